// Types and small device helpers that the MFMA kernels share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace lora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Read-only global memory.
template <typename T> using gptr = const __attribute__((address_space(1))) T *;
template <typename T> __device__ __forceinline__ gptr<T> as_global(const void *p) { return (gptr<T>)(p); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint32_t f32_to_bf16(float f)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); // nearest even, NaN stays a (quiet) NaN
}
// two fp32 -> packed bf16 (lo in bits 15:0), one conversion instruction
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

// s_waitcnt immediates (vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8; the
// others at their largest: no wait), written through the builtin, so that the
// compiler's own wait insertion knows about them.
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); } // vmcnt(n)
constexpr int wait_vm_lds0(int n) { return wait_vm(n) & ~(15 << 8); }                       // vmcnt(n) and lgkmcnt(0)
constexpr int kWaitLds0 = 15 | (3 << 14) | (7 << 4);                                        // lgkmcnt(0) alone

// 16 bytes per lane from global memory to LDS at m0 + 16 lane.  The compiler does
// not see this write to LDS; the kernel waits for it with an explicit vmcnt before
// the barrier that publishes the data.  m0 is a reserved register (never allocated
// by the compiler) and no other code in these kernels reads it.  A load to LDS needs a
// wait state behind a scalar write of m0, which the compiler does not add inside an asm
// statement: hence the s_nop, here and wherever else m0 is written.
__device__ __forceinline__ void dma16(const void *g, uint32_t lds_byte)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds_byte) : "memory");
}
// What direct loads take for places outside.
__device__ const uint32_t g_zeros[4] = {0, 0, 0, 0};

// Lane i of every 16 lanes gives the address of 4 elements of row i / 4, at
// column group i % 4, and receives column i of the 4 rows.
__device__ __forceinline__ u32x2 read_tr(const char *lds)
{
    typedef __attribute__((address_space(3))) s16x4 lds4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(lds)));
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

} // namespace
} // namespace lora
