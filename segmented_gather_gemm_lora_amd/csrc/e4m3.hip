// Quantization to OCP E4M3 with a scale for each block, on gfx950.
//
// A block is 128 adjacent elements of a row (activations, gradients) or 128 x 128
// elements (weights); the last ones of a matrix are ragged.  With amax the largest
// magnitude of a block:
//     s = max(fp32(amax / 448), 2^-126), or
//     s = 2^e, the least e in [-126, 127] with amax <= 448 2^e   (E8M0: the byte e + 127)
//     code = the E4M3 value nearest to x / s, ties to even, from the exact quotient
// A block that holds an infinity or a NaN gets a NaN scale and codes of 0.
//
// The quotient is rounded once.  bf16 values against a scale that comes from one of
// them meet the middle of two codes often (small whole ratios), and a quotient rounded to
// fp32 first falls on it when it was next to it.  So x and s are scaled by a power of two
// (s into [1, 2), no subnormals), q = x / s is formed to within a bit, its exact remainder
// x - q s (one fma) says on which side x / s lies, and a q with an even last bit is moved
// to its odd neighbour on that side ("round to odd", Boldo and Melquiond): the
// hardware's rounding of that to 4 bits is the rounding of the exact quotient.
//
// Memory-bound: x is read once, codes written once.  Rows form: 16 lanes hold a group
// (8 elements each: 16 bytes of bf16), a workgroup 16 rows x U groups, so that the scales
// of 16 rows, which lie side by side, leave as 64 bytes.  Block form: a workgroup holds a
// block in registers.
#include "device.h"
#include "internal.h"

namespace lora {
namespace {

constexpr int kG = 128;
typedef u32x4 u32x4_2 __attribute__((aligned(2)));
typedef u32x4 u32x4_4 __attribute__((aligned(4)));
typedef u32x2 u32x2_1 __attribute__((aligned(1)));

struct QuantArgs {
    const void *x;
    int64_t ldx;
    int32_t rows, cols; // of the result; columns of x
    const int32_t *perm; // row p of the result is row perm[p] of x (-1: zeros); null: row p
    uint8_t *codes;
    int64_t ldq;
    int32_t qcols; // columns written (cols, or more: zeros)
    void *scales;
    int64_t lds;
};

// Eight elements from column c of a row; past the row's end zeros.
template <int DT> __device__ __forceinline__ void load8(const void *x, int64_t row, int c, int cols, float (&f)[8])
{
    if constexpr (DT == LORA_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(x) + row + c;
        if (c + 8 <= cols) {
            const u32x4 u = *reinterpret_cast<const u32x4_2 *>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? bf16_to_f32(p[i]) : 0.f;
        }
    } else {
        const float *p = static_cast<const float *>(x) + row + c;
        if (c + 8 <= cols) {
            const u32x4 u = *reinterpret_cast<const u32x4_4 *>(p), w = *reinterpret_cast<const u32x4_4 *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = __uint_as_float(u[i]);
                f[4 + i] = __uint_as_float(w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? p[i] : 0.f;
        }
    }
}

// Magnitudes as whole numbers: they order as the values do, and NaN is above infinity.
__device__ __forceinline__ uint32_t top8(const float (&f)[8], uint32_t top)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return top;
}

// The scale of a block: as it is stored, and what the quotients take.
struct Scale {
    uint32_t stored; // fp32 bits, or the E8M0 byte
    float s, inv;    // s in [1, 2) and 1 / s (E8M0: 1)
    int shift;       // x and s are multiplied by 2^shift first
    bool bad;        // an infinity or a NaN
};
template <bool E8> __device__ __forceinline__ Scale scale_of(uint32_t top)
{
    Scale r;
    r.bad = top >= 0x7F800000u;
    const float amax = __uint_as_float(top);
    if constexpr (E8) {
        int e;
        const float m = frexpf(amax, &e); // amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        e = amax > 0.f ? e - 9 + (m > 0.875f) : -126;
        e = min(max(e, -126), 127);
        r.stored = r.bad ? 255u : uint32_t(e + 127);
        r.s = r.inv = 1.f;
        r.shift = -e;
    } else {
        const float s = fmaxf(amax / 448.f, 0x1p-126f);
        const int e = int(__float_as_uint(s) >> 23) - 127;
        r.stored = r.bad ? 0x7FC00000u : __float_as_uint(s);
        r.shift = -e;
        r.s = ldexpf(s, -e);
        r.inv = 1.f / r.s;
    }
    return r;
}

// x / s, rounded to odd (E8M0: exact).
template <bool E8> __device__ __forceinline__ float quotient(float x, const Scale &sc)
{
    const float v = ldexpf(x, sc.shift);
    if constexpr (E8) return v;
    float q = v * sc.inv;
    q = fmaf(fmaf(-q, sc.s, v), sc.inv, q);
    const float rest = fmaf(-q, sc.s, v); // exact: q is within a bit of v / s
    const uint32_t b = __float_as_uint(q);
    const int away = (__float_as_uint(rest) ^ b) >> 31 ? -1 : 1; // v / s is further from 0 than q
    return rest != 0.f && !(b & 1) ? __uint_as_float(b + away) : q;
}

template <bool E8> __device__ __forceinline__ u32x2 codes8(const float (&f)[8], const Scale &sc)
{
    u32x2 out{};
    if (sc.bad) return out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(quotient<E8>(f[4 * h + i], sc), -448.f), 448.f);
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
        out[h] = uint32_t(w);
    }
    return out;
}

__device__ __forceinline__ void store8(uint8_t *p, int c, int cols, u32x2 w)
{
    if (c + 8 <= cols) {
        *reinterpret_cast<u32x2_1 *>(p + c) = w;
        return;
    }
    for (int i = 0; i < 8; ++i)
        if (c + i < cols) p[c + i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
}

template <int DT, bool E8, int U> __global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a)
{
    __shared__ uint32_t sc_lds[U][16];
    const int tid = threadIdx.x, l = tid & 15, i = tid >> 4;
    const int64_t p = int64_t(blockIdx.x) * 16 + i;
    const int groups = (a.cols + kG - 1) / kG;
    int64_t row = p < a.rows ? p : -1;
    if (a.perm && row >= 0) row = a.perm[row];
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (int(blockIdx.y) * U + u) * kG + 8 * l;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[u][k] = 0.f;
        if (row >= 0 && c < a.cols) load8<DT>(a.x, row * a.ldx, c, a.cols, f[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (int(blockIdx.y) * U + u) * kG + 8 * l;
        uint32_t top = top8(f[u], 0);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = max(top, uint32_t(__shfl_xor(int(top), d)));
        const Scale sc = scale_of<E8>(top);
        if (p < a.rows && c < a.qcols) store8(a.codes + p * a.ldq, c, a.qcols, codes8<E8>(f[u], sc));
        if (l == 0) sc_lds[u][i] = sc.stored;
    }
    __syncthreads();
    const int u = tid >> 4, g = int(blockIdx.y) * U + u;
    const int64_t q = int64_t(blockIdx.x) * 16 + l;
    if (u < U && g < groups && q < a.rows) {
        if constexpr (E8) static_cast<uint8_t *>(a.scales)[g * a.lds + q] = uint8_t(sc_lds[u][l]);
        else static_cast<uint32_t *>(a.scales)[g * a.lds + q] = sc_lds[u][l];
    }
}

template <int DT, bool E8> __global__ __launch_bounds__(256) void quantize_blocks_kernel(QuantArgs a)
{
    __shared__ uint32_t tops[4];
    const int tid = threadIdx.x, l = tid & 15, i = tid >> 4;
    const int r0 = int(blockIdx.x) * kG, c = int(blockIdx.y) * kG + 8 * l;
    float f[8][8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = r0 + i + 16 * j;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[j][k] = 0.f;
        if (r < a.rows && c < a.cols) load8<DT>(a.x, r * a.ldx, c, a.cols, f[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = top8(f[j], top);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, uint32_t(__shfl_xor(int(top), d)));
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const Scale sc = scale_of<E8>(top);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t r = r0 + i + 16 * j;
        if (r < a.rows && c < a.cols) store8(a.codes + r * a.ldq, c, a.cols, codes8<E8>(f[j], sc));
    }
    if (tid == 0) {
        const int64_t at = int64_t(blockIdx.x) * a.lds + blockIdx.y;
        if constexpr (E8) static_cast<uint8_t *>(a.scales)[at] = uint8_t(sc.stored);
        else static_cast<uint32_t *>(a.scales)[at] = sc.stored;
    }
}

template <int DT, bool E8> void go(hipStream_t s, const QuantArgs &a, int block_rows)
{
    const int qg = (a.qcols + kG - 1) / kG;
    if (block_rows == kG) {
        launch_kernel(quantize_blocks_kernel<DT, E8>, dim3(unsigned((a.rows + kG - 1) / kG), unsigned(qg)), dim3(256), 0, s,
                      a);
        return;
    }
    const int64_t rt = (int64_t(a.rows) + 15) / 16;
    // four groups a workgroup where that still fills the chip twice over
    if (rt * qg >= 4 * 512)
        launch_kernel(quantize_rows_kernel<DT, E8, 4>, dim3(unsigned(rt), unsigned((qg + 3) / 4)), dim3(256), 0, s, a);
    else
        launch_kernel(quantize_rows_kernel<DT, E8, 1>, dim3(unsigned(rt), unsigned(qg)), dim3(256), 0, s, a);
}

} // namespace

int launch_quantize(hipStream_t s, const QuantCall &q)
{
    QuantArgs a{};
    a.x = q.x;
    a.ldx = q.ldx;
    a.rows = q.rows;
    a.cols = q.cols;
    a.perm = q.perm;
    a.codes = static_cast<uint8_t *>(q.codes);
    a.ldq = q.ldq;
    a.qcols = q.pad ? (q.cols + kG - 1) / kG * kG : q.cols;
    a.scales = q.scales;
    a.lds = q.lds;
    if (q.rows == 0) return LORA_OK;
    const bool e8 = q.scale_type == LORA_SCALE_E8M0;
    if (q.dtype == LORA_BF16) {
        if (e8) go<LORA_BF16, true>(s, a, q.block_rows);
        else go<LORA_BF16, false>(s, a, q.block_rows);
    } else {
        if (e8) go<LORA_F32, true>(s, a, q.block_rows);
        else go<LORA_F32, false>(s, a, q.block_rows);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(LORA_ERR_HIP, "quantize launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

} // namespace lora
