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
// block in registers.  64 x 4096 bf16 in 3.2 us (a launch's latency), 12250 x 4105 fp32 in
// 128 x 128 blocks in 60 (4.2 TB/s; a large copy moves 5.1).
#include "e4m3.h"

namespace lora {
namespace {

constexpr int kG = LORA_SCALE_BLOCK;

template <int DT, bool E8, int U> __global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a)
{
    quantize_rows<DT, E8, U>(a, blockIdx.x, blockIdx.y);
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
    if (quant_groups(a) == 4)
        launch_kernel(quantize_rows_kernel<DT, E8, 4>, dim3(unsigned(rt), unsigned((qg + 3) / 4)), dim3(256), 0, s, a);
    else
        launch_kernel(quantize_rows_kernel<DT, E8, 1>, dim3(unsigned(rt), unsigned(qg)), dim3(256), 0, s, a);
}

} // namespace

int launch_quantize(hipStream_t s, const QuantCall &q)
{
    const QuantArgs a = quant_args(q);
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
