// Quantization to E4M3 on the device: scales, codes, and the rows form, which other launches take
// along.  What is computed, and why so, stands in e4m3.hip.
#pragma once

#include "device.h"
#include "internal.h"

namespace lora {
namespace {

constexpr int kScaleGroup = LORA_SCALE_BLOCK;
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

// 16 rows (from 16 bx) x U groups (from U by) by 256 threads; a workgroup of NW times as many
// takes the groups from U NW by.
template <int DT, bool E8, int U, int NW = 1>
__device__ __forceinline__ void quantize_rows(const QuantArgs &a, unsigned bx, unsigned by)
{
    __shared__ uint32_t sc_all[NW][U][16];
    const int part = threadIdx.x >> 8, tid = threadIdx.x & 255, l = tid & 15, i = tid >> 4;
    auto &sc_lds = sc_all[part];
    by = by * NW + part;
    const int64_t p = int64_t(bx) * 16 + i;
    const int groups = (a.cols + kScaleGroup - 1) / kScaleGroup;
    int64_t row = p < a.rows ? p : -1;
    if (a.perm && row >= 0) row = a.perm[row];
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (int(by) * U + u) * kScaleGroup + 8 * l;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[u][k] = 0.f;
        if (row >= 0 && c < a.cols) load8<DT>(a.x, row * a.ldx, c, a.cols, f[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = (int(by) * U + u) * kScaleGroup + 8 * l;
        uint32_t top = top8(f[u], 0);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = max(top, uint32_t(__shfl_xor(int(top), d)));
        const Scale sc = scale_of<E8>(top);
        if (p < a.rows && c < a.qcols) store8(a.codes + p * a.ldq, c, a.qcols, codes8<E8>(f[u], sc));
        if (l == 0) sc_lds[u][i] = sc.stored;
    }
    __syncthreads();
    const int u = i, g = int(by) * U + u;
    const int64_t q = int64_t(bx) * 16 + l;
    if (u < U && g < groups && q < a.rows) {
        if constexpr (E8) static_cast<uint8_t *>(a.scales)[g * a.lds + q] = uint8_t(sc_lds[u][l]);
        else static_cast<uint32_t *>(a.scales)[g * a.lds + q] = sc_lds[u][l];
    }
}

// The arguments of a call in rows.
inline QuantArgs quant_args(const QuantCall &q)
{
    QuantArgs a{};
    a.x = q.x;
    a.ldx = q.ldx;
    a.rows = q.rows;
    a.cols = q.cols;
    a.perm = q.perm;
    a.codes = static_cast<uint8_t *>(q.codes);
    a.ldq = q.ldq;
    a.qcols = q.pad ? (q.cols + kScaleGroup - 1) / kScaleGroup * kScaleGroup : q.cols;
    a.scales = q.scales;
    a.lds = q.lds;
    return a;
}
// Groups of a workgroup of the rows form: four where that still fills the chip twice over.
inline int quant_groups(const QuantArgs &a)
{
    const int64_t rt = (int64_t(a.rows) + 15) / 16, qg = (a.qcols + kScaleGroup - 1) / kScaleGroup;
    return rt * qg >= 4 * 512 ? 4 : 1;
}

// Rows that another launch of bf16 rows quantizes along: its workgroups from `first` on, each of 256 NW threads.
struct QuantAlong {
    QuantArgs q;
    unsigned first, gx; // first workgroup, workgroups along the rows
    int groups;
    bool e8;
};
template <int NW> __device__ __forceinline__ void quantize_along(const QuantAlong &along, unsigned workgroup)
{
    const unsigned b = workgroup - along.first, bx = b % along.gx, by = b / along.gx;
    if (along.groups == 4) {
        if (along.e8) quantize_rows<LORA_BF16, true, 4, NW>(along.q, bx, by);
        else quantize_rows<LORA_BF16, false, 4, NW>(along.q, bx, by);
    } else {
        if (along.e8) quantize_rows<LORA_BF16, true, 1, NW>(along.q, bx, by);
        else quantize_rows<LORA_BF16, false, 1, NW>(along.q, bx, by);
    }
}
// q behind `first` workgroups of the launch; *grid: workgroups of both.
inline QuantAlong quant_along(const QuantCall &q, int64_t first, int nw, int64_t *grid)
{
    QuantAlong along{};
    along.q = quant_args(q);
    along.groups = quant_groups(along.q);
    along.e8 = q.scale_type == LORA_SCALE_E8M0;
    along.gx = unsigned((int64_t(q.rows) + 15) / 16);
    along.first = unsigned(first);
    const int64_t each = int64_t(along.groups) * nw, qg = along.q.qcols / kScaleGroup;
    *grid = first + (qg + each - 1) / each * along.gx;
    return along;
}

} // namespace
} // namespace lora
