// Products with an E4M3 base that has a scale for each block of 128, on gfx950:
//
//     y[t, n] = sum_b sx[b, t] sw[n / 128, b] sum_{k in block b} qx[t, k] qw[n, k]
//
// with qx, sx the codes and scales of 1 x 128 groups of the rows and qw, sw those of 128 x
// 128 blocks of W [d_out, d_in].  lora_linear_e4m3_block is that product;
// lora_fused_linear_e4m3_block quantizes x itself and adds every token's correction
// scale_s (x A_s) B_s from the unquantized x, as further steps of the same accumulators.
//
// One workgroup computes 16 TN WN columns x 16 TM WM rows with WN x WM waves on
// v_mfma_f32_16x16x128_f8f6f4, whose 128 is a block: one instruction is the inner sum of 16
// columns and 16 rows.  E8M0 scales: the instruction takes the two scale bytes itself and
// accumulates.  fp32 scales: it takes the power of two of W's, starts from 0, and its result enters the fp32
// accumulators with one fma a value (a lane's four values are one row's, so the rest of W's scale and the row's
// scale are one factor in a register a row tile).  MFMA rows are columns of W, MFMA columns are rows of x.
//
// A stage is a block: 128 bytes of each row of W and of x, and the rows' scales, brought
// to LDS by direct loads.  16-byte unit u of row r lies in slot u ^ (r % 8), so that 8
// rows at one unit cover all banks.  Of the 128 a lane takes units g and g + 4 (g = lane /
// 16) on both sides: within a block the order of k does not matter.  The rows of W are
// placed so that a lane ends with 4 TN adjacent columns of a row.
//
// Precision.  The 8-bit instructions add the products of 8 adjacent k at a fixed point,
// 2^-13 below the power of two of the largest, and the eights in fp32 (measured with exact
// powers of two: 2^16 + 2^3 is kept, 2^16 + 2^2 gives 2^16).  On hidden states that is 4e-5 of a
// result, 50 times below the rounding to bf16, so bf16 results and dx take them.  fp32 results
// do not: their codes are widened to bf16 (exactly: 4 significant bits) and multiplied on
// v_mfma_f32_16x16x32_bf16, whose sums are fp32's, at half the rate and a conversion for
// each operand.
//
// The rows' gradient, dx = (sdy qdy) (sw qw), sums over d_out, along which W is not
// contiguous: a stage is then 128 rows of 16 TN WN bytes of W, read with
// ds_read_b64_tr_b8, which hands a lane one column of 8 rows; unit u of row r lies in
// slot u ^ (r % 8), so that those 8 rows cover all banks.  It writes fp32 sums (few tiles are
// split along d_out), which the gradient's last launch adds, with u A.
//
// What bounds it: a stage's loads.  4096 rows, 4096 -> 14336, E8M0 scales: 236 us (2.0
// PFLOP/s), the matrix units busy 44% of the cycles, no LDS conflicts; 64 KB a stage come
// from the L2 while the stage before is multiplied, and LDS holds two.  fp32 scales: 265
// us, with fresh results and four fmas for each matrix instruction.
#include "device.h"
#include "internal.h"

#include <algorithm>

namespace lora {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
constexpr int kG = 128;

// Read-only memory at a wave-uniform address: scalar loads.
template <typename T> using cptr = const __attribute__((address_space(4))) T *;

struct BlockArgs {
    const uint8_t *x; // codes [T][ldx]
    int64_t ldx;
    const void *sx; // [groups][lds]
    int64_t lds;
    const uint8_t *W; // codes [n][k]
    const void *sw;   // [n / 128][groups]
    int k, n, T;
    const int32_t *perm; // output row of each row (-1: none); null: the row itself
    void *y;
    int64_t ldy;
    int vec_y; // whole aligned 16-byte pieces of y
    int tiles_m, tiles_n;
    int whole; // tiles that are not halved
    // the correction
    const int32_t *segidx;
    const lora_seg_desc *seg;
    int nseg; // records (of a device plan: room for them)
    int Tp;
    const int32_t *tp_dev;
    const uint16_t *vh;
    int64_t ldh;
    const float *v; // up to 64 rows: the shrink's slices of v, and their layout
    int64_t ldw, sl_stride;
    int nsl;
    int per; // gradient: stages of a split; split i writes rows i T .. of y
};

template <int TN_, int TM_, int WN_, int WM_, int STAGES> struct Shape {
    static constexpr int TN = TN_, TM = TM_, WN = WN_, WM = WM_, kStages = STAGES;
    static constexpr int kBN = 16 * TN * WN, kBM = 16 * TM * WM, kWaves = WN * WM, kThreads = 64 * kWaves;
    static constexpr int kWBytes = kBN * kG, kXBytes = kBM * kG;
    static constexpr int kSBytes = kBM <= 64 ? 256 : 4 * kBM; // the rows' scales
    static constexpr int kStageBytes = kWBytes + kXBytes + kSBytes;
    static constexpr int kWavesPerSimd = kWaves * (160 * 1024 / (kStages * kStageBytes)) / 4;
    static constexpr int kWDma = kWBytes / 1024 / kWaves, kXDma = kXBytes / 1024 / kWaves;
    static constexpr int kDma = kWDma + kXDma + 1; // direct loads of a wave in a stage
    static_assert(kWDma * kWaves * 1024 == kWBytes && kXDma * kWaves * 1024 == kXBytes, "stage split");
    static_assert(kStages * kStageBytes <= 160 * 1024, "LDS budget");
    static_assert(kDma * (kStages - 2) <= 63, "vmcnt range");
    static_assert(16 * TN <= kG && kG % (16 * TN) == 0, "a wave's columns lie in one block");
    static constexpr bool kHalved = TN == 8; // its last tiles may be halves
    typedef Shape<TN / 2, TM, WN, WM, STAGES> Half;
};

__device__ __forceinline__ void dma4(const void *g, uint32_t lds_byte)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(g), "s"(lds_byte) : "memory");
}

// A byte per lane, which becomes a word in LDS.
__device__ __forceinline__ void dma1(const void *g, uint32_t lds_byte)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, off" ::"v"(g), "s"(lds_byte) : "memory");
}

// dma16 from a wave-uniform base plus a 32-bit per-lane byte offset.
__device__ __forceinline__ void dma16s(const void *base, uint32_t off, uint32_t lds_byte)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds_byte) : "memory");
}

// Column of a wave's tile t that MFMA row m stands for: lane group g ends with columns
// 4 TN g + 4 t + q.
template <int TN> __device__ __forceinline__ int wave_col(int m, int t) { return (m >> 2) * (4 * TN) + 4 * t + (m & 3); }

// Ranks jj .. jj + 7 of a row of B whose rank r is any: the 16 bytes from element `at` of the matrix (its
// elements go on in the next row), or at the matrix's end those before it.  n r >= 8 elements.
// Ranks one by one: 201 rows of ranks 5, 24 and 100, 4224 -> 4880, 49 us, 29 so; 64 rows of 32 such adapters
// 31 and 25.
typedef u32x4 u32x4_half __attribute__((aligned(2)));
__device__ __forceinline__ u32x4 eight_of(gptr<uint16_t> B, int64_t at, int64_t elements)
{
    return *(gptr<u32x4_half>)(B + (at < elements - 8 ? at : elements - 8));
}
// What eight_of() has brought, moved to its place, and zeros for what are not the row's ranks (`left` of them).
__device__ __forceinline__ u32x4 own_eight(u32x4 u, int64_t at, int64_t elements, int left)
{
    const int late = at > elements - 8 ? int(at - (elements - 8)) : 0; // only in the matrix's last rows
    if (__any(late > 0)) {
        uint64_t lo = uint64_t(u[0]) | uint64_t(u[1]) << 32, hi = uint64_t(u[2]) | uint64_t(u[3]) << 32;
        const int by = 16 * (late & 3);
        if (late & 4) lo = hi, hi = 0;
        if (by) lo = lo >> by | hi << (64 - by), hi >>= by;
        if (late > 7) lo = 0;
        u = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] &= (2 * e < left ? 0xFFFFu : 0u) | (2 * e + 1 < left ? 0xFFFF0000u : 0u);
    return u;
}
// The same one by one, of a matrix of fewer than 8 elements.
__device__ __forceinline__ u32x4 few_ranks(gptr<uint16_t> row, int jj, int r)
{
    u32x4 u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = jj + 2 * e;
        const uint32_t lo = row[j < r ? j : 0], hi = row[j + 1 < r ? j + 1 : 0];
        u[e] = (j < r ? lo : 0) | (j + 1 < r ? hi << 16 : 0);
    }
    return u;
}

// The correction of the segments that meet a wave's rows (at most one a row), on bf16
// MFMA: a step is 16 ranks of one segment, A = B_s rows (lane groups 0, 2: the first 8 ranks,
// 1, 3: the others), B = scale_s v in two halves (groups 0, 1: hi, 2, 3: lo).  Only the row tiles that the
// segment meets are multiplied, and of those only its own rows take the result: what is
// not finite in one adapter stays with its rows.  Ranks are the outer loop: the rows' v of 16
// ranks is then loaded once for all segments.
//
// kRing (every rank is a multiple of 8): B_s comes by direct loads through a ring of
// steps in LDS that is the wave's own, several steps ahead: short segments are chains of
// loads that depend on nothing but their segment, and one step at a time took over 2 us.
template <int TN, int TM, int SR, bool kRing, int kBytes>
__device__ __forceinline__ void correction(const BlockArgs &a, int Tp, int pw0, int cw0, int lane, char *mine, uint32_t mine_lds,
                                           floatx4 (&acc)[TN][TM])
{
    constexpr int kSlot = 512 * TN, kLoads = TN / 2, kDepth = kBytes / kSlot < 4 ? kBytes / kSlot : 4;
    static_assert(kDepth >= 2 && 16 * TM <= 64, "ring, segments of a wave");
    const int m = lane & 15, g = lane >> 4;
    // lane l: the segment of row l % 16 of the wave's row tile l / 16, if that is the first of the
    // wave's rows in it
    const int mt = lane >> 4 < TM ? lane >> 4 : TM - 1, mp = pw0 + SR * mt + m;
    const lora_seg_desc *d = a.seg + as_global<int32_t>(a.segidx)[mp < Tp ? mp : Tp - 1];
    const uint64_t dB = d->B;
    const uint32_t Blo = uint32_t(dB), Bhi = uint32_t(dB >> 32);
    const int start = d->start, len = d->len, drank = d->rank;
    const bool first = mp == start || (m == 0 && (mt == 0 || start >= mp - SR + 16));
    const int rank = first && mp < Tp && lane < 16 * TM ? drank : 0;
    // Here, and below, what the compiler loaded has landed before the ring's loads, which it does not
    // count: else it would wait for all of them in every step.
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    auto lane_of = [](int v, int l) { return __builtin_amdgcn_readlane(v, l); };
    const int c00 = cw0 < a.n ? cw0 : a.n - 1; // columns are counted from here: B may span more than 4 GiB
    auto whole_of = [&](int l) {
        return reinterpret_cast<const uint16_t *>(uint64_t(uint32_t(lane_of(int(Blo), l))) | uint64_t(uint32_t(lane_of(int(Bhi), l))) << 32);
    };
    auto base_of = [&](int l, int r) { return whole_of(l) + int64_t(c00) * r; };
    auto next = [&](int &q, uint64_t &left) { // the next step (16 ranks q, segment), or -1
        while (left == 0) {
            left = __ballot(rank > 16 * ++q);
            if (left == 0) return -1;
        }
        const int l = __builtin_ctzll(left);
        left &= left - 1;
        return l;
    };
    int pq = -1, issued = 0, done = 0; // steps whose loads are out
    uint64_t pleft = 0;
    bool more = true;
    int col[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) { // LDS row 32 k + lane / 2 of a step, half lane % 2
        const int rho = 32 * k + (lane >> 1), c = cw0 + wave_col<TN>(rho & 15, rho >> 4);
        col[k] = (c < a.n ? c : a.n - 1) - c00;
    }
    auto issue = [&] {
        const int l = next(pq, pleft);
        if (l < 0) {
            more = false;
            return;
        }
        const int r = lane_of(rank, l), half = 16 * pq + 8 < r ? lane & 1 : 0;
        const void *B = base_of(l, r);
        const uint32_t to = mine_lds + uint32_t(issued % kDepth) * kSlot;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) dma16s(B, uint32_t(col[k]) * uint32_t(2 * r) + uint32_t(32 * pq + 16 * half), to + 1024 * k);
        ++issued;
    };
    if constexpr (kRing)
        for (int i = 0; i < kDepth && more; ++i) issue();
    int q = -1, vq = -1;
    uint64_t left = 0;
    u32x4 v[TM];
    for (;;) {
        const int l = next(q, left);
        if (l < 0) break;
        if (q != vq) {
            vq = q;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int p = pw0 + SR * i + m;
                v[i] = *(gptr<u32x4>)(as_global<uint16_t>(a.vh) + int64_t(p < Tp ? p : Tp - 1) * a.ldh + 32 * q + 8 * g);
            }
            if constexpr (kRing) __builtin_amdgcn_s_waitcnt(wait_vm(0));
        }
        const int r = lane_of(rank, l), p0 = lane_of(start, l), p1 = p0 + lane_of(len, l);
        const int jj = 16 * q + 8 * (g & 1);
        bf16x8 b[TN];
        if constexpr (kRing) {
            // this step's loads have landed: with a full ring all but those of the later ones
            if (issued - done == kDepth) __builtin_amdgcn_s_waitcnt(wait_vm(kLoads * (kDepth - 1)));
            else __builtin_amdgcn_s_waitcnt(wait_vm(0));
            const char *at = mine + (done % kDepth) * kSlot + m * 32 + (g & 1) * 16;
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                u32x4 u = *reinterpret_cast<const u32x4 *>(at + 512 * t);
                if (jj >= r) u = u32x4{};
                b[t] = __builtin_bit_cast(bf16x8, u);
            }
            ++done;
            __builtin_amdgcn_s_waitcnt(kWaitLds0); // read before the place is filled again
            if (more) issue();
        } else {
            const gptr<uint16_t> B = as_global<uint16_t>(whole_of(l));
            const int64_t elements = int64_t(a.n) * r;
            auto at = [&](int t) {
                const int c = cw0 + wave_col<TN>(m, t);
                return int64_t(c < a.n ? c : a.n - 1) * r;
            };
            u32x4 raw[TN];
            if (elements >= 8) {
#pragma unroll
                for (int t = 0; t < TN; ++t) raw[t] = eight_of(B, at(t) + jj, elements);
#pragma unroll
                for (int t = 0; t < TN; ++t) raw[t] = own_eight(raw[t], at(t) + jj, elements, r - jj);
            } else {
#pragma unroll
                for (int t = 0; t < TN; ++t) raw[t] = few_ranks(B + at(t), jj, r);
            }
#pragma unroll
            for (int t = 0; t < TN; ++t) b[t] = __builtin_bit_cast(bf16x8, raw[t]);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int t0 = pw0 + SR * i;
            if (p0 >= t0 + 16 || p1 <= t0) continue; // wave-uniform
            const bool in = t0 + m >= p0 && t0 + m < p1;
            const bf16x8 vi = __builtin_bit_cast(bf16x8, v[i]);
            constexpr int kAtOnce = TN < 4 ? TN : 4; // so many results wait for their choice together
#pragma unroll
            for (int t = 0; t < TN; t += kAtOnce) {
                floatx4 y[kAtOnce];
#pragma unroll
                for (int h = 0; h < kAtOnce; ++h) y[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[t + h], vi, acc[t + h][i], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int h = 0; h < kAtOnce; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t + h][i][e] = in ? y[h][e] : acc[t + h][i][e];
            }
        }
    }
}

// Row p's values of columns c0 .. c0 + 4 TN - 1.
template <int TN, bool F32OUT>
__device__ __forceinline__ void store_row(const BlockArgs &a, int64_t row, int c0, const float (&v)[4 * TN])
{
    constexpr int kPiece = F32OUT ? 4 : 8;
#pragma unroll
    for (int h = 0; h < 4 * TN / kPiece; ++h) {
        const int c = c0 + h * kPiece;
        const float *f = v + h * kPiece;
        if (a.vec_y && c + kPiece <= a.n) {
            u32x4 w;
            if constexpr (F32OUT) w = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
            else w = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
            *reinterpret_cast<u32x4 *>(static_cast<char *>(a.y) + (row * a.ldy + c) * (F32OUT ? 4 : 2)) = w;
        } else {
#pragma unroll
            for (int q = 0; q < kPiece; ++q)
                if (c + q < a.n) {
                    if constexpr (F32OUT) static_cast<float *>(a.y)[row * a.ldy + c + q] = f[q];
                    else static_cast<uint16_t *>(a.y)[row * a.ldy + c + q] = uint16_t(f32_to_bf16(f[q]));
                }
        }
    }
}

// 32 codes as four operands of 8 bf16, times a power of two, exactly (2^-100 to 2^100 of 4 significant bits).
struct Wide {
    bf16x8 v[4];
};
__device__ __forceinline__ Wide widen(const i32x8 &c, float power)
{
    Wide w;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        u32x4 u;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            u[2 * q] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(uint32_t(c[2 * h + q]), power, false));
            u[2 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(uint32_t(c[2 * h + q]), power, true));
        }
        w.v[h] = __builtin_bit_cast(bf16x8, u);
    }
    return w;
}

// W's scale as the byte of a power of two and a factor: value = f 2^(e - 127).  The product of two scales may
// leave fp32's range where its product with a block's sum does not (or the sum is 0), so it is never formed: 2^(e - 127)
// goes into the sum, through the matrix instruction or the widened codes, and f with the row's scale into the
// accumulators.  e is held in 2^-100 .. 2^100, where no sum of a block (2^-18 to 2^25) leaves the range; f is in [1, 2)
// there.  So the factor f sx overflows for scales whose product is 2^228 and more alone, and loses bits
// where sx is subnormal.
struct WScale {
    int e;
    float f;
};
__device__ __forceinline__ float e8m0(int e)
{
    return e == 255 ? __uint_as_float(0x7FC00000u) : e ? __uint_as_float(uint32_t(e) << 23) : 0x1p-127f;
}
template <bool E8> __device__ __forceinline__ WScale wscale_of(uint32_t word)
{
    const int e = min(max(E8 ? int(word) : int(word >> 23 & 255), 27), 227);
    return WScale{e, ldexpf(E8 ? e8m0(int(word)) : __uint_as_float(word), 127 - e)};
}

// One block with fp32 sums: acc += f (power W x) on bf16 MFMA.
template <int TN, int TM, class WF>
__device__ __forceinline__ void exact_block(const i32x8 (&xf)[TM], float power, const float (&f)[TM], floatx4 (&acc)[TN][TM], const WF &wfrag)
{
    Wide x[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) x[i] = widen(xf[i], 1.f);
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        const Wide w = widen(wfrag(t), power);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            floatx4 p{};
#pragma unroll
            for (int h = 0; h < 4; ++h) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[h], x[i].v[h], p, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[t][i][q] = fmaf(p[q], f[i], acc[t][i][q]);
        }
    }
}

// What a kernel computes: the product into bf16 or fp32, the fused layer, or the rows'
// gradient.
enum Form { kBf16, kF32, kFused, kFusedAnyRank, kGradient };
constexpr bool is_fused(Form f) { return f == kFused || f == kFusedAnyRank; }
// Whether the matrix instruction takes both scales whole.
constexpr bool own_scales(bool e8, Form f) { return e8 && f != kF32; }

// The scales of W that a wave meets in 64 blocks, one a lane: a byte, and where the instruction does not take
// it all a factor.
struct WScales {
    uint32_t e;
    float f;
};
template <bool E8, Form F> __device__ __forceinline__ WScales wscales_at(const void *sw, int64_t at)
{
    if constexpr (own_scales(E8, F)) return WScales{as_global<uint8_t>(sw)[at], 1.f};
    const WScale w = wscale_of<E8>(E8 ? as_global<uint8_t>(sw)[at] : as_global<uint32_t>(sw)[at]);
    return WScales{uint32_t(w.e), w.f};
}
__device__ __forceinline__ WScale wscale_from(const WScales &all, int l)
{
    return WScale{__builtin_amdgcn_readlane(int(all.e), l),
                  __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(all.f)), l)))};
}
// A row's factor: what is left of W's scale, and its own (a byte or fp32 bits).
template <bool E8> __device__ __forceinline__ float factor(const WScale &w, uint32_t sx) { return w.f * (E8 ? e8m0(int(sx)) : __uint_as_float(sx)); }

// A workgroup's tile: its place, the loads of its stages and the fragments in them.
// k is the summed axis and n the columns of W [n][k], or of W [k][n] (kGradient).
template <class S, bool E8, Form F> struct Tile {
    static constexpr int TN = S::TN, TM = S::TM;
    static constexpr bool WT = F == kGradient;
    // Direct loads: load i of a part fills 64 units of 16 bytes, a lane the one in row
    // (64 i + lane) / units-of-a-row, slot (64 i + lane) % units-of-a-row, which holds unit
    // slot ^ (row % 8).
    static constexpr int kWUnits = WT ? S::kBN / 16 : 8;
    // Row tile i of a wave is kStrips * i below its first: neighbouring rows, which may be many short
    // segments, are every wave's (2304 rows, the 288 last of 70 adapters of ranks 8 to 64: 121 us with
    // a wave's tiles side by side, 90 so).
    static constexpr int kStrips = 16 * S::WM;
    const BlockArgs &a;
    char *lds;
    uint32_t lds0;
    int lane, wave, m, g, wn, wm;
    int m0, n0, split, blocks, k0, k1, pw0, cw0;
    int unit, spart;
    uint32_t woff[S::kWDma], xoff[S::kXDma];
    const char *sxp;
    int64_t sstep, sw0, sw1;
    int u0, u1;

    // tile: its number; half: columns it starts behind its first
    __device__ __forceinline__ Tile(const BlockArgs &args, char *l, int tile, int cols, int half) : a(args), lds(l)
    {
        const int tid = threadIdx.x;
        lane = tid & 63;
        wave = uniform(tid >> 6);
        m = lane & 15;
        g = lane >> 4;
        wn = wave / S::WM;
        wm = wave % S::WM;
        lds0 = uint32_t(uintptr_t((__attribute__((address_space(3))) char *)(lds)));
        // row tiles fastest, then columns, then splits
        m0 = tile % a.tiles_m * S::kBM;
        tile /= a.tiles_m;
        n0 = tile % a.tiles_n * cols + half;
        split = tile / a.tiles_n;
        blocks = (a.k + kG - 1) / kG; // of the summed axis
        k0 = WT ? split * a.per : 0;
        k1 = WT ? min(k0 + a.per, blocks) : blocks;
        pw0 = m0 + 16 * wm;
        cw0 = n0 + 16 * TN * wn;
        // the wave's block of columns: those past n repeat the last ones and are not stored
        const int nb = (cw0 < a.n ? cw0 : a.n - 1) / kG;
        sw0 = WT ? nb : int64_t(nb) * blocks;
        sw1 = WT ? (a.n + kG - 1) / kG : 1;
        u0 = (g ^ (m & 7)) << 4;
        u1 = ((g + 4) ^ (m & 7)) << 4;
        unit = (lane & 7) ^ (lane >> 3);
#pragma unroll
        for (int j = 0; j < S::kWDma; ++j) {
            const int rho = wrow(j), rp = rho % (16 * TN);
            if constexpr (WT) {
                const int c = n0 + 16 * ((lane % kWUnits) ^ (rho & 7)); // n is a multiple of 16
                woff[j] = uint32_t(int64_t(rho) * a.n + (c < a.n ? c : a.n - 16));
            } else {
                const int c = n0 + rho / (16 * TN) * (16 * TN) + wave_col<TN>(rp & 15, rp >> 4);
                woff[j] = uint32_t(int64_t(c < a.n ? c : a.n - 1) * a.k + 16 * unit);
            }
        }
#pragma unroll
        for (int j = 0; j < S::kXDma; ++j) {
            const int p = m0 + (wave * S::kXDma + j) * 8 + (lane >> 3);
            xoff[j] = uint32_t((p < a.T ? p : a.T - 1) * a.ldx + 16 * unit);
        }
        // scales: a wave brings 64 rows', a word each (rows of E8M0 scales may start at any byte); others
        // repeat them
        constexpr int kSParts = (S::kBM + 63) / 64;
        spart = wave % kSParts;
        int sp = m0 + spart * 64 + lane;
        sp = sp < a.T ? sp : a.T - 1;
        sxp = static_cast<const char *>(a.sx) + int64_t(sp) * (E8 ? 1 : 4);
        sstep = a.lds * (E8 ? 1 : 4);
    }
    __device__ __forceinline__ int wrow(int j) const { return ((wave * S::kWDma + j) * 64 + lane) / kWUnits; }

    // Loads part, part + parts, ... of stage kt, to its slot of the ring (past the last stage, the
    // last one's data again, so that every stage has the same number of loads).  No branches: they
    // would keep the matrix instructions around them apart.  Of what lies past k, x's codes
    // are zeros (the fused forms pad them, else the lane loads zeros), and W's are others of the same
    // column, so that a NaN code reaches only results that are NaN in any case.
    __device__ __forceinline__ void issue(int kt, int part = 0, int parts = 1) const
    {
        const uint32_t base = lds0 + uint32_t((kt - k0) % S::kStages) * S::kStageBytes;
        kt = kt < k1 ? kt : k1 - 1;
        const uint8_t *wb = a.W + int64_t(kt) * kG * (WT ? a.n : 1), *xb = a.x + int64_t(kt) * kG;
        const uint32_t wl = base + uint32_t(wave * S::kWDma) * 1024, xl = base + S::kWBytes + uint32_t(wave * S::kXDma) * 1024;
        const bool in = kt * kG + 16 * unit < a.k;
#pragma unroll
        for (int j = 0; j < S::kWDma; ++j) {
            if (j % parts != part) continue;
            uint32_t off = woff[j];
            if constexpr (WT) off -= uint32_t(max(kt * kG + wrow(j) - (a.k - 1), 0)) * uint32_t(a.n);
            else off -= in ? 0u : uint32_t(16 * unit);
            dma16s(wb, off, wl + 1024 * j);
        }
#pragma unroll
        for (int j = 0; j < S::kXDma; ++j) {
            if ((S::kWDma + j) % parts != part) continue;
            if constexpr (is_fused(F) || F == kGradient) dma16s(xb, xoff[j], xl + 1024 * j);
            else dma16(in ? static_cast<const void *>(xb + xoff[j]) : g_zeros, xl + 1024 * j);
        }
        if ((S::kWDma + S::kXDma) % parts == part) {
            const uint32_t to = base + S::kWBytes + S::kXBytes + uint32_t(spart) * 256;
            if constexpr (E8) dma1(sxp + kt * sstep, to);
            else dma4(sxp + kt * sstep, to);
        }
    }

    __device__ __forceinline__ const char *stage(int kt) const { return lds + ((kt - k0) % S::kStages) * S::kStageBytes; }
    __device__ __forceinline__ i32x8 frag(const char *row) const
    {
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(row + u0), hi = *reinterpret_cast<const u32x4 *>(row + u1);
        return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]), int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    }
    __device__ __forceinline__ i32x8 wfrag(const char *st, int t) const
    {
        if constexpr (WT) { // 16 rows at 16 g and 16 at 64 + 16 g, 8 at a time
            const char *p = st + (16 * g + (m >> 1)) * S::kBN + (((TN * wn + t) ^ (m >> 1)) << 4) + 8 * (m & 1);
            typedef __attribute__((address_space(3))) i32x2 lds2;
            i32x2 r[4];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                r[h] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2 *)(p + (8 * (h & 1) + 64 * (h >> 1)) * S::kBN));
            return i32x8{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
        } else {
            return frag(st + (16 * (TN * wn + t) + m) * kG);
        }
    }
    __device__ __forceinline__ i32x8 xfrag(const char *st, int i) const { return frag(st + S::kWBytes + (16 * wm + kStrips * i + m) * kG); }

    // The scales of block kt: bytes, and the rows' factors where the instruction does not take both.
    struct Scales {
        int wb, xb[TM];
        float f[TM];
    };
    // W's scales of the 64 stages from kt, one a lane.  A scalar load in each
    // stage would make every wait for LDS in it a wait for that load too (they return out of
    // order): fp32 results of 65 x 1024, summed axis 4096, took 53 us with them and 42 without (27.5 since codes
    // are widened in one instruction), one row of 12288 columns 12.5 and 11.1.
    __device__ __forceinline__ WScales wscales(int kt) const
    {
        return wscales_at<E8, F>(a.sw, sw0 + (kt + lane < k1 ? kt + lane : k1 - 1) * sw1);
    }
    __device__ __forceinline__ Scales scales(const char *st, const WScale &w) const
    {
        Scales r;
        r.wb = w.e;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const uint32_t sx = *reinterpret_cast<const uint32_t *>(st + S::kWBytes + S::kXBytes + 4 * (16 * wm + m + kStrips * i));
            if constexpr (own_scales(E8, F)) r.xb[i] = int(sx);
            else r.f[i] = factor<E8>(w, sx);
        }
        return r;
    }

    // acc += the block's product of one column tile with every row tile
    __device__ __forceinline__ void multiply(const i32x8 &wf, const i32x8 (&xf)[TM], const Scales &sc, floatx4 (&acc)[TM]) const
    {
        static_assert(E8, "the instruction's own scales");
#pragma unroll
        for (int i = 0; i < TM; ++i)
            acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf[i], acc[i], 0, 0, 0, sc.wb, 0, sc.xb[i]);
    }

    // Behind the last stage: its place in LDS is free when every wave is past its reads.
    __device__ __forceinline__ void correct(floatx4 (&acc)[TN][TM]) const
    {
        if constexpr (is_fused(F)) {
            __builtin_amdgcn_s_waitcnt(kWaitLds0);
            __builtin_amdgcn_s_barrier();
            constexpr int kBytes = S::kStages * S::kStageBytes / S::kWaves / 1024 * 1024;
            const int Tp = a.tp_dev ? uniform(*a.tp_dev) : a.Tp;
            if (pw0 < Tp)
                correction<TN, TM, kStrips, F == kFused, kBytes>(a, Tp, pw0, cw0, lane, lds + wave * kBytes, lds0 + uint32_t(wave) * kBytes, acc);
        }
    }

    __device__ __forceinline__ void store(const floatx4 (&acc)[TN][TM]) const
    {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int p = pw0 + kStrips * i + m;
            if (p >= a.T) continue;
            if constexpr (WT) { // lane: columns 16 t + 4 g .. + 3
                float *o = static_cast<float *>(a.y) + (int64_t(split) * a.T + p) * a.n + cw0 + 4 * g;
#pragma unroll
                for (int t = 0; t < TN; ++t)
                    if (cw0 + 16 * t < a.n) *reinterpret_cast<floatx4 *>(o + 16 * t) = acc[t][i];
            } else {
                const int row = a.perm ? as_global<int32_t>(a.perm)[p] : p;
                if (row < 0) continue;
                float v[4 * TN];
#pragma unroll
                for (int t = 0; t < TN; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[4 * t + q] = acc[t][i][q];
                store_row<TN, F == kF32>(a, row, cw0 + 4 * TN * g, v);
            }
        }
    }
};

template <class S, bool E8, Form F> __device__ __forceinline__ void multiply_tile(const BlockArgs &a, char *lds, int tile, int cols, int half)
{
    constexpr int TN = S::TN, TM = S::TM;
    Tile<S, E8, F> T(a, lds, tile, cols, half);
    floatx4 acc[TN][TM];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[t][i] = floatx4{};
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) T.issue(T.k0 + s);
    WScales ws{};
    for (int kt = T.k0; kt < T.k1; ++kt) {
        if (((kt - T.k0) & 63) == 0) ws = T.wscales(kt);
        const WScale w = wscale_from(ws, (kt - T.k0) & 63);
        // this wave's loads of stage kt have landed and its reads of stage kt - 1 are
        // done; past the barrier that holds for every wave
        __builtin_amdgcn_s_waitcnt(wait_vm_lds0(S::kDma * (S::kStages - 2)));
        __builtin_amdgcn_s_barrier();
        const char *st = T.stage(kt);
        i32x8 xf[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) xf[i] = T.xfrag(st, i);
        const i32x8 w0 = T.wfrag(st, 0);
        const auto sc = T.scales(st, w);
        const i32x8 w1 = T.wfrag(st, 1);
        // the next stage's loads go out while these reads come back
        T.issue(kt + S::kStages - 1);
        if constexpr (F == kF32) {
            exact_block<TN, TM>(xf, e8m0(sc.wb), sc.f, acc, [&](int t) { return t ? T.wfrag(st, t) : w0; });
        } else if constexpr (E8) {
#pragma unroll
            for (int t = 0; t < TN; ++t) T.multiply(t ? t == 1 ? w1 : T.wfrag(st, t) : w0, xf, sc, acc[t]);
        } else {
            // the fmas of a column tile go between the matrix instructions of the next
            constexpr int NW = 3;
            i32x8 wf[NW] = {w0, w1};
            floatx4 q[2][TM];
#pragma unroll
            for (int t = 0; t <= TN; ++t) {
                __builtin_amdgcn_sched_barrier(0);
                if (NW > 2 ? t + 2 < TN : t > 0 && t + 1 < TN) wf[(t + NW - 1) % NW] = T.wfrag(st, t + NW - 1);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    if (t < TN)
                        q[t & 1][i] =
                            __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[t % NW], xf[i], floatx4{}, 0, 0, 0, sc.wb, 0, 127);
                    if (t > 0)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[t - 1][i][e] = fmaf(q[(t - 1) & 1][i][e], sc.f[i], acc[t - 1][i][e]);
                }
            }
        }
    }
    // no direct load may still be writing this workgroup's LDS when it ends
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    T.correct(acc);
    T.store(acc);
}

// A contiguous run of n tiles for each XCD.
__device__ __forceinline__ int own_run(int b, int n) { return (n & 7) == 0 ? (b & 7) * (n >> 3) + (b >> 3) : b; }

template <class S, bool E8, Form F>
__global__ __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(S::kWavesPerSimd, S::kWavesPerSimd)))
void block_gemm_kernel(BlockArgs a)
{
    __shared__ __attribute__((aligned(1024))) char lds[S::kStages * S::kStageBytes];
    const int b = blockIdx.x;
    if constexpr (S::kHalved) {
        if (b >= a.whole) {
            const int c = own_run(b - a.whole, int(gridDim.x) - a.whole);
            multiply_tile<typename S::Half, E8, F>(a, lds, a.whole + c / 2, S::kBN, c % 2 * (S::kBN / 2));
            return;
        }
        multiply_tile<S, E8, F>(a, lds, own_run(b, a.whole), S::kBN, 0);
    } else {
        multiply_tile<S, E8, F>(a, lds, own_run(b, gridDim.x), S::kBN, 0);
    }
}

// Up to 64 rows: bound by reading W once.  A workgroup has 16 TN columns and all rows; its 8 waves
// take every eighth block each, straight from memory in MFMA order (a wave's 16 columns of a
// block are whole 128-byte lines), with 8 KB of W a wave on the way: 64 KB a CU, which
// is what HBM's latency takes.  The waves' sums meet in LDS.  x's codes (at most 64 rows) are
// read by every workgroup from L2; TN grows with the columns, so that there are about 256.
// 4096 -> 4096, fp32 scales: 1 row 5.8 us (2.9 TB/s), 16 6.7, 32 8.6, 64 12.3: 64 rows' codes are 64 MB from the L2.
constexpr int kFew = 64;
constexpr int kMaxSlices = 4; // of the shrink
constexpr int kFewWaves = 8;
template <int TN, int TM, bool E8, Form F> __global__ __launch_bounds__(64 * kFewWaves) void block_few_kernel(BlockArgs a)
{
    // blocks of the wave whose loads are out: four where the registers hold them
    constexpr int D = TN * TM <= 4 && !(F == kF32 && TM == 4) ? 4 : 2;
    constexpr int kPitch = 16 * TN + 4;
    constexpr int kSum = kFewWaves * 16 * TM * kPitch * 4;
    constexpr int kV = is_fused(F) ? 16 * TM * 2 * LORA_MAX_RANK * 2 : 0;
    __shared__ __attribute__((aligned(16))) char lds[kSum > kV ? kSum : kV];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int c0 = int(blockIdx.x) * 16 * TN;
    const int blocks = (a.k + kG - 1) / kG;
    const int nb = (c0 < a.n ? c0 : a.n - 1) / kG;

    const gptr<char> W = as_global<char>(a.W), X = as_global<char>(a.x), SX = as_global<char>(a.sx);
    uint32_t woff[TN];
    int64_t xoff[TM];
    int xrow[TM];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        const int c = c0 + 16 * t + m;
        woff[t] = uint32_t(int64_t(c < a.n ? c : a.n - 1) * a.k);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int p = 16 * i + m;
        xrow[i] = p < a.T ? p : a.T - 1;
        xoff[i] = xrow[i] * a.ldx;
    }
    struct Row {
        u32x4 lo, hi;
    };
    // units g and g + 4 of a row's block; past k those of another place of the row
    auto load = [&](gptr<char> row, int kb) {
        const int k = kb * kG + 16 * g;
        return Row{*(gptr<u32x4>)(row + (k < a.k ? k : 0)), *(gptr<u32x4>)(row + (k + 64 < a.k ? k + 64 : 0))};
    };
    auto operand = [](const Row &r) {
        return i32x8{int(r.lo[0]), int(r.lo[1]), int(r.lo[2]), int(r.lo[3]), int(r.hi[0]), int(r.hi[1]), int(r.hi[2]), int(r.hi[3])};
    };
    struct Operands {
        Row w[TN], x[TM];
        uint32_t sx[TM]; // fp32 bits or a byte
    };
    // The wave's block j, from another place in each workgroup of an XCD: rows are often a
    // power of two apart, so that one block of all rows lies in few channels of the L2.
    const int turn = int(blockIdx.x >> 3) % blocks;
    auto block_of = [&](int j) {
        const int kb = wave + kFewWaves * j + turn;
        return wave + kFewWaves * j >= blocks ? blocks : kb < blocks ? kb : kb - blocks;
    };
    auto load_block = [&](int j, Operands &o) {
        int kb = block_of(j);
        kb = kb < blocks ? kb : blocks - 1;
#pragma unroll
        for (int t = 0; t < TN; ++t) o.w[t] = load(W + woff[t], kb);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            o.x[i] = load(X + xoff[i], kb);
            const int64_t at = kb * a.lds + xrow[i];
            if constexpr (E8) o.sx[i] = *(gptr<uint8_t>)(SX + at);
            else o.sx[i] = *(gptr<uint32_t>)(SX + 4 * at);
        }
    };
    floatx4 acc[TN][TM];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[t][i] = floatx4{};
    // W's scales of the wave's next 64 blocks, one a lane
    WScales wsv{};
    auto load_scales = [&](int j) {
        const int kb = block_of(j + lane);
        wsv = wscales_at<E8, F>(a.sw, int64_t(nb) * blocks + (kb < blocks ? kb : 0));
    };
    auto multiply = [&](int j, Operands &o) {
        const int kb = block_of(j);
        if (kb >= blocks) return; // wave-uniform
        const WScale w = wscale_from(wsv, j & 63);
        const int k = kb * kG + 16 * g;
        auto xfrag = [&](int i) { // past k x's codes are zeros
            if (k >= a.k) o.x[i].lo = u32x4{};
            if (k + 64 >= a.k) o.x[i].hi = u32x4{};
            return operand(o.x[i]);
        };
        if constexpr (F == kF32) {
            i32x8 xf[TM];
            float f[TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                xf[i] = xfrag(i);
                f[i] = factor<E8>(w, o.sx[i]);
            }
            exact_block<TN, TM>(xf, e8m0(w.e), f, acc, [&](int t) { return operand(o.w[t]); });
        } else {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const i32x8 xf = xfrag(i);
                const float f = E8 ? 1.f : factor<E8>(w, o.sx[i]);
#pragma unroll
                for (int t = 0; t < TN; ++t) {
                    const floatx4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(o.w[t]), xf, E8 ? acc[t][i] : floatx4{}, 0,
                                                                                       0, 0, w.e, 0, E8 ? int(o.sx[i]) : 127);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[t][i][q] = E8 ? p[q] : fmaf(p[q], f, acc[t][i][q]);
                }
            }
        }
    };
    const int mine = wave < blocks ? (blocks - wave + kFewWaves - 1) / kFewWaves : 0; // blocks of this wave
    // lane l: the wave's segment l (records past the last have rank 0), loaded
    // before all others, so that no step waits for its own.
    uint32_t Blo = 0, Bhi = 0;
    int srank = 0, sstart = 0, slen = 0;
    float sscale = 0.f;
    if constexpr (is_fused(F))
        if (a.nseg > 0) {
            static_assert(kFew <= 8 * kFewWaves, "a wave's segments");
            const int at = wave + kFewWaves * (lane & 7);
            const lora_seg_desc *d = a.seg + (at < a.nseg ? at : a.nseg - 1);
            const uint64_t B = d->B;
            Blo = uint32_t(B), Bhi = uint32_t(B >> 32);
            srank = d->rank, sstart = d->start, slen = d->len, sscale = d->scale;
            if (at >= a.nseg) srank = 0;
        }
    Operands ring[D];
    load_scales(0);
#pragma unroll
    for (int d = 0; d < D; ++d) load_block(d, ring[d]);

    // The correction.  v = the sum of the shrink's slices, in two bf16 halves in the order of
    // v_halves(), goes to LDS; the segments are dealt to the waves, and kAhead steps of 16 ranks
    // are loaded at a time, the first before the products.  What a load brings is only looked at when
    // all of them are out (v's slices, a step's ranks past the last): 64 rows of 32 adapters 15.7 -> 14.4 us.
    constexpr int kAhead = 4 / TN;
    struct Step {
        u32x4 b[TN];
        int l, j0; // segment, or -1; first rank
    };
    const int pitch = int(a.ldh);
    int s_at = 0, j_at = 0, S = 0; // of the wave's segments
    auto lane_of = [](int v, int l) { return __builtin_amdgcn_readlane(v, l); };
    Step step[kAhead];
    auto load_steps = [&] {
#pragma unroll
        for (Step &f : step) {
            f.l = -1;
            if (s_at >= S) continue;
            const gptr<uint16_t> Bs = as_global<uint16_t>(reinterpret_cast<const void *>(
                uint64_t(uint32_t(lane_of(int(Blo), s_at))) | uint64_t(uint32_t(lane_of(int(Bhi), s_at))) << 32));
            const int r = lane_of(srank, s_at);
            f.l = s_at;
            f.j0 = j_at;
            const int jj = f.j0 + 8 * (g & 1);
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                const int c = c0 + 16 * t + m;
                const int64_t at = int64_t(c < a.n ? c : a.n - 1) * r, elements = int64_t(a.n) * r;
                f.b[t] = elements >= 8 ? eight_of(Bs, at + jj, elements) : few_ranks(Bs + at, jj, r);
            }
            j_at += 16;
            if (j_at >= r) {
                j_at = 0;
                ++s_at;
            }
        }
    };
    auto add_steps = [&] {
#pragma unroll
        for (const Step &f : step) {
            if (f.l < 0) continue;
            const int p0 = lane_of(sstart, f.l), p1 = p0 + lane_of(slen, f.l);
            const float scale = __uint_as_float(uint32_t(lane_of(int(__float_as_uint(sscale)), f.l)));
            const int jj = f.j0 + 8 * (g & 1);
            const int left = lane_of(srank, f.l) - jj; // ranks of this lane's 8 (LDS holds any bits past r)
            u32x4 b[TN];
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                const int c = c0 + 16 * t + m;
                const int64_t elements = int64_t(a.n) * (left + jj);
                b[t] = elements >= 8 ? own_eight(f.b[t], int64_t(c < a.n ? c : a.n - 1) * (left + jj) + jj, elements, left) : f.b[t];
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if (p0 >= 16 * i + 16 || p1 <= 16 * i) continue; // wave-uniform
                const bool in = 16 * i + m >= p0 && 16 * i + m < p1;
                u32x4 v = *reinterpret_cast<const u32x4 *>(lds + ((16 * i + m) * pitch + 2 * f.j0 + 8 * g) * 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] &= (2 * e < left ? 0xFFFFu : 0u) | (2 * e + 1 < left ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int t = 0; t < TN; ++t) {
                    const floatx4 y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[t]),
                                                                              __builtin_bit_cast(bf16x8, v), floatx4{}, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][i][e] = in ? fmaf(scale, y[e], acc[t][i][e]) : acc[t][i][e];
                }
            }
        }
    };
    if constexpr (is_fused(F)) {
        const int Tp = a.tp_dev ? *(cptr<int32_t>)(a.tp_dev) : a.Tp;
        S = __builtin_popcountll(__ballot(lane < 8 && srank > 0));
        load_steps(); // before v, which waits for the loads above
        for (int e = tid; e < Tp * (pitch / 8); e += 64 * kFewWaves) { // 4 ranks of a row a thread
            const int p = e / (pitch / 8), j = e % (pitch / 8) * 4;
            const int64_t at = p * a.ldw + (j < a.ldw ? j : 0);
            // every slice's load goes out before the first is added (choices, not branches)
            floatx4 u[kMaxSlices], v{};
#pragma unroll
            for (int c = 0; c < kMaxSlices; ++c) u[c] = *(gptr<floatx4>)(as_global<float>(a.v) + (c < a.nsl ? c : 0) * a.sl_stride + at);
#pragma unroll
            for (int c = 0; c < kMaxSlices; ++c)
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = c < a.nsl ? v[x] + u[c][x] : v[x];
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                hi[x] = f32_to_bf16(v[x]);
                lo[x] = f32_to_bf16(v[x] - bf16_to_f32(hi[x]));
            }
            char *to = lds + (p * pitch + 32 * (j >> 4) + (j & 15)) * 2;
            *reinterpret_cast<u32x2 *>(to) = u32x2{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
            *reinterpret_cast<u32x2 *>(to + 32) = u32x2{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
        }
    }
    for (int j = 0; j < mine; j += D) {
        if (j && (j & 63) == 0) load_scales(j);
#pragma unroll
        for (int d = 0; d < D; ++d) {
            multiply(j + d, ring[d]);
            if (j + d + D < mine) load_block(j + d + D, ring[d]);
        }
    }
    if constexpr (is_fused(F)) {
        __syncthreads();
        for (;;) {
            add_steps();
            if (s_at >= S) break;
            load_steps();
        }
        __syncthreads(); // v's place is the sums' now
    }

    // the waves' sums, in wave order
    float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i)
            *reinterpret_cast<floatx4 *>(sums + (wave * 16 * TM + 16 * i + m) * kPitch + 16 * t + 4 * g) = acc[t][i];
    __syncthreads();
    for (int e = tid; e < a.T * 4 * TN; e += 64 * kFewWaves) {
        const int p = e / (4 * TN), c = e % (4 * TN) * 4;
        floatx4 y{};
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) {
            const floatx4 u = *reinterpret_cast<const floatx4 *>(sums + (w * 16 * TM + p) * kPitch + c);
#pragma unroll
            for (int x = 0; x < 4; ++x) y[x] += u[x];
        }
        const int row = a.perm ? a.perm[p] : p;
        if (row < 0) continue;
        const int n = c0 + c;
        if constexpr (F == kF32) {
            float *o = static_cast<float *>(a.y) + row * a.ldy + n;
            if (a.vec_y && n + 4 <= a.n) *reinterpret_cast<floatx4 *>(o) = y;
            else
                for (int x = 0; x < 4; ++x)
                    if (n + x < a.n) o[x] = y[x];
        } else {
            uint16_t *o = static_cast<uint16_t *>(a.y) + row * a.ldy + n;
            if (a.vec_y && n + 4 <= a.n) *reinterpret_cast<u32x2 *>(o) = u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            else
                for (int x = 0; x < 4; ++x)
                    if (n + x < a.n) o[x] = uint16_t(f32_to_bf16(y[x]));
        }
    }
}

template <int TN, Form F> void go_few_rows(hipStream_t s, const BlockArgs &a, bool e8, dim3 grid)
{
    const dim3 block(64 * kFewWaves);
    const int tm = a.T <= 16 ? 1 : a.T <= 32 ? 2 : 4;
    if (e8) {
        if (tm == 1) launch_kernel(block_few_kernel<TN, 1, true, F>, grid, block, 0, s, a);
        else if (tm == 2) launch_kernel(block_few_kernel<TN, 2, true, F>, grid, block, 0, s, a);
        else if constexpr (TN <= (F == kF32 ? 1 : 2)) launch_kernel(block_few_kernel<TN, 4, true, F>, grid, block, 0, s, a);
    } else {
        if (tm == 1) launch_kernel(block_few_kernel<TN, 1, false, F>, grid, block, 0, s, a);
        else if (tm == 2) launch_kernel(block_few_kernel<TN, 2, false, F>, grid, block, 0, s, a);
        else if constexpr (TN <= (F == kF32 ? 1 : 2)) launch_kernel(block_few_kernel<TN, 4, false, F>, grid, block, 0, s, a);
    }
}

// Columns, in sixteens, of a workgroup of up to 64 rows, and the workgroups.
struct FewGrid {
    int tn;
    int64_t workgroups;
    FewGrid(int32_t T, int32_t n, bool f32)
    {
        // about a workgroup for each CU
        // (the registers of 64 rows hold fewer columns)
        const int tiles = (n + 15) / 16, most = T <= 32 ? 4 : f32 ? 1 : 2;
        tn = std::min(most, tiles <= 256 ? 1 : tiles <= 512 ? 2 : 4);
        workgroups = (int64_t(tiles) + tn - 1) / tn;
    }
};

template <Form F> int go_few(hipStream_t s, const BlockArgs &a, bool e8)
{
    const FewGrid f(a.T, a.n, F == kF32);
    const dim3 grid{unsigned(f.workgroups)};
    if (f.tn == 1) go_few_rows<1, F>(s, a, e8, grid);
    else if (f.tn == 2) go_few_rows<2, F>(s, a, e8, grid);
    else go_few_rows<4, F>(s, a, e8, grid); // up to 32 rows
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(LORA_ERR_HIP, "block product launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

typedef Shape<8, 4, 2, 4, 2> Large;  // 256 columns x 256 rows, 8 waves
typedef Shape<4, 4, 2, 2, 2> Medium; // 128 x 128, 4 waves, two workgroups on a CU
typedef Shape<2, 2, 4, 2, 3> Small;  // 128 x 64, 8 waves

template <class S, Form F> int go(hipStream_t s, BlockArgs &a, bool e8, int splits = 1)
{
    a.tiles_m = (a.T + S::kBM - 1) / S::kBM;
    a.tiles_n = (a.n + S::kBN - 1) / S::kBN;
    const int64_t tiles = int64_t(a.tiles_m) * a.tiles_n * splits;
    // Where whole rounds of workgroups (one on a CU) leave at most half a round of tiles, those
    // are halves of 128 columns (summed axis 4096, fp32 scales / E8M0, us: 4096 x 4352 119 -> 100 / 103 -> 89,
    // 2304 x 8192 119 -> 100 / 104 -> 89, 4096 x 14336 280 -> 265 / 248 -> 236).
    const int rest = S::kHalved && tiles > 256 && splits == 1 && tiles % 256 <= 128 ? int(tiles % 256) : 0;
    a.whole = int(tiles) - rest;
    const dim3 grid{unsigned(tiles + rest)}, block(S::kThreads);
    if (e8) launch_kernel(block_gemm_kernel<S, true, F>, grid, block, 0, s, a);
    else launch_kernel(block_gemm_kernel<S, false, F>, grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(LORA_ERR_HIP, "block product launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

template <class S> int64_t tiles_of(int32_t T, int32_t n) { return (int64_t(T) + S::kBM - 1) / S::kBM * ((int64_t(n) + S::kBN - 1) / S::kBN); }

// The tile of a product of T rows and n columns.  A round of Large, Medium and Small tiles
// over the chip takes about 1.6, 0.8 and 0.5 us for each block of the summed axis (Medium
// and Small 0.9 and 0.8 with two workgroups on a CU), so the smallest tile whose workgroups
// run all at once is taken, two of them on a CU, and the largest where none does.  Summed
// axis 4096, rows x columns, us of Small / Medium / Large:
//    128 x  4096   17 / 27 / 53      517 x 12288   52 /  41 /  59     4096 x 4096  108 /  83 /  71
//   1024 x  4096   28 / 29 / 56     1024 x 12288   79 /  64 /  62    2304 x 12288  186 / 151 / 136
// An fp32 result takes four times the matrix instructions and widens each code that it reads, which
// larger tiles do less often; Large ones do not fit the registers.  Small / Medium, 517 x 1531 (summed axis 1008)
// 13 / 21, 517 x 4096 44 / 42, 1024 x 4096 47 / 45.
enum Size { kSmall, kMedium, kLarge };
inline Size size_of(int32_t T, int32_t n, bool f32)
{
    if (tiles_of<Small>(T, n) <= (f32 ? 256 : 512)) return kSmall;
    return f32 || tiles_of<Medium>(T, n) <= 512 ? kMedium : kLarge;
}

// More workgroups than a launch has are refused, before anything of the call runs.  A rest of
// halved tiles is at most 128 more.
inline int check_tiles(int64_t tiles, int threads)
{
    if (tiles + 128 > most_workgroups(threads)) return fail(LORA_ERR_ARG, "block product: too many tiles");
    return LORA_OK;
}
template <class S> int check_shape(int32_t T, int32_t n, int splits) { return check_tiles(tiles_of<S>(T, n) * splits, S::kThreads); }
inline int check_size(Size size, int32_t T, int32_t n, int splits)
{
    return size == kLarge ? check_shape<Large>(T, n, splits) : size == kMedium ? check_shape<Medium>(T, n, splits) : check_shape<Small>(T, n, splits);
}
inline int check_product(int32_t T, int32_t n, bool f32)
{
    if (T <= kFew) return check_tiles(FewGrid(T, n, f32).workgroups, 64 * kFewWaves);
    return check_size(size_of(T, n, f32), T, n, 1);
}

template <Form F> int launch_product(hipStream_t s, BlockArgs &a, bool e8)
{
    if (a.T <= kFew) return go_few<F == kFusedAnyRank ? kFused : F>(s, a, e8);
    const Size size = size_of(a.T, a.n, F == kF32);
    if constexpr (F != kF32)
        if (size == kLarge) return go<Large, F>(s, a, e8);
    return size == kMedium ? go<Medium, F>(s, a, e8) : go<Small, F>(s, a, e8);
}

// Tile and splits of the rows' gradient: as many splits of the summed axis as fill the
// chip once, with at least 4 blocks each.
struct GradientPlan {
    Size size;
    int splits, per;
    GradientPlan(int32_t T, int32_t d_in, int32_t d_out)
    {
        size = size_of(T, d_in, false);
        const int64_t tiles = size == kLarge ? tiles_of<Large>(T, d_in) : size == kMedium ? tiles_of<Medium>(T, d_in) : tiles_of<Small>(T, d_in);
        const int blocks = (d_out + kG - 1) / kG;
        const int most = int(std::max<int64_t>(1, std::min<int64_t>({256 / tiles, blocks / 4, 16})));
        per = (blocks + most - 1) / most;
        splits = (blocks + per - 1) / per;
    }
    // floats of the sums of a batch of up to T rows: a batch of fewer has more splits
    static size_t sums(int32_t T, int32_t d_in)
    {
        const size_t one = size_t(T) * size_t(d_in);
        return std::max(one, std::min(16 * one, size_t(256) * 256 * 256));
    }
};

// Workspace of the fused call: the shrink's slice partials, v's halves, x's codes (rows of
// whole blocks) and scales (rows padded to 4).
int64_t vh_pitch(int32_t max_rank) { return 2 * int64_t((max_rank + 15) / 16 * 16); }
struct FusedBlockWs {
    size_t vh, codes, scales, end;
    int64_t ldq, lds;
    FusedBlockWs(int32_t T, int32_t d_in, int32_t max_rank)
    {
        const int64_t groups = (int64_t(d_in) + kG - 1) / kG;
        ldq = groups * kG;
        lds = (int64_t(T) + 3) / 4 * 4;
        vh = up256(combined_workspace_bytes(T, d_in, max_rank));
        codes = vh + up256(size_t(T) * size_t(vh_pitch(max_rank)) * 2);
        scales = codes + up256(size_t(T) * size_t(ldq));
        end = scales + up256(size_t(groups) * size_t(lds) * 4);
    }
};

// Workspace of the gradient call: the adapters' gradients', then dy's codes and scales and
// the fp32 sums of dx.
struct GradientWs {
    size_t codes, scales, parts, end;
    int64_t ldq, lds;
    GradientWs(int32_t T, int32_t d_in, int32_t d_out, int32_t max_rank)
    {
        const int64_t groups = (int64_t(d_out) + kG - 1) / kG;
        ldq = groups * kG;
        lds = (int64_t(T) + 3) / 4 * 4;
        codes = up256(sgmv_backward_workspace_bytes(T, d_in, d_out, max_rank));
        scales = codes + up256(size_t(T) * size_t(ldq));
        parts = scales + up256(size_t(groups) * size_t(lds) * 4);
        end = parts + GradientPlan::sums(T, d_in) * 4;
    }
};

} // namespace

int launch_linear_block(hipStream_t s, const LinearBlockCall &c)
{
    if (c.T == 0) return LORA_OK;
    BlockArgs a{};
    a.x = static_cast<const uint8_t *>(c.x);
    a.ldx = c.ldx;
    a.sx = c.sx;
    a.lds = c.lds;
    a.W = static_cast<const uint8_t *>(c.W);
    a.sw = c.sw;
    a.k = c.d_in;
    a.n = c.d_out;
    a.T = c.T;
    a.y = c.y;
    a.ldy = c.ldy;
    const int es = c.out_dtype == LORA_F32 ? 4 : 2;
    a.vec_y = aligned16(c.y) && c.ldy * es % 16 == 0;
    const bool e8 = c.scale_type == LORA_SCALE_E8M0;
    const int st = check_product(c.T, c.d_out, c.out_dtype == LORA_F32);
    if (st) return st;
    return c.out_dtype == LORA_F32 ? launch_product<kF32>(s, a, e8) : launch_product<kBf16>(s, a, e8);
}

size_t fused_block_workspace_bytes(int32_t T, int32_t d_in, int32_t max_rank) { return FusedBlockWs(T, d_in, max_rank).end; }

int launch_fused_linear_block(hipStream_t s, const ShrinkArgs &sa, const void *W0, const void *sw, int scale_type,
                              const ExpandArgs &ea, const PlanView &p, void *ws)
{
    const int T = p.h->num_tokens;
    const int max_rank = p.h->max_rank < 1 ? 1 : p.h->max_rank;
    const FusedBlockWs w(T, sa.d_in, max_rank);
    char *base = static_cast<char *>(ws);
    BlockArgs a{};
    a.perm = reinterpret_cast<const int32_t *>(p.dev + p.h->perm_offset);
    QuantCall q{};
    q.dtype = LORA_BF16;
    q.x = sa.x;
    q.ldx = sa.ldx;
    q.rows = T;
    q.cols = sa.d_in;
    q.perm = a.perm;
    q.codes = base + w.codes;
    q.ldq = w.ldq;
    q.pad = true;
    q.block_rows = 1;
    q.scale_type = scale_type;
    q.scales = base + w.scales;
    q.lds = w.lds;
    int st = check_product(T, ea.d_out, false);
    if (st) return st;
    uint16_t *vh = reinterpret_cast<uint16_t *>(base + w.vh);
    a.ldh = vh_pitch(max_rank);
    a.nsl = 0;
    if (p.h->num_sorted > 0) {
        a.v = static_cast<const float *>(ws);
        st = T <= kFew ? launch_sgmv_shrink_quantize(s, sa, p, static_cast<float *>(ws), &a.ldw, &a.sl_stride, &a.nsl, q)
                       : launch_v_halves(s, sa, p, ws, vh, a.ldh, 0.f, &q);
        if (st) return st;
        if (a.nsl > kMaxSlices) return fail(LORA_ERR_ARG, "block product: %d d_in slices > %d", a.nsl, kMaxSlices);
    } else if ((st = launch_quantize(s, q))) {
        return st;
    }
    a.x = static_cast<const uint8_t *>(q.codes);
    a.ldx = w.ldq;
    a.sx = q.scales;
    a.lds = w.lds;
    a.W = static_cast<const uint8_t *>(W0);
    a.sw = sw;
    a.k = sa.d_in;
    a.n = ea.d_out;
    a.T = T;
    a.y = ea.y;
    a.ldy = ea.ldy;
    a.vec_y = 1;
    a.segidx = reinterpret_cast<const int32_t *>(p.dev + p.h->segidx_offset);
    a.seg = reinterpret_cast<const lora_seg_desc *>(p.dev + p.h->seg_offset);
    a.Tp = p.h->num_sorted;
    a.nseg = p.h->num_sorted > 0 ? p.h->num_segments : 0;
    a.tp_dev = plan_sorted_dev(p);
    a.vh = vh;
    const bool e8 = scale_type == LORA_SCALE_E8M0;
    return ranks_of_8(p) ? launch_product<kFused>(s, a, e8) : launch_product<kFusedAnyRank>(s, a, e8);
}

size_t fused_block_backward_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t max_rank)
{
    return GradientWs(T, d_in, d_out, max_rank).end;
}

int launch_fused_block_backward(hipStream_t s, const BackwardArgs &b, const void *W0, const void *sw, int scale_type,
                                const PlanView &p, void *ws)
{
    const lora_plan_header *h = p.h;
    const int T = h->num_tokens;
    const GradientWs w(T, b.d_in, b.d_out, h->max_rank < 1 ? 1 : h->max_rank);
    const GradientPlan g(T, b.d_in, b.d_out);
    char *base = static_cast<char *>(ws);
    int st = check_size(g.size, T, b.d_in, g.splits);
    if (!st) st = check_dx_join(b, p);
    if (st) return st;
    QuantCall q{};
    q.dtype = LORA_BF16;
    q.x = b.dy;
    q.ldx = b.lddy;
    q.rows = T;
    q.cols = b.d_out;
    q.perm = reinterpret_cast<const int32_t *>(p.dev + h->perm_offset);
    q.codes = base + w.codes;
    q.ldq = w.ldq;
    q.pad = true;
    q.block_rows = 1;
    q.scale_type = scale_type;
    q.scales = base + w.scales;
    q.lds = w.lds;
    if (h->num_sorted > 0) { // the adapters' gradients, and u
        BackwardArgs adapters = b;
        adapters.dx = nullptr;
        const uint16_t *ur;
        int64_t ldu;
        st = launch_sgmv_backward(s, adapters, p, ws, &ur, &ldu, &q);
    } else {
        st = launch_quantize(s, q);
    }
    if (st) return st;
    BlockArgs a{};
    a.x = static_cast<const uint8_t *>(q.codes);
    a.ldx = w.ldq;
    a.sx = q.scales;
    a.lds = w.lds;
    a.W = static_cast<const uint8_t *>(W0);
    a.sw = sw;
    a.k = b.d_out;
    a.n = b.d_in;
    a.T = T;
    a.y = base + w.parts;
    a.per = g.per;
    const bool e8 = scale_type == LORA_SCALE_E8M0;
    if (g.size == kLarge) st = go<Large, kGradient>(s, a, e8, g.splits);
    else if (g.size == kMedium) st = go<Medium, kGradient>(s, a, e8, g.splits);
    else st = go<Small, kGradient>(s, a, e8, g.splits);
    if (st) return st;
    return launch_dx_join(s, b, p, ws, reinterpret_cast<const float *>(base + w.parts), g.splits);
}

} // namespace lora
