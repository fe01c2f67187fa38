// Input gradient of the fused adapted layer on gfx950:
//
//     dx[t] = dy[t] W0 + u[t] A_s          (W0 [d_out, d_in], A_s [r, d_in])
//
// for every token t, overwriting dx, with u = s dy B from the backward shrink
// (backward.hip), in bf16 hi and lo halves.  One GEMM over the plan's rows: the
// summed axis is d_out, and u A is appended to it as further steps (a step of 32
// holds 16 ranks: u's hi halves, then its lo halves, against the same 16 rows
// of A), so that the correction costs ceil(r / 16) steps per segment that meets a
// tile and no code of its own.
//
// A workgroup computes 256 columns x ROWS plan rows with 8 waves.  The summed
// axis advances 32 per stage through a ring of LDS stages filled by direct
// global-to-LDS loads (16 bytes per lane) issued kStages - 1 stages ahead.
// W0 (and A) are contiguous along the columns, not along the summed axis that
// MFMA wants in a lane: their part of a stage holds 32 rows of 512 bytes, read
// with ds_read_b64_tr_b16, which hands each lane one column of 4 rows.  Unit
// (16 bytes) un of row q lies in slot un ^ 4 (q % 4): the 4 rows of a read fall in
// distinct banks.  The dy (u) part holds rows of 64 bytes, unit un of row q in
// slot un ^ (q / 2 % 4).
// Units that lie outside (rows of another segment, ranks past r, the summed
// axis past d_out) are loaded from a block of zeros.
//
// Few tiles (a narrow d_in, few rows) leave most CUs idle, so the stages are split:
// each split writes fp32 sums to the workspace, and a last launch (the backward's
// dx kernel) adds them in split order, and u A.  With 200 adapters over 1024
// tokens the correction took 20 us as steps of the split GEMM (117 us, 96
// without); the last launch, which sums the parts in any case, takes 22 us with it.
#include "device.h"
#include "internal.h"

#include <algorithm>

namespace lora {
namespace {

constexpr int kCols = 256;    // columns per workgroup
constexpr int kBK = 32;       // summed axis per stage
constexpr int kThreads = 512; // 8 waves
constexpr int kStages = 4;
constexpr int kWBytes = kBK * kCols * 2; // W0 part of a stage: 16 KB
constexpr int kMaxSplits = 16;
constexpr int kFill = 256; // workgroups that fill the chip

// WC column groups of waves (8 / WC row groups); a wave has TM row tiles and TN
// column tiles of 16.
template <int ROWS> struct Shape;
template <> struct Shape<256> {
    static constexpr int WC = 4, TM = 8, TN = 4;
};
template <> struct Shape<64> {
    static constexpr int WC = 8, TM = 4, TN = 2;
};

// Read-only memory at a wave-uniform address: scalar loads, which wait for no
// vector load in flight.
template <typename T> using cptr = const __attribute__((address_space(4))) T *;
template <typename T> __device__ __forceinline__ cptr<T> as_const(const T *p) { return (cptr<T>)(p); }
__device__ __forceinline__ int wave_sum(int v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return uniform(v);
}

struct DgradArgs {
    const uint16_t *dy;
    int64_t lddy;
    const uint16_t *W0;
    const uint16_t *tail; // [T][8]: dy's last d_out % 8 columns and zeros, or null
    int d_in, d_out;
    const int32_t *perm;
    const int32_t *segidx;
    const lora_seg_desc *seg;
    const uint16_t *ur; // u as MFMA operands: [16 positions][16-rank tile][lane 16 g + position % 16][8 ranks]
    int64_t ldu;        // elements from 16 positions to the next
    int T, Tp;
    uint16_t *dx;
    int64_t lddx;
    float *part; // [split][T][d_in] when splits > 1
    int tiles_m, tiles_n, splits;
};

// Rows' columns d_out / 8 * 8 .. d_out - 1, padded with zeros to 8.
__global__ __launch_bounds__(256) void dgrad_tail_kernel(const uint16_t *__restrict__ dy, int64_t lddy, int T, int d_out,
                                                         uint16_t *__restrict__ tail)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= T * 8) return;
    const int t = i >> 3, c = d_out / 8 * 8 + (i & 7);
    tail[i] = c < d_out ? dy[int64_t(t) * lddy + c] : 0;
}

template <int ROWS>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void dgrad_kernel(DgradArgs a)
{
    typedef Shape<ROWS> G;
    constexpr int kXBytes = ROWS * kBK * 2, kStageBytes = kWBytes + kXBytes;
    constexpr int kWDma = kWBytes / 1024 / 8;                    // W0 loads of a wave per stage: 2
    constexpr int kXDma = kXBytes / 1024 >= 8 ? kXBytes / 1024 / 8 : 1;
    constexpr bool kXAll = kXBytes / 1024 >= 8;                  // every wave loads dy rows
    static_assert(kStages * kStageBytes <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char lds[kStages * kStageBytes];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int wr = wave / G::WC, wc = wave % G::WC;
    const uint32_t lds0 = uint32_t(uintptr_t((__attribute__((address_space(3))) char *)(lds)));

    // Row tiles fastest, then columns, then splits; a contiguous run per XCD.
    const int nwg = a.tiles_m * a.tiles_n * a.splits;
    int id = blockIdx.x;
    if ((nwg & 7) == 0) id = (id & 7) * (nwg >> 3) + (id >> 3);
    const int m0 = (id % a.tiles_m) * ROWS;
    id /= a.tiles_m;
    const int c0 = (id % a.tiles_n) * kCols, split = id / a.tiles_n;
    const int nk = (a.d_out + kBK - 1) / kBK; // stages of the base product

    // The stages of the base product, shared by the splits, then (one split) the
    // correction steps of the segments s0 .. s1 that meet the tile.
    int s0 = 0, s1 = -1, ncorr = 0;
    if (a.splits == 1 && m0 < a.Tp) {
        s0 = uniform(a.segidx[m0]);
        s1 = uniform(a.segidx[min(m0 + ROWS, a.Tp) - 1]);
        for (int s = s0; s <= s1; s += 64) ncorr += wave_sum(s + lane <= s1 ? (a.seg[s + lane].rank + 15) >> 4 : 0);
    }
    const int k_begin = int(int64_t(nk) * split / a.splits);
    const int nbase = int(int64_t(nk) * (split + 1) / a.splits) - k_begin, nst = nbase + ncorr;

    // This lane's units.  W0 part: slot 64 i + lane of the stage, i = 2 wave + j:
    // row slot / 32.  dy part: row slot / 4.
    const char *zeros = reinterpret_cast<const char *>(g_zeros);
    int wrow[kWDma], wcol[kWDma];
    const char *wp[kWDma];
#pragma unroll
    for (int j = 0; j < kWDma; ++j) {
        const int slot = (wave * kWDma + j) * 64 + lane;
        wrow[j] = slot >> 5;
        const int c = c0 + 8 * ((slot & 31) ^ ((wrow[j] & 3) << 2));
        wcol[j] = c < a.d_in ? c : 0; // past d_in: columns that are not stored
        wp[j] = reinterpret_cast<const char *>(a.W0 + int64_t(k_begin * kBK + wrow[j]) * a.d_in + wcol[j]);
    }
    const bool xw = kXAll || wave < kXBytes / 1024;
    int xpos[kXDma], xk[kXDma], xtok[kXDma];
    const char *xp[kXDma];
#pragma unroll
    for (int j = 0; j < kXDma; ++j) {
        const int slot = ((xw ? wave : 0) * kXDma + j) * 64 + lane, row = slot >> 2;
        xpos[j] = m0 + row;
        xk[j] = 8 * ((slot & 3) ^ ((row >> 1) & 3));
        xtok[j] = a.perm[xpos[j] < a.T ? xpos[j] : a.T - 1];
        xp[j] = reinterpret_cast<const char *>(a.dy + int64_t(xtok[j]) * a.lddy + k_begin * kBK + xk[j]);
    }

    // Stage i of this run: nbase base stages, then the correction.
    int is = s0, ij = 0; // the next correction step to load, and its segment (read ahead)
    uint64_t nA = 0;
    int nr = 0, nfirst = 0, nlen = 0;
    auto read_seg = [&] {
        const cptr<lora_seg_desc> d = as_const(a.seg + is);
        nA = d->A, nr = d->rank, nfirst = d->start, nlen = d->len;
    };
    if (nst > nbase) read_seg();
    auto issue = [&](int i) {
        const uint32_t wbase = lds0 + uint32_t((i % kStages) * kStageBytes + wave * kWDma * 1024);
        const uint32_t xbase = lds0 + uint32_t((i % kStages) * kStageBytes + kWBytes + wave * kXDma * 1024);
        const int k0 = (k_begin + i) * kBK;
        if (i < nbase) {
            if (k0 + kBK <= a.d_out) {
#pragma unroll
                for (int j = 0; j < kWDma; ++j) dma16(wp[j], wbase + j * 1024);
                if (xw) {
#pragma unroll
                    for (int j = 0; j < kXDma; ++j) dma16(xp[j], xbase + j * 1024);
                }
#pragma unroll
                for (int j = 0; j < kWDma; ++j) wp[j] += int64_t(kBK) * a.d_in * 2;
#pragma unroll
                for (int j = 0; j < kXDma; ++j) xp[j] += kBK * 2;
            } else { // the last, partial stage
#pragma unroll
                for (int j = 0; j < kWDma; ++j) dma16(k0 + wrow[j] < a.d_out ? wp[j] : zeros, wbase + j * 1024);
                if (xw) {
#pragma unroll
                    for (int j = 0; j < kXDma; ++j) {
                        const int k = k0 + xk[j];
                        const char *p = k + 8 <= a.d_out ? xp[j]
                                        : k < a.d_out    ? reinterpret_cast<const char *>(a.tail + int64_t(xtok[j]) * 8)
                                                         : zeros;
                        dma16(p, xbase + j * 1024);
                    }
                }
            }
        } else if (i < nst) {
            const int r = nr, first = nfirst, last = nfirst + nlen;
            const uint16_t *A = reinterpret_cast<const uint16_t *>(nA);
#pragma unroll
            for (int j = 0; j < kWDma; ++j) {
                const int rank = ij + (wrow[j] & 15);
                const char *p = reinterpret_cast<const char *>(A + int64_t(rank) * a.d_in + wcol[j]);
                dma16(rank < r ? p : zeros, wbase + j * 1024);
            }
            if (xw) {
#pragma unroll
                for (int j = 0; j < kXDma; ++j) {
                    // unit xk / 8: hi parts of ranks 0 .. 7, 8 .. 15, then lo parts
                    const char *p = reinterpret_cast<const char *>(a.ur + int64_t(xpos[j] >> 4) * a.ldu + 32 * ij + 16 * xk[j] + 8 * (xpos[j] & 15));
                    dma16(xpos[j] >= first && xpos[j] < last ? p : zeros, xbase + j * 1024);
                }
            }
            ij += 16;
            if (ij >= r) {
                ij = 0;
                is = min(is + 1, s1);
                read_seg();
            }
        } else { // past the end: keeps the number of loads in flight
#pragma unroll
            for (int j = 0; j < kWDma; ++j) dma16(zeros, wbase + j * 1024);
            if (xw) {
#pragma unroll
                for (int j = 0; j < kXDma; ++j) dma16(zeros, xbase + j * 1024);
            }
        }
    };

    // This lane's fragment places in a stage.  dy rows of a wave's row tiles are
    // 1024 bytes apart; W0: tiles t and t + 1 are the halves of one unit, tiles t + 2
    // lie 4 units on, the second 4 rows of a fragment 4 rows on.
    const int xr = wr * G::TM * 16 + m;
    const uint32_t xoff = uint32_t(kWBytes + xr * 64 + ((g ^ ((xr >> 1) & 3)) << 4));
    uint32_t woff[G::TN / 2];
#pragma unroll
    for (int t = 0; t < G::TN / 2; ++t) {
        const int row = 8 * g + (m >> 2), un = wc * 2 * G::TN + t * 4 + (m & 3);
        woff[t] = uint32_t(row * kCols * 2 + ((un ^ ((row & 3) << 2)) << 4));
    }
    auto read_w = [&](const char *st, bf16x8(&wf)[G::TN]) {
#pragma unroll
        for (int t = 0; t < G::TN; ++t) {
            const char *p = st + woff[t >> 1] + 8 * (t & 1);
            const u32x2 lo = read_tr(p), hi = read_tr(p + 4 * kCols * 2);
            wf[t] = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
        }
    };
    constexpr int kHalf = G::TM / 2; // row tiles are read and multiplied in two halves
    auto read_x = [&](const char *st, int half, bf16x8(&xf)[kHalf]) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            xf[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(st + xoff + (half * kHalf + k) * 1024));
    };

    floatx4 acc[G::TN][G::TM];
#pragma unroll
    for (int t = 0; t < G::TN; ++t)
#pragma unroll
        for (int i = 0; i < G::TM; ++i) acc[t][i] = floatx4{};

    // Stage i + 1 is there and stage i's slot free: this wave's reads of stage i and
    // its loads of stage i + 1 are done (later ones may be in flight), and every
    // wave's.  Refills the slot.
    auto next_stage = [&](int i) {
        asm volatile("" ::: "memory");
        if (xw) __builtin_amdgcn_s_waitcnt(wait_vm_lds0((kWDma + kXDma) * (kStages - 2)));
        else __builtin_amdgcn_s_waitcnt(wait_vm_lds0(kWDma * (kStages - 2)));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(i + kStages);
    };
    // Base stage i: the second half of its rows is read while the first half's
    // products run, and the next stage's columns and first half while the second
    // half's do.  w0: its column fragments, w1: the next stage's.
    bf16x8 wa[G::TN], wb[G::TN], xa[kHalf], xb[kHalf];
    auto base_stage = [&](int i, bf16x8(&w0)[G::TN], bf16x8(&w1)[G::TN]) {
        read_x(lds + (i % kStages) * kStageBytes, 1, xb);
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
#pragma unroll
            for (int t = 0; t < G::TN; ++t)
                acc[t][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0[t], xa[k], acc[t][k], 0, 0, 0);
        next_stage(i);
        const char *st = lds + ((i + 1) % kStages) * kStageBytes;
        read_w(st, w1);
        read_x(st, 0, xa);
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
#pragma unroll
            for (int t = 0; t < G::TN; ++t)
                acc[t][kHalf + k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0[t], xb[k], acc[t][kHalf + k], 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) issue(i);
    if (xw) __builtin_amdgcn_s_waitcnt(wait_vm((kWDma + kXDma) * (kStages - 1)));
    else __builtin_amdgcn_s_waitcnt(wait_vm(kWDma * (kStages - 1)));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read_w(lds, wa);
    read_x(lds, 0, xa);
    int i = 0;
    for (; i + 1 < nbase; i += 2) {
        base_stage(i, wa, wb);
        base_stage(i + 1, wb, wa);
    }
    if (i < nbase) base_stage(i++, wa, wb);
    // Correction: a step's products go to the rows of its segment alone, so that a
    // NaN or infinity in one adapter (times the other rows' zeros) stays with it.
    for (int cs = s0, cj = 0; i < nst; ++i) {
        const cptr<lora_seg_desc> d = as_const(a.seg + cs);
        const int first = d->start, last = first + d->len;
        const char *st = lds + (i % kStages) * kStageBytes;
        read_w(st, wa);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            read_x(st, h, xa);
#pragma unroll
            for (int k = 0; k < kHalf; ++k) {
                const int p0 = m0 + (wr * G::TM + h * kHalf + k) * 16;
                if (p0 + 16 <= first || p0 >= last) continue; // wave-uniform
                const bool mine = p0 + m >= first && p0 + m < last;
#pragma unroll
                for (int t = 0; t < G::TN; ++t) {
                    const floatx4 v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[t], xa[k], floatx4{}, 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[t][h * kHalf + k][q] += mine ? v[q] : 0.f;
                }
            }
        }
        cj += 16;
        if (cj >= d->rank) {
            cj = 0;
            ++cs;
        }
        next_stage(i);
    }
    // no direct load may still be writing this workgroup's LDS when it ends
    __builtin_amdgcn_s_waitcnt(wait_vm(0));

    // lane: 16 columns (8 for TN = 2) of each of its rows, as 16-byte pieces
#pragma unroll
    for (int k = 0; k < G::TM; ++k) {
        const int p = m0 + (wr * G::TM + k) * 16 + m;
        if (p >= a.T) continue;
#pragma unroll
        for (int h = 0; h < G::TN / 2; ++h) {
            const int c = c0 + wc * 16 * G::TN + h * 32 + g * 8;
            if (c >= a.d_in) continue; // d_in is a multiple of 8
            const floatx4 lo = acc[2 * h][k], hi = acc[2 * h + 1][k];
            if (a.splits > 1) {
                float *o = a.part + (int64_t(split) * a.T + p) * a.d_in + c;
                *reinterpret_cast<floatx4 *>(o) = lo;
                *reinterpret_cast<floatx4 *>(o + 4) = hi;
            } else {
                *reinterpret_cast<u32x4 *>(a.dx + int64_t(a.perm[p]) * a.lddx + c) =
                    u32x4{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
            }
        }
    }
}

// Splits of the summed axis: as many as fill the chip in one round, with at
// least 16 stages each (GEMM and join, us, at 8 / 16 splits: 64 rows, 4096 columns,
// d_out 4096 18.7 / 22.5, d_out 14336 39.9 / 35.3; 8 rows, 2048 columns, d_out 8192
// 21.2 / 19.0).
int splits_of(int64_t tiles, int32_t d_out)
{
    const int64_t stages = (int64_t(d_out) + kBK - 1) / kBK;
    return int(std::max<int64_t>(1, std::min<int64_t>({kFill / tiles, stages / 16, kMaxSplits})));
}

// Stages that a CU goes through one after the other: rounds of workgroups, times a
// workgroup's.
int64_t stages_of_cu(int64_t tiles, int32_t d_out)
{
    const int64_t splits = splits_of(tiles, d_out), stages = (int64_t(d_out) + kBK - 1) / kBK;
    return (tiles * splits + kFill - 1) / kFill * ((stages + splits - 1) / splits);
}

// Rows of a tile.  A stage takes 0.39 us with 64 rows and 0.87 with 256, which also
// begin and end later (by the time of some 40 of the small stages): so 256 where 64
// rows would go through more than 2 s + 36 stages, s those of 256 rows.  Over 260
// sizes (T 96 to 2048, d_in and d_out 1024 to 14336) the other choice would have been
// over 5% faster in 10, by 28% at most.  64 / 256 rows, us, u, GEMM and join.  d 4096 ->
// 4096: 256 rows 30 / 39, 512 40 / 51, 640 54 / 52, 1024 55 / 64 (256 is taken), 1536
// 100 / 82; d_in 4096, d_out 14336: 192 rows 68 / 71, 384 117 / 89, 1024 198 / 138; d_in
// 1024, d_out 8192: 512 rows 33 / 42, 1024 43 / 54.
int rows_of(int32_t T, int32_t d_in, int32_t d_out)
{
    const int64_t cols = (int64_t(d_in) + kCols - 1) / kCols;
    const int64_t few = stages_of_cu((int64_t(T) + 63) / 64 * cols, d_out);
    return few <= 2 * stages_of_cu((int64_t(T) + 255) / 256 * cols, d_out) + 36 ? 64 : 256;
}

// dy's tail columns, and the splits' sums: splits x tiles <= kFill tiles of at most
// 256 x 256, and at most kMaxSplits of T x d_in.
size_t tail_bytes(int32_t T) { return up256(size_t(T) * 16); }
size_t part_bytes(int32_t T, int32_t d_in)
{
    return std::min(size_t(kFill) * 256 * kCols * 4, up256(size_t(T) * size_t(d_in) * 4 * kMaxSplits));
}

} // namespace

size_t fused_backward_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t max_rank)
{
    return up256(sgmv_backward_workspace_bytes(T, d_in, d_out, max_rank)) + tail_bytes(T) + part_bytes(T, d_in);
}

int launch_fused_backward(hipStream_t s, const BackwardArgs &b, const void *W0, const PlanView &p, void *ws)
{
    const lora_plan_header *h = p.h;
    const int T = h->num_tokens;
    const int max_rank = h->max_rank < 1 ? 1 : h->max_rank;
    DgradArgs a{};
    const int rows = rows_of(T, b.d_in, b.d_out);
    a.tiles_m = (T + rows - 1) / rows;
    a.tiles_n = (b.d_in + kCols - 1) / kCols;
    const int64_t tiles = int64_t(a.tiles_m) * a.tiles_n;
    if (tiles > most_workgroups(kThreads)) return fail(LORA_ERR_ARG, "fused backward: too many tiles");
    a.splits = splits_of(tiles, b.d_out);
    if (T > (1 << 27))
        return fail(LORA_ERR_ARG, "fused backward: too many rows");
    char *w = static_cast<char *>(ws) + up256(sgmv_backward_workspace_bytes(T, b.d_in, b.d_out, max_rank));
    // the adapters' gradients, and u
    if (h->num_sorted > 0) {
        BackwardArgs q = b;
        q.dx = nullptr;
        const int st = launch_sgmv_backward(s, q, p, ws, &a.ur, &a.ldu);
        if (st) return st;
    }
    a.dy = static_cast<const uint16_t *>(b.dy);
    a.lddy = b.lddy;
    a.W0 = static_cast<const uint16_t *>(W0);
    a.d_in = b.d_in;
    a.d_out = b.d_out;
    a.perm = reinterpret_cast<const int32_t *>(p.dev + h->perm_offset);
    a.segidx = reinterpret_cast<const int32_t *>(p.dev + h->segidx_offset);
    a.seg = reinterpret_cast<const lora_seg_desc *>(p.dev + h->seg_offset);
    a.T = T;
    a.Tp = h->num_sorted;
    a.dx = static_cast<uint16_t *>(b.dx);
    a.lddx = b.lddx;
    a.part = reinterpret_cast<float *>(w + tail_bytes(T));
    hipError_t e = hipSuccess;
    if (b.d_out % 8) {
        uint16_t *tail = reinterpret_cast<uint16_t *>(w);
        a.tail = tail;
        launch_kernel(dgrad_tail_kernel, dim3(unsigned((int64_t(T) * 8 + 255) / 256)), dim3(256), 0, s, a.dy, a.lddy, T,
                      a.d_out, tail);
        if ((e = hipGetLastError()) != hipSuccess)
            return fail(LORA_ERR_HIP, "fused backward tail launch: %s", hipGetErrorString(e));
    }
    const dim3 grid{unsigned(tiles * a.splits)};
    if (rows == 64) launch_kernel(dgrad_kernel<64>, grid, dim3(kThreads), 0, s, a);
    else launch_kernel(dgrad_kernel<256>, grid, dim3(kThreads), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return fail(LORA_ERR_HIP, "fused backward launch: %s", hipGetErrorString(e));
    if (a.splits > 1) return launch_dx_join(s, b, p, ws, a.part, a.splits);
    return LORA_OK;
}

} // namespace lora
