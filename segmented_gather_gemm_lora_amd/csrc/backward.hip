// Gradients of the segmented correction y[t] += s (x[t] A^T) B^T on gfx950, for
// the adapters of many requests at once (A_i [r, d_in], B_i [d_out, r] row-major,
// s = alpha_i / r_i, dy the gradient of y):
//
//     u[p, :] = s dy[perm p, :] B        v[p, :] = s x[perm p, :] A^T
//     dx[perm p, :] += u[p, :] A
//     dA = sum over the segment's p of u[p, :]^T x[perm p, :]
//     dB = sum over the segment's p of dy[perm p, :]^T v[p, :]
//
// u and v are full sums over d_out and d_in, so dA and dB can only start when
// they are known: x and dy are read twice.  Launches:
//  1. bwd_shrink_kernel: u and v of every block of 16 rows (one workgroup per
//     block and side, its waves split the long axis and are summed in LDS in
//     wave order), stored in the forms that the next launches multiply with;
//     one more workgroup lists the work items of launch 2.  Many long segments of
//     large ranks: bwd_shrink_ring_kernel, 64 rows per workgroup;
//  2. bwd_out_kernel: dA, dB and dx.  An item of dA and dB is one segment's rows
//     inside one span of `span` sorted positions; a workgroup takes 256 columns of
//     x or dy of it.  A segment inside one span is written at once; the sums of a
//     segment that crosses spans go to the workspace.  Further workgroups take 256
//     columns of dx for a block of 16 rows or a chunk of 64;
//  3. bwd_reduce_kernel: adds those partial sums in span order (a fixed order:
//     the gradients do not change from run to run).
//
// Access shape.  A vector load or store costs the L1 one access per run of lanes
// with consecutive addresses, so every large access has 8 or more adjacent lanes on
// one row's consecutive 16 bytes (operands loaded straight into MFMA's lane order,
// 16 rows x 4 pieces that are 16 lanes apart, cost 51 accesses per load: the shrink
// of 4096 rows of rank 16 took 27 us so, 21 as it is).  Rows go to a wave's own LDS tile and are
// read back in MFMA's order; u and v are stored in that order by launch 1; results
// leave with consecutive columns in consecutive lanes.
//
// The transposed operands.  MFMA wants, in each lane, consecutive elements of
// the summed axis.  x, dy (summed over rows for dA, dB), A (summed over its
// rows for dx) and B (summed over its rows for u) are contiguous along the
// other axis: their LDS tiles are read with ds_read_b64_tr_b16, which hands lane i
// of every 16 lanes column i of 4 rows.  fp32 operands go to
// v_mfma_f32_16x16x4_f32, which takes one element per lane.
//
// Precision.  u and v are fp32 sums.  For dA and dB they are fed to bf16 MFMA
// as three bf16 parts (hi + mid + lo, 24 significant bits: all of an fp32), so the
// fp32 gradients keep fp32 accuracy; for dx, which is rounded to bf16, as two
// (16 significant bits, as in the forward's expand).  fp32 calls multiply
// exactly.
#include "e4m3.h"

#include <algorithm>
#include <type_traits>

namespace lora {
namespace {

typedef __attribute__((address_space(1))) float *gfloat; // written
typedef __attribute__((address_space(1))) floatx4 *gfloatx4;

__device__ __forceinline__ bf16x8 join8(u32x2 a, u32x2 b)
{
    return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}

// 16 bytes at a wave-uniform base (kept in scalar registers) plus a lane's 32-bit
// byte offset: no 64-bit address per load in vector registers.
__device__ __forceinline__ u32x4 load16(const void *base, uint32_t off)
{
    return *(gptr<u32x4>)(as_global<char>(base) + off);
}
// 16 bytes from or to a place that is aligned to its elements alone.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <class T> __device__ __forceinline__ u32x4 load16_any(gptr<T> p) { return *(gptr<u32x4_any>)(p); }

constexpr int kWin = 32; // sorted positions of one step over rows; u and v are stored in windows of it
constexpr int kPieces = 64 * 16; // bytes of one operand: 16 per lane

template <int DT> struct Elem;
template <> struct Elem<LORA_BF16> {
    using T = uint16_t;
    using F = bf16x8;              // operand of one MFMA step
    static constexpr int kVec = 8; // elements of the summed axis per lane
    static constexpr int kStep = 32;
    static constexpr int kParts = 3; // operands of a window and 16 ranks: hi, mid, lo of 32 positions
};
template <> struct Elem<LORA_F32> {
    using T = float;
    using F = floatx4;
    static constexpr int kVec = 4;
    static constexpr int kStep = 16;
    static constexpr int kParts = 2; // 16 positions each
};

template <int DT>
__device__ __forceinline__ floatx4 mma(const typename Elem<DT>::F &a, const typename Elem<DT>::F &b, floatx4 c)
{
    if constexpr (DT == LORA_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
}

// A lane's 16 output columns of a 64-column wave tile, as (MFMA tile t, D row
// 4 g + q): 16-byte pieces that make 64 contiguous bytes over the 4 lane
// groups.  MFMA row m of tile t stands for column col(m >> 2, 4 t + (m & 3)).
template <int DT> __device__ __forceinline__ int col(int g, int v)
{
    constexpr int E = DT == LORA_BF16 ? 8 : 4;
    return (v / E) * 4 * E + g * E + v % E;
}

struct Item {
    uint64_t grad_A, grad_B; // the adapter's gradients, 0: not wanted
    int32_t begin, end;      // sorted positions
    int32_t rank;
    int32_t slot;            // partial sums' place, -1: the gradient itself
};
static_assert(sizeof(Item) == 32, "one record per item");
struct Split { // a segment whose sums lie in `count` slots from slot0
    int32_t seg, slot0, count, reserved;
};

struct BwdArgs {
    const void *x, *dy;
    int64_t ldx, lddy;
    int d_in, d_out;
    const lora_seg_desc *seg;
    const lora_blk_desc *blk;
    const lora_chunk_desc *chunk;
    const int32_t *perm;
    int S, nblk, nchunk;
    int nt;         // 16-rank tiles of the largest rank
    // u and v as MFMA operands (16 bytes a lane, lane = 16 g + m):
    char *ut, *vt;  // [window][part][tile]: rank m of the tile, bf16 positions 8 g .. + 7 (fp32 4 g .. + 3)
    char *ur;       // [16 positions][tile]: position m, bf16 ranks 8 (g % 2) .. + 7 of the hi (g < 2) or lo
                    // part, fp32 ranks 4 g .. + 3
    Item *items;
    Split *segsplits;
    float *part;
    int64_t part_stride;
    int span, nitems, nsplit;
    const uint64_t *grad_A, *grad_B;
    int accumulate;
    int sides; // bit 0: v is wanted, bit 1: u
    // launch 2: column tiles of x and of both, groups of 64 ranks, gradient workgroups,
    // column tiles of dx
    int tiles_A, tiles, groups, ngrad, tiles_x;
    bool chunks; // dx by chunks of 64 rows, else by blocks of 16
    void *dx;
    int64_t lddx;
    // JOIN: the sums of a base product in parts, [splits][T][d_in] by plan rows
    const float *joins;
    int splits, T, Tp;
};

// ----------------------------------------------------------------------------
// Launch 1.  One workgroup: 16 rows, all ranks, one side.
// Side 0: v, K = d_in, W = A (row j is rank j, contiguous along K).
// Side 1: u, K = d_out, W = B (row k holds the ranks).
// ----------------------------------------------------------------------------
// Elements k .. of a row, 0 past K, one by one.
template <int DT> __device__ __forceinline__ u32x4 load_row(gptr<typename Elem<DT>::T> row, int k, int K)
{
    using E = Elem<DT>;
    typename E::F f;
#pragma unroll
    for (int e = 0; e < E::kVec; ++e) {
        const typename E::T w = row[k + e < K ? k + e : K - 1];
        if constexpr (DT == LORA_BF16) f[e] = __builtin_bit_cast(__bf16, uint16_t(k + e < K ? w : 0));
        else f[e] = k + e < K ? w : 0.f;
    }
    return __builtin_bit_cast(u32x4, f);
}

// Work items: the segments cut at multiples of `span`.  One workgroup.
__device__ void list_items(const BwdArgs &a, int *scan, int nthreads)
{
    const int tid = threadIdx.x;
    int item0 = 0, slot0 = 0, split0 = 0;
    for (int s0 = 0; s0 < a.S; s0 += nthreads) {
        const int s = s0 + tid;
        int start = 0, end = 0, n = 0, r = 0;
        uint64_t gA = 0, gB = 0;
        if (s < a.S) {
            const lora_seg_desc &d = a.seg[s];
            start = d.start;
            end = start + d.len;
            r = d.rank;
            n = (end - 1) / a.span - start / a.span + 1;
            gA = a.grad_A ? a.grad_A[d.adapter] : 0;
            gB = a.grad_B ? a.grad_B[d.adapter] : 0;
        }
        const int ns = n > 1 ? n : 0, nq = n > 1 ? 1 : 0;
        // sums before this thread: over its wave's lanes, then the waves'
        const int own[3] = {n, ns, nq}, lane = tid & 63, wave = tid >> 6;
        int upto[3] = {n, ns, nq}, total[3] = {0, 0, 0};
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const int v = __shfl_up(upto[q], d);
                if (lane >= d) upto[q] += v;
            }
        if (lane == 63)
            for (int q = 0; q < 3; ++q) scan[3 * wave + q] = upto[q];
        __syncthreads();
        for (int w = 0; w < nthreads >> 6; ++w)
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const int v = scan[3 * w + q];
                if (w < wave) upto[q] += v;
                total[q] += v;
            }
        const int it = item0 + upto[0] - own[0], sl = slot0 + upto[1] - own[1], sp = split0 + upto[2] - own[2];
        for (int i = 0; i < n; ++i) {
            const int b = i == 0 ? start : (start / a.span + i) * a.span;
            const int e = i == n - 1 ? end : (start / a.span + i + 1) * a.span;
            a.items[it + i] = Item{gA, gB, b, e, r, n > 1 ? sl + i : -1};
        }
        if (nq) a.segsplits[sp] = Split{s, sl, n, 0};
        item0 += total[0];
        slot0 += total[1];
        split0 += total[2];
        __syncthreads();
    }
}

// v = h + mid + low, three bf16 (24 bits); an infinity or NaN has no rest.
struct Parts {
    uint32_t h, mid, low;
};
__device__ __forceinline__ Parts parts_of(float v)
{
    Parts p;
    p.h = f32_to_bf16(v);
    const float rest = (p.h & 0x7f80u) != 0x7f80u ? v - bf16_to_f32(p.h) : 0.f;
    p.mid = f32_to_bf16(rest);
    p.low = f32_to_bf16(rest - bf16_to_f32(p.mid));
    return p;
}

// One value of u (side 1) or v, scaled: position p, rank 16 t + jm (0 past the
// segment's rank), in the operands that launch 2 reads.
template <int DT> __device__ __forceinline__ void store_uv(const BwdArgs &a, int side, int p, int t, int jm, float v)
{
    char *parts = side ? a.ut : a.vt, *ur = a.ur + (int64_t(p >> 4) * a.nt + t) * kPieces;
    if constexpr (DT == LORA_BF16) {
        const Parts f = parts_of(v);
        const int at = (((p & 31) >> 3) * 16 + jm) * 8 + (p & 7);
        uint16_t *o = reinterpret_cast<uint16_t *>(parts + (int64_t(p / kWin) * 3 * a.nt + t) * kPieces) + at;
        const int64_t part = int64_t(a.nt) * kPieces / 2;
        o[0] = uint16_t(f.h);
        o[part] = uint16_t(f.mid);
        o[2 * part] = uint16_t(f.low);
        if (side) {
            uint16_t *u = reinterpret_cast<uint16_t *>(ur) + ((jm >> 3) * 16 + (p & 15)) * 8 + (jm & 7);
            u[0] = uint16_t(f.h);
            u[2 * 16 * 8] = uint16_t(f.mid);
        }
    } else {
        float *o = reinterpret_cast<float *>(parts + ((int64_t(p / kWin) * 2 + ((p & 31) >> 4)) * a.nt + t) * kPieces);
        o[(((p & 15) >> 2) * 16 + jm) * 4 + (p & 3)] = v;
        if (side) reinterpret_cast<float *>(ur)[((jm >> 2) * 16 + (p & 15)) * 4 + (jm & 3)] = v;
    }
}

constexpr int kShrinkWaves = 8;

// A wave advances 128 bytes of every row at a time (a pair of steps: 64 elements in
// bf16, 32 in fp32).  Rows of x (dy) and of A are loaded as 8 rows x 128 bytes per
// instruction, B as pieces of 16 bytes in the order of its rows, and kept in the
// wave's LDS tile: rows of 128 bytes with unit (16 bytes) un of row q in slot
// un ^ (q % 8), B as below.
template <int DT, int RT> struct ShrinkTile {
    static constexpr int kPair = 2 * Elem<DT>::kStep;     // elements of the long axis
    static constexpr int kX = 2048;                       // bytes: x rows
    static constexpr int kRowB = DT == LORA_BF16 ? 32 * RT : 64 * RT + 16; // bytes of a row of B's tile
    static constexpr int kB = kPair * kRowB;
    static constexpr int kW = kB > RT * 2048 ? kB : RT * 2048;
    static constexpr int kBytes = kX + kW;
};

// One side's operands of a workgroup: rows of x or dy, and A or B.
struct ShrinkSide {
    const void *src, *mat;
    int64_t ld;
    int K, r, rt0;
    const int32_t *rows;
    int n;
};

// A pair's loads, in registers.
template <int DT, int RT> struct ShrinkOps {
    static constexpr int kWs = RT * 2; // loads of W (B: 64 rows of 2 RT pieces, fp32 32 rows of 4 RT)
    u32x4 x[2], w[kWs];
};

// B's place in the tile.  bf16: 32-byte granules (one rank tile of a row), moved so
// that the 4 rows of a transposing read fall in distinct banks; fp32: padded rows.
template <int DT, int RT> __device__ __forceinline__ int b_at(int k, int byte)
{
    if constexpr (DT == LORA_BF16)
        return k * 32 * RT + (((byte >> 5) ^ ((RT == 4 ? k >> 1 : k >> 2) & (RT - 1))) << 5) + (byte & 31);
    else return k * (64 * RT + 16) + byte;
}

// FULL: everything that is loaded lies inside.  VEC: rows are whole aligned 16-byte
// pieces below 4 GiB (xoff: byte offsets); else at any alignment (xoff: tokens).
// BANY: B's rows are not whole 16-byte pieces.
template <int DT, bool VEC, int SIDE, bool BANY, bool FULL, int RT>
__device__ __forceinline__ void shrink_load(ShrinkOps<DT, RT> &o, const ShrinkSide &sd, const uint32_t (&xoff)[2],
                                            int k, int lane)
{
    using E = Elem<DT>;
    using T = typename E::T;
    constexpr int es = int(sizeof(T));
    const int kl = k + E::kVec * (lane & 7); // this lane's first element of a row
    const char *xb = static_cast<const char *>(sd.src) + int64_t(k) * es;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (FULL && VEC) {
                o.x[h] = load16(xb, xoff[h]);
            } else {
                const gptr<T> row = VEC ? (gptr<T>)(as_global<char>(sd.src) + xoff[h]) - E::kVec * (lane & 7)
                                        : as_global<T>(sd.src) + int64_t(xoff[h]) * sd.ld;
                if constexpr (FULL) o.x[h] = load16_any(row + kl);
                else o.x[h] = load_row<DT>(row, kl, sd.K);
            }
        }
#pragma unroll
    for (int i = 0; i < o.kWs; ++i) {
        if constexpr (SIDE == 0) { // rank rows 16 (i / 2) + 8 (i % 2) + lane / 8
            const int j = 16 * sd.rt0 + 8 * i + (lane >> 3);
            const gptr<T> row = as_global<T>(sd.mat) + int64_t(j < sd.r ? j : sd.r - 1) * sd.K;
            if constexpr (FULL && VEC)
                o.w[i] = load16(static_cast<const char *>(sd.mat) + int64_t(k) * es,
                                uint32_t(j < sd.r ? j : sd.r - 1) * uint32_t(sd.K * es) + 16 * (lane & 7));
            else if constexpr (FULL) o.w[i] = load16_any(row + kl);
            else o.w[i] = load_row<DT>(row, kl, sd.K);
        } else { // piece lane + 64 i of the pair's rows of B
            constexpr int kPer = 16 * RT / E::kVec; // pieces of a row
            const int q = lane + 64 * i, kr = k + q / kPer, j = 16 * sd.rt0 + E::kVec * (q % kPer);
            const int jj = j < sd.r ? j : 0; // past r: columns that nothing reads
            const gptr<T> B = as_global<T>(sd.mat);
            if constexpr (FULL && !BANY)
                o.w[i] = load16(static_cast<const char *>(sd.mat) + int64_t(k) * sd.r * es, uint32_t((q / kPer) * sd.r + jj) * es);
            else if constexpr (FULL) o.w[i] = load16_any(B + (int64_t(kr) * sd.r + jj));
            else {
                o.w[i] = load_row<DT>(B + int64_t(kr < sd.K ? kr : sd.K - 1) * sd.r, jj, sd.r);
                if (kr >= sd.K) o.w[i] = u32x4{};
            }
        }
    }
}

template <int DT, int SIDE, int RT>
__device__ __forceinline__ void shrink_put(const ShrinkOps<DT, RT> &o, char *tile, int lane)
{
    constexpr int kX = ShrinkTile<DT, RT>::kX;
    const int q0 = lane >> 3;
    const int at = q0 * 128 + (((lane & 7) ^ q0) << 4); // rows 8 on: 1024 bytes on, the same slot
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4 *>(tile + h * 1024 + at) = o.x[h];
#pragma unroll
    for (int i = 0; i < o.kWs; ++i) {
        if constexpr (SIDE == 0) {
            *reinterpret_cast<u32x4 *>(tile + kX + i * 1024 + at) = o.w[i];
        } else {
            constexpr int kPer = 16 * RT / Elem<DT>::kVec;
            const int q = lane + 64 * i;
            *reinterpret_cast<u32x4 *>(tile + kX + b_at<DT, RT>(q / kPer, 16 * (q % kPer))) = o.w[i];
        }
    }
}

template <int DT, int SIDE, int RT>
__device__ __forceinline__ void shrink_mma(floatx4 (&acc)[RT], const char *tile, int lane)
{
    using E = Elem<DT>;
    using F = typename E::F;
    constexpr int kX = ShrinkTile<DT, RT>::kX;
    const int m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        auto row_frag = [&](const char *rows) { // row m, unit 4 s + g
            return __builtin_bit_cast(F, *reinterpret_cast<const u32x4 *>(rows + m * 128 + (((4 * s + g) ^ (m & 7)) << 4)));
        };
        F wf[RT];
        const F xf = row_frag(tile);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if constexpr (SIDE == 0) {
                wf[i] = row_frag(tile + kX + i * 2048);
            } else if constexpr (DT == LORA_BF16) {
                u32x2 t[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) t[b] = read_tr(tile + kX + b_at<DT, RT>(32 * s + 8 * g + 4 * b + (m >> 2), 32 * i + 8 * (m & 3)));
                wf[i] = join8(t[0], t[1]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    wf[i][e] = *reinterpret_cast<const float *>(tile + kX + b_at<DT, RT>(16 * s + 4 * g + e, 4 * (16 * i + m)));
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = mma<DT>(xf, wf[i], acc[i]);
    }
}

// This wave's part of the sums: NP pairs at a time (one rank tile: 2, else 1; 1 or 3
// there and 2 for more tiles measured no faster), the next ones' loads in flight while
// the current ones are multiplied.
template <int DT, bool VEC, int SIDE, bool BANY, int RT, int NP>
__device__ __forceinline__ void shrink_sum(floatx4 (&acc)[RT], const ShrinkSide &sd, char *tile, int wave, int lane)
{
    using E = Elem<DT>;
    using Tl = ShrinkTile<DT, RT>;
    constexpr int kChunk = NP * Tl::kPair, kNext = kShrinkWaves * kChunk;
    uint32_t xoff[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) { // rows past n: never stored
            const uint32_t t = uint32_t(sd.rows[min(8 * h + (lane >> 3), sd.n - 1)]);
            xoff[h] = VEC ? t * uint32_t(sd.ld * int(sizeof(typename E::T))) + 16 * (lane & 7) : t;
        }
    // pieces of rows of B that hold fewer or other ranks reach up to kVec - 1
    // elements into the rows after, so they keep kVec rows from B's end
    const int last = sd.K - kChunk - (SIDE == 1 && BANY ? E::kVec : 0);
    ShrinkOps<DT, RT> o[NP];
    int k = wave * kChunk;
    auto load = [&] {
#pragma unroll
        for (int q = 0; q < NP; ++q) shrink_load<DT, VEC, SIDE, BANY, true>(o[q], sd, xoff, k + q * Tl::kPair, lane);
    };
    if (k <= last) load();
    while (k <= last) {
#pragma unroll
        for (int q = 0; q < NP; ++q) shrink_put<DT, SIDE>(o[q], tile + q * Tl::kBytes, lane);
        k += kNext;
        if (k <= last) load();
#pragma unroll
        for (int q = 0; q < NP; ++q) shrink_mma<DT, SIDE>(acc, tile + q * Tl::kBytes, lane);
    }
    for (; k < sd.K; k += kNext) // the last, partial chunk
        for (int q = 0; q < NP && k + q * Tl::kPair < sd.K; ++q) {
            shrink_load<DT, VEC, SIDE, BANY, false>(o[0], sd, xoff, k + q * Tl::kPair, lane);
            shrink_put<DT, SIDE>(o[0], tile, lane);
            shrink_mma<DT, SIDE>(acc, tile, lane);
        }
}

// Where the work of launch 1 goes on.  Workgroup b runs on XCD b % 8: an XCD takes a
// run of consecutive units, so that a segment's A and B are fetched into few L2s;
// the list of items first (one workgroup), then the longer side, and each group of
// 64 ranks by itself.  False: nothing (more) to do here.
__device__ __forceinline__ bool shrink_unit(const BwdArgs &a, int units, int *scan, int &unit, int &side, int &group)
{
    const int run = (units + 7) / 8, q = int(blockIdx.x >> 3) - 1;
    if (q < 0) {
        if (blockIdx.x == 0) list_items(a, scan, blockDim.x);
        return false;
    }
    unit = int(blockIdx.x % 8) * run + q % run;
    const bool both = a.sides == 3;
    side = both ? (q / run % 2 == 0) == (a.d_out >= a.d_in) : a.sides - 1;
    group = both ? q / run / 2 : q / run;
    return unit < units;
}

// A workgroup takes a block of 16 rows and 64 ranks (all of them by one workgroup:
// 517 rows of ranks to 100, 22 us, 10 so); its waves share the long axis.  Four rank
// tiles: 2 waves per SIMD, so that the loads ahead stay in registers (left to
// itself the compiler makes 4 fit: mixed ranks 65 us, 58 so).
template <int DT, bool VEC, int RT> __device__ __forceinline__ void shrink_block(const BwdArgs &a)
{
    constexpr int W = kShrinkWaves, NP = RT == 1 ? 2 : 1;
    constexpr int kTile = NP * ShrinkTile<DT, RT>::kBytes;
    constexpr int kLds = std::max(W * kTile, W * RT * 1024); // tiles, or the waves' sums
    static_assert(kLds <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(16))) char lds[kLds];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    int unit, side, group;
    if (!shrink_unit(a, a.nblk, reinterpret_cast<int *>(lds), unit, side, group)) return;
    const lora_blk_desc *d = a.blk + unit;
    const int r = d->rank, n = d->n, p0 = d->p0;
    const float scale = d->scale;
    const void *mat = reinterpret_cast<const void *>(side ? d->B : d->A);
    const int rt0 = RT * group;
    if (16 * rt0 >= r) return;
    const ShrinkSide sd = side ? ShrinkSide{a.dy, mat, a.lddy, a.d_out, r, rt0, d->rows, n} : ShrinkSide{a.x, mat, a.ldx, a.d_in, r, rt0, d->rows, n};
    const int ntiles = (r + 15) >> 4;
    char *tile = lds + wave * kTile;
    floatx4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = floatx4{};
    if (side == 0) shrink_sum<DT, VEC, 0, false, RT, NP>(acc, sd, tile, wave, lane);
    else if (r % Elem<DT>::kVec) shrink_sum<DT, VEC, 1, true, RT, NP>(acc, sd, tile, wave, lane);
    else shrink_sum<DT, VEC, 1, false, RT, NP>(acc, sd, tile, wave, lane);
    // lane l of tile i holds D[row 4 (l / 16) + q][rank l % 16]
    float *red = reinterpret_cast<float *>(lds);
    __syncthreads(); // every wave is past its tiles, and past the last sums
#pragma unroll
    for (int i = 0; i < RT; ++i) *reinterpret_cast<floatx4 *>(red + ((wave * RT + i) * 64 + lane) * 4) = acc[i];
    __syncthreads();
    for (int idx = tid; idx < RT * 256; idx += W * 64) {
        const int i = idx >> 8, l2 = (idx >> 2) & 63, q4 = idx & 3;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += red[((w * RT + i) * 64 + l2) * 4 + q4];
        const int mm = 4 * (l2 >> 4) + q4, t = rt0 + i, jm = l2 & 15, j = 16 * t + jm;
        if (mm >= n || t >= ntiles) continue;
        const int p = p0 + mm;
        const float v = j < r ? sum * scale : 0.f;
        store_uv<DT>(a, side, p, t, jm, v);
    }
}
template <int DT, bool VEC, int RT>
__global__ __launch_bounds__(kShrinkWaves * 64) __attribute__((amdgpu_waves_per_eu(2, RT == 4 ? 2 : 8))) void bwd_shrink_kernel(BwdArgs a)
{
    shrink_block<DT, VEC, RT>(a);
}
// And dy's rows quantized by further workgroups, a launch less and dy read from memory once: 64 rows of
// 4096 columns 6.6 us (6.8 and 3.2 in two), 4096 rows 37 (24.4 and 17.9).
template <int RT>
__global__ __launch_bounds__(kShrinkWaves * 64) __attribute__((amdgpu_waves_per_eu(2, RT == 4 ? 2 : 8)))
void bwd_shrink_quantize_kernel(BwdArgs a, QuantAlong along)
{
    if (blockIdx.x < along.first) shrink_block<LORA_BF16, true, RT>(a);
    else quantize_along<kShrinkWaves / 4>(along, blockIdx.x);
}

// The same for many long segments (bf16, VEC, ranks above 32, multiples of 8): a
// workgroup takes a chunk of up to 64 rows, a wave 16 of them and 64 ranks, over the
// whole long axis.  Stages of 128 bytes of every row come through a ring of LDS tiles
// filled by direct global-to-LDS loads, kRing - 1 stages ahead, so A and B are read
// once for 64 rows.  16384 rows of rank 64, d 4096: 98 us (the loads alone 83, the
// bytes at the copy rate 52; ring of 4: 104), by blocks of 16 rows 125.
constexpr int kRing = 3;

__global__ __launch_bounds__(256) void bwd_shrink_ring_kernel(BwdArgs a)
{
    constexpr int RT = 4, kXBytes = 64 * 128, kWBytes = 64 * 128, kStage = kXBytes + kWBytes;
    constexpr int kDma = 2; // loads of x, and of W, of a wave per stage
    __shared__ __attribute__((aligned(1024))) char lds[kRing * kStage];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), m = lane & 15, g = lane >> 4;
    int unit, side, group;
    if (!shrink_unit(a, a.nchunk, reinterpret_cast<int *>(lds), unit, side, group)) return;
    const lora_chunk_desc *d = a.chunk + unit;
    const int r = d->rank, n = d->n, p0 = d->p0;
    const float scale = d->scale;
    const int rt0 = RT * group;
    if (16 * rt0 >= r) return;
    const int K = side ? a.d_out : a.d_in, nst = (K + 63) / 64;
    const uint32_t lds0 = uint32_t(uintptr_t((__attribute__((address_space(3))) char *)(lds)));
    const char *zeros = reinterpret_cast<const char *>(g_zeros);
    // x: instruction 2 wave + j, row 8 i + lane / 8, slot lane % 8 holds unit slot ^ (row % 8)
    const int un = (lane & 7) ^ (lane >> 3);
    const char *xp[kDma];
#pragma unroll
    for (int j = 0; j < kDma; ++j) {
        const int row = d->rows[min(8 * (2 * wave + j) + (lane >> 3), n - 1)]; // past n: not stored
        xp[j] = side ? static_cast<const char *>(a.dy) + (int64_t(row) * a.lddy + 8 * un) * 2
                     : static_cast<const char *>(a.x) + (int64_t(row) * a.ldx + 8 * un) * 2;
    }
    // W: instruction 2 wave + j.  A: as x; B: row k of 8 slots, 32-byte granules
    // moved as in b_at
    const char *wp[kDma];
    int wk[kDma];
    const int64_t step = side ? int64_t(64) * r * 2 : 128;
#pragma unroll
    for (int j = 0; j < kDma; ++j) {
        const int s = (kDma * wave + j) * 64 + lane;
        if (side == 0) {
            const int rank = 16 * rt0 + (s >> 3);
            wk[j] = 8 * un;
            wp[j] = reinterpret_cast<const char *>(d->A) + (int64_t(rank < r ? rank : r - 1) * K + 8 * un) * 2;
        } else {
            const int k = s >> 3, pos = s & 7, gran = (pos >> 1) ^ ((k >> 1) & 3), rank = 16 * (rt0 + gran) + 8 * (pos & 1);
            wk[j] = k;
            wp[j] = reinterpret_cast<const char *>(d->B) + (int64_t(k) * r + (rank < r ? rank : 0)) * 2;
        }
    }
    auto issue = [&](int i) {
        const uint32_t xbase = lds0 + uint32_t((i % kRing) * kStage + wave * kDma * 1024);
        const uint32_t wbase = lds0 + uint32_t((i % kRing) * kStage + kXBytes + wave * kDma * 1024);
        const int k0 = 64 * i;
        // past K (the last stage, and stages past the last): zeros
#pragma unroll
        for (int j = 0; j < kDma; ++j) dma16(k0 + 8 * un < K ? xp[j] + int64_t(k0) * 2 : zeros, xbase + j * 1024);
#pragma unroll
        for (int j = 0; j < kDma; ++j) dma16(k0 + wk[j] < K ? wp[j] + i * step : zeros, wbase + j * 1024);
    };
    floatx4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = floatx4{};
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue(i);
    for (int i = 0; i < nst; ++i) {
        // this wave's loads of stage i are done, then every wave's, and every wave
        // has read stage i - 1
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(wait_vm_lds0(2 * kDma * (kRing - 2)));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(i + kRing - 1);
        const char *xt = lds + (i % kRing) * kStage + wave * 2048, *wt = lds + (i % kRing) * kStage + kXBytes;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = m * 128 + (((4 * s + g) ^ (m & 7)) << 4);
            const bf16x8 xf = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(xt + at));
#pragma unroll
            for (int q = 0; q < RT; ++q) {
                bf16x8 wf;
                if (side == 0) {
                    wf = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(wt + q * 2048 + at));
                } else {
                    u32x2 t[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) t[b] = read_tr(wt + b_at<LORA_BF16, RT>(32 * s + 8 * g + 4 * b + (m >> 2), 32 * q + 8 * (m & 3)));
                    wf = join8(t[0], t[1]);
                }
                acc[q] = mma<LORA_BF16>(xf, wf, acc[q]);
            }
        }
    }
    // no direct load may still be writing the ring, and every wave is past its reads
    __builtin_amdgcn_s_waitcnt(wait_vm_lds0(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // u or v through LDS, so that whole 16-byte pieces of the operands are stored
    // (by single values: 14 us more for 16384 rows of rank 64)
    constexpr int kPitch = 16 * RT + 1;
    static_assert(64 * kPitch * 4 <= kRing * kStage, "the sums fit the ring");
    float *sum = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sum[(16 * wave + 4 * g + q) * kPitch + 16 * i + m] = 16 * (rt0 + i) + m < r ? acc[i][q] * scale : 0.f;
    __syncthreads();
    const int cols = min(16 * RT, ((r + 15) & ~15) - 16 * rt0), oct0 = p0 >> 3, octs = ((p0 + n - 1) >> 3) - oct0 + 1;
    const int64_t part = int64_t(a.nt) * kPieces / 2;
    for (int idx = tid; idx < octs * cols; idx += 256) {
        const int oct = idx / cols, j = idx - oct * cols, p = 8 * (oct0 + oct), row = p - p0;
        uint16_t *o = reinterpret_cast<uint16_t *>((side ? a.ut : a.vt) + (int64_t(p / kWin) * 3 * a.nt + rt0 + (j >> 4)) * kPieces) +
                      (((p & 31) >> 3) * 16 + (j & 15)) * 8;
        if (row >= 0 && row + 8 <= n) {
            u32x4 w[3];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Parts f0 = parts_of(sum[(row + 2 * e) * kPitch + j]), f1 = parts_of(sum[(row + 2 * e + 1) * kPitch + j]);
                w[0][e] = f0.h | f1.h << 16, w[1][e] = f0.mid | f1.mid << 16, w[2][e] = f0.low | f1.low << 16;
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x4 *>(o + q * part) = w[q];
        } else {
            for (int e = max(0, -row); e < 8 && row + e < n; ++e) {
                const Parts f = parts_of(sum[(row + e) * kPitch + j]);
                o[e] = uint16_t(f.h), o[part + e] = uint16_t(f.mid), o[2 * part + e] = uint16_t(f.low);
            }
        }
    }
    if (side)
        for (int idx = tid; idx < n * (cols >> 3); idx += 256) {
            const int c8 = idx / n, row = idx - c8 * n, p = p0 + row;
            uint16_t *u = reinterpret_cast<uint16_t *>(a.ur + (int64_t(p >> 4) * a.nt + rt0 + (c8 >> 1)) * kPieces) +
                          ((c8 & 1) * 16 + (p & 15)) * 8;
            u32x4 w[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Parts f0 = parts_of(sum[row * kPitch + 8 * c8 + 2 * e]), f1 = parts_of(sum[row * kPitch + 8 * c8 + 2 * e + 1]);
                w[0][e] = f0.h | f1.h << 16, w[1][e] = f0.mid | f1.mid << 16;
            }
            *reinterpret_cast<u32x4 *>(u) = w[0];
            *reinterpret_cast<u32x4 *>(u + 2 * 16 * 8) = w[1];
        }
}

// ----------------------------------------------------------------------------
// Launch 2.  A wave: 64 columns of x (dA) or dy (dB), one item's rows, the
// ranks in groups of 16 RT.
// ----------------------------------------------------------------------------
constexpr int kGradWaves = 4;
constexpr int kMaxSpan = 2048;
constexpr int kOutPitch = 272, kWaveTile = 16 * kOutPitch; // a wave's LDS: 32 rows of 128 bytes, or 16 rows of results
constexpr int kTileCols = 64 * kGradWaves; // columns of a workgroup

// The wave's column fragments of one window, from its LDS tile: 32 rows of 128
// bytes, unit 16 bytes, unit un of row q in slot un ^ (4 if q & 2): 4 rows
// of a fragment read then fall in distinct banks.
__device__ __forceinline__ int tile_at(int q, int un) { return q * 128 + ((un ^ ((q & 2) << 1)) << 4); }
// Rows 8 g .. + 7 of the 4 columns in half `half` of unit `un` (this lane's piece, of
// the 16 columns that 4 lanes name).
__device__ __forceinline__ bf16x8 tile_frag(const char *tile, int un, int half, int m, int g)
{
    u32x2 h[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) h[b] = read_tr(tile + tile_at(8 * g + 4 * b + (m >> 2), un) + 8 * half);
    return join8(h[0], h[1]);
}

// Operands of one window.  bf16: rows by 16 bytes, row (lane / 8) + 8 i, column
// 8 (lane % 8), to be turned through the tile; fp32: the column fragments
// themselves, in two halves of 16 rows.
template <int DT, int RT> struct GradOps {
    static constexpr int kHalves = DT == LORA_BF16 ? 1 : 2;
    typename Elem<DT>::F xf[kHalves][4];
    typename Elem<DT>::F uf[RT][Elem<DT>::kParts]; // fp32: of the two halves
};

struct GradSide {
    const void *src, *parts; // x and u (dA) or dy and v (dB)
    int64_t ld;
    int D;
};

// Four rank tiles (bf16): a window's 12 operands of u or v are three times the bytes of a
// wave's columns, and the same for the 4 waves, which fetch them once for all, by
// direct loads into LDS (each wave by itself: L1-bound, 16384 rows of rank 64 95 us, 74
// so).
template <int DT, int RT> constexpr bool kShareU = DT == LORA_BF16 && RT == 4;
constexpr int kShareBytes = 12 * kPieces; // one window; two lie in LDS

__device__ __forceinline__ void share_load(const BwdArgs &a, const GradSide &sd, int w, int rt0, uint32_t lds_byte, int wave, int lane)
{
    const char *win = static_cast<const char *>(sd.parts) + int64_t(w) * 3 * a.nt * kPieces + 16 * lane;
#pragma unroll
    for (int k = 0; k < 12 / kGradWaves; ++k) {
        const int piece = 12 / kGradWaves * wave + k, t = min(rt0 + (piece & 3), a.nt - 1); // past the last tile: not stored
        dma16(win + ((piece >> 2) * a.nt + t) * kPieces, lds_byte + uint32_t((w & 1) * kShareBytes + piece * kPieces));
    }
}

// WHOLE: all 64 columns lie in the row (not asked for by VEC).
template <int DT, bool VEC, bool WHOLE, int RT>
__device__ __forceinline__ void grad_load(GradOps<DT, RT> &o, const BwdArgs &a, const GradSide &sd, int begin, int end,
                                          int w, int c0, int rt0, const int32_t *tok, int lane)
{
    using E = Elem<DT>;
    using T = typename E::T;
    const int m = lane & 15, g = lane >> 4;
    const int base = w * kWin;
    if constexpr (!kShareU<DT, RT>) {
        const char *win = static_cast<const char *>(sd.parts) + int64_t(w) * E::kParts * a.nt * kPieces;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int t = min(rt0 + i, a.nt - 1); // past the last tile: not stored
#pragma unroll
            for (int q = 0; q < E::kParts; ++q)
                o.uf[i][q] = __builtin_bit_cast(typename E::F, load16(win + (q * a.nt + t) * kPieces, 16 * lane));
        }
    }
    auto token = [&](int p) { return tok[min(max(p, begin), end - 1) - begin]; };
    if constexpr (DT == LORA_BF16 && VEC) {
        const char *src = static_cast<const char *>(sd.src) + int64_t(c0) * 2;
        // past the row: columns that are not stored
        const uint32_t cc = c0 + 8 * (lane & 7) < sd.D ? 16 * (lane & 7) : 0, pitch = uint32_t(sd.ld * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o.xf[0][i] = __builtin_bit_cast(bf16x8, load16(src, uint32_t(token(base + (lane >> 3) + 8 * i)) * pitch + cc));
    } else if constexpr (DT == LORA_BF16) {
        const gptr<T> src = as_global<T>(sd.src);
        const int c = c0 + 8 * (lane & 7);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const gptr<T> row = src + int64_t(token(base + (lane >> 3) + 8 * i)) * sd.ld;
            if constexpr (WHOLE) o.xf[0][i] = __builtin_bit_cast(bf16x8, load16_any(row + c));
            else o.xf[0][i] = __builtin_bit_cast(bf16x8, load_row<DT>(row, c, sd.D));
        }
    } else {
        const gptr<T> src = as_global<T>(sd.src);
#pragma unroll
        for (int h = 0; h < o.kHalves; ++h)
#pragma unroll
            for (int e = 0; e < E::kVec; ++e) {
                const gptr<T> row = src + int64_t(token(base + 16 * h + E::kVec * g + e)) * sd.ld;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    o.xf[h][t][e] = row[min(c0 + 16 * t + m, sd.D - 1)];
                }
            }
    }
}

template <int DT, int RT>
__device__ __forceinline__ void grad_mma(GradOps<DT, RT> &o, floatx4 (&acc)[4][RT], int side, int begin, int end, int w,
                                         char *tile, const char *share, int lane)
{
    using E = Elem<DT>;
    using F = typename E::F;
    const int m = lane & 15, g = lane >> 4, base = w * kWin;
    if constexpr (kShareU<DT, RT>) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int q = 0; q < E::kParts; ++q)
                o.uf[i][q] = __builtin_bit_cast(F, *reinterpret_cast<const u32x4 *>(share + (w & 1) * kShareBytes + ((4 * q + i) * 64 + lane) * 16));
    }
    if (base < begin || base + kWin > end) { // rows outside: zero on both sides (wave-uniform)
        auto in = [&](int p) { return p >= begin && p < end; };
#pragma unroll
        for (int h = 0; h < o.kHalves; ++h) {
            u32x4 keep; // this lane's elements of the summed axis
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (DT == LORA_BF16)
                    keep[e] = (in(base + 8 * g + 2 * e) ? 0xffffu : 0u) | (in(base + 8 * g + 2 * e + 1) ? 0xffff0000u : 0u);
                else keep[e] = in(base + 16 * h + 4 * g + e) ? ~0u : 0u;
            }
            auto mask = [&](F &f) { f = __builtin_bit_cast(F, __builtin_bit_cast(u32x4, f) & keep); };
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int q = 0; q < E::kParts; ++q)
                    if (DT == LORA_BF16 || q == h) mask(o.uf[i][q]);
            if constexpr (DT == LORA_BF16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!in(base + (lane >> 3) + 8 * i)) o.xf[0][i] = bf16x8{};
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) mask(o.xf[h][t]);
            }
        }
    }
    if constexpr (DT == LORA_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x4 *>(tile + tile_at((lane >> 3) + 8 * i, lane & 7)) = __builtin_bit_cast(u32x4, o.xf[0][i]);
    }
#pragma unroll
    for (int h = 0; h < o.kHalves; ++h) {
        F xf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if constexpr (DT == LORA_BF16) xf[t] = tile_frag(tile, 2 * t + ((m & 3) >> 1), m & 1, m, g);
            else xf[t] = o.xf[h][t];
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int q = 0; q < E::kParts; ++q)
                if (DT == LORA_BF16 || q == h) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        acc[t][i] = side ? mma<DT>(o.uf[i][q], xf[t], acc[t][i]) : mma<DT>(xf[t], o.uf[i][q], acc[t][i]);
                }
    }
}

template <int DT, bool VEC, bool WHOLE, int RT>
__device__ __forceinline__ void grad_item(const BwdArgs &a, const GradSide &sd, int side, int begin, int end, int c0, int rt0,
                                          int r, float *dst, bool add, bool stream, bool idle, const int32_t *tok, char *tile,
                                          char *share, int lane)
{
    const int w1 = (end - 1) / kWin;
    floatx4 acc[4][RT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[t][i] = floatx4{};
    // Four rank tiles: the next window's loads are issued before the current one's
    // products (16384 rows of rank 64: 106 us, 118 without, before they were shared).  Fewer: more waves fit
    // instead (rank 16, 4096 rows: 17.2 us, 18.8 with).
    GradOps<DT, RT> o0;
    int w = begin / kWin;
    const int wave = uniform(threadIdx.x >> 6);
    const uint32_t share_at = uint32_t(uintptr_t((__attribute__((address_space(3))) char *)(share)));
    if (kShareU<DT, RT>) share_load(a, sd, w, rt0, share_at, wave, lane);
    grad_load<DT, VEC, WHOLE>(o0, a, sd, begin, end, w, c0, rt0, tok, lane);
    for (;;) {
        GradOps<DT, RT> o1;
        if (kShareU<DT, RT>) {
            // window w is there, every wave's part of it, and every wave is past the one before
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(wait_vm_lds0(0));
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (w < w1) share_load(a, sd, w + 1, rt0, share_at, wave, lane);
        }
        if (RT == 4 && w < w1) grad_load<DT, VEC, WHOLE>(o1, a, sd, begin, end, w + 1, c0, rt0, tok, lane);
        grad_mma(o0, acc, side, begin, end, w, tile, share, lane);
        if (++w > w1) break;
        if (RT == 4) o0 = o1;
        else grad_load<DT, VEC, WHOLE>(o0, a, sd, begin, end, w, c0, rt0, tok, lane);
    }
    if (idle) return;
    // dA (side 0): D rows are columns of x, D columns ranks; dB: D rows are ranks, D
    // columns columns of dy (rows of dB).  A lane's 4 sums are consecutive in the
    // gradient; 16 ranks x 64 columns turn in the wave's tile, so that they leave
    // with 16 bytes from each of 16 (dB: 4) adjacent lanes for a row.
    const int m = lane & 15, g = lane >> 4;
    const gfloat gdst = (gfloat)dst; // (generic stores would be waited for with the tile's reads)
    const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15) == 0 && ((side ? r : sd.D) & 3) == 0;
    auto put4 = [&](gfloat o, const floatx4 &v, int n) {
        if (n <= 0) return;
        if (vec) { // n is a multiple of 4
            const floatx4 f = add ? *(gfloatx4)o + v : v;
            // Gradients are not read here again, partial sums are (200 adapters of 5
            // rows, d_out 12288: 55 us with plain stores, 46 so; ranks up to 64 over 128
            // adapters, 72 and 82: plain there).  The two empty statements keep the
            // compiler from making the two stores one.
            if (stream) {
                asm volatile("");
                __builtin_nontemporal_store(f, (gfloatx4)o);
                asm volatile("");
            } else {
                *(gfloatx4)o = f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) o[e] = add ? o[e] + v[e] : v[e];
        }
    };
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int j0 = 16 * (rt0 + i);
        if (side == 0) {
#pragma unroll
            for (int t = 0; t < 4; ++t) *reinterpret_cast<floatx4 *>(tile + m * kOutPitch + 4 * (16 * t + 4 * g)) = acc[t][i];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int j = 4 * h + g, c = c0 + 4 * m;
                const floatx4 v = *reinterpret_cast<const floatx4 *>(tile + j * kOutPitch + 16 * m);
                if (j0 + j < r) put4(gdst + int64_t(j0 + j) * sd.D + c, v, sd.D - c);
            }
        } else {
            // rows of 64 bytes, unit un of row q in slot un ^ (q / 2 % 4)
#pragma unroll
            for (int t = 0; t < 4; ++t) *reinterpret_cast<floatx4 *>(tile + (16 * t + m) * 64 + ((g ^ ((m >> 1) & 3)) << 4)) = acc[t][i];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int q = 16 * h + (lane >> 2), un = lane & 3, j = j0 + 4 * un;
                const floatx4 v = *reinterpret_cast<const floatx4 *>(tile + q * 64 + ((un ^ ((q >> 1) & 3)) << 4));
                if (c0 + q < sd.D) put4(gdst + int64_t(c0 + q) * r + j, v, r - j);
            }
        }
    }
}

// RT: rank tiles that a wave holds (the plan's largest rank, at most 4: higher
// ranks are `groups` of 64, a workgroup each).
template <int DT, bool VEC, int RT>
__device__ __forceinline__ void grad_unit(const BwdArgs &a, int id, char *tiles_lds, int32_t *tok, char *share)
{
    const int tl = id % a.tiles, group = id / a.tiles % a.groups;
    const Item it = a.items[id / a.tiles / a.groups];
    if (64 * group >= it.rank) return;
    const int side = tl >= a.tiles_A;
    const uint64_t grad = side ? it.grad_B : it.grad_A;
    if (!grad) return; // this adapter's gradient is not wanted
    for (int i = threadIdx.x; i < it.end - it.begin; i += kGradWaves * 64) tok[i] = a.perm[it.begin + i];
    __syncthreads();
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = it.rank;
    const GradSide sd = side ? GradSide{a.dy, a.vt, a.lddy, a.d_out} : GradSide{a.x, a.ut, a.ldx, a.d_in};
    int c0 = (side ? tl - a.tiles_A : tl) * (64 * kGradWaves) + 64 * wave;
    const int left = r - 64 * group;
    // a wave past the columns does its part of shared windows (on the first columns,
    // which it does not store)
    const bool idle = c0 >= sd.D;
    if (idle && !(DT == LORA_BF16 && RT >= 4 && left > 32)) return;
    if (idle) c0 = 0;
    float *dst = reinterpret_cast<float *>(grad);
    bool add = a.accumulate;
    if (it.slot >= 0) {
        dst = a.part + it.slot * a.part_stride + (side ? int64_t(r) * a.d_in : 0);
        add = false;
    }
    char *tile = tiles_lds + wave * kWaveTile;
    auto ranks = [&](auto whole) {
        constexpr bool W = decltype(whole)::value;
        if (RT >= 4 && left > 32)
            grad_item<DT, VEC, W, RT >= 4 ? 4 : 1>(a, sd, side, it.begin, it.end, c0, 4 * group, r, dst, add, RT < 4 && it.slot < 0, idle, tok, tile, share, lane);
        else if (RT >= 2 && left > 16)
            grad_item<DT, VEC, W, RT >= 2 ? 2 : 1>(a, sd, side, it.begin, it.end, c0, 4 * group, r, dst, add, RT < 4 && it.slot < 0, idle, tok, tile, share, lane);
        else grad_item<DT, VEC, W, 1>(a, sd, side, it.begin, it.end, c0, 4 * group, r, dst, add, RT < 4 && it.slot < 0, idle, tok, tile, share, lane);
    };
    if constexpr (VEC || DT == LORA_F32) ranks(std::true_type{});
    else if (c0 + 64 <= sd.D) ranks(std::true_type{});
    else ranks(std::false_type{});
}

// ----------------------------------------------------------------------------
// dx.  A wave: 64 columns, the up to 16 RB rows of a block or a chunk.
// ----------------------------------------------------------------------------
constexpr int kDxWaves = kGradWaves;

// JOIN: dx is not read but set, to the sum of the parts of a base product plus u A,
// for every row of the plan, by blocks of 16 rows (those past the plan's: rows
// without an adapter).
template <int DT, bool VEC, bool JOIN, int RB>
__device__ __forceinline__ void dx_unit(const BwdArgs &a, int id, char *tiles_lds)
{
    static_assert(RB == 1 || (RB == 4 && !JOIN), "a block or a chunk");
    using E = Elem<DT>;
    using T = typename E::T;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), m = lane & 15, g = lane >> 4;
    const int unit = id / a.tiles_x;
    const int c0 = int(id % a.tiles_x) * (64 * kDxWaves) + 64 * wave;
    if (c0 >= a.d_in) return;
    int r = 0, p0 = 0, n = 0;
    const void *A = nullptr;
    auto take = [&](const auto *d) {
        r = d->rank, n = d->n, p0 = d->p0;
        A = reinterpret_cast<const void *>(d->A);
    };
    if constexpr (RB == 4) take(a.chunk + unit);
    else if (!JOIN || unit < a.nblk) take(a.blk + unit);
    else p0 = a.Tp + 16 * (unit - a.nblk), n = min(16, a.T - p0);
    char *tile = tiles_lds + wave * kWaveTile;
    // operands of 16 ranks: u of 4 row blocks, and A by rows (bf16: rank
    // (lane / 8) + 8 i, column 8 (lane % 8)) or by column fragments (fp32)
    struct Ops {
        typename E::F uf[RB], af[4];
    };
    // u of row m of block i (past n: not stored), where launch 1 put its position
    uint32_t uoff[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int p = p0 + min(16 * i + m, n - 1);
        uoff[i] = uint32_t((p >> 4) - (p0 >> 4)) * uint32_t(a.nt * kPieces) + uint32_t(g * 16 + (p & 15)) * 16;
    }
    const char *ur = a.ur + int64_t(p0 >> 4) * a.nt * kPieces;
    const bool whole = c0 + 64 <= a.d_in; // every piece of this wave lies in its row
    const uint32_t acol = c0 + 8 * (lane & 7) < a.d_in ? 16 * (lane & 7) : 0;
    auto load = [&](Ops &o, int j0) {
#pragma unroll
        for (int i = 0; i < RB; ++i) o.uf[i] = __builtin_bit_cast(typename E::F, load16(ur + (j0 >> 4) * kPieces, uoff[i]));
        if constexpr (DT == LORA_BF16) {
            const char *base = static_cast<const char *>(A) + (int64_t(j0) * a.d_in + c0) * 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = (lane >> 3) + 8 * i;
                const uint32_t row = uint32_t(j0 + j < r ? j : 0) * uint32_t(a.d_in * 2);
                u32x4 w;
                if constexpr (VEC) w = load16(base, row + acol);
                else if (whole) w = load16_any(as_global<char>(base) + (row + acol)); // wave-uniform
                else w = load_row<DT>(as_global<T>(base + row), 8 * (lane & 7), a.d_in - c0);
                if (j0 + j >= r) w = u32x4{};
                o.af[i] = __builtin_bit_cast(bf16x8, w);
            }
        } else {
            const gptr<T> Af = as_global<T>(A);
#pragma unroll
            for (int e = 0; e < E::kVec; ++e) {
                const int j = j0 + 4 * g + e;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const T w = Af[int64_t(j < r ? j : r - 1) * a.d_in + min(c0 + 16 * t + m, a.d_in - 1)];
                    o.af[t][e] = j < r ? w : 0.f;
                }
            }
        }
    };
    floatx4 acc[4][RB]; // column tile, row block
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[t][i] = floatx4{};
    auto products = [&](const Ops &o, int s) {
        typename E::F af[4];
        if constexpr (DT == LORA_BF16) {
            char *tl = tile + (s & 1) * 2048;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<u32x4 *>(tl + tile_at((lane >> 3) + 8 * i, lane & 7)) = __builtin_bit_cast(u32x4, o.af[i]);
            // k slots of lane groups 0, 1 meet u's hi parts, 2, 3 its lo parts, of the same ranks
#pragma unroll
            for (int t = 0; t < 4; ++t) af[t] = tile_frag(tl, (t >> 1) * 4 + (m & 3), t & 1, m, g & 1);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) af[t] = o.af[t];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < RB; ++i) acc[t][i] = mma<DT>(af[t], o.uf[i], acc[t][i]);
    };
    // The first operands, then what is added to (needed last), then each next step's
    // operands before the products of the current one.  Results leave through the
    // wave's tile by rows: bf16 rows (lane / 8) + 8 h of a block, 8 columns at
    // 8 (lane % 8); fp32 and JOIN rows (lane / 16) + 4 h, 4 columns at 4 (lane % 16).
    constexpr bool kBy8 = DT == LORA_BF16 && !JOIN;
    constexpr int H = kBy8 ? 2 : 4, kC = kBy8 ? 8 : 4;
    const int orow = kBy8 ? lane >> 3 : lane >> 4, oc = c0 + kC * (kBy8 ? lane & 7 : lane & 15);
    Ops o0, o1;
    if (!JOIN || r) load(o0, 0);
    T *out[RB][H];
    u32x4 y[RB][H];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int h = 0; h < H; ++h) {
            out[i][h] = static_cast<T *>(a.dx) + int64_t(a.perm[p0 + min(16 * i + orow + (16 / H) * h, n - 1)]) * a.lddx;
            if constexpr (!JOIN) {
                const gptr<T> row = as_global<T>(out[i][h]);
                if constexpr (VEC) y[i][h] = *(gptr<u32x4>)(row + (oc < a.d_in ? oc : 0)); // past d_in: not stored
                else if (whole) y[i][h] = load16_any(row + oc);
                else y[i][h] = load_row<DT>(row, oc, a.d_in);
            }
        }
    floatx4 base[H]; // JOIN: the sums of the parts
    if constexpr (JOIN) {
#pragma unroll
        for (int h = 0; h < H; ++h) base[h] = floatx4{};
        const float *q = a.joins + int64_t(p0) * a.d_in + (oc < a.d_in ? oc : 0);
        for (int k = 0; k < a.splits; ++k, q += int64_t(a.T) * a.d_in)
#pragma unroll
            for (int h = 0; h < H; ++h) base[h] += *reinterpret_cast<const floatx4 *>(q + int64_t(min(orow + 4 * h, n - 1)) * a.d_in);
    }
    for (int j0 = 0; !JOIN || r;) {
        if (j0 + 16 < r) load(o1, j0 + 16);
        products(o0, 0);
        if ((j0 += 16) >= r) break;
        if (j0 + 16 < r) load(o0, j0 + 16);
        products(o1, 1);
        if ((j0 += 16) >= r) break;
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        // rows of kOutPitch bytes: 16 rows' equal columns fall in distinct banks
#pragma unroll
        for (int t = 0; t < 4; ++t)
            *reinterpret_cast<floatx4 *>(tile + m * kOutPitch + 4 * (DT == LORA_BF16 ? col<DT>(g, 4 * t) : 16 * t + 4 * g)) = acc[t][i];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int row = orow + (16 / H) * h;
            const floatx4 *f = reinterpret_cast<const floatx4 *>(tile + row * kOutPitch + 4 * (oc - c0));
            if (16 * i + row >= n || oc >= a.d_in) continue;
            if constexpr (kBy8) {
                const floatx4 lo = f[0], hi = f[1];
                u32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f0 = e < 2 ? lo[2 * e] : hi[2 * e - 4], f1 = e < 2 ? lo[2 * e + 1] : hi[2 * e - 3];
                    o[e] = pack_bf16x2(bf16_to_f32(y[i][h][e] & 0xffffu) + f0, bf16_to_f32(y[i][h][e] >> 16) + f1);
                }
                if constexpr (VEC) *reinterpret_cast<u32x4 *>(out[i][h] + oc) = o;
                else if (whole) *reinterpret_cast<u32x4_any *>(out[i][h] + oc) = o;
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (oc + e < a.d_in) out[i][h][oc + e] = uint16_t(o[e >> 1] >> (16 * (e & 1)));
            } else if constexpr (JOIN) { // d_in is a multiple of 8
                const floatx4 v = base[h] + f[0];
                *reinterpret_cast<u32x2 *>(out[i][h] + oc) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            } else {
                const floatx4 v = __builtin_bit_cast(floatx4, y[i][h]) + f[0];
                if constexpr (VEC) *reinterpret_cast<floatx4 *>(out[i][h] + oc) = v;
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (oc + e < a.d_in) out[i][h][oc + e] = v[e];
            }
        }
    }
}

// Launch 2: the gradients' workgroups, then dx's (they read the same u).
// Waves per SIMD that the registers allow without spills.
constexpr int out_waves(int dt, bool vec, int rt)
{
    if (dt == LORA_F32) return rt == 1 ? 4 : rt == 2 ? 3 : 1;
    return rt == 1 ? 5 : rt == 2 ? (vec ? 4 : 3) : (vec ? 2 : 1);
}
template <int DT, bool VEC, int RT>
__global__ __launch_bounds__(kGradWaves * 64, out_waves(DT, VEC, RT)) void bwd_out_kernel(BwdArgs a)
{
    __shared__ __attribute__((aligned(16))) char tiles_lds[kGradWaves * kWaveTile];
    __shared__ int32_t tok[kMaxSpan];
    __shared__ __attribute__((aligned(16))) char share[kShareU<DT, RT> ? 2 * kShareBytes : 16];
    if (int(blockIdx.x) < a.ngrad) grad_unit<DT, VEC, RT>(a, blockIdx.x, tiles_lds, tok, share);
    else if (RT >= 4 && a.chunks) dx_unit<DT, VEC, false, RT >= 4 ? 4 : 1>(a, int(blockIdx.x) - a.ngrad, tiles_lds);
    else dx_unit<DT, VEC, false, 1>(a, int(blockIdx.x) - a.ngrad, tiles_lds);
}

// Launch 3: gradient = sum of a split segment's slots, in slot order.
__global__ __launch_bounds__(256) void bwd_reduce_kernel(BwdArgs a)
{
    const Split sp = a.segsplits[blockIdx.y];
    const lora_seg_desc *sd = a.seg + sp.seg;
    const int64_t nA = int64_t(sd->rank) * a.d_in, n = nA + int64_t(sd->rank) * a.d_out;
    const uint64_t gA = a.grad_A ? a.grad_A[sd->adapter] : 0, gB = a.grad_B ? a.grad_B[sd->adapter] : 0;
    for (int64_t e = 4 * (int64_t(blockIdx.x) * 256 + threadIdx.x); e < n; e += 4 * int64_t(gridDim.x) * 256) {
        // slots start at multiples of 4; a group of 4 may reach from dA into dB
        const bool wA = e < nA && gA, wB = e + 3 >= nA && gB;
        if (!wA && !wB) continue;
        const float *src = a.part + sp.slot0 * a.part_stride + e;
        floatx4 sum = floatx4{};
        for (int q = 0; q < sp.count; ++q) sum += *reinterpret_cast<const floatx4 *>(src + q * a.part_stride);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = e + i;
            if (k >= n) break;
            const uint64_t base = k < nA ? gA : gB;
            if (!base) continue;
            float *dst = reinterpret_cast<float *>(base) + (k < nA ? k : k - nA);
            *dst = a.accumulate ? *dst + sum[i] : sum[i];
        }
    }
}

// The last launch of the fused layer's backward.
template <bool VEC> __global__ __launch_bounds__(kDxWaves * 64, 4) void bwd_join_kernel(BwdArgs a)
{
    __shared__ __attribute__((aligned(16))) char tiles_lds[kDxWaves * kWaveTile];
    dx_unit<LORA_BF16, VEC, true, 1>(a, blockIdx.x, tiles_lds);
}

// Sorted positions of one span, a power of two of windows.  Items of the whole
// batch are wanted, since a segment over k spans costs k partial sums and a launch:
// the widest span (up to kLong rows, 16 windows one after the other) that still
// gives the chip kEnough workgroups.  At most kSpans spans, so that the bytes of
// partial sums stay bounded, and none that a few rows would need.
constexpr int kMinSpan = 64, kLong = 512, kSpans = 16, kEnough = 1024;
int span_of(int64_t rows, int64_t segments, int64_t wgs_per_item)
{
    if (rows <= 256) return 256;
    int span = kMinSpan;
    while (span < kMaxSpan && rows / span > kSpans) span *= 2;
    while (span < kLong && (segments + rows / (2 * span)) * wgs_per_item >= kEnough) span *= 2;
    return span;
}
// Borders of spans inside `rows` sorted positions, at most, for any span that
// span_of gives for them or for fewer.
size_t most_borders(size_t rows) { return std::max(std::min(rows / kMinSpan, size_t(kSpans)), rows / kMaxSpan); }

struct Layout {
    size_t ut, vt, ur, items, splits, part, bytes;
    int64_t part_stride;
};

// For up to `rows` adapted tokens; the partial sums of a segment cut into k
// items cross k - 1 span borders, so there are at most two for each border.
Layout layout_of(int32_t rows, int32_t d_in, int32_t d_out, int32_t max_rank)
{
    Layout l{};
    const size_t r16 = size_t(max_rank + 15) / 16 * 16, n = size_t(rows);
    const size_t windows = (n + kWin - 1) / kWin;
    l.ut = 0;
    l.vt = l.ut + windows * 3 * (r16 / 16) * kPieces; // three bf16 parts; fp32 takes two thirds
    l.ur = l.vt + windows * 3 * (r16 / 16) * kPieces;
    l.items = l.ur + (n + 15) / 16 * (r16 / 16) * kPieces;
    const size_t borders = most_borders(n);
    l.splits = l.items + up256((n + borders) * sizeof(Item));
    l.part = l.splits + up256(borders * sizeof(Split));
    l.part_stride = (int64_t(max_rank) * (int64_t(d_in) + d_out) + 3) / 4 * 4;
    l.bytes = l.part + 2 * borders * size_t(l.part_stride) * 4;
    return l;
}

int checked(const char *what)
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? LORA_OK : fail(LORA_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

template <int DT, bool VEC> int run_shrink(hipStream_t s, const BwdArgs &a, unsigned nside, bool ranks8, const QuantCall *quant)
{
    int st = LORA_OK;
    // The ring where 64-row workgroups fill the chip and are mostly whole: d 4096,
    // ring / blocks of 16 rows, us.  Rank 64: 4096 rows 41 / 41, 8192 54 / 66, 16384
    // 98 / 125, 32768 159 / 231; rank 32: 44 / 42, 84 / 80, 146 / 151 from 8192 rows;
    // rank 16: 78 / 67 for 16384.
    if (DT == LORA_BF16 && VEC && ranks8 && a.nt > 2 && int64_t(a.nchunk) * nside >= 256 && a.Tp / a.nchunk >= 32) {
        const dim3 grid((unsigned(a.nchunk) + 7) / 8 * nside * a.groups * 8 + 8), block(256);
        if (quant) st = launch_quantize(s, *quant);
        if (st) return st;
        launch_kernel(bwd_shrink_ring_kernel, grid, block, 0, s, a);
        return checked("backward shrink");
    }
    const dim3 grid((unsigned(a.nblk) + 7) / 8 * nside * a.groups * 8 + 8), block(kShrinkWaves * 64);
    if (quant) {
        int64_t both;
        const QuantAlong along = quant_along(*quant, grid.x, kShrinkWaves / 4, &both);
        if (DT == LORA_BF16 && VEC && quant->pad && both <= most_workgroups(kShrinkWaves * 64)) {
            const dim3 all{unsigned(both)};
            if (a.nt <= 1) launch_kernel(bwd_shrink_quantize_kernel<1>, all, block, 0, s, a, along);
            else if (a.nt <= 2) launch_kernel(bwd_shrink_quantize_kernel<2>, all, block, 0, s, a, along);
            else launch_kernel(bwd_shrink_quantize_kernel<4>, all, block, 0, s, a, along);
            return checked("backward shrink and quantize");
        }
        st = launch_quantize(s, *quant);
        if (st) return st;
    }
    if (a.nt <= 1) launch_kernel(bwd_shrink_kernel<DT, VEC, 1>, grid, block, 0, s, a);
    else if (a.nt <= 2) launch_kernel(bwd_shrink_kernel<DT, VEC, 2>, grid, block, 0, s, a);
    else launch_kernel(bwd_shrink_kernel<DT, VEC, 4>, grid, block, 0, s, a);
    return checked("backward shrink");
}
template <int DT, bool VEC> void run_out(hipStream_t s, const BwdArgs &a, dim3 grid)
{
    const dim3 block(kGradWaves * 64);
    if (a.nt <= 1) launch_kernel(bwd_out_kernel<DT, VEC, 1>, grid, block, 0, s, a);
    else if (a.nt <= 2) launch_kernel(bwd_out_kernel<DT, VEC, 2>, grid, block, 0, s, a);
    else launch_kernel(bwd_out_kernel<DT, VEC, 4>, grid, block, 0, s, a);
}

} // namespace

size_t sgmv_backward_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t max_rank)
{
    return layout_of(T, d_in, d_out, max_rank).bytes;
}

static BwdArgs make_args(const BackwardArgs &b, const PlanView &p, const Layout &l, void *ws)
{
    const lora_plan_header *h = p.h;
    char *w = static_cast<char *>(ws);
    BwdArgs a{};
    a.x = b.x;
    a.ldx = b.ldx;
    a.dy = b.dy;
    a.lddy = b.lddy;
    a.d_in = b.d_in;
    a.d_out = b.d_out;
    a.seg = reinterpret_cast<const lora_seg_desc *>(p.dev + h->seg_offset);
    a.blk = reinterpret_cast<const lora_blk_desc *>(p.dev + h->blk_offset);
    a.chunk = reinterpret_cast<const lora_chunk_desc *>(p.dev + h->chunk_offset);
    a.perm = reinterpret_cast<const int32_t *>(p.dev + h->perm_offset);
    a.S = h->num_segments;
    a.nblk = h->num_blocks;
    a.nchunk = h->num_chunks;
    a.nt = (h->max_rank + 15) / 16;
    a.ut = w + l.ut;
    a.vt = w + l.vt;
    a.ur = w + l.ur;
    a.items = reinterpret_cast<Item *>(w + l.items);
    a.splits = 1;
    a.segsplits = reinterpret_cast<Split *>(w + l.splits);
    a.part = reinterpret_cast<float *>(w + l.part);
    a.part_stride = l.part_stride;
    a.grad_A = b.grad_A;
    a.grad_B = b.grad_B;
    a.accumulate = b.accumulate;
    a.dx = b.dx;
    a.lddx = b.lddx;
    a.tiles_x = (a.d_in + kTileCols - 1) / kTileCols;
    a.T = h->num_tokens;
    a.Tp = h->num_sorted;
    return a;
}

int launch_sgmv_backward(hipStream_t s, const BackwardArgs &b, const PlanView &p, void *ws, const uint16_t **u_rows,
                         int64_t *ldu, const QuantCall *quant)
{
    const lora_plan_header *h = p.h;
    const Layout l = layout_of(h->num_sorted, b.d_in, b.d_out, h->max_rank);
    BwdArgs a = make_args(b, p, l, ws);
    a.sides = (b.grad_B ? 1 : 0) | (b.grad_A || b.dx || u_rows ? 2 : 0);
    if (u_rows) {
        *u_rows = reinterpret_cast<const uint16_t *>(a.ur);
        *ldu = int64_t(a.nt) * kPieces / 2;
    }
    if (!a.sides) return LORA_OK;
    a.tiles_A = a.grad_A ? (a.d_in + kTileCols - 1) / kTileCols : 0;
    a.tiles = a.tiles_A + (a.grad_B ? (a.d_out + kTileCols - 1) / kTileCols : 0);
    a.groups = (a.nt + 3) / 4;
    a.span = span_of(h->num_sorted, h->num_segments, int64_t(a.tiles) * a.groups);
    const lora_seg_desc *hs = reinterpret_cast<const lora_seg_desc *>(reinterpret_cast<const char *>(h) + h->seg_offset);
    bool ranks8 = true;
    for (int i = 0; i < h->num_segments; ++i) {
        const int n = (hs[i].start + hs[i].len - 1) / a.span - hs[i].start / a.span + 1;
        a.nitems += n;
        a.nsplit += n > 1;
        ranks8 = ranks8 && hs[i].rank % 8 == 0;
    }

    if (a.nsplit > 65535) return fail(LORA_ERR_ARG, "backward: %d segments over several spans (> 65535)", a.nsplit);

    const int64_t ngrad = int64_t(a.nitems) * a.tiles * a.groups;
    // dx by chunks of 64 rows where they fill the chip (16384 rows of rank 64: launch
    // 2 took 149 us so, 217 by blocks; 517 rows of ranks to 100: 19, 14 by blocks),
    // and not beside gradients of one or two rank tiles, whose launch would take
    // twice its registers (4096 rows of rank 16: 70 us, 29 by blocks).
    a.chunks = a.nt >= 3 && int64_t(a.nchunk) * a.tiles_x >= 512;
    const int64_t ndx = a.dx ? int64_t(a.chunks ? a.nchunk : a.nblk) * a.tiles_x : 0;
    // launch 1: at most (blocks + 7 and 8 more) workgroups for a side and group of ranks
    if (ngrad + ndx > most_workgroups(kGradWaves * 64) ||
        (int64_t(a.nblk) + 15) * 2 * a.groups > most_workgroups(kShrinkWaves * 64))
        return fail(LORA_ERR_ARG, "backward: too many work items");
    a.ngrad = int(ngrad);

    const bool bf16 = b.dtype == LORA_BF16;
    const bool vec = b.vec_x && b.vec_dy && (!a.dx || b.vec_dx);
    const unsigned nside = a.sides == 3 ? 2 : 1;
    int st;
    if (bf16 && vec) st = run_shrink<LORA_BF16, true>(s, a, nside, ranks8, quant);
    else if (bf16) st = run_shrink<LORA_BF16, false>(s, a, nside, ranks8, quant);
    else if (vec) st = run_shrink<LORA_F32, true>(s, a, nside, ranks8, quant);
    else st = run_shrink<LORA_F32, false>(s, a, nside, ranks8, quant);
    if (st || ngrad + ndx == 0) return st;
    const dim3 grid{unsigned(ngrad + ndx)};
    if (bf16 && vec) run_out<LORA_BF16, true>(s, a, grid);
    else if (bf16) run_out<LORA_BF16, false>(s, a, grid);
    else if (vec) run_out<LORA_F32, true>(s, a, grid);
    else run_out<LORA_F32, false>(s, a, grid);
    if ((st = checked("backward gradient"))) return st;
    if (a.tiles && a.nsplit) {
        const int64_t units = (l.part_stride / 4 + 255) / 256;
        launch_kernel(bwd_reduce_kernel, dim3(unsigned(std::min<int64_t>(units, 1024)), unsigned(a.nsplit)), dim3(256), 0, s, a);
        return checked("backward reduce");
    }
    return LORA_OK;
}

static int64_t join_workgroups(const BackwardArgs &b, const lora_plan_header *h)
{
    return (int64_t(h->num_blocks) + (h->num_tokens - h->num_sorted + 15) / 16) * ((b.d_in + kTileCols - 1) / kTileCols);
}
int check_dx_join(const BackwardArgs &b, const PlanView &p)
{
    if (join_workgroups(b, p.h) > most_workgroups(kDxWaves * 64)) return fail(LORA_ERR_ARG, "backward: too many dx tiles");
    return LORA_OK;
}

int launch_dx_join(hipStream_t s, const BackwardArgs &b, const PlanView &p, void *ws, const float *parts, int splits)
{
    const lora_plan_header *h = p.h;
    BwdArgs a = make_args(b, p, layout_of(h->num_sorted, b.d_in, b.d_out, h->max_rank), ws);
    a.joins = parts;
    a.splits = splits;
    const int st = check_dx_join(b, p);
    if (st) return st;
    const dim3 grid{unsigned(join_workgroups(b, h))}, block(kDxWaves * 64);
    if (b.vec_dx) launch_kernel(bwd_join_kernel<true>, grid, block, 0, s, a);
    else launch_kernel(bwd_join_kernel<false>, grid, block, 0, s, a);
    return checked("backward join");
}

} // namespace lora
