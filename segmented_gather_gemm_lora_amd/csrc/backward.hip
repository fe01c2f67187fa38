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
//     one more workgroup lists the work items of launch 2;
//  2. bwd_grad_kernel: dA and dB.  An item is one segment's rows inside one
//     span of `span` sorted positions; an item covers 256 columns of x or dy per
//     workgroup.  A segment inside one span is written at once; the sums of a
//     segment that crosses spans go to the workspace;
//  3. bwd_reduce_kernel: adds those partial sums in span order (a fixed order:
//     the gradients do not change from run to run);
//  4. bwd_dx_kernel: dx, one workgroup per 64-row chunk and 256 columns.
//
// The transposed operands.  MFMA wants, in each lane, consecutive elements of
// the summed axis.  x, dy (summed over rows for dA, dB), A (summed over its
// rows for dx) and B (summed over its rows for u) are contiguous along the
// other axis.  Rows are loaded with 16 bytes per lane into a wave's own LDS
// tile and read back with ds_read_b64_tr_b16, which hands lane i of every 16
// lanes column i of 4 rows.  fp32 operands go to v_mfma_f32_16x16x4_f32, which
// takes one element per lane: they are loaded where they are needed.
//
// Precision.  u and v are fp32 sums.  For dA and dB they are fed to bf16 MFMA
// as three bf16 parts (hi + mid + lo, 24 significant bits: all of an fp32), so the
// fp32 gradients keep fp32 accuracy; for dx, which is rounded to bf16, as two
// (16 significant bits, as in the forward's expand).  fp32 calls multiply
// exactly.
#include "internal.h"

#include <algorithm>

namespace lora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <typename T> using gptr = const __attribute__((address_space(1))) T *;
template <typename T> __device__ __forceinline__ gptr<T> as_global(const void *p) { return (gptr<T>)(p); }

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint32_t f32_to_bf16(float f)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); // nearest even, NaN stays NaN
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

// Lane i of every 16 lanes gives the address of 4 elements of row i / 4, at
// column group i % 4, and receives column i of the 4 rows.
__device__ __forceinline__ u32x2 read_tr(const char *lds)
{
    typedef __attribute__((address_space(3))) s16x4 lds4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(lds)));
}
__device__ __forceinline__ bf16x8 join8(u32x2 a, u32x2 b)
{
    return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
}

constexpr int kWin = 32; // sorted positions of one step over rows; u and v are stored in windows of it

template <int DT> struct Elem;
template <> struct Elem<LORA_BF16> {
    using T = uint16_t;
    using F = bf16x8;              // operand of one MFMA step
    static constexpr int kVec = 8; // elements of the summed axis per lane
    static constexpr int kStep = 32;
    static constexpr int kParts = 3;  // u and v for dA, dB
    static constexpr int kPart = 2;   // bytes of a part's element
};
template <> struct Elem<LORA_F32> {
    using T = float;
    using F = floatx4;
    static constexpr int kVec = 4;
    static constexpr int kStep = 16;
    static constexpr int kParts = 1;
    static constexpr int kPart = 4;
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
    int32_t seg;
    int32_t begin, end; // sorted positions
    int32_t slot;       // partial sums' place, -1: the gradient itself
};
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
    int r16;        // largest rank, rounded up to 16
    char *ut, *vt;  // u and v in windows: [window][part][rank][32 positions]
    char *ur;       // u in rows: bf16 [position][16 ranks hi, 16 ranks lo ...], fp32 [position][ranks]
    Item *items;
    Split *splits;
    float *part;
    int64_t part_stride;
    int span, nitems, nsplit;
    const uint64_t *grad_A, *grad_B;
    int accumulate;
    int sides; // bit 0: v is wanted, bit 1: u
    void *dx;
    int64_t lddx;
};

// ----------------------------------------------------------------------------
// Launch 1.  One workgroup: 16 rows, all ranks, one side.
// Side 0: v, K = d_in, W = A (row j is rank j, contiguous along K).
// Side 1: u, K = d_out, W = B (row k holds the ranks).
// ----------------------------------------------------------------------------
template <int DT, bool VEC>
__device__ __forceinline__ typename Elem<DT>::F load_row(gptr<typename Elem<DT>::T> row, int k, int K)
{
    using E = Elem<DT>;
    typename E::F f;
    if constexpr (VEC) { // K is a multiple of kVec
        const int kk = k < K ? k : K - E::kVec;
        f = __builtin_bit_cast(typename E::F, *(gptr<u32x4>)(row + kk));
        if (k >= K) f = typename E::F{};
    } else {
#pragma unroll
        for (int e = 0; e < E::kVec; ++e) {
            const typename E::T w = row[k + e < K ? k + e : K - 1];
            if constexpr (DT == LORA_BF16) f[e] = __builtin_bit_cast(__bf16, uint16_t(k + e < K ? w : 0));
            else f[e] = k + e < K ? w : 0.f;
        }
    }
    return f;
}

// Column j of rows k .. k + kVec - 1 of B (row pitch r), element by element.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::F load_col(gptr<typename Elem<DT>::T> B, int r, int j, int k, int K)
{
    using E = Elem<DT>;
    typename E::F f;
    const int jj = j < r ? j : r - 1; // past r: a column that nothing reads
#pragma unroll
    for (int e = 0; e < E::kVec; ++e) {
        const typename E::T w = B[int64_t(k + e < K ? k + e : K - 1) * r + jj];
        if constexpr (DT == LORA_BF16) f[e] = __builtin_bit_cast(__bf16, uint16_t(k + e < K ? w : 0));
        else f[e] = k + e < K ? w : 0.f;
    }
    return f;
}

// Work items: the segments cut at multiples of `span`.  One workgroup.
__device__ void list_items(const BwdArgs &a, int *scan, int nthreads)
{
    const int tid = threadIdx.x;
    int item0 = 0, slot0 = 0, split0 = 0;
    for (int s0 = 0; s0 < a.S; s0 += nthreads) {
        const int s = s0 + tid;
        int start = 0, end = 0, n = 0;
        if (s < a.S) {
            start = a.seg[s].start;
            end = start + a.seg[s].len;
            n = (end - 1) / a.span - start / a.span + 1;
        }
        const int ns = n > 1 ? n : 0, nq = n > 1 ? 1 : 0;
        int *sc[3] = {scan, scan + nthreads, scan + 2 * nthreads};
        int val[3] = {n, ns, nq};
        for (int q = 0; q < 3; ++q) sc[q][tid] = val[q];
        __syncthreads();
        for (int d = 1; d < nthreads; d <<= 1) {
            int add[3];
            for (int q = 0; q < 3; ++q) add[q] = tid >= d ? sc[q][tid - d] : 0;
            __syncthreads();
            for (int q = 0; q < 3; ++q) sc[q][tid] += add[q];
            __syncthreads();
        }
        const int it = item0 + sc[0][tid] - n, sl = slot0 + sc[1][tid] - ns, sp = split0 + sc[2][tid] - nq;
        for (int i = 0; i < n; ++i) {
            const int b = i == 0 ? start : (start / a.span + i) * a.span;
            const int e = i == n - 1 ? end : (start / a.span + i + 1) * a.span;
            a.items[it + i] = Item{s, b, e, n > 1 ? sl + i : -1};
        }
        if (nq) a.splits[sp] = Split{s, sl, n, 0};
        item0 += sc[0][nthreads - 1];
        slot0 += sc[1][nthreads - 1];
        split0 += sc[2][nthreads - 1];
        __syncthreads();
    }
}

constexpr int kShrinkWaves = 8;

template <int DT, bool VEC, int RT>
__global__ __launch_bounds__(kShrinkWaves * 64) void bwd_shrink_kernel(BwdArgs a)
{
    using E = Elem<DT>;
    using T = typename E::T;
    using F = typename E::F;
    constexpr int W = kShrinkWaves, NS = RT >= 4 ? 2 : 4;
    constexpr int kTile = 1024 * RT; // LDS of one step's B tile: 32 rows of 16 RT ranks
    constexpr int kRed = W * RT * 1024, kTiles = W * 2 * kTile;
    constexpr int kScan = 3 * 4 * W * 64;
    constexpr int kLds = kRed > kTiles ? kRed : kTiles;
    __shared__ __attribute__((aligned(16))) char lds[kLds > kScan ? kLds : kScan];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int m = lane & 15, g = lane >> 4;
    const int nside = a.sides == 3 ? 2 : 1;
    if (int(blockIdx.x) == a.nblk * nside) {
        list_items(a, reinterpret_cast<int *>(lds), W * 64);
        return;
    }
    const int blk = blockIdx.x / nside;
    const int side = a.sides == 3 ? int(blockIdx.x) % 2 : a.sides - 1;
    const lora_blk_desc *d = a.blk + blk;
    const int r = d->rank, n = d->n, p0 = d->p0;
    const float scale = d->scale;
    const int row = d->rows[m] >= 0 ? d->rows[m] : d->rows[0]; // past n: never stored
    const int K = side ? a.d_out : a.d_in;
    const gptr<T> src = as_global<T>(side ? a.dy : a.x) + int64_t(row) * (side ? a.lddy : a.ldx);
    const gptr<T> mat = as_global<T>(reinterpret_cast<const void *>(side ? d->B : d->A));
    const int ntiles = (r + 15) >> 4;
    const bool bvec = VEC && DT == LORA_BF16 && (r & 7) == 0; // B rows are whole 16-byte pieces

    for (int rt0 = 0; rt0 < ntiles; rt0 += RT) {
        floatx4 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = floatx4{};
        for (int kb = wave * NS * E::kStep; kb < K; kb += W * NS * E::kStep) {
            F xf[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) xf[s] = load_row<DT, VEC>(src, kb + s * E::kStep + E::kVec * g, K);
            if (side == 0) {
                F wf[NS][RT];
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const int j = 16 * (rt0 + i) + m;
                        wf[s][i] = load_row<DT, VEC>(mat + int64_t(j < r ? j : r - 1) * K, kb + s * E::kStep + E::kVec * g, K);
                    }
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < RT; ++i) acc[i] = mma<DT>(xf[s], wf[s][i], acc[i]);
            } else if (bvec) {
                if constexpr (DT == LORA_BF16) {
                    // 32 rows x 2 RT pieces of 16 bytes, RT pieces a lane
                    u32x4 w[NS][RT];
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            const int q = lane + 64 * i, kr = kb + 32 * s + q / (2 * RT), j = 16 * rt0 + 8 * (q % (2 * RT));
                            w[s][i] = *(gptr<u32x4>)(mat + int64_t(kr < K ? kr : K - 1) * r + (j < r ? j : 0));
                            if (kr >= K) w[s][i] = u32x4{};
                        }
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        // 32-byte granules (one rank tile of a row), moved so that 4 rows of a
                        // tile fall in distinct banks
                        char *tile = lds + (wave * 2 + (s & 1)) * kTile;
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            const int q = lane + 64 * i, kr = q / (2 * RT), pc = q % (2 * RT);
                            const int gran = (pc >> 1) ^ ((RT == 4 ? kr >> 1 : kr >> 2) & (RT - 1));
                            *reinterpret_cast<u32x4 *>(tile + kr * 32 * RT + gran * 32 + (pc & 1) * 16) = w[s][i];
                        }
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            u32x2 h[2];
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const int kr = 8 * g + 4 * b + (m >> 2);
                                const int gran = i ^ ((RT == 4 ? kr >> 1 : kr >> 2) & (RT - 1));
                                h[b] = read_tr(tile + kr * 32 * RT + gran * 32 + (m & 3) * 8);
                            }
                            acc[i] = mma<DT>(xf[s], join8(h[0], h[1]), acc[i]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        acc[i] = mma<DT>(xf[s], load_col<DT>(mat, r, 16 * (rt0 + i) + m, kb + s * E::kStep + E::kVec * g, K), acc[i]);
            }
        }
        // lane l of tile i holds D[row 4 (l / 16) + q][rank l % 16]
        float *red = reinterpret_cast<float *>(lds);
        __syncthreads(); // the tiles of every wave are read
#pragma unroll
        for (int i = 0; i < RT; ++i) *reinterpret_cast<floatx4 *>(red + ((wave * RT + i) * 64 + lane) * 4) = acc[i];
        __syncthreads();
        for (int idx = tid; idx < RT * 256; idx += W * 64) {
            const int i = idx >> 8, l2 = (idx >> 2) & 63, q = idx & 3;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) sum += red[((w * RT + i) * 64 + l2) * 4 + q];
            const int mm = 4 * (l2 >> 4) + q, j = 16 * (rt0 + i) + (l2 & 15);
            if (mm >= n || rt0 + i >= ntiles) continue;
            const int p = p0 + mm;
            const float t = j < r ? sum * scale : 0.f;
            char *win = (side ? a.ut : a.vt) + int64_t(p / kWin) * E::kParts * a.r16 * kWin * E::kPart;
            const int at = j * kWin + p % kWin;
            if constexpr (DT == LORA_BF16) {
                const uint32_t h = f32_to_bf16(t);
                const bool fin = (h & 0x7f80u) != 0x7f80u; // an infinity or NaN has no rest
                const float rest = fin ? t - bf16_to_f32(h) : 0.f;
                const uint32_t mid = f32_to_bf16(rest);
                uint16_t *o = reinterpret_cast<uint16_t *>(win) + at;
                o[0] = uint16_t(h);
                o[a.r16 * kWin] = uint16_t(mid);
                o[2 * a.r16 * kWin] = uint16_t(f32_to_bf16(rest - bf16_to_f32(mid)));
                if (side) {
                    uint16_t *u = reinterpret_cast<uint16_t *>(a.ur) + int64_t(p) * 2 * a.r16 + 32 * (j >> 4) + (j & 15);
                    u[0] = uint16_t(h);
                    u[16] = uint16_t(mid);
                }
            } else {
                reinterpret_cast<float *>(win)[at] = t;
                if (side) reinterpret_cast<float *>(a.ur)[int64_t(p) * a.r16 + j] = t;
            }
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------
// Launch 2.  A wave: 64 columns of x (dA) or dy (dB), one item's rows, the
// ranks in groups of 16 RT.
// ----------------------------------------------------------------------------
constexpr int kGradWaves = 4;
constexpr int kMaxSpan = 2048;

// The wave's column fragments of one window, from its LDS tile: 32 rows of 128
// bytes, unit 16 bytes, unit un of row q in slot un ^ (4 if q & 2): 4 rows
// of a fragment read then fall in distinct banks.
__device__ __forceinline__ int tile_at(int q, int un) { return q * 128 + ((un ^ ((q & 2) << 1)) << 4); }
__device__ __forceinline__ bf16x8 tile_frag(const char *tile, int t, int m, int g, int step)
{
    // rows step * g .. + 7, columns of tile t: 8-byte pieces of 4 columns
    const int un = (t >> 1) * 4 + (m & 3);
    u32x2 h[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) h[b] = read_tr(tile + tile_at(step * g + 4 * b + (m >> 2), un) + (t & 1) * 8);
    return join8(h[0], h[1]);
}

// Stores 4 consecutive fp32 sums.
__device__ __forceinline__ void put4(float *dst, floatx4 v, int n, bool vec, bool add)
{
    if (vec) {
        if (add) v += *reinterpret_cast<const floatx4 *>(dst);
        *reinterpret_cast<floatx4 *>(dst) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) dst[e] = add ? dst[e] + v[e] : v[e];
    }
}

template <int DT, bool VEC, int RT>
__device__ __forceinline__ void grad_item(const BwdArgs &a, const Item &it, int side, int c0, int rt0, int r,
                                          float *dst, bool add, const int32_t *tok, char *tile)
{
    using E = Elem<DT>;
    using T = typename E::T;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int D = side ? a.d_out : a.d_in;
    const gptr<T> src = as_global<T>(side ? a.dy : a.x);
    const int64_t ld = side ? a.lddy : a.ldx;
    const char *ft = side ? a.vt : a.ut;
    const int w0 = it.begin / kWin, w1 = (it.end - 1) / kWin;
    floatx4 acc[4][RT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[t][i] = floatx4{};

    for (int w = w0; w <= w1; ++w) {
        const int base = w * kWin;
        const bool edge = base < it.begin || base + kWin > it.end; // wave-uniform
        const char *win = ft + int64_t(w) * E::kParts * a.r16 * kWin * E::kPart;
        if constexpr (DT == LORA_BF16) {
            bf16x8 xf[4];
            if constexpr (VEC) {
                // row (lane / 8) + 8 i of the window, 16 bytes at column 8 (lane % 8)
                int cc = c0 + 8 * (lane & 7);
                cc = cc < D ? cc : 0; // past the row: columns that are not stored
                u32x4 xr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = base + (lane >> 3) + 8 * i;
                    const int pc = min(max(p, it.begin), it.end - 1);
                    xr[i] = *(gptr<u32x4>)(src + int64_t(tok[pc - it.begin]) * ld + cc);
                    if (edge && p != pc) xr[i] = u32x4{};
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<u32x4 *>(tile + tile_at((lane >> 3) + 8 * i, lane & 7)) = xr[i];
#pragma unroll
                for (int t = 0; t < 4; ++t) xf[t] = tile_frag(tile, t, m, g, 8);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int p = base + 8 * g + e;
                    const int pc = min(max(p, it.begin), it.end - 1);
                    const gptr<T> row = src + int64_t(tok[pc - it.begin]) * ld;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int cc = min(c0 + col<DT>(m >> 2, 4 * t + (m & 3)), D - 1);
                        const uint16_t h = row[cc];
                        xf[t][e] = __builtin_bit_cast(__bf16, uint16_t(p == pc ? h : 0));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                // ranks past r16 (the last group): clamped, not stored
                const int j = min(16 * (rt0 + i), a.r16 - 16) + m;
#pragma unroll
                for (int q = 0; q < E::kParts; ++q) {
                    u32x4 uw = *(gptr<u32x4>)(as_global<uint16_t>(win) + (q * a.r16 + j) * kWin + 8 * g);
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int p = base + 8 * g + 2 * e;
                            if (p < it.begin || p >= it.end) uw[e] &= 0xffff0000u;
                            if (p + 1 < it.begin || p + 1 >= it.end) uw[e] &= 0x0000ffffu;
                        }
                    }
                    const bf16x8 uf = __builtin_bit_cast(bf16x8, uw);
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        acc[t][i] = side ? mma<DT>(uf, xf[t], acc[t][i]) : mma<DT>(xf[t], uf, acc[t][i]);
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                floatx4 xf[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int p = base + 16 * h + 4 * g + e;
                    const int pc = min(max(p, it.begin), it.end - 1);
                    const gptr<T> row = src + int64_t(tok[pc - it.begin]) * ld;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int cc = min(c0 + col<DT>(m >> 2, 4 * t + (m & 3)), D - 1);
                        const float f = row[cc];
                        xf[t][e] = p == pc ? f : 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const int j = min(16 * (rt0 + i), a.r16 - 16) + m;
                    floatx4 uf = *(gptr<floatx4>)(as_global<float>(win) + j * kWin + 16 * h + 4 * g);
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int p = base + 16 * h + 4 * g + e;
                            if (p < it.begin || p >= it.end) uf[e] = 0.f;
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        acc[t][i] = side ? mma<DT>(uf, xf[t], acc[t][i]) : mma<DT>(xf[t], uf, acc[t][i]);
                }
            }
        }
    }
    // dA (side 0): D rows are columns of x, D columns are ranks.  dB: D rows
    // are ranks, D columns are columns of dy (rows of dB).
    const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15) == 0 && ((side ? r : D) & 3) == 0;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (side == 0) {
                const int j = 16 * (rt0 + i) + m, c = c0 + col<DT>(g, 4 * t);
                if (j < r && c < D) put4(dst + int64_t(j) * D + c, acc[t][i], D - c, vec, add);
            } else {
                const int c = c0 + col<DT>(m >> 2, 4 * t + (m & 3)), j = 16 * (rt0 + i) + 4 * g;
                if (c < D && j < r) put4(dst + int64_t(c) * r + j, acc[t][i], r - j, vec, add);
            }
        }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kGradWaves * 64) void bwd_grad_kernel(BwdArgs a, int tiles_A, int tiles)
{
    __shared__ __attribute__((aligned(16))) char tiles_lds[kGradWaves * 4096];
    __shared__ int32_t tok[kMaxSpan];
    const int item = blockIdx.x / tiles, tl = blockIdx.x % tiles;
    const Item it = a.items[item];
    const int side = tl >= tiles_A;
    const lora_seg_desc *sd = a.seg + it.seg;
    const int r = sd->rank;
    const uint64_t grad = (side ? a.grad_B : a.grad_A)[sd->adapter];
    if (!grad) return; // this adapter's gradient is not wanted
    for (int i = threadIdx.x; i < it.end - it.begin; i += kGradWaves * 64) tok[i] = a.perm[it.begin + i];
    __syncthreads();
    const int wave = threadIdx.x >> 6;
    const int c0 = (side ? tl - tiles_A : tl) * (64 * kGradWaves) + 64 * wave;
    if (c0 >= (side ? a.d_out : a.d_in)) return;
    float *dst = reinterpret_cast<float *>(grad);
    bool add = a.accumulate;
    if (it.slot >= 0) {
        dst = a.part + it.slot * a.part_stride + (side ? int64_t(r) * a.d_in : 0);
        add = false;
    }
    char *tile = tiles_lds + wave * 4096;
    for (int rt0 = 0; 16 * rt0 < r;) {
        if (r - 16 * rt0 <= 16) {
            grad_item<DT, VEC, 1>(a, it, side, c0, rt0, r, dst, add, tok, tile);
            rt0 += 1;
        } else if (r - 16 * rt0 <= 32) {
            grad_item<DT, VEC, 2>(a, it, side, c0, rt0, r, dst, add, tok, tile);
            rt0 += 2;
        } else {
            grad_item<DT, VEC, 4>(a, it, side, c0, rt0, r, dst, add, tok, tile);
            rt0 += 4;
        }
    }
}

// Launch 3: gradient = sum of a split segment's slots, in slot order.
__global__ __launch_bounds__(256) void bwd_reduce_kernel(BwdArgs a)
{
    const Split sp = a.splits[blockIdx.y];
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

// ----------------------------------------------------------------------------
// Launch 4.  A wave: 64 columns of dx, the up to 64 rows of one chunk.
// ----------------------------------------------------------------------------
constexpr int kDxWaves = 4;

template <int DT, bool VEC>
__global__ __launch_bounds__(kDxWaves * 64) void bwd_dx_kernel(BwdArgs a, int tiles)
{
    using E = Elem<DT>;
    using T = typename E::T;
    using F = typename E::F;
    __shared__ __attribute__((aligned(16))) char tiles_lds[kDxWaves * 2 * 2048];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const lora_chunk_desc *d = a.chunk + blockIdx.x / tiles;
    const int c0 = int(blockIdx.x % tiles) * (64 * kDxWaves) + 64 * wave;
    if (c0 >= a.d_in) return;
    const int r = d->rank, n = d->n, p0 = d->p0;
    const gptr<T> A = as_global<T>(reinterpret_cast<const void *>(d->A));
    char *tile = tiles_lds + wave * 4096;
    floatx4 acc[4][4]; // column tile, row block
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = floatx4{};
    for (int j0 = 0, s = 0; j0 < r; j0 += 16, ++s) {
        F uf[4], af[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + min(16 * i + m, n - 1); // past n: not stored
            if constexpr (DT == LORA_BF16)
                uf[i] = __builtin_bit_cast(F, *(gptr<u32x4>)(as_global<uint16_t>(a.ur) + int64_t(p) * 2 * a.r16 + 2 * j0 + 8 * g));
            else
                uf[i] = *(gptr<floatx4>)(as_global<float>(a.ur) + int64_t(p) * a.r16 + j0 + 4 * g);
        }
        if constexpr (DT == LORA_BF16 && VEC) {
            char *tl = tile + (s & 1) * 2048;
            int cc = c0 + 8 * (lane & 7);
            cc = cc < a.d_in ? cc : 0;
            u32x4 w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = j0 + (lane >> 3) + 8 * i;
                w[i] = *(gptr<u32x4>)(A + int64_t(j < r ? j : r - 1) * a.d_in + cc);
                if (j >= r) w[i] = u32x4{};
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4 *>(tl + tile_at((lane >> 3) + 8 * i, lane & 7)) = w[i];
            // k slots of lane groups 0, 1 meet u's hi parts, 2, 3 its lo parts, of the same ranks
#pragma unroll
            for (int t = 0; t < 4; ++t) af[t] = tile_frag(tl, t, m, g & 1, 8);
        } else {
#pragma unroll
            for (int e = 0; e < E::kVec; ++e) {
                const int j = DT == LORA_BF16 ? j0 + 8 * (g & 1) + e : j0 + 4 * g + e;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int cc = min(c0 + col<DT>(m >> 2, 4 * t + (m & 3)), a.d_in - 1);
                    const T w = A[int64_t(j < r ? j : r - 1) * a.d_in + cc];
                    if constexpr (DT == LORA_BF16) af[t][e] = __builtin_bit_cast(__bf16, uint16_t(j < r ? w : 0));
                    else af[t][e] = j < r ? w : 0.f;
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = mma<DT>(af[t], uf[i], acc[t][i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (16 * i + m >= n) continue;
        T *row = static_cast<T *>(a.dx) + int64_t(d->rows[16 * i + m]) * a.lddx;
        if constexpr (DT == LORA_BF16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = c0 + col<DT>(g, 8 * h);
                const floatx4 lo = acc[2 * h][i], hi = acc[2 * h + 1][i];
                if constexpr (VEC) {
                    if (c >= a.d_in) continue;
                    const u32x4 y = *reinterpret_cast<const u32x4 *>(row + c);
                    u32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f0 = e < 2 ? lo[2 * e] : hi[2 * e - 4], f1 = e < 2 ? lo[2 * e + 1] : hi[2 * e - 3];
                        o[e] = pack_bf16x2(bf16_to_f32(y[e] & 0xffffu) + f0, bf16_to_f32(y[e] >> 16) + f1);
                    }
                    *reinterpret_cast<u32x4 *>(row + c) = o;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < a.d_in)
                            row[c + e] = uint16_t(f32_to_bf16(bf16_to_f32(row[c + e]) + (e < 4 ? lo[e & 3] : hi[e & 3])));
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int c = c0 + col<DT>(g, 4 * t);
                if (c < a.d_in) put4(row + c, acc[t][i], a.d_in - c, VEC, true);
            }
        }
    }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Sorted positions of one span, a whole number of windows: up to kSpans spans
// for the rows, so that the bytes of partial sums stay bounded.
constexpr int kMinSpan = 128, kSpans = 16;
int span_of(int32_t rows)
{
    int span = kMinSpan;
    while (span < kMaxSpan && rows / span > kSpans) span *= 2;
    return span;
}

struct Layout {
    size_t ut, vt, ur, items, splits, part, bytes;
    int64_t part_stride;
    int span;
};

// For up to `rows` adapted tokens; the partial sums of a segment cut into k
// items cross k - 1 span borders, so there are at most two for each border.
Layout layout_of(int32_t rows, int32_t d_in, int32_t d_out, int32_t max_rank)
{
    Layout l{};
    const size_t r16 = size_t(max_rank + 15) / 16 * 16, n = size_t(rows);
    const size_t windows = (n + kWin - 1) / kWin;
    l.span = span_of(rows);
    l.ut = 0;
    l.vt = l.ut + up256(windows * kWin * r16 * 6); // three bf16 parts; fp32 takes 4 of the 6 bytes
    l.ur = l.vt + up256(windows * kWin * r16 * 6);
    l.items = l.ur + up256(n * r16 * 4);
    // span borders inside rows / span of any fewer rows, too: the size grows with `rows`
    const size_t borders = std::max(std::min(n / kMinSpan, size_t(kSpans)), n / kMaxSpan);
    l.splits = l.items + up256((n + borders) * sizeof(Item));
    l.part = l.splits + up256(borders * sizeof(Split));
    l.part_stride = (int64_t(max_rank) * (int64_t(d_in) + d_out) + 3) / 4 * 4;
    l.bytes = l.part + 2 * borders * size_t(l.part_stride) * 4;
    return l;
}

template <int DT, bool VEC> void run_shrink(hipStream_t s, const BwdArgs &a, int nside)
{
    const dim3 grid(unsigned(a.nblk) * nside + 1), block(kShrinkWaves * 64);
    if (a.r16 <= 16) launch_kernel(bwd_shrink_kernel<DT, VEC, 1>, grid, block, 0, s, a);
    else if (a.r16 <= 32) launch_kernel(bwd_shrink_kernel<DT, VEC, 2>, grid, block, 0, s, a);
    else launch_kernel(bwd_shrink_kernel<DT, VEC, 4>, grid, block, 0, s, a);
}

int checked(const char *what)
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? LORA_OK : fail(LORA_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

} // namespace

size_t sgmv_backward_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t max_rank)
{
    return layout_of(T, d_in, d_out, max_rank).bytes;
}

int launch_sgmv_backward(hipStream_t s, const BackwardArgs &b, const PlanView &p, void *ws, const uint16_t **u_rows,
                         int64_t *ldu)
{
    const lora_plan_header *h = p.h;
    const Layout l = layout_of(h->num_sorted, b.d_in, b.d_out, h->max_rank);
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
    a.r16 = (h->max_rank + 15) / 16 * 16;
    a.ut = w + l.ut;
    a.vt = w + l.vt;
    a.ur = w + l.ur;
    a.items = reinterpret_cast<Item *>(w + l.items);
    a.splits = reinterpret_cast<Split *>(w + l.splits);
    a.part = reinterpret_cast<float *>(w + l.part);
    a.part_stride = l.part_stride;
    a.span = l.span;
    a.grad_A = b.grad_A;
    a.grad_B = b.grad_B;
    a.accumulate = b.accumulate;
    a.dx = b.dx;
    a.lddx = b.lddx;
    a.sides = (b.grad_B ? 1 : 0) | (b.grad_A || b.dx || u_rows ? 2 : 0);
    if (u_rows) {
        *u_rows = reinterpret_cast<const uint16_t *>(a.ur);
        *ldu = 2 * int64_t(a.r16);
    }
    if (!a.sides) return LORA_OK;
    const lora_seg_desc *hs = reinterpret_cast<const lora_seg_desc *>(reinterpret_cast<const char *>(h) + h->seg_offset);
    for (int i = 0; i < h->num_segments; ++i) {
        const int n = (hs[i].start + hs[i].len - 1) / a.span - hs[i].start / a.span + 1;
        a.nitems += n;
        a.nsplit += n > 1;
    }

    if (a.nsplit > 65535) return fail(LORA_ERR_ARG, "backward: %d segments over several spans (> 65535)", a.nsplit);

    const bool bf16 = b.dtype == LORA_BF16;
    const bool vec = b.vec_x && b.vec_dy;
    const int nside = a.sides == 3 ? 2 : 1;
    if (bf16 && vec) run_shrink<LORA_BF16, true>(s, a, nside);
    else if (bf16) run_shrink<LORA_BF16, false>(s, a, nside);
    else if (vec) run_shrink<LORA_F32, true>(s, a, nside);
    else run_shrink<LORA_F32, false>(s, a, nside);
    int st = checked("backward shrink");
    if (st) return st;

    constexpr int kCols = 64 * kGradWaves;
    const int tiles_A = a.grad_A ? (a.d_in + kCols - 1) / kCols : 0;
    const int tiles = tiles_A + (a.grad_B ? (a.d_out + kCols - 1) / kCols : 0);
    if (tiles) {
        const int64_t nwg = int64_t(a.nitems) * tiles;
        if (nwg > (int64_t(1) << 31) - 1) return fail(LORA_ERR_ARG, "backward: too many work items");
        const dim3 grid{unsigned(nwg)}, block(kGradWaves * 64);
        if (bf16 && vec) launch_kernel(bwd_grad_kernel<LORA_BF16, true>, grid, block, 0, s, a, tiles_A, tiles);
        else if (bf16) launch_kernel(bwd_grad_kernel<LORA_BF16, false>, grid, block, 0, s, a, tiles_A, tiles);
        else launch_kernel(bwd_grad_kernel<LORA_F32, false>, grid, block, 0, s, a, tiles_A, tiles);
        if ((st = checked("backward gradient"))) return st;
        if (a.nsplit) {
            const int64_t units = (l.part_stride / 4 + 255) / 256;
            launch_kernel(bwd_reduce_kernel, dim3(unsigned(std::min<int64_t>(units, 1024)), unsigned(a.nsplit)), dim3(256),
                          0, s, a);
            if ((st = checked("backward reduce"))) return st;
        }
    }
    if (a.dx) {
        const int tx = (a.d_in + 64 * kDxWaves - 1) / (64 * kDxWaves);
        const int64_t nwg = int64_t(a.nchunk) * tx;
        if (nwg > (int64_t(1) << 31) - 1) return fail(LORA_ERR_ARG, "backward: too many dx tiles");
        const dim3 grid{unsigned(nwg)}, block(kDxWaves * 64);
        const bool vx = vec && b.vec_dx;
        if (bf16 && vx) launch_kernel(bwd_dx_kernel<LORA_BF16, true>, grid, block, 0, s, a, tx);
        else if (bf16) launch_kernel(bwd_dx_kernel<LORA_BF16, false>, grid, block, 0, s, a, tx);
        else if (vx) launch_kernel(bwd_dx_kernel<LORA_F32, true>, grid, block, 0, s, a, tx);
        else launch_kernel(bwd_dx_kernel<LORA_F32, false>, grid, block, 0, s, a, tx);
        if ((st = checked("backward dx"))) return st;
    }
    return LORA_OK;
}

} // namespace lora
