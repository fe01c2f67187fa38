// Plans built on the device: the tokens of a batch, given as requests (a length and an
// adapter each) or as one adapter a token, sorted by adapter into the segments, 16-row
// blocks and 64-row chunks that the SGMV and fused calls read, in one launch and with no
// value that the host has to see ("Multi-LoRA Serving in Production ..." (llms.blog),
// section "Punica and Segmented Gather Matrix-Vector Multiplication (SGMV)": contiguous
// segments whose tokens reference one adapter).  The order is the host builder's: adapters
// ascending, a segment's tokens in their order, tokens without an adapter behind them, and
// rows that no request owns (padding of a captured batch) last, with perm = -1.
//
// A stable counting sort in which no workgroup waits for another: each counts all the
// requests by adapter into LDS (and, beside it, those before its own rows), which is a few
// loads of 4 bytes a thread, and scans the counts over the adapters itself.  It then knows
// the place of every segment, block and chunk, so it ranks and scatters its own kRows rows
// (equal adapters of a wave are matched by one ballot for each bit of the id, then the
// waves add their counts in turn) and writes its share of the records.  Every word of the
// plan has one writer, and results do not depend on the order of the atomics, which add
// whole numbers.  What bounds it is the latency of that chain; a grid-wide sort in several
// launches would pay a launch for each step.
#include "device.h"
#include "internal.h"

namespace lora {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kRows = 256; // rows that a workgroup ranks and scatters
// Blocks, and chunks, of a workgroup: its share of T / 16 + min(T, N) and less than 16 more.
constexpr int kRecords = 512;
static_assert(kRows / 16 + kRows + 16 <= kRecords && 2 * kRecords <= kThreads, "a thread for each record");
static_assert(sizeof(lora_blk_desc) == 128 && sizeof(lora_chunk_desc) == 320 && sizeof(lora_seg_desc) == 40, "records");

struct DevicePlanArgs {
    const int32_t *adapters, *lengths; // [R]; lengths nullptr: 1 each
    const uint64_t *A, *B;
    const int32_t *rank;
    const float *alpha;
    int32_t T, R, N, max_rank, rank_step;
    int32_t S, nb, nc; // records in the tables
    char *base;        // the plan
    lora_plan_header h;
};

// Dynamic LDS: five words for each adapter.
struct Tables {
    int32_t *len;    // rows of the adapter
    int32_t *before; // those before this workgroup's rows, then also those of its earlier waves
    int32_t *start;  // first sorted position
    int32_t *blk0;   // first block
    uint32_t *sc;    // segment (low half) and first chunk
};

__device__ __forceinline__ int wave_scan(int v, int lane) // inclusive
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

__global__ __launch_bounds__(kThreads) void plan_device_kernel(DevicePlanArgs a)
{
    extern __shared__ int32_t dyn[];
    __shared__ int32_t part[4][kWaves];
    __shared__ int32_t mark[kRows], last[kRows / 64];
    __shared__ int32_t rows_of[2][kRecords];
    __shared__ int32_t sums[8]; // rows before this workgroup's without an adapter, rows of all requests
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t0 = blockIdx.x * kRows;
    const Tables tb{dyn, dyn + a.N, dyn + 2 * a.N, dyn + 3 * a.N, reinterpret_cast<uint32_t *>(dyn + 4 * a.N)};

    for (int i = tid; i < a.N; i += kThreads) {
        tb.len[i] = 0;
        tb.before[i] = 0;
    }
    if (tid < kRows) mark[tid] = 0;
    if (tid < 8) sums[tid] = 0;
    __syncthreads();

    // an adapter whose id or rank breaks the call's terms counts as none
    auto adapter_of = [&](int q) {
        const int id = a.adapters[q];
        if (uint32_t(id) >= uint32_t(a.N)) return -1;
        const int r = a.rank[id];
        return r >= 1 && r <= a.max_rank && r % a.rank_step == 0 ? id : -1;
    };

    // ---- requests: counts by adapter, and the request of each own row
    int64_t carry = 0; // rows of the requests of the rounds before
    for (int q0 = 0; q0 < a.R; q0 += kThreads) {
        const int q = q0 + tid;
        const int id = q < a.R ? adapter_of(q) : -1;
        int s, e;
        if (a.lengths) {
            // lengths below 0 count as 0, and rows past T are cut off; a length is cut
            // to T + 1, so that 1024 of them stay below 2^31
            const int len = q < a.R ? min(max(a.lengths[q], 0), a.T + 1) : 0;
            const int incl = wave_scan(len, lane);
            if (lane == 63) part[0][wave] = incl;
            __syncthreads();
            int64_t base = carry;
            int64_t all = 0;
            for (int w = 0; w < kWaves; ++w) {
                if (w < wave) base += part[0][w];
                all += part[0][w];
            }
            carry += all;
            __syncthreads();
            s = int(min(base + incl - len, int64_t(a.T)));
            e = int(min(base + incl, int64_t(a.T)));
        } else {
            s = min(q, a.R);
            e = min(q + 1, a.R);
        }
        // a run of single rows of one adapter is one addition of its wave, not 64 in turn
        if (!a.lengths) {
            const uint64_t on = __ballot(e > s);
            const int first = on ? __shfl(id, __ffsll(static_cast<unsigned long long>(on)) - 1) : -1;
            if (on && __ballot(e > s && id == first) == on) {
                const int b = __popcll(__ballot(e > s && s < t0));
                if (lane == 0) {
                    if (first >= 0) {
                        atomicAdd(&tb.len[first], __popcll(on));
                        if (b) atomicAdd(&tb.before[first], b);
                    } else if (b) {
                        atomicAdd(&sums[0], b);
                    }
                }
                if (e > s && s >= t0 && s < t0 + kRows) mark[s - t0] = q + 1;
                continue;
            }
        }
        if (e > s) {
            const int b = min(max(t0 - s, 0), e - s);
            if (id >= 0) {
                atomicAdd(&tb.len[id], e - s);
                if (b) atomicAdd(&tb.before[id], b);
            } else if (b) {
                atomicAdd(&sums[0], b);
            }
            if (e > t0 && s < t0 + kRows) mark[max(s - t0, 0)] = q + 1;
        }
    }
    const int total = a.lengths ? int(min(carry, int64_t(a.T))) : a.R;
    __syncthreads();

    // ---- scan over the adapters: rows, segments, blocks, chunks
    const int per = (a.N + kThreads - 1) / kThreads;
    const int i0 = min(tid * per, a.N), i1 = min(i0 + per, a.N);
    int own[4] = {0, 0, 0, 0};
    int top_len = 0, top_rank = 0;
    for (int i = i0; i < i1; ++i) {
        const int c = tb.len[i];
        own[0] += c;
        own[1] += c > 0;
        own[2] += (c + 15) >> 4;
        own[3] += (c + 63) >> 6;
        if (blockIdx.x == 0 && c) {
            top_len = max(top_len, c);
            top_rank = max(top_rank, a.rank[i]);
        }
    }
    int at[4], all[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        at[k] = wave_scan(own[k], lane);
        if (lane == 63) part[k][wave] = at[k];
        at[k] -= own[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        all[k] = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) at[k] += part[k][w];
            all[k] += part[k][w];
        }
    }
    for (int i = i0; i < i1; ++i) {
        const int c = tb.len[i];
        tb.start[i] = at[0];
        tb.sc[i] = uint32_t(at[1]) | (uint32_t(at[3]) << 16);
        tb.blk0[i] = at[2];
        at[0] += c;
        at[1] += c > 0;
        at[2] += (c + 15) >> 4;
        at[3] += (c + 63) >> 6;
    }
    const int sorted = all[0], n_seg = all[1], n_blk = all[2], n_chunk = all[3];

    // ---- the adapter of each own row: requests ascend along the rows, so the last mark
    // at or before a row is its request
    int id = -1, row = 0;
    const int t = t0 + tid;
    const bool mine = tid < kRows; // whole waves
    if (mine) {
        int q = mark[tid];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(q, d);
            if (lane >= d) q = max(q, o);
        }
        row = q;
        if (lane == 63) last[wave] = q;
    }
    __syncthreads();
    if (mine) {
        for (int w = 0; w < wave; ++w) row = max(row, last[w]);
        if (t < total && row > 0) id = adapter_of(row - 1);
    }
    const bool live = mine && t < total;
    // equal ids of a wave: one ballot a bit (none counts as N)
    uint64_t same = __ballot(live);
    const int key = id < 0 ? a.N : id;
    if (mine)
        for (int b = 0; (a.N >> b) != 0; ++b) {
            const uint64_t one = __ballot((key >> b) & 1);
            same &= (key >> b) & 1 ? one : ~one;
        }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1)), count = __popcll(same);
    int32_t *counter = id < 0 ? &sums[0] : &tb.before[id];
    int pos = 0; // place among the adapter's rows
    for (int w = 0; w < kRows / 64; ++w) {
        if (w == wave && live) {
            pos = *counter + rank;
            __builtin_amdgcn_wave_barrier();
            if (rank == 0) *counter = pos + count;
        }
        __syncthreads();
    }

    // ---- the own rows
    auto *perm = reinterpret_cast<int32_t *>(a.base + a.h.perm_offset);
    auto *segidx = reinterpret_cast<int32_t *>(a.base + a.h.segidx_offset);
    auto *blk = reinterpret_cast<lora_blk_desc *>(a.base + a.h.blk_offset);
    auto *chunk = reinterpret_cast<lora_chunk_desc *>(a.base + a.h.chunk_offset);
    if (mine && t < a.T) {
        if (id >= 0) {
            const uint32_t sc = tb.sc[id];
            const int p = tb.start[id] + pos;
            perm[p] = t;
            segidx[p] = int(sc & 0xFFFF);
            blk[tb.blk0[id] + (pos >> 4)].rows[pos & 15] = t;
            chunk[(sc >> 16) + (pos >> 6)].rows[pos & 63] = t;
        } else {
            const int p = live ? sorted + pos : t;
            perm[p] = live ? t : -1;
            segidx[p] = -1;
        }
    }

    // ---- this workgroup's share of the records; rows that they hold were written above
    // or by the rows' own workgroups
    const int wgs = gridDim.x, wg = blockIdx.x;
    auto *seg = reinterpret_cast<lora_seg_desc *>(a.base + a.h.seg_offset);
    char *soa = a.base + a.h.soa_offset;
    auto *sA = reinterpret_cast<uint64_t *>(soa), *sB = sA + a.S;
    auto *s_ptr = reinterpret_cast<int32_t *>(sB + a.S);
    int32_t *s_id = s_ptr + a.S + 1, *s_rank = s_id + a.S;
    auto *s_scale = reinterpret_cast<float *>(s_rank + a.S);
    for (int i = wg * kThreads + tid; i < max(a.N, a.S); i += wgs * kThreads) {
        if (i < a.N && tb.len[i] > 0) {
            const int s = int(tb.sc[i] & 0xFFFF);
            lora_seg_desc d;
            d.A = a.A[i];
            d.B = a.B[i];
            d.start = tb.start[i];
            d.len = tb.len[i];
            d.rank = a.rank[i];
            d.adapter = i;
            d.scale = a.alpha[i] / float(d.rank);
            d.blk0 = tb.blk0[i];
            seg[s] = d;
            sA[s] = d.A;
            sB[s] = d.B;
            s_ptr[s] = d.start;
            s_id[s] = i;
            s_rank[s] = d.rank;
            s_scale[s] = d.scale;
        }
        if (i >= n_seg && i < a.S) { // no such segment
            seg[i] = lora_seg_desc{};
            sA[i] = 0;
            sB[i] = 0;
            s_ptr[i] = sorted;
            s_id[i] = -1;
            s_rank[i] = 0;
            s_scale[i] = 0.f;
        }
    }
    // the adapter of block or chunk x: the last one whose first is not past x (adapters
    // without rows share the first of the next one that has some)
    auto find = [&](auto first, int x) {
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first(mid) <= x) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    // This workgroup's blocks x0 + i and chunks y0 + i: a thread each writes the record's head (its
    // first 64 bytes) and leaves its rows' count, then the waves fill the places past it.
    const int per_b = (a.nb + wgs - 1) / wgs, per_c = (a.nc + wgs - 1) / wgs;
    const int x0 = wg * per_b, y0 = wg * per_c;
    const bool is_chunk = tid >= kRecords;
    const int i = is_chunk ? tid - kRecords : tid, x = (is_chunk ? y0 : x0) + i;
    if (i < (is_chunk ? per_c : per_b) && x < (is_chunk ? a.nc : a.nb)) {
        u32x4 w[4] = {};
        int n = 0;
        if (x < (is_chunk ? n_chunk : n_blk)) {
            const int ad = is_chunk ? find([&](int j) { return int(tb.sc[j] >> 16); }, x) : find([&](int j) { return tb.blk0[j]; }, x);
            const int c = x - (is_chunk ? int(tb.sc[ad] >> 16) : tb.blk0[ad]), rows = is_chunk ? 64 : 16;
            const uint64_t A = a.A[ad], B = a.B[ad];
            const int r = a.rank[ad];
            const float scale = a.alpha[ad] / float(r);
            n = min(tb.len[ad] - c * rows, rows);
            w[0] = u32x4{uint32_t(A), uint32_t(A >> 32), uint32_t(B), uint32_t(B >> 32)};
            w[1] = u32x4{__float_as_uint(scale), uint32_t(r), uint32_t(n), uint32_t(tb.start[ad] + c * rows)};
            w[2][0] = tb.sc[ad] & 0xFFFF;
            if (is_chunk) {
                w[2][1] = uint32_t(tb.blk0[ad] + 4 * c);
                w[2][2] = uint32_t((n + 15) >> 4);
            }
        }
        auto *to = is_chunk ? reinterpret_cast<u32x4 *>(chunk + x) : reinterpret_cast<u32x4 *>(blk + x);
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = w[k];
        rows_of[is_chunk][i] = n;
    }
    __syncthreads();
    for (int k = tid >> 4; k < per_b && x0 + k < a.nb; k += kThreads / 16)
        if ((tid & 15) >= rows_of[0][k]) blk[x0 + k].rows[tid & 15] = -1;
    for (int k = wave; k < per_c && y0 + k < a.nc; k += kWaves)
        if (lane >= rows_of[1][k]) chunk[y0 + k].rows[lane] = -1;

    // ---- the header
    if (wg != 0) return;
    __syncthreads();
    if (tid < 2) part[tid][0] = 0;
    __syncthreads();
    atomicMax(&part[0][0], top_rank);
    atomicMax(&part[1][0], top_len);
    __syncthreads();
    if (tid == 0) {
        lora_plan_header h = a.h;
        h.num_tokens = total;
        h.num_sorted = sorted;
        h.num_segments = n_seg;
        h.num_blocks = n_blk;
        h.max_rank = part[0][0];
        h.max_len = part[1][0];
        h.num_chunks = n_chunk;
        *reinterpret_cast<lora_plan_header *>(a.base) = h;
        s_ptr[a.S] = sorted;
    }
}

} // namespace

int launch_plan_device(hipStream_t s, const DevicePlanCall &c, const lora_plan_header &h, void *dev)
{
    DevicePlanArgs a{};
    a.adapters = c.adapters;
    a.lengths = c.lengths;
    a.A = c.pool_A;
    a.B = c.pool_B;
    a.rank = c.pool_rank;
    a.alpha = c.pool_alpha;
    a.T = h.num_tokens;
    a.R = c.n_requests;
    a.N = c.n_adapters;
    a.max_rank = c.max_rank;
    a.rank_step = c.rank_multiple;
    a.S = h.num_segments;
    a.nb = h.num_blocks;
    a.nc = h.num_chunks;
    a.base = static_cast<char *>(dev);
    a.h = h;
    const size_t shm = size_t(5) * size_t(c.n_adapters) * 4;
    // more than the 64 KB that a launch takes unasked
    if (shm > 48 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(plan_device_kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize,
                                                 LORA_DEVICE_PLAN_MAX_ADAPTERS * 5 * 4);
        if (e != hipSuccess) return fail(LORA_ERR_HIP, "device plan LDS: %s", hipGetErrorString(e));
    }
    launch_kernel(plan_device_kernel, dim3(unsigned((a.T + kRows - 1) / kRows)), dim3(kThreads), shm, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(LORA_ERR_HIP, "device plan launch: %s", hipGetErrorString(e));
    return LORA_OK;
}

} // namespace lora
