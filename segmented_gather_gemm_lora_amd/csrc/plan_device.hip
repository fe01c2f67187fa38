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
// loads of 4 bytes a thread, and scans the counts over the adapters itself (two packed counts a
// word).  It then knows
// the place of every segment, block and chunk, so it ranks and scatters its own kRows rows
// (equal adapters of a wave are matched by one ballot for each bit of the id, then the
// waves add their counts in turn) and writes its share of the records.  Every word of the
// plan has one writer, and results do not depend on the order of the atomics, which add
// whole numbers.  What bounds it is the latency of that chain (64 requests 6.8 us; 16384 rows,
// 600 requests, 2000 adapters 11.1); a grid-wide sort in several launches would pay a launch for
// each step.
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

// Inclusive scans of a wave by lane shifts within 16 lanes, then from their last lanes.
template <class Op> __device__ __forceinline__ uint32_t wave_scan(uint32_t v, Op op)
{
    v = op(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xf, 0xf, true)));
    v = op(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xf, 0xf, true)));
    v = op(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xf, 0xf, true)));
    v = op(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xf, 0xf, true)));
    v = op(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xa, 0xf, false)));
    v = op(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xc, 0xf, false)));
    return v;
}
struct Add {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a + b; }
};
struct Max {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};
// Two counts in a word: rows (low 17 bits) and segments, or blocks (low 16) and chunks.
constexpr int kRowBits = 17, kBlkBits = 16;

__global__ __launch_bounds__(kThreads) void plan_device_kernel(DevicePlanArgs a)
{
    extern __shared__ int32_t dyn[];
    __shared__ uint32_t part[4][kWaves];
    __shared__ int32_t mark[kRows], id_at[kRows], last[kRows / 64];
    __shared__ int32_t owner[2][kRecords], rows_of[2][kRecords];
    __shared__ int32_t none[1]; // rows without an adapter before this workgroup's
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wgs = gridDim.x, wg = blockIdx.x;
    const int t0 = wg * kRows;
    const Tables tb{dyn, dyn + a.N, dyn + 2 * a.N, dyn + 3 * a.N, reinterpret_cast<uint32_t *>(dyn + 4 * a.N)};

    for (int i = tid; i < a.N; i += kThreads) {
        tb.len[i] = 0;
        tb.before[i] = 0;
    }
    if (tid < kRows) mark[tid] = 0;
    for (int i = tid; i < 2 * kRecords; i += kThreads) owner[0][i] = -1;
    if (tid == 0) none[0] = 0;
    __syncthreads();

    // an adapter whose id or rank breaks the call's terms counts as none
    auto adapter_of = [&](int q) {
        const int id = a.adapters[q];
        if (uint32_t(id) >= uint32_t(a.N)) return -1;
        const int r = a.rank[id];
        return r >= 1 && r <= a.max_rank && r % a.rank_step == 0 ? id : -1;
    };

    // ---- requests: counts by adapter, and the request of each own row (its place, counted
    // from 1, at its first own row; its adapter beside it)
    int64_t carry = 0; // rows of the requests of the rounds before
    for (int q0 = 0; q0 < a.R; q0 += kThreads) {
        const int q = q0 + tid;
        const int id = q < a.R ? adapter_of(q) : -1;
        int s, e;
        if (a.lengths) {
            // lengths below 0 count as 0, and rows past T are cut off; a length is cut
            // to T + 1, so that 1024 of them stay below 2^31
            const int len = q < a.R ? min(max(a.lengths[q], 0), a.T + 1) : 0;
            const int incl = int(wave_scan(uint32_t(len), Add{}));
            if (lane == 63) part[0][wave] = uint32_t(incl);
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
        if (e > max(s, t0) && s < t0 + kRows) {
            const int at = max(s - t0, 0);
            mark[at] = at + 1;
            id_at[at] = id;
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
                        atomicAdd(&none[0], b);
                    }
                }
                continue;
            }
        }
        if (e > s) {
            const int b = min(max(t0 - s, 0), e - s);
            if (id >= 0) {
                atomicAdd(&tb.len[id], e - s);
                if (b) atomicAdd(&tb.before[id], b);
            } else if (b) {
                atomicAdd(&none[0], b);
            }
        }
    }
    const int total = a.lengths ? int(min(carry, int64_t(a.T))) : a.R;
    __syncthreads();

    // ---- scan over the adapters: rows and segments, blocks and chunks
    const int per = (a.N + kThreads - 1) / kThreads;
    const int i0 = min(tid * per, a.N), i1 = min(i0 + per, a.N);
    auto counts = [&](int c) {
        return u32x2{uint32_t(c) | uint32_t(c > 0) << kRowBits, uint32_t((c + 15) >> 4) | uint32_t((c + 63) >> 6) << kBlkBits};
    };
    uint32_t rs = 0, bc = 0, top_len = 0;
    for (int i = i0; i < i1; ++i) {
        const u32x2 c = counts(tb.len[i]);
        rs += c[0];
        bc += c[1];
        top_len = max(top_len, uint32_t(tb.len[i]));
    }
    const uint32_t rs1 = wave_scan(rs, Add{}), bc1 = wave_scan(bc, Add{});
    // ---- and the adapter of each own row: requests ascend along the rows, so the last mark
    // at or before a row is its request's
    const int t = t0 + tid;
    const bool mine = tid < kRows; // whole waves
    int row = mine ? int(wave_scan(uint32_t(mark[tid]), Max{})) : 0;
    if (lane == 63) {
        part[0][wave] = rs1;
        part[1][wave] = bc1;
        if (mine) last[wave] = row;
    }
    __syncthreads();
    rs = rs1 - rs;
    bc = bc1 - bc;
    uint32_t all_rs = 0, all_bc = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t x = part[0][w], y = part[1][w];
        rs += w < wave ? x : 0;
        bc += w < wave ? y : 0;
        all_rs += x;
        all_bc += y;
    }
    constexpr uint32_t kRowMask = (1u << kRowBits) - 1, kBlkMask = (1u << kBlkBits) - 1;
    const int sorted = int(all_rs & kRowMask), n_seg = int(all_rs >> kRowBits);
    const int n_blk = int(all_bc & kBlkMask), n_chunk = int(all_bc >> kBlkBits);
    // this workgroup's share of the blocks and chunks: their adapters
    const int per_b = (a.nb + wgs - 1) / wgs, per_c = (a.nc + wgs - 1) / wgs;
    const int x0 = wg * per_b, y0 = wg * per_c;
    for (int i = i0; i < i1; ++i) {
        const u32x2 c = counts(tb.len[i]);
        const int blk = int(bc & kBlkMask), chk = int(bc >> kBlkBits);
        tb.start[i] = int(rs & kRowMask);
        tb.sc[i] = (rs >> kRowBits) | uint32_t(chk) << 16;
        tb.blk0[i] = blk;
        rs += c[0];
        bc += c[1];
        for (int x = max(blk, x0); x < min(int(bc & kBlkMask), x0 + per_b); ++x) owner[0][x - x0] = i;
        for (int y = max(chk, y0); y < min(int(bc >> kBlkBits), y0 + per_c); ++y) owner[1][y - y0] = i;
    }
    int id = -1;
    if (mine) {
        for (int w = 0; w < wave; ++w) row = max(row, last[w]);
        if (t < total && row > 0) id = id_at[row - 1];
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
    int32_t *counter = id < 0 ? &none[0] : &tb.before[id];
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
    // the adapters' tables, for the records below, are on the way meanwhile
    struct Adapter {
        uint64_t A, B;
        int rank;
        float alpha;
    };
    auto adapter = [&](int i) { return Adapter{a.A[i], a.B[i], a.rank[i], a.alpha[i]}; };
    // a thread for each of this workgroup's records, blocks first
    const bool is_chunk = tid >= kRecords;
    const int rec = is_chunk ? tid - kRecords : tid, x = (is_chunk ? y0 : x0) + rec;
    const bool writes = rec < (is_chunk ? per_c : per_b) && x < (is_chunk ? a.nc : a.nb);
    const int own = writes ? owner[is_chunk][rec] : -1;
    // and for its share of the adapters, whose segments it writes
    const int sg = wg * kThreads + tid;
    const bool has = sg < a.N && tb.len[sg] > 0;
    Adapter ra{}, sa{};
    if (own >= 0) ra = adapter(own);
    if (has) sa = adapter(sg);

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
            if (a.S > 0) segidx[p] = -1; // without adapters the plan has no such table
        }
    }

    // ---- the records' heads (their first 64 bytes); the places past their rows are filled below
    if (writes) {
        u32x4 w[4] = {};
        int n = 0;
        if (own >= 0) {
            const uint32_t sc = tb.sc[own];
            const int c = x - (is_chunk ? int(sc >> 16) : tb.blk0[own]), rows = is_chunk ? 64 : 16;
            n = min(tb.len[own] - c * rows, rows);
            w[0] = u32x4{uint32_t(ra.A), uint32_t(ra.A >> 32), uint32_t(ra.B), uint32_t(ra.B >> 32)};
            w[1] = u32x4{__float_as_uint(ra.alpha / float(ra.rank)), uint32_t(ra.rank), uint32_t(n), uint32_t(tb.start[own] + c * rows)};
            w[2][0] = sc & 0xFFFF;
            if (is_chunk) {
                w[2][1] = uint32_t(tb.blk0[own] + 4 * c);
                w[2][2] = uint32_t((n + 15) >> 4);
            }
        }
        auto *to = is_chunk ? reinterpret_cast<u32x4 *>(chunk + x) : reinterpret_cast<u32x4 *>(blk + x);
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = w[k];
        rows_of[is_chunk][rec] = n;
    }
    // ---- segments
    auto *seg = reinterpret_cast<lora_seg_desc *>(a.base + a.h.seg_offset);
    char *soa = a.base + a.h.soa_offset;
    auto *sA = reinterpret_cast<uint64_t *>(soa), *sB = sA + a.S;
    auto *s_ptr = reinterpret_cast<int32_t *>(sB + a.S);
    int32_t *s_id = s_ptr + a.S + 1, *s_rank = s_id + a.S;
    auto *s_scale = reinterpret_cast<float *>(s_rank + a.S);
    auto write_segment = [&](int i, const Adapter &ad) {
        const int s = int(tb.sc[i] & 0xFFFF);
        const lora_seg_desc d{ad.A, ad.B, tb.start[i], tb.len[i], ad.rank, i, ad.alpha / float(ad.rank), tb.blk0[i]};
        seg[s] = d;
        sA[s] = d.A;
        sB[s] = d.B;
        s_ptr[s] = d.start;
        s_id[s] = i;
        s_rank[s] = d.rank;
        s_scale[s] = d.scale;
    };
    if (has) write_segment(sg, sa);
    for (int i = sg + wgs * kThreads; i < a.N; i += wgs * kThreads)
        if (tb.len[i] > 0) write_segment(i, adapter(i));
    for (int i = n_seg + sg; i < a.S; i += wgs * kThreads) { // no such segment
        seg[i] = lora_seg_desc{};
        sA[i] = 0;
        sB[i] = 0;
        s_ptr[i] = sorted;
        s_id[i] = -1;
        s_rank[i] = 0;
        s_scale[i] = 0.f;
    }
    // the largest rank and length, of workgroup 0's header
    if (wg == 0) {
        uint32_t top_rank = 0;
        for (int i = tid; i < a.N; i += kThreads)
            if (tb.len[i] > 0) top_rank = max(top_rank, uint32_t(i == sg ? sa.rank : a.rank[i]));
        top_rank = wave_scan(top_rank, Max{});
        top_len = wave_scan(top_len, Max{});
        if (lane == 63) {
            part[2][wave] = top_rank;
            part[3][wave] = top_len;
        }
    }
    __syncthreads();
    for (int k = tid >> 4; k < per_b && x0 + k < a.nb; k += kThreads / 16)
        if ((tid & 15) >= rows_of[0][k]) blk[x0 + k].rows[tid & 15] = -1;
    for (int k = wave; k < per_c && y0 + k < a.nc; k += kWaves)
        if (lane >= rows_of[1][k]) chunk[y0 + k].rows[lane] = -1;
    if (wg == 0 && tid == 0) {
        lora_plan_header h = a.h;
        h.num_tokens = total;
        h.num_sorted = sorted;
        h.num_segments = n_seg;
        h.num_blocks = n_blk;
        h.num_chunks = n_chunk;
        h.max_rank = h.max_len = 0;
        for (int w = 0; w < kWaves; ++w) {
            h.max_rank = max(h.max_rank, int(part[2][w]));
            h.max_len = max(h.max_len, int(part[3][w]));
        }
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
