// AdamW over many tensors in one launch on gfx950, for the fp32 masters of the
// adapters of a pool:
//
//     g = c grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g g
//     p = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// with lr, b1, b2, eps, wd, c, t of the tensor's group (an adapter: every
// tenant's training run has its own), read from device memory, and optionally a
// bf16 copy of p (the matrix that the forward reads).
//
// States are fp32 or 8 bits.  8 bits: a block of 256 elements has one scale
// 2^(e - 127), e a byte, and a code per element: m as OCP E4M3, v (never
// negative) as an unsigned float of 5 exponent bits (bias 15) and 3 mantissa
// bits.  e is the least that keeps the block's largest magnitude below 1.75 2^8
// (m) or 1.75 2^16 (v) scales.  Rounding is stochastic: v moves by 0.1% a step
// (b2 = 0.999) and its codes are 6 to 12% apart, so rounding to nearest would
// never move it; a value between two codes goes up with the probability of its
// distance, so the stored state is right on average.  The 32 random bits of an
// element (16 each for m and v) are a hash of the group's seed and step, the
// tensor's number and the element's index.  A positive v never becomes 0, which
// would make the next quotient arbitrarily large.  A non-finite m or v is stored
// as NaN and does not enter its block's scale.  The update of p uses m and v
// before they are rounded.
//
// One workgroup takes one chunk, described by one record (addresses at the
// chunk's start), and a wave 256 consecutive elements at a time, so that a
// state block's maximum is a reduction over one wave.
#include "device.h"
#include "internal.h"

#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

namespace lora {
namespace {

constexpr int kBlock = LORA_ADAM_BLOCK; // elements of a state block: 4 per lane of a wave
constexpr int kAdamThreads = 256;
constexpr int kRow = 4 * kAdamThreads; // elements that a workgroup takes at a time
// Elements of a chunk: one row, or two where there are many with 8-bit states, whose
// arithmetic shows (the record, the group's numbers and its powers are read and formed
// once for both).  8-bit states, one / two rows, us.  fp32 gradients: 0.5 M elements
// 4.8 / 5.6, 1 M 6.5 / 6.7, 2 M 10.8 / 10.1, 8 M 34 / 31, 24 M 90 / 82, 48 M 171 / 166;
// from 64 M on 5% the other way for steps one after the other (96 M 330 / 347), nothing
// with other work between, and the first steps 520 / 480: left alone.  bf16 gradients:
// 1 M 6.7 / 7.4, 1.5 M 9.0 / 9.2, 24 M 90 / 82, 96 M 308 / 285, 128 M 401 / 373.  fp32
// states, 16.8 M elements: 80 / 88.
constexpr int64_t kFewElements = 1 << 21;
int chunk_of(int64_t elements, bool eight) { return eight && elements > kFewElements ? 2 * kRow : kRow; }

constexpr uint32_t kAdamMagic = 0x4C6F4164u;

struct AdamChunk {
    uint64_t param, grad, copy, m, v, m_scale, v_scale; // at the chunk's first element
    uint32_t e0;     // index of the first element in its tensor
    int32_t n;       // elements
    int32_t group;
    uint32_t tensor; // the tensor's number
    uint64_t reserved;
};
static_assert(sizeof(AdamChunk) == 80, "chunk record");

struct AdamHeader {
    uint32_t magic;
    int32_t state, grad_dtype, n_groups;
    int64_t n_chunks;
    uint64_t bytes;
};
static_assert(sizeof(AdamHeader) == 32, "plan header");

// Multiply and xor-shift mixing of 32 bits (the fractions of sqrt 2 and sqrt 3
// as odd multipliers): every input bit reaches every output bit.
__device__ __forceinline__ uint32_t mix(uint32_t h)
{
    h ^= h >> 16;
    h *= 0x6A09E667u;
    h ^= h >> 15;
    h *= 0xBB67AE85u;
    return h ^ (h >> 16);
}

// Largest of 64 lanes' values.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
#define LORA_MAX_DPP(ctrl, rows) x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), ctrl, rows, 0xf, false)))
    LORA_MAX_DPP(0xB1, 0xf);  // lane ^ 1
    LORA_MAX_DPP(0x4E, 0xf);  // lane ^ 2
    LORA_MAX_DPP(0x124, 0xf); // rotations inside 16 lanes
    LORA_MAX_DPP(0x128, 0xf);
    LORA_MAX_DPP(0x142, 0xa); // lane 15 of rows 0 and 2 to rows 1 and 3
    LORA_MAX_DPP(0x143, 0xc); // lane 31 to rows 2 and 3
#undef LORA_MAX_DPP
    return uint32_t(__builtin_amdgcn_readlane(int(x), 63));
}

// The 8-bit formats: BIAS of the exponent, TOP = exponent of the largest code.
struct M8 {
    static constexpr int kBias = 7, kTop = 8;
    static constexpr uint32_t kMax = 0x7E, kNan = 0x7F;
};
struct V8 {
    static constexpr int kBias = 15, kTop = 16;
    static constexpr uint32_t kMax = 0xFE, kNan = 0xFF;
};

// Scale byte of a block whose largest magnitude has these bits.
template <class Q> __device__ __forceinline__ int scale_of(uint32_t most)
{
    const int e = int(most >> 23) + ((most & 0x7fffffu) >= 0x600000u) - Q::kTop;
    return min(max(e, 1), 254);
}
// |a| on the block's scale, as the code's magnitude: moved so that the code's
// exponent field lies in the fp32 one (its subnormals are fp32 subnormals), the
// code is the top bits; the noise is added below them.
template <class Q> __device__ __forceinline__ uint32_t encode(float a, int e, uint32_t noise16)
{
    const uint32_t bits = __float_as_uint(__builtin_ldexpf(__builtin_fabsf(a), Q::kBias - e)) + (noise16 << 4);
    const uint32_t c = min(bits >> 20, Q::kMax);
    return __builtin_isfinite(a) ? c : Q::kNan;
}
// 4 codes of m: the hardware's E4M3 conversion, then the scale 2^(e - 127).
__device__ __forceinline__ floatx4 decode_m(uint32_t w, int e)
{
    typedef float floatx2 __attribute__((ext_vector_type(2)));
    const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    const float scale = __uint_as_float(uint32_t(e) << 23);
    return floatx4{a[0] * scale, a[1] * scale, b[0] * scale, b[1] * scale};
}
// A code of v: its bits in the fp32 exponent and mantissa, then the scale.
__device__ __forceinline__ float decode_v(uint32_t c, int e)
{
    const float f = __builtin_ldexpf(__uint_as_float(c << 20), e - V8::kBias);
    return c == V8::kNan ? __builtin_nanf("") : f;
}

// Everything of a step is touched once: fp32 accesses are non-temporal (128
// adapters of rank 16, 503 MB: 96 us without, 80 us with).
//
// 4 consecutive elements from a 16-byte (fp32) or 8-byte (bf16) aligned place; past n: 0.
__device__ __forceinline__ floatx4 get4(const float *p, int n)
{
    if (n >= 4) return __builtin_nontemporal_load(reinterpret_cast<const floatx4 *>(p));
    floatx4 f{};
    for (int i = 0; i < n; ++i) f[i] = p[i];
    return f;
}
__device__ __forceinline__ floatx4 get4(const uint16_t *p, int n)
{
    floatx4 f{};
    if (n >= 4) {
        const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
        return floatx4{bf16_to_f32(w[0] & 0xffffu), bf16_to_f32(w[0] >> 16), bf16_to_f32(w[1] & 0xffffu), bf16_to_f32(w[1] >> 16)};
    }
    for (int i = 0; i < n; ++i) f[i] = bf16_to_f32(p[i]);
    return f;
}
__device__ __forceinline__ uint32_t get4(const uint8_t *p, int n)
{
    if (n >= 4) return *reinterpret_cast<const uint32_t *>(p);
    uint32_t w = 0;
    for (int i = 0; i < n; ++i) w |= uint32_t(p[i]) << (8 * i);
    return w;
}
__device__ __forceinline__ void put4(float *p, floatx4 f, int n)
{
    if (n >= 4) __builtin_nontemporal_store(f, reinterpret_cast<floatx4 *>(p));
    else
        for (int i = 0; i < n; ++i) p[i] = f[i];
}
__device__ __forceinline__ void put4(uint16_t *p, floatx4 f, int n)
{
    const u32x2 w = {f32_to_bf16(f[0]) | (f32_to_bf16(f[1]) << 16), f32_to_bf16(f[2]) | (f32_to_bf16(f[3]) << 16)};
    if (n >= 4) *reinterpret_cast<u32x2 *>(p) = w;
    else
        for (int i = 0; i < n; ++i) p[i] = uint16_t(w[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void put4(uint8_t *p, uint32_t w, int n)
{
    if (n >= 4) *reinterpret_cast<uint32_t *>(p) = w;
    else
        for (int i = 0; i < n; ++i) p[i] = uint8_t(w >> (8 * i));
}

// 1 - b^t in 64 bits: with t in the thousands and b near 1 an fp32 power is off
// by more than the fp32 quotient it goes into.
__device__ __forceinline__ float one_minus_power(float b, int t)
{
    double p = 1.0, q = double(b);
    for (uint32_t n = uint32_t(t); n; n >>= 1, q *= q)
        if (n & 1) p *= q;
    return float(1.0 - p);
}

// (m / bc1) / (sqrt(v / bc2) + eps).  fp32 states: IEEE quotients and root, behind
// the memory's time (16.8 M elements: 80 us with these or with the form below).
// 8-bit states: products with the reciprocals of bc1 and bc2, root and reciprocal to
// 1 ulp each, of an update that is far below p (100 M elements with bf16 gradients:
// 283 us so, 331 with IEEE ones).  The root instruction takes subnormals as 0, so small
// arguments are moved up for it (no time either).
template <bool BITS8>
__device__ __forceinline__ float update(float m, float v, float bc1, float bc2, float ib1, float ib2, float eps)
{
#pragma clang fp contract(off)
    if constexpr (!BITS8) return (m / bc1) / (__builtin_sqrtf(v / bc2) + eps);
    const float x = v * ib2;
    const bool small = x < 0x1p-96f;
    const float root = __builtin_amdgcn_sqrtf(small ? x * 0x1p64f : x) * (small ? 0x1p-32f : 1.0f);
    return (m * ib1) * __builtin_amdgcn_rcpf(root + eps);
}

// A lane's 4 elements of a row, as loaded.
template <bool BITS8, class G> struct AdamRow {
    floatx4 p, g, m, v;
    uint32_t mc, vc;
    int me, ve;
    __device__ __forceinline__ void load(const AdamChunk &c, int at)
    {
        const int n = c.n - at, lat = n > 0 ? at : 0, ln = n > 0 ? n : 0; // past the end: nothing
        p = get4(reinterpret_cast<const float *>(c.param) + lat, ln);
        g = get4(reinterpret_cast<const G *>(c.grad) + lat, ln);
        if constexpr (BITS8) {
            mc = get4(reinterpret_cast<const uint8_t *>(c.m) + lat, ln);
            vc = get4(reinterpret_cast<const uint8_t *>(c.v) + lat, ln);
            const int b = at / kBlock * kBlock < c.n ? at / kBlock : 0; // state block (one per wave)
            me = reinterpret_cast<const uint8_t *>(c.m_scale)[b];
            ve = reinterpret_cast<const uint8_t *>(c.v_scale)[b];
        } else {
            m = get4(reinterpret_cast<const float *>(c.m) + lat, ln);
            v = get4(reinterpret_cast<const float *>(c.v) + lat, ln);
        }
    }
};

template <bool BITS8, class G>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(const AdamChunk *__restrict__ chunks,
                                                             const lora_adam_hyper *__restrict__ hyper)
{
#pragma clang fp contract(off)
    const AdamChunk &c = chunks[blockIdx.x];
    int at = 4 * int(threadIdx.x); // this lane's first element of the row, in the chunk
    AdamRow<BITS8, G> row;
    row.load(c, at);
    const lora_adam_hyper h = hyper[c.group];
    if (h.step < 1) return; // a group that rests
    const float bc1 = one_minus_power(h.beta1, h.step), bc2 = one_minus_power(h.beta2, h.step);
    const float c1 = 1.0f - h.beta1, c2 = 1.0f - h.beta2;
    const float ib1 = 1.0f / bc1, ib2 = 1.0f / bc2;
    const uint32_t key = mix(mix(h.seed + uint32_t(h.step) * 0x9E3779B9u) + c.tensor * 0x510E527Fu);
    while (at / kBlock * kBlock < c.n) { // wave-uniform
        floatx4 p = row.p, g = row.g, m = row.m, v = row.v;
        if constexpr (BITS8) {
            m = decode_m(row.mc, row.me);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = decode_v((row.vc >> (8 * i)) & 0xffu, row.ve);
        }
        const int here = at;
        at += kRow;
        if (at / kBlock * kBlock < c.n) row.load(c, at); // the next row's, while this one is computed
        const int n = c.n - here, b = here / kBlock; // elements from here, may be <= 0; state block
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float gi = g[i] * h.grad_scale;
            m[i] = h.beta1 * m[i] + c1 * gi;
            v[i] = h.beta2 * v[i] + c2 * (gi * gi);
            p[i] = p[i] - h.lr * (h.weight_decay * p[i] + update<BITS8>(m[i], v[i], bc1, bc2, ib1, ib2, h.eps));
        }
        uint32_t mc = 0, vc = 0;
        if constexpr (BITS8) {
            uint32_t mm = 0, vm = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t ma = __float_as_uint(m[i]) & 0x7fffffffu, va = __float_as_uint(v[i]) & 0x7fffffffu;
                if (i < n) {
                    mm = max(mm, ma < 0x7f800000u ? ma : 0u);
                    vm = max(vm, va < 0x7f800000u ? va : 0u);
                }
            }
            const int me = scale_of<M8>(wave_max(mm)), ve = scale_of<V8>(wave_max(vm));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t rnd = mix((c.e0 + uint32_t(here + i)) * 0x9E3779B9u + key);
                const uint32_t qm = encode<M8>(m[i], me, rnd & 0xffffu) | (m[i] < 0.f ? 0x80u : 0u);
                uint32_t qv = encode<V8>(v[i], ve, rnd >> 16);
                if (v[i] > 0.f && qv == 0) qv = 1;
                mc |= qm << (8 * i);
                vc |= qv << (8 * i);
            }
            if ((threadIdx.x & 63) == 0) {
                reinterpret_cast<uint8_t *>(c.m_scale)[b] = uint8_t(me);
                reinterpret_cast<uint8_t *>(c.v_scale)[b] = uint8_t(ve);
            }
        }
        if (n > 0) {
            put4(reinterpret_cast<float *>(c.param) + here, p, n);
            if (c.copy) put4(reinterpret_cast<uint16_t *>(c.copy) + here, p, n);
            if constexpr (BITS8) {
                put4(reinterpret_cast<uint8_t *>(c.m) + here, mc, n);
                put4(reinterpret_cast<uint8_t *>(c.v) + here, vc, n);
            } else {
                put4(reinterpret_cast<float *>(c.m) + here, m, n);
                put4(reinterpret_cast<float *>(c.v) + here, v, n);
            }
        }
    }
}

// The values of 8-bit states; both formats' values are bf16 values (4
// significant bits times a power of two in bf16's range).  16 elements a thread,
// in accesses of 16 bytes where they are whole.
__global__ __launch_bounds__(256) void adam_values_kernel(int64_t n, const uint8_t *__restrict__ m,
                                                          const uint8_t *__restrict__ ms, const uint8_t *__restrict__ v,
                                                          const uint8_t *__restrict__ vs, uint16_t *__restrict__ mo,
                                                          uint16_t *__restrict__ vo)
{
    const int64_t at = 16 * (int64_t(blockIdx.x) * 256 + threadIdx.x);
    if (at >= n) return;
    auto side = [&](const uint8_t *codes, const uint8_t *scales, uint16_t *out, auto values) {
        const int e = scales[at / kBlock];
        if (n - at >= 16) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(codes + at);
            u32x4 o[2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const floatx4 f = values(w[q], e);
                o[q >> 1][2 * (q & 1)] = f32_to_bf16(f[0]) | (f32_to_bf16(f[1]) << 16);
                o[q >> 1][2 * (q & 1) + 1] = f32_to_bf16(f[2]) | (f32_to_bf16(f[3]) << 16);
            }
            *reinterpret_cast<u32x4 *>(out + at) = o[0];
            *reinterpret_cast<u32x4 *>(out + at + 8) = o[1];
        } else {
            for (int64_t k = at; k < n; k += 4)
                put4(out + k, values(get4(codes + k, int(n - k)), e), int(n - k));
        }
    };
    if (m) side(m, ms, mo, [](uint32_t w, int e) { return decode_m(w, e); });
    if (v) side(v, vs, vo, [](uint32_t w, int e) {
        return floatx4{decode_v(w & 0xffu, e), decode_v((w >> 8) & 0xffu, e), decode_v((w >> 16) & 0xffu, e), decode_v(w >> 24, e)};
    });
}

// The plan's header; nullptr with the error set.
const AdamHeader *check_adam_plan(const void *plan)
{
    if (!plan) {
        fail(LORA_ERR_ARG, "the plan's host buffer is NULL");
        return nullptr;
    }
    if (reinterpret_cast<uintptr_t>(plan) & 15u) {
        fail(LORA_ERR_ALIGN, "the plan's host buffer is not 16-byte aligned");
        return nullptr;
    }
    const auto *h = static_cast<const AdamHeader *>(plan);
    if (h->magic != kAdamMagic || h->n_chunks < 0) {
        fail(LORA_ERR_PLAN, "buffer holds no built AdamW plan");
        return nullptr;
    }
    return h;
}
int plan_status(const void *plan)
{
    return !plan ? LORA_ERR_ARG : (reinterpret_cast<uintptr_t>(plan) & 15u) ? LORA_ERR_ALIGN : LORA_ERR_PLAN;
}

bool sizes_ok(const lora_adam_tensor *t, int32_t n)
{
    if (n < 0 || (n > 0 && !t)) return false;
    for (int32_t i = 0; i < n; ++i)
        if (t[i].n < 0 || t[i].n > LORA_ADAM_MAX_ELEMENTS) return false;
    return true;
}

int64_t elements_of(const lora_adam_tensor *t, int32_t n)
{
    int64_t e = 0;
    for (int32_t i = 0; i < n; ++i) e += t[i].n;
    return e;
}
int64_t chunks_of(const lora_adam_tensor *t, int32_t n, int chunk)
{
    int64_t c = 0;
    for (int32_t i = 0; i < n; ++i) c += (t[i].n + chunk - 1) / chunk;
    return c;
}

} // namespace
} // namespace lora

using namespace lora;

extern "C" {

size_t lora_adamw_plan_bytes(const lora_adam_tensor *tensors, int32_t n_tensors)
{
    // the larger of both states' plans: chunks of one row
    if (!sizes_ok(tensors, n_tensors)) return 0;
    return sizeof(AdamHeader) + sizeof(AdamChunk) * size_t(chunks_of(tensors, n_tensors, kRow));
}

int lora_adamw_plan(const lora_adam_tensor *tensors, int32_t n_tensors, int32_t n_groups, int state, int grad_dtype,
                    void *plan_host, size_t plan_bytes)
{
    clear_error();
    if (n_tensors < 0) return fail(LORA_ERR_ARG, "n_tensors %d < 0", n_tensors);
    if (n_tensors > 0 && !tensors) return fail(LORA_ERR_ARG, "tensors is NULL");
    if (n_groups < 0) return fail(LORA_ERR_ARG, "n_groups %d < 0", n_groups);
    if (state != LORA_ADAM_F32 && state != LORA_ADAM_8BIT) return fail(LORA_ERR_DTYPE, "unknown state format %d", state);
    if (grad_dtype != LORA_F32 && grad_dtype != LORA_BF16) return fail(LORA_ERR_DTYPE, "unknown dtype %d", grad_dtype);
    if (!plan_host) return fail(LORA_ERR_ARG, "plan_host is NULL");
    if (!aligned16(plan_host)) return fail(LORA_ERR_ALIGN, "plan_host is not 16-byte aligned");
    static_cast<AdamHeader *>(plan_host)->magic = 0;
    // everything that is written, to find memory that two tensors share
    struct Range {
        uint64_t lo, hi;
        int32_t tensor;
    };
    std::vector<Range> ranges;
    try {
        ranges.reserve(size_t(n_tensors) * 6);
    } catch (const std::bad_alloc &) {
        return fail(LORA_ERR_WORKSPACE, "no host memory for %d tensors", n_tensors);
    }
    const bool eight = state == LORA_ADAM_8BIT;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const lora_adam_tensor &t = tensors[i];
        if (t.n < 0 || t.n > LORA_ADAM_MAX_ELEMENTS)
            return fail(LORA_ERR_ARG, "tensor %d: %lld elements outside [0, 2^31 - 1]", i, (long long)t.n);
        if (t.group < 0 || t.group >= n_groups)
            return fail(LORA_ERR_ARG, "tensor %d: group %d outside [0, %d)", i, t.group, n_groups);
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale)))
            return fail(LORA_ERR_ARG, "tensor %d: a NULL address", i);
        if ((t.param | t.grad | t.copy | t.m | t.v) & 15u)
            return fail(LORA_ERR_ALIGN, "tensor %d: an address is not 16-byte aligned", i);
        const uint64_t n = uint64_t(t.n), blocks = (n + kBlock - 1) / kBlock, es = eight ? 1 : 4;
        ranges.push_back({t.param, t.param + 4 * n, i});
        if (t.copy) ranges.push_back({t.copy, t.copy + 2 * n, i});
        ranges.push_back({t.m, t.m + es * n, i});
        ranges.push_back({t.v, t.v + es * n, i});
        if (eight) {
            ranges.push_back({t.m_scale, t.m_scale + blocks, i});
            ranges.push_back({t.v_scale, t.v_scale + blocks, i});
        }
    }
    std::sort(ranges.begin(), ranges.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    for (size_t k = 1; k < ranges.size(); ++k)
        if (ranges[k].lo < ranges[k - 1].hi)
            return fail(LORA_ERR_ARG, "tensors %d and %d share memory that is written",
                        std::min(ranges[k].tensor, ranges[k - 1].tensor), std::max(ranges[k].tensor, ranges[k - 1].tensor));
    // gradients are read by one workgroup while others write: they may share memory
    // with each other, not with what is written
    for (int32_t i = 0; i < n_tensors; ++i) {
        const uint64_t lo = tensors[i].grad, hi = lo + (grad_dtype == LORA_BF16 ? 2 : 4) * uint64_t(tensors[i].n);
        // the last written range that starts below hi ends last too
        auto it = std::lower_bound(ranges.begin(), ranges.end(), hi, [](const Range &r, uint64_t at) { return r.lo < at; });
        if (hi > lo && it != ranges.begin() && (--it)->hi > lo)
            return fail(LORA_ERR_ARG, "the gradient of tensor %d shares memory with what is written of tensor %d", i, it->tensor);
    }
    const int chunk = chunk_of(elements_of(tensors, n_tensors), eight);
    const int64_t n_chunks = chunks_of(tensors, n_tensors, chunk);
    const size_t need = sizeof(AdamHeader) + sizeof(AdamChunk) * size_t(n_chunks);
    if (plan_bytes < need) return fail(LORA_ERR_WORKSPACE, "plan buffer of %zu B < %zu B needed", plan_bytes, need);
    auto *h = static_cast<AdamHeader *>(plan_host);
    auto *ch = reinterpret_cast<AdamChunk *>(h + 1);
    for (int32_t i = 0; i < n_tensors; ++i) {
        const lora_adam_tensor &t = tensors[i];
        const uint64_t gs = grad_dtype == LORA_BF16 ? 2 : 4, es = eight ? 1 : 4;
        for (int64_t e = 0; e < t.n; e += chunk, ++ch) {
            std::memset(ch, 0, sizeof *ch);
            ch->param = t.param + 4 * uint64_t(e);
            ch->grad = t.grad + gs * uint64_t(e);
            ch->copy = t.copy ? t.copy + 2 * uint64_t(e) : 0;
            ch->m = t.m + es * uint64_t(e);
            ch->v = t.v + es * uint64_t(e);
            ch->m_scale = eight ? t.m_scale + uint64_t(e) / kBlock : 0;
            ch->v_scale = eight ? t.v_scale + uint64_t(e) / kBlock : 0;
            ch->e0 = uint32_t(e);
            ch->n = int32_t(std::min<int64_t>(chunk, t.n - e));
            ch->group = t.group;
            ch->tensor = uint32_t(i);
        }
    }
    h->state = state;
    h->grad_dtype = grad_dtype;
    h->n_groups = n_groups;
    h->n_chunks = n_chunks;
    h->bytes = need;
    h->magic = kAdamMagic;
    return LORA_OK;
}

int lora_adamw_upload(const void *plan_host, void *plan_dev, size_t dev_bytes, void *stream)
{
    clear_error();
    const AdamHeader *h = check_adam_plan(plan_host);
    if (!h) return plan_status(plan_host);
    if (!plan_dev) return fail(LORA_ERR_ARG, "plan_dev is NULL");
    if (!aligned16(plan_dev)) return fail(LORA_ERR_ALIGN, "plan_dev is not 16-byte aligned");
    if (dev_bytes < h->bytes) return fail(LORA_ERR_WORKSPACE, "plan_dev of %zu B < %zu B", dev_bytes, size_t(h->bytes));
    const hipError_t e = hipMemcpyAsync(plan_dev, plan_host, h->bytes, hipMemcpyHostToDevice, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? LORA_OK : fail(LORA_ERR_HIP, "hipMemcpyAsync: %s", hipGetErrorString(e));
}

int lora_adamw(void *stream, const void *plan_host, const void *plan_dev, const lora_adam_hyper *hyper_dev,
               int32_t n_groups)
{
    clear_error();
    const AdamHeader *h = check_adam_plan(plan_host);
    if (!h) return plan_status(plan_host);
    if (n_groups < h->n_groups)
        return fail(LORA_ERR_ARG, "%d groups of parameters; the plan's tensors use %d", n_groups, h->n_groups);
    if (h->n_chunks == 0) return LORA_OK;
    if (!plan_dev || !hyper_dev) return fail(LORA_ERR_ARG, "plan_dev or hyper_dev is NULL");
    if (!aligned16(plan_dev) || !aligned16(hyper_dev))
        return fail(LORA_ERR_ALIGN, "plan_dev or hyper_dev is not 16-byte aligned");
    if (h->n_chunks > most_workgroups(kAdamThreads))
        return fail(LORA_ERR_ARG, "%lld chunks of elements are more than one launch has", (long long)h->n_chunks);
    const auto *ch = reinterpret_cast<const AdamChunk *>(static_cast<const AdamHeader *>(plan_dev) + 1);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid{unsigned(h->n_chunks)}, block(kAdamThreads);
    const bool eight = h->state == LORA_ADAM_8BIT, gb = h->grad_dtype == LORA_BF16;
    if (eight && gb) launch_kernel(adamw_kernel<true, uint16_t>, grid, block, 0, s, ch, hyper_dev);
    else if (eight) launch_kernel(adamw_kernel<true, float>, grid, block, 0, s, ch, hyper_dev);
    else if (gb) launch_kernel(adamw_kernel<false, uint16_t>, grid, block, 0, s, ch, hyper_dev);
    else launch_kernel(adamw_kernel<false, float>, grid, block, 0, s, ch, hyper_dev);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? LORA_OK : fail(LORA_ERR_HIP, "AdamW launch: %s", hipGetErrorString(e));
}

int lora_adam_state_values(void *stream, int64_t n, const void *m, const void *m_scale, const void *v,
                           const void *v_scale, void *m_out, void *v_out)
{
    clear_error();
    if (n < 0) return fail(LORA_ERR_ARG, "n %lld < 0", (long long)n);
    if (n == 0 || (!m && !v)) return LORA_OK;
    if ((m && (!m_scale || !m_out)) || (v && (!v_scale || !v_out))) return fail(LORA_ERR_ARG, "a scale or output is NULL");
    if ((m && (!aligned16(m) || !aligned16(m_out))) || (v && (!aligned16(v) || !aligned16(v_out))))
        return fail(LORA_ERR_ALIGN, "codes or outputs are not 16-byte aligned");
    const int64_t nwg = (n + 4095) / 4096;
    if (nwg > most_workgroups(256)) return fail(LORA_ERR_ARG, "n %lld is too large", (long long)n);
    launch_kernel(adam_values_kernel, dim3(unsigned(nwg)), dim3(256), 0, static_cast<hipStream_t>(stream), n,
                  static_cast<const uint8_t *>(m), static_cast<const uint8_t *>(m_scale), static_cast<const uint8_t *>(v),
                  static_cast<const uint8_t *>(v_scale), static_cast<uint16_t *>(m_out), static_cast<uint16_t *>(v_out));
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? LORA_OK : fail(LORA_ERR_HIP, "state values launch: %s", hipGetErrorString(e));
}

} // extern "C"
