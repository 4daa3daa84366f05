// ninfer_sample: the next token of every row of logits, by temperature, top-k,
// top-p and min-p from given random numbers.
//
// What is kept is a beginning of the tokens in falling order of their logits (equal ones in rising order of their
// place), so that a border, a logit's order-preserving 32-bit key and the place of its last equal one, describes it: top-k and
// top-p each find one by descending through the key's bits (11, 11 and 10 at a time) with histograms in shared memory, of
// counts or of weights. The token is then the first whose running sum in the order of the row passes the
// random number's share of the whole.
//
// Weights are whole numbers (units of 2^-kScale of the largest one), exact to 2^-30 of themselves: sums of them do not
// depend on the order in which threads and CTAs add, which makes borders and choices the same however a row is divided. A
// weight is 2^t, t = (x - m) log2(e) / T in two floats: a table of 64 powers for the fraction's first six bits, the
// exponential's series for the rest, everything else in integers.
//
// A row is divided among the CTAs of a cluster, which exchange maxima, sums and histograms through distributed shared memory.
#include <cmath>

#include "decode.cuh"
#include "gemv.h"
#include "ninfer_layer.h"

namespace ninfer {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 2048, kMostCluster = 8;

// 2^(30 + j / 64), rounded
__device__ const uint32_t kPowers[64] = {
    0x40000000, 0x40b268fa, 0x4166c34c, 0x421d1462, 0x42d561b4, 0x438fb0cb, 0x444c0740, 0x450a6abb,
    0x45cae0f2, 0x468d6fae, 0x47521cc6, 0x4818ee22, 0x48e1e9ba, 0x49ad1598, 0x4a7a77d4, 0x4b4a169c,
    0x4c1bf829, 0x4cf022ca, 0x4dc69cdd, 0x4e9f6cd4, 0x4f7a9930, 0x50582888, 0x51382182, 0x521a8ad7,
    0x52ff6b55, 0x53e6c9da, 0x54d0ad5a, 0x55bd1cdb, 0x56ac1f75, 0x579dbc57, 0x5891fac1, 0x5988e209,
    0x5a82799a, 0x5b7ec8f2, 0x5c7dd7a4, 0x5d7fad59, 0x5e8451d0, 0x5f8bccdb, 0x60962665, 0x61a3666d,
    0x62b39509, 0x63c6ba64, 0x64dcdec3, 0x65f60a7f, 0x6712460b, 0x683199ed, 0x69540ec9, 0x6a79ad56,
    0x6ba27e65, 0x6cce8ae1, 0x6dfddbcc, 0x6f307a41, 0x70666f76, 0x719fc4b9, 0x72dc8374, 0x741cb528,
    0x75606374, 0x76a7980f, 0x77f25cce, 0x7940bb9e, 0x7a92be8b, 0x7be86fba, 0x7d41d96e, 0x7e9f0606};

struct SampleParams {
    ninfer_sample_args a;
    uint32_t slice;         // tokens a CTA, a multiple of 8
    int scale;              // weights are whole multiples of 2^-scale
};

__device__ __forceinline__ uint64_t ld_cluster_u64(const void *local, uint32_t rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_cluster_v2(const void *local, uint32_t rank) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u64(const void *local, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "l"(v) : "memory");
}

// Order-preserving key of a logit without NaN; equal values (both zeros) have equal keys.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }
constexpr uint32_t kLowest = 0x007fffffu;       // the key of -infinity

struct Shared {
    uint32_t powers[64];
    uint64_t part[kWarps], slot[2], total, found[2], totals[kBins];
    uint2 hist[kBins];      // low and high words
    uint64_t above, inside;
    uint32_t bin;
    float c_hi, c_lo;
};

template <int kDtype>
struct Row {
    const void *x;
    Shared &s;
    uint32_t lo, hi;        // this CTA's tokens
    uint32_t rank, ranks;
    int scale;
    uint32_t phase = 0;
    // the row's largest logit, log2(e) / temperature in two floats
    float m = 0.f, c_hi = 0.f, c_lo = 0.f;
    // what is kept: keys above `border`, and at it those up to place `last`; weights of at least `least`
    uint32_t border = kLowest + 1, last = ~0u;
    uint64_t least = 0;

    __device__ Row(const void *x, Shared &s, uint32_t lo, uint32_t hi, int scale)
        : x(x), s(s), lo(lo), hi(hi), rank(cluster_ctarank()), ranks(cluster_nctarank()), scale(scale) {}

    __device__ __forceinline__ uint32_t key(uint32_t i) const {
        const float v = load1(x, i, kDtype);
        return v == v ? key_of(v) : kLowest;
    }
    __device__ __forceinline__ bool kept(uint32_t key, uint32_t i) const { return key > border || (key == border && i <= last); }

    // t as two floats; false where 2^t is no more than 2^-100 (or the logit infinitely far away)
    __device__ __forceinline__ bool exponent(float v, float &p, float &rest) const {
        p = rest = 0.f;
        if (v == m) return true;
        const float d = v - m, b = d + m, e = (v - b) + (m - (b - d)) * -1.f;     // d + e = v - m exactly
        p = d * c_hi;
        if (!(p >= -100.f)) return false;
        rest = fmaf(d, c_hi, -p) + fmaf(d, c_lo, e * c_hi);
        return true;
    }
    __device__ __forceinline__ uint64_t weight(uint32_t key) const {
        float p, rest;
        if (!exponent(logit_of(key), p, rest)) return 0;
        const int n = __float2int_rn(p * 64.f);
        const float r = fmaf((float)n, -1.f / 64.f, p) + rest;       // exact but for `rest`, at most 1 / 128
        const float y = r * fmaf(r, fmaf(r, 0.05550411f, 0.24022651f), 0.69314718f);        // 2^r - 1
        const int power = (int)s.powers[n & 63];
        const uint32_t w = (uint32_t)(power + __mulhi(power, __float2int_rn(y * 0x1p32f)));     // of 2^(t - n / 64's whole part), times 2^30
        const int shift = (n >> 6) + scale - 30;
        if (shift >= 0) return (uint64_t)w << shift;
        return shift < -31 ? 0 : ((uint64_t)w + (1ull << (-shift - 1))) >> -shift;
    }

    __device__ uint64_t block_sum(uint64_t v) {
#pragma unroll
        for (int k = 16; k; k /= 2) v += __shfl_xor_sync(~0u, v, k);
        __syncthreads();
        if (threadIdx.x % 32 == 0) s.part[threadIdx.x / 32] = v;
        __syncthreads();
        v = threadIdx.x % 32 < kWarps ? s.part[threadIdx.x % 32] : 0;
#pragma unroll
        for (int k = 16; k; k /= 2) v += __shfl_xor_sync(~0u, v, k);
        return v;
    }
    __device__ uint64_t block_max(uint64_t v) {
#pragma unroll
        for (int k = 16; k; k /= 2) v = max(v, __shfl_xor_sync(~0u, v, k));
        __syncthreads();
        if (threadIdx.x % 32 == 0) s.part[threadIdx.x / 32] = v;
        __syncthreads();
        v = threadIdx.x % 32 < kWarps ? s.part[threadIdx.x % 32] : 0;
#pragma unroll
        for (int k = 16; k; k /= 2) v = max(v, __shfl_xor_sync(~0u, v, k));
        return v;
    }
    // Puts one value of each CTA where the others see it. The slot of two exchanges ago is free: every CTA has read it
    // before it came to the barrier of the last one.
    __device__ void exchange(uint64_t v) {
        phase ^= 1;
        if (threadIdx.x == 0) s.slot[phase] = v;
        cluster_sync();
    }
    __device__ uint64_t cluster_sum(uint64_t v) {
        exchange(block_sum(v));
        uint64_t t = 0;
        for (uint32_t r = 0; r < ranks; ++r) t += ld_cluster_u64(&s.slot[phase], r);
        return t;
    }
    __device__ uint64_t cluster_max(uint64_t v) {
        exchange(block_max(v));
        uint64_t t = 0;
        for (uint32_t r = 0; r < ranks; ++r) t = max(t, ld_cluster_u64(&s.slot[phase], r));
        return t;
    }

    // The first place, in the order of the row, at which the running sum of value(place) passes `target` (which the
    // whole sum does).
    template <class F>
    __device__ uint32_t locate(uint64_t target, F value) {
        const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const uint32_t each = ((hi - lo + kWarps - 1) / kWarps + 31) / 32 * 32;
        const uint32_t from = min(lo + warp * each, hi), to = min(from + each, hi);
        uint64_t sum = 0;
        for (uint32_t i = from + lane; i < to; i += 32) sum += value(i);
#pragma unroll
        for (int k = 16; k; k /= 2) sum += __shfl_xor_sync(~0u, sum, k);
        __syncthreads();
        if (lane == 0) s.part[warp] = sum;
        __syncthreads();
        uint64_t before = 0, all = 0;
        for (uint32_t w = 0; w < kWarps; ++w) {
            if (w < warp) before += s.part[w];
            all += s.part[w];
        }
        exchange(all);
        for (uint32_t r = 0; r < rank; ++r) before += ld_cluster_u64(&s.slot[phase], r);
        if (target >= before && target - before < sum) {            // one warp of the cluster
            uint64_t run = target - before;                          // what is still to be passed
            for (uint32_t i0 = from; i0 < to; i0 += 32) {
                uint64_t v = i0 + lane < to ? value(i0 + lane) : 0;
#pragma unroll
                for (int k = 1; k < 32; k *= 2) {
                    const uint64_t u = __shfl_up_sync(~0u, v, k);
                    if (lane >= (uint32_t)k) v += u;
                }
                const uint32_t passed = __ballot_sync(~0u, v > run);
                if (passed) {
                    if (lane < ranks) st_cluster_u64(&s.found[phase], lane, i0 + __ffs(passed) - 1);
                    break;
                }
                run -= __shfl_sync(~0u, v, 31);
            }
        }
        cluster_sync();
        return (uint32_t)s.found[phase];
    }

    // Moves the border to where the kept tokens' counts (kWeighted: weights), from the largest on, reach `target`, which
    // their sum does; its last token included.
    template <bool kWeighted>
    __device__ void cut(uint64_t target) {
        uint32_t prefix = 0;
        uint64_t above = 0;
        for (int level = 0; level < 3; ++level) {
            const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
            for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = make_uint2(0, 0);
            __syncthreads();
            for (uint32_t i = lo + threadIdx.x; i < hi; i += kThreads) {
                const uint32_t k = key(i);
                if (!kept(k, i) || (level && k >> (shift + bits) != prefix)) continue;
                uint2 *bin = &s.hist[k >> shift & ((1u << bits) - 1)];
                if (kWeighted) {
                    const uint64_t w = weight(k);
                    const uint32_t old = atomicAdd(&bin->x, (uint32_t)w);
                    const uint32_t more = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
                    if (more) atomicAdd(&bin->y, more);
                } else atomicAdd(&bin->x, 1u);
            }
            cluster_sync();
            // each CTA adds up its part of the bins and gives the sums to all
            const uint32_t each = kBins / ranks;
            for (uint32_t i = threadIdx.x; i < each; i += kThreads) {
                const uint32_t b = rank * each + i;
                uint64_t t = 0;
                for (uint32_t r = 0; r < ranks; ++r) {
                    const uint2 v = ld_cluster_v2(&s.hist[b], r);
                    t += (uint64_t)v.y << 32 | v.x;
                }
                for (uint32_t r = 0; r < ranks; ++r) st_cluster_u64(&s.totals[b], r, t);
            }
            cluster_sync();
            // from the highest bin on: the one in which the sum reaches the target
            constexpr int kEach = kBins / kThreads;
            const uint32_t top = kBins - 1 - threadIdx.x * kEach, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
            uint64_t t[kEach], mine = 0;
#pragma unroll
            for (int j = 0; j < kEach; ++j) mine += t[j] = s.totals[top - j];
            uint64_t run = mine;
#pragma unroll
            for (int k = 1; k < 32; k *= 2) {
                const uint64_t u = __shfl_up_sync(~0u, run, k);
                if (lane >= (uint32_t)k) run += u;
            }
            if (lane == 31) s.part[warp] = run;
            __syncthreads();
            run += above - mine;
            for (uint32_t w = 0; w < warp; ++w) run += s.part[w];
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                if (run < target && target - run <= t[j]) {
                    s.above = run;
                    s.inside = t[j];
                    s.bin = top - j;
                }
                run += t[j];
            }
            __syncthreads();
            above = s.above;
            prefix = prefix << bits | s.bin;
            __syncthreads();
        }
        // the border's key is known; of the tokens that share it, the first in the row's order
        const uint64_t each = kWeighted ? weight(prefix) : 1, ties = s.inside / each;
        const uint64_t wanted = (target - above + each - 1) / each;
        uint32_t at = prefix == border ? last : ~0u;
        if (wanted < ties) {
            const uint32_t old = border, old_last = last;
            at = locate(wanted - 1, [&](uint32_t i) -> uint64_t { return key(i) == prefix && (prefix != old || i <= old_last); });
        }
        border = prefix;
        last = at;
    }
};

template <int kDtype>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x;
    if (tid < 64) s.powers[tid] = kPowers[tid];
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_sample_args &a = p.a;
    const uint32_t ranks = cluster_nctarank(), vocab = (uint32_t)a.vocab;
    const uint64_t b = blockIdx.x / ranks;
    const uint32_t lo = min(cluster_ctarank() * p.slice, vocab), hi = min(lo + p.slice, vocab);
    Row<kDtype> row(static_cast<const uint8_t *>(a.logits) + b * a.stride * (kDtype == NINFER_F32 ? 4 : 2), s, lo, hi, p.scale);

    const float temperature = a.temperature ? a.temperature[b] : 1.f, top_p = a.top_p ? a.top_p[b] : 1.f;
    const float min_p = a.min_p ? a.min_p[b] : 0.f, random = a.random[b];
    const int32_t top_k = a.top_k ? a.top_k[b] : 0;
    if (tid == 0) {
        const double c = 1.4426950408889634 / (double)temperature;
        s.c_hi = (float)c;
        s.c_lo = (float)(c - (double)s.c_hi);
    }
    // the largest logit, the first place that has it; how many take part
    uint64_t best = 0, count = 0;
    for (uint32_t i = lo + tid; i < hi; i += kThreads) {
        const uint32_t k = row.key(i);
        count += k > kLowest;
        best = max(best, (uint64_t)k << 32 | (uint32_t)~i);
    }
    best = row.cluster_max(best);
    const bool lead = tid == 0 && row.rank == 0;
    const uint32_t top = (uint32_t)(best >> 32);
    if (top <= kLowest || !(temperature > 0.f)) {
        if (lead) {
            a.tokens[b] = top <= kLowest ? -1 : (int32_t)~(uint32_t)best;
            if (a.logprobs) a.logprobs[b] = top <= kLowest ? -INFINITY : 0.f;
        }
        cluster_sync();         // no CTA leaves while another reads its shared memory
        return;
    }
    row.m = logit_of(top);
    row.c_hi = s.c_hi;
    row.c_lo = isfinite(s.c_hi) ? s.c_lo : 0.f;
    auto weight_at = [&](uint32_t i) -> uint64_t {
        const uint32_t k = row.key(i);
        if (!row.kept(k, i)) return 0;
        const uint64_t w = row.weight(k);
        return w >= row.least ? w : 0;
    };
    auto whole = [&]() {
        uint64_t sum = 0;
        for (uint32_t i = lo + tid; i < hi; i += kThreads) sum += weight_at(i);
        return row.cluster_sum(sum);
    };
    if (top_k > 0) {
        count = row.cluster_sum(count);
        if ((uint64_t)top_k < count) row.template cut<false>((uint64_t)top_k);
    }
    if (top_p < 1.f) {
        const uint64_t sum = whole();
        const double target = ceil((double)fmaxf(top_p, 0.f) * (double)sum);
        row.template cut<true>(max((uint64_t)target, (uint64_t)1));
    }
    if (min_p > 0.f) row.least = (uint64_t)ceil(ldexp((double)fminf(min_p, 1.f), p.scale));
    const uint64_t sum = whole();
    const uint64_t share = (uint64_t)((double)fminf(fmaxf(random, 0.f), 1.f) * (double)sum);
    const uint32_t token = row.locate(min(share, sum - 1), weight_at);
    if (lead) {
        a.tokens[b] = (int32_t)token;
        if (a.logprobs) {
            float t, rest;
            row.exponent(logit_of(row.key(token)), t, rest);
            // ln of the sum in units of the largest weight, which is 2^scale and among those kept
            const uint64_t others = sum - (1ull << p.scale);
            const float of = (float)((double)others * ldexp(1.0, -p.scale));
            a.logprobs[b] = (t + rest) * 0.69314718f - log1pf(of);
        }
    }
    cluster_sync();
}

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_sample(const ninfer_sample_args *args, ninfer_stream stream) {
    if (!args || !args->logits || !args->random || !args->tokens)
        return fail(NINFER_ERR_INVALID_ARGUMENT, "sample: NULL args, logits, random or tokens");
    const ninfer_sample_args &a = *args;
    if (!dtype_valid(a.dtype)) return fail(NINFER_ERR_INVALID_ARGUMENT, "sample: dtype %d unsupported", a.dtype);
    if (a.reserved) return fail(NINFER_ERR_INVALID_ARGUMENT, "sample: reserved must be 0");
    if (!a.rows || !a.vocab || a.vocab > (1ull << 30))
        return fail(NINFER_ERR_SHAPE, "sample: %llu rows of %llu", (unsigned long long)a.rows, (unsigned long long)a.vocab);
    if (a.rows > 1 && a.stride < a.vocab) return fail(NINFER_ERR_SHAPE, "sample: row stride below vocab");
    if (a.rows > 0x7fffffffull / kMostCluster || (a.rows > 1 && a.stride >= (1ull << 40)))
        return fail(NINFER_ERR_OVERFLOW, "sample: too many rows, or a stride of 2^40 or more");
    if (!aligned(a.logits, dtype_size(a.dtype))) return fail(NINFER_ERR_ALIGNMENT, "sample: logits are not aligned to their elements");
    for (const void *q : {(const void *)a.temperature, (const void *)a.top_p, (const void *)a.min_p, (const void *)a.top_k,
                          (const void *)a.random, (const void *)a.tokens, (const void *)a.logprobs})
        if (!aligned(q, 4)) return fail(NINFER_ERR_ALIGNMENT, "sample: controls and outputs must be 4-byte aligned");
    SampleParams p;
    p.a = a;
    int bits = 1;
    while ((1ull << bits) < a.vocab) ++bits;
    p.scale = 62 - bits;
    const unsigned ranks = kMostCluster;
    p.slice = (uint32_t)((a.vocab + ranks - 1) / ranks + 7) / 8 * 8;
    const auto kernel = a.dtype == NINFER_F32    ? sample_kernel<NINFER_F32>
                        : a.dtype == NINFER_BF16 ? sample_kernel<NINFER_BF16>
                                                 : sample_kernel<NINFER_F16>;
    return launch_clusters("sample", ranks, kernel, dim3((unsigned)(a.rows * ranks)), dim3(kThreads), 0, (cudaStream_t)stream, p);
}
