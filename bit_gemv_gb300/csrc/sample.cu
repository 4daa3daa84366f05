// ninfer_sample: the next token of every row of logits, by temperature, top-k,
// top-p and min-p from given random numbers.
//
// What is kept is a beginning of the tokens in falling order of their logits (equal ones in rising order of their
// place), so that a border, a logit's order-preserving 32-bit key and the place of its last equal one, describes it, whatever the
// number of tokens. The token is then the first whose running sum in the order of the row passes the random number's share
// of the whole.
//
// Weights are whole numbers (units of 2^-scale of the largest one), exact to 2^-30 of themselves but for the rounding of x - m: sums
// of them do not depend on the order in which threads and CTAs add, which makes borders and choices the same however a row is
// divided. A weight is 2^t, t = (x - m) log2(e) / T in two floats: a table of 64 powers for the fraction's first six bits, the
// exponential's series for the rest, everything else in integers. Shares of sums are products of whole numbers too.
//
// A row is divided among the CTAs of a cluster, which hold it in shared memory (read once from HBM) and exchange maxima, sums and
// histograms through distributed shared memory. Whatever keeps few tokens is chosen from by the first CTA alone, to which all
// push the tokens that may be kept, so that the others end: those of min-p by their weight; for top-k and top-p (whose sum over all tokens is
// taken first) down to where a histogram of one logit for each thread, its largest, reaches the count or the share, which is
// hardly further than where all logits do. Other borders are found in two passes: a histogram of 2048 bins, 1/64 of a
// power of two wide, from the largest logit down, of counts (top-k) or weights to 16 bits (top-p), tells the bin or the few bins
// in which it lies; their tokens, seldom more than a few hundred, are sorted by the first CTA, which adds their exact weights
// to the exact sum of what lies above. Where more than 2048 tokens lie there (equal logits without end), the border comes from the
// key's bits, eight at a time.
//
// What bounds it: not HBM (greedy rows, 64 of 248320 fp32 logits, 64 MB, 26 us, held like others); about 40 instructions for each exact weight (normal
// logits of deviation 2.5, temperature alone: 87 us; large nuclei, which need them twice: 240 to 300), and the chain of a cluster's exchanges (top-k 62,
// min-p 52; one row 11 to 13 us, 49 with a nucleus of most of the row).
#include <cfloat>
#include <cmath>
#include <cstddef>

#include "decode.cuh"
#include "gemv.h"
#include "ninfer_layer.h"
#include "overlap.h"

namespace ninfer {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kResident = 2;    // CTAs an SM
constexpr uint32_t kBins = 2048, kListed = 2048, kFew = 1024, kMostCluster = 16;
constexpr uint32_t kSliceBytes = 64 * 1024, kMostSliceBytes = 176 * 1024, kLeastSlice = 2048;  // two CTAs an SM, one; tokens

// Added to a float below 2^22, it leaves the nearest whole number in the last bits (conversions go at a sixteenth of the rate of additions);
// kDown, with the sum rounded down, the whole part of one from 0 to 2^23.
constexpr float kRound = 12582912.f, kDown = 8388608.f;

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
    uint32_t vectors;       // 16-byte vectors of a row a CTA
    int scale;              // weights are whole multiples of 2^-scale
    bool held;              // in shared memory
    uint32_t few_k;         // top_k up to which the tokens that may be kept are listed
    float unit, slack;      // of the histogram's weights: a bin's largest is `unit`; sums are too small by less than `slack` of themselves
};

__device__ __forceinline__ uint64_t ld_cluster_u64(const void *local, uint32_t rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const void *local, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u64(const void *local, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(const void *local, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(local), rank)), "r"(v) : "memory");
}

// The cluster's barrier, which wants whole warps.
__device__ __forceinline__ void join() {
    __syncwarp();
    cluster_sync();
}

// Order-preserving key of a logit without NaN; equal values (both zeros) have equal keys.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }

// f * whole for 0 <= f <= 1, exactly, rounded down (up).
__device__ __forceinline__ uint64_t times(float f, uint64_t whole, bool up) {
    const uint32_t bits = __float_as_uint(f), e = max(bits >> 23, 1u), k = 150 - e;      // f = mantissa 2^-k, k from 23 on
    const uint64_t mantissa = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
    const uint64_t low = whole * mantissa, high = __umul64hi(whole, mantissa);
    uint64_t t = k < 64 ? high << (64 - k) | low >> k : k < 128 ? high >> (k - 64) : 0;
    if (up && (k < 64 ? low << (64 - k) : low | (k < 128 ? k > 64 ? high << (128 - k) : 0 : high))) ++t;
    return t;
}

struct alignas(16) Shared {
    uint32_t powers[64];
    uint64_t part[kWarps], slot[2][2][kMostCluster], found[2];
    alignas(16) uint32_t hist[kBins];           // hist and totals: together also the weights of kListed tokens
    alignas(16) uint32_t totals[kBins];
    alignas(16) uint64_t sorted[kListed];
    uint32_t listed, taken, lowest;             // listed: by this CTA; taken: of the first CTA's `sorted`
    struct {
        uint64_t above, inside;
        uint32_t bin, bin2, border, last;
    } cut;
    uint64_t target, all;
};

static_assert(offsetof(Shared, hist) % 16 == 0 && offsetof(Shared, totals) == offsetof(Shared, hist) + kBins * 4 && offsetof(Shared, totals) % 16 == 0 &&
                  offsetof(Shared, sorted) % 16 == 0 && 2 * kBins * 4 >= kListed * 8 && kBins == 4 * kThreads && kListed == 4 * kThreads,
              "vector loads, and arrays that serve twice");

template <int kDtype>
struct Row {
    static constexpr int kEs = kDtype == NINFER_F32 ? 4 : 2, kVec = 16 / kEs;
    const uint8_t *x;
    Shared *shared;
    bool held;                  // the slice, in shared memory
    bool infinite = false;      // some logits are +infinity: they count as 0, all others as -infinity
    uint32_t vocab, shift;      // elements between the last 16-byte boundary and the row's first
    uint32_t v0, v1;            // this CTA's 16-byte vectors, counted from that boundary
    uint32_t rank, ranks;
    int right;                  // 61 - the weights' scale
    uint64_t half;              // of its unit, that far to the left
    uint32_t phase = 0;
    // the row's largest logit, log2(e) / temperature in two floats
    float m = 0.f, c_hi = 0.f, c_lo = 0.f;
    // what is kept: logits above `border`, and at it those up to place `last`; weights of at least `least`
    float border = -FLT_MAX;
    uint32_t last = ~0u;
    uint64_t least = 0;

    __device__ Row(const uint8_t *x, Shared *shared, bool held, uint32_t vocab, int scale) : x(x), shared(shared), held(held), vocab(vocab), right(61 - scale), half((1ull << right) >> 1) {
        shift = (uint32_t)(reinterpret_cast<uintptr_t>(x) & 15) / kEs;
        rank = cluster_ctarank();
        ranks = cluster_nctarank();
    }

    // The 16 bytes of vector v from global memory; -infinity for what is not of the row
    __device__ __forceinline__ uint4 read(uint32_t v) const {
        const int64_t first = (int64_t)v * kVec - shift;
        if (first >= 0 && first + kVec <= vocab) return *reinterpret_cast<const uint4 *>(x + first * kEs);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t i = first + j;
            const bool in = i >= 0 && i < vocab;
            if (kEs == 4) w[j] = in ? reinterpret_cast<const uint32_t *>(x)[i] : 0xff800000u;
            else {
                const uint32_t h = in ? reinterpret_cast<const uint16_t *>(x)[i] : kDtype == NINFER_BF16 ? 0xff80u : 0xfc00u;
                w[j / 2] = j & 1 ? w[j / 2] | h << 16 : h;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // f(four neighbouring logits, the first's place) for the 16-byte vectors from, from + step ... before `to`; NaN and what is not of the row as
    // -infinity. Four at once, and f without branches but one around them all: a thread has few logits, and a chain of dependent
    // instructions takes 150 to 250 cycles for each.
    template <class F>
    __device__ __forceinline__ void over(uint32_t from, uint32_t to, uint32_t step, F f) const {
        extern __shared__ __align__(16) uint4 slice[];
#pragma unroll 1
        for (uint32_t i = from; i < to; i += step) {
            uint4 u;
            if (held) u = slice[i - v0];
            else u = read(i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int q = 0; q < kVec; q += 4) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = fmaxf(element(w, q + j), -INFINITY);
                if (infinite) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = v[j] == INFINITY ? 0.f : -INFINITY;
                }
                f(v, i * kVec - shift + q);
            }
        }
    }
    static __device__ __forceinline__ float element(const uint32_t (&w)[4], int j) {
        const uint32_t h = w[j * kEs / 4];
        return kEs == 4 ? __uint_as_float(h)
               : kDtype == NINFER_BF16 ? __uint_as_float(j & 1 ? h & 0xffff0000u : h << 16)
                                       : __half2float(__ushort_as_half((uint16_t)(j & 1 ? h >> 16 : h & 0xffff)));
    }
    template <class F>
    __device__ __forceinline__ void each(F f) const { over(v0 + threadIdx.x, v1, kThreads, f); }
    // The sum of value(x) over the places for which wanted(x, place) says so; the value of -infinity is 0.
    template <class W, class V>
    __device__ __forceinline__ uint64_t sum_over(uint32_t from, uint32_t to, uint32_t step, W wanted, V value) const {
        uint64_t sum = 0;
        over(from, to, step, [&](const float (&v)[4], uint32_t i) {
            bool in[4], any = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) any |= in[j] = wanted(v[j], i + j);
            if (!any) return;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += value(in[j] ? v[j] : -INFINITY);
        });
        return sum;
    }

    __device__ __forceinline__ float logit_at(uint32_t i) const {
        const float v = fmaxf(load1(x, i, kDtype), -INFINITY);
        return !infinite ? v : v == INFINITY ? 0.f : -INFINITY;
    }
    __device__ __forceinline__ bool kept(float v, uint32_t i) const { return v > border || (v == border && i <= last); }

    // t as two floats (but for the rounding of x - m: 2^-24 t, another one for each token); -100 and less as -100 (and `rest` without a
    // meaning)
    __device__ __forceinline__ float exponent(float v, float &rest) const {
        const float d = v - m, p = d * c_hi;
        rest = fmaf(d, c_lo, fmaf(d, c_hi, -p));
        return fmaxf(p, -100.f);
    }
    __device__ __forceinline__ uint64_t weight(float v) const {
        float rest;
        const float p = exponent(v, rest);
        const float z = fmaf(p, 64.f, kRound);
        const int n = __float_as_int(z) - __float_as_int(kRound);
        const float r = fmaf(z - kRound, -1.f / 64.f, p) + rest;     // exact but for `rest`, at most 1 / 128
        const float y = r * fmaf(r, fmaf(r, 0.05550411f, 0.24022651f), 0.69314718f);        // 2^r - 1
        const int power = (int)shared->powers[n & 63];
        // of 2^(t - n / 64's whole part), times 2^30
        uint32_t w = (uint32_t)(power + __mulhi(power, (__float_as_int(fmaf(y, 0x1p29f, kRound)) - __float_as_int(kRound)) << 3));
        // times 2^(n / 64 + scale - 30), rounded: to the left up to 31, where more than that to the right is left out before, and to the
        // right by the same for all tokens. Nothing is left of what is 2^-100 and less, whatever w.
        const int left = max((n >> 6) + 31, 0), before = left - 31 - (n >> 6);
        w = before < 32 ? w >> before : 0;
        return ((uint64_t)w * (1u << left) + half) >> right;
    }
    // How many bins a logit lies below the largest one, with a fraction; falling logits have rising ones. NaN, which is below no number of
    // bins, for a logit of -infinity at an infinite temperature.
    __device__ __forceinline__ float below(float v, float scale) const { return (m - v) * scale; }
    __device__ __forceinline__ float below(float v) const { return below(v, c_hi * 64.f); }

    // Sum over the CTA; every thread gets it.
    __device__ uint64_t block_sum(uint64_t v) {
#pragma unroll
        for (int k = 16; k; k /= 2) v += __shfl_xor_sync(~0u, v, k);
        __syncthreads();
        if (threadIdx.x % 32 == 0) shared->part[threadIdx.x / 32] = v;
        __syncthreads();
        v = threadIdx.x % 32 < kWarps ? shared->part[threadIdx.x % 32] : 0;
#pragma unroll
        for (int k = 8; k; k /= 2) v += __shfl_xor_sync(~0u, v, k);
        return __shfl_sync(~0u, v, 0);
    }
    // Gives two values of each CTA to all. The slots of two exchanges ago are free: every CTA has read its own before it came to the
    // barrier of the last one. Nothing of another CTA is read behind the barrier, so that a CTA may end there.
    __device__ void exchange(uint64_t v, uint64_t w = 0) {
        phase ^= 1;
        if (threadIdx.x < ranks) {
            st_cluster_u64(&shared->slot[phase][0][rank], threadIdx.x, v);
            st_cluster_u64(&shared->slot[phase][1][rank], threadIdx.x, w);
        }
        join();
    }
    // The sums of both over the cluster.
    __device__ uint64_t collect(int which = 0) const {
        uint64_t t = threadIdx.x % 32 < ranks ? shared->slot[phase][which][threadIdx.x % 32] : 0;
#pragma unroll
        for (int k = 8; k; k /= 2) t += __shfl_xor_sync(~0u, t, k);
        return __shfl_sync(~0u, t, 0);
    }
    __device__ uint64_t cluster_sum(uint64_t v) {
        exchange(block_sum(v));
        return collect();
    }
    // The largest v over the cluster, and the least of least_key.
    __device__ uint64_t cluster_max(uint64_t v, uint32_t &least_key) {
        const uint32_t lane = threadIdx.x % 32;
        const uint32_t low = __reduce_min_sync(~0u, least_key);
        if (lane == 0) atomicMin(&shared->lowest, low);
#pragma unroll
        for (int k = 16; k; k /= 2) v = max(v, __shfl_xor_sync(~0u, v, k));
        if (lane == 0) shared->part[threadIdx.x / 32] = v;
        __syncthreads();
        v = lane < kWarps ? shared->part[lane] : 0;
#pragma unroll
        for (int k = 8; k; k /= 2) v = max(v, __shfl_xor_sync(~0u, v, k));
        exchange(v, shared->lowest);
        v = lane < ranks ? shared->slot[phase][0][lane] : 0;
        least_key = __reduce_min_sync(~0u, lane < ranks ? (uint32_t)shared->slot[phase][1][lane] : ~0u);
#pragma unroll
        for (int k = 8; k; k /= 2) v = max(v, __shfl_xor_sync(~0u, v, k));
        return __shfl_sync(~0u, v, 0);
    }

    // Vectors of a warp, where each has neighbouring ones.
    __device__ __forceinline__ uint32_t warps_part() const { return (v1 - v0 + kWarps - 1) / kWarps; }
    // The first place, in the order of the row, at which the running sum of value(x) over the wanted ones passes target(whole sum).
    // sum(from, to): the thread's part of that sum, over vectors from, from + 32 ..., where it is known cheaper than by adding all up.
    template <class T, class S, class W, class V>
    __device__ uint32_t locate(T target, S part_sum, W wanted, V value, uint64_t *whole = nullptr) {
        const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const uint32_t part = warps_part(), from = min(v0 + warp * part, v1);
        uint64_t sum = part_sum(from + lane, min(from + part, v1));
        uint64_t before;                        // what lies before this CTA, then before its part that has the token, then the part's part
        uint32_t at;
        warps_sums(sum);
        exchange(shared->all);
        const uint64_t total = collect();
        if (whole) *whole = total;
        before = lane < rank ? shared->slot[phase][0][lane] : 0;
#pragma unroll
        for (int k = 8; k; k /= 2) before += __shfl_xor_sync(~0u, before, k);
        before = __shfl_sync(~0u, before, 0);
        const uint64_t goal = target(total);
        if (goal >= before && goal - before < shared->all) {              // one CTA of the cluster
            at = passing(goal - before, before);
            const uint32_t first = v0 + at * part, end = min(first + part, v1), less = (part + kWarps - 1) / kWarps;
            const uint32_t here = min(first + warp * less, end);
            sum = sum_over(here + lane, min(here + less, end), 32, wanted, value);
            __syncthreads();
            warps_sums(sum);
            at = passing(goal - before, before);
            if (warp == at) {
                uint64_t run = goal - before;                        // what is still to be passed
                const uint32_t until = min((here + less) * kVec - shift, vocab);
                for (uint32_t i = here ? here * kVec - shift : 0; i < until; i += 32) {
                    uint64_t u = 0;
                    if (i + lane < until) {
                        const float v = logit_at(i + lane);
                        if (wanted(v, i + lane)) u = value(v);
                    }
#pragma unroll
                    for (int k = 1; k < 32; k *= 2) {
                        const uint64_t w = __shfl_up_sync(~0u, u, k);
                        if (lane >= (uint32_t)k) u += w;
                    }
                    const uint32_t passed = __ballot_sync(~0u, u > run);
                    if (passed) {
                        if (lane < ranks) st_cluster_u64(&shared->found[phase], lane, i + __ffs(passed) - 1);
                        break;
                    }
                    run -= __shfl_sync(~0u, u, 31);
                }
            }
        }
        join();
        return (uint32_t)shared->found[phase];
    }
    // Each warp's sum of v in shared->part, all of them in shared->all.
    __device__ void warps_sums(uint64_t v) {
        const uint32_t lane = threadIdx.x % 32;
#pragma unroll
        for (int k = 16; k; k /= 2) v += __shfl_xor_sync(~0u, v, k);
        __syncthreads();
        if (lane == 0) shared->part[threadIdx.x / 32] = v;
        __syncthreads();
        uint64_t t = lane < kWarps ? shared->part[lane] : 0;
#pragma unroll
        for (int k = 8; k; k /= 2) t += __shfl_xor_sync(~0u, t, k);
        if (threadIdx.x == 0) shared->all = t;
        __syncthreads();
    }
    // Which warp's sum passes `run`; adds those before it to `before`.
    __device__ uint32_t passing(uint64_t run, uint64_t &before) const {
        const uint32_t lane = threadIdx.x % 32;
        const uint64_t mine = lane < kWarps ? shared->part[lane] : 0;
        uint64_t sum = mine;
#pragma unroll
        for (int k = 1; k < kWarps; k *= 2) {
            const uint64_t u = __shfl_up_sync(~0u, sum, k);
            if (lane >= (uint32_t)k) sum += u;
        }
        const uint32_t at = __ffs(__ballot_sync(~0u, lane < kWarps && sum > run)) - 1;
        before += __shfl_sync(~0u, sum - mine, at);
        return at;
    }

    // Adds up the cluster's histograms (counts, or weights of which a bin's largest times `unit` is 1) into `totals` of every CTA: a part each.
    template <bool kWeights>
    __device__ void merge(float unit) {
        join();
        // a lane a bin: 32 neighbouring ones of each CTA at once
        const uint32_t part = kBins / ranks;
        for (uint32_t i = threadIdx.x; i < part; i += kThreads) {
            const uint32_t b = rank * part + i;
            uint32_t word[kMostCluster];
#pragma unroll
            for (uint32_t r = 0; r < kMostCluster; ++r) word[r] = r < ranks ? ld_cluster_u32(&shared->hist[b], r) : 0;
            uint64_t t = 0;
#pragma unroll
            for (uint32_t r = 0; r < kMostCluster; ++r) t += word[r];
            // a weight as a float, of the row's largest one
            const uint32_t sum = kWeights ? __float_as_uint((float)t * unit * exp2f((float)b * (-1.f / 64.f))) : (uint32_t)t;
#pragma unroll
            for (uint32_t r = 0; r < kMostCluster; ++r)
                if (r < ranks) st_cluster_u32(&shared->totals[b], r, sum);
        }
        join();
    }
    // Running sums over the bins' totals up to and with this thread's bins 4 tid .. 4 tid + 3.
    template <class T>
    __device__ void running(T (&sums)[4]) {
        const uint4 u = *reinterpret_cast<const uint4 *>(&shared->totals[threadIdx.x * 4]);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w}, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        T v[4], run = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = sizeof(T) == 4 ? (T)__uint_as_float(w[j]) : (T)w[j];
            run += v[j];
        }
        const T mine = run;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) {
            const T o = __shfl_up_sync(~0u, run, k);
            if (lane >= (uint32_t)k) run += o;
        }
        __syncthreads();
        T *parts = reinterpret_cast<T *>(shared->part);
        if (lane == 31) parts[warp] = run;
        __syncthreads();
        run -= mine;
        for (uint32_t k = 0; k < warp; ++k) run += parts[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[j] = run += v[j];
    }

    __device__ void clear() {
        for (uint32_t i = threadIdx.x; i < kBins; i += kThreads) shared->hist[i] = 0;
        if (threadIdx.x == 0) {
            shared->listed = shared->taken = 0;     // for lists behind the next barrier of the cluster
            shared->cut.bin = shared->cut.bin2 = kBins;
        }
        __syncthreads();
    }
    // A logit's weight into its bin, if it has one.
    __device__ __forceinline__ void count(float v, bool in, float unit) {
        const float at = below(v), z = __fadd_rd(at, kDown);
        // 2^-x of the bin's fraction by its series, within 2^-22
        const float part = (at - (z - kDown)) * (1.f / 64.f), share = fmaf(part, fmaf(part, 0.2402f, -0.69314718f), 1.f) * unit;
        if (in && at < (float)kBins) atomicAdd(&shared->hist[__float_as_uint(z) & (kBins - 1)], __float_as_uint(__fadd_rd(share, kDown)) & 0x7fffffu);
    }
    // Puts a token into the first CTA's `sorted`.
    __device__ __forceinline__ void list(float v, uint32_t place) {
        atomicAdd(&shared->listed, 1u);
        uint32_t at;
        asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(at) : "r"(mapa_shared(smem_u32(&shared->taken), 0)) : "memory");
        if (at < kListed) st_cluster_u64(&shared->sorted[at], 0, (uint64_t)key_of(v) << 32 | (uint32_t)~place);
    }

    // `sorted`, (key, place) of each, in falling order of keys and rising of places, with zeros behind the n first.
    __device__ void sort(uint32_t n) {
        __syncthreads();
        if (n <= kThreads) {        // each one's number is how many are larger
            const uint64_t mine = threadIdx.x < n ? shared->sorted[threadIdx.x] : 0;
            if (threadIdx.x == n) shared->sorted[n] = 0;
            __syncthreads();
            uint32_t larger = 0;
            if (threadIdx.x < n)
                for (uint32_t i = 0; i < n; i += 2) {
                    const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&shared->sorted[i]);
                    larger += (two.x > mine) + (two.y > mine);
                }
            __syncthreads();
            if (threadIdx.x < n) shared->sorted[larger] = mine;
            __syncthreads();
            return;
        }
        uint32_t size = 1024;
        while (size < n) size *= 2;
        for (uint32_t i = n + threadIdx.x; i < size; i += kThreads) shared->sorted[i] = 0;
        __syncthreads();
        for (uint32_t k = 2; k <= size; k *= 2)
            for (uint32_t j = k / 2; j; j /= 2) {
                for (uint32_t i = threadIdx.x; i < size / 2; i += kThreads) {
                    const uint32_t a = 2 * i - (i & (j - 1)), b = a + j;
                    const uint64_t x = shared->sorted[a], y = shared->sorted[b];
                    if ((x < y) == ((a & k) == 0)) {
                        shared->sorted[a] = y;
                        shared->sorted[b] = x;
                    }
                }
                // pairs less than 64 apart stay with a warp
                if (j > 32 || j == 1) __syncthreads();
                else __syncwarp();
            }
    }
    // Running sums of w (4 a thread: numbers 4 tid .. 4 tid + 3) up to and with each.
    __device__ void scan(const uint64_t (&w)[4], uint64_t (&sums)[4]) {
        const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
        uint64_t run = (w[0] + w[1]) + (w[2] + w[3]);
        const uint64_t mine = run;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) {
            const uint64_t o = __shfl_up_sync(~0u, run, k);
            if (lane >= (uint32_t)k) run += o;
        }
        __syncthreads();
        if (lane == 31) shared->part[warp] = run;
        __syncthreads();
        run -= mine;
        for (uint32_t k = 0; k < warp; ++k) run += shared->part[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[j] = run += w[j];
    }
    // Running sums of the weights of `sorted`.
    __device__ void sorted_sums(uint32_t n, uint64_t (&w)[4], uint64_t (&sums)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t i = threadIdx.x * 4 + j;
            w[j] = i < n ? weight(logit_of((uint32_t)(shared->sorted[i] >> 32))) : 0;
        }
        scan(w, sums);
    }
    // Gives the border that the first CTA has put into shared->cut to all.
    __device__ void adopt() {
        phase ^= 1;
        if (rank == 0 && threadIdx.x < ranks) {
            st_cluster_u64(&shared->found[phase], threadIdx.x, (uint64_t)shared->cut.border << 32 | shared->cut.last);
        }
        join();
        border = logit_of((uint32_t)(shared->found[phase] >> 32));
        last = (uint32_t)shared->found[phase];
    }

    // Moves the border to where the kept tokens' counts (kWeighted: weights), from the largest on, reach `target`, which
    // their sum does, its last token included; by the keys' bits, eight at a time.
    template <bool kWeighted>
    __device__ __forceinline__ void by_bits(uint64_t target) {
        uint2 *hist = reinterpret_cast<uint2 *>(shared->hist);                // low and high words
        uint64_t *totals = reinterpret_cast<uint64_t *>(shared->totals);
        uint32_t prefix = 0;
        uint64_t above = 0;
        for (int shift_ = 24; shift_ >= 0; shift_ -= 8) {
            __syncthreads();
            if (threadIdx.x < 256) hist[threadIdx.x] = make_uint2(0, 0);
            __syncthreads();
            each([&](const float (&v)[4], uint32_t i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t k = key_of(v[j]);
                    if (!kept(v[j], i + j) || (shift_ < 24 && k >> (shift_ + 8) != prefix)) continue;
                    uint2 *bin = &hist[k >> shift_ & 255];
                    if (kWeighted) {
                        const uint64_t w = weight(v[j]);
                        const uint32_t old = atomicAdd(&bin->x, (uint32_t)w);
                        const uint32_t more = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
                        if (more) atomicAdd(&bin->y, more);
                    } else atomicAdd(&bin->x, 1u);
                }
            });
            join();
            if (threadIdx.x < 256) {
                // a lane a CTA
                const uint32_t from = threadIdx.x % ranks, b = rank * (256 / ranks) + threadIdx.x / ranks;
                uint64_t t = ld_cluster_u64(&hist[b], from);
                for (uint32_t k = ranks / 2; k; k /= 2) t += __shfl_xor_sync(~0u, t, k);
                st_cluster_u64(&totals[b], from, t);
            }
            join();
            // from the highest bin on: the one in which the sum reaches the target
            const uint64_t mine = threadIdx.x < 256 ? totals[255 - threadIdx.x] : 0;
            uint64_t sums[4], w[4] = {mine, 0, 0, 0};
            scan(w, sums);
            const uint64_t before = above + sums[0] - mine;
            if (mine && before < target && target - before <= mine) {
                shared->cut.above = before;
                shared->cut.inside = mine;
                shared->cut.bin = 255 - threadIdx.x;
            }
            __syncthreads();
            above = shared->cut.above;
            prefix = prefix << 8 | shared->cut.bin;
        }
        // the border's key is known; of the tokens that share it, the first in the row's order
        const float edge = logit_of(prefix);
        const uint64_t one = kWeighted ? weight(edge) : 1, ties = shared->cut.inside / one;
        const uint64_t wanted = (target - above + one - 1) / one;
        uint32_t at = edge == border ? last : ~0u;
        if (wanted < ties) {
            auto tied = [&](float v, uint32_t i) { return v == edge && kept(v, i); };
            auto one_each = [](float v) -> uint64_t { return v > -INFINITY; };
            at = locate([&](uint64_t) { return wanted - 1; }, [&](uint32_t from, uint32_t to) { return sum_over(from, to, 32, tied, one_each); }, tied, one_each);
        }
        border = edge;
        last = at;
    }
};

// The row with its border moved, for the rows that come to it; out of line, and of a copy, so that others stay in registers.
template <bool kWeighted, int kDtype>
__device__ __noinline__ Row<kDtype> cut_by_bits(Row<kDtype> row, uint64_t target) {
    row.template by_bits<kWeighted>(target);
    return row;
}

template <int kDtype>
__global__ void __launch_bounds__(kThreads, kResident) sample_kernel(const __grid_constant__ SampleParams p) {
    using R = Row<kDtype>;
    extern __shared__ __align__(16) uint4 slice[];
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x, lane = tid % 32;
    if (tid < 64) s.powers[tid] = kPowers[tid];
    if (tid == 64) {
        s.lowest = ~0u;
        s.listed = s.taken = 0;
    }
    __syncthreads();
    cluster_arrive();
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_sample_args &a = p.a;
    const uint32_t ranks = cluster_nctarank(), vocab = (uint32_t)a.vocab;
    const uint64_t b = blockIdx.x / ranks;
    R row(static_cast<const uint8_t *>(a.logits) + b * a.stride * R::kEs, &s, p.held, vocab, p.scale);
    const uint32_t all = (row.shift + vocab + R::kVec - 1) / R::kVec;      // the row's 16-byte vectors, from the boundary before it
    row.v0 = min(row.rank * p.vectors, all);
    row.v1 = min(row.v0 + p.vectors, all);

    const float temperature = a.temperature ? a.temperature[b] : 1.f, top_p = a.top_p ? a.top_p[b] : 1.f;
    const float min_p = a.min_p ? a.min_p[b] : 0.f, random = a.random[b];
    const int32_t top_k = a.top_k ? a.top_k[b] : 0;
    // the row into shared memory, and its largest logit, with the first place that has it where that is the answer
    const bool greedy = !(temperature > 0.f);
    float most = -INFINITY;
    uint32_t place = ~0u;
    auto larger = [&](float v, uint32_t i) {
        if (v > most) {
            most = v;
            place = i;
        }
    };
    if (p.held) {
        constexpr int kAhead = 8;
        for (uint32_t v = row.v0 + tid; v < row.v1; v += kAhead * kThreads) {
            uint4 u[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (v + j * kThreads < row.v1) u[j] = row.read(v + j * kThreads);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (v + j * kThreads >= row.v1) break;
                slice[v + j * kThreads - row.v0] = u[j];
                const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
                for (int e = 0; e < R::kVec; ++e) {
                    const float y = R::element(w, e);
                    if (greedy) larger(y, (v + j * kThreads) * R::kVec - row.shift + e);
                    else most = fmaxf(most, y);
                }
            }
        }
    } else
        row.each([&](const float (&v)[4], uint32_t i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) larger(v[j], i + j);
        });
    uint32_t lowest = most == -INFINITY ? ~0u : key_of(most);       // of the threads' largest, which top-k looks at
    __syncwarp();
    cluster_wait();         // every CTA of the row has begun: what follows is stored into the others' shared memory
    const uint64_t best = row.cluster_max((uint64_t)key_of(most) << 32 | (uint32_t)~place, lowest);
    const float top = logit_of((uint32_t)(best >> 32));
    const bool lead = tid == 0 && row.rank == 0, none = top == -INFINITY;
    if (none || greedy) {
        if (lead) {
            a.tokens[b] = none ? -1 : (int32_t)~(uint32_t)best;
            if (a.logprobs) a.logprobs[b] = none ? -INFINITY : 0.f;
        }
        return;
    }
    row.infinite = top == INFINITY;
    row.m = row.infinite ? 0.f : top;
    if (row.infinite) most = most == INFINITY ? 0.f : -INFINITY;
    // log2(e) / temperature, of which 64 times (bins) are a float too
    const float warm = fmaxf(temperature, 0x1p-119f);
    row.c_hi = __fdiv_rn(1.44269504f, warm);
    row.c_lo = __fdiv_rn(fmaf(-row.c_hi, warm, 1.44269504f) + 1.92596299e-8f, warm);
    if (!isfinite(row.c_lo)) row.c_lo = 0.f;
    if (min_p > 0.f) row.least = times(fminf(min_p, 1.f), 1ull << p.scale, true);
    const bool by_k = top_k > 0 && (uint32_t)top_k < vocab, by_p = top_p < 1.f, by_m = min_p > 0.f;
    // the share of a whole that the random number says, and the logarithm of a token's share
    auto share = [&](uint64_t whole) {
        return min(times(fminf(fmaxf(random, 0.f), 1.f), whole, false), whole - 1);
    };
    auto answer = [&](uint32_t token, float logit, uint64_t whole) {
        a.tokens[b] = (int32_t)token;
        if (!a.logprobs) return;
        float rest;
        const float t = row.exponent(logit, rest);
        // the sum in units of the largest weight, which is 2^scale and among those kept
        a.logprobs[b] = (t + rest) * 0.69314718f - log1pf((float)(whole - (1ull << p.scale)) * __uint_as_float((uint32_t)(127 - p.scale) << 23));
    };

    // few tokens kept: those down to bin `few` hold them all
    uint32_t few = kBins;
    auto reach = [&](uint64_t wanted) {     // the bin in which the counts reach it, what lies above, and both
        uint64_t sums[4];
        row.running(sums);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint64_t before = sums[j] - s.totals[tid * 4 + j];
            if (before < wanted && sums[j] >= wanted) {
                s.cut.bin = tid * 4 + j;
                s.cut.above = before;
                s.cut.inside = sums[j];
            }
        }
        __syncthreads();
        return s.cut.bin;
    };
    // What may be kept lies less than `limit` below the largest, in units of `scale`. With one logit for each thread, its largest: where top_k
    // of those are, or as much weight as top_p wants, all that is kept is, and hardly more than that while it is few.
    float limit = INFINITY, scale = row.c_hi * 64.f;
    uint64_t all_weights = 0;
    if (by_k) {
        if ((uint32_t)top_k <= p.few_k) {
            scale = (float)(kBins - 1) / (row.m - logit_of(lowest));
            if (!(fabsf(scale) < FLT_MAX)) scale = 0.f;            // one logit only; otherwise what lies off by rounding goes to the last bin
            row.clear();
            if (most > -INFINITY) atomicAdd(&s.hist[min((uint32_t)row.below(most, scale), kBins - 1)], 1u);
            row.template merge<false>(1.f);
            few = reach((uint32_t)top_k);
            limit = few < kBins - 1 ? (float)(few + 1) : INFINITY;
        }
    } else if (by_p) {
        uint64_t sum = row.sum_over(row.v0 + tid, row.v1, kThreads, [](float v, uint32_t) { return v > -INFINITY; }, [&](float v) { return row.weight(v); });
        sum = row.block_sum(sum);
        row.exchange(sum);
        all_weights = row.collect();
        row.clear();
        row.count(most, most > -INFINITY, p.unit);
        row.template merge<true>(1.f / p.unit);
        float sums[4];
        row.running(sums);
        const float goal = (float)times(fmaxf(top_p, 0.f), all_weights, true) * __uint_as_float((uint32_t)(127 - p.scale) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (sums[j] * (1.f - p.slack) >= goal) atomicMin(&s.cut.bin, tid * 4 + j);
        __syncthreads();
        few = s.cut.bin;
        limit = (float)(few + 1);
    } else if (by_m) {
        few = 0;
        limit = -64.f * log2f(fminf(min_p, 1.f)) * (1.f + 0x1p-20f) + 0.01f;      // a little more, for what the logarithm and `below` round
    }
    if (few < kBins) {
        row.each([&](const float (&v)[4], uint32_t i) {
            bool in[4], any = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) any |= in[j] = v[j] > -INFINITY && row.below(v[j], scale) < limit;
            if (!any) return;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in[j]) row.list(v[j], i + j);
        });
        __syncthreads();
        row.exchange(s.listed);
        const uint32_t n = (uint32_t)row.collect();
        if (n <= kListed) {
            if (row.rank == 0) {
                row.sort(n);
                uint64_t w[4], sums[4];
                row.sorted_sums(n, w, sums);
                // A, its sum, and where B and C end: a number of `sorted` each
                const uint32_t first_k = by_k ? min((uint32_t)top_k, n) : n;
                uint64_t whole = 0;
                if (first_k && tid == (first_k - 1) / 4) s.target = sums[(first_k - 1) % 4];
                __syncthreads();
                whole = s.target;
                __syncthreads();
                if (tid == 0) s.cut.bin2 = 0;
                __syncthreads();
                if (!by_k && by_p) whole = all_weights;
                const uint64_t goal = by_p ? max(times(fmaxf(top_p, 0.f), whole, true), (uint64_t)1) : ~0ull;
                uint64_t mine = 0;
                uint32_t end = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t i = tid * 4 + j;
                    const bool in = i < first_k && sums[j] - w[j] < goal && w[j] >= row.least;
                    if (in) {
                        mine += w[j];
                        end = i + 1;
                    }
                }
                end = __reduce_max_sync(~0u, end);
                if (lane == 0) atomicMax(&s.cut.bin2, end);
                whole = row.block_sum(mine);        // of those kept: the first s.cut.bin2
                const uint32_t kept = s.cut.bin2;
                const uint64_t passed = share(whole);
                // sorted by places, the one whose running sum is the first past the share
                uint64_t *weights = reinterpret_cast<uint64_t *>(s.hist);       // hist and totals, which are done with
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t i = tid * 4 + j;
                    if (i >= kept) break;
                    weights[i] = w[j];
                    s.sorted[i] = (s.sorted[i] & 0xffffffffull) << 32 | i;      // ~place, number
                }
                row.sort(kept);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = tid * 4 + j < kept ? weights[(uint32_t)s.sorted[tid * 4 + j]] : 0;
                row.scan(w, sums);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (sums[j] - w[j] <= passed && passed < sums[j]) {
                        const uint32_t place = ~(uint32_t)(s.sorted[tid * 4 + j] >> 32);
                        answer(place, row.logit_at(place), whole);
                    }
            }
            return;
        }
    }
    if (by_k) {
        // many: the border alone
        row.clear();
        row.each([&](const float (&v)[4], uint32_t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float at = row.below(v[j]);
                if (at < (float)kBins) atomicAdd(&s.hist[__float_as_uint(__fadd_rd(at, kDown)) & (kBins - 1)], 1u);
            }
        });
        row.template merge<false>(1.f);
        const uint32_t bin = reach((uint32_t)top_k);
        const uint64_t above = s.cut.above, inside = s.cut.inside - above;
        __syncthreads();
        if (bin < kBins && inside <= kListed) {
            row.each([&](const float (&v)[4], uint32_t i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float at = row.below(v[j]);
                    if (at >= (float)bin && at < (float)(bin + 1)) row.list(v[j], i + j);
                }
            });
            join();
            if (row.rank == 0) {
                row.sort((uint32_t)inside);
                if (tid == 0) {
                    const uint64_t e = s.sorted[(uint32_t)(top_k - above) - 1];
                    s.cut.border = (uint32_t)(e >> 32);
                    s.cut.last = (uint32_t)~e;
                }
                __syncthreads();
            }
            row.adopt();
        } else {
            uint64_t count = 0;
            row.each([&](const float (&v)[4], uint32_t) {
#pragma unroll
                for (int j = 0; j < 4; ++j) count += v[j] > -INFINITY;
            });
            count = row.cluster_sum(count);
            if ((uint64_t)top_k < count) row = cut_by_bits<false>(row, (uint64_t)top_k);
        }
    }
    // by warps' parts: the exact weights of what is surely kept, and from where to where it is not sure
    uint64_t sure_sum = 0;
    float sure = 0.f, unsure = INFINITY;
    if (by_p) {
        // the exact sum, and the weights by bins
        row.clear();
        uint64_t sum = 0;
        row.each([&](const float (&v)[4], uint32_t i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = row.kept(v[j], i + j);
                if (by_k) {
                    const uint64_t w = row.weight(v[j]);
                    sum += in ? w : 0;
                }
                row.count(v[j], in, p.unit);
            }
        });
        if (by_k) {
            sum = row.block_sum(sum);
            row.exchange(sum);
            sum = row.collect();
        } else sum = all_weights;
        const uint64_t target = max(times(fmaxf(top_p, 0.f), sum, true), (uint64_t)1);
        row.template merge<true>(1.f / p.unit);
        // the border lies between where the bins' sums with all that they may lack reach the target and where they do with as much less
        const float goal = (float)target * __uint_as_float((uint32_t)(127 - p.scale) << 23);
        float sums[4];
        row.running(sums);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (sums[j] * (1.f + p.slack) >= goal) atomicMin(&s.cut.bin, tid * 4 + j);
            if (sums[j] * (1.f - p.slack) >= goal) atomicMin(&s.cut.bin2, tid * 4 + j);
        }
        __syncthreads();
        const uint32_t bin = s.cut.bin, bin2 = s.cut.bin2;
        bool done = bin2 < kBins;
        if (done) {
            uint64_t over = 0;
            const float low = (float)bin, limit = (float)(bin2 + 1);
            const uint32_t part = row.warps_part(), from = min(row.v0 + tid / 32 * part, row.v1);
            row.over(from + lane, min(from + part, row.v1), 32, [&](const float (&v)[4], uint32_t i) {
                bool in[4], any = false;
                float at[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    at[j] = row.below(v[j]);
                    any |= in[j] = at[j] < limit && row.kept(v[j], i + j);
                }
                if (!any) return;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t w = row.weight(v[j]);
                    over += in[j] && at[j] < low ? w : 0;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in[j] && at[j] >= low) row.list(v[j], i + j);
            });
            const uint64_t mine = over;
            over = row.block_sum(over);
            row.exchange(over, s.listed);
            over = row.collect();
            const uint32_t n = (uint32_t)row.collect(1);
            done = n <= kListed;
            if (done) {
                if (row.rank == 0) {
                    row.sort(n);
                    uint64_t w[4], sums_[4];
                    row.sorted_sums(n, w, sums_);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t i = tid * 4 + j;
                        if (i < n && over + sums_[j] - w[j] < target && over + sums_[j] >= target) {
                            s.cut.border = (uint32_t)(s.sorted[i] >> 32);
                            s.cut.last = (uint32_t)~s.sorted[i];
                        }
                    }
                    __syncthreads();
                }
                row.adopt();
                if (!by_m) {
                    sure_sum = mine;
                    sure = low;
                    unsure = limit;
                }
            }
        }
        if (!done) row = cut_by_bits<true>(row, target);
    }
    uint64_t whole;
    const uint64_t least = row.least;
    auto kept = [&](float v, uint32_t i) { return row.kept(v, i); };
    auto value = [&](float v) -> uint64_t {
        const uint64_t w = row.weight(v);
        return w >= least ? w : 0;
    };
    const uint32_t token = row.locate(
        share,
        [&](uint32_t from, uint32_t to) {
            return sure_sum + row.sum_over(from, to, 32, [&](float v, uint32_t i) {
                const float at = row.below(v);
                return !(at < sure) && !(at >= unsure) && row.kept(v, i);
            }, value);
        },
        kept, value, &whole);
    if (lead) answer(token, row.logit_at(token), whole);
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
    // a row's controls have been read when its results are written
    const Span logits(a.logits, a.vocab * dtype_size(a.dtype), a.rows, a.stride * dtype_size(a.dtype));
    const Span chosen(a.tokens, a.rows * 4), logprobs(a.logprobs, a.rows * 4);
    bool shared = chosen.meets(logprobs) || chosen.meets(logits) || logprobs.meets(logits);
    for (const void *q : {(const void *)a.temperature, (const void *)a.top_p, (const void *)a.min_p, (const void *)a.top_k, (const void *)a.random}) {
        const Span in(q, a.rows * 4);
        shared = shared || (chosen.meets(in) && !chosen.same(in)) || (logprobs.meets(in) && !logprobs.same(in));
    }
    if (shared) return fail(NINFER_ERR_INVALID_ARGUMENT, "sample: tokens and logprobs may not overlap logits, each other or parts of the controls");
    DeviceInfo d;
    int st = device_info(&d);
    if (st) return st;
    SampleParams p;
    p.a = a;
    int bits = 1;
    while ((1ull << bits) < a.vocab) ++bits;
    p.scale = 62 - bits;
    // CTAs a row: as many as make a slice fit two times into an SM, more where few rows leave SMs without work
    const uint64_t es = dtype_size(a.dtype), vectors = (a.vocab * es + 15) / 16 + 1;
    unsigned ranks = 1;
    while (ranks < kMostCluster && ((vectors + ranks - 1) / ranks * 16 > kSliceBytes ||
                                    (a.rows * ranks * 2 <= (uint64_t)d.sms * kResident && a.vocab > (uint64_t)ranks * kLeastSlice)))
        ranks *= 2;
    p.vectors = (uint32_t)((vectors + ranks - 1) / ranks);
    // a CTA's sums in 32 bits; beside a unit's rounding, the bins' and the floats' that add them up are under 2^-12
    const uint64_t tokens = p.vectors * (16 / es);
    p.unit = (float)std::min<uint64_t>(65535, 0xfffffff0ull / tokens);
    p.slack = 0x1p-12f + 1.02f / p.unit;
    p.held = p.vectors * 16ull <= kMostSliceBytes;
    // Listing costs by top_k, a border's histogram by the tokens of a thread, so that the one ends where top_k is 12 times these (us, listed and
    // by histogram: a row of 248320 with top_k 200 14.5 and 17.8, 400 21.0 and 18.1; 64 rows of 4099, 50 12.2 and 13.0, 200 16.4 and 13.4). Where
    // clusters have to wait for others, listing frees most of their CTAs sooner (64 rows of 248320, 800 92 and 117, 1024 119 and 119). Fewer threads than
    // top_k or hardly more have no maxima that bound it (256 rows of 32003 in a CTA each, 380 42.7 and 45.5, 800 54.9 and 48.0).
    const uint64_t each = (a.vocab + ranks * kThreads - 1) / (ranks * kThreads), most = ranks * kThreads * 4 / 5;
    p.few_k = (uint32_t)std::min<uint64_t>(most, a.rows * ranks > (uint64_t)d.sms * kResident ? kFew : std::min<uint64_t>(kFew, 12 * each));
    const auto kernel = a.dtype == NINFER_F32    ? sample_kernel<NINFER_F32>
                        : a.dtype == NINFER_BF16 ? sample_kernel<NINFER_BF16>
                                                 : sample_kernel<NINFER_F16>;
    const uint32_t smem = p.held ? p.vectors * 16 : 0;
    st = set_smem_attribute(reinterpret_cast<const void *>(kernel), kMostSliceBytes);
    if (!st && ranks > 8) st = set_wide_clusters(reinterpret_cast<const void *>(kernel));
    if (st) return st;
    return launch_clusters("sample", ranks, kernel, dim3((unsigned)(a.rows * ranks)), dim3(kThreads), smem, (cudaStream_t)stream, p);
}
