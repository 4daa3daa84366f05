// ninfer_gated_delta: the gated delta rule, S <- e^g S + beta k (v - e^g S^T k)^T,
// out = scale S^T q, over a k_dim x v_dim state of fp32 per request and value head.
//
// The columns of a state do not see each other: S^T k, u = beta (v - e^g S^T k), the update k u^T and S^T q need, for
// one column of S, only that column and the k and q that all columns share. The kernels divide the states by columns.
//
// One token a request (step_kernel): with a = S^T k and b = S^T q of the old state, out = scale (e^g b + (k . q) u), so
// that one pass over the state gives both sums and a second one, in registers, updates it: the state is read once and
// written once, and HBM bounds it.
// Several (prepare_kernel, chunk_kernel): 32 tokens at once, by matrix products whose state stays in registers from a
// request's first token to its last. The chain of dependent products bounds it (the tensor cores are busy for a third of it).
//
// Measured: 64 requests of one token, 48 states of 128 x 128 each, 405 MB, 69 us (5.9 TB/s; with 128 columns a CTA, one CTA an SM, 104).
// A prompt of 8001 tokens with 48 heads: 93 us of preparation and 522 of chunks, 2.07 us each, 620 in all; token by token in fp32, four
// lanes a column, 7390.
#include <cmath>

#include "decode.cuh"
#include "gemv.h"
#include "ninfer_layer.h"
#include "overlap.h"

namespace ninfer {
namespace {

constexpr int kStepThreads = 256;

struct DeltaParams {
    ninfer_gated_delta_args a;
    FastDiv slabs, heads, group;    // of a head's columns, value heads, value heads a key head
};

struct Part {
    uint32_t request, head, key_head, column;   // `column`: the slab's first
    uint64_t state;                             // element of the state's first
    bool none, fresh;
};

// What block `index` works on; none: the request has no slot.
__device__ __forceinline__ Part part_of(const DeltaParams &p, uint32_t index, uint32_t slab) {
    const ninfer_gated_delta_args &a = p.a;
    const uint32_t row = p.slabs.div(index);
    Part t;
    t.column = (index - row * p.slabs.d) * slab;
    t.request = p.heads.div(row);
    t.head = row - t.request * p.heads.d;
    t.key_head = p.group.div(t.head);
    const int64_t slot = a.state_slots ? (int64_t)a.state_slots[t.request] : (int64_t)t.request;
    t.none = slot < 0 || (uint64_t)slot >= a.slots;
    if (slot >= 0 && t.none && a.status && threadIdx.x == 0) atomicOr(a.status, NINFER_DELTA_BAD_SLOT);
    t.fresh = a.lengths && a.lengths[t.request] <= 0;
    t.state = t.none ? 0 : (uint64_t)slot * a.slot_stride + (uint64_t)t.head * a.k_dim * a.v_dim;
    return t;
}

// One token a request. kLanes lanes hold a row's columns, four each; 256 / kLanes rows at a time, kIter times.
template <int kLanes, int kIter>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const __grid_constant__ DeltaParams p) {
    constexpr int kRows = kStepThreads / kLanes, kSlab = kLanes * 4, kWarps = kStepThreads / 32;
    __shared__ float ks[256], qs[256], dots[3][kWarps], part[kWarps][2][kSlab];
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_gated_delta_args &a = p.a;
    const Part t = part_of(p, blockIdx.x, kSlab);
    if (t.none) return;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32, k_dim = (uint32_t)a.k_dim, v_dim = (uint32_t)a.v_dim;
    const uint32_t first = tid / kLanes, column = t.column + tid % kLanes * 4;
    const bool inside = column < v_dim;
    float4 *state = reinterpret_cast<float4 *>(a.state + t.state + column);
    const uint32_t step = v_dim / 4;        // float4 a row
    float4 s[kIter];
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
        s[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t r = first + j * kRows;
        if (r < k_dim && inside && !t.fresh) s[j] = state[r * step];
    }
    const uint64_t token = t.request;
    float k = 0.f, q = 0.f;
    if (tid < k_dim) {
        k = load1(a.k, token * a.k_token_stride + t.key_head * a.k_head_stride + tid, a.dtype);
        q = load1(a.q, token * a.q_token_stride + t.key_head * a.q_head_stride + tid, a.dtype);
    }
    float v[4] = {};
    if (inside) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load1(a.v, token * a.v_token_stride + t.head * a.v_head_stride + column + i, a.dtype);
    }
    const float decay = expf(a.log_decay[token * a.decay_stride + t.head]), beta = a.beta[token * a.beta_stride + t.head];
    ks[tid] = k;
    qs[tid] = q;
    float kk = k * k, qq = q * q, kq = k * q;
#pragma unroll
    for (int i = 16; i; i /= 2) {
        kk += __shfl_xor_sync(~0u, kk, i);
        qq += __shfl_xor_sync(~0u, qq, i);
        kq += __shfl_xor_sync(~0u, kq, i);
    }
    if (lane == 0) {
        dots[0][warp] = kk;
        dots[1][warp] = qq;
        dots[2][warp] = kq;
    }
    __syncthreads();
    kk = qq = kq = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        kk += dots[0][w];
        qq += dots[1][w];
        kq += dots[2][w];
    }
    const float k_scale = a.norm_eps < 0.f ? 1.f : 1.f / sqrtf(kk + a.norm_eps), q_scale = a.norm_eps < 0.f ? 1.f : 1.f / sqrtf(qq + a.norm_eps);
    float x[8] = {};        // S^T k and S^T q of the four columns
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
        const uint32_t r = first + j * kRows;
        const float kr = r < 256 ? ks[r] : 0.f, qr = r < 256 ? qs[r] : 0.f;
        x[0] = fmaf(s[j].x, kr, x[0]);
        x[1] = fmaf(s[j].y, kr, x[1]);
        x[2] = fmaf(s[j].z, kr, x[2]);
        x[3] = fmaf(s[j].w, kr, x[3]);
        x[4] = fmaf(s[j].x, qr, x[4]);
        x[5] = fmaf(s[j].y, qr, x[5]);
        x[6] = fmaf(s[j].z, qr, x[6]);
        x[7] = fmaf(s[j].w, qr, x[7]);
    }
#pragma unroll
    for (int i = kLanes; i < 32; i *= 2)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += __shfl_xor_sync(~0u, x[j], i);
    if (lane < kLanes) {
        *reinterpret_cast<float4 *>(&part[warp][0][lane * 4]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(&part[warp][1][lane * 4]) = make_float4(x[4], x[5], x[6], x[7]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float4 m = *reinterpret_cast<const float4 *>(&part[w][0][tid % kLanes * 4]), n = *reinterpret_cast<const float4 *>(&part[w][1][tid % kLanes * 4]);
        x[0] += m.x; x[1] += m.y; x[2] += m.z; x[3] += m.w;
        x[4] += n.x; x[5] += n.y; x[6] += n.z; x[7] += n.w;
    }
    if (!inside) return;
    float u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = beta * (v[i] - decay * (k_scale * x[i]));
    if (first == 0) {
        const uint64_t at = (token * a.v_heads + t.head) * v_dim + column;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store1(a.out, at + i, a.out_dtype, a.scale * q_scale * (decay * x[4 + i] + k_scale * kq * u[i]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] *= k_scale;
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
        const uint32_t r = first + j * kRows;
        if (r >= k_dim) break;
        const float kr = ks[r];
        s[j].x = fmaf(kr, u[0], decay * s[j].x);
        s[j].y = fmaf(kr, u[1], decay * s[j].y);
        s[j].z = fmaf(kr, u[2], decay * s[j].z);
        s[j].w = fmaf(kr, u[3], decay * s[j].w);
        state[r * step] = s[j];
    }
}

// ---------------------------------------------------------------- prompts ---
// A request's tokens go in chunks of 32. With G_t the chunk's log decays summed up to and with token t, S the state before it,
//   U = T diag(beta) (V - diag(e^G) K S),     T = (I + A)^-1, A_ts = beta_t e^(G_t - G_s) k_t . k_s for s < t, else 0
//   O = scale (diag(e^G) Q S + P U),          P_ts = e^(G_t - G_s) q_t . k_s for s <= t, else 0
//   S <- e^(G_last) S + K^T diag(e^(G_last - G)) U
// T diag(beta) and P need no state: prepare_kernel makes them for all chunks at once, chunk_kernel goes through them.
// Every row of K and Q is a row of binary16 times its own scale. T's rows take their keys' scales, so that U comes out as what it adds to the
// state, of one size with it, and P is made of the rows without their scales: a small key or query beside large ones keeps its bits.
constexpr int kChunk = 32, kPrepareThreads = 128;
constexpr int kNumbers = 132;                                       // floats of a chunk and head: below
enum { kOfK = 0, kOfQ = 32, kOfU = 64, kOfP = 96, kLeft = 128, kOfT };   // e^G k's scale, scale e^G q's, e^(G_last - G), scale q's and P's; e^G_last, T's
constexpr uint32_t kTriStride = kChunk * 2 + 16, kTrianglesBytes = 4 * kChunk * kTriStride;     // T high and low, P high and low
constexpr uint32_t kHeadBytes = kTrianglesBytes + kNumbers * 4;

// What lies in the workspace: for every chunk and key head K and Q as binary16 (f32: two terms each), [term][K, Q][token][k_dim];
// then for every chunk and value head the triangles, [which][t][s], and the numbers. Rows are 16 bytes longer than their elements, as
// they are to lie in shared memory (eight of them in different banks), so that one copy moves a chunk's.
struct ChunkParams {
    DeltaParams d;
    uint8_t *rows, *heads;
    uint64_t rows_bytes;        // of a chunk and key head
    uint32_t wide;              // k_dim rounded up to the kernel's steps of 16
    uint32_t slab;              // columns of a state a CTA
    uint32_t *error;            // the library's error word
    long long wait_limit;
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void load_matrices_turned(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void store_matrices_turned(uint32_t at, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// 16 bytes from global to shared memory; an arrival at a barrier once the thread's copies so far have landed.
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Two floats as two binary16 terms each: 22 bits of every value from 2^-14 of 1 on.
__device__ __forceinline__ void split(float x, float y, uint32_t &high, uint32_t &low) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    high = *reinterpret_cast<const uint32_t *>(&h);
    low = *reinterpret_cast<const uint32_t *>(&l);
}

// The power of two that takes `most` (a row's largest magnitude) to 2^13 .. 2^14, so that its binary16 terms lose nothing
// above 2^-38 of it, and its inverse.
__device__ __forceinline__ float power_for(float most) { return __uint_as_float((uint32_t)min(max(267 - (int)(__float_as_uint(most) >> 23), 1), 253) << 23); }
__device__ __forceinline__ float inverse_power(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
    return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}
// The largest magnitude; NaN where one is.
__device__ __forceinline__ float most_of(float m, float v, float w) {
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(v), "f"(w));
    return m;
}
__device__ __forceinline__ float most_of(float m, float v) { return most_of(m, v, v); }

// What is not finite goes into no product with other tokens' values: zeros times it would make NaN of earlier ones, and the power of two
// that fits it zeros. Of two columns by 32 tokens (y[n][e]: token 8 n + 2 (lane % 4) + e % 2 of column e / 2, the same two of a quad of lanes) the
// first tokens that are not finite, in a byte each.
constexpr uint32_t kAllFinite = kChunk | kChunk << 8;
__device__ __forceinline__ uint32_t first_spoilt(const float (&y)[4][4]) {
    uint32_t first[2] = {kChunk, kChunk};
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (!(fabsf(y[n][e]) < INFINITY)) first[e / 2] = min(first[e / 2], n * 8 + threadIdx.x % 4 * 2 + e % 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 1; k < 4; k *= 2) first[i] = min(first[i], __shfl_xor_sync(~0u, first[i], k));
    return first[0] | first[1] << 8;
}
// `value` instead of the values from there on, of kCount times 8 tokens from 8 n0 on.
template <int kCount>
__device__ __forceinline__ void from_spoilt(uint32_t first, float (&y)[kCount][4], float value, uint32_t n0 = 0) {
#pragma unroll
    for (int n = 0; n < kCount; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((n0 + n) * 8 + threadIdx.x % 4 * 2 + e % 2 >= (first >> e / 2 * 8 & 255)) y[n][e] = value;
}

// A request's tokens, and the chunks that are its own: distinct ones for requests whose tokens are, in whatever order they lie. A chunk of 32 tokens
// holds one with 31 over a multiple of 32, whose 32nd is its number; a request's last chunk, if it has fewer, comes behind all those.
struct Range {
    int32_t begin, end;
    uint32_t first, whole, last, chunks;        // number of the first whole chunk, how many, number of one with fewer tokens, chunks in all
};
__device__ __forceinline__ Range range_of(const ninfer_gated_delta_args &a, uint32_t request) {
    const int32_t most = (int32_t)a.tokens;
    Range r;
    r.begin = min(max(a.offsets[request], 0), most);
    r.end = min(max(a.offsets[request + 1], 0), most);
    const uint32_t count = r.end > r.begin ? r.end - r.begin : 0;
    r.first = (uint32_t)r.begin / kChunk;
    r.whole = count / kChunk;
    r.last = (uint32_t)most / kChunk + request;
    r.chunks = (count + kChunk - 1) / kChunk;
    return r;
}

constexpr uint32_t kTriRow = kChunk + 4, kTriSmem = kPrepareThreads / 32 * kChunk * kTriRow * 4;

// 32 rows by 32 columns, a lane's `x` its column, as two binary16 matrices under the power of two that fits the largest; its inverse.
__device__ __forceinline__ float put_matrix(uint8_t *to, const float (&x)[kChunk], float most, uint32_t lane) {
#pragma unroll
    for (int k = 16; k; k /= 2) most = fmaxf(most, __shfl_xor_sync(~0u, most, k));
    const float up = power_for(most);
#pragma unroll
    for (int t = 0; t < kChunk; ++t) {
        const float y = x[t] * up;
        const __half high = __float2half_rn(y);
        __half *at = reinterpret_cast<__half *>(to + t * kTriStride) + lane;
        at[0] = high;
        at[kChunk * kTriStride / 2] = __float2half_rn(y - __half2float(high));
    }
    return inverse_power(up);
}

// A CTA for every chunk and key head. kTerms: binary16 terms of k and q, 1 where they have 16 bits themselves.
template <int kTerms>
__global__ void __launch_bounds__(kPrepareThreads, 6) prepare_kernel(const __grid_constant__ ChunkParams p) {
    extern __shared__ __align__(16) uint8_t smem[];     // K and Q in binary16, rows of p.wide + 8; then a triangle of each warp
    __shared__ float dots[2][kChunk][kChunk + 1], scales[2][kChunk];
    __shared__ float4 sums[kPrepareThreads / 32][kChunk];      // the log decays' sums in two floats, beta
    __shared__ uint32_t found;
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_gated_delta_args &a = p.d.a;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32, k_dim = (uint32_t)a.k_dim;
    const uint32_t chunk = blockIdx.x / (uint32_t)a.k_heads, key_head = blockIdx.x % (uint32_t)a.k_heads;
    // the request that this chunk belongs to
    const uint32_t whole = (uint32_t)a.tokens / kChunk;
    if (tid == 0) found = ~0u;
    __syncthreads();
    if (chunk < whole)
        for (uint32_t r = tid; r < (uint32_t)a.requests; r += kPrepareThreads) {
            const Range c = range_of(a, r);
            if (chunk - c.first < c.whole) found = r;
        }
    __syncthreads();
    const uint32_t request = chunk < whole ? found : chunk - whole;
    if (request == ~0u) return;
    const Range range = range_of(a, request);
    const uint32_t place = chunk < whole ? chunk - range.first : range.whole;        // among the request's
    if (place >= range.chunks) return;
    const int32_t first = range.begin + (int32_t)place * kChunk, count = min(range.end - first, kChunk);
    // rows of K, then of Q: their norms, and their elements times a power of two
    const uint32_t stride = p.wide * 2 + 16, term_bytes = 2 * kChunk * stride;
    uint8_t *rows = p.rows + (uint64_t)blockIdx.x * p.rows_bytes;
    // 16 lanes a row where it has no more than 128 elements
    const uint32_t row_lanes = p.wide <= 128 ? 16 : 32, at_once = kPrepareThreads / row_lanes, e0 = tid % row_lanes * 8;
    const bool low_dim = e0 < k_dim, in_row = e0 < p.wide;
    // each head's decays of this lane's token; the first ones before the rows, so that they are there when the triangles are made
    const bool on = (int32_t)lane < count;
    const uint32_t group = p.d.group.d;
    const uint64_t decays_at = (first + (on ? lane : 0)) * a.decay_stride + key_head * group, betas_at = (first + (on ? lane : 0)) * a.beta_stride + key_head * group;
    float g = 0.f, beta = 0.f;
    if (on && warp < group) {
        g = a.log_decay[decays_at + warp];
        beta = a.beta[betas_at + warp];
    }
    constexpr uint32_t kBatch = 8 / kTerms;     // rows on their way at once
    uint4 raw[kBatch][kTerms];
    for (uint32_t i0 = tid / row_lanes; i0 < 2 * kChunk; i0 += kBatch * at_once) {
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) {
            const uint32_t i = i0 + j * at_once, t = i % kChunk, q = i / kChunk;
#pragma unroll
            for (int e = 0; e < kTerms; ++e) raw[j][e] = make_uint4(0, 0, 0, 0);
            if ((int32_t)t < count && low_dim) {
                const uint64_t token = first + t;
                const uint64_t at = q ? token * a.q_token_stride + key_head * a.q_head_stride : token * a.k_token_stride + key_head * a.k_head_stride;
                const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(q ? a.q : a.k) + (at + e0) * kTerms);
#pragma unroll
                for (int e = 0; e < kTerms; ++e) raw[j][e] = __ldg(from + e);
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) {
            const uint32_t i = i0 + j * at_once, t = i % kChunk, q = i / kChunk;
            float x[8], sum = 0.f, most = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint4 &r = raw[j][kTerms == 2 ? e / 4 : 0];
                const uint32_t words[4] = {r.x, r.y, r.z, r.w}, word = words[kTerms == 2 ? e % 4 : e / 2];
                if (kTerms == 2) x[e] = __uint_as_float(word);
                else if (a.dtype == NINFER_BF16) x[e] = __uint_as_float(e % 2 ? word & 0xffff0000u : word << 16);
                else x[e] = __half2float(__ushort_as_half((unsigned short)(e % 2 ? word >> 16 : word & 0xffffu)));
                sum = fmaf(x[e], x[e], sum);
                if (e % 2) most = most_of(most, x[e - 1], x[e]);
            }
            if (row_lanes == 32) {
                sum += __shfl_xor_sync(~0u, sum, 16);
                most = most_of(most, __shfl_xor_sync(~0u, most, 16));
            }
#pragma unroll
            for (int e = 8; e; e /= 2) {
                sum += __shfl_xor_sync(~0u, sum, e);
                most = most_of(most, __shfl_xor_sync(~0u, most, e));
            }
            if (!(most < INFINITY)) {       // a row that is not finite: zeros
                most = 0.f;
                sum = NAN;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
            }
            const float up = power_for(most);
            if (e0 == 0) scales[q][t] = (int32_t)t >= count ? 0.f : inverse_power(up) * (a.norm_eps < 0.f ? (sum == sum ? 1.f : NAN) : 1.f / sqrtf(sum + a.norm_eps));
            uint32_t high[4], low[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split(x[2 * e] * up, x[2 * e + 1] * up, high[e], low[e]);
            if (in_row) {
                const uint4 h = make_uint4(high[0], high[1], high[2], high[3]), l = make_uint4(low[0], low[1], low[2], low[3]);
                *reinterpret_cast<uint4 *>(smem + i * stride + e0 * 2) = h;
                *reinterpret_cast<uint4 *>(rows + i * stride + e0 * 2) = h;
                if (kTerms == 2) {
                    *reinterpret_cast<uint4 *>(smem + term_bytes + i * stride + e0 * 2) = l;
                    *reinterpret_cast<uint4 *>(rows + term_bytes + i * stride + e0 * 2) = l;
                }
            }
        }
    }
    __syncthreads();
    // a query's scale spoils its own result alone; a key's all that follows (below), and enters no product
    const bool bad_key = !(scales[0][lane] < INFINITY);
    __syncthreads();
    if (warp == 0 && bad_key) scales[0][lane] = 0.f;
    __syncthreads();
    // (K, Q) K^T: 16 rows a warp
    {
        // The tensor core cuts sums off towards zero: even and odd steps, and fp32's lower terms, have sums of their own.
        float d[4][4] = {}, odd[4][4] = {}, lower[kTerms == 2 ? 4 : 1][4] = {};
        const uint32_t base = smem_u32(smem), from_a = base + (warp * 16 + lane % 16) * stride + lane / 16 * 16;
        const uint32_t from_b = base + (lane % 8 + lane / 16 * 8) * stride + lane / 8 % 2 * 16;
        for (uint32_t k0 = 0; k0 < p.wide; k0 += 32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = (k0 + h * 16) * 2;
                float(&sum)[4][4] = h ? odd : d;
                uint32_t x[kTerms][4], y[4];
#pragma unroll
                for (int e = 0; e < kTerms; ++e) load_matrices(x[e], from_a + e * term_bytes + k);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    load_matrices(y, from_b + n * 16 * stride + k);
                    mma(sum[2 * n], x[0], y[0], y[1]);
                    mma(sum[2 * n + 1], x[0], y[2], y[3]);
                    if (kTerms == 2) {
                        mma(lower[2 * n], x[kTerms - 1], y[0], y[1]);
                        mma(lower[2 * n + 1], x[kTerms - 1], y[2], y[3]);
                        load_matrices(y, from_b + term_bytes + n * 16 * stride + k);
                        mma(lower[2 * n], x[0], y[0], y[1]);
                        mma(lower[2 * n + 1], x[0], y[2], y[3]);
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t t = warp % 2 * 16 + lane / 4 + e / 2 * 8, u = n * 8 + lane % 4 * 2 + e % 2;
                const float dot = d[n][e] + odd[n][e] + (kTerms == 2 ? lower[kTerms == 2 ? n : 0][e] : 0.f);
                dots[warp / 2][t][u] = warp / 2 ? dot : dot * scales[0][t] * scales[0][u];       // of Q: without the scales
            }
    }
    __syncthreads();
    // A warp a value head: lane s has column s of both triangles. Log decays are added up in units of ln 2 and in two floats, so that
    // differences of far sums are as exact as those of near ones; 2^(+-2^15) is all the same.
    float(*tri)[kChunk][kTriRow] = reinterpret_cast<float(*)[kChunk][kTriRow]>(smem);
    for (uint32_t i = warp; i < group; i += kPrepareThreads / 32) {
        const uint32_t head = key_head * group + i;
        if (on && i != warp) {
            g = a.log_decay[decays_at + i];
            beta = a.beta[betas_at + i];
        }
        // A decay, beta or key that is not finite makes all of the state NaN (a decay of -infinity zeros): the chunks' kernel does that from the first
        // such token on, and here they count as zeros.
        const bool spoils = !(g < INFINITY) || !(fabsf(beta) < INFINITY) || bad_key;
        const uint32_t bad = __ballot_sync(~0u, spoils);
        if (spoils) g = beta = 0.f;
        const float bound = fminf(fmaxf(g, -32768.f), 32768.f);
        float high = bound * 1.44269504f, low = fmaf(bound, 1.44269504f, -high) + bound * 1.92596299e-8f;
#pragma unroll
        for (int k = 1; k < 32; k *= 2) {
            const float u = __shfl_up_sync(~0u, high, k), v = __shfl_up_sync(~0u, low, k);
            if (lane >= (uint32_t)k) {
                const float sum = high + u, w = sum - high;
                low += v + ((high - (sum - w)) + (u - w));
                high = sum;
            }
        }
        const float last_high = __shfl_sync(~0u, high, 31), last_low = __shfl_sync(~0u, low, 31);
        sums[warp][lane] = make_float4(high, low, beta, 0.f);
        __syncwarp();
        uint8_t *to = p.heads + ((uint64_t)chunk * a.v_heads + head) * kHeadBytes;       // T high and low, P high and low, the numbers
        float pp[kChunk], tt[kChunk], most_p = 0.f, most_t = 0.f;
#pragma unroll
        for (int t = 0; t < kChunk; ++t) {
            const float4 at = sums[warp][t];
            const float fade = exp2f((at.x - high) + (at.y - low));
            tri[warp][t][lane] = (int)lane < t ? at.z * fade * dots[0][t][lane] : 0.f;
            pp[t] = (int)lane <= t ? fade * dots[1][t][lane] : 0.f;
            most_p = fmaxf(most_p, fabsf(pp[t]));
        }
        const float of_p = put_matrix(to + 2 * kChunk * kTriStride, pp, most_p, lane);      // first, so that its registers are free for T
        __syncwarp();
#pragma unroll
        for (int t = 0; t < kChunk; ++t) {
            float sum4[4] = {(int)lane == t ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < t; m += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&tri[warp][t][m]);
                sum4[0] = fmaf(-x.x, tt[m], sum4[0]);
                if (m + 1 < t) sum4[1] = fmaf(-x.y, tt[m + 1], sum4[1]);
                if (m + 2 < t) sum4[2] = fmaf(-x.z, tt[m + 2], sum4[2]);
                if (m + 3 < t) sum4[3] = fmaf(-x.w, tt[m + 3], sum4[3]);
            }
            tt[t] = (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
        }
#pragma unroll
        for (int t = 0; t < kChunk; ++t) most_t = fmaxf(most_t, fabsf(tt[t] *= beta * scales[0][t]));
        __syncwarp();
        const float of_t = put_matrix(to, tt, most_t, lane);
        float *numbers = reinterpret_cast<float *>(to + kTrianglesBytes);
        const float fade = exp2f(high + low);
        numbers[kOfK + lane] = bad & (~0u >> (31 - lane)) ? NAN : fade * scales[0][lane];
        numbers[kOfQ + lane] = a.scale * fade * scales[1][lane];
        numbers[kOfU + lane] = exp2f((last_high - high) + (last_low - low));
        numbers[kOfP + lane] = a.scale * scales[1][lane] * of_p;
        if (lane < 2) numbers[kLeft + lane] = lane == 0 ? exp2f(last_high + last_low) : of_t;
    }
}

// Columns of a state a CTA: where that makes no more CTAs than SMs 16, 32 or up to 48 (8001 tokens with 16 heads of 128 columns by 16, 32 and
// 48: 420, 475 and 592 us; 48 heads by 48 and by 32 columns, two CTAs an SM: 620 and 716), else 32, two CTAs an SM of which one begins or ends
// while the other computes (64 prompts of 33 tokens with 48 heads 322 us, of 128 tokens 567; with 48 columns 440 and 721), or 64 where
// shared memory has no room for two.
// With up to 48 (3 pairs of warps) the two warps without columns take from the pairs' chain what is not of it: the results (P U and Q S), made
// by one of them (the other copies) or, with a ninth warp that copies, by both; for 8001 tokens with 48 heads 78 us less than by the pairs themselves.
// What a pair hands over: U and Q S of 16 columns by 32 tokens, two buffers.
constexpr uint32_t kResultWarp = 6, kHandedBytes = 8 * 32 * 16;
// The ninth warp is there where it leaves the others registers enough: 168 a thread instead of 255.
__host__ __device__ constexpr int chunk_threads(int steps, int columns) { return columns == 32 ? 128 : columns == 48 && steps < 4 ? 288 : 256; }

// Shared memory: the stages (chunks at once), the results' turning (16 tokens by 16 columns a warp), the pairs' sums (one buffer or two),
// what is handed over.
__host__ __device__ constexpr uint32_t values_of(int columns) { return columns == 32 ? 32 : 64; }      // columns of V that are copied
__host__ __device__ constexpr uint32_t stage_bytes_of(uint32_t wide, int terms, int columns) {
    return terms * 2 * kChunk * (wide * 2 + 16) + kHeadBytes + kChunk * (values_of(columns) * (terms == 2 ? 4 : 2) + 16);
}
__host__ __device__ constexpr uint32_t turning_of(int columns) { return (columns == 48 ? 2 : columns / 8) * (kChunk / 2 * 80); }
__host__ __device__ constexpr uint32_t sums_bytes_of(int columns) { return columns / 8 * 6 * 32 * 16; }
__host__ __device__ constexpr uint32_t smem_of(uint32_t wide, int terms, int columns, uint32_t stages, uint32_t sums) {
    return stages * stage_bytes_of(wide, terms, columns) + turning_of(columns) + sums * sums_bytes_of(columns) + (columns == 48 ? 6 * kHandedBytes : 0);
}
__host__ __device__ constexpr uint32_t room_of(int columns) { return (columns == 32 ? 113 : 227) * 1024 - 384; }       // less what has its place at compile time
__host__ __device__ constexpr uint32_t sums_of(uint32_t wide, int terms, int columns) { return smem_of(wide, terms, columns, 2, 2) <= room_of(columns) ? 2 : 1; }
__host__ __device__ constexpr uint32_t stages_of(uint32_t wide, int terms, int columns) {
    return smem_of(wide, terms, columns, 3, sums_of(wide, terms, columns)) <= room_of(columns) ? 3 : 2;
}
__host__ __device__ constexpr uint32_t chunk_smem_of(uint32_t wide, int terms, int columns) {
    return smem_of(wide, terms, columns, stages_of(wide, terms, columns), sums_of(wide, terms, columns));
}

// Columns where there are more states than SMs.
__host__ __device__ constexpr int many_columns(uint32_t wide, int terms) { return smem_of(wide, terms, 32, 2, 1) <= room_of(32) ? 32 : 64; }

// 16 columns by 32 tokens as the A operand, each column times its power of two.
__device__ __forceinline__ void halves(const float (&y)[4][4], float p0, float p1, uint32_t (&high)[2][4], uint32_t (&low)[2][4]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            split(y[2 * k + h][0] * p0, y[2 * k + h][1] * p0, high[k][2 * h], low[k][2 * h]);
            split(y[2 * k + h][2] * p1, y[2 * k + h][3] * p1, high[k][2 * h + 1], low[k][2 * h + 1]);
        }
}
// 16 tokens of a matrix's rows as the B operand, of both of its terms.
__device__ __forceinline__ void load_terms(uint32_t (&b)[2][4], uint32_t from) {
    load_matrices(b[0], from);
    load_matrices(b[1], from + kChunk * kTriStride);
}
__device__ __forceinline__ void times(float (&y)[4], const uint32_t (&high)[4], const uint32_t (&low)[4], const uint32_t (&b)[2][4], int i, int term) {
    mma(y, term == 2 ? low : high, b[term == 1][2 * i], b[term == 1][2 * i + 1]);
}
// A lower triangle whose first term lies at `from` (this lane's row and column of the first 16 by 16); u += A times it.
__device__ __forceinline__ void load_triangle(uint32_t (&t00)[2][4], uint32_t (&t01)[2][4], uint32_t (&t11)[2][4], uint32_t from) {
    load_terms(t00, from);
    load_terms(t01, from + 16 * kTriStride);
    load_terms(t11, from + 16 * kTriStride + 32);
}
__device__ __forceinline__ void times_triangle(float (&u)[4][4], const uint32_t (&high)[2][4], const uint32_t (&low)[2][4], const uint32_t (&t00)[2][4],
                                               const uint32_t (&t01)[2][4], const uint32_t (&t11)[2][4]) {
#pragma unroll
    for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            times(u[i], high[0], low[0], t00, i, term);
            times(u[2 + i], high[0], low[0], t01, i, term);
        }
#pragma unroll
    for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int i = 0; i < 2; ++i) times(u[2 + i], high[1], low[1], t11, i, term);
}
// 16 tokens by 16 columns to where this lane's first 16 bytes go, turned in shared memory at `at`; `left` tokens there are.
struct Results {
    uint32_t es, row;       // bytes an element, this lane's token
    uint64_t step;          // bytes a token
    bool on;
};
__device__ __forceinline__ void put_results(const Results &r, int dtype, uint8_t *smem, uint32_t at, uint8_t *to, const float (&o)[2][4], int32_t left, uint32_t lane) {
    if (dtype == NINFER_F32) {
        uint8_t *turned = smem + at + lane % 4 * 160 + lane / 4 * 4;
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<float *>(turned + (i / 4 * 8 + i % 2) * 80 + i / 2 % 2 * 32) = o[i / 4][i % 4];
    } else {
        uint32_t x[4];          // pairs of tokens, turned as they are stored
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(o[i / 2][i % 2 * 2], o[i / 2][i % 2 * 2 + 1]);
            const __half2 h = __floats2half2_rn(o[i / 2][i % 2 * 2], o[i / 2][i % 2 * 2 + 1]);
            x[i] = dtype == NINFER_BF16 ? *reinterpret_cast<const uint32_t *>(&b) : *reinterpret_cast<const uint32_t *>(&h);
        }
        store_matrices_turned(smem_u32(smem) + at + (lane % 8 + lane / 16 * 8) * 80 + lane / 8 % 2 * 16, x);
    }
    __syncwarp();
    const uint8_t *from = smem + at + r.row * 80 + lane % r.es * 16;
    if (r.on && (int32_t)r.row < left) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
    if (r.es == 4 && r.on && (int32_t)r.row + 8 < left) *reinterpret_cast<uint4 *>(to + 8 * r.step) = *reinterpret_cast<const uint4 *>(from + 8 * 80);
    __syncwarp();
}

// 16 to 64 columns of one state a CTA, 16 a pair of warps, of which each has half of the columns' k; the state stays in the
// accumulators' layout of mma, transposed (rows are columns of S, columns k), which is the layout of the A operand of the
// products with K and Q, and U, made the same way, that of the products with P and K. Every factor that is not exact in binary16 enters
// as two terms, scaled row by row. The pair adds up its halves of K S and Q S through shared memory, has U twice, and shares out the
// outputs by tokens where no other warp makes them. One warp keeps the next chunks coming (bulk copies, mbarriers); nothing else holds pairs together, so
// that of two pairs on a scheduler one multiplies while the other splits and scales.
// kSteps: steps of 16 of k_dim of a warp; kTerms: terms of k and q. The CTAs an SM are said to ptxas, which otherwise
// takes fewer registers and loads later (173 for 207, 59 us more for the same prompt).
template <int kSteps, int kTerms, int kColumns>
__global__ void __launch_bounds__(chunk_threads(kSteps, kColumns), kColumns == 32 ? 2 : 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    constexpr uint32_t kRowStride = kSteps * 64 + 16, kTermBytes = 2 * kChunk * kRowStride;
    constexpr bool kResults = kColumns == 48, kNinth = chunk_threads(kSteps, kColumns) > 256;       // a warp that copies
    constexpr uint32_t kStages = stages_of(kSteps * 32, kTerms, kColumns), kTri = kTerms * kTermBytes, kNumbersAt = kTri + kTrianglesBytes, kV = kTri + kHeadBytes;
    constexpr uint32_t kSums = sums_of(kSteps * 32, kTerms, kColumns), es = kTerms == 2 ? 4 : 2, v_stride = values_of(kColumns) * es + 16, stage_bytes = kV + kChunk * v_stride;
    static_assert(stage_bytes == stage_bytes_of(kSteps * 32, kTerms, kColumns));
    static_assert(chunk_smem_of(kSteps * 32, kTerms, kColumns) <= room_of(kColumns));
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], handed[3][2], taken[3][2];
    __shared__ uint32_t spoilt[kResults ? 3 : 1][2][8];      // handed over too
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_gated_delta_args &a = p.d.a;
    const Part part = part_of(p.d, blockIdx.x, p.slab);
    if (part.none) return;
    const Range range = range_of(a, part.request);
    if (!range.chunks) return;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32, k_dim = (uint32_t)a.k_dim, v_dim = (uint32_t)a.v_dim;
    const uint32_t base = smem_u32(smem), columns = min(v_dim - part.column, p.slab);
    if (tid == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&full[i]), 1 + 32);          // the bulk copies, and each lane's of the values
            mbar_init(smem_u32(&empty[i]), (columns + 15) / 16 * 2 + kResults);
        }
        for (uint32_t i = 0; kResults && i < 6; ++i) {
            mbar_init(smem_u32(&handed[i / 2][i % 2]), 2);       // a pair's warps
            mbar_init(smem_u32(&taken[i / 2][i % 2]), 1);
        }
        fence_mbar_init();
    }
    __syncthreads();
    const uint32_t pair = warp / 2, half = warp % 2;
    const bool bf16 = a.dtype == NINFER_BF16;
    constexpr uint32_t kSumsAt = kStages * stage_bytes + turning_of(kColumns), kHandedAt = kSumsAt + kSums * sums_bytes_of(kColumns);
    const uint32_t out_at = kStages * stage_bytes + (kResults ? warp % 2 : warp) * (kChunk / 2 * 80);
    const uint32_t mine = part.column + pair * 16, column = mine + lane / 4;         // this thread's: column, column + 8
    const uint32_t b_row = lane % 8 + lane / 16 * 8, b_col = lane / 8 % 2 * 16;          // of the four matrices that a lane addresses
    const uint32_t t_row = lane % 16, t_col = lane / 16 * 16, half_col = half * kSteps * 32;
    uint32_t sent = 0;
    bool good = true;       // once a wait has run out, none is made and nothing is stored
    // The copying warp's: chunk j into its stage, which all warps have left. Lanes whose 16 bytes of values lie past the last column copy
    // the last ones there are; what they get is part of no result.
    constexpr uint32_t kUnits = values_of(kColumns) * es / 16;
    constexpr int32_t kRowsAtOnce = 32 / kUnits;
    const uint8_t *next_v = static_cast<const uint8_t *>(a.v) +
                            ((uint64_t)(range.begin + lane / kUnits) * a.v_token_stride + part.head * a.v_head_stride + part.column) * es + min(lane % kUnits, columns * es / 16 - 1) * 16;
    const uint64_t v_step = kRowsAtOnce * a.v_token_stride * es;
    auto send = [&](uint32_t j) {
        if (j >= kStages) good = !__any_sync(~0u, !(good && mbar_wait(smem_u32(&empty[j % kStages]), (j / kStages - 1) & 1, p.error, p.wait_limit)));
        if (!good) return;
        const uint32_t stage = base + j % kStages * stage_bytes, bar = smem_u32(&full[j % kStages]);
        const int32_t left = range.end - range.begin - (int32_t)j * kChunk - (int32_t)(lane / kUnits);      // tokens from this lane's first on
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, kTri + kHeadBytes);
            const uint32_t chunk = j < range.whole ? range.first + j : range.last;
            bulk_g2s(stage, p.rows + (uint64_t)(chunk * (uint32_t)a.k_heads + part.key_head) * p.rows_bytes, kTri, bar);
            bulk_g2s(stage + kTri, p.heads + ((uint64_t)chunk * a.v_heads + part.head) * kHeadBytes, kHeadBytes, bar);
        }
        // the values, 16 bytes at a time (a bulk copy a row took 80 cycles to issue, each)
        const uint32_t to = stage + kV + lane / kUnits * v_stride + lane % kUnits * 16;
        const uint8_t *from = next_v;
        if (left >= kChunk) {
#pragma unroll
            for (int32_t i = 0; i < kChunk / kRowsAtOnce; ++i, from += v_step) copy16(to + i * kRowsAtOnce * v_stride, from);
        } else {
            for (int32_t i = 0; i * kRowsAtOnce < left; ++i, from += v_step) copy16(to + i * kRowsAtOnce * v_stride, from);
        }
        next_v += v_step * (kChunk / kRowsAtOnce);
        copies_arrive(bar);
        sent = j + 1;
    };
    // No CTA ends with copies under way, not where a wait has run out either: at least a millisecond for them to land.
    constexpr long long kLanding = 2000000;
    auto drain = [&]() {
        for (uint32_t j = sent > kStages ? sent - kStages : 0; j < sent; ++j) mbar_wait(smem_u32(&full[j % kStages]), j / kStages & 1, p.error, max(p.wait_limit, kLanding));
    };
    // a lane's first 16 bytes of results: of 16 tokens by 16 columns, two (f32: four) a token
    const uint32_t out_es = a.out_dtype == NINFER_F32 ? 4 : 2, out_col = lane % out_es * 16 / out_es;
    const uint64_t out_step = a.v_heads * v_dim * out_es;
    Results results = {out_es, lane / out_es, out_step, mine + out_col < v_dim};
    uint8_t *to_out = static_cast<uint8_t *>(a.out) + (uint64_t)(range.begin + results.row) * out_step + ((uint64_t)part.head * v_dim + part.column + out_col) * out_es;
    uint32_t slot = 0, parity = 0;
    // who copies: a ninth warp, or one without columns, or the first beside its other work
    const uint32_t sender = kNinth ? 8 : kResults ? kResultWarp + 1 : 0;
    if ((kNinth || kResults) && warp == sender) {
        for (uint32_t j = 0; j < range.chunks && good; ++j) send(j);
        drain();
        return;
    }
    constexpr uint32_t kResultWarps = kNinth ? 2 : 1;       // each has its chunks
    if (kResults && warp >= kResultWarp && warp < kResultWarp + kResultWarps) {
        to_out += (warp - kResultWarp) * kChunk * out_step;
        for (uint32_t j = warp - kResultWarp; j < range.chunks; j += kResultWarps) {
            slot = j % kStages;
            parity = j / kStages & 1;
            good = !__any_sync(~0u, !(good && mbar_wait(smem_u32(&full[slot]), parity, p.error, p.wait_limit)));
            const uint32_t stage = base + slot * stage_bytes;
            const float *numbers = reinterpret_cast<const float *>(smem + slot * stage_bytes + kNumbersAt);
            const int32_t count = min(range.end - range.begin - (int32_t)j * kChunk, kChunk);
            for (uint32_t g = 0; g * 16 < columns; ++g) {
                good = !__any_sync(~0u, !(good && mbar_wait(smem_u32(&handed[g][j % 2]), j / 2 & 1, p.error, p.wait_limit)));
                const float4 *from = reinterpret_cast<const float4 *>(smem + kHandedAt + (g * 2 + j % 2) * kHandedBytes) + lane;
                float u[4][4], qs[4][4], o[4][4] = {}, m0 = 0.f, m1 = 0.f;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float4 x = from[n * 32], y = from[(4 + n) * 32];
                    u[n][0] = x.x; u[n][1] = x.y; u[n][2] = x.z; u[n][3] = x.w;
                    qs[n][0] = y.x; qs[n][1] = y.y; qs[n][2] = y.z; qs[n][3] = y.w;
                    m0 = fmaxf(m0, fmaxf(fabsf(x.x), fabsf(x.y)));
                    m1 = fmaxf(m1, fmaxf(fabsf(x.z), fabsf(x.w)));
                }
                const uint32_t first = spoilt[g][j % 2][lane / 4];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&taken[g][j % 2]));
                const float p0 = power_for(quad_max(m0)), p1 = power_for(quad_max(m1));
                uint32_t high[2][4], low[2][4];
                halves(u, p0, p1, high, low);
                uint32_t t00[2][4], t01[2][4], t11[2][4];
                load_triangle(t00, t01, t11, stage + kTri + (2 * kChunk + b_row) * kTriStride + b_col);
                times_triangle(o, high, low, t00, t01, t11);
                const float g0 = inverse_power(p0), g1 = inverse_power(p1);
                if (first != kAllFinite) from_spoilt(first, o, NAN);
                if (!good) continue;
                results.on = part.column + g * 16 + out_col < v_dim;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float y[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float2 of_q = *reinterpret_cast<const float2 *>(numbers + kOfQ + (h * 2 + n) * 8 + lane % 4 * 2);
                        const float2 of_p = *reinterpret_cast<const float2 *>(numbers + kOfP + (h * 2 + n) * 8 + lane % 4 * 2);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[n][e] = fmaf(e % 2 ? of_q.y : of_q.x, qs[2 * h + n][e], o[2 * h + n][e] * (e / 2 ? g1 : g0) * (e % 2 ? of_p.y : of_p.x));
                    }
                    put_results(results, a.out_dtype, smem, out_at, to_out + (uint64_t)h * 16 * out_step + g * 16 * out_es, y, count - h * 16, lane);
                }
            }
            to_out += kResultWarps * kChunk * out_step;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));
        }
        return;
    }
    if (pair * 16 >= columns) return;      // whole pairs
    if (warp == sender)
        for (uint32_t j = 0; j < min(kStages - 1, range.chunks); ++j) send(j);
    to_out += (uint64_t)half * 16 * out_step + pair * 16 * out_es;
    // s[n][e]: k = 16 kSteps half + 8 n + 2 (lane % 4) + e % 2 of column (e / 2: + 8)
    float s[2 * kSteps][4];
    float *state = a.state + part.state;
    const uint32_t k_first = half * kSteps * 16 + lane % 4 * 2;
#pragma unroll
    for (int n = 0; n < 2 * kSteps; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t k = k_first + n * 8 + e % 2, c = column + e / 2 * 8;
            s[n][e] = k < k_dim && c < v_dim && !part.fresh ? state[k * v_dim + c] : 0.f;
        }
    for (uint32_t j = 0; j < range.chunks; ++j) {
        good = !__any_sync(~0u, !(good && mbar_wait(smem_u32(&full[slot]), parity, p.error, p.wait_limit)));
        const uint32_t stage = base + slot * stage_bytes;
        const uint8_t *here = smem + slot * stage_bytes;
        const float *numbers = reinterpret_cast<const float *>(here + kNumbersAt);
        const int32_t count = min(range.end - range.begin - (int32_t)j * kChunk, kChunk);
        {
            // S^T times K^T and Q^T: x[0..3] tokens of K, x[4..7] of Q
            float x[8][4] = {}, up0, up1;
            {
                float m[4] = {};
#pragma unroll
                for (int n = 0; n < 2 * kSteps; ++n) {
                    m[n % 2] = fmaxf(m[n % 2], fmaxf(fabsf(s[n][0]), fabsf(s[n][1])));
                    m[2 + n % 2] = fmaxf(m[2 + n % 2], fmaxf(fabsf(s[n][2]), fabsf(s[n][3])));
                }
                up0 = power_for(quad_max(fmaxf(m[0], m[1])));
                up1 = power_for(quad_max(fmaxf(m[2], m[3])));
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                uint32_t high[4], low[4], y[4][4];
                const uint32_t from = stage + b_row * kRowStride + half_col + k * 32 + b_col;
#pragma unroll
                for (int n = 0; n < 4; ++n) load_matrices(y[n], from + n * 16 * kRowStride);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    split(s[2 * k + h][0] * up0, s[2 * k + h][1] * up0, high[2 * h], low[2 * h]);
                    split(s[2 * k + h][2] * up1, s[2 * k + h][3] * up1, high[2 * h + 1], low[2 * h + 1]);
                }
                // each accumulator again after eight products
#pragma unroll
                for (int n = 0; n < 8; ++n) mma(x[n], high, y[n / 2][n % 2 * 2], y[n / 2][n % 2 * 2 + 1]);
#pragma unroll
                for (int n = 0; n < 8; ++n) mma(x[n], low, y[n / 2][n % 2 * 2], y[n / 2][n % 2 * 2 + 1]);
                if (kTerms == 2) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) load_matrices(y[n], from + kTermBytes + n * 16 * kRowStride);
#pragma unroll
                    for (int n = 0; n < 8; ++n) mma(x[n], high, y[n / 2][n % 2 * 2], y[n / 2][n % 2 * 2 + 1]);
                }
            }
            if (warp == sender && j + kStages - 1 < range.chunks) send(j + kStages - 1);
            {
                const float down0 = inverse_power(up0), down1 = inverse_power(up1);
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] *= e / 2 ? down1 : down0;
            }
            // the pair's halves: all of K S to both, of Q S the first 16 tokens to the first. Two buffers: who writes one again has
            // passed the barrier between, and with it the other's reads.
            float4 *sums = reinterpret_cast<float4 *>(smem + kSumsAt) + (j % kSums * (kColumns / 8) + warp) * 6 * 32 + lane;
            const float4 *others = reinterpret_cast<const float4 *>(smem + kSumsAt) + (j % kSums * (kColumns / 8) + (warp ^ 1)) * 6 * 32 + lane;
#pragma unroll
            for (int n = 0; n < 4; ++n) sums[n * 32] = make_float4(x[n][0], x[n][1], x[n][2], x[n][3]);
#pragma unroll
            for (int n = 0; n < 2; ++n)
                sums[(4 + n) * 32] = half ? make_float4(x[4 + n][0], x[4 + n][1], x[4 + n][2], x[4 + n][3]) : make_float4(x[6 + n][0], x[6 + n][1], x[6 + n][2], x[6 + n][3]);
            // meanwhile the values, and the numbers
            float w[4][4];
            if (kTerms == 2) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[n][e] = *reinterpret_cast<const float *>(here + kV + (n * 8 + lane % 4 * 2 + e % 2) * v_stride + (pair * 16 + lane / 4 + e / 2 * 8) * es);
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {       // 16 tokens: pairs of them, of this thread's two columns
                    uint32_t v[4];
                    load_matrices_turned(v, stage + kV + (k * 16 + b_row) * v_stride + pair * 32 + b_col);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
                        w[2 * k + i / 2][i % 2 * 2] = bf16 ? __uint_as_float(v[i] << 16) : f.x;
                        w[2 * k + i / 2][i % 2 * 2 + 1] = bf16 ? __uint_as_float(v[i] & 0xffff0000u) : f.y;
                    }
                }
            }
            if (count < kChunk) {       // rows that were not copied
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n * 8 + (int32_t)(lane % 4) * 2 + e % 2 >= count) w[n][e] = 0.f;
            }
            named_barrier(1 + pair, 64);
            // W = V - e^G K S, then U = T diag(beta) W, times the keys' scales
            float m0 = 0.f, m1 = 0.f, qs[2][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 f = *reinterpret_cast<const float2 *>(numbers + kOfK + n * 8 + lane % 4 * 2);
                const float4 o = others[n * 32];
                const float oe[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) w[n][e] -= (e % 2 ? f.y : f.x) * (x[n][e] + oe[e]);
                m0 = most_of(m0, w[n][0], w[n][1]);
                m1 = most_of(m1, w[n][2], w[n][3]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float4 o = others[(4 + n) * 32];
                const float oe[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) qs[n][e] = (half ? x[6 + n][e] : x[4 + n][e]) + oe[e];
            }
            if (kSums == 1) named_barrier(1 + pair, 64);
            uint32_t high[2][4], low[2][4], t00[2][4], t01[2][4], t11[2][4];
            load_triangle(t00, t01, t11, stage + kTri + b_row * kTriStride + b_col);        // ahead of the branch
            float u[4][4] = {};
            // W of a column is zero from its first token on that is not finite; that token's result and later ones are NaN, and so is the state
            // (520 us for the prompt of 8001 tokens, 514 without the test; values tested before the pair's barrier, which waits for it: 541)
            const bool odd = !(most_of(m0, m1) < INFINITY);
            m0 = quad_max(m0);
            m1 = quad_max(m1);
            uint32_t first = kAllFinite;
            if (__any_sync(~0u, odd)) {
                first = first_spoilt(w);
                from_spoilt(first, w, 0.f);
                m0 = m1 = 0.f;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    m0 = fmaxf(m0, fmaxf(fabsf(w[n][0]), fabsf(w[n][1])));
                    m1 = fmaxf(m1, fmaxf(fabsf(w[n][2]), fabsf(w[n][3])));
                }
                m0 = quad_max(m0);
                m1 = quad_max(m1);
            }
            float p0 = power_for(m0), p1 = power_for(m1);
            halves(w, p0, p1, high, low);
            times_triangle(u, high, low, t00, t01, t11);
            const float of_t = numbers[kOfT], f0 = of_t * inverse_power(p0), f1 = of_t * inverse_power(p1);
            m0 = m1 = 0.f;
            float n0 = 0.f, n1 = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 f = *reinterpret_cast<const float2 *>(numbers + kOfU + n * 8 + lane % 4 * 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    u[n][e] *= e / 2 ? f1 : f0;
                    w[n][e] = u[n][e] * (e % 2 ? f.y : f.x);
                }
                m0 = fmaxf(m0, fmaxf(fabsf(u[n][0]), fabsf(u[n][1])));
                m1 = fmaxf(m1, fmaxf(fabsf(u[n][2]), fabsf(u[n][3])));
                n0 = fmaxf(n0, fmaxf(fabsf(w[n][0]), fabsf(w[n][1])));
                n1 = fmaxf(n1, fmaxf(fabsf(w[n][2]), fabsf(w[n][3])));
            }
            float o[2][4] = {}, g0 = 0.f, g1 = 0.f;
            if constexpr (kResults) {       // handed over
                if (j >= 2) good = !__any_sync(~0u, !(good && mbar_wait(smem_u32(&taken[pair][j % 2]), (j / 2 - 1) & 1, p.error, p.wait_limit)));
                float4 *to = reinterpret_cast<float4 *>(smem + kHandedAt + (pair * 2 + j % 2) * kHandedBytes) + half * 64 + lane;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    to[n * 32] = half ? make_float4(u[2 + n][0], u[2 + n][1], u[2 + n][2], u[2 + n][3]) : make_float4(u[n][0], u[n][1], u[n][2], u[n][3]);
                    to[(4 + n) * 32] = make_float4(qs[n][0], qs[n][1], qs[n][2], qs[n][3]);
                }
                if (!half && lane % 4 == 0) spoilt[pair][j % 2][lane / 4] = first;
                __syncwarp();
                if (lane == 0 && good) mbar_arrive(smem_u32(&handed[pair][j % 2]));      // else there are no results
            } else {        // P U for this warp's 16 tokens
                p0 = power_for(quad_max(m0));
                p1 = power_for(quad_max(m1));
                halves(u, p0, p1, high, low);
                uint32_t t0[2][4], t1[2][4];
                const uint32_t from = stage + kTri + (2 * kChunk + b_row) * kTriStride + b_col;
                load_terms(t0, from + half * 16 * kTriStride);
                load_terms(t1, from + 16 * kTriStride + 32);
#pragma unroll
                for (int term = 0; term < 3; ++term)
#pragma unroll
                    for (int i = 0; i < 2; ++i) times(o[i], high[0], low[0], t0, i, term);
                if (half) {
#pragma unroll
                    for (int term = 0; term < 3; ++term)
#pragma unroll
                        for (int i = 0; i < 2; ++i) times(o[i], high[1], low[1], t1, i, term);
                }
                g0 = inverse_power(p0);
                g1 = inverse_power(p1);
            }
            // S^T = e^G_last S^T + (e^(G_last - G) U)^T K; the products begin at zero and are added rounded to nearest
            p0 = power_for(quad_max(n0));
            p1 = power_for(quad_max(n1));
            halves(w, p0, p1, high, low);
            const float left = numbers[kLeft], d0 = inverse_power(p0), d1 = inverse_power(p1);
            const float left0 = (first & 255) < kChunk ? NAN : left, left1 = first >> 8 < kChunk ? NAN : left;
            constexpr int kAtOnce = kSteps % 2 ? 1 : 2;
#pragma unroll
            for (int n0_ = 0; n0_ < kSteps; n0_ += kAtOnce) {
                float y[2 * kAtOnce][4] = {};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t b[kAtOnce][4];
                    const uint32_t from = stage + (k * 16 + t_row) * kRowStride + half_col + n0_ * 32 + t_col;
#pragma unroll
                    for (int m = 0; m < kAtOnce; ++m) load_matrices_turned(b[m], from + m * 32);
#pragma unroll
                    for (int m = 0; m < 2 * kAtOnce; ++m) mma(y[m], high[k], b[m / 2][m % 2 * 2], b[m / 2][m % 2 * 2 + 1]);
#pragma unroll
                    for (int m = 0; m < 2 * kAtOnce; ++m) mma(y[m], low[k], b[m / 2][m % 2 * 2], b[m / 2][m % 2 * 2 + 1]);
                    if (kTerms == 2) {
#pragma unroll
                        for (int m = 0; m < kAtOnce; ++m) load_matrices_turned(b[m], from + kTermBytes + m * 32);
#pragma unroll
                        for (int m = 0; m < 2 * kAtOnce; ++m) mma(y[m], high[k], b[m / 2][m % 2 * 2], b[m / 2][m % 2 * 2 + 1]);
                    }
                }
#pragma unroll
                for (int m = 0; m < 2 * kAtOnce; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[2 * n0_ + m][e] = fmaf(y[m][e], e / 2 ? d1 : d0, (e / 2 ? left1 : left0) * s[2 * n0_ + m][e]);
            }
            float2 of_q[2], of_p[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                of_q[n] = *reinterpret_cast<const float2 *>(numbers + kOfQ + (half * 2 + n) * 8 + lane % 4 * 2);
                of_p[n] = *reinterpret_cast<const float2 *>(numbers + kOfP + (half * 2 + n) * 8 + lane % 4 * 2);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));
            if (++slot == kStages) {
                slot = 0;
                parity ^= 1;
            }
            if (!kResults && good) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[n][e] = fmaf(e % 2 ? of_q[n].y : of_q[n].x, qs[n][e], o[n][e] * (e / 2 ? g1 : g0) * (e % 2 ? of_p[n].y : of_p[n].x));
                if (first != kAllFinite) from_spoilt(first, o, NAN, half * 2);
                put_results(results, a.out_dtype, smem, out_at, to_out, o, count - (int32_t)half * 16, lane);
                to_out += kChunk * out_step;
            }
        }
    }
    if (!good) {
        if (warp == sender) drain();
        return;
    }
#pragma unroll
    for (int n = 0; n < 2 * kSteps; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t k = k_first + n * 8 + e % 2, c = column + e / 2 * 8;
            if (k < k_dim && c < v_dim) state[k * v_dim + c] = s[n][e];
        }
}

using ChunkKernel = void (*)(ChunkParams);
template <int kSteps, int kTerms>
ChunkKernel chunk_kernel_at(int columns) {
    if (columns == 48) return chunk_kernel<kSteps, kTerms, 48>;
    return chunk_kernel<kSteps, kTerms, many_columns(kSteps * 32, kTerms)>;
}
template <int kTerms>
ChunkKernel chunk_kernel_of(uint32_t wide, int columns) {
    return wide == 64    ? chunk_kernel_at<2, kTerms>(columns)
           : wide == 96  ? chunk_kernel_at<3, kTerms>(columns)
           : wide == 128 ? chunk_kernel_at<4, kTerms>(columns)
                         : chunk_kernel_at<8, kTerms>(columns);
}

// k_dim rounded up to what the kernel has instances for
uint32_t wide_of(uint64_t k_dim) { return k_dim <= 64 ? 64 : k_dim <= 96 ? 96 : k_dim <= 128 ? 128 : 256; }

uint64_t rows_bytes_of(int terms, uint64_t k_dim) { return (uint64_t)terms * 2 * kChunk * (wide_of(k_dim) * 2 + 16); }

int check_sizes(uint64_t tokens, uint64_t requests, uint64_t k_heads, uint64_t v_heads, uint64_t k_dim, uint64_t v_dim) {
    if (!tokens || tokens > 0x7fffffffull || !requests || requests > 0x7fffffffull)
        return fail(NINFER_ERR_SHAPE, "gated delta: %llu tokens of %llu requests", (unsigned long long)tokens, (unsigned long long)requests);
    if (!k_heads || !v_heads || v_heads > 65535 || v_heads % k_heads)
        return fail(NINFER_ERR_SHAPE, "gated delta: %llu value heads for %llu key heads", (unsigned long long)v_heads, (unsigned long long)k_heads);
    if (!k_dim || !v_dim || k_dim % 8 || v_dim % 8 || k_dim > 256 || v_dim > 256)
        return fail(NINFER_ERR_SHAPE, "gated delta: k_dim %llu and v_dim %llu must be multiples of 8 up to 256", (unsigned long long)k_dim,
                    (unsigned long long)v_dim);
    return NINFER_OK;
}

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_gated_delta_workspace(uint64_t tokens, uint64_t requests, uint64_t k_heads, uint64_t v_heads, uint64_t k_dim,
                                            uint64_t v_dim, uint64_t *bytes) {
    if (!bytes) return fail(NINFER_ERR_INVALID_ARGUMENT, "gated delta workspace: NULL bytes");
    const int st = check_sizes(tokens, requests, k_heads, v_heads, k_dim, v_dim);
    if (st) return st;
    // of calls with offsets, whichever dtype; a call without them needs none
    const uint64_t chunks = tokens / kChunk + requests;
    if (chunks * k_heads > 0x7fffffffull) return fail(NINFER_ERR_OVERFLOW, "gated delta: too many tokens and key heads");
    *bytes = chunks * (k_heads * 2 * rows_bytes_of(1, k_dim) + v_heads * kHeadBytes);
    return NINFER_OK;
}

extern "C" int ninfer_gated_delta(const ninfer_gated_delta_args *args, void *workspace, uint64_t workspace_bytes, ninfer_stream stream) {
    if (!args || !args->q || !args->k || !args->v || !args->log_decay || !args->beta || !args->state || !args->out)
        return fail(NINFER_ERR_INVALID_ARGUMENT, "gated delta: NULL args, q, k, v, log_decay, beta, state or out");
    const ninfer_gated_delta_args &a = *args;
    if (!dtype_valid(a.dtype) || !dtype_valid(a.out_dtype))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "gated delta: dtype %d or out dtype %d unsupported", a.dtype, a.out_dtype);
    if (!std::isfinite(a.scale) || !std::isfinite(a.norm_eps)) return fail(NINFER_ERR_INVALID_ARGUMENT, "gated delta: scale and norm_eps must be finite");
    int st = check_sizes(a.tokens, a.requests, a.k_heads, a.v_heads, a.k_dim, a.v_dim);
    if (st) return st;
    if (!a.offsets && a.tokens != a.requests)
        return fail(NINFER_ERR_SHAPE, "gated delta: %llu tokens of %llu requests without offsets", (unsigned long long)a.tokens, (unsigned long long)a.requests);
    const uint64_t whole = a.v_heads * a.k_dim * a.v_dim;
    if (!a.slots || a.slots > 0x7fffffffull || (!a.state_slots && a.slots < a.requests) || (a.slots > 1 && a.slot_stride < whole))
        return fail(NINFER_ERR_SHAPE, "gated delta: %llu slots of stride %llu", (unsigned long long)a.slots, (unsigned long long)a.slot_stride);
    if ((a.tokens > 1 && (a.decay_stride < a.v_heads || a.beta_stride < a.v_heads)))
        return fail(NINFER_ERR_SHAPE, "gated delta: decay or beta stride below v_heads");
    const uint64_t unit = 16 / dtype_size(a.dtype);
    const struct {
        const void *p;
        uint64_t token, head, heads;
    } tensors[] = {{a.q, a.q_token_stride, a.q_head_stride, a.k_heads},
                   {a.k, a.k_token_stride, a.k_head_stride, a.k_heads},
                   {a.v, a.v_token_stride, a.v_head_stride, a.v_heads}};
    for (const auto &t : tensors) {
        const uint64_t token = a.tokens > 1 ? t.token : 0, head = t.heads > 1 ? t.head : 0;
        if (!aligned(t.p, 16) || token % unit || head % unit)
            return fail(NINFER_ERR_ALIGNMENT, "gated delta: q, k and v must have bases and strides of 16 bytes' multiples");
        if (token >= (1ull << 40) || head >= (1ull << 40)) return fail(NINFER_ERR_OVERFLOW, "gated delta: a stride of 2^40 or more");
    }
    if (a.decay_stride >= (1ull << 40) || a.beta_stride >= (1ull << 40) || a.slot_stride >= (1ull << 40))
        return fail(NINFER_ERR_OVERFLOW, "gated delta: a stride of 2^40 or more");
    if (!aligned(a.state, 16) || (a.slots > 1 && a.slot_stride % 4) || !aligned(a.out, 16))
        return fail(NINFER_ERR_ALIGNMENT, "gated delta: state (with slot_stride) and out must be 16-byte aligned");
    for (const void *q : {(const void *)a.log_decay, (const void *)a.beta, (const void *)a.state_slots, (const void *)a.offsets,
                          (const void *)a.lengths, (const void *)a.status})
        if (!aligned(q, 4)) return fail(NINFER_ERR_ALIGNMENT, "gated delta: decays, betas and index arrays must be 4-byte aligned");
    uint64_t need = 0;
    if (a.offsets) st = ninfer_gated_delta_workspace(a.tokens, a.requests, a.k_heads, a.v_heads, a.k_dim, a.v_dim, &need);
    if (st) return st;
    if (need && !workspace) return fail(NINFER_ERR_INVALID_ARGUMENT, "gated delta: NULL workspace");
    if (workspace_bytes < need) return fail(NINFER_ERR_SIZE_MISMATCH, "gated delta: workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                                            (unsigned long long)need);
    if (need && !aligned(workspace, 256)) return fail(NINFER_ERR_ALIGNMENT, "gated delta: workspace must be 256-byte aligned");
    DeltaParams p;
    p.a = a;
    p.heads = FastDiv((uint32_t)a.v_heads);
    p.group = FastDiv((uint32_t)(a.v_heads / a.k_heads));
    const uint64_t rows = a.requests * a.v_heads;       // below 2^47; of at most eight slabs each
    if (rows * ((a.v_dim + 31) / 32) > 0x7fffffffull) return fail(NINFER_ERR_OVERFLOW, "gated delta: too many requests and heads");
    const uint64_t es = dtype_size(a.dtype);
    const auto heads = [&](const void *p, uint64_t dim, uint64_t token, uint64_t n, uint64_t head) { return Span(p, dim * es, a.tokens, token * es, n, head * es); };
    const Span out(a.out, a.tokens * a.v_heads * a.v_dim * dtype_size(a.out_dtype)), v = heads(a.v, a.v_dim, a.v_token_stride, a.v_heads, a.v_head_stride);
    const Span written[] = {out, Span(a.state, whole * 4, a.slots, a.slot_stride * 4), Span(a.status, 4), Span(workspace, need)};
    const Span inputs[] = {heads(a.q, a.k_dim, a.q_token_stride, a.k_heads, a.q_head_stride), heads(a.k, a.k_dim, a.k_token_stride, a.k_heads, a.k_head_stride),
                           out.same(v) && a.out_dtype == a.dtype ? Span() : v, Span(a.log_decay, a.v_heads * 4, a.tokens, a.decay_stride * 4),
                           Span(a.beta, a.v_heads * 4, a.tokens, a.beta_stride * 4), Span(a.state_slots, a.requests * 4), Span(a.offsets, (a.requests + 1) * 4),
                           Span(a.lengths, a.requests * 4)};
    bool shared = false;
    for (const Span &o : written) {
        for (const Span &i : inputs) shared = shared || o.meets(i);
        for (const Span &w : written) shared = shared || (&w != &o && o.meets(w));
    }
    if (shared) return fail(NINFER_ERR_INVALID_ARGUMENT, "gated delta: out may be v without gaps, of one dtype; no other of out, state, status and workspace overlaps anything");
    const auto grid = [&](uint64_t slab, unsigned *blocks) {
        const uint64_t slabs = (a.v_dim + slab - 1) / slab;
        p.slabs = FastDiv((uint32_t)slabs);
        *blocks = (unsigned)(rows * slabs);
    };
    unsigned blocks;
    const cudaStream_t s = (cudaStream_t)stream;
    if (!a.offsets) {
        // 32 columns a CTA while three of them an SM, which is how many run at once, are enough for all, else 64. 48 heads of 128 by 128, 2
        // requests 5.7 us by 32 and 6.2 by 64 columns, 4 requests 10.0 and 7.2; 8 heads of 256 by 256, 6 requests 7.7 and 8.0, 8 requests 10.9 and 8.7.
        DeviceInfo d;
        st = device_info(&d);
        if (st) return st;
        const bool narrow = rows * ((a.v_dim + 31) / 32) <= 3ull * d.sms;
        const int lanes = narrow || a.v_dim <= 32 ? 8 : 16;
        grid(lanes * 4, &blocks);
        const bool small = a.k_dim <= (uint64_t)(8 * kStepThreads / lanes);
        const auto kernel = lanes == 8 ? step_kernel<8, 8> : small ? step_kernel<16, 8> : step_kernel<16, 16>;
        return launch_dependent("gated delta", kernel, dim3(blocks), dim3(kStepThreads), 0, s, p);
    }
    DeviceInfo d;
    st = device_info(&d);
    if (st) return st;
    const int terms = a.dtype == NINFER_F32 ? 2 : 1;
    int columns = many_columns(wide_of(a.k_dim), terms), slab = columns;
    for (int most = 48; most >= 16 && rows * ((a.v_dim + most - 1) / most) <= (uint64_t)d.sms; most -= 16) {
        columns = 48;
        slab = most;
    }
    grid((uint64_t)slab, &blocks);
    const uint64_t chunks = a.tokens / kChunk + a.requests;
    ChunkParams c;
    c.d = p;
    c.wide = wide_of(a.k_dim);
    c.slab = (uint32_t)slab;
    c.rows_bytes = rows_bytes_of(terms, a.k_dim);
    c.rows = static_cast<uint8_t *>(workspace);
    c.heads = c.rows + chunks * a.k_heads * c.rows_bytes;
    st = device_error_word(&c.error);
    if (st) return st;
    c.wait_limit = wait_limit_cycles();
    const uint32_t prepare_smem = std::max((uint32_t)c.rows_bytes, kTriSmem);
    const uint32_t chunk_smem = chunk_smem_of(c.wide, terms, columns);
    const auto prepare = terms == 2 ? prepare_kernel<2> : prepare_kernel<1>;
    const auto chunk = terms == 2 ? chunk_kernel_of<2>(c.wide, columns) : chunk_kernel_of<1>(c.wide, columns);
    st = set_smem_attribute(reinterpret_cast<const void *>(prepare), (int)prepare_smem);
    if (!st) st = set_smem_attribute(reinterpret_cast<const void *>(chunk), (int)chunk_smem);
    if (!st) st = launch_dependent("gated delta", prepare, dim3((unsigned)(chunks * a.k_heads)), dim3(kPrepareThreads), prepare_smem, s, c);
    if (!st) st = launch_dependent("gated delta", chunk, dim3(blocks), dim3((unsigned)chunk_threads((int)c.wide / 32, columns)), chunk_smem, s, c);
    return st;
}
