// Kernels of ninfer_kv_attention: attention of one new token per request over a
// paged cache.
//
// Mathematics. One pass over the keys with a running maximum m and sum l per
// query head: scores above m rescale what was summed by 2^{m_old - m_new} (scores are
// kept in units of log2). Parts of a row that different warps or CTAs
// summed are joined the same way, with M = max m_i: l = sum 2^{m_i - M} l_i.
//
// What bounds it. Every key and value is used by the few query heads of its
// group (4 * group flops an element), so HBM does; the tensor cores only have
// to keep up, and mma.sync.m16n8k16 serves (11 % of the tensor pipe's cycles on a
// 16-bit cache, 17 % on an 8-bit one).
//   scores   A = 16 keys, B = 8 heads' queries;
//   values   A = 16 elements of the values transposed (ldmatrix.trans), B = 8 heads' weights,
//            transposed from the scores' accumulators in the registers (movmatrix).
// The 8 heads of a row are the narrow side of both, so that a group of eight wastes
// nothing. Queries as the A operand, with their remainders in the rows that a group
// of eight leaves empty, took twice the mmas: 231 against 203 us for 1.2 GB of 8-bit
// keys and values. 32-bit operands enter as sums of 16-bit terms, one mma each.
//
// Split. The keys of every (request, key head, 8 or 16 query heads), a row, are cut into
// units of 8 KB of keys and 8 KB of values; all units of the call form one
// line, on which a row's beginning counts as some units more, and of which each CTA
// (one an SM) and in it each warp takes an equal, contiguous part, so that any mix of
// lengths keeps every SM busy. A warp writes a row that lies in its part whole; cut
// rows are joined in the CTA, and rows cut between CTAs by a second, small kernel. Few
// short rows go without all that: a CTA or a cluster of CTAs for each, which joins its
// parts through distributed shared memory. Groups of more than eight heads take
// sixteen to a row up to 128 elements (8 key heads, 16 requests of 8000 to 24000 keys:
// groups of 16 162 us, with two rows of eight 273 us, groups of 8 155 us); what is
// past that makes further rows of the same keys.
//
// Loads. Each warp has a ring of three 8 KB items in shared memory, keys and
// values of its units in turn, filled by 16-byte asynchronous copies of all lanes
// (swizzled, so that ldmatrix is free of bank conflicts); no warp waits for
// another one until its part is done. Up to 192 KB an SM are in flight, and a warp
// hardly ever waits for a copy to land (under 1 % of a long row's time). Tensor-map boxes in
// their place cost 105 to 185 cycles each to issue, a box a page and 128 bytes: 94.5 against
// 88.4 us for one row of 131071 keys in pages of 64, 132 against 119 us for 8-bit rows of
// 80 elements in pages of 24. Keys outside a request are filled with zeros in shared
// memory, so that nothing a page holds behind them reaches a product.
//
// Measured, from the fastest machine to the slowest (a plain copy runs at 6685 to 6791 GB/s): 128 requests of
// 1000 to 16000 keys, 2.85 GB, 438 to 449 us (6.51 to 6.36 TB/s); one of 131071, 537 MB, 87.8 to 89.8 us (6.11 to
// 5.98 TB/s); 16 of 20000 to 60000 on an 8-bit cache, 1.2 GB, 188 to 212 us (6.39 to 5.66 TB/s); 32 of 200 to 4500, 184 MB,
// 39.5 to 40.5 us, of which about 12 are the beginning and the joins.
#pragma once

#include <cmath>

#include "decode.cuh"
#include "gemv.h"

namespace ninfer {
namespace attention {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kItems = 3;
constexpr uint32_t kItemBytes = 8192;
constexpr uint32_t kRingBytes = kWarps * kItems * kItemBytes;
constexpr uint32_t kNone = 0xffffffffu;
// What beginning a row costs, in units: its queries, its first copies, its output. 0, 1, 2, 3 and 4
// measured 42.7, 41.4, 40.5, 39.5 and 39.6 us for 32 requests of 200 to 4500 keys and 24.2, 21.7, 20.2,
// 20.2 and 21.5 us for 24 of 1 to 3001 with 16 key heads each; no change for long rows.
constexpr uint32_t kRowCost = 3;

struct AttentionParams {
    const uint8_t *k, *v;
    const void *q;
    const int32_t *table, *lengths;
    void *out;
    float *lse;
    uint4 *meta;                        // per CTA: row of its tail, whether its head part ends a row, and has one
    float2 *cta_ml;                     // [CTA][2][heads of a row]: m, l
    float4 *cta_o, *warp_o;             // [CTA][2] and [CTA][warp] sums, in fragment order
    int64_t q_request, q_head, table_stride;
    uint64_t page_bytes, token_bytes, head_bytes;       // strides of the pools
    float scale, v_scale;               // scale: of scores, in log2
    uint32_t requests, run, q_heads, group, head_dim, head_rows, pages, piece_log, window, most;
    uint32_t by_row, cluster_log;       // whether each cluster of 2^cluster_log CTAs has one row, and no other
    FastDiv page, tiles, heads;         // tokens a page, rows a key head, rows a request
    int q_dtype, out_dtype;
};

// 16 bytes into shared memory, or zeros where `bytes` is 0 (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but the last n groups of this thread's copies have landed.
template <int n>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two 8-bit floats as two binary16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

// What depends on the cache's type and the padded head width. Operands of the
// tensor cores are bfloat16 for a bfloat16 cache and binary16 for the other two.
template <int kDtype, int kWidth_, int kUsed, int kHeadTiles_>
struct Shape {
    static constexpr int kWidth = kWidth_;                      // elements of a row in shared memory
    static constexpr bool kBf16 = kDtype == NINFER_BF16, kBytes8 = kDtype == NINFER_E4M3;
    static constexpr int kHeadTiles = kHeadTiles_, kHeads = 8 * kHeadTiles;      // query heads of a row: 8 or 16
    static constexpr int kEs = kBytes8 ? 1 : 2;
    static constexpr int kKeys = kItemBytes / (kWidth * kEs);   // of a unit: 16, 32 or 64
    static constexpr int kSteps = kUsed / 16;                   // 16-element steps of a row that are computed
    static constexpr int kKeyTiles = kKeys / 16;
    // binary16 weights carry a factor 2^14: weights down to 2^-38 of the largest one keep a value
    static constexpr float kBias = kBf16 ? 0.f : 14.f;

    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        if (kBf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            return *reinterpret_cast<const uint32_t *>(&h);
        }
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        if (kBf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    // x as a sum of 16-bit values: the nearest one, the nearest to what remains, and so on
    template <int kTerms>
    static __device__ __forceinline__ void split(float a, float b, uint32_t (&term)[kTerms]) {
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {
            term[i] = pack(a, b);
            const float2 f = unpack(term[i]);
            a -= f.x;
            b -= f.y;
        }
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        if (kBf16)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    // Element of a row that accumulator row g (+ 8 * half) of value tile `tile` stands for.
    // 8-bit values leave ldmatrix.trans in pairs, so that rows g and g + 8 are neighbours.
    static __device__ __forceinline__ int element(int tile, int g, int half) {
        return 16 * tile + (kBytes8 ? 2 * g + half : g + 8 * half);
    }
};

// Keys of a request, and how many units they take.
struct Row {
    uint32_t from, end, units;
};

template <int kKeys>
__device__ __forceinline__ Row row_of(const AttentionParams &p, uint32_t request) {
    Row r;
    const int32_t n = p.lengths[request];
    r.end = n <= 0 ? 0u : min((uint32_t)n, p.most);
    r.from = p.window && r.end > p.window ? r.end - p.window : 0u;
    r.units = r.end ? (r.end + kKeys - 1) / kKeys - r.from / kKeys : 0u;
    return r;
}

// A place on the line of units.
struct Cursor {
    uint32_t request, head, unit;       // head: of the request's rows
    Row row;
};

template <int kKeys>
__device__ __forceinline__ void advance(const AttentionParams &p, Cursor &c) {
    if (++c.unit < c.row.units) return;
    c.unit = 0;
    if (++c.head < p.head_rows) return;
    c.head = 0;
    while (++c.request < p.requests) {
        c.row = row_of<kKeys>(p, c.request);
        if (c.row.units) return;
    }
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Where the output of a row, or of eight of its heads, lies.
struct Place {
    uint64_t head;      // the first query head
    uint32_t heads;     // how many
    __device__ __forceinline__ Place eight(int tile) const {
        return Place{head + 8 * tile, heads > 8u * tile ? min(8u, heads - 8 * tile) : 0u};
    }
};

template <class S>
__device__ __forceinline__ Place place_of(const AttentionParams &p, uint32_t request, uint32_t hr) {
    const uint32_t kvh = p.tiles.div(hr), first = (hr - kvh * p.tiles.d) * S::kHeads;
    return Place{(uint64_t)request * p.q_heads + kvh * p.group + first, min((uint32_t)S::kHeads, p.group - first)};
}

template <class S>
__device__ __forceinline__ Place place_of(const AttentionParams &p, uint32_t row) {
    const uint32_t request = p.heads.div(row);
    return place_of<S>(p, request, row - request * p.head_rows);
}

// One value tile of eight heads of a finished row, times r0 and r1 (v_scale / l of heads 2 t and 2 t + 1).
// 16-bit outputs are transposed in the registers, so that a lane has neighbouring elements of one head.
template <class S>
__device__ __forceinline__ void store_tile(const AttentionParams &p, const Place &at, int tile, int lane, const float4 &o, float r0,
                                           float r1) {
    const uint32_t g = lane >> 2, t = lane & 3;
    const float a = o.x * r0, b = o.y * r1, c = o.z * r0, d = o.w * r1;
    if (p.out_dtype == NINFER_F32) {
        float *to = static_cast<float *>(p.out) + (at.head + 2 * t) * p.head_dim;
        const uint32_t e = S::element(tile, g, 0), f = S::element(tile, g, 1);
        const bool first = 2 * t < at.heads, second = 2 * t + 1 < at.heads;
        if (e < p.head_dim) {
            if (first) to[e] = a;
            if (second) to[p.head_dim + e] = b;
        }
        if (f < p.head_dim) {
            if (first) to[f] = c;
            if (second) to[p.head_dim + f] = d;
        }
        return;
    }
    const bool bf = p.out_dtype == NINFER_BF16;
    const __nv_bfloat162 b0 = __floats2bfloat162_rn(a, b), b1 = __floats2bfloat162_rn(c, d);
    const __half2 h0 = __floats2half2_rn(a, b), h1 = __floats2half2_rn(c, d);
    // now lane (g, t) has head g's elements: 2 t and 2 t + 1 of the tile's first eight, and of its last eight
    const uint32_t x = movmatrix(bf ? *reinterpret_cast<const uint32_t *>(&b0) : *reinterpret_cast<const uint32_t *>(&h0));
    const uint32_t y = movmatrix(bf ? *reinterpret_cast<const uint32_t *>(&b1) : *reinterpret_cast<const uint32_t *>(&h1));
    if (g >= at.heads) return;
    uint16_t *to = static_cast<uint16_t *>(p.out) + (at.head + g) * p.head_dim + 16 * tile;
    if (S::kBytes8) {       // x: even elements 4 t, 4 t + 2; y: the odd ones between them
        if (16 * tile < (int)p.head_dim)
            *reinterpret_cast<uint2 *>(to + 4 * t) = make_uint2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
    } else {
        if (16 * tile < (int)p.head_dim) *reinterpret_cast<uint32_t *>(to + 2 * t) = x;
        if (16 * tile + 8 < (int)p.head_dim) *reinterpret_cast<uint32_t *>(to + 8 + 2 * t) = y;
    }
}

// ln of the sum of e^score for head `h` of `at`.
template <class S>
__device__ __forceinline__ void store_lse(const AttentionParams &p, const Place &at, uint32_t h, float m, float l) {
    if (p.lse && h < at.heads) p.lse[at.head + h] = l == 0.f ? -INFINITY : (m - S::kBias) * 0.693147180559945f + logf(l);
}

// What the sums of a row are multiplied by in the end; a row without weights gives zeros.
__device__ __forceinline__ float scale_of(const AttentionParams &p, float l) { return l == 0.f ? 0.f : p.v_scale / l; }

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// Parts of one value tile for heads 2 t and 2 t + 1, joined one by one.
struct Joined {
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float4 ml, float4 x) {      // ml: m and l of the two heads
        const float n0 = fmaxf(m0, ml.x), n1 = fmaxf(m1, ml.z);
        const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
        const float f0 = exp2_approx(m0 - u0), f1 = exp2_approx(m1 - u1), g0 = exp2_approx(ml.x - u0), g1 = exp2_approx(ml.z - u1);
        l0 = l0 * f0 + ml.y * g0;
        l1 = l1 * f1 + ml.w * g1;
        a.x = a.x * f0 + x.x * g0;
        a.y = a.y * f1 + x.y * g1;
        a.z = a.z * f0 + x.z * g0;
        a.w = a.w * f1 + x.w * g1;
        m0 = n0;
        m1 = n1;
    }
};

template <class S>
__device__ __forceinline__ void store_joined(const AttentionParams &p, const Place &at, int tile, int lane, const Joined &s) {
    store_tile<S>(p, at, tile, lane, s.a, scale_of(p, s.l0), scale_of(p, s.l1));
    if (tile == 0 && lane < 4) {
        store_lse<S>(p, at, 2 * lane, s.m0, s.l0);
        store_lse<S>(p, at, 2 * lane + 1, s.m1, s.l1);
    }
}

// kFull: as exact as fp32 operands. Queries and weights then enter as three bfloat16
// or two binary16 terms (24 and 22 bits). Otherwise the queries are of a 16-bit type
// that one term holds, and the output is rounded to 16 bits: weights have two
// bfloat16 terms (one would add as much error as that rounding), and one binary16
// term where the output is bfloat16 (2^-12 against 2^-9: the error grows by less than 1 %).
template <class S, bool kFull>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttentionParams p) {
    constexpr int kKeys = S::kKeys, kWidth = S::kWidth, kSteps = S::kSteps, kTiles = kSteps, kHeadTiles = S::kHeadTiles, kPart = kHeadTiles * kTiles * 32;
    constexpr int kQueryTerms = kFull ? S::kBf16 ? 3 : 2 : 1, kWeightTerms = S::kBf16 ? kFull ? 3 : 2 : kFull ? 2 : 1;
    extern __shared__ uint8_t ring_raw[];
    __shared__ uint64_t s_sum[kWarps], s_upto[kThreads];
    __shared__ uint32_t s_row[2 * kWarps], s_flags[2 * kWarps];
    __shared__ float2 s_ml[2 * kWarps][S::kHeads], s_total[2 * kWarps][S::kHeads];
    __shared__ float s_factor[2 * kWarps][S::kHeads];
    __shared__ __align__(16) float2 s_cta_ml[S::kHeads];     // of this CTA's part of the cluster's row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring_skip = (1024 - (smem_u32(ring_raw) & 1023)) & 1023;
    const uint32_t ring = smem_u32(ring_raw) + ring_skip + warp * (kItems * kItemBytes);
    if (lane < 2) s_row[2 * warp + lane] = kNone;
    if (threadIdx.x < S::kHeads) s_cta_ml[threadIdx.x] = make_float2(-INFINITY, -1.f);      // no sums (they are never negative)
    pdl_launch_dependents();
    pdl_wait();

    // ---- this warp's part of the line ----
    Cursor ld;
    uint32_t left = 0;          // of this warp's part: units, and kRowCost for each row that begins after the first
    bool empties = false;       // whether any request has no keys
    if (p.by_row) {
        const uint32_t row = blockIdx.x >> p.cluster_log, rank = blockIdx.x - (row << p.cluster_log);
        ld.request = p.heads.div(row);
        ld.head = row - ld.request * p.head_rows;
        ld.row = row_of<kKeys>(p, ld.request);
        // equal parts for the cluster's CTAs, and in them for the warps
        const uint32_t share = ld.row.units >> p.cluster_log, more = ld.row.units - (share << p.cluster_log);
        const uint32_t n = share + (rank < more), warp_share = n / kWarps, warp_more = n % kWarps;
        ld.unit = rank * share + min(rank, more) + warp * warp_share + min((uint32_t)warp, warp_more);
        left = warp_share + (warp < warp_more);
        empties = ld.row.units == 0 && ld.head == 0 && rank == 0;
    } else {
        const uint32_t r0 = min(threadIdx.x * p.run, p.requests), r1 = min(r0 + p.run, p.requests);
        uint64_t mine = 0;
        for (uint32_t r = r0; r < r1; ++r) {
            const uint32_t units = row_of<kKeys>(p, r).units;
            mine += units ? units + kRowCost : 0u;
            empties |= units == 0;
        }
        mine *= p.head_rows;
        uint64_t upto = mine;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const uint64_t a = __shfl_up_sync(~0u, upto, s);
            if (lane >= s) upto += a;
        }
        if (lane == 31) s_sum[warp] = upto;
        s_upto[threadIdx.x] = upto;     // within the warp
        empties = __syncthreads_or(empties);
        uint64_t total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += s_sum[w];
        // equal parts for the CTAs, of at least a unit a warp, and in them for the warps
        const uint32_t ctas = (uint32_t)min((uint64_t)gridDim.x, (total + kWarps - 1) / kWarps);
        uint64_t at = 0, n = 0;
        if (blockIdx.x < ctas) {
            const uint64_t share = total >> 32 ? total / ctas : (uint32_t)total / ctas;
            const uint32_t more = (uint32_t)(total - share * ctas);
            n = share + (blockIdx.x < more);
            at = blockIdx.x * share + min(blockIdx.x, more);
        }
        const uint32_t more = (uint32_t)n % kWarps;
        left = (uint32_t)(n / kWarps) + (warp < more);
        at += warp * (n / kWarps) + min((uint32_t)warp, more);
        if (left) {
            // the first run of requests that ends past `at`, then the request in it
            int w = 0;
            while (s_sum[w] <= at) at -= s_sum[w++];
            const uint32_t past = __ballot_sync(~0u, s_upto[32 * w + lane] > at), k = __ffs(past) - 1;
            if (k) at -= s_upto[32 * w + k - 1];
            const uint32_t run = 32 * w + k;
            ld.request = run * p.run;
            ld.row = row_of<kKeys>(p, ld.request);
            uint32_t size = ld.row.units ? ld.row.units + kRowCost : 0u;        // of one of the request's rows
            while (at >= (uint64_t)size * p.head_rows) {
                at -= (uint64_t)size * p.head_rows;
                ld.row = row_of<kKeys>(p, ++ld.request);
                size = ld.row.units ? ld.row.units + kRowCost : 0u;
            }
            ld.head = at >> 32 ? (uint32_t)(at / size) : (uint32_t)at / size;
            const uint32_t in_row = (uint32_t)(at - (uint64_t)ld.head * size), paid = min(in_row, kRowCost);
            ld.unit = in_row - paid;
            left -= min(left, kRowCost - paid);
        }
    }

    // ---- the ring: keys and values of the units in turn ----
    Cursor cp = ld;
    // A part that ends within the cost of a row's beginning leaves that row to the next part.
    auto spend = [](uint32_t left, bool row_ends) { return --left, row_ends ? left - min(left, kRowCost) : left; };
    uint32_t due = left, slot_in = 0, slot_out = 0;         // due: of what is not loaded yet
    constexpr int kRowUnits = kWidth * S::kEs / 16, kRowsAtOnce = 32 / kRowUnits;   // 16-byte units a row, rows a copy of the warp
    constexpr int kPieces = (kKeys + 31) / 32;
    // The unit that is loaded next is in pieces of 2^piece_log keys, each within one page; lane q has pieces q and q + 32.
    int32_t page[kPieces];
    uint32_t token[kPieces];
    const uint32_t pieces = kKeys >> p.piece_log;
    auto find_pages = [&] {
        const uint32_t base = (ld.row.from / kKeys + ld.unit) * kKeys;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t key = base + ((lane + 32 * i) << p.piece_log);
            page[i] = -1;
            if (lane + 32u * i < pieces && key < ld.row.end) {
                const uint32_t pg = p.page.div(key);
                token[i] = key - pg * p.page.d;
                page[i] = p.table[(int64_t)ld.request * p.table_stride + pg];
            }
        }
    };
    const uint32_t unit = lane & (kRowUnits - 1), unit_row = lane / kRowUnits;
    const uint32_t column = (unit >> 3) * (kKeys * 128) + unit_row * 128, turn = ((unit & 7) ^ (unit_row & 7)) << 4;
    const uint32_t in_piece = (1u << p.piece_log) - 1;
    auto load_item = [&](const uint8_t *pool) {
        // keys before `lo` or from `hi` on, and all of a unit past the head, are filled with zeros
        const uint32_t base = (ld.row.from / kKeys + ld.unit) * kKeys + unit_row;
        const uint32_t lo = ld.row.from > base ? ld.row.from - base : 0u;
        const uint32_t hi = unit * (16 / S::kEs) < p.head_dim && ld.row.end > base ? ld.row.end - base : 0u;
        const uint32_t to = ring + slot_in * kItemBytes + column;
        const uint64_t head = p.tiles.div(ld.head) * p.head_bytes;
        uint64_t at[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            at[i] = (uint32_t)page[i] < p.pages ? reinterpret_cast<uint64_t>(pool) + (uint32_t)page[i] * p.page_bytes + token[i] * p.token_bytes + head : 0u;
        const uint64_t none = reinterpret_cast<uint64_t>(pool), own = unit * 16;
        // where lane `unit_row`'s row of copy k comes from, or 0
        auto row_at = [&](int k) {
            const uint32_t r = k * kRowsAtOnce + unit_row, q = r >> p.piece_log;
            uint64_t from = __shfl_sync(~0u, at[0], q & 31);
            if (kPieces > 1) {
                const uint64_t more = __shfl_sync(~0u, at[kPieces - 1], q & 31);
                if (q >= 32) from = more;
            }
            return from;
        };
        auto copy = [&](int k, uint64_t from, bool on) {
            const uint32_t r = k * kRowsAtOnce;
            from += ((r + unit_row) & in_piece) * p.token_bytes + own;
            copy16(to + r * 128 + (turn ^ (r & 7) << 4), reinterpret_cast<const uint8_t *>(on ? from : none), on ? 16 : 0);
        };
        constexpr int kCopies = kKeys / kRowsAtOnce;
        if constexpr (S::kBytes8) {
#pragma unroll
            for (int k = 0; k < kCopies; ++k) {
                const uint64_t from = row_at(k);
                copy(k, from, from && k * kRowsAtOnce >= lo && k * kRowsAtOnce < hi);
            }
        } else {
            // 16-bit rows: units that lie in the request and in pages whole go without a test a copy (2.85 GB: 446
            // against 451 us); 8-bit rows took 2 to 5 % longer that way
            const bool whole = base >= ld.row.from + unit_row && base - unit_row + kKeys <= ld.row.end && pieces <= 32 && (at[0] || lane >= pieces);
            if (__all_sync(~0u, whole)) {
                const bool on = unit * (16 / S::kEs) < p.head_dim;
#pragma unroll
                for (int k = 0; k < kCopies; ++k) {
                    const uint32_t r = k * kRowsAtOnce + unit_row;
                    const uint64_t from = __shfl_sync(~0u, at[0], r >> p.piece_log) + ((r & in_piece) * (uint32_t)p.token_bytes + unit * 16);
                    copy16(to + k * kRowsAtOnce * 128 + (turn ^ (k * kRowsAtOnce & 7) << 4), reinterpret_cast<const uint8_t *>(from), on ? 16 : 0);
                }
            } else {
#pragma unroll 4
                for (int k = 0; k < kCopies; ++k) {
                    const uint64_t from = row_at(k);
                    copy(k, from, from && k * kRowsAtOnce >= lo && k * kRowsAtOnce < hi);
                }
            }
        }
        slot_in = slot_in == kItems - 1 ? 0 : slot_in + 1;
    };
    // one group an item, empty ones at the end, so that the oldest of three is always the one waited for
    auto load_keys = [&] {
        if (due) load_item(p.k);
        copies_commit();
    };
    auto load_values = [&] {
        if (due) {
            load_item(p.v);
            due = spend(due, ld.unit + 1 == ld.row.units);
            if (due) {
                advance<kKeys>(p, ld);
                find_pages();       // read early: the next unit's keys are asked for half a unit later
            }
        }
        copies_commit();
    };
    if (left) find_pages();
    auto wait_item = [&] {
        copies_wait<kItems - 1>();
        __syncwarp();
    };
    auto release_item = [&] {
        __syncwarp();
        slot_out = slot_out == kItems - 1 ? 0 : slot_out + 1;
    };

    // ---- the units ----
    // q[.][i][j]: elements 16 i .. 16 i + 15 of head g of each eight, the terms of the half j of a B operand.
    // m, l, sc, o: of heads 2 t and 2 t + 1 of each eight, as an accumulator has them.
    uint32_t q[kHeadTiles][kSteps][2][kQueryTerms];
    float o[kHeadTiles][kTiles][4], m0[kHeadTiles], m1[kHeadTiles], l0[kHeadTiles], l1[kHeadTiles], sc0[kHeadTiles], sc1[kHeadTiles];
    bool fresh = true, begun = false, primed = false;   // a new row's queries are due; it began in this part; loads run
    const uint32_t lane_row = lane & 7, lane_mat = lane >> 3;
    while (left) {
        const bool ends = cp.unit + 1 == cp.row.units;
        left = spend(left, ends);
        if (fresh) {
            fresh = false;
            begun = cp.unit == 0;
            const uint32_t kvh = p.tiles.div(cp.head), first = (cp.head - kvh * p.tiles.d) * S::kHeads + g;
#pragma unroll
            for (int ht = 0; ht < kHeadTiles; ++ht) {
                m0[ht] = m1[ht] = -INFINITY;
                l0[ht] = l1[ht] = 0.f;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) o[ht][i][0] = o[ht][i][1] = o[ht][i][2] = o[ht][i][3] = 0.f;
                const uint32_t h = first + 8 * ht;
                const int64_t at = (int64_t)cp.request * p.q_request + (int64_t)(kvh * p.group + h) * p.q_head;
                // all of a lane's loads first, then the first unit's copies, then the conversions
                float2 x[kSteps][2];
                const bool wide = p.q_dtype == NINFER_F32;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) x[i][0] = x[i][1] = make_float2(0.f, 0.f);
                // head_dim ends on a multiple of 8 (8-bit caches: 16), so that the lanes of a load stop together
                if (wide && h < p.group) {
                    const float2 *from = reinterpret_cast<const float2 *>(static_cast<const float *>(p.q) + at + (S::kBytes8 ? 4 : 2) * t);
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (16 * i + (S::kBytes8 ? 0 : 8 * j) < (int)p.head_dim) x[i][j] = from[8 * i + (S::kBytes8 ? j : 4 * j)];
                } else if (h < p.group) {
                    const uint32_t *from = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.q) + at + (S::kBytes8 ? 4 : 2) * t);
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (16 * i + (S::kBytes8 ? 0 : 8 * j) < (int)p.head_dim)
                                x[i][j].x = __uint_as_float(from[8 * i + (S::kBytes8 ? j : 4 * j)]);
                }
                if (!primed && ht == 0) {
                    load_keys();
                    load_values();
                }
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (!wide) {
                            const uint32_t u = __float_as_uint(x[i][j].x);
                            x[i][j] = p.q_dtype == NINFER_BF16 ? make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u))
                                                               : __half22float2(*reinterpret_cast<const __half2 *>(&u));
                        }
                        top = fmaxf(top, fmaxf(fabsf(x[i][j].x), fabsf(x[i][j].y)));
                    }
                float sc = p.scale, down = 1.f;
                if (!S::kBf16) {
                    // binary16 operands: a power of two brings the head's largest element to between 2^14 and 2^15, so that
                    // elements 2^-28 of it still have all of their bits (keys of zero may meet the largest one)
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    const int e = top > 0.f && top < INFINITY ? min(max((int)(__float_as_uint(top) >> 23), 27), 254) : 127 + 14;
                    down = __uint_as_float((uint32_t)(254 + 14 - e) << 23);
                    sc *= __uint_as_float((uint32_t)(e - 14) << 23);
                }
                sc0[ht] = __shfl_sync(~0u, sc, 8 * t);
                sc1[ht] = __shfl_sync(~0u, sc, 8 * t + 4);
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a = x[i][j].x * down, b = x[i][j].y * down;
                        S::split(a, b, q[ht][i][j]);
                        if (isinf(a) || isinf(b))                           // nothing remains: inf - inf
#pragma unroll
                            for (int k = 1; k < kQueryTerms; ++k) q[ht][i][j][k] = 0;
                    }
            }
            if (!primed) load_keys();
            primed = true;
        }
        const uint32_t base = (cp.row.from / kKeys + cp.unit) * kKeys;
        const bool edge = base < cp.row.from || base + kKeys > cp.row.end;

        // scores: keys g and g + 8 of each 16, heads 2 t and 2 t + 1
        wait_item();
        float s[kHeadTiles][S::kKeyTiles][4], r[kHeadTiles][S::kKeyTiles][4];        // of the queries' first terms, of the others
        float before[kHeadTiles][S::kKeyTiles][4];       // exact results of more than 128 elements: of all but the last 64
#pragma unroll
        for (int ht = 0; ht < kHeadTiles; ++ht)
#pragma unroll
            for (int i = 0; i < S::kKeyTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[ht][i][j] = r[ht][i][j] = before[ht][i][j] = 0.f;
        uint32_t item = ring + slot_out * kItemBytes;
        {
            const uint32_t lane_at = item + ((lane_mat & 1) * 8 + lane_row) * 128;
            constexpr int kUnits = S::kBytes8 ? 1 : 2;      // 16-byte units a step
#pragma unroll
            for (int i = 0; i < kSteps; i += 2 / kUnits) {
                if (kFull && kSteps > 8 && i && i % 4 == 0)      // (see add_values)
#pragma unroll
                    for (int ht = 0; ht < kHeadTiles; ++ht)
#pragma unroll
                        for (int n = 0; n < S::kKeyTiles; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                before[ht][n][j] += s[ht][n][j];
                                s[ht][n][j] = 0.f;
                            }
                const uint32_t unit = kUnits * i, at = lane_at + (unit >> 3) * (kKeys * 128) + ((((unit & 7) + (lane_mat >> 1)) ^ lane_row) << 4);
#pragma unroll
                for (int n = 0; n < S::kKeyTiles; ++n) {
                    uint32_t k[4];
                    ldmatrix4(k, at + n * 2048);
                    if constexpr (!S::kBytes8) {
#pragma unroll
                        for (int ht = 0; ht < kHeadTiles; ++ht) {
                            S::mma(s[ht][n], k, q[ht][i][0][0], q[ht][i][1][0]);
#pragma unroll
                            for (int m = 1; m < kQueryTerms; ++m) S::mma(r[ht][n], k, q[ht][i][0][m], q[ht][i][1][m]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t a[4] = {e4m3x2_to_f16x2(k[2 * j]), e4m3x2_to_f16x2(k[2 * j + 1]),
                                                   e4m3x2_to_f16x2(k[2 * j] >> 16), e4m3x2_to_f16x2(k[2 * j + 1] >> 16)};
#pragma unroll
                            for (int ht = 0; ht < kHeadTiles; ++ht) {
                                S::mma(s[ht][n], a, q[ht][i + j][0][0], q[ht][i + j][1][0]);
#pragma unroll
                                for (int m = 1; m < kQueryTerms; ++m) S::mma(r[ht][n], a, q[ht][i + j][0][m], q[ht][i + j][1][m]);
                            }
                        }
                    }
                }
            }
        }
        release_item();
        load_values();      // of the next unit
        // weights, transposed to a B operand: head g, keys 2 t and 2 t + 1 of each eight
        uint32_t w[kHeadTiles][S::kKeyTiles][2][kWeightTerms];
#pragma unroll
        for (int ht = 0; ht < kHeadTiles; ++ht) {
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < S::kKeyTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // an infinite score stands: a term of 0 times an infinite key is NaN
                    if constexpr (kFull && kSteps > 8) s[ht][i][j] += before[ht][i][j];
                    if constexpr (kFull) s[ht][i][j] = isinf(s[ht][i][j]) ? s[ht][i][j] : s[ht][i][j] + r[ht][i][j];
                    s[ht][i][j] *= j & 1 ? sc1[ht] : sc0[ht];
                    if (edge) {
                        const uint32_t key = base + 16 * i + g + (j & 2 ? 8 : 0);
                        if (key < cp.row.from || key >= cp.row.end) s[ht][i][j] = -INFINITY;
                    }
                    if (j & 1) top1 = fmaxf(top1, s[ht][i][j]);
                    else top0 = fmaxf(top0, s[ht][i][j]);
                }
#pragma unroll
            for (int b = 4; b <= 16; b <<= 1) {
                top0 = fmaxf(top0, __shfl_xor_sync(~0u, top0, b));
                top1 = fmaxf(top1, __shfl_xor_sync(~0u, top1, b));
            }
            top0 = fmaxf(m0[ht], top0);
            top1 = fmaxf(m1[ht], top1);
            if (__any_sync(~0u, top0 != m0[ht] || top1 != m1[ht])) {
                const float f0 = top0 == -INFINITY ? 1.f : exp2_approx(m0[ht] - top0), f1 = top1 == -INFINITY ? 1.f : exp2_approx(m1[ht] - top1);
                l0[ht] *= f0;
                l1[ht] *= f1;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    o[ht][i][0] *= f0;
                    o[ht][i][1] *= f1;
                    o[ht][i][2] *= f0;
                    o[ht][i][3] *= f1;
                }
                m0[ht] = top0;
                m1[ht] = top1;
            }
            const float shift0 = (m0[ht] == -INFINITY ? 0.f : m0[ht]) - S::kBias, shift1 = (m1[ht] == -INFINITY ? 0.f : m1[ht]) - S::kBias;
#pragma unroll
            for (int i = 0; i < S::kKeyTiles; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float a = exp2_approx(s[ht][i][2 * j] - shift0), b = exp2_approx(s[ht][i][2 * j + 1] - shift1);
                    l0[ht] += a;
                    l1[ht] += b;
                    S::split(a, b, w[ht][i][j]);
#pragma unroll
                    for (int m = 0; m < kWeightTerms; ++m) w[ht][i][j][m] = movmatrix(w[ht][i][j][m]);
                }
        }

        // The matrix unit cuts its sums off where they are aligned, always towards zero: over the 2200 keys of a
        // warp's part that added up to 5e-6 of the result. Exact results therefore sum every 16 keys by themselves and
        // add them rounded: 6e-7, for 0.3 to 4 % of the time (24 x 1 to 3001 keys, 16 heads of 80: 20.5 us before, 21.0 now).
        auto add_values = [](float (&to)[4], const uint32_t (&a)[4], const uint32_t (&w)[2][kWeightTerms]) {
            float own[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < kWeightTerms; ++m) S::mma(kFull ? own : to, a, w[0][m], w[1][m]);
#pragma unroll
            for (int j = 0; j < 4 * kFull; ++j) to[j] += own[j];
        };
        wait_item();
        item = ring + slot_out * kItemBytes;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk) {
            if constexpr (!S::kBytes8) {
                const uint32_t lane_at = item + (16 * kk + (lane_mat >> 1) * 8 + lane_row) * 128;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    uint32_t a[4];
                    ldmatrix4_trans(a, lane_at + (i >> 2) * (kKeys * 128) + (((2 * (i & 3) + (lane_mat & 1)) ^ lane_row) << 4));
#pragma unroll
                    for (int ht = 0; ht < kHeadTiles; ++ht) add_values(o[ht][i], a, w[ht][kk]);
                }
            } else {
                const uint32_t lane_at = item + (16 * kk + (lane_mat & 1) * 8 + lane_row) * 128;
#pragma unroll
                for (int i = 0; i < kTiles; i += 2) {
                    uint32_t r[4];
                    ldmatrix4_trans(r, lane_at + (i >> 3) * (kKeys * 128) + ((((i & 7) + (lane_mat >> 1)) ^ lane_row) << 4));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t x = __byte_perm(r[2 * j], 0, 0x3120), y = __byte_perm(r[2 * j + 1], 0, 0x3120);
                        const uint32_t a[4] = {e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y),
                                               e4m3x2_to_f16x2(y >> 16)};
#pragma unroll
                        for (int ht = 0; ht < kHeadTiles; ++ht) add_values(o[ht][i + j], a, w[ht][kk]);
                    }
                }
            }
        }
        release_item();
        load_keys();        // of the unit after that

        if (ends || !left) {
            const bool whole = begun && ends && !p.cluster_log;
            const int slot = 2 * warp + (begun ? 1 : 0);
            // at the end of the warp's part its ring is free, and holds the sums until they are joined
            float4 *to = left ? p.warp_o + ((uint64_t)blockIdx.x * kWarps + warp) * kPart
                              : reinterpret_cast<float4 *>(ring_raw + ring_skip + warp * (kItems * kItemBytes)) + (slot & 1) * kPart;
#pragma unroll
            for (int ht = 0; ht < kHeadTiles; ++ht) {
                float a0 = l0[ht], a1 = l1[ht];
#pragma unroll
                for (int b = 4; b <= 16; b <<= 1) {
                    a0 += __shfl_xor_sync(~0u, a0, b);
                    a1 += __shfl_xor_sync(~0u, a1, b);
                }
                if (whole) {
                    const Place at = place_of<S>(p, cp.request, cp.head).eight(ht);
                    const float r0 = scale_of(p, a0), r1 = scale_of(p, a1);
#pragma unroll
                    for (int i = 0; i < kTiles; ++i)
                        store_tile<S>(p, at, i, lane, make_float4(o[ht][i][0], o[ht][i][1], o[ht][i][2], o[ht][i][3]), r0, r1);
                    if (g == 0) {
                        store_lse<S>(p, at, 2 * t, m0[ht], a0);
                        store_lse<S>(p, at, 2 * t + 1, m1[ht], a1);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kTiles; ++i)
                        to[32 * (ht * kTiles + i) + lane] = make_float4(o[ht][i][0], o[ht][i][1], o[ht][i][2], o[ht][i][3]);
                    if (g == 0) {
                        s_ml[slot][8 * ht + 2 * t] = make_float2(m0[ht], a0);
                        s_ml[slot][8 * ht + 2 * t + 1] = make_float2(m1[ht], a1);
                    }
                }
            }
            if (lane == 0 && !whole) {
                s_row[slot] = cp.request * p.head_rows + cp.head;
                s_flags[slot] = (begun ? 1u : 0u) | (ends ? 2u : 0u) | (left ? 4u : 0u);
            }
            fresh = true;
        }
        advance<kKeys>(p, cp);
    }
    if (empties) {
        // requests without keys: by_row CTAs look at their own, others share them out
        const uint32_t step = p.by_row ? p.requests : gridDim.x;
        for (uint32_t r = p.by_row ? p.heads.div(blockIdx.x >> p.cluster_log) : blockIdx.x; r < p.requests; r += step) {
            if (row_of<kKeys>(p, r).units) continue;
            for (uint32_t i = threadIdx.x; i < p.q_heads * p.head_dim; i += kThreads)
                store1(p.out, (uint64_t)r * p.q_heads * p.head_dim + i, p.out_dtype, 0.f);
            if (p.lse)
                for (uint32_t i = threadIdx.x; i < p.q_heads; i += kThreads) p.lse[(uint64_t)r * p.q_heads + i] = -INFINITY;
        }
    }
    __syncthreads();

    // ---- rows cut between warps, joined in order; what is still cut goes to the cluster or the second kernel ----
    // slot j of a warp's parts: row, flags, and the slots that hold parts of the same row
    const int mine = lane & (2 * kWarps - 1);
    const uint32_t slot_row = s_row[mine], slot_flags = s_flags[mine];
    const uint32_t slot_mask = __match_any_sync(~0u, slot_row) & (slot_row == kNone ? 0u : (1u << (2 * kWarps)) - 1);
    {
        const int j = threadIdx.x >> 4, h = threadIdx.x & (S::kHeads - 1);     // (two threads an entry of eight heads, the same value)
        const uint32_t mask = __shfl_sync(~0u, slot_mask, j);
        float2 ml[2 * kWarps];
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kWarps; ++i) {
            ml[i] = mask >> i & 1 ? s_ml[i][h] : make_float2(-INFINITY, 0.f);
            top = fmaxf(top, ml[i].x);
        }
        const float u = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < 2 * kWarps; ++i) sum = fmaf(ml[i].y, exp2_approx(ml[i].x - u), sum);
        s_total[j][h] = make_float2(top, sum);
        s_factor[j][h] = mask >> j & 1 ? exp2_approx(s_ml[j][h].x - u) : 0.f;
    }
    __syncthreads();
    // behind the two parts that warp 0's ring may hold, room for what the cluster's other CTAs read
    static_assert(3 * kPart * sizeof(float4) <= kItems * kItemBytes, "three parts fit a warp's ring");
    float4 *cta_o = reinterpret_cast<float4 *>(ring_raw + ring_skip) + 2 * kPart;
    uint4 meta = make_uint4(kNone, 0, 0, 0);
    uint32_t starts = __ballot_sync(~0u, lane < 2 * kWarps && (slot_mask & ((2u << lane) - 1)) == 1u << lane);
    for (; starts; starts &= starts - 1) {
        const int i = __ffs(starts) - 1;
        const uint32_t row = __shfl_sync(~0u, slot_row, i), mask = __shfl_sync(~0u, slot_mask, i);
        const bool begins = __shfl_sync(~0u, slot_flags, i) & 1, ends = __shfl_sync(~0u, slot_flags, 31 - __clz(mask)) & 2;
        const bool whole = begins && ends && !p.cluster_log;
        const uint32_t outside = __ballot_sync(~0u, slot_flags & 4);        // slots whose sums lie in the workspace
        const uint64_t part = (uint64_t)blockIdx.x * 2 + (begins ? 1 : 0);
        const Place place = place_of<S>(p, row);
        for (int job = warp; job < kHeadTiles * kTiles; job += kWarps) {
            const int ht = kHeadTiles == 1 ? 0 : job / kTiles, tile = job - ht * kTiles, h0 = 8 * ht + 2 * t;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), x[kWarps];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int n = 0; n < kWarps; ++n) {
                    const int j = kWarps * half + n;
                    x[n] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (!(mask >> j & 1)) continue;
                    const float4 *from = outside >> j & 1 ? p.warp_o + ((uint64_t)blockIdx.x * kWarps + (j >> 1)) * kPart
                                                          : reinterpret_cast<const float4 *>(ring_raw + ring_skip + (j >> 1) * (kItems * kItemBytes)) + (j & 1) * kPart;
                    x[n] = from[32 * job + lane];
                }
#pragma unroll
                for (int n = 0; n < kWarps; ++n) {
                    const int j = kWarps * half + n;
                    const bool on = mask >> j & 1;
                    const float f0 = on ? s_factor[j][h0] : 0.f, f1 = on ? s_factor[j][h0 + 1] : 0.f;
                    a.x = fmaf(x[n].x, f0, a.x);
                    a.y = fmaf(x[n].y, f1, a.y);
                    a.z = fmaf(x[n].z, f0, a.z);
                    a.w = fmaf(x[n].w, f1, a.w);
                }
            }
            if (whole) store_tile<S>(p, place.eight(ht), tile, lane, a, scale_of(p, s_total[i][h0].y), scale_of(p, s_total[i][h0 + 1].y));
            else if (p.cluster_log) cta_o[32 * job + lane] = a;
            else p.cta_o[part * kPart + 32 * job + lane] = a;
        }
        if (warp == 0 && lane < S::kHeads) {
            const float2 ml = s_total[i][lane];
            if (whole) store_lse<S>(p, place, lane, ml.x, ml.y);
            else if (p.cluster_log) s_cta_ml[lane] = ml;
            else p.cta_ml[part * S::kHeads + lane] = ml;
        }
        if (!whole) {
            if (begins) meta.x = row;
            else {
                meta.y = ends ? 1u : 0u;
                meta.z = 1u;
            }
        }
    }
    if (!p.by_row) {
        if (threadIdx.x == 0) p.meta[blockIdx.x] = meta;
        return;
    }
    if (!p.cluster_log) return;

    // ---- the cluster's row: each CTA joins some of its value tiles, from all CTAs' shared memory ----
    const uint32_t row = blockIdx.x >> p.cluster_log, ctas = 1u << p.cluster_log, rank = blockIdx.x - (row << p.cluster_log);
    cluster_sync();
    const Place place = place_of<S>(p, row);
    for (int job = rank * kWarps + warp; job < kHeadTiles * kTiles; job += kWarps << p.cluster_log) {
        const int ht = kHeadTiles == 1 ? 0 : job / kTiles;
        Joined sum;
        for (uint32_t c = 0; c < ctas; ++c) {
            const float4 ml = load_cluster(mapa_shared(smem_u32(&s_cta_ml[8 * ht + 2 * t]), c));
            // a CTA without keys has written no sums; one whose scores are all NaN or -infinity has
            if (ml.y < 0.f) continue;
            sum.add(ml, load_cluster(mapa_shared(smem_u32(cta_o + 32 * job + lane), c)));
        }
        store_joined<S>(p, place.eight(ht), job - ht * kTiles, lane, sum);
    }
    cluster_sync();             // no CTA goes while another reads its shared memory
}

// Joins the rows that were cut between CTAs: block (c, value tile of eight heads) takes the row whose
// first part is CTA c's tail, if there is one, through the head parts of the
// following CTAs up to the one that ends it.
template <class S>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ AttentionParams p, uint32_t ctas) {
    constexpr int kTiles = S::kSteps, kPart = S::kHeadTiles * kTiles * 32;
    __shared__ uint32_t s_last;
    __shared__ float4 s_ml[kWarps][4], s_o[kWarps][32];     // m and l of heads 2 t and 2 t + 1
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
    const uint32_t c = blockIdx.x, job = blockIdx.y, ht = job / kTiles, tile = job - ht * kTiles;
    if (threadIdx.x == 0) s_last = ctas - 1;
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t row = p.meta[c].x;
    __syncthreads();
    for (uint32_t i = c + 1 + threadIdx.x; i < ctas; i += kThreads) {
        const uint4 meta = p.meta[i];
        if (meta.z && meta.y) {
            atomicMin(&s_last, i);
            break;
        }
    }
    if (row == kNone) return;
    __syncthreads();
    // part 0 is CTA c's tail, part i the head of CTA c + i; each warp joins every eighth, then the warps
    const uint32_t parts = s_last - c + 1;
    Joined sum;
#pragma unroll 4
    for (uint32_t i = warp; i < parts; i += kWarps) {
        const uint64_t at = (uint64_t)(c + i) * 2 + (i ? 0 : 1);
        sum.add(reinterpret_cast<const float4 *>(p.cta_ml)[(at * S::kHeadTiles + ht) * 4 + t], p.cta_o[at * kPart + 32 * job + lane]);
    }
    if (lane < 4) s_ml[warp][lane] = make_float4(sum.m0, sum.l0, sum.m1, sum.l1);
    s_o[warp][lane] = sum.a;
    __syncthreads();
    if (warp) return;
    for (uint32_t w = 1; w < min(parts, (uint32_t)kWarps); ++w) sum.add(s_ml[w][t], s_o[w][lane]);
    const Place place = place_of<S>(p, row).eight(ht);
    store_joined<S>(p, place, tile, lane, sum);
}

struct Instance {
    void (*attention)(const AttentionParams), (*join)(const AttentionParams, uint32_t);
    uint32_t used, keys, heads;         // elements computed, keys of a unit, query heads of a row
};

template <int kDtype, int kWidth, int kUsed, int kHeadTiles = 1>
Instance instance(bool full) {
    using S = Shape<kDtype, kWidth, kUsed, kHeadTiles>;
    return Instance{full ? attention_kernel<S, true> : attention_kernel<S, false>, join_kernel<S>, kUsed, (uint32_t)S::kKeys,
                    (uint32_t)S::kHeads};
}

// The instances of one cache type each, in files of their own so that they compile side by side.
// Rows are 128, 256 or 512 bytes in shared memory (64, 128 or 256 elements, of 8 bits 128 or 256).
Instance instance_bf16(uint64_t head_dim, uint64_t group, bool full);
Instance instance_f16(uint64_t head_dim, uint64_t group, bool full);
Instance instance_e4m3(uint64_t head_dim, uint64_t group, bool full);

}  // namespace attention
}  // namespace ninfer
