// ninfer_kv_attention: attention of one new token per request over a paged cache.
//
// One pass over the keys with a running maximum m and sum l: a new score s
// rescales what was summed by e^{m - max(m, s)}. One CTA per (request, query
// head); its warps take every eighth key, each lane eight elements of the row,
// and join their (m, l, sum) at the end.
#include <cmath>

#include "decode.cuh"

namespace ninfer {
namespace {

struct AttentionParams {
    const void *q;
    const uint8_t *k, *v;
    const int32_t *table, *lengths;
    void *out;
    float *lse;
    uint64_t q_request, q_head, table_stride, page_stride, token_stride, head_stride, window;
    float scale, v_scale;       // scores: scale * k_scale
    uint32_t q_heads, group, head_dim, table_pages, pages;
    FastDiv page;
    int q_dtype, out_dtype, dtype;
};

__device__ __forceinline__ void load_cache8(const uint8_t *base, uint64_t idx, int dtype, float (&x)[8]) {
    if (dtype != NINFER_E4M3) {
        load8(base, idx, dtype, x);
        return;
    }
    const uint2 u = *reinterpret_cast<const uint2 *>(base + idx);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = ((j & 2) ? u.y : u.x) >> (16 * (j & 1));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffff), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}

__global__ void __launch_bounds__(256) attention_kernel(const AttentionParams p) {
    __shared__ float s_m[8], s_l[8], s_o[8][256];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t r = blockIdx.x / p.q_heads;
    const uint32_t h = blockIdx.x % p.q_heads, kvh = h / p.group, e = lane * 8;
    const bool on = e < p.head_dim;
    int64_t n = p.lengths[r];
    const int64_t most = (int64_t)p.table_pages * p.page.d;
    n = n < 0 ? 0 : n > most ? most : n;
    const int64_t from = p.window && (uint64_t)n > p.window ? n - (int64_t)p.window : 0;
    float q[8] = {}, o[8] = {}, m = -INFINITY, l = 0.f;
    if (on) load8(p.q, r * p.q_request + h * p.q_head + e, p.q_dtype, q);
    for (int64_t j = from + warp; j < n; j += 8) {
        const uint32_t pg = p.page.div((uint32_t)j);
        const int32_t page = p.table[r * p.table_stride + pg];
        const bool held = on && page >= 0 && (uint32_t)page < p.pages;
        const uint64_t at = (uint64_t)(held ? page : 0) * p.page_stride + (uint64_t)((uint32_t)j - pg * p.page.d) * p.token_stride +
                            kvh * p.head_stride + e;
        float k[8] = {}, v[8] = {}, s = 0.f;
        if (held) {
            load_cache8(p.k, at, p.dtype, k);
            load_cache8(p.v, at, p.dtype, v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int b = 16; b; b >>= 1) s += __shfl_xor_sync(~0u, s, b);
        s *= p.scale;
        const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - mu), w = expf(s - mu);
        l = fmaf(l, f, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(o[i], f, w * v[i]);
        m = mn;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    if (on)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_o[warp][e + i] = o[i];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < 8; ++w) top = fmaxf(top, s_m[w]);
    const float mu = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < 8; ++w) sum += s_l[w] * expf(s_m[w] - mu);
    const uint64_t row = r * p.q_heads + h;
    if (threadIdx.x == 0 && p.lse) p.lse[row] = top + logf(sum);
    if (threadIdx.x < p.head_dim) {
        float acc = 0.f;
        for (int w = 0; w < 8; ++w) acc += s_o[w][threadIdx.x] * expf(s_m[w] - mu);
        store1(p.out, row * p.head_dim + threadIdx.x, p.out_dtype, sum == 0.f ? 0.f : acc / sum * p.v_scale);
    }
}

int check_heads(const ninfer_kv_cache *cache, uint64_t requests, uint64_t q_heads) {
    if (!requests || !q_heads || requests > 0x7fffffffull || q_heads > 0x7fffffffull)
        return fail(NINFER_ERR_SHAPE, "attention: %llu requests of %llu heads", (unsigned long long)requests,
                    (unsigned long long)q_heads);
    if (q_heads % cache->kv_heads)
        return fail(NINFER_ERR_SHAPE, "attention: %llu query heads are not a multiple of %llu key heads",
                    (unsigned long long)q_heads, (unsigned long long)cache->kv_heads);
    if (requests * q_heads > 0x7fffffffull) return fail(NINFER_ERR_OVERFLOW, "attention: requests * q_heads over 2^31 - 1");
    return NINFER_OK;
}

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_kv_attention_workspace(const ninfer_kv_cache *cache, uint64_t requests, uint64_t q_heads,
                                             uint64_t *bytes) {
    int st = check_cache(cache, "attention workspace");
    if (!st) st = check_heads(cache, requests, q_heads);
    if (st) return st;
    if (!bytes) return fail(NINFER_ERR_INVALID_ARGUMENT, "attention workspace: NULL output");
    *bytes = 0;
    return NINFER_OK;
}

extern "C" int ninfer_kv_attention(const void *q, int q_dtype, uint64_t requests, uint64_t q_heads,
                                   uint64_t q_request_stride, uint64_t q_head_stride, const ninfer_kv_cache *cache,
                                   const int32_t *block_table, uint64_t table_pages, uint64_t table_stride,
                                   const int32_t *lengths, float scale, uint64_t window, void *out, int out_dtype,
                                   float *lse, void *workspace, uint64_t workspace_bytes, ninfer_stream stream) {
    uint64_t need = 0;
    int st = ninfer_kv_attention_workspace(cache, requests, q_heads, &need);
    if (st) return st;
    if (!q || !block_table || !lengths || !out)
        return fail(NINFER_ERR_INVALID_ARGUMENT, "attention: NULL q, block_table, lengths or out");
    if (!dtype_valid(q_dtype) || !dtype_valid(out_dtype))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "attention: q dtype %d or out dtype %d unsupported", q_dtype, out_dtype);
    if (!std::isfinite(scale)) return fail(NINFER_ERR_INVALID_ARGUMENT, "attention: scale must be finite");
    if (!table_pages || table_pages > 0x7fffffffull || (requests > 1 && table_stride < table_pages))
        return fail(NINFER_ERR_SHAPE, "attention: block table of %llu pages a row, %llu apart",
                    (unsigned long long)table_pages, (unsigned long long)table_stride);
    if (table_pages > 0x7fffffffull / cache->page_size)
        return fail(NINFER_ERR_OVERFLOW, "attention: table_pages * page_size over 2^31 - 1");
    const uint64_t unit = 16 / dtype_size(q_dtype);
    if (!aligned(q, 16) || !aligned(out, 16) || (requests > 1 && q_request_stride % unit) || (q_heads > 1 && q_head_stride % unit))
        return fail(NINFER_ERR_ALIGNMENT, "attention: q, out and the strides of q must be 16-byte aligned");
    if (!aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(lse, 4))
        return fail(NINFER_ERR_ALIGNMENT, "attention: block_table, lengths and lse must be 4-byte aligned");
    if (need && (!workspace || workspace_bytes < need))
        return fail(NINFER_ERR_SIZE_MISMATCH, "attention: workspace of %llu bytes needed, %llu given",
                    (unsigned long long)need, (unsigned long long)workspace_bytes);
    if (need && !aligned(workspace, 256)) return fail(NINFER_ERR_ALIGNMENT, "attention: workspace must be 256-byte aligned");
    AttentionParams p;
    p.q = q;
    p.k = static_cast<const uint8_t *>(cache->k);
    p.v = static_cast<const uint8_t *>(cache->v);
    p.table = block_table;
    p.lengths = lengths;
    p.out = out;
    p.lse = lse;
    p.q_request = q_request_stride;
    p.q_head = q_head_stride;
    p.table_stride = table_stride;
    p.page_stride = cache->page_stride;
    p.token_stride = cache->token_stride;
    p.head_stride = cache->head_stride;
    p.window = window;
    p.scale = scale * cache->k_scale;
    p.v_scale = cache->v_scale;
    p.q_heads = (uint32_t)q_heads;
    p.group = (uint32_t)(q_heads / cache->kv_heads);
    p.head_dim = (uint32_t)cache->head_dim;
    p.table_pages = (uint32_t)table_pages;
    p.pages = (uint32_t)cache->pages;
    p.page = FastDiv((uint32_t)cache->page_size);
    p.q_dtype = q_dtype;
    p.out_dtype = out_dtype;
    p.dtype = cache->dtype;
    return launch_dependent("attention", attention_kernel, dim3((unsigned)(requests * q_heads)), dim3(256), 0,
                            (cudaStream_t)stream, p);
}
