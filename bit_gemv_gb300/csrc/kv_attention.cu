// ninfer_kv_attention: argument checks, workspace, the choice of an instance and of
// how the work is divided. The kernels are in kv_attention.cuh.
#include "kv_attention.cuh"

namespace ninfer {
namespace {

using namespace attention;

Instance instance_of(const ninfer_kv_cache *c, uint64_t q_heads, int q_dtype, int out_dtype) {
    const uint64_t group = q_heads / c->kv_heads;
    if (c->dtype == NINFER_BF16) return instance_bf16(c->head_dim, group, q_dtype != NINFER_BF16 || out_dtype == NINFER_F32);
    const bool full = q_dtype == NINFER_F32 || out_dtype != NINFER_BF16;
    return c->dtype == NINFER_F16 ? instance_f16(c->head_dim, group, full) : instance_e4m3(c->head_dim, group, full);
}

struct Layout {
    uint64_t ml, cta_o, warp_o, bytes;      // offsets in the workspace
};

Layout layout(uint32_t ctas, const Instance &in) {
    const uint64_t part = (uint64_t)in.used * in.heads * sizeof(float);
    Layout w;
    w.ml = (uint64_t)ctas * sizeof(uint4);
    w.cta_o = (w.ml + (uint64_t)ctas * 2 * in.heads * sizeof(float2) + 255) / 256 * 256;
    w.warp_o = w.cta_o + ctas * 2 * part;
    w.bytes = w.warp_o + (uint64_t)ctas * kWarps * part;
    return w;
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
    DeviceInfo d;
    st = device_info(&d);
    if (st) return st;
    *bytes = layout(d.sms, instance_of(cache, q_heads, NINFER_F32, NINFER_F32)).bytes;
    return NINFER_OK;
}

extern "C" int ninfer_kv_attention(const void *q, int q_dtype, uint64_t requests, uint64_t q_heads,
                                   uint64_t q_request_stride, uint64_t q_head_stride, const ninfer_kv_cache *cache,
                                   const int32_t *block_table, uint64_t table_pages, uint64_t table_stride,
                                   const int32_t *lengths, float scale, uint64_t window, void *out, int out_dtype,
                                   float *lse, void *workspace, uint64_t workspace_bytes, ninfer_stream stream) {
    int st = check_cache(cache, "attention");
    if (!st) st = check_heads(cache, requests, q_heads);
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
    DeviceInfo d;
    st = device_info(&d);
    if (st) return st;
    const Instance in = instance_of(cache, q_heads, q_dtype, out_dtype);
    const Layout w = layout(d.sms, in);
    if (!workspace || workspace_bytes < w.bytes)
        return fail(NINFER_ERR_SIZE_MISMATCH, "attention: workspace of %llu bytes needed, %llu given",
                    (unsigned long long)w.bytes, (unsigned long long)(workspace ? workspace_bytes : 0));
    if (!aligned(workspace, 256)) return fail(NINFER_ERR_ALIGNMENT, "attention: workspace must be 256-byte aligned");
    AttentionParams p;
    // a piece of a unit lies in one page: the largest power of two that divides page_size, up to a unit's keys
    uint32_t piece = in.keys;
    while (cache->page_size % piece) piece /= 2;
    constexpr int kSmem = kRingBytes + 1024;
    st = set_smem_attribute(reinterpret_cast<const void *>(in.attention), kSmem);
    if (st) return st;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.q = q;
    p.table = block_table;
    p.lengths = lengths;
    p.out = out;
    p.lse = lse;
    p.meta = reinterpret_cast<uint4 *>(ws);
    p.cta_ml = reinterpret_cast<float2 *>(ws + w.ml);
    p.cta_o = reinterpret_cast<float4 *>(ws + w.cta_o);
    p.warp_o = reinterpret_cast<float4 *>(ws + w.warp_o);
    p.q_request = (int64_t)q_request_stride;
    p.q_head = (int64_t)q_head_stride;
    p.table_stride = (int64_t)table_stride;
    p.scale = scale * cache->k_scale * 1.44269504088896f;
    p.v_scale = cache->v_scale;
    p.requests = (uint32_t)requests;
    p.run = (uint32_t)((requests + kThreads - 1) / kThreads);
    p.q_heads = (uint32_t)q_heads;
    p.group = (uint32_t)(q_heads / cache->kv_heads);
    p.head_dim = (uint32_t)cache->head_dim;
    p.tiles = FastDiv((p.group + in.heads - 1) / in.heads);
    p.head_rows = (uint32_t)cache->kv_heads * p.tiles.d;
    p.heads = FastDiv(p.head_rows);
    p.pages = (uint32_t)cache->pages;
    p.piece_log = (uint32_t)__builtin_ctz(piece);
    const uint64_t es = cache_dtype_size(cache->dtype);
    p.k = static_cast<const uint8_t *>(cache->k);
    p.v = static_cast<const uint8_t *>(cache->v);
    p.page_bytes = cache->page_stride * es;
    p.token_bytes = cache->token_stride * es;
    p.head_bytes = cache->head_stride * es;
    p.most = (uint32_t)(table_pages * cache->page_size);
    p.window = window < p.most ? (uint32_t)window : 0;
    p.page = FastDiv((uint32_t)cache->page_size);
    p.q_dtype = q_dtype;
    p.out_dtype = out_dtype;
    // Few and short rows: a CTA, or a cluster of two, four or eight, for each, without a schedule and
    // a second kernel. The lengths are on the device, so that the table's width (or the window) stands for the longest row:
    // short rows under a table that is wider than these sizes are divided like long ones. On the GPU that costs 5 us (clusters: 7) and 1.8 us for every 8 units of a
    // CTA's part of the longest row; the division of the line costs 9 us (256 elements: 11) and
    // 1.8 us for every unit a warp. Measured, rows of 128 elements in 16 bits, clusters against the line:
    //   4 rows of 64 units 9.1 / 9.7 us, of 80 10.2 / 9.9;  16 of 32 8.0 / 9.5, of 80 10.9 / 10.2;  32 of 64
    //   9.8 / 11.8, of 128 13.1 / 13.4;  64 of 64 12.3 / 13.4, of 80 15.0 / 15.0;  144 (a CTA each) of 32 11.0 / 15.3.
    // Past 32 units a CTA, rows of different lengths would leave most of the SMs waiting. Clusters of
    // eight and four do not fill every SM (their SMs are neighbours): 5/6 and 9/10 are counted on.
    const uint64_t rows = requests * p.head_rows, sms = d.sms;
    const uint64_t longest = p.window ? std::min<uint64_t>(p.window, p.most) : p.most, units = (longest + in.keys - 1) / in.keys;
    const uint64_t room[4] = {sms, sms, sms * 9 / 10, sms * 5 / 6};
    p.by_row = 0;
    for (p.cluster_log = 4; p.cluster_log-- > 0;) {
        const uint64_t size = 1ull << p.cluster_log, ctas = rows * size;
        p.by_row = ctas <= room[p.cluster_log] && (size == 1 || units > 4 * size) && units <= 32 * size &&
                   units * (sms - ctas) <= (size == 1 ? 20 : 8 * size) * sms;
        if (p.by_row) break;
    }
    if (!p.by_row) p.cluster_log = 0;
    const unsigned cluster = 1u << p.cluster_log;
    st = launch_clusters("attention", cluster, in.attention, dim3((unsigned)(p.by_row ? rows * cluster : sms)), dim3(kThreads), kSmem,
                         (cudaStream_t)stream, p);
    if (st || p.by_row) return st;
    return launch_dependent("attention join", in.join, dim3(d.sms, in.used / 16 * in.heads / 8), dim3(kThreads), 0, (cudaStream_t)stream, p,
                            (uint32_t)d.sms);
}
