// ninfer_kv_append: new keys and values into the slots of a paged cache, and the
// rules of the cache description.
//
// Pure data movement: each source element is read once and each stored element
// written once, so HBM bounds it (latency, for the few rows of a decode step).
// One thread moves one 16-byte unit of the stored row (8 or 16 elements) of K and of V,
// all of its loads under way at once: 30011 tokens of 4 x 256 from fp32 rows into a bfloat16
// cache, 369 MB, 53.5 us (6.9 TB/s, the rate of a copy; K and V in threads of their own: 59.9 us).
// Scales cost what it takes to round their quotients once: the same tokens from bfloat16 into 8 bits 41.5 us for a power of
// two and for 0.0137, 58 for 0.3 (where each third bfloat16 value gives a quotient near a halfway point), 31.5 without a
// scale; from fp32 45.4 and 44.8; from bfloat16 into bfloat16 51 by 0.5, 72 by 0.3, 39.1 without. With an fp32 division
// each, which rounds twice, those with a scale took 49, 47 and 49.5 us.
#include "decode.cuh"

namespace ninfer {

int check_cache(const ninfer_kv_cache *c, const char *who) {
    if (!c || !c->k || !c->v) return fail(NINFER_ERR_INVALID_ARGUMENT, "%s: NULL cache, k or v", who);
    if (!cache_dtype_valid(c->dtype)) return fail(NINFER_ERR_INVALID_ARGUMENT, "%s: cache dtype %d unsupported", who, c->dtype);
    if (!(c->k_scale > 0) || !(c->v_scale > 0) || !std::isfinite(c->k_scale) || !std::isfinite(c->v_scale))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "%s: cache scales must be finite and positive", who);
    if (c->reserved) return fail(NINFER_ERR_INVALID_ARGUMENT, "%s: cache.reserved must be 0", who);
    const uint64_t es = cache_dtype_size(c->dtype), unit = 16 / es, most = 0x7fffffffull;
    if (!c->pages || !c->page_size || !c->kv_heads || c->pages > most || c->page_size > most || c->kv_heads > 65535)
        return fail(NINFER_ERR_SHAPE, "%s: cache of %llu pages of %llu tokens, %llu heads", who,
                    (unsigned long long)c->pages, (unsigned long long)c->page_size, (unsigned long long)c->kv_heads);
    if (!c->head_dim || c->head_dim > 256 || c->head_dim % unit)
        return fail(NINFER_ERR_SHAPE, "%s: head_dim %llu is not a multiple of %llu up to 256", who,
                    (unsigned long long)c->head_dim, (unsigned long long)unit);
    const uint64_t strides[3] = {c->pages > 1 ? c->page_stride : 0, c->page_size > 1 ? c->token_stride : 0,
                                 c->kv_heads > 1 ? c->head_stride : 0};
    for (uint64_t s : strides) {
        if (s % unit) return fail(NINFER_ERR_ALIGNMENT, "%s: cache strides must be multiples of 16 bytes", who);
        if (s >= (1ull << 40) / es) return fail(NINFER_ERR_OVERFLOW, "%s: cache stride of 2^40 bytes or more", who);
    }
    if (strides[1] >= (1ull << 25) / es) return fail(NINFER_ERR_OVERFLOW, "%s: cache token_stride of 2^25 bytes or more", who);
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(NINFER_ERR_ALIGNMENT, "%s: k and v must be 16-byte aligned", who);
    return NINFER_OK;
}

namespace {

struct AppendParams {
    const uint8_t *src[2];              // k_new, v_new
    uint8_t *dst[2];                    // cache.k, cache.v
    uint64_t src_token[2], src_head[2]; // source strides, elements
    uint64_t page_stride, token_stride, head_stride;
    float scale[2], inverse[2];         // 1 / scale, 0 where that is not a normal number
    bool exact[2];                      // scale is a power of two
    const int64_t *slots;
    uint64_t slot_count;                // of the cache
    uint32_t total;                     // 16-byte units of one of the two
    FastDiv units, heads, page;         // units a head, heads, tokens a page
    int src_dtype;
    int32_t *status;
};

// Eight floats, each divided by its scale, as 16 bytes of bf16 or f16 (kEs 2) or 8 bytes of e4m3 (kEs 1).
template <int kDtype>
__device__ __forceinline__ void pack8(const float (&x)[8], uint32_t *out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kDtype == NINFER_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            out[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else if (kDtype == NINFER_F16) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            out[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const uint32_t q = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            out[i / 2] = i & 1 ? out[i / 2] | (q << 16) : q;
        }
    }
}

// Bits of an fp32 value below half a step of the cache's type: where they are zero it may lie halfway between
// two values of that type.
template <int kDtype>
constexpr uint32_t kBelow = (1u << (kDtype == NINFER_BF16 ? 15 : kDtype == NINFER_F16 ? 12 : 19)) - 1;

// `near`, a value with zeros for those bits, or its neighbour on the side that the remainder r = x - near * scale tells:
// rounding it to the cache's type is rounding x / scale once. `other` where there is no remainder (infinite x, NaN).
__device__ __forceinline__ float beside(float near, float other, float r) {
    const int32_t bits = __float_as_int(near), step = (__float_as_int(r) ^ bits) >> 31 | 1;
    return r != r ? other : __int_as_float(r == 0.f ? bits : bits + step);
}

// x / scale from the fp32 quotient; for values that few caches see.
template <int kDtype>
__device__ __noinline__ float quotient(float x, float scale) {
    const float q = __fdiv_rn(x, scale);
    if (__float_as_uint(q) & kBelow<kDtype>) return q;
    // the remainder's lowest bit is at least 2^-36 of x, so that it is exact (and not lost under 2^-149) from 2^-113 on
    const float up = fabsf(x) < 0x1p-100f ? 0x1p64f : 1.f;
    return beside(q, q, fmaf(-q, scale * up, x * up));
}

// x / scale for one rounding to the cache's type, which pack8 does. The product with 1 / scale is x / scale where scale is
// a power of two, and otherwise at most two units in its last place off, so that it rounds as x / scale does unless it
// lies within three of a halfway point. Under 2^-100 a remainder, and a product that bfloat16 holds, may lose bits.
template <int kDtype>
__device__ __forceinline__ void divide8(float (&x)[8], float scale, float inverse, bool exact) {
    float q[8];
    bool near = false, small = inverse == 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = x[i] * inverse;
        near |= ((__float_as_uint(q[i]) + 3) & kBelow<kDtype>) <= 6;
        small |= (kDtype == NINFER_BF16 ? fminf(fabsf(x[i]), fabsf(q[i])) : fabsf(x[i])) < 0x1p-100f && x[i] != 0.f;
    }
    if (small) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = quotient<kDtype>(x[i], scale);
        return;
    }
    if (near && !exact) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = __float_as_uint(q[i]) + 3;
            const float mid = __uint_as_float(bits & ~kBelow<kDtype>);
            if ((bits & kBelow<kDtype>) <= 6) q[i] = beside(mid, q[i], fmaf(-mid, scale, x[i]));
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = q[i];
}

// kScaled: a scale that is not 1. Caches without one go without the registers for it (32 against 40 or more: bfloat16
// into bfloat16 39.1 us, 43.8 in one instance for both). The least CTAs an SM are what each instance's registers allow
// with few spills or none (16-bit with a scale: 5, 6 and 8 CTAs 53.4, 50.7 and 60.0 us by 0.5).
template <int kDtype, bool kScaled>
__global__ void __launch_bounds__(256, kDtype == NINFER_E4M3 ? (kScaled ? 4 : 5) : kScaled ? 6 : 8) append_kernel(const __grid_constant__ AppendParams p) {
    constexpr uint32_t kEs = kDtype == NINFER_E4M3 ? 1 : 2, kUnit = 16 / kEs;
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;      // total < 2^31: the host splits longer calls
    if (i >= p.total) return;
    const uint32_t head_row = p.units.div(i), unit = i - head_row * p.units.d;
    const uint32_t token = p.heads.div(head_row), head = head_row - token * p.heads.d;
    const int64_t slot = p.slots[token];
    float x[2][kUnit];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint64_t from = token * p.src_token[w] + head * p.src_head[w] + unit * kUnit;
#pragma unroll
        for (uint32_t j = 0; j < kUnit; j += 8) load8(p.src[w], from + j, p.src_dtype, *reinterpret_cast<float(*)[8]>(x[w] + j));
    }
    if (slot < 0) return;
    if ((uint64_t)slot >= p.slot_count) {
        if (p.status && unit == 0 && head == 0) atomicOr(p.status, NINFER_KV_BAD_SLOT);
        return;
    }
    uint64_t page, in;
    if (p.slot_count >> 32) {
        page = (uint64_t)slot / p.page.d;
        in = (uint64_t)slot % p.page.d;
    } else {
        page = p.page.div((uint32_t)slot);
        in = (uint32_t)slot - (uint32_t)page * p.page.d;
    }
    const uint64_t to = (page * p.page_stride + in * p.token_stride + head * p.head_stride + unit * kUnit) * kEs;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t o[4];
#pragma unroll
        for (uint32_t j = 0; j < kUnit; j += 8) {
            float(&eight)[8] = *reinterpret_cast<float(*)[8]>(x[w] + j);
            if (kScaled) divide8<kDtype>(eight, p.scale[w], p.inverse[w], p.exact[w]);
            pack8<kDtype>(eight, o + j / 4);
        }
        *reinterpret_cast<uint4 *>(p.dst[w] + to) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <int kDtype>
auto kernel_of(bool scaled) {
    return scaled ? append_kernel<kDtype, true> : append_kernel<kDtype, false>;
}

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_kv_append(const void *k_new, const void *v_new, int src_dtype, uint64_t tokens,
                                uint64_t k_token_stride, uint64_t k_head_stride, uint64_t v_token_stride,
                                uint64_t v_head_stride, const int64_t *slots, const ninfer_kv_cache *cache,
                                int32_t *status, ninfer_stream stream) {
    int st = check_cache(cache, "append");
    if (st) return st;
    if (!k_new || !v_new || !slots) return fail(NINFER_ERR_INVALID_ARGUMENT, "append: NULL k_new, v_new or slots");
    if (!dtype_valid(src_dtype)) return fail(NINFER_ERR_INVALID_ARGUMENT, "append: source dtype %d unsupported", src_dtype);
    const uint64_t es = cache_dtype_size(cache->dtype), unit = 16 / es, aligned_elems = 16 / dtype_size(src_dtype);
    if (tokens == 0 || tokens > 0x7fffffffull) return fail(NINFER_ERR_SHAPE, "append: tokens must be 1 to 2^31 - 1");
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(slots, 8) || (status && !aligned(status, 4)))
        return fail(NINFER_ERR_ALIGNMENT, "append: k_new and v_new must be 16-byte, slots 8-byte aligned");
    if ((tokens > 1 && (k_token_stride % aligned_elems || v_token_stride % aligned_elems)) ||
        (cache->kv_heads > 1 && (k_head_stride % aligned_elems || v_head_stride % aligned_elems)))
        return fail(NINFER_ERR_ALIGNMENT, "append: source strides must be multiples of 16 bytes");
    AppendParams p;
    const uint64_t units = cache->head_dim / unit, per_token = units * cache->kv_heads;
    p.dst[0] = static_cast<uint8_t *>(cache->k);
    p.dst[1] = static_cast<uint8_t *>(cache->v);
    p.src_token[0] = k_token_stride;
    p.src_token[1] = v_token_stride;
    p.src_head[0] = k_head_stride;
    p.src_head[1] = v_head_stride;
    p.page_stride = cache->page_stride;
    p.token_stride = cache->token_stride;
    p.head_stride = cache->head_stride;
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    for (int w = 0; w < 2; ++w) {
        int e;
        p.inverse[w] = std::isnormal(1.f / p.scale[w]) ? 1.f / p.scale[w] : 0.f;
        p.exact[w] = p.inverse[w] != 0.f && std::frexp(p.scale[w], &e) == 0.5f;
    }
    p.slot_count = cache->pages * cache->page_size;
    p.units = FastDiv((uint32_t)units);
    p.heads = FastDiv((uint32_t)cache->kv_heads);
    p.page = FastDiv((uint32_t)cache->page_size);
    p.src_dtype = src_dtype;
    p.status = status;
    const bool scaled = cache->k_scale != 1.f || cache->v_scale != 1.f;
    const auto kernel = cache->dtype == NINFER_BF16  ? kernel_of<NINFER_BF16>(scaled)
                        : cache->dtype == NINFER_F16 ? kernel_of<NINFER_F16>(scaled)
                                                     : kernel_of<NINFER_E4M3>(scaled);
    // fewer than 2^31 units a launch: the kernel counts them in 32 bits
    const uint64_t step = ((1ull << 31) - 1) / per_token;
    for (uint64_t t = 0; t < tokens; t += step) {
        const uint64_t n = tokens - t < step ? tokens - t : step;
        p.src[0] = static_cast<const uint8_t *>(k_new) + t * k_token_stride * dtype_size(src_dtype);
        p.src[1] = static_cast<const uint8_t *>(v_new) + t * v_token_stride * dtype_size(src_dtype);
        p.slots = slots + t;
        p.total = (uint32_t)(n * per_token);
        st = launch_dependent("append", kernel, dim3((p.total + 255) / 256), dim3(256), 0,
                              (cudaStream_t)stream, p);
        if (st) return st;
    }
    return NINFER_OK;
}
