// ninfer_logits_process: penalties for repeated tokens, biases and grammar masks
// on the logits of the output head.
//
// One pass over the logits (read once, written once): HBM bounds a batch,
// latency a single row. A CTA owns a slice of one row's tokens and keeps a
// table of them in shared memory, one entry a token: how often it was answered,
// whether it was seen in the prompt, whether it has a bias; the slice's mask words
// stand behind it. It asks for the row's history, its mask words, its biases and its first
// logits at once, enters them into the table, and streams the slice through. Tokens
// with a bias are left out there and done one by one from the list, so that the
// biases need no table of their own.
//
// Slices. Every CTA of a row reads the row's whole history, so slices are as large
// as the table of a third of an SM allows, and as many as fill the SMs once: 64
// rows are 7 slices of about 35,500 tokens each. Twice as many measured 2 us less for
// 64 rows and 2 to 4 us more for 11 to 47.
//
// Measured: 64 rows of 248320 fp32 logits with histories of 16 to 8000 tokens, 28.1 to 28.7 us for
// 128 MB (18.8 us at the rate of a copy): 3.7 us until the table stands, 18 us of streaming, and the
// launch. Copying the untouched tokens at once, and doing the touched ones after the
// table, took 52 us (a dependent read for each of them). One row takes 2.3 us on the GPU.
#include <cmath>

#include "decode.cuh"
#include "gemv.h"

namespace ninfer {
namespace {

constexpr int kThreads = 384, kResident = 3;        // CTAs an SM
constexpr uint32_t kSmemBytes = 76800;              // of a CTA: three fit an SM
constexpr uint32_t kMostNarrow = 36096, kMostWide = 18560;      // tokens of a slice: (16 or 32) + 1 bits each
constexpr uint32_t kLeast = 2048;                   // tokens of a slice: a 16-byte load a thread

struct LogitsParams {
    const void *x;
    void *out;
    uint64_t x_stride, out_stride;
    ninfer_logits_controls c;
    int32_t *status;
    uint32_t vocab, slices, slice, mask_at;     // mask_at: word of shared memory where the mask words begin
    int dtype;
};

// Table entries. Histories below 2^14 tokens take 16 bits a token, longer ones 32.
template <bool kWide>
struct Entry;
template <>
struct Entry<false> {
    using Word = uint16_t;
    static constexpr uint32_t kPrompt = 0x8000u, kBias = 0x4000u, kCount = 0x3fffu;
    static __device__ __forceinline__ void set(uint32_t *table, uint32_t i, uint32_t flag) { atomicOr(table + (i >> 1), flag << (16 * (i & 1))); }
    static __device__ __forceinline__ void add(uint32_t *table, uint32_t i) { atomicAdd(table + (i >> 1), 1u << (16 * (i & 1))); }
};
template <>
struct Entry<true> {
    using Word = uint32_t;
    static constexpr uint32_t kPrompt = 0x80000000u, kBias = 0x40000000u, kCount = 0x3fffffffu;
    static __device__ __forceinline__ void set(uint32_t *table, uint32_t i, uint32_t flag) { atomicOr(table + i, flag); }
    static __device__ __forceinline__ void add(uint32_t *table, uint32_t i) { atomicAdd(table + i, 1u); }
};

template <int kDtype>
__device__ __forceinline__ float value(uint32_t w, int half) {
    if (kDtype == NINFER_F32) return __uint_as_float(w);
    if (kDtype == NINFER_BF16) return __uint_as_float(half ? w & 0xffff0000u : w << 16);
    return __half2float(__ushort_as_half((uint16_t)(half ? w >> 16 : w & 0xffff)));
}

template <int kDtype, bool kWide>
__global__ void __launch_bounds__(kThreads, kResident) logits_kernel(const __grid_constant__ LogitsParams p) {
    using E = Entry<kWide>;
    constexpr int kEs = kDtype == NINFER_F32 ? 4 : 2, kVec = 16 / kEs, kAhead = 2, kQuads = 6;
    constexpr int kMaskWords = ((kWide ? kMostWide : kMostNarrow) / 32 + kThreads - 1) / kThreads;
    extern __shared__ __align__(16) uint32_t table[];
    const uint32_t tid = threadIdx.x, row = blockIdx.x / p.slices, first = blockIdx.x % p.slices * p.slice;
    const uint32_t size = min(p.slice, p.vocab - first);
    for (uint32_t i = tid; i * 16 < size * (uint32_t)sizeof(typename E::Word); i += kThreads)
        reinterpret_cast<uint4 *>(table)[i] = make_uint4(0, 0, 0, 0);
    pdl_launch_dependents();
    pdl_wait();
    const uint8_t *x = static_cast<const uint8_t *>(p.x) + (row * p.x_stride + first) * kEs;
    uint8_t *out = static_cast<uint8_t *>(p.out) + (row * p.out_stride + first) * kEs;
    // the row's numbers, all asked for at once
    int32_t n = 0, told = 0, bias_from = 0, bias_to = 0, mask_row = -1;
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if (p.c.history) n = p.c.history_lengths[row];
    if (p.c.prompt_lengths) told = p.c.prompt_lengths[row];
    if (p.c.bias_ids) {
        bias_from = p.c.bias_offsets[row];
        bias_to = p.c.bias_offsets[row + 1];
    }
    if (p.c.mask) mask_row = p.c.mask_rows ? p.c.mask_rows[row] : (int32_t)row;
    if (p.c.repetition) rep = p.c.repetition[row];
    if (p.c.presence) pres = p.c.presence[row];
    if (p.c.frequency) freq = p.c.frequency[row];
    // rows on 16-byte boundaries go in vectors, others (and the last few tokens) one by one
    const uint32_t vecs = (p.x_stride * kEs) % 16 == 0 && (p.out_stride * kEs) % 16 == 0 ? size / kVec : 0;
    int bad = 0;
    n = min(max(n, 0), (int32_t)p.c.history_stride);
    const int32_t *h = p.c.history + row * p.c.history_stride;
    const bool quads = p.c.history_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.c.history) & 15) == 0;
    // the history before the logits, which would hold it up
    uint4 v[kQuads], ahead[kAhead];
    auto read_history = [&](int32_t i0) {
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const int32_t i = i0 + 4 * kThreads * k;
            v[k] = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (i >= n) continue;
            if (quads) v[k] = *reinterpret_cast<const uint4 *>(h + i);      // rows are whole quads long
            else {
                v[k].x = h[i];
                if (i + 1 < n) v[k].y = h[i + 1];
                if (i + 2 < n) v[k].z = h[i + 2];
                if (i + 3 < n) v[k].w = h[i + 3];
            }
        }
    };
    read_history(4 * tid);
    // a thread's first bias and its mask words; unsigned, so that an offset near 2^31 - 1 stays past the last entry
    const uint32_t b0 = min(max(bias_from, 0), (int32_t)p.c.bias_count), b1 = min(max(bias_to, 0), (int32_t)p.c.bias_count);
    const bool biased = b0 + tid < b1;
    uint32_t bias_token = ~0u;
    float bias_value = 0.f;
    if (biased) {
        bias_token = (uint32_t)p.c.bias_ids[b0 + tid];
        bias_value = p.c.bias_values[b0 + tid];
    }
    if (mask_row >= 0 && (uint64_t)mask_row >= p.c.mask_row_count) {
        bad = NINFER_LOGITS_BAD_TOKEN;
        mask_row = -1;
    }
    uint32_t *mask = table + p.mask_at, words[kMaskWords];
    if (mask_row >= 0) {
        const uint32_t *from = p.c.mask + mask_row * p.c.mask_stride + (first >> 5);
#pragma unroll
        for (int k = 0; k < kMaskWords; ++k)
            if ((tid + k * kThreads) * 32 < size) words[k] = from[tid + k * kThreads];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (tid + k * kThreads < vecs) ahead[k] = reinterpret_cast<const uint4 *>(x)[tid + k * kThreads];
    __syncthreads();            // the table is empty
    for (int32_t i0 = 4 * tid; i0 < n; i0 += 4 * kThreads * kQuads) {
        if (i0 != 4 * (int32_t)tid) read_history(i0);
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int32_t i = i0 + 4 * kThreads * k + j;
                if (i >= n) break;
                if (w[j] >= p.vocab) bad = NINFER_LOGITS_BAD_TOKEN;
                const uint32_t at = w[j] - first;
                if (at >= size) continue;
                if (i < told) E::set(table, at, E::kPrompt);
                else E::add(table, at);
            }
        }
    }
    if (biased && bias_token >= p.vocab) bad = NINFER_LOGITS_BAD_TOKEN;
    float bias_logit = 0.f;                 // of this thread's first bias, if it lies in the slice
    bias_token -= first;
    if (bias_token < size) {
        E::set(table, bias_token, E::kBias);
        bias_logit = load1(x, bias_token, kDtype);
    }
    for (uint32_t i = b0 + tid + kThreads; i < b1; i += kThreads) {
        const uint32_t v = (uint32_t)p.c.bias_ids[i];
        if (v >= p.vocab) bad = NINFER_LOGITS_BAD_TOKEN;
        if (v - first < size) E::set(table, v - first, E::kBias);
    }
    if (mask_row >= 0) {
#pragma unroll
        for (int k = 0; k < kMaskWords; ++k)
            if ((tid + k * kThreads) * 32 < size) mask[tid + k * kThreads] = words[k];
    }
    __syncthreads();

    const typename E::Word *entries = reinterpret_cast<const typename E::Word *>(table);
    // The product with the reciprocal rounds once more than a division (of each seen token: 29.5 against 28.4 us for the
    // 64 rows); a repetition whose reciprocal is no normal number would lose bits or the value, and divides.
    const float less = 1.f / rep;
    const bool divide = !(fabsf(less) >= 0x1p-126f && fabsf(less) < INFINITY);
    auto penalised = [&](float v, uint32_t e) {         // an empty entry leaves v as it is
        if (divide) v = e ? v > 0.f ? v / rep : v * rep : v;
        else v *= e ? v > 0.f ? less : rep : 1.f;
        return v - (e & E::kCount ? fmaf(freq, (float)(e & E::kCount), pres) : 0.f);
    };
    auto one = [&](uint32_t i, float v, float bias) {       // token `i` of the slice, whose logit is v
        v = penalised(v, entries[i] & (E::kPrompt | E::kCount)) + bias;
        if (mask_row >= 0 && !(mask[i >> 5] >> (i & 31) & 1)) v = -INFINITY;
        store1(out, i, kDtype, v);
    };
    if (bias_token < size) one(bias_token, bias_logit, bias_value);
    constexpr uint32_t kLowest = kDtype == NINFER_F32 ? 0xff800000u : kDtype == NINFER_BF16 ? 0xff80ff80u : 0xfc00fc00u;  // -infinity
    for (uint32_t g0 = tid; g0 < vecs; g0 += kAhead * kThreads) {
        uint4 now[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            now[k] = ahead[k];
            const uint32_t g = g0 + (kAhead + k) * kThreads;
            if (g < vecs) ahead[k] = reinterpret_cast<const uint4 *>(x)[g];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint32_t g = g0 + k * kThreads;
            if (g >= vecs) break;
            uint32_t w[4] = {now[k].x, now[k].y, now[k].z, now[k].w};
            // the vector's entries: kVec of them, 8 to 32 bytes
            uint32_t e[kVec * sizeof(typename E::Word) / 4], any = 0;
#pragma unroll
            for (int j = 0; j < (int)(sizeof e / 4); ++j) {
                e[j] = table[g * (sizeof e / 4) + j];
                any |= e[j];
            }
            uint32_t bits = ~0u;
            if (mask_row >= 0) bits = mask[g * kVec >> 5] >> (g * kVec & 31);
            if (any & (kWide ? E::kBias : E::kBias * 0x10001u)) {
                // a token with a bias is among them: the others alone
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (!(entries[g * kVec + j] & E::kBias)) one(g * kVec + j, value<kDtype>(w[j * kEs / 4], j & 1), 0.f);
                continue;
            }
            if (any) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const uint32_t ej = kWide ? e[j] : e[j / 2] >> (16 * (j & 1)) & 0xffffu;
                    const float v = penalised(value<kDtype>(w[j * kEs / 4], j & 1), ej);
                    if (kDtype == NINFER_F32) w[j] = __float_as_uint(v);
                    else {
                        const uint32_t r = kDtype == NINFER_BF16 ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v))
                                                                 : (uint32_t)__half_as_ushort(__float2half_rn(v));
                        w[j / 2] = j & 1 ? (w[j / 2] & 0xffffu) | r << 16 : (w[j / 2] & 0xffff0000u) | r;
                    }
                }
            }
            if (~bits & ((1u << kVec) - 1)) {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (!(bits >> j & 1)) {
                        if (kDtype == NINFER_F32) w[j] = kLowest;
                        else w[j / 2] = j & 1 ? (w[j / 2] & 0xffffu) | (kLowest & 0xffff0000u) : (w[j / 2] & 0xffff0000u) | (kLowest & 0xffffu);
                    }
            }
            reinterpret_cast<uint4 *>(out)[g] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    for (uint32_t i = vecs * kVec + tid; i < size; i += kThreads)
        if (!(entries[i] & E::kBias)) one(i, load1(x, i, kDtype), 0.f);
    for (uint32_t i = b0 + tid + kThreads; i < b1; i += kThreads) {
        const uint32_t at = (uint32_t)p.c.bias_ids[i] - first;
        if (at < size) one(at, load1(x, at, kDtype), p.c.bias_values[i]);
    }
    if (bad && p.status) atomicOr(p.status, bad);
}

template <bool kWide>
auto kernel_of(int dtype) {
    return dtype == NINFER_F32    ? logits_kernel<NINFER_F32, kWide>
           : dtype == NINFER_BF16 ? logits_kernel<NINFER_BF16, kWide>
                                  : logits_kernel<NINFER_F16, kWide>;
}

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_logits_process(const void *logits, uint64_t logits_stride, void *out, uint64_t out_stride, int dtype,
                                     uint64_t rows, uint64_t vocab, const ninfer_logits_controls *controls,
                                     int32_t *status, ninfer_stream stream) {
    if (!logits || !out || !controls) return fail(NINFER_ERR_INVALID_ARGUMENT, "logits: NULL logits, out or controls");
    const ninfer_logits_controls &c = *controls;
    if (!dtype_valid(dtype)) return fail(NINFER_ERR_INVALID_ARGUMENT, "logits: dtype %d unsupported", dtype);
    if (c.history && !c.history_lengths) return fail(NINFER_ERR_INVALID_ARGUMENT, "logits: history without history_lengths");
    if (!c.bias_offsets != !c.bias_ids || !c.bias_ids != !c.bias_values)
        return fail(NINFER_ERR_INVALID_ARGUMENT, "logits: bias_offsets, bias_ids and bias_values go together");
    if (!rows || !vocab || rows > 0x7fffffffull || vocab > 0x7fffffffull)
        return fail(NINFER_ERR_SHAPE, "logits: %llu rows of %llu", (unsigned long long)rows, (unsigned long long)vocab);
    if (rows > 1 && (logits_stride < vocab || out_stride < vocab))
        return fail(NINFER_ERR_SHAPE, "logits: row stride below vocab");
    if (logits == out && logits_stride != out_stride) return fail(NINFER_ERR_SHAPE, "logits: in place needs equal strides");
    if (c.mask && c.mask_stride < (vocab + 31) / 32 && c.mask_row_count > 1)
        return fail(NINFER_ERR_SHAPE, "logits: mask_stride below vocab / 32 words");
    if (c.mask && (!c.mask_row_count || (!c.mask_rows && c.mask_row_count < rows)))
        return fail(NINFER_ERR_SHAPE, "logits: %llu mask rows for %llu rows", (unsigned long long)c.mask_row_count,
                    (unsigned long long)rows);
    // what a table entry counts to; the kernel's 32-bit history indices pass it by less than 2^14
    if (c.history && c.history_stride > Entry<true>::kCount) return fail(NINFER_ERR_SHAPE, "logits: history_stride over 2^30 - 1");
    if (c.bias_ids && c.bias_count > 0x7fffffffull) return fail(NINFER_ERR_SHAPE, "logits: bias_count over 2^31 - 1");
    if (!aligned(logits, 16) || !aligned(out, 16)) return fail(NINFER_ERR_ALIGNMENT, "logits: logits and out must be 16-byte aligned");
    for (const void *a : {(const void *)c.history, (const void *)c.history_lengths, (const void *)c.prompt_lengths,
                          (const void *)c.repetition, (const void *)c.presence, (const void *)c.frequency,
                          (const void *)c.bias_offsets, (const void *)c.bias_ids, (const void *)c.bias_values,
                          (const void *)c.mask, (const void *)c.mask_rows, (const void *)status})
        if (!aligned(a, 4)) return fail(NINFER_ERR_ALIGNMENT, "logits: control buffers must be 4-byte aligned");
    DeviceInfo d;
    int st = device_info(&d);
    if (st) return st;
    const bool wide = c.history && c.history_stride > Entry<false>::kCount;
    // a slice: at most a table, at least kLeast tokens, and as many as fill the SMs once
    const uint64_t most = wide ? kMostWide : kMostNarrow, slots = (uint64_t)d.sms * kResident;
    uint64_t slices = slots / rows;
    slices = std::min(std::max(slices, (vocab + most - 1) / most), std::max((vocab + kLeast - 1) / kLeast, (vocab + most - 1) / most));
    LogitsParams p;
    p.slice = (uint32_t)std::min<uint64_t>(((vocab + slices - 1) / slices + 127) / 128 * 128, most);
    slices = (vocab + p.slice - 1) / p.slice;
    p.x = logits;
    p.out = out;
    p.x_stride = logits_stride;
    p.out_stride = out_stride;
    p.c = c;
    p.status = status;
    p.vocab = (uint32_t)vocab;
    p.slices = (uint32_t)slices;
    p.dtype = dtype;
    if (rows * slices > 0x7fffffffull) return fail(NINFER_ERR_OVERFLOW, "logits: rows * vocab too large");
    const auto kernel = wide ? kernel_of<true>(dtype) : kernel_of<false>(dtype);
    st = set_smem_attribute(reinterpret_cast<const void *>(kernel), kSmemBytes);
    if (st) return st;
    p.mask_at = p.slice * (wide ? 4 : 2) / 4;
    const size_t smem = p.mask_at * 4 + p.slice / 8;
    return launch_dependent("logits", kernel, dim3((unsigned)(rows * slices)), dim3(kThreads), smem, (cudaStream_t)stream, p);
}
