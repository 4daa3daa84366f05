// ninfer_logits_process: penalties for repeated tokens, biases and grammar masks
// on the logits of the output head.
//
// One pass over the logits (read once, written once): HBM bounds a batch,
// latency a single row. A CTA owns a slice of one row's tokens. It first
// enters the row's history into a table of counts in shared memory, one word a
// token of its slice (bit 31: seen at all, the rest: how often after the
// prompt), and the biases into a second table, then streams the slice through.
#include <cmath>

#include "decode.cuh"
#include "gemv.h"

namespace ninfer {
namespace {

constexpr uint32_t kSlice = 8192;       // tokens of a CTA: 64 KB of tables
constexpr int kThreads = 512;
constexpr uint32_t kSeen = 0x80000000u;

struct LogitsParams {
    const void *x;
    void *out;
    uint64_t x_stride, out_stride;
    ninfer_logits_controls c;
    int32_t *status;
    uint32_t vocab, slices;
    int dtype;
};

__global__ void __launch_bounds__(kThreads) logits_kernel(const LogitsParams p) {
    extern __shared__ __align__(16) uint32_t tables[];
    uint32_t *count = tables;
    float *bias = reinterpret_cast<float *>(tables + kSlice);
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t tid = threadIdx.x, row = blockIdx.x / p.slices;
    const uint32_t first = blockIdx.x % p.slices * kSlice, size = min(kSlice, p.vocab - first);
    for (uint32_t i = tid; i < kSlice; i += kThreads) {
        count[i] = 0;
        bias[i] = 0.f;
    }
    __syncthreads();
    int bad = 0;
    if (p.c.history) {
        const int64_t most = (int64_t)p.c.history_stride;
        const int64_t n = min((int64_t)max(p.c.history_lengths[row], 0), most);
        const int64_t told = p.c.prompt_lengths ? p.c.prompt_lengths[row] : 0;
        const int32_t *h = p.c.history + row * p.c.history_stride;
        for (int64_t i = tid; i < n; i += kThreads) {
            const uint32_t v = (uint32_t)h[i];
            if (v >= p.vocab) bad |= NINFER_LOGITS_BAD_TOKEN;
            if (v - first < size) {
                atomicOr(count + (v - first), kSeen);
                if (i >= told) atomicAdd(count + (v - first), 1u);
            }
        }
    }
    if (p.c.bias_ids) {
        const int64_t all = (int64_t)p.c.bias_count;
        const int64_t b0 = max((int64_t)p.c.bias_offsets[row], (int64_t)0), b1 = min((int64_t)p.c.bias_offsets[row + 1], all);
        for (int64_t i = b0 + tid; i < b1; i += kThreads) {
            const uint32_t v = (uint32_t)p.c.bias_ids[i];
            if (v >= p.vocab) bad |= NINFER_LOGITS_BAD_TOKEN;
            if (v - first < size) bias[v - first] = p.c.bias_values[i];
        }
    }
    __syncthreads();
    const float rep = p.c.repetition ? p.c.repetition[row] : 1.f, pres = p.c.presence ? p.c.presence[row] : 0.f;
    const float freq = p.c.frequency ? p.c.frequency[row] : 0.f;
    const uint32_t *mask = nullptr;
    if (p.c.mask) {
        const int64_t m = p.c.mask_rows ? (int64_t)p.c.mask_rows[row] : (int64_t)row;
        if (m >= (int64_t)p.c.mask_row_count) bad |= NINFER_LOGITS_BAD_TOKEN;
        else if (m >= 0) mask = p.c.mask + m * p.c.mask_stride;
    }
    for (uint32_t i = tid; i < size; i += kThreads) {
        float x = load1(p.x, row * p.x_stride + first + i, p.dtype);
        const uint32_t c = count[i];
        if (c) x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
        if (c & ~kSeen) x -= freq * (float)(c & ~kSeen) + pres;
        x += bias[i];
        const uint32_t v = first + i;
        if (mask && !(mask[v >> 5] >> (v & 31) & 1)) x = -INFINITY;
        store1(p.out, row * p.out_stride + v, p.dtype, x);
    }
    if (bad && p.status) atomicOr(p.status, bad);
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
    if (c.history && c.history_stride > 0x7fffffffull) return fail(NINFER_ERR_SHAPE, "logits: history_stride over 2^31 - 1");
    if (c.bias_ids && c.bias_count > 0x7fffffffull) return fail(NINFER_ERR_SHAPE, "logits: bias_count over 2^31 - 1");
    if (!aligned(logits, 16) || !aligned(out, 16)) return fail(NINFER_ERR_ALIGNMENT, "logits: logits and out must be 16-byte aligned");
    for (const void *a : {(const void *)c.history, (const void *)c.history_lengths, (const void *)c.prompt_lengths,
                          (const void *)c.repetition, (const void *)c.presence, (const void *)c.frequency,
                          (const void *)c.bias_offsets, (const void *)c.bias_ids, (const void *)c.bias_values,
                          (const void *)c.mask, (const void *)c.mask_rows, (const void *)status})
        if (!aligned(a, 4)) return fail(NINFER_ERR_ALIGNMENT, "logits: control buffers must be 4-byte aligned");
    LogitsParams p;
    p.x = logits;
    p.out = out;
    p.x_stride = logits_stride;
    p.out_stride = out_stride;
    p.c = c;
    p.status = status;
    p.vocab = (uint32_t)vocab;
    p.slices = (uint32_t)((vocab + kSlice - 1) / kSlice);
    p.dtype = dtype;
    if (rows * p.slices > 0x7fffffffull) return fail(NINFER_ERR_OVERFLOW, "logits: rows * vocab too large");
    constexpr int kBytes = kSlice * 8;
    const int st = ninfer::set_smem_attribute(reinterpret_cast<const void *>(logits_kernel), kBytes);
    if (st) return st;
    return launch_dependent("logits", logits_kernel, dim3((unsigned)(rows * p.slices)), dim3(kThreads), kBytes,
                            (cudaStream_t)stream, p);
}
