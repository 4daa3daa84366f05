// ninfer_rotary: rotary positions of queries and keys, with their heads' norms
// before it; ninfer_rotary_frequencies: the table of frequencies (host).
//
// Queries and keys are read once and written once: HBM bounds a prompt, latency a decode step. An angle is
// a whole number of 2^-64 turns: position times frequency modulo 2^64 is exact in integers, and what
// remains of it, as a signed fraction, goes through sincospif, so that position 2^31 is as exact as position 1
// without 64-bit floats. The sines and cosines of a token serve all of its heads: a CTA takes one
// token, asks for its first heads, puts the sines and cosines into shared memory and then turns its heads,
// a few lanes each, 8 elements a lane, with as many threads as take them in the fewest rounds.
//
// Measured: 30011 tokens of 40 heads of 128 in bfloat16, neighbouring pairs, 615 MB, 102 us (6.0 TB/s). Heads asked for only after the sines and
// cosines: 140; 256 threads for every token: 125; 64 registers a thread instead of 48: 109. Halves, whose partners are eight shuffles of a lane
// away, 168 us, with norms (a weight, a root and a quotient a head) 209; 28 heads of 256 with 64 elements turned, halves, 861 MB, 161 and with norms 214.
#include <cmath>

#include "decode.cuh"
#include "gemv.h"
#include "ninfer_layer.h"
#include "overlap.h"

namespace ninfer {
namespace {

constexpr int kThreads = 256;

struct RotaryParams {
    ninfer_rotary_args a;
    uint32_t heads, q_heads, half;      // heads: q_heads + kv_heads; half: rotary_dim / 2
    float inverse;              // 1 / head_dim
};

// Heads of a team under way at once.
__host__ __device__ constexpr uint32_t ahead_of(int dtype) { return dtype == NINFER_F32 ? 2 : 4; }

// kLanes: lanes of a head, 8 elements each. kPairs: 0 neighbours; 1 halves whose distance is a multiple of 8 (partners in another
// lane, the same place); 2 other halves (the head goes through shared memory).
template <int kDtype, int kLanes, int kPairs>
__global__ void __launch_bounds__(kThreads, 5) rotary_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ __align__(16) float2 turn[128];
    __shared__ float row[kPairs == 2 ? kThreads / kLanes : 1][kPairs == 2 ? kLanes * 8 : 1];
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_rotary_args &a = p.a;
    const uint32_t token = blockIdx.x, tid = threadIdx.x;
    const int32_t position = a.positions[token];
    if (position < 0) return;
    const uint32_t lane = tid % kLanes, team = tid / kLanes, e = lane * 8;
    const bool inside = e < a.head_dim;
    // a few heads of each team asked for at once, the first ones before the sines and cosines
    constexpr uint32_t kAhead = ahead_of(kDtype);
    const uint32_t teams = blockDim.x / kLanes;
    Raw8 raw[kAhead];
    const uint64_t q_in = token * a.q_token_stride + e, k_in = token * a.k_token_stride + e;
    const uint64_t q_to = token * a.q_out_token_stride + e, k_to = token * a.k_out_token_stride + e;
    auto fetch = [&](uint32_t h0) {
#pragma unroll
        for (uint32_t j = 0; j < kAhead; ++j) {
            const uint32_t h = h0 + j * teams + team;
            const bool key = h >= p.q_heads;
            const uint32_t head = key ? h - p.q_heads : h;
            if (inside && h < p.heads) raw[j] = raw8(key ? a.k : a.q, (key ? k_in : q_in) + head * (key ? a.k_head_stride : a.q_head_stride), kDtype);
        }
    };
    fetch(0);
    for (uint32_t i = tid; i < p.half; i += blockDim.x) {
        const int64_t part = (int64_t)((uint64_t)position * a.frequencies[i]);
        float s, c;
        sincospif(__ll2float_rn(part) * 0x1p-63f, &s, &c);
        turn[i] = make_float2(c * a.magnitude, s * a.magnitude);
    }
    __syncthreads();
    for (uint32_t h0 = 0; h0 < p.heads; h0 += kAhead * teams) {
      if (h0) fetch(h0);
#pragma unroll
      for (uint32_t j = 0; j < kAhead; ++j) {
        const uint32_t h = h0 + j * teams + team;
        if (h - team >= p.heads) break;
        const bool on = inside && h < p.heads, key = h >= p.q_heads;
        const uint32_t head = key ? h - p.q_heads : h;
        float x[8] = {};
        if (on) widen(raw[j], kDtype, x);
        const void *weight = key ? a.k_weight : a.q_weight;
        if (a.q_weight || a.k_weight) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int k = kLanes / 2; k; k /= 2) sum += __shfl_xor_sync(~0u, sum, k);
            if (weight && on) {
                const float scale = 1.f / sqrtf(fmaf(sum, p.inverse, a.eps));
                float w[8];
                load8(weight, e, a.weight_dtype, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * scale * (w[i] + a.weight_offset);
            }
        }
        if (kPairs == 0) {
            if (e + 8 <= a.rotary_dim) {
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(&turn[(e + i) / 2]);
                    const float u = x[i], v = x[i + 1], w = x[i + 2], y = x[i + 3];
                    x[i] = u * t.x - v * t.y;
                    x[i + 1] = v * t.x + u * t.y;
                    x[i + 2] = w * t.z - y * t.w;
                    x[i + 3] = y * t.z + w * t.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    if (e + i >= a.rotary_dim) break;
                    const float2 t = turn[(e + i) / 2];
                    const float u = x[i], v = x[i + 1];
                    x[i] = u * t.x - v * t.y;
                    x[i + 1] = v * t.x + u * t.y;
                }
            }
        } else if (kPairs == 1) {
            const uint32_t apart = p.half / 8;
            const bool low = e < p.half, turned = e < a.rotary_dim;
            const uint32_t from = !turned ? lane : low ? lane + apart : lane - apart;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(~0u, x[i], from, kLanes);
            if (turned) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 t = *reinterpret_cast<const float4 *>(&turn[(low ? e : e - p.half) + i]);
                    x[i] = fmaf(x[i], t.x, low ? -y[i] * t.y : y[i] * t.y);
                    x[i + 1] = fmaf(x[i + 1], t.z, low ? -y[i + 1] * t.w : y[i + 1] * t.w);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) row[team][e + i] = x[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (e + i >= a.rotary_dim) break;
                const bool low = e + i < p.half;
                const float2 t = turn[low ? e + i : e + i - p.half];
                const float y = row[team][low ? e + i + p.half : e + i - p.half];
                x[i] = low ? x[i] * t.x - y * t.y : x[i] * t.x + y * t.y;
            }
            __syncwarp();
        }
        if (on)
            store8(key ? a.k_out : a.q_out, (key ? k_to : q_to) + head * (key ? a.k_out_head_stride : a.q_out_head_stride), kDtype, x);
      }
    }
}

template <int kDtype, int kLanes>
auto kernel_of(int pairs) {
    return pairs == 0 ? rotary_kernel<kDtype, kLanes, 0> : pairs == 1 ? rotary_kernel<kDtype, kLanes, 1> : rotary_kernel<kDtype, kLanes, 2>;
}

template <int kDtype>
auto kernel_of(unsigned lanes, int pairs) {
    return lanes == 8 ? kernel_of<kDtype, 8>(pairs) : lanes == 16 ? kernel_of<kDtype, 16>(pairs) : kernel_of<kDtype, 32>(pairs);
}

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_rotary_frequencies(uint64_t rotary_dim, double base, int scaling, double factor, double context,
                                         double slow, double fast, uint64_t *frequencies, float *magnitude) {
    if (!frequencies || !magnitude) return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary frequencies: NULL frequencies or magnitude");
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 256)
        return fail(NINFER_ERR_SHAPE, "rotary frequencies: rotary_dim %llu is not even and 2 to 256", (unsigned long long)rotary_dim);
    const bool parts = scaling == NINFER_ROTARY_DIMENSIONS || scaling == NINFER_ROTARY_TURNS;
    if (!parts && scaling != NINFER_ROTARY_NONE && scaling != NINFER_ROTARY_LINEAR)
        return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary frequencies: scaling %d unknown", scaling);
    if (!(base > 1) || !std::isfinite(base) || (scaling != NINFER_ROTARY_NONE && (!(factor >= 1) || !std::isfinite(factor))))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary frequencies: base must be over 1, factor 1 or more");
    if (parts && (!(context > 0) || !std::isfinite(context) || !(slow > 0) || !(fast > slow) || !std::isfinite(fast)))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary frequencies: context must be positive, 0 < slow < fast");
    const double turn = 6.283185307179586476925286766559, dim = (double)rotary_dim;
    double first = 0, last = 1;
    if (scaling == NINFER_ROTARY_DIMENSIONS) {
        // the pair that turns n times within the context: context base^(-2 i / dim) / 2 pi = n
        const auto pair = [&](double n) { return dim * std::log(context / (n * turn)) / (2 * std::log(base)); };
        first = std::max(std::floor(pair(fast)), 0.0);
        last = std::min(std::ceil(pair(slow)), dim - 1);
    }
    for (uint64_t i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / dim);
        double ramp = scaling == NINFER_ROTARY_NONE ? 0 : 1;
        if (scaling == NINFER_ROTARY_DIMENSIONS) ramp = ((double)i - first) / std::max(last - first, 0.001);
        if (scaling == NINFER_ROTARY_TURNS) ramp = 1 - (context * f / turn - slow) / (fast - slow);
        ramp = std::min(std::max(ramp, 0.0), 1.0);
        // f / 2 pi < 1 / 6, so that 2^64 of it fit
        const double turns = (ramp == 0 ? f : f / factor * ramp + f * (1 - ramp)) / turn;
        frequencies[i] = (uint64_t)(turns * 0x1p64);
    }
    *magnitude = scaling == NINFER_ROTARY_DIMENSIONS ? (float)(0.1 * std::log(factor) + 1) : 1.f;
    return NINFER_OK;
}

extern "C" int ninfer_rotary(const ninfer_rotary_args *args, ninfer_stream stream) {
    if (!args || !args->q || !args->q_out || !args->positions || !args->frequencies)
        return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary: NULL args, q, q_out, positions or frequencies");
    const ninfer_rotary_args &a = *args;
    if (!a.k != !a.k_out) return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary: k and k_out go together");
    if (!dtype_valid(a.dtype) || ((a.q_weight || a.k_weight) && !dtype_valid(a.weight_dtype)))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary: dtype %d or weight dtype %d unsupported", a.dtype, a.weight_dtype);
    if (!std::isfinite(a.magnitude) || !std::isfinite(a.weight_offset) || !(a.eps >= 0.f) || !std::isfinite(a.eps))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary: magnitude and weight_offset must be finite, eps finite and 0 or more");
    if (!a.tokens || a.tokens > 0x7fffffffull || !a.q_heads || a.q_heads > 65535 || (a.k && (!a.kv_heads || a.kv_heads > 65535)))
        return fail(NINFER_ERR_SHAPE, "rotary: %llu tokens of %llu and %llu heads", (unsigned long long)a.tokens,
                    (unsigned long long)a.q_heads, (unsigned long long)a.kv_heads);
    if (!a.head_dim || a.head_dim % 8 || a.head_dim > 256 || a.rotary_dim < 2 || a.rotary_dim % 2 || a.rotary_dim > a.head_dim)
        return fail(NINFER_ERR_SHAPE, "rotary: head_dim %llu must be a multiple of 8 up to 256, rotary_dim %llu even and 2 to it",
                    (unsigned long long)a.head_dim, (unsigned long long)a.rotary_dim);
    const uint64_t es = dtype_size(a.dtype), unit = 16 / es;
    const struct {
        const void *p;
        uint64_t token, head, heads;
    } tensors[] = {{a.q, a.q_token_stride, a.q_head_stride, a.q_heads},
                   {a.q_out, a.q_out_token_stride, a.q_out_head_stride, a.q_heads},
                   {a.k, a.k_token_stride, a.k_head_stride, a.kv_heads},
                   {a.k_out, a.k_out_token_stride, a.k_out_head_stride, a.kv_heads}};
    for (const auto &t : tensors) {
        if (!t.p) continue;
        const uint64_t token = a.tokens > 1 ? t.token : 0, head = t.heads > 1 ? t.head : 0;
        if (!aligned(t.p, 16) || token % unit || head % unit)
            return fail(NINFER_ERR_ALIGNMENT, "rotary: q, k and their outputs must have bases and strides of 16 bytes' multiples");
        if (token >= (1ull << 40) || head >= (1ull << 40)) return fail(NINFER_ERR_OVERFLOW, "rotary: a stride of 2^40 or more");
    }
    if (!aligned(a.positions, 4) || !aligned(a.frequencies, 8) || !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16))
        return fail(NINFER_ERR_ALIGNMENT, "rotary: positions must be 4-byte, frequencies 8-byte, weights 16-byte aligned");
    const auto span = [&](const void *p, uint64_t token, uint64_t heads, uint64_t head) { return p ? Span(p, a.head_dim * es, a.tokens, token * es, heads, head * es) : Span(); };
    const Span q = span(a.q, a.q_token_stride, a.q_heads, a.q_head_stride), q_out = span(a.q_out, a.q_out_token_stride, a.q_heads, a.q_out_head_stride);
    const Span k = span(a.k, a.k_token_stride, a.kv_heads, a.k_head_stride), k_out = span(a.k_out, a.k_out_token_stride, a.kv_heads, a.k_out_head_stride);
    const bool q_here = q_out.same(q), k_here = k_out.same(k);
    bool shared = (!q_here && q_out.meets(q)) || (!k_here && k_out.meets(k)) || !q_out.simple() || !k_out.simple() || q_out.meets(k_out) ||
                  (!k_here && q_out.meets(k)) || (!q_here && k_out.meets(q));
    const uint64_t weight_bytes = a.q_weight || a.k_weight ? a.head_dim * dtype_size(a.weight_dtype) : 0;
    for (const Span &in : {Span(a.positions, a.tokens * 4), Span(a.frequencies, a.rotary_dim * 4), Span(a.q_weight, weight_bytes), Span(a.k_weight, weight_bytes)})
        shared = shared || q_out.meets(in) || k_out.meets(in);
    if (shared) return fail(NINFER_ERR_INVALID_ARGUMENT, "rotary: an output may be its own input with the same strides, and overlaps nothing else");
    RotaryParams p;
    p.a = a;
    p.half = (uint32_t)(a.rotary_dim / 2);
    p.q_heads = (uint32_t)a.q_heads;
    p.heads = (uint32_t)(a.q_heads + (a.k ? a.kv_heads : 0));
    p.inverse = 1.f / (float)a.head_dim;
    const unsigned lanes = a.head_dim <= 64 ? 8 : a.head_dim <= 128 ? 16 : 32;
    const int pairs = a.interleaved ? 0 : p.half % 8 == 0 ? 1 : 2;
    const auto kernel = a.dtype == NINFER_F32    ? kernel_of<NINFER_F32>(lanes, pairs)
                        : a.dtype == NINFER_BF16 ? kernel_of<NINFER_BF16>(lanes, pairs)
                                                 : kernel_of<NINFER_F16>(lanes, pairs);
    // as many teams as take the heads in the fewest rounds
    const unsigned ahead = ahead_of(a.dtype), rounds = (p.heads * lanes + ahead * kThreads - 1) / (ahead * kThreads);
    const unsigned teams = (p.heads + ahead * rounds - 1) / (ahead * rounds), threads = (teams * lanes + 31) / 32 * 32;
    return launch_dependent("rotary", kernel, dim3((unsigned)a.tokens), dim3(threads), 0, (cudaStream_t)stream, p);
}
