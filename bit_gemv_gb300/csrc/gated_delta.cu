// ninfer_gated_delta: the gated delta rule, S <- e^g S + beta k (v - e^g S^T k)^T,
// out = scale S^T q, over a k_dim x v_dim state of fp32 per request and value head.
//
// The columns of a state do not see each other: S^T k, u = beta (v - e^g S^T k), the update k u^T and S^T q need, for
// one column of S, only that column and the k and q that all columns share. Both kernels divide the states by columns.
// With a = S^T k and b = S^T q of the old state, out = scale (e^g b + (k . q) u): one pass over the state gives both sums,
// a second one, in registers, updates it.
//
// One token a request (step_kernel): the state is read once and written once, and HBM bounds it.
// Several (run_kernel): the state stays in registers from a request's first token to its last, four lanes a
// column; fp32 multiply-adds, 3 k_dim v_dim of them a token, bound it, and latency where few heads are under way.
#include <cmath>

#include "decode.cuh"
#include "gemv.h"
#include "ninfer_layer.h"

namespace ninfer {
namespace {

constexpr int kStepThreads = 256, kRunThreads = 128, kRunColumns = 32, kTile = 16;

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

// Any number of tokens a request. Four lanes hold a column: lane i of them the rows 16 j + 4 i .. 16 j + 4 i + 3, so that
// the four read 64 neighbouring bytes of k and q. kGroups: 16-row groups of k_dim, rounded up to 4, 8 or 16.
template <int kGroups>
__global__ void __launch_bounds__(kRunThreads) run_kernel(const __grid_constant__ DeltaParams p) {
    constexpr int kDim = kGroups * 16;
    __shared__ __align__(16) float ks[kTile][kDim], qs[kTile][kDim];
    __shared__ float vs[kTile][kRunColumns], numbers[3][kTile];     // e^g, beta, k . q
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_gated_delta_args &a = p.a;
    const Part t = part_of(p, blockIdx.x, kRunColumns);
    if (t.none) return;
    const int32_t most = (int32_t)a.tokens;
    const int32_t begin = a.offsets ? min(max(a.offsets[t.request], 0), most) : (int32_t)t.request;
    const int32_t end = a.offsets ? min(max(a.offsets[t.request + 1], 0), most) : begin + 1;
    if (begin >= end) return;
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32, k_dim = (uint32_t)a.k_dim, v_dim = (uint32_t)a.v_dim;
    const uint32_t mine = warp * 8 + lane / 4, column = t.column + mine, part = lane % 4 * 4;
    const bool inside = column < v_dim;
    float *state = a.state + t.state + column;
    float s[kGroups][4];
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = j * 16 + part + i;
            s[j][i] = r < k_dim && inside && !t.fresh ? state[r * v_dim] : 0.f;
        }
    for (int32_t t0 = begin; t0 < end; t0 += kTile) {
        const int32_t count = min(end - t0, kTile);
        __syncthreads();
        // a warp a token: its k and q, normalised; its numbers and values
        for (int32_t i = warp; i < count; i += kRunThreads / 32) {
            const uint64_t token = t0 + i;
            float k[8] = {}, q[8] = {}, kk = 0.f, qq = 0.f, kq = 0.f;
            if (lane * 8 < k_dim) {
                load8(a.k, token * a.k_token_stride + t.key_head * a.k_head_stride + lane * 8, a.dtype, k);
                load8(a.q, token * a.q_token_stride + t.key_head * a.q_head_stride + lane * 8, a.dtype, q);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kk = fmaf(k[e], k[e], kk);
                qq = fmaf(q[e], q[e], qq);
                kq = fmaf(k[e], q[e], kq);
            }
#pragma unroll
            for (int e = 16; e; e /= 2) {
                kk += __shfl_xor_sync(~0u, kk, e);
                qq += __shfl_xor_sync(~0u, qq, e);
                kq += __shfl_xor_sync(~0u, kq, e);
            }
            const float k_scale = a.norm_eps < 0.f ? 1.f : 1.f / sqrtf(kk + a.norm_eps);
            const float q_scale = a.norm_eps < 0.f ? 1.f : 1.f / sqrtf(qq + a.norm_eps);
            if (lane * 8 < kDim) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ks[i][lane * 8 + e] = k[e] * k_scale;
                    qs[i][lane * 8 + e] = q[e] * q_scale;
                }
            }
            vs[i][lane] = t.column + lane < v_dim ? load1(a.v, token * a.v_token_stride + t.head * a.v_head_stride + t.column + lane, a.dtype) : 0.f;
            if (lane == 0) {
                numbers[0][i] = expf(a.log_decay[token * a.decay_stride + t.head]);
                numbers[1][i] = a.beta[token * a.beta_stride + t.head];
                numbers[2][i] = kq * k_scale * q_scale;
            }
        }
        __syncthreads();
        for (int32_t i = 0; i < count; ++i) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const float4 k = *reinterpret_cast<const float4 *>(&ks[i][j * 16 + part]), q = *reinterpret_cast<const float4 *>(&qs[i][j * 16 + part]);
                x = fmaf(s[j][0], k.x, x);
                x = fmaf(s[j][1], k.y, x);
                x = fmaf(s[j][2], k.z, x);
                x = fmaf(s[j][3], k.w, x);
                y = fmaf(s[j][0], q.x, y);
                y = fmaf(s[j][1], q.y, y);
                y = fmaf(s[j][2], q.z, y);
                y = fmaf(s[j][3], q.w, y);
            }
            x += __shfl_xor_sync(~0u, x, 1);
            y += __shfl_xor_sync(~0u, y, 1);
            x += __shfl_xor_sync(~0u, x, 2);
            y += __shfl_xor_sync(~0u, y, 2);
            const float decay = numbers[0][i], u = numbers[1][i] * (vs[i][mine] - decay * x);
            if (lane % 4 == 0 && inside)
                store1(a.out, ((uint64_t)(t0 + i) * a.v_heads + t.head) * v_dim + column, a.out_dtype, a.scale * (decay * y + numbers[2][i] * u));
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const float4 k = *reinterpret_cast<const float4 *>(&ks[i][j * 16 + part]);
                s[j][0] = fmaf(k.x, u, decay * s[j][0]);
                s[j][1] = fmaf(k.y, u, decay * s[j][1]);
                s[j][2] = fmaf(k.z, u, decay * s[j][2]);
                s[j][3] = fmaf(k.w, u, decay * s[j][3]);
            }
        }
    }
    if (!inside) return;
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = j * 16 + part + i;
            if (r < k_dim) state[r * v_dim] = s[j][i];
        }
}

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
    *bytes = 0;
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
    uint64_t need;
    st = ninfer_gated_delta_workspace(a.tokens, a.requests, a.k_heads, a.v_heads, a.k_dim, a.v_dim, &need);
    if (st) return st;
    if (need && !workspace) return fail(NINFER_ERR_INVALID_ARGUMENT, "gated delta: NULL workspace");
    if (workspace_bytes < need) return fail(NINFER_ERR_SIZE_MISMATCH, "gated delta: workspace of %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                                            (unsigned long long)need);
    if (need && !aligned(workspace, 256)) return fail(NINFER_ERR_ALIGNMENT, "gated delta: workspace must be 256-byte aligned");
    DeltaParams p;
    p.a = a;
    p.heads = FastDiv((uint32_t)a.v_heads);
    p.group = FastDiv((uint32_t)(a.v_heads / a.k_heads));
    const uint64_t rows = a.requests * a.v_heads;
    const auto grid = [&](uint64_t slab, unsigned *blocks) {
        const uint64_t slabs = (a.v_dim + slab - 1) / slab;
        p.slabs = FastDiv((uint32_t)slabs);
        *blocks = (unsigned)(rows * slabs);
        return rows * slabs <= 0x7fffffffull;
    };
    unsigned blocks;
    const cudaStream_t s = (cudaStream_t)stream;
    if (!a.offsets) {
        // whole rows of a state where there are enough of them for the SMs, else narrow slabs
        DeviceInfo d;
        st = device_info(&d);
        if (st) return st;
        const bool narrow = rows * ((a.v_dim + 127) / 128) < 2ull * d.sms;
        const int lanes = narrow || a.v_dim <= 32 ? 8 : a.k_dim > 128 || a.v_dim <= 64 ? 16 : 32;
        if (!grid(lanes * 4, &blocks)) return fail(NINFER_ERR_OVERFLOW, "gated delta: too many requests and heads");
        const bool small = a.k_dim <= (uint64_t)(8 * kStepThreads / lanes);
        const auto kernel = lanes == 8    ? step_kernel<8, 8>
                            : lanes == 16 ? (small ? step_kernel<16, 8> : step_kernel<16, 16>)
                                          : (small ? step_kernel<32, 8> : step_kernel<32, 16>);
        return launch_dependent("gated delta", kernel, dim3(blocks), dim3(kStepThreads), 0, s, p);
    }
    if (!grid(kRunColumns, &blocks)) return fail(NINFER_ERR_OVERFLOW, "gated delta: too many requests and heads");
    const auto kernel = a.k_dim <= 64 ? run_kernel<4> : a.k_dim <= 128 ? run_kernel<8> : run_kernel<16>;
    return launch_dependent("gated delta", kernel, dim3(blocks), dim3(kRunThreads), 0, s, p);
}
