// ninfer_norm: root-mean-square norm of groups of a row, with the residual's
// addition before it and a gate behind it.
//
// Each element is read once and written once, so HBM bounds a prompt and latency a single row. A group's
// values stay in the registers of the threads that read them between the sum of squares and the product:
// of a few lanes for the heads of a row (norm_team_kernel), of a CTA for a hidden state (norm_row_kernel). Only groups of more
// than 32768 elements are read twice (norm_long_kernel).
//
// Measured: 8192 rows of 5120 with a residual, all bfloat16, 336 MB, 49.2 to 50.0 us (6.7 to 6.8 TB/s, the rate of a copy); 4001 rows of 48
// heads of 128 with gates, 147 MB, 26.3 us (5.6 TB/s, at 73 % of the issue slots). Reciprocal square roots, powers and reciprocals
// are the fast ones, within 4 2^-24: with the exact ones' sequences 55 and 39 us. (A gate's exponent in one float, 2^-24 z off, 25.2.)
// Rows off 16-byte boundaries go an element at a time (8192 of 5119 with a residual 224 us), groups over 32768 by one CTA twice (512 of 40000
// 55 us, 1.5 TB/s; one of 262144 118).
#include <cmath>

#include "decode.cuh"
#include "gemv.h"
#include "ninfer_layer.h"
#include "overlap.h"

namespace ninfer {
namespace {

constexpr int kTeamThreads = 256;
constexpr uint32_t kMostTeam = 256, kMostRow = 32768;   // elements of a group: 8 a lane, 32 a thread

struct NormParams {
    ninfer_norm_args a;
    FastDiv groups;         // of a row
    uint32_t total;         // groups in all
    float inverse;          // 1 / group
};

// y z / (1 + e^-z) as y z E / (1 + E) with E = e^z (from 44 on the quotient is 1): no sum overflows, and nothing is lost down to the least number.
// E = 2^2t e^d with t = z log2(e) / 2 rounded, whose power is a normal number, and d = z - 2 t ln 2 what that left out; within 14 2^-24
// (2^t 4, twice; ln 2's own rounding 5 at z = -104; the sum 1).
__device__ __forceinline__ float gated(float y, float z) {
    const float a = fminf(z, 44.f), t = a * 0.72134752f;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e *= e;
    e = fmaf(e, fmaf(t, -1.38629436f, a), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return e * r * (y * z);
}

// Where element `at` of group `group` lies in the row's tensors.
struct Place {
    uint64_t row;
    uint32_t first;     // of the group within its row
};

__device__ __forceinline__ Place place_of(const NormParams &p, uint32_t index) {
    const uint32_t row = p.groups.div(index);
    return {row, (index - row * p.groups.d) * (uint32_t)p.a.group};
}

// A group to a team of kLanes lanes, 8 elements a lane. kType: the type of x, gate and out where they have one and the weight is
// float (or there is none), and there is no residual; -1 for all else. (A lane has few elements, so that the branches on four types and the
// addresses are a third of the instructions that bound this kernel: the gated heads above 26 us, with a weight of 16 bits 32.)
template <int kLanes, int kType>
__global__ void __launch_bounds__(kTeamThreads) norm_team_kernel(const __grid_constant__ NormParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_norm_args &a = p.a;
    constexpr bool kOne = kType >= 0;
    const int x_dtype = kOne ? kType : a.x_dtype, gate_dtype = kOne ? kType : a.gate_dtype, out_dtype = kOne ? kType : a.out_dtype;
    const int weight_dtype = kOne ? (int)NINFER_F32 : a.weight_dtype;
    const uint32_t index = blockIdx.x * (kTeamThreads / kLanes) + threadIdx.x / kLanes, e = threadIdx.x % kLanes * 8;
    const bool on = index < p.total && e < a.group;
    const Place at = place_of(p, on ? index : 0);
    const uint64_t col = at.first + e;
    Raw8 x, r, z, w;
    if (on) {
        x = raw8(a.x, at.row * a.x_stride + col, x_dtype);
        if (!kOne && a.residual) r = raw8(a.residual, at.row * a.residual_stride + col, a.residual_dtype);
        if (a.gate) z = raw8(a.gate, at.row * a.gate_stride + col, gate_dtype);
        if (a.weight) w = raw8(a.weight, e, weight_dtype);
    }
    float s[8] = {}, t[8], sum = 0.f;
    if (on) {
        widen(x, x_dtype, s);
        if (!kOne && a.residual) {
            widen(r, a.residual_dtype, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += t[i];
            if (a.sum) store8(a.sum, at.row * a.sum_stride + col, a.residual_dtype, s);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(s[i], s[i], sum);
#pragma unroll
    for (int k = kLanes / 2; k; k /= 2) sum += __shfl_xor_sync(~0u, sum, k);
    if (!on) return;
    const float scale = rsqrtf(fmaf(sum, p.inverse, a.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= scale;
    if (a.weight) {
        widen(w, weight_dtype, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] *= t[i] + a.weight_offset;
    }
    if (a.gate) {
        widen(z, gate_dtype, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = gated(s[i], t[i]);
    }
    store8(a.out, at.row * a.out_stride + col, out_dtype, s);
}

template <int kLanes>
auto team_kernel_of(int type) {
    return type == NINFER_BF16 ? norm_team_kernel<kLanes, NINFER_BF16> : type == NINFER_F16 ? norm_team_kernel<kLanes, NINFER_F16> : norm_team_kernel<kLanes, -1>;
}

// The CTA's sum; every thread gets it, the same bits.
__device__ __forceinline__ float sum_of_all(float v) {
    __shared__ float part[32];
#pragma unroll
    for (int k = 16; k; k /= 2) v += __shfl_xor_sync(~0u, v, k);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = threadIdx.x % 32 < blockDim.x / 32 ? part[threadIdx.x % 32] : 0.f;
#pragma unroll
    for (int k = 16; k; k /= 2) v += __shfl_xor_sync(~0u, v, k);
    return v;
}

// A group to a CTA, kPer times 8 elements a thread: neighbouring ones in vectors, or (rows off 16-byte boundaries,
// groups of no multiple of 8) one by one.
template <int kPer, bool kVec>
__global__ void __launch_bounds__(1024) norm_row_kernel(const __grid_constant__ NormParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_norm_args &a = p.a;
    const Place at = place_of(p, blockIdx.x);
    const uint32_t group = (uint32_t)a.group, threads = blockDim.x, tid = threadIdx.x;
    const uint64_t x_at = at.row * a.x_stride + at.first, r_at = at.row * a.residual_stride + at.first;
    const uint64_t z_at = at.row * a.gate_stride + at.first, sum_at = at.row * a.sum_stride + at.first;
    const uint64_t out_at = at.row * a.out_stride + at.first;
    float s[kPer][8], sum = 0.f;
    if (kVec) {
        Raw8 x[kPer], r[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t e = (tid + j * threads) * 8;
            if (e >= group) continue;
            x[j] = raw8(a.x, x_at + e, a.x_dtype);
            if (a.residual) r[j] = raw8(a.residual, r_at + e, a.residual_dtype);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t e = (tid + j * threads) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] = 0.f;
            if (e >= group) continue;
            widen(x[j], a.x_dtype, s[j]);
            if (a.residual) {
                float t[8];
                widen(r[j], a.residual_dtype, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[j][i] += t[i];
                if (a.sum) store8(a.sum, sum_at + e, a.residual_dtype, s[j]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t e = tid + (j * 8 + i) * threads;
                s[j][i] = 0.f;
                if (e >= group) continue;
                s[j][i] = load1(a.x, x_at + e, a.x_dtype);
                if (a.residual) {
                    s[j][i] += load1(a.residual, r_at + e, a.residual_dtype);
                    if (a.sum) store1(a.sum, sum_at + e, a.residual_dtype, s[j][i]);
                }
            }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(s[j][i], s[j][i], sum);
    const float scale = rsqrtf(fmaf(sum_of_all(sum), p.inverse, a.eps));
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (kVec) {
            const uint32_t e = (tid + j * threads) * 8;
            if (e >= group) break;
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j][i] *= scale;
            if (a.weight) {
                widen(raw8(a.weight, e, a.weight_dtype), a.weight_dtype, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[j][i] *= t[i] + a.weight_offset;
            }
            if (a.gate) {
                widen(raw8(a.gate, z_at + e, a.gate_dtype), a.gate_dtype, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[j][i] = gated(s[j][i], t[i]);
            }
            store8(a.out, out_at + e, a.out_dtype, s[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t e = tid + (j * 8 + i) * threads;
                if (e >= group) break;
                float y = s[j][i] * scale;
                if (a.weight) y *= load1(a.weight, e, a.weight_dtype) + a.weight_offset;
                if (a.gate) y = gated(y, load1(a.gate, z_at + e, a.gate_dtype));
                store1(a.out, out_at + e, a.out_dtype, y);
            }
        }
    }
}

// A group of any size to a CTA, read twice; an element's outputs are written by the thread that reads it last.
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const ninfer_norm_args &a = p.a;
    const Place at = place_of(p, blockIdx.x);
    const uint64_t x_at = at.row * a.x_stride + at.first, r_at = at.row * a.residual_stride + at.first;
    auto value = [&](uint64_t e) {
        float s = load1(a.x, x_at + e, a.x_dtype);
        if (a.residual) s += load1(a.residual, r_at + e, a.residual_dtype);
        return s;
    };
    float sum = 0.f;
    for (uint64_t e = threadIdx.x; e < a.group; e += 1024) {
        const float s = value(e);
        sum = fmaf(s, s, sum);
    }
    const float scale = rsqrtf(fmaf(sum_of_all(sum), p.inverse, a.eps));
    for (uint64_t e = threadIdx.x; e < a.group; e += 1024) {
        const float s = value(e);
        float y = s * scale;
        if (a.weight) y *= load1(a.weight, e, a.weight_dtype) + a.weight_offset;
        if (a.gate) y = gated(y, load1(a.gate, at.row * a.gate_stride + at.first + e, a.gate_dtype));
        if (a.sum) store1(a.sum, at.row * a.sum_stride + at.first + e, a.residual_dtype, s);
        store1(a.out, at.row * a.out_stride + at.first + e, a.out_dtype, y);
    }
}

}  // namespace
}  // namespace ninfer

using namespace ninfer;

extern "C" int ninfer_norm(const ninfer_norm_args *args, ninfer_stream stream) {
    if (!args || !args->x || !args->out) return fail(NINFER_ERR_INVALID_ARGUMENT, "norm: NULL args, x or out");
    const ninfer_norm_args &a = *args;
    if (a.sum && !a.residual) return fail(NINFER_ERR_INVALID_ARGUMENT, "norm: sum without a residual");
    if (a.reserved) return fail(NINFER_ERR_INVALID_ARGUMENT, "norm: reserved must be 0");
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps) || !std::isfinite(a.weight_offset))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "norm: eps must be finite and 0 or more, weight_offset finite");
    if (!a.rows || !a.cols || !a.group || a.cols % a.group || a.cols > 0x7fffffffull)
        return fail(NINFER_ERR_SHAPE, "norm: %llu rows of %llu in groups of %llu", (unsigned long long)a.rows,
                    (unsigned long long)a.cols, (unsigned long long)a.group);
    const struct {
        const void *p;
        uint64_t stride;
        int dtype;
        const char *name;
    } tensors[] = {{a.x, a.x_stride, a.x_dtype, "x"},
                   {a.residual, a.residual_stride, a.residual_dtype, "residual"},
                   {a.sum, a.sum_stride, a.residual_dtype, "sum"},
                   {a.gate, a.gate_stride, a.gate_dtype, "gate"},
                   {a.out, a.out_stride, a.out_dtype, "out"},
                   {a.weight, a.cols, a.weight_dtype, "weight"}};
    bool vec = a.group % 8 == 0;
    for (const auto &t : tensors) {
        if (!t.p) continue;
        if (!dtype_valid(t.dtype)) return fail(NINFER_ERR_INVALID_ARGUMENT, "norm: %s dtype %d unsupported", t.name, t.dtype);
        const size_t es = dtype_size(t.dtype);
        if (!aligned(t.p, es)) return fail(NINFER_ERR_ALIGNMENT, "norm: %s is not aligned to its elements", t.name);
        if (a.rows > 1 && t.stride < a.cols) return fail(NINFER_ERR_SHAPE, "norm: %s stride below cols", t.name);
        if (a.rows > 1 && t.stride >= (1ull << 40)) return fail(NINFER_ERR_OVERFLOW, "norm: %s stride of 2^40 or more", t.name);
        vec = vec && aligned(t.p, 16) && (a.rows == 1 || t.p == a.weight || t.stride * es % 16 == 0);
    }
    const uint64_t groups = a.cols / a.group;
    uint64_t total;
    if (!mul_ok(a.rows, groups, &total) || total > 0x7fffffffull)
        return fail(NINFER_ERR_OVERFLOW, "norm: rows * groups over 2^31 - 1");
    // in place only where every element is written where it was read
    const auto span = [&](const void *p, uint64_t stride, int dtype) { return Span(p, a.cols * dtype_size(dtype), a.rows, stride * dtype_size(dtype)); };
    const Span x = span(a.x, a.x_stride, a.x_dtype), gate = a.gate ? span(a.gate, a.gate_stride, a.gate_dtype) : Span(), out = span(a.out, a.out_stride, a.out_dtype);
    const Span residual = a.residual ? span(a.residual, a.residual_stride, a.residual_dtype) : Span(), sum = a.sum ? span(a.sum, a.sum_stride, a.residual_dtype) : Span();
    const Span weight = a.weight ? Span(a.weight, a.group * dtype_size(a.weight_dtype)) : Span();
    if ((out.meets(x) && !(out.same(x) && a.out_dtype == a.x_dtype)) || (out.meets(gate) && !(out.same(gate) && a.out_dtype == a.gate_dtype)) ||
        (sum.meets(residual) && !sum.same(residual)) || out.meets(residual) || out.meets(sum) || out.meets(weight) || sum.meets(x) || sum.meets(gate) || sum.meets(weight))
        return fail(NINFER_ERR_INVALID_ARGUMENT, "norm: out may be x or gate, sum the residual, with the same stride and dtype; no other outputs overlap");
    NormParams p;
    p.a = a;
    p.groups = FastDiv((uint32_t)groups);
    p.total = (uint32_t)total;
    p.inverse = 1.f / (float)a.group;
    const cudaStream_t st = (cudaStream_t)stream;
    if (vec && a.group <= kMostTeam) {
        const unsigned lanes = a.group <= 32 ? 4 : a.group <= 64 ? 8 : a.group <= 128 ? 16 : 32;
        const bool one = !a.residual && a.out_dtype == a.x_dtype && (!a.gate || a.gate_dtype == a.x_dtype) && (!a.weight || a.weight_dtype == NINFER_F32);
        const int type = one ? a.x_dtype : -1;
        const auto kernel = lanes == 4    ? team_kernel_of<4>(type)
                            : lanes == 8  ? team_kernel_of<8>(type)
                            : lanes == 16 ? team_kernel_of<16>(type)
                                          : team_kernel_of<32>(type);
        const unsigned teams = kTeamThreads / lanes;
        return launch_dependent("norm", kernel, dim3((unsigned)((total + teams - 1) / teams)), dim3(kTeamThreads), 0, st, p);
    }
    if (a.group > kMostRow) return launch_dependent("norm", norm_long_kernel, dim3(p.total), dim3(1024), 0, st, p);
    const unsigned eights = (unsigned)((a.group + 7) / 8);
    // 8 elements a thread where the CTA's threads reach, 16 where rows of more than 4096 are more than about an SM each (8192 rows of 5120 49.9 us
    // by 16 and 54.0 by 8, of 6144 61.2 and 74.3; 152 rows of 5120 3.5 and 3.0; 8192 rows of 4096 41.0 and 42.2, 1024 of them 8.3 and 7.7)
    const unsigned per = eights > 2048 ? 4 : eights > 512 && total > 256 ? 2 : eights > 1024 ? 2 : 1;
    const unsigned threads = (eights + 32 * per - 1) / (32 * per) * 32;
    const auto kernel = vec ? (per == 4 ? norm_row_kernel<4, true> : per == 2 ? norm_row_kernel<2, true> : norm_row_kernel<1, true>)
                            : (per == 4 ? norm_row_kernel<4, false> : per == 2 ? norm_row_kernel<2, false> : norm_row_kernel<1, false>);
    return launch_dependent("norm", kernel, dim3(p.total), dim3(threads), 0, st, p);
}
