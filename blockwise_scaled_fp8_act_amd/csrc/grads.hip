// gfx950 global gradient norm over many tensors and clipping: norm = sqrt(sum of squares), out = g c with
// c = min(1, max_norm / (norm + eps)). A launch takes the addresses of up to kGradTensors tensors in its
// arguments, so a call copies no table to the device. Squares and sums are in 64 bits, in an order that
// depends on the sizes alone: no gradient overflows its square, and the norm is the same on every call.
// Bound by the memory traffic: every gradient is read once for the norm and once for the clipped copy.
#include "row_codes.hpp"
#include "schedule.hpp"

namespace bsfp8 {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kVec = 8, kStep = kThreads * kVec;
static_assert(sched::kGradUnit == kStep, "a unit is a step of the workgroup");

// The values of one step: value j of piece `at` + 8 tid, zero at or past n. VEC: 16-byte aligned tensors.
template <bool F32>
__device__ __forceinline__ void load_step(const void* p, int64_t at, int64_t n, bool vec, float (&v)[kVec]) {
    if (vec && at + kVec <= n) {
        load8_of<F32>(p, at, v);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = at + j < n ? load_of(p, at + j, F32) : 0.0f;
    }
}

// Calls f(tensor, first value, one past the last) for the run of units that a workgroup of `blocks` takes.
template <typename F>
__device__ __forceinline__ void for_units(const GradTable& t, F f) {
    const int64_t units = t.first[t.count];
    int64_t u = units * blockIdx.x / gridDim.x;
    const int64_t end = units * (blockIdx.x + 1) / gridDim.x;
    int lo = 0, hi = t.count - 1;  // the last tensor that begins at or before u
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.first[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    for (int i = lo; u < end; ++i) {
        const int64_t from = (u - t.first[i]) * sched::kGradUnit, stop = min(end, t.first[i + 1]);
        if (stop > u) f(i, from, min((stop - t.first[i]) * sched::kGradUnit, t.n[i]));
        u = max(u, stop);
    }
}

template <bool F32>
__device__ __forceinline__ double squares(const void* p, int64_t from, int64_t to) {
    const bool vec = reinterpret_cast<uintptr_t>(p) % 16 == 0;
    double sum[2] = {0.0, 0.0};
    for (int64_t at = from + threadIdx.x * kVec; at < to; at += kStep) {
        float v[kVec];
        load_step<F32>(p, at, to, vec, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const double d = v[j];
            sum[j & 1] = fma(d, d, sum[j & 1]);
        }
    }
    return sum[0] + sum[1];
}

__global__ __launch_bounds__(kThreads) void squares_kernel(GradTable t, double* partial) {
    __shared__ double part[kWaves];
    double sum = 0.0;
    for_units(t, [&](int i, int64_t from, int64_t to) {
        sum += t.in_f32[i] ? squares<true>(t.in[i], from, to) : squares<false>(t.in[i], from, to);
    });
    sum = block_sum<kWaves>(sum, part);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from the workgroups' sums; every workgroup that asks gets the same bits.
__device__ __forceinline__ double norm_of(const double* partial, int64_t count, double* part) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) sum += partial[i];
    return sqrt(block_sum<kWaves>(sum, part));
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const double* partial, int64_t count, float* norm) {
    __shared__ double part[kWaves];
    const double v = norm_of(partial, count, part);
    if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <bool IN_F32, bool OUT_F32>
__device__ __forceinline__ void scale(const void* in, void* out, int64_t from, int64_t to, float c) {
    const bool vec = (reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) % 16 == 0;
    for (int64_t at = from + threadIdx.x * kVec; at < to; at += kStep) {
        float v[kVec];
        load_step<IN_F32>(in, at, to, vec, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] *= c;
        if (vec && at + kVec <= to) {
            store8_of<OUT_F32>(out, at, v);
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (at + j >= to) continue;
                if (OUT_F32) static_cast<float*>(out)[at + j] = v[j];
                else static_cast<uint16_t*>(out)[at + j] = to_bf16_bits(v[j]);
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void clip_kernel(GradTable t, const double* partial, int64_t count, float max_norm, float eps,
                                                        float* norm) {
    __shared__ double part[kWaves];
    const double v = norm_of(partial, count, part);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(v);
    // a norm that is not finite leaves the gradients as they are: the caller sees it in the norm
    const double ratio = static_cast<double>(max_norm) / (v + static_cast<double>(eps));
    const float c = isfinite(v) && ratio < 1.0 ? static_cast<float>(ratio) : 1.0f;
    for_units(t, [&](int i, int64_t from, int64_t to) {
        if (c == 1.0f && t.in[i] == t.out[i]) return;  // in place: nothing to do
        if (t.in_f32[i]) {
            if (t.out_f32[i]) scale<true, true>(t.in[i], t.out[i], from, to, c);
            else scale<true, false>(t.in[i], t.out[i], from, to, c);
        } else {
            if (t.out_f32[i]) scale<false, true>(t.in[i], t.out[i], from, to, c);
            else scale<false, false>(t.in[i], t.out[i], from, to, c);
        }
    });
}

}  // namespace

hipError_t launch_grad_squares(const GradTable& t, double* partial, hipStream_t stream) {
    squares_kernel<<<static_cast<unsigned>(sched::grad_blocks(t.first[t.count])), kThreads, 0, stream>>>(t, partial);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const double* partial, int64_t count, float* norm, hipStream_t stream) {
    norm_kernel<<<1, kThreads, 0, stream>>>(partial, count, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTable& t, const double* partial, int64_t count, float max_norm, float eps, float* norm,
                            hipStream_t stream) {
    clip_kernel<<<static_cast<unsigned>(sched::grad_blocks(t.first[t.count])), kThreads, 0, stream>>>(t, partial, count, max_norm, eps, norm);
    return hipGetLastError();
}

}  // namespace bsfp8
