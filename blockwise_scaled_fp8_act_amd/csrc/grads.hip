// gfx950 global gradient norm over many tensors and clipping: norm = sqrt(sum of squares), out = g c with
// c = min(1, max_norm / (norm + eps)). A launch takes the addresses of up to kGradTensors tensors in its
// arguments, so a call copies no table to the device. Squares and sums are in 64 bits, in an order that sizes, types
// and alignment decide: no gradient overflows its square, and the norm is the same on every call.
// Bound by the memory traffic: every gradient is read once for the norm and once for the clipped copy.
#include "row_codes.hpp"
#include "schedule.hpp"

namespace bsfp8 {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kVec = 8, kStep = kThreads * kVec;
constexpr int kAhead = 8;  // steps whose loads are on the way together: long runs of reads, then of writes
static_assert(sched::kGradUnit == kStep, "a unit is a step of the workgroup");

// A thread's values of a step: eight side by side where all tensors are bf16, else four and, half a step
// further, four, so that 16-byte pieces of fp32 lie side by side over the lanes.
template <bool F32, bool ONCE>
__device__ __forceinline__ void load4_of(const void* p, int64_t at, float* f) {
    if constexpr (F32) {
        const rc_f32x4 v = load_piece<ONCE>(reinterpret_cast<const rc_f32x4*>(static_cast<const float*>(p) + at));
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = v[j];
    } else {
        const u32x2 v = load_piece<ONCE>(reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + at));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f[2 * j] = bf16_lo(v[j]);
            f[2 * j + 1] = bf16_hi(v[j]);
        }
    }
}
template <bool F32, bool WIDE, bool ONCE>
__device__ __forceinline__ void load_step(const void* p, int64_t base, float (&v)[kVec]) {
    if constexpr (WIDE) {
        load8_of<false, ONCE>(p, base + kVec * threadIdx.x, v);
    } else {
        load4_of<F32, ONCE>(p, base + 4 * threadIdx.x, v);
        load4_of<F32, ONCE>(p, base + kStep / 2 + 4 * threadIdx.x, v + 4);
    }
}
template <bool ONCE, typename V>
__device__ __forceinline__ void store_piece(V* p, V v) {
    if (ONCE) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool F32, bool WIDE, bool ONCE>
__device__ __forceinline__ void store_step(void* p, int64_t base, const float (&v)[kVec]) {
    if constexpr (WIDE) {
        store_piece<ONCE>(reinterpret_cast<rc_u32x4*>(static_cast<uint16_t*>(p) + base + kVec * threadIdx.x),
                          rc_u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = base + h * (kStep / 2) + 4 * threadIdx.x;
            const float* f = v + 4 * h;
            if constexpr (F32) store_piece<ONCE>(reinterpret_cast<rc_f32x4*>(static_cast<float*>(p) + at), rc_f32x4{f[0], f[1], f[2], f[3]});
            else store_piece<ONCE>(reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + at), u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])});
        }
    }
}

// Calls f(tensor, its first value, one past the last) for the run of units that this workgroup takes.
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

template <bool F32, bool ONCE>
__device__ __forceinline__ double squares(const void* p, int64_t from, int64_t to) {
    double sum[kAhead] = {};
    const auto add = [&](const float (&v)[kVec], double& s) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const double d = v[j];
            s = fma(d, d, s);
        }
    };
    if (reinterpret_cast<uintptr_t>(p) % 16 == 0) {
        for (; from + kAhead * kStep <= to; from += kAhead * kStep) {
            float v[kAhead][kVec];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load_step<F32, !F32, ONCE>(p, from + k * kStep, v[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) add(v[k], sum[k]);
        }
        for (; from + kStep <= to; from += kStep) {
            float v[kVec];
            load_step<F32, !F32, ONCE>(p, from, v);
            add(v, sum[0]);
        }
    }
    for (int64_t at = from + threadIdx.x; at < to; at += kThreads) {
        const double d = load_of(p, at, F32);
        sum[1] = fma(d, d, sum[1]);
    }
    return ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
}

// PAST: past the caches, which cannot hold the gradients until the second pass (1.6 GB: 303 us through them,
// 237 past them, 6.8 TB/s).
template <bool PAST>
__global__ __launch_bounds__(kThreads) void squares_kernel(GradTable t, double* partial) {
    __shared__ double part[kWaves];
    double sum = 0.0;
    for_units(t, [&](int i, int64_t from, int64_t to) {
        sum += t.in_f32[i] ? squares<true, PAST>(t.in[i], from, to) : squares<false, PAST>(t.in[i], from, to);
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

// Below 2^-126 by `wide`, in 64 bits, a value a lane: the factor has lost digits in fp32 there, or is 0, while the products of
// large gradients are ordinary. Rare, so it has no pieces.
template <bool IN_F32, bool OUT_F32, bool PAST>
__device__ __forceinline__ void scale(const void* in, void* out, int64_t from, int64_t to, float c, double wide) {
    constexpr bool kWide = !IN_F32 && !OUT_F32;
    const auto store = [&](int64_t at, float v) {
        if (OUT_F32) static_cast<float*>(out)[at] = v;
        else static_cast<uint16_t*>(out)[at] = to_bf16_bits(v);
    };
    if (wide < 0x1p-126 && wide > 0.0) {
        for (int64_t at = from + threadIdx.x; at < to; at += kThreads)
            store(at, static_cast<float>(static_cast<double>(load_of(in, at, IN_F32)) * wide));
        return;
    }
    if ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) % 16 == 0) {
        for (; from + kAhead * kStep <= to; from += kAhead * kStep) {
            float v[kAhead][kVec];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load_step<IN_F32, kWide, PAST>(in, from + k * kStep, v[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[k][j] *= c;
                store_step<OUT_F32, kWide, PAST>(out, from + k * kStep, v[k]);
            }
        }
        for (; from + kStep <= to; from += kStep) {
            float v[kVec];
            load_step<IN_F32, kWide, PAST>(in, from, v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] *= c;
            store_step<OUT_F32, kWide, PAST>(out, from, v);
        }
    }
    for (int64_t at = from + threadIdx.x; at < to; at += kThreads) store(at, load_of(in, at, IN_F32) * c);
}

// 1.6 GB of bf16 into 3.2 GB of fp32: 939 us, 5.1 TB/s, what a copy reaches (976 with the stores through the
// caches, 957 with four steps ahead).
template <bool PAST>
__global__ __launch_bounds__(kThreads) void clip_kernel(GradTable t, const double* partial, int64_t count, float max_norm, float eps, float* norm) {
    __shared__ double part[kWaves];
    const double v = norm_of(partial, count, part);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(v);
    // in 64 bits the norm is finite unless a gradient is not: then all stay as they are. Beyond fp32 alone (norm[0] reads
    // infinity) the gradients are finite, and so are the clipped ones.
    const double ratio = static_cast<double>(max_norm) / (v + static_cast<double>(eps));
    const float c = isfinite(v) && ratio < 1.0 ? static_cast<float>(ratio) : 1.0f;
    for_units(t, [&](int i, int64_t from, int64_t to) {
        if (c == 1.0f && t.in[i] == t.out[i]) return;  // in place: nothing to do
        if (t.in_f32[i]) {
            if (t.out_f32[i]) scale<true, true, PAST>(t.in[i], t.out[i], from, to, c, ratio);
            else scale<true, false, PAST>(t.in[i], t.out[i], from, to, c, ratio);
        } else {
            if (t.out_f32[i]) scale<false, true, PAST>(t.in[i], t.out[i], from, to, c, ratio);
            else scale<false, false, PAST>(t.in[i], t.out[i], from, to, c, ratio);
        }
    });
}

}  // namespace

hipError_t launch_grad_squares(const GradTable& t, bool past, double* partial, hipStream_t stream) {
    const unsigned grid = static_cast<unsigned>(sched::grad_blocks(t.first[t.count]));
    if (past) squares_kernel<true><<<grid, kThreads, 0, stream>>>(t, partial);
    else squares_kernel<false><<<grid, kThreads, 0, stream>>>(t, partial);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const double* partial, int64_t count, float* norm, hipStream_t stream) {
    norm_kernel<<<1, kThreads, 0, stream>>>(partial, count, norm);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTable& t, bool past, const double* partial, int64_t count, float max_norm, float eps, float* norm,
                            hipStream_t stream) {
    const unsigned grid = static_cast<unsigned>(sched::grad_blocks(t.first[t.count]));
    if (past) clip_kernel<true><<<grid, kThreads, 0, stream>>>(t, partial, count, max_norm, eps, norm);
    else clip_kernel<false><<<grid, kThreads, 0, stream>>>(t, partial, count, max_norm, eps, norm);
    return hipGetLastError();
}

}  // namespace bsfp8
