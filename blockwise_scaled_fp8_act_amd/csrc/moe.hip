// gfx950 kernels of a mixture-of-experts layer around the grouped FP8 GEMMs: routing (forward and
// backward), the plan that sorts the chosen (token, choice) pairs by expert, the dispatch of tokens
// into expert order with their 1x128 quantization, and the weighted return of the experts' rows
// (forward and backward). Definitions and layouts: blockwise_fp8.h. All are bound by memory traffic
// or by launch latency; none allocates, and no result depends on the order of atomics.
#include "device_common.hpp"
#include "launch.hpp"

namespace bsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;  // waves per workgroup of the wave-per-item kernels
constexpr float kSumFloor = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const f2v v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf2v));
}
__device__ __forceinline__ uint16_t to_bf16(float f) { return static_cast<uint16_t>(pack_bf16x2(f, 0.0f)); }

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = to_bf16(v); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// Orders one wave's LDS writes before its later LDS reads (no other wave is involved).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ------------------------------------------------------------------------------------- routing
// One wave a token; lane l holds the experts l, l + 64, ... . Scores and keys are in 64 bits: the
// choice is made between values that may lie closer together than fp32 rounding, and the chosen
// experts are whole numbers, so the comparison must not depend on how a score was rounded.
template <typename LT, int V>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const LT* logits, int64_t T, int E, int64_t ld,
                                                            const float* bias, int softmax, int k, int groups,
                                                            int top_groups, int renormalize, float scale,
                                                            float* weights, int32_t* ids) {
    extern __shared__ double lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
    if (t >= T) return;
    const LT* row = logits + t * ld;

    float z[V];
    bool bad = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        z[v] = e < E ? load_logit(row + e) : -INFINITY;
        bad = bad || z[v] != z[v] || (softmax && z[v] == INFINITY);
    }
    if (__any(bad)) {  // no probabilities: no expert, NaN weights
        if (lane < k) {
            weights[t * k + lane] = NAN;
            ids[t * k + lane] = -1;
        }
        return;
    }
    float top = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, z[v]);
    top = wave_max(top);
    double total = 1.0;
    if (softmax && (bias != nullptr || !renormalize)) {
        total = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) total += z[v] == -INFINITY ? 0.0 : exp(static_cast<double>(z[v]) - top);
        total = wave_sum(total);
    }
    const auto score = [&](float x) -> double {
        return softmax ? exp(static_cast<double>(x) - top) / total : 1.0 / (1.0 + exp(-static_cast<double>(x)));
    };
    double key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        key[v] = z[v];
        if (bias != nullptr && z[v] != -INFINITY) {
            key[v] = score(z[v]) + static_cast<double>(bias[e]);
            if (key[v] != key[v]) key[v] = -INFINITY;  // a NaN bias takes its expert out
        }
    }

    if (groups > 1) {
        // keys to LDS; lane g values the groups g, g + 64, ... and ranks them
        double* mine = lds + static_cast<int64_t>(wave) * (E + groups);
        double* value = mine + E;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 64 + lane < E) mine[v * 64 + lane] = key[v];
        wave_lds_fence();
        const int size = E / groups;
        for (int g = lane; g < groups; g += 64) {
            double a = -INFINITY, b = -INFINITY;  // the two largest keys
            for (int i = 0; i < size; ++i) {
                const double x = mine[g * size + i];
                if (x > a) {
                    b = a;
                    a = x;
                } else if (x > b) {
                    b = x;
                }
            }
            value[g] = bias != nullptr && b != -INFINITY ? a + b : a;
        }
        wave_lds_fence();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            if (e >= E) continue;
            const int g = e / size;
            const double x = value[g];
            int rank = 0;
            for (int i = 0; i < groups; ++i) rank += value[i] > x || (value[i] == x && i < g) ? 1 : 0;
            if (rank >= top_groups) key[v] = -INFINITY;
        }
    }

    int id = -1;  // lane j: the j-th choice
    for (int j = 0; j < k; ++j) {
        double best = -INFINITY;
        int at = E;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > best) {
                best = key[v];
                at = v * 64 + lane;
            }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double ob = __shfl_xor(best, m);
            const int oa = __shfl_xor(at, m);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
        if (best == -INFINITY) break;  // nothing left: the remaining choices stay -1
        if (lane == j) id = at;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 64 + lane == at) key[v] = -INFINITY;
    }

    const float zc = id >= 0 ? load_logit(row + id) : -INFINITY;
    double w = 0.0;
    if (softmax && renormalize) {  // softmax over the chosen logits: the row's own sum cancels
        const float ztop = wave_max(zc);
        const double x = id >= 0 ? exp(static_cast<double>(zc) - ztop) : 0.0;
        w = x / wave_sum(x);
    } else {
        w = id >= 0 ? score(zc) : 0.0;
        if (renormalize) w /= fmax(wave_sum(w), static_cast<double>(kSumFloor));
    }
    if (lane < k) {
        weights[t * k + lane] = id >= 0 ? static_cast<float>(scale * w) : 0.0f;
        ids[t * k + lane] = id;
    }
}

// One wave a token: the gradient of the chosen weights, spread over the row's logits.
//   softmax, renormalized: dz = s q (dw - sum q dw) on the chosen experts, q = softmax over them;
//   softmax:               dz = p (dp - sum dp p) on all experts, dp = s dw on the chosen ones;
//   sigmoid:               dz = dp p (1 - p) on the chosen ones, dp = s (dw - sum dw p / D) / D when
//                          renormalized (D the sum of the chosen p, a constant where it is floored).
template <typename LT, int V>
__global__ __launch_bounds__(64 * kWaves) void route_backward_kernel(const LT* logits, int64_t T, int E, int64_t ld,
                                                                     int softmax, int k, int renormalize, float scale,
                                                                     const int32_t* ids, const float* dweights,
                                                                     LT* dlogits, int64_t ldd) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
    if (t >= T) return;
    const LT* row = logits + t * ld;

    int id = lane < k ? ids[t * k + lane] : -1;
    if (id < 0 || id >= E) id = -1;
    const float dw = id >= 0 ? dweights[t * k + lane] : 0.0f;
    const float zc = id >= 0 ? load_logit(row + id) : -INFINITY;
    float dz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dz[v] = 0.0f;
    float add = 0.0f;  // lane j: what the j-th choice adds to its expert's dz
    if (__any(id >= 0)) {
        if (softmax && renormalize) {
            const float ztop = wave_max(zc);  // lanes without a choice hold -inf
            const float x = id >= 0 ? expf(zc - ztop) : 0.0f;
            const float q = x / wave_sum(x);
            add = scale * q * (dw - wave_sum(q * dw));
        } else if (softmax) {
            float z[V], p[V], top = -INFINITY, total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int e = v * 64 + lane;
                z[v] = e < E ? load_logit(row + e) : -INFINITY;
                top = fmaxf(top, z[v]);
            }
            top = wave_max(top);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] = expf(z[v] - top);
                total += p[v];
            }
            total = wave_sum(total);
            const float q = id >= 0 ? expf(zc - top) / total : 0.0f;
            const float sum = wave_sum(scale * dw * q);
#pragma unroll
            for (int v = 0; v < V; ++v) dz[v] = -(p[v] / total) * sum;
            add = scale * dw * q;
        } else {
            const float q = id >= 0 ? 1.0f / (1.0f + expf(-zc)) : 0.0f;
            float dq = scale * dw;
            if (renormalize) {
                const float sum = wave_sum(q), D = fmaxf(sum, kSumFloor);
                const float mean = wave_sum(q * dw) / D;
                dq = scale * (dw - (sum < kSumFloor ? 0.0f : mean)) / D;
            }
            add = id >= 0 ? dq * q * (1.0f / (1.0f + expf(zc))) : 0.0f;
        }
        for (int j = 0; j < k; ++j) {
            const int at = __builtin_amdgcn_readlane(id, j);
            const float x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(add), j));
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (at == v * 64 + lane) dz[v] += x;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v * 64 + lane < E) store_logit(dlogits + t * ldd + v * 64 + lane, dz[v]);
}

// ---------------------------------------------------------------------------------------- plan
// A stable counting sort of the P = T k pairs into E + 1 bins (bin E: no expert here). Each wave
// walks its own contiguous run of pairs, 64 at a time; a pair's rank among the equal bins of its 64
// comes from one ballot per bit of the bin number, and one lane per distinct bin advances the
// wave's own counter, so no atomics decide an order. With more than one workgroup a first kernel
// counts each workgroup's bins, and every workgroup sums the counts it needs.
constexpr int kPlanWaves = 8;

struct PlanArgs {
    const int32_t* ids;
    int64_t P;
    int E;
    int64_t seg;       // pairs per workgroup, a multiple of 64 * kPlanWaves
    int32_t* counts;   // [workgroups][E + 1], used with more than one workgroup
    int64_t* offsets;
    int32_t* slots;
    int32_t* rows;
};

__device__ __forceinline__ int plan_bin(const PlanArgs& a, int64_t p) {
    const int id = a.ids[p];
    return id >= 0 && id < a.E ? id : a.E;
}

__global__ __launch_bounds__(64 * kPlanWaves) void plan_count_kernel(PlanArgs a) {
    extern __shared__ int32_t hist[];
    const int tid = threadIdx.x, bins = a.E + 1;
    for (int b = tid; b < bins; b += 64 * kPlanWaves) hist[b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * a.seg, hi = min(lo + a.seg, a.P);
    for (int64_t p = lo + tid; p < hi; p += 64 * kPlanWaves) atomicAdd(&hist[plan_bin(a, p)], 1);
    __syncthreads();
    for (int b = tid; b < bins; b += 64 * kPlanWaves) a.counts[static_cast<int64_t>(blockIdx.x) * bins + b] = hist[b];
}

// Lanes of this wave whose bin equals this lane's, among the lanes of `active`.
__device__ __forceinline__ uint64_t same_bin(int bin, int bits, uint64_t active) {
    uint64_t m = active;
    for (int i = 0; i < bits; ++i) {
        const uint64_t one = __ballot((bin >> i) & 1);
        m &= (bin >> i) & 1 ? one : ~one;
    }
    return m;
}

__global__ __launch_bounds__(64 * kPlanWaves) void plan_kernel(PlanArgs a) {
    extern __shared__ int32_t base[];  // [kPlanWaves][bins] counts, then each wave's next row of a bin
    __shared__ int32_t wave_total[kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = a.E + 1;
    const int bits = 32 - __builtin_clz(a.E);  // E itself needs a place
    for (int b = tid; b < bins * kPlanWaves; b += 64 * kPlanWaves) base[b] = 0;
    __syncthreads();

    const int64_t run = a.seg / kPlanWaves;
    const int64_t lo = blockIdx.x * a.seg + wave * run, hi = min(lo + run, a.P);
    int32_t* const own = base + wave * bins;
    const uint64_t below = (uint64_t{1} << lane) - 1;
    for (int64_t p0 = lo; p0 < hi; p0 += 64) {
        const bool in = p0 + lane < hi;
        const int bin = in ? plan_bin(a, p0 + lane) : 0;
        const uint64_t m = same_bin(bin, bits, __ballot(in));
        if (in && (m & below) == 0) own[bin] += __popcll(m);
        wave_lds_fence();
    }
    __syncthreads();

    // first row of each bin for this workgroup: the bins before it, and its own bin in the
    // workgroups before this one; bins in runs of 64 * kPlanWaves, carried on
    int32_t carry = 0;
    for (int b0 = 0; b0 < bins; b0 += 64 * kPlanWaves) {
        const int b = b0 + tid;
        int32_t all = 0, before = 0;
        if (b < bins) {
            if (gridDim.x == 1) {
                for (int w = 0; w < kPlanWaves; ++w) all += base[w * bins + b];
            } else {
                for (unsigned g = 0; g < gridDim.x; ++g) {
                    const int32_t c = a.counts[static_cast<int64_t>(g) * bins + b];
                    all += c;
                    before += g < blockIdx.x ? c : 0;
                }
            }
        }
        int32_t sum = all;  // inclusive scan over the workgroup's threads
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 63) wave_total[wave] = sum;
        __syncthreads();
        int32_t start = carry + sum - all;
        for (int w = 0; w < kPlanWaves; ++w) {
            if (w < wave) start += wave_total[w];
            carry += wave_total[w];
        }
        if (b < bins) {
            if (blockIdx.x == 0) a.offsets[b] = start;
            int32_t next = start + before;
            for (int w = 0; w < kPlanWaves; ++w) {
                const int32_t c = base[w * bins + b];
                base[w * bins + b] = next;
                next += c;
            }
        }
        __syncthreads();
    }

    for (int64_t p0 = lo; p0 < hi; p0 += 64) {
        const bool in = p0 + lane < hi;
        const int64_t p = p0 + lane;
        const int bin = in ? plan_bin(a, p) : 0;
        const uint64_t m = same_bin(bin, bits, __ballot(in));
        const int32_t row = own[bin] + __popcll(m & below);
        wave_lds_fence();
        if (in && (m & below) == 0) own[bin] = row + __popcll(m);
        wave_lds_fence();
        if (in) {
            a.slots[p] = bin < a.E ? row : -1 - row;
            a.rows[row] = bin < a.E ? static_cast<int32_t>(p) : -1;
        }
    }
}

// ------------------------------------------------------------------------------------ dispatch
// One wave takes 1024 columns of a token: 16 a lane, so a 1x128 group is 8 lanes. The token is read
// and quantized once and its codes written to each of its k rows (a pass in row order would read
// the token k times). A dropped pair's padding row is zeroed by the pair's own token, so every row
// is written exactly once.
template <bool VEC>
__global__ __launch_bounds__(64 * kWaves) void dispatch_kernel(const uint16_t* x, int64_t T, int64_t H, int64_t ldx,
                                                               const int32_t* slots, int k, int64_t chunks,
                                                               uint8_t* q, int64_t ldq, float* a_s, uint16_t* copy,
                                                               int64_t ldcopy) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    if (unit >= T * chunks) return;
    const int64_t t = unit / chunks, col = (unit - t * chunks) * 1024 + lane * 16;
    const int64_t R = T * k;
    const bool in = col < H;

    u32x4 w[2] = {};  // 16 bf16
    if (VEC) {
        if (in) {
            const u32x4* p = reinterpret_cast<const u32x4*>(x + t * ldx + col);
            w[0] = p[0];
            w[1] = p[1];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (col + i < H) w[i >> 3][(i >> 1) & 3] |= static_cast<uint32_t>(x[t * ldx + col + i]) << (16 * (i & 1));
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t d = w[i >> 2][i & 3];
        amax = max(amax, max(abs_bits(bf16_lo(d)), abs_bits(bf16_hi(d))));
    }
    amax = max(amax, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(amax), 0xB1, 0xF, 0xF, false)));
    amax = max(amax, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(amax), 0x4E, 0xF, 0xF, false)));
    amax = max(amax, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(amax), 0x141, 0xF, 0xF, false)));
    const GroupScale g = group_scale<false>(__uint_as_float(amax));
    u32x4 code;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t d0 = w[i >> 1][(2 * i) & 3], d1 = w[i >> 1][(2 * i + 1) & 3];
        code[i] = encode4_in_range<false>(bf16_lo(d0) * g.m, bf16_hi(d0) * g.m, bf16_lo(d1) * g.m, bf16_hi(d1) * g.m);
    }
    if (!in) return;
    for (int j = 0; j < k; ++j) {
        const int32_t slot = slots[t * k + j];
        const int64_t r = slot >= 0 ? slot : -1 - static_cast<int64_t>(slot);
        if (r >= R) continue;
        const uint32_t keep = slot >= 0 ? 0xFFFFFFFFu : 0u;
        const u32x4 c = code & keep, w0 = w[0] & keep, w1 = w[1] & keep;
        if (VEC) {
            *reinterpret_cast<u32x4*>(q + r * ldq + col) = c;
            if (copy != nullptr) {
                u32x4* p = reinterpret_cast<u32x4*>(copy + r * ldcopy + col);
                p[0] = w0;
                p[1] = w1;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (col + i >= H) continue;
                q[r * ldq + col + i] = static_cast<uint8_t>(c[i >> 2] >> (8 * (i & 3)));
                if (copy != nullptr)
                    copy[r * ldcopy + col + i] = static_cast<uint16_t>((i < 8 ? w0 : w1)[(i >> 1) & 3] >> (16 * (i & 1)));
            }
        }
        if ((lane & 7) == 0) a_s[(col >> 7) * R + r] = slot >= 0 ? g.s : 0.0f;
    }
}

// ------------------------------------------------------------------------------------- combine
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* p, int64_t left, float (&f)[8]) {
    if (VEC) {
        const u32x4 w = left > 0 ? *reinterpret_cast<const u32x4*>(p) : u32x4{};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < left ? bf16_to_f32(p[i]) : 0.0f;
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* p, int64_t left, const float (&f)[8]) {
    if (VEC) {
        if (left > 0)
            *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                                pack_bf16x2(f[6], f[7])};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = to_bf16(f[i]);
    }
}

// One wave takes 512 columns of a token, 8 a lane, and adds its k rows in order of the choices in
// fp32. A dropped pair adds weight * 0: nothing, unless its weight is NaN (a token whose logits
// were), which then shows in the token's output.
template <bool VEC>
__global__ __launch_bounds__(64 * kWaves) void combine_kernel(const uint16_t* rows, int64_t R, int64_t ldr,
                                                              const int32_t* slots, const float* weights, int64_t T,
                                                              int k, int64_t H, int64_t chunks, uint16_t* y,
                                                              int64_t ldy) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    if (unit >= T * chunks) return;
    const int64_t t = unit / chunks, col = (unit - t * chunks) * 512 + lane * 8;
    float acc[8] = {};
    for (int j = 0; j < k; ++j) {
        const int32_t slot = slots[t * k + j];
        const float w = weights != nullptr ? weights[t * k + j] : 1.0f;
        float f[8] = {};
        if (slot >= 0 && slot < R) load8<VEC>(rows + slot * ldr + col, H - col, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += w * f[i];
    }
    store8<VEC>(y + t * ldy + col, H - col, acc);
}

// One workgroup a token: drows[slot] = w dy and dweights = <dy, rows[slot]>, choice by choice, so a
// dot product is one running sum a thread and one reduction.
template <bool VEC>
__global__ __launch_bounds__(64 * kWaves) void combine_backward_kernel(const uint16_t* dy, int64_t lddy,
                                                                       const uint16_t* rows, int64_t ldr,
                                                                       const int32_t* slots, const float* weights,
                                                                       int64_t T, int k, int64_t H, uint16_t* drows,
                                                                       int64_t lddr, float* dweights) {
    __shared__ float part[kWaves][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x, R = T * k;
    for (int j = 0; j < k; ++j) {
        const int32_t slot = slots[t * k + j];
        const int64_t r = slot >= 0 ? slot : -1 - static_cast<int64_t>(slot);
        if (r >= R) {
            if (lane == 0) part[wave][j] = 0.0f;
            continue;
        }
        const float w = slot >= 0 ? weights[t * k + j] : 0.0f;
        float dot = 0.0f;
        for (int64_t col = tid * 8; col < H; col += 64 * kWaves * 8) {
            float g[8], f[8] = {}, d[8];
            load8<VEC>(dy + t * lddy + col, H - col, g);
            if (slot >= 0) load8<VEC>(rows + r * ldr + col, H - col, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = slot >= 0 ? w * g[i] : 0.0f;
                if (slot >= 0) dot += g[i] * f[i];
            }
            store8<VEC>(drows + r * lddr + col, H - col, d);
        }
        dot = wave_sum(dot);
        if (lane == 0) part[wave][j] = dot;
    }
    __syncthreads();
    if (tid < k) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += part[w][tid];
        dweights[t * k + tid] = s;
    }
}

bool rows16(const void* p, int64_t ld_bytes) { return (reinterpret_cast<uintptr_t>(p) % 16 == 0) && ld_bytes % 16 == 0; }

}  // namespace

template <typename LT, int V>
static hipError_t route_v(const LT* logits, int64_t T, int E, int64_t ld, const RouteRule& r, const float* bias,
                          float* weights, int32_t* ids, hipStream_t stream) {
    const int64_t blocks = (T + kWaves - 1) / kWaves;
    const size_t lds = r.groups > 1 ? sizeof(double) * kWaves * (E + r.groups) : 0;
    route_kernel<LT, V><<<dim3(static_cast<unsigned>(blocks)), 64 * kWaves, lds, stream>>>(
        logits, T, E, ld, bias, r.softmax, r.k, r.groups, r.top_groups, r.renormalize, r.scale, weights, ids);
    return hipGetLastError();
}

template <typename LT, int V>
static hipError_t route_backward_v(const LT* logits, int64_t T, int E, int64_t ld, const RouteRule& r, const int32_t* ids,
                                   const float* dweights, LT* dlogits, int64_t ldd, hipStream_t stream) {
    const int64_t blocks = (T + kWaves - 1) / kWaves;
    route_backward_kernel<LT, V><<<dim3(static_cast<unsigned>(blocks)), 64 * kWaves, 0, stream>>>(
        logits, T, E, ld, r.softmax, r.k, r.renormalize, r.scale, ids, dweights, dlogits, ldd);
    return hipGetLastError();
}

// Experts per lane: the smallest of 1, 2, 4, 8, 16 that holds E <= 1024.
#define BSFP8_BY_EXPERTS(call)                  \
    (E <= 64    ? call(1)                       \
     : E <= 128 ? call(2)                       \
     : E <= 256 ? call(4)                       \
     : E <= 512 ? call(8)                       \
                : call(16))

template <typename LT>
static hipError_t route_t(const void* logits, int64_t T, int E, int64_t ld, const RouteRule& r, const float* bias,
                          float* weights, int32_t* ids, hipStream_t stream) {
#define CALL(V) route_v<LT, V>(static_cast<const LT*>(logits), T, E, ld, r, bias, weights, ids, stream)
    return BSFP8_BY_EXPERTS(CALL);
#undef CALL
}

template <typename LT>
static hipError_t route_backward_t(const void* logits, int64_t T, int E, int64_t ld, const RouteRule& r, const int32_t* ids,
                                   const float* dweights, void* dlogits, int64_t ldd, hipStream_t stream) {
#define CALL(V) route_backward_v<LT, V>(static_cast<const LT*>(logits), T, E, ld, r, ids, dweights, static_cast<LT*>(dlogits), ldd, stream)
    return BSFP8_BY_EXPERTS(CALL);
#undef CALL
}

hipError_t launch_route(const void* logits, bool f32, int64_t T, int E, int64_t ld, const RouteRule& r, const float* bias,
                        float* weights, int32_t* ids, hipStream_t stream) {
    return f32 ? route_t<float>(logits, T, E, ld, r, bias, weights, ids, stream)
               : route_t<uint16_t>(logits, T, E, ld, r, bias, weights, ids, stream);
}

hipError_t launch_route_backward(const void* logits, bool f32, int64_t T, int E, int64_t ld, const RouteRule& r,
                                 const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd,
                                 hipStream_t stream) {
    return f32 ? route_backward_t<float>(logits, T, E, ld, r, ids, dweights, dlogits, ldd, stream)
               : route_backward_t<uint16_t>(logits, T, E, ld, r, ids, dweights, dlogits, ldd, stream);
}

hipError_t launch_plan(const int32_t* ids, int64_t P, int E, int64_t* offsets, int32_t* slots, int32_t* rows,
                       int32_t* workspace, hipStream_t stream) {
    const int64_t blocks = sched::plan_blocks(P), seg = sched::plan_segment(P);
    const PlanArgs a{ids, P, E, seg, workspace, offsets, slots, rows};
    if (blocks > 1) {
        plan_count_kernel<<<dim3(static_cast<unsigned>(blocks)), 64 * kPlanWaves, sizeof(int32_t) * (E + 1), stream>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    plan_kernel<<<dim3(static_cast<unsigned>(blocks)), 64 * kPlanWaves, sizeof(int32_t) * (E + 1) * kPlanWaves, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_dispatch(const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const int32_t* slots, int k, uint8_t* q,
                           int64_t ldq, float* a_s, uint16_t* copy, int64_t ldcopy, hipStream_t stream) {
    const int64_t chunks = (H + 1023) / 1024, blocks = (T * chunks + kWaves - 1) / kWaves;
    if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
    const bool vec = H % 16 == 0 && rows16(x, 2 * ldx) && rows16(q, ldq) && (copy == nullptr || rows16(copy, 2 * ldcopy));
    const dim3 grid(static_cast<unsigned>(blocks));
    if (vec)
        dispatch_kernel<true><<<grid, 64 * kWaves, 0, stream>>>(x, T, H, ldx, slots, k, chunks, q, ldq, a_s, copy, ldcopy);
    else
        dispatch_kernel<false><<<grid, 64 * kWaves, 0, stream>>>(x, T, H, ldx, slots, k, chunks, q, ldq, a_s, copy, ldcopy);
    return hipGetLastError();
}

hipError_t launch_combine(const uint16_t* rows, int64_t R, int64_t ldr, const int32_t* slots, const float* weights,
                          int64_t T, int k, int64_t H, uint16_t* y, int64_t ldy, hipStream_t stream) {
    const int64_t chunks = (H + 511) / 512, blocks = (T * chunks + kWaves - 1) / kWaves;
    if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
    const bool vec = H % 8 == 0 && rows16(rows, 2 * ldr) && rows16(y, 2 * ldy);
    const dim3 grid(static_cast<unsigned>(blocks));
    if (vec)
        combine_kernel<true><<<grid, 64 * kWaves, 0, stream>>>(rows, R, ldr, slots, weights, T, k, H, chunks, y, ldy);
    else
        combine_kernel<false><<<grid, 64 * kWaves, 0, stream>>>(rows, R, ldr, slots, weights, T, k, H, chunks, y, ldy);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const uint16_t* dy, int64_t lddy, const uint16_t* rows, int64_t ldr,
                                   const int32_t* slots, const float* weights, int64_t T, int k, int64_t H,
                                   uint16_t* drows, int64_t lddr, float* dweights, hipStream_t stream) {
    const bool vec = H % 8 == 0 && rows16(dy, 2 * lddy) && rows16(rows, 2 * ldr) && rows16(drows, 2 * lddr);
    const dim3 grid(static_cast<unsigned>(T));
    if (vec)
        combine_backward_kernel<true><<<grid, 64 * kWaves, 0, stream>>>(dy, lddy, rows, ldr, slots, weights, T, k, H, drows,
                                                                       lddr, dweights);
    else
        combine_backward_kernel<false><<<grid, 64 * kWaves, 0, stream>>>(dy, lddy, rows, ldr, slots, weights, T, k, H, drows,
                                                                        lddr, dweights);
    return hipGetLastError();
}

}  // namespace bsfp8
