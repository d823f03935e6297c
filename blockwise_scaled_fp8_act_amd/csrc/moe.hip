// gfx950 kernels of a mixture-of-experts layer around the grouped FP8 GEMMs: routing (forward and
// backward), the plan that sorts the chosen (token, choice) pairs by expert, the dispatch of tokens
// into expert order with their 1x128 quantization, and the weighted return of the experts' rows
// (forward and backward). Definitions and layouts: blockwise_fp8.h. All are bound by memory traffic
// or by launch latency; none allocates, and no result depends on the order of atomics.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"

namespace bsfp8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
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

// Below this logit sigmoid scores are formed in 64 bits: 1 / (1 + exp(-z)) in fp32 is 0 from -88.7 on,
// where exp(-z) overflows, while the score and a floored sum of such still give ordinary weights.
constexpr float kFarLogit = -80.0f;
__device__ __forceinline__ double far_score(float z) { return 1.0 / (1.0 + exp(-static_cast<double>(z))); }

// Sum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ double sum_row16(double v) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// ------------------------------------------------------------------------------------- routing
// Scores and keys that decide a choice are compared in 64 bits: the choice is made between values
// that may lie closer together than fp32 rounding, and its results are whole numbers.
struct RouteArgs {
    int64_t T;
    int E;
    int64_t ld;
    const float* bias;
    int softmax, k, groups, top_groups, renormalize;
    float scale;
    float* weights;
    int32_t* ids;
    int vec, bias_vec;  // rows of the logits, the bias are 16-byte aligned
    int size;           // experts a group
    int shift;          // a group is 2^shift of a kernel's runs; -1: it is not
};

// One token, by a whole wave, everything in 64 bits; lane l holds the experts l, l + 64, ... . `lds`:
// E + groups doubles of this wave's own when groups > 1.
template <typename LT, int V>
__device__ __forceinline__ void route_token(const LT* row, int64_t t, const RouteArgs& a, double* lds, int lane) {
    const int E = a.E, k = a.k;
    float z[V];
    bool bad = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        z[v] = e < E ? load_logit(row + e) : -INFINITY;
        bad = bad || z[v] != z[v] || (a.softmax && z[v] == INFINITY);
    }
    if (__any(bad)) {  // no probabilities: no expert, NaN weights
        if (lane < k) {
            a.weights[t * k + lane] = NAN;
            a.ids[t * k + lane] = -1;
        }
        return;
    }
    float top = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = fmaxf(top, z[v]);
    top = wave_max(top);
    double total = 1.0;
    if (a.softmax && (a.bias != nullptr || !a.renormalize)) {
        total = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) total += z[v] == -INFINITY ? 0.0 : exp(static_cast<double>(z[v]) - top);
        total = wave_sum(total);
    }
    const auto score = [&](float x) -> double {
        return a.softmax ? exp(static_cast<double>(x) - top) / total : 1.0 / (1.0 + exp(-static_cast<double>(x)));
    };
    double key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        key[v] = z[v];
        if (a.bias != nullptr && z[v] != -INFINITY) {
            key[v] = score(z[v]) + static_cast<double>(a.bias[e]);
            if (key[v] != key[v]) key[v] = -INFINITY;  // a NaN bias takes its expert out
        }
    }

    if (a.groups > 1) {
        // keys to LDS; lane g values the groups g, g + 64, ... and ranks them
        double* value = lds + E;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 64 + lane < E) lds[v * 64 + lane] = key[v];
        wave_lds_fence();
        const int size = E / a.groups;
        for (int g = lane; g < a.groups; g += 64) {
            double first = -INFINITY, second = -INFINITY;  // the two largest keys
            for (int i = 0; i < size; ++i) {
                const double x = lds[g * size + i];
                second = fmax(second, fmin(first, x));
                first = fmax(first, x);
            }
            value[g] = a.bias != nullptr && second != -INFINITY ? first + second : first;
        }
        wave_lds_fence();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            if (e >= E) continue;
            const int g = e / size;
            const double x = value[g];
            int rank = 0;
            for (int i = 0; i < a.groups; ++i) rank += value[i] > x || (value[i] == x && i < g) ? 1 : 0;
            if (rank >= a.top_groups) key[v] = -INFINITY;
        }
        wave_lds_fence();
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
    if (a.softmax && a.renormalize) {  // softmax over the chosen logits: the row's own sum cancels
        const float ztop = wave_max(zc);
        const double x = id >= 0 ? exp(static_cast<double>(zc) - ztop) : 0.0;
        w = x / wave_sum(x);
    } else {
        w = id >= 0 ? score(zc) : 0.0;
        const double sum = wave_sum(w);
        if (a.renormalize) w /= fmax(sum, static_cast<double>(kSumFloor));
    }
    if (lane < k) {
        a.weights[t * k + lane] = id >= 0 ? static_cast<float>(a.scale * w) : 0.0f;
        a.ids[t * k + lane] = id;
    }
}

// Every rule the kernel below does not take: more than 16 choices, more groups than its lanes. One wave
// a token.
template <typename LT, int V>
__global__ __launch_bounds__(64 * kWaves) void route_wide_kernel(const LT* logits, RouteArgs a) {
    extern __shared__ double lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
    if (t >= a.T) return;
    route_token<LT, V>(logits + t * a.ld, t, a, lds + static_cast<int64_t>(wave) * (a.E + a.groups), lane);
}

// fp32 as an unsigned number of the same order, and back.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
constexpr uint32_t kLeastKey = 0x00800000u;  // below: -inf (and the packed 0 of a taken or missing expert)

template <int L>
__device__ __forceinline__ uint32_t team_umax(uint32_t v) {
    v = umax_row16(v);
    if (L == 64) {
        auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(r[0], r[1]);
        r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(r[0], r[1]);
    }
    return v;
}

// Sum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float sum_row16(float v) {
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0xB1, 0xF, 0xF, false));
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x4E, 0xF, 0xF, false));
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x141, 0xF, 0xF, false));
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x140, 0xF, 0xF, false));
    return v;
}
template <int L>
__device__ __forceinline__ float team_sum(float v) {
    v = sum_row16(v);
    if (L == 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}

// How many of the other 15 lanes of the row come before this one: a larger key, or the same and a
// smaller index.
template <int R = 1>
__device__ __forceinline__ int rank_row16(double key, int idx) {
    if constexpr (R == 16) {
        return 0;
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, key);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), 0x120 + R, 0xF, 0xF, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), 0x120 + R, 0xF, 0xF, false);
        const int oi = __builtin_amdgcn_update_dpp(0, idx, 0x120 + R, 0xF, 0xF, false);
        const double ok = __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
        return (ok > key || (ok == key && oi < idx) ? 1 : 0) + rank_row16<R + 1>(key, idx);
    }
}

// Descending sort of V values in registers: odd-even merge network.
template <int V>
__device__ __forceinline__ void sort_descending(uint32_t (&s)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (j + i + q < V && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
                        const uint32_t x = s[j + i], y = s[j + i + q];
                        s[j + i] = max(x, y);
                        s[j + i + q] = min(x, y);
                    }
}

template <int V>
__device__ __forceinline__ void load_run(const float* p, bool vec, int left, float (&z)[V]) {
    if (V % 4 == 0 && vec) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const float4 f = v < left ? *reinterpret_cast<const float4*>(p + v) : float4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            z[v] = f.x;
            z[v + 1] = f.y;
            z[v + 2] = f.z;
            z[v + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = v < left ? p[v] : -INFINITY;
    }
}
template <int V>
__device__ __forceinline__ void load_run(const uint16_t* p, bool vec, int left, float (&z)[V]) {
    if (V % 4 == 0 && vec) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const uint2 w = v < left ? *reinterpret_cast<const uint2*>(p + v) : uint2{0xFF80FF80u, 0xFF80FF80u};
            z[v] = bf16_lo(w.x);
            z[v + 1] = bf16_hi(w.x);
            z[v + 2] = bf16_lo(w.y);
            z[v + 3] = bf16_hi(w.y);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = v < left ? bf16_to_f32(p[v]) : -INFINITY;
    }
}

enum RouteKey { kKeyLogit, kKeySigmoid, kKeySoftmax };
// Bounds of a score's error in fp32, from one unit of the last place in each of the hardware's exp2 and
// reciprocal. Sigmoid: 3 half units for the sum and the reciprocal and 0.8 from the exponential (p (1 -
// p) |z| is at most 0.23): 3.8 * 2^-24 of 8. Softmax: a sum 21 roundings deep (15 in a lane, 6 across), its
// terms' errors weighted by themselves, the quotient: 25 * 2^-24 of 32, at a score of 1.
constexpr float kSigmoidError = 4.8e-7f;  // 2^-21
constexpr float kSoftmaxError = 2e-6f;    // 2^-19
constexpr float kKeyRounding = 6e-8f;     // 2^-24, of a key or a sum: the rounding of an addition

// L lanes a token (16, four tokens a wave, up to 256 experts; 64 up to 1024), V consecutive experts a
// lane. Candidates come from fp32 keys cut to make room for the expert's index in the low bits: then
// one unsigned maximum over the lanes (a DPP step each) yields key and index, and the owner drops
// the head of its sorted run. Where neighbours among the k + 2 (at most 16) best are too close for the
// cut keys to order them, the candidates are ranked by their exact keys, one a lane. Where the cut
// keys cannot tell that the k best are among the candidates (the k-th too close to the best key that is
// none: four nearly equal keys at the border, three for k = 15, two for k = 16),
// the choices are made one by one from 64-bit keys; where fp32 cannot tell which groups are kept,
// the groups are valued again in 64 bits. KEY: the logits, which are exact, or a score + bias.
// 16384 tokens of 256 experts in groups 10.8 us in a graph, 12.3-12.9 with inputs that change (15.7 where
// each lane formed its own exact keys; 48 with one wave a token and 64-bit shuffles; their bytes alone
// 3.4), with a softmax and no groups 10.7 and 12.6 (16.3), one token 4.2 us. Vector issue is about half
// of that: 880 instructions a wave of four tokens, nearly half of them the sort and the takes, 14
// thousand of 26 thousand cycles, all waves in one round. The launch ends with its slowest waves, most
// likely those with exact keys: the cut's tolerance (2^-14 of a key at 256 experts) holds neighbours of
// 4% of the tokens, so of 15% of the waves, where fp32's own error would hold those of 0.05%.
template <typename LT, int V, int L, RouteKey KEY>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const LT* logits, RouteArgs a) {
    extern __shared__ double lds[];
    constexpr bool BIAS = KEY != kKeyLogit, SOFTMAX_KEY = KEY == kKeySoftmax;
    constexpr int kTokens = 64 / L;
    constexpr uint32_t kIndex = L * V - 1;  // low bits of a packed key
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int team = lane / L, sub = lane % L;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens;
    if (t0 >= a.T) return;
    const int64_t t = t0 + team;
    const bool live = t < a.T;
    const LT* row = logits + (live ? t : a.T - 1) * a.ld;
    const int E = a.E, k = a.k, e0 = sub * V;
    const uint64_t team_lanes = (L == 64 ? ~uint64_t{0} : (uint64_t{1} << L) - 1) << (team * L);
    const auto team_any = [&](bool x) { return (__ballot(x) & team_lanes) != 0; };

    float z[V];
    load_run<V>(row + e0, a.vec && E % 4 == 0, E - e0, z);
    float key[V];  // starts as the bias: on the way with the logits
    if (BIAS) load_run<V>(a.bias + e0, a.bias_vec && E % 4 == 0, E - e0, key);
    bool bad = false;
    uint32_t low = 0;  // bits that the cut keys lose
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (!BIAS) z[v] += 0.0f;  // -0 and 0 are the same key
        bad = bad || z[v] != z[v] || (a.softmax && z[v] == INFINITY);
        low |= z[v] == -INFINITY ? 0u : __float_as_uint(z[v]) & kIndex;
    }
    bad = team_any(bad);
    const bool exact = !BIAS && (sizeof(LT) == 2 || !team_any(low != 0));

    float total = 1.0f, top = 0.0f;  // softmax: the row's sum of exp(z - top)
    if (SOFTMAX_KEY || (!BIAS && a.softmax && !a.renormalize)) {
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) m = max(m, ordered(z[v]));
        top = from_ordered(team_umax<L>(m));
        total = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) total += z[v] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((z[v] - top) * 1.44269504f);
        total = team_sum<L>(total);
    }
    constexpr float key_error = SOFTMAX_KEY ? kSoftmaxError : kSigmoidError;
    if (BIAS) {
        if (SOFTMAX_KEY) {
            const float inverse = __builtin_amdgcn_rcpf(total);
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] += __builtin_amdgcn_exp2f((z[v] - top) * 1.44269504f) * inverse;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                key[v] += __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z[v] * -1.44269504f));
        }
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] != key[v] || z[v] == -INFINITY ? -INFINITY : key[v];
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = z[v];
    }
    // The exact key of an expert: score in 64 bits + bias. The softmax's sum in 64 bits is made where a
    // key is first asked for (prepare_exact before exact_key, in uniform control flow). What follows is
    // rare, but the launch waits for the last wave: the whole wave works for a team that asks.
    double total64 = 0.0;
    const auto asks = [&](uint64_t lanes, int x) { return (lanes >> (x * L) & (L == 64 ? ~uint64_t{0} : (uint64_t{1} << L) - 1)) != 0; };
    constexpr int kSteps = (L * V + 63) / 64;
    const auto prepare_exact = [&](uint64_t lanes) {
        if (!SOFTMAX_KEY) return;
        lanes &= __ballot(total64 == 0.0);
#pragma unroll 1
        for (int x = 0; x < kTokens; ++x) {
            if (!asks(lanes, x)) continue;
            const LT* const other = logits + min(t0 + x, a.T - 1) * a.ld;
            const float other_top = __shfl(top, x * L);
            double sum = 0.0;
#pragma unroll 4
            for (int v = 0; v < kSteps; ++v) {
                const int e = v * 64 + lane;
                const float y = load_logit(other + min(e, E - 1));
                sum += e >= E || y == -INFINITY ? 0.0 : exp(static_cast<double>(y) - other_top);
            }
            sum = wave_sum(sum);
            if (team == x) total64 = sum;
        }
    };
    const auto exact_key_of = [&](float x, int e, float row_top, double row_total) -> double {
        if (!BIAS) return x + 0.0f;
        const double y = exp(SOFTMAX_KEY ? static_cast<double>(x) - row_top : -static_cast<double>(x));
        return (SOFTMAX_KEY ? y / row_total : 1.0 / (1.0 + y)) + static_cast<double>(a.bias[e]);
    };
    const auto exact_key = [&](float x, int e) { return exact_key_of(x, e, top, total64); };

    // doubles of LDS a token has: its keys, a group's run padded to an odd length, and the groups' values
    const int size = a.size, pitch = size | 1, area = a.groups * (pitch + 1);
    uint32_t dropped = 0;  // bit v: the group of expert e0 + v is not kept
    if (a.groups > 1) {
        double* const mine64 = lds + static_cast<int64_t>(wave * kTokens + team) * area;
        float* const mine = reinterpret_cast<float*>(mine64);
        float* const value = mine + a.groups * pitch;
        // a group of whole runs, 1, 2, 4, 8 or 16 of them, is valued in registers; any other through LDS
        const bool regular = a.shift >= 0;
        float first = -INFINITY, second = -INFINITY;
        int group = sub;  // the group this lane values
        if (regular) {
            group = sub >> a.shift;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                second = __builtin_amdgcn_fmed3f(first, second, key[v]);
                first = fmaxf(first, key[v]);
            }
            const auto join = [&](int of, int os) {
                const float x = __uint_as_float(of), y = __uint_as_float(os);
                second = fmaxf(fminf(first, x), fmaxf(second, y));
                first = fmaxf(first, x);
            };
#define BSFP8_JOIN(ctrl)                                                                              \
    join(__builtin_amdgcn_update_dpp(0, __float_as_uint(first), ctrl, 0xF, 0xF, false),               \
         __builtin_amdgcn_update_dpp(0, __float_as_uint(second), ctrl, 0xF, 0xF, false))
            if (a.shift >= 1) BSFP8_JOIN(0xB1);
            if (a.shift >= 2) BSFP8_JOIN(0x4E);
            if (a.shift >= 3) BSFP8_JOIN(0x141);
            if (a.shift >= 4) BSFP8_JOIN(0x140);
#undef BSFP8_JOIN
        } else {
            // lane g reads run g, at an odd distance from its neighbours: no bank twice
            const int spare = 2 * area - 1;  // past the keys and group values: for lanes past E
            int i = e0 % size, at = e0 / size * pitch + i;
#pragma unroll 4
            for (int v = 0; v < V; ++v) {
                mine[e0 + v < E ? at : spare] = key[v];
                ++i;
                ++at;
                if (i == size) {
                    i = 0;
                    at += pitch - size;
                }
            }
            wave_lds_fence();
            if (sub < a.groups)
                for (int j = 0; j < size; ++j) {
                    const float x = mine[sub * pitch + j];
                    second = fmaxf(second, fminf(first, x));
                    first = fmaxf(first, x);
                }
        }
        // Ranks of the groups. With exact keys they are exact. Else a sum of two keys is off by two scores'
        // errors, the keys' roundings and its own, a difference of two sums by twice that (each group
        // with the larger keys of the two sees the pair), and a border inside it is open.
        float tol = 0.0f;
        if (BIAS) {
            const float big = fmaxf(fabsf(first), second == -INFINITY ? 0.0f : fabsf(second));
            tol = first == -INFINITY ? 0.0f : 4.0f * key_error + 8.0f * kKeyRounding * big;
            if (second != -INFINITY) first += second;
        }
        wave_lds_fence();
        if (group < a.groups) value[group] = first;
        wave_lds_fence();
        int before = 0, maybe = 0;
        const float high = first + tol, low = tol < INFINITY ? first - tol : -INFINITY;
#pragma unroll 4
        for (int j = 0; j < a.groups; ++j) {
            const float x = value[j];
            if (BIAS) {
                before += x > high ? 1 : 0;
                maybe += x >= low ? 1 : 0;  // itself, at least
            } else {
                before += x > first || (x == first && j < group) ? 1 : 0;
            }
        }
        bool keep = group < a.groups && before < a.top_groups;
        bool lanes_keep = regular;  // keep is about the lane's own experts
        const uint64_t doubt = BIAS ? __ballot(keep && maybe > a.top_groups && !bad && live) : 0;
        if (doubt != 0) {
            wave_lds_fence();
            prepare_exact(doubt);
#pragma unroll 1
            for (int x = 0; x < kTokens; ++x) {
                if (!asks(doubt, x)) continue;
                const LT* const other = logits + (t0 + x) * a.ld;
                const float other_top = __shfl(top, x * L);
                const double other_total = __shfl(total64, x * L);
                double* const keys = lds + static_cast<int64_t>(wave * kTokens + x) * area;
#pragma unroll 4
                for (int v = 0; v < kSteps; ++v) {
                    const int e = v * 64 + lane;
                    const float z1 = load_logit(other + min(e, E - 1));
                    const double y = exact_key_of(z1, min(e, E - 1), other_top, other_total);
                    const int g = e / size;
                    if (e < E) keys[g * pitch + e - g * size] = z1 == -INFINITY || y != y ? -INFINITY : y;
                }
            }
            wave_lds_fence();
        }
        if ((doubt & team_lanes) != 0) {
            double* const value64 = mine64 + a.groups * pitch;
            double one = -INFINITY, two = -INFINITY;
            if (sub < a.groups) {
#pragma unroll 8
                for (int j = 0; j < size; ++j) {
                    const double x = mine64[sub * pitch + j];
                    two = fmax(two, fmin(one, x));
                    one = fmax(one, x);
                }
                if (two != -INFINITY) one += two;
                value64[sub] = one;
            }
            wave_lds_fence();
            int rank = 0;
            if (sub < a.groups)
#pragma unroll 4
                for (int j = 0; j < a.groups; ++j) rank += value64[j] > one || (value64[j] == one && j < sub) ? 1 : 0;
            keep = sub < a.groups && rank < a.top_groups;
            lanes_keep = false;
        }
        if (lanes_keep) {
            dropped = keep ? 0u : ~0u;
        } else {
            const uint64_t kept = (__ballot(keep) & team_lanes) >> (team * L);  // bit g: group g
            int g = e0 / size, i = e0 - g * size;
#pragma unroll 1
            for (int v = 0; v < V; ++v) {
                dropped |= ((kept >> g) & 1 ? 0u : 1u) << v;
                if (++i == size) {
                    i = 0;
                    ++g;
                }
            }
        }
    }

    // packed keys; -inf stays below kLeastKey
    uint32_t run[V];
#pragma unroll
    for (int v = 0; v < V; ++v) run[v] = (ordered(key[v]) & ~kIndex) | ((kIndex - e0) ^ v);
    if (dropped != 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if ((dropped >> v) & 1) run[v] = 0;
    }
    sort_descending<V>(run);

    const int m = min(k + 2, 16);
    uint32_t mine = 0, at_k = 0;  // lane j: the j-th candidate; every lane: the k-th
    const auto take = [&](int j, auto depth) {  // the best head; its run moves up, as far as m takes can reach
        constexpr int kDepth = decltype(depth)::value < V ? decltype(depth)::value : V;
        const uint32_t best = team_umax<L>(run[0]);
        if (sub == j) mine = best;
        if (j == k - 1) at_k = best;
        const uint32_t own = run[0] == best ? ~0u : 0u;  // a bit select: "own ? a : b" becomes an indexed read
#pragma unroll
        for (int v = 0; v < kDepth; ++v) run[v] = ((v + 1 < V ? run[v + 1 < V ? v + 1 : v] : 0u) & own) | (run[v] & ~own);
    };
    if (m <= 10) {
        const auto takes = [&](auto self, auto at) {
            constexpr int j = decltype(at)::value;
            if constexpr (j < 10) {
                if (j >= m) return;
                take(j, std::integral_constant<int, 10 - j>{});
                self(self, std::integral_constant<int, j + 1>{});
            }
        };
        takes(takes, std::integral_constant<int, 0>{});
    } else {
        for (int j = 0; j < m; ++j) take(j, std::integral_constant<int, 16>{});
    }
    const uint32_t next = team_umax<L>(run[0]);

    // Whether two packed keys, x before y, may stand for keys in the other order.
    const auto close = [&](uint32_t x, uint32_t y) {
        if (exact || y < kLeastKey) return false;
        if (!BIAS) return (x & ~kIndex) == (y & ~kIndex);
        const float f = from_ordered(x & ~kIndex), h = from_ordered(y & ~kIndex), big = fmaxf(fabsf(f), fabsf(h));
        return !(f - h > 2.0f * (key_error + kKeyRounding * big) + big * (2.0f * (kIndex + 1) * 1.1920929e-7f));
    };
    const bool open = close(at_k, next);  // an expert that is no candidate may be among the k best
    const uint32_t after = __builtin_amdgcn_update_dpp(0, mine, 0x101, 0xF, 0xF, false);  // the next lane's

    bool have = sub < 16 && mine >= kLeastKey;
    int id = have ? static_cast<int>(kIndex - (mine & kIndex)) : 0x7FFFFFFF;
    float zc = have ? load_logit(row + id) : -INFINITY;
    int rank = sub;
    const uint64_t near = __ballot(have && sub < k && close(mine, after) && live && !bad);
    if (near != 0) {  // by the exact keys
        prepare_exact(near);
        double full = -INFINITY;
        if (have) full = exact_key(zc, id);
        const int exact_rank = rank_row16(full, id);  // lanes without a candidate: -inf, last
        if ((near & team_lanes) != 0) rank = exact_rank;
    }
    bool chosen = have && rank < k;
    const uint64_t opens = __ballot(open && live && !bad);
    if (opens != 0) {  // choice by choice from 64-bit keys in LDS
        double* const key64 = lds + static_cast<int64_t>(wave * kTokens + team) * area;
        wave_lds_fence();
        prepare_exact(opens);
#pragma unroll 4
        for (int v = 0; v < V; ++v) {
            const int e = min(e0 + v, E - 1);
            const float x = load_logit(row + e);
            const double y = exact_key(x, e);
            if (e0 + v < E) key64[e0 + v] = x == -INFINITY || y != y || ((dropped >> v) & 1) ? -INFINITY : y;
        }
        int found = -1;
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            wave_lds_fence();
            double best = -INFINITY;
            int at = E;
#pragma unroll 1
            for (int e = e0; e < min(e0 + V, E); ++e) {
                const double x = key64[e];
                if (x > best) {
                    best = x;
                    at = e;
                }
            }
#pragma unroll 1
            for (int x = 1; x < L; x <<= 1) {
                const double ob = __shfl_xor(best, x);
                const int oa = __shfl_xor(at, x);
                if (ob > best || (ob == best && oa < at)) {
                    best = ob;
                    at = oa;
                }
            }
            if (sub == j && best != -INFINITY) found = at;
            wave_lds_fence();
            if (at >= e0 && at < min(e0 + V, E)) key64[at] = -INFINITY;
        }
        if (open) {
            have = chosen = found >= 0;
            id = found;
            rank = sub;
            zc = have ? load_logit(row + id) : -INFINITY;
        }
    }

    float w;
    if (a.softmax && a.renormalize) {
        const float ztop = from_ordered(umax_row16(chosen ? ordered(zc) : 0u));
        w = chosen ? expf(zc - ztop) : 0.0f;
        const float sum = sum_row16(w);
        w /= sum;
    } else {
        w = a.softmax ? expf(zc - top) / total : 1.0f / (1.0f + expf(-zc));
        if (!chosen) w = 0.0f;
        const float sum = sum_row16(w);
        if (a.renormalize) w /= fmaxf(sum, kSumFloor);
    }
    w *= a.scale;
    const uint64_t far = __ballot(!a.softmax && chosen && zc < kFarLogit && live && !bad);
    if (far != 0) {
        const double p = chosen ? far_score(zc) : 0.0, sum = sum_row16(p);
        if ((far & team_lanes) != 0) w = static_cast<float>(a.scale * (a.renormalize ? p / fmax(sum, static_cast<double>(kSumFloor)) : p));
    }
    if (live && sub < k) {
        if (bad) {  // no probabilities: no expert, NaN weights
            a.weights[t * k + sub] = NAN;
            a.ids[t * k + sub] = -1;
        } else if (!have) {  // the candidates fill the lanes from 0 on: this choice found no expert
            a.weights[t * k + sub] = 0.0f;
            a.ids[t * k + sub] = -1;
        }
    }
    if (live && !bad && chosen) {
        a.weights[t * k + rank] = w;
        a.ids[t * k + rank] = id;
    }
}

// A choice's part of the sigmoid gradient in 64 bits; p: its score, sum, dot: the sums of p, p dw.
__device__ __forceinline__ float far_gradient(double p, double sum, double dot, float z, float dw, int renormalize, float scale) {
    const double D = renormalize ? fmax(sum, static_cast<double>(kSumFloor)) : 1.0;
    const double mean = renormalize && sum >= kSumFloor ? dot / D : 0.0;
    return static_cast<float>(scale * (p / D * (dw - mean)) * far_score(-z));
}

// One wave a token: the gradient of the chosen weights, spread over the row's logits.
//   softmax, renormalized: dz = s q (dw - sum q dw) on the chosen experts, q = softmax over them;
//   softmax:               dz = p (dp - sum dp p) on all experts, dp = s dw on the chosen ones;
//   sigmoid:               dz = s q (dw - sum dw q) (1 - p) on the chosen ones, q = p / D, when renormalized
//                          (D the sum of the chosen p; floored it is a constant, without the sum of
//                          dw q), else dz = s p dw (1 - p). p is divided first: q is at most 1, while
//                          dw / D overflows where the scores are small.
// For more than 16 choices or 256 experts; the rest: route_backward_team_kernel.
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
            float q = id >= 0 ? 1.0f / (1.0f + expf(-zc)) : 0.0f, mean = 0.0f;
            if (renormalize) {
                const float sum = wave_sum(q);
                q /= fmaxf(sum, kSumFloor);
                mean = sum < kSumFloor ? 0.0f : wave_sum(q * dw);
            }
            add = scale * (q * (dw - mean) * (1.0f / (1.0f + expf(zc))));
            if (__any(id >= 0 && zc < kFarLogit)) {
                const double p = id >= 0 ? far_score(zc) : 0.0;
                add = far_gradient(p, wave_sum(p), wave_sum(p * dw), zc, dw, renormalize, scale);
            }
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

template <int V>
__device__ __forceinline__ void store_run(float* p, bool vec, int left, const float (&z)[V]) {
    if (V % 4 == 0 && vec) {
#pragma unroll
        for (int v = 0; v < V; v += 4)
            if (v < left) *reinterpret_cast<float4*>(p + v) = float4{z[v], z[v + 1], z[v + 2], z[v + 3]};
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < left) p[v] = z[v];
    }
}
template <int V>
__device__ __forceinline__ void store_run(uint16_t* p, bool vec, int left, const float (&z)[V]) {
    if (V % 4 == 0 && vec) {
#pragma unroll
        for (int v = 0; v < V; v += 4)
            if (v < left) *reinterpret_cast<uint2*>(p + v) = uint2{pack_bf16x2(z[v], z[v + 1]), pack_bf16x2(z[v + 2], z[v + 3])};
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < left) p[v] = to_bf16(z[v]);
    }
}

// The same for up to 16 choices and 256 experts: 16 lanes a token, sums by DPP; a lane holds four
// experts of every 64, so that a token's lanes store whole lines, and the choices, which differ, find
// their experts through LDS. 8191 rows of 64 experts in bf16 2.5 us (with a wave a token and sums by
// shuffles 4.2), 16384 of 256 with sigmoid scores in fp32 5.9-6.4 (10.6; 8.4 with a comparison for every
// choice and expert), with the plain softmax 9.7 (12.8).
template <typename LT, int V>
__global__ __launch_bounds__(64 * kWaves) void route_backward_team_kernel(const LT* logits, int64_t T, int E, int64_t ld,
                                                                          int softmax, int k, int renormalize, float scale,
                                                                          const int32_t* ids, const float* dweights,
                                                                          LT* dlogits, int64_t ldd, int vec, int dvec) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & 15;
    constexpr int C = V < 4 ? V : 4;  // consecutive experts
    const int e0 = sub * C;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * 4;
    if (t0 >= T) return;
    const bool live = t0 + (lane >> 4) < T;
    const int64_t t = live ? t0 + (lane >> 4) : T - 1;
    const LT* row = logits + t * ld;

    int id = sub < k ? ids[t * k + sub] : -1;
    float dw = sub < k ? dweights[t * k + sub] : 0.0f;
    const bool have = id >= 0 && id < E;
    if (!have) {
        id = -1;
        dw = 0.0f;
    }
    const float zc = have ? load_logit(row + id) : -INFINITY;
    float dz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dz[v] = 0.0f;
    __shared__ __attribute__((aligned(16))) float spread[kWaves * 4][16 * V];
    float* const mine = spread[wave * 4 + (lane >> 4)];
#pragma unroll
    for (int c = 0; c < V / C; ++c)
#pragma unroll
        for (int i = 0; i < C; ++i) mine[64 * c + e0 + i] = 0.0f;
    wave_lds_fence();
    float add = 0.0f;  // what this lane's choice adds to its expert's dz
    if (softmax && renormalize) {
        const float ztop = from_ordered(umax_row16(ordered(zc)));
        const float x = have ? expf(zc - ztop) : 0.0f;
        const float q = x / sum_row16(x);
        add = scale * q * (dw - sum_row16(have ? q * dw : 0.0f));
    } else if (softmax) {
        float z[V], total = 0.0f;
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < V / C; ++c) {
            float part[C];
            load_run<C>(row + 64 * c + e0, vec && E % 4 == 0, E - 64 * c - e0, part);
#pragma unroll
            for (int i = 0; i < C; ++i) z[C * c + i] = part[i];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) m = max(m, ordered(z[v]));
        const float top = from_ordered(umax_row16(m));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = expf(z[v] - top);
            total += z[v];
        }
        total = sum_row16(total);
        const float q = have ? expf(zc - top) / total : 0.0f;
        add = scale * dw * q;
        const float sum = sum_row16(have ? add : 0.0f);
        const bool any = sum_row16(have ? 1.0f : 0.0f) != 0.0f;
        const float f = any ? -(sum / total) : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) dz[v] = any ? z[v] * f : 0.0f;
    } else {
        float q = have ? 1.0f / (1.0f + expf(-zc)) : 0.0f, mean = 0.0f;
        if (renormalize) {
            const float sum = sum_row16(q);
            q /= fmaxf(sum, kSumFloor);
            mean = sum < kSumFloor ? 0.0f : sum_row16(q * dw);
        }
        add = scale * (q * (dw - mean) * (1.0f / (1.0f + expf(zc))));
        const uint64_t far = __ballot(have && zc < kFarLogit);
        if (far != 0) {
            const double p = have ? far_score(zc) : 0.0;
            const float x = far_gradient(p, sum_row16(p), sum_row16(p * dw), zc, dw, renormalize, scale);
            if (((far >> (lane & 48)) & 0xFFFF) != 0) add = x;
        }
    }
    if (have) __hip_atomic_fetch_add(mine + id, add, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
    wave_lds_fence();
    if (!live) return;
#pragma unroll
    for (int c = 0; c < V / C; ++c) {
        float part[C];
#pragma unroll
        for (int i = 0; i < C; ++i) part[i] = dz[C * c + i] + mine[64 * c + e0 + i];
        store_run<C>(dlogits + t * ldd + 64 * c + e0, dvec && E % 4 == 0, E - 64 * c - e0, part);
    }
}

// ---------------------------------------------------------------------------------------- plan
// A stable counting sort of the P = T k pairs into E + 1 bins (bin E: no expert here). A workgroup
// takes its pairs in rounds; in a round each wave has S steps of 64 pairs, loaded together. A pair's
// rank among the equal bins of its 64 comes from one ballot per bit of the bin number, and one lane
// per distinct bin advances the wave's own counter, step after step, so no atomics decide an order.
// Up to 8192 pairs are one round of one workgroup, which gathers the rows in LDS and stores them in
// order. With more (MANY) a first kernel counts each workgroup's bins, and every workgroup sums the
// counts it needs. Latency-bound, in a graph: 512 pairs 3.0 us, 4096 6.2, 8192 8.7 (10.8 with the rows
// scattered to memory), 65536 pairs of 64 experts 9.0 with the counting launch (19 with the counts
// summed one workgroup after the other).
constexpr int kCountThreads = 512, kCountSteps = 4;
constexpr int kBinBits = 11;  // bins 0 to 1024
typedef uint32_t u32_pair __attribute__((may_alias));  // two 16-bit counters

struct PlanArgs {
    const int32_t* ids;
    int64_t P;
    int E;
    int64_t seg;       // pairs per workgroup, whole rounds
    int32_t* counts;   // [workgroups][E + 1], used with more than one workgroup
    int64_t* offsets;
    int32_t* slots;
    int32_t* rows;
};

__device__ __forceinline__ int plan_bin(int32_t id, int E) { return id >= 0 && id < E ? id : E; }

__global__ __launch_bounds__(kCountThreads) void plan_count_kernel(PlanArgs a) {
    extern __shared__ int32_t hist[];
    const int tid = threadIdx.x, bins = a.E + 1;
    for (int b = tid; b < bins; b += kCountThreads) hist[b] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * a.seg, hi = min(lo + a.seg, a.P);
    for (int64_t p0 = lo; p0 < hi; p0 += kCountSteps * kCountThreads) {
        int32_t id[kCountSteps];
#pragma unroll
        for (int s = 0; s < kCountSteps; ++s) id[s] = p0 + s * kCountThreads + tid < hi ? a.ids[p0 + s * kCountThreads + tid] : 0;
#pragma unroll
        for (int s = 0; s < kCountSteps; ++s)
            if (p0 + s * kCountThreads + tid < hi) atomicAdd(&hist[plan_bin(id[s], a.E)], 1);
    }
    __syncthreads();
    for (int b = tid; b < bins; b += kCountThreads) a.counts[static_cast<int64_t>(blockIdx.x) * bins + b] = hist[b];
}

template <int W, int S, bool MANY>
__global__ __launch_bounds__(64 * W) void plan_kernel(PlanArgs a) {
    constexpr int kThreads = 64 * W, kRound = sched::plan_round(W, S);
    extern __shared__ int32_t bin_lds[];
    static_assert(kRound <= 0xFFFF, "a wave's place in a bin is kept in 16 bits");
    __shared__ int32_t wave_total[W];
    __shared__ uint16_t row_pair[MANY ? 2 : kRound];  // without MANY: a row's pair, kNoPair for none
    constexpr uint16_t kNoPair = 0xFFFF;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = a.E + 1;
    const int bits = 32 - __builtin_clz(a.E);  // E itself needs a place
    int32_t* const next = bin_lds;     // [bins]: this workgroup's next row of a bin
    int32_t* const all = next + bins;  // [bins]: pairs of a bin
    // [W][bins]: a wave's pairs of a bin in this round, then those of the waves before it
    uint16_t* const wave_bins = reinterpret_cast<uint16_t*>(all + bins);
    const int pitch = (bins + 1) & ~1;  // whole words a wave
    const int64_t lo = blockIdx.x * a.seg, hi = min(lo + a.seg, a.P);
    u32_pair* const own = reinterpret_cast<u32_pair*>(wave_bins + wave * pitch);

    for (int64_t p0 = lo; p0 == lo || (MANY && p0 < hi); p0 += kRound) {
        // a short round is spread over all waves
        const int steps = static_cast<int>((min(hi - p0, int64_t{kRound}) + kThreads - 1) / kThreads);
        const int64_t mine = p0 + wave * 64 * steps + lane;
        const auto in = [&](int s) { return s < steps && mine + 64 * s < hi; };
        int32_t id[S], rank[S];
#pragma unroll
        for (int s = 0; s < S; ++s) id[s] = lo < hi ? a.ids[in(s) ? mine + 64 * s : lo] : 0;
        for (int b = tid; b < pitch * W / 2; b += kThreads) reinterpret_cast<u32_pair*>(wave_bins)[b] = 0;
        if (MANY && p0 == lo) {
            // bins of all workgroups, and of those before this one: parts of the workgroups side by side
            for (int b = tid; b < bins; b += kThreads) next[b] = all[b] = 0;
            __syncthreads();
            const int parts = bins < kThreads ? kThreads / bins : 1, part = bins < kThreads ? tid / bins : 0;
            if (part < parts)
                for (int b = bins < kThreads ? tid - part * bins : tid; b < bins; b += kThreads) {
                    int32_t total = 0, before = 0;
#pragma unroll 8
                    for (int g = part; g < static_cast<int>(gridDim.x); g += parts) {
                        const int32_t c = a.counts[static_cast<int64_t>(g) * bins + b];
                        total += c;
                        before += g < static_cast<int>(blockIdx.x) ? c : 0;
                    }
                    atomicAdd(&all[b], total);  // whole numbers: the order changes nothing
                    atomicAdd(&next[b], before);
                }
        }
        __syncthreads();
        // Ranks inside the wave's run: the first lane of a bin adds all of its 64 pairs to the wave's counter.
        // The wave's LDS operations keep their order, so the steps' counters come back without a wait
        // between them.
        uint32_t low[S], high[S], old[S];  // lanes with this lane's bin
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint64_t m = __ballot(in(s));
            low[s] = static_cast<uint32_t>(m);
            high[s] = static_cast<uint32_t>(m >> 32);
            id[s] = plan_bin(id[s], a.E);
        }
#pragma unroll
        for (int i = 0; i < kBinBits; ++i)
            if (i < bits) {
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const int bit = (id[s] << (31 - i)) >> 31;  // all ones or zeros
                    const uint64_t ones = __ballot(bit != 0);
                    low[s] &= ~(static_cast<uint32_t>(ones) ^ bit);
                    high[s] &= ~(static_cast<uint32_t>(ones >> 32) ^ bit);
                }
            }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            rank[s] = __builtin_amdgcn_mbcnt_hi(high[s], __builtin_amdgcn_mbcnt_lo(low[s], 0));
            old[s] = 0;
            if (in(s) && rank[s] == 0)
                old[s] = __hip_atomic_fetch_add(own + (id[s] >> 1), static_cast<uint32_t>(__popc(low[s]) + __popc(high[s])) << 16 * (id[s] & 1),
                                                __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int first = low[s] != 0 ? __ffs(low[s]) - 1 : 31 + __ffs(high[s]);
            rank[s] += __shfl(old[s], first) >> 16 * (id[s] & 1) & 0xFFFF;
        }
        __syncthreads();
        // first round: where each bin starts (bins in runs of the workgroup's threads, carried on)
        if (p0 == lo) {
            int32_t carry = 0;
            for (int b0 = 0; b0 < bins; b0 += kThreads) {
                const int b = b0 + tid;
                int32_t n = 0;
                if (b < bins) {
                    if (MANY) n = all[b];
                    else
#pragma unroll
                        for (int w = 0; w < W; ++w) n += wave_bins[w * pitch + b];
                }
                int32_t sum = n;
                for (int d = 1; d < 64; d <<= 1) {
                    const int32_t o = __shfl_up(sum, d);
                    if (lane >= d) sum += o;
                }
                if (lane == 63) wave_total[wave] = sum;
                __syncthreads();
                int32_t start = carry + sum - n;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (w < wave) start += wave_total[w];
                    carry += wave_total[w];
                }
                if (b < bins) {
                    if (blockIdx.x == 0) a.offsets[b] = start;
                    next[b] = start + (MANY ? next[b] : 0);
                }
                __syncthreads();
            }
        }
        for (int b = tid; b < bins; b += kThreads) {
            uint16_t c[W], before = 0;
#pragma unroll
            for (int w = 0; w < W; ++w) c[w] = wave_bins[w * pitch + b];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                wave_bins[w * pitch + b] = before;
                before += c[w];
            }
            all[b] = before;  // of this round
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int64_t p = mine + 64 * s;
            if (!in(s)) continue;
            const int32_t row = next[id[s]] + wave_bins[wave * pitch + id[s]] + rank[s];
            a.slots[p] = id[s] < a.E ? row : -1 - row;
            if (MANY) a.rows[row] = id[s] < a.E ? static_cast<int32_t>(p) : -1;
            else row_pair[row] = id[s] < a.E ? static_cast<uint16_t>(p) : kNoPair;
        }
        __syncthreads();
        if (MANY) {
            for (int b = tid; b < bins; b += kThreads) next[b] += all[b];
        } else {  // rows in order: stores of whole lines (a CU scatters a word a clock)
            for (int r = tid; r < static_cast<int>(a.P); r += kThreads) a.rows[r] = row_pair[r] == kNoPair ? -1 : row_pair[r];
        }
    }
}

// ------------------------------------------------------------------------------------ dispatch
// Outputs that this launch does not read: past the caches, a wave's instruction whole lines.
__device__ __forceinline__ void stream_store(u32x4* p, u32x4 v) { __builtin_nontemporal_store(v, p); }
__device__ __forceinline__ void stream_store(u32x2* p, u32x2 v) { __builtin_nontemporal_store(v, p); }

// One wave takes 1024 columns of a token in two pieces of 512, 8 a lane, so a 1x128 group is a row of
// 16 lanes and every store of a wave is one run of 512 (codes) or 1024 bytes (copy): with 16 columns a
// lane the copy's two stores interleaved, and past the caches half-written lines cost 314 us against
// 184 (8192 tokens x 8, 4096 columns). The token is read and quantized once and written to each of
// its k rows (in row order it would be read k times). A dropped pair's padding row is zeroed by the
// pair's own token, so every row is written exactly once. The scales of a column are 4 bytes a
// token, 32 rows a line: workgroups of one XCD (blockIdx % 8) take consecutive tokens, so that its L2
// collects the lines (without copy 64 -> 53 us, 6.5 TB/s of 0.34 GB; with it 158 us, 5.6 TB/s). Bound
// by the writes.
template <bool VEC>
__global__ __launch_bounds__(64 * kWaves) void dispatch_kernel(const uint16_t* x, int64_t T, int64_t H, int64_t ldx,
                                                               const int32_t* slots, int k, int64_t chunks,
                                                               uint8_t* q, int64_t ldq, float* a_s, uint16_t* copy,
                                                               int64_t ldcopy) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t block = static_cast<int64_t>(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    const int64_t unit = block * kWaves + wave;
    if (unit >= T * chunks) return;
    const int64_t t = unit / chunks, c0 = (unit - t * chunks) * 1024, R = T * k;

    u32x4 w[2];  // 8 bf16 of each piece
    u32x2 code[2];
    float scale[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int64_t col = c0 + 512 * p + lane * 8;
        w[p] = u32x4{};
        if (VEC) {
            if (col < H) w[p] = *reinterpret_cast<const u32x4*>(x + t * ldx + col);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < H) w[p][i >> 1] |= static_cast<uint32_t>(x[t * ldx + col + i]) << (16 * (i & 1));
        }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = max(amax, max(abs_bits(bf16_lo(w[p][i])), abs_bits(bf16_hi(w[p][i]))));
        const GroupScale g = group_scale<false>(__uint_as_float(umax_row16(amax)));
        scale[p] = g.s;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            code[p][i] = encode4_in_range<false>(bf16_lo(w[p][2 * i]) * g.m, bf16_hi(w[p][2 * i]) * g.m,
                                                 bf16_lo(w[p][2 * i + 1]) * g.m, bf16_hi(w[p][2 * i + 1]) * g.m);
    }
    const int32_t mine = lane < k ? slots[t * k + lane] : 0;
    for (int j = 0; j < k; ++j) {
        const int32_t slot = __builtin_amdgcn_readlane(mine, j);
        const int64_t r = slot >= 0 ? slot : -1 - static_cast<int64_t>(slot);
        if (r >= R) continue;
        const uint32_t keep = slot >= 0 ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int64_t col = c0 + 512 * p + lane * 8;
            if (col >= H) continue;
            const u32x2 c = code[p] & keep;
            const u32x4 v = w[p] & keep;
            if (VEC) {
                stream_store(reinterpret_cast<u32x2*>(q + r * ldq + col), c);
                if (copy != nullptr) stream_store(reinterpret_cast<u32x4*>(copy + r * ldcopy + col), v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (col + i >= H) continue;
                    q[r * ldq + col + i] = static_cast<uint8_t>(c[i >> 2] >> (8 * (i & 3)));
                    if (copy != nullptr) copy[r * ldcopy + col + i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
                }
            }
            if ((lane & 15) == 0) a_s[(col >> 7) * R + r] = slot >= 0 ? scale[p] : 0.0f;
        }
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
            stream_store(reinterpret_cast<u32x4*>(p), u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])});
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = to_bf16(f[i]);
    }
}

// Choices whose rows are on the way together (a token's rows lie anywhere: each is a round trip).
constexpr int kBatch = 8;

// One wave takes 512 columns of a token, 8 a lane, and adds its k rows in order of the choices in
// fp32. A dropped pair adds weight * 0: nothing, unless its weight is NaN (a token whose logits
// were), which then shows in the token's output. Bound by the rows' traffic: 8192 tokens x 8 of 4096
// columns 111 us, 5.4 TB/s (138 us with a row at a time).
template <bool VEC>
__global__ __launch_bounds__(64 * kWaves) void combine_kernel(const uint16_t* rows, int64_t R, int64_t ldr,
                                                              const int32_t* slots, const float* weights, int64_t T,
                                                              int k, int64_t H, int64_t chunks, uint16_t* y,
                                                              int64_t ldy) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
    if (unit >= T * chunks) return;
    const int64_t t = unit / chunks, col = (unit - t * chunks) * 512 + lane * 8;
    // lane j: the j-th choice
    const int32_t slot = lane < k ? slots[t * k + lane] : -1;
    const float weight = lane < k ? (weights != nullptr ? weights[t * k + lane] : 1.0f) : 0.0f;
    float acc[8] = {};
    for (int j0 = 0; j0 < k; j0 += kBatch) {
        float f[kBatch][8];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int32_t r = j0 + j < k ? __builtin_amdgcn_readlane(slot, j0 + j) : -1;
            const bool there = r >= 0 && r < R;
            load8<VEC>(rows + (there ? r * ldr : 0) + col, there ? H - col : 0, f[j]);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float w = j0 + j < k ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j0 + j)) : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[j][i], acc[i]);
        }
    }
    store8<VEC>(y + t * ldy + col, H - col, acc);
}

// One workgroup a token: drows[slot] = w dy and dweights = <dy, rows[slot]>, a batch of choices at a
// time: dy is read once a batch, a dot product is one running sum a thread and one reduction. The same
// sizes: 222 us, 5.1 TB/s read and written.
template <bool VEC>
__global__ __launch_bounds__(64 * kWaves) void combine_backward_kernel(const uint16_t* dy, int64_t lddy,
                                                                       const uint16_t* rows, int64_t ldr,
                                                                       const int32_t* slots, const float* weights,
                                                                       int64_t T, int k, int64_t H, uint16_t* drows,
                                                                       int64_t lddr, float* dweights) {
    __shared__ float part[kWaves][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t t = blockIdx.x, R = T * k;
    const int32_t slot = lane < k ? slots[t * k + lane] : -1;
    const float weight = lane < k ? weights[t * k + lane] : 0.0f;
    for (int j0 = 0; j0 < k; j0 += kBatch) {
        float dot[kBatch] = {};
        for (int64_t col = tid * 8; col < H; col += 64 * kWaves * 8) {
            float g[8], f[kBatch][8];
            load8<VEC>(dy + t * lddy + col, H - col, g);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int32_t r = j0 + j < k ? __builtin_amdgcn_readlane(slot, j0 + j) : -1;
                const bool there = r >= 0 && r < R;
                load8<VEC>(rows + (there ? r * ldr : 0) + col, there ? H - col : 0, f[j]);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (j0 + j >= k) continue;
                const int32_t sl = __builtin_amdgcn_readlane(slot, j0 + j);
                const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j0 + j));
                const int64_t r = sl >= 0 ? sl : -1 - static_cast<int64_t>(sl);
                if (r >= R) continue;
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d[i] = sl >= 0 ? w * g[i] : 0.0f;
                    if (sl >= 0) dot[j] = fmaf(g[i], f[j][i], dot[j]);
                }
                store8<VEC>(drows + r * lddr + col, H - col, d);
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float sum = wave_sum(dot[j]);
            if (lane == 0 && j0 + j < k) part[wave][j0 + j] = sum;
        }
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
static hipError_t route_wide(const LT* logits, const RouteArgs& a, hipStream_t stream) {
    const int64_t blocks = (a.T + kWaves - 1) / kWaves;
    const size_t lds = a.groups > 1 ? sizeof(double) * kWaves * (a.E + a.groups) : 0;
    route_wide_kernel<LT, V><<<dim3(static_cast<unsigned>(blocks)), 64 * kWaves, lds, stream>>>(logits, a);
    return hipGetLastError();
}

template <typename LT, int V, int L>
static hipError_t route_teams(const LT* logits, RouteArgs a, hipStream_t stream) {
    const int runs = a.size / V;
    a.shift = a.size % V == 0 && (runs & (runs - 1)) == 0 && runs <= 16 ? __builtin_ctz(runs) : -1;
    const int64_t per = kWaves * (64 / L), blocks = (a.T + per - 1) / per;
    const size_t lds = sizeof(double) * per * a.groups * ((a.size | 1) + 1);
    const dim3 grid(static_cast<unsigned>(blocks));
    if (a.bias == nullptr)
        route_kernel<LT, V, L, kKeyLogit><<<grid, 64 * kWaves, lds, stream>>>(logits, a);
    else if (a.softmax)
        route_kernel<LT, V, L, kKeySoftmax><<<grid, 64 * kWaves, lds, stream>>>(logits, a);
    else
        route_kernel<LT, V, L, kKeySigmoid><<<grid, 64 * kWaves, lds, stream>>>(logits, a);
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

template <typename LT, int V>
static hipError_t route_backward_team(const LT* logits, int64_t T, int E, int64_t ld, const RouteRule& r, const int32_t* ids,
                                      const float* dweights, LT* dlogits, int64_t ldd, hipStream_t stream) {
    const int64_t blocks = (T + 4 * kWaves - 1) / (4 * kWaves);
    route_backward_team_kernel<LT, V><<<dim3(static_cast<unsigned>(blocks)), 64 * kWaves, 0, stream>>>(
        logits, T, E, ld, r.softmax, r.k, r.renormalize, r.scale, ids, dweights, dlogits, ldd, rows16(logits, ld * sizeof(LT)),
        rows16(dlogits, ldd * sizeof(LT)));
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
static hipError_t route_t(const LT* logits, const RouteArgs& a, hipStream_t stream) {
    const int E = a.E;
    const bool wide = a.k > 16 || a.groups > (E <= 256 ? 16 : 64);
    if (wide) {
#define CALL(V) route_wide<LT, V>(logits, a, stream)
        return BSFP8_BY_EXPERTS(CALL);
#undef CALL
    }
    if (E <= 16) return route_teams<LT, 1, 16>(logits, a, stream);
    if (E <= 64) return route_teams<LT, 4, 16>(logits, a, stream);
    if (E <= 128) return route_teams<LT, 8, 16>(logits, a, stream);
    if (E <= 256) return route_teams<LT, 16, 16>(logits, a, stream);
    if (E <= 512) return route_teams<LT, 8, 64>(logits, a, stream);
    return route_teams<LT, 16, 64>(logits, a, stream);
}

template <typename LT>
static hipError_t route_backward_t(const void* logits, int64_t T, int E, int64_t ld, const RouteRule& r, const int32_t* ids,
                                   const float* dweights, void* dlogits, int64_t ldd, hipStream_t stream) {
    if (r.k <= 16 && E <= 256) {
#define CALL(V) route_backward_team<LT, V>(static_cast<const LT*>(logits), T, E, ld, r, ids, dweights, static_cast<LT*>(dlogits), ldd, stream)
        return E <= 16 ? CALL(1) : E <= 64 ? CALL(4) : E <= 128 ? CALL(8) : CALL(16);
#undef CALL
    }
#define CALL(V) route_backward_v<LT, V>(static_cast<const LT*>(logits), T, E, ld, r, ids, dweights, static_cast<LT*>(dlogits), ldd, stream)
    return BSFP8_BY_EXPERTS(CALL);
#undef CALL
}

hipError_t launch_route(const void* logits, bool f32, int64_t T, int E, int64_t ld, const RouteRule& r, const float* bias,
                        float* weights, int32_t* ids, hipStream_t stream) {
    const RouteArgs a{T, E, ld, bias, r.softmax, r.k, r.groups, r.top_groups, r.renormalize, r.scale, weights, ids,
                      rows16(logits, ld * (f32 ? 4 : 2)), rows16(bias, 0), E / r.groups, -1};
    return f32 ? route_t(static_cast<const float*>(logits), a, stream) : route_t(static_cast<const uint16_t*>(logits), a, stream);
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
        plan_count_kernel<<<dim3(static_cast<unsigned>(blocks)), kCountThreads, sizeof(int32_t) * (E + 1), stream>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const int waves = sched::plan_waves(P), steps = sched::plan_steps(P);
    const size_t lds = (E + 1) * 2 * sizeof(int32_t) + (E + 2) / 2 * 2 * waves * sizeof(uint16_t);
    const dim3 grid(static_cast<unsigned>(blocks));
    if (blocks > 1)
        plan_kernel<8, 4, true><<<grid, 64 * 8, lds, stream>>>(a);
    else if (steps == 8)
        plan_kernel<16, 8, false><<<grid, 64 * 16, lds, stream>>>(a);
    else if (waves == 16)
        plan_kernel<16, 4, false><<<grid, 64 * 16, lds, stream>>>(a);
    else if (steps == 1)
        plan_kernel<8, 1, false><<<grid, 64 * 8, lds, stream>>>(a);
    else
        plan_kernel<8, 4, false><<<grid, 64 * 8, lds, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_dispatch(const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const int32_t* slots, int k, uint8_t* q,
                           int64_t ldq, float* a_s, uint16_t* copy, int64_t ldcopy, hipStream_t stream) {
    const int64_t chunks = (H + 1023) / 1024, blocks = (T * chunks + 8 * kWaves - 1) / (8 * kWaves) * 8;
    const bool vec = H % 8 == 0 && rows16(x, 2 * ldx) && reinterpret_cast<uintptr_t>(q) % 8 == 0 && ldq % 8 == 0 &&
                     (copy == nullptr || rows16(copy, 2 * ldcopy));
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
