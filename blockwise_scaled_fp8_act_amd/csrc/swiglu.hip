// gfx950 gated activation with 8-bit codes, and its gradient: of gu [T, 2 F], gate g and up u,
//   v = g sig(g) u,   dg = dy u sig(g) (1 + g (1 - sig(g))),   du = dy g sig(g),   sig(g) = 1 / (1 + exp(-g)),
// formed in fp32 and written as e4m3 codes in 1x128 groups (for a training step in both groupings), as int8
// rows, or in bf16. Bound by the memory traffic: the inputs are read once, the values never leave the
// registers in a wider type unless they are asked for. Measured: 8192 x 4096 in both groupings 36 to 44 us (4.6 to 5.6 TB/s),
// the gradient in both 66 to 73 (4.6 to 5.1), in bf16 56 (6.0); 64 x 5120 rows 3.7, as int8 3.6 (16384 x 5120 81, 5.2 TB/s),
// 1000 x 1408 with a bf16 copy 4.2.
#include "row_codes.hpp"
#include "schedule.hpp"
#include "tile_codes.hpp"

namespace bsfp8 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// exp(x): x log2(e) in two parts, since rounding the product alone costs |x| 2^-24.
__device__ __forceinline__ float exp_of(float x) {
    const float hi = x * 1.44269504f, lo = fmaf(x, 1.92596e-8f, fmaf(x, 1.44269504f, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    return fmaf(e * 0.693147181f, lo, e);
}

// 1 / d for ordinary d, the instruction's result (within an ulp) corrected by one step of Newton's method.
__device__ __forceinline__ float reciprocal(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return fmaf(fmaf(-d, r, 1.0f), r, r);
}

// Where |g| <= 80 neither sig = 1 / (1 + t) with t = exp(-g) nor 1 - sig = t sig nor g sig leaves fp32's ordinary range,
// and none is formed with cancellation. Beyond, sig is 1 to fp32, or exp(g) to 2^-115: that leaves
// fp32's ordinary range while g sig u need not (u is as large as 3e38), so it is taken in 64 bits, from the
// fourth power of exp(g / 4). Eight values share the test for it.
constexpr float kFar = 80.0f;
__device__ __forceinline__ float far_product(float a, float b, float c, float g) {
    double e = exp_of(0.25f * fmaxf(g, -800.0f));
    e *= e;
    return static_cast<float>(static_cast<double>(a) * b * c * (e * e));
}
__device__ __forceinline__ bool any_far(const float (&g)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(g[j]));
    return top > kFar;
}

// v = g sig(g) u
__device__ __forceinline__ void swiglu8(const float (&g)[8], const float (&u)[8], float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (g[j] * reciprocal(1.0f + exp_of(-g[j]))) * u[j];
    if (__builtin_expect(any_far(g), 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (fabsf(g[j]) > kFar) v[j] = g[j] > 0.0f ? g[j] * u[j] : far_product(g[j], u[j], 1.0f, g[j]);
    }
}
__device__ __forceinline__ float swiglu(float g, float u) {
    const float g8[8] = {g}, u8[8] = {u};
    float v[8];
    swiglu8(g8, u8, v);
    return v[0];
}

// dg = (dy u) d with d = sig (1 + g (1 - sig)), |d| < 1.1, and du = (g sig) dy. dy u of two bf16 is whole in fp32 but at its
// ends: below 2^-126 it is off by 2^-150, which d does not enlarge; beyond kHuge, where it may pass fp32 while dg need
// not, dg is formed in 64 bits (with u sig (1 + g (1 - sig)) first, u of 3.2e38 and dy of 0.01 gave an infinity, and
// its group's scale with it, and u of 1e-11 at a gate of -79 lost all but 27 steps before a large dy).
constexpr float kHuge = 0x1p127f;
__device__ __forceinline__ float gate_factor(float g, float& sig) {
    const float t = exp_of(-g);
    sig = reciprocal(1.0f + t);
    return sig * fmaf(g, t * sig, 1.0f);
}
__device__ __forceinline__ void swiglu_grad8(const float (&dy)[8], const float (&g)[8], const float (&u)[8], float (&dg)[8], float (&du)[8]) {
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float sig;
        const float d = gate_factor(g[j], sig);
        const float p = dy[j] * u[j];
        most = fmaxf(most, fabsf(p));
        dg[j] = p * d;
        du[j] = (g[j] * sig) * dy[j];
    }
    if (__builtin_expect(any_far(g) || most > kHuge, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (fabsf(g[j]) > kFar) {
                dg[j] = g[j] > 0.0f ? dy[j] * u[j] : far_product(1.0f + g[j], u[j], dy[j], g[j]);
                du[j] = g[j] > 0.0f ? g[j] * dy[j] : far_product(g[j], dy[j], 1.0f, g[j]);
            } else if (fabsf(dy[j] * u[j]) > kHuge) {
                float sig;
                dg[j] = static_cast<float>(static_cast<double>(gate_factor(g[j], sig)) * u[j] * dy[j]);
            }
        }
    }
}

// A row of TPR threads, NC pieces of 8 columns each. ANY: rows that begin anywhere, of any length; without it all rows in
// 16-byte pieces (codes in 8-byte ones).
template <int TPR, int NC, bool ANY>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, int64_t per_xcd, RowCodes out) {
    __shared__ uint32_t part_max[kWaves];
    const int tid = threadIdx.x % TPR;
    const int64_t row = xcd_block(blockIdx.x, per_xcd) * (kThreads / TPR) + threadIdx.x / TPR;
    if (row >= T) return;
    rc_u32x4 g[NC], u[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = row * ldgu + (c < F ? c : 0);
        g[i] = load8_bf16<false, ANY>(gu + at, F - c);
        u[i] = load8_bf16<false, ANY>(gu + at + F, F - c);
    }
    float v[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float gf[8], uf[8];
        unpack8(g[i], gf);
        unpack8(u[i], uf);
        swiglu8(gf, uf, v[i]);  // of zeros: zero
        if (!ANY && 8 * (static_cast<int64_t>(i) * TPR + tid) >= F)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
    emit_row<TPR, NC, ANY>(out, row, T, F, tid, v, part_max);
}

// Longer rows.
__global__ __launch_bounds__(kThreads) void swiglu_long_kernel(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, RowCodes out) {
    __shared__ uint32_t part_max[kWaves];
    const int64_t row = blockIdx.x;
    const uint16_t* p = gu + row * ldgu;
    emit_row_any<kWaves>(out, row, T, F, [&](int64_t c) { return swiglu(bf16_to_f32(p[c]), bf16_to_f32(p[F + c])); }, part_max);
}

template <bool FNUZ, bool WHOLE>
__global__ __launch_bounds__(kTileThreads) void swiglu_dual_kernel(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    rc_u32x4 g[kTileRows], u[kTileRows];
    load_tile<WHOLE>(gu, ldgu, row, T, c0, c, F, g);
    load_tile<WHOLE>(gu + F, ldgu, row, T, c0, c, F, u);
    float v[kTileRows][8];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        float gf[8], uf[8];
        unpack8(g[i], gf);
        unpack8(u[i], uf);
        swiglu8(gf, uf, v[i]);
    }
    emit_tile<FNUZ, true>(out, r0, c0, T, F, v, lds);
}

// The gradient's tile of the columns c0 .. c0 + 127 of [T, 2 F]: of one half, or of both (a group of 128 may lie in
// both, and so may a thread's eight columns).
template <bool FNUZ>
__global__ __launch_bounds__(kTileThreads, 4) void swiglu_backward_dual_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu,
                                                                              int64_t T, int64_t F, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    float v[kTileRows][8], dg[8], du[8];
    if (c0 + kGroup <= F || (c0 >= F && c0 + kGroup <= 2 * F)) {
        const int64_t half = c0 < F ? 0 : F;
        rc_u32x4 d[kTileRows], g[kTileRows], u[kTileRows];
        load_tile<true>(dy, lddy, row, T, c0 - half, c - half, F, d);
        load_tile<true>(gu, ldgu, row, T, c0 - half, c - half, F, g);
        load_tile<true>(gu + F, ldgu, row, T, c0 - half, c - half, F, u);
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            float df[8], gf[8], uf[8];
            unpack8(d[i], df);
            unpack8(g[i], gf);
            unpack8(u[i], uf);
            swiglu_grad8(df, gf, uf, dg, du);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = half == 0 ? dg[j] : du[j];
        }
    } else {
        const bool both = c < F && c + 8 > F;
        const int64_t f = c < F ? c : c - F;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            float d[8], g[8], u[8];
            const int64_t n = row + i < T ? F - f : 0;  // of the half, from f on
            load8_of<false, false, true>(dy, (row + i) * lddy + f, d, n);
            load8_of<false, false, true>(gu, (row + i) * ldgu + f, g, n);
            load8_of<false, false, true>(gu + F, (row + i) * ldgu + f, u, n);
            if (both && n > 0) {  // the rest from the other half's beginning
#pragma unroll
                for (int j = 1; j < 8; ++j) {
                    const int64_t k = c + j - F;
                    if (k < 0 || k >= F) continue;
                    d[j] = bf16_to_f32(dy[(row + i) * lddy + k]);
                    g[j] = bf16_to_f32(gu[(row + i) * ldgu + k]);
                    u[j] = bf16_to_f32(gu[(row + i) * ldgu + F + k]);
                }
            }
            swiglu_grad8(d, g, u, dg, du);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = c + j < F ? dg[j] : du[j];
        }
    }
    emit_tile<FNUZ, true>(out, r0, c0, T, 2 * F, v, lds);
}

// Whole tiles of both halves (F a multiple of 128): gate and up gradients of the same inputs.
template <bool FNUZ>
__global__ __launch_bounds__(kTileThreads) void swiglu_backward_tiles_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu,
                                                                            int64_t T, int64_t F, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    rc_u32x4 d[kTileRows], g[kTileRows], u[kTileRows];
    load_tile<true>(dy, lddy, row, T, c0, c, F, d);
    load_tile<true>(gu, ldgu, row, T, c0, c, F, g);
    load_tile<true>(gu + F, ldgu, row, T, c0, c, F, u);
    float dg[kTileRows][8], du[kTileRows][8];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        float df[8], gf[8], uf[8];
        unpack8(d[i], df);
        unpack8(g[i], gf);
        unpack8(u[i], uf);
        swiglu_grad8(df, gf, uf, dg[i], du[i]);
    }
    emit_tile<FNUZ, true>(out, r0, c0, T, 2 * F, dg, lds);
    emit_tile<FNUZ, true, true>(out, r0, c0 + F, T, 2 * F, du, lds);
}

template <bool ANY>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu, int64_t T,
                                                                  int64_t F, int64_t chunks, uint16_t* dgu, int64_t lddgu) {
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    const int64_t row = unit / chunks, c = (unit - row * chunks) * 512 + (threadIdx.x & 63) * 8;
    if (row >= T || c >= F) return;
    float d[8], g[8], u[8], dg[8], du[8];
    load8_of<false, false, ANY>(dy, row * lddy + c, d, F - c);
    load8_of<false, false, ANY>(gu, row * ldgu + c, g, F - c);
    load8_of<false, false, ANY>(gu + F, row * ldgu + c, u, F - c);
    swiglu_grad8(d, g, u, dg, du);
    store8_of<false, ANY>(dgu, row * lddgu + c, dg, F - c);
    store8_of<false, ANY>(dgu + F, row * lddgu + c, du, F - c);
}

dim3 tiles(int64_t T, int64_t C) {
    return dim3(static_cast<unsigned>((C + kGroup - 1) / kGroup), static_cast<unsigned>((T + kGroup - 1) / kGroup));
}

template <bool ANY>
void launch_rows(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, const RowCodes& out, hipStream_t stream) {
    const bool wave = F <= sched::kRowWaveMax;
    const int64_t blocks = wave ? (T + kWaves - 1) / kWaves : T, per_xcd = (blocks + kXcds - 1) / kXcds;
    const unsigned grid = static_cast<unsigned>(per_xcd * kXcds);
#define BSFP8_SWIGLU(TPR, NC) swiglu_kernel<TPR, NC, ANY><<<grid, kThreads, 0, stream>>>(gu, ldgu, T, F, per_xcd, out)
    if (wave) {
        if (F <= 512) BSFP8_SWIGLU(64, 1);
        else BSFP8_SWIGLU(64, 2);
    } else {
        switch ((F + 2047) / 2048) {
            case 1: BSFP8_SWIGLU(256, 1); break;
            case 2: BSFP8_SWIGLU(256, 2); break;
            case 3: BSFP8_SWIGLU(256, 3); break;
            case 4: BSFP8_SWIGLU(256, 4); break;
            case 5: case 6: BSFP8_SWIGLU(256, 6); break;
            default: BSFP8_SWIGLU(256, 8); break;
        }
    }
#undef BSFP8_SWIGLU
}

}  // namespace

hipError_t launch_swiglu(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, const RowCodes& out, hipStream_t stream) {
    if (F > sched::kRowMax) swiglu_long_kernel<<<static_cast<unsigned>(T), kThreads, 0, stream>>>(gu, ldgu, T, F, out);
    else if (F % 8 == 0 && rows16(gu, 2 * ldgu) && whole_codes(out)) launch_rows<false>(gu, ldgu, T, F, out, stream);
    else launch_rows<true>(gu, ldgu, T, F, out, stream);
    return hipGetLastError();
}

hipError_t launch_swiglu_dual(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, const TileCodes& out, bool fnuz,
                              hipStream_t stream) {
    const auto go = [&](auto fz, auto whole) {
        swiglu_dual_kernel<decltype(fz)::value, decltype(whole)::value><<<tiles(T, F), kTileThreads, 0, stream>>>(gu, ldgu, T, F, out);
    };
    if (F % kGroup == 0) fnuz ? go(std::true_type{}, std::true_type{}) : go(std::false_type{}, std::true_type{});
    else fnuz ? go(std::true_type{}, std::false_type{}) : go(std::false_type{}, std::false_type{});
    return hipGetLastError();
}

hipError_t launch_swiglu_backward_dual(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F,
                                       const TileCodes& out, bool fnuz, hipStream_t stream) {
    if (F % kGroup == 0) {
        if (fnuz) swiglu_backward_tiles_kernel<true><<<tiles(T, F), kTileThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, out);
        else swiglu_backward_tiles_kernel<false><<<tiles(T, F), kTileThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, out);
    } else if (fnuz) {
        swiglu_backward_dual_kernel<true><<<tiles(T, 2 * F), kTileThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, out);
    } else {
        swiglu_backward_dual_kernel<false><<<tiles(T, 2 * F), kTileThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, out);
    }
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F,
                                  uint16_t* dgu, int64_t lddgu, hipStream_t stream) {
    const int64_t chunks = (F + 511) / 512, blocks = (T * chunks + kWaves - 1) / kWaves;
    const unsigned grid = static_cast<unsigned>(blocks);
    // both halves on whole pieces: F a multiple of 8
    if (F % 8 == 0 && rows16(dy, 2 * lddy) && rows16(gu, 2 * ldgu) && rows16(dgu, 2 * lddgu))
        swiglu_backward_kernel<false><<<grid, kThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, chunks, dgu, lddgu);
    else
        swiglu_backward_kernel<true><<<grid, kThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, chunks, dgu, lddgu);
    return hipGetLastError();
}

}  // namespace bsfp8
