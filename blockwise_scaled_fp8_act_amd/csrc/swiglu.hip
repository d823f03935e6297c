// gfx950 gated activation with 8-bit codes, and its gradient: of gu [T, 2 F], gate g and up u,
//   v = g sig(g) u,   dg = dy u sig(g) (1 + g (1 - sig(g))),   du = dy g sig(g),   sig(g) = 1 / (1 + exp(-g)),
// formed in fp32 and written as e4m3 codes in 1x128 groups (for a training step in both groupings), as int8
// rows, or in bf16. Bound by the memory traffic: the inputs are read once, the values never leave the
// registers in a wider type unless they are asked for.
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

// Where |g| <= 80 nothing leaves fp32's ordinary range: with t = exp(-g), sig = 1 / (1 + t) and
// 1 - sig = t sig, neither with cancellation. Beyond, sig is 1 to fp32, or exp(g) to 2^-115: that leaves
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

// dg = dy u sig (1 + g (1 - sig)), du = dy g sig
__device__ __forceinline__ void swiglu_grad8(const float (&dy)[8], const float (&g)[8], const float (&u)[8], float (&dg)[8], float (&du)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = exp_of(-g[j]), sig = reciprocal(1.0f + t);
        dg[j] = (u[j] * (sig * fmaf(g[j], t * sig, 1.0f))) * dy[j];
        du[j] = (g[j] * sig) * dy[j];
    }
    if (__builtin_expect(any_far(g), 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (fabsf(g[j]) > kFar) {
                dg[j] = g[j] > 0.0f ? u[j] * dy[j] : far_product(1.0f + g[j], u[j], dy[j], g[j]);
                du[j] = g[j] > 0.0f ? g[j] * dy[j] : far_product(g[j], dy[j], 1.0f, g[j]);
            }
    }
}

// A row of TPR threads, NC pieces of 8 columns each.
template <int TPR, int NC>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, int64_t per_xcd, RowCodes out) {
    __shared__ uint32_t part_max[kWaves];
    const int tid = threadIdx.x % TPR;
    const int64_t row = xcd_block(blockIdx.x, per_xcd) * (kThreads / TPR) + threadIdx.x / TPR;
    if (row >= T) return;
    rc_u32x4 g[NC], u[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = row * ldgu + (c < F ? c : 0);
        g[i] = *reinterpret_cast<const rc_u32x4*>(gu + at);
        u[i] = *reinterpret_cast<const rc_u32x4*>(gu + at + F);
    }
    float v[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const bool in = 8 * (static_cast<int64_t>(i) * TPR + tid) < F;
        float gf[8], uf[8];
        unpack8(g[i], gf);
        unpack8(u[i], uf);
        swiglu8(gf, uf, v[i]);
        if (!in)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
    emit_row<TPR, NC>(out, row, T, F, tid, v, part_max);
}

__global__ __launch_bounds__(kThreads) void swiglu_any_kernel(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, RowCodes out) {
    __shared__ uint32_t part_max[kWaves];
    const int64_t row = blockIdx.x;
    const uint16_t* p = gu + row * ldgu;
    emit_row_any<kWaves>(out, row, T, F, [&](int64_t c) { return swiglu(bf16_to_f32(p[c]), bf16_to_f32(p[F + c])); }, part_max);
}

// Eight columns of a row of a [*, ld] bf16 tensor; zero outside.
template <bool VEC, bool ONCE = false>
__device__ __forceinline__ void load_cols(const uint16_t* p, int64_t ld, int64_t row, int64_t T, int64_t c, int64_t C, float (&f)[8]) {
    const bool in = row < T;
    if (VEC) {
        load8_of<false, ONCE>(p, in && c < C ? row * ld + c : 0, f);
        if (!(in && c < C))
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = in && c + j < C ? bf16_to_f32(p[row * ld + c + j]) : 0.0f;
    }
}

template <bool FNUZ, bool VEC>
__global__ __launch_bounds__(kTileThreads) void swiglu_dual_kernel(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    float v[kTileRows][8], u[kTileRows][8];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        load_cols<VEC>(gu, ldgu, row + i, T, c, F, v[i]);
        load_cols<VEC>(gu + F, ldgu, row + i, T, c, F, u[i]);
    }
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        float w[8];
        swiglu8(v[i], u[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = w[j];
    }
    emit_tile<FNUZ, true, VEC, VEC>(out, r0, c0, T, F, v, lds);
}

// The gradient's tile of the columns c0 .. c0 + 127 of [T, 2 F], which may hold columns of both halves.
template <bool FNUZ>
__global__ __launch_bounds__(kTileThreads) void swiglu_backward_dual_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu,
                                                                           int64_t T, int64_t F, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    float v[kTileRows][8];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        float d[8], g[8], u[8], dg[8], du[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t at = c + j, f = at < F ? at : at - F;
            const bool in = row + i < T && at < 2 * F;
            const uint16_t* p = gu + (row + i) * ldgu + f;
            d[j] = in ? bf16_to_f32(dy[(row + i) * lddy + f]) : 0.0f;
            g[j] = in ? bf16_to_f32(p[0]) : 0.0f;
            u[j] = in ? bf16_to_f32(p[F]) : 0.0f;
        }
        swiglu_grad8(d, g, u, dg, du);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = c + j < F ? dg[j] : du[j];
    }
    emit_tile<FNUZ, true, false, false>(out, r0, c0, T, 2 * F, v, lds);
}

// Whole tiles of both halves (F a multiple of 128): gate and up gradients of the same inputs.
template <bool FNUZ>
__global__ __launch_bounds__(kTileThreads) void swiglu_backward_tiles_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu,
                                                                            int64_t T, int64_t F, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    float dg[kTileRows][8], du[kTileRows][8];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        float d[8], g[8], u[8];
        load_cols<true>(dy, lddy, row + i, T, c, F, d);
        load_cols<true>(gu, ldgu, row + i, T, c, F, g);
        load_cols<true>(gu + F, ldgu, row + i, T, c, F, u);
        swiglu_grad8(d, g, u, dg[i], du[i]);
    }
    emit_tile<FNUZ, true, true, true>(out, r0, c0, T, 2 * F, dg, lds);
    emit_tile<FNUZ, true, true, true, true>(out, r0, c0 + F, T, 2 * F, du, lds);
}

template <bool VEC>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu, int64_t T,
                                                                  int64_t F, int64_t chunks, uint16_t* dgu, int64_t lddgu) {
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    const int64_t row = unit / chunks, c = (unit - row * chunks) * 512 + (threadIdx.x & 63) * 8;
    if (row >= T || c >= F) return;
    float d[8], g[8], u[8], dg[8], du[8];
    load_cols<VEC>(dy, lddy, row, T, c, F, d);
    load_cols<VEC>(gu, ldgu, row, T, c, F, g);
    load_cols<VEC>(gu + F, ldgu, row, T, c, F, u);
    swiglu_grad8(d, g, u, dg, du);
    uint16_t* p = dgu + row * lddgu + c;
    if (VEC) {
        store8_of<false>(p, 0, dg);
        store8_of<false>(p, F, du);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < F) {
                p[j] = to_bf16_bits(dg[j]);
                p[F + j] = to_bf16_bits(du[j]);
            }
    }
}

bool rows16(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bytes % 16 == 0; }
bool rows8(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && bytes % 8 == 0; }
bool tiles_vec(const TileCodes& o, int64_t T) { return rows8(o.q, o.ldq) && T % 16 == 0 && rows16(o.qT, o.ldqT); }
dim3 tiles(int64_t T, int64_t C) {
    return dim3(static_cast<unsigned>((C + kGroup - 1) / kGroup), static_cast<unsigned>((T + kGroup - 1) / kGroup));
}

}  // namespace

hipError_t launch_swiglu(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, const RowCodes& out, hipStream_t stream) {
    const bool vec = F % 8 == 0 && F <= sched::kRowMax && rows16(gu, 2 * ldgu) && (out.codes == kCodesNone || rows8(out.q, out.ldq)) &&
                     (out.y == nullptr || rows16(out.y, 2 * out.ldy));
    if (!vec) {
        swiglu_any_kernel<<<static_cast<unsigned>(T), kThreads, 0, stream>>>(gu, ldgu, T, F, out);
        return hipGetLastError();
    }
    const bool wave = F <= sched::kRowWaveMax;
    const int64_t blocks = wave ? (T + kWaves - 1) / kWaves : T, per_xcd = (blocks + kXcds - 1) / kXcds;
    const unsigned grid = static_cast<unsigned>(per_xcd * kXcds);
#define BSFP8_SWIGLU(TPR, NC) swiglu_kernel<TPR, NC><<<grid, kThreads, 0, stream>>>(gu, ldgu, T, F, per_xcd, out)
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
    return hipGetLastError();
}

hipError_t launch_swiglu_dual(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, const TileCodes& out, bool fnuz,
                              hipStream_t stream) {
    const bool vec = F % 8 == 0 && rows16(gu, 2 * ldgu) && tiles_vec(out, T);
    const dim3 grid = tiles(T, F);
    if (fnuz && vec) swiglu_dual_kernel<true, true><<<grid, kTileThreads, 0, stream>>>(gu, ldgu, T, F, out);
    else if (fnuz) swiglu_dual_kernel<true, false><<<grid, kTileThreads, 0, stream>>>(gu, ldgu, T, F, out);
    else if (vec) swiglu_dual_kernel<false, true><<<grid, kTileThreads, 0, stream>>>(gu, ldgu, T, F, out);
    else swiglu_dual_kernel<false, false><<<grid, kTileThreads, 0, stream>>>(gu, ldgu, T, F, out);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward_dual(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F,
                                       const TileCodes& out, bool fnuz, hipStream_t stream) {
    if (F % kGroup == 0 && rows16(dy, 2 * lddy) && rows16(gu, 2 * ldgu) && tiles_vec(out, T)) {
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
    if (F % 8 == 0 && rows16(dy, 2 * lddy) && rows16(gu, 2 * ldgu) && rows16(dgu, 2 * lddgu))
        swiglu_backward_kernel<true><<<grid, kThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, chunks, dgu, lddgu);
    else
        swiglu_backward_kernel<false><<<grid, kThreads, 0, stream>>>(dy, lddy, gu, ldgu, T, F, chunks, dgu, lddgu);
    return hipGetLastError();
}

}  // namespace bsfp8
