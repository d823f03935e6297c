// Device helper of the operators that write their values in both groupings of a training step: the codes
// of a tile of 128 rows and 128 columns held in registers, row-wise in 1x128 groups and, transposed,
// column-wise in 128x1 groups. A tile holds exactly one group of every row and of every column.
#pragma once

#include "row_codes.hpp"

namespace bsfp8 {

constexpr int kTileThreads = 512;
constexpr int kTileRows = 4;  // a thread's consecutive rows, of 8 columns: 16 lanes make a row of the tile

// The transposed code tile and, before it in the same place, the column maxima of the 32 row groups.
struct TileLds {
    union {
        uint4 tile[kGroup * 8];  // [column][8 chunks of 16 rows], the chunk swizzled by the column's eights
        uint32_t red[32][kGroup + 1];
    };
    float mult[kGroup];
};

// The value of lane l of the 16 lanes of a DPP row, in all of them.
template <int L>
__device__ __forceinline__ float row16_lane(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), 0x150 + L, 0xF, 0xF, false));
}

// Eight columns from c = c0 + 8 (t % 16) on of the rows row + i, row = r0 + 4 (t / 16), of a [T, C] tensor (row stride
// ld); zero outside. WHOLE: C is a multiple of 128, so there is no branch, at whose end all loads would be waited for (the
// gradient's three inputs, 8192 x 4096: 70.6 -> 65.6 us).
template <bool WHOLE>
__device__ __forceinline__ void load_tile(const uint16_t* p, int64_t ld, int64_t row, int64_t T, int64_t c0, int64_t c, int64_t C,
                                          rc_u32x4 (&w)[kTileRows]) {
    if (WHOLE || c0 + kGroup <= C) {
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) w[i] = load8_bf16<false, true>(p + (row + i < T ? row + i : 0) * ld + c);
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) w[i] = row + i < T ? w[i] : rc_u32x4{0, 0, 0, 0};
    } else {
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) w[i] = load8_bf16<false, true>(p + (row + i) * ld + c, row + i < T ? C - c : 0);
    }
}
template <bool WHOLE>
__device__ __forceinline__ void load_tile(const float* p, int64_t ld, int64_t row, int64_t T, int64_t c0, int64_t c, int64_t C,
                                          float (&v)[kTileRows][8]) {
    if (WHOLE || c0 + kGroup <= C) {
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) load8_of<true, false, true>(p, (row + i < T ? row + i : 0) * ld + c, v[i]);
#pragma unroll
        for (int i = 0; i < kTileRows; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = row + i < T ? v[i][j] : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) load8_of<true, false, true>(p, (row + i) * ld + c, v[i], row + i < T ? C - c : 0);
    }
}

// v[i][j]: row r0 + 4 (t / 16) + i, column c0 + 8 (t % 16) + j; zero outside the [T, C] tensor. Code rows
// may begin anywhere: pieces of 8 and 16 bytes go to any address in one store (rows of qT are T bytes long by default, and
// T is what a batch happens to hold: gated activation of 8191 x 4096 46 us, byte by byte 143, its gradient 67 and 302;
// 8192 rows 44 and 65). Every thread of the workgroup calls it, with AGAIN for a second tile through the same LDS.
template <bool FNUZ, bool ROWS, bool AGAIN = false>
__device__ __forceinline__ void emit_tile(const TileCodes& out, int64_t r0, int64_t c0, int64_t T, int64_t C, const float (&v)[kTileRows][8],
                                          TileLds& lds) {
    const int t = threadIdx.x, cg = t & 15, rg = t >> 4;
    const int64_t c = c0 + cg * 8;
    const auto encode = [](float a, float b, float d, float e) { return encode4_in_range<FNUZ>(a, b, d, e); };

    // column maxima of this thread's rows, then of all in LDS
    if (AGAIN) __syncthreads();  // every thread has read the tile before
    uint32_t mag[kTileRows][8];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) mag[i][j] = abs_bits(v[i][j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) lds.red[rg][cg * 8 + j] = max(max(mag[0][j], mag[1][j]), max(mag[2][j], mag[3][j]));
    if (ROWS) {
        // lane l of a row's 16 forms the scale pair of row l % 4 (two divisions), and all take each row's
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            uint32_t am = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) am = max(am, mag[i][j]);
            am = umax_row16(am);
            mine = (cg & 3) == i ? am : mine;
        }
        const GroupScale own = fp8_scale<FNUZ>(mine);
        const GroupScale g[kTileRows] = {{row16_lane<0>(own.s), row16_lane<0>(own.m)}, {row16_lane<1>(own.s), row16_lane<1>(own.m)},
                                         {row16_lane<2>(own.s), row16_lane<2>(own.m)}, {row16_lane<3>(own.s), row16_lane<3>(own.m)}};
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            const int64_t r = r0 + rg * kTileRows + i;
            if (r >= T) continue;
            const uint32_t w0 = encode(v[i][0] * g[i].m, v[i][1] * g[i].m, v[i][2] * g[i].m, v[i][3] * g[i].m);
            const uint32_t w1 = encode(v[i][4] * g[i].m, v[i][5] * g[i].m, v[i][6] * g[i].m, v[i][7] * g[i].m);
            if (c < C) store8_codes<true>(out.q + r * out.ldq + c, make_uint2(w0, w1), C - c);
            if (cg == 0) out.a_s[c0 / kGroup * T + r] = g[i].s;
        }
    }
    __syncthreads();
    if (t < kGroup) {
        uint32_t am = 0;
#pragma unroll 8
        for (int r = 0; r < 32; ++r) am = max(am, lds.red[r][t]);
        const GroupScale g = fp8_scale<FNUZ>(am);
        lds.mult[t] = g.m;
        if (c0 + t < C) out.s[r0 / kGroup * C + c0 + t] = g.s;
    }
    __syncthreads();
    // column j of my eight: the codes of my four rows are a dword of the transposed tile
    uint32_t* tw = reinterpret_cast<uint32_t*>(lds.tile);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int cl = cg * 8 + j;
        const float m = lds.mult[cl];
        tw[cl * 32 + (((rg >> 2) ^ (cg & 7)) * 4) + (rg & 3)] = encode(v[0][j] * m, v[1][j] * m, v[2][j] * m, v[3][j] * m);
    }
    __syncthreads();
    // eight consecutive lanes write a column's 128 codes: whole lines of qT
    const int chunk = t & 7;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int cl = p * 64 + (t >> 3);
        const int64_t col = c0 + cl, r = r0 + chunk * 16;
        if (col >= C) continue;
        const uint4 w = lds.tile[cl * 8 + (chunk ^ ((cl >> 3) & 7))];
        uint8_t* q = out.qT + col * out.ldqT + r;
        if (r + 16 <= T) {
            *reinterpret_cast<rc_u32x4_any*>(q) = rc_u32x4_any{w.x, w.y, w.z, w.w};
        } else {
            const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 15; ++j)
                if (r + j < T) q[j] = static_cast<uint8_t>(d[j >> 2] >> (8 * (j & 3)));
        }
    }
}

}  // namespace bsfp8
