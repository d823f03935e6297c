// gfx950 expert products for few rows an expert (gemm_1x128_128x128_routed): C[r, :] = A[row(r), :]
// B_e^T over the row ranges of a mixture-of-experts plan, float8_e4m3fn operands with 1x128 scales on
// A and 128x128 block scales on B, bf16 out, optionally with the gate and up halves of B joined as
// silu(gate) * up before the one rounding.
//
// With few rows an expert the experts' weights are read once and hardly reused: the bound is their
// traffic from HBM. So B does not go through LDS: every wave reads its own 16-column blocks of B
// straight into the registers a v_mfma_f32_16x16x128_f8f6f4 takes them from, and no barrier stands
// between a wave and its next load. A (a few rows, read by every workgroup of its expert) comes from
// L2 the same way. The waves of a workgroup split K between them and join their fp32 totals through
// LDS in a fixed order. As in the other GEMMs a K-block's partial comes out of one matrix
// instruction, is multiplied by its two scales and added to an fp32 total.
#include "device_common.hpp"
#include "geometry.hpp"
#include "launch.hpp"

namespace bsfp8 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4f mfma_fp8_16x16x128(const v8i& a, const v8i& b) {
    const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const f2v v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf2v));
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// A lane's 32 codes of a K-block row: the 16-byte chunks g and g + 4 of its 128 bytes, g = lane / 16.
// The matrix instruction sums over k whichever k a lane's bytes stand for, as long as A and B agree;
// this order makes each load of a wave read 64 contiguous bytes of every row.
__device__ __forceinline__ v8i load_frag(const uint8_t* p) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(p), hi = *reinterpret_cast<const u32x4*>(p + 64);
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

struct RowTile {
    int e;            // expert, -1: no such tile
    int64_t m0, end;  // its rows of C
};

// The tile-th tile of TM rows over all experts, from the device boundaries (clamped into [0, M] and
// to non-decreasing order): lane l takes expert 64 i + l, a running maximum orders the boundaries and
// a running sum of the experts' tile counts finds the tile. Every lane returns the same.
template <int TM>
__device__ __forceinline__ RowTile find_tile(const int64_t* offsets, int64_t E, int64_t M, int64_t tile, int lane) {
    int64_t floor_at = 0, first = 0;  // largest boundary so far, tiles of the experts before
    for (int64_t e0 = 0; e0 < E; e0 += 64) {
        const int64_t e = e0 + lane;
        int64_t lo = e < E ? min(max(offsets[e], int64_t{0}), M) : 0;
        int64_t hi = e < E ? min(max(offsets[e + 1], int64_t{0}), M) : 0;
        lo = max(lo, floor_at);
        hi = max(hi, lo);
        for (int d = 1; d < 64; d <<= 1) {  // boundaries up to and with this lane's upper one
            const int64_t o = __shfl_up(hi, d);
            if (lane >= d) hi = max(hi, o);
        }
        const int64_t before = __shfl_up(hi, 1);
        if (lane > 0) lo = max(lo, before);
        const int64_t n = e < E ? (hi - lo + TM - 1) / TM : 0;
        int64_t sum = n;
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const int64_t start = first + sum - n;
        const uint64_t hit = __ballot(tile >= start && tile < start + n);
        if (hit != 0) {
            const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
            RowTile r;
            r.e = static_cast<int>(e0) + at;
            r.m0 = __shfl(lo, at) + (tile - __shfl(start, at)) * TM;
            r.end = min(__shfl(hi, at), r.m0 + TM);
            return r;
        }
        first += __shfl(sum, 63);
        floor_at = __shfl(hi, 63);
    }
    return RowTile{-1, 0, 0};
}

// MS 16-row subtiles, two 16-column subtiles of B (with SWIGLU one of the gate half and the same
// columns of the up half) and KW waves that split the K-blocks.
template <int MS, bool SWIGLU, int KW>
__global__ __launch_bounds__(64 * KW) void routed_kernel(RoutedArgs a) {
    constexpr int TM = 16 * MS, NS = 2, kOut = SWIGLU ? 16 : 32;
    __shared__ float red[KW][MS * NS * 4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t tile = blockIdx.x / a.col_tiles;
    const int64_t n0 = (blockIdx.x - tile * a.col_tiles) * kOut;
    const RowTile rt = find_tile<TM>(a.offsets, a.E, a.M, tile, lane);
    if (rt.e < 0) return;

    const int i16 = lane & 15, g = lane >> 4;
    // this lane's row of each 16-row subtile; rows past the tile read its last row and are not stored
    const uint8_t* ap[MS];
    const float* as[MS];
    bool known[MS];
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        const int64_t r = min(rt.m0 + 16 * m + i16, rt.end - 1);
        int64_t src = a.rows != nullptr ? a.rows[r] : r;
        if (a.rows != nullptr) src = src >= 0 ? src / a.k : -1;
        known[m] = src >= 0 && src < a.a_rows;
        if (!known[m]) src = 0;
        ap[m] = a.a + src * a.lda + g * 16;
        as[m] = a.a_s + src;
    }
    const uint8_t* bp[NS];
    const float* bs[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const int64_t first = SWIGLU ? n0 + s * a.N : n0 + 16 * s;   // N: output columns
        const int64_t row = SWIGLU ? min(first + i16, (s + 1) * a.N - 1) : min(first + i16, a.N - 1);
        bp[s] = a.b + rt.e * a.b_stride + row * a.ldb + g * 16;
        // the lane's four outputs are columns first + 4 g .. + 3, inside one 128-column block
        const int64_t nb = min(first + 4 * g, (SWIGLU ? (s + 1) * a.N : a.N) - 1) / kGroup;
        bs[s] = a.b_s + rt.e * a.bs_stride + nb * a.bs_nb;
    }

    const int64_t Kb = a.K / kGroup;
    const int64_t kb0 = Kb * wave / KW, kb1 = Kb * (wave + 1) / KW;
    v4f tot[MS][NS] = {};
    for (int64_t kb = kb0; kb < kb1; ++kb) {
        v8i bf[NS];
        float sb[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            bf[s] = load_frag(bp[s] + kb * kGroup);
            sb[s] = bs[s][kb * a.bs_kb];
        }
#pragma unroll
        for (int m = 0; m < MS; ++m) {
            const v8i af = load_frag(ap[m] + kb * kGroup);
            const float sa = as[m][kb * a.a_rows];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const v4f p = mfma_fp8_16x16x128(bf[s], af);
                const float f = sa * sb[s];
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[m][s][i] = fmaf(p[i], f, tot[m][s][i]);
            }
        }
    }

#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][(m * NS + s) * 4 + i][lane] = tot[m][s][i];
    __syncthreads();

    // units of one output subtile (a gate and up pair with SWIGLU), dealt to the waves
    constexpr int kUnits = SWIGLU ? MS : MS * NS;
    for (int u = wave; u < kUnits; u += KW) {
        const int m = SWIGLU ? u : u / NS, s = SWIGLU ? 0 : u % NS;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                x += red[w][(m * NS + s) * 4 + i][lane];
                if (SWIGLU) y += red[w][(m * NS + 1) * 4 + i][lane];
            }
            v[i] = SWIGLU ? silu(x) * y : x;
        }
        bool ok = true;
#pragma unroll
        for (int q = 0; q < MS; ++q)
            if (q == m) ok = known[q];
        const int64_t r = rt.m0 + 16 * m + i16;
        const int64_t n = n0 + 16 * s + 4 * g;
        if (r >= rt.end || n >= a.N) continue;
        if (!ok) v[0] = v[1] = v[2] = v[3] = 0.0f;
        const uint32_t w0 = pack_bf16x2(v[0], v[1]), w1 = pack_bf16x2(v[2], v[3]);
        uint16_t* c = a.c + r * a.ldc + n;
        if (a.c_vec && n + 4 <= a.N) {
            *reinterpret_cast<uint2*>(c) = uint2{w0, w1};
        } else {
            const uint16_t h[4] = {static_cast<uint16_t>(w0), static_cast<uint16_t>(w0 >> 16), static_cast<uint16_t>(w1),
                                   static_cast<uint16_t>(w1 >> 16)};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) c[i] = h[i];
        }
    }
}

template <int MS, bool SWIGLU, int KW>
hipError_t launch(RoutedArgs a, hipStream_t stream) {
    const int64_t kOut = SWIGLU ? 16 : 32;
    a.col_tiles = (a.N + kOut - 1) / kOut;
    const int64_t blocks = sched::routed_row_tiles(a.M, a.E, 16 * MS) * a.col_tiles;
    if (blocks > 0x7FFFFFFFLL) return hipErrorInvalidValue;
    routed_kernel<MS, SWIGLU, KW><<<dim3(static_cast<unsigned>(blocks)), 64 * KW, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_routed(RoutedArgs a, bool swiglu, hipStream_t stream) {
    a.c_vec = (reinterpret_cast<uintptr_t>(a.c) % 8 == 0) && a.ldc % 4 == 0;
    switch (sched::routed_subtiles(a.M, a.E)) {
        case 1: return swiglu ? launch<1, true, 4>(a, stream) : launch<1, false, 4>(a, stream);
        case 2: return swiglu ? launch<2, true, 4>(a, stream) : launch<2, false, 4>(a, stream);
        default: return swiglu ? launch<4, true, 4>(a, stream) : launch<4, false, 4>(a, stream);
    }
}

}  // namespace bsfp8
