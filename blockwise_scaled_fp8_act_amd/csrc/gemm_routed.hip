// gfx950 expert products for few rows an expert (gemm_1x128_128x128_routed): C[r, :] = A[row(r), :]
// B_e^T over the row ranges of a mixture-of-experts plan, float8_e4m3fn operands with 1x128 scales on
// A and 128x128 block scales on B, bf16 out, optionally with the gate and up halves of B joined as
// silu(gate) * up before the one rounding.
//
// With few rows an expert the experts' weights are read once and hardly reused: the bound is their
// traffic from HBM. Two kernels: tiles straight into registers, whose waves read what a matrix
// instruction takes from them and wait for nobody, for problems of few workgroups, where latency
// counts; and 64-row tiles through LDS, whose waves share what they load. sched::routed_kernel has
// the rule and both sides' times. In both, as in the other GEMMs, a K-block's partial comes out of
// one v_mfma_f32_16x16x128_f8f6f4 a subtile, is multiplied by its two scales and added to an fp32
// total; A and B rows are read through plain 64-bit addresses, rows and columns past an end repeat
// the last one and are not stored.
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
    int e;           // expert, -1: no such tile
    int32_t m0, end; // its rows of C
};

// The tile-th tile of TM rows over all experts, from the device boundaries (clamped into [0, M] and
// to non-decreasing order): lane l takes expert 64 i + l, a running maximum orders the boundaries and
// a running sum of the experts' tile counts finds the tile. Every lane returns the same.
template <int TM>
__device__ __forceinline__ RowTile find_tile(const int64_t* offsets, int E, int32_t M, int32_t tile, int lane) {
    int32_t floor_at = 0, first = 0;  // largest boundary so far, tiles of the experts before
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        const auto bound = [&](int i) { return static_cast<int32_t>(min(max(offsets[i], int64_t{0}), static_cast<int64_t>(M))); };
        int32_t lo = e < E ? max(bound(e), floor_at) : 0;
        int32_t hi = e < E ? max(bound(e + 1), lo) : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {  // boundaries up to and with this lane's upper one
            const int32_t o = __shfl_up(hi, d);
            if (lane >= d) hi = max(hi, o);
        }
        const int32_t before = __shfl_up(hi, 1);
        if (lane > 0) lo = max(lo, before);
        const int32_t n = e < E ? (hi - lo + TM - 1) / TM : 0;
        int32_t sum = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const int32_t start = first + sum - n;
        const uint64_t hit = __ballot(tile >= start && tile < start + n);
        if (hit != 0) {
            const int at = __ffsll(static_cast<unsigned long long>(hit)) - 1;
            const int32_t m0 = __builtin_amdgcn_readlane(lo, at) + (tile - __builtin_amdgcn_readlane(start, at)) * TM;
            return RowTile{e0 + at, m0, min(__builtin_amdgcn_readlane(hi, at), m0 + TM)};
        }
        first = __builtin_amdgcn_readlane(first + sum, 63);
        floor_at = __builtin_amdgcn_readlane(hi, 63);
    }
    return RowTile{-1, 0, 0};
}

// Four consecutive columns of one row of C, n on; columns past the end are not written.
__device__ __forceinline__ void store4(const RoutedArgs& a, int64_t r, int64_t n, const float (&v)[4]) {
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

// ---- Straight into registers: a tile of 16 MS rows by NS 16-column subtiles of B (with SWIGLU half
// of them of the gate half, half the same columns of the up half), whose K-blocks WK waves split.
// Each wave keeps D K-blocks' operands on the way: no barrier before the end. One row each of 8 experts
// of 2048 x 4096: 13.6 us, 67 MB at 4.9 TB/s; four waves, three blocks and two subtiles were the best
// of 4 or 8, 2 to 4 and 2 or 4 (the others 14.2-16.2 us).
template <int MS, int NS, int WK, int D, bool SWIGLU>
__global__ __launch_bounds__(64 * WK) void routed_kernel(RoutedArgs a) {
    constexpr int TM = 16 * MS, kPairs = SWIGLU ? NS / 2 : NS, kOut = 16 * kPairs;
    __shared__ float red[WK][MS * NS * 4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t tile = blockIdx.x / static_cast<uint32_t>(a.col_tiles);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x - tile * a.col_tiles) * kOut;
    const RowTile rt = find_tile<TM>(a.offsets, static_cast<int>(a.E), static_cast<int32_t>(a.M), tile, lane);
    if (rt.e < 0) return;

    const int i16 = lane & 15, g = lane >> 4;
    // this lane's row of each 16-row subtile; rows past the tile read its last row and are not stored
    const uint8_t* ap[MS];
    const float* as[MS];
    bool known[MS];
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        const int64_t r = min(rt.m0 + 16 * m + i16, rt.end - 1);
        int64_t src = r;
        if (a.rows != nullptr) {
            const int32_t pair = a.rows[r];
            src = pair >= 0 ? static_cast<uint32_t>(pair) / static_cast<uint32_t>(a.k) : -1;
        }
        known[m] = src >= 0 && src < a.a_rows;
        if (!known[m]) src = 0;
        ap[m] = a.a + src * a.lda + g * 16;
        as[m] = a.a_s + src;
    }
    const uint8_t* bp[NS];
    const float* bs[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        // N: output columns. Subtile s is columns first .. first + 15 of C, of the gate or up half of B.
        const int64_t half = SWIGLU ? (s & 1) * a.N : 0, first = min(n0 + 16 * (SWIGLU ? s / 2 : s), a.N - 1);
        bp[s] = a.b + rt.e * a.b_stride + (half + min(first + i16, a.N - 1)) * a.ldb + g * 16;
        bs[s] = a.b_s + rt.e * a.bs_stride + (half + first) / kGroup * a.bs_nb;  // 16 columns lie in one block of 128
    }

    const int Kb = static_cast<int>(a.K / kGroup);
    const int kb0 = Kb * wave / WK, kb1 = Kb * (wave + 1) / WK;
    v4f tot[MS][NS] = {};
    v8i af[D][MS], bf[D][NS];
    float sa[D][MS], sb[D][NS];
    const auto load = [&](int d, int kb) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            bf[d][s] = load_frag(bp[s] + static_cast<int64_t>(kb) * kGroup);
            sb[d][s] = bs[s][kb * a.bs_kb];
        }
#pragma unroll
        for (int m = 0; m < MS; ++m) {
            af[d][m] = load_frag(ap[m] + static_cast<int64_t>(kb) * kGroup);
            sa[d][m] = as[m][kb * a.a_rows];
        }
    };
    const auto multiply = [&](int d) {
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const v4f p = mfma_fp8_16x16x128(bf[d][s], af[d][m]);
                const float f = sa[d][m] * sb[d][s];
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[m][s][i] = fmaf(p[i], f, tot[m][s][i]);
            }
    };
    // D - 1 K-blocks ahead; past the end the last block is loaded again and not used
    if (kb0 < kb1) {
#pragma unroll
        for (int d = 0; d + 1 < D; ++d) load(d, min(kb0 + d, kb1 - 1));
        int kb = kb0;
        for (; kb + D <= kb1; kb += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                load((d + D - 1) % D, min(kb + d + D - 1, kb1 - 1));
                multiply(d);
            }
        }
#pragma unroll
        for (int d = 0; d + 1 < D; ++d)
            if (kb + d < kb1) multiply(d);
    }

#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][(m * NS + s) * 4 + i][lane] = tot[m][s][i];
    __syncthreads();
    // Output subtiles (a gate and up pair with SWIGLU): the waves take turns.
#pragma unroll
    for (int u = 0; u < MS * kPairs; ++u) {
        if (u % WK != wave) continue;
        const int m = u / kPairs, j = u % kPairs, s = SWIGLU ? 2 * j : j;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                x += red[w][(m * NS + s) * 4 + i][lane];
                if (SWIGLU) y += red[w][(m * NS + s + 1) * 4 + i][lane];
            }
            v[i] = !known[m] ? 0.0f : SWIGLU ? silu(x) * y : x;
        }
        const int64_t r = rt.m0 + 16 * m + i16;
        if (r < rt.end) store4(a, r, n0 + 16 * j + 4 * g, v);
    }
}

template <int MS, int NS, int WK, int D, bool SWIGLU>
hipError_t launch(RoutedArgs a, hipStream_t stream) {
    constexpr int64_t kOut = 16 * (SWIGLU ? NS / 2 : NS);
    a.col_tiles = (a.N + kOut - 1) / kOut;
    const int64_t blocks = sched::routed_row_tiles(a.M, a.E, 16 * MS) * a.col_tiles;
    routed_kernel<MS, NS, WK, D, SWIGLU><<<dim3(static_cast<unsigned>(blocks)), 64 * WK, 0, stream>>>(a);
    return hipGetLastError();
}

// ---- Tiles through LDS, for more rows an expert: 64 rows by 128 rows of B, eight waves of 32 x 32
// (two by four). Every K-block's operands go global -> LDS with direct loads, S stages deep, one
// barrier a K-block; waves share each other's rows, so a K-block of A and B crosses L2 once a
// workgroup. Three stages are 75 KB: two workgroups a CU, one's latency under the other's loads (two
// stages 118 us, four, one workgroup a CU, 103, three 99 for 16 rows of 64 experts, gated 1024 x 4096).
// Bound by HBM: that case, past the caches, 92-98 us, is 451 MB at 4.9 TB/s; 60 rows of 64 experts of
// 5120 x 1280 take 101 us against 90 for their bytes (register tiles 160 and more).
namespace tiled {

constexpr int kTM = 64, kTN = 128, kWaves = 8;
constexpr int kB = kTM * 8, kSA = kB + kTN * 8, kSB = kSA + 16, kStage = kSB + 16;  // in 16-byte units

// A direct load to LDS address lds + BYTES * lane, BYTES (4 or 16) a lane; STREAM: past the caches.
template <int BYTES, bool STREAM = false>
__device__ __forceinline__ void dma(uint32_t lds, const void* p) {
    uint32_t saved;
    if (BYTES == 16 && STREAM)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %2, off sc1 nt\n\ts_mov_b32 m0, %0"
                     : "=&s"(saved) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory");
    else if (BYTES == 16)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
                     : "=&s"(saved) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory");
    else
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tglobal_load_lds_dword %2, off\n\ts_mov_b32 m0, %0"
                     : "=&s"(saved) : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Waits until at most `later` blocks' loads (L each, later <= MAX) of this wave are on the way.
template <int L, int MAX>
__device__ __forceinline__ void wait_block(int later) {
    if constexpr (MAX == 0) {
        wait_loads<0>();
    } else {
        if (later >= MAX) wait_loads<L * MAX>();
        else wait_block<L, MAX - 1>(later);
    }
}

// STREAM: B past the caches, where an expert's rows fit one tile and its weights are read once.
template <int S, bool SWIGLU, bool STREAM>
__global__ __launch_bounds__(64 * kWaves) void routed_kernel(RoutedArgs a) {
    __shared__ u32x4 smem[S * kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1, i16 = lane & 15, g = lane >> 4;
    const int32_t tile = blockIdx.x / static_cast<uint32_t>(a.col_tiles);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x - tile * a.col_tiles) * (SWIGLU ? kTN / 2 : kTN);
    const RowTile rt = find_tile<kTM>(a.offsets, static_cast<int>(a.E), static_cast<int32_t>(a.M), tile, lane);
    if (rt.e < 0) return;

    // Load q of a stage: 8 rows of 128 bytes, a lane one 16-byte chunk, put where lds_swizzle of the
    // row says. Wave w loads A rows 8 w .. and B rows 16 w .. + 15; rows past the end repeat the last.
    const int lr = lane >> 3;
    const auto source_row = [&](int64_t r) {  // A's row for row r of C, -1: none
        if (a.rows == nullptr) return r;
        const int32_t pair = a.rows[r];
        const int64_t src = pair >= 0 ? static_cast<uint32_t>(pair) / static_cast<uint32_t>(a.k) : -1;
        return src < a.a_rows ? src : -1;
    };
    const int64_t arow = max(source_row(min(rt.m0 + 8 * wave + lr, rt.end - 1)), int64_t{0});
    const uint8_t* ap = a.a + arow * a.lda + 16 * ((lane & 7) ^ geom::lds_swizzle(8 * wave + lr));
    const uint8_t* bp[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = 16 * wave + 8 * q + lr;  // of the tile: with SWIGLU 16 gate, 16 up, ...
        const int64_t n = SWIGLU ? min(n0 + 16 * (row >> 5) + (row & 15), a.N - 1) + ((row >> 4) & 1) * a.N : min(n0 + row, a.N - 1);
        bp[q] = a.b + rt.e * a.b_stride + n * a.ldb + 16 * ((lane & 7) ^ geom::lds_swizzle(row));
    }
    // wave 0 loads the A scales of the 64 rows, wave 1 the B scale (lanes 32 on: of the up half)
    const float* sp = a.a_s + max(source_row(min(rt.m0 + lane, rt.end - 1)), int64_t{0});
    int64_t s_step = a.a_rows;
    if (wave == 1) {
        sp = a.b_s + rt.e * a.bs_stride + (n0 + (SWIGLU && lane >= 32 ? a.N : 0)) / kGroup * a.bs_nb;
        s_step = a.bs_kb;
    }
    const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
    const auto issue = [&](int kb, int stage) {
        const uint32_t base = lds0 + static_cast<uint32_t>(stage * kStage * 16);
        const int64_t adv = static_cast<int64_t>(kb) * kGroup;
        dma<16>(base + 64 * wave * 16, ap + adv);
        dma<16, STREAM>(base + (kB + 128 * wave) * 16, bp[0] + adv);
        dma<16, STREAM>(base + (kB + 128 * wave + 64) * 16, bp[1] + adv);
        if (wave < 2) dma<4>(base + (wave == 0 ? kSA : kSB) * 16, sp + kb * s_step);
    };

    const int Kb = static_cast<int>(a.K / kGroup);
    v4f tot[2][2] = {};
#pragma unroll
    for (int kb = 0; kb < S - 1; ++kb)
        if (kb < Kb) issue(kb, kb);
    int stage = 0, into = S - 1;  // of block kb, and of block kb + S - 1
    const int sw = geom::lds_swizzle(i16);
    for (int kb = 0; kb < Kb; ++kb) {
        // block kb has landed for every wave, and no wave reads the stage of block kb - 1 any more
        const int later = min(S - 2, Kb - 1 - kb);
        if (wave < 2) wait_block<4, S - 2>(later);
        else wait_block<3, S - 2>(later);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kb + S - 1 < Kb) issue(kb + S - 1, into);
        const u32x4* st = smem + stage * kStage;
        const auto frag = [&](int unit) {
            const u32x4 lo = st[unit + (g ^ sw)], hi = st[unit + ((g + 4) ^ sw)];
            return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
        };
        const float* sa = reinterpret_cast<const float*>(st + kSA);
        const float* sb = reinterpret_cast<const float*>(st + kSB);
        v8i af[2], bf[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) af[m] = frag((32 * wm + 16 * m + i16) * 8);
#pragma unroll
        for (int s = 0; s < 2; ++s) bf[s] = frag(kB + (32 * wn + 16 * s + i16) * 8);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const v4f p = mfma_fp8_16x16x128(bf[s], af[m]);
                const float f = sa[32 * wm + 16 * m + i16] * sb[SWIGLU && s == 1 ? 32 : 0];
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[m][s][i] = fmaf(p[i], f, tot[m][s][i]);
            }
        stage = stage + 1 == S ? 0 : stage + 1;
        into = into + 1 == S ? 0 : into + 1;
    }

#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int64_t r = rt.m0 + 32 * wm + 16 * m + i16;
        if (r >= rt.end) continue;
        const bool known = source_row(r) >= 0;
#pragma unroll
        for (int s = 0; s < (SWIGLU ? 1 : 2); ++s) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = !known ? 0.0f : SWIGLU ? silu(tot[m][0][i]) * tot[m][1][i] : tot[m][s][i];
            store4(a, r, n0 + (SWIGLU ? 16 * wn : 32 * wn + 16 * s) + 4 * g, v);
        }
    }
}

template <int S, bool SWIGLU>
hipError_t launch(RoutedArgs a, bool once, hipStream_t stream) {
    constexpr int64_t kOut = SWIGLU ? kTN / 2 : kTN;
    a.col_tiles = (a.N + kOut - 1) / kOut;
    const int64_t blocks = sched::routed_row_tiles(a.M, a.E, kTM) * a.col_tiles;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (once)
        routed_kernel<S, SWIGLU, true><<<grid, 64 * kWaves, 0, stream>>>(a);
    else
        routed_kernel<S, SWIGLU, false><<<grid, 64 * kWaves, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace tiled

}  // namespace

hipError_t launch_gemm_routed(RoutedArgs a, bool swiglu, hipStream_t stream) {
    a.c_vec = (reinterpret_cast<uintptr_t>(a.c) % 8 == 0) && a.ldc % 4 == 0;
    const bool once = sched::routed_reads_once(a.M, a.N, a.E, swiglu);
    switch (sched::routed_kernel(a.M, a.N, a.K, a.E, swiglu)) {
        case sched::kRoutedRegisters16: return swiglu ? launch<1, 2, 4, 3, true>(a, stream) : launch<1, 2, 4, 3, false>(a, stream);
        case sched::kRoutedRegisters32: return swiglu ? launch<2, 2, 4, 3, true>(a, stream) : launch<2, 2, 4, 3, false>(a, stream);
        default: return swiglu ? tiled::launch<3, true>(a, once, stream) : tiled::launch<3, false>(a, once, stream);
    }
}

}  // namespace bsfp8
