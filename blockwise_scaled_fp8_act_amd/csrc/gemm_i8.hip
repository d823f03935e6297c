// gfx950 int8 product: C[m, n] (bf16) = a_s[m] b_s[n] sum_k A[m, k] B[n, k], the sum exact in int32.
//   * one v_mfma_i32_16x16x64_i8 a 16 x 16 subtile and 64 bytes of K, accumulating in place: the scales come
//     once, at the end, so the matrix cores wait for nothing in between;
//   * B is the first operand, so a lane's four sums are four consecutive columns of one row of C;
//   * operands go from memory straight to LDS by buffer loads whose resources end with the tensor: rows past
//     an end read as zero. Of a partial last K-block the bytes at and past K are zeroed in A's fragments
//     alone, which makes every product with them zero.
#include "device_common.hpp"
#include "geometry.hpp"
#include "launch.hpp"

namespace bsfp8 {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, static_cast<int>(bytes), 0x00020000);
}

// 16 bytes a lane from the resource to LDS address lds + 16 * lane.
__device__ __forceinline__ void dma16(uint32_t lds, __amdgpu_buffer_rsrc_t r, uint32_t voff) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "buffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(r)
        : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Bytes of a tile's rows that may be read: the last row ends with the 16 bytes that hold its last code.
__device__ __forceinline__ int64_t tile_bytes(int64_t rows, int64_t ld, int64_t K) {
    return rows > 0 ? (rows - 1) * ld + ((K + 15) & ~int64_t{15}) : 0;
}

// BM x BN tiles of C in waves of WM x WN. LDS stage: A rows, then B rows, 128 bytes of K each, the 16-byte
// chunks of a row swizzled by (row / 2) % 8 (geom::lds_swizzle), so that a fragment's reads hit all banks.
template <int BM, int BN, int WM, int WN>
struct Tile {
    static constexpr int kWavesM = BM / WM, kWaves = kWavesM * (BN / WN), kThreads = 64 * kWaves;
    static constexpr int kMS = WM / 16, kNS = WN / 16;
    static constexpr int kLoads = (BM + BN) / 8 / kWaves;  // 8 rows each
    static constexpr int kStage = (BM + BN) * 8;           // 16-byte units
    static_assert((BM + BN) % (8 * kWaves) == 0, "whole loads a wave");
};

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((Tile<BM, BN, WM, WN>::kThreads), 1) void gemm_i8_kernel(I8Args g, int mt, int nt, int c_vec) {
    using C = Tile<BM, BN, WM, WN>;
    __shared__ u32x4 smem[2 * C::kStage];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % C::kWavesM, wn = wave / C::kWavesM, l16 = lane & 15, lg = lane >> 4;
    int tm, tn;
    geom::tile_of(blockIdx.x, mt, nt, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.a + m0 * g.lda, tile_bytes(min(g.M - m0, int64_t{BM}), g.lda, g.K));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.b + n0 * g.ldb, tile_bytes(min(g.N - n0, int64_t{BN}), g.ldb, g.K));
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem)));
    const int Kb = static_cast<int>((g.K + kGroup - 1) / kGroup);

    // load p of a wave: rows 8 r .. of A (r < BM / 8) or of B
    auto issue = [&](int kb, int stage) {
#pragma unroll
        for (int p = 0; p < C::kLoads; ++p) {
            const int r = wave * C::kLoads + p;
            const bool is_a = r < BM / 8;
            const int q = is_a ? r : r - BM / 8;
            const uint32_t off = static_cast<uint32_t>((8 * q + (lane >> 3)) * (is_a ? g.lda : g.ldb)) + 16 * geom::fast_operand_chunk(q, lane);
            dma16(lds0 + static_cast<uint32_t>(stage * C::kStage + 64 * r) * 16, is_a ? ra : rb, off + static_cast<uint32_t>(kb * kGroup));
        }
    };

    i32x4 acc[C::kMS][C::kNS];
#pragma unroll
    for (int i = 0; i < C::kMS; ++i)
#pragma unroll
        for (int j = 0; j < C::kNS; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    const int sw = geom::lds_swizzle(l16);
    if (Kb > 0) issue(0, 0);
    for (int kb = 0; kb < Kb; ++kb) {
        wait_loads<0>();
        lds_barrier();  // block kb is there, and no wave reads the other stage any more
        if (kb + 1 < Kb) issue(kb + 1, (kb + 1) & 1);
        const u32x4* st = smem + (kb & 1) * C::kStage;
        const int keep = static_cast<int>(min(g.K - static_cast<int64_t>(kb) * kGroup, int64_t{kGroup}));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = (lg + 4 * h) ^ sw;
            i32x4 a[C::kMS], b[C::kNS];
#pragma unroll
            for (int i = 0; i < C::kMS; ++i) {
                a[i] = __builtin_bit_cast(i32x4, st[(WM * wm + 16 * i + l16) * 8 + pos]);
                if (keep < kGroup)
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int left = keep - 16 * (lg + 4 * h) - 4 * d;
                        a[i][d] &= left >= 4 ? -1 : left <= 0 ? 0 : (1 << (8 * left)) - 1;
                    }
            }
#pragma unroll
            for (int j = 0; j < C::kNS; ++j) b[j] = __builtin_bit_cast(i32x4, st[BM * 8 + (WN * wn + 16 * j + l16) * 8 + pos]);
#pragma unroll
            for (int i = 0; i < C::kMS; ++i)
#pragma unroll
                for (int j = 0; j < C::kNS; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j], a[i], acc[i][j], 0, 0, 0);
        }
    }

#pragma unroll
    for (int i = 0; i < C::kMS; ++i) {
        const int64_t m = m0 + WM * wm + 16 * i + l16;
        if (m >= g.M) continue;
        const float as = Kb > 0 ? g.a_s[m] : 0.0f;
#pragma unroll
        for (int j = 0; j < C::kNS; ++j) {
            const int64_t n = n0 + WN * wn + 16 * j + 4 * lg;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (static_cast<float>(acc[i][j][e]) * as) * (Kb > 0 && n + e < g.N ? g.b_s[n + e] : 0.0f);
            const uint32_t w0 = pack_bf16x2(v[0], v[1]), w1 = pack_bf16x2(v[2], v[3]);
            uint16_t* c = g.c + m * g.ldc + n;
            if (c_vec && n + 4 <= g.N) {
                *reinterpret_cast<uint2*>(c) = make_uint2(w0, w1);
            } else {
                const uint16_t h[4] = {static_cast<uint16_t>(w0), static_cast<uint16_t>(w0 >> 16), static_cast<uint16_t>(w1),
                                       static_cast<uint16_t>(w1 >> 16)};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < g.N) c[e] = h[e];
            }
        }
    }
}

}  // namespace

hipError_t launch_gemm_i8(const I8Args& g, int cus, hipStream_t stream) {
    const int c_vec = reinterpret_cast<uintptr_t>(g.c) % 8 == 0 && g.ldc % 4 == 0;
    const auto tiles = [&](int64_t bm, int64_t bn) { return ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn); };
#define BSFP8_I8(BM, BN, WM, WN)                                                                                         \
    gemm_i8_kernel<BM, BN, WM, WN><<<static_cast<unsigned>(tiles(BM, BN)), Tile<BM, BN, WM, WN>::kThreads, 0, stream>>>( \
        g, static_cast<int>((g.M + BM - 1) / BM), static_cast<int>((g.N + BN - 1) / BN), c_vec)
    if (tiles(256, 256) >= cus / 2) BSFP8_I8(256, 256, 64, 128);
    else if (tiles(128, 128) >= cus / 2) BSFP8_I8(128, 128, 64, 64);
    else BSFP8_I8(64, 64, 32, 32);
#undef BSFP8_I8
    return hipGetLastError();
}

}  // namespace bsfp8
