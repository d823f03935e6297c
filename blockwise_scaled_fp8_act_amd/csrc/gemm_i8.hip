// gfx950 int8 product: C[m, n] (bf16) = a_s[m] b_s[n] sum_k A[m, k] B[n, k], the sum exact in int32.
//   * one v_mfma_i32_16x16x64_i8 a 16 x 16 subtile and 64 bytes of K, accumulating in place: the scales come
//     once, at the end, so the matrix cores wait for nothing in between;
//   * B is the first operand, so a lane's four sums are four consecutive columns of one row of C;
//   * operands go from memory straight to LDS by buffer loads whose resources end with the tensor: rows past
//     an end read as zero. Of a partial last K-block the bytes at and past K are zeroed in A's fragments
//     alone, which makes every product with them zero.
// Three kernels; sched::i8_kernel has the rule between them and the tiles' measured costs:
//   * rows of B straight to the lanes (a few rows of A): bound by reading B once;
//   * tiles with several K-blocks in LDS: problems whose 256 x 256 tiles would leave compute units idle;
//   * 256 x 256 tiles, bound by the card's power: the matrix cores are busy for 60% of the cycles, at a clock
//     that has come down from 2.4 to 1.9 GHz.
#include <type_traits>

#include "device_common.hpp"
#include "geometry.hpp"
#include "launch.hpp"
#include "schedule.hpp"

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

// 16 bytes a lane from the resource to LDS address lds + 16 * lane; PAST: not kept in the caches.
template <bool PAST = false>
__device__ __forceinline__ void dma16(uint32_t lds, __amdgpu_buffer_rsrc_t r, uint32_t voff) {
    uint32_t saved;
    if (PAST)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tbuffer_load_dwordx4 %2, %3, 0 offen nt lds\n\ts_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(r)
                     : "memory");
    else
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
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

// The offset of a K-block past the last: beyond every resource (their sizes and the lanes' offsets are below
// 2^31), so its loads write zeros to LDS and the count of loads under way stays the same.
constexpr uint32_t kPastEnd = 0x80000000u;

// The block of K with which the workgroups of an XCD begin, of Kb.
__device__ __forceinline__ int first_block(int Kb) { return static_cast<int>(blockIdx.x % geom::kXcds) * Kb / geom::kXcds; }

// Zeroes the bytes of a lane's 16 that lie at or past `left`.
__device__ __forceinline__ void keep_bytes(i32x4& v, int left) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int l = left - 4 * d;
        v[d] &= l >= 4 ? -1 : l <= 0 ? 0 : (1 << (8 * l)) - 1;
    }
}

// The output columns n .. n + 3: their scales, zero past the end or without a sum (K == 0).
__device__ __forceinline__ void column_scales(const I8Args& g, int64_t n, float (&s)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = g.K > 0 && n + e < g.N ? g.b_s[n + e] : 0.0f;
}
__device__ __forceinline__ uint2 scaled4(const i32x4& sum, float as, const float (&bs)[4]) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (static_cast<float>(sum[e]) * as) * bs[e];
    return make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Writes a wave's WM x WN block of C, rows from m0 and columns from n0 on, through its own part of LDS, so that a
// store's lanes write whole runs of a row, wherever rows begin (2048 x 1408 x 1280 11.6 us, with eight bytes a lane from the
// registers 13.4; 2048 x 4096 x 4096 43 and 46). 16-byte chunk c of row r lies at c ^ (r % chunks). PAST: past the caches.
template <int WM, int WN, bool PAST>
__device__ __forceinline__ void store_block(const I8Args& g, const i32x4 (&acc)[WM / 16][WN / 16], int64_t m0, int64_t n0, uint8_t* own, int lane) {
    constexpr int kChunks = WN / 8;  // of a row
    const int l16 = lane & 15, lg = lane >> 4;
#pragma unroll
    for (int j = 0; j < WN / 16; ++j) {
        float bs[4];
        column_scales(g, n0 + 16 * j + 4 * lg, bs);
#pragma unroll
        for (int i = 0; i < WM / 16; ++i) {
            const int r = 16 * i + l16;
            const float as = g.K > 0 && m0 + r < g.M ? g.a_s[m0 + r] : 0.0f;
            *reinterpret_cast<uint2*>(own + r * (2 * WN) + (((2 * j + (lg >> 1)) ^ (r & (kChunks - 1))) * 16) + 8 * (lg & 1)) = scaled4(acc[i][j], as, bs);
        }
    }
    wave_lds_fence();  // the pieces read below are other lanes' writes
#pragma unroll
    for (int p = 0; p < (WM * kChunks + 63) / 64; ++p) {
        const int r = (64 * p + lane) / kChunks, c = lane % kChunks;
        const int64_t m = m0 + r, n = n0 + 8 * c;
        if (r >= WM || m >= g.M || n >= g.N) continue;
        const u32x4 v = *reinterpret_cast<const u32x4*>(own + r * (2 * WN) + ((c ^ (r & (kChunks - 1))) * 16));
        uint16_t* to = g.c + m * g.ldc + n;
        if (n + 8 <= g.N) {
            if (PAST) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(to));
            else *reinterpret_cast<u32x4_any*>(to) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (n + e < g.N) to[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// ---- Tiles of BM x BN in waves of WM x WN, STAGES blocks of KS bytes of K in LDS, loads STAGES - 1 blocks
// ahead of the products. A row of a stage has its 16-byte chunks swizzled by the row, so that the 16 rows of a
// fragment's read fall on all banks: chunk c at c ^ swizzle(row). One barrier a block. With few workgroups a
// block's time is one wait, barrier and chain of reads and products, so blocks are long (256 bytes) for the
// small tiles; with two workgroups on a CU each hides the other's waits.
// The blocks of K come in an order that begins elsewhere for other workgroups (the sum is whole, so any order gives
// the same bits): rows lie a multiple of a KB apart, so workgroups that all read one block at a time reach only
// an eighth or fewer of HBM's channels. PAST, for weights that are read once and by so many workgroups that
// HBM is the bound: every column of tiles begins with another block, and B is read past the caches (16 rows by
// 14336 x 4096 14.7 us without both, 13.2 with the second, 11.5 with both, 5.1 TB/s). Else the workgroups of an
// XCD, which share rows in its L2, begin together (512 x 5120 x 5120 in 64 x 128 tiles 39.8 -> 36.3 us).
// 64 x 5120 x 5120 12.6 us, 1000 x 1000 x 1288 8.3. What most likely bounds a tile: the loads into LDS, some 32 bytes a cycle and CU. A
// 128 x 128 tile's block of 32 KB takes 1080 cycles, its products 512; with loads that all lie out of range it takes as
// long (512 x 5120 x 5120 24.4 us of 31.5, the rest is HBM's). So fragments read half a block ahead (31.6), waves of 64 x 64
// with half of a block's K each, which read a third less from LDS (32.2), and other orders of the blocks in an XCD (31.2)
// gain nothing.
template <int BM, int BN, int WM, int WN, int STAGES, int KS, bool PAST>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void tile_kernel(I8Args g, int mt, int nt) {
    constexpr int kWavesM = BM / WM, kWaves = kWavesM * (BN / WN), kMS = WM / 16, kNS = WN / 16;
    constexpr int kChunks = KS / 16, kRows = 64 / kChunks;  // of a row; rows of one load
    constexpr int kStage = (BM + BN) * kChunks, kLoads = (BM + BN) / kRows / kWaves;
    static_assert((BM + BN) % (kRows * kWaves) == 0 && BM % kRows == 0, "whole loads a wave");
    static_assert((STAGES - 2) * kLoads <= 63, "loads under way that can be counted");
    static_assert(KS == 128 || KS == 256, "swizzles of these");
    __shared__ u32x4 smem[STAGES * kStage];
    const auto swizzle = [](int row) { return KS == 128 ? geom::lds_swizzle(row) : row & 15; };
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % kWavesM, wn = wave / kWavesM, l16 = lane & 15, lg = lane >> 4;
    int tm, tn;
    geom::tile_of(blockIdx.x, mt, nt, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.a + m0 * g.lda, tile_bytes(min(g.M - m0, int64_t{BM}), g.lda, g.K));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.b + n0 * g.ldb, tile_bytes(min(g.N - n0, int64_t{BN}), g.ldb, g.K));
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem)));
    const int Kb = static_cast<int>((g.K + KS - 1) / KS);
    const int start = PAST ? tn % max(Kb, 1) : first_block(Kb);
    const auto block = [&](int i) { return i + start < Kb ? i + start : i + start - Kb; };  // the i-th

    // load p of a wave: kRows rows of A, or of B behind them
    uint32_t off[kLoads];
#pragma unroll
    for (int p = 0; p < kLoads; ++p) {
        const int r = wave * kLoads + p;
        const bool is_a = r < BM / kRows;
        const int row = kRows * (is_a ? r : r - BM / kRows) + lane / kChunks;
        off[p] = static_cast<uint32_t>(row * (is_a ? g.lda : g.ldb)) + 16 * ((lane % kChunks) ^ swizzle(row));
    }
    const auto issue = [&](int i, int stage) {
        const uint32_t k = i < Kb ? static_cast<uint32_t>(block(i) * KS) : kPastEnd;
#pragma unroll
        for (int p = 0; p < kLoads; ++p) {
            const int r = wave * kLoads + p;
            const uint32_t to = lds0 + static_cast<uint32_t>(stage * kStage + 64 * r) * 16;
            if (r < BM / kRows) dma16(to, ra, off[p] + k);
            else dma16<PAST>(to, rb, off[p] + k);
        }
    };

    i32x4 acc[kMS][kNS];
#pragma unroll
    for (int i = 0; i < kMS; ++i)
#pragma unroll
        for (int j = 0; j < kNS; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    if (Kb > 0) {
#pragma unroll
        for (int t = 0; t < STAGES - 1; ++t) issue(t, t);
    }
    const int sw = swizzle(l16);
    int stage = 0;
    for (int n = 0; n < Kb; ++n) {
        wait_loads<(STAGES - 2) * kLoads>();
        lds_barrier();  // the n-th block is there, and no wave reads the stage before it any more
        issue(n + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
        const u32x4* st = smem + stage * kStage;
        i32x4 a[KS / 64][kMS], b[KS / 64][kNS];
#pragma unroll
        for (int h = 0; h < KS / 64; ++h) {
            const int pos = (lg + 4 * h) ^ sw;
#pragma unroll
            for (int i = 0; i < kMS; ++i) a[h][i] = __builtin_bit_cast(i32x4, st[(WM * wm + 16 * i + l16) * kChunks + pos]);
#pragma unroll
            for (int j = 0; j < kNS; ++j) b[h][j] = __builtin_bit_cast(i32x4, st[(BM + WN * wn + 16 * j + l16) * kChunks + pos]);
        }
        const int64_t keep = g.K - static_cast<int64_t>(block(n)) * KS;
        if (keep < KS) {
#pragma unroll
            for (int h = 0; h < KS / 64; ++h)
#pragma unroll
                for (int i = 0; i < kMS; ++i) keep_bytes(a[h][i], static_cast<int>(keep) - 16 * (lg + 4 * h));
        }
#pragma unroll
        for (int h = 0; h < KS / 64; ++h)
#pragma unroll
            for (int i = 0; i < kMS; ++i)
#pragma unroll
                for (int j = 0; j < kNS; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[h][j], a[h][i], acc[i][j], 0, 0, 0);
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    wait_loads<0>();  // the last blocks' empty loads: none may land after the workgroup's LDS is given away

    lds_barrier();    // and no wave reads the stages any more
    static_assert(STAGES * kStage * 16 >= BM * BN * 2, "the tile of C fits the stages");
    store_block<WM, WN, false>(g, acc, m0 + WM * wm, n0 + WN * wn, reinterpret_cast<uint8_t*>(smem) + wave * (WM * WN * 2), lane);
}

// ---- 256 x 256 tiles, eight waves of 64 x 128 (two a SIMD), two stages of 128 bytes of K. A wave reads the
// fragments of half a block (64 bytes) while it multiplies the half before, and the one barrier a block comes
// after its first half: by then every wave has read the whole stage, so the loads of the block after next go
// there, a block's time before they are needed. 16384 x 5120 x 5120 358 to 381 us, 2.25 to 2.4 Pop/s (400 us with reads and
// products of a block in turn); 4096^3 65 us (67 with all workgroups beginning at one block); 8192^3 437 us, 2.51.
// Bound by power: the same loop over zeros takes 402. Not better: 32 x 32 x 32 instructions (488), a ring of five half
// blocks (473, in 6% fewer cycles at a lower clock), four waves of 128 x 128 (550).
constexpr int kBig = 256;
__global__ __launch_bounds__(512, 1) void big_kernel(I8Args g, int mt, int nt) {
    constexpr int WM = 64, WN = 128, kMS = WM / 16, kNS = WN / 16, kHalf = kBig * 8, kStage = 2 * kHalf;  // 16-byte units
    __shared__ u32x4 smem[2 * kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 3, wn = wave >> 2, l16 = lane & 15, lg = lane >> 4;
    int tm, tn;
    geom::tile_of(blockIdx.x, mt, nt, tm, tn);
    const int64_t m0 = static_cast<int64_t>(tm) * kBig, n0 = static_cast<int64_t>(tn) * kBig;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.a + m0 * g.lda, tile_bytes(min(g.M - m0, int64_t{kBig}), g.lda, g.K));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(g.b + n0 * g.ldb, tile_bytes(min(g.N - n0, int64_t{kBig}), g.ldb, g.K));
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem)));
    // the whole blocks, from first_block on and around, then the partial one
    const int Kb = static_cast<int>((g.K + kGroup - 1) / kGroup), whole = static_cast<int>(g.K / kGroup), start = first_block(whole);
    const auto block = [&](int i) { return i >= whole ? i : i + start < whole ? i + start : i + start - whole; };

    // a wave loads 32 rows of A and 32 of B a block, 8 a load; the chunk differs between even and odd loads
    uint32_t offa[2], offb[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        offa[q] = static_cast<uint32_t>((32 * wave + 8 * q + (lane >> 3)) * g.lda) + 16 * geom::fast_operand_chunk(q, lane);
        offb[q] = static_cast<uint32_t>((32 * wave + 8 * q + (lane >> 3)) * g.ldb) + 16 * geom::fast_operand_chunk(q, lane);
    }
    const uint32_t stepa = static_cast<uint32_t>(16 * g.lda), stepb = static_cast<uint32_t>(16 * g.ldb);
    const auto issue = [&](int i, int stage) {
        const uint32_t k = static_cast<uint32_t>(block(i) * kGroup), to = lds0 + static_cast<uint32_t>(stage * kStage + 256 * wave) * 16;
#pragma unroll
        for (int p = 0; p < 4; ++p) dma16(to + p * 1024, ra, offa[p & 1] + (p >> 1) * stepa + k);
#pragma unroll
        for (int p = 0; p < 4; ++p) dma16(to + kHalf * 16 + p * 1024, rb, offb[p & 1] + (p >> 1) * stepb + k);
    };

    i32x4 acc[kMS][kNS];
#pragma unroll
    for (int i = 0; i < kMS; ++i)
#pragma unroll
        for (int j = 0; j < kNS; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    if (Kb > 0) {
        const int sw = geom::lds_swizzle(l16);
        const u32x4* la = smem + (WM * wm + l16) * 8;
        const u32x4* lb = smem + kHalf + (WN * wn + l16) * 8;
        i32x4 a[2][kMS], b[2][kNS];
        const auto read = [&](int half, int stage) {
            const int at = stage * kStage + ((lg + 4 * half) ^ sw);
#pragma unroll
            for (int i = 0; i < kMS; ++i) a[half][i] = __builtin_bit_cast(i32x4, la[at + 128 * i]);
#pragma unroll
            for (int j = 0; j < kNS; ++j) b[half][j] = __builtin_bit_cast(i32x4, lb[at + 128 * j]);
        };
        const auto multiply = [&](int half) {
#pragma unroll
            for (int j = 0; j < kNS; ++j)
#pragma unroll
                for (int i = 0; i < kMS; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[half][j], a[half][i], acc[i][j], 0, 0, 0);
        };
        // twelve reads spread over the 32 products
        const auto spread = [&]() {
#pragma unroll
            for (int r = 0; r < kMS + kNS; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, kMS * kNS - kMS - kNS, 0);
            __builtin_amdgcn_sched_barrier(0);
        };
        issue(0, 0);
        wait_loads<0>();
        lds_barrier();
        if (Kb > 1) issue(1, 1);
        read(0, 0);
        const int left = whole < Kb ? static_cast<int>(g.K - static_cast<int64_t>(whole) * kGroup) : kGroup;  // bytes of the last block
        for (int kb = 0; kb < Kb - 1; ++kb) {
            const int s = kb & 1;
            __builtin_amdgcn_sched_barrier(0);
            read(1, s);
            multiply(0);
            spread();
            wait_loads<0>();
            lds_barrier();  // block kb + 1 is there, and no wave reads stage s any more
            if (kb + 2 < Kb) issue(kb + 2, s);
            __builtin_amdgcn_sched_barrier(0);
            read(0, s ^ 1);
            multiply(1);
            spread();
        }
        // the last block, of whose bytes `left` count
        read(1, (Kb - 1) & 1);
#pragma unroll
        for (int i = 0; i < kMS; ++i) {
            keep_bytes(a[0][i], left - 16 * lg);
            keep_bytes(a[1][i], left - 16 * (lg + 4));
        }
        multiply(0);
        multiply(1);
    }

    lds_barrier();
    store_block<WM, WN, true>(g, acc, m0 + WM * wm, n0 + WN * wn, reinterpret_cast<uint8_t*>(smem) + wave * (WM * WN * 2), lane);
}

// ---- One to four rows of A: four columns a workgroup, whose waves take a KB of each in turn, 16 bytes a lane,
// and add products of four bytes. B is read once, past the caches, in pieces of a KB: one row, 14336 x 4096
// 10.5 us, 5.6 TB/s (14.2 in 16-row tiles whose loads read 256 bytes of a row).
constexpr int kCols = 4, kPiece = 1024;
template <int ROWS>
__global__ __launch_bounds__(256) void rows_kernel(I8Args g) {
    __shared__ int part[4][kCols][ROWS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kCols;
    const uint8_t* pb[kCols];
#pragma unroll
    for (int r = 0; r < kCols; ++r) pb[r] = g.b + min(n0 + r, g.N - 1) * g.ldb;
    int acc[kCols][ROWS] = {};
    const int K = static_cast<int>(g.K);
    for (int k0 = wave * kPiece; k0 < K; k0 += 4 * kPiece) {
        const int k = k0 + 16 * lane, at = k < K ? k : 0;
        i32x4 a[ROWS], b[kCols];
#pragma unroll
        for (int r = 0; r < kCols; ++r) b[r] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pb[r] + at));
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
            a[m] = *reinterpret_cast<const i32x4*>(g.a + m * g.lda + at);
            keep_bytes(a[m], K - k);
        }
#pragma unroll
        for (int r = 0; r < kCols; ++r)
#pragma unroll
            for (int m = 0; m < ROWS; ++m)
#pragma unroll
                for (int d = 0; d < 4; ++d) acc[r][m] = __builtin_amdgcn_sdot4(a[m][d], b[r][d], acc[r][m], false);
    }
#pragma unroll
    for (int r = 0; r < kCols; ++r)
#pragma unroll
        for (int m = 0; m < ROWS; ++m) {
            int v = acc[r][m];
            v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false);   // the pair's other lane
            v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false);   // the other pair of four
            v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false);  // the other four of eight
            v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false);  // the other eight of sixteen
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            if (lane == 0) part[wave][r][m] = v;
        }
    __syncthreads();
    if (threadIdx.x < kCols * ROWS) {
        const int r = threadIdx.x % kCols, m = threadIdx.x / kCols;
        const int64_t n = n0 + r;
        if (n < g.N) {
            const int sum = part[0][r][m] + part[1][r][m] + part[2][r][m] + part[3][r][m];
            const float v = K > 0 ? (static_cast<float>(sum) * g.a_s[m]) * g.b_s[n] : 0.0f;
            g.c[m * g.ldc + n] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
        }
    }
}

}  // namespace

hipError_t launch_gemm_i8(const I8Args& g, int cus, hipStream_t stream) {
    const sched::I8Kernel kernel = sched::i8_kernel(g.M, g.N, g.K, cus);
    const sched::I8Tile tile = sched::kI8Tiles[kernel];
    const int mt = static_cast<int>(sched::cdiv(g.M, tile.bm)), nt = static_cast<int>(sched::cdiv(g.N, tile.bn));
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(mt) * nt);
    const bool past = sched::i8_reads_once(g.M, g.N, kernel, cus);
#define BSFP8_TILE(BM, BN, WM, WN, STAGES, KS)                                                                      \
    do {                                                                                                            \
        constexpr int kThreads = 64 * (BM / WM) * (BN / WN);                                                        \
        if (past) tile_kernel<BM, BN, WM, WN, STAGES, KS, true><<<grid, kThreads, 0, stream>>>(g, mt, nt);   \
        else tile_kernel<BM, BN, WM, WN, STAGES, KS, false><<<grid, kThreads, 0, stream>>>(g, mt, nt);       \
    } while (0)
    switch (kernel) {
        case sched::kI8Rows:
            switch (g.M) {
                case 1: rows_kernel<1><<<grid, 256, 0, stream>>>(g); break;
                case 2: rows_kernel<2><<<grid, 256, 0, stream>>>(g); break;
                case 3: rows_kernel<3><<<grid, 256, 0, stream>>>(g); break;
                default: rows_kernel<4><<<grid, 256, 0, stream>>>(g); break;
            }
            break;
        case sched::kI8Tile32x32: BSFP8_TILE(32, 32, 16, 16, 4, 256); break;
        case sched::kI8Tile32x64: BSFP8_TILE(32, 64, 32, 16, 3, 256); break;
        case sched::kI8Tile64x64: BSFP8_TILE(64, 64, 16, 32, 4, 256); break;
        case sched::kI8Tile64x128: tile_kernel<64, 128, 32, 32, 3, 128, false><<<grid, 512, 0, stream>>>(g, mt, nt); break;
        case sched::kI8Tile128x128: tile_kernel<128, 128, 32, 64, 4, 128, false><<<grid, 512, 0, stream>>>(g, mt, nt); break;
        case sched::kI8Tile128x128Two: tile_kernel<128, 128, 32, 64, 2, 128, false><<<grid, 512, 0, stream>>>(g, mt, nt); break;
        default: big_kernel<<<grid, 512, 0, stream>>>(g, mt, nt); break;
    }
#undef BSFP8_TILE
    return hipGetLastError();
}

}  // namespace bsfp8
