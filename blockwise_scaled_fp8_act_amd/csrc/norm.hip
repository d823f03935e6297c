// gfx950 root-mean-square norm with the residual's addition and 8-bit codes, and its gradient:
//   h = x + residual (rounded to the residual's type, or x itself);  r = 1 / sqrt(mean(h^2) + eps);
//   v = (h r) w in fp32, written as e4m3 codes with 1x128 scales, as int8 rows, or in bf16.
// The sum of squares is in 64 bits: a bf16 value's square has no room in fp32 from 1.8e19 on, and the
// conversions cost nothing next to the memory traffic that bounds these kernels. Measured: 16384 x 5120 bf16 with
// residual, codes and a bf16 copy 147 us, 5.1 TB/s (a device copy reaches 5.2); 8192 x 4096 with an fp32 residual 75 us
// (4.9 TB/s), the 128x1 codes 26 (6.4, h partly in the last-level cache), the gradient 82 (5.8) and the weight's sum 4.8;
// one row 2.9.
#include "row_codes.hpp"
#include "schedule.hpp"
#include "tile_codes.hpp"

namespace bsfp8 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
enum { kResNone = 0, kResBf16 = 1, kResF32 = 2 };

// 1 / sqrt(sum / H + eps), rounded to fp32: the instruction's 2^-23 squared by one step of Newton's method. A square
// root and a division in 64 bits are sixty instructions, for which every row waits (3000 x 1280 8.0 -> 7.2 us, one row
// of 4096 3.1 -> 2.9).
__device__ __forceinline__ float rstd_of(double sum, double per_column, float eps) {
    const double m = fma(sum, per_column, static_cast<double>(eps)), y = __builtin_amdgcn_rsq(m);
    const double e = fma(-m * y, y, 1.0);
    return static_cast<float>(isinf(m) ? 0.0 : fma(0.5 * y, e, y));
}

// v = (h r) w, rounded after each product
__device__ __forceinline__ float normed(float h, float r, float w) { return (h * r) * w; }

// A row of TPR threads, NC pieces of 8 columns each, held in registers: H <= 8 TPR NC. 256 / TPR rows a workgroup. ANY:
// rows that begin anywhere, of any length; without it all rows in 16-byte pieces (codes in 8-byte ones).
template <int RES, int TPR, int NC, bool ANY>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a, RowCodes out) {
    __shared__ double part[kWaves];
    __shared__ uint32_t part_max[kWaves];
    constexpr int kRows = kThreads / TPR;
    const int tid = threadIdx.x % TPR;
    const int64_t row = xcd_block(blockIdx.x, a.per_xcd) * kRows + threadIdx.x / TPR;
    if (row >= a.T) return;  // a whole wave, and with more than one wave a row the whole workgroup

    rc_u32x4 xw[NC];
    float h[NC][8], w[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = c < a.H ? c : 0, n = a.H - c;
        xw[i] = load8_bf16<true, ANY>(a.x + row * a.ldx + at, n);
        if (RES != kResNone) load8_of<RES == kResF32, true, ANY>(a.residual, row * a.ldr + at, h[i], n);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = c < a.H ? c : 0;
        if (a.w_f32) load8_of<true, false, ANY>(a.weight, at, w[i], a.H - c);
        else load8_of<false, false, ANY>(a.weight, at, w[i], a.H - c);
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
        float x[8];
        unpack8(xw[i], x);
        if (RES == kResNone) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = x[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += x[j];
            if (RES == kResBf16) {  // the sum as it is kept
                const rc_u32x4 k = pack8(h[i]);
                unpack8(k, h[i]);
                if (c < a.H) store8_bf16<ANY>(static_cast<uint16_t*>(a.h) + row * a.ldh + c, k, a.H - c);
            } else if (c < a.H) {
                store8_of<true, ANY>(a.h, row * a.ldh + c, h[i], a.H - c);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c >= a.H) h[i][j] = 0.0f;
            const double d = h[i][j];
            sum = fma(d, d, sum);
        }
    }
    const float r = rstd_of(block_sum<TPR / 64>(sum, part), a.per_column, a.eps);
    if (a.rstd != nullptr && tid == 0) a.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = c + (ANY ? j : 0) < a.H ? normed(h[i][j], r, w[i][j]) : 0.0f;
    }
    emit_row<TPR, NC, ANY>(out, row, a.T, a.H, tid, h, part_max);
}

// Longer rows: a workgroup each, which is read again for each pass. A thread reads
// back the sums that it wrote itself (a wave takes the same 128 columns in every pass).
template <int RES>
__global__ __launch_bounds__(kThreads) void norm_long_kernel(NormArgs a, RowCodes out) {
    __shared__ double part[kWaves];
    __shared__ uint32_t part_max[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    double sum = 0.0;
    for (int64_t c0 = wave * kGroup; c0 < a.H; c0 += kWaves * kGroup)
        for (int j = 0; j < 2; ++j) {
            const int64_t c = c0 + 64 * j + lane;
            if (c >= a.H) continue;
            float h = bf16_to_f32(a.x[row * a.ldx + c]);
            if (RES == kResBf16) {
                const uint16_t k = to_bf16_bits(h + bf16_to_f32(static_cast<const uint16_t*>(a.residual)[row * a.ldr + c]));
                static_cast<uint16_t*>(a.h)[row * a.ldh + c] = k;
                h = bf16_to_f32(k);
            } else if (RES == kResF32) {
                h += static_cast<const float*>(a.residual)[row * a.ldr + c];
                static_cast<float*>(a.h)[row * a.ldh + c] = h;
            }
            const double d = h;
            sum = fma(d, d, sum);
        }
    const float r = rstd_of(block_sum<kWaves>(sum, part), a.per_column, a.eps);
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = r;
    const auto value = [&](int64_t c) {
        const float h = RES == kResNone ? bf16_to_f32(a.x[row * a.ldx + c]) : load_of(a.h, row * a.ldh + c, RES == kResF32);
        return normed(h, r, load_of(a.weight, c, a.w_f32));
    };
    emit_row_any<kWaves>(out, row, a.T, a.H, value, part_max);
}

// The normed rows in 128x1 groups, transposed: v is formed again from h and r.
template <bool FNUZ, bool H_F32, bool WHOLE>
__global__ __launch_bounds__(kTileThreads) void norm_rhs_kernel(const void* h, int64_t ldh, const void* weight, bool w_f32,
                                                               const float* rstd, int64_t T, int64_t H, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    float v[kTileRows][8], w[8], r[kTileRows];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) r[i] = rstd[row + i < T ? row + i : 0];
    if (w_f32) load8_of<true, false, true>(weight, c < H ? c : 0, w, H - c);
    else load8_of<false, false, true>(weight, c < H ? c : 0, w, H - c);
    if constexpr (H_F32) {
        load_tile<WHOLE>(static_cast<const float*>(h), ldh, row, T, c0, c, H, v);
    } else {
        rc_u32x4 k[kTileRows];
        load_tile<WHOLE>(static_cast<const uint16_t*>(h), ldh, row, T, c0, c, H, k);
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) unpack8(k[i], v[i]);
    }
#pragma unroll
    for (int i = 0; i < kTileRows; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = row + i < T && c + j < H ? normed(v[i][j], r[i], w[j]) : 0.0f;
    emit_tile<FNUZ, false>(out, r0, c0, T, H, v, lds);
}

// Eight values as they lie in memory.
template <bool F32>
struct Held {
    rc_u32x4 w;
    template <bool ANY>
    __device__ __forceinline__ void load(const void* p, int64_t at, int64_t n) {
        w = load8_bf16<false, ANY>(static_cast<const uint16_t*>(p) + at, n);
    }
    __device__ __forceinline__ void values(float (&f)[8]) const { unpack8(w, f); }
};
template <>
struct Held<true> {
    float v[8];
    template <bool ANY>
    __device__ __forceinline__ void load(const void* p, int64_t at, int64_t n) {
        load8_of<true, false, ANY>(p, at, v, n);
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[j];
    }
};

// Gradient. With g = dy w and n = h r: dx = dh + r (g - n mean(g n)), dw = sum over the rows of dy n. TPR threads
// take a row at a time, NC pieces of 8 columns each, and keep their part of dw in registers; a workgroup's rows, 256 /
// TPR side by side, are every gridDim-th. Its parts are added in order of the waves, those of the workgroups by the
// second kernel, in order too. Rows of up to kRowWaveMax columns take a wave, which waits for no other (16384 x 1000
// 27 us, 58 with a workgroup a row; 3000 x 1000 7.9 and 12); longer ones gain nothing by it (8192 x 2048 in fp32 45 and 39).
// The next row's loads are on the way while a row is summed, where the registers hold both (8192 x 2048 33 -> 25 us,
// 8192 x 4096 50 -> 46). ANY as in norm_kernel.
template <bool H_F32, int TPR, int NC, bool ANY>
__global__ __launch_bounds__(kThreads) void norm_backward_kernel(NormBackwardArgs a) {
    constexpr int kRows = kThreads / TPR;
    constexpr bool kAhead = NC <= 2;
    __shared__ float part[2][kWaves];
    __shared__ alignas(16) float sums[kRows > 1 ? kRows : 1][kRows > 1 ? 8 * TPR * NC : 1];
    const int tid = threadIdx.x % TPR, side = threadIdx.x / TPR;
    float w[NC][8], dw[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = c < a.H ? c : 0;
        if (a.w_f32) load8_of<true, false, ANY>(a.weight, at, w[i], a.H - c);
        else load8_of<false, false, ANY>(a.weight, at, w[i], a.H - c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = 0.0f;
            if (!ANY && c >= a.H) w[i][j] = 0.0f;
        }
    }
    rc_u32x4 dy_next[NC];
    Held<H_F32> h_next[NC], dh_next[NC];
    float r_next = 0.0f;
    const auto load = [&](int64_t row) {
        r_next = a.rstd[row];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = c < a.H ? c : 0;
            dy_next[i] = load8_bf16<false, ANY>(a.dy + row * a.lddy + at, a.H - c);
            h_next[i].template load<ANY>(a.h, row * a.ldh + at, a.H - c);
            if (a.dh != nullptr) dh_next[i].template load<ANY>(a.dh, row * a.lddh + at, a.H - c);
        }
    };
    const int64_t step = kRows * static_cast<int64_t>(gridDim.x);
    int64_t row = blockIdx.x + static_cast<int64_t>(side) * gridDim.x;
    if (kAhead && row < a.T) load(row);
    for (int turn = 0; row < a.T; row += step, turn ^= 1) {
        if (!kAhead) load(row);
        const float r = r_next;
        float n[NC][8], dy[NC][8], dh[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            unpack8(dy_next[i], dy[i]);
            h_next[i].values(n[i]);
            if (a.dh != nullptr) dh_next[i].values(dh[i]);
        }
        if (kAhead && row + step < a.T) load(row + step);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[i][j] *= r;
                if (c + (ANY ? j : 0) >= a.H) n[i][j] = dy[i][j] = 0.0f;
                dw[i][j] = fmaf(dy[i][j], n[i][j], dw[i][j]);
                sum = fmaf(dy[i][j] * w[i][j], n[i][j], sum);
            }
        }
        // two buffers in turn: the next row's sums are written before every wave has read these
        const float mean = block_sum<TPR / 64>(sum, part[turn]) / static_cast<float>(a.H);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = r * (dy[i][j] * w[i][j] - n[i][j] * mean);
                if (a.dh != nullptr) d[j] += dh[i][j];
            }
            if (c < a.H) store8_of<H_F32, ANY>(a.dx, row * a.lddx + c, d, a.H - c);
        }
    }
    float* out = a.partial + blockIdx.x * a.H;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
            if (c < a.H) store8_of<true, ANY>(out, c, dw[i], a.H - c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) store8_of<true>(sums[side], 8 * (i * TPR + tid), dw[i]);
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += kThreads) {
            float sum = sums[0][c];
#pragma unroll
            for (int k = 1; k < kRows; ++k) sum += sums[k][c];
            out[c] = sum;
        }
    }
}

// Longer rows: the parts of dw are kept in memory, a column always by one thread.
template <bool H_F32>
__global__ __launch_bounds__(kThreads) void norm_backward_long_kernel(NormBackwardArgs a) {
    __shared__ float part[2][kWaves];
    float* dw = a.partial + blockIdx.x * a.H;
    for (int64_t c = threadIdx.x; c < a.H; c += kThreads) dw[c] = 0.0f;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const float r = a.rstd[row];
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < a.H; c += kThreads) {
            const float dy = bf16_to_f32(a.dy[row * a.lddy + c]), n = load_of(a.h, row * a.ldh + c, H_F32) * r;
            dw[c] = fmaf(dy, n, dw[c]);
            sum = fmaf(dy * load_of(a.weight, c, a.w_f32), n, sum);
        }
        const float mean = block_sum<kWaves>(sum, part[turn]) / static_cast<float>(a.H);
        for (int64_t c = threadIdx.x; c < a.H; c += kThreads) {
            const float dy = bf16_to_f32(a.dy[row * a.lddy + c]), n = load_of(a.h, row * a.ldh + c, H_F32) * r;
            float d = r * (dy * load_of(a.weight, c, a.w_f32) - n * mean);
            if (a.dh != nullptr) d += load_of(a.dh, row * a.lddh + c, H_F32);
            if (H_F32) static_cast<float*>(a.dx)[row * a.lddx + c] = d;
            else static_cast<uint16_t*>(a.dx)[row * a.lddx + c] = to_bf16_bits(d);
        }
    }
}

// dw[c] = the sum of the G parts of column c: 16 columns a workgroup, 64 runs of parts side by side.
constexpr int kSumCols = 16, kSumRuns = 64, kSumEach = 8;
__global__ __launch_bounds__(kSumCols* kSumRuns) void norm_weight_kernel(const float* partial, int64_t G, int64_t H, void* dweight, bool w_f32) {
    __shared__ float part[kSumRuns][kSumCols + 1];
    const int col = threadIdx.x % kSumCols, run = threadIdx.x / kSumCols;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kSumCols + col;
    static_assert(sched::kNormBackwardBlocks == kSumRuns * kSumEach, "a run's parts are on the way together");
    float v[kSumEach];
#pragma unroll
    for (int k = 0; k < kSumEach; ++k) {
        const int64_t g = run + k * kSumRuns;
        v[k] = g < G && c < H ? partial[g * H + c] : 0.0f;
    }
    float sum = v[0];
#pragma unroll
    for (int k = 1; k < kSumEach; ++k) sum += v[k];
    part[run][col] = sum;
    __syncthreads();
    if (run != 0 || c >= H) return;
#pragma unroll 8
    for (int i = 1; i < kSumRuns; ++i) sum += part[i][col];
    if (w_f32) static_cast<float*>(dweight)[c] = sum;
    else static_cast<uint16_t*>(dweight)[c] = to_bf16_bits(sum);
}

template <int RES, bool ANY>
void launch_rows(NormArgs a, const RowCodes& out, hipStream_t stream) {
    const bool wave = a.H <= sched::kRowWaveMax;
    const int64_t blocks = wave ? (a.T + kWaves - 1) / kWaves : a.T;
    a.per_xcd = (blocks + kXcds - 1) / kXcds;
    const unsigned grid = static_cast<unsigned>(a.per_xcd * kXcds);
#define BSFP8_NORM(TPR, NC) norm_kernel<RES, TPR, NC, ANY><<<grid, kThreads, 0, stream>>>(a, out)
    if (wave) {
        if (a.H <= 512) BSFP8_NORM(64, 1);
        else BSFP8_NORM(64, 2);
    } else {
        switch ((a.H + 2047) / 2048) {
            case 1: BSFP8_NORM(256, 1); break;
            case 2: BSFP8_NORM(256, 2); break;
            case 3: BSFP8_NORM(256, 3); break;
            case 4: BSFP8_NORM(256, 4); break;
            case 5: case 6: BSFP8_NORM(256, 6); break;
            default: BSFP8_NORM(256, 8); break;
        }
    }
#undef BSFP8_NORM
}

template <int RES>
hipError_t launch_res(const NormArgs& a, const RowCodes& out, hipStream_t stream) {
    const int64_t rs = RES == kResF32 ? 4 : 2;
    const bool whole = a.H % 8 == 0 && rows16(a.x, 2 * a.ldx) && rows16(a.weight, 0) && whole_codes(out) &&
                       (RES == kResNone || (rows16(a.residual, rs * a.ldr) && rows16(a.h, rs * a.ldh)));
    if (a.H > sched::kRowMax) norm_long_kernel<RES><<<static_cast<unsigned>(a.T), kThreads, 0, stream>>>(a, out);
    else if (whole) launch_rows<RES, false>(a, out, stream);
    else launch_rows<RES, true>(a, out, stream);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(NormArgs a, const RowCodes& out, hipStream_t stream) {
    a.per_column = 1.0 / static_cast<double>(a.H);
    if (a.residual == nullptr) return launch_res<kResNone>(a, out, stream);
    return a.res_f32 ? launch_res<kResF32>(a, out, stream) : launch_res<kResBf16>(a, out, stream);
}

hipError_t launch_rms_norm_rhs(const void* h, bool h_f32, int64_t ldh, const void* weight, bool w_f32, const float* rstd, int64_t T,
                               int64_t H, uint8_t* qT, int64_t ldqT, float* s, bool fnuz, hipStream_t stream) {
    const TileCodes out{nullptr, 0, nullptr, qT, ldqT, s};
    const dim3 grid(static_cast<unsigned>((H + kGroup - 1) / kGroup), static_cast<unsigned>((T + kGroup - 1) / kGroup));
    const auto go = [&](auto fz, auto f32) {
        constexpr bool FZ = decltype(fz)::value, F32 = decltype(f32)::value;
        if (H % kGroup == 0) norm_rhs_kernel<FZ, F32, true><<<grid, kTileThreads, 0, stream>>>(h, ldh, weight, w_f32, rstd, T, H, out);
        else norm_rhs_kernel<FZ, F32, false><<<grid, kTileThreads, 0, stream>>>(h, ldh, weight, w_f32, rstd, T, H, out);
    };
    if (fnuz) h_f32 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    else h_f32 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, bool h_f32, hipStream_t stream) {
    const int64_t hs = h_f32 ? 4 : 2, G = sched::norm_backward_blocks(a.T);
    const bool whole = a.H % 8 == 0 && rows16(a.dy, 2 * a.lddy) && rows16(a.h, hs * a.ldh) && rows16(a.weight, 0) &&
                       (a.dh == nullptr || rows16(a.dh, hs * a.lddh)) && rows16(a.dx, hs * a.lddx);
    const unsigned grid = static_cast<unsigned>(G);
    const auto rows = [&](auto f32, auto any) {
        constexpr bool F32 = decltype(f32)::value, ANY = decltype(any)::value;
#define BSFP8_BACKWARD(TPR, NC) norm_backward_kernel<F32, TPR, NC, ANY><<<grid, kThreads, 0, stream>>>(a)
        if (a.H <= 512) BSFP8_BACKWARD(64, 1);
        else if (a.H <= sched::kRowWaveMax) BSFP8_BACKWARD(64, 2);
        else if (a.H <= 2048) BSFP8_BACKWARD(256, 1);
        else if (a.H <= 4096) BSFP8_BACKWARD(256, 2);
        else if (a.H <= 3 * 2048) BSFP8_BACKWARD(256, 3);
        else if (a.H <= 8192) BSFP8_BACKWARD(256, 4);
        else BSFP8_BACKWARD(256, 8);
#undef BSFP8_BACKWARD
    };
    const auto go = [&](auto f32) {
        if (a.H > sched::kRowMax) norm_backward_long_kernel<decltype(f32)::value><<<grid, kThreads, 0, stream>>>(a);
        else if (whole) rows(f32, std::false_type{});
        else rows(f32, std::true_type{});
    };
    if (G > 0) h_f32 ? go(std::true_type{}) : go(std::false_type{});  // without rows only the weight's gradient, 0, is written
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm_weight_kernel<<<static_cast<unsigned>((a.H + kSumCols - 1) / kSumCols), kSumCols * kSumRuns, 0, stream>>>(a.partial, G, a.H, a.dweight,
                                                                                                                   a.w_f32);
    return hipGetLastError();
}

}  // namespace bsfp8
