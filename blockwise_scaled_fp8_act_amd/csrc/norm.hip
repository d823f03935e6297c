// gfx950 root-mean-square norm with the residual's addition and 8-bit codes, and its gradient:
//   h = x + residual (rounded to the residual's type, or x itself);  r = 1 / sqrt(mean(h^2) + eps);
//   v = (h r) w in fp32, written as e4m3 codes with 1x128 scales, as int8 rows, or in bf16.
// The sum of squares is in 64 bits: a bf16 value's square has no room in fp32 from 1.8e19 on, and the
// conversions cost nothing next to the memory traffic that bounds these kernels.
#include "row_codes.hpp"
#include "schedule.hpp"
#include "tile_codes.hpp"

namespace bsfp8 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
enum { kResNone = 0, kResBf16 = 1, kResF32 = 2 };

// 1 / sqrt(sum / H + eps), rounded to fp32.
__device__ __forceinline__ float rstd_of(double sum, int64_t H, float eps) {
    return static_cast<float>(1.0 / sqrt(sum / static_cast<double>(H) + static_cast<double>(eps)));
}

// v = (h r) w, rounded after each product
__device__ __forceinline__ float normed(float h, float r, float w) { return (h * r) * w; }

// A row of TPR threads, NC pieces of 8 columns each, held in registers: H <= 8 TPR NC, everything in
// 16-byte pieces. 256 / TPR rows a workgroup.
template <int RES, int TPR, int NC>
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
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = c < a.H ? c : 0;
        xw[i] = load_piece<true>(reinterpret_cast<const rc_u32x4*>(a.x + row * a.ldx + at));
        if (RES != kResNone) load8_of<RES == kResF32, true>(a.residual, row * a.ldr + at, h[i]);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid), at = c < a.H ? c : 0;
        if (a.w_f32) load8_of<true>(a.weight, at, w[i]);
        else load8_of<false>(a.weight, at, w[i]);
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
                const rc_u32x4 k = {pack_bf16(h[i][0], h[i][1]), pack_bf16(h[i][2], h[i][3]), pack_bf16(h[i][4], h[i][5]),
                                    pack_bf16(h[i][6], h[i][7])};
                unpack8(k, h[i]);
                if (c < a.H) *reinterpret_cast<rc_u32x4*>(static_cast<uint16_t*>(a.h) + row * a.ldh + c) = k;
            } else if (c < a.H) {
                store8_of<true>(a.h, row * a.ldh + c, h[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c >= a.H) h[i][j] = 0.0f;
            const double d = h[i][j];
            sum = fma(d, d, sum);
        }
    }
    const float r = rstd_of(block_sum<TPR / 64>(sum, part), a.H, a.eps);
    if (a.rstd != nullptr && tid == 0) a.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const bool in = 8 * (static_cast<int64_t>(i) * TPR + tid) < a.H;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = in ? normed(h[i][j], r, w[i][j]) : 0.0f;
    }
    emit_row<TPR, NC>(out, row, a.T, a.H, tid, h, part_max);
}

// Any length, stride and alignment: a workgroup a row, which is read again for each pass. A thread reads
// back the sums that it wrote itself (a wave takes the same 128 columns in every pass).
template <int RES>
__global__ __launch_bounds__(kThreads) void norm_any_kernel(NormArgs a, RowCodes out) {
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
    const float r = rstd_of(block_sum<kWaves>(sum, part), a.H, a.eps);
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = r;
    const auto value = [&](int64_t c) {
        const float h = RES == kResNone ? bf16_to_f32(a.x[row * a.ldx + c]) : load_of(a.h, row * a.ldh + c, RES == kResF32);
        return normed(h, r, load_of(a.weight, c, a.w_f32));
    };
    emit_row_any<kWaves>(out, row, a.T, a.H, value, part_max);
}

// The normed rows in 128x1 groups, transposed: v is formed again from h and r.
template <bool FNUZ, bool H_F32, bool VEC_X, bool VEC_T>
__global__ __launch_bounds__(kTileThreads) void norm_rhs_kernel(const void* h, int64_t ldh, const void* weight, bool w_f32,
                                                               const float* rstd, int64_t T, int64_t H, TileCodes out) {
    __shared__ TileLds lds;
    const int t = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
    const int64_t row = r0 + (t >> 4) * kTileRows, c = c0 + (t & 15) * 8;
    float v[kTileRows][8], w[8], r[kTileRows];
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        const bool in = row + i < T;
        r[i] = in ? rstd[row + i] : 0.0f;
        if (VEC_X) {
            load8_of<H_F32>(h, in && c < H ? (row + i) * ldh + c : 0, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = in && c + j < H ? load_of(h, (row + i) * ldh + c + j, H_F32) : 0.0f;
        }
    }
    if (VEC_X) {
        if (w_f32) load8_of<true>(weight, c < H ? c : 0, w);
        else load8_of<false>(weight, c < H ? c : 0, w);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = c + j < H ? load_of(weight, c + j, w_f32) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kTileRows; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = row + i < T && c + j < H ? normed(v[i][j], r[i], w[j]) : 0.0f;
    emit_tile<FNUZ, false, false, VEC_T>(out, r0, c0, T, H, v, lds);
}

// Gradient. With g = dy w and n = h r: dx = dh + r (g - n mean(g n)), dw = sum over the rows of dy n. A
// workgroup takes every gridDim-th row and keeps its part of dw in registers (NC pieces of 8 columns a
// thread); the parts are added by the second kernel, in order.
template <bool H_F32, int NC>
__global__ __launch_bounds__(kThreads) void norm_backward_kernel(NormBackwardArgs a) {
    __shared__ float part[2][kWaves];
    const int tid = threadIdx.x;
    float w[NC][8], dw[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * kThreads + tid), at = c < a.H ? c : 0;
        if (a.w_f32) load8_of<true>(a.weight, at, w[i]);
        else load8_of<false>(a.weight, at, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = 0.0f;
            if (c >= a.H) w[i][j] = 0.0f;
        }
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
        const float r = a.rstd[row];
        float n[NC][8], dy[NC][8], dh[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * kThreads + tid), at = c < a.H ? c : 0;
            load8_of<false>(a.dy, row * a.lddy + at, dy[i]);
            load8_of<H_F32>(a.h, row * a.ldh + at, n[i]);
            if (a.dh != nullptr) load8_of<H_F32>(a.dh, row * a.lddh + at, dh[i]);
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const bool in = 8 * (static_cast<int64_t>(i) * kThreads + tid) < a.H;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[i][j] *= r;
                if (!in) n[i][j] = dy[i][j] = 0.0f;
                dw[i][j] = fmaf(dy[i][j], n[i][j], dw[i][j]);
                sum = fmaf(dy[i][j] * w[i][j], n[i][j], sum);
            }
        }
        // two buffers in turn: the next row's sums are written before every wave has read these
        const float mean = block_sum<kWaves>(sum, part[turn]) / static_cast<float>(a.H);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * kThreads + tid);
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = r * (dy[i][j] * w[i][j] - n[i][j] * mean);
                if (a.dh != nullptr) d[j] += dh[i][j];
            }
            if (c < a.H) store8_of<H_F32>(a.dx, row * a.lddx + c, d);
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * kThreads + tid);
        if (c < a.H) store8_of<true>(a.partial, blockIdx.x * a.H + c, dw[i]);
    }
}

// Any length, stride and alignment: the parts of dw are kept in memory, a column always by one thread.
template <bool H_F32>
__global__ __launch_bounds__(kThreads) void norm_backward_any_kernel(NormBackwardArgs a) {
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

bool rows16(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bytes % 16 == 0; }
bool rows8(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && bytes % 8 == 0; }

bool codes_vec(const RowCodes& o) {
    return (o.codes == kCodesNone || rows8(o.q, o.ldq)) && (o.y == nullptr || rows16(o.y, 2 * o.ldy));
}

template <int RES>
hipError_t launch_res(NormArgs a, const RowCodes& out, hipStream_t stream) {
    const bool vec = a.H % 8 == 0 && a.H <= sched::kRowMax && rows16(a.x, 2 * a.ldx) && rows16(a.weight, 0) && codes_vec(out) &&
                     (RES == kResNone || (rows16(a.residual, (RES == kResF32 ? 4 : 2) * a.ldr) && rows16(a.h, (RES == kResF32 ? 4 : 2) * a.ldh)));
    if (!vec) {
        norm_any_kernel<RES><<<static_cast<unsigned>(a.T), kThreads, 0, stream>>>(a, out);
        return hipGetLastError();
    }
    const bool wave = a.H <= sched::kRowWaveMax;
    const int64_t blocks = wave ? (a.T + kWaves - 1) / kWaves : a.T;
    a.per_xcd = (blocks + kXcds - 1) / kXcds;
    const unsigned grid = static_cast<unsigned>(a.per_xcd * kXcds);
#define BSFP8_NORM(TPR, NC) norm_kernel<RES, TPR, NC><<<grid, kThreads, 0, stream>>>(a, out)
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
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(NormArgs a, const RowCodes& out, hipStream_t stream) {
    if (a.residual == nullptr) return launch_res<kResNone>(a, out, stream);
    return a.res_f32 ? launch_res<kResF32>(a, out, stream) : launch_res<kResBf16>(a, out, stream);
}

hipError_t launch_rms_norm_rhs(const void* h, bool h_f32, int64_t ldh, const void* weight, bool w_f32, const float* rstd, int64_t T,
                               int64_t H, uint8_t* qT, int64_t ldqT, float* s, bool fnuz, hipStream_t stream) {
    const bool vx = H % 8 == 0 && rows16(h, (h_f32 ? 4 : 2) * ldh) && rows16(weight, 0), vt = T % 16 == 0 && rows16(qT, ldqT);
    const TileCodes out{nullptr, 0, nullptr, qT, ldqT, s};
    const dim3 grid(static_cast<unsigned>((H + kGroup - 1) / kGroup), static_cast<unsigned>((T + kGroup - 1) / kGroup));
    const auto go = [&](auto fz, auto f32) {
        constexpr bool FZ = decltype(fz)::value, F32 = decltype(f32)::value;
        if (vx && vt) norm_rhs_kernel<FZ, F32, true, true><<<grid, kTileThreads, 0, stream>>>(h, ldh, weight, w_f32, rstd, T, H, out);
        else if (vx) norm_rhs_kernel<FZ, F32, true, false><<<grid, kTileThreads, 0, stream>>>(h, ldh, weight, w_f32, rstd, T, H, out);
        else norm_rhs_kernel<FZ, F32, false, false><<<grid, kTileThreads, 0, stream>>>(h, ldh, weight, w_f32, rstd, T, H, out);
    };
    if (fnuz) h_f32 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    else h_f32 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, bool h_f32, hipStream_t stream) {
    const int64_t hs = h_f32 ? 4 : 2, G = sched::norm_backward_blocks(a.T);
    const bool vec = a.H % 8 == 0 && a.H <= sched::kRowMax && rows16(a.dy, 2 * a.lddy) && rows16(a.h, hs * a.ldh) && rows16(a.weight, 0) &&
                     (a.dh == nullptr || rows16(a.dh, hs * a.lddh)) && rows16(a.dx, hs * a.lddx) && rows16(a.partial, 0);
    const unsigned grid = static_cast<unsigned>(G);
    const auto go = [&](auto f32) {
        constexpr bool F32 = decltype(f32)::value;
        if (!vec) norm_backward_any_kernel<F32><<<grid, kThreads, 0, stream>>>(a);
        else if (a.H <= 2048) norm_backward_kernel<F32, 1><<<grid, kThreads, 0, stream>>>(a);
        else if (a.H <= 4096) norm_backward_kernel<F32, 2><<<grid, kThreads, 0, stream>>>(a);
        else if (a.H <= 3 * 2048) norm_backward_kernel<F32, 3><<<grid, kThreads, 0, stream>>>(a);
        else if (a.H <= 8192) norm_backward_kernel<F32, 4><<<grid, kThreads, 0, stream>>>(a);
        else norm_backward_kernel<F32, 8><<<grid, kThreads, 0, stream>>>(a);
    };
    if (G > 0) h_f32 ? go(std::true_type{}) : go(std::false_type{});  // without rows only the weight's gradient, 0, is written
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm_weight_kernel<<<static_cast<unsigned>((a.H + kSumCols - 1) / kSumCols), kSumCols * kSumRuns, 0, stream>>>(a.partial, G, a.H, a.dweight,
                                                                                                                   a.w_f32);
    return hipGetLastError();
}

}  // namespace bsfp8
