// gfx950 int8 row quantizer: x [T, H] bf16 -> codes with one scale a row (a token's activations, or an
// output channel's weights): s = max(amax, 1e-12) / 127, q = rint(x * (127 / max(amax, 1e-12))). A row
// stays in registers between its maximum and its codes (of up to sched::kRowMax values; longer ones are read
// twice); bound by the memory traffic, for few rows by the launch: 1000 x 1288 3.3 us.
#include "row_codes.hpp"
#include "schedule.hpp"

namespace bsfp8 {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// ANY: rows that begin anywhere, of any length; without it 16-byte pieces (codes 8-byte ones).
template <int TPR, int NC, bool ANY>
__global__ __launch_bounds__(kThreads) void rows_kernel(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, int64_t per_xcd, RowCodes out) {
    __shared__ uint32_t part[kWaves];
    const int tid = threadIdx.x % TPR;
    const int64_t row = xcd_block(blockIdx.x, per_xcd) * (kThreads / TPR) + threadIdx.x / TPR;
    if (row >= T) return;
    float v[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
        load8_of<false, false, ANY>(x, row * ldx + (c < H ? c : 0), v[i], H - c);
        if (!ANY && c >= H)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
    emit_row<TPR, NC, ANY>(out, row, T, H, tid, v, part);
}

__global__ __launch_bounds__(kThreads) void rows_long_kernel(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, RowCodes out) {
    __shared__ uint32_t part[kWaves];
    const int64_t row = blockIdx.x;
    const uint16_t* p = x + row * ldx;
    emit_row_any<kWaves>(out, row, T, H, [&](int64_t c) { return bf16_to_f32(p[c]); }, part);
}

template <bool ANY>
void launch_rows(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, const RowCodes& out, hipStream_t stream) {
    const bool wave = H <= sched::kRowWaveMax;
    const int64_t blocks = wave ? (T + kWaves - 1) / kWaves : T, per_xcd = (blocks + kXcds - 1) / kXcds;
    const unsigned grid = static_cast<unsigned>(per_xcd * kXcds);
#define BSFP8_ROWS(TPR, NC) rows_kernel<TPR, NC, ANY><<<grid, kThreads, 0, stream>>>(x, ldx, T, H, per_xcd, out)
    if (wave) {
        if (H <= 512) BSFP8_ROWS(64, 1);
        else BSFP8_ROWS(64, 2);
    } else {
        switch ((H + 2047) / 2048) {
            case 1: BSFP8_ROWS(256, 1); break;
            case 2: BSFP8_ROWS(256, 2); break;
            case 3: BSFP8_ROWS(256, 3); break;
            case 4: BSFP8_ROWS(256, 4); break;
            case 5: case 6: BSFP8_ROWS(256, 6); break;
            default: BSFP8_ROWS(256, 8); break;
        }
    }
#undef BSFP8_ROWS
}

}  // namespace

hipError_t launch_quantize_rows_i8(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, uint8_t* q, int64_t ldq, float* s,
                                   hipStream_t stream) {
    const RowCodes out{kCodesI8, q, ldq, s, nullptr, 0};
    if (H > sched::kRowMax) rows_long_kernel<<<static_cast<unsigned>(T), kThreads, 0, stream>>>(x, ldx, T, H, out);
    else if (H % 8 == 0 && rows16(x, 2 * ldx) && whole_codes(out)) launch_rows<false>(x, ldx, T, H, out, stream);
    else launch_rows<true>(x, ldx, T, H, out, stream);
    return hipGetLastError();
}

}  // namespace bsfp8
