// Host-side launchers of the gfx950 kernels (internal to the library; the C ABI validates first).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "schedule.hpp"

namespace bsfp8 {

// fnuz: float8_e4m3fnuz codes (FP8_MAX 240) instead of float8_e4m3fn (FP8_MAX 448).
// strip_loads: 0 = automatic (row strips of sched::lhs_strip_loads pieces per thread where the
// alignment allows, else tiles); 1, 2, 4, 8 or 16 = row strips of that many where the alignment
// allows; -1 = always the tile kernel.
hipError_t launch_quantize_lhs(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* q,
                               int64_t ldq, float* a_s, bool fnuz, int strip_loads, hipStream_t stream);
hipError_t launch_quantize_dual(const uint16_t* x, int64_t R, int64_t C, int64_t ldx, uint8_t* q,
                                int64_t ldq, float* a_s, uint8_t* qT, int64_t ldqT, float* s,
                                bool fnuz, hipStream_t stream);
// 128x1 groups that restart at every expert's first token, written in the 128-padded token layout
// (see quantize_rhs_grouped_kernel); padded: E + 1 padded boundaries (device memory, written).
hipError_t launch_quantize_rhs_grouped(const uint16_t* x, int64_t T, int64_t N, int64_t ldx, const int64_t* offsets,
                                      int64_t E, uint8_t* qT, int64_t ldqT, float* s, int64_t* padded, bool fnuz,
                                      hipStream_t stream);
hipError_t launch_quantize_rhs(const uint16_t* x, int64_t K, int64_t N, int64_t ldx, uint8_t* qT,
                               int64_t ldqT, float* s, bool fnuz, hipStream_t stream);
hipError_t launch_quantize_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldw, uint8_t* q,
                                  int64_t ldq, uint8_t* qT, int64_t ldqT, float* s, bool fnuz,
                                  hipStream_t stream);
// quantize_lhs(x) and quantize_weight_128x128(w) in one launch
hipError_t launch_quantize_step(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* qx,
                                int64_t ldqx, float* sx, const uint16_t* w, int64_t N, int64_t Kw,
                                int64_t ldw, uint8_t* qw, int64_t ldqw, uint8_t* qwT, int64_t ldqwT,
                                float* sw, bool fnuz, hipStream_t stream);
hipError_t launch_encode(const float* x, uint8_t* q, int64_t n, bool fnuz, hipStream_t stream);

// b-scale addressing of the GEMM: kind 0 = one scale per (K-block, 128-column block) at
// b_s[nb * stride_nb + kb * stride_kb]; kind 1 = one scale per (K-block, column) at b_s[kb * N + n].
struct BScale {
    const float* ptr;
    int64_t stride_nb;
    int64_t stride_kb;
    int per_column;
};

// Compute units of the current device (cached per device after the first query).
int device_cus();

// SplitPlan, gemm_split_plan and gemm_split_plan_forced: schedule.hpp.

// The allocation-free GEMM's scratch: a device array of gemm_scratch_bytes() bytes per device;
// gemm_scratch gives its address on the current device (looked up once per device).
int64_t gemm_scratch_bytes();
hipError_t gemm_scratch(float** out);

// fnuz: both operands hold float8_e4m3fnuz codes (general kernel, f16 matrix instructions).
// plan.S > 1 needs `workspace` (plan.bytes, 256-byte aligned, device memory) for the partial tiles.
hipError_t launch_gemm(const uint8_t* a, int64_t lda, const float* a_s, const uint8_t* b,
                       int64_t ldb, BScale bs, uint16_t* c, int64_t ldc, int64_t M, int64_t N,
                       int64_t K, bool fnuz, const SplitPlan& plan, float* workspace, int cus,
                       hipStream_t stream);

// Expert-grouped GEMMs (fast kernel; K % 128 == 0). offsets: E + 1 device int64 boundaries.
hipError_t launch_gemm_grouped_rows(const uint8_t* a, int64_t lda, const float* a_s,
                                    const uint8_t* b, int64_t ldb, int64_t b_stride, BScale bs,
                                    int64_t bs_stride, const int64_t* offsets, int64_t E,
                                    uint16_t* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                    hipStream_t stream);
hipError_t launch_gemm_grouped_k(const uint8_t* a, int64_t lda, const float* a_s, const uint8_t* b,
                                 int64_t ldb, const float* b_s, const int64_t* offsets, int64_t E,
                                 uint16_t* c, int64_t ldc, int64_t c_stride, int64_t M, int64_t N,
                                 int64_t K, int32_t* status, hipStream_t stream);

// Routing of a mixture-of-experts layer (moe.hip); the rule's fields as in moe_route.
struct RouteRule {
    bool softmax;
    int k, groups, top_groups;
    bool renormalize;
    float scale;
};
hipError_t launch_route(const void* logits, bool f32, int64_t T, int E, int64_t ld, const RouteRule& r, const float* bias,
                        float* weights, int32_t* ids, hipStream_t stream);
hipError_t launch_route_backward(const void* logits, bool f32, int64_t T, int E, int64_t ld, const RouteRule& r,
                                 const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd,
                                 hipStream_t stream);
// workspace: sched::plan_blocks(P) * (E + 1) int32 when plan_blocks(P) > 1, else unused
hipError_t launch_plan(const int32_t* ids, int64_t P, int E, int64_t* offsets, int32_t* slots, int32_t* rows,
                       int32_t* workspace, hipStream_t stream);
hipError_t launch_dispatch(const uint16_t* x, int64_t T, int64_t H, int64_t ldx, const int32_t* slots, int k, uint8_t* q,
                           int64_t ldq, float* a_s, uint16_t* copy, int64_t ldcopy, hipStream_t stream);
hipError_t launch_combine(const uint16_t* rows, int64_t R, int64_t ldr, const int32_t* slots, const float* weights,
                          int64_t T, int k, int64_t H, uint16_t* y, int64_t ldy, hipStream_t stream);
hipError_t launch_combine_backward(const uint16_t* dy, int64_t lddy, const uint16_t* rows, int64_t ldr,
                                   const int32_t* slots, const float* weights, int64_t T, int k, int64_t H,
                                   uint16_t* drows, int64_t lddr, float* dweights, hipStream_t stream);

// Expert products for few rows an expert (gemm_routed.hip). N: output columns (with swiglu B_e has
// 2 N rows). col_tiles and c_vec are set by the launcher.
struct RoutedArgs {
    const uint8_t* a;
    int64_t lda;
    const float* a_s;
    int64_t a_rows;
    const int32_t* rows;  // nullptr: row r of C reads row r of A
    int64_t k;
    const uint8_t* b;
    int64_t ldb, b_stride;
    const float* b_s;
    int64_t bs_stride, bs_nb, bs_kb;
    const int64_t* offsets;
    int64_t E;
    uint16_t* c;
    int64_t ldc, M, N, K;
    int64_t col_tiles;
    int c_vec;
};
hipError_t launch_gemm_routed(RoutedArgs a, bool swiglu, hipStream_t stream);

// Codes that an operator writes its rows in (BSFP8_CODES_*).
constexpr int kCodesNone = 0, kCodesE4m3Fn = 1, kCodesE4m3Fnuz = 2, kCodesI8 = 3;
struct RowCodes {
    int codes;
    uint8_t* q;  // [T, H], row stride ldq
    int64_t ldq;
    float* s;    // e4m3: column-major [T, ceil(H/128)], ld T; int8: [T]
    uint16_t* y; // nullptr, or the values in bf16, row stride ldy
    int64_t ldy;
};

// RMS norm (norm.hip). residual and h: both nullptr, or both set and of one type.
struct NormArgs {
    const uint16_t* x;
    int64_t ldx;
    const void* residual;
    int64_t ldr;
    bool res_f32;
    const void* weight;
    bool w_f32;
    float eps;
    void* h;
    int64_t ldh;
    float* rstd;  // nullptr: not written
    int64_t T, H;
    int64_t per_xcd;  // these two are set by the launcher
    double per_column;
};
hipError_t launch_rms_norm(NormArgs a, const RowCodes& out, hipStream_t stream);
hipError_t launch_rms_norm_rhs(const void* h, bool h_f32, int64_t ldh, const void* weight, bool w_f32, const float* rstd, int64_t T,
                               int64_t H, uint8_t* qT, int64_t ldqT, float* s, bool fnuz, hipStream_t stream);
struct NormBackwardArgs {
    const uint16_t* dy;
    int64_t lddy;
    const void* h;
    int64_t ldh;
    const void* weight;
    bool w_f32;
    const float* rstd;
    const void* dh;  // nullptr, or of h's type
    int64_t lddh;
    void* dx;  // of h's type
    int64_t lddx;
    void* dweight;  // of the weight's type
    float* partial; // sched::norm_backward_blocks(T) rows of H sums
    int64_t T, H;
};
hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, bool h_f32, hipStream_t stream);

// SwiGLU (swiglu.hip): gu [T, 2 F], gate then up.
hipError_t launch_swiglu(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, const RowCodes& out, hipStream_t stream);
struct TileCodes {
    uint8_t* q;
    int64_t ldq;
    float* a_s;
    uint8_t* qT;
    int64_t ldqT;
    float* s;
};
hipError_t launch_swiglu_dual(const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F, const TileCodes& out, bool fnuz,
                              hipStream_t stream);
hipError_t launch_swiglu_backward(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F,
                                  uint16_t* dgu, int64_t lddgu, hipStream_t stream);
hipError_t launch_swiglu_backward_dual(const uint16_t* dy, int64_t lddy, const uint16_t* gu, int64_t ldgu, int64_t T, int64_t F,
                                       const TileCodes& out, bool fnuz, hipStream_t stream);

// int8 rows (quantize_i8.hip) and products (gemm_i8.hip).
hipError_t launch_quantize_rows_i8(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, uint8_t* q, int64_t ldq, float* s,
                                   hipStream_t stream);
struct I8Args {
    const uint8_t* a;
    int64_t lda;
    const float* a_s;
    const uint8_t* b;
    int64_t ldb;
    const float* b_s;
    uint16_t* c;
    int64_t ldc, M, N, K;
};
hipError_t launch_gemm_i8(const I8Args& a, int cus, hipStream_t stream);

// Gradients of many tensors (grads.hip): the tensors of one launch, in units of sched::kGradUnit values.
constexpr int kGradTensors = 96;
struct GradTable {
    const void* in[kGradTensors];
    void* out[kGradTensors];  // clip only
    int64_t n[kGradTensors];
    int64_t first[kGradTensors + 1];  // units before tensor i; the last one: all
    uint8_t in_f32[kGradTensors], out_f32[kGradTensors];
    int count;
};
static_assert(sizeof(GradTable) <= 3800, "kernel arguments fit 4 KB");
// past: past the caches (sched::grads_past_caches)
hipError_t launch_grad_squares(const GradTable& t, bool past, double* partial, hipStream_t stream);
hipError_t launch_grad_norm(const double* partial, int64_t count, float* norm, hipStream_t stream);
// norm: nullptr where another launch of the call writes it
hipError_t launch_grad_clip(const GradTable& t, bool past, const double* partial, int64_t count, float max_norm, float eps, float* norm,
                            hipStream_t stream);

}  // namespace bsfp8
