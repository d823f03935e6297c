// C ABI of the blockwise FP8 library: argument validation (before any HIP call), a per-device
// gfx950 check, and launches on the caller's stream. Declarations and contracts: blockwise_fp8.h.
#include "blockwise_fp8.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "launch.hpp"

namespace {

constexpr int64_t kGroupEdge = 128;
constexpr int64_t kMaxGridY = 65535;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 0 = unknown, 1 = gfx950, 2 = other. Indexed by HIP device ordinal.
std::atomic<int> g_arch_state[64];

int check_device() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return BSFP8_EHIP;
    if (dev < 0 || dev >= 64) return BSFP8_EDEVICE;
    int st = g_arch_state[dev].load(std::memory_order_relaxed);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return BSFP8_EHIP;
        st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
        g_arch_state[dev].store(st, std::memory_order_relaxed);
    }
    return st == 1 ? BSFP8_OK : BSFP8_EDEVICE;
}

int finish(hipError_t e) { return e == hipSuccess ? BSFP8_OK : BSFP8_EHIP; }

// Compute units per device ordinal, queried once (0 = not yet known).
std::atomic<int> g_cus[64];

}  // namespace

int bsfp8::device_cus() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int cus = g_cus[dev].load(std::memory_order_relaxed);
    if (cus == 0) {
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
            cus = 256;
        g_cus[dev].store(cus, std::memory_order_relaxed);
    }
    return cus;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The GEMM kernels read every operand and scale tensor through buffer resources of at most 2^31
// bytes (a 256-row band of an operand, a whole scale tensor), so that an out-of-range lane offset
// (2^31 plus a per-K-block advance below 2^31) is always past the end.
constexpr int64_t kMaxRange = 0x80000000LL;
constexpr int64_t kMaxOperandLd = kMaxRange / 256;

int validate_gemm(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb,
                  const float* b_s, const void* c, int64_t ldc, int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0) return BSFP8_EINVAL;
    if (M == 0 || N == 0) return BSFP8_OK;
    if (c == nullptr || ldc < N) return BSFP8_EINVAL;
    if (cdiv(M, kGroupEdge) > kMaxGridY) return BSFP8_EINVAL;
    if (K == 0) return BSFP8_OK;
    if (a == nullptr || b == nullptr || a_s == nullptr || b_s == nullptr) return BSFP8_EINVAL;
    if (lda < K || ldb < K) return BSFP8_EINVAL;
    if (lda > kMaxOperandLd || ldb > kMaxOperandLd) return BSFP8_EINVAL;
    if (4 * M * cdiv(K, kGroupEdge) > kMaxRange) return BSFP8_EINVAL;
    if (!aligned16(a) || !aligned16(b) || (lda % 16) != 0 || (ldb % 16) != 0) return BSFP8_EALIGN;
    return BSFP8_OK;
}

// Split-K workspaces (shapes whose output tiles cannot fill the chip) come from a per-device
// stream-ordered memory pool whose memory is never returned to the system, so a call allocates
// from the driver only until the pool has grown to its largest workspace, and calls on different
// streams never share a buffer.
constexpr int64_t kMaxSplitWorkspace = 256LL << 20;
std::mutex g_pool_mutex;
hipMemPool_t g_pools[64];

hipError_t device_pool(hipMemPool_t* out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_pool_mutex);
    if (g_pools[dev] == nullptr) {
        hipMemPoolProps props;
        std::memset(&props, 0, sizeof(props));
        props.allocType = hipMemAllocationTypePinned;
        props.handleTypes = hipMemHandleTypeNone;
        props.location.type = hipMemLocationTypeDevice;
        props.location.id = dev;
        hipMemPool_t pool = nullptr;
        if ((e = hipMemPoolCreate(&pool, &props)) != hipSuccess) return e;
        uint64_t keep = UINT64_MAX;
        if ((e = hipMemPoolSetAttribute(pool, hipMemPoolAttrReleaseThreshold, &keep)) != hipSuccess) return e;
        g_pools[dev] = pool;
    }
    *out = g_pools[dev];
    return hipSuccess;
}

// BSFP8_GEMM_SPLIT, BSFP8_GEMM_TILE_M, BSFP8_GEMM_TILE_N, BSFP8_GEMM_THIN_STAGES and
// BSFP8_GEMM_THIN_WAVES (environment, read at each call): a slice count (1 = never split), a tile
// height (256 or 128: the fast kernel; 64: the thin kernel), the thin kernel's tile width (32, 64 or
// 128), its LDS stages (2, 3, 4, 6, 8 or 12, as far as the tile's stages fit the LDS) and its waves
// per workgroup (4, or 8 for tiles of 64 or 128 columns; other values fail with BSFP8_EHIP) that
// replace the automatic choices of gemm_split_plan, so tests and benchmarks can run every schedule
// on any shape. Unset or empty: automatic.
int env_int(const char* name) {
    const char* v = std::getenv(name);
    if (v == nullptr || *v == 0) return 0;
    const long s = std::strtol(v, nullptr, 10);
    return s < 1 ? 1 : (s > 65535 ? 65535 : static_cast<int>(s));
}

// The GEMM with its K split when the plan asks for it. The workspace is allocated and freed in
// stream order around the two kernels, or, with use_scratch, is the library's static scratch
// (nothing allocated; a plan larger than the scratch is BSFP8_ESCRATCH).
int run_gemm(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb,
             bsfp8::BScale bs, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K, bool fnuz,
             bool use_scratch, hipStream_t stream) {
    const int cus = bsfp8::device_cus();
    const int forced_s = env_int("BSFP8_GEMM_SPLIT"), forced_bm = env_int("BSFP8_GEMM_TILE_M");
    const int forced_bn = env_int("BSFP8_GEMM_TILE_N");
    bsfp8::SplitPlan plan =
        forced_s || forced_bm || forced_bn
            ? bsfp8::gemm_split_plan_forced(M, N, K, fnuz, cus, forced_s, forced_bm, forced_bn, kMaxSplitWorkspace)
            : bsfp8::gemm_split_plan(M, N, K, fnuz, cus, kMaxSplitWorkspace);
    if (plan.bm == bsfp8::geom::kThinBM) {
        plan.stages = env_int("BSFP8_GEMM_THIN_STAGES");
        plan.waves = env_int("BSFP8_GEMM_THIN_WAVES");
    }
    // A partial last round of 256 x 256 tiles: the leading columns as one GEMM, the tail columns
    // with K split (schedule.hpp, gemm_column_split). Automatic schedules with 128 x 128 B scales
    // only; BSFP8_GEMM_COLUMN_SPLIT=0 turns it off.
    const char* col_env = std::getenv("BSFP8_GEMM_COLUMN_SPLIT");
    const bool col_off = col_env != nullptr && col_env[0] == '0';
    if (!fnuz && !bs.per_column && !forced_s && !forced_bm && !forced_bn && !col_off) {
        const bsfp8::ColumnSplit cs = bsfp8::gemm_column_split(M, N, K, cus, kMaxSplitWorkspace);
        if (cs.n1 > 0 && (!use_scratch || cs.tail.bytes <= bsfp8::gemm_scratch_bytes())) {
            float* ws = nullptr;
            hipMemPool_t pool = nullptr;
            if (use_scratch) {
                if (bsfp8::gemm_scratch(&ws) != hipSuccess) return BSFP8_EHIP;
            } else {
                if (device_pool(&pool) != hipSuccess) return BSFP8_EHIP;
                if (hipMallocFromPoolAsync(reinterpret_cast<void**>(&ws), static_cast<size_t>(cs.tail.bytes), pool,
                                           stream) != hipSuccess)
                    return BSFP8_EHIP;
            }
            const uint8_t* a8 = static_cast<const uint8_t*>(a);
            const uint8_t* b8 = static_cast<const uint8_t*>(b);
            uint16_t* c16 = static_cast<uint16_t*>(c);
            hipError_t e = bsfp8::launch_gemm(a8, lda, a_s, b8, ldb, bs, c16, ldc, M, cs.n1, K, false, plan, nullptr,
                                              cus, stream);
            if (e == hipSuccess) {
                bsfp8::BScale bs_tail = bs;
                bs_tail.ptr = bs.ptr + (cs.n1 / bsfp8::geom::kBlockK) * bs.stride_nb;
                e = bsfp8::launch_gemm(a8, lda, a_s, b8 + cs.n1 * ldb, ldb, bs_tail, c16 + cs.n1, ldc, M, N - cs.n1, K,
                                       false, cs.tail, ws, cus, stream);
            }
            const hipError_t f = (!use_scratch && ws != nullptr) ? hipFreeAsync(ws, stream) : hipSuccess;
            return finish(e != hipSuccess ? e : f);
        }
    }
    if (use_scratch) {
        if (plan.bytes > bsfp8::gemm_scratch_bytes()) return BSFP8_ESCRATCH;
        float* ws = nullptr;
        if (plan.S > 1 && bsfp8::gemm_scratch(&ws) != hipSuccess) return BSFP8_EHIP;
        return finish(bsfp8::launch_gemm(static_cast<const uint8_t*>(a), lda, a_s, static_cast<const uint8_t*>(b),
                                         ldb, bs, static_cast<uint16_t*>(c), ldc, M, N, K, fnuz, plan, ws, cus,
                                         stream));
    }
    float* ws = nullptr;
    if (plan.S > 1) {
        hipMemPool_t pool = nullptr;
        if (device_pool(&pool) != hipSuccess) return BSFP8_EHIP;
        if (hipMallocFromPoolAsync(reinterpret_cast<void**>(&ws), static_cast<size_t>(plan.bytes), pool, stream) !=
            hipSuccess)
            return BSFP8_EHIP;
    }
    const hipError_t e = bsfp8::launch_gemm(static_cast<const uint8_t*>(a), lda, a_s, static_cast<const uint8_t*>(b),
                                            ldb, bs, static_cast<uint16_t*>(c), ldc, M, N, K, fnuz, plan, ws,
                                            cus, stream);
    const hipError_t f = ws != nullptr ? hipFreeAsync(ws, stream) : hipSuccess;
    return finish(e != hipSuccess ? e : f);
}

// BSFP8_QUANT_LHS_STRIP (environment, read at each call): 1, 2, 4, 8 or 16 runs quantize_lhs in
// row strips of that many 16-byte pieces per thread wherever the alignment allows, 0 always in
// tiles, so tests and benchmarks can compare the variants. Unset or empty: automatic.
int env_lhs_strip() {
    const char* v = std::getenv("BSFP8_QUANT_LHS_STRIP");
    if (v == nullptr || *v == 0) return 0;
    const long n = std::strtol(v, nullptr, 10);
    return n == 1 || n == 2 || n == 4 || n == 8 || n == 16 ? static_cast<int>(n) : -1;
}

int quantize_lhs_impl(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, int64_t ldq,
                      float* a_s, bool fnuz, void* stream) {
    if (M < 0 || K < 0) return BSFP8_EINVAL;
    if (M == 0 || K == 0) return BSFP8_OK;
    if (x == nullptr || q == nullptr || a_s == nullptr) return BSFP8_EINVAL;
    if (ldx < K || ldq < K) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_quantize_lhs(static_cast<const uint16_t*>(x), M, K, ldx,
                                             static_cast<uint8_t*>(q), ldq, a_s, fnuz, env_lhs_strip(),
                                             static_cast<hipStream_t>(stream)));
}

int quantize_rhs_impl(const void* x, int64_t K, int64_t N, int64_t ldx, void* qT, int64_t ldqT,
                      float* s, bool fnuz, void* stream) {
    if (K < 0 || N < 0) return BSFP8_EINVAL;
    if (K == 0 || N == 0) return BSFP8_OK;
    if (x == nullptr || qT == nullptr || s == nullptr) return BSFP8_EINVAL;
    if (ldx < N || ldqT < K) return BSFP8_EINVAL;
    if (cdiv(K, kGroupEdge) > kMaxGridY) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_quantize_rhs(static_cast<const uint16_t*>(x), K, N, ldx,
                                             static_cast<uint8_t*>(qT), ldqT, s, fnuz,
                                             static_cast<hipStream_t>(stream)));
}

int quantize_rhs_grouped_impl(const void* x, int64_t T, int64_t N, int64_t ldx, const int64_t* offsets, int64_t E,
                              void* qT, int64_t ldqT, float* s, int64_t* padded, bool fnuz, void* stream) {
    if (T < 0 || N < 0 || E < 0) return BSFP8_EINVAL;
    if (offsets == nullptr || padded == nullptr) return BSFP8_EINVAL;
    const int64_t groups = cdiv(T, kGroupEdge) + E;  // bound on the padded groups
    if (groups > kMaxGridY || cdiv(N, 64) > 0x7FFFFFFFLL) return BSFP8_EINVAL;
    if (T > 0 && N > 0) {
        if (x == nullptr || qT == nullptr || s == nullptr) return BSFP8_EINVAL;
        if (ldx < N || ldqT < groups * kGroupEdge) return BSFP8_EINVAL;
    }
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_quantize_rhs_grouped(static_cast<const uint16_t*>(x), T, N, ldx, offsets, E,
                                                     static_cast<uint8_t*>(qT), ldqT, s, padded, fnuz,
                                                     static_cast<hipStream_t>(stream)));
}

int quantize_weight_impl(const void* w, int64_t N, int64_t K, int64_t ldw, void* q, int64_t ldq,
                         void* qT, int64_t ldqT, float* s, bool fnuz, void* stream) {
    if (N < 0 || K < 0) return BSFP8_EINVAL;
    if (N == 0 || K == 0) return BSFP8_OK;
    if (w == nullptr || q == nullptr || s == nullptr) return BSFP8_EINVAL;
    if (ldw < K || ldq < K || (qT != nullptr && ldqT < N)) return BSFP8_EINVAL;
    if (cdiv(N, kGroupEdge) > kMaxGridY) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_quantize_weight(static_cast<const uint16_t*>(w), N, K, ldw,
                                                static_cast<uint8_t*>(q), ldq,
                                                static_cast<uint8_t*>(qT), ldqT, s, fnuz,
                                                static_cast<hipStream_t>(stream)));
}

int quantize_dual_impl(const void* x, int64_t R, int64_t C, int64_t ldx, void* q, int64_t ldq,
                       float* a_s, void* qT, int64_t ldqT, float* s, bool fnuz, void* stream) {
    if (R < 0 || C < 0) return BSFP8_EINVAL;
    if (R == 0 || C == 0) return BSFP8_OK;
    if (x == nullptr || q == nullptr || a_s == nullptr || qT == nullptr || s == nullptr) return BSFP8_EINVAL;
    if (ldx < C || ldq < C || ldqT < R) return BSFP8_EINVAL;
    if (cdiv(R, kGroupEdge) > kMaxGridY || cdiv(C, kGroupEdge) > 0x7FFFFFFFLL) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_quantize_dual(static_cast<const uint16_t*>(x), R, C, ldx,
                                              static_cast<uint8_t*>(q), ldq, a_s,
                                              static_cast<uint8_t*>(qT), ldqT, s, fnuz,
                                              static_cast<hipStream_t>(stream)));
}

int quantize_step_impl(const void* x, int64_t M, int64_t K, int64_t ldx, void* qx, int64_t ldqx,
                       float* sx, const void* w, int64_t N, int64_t Kw, int64_t ldw, void* qw,
                       int64_t ldqw, void* qwT, int64_t ldqwT, float* sw, bool fnuz, void* stream) {
    if (M < 0 || K < 0 || N < 0 || Kw < 0) return BSFP8_EINVAL;
    const bool x_empty = M == 0 || K == 0, w_empty = N == 0 || Kw == 0;
    if (!x_empty && (x == nullptr || qx == nullptr || sx == nullptr || ldx < K || ldqx < K)) return BSFP8_EINVAL;
    if (!w_empty && (w == nullptr || qw == nullptr || sw == nullptr || ldw < Kw || ldqw < Kw ||
                     (qwT != nullptr && ldqwT < N)))
        return BSFP8_EINVAL;
    if (x_empty && w_empty) return BSFP8_OK;
    if (x_empty) return quantize_weight_impl(w, N, Kw, ldw, qw, ldqw, qwT, ldqwT, sw, fnuz, stream);
    if (w_empty) return quantize_lhs_impl(x, M, K, ldx, qx, ldqx, sx, fnuz, stream);
    if (cdiv(M, kGroupEdge) * cdiv(K, kGroupEdge) + cdiv(N, kGroupEdge) * cdiv(Kw, kGroupEdge) > 0x7FFFFFFFLL)
        return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_quantize_step(
        static_cast<const uint16_t*>(x), M, K, ldx, static_cast<uint8_t*>(qx), ldqx, sx,
        static_cast<const uint16_t*>(w), N, Kw, ldw, static_cast<uint8_t*>(qw), ldqw,
        static_cast<uint8_t*>(qwT), ldqwT, sw, fnuz, static_cast<hipStream_t>(stream)));
}

// Floats a strided 128x128 scale tensor spans (the largest index read, plus one).
int64_t bscale_extent(int64_t N, int64_t K, int64_t bs_nb, int64_t bs_kb) {
    return (cdiv(N, kGroupEdge) - 1) * bs_nb + (cdiv(K, kGroupEdge) - 1) * bs_kb + 1;
}

int gemm_128x128_impl(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb,
                      const float* b_s, int64_t bs_stride_nb, int64_t bs_stride_kb, void* c,
                      int64_t ldc, int64_t M, int64_t N, int64_t K, bool fnuz, void* stream,
                      bool use_scratch = false) {
    if (int rc = validate_gemm(a, lda, a_s, b, ldb, b_s, c, ldc, M, N, K)) return rc;
    if (M == 0 || N == 0) return BSFP8_OK;
    if (bs_stride_nb < 0 || bs_stride_kb < 0) return BSFP8_EINVAL;
    if (K > 0 && 4 * bscale_extent(N, K, bs_stride_nb, bs_stride_kb) > kMaxRange) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    bsfp8::BScale bs{b_s, bs_stride_nb, bs_stride_kb, 0};
    return run_gemm(a, lda, a_s, b, ldb, bs, c, ldc, M, N, K, fnuz, use_scratch, static_cast<hipStream_t>(stream));
}

int gemm_128x1_impl(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb,
                    const float* b_s, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                    bool fnuz, void* stream, bool use_scratch = false) {
    if (int rc = validate_gemm(a, lda, a_s, b, ldb, b_s, c, ldc, M, N, K)) return rc;
    if (M == 0 || N == 0) return BSFP8_OK;
    if (4 * N * cdiv(K, kGroupEdge) > kMaxRange) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    bsfp8::BScale bs{b_s, 0, 0, 1};
    return run_gemm(a, lda, a_s, b, ldb, bs, c, ldc, M, N, K, fnuz, use_scratch, static_cast<hipStream_t>(stream));
}

// Limits of the mixture-of-experts entry points: one lane holds a choice, and the experts of a row
// (of a bin) fit a wave's registers (a workgroup's LDS).
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxChoices = 64;
constexpr int64_t kMaxPairs = 0x7FFFFFFF;
constexpr int64_t kMaxWaves = (int64_t{1} << 26) - 64;  // a launch's lanes are counted in 32 bits; whole workgroups

// The pairs of T tokens with k choices each are numbered in 32 bits.
bool pairs_ok(int64_t T, int64_t k) { return T >= 0 && k >= 1 && k <= kMaxChoices && T <= kMaxPairs / k; }

int validate_route(int dtype, int64_t T, int64_t E, int64_t ld, int score, int64_t k, float scale) {
    if (!pairs_ok(T, k) || E < 1 || E > kMaxExperts || k > E) return BSFP8_EINVAL;
    if ((dtype != BSFP8_BF16 && dtype != BSFP8_F32) || (score != BSFP8_SOFTMAX && score != BSFP8_SIGMOID))
        return BSFP8_EINVAL;
    if (ld < E || !std::isfinite(scale) || T > kMaxWaves) return BSFP8_EINVAL;
    return BSFP8_OK;
}

// Limits of the operators that take rows of tokens: a workgroup of four waves a row.
constexpr int64_t kMaxRows = (int64_t{1} << 24) - 16;
constexpr int64_t kMaxI8K = 131071;  // 2^14 K < 2^31
// A launch's lanes are counted in 32 bits: 512 for each 128 columns, 1024 for each 16.
constexpr int64_t kMaxTileColumns = (int64_t{1} << 30) - 128, kMaxBackwardColumns = (int64_t{1} << 26) - 16;

bool dtype_ok(int d) { return d == BSFP8_BF16 || d == BSFP8_F32; }
bool fp8_codes(int codes) { return codes == BSFP8_CODES_E4M3FN || codes == BSFP8_CODES_E4M3FNUZ; }

// Outputs of an operator that writes rows as codes.
int validate_codes(int64_t T, int64_t H, int codes, const void* q, int64_t ldq, const float* s, const void* y, int64_t ldy) {
    if (T < 0 || H < 0 || T > kMaxRows || H > 0x7FFFFFFF) return BSFP8_EINVAL;
    if (codes != BSFP8_CODES_NONE && codes != BSFP8_CODES_INT8 && !fp8_codes(codes)) return BSFP8_EINVAL;
    if (T == 0 || H == 0) return BSFP8_OK;
    if ((codes == BSFP8_CODES_NONE) != (q == nullptr) || (q == nullptr) != (s == nullptr)) return BSFP8_EINVAL;
    if (q == nullptr && y == nullptr) return BSFP8_EINVAL;
    if ((q != nullptr && ldq < H) || (y != nullptr && ldy < H)) return BSFP8_EINVAL;
    return BSFP8_OK;
}

// Outputs in both groupings of a [T, C] tensor.
int validate_tiles(int64_t T, int64_t C, int codes, const void* q, int64_t ldq, const float* a_s, const void* qT, int64_t ldqT,
                   const float* s) {
    if (T < 0 || C < 0 || C > kMaxTileColumns || cdiv(T, kGroupEdge) > kMaxGridY || !fp8_codes(codes)) return BSFP8_EINVAL;
    if (T == 0 || C == 0) return BSFP8_OK;
    if (q == nullptr || a_s == nullptr || qT == nullptr || s == nullptr || ldq < C || ldqT < T) return BSFP8_EINVAL;
    return BSFP8_OK;
}

// The tensors of grad_norm and clip_grads; the number of their launches' workgroups, or -1.
int64_t grad_partials(const int64_t* sizes, int64_t count) {
    if (count < 0 || count > 0xFFFFFF || (count > 0 && sizes == nullptr)) return -1;
    int64_t partials = 0, units = 0, in_launch = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > (int64_t{1} << 48)) return -1;
        if (sizes[i] == 0) continue;
        units += cdiv(sizes[i], bsfp8::sched::kGradUnit);
        if (++in_launch == bsfp8::kGradTensors) {
            partials += bsfp8::sched::grad_blocks(units);
            units = in_launch = 0;
        }
    }
    return partials + (in_launch > 0 ? bsfp8::sched::grad_blocks(units) : 0);
}

double grad_bytes(const int64_t* sizes, const int* dtypes, int64_t count) {
    double bytes = 0;
    for (int64_t i = 0; i < count; ++i) bytes += static_cast<double>(sizes[i]) * (dtypes[i] == BSFP8_F32 ? 4 : 2);
    return bytes;
}

// No output shares memory with another tensor of the call, but with its own gradient as a whole.
bool outputs_apart(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes, const int* out_dtypes,
                   int64_t count) {
    struct Range {
        uintptr_t from, to;
        int64_t i;
    };
    const auto bytes = [&](int64_t i, int d) { return static_cast<uintptr_t>(sizes[i]) * (d == BSFP8_F32 ? 4 : 2); };
    std::vector<Range> out;
    out.reserve(static_cast<size_t>(count));
    for (int64_t i = 0; i < count; ++i)
        if (sizes[i] > 0) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(outs[i]);
            out.push_back({p, p + bytes(i, out_dtypes[i]), i});
        }
    const auto before = [](const Range& a, const Range& b) { return a.from < b.from; };
    if (!std::is_sorted(out.begin(), out.end(), before)) std::sort(out.begin(), out.end(), before);
    for (size_t k = 1; k < out.size(); ++k)
        if (out[k].from < out[k - 1].to) return false;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t from = reinterpret_cast<uintptr_t>(grads[i]), to = from + bytes(i, dtypes[i]);
        if (grads[i] == outs[i] && dtypes[i] == out_dtypes[i]) continue;  // the outputs are apart, so this one meets no other
        // the outputs end in order, too: the first that ends behind `from`
        const auto at = std::upper_bound(out.begin(), out.end(), from, [](uintptr_t v, const Range& r) { return v < r.to; });
        if (at != out.end() && at->from < to) return false;
    }
    return true;
}

// Calls f(table, workgroups before) for each launch of the tensors that hold values.
template <typename F>
hipError_t for_grad_tables(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes,
                           const int* out_dtypes, int64_t count, F f) {
    bsfp8::GradTable t;
    t.count = 0;
    t.first[0] = 0;
    int64_t before = 0;
    const auto flush = [&]() {
        if (t.count == 0) return hipSuccess;
        const hipError_t e = f(t, before);
        before += bsfp8::sched::grad_blocks(t.first[t.count]);
        t.count = 0;
        return e;
    };
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const int k = t.count++;
        t.in[k] = grads[i];
        t.out[k] = outs != nullptr ? outs[i] : nullptr;
        t.n[k] = sizes[i];
        t.first[k + 1] = t.first[k] + cdiv(sizes[i], bsfp8::sched::kGradUnit);
        t.in_f32[k] = dtypes[i] == BSFP8_F32;
        t.out_f32[k] = outs != nullptr && out_dtypes[i] == BSFP8_F32;
        if (t.count == bsfp8::kGradTensors)
            if (const hipError_t e = flush()) return e;
    }
    return flush();
}

int validate_grads(const void* const* grads, const int64_t* sizes, const int* dtypes, int64_t count, const float* norm,
                   const void* workspace, int64_t workspace_bytes) {
    const int64_t partials = grad_partials(sizes, count);
    if (partials < 0 || norm == nullptr || (count > 0 && (grads == nullptr || dtypes == nullptr))) return BSFP8_EINVAL;
    if (partials > 0 && (workspace == nullptr || workspace_bytes < 8 * partials)) return BSFP8_EINVAL;
    if ((reinterpret_cast<uintptr_t>(workspace) & 7) != 0) return BSFP8_EINVAL;
    for (int64_t i = 0; i < count; ++i) {
        if (!dtype_ok(dtypes[i]) || (sizes[i] > 0 && grads[i] == nullptr)) return BSFP8_EINVAL;
        if (sizes[i] > 0 && reinterpret_cast<uintptr_t>(grads[i]) % (dtypes[i] == BSFP8_F32 ? 4 : 2) != 0) return BSFP8_EINVAL;
    }
    return BSFP8_OK;
}

int encode_impl(const float* x, void* q, int64_t n, bool fnuz, void* stream) {
    if (n < 0) return BSFP8_EINVAL;
    if (n == 0) return BSFP8_OK;
    if (x == nullptr || q == nullptr) return BSFP8_EINVAL;
    if (!aligned16(x) || (reinterpret_cast<uintptr_t>(q) & 3) != 0) return BSFP8_EALIGN;
    if ((n + 1023) / 1024 > 0x7FFFFFFFLL) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_encode(x, static_cast<uint8_t*>(q), n, fnuz,
                                       static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

const char* bsfp8_status_string(int status) {
    switch (status) {
        case BSFP8_OK: return "ok";
        case BSFP8_EINVAL: return "invalid argument";
        case BSFP8_EALIGN: return "operand rows not 16-byte aligned";
        case BSFP8_EDEVICE: return "current device is not gfx950";
        case BSFP8_EHIP: return "HIP call or kernel launch failed";
        case BSFP8_ESCRATCH: return "the K-split workspace exceeds the allocation-free scratch";
        default: return "unknown status";
    }
}

int quantize_lhs(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, int64_t ldq,
                 float* a_s, void* stream) {
    return quantize_lhs_impl(x, M, K, ldx, q, ldq, a_s, false, stream);
}

int quantize_lhs_fnuz(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, int64_t ldq,
                      float* a_s, void* stream) {
    return quantize_lhs_impl(x, M, K, ldx, q, ldq, a_s, true, stream);
}

int quantize_rhs(const void* x, int64_t K, int64_t N, int64_t ldx, void* qT, int64_t ldqT,
                 float* s, void* stream) {
    return quantize_rhs_impl(x, K, N, ldx, qT, ldqT, s, false, stream);
}

int quantize_rhs_fnuz(const void* x, int64_t K, int64_t N, int64_t ldx, void* qT, int64_t ldqT,
                      float* s, void* stream) {
    return quantize_rhs_impl(x, K, N, ldx, qT, ldqT, s, true, stream);
}

int quantize_weight_128x128(const void* w, int64_t N, int64_t K, int64_t ldw, void* q,
                            int64_t ldq, void* qT, int64_t ldqT, float* s, void* stream) {
    return quantize_weight_impl(w, N, K, ldw, q, ldq, qT, ldqT, s, false, stream);
}

int quantize_weight_128x128_fnuz(const void* w, int64_t N, int64_t K, int64_t ldw, void* q,
                                 int64_t ldq, void* qT, int64_t ldqT, float* s, void* stream) {
    return quantize_weight_impl(w, N, K, ldw, q, ldq, qT, ldqT, s, true, stream);
}

int gemm_1x128_128x128(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb,
                       const float* b_s, int64_t bs_stride_nb, int64_t bs_stride_kb, void* c,
                       int64_t ldc, int64_t M, int64_t N, int64_t K, void* stream) {
    return gemm_128x128_impl(a, lda, a_s, b, ldb, b_s, bs_stride_nb, bs_stride_kb, c, ldc, M, N, K,
                             false, stream);
}

int gemm_1x128_128x128_noalloc(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb,
                               const float* b_s, int64_t bs_stride_nb, int64_t bs_stride_kb, void* c,
                               int64_t ldc, int64_t M, int64_t N, int64_t K, void* stream) {
    return gemm_128x128_impl(a, lda, a_s, b, ldb, b_s, bs_stride_nb, bs_stride_kb, c, ldc, M, N, K,
                             false, stream, true);
}

int gemm_1x128_128x128_fnuz(const void* a, int64_t lda, const float* a_s, const void* b,
                            int64_t ldb, const float* b_s, int64_t bs_stride_nb,
                            int64_t bs_stride_kb, void* c, int64_t ldc, int64_t M, int64_t N,
                            int64_t K, void* stream) {
    return gemm_128x128_impl(a, lda, a_s, b, ldb, b_s, bs_stride_nb, bs_stride_kb, c, ldc, M, N, K,
                             true, stream);
}

int gemm_1x128_128x1(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb,
                     const float* b_s, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                     void* stream) {
    return gemm_128x1_impl(a, lda, a_s, b, ldb, b_s, c, ldc, M, N, K, false, stream);
}

int gemm_1x128_128x1_fnuz(const void* a, int64_t lda, const float* a_s, const void* b,
                          int64_t ldb, const float* b_s, void* c, int64_t ldc, int64_t M,
                          int64_t N, int64_t K, void* stream) {
    return gemm_128x1_impl(a, lda, a_s, b, ldb, b_s, c, ldc, M, N, K, true, stream);
}

int quantize_lhs_and_rhs(const void* x, int64_t R, int64_t C, int64_t ldx, void* q, int64_t ldq,
                         float* a_s, void* qT, int64_t ldqT, float* s, void* stream) {
    return quantize_dual_impl(x, R, C, ldx, q, ldq, a_s, qT, ldqT, s, false, stream);
}

int quantize_lhs_and_rhs_fnuz(const void* x, int64_t R, int64_t C, int64_t ldx, void* q,
                              int64_t ldq, float* a_s, void* qT, int64_t ldqT, float* s,
                              void* stream) {
    return quantize_dual_impl(x, R, C, ldx, q, ldq, a_s, qT, ldqT, s, true, stream);
}

int quantize_rhs_grouped(const void* x, int64_t T, int64_t N, int64_t ldx, const int64_t* offsets, int64_t E,
                         void* qT, int64_t ldqT, float* s, int64_t* padded_offsets, void* stream) {
    return quantize_rhs_grouped_impl(x, T, N, ldx, offsets, E, qT, ldqT, s, padded_offsets, false, stream);
}

int quantize_rhs_grouped_fnuz(const void* x, int64_t T, int64_t N, int64_t ldx, const int64_t* offsets,
                              int64_t E, void* qT, int64_t ldqT, float* s, int64_t* padded_offsets,
                              void* stream) {
    return quantize_rhs_grouped_impl(x, T, N, ldx, offsets, E, qT, ldqT, s, padded_offsets, true, stream);
}

int gemm_1x128_128x128_grouped(const void* a, int64_t lda, const float* a_s, const void* b,
                               int64_t ldb, int64_t b_stride, const float* b_s, int64_t bs_stride,
                               int64_t bs_stride_nb, int64_t bs_stride_kb, const int64_t* offsets,
                               int64_t E, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                               void* stream) {
    if (E < 0 || K < 0) return BSFP8_EINVAL;
    if (E == 0 || M == 0 || N == 0) return M < 0 || N < 0 ? BSFP8_EINVAL : BSFP8_OK;
    if (K == 0 || K % kGroupEdge != 0) return BSFP8_EINVAL;
    if (int rc = validate_gemm(a, lda, a_s, b, ldb, b_s, c, ldc, M, N, K)) return rc;
    if (offsets == nullptr || b_stride < 0 || bs_stride < 0 || bs_stride_nb < 0 || bs_stride_kb < 0)
        return BSFP8_EINVAL;
    if (4 * bscale_extent(N, K, bs_stride_nb, bs_stride_kb) > kMaxRange) return BSFP8_EINVAL;
    if (b_stride % 16 != 0) return BSFP8_EALIGN;
    if (int rc = check_device()) return rc;
    bsfp8::BScale bs{b_s, bs_stride_nb, bs_stride_kb, 0};
    return finish(bsfp8::launch_gemm_grouped_rows(
        static_cast<const uint8_t*>(a), lda, a_s, static_cast<const uint8_t*>(b), ldb, b_stride, bs,
        bs_stride, offsets, E, static_cast<uint16_t*>(c), ldc, M, N, K,
        static_cast<hipStream_t>(stream)));
}

int gemm_1x128_128x1_grouped(const void* a, int64_t lda, const float* a_s, const void* b,
                             int64_t ldb, const float* b_s, const int64_t* offsets, int64_t E,
                             void* c, int64_t ldc, int64_t c_stride, int64_t M, int64_t N,
                             int64_t K, int32_t* status, void* stream) {
    if (E < 0 || K < 0) return BSFP8_EINVAL;
    if (E == 0 || M == 0 || N == 0) return M < 0 || N < 0 ? BSFP8_EINVAL : BSFP8_OK;
    if (K == 0 || K % kGroupEdge != 0 || E > 65535) return BSFP8_EINVAL;
    if (int rc = validate_gemm(a, lda, a_s, b, ldb, b_s, c, ldc, M, N, K)) return rc;
    if (4 * N * cdiv(K, kGroupEdge) > kMaxRange) return BSFP8_EINVAL;
    if (offsets == nullptr) return BSFP8_EINVAL;
    if (E > 1 && c_stride < (M - 1) * ldc + N) return BSFP8_EINVAL;  // expert outputs must not overlap
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_gemm_grouped_k(
        static_cast<const uint8_t*>(a), lda, a_s, static_cast<const uint8_t*>(b), ldb, b_s, offsets,
        E, static_cast<uint16_t*>(c), ldc, c_stride, M, N, K, status, static_cast<hipStream_t>(stream)));
}

int quantize_lhs_and_weight(const void* x, int64_t M, int64_t K, int64_t ldx, void* qx, int64_t ldqx,
                            float* sx, const void* w, int64_t N, int64_t Kw, int64_t ldw, void* qw,
                            int64_t ldqw, void* qwT, int64_t ldqwT, float* sw, void* stream) {
    return quantize_step_impl(x, M, K, ldx, qx, ldqx, sx, w, N, Kw, ldw, qw, ldqw, qwT, ldqwT, sw, false,
                              stream);
}

int quantize_lhs_and_weight_fnuz(const void* x, int64_t M, int64_t K, int64_t ldx, void* qx,
                                 int64_t ldqx, float* sx, const void* w, int64_t N, int64_t Kw,
                                 int64_t ldw, void* qw, int64_t ldqw, void* qwT, int64_t ldqwT,
                                 float* sw, void* stream) {
    return quantize_step_impl(x, M, K, ldx, qx, ldqx, sx, w, N, Kw, ldw, qw, ldqw, qwT, ldqwT, sw, true,
                              stream);
}

int encode_e4m3_f32(const float* x, void* q, int64_t n, void* stream) {
    return encode_impl(x, q, n, false, stream);
}

int encode_e4m3fnuz_f32(const float* x, void* q, int64_t n, void* stream) {
    return encode_impl(x, q, n, true, stream);
}

int moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias, int score,
              int64_t k, int64_t groups, int64_t top_groups, int renormalize, float scale, float* weights,
              int32_t* ids, void* stream) {
    if (int rc = validate_route(dtype, T, E, ld, score, k, scale)) return rc;
    if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups || k > top_groups * (E / groups))
        return BSFP8_EINVAL;
    if (T == 0) return BSFP8_OK;
    if (logits == nullptr || weights == nullptr || ids == nullptr) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    const bsfp8::RouteRule rule{score == BSFP8_SOFTMAX, static_cast<int>(k), static_cast<int>(groups),
                                static_cast<int>(top_groups), renormalize != 0, scale};
    return finish(bsfp8::launch_route(logits, dtype == BSFP8_F32, T, static_cast<int>(E), ld, rule, bias, weights, ids,
                                      static_cast<hipStream_t>(stream)));
}

int moe_route_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, int score, int64_t k,
                       int renormalize, float scale, const int32_t* ids, const float* dweights, void* dlogits,
                       int64_t lddl, void* stream) {
    if (int rc = validate_route(dtype, T, E, ld, score, k, scale)) return rc;
    if (lddl < E) return BSFP8_EINVAL;
    if (T == 0) return BSFP8_OK;
    if (logits == nullptr || ids == nullptr || dweights == nullptr || dlogits == nullptr) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    const bsfp8::RouteRule rule{score == BSFP8_SOFTMAX, static_cast<int>(k), 1, 1, renormalize != 0, scale};
    return finish(bsfp8::launch_route_backward(logits, dtype == BSFP8_F32, T, static_cast<int>(E), ld, rule, ids,
                                               dweights, dlogits, lddl, static_cast<hipStream_t>(stream)));
}

int64_t moe_plan_workspace(int64_t T, int64_t k, int64_t E) {
    if (!pairs_ok(T, k) || E < 1 || E > kMaxExperts) return -1;
    const int64_t blocks = bsfp8::sched::plan_blocks(T * k);
    return blocks > 1 ? blocks * (E + 1) * static_cast<int64_t>(sizeof(int32_t)) : 0;
}

int moe_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int64_t* offsets, int32_t* slots, int32_t* rows,
             void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = moe_plan_workspace(T, k, E);
    if (need < 0 || offsets == nullptr) return BSFP8_EINVAL;
    if (T > 0 && (ids == nullptr || slots == nullptr || rows == nullptr)) return BSFP8_EINVAL;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BSFP8_EINVAL;
    if ((reinterpret_cast<uintptr_t>(workspace) & 3) != 0) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_plan(ids, T * k, static_cast<int>(E), offsets, slots, rows,
                                     static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)));
}

int moe_dispatch(const void* x, int64_t T, int64_t H, int64_t ldx, const int32_t* slots, int64_t k, void* q, int64_t ldq,
                 float* a_s, void* copy, int64_t ldcopy, void* stream) {
    if (!pairs_ok(T, k) || H < 0) return BSFP8_EINVAL;
    if (T == 0 || H == 0) return BSFP8_OK;
    if (x == nullptr || slots == nullptr || q == nullptr || a_s == nullptr) return BSFP8_EINVAL;
    if (ldx < H || ldq < H || (copy != nullptr && ldcopy < H)) return BSFP8_EINVAL;
    if (cdiv(H, 1024) > kMaxWaves / T) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_dispatch(static_cast<const uint16_t*>(x), T, H, ldx, slots, static_cast<int>(k),
                                         static_cast<uint8_t*>(q), ldq, a_s, static_cast<uint16_t*>(copy), ldcopy,
                                         static_cast<hipStream_t>(stream)));
}

int moe_combine(const void* rows, int64_t R, int64_t ldr, const int32_t* slots, const float* weights, int64_t T,
                int64_t k, int64_t H, void* y, int64_t ldy, void* stream) {
    if (!pairs_ok(T, k) || H < 0 || R < 0) return BSFP8_EINVAL;
    if (T == 0 || H == 0) return BSFP8_OK;
    if ((rows == nullptr && R > 0) || slots == nullptr || y == nullptr) return BSFP8_EINVAL;
    if (ldr < H || ldy < H || cdiv(H, 512) > kMaxWaves / T) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_combine(static_cast<const uint16_t*>(rows), R, ldr, slots, weights, T,
                                        static_cast<int>(k), H, static_cast<uint16_t*>(y), ldy,
                                        static_cast<hipStream_t>(stream)));
}

int moe_combine_backward(const void* dy, int64_t lddy, const void* rows, int64_t ldr, const int32_t* slots,
                         const float* weights, int64_t T, int64_t k, int64_t H, void* drows, int64_t lddr,
                         float* dweights, void* stream) {
    if (!pairs_ok(T, k) || H < 0) return BSFP8_EINVAL;
    if (T == 0) return BSFP8_OK;
    if (slots == nullptr || weights == nullptr || dweights == nullptr) return BSFP8_EINVAL;
    if (H > 0 && (dy == nullptr || rows == nullptr || drows == nullptr)) return BSFP8_EINVAL;
    if (lddy < H || ldr < H || lddr < H || T > kMaxWaves / 4) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_combine_backward(
        static_cast<const uint16_t*>(dy), lddy, static_cast<const uint16_t*>(rows), ldr, slots, weights, T,
        static_cast<int>(k), H, static_cast<uint16_t*>(drows), lddr, dweights, static_cast<hipStream_t>(stream)));
}

int gemm_1x128_128x128_routed(const void* a, int64_t lda, const float* a_s, int64_t a_rows, const int32_t* rows,
                              int64_t k, const void* b, int64_t ldb, int64_t b_stride, const float* b_s,
                              int64_t bs_stride, int64_t bs_stride_nb, int64_t bs_stride_kb, const int64_t* offsets,
                              int64_t E, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K, int swiglu,
                              void* stream) {
    if (E < 0 || M < 0 || N < 0 || K < 0 || a_rows < 0) return BSFP8_EINVAL;
    if (E == 0 || M == 0 || N == 0) return BSFP8_OK;
    if (K == 0 || K % kGroupEdge != 0 || (swiglu != 0 && N % kGroupEdge != 0)) return BSFP8_EINVAL;
    if (a == nullptr || a_s == nullptr || b == nullptr || b_s == nullptr || offsets == nullptr || c == nullptr)
        return BSFP8_EINVAL;
    if (E > kMaxExperts || M > kMaxPairs || a_rows < 1 || k < 1 || k > kMaxChoices) return BSFP8_EINVAL;
    if (rows == nullptr && a_rows < M) return BSFP8_EINVAL;
    if (!bsfp8::sched::routed_fits(M, N, K, E, swiglu != 0)) return BSFP8_EINVAL;
    if (lda < K || ldb < K || ldc < N || b_stride < 0 || bs_stride < 0 || bs_stride_nb < 0 || bs_stride_kb < 0)
        return BSFP8_EINVAL;
    if (!aligned16(a) || !aligned16(b) || lda % 16 != 0 || ldb % 16 != 0 || b_stride % 16 != 0) return BSFP8_EALIGN;
    if (int rc = check_device()) return rc;
    const bsfp8::RoutedArgs args{static_cast<const uint8_t*>(a), lda, a_s, a_rows, rows, k,
                                 static_cast<const uint8_t*>(b), ldb, b_stride, b_s, bs_stride, bs_stride_nb,
                                 bs_stride_kb, offsets, E, static_cast<uint16_t*>(c), ldc, M, N, K, 0, 0};
    return finish(bsfp8::launch_gemm_routed(args, swiglu != 0, static_cast<hipStream_t>(stream)));
}

int rms_norm_quantize(const void* x, int64_t T, int64_t H, int64_t ldx, const void* residual, int res_dtype, int64_t ldr,
                      const void* weight, int w_dtype, float eps, void* h, int64_t ldh, float* rstd, int codes, void* q,
                      int64_t ldq, float* s, void* y, int64_t ldy, void* stream) {
    if (int rc = validate_codes(T, H, codes, q, ldq, s, y, ldy)) return rc;
    if (!dtype_ok(res_dtype) || !dtype_ok(w_dtype) || !(eps > 0.0f) || !std::isfinite(eps)) return BSFP8_EINVAL;
    if (T == 0 || H == 0) return BSFP8_OK;
    if (x == nullptr || weight == nullptr || ldx < H || (residual == nullptr) != (h == nullptr)) return BSFP8_EINVAL;
    if (residual != nullptr && (ldr < H || ldh < H)) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    const bsfp8::NormArgs a{static_cast<const uint16_t*>(x), ldx, residual, ldr, res_dtype == BSFP8_F32, weight,
                            w_dtype == BSFP8_F32, eps, h, ldh, rstd, T, H, 0, 0.0};
    const bsfp8::RowCodes out{codes, static_cast<uint8_t*>(q), ldq, s, static_cast<uint16_t*>(y), ldy};
    return finish(bsfp8::launch_rms_norm(a, out, static_cast<hipStream_t>(stream)));
}

int rms_norm_quantize_rhs(const void* h, int h_dtype, int64_t T, int64_t H, int64_t ldh, const void* weight, int w_dtype,
                          const float* rstd, int codes, void* qT, int64_t ldqT, float* s, void* stream) {
    if (T < 0 || H < 0 || H > kMaxTileColumns || cdiv(T, kGroupEdge) > kMaxGridY || !fp8_codes(codes)) return BSFP8_EINVAL;
    if (!dtype_ok(h_dtype) || !dtype_ok(w_dtype)) return BSFP8_EINVAL;
    if (T == 0 || H == 0) return BSFP8_OK;
    if (h == nullptr || weight == nullptr || rstd == nullptr || qT == nullptr || s == nullptr || ldh < H || ldqT < T)
        return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_rms_norm_rhs(h, h_dtype == BSFP8_F32, ldh, weight, w_dtype == BSFP8_F32, rstd, T, H,
                                             static_cast<uint8_t*>(qT), ldqT, s, codes == BSFP8_CODES_E4M3FNUZ,
                                             static_cast<hipStream_t>(stream)));
}

int64_t rms_norm_backward_workspace(int64_t T, int64_t H) {
    if (T < 0 || H < 0 || T > kMaxRows || H > kMaxBackwardColumns) return -1;
    return bsfp8::sched::norm_backward_blocks(T) * H * static_cast<int64_t>(sizeof(float));
}

int rms_norm_backward(const void* dy, int64_t lddy, const void* h, int h_dtype, int64_t ldh, const void* weight, int w_dtype,
                      const float* rstd, const void* dh, int64_t lddh, int64_t T, int64_t H, void* dx, int64_t lddx,
                      void* dweight, void* workspace, int64_t workspace_bytes, void* stream) {
    const int64_t need = rms_norm_backward_workspace(T, H);
    if (need < 0 || !dtype_ok(h_dtype) || !dtype_ok(w_dtype)) return BSFP8_EINVAL;
    if (H == 0) return BSFP8_OK;
    if (weight == nullptr || dweight == nullptr) return BSFP8_EINVAL;
    if (T > 0) {
        if (dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr) return BSFP8_EINVAL;
        if (lddy < H || ldh < H || lddx < H || (dh != nullptr && lddh < H)) return BSFP8_EINVAL;
        if (workspace == nullptr || workspace_bytes < need) return BSFP8_EINVAL;
    }
    if ((reinterpret_cast<uintptr_t>(workspace) & 15) != 0) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    const bsfp8::NormBackwardArgs a{static_cast<const uint16_t*>(dy), lddy, h, ldh, weight, w_dtype == BSFP8_F32, rstd, dh,
                                    lddh, dx, lddx, dweight, static_cast<float*>(workspace), T, H};
    return finish(bsfp8::launch_rms_norm_backward(a, h_dtype == BSFP8_F32, static_cast<hipStream_t>(stream)));
}

int swiglu_quantize(const void* gu, int64_t T, int64_t F, int64_t ldgu, int codes, void* q, int64_t ldq, float* s, void* y,
                    int64_t ldy, void* stream) {
    if (int rc = validate_codes(T, F, codes, q, ldq, s, y, ldy)) return rc;
    if (T == 0 || F == 0) return BSFP8_OK;
    if (gu == nullptr || ldgu < 2 * F) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    const bsfp8::RowCodes out{codes, static_cast<uint8_t*>(q), ldq, s, static_cast<uint16_t*>(y), ldy};
    return finish(bsfp8::launch_swiglu(static_cast<const uint16_t*>(gu), ldgu, T, F, out, static_cast<hipStream_t>(stream)));
}

int swiglu_quantize_lhs_and_rhs(const void* gu, int64_t T, int64_t F, int64_t ldgu, int codes, void* q, int64_t ldq, float* a_s,
                                void* qT, int64_t ldqT, float* s, void* stream) {
    if (int rc = validate_tiles(T, F, codes, q, ldq, a_s, qT, ldqT, s)) return rc;
    if (T == 0 || F == 0) return BSFP8_OK;
    if (gu == nullptr || ldgu < 2 * F) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    const bsfp8::TileCodes out{static_cast<uint8_t*>(q), ldq, a_s, static_cast<uint8_t*>(qT), ldqT, s};
    return finish(bsfp8::launch_swiglu_dual(static_cast<const uint16_t*>(gu), ldgu, T, F, out, codes == BSFP8_CODES_E4M3FNUZ,
                                            static_cast<hipStream_t>(stream)));
}

int swiglu_backward(const void* dy, int64_t lddy, const void* gu, int64_t ldgu, int64_t T, int64_t F, void* dgu, int64_t lddgu,
                    void* stream) {
    if (T < 0 || F < 0 || F > 0x3FFFFFFF) return BSFP8_EINVAL;
    if (T == 0 || F == 0) return BSFP8_OK;
    if (dy == nullptr || gu == nullptr || dgu == nullptr || lddy < F || ldgu < 2 * F || lddgu < 2 * F) return BSFP8_EINVAL;
    if (cdiv(F, 512) > kMaxWaves / T) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_swiglu_backward(static_cast<const uint16_t*>(dy), lddy, static_cast<const uint16_t*>(gu), ldgu, T,
                                                F, static_cast<uint16_t*>(dgu), lddgu, static_cast<hipStream_t>(stream)));
}

int swiglu_backward_quantize(const void* dy, int64_t lddy, const void* gu, int64_t ldgu, int64_t T, int64_t F, int codes, void* q,
                             int64_t ldq, float* a_s, void* qT, int64_t ldqT, float* s, void* stream) {
    if (F < 0 || F > 0x3FFFFFFF) return BSFP8_EINVAL;
    if (int rc = validate_tiles(T, 2 * F, codes, q, ldq, a_s, qT, ldqT, s)) return rc;
    if (T == 0 || F == 0) return BSFP8_OK;
    if (dy == nullptr || gu == nullptr || lddy < F || ldgu < 2 * F) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    const bsfp8::TileCodes out{static_cast<uint8_t*>(q), ldq, a_s, static_cast<uint8_t*>(qT), ldqT, s};
    return finish(bsfp8::launch_swiglu_backward_dual(static_cast<const uint16_t*>(dy), lddy, static_cast<const uint16_t*>(gu), ldgu, T,
                                                     F, out, codes == BSFP8_CODES_E4M3FNUZ, static_cast<hipStream_t>(stream)));
}

int quantize_rows_i8(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, int64_t ldq, float* s, void* stream) {
    if (M < 0 || K < 0 || M > kMaxRows || K > 0x7FFFFFFF) return BSFP8_EINVAL;
    if (M == 0 || K == 0) return BSFP8_OK;
    if (x == nullptr || q == nullptr || s == nullptr || ldx < K || ldq < K) return BSFP8_EINVAL;
    if (int rc = check_device()) return rc;
    return finish(bsfp8::launch_quantize_rows_i8(static_cast<const uint16_t*>(x), ldx, M, K, static_cast<uint8_t*>(q), ldq, s,
                                                 static_cast<hipStream_t>(stream)));
}

int gemm_i8(const void* a, int64_t lda, const float* a_s, const void* b, int64_t ldb, const float* b_s, void* c, int64_t ldc,
            int64_t M, int64_t N, int64_t K, void* stream) {
    if (M < 0 || N < 0 || K < 0 || K > kMaxI8K) return BSFP8_EINVAL;
    if (M == 0 || N == 0) return BSFP8_OK;
    if (c == nullptr || ldc < N || cdiv(M, 64) > ((int64_t{1} << 22) - 1) / cdiv(N, 64)) return BSFP8_EINVAL;
    if (K > 0) {
        if (a == nullptr || a_s == nullptr || b == nullptr || b_s == nullptr || lda < K || ldb < K) return BSFP8_EINVAL;
        if (lda > kMaxOperandLd || ldb > kMaxOperandLd) return BSFP8_EINVAL;
        if (!aligned16(a) || !aligned16(b) || lda % 16 != 0 || ldb % 16 != 0) return BSFP8_EALIGN;
    }
    if (int rc = check_device()) return rc;
    const bsfp8::I8Args args{static_cast<const uint8_t*>(a), lda, a_s, static_cast<const uint8_t*>(b), ldb, b_s,
                             static_cast<uint16_t*>(c), ldc, M, N, K};
    return finish(bsfp8::launch_gemm_i8(args, bsfp8::device_cus(), static_cast<hipStream_t>(stream)));
}

int64_t grad_workspace(const int64_t* sizes, int64_t count) {
    const int64_t partials = grad_partials(sizes, count);
    return partials < 0 ? -1 : 8 * partials;
}

int grad_norm(const void* const* grads, const int64_t* sizes, const int* dtypes, int64_t count, float* norm, void* workspace,
              int64_t workspace_bytes, void* stream) {
    if (int rc = validate_grads(grads, sizes, dtypes, count, norm, workspace, workspace_bytes)) return rc;
    if (int rc = check_device()) return rc;
    double* partial = static_cast<double*>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool past = bsfp8::sched::grads_past_caches(grad_bytes(sizes, dtypes, count));
    const hipError_t e = for_grad_tables(grads, nullptr, sizes, dtypes, nullptr, count, [&](const bsfp8::GradTable& t, int64_t before) {
        return bsfp8::launch_grad_squares(t, past, partial + before, st);
    });
    if (e != hipSuccess) return BSFP8_EHIP;
    return finish(bsfp8::launch_grad_norm(partial, grad_partials(sizes, count), norm, st));
}

int clip_grads(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes, const int* out_dtypes,
               int64_t count, float max_norm, float eps, float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
    if (int rc = validate_grads(grads, sizes, dtypes, count, norm, workspace, workspace_bytes)) return rc;
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || !std::isfinite(eps)) return BSFP8_EINVAL;
    if (count > 0 && (outs == nullptr || out_dtypes == nullptr)) return BSFP8_EINVAL;
    for (int64_t i = 0; i < count; ++i) {
        if (!dtype_ok(out_dtypes[i]) || (sizes[i] > 0 && outs[i] == nullptr)) return BSFP8_EINVAL;
        if (sizes[i] > 0 && reinterpret_cast<uintptr_t>(outs[i]) % (out_dtypes[i] == BSFP8_F32 ? 4 : 2) != 0) return BSFP8_EINVAL;
    }
    try {
        if (!outputs_apart(grads, outs, sizes, dtypes, out_dtypes, count)) return BSFP8_EINVAL;
    } catch (const std::bad_alloc&) {
        return BSFP8_EHIP;
    }
    if (int rc = check_device()) return rc;
    double* partial = static_cast<double*>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t partials = grad_partials(sizes, count);
    if (partials == 0) return finish(bsfp8::launch_grad_norm(partial, 0, norm, st));
    const bool past = bsfp8::sched::grads_past_caches(grad_bytes(sizes, dtypes, count) + grad_bytes(sizes, out_dtypes, count));
    hipError_t e = for_grad_tables(grads, outs, sizes, dtypes, out_dtypes, count, [&](const bsfp8::GradTable& t, int64_t before) {
        return bsfp8::launch_grad_squares(t, past, partial + before, st);
    });
    if (e != hipSuccess) return BSFP8_EHIP;
    // the first launch of the clipped copies writes the norm
    return finish(for_grad_tables(grads, outs, sizes, dtypes, out_dtypes, count, [&](const bsfp8::GradTable& t, int64_t before) {
        return bsfp8::launch_grad_clip(t, past, partial, partials, max_norm, eps, before == 0 ? norm : nullptr, st);
    }));
}

}  // extern "C"
