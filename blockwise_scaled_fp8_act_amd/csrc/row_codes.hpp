// Device helpers of the operators that form values row by row and write them as 8-bit codes: sums and
// maxima over the threads of a row, scales, codes, and the order of workgroups over the rows.
#pragma once

#include "device_common.hpp"
#include "launch.hpp"

namespace bsfp8 {

typedef uint32_t rc_u32x4 __attribute__((ext_vector_type(4)));
typedef float rc_f32x4 __attribute__((ext_vector_type(4)));
typedef float rc_f2 __attribute__((ext_vector_type(2)));
typedef __bf16 rc_bf2 __attribute__((ext_vector_type(2)));

constexpr float kI8Max = 127.0f;
constexpr int kXcds = 8;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const rc_f2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, rc_bf2));
}
__device__ __forceinline__ uint16_t to_bf16_bits(float v) { return static_cast<uint16_t>(pack_bf16(v, 0.0f)); }

// Workgroups go to the XCDs in turn: workgroup b takes block (b % 8) per_xcd + b / 8, so that an XCD
// walks consecutive rows and its L2 collects the lines of the column-major scales, of which a row
// writes four bytes each.
__device__ __forceinline__ int64_t xcd_block(uint32_t b, int64_t per_xcd) {
    return static_cast<int64_t>(b % kXcds) * per_xcd + b / kXcds;
}

// The scale pair of a group from its largest magnitude (bit pattern). A group that holds a NaN has scale
// NaN and NaN multipliers, one that holds an infinity scale infinity: what it stands for is not finite
// in either case, also in int8, which has no code for that.
template <bool FNUZ = false>
__device__ __forceinline__ GroupScale fp8_scale(uint32_t amax) {
    GroupScale g = group_scale<FNUZ>(__uint_as_float(amax));
    if (amax > 0x7F800000u) g.s = g.m = __uint_as_float(amax);
    return g;
}
__device__ __forceinline__ GroupScale i8_scale(uint32_t amax) {
    const float a = fmaxf(__uint_as_float(amax), kAmaxEps);
    GroupScale g{a / kI8Max, kI8Max / a};
    if (amax > 0x7F800000u) g.s = g.m = __uint_as_float(amax);
    return g;
}

// The whole number nearest to v, ties to even, as a byte, for |v| <= 127 (1 + 2^-22): 1.5 2^23 + v is
// rounded at its last bit, which counts ones, and the low byte is the number in two's complement. The sum
// must not join the product before it: the definition rounds that to fp32 first.
__device__ __forceinline__ uint32_t i8_bits(float v) {
#pragma clang fp contract(off)
    return __float_as_uint(v + 12582912.0f);
}
__device__ __forceinline__ uint32_t i8_codes4(float a, float b, float c, float d) {
    const uint32_t lo = __builtin_amdgcn_perm(i8_bits(b), i8_bits(a), 0x0C0C0400u);
    return __builtin_amdgcn_perm(i8_bits(d), i8_bits(c), 0x04000C0Cu) | lo;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float m, int codes) {
#pragma clang fp contract(off)
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = v[j] * m;
    if (codes == kCodesI8) return make_uint2(i8_codes4(p[0], p[1], p[2], p[3]), i8_codes4(p[4], p[5], p[6], p[7]));
    uint2 w = make_uint2(encode4_in_range(p[0], p[1], p[2], p[3]), encode4_in_range(p[4], p[5], p[6], p[7]));
    if (codes == kCodesE4m3Fnuz) w = make_uint2(drop_negative_zero(w.x), drop_negative_zero(w.y));
    return w;
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
    uint32_t am = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) am = max(am, abs_bits(v[j]));
    return am;
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), CTRL, 0xF, 0xF, false));
}

// The sum over a wave, the same in every lane: within 16 lanes by DPP (the lanes of a pair, of a pair of
// pairs, mirrored halves and rows), then across the four rows.
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    v += dpp_f64<0x140>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f32<0xB1>(v);
    v += dpp_f32<0x4E>(v);
    v += dpp_f32<0x141>(v);
    v += dpp_f32<0x140>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// The same over the WAVES waves of a workgroup, in order of the waves. `part` is the caller's LDS, not
// written by another reduction before the next barrier.
template <int WAVES, typename V>
__device__ __forceinline__ V block_sum(V v, V* part) {
    v = wave_sum(v);
    if constexpr (WAVES == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    V sum = part[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) sum += part[i];
    return sum;
}
template <int WAVES>
__device__ __forceinline__ uint32_t block_umax(uint32_t v, uint32_t* part) {
    v = umax_wave(v);
    if constexpr (WAVES == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t top = part[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) top = max(top, part[i]);
    return top;
}

// The same types at any address: loads and stores of these are single instructions too.
typedef uint32_t rc_u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t rc_u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float rc_f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// Eight consecutive bf16 or fp32. ONCE: nothing here reads them again, so they are not kept in the caches (the
// norm with an fp32 residual, 8192 x 4096: 80 -> 75 us). ANY: at any address, and of the eight the first n alone (the
// others are 0, and are not touched); without it all eight are there, 16-byte aligned.
__device__ __forceinline__ void unpack8(rc_u32x4 w, float (&f)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        f[2 * d] = bf16_lo(w[d]);
        f[2 * d + 1] = bf16_hi(w[d]);
    }
}
template <bool ONCE, typename V>
__device__ __forceinline__ V load_piece(const V* p) {
    return ONCE ? __builtin_nontemporal_load(p) : *p;
}
// Not through load_piece: a deduced type loses the small alignment, and the load would count as 16-byte aligned.
template <bool ONCE>
__device__ __forceinline__ rc_u32x4 load_any(const uint16_t* p) {
    const rc_u32x4_any* q = reinterpret_cast<const rc_u32x4_any*>(p);
    return ONCE ? __builtin_nontemporal_load(q) : *q;
}
template <bool ONCE>
__device__ __forceinline__ rc_f32x4 load_any(const float* p) {
    const rc_f32x4_any* q = reinterpret_cast<const rc_f32x4_any*>(p);
    return ONCE ? __builtin_nontemporal_load(q) : *q;
}
template <bool ONCE = false, bool ANY = false>
__device__ __forceinline__ rc_u32x4 load8_bf16(const uint16_t* p, int64_t n = 8) {
    if (!ANY) return load_piece<ONCE>(reinterpret_cast<const rc_u32x4*>(p));
    if (n >= 8) return load_any<ONCE>(p);
    rc_u32x4 w = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < n) w[j / 2] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
    return w;
}
template <bool F32, bool ONCE = false, bool ANY = false>
__device__ __forceinline__ void load8_of(const void* p, int64_t at, float (&f)[8], int64_t n = 8) {
    if constexpr (!F32) {
        unpack8(load8_bf16<ONCE, ANY>(static_cast<const uint16_t*>(p) + at, n), f);
    } else {
        const float* q = static_cast<const float*>(p) + at;
        if (!ANY || n >= 8) {
            rc_f32x4 lo, hi;
            if (ANY) {
                lo = load_any<ONCE>(q);
                hi = load_any<ONCE>(q + 4);
            } else {
                lo = load_piece<ONCE>(reinterpret_cast<const rc_f32x4*>(q));
                hi = load_piece<ONCE>(reinterpret_cast<const rc_f32x4*>(q + 4));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j] = lo[j];
                f[4 + j] = hi[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = j < n ? q[j] : 0.0f;
        }
    }
}
__device__ __forceinline__ float load_of(const void* p, int64_t at, bool f32) {
    return f32 ? static_cast<const float*>(p)[at] : bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
}
// What store8_of writes of bf16.
__device__ __forceinline__ rc_u32x4 pack8(const float (&f)[8]) {
    return rc_u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}
template <bool ANY = false>
__device__ __forceinline__ void store8_bf16(uint16_t* p, rc_u32x4 w, int64_t n = 8) {
    if (!ANY) {
        *reinterpret_cast<rc_u32x4*>(p) = w;
    } else if (n >= 8) {
        *reinterpret_cast<rc_u32x4_any*>(p) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) p[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
    }
}
template <bool F32, bool ANY = false>
__device__ __forceinline__ void store8_of(void* p, int64_t at, const float (&f)[8], int64_t n = 8) {
    if constexpr (!F32) {
        store8_bf16<ANY>(static_cast<uint16_t*>(p) + at, pack8(f), n);
    } else {
        float* q = static_cast<float*>(p) + at;
        const rc_f32x4 lo = {f[0], f[1], f[2], f[3]}, hi = {f[4], f[5], f[6], f[7]};
        if (!ANY) {
            reinterpret_cast<rc_f32x4*>(q)[0] = lo;
            reinterpret_cast<rc_f32x4*>(q)[1] = hi;
        } else if (n >= 8) {
            *reinterpret_cast<rc_f32x4_any*>(q) = lo;
            *reinterpret_cast<rc_f32x4_any*>(q + 4) = hi;
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < n) q[j] = f[j];
        }
    }
}
template <bool ANY = false>
__device__ __forceinline__ void store8_codes(uint8_t* p, uint2 w, int64_t n = 8) {
    if (!ANY) {
        *reinterpret_cast<uint2*>(p) = w;
    } else if (n >= 8) {
        *reinterpret_cast<rc_u32x2_any*>(p) = rc_u32x2_any{w.x, w.y};
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < n) p[j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
}

// Writes the values v of one row as codes and scales, and in bf16 where out.y is set. The row's TPR
// threads (thread `tid`) hold the columns 8 (i TPR + tid) .. + 7 in v[i]; columns >= H are zero there,
// and without ANY H is a multiple of 8. A 1x128 group is one DPP row of 16 lanes.
template <int TPR, int NC, bool ANY>
__device__ __forceinline__ void emit_row(const RowCodes& out, int64_t row, int64_t T, int64_t H, int tid, const float (&v)[NC][8],
                                         uint32_t* part) {
    if (out.y != nullptr) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
            if (c < H) store8_of<false, ANY>(out.y, row * out.ldy + c, v[i], H - c);
        }
    }
    if (out.codes == kCodesNone) return;
    if (out.codes == kCodesI8) {
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < NC; ++i) am = max(am, amax8(v[i]));
        const GroupScale g = i8_scale(block_umax<TPR / 64>(am, part));
        if (tid == 0) out.s[row] = g.s;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
            if (c < H) store8_codes<ANY>(out.q + row * out.ldq + c, codes8(v[i], g.m, kCodesI8), H - c);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * (static_cast<int64_t>(i) * TPR + tid);
        const uint32_t am = umax_row16(amax8(v[i]));
        const GroupScale g = out.codes == kCodesE4m3Fnuz ? fp8_scale<true>(am) : fp8_scale<false>(am);
        if (c < H) {
            store8_codes<ANY>(out.q + row * out.ldq + c, codes8(v[i], g.m, out.codes), H - c);
            if ((tid & 15) == 0) out.s[c / kGroup * T + row] = g.s;
        }
    }
}

// The same for a row of any length: `value(c)` gives the value of column c, and is called
// again for each pass. One workgroup of WAVES waves; a wave takes a group of 128 columns at a time, lane
// l its columns l and l + 64.
template <int WAVES, typename F>
__device__ __forceinline__ void emit_row_any(const RowCodes& out, int64_t row, int64_t T, int64_t H, F value, uint32_t* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t Hb = (H + kGroup - 1) / kGroup;
    float m_row = 0.0f;
    if (out.codes == kCodesI8) {
        uint32_t am = 0;
        for (int64_t b = wave; b < Hb; b += WAVES)
            for (int j = 0; j < 2; ++j) {
                const int64_t c = b * kGroup + 64 * j + lane;
                if (c < H) am = max(am, abs_bits(value(c)));
            }
        const GroupScale g = i8_scale(block_umax<WAVES>(am, part));
        if (threadIdx.x == 0) out.s[row] = g.s;
        m_row = g.m;
    }
    for (int64_t b = wave; b < Hb; b += WAVES) {
        float v[2];
        for (int j = 0; j < 2; ++j) {
            const int64_t c = b * kGroup + 64 * j + lane;
            v[j] = c < H ? value(c) : 0.0f;
        }
        float m = m_row;
        if (out.codes == kCodesE4m3Fn || out.codes == kCodesE4m3Fnuz) {
            const uint32_t am = umax_wave(max(abs_bits(v[0]), abs_bits(v[1])));
            const GroupScale g = out.codes == kCodesE4m3Fnuz ? fp8_scale<true>(am) : fp8_scale<false>(am);
            if (lane == 0) out.s[b * T + row] = g.s;
            m = g.m;
        }
        for (int j = 0; j < 2; ++j) {
            const int64_t c = b * kGroup + 64 * j + lane;
            if (c >= H) continue;
            if (out.y != nullptr) out.y[row * out.ldy + c] = to_bf16_bits(v[j]);
            if (out.codes == kCodesNone) continue;
            const float p = v[j] * m;
            uint32_t w = (out.codes == kCodesI8 ? i8_bits(p) : encode4_in_range(p, 0.0f, 0.0f, 0.0f)) & 0xFFu;
            if (out.codes == kCodesE4m3Fnuz && w == 0x80u) w = 0;
            out.q[row * out.ldq + c] = static_cast<uint8_t>(w);
        }
    }
}

// Whether rows of a byte stride begin on whole pieces.
inline bool rows16(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bytes % 16 == 0; }
inline bool rows8(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && bytes % 8 == 0; }
inline bool whole_codes(const RowCodes& o) {
    return (o.codes == kCodesNone || rows8(o.q, o.ldq)) && (o.y == nullptr || rows16(o.y, 2 * o.ldy));
}

}  // namespace bsfp8
