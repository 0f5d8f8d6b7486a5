// Per-row 8-bit codes (E4M3 and symmetric INT8) shared by the kernels that write such rows: the
// row quantizers, and the norm, the gate and the cache write that quantize what they compute.
// All of them give the codes and scales that the row quantizers give for the same binary32
// values.
#pragma once

#include "w4_internal.h"

namespace w4 {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr double kFp8Max = 448.0;

// E4M3 rounding of a magnitude m <= 448: u = m in units of its grid step 2^(ex-3)
// (ex = its binary exponent, at least -6); scaling by a power of two is exact
__device__ __forceinline__ double e4m3_units(double m, int& ex) {
    int e = 0;
    (void)frexp(m, &e);                            // m = f * 2^e, f in [0.5, 1)
    ex = max(e - 1, -6);
    return ldexp(m, 3 - ex);
}

// byte of the rounded magnitude q * 2^(ex-3) with the given sign bit
__device__ __forceinline__ uint32_t e4m3_encode(uint32_t sign, double q, int ex) {
    const double r = fmin(ldexp(q, ex - 3), kFp8Max);
    if (r == 0.0) return sign;
    if (r < 0x1p-6) return sign | (uint32_t)(r * 512.0);   // subnormal: r = m * 2^-9
    int E = 0;
    const double f = frexp(r, &E);                 // r = (2f) * 2^(E-1)
    return sign | ((uint32_t)(E + 6) << 3) | (uint32_t)((2.0 * f - 1.0) * 8.0);
}

// E4M3 byte of a binary64 quotient t (the rounding described at the top of the file)
__device__ __forceinline__ uint32_t e4m3_byte(double t) {
    if (t == 0.0) return 0u;
    int ex = 0;
    const double u = e4m3_units(fmin(fabs(t), kFp8Max), ex);
    return e4m3_encode(t < 0.0 ? 0x80u : 0u, rint(u), ex);
}

// The codes without binary64 arithmetic per value.  r32 is 1 / s (correctly rounded in
// binary64, then to binary32), so t = v * r32 in binary32 is within 2^-23 relative of v / s
// and of its correctly rounded binary64 quotient.  In grid units (below 16 for E4M3, below
// 128 for INT8) the two differ by less than 2^-19 and 2^-16; where t lies more than 2^-17
// (E4M3) or 2^-13 (INT8) from a rounding boundary both give the same code.  The other
// values (windows of 2^-16 and 2^-12 per unit: about 1.5 in 10^5 and 2.4 in 10^4),
// non-finite ones and scales outside [2^-100, 2^100] take the binary64 quotient.  An E4M3
// quotient below 2^-12 rounds to a zero with the sign of v.
__device__ __forceinline__ bool clear_of_half(float u, float margin) {
    return fabsf(__builtin_amdgcn_fractf(u) - 0.5f) > margin;
}

__device__ __forceinline__ uint32_t e4m3_byte_recip(float v, double s, float r32, bool rcp_ok) {
    if (rcp_ok) {
        const float m = fabsf(v * r32);
        const uint32_t sign = v < 0.0f ? 0x80u : 0u;
        if (m < 0x1p-12f) return sign;
        const int ex = max(__builtin_amdgcn_frexp_expf(m) - 1, -6);   // binary exponent
        const float u = ldexpf(m, 3 - ex);                              // in units of 2^(ex-3)
        // below 448 * (1 + 2^-22), so u < 14.5 at ex = 8: no value rounds past 448
        if (clear_of_half(u, 0x1p-17f)) {
            // the byte of q * 2^(ex-3): exponent field ex + 7 and mantissa q - 8 for
            // 8 <= q <= 16 (q = 16 carries into the exponent), the subnormal q < 8 at ex = -6
            return sign | (uint32_t)(8 * ex + 48 + (int)rintf(u));
        }
    }
    return e4m3_byte((double)v / s);
}

template <bool IN_BF16>
__device__ __forceinline__ void load8(const void* a, int64_t i, float* v) {
    if constexpr (IN_BF16) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a) + i);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        }
    } else {
        const u32x4_t w0 = *reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a) + i);
        const u32x4_t w1 = *reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a) + i + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = __uint_as_float(w0[q]);
            v[4 + q] = __uint_as_float(w1[q]);
        }
    }
}

// INT8 (symmetric, page "Quantization" › "How it really works" and "Code"): the step is the
// row's largest magnitude over 127 (1 for an all-zero row), in binary64; code = the
// binary64 quotient rounded to the nearest integer, halves to even, clamped to [-128, 127].
__device__ __forceinline__ uint32_t int8_byte(double t) {
    const double q = fmin(fmax(rint(t), -128.0), 127.0);
    return (uint32_t)(uint8_t)(int8_t)(int)q;
}

__device__ __forceinline__ uint32_t int8_byte_recip(float v, double s, float r32, bool rcp_ok) {
    const float t = v * r32;
    if (rcp_ok && clear_of_half(t, 0x1p-13f))   // |t| <= 127 (1 + 2^-22): no clamp needed
        return (uint32_t)(uint8_t)(int8_t)(int)rintf(t);
    return int8_byte((double)v / s);
}

template <bool INT8>
__device__ __forceinline__ uint2 w8_codes8(const float* v, double s, float rs, bool rcp_ok) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (INT8) {
            lo |= int8_byte_recip(v[q], s, rs, rcp_ok) << (8 * q);
            hi |= int8_byte_recip(v[4 + q], s, rs, rcp_ok) << (8 * q);
        } else {
            lo |= e4m3_byte_recip(v[q], s, rs, rcp_ok) << (8 * q);
            hi |= e4m3_byte_recip(v[4 + q], s, rs, rcp_ok) << (8 * q);
        }
    }
    return make_uint2(lo, hi);
}

// The same codes for the kernels that have 8 values of a row in registers, with one branch for
// all of them; rcp_ok has to be false where one of them is not finite.  E4M3: t = v * r32 is within 2^-23 relative of v / s, and rounding is monotonic,
// so where t (1 - 2^-21) and t (1 + 2^-21) have the same byte it is the byte of v / s; about one
// value in 10^5 differs and sends the 8 to the binary64 quotients.  The conversion instruction
// rounds halves to even, subnormals included, and keeps the sign of a value that rounds to zero;
// the 0 added to the product makes an exact -0 the code 0x00.  INT8: v * r32 + 1.5 * 2^23 in one
// FMA leaves the nearest integer i in the low bits (halves to even), and v * r32 - i in another
// how far it is; within 2^-15 of a half (r32 accounts for 127 * 2^-24) the quotient decides.
template <bool INT8>
__device__ __forceinline__ uint2 w8_codes8_of(const float* v, double s, float rs, bool rcp_ok) {
    uint32_t w[2];
    if constexpr (INT8) {
        float far = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float x = v[4 * h + q];
                const float i = fmaf(x, rs, 0x1.8p23f);
                b[q] = __float_as_uint(i);
                far = fmaxf(far, fabsf(fmaf(x, rs, 0x1.8p23f - i)));
            }
            // byte 0 of each word
            w[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                         __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
        }
        if (rcp_ok && far < 0.5f - 0x1p-15f) return make_uint2(w[0], w[1]);
    } else {
        uint32_t differ = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int lo = 0, hi = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float t0 = fmaf(v[4 * h + 2 * q], rs, 0.0f), t1 = fmaf(v[4 * h + 2 * q + 1], rs, 0.0f);
                const float k0 = 1.0f - 0x1p-21f, k1 = 1.0f + 0x1p-21f;
                if (q == 0) {
                    lo = __builtin_amdgcn_cvt_pk_fp8_f32(t0 * k0, t1 * k0, lo, false);
                    hi = __builtin_amdgcn_cvt_pk_fp8_f32(t0 * k1, t1 * k1, hi, false);
                } else {
                    lo = __builtin_amdgcn_cvt_pk_fp8_f32(t0 * k0, t1 * k0, lo, true);
                    hi = __builtin_amdgcn_cvt_pk_fp8_f32(t0 * k1, t1 * k1, hi, true);
                }
            }
            differ |= (uint32_t)(lo ^ hi);
            w[h] = (uint32_t)lo;
        }
        if (rcp_ok && differ == 0) return make_uint2(w[0], w[1]);
    }
    return w8_codes8<INT8>(v, s, rs, rcp_ok);
}

}  // namespace
}  // namespace w4
