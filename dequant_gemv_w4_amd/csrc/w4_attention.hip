// Attention of new tokens over the paged cache:
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q.k_j - max),
// over the keys that a query sees, in one pass with the running maximum and sum of the softmax.
// The index arithmetic (tiles, parts, pages) is in w4_paging.h.
//
// Both kernels multiply on the matrix cores with the keys as rows and the query rows as columns
// (32x32x16 in attend_wide, 16x16x32 in attend_narrow): S^T = K Q^T leaves each lane one query row and
// a half or a quarter of the keys, so the running maximum is one or two exchanges between lanes, and
// the same registers, rounded to bfloat16, are the right operand of O^T += V^T P^T without any
// movement: which key stands at which place of that product's inner dimension is free, and the left
// operand follows (half h of the lanes holds the keys 4h..4h+3 and 8+4h..8+4h+3 of each 16, quarter h
// the keys 4h..4h+3 and 16+4h..16+4h+3 of 32).  V stays in its row order and is turned by
// ds_read_b64_tr_b16, which gives a lane four keys of one column.
//
// Rounding: scores, maximum, sum and O are binary32; the sum takes the unrounded P.  For the matrix unit
// attend_wide rounds P to bfloat16 (each weight within 2^-8 relative; the same size as the rounding of
// the bfloat16 output, and averaged over the keys: outputs are 1.4 times as far from 64 bits as an
// unrounded P would leave them).  attend_narrow, which waits for memory, multiplies V by what that
// rounding leaves as well (P = p + rest, both bfloat16, together within 2^-16): a decode step of 32
// requests takes 153.0 us instead of 152.3.  E4M3 codes enter as exact bfloat16 values; the scale of a
// key's row multiplies its scores, that of a value's row its P, both in binary32.
//
// attend_wide: 256 rows a workgroup, 8 waves of 32 rows; tiles of 64 keys pass through LDS for
// all of them, the next tiles' loads in flight, and the two waves of a SIMD take turns on the matrix
// unit.  Bound by the matrix unit and LDS together: two chunks of up to 2048 tokens over up to 6144
// cached (64 heads, 8 kv heads, 0.79 Tflop) take 722 to 763 us on different cards, 1.03 to 1.09 PFLOP/s
// where a large bfloat16 product of the vendor's library reaches 1.37; the matrix unit is busy for 51 % of
// the cycles, and the products without their LDS reads take 0.55 of the time.  64 rows a wave would halve
// those reads, with 512 registers and one wave a SIMD, which then has none to take turns with; half of
// those registers are out of the vector unit's reach, and the compiler moves 256 values a step for that.
// attend_narrow: 16 rows or 32, for single tokens: the waves take 32-key tiles in turn, each with its own
// piece of LDS, and join their sums at the end.  (Products of 32 rows for 8 rows, twice the registers and
// matrix work: 157.0 us instead of 152.9 for single tokens of 32 requests over up to 8192 cached, 86.2
// instead of 80.6 over 100,000 in E4M3, 13.8 instead of 12.8 for one request over 1000.)  Bound by
// memory: these 32 requests' 852 MB come at 5.6 TB/s, a plain read's rate being 5.9.  A short context is
// bound by latency: one request over 1000 keys (16 MB) takes 11.2 us, 8.3 of them one chain of lengths,
// table entries, rows, products and the waves' join, and 3 the launch that joins the parts.  Code that
// the chain runs once is paid at the rate at which instructions arrive (600 more cost 1.5 us: two tiles
// of loads in flight instead of one, in a loop unrolled by two, were dropped for that).
// Either may split the keys of a tile over several workgroups, which then leave (m, l, O / l) in
// the workspace for combine_kernel.
//
// Masked keys: scores are set to -inf by selection, so NaN there is harmless.  A masked value row
// meets a weight of zero in the matrix unit, where an infinity or NaN would survive as NaN: rows
// past the context are replaced by zeros when they are staged, and a query row whose result is not
// finite is computed again by attend_row, which skips masked keys.
#include "w4a16.h"
#include "w4_codes.h"
#include "w4_internal.h"
#include "w4_paging.h"

#include <type_traits>

namespace w4 {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr float kNegInf = -__builtin_huge_valf();
// O is rescaled when a row's maximum grows by more than this (in powers of two); until then the
// weights are up to 2^8 and the sums stay far inside binary32
constexpr float kSlack = 8.0f;

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const f32x2_t f = {a, b};
    const bf16x2_t h = __builtin_convertvector(f, bf16x2_t);
    return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// 16 bytes of E4M3 codes -> 16 bfloat16 values (exact)
__device__ __forceinline__ void fp8_to_bf16(const u32x4_t c, u32x4_t& lo, u32x4_t& hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false);
        const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true);
        const uint32_t ua = __builtin_bit_cast(uint32_t, a), ub = __builtin_bit_cast(uint32_t, b);
        if (i < 2) {
            lo[2 * i] = ua;
            lo[2 * i + 1] = ub;
        } else {
            hi[2 * (i - 2)] = ua;
            hi[2 * (i - 2) + 1] = ub;
        }
    }
}

// Places of 16-byte chunk c of key row r in LDS.  K is read 16 rows at a time at one chunk: the
// rows' chunks go to different bank groups.  V is read as 4 rows of 64 bytes: the rows go to
// different quarters of the banks.
template <int D>
__device__ __forceinline__ int k_place(int r, int c) {
    return r * (2 * D) + 16 * (D == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7));
}
template <int D>
__device__ __forceinline__ int v_place(int r, int c) {
    return r * (2 * D) + 16 * (c ^ (D == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2) ^ (((r >> 2) & 1) << 1));
}

__device__ __forceinline__ uint64_t read_tr(const uint8_t* p) {
    typedef __attribute__((address_space(3))) s16x4_t* lds_t;
    const s16x4_t r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p));
    return __builtin_bit_cast(uint64_t, r);
}

// Stages the 16 bytes that a lane loaded of key row r (chunk c of the stored row), zeros where r is not
// below `left` (the same for the wave; the rows of most tiles all stay).
template <int D, bool FP8, bool IS_V>
__device__ __forceinline__ void stage(uint8_t* tile, int r, int c, u32x4_t w, int left) {
    if (left < kKeyTile) {
        if (r >= left) w = u32x4_t{0u, 0u, 0u, 0u};
    }
    if constexpr (FP8) {
        u32x4_t lo, hi;
        fp8_to_bf16(w, lo, hi);
        *reinterpret_cast<u32x4_t*>(tile + (IS_V ? v_place<D>(r, 2 * c) : k_place<D>(r, 2 * c))) = lo;
        *reinterpret_cast<u32x4_t*>(tile + (IS_V ? v_place<D>(r, 2 * c + 1) : k_place<D>(r, 2 * c + 1))) = hi;
    } else {
        *reinterpret_cast<u32x4_t*>(tile + (IS_V ? v_place<D>(r, c) : k_place<D>(r, c))) = w;
    }
}

// The running state of 32 query rows: lane % 32 is the row, lane / 32 picks half of the keys in
// the scores and half of the columns in O (register r of block i: column 32 i + 8 (r / 4) +
// 4 (lane / 32) + r % 4).  l is the lane's own part of the sum.
template <int D>
struct Rows {
    u32x4_t q[D / 16];
    f32x16_t o[D / 32];
    float m, l;
};

template <int D>
__device__ __forceinline__ void clear_rows(Rows<D>& s) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s.o[i][r] = 0.0f;
    s.m = kNegInf;
    s.l = 0.0f;
}

// A step of attend_wide takes 64 keys in three parts.  The products read their left operands from LDS,
// which answers after about 130 cycles; a product takes 32.  The operands of four products are read
// while the four before them are in the matrix unit, and held to that order: left alone the compiler
// reads two to eight ahead, by what registers seem free (a chunk of 2048 + 1889 tokens: 737 us when it
// read eight ahead, 790 with two).
__device__ __forceinline__ void hold_order() { __builtin_amdgcn_sched_barrier(0); }

// scores: z = K q for the staged keys kt.
template <int D>
__device__ __forceinline__ void scores(const Rows<D>& s, const uint8_t* kt, f32x16_t (&z)[2]) {
    constexpr int kGroups = D / 32;
    const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    auto operand = [&](int d, int b) {
        return *reinterpret_cast<const u32x4_t*>(kt + k_place<D>(32 * b + l32, 2 * d + half));
    };
    auto multiply = [&](u32x4_t a, int d, int b) {
        z[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, s.q[d]), z[b], 0, 0, 0);
    };
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) z[b][r] = 0.0f;
    u32x4_t a[2][4];
#pragma unroll
    for (int g = 0; g <= kGroups; ++g) {
        if (g < kGroups) {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[g & 1][j] = operand(2 * g + j / 2, j % 2);
        }
        hold_order();
        if (g > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) multiply(a[(g - 1) & 1][j], 2 * (g - 1) + j / 2, j % 2);
        }
        hold_order();
    }
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}
__device__ __forceinline__ f32x4_t read_lds_f32x4(uint32_t address) {
    return *(__attribute__((address_space(3))) const f32x4_t*)(uintptr_t)address;
}

// Maximum over a lane and the one 32 lanes away.
__device__ __forceinline__ float half_max(float x) {
    const uint32_t u = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// Over the four lanes that are multiples of 16 apart.
__device__ __forceinline__ float quarter_max(float x) {
    const uint32_t u = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

// weights: the running maximum and sum, and the bfloat16 weights p (as the right operand of 16 keys
// each: p[4 c .. 4 c + 3]).  ks, vs: LDS addresses of the scales of the keys' and values' rows, from
// row 4 half on (FP8); first: position of the first key; the row sees the `count` keys from lo; mask:
// whether the step reaches outside some row's.
template <int D, bool FP8>
__device__ __forceinline__ void weights(Rows<D>& s, f32x16_t (&z)[2], uint32_t (&p)[16], uint32_t ks, uint32_t vs,
                                        float scale, int first, int lo, int count, bool mask) {
    const int half = (threadIdx.x & 63) >> 5;
    if constexpr (FP8) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4_t f = read_lds_f32x4(ks + 4 * (32 * b + 8 * i));
#pragma unroll
                for (int j = 0; j < 4; ++j) z[b][4 * i + j] *= f[j];
            }
    }
    if (mask) {
        const uint32_t from = (uint32_t)(first + 4 * half - lo);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (from + (32 * b + 8 * (r >> 2) + (r & 3)) >= (uint32_t)count) z[b][r] = kNegInf;
    }
    float mx = z[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, z[b][r]);
    mx = half_max(mx) * scale;                               // scale > 0
    if (__any(mx > s.m + kSlack)) {
        const float m = fmaxf(s.m, mx);
        const float f = m == s.m ? 1.0f : exp2_fast(s.m - m);
        s.m = m;
        s.l *= f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) s.o[i][r] *= f;
    }
    const float sub = s.m == kNegInf ? 0.0f : s.m;           // nothing seen yet: every weight is 0
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        f32x4_t f = {1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e0 = exp2_fast(fmaf(z[b][2 * i], scale, -sub));
            const float e1 = exp2_fast(fmaf(z[b][2 * i + 1], scale, -sub));
            sum[0] += e0;
            sum[1] += e1;
            float w0 = e0, w1 = e1;
            if constexpr (FP8) {
                if ((i & 1) == 0) f = read_lds_f32x4(vs + 4 * (32 * b + 4 * i));
                w0 *= f[2 * (i & 1)];
                w1 *= f[2 * (i & 1) + 1];
            }
            p[8 * b + i] = bf16_pair(w0, w1);
        }
    }
    s.l += sum[0] + sum[1];
}

// accumulate: O += V p for the staged values vt.
template <int D>
__device__ __forceinline__ void accumulate(Rows<D>& s, const uint8_t* vt, const uint32_t (&p)[16]) {
    constexpr int kBlocks = D / 32, kSteps = 4 / kBlocks;    // blocks of columns; steps of 16 keys in a group
    constexpr int kGroups = 4 / kSteps;
    const int lane = threadIdx.x & 63, half = lane >> 5, i16 = lane & 15, g16 = (lane >> 4) & 1;
    auto operand = [&](int c, int i) {                       // 16 keys, 32 columns
        const int r0 = 16 * c + 4 * half + (i16 >> 2);
        const int chunk = 4 * i + 2 * g16 + ((i16 & 3) >> 1), off = 8 * (i16 & 1);
        const uint64_t a0 = read_tr(vt + v_place<D>(r0, chunk) + off);
        const uint64_t a1 = read_tr(vt + v_place<D>(r0 + 8, chunk) + off);
        return u32x4_t{(uint32_t)a0, (uint32_t)(a0 >> 32), (uint32_t)a1, (uint32_t)(a1 >> 32)};
    };
    auto multiply = [&](u32x4_t a, int c, int i) {
        const u32x4_t pb = {p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]};
        s.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                         __builtin_bit_cast(bf16x8_t, pb), s.o[i], 0, 0, 0);
    };
    u32x4_t a[2][4];
#pragma unroll
    for (int g = 0; g <= kGroups; ++g) {
        if (g < kGroups) {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[g & 1][j] = operand(g * kSteps + j / kBlocks, j % kBlocks);
        }
        hold_order();
        if (g > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) multiply(a[(g - 1) & 1][j], (g - 1) * kSteps + j / kBlocks, j % kBlocks);
        }
        hold_order();
    }
}

// The running state of attend_narrow's 16 N query rows: lane % 16 is the row of each 16, lane / 16 picks a
// quarter of the keys in the scores and of the columns in O (register r of block i: column 16 i +
// 4 (lane / 16) + r).  l is the lane's own part of the sum.
template <int D, int N>
struct Few {
    u32x4_t q[N][D / 32];
    f32x4_t o[N][D / 16];
    float m[N], l[N];
    int lo[N], count[N];                                     // the rows see `count` keys from lo on
};

// A step of attend_narrow: the 32 staged keys from position `first` on.  sc: LDS address of the keys' row
// scales from row 4 (lane / 16) on, the values' 32 floats on; mask: whether the step reaches outside some
// row's keys.
template <int D, bool FP8, int N>
__device__ __forceinline__ void step_narrow(Few<D, N>& s, const uint8_t* kt, const uint8_t* vt, uint32_t sc, float scale,
                                            int first, bool mask) {
    const int lane = threadIdx.x & 63, i16 = lane & 15, quarter = lane >> 4;
    f32x4_t z[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int b = 0; b < 2; ++b) z[n][b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const u32x4_t k = *reinterpret_cast<const u32x4_t*>(kt + k_place<D>(16 * b + i16, 4 * d + quarter));
#pragma unroll
            for (int n = 0; n < N; ++n)
                z[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k),
                                                                  __builtin_bit_cast(bf16x8_t, s.q[n][d]), z[n][b], 0, 0, 0);
        }
    if constexpr (FP8) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const f32x4_t f = read_lds_f32x4(sc + 64 * b);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) z[n][b][r] *= f[r];
        }
    }
    if (mask) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t from = (uint32_t)(first + 4 * quarter - s.lo[n]);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (from + (16 * b + r) >= (uint32_t)s.count[n]) z[n][b][r] = kNegInf;
        }
    }
    float mx[N];
    bool grow = false;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        mx[n] = z[n][0][0];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) mx[n] = fmaxf(mx[n], z[n][b][r]);
        mx[n] = quarter_max(mx[n]) * scale;                  // scale > 0
        grow |= mx[n] > s.m[n] + kSlack;
    }
    if (__any(grow)) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float m = fmaxf(s.m[n], mx[n]);
            const float f = m == s.m[n] ? 1.0f : exp2_fast(s.m[n] - m);
            s.m[n] = m;
            s.l[n] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s.o[n][i][r] *= f;
        }
    }
    u32x4_t p[N], rest[N];                                   // and what the rounding left, itself within 2^-8
    float sub[N], sum[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        sub[n] = s.m[n] == kNegInf ? 0.0f : s.m[n];          // nothing seen yet: every weight is 0
        sum[n] = 0.0f;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        f32x4_t f = {1.0f, 1.0f, 1.0f, 1.0f};
        if constexpr (FP8) f = read_lds_f32x4(sc + 128 + 64 * b);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float e0 = exp2_fast(fmaf(z[n][b][2 * i], scale, -sub[n]));
                const float e1 = exp2_fast(fmaf(z[n][b][2 * i + 1], scale, -sub[n]));
                sum[n] += e0 + e1;
                const float w0 = FP8 ? e0 * f[2 * i] : e0, w1 = FP8 ? e1 * f[2 * i + 1] : e1;
                const uint32_t w = bf16_pair(w0, w1);
                p[n][2 * b + i] = w;
                rest[n][2 * b + i] = bf16_pair(w0 - __uint_as_float(w << 16), w1 - __uint_as_float(w & 0xFFFF0000u));
            }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) s.l[n] += sum[n];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {                       // 16 columns, the 32 keys in the order of p
        const int chunk = 2 * i + ((i16 & 3) >> 1), off = 8 * (i16 & 1), r0 = 4 * quarter + (i16 >> 2);
        const uint64_t a0 = read_tr(vt + v_place<D>(r0, chunk) + off);
        const uint64_t a1 = read_tr(vt + v_place<D>(r0 + 16, chunk) + off);
        const bf16x8_t v = __builtin_bit_cast(
            bf16x8_t, u32x4_t{(uint32_t)a0, (uint32_t)(a0 >> 32), (uint32_t)a1, (uint32_t)(a1 >> 32)});
#pragma unroll
        for (int n = 0; n < N; ++n) {
            s.o[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8_t, p[n]), s.o[n][i], 0, 0, 0);
            s.o[n][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8_t, rest[n]), s.o[n][i], 0, 0, 0);
        }
    }
}

// The last sequence b with key(cu[b], b) <= x, by all lanes of a wave: 64 sequences at a time, so two
// rounds of loads for up to 4096 sequences.  The sequence's own numbers are loaded in the same round.
template <typename Key>
__device__ __forceinline__ Seq find_seq(const AttendArgs& a, Key key, int x, int& found) {
    const int lane = threadIdx.x & 63;
    auto below = [&](int cu, int b) { return b < a.B && key(min(max(cu, 0), a.T), b) <= x; };
    int base = 0;
    if (a.B > 64) {
        const int b = lane * 64;
        base = __builtin_amdgcn_readfirstlane(max(__popcll(__ballot(below(a.cu[min(b, a.B - 1)], b))) - 1, 0) * 64);
    }
    const int b = min(base + lane, a.B - 1);
    const int cu0 = a.cu[b], cu1 = a.cu[b + 1], len = a.lens[b];
    const int at = __builtin_amdgcn_readfirstlane(max(__popcll(__ballot(below(cu0, base + lane))) - 1, 0));
    found = base + at;
    return clamp_seq(__builtin_amdgcn_readlane(cu0, at), __builtin_amdgcn_readlane(cu1, at),
                     __builtin_amdgcn_readlane(len, at), a.T, a.capacity);
}

__device__ __forceinline__ Seq load_seq(const AttendArgs& a, int b) {
    return clamp_seq(a.cu[b], a.cu[b + 1], a.lens[b], a.T, a.capacity);
}

// Row of the cache that holds a key (times D elements), or -1 where the table names no page.
__device__ __forceinline__ int64_t key_row(const AttendArgs& a, int b, int kv, int64_t key) {
    const int64_t page = checked_page(a.table[(int64_t)b * a.max_pages + (key >> a.page_shift)], a.pages);
    if (page < 0) return -1;
    return ((page * a.kv_heads + kv) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
}

// One query row over keys [k0, k1) by one wave, D / 64 columns a lane, skipping masked keys; O is
// kept divided by the sum, so values near the end of the range do not overflow.
template <int D, bool FP8>
__device__ void attend_row(const AttendArgs& a, int b, int kv, int64_t row, int64_t k0, int64_t k1,
                           int lo, int hi, float* o, float& m_out, float& l_out) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    float q[E], m = kNegInf, l = 0.0f;
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float((uint32_t)a.q[row * D + lane * E + e] << 16);
        o[e] = 0.0f;
    }
    const int64_t last = imin(k1 - 1, hi), page_rows = (int64_t)1 << a.page_shift;
    for (int64_t j = k0 > lo ? k0 : lo; j <= last;) {
        const int64_t at = key_row(a, b, kv, j);
        float z = 0.0f, v[E], count = 1.0f;
        for (int e = 0; e < E; ++e) v[e] = 0.0f;
        if (at < 0) {                                        // zeros up to the end of the page
            const int64_t next = imin(last + 1, (j / page_rows + 1) * page_rows);
            count = (float)(next - j);
            j = next;
        } else {
            for (int e = 0; e < E; ++e) {
                const int64_t i = at * D + lane * E + e;
                float k;
                if constexpr (FP8) {
                    k = __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(a.k)[i], 0) * a.k_scales[at];
                    v[e] = __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(a.v)[i], 0) * a.v_scales[at];
                } else {
                    k = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.k)[i] << 16);
                    v[e] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.v)[i] << 16);
                }
                z = fmaf(q[e], k, z);
            }
            for (int off = 32; off > 0; off >>= 1) z += __shfl_xor(z, off);
            z *= a.scale_log2;
            ++j;
        }
        const float mn = z != z ? z : fmaxf(m, z);
        const float keep = mn == m ? 1.0f : exp2_fast(m - mn);
        const float p = mn == kNegInf ? 0.0f : count * exp2_fast(z - mn);
        const float ln = l * keep + p;
        if (!(ln == 0.0f)) {
            const float fo = l * keep / ln, fv = p / ln;
            for (int e = 0; e < E; ++e) o[e] = (fo == 0.0f ? 0.0f : o[e] * fo) + v[e] * fv;
        }
        l = ln;
        m = mn;
    }
    m_out = m;
    l_out = l;
}

// What a row's sum of weights divides by: a row that sees no key gives zeros, one that sees keys
// of weight zero only (every score -inf) 0/0 like the formula.
__device__ __forceinline__ float inverse(float l, bool sees) {
    return l == 0.0f ? (sees ? __builtin_nanf("") : 0.0f) : 1.0f / l;
}

struct Tile {
    Seq seq;
    Span span;
    int b;
    int64_t part_row;  // the tile's first row in the workspace
    int row0;          // first row of the tile in its sequence
    int rows;          // rows of the sequence
    int k0, k1;        // keys of this workgroup's part
    bool run;
};

// Tile number `index` of R rows: of attend_wide's (R = kWideRows) or attend_narrow's.
template <int R>
__device__ __forceinline__ Tile find_tile(const AttendArgs& a, uint32_t index, int part, int& kv) {
    constexpr bool WIDE = R == kWideRows;
    Tile t;
    const int G = a.group;
    const int tile = __builtin_amdgcn_readfirstlane((int)(index / (uint32_t)a.kv_heads));
    kv = (int)index - tile * a.kv_heads;
    t.part_row = (int64_t)index * R;
    if (!WIDE && a.both) {
        t.b = few_sequence(tile, a.B);
        t.row0 = few_row0(tile, a.B, R);
        t.seq = load_seq(a, t.b);
    } else {
        const bool by_token = !WIDE && a.T == a.B;
        auto first = [&](int cu_b, int b) { return by_token ? token_tile(cu_b, G, R) : first_tile(cu_b, b, G, R); };
        t.seq = find_seq(a, first, tile, t.b);
        t.row0 = (tile - first(t.seq.start, t.b)) * R;
    }
    t.rows = t.seq.n * G;
    t.run = tile_runs(WIDE, a.both, t.row0, t.rows, a.few_tiles);
    if (!t.run) return t;
    const int reach = a.window > 0 ? min(t.seq.ctx, a.window) : t.seq.ctx;
    const int parts = !WIDE ? (a.both && t.rows > R ? a.narrow_fill : a.narrow_parts) : reach < kWideEven ? a.wide_fill : a.wide_parts;
    t.span = seen_span(key_span(t.seq, t.row0, min(R, t.rows - t.row0), G, a.window, parts, WIDE ? kWideLeast : kNarrowLeast));
    t.run = part < t.span.parts;
    if (!t.run) return t;
    t.k0 = t.span.begin + part * t.span.chunk;
    t.k1 = min(t.span.end - t.k0, t.span.chunk) + t.k0;
    return t;
}

// The place of a row of the tile: its row in q and o, and the keys it sees.
struct Place {
    int row;           // token * heads + head
    int lo, hi, count; // lo <= key <= hi
    bool real;
};
__device__ __forceinline__ Place row_place(const AttendArgs& a, const Tile& t, int kv, int r) {
    Place p;
    p.real = r < t.rows;
    const int token = p.real ? quotient(r, a.group) : 0;
    p.row = (t.seq.start + token) * a.heads + kv * a.group + (p.real ? r - token * a.group : 0);
    p.hi = p.real ? t.seq.ctx - t.seq.n + token : -1;
    p.lo = a.window > 0 ? max(0, p.hi - a.window + 1) : 0;
    p.count = max(0, p.hi - p.lo + 1);
    return p;
}

// Rows past the last stand for the first: what comes of them is not stored.
template <int N>
__device__ __forceinline__ void load_q(const uint16_t* q, u32x4_t (&out)[N], int step) {
#pragma unroll
    for (int d = 0; d < N; ++d) out[d] = *reinterpret_cast<const u32x4_t*>(q + d * step);
}
// The wait for these loads: left to the first product, inside the loop, it would be a wait for the tile
// loads in flight at every step.  attend_narrow has it behind the first tile's loads.
template <int N>
__device__ __forceinline__ void wait_q(u32x4_t (&q)[N]) {
#pragma unroll
    for (int d = 0; d < N; ++d) asm volatile("" : "+v"(q[d]));
}

// Stores 4 neighbouring columns of a row that are already divided by its sum.
template <bool WIDE>
struct Parts {
    float* o;          // [parts][rows of all tiles][D]
    float* ml;         // [parts][rows of all tiles][2]
    int64_t rows;
    __device__ explicit Parts(const AttendArgs& a)
        : o(WIDE ? a.wide_o : a.narrow_o), ml(WIDE ? a.wide_ml : a.narrow_ml),
          rows(WIDE ? a.wide_rows : a.narrow_rows) {}
    __device__ int64_t at(const Tile& t, int part, int r) const { return part * rows + t.part_row + r; }
};

template <bool WIDE>
__device__ __forceinline__ void store4(const AttendArgs& a, const Tile& t, int part, int r, int64_t row,
                                       int D, int col, f32x4_t v) {
    if (t.span.parts == 1) {
        const uint2 w = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
        *reinterpret_cast<uint2*>(a.o + row * D + col) = w;
    } else {
        const Parts<WIDE> w(a);
        *reinterpret_cast<f32x4_t*>(w.o + w.at(t, part, r) * D + col) = v;
    }
}

template <bool WIDE>
__device__ __forceinline__ void store_ml(const AttendArgs& a, const Tile& t, int part, int r, float m, float l) {
    const Parts<WIDE> w(a);
    float* p = w.ml + 2 * w.at(t, part, r);
    p[0] = m;
    p[1] = l;
}

// Computes the rows of `bad` (one bit per row from row r0 of the tile) again.
template <int D, bool FP8, bool WIDE>
__device__ void redo_rows(const AttendArgs& a, const Tile& t, int part, int kv, int r0, uint32_t bad) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    while (bad) {
        const int r = r0 + __ffs(bad) - 1;
        bad &= bad - 1;
        const Place p = row_place(a, t, kv, t.row0 + r);
        float o[E], m, l;
        attend_row<D, FP8>(a, t.b, kv, p.row, t.k0, t.k1, p.lo, p.hi, o, m, l);
        if (t.span.parts == 1) {
            const bool sees = p.hi >= 0;
            for (int e = 0; e < E; ++e) {
                const float v = l == 0.0f && sees ? __builtin_nanf("") : o[e];
                a.o[(int64_t)p.row * D + lane * E + e] = (uint16_t)bf16_pair(v, v);
            }
        } else {
            const Parts<WIDE> w(a);
            for (int e = 0; e < E; ++e) w.o[w.at(t, part, r) * D + lane * E + e] = o[e];
            if (lane == 0) store_ml<WIDE>(a, t, part, r, m, l);
        }
    }
}

// The rows of one sequence and kv head, for loads whose page is the same for a whole wave: offsets
// are formed once per 16 keys, in scalar registers.
template <int ROW_BYTES>
struct Rows16 {
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t* table;
    uint32_t pages, page_bytes, worst;                       // worst: the largest page number met
    int shift, end;                                          // keys below `end` are wanted

    __device__ Rows16(const AttendArgs& a, int b, int kv, int end_) {
        const int64_t head = (int64_t)kv << a.page_shift;
        k = static_cast<const uint8_t*>(a.k) + head * ROW_BYTES;
        v = static_cast<const uint8_t*>(a.v) + head * ROW_BYTES;
        ks = a.k_scales + head;
        vs = a.v_scales + head;
        table = a.table + (int64_t)b * a.max_pages;
        pages = (uint32_t)a.pages;
        page_bytes = (uint32_t)(a.kv_heads * ROW_BYTES) << a.page_shift;   // < 2^31
        shift = a.page_shift;
        end = end_;
        worst = 0;
    }
    __device__ __forceinline__ bool missing() const { return worst >= pages; }
    // Table entry of a key (the same for the wave); keys past the end read the last one's.
    __device__ __forceinline__ int entry(int key) const {
        // through the scalar cache: the answer does not pass in the order of the vector loads
        const auto t = (__attribute__((address_space(4))) const int32_t*)(uintptr_t)table;
        return t[(uint32_t)(min(__builtin_amdgcn_readfirstlane(key), end - 1) >> shift)];
    }
    // The same with a key for each lane.
    __device__ __forceinline__ int entry_by_lane(int key) const { return table[(uint32_t)(min(key, end - 1) >> shift)]; }
    // Byte offset of the row of `key` (a multiple of 16, the same for the wave) by its entry.  For a
    // page that the cache does not have it is that of a row of its last page: the kernel then computes
    // its rows again (attend_row).
    __device__ __forceinline__ uint64_t offset(int e, int key) {
        worst = max(worst, (uint32_t)e);
        return (uint64_t)min((uint32_t)e, pages - 1) * page_bytes + (uint32_t)((key & ((1 << shift) - 1)) * ROW_BYTES);
    }
};

__device__ __forceinline__ u32x4_t load16(const uint8_t* base, uint64_t offset, uint32_t lane_byte) {
    return *reinterpret_cast<const u32x4_t*>(base + offset + lane_byte);
}

// 16 bytes a lane from the cache straight into LDS: lane l of the wave writes bytes [16 l, 16 l + 16)
// after the wave-uniform LDS address.  Inline assembly, so that the compiler does not hold the LDS
// reads of other tiles back behind these loads; the kernel waits for them itself (vmcnt) before the
// barrier that publishes them.
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t lane_byte, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(lane_byte), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory", "m0");
}

constexpr int kThreads = 512;                                // of either kernel: 8 waves
constexpr int kWideStages = 4;

// LDS of either kernel: the keys, the values and the rest.  Three arrays, not one: the offset in an LDS
// instruction ends at 64 KB, and within one array every place of the values would take registers for
// addresses of its own.
template <int D>
struct Lds {
    uint8_t (&k)[kWideStages * kKeyTile * 2 * D];
    uint8_t (&v)[kWideStages * kKeyTile * 2 * D];
    union Rest {
        struct {
            float scales[2][kWideStages][kKeyTile];          // of keys, of values
            int any_missing;
        } wide;
        struct {
            float scales[kThreads / 64][2 * 32];
            float m[kThreads / 64][kFewRows], l[kThreads / 64][kFewRows];
            uint32_t redo;
        } narrow;
        __device__ Rest() {}
    } &rest;
};

// Tile `index` of the wide ones, its part `part` of the keys.
template <int D, bool FP8>
__device__ __forceinline__ void attend_wide(const AttendArgs& a, uint32_t index, int part, const Lds<D>& lds) {
    constexpr int kRowBytes = FP8 ? D : 2 * D;               // of a cached row
    constexpr int kChunks = kRowBytes / 16;
    constexpr int kStepRows = kThreads / kChunks;        // rows that one load of all threads covers
    constexpr int kLoads = kStepRows >= kKeyTile ? 1 : kKeyTile / kStepRows;
    constexpr int kTileBytes = kKeyTile * 2 * D;
    auto& kt = reinterpret_cast<uint8_t(&)[kWideStages][kTileBytes]>(lds.k);
    auto& vt = reinterpret_cast<uint8_t(&)[kWideStages][kTileBytes]>(lds.v);
    auto& sc_lds = lds.rest.wide.scales;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    int kv;
    const Tile t = find_tile<kWideRows>(a, index, part, kv);
    if (!t.run) return;
    Place p = row_place(a, t, kv, t.row0 + 32 * wave + (lane & 31));
    Rows<D> s;
    load_q(a.q + (int64_t)p.row * D + 8 * (lane >> 5), s.q, 16);
    wait_q(s.q);                                             // behind the first tile's loads: 1.6 % slower
    clear_rows<D>(s);
    // keys that any row of this wave sees, and those that all of them see
    int any_lo = p.real ? p.lo : W4_MAX_CONTEXT, any_hi = p.hi, all_lo = p.lo, all_hi = p.real ? p.hi : W4_MAX_CONTEXT;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        any_lo = min(any_lo, __shfl_xor(any_lo, off));
        any_hi = max(any_hi, __shfl_xor(any_hi, off));
        all_lo = max(all_lo, __shfl_xor(all_lo, off));
        all_hi = min(all_hi, __shfl_xor(all_hi, off));
    }
    any_lo = __builtin_amdgcn_readfirstlane(any_lo);
    any_hi = __builtin_amdgcn_readfirstlane(any_hi);
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);

    // the same for all, which the compiler has to know for what follows to stay in scalar registers
    const int k0 = __builtin_amdgcn_readfirstlane((int)t.k0), k1 = __builtin_amdgcn_readfirstlane((int)t.k1);
    const int tiles = (k1 - k0 + kKeyTile - 1) / kKeyTile;
    const int crow = tid / kChunks, chunk = tid % kChunks;
    const bool loads = kStepRows * kLoads == kKeyTile || crow < kKeyTile;   // else more threads than chunks
    // The rows that one load of a wave covers lie in one aligned group of 16, so in one page.
    const int granule = __builtin_amdgcn_readfirstlane(crow & ~15) & (kKeyTile - 1);
    Rows16<kRowBytes> rows(a, __builtin_amdgcn_readfirstlane(t.b), __builtin_amdgcn_readfirstlane(kv), k1);
    int entry[kLoads];                                       // of the tile whose keys are brought next
    uint64_t off[kLoads];                                    // of the tile whose values are brought next
    auto look_up = [&](int i) {                              // read here, used by locate
#pragma unroll
        for (int c = 0; c < kLoads; ++c) entry[c] = rows.entry(k0 + i * kKeyTile + granule + c * kStepRows);
    };
    auto locate = [&](int i) {
#pragma unroll
        for (int c = 0; c < kLoads; ++c) off[c] = rows.offset(entry[c], k0 + i * kKeyTile + granule + c * kStepRows);
    };
    // Rows of a tile that are past the part become zeros, so that what lies there in the cache does not
    // meet a weight of zero.
    auto left = [&](int i) { return k1 - k0 - i * kKeyTile; };

    // A bfloat16 tile goes straight into LDS: a lane loads the chunk whose place it is.  An E4M3 tile
    // passes through registers (kw, vw), where its codes are widened.
    const int crow16 = crow & 15;
    const uint32_t lane_k = crow16 * kRowBytes + (FP8 ? 16 * chunk : k_place<D>(crow, chunk) - crow * 2 * D);
    const uint32_t lane_v = crow16 * kRowBytes + (FP8 ? 16 * chunk : v_place<D>(crow, chunk) - crow * 2 * D);
    const uint32_t lds_k = lds_address(&kt[0][0]) + wave * 1024, lds_v = lds_address(&vt[0][0]) + wave * 1024;
    u32x4_t kw, vw;
    float sc = 1.0f;
    auto bring = [&](int i, bool values) {
        const uint8_t* from = values ? rows.v : rows.k;
        const uint32_t lane_byte = values ? lane_v : lane_k;
        if constexpr (FP8) {
            static_assert(!FP8 || kLoads == 1, "one row a thread");
            (values ? vw : kw) = load16(from, off[0], lane_byte);
            if (!values) sc = (chunk & 1 ? rows.vs : rows.ks)[off[0] / kRowBytes + crow16];
        } else {
            const uint32_t lds = (values ? lds_v : lds_k) + (i % kWideStages) * kTileBytes;
            if (left(i) >= kKeyTile) {
#pragma unroll
                for (int c = 0; c < kLoads; ++c) load_lds16(from + off[c], lane_byte, lds + c * (kStepRows * 2 * D));
            } else {
                uint8_t* tile = values ? vt[i % kWideStages] : kt[i % kWideStages];
#pragma unroll
                for (int c = 0; c < kLoads; ++c) {
                    if (crow + c * kStepRows < left(i))
                        load_lds16(from + off[c], lane_byte, lds + c * (kStepRows * 2 * D));
                    else
                        *reinterpret_cast<u32x4_t*>(tile + c * (kStepRows * 2 * D) + 16 * tid) = u32x4_t{0u, 0u, 0u, 0u};
                }
            }
        }
    };
    auto put = [&](int i, bool values) {                     // FP8: what bring loaded
        if (!loads) return;
        int at = i % kWideStages;
        asm volatile("" : "+s"(at));                         // addresses formed here, not kept for every place
        if (values) {
            stage<D, true, true>(vt[at], crow, chunk, vw, left(i));
        } else {
            stage<D, true, false>(kt[at], crow, chunk, kw, left(i));
            if (chunk < 2) sc_lds[chunk][at][crow] = crow < left(i) ? sc : 1.0f;
        }
    };
    // Waits for this wave's LDS accesses and then for the other waves; loads of the cache stay in
    // flight, and nothing is moved across.
    auto meet = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Tiles that some row of this wave sees, and those among them that all rows see whole.
    const int seen_lo = (any_lo - k0) >> 6, seen_hi = min(tiles - 1, (any_hi - k0) >> 6);
    const int whole_lo = (all_lo - k0 + kKeyTile - 1) >> 6, whole_hi = ((all_hi - k0 + 1) >> 6) - 1;
    static_assert(kKeyTile == 64, "shifts by 6");
    auto seen = [&](int i) { return i >= seen_lo && i <= seen_hi; };

    // Waves 0-3 and 4-7 (one of either on each SIMD) take turns: while one half is on the matrix
    // unit with O += V(i) P(i) and S = K(i+1) q, the other is on the vector unit with the weights of
    // its tile.  Phase by phase (A: weights, B: products; a barrier after each), the second half one
    // phase behind:
    //     phase        2i            2i+1          2i+2
    //     waves 0-3    A(i)          B(i)          A(i+1)
    //     waves 4-7    B(i-1)        A(i)          B(i)
    // "Pair n", V(n) and K(n+1), is read in phases 2n+1 and 2n+2; LDS has four places for either.
    // Each wave brings its share of pair n at the end of its A: of a bfloat16 cache at A(n-2) of waves
    // 0-3 and A(n-3) of waves 4-7, phases 2n-4 and 2n-5, two pairs ahead of the one that has landed
    // by the end of that phase; its place was pair n-4's, read last in phase 2n-6.  E4M3 rows are one
    // pair ahead in registers and staged in phases 2n (A(n)) and 2n-1 (A(n-1)).  Row scales come with
    // the keys of their tile: those of tile i are staged in phase 2i-2 at the latest, read in A(i), and
    // written over by those of tile i+4 in phase 2i+5 at the earliest.
    constexpr int kAhead = FP8 ? 1 : 2;                      // pairs in flight
    const int behind = wave >> 2;                            // 1 for waves 4-7
    uint32_t sc_lane = lds_address(&sc_lds[0][0][0]) + 16 * (lane >> 5);
    asm volatile("" : "+v"(sc_lane));                        // one register for all places
    f32x16_t z[2];
    uint32_t pw[16];
    if (tid == 0) lds.rest.wide.any_missing = 0;
    if (tiles > 0) {
        const int early = rows.entry_by_lane(k0 + 16 * lane);   // of the first 16 groups of 16 keys, in one load
        for (int i = 0; i <= kAhead + 1; ++i) {              // K(0), V(0), K(1), V(1) ...
            if (i >= tiles) break;
            static_assert((kAhead + 2) * kKeyTile <= 64 * 16, "a lane for each group");
#pragma unroll
            for (int c = 0; c < kLoads; ++c)
                entry[c] = __builtin_amdgcn_readlane(early, (i * kKeyTile + granule + c * kStepRows) >> 4);
            locate(i);
            bring(i, false);
            if (FP8 && i <= 1) put(i, false);
            if (i <= kAhead) bring(i, true);
            if (FP8 && i == 0) put(i, true);
            if (!FP8 && i == 1) {                            // K(0), V(0) and K(1) are needed at once
                if (left(1) >= kKeyTile)
                    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
                else
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
        }
        if (!FP8 && tiles < 2) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    meet();
    if (seen(0)) scores<D>(s, kt[0], z);
    if (behind) meet();
    // One step, tile i in place S = i % kWideStages.
    auto step = [&](auto place, int i) {
        constexpr int S = decltype(place)::value;
        const int n = i + behind;
        look_up(n + kAhead + 1);
        if (seen(i))
            weights<D, FP8>(s, z, pw, sc_lane + 4 * S * kKeyTile, sc_lane + 4 * (kWideStages + S) * kKeyTile, a.scale_log2,
                            k0 + i * kKeyTile, p.lo, p.count, i < whole_lo || i > whole_hi);
        if (n >= 1 && n < tiles) {
            if constexpr (FP8) {
                put(n, true);
                if (n + 1 < tiles) put(n + 1, false);
            } else if (left(n + 2) >= kKeyTile) {            // pair n + 1 may stay in flight
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kLoads) : "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
            if (n + kAhead < tiles) bring(n + kAhead, true);
            if (n + kAhead + 1 < tiles) {
                locate(n + kAhead + 1);
                bring(n + kAhead + 1, false);
            }
        }
        meet();
        __builtin_amdgcn_s_setprio(1);
        if (seen(i)) accumulate<D>(s, vt[S], pw);
        if (seen(i + 1)) scores<D>(s, kt[(S + 1) % kWideStages], z);
        __builtin_amdgcn_s_setprio(0);
        meet();
    };
    static_assert(kWideStages == 4, "the loop is unrolled over the places");
    for (int i = 0; i < tiles; i += 4) {
        step(std::integral_constant<int, 0>(), i);
        if (i + 1 < tiles) step(std::integral_constant<int, 1>(), i + 1);
        if (i + 2 < tiles) step(std::integral_constant<int, 2>(), i + 2);
        if (i + 3 < tiles) step(std::integral_constant<int, 3>(), i + 3);
    }
    if (!behind) meet();
    if (rows.missing()) lds.rest.wide.any_missing = 1;
    __syncthreads();
    const bool missing = lds.rest.wide.any_missing != 0;
    if (missing && tid == 0 && a.status) atomicOr(a.status, kStatusPage);

    // where the row goes is found again here: kept through the loop it would cost registers
    int r = 32 * wave + (lane & 31);
    asm volatile("" : "+v"(r));
    p = row_place(a, t, kv, t.row0 + r);
    const float l = s.l + __shfl_xor(s.l, 32);
    const bool whole = t.span.parts == 1;
    const float inv = inverse(l, whole && p.hi >= 0);
    const int half = lane >> 5;
    bool bad = !isfinite(l);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f32x4_t v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bad |= !isfinite(s.o[i][4 * g + j]);
                v[j] = s.o[i][4 * g + j] * inv;
            }
            if (p.real) store4<true>(a, t, part, r, p.row, D, 32 * i + 8 * g + 4 * half, v);
        }
    if (p.real && !whole && half == 0) store_ml<true>(a, t, part, r, s.m, l);
    const uint64_t mask = __ballot((bad || missing) && p.real);
    const uint32_t again = (uint32_t)mask | (uint32_t)(mask >> 32);
    if (again) {
        __threadfence();                                     // the rows' first results have landed
        redo_rows<D, FP8, true>(a, t, part, kv, 32 * wave, again);
    }
}

constexpr int kNarrowWaves = kThreads / 64;

// Tile `index` of the narrow ones, its part `part` of the keys.
template <int D, bool FP8, int N>
__device__ __forceinline__ void attend_narrow(const AttendArgs& a, uint32_t index, int part, const Lds<D>& lds) {
    constexpr int kRows = 16 * N;
    constexpr int kKeys = 32;                                // of a wave's tile
    constexpr int kRowBytes = FP8 ? D : 2 * D;
    constexpr int kChunks = kRowBytes / 16;
    constexpr int kStepRows = 64 / kChunks;                  // rows that one load of the wave covers
    constexpr int kLoads = kKeys / kStepRows;
    constexpr int kTileBytes = kKeys * 2 * D;
    static_assert(kNarrowWaves * kTileBytes <= sizeof(lds.k) && kTileBytes >= 16 * D * 4 && N <= 2,
                  "a tile a wave, and at the end its O in the place of the keys and, of rows past 16, the values");
    auto& scales = lds.rest.narrow.scales;
    auto& lds_m = lds.rest.narrow.m;
    auto& lds_l = lds.rest.narrow.l;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    int kv;
    const Tile t = find_tile<kRows>(a, index, part, kv);
    if (!t.run) return;
    const int i16 = lane & 15, quarter = lane >> 4;
    Few<D, N> s;
    int all_lo = 0, all_hi = W4_MAX_CONTEXT;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const Place p = row_place(a, t, kv, t.row0 + 16 * n + i16);
        load_q(a.q + (int64_t)p.row * D + 8 * quarter, s.q[n], 32);
        s.lo[n] = p.lo;
        s.count[n] = p.count;
        all_lo = max(all_lo, p.lo);
        all_hi = min(all_hi, p.real ? p.hi : W4_MAX_CONTEXT);
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
        all_lo = max(all_lo, __shfl_xor(all_lo, off));
        all_hi = min(all_hi, __shfl_xor(all_hi, off));
    }
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);

    // the same for all, which the compiler has to know for what follows to stay in scalar registers
    const int k0 = __builtin_amdgcn_readfirstlane((int)t.k0), k1 = __builtin_amdgcn_readfirstlane((int)t.k1);
    uint8_t* kt = lds.k + wave * kTileBytes;
    uint8_t* vt = lds.v + wave * kTileBytes;
    const int crow = lane / kChunks, chunk = lane % kChunks;
    const uint32_t lane_byte = (crow & 15) * kRowBytes + 16 * chunk;
    // A page holds 16 keys at least and tiles begin at multiples of 16, so either half of a tile
    // lies in one page: two lookups a tile, the same for all lanes.
    Rows16<kRowBytes> rows(a, __builtin_amdgcn_readfirstlane(t.b), __builtin_amdgcn_readfirstlane(kv), k1);
    int entry[2];                                            // table entries of the next tile
    u32x4_t kw[kLoads], vw[kLoads];
    float sc = 1.0f;
    auto look_up = [&](int i, int* e) {                      // read here, used a tile later
#pragma unroll
        for (int h = 0; h < 2; ++h) e[h] = rows.entry(k0 + i * kKeys + 16 * h);
    };
    auto fetch = [&](int i) {
        uint64_t off[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) off[h] = rows.offset(entry[h], k0 + i * kKeys + 16 * h);
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            const uint64_t from = off[(c * kStepRows) >> 4] + (c * kStepRows & 15) * kRowBytes;
            kw[c] = load16(rows.k, from, lane_byte);
            vw[c] = load16(rows.v, from, lane_byte);
        }
        if constexpr (FP8) {
            const uint64_t at = (lane & 16 ? off[1] : off[0]) / kRowBytes + (lane & 15);
            sc = (lane < 32 ? rows.ks : rows.vs)[at];
        }
    };
    const uint32_t sc_lane = lds_address(scales[wave]) + 16 * quarter;
    const int tiles = (k1 - k0 + kKeys - 1) / kKeys;
    if (wave < tiles) {
        look_up(wave, entry);
        fetch(wave);
        look_up(wave + kNarrowWaves, entry);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        wait_q(s.q[n]);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) s.o[n][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        s.m[n] = kNegInf;
        s.l[n] = 0.0f;
    }
    for (int i = wave; i < tiles; i += kNarrowWaves) {
        const int first = k0 + i * kKeys;
        int later[2];
        look_up(i + 2 * kNarrowWaves, later);                // there by the time these rows are
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            const int row = c * kStepRows + crow;
            stage<D, FP8, false>(kt, row, chunk, kw[c], k1 - first);
            stage<D, FP8, true>(vt, row, chunk, vw[c], k1 - first);
        }
        if constexpr (FP8) scales[wave][lane] = first + (lane & 31) < k1 ? sc : 1.0f;
        if (i + kNarrowWaves < tiles) {
            fetch(i + kNarrowWaves);
            entry[0] = later[0];
            entry[1] = later[1];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // rows staged by other lanes
        step_narrow<D, FP8, N>(s, kt, vt, sc_lane, a.scale_log2, first, first < all_lo || first + kKeys - 1 > all_hi);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // read before the next rows land
    }

    // Join the waves: O of wave w counts 2^(m_w - m).
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float l = s.l[n] + __shfl_xor(s.l[n], 16);
        l += __shfl_xor(l, 32);
        if (lane < 16) {
            lds_m[wave][16 * n + lane] = s.m[n];
            lds_l[wave][16 * n + lane] = l;
        }
        float* own = reinterpret_cast<float*>(n == 0 ? kt : vt);
        // row r's groups of 4 columns are rotated by r, so that the rows do not share banks
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<f32x4_t*>(own + i16 * D + 4 * ((4 * i + quarter + i16) & (D / 4 - 1))) = s.o[n][i];
    }
    __syncthreads();
    constexpr int kGroups = D / 4;                           // a thread joins 4 columns of a row
    uint32_t bad_rows = 0;
    const bool whole = t.span.parts == 1;
    const int rows_here = min(kRows, t.rows - t.row0);
    for (int i = tid; i < rows_here * kGroups; i += kThreads) {
        const int row = i / kGroups, g = i % kGroups;
        float m = kNegInf;
#pragma unroll
        for (int w = 0; w < kNarrowWaves; ++w) m = fmaxf(m, lds_m[w][row]);
        float sum = 0.0f;
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kNarrowWaves; ++w) {
            const float mw = lds_m[w][row];
            const float f = mw == kNegInf ? 0.0f : exp2_fast(mw - m);
            const uint8_t* from = (N == 1 || row < 16 ? lds.k : lds.v) + w * kTileBytes;
            const f32x4_t ow = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(from) + (row & 15) * D +
                                                                4 * ((g + (row & 15)) & (kGroups - 1)));
            sum += f * lds_l[w][row];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += f * ow[j];
        }
        bool bad = !isfinite(sum);
        const Place pr = row_place(a, t, kv, t.row0 + row);
        const float inv = inverse(sum, whole && pr.hi >= 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bad |= !isfinite(v[j]);
            v[j] *= inv;
        }
        if (bad) bad_rows |= 1u << row;
        store4<false>(a, t, part, row, pr.row, D, 4 * g, v);
        if (g == 0 && !whole) store_ml<false>(a, t, part, row, m, sum);
    }
    if (tid == 0) lds.rest.narrow.redo = 0;
    __syncthreads();
    if (rows.missing()) {
        bad_rows = (uint32_t)(((uint64_t)1 << rows_here) - 1);
        if (lane == 0 && a.status) atomicOr(a.status, kStatusPage);
    }
    if (bad_rows) atomicOr(&lds.rest.narrow.redo, bad_rows);
    __syncthreads();
    if (lds.rest.narrow.redo) {
        __threadfence();                                     // the rows' first results have landed
        __syncthreads();
        if (wave == 0) redo_rows<D, FP8, false>(a, t, part, kv, 0, lds.rest.narrow.redo);
    }
}

#define W4_ATTEND_LDS(D)                                                                            \
    __shared__ __attribute__((aligned(16))) uint8_t lds_k[kWideStages * kKeyTile * 2 * (D)];         \
    __shared__ __attribute__((aligned(16))) uint8_t lds_v[kWideStages * kKeyTile * 2 * (D)];         \
    __shared__ __attribute__((aligned(16))) typename Lds<(D)>::Rest lds_rest;                        \
    const Lds<(D)> lds = {lds_k, lds_v, lds_rest}

template <int D, bool FP8, int N>
__global__ __launch_bounds__(kThreads, 2) void attend_narrow_kernel(AttendArgs a) {
    W4_ATTEND_LDS(D);
    attend_narrow<D, FP8, N>(a, blockIdx.x, blockIdx.y, lds);
}

// Both kinds of tiles in one launch: the wide ones first, of them those last in their sequence, which
// see the most keys.
template <int D, bool FP8>
__global__ __launch_bounds__(kThreads, 2) void attend_kernel(AttendArgs a) {
    W4_ATTEND_LDS(D);
    const uint32_t wide = (uint32_t)a.wide_tiles * a.wide_parts, number = blockIdx.y * gridDim.x + blockIdx.x;
    if (number >= wide + (uint32_t)a.narrow_tiles * a.narrow_parts) return;
    const bool first = number < wide;
    const uint32_t index = first ? number : number - wide, tiles = first ? a.wide_tiles : a.narrow_tiles;
    const uint32_t part = __builtin_amdgcn_readfirstlane(index / tiles);   // the division leaves scalar registers
    if (first)
        attend_wide<D, FP8>(a, tiles - 1 - (index - part * tiles), part, lds);
    else
        attend_narrow<D, FP8, kFewRows / 16>(a, index - part * tiles, part, lds);
}

// Joins the parts of the rows that were split: one wave a row, the tiles numbered as in the
// launch that wrote them.  What the parts left is loaded before it is known how many there are (the
// launch allows a.*_parts, at most 64), so that the sequence and the parts cost one wait.
template <int D, int R>
__device__ __forceinline__ void combine_rows(const AttendArgs& a, uint32_t set) {
    constexpr bool WIDE = R == kWideRows;
    constexpr int E = D / 64, kSets = R / 4;
    const int lane = threadIdx.x & 63;
    const int r = (int)(set % kSets) * 4 + (threadIdx.x >> 6);
    const int most = WIDE ? a.wide_parts : a.narrow_parts;
    const int64_t rows = WIDE ? a.wide_rows : a.narrow_rows;
    const int64_t row = (int64_t)(set / kSets) * R + r;
    const float* ml = (WIDE ? a.wide_ml : a.narrow_ml) + 2 * row;
    const float* po = (WIDE ? a.wide_o : a.narrow_o) + row * D + lane * E;
    const int mine = min(lane, most - 1);
    float mp = ml[2 * mine * rows], lp = ml[2 * mine * rows + 1];
    float x[4][E];
    auto load = [&](int p0) {                                // of four parts at once
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) x[j][e] = po[min(p0 + j, most - 1) * rows * D + e];
    };
    load(0);
    int kv;
    const Tile t = find_tile<R>(a, set / kSets, 0, kv);
    if (!t.run || t.span.parts == 1 || t.row0 + r >= t.rows) return;
    const Place place = row_place(a, t, kv, t.row0 + r);
    // lane p weighs part p: 2^(m_p - m) l_p, 0 where the part has nothing of weight
    const int parts = t.span.parts;
    if (lane >= parts) {
        mp = kNegInf;
        lp = 0.0f;
    }
    float m = mp;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    const float f = lp == 0.0f ? 0.0f : exp2_fast(mp - m) * lp;   // NaN where lp or mp is
    float sum = f;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    for (int p0 = 0; p0 < parts; p0 += 4) {
        if (p0 > 0) load(p0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float fp = p0 + j < parts ? __shfl(f, p0 + j) : 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += fp == 0.0f ? 0.0f : fp * x[j][e];
        }
    }
    const float inv = inverse(sum, place.hi >= 0);
    if constexpr (E == 2)
        *reinterpret_cast<uint32_t*>(a.o + (int64_t)place.row * D + 2 * lane) = bf16_pair(o[0] * inv, o[1] * inv);
    else
        a.o[(int64_t)place.row * D + lane] = (uint16_t)bf16_pair(o[0] * inv, o[0] * inv);
}

template <int D>
__global__ __launch_bounds__(256) void combine_kernel(AttendArgs a) {
    const uint32_t narrow = (uint32_t)(a.narrow_rows / 4);
    if (blockIdx.x >= narrow)
        combine_rows<D, kWideRows>(a, blockIdx.x - narrow);
    else if (a.narrow_tile == 16)
        combine_rows<D, 16>(a, blockIdx.x);
    else
        combine_rows<D, kFewRows>(a, blockIdx.x);
}

}  // namespace

static int64_t split_rows(bool wide, const AttendPlan& p) {
    const int64_t tiles = wide ? p.wide_tiles : p.narrow_tiles;
    return (wide ? p.wide_parts : p.narrow_parts) > 1 ? tiles * (wide ? kWideRows : p.narrow_tile) : 0;
}

size_t attend_workspace(int64_t D, const AttendPlan& p) {
    return (size_t)(split_rows(false, p) * p.narrow_parts + split_rows(true, p) * p.wide_parts) * (D + 2) * 4;
}

template <int D, bool FP8>
static hipError_t launch_attend_d(const AttendArgs& a, const AttendPlan& p, hipStream_t s) {
    if (p.both) {
        // a dimension of a grid holds less than 2^32 threads
        const int64_t n = p.wide_tiles * p.wide_parts + p.narrow_tiles * p.narrow_parts, x = imin(n, 1 << 22);
        hipLaunchKernelGGL((attend_kernel<D, FP8>), dim3((unsigned)x, (unsigned)ceil_div(n, x)), dim3(kThreads), 0, s, a);
    } else {
        const dim3 grid((unsigned)p.narrow_tiles, (unsigned)p.narrow_parts), block(kThreads);
        if (p.narrow_tile == 16)
            hipLaunchKernelGGL((attend_narrow_kernel<D, FP8, 1>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((attend_narrow_kernel<D, FP8, kFewRows / 16>), grid, block, 0, s, a);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.wide_rows + a.narrow_rows > 0) {
        hipLaunchKernelGGL(combine_kernel<D>, dim3((unsigned)((a.wide_rows + a.narrow_rows) / 4)), dim3(256), 0, s, a);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_attend(AttendArgs a, int head_dim, bool fp8, const AttendPlan& p, void* workspace, hipStream_t s) {
    a.both = p.both;
    a.narrow_tile = p.narrow_tile;
    a.few_tiles = p.few_tiles;
    a.narrow_tiles = (int)p.narrow_tiles;
    a.wide_tiles = (int)p.wide_tiles;
    a.narrow_parts = p.narrow_parts;
    a.wide_parts = p.wide_parts;
    a.wide_fill = p.wide_fill;
    a.narrow_fill = p.narrow_fill;
    a.narrow_rows = split_rows(false, p);
    a.wide_rows = split_rows(true, p);
    a.narrow_o = static_cast<float*>(workspace);
    a.wide_o = a.narrow_o + a.narrow_rows * p.narrow_parts * head_dim;
    a.narrow_ml = a.wide_o + a.wide_rows * p.wide_parts * head_dim;
    a.wide_ml = a.narrow_ml + a.narrow_rows * p.narrow_parts * 2;
    if (head_dim == 128) return fp8 ? launch_attend_d<128, true>(a, p, s) : launch_attend_d<128, false>(a, p, s);
    return fp8 ? launch_attend_d<64, true>(a, p, s) : launch_attend_d<64, false>(a, p, s);
}

}  // namespace w4
