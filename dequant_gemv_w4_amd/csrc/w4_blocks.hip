// The INT8 cache: rows written as codes with one scale for each block of 16 rows (of a page and kv head),
// and the rows of any cache read back as values.
//
// Write: with m the largest magnitude that a call writes into a block, old the block's scale (0 where its
// first row is written, for the block then begins anew) and S = m / 127 in binary64 if that is larger than old,
// else old:   scale = S, code = round(y / S), and of the block's other rows, where the scale has grown,
// code = round(code / (S / old)).  All quotients are those of binary64 (a new block's codes are the row
// quantizer's for its 16 rows as one).
//
// One wave takes a block of one kv head, K or V: D / 16 lanes a row, so that all 16 rows are in registers, the
// largest value is found by shuffles and a row is either written from its token or, where the scale grows,
// rescaled.  The tokens of a block stand next to each other in the batch, so a workgroup finds the blocks that begin
// within its window of tokens by looking at each token's slot and the one before; the query heads of a token are
// other workgroups of the same launch.  Bound by memory where tokens are many: two prompts of up to 2048 tokens of 32 +
// 64 heads in bfloat16 (132 MB) take 32 us without rotation, 4.2 TB/s (a 4 GiB copy: 4.7), 37 with; by one chain
// of loads where they are few: 64 tokens of 64 + 16 heads in binary32 5.7 us.
#include "w4_codes.h"
#include "w4_internal.h"
#include "w4_paging.h"

namespace w4 {
namespace {

constexpr int kBlockRows = 16;
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxPairs = 64;   // head_dim 128
constexpr float kLeastMax = 0x1p-93f;                        // a block below it counts as zeros
constexpr float kLeastScale = (float)(0x1p-93 / 127.0);      // of those that a write leaves; values below kLeastMax pass 127 of a smaller one

__device__ __forceinline__ uint32_t bf16_pair2(float a, float b) {
    typedef float f2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
    const f2_t f = {a, b};
    const b2_t h = __builtin_convertvector(f, b2_t);
    return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ u32x4_t bf16_of8(const float* v) {
    u32x4_t a;
#pragma unroll
    for (int q = 0; q < 4; ++q) a[q] = bf16_pair2(v[2 * q], v[2 * q + 1]);
    return a;
}

// What codes are divided by: S, and 1 / S correctly rounded to binary64 and binary32.
struct Step {
    double s, r;
    float r32;
    __device__ explicit Step(double by) : s(by), r(1.0 / by), r32((float)r) {}
};

// round(v / S) of 8 values as bytes, |v / S| <= 128.  fma(v, r32, 1.5 * 2^23) has the nearest whole number in its
// low bits and what it leaves tells how near a half is; v * r32 is within 128 * 2^-23 of v / S, so only nearer than
// 2^-15 the binary64 quotient has to decide.  That quotient in three operations: with r the rounded reciprocal and
// q = v r, q + (v - q S) r rounds to the correctly rounded v / S (Markstein).
__device__ __forceinline__ uint2 int8_codes8(const float* v, const Step& by) {
    uint32_t w[2];
    float far = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float x = v[4 * h + q], i = fmaf(x, by.r32, 0x1.8p23f);
            b[q] = __float_as_uint(i);
            far = fmaxf(far, fabsf(fmaf(x, by.r32, 0x1.8p23f - i)));
        }
        w[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
    }
    if (far >= 0.5f - 0x1p-15f) {
        w[0] = w[1] = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const double x = v[q], t = x * by.r;
            w[q >> 2] |= (uint32_t)(uint8_t)(int8_t)(int)rint(fma(fma(-t, by.s, x), by.r, t)) << (8 * (q & 3));
        }
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void values_of8(uint2 c, float* v) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = (float)(int8_t)(c.x >> (8 * q));
        v[4 + q] = (float)(int8_t)(c.y >> (8 * q));
    }
}

// The 16 elements of a head that a lane holds: pairs of a rotation are within it.
struct Chunks {
    int c0, c1;   // two runs of 8
    bool turns;
};
__device__ __forceinline__ Chunks chunks_of(const RopeArgs& a, int u) {
    Chunks c;
    c.turns = u < (a.rotary >> 4);
    const bool split = c.turns && !a.interleaved;
    c.c0 = split ? 8 * u : 16 * u;
    c.c1 = split ? 8 * u + (a.rotary >> 1) : 16 * u + 8;
    return c;
}

__device__ __forceinline__ void turn(const RopeArgs& a, const float* cs, const float* sn, int u, float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float c = cs[8 * u + j], s = sn[8 * u + j];
        if (a.interleaved) {
            const float x0 = v[2 * j], x1 = v[2 * j + 1];
            v[2 * j] = x0 * c - x1 * s;
            v[2 * j + 1] = x0 * s + x1 * c;
        } else {
            const float x0 = v[j], x1 = v[8 + j];
            v[j] = x0 * c - x1 * s;
            v[8 + j] = x0 * s + x1 * c;
        }
    }
}

// Cosines and sines of the pairs of n tokens from t on.
__device__ __forceinline__ void angles(const RopeArgs& a, int64_t t, int n, float (*cs)[kMaxPairs], float (*sn)[kMaxPairs]) {
    const int pair = threadIdx.x & (kMaxPairs - 1);
    if (pair >= a.rotary >> 1) return;
    for (int i = threadIdx.x / kMaxPairs; i < n; i += kThreads / kMaxPairs) {
        const double turns = (double)a.positions[t + i] * a.freqs[pair] * 0.15915494309189533577;
        const float part = (float)(turns - rint(turns));     // [-1/2, 1/2]
        float s, c;
        sincospif(2.0f * part, &s, &c);
        cs[i][pair] = c * a.amplitude;
        sn[i][pair] = s * a.amplitude;
    }
}

// Query heads of token t.
template <bool XF32>
__device__ __forceinline__ void write_q(const RopeArgs& a, int64_t t, int part, float (*cs)[kMaxPairs], float (*sn)[kMaxPairs]) {
    const int lanes = a.head_dim >> 4;
    const int item = part * kThreads + threadIdx.x, head = item / lanes, u = item & (lanes - 1);
    const int64_t slot = a.slots[t];
    const Chunks c = chunks_of(a, u);
    float v[16];
    const bool active = head < a.heads;
    if (active) {
        const int64_t from = (t * (a.heads + 2 * a.kv_heads) + head) * a.head_dim;
        load8<!XF32>(a.qkv, from + c.c0, v);
        load8<!XF32>(a.qkv, from + c.c1, v + 8);
    }
    angles(a, t, 1, cs, sn);
    __syncthreads();
    if (slot < 0 || slot >= a.pages << a.page_shift || !active) return;
    if (c.turns) turn(a, cs[0], sn[0], u, v);
    uint16_t* q = a.q + (t * a.heads + head) * a.head_dim;
    *reinterpret_cast<u32x4_t*>(q + c.c0) = bf16_of8(v);
    *reinterpret_cast<u32x4_t*>(q + c.c1) = bf16_of8(v + 8);
}

// The block that begins with token t, in slot `slot`: heads of K and V, wave by wave.
template <bool XF32, int D>
__device__ __forceinline__ void write_block(const RopeArgs& a, int64_t t, int64_t slot, int part, int parts,
                                            float (*cs)[kMaxPairs], float (*sn)[kMaxPairs]) {
    constexpr int kLanes = D / 16, kGroups = 64 / kLanes, kRows = kBlockRows / kGroups;   // rows of a lane
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t block = slot >> 4;
    if (slot >= a.pages << a.page_shift) {
        if (part == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, kStatusPage);
        return;
    }
    // the tokens that follow in the same block, and their rows
    const int64_t near = t + (lane & 15);
    const int64_t theirs = near < a.T ? a.slots[near] : -1;
    const uint64_t others = ~__ballot(theirs >> 4 == block) & 0xFFFF;
    const int n = others ? __builtin_ctzll(others) : kBlockRows;
    const int row_of = (int)theirs & 15;
    const bool anew = __any(lane < n && row_of == 0);
    const int group = lane / kLanes, u = lane % kLanes;
    int token[kRows];                                        // of my rows; -1: not written
#pragma unroll
    for (int i = 0; i < kRows; ++i) token[i] = -1;
    for (int j = 0; j < n; ++j) {
        const int r = __builtin_amdgcn_readlane(row_of, j);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (r == i * kGroups + group) token[i] = j;
    }
    if (a.rotary > 0) {
        __syncthreads();                                     // those of the block before are read
        angles(a, t, n, cs, sn);
        __syncthreads();
    }
    const Chunks ck = chunks_of(a, u);
    const int page_rows = 1 << a.page_shift;
    for (int item = part * kWaves + wave; item < 2 * a.kv_heads; item += parts * kWaves) {
        const bool is_v = item >= a.kv_heads;
        const int kvh = item - (is_v ? a.kv_heads : 0);
        const Chunks c = is_v ? Chunks{16 * u, 16 * u + 8, false} : ck;
        const int64_t row0 = (((slot >> a.page_shift) * a.kv_heads + kvh) << a.page_shift) + (slot & (page_rows - 1) & ~15);
        float* scale = (is_v ? a.v_scales : a.k_scales) + (row0 >> 4);
        uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v : a.k) + row0 * D;
        float v[kRows][16];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (token[i] >= 0) {
                const int64_t from = ((t + token[i]) * (a.heads + 2 * a.kv_heads) + a.heads + item) * D;
                load8<!XF32>(a.qkv, from + c.c0, v[i]);
                load8<!XF32>(a.qkv, from + c.c1, v[i] + 8);
            }
        }
        float old = anew ? 0.0f : *scale;
        old = old >= kLeastScale && old < __builtin_huge_valf() ? old : 0.0f;
        float most = 0.0f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (token[i] < 0) continue;
            if (c.turns) turn(a, cs[token[i]], sn[token[i]], u, v[i]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (!(fabsf(v[i][j]) < __builtin_huge_valf())) {
                    bad = true;
                    v[i][j] = 0.0f;
                }
                most = fmaxf(most, fabsf(v[i][j]));
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor(most, off));
        const double need = most < kLeastMax ? 0.0 : (double)most / 127.0;
        const bool more = (float)need > old;
        const Step S(more ? need : old > 0.0f ? (double)old : 1.0);
        if (__any(bad) && lane == 0 && a.status) atomicOr(a.status, kStatusNonfinite);
        if (lane == 0) *scale = more ? (float)need : old;
        const bool grown = more && !anew;                    // the same for the wave
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            uint8_t* row = codes + (i * kGroups + group) * D;
            if (token[i] >= 0) {
                *reinterpret_cast<uint2*>(row + c.c0) = int8_codes8(v[i], S);
                *reinterpret_cast<uint2*>(row + c.c1) = int8_codes8(v[i] + 8, S);
            } else if (grown) {
                const u32x4_t w = *reinterpret_cast<const u32x4_t*>(row + 16 * u);
                float x[16];
                values_of8(make_uint2(w[0], w[1]), x);
                values_of8(make_uint2(w[2], w[3]), x + 8);
                const Step by(old > 0.0f ? S.s / old : 0x1p60);   // a scale of 0: all codes become 0
                const uint2 lo = int8_codes8(x, by), hi = int8_codes8(x + 8, by);
                *reinterpret_cast<u32x4_t*>(row + 16 * u) = u32x4_t{lo.x, lo.y, hi.x, hi.y};
            }
        }
    }
}

// Workgroups of blocks first: of the `window` tokens from window * w on, those that begin one, one after the other.
struct WriteGrid {
    int window, q_parts, kv_parts;
    uint32_t blocks, all;   // workgroups of blocks; of all
};
template <bool XF32, int D>
__global__ __launch_bounds__(kThreads) void write_blocks_kernel(RopeArgs a, WriteGrid g) {
    __shared__ float cs[kBlockRows][kMaxPairs], sn[kBlockRows][kMaxPairs];
    const uint32_t number = blockIdx.y * gridDim.x + blockIdx.x;
    if (number >= g.all) return;
    if (number >= g.blocks) {
        const uint32_t q = number - g.blocks, t = q / (uint32_t)g.q_parts;
        write_q<XF32>(a, t, (int)(q - t * g.q_parts), cs, sn);
        return;
    }
    const uint32_t w = number / (uint32_t)g.kv_parts;
    const int part = (int)(number - w * g.kv_parts), lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)w * g.window, t = t0 + lane;
    const int64_t slot = lane < g.window && t < a.T ? a.slots[t] : -1;
    const int64_t before = slot >= 0 && t > 0 ? a.slots[t - 1] : -1;
    uint64_t begin = __ballot(slot >= 0 && slot >> 4 != before >> 4);
    while (begin) {
        const int i = __builtin_ctzll(begin);
        begin &= begin - 1;
        write_block<XF32, D>(a, t0 + i, __shfl(slot, i), part, g.kv_parts, cs, sn);
    }
}

// --------------------------------------------------------------------------
// Rows read back
// --------------------------------------------------------------------------
//
// Bound by memory, if the address of an element costs few instructions: a thread keeps to one place of a token's row, 16
// bytes of it in the output, and goes through tokens, four of them on their way.  Where a wave's 64 places are of one
// token (WHOLE) what depends on the slot is formed once for all in scalar registers.  65,536 tokens of 8 INT8 heads of
// 128 take 77 us as bfloat16 rows (403 MB, 5.2 TB/s); with a place found again for each 8 elements 101.  The stores are
// non-temporal: 87 us otherwise.

constexpr int kReadTokens = 4;

template <int TYPE, bool F32, bool WHOLE>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(ReadArgs a, int places_shift) {
    constexpr int E = F32 ? 4 : 8;                           // elements of a place
    typedef uint32_t raw_t __attribute__((ext_vector_type(TYPE == 0 ? E / 2 : E / 4 < 2 ? 2 : E / 4)));
    const int places = 2 * a.kv_heads * a.head_dim / E;      // of a token, here at most 1 << places_shift of them
    const int place = ((int)blockIdx.y << places_shift) + ((int)threadIdx.x & ((1 << places_shift) - 1));
    const int beside = kThreads >> places_shift;             // tokens at once
    const int head_shift = (a.head_dim == 128 ? 7 : 6) - (F32 ? 2 : 3);   // places of a head
    const bool is_v = (place >> head_shift) >= a.kv_heads, real = place < places;
    const int kvh = (place >> head_shift) - (is_v ? a.kv_heads : 0), at = E * (place & ((1 << head_shift) - 1));
    const int64_t head_row = (int64_t)kvh << a.page_shift;
    const uint8_t* from = static_cast<const uint8_t*>(is_v ? a.v : a.k) + (head_row * a.head_dim + at) * (TYPE == 0 ? 2 : 1);
    const float* scales = (is_v ? a.v_scales : a.k_scales) + (TYPE == 2 ? head_row >> 4 : head_row);
    const uint32_t page_rows = (uint32_t)a.kv_heads << a.page_shift;   // at most 2^22
    const int64_t t0 = (int64_t)blockIdx.x * (beside * kReadTokens), end = a.pages << a.page_shift;
    raw_t w[kReadTokens];
    float s[kReadTokens];
    int64_t slot[kReadTokens], t[kReadTokens];
#pragma unroll
    for (int q = 0; q < kReadTokens; ++q) {
        const int first = (int)(threadIdx.x >> places_shift) + q * beside;
        t[q] = t0 + (WHOLE ? __builtin_amdgcn_readfirstlane(first) : first);
        const int64_t known = t[q] < a.n ? t[q] : a.n - 1;
        if constexpr (WHOLE)                                 // through the scalar cache
            slot[q] = ((__attribute__((address_space(4))) const int64_t*)(uintptr_t)a.slots)[known];
        else
            slot[q] = a.slots[known];
        if (t[q] >= a.n) slot[q] = -1;
    }
#pragma unroll
    for (int q = 0; q < kReadTokens; ++q) {
        // rows that are left out (negative, or past the cache) read the cache's first one
        const int64_t here = slot[q] >= 0 && slot[q] < end ? slot[q] : 0;
        const uint64_t row = (uint64_t)(uint32_t)(here >> a.page_shift) * page_rows + (uint32_t)(here & ((1 << a.page_shift) - 1));
        if (!real) continue;
        const uint8_t* p = from + row * (a.head_dim * (TYPE == 0 ? 2 : 1));
        if constexpr (TYPE != 0 && F32)
            w[q][0] = *reinterpret_cast<const uint32_t*>(p);
        else
            w[q] = *reinterpret_cast<const raw_t*>(p);
        if constexpr (TYPE != 0) s[q] = scales[TYPE == 2 ? row >> 4 : row];
    }
#pragma unroll
    for (int q = 0; q < kReadTokens; ++q) {
        if (slot[q] >= end && place == 0 && a.status) atomicOr(a.status, kStatusPage);
        if (slot[q] < 0 || slot[q] >= end || !real) continue;
        u32x4_t* to = static_cast<u32x4_t*>(a.out) + (t[q] * places + place);
        if constexpr (TYPE == 0 && !F32) {
            __builtin_nontemporal_store(w[q], to);
            continue;
        }
        float v[E];
        if constexpr (TYPE == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __uint_as_float(e % 2 ? w[q][e / 2] & 0xFFFF0000u : w[q][e / 2] << 16);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint32_t c = w[q][e / 4] >> (8 * (e % 4));
                v[e] = s[q] * (TYPE == 2 ? (float)(int8_t)c : __builtin_amdgcn_cvt_f32_fp8(c, 0));
            }
        }
        if constexpr (F32)
            __builtin_nontemporal_store(u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, to);
        else
            __builtin_nontemporal_store(bf16_of8(v), to);
    }
}

}  // namespace

hipError_t launch_write_blocks(const RopeArgs& a, bool x_f32, hipStream_t s) {
    WriteGrid g;
    // Blocks that begin within a window are written one after the other (2.6 us each), and a workgroup whose window has
    // none ends at once, at the cost of its launch.  us with windows of 1, 4 and 16 (32 heads, 8 kv heads of 128): 64
    // single tokens 5.1, 12, 46, 256 6.6, 12, 40, 1024 19, 17, 39, 4096 72, 60, 57; a prompt of 256 9.5, 7.2, 11, 1000
    // 19, 11, 12, 2048 36, 21, 14, 8192 137, 74, 37 (32 kv heads 224, 166, 95).
    g.window = a.T <= 256 ? 1 : a.T <= 1024 ? 4 : kBlockRows;
    g.q_parts = (int)ceil_div((int64_t)a.heads * (a.head_dim / 16), kThreads);
    g.kv_parts = (int)ceil_div(2 * a.kv_heads, kWaves);
    g.blocks = (uint32_t)(ceil_div(a.T, g.window) * g.kv_parts);
    g.all = g.blocks + (uint32_t)(a.T * g.q_parts);
    const int64_t x = imin(g.all, 1 << 20);                  // a dimension of a grid holds less than 2^32 threads
    const dim3 grid((unsigned)x, (unsigned)ceil_div(g.all, x)), block(kThreads);
    if (a.head_dim == 128) {
        if (x_f32)
            hipLaunchKernelGGL((write_blocks_kernel<true, 128>), grid, block, 0, s, a, g);
        else
            hipLaunchKernelGGL((write_blocks_kernel<false, 128>), grid, block, 0, s, a, g);
    } else {
        if (x_f32)
            hipLaunchKernelGGL((write_blocks_kernel<true, 64>), grid, block, 0, s, a, g);
        else
            hipLaunchKernelGGL((write_blocks_kernel<false, 64>), grid, block, 0, s, a, g);
    }
    return hipGetLastError();
}

template <int TYPE, bool F32>
static hipError_t launch_read_type(const ReadArgs& a, hipStream_t s) {
    const int places = 2 * a.kv_heads * a.head_dim / (F32 ? 4 : 8);   // 16 at least
    int shift = 4;
    while ((1 << shift) < places && (1 << shift) < kThreads) ++shift;
    const int64_t tokens = (kThreads >> shift) * kReadTokens;
    const dim3 grid((unsigned)ceil_div(a.n, tokens), (unsigned)ceil_div(places, 1 << shift)), block(kThreads);
    if (shift >= 6)
        hipLaunchKernelGGL((cache_read_kernel<TYPE, F32, true>), grid, block, 0, s, a, shift);
    else
        hipLaunchKernelGGL((cache_read_kernel<TYPE, F32, false>), grid, block, 0, s, a, shift);
    return hipGetLastError();
}

hipError_t launch_cache_read(const ReadArgs& a, int type, bool out_f32, hipStream_t s) {
    if (type == 0) return out_f32 ? launch_read_type<0, true>(a, s) : launch_read_type<0, false>(a, s);
    if (type == 1) return out_f32 ? launch_read_type<1, true>(a, s) : launch_read_type<1, false>(a, s);
    return out_f32 ? launch_read_type<2, true>(a, s) : launch_read_type<2, false>(a, s);
}

}  // namespace w4
