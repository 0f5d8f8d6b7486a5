// Row operators between the products of a decoder layer: the root-mean-square norm with the
// residual's addition, and the gate silu(g) * u.  Either writes binary32 or bfloat16 rows for the
// 4-bit products, or E4M3 / INT8 codes with one scale per row for the 8-bit products.
//
// Norm:  h = x + r, rounded to the residual's type and stored; y_i = h_i * s * w_i with
//        s = 1 / sqrt(mean_j h_j^2 + eps).  The squares are summed in binary64: a bfloat16 or
//        binary32 square leaves binary32's range at 2^64, and the sum costs nothing here (the
//        binary64 FMA issues at the binary32 rate).  s is rounded to binary32 once, the two
//        products are binary32.  h is normalized as it is stored, so that a later reader of the
//        residual sees the row that was normalized.
// Gate:  y_i = g_i / (1 + exp(-g_i)) * u_i in binary32; with t = exp(-|g_i|) a negative g_i gives
//        g_i t / (1 + t).  Values depend on no others, so value rows are spread over all compute
//        units whatever their number; code rows take a workgroup each.
// Codes: the row's largest |y| gives the scale, then each y its code, with the functions of the
//        row quantizers: the result is that of w4_rmsnorm / w4_silu_mul to binary32 followed by
//        w4_fp8_quantize_rows / w4_int8_quantize_rows, bit for bit, without the 8 bytes a value
//        that the binary32 row in between would move.
//
// Every kernel is bound by memory: each input is read once and each output written once.  A
// workgroup holds a whole row in registers between the reductions (C chunks of 8 values a
// thread, all loads issued before the first is used).  Measured: norm of 4096 x 8192 bfloat16 with
// residual to E4M3 53 us, 4.4 TB/s (a copy of 4 GiB reaches 4.8); gate of 2049 x 11008 bfloat16 to
// INT8 30 us, 3.8 TB/s, of 4096 x 28672 to E4M3 125 us, 4.7 TB/s.  Few rows are bound by latency: norm
// of one row of 8192 3.7 us, of which the launch is about half; gate of 16 x 28672 binary32 to
// bfloat16 2.5 us, to codes (one workgroup a row, for the row's largest value) 11 us.
#include "w4_codes.h"
#include "w4_internal.h"

namespace w4 {
namespace {

constexpr int kMaxWaves = 16;

// 8 values as they are stored: loads of a row are issued together and widened when they are used.
template <bool F32>
struct Raw {
    u32x4_t w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const u32x4_t* s = reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
        w[0] = s[0];
        if constexpr (F32) w[1] = s[1];
    }
    __device__ __forceinline__ float get(int q) const {
        if constexpr (F32) return __uint_as_float(w[q >> 2][q & 3]);
        return __uint_as_float(q & 1 ? w[0][q >> 1] & 0xFFFF0000u : w[0][q >> 1] << 16);
    }
};

// Sum or maximum over the workgroup; every thread gets it, in one order for one row.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    for (int w = 0; w < waves; ++w) t += red[w];
    return t;
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    const int waves = blockDim.x >> 6;
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = red[0];
    for (int w = 1; w < waves; ++w) t = fmaxf(t, red[w]);
    return t;
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef float f2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
    const f2_t f = {a, b};
    const b2_t h = __builtin_convertvector(f, b2_t);   // nearest, halves to even
    return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ void store8(void* p, bool f32, int64_t i, const float* v) {
    if (f32) {
        u32x4_t a, b;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            a[q] = __float_as_uint(v[q]);
            b[q] = __float_as_uint(v[4 + q]);
        }
        u32x4_t* d = reinterpret_cast<u32x4_t*>(static_cast<float*>(p) + i);
        d[0] = a;
        d[1] = b;
    } else {
        u32x4_t a;
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = bf16_pair(v[2 * q], v[2 * q + 1]);
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i) = a;
    }
}

// Writes one row held as C chunks per thread (chunk c of thread t: values (t + c * threads) * 8).
template <int C>
__device__ __forceinline__ void write_row(const RowOut& o, int64_t row, int64_t K, const float* y,
                                          float* red) {
    const int step = blockDim.x * 8, first = threadIdx.x * 8;
    if (o.kind == RowOut::kF32 || o.kind == RowOut::kBf16) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (first + c * step < K)
                store8(o.y, o.kind == RowOut::kF32, row * K + first + c * step, &y[8 * c]);
        return;
    }
    // the largest magnitude, and whether all are finite: x - x is 0 for a finite x only
    float amax = 0.0f, off = 0.0f;
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) {
        amax = fmaxf(amax, fabsf(y[i]));
        off += y[i] - y[i];
    }
    amax = block_max(amax, red);
    if (off != 0.0f && o.status) atomicOr(o.status, kStatusNonfinite);
    const bool int8 = o.kind == RowOut::kInt8;
    const double s = amax == 0.0f ? 1.0 : (double)amax / (int8 ? 127.0 : kFp8Max);
    if (threadIdx.x == 0) o.scales[row] = (float)s;
    const float rs = (float)(1.0 / s);
    // values that are not finite take the quotients, so that their bytes are the row quantizers' too
    const bool ok = s >= 0x1p-100 && s <= 0x1p100 && off == 0.0f;
    uint8_t* dst = static_cast<uint8_t*>(o.y) + row * K + first;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (first + c * step >= K) continue;
        const uint2 w = int8 ? w8_codes8_of<true>(&y[8 * c], s, rs, ok) : w8_codes8_of<false>(&y[8 * c], s, rs, ok);
        *reinterpret_cast<uint2*>(dst + c * step) = w;
    }
}

// One workgroup a row; a dimension of a launch holds fewer than 2^32 threads, so the rows lie in two.
constexpr int64_t kGridRows = 65535;
__device__ __forceinline__ int64_t row_of_block() { return blockIdx.y * kGridRows + blockIdx.x; }
dim3 row_grid(int64_t rows) {
    return dim3((unsigned)(rows < kGridRows ? rows : kGridRows), (unsigned)((rows + kGridRows - 1) / kGridRows));
}

enum Residual { kNone, kBf16Residual, kF32Residual };

template <int C, bool XF32, int R>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(RmsnormArgs a, RowOut o) {
    __shared__ double red_d[kMaxWaves];
    __shared__ float red_f[kMaxWaves];
    const int K = (int)a.K, step = blockDim.x * 8, first = threadIdx.x * 8;
    const int64_t row = row_of_block();
    if (row >= a.rows) return;
    const int64_t base = row * K;
    Raw<XF32> x[C];
    Raw<R == kF32Residual> r[R == kNone ? 1 : C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (first + c * step >= K) continue;
        x[c].load(a.x, base + first + c * step);
        if constexpr (R != kNone) r[c].load(a.r, base + first + c * step);
    }
    float h[8 * C];
    double sum[2] = {0.0, 0.0};
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = first + c * step;
        if (i >= K) {
#pragma unroll
            for (int q = 0; q < 8; ++q) h[8 * c + q] = 0.0f;
            continue;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            h[8 * c + q] = x[c].get(q);
            if constexpr (R != kNone) h[8 * c + q] += r[c].get(q);
        }
        if constexpr (R != kNone) store8(a.r_out, R == kF32Residual, base + i, &h[8 * c]);
        if constexpr (R == kBf16Residual) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t b = bf16_pair(h[8 * c + 2 * q], h[8 * c + 2 * q + 1]);
                h[8 * c + 2 * q] = __uint_as_float(b << 16);
                h[8 * c + 2 * q + 1] = __uint_as_float(b & 0xFFFF0000u);
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
            sum[q & 1] = fma((double)h[8 * c + q], (double)h[8 * c + q], sum[q & 1]);
    }
    const double ss = block_sum(sum[0] + sum[1], red_d);
    const float s = (float)(1.0 / sqrt(ss / (double)K + (double)a.eps));
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = first + c * step;
        if (i >= K) continue;
        if (a.w_f32) {
            Raw<true> w;
            w.load(a.w, i);
#pragma unroll
            for (int q = 0; q < 8; ++q) h[8 * c + q] = h[8 * c + q] * s * w.get(q);
        } else {
            Raw<false> w;
            w.load(a.w, i);
#pragma unroll
            for (int q = 0; q < 8; ++q) h[8 * c + q] = h[8 * c + q] * s * w.get(q);
        }
    }
    write_row<C>(o, row, K, h, red_f);
}

// exp(-|x|) = 2^n 2^f, n the nearest integer to -|x| / ln 2: f is exact to one rounding, 2^f in
// [0.7, 1.42] comes from the exponential unit (1 unit in the last place), so the result is within
// 2.4 half units; 1 / (1 + t) is the reciprocal unit's value improved by one Newton step (1 + t lies
// in [1, 2]).  About 20 instructions a value instead of 40 with the library's exponential and IEEE
// division, which took as long as the row's bytes.
__device__ __forceinline__ float silu_mul(float x, float u) {
    const float a = fminf(fabsf(x), 200.0f);                 // exp(-200) is 0 in binary32
    const float n = rintf(a * -0x1.715476p0f);               // 1 / ln 2
    float f = fmaf(a, -0x1.715476p0f, -n);
    f = fmaf(a, -0x1.4ae0c0p-26f, f);                        // the rest of 1 / ln 2
    const float t = ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    const float d = 1.0f + t;
    const float r = __builtin_amdgcn_rcpf(d);
    const float inv = fmaf(r, fmaf(-d, r, 1.0f), r);
    return (x < 0.0f ? x * t : x) * inv * u;
}

// Value rows: 8 values a thread.
template <bool XF32>
__global__ __launch_bounds__(256) void silu_mul_values_kernel(const void* gu, int64_t rows, int64_t F,
                                                              void* y, bool y_f32) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    const int64_t row = blockIdx.z * kGridRows + blockIdx.y;
    if (i >= F || row >= rows) return;
    Raw<XF32> g, u;
    g.load(gu, row * 2 * F + i);
    u.load(gu, row * 2 * F + F + i);
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = silu_mul(g.get(q), u.get(q));
    store8(y, y_f32, row * F + i, v);
}

template <int C, bool XF32>
__global__ __launch_bounds__(1024) void silu_mul_kernel(const void* gu, int64_t rows, int64_t width, RowOut o) {
    __shared__ float red_f[kMaxWaves];
    const int F = (int)width, step = blockDim.x * 8, first = threadIdx.x * 8;
    const int64_t row = row_of_block();
    if (row >= rows) return;
    const int64_t base = row * 2 * F;
    Raw<XF32> g[C], u[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (first + c * step >= F) continue;
        g[c].load(gu, base + first + c * step);
        u[c].load(gu, base + F + first + c * step);
    }
    float y[8 * C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (first + c * step >= F) {
#pragma unroll
            for (int q = 0; q < 8; ++q) y[8 * c + q] = 0.0f;
            continue;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) y[8 * c + q] = silu_mul(g[c].get(q), u[c].get(q));
    }
    write_row<C>(o, row, F, y, red_f);
}

// Threads and chunks of a row of K values.  Few rows: one chunk a thread, so that a row's latency
// is shortest.  From 512 rows on two, so that several workgroups share a compute unit and one
// loads while another computes: 4096 x 8192 bfloat16 with residual to E4M3 takes 53 us with two
// chunks (512 threads), 57 with four, 63 with one.  `wide` raises that to eight for rows past 16384
// values where the registers allow it (bfloat16 gate rows): 4096 x 28672 to E4M3 takes 125 us
// with 448 threads, of which two workgroups fit, 174 with 896, of which one does; binary32 rows
// spill there (1024 x 28672: 75 us with eight, 65 with four).  Past 32768 values a row needs eight with
// any type, and a binary32 norm with a binary32 residual then spills 89 registers: 1024 x 65536 to E4M3 takes
// 276 us, where a copy of its bytes takes 182.
struct RowShape {
    int threads;
    int chunks;
};

RowShape row_shape(int64_t rows, int64_t K, bool wide) {
    const int64_t n = K / 8;
    int c = rows < 512 ? 1 : wide && K > 16384 ? 8 : 2;
    while (c > 1 && (n + c - 1) / c < 256) c >>= 1;
    while ((n + c - 1) / c > 1024) c <<= 1;
    return {(int)(((n + c - 1) / c + 63) / 64 * 64), c};
}

template <int C, bool XF32>
void launch_norm(const RmsnormArgs& a, const RowOut& o, dim3 grid, dim3 block, hipStream_t s) {
    if (!a.r)
        hipLaunchKernelGGL((rmsnorm_kernel<C, XF32, kNone>), grid, block, 0, s, a, o);
    else if (a.r_f32)
        hipLaunchKernelGGL((rmsnorm_kernel<C, XF32, kF32Residual>), grid, block, 0, s, a, o);
    else
        hipLaunchKernelGGL((rmsnorm_kernel<C, XF32, kBf16Residual>), grid, block, 0, s, a, o);
}

template <int C>
void launch_norm_x(const RmsnormArgs& a, const RowOut& o, dim3 grid, dim3 block, hipStream_t s) {
    if (a.x_f32)
        launch_norm<C, true>(a, o, grid, block, s);
    else
        launch_norm<C, false>(a, o, grid, block, s);
}

template <int C>
void launch_gate_x(const void* gu, bool f32, int64_t rows, int64_t F, const RowOut& o, dim3 grid, dim3 block,
                   hipStream_t s) {
    if (f32)
        hipLaunchKernelGGL((silu_mul_kernel<C, true>), grid, block, 0, s, gu, rows, F, o);
    else
        hipLaunchKernelGGL((silu_mul_kernel<C, false>), grid, block, 0, s, gu, rows, F, o);
}

}  // namespace

hipError_t launch_rmsnorm(const RmsnormArgs& a, const RowOut& o, hipStream_t s) {
    const RowShape sh = row_shape(a.rows, a.K, false);
    const dim3 grid = row_grid(a.rows), block((unsigned)sh.threads);
    switch (sh.chunks) {
        case 1: launch_norm_x<1>(a, o, grid, block, s); break;
        case 2: launch_norm_x<2>(a, o, grid, block, s); break;
        case 4: launch_norm_x<4>(a, o, grid, block, s); break;
        default: launch_norm_x<8>(a, o, grid, block, s); break;
    }
    return hipGetLastError();
}

hipError_t launch_silu_mul(const void* gu, bool f32, int64_t rows, int64_t F, const RowOut& o,
                           hipStream_t s) {
    if (o.kind == RowOut::kF32 || o.kind == RowOut::kBf16) {
        const dim3 r = row_grid(rows), grid((unsigned)((F / 8 + 255) / 256), r.x, r.y), block(256);
        if (f32)
            hipLaunchKernelGGL(silu_mul_values_kernel<true>, grid, block, 0, s, gu, rows, F, o.y, o.kind == RowOut::kF32);
        else
            hipLaunchKernelGGL(silu_mul_values_kernel<false>, grid, block, 0, s, gu, rows, F, o.y, o.kind == RowOut::kF32);
        return hipGetLastError();
    }
    const RowShape sh = row_shape(rows, F, !f32);
    const dim3 grid = row_grid(rows), block((unsigned)sh.threads);
    switch (sh.chunks) {
        case 1: launch_gate_x<1>(gu, f32, rows, F, o, grid, block, s); break;
        case 2: launch_gate_x<2>(gu, f32, rows, F, o, grid, block, s); break;
        case 4: launch_gate_x<4>(gu, f32, rows, F, o, grid, block, s); break;
        default: launch_gate_x<8>(gu, f32, rows, F, o, grid, block, s); break;
    }
    return hipGetLastError();
}

}  // namespace w4
