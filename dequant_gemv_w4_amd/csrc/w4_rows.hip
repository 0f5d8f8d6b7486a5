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
//        g_i t / (1 + t).
// Codes: the row's largest |y| gives the scale, then each y its code, with the functions of the
//        row quantizers: the result is that of w4_rmsnorm / w4_silu_mul to binary32 followed by
//        w4_fp8_quantize_rows / w4_int8_quantize_rows, bit for bit, without the 8 bytes a value
//        that the binary32 row in between would move.
//
// Every kernel is bound by memory: each input is read once and each output written once.  A
// workgroup holds a whole row in registers between the reductions (C chunks of 8 values a
// thread, all loads issued before the first is used).
#include "w4_codes.h"
#include "w4_internal.h"

namespace w4 {
namespace {

constexpr int kMaxWaves = 16;

__device__ __forceinline__ void load8_any(const void* p, bool f32, int64_t i, float* v) {
    if (f32)
        load8<false>(p, i, v);
    else
        load8<true>(p, i, v);
}

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
                                          bool finite, float* red) {
    const int64_t step = (int64_t)blockDim.x * 8;
    const int64_t first = (int64_t)threadIdx.x * 8;
    if (o.kind == RowOut::kF32 || o.kind == RowOut::kBf16) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (first + c * step < K)
                store8(o.y, o.kind == RowOut::kF32, row * K + first + c * step, &y[8 * c]);
        return;
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) amax = fmaxf(amax, fabsf(y[i]));
    amax = block_max(amax, red);
    if (!finite && o.status) atomicOr(o.status, 1u);
    const bool int8 = o.kind == RowOut::kInt8;
    const double s = amax == 0.0f ? 1.0 : (double)amax / (int8 ? 127.0 : kFp8Max);
    if (threadIdx.x == 0) o.scales[row] = (float)s;
    const float rs = (float)(1.0 / s);
    const bool ok = s >= 0x1p-100 && s <= 0x1p100;
    uint8_t* dst = static_cast<uint8_t*>(o.y) + row * K + first;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (first + c * step >= K) continue;
        const uint2 w = int8 ? w8_codes8<true>(&y[8 * c], s, rs, ok) : w8_codes8<false>(&y[8 * c], s, rs, ok);
        *reinterpret_cast<uint2*>(dst + c * step) = w;
    }
}

template <int C>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(RmsnormArgs a, RowOut o) {
    __shared__ double red_d[kMaxWaves];
    __shared__ float red_f[kMaxWaves];
    const int64_t step = (int64_t)blockDim.x * 8;
    const int64_t first = (int64_t)threadIdx.x * 8;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = row * a.K;
        float h[8 * C], w[8 * C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t i = first + c * step;
            if (i < a.K) {
                load8_any(a.x, a.x_f32, base + i, &h[8 * c]);
                load8_any(a.w, a.w_f32, i, &w[8 * c]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) h[8 * c + q] = w[8 * c + q] = 0.0f;
            }
        }
        if (a.r) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t i = first + c * step;
                if (i >= a.K) continue;
                float r[8];
                load8_any(a.r, a.r_f32, base + i, r);
#pragma unroll
                for (int q = 0; q < 8; ++q) r[q] += h[8 * c + q];
                store8(a.r_out, a.r_f32, base + i, r);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t b = bf16_pair(r[2 * q], r[2 * q + 1]);
                    h[8 * c + 2 * q] = a.r_f32 ? r[2 * q] : __uint_as_float(b << 16);
                    h[8 * c + 2 * q + 1] = a.r_f32 ? r[2 * q + 1] : __uint_as_float(b & 0xFFFF0000u);
                }
            }
        }
        double sum[2] = {0.0, 0.0};
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) sum[i & 1] = fma((double)h[i], (double)h[i], sum[i & 1]);
        const double ss = block_sum(sum[0] + sum[1], red_d);
        const float s = (float)(1.0 / sqrt(ss / (double)a.K + (double)a.eps));
        bool finite = true;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) {
            h[i] = h[i] * s * w[i];
            finite &= isfinite(h[i]);
        }
        write_row<C>(o, row, a.K, h, finite, red_f);
        __syncthreads();   // the next row's reductions write red_d and red_f again
    }
}

template <int C>
__global__ __launch_bounds__(1024) void silu_mul_kernel(const void* gu, bool f32, int64_t rows, int64_t F,
                                                        RowOut o) {
    __shared__ float red_f[kMaxWaves];
    const int64_t step = (int64_t)blockDim.x * 8;
    const int64_t first = (int64_t)threadIdx.x * 8;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        float g[8 * C], u[8 * C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t i = first + c * step;
            if (i < F) {
                load8_any(gu, f32, row * 2 * F + i, &g[8 * c]);
                load8_any(gu, f32, row * 2 * F + F + i, &u[8 * c]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) g[8 * c + q] = u[8 * c + q] = 0.0f;
            }
        }
        bool finite = true;
#pragma unroll
        for (int i = 0; i < 8 * C; ++i) {
            const float t = expf(-fabsf(g[i]));              // never overflows
            g[i] = (g[i] < 0.0f ? g[i] * t : g[i]) / (1.0f + t) * u[i];
            finite &= isfinite(g[i]);
        }
        write_row<C>(o, row, F, g, finite, red_f);
        __syncthreads();
    }
}

// Threads and chunks of a row of K values.
struct RowShape {
    int threads;
    int chunks;
};

RowShape row_shape(int64_t rows, int64_t K) {
    (void)rows;
    if (K <= 512) return {64, 1};
    if (K <= 2048) return {256, 1};
    if (K <= 8192) return {256, 4};
    if (K <= 32768) return {1024, 4};
    return {1024, 8};
}

// a launch holds fewer than 2^32 threads: longer inputs are walked in steps of the grid
unsigned row_grid(int64_t rows) { return (unsigned)(rows < (1 << 20) ? rows : (1 << 20)); }

}  // namespace

#define W4_ROW_LAUNCH(KERNEL, ...)                                                             \
    switch (sh.chunks) {                                                                       \
        case 1: hipLaunchKernelGGL(KERNEL<1>, grid, block, 0, s, __VA_ARGS__); break;          \
        case 2: hipLaunchKernelGGL(KERNEL<2>, grid, block, 0, s, __VA_ARGS__); break;          \
        case 4: hipLaunchKernelGGL(KERNEL<4>, grid, block, 0, s, __VA_ARGS__); break;          \
        default: hipLaunchKernelGGL(KERNEL<8>, grid, block, 0, s, __VA_ARGS__); break;         \
    }

hipError_t launch_rmsnorm(const RmsnormArgs& a, const RowOut& o, hipStream_t s) {
    const RowShape sh = row_shape(a.rows, a.K);
    const dim3 grid(row_grid(a.rows)), block((unsigned)sh.threads);
    W4_ROW_LAUNCH(rmsnorm_kernel, a, o)
    return hipGetLastError();
}

hipError_t launch_silu_mul(const void* gu, bool f32, int64_t rows, int64_t F, const RowOut& o,
                           hipStream_t s) {
    const RowShape sh = row_shape(rows, F);
    const dim3 grid(row_grid(rows)), block((unsigned)sh.threads);
    W4_ROW_LAUNCH(silu_mul_kernel, gu, f32, rows, F, o)
    return hipGetLastError();
}

}  // namespace w4
