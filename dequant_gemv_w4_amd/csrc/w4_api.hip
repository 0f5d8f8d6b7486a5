// C-ABI entry points of libw4a16: argument validation, device check, launch.
// The kernels live in w4_quantize.hip, w4_gemv.hip, w4_gemv_mfma.hip, w4_gemm.hip, w4_w8a8.hip,
// w4_rows.hip, w4_cache.hip and w4_attention.hip.
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "w4a16.h"
#include "w4_internal.h"
#include "w4_paging.h"

namespace {

thread_local std::string g_last_hip_error;

constexpr int kMaxDevices = 64;
std::atomic<int> g_arch_state[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

w4_status hip_fail(hipError_t e) {
    g_last_hip_error = hipGetErrorString(e);
    return W4_ERR_HIP;
}

w4_status check_arch() {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return W4_ERR_ARCH;
    int st = g_arch_state[dev].load(std::memory_order_acquire);
    if (st == 0) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess) return hip_fail(e);
        st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
        g_arch_state[dev].store(st, std::memory_order_release);
    }
    return st == 1 ? W4_OK : W4_ERR_ARCH;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

w4_status check_nk(int64_t n, int64_t k) {
    if (n < 1 || k < W4_GROUP || k % W4_GROUP != 0) return W4_ERR_SHAPE;
    if (n > (int64_t)0x7FFFFFFF || k > (int64_t)0x7FFFFFFF) return W4_ERR_SHAPE;
    return W4_OK;
}

w4_status to_fmt(const w4_format* in, w4::Fmt* out) {
    if (!in) return W4_ERR_NULL;
    if ((in->group != 32 && in->group != 64 && in->group != 128) ||
        (in->scale_bf16 != 0 && in->scale_bf16 != 1) ||
        (in->zero_bits != 4 && in->zero_bits != 8) || (in->symmetric != 0 && in->symmetric != 1))
        return W4_ERR_UNSUPPORTED;
    out->group = in->group;
    out->scale_bf16 = in->scale_bf16 == 1;
    out->zero4 = in->zero_bits == 4;
    out->symmetric = in->symmetric == 1;
    return W4_OK;
}

bool is_dtype(w4_dtype t) { return t == W4_F32 || t == W4_BF16; }

w4_status check_rows(int64_t rows, int64_t k) {
    if (rows < 1 || rows > (int64_t)INT32_MAX || k < W4_GROUP || k % W4_GROUP != 0 ||
        k > W4_ROWS_MAX_K)
        return W4_ERR_SHAPE;
    return W4_OK;
}

// Geometry of a paged cache (the pointers apart); *shift is log2(page_size).
w4_status check_page_size(int32_t page_size, int* shift) {
    if (page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)) != 0)
        return W4_ERR_UNSUPPORTED;
    *shift = __builtin_ctz((unsigned)page_size);
    return W4_OK;
}

w4_status check_cache(const w4_kv_cache* c, int* shift) {
    if (!c) return W4_ERR_NULL;
    if (c->type != W4_CACHE_BF16 && c->type != W4_CACHE_FP8 && c->type != W4_CACHE_INT8) return W4_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return W4_ERR_UNSUPPORTED;
    const w4_status st = check_page_size(c->page_size, shift);
    if (st != W4_OK) return st;
    if (c->kv_heads < 1 || c->kv_heads > 1024 || c->pages < 1 || c->pages > (int64_t)INT32_MAX ||
        c->pages * c->page_size >= ((int64_t)1 << 40) / c->kv_heads)
        return W4_ERR_SHAPE;
    return W4_OK;
}

w4_status check_cache_pointers(const w4_kv_cache* c) {
    if (!c->k || !c->v) return W4_ERR_NULL;
    if (c->type != W4_CACHE_BF16 && (!c->k_scales || !c->v_scales)) return W4_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 4) ||
        !aligned(c->v_scales, 4))
        return W4_ERR_ALIGN;
    return W4_OK;
}

w4_status check_heads(int64_t T, int64_t heads, const w4_kv_cache* c) {
    if (T < 1 || T > W4_MAX_TOKENS || heads < c->kv_heads || heads % c->kv_heads != 0 ||
        heads > 65536 || heads >= ((int64_t)1 << 26) / T)
        return W4_ERR_SHAPE;
    return W4_OK;
}

// The kernels' number of a cache type.
int cache_kind(const w4_kv_cache* c) { return c->type == W4_CACHE_INT8 ? 2 : c->type == W4_CACHE_FP8 ? 1 : 0; }

w4_status check_batch(int64_t B, int64_t max_pages, int64_t page_size) {
    if (B < 1 || B > W4_MAX_SEQUENCES || max_pages < 1 || max_pages > W4_MAX_CONTEXT / page_size)
        return W4_ERR_SHAPE;
    return W4_OK;
}

w4_status check_rope(const w4_rope* r) {
    if (!r) return W4_ERR_NULL;
    if (r->scaling < W4_ROPE_NONE || r->scaling > W4_ROPE_RAMP || r->reserved != 0 ||
        (r->interleaved != 0 && r->interleaved != 1) || r->rotary_dim < 16 ||
        r->rotary_dim % 16 != 0 || r->rotary_dim > 128)
        return W4_ERR_UNSUPPORTED;
    if (!(r->base > 1.0) || !std::isfinite(r->base)) return W4_ERR_VALUE;
    if (r->scaling == W4_ROPE_NONE) return W4_OK;
    if (!(r->factor >= 1.0) || !std::isfinite(r->factor)) return W4_ERR_VALUE;
    if (r->scaling == W4_ROPE_LINEAR) return W4_OK;
    if (!(r->low > 0.0) || !(r->high > r->low) || !std::isfinite(r->high) ||
        r->original_positions < 1)
        return W4_ERR_VALUE;
    return W4_OK;
}

double rope_amplitude(const w4_rope* r) {
    return r->scaling == W4_ROPE_RAMP ? 1.0 + 0.1 * std::log(r->factor) : 1.0;
}

}  // namespace

// Workspace of w4_gemm_noalloc.  In host code this name is only a stand-in for the
// symbol: its device address (one per GPU) comes from hipGetSymbolAddress and is the
// only form passed to kernels.
static __device__ __align__(256) uint8_t scratch[W4_GEMM_NOALLOC_MAX_WORKSPACE];

namespace {

std::atomic<void*> g_scratch_addr[kMaxDevices];
std::mutex g_scratch_mu;

// Device address of the current device's scratch, looked up once per device.
w4_status scratch_address(void** out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return W4_ERR_ARCH;
    void* p = g_scratch_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        p = g_scratch_addr[dev].load(std::memory_order_relaxed);
        if (!p) {
            e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            if (e != hipSuccess) return hip_fail(e);
            if (!p) return W4_ERR_WORKSPACE;
            g_scratch_addr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return W4_OK;
}

}  // namespace

extern "C" {

const char* w4_status_string(w4_status s) {
    switch (s) {
        case W4_OK: return "ok";
        case W4_ERR_NULL: return "null pointer";
        case W4_ERR_SHAPE: return "unsupported shape";
        case W4_ERR_ALIGN: return "misaligned pointer";
        case W4_ERR_DTYPE: return "unsupported dtype";
        case W4_ERR_UNSUPPORTED: return "unsupported format";
        case W4_ERR_ARCH: return "device is not gfx950";
        case W4_ERR_WORKSPACE: return "workspace missing or too small";
        case W4_ERR_HIP: return "HIP runtime error";
        case W4_ERR_BUFFER: return "destination buffer too small";
        case W4_ERR_VALUE: return "argument value out of range";
    }
    return "unknown status";
}

const char* w4_last_hip_error(void) { return g_last_hip_error.c_str(); }

int w4_format_version(void) { return W4_FORMAT_VERSION; }

static w4_status quantize_common(const void* W, w4_dtype wt, int64_t N, int64_t K,
                                 uint8_t* packed, uint16_t* scales_f16, uint8_t* zeros,
                                 uint32_t* d_status, bool symmetric, hipStream_t stream) {
    if (!W || !packed || !scales_f16 || !zeros) return W4_ERR_NULL;
    if (wt != W4_F32 && wt != W4_BF16) return W4_ERR_DTYPE;
    w4_status st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(scales_f16, 2) ||
        (d_status && !aligned(d_status, 4)))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    w4::Fmt f;
    f.symmetric = symmetric;
    hipError_t e = w4::launch_quantize(W, wt == W4_BF16, f, N * (K / W4_GROUP), packed,
                                       scales_f16, zeros, d_status, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_quantize(const void* W, w4_dtype wt, int64_t N, int64_t K, uint8_t* packed,
                      uint16_t* scales_f16, uint8_t* zeros, uint32_t* d_status,
                      hipStream_t stream) {
    return quantize_common(W, wt, N, K, packed, scales_f16, zeros, d_status, false, stream);
}

w4_status w4_quantize_symmetric(const void* W, w4_dtype wt, int64_t N, int64_t K,
                                uint8_t* packed, uint16_t* scales_f16, uint8_t* zeros,
                                uint32_t* d_status, hipStream_t stream) {
    return quantize_common(W, wt, N, K, packed, scales_f16, zeros, d_status, true, stream);
}

size_t w4_prepared_bytes(int64_t N, int64_t K) {
    if (check_nk(N, K) != W4_OK) return 0;
    return (size_t)w4::prepared_total(N, K);
}

w4_status w4_prepare(const uint8_t* packed, const uint16_t* scales_f16, const uint8_t* zeros,
                     int64_t N, int64_t K, void* prepared, size_t prepared_bytes,
                     hipStream_t stream) {
    if (!packed || !scales_f16 || !zeros || !prepared) return W4_ERR_NULL;
    w4_status st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (!aligned(packed, 16) || !aligned(scales_f16, 2) || !aligned(prepared, 256))
        return W4_ERR_ALIGN;
    if (prepared_bytes < w4_prepared_bytes(N, K)) return W4_ERR_BUFFER;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_prepare(packed, scales_f16, zeros, N, K, w4::Fmt{},
                                      static_cast<uint8_t*>(prepared), stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_unprepare(const void* prepared, int64_t N, int64_t K, uint8_t* packed,
                       uint16_t* scales_f16, uint8_t* zeros, hipStream_t stream) {
    if (!packed || !scales_f16 || !zeros || !prepared) return W4_ERR_NULL;
    w4_status st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (!aligned(packed, 16) || !aligned(scales_f16, 2) || !aligned(prepared, 256))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_unprepare(static_cast<const uint8_t*>(prepared), N, K, w4::Fmt{}, packed,
                                        scales_f16, zeros, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_gemv(const void* prepared, int64_t N, int64_t K, const void* x, w4_dtype xt,
                  int64_t M, void* y, w4_dtype yt, hipStream_t stream) {
    if (!prepared || !x || !y) return W4_ERR_NULL;
    if ((xt != W4_F32 && xt != W4_BF16) || (yt != W4_F32 && yt != W4_BF16)) return W4_ERR_DTYPE;
    w4_status st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (K > W4_GEMV_MAX_K || M < 1 || M > W4_GEMV_MAX_M) return W4_ERR_SHAPE;
    if (!aligned(prepared, 256) || !aligned(x, 16) || !aligned(y, yt == W4_F32 ? 4 : 2))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_gemv(static_cast<const uint8_t*>(prepared), N, K, x, xt == W4_F32,
                                   M, y, yt == W4_BF16, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

size_t w4_zeros_bytes(int64_t N, int64_t K, const w4_format* fmt) {
    w4::Fmt f;
    if (to_fmt(fmt, &f) != W4_OK || check_nk(N, K) != W4_OK) return 0;
    const int64_t groups = N * (K / f.group);
    return (size_t)(f.zero4 ? (groups + 1) / 2 : groups);
}

w4_status w4_quantize_fmt(const void* W, w4_dtype wt, int64_t N, int64_t K,
                          const w4_format* fmt, uint8_t* packed, uint16_t* scales,
                          uint8_t* zeros, uint32_t* d_status, hipStream_t stream) {
    if (!W || !packed || !scales || !zeros || !fmt) return W4_ERR_NULL;
    w4::Fmt f;
    w4_status st = to_fmt(fmt, &f);
    if (st != W4_OK) return st;
    if (wt != W4_F32 && wt != W4_BF16) return W4_ERR_DTYPE;
    st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(scales, 2) ||
        (d_status && !aligned(d_status, 4)))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_quantize(W, wt == W4_BF16, f, N * (K / f.group), packed, scales,
                                       zeros, d_status, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

size_t w4_prepared_bytes_fmt(int64_t N, int64_t K, const w4_format* fmt) {
    w4::Fmt f;
    if (to_fmt(fmt, &f) != W4_OK || check_nk(N, K) != W4_OK) return 0;
    return (size_t)w4::prepared_total_g(N, K, f.group);
}

w4_status w4_prepare_fmt(const uint8_t* packed, const uint16_t* scales, const uint8_t* zeros,
                         int64_t N, int64_t K, const w4_format* fmt, void* prepared,
                         size_t prepared_bytes, hipStream_t stream) {
    if (!packed || !scales || !zeros || !prepared || !fmt) return W4_ERR_NULL;
    w4::Fmt f;
    w4_status st = to_fmt(fmt, &f);
    if (st != W4_OK) return st;
    st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (!aligned(packed, 16) || !aligned(scales, 2) || !aligned(prepared, 256))
        return W4_ERR_ALIGN;
    if (prepared_bytes < w4_prepared_bytes_fmt(N, K, fmt)) return W4_ERR_BUFFER;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_prepare(packed, scales, zeros, N, K, f,
                                      static_cast<uint8_t*>(prepared), stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_unprepare_fmt(const void* prepared, int64_t N, int64_t K, const w4_format* fmt,
                           uint8_t* packed, uint16_t* scales, uint8_t* zeros,
                           hipStream_t stream) {
    if (!packed || !scales || !zeros || !prepared || !fmt) return W4_ERR_NULL;
    w4::Fmt f;
    w4_status st = to_fmt(fmt, &f);
    if (st != W4_OK) return st;
    st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (!aligned(packed, 16) || !aligned(scales, 2) || !aligned(prepared, 256))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_unprepare(static_cast<const uint8_t*>(prepared), N, K, f, packed,
                                        scales, zeros, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_gemv_fmt(const void* prepared, int64_t N, int64_t K, const w4_format* fmt,
                      const void* x, w4_dtype xt, int64_t M, void* y, w4_dtype yt,
                      hipStream_t stream) {
    if (!fmt) return W4_ERR_NULL;
    w4::Fmt f;
    w4_status st = to_fmt(fmt, &f);
    if (st != W4_OK) return st;
    if (f.group == W4_GROUP && !f.scale_bf16)
        return w4_gemv(prepared, N, K, x, xt, M, y, yt, stream);
    if (!prepared || !x || !y) return W4_ERR_NULL;
    if ((xt != W4_F32 && xt != W4_BF16) || (yt != W4_F32 && yt != W4_BF16)) return W4_ERR_DTYPE;
    st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (K > W4_GEMV_MAX_K || M < 1 || M > W4_GEMV_MAX_M) return W4_ERR_SHAPE;
    if (!aligned(prepared, 256) || !aligned(x, 16) || !aligned(y, yt == W4_F32 ? 4 : 2))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_gemv_dot2(static_cast<const uint8_t*>(prepared), N, K, f.group,
                                        f.scale_bf16, x, xt == W4_F32, M, y, yt == W4_BF16,
                                        stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

size_t w4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || check_nk(N, K) != W4_OK || K > W4_GEMM_MAX_K) return 0;
    return w4::gemm_workspace(M, K);
}

w4_status w4_gemm(const void* prepared, int64_t N, int64_t K, const void* X, int64_t M, void* Y,
                  w4_dtype yt, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!prepared || !X || !Y) return W4_ERR_NULL;
    if (yt != W4_F32 && yt != W4_BF16) return W4_ERR_DTYPE;
    w4_status st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (K > W4_GEMM_MAX_K || M < 1 || (M + 127) / 128 > 65535) return W4_ERR_SHAPE;
    // the tile count (128 x 256 output tiles, padded to a multiple of 8) is a grid size
    if (((M + 127) / 128) * ((N + 255) / 256) > (int64_t)INT32_MAX - 8) return W4_ERR_SHAPE;
    if (!workspace || workspace_bytes < w4_gemm_workspace_bytes(M, N, K)) return W4_ERR_WORKSPACE;
    if (!aligned(prepared, 256) || !aligned(X, 16) || !aligned(Y, yt == W4_F32 ? 4 : 2) ||
        !aligned(workspace, 16))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_gemm(static_cast<const uint8_t*>(prepared), N, K, X, M, Y,
                                   yt == W4_BF16, workspace, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_gemm_noalloc(const void* prepared, int64_t N, int64_t K, const void* X, int64_t M,
                          void* Y, w4_dtype yt, hipStream_t stream) {
    if (!prepared || !X || !Y) return W4_ERR_NULL;
    if (yt != W4_F32 && yt != W4_BF16) return W4_ERR_DTYPE;
    w4_status st = check_nk(N, K);
    if (st != W4_OK) return st;
    if (K > W4_GEMM_MAX_K || M < 1 || (M + 127) / 128 > 65535) return W4_ERR_SHAPE;
    if (((M + 127) / 128) * ((N + 255) / 256) > (int64_t)INT32_MAX - 8) return W4_ERR_SHAPE;
    if (w4_gemm_workspace_bytes(M, N, K) > W4_GEMM_NOALLOC_MAX_WORKSPACE) return W4_ERR_WORKSPACE;
    if (!aligned(prepared, 256) || !aligned(X, 16) || !aligned(Y, yt == W4_F32 ? 4 : 2))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    void* ws = nullptr;
    st = scratch_address(&ws);
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_gemm(static_cast<const uint8_t*>(prepared), N, K, X, M, Y,
                                   yt == W4_BF16, ws, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_fp8_quantize_rows(const void* A, w4_dtype at, int64_t rows, int64_t K,
                               uint8_t* codes, float* scales, uint32_t* d_status,
                               hipStream_t stream) {
    if (!A || !codes || !scales) return W4_ERR_NULL;
    if (at != W4_F32 && at != W4_BF16) return W4_ERR_DTYPE;
    if (rows < 1 || rows > (int64_t)INT32_MAX || K < W4_GROUP || K % W4_GROUP != 0 ||
        K > W4_FP8_MAX_K)
        return W4_ERR_SHAPE;
    if (!aligned(A, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(d_status, 4))
        return W4_ERR_ALIGN;
    w4_status st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_w8_quantize_rows(A, at == W4_BF16, rows, K, codes, scales,
                                                d_status, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_fp8_gemm(const uint8_t* xq, const float* sx, int64_t M, const uint8_t* wq,
                      const float* sw, int64_t N, int64_t K, void* Y, w4_dtype yt,
                      hipStream_t stream) {
    if (!xq || !sx || !wq || !sw || !Y) return W4_ERR_NULL;
    if (yt != W4_F32 && yt != W4_BF16) return W4_ERR_DTYPE;
    if (M < 1 || N < 1 || M > (int64_t)INT32_MAX || N > (int64_t)INT32_MAX || K < W4_GROUP ||
        K % W4_GROUP != 0 || K > W4_FP8_MAX_K)
        return W4_ERR_SHAPE;
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    if (tiles > (int64_t)INT32_MAX) return W4_ERR_SHAPE;
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
        !aligned(Y, yt == W4_F32 ? 4 : 2))
        return W4_ERR_ALIGN;
    w4_status st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_fp8_gemm(xq, sx, M, wq, sw, N, K, Y, yt == W4_BF16, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_int8_quantize_rows(const void* A, w4_dtype at, int64_t rows, int64_t K,
                                int8_t* codes, float* scales, uint32_t* d_status,
                                hipStream_t stream) {
    if (!A || !codes || !scales) return W4_ERR_NULL;
    if (at != W4_F32 && at != W4_BF16) return W4_ERR_DTYPE;
    if (rows < 1 || rows > (int64_t)INT32_MAX || K < W4_GROUP || K % W4_GROUP != 0 ||
        K > W4_FP8_MAX_K)
        return W4_ERR_SHAPE;
    if (!aligned(A, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(d_status, 4))
        return W4_ERR_ALIGN;
    w4_status st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_w8_quantize_rows(A, at == W4_BF16, rows, K,
                                                reinterpret_cast<uint8_t*>(codes), scales,
                                                d_status, stream, true);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_int8_gemm(const int8_t* xq, const float* sx, int64_t M, const int8_t* wq,
                       const float* sw, int64_t N, int64_t K, void* Y, w4_dtype yt,
                       hipStream_t stream) {
    if (!xq || !sx || !wq || !sw || !Y) return W4_ERR_NULL;
    if (yt != W4_F32 && yt != W4_BF16) return W4_ERR_DTYPE;
    if (M < 1 || N < 1 || M > (int64_t)INT32_MAX || N > (int64_t)INT32_MAX || K < W4_GROUP ||
        K % W4_GROUP != 0 || K > W4_FP8_MAX_K)
        return W4_ERR_SHAPE;
    const int64_t tiles = ((M + 127) / 128) * ((N + 255) / 256);
    if (tiles > (int64_t)INT32_MAX) return W4_ERR_SHAPE;
    if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
        !aligned(Y, yt == W4_F32 ? 4 : 2))
        return W4_ERR_ALIGN;
    w4_status st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_int8_gemm(reinterpret_cast<const uint8_t*>(xq), sx, M,
                                        reinterpret_cast<const uint8_t*>(wq), sw, N, K, Y,
                                        yt == W4_BF16, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

static w4_status rmsnorm_common(const void* x, w4_dtype xt, const void* residual,
                                void* residual_out, w4_dtype rt, const void* weight, w4_dtype wt,
                                float eps, int64_t rows, int64_t K, const w4::RowOut& out,
                                hipStream_t stream) {
    const bool codes = out.kind == w4::RowOut::kFp8 || out.kind == w4::RowOut::kInt8;
    if (!x || !weight || !out.y || (codes && !out.scales) || !residual != !residual_out)
        return W4_ERR_NULL;
    if (!is_dtype(xt) || !is_dtype(wt) || (residual && !is_dtype(rt))) return W4_ERR_DTYPE;
    w4_status st = check_rows(rows, K);
    if (st != W4_OK) return st;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return W4_ERR_VALUE;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
        !aligned(weight, 16) || !aligned(out.y, 16) || !aligned(out.scales, 4) ||
        !aligned(out.status, 4))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    w4::RmsnormArgs a;
    a.x = x;
    a.r = residual;
    a.r_out = residual_out;
    a.w = weight;
    a.x_f32 = xt == W4_F32;
    a.r_f32 = rt == W4_F32;
    a.w_f32 = wt == W4_F32;
    a.eps = eps;
    a.rows = rows;
    a.K = K;
    const hipError_t e = w4::launch_rmsnorm(a, out, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_rmsnorm(const void* x, w4_dtype xt, const void* residual, void* residual_out,
                     w4_dtype rt, const void* weight, w4_dtype wt, float eps, int64_t rows,
                     int64_t K, void* y, w4_dtype yt, hipStream_t stream) {
    if (!is_dtype(yt)) return W4_ERR_DTYPE;
    const w4::RowOut out = {yt == W4_F32 ? w4::RowOut::kF32 : w4::RowOut::kBf16, y, nullptr, nullptr};
    return rmsnorm_common(x, xt, residual, residual_out, rt, weight, wt, eps, rows, K, out, stream);
}

w4_status w4_rmsnorm_fp8(const void* x, w4_dtype xt, const void* residual, void* residual_out,
                         w4_dtype rt, const void* weight, w4_dtype wt, float eps, int64_t rows,
                         int64_t K, uint8_t* codes, float* scales, uint32_t* d_status,
                         hipStream_t stream) {
    const w4::RowOut out = {w4::RowOut::kFp8, codes, scales, d_status};
    return rmsnorm_common(x, xt, residual, residual_out, rt, weight, wt, eps, rows, K, out, stream);
}

w4_status w4_rmsnorm_int8(const void* x, w4_dtype xt, const void* residual, void* residual_out,
                          w4_dtype rt, const void* weight, w4_dtype wt, float eps, int64_t rows,
                          int64_t K, int8_t* codes, float* scales, uint32_t* d_status,
                          hipStream_t stream) {
    const w4::RowOut out = {w4::RowOut::kInt8, codes, scales, d_status};
    return rmsnorm_common(x, xt, residual, residual_out, rt, weight, wt, eps, rows, K, out, stream);
}

static w4_status silu_mul_common(const void* gate_up, w4_dtype gt, int64_t rows, int64_t F,
                                 const w4::RowOut& out, hipStream_t stream) {
    const bool codes = out.kind == w4::RowOut::kFp8 || out.kind == w4::RowOut::kInt8;
    if (!gate_up || !out.y || (codes && !out.scales)) return W4_ERR_NULL;
    if (!is_dtype(gt)) return W4_ERR_DTYPE;
    w4_status st = check_rows(rows, F);
    if (st != W4_OK) return st;
    if (!aligned(gate_up, 16) || !aligned(out.y, 16) || !aligned(out.scales, 4) ||
        !aligned(out.status, 4))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    const hipError_t e = w4::launch_silu_mul(gate_up, gt == W4_F32, rows, F, out, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_silu_mul(const void* gate_up, w4_dtype gt, int64_t rows, int64_t F, void* y,
                      w4_dtype yt, hipStream_t stream) {
    if (!is_dtype(yt)) return W4_ERR_DTYPE;
    const w4::RowOut out = {yt == W4_F32 ? w4::RowOut::kF32 : w4::RowOut::kBf16, y, nullptr, nullptr};
    return silu_mul_common(gate_up, gt, rows, F, out, stream);
}

w4_status w4_silu_mul_fp8(const void* gate_up, w4_dtype gt, int64_t rows, int64_t F,
                          uint8_t* codes, float* scales, uint32_t* d_status, hipStream_t stream) {
    const w4::RowOut out = {w4::RowOut::kFp8, codes, scales, d_status};
    return silu_mul_common(gate_up, gt, rows, F, out, stream);
}

w4_status w4_silu_mul_int8(const void* gate_up, w4_dtype gt, int64_t rows, int64_t F,
                           int8_t* codes, float* scales, uint32_t* d_status, hipStream_t stream) {
    const w4::RowOut out = {w4::RowOut::kInt8, codes, scales, d_status};
    return silu_mul_common(gate_up, gt, rows, F, out, stream);
}

w4_status w4_rope_frequencies(const w4_rope* rope, double* freqs, double* amplitude) {
    if (!freqs) return W4_ERR_NULL;
    const w4_status st = check_rope(rope);
    if (st != W4_OK) return st;
    const int half = rope->rotary_dim / 2;
    const double two_pi = 6.283185307179586476925;
    double first = 0.0, last = 0.0;                          // pairs between which the ramp rises
    if (rope->scaling == W4_ROPE_RAMP) {
        const auto pair_of = [&](double turns) {
            return half * std::log((double)rope->original_positions / (two_pi * turns)) /
                   std::log(rope->base);
        };
        first = std::floor(pair_of(rope->high));
        last = std::ceil(pair_of(rope->low));
        // a ramp that ends ahead of the first pair or begins behind the last place stays there
        if (last >= 0.0 && first <= 2.0 * half - 1.0) {
            first = std::fmax(0.0, first);
            last = std::fmin(2.0 * half - 1.0, last);
        }
        if (first == last) last += 0.001;
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(rope->base, -(double)i / half);
        switch (rope->scaling) {
            case W4_ROPE_LINEAR: f /= rope->factor; break;
            case W4_ROPE_BANDS: {
                const double turns = (double)rope->original_positions * f / two_pi;
                const double k = std::fmin(1.0, std::fmax(0.0, (turns - rope->low) / (rope->high - rope->low)));
                f *= k + (1.0 - k) / rope->factor;
                break;
            }
            case W4_ROPE_RAMP: {
                const double r = std::fmin(1.0, std::fmax(0.0, (i - first) / (last - first)));
                f *= 1.0 - r + r / rope->factor;
                break;
            }
            default: break;
        }
        freqs[i] = f;
    }
    if (amplitude) *amplitude = rope_amplitude(rope);
    return W4_OK;
}

// What a write into a cache takes, without rotation.
static w4::RopeArgs rope_args(const w4_kv_cache* cache, int shift, const void* qkv, int64_t T, int64_t heads,
                              const int64_t* slots, void* q, uint32_t* d_status) {
    w4::RopeArgs a = {};
    a.qkv = qkv;
    a.slots = slots;
    a.q = static_cast<uint16_t*>(q);
    a.k = cache->k;
    a.v = cache->v;
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.status = d_status;
    a.T = T;
    a.pages = cache->pages;
    a.heads = (int)heads;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.page_shift = shift;
    a.amplitude = 1.0f;
    return a;
}

static hipError_t launch_cache_write(const w4::RopeArgs& a, w4_dtype xt, int type, hipStream_t stream) {
    if (type == W4_CACHE_INT8) return w4::launch_write_blocks(a, xt == W4_F32, stream);
    return w4::launch_rope_cache(a, xt == W4_F32, type == W4_CACHE_FP8, stream);
}

w4_status w4_rope_cache(const void* qkv, w4_dtype xt, int64_t T, int64_t heads,
                        const w4_kv_cache* cache, const int32_t* positions, const int64_t* slots,
                        const w4_rope* rope, const double* d_freqs, void* q, uint32_t* d_status,
                        hipStream_t stream) {
    if (!qkv || !cache || !positions || !slots || !rope || !d_freqs || !q) return W4_ERR_NULL;
    if (!is_dtype(xt)) return W4_ERR_DTYPE;
    int shift = 0;
    w4_status st = check_cache(cache, &shift);
    if (st == W4_OK) st = check_cache_pointers(cache);
    if (st == W4_OK) st = check_heads(T, heads, cache);
    if (st == W4_OK) st = check_rope(rope);
    if (st != W4_OK) return st;
    if (rope->rotary_dim > cache->head_dim) return W4_ERR_SHAPE;
    if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(positions, 4) || !aligned(slots, 8) ||
        !aligned(d_freqs, 8) || !aligned(d_status, 4))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    w4::RopeArgs a = rope_args(cache, shift, qkv, T, heads, slots, q, d_status);
    a.positions = positions;
    a.freqs = d_freqs;
    a.rotary = rope->rotary_dim;
    a.interleaved = rope->interleaved;
    a.amplitude = (float)rope_amplitude(rope);
    const hipError_t e = launch_cache_write(a, xt, cache->type, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_cache_write(const void* qkv, w4_dtype xt, int64_t T, int64_t heads, const w4_kv_cache* cache,
                         const int64_t* slots, void* q, uint32_t* d_status, hipStream_t stream) {
    if (!qkv || !cache || !slots || (heads != 0 && !q)) return W4_ERR_NULL;
    if (!is_dtype(xt)) return W4_ERR_DTYPE;
    int shift = 0;
    w4_status st = check_cache(cache, &shift);
    if (st == W4_OK) st = check_cache_pointers(cache);
    if (st == W4_OK) st = check_heads(T, heads == 0 ? cache->kv_heads : heads, cache);
    if (st != W4_OK) return st;
    if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(slots, 8) || !aligned(d_status, 4)) return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    w4::RopeArgs a = rope_args(cache, shift, qkv, T, heads, slots, q, d_status);
    const hipError_t e = launch_cache_write(a, xt, cache->type, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_cache_read(const w4_kv_cache* cache, const int64_t* slots, int64_t n, void* kv, w4_dtype yt,
                        uint32_t* d_status, hipStream_t stream) {
    if (!cache || !slots || !kv) return W4_ERR_NULL;
    if (!is_dtype(yt)) return W4_ERR_DTYPE;
    int shift = 0;
    w4_status st = check_cache(cache, &shift);
    if (st == W4_OK) st = check_cache_pointers(cache);
    if (st != W4_OK) return st;
    if (n < 1 || n > W4_MAX_TOKENS) return W4_ERR_SHAPE;
    if (!aligned(slots, 8) || !aligned(kv, 16) || !aligned(d_status, 4)) return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    w4::ReadArgs a;
    a.k = cache->k;
    a.v = cache->v;
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.slots = slots;
    a.out = kv;
    a.status = d_status;
    a.n = n;
    a.pages = cache->pages;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.page_shift = shift;
    const hipError_t e = w4::launch_cache_read(a, cache_kind(cache), yt == W4_F32, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_block_tables(const int32_t* new_lens, const int32_t* lens_in, int64_t B,
                          const int32_t* free_pages, int64_t free_capacity,
                          const int32_t* free_count_in, int32_t* lens_out,
                          int32_t* free_count_out, int32_t* block_table, int64_t max_pages,
                          int32_t page_size, int32_t* cu_q, int32_t* positions, int64_t* slots,
                          int64_t T, uint32_t* d_status, hipStream_t stream) {
    if (!new_lens || !lens_in || (!free_pages && free_capacity != 0) || !free_count_in ||
        !lens_out || !free_count_out || !block_table || !cu_q || !positions || !slots)
        return W4_ERR_NULL;
    int shift = 0;
    w4_status st = check_page_size(page_size, &shift);
    if (st != W4_OK) return st;
    st = check_batch(B, max_pages, page_size);
    if (st != W4_OK) return st;
    if (T < 1 || T > W4_MAX_TOKENS || free_capacity < 0 || free_capacity > (int64_t)INT32_MAX)
        return W4_ERR_SHAPE;
    if (!aligned(new_lens, 4) || !aligned(lens_in, 4) || !aligned(free_pages, 4) ||
        !aligned(free_count_in, 4) || !aligned(lens_out, 4) || !aligned(free_count_out, 4) ||
        !aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(positions, 4) ||
        !aligned(slots, 8) || !aligned(d_status, 4))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    w4::TableArgs a;
    a.new_lens = new_lens;
    a.lens_in = lens_in;
    a.free_pages = free_pages;
    a.count_in = free_count_in;
    a.lens_out = lens_out;
    a.count_out = free_count_out;
    a.table = block_table;
    a.cu = cu_q;
    a.positions = positions;
    a.slots = slots;
    a.status = d_status;
    a.free_capacity = free_capacity;
    a.max_pages = max_pages;
    a.T = T;
    a.B = (int)B;
    a.page_shift = shift;
    const hipError_t e = w4::launch_block_tables(a, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

size_t w4_paged_attention_workspace_bytes(int64_t T, int64_t heads, const w4_kv_cache* cache,
                                          int64_t B, int64_t max_pages) {
    int shift = 0;
    if (check_cache(cache, &shift) != W4_OK || check_heads(T, heads, cache) != W4_OK ||
        check_batch(B, max_pages, cache->page_size) != W4_OK)
        return 0;
    w4::AttendPlan plan;
    w4::plan_attend(T, B, heads, cache->kv_heads, max_pages << shift,
                    cache->type != W4_CACHE_BF16, &plan);
    return w4::attend_workspace(cache->head_dim, plan);
}

static w4_status attend_common(const void* q, int64_t T, int64_t heads, const w4_kv_cache* cache,
                               const int32_t* block_table, int64_t max_pages, const int32_t* cu_q,
                               const int32_t* lens, int64_t B, float scale, int64_t window, const w4_scores& scores,
                               void* o, void* workspace, size_t workspace_bytes, uint32_t* d_status,
                               hipStream_t stream) {
    if (!q || !cache || !block_table || !cu_q || !lens || !o) return W4_ERR_NULL;
    int shift = 0;
    w4_status st = check_cache(cache, &shift);
    if (st == W4_OK) st = check_cache_pointers(cache);
    if (st == W4_OK) st = check_heads(T, heads, cache);
    if (st == W4_OK) st = check_batch(B, max_pages, cache->page_size);
    if (st != W4_OK) return st;
    if (scores.reserved != 0) return W4_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0) return W4_ERR_VALUE;
    if (scores.cap != 0.0f && !(scale <= 256.0f && scores.cap >= 0x1p-20f * scale && scores.cap <= 0x1p20f * scale))
        return W4_ERR_VALUE;
    w4::AttendPlan plan;
    w4::plan_attend(T, B, heads, cache->kv_heads, max_pages << shift,
                    cache->type != W4_CACHE_BF16, &plan);
    const size_t need = w4::attend_workspace(cache->head_dim, plan);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4_ERR_WORKSPACE;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(block_table, 4) || !aligned(cu_q, 4) ||
        !aligned(lens, 4) || !aligned(scores.slopes, 4) || !aligned(scores.first_keys, 4) ||
        !aligned(scores.prefix_lens, 4) || !aligned(workspace, 16) || !aligned(d_status, 4))
        return W4_ERR_ALIGN;
    st = check_arch();
    if (st != W4_OK) return st;
    w4::AttendArgs a = {};
    a.q = static_cast<const uint16_t*>(q);
    a.o = static_cast<uint16_t*>(o);
    a.k = cache->k;
    a.v = cache->v;
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.table = block_table;
    a.cu = cu_q;
    a.lens = lens;
    a.status = d_status;
    a.T = (int)T;
    a.capacity = (int)(max_pages << shift);
    a.pages = cache->pages;
    a.max_pages = max_pages;
    a.B = (int)B;
    a.heads = (int)heads;
    a.kv_heads = cache->kv_heads;
    a.group = (int)(heads / cache->kv_heads);
    a.page_shift = shift;
    a.window = (int)(window < W4_MAX_CONTEXT ? window : 0);   // wider than any context: none
    a.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    a.slopes = scores.slopes;
    a.first = scores.first_keys;
    a.prefix = scores.prefix_lens;
    a.ranges = a.first || a.prefix;
    if (scores.cap != 0.0f) {
        // tanh(y) / y of y^2 in [0, 0.28^2], met at the Chebyshev nodes 0.0392 (1 + cos((2 i + 1) pi / 6)): within 7.8e-7
        const double k[3] = {0.9999992246769208, -0.3331550113021886, 0.1272063837601273};
        const double log2e = 1.4426950408889634074, y = (double)scale / scores.cap, s = scale * log2e;
        a.cap_log2 = (float)(scores.cap * log2e);
        a.cap_exp = (float)(2.0 * y * log2e);
        a.cap_small = (float)(0.28 / y);
        a.cap_c1 = (float)(s * k[0]);
        a.cap_c3 = (float)(s * y * y * k[1]);
        a.cap_c5 = (float)(s * y * y * y * y * k[2]);
    }
    const hipError_t e = w4::launch_attend(a, cache->head_dim, cache_kind(cache), plan, workspace, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

w4_status w4_paged_attention(const void* q, int64_t T, int64_t heads, const w4_kv_cache* cache,
                             const int32_t* block_table, int64_t max_pages, const int32_t* cu_q,
                             const int32_t* lens, int64_t B, float scale, int64_t window, void* o,
                             void* workspace, size_t workspace_bytes, uint32_t* d_status,
                             hipStream_t stream) {
    return attend_common(q, T, heads, cache, block_table, max_pages, cu_q, lens, B, scale, window, w4_scores{}, o,
                         workspace, workspace_bytes, d_status, stream);
}

w4_status w4_paged_attention_scores(const void* q, int64_t T, int64_t heads, const w4_kv_cache* cache,
                                    const int32_t* block_table, int64_t max_pages, const int32_t* cu_q,
                                    const int32_t* lens, int64_t B, float scale, int64_t window,
                                    const w4_scores* scores, void* o, void* workspace, size_t workspace_bytes,
                                    uint32_t* d_status, hipStream_t stream) {
    if (!scores) return W4_ERR_NULL;
    return attend_common(q, T, heads, cache, block_table, max_pages, cu_q, lens, B, scale, window, *scores, o,
                         workspace, workspace_bytes, d_status, stream);
}

w4_status w4_stream_read(const void* buf, size_t bytes, uint32_t* sink, hipStream_t stream) {
    if (!buf || !sink) return W4_ERR_NULL;
    if (bytes == 0 || bytes % 16 != 0) return W4_ERR_SHAPE;
    if (!aligned(buf, 16) || !aligned(sink, 4)) return W4_ERR_ALIGN;
    w4_status st = check_arch();
    if (st != W4_OK) return st;
    hipError_t e = w4::launch_stream_read(buf, (int64_t)bytes, sink, stream);
    return e == hipSuccess ? W4_OK : hip_fail(e);
}

}  // extern "C"
