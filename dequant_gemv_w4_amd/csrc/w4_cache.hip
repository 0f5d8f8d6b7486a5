// What stands between the fused q|k|v product and the attention: rotary positions with the write
// of K and V into the paged cache, and the block tables and slots that the write goes by.
//
// Rotary positions: the pair (x0, x1) of a head at position p turns by the angle p * f,
//     (A (x0 cos - x1 sin), A (x0 sin + x1 cos)),
// with f and the amplitude A from w4_rope_frequencies.  Pairs are (i, i + R/2) of the first R
// elements of a head, or (2i, 2i+1).  p * f passes 2^24 turns' worth of binary32 at far
// positions, so the turns p * f / 2 pi are formed in binary64 and only their fraction goes on in
// binary32 (angles are off by less than 2^-24 turns wherever p * f < 2^28).  A workgroup takes
// one token, so the R/2 sines and cosines are formed once for all heads.
//
// Bound by memory: each row is read once and written once.  A lane takes two chunks of 8
// elements that hold 8 whole pairs, so no element moves between lanes, and D / 16 neighbouring
// lanes hold a head, which gives the E4M3 row its largest value by shuffles.  4096 tokens of 32 + 64
// heads of 128 in bfloat16 (201 MB) take 44.5 us, 4.5 TB/s; 16 tokens of 64 + 16 heads into E4M3 3.4 us.
#include "w4_codes.h"
#include "w4_internal.h"
#include "w4_paging.h"

namespace w4 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 64;   // head_dim 128

__device__ __forceinline__ uint32_t bf16_pair2(float a, float b) {
    typedef float f2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
    const f2_t f = {a, b};
    const b2_t h = __builtin_convertvector(f, b2_t);
    return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, const float* v) {
    u32x4_t a;
#pragma unroll
    for (int q = 0; q < 4; ++q) a[q] = bf16_pair2(v[2 * q], v[2 * q + 1]);
    *reinterpret_cast<u32x4_t*>(p) = a;
}

template <bool XF32, bool FP8>
__global__ __launch_bounds__(kRopeThreads) void rope_cache_kernel(RopeArgs a) {
    __shared__ float cs[kMaxPairs], sn[kMaxPairs];
    const int64_t t = blockIdx.x;
    const int D = a.head_dim;
    const int lanes = D >> 4;                                // lanes of a head: 4 or 8
    const int half = a.rotary >> 1;
    const int item = blockIdx.y * kRopeThreads + threadIdx.x;
    const int head = item / lanes, u = item & (lanes - 1);
    const bool active = head < a.heads + 2 * a.kv_heads;
    const bool split = u < (a.rotary >> 4) && !a.interleaved;
    const int c0 = split ? 8 * u : 16 * u;
    const int c1 = split ? 8 * u + half : 16 * u + 8;
    // the row's values are on their way while the angles are formed
    float v[16];
    if (active) {
        const int64_t from = (t * (a.heads + 2 * a.kv_heads) + head) * D;
        load8<!XF32>(a.qkv, from + c0, v);
        load8<!XF32>(a.qkv, from + c1, v + 8);
    }
    const int64_t slot = a.slots[t];
    if ((int)threadIdx.x < half) {
        const double turns = (double)a.positions[t] * a.freqs[threadIdx.x] * 0.15915494309189533577;
        const float part = (float)(turns - rint(turns));     // [-1/2, 1/2]
        float s, c;
        sincospif(2.0f * part, &s, &c);
        cs[threadIdx.x] = c * a.amplitude;
        sn[threadIdx.x] = s * a.amplitude;
    }
    __syncthreads();
    if (slot < 0 || !active) return;                         // padding: nothing is written
    if (slot >= a.pages << a.page_shift) {
        if (item == 0 && a.status) atomicOr(a.status, kStatusPage);
        return;
    }
    if (u < (a.rotary >> 4) && head < a.heads + a.kv_heads) {
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
    if (head < a.heads) {
        uint16_t* q = a.q + (t * a.heads + head) * D;
        store8_bf16(q + c0, v);
        store8_bf16(q + c1, v + 8);
        return;
    }
    const bool is_v = head >= a.heads + a.kv_heads;
    const int kvh = head - a.heads - (is_v ? a.kv_heads : 0);
    const int64_t page = slot >> a.page_shift;
    const int64_t row = ((page * a.kv_heads + kvh) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
    if constexpr (!FP8) {
        uint16_t* dst = static_cast<uint16_t*>(is_v ? a.v : a.k) + row * D;
        store8_bf16(dst + c0, v);
        store8_bf16(dst + c1, v + 8);
    } else {
        float amax = 0.0f, off = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            amax = fmaxf(amax, fabsf(v[j]));
            off += v[j] - v[j];                              // 0 for finite values only
        }
        for (int d = lanes >> 1; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
        const double s = amax == 0.0f ? 1.0 : (double)amax / kFp8Max;
        const float rs = (float)(1.0 / s);
        // values that are not finite take the quotients, so that their bytes are the row quantizers' too
        const bool ok = s >= 0x1p-100 && s <= 0x1p100 && off == 0.0f;
        if (u == 0) (is_v ? a.v_scales : a.k_scales)[row] = (float)s;
        uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v : a.k) + row * D;
        *reinterpret_cast<uint2*>(dst + c0) = w8_codes8_of<false>(v, s, rs, ok);
        *reinterpret_cast<uint2*>(dst + c1) = w8_codes8_of<false>(v + 8, s, rs, ok);
        if (off != 0.0f && a.status) atomicOr(a.status, kStatusNonfinite);
    }
}

// --------------------------------------------------------------------------
// Block tables and slots
// --------------------------------------------------------------------------
//
// Two exclusive sums over the requests, of their new tokens and of the pages they take, place
// everything; each new token then finds its request by a search in the first sum.  Every
// workgroup scans the requests itself (8 bytes a request, read from the cache by all but the
// first), which is cheaper than a launch of its own.  Bound by the latency of that scan and of the
// search behind it: 64 requests with a token each take 5.3 us, 256 with 8252 tokens 7.4.  The new
// lengths and the rest of the list are written by the first workgroup, unless others may still read
// the old ones in their place: with more than one workgroup and an update in place a second launch
// writes them.

constexpr int kTableThreads = 1024;

struct Scan {
    int cu[kMaxSeqs + 1];        // first token of each request
    int taken[kMaxSeqs];         // pages taken ahead of it
    int cached[kMaxSeqs];        // its cached tokens; -1: not served
    long long wave_n[kTableThreads / 64], wave_p[kTableThreads / 64];
    long long carry_n, carry_p, served_p;
    unsigned status;
    int pages_short;             // some request's pages are not there
};

// Where the pages run out the sums hold requests that take none.  Then one wave goes through the requests in
// order, 64 at a time: those that need more than is left by now are refused at once, and of the others all
// are served up to the first whose pages are not there, which is refused, and so on behind it.  64 requests
// of which 63 are short take 8.3 us instead of the 7.4 of the sums alone, 4096 of which 4095 are 75
// instead of 29; where none is short nothing is spent.
__device__ __forceinline__ void serve_in_order(const TableArgs& a, Scan& sc, int64_t count) {
    const int lane = threadIdx.x;
    if (lane < 64) {
        long long left = count;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
            const int b = b0 + lane;
            long long need = 0;                              // of requests that are neither served nor refused yet
            if (b < a.B && sc.cached[b] >= 0)
                need = page_need(a.lens_in[b], a.new_lens[b], (int64_t)1 << a.page_shift, a.max_pages).take;
            while (__any(need > 0)) {
                if (need > left) {
                    sc.cached[b] = -1;
                    need = 0;
                }
                long long sum = need;
#pragma unroll
                for (int off = 1; off < 64; off <<= 1) {
                    const long long up = __shfl_up(sum, off);
                    if (lane >= off) sum += up;
                }
                const uint64_t over = __ballot(sum > left);
                const int first = over ? __builtin_ctzll(over) : 64;   // one that needs pages
                if (need > 0 && lane < first) sc.taken[b] = (int)(count - left + sum - need);
                if (lane == first) sc.cached[b] = -1;
                const long long all = __shfl(sum, first > 0 ? first - 1 : 0);
                if (first > 0) left -= all;
                if (lane <= first) need = 0;
            }
        }
        if (lane == 0) sc.served_p = count - left;
    }
    __syncthreads();
}

__device__ __forceinline__ void scan_requests(const TableArgs& a, Scan& sc) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0) {
        sc.carry_n = sc.carry_p = sc.served_p = 0;
        sc.status = 0;
        sc.pages_short = 0;
    }
    __syncthreads();
    const int64_t count = imin(imax(*a.count_in, 0), a.free_capacity);
    const int64_t page = 1 << a.page_shift;
    for (int b0 = 0; b0 < a.B; b0 += kTableThreads) {
        const int b = b0 + tid;
        const int64_t len = b < a.B ? a.lens_in[b] : 0;
        const int64_t fresh = b < a.B ? a.new_lens[b] : 0;
        const Need d = page_need(len, fresh, page, a.max_pages);
        long long n = fresh > 0 ? fresh : 0, p = d.take;
        const long long own_n = n, own_p = p;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const long long un = __shfl_up(n, off), up = __shfl_up(p, off);
            if (lane >= off) {
                n += un;
                p += up;
            }
        }
        if (lane == 63) {
            sc.wave_n[wave] = n;
            sc.wave_p[wave] = p;
        }
        __syncthreads();
        long long before_n = sc.carry_n, before_p = sc.carry_p;
        for (int w = 0; w < wave; ++w) {
            before_n += sc.wave_n[w];
            before_p += sc.wave_p[w];
        }
        const long long start = before_n + n - own_n, ahead = before_p + p - own_p;
        if (b < a.B) {
            unsigned st = 0;
            if (len < 0 || fresh < 0 || start + own_n > a.T) st |= kStatusLength;
            else if (!d.fits) st |= kStatusPagesShort;
            sc.cu[b] = (int)imin(start, a.T);
            sc.taken[b] = (int)imin(ahead, INT32_MAX);
            sc.cached[b] = st ? -1 : (int)len;
            if (!st && own_p > 0) {
                if (ahead + own_p > count) {                 // at least the first of these is refused
                    st |= kStatusPagesShort;
                    sc.pages_short = 1;
                } else {
                    atomicMax(&sc.served_p, ahead + own_p);
                }
            }
            if (st) atomicOr(&sc.status, st);
        }
        __syncthreads();
        if (tid == kTableThreads - 1) {
            sc.carry_n = before_n + n;
            sc.carry_p = before_p + p;
        }
        __syncthreads();
    }
    if (tid == 0) sc.cu[a.B] = (int)imin(sc.carry_n, a.T);
    __syncthreads();
    if (sc.pages_short) serve_in_order(a, sc, count);
}

__device__ __forceinline__ void write_lengths(const TableArgs& a, const Scan& sc) {
    const int64_t count = imin(imax(*a.count_in, 0), a.free_capacity);
    for (int b = threadIdx.x; b < a.B; b += kTableThreads) {
        const int len = a.lens_in[b];
        a.lens_out[b] = sc.cached[b] < 0 ? len : len + a.new_lens[b];
    }
    __syncthreads();                                         // count_out may be count_in
    if (threadIdx.x == 0) {
        *a.count_out = (int)(count - sc.served_p);
        if (sc.status && a.status) atomicOr(a.status, sc.status);
    }
}

// lengths: whether the first workgroup writes them.
__global__ __launch_bounds__(kTableThreads) void block_tables_kernel(TableArgs a, bool lengths) {
    __shared__ Scan sc;
    scan_requests(a, sc);
    const int64_t count = imin(imax(*a.count_in, 0), a.free_capacity);
    const int total = sc.cu[a.B];
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b <= a.B; b += kTableThreads) a.cu[b] = sc.cu[b];
    const int64_t page_size = 1 << a.page_shift;
    for (int64_t t = (int64_t)blockIdx.x * kTableThreads + threadIdx.x; t < a.T;
         t += (int64_t)gridDim.x * kTableThreads) {
        if (t >= total) {
            a.positions[t] = 0;
            a.slots[t] = -1;
            continue;
        }
        int lo = 0, hi = a.B;                                // cu[lo] <= t < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sc.cu[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        if (sc.cached[lo] < 0) {
            a.positions[t] = 0;
            a.slots[t] = -1;
            continue;
        }
        const int64_t pos = (int64_t)sc.cached[lo] + (t - sc.cu[lo]);
        const int64_t at = pos >> a.page_shift;
        const int64_t have = (sc.cached[lo] + page_size - 1) >> a.page_shift;
        int32_t* entry = a.table + (int64_t)lo * a.max_pages + at;
        int64_t page;
        if (at >= have) {
            page = a.free_pages[count - 1 - (sc.taken[lo] + at - have)];
            if ((pos & (page_size - 1)) == 0) *entry = (int32_t)page;   // its first token writes it
        } else {
            page = *entry;
        }
        a.positions[t] = (int32_t)pos;
        a.slots[t] = page < 0 ? -1 : (page << a.page_shift) + (pos & (page_size - 1));
    }
    if (lengths && blockIdx.x == 0) {
        __syncthreads();
        write_lengths(a, sc);
    }
}

__global__ __launch_bounds__(kTableThreads) void table_lengths_kernel(TableArgs a) {
    __shared__ Scan sc;
    scan_requests(a, sc);
    write_lengths(a, sc);
}

}  // namespace

hipError_t launch_rope_cache(const RopeArgs& a, bool x_f32, bool fp8, hipStream_t s) {
    const int64_t items = (int64_t)(a.heads + 2 * a.kv_heads) * (a.head_dim / 16);
    const dim3 grid((unsigned)a.T, (unsigned)ceil_div(items, kRopeThreads)), block(kRopeThreads);
    if (x_f32 && fp8)
        hipLaunchKernelGGL((rope_cache_kernel<true, true>), grid, block, 0, s, a);
    else if (x_f32)
        hipLaunchKernelGGL((rope_cache_kernel<true, false>), grid, block, 0, s, a);
    else if (fp8)
        hipLaunchKernelGGL((rope_cache_kernel<false, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((rope_cache_kernel<false, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_block_tables(const TableArgs& a, hipStream_t s) {
    // One workgroup up to 8 tokens a thread, then more: 256 requests with 8252 tokens take 13 us either
    // way in place, 7.5 apart.
    const int64_t wgs = a.T <= 8 * kTableThreads ? 1 : imin(ceil_div(a.T, kTableThreads), 256);
    const bool in_place = a.lens_out == a.lens_in || a.count_out == a.count_in;
    const bool at_once = wgs == 1 || !in_place;
    hipLaunchKernelGGL(block_tables_kernel, dim3((unsigned)wgs), dim3(kTableThreads), 0, s, a, at_once);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || at_once) return e;
    hipLaunchKernelGGL(table_lengths_kernel, dim3(1), dim3(kTableThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace w4
