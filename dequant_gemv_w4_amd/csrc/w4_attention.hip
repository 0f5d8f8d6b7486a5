// Launches of the attention (w4_attention.h): the plain causal form over bfloat16 and E4M3 caches, the join
// of the parts, and which of the other sources a call goes to.
#include "w4_attention.h"

namespace w4 {

static int64_t split_rows(bool wide, const AttendPlan& p) {
    const int64_t tiles = wide ? p.wide_tiles : p.narrow_tiles;
    return (wide ? p.wide_parts : p.narrow_parts) > 1 ? tiles * (wide ? kWideRows : p.narrow_tile) : 0;
}

size_t attend_workspace(int64_t D, const AttendPlan& p) {
    return (size_t)(split_rows(false, p) * p.narrow_parts + split_rows(true, p) * p.wide_parts) * (D + 2) * 4;
}

template <int MOD>
static hipError_t launch_combine(const AttendArgs& a, int head_dim, hipStream_t s) {
    const dim3 grid((unsigned)((a.wide_rows + a.narrow_rows) / 4)), block(256);
    if (head_dim == 128)
        hipLaunchKernelGGL((combine_kernel<128, MOD>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((combine_kernel<64, MOD>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_attend(AttendArgs a, int head_dim, int type, const AttendPlan& p, void* workspace, hipStream_t s) {
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
    const int mod = (a.ranges ? kRanges : 0) | (a.slopes ? kBias : 0) | (a.cap_log2 != 0.0f ? kCap : 0);
    hipError_t e;
    if (type == kInt8Rows)
        e = launch_attend_int8(a, head_dim, mod ? mod | kRanges : 0, p, s);
    else if (mod)
        e = type == kFp8Rows ? launch_attend_scores_fp8(a, head_dim, mod | kRanges, p, s)
                             : launch_attend_scores_bf16(a, head_dim, mod | kRanges, p, s);
    else
        e = type == kFp8Rows ? launch_attend_type<kFp8Rows, 0>(a, head_dim, p, s) : launch_attend_type<kBf16Rows, 0>(a, head_dim, p, s);
    if (e != hipSuccess || a.wide_rows + a.narrow_rows == 0) return e;
    return mod ? launch_combine<kRanges>(a, head_dim, s) : launch_combine<0>(a, head_dim, s);
}

}  // namespace w4
