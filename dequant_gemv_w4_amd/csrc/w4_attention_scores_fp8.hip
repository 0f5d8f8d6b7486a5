// The attention (w4_attention.h) with capped scores, a bias by distance or key ranges, over E4M3 caches.
#include "w4_attention.h"

namespace w4 {

hipError_t launch_attend_scores_fp8(const AttendArgs& a, int head_dim, int mod, const AttendPlan& p, hipStream_t s) {
    switch (mod) {
        case kRanges: return launch_attend_type<kFp8Rows, kRanges>(a, head_dim, p, s);
        case kRanges | kBias: return launch_attend_type<kFp8Rows, kRanges | kBias>(a, head_dim, p, s);
        case kRanges | kCap: return launch_attend_type<kFp8Rows, kRanges | kCap>(a, head_dim, p, s);
        default: return launch_attend_type<kFp8Rows, kRanges | kBias | kCap>(a, head_dim, p, s);
    }
}

}  // namespace w4
