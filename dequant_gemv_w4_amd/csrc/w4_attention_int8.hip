// The attention (w4_attention.h) over INT8 caches.
#include "w4_attention.h"

namespace w4 {

hipError_t launch_attend_int8(const AttendArgs& a, int head_dim, int mod, const AttendPlan& p, hipStream_t s) {
    switch (mod) {
        case 0: return launch_attend_type<kInt8Rows, 0>(a, head_dim, p, s);
        case kRanges: return launch_attend_type<kInt8Rows, kRanges>(a, head_dim, p, s);
        case kRanges | kBias: return launch_attend_type<kInt8Rows, kRanges | kBias>(a, head_dim, p, s);
        case kRanges | kCap: return launch_attend_type<kInt8Rows, kRanges | kCap>(a, head_dim, p, s);
        default: return launch_attend_type<kInt8Rows, kRanges | kBias | kCap>(a, head_dim, p, s);
    }
}

}  // namespace w4
