// fa_fwd_ranges.cuh -- how the forward kernels read the visible-key intervals
// of fa_mask_ranges.
#pragma once

#include "fa_params.h"

namespace fa {

// The keys a 128-row tile of a problem with visible-key intervals may see:
// the bounds of its two 64-row blocks.  *first / *last: no key if last < first.
__device__ __forceinline__ void tile_range(const BwdParams &p, int b, int m, int lk, long long *first,
                                           long long *last) {
    const int4 *blk = p.mr_block + (long long)b * (p.mr_rows / 64) + 2 * m;
    const int4 u = __ldg(blk), v = __ldg(blk + 1);
    *first = max(0, min(u.x, v.x));
    *last = (long long)min(lk, max(u.y, v.y)) - 1;
}
// The visible keys [*kmin, *kmax] of query row qi (none if kmax < kmin).
__device__ __forceinline__ void row_range(const BwdParams &p, int b, int qi, int lq, int lk, int *kmin, int *kmax) {
    *kmin = 0;
    *kmax = -1;
    if (qi < lq) {
        const int2 r = __ldg(p.mr_row + (long long)b * p.mr_rows + qi);
        *kmin = max(r.x, 0);
        *kmax = min(r.y, lk) - 1;
    }
}

}  // namespace fa
