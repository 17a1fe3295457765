// fa_ranges.cu -- the visible keys of every query row of a self-attention
// problem with documents, prefixes and windows, as intervals, and the tables
// by which the attention kernels skip what no row sees.
//
// Row i of a sequence of S tokens sees the keys [lo_i, hi_i) with
//   s, e  first and past-the-end position of i's document (a run of equal ids;
//         without ids the whole sequence),
//   lo = max(s, i - window_left),  hi = min(e, i + window_right + 1),
//   hi = max(hi, min(e, s + prefix length of the document)) with a prefix,
// and none if its document id is negative.  Every such mask is an interval per
// row, so an attention kernel needs two compares per element of an edge tile
// and no [S, S] tensor.
//
// What bounds it: 4 bytes read and 8 written per row, so a few launches'
// latency at every size in use.  Rows are independent apart from their
// document's two ends: a CTA of 1024 rows finds those of its own rows by a
// block scan and searches outwards only for the documents that cross its
// edges, 4096 ids per step, so no pass over the whole sequence is serial.
#include "fa_device.cuh"
#include "fa_ranges.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                       // rows per thread
constexpr int kTile = kThreads * kPer;        // rows per CTA
constexpr int kReach = 16;                    // ids per thread and search step
static_assert(kTile <= 4096 && kThreads * kReach <= 4096, "kMaxRangeSeq leaves two such steps");

struct MaskArgs {
    const int *doc;        // [B, S], null: one document per sequence
    const int *prefix;     // null: none
    int prefix_row, prefix_tok;   // strides of prefix: entry b * row + s * tok
    int B, S, wl, wr;      // wl / wr < 0: unbounded
};

// Maximum over the block; every thread gets it.
__device__ __forceinline__ int block_max(int v, int *sh) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    int r = sh[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) r = max(r, sh[i]);
    return r;
}

// Inclusive running maximum over the block's threads in thread order
// (exclusive value returned).
__device__ __forceinline__ int block_scan_max_excl(int v, int *sh, int first) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = max(x, y);
    }
    __syncthreads();
    if (lane == 31) sh[w] = x;
    __syncthreads();
    int r = first;
    for (int i = 0; i < w; ++i) r = max(r, sh[i]);
    const int up = __shfl_up_sync(0xffffffffu, x, 1);
    return lane > 0 ? max(r, up) : r;
}

// The keys [x, y) row i of the document [start, end) sees.
__device__ __forceinline__ int2 row_interval(const MaskArgs &a, int b, int i, int start, int end) {
    int lo = start, hi = end;
    if (a.wl >= 0) lo = max(lo, i - min(a.wl, i));
    if (a.wr >= 0) hi = min(hi, i + 1 + min(a.wr, a.S - 1 - i));
    if (a.prefix) {
        const int n = __ldg(a.prefix + (long long)b * a.prefix_row + (long long)start * a.prefix_tok);
        hi = max(hi, start + min(max(n, 0), end - start));
    }
    return make_int2(lo, hi);
}

__global__ void __launch_bounds__(kThreads) row_ranges_kernel(MaskArgs a, RangeTables t) {
    __shared__ int sh[kThreads / 32];
    const int b = blockIdx.y, base = blockIdx.x * kTile, S = a.S;
    const int i0 = base + threadIdx.x * kPer;
    const int *doc = a.doc ? a.doc + (long long)b * S : nullptr;
    int start[kPer], end[kPer];
    bool live[kPer];
    if (doc) {
        // id of the row before, of the thread's rows and of the row behind
        int id[kPer + 2];
#pragma unroll
        for (int k = 0; k < kPer + 2; ++k) {
            const int i = i0 - 1 + k;
            id[k] = (i >= 0 && i < S) ? __ldg(doc + i) : 0;
        }
        // start: the last position <= i where a document begins.  Begins of the
        // thread's rows, then a running maximum over the block; a document
        // begun before the tile is looked for backwards.
        int last = -1;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = i0 + k;
            if (i < S && (i == 0 || id[k + 1] != id[k])) last = i;
            start[k] = last;
        }
        int before = 0;   // begin of the document that holds the tile's first row
        for (int top = base; top > 0; top -= kThreads * kReach) {
            int found = -1;
#pragma unroll 4
            for (int k = 0; k < kReach; ++k) {
                const int i = top - (k * kThreads + (int)threadIdx.x);
                if (i > 0 && i < S && __ldg(doc + i) != __ldg(doc + i - 1)) found = max(found, i);
            }
            found = block_max(found, sh);
            if (found >= 0) { before = found; break; }
        }
        const int carry = block_scan_max_excl(last, sh, before);
#pragma unroll
        for (int k = 0; k < kPer; ++k) start[k] = start[k] >= 0 ? start[k] : carry;
        // end: the first position > i where a document begins (or S), the same
        // from the other side: positions mirrored, so that the minimum to the
        // right is a running maximum in reversed thread order
        int next = -1;   // S - position: larger is nearer; -1: none
#pragma unroll
        for (int k = kPer - 1; k >= 0; --k) {
            const int i = i0 + k + 1;   // does a document begin behind row i0 + k?
            if (i < S && id[k + 2] != id[k + 1]) next = S - i;
            else if (i == S) next = 0;
            end[k] = next;
        }
        int behind = 0;
        for (int from = base + kTile; from < S; from += kThreads * kReach) {
            int found = -1;
#pragma unroll 4
            for (int k = 0; k < kReach; ++k) {
                const int i = from + k * kThreads + (int)threadIdx.x;
                if (i < S && __ldg(doc + i) != __ldg(doc + i - 1)) found = max(found, S - i);
            }
            found = block_max(found, sh);
            if (found >= 0) { behind = found; break; }
        }
        // reversed thread order: exchange through shared memory, scan, back
        __shared__ int rev[kThreads];
        __syncthreads();
        rev[kThreads - 1 - threadIdx.x] = next;
        __syncthreads();
        const int mine = rev[threadIdx.x];
        const int rc = block_scan_max_excl(mine, sh, behind);
        __syncthreads();
        rev[kThreads - 1 - threadIdx.x] = rc;
        __syncthreads();
        const int carry_end = rev[threadIdx.x];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            end[k] = S - (end[k] >= 0 ? end[k] : carry_end);
            live[k] = i0 + k < S && id[k + 1] >= 0;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            start[k] = 0;
            end[k] = S;
            live[k] = i0 + k < S;
        }
    }
    // the rows' intervals, and the bounds of the 64-row block (16 threads)
    int2 r[kPer];
    int min_lo = 0x7fffffff, max_hi = 0, max_lo = 0, min_hi = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = i0 + k;
        r[k] = make_int2(0, 0);
        if (live[k]) {
            r[k] = row_interval(a, b, i, start[k], end[k]);
            const int lo = r[k].x, hi = r[k].y;
            min_lo = min(min_lo, lo);
            max_hi = max(max_hi, hi);
        }
        if (i < S) {
            max_lo = max(max_lo, r[k].x);
            min_hi = min(min_hi, r[k].y);
        }
    }
    if (i0 < t.rows) {   // t.rows is a multiple of 128: whole threads
        int4 *dst = reinterpret_cast<int4 *>(t.row + (long long)b * t.rows + i0);
        dst[0] = make_int4(r[0].x, r[0].y, r[1].x, r[1].y);
        dst[1] = make_int4(r[2].x, r[2].y, r[3].x, r[3].y);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        min_lo = min(min_lo, __shfl_xor_sync(0xffffffffu, min_lo, o));
        max_hi = max(max_hi, __shfl_xor_sync(0xffffffffu, max_hi, o));
        max_lo = max(max_lo, __shfl_xor_sync(0xffffffffu, max_lo, o));
        min_hi = min(min_hi, __shfl_xor_sync(0xffffffffu, min_hi, o));
    }
    if ((threadIdx.x & 15) == 0 && i0 < t.rows)
        t.block[(long long)b * (t.rows / 64) + i0 / 64] = make_int4(min_lo, max_hi, max_lo, min_hi);
}

// ------------------------------------------------------------------ tables
// For the 64-row blocks m of a sequence and its 128-key blocks n: a row block
// that sees keys touches the key blocks [f_m, l_m].  The row blocks a unit of
// key block n works on are [a_n, b_n],
//   b_n = max{m : f_m' <= n for some m' >= m} = the last m whose suffix minimum
//         of f is <= n,
//   a_n = the first m whose prefix maximum of l is >= n,
// which for documents, prefixes and windows (f and l rise with m) is exactly
// the blocks that touch n, and for any intervals holds them all.  Both ends
// rise with n, so the key blocks that work on m are contiguous and start at
// first[m], the suffix minimum of f: the deterministic order counts from it.
constexpr int kTabThreads = 1024;

__device__ __forceinline__ int scan_op(int x, int y, bool mx) { return mx ? max(x, y) : min(x, y); }

// Inclusive scan (maximum or minimum) over the block's threads in thread
// order, `carry` before the first; *total gets the whole block's value.
__device__ __forceinline__ int block_scan_incl(int v, bool mx, int carry, int *sh, int *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = scan_op(x, y, mx);
    }
    __syncthreads();
    if (lane == 31) sh[w] = x;
    __syncthreads();
    int r = carry, all = carry;
    for (int i = 0; i < kTabThreads / 32; ++i) {
        if (i < w) r = scan_op(r, sh[i], mx);
        all = scan_op(all, sh[i], mx);
    }
    *total = all;
    return scan_op(r, x, mx);
}

// The row blocks [x, y) a unit of key block n works on, from the suffix minimum
// `first` and the prefix maximum `last`.
__device__ __forceinline__ int2 key_blocks(const int *first, const int *last, int nm, int n) {
    int lo = 0, hi = nm;                    // number of m with first[m] <= n
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= n) lo = mid + 1;
        else hi = mid;
    }
    const int end = lo;
    lo = 0, hi = nm;                        // first m with last[m] >= n
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (last[mid] >= n) hi = mid;
        else lo = mid + 1;
    }
    return lo < end ? make_int2(lo, end) : make_int2(0, 0);
}

// The row blocks of [r.x, r.y) whose rows all see the whole key block n, as one
// run [x, y): the first there is (documents, prefixes and windows leave one).  A
// whole warp, 32 blocks at a time.
__device__ __forceinline__ int2 open_run(const int4 *block, int n, int2 r) {
    const int lane = threadIdx.x & 31, lo = n * kBlockN, hi = lo + kBlockN;
    int x = -1;
    for (int m0 = r.x; m0 < r.y; m0 += 32) {
        const int m = m0 + lane;
        bool open = false;
        if (m < r.y) {
            const int4 e = block[m];
            open = e.z <= lo && e.w >= hi;
        }
        uint32_t bits = __ballot_sync(0xffffffffu, open);
        if (x < 0) {
            if (bits == 0u) continue;
            const int at = __ffs((int)bits) - 1;
            x = m0 + at;
            bits |= (1u << at) - 1u;   // looked for: the first that is shut
        }
        if (bits != 0xffffffffu) return make_int2(x, m0 + __ffs((int)~bits) - 1);
    }
    return x < 0 ? make_int2(0, 0) : make_int2(x, r.y);
}

// Longest first: the order in which the backward takes a sequence's key blocks
// (documents leave units of very different lengths, and a long one begun last
// keeps the rest waiting).  The rank of a block is counted; past kRanked
// blocks there are so many units that the order does not matter.
constexpr int kRanked = 512;
__device__ __forceinline__ int rank_of(const int2 *key, int nn, int n, int2 mine) {
    const int len = mine.y - mine.x;
    int r = 0;
#pragma unroll 4
    for (int i = 0; i < nn; ++i) {
        const int l = key[i].y - key[i].x;
        r += l > len || (l == len && i < n);
    }
    return r;
}

__global__ void __launch_bounds__(kTabThreads) range_tables_kernel(RangeTables t) {
    __shared__ int sh[kTabThreads / 32];
    __shared__ int2 s_key[kRanked];
    const int b = blockIdx.x, nm = t.rows / 64, nn = t.rows / kBlockN, tid = threadIdx.x;
    const int4 *blk = t.block + (long long)b * nm;
    int *first = t.first + (long long)b * nm, *last = t.last + (long long)b * nm;
    int carry = -1;
    for (int m0 = 0; m0 < nm; m0 += kTabThreads) {
        const int m = m0 + tid;
        int l = -1;
        if (m < nm) {
            const int4 e = blk[m];
            if (e.y > e.x) l = (e.y - 1) / kBlockN;
        }
        const int v = block_scan_incl(l, true, carry, sh, &carry);
        if (m < nm) last[m] = v;
    }
    carry = 0x7fffffff;
    for (int m0 = 0; m0 < nm; m0 += kTabThreads) {
        const int m = nm - 1 - (m0 + tid);   // from the end
        int f = 0x7fffffff;
        if (m >= 0) {
            const int4 e = blk[m];
            if (e.y > e.x) f = e.x / kBlockN;
        }
        const int v = block_scan_incl(f, false, carry, sh, &carry);
        if (m >= 0) first[m] = v;
    }
    __syncthreads();   // the block's own writes, read back below
    for (int n = tid; n < nn; n += kTabThreads) {
        const int2 r = key_blocks(first, last, nm, n);
        t.key[(long long)b * nn + n] = make_int4(r.x, r.y, 0, 0);
        if (nn <= kRanked) s_key[n] = r;
    }
    __syncthreads();
    for (int n = tid; n < nn; n += kTabThreads)
        t.order[(long long)b * nn + (nn <= kRanked ? rank_of(s_key, nn, n, s_key[n]) : n)] = n;
}

// The runs of whole row blocks, a warp per key block.
__global__ void __launch_bounds__(256) range_runs_kernel(RangeTables t) {
    const int b = blockIdx.y, nm = t.rows / 64, nn = t.rows / kBlockN;
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= nn) return;
    int4 *key = t.key + (long long)b * nn + n;
    const int4 r = *key;
    const int2 run = open_run(t.block + (long long)b * nm, n, make_int2(r.x, r.y));
    if ((threadIdx.x & 31) == 0) *key = make_int4(r.x, r.y, run.x, run.y);
}

// ------------------------------------------------------- short sequences
// Up to kShort rows: one CTA per sequence, eight rows per thread, so one launch
// does both steps, no document end is searched for, and the tables are one
// warp's work.
constexpr int kShortThreads = 1024, kShortPer = 8, kShort = kShortThreads * kShortPer;
constexpr int kShortBlocks = kShort / 64;

// Exclusive running maximum over the block's threads, `first` before the first.
__device__ __forceinline__ int short_scan_excl(int v, int first, int *sh) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = max(x, y);
    }
    if (lane == 31) sh[w] = x;
    __syncthreads();
    const int before = __reduce_max_sync(0xffffffffu, lane < w ? sh[lane] : first);
    const int up = __shfl_up_sync(0xffffffffu, x, 1);
    return lane > 0 ? max(before, up) : before;
}
// The same from the other end: what lies behind a thread.
__device__ __forceinline__ int short_scan_excl_back(int v, int first, int *sh) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, x, o);
        if (lane + o < 32) x = max(x, y);
    }
    if (lane == 0) sh[w] = x;
    __syncthreads();
    const int behind = __reduce_max_sync(0xffffffffu, lane > w && lane < nw ? sh[lane] : first);
    const int dn = __shfl_down_sync(0xffffffffu, x, 1);
    return lane < 31 ? max(behind, dn) : behind;
}

__global__ void __launch_bounds__(kShortThreads) short_ranges_kernel(MaskArgs a, RangeTables t) {
    __shared__ int sh[2][kShortThreads / 32];
    __shared__ int s_first[kShortBlocks], s_last[kShortBlocks];
    __shared__ int2 s_key[kShortBlocks / 2];
    __shared__ int4 s_block[kShortBlocks];
    const int b = blockIdx.x, S = a.S, tid = threadIdx.x, i0 = tid * kShortPer;
    const int *doc = a.doc ? a.doc + (long long)b * S : nullptr;
    int start[kShortPer], end[kShortPer];
    bool live[kShortPer];
    if (doc) {
        int id[kShortPer + 2];
        if ((S & 3) == 0 && (reinterpret_cast<uintptr_t>(doc) & 15u) == 0) {
            // 16-byte loads; the neighbours' ids come from the neighbour lanes
#pragma unroll
            for (int k = 0; k < kShortPer; k += 4) {
                const int4 v = i0 + k < S ? __ldg(reinterpret_cast<const int4 *>(doc + i0 + k)) : make_int4(0, 0, 0, 0);
                id[k + 1] = v.x, id[k + 2] = v.y, id[k + 3] = v.z, id[k + 4] = v.w;
            }
            id[0] = __shfl_up_sync(0xffffffffu, id[kShortPer], 1);
            id[kShortPer + 1] = __shfl_down_sync(0xffffffffu, id[1], 1);
            if ((tid & 31) == 0) id[0] = (i0 > 0 && i0 <= S) ? __ldg(doc + i0 - 1) : 0;
            if ((tid & 31) == 31) id[kShortPer + 1] = i0 + kShortPer < S ? __ldg(doc + i0 + kShortPer) : 0;
        } else {
#pragma unroll
            for (int k = 0; k < kShortPer + 2; ++k) {
                const int i = i0 - 1 + k;
                id[k] = (i >= 0 && i < S) ? __ldg(doc + i) : 0;
            }
        }
        int last = -1, next = -1;   // as in row_ranges_kernel
#pragma unroll
        for (int k = 0; k < kShortPer; ++k) {
            const int i = i0 + k;
            if (i < S && (i == 0 || id[k + 1] != id[k])) last = i;
            start[k] = last;
        }
#pragma unroll
        for (int k = kShortPer - 1; k >= 0; --k) {
            const int i = i0 + k + 1;
            if (i < S && id[k + 2] != id[k + 1]) next = S - i;
            else if (i == S) next = 0;
            end[k] = next;
        }
        const int carry = short_scan_excl(last, 0, sh[0]);
        const int carry_end = short_scan_excl_back(next, 0, sh[1]);
#pragma unroll
        for (int k = 0; k < kShortPer; ++k) {
            start[k] = start[k] >= 0 ? start[k] : carry;
            end[k] = S - (end[k] >= 0 ? end[k] : carry_end);
            live[k] = i0 + k < S && id[k + 1] >= 0;
        }
    } else {
#pragma unroll
        for (int k = 0; k < kShortPer; ++k) {
            start[k] = 0;
            end[k] = S;
            live[k] = i0 + k < S;
        }
    }
    int2 r[kShortPer];
    int min_lo = 0x7fffffff, max_hi = 0, max_lo = 0, min_hi = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kShortPer; ++k) {
        const int i = i0 + k;
        r[k] = make_int2(0, 0);
        if (live[k]) {
            r[k] = row_interval(a, b, i, start[k], end[k]);
            min_lo = min(min_lo, r[k].x);
            max_hi = max(max_hi, r[k].y);
        }
        if (i < S) {
            max_lo = max(max_lo, r[k].x);
            min_hi = min(min_hi, r[k].y);
        }
    }
    if (i0 < t.rows) {
        int4 *dst = reinterpret_cast<int4 *>(t.row + (long long)b * t.rows + i0);
#pragma unroll
        for (int k = 0; k < kShortPer / 2; ++k)
            dst[k] = make_int4(r[2 * k].x, r[2 * k].y, r[2 * k + 1].x, r[2 * k + 1].y);
    }
    const int nm = t.rows / 64, nn = t.rows / kBlockN;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {   // 64 rows: eight threads
        min_lo = min(min_lo, __shfl_xor_sync(0xffffffffu, min_lo, o));
        max_hi = max(max_hi, __shfl_xor_sync(0xffffffffu, max_hi, o));
        max_lo = max(max_lo, __shfl_xor_sync(0xffffffffu, max_lo, o));
        min_hi = min(min_hi, __shfl_xor_sync(0xffffffffu, min_hi, o));
    }
    if ((tid & 7) == 0 && tid / 8 < nm) {
        const int m = tid / 8;
        s_block[m] = make_int4(min_lo, max_hi, max_lo, min_hi);
        t.block[(long long)b * nm + m] = s_block[m];
        s_first[m] = max_hi > min_lo ? min_lo / kBlockN : 0x7fffffff;
        s_last[m] = max_hi > min_lo ? (max_hi - 1) / kBlockN : -1;
    }
    __syncthreads();
    if (tid < 32) {
        // suffix minimum of first, prefix maximum of last: four blocks per lane
        constexpr int PER = kShortBlocks / 32;
        int f[PER], l[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int m = tid * PER + k;
            f[k] = m < nm ? s_first[m] : 0x7fffffff;
            l[k] = m < nm ? s_last[m] : -1;
        }
#pragma unroll
        for (int k = 1; k < PER; ++k) {
            l[k] = max(l[k], l[k - 1]);
            f[PER - 1 - k] = min(f[PER - 1 - k], f[PER - k]);
        }
        int lt = l[PER - 1], ft = f[0];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, lt, o), z = __shfl_down_sync(0xffffffffu, ft, o);
            if (tid >= o) lt = max(lt, y);
            if (tid + o < 32) ft = min(ft, z);
        }
        int lb = __shfl_up_sync(0xffffffffu, lt, 1), fb = __shfl_down_sync(0xffffffffu, ft, 1);
        if (tid == 0) lb = -1;
        if (tid == 31) fb = 0x7fffffff;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int m = tid * PER + k;
            if (m < nm) {
                s_first[m] = min(f[k], fb);
                s_last[m] = max(l[k], lb);
                t.first[(long long)b * nm + m] = s_first[m];
            }
        }
    }
    __syncthreads();
    for (int n = tid; n < nn; n += blockDim.x) s_key[n] = key_blocks(s_first, s_last, nm, n);
    __syncthreads();
    for (int n = tid >> 5; n < nn; n += blockDim.x >> 5) {   // a warp per key block
        const int2 r = s_key[n], run = open_run(s_block, n, r);
        if ((tid & 31) == 0) t.key[(long long)b * nn + n] = make_int4(r.x, r.y, run.x, run.y);
    }
    for (int n = tid; n < nn; n += blockDim.x) t.order[(long long)b * nn + rank_of(s_key, nn, n, s_key[n])] = n;
}

}  // namespace

cudaError_t launch_mask_ranges(const int *doc, const int *prefix, int prefix_per_token, int B, int S, int wl,
                               int wr, const RangeTables &t, cudaStream_t stream) {
    MaskArgs a{doc, prefix, prefix_per_token ? S : 1, prefix_per_token ? 1 : 0, B, S, wl, wr};
    if (S <= kShort) {
        const int threads = (t.rows / kShortPer + 31) / 32 * 32;
        short_ranges_kernel<<<(unsigned)B, threads, 0, stream>>>(a, t);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)((t.rows + kTile - 1) / kTile), (unsigned)B);
    row_ranges_kernel<<<grid, kThreads, 0, stream>>>(a, t);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    range_tables_kernel<<<(unsigned)B, kTabThreads, 0, stream>>>(t);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    range_runs_kernel<<<dim3((unsigned)((t.rows / kBlockN + 7) / 8), (unsigned)B), 256, 0, stream>>>(t);
    return cudaGetLastError();
}

}  // namespace fa
