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

__global__ void __launch_bounds__(kTabThreads) range_tables_kernel(RangeTables t) {
    __shared__ int sh[kTabThreads / 32];
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
        t.key[(long long)b * nn + n] = key_blocks(first, last, nm, n);
    }
}

// ------------------------------------------------------- short sequences
// Up to kShort rows: one CTA per sequence holds everything, eight rows per
// thread, so one launch does both steps and no document end is searched for.
// Measured (2 launches -> this): @SHORT@
constexpr int kShortThreads = 1024, kShortPer = 8, kShort = kShortThreads * kShortPer;
constexpr int kShortBlocks = kShort / 64;

__global__ void __launch_bounds__(kShortThreads) short_ranges_kernel(MaskArgs a, RangeTables t) {
    __shared__ int sh[kShortThreads / 32];
    __shared__ int rev[kShortThreads];
    __shared__ int s_first[kShortBlocks], s_last[kShortBlocks];
    const int b = blockIdx.x, S = a.S, tid = threadIdx.x, i0 = tid * kShortPer;
    const int *doc = a.doc ? a.doc + (long long)b * S : nullptr;
    int start[kShortPer], end[kShortPer];
    bool live[kShortPer];
    if (doc) {
        int id[kShortPer + 2];
#pragma unroll
        for (int k = 0; k < kShortPer + 2; ++k) {
            const int i = i0 - 1 + k;
            id[k] = (i >= 0 && i < S) ? __ldg(doc + i) : 0;
        }
        int last = -1, next = -1, all;   // as in row_ranges_kernel
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
        // inclusive scans; a thread takes its neighbour's value
        rev[tid] = block_scan_incl(last, true, 0, sh, &all);
        __syncthreads();
        const int carry = tid > 0 ? rev[tid - 1] : 0;
        __syncthreads();
        rev[kShortThreads - 1 - tid] = next;
        __syncthreads();
        const int mirrored = rev[tid];
        const int scan = block_scan_incl(mirrored, true, 0, sh, &all);
        rev[tid] = scan;   // every thread has read its mirrored value (the scan's barriers)
        __syncthreads();
        const int carry_end = tid < kShortThreads - 1 ? rev[kShortThreads - 2 - tid] : 0;
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
    if ((tid & 7) == 0) {
        const int m = tid / 8;   // of kShortBlocks
        if (m < nm) t.block[(long long)b * nm + m] = make_int4(min_lo, max_hi, max_lo, min_hi);
        const bool some = m < nm && max_hi > min_lo;
        s_first[m] = some ? min_lo / kBlockN : 0x7fffffff;
        s_last[m] = some ? (max_hi - 1) / kBlockN : -1;
    }
    // suffix minimum of first, prefix maximum of last, in log steps
    for (int o = 1; o < kShortBlocks; o <<= 1) {
        __syncthreads();
        int f = 0, l = 0;
        if (tid < kShortBlocks) {
            f = tid + o < kShortBlocks ? min(s_first[tid], s_first[tid + o]) : s_first[tid];
            l = tid >= o ? max(s_last[tid], s_last[tid - o]) : s_last[tid];
        }
        __syncthreads();
        if (tid < kShortBlocks) {
            s_first[tid] = f;
            s_last[tid] = l;
        }
    }
    __syncthreads();
    if (tid < nm) t.first[(long long)b * nm + tid] = s_first[tid];
    if (tid < nn) {
        const int2 r2 = key_blocks(s_first, s_last, nm, tid);
        t.key[(long long)b * nn + tid] = r2;
    }
}

}  // namespace

cudaError_t launch_mask_ranges(const int *doc, const int *prefix, int prefix_per_token, int B, int S, int wl,
                               int wr, const RangeTables &t, cudaStream_t stream) {
    MaskArgs a{doc, prefix, prefix_per_token ? S : 1, prefix_per_token ? 1 : 0, B, S, wl, wr};
    if (S <= kShort) {
        short_ranges_kernel<<<(unsigned)B, kShortThreads, 0, stream>>>(a, t);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)((t.rows + kTile - 1) / kTile), (unsigned)B);
    row_ranges_kernel<<<grid, kThreads, 0, stream>>>(a, t);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    range_tables_kernel<<<(unsigned)B, kTabThreads, 0, stream>>>(t);
    return cudaGetLastError();
}

}  // namespace fa
