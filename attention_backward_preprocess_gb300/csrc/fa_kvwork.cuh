// fa_kvwork.cuh -- what the attention kernels over a paged cache share, whatever
// their values are held in: how the work is counted and split over the workers
// (warps), and how the pieces of a segment that several of them held are joined.
//
// Fragments.  A worker's accumulator of 16-dim part dm holds two dims of two rows
// a lane (r8 = lane / 4, q4 = lane % 4): rows 2 q4, + 1 of its 8, and dims
// 16 dm + r8, + 8 (kPairs false) or two neighbours, 32 (dm / 2) + 4 r8 +
// 2 (dm % 2), + 1 (kPairs true).
#pragma once

#include "fa_device.cuh"
#include "fa_kvcache.h"
#include "fa_params.h"

namespace fa {
namespace {

constexpr int kTile = 64;   // keys per step
constexpr float kLazy = 8.f;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 2-D tiled load (bytes along a row, row) completing on an mbarrier.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// an 8x8 block of 16-bit values transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// over the lanes of equal lane % 4 (the keys of a row pair)
__device__ __forceinline__ float keys_max(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float keys_sum(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// First key any of the sequence's queries sees.
__device__ __forceinline__ int kv_first(const KvAttnParams &p, int n) {
    return p.window < 0 ? 0 : max(0, n - p.Sq - min(p.window, n));
}
__device__ __forceinline__ int kv_tiles(const KvAttnParams &p, int n) {
    return (n + kTile - 1) / kTile - kv_first(p, n) / kTile;
}
// Work is shared out in half tiles: a segment of nt tiles counts 2 nt + 2, for
// opening and closing it takes about as long as a tile.  A border x half tiles
// into a segment lies before tile kv_border(x); tile t belongs to the worker
// that holds half tile 2 t + 2.  (Shared out by tiles alone, workers with short
// sequences took 145 k cycles where the mean was 118 k.)
__device__ __forceinline__ int kv_units(int nt) { return nt > 0 ? 2 * nt + 2 : 0; }
__device__ __forceinline__ int kv_border(int x) { return max(x - 1, 0) / 2; }

// A worker's place in the work: tile t of [t0, t1) of sequence b, kv head hk and
// row group rg.
struct Cursor {
    int b, hk, rg, t, t0, t1, n, lo;
    __device__ __forceinline__ void open(const KvAttnParams &p, const int *lens) {   // sequence b
        n = lens[b];
        lo = kv_first(p, n);
        t0 = lo / kTile;
        t1 = (n + kTile - 1) / kTile;
    }
    __device__ __forceinline__ void next(const KvAttnParams &p, const int *lens) {
        if (++t < t1) return;
        t = 0;   // (the end of all work: 0)
        if (++rg == p.groups) {
            rg = 0;
            if (++hk == p.c.Hkv) {
                hk = 0;
                do {
                    if (++b >= p.B) return;   // the end of all work
                    open(p, lens);
                } while (t1 <= t0);
            }
        }
        t = t0;
    }
};

// The work: half tiles of one head and row group of sequences 0 .. b into s_pre,
// their tokens into s_len (0 where the length is outside the table), and the sum
// back, to every thread of the CTA of W warps.  Rows of sequences without a key
// are written here.
template <int W, int D>
__device__ __forceinline__ int kv_count(const KvAttnParams &p, int *s_pre, int *s_len, int *s_warp, int warp, int lane) {
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += W * 32) {
        const int b = b0 + threadIdx.x;
        int x = 0;
        if (b < p.B) {
            int n = __ldg(p.len + b);
            if (n < 0 || (long long)n > (long long)p.c.max_pages * p.c.page) {
                if (blockIdx.x == 0) atomicOr(p.c.err, kErrBadLength);
                n = 0;
            }
            x = kv_units(kv_tiles(p, n));
            s_len[b] = n;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        int add = carry, all = carry;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int v = s_warp[i];
            if (i < warp) add += v;
            all += v;
        }
        if (b < p.B) s_pre[b] = x + add;
        carry = all;
        __syncthreads();
    }
    // sequences without a key: zeros
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (s_pre[b] - (b > 0 ? s_pre[b - 1] : 0) > 0) continue;
        uint32_t *o = reinterpret_cast<uint32_t *>(p.o) + (long long)b * p.Sq * p.Hq * (D / 2);
        for (int i = threadIdx.x; i < p.Sq * p.Hq * (D / 2); i += W * 32) o[i] = 0u;
        if (p.lse)
            for (int i = threadIdx.x; i < p.Sq * p.Hq; i += W * 32) p.lse[(long long)b * p.Sq * p.Hq + i] = -INFINITY;
    }
    return carry;
}

// A worker's share [w0, w1) of the half tiles of all heads and row groups: total /
// N each, one more for the first total % N.
struct KvShare {
    int wid, N, share, more, w0, w1;
    // (total: the host keeps it below 2^31.)  A worker holds at least two tiles'
    // worth, so that few pieces are made of little work; from N on they hold none.
    __device__ __forceinline__ KvShare(const KvAttnParams &p, int wid_, int total) {
        wid = wid_;
        N = min(p.workers, max(total / 4, 1));
        share = total / N;
        more = total - share * N;
        w0 = wid * share + min(wid, more);
        w1 = w0 + share + (wid < more ? 1 : 0);
    }
    __device__ __forceinline__ int worker_of(int w) const {
        const int head = (share + 1) * more;
        return w < head ? w / (share + 1) : more + (w - head) / share;
    }
};

// The tile behind a border (past the last one: b == B).
__device__ __forceinline__ void kv_place(const KvAttnParams &p, const int *s_pre, const int *s_len, int per_tile, int w,
                                         Cursor &c) {
    const int u = w / per_tile;   // the border over the sequences, if every half tile came once
    int lo = 0, hi = p.B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid] > u) hi = mid;
        else lo = mid + 1;
    }
    c.b = lo;
    c.hk = c.rg = c.t = 0;
    if (lo == p.B) return;
    c.open(p, s_len);
    const int in = w - (lo > 0 ? s_pre[lo - 1] : 0) * per_tile, units = kv_units(c.t1 - c.t0);
    const int seg = in / units;
    c.hk = seg / p.groups;
    c.rg = seg - c.hk * p.groups;
    c.t = c.t0 + kv_border(in - seg * units) - 1;
    c.next(p, s_len);   // (a border behind a segment's last tile: the next one's first)
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : l == 0.f ? -INFINITY : l;
}
// What turns a row's accumulator into its output: 2^(R - m) / l (0 for a row
// that saw nothing).
__device__ __forceinline__ float out_factor(float R, float m, float l) { return l == 0.f ? 0.f : ex2(R - m) / l; }

// Output rows of a piece: acc is one 16-dim part dm of them, already scaled.
template <int D, typename T, bool kPairs>
__device__ __forceinline__ void store_rows(const KvAttnParams &p, int b, int hk, int row0, int lane,
                                           float (&acc)[4], int dm) {
    const int r8 = lane >> 2, q4 = lane & 3;
    auto at = [&](int row) __attribute__((always_inline)) -> T * {
        const int i = row / p.G, hq = hk * p.G + row % p.G;
        return reinterpret_cast<T *>(p.o) + (((long long)b * p.Sq + i) * p.Hq + hq) * D;
    };
    if (kPairs) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (row0 + 2 * q4 + e < p.Sq * p.G)
                *reinterpret_cast<uint32_t *>(at(row0 + 2 * q4 + e) + 32 * (dm >> 1) + 4 * r8 + 2 * (dm & 1)) =
                    Cvt<T>::pack(acc[e], acc[2 + e]);
        return;
    }
    // two 8x8 blocks (dims x rows), transposed: lane gets row r8, dims 2 q4, + 1
    const uint32_t lo = transpose8(Cvt<T>::pack(acc[0], acc[1]));
    const uint32_t hi = transpose8(Cvt<T>::pack(acc[2], acc[3]));
    if (row0 + r8 < p.Sq * p.G) {
        T *dst = at(row0 + r8) + 16 * dm + 2 * q4;
        *reinterpret_cast<uint32_t *>(dst) = lo;
        *reinterpret_cast<uint32_t *>(dst + 8) = hi;
    }
}

// Rows 2 q4 + e of one row block, one 16-dim part, over several pieces.
struct Joined {
    float4 v;
    float m[2], l[2], r[2];
};
__device__ __forceinline__ void joined_zero(Joined &x) {
    x.v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 2; ++e) x.m[e] = x.r[e] = -INFINITY, x.l[e] = 0.f;
}
// x += a piece's values and (m, l, R) of the two rows, against the larger maxima
__device__ __forceinline__ void joined_add(Joined &x, float4 v, const float (&m)[2], const float (&l)[2],
                                           const float (&r)[2]) {
    float g[2], h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(x.m[e], m[e]), rn = fmaxf(x.r[e], r[e]);
        const float m0 = mn == -INFINITY ? 0.f : mn, r0 = rn == -INFINITY ? 0.f : rn;
        x.l[e] = x.l[e] * ex2(x.m[e] - m0) + l[e] * ex2(m[e] - m0);
        g[e] = ex2(x.r[e] - r0);
        h[e] = ex2(r[e] - r0);
        x.m[e] = mn;
        x.r[e] = rn;
    }
    x.v.x = fmaf(v.x, h[0], x.v.x * g[0]);
    x.v.y = fmaf(v.y, h[1], x.v.y * g[1]);
    x.v.z = fmaf(v.z, h[0], x.v.z * g[0]);
    x.v.w = fmaf(v.w, h[1], x.v.w * g[1]);
}
// Every `step`-th piece of workers from .. to (piece 1 of worker `first`, piece 0
// of the others), in order.
template <int NR, int DM>
__device__ __forceinline__ void join_pieces(const KvAttnParams &p, int from, int to, int step, int first, int nr,
                                            int dm, int row0, int lane, Joined &x) {
    constexpr int PIECE = NR * DM * 128;
    const int q4 = lane & 3;
    joined_zero(x);
#pragma unroll 4
    for (int w = from; w <= to; w += step) {
        const long long at = (long long)w * 2 + (w == first ? 1 : 0);
        const float4 v = *(reinterpret_cast<const float4 *>(p.acc + at * PIECE + nr * DM * 128) + 32 * dm + lane);
        float m[2], l[2], r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {   // rows past the last carry no statistics
            const float4 st = row0 + 2 * q4 + e < p.Sq * p.G ? p.stat[at * (NR * 8) + nr * 8 + 2 * q4 + e]
                                                             : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
            m[e] = st.x, l[e] = st.y, r[e] = st.z;
        }
        joined_add(x, v, m, l, r);
    }
}

template <int D, typename T, bool kPairs>
__device__ __forceinline__ void finish_rows(const KvAttnParams &p, const Joined &x, int b, int hk, int row0, int dm,
                                            int lane) {
    const float f0 = out_factor(x.r[0], x.m[0], x.l[0]), f1 = out_factor(x.r[1], x.m[1], x.l[1]);
    float o[4] = {x.v.x * f0, x.v.y * f1, x.v.z * f0, x.v.w * f1};
    store_rows<D, T, kPairs>(p, b, hk, row0, lane, o, dm);
    if (p.lse && dm == 0 && lane < 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = row0 + 2 * lane + e;
            if (row < p.Sq * p.G)
                p.lse[((long long)b * p.Hq + hk * p.G + row % p.G) * p.Sq + row / p.G] = lse_of(x.m[e], x.l[e]);
        }
    }
}

// Programmatic dependent launch: the second kernel's CTAs may be set up while
// the first still runs, and wait here for its results.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------------- join
// One CTA per kJoinWorkers workers and 16 dims: for each of the workers in which
// a segment ends that began before it, the segment's pieces are joined and
// finished.  A warp takes a segment of few pieces by itself; of one of many the
// kParts warps take every kParts-th piece and add their sums in order.
// Joining in the attention kernel instead (the last holder in a CTA) kept
// 17 to 20 thousand cycles of a worker's 115 for itself, most of them the first
// run through code that is used once.  Eight workers and eight warps a CTA: 67 us
// for 64 requests of 256 to 8192 tokens, 48 for two of up to 64k (calls); 16
// workers 68 and 48, 32 workers 73 and 49, four of each 65 and 52.
constexpr int kParts = 8, kJoinWorkers = 8, kFew = 8;

template <int D, int NR, typename T, bool kPairs>
__global__ void __launch_bounds__(32 * kParts) kv_join_kernel(const __grid_constant__ KvAttnParams p) {
    constexpr int DM = D / 16;
    __shared__ Joined s_x[kParts - 1][32];
    const int part = threadIdx.x / 32, lane = threadIdx.x % 32, dm = blockIdx.y;
    pdl_wait();
    const int w_lane = blockIdx.x * kJoinWorkers + lane;
    int4 mine = make_int4(-1, 0, 0, 0);
    if (lane < kJoinWorkers && w_lane < p.workers) mine = p.meta[w_lane];
    int turn = 0;
#pragma unroll 1
    for (int i = 0; i < kJoinWorkers; ++i) {
        const int seg = __shfl_sync(0xffffffffu, mine.x, i), b = __shfl_sync(0xffffffffu, mine.y, i);
        const int first = __shfl_sync(0xffffffffu, mine.z, i), ends = __shfl_sync(0xffffffffu, mine.w, i);
        const int w = blockIdx.x * kJoinWorkers + i;
        if (seg < 0 || ends == 0) continue;
        const bool few = w - first < kFew;
        if (few && turn++ % kParts != part) continue;
#pragma unroll 1
        for (int nr = 0; nr < NR; ++nr) {
            const int row0 = ((seg % p.groups) * NR + nr) * 8;
            Joined x;
            join_pieces<NR, DM>(p, few ? first : first + part, w, few ? 1 : kParts, first, nr, dm, row0, lane, x);
            if (!few) {
                if (part > 0) s_x[part - 1][lane] = x;
                __syncthreads();   // (many pieces: every warp of the CTA is here)
                if (part == 0)
#pragma unroll 1
                    for (int k = 0; k < kParts - 1; ++k) {
                        const Joined &y = s_x[k][lane];
                        joined_add(x, y.v, y.m, y.l, y.r);
                    }
                __syncthreads();
                if (part > 0) continue;
            }
            finish_rows<D, T, kPairs>(p, x, b, seg / p.groups, row0, dm, lane);
        }
    }
}

// The join behind an attention kernel on the same stream, set up while that one runs.
template <int D, int NR, typename T, bool kPairs>
cudaError_t launch_join(const KvAttnParams &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.workers + kJoinWorkers - 1) / kJoinWorkers), D / 16);
    cfg.blockDim = dim3(32 * kParts);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NR, T, kPairs>, p);
}

}  // namespace
}  // namespace fa
