// fa_kvwork.cuh -- what the attention kernels over a paged cache share, whatever
// their values are held in: how the work is counted and split over the workers
// (warps), and the fragments' small operations.  A lane of a worker: r8 = lane / 4,
// q4 = lane % 4.
#pragma once

#include "fa_device.cuh"
#include "fa_kvcache.h"
#include "fa_params.h"

namespace fa {
namespace {

constexpr int kTile = 64;   // keys per step
constexpr float kLazy = 8.f;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// four e4m3 bytes -> two f16 pairs (exact), low bytes first
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// two fp32 -> two e4m3 bytes, lo in the low byte (nearest even, saturating)
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// magnitudes of two 16-bit floats compare as their bits do
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

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
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
// Work is shared out in half tiles: a segment of nt tiles counts 2 nt + kOpen, for
// opening and closing it takes time as well.  A border x half tiles into a segment
// lies before tile kv_border(x); tile t belongs to the worker that holds half tile
// 2 t + kOpen.  (8-bit, shared out by tiles alone: workers with short sequences took
// 145 k cycles where the mean was 118 k.)
template <int kOpen> __device__ __forceinline__ int kv_units(int nt) { return nt > 0 ? 2 * nt + kOpen : 0; }
template <int kOpen> __device__ __forceinline__ int kv_border(int x) { return max(x - kOpen + 1, 0) / 2; }

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
template <int W, int D, int kOpen>
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
            x = kv_units<kOpen>(kv_tiles(p, n));
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
template <int kOpen>
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
    const int in = w - (lo > 0 ? s_pre[lo - 1] : 0) * per_tile, units = kv_units<kOpen>(c.t1 - c.t0);
    const int seg = in / units;
    c.hk = seg / p.groups;
    c.rg = seg - c.hk * p.groups;
    c.t = c.t0 + kv_border<kOpen>(in - seg * units) - 1;
    c.next(p, s_len);   // (a border behind a segment's last tile: the next one's first)
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : l == 0.f ? -INFINITY : l;
}
// What turns a row's accumulator into its output: 2^(R - m) / l (0 for a row
// that saw nothing).
__device__ __forceinline__ float out_factor(float R, float m, float l) { return l == 0.f ? 0.f : ex2(R - m) / l; }

// Programmatic dependent launch: the second kernel's CTAs may be set up while
// the first still runs, and wait here for its results.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace
}  // namespace fa
