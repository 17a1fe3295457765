// fa_kvcache.cu -- the 8-bit paged key / value cache: appending to it and the
// attention of a sequence's last tokens over it.
//
// Values are e4m3 with one scale per (page, kv head), a power of two 2^e with
// the smallest e for which the page's largest magnitude fits 448 * 2^e.  A
// power of two costs no precision (e4m3 is a floating type) and makes the
// division by the scale, and moving a page to a larger scale, exact but for
// values that become subnormal.
//
// K lies token by token, V dim by dim, so that in both products the 16-byte
// pieces a lane reads are contiguous along the axis the tensor core contracts.
#include <cuda_fp8.h>

#include "fa_device.cuh"
#include "fa_kvcache.h"
#include "fa_params.h"

namespace fa {
namespace {

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

// ------------------------------------------------------------------ append
// One CTA per (page a sequence's new tokens touch, kv head, K or V).  It reads
// the tokens once (into shared memory, their largest magnitude on the way),
// settles the page's scale, moves tokens the page held before to it if it
// grew, and writes the new ones.  The CTA owns the page, so bytes are merged
// without atomics.  What bounds it: 3 bytes moved per value, and for a
// decoding step the latency of one read, one reduction and one write.
constexpr int kAppendThreads = 128;

// smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), held in [-120, 120]
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, -120), 120);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 16 stored bytes moved to another scale, those from byte `n` on left alone
__device__ __forceinline__ void requantise(uint32_t (&w)[4], float ratio, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, b;
        e4m3x4_to_f16(w[i], a, b);
        const float2 x = Cvt<__half>::unpack(a), y = Cvt<__half>::unpack(b);
        const uint32_t r = f32_to_e4m3x2(x.x * ratio, x.y * ratio) | f32_to_e4m3x2(y.x * ratio, y.y * ratio) << 16;
        const int k = min(max(n - 4 * i, 0), 4);
        const uint32_t keep = k >= 4 ? 0u : 0xffffffffu << (8 * k);
        w[i] = (w[i] & keep) | (r & ~keep);
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p, int per_seq) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ float s_max[kAppendThreads / 32];
    const int ps = p.c.page, tid = threadIdx.x;
    const int b = blockIdx.x / per_seq, h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int len = p.len[b];
    const int row0 = p.cu ? p.cu[b] : b * p.max_new;
    const int n = p.cu ? p.cu[b + 1] - row0 : p.max_new;
    // lengths outside what the call said, or tokens past the table: the
    // sequence is left alone and the call reports it
    if (n < 0 || n > p.max_new || row0 < 0 || len < 0 || (long long)len + n > (long long)p.c.max_pages * ps) {
        if (tid == 0) atomicOr(p.c.err, kErrBadLength);
        return;
    }
    const int pi = len / ps + blockIdx.x % per_seq;                 // page of the sequence
    const int from = max(len, pi * ps), to = min(len + n, pi * ps + ps);
    if (from >= to) return;
    const int page = p.c.table[(long long)b * p.c.max_pages + pi];
    if (page < 0 || page >= p.c.num_pages) {
        if (tid == 0) atomicOr(p.c.err, kErrBadPage);
        return;
    }
    const int held = from - pi * ps, T_new = to - from;   // tokens before, new tokens
    const long long ph = (long long)page * p.c.Hkv + h;
    float *scale = (is_v ? p.c.v_scale : p.c.k_scale) + ph;
    uint8_t *base = (is_v ? p.c.v : p.c.k) + ph * ps * D;
    const float old = held > 0 ? *scale : 0.f;
    // the new tokens into shared memory, rows of D 16-bit values
    constexpr int CH = D / 8;   // 16-byte pieces of a row
    const T *src = reinterpret_cast<const T *>(is_v ? p.v : p.k) + ((long long)(row0 + from - len) * p.c.Hkv + h) * D;
    uint4 *rows = reinterpret_cast<uint4 *>(smem_raw);
    float amax = 0.f;
    for (int i = tid; i < T_new * CH; i += kAppendThreads) {
        const int t = i / CH, c = i % CH;
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + (long long)t * p.c.Hkv * D) + c);
        rows[i] = v;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // NaN and infinities do not set the scale (stored as NaN / saturated)
            const float2 f = Cvt<T>::unpack(w[k]);
            const float x = fabsf(f.x), y = fabsf(f.y);
            amax = x < INFINITY ? fmaxf(amax, x) : amax;
            amax = y < INFINITY ? fmaxf(amax, y) : amax;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();   // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
    const float now = fmaxf(old, pow2(scale_exponent(amax)));
    const float ratio = old / now, inv = 1.f / now;   // powers of two: exact
    if (tid == 0) *scale = now;
    const bool move = held > 0 && ratio != 1.f;
    const T *xs = reinterpret_cast<const T *>(smem_raw);
    if (!is_v) {
        if (move) {
            for (int i = tid; i < held * (D / 16); i += kAppendThreads) {
                uint4 *at = reinterpret_cast<uint4 *>(base) + i;
                const uint4 v = *at;
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
                requantise(w, ratio, 16);
                *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        for (int i = tid; i < T_new * (D / 16); i += kAppendThreads) {
            const uint32_t *x = reinterpret_cast<const uint32_t *>(xs) + 8 * i;
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 a = Cvt<T>::unpack(x[2 * k]), c = Cvt<T>::unpack(x[2 * k + 1]);
                w[k] = f32_to_e4m3x2(a.x * inv, a.y * inv) | f32_to_e4m3x2(c.x * inv, c.y * inv) << 16;
            }
            reinterpret_cast<uint4 *>(base + (long long)held * D)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return;
    }
    // V: 16 tokens of one dim per piece; lanes go along the dims, so the reads
    // of shared memory are rows.  A piece with bytes of before, or past the
    // last token, is read first.
    const int g0 = move ? 0 : held / 16, g1 = (held + T_new + 15) / 16;
    for (int i = tid; i < (g1 - g0) * D; i += kAppendThreads) {
        const int g = g0 + i / D, d = i % D, t0 = 16 * g - held;   // t0: new token of the piece's first byte
        uint4 *at = reinterpret_cast<uint4 *>(base + (long long)d * ps + 16 * g);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (t0 < 0 || t0 + 16 > T_new) {
            const uint4 v = *at;
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            if (move && t0 < 0) requantise(w, ratio, -t0);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f[4];
            uint32_t put = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + 4 * k + j;
                const bool in = t >= 0 && t < T_new;
                f[j] = in ? static_cast<float>(xs[t * D + d]) * inv : 0.f;
                put |= in ? 0xffu << (8 * j) : 0u;
            }
            const uint32_t r = f32_to_e4m3x2(f[0], f[1]) | f32_to_e4m3x2(f[2], f[3]) << 16;
            w[k] = (w[k] & ~put) | (r & put);
        }
        *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// --------------------------------------------------------------- attention
// For one kv head the G query heads of a group times Sq tokens are the rows of
// one tile: S = Q K^T and O = P V run as m16n8k16 products over 64 keys at a
// time.  Bytes bound it (2 D bytes per key against 4 D flops per row and key),
// so the design keeps reads in flight: every warp is a worker of its own with
// a contiguous share of all (sequence, kv head, row group, 64-key tile) work,
// each lane copies the pieces of K and V it needs itself into a ring in shared
// memory (cp.async, no barrier: a lane reads only what it copied), and e4m3
// becomes f16 in registers on the way into the tensor core.  Equal shares
// whatever the lengths; a (sequence, kv head) cut between workers leaves
// pieces that a second kernel joins in a fixed order.
//
// e4m3 fits f16 exactly.  Q (bf16 or f16) enters as f16 under a power of two
// per row that brings its largest magnitude to [2^14, 2^15): exact but for
// values 2^-29 below that.  P enters as f16 <= 2^8 against a running maximum R
// of score + log2(V scale), so the V scales cost no range; the row sums keep
// the running maximum of the scores alone.
//
// Fragments.  The contracted axis may be permuted at will if both operands
// agree: a lane holds 16 consecutive bytes of a key's row (K) or of a dim's
// row of tokens (V), i.e. four k-steps of four values.  Column n of S tile (u,
// h) is key 16 (n / 2) + 4 u + 2 h + n % 2, which puts a lane's P where the
// product with V wants it, and all a lane's keys into one 16-key group, hence
// one page and one scale.
constexpr int kTile = 64;   // keys per step
constexpr float kLazy = 8.f;

template <int D>
struct KvCfg {
    static constexpr int kWarps = (D == 128) ? 6 : 8;
    static constexpr int kStages = (D == 128) ? 2 : 3;
    static constexpr int KB = kTile * D;                 // bytes of a K (or V) tile
    static constexpr int SMEM = kWarps * kStages * 2 * KB;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Tokens of sequence b, 0 where the length is outside the table.
__device__ __forceinline__ int kv_len(const KvAttnParams &p, int b) {
    const int n = __ldg(p.len + b);
    return (n < 0 || (long long)n > (long long)p.c.max_pages * p.c.page) ? 0 : n;
}
// First key any of the sequence's queries sees.
__device__ __forceinline__ int kv_first(const KvAttnParams &p, int n) {
    return p.window < 0 ? 0 : max(0, n - p.Sq - min(p.window, n));
}
__device__ __forceinline__ int kv_tiles(const KvAttnParams &p, int n) {
    return (n + kTile - 1) / kTile - kv_first(p, n) / kTile;
}

// A worker's place in the work: tile t of [t0, t1) of (sequence b, head and row
// group s).
struct Cursor {
    int b, s, t, t0, t1, n, lo;
    __device__ __forceinline__ void open(const KvAttnParams &p) {   // sequence b
        n = kv_len(p, b);
        lo = kv_first(p, n);
        t0 = lo / kTile;
        t1 = (n + kTile - 1) / kTile;
    }
    __device__ __forceinline__ void next(const KvAttnParams &p) {
        if (++t < t1) return;
        if (++s == p.c.Hkv * p.groups) {
            s = 0;
            do {
                if (++b >= p.B) return;   // the end of all work
                open(p);
            } while (t1 <= t0);
        }
        t = t0;
    }
};

__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : l == 0.f ? -INFINITY : l;
}

template <int D, typename T, bool kCap>
__global__ void __launch_bounds__(KvCfg<D>::kWarps * 32, 1) kv_attn_kernel(const __grid_constant__ KvAttnParams p) {
    using C = KvCfg<D>;
    constexpr int W = C::kWarps, ST = C::kStages, KS = D / 16;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ int s_pre[kKvMaxSeqs];   // tiles of sequences 0 .. b, inclusive
    __shared__ int s_warp[W];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r8 = lane >> 2, q4 = lane & 3;

    // ---- the work: tiles per sequence, summed
    const int per_tile = p.c.Hkv * p.groups;
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += W * 32) {
        const int b = b0 + threadIdx.x;
        int x = 0;
        if (b < p.B) {
            const int n = __ldg(p.len + b);
            if (n < 0 || (long long)n > (long long)p.c.max_pages * p.c.page) {
                if (blockIdx.x == 0) atomicOr(p.c.err, kErrBadLength);
            } else {
                x = kv_tiles(p, n);
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        int add = carry, all = carry;
        for (int i = 0; i < W; ++i) {
            if (i < warp) add += s_warp[i];
            all += s_warp[i];
        }
        if (b < p.B) s_pre[b] = x + add;
        carry = all;
        __syncthreads();
    }
    // sequences without a key: zeros
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (s_pre[b] - (b > 0 ? s_pre[b - 1] : 0) > 0) continue;
        uint32_t *o = reinterpret_cast<uint32_t *>(reinterpret_cast<T *>(p.o) + (long long)b * p.Sq * p.Hq * D);
        for (int i = threadIdx.x; i < p.Sq * p.Hq * (D / 2); i += W * 32) o[i] = 0u;
        if (p.lse)
            for (int i = threadIdx.x; i < p.Sq * p.Hq; i += W * 32) p.lse[(long long)b * p.Sq * p.Hq + i] = -INFINITY;
    }
    const long long total = (long long)carry * per_tile;
    // shares of the workers: worker c takes tiles [c total / N, (c + 1) total / N)
    const int wid = blockIdx.x * W + warp;
    const long long N = min((long long)p.workers, total);
    if (lane == 0 && wid < p.workers) p.meta[wid] = make_int4(-1, 0, 0, 0);
    if (wid >= N) return;
    const long long w0 = total * wid / N, w1 = total * (wid + 1) / N;
    auto worker_of = [&](long long w) -> int { return (int)(((w + 1) * N - 1) / total); };

    Cursor pc;   // what is loaded next
    {
        const int u = (int)(w0 / per_tile);   // tile over the sequences, if every tile came once
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] > u) hi = mid;
            else lo = mid + 1;
        }
        pc.b = lo;
        pc.open(p);
        const long long in = w0 - (long long)(lo > 0 ? s_pre[lo - 1] : 0) * per_tile;
        const int nt = pc.t1 - pc.t0;
        pc.s = (int)(in / nt);
        pc.t = pc.t0 + (int)(in - (long long)pc.s * nt);
    }
    Cursor cc = pc;   // what is computed next
    int left = (int)(w1 - w0), to_load = left;

    const uint32_t ring = smem_u32(smem_raw) + warp * (ST * 2 * C::KB) + 16 * lane;
    // page of 16-key group (lane % 4) of the tile at pc, and the lookup of the next
    auto lookup = [&](const Cursor &c) -> int {
        const int tok = kTile * c.t + 16 * q4;
        if (tok >= c.n || tok + 16 <= c.lo) return -1;    // a group nobody sees: not read
        const int page = __ldg(p.c.table + (long long)c.b * p.c.max_pages + tok / p.c.page);
        if (page < 0 || page >= p.c.num_pages) {
            atomicOr(p.c.err, kErrBadPage);
            return -1;
        }
        return page;
    };
    int pg = lookup(pc);
    float ksc[ST], vsc[ST];   // scales of the lane's group, tiles in the ring
    // K of the tile at pc into slot st (and its scales), then V of the same tile
    auto load_k = [&](int st) __attribute__((always_inline)) {
        if (to_load > 0) {
            const int hk = pc.s / p.groups;
            ksc[st] = 0.f;
            vsc[st] = 0.f;
            if (pg >= 0) {
                ksc[st] = __ldg(p.c.k_scale + (long long)pg * p.c.Hkv + hk);
                vsc[st] = __ldg(p.c.v_scale + (long long)pg * p.c.Hkv + hk);
            }
            const int grp = r8 >> 1;
            const int page = __shfl_sync(0xffffffffu, pg, grp);
            const int in_page = (kTile * pc.t + 16 * grp) % p.c.page + (r8 & 1);
            const uint8_t *src = p.c.k + (((long long)max(page, 0) * p.c.Hkv + hk) * p.c.page + in_page) * D + 16 * q4;
#pragma unroll
            for (int ut = 0; ut < 8; ++ut)
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh)
                    cp_async16(ring + st * 2 * C::KB + 512 * (ut * (D / 64) + hh), src + 2 * ut * D + 64 * hh, page >= 0);
        }
        cp_commit();
    };
    auto load_v = [&](int st) __attribute__((always_inline)) {
        if (to_load > 0) {
            const int hk = pc.s / p.groups;
            const int in_page = (kTile * pc.t + 16 * q4) % p.c.page;
            const uint8_t *src = p.c.v + (((long long)max(pg, 0) * p.c.Hkv + hk) * D + r8) * p.c.page + in_page;
#pragma unroll
            for (int dt = 0; dt < D / 8; ++dt)
                cp_async16(ring + st * 2 * C::KB + C::KB + 512 * dt, src + (long long)8 * dt * p.c.page, pg >= 0);
            if (--to_load > 0) {
                pc.next(p);
                pg = lookup(pc);
            }
        }
        cp_commit();
    };
    // (the slots are compile-time constants: the scales stay in registers)
#pragma unroll
    for (int st = 0; st < ST; ++st) {
        load_k(st);
        load_v(st);
    }

    // ---- state of the segment being computed
    uint32_t qa[KS][4];          // Q fragments (f16)
    float fr[2];                 // per row r8, r8 + 8: undoes Q's power of two, times c log2(e) (or the cap's factor)
    int lo_r[2], hi_r[2];        // visible keys of the two rows
    float acc[D / 8][4];
    float m_run[2], l_run[2], R[2];
    bool fresh = true, begins = false;
    auto open_segment = [&]() __attribute__((always_inline)) {
        const int hk = cc.s / p.groups, rg = cc.s % p.groups;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = rg * 16 + r8 + 8 * j;
            const bool live = row < p.Sq * p.G;
            const int i = live ? row / p.G : p.Sq - 1, g = live ? row % p.G : 0;
            const T *src = reinterpret_cast<const T *>(p.q) + (((long long)cc.b * p.Sq + i) * p.Hq + hk * p.G + g) * D + 16 * q4;
            uint32_t raw[D / 64][8];
            float amax = 0.f;
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh) {
                const uint4 a = live ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * hh)) : make_uint4(0, 0, 0, 0);
                const uint4 c = live ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * hh) + 1) : make_uint4(0, 0, 0, 0);
                raw[hh][0] = a.x, raw[hh][1] = a.y, raw[hh][2] = a.z, raw[hh][3] = a.w;
                raw[hh][4] = c.x, raw[hh][5] = c.y, raw[hh][6] = c.z, raw[hh][7] = c.w;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 f = Cvt<T>::unpack(raw[hh][k]);
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            amax = quad_max(amax);
            const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
            const float up = pow2(14 - min(e, 126)), down = pow2(min(e, 126) - 14);
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
                for (int k = 0; k < 8; ++k) {   // piece k of the row: k-step 4 hh + k / 2, register j + 2 (k % 2)
                    const float2 f = Cvt<T>::unpack(raw[hh][k]);
                    qa[4 * hh + k / 2][j + 2 * (k & 1)] = Cvt<__half>::pack(f.x * up, f.y * up);
                }
            fr[j] = down * (kCap ? p.cap_k : p.scale_log2);
            hi_r[j] = cc.n - p.Sq + i;
            lo_r[j] = p.window < 0 ? 0 : max(0, hi_r[j] - p.window);
            m_run[j] = R[j] = -INFINITY;
            l_run[j] = 0.f;
        }
#pragma unroll
        for (int dt = 0; dt < D / 8; ++dt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[dt][i] = 0.f;
        begins = cc.t == cc.t0;
        fresh = false;
    };
    // the rows' results, or the piece's for the join
    auto close_segment = [&](bool ends) __attribute__((always_inline)) {
        const int hk = cc.s / p.groups, rg = cc.s % p.groups;
        const bool whole = begins && ends;
        const int piece = begins ? 1 : 0;
        if (!whole && !begins && lane == 0) {
            // the segment's first tile in the order of all work
            const long long first = (long long)(cc.b > 0 ? s_pre[cc.b - 1] : 0) * per_tile + (long long)cc.s * (cc.t1 - cc.t0);
            p.meta[wid] = make_int4(cc.s, worker_of(first), ends ? 1 : 0, cc.b);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float l = quad_sum(l_run[j]);
            const int row = rg * 16 + r8 + 8 * j;
            if (row >= p.Sq * p.G) continue;
            if (whole) {
                const int i = row / p.G, hq = hk * p.G + row % p.G;
                const float f = l == 0.f ? 0.f : ex2(R[j] - m_run[j]) / l;
                T *dst = reinterpret_cast<T *>(p.o) + (((long long)cc.b * p.Sq + i) * p.Hq + hq) * D + 2 * q4;
#pragma unroll
                for (int dt = 0; dt < D / 8; ++dt)
                    *reinterpret_cast<uint32_t *>(dst + 8 * dt) =
                        l == 0.f ? 0u : Cvt<T>::pack(acc[dt][2 * j] * f, acc[dt][2 * j + 1] * f);
                if (p.lse && q4 == 0) p.lse[((long long)cc.b * p.Hq + hq) * p.Sq + i] = lse_of(m_run[j], l);
            } else {
                const long long at = ((long long)wid * 2 + piece) * 16 + r8 + 8 * j;
                float *dst = p.acc + at * D + 2 * q4;
#pragma unroll
                for (int dt = 0; dt < D / 8; ++dt)
                    *reinterpret_cast<float2 *>(dst + 8 * dt) = make_float2(acc[dt][2 * j], acc[dt][2 * j + 1]);
                if (q4 == 0) p.stat[at] = make_float4(m_run[j], l, R[j], 0.f);
            }
        }
        fresh = true;
    };

    auto step = [&](int st) __attribute__((always_inline)) {
        if (fresh) open_segment();
        const uint32_t kt = ring + st * 2 * C::KB, vt = kt + C::KB;
        // S = Q K^T
        cp_wait<2 * ST - 1>();
        float s[8][4];
#pragma unroll
        for (int ut = 0; ut < 8; ++ut) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[ut][i] = 0.f;
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh) {
                const uint4 v = ld_shared_v4(kt + 512 * (ut * (D / 64) + hh));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16(w[k], b0, b1);
                    mma_f16(s[ut], qa[4 * hh + k], b0, b1);
                }
            }
        }
        const float ks = ksc[st], vs = vsc[st];
        const int key0 = kTile * cc.t + 16 * q4;   // first key of the lane's group
        const int n = cc.n;
        const bool ends = cc.t + 1 == cc.t1;
        load_k(st);   // the slot's K has been read
        const float ev = vs > 0.f ? log2f(vs) : -INFINITY;   // exact for a power of two
        // scores in log2 units; a tile inside every row's keys takes no compare
        const bool edge = __any_sync(0xffffffffu, kTile * cc.t < max(lo_r[0], lo_r[1]) ||
                                                      kTile * cc.t + kTile - 1 > min(hi_r[0], hi_r[1]));
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int ut = 0; ut < 8; ++ut)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x0 = s[ut][2 * j] * (fr[j] * ks), x1 = s[ut][2 * j + 1] * (fr[j] * ks);
                const int key = key0 + 2 * ut;
                const bool off0 = key < lo_r[j] || key > hi_r[j], off1 = key + 1 < lo_r[j] || key + 1 > hi_r[j];
                if (kCap) {
                    float r0, r1;
                    if (edge) {   // what lies behind the last token may be NaN: not into the pair
                        x0 = off0 ? 0.f : x0;
                        x1 = off1 ? 0.f : x1;
                    }
                    cap_r2(x0, x1, r0, r1);
                    x0 = fmaf(-2.f * p.cap_log2, r0, p.cap_log2);
                    x1 = fmaf(-2.f * p.cap_log2, r1, p.cap_log2);
                }
                if (edge) {
                    if (off0) x0 = -INFINITY;
                    if (off1) x1 = -INFINITY;
                }
                s[ut][2 * j] = x0;
                s[ut][2 * j + 1] = x1;
                mx[j] = fmaxf(mx[j], fmaxf(x0, x1));
            }
        uint32_t pa[4][4];
        float mref[2], rref[2];
        bool grow = false;
        float ry[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float y = quad_max(mx[j] + ev);
            const float m = fmaxf(m_run[j], quad_max(mx[j]));
            mref[j] = m == -INFINITY ? 0.f : m;
            l_run[j] *= ex2(m_run[j] - mref[j]);   // -inf before the first key: 0
            m_run[j] = m;
            ry[j] = R[j];
            if (y > R[j] + kLazy || R[j] == -INFINITY) {
                ry[j] = fmaxf(R[j], y);
                grow |= ry[j] != R[j];
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float a = ry[j] == R[j] ? 1.f : ex2(R[j] - ry[j]);
#pragma unroll
                for (int dt = 0; dt < D / 8; ++dt) {
                    acc[dt][2 * j] *= a;
                    acc[dt][2 * j + 1] *= a;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            R[j] = ry[j];
            rref[j] = R[j] == -INFINITY ? INFINITY : R[j] - ev;   // no weight yet: P = 0
            float sum = 0.f;
#pragma unroll
            for (int ut = 0; ut < 8; ++ut) {
                const float x0 = s[ut][2 * j], x1 = s[ut][2 * j + 1];
                sum += ex2(x0 - mref[j]) + ex2(x1 - mref[j]);
                // k-step ut / 2: register j (first eight columns) or 2 + j
                pa[ut >> 1][j + 2 * (ut & 1)] = Cvt<__half>::pack(ex2(x0 - rref[j]), ex2(x1 - rref[j]));
            }
            l_run[j] += sum;
        }
        // O += P V
        cp_wait<2 * ST - 1>();
        const int nv = n - key0;   // tokens of the group that exist: bytes behind them hold anything
        const bool tail = __any_sync(0xffffffffu, nv < 16);
#pragma unroll
        for (int dt = 0; dt < D / 8; ++dt) {
            const uint4 v = ld_shared_v4(vt + 512 * dt);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (tail) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = min(max(nv - 4 * k, 0), 4);
                    w[k] = c >= 4 ? w[k] : w[k] & ((1u << (8 * c)) - 1u);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t b0, b1;
                e4m3x4_to_f16(w[k], b0, b1);
                mma_f16(acc[dt], pa[k], b0, b1);
            }
        }
        load_v(st);
        --left;
        if (ends || left == 0) close_segment(ends);
        if (left > 0) cc.next(p);
    };
    while (true) {
#pragma unroll
        for (int st = 0; st < ST; ++st) {
            step(st);
            if (left == 0) {
                cp_wait<0>();
                return;
            }
        }
    }
}

// ------------------------------------------------------------------- join
// One CTA per worker whose share begins inside a segment that ends in it: the
// pieces of that segment (piece 1 of its first worker, piece 0 of the others)
// joined in worker order, one warp per row at a time.
template <int D, typename T>
__global__ void __launch_bounds__(128) kv_join_kernel(const __grid_constant__ KvAttnParams p) {
    const int wid = blockIdx.x;
    const int4 me = p.meta[wid];
    if (me.x < 0 || me.z == 0) return;
    const int hk = me.x / p.groups, rg = me.x % p.groups, first = me.y, b = me.w;
    constexpr int V = D / 32;   // dims per lane
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int r = warp; r < 16; r += 4) {
        const int row = rg * 16 + r;
        if (row >= p.Sq * p.G) break;
        auto slot = [&](int w) -> long long { return ((long long)w * 2 + (w == first ? 1 : 0)) * 16 + r; };
        float M = -INFINITY, RM = -INFINITY;
        for (int w = first + lane; w <= wid; w += 32) {
            const float4 st = p.stat[slot(w)];
            M = fmaxf(M, st.x);
            RM = fmaxf(RM, st.z);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            RM = fmaxf(RM, __shfl_xor_sync(0xffffffffu, RM, o));
        }
        const float m0 = M == -INFINITY ? 0.f : M, r0 = RM == -INFINITY ? 0.f : RM;
        float l = 0.f, x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 0.f;
#pragma unroll 4
        for (int w = first; w <= wid; ++w) {
            const float4 st = p.stat[slot(w)];
            l += st.y * ex2(st.x - m0);
            const float f = ex2(st.z - r0);
            const float *src = p.acc + slot(w) * D + V * lane;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(src + i);
                x[i] = fmaf(v.x, f, x[i]);
                x[i + 1] = fmaf(v.y, f, x[i + 1]);
            }
        }
        const int i = row / p.G, hq = hk * p.G + row % p.G;
        const float f = l == 0.f ? 0.f : ex2(r0 - m0) / l;
        uint32_t *dst = reinterpret_cast<uint32_t *>(reinterpret_cast<T *>(p.o) + (((long long)b * p.Sq + i) * p.Hq + hq) * D + V * lane);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) dst[k] = l == 0.f ? 0u : Cvt<T>::pack(x[2 * k] * f, x[2 * k + 1] * f);
        if (p.lse && lane == 0) p.lse[((long long)b * p.Hq + hq) * p.Sq + i] = lse_of(M, l);
    }
}

template <int D, typename T, bool kCap>
cudaError_t launch_attn_t(KvAttnParams p, int sms, cudaStream_t stream) {
    using C = KvCfg<D>;
    auto kern = kv_attn_kernel<D, T, kCap>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int grid = sms < kKvSms ? sms : kKvSms;
    p.workers = grid * C::kWarps;
    kern<<<grid, C::kWarps * 32, C::SMEM, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    kv_join_kernel<D, T><<<p.workers, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int D, typename T>
cudaError_t launch_append_t(const KvAppendParams &p, cudaStream_t stream) {
    // pages a sequence's new tokens can touch: from anywhere in the first one
    const long long per_seq = ((long long)p.max_new + p.c.page - 2) / p.c.page + 1;
    if (per_seq * p.B > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int smem = (p.max_new < p.c.page ? p.max_new : p.c.page) * D * 2;
    const dim3 grid((unsigned)(per_seq * p.B), (unsigned)p.c.Hkv, 2);
    kv_append_kernel<D, T><<<grid, kAppendThreads, smem, stream>>>(p, (int)per_seq);
    return cudaGetLastError();
}

}  // namespace

int kv_warps(int D) { return D == 128 ? KvCfg<128>::kWarps : KvCfg<64>::kWarps; }

size_t kv_workspace_bytes(int D) {
    const size_t n = (size_t)kKvSms * kv_warps(D);
    return n * 2 * 16 * D * sizeof(float) + n * 2 * 16 * sizeof(float4) + n * sizeof(int4);
}

cudaError_t launch_kv_append(const KvAppendParams &p, int D, int bf16, cudaStream_t stream) {
    if (D == 128)
        return bf16 ? launch_append_t<128, __nv_bfloat16>(p, stream) : launch_append_t<128, __half>(p, stream);
    return bf16 ? launch_append_t<64, __nv_bfloat16>(p, stream) : launch_append_t<64, __half>(p, stream);
}

cudaError_t launch_kv_attn(const KvAttnParams &p, int D, int bf16, int sms, cudaStream_t stream) {
    const bool cap = p.cap_log2 > 0.f;
    if (D == 128) {
        if (bf16)
            return cap ? launch_attn_t<128, __nv_bfloat16, true>(p, sms, stream)
                       : launch_attn_t<128, __nv_bfloat16, false>(p, sms, stream);
        return cap ? launch_attn_t<128, __half, true>(p, sms, stream) : launch_attn_t<128, __half, false>(p, sms, stream);
    }
    if (bf16)
        return cap ? launch_attn_t<64, __nv_bfloat16, true>(p, sms, stream)
                   : launch_attn_t<64, __nv_bfloat16, false>(p, sms, stream);
    return cap ? launch_attn_t<64, __half, true>(p, sms, stream) : launch_attn_t<64, __half, false>(p, sms, stream);
}

}  // namespace fa
