// fa_kvcache.cu -- the 8-bit paged key / value cache: appending to it and the
// attention of a sequence's last tokens over it.
//
// Values are e4m3 with one scale per (page, kv head), a power of two 2^e with
// the smallest e for which the page's largest magnitude fits 448 * 2^e.  A
// power of two costs no precision (e4m3 is a floating type) and makes the
// division by the scale, and moving a page to a larger scale, exact but for
// values that become subnormal.  A page filled elsewhere may keep another scale;
// its values are rounded once all the same (div_to_odd).
//
// K lies token by token, V dim by dim, so that in both products the 16-byte
// pieces a lane reads are contiguous along the axis the tensor core contracts.
#include <type_traits>

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
// Prompts (51 MB moved, nothing in L2 before) take 16.5 us, 3.1 TB/s: three
// dependent reads from memory per CTA, in two waves of CTAs.  With 128 threads
// 18.0; with loads that the compiler was left to batch 20.4; with floats compared
// and every byte of V tested 18.0 (but 12.6 against 10.6 with the tokens in L2).

// smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), held in [-120, 120]
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, -120), 120);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// x / s and x r in 32 bits, rounded to odd: cut off, and the last bit set if
// anything was.  Rounding that to e4m3's four bits to nearest even then gives what
// rounding the exact value would, as a nearest 32-bit value need not (it may land on
// a tie).  Results whose cut-off part is itself below 32 bits' range are far below
// half of e4m3's smallest value.
__device__ __forceinline__ float to_odd(float q, float rest) {
    return rest < 0.f || rest > 0.f ? __uint_as_float(__float_as_uint(q) | 1u) : q;   // (NaN: as it is)
}
__device__ __forceinline__ float div_to_odd(float x, float s) {
    const float q = __fdiv_rz(x, s);
    return to_odd(q, fmaf(-q, s, x));
}
__device__ __forceinline__ float mul_to_odd(float x, float r) {
    const float q = __fmul_rz(x, r);
    return to_odd(q, fmaf(x, r, -q));
}

// 16 stored bytes moved to another scale, those from byte `n` on left alone
__device__ __forceinline__ void requantise(uint32_t (&w)[4], float ratio, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, b;
        e4m3x4_to_f16(w[i], a, b);
        const float2 x = Cvt<__half>::unpack(a), y = Cvt<__half>::unpack(b);
        const uint32_t r = f32_to_e4m3x2(mul_to_odd(x.x, ratio), mul_to_odd(x.y, ratio)) |
                           f32_to_e4m3x2(mul_to_odd(y.x, ratio), mul_to_odd(y.y, ratio)) << 16;
        const int k = min(max(n - 4 * i, 0), 4);
        const uint32_t keep = k >= 4 ? 0u : 0xffffffffu << (8 * k);
        w[i] = (w[i] & keep) | (r & ~keep);
    }
}

// magnitudes of two 16-bit floats compare as their bits do
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int D, typename T, int kThreads>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p, int per_seq) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_max[kThreads / 32];
    const int ps = p.c.page, tid = threadIdx.x;
    const int b = blockIdx.x / per_seq, h = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int len = p.len[b];
    const int row0 = p.cu ? p.cu[b] : b * p.max_new;
    const int n = p.cu ? p.cu[b + 1] - row0 : p.max_new;
    // lengths or rows outside what the call said, or tokens past the table: the
    // sequence is left alone and the call reports it
    if (n < 0 || n > p.max_new || row0 < 0 || (long long)row0 + n > p.rows || len < 0 || (long long)len + n > (long long)p.c.max_pages * ps) {
        if (tid == 0) atomicOr(p.c.err, kErrBadLength);
        return;
    }
    const int pi = len / ps + blockIdx.x % per_seq;                 // page of the sequence
    const int from = max(len, pi * ps), to = min(len + n, pi * ps + ps);
    if (from >= to) return;
    // (read here, looked at once the tokens are on their way)
    const int page = p.c.table[(long long)b * p.c.max_pages + pi];
    const int held = from - pi * ps, T_new = to - from;   // tokens before, new tokens
    // the new tokens into shared memory, rows of D 16-bit values
    constexpr int CH = D / 8, PER = kThreads == 128 ? 2 : 4;   // 16-byte pieces of a row, and per thread
    const T *src = reinterpret_cast<const T *>(is_v ? p.v : p.k) + ((long long)(row0 + from - len) * p.c.Hkv + h) * D;
    uint4 *rows = reinterpret_cast<uint4 *>(smem_raw);
    uint32_t top = 0u;   // largest magnitudes, as bits: of the low and of the high halves
    for (int i0 = tid; i0 < T_new * CH; i0 += PER * kThreads) {
        uint4 v[PER];   // all on their way at once
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = i0 + k * kThreads, t = i / CH, c = i % CH;
            v[k] = i < T_new * CH ? __ldg(reinterpret_cast<const uint4 *>(src + (long long)t * p.c.Hkv * D) + c)
                                  : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = i0 + k * kThreads;
            if (i < T_new * CH) rows[i] = v[k];
            top = max_u16x2(max_u16x2(top, v[k].x & 0x7fff7fffu), v[k].y & 0x7fff7fffu);
            top = max_u16x2(max_u16x2(top, v[k].z & 0x7fff7fffu), v[k].w & 0x7fff7fffu);
        }
    }
    constexpr uint32_t kInf = Cvt<T>::is_bf16 ? 0x7f80u : 0x7c00u;
    top = max(top >> 16, top & 0xffffu);
    if (top >= kInf) {
        // NaN and infinities do not set the scale (stored as NaN / saturated): the
        // thread's pieces again without them
        top = 0u;
        for (int i = tid; i < T_new * CH; i += kThreads)
            for (int k = 0; k < 8; ++k) {
                const uint32_t x = reinterpret_cast<const uint16_t *>(rows + i)[k] & 0x7fffu;
                top = x < kInf ? max(top, x) : top;
            }
    }
    if (page < 0 || page >= p.c.num_pages) {   // (the whole CTA)
        if (tid == 0) atomicOr(p.c.err, kErrBadPage);
        return;
    }
    const long long ph = (long long)page * p.c.Hkv + h;
    float *scale = (is_v ? p.c.v_scale : p.c.k_scale) + ph;
    uint8_t *base = (is_v ? p.c.v : p.c.k) + ph * ps * D;
    const float old = held > 0 ? *scale : 0.f;
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) s_max[tid >> 5] = top;
    __syncthreads();   // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, s_max[i]);
    const float amax = Cvt<T>::unpack(top).x;
    const float now = fmaxf(old, pow2(scale_exponent(amax)));
    // exact: ratio, for now is old or a power of two; inv, where now is a power of two
    const float ratio = old / now, inv = 1.f / now;
    if (tid == 0) *scale = now;
    const bool move = held > 0 && ratio != 1.f;
    const T *xs = reinterpret_cast<const T *>(smem_raw);
    // (a scale that is no power of two takes a copy of the rest that divides)
    auto store = [&](auto exact_tag) __attribute__((always_inline)) {
        constexpr bool kExact = decltype(exact_tag)::value;
        auto scaled = [&](float x) __attribute__((always_inline)) -> float { return kExact ? x * inv : div_to_odd(x, now); };
        if (!is_v) {
            if (move) {
                for (int i = tid; i < held * (D / 16); i += kThreads) {
                    uint4 *at = reinterpret_cast<uint4 *>(base) + i;
                    const uint4 v = *at;
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    requantise(w, ratio, 16);
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            for (int i = tid; i < T_new * (D / 16); i += kThreads) {
                const uint32_t *x = reinterpret_cast<const uint32_t *>(xs) + 8 * i;
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 a = Cvt<T>::unpack(x[2 * k]), c = Cvt<T>::unpack(x[2 * k + 1]);
                    w[k] = f32_to_e4m3x2(scaled(a.x), scaled(a.y)) | f32_to_e4m3x2(scaled(c.x), scaled(c.y)) << 16;
                }
                reinterpret_cast<uint4 *>(base + (long long)held * D)[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            return;
        }
        // V: pieces of 16 tokens of one dim; lanes go along the dims, so the reads of
        // shared memory are rows.  Pieces all of whose tokens are new take two dims a
        // thread and no test per byte; a piece with bytes of before, or past the last
        // token, is read first.
        const int g0 = move ? 0 : held / 16;
        int g1 = (held + T_new + 15) / 16;
        const int ga = (held + 15) / 16, gw = max((held + T_new) / 16 - ga, 0);   // pieces [ga, ga + gw) are whole
#pragma unroll 1
        for (int i = tid; i < gw * (D / 2); i += kThreads) {
            const int g = ga + i / (D / 2), d = 2 * (i % (D / 2));
            const T *x = xs + (16 * g - held) * D + d;
            uint32_t w0[4], w1[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = Cvt<T>::unpack(*reinterpret_cast<const uint32_t *>(x + (4 * k + j) * D));
                w0[k] = f32_to_e4m3x2(scaled(f[0].x), scaled(f[1].x)) | f32_to_e4m3x2(scaled(f[2].x), scaled(f[3].x)) << 16;
                w1[k] = f32_to_e4m3x2(scaled(f[0].y), scaled(f[1].y)) | f32_to_e4m3x2(scaled(f[2].y), scaled(f[3].y)) << 16;
            }
            uint4 *at = reinterpret_cast<uint4 *>(base + (long long)d * ps + 16 * g);
            *at = make_uint4(w0[0], w0[1], w0[2], w0[3]);
            at[ps / 16] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        }
        g1 -= gw;
#pragma unroll 1
        for (int i = tid; i < (g1 - g0) * D; i += kThreads) {
            int g = g0 + i / D;
            if (gw > 0 && g >= ga) g += gw;   // over the whole ones
            const int d = i % D, t0 = 16 * g - held;   // t0: new token of the piece's first byte
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
                    f[j] = in ? scaled(static_cast<float>(xs[t * D + d])) : 0.f;
                    put |= in ? 0xffu << (8 * j) : 0u;
                }
                const uint32_t r = f32_to_e4m3x2(f[0], f[1]) | f32_to_e4m3x2(f[2], f[3]) << 16;
                w[k] = (w[k] & ~put) | (r & put);
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
    };
    if ((__float_as_uint(now) & 0x7fffffu) == 0u) store(std::true_type{});
    else store(std::false_type{});
}

// --------------------------------------------------------------- attention
// For one kv head the G query heads of a group times Sq tokens are the rows of
// one product: S^T = K Q^T and O^T = V^T P^T run as m16n8k16 products over 64
// keys at a time, keys (then dims) along M and the rows along N, so a decoding
// step's few rows pad to 8 and not to 16.  Bytes bound it (2 D bytes per key
// against 4 D flops per row and key), so the design keeps reads in flight:
// every warp is a worker of its own with a contiguous share of all (sequence,
// kv head, row group, 64-key tile) work and its own K and V slot in shared
// memory, filled by bulk copies (one per 16 keys of K, one per page of V) that
// go out as soon as the slot has been read.  (With a 16-byte cp.async per lane
// instead, 3600 of a tile's 8200 cycles went by issuing the 32 copies.)  Equal shares whatever the lengths; a (sequence, kv head) cut
// between workers leaves pieces that a second kernel joins in a fixed order.
//
// K goes to the tensor core as it lies.  Q is split into e4m3 parts, each what
// the one before left, times 16: a bf16 value (8 significant bits) is two
// parts of four bits, an f16 value (11) three, under a power of two per row
// that brings its largest magnitude to [2^7, 2^8).  The parts are exact but for
// values more than 2^13 below that (the last part's smallest step, 2^-13 or
// 2^-17 of the row's units); their products run in accumulators of their own,
// the e4m3 product adds in full 32 bits (measured: within 2^-22 of the sum of
// magnitudes), and it is four times as fast per key as the f16 one behind two
// conversions per value.  For V, e4m3 fits f16 exactly; P enters as f16 <= 2^8
// against a running maximum R of score + log2(V scale), so the V scales cost no
// range; the row sums keep the running maximum of the scores alone.
//
// Fragments.  The contracted axis may be permuted at will if both operands
// agree: a lane holds 16 consecutive bytes of a key's row (K) or of a dim's
// row of tokens (V).  Row 8 h + r of S^T tile t is key 16 (r / 2) + r % 2 + 4 t
// + 2 h: all keys of a lane are then of one 16-key group (one page, one scale),
// and the 8x8 blocks of P, transposed across the lanes (movmatrix), are where
// the product with V wants them.
constexpr int kTile = 64;   // keys per step
constexpr float kLazy = 8.f;
template <typename T> constexpr int kQParts = Cvt<T>::is_bf16 ? 2 : 3;

// NR: 8-row blocks of a worker's rows (1 or 2).  Warps per CTA: at D = 128, 8
// with up to 255 registers each stream at 21 bytes per cycle and SM; 12 with
// 168 spill, and every part of a step took 1.6 to 3 times as long (75 against
// 66 us on 64 requests of 256 to 8192 tokens).
template <int D, int NR>
struct KvCfg {
    static constexpr int kWarps = (D == 128 || NR == 2) ? 8 : 12;
    static constexpr int KB = kTile * D;                 // bytes of a K (or V) tile
    static constexpr int VB = KB + 128;                  // V's blocks lie apart (kv_block_pad)
    static constexpr int SMEM = kWarps * (KB + VB);
    static constexpr int PIECE = NR * 8 * D;             // floats of a piece
    static_assert(kWarps <= kv_max_warps(D), "the workspace holds that many workers per SM");
    static_assert(SMEM + 8 * kKvMaxSeqs + 2048 <= 232448, "shared memory overflow");
};

// 2-D tiled load (bytes along a row, row) completing on an mbarrier.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
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

// the low c bytes of a word (none below 0, all from 4 on)
__device__ __forceinline__ uint32_t bytes_below(int c) { return c >= 4 ? 0xffffffffu : (1u << (8 * max(c, 0))) - 1u; }

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

__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : l == 0.f ? -INFINITY : l;
}
// What turns a row's accumulator into its output: 2^(R - m) / l (0 for a row
// that saw nothing).
__device__ __forceinline__ float out_factor(float R, float m, float l) { return l == 0.f ? 0.f : ex2(R - m) / l; }

// Output rows of a piece in fragment order: acc[dm] holds dims 16 dm + r8 (and
// + 8) of rows row0 + 2 q4, + 1, already scaled.
template <int D, typename T>
__device__ __forceinline__ void store_rows(const KvAttnParams &p, int b, int hk, int row0, int lane,
                                           float (&acc)[4], int dm) {
    const int r8 = lane >> 2, q4 = lane & 3;
    // two 8x8 blocks (dims x rows), transposed: lane gets row r8, dims 2 q4, + 1
    const uint32_t lo = transpose8(Cvt<T>::pack(acc[0], acc[1]));
    const uint32_t hi = transpose8(Cvt<T>::pack(acc[2], acc[3]));
    const int row = row0 + r8;
    if (row < p.Sq * p.G) {
        const int i = row / p.G, hq = hk * p.G + row % p.G;
        T *dst = reinterpret_cast<T *>(p.o) + (((long long)b * p.Sq + i) * p.Hq + hq) * D + 16 * dm + 2 * q4;
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

template <int D, typename T>
__device__ __forceinline__ void finish_rows(const KvAttnParams &p, const Joined &x, int b, int hk, int row0, int dm,
                                            int lane) {
    const float f0 = out_factor(x.r[0], x.m[0], x.l[0]), f1 = out_factor(x.r[1], x.m[1], x.l[1]);
    float o[4] = {x.v.x * f0, x.v.y * f1, x.v.z * f0, x.v.w * f1};
    store_rows<D, T>(p, b, hk, row0, lane, o, dm);
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

template <int D, int NR, typename T, bool kCap>
__global__ void __launch_bounds__(KvCfg<D, NR>::kWarps * 32, 1)
    kv_attn_kernel(const __grid_constant__ KvAttnParams p, const __grid_constant__ CUtensorMap map_v) {
    using C = KvCfg<D, NR>;
    constexpr int W = C::kWarps, HH = D / 64, K32 = D / 32, DM = D / 16, QP = kQParts<T>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ int s_pre[kKvMaxSeqs];   // half tiles of one head and row group of sequences 0 .. b, inclusive
    __shared__ int s_len[kKvMaxSeqs];   // their tokens, 0 where the length is outside the table
    __shared__ int s_warp[W];
    __shared__ __align__(8) uint64_t s_bar[W][2];   // K, V of the worker's tile landed
    __shared__ int s_abort;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r8 = lane >> 2, q4 = lane & 3;

    if (threadIdx.x == 0) s_abort = 0;
    if (lane == 0) p.meta[blockIdx.x * W + warp] = make_int4(-1, 0, 0, 0);
    if (lane < 2) {
        mbar_init(smem_u32(&s_bar[warp][lane]), 1);
        fence_mbar_init();
    }
    // ---- the work: tiles per sequence, summed
    const int per_tile = p.c.Hkv * p.groups;
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
        uint32_t *o = reinterpret_cast<uint32_t *>(reinterpret_cast<T *>(p.o) + (long long)b * p.Sq * p.Hq * D);
        for (int i = threadIdx.x; i < p.Sq * p.Hq * (D / 2); i += W * 32) o[i] = 0u;
        if (p.lse)
            for (int i = threadIdx.x; i < p.Sq * p.Hq; i += W * 32) p.lse[(long long)b * p.Sq * p.Hq + i] = -INFINITY;
    }
    const int total = carry * per_tile;   // (the host keeps it below 2^31)
    // shares of the workers: total / N half tiles each, one more for the first
    // total % N; a worker holds at least two tiles' worth, so that few pieces
    // are made of little work
    const int wid = blockIdx.x * W + warp, N = min(p.workers, max(total / 4, 1));
    pdl_launch();
    if (wid >= N || total == 0) return;
    const int share = total / N, more = total - share * N;
    const int w0 = wid * share + min(wid, more), w1 = w0 + share + (wid < more ? 1 : 0);
    auto worker_of = [&](int w) -> int {
        const int head = (share + 1) * more;
        return w < head ? w / (share + 1) : more + (w - head) / share;
    };
    // the tile behind a border (past the last one: b == B)
    auto place = [&](int w, Cursor &c) {
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
    };
    Cursor pc, end;   // what is loaded next, and where the worker stops
    {
        Cursor c;   // even lanes place the one, odd lanes the other
        place(lane & 1 ? w1 : w0, c);
        auto from = [&](int src, Cursor &d) {
            d.b = __shfl_sync(0xffffffffu, c.b, src), d.hk = __shfl_sync(0xffffffffu, c.hk, src);
            d.rg = __shfl_sync(0xffffffffu, c.rg, src), d.t = __shfl_sync(0xffffffffu, c.t, src);
        };
        from(0, pc);
        from(1, end);
        const int t = pc.t;
        if (pc.b < p.B) pc.open(p, s_len);
        pc.t = t;
    }
    auto at_end = [&](const Cursor &c) -> bool {
        return c.b == end.b && c.hk == end.hk && c.rg == end.rg && c.t == end.t;
    };
    if (at_end(pc)) return;
    Cursor cc = pc;   // what is computed next
    {   // the first rows of Q on their way while the block table is read
        const int row = cc.rg * NR * 8 + r8;
        if (row < p.Sq * p.G) {
            const T *src = reinterpret_cast<const T *>(p.q) +
                           (((long long)cc.b * p.Sq + row / p.G) * p.Hq + cc.hk * p.G + row % p.G) * D + q4 * (D / 4);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
        }
    }
    bool loads = true;   // pc is a tile of this worker's

    const uint32_t kt = smem_u32(smem_raw) + warp * (C::KB + C::VB), vt = kt + C::KB;
    const uint32_t k_bar = smem_u32(&s_bar[warp][0]), v_bar = smem_u32(&s_bar[warp][1]);
    const WaitCtl wctl{&s_abort, p.c.err, p.budget_ns};
    uint32_t phase = 0;   // of both barriers: the tile being computed
    bool ahead = false;   // gave up with the next tile's K on its way
    // V in shared memory: 64 / bw blocks of bw tokens, D rows each, a pad apart
    const int bw = p.v_block, v_step = D * bw + p.v_pad;
    // this lane's 16 tokens of dim r8, and its keys' rows
    const uint32_t v_at = vt + (16 * q4 / bw) * v_step + (16 * q4) % bw + r8 * bw;
    const uint32_t k_at = kt + (16 * (r8 >> 1) + (r8 & 1)) * D + 16 * q4;
    // 16-key group x of a sequence: its page, and its place in the page
    auto page_of = [&](int x) -> int { return p.page_magic ? __umulhi((uint32_t)x, p.page_magic) : x; };
    const int page16 = p.c.page / 16;
    // page of group (lane % 4) of a tile
    auto lookup = [&](const Cursor &c) -> int {
        const int x = 4 * c.t + q4;
        if (16 * x >= c.n || 16 * x + 16 <= c.lo) return -1;    // a group nobody sees: not read
        const int page = __ldg(p.c.table + (long long)c.b * p.c.max_pages + page_of(x));
        if (page < 0 || page >= p.c.num_pages) {
            atomicOr(p.c.err, kErrBadPage);
            return -1;
        }
        return page;
    };
    int pg = lookup(pc);
    float ksc = -1.f, vsc = 0.f;   // scales of group r8 / 2 (a lane's keys) of the loaded tile
    bool v_ok = false;            // the lane's 16 tokens (group q4) of it are there
    // K of the tile at pc (and its scales), then V of the same tile.  Lanes 0-3
    // copy a group of 16 keys each; groups not read are masked.
    auto load_k = [&]() __attribute__((always_inline)) {
        if (!loads) return;
        const int page = __shfl_sync(0xffffffffu, pg, r8 >> 1);   // (also: every lane has read the slot)
        const long long ph = (long long)max(page, 0) * p.c.Hkv + pc.hk;
        ksc = page >= 0 ? __ldg(p.c.k_scale + ph) : -1.f;   // negative: not read
        vsc = page >= 0 ? __ldg(p.c.v_scale + ph) : 0.f;
        const bool mine = lane < 4 && pg >= 0;
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(k_bar, n * 16 * D);
        __syncwarp();
        if (mine) {
            const int x = 4 * pc.t + lane;
            const long long row = ((long long)pg * p.c.Hkv + pc.hk) * p.c.page + 16 * (x - page_of(x) * page16);
            bulk_load(kt + lane * 16 * D, p.c.k + row * D, 16 * D, k_bar);
        }
    };
    auto load_v = [&]() __attribute__((always_inline)) {
        if (!loads) return;
        // lanes 0 .. 64 / bw - 1 copy a block of bw tokens each, if one of its
        // groups is read (the groups of a block share a page)
        v_ok = pg >= 0;
        const uint32_t ok = __ballot_sync(0xffffffffu, pg >= 0) & 15u;
        const int per = bw / 16, first = lane * per;          // the block's groups
        int page = -1;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int pgg = __shfl_sync(0xffffffffu, pg, g);
            if (g >= first && g < first + per) page = max(page, pgg);
        }
        const bool mine = lane < 64 / bw && (ok >> first & ((1u << per) - 1u)) != 0u;
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(v_bar, n * bw * D);
        __syncwarp();
        if (mine) {
            const long long ph = (long long)page * p.c.Hkv + pc.hk;
            const uint32_t dst = vt + lane * v_step;
            if (bw == p.c.page) {
                bulk_load(dst, p.c.v + ph * D * bw, bw * D, v_bar);
            } else {
                const int x = 4 * pc.t + first;
                tma_load_2d(dst, &map_v, v_bar, 16 * (x - page_of(x) * page16), (int)(ph * D));
            }
        }
        pc.next(p, s_len);
        loads = !at_end(pc);
        if (loads) pg = lookup(pc);
    };
    load_k();
    load_v();

    // ---- state of the segment being computed: row block nr, row 2 q4 + e of it
    uint32_t qb[NR][QP][K32][2];   // parts of Q (e4m3): row r8 of the block
    float fr[NR][2];             // undoes Q's power of two, times c log2(e) (or the cap's factor)
    int lo_r[NR][2], hi_r[NR][2];   // visible keys
    int lo_all = 0, hi_all = 0;     // keys every row of the worker sees
    float acc[NR][DM][4];
    float m_run[NR][2], l_run[NR][2], R[NR][2];
    bool fresh = true, begins = false;
    while (true) {
        if (fresh) {
            lo_all = 0, hi_all = 0x7fffffff;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                const int row = (cc.rg * NR + nr) * 8 + r8;
                const bool live = row < p.Sq * p.G;
                const int i = live ? row / p.G : p.Sq - 1, g = live ? row % p.G : 0;
                const T *src = reinterpret_cast<const T *>(p.q) + (((long long)cc.b * p.Sq + i) * p.Hq + cc.hk * p.G + g) * D + 16 * q4;
                uint32_t raw[HH][8];
                float amax = 0.f;
#pragma unroll
                for (int hh = 0; hh < HH; ++hh) {
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
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126);
                const float up = pow2(7 - e), down = pow2(e - 7) * (kCap ? p.cap_k : p.scale_log2);
#pragma unroll
                for (int hh = 0; hh < HH; ++hh)
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {   // words k, k + 1: four dims, register (k / 2) % 2 of k-step 2 hh + k / 4
                        const float2 a = Cvt<T>::unpack(raw[hh][k]), c = Cvt<T>::unpack(raw[hh][k + 1]);
                        float x[4] = {a.x * up, a.y * up, c.x * up, c.y * up};
#pragma unroll
                        for (int part = 0; part < QP; ++part) {
                            const uint32_t w = f32_to_e4m3x2(x[0], x[1]) | f32_to_e4m3x2(x[2], x[3]) << 16;
                            qb[nr][part][2 * hh + k / 4][(k / 2) & 1] = w;
                            uint32_t lo, hi;
                            e4m3x4_to_f16(w, lo, hi);
                            const float2 y = Cvt<__half>::unpack(lo), z = Cvt<__half>::unpack(hi);
                            x[0] = (x[0] - y.x) * 16.f, x[1] = (x[1] - y.y) * 16.f;
                            x[2] = (x[2] - z.x) * 16.f, x[3] = (x[3] - z.y) * 16.f;
                        }
                    }
                // a NaN or infinite query: what is left of it is NaN, for its own row only
                const float dn = amax < INFINITY ? down : NAN;
                const int hi = cc.n - p.Sq + i;
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {   // the rows a lane's scores belong to
                    fr[nr][e2] = __shfl_sync(0xffffffffu, dn, 4 * (2 * q4 + e2));
                    hi_r[nr][e2] = __shfl_sync(0xffffffffu, hi, 4 * (2 * q4 + e2));
                    lo_r[nr][e2] = p.window < 0 ? 0 : max(0, hi_r[nr][e2] - p.window);
                    lo_all = max(lo_all, lo_r[nr][e2]);
                    hi_all = min(hi_all, hi_r[nr][e2]);
                    m_run[nr][e2] = R[nr][e2] = -INFINITY;
                    l_run[nr][e2] = 0.f;
                }
#pragma unroll
                for (int dm = 0; dm < DM; ++dm)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[nr][dm][k] = 0.f;
            }
            lo_all = __reduce_max_sync(0xffffffffu, lo_all);
            hi_all = __reduce_min_sync(0xffffffffu, hi_all);
            begins = cc.t == cc.t0;
            fresh = false;
        }
        // ---- S^T = K Q^T
        if (!mbar_wait_warp(k_bar, phase, wctl)) break;
        float s[NR][4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t a[K32][4];
#pragma unroll
            for (int hh = 0; hh < HH; ++hh) {
                const uint4 v = ld_shared_v4(k_at + 4 * t * D + 64 * hh), u = ld_shared_v4(k_at + (4 * t + 2) * D + 64 * hh);
                a[2 * hh][0] = v.x, a[2 * hh][1] = u.x, a[2 * hh][2] = v.y, a[2 * hh][3] = u.y;
                a[2 * hh + 1][0] = v.z, a[2 * hh + 1][1] = u.z, a[2 * hh + 1][2] = v.w, a[2 * hh + 1][3] = u.w;
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                // the last part first, a sixteenth of its sum under the next
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nr][t][i] = 0.f;
#pragma unroll
                for (int q = QP - 1; q >= 0; --q) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[nr][t][i] = q < QP - 1 ? s[nr][t][i] * 0.0625f : s[nr][t][i];
#pragma unroll
                    for (int k = 0; k < K32; ++k) mma_e4m3(s[nr][t], a[k], qb[nr][q][k][0], qb[nr][q][k][1]);
                }
            }
        }
        const float ks = ksc, vs = vsc;
        const int key0 = kTile * cc.t + 16 * (r8 >> 1) + (r8 & 1);   // the lane's keys: key0 + 2 u
        const bool ends = cc.t + 1 == cc.t1;
        const bool v_here = v_ok;
        load_k();   // this tile's K has been read
        const float ev = vs > 0.f ? lg2_approx(vs) : -INFINITY;
        // a tile inside every row's keys, all its pages read, takes no compare
        const bool edge = __any_sync(0xffffffffu, ks < 0.f) || kTile * cc.t < lo_all || kTile * cc.t + kTile - 1 > hi_all;
        uint32_t pt[NR][4][2];   // P^T blocks, transposed: the B operand of O^T
        // scores in log2 units, masked; per block of rows
        auto scores = [&](auto edge_tag, int nr, float (&mx)[2]) __attribute__((always_inline)) {
            constexpr bool kEdge = decltype(edge_tag)::value;
            const uint64_t f2 = f2_pack(fr[nr][0] * ks, fr[nr][1] * ks);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                float2 x = f2_unpack(f2_mul(f2_pack(s[nr][u >> 1][2 * (u & 1)], s[nr][u >> 1][2 * (u & 1) + 1]), f2));
                const int key = key0 + 2 * u;
                const bool off0 = kEdge && (ks < 0.f || key < lo_r[nr][0] || key > hi_r[nr][0]);
                const bool off1 = kEdge && (ks < 0.f || key < lo_r[nr][1] || key > hi_r[nr][1]);
                if (kCap) {
                    // what lies behind the last token may be NaN: not into the pair
                    if (off0) x.x = 0.f;
                    if (off1) x.y = 0.f;
                    float r0, r1;
                    cap_r2(x.x, x.y, r0, r1);
                    x.x = fmaf(-2.f * p.cap_log2, r0, p.cap_log2);
                    x.y = fmaf(-2.f * p.cap_log2, r1, p.cap_log2);
                }
                if (off0) x.x = -INFINITY;
                if (off1) x.y = -INFINITY;
                s[nr][u >> 1][2 * (u & 1)] = x.x;
                s[nr][u >> 1][2 * (u & 1) + 1] = x.y;
                mx[0] = fmaxf(mx[0], x.x);
                mx[1] = fmaxf(mx[1], x.y);
            }
        };
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            float mx[2] = {-INFINITY, -INFINITY};
            if (edge) scores(std::true_type{}, nr, mx);
            else scores(std::false_type{}, nr, mx);
            // p = 2^(x - m) for the row sum; P = 2^(x + ev - R) = p 2^(ev + m - R)
            // for the product, one exp2 for both unless that factor leaves 32
            // bits (V scales more than 2^100 apart)
            float mref[2], rref[2], fv[2], grow[2];
            bool any_grow = false, wide = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float y = keys_max(mx[e] + ev);
                const float m = fmaxf(m_run[nr][e], keys_max(mx[e]));
                mref[e] = m == -INFINITY ? 0.f : m;
                l_run[nr][e] *= ex2(m_run[nr][e] - mref[e]);   // -inf before the first key: 0
                m_run[nr][e] = m;
                grow[e] = 1.f;
                if (y > R[nr][e] + kLazy || (R[nr][e] == -INFINITY && y > R[nr][e])) {
                    grow[e] = ex2(R[nr][e] - y);
                    R[nr][e] = y;
                    any_grow = true;
                }
                rref[e] = R[nr][e] == -INFINITY ? INFINITY : R[nr][e] - ev;   // no weight yet: P = 0
                wide |= mref[e] - rref[e] > 100.f;
                fv[e] = ex2(mref[e] - rref[e]);
            }
            if (__any_sync(0xffffffffu, any_grow || wide)) {
                const uint64_t g2 = f2_pack(grow[0], grow[1]);
#pragma unroll
                for (int dm = 0; dm < DM; ++dm)
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 v = f2_unpack(f2_mul(f2_pack(acc[nr][dm][k], acc[nr][dm][k + 1]), g2));
                        acc[nr][dm][k] = v.x;
                        acc[nr][dm][k + 1] = v.y;
                    }
                wide = __any_sync(0xffffffffu, wide);
            }
            const uint64_t nm = f2_pack(-mref[0], -mref[1]), f2 = f2_pack(fv[0], fv[1]);
            uint64_t sum = 0ull;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float2 x = f2_unpack(f2_add(f2_pack(s[nr][u >> 1][2 * (u & 1)], s[nr][u >> 1][2 * (u & 1) + 1]), nm));
                const uint64_t p2 = f2_pack(ex2(x.x), ex2(x.y));
                sum = f2_add(sum, p2);
                const float2 w = f2_unpack(f2_mul(p2, f2));
                pt[nr][u >> 1][u & 1] = Cvt<__half>::pack(w.x, w.y);
            }
            if (wide) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    pt[nr][u >> 1][u & 1] = Cvt<__half>::pack(ex2(s[nr][u >> 1][2 * (u & 1)] - rref[0]),
                                                              ex2(s[nr][u >> 1][2 * (u & 1) + 1] - rref[1]));
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) pt[nr][u >> 1][u & 1] = transpose8(pt[nr][u >> 1][u & 1]);
            const float2 t = f2_unpack(sum);
            l_run[nr][0] += t.x;
            l_run[nr][1] += t.y;
        }
        // ---- O^T += V^T P^T
        if (!mbar_wait_warp(v_bar, phase, wctl)) {
            ahead = loads;
            break;
        }
        phase ^= 1u;
        // tokens of the V group that some row sees: bytes before and behind them
        // hold anything (such a tile has keys a row does not see)
        const int v0 = kTile * cc.t + 16 * q4;
        const int v_from = cc.lo - v0, v_to = v_here ? cc.n - v0 : 0;
#pragma unroll
        for (int dm = 0; dm < DM; ++dm) {
            const uint4 v = ld_shared_v4(v_at + 16 * dm * bw), u = ld_shared_v4(v_at + (16 * dm + 8) * bw);
            uint32_t w[4] = {v.x, v.y, v.z, v.w}, x[4] = {u.x, u.y, u.z, u.w};
            if (edge) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t keep = bytes_below(v_to - 4 * k) & ~bytes_below(v_from - 4 * k);
                    w[k] &= keep;
                    x[k] &= keep;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t a[4];
                e4m3x4_to_f16(w[k], a[0], a[2]);
                e4m3x4_to_f16(x[k], a[1], a[3]);
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) mma_f16(acc[nr][dm], a, pt[nr][k][0], pt[nr][k][1]);
            }
        }
        load_v();
        Cursor nx = cc;
        nx.next(p, s_len);
        const bool done = at_end(nx);
        if (ends || done) {
            // the rows' results, or the piece's for the join
            const int hk = cc.hk, rg = cc.rg, seg = hk * p.groups + rg;
            const bool whole = begins && ends;
            if (!begins && lane == 0) {
                // piece 0, of a segment begun before: whose first tile's holder
                const int unit0 = (cc.b > 0 ? s_pre[cc.b - 1] : 0) * per_tile + seg * kv_units(cc.t1 - cc.t0);
                p.meta[wid] = make_int4(seg, cc.b, worker_of(unit0 + 2), ends ? 1 : 0);
            }
            const long long at = (long long)wid * 2 + (begins ? 1 : 0);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                const int row0 = (rg * NR + nr) * 8;
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float l = keys_sum(l_run[nr][e]);
                    f[e] = out_factor(R[nr][e], m_run[nr][e], l);
                    const int row = row0 + 2 * q4 + e;
                    if (r8 == 0 && row < p.Sq * p.G) {
                        if (!whole)
                            p.stat[at * (NR * 8) + nr * 8 + 2 * q4 + e] = make_float4(m_run[nr][e], l, R[nr][e], 0.f);
                        else if (p.lse)
                            p.lse[((long long)cc.b * p.Hq + hk * p.G + row % p.G) * p.Sq + row / p.G] =
                                lse_of(m_run[nr][e], l);
                    }
                }
                if (whole) {
#pragma unroll
                    for (int dm = 0; dm < DM; ++dm) {
                        // (a row without keys: its sums are 0, and so is the factor)
                        float o[4] = {acc[nr][dm][0] * f[0], acc[nr][dm][1] * f[1], acc[nr][dm][2] * f[0],
                                      acc[nr][dm][3] * f[1]};
                        store_rows<D, T>(p, cc.b, hk, row0, lane, o, dm);
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.acc + at * C::PIECE + nr * 8 * D) + lane;
#pragma unroll
                    for (int dm = 0; dm < DM; ++dm)
                        dst[32 * dm] = make_float4(acc[nr][dm][0], acc[nr][dm][1], acc[nr][dm][2], acc[nr][dm][3]);
                }
            }
            fresh = true;
        }
        if (done) return;
        cc = nx;
    }
    {
        // a wait ran out: the copies in flight land before the CTA's memory goes
        mbar_wait_drain_warp(k_bar, phase, p.c.err, p.budget_ns);
        mbar_wait_drain_warp(v_bar, phase, p.c.err, p.budget_ns);
        if (ahead) mbar_wait_drain_warp(k_bar, phase ^ 1u, p.c.err, p.budget_ns);
    }
}

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

template <int D, int NR, typename T>
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
            finish_rows<D, T>(p, x, b, seg / p.groups, row0, dm, lane);
        }
    }
}

template <int D, int NR, typename T, bool kCap>
cudaError_t launch_attn_t(KvAttnParams p, const CUtensorMap &map_v, int sms, cudaStream_t stream) {
    using C = KvCfg<D, NR>;
    auto kern = kv_attn_kernel<D, NR, T, kCap>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int grid = sms < kKvSms ? sms : kKvSms;
    p.workers = grid * C::kWarps;
    p.groups = (p.G * p.Sq + 8 * NR - 1) / (8 * NR);
    // x / (page / 16) as a product: exact for x below 2^29 and divisors up to 8
    const uint32_t d = (uint32_t)p.c.page / 16;
    p.page_magic = d > 1 ? (uint32_t)((1ull << 32) / d + 1) : 0u;
    kern<<<grid, C::kWarps * 32, C::SMEM, stream>>>(p, map_v);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.workers + kJoinWorkers - 1) / kJoinWorkers), D / 16);
    cfg.blockDim = dim3(32 * kParts);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NR, T>, p);
}

template <int D, typename T>
cudaError_t launch_attn_dt(const KvAttnParams &p, const CUtensorMap &mv, int sms, cudaStream_t stream) {
    const bool cap = p.cap_log2 > 0.f;
    if (p.G * p.Sq <= 8)
        return cap ? launch_attn_t<D, 1, T, true>(p, mv, sms, stream) : launch_attn_t<D, 1, T, false>(p, mv, sms, stream);
    return cap ? launch_attn_t<D, 2, T, true>(p, mv, sms, stream) : launch_attn_t<D, 2, T, false>(p, mv, sms, stream);
}

template <int D, typename T>
cudaError_t launch_append_t(const KvAppendParams &p, cudaStream_t stream) {
    // pages a sequence's new tokens can touch: from anywhere in the first one
    const long long per_seq = ((long long)p.max_new + p.c.page - 2) / p.c.page + 1;
    if (per_seq * p.B > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int smem = (p.max_new < p.c.page ? p.max_new : p.c.page) * D * 2;
    const dim3 grid((unsigned)(per_seq * p.B), (unsigned)p.c.Hkv, 2);
    // (a decoding step's one token a page: 5.4 us a call with 128 threads, 6.2 with 256)
    if (smem > 4096) kv_append_kernel<D, T, 256><<<grid, 256, smem, stream>>>(p, (int)per_seq);
    else kv_append_kernel<D, T, 128><<<grid, 128, smem, stream>>>(p, (int)per_seq);
    return cudaGetLastError();
}

}  // namespace

size_t kv_workspace_bytes(int D) {
    // two pieces of up to 16 rows per worker, and what its piece 0 is
    const size_t n = (size_t)kKvSms * kv_max_warps(D);
    return kv_pieces_bytes(n, D) + n * sizeof(int4);
}

cudaError_t launch_kv_append(const KvAppendParams &p, int D, int bf16, cudaStream_t stream) {
    if (D == 128)
        return bf16 ? launch_append_t<128, __nv_bfloat16>(p, stream) : launch_append_t<128, __half>(p, stream);
    return bf16 ? launch_append_t<64, __nv_bfloat16>(p, stream) : launch_append_t<64, __half>(p, stream);
}

cudaError_t launch_kv_attn(const KvAttnParams &p, const CUtensorMap &mv, int D, int bf16, int sms,
                           cudaStream_t stream) {
    if (D == 128)
        return bf16 ? launch_attn_dt<128, __nv_bfloat16>(p, mv, sms, stream)
                    : launch_attn_dt<128, __half>(p, mv, sms, stream);
    return bf16 ? launch_attn_dt<64, __nv_bfloat16>(p, mv, sms, stream)
                : launch_attn_dt<64, __half>(p, mv, sms, stream);
}

}  // namespace fa
