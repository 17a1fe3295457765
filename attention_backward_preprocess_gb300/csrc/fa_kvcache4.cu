// fa_kvcache4.cu -- the 4-bit paged key / value cache: appending to it, reading
// it back, and the attention of a sequence's last tokens over it.
//
// A value is middle + scale (c - 8) for a code c in 0 .. 15, with a bf16 (scale,
// middle) pair per 64 dims of a token.  Unsigned codes, because they reach the
// tensor core at one logical operation per two of them: below 2^11 the bits of an
// f16 number are that number in units of 2^-24, so masking a word of eight codes
// with 0x000f000f leaves two f16 operands c 2^-24, and with 0x00f000f0 two of 16 c
// 2^-24.  What the units and the 16 do is undone on the other operand or the result.
#include <atomic>
#include <type_traits>

#include "fa_device.cuh"
#include "fa_kvcache.h"
#include "fa_kvwork.cuh"
#include "fa_params.h"

namespace fa {
namespace {

// ------------------------------------------------------- rows of a ragged call
// What the append and the read have in common: rows cu[b] .. cu[b + 1] are tokens of
// sequence b, and each needs its place in the cache.
struct Ragged {
    KvCacheParams c;
    const int *cu, *len, *first;   // cu null: max_new rows each; first null: 0
    int B, rows, max_new;          // max_new < 0: a read
    // Rows [at, at + n) of a sequence as the call said, of tokens that are there (read) or
    // fit the table (append)?
    __device__ __forceinline__ bool fits(int at, int n, int held, int from) const {
        const long long cap = (long long)c.max_pages * c.page;
        if (n < 0 || at < 0 || (long long)at + n > rows || held < 0) return false;
        if (max_new < 0) return from >= 0 && (long long)from + n <= held && held <= cap;
        return n <= max_new && (long long)held + n <= cap;
    }
};

// (borders may be anything: the difference as 32 bits hold it)
__device__ __forceinline__ int rows_between(int at, int end) { return (int)((unsigned)end - (unsigned)at); }

constexpr int kRagged = 256;   // threads of a CTA
constexpr int kMaxRows = 16;   // rows of it

// Places of the CTA's rows, in tokens of one head: (page Hkv) page_size + slot, so that
// head h's is h page_size further; -1 for a row to be left alone (of no sequence, of one
// that is not as the call said, or on a bad page, which is reported).  All sequences'
// borders and lengths are read at once (up to kRagged sequences) where a search would
// read one border after the other: two dependent reads, this and the table's.
__device__ __forceinline__ void place_rows(const Ragged &r, int row0, int n_rows, long long (&s_at)[kMaxRows]) {
    __shared__ int s_cu[kRagged + 1], s_len[kRagged], s_first[kRagged], s_n[kRagged / 32];
    const int tid = threadIdx.x;
    const bool staged = r.B <= kRagged;
    int before = 0;   // sequences that end at or before row0
    if (r.cu)
        for (int b = tid; b < r.B; b += kRagged) {
            const int end = __ldg(r.cu + b + 1);
            if (staged) {
                s_cu[b + 1] = end, s_len[b] = __ldg(r.len + b), s_first[b] = r.first ? __ldg(r.first + b) : 0;
                if (b == 0) s_cu[0] = __ldg(r.cu);
            }
            before += end <= row0 ? 1 : 0;
        }
    before = __reduce_add_sync(0xffffffffu, before);
    if (tid % 32 == 0) s_n[tid / 32] = before;
    __syncthreads();
    if (tid < n_rows) {
        const int row = row0 + tid;
        int b = 0, at, n, held, from;
        auto end = [&](int i) { return staged ? s_cu[i + 1] : __ldg(r.cu + i + 1); };
        if (r.cu) {
#pragma unroll
            for (int i = 0; i < kRagged / 32; ++i) b += s_n[i];
            int hi = r.B;
            while (b < hi) {   // (the first row: b already; a later one: a few steps)
                const int mid = end(b) > row ? b : (b + hi) >> 1;
                if (end(mid) <= row) b = mid + 1;
                else hi = mid;
            }
        } else {
            b = row / r.max_new;
        }
        long long place = -1;
        if (b < r.B) {
            at = !r.cu ? b * r.max_new : staged ? s_cu[b] : __ldg(r.cu + b);
            n = !r.cu ? r.max_new : rows_between(at, end(b));
            held = r.cu && staged ? s_len[b] : __ldg(r.len + b);
            from = !r.first ? 0 : staged ? s_first[b] : __ldg(r.first + b);
            if (row >= at && r.fits(at, n, held, from)) {
                const int token = (r.max_new < 0 ? from : held) + (row - at), i = token / r.c.page;
                const int page = __ldg(r.c.table + (long long)b * r.c.max_pages + i);
                if (page < 0 || page >= r.c.num_pages) atomicOr(r.c.err, kErrBadPage);
                else place = (long long)page * r.c.Hkv * r.c.page + (token - i * r.c.page);
            }
        }
        s_at[tid] = place;
    }
    __syncthreads();
}
// Reports sequences that are not as the call said; one CTA, behind its own work.
__device__ __forceinline__ void check_ragged(const Ragged &r) {
    if (blockIdx.x != 0 || blockIdx.y != 0) return;
    for (int b = threadIdx.x; b < r.B; b += kRagged) {
        const int at = r.cu ? r.cu[b] : b * r.max_new, n = r.cu ? rows_between(at, r.cu[b + 1]) : r.max_new;
        if (!r.fits(at, n, r.len[b], r.first ? r.first[b] : 0)) atomicOr(r.c.err, kErrBadLength);
    }
}

// A thread's part of a CTA's rows: 16 dims of K or V of one head, two 16-byte pieces of a
// group of 64 dims, of every step-th row: a row costs no division.  The group's l-th of
// four threads has pieces 2 l and 2 l + 1 (kNext 1: the codes are stored in whole sectors,
// the pieces' second load meets the first one's) or l and l + 4 (kNext 4: the pieces are
// stored in whole sectors).  CTAs go over the rows along x, over rows of more than kRagged
// parts along y.
template <int D, int kNext> struct Part {
    static constexpr int CH = D / 8, N = D / 16;   // pieces and parts of a head
    int row, step, side, at;     // first row, rows from one to the next; pieces of K's (or V's) row, and the first one's place
    bool is_v, live;
    long long in_cache;          // pieces from a token's place to this one: of its head, and the dims
    __device__ __forceinline__ Part(const KvCacheParams &c) {
        side = c.Hkv * CH;
        const int all = 2 * c.Hkv * N, width = min(all, kRagged), tid = threadIdx.x;
        row = tid / width;
        step = kRagged / width;
        const int col = blockIdx.y * kRagged + tid - row * width;
        live = row < step && col < all;
        is_v = 2 * col >= all;
        const int part = col - (is_v ? all / 2 : 0), head = part / N, in = part % N / 4 * 8 + part % 4 * (kNext == 1 ? 2 : 1);
        at = head * CH + in;
        in_cache = (long long)head * c.page * CH + in;
    }
};

constexpr float kLeastScale = 0x1p-60f, kFifteenths = 8947849.f * 0x1p-26f;   // 2 / 15

template <typename T> __device__ __forceinline__ constexpr float largest() { return std::is_same_v<T, __half> ? 65504.f : 0x1.fep127f; }
// The smaller, the larger of two pairs of 16-bit floats, NaN if either is.
template <typename T> __device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T> __device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_s16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// ------------------------------------------------------------------ append
// A thread takes 16 dims of one new token; the four threads of a group of 64 share its
// least and largest value by shuffles.  Every token is written by itself, so nothing of
// the cache is read.  A thread's first loads (two tokens' parts) go out before the rows'
// places are looked up.  Prompts of 8256 tokens (8 heads of 128): 14.3 us, 43 MB.  Neither
// instructions nor occupancy bound it: 4 to 8 operations a value, four to six CTAs an
// SM and all of a thread's rows under way by asynchronous copies came out at 14.2 to 14.5.
template <int D, typename T>
__global__ void __launch_bounds__(kRagged) kv4_append_kernel(const __grid_constant__ KvAppendParams p, int per_cta) {
    __shared__ long long s_at[kMaxRows];
    constexpr int CH = D / 8, PER = 2;
    const Ragged ragged{p.c, p.cu, p.len, nullptr, p.B, p.rows, p.max_new};
    const int row0 = blockIdx.x * per_cta, rows = min(per_cta, p.rows - row0);
    const Part<D, 1> me(p.c);
    const uint4 *src = reinterpret_cast<const uint4 *>(me.is_v ? p.v : p.k) + (long long)row0 * me.side + me.at;
    uint32_t *const codes_at = reinterpret_cast<uint32_t *>(me.is_v ? p.c.v : p.c.k);
    uint32_t *const scales_at = reinterpret_cast<uint32_t *>(me.is_v ? p.c.v_scale : p.c.k_scale);
    uint4 x[PER][2];
    auto load = [&](int r0) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int r = r0 + k * me.step;
            x[k][0] = x[k][1] = make_uint4(0u, 0u, 0u, 0u);
            if (me.live && r < rows) {
                const uint4 *from = src + (long long)r * me.side;
                x[k][0] = __ldcs(from), x[k][1] = __ldcs(from + 1);
            }
        }
    };
    load(me.row);
    place_rows(ragged, row0, rows, s_at);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += PER * me.step) {   // (all threads: groups stay whole)
        if (r0 > 0) load(r0 + me.row);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int r = r0 + me.row + k * me.step;
            if (r0 + k * me.step >= rows) break;
            const uint32_t w[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
            // least and largest values of the pairs' halves; then (least, -largest) of the group: NaN
            // or infinite exactly where the group has such a value
            uint32_t a = w[0], b = w[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) a = min2_nan<T>(a, w[j]), b = max2_nan<T>(b, w[j]);
            b ^= 0x80008000u;
            uint32_t ends = min2_nan<T>(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) ends = min2_nan<T>(ends, __shfl_xor_sync(0xffffffffu, ends, o));
            const float2 lh = Cvt<T>::unpack(ends);
            const float lo = lh.x, hi = -lh.y;
            const bool bad = !(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY);
            const float mid = __bfloat162float(__float2bfloat16_rn(__fadd_rn(0.5f * lo, 0.5f * hi)));
            const float far = fmaxf(__fsub_rn(hi, mid), __fsub_rn(mid, lo)) * kFifteenths;
            const float scale = fmaxf(__uint_as_float((__float_as_uint(far) + 0xffffu) & 0xffff0000u), kLeastScale);
            const float inv = __frcp_rn(scale);
            // Rounded to nearest even by adding 1.5 2^23 (and 8): the sum's low 16 bits are the code.
            // Distances are at most 7.5 scales and a hair, so only 16 needs clamping.  (Conversions
            // run at a quarter of the rate.  Single products: a packed one and the sum behind it came out
            // rounded once.)
            const uint64_t mid2 = f2_pack(-mid, -mid), whole2 = f2_pack(12582920.f, 12582920.f);
            uint32_t c[8][2];   // of dims 2 i, + 1
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 y = Cvt<T>::unpack(w[i]);
                const float2 d = f2_unpack(f2_add(f2_pack(y.x, y.y), mid2));
                const float2 t = f2_unpack(f2_add(f2_pack(__fmul_rn(d.x, inv), __fmul_rn(d.y, inv)), whole2));
                c[i][0] = __float_as_uint(t.x), c[i][1] = __float_as_uint(t.y);
            }
            uint32_t h[2];   // eight codes each
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                h[i] = 0u;
#pragma unroll
                for (int j = 3; j >= 0; --j)   // codes j and j + 4: 16 bits apart
                    h[i] = h[i] * 16u + min_s16x2(__byte_perm(c[4 * i + j / 2][j & 1], c[4 * i + 2 + j / 2][j & 1], 0x5410), 0x000f000fu);
            }
            // The least value may be half a scale from codes 0 and 1 and rounded to 0; where the type has no such
            // value, codes 0 become 1.
            if (fmaf(-8.f, scale, mid) < -largest<T>()) {
#pragma unroll
                for (int i = 0; i < 2; ++i) h[i] |= ~(h[i] | h[i] >> 1 | h[i] >> 2 | h[i] >> 3) & 0x11111111u;
            }
            if (!me.live || r >= rows) continue;
            const long long place = s_at[r];
            if (place >= 0) {
                const long long at = place * CH + me.in_cache;
                *reinterpret_cast<uint2 *>(codes_at + at) = bad ? make_uint2(0x88888888u, 0x88888888u) : make_uint2(h[0], h[1]);
                if ((me.at & 7) == 0)
                    scales_at[at >> 3] = bad ? 0x7fc00000u | __float_as_uint(kLeastScale) >> 16
                                             : __float_as_uint(scale) >> 16 | (__float_as_uint(mid) & 0xffff0000u);
            }
        }
    }
    check_ragged(ragged);
}

// -------------------------------------------------------------------- read
// A thread takes 16 dims of one token, two words of codes and one of scale and middle in,
// two 16-byte pieces out; four tokens' at a time.  Codes become numbers in pairs, as f16 (1024 +
// c, and 1024 + 16 c over 16, less what brings them to c - 8, all exact).  With eight dims a
// thread and a shift, a mask and an addition for each code, contexts of 13 k tokens took 18.4 us
// where this takes 14.4.
template <int D, typename T>
__global__ void __launch_bounds__(kRagged) kv4_read_kernel(const __grid_constant__ KvReadParams p, int per_cta) {
    __shared__ long long s_at[kMaxRows];
    constexpr int CH = D / 8, PER = 4;
    const Ragged ragged{p.c, p.cu, p.len, p.first, p.B, p.rows, -1};
    const int row0 = blockIdx.x * per_cta, rows = min(per_cta, p.rows - row0);
    const Part<D, 4> me(p.c);
    const uint32_t *const codes_at = reinterpret_cast<const uint32_t *>(me.is_v ? p.c.v : p.c.k);
    const uint32_t *const scales_at = reinterpret_cast<const uint32_t *>(me.is_v ? p.c.v_scale : p.c.k_scale);
    uint4 *const dst = reinterpret_cast<uint4 *>(me.is_v ? p.v : p.k) + (long long)row0 * me.side + me.at;
    place_rows(ragged, row0, rows, s_at);
    if (me.live) {
#pragma unroll 1
        for (int r0 = me.row; r0 < rows; r0 += PER * me.step) {
            uint32_t c[PER][2], sm[PER];
            bool there[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int r = r0 + k * me.step;
                const long long place = r < rows ? s_at[r] : -1;
                there[k] = place >= 0;
                if (there[k]) {
                    const long long at = place * CH + me.in_cache;
                    c[k][0] = __ldcs(codes_at + at), c[k][1] = __ldcs(codes_at + at + 4);
                    sm[k] = __ldg(scales_at + (at >> 3));
                }
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (!there[k]) continue;
                const float scale = __uint_as_float(sm[k] << 16), mid = __uint_as_float(sm[k] & 0xffff0000u);
                uint4 *const to = dst + (long long)(r0 + k * me.step) * me.side;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {   // codes j and j + 4
                        const uint32_t w = c[k][i] >> (8 * (j >> 1)), v = (w & (j & 1 ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
                        const __half2 n = *reinterpret_cast<const __half2 *>(&v);
                        const float2 y = __half22float2(j & 1 ? __hfma2(n, __half2half2(__ushort_as_half(0x2c00)), __half2half2(__ushort_as_half(0xd480)))
                                                              : __hadd2(n, __half2half2(__ushort_as_half(0xe408))));
                        const float2 x = f2_unpack(f2_fma(f2_pack(scale, scale), f2_pack(y.x, y.y), f2_pack(mid, mid)));
                        f[j] = x.x, f[j + 4] = x.y;
                    }
                    __stcs(to + 4 * i, make_uint4(Cvt<T>::pack(f[0], f[1]), Cvt<T>::pack(f[2], f[3]), Cvt<T>::pack(f[4], f[5]),
                                                  Cvt<T>::pack(f[6], f[7])));
                }
            }
        }
    }
    check_ragged(ragged);
}

// --------------------------------------------------------------- attention
// The rows of a kv head's query group times Sq tokens lie along N of m16n8k16
// products, keys (then dims) along M, and the work is shared out as in the 8-bit kernel:
// every warp a worker with a contiguous share of all 64-key tiles.  Bytes should bound
// it (D + D / 8 per key against 4 D flops per row and key); a key's codes take about as
// many instructions to multiply as the memory takes cycles to bring them, so the design
// spares instructions, and each worker has a ring of tiles (codes of K and V, their scales)
// in shared memory, all but one under way.  Four more warps look up the pages and start the
// copies, two workers' each; the workers take over most of their registers.
//
// S^T.  A key's row of codes is D / 2 bytes; ldmatrix hands lane (r8, q4) the word
// of dims 32 j + 8 q4 .. + 7 of key r8: masked, the operands (d0, d4), 16 (d1, d5),
// (d2, d6), 16 (d3, d7).  The contracted axis may be permuted and scaled as long as
// Q's side agrees: Q lies as f16 under a power of two per row that brings its largest
// value to [2^14, 2^15), the odd dims at a sixteenth.  (bf16's 8 bits and f16's 11 fit
// but for values 2^29 below the row's largest.)  A group's part of the score is scale a +
// (middle - 8 scale) Q_g, a from the product and Q_g the sum of Q over the group.  The second
// term is a product of its own: the keys' (scale, middle) words as they lie, two bf16 operands,
// against (-8 Q_g, Q_g) in three bf16 parts.
//
// O^T.  ldmatrix.trans hands lane (r8, q4) 16-bit pieces of tokens 2 q4, + 1: dims 32
// j + 4 r8 .. + 3 of both, which masked are operands of one dim (or 16 times it) of
// two neighbouring tokens, so P^T is needed in the keys' own order and the 16 falls
// on whole rows of the result.  V's scales go into P: P_g = p scale_g in f16, at most
// 2^14 against a running reference R of score + log2(largest scale of the key); p's own
// reference, for sums and middles, is the score alone.  The middles' part, sum p middle_g,
// is kept in 32 bits per row and group, and so is 8 sum P_g, by a product with a
// constant operand, from the rounded P_g that the codes were multiplied with: the two
// cancel as exactly as the codes demand.
//
// Codes are finite whatever their bits, so only scores and scales of hidden keys
// are masked.
//
// Measured (64 requests of 256 to 8192 tokens, 32 / 8 heads of 128; two of 64 k capped),
// the call with its join: 41.2 and 31.1 us, 4.07 TB/s and 3.45; three rows of 8 / 2 heads of
// 64 over 200 tokens 12.3.  By events around the call, which add 9 us, over 140 k tokens in 64
// requests: 32, 64 and 128 heads on 8 (4, 8, 16 rows) 50.2, 50.2 and 66.8 us (capped 50.2, 52.2, 75.8).
// What else was measured (against 41.0, 31.0 and 12.3):
//   each worker starting its own copies: 41.6, 32.8 and 14.3;
//   and with that: scores by e4m3 products (Q in parts, three operations a word of codes
//   where f16 takes five): 57 us where f16 took 47;
//   12 workers an SM (16 or 32 keys at a time fit 168 registers): 44.9 and 34.6; 10: 50.4 and
//   37.4; 6: 54 and 39; one tile a worker: 50.9 and 39;
//   rows 4 .. 7 left idle where there are four (kSplit): 45.1 and 34.8.
// Three tiles a worker: 43.3 and 31.9.
constexpr uint32_t kLoMask = 0x000f000fu, kHiMask = 0x00f000f0u;
// R is at most this far below m, so that 2^(m - R + 6) p stays in 32 bits where the top keys' V scales
// are 0: what scales of 2^-100 reach, and the references' slack.  What P_g loses to it weighs below 2^-130.
constexpr float kFarBelow = 108.f;

constexpr int kKv4Smem = 232448 - 1024;   // of a CTA, what is not dynamic set aside

template <int D, int NR>
struct Kv4Cfg {
    static constexpr int kWarps = 8, kThreads = (kWarps + 4) * 32;   // workers; and the four warps that load
    // Registers of a thread: as launched (what three warps a scheduler may have), a worker's, a loading warp's.
    static constexpr int kRegs = 168, kWorkRegs = 224, kLoadRegs = 56;
    static_assert(kWarps * kWorkRegs + 4 * kLoadRegs <= (kWarps + 4) * kRegs, "the launch's registers are shared out");
    static constexpr int kStep = NR == 1 ? 4 : 2;   // 16-key products at a time
    static constexpr int KB = kTile * D / 2;             // codes of a K (or V) tile
    static constexpr int SB = kTile * (D / 64) * 4;      // its scales
    static constexpr int STAGE = 2 * (KB + SB);
    static constexpr int kStages = D == 64 ? 4 : 2;
    // shared memory of a CTA for B sequences (1008: to a whole pattern)
    static constexpr int smem(int B) { return 1008 + kWarps * kStages * STAGE + 8 * B; }
    static_assert(smem(kKvMaxSeqs) <= kKv4Smem, "shared memory overflow");
    static_assert(kWarps <= kKv4MaxWarps, "the workspace holds that many workers per SM");
    static_assert(STAGE % 512 == 0 && KB % 512 == 0, "swizzled tiles start on whole patterns");
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t row_addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(row_addr)
                 : "memory");
}
__device__ __forceinline__ void ld_shared_words(uint32_t addr, uint32_t (&v)[1]) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ld_shared_words(uint32_t addr, uint32_t (&v)[2]) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float log2_scale(float x) {   // (below 2^-126: -inf)
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float scale_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float middle_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Q's operands from a row's dims 32 j + 8 q4 .. + 7, `up` its power of two: the two
// registers each of the two products of a chunk; what they sum to is added to `sum`.
template <typename T>
__device__ __forceinline__ void q_operands(uint4 raw, float up, uint32_t (&b)[4], float &sum) {
    const float2 a = Cvt<T>::unpack(raw.x), c = Cvt<T>::unpack(raw.y), d = Cvt<T>::unpack(raw.z), e = Cvt<T>::unpack(raw.w);
    const float od = up * 0.0625f;
    b[0] = Cvt<__half>::pack(a.x * up, d.x * up);   // dims 0, 4
    b[1] = Cvt<__half>::pack(a.y * od, d.y * od);   // dims 1, 5
    b[2] = Cvt<__half>::pack(c.x * up, e.x * up);   // dims 2, 6
    b[3] = Cvt<__half>::pack(c.y * od, e.y * od);   // dims 3, 7
    sum += up * (((a.x + a.y) + (c.x + c.y)) + ((d.x + d.y) + (e.x + e.y)));
}

// Two dims of two rows: v is (row 2 q4, dim d), (row + 1, d), (row, d + 1), (row + 1, d + 1)
// with d = 32 (dm / 2) + 4 r8 + 2 (dm % 2).
template <int D, typename T>
__device__ __forceinline__ void store_pairs(const KvAttnParams &p, int b, int hk, int row0, int lane, float4 v, int dm) {
    const int row = row0 + 2 * (lane & 3), d = 32 * (dm >> 1) + 4 * (lane >> 2) + 2 * (dm & 1);
    const uint32_t w[2] = {Cvt<T>::pack(v.x, v.z), Cvt<T>::pack(v.y, v.w)};
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (row + e < p.Sq * p.G) {
            const int i = (row + e) / p.G, hq = hk * p.G + (row + e) % p.G;
            *reinterpret_cast<uint32_t *>(reinterpret_cast<T *>(p.o) + (((long long)b * p.Sq + i) * p.Hq + hq) * D + d) = w[e];
        }
}

// Does the phase of that parity lie behind?  (Without waiting.)
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Waits for a phase, within the budget and, if it heeds an abort, until there is one.
// (Inline: no calls where warps have registers of their own number.)
template <bool kHeeds>
__device__ __forceinline__ bool kv4_wait(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    uint64_t since = 0;
#pragma unroll 1
    for (int i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (i & 31) continue;
        if (kHeeds && *w.abort_flag) return false;
        const uint64_t now = globaltimer_ns();
        if (since == 0) since = now;
        if ((long long)(now - since) > w.budget_ns) {
            raise_error(w, kErrWaitTimeout);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool kv4_wait_warp(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    int ok = 1;
    if ((threadIdx.x & 31) == 0) ok = kv4_wait<true>(bar, parity, w);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();   // (what lane 0 has waited for is there for all lanes: a shuffle alone orders no memory)
    return ok != 0;
}

// The warps that load the workers' tiles, two workers each: lane 16 j + 4 i + k copies part k
// (K's codes, V's codes, K's scales, V's) of block i (bw tokens of one page) of worker 2 warp + j's.
template <int D, int NR>
__device__ __forceinline__ void kv4_loads(const KvAttnParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v,
                                          const int *s_pre, const int *s_len, int per_tile, int total, uint32_t tiles,
                                          uint32_t full, uint32_t empty, uint32_t *s_ok, int warp, int lane, const WaitCtl &wctl) {
    using C = Kv4Cfg<D, NR>;
    constexpr int GR = D / 64, ST = C::kStages;
    static_assert(C::kWarps == 8, "two workers a loading warp");
    const int half = lane & 16, worker = 2 * warp + (lane >> 4), blk = lane >> 2 & 3, part = lane & 3;
    const bool leads = (lane & 15) == 0;
    Cursor pc, end;   // what is loaded next, and where the worker stops
    bool left;
    {
        const KvShare sh(p, blockIdx.x * C::kWarps + worker, total);
        left = sh.wid < sh.N && total > 0;
        Cursor c;   // even lanes place the one, odd lanes the other
        c.b = c.hk = c.rg = c.t = 0;
        if (left) kv_place<kKv4Open>(p, s_pre, s_len, per_tile, lane & 1 ? sh.w1 : sh.w0, c);
        __syncwarp();
        auto from = [&](int src, Cursor &d) {
            d.b = __shfl_sync(0xffffffffu, c.b, src), d.hk = __shfl_sync(0xffffffffu, c.hk, src);
            d.rg = __shfl_sync(0xffffffffu, c.rg, src), d.t = __shfl_sync(0xffffffffu, c.t, src);
        };
        from(half, pc);
        from(half + 1, end);
        const int t = pc.t;
        if (left && pc.b < p.B) pc.open(p, s_len);
        pc.t = t;
    }
    auto at_end = [&]() -> bool { return pc.b == end.b && pc.hk == end.hk && pc.rg == end.rg && pc.t == end.t; };
    left = left && !at_end();
    const int bw = p.v_block, page16 = p.c.page / 16;
    auto page_of = [&](int x) -> int { return p.page_magic ? __umulhi((uint32_t)x, p.page_magic) : x; };
    // The page of the lane's block of the tile at pc, -1 if no query sees it.
    auto lookup = [&]() __attribute__((always_inline)) -> int {
        const int x = 4 * pc.t + blk * (bw / 16);
        if (blk * bw >= 64 || 16 * x >= pc.n || 16 * x + bw <= pc.lo) return -1;
        const int page = __ldg(p.c.table + (long long)pc.b * p.c.max_pages + page_of(x));
        if (page < 0 || page >= p.c.num_pages) {
            atomicOr(p.c.err, kErrBadPage);
            return -1;
        }
        return page;
    };
    // where the lane's copies land in a stage, and its part's scales
    const uint32_t ring = tiles + worker * (ST * C::STAGE) + (part < 2 ? part * C::KB + blk * bw * (D / 2)
                                                                       : 2 * C::KB + (part & 1) * C::SB + blk * bw * (4 * GR));
    const uint32_t *const scales = reinterpret_cast<const uint32_t *>(part & 1 ? p.c.v_scale : p.c.k_scale);
    full += worker * (8 * C::kStages), empty += worker * (8 * C::kStages), s_ok += worker * C::kStages;
    int pg = left ? lookup() : -1, s = 0, loaded = 0, idle = 0;
    uint32_t phase = 0;
    uint64_t since = 0;
    while (__any_sync(0xffffffffu, left)) {
        bool go = left && leads && mbar_test(empty + 8 * s, phase ^ 1u);
        go = __shfl_sync(0xffffffffu, go, half);
        if (!__any_sync(0xffffffffu, go)) {
            if ((++idle & 255) == 0) {   // (the workers' own waits are bounded: a second bound)
                const uint64_t now = globaltimer_ns();
                if (since == 0) since = now;
                if (twice_over(now - since, p.budget_ns)) raise_error(wctl, kErrWaitTimeout);
                __syncwarp();
            }
            if (__any_sync(0xffffffffu, *wctl.abort_flag != 0)) break;
            __nanosleep(40);
            continue;
        }
        idle = 0, since = 0;
        const uint32_t b = __ballot_sync(0xffffffffu, pg >= 0 && part == 0) >> half;
        if (go && leads) {
            s_ok[s] = (b & 1u) | (b >> 3 & 2u) | (b >> 6 & 4u) | (b >> 9 & 8u);
            mbar_arrive_expect_tx(full + 8 * s, (uint32_t)(__popc(b & 0xffffu) * bw) * (D + 8 * GR));
        }
        __syncwarp();
        if (go) {
            if (pg >= 0) {
                const int x = 4 * pc.t + blk * (bw / 16);
                const int row = (pg * p.c.Hkv + pc.hk) * p.c.page + 16 * (x - page_of(x) * page16);   // (below 2^31)
                const uint32_t dst = ring + s * C::STAGE;
                if (part < 2) tma_load_2d(dst, part ? &map_v : &map_k, full + 8 * s, 0, row);
                else bulk_load(dst, scales + (long long)row * GR, bw * 4 * GR, full + 8 * s);
            }
            ++loaded;
            if (++s == ST) s = 0, phase ^= 1u;
            pc.next(p, s_len);
            left = !at_end();
            if (left) pg = lookup();
        }
        __syncwarp();
    }
    if (leads)   // the copies in flight land before the CTA's memory goes, whatever the workers do
        for (int k = max(loaded - ST, 0); k < loaded; ++k)
            kv4_wait<false>(full + 8 * (k % ST), k / ST & 1, wctl);
}

// kSplit: at most four rows (NR is 1).  Lanes q4 >= 2, whose rows 4 .. 7 there are not, take
// the softmax of every second 16 keys off their neighbours q4 - 2.
template <int D, int NR, typename T, bool kCap, bool kSplit>
__global__ void __launch_bounds__(Kv4Cfg<D, NR>::kThreads, 1)
    kv4_attn_kernel(const __grid_constant__ KvAttnParams p, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v) {
    using C = Kv4Cfg<D, NR>;
    constexpr int W = C::kWarps, KS = C::kStep, J = D / 32, GR = D / 64, DM = D / 16, ST = C::kStages;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ int s_warp[W + 4];
    __shared__ __align__(8) uint64_t s_full[W][C::kStages], s_empty[W][C::kStages];   // a stage's tile landed, was used
    __shared__ uint32_t s_ok[W][C::kStages];   // its blocks that were read
    __shared__ int s_abort;
    const uint32_t tiles = (smem_u32(smem_raw) + 1023u) & ~1023u;
    int *s_pre = reinterpret_cast<int *>(smem_raw + (tiles - smem_u32(smem_raw)) + W * ST * C::STAGE), *s_len = s_pre + p.B;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int r8 = lane >> 2, q4 = lane & 3;
    // the rows a lane's scores belong to: 2 qr, + 1; which of two 16-key products it takes (kSplit)
    const int qr = kSplit ? q4 & 1 : q4, odd = kSplit ? q4 >> 1 : 0;
    static_assert(!kSplit || (NR == 1 && KS % 2 == 0), "pairs of products");
    constexpr int KU = kSplit ? KS / 2 : KS;   // 16-key products whose softmax a lane takes part in

    // The block table and Q on their way from memory while the lengths are read: a line a
    // thread (what lies further comes when it is wanted).
    {
        const long long line = (long long)(blockIdx.x * C::kThreads + threadIdx.x) * 128;
        if (line < (long long)p.B * p.c.max_pages * 4)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(p.c.table) + line));
        if (line < (long long)p.B * p.Sq * p.Hq * D * 2)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char *>(p.q) + line));
    }
    if (threadIdx.x == 32) prefetch_tmap(&map_k), prefetch_tmap(&map_v);
    if (threadIdx.x == 0) s_abort = 0;
    if (warp < W) {
        if (lane == 0) p.meta[blockIdx.x * W + warp] = make_int4(-1, 0, 0, 0);
        if (lane < ST) {
            mbar_init(smem_u32(&s_full[warp][lane]), 1);
            mbar_init(smem_u32(&s_empty[warp][lane]), 1);
            fence_mbar_init();
        }
    }
    const int per_tile = p.c.Hkv * p.groups;
    const int total = kv_count<W + 4, D, kKv4Open>(p, s_pre, s_len, s_warp, warp, lane) * per_tile;   // (the host keeps it below 2^31)
    pdl_launch();
    const WaitCtl wctl{&s_abort, p.c.err, p.budget_ns};
    if (warp >= W) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLoadRegs));
        kv4_loads<D, NR>(p, map_k, map_v, s_pre, s_len, per_tile, total, tiles, smem_u32(&s_full[0][0]), smem_u32(&s_empty[0][0]),
                         &s_ok[0][0], warp - W, lane, wctl);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kWorkRegs));
    const int wid = blockIdx.x * W + warp;
    const KvShare sh(p, wid, total);
    if (wid >= sh.N || total == 0) return;
    Cursor cc, end;   // what is computed next, and where the worker stops
    {
        Cursor c;   // even lanes place the one, odd lanes the other
        kv_place<kKv4Open>(p, s_pre, s_len, per_tile, lane & 1 ? sh.w1 : sh.w0, c);
        auto from = [&](int src, Cursor &d) {
            d.b = __shfl_sync(0xffffffffu, c.b, src), d.hk = __shfl_sync(0xffffffffu, c.hk, src);
            d.rg = __shfl_sync(0xffffffffu, c.rg, src), d.t = __shfl_sync(0xffffffffu, c.t, src);
        };
        from(0, cc);
        from(1, end);
        const int t = cc.t;
        if (cc.b < p.B) cc.open(p, s_len);
        cc.t = t;
    }
    auto at_end = [&](const Cursor &c) -> bool {
        return c.b == end.b && c.hk == end.hk && c.rg == end.rg && c.t == end.t;
    };
    if (at_end(cc)) return;

    const uint32_t ring = tiles + warp * (ST * C::STAGE);
    const uint32_t full = smem_u32(&s_full[warp][0]), empty = smem_u32(&s_empty[warp][0]);
    float2 *const stat = reinterpret_cast<float2 *>(p.stat);   // (m, l) of a piece's rows
    const int bw = p.v_block;
    const uint32_t whole_tile = (1u << (64 / bw)) - 1u;
    // Q's rows of the segment that comes next, on their way to this SM: lane (r8, q4) a quarter
    // of row r8
    auto prefetch_q = [&](const Cursor &c) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = (c.rg * NR + nr) * 8 + r8;
            if (row < p.Sq * p.G) {
                const uint16_t *src = reinterpret_cast<const uint16_t *>(p.q) +
                                      (((long long)c.b * p.Sq + row / p.G) * p.Hq + c.hk * p.G + row % p.G) * D + q4 * (D / 4);
                asm volatile("prefetch.global.L1 [%0];" ::"l"(src));
            }
        }
    };
    // ldmatrix: lane l gives the address of row l % 8 of matrix l / 8, matrices being the
    // 16-byte chunks of eight keys (D = 64: of sixteen).  Chunks lie as the tensor loads
    // swizzle them: chunk c of row r at c ^ (r / 2 % 4) (64-byte rows), c ^ (r / 4 % 2) (32).
    const int lr = lane & 7, lm = lane >> 3;
    const uint32_t lm_at = D == 128 ? lr * 64 + ((lm ^ (lr >> 1)) << 4)
                                    : ((lm >> 1) * 8 + lr) * 32 + (((lm & 1) ^ (lr >> 2)) << 4);

    // over the lanes that hold a row's keys
    auto row_max = [&](float v) __attribute__((always_inline)) -> float {
        v = keys_max(v);
        return kSplit ? fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2)) : v;
    };
    auto row_sum = [&](float v) __attribute__((always_inline)) -> float {
        v = keys_sum(v);
        return kSplit ? v + __shfl_xor_sync(0xffffffffu, v, 2) : v;
    };
    // ---- state of the segment being computed: row block nr, row 2 qr + e of it
    uint32_t qb[NR][J][4];       // Q's operands
    uint32_t qz[NR][2];          // its sums per group, as the operand of scales and middles
    float fr[NR][2];             // undoes the units and Q's power of two, times c log2(e) (or the cap's factor); > 0
    int lo_r[NR][2], hi_r[NR][2];   // visible keys
    int lo_all = 0, hi_all = 0;     // keys every row of the worker sees
    float acc[NR][DM][4];        // 2^-24 sum P_g c: dims 32 (dm / 2) + 4 r8 + 2 (dm % 2), and 16 times the next
    float eight[NR][GR][4];      // 2^-24 8 sum P_g
    float zc[NR][GR][2];         // the lane's part of sum p middle_g
    float m[NR][2], R[NR][2];    // what p = 2^(score - m) and P_g = 2^(score - R + 6) scale_g refer to
    float mr[NR][2], fv[NR][2];  // m (0 before the first key), 2^(m - R + 6) (0 before the first scale)
    float l_run[NR][2];          // the lane's part of sum p
    bool fresh = true, begins = false;
    int s_at = 0;
    uint32_t phase = 0;   // of stage s_at's barrier
    while (true) {
        if (fresh) {
            lo_all = 0, hi_all = 0x7fffffff;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                const int row = (cc.rg * NR + nr) * 8 + r8;
                const bool live = row < p.Sq * p.G;
                const int i = live ? row / p.G : p.Sq - 1, g = live ? row % p.G : 0;
                const T *src = reinterpret_cast<const T *>(p.q) + (((long long)cc.b * p.Sq + i) * p.Hq + cc.hk * p.G + g) * D + 8 * q4;
                uint4 raw[J];
                uint32_t top = 0u;   // largest magnitudes as bits
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    raw[j] = live ? __ldg(reinterpret_cast<const uint4 *>(src + 32 * j)) : make_uint4(0, 0, 0, 0);
                    top = max_u16x2(max_u16x2(top, raw[j].x & 0x7fff7fffu), raw[j].y & 0x7fff7fffu);
                    top = max_u16x2(max_u16x2(top, raw[j].z & 0x7fff7fffu), raw[j].w & 0x7fff7fffu);
                }
                top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
                top = max(top >> 16, top & 0xffffu);
                const float amax = Cvt<T>::unpack(top).x;
                const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126);
                // (down: the smaller products first, and held within the finite numbers above 0: a row of next to
                // nothing scores 0, and a hidden key's -inf stays what it is)
                const float up = pow2(14 - e), c = kCap ? p.cap_k : p.scale_log2;
                const float down = fminf(fmaxf(e < 14 ? pow2(e - 14) * 0x1p24f * c : pow2(e - 14) * c * 0x1p24f, 0x1p-126f), 0x1.fffffep127f);
                float sum[2] = {0.f, 0.f};
                // A NaN or infinite query goes on as zeros (a NaN would get past the -inf of keys that it does not
                // see); its row sum is NaN where it sees a key.
                const bool fine = amax < INFINITY;
#pragma unroll
                for (int j = 0; j < J; ++j)
                    q_operands<T>(fine ? raw[j] : make_uint4(0u, 0u, 0u, 0u), fine ? up : 1.f, qb[nr][j], sum[j / 2]);
                const float dn = fine ? down : 1.f;
                const int hi = cc.n - p.Sq + i;
                const float l0 = fine || hi < 0 ? 0.f : NAN;
#pragma unroll
                for (int g2 = 0; g2 < GR; ++g2) {
                    sum[g2] += __shfl_xor_sync(0xffffffffu, sum[g2], 1);
                    sum[g2] += __shfl_xor_sync(0xffffffffu, sum[g2], 2);
                }
                // (-8 Q_g, Q_g) against a key's (scale, middle) pairs: Q_g as three bf16 parts, lane q4
                // the first or second part of group q4 % 2 and (below) the third (one group: part q4)
                {
                    const float z0 = sum[GR == 2 ? q4 & 1 : 0] * 0x1p-24f;
                    const float p0 = Cvt<__nv_bfloat16>::unpack(Cvt<__nv_bfloat16>::pack(z0, 0.f)).x;
                    const float p1 = Cvt<__nv_bfloat16>::unpack(Cvt<__nv_bfloat16>::pack(z0 - p0, 0.f)).x;
                    const float p2 = Cvt<__nv_bfloat16>::unpack(Cvt<__nv_bfloat16>::pack(z0 - p0 - p1, 0.f)).x;
                    const int part = GR == 2 ? q4 >> 1 : q4;
                    const float a = part == 0 ? p0 : part == 1 ? p1 : part == 2 ? p2 : 0.f, b = GR == 2 && q4 < 2 ? p2 : 0.f;
                    qz[nr][0] = Cvt<__nv_bfloat16>::pack(-8.f * a, a);
                    qz[nr][1] = Cvt<__nv_bfloat16>::pack(-8.f * b, b);
                }
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {   // the rows a lane's scores belong to
                    const int src_lane = 4 * (2 * qr + e2);
                    fr[nr][e2] = __shfl_sync(0xffffffffu, dn, src_lane);
                    hi_r[nr][e2] = __shfl_sync(0xffffffffu, hi, src_lane);
                    lo_r[nr][e2] = p.window < 0 ? 0 : max(0, hi_r[nr][e2] - p.window);
                    lo_all = max(lo_all, lo_r[nr][e2]);
                    hi_all = min(hi_all, hi_r[nr][e2]);
                    m[nr][e2] = R[nr][e2] = -INFINITY;
                    mr[nr][e2] = fv[nr][e2] = 0.f;
                    l_run[nr][e2] = __shfl_sync(0xffffffffu, l0, src_lane);
#pragma unroll
                    for (int g2 = 0; g2 < GR; ++g2) zc[nr][g2][e2] = 0.f;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int dm = 0; dm < DM; ++dm) acc[nr][dm][k] = 0.f;
#pragma unroll
                    for (int g2 = 0; g2 < GR; ++g2) eight[nr][g2][k] = 0.f;
                }
            }
            lo_all = __reduce_max_sync(0xffffffffu, lo_all);
            hi_all = __reduce_min_sync(0xffffffffu, hi_all);
            begins = cc.t == cc.t0;
            fresh = false;
        }
        Cursor nx = cc;
        nx.next(p, s_len);
        const bool done = at_end(nx), ends = cc.t + 1 == cc.t1;
        if (ends && !done) prefetch_q(nx);
        if (!kv4_wait_warp(full + 8 * s_at, phase, wctl)) return;   // (the copies in flight: the loading warp waits for them)
        const uint32_t kt = ring + s_at * C::STAGE, vt = kt + C::KB;
        const uint32_t ks_at = kt + 2 * C::KB + r8 * (4 * GR), vs_at = ks_at + C::SB;
        const uint32_t ok = *reinterpret_cast<volatile uint32_t *>(&s_ok[warp][s_at]);
        // a tile inside every row's keys, all its pages read, takes no compare
        const bool edge = ok != whole_tile || kTile * cc.t < lo_all || kTile * cc.t + kTile - 1 > hi_all;
#pragma unroll 1
        for (int t0 = 0; t0 < 4; t0 += KS) {
            // ---- S^T = K Q^T: scores of keys 16 t + r8 (+ 8), rows 2 q4, + 1
            float x[NR][KS][4];
            uint32_t vsm[2 * KU][GR];   // V's (scale, middle) of the lane's keys, 0 for keys nobody sees
            // product of its keys u (two each): rows r8 (+ 8) of it
            auto tile_of = [&](int u) __attribute__((always_inline)) -> int { return t0 + (kSplit ? (u & ~1) + odd : u >> 1); };
#pragma unroll
            for (int u = 0; u < 2 * KU; ++u) ld_shared_words(vs_at + (16 * tile_of(u) + 8 * (u & 1)) * (4 * GR), vsm[u]);
#pragma unroll
            for (int tt = 0; tt < KS; ++tt) {
                const uint32_t at = kt + (t0 + tt) * (16 * D / 2) + lm_at;
                uint32_t w[2][J];   // key r8, key r8 + 8: the words of chunk j
                if constexpr (D == 128) {
                    ldmatrix_x4(at, w[0]);
                    ldmatrix_x4(at + 512, w[1]);
                } else {
                    uint32_t r[4];
                    ldmatrix_x4(at, r);
                    w[0][0] = r[0], w[0][1] = r[1], w[1][0] = r[2], w[1][1] = r[3];
                }
                uint32_t sm[2][GR];   // (scale, middle) of keys r8, r8 + 8
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) ld_shared_words(ks_at + (16 * (t0 + tt) + 8 * hh) * (4 * GR), sm[hh]);
                float a[NR][GR][4];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int g = 0; g < GR; ++g)
#pragma unroll
                        for (int k = 0; k < 4; ++k) a[nr][g][k] = 0.f;
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = w[0][j] >> (8 * h), v = w[1][j] >> (8 * h);
                        const uint32_t A[4] = {u & kLoMask, v & kLoMask, u & kHiMask, v & kHiMask};
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) mma_f16(a[nr][j / 2], A, qb[nr][j][2 * h], qb[nr][j][2 * h + 1]);
                    }
                const uint32_t w0 = GR == 2 && (q4 & 1) ? sm[0][GR - 1] : sm[0][0], w1 = GR == 2 && (q4 & 1) ? sm[1][GR - 1] : sm[1][0];
                const uint32_t Z[4] = {w0, w1, w0, w1};
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float y[4] = {0.f, 0.f, 0.f, 0.f};   // sum over the groups of (middle - 8 scale) Q_g
                    mma_bf16(y, Z, qz[nr][0], qz[nr][1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int g = 0; g < GR; ++g) y[k] = fmaf(scale_of(sm[k >> 1][g]), a[nr][g][k], y[k]);
                        x[nr][tt][k] = y[k];
                    }
                }
            }
            if (kSplit) {
#pragma unroll
                for (int i = 0; i < KU; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float own = x[0][2 * i][k], other = x[0][2 * i + 1][k];
                        const float got = __shfl_xor_sync(0xffffffffu, other, 2);   // (of lanes q4 < 2; they ignore theirs)
                        x[0][i][k] = odd ? got : own;
                    }
            }
            // ---- softmax, and V's scales
            uint32_t hidden = 0u;   // (under a cap) a bit per score
            if (edge) {
                const int per = bw / 16;
#pragma unroll
                for (int u = 0; u < 2 * KU; ++u) {
                    const int t = tile_of(u), key = kTile * cc.t + 16 * t + 8 * (u & 1) + r8;
                    const bool gone = !(ok >> (per == 4 ? 0 : per == 2 ? t >> 1 : t) & 1u) || key >= cc.n || key < cc.lo;
#pragma unroll
                    for (int g = 0; g < GR; ++g) vsm[u][g] = gone ? 0u : vsm[u][g];
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (gone || key < lo_r[nr][e] || key > hi_r[nr][e]) {
                                // (what lies behind the last token may be NaN: not into the cap's pair)
                                x[nr][u >> 1][2 * (u & 1) + e] = kCap ? 0.f : -INFINITY;
                                if (kCap) hidden |= 1u << ((nr * 2 * KU + u) * 2 + e);
                            }
                }
            }
            float top = 0.f;   // largest scale of the lane's keys
#pragma unroll
            for (int u = 0; u < 2 * KU; ++u)
                top = GR == 2 ? max3(top, scale_of(vsm[u][0]), scale_of(vsm[u][GR - 1])) : fmaxf(top, scale_of(vsm[u][0]));
            const float ev = log2_scale(top);
            uint32_t pt[NR][GR][2 * KU];   // P_g^T blocks, transposed: the B operands of O^T
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                if (kCap) {
#pragma unroll
                    for (int i = 0; i < KU; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {   // (a pair is of two keys: a row's scores are its own affair)
                            float &a = x[nr][i][e], &b = x[nr][i][2 + e], ra, rb;
                            cap_r2(a * fr[nr][e], b * fr[nr][e], ra, rb);
                            a = fmaf(-2.f * p.cap_log2, ra, p.cap_log2);
                            b = fmaf(-2.f * p.cap_log2, rb, p.cap_log2);
                            if (edge && (hidden >> ((nr * KU + i) * 4 + e) & 1u)) a = -INFINITY;
                            if (edge && (hidden >> ((nr * KU + i) * 4 + e) & 4u)) b = -INFINITY;
                        }
                }
                // The references move only where a lane's largest score, or that plus its
                // largest log2 scale, is 8 above them: mostly in a segment's first tile.
                // (R then to the largest sum of a key's own two.)
                float mx[2];
                bool moves = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float y = fmaxf(x[nr][0][e], x[nr][0][2 + e]);
#pragma unroll
                    for (int tt = 1; tt < KU; ++tt) y = max3(y, x[nr][tt][e], x[nr][tt][2 + e]);
                    mx[e] = kCap ? y : y * fr[nr][e];
                    moves |= mx[e] > m[nr][e] + kLazy || mx[e] + ev > R[nr][e] + kLazy;
                }
                if (__any_sync(0xffffffffu, moves)) {
                    float grow[2], my[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int u = 0; u < 2 * KU; ++u) {
                        const float lg = log2_scale(fmaxf(scale_of(vsm[u][0]), scale_of(vsm[u][GR - 1])));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float y = x[nr][u >> 1][2 * (u & 1) + e];
                            my[e] = fmaxf(my[e], kCap ? y + lg : fmaf(y, fr[nr][e], lg));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mn = fmaxf(m[nr][e], row_max(mx[e])), y = row_max(my[e]);
                        mr[nr][e] = mn == -INFINITY ? 0.f : mn;
                        const float shrink = ex2(m[nr][e] - mr[nr][e]);   // -inf before the first key: 0
                        m[nr][e] = mn;
                        l_run[nr][e] *= shrink;
#pragma unroll
                        for (int g = 0; g < GR; ++g) zc[nr][g][e] *= shrink;
                        grow[e] = 1.f;
                        float r = y > R[nr][e] + kLazy || R[nr][e] == -INFINITY ? y : R[nr][e];
                        if (r > -INFINITY) r = fmaxf(r, mn - kFarBelow);
                        if (r > R[nr][e]) {
                            grow[e] = ex2(R[nr][e] - r);
                            R[nr][e] = r;
                        }
                        fv[nr][e] = R[nr][e] == -INFINITY ? 0.f : ex2(mr[nr][e] - R[nr][e] + 6.f);
                    }
                    auto times = [&](float (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] *= grow[k & 1];
                    };
#pragma unroll
                    for (int dm = 0; dm < DM; ++dm) times(acc[nr][dm]);
#pragma unroll
                    for (int g = 0; g < GR; ++g) times(eight[nr][g]);
                }
                const uint64_t fr2 = f2_pack(fr[nr][0], fr[nr][1]), nm = f2_pack(-mr[nr][0], -mr[nr][1]);
                const uint64_t fv2 = f2_pack(fv[nr][0], fv[nr][1]);
                uint64_t sum = f2_pack(l_run[nr][0], l_run[nr][1]);
#pragma unroll
                for (int u = 0; u < 2 * KU; ++u) {
                    const uint64_t x2 = f2_pack(x[nr][u >> 1][2 * (u & 1)], x[nr][u >> 1][2 * (u & 1) + 1]);
                    const float2 y = f2_unpack(kCap ? f2_add(x2, nm) : f2_fma(x2, fr2, nm));
                    const float2 pp = make_float2(ex2(y.x), ex2(y.y));
                    const uint64_t p2 = f2_pack(pp.x, pp.y);
                    sum = f2_add(sum, p2);
                    const float2 w = f2_unpack(f2_mul(p2, fv2));
#pragma unroll
                    for (int g = 0; g < GR; ++g) {
                        const float mid = middle_of(vsm[u][g]), sc = scale_of(vsm[u][g]);
                        // (a row that does not see the key: nothing, whatever the middle)
                        zc[nr][g][0] = fmaf(pp.x, edge && y.x == -INFINITY ? 0.f : mid, zc[nr][g][0]);
                        zc[nr][g][1] = fmaf(pp.y, edge && y.y == -INFINITY ? 0.f : mid, zc[nr][g][1]);
                        pt[nr][g][u] = transpose8(Cvt<__half>::pack(w.x * sc, w.y * sc));
                    }
                }
                const float2 l2 = f2_unpack(sum);
                l_run[nr][0] = l2.x, l_run[nr][1] = l2.y;
            }
            // ---- O^T += V^T P^T
            constexpr uint32_t kEight[4] = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
#pragma unroll
            for (int tt = 0; tt < KS; ++tt) {
                // (kSplit: rows 4 .. 7 of P are rows 0 .. 3 of the pair's second product, and what they
                // sum to, of this one's V, goes unread)
                uint32_t P[NR][GR][2];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int g = 0; g < GR; ++g)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            P[nr][g][k] = pt[nr][g][2 * (kSplit ? tt / 2 : tt) + k];
                            if (kSplit && (tt & 1)) P[nr][g][k] = __shfl_xor_sync(0xffffffffu, P[nr][g][k], 16);
                        }
                const uint32_t at = vt + (t0 + tt) * (16 * D / 2) + lm_at;
                uint32_t w[2][J];   // tokens 2 q4, + 1 and 8 further: dims 32 j + 4 r8 ..
                if constexpr (D == 128) {
                    ldmatrix_x4_trans(at, w[0][0], w[0][1], w[0][2], w[0][3]);
                    ldmatrix_x4_trans(at + 512, w[1][0], w[1][1], w[1][2], w[1][3]);
                } else {
                    ldmatrix_x4_trans(at, w[0][0], w[0][1], w[1][0], w[1][1]);
                }
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u = w[0][j] >> (8 * h), v = w[1][j] >> (8 * h);
                        const uint32_t A[4] = {u & kLoMask, u & kHiMask, v & kLoMask, v & kHiMask};
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) mma_f16(acc[nr][2 * j + h], A, P[nr][j / 2][0], P[nr][j / 2][1]);
                    }
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int g = 0; g < GR; ++g) mma_f16(eight[nr][g], kEight, P[nr][g][0], P[nr][g][1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s_at);
        if (++s_at == ST) s_at = 0, phase ^= 1u;
        if (ends || done) {
            // the rows' results, or the piece's for the join
            const int hk = cc.hk, rg = cc.rg, seg = hk * p.groups + rg;
            const bool whole = begins && ends;
            if (!begins && lane == 0) {
                // piece 0, of a segment begun before: the holders of its first and last tiles
                const int units = kv_units<kKv4Open>(cc.t1 - cc.t0), unit0 = (cc.b > 0 ? s_pre[cc.b - 1] : 0) * per_tile + seg * units;
                p.meta[wid] = make_int4(seg, cc.b, sh.worker_of(unit0 + kKv4Open), sh.worker_of(unit0 + units - 2));
            }
            const long long at = (long long)wid * 2 + (begins ? 1 : 0);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                const int row0 = (rg * NR + nr) * 8;
                float f[2], z[GR][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float l = row_sum(l_run[nr][e]), out = whole ? out_factor(0.f, 0.f, l) : 1.f;
#pragma unroll
                    for (int g = 0; g < GR; ++g) z[g][e] = row_sum(zc[nr][g][e]) * out;
                    // what brings acc from R to m
                    f[e] = R[nr][e] == -INFINITY ? 0.f : ex2(R[nr][e] - mr[nr][e]) * out;
                    const int row = row0 + 2 * q4 + e;
                    if (r8 == 0 && row < p.Sq * p.G) {
                        if (!whole)
                            stat[at * (NR * 8) + nr * 8 + 2 * q4 + e] = make_float2(m[nr][e], l);
                        else if (p.lse)
                            p.lse[((long long)cc.b * p.Hq + hk * p.G + row % p.G) * p.Sq + row / p.G] = lse_of(m[nr][e], l);
                    }
                }
                T *dst[2] = {nullptr, nullptr};   // rows 2 q4, + 1 of the output, dim 4 r8
                if (whole)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = row0 + 2 * q4 + e;
                        if (row < p.Sq * p.G)
                            dst[e] = reinterpret_cast<T *>(p.o) + (((long long)cc.b * p.Sq + row / p.G) * p.Hq + hk * p.G + row % p.G) * D + 4 * r8;
                    }
                float4 *const piece = reinterpret_cast<float4 *>(p.acc + at * (NR * 8 * D) + nr * 8 * D) + lane;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float o[2][4];   // dims 32 j + 4 r8 + 2 h, + 1 of the two rows
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = fmaf(acc[nr][2 * j + h][k], k < 2 ? 1.f : 0.0625f, -eight[nr][j / 2][k & 1]);
                            o[h][k] = fmaf(a * 0x1p18f, f[k & 1], z[j / 2][k & 1]);
                        }
                    if (!whole) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) piece[32 * (2 * j + h)] = make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (dst[e])
                                *reinterpret_cast<uint2 *>(dst[e] + 32 * j) =
                                    make_uint2(Cvt<T>::pack(o[0][e], o[0][2 + e]), Cvt<T>::pack(o[1][e], o[1][2 + e]));
                    }
                }
            }
            fresh = true;
        }
        if (done) return;
        cc = nx;
    }
}

// ------------------------------------------------------------------- join
// One CTA per worker.  The workers first .. last that held a segment have a piece of it
// each (piece 1 of the first, piece 0 of the others); the CTAs of the others put them
// together, H of them (a power of two, as many as there are up to kHelpers) a 1 / H of
// the segment's values each, with H sets of threads that take every H-th piece and are
// added in a tree.  So every thread has a few pieces to read at once, two
// pieces or two hundred.  Latency bounds it: three dependent reads.
constexpr int kHelpers = 32;

// Two float4s a thread: with one the call over 64 requests takes 43.0 us, with two 41.0,
// with four 42.7 (two contexts of 64 k: 32.8, 32.8, 34.8).
template <int D, int NR>
__global__ void __launch_bounds__(D) kv4_join_kernel(const __grid_constant__ KvAttnParams p) {
    constexpr int V = 2, N = 2 * D / V;   // threads; float4s of eight rows of a piece: V times that
    constexpr int kMost = N / 4 < kHelpers ? N / 4 : kHelpers;   // (a thread's float4s are of the same two rows)
    __shared__ float4 s_v[V][N], s_s[N];
    const int tid = threadIdx.x, w = blockIdx.x;
    pdl_wait();
    const int4 meta = p.meta[w];   // segment, sequence, first and last worker
    const int first = meta.z, last = meta.w, others = last - first;
    if (meta.x < 0) return;
    const int H = 1 << (31 - __clz(min(others, kMost))), h = w - first - 1;
    if (h >= H) return;
    const int F = N / H, set = tid / F, q = h * F * V + tid % F;   // float4s q + v F
    const int hk = meta.x / p.groups, rg = meta.x - hk * p.groups;
#pragma unroll 1
    for (int nr = 0; nr < NR; ++nr) {
        float4 x[V], t = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);   // t: m, l of the two rows
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4 (&y)[V], float4 s) __attribute__((always_inline)) {
            const float m0 = fmaxf(t.x, s.x), m1 = fmaxf(t.z, s.z);
            const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
            const float a0 = ex2(t.x - r0), a1 = ex2(t.z - r1), b0 = ex2(s.x - r0), b1 = ex2(s.z - r1);
            t = make_float4(m0, fmaf(s.y, b0, t.y * a0), m1, fmaf(s.w, b1, t.w * a1));
#pragma unroll
            for (int v = 0; v < V; ++v)
                x[v] = make_float4(fmaf(y[v].x, b0, x[v].x * a0), fmaf(y[v].y, b1, x[v].y * a1), fmaf(y[v].z, b0, x[v].z * a0),
                                   fmaf(y[v].w, b1, x[v].w * a1));
        };
#pragma unroll 2
        for (int i = first + set; i <= last; i += H) {
            const long long at = ((long long)i * 2 + (i == first ? 1 : 0)) * NR + nr;
            float4 y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = reinterpret_cast<const float4 *>(p.acc + at * (8 * D))[q + v * F];
            add(y, reinterpret_cast<const float4 *>(p.stat)[at * 4 + (q & 3)]);
        }
#pragma unroll 1
        for (int o = H / 2; o > 0; o >>= 1) {
            if (set >= o && set < 2 * o) {
#pragma unroll
                for (int v = 0; v < V; ++v) s_v[v][tid] = x[v];
                s_s[tid] = t;
            }
            __syncthreads();
            if (set < o) {
                float4 y[V];
#pragma unroll
                for (int v = 0; v < V; ++v) y[v] = s_v[v][tid + o * F];
                add(y, s_s[tid + o * F]);
            }
        }
        if (set == 0) {
            const float f0 = t.y == 0.f ? 0.f : 1.f / t.y, f1 = t.w == 0.f ? 0.f : 1.f / t.w;
            const int row0 = (rg * NR + nr) * 8;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 o = make_float4(x[v].x * f0, x[v].y * f1, x[v].z * f0, x[v].w * f1);
                const int at = q + v * F;
                if (p.bf16) store_pairs<D, __nv_bfloat16>(p, meta.y, hk, row0, at % 32, o, at / 32);
                else store_pairs<D, __half>(p, meta.y, hk, row0, at % 32, o, at / 32);
            }
            if (p.lse && q < 4) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = row0 + 2 * q + e;
                    if (row < p.Sq * p.G)
                        p.lse[((long long)meta.y * p.Hq + hk * p.G + row % p.G) * p.Sq + row / p.G] =
                            e ? lse_of(t.z, t.w) : lse_of(t.x, t.y);
                }
            }
        }
        if (NR > 1) __syncthreads();
    }
}

template <int D, int NR, typename T, bool kCap, bool kSplit>
cudaError_t launch_attn(KvAttnParams p, const CUtensorMap &mk, const CUtensorMap &mv, int sms, cudaStream_t stream) {
    using C = Kv4Cfg<D, NR>;
    auto kern = kv4_attn_kernel<D, NR, T, kCap, kSplit>;
    const int smem = C::smem(p.B);
    // Registers of the code as built: workers would wait for those that a smaller launch has not got.
    static std::atomic<int> regs{0};
    cudaError_t e;
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes a;
        if ((e = cudaFuncGetAttributes(&a, kern)) != cudaSuccess) return e;
        regs.store(a.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < C::kRegs) return cudaErrorInvalidConfiguration;
    // (the limit is the kernel's, not the call's: the same for all of them, or a call of fewer sequences
    // could lower it under another thread's launch)
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(kKvMaxSeqs))) != cudaSuccess) return e;
    const int grid = sms < kKvSms ? sms : kKvSms;
    p.workers = grid * C::kWarps;
    p.groups = (p.G * p.Sq + 8 * NR - 1) / (8 * NR);
    // x / (page / 16) as a product: exact for x below 2^29 and divisors up to 8
    const uint32_t d = (uint32_t)p.c.page / 16;
    p.page_magic = d > 1 ? (uint32_t)((1ull << 32) / d + 1) : 0u;
    kern<<<grid, C::kThreads, smem, stream>>>(p, mk, mv);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};   // set up while the attention runs
    cfg.gridDim = dim3((unsigned)p.workers);
    cfg.blockDim = dim3(D);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NR>, p);
}

template <int D, typename T>
cudaError_t launch_attn_d(const KvAttnParams &p, const CUtensorMap &mk, const CUtensorMap &mv, int sms, cudaStream_t stream) {
    const bool cap = p.cap_log2 > 0.f;
    const int rows = p.G * p.Sq;
    if (rows <= 4)
        return cap ? launch_attn<D, 1, T, true, true>(p, mk, mv, sms, stream) : launch_attn<D, 1, T, false, true>(p, mk, mv, sms, stream);
    if (rows <= 8)
        return cap ? launch_attn<D, 1, T, true, false>(p, mk, mv, sms, stream) : launch_attn<D, 1, T, false, false>(p, mk, mv, sms, stream);
    return cap ? launch_attn<D, 2, T, true, false>(p, mk, mv, sms, stream) : launch_attn<D, 2, T, false, false>(p, mk, mv, sms, stream);
}

// CTAs of a ragged call: about `each` parts a thread, fewer rows where that would
// leave SMs idle.
template <int D> dim3 ragged_grid(int rows, int Hkv, int each, int sms, int *per_cta) {
    const long long parts = 2LL * Hkv * (D / 16), n = each * kRagged / parts, most = rows / (4 * sms);
    const long long m = n < most ? n : most;
    *per_cta = (int)(m < 1 ? 1 : m > kMaxRows ? kMaxRows : m);
    return dim3((unsigned)(((long long)rows + *per_cta - 1) / *per_cta), (unsigned)((parts + kRagged - 1) / kRagged));
}

template <int D, typename T>
cudaError_t launch_append_t(const KvAppendParams &p, int sms, cudaStream_t stream) {
    int per;
    const dim3 grid = ragged_grid<D>(p.rows, p.c.Hkv, 4, sms, &per);
    kv4_append_kernel<D, T><<<grid, kRagged, 0, stream>>>(p, per);
    return cudaGetLastError();
}
template <int D, typename T>
cudaError_t launch_read_t(const KvReadParams &p, int sms, cudaStream_t stream) {
    int per;
    const dim3 grid = ragged_grid<D>(p.rows, p.c.Hkv, 4, sms, &per);
    kv4_read_kernel<D, T><<<grid, kRagged, 0, stream>>>(p, per);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const KvAppendParams &p, int D, int bf16, int sms, cudaStream_t stream) {
    if (D == 128)
        return bf16 ? launch_append_t<128, __nv_bfloat16>(p, sms, stream) : launch_append_t<128, __half>(p, sms, stream);
    return bf16 ? launch_append_t<64, __nv_bfloat16>(p, sms, stream) : launch_append_t<64, __half>(p, sms, stream);
}

cudaError_t launch_kv4_read(const KvReadParams &p, int D, int bf16, int sms, cudaStream_t stream) {
    if (D == 128) return bf16 ? launch_read_t<128, __nv_bfloat16>(p, sms, stream) : launch_read_t<128, __half>(p, sms, stream);
    return bf16 ? launch_read_t<64, __nv_bfloat16>(p, sms, stream) : launch_read_t<64, __half>(p, sms, stream);
}

cudaError_t launch_kv4_attn(const KvAttnParams &p, const CUtensorMap &mk, const CUtensorMap &mv, int D, int sms,
                            cudaStream_t stream) {
    if (D == 128)
        return p.bf16 ? launch_attn_d<128, __nv_bfloat16>(p, mk, mv, sms, stream) : launch_attn_d<128, __half>(p, mk, mv, sms, stream);
    return p.bf16 ? launch_attn_d<64, __nv_bfloat16>(p, mk, mv, sms, stream) : launch_attn_d<64, __half>(p, mk, mv, sms, stream);
}

}  // namespace fa
