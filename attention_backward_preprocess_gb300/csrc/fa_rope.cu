// fa_rope.cu -- rotary positions: pairs of dims of q and k turned by an angle
// that goes with the row's position, forward and (the other way round) backward.
//
// a' = f (a cos - b sin), b' = f (b cos + a sin), in 32 bits and rounded once.  Each
// element is read and written once, so bytes bound it where it moves in 16-byte pieces;
// single pairs (kScalar) are bound by their instructions, one per two bytes, and by reads
// that wait for each other.  The angles: p w / (2 pi)
// turns, as a 64-bit fixed-point product whose overflow drops the whole turns, so
// that no position is too far for its angle; its upper 32 bits, as a signed part of
// half a turn (24 bits of them, in f32), go to sincospif.  A CTA works out the cosines and sines of its few
// rows once, in shared memory, while its first loads are under way; all heads of
// q and k use them.
#include "fa_device.cuh"
#include "fa_rope.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;     // rows of a CTA
constexpr int kMaxPairs = 128;  // of a head (D <= 256)

// Pieces of a head a thread takes at a time:
//  kHalves       R / 16 of eight pairs (dims 8u .. and R / 2 + 8u ..), then eight dims each behind R
//  kInterleaved  D / 8 of eight dims: four pairs, fewer at the end of R (pairs do not straddle pieces)
//  kScalar       R / 2 of one pair (halves that are not whole 16-byte pieces), then one dim each
enum RopeKind { kHalves, kInterleaved, kScalar };

// two dims of a and their partners in b, by (cos, sin, cos, sin)
template <typename T> __device__ __forceinline__ void turn(uint32_t &a, uint32_t &b, float4 c) {
    const float2 x = Cvt<T>::unpack(a), y = Cvt<T>::unpack(b);
    a = Cvt<T>::pack(x.x * c.x - y.x * c.y, x.y * c.z - y.y * c.w);
    b = Cvt<T>::pack(y.x * c.x + x.x * c.y, y.y * c.z + x.y * c.w);
}
// a pair in one word
template <typename T> __device__ __forceinline__ void turn_pair(uint32_t &a, float cs, float sn) {
    const float2 v = Cvt<T>::unpack(a);
    a = Cvt<T>::pack(v.x * cs - v.y * sn, v.y * cs + v.x * sn);
}

// A thread keeps its piece u of a head and goes from head to head (and row to row) of
// the CTA: a piece then costs no division (but for sequences that do not follow each other
// as rows do, where each address has one: 57.3 us where evenly spaced ones take 56.4, by
// events around the call) and its cosines' place is known.  2 x 8192
// rows of 40 heads of 128: 52.5 us (6.39 TB/s, 94 % of a copy's rate) at five CTAs an SM, 53
// at six (registers in memory), 57.4 at seven; 55.4 with twice the rows a CTA, 55.3 with the
// cosines in the pairs' order, 57.4 with two divisions a piece besides.  By events around a call,
// which add 5 us: whole heads in halves 57.3, interleaved 70.3; half of a head turned, 67.6 and
// 69.6; kScalar, 24 of 96 dims 235 us (1.07 TB/s), 20 of 80 dims 215 (0.98; interleaved 47.1).
template <typename T, RopeKind kKind>
__global__ void __launch_bounds__(kThreads, 5) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 s_cs[kMaxRows][kMaxPairs];   // factor (cos, sin)
    const int row0 = blockIdx.x * p.rows_per_cta;   // (rows are below 2^31)
    const int rows = min(p.rows_per_cta, p.B * p.S - row0);
    const int half = p.R / 2, heads = p.heads[0] + p.heads[1];
    const int h0 = p.by_units ? (int)__umulhi((uint32_t)threadIdx.x, p.by_units) : threadIdx.x, u = threadIdx.x - h0 * p.units;
    const bool live = h0 < p.heads_at_once;
    // a piece's first dim, and (halves) the other one's
    const int d0 = kKind == kHalves ? (8 * u < half ? 8 * u : p.R + 8 * u - half)
                   : kKind == kInterleaved ? 8 * u : (u < half ? u : u + half);
    constexpr int kPairs = kKind == kHalves ? 8 : 4;   // of a piece
    const int pieces = (half + kPairs - 1) / kPairs;   // that turn
    const bool turns = kKind == kInterleaved || (kKind == kHalves ? 8 * u < half : u < half);
    struct At {
        int r, h;   // row of the CTA, head of q and k together
    };
    auto next = [&](At &x) {
        x.r += p.step_rows, x.h += p.step_heads;
        if (x.h >= heads) x.h -= heads, ++x.r;
    };
    auto offset = [&](const At &x, int t, const long long (&st)[3]) -> long long {
        const int row = row0 + x.r, b = p.batches > 1 ? row / p.S : 0;
        return b * st[0] + (row - b * p.S) * st[1] + (x.h - (t ? p.heads[0] : 0)) * st[2] + d0;
    };
    auto in_at = [&](const At &x) {
        const int t = x.h >= p.heads[0] ? 1 : 0;
        return reinterpret_cast<const T *>(p.t[t].in) + offset(x, t, p.t[t].is);
    };
    auto out_at = [&](const At &x) {
        const int t = x.h >= p.heads[0] ? 1 : 0;
        return reinterpret_cast<T *>(p.t[t].out) + offset(x, t, p.t[t].os);
    };
    // two pieces at a time, both on their way before the cosines are worked out
    uint4 a0, c0, a1, c1;
    At at0, at1;
    auto load = [&](const At &x, uint4 &a, uint4 &c) __attribute__((always_inline)) {
        if (kKind == kScalar || !live || x.r >= rows) return;
        const T *in = in_at(x);
        a = __ldcs(reinterpret_cast<const uint4 *>(in));
        if (kKind == kHalves && turns) c = __ldcs(reinterpret_cast<const uint4 *>(in + half));
    };
    at0.r = h0 / heads, at0.h = h0 - at0.r * heads;
    at1 = at0, next(at1);
    load(at0, a0, c0);
    load(at1, a1, c1);
    for (int i = threadIdx.x; i < rows * half; i += kThreads) {
        const int r = i / half, j = i - r * half, row = row0 + r, b = row / p.S;
        const long long pos = p.positions ? p.positions[row] : (long long)(row - b * p.S) + (p.offsets ? p.offsets[b] : 0);
        const unsigned long long turns_at = (unsigned long long)pos * p.steps[j];
        float sn, cs;
        sincospif((float)(int)(turns_at >> 32) * 0x1p-31f, &sn, &cs);
        // pairs in twos: the first two of every piece, then the next two of every piece ..., so that
        // neighbouring pieces' reads lie side by side (in the pairs' order, four times the wavefronts)
        const int at = kKind == kScalar ? j : ((j % kPairs / 2) * pieces + j / kPairs) * 2 + j % 2;
        s_cs[r][at] = make_float2(cs * p.factor, sn * (p.inverse ? -p.factor : p.factor));
    }
    __syncthreads();
    auto store = [&](const At &x, uint4 a, uint4 c) __attribute__((always_inline)) {
        if (x.r >= rows) return;
        T *out = out_at(x);
        const float2 *cs = s_cs[x.r];
        if (kKind == kHalves) {
            if (turns) {
                const float4 *q = reinterpret_cast<const float4 *>(cs) + u;
                turn<T>(a.x, c.x, q[0]);
                turn<T>(a.y, c.y, q[pieces]);
                turn<T>(a.z, c.z, q[2 * pieces]);
                turn<T>(a.w, c.w, q[3 * pieces]);
                __stcs(reinterpret_cast<uint4 *>(out + half), c);
            }
            __stcs(reinterpret_cast<uint4 *>(out), a);
        } else if (kKind == kInterleaved) {
            const float4 *q = reinterpret_cast<const float4 *>(cs) + min(u, pieces - 1);   // (beyond R: not looked at)
            const float4 v0 = q[0], v1 = q[pieces];
            if (4 * u < half) turn_pair<T>(a.x, v0.x, v0.y);
            if (4 * u + 1 < half) turn_pair<T>(a.y, v0.z, v0.w);
            if (4 * u + 2 < half) turn_pair<T>(a.z, v1.x, v1.y);
            if (4 * u + 3 < half) turn_pair<T>(a.w, v1.z, v1.w);
            __stcs(reinterpret_cast<uint4 *>(out), a);
        } else {
            const T *in = in_at(x);
            if (turns) {
                const float v = static_cast<float>(in[0]), y = static_cast<float>(in[half]);
                const float2 w = cs[u];
                const uint32_t both = Cvt<T>::pack(v * w.x - y * w.y, y * w.x + v * w.y);
                reinterpret_cast<uint16_t *>(out)[0] = (uint16_t)both;
                reinterpret_cast<uint16_t *>(out)[half] = (uint16_t)(both >> 16);
            } else {
                out[0] = in[0];
            }
        }
    };
    if (!live) return;
#pragma unroll 1
    while (at0.r < rows) {
        store(at0, a0, c0);
        store(at1, a1, c1);
        at0 = at1, next(at0);
        at1 = at0, next(at1);
        load(at0, a0, c0);
        load(at1, a1, c1);
    }
}

template <typename T>
cudaError_t launch(const RopeParams &p, RopeKind kind, cudaStream_t stream) {
    const int grid = (int)(((long long)p.B * p.S + p.rows_per_cta - 1) / p.rows_per_cta);
    if (kind == kHalves) rope_kernel<T, kHalves><<<grid, kThreads, 0, stream>>>(p);
    else if (kind == kInterleaved) rope_kernel<T, kInterleaved><<<grid, kThreads, 0, stream>>>(p);
    else rope_kernel<T, kScalar><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int interleaved, int bf16, int sms, cudaStream_t stream) {
    const RopeKind kind = interleaved ? kInterleaved : p.R % 16 == 0 ? kHalves : kScalar;
    // (in place, the dims behind R stay)
    p.units = kind == kInterleaved ? (p.in_place ? (p.R + 7) / 8 : p.D / 8)
              : kind == kHalves    ? p.R / 16 + (p.in_place ? 0 : (p.D - p.R) / 8)
                                   : p.R / 2 + (p.in_place ? 0 : p.D - p.R);
    const long long heads = p.heads[0] + p.heads[1], per_row = heads * p.units, rows = (long long)p.B * p.S;
    // rows of a CTA: about four pieces a thread, fewer where that would leave SMs idle
    long long n = 4 * kThreads / per_row;
    n = n < rows / (4 * sms) ? n : rows / (4 * sms);
    p.rows_per_cta = (int)(n < 1 ? 1 : n > kMaxRows ? kMaxRows : n);
    p.heads_at_once = kThreads / p.units;   // (a head has at most 256 pieces)
    p.step_rows = p.heads_at_once / (int)heads;
    p.step_heads = p.heads_at_once % (int)heads;
    // thread / units as the upper half of a product: exact below 2^16
    p.by_units = p.units > 1 ? (uint32_t)((1ull << 32) / (unsigned)p.units + 1) : 0u;
    // sequences whose rows follow each other as rows do are one
    p.batches = 1;
    for (int i = 0; i < 2 && p.heads[i] > 0; ++i)
        if (p.B > 1 && (p.t[i].is[0] != p.S * p.t[i].is[1] || p.t[i].os[0] != p.S * p.t[i].os[1])) p.batches = p.B;
    return bf16 ? launch<__nv_bfloat16>(p, kind, stream) : launch<__half>(p, kind, stream);
}

}  // namespace fa
