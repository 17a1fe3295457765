// fa_rope.cu -- rotary positions: pairs of dims of q and k turned by an angle
// that goes with the row's position, forward and (the other way round) backward.
//
// a' = f (a cos - b sin), b' = f (b cos + a sin), in 32 bits and rounded once.  Each
// element is read and written once, so bytes bound it.  The angles: p w / (2 pi)
// turns, as a 64-bit fixed-point product whose overflow drops the whole turns, so
// that no position is too far for its angle; its upper 32 bits, as a signed part of
// half a turn, go to sincospif.  A CTA works out the cosines and sines of its few
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

template <typename T>
__device__ __forceinline__ void turn(uint32_t &a, uint32_t &b, float2 c0, float2 c1) {
    const float2 x = Cvt<T>::unpack(a), y = Cvt<T>::unpack(b);
    a = Cvt<T>::pack(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
    b = Cvt<T>::pack(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
}

template <typename T, RopeKind kKind>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 s_cs[kMaxRows][kMaxPairs];   // factor (cos, sin)
    const int row0 = blockIdx.x * p.rows_per_cta;   // (rows are below 2^31)
    const int rows = min(p.rows_per_cta, p.B * p.S - row0);
    const int half = p.R / 2, per_row = (p.heads[0] + p.heads[1]) * p.units;
    // where item i of the CTA lies: its row, and the addresses of its head
    auto where = [&](int i, int &r, int &u, const T *&in, T *&out) {
        r = (int)__umulhi((uint32_t)i, p.by_row);
        const int in_row = i - r * per_row;
        int h = p.by_units ? (int)__umulhi((uint32_t)in_row, p.by_units) : in_row;
        u = in_row - h * p.units;
        const int t = h >= p.heads[0] ? 1 : 0;
        h -= t ? p.heads[0] : 0;
        const int row = row0 + r, b = p.B > 1 ? row / p.S : 0, s = row - b * p.S;
        const RopeTensor &x = p.t[t];
        in = reinterpret_cast<const T *>(x.in) + (b * x.is[0] + s * x.is[1] + h * x.is[2]);
        out = reinterpret_cast<T *>(x.out) + (b * x.os[0] + s * x.os[1] + h * x.os[2]);
    };
    const int items = rows * per_row;
    constexpr int PER = kKind == kScalar ? 1 : 2;
    uint4 a[PER], c[PER];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= items) break;
            int r, u;
            const T *in;
            T *out;
            where(i, r, u, in, out);
            if (kKind == kHalves) {
                if (8 * u < half) {
                    a[k] = __ldcs(reinterpret_cast<const uint4 *>(in + 8 * u));
                    c[k] = __ldcs(reinterpret_cast<const uint4 *>(in + half + 8 * u));
                } else {
                    a[k] = __ldcs(reinterpret_cast<const uint4 *>(in + p.R + 8 * u - half));
                }
            } else if (kKind == kInterleaved) {
                a[k] = __ldcs(reinterpret_cast<const uint4 *>(in + 8 * u));
            }
        }
    };
    load(threadIdx.x);
    for (int i = threadIdx.x; i < rows * half; i += kThreads) {
        const int r = i / half, j = i - r * half, row = row0 + r, b = row / p.S;
        const long long pos = p.positions ? p.positions[row] : (long long)(row - b * p.S) + (p.offsets ? p.offsets[b] : 0);
        const unsigned long long turns = (unsigned long long)pos * p.steps[j];
        float sn, cs;
        sincospif((float)(int)(turns >> 32) * 0x1p-31f, &sn, &cs);
        s_cs[r][j] = make_float2(cs * p.factor, sn * (p.inverse ? -p.factor : p.factor));
    }
    __syncthreads();
    for (int i0 = threadIdx.x; i0 < items; i0 += PER * kThreads) {
        if (i0 != (int)threadIdx.x) load(i0);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= items) break;
            int r, u;
            const T *in;
            T *out;
            where(i, r, u, in, out);
            const float2 *cs = s_cs[r];
            if (kKind == kHalves) {
                if (8 * u < half) {
                    const float4 *q = reinterpret_cast<const float4 *>(cs + 8 * u);
                    uint32_t *x = &a[k].x, *y = &c[k].x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 v = q[j];
                        turn<T>(x[j], y[j], make_float2(v.x, v.y), make_float2(v.z, v.w));
                    }
                    __stcs(reinterpret_cast<uint4 *>(out + 8 * u), a[k]);
                    __stcs(reinterpret_cast<uint4 *>(out + half + 8 * u), c[k]);
                } else {
                    __stcs(reinterpret_cast<uint4 *>(out + p.R + 8 * u - half), a[k]);
                }
            } else if (kKind == kInterleaved) {
                uint32_t *x = &a[k].x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int pair = 4 * u + j;
                    if (pair < half) {
                        const float2 v = Cvt<T>::unpack(x[j]), w = cs[pair];
                        x[j] = Cvt<T>::pack(v.x * w.x - v.y * w.y, v.y * w.x + v.x * w.y);
                    }
                }
                __stcs(reinterpret_cast<uint4 *>(out + 8 * u), a[k]);
            } else {
                if (u < half) {
                    const float v = static_cast<float>(in[u]), y = static_cast<float>(in[u + half]);
                    const float2 w = cs[u];
                    const uint32_t both = Cvt<T>::pack(v * w.x - y * w.y, y * w.x + v * w.y);
                    reinterpret_cast<uint16_t *>(out)[u] = (uint16_t)both;
                    reinterpret_cast<uint16_t *>(out)[u + half] = (uint16_t)(both >> 16);
                } else {
                    out[u + half] = in[u + half];
                }
            }
        }
    }
}

// x / d as the upper half of x m: exact for x d < 2^32 (0 where d is 1).  Here x is below
// heads times units and d a head's units: at most 2^16 256^2
uint32_t magic(uint32_t d) { return d > 1 ? (uint32_t)((1ull << 32) / d + 1) : 0u; }

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
    // rows of a CTA: about four items a thread, fewer where that would leave SMs idle
    long long n = 4 * kThreads / per_row;
    n = n < rows / (4 * sms) ? n : rows / (4 * sms);
    p.rows_per_cta = (int)(n < 1 ? 1 : n > kMaxRows ? kMaxRows : n);
    if (per_row == 1) p.rows_per_cta = 1;
    p.by_units = magic((uint32_t)p.units);                                      // divides an item of a row
    p.by_row = p.rows_per_cta > 1 ? magic((uint32_t)per_row) : 0u;              // (then a row has at most 512 items)
    return bf16 ? launch<__nv_bfloat16>(p, kind, stream) : launch<__half>(p, kind, stream);
}

}  // namespace fa
