// fa_fwd_duo.cu -- the forward pass (O and LSE, as in fa_fwd_tc.cu) for capped
// scores and for fa_mask_ranges' interval masks.
//
// One CTA per (128-query tile, sequence, query head), the longest causal rows
// first, two CTAs to an SM: each has half of tensor memory, shared memory and
// registers and works in 64-key blocks.  An interval mask leaves a tile few
// key blocks (documents of a thousand tokens: about five of 128 keys), and a
// capped score takes the softmax twice a plain one's time, so with one
// CTA per SM (fa_fwd_tc.cu's shape) most of the time goes by in one warp's
// chain of latencies at a time: a tile set up, its first K on the way, P V of
// the last block, O written, exp2 and reciprocal behind one another.  Here the
// other CTA's work fills it.  Measured (8192 tokens of packed documents, 32 / 8
// heads, D = 128, us | 4 x 16 heads x 2048, causal, cap 50): one CTA per tile
// and SM, 128-key blocks 204 | -; two warps per row (fa_fwd_split.cu) - | 126;
// a persistent CTA per SM that overlaps one tile's end with the next one's
// start 165 | 154; two CTAs of 128-key blocks with one S buffer 222 | 180;
// this one 118 | 124, 111 | 102 with scores taken in packed pairs, 111 | 92 with
// the cap's tanh by a polynomial where a warp's scores lie within half the cap (111
// | 93 since hidden keys are told from visible scores of -inf by their bits):
// exp2, reciprocal and exp2 again, 12 of the exponential unit's cycles per score
// and warp, were 1 / 2 of the time (unit 45 % busy, two warps per scheduler).
// What is left at 8192 tokens: per 64-key block 1480 cycles in each of two CTAs,
// of which 640 are MMA (128 x 64 SS steps at 48 cycles for 32 of math), and 9000
// of a tile's 29000 cycles from launch to first S and from last S to O.
//
// Per block: S = Q K^T (tcgen05 SS, 128 x 64), P = exp2(S c log2e - m) as 16-bit
// pairs into one of two TMEM buffers, O += P V (TS).  S has one buffer, free
// once the softmax warps hold it in registers: S of block n + 1 is issued then,
// and P of block n behind O += P V of block n - 2, which was issued before S of
// block n and is complete with it.   (With two S buffers, P over half
// of its own, S waited for that product: 112 | 93 us.)  K and V have
// rings of their own (a K slot is free once its S is done).  The running
// maximum is raised only past 2^8, as in fa_fwd_tc.cu.
//
// Warps: 0 TMA producer, 1 MMA issuer, 4-7 softmax (thread = query row of its
// TMEM lane quarter), 2-3 idle.
#include <type_traits>

#include "fa_device.cuh"
#include "fa_fwd_common.h"
#include "fa_fwd_ranges.cuh"
#include "fa_params.h"

namespace fa {
namespace {

template <int kD, typename T>
struct DuoCfg {
    static constexpr int D = kD;
    static constexpr int BM = 128, BN = 64;
    static constexpr int kStages = (kD == 128) ? 2 : 4;   // slots of the K ring and of the V ring
    static constexpr int kThreads = 8 * 32;
    static constexpr int W_SM = 4;                         // first softmax warp
    // TMEM: S | P x2 (16-bit pairs) | O
    static constexpr int TM_S = 0, TM_P = BN, TM_O = 2 * BN, TM_COLS = 256;
    static_assert(TM_O + D <= TM_COLS, "TMEM overflow");
    static constexpr int Q_BYTES = BM * D * 2, KV_BYTES = BN * D * 2;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + Q_BYTES;
    static constexpr int OFF_V = OFF_K + kStages * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + kStages * KV_BYTES;
    static constexpr int k_full(int s) { return 8 + s; }
    static constexpr int k_empty(int s) { return 8 + kStages + s; }
    static constexpr int v_full(int s) { return 8 + 2 * kStages + s; }
    static constexpr int v_empty(int s) { return 8 + 3 * kStages + s; }
    static constexpr int NUM_BARS = 8 + 4 * kStages;
    static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;   // TMEM slot, abort flag
    static constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;   // + alignment slack
    // two CTAs to an SM (228 KB, 1 KB of it per CTA beside its own) and no third,
    // which would wait for tensor memory
    static_assert(2 * (SMEM_BYTES + 1024) <= 233472 && 3 * (SMEM_BYTES + 1024) > 233472, "two CTAs per SM");
    static constexpr uint32_t IDESC_S = make_idesc(128, BN, Cvt<T>::is_bf16, false, false);
    static constexpr uint32_t IDESC_PV = make_idesc(128, D, Cvt<T>::is_bf16, false, true);
};

enum {
    U_Q_FULL = 0,     // (its second phase: every MMA done)
    U_S_FULL = 1,     // S of the block complete
    U_S_FREE = 2,     // S in the registers of the 4 softmax warps
    U_P_FULL = 3,     // +b: P written (and O rescaled) by the 4 softmax warps
    U_PV_DONE = 5,    // +b: O += P V of the block with P buffer b complete
    U_O_FINAL = 7,    // (the rings' barriers follow)
};

constexpr float kRescaleLog2 = 8.f;   // how far P's maximum may lag (log2 units)

template <int kD, typename T, int kFlags>
__global__ void __launch_bounds__(DuoCfg<kD, T>::kThreads, 2)
    fwd_duo_kernel(const __grid_constant__ BwdParams p, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, void *o_out,
                   float *lse_out, int nmb) {
    using C = DuoCfg<kD, T>;
    constexpr int D = C::D, BM = C::BM, BN = C::BN, S = C::kStages;
    constexpr bool kCap = (kFlags & kFwdCap) != 0, kRange = (kFlags & kFwdRange) != 0;
    // ---- tile of this CTA: longest causal rows first
    const int bh = blockIdx.x % (p.B * p.Hq);
    const int m = nmb - 1 - blockIdx.x / (p.B * p.Hq);
    const int b = bh / p.Hq, h = bh - b * p.Hq, hk = h / p.G;
    // varlen lengths outside the planned maps: the sequence is left alone and
    // the call reports the error (uniform: the whole CTA leaves)
    if (p.varlen && !varlen_seq_ok(p, b)) {
        if (threadIdx.x == 0 && h == 0 && m == nmb - 1) atomicOr(p.err, kErrBadLength);
        return;
    }
    const int q0 = p.varlen ? p.cu_q[b] : 0, k0 = p.varlen ? p.cu_k[b] : 0;
    const int lq = used_len_q(p, b), lk = used_len_k(p, b);
    if (m * BM >= lq) return;                       // uniform: the whole CTA leaves
    const int diag = lk - lq, bidx = p.varlen ? 0 : b;
    // key blocks [n_begin, n_begin + nblk) hold every key some row of the tile sees
    long long first_key = max(0LL, (long long)m * BM + diag - p.win_lo);
    long long last_key = min((long long)lk - 1, (long long)m * BM + BM - 1 + diag + p.win_hi);
    if (kRange && p.mr_row) tile_range(p, b, m, lk, &first_key, &last_key);
    const int n_begin = (int)(first_key / BN);
    const int nblk = last_key < first_key ? 0 : (int)(last_key / BN) + 1 - n_begin;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 16);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(bar(U_Q_FULL), 1);
        mbar_init(bar(U_S_FULL), 1);
        mbar_init(bar(U_S_FREE), 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(U_P_FULL + i), 4);
            mbar_init(bar(U_PV_DONE + i), 1);
        }
        mbar_init(bar(U_O_FINAL), 1);
        for (int s = 0; s < 4 * S; ++s) mbar_init(bar(C::k_full(s)), 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl w{abort_flag, p.err, p.budget_ns};

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0 && nblk > 0) {
            mbar_arrive_expect_tx(bar(U_Q_FULL), C::Q_BYTES);
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
                tma_load_4d(sbase + C::OFF_Q + hh * BM * 128, &map_q, bar(U_Q_FULL), hh * 64, h, q0 + m * BM, bidx);
            int k_armed = -1, v_armed = -1;   // the last block whose load was issued
            auto load = [&](const CUtensorMap *map, uint32_t off, int full, int empty, int n, int &armed) -> bool {
                const int st = n % S;
                if (n >= S && !mbar_wait(bar(empty + st), (uint32_t)(n / S - 1) & 1u, w)) return false;
                mbar_arrive_expect_tx(bar(full + st), C::KV_BYTES);
                armed = n;
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh)
                    tma_load_4d(sbase + off + st * C::KV_BYTES + hh * BN * 128, map, bar(full + st), hh * 64, hk,
                                k0 + (n_begin + n) * BN, bidx);
                return true;
            };
            for (int n = 0; n < nblk; ++n) {
                if (!load(&map_k, C::OFF_K, C::k_full(0), C::k_empty(0), n, k_armed)) break;
                if (!load(&map_v, C::OFF_V, C::v_full(0), C::v_empty(0), n, v_armed)) break;
            }
            // wind-down: no K/V load may land after the CTA exits (after an abort
            // its consumers may not have waited for it).  The Q load needs no wait
            // here: it is issued first, and the MMA warp waits for it with the
            // whole budget before any wait can run out.
            for (int n = max(k_armed + 1 - S, 0); n <= k_armed; ++n)
                mbar_wait_drain(bar(C::k_full(n % S)), (uint32_t)(n / S) & 1u, p.err, p.budget_ns);
            for (int n = max(v_armed + 1 - S, 0); n <= v_armed; ++n)
                mbar_wait_drain(bar(C::v_full(n % S)), (uint32_t)(n / S) & 1u, p.err, p.budget_ns);
        }
    } else if (warp == 1) {
        // ----------------------------------------------------------- MMA issuer
        // S of block n is issued before O += P V of block n - 1.
        if (nblk > 0) {
            const uint64_t dQ_k = sw128_desc(sbase + C::OFF_Q, 16, 1024);
            bool ok = mbar_wait_warp(bar(U_Q_FULL), 0, w);
            auto issue_pv = [&](int n) -> bool {
                const int bb = n & 1, st = n % S;
                if (!mbar_wait_warp(bar(C::v_full(st)), (uint32_t)(n / S) & 1u, w)) return false;
                if (!mbar_wait_warp(bar(U_P_FULL + bb), (uint32_t)(n >> 1) & 1u, w)) return false;
                tc_fence_after();
                // P (queries x keys) from TMEM, V (keys x d) MN-major, K step = 16
                // keys = 2048 bytes of the swizzled tile
                const uint64_t dV_mn = sw128_desc(sbase + C::OFF_V + st * C::KV_BYTES, BN * 128, 1024);
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk)
                    mma_ts_warp(tmem + C::TM_O, tmem + C::TM_P + bb * (BN / 2) + 8 * kk, desc_add(dV_mn, kk * 2048),
                                C::IDESC_PV, (n > 0 || kk > 0) ? 1u : 0u);
                mma_commit_warp(bar(U_PV_DONE + bb));
                mma_commit_warp(bar(C::v_empty(st)));
                return true;
            };
            for (int n = 0; ok && n < nblk; ++n) {
                const int st = n % S;
                if (!(ok = mbar_wait_warp(bar(C::k_full(st)), (uint32_t)(n / S) & 1u, w))) break;
                if (n >= 1 && !(ok = mbar_wait_warp(bar(U_S_FREE), (uint32_t)(n - 1) & 1u, w))) break;
                tc_fence_after();
                const uint64_t dK_k = sw128_desc(sbase + C::OFF_K + st * C::KV_BYTES, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ko = (kk / 4) * (BN * 128) + (kk % 4) * 32;
                    const uint32_t qo = (kk / 4) * (BM * 128) + (kk % 4) * 32;
                    mma_ss_warp(tmem + C::TM_S, desc_add(dQ_k, qo), desc_add(dK_k, ko), C::IDESC_S, kk > 0);
                }
                mma_commit_warp(bar(U_S_FULL));
                mma_commit_warp(bar(C::k_empty(st)));
                if (n >= 1 && !(ok = issue_pv(n - 1))) break;
            }
            if (ok && issue_pv(nblk - 1)) mma_commit_warp(bar(U_O_FINAL));
            // make sure no MMA is still running before tensor memory is freed
            mma_commit_warp(bar(U_Q_FULL));
            mbar_wait_drain_warp(bar(U_Q_FULL), 1, p.err, p.budget_ns);
        }
    } else if (warp >= C::W_SM) {
        // ------------------------------------------------------------- softmax
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;          // query row of the tile
        const int qi = m * BM + r;                  // query index within the sequence
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        // keys [kmin, kmax] are visible to this row (none if kmax < kmin)
        int kmin = (int)max(0LL, (long long)qi + diag - p.win_lo);
        int kmax = (int)min((long long)lk - 1, (long long)qi + diag + p.win_hi);
        if (kRange && p.mr_row) row_range(p, b, qi, lq, lk, &kmin, &kmax);
        // softcap tanh(s / softcap) log2 e = y q(y^2) for y = s log2 e within half the
        // cap (raw scores within tanh_top)
        float tq[4] = {};
        if (kCap) cap_poly(p.cap_log2, tq);
        const float tanh_top = 0.5f * p.cap_log2 / p.scale_log2;
        float m_run = -INFINITY, l_run = 0.f;       // running max (log2 units), row sum
        bool ok = true;
        for (int n = 0; n < nblk; ++n) {
            const int bb = n & 1;
            const int kb = (n_begin + n) * BN;
            if (!(ok = mbar_wait_warp(bar(U_S_FULL), (uint32_t)n & 1u, w))) break;
            tc_fence_after();
            const uint32_t scol = lane_addr + C::TM_S, pcol = lane_addr + C::TM_P + bb * (BN / 2);
            // element e of the block (key kb + e) is visible iff lo <= e <= hi
            const int lo = kmin - kb, hi = kmax - kb;
            const bool edge = __any_sync(0xffffffffu, lo > 0 || hi < BN - 1);
            float alpha = 1.f, m_use = m_run;
            uint64_t sumv[4] = {0ull, 0ull, 0ull, 0ull};   // row sum: pairs, four independent chains
            // One block.  kMask: hidden keys are masked.  Under a cap the pass without
            // masks takes the tanh by its polynomial, and gives up (false, nothing
            // written) on a score beyond half the cap; the pass with masks takes
            // any.  (Two bodies, not four: a body runs from the instruction cache
            // only when it is not alone in its block.)
            auto block_pass = [&](auto mask_tag) __attribute__((always_inline)) -> bool {
                constexpr bool kMask = decltype(mask_tag)::value, kPoly = kCap && !kMask;
                uint32_t sr[BN / 32][32];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) tmem_ld32(scol + 32 * c, sr[c]);
                tmem_wait_ld();
                if (kPoly) {
                    float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < BN; e += 2)
                        top[e / 2 & 3] = max3_abs(top[e / 2 & 3], sr[e / 32][e % 32], sr[e / 32][e % 32 + 1]);
                    if (!__all_sync(0xffffffffu, fmaxf(max3(top[0], top[1], top[2]), top[3]) <= tanh_top)) return false;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(U_S_FREE));
                // hidden keys at -inf: one bit test and one select per score
                uint32_t in[BN / 32];   // kMask: bit i of word c: key 32 c + i is visible
                bool none = false;      // kMask: no key of the block is
                if (kMask) {
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        const uint32_t below = (uint32_t)((1ull << min(max(lo - 32 * c, 0), 32)) - 1ull);
                        in[c] = (uint32_t)((1ull << min(max(hi + 1 - 32 * c, 0), 32)) - 1ull) & ~below;
#pragma unroll
                        for (int i = 0; i < 32; ++i) sr[c][i] = (in[c] >> i & 1u) ? sr[c][i] : 0xff800000u;
                    }
                    none = (in[0] | in[BN / 32 - 1]) == 0u;
                    static_assert(BN == 64, "two words");
                }
                // pass 1: maximum of the raw scores, scaled (or capped: tanh
                // rises) once, in eight independent chains
                float mxv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mxv[i] = __uint_as_float(sr[0][i]);
#pragma unroll
                for (int e = 8; e < BN; e += 2)
                    mxv[e / 2 & 7] = max3(mxv[e / 2 & 7], __uint_as_float(sr[e / 32][e % 32]), __uint_as_float(sr[e / 32][e % 32 + 1]));
                float mx = fmaxf(max3(max3(mxv[0], mxv[1], mxv[2]), mxv[3], mxv[4]), max3(mxv[5], mxv[6], mxv[7]));
                if (kPoly) {
                    const float y = mx * p.scale_log2, u = y * y;
                    mx = y * fmaf(u, fmaf(u, fmaf(u, tq[3], tq[2]), tq[1]), tq[0]);
                } else if (kCap) {
                    float r0, r1;
                    cap_r2(mx * p.cap_k, 0.f, r0, r1);
                    mx = none ? -INFINITY : fmaf(-2.f * p.cap_log2, r0, p.cap_log2);
                } else {
                    mx *= p.scale_log2;
                }
                const float m_new = fmaxf(m_run, mx);
                m_use = (m_run == -INFINITY || m_new > m_run + kRescaleLog2) ? m_new : m_run;
                alpha = (m_use == m_run) ? 1.f : ex2(m_run - m_use);
                const float mref = (m_use == -INFINITY) ? 0.f : m_use;
                const float cl = kCap && !kPoly ? p.cap_log2 - mref : -mref, cm = -2.f * p.cap_log2;
                const uint64_t cl2 = f2_pack(cl, cl), cm2 = f2_pack(cm, cm), one2 = f2_pack(1.f, 1.f);
                const uint64_t k2 = kCap && !kPoly ? f2_pack(p.cap_k, p.cap_k) : f2_pack(p.scale_log2, p.scale_log2);
                // pass 2: P as pairs into the first BN/2 columns
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t raw = f2_pack(__uint_as_float(sr[c][2 * i]), __uint_as_float(sr[c][2 * i + 1]));
                        float2 x;
                        if (kPoly) {
                            const uint64_t y = f2_mul(raw, k2), u = f2_mul(y, y);
                            uint64_t t = f2_fma(u, f2_pack(tq[3], tq[3]), f2_pack(tq[2], tq[2]));
                            t = f2_fma(u, t, f2_pack(tq[1], tq[1]));
                            t = f2_fma(u, t, f2_pack(tq[0], tq[0]));
                            x = f2_unpack(f2_fma(y, t, cl2));
                        } else if (kCap) {
                            // (cap_r2 on packed pairs)
                            const float2 z = f2_unpack(f2_mul(raw, k2));
                            const float2 a = f2_unpack(f2_add(f2_pack(cap_exp(z.x), cap_exp(z.y)), one2));
                            const float rr = rcp_approx(a.x * a.y);
                            x = f2_unpack(f2_fma(f2_mul(f2_pack(rr, rr), f2_pack(a.y, a.x)), cm2, cl2));
                        } else {
                            x = f2_unpack(f2_fma(raw, k2, cl2));
                        }
                        float p0 = ex2(x.x), p1 = ex2(x.y);
                        if (kCap && kMask) {   // the cap of -inf is -softcap
                            p0 = (in[c] >> (2 * i) & 1u) ? p0 : 0.f;
                            p1 = (in[c] >> (2 * i + 1) & 1u) ? p1 : 0.f;
                        }
                        sumv[i & 3] = f2_add(sumv[i & 3], f2_pack(p0, p1));
                        pk[i] = Cvt<T>::pack(p0, p1);
                    }
                    tmem_st16(pcol + 16 * c, pk);
                }
                return true;
            };
            if (edge || !block_pass(std::false_type{})) block_pass(std::true_type{});
            const float2 sum = f2_unpack(f2_add(f2_add(sumv[0], sumv[1]), f2_add(sumv[2], sumv[3])));
            l_run = l_run * alpha + (sum.x + sum.y);
            m_run = m_use;
            // O holds the blocks < n: rescale it when a row's maximum moved
            if (n > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                if (!(ok = mbar_wait_warp(bar(U_PV_DONE + ((n - 1) & 1)), (uint32_t)((n - 1) >> 1) & 1u, w))) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t orr[32];
                    tmem_ld32(lane_addr + C::TM_O + 32 * c, orr);
                    tmem_wait_ld();
                    uint32_t olo[16], ohi[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        olo[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
                        ohi[i] = __float_as_uint(__uint_as_float(orr[16 + i]) * alpha);
                    }
                    tmem_st16(lane_addr + C::TM_O + 32 * c, olo);
                    tmem_st16(lane_addr + C::TM_O + 32 * c + 16, ohi);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(U_P_FULL + bb));
        }
        // ---------------------------------------------------------- epilogue
        // O = acc / l, LSE = (m + log2 l) ln 2; a row that sees no key gets O = 0
        // and LSE = -inf, a row of NaN scores NaN
        if (ok && nblk > 0) {
            ok = mbar_wait_warp(bar(U_O_FINAL), 0, w);
            tc_fence_after();
        }
        if (ok) {
            const bool live = qi < lq;
            const long long row = p.varlen ? (long long)q0 + qi : (long long)b * p.Sq + qi;
            if (live) {
                float *lse_dst = p.varlen ? lse_out + (long long)h * p.cu_q[p.B] + q0 + qi
                                          : lse_out + ((long long)b * p.Hq + h) * p.Sq + qi;
                *lse_dst = l_run > 0.f ? (m_run + log2f(l_run)) * 0.69314718055994531f
                                       : l_run == 0.f ? -INFINITY : l_run;
            }
            const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
            T *dst = reinterpret_cast<T *>(o_out) + (row * p.Hq + h) * p.Dhv;   // Dhv <= D columns
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t orr[32];
                if (nblk > 0) {
                    tmem_ld32(lane_addr + C::TM_O + 32 * c, orr);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) orr[i] = 0u;
                }
                if (live) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[i] = Cvt<T>::pack(__uint_as_float(orr[2 * i]) * inv, __uint_as_float(orr[2 * i + 1]) * inv);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (32 * c + 8 * i < p.Dhv)
                            reinterpret_cast<uint4 *>(dst + 32 * c)[i] =
                                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::TM_COLS);
}

template <int kD, typename T, int kFlags>
cudaError_t launch_duo_t(const BwdParams &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                         void *o, float *lse, int max_lq, cudaStream_t stream) {
    using C = DuoCfg<kD, T>;
    auto kern = fwd_duo_kernel<kD, T, kFlags>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const int nmb = (max_lq + C::BM - 1) / C::BM;
    const long long grid = (long long)nmb * p.B * p.Hq;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kern<<<(unsigned)grid, C::kThreads, C::SMEM_BYTES, stream>>>(p, mq, mk, mv, o, lse, nmb);
    return cudaGetLastError();
}

template <int kD, typename T>
cudaError_t launch_duo_flags(const BwdParams &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                             void *o, float *lse, int max_lq, int flags, cudaStream_t stream) {
    if (flags == kFwdRange) return launch_duo_t<kD, T, kFwdRange>(p, mq, mk, mv, o, lse, max_lq, stream);
    return launch_duo_t<kD, T, kFwdCap | kFwdRange>(p, mq, mk, mv, o, lse, max_lq, stream);
}

}  // namespace

// Key rows of one TMA box for K / V.
int fwd_duo_block_n() { return DuoCfg<128, __nv_bfloat16>::BN; }

cudaError_t launch_fwd_duo(const BwdParams &p, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                           void *o, float *lse, int max_lq, int bf16, int flags, cudaStream_t stream) {
    if (p.D == 128)
        return bf16 ? launch_duo_flags<128, __nv_bfloat16>(p, q, k, v, o, lse, max_lq, flags, stream)
                    : launch_duo_flags<128, __half>(p, q, k, v, o, lse, max_lq, flags, stream);
    return bf16 ? launch_duo_flags<64, __nv_bfloat16>(p, q, k, v, o, lse, max_lq, flags, stream)
                : launch_duo_flags<64, __half>(p, q, k, v, o, lse, max_lq, flags, stream);
}

}  // namespace fa
