// fa_api.cu -- the C ABI declared in include/fa.h: argument validation,
// workspace planning, TMA tensor-map encoding and the kernel launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fa.h"
#include "fa_kvcache.h"
#include "fa_params.h"
#include "fa_ranges.h"

namespace fa {
cudaError_t launch_schedule(const BwdParams &p, cudaStream_t stream);
cudaError_t launch_preprocess(const BwdParams &p, int bf16, cudaStream_t stream);
cudaError_t launch_postprocess(const BwdParams &p, int bf16, cudaStream_t stream);
cudaError_t launch_dbias_zero(const BwdParams &p, int bm, cudaStream_t stream);
cudaError_t launch_fwd_tc(const BwdParams &p, const CUtensorMap &q, const CUtensorMap &k,
                          const CUtensorMap &v, void *o, float *lse, int max_lq, int bf16, int sms,
                          cudaStream_t stream);
int fwd_block_m();
int fwd_block_n(const BwdParams &p, int sms);
int *fwd_error_word();
cudaError_t launch_error_or(const int *from, int *word, cudaStream_t stream);
cudaError_t launch_bwd_main(const BwdParams &p, const CUtensorMap &q, const CUtensorMap &k,
                            const CUtensorMap &v, const CUtensorMap &dout, const CUtensorMap &dk,
                            const CUtensorMap &dv, int bf16, int grid, cudaStream_t stream);
int main_block_m(int D);
cudaError_t launch_bwd_wide(const BwdParams &p, const CUtensorMap &q, const CUtensorMap &k,
                            const CUtensorMap &v, const CUtensorMap &dout, int bf16, int grid,
                            cudaStream_t stream);
int wide_block_m();
int wide_halves(int Dq_tile, int Dv_tile);
}  // namespace fa

namespace {

std::atomic<long long> g_budget_ns{2000000000LL};

constexpr float kLog2e = 1.4426950408889634f;

// Bounds of a soft cap.  The capped score's error is absolute, about softcap *
// 2^-21 (fa_device.cuh): at 1000 that is the size of fp16's rounding of P.
// Below 1 / 1000 every score is the same to the softmax.
constexpr float kMinSoftcap = 1e-3f, kMaxSoftcap = 1000.f;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Tile width a head dim runs at: 64, 128 or 256 (the columns past D are
// zero-filled by the TMA loads; the FlashAttention postprocess page likewise
// pads the head dim to a multiple of its block size).
int pad_d(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Backward tile width of a query / key head dim.  D = 64 runs in the 128-wide
// tile (its upper 64 columns zero) for dense problems of at least 4096 keys:
// its softmax, not the tensor core, sets the step time, and the wider tile's
// 64-query steps carry half the elementwise work per step (B = 2, 32 / 8
// heads, 8192 keys, causal: main kernel 2.204 -> 1.911 ms).  Shorter and
// varlen problems keep the 64-wide tile, whose 128-query steps halve the unit
// transitions (16 sequences of 256..2048 keys: 0.378 against 0.435 ms).
int bwd_pad_d(int D, int Sk, bool varlen) {
    if (D <= 64 && !varlen && Sk >= 4096) return 128;
    return pad_d(D);
}

// Head dims with a kernel: a query / key dim D that is a multiple of 8 in
// [64, 256]; a value dim Dv (0: equal to D) that is a multiple of 8 in
// [8, 256].  One head dim of at most 128 runs in the main kernel; a head dim
// above 128, or Dv != D (then D > 64), runs in the wide kernel.
bool head_dims_ok(int D, int Dv) {
    if (D < 64 || D > 256 || D % 8 != 0) return false;
    if (Dv == 0 || Dv == D) return true;
    return Dv >= 8 && Dv <= 256 && Dv % 8 == 0 && D > 64;
}
bool wide_dims(int D, int Dv) { return D > 128 || (Dv != 0 && Dv != D); }
int value_tile(int D, int Dv) {   // tile width of the value side
    return wide_dims(D, Dv) ? ((Dv == 0 ? D : Dv) <= 128 ? 128 : 256) : pad_d(D);
}

struct Layout {
    size_t err, ntiles, tiles, dvec, lse2, dqacc, sem, total;  // byte offsets / size
    long long rows, rows_per_head;
    int sq_round, max_tiles;
};

bool plan(int B, int Sq, int Sk, int Hq, int Hkv, int D, int varlen, int deterministic,
          Layout *L) {
    if (B <= 0 || Sq <= 0 || Sk <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv) return false;
    const long long T = fa::kRowTile;
    L->sq_round = (int)round_up((size_t)Sq, T);
    if (varlen) {
        L->rows_per_head = (long long)round_up((size_t)B * ((size_t)Sq + T), T);
        L->rows = (long long)Hq * L->rows_per_head;
    } else {
        L->rows_per_head = L->sq_round;
        L->rows = (long long)B * Hq * L->sq_round;
    }
    const long long tiles = (long long)B * ((Sk + fa::kBlockN - 1) / fa::kBlockN) * Hkv;
    if (tiles > (1LL << 30)) return false;
    L->max_tiles = (int)tiles;
    size_t off = 0;
    L->err = off;       off += 256;
    L->ntiles = off;    off += 256;
    L->tiles = off;     off = round_up(off + (size_t)tiles * 16, 256);
    L->dvec = off;      off = round_up(off + (size_t)L->rows * 4, 256);
    L->lse2 = off;      off = round_up(off + (size_t)L->rows * 4, 256);
    L->dqacc = off;     off = round_up(off + (size_t)L->rows * bwd_pad_d(D, Sk, varlen) * 4, 256);
    L->sem = off;       off = round_up(off + (deterministic ? (size_t)(L->rows / 64) * 4 : 0), 256);
    L->total = off;
    return true;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

fa_status check_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return FA_ERR_CUDA;
    if (major != 10 || minor != 3) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

fa_status check_shape(int B, int Sq, int Sk, int Hq, int Hkv, int D, fa_dtype dtype,
                      const int *cu_q, const int *cu_k) {
    if (B <= 0 || Sq <= 0 || Sk <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return FA_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if ((cu_q == nullptr) != (cu_k == nullptr)) return FA_ERR_INVALID_ARG;
    if (!head_dims_ok(D, 0)) return FA_ERR_UNSUPPORTED;
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
    // TMA coordinates are 32-bit
    if ((long long)B * Sq > (1LL << 31) - 1 || (long long)B * Sk > (1LL << 31) - 1)
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// ----------------------------------------------------------- tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

// 4-D map over a [batch, rows, heads, D] 16-bit tensor (d innermost; strides
// st in elements: batch, row, head), box of 64 d x 1 head x box_rows rows,
// 128-byte swizzle, zero fill out of bounds.
bool encode_rows_map(CUtensorMap *m, const void *base, int D, int H, long long rows, int batch,
                     int box_rows, int bf16, const long long (&st)[3]) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)rows, (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)st[2] * 2, (cuuint64_t)st[1] * 2, (cuuint64_t)st[0] * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                    const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 2-D map over the cache's V as rows of page bytes, box of block tokens x D dims.
bool encode_v_map(CUtensorMap *m, const void *base, int page, long long rows, int block, int D) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)page, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)page};
    const cuuint32_t box[2] = {(cuuint32_t)block, (cuuint32_t)D};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------- workspace of the library's
// A call that brings no workspace takes one from a memory pool of the library's,
// allocated and freed in the order of the call's stream: calls in flight together
// never share one, and a block is given to another stream only once the work that
// used it is over (or, captured, belongs to its graph).  The pool keeps what it
// has, so a steady program allocates nothing from the driver; it makes no stream
// wait for another one's block.
std::mutex g_pool_mutex;
std::vector<cudaMemPool_t> g_pools;   // per device, made by its first call

bool library_pool(cudaMemPool_t *out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lk(g_pool_mutex);
    if ((int)g_pools.size() <= dev) g_pools.resize(dev + 1, nullptr);
    if (!g_pools[dev]) {
        cudaMemPoolProps props;
        std::memset(&props, 0, sizeof(props));
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        cudaMemPool_t pool = nullptr;
        if (cudaMemPoolCreate(&pool, &props) != cudaSuccess) return false;
        uint64_t keep = UINT64_MAX;
        int off = 0;
        if (cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep) != cudaSuccess ||
            cudaMemPoolSetAttribute(pool, cudaMemPoolReuseAllowInternalDependencies, &off) != cudaSuccess) {
            cudaMemPoolDestroy(pool);
            return false;
        }
        g_pools[dev] = pool;
    }
    *out = g_pools[dev];
    return true;
}

// The workspace of one call.
struct CallWorkspace {
    void *ptr = nullptr;
    cudaStream_t stream = nullptr;

    fa_status take(size_t bytes, cudaStream_t s) {
        cudaMemPool_t pool;
        if (!library_pool(&pool) || cudaMallocFromPoolAsync(&ptr, bytes, pool, s) != cudaSuccess) {
            ptr = nullptr;
            cudaGetLastError();   // not left for the next launch's check to find
            return FA_ERR_CUDA;
        }
        stream = s;
        return FA_OK;
    }
    CallWorkspace() = default;
    CallWorkspace(const CallWorkspace &) = delete;
    CallWorkspace &operator=(const CallWorkspace &) = delete;
    ~CallWorkspace() {
        if (ptr) cudaFreeAsync(ptr, stream);
    }
};

// Totals of the packed varlen tensors (cu[B]); read back from the device.
fa_status varlen_totals(const int *cu_q, const int *cu_k, int B, cudaStream_t stream,
                        long long *tq, long long *tk) {
    int h[2] = {0, 0};
    if (cudaMemcpyAsync(&h[0], cu_q + B, sizeof(int), cudaMemcpyDeviceToHost, stream) !=
            cudaSuccess ||
        cudaMemcpyAsync(&h[1], cu_k + B, sizeof(int), cudaMemcpyDeviceToHost, stream) !=
            cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
        return FA_ERR_CUDA;
    if (h[0] < 0 || h[1] < 0) return FA_ERR_INVALID_ARG;
    *tq = h[0];
    *tk = h[1];
    return FA_OK;
}

// The packed row counts of a varlen call: the caller's (fa_ext total_q /
// total_k, both > 0), which need no host synchronisation, else cu[B] read
// back from the device.  Every sequence fits the planned layout only if the
// totals are at most B times the maximum lengths; the kernels check
// cu_seqlens against the totals and the maximum lengths (kErrBadLength).
fa_status packed_totals(const fa_ext *ext, const int *cu_q, const int *cu_k, int B, int Sq,
                        int Sk, cudaStream_t stream, long long *tq, long long *tk) {
    if (ext && (ext->total_q != 0 || ext->total_k != 0)) {
        *tq = ext->total_q;
        *tk = ext->total_k;
    } else {
        fa_status st = varlen_totals(cu_q, cu_k, B, stream, tq, tk);
        if (st != FA_OK) return st;
    }
    if (*tq > (long long)B * Sq || *tk > (long long)B * Sk) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Host check of the caller's packed totals (before the device is touched):
// varlen only, both positive, at most B times the maximum lengths.
fa_status check_ext_totals(const fa_ext *ext, bool varlen, int B, int Sq, int Sk) {
    if (!ext || (ext->total_q == 0 && ext->total_k == 0)) return FA_OK;
    if (!varlen || ext->total_q <= 0 || ext->total_k <= 0) return FA_ERR_INVALID_ARG;
    if (ext->total_q > (long long)B * Sq || ext->total_k > (long long)B * Sk) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// Strides of a [batch, rows, H, D] tensor: the caller's (all zero: contiguous),
// else contiguous.  A packed varlen tensor has no batch stride.
fa_status set_strides(long long (&dst)[3], const long long *given, int varlen, long long rows, int H, int D) {
    dst[2] = D;
    dst[1] = (long long)H * D;
    dst[0] = rows * H * D;
    if (!given || (given[0] == 0 && given[1] == 0 && given[2] == 0)) return FA_OK;
    for (int i = varlen ? 1 : 0; i < 3; ++i) {
        // the tensor maps' terms: multiples of 16 bytes below 2^40 bytes
        if (given[i] <= 0 || (given[i] & 7) || given[i] >= (1LL << 39)) return FA_ERR_INVALID_ARG;
        dst[i] = given[i];
    }
    return FA_OK;
}

// The strides of q, k, v, o and dout, once the head dims and lengths are known
// (rq / rk: rows of the query and key side of one batch entry).
fa_status apply_strides(fa::BwdParams &p, const fa_ext *ext, long long rq, long long rk) {
    fa_status st;
    if ((st = set_strides(p.sq, ext ? ext->q_stride : nullptr, p.varlen, rq, p.Hq, p.Dh)) != FA_OK) return st;
    if ((st = set_strides(p.sk, ext ? ext->k_stride : nullptr, p.varlen, rk, p.Hkv, p.Dh)) != FA_OK) return st;
    if ((st = set_strides(p.sv, ext ? ext->v_stride : nullptr, p.varlen, rk, p.Hkv, p.Dhv)) != FA_OK) return st;
    if ((st = set_strides(p.so, ext ? ext->o_stride : nullptr, p.varlen, rq, p.Hq, p.Dhv)) != FA_OK) return st;
    return set_strides(p.sdo, ext ? ext->dout_stride : nullptr, p.varlen, rq, p.Hq, p.Dhv);
}

struct Prepared {
    fa::BwdParams p;
    Layout L;
    long long total_q, total_k;
};

int sm_count() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 1;
}

// The visible band, ALiBi slopes and used lengths of the parameter block
// (ext NULL: none, only the causal mask).
fa_status apply_ext(fa::BwdParams &p, int causal, const fa_ext *ext) {
    int wl = -1, wr = -1;
    p.alibi = nullptr;
    p.alibi_bstride = 0;
    p.seqused_q = p.seqused_k = nullptr;
    p.bias = nullptr;
    p.bias_bs = p.bias_hs = p.bias_rs = 0;
    p.dbias = nullptr;
    p.drop_t = 0;
    p.drop_key0 = p.drop_key1 = p.drop_offset = 0;
    p.drop_scale = 1.f;
    p.drop_mask = nullptr;
    p.drop_mask_w = 0;
    p.Dhv = p.Dh;
    p.Dv = p.D;
    if (ext) {
        if (ext->head_dim_v != 0) {
            if (!head_dims_ok(p.Dh, ext->head_dim_v)) return FA_ERR_UNSUPPORTED;
            p.Dhv = ext->head_dim_v;
        }
        wl = ext->window_left;
        wr = ext->window_right;
        if (wl < -1 || wr < -1) return FA_ERR_INVALID_ARG;
        if (ext->alibi_slopes) {
            if ((reinterpret_cast<uintptr_t>(ext->alibi_slopes) & 3u) ||
                (ext->alibi_batch_stride != 0 && ext->alibi_batch_stride != p.Hq))
                return FA_ERR_INVALID_ARG;
            p.alibi = ext->alibi_slopes;
            p.alibi_bstride = ext->alibi_batch_stride;
        }
        if ((reinterpret_cast<uintptr_t>(ext->seqused_q) & 3u) ||
            (reinterpret_cast<uintptr_t>(ext->seqused_k) & 3u))
            return FA_ERR_INVALID_ARG;
        p.seqused_q = ext->seqused_q;
        p.seqused_k = ext->seqused_k;
        if (ext->bias) {
            if (p.varlen) return FA_ERR_UNSUPPORTED;
            if (!aligned16(ext->bias) || ext->bias_batch_stride < 0 || ext->bias_head_stride < 0 ||
                ext->bias_row_stride < p.Sk || (ext->bias_batch_stride & 7) ||
                (ext->bias_head_stride & 7) || (ext->bias_row_stride & 7))
                return FA_ERR_INVALID_ARG;
            p.bias = ext->bias;
            p.bias_bs = ext->bias_batch_stride;
            p.bias_hs = ext->bias_head_stride;
            p.bias_rs = ext->bias_row_stride;
        }
        if (ext->dbias) {
            if (p.varlen) return FA_ERR_UNSUPPORTED;
            if ((reinterpret_cast<uintptr_t>(ext->dbias) & 1u)) return FA_ERR_INVALID_ARG;
            p.dbias = ext->dbias;
        }
        const float dp = ext->dropout_p;
        if (!(dp >= 0.f && dp < 1.f)) return FA_ERR_INVALID_ARG;
        p.drop_t = std::min(255, (int)(dp * 256.f + 0.5f));
        p.drop_key0 = (uint32_t)ext->dropout_seed;
        p.drop_key1 = (uint32_t)(ext->dropout_seed >> 32);
        p.drop_offset = ext->dropout_offset;
        p.drop_scale = 256.f / (float)(256 - p.drop_t);
        if (ext->dropout_mask && p.drop_t > 0) {
            if (reinterpret_cast<uintptr_t>(ext->dropout_mask) & 3u) return FA_ERR_INVALID_ARG;
            p.drop_mask = ext->dropout_mask;
            p.drop_mask_w = (p.Sk + 31) / 32;
        }
    }
    p.cap_log2 = p.cap_k = 0.f;
    p.mr_row = nullptr;
    if (ext && (ext->softcap != 0.f || ext->mask_ranges)) {
        // the capped and interval instances carry no other score extension
        if (ext->softcap != 0.f) {
            if (!(ext->softcap >= kMinSoftcap && ext->softcap <= kMaxSoftcap)) return FA_ERR_INVALID_ARG;
            p.cap_log2 = ext->softcap * kLog2e;
            p.cap_k = 2.f * p.scale_log2 / ext->softcap;
            if (!std::isfinite(p.cap_k)) return FA_ERR_INVALID_ARG;
        }
        if (ext->mask_ranges) {
            if (p.varlen) return FA_ERR_UNSUPPORTED;
            if (p.Sq != p.Sk || causal || wl != -1 || wr != -1) return FA_ERR_INVALID_ARG;
            if (reinterpret_cast<uintptr_t>(ext->mask_ranges) & 255u) return FA_ERR_INVALID_ARG;
            const size_t need = fa_mask_ranges_bytes(p.B, p.Sq);
            if (need == 0 || ext->mask_ranges_bytes < need) return FA_ERR_INVALID_ARG;
            const fa::RangeTables t = fa::range_tables(const_cast<void *>(ext->mask_ranges), p.B, p.Sq);
            p.mr_row = t.row;
            p.mr_block = t.block;
            p.mr_key = t.key;
            p.mr_first = t.first;
            p.mr_order = t.order;
            p.mr_rows = t.rows;
        }
        if (p.alibi || p.bias || p.dbias || p.drop_t > 0 || wide_dims(p.Dh, p.Dhv)) return FA_ERR_UNSUPPORTED;
    }
    p.win_lo = (wl < 0 || wl >= fa::kNoWindow) ? fa::kNoWindow : wl;
    p.win_hi = (wr < 0 || wr >= fa::kNoWindow) ? fa::kNoWindow : wr;
    if (causal) p.win_hi = std::min(p.win_hi, 0);
    if (wide_dims(p.Dh, p.Dhv)) {
        // the wide kernel's tile widths (128 or 256 on each side); it has the
        // band masks (causal, both window edges) and used lengths
        p.D = p.Dh <= 128 ? 128 : 256;
        p.Dv = value_tile(p.Dh, p.Dhv);
        if (p.alibi || p.bias || p.dbias || p.drop_t > 0) return FA_ERR_UNSUPPORTED;
    }
    return FA_OK;
}

fa_status prepare(const void *q, const void *k, const void *v, const void *o, const void *dout,
                  const float *lse, void *dq, void *dk, void *dv, int B, int Sq, int Sk, int Hq,
                  int Hkv, int D, float scale, int causal, const int *cu_q, const int *cu_k,
                  int deterministic, fa_dtype dtype, void *ws, size_t ws_bytes,
                  cudaStream_t stream, Prepared *out, const fa_ext *ext = nullptr) {
    fa_status st = check_shape(B, Sq, Sk, Hq, Hkv, D, dtype, cu_q, cu_k);
    if (st != FA_OK) return st;
    if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, o, dout, lse, dq, dk, dv};
    for (const void *ptr : ptrs)
        if (ptr && !aligned16(ptr)) return FA_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return FA_ERR_INVALID_ARG;
    Layout L;
    if (!plan(B, Sq, Sk, Hq, Hkv, D, cu_q != nullptr, deterministic, &L)) return FA_ERR_INVALID_ARG;
    if (ws_bytes < L.total) return FA_ERR_INVALID_ARG;
    uint8_t *w = static_cast<uint8_t *>(ws);
    fa::BwdParams &p = out->p;
    std::memset(&p, 0, sizeof(p));
    p.q = q; p.k = k; p.v = v; p.o = o; p.dout = dout; p.lse = lse;
    p.dq = dq; p.dk = dk; p.dv = dv;
    p.B = B; p.Sq = Sq; p.Sk = Sk; p.Hq = Hq; p.Hkv = Hkv; p.D = bwd_pad_d(D, Sk, cu_q != nullptr);
    p.Dh = D;
    p.G = Hq / Hkv;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.causal = causal ? 1 : 0;
    p.deterministic = deterministic ? 1 : 0;
    p.varlen = cu_q != nullptr;
    p.cu_q = cu_q; p.cu_k = cu_k;
    // the extensions are host arguments too: checked before the device is
    if ((st = apply_ext(p, causal, ext)) != FA_OK) return st;
    if ((st = check_ext_totals(ext, cu_q != nullptr, B, Sq, Sk)) != FA_OK) return st;
    if ((st = apply_strides(p, ext, Sq, Sk)) != FA_OK) return st;   // (before any launch)
    // the wide kernel adds dQ without the deterministic order
    if (deterministic && wide_dims(p.Dh, p.Dhv)) return FA_ERR_UNSUPPORTED;
    st = check_device();
    if (st != FA_OK) return st;
    long long tq = (long long)B * Sq, tk = (long long)B * Sk;
    if (cu_q) {
        if ((st = packed_totals(ext, cu_q, cu_k, B, Sq, Sk, stream, &tq, &tk)) != FA_OK) return st;
        p.total_q = tq;
        p.total_k = tk;
        if ((st = apply_strides(p, ext, tq, tk)) != FA_OK) return st;
    }
    p.err = reinterpret_cast<int *>(w + L.err);
    p.ntiles = reinterpret_cast<int *>(w + L.ntiles);
    p.unit_counter = reinterpret_cast<int *>(w + L.ntiles) + 1;
    p.tiles = reinterpret_cast<int4 *>(w + L.tiles);
    p.max_tiles = L.max_tiles;
    p.num_units = L.max_tiles;
    // Unit order of the dense main kernel: the smallest group of (batch, kv
    // head) pairs -- a divisor of B * Hkv, so that no short group comes last --
    // whose units number at least 1.5 times the grid.
    // Deterministic mode adds each row block's contributions in n-block
    // order, so the units of one (sequence, kv head) wait on one another;
    // there, all pairs are interleaved (plain n-block-major order), so that
    // few units of any one chain run at the same time.
    // Varlen (the scheduler kernel builds the list): groups of consecutive
    // sequences of at least 1.5 grids of units each, the same idea; in
    // deterministic mode none (0: the plain order).
    p.unit_group = B * Hkv;
    // With intervals all pairs are one group: its units go out longest first
    // (fa_ranges.cu), and a second group's long ones would begin half way.
    if (!cu_q && !deterministic && !p.mr_row) {
        const int nblk = (Sk + fa::kBlockN - 1) / fa::kBlockN;
        const long long grid = std::min<long long>(L.max_tiles, sm_count());
        for (int g = 1; g <= B * Hkv; ++g)
            if ((B * Hkv) % g == 0 && 2LL * g * nblk >= 3 * grid) { p.unit_group = g; break; }
    } else if (cu_q) {
        const long long grid = std::min<long long>(L.max_tiles, sm_count());
        p.unit_group = deterministic ? 0 : (int)std::max<long long>(1, 3 * grid / 2);
    }
    p.dvec = reinterpret_cast<float *>(w + L.dvec);
    p.lse2 = reinterpret_cast<float *>(w + L.lse2);
    p.dqacc = reinterpret_cast<float *>(w + L.dqacc);
    p.sem = deterministic ? reinterpret_cast<int *>(w + L.sem) : nullptr;
    p.rows = L.rows;
    p.rows_per_head = L.rows_per_head;
    p.sq_round = L.sq_round;
    p.budget_ns = g_budget_ns.load();
    out->L = L;
    out->total_q = tq;
    out->total_k = tk;
    return FA_OK;
}

fa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

fa_status run_preprocess(const Prepared &P, fa_dtype dtype, cudaStream_t stream) {
    if (!P.p.o || !P.p.dout || !P.p.lse) return FA_ERR_INVALID_ARG;
    return cuda_status(fa::launch_preprocess(P.p, dtype == FA_BF16, stream));
}

// dBias (dense, main kernel only): the main kernel writes dS of the tiles it
// visits, the rest is 0.  A kernel that decodes the same units writes those
// zeros when 16-byte stores fit the tensor; else the whole tensor is zeroed
// first.
fa_status zero_dbias(const Prepared &P, cudaStream_t stream) {
    const fa::BwdParams &p = P.p;
    if ((reinterpret_cast<uintptr_t>(p.dbias) & 15u) == 0 && (p.Sk & 7) == 0)
        return cuda_status(fa::launch_dbias_zero(p, fa::main_block_m(p.D), stream));
    const size_t n = (size_t)p.B * p.Hq * p.Sq * p.Sk * 2;
    return cudaMemsetAsync(p.dbias, 0, n, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status run_main(const Prepared &P, fa_dtype dtype, cudaStream_t stream) {
    const fa::BwdParams &p = P.p;
    const bool wide = wide_dims(p.Dh, p.Dhv);
    const int bm = wide ? fa::wide_block_m() : fa::main_block_m(p.D);
    const int bf16 = dtype == FA_BF16;
    CUtensorMap mq, mk, mv, mdo;
    const long long rq = p.varlen ? P.total_q : p.Sq, rk = p.varlen ? P.total_k : p.Sk;
    const int nb = p.varlen ? 1 : p.B;
    if (rq <= 0 || rk <= 0) return FA_ERR_INVALID_ARG;
    if (!p.q || !p.k || !p.v || !p.dout || !p.dk || !p.dv) return FA_ERR_INVALID_ARG;
    if (!encode_rows_map(&mq, p.q, p.Dh, p.Hq, rq, nb, bm, bf16, p.sq) ||
        !encode_rows_map(&mdo, p.dout, p.Dhv, p.Hq, rq, nb, bm, bf16, p.sdo) ||
        !encode_rows_map(&mk, p.k, p.Dh, p.Hkv, rk, nb, fa::kBlockN, bf16, p.sk) ||
        !encode_rows_map(&mv, p.v, p.Dhv, p.Hkv, rk, nb, fa::kBlockN, bf16, p.sv))
        return FA_ERR_CUDA;
    if (p.varlen) {
        // the unit list depends on the device-resident cu_seqlens
        if (fa::launch_schedule(p, stream) != cudaSuccess) return FA_ERR_CUDA;
    }
    if (wide) {
        // units: key-block units times column halves
        const long long units = (long long)p.max_tiles * fa::wide_halves(p.D, p.Dv);
        const int grid = (int)std::min<long long>(units, sm_count());
        return cuda_status(fa::launch_bwd_wide(p, mq, mk, mv, mdo, bf16, grid, stream));
    }
    // dK / dV leave the main kernel through tensor stores of the same geometry as K / V
    CUtensorMap mdk, mdv;
    long long sdk[3], sdv[3];   // the outputs are contiguous
    set_strides(sdk, nullptr, p.varlen, rk, p.Hkv, p.Dh);
    set_strides(sdv, nullptr, p.varlen, rk, p.Hkv, p.Dhv);
    if (!encode_rows_map(&mdk, p.dk, p.Dh, p.Hkv, rk, nb, fa::kBlockN, bf16, sdk) ||
        !encode_rows_map(&mdv, p.dv, p.Dhv, p.Hkv, rk, nb, fa::kBlockN, bf16, sdv))
        return FA_ERR_CUDA;
    const int grid = (int)std::min<long long>(p.max_tiles, sm_count());
    return cuda_status(fa::launch_bwd_main(p, mq, mk, mv, mdo, mdk, mdv, bf16, grid, stream));
}

fa_status run_postprocess(const Prepared &P, fa_dtype dtype, cudaStream_t stream) {
    if (!P.p.dq) return FA_ERR_INVALID_ARG;
    return cuda_status(fa::launch_postprocess(P.p, dtype == FA_BF16, stream));
}

fa_status read_error_word(int *err_dev, cudaStream_t stream, bool clear) {
    int h = 0;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return FA_ERR_CUDA;
    if (cudaMemcpy(&h, err_dev, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return FA_ERR_CUDA;
    if (clear && h != 0 && cudaMemset(err_dev, 0, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
    // kErrBadLength: cu_seqlens or cached lengths against the sizes given; kErrBadPage
    if (h & 12) return FA_ERR_INVALID_ARG;
    return h ? FA_ERR_TIMEOUT : FA_OK;
}

}  // namespace

extern "C" {

const char *fa_status_string(fa_status s) {
    switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "device-side wait timed out";
    case FA_ERR_SCRATCH_LIMIT: return "problem needs more scratch than the fixed no-alloc array";
    }
    return "unknown status";
}

long long fa_set_wait_timeout_ns(long long ns) {
    if (ns <= 0) return g_budget_ns.load();
    return g_budget_ns.exchange(ns);
}

size_t fa_bwd_workspace_bytes(int B, int Sq, int Sk, int Hq, int Hkv, int D, int varlen,
                              int deterministic) {
    Layout L;
    if (!head_dims_ok(D, 0)) return 0;
    if (!plan(B, Sq, Sk, Hq, Hkv, D, varlen, deterministic, &L)) return 0;
    return L.total;
}

fa_status fa_bwd_workspace_layout(int B, int Sq, int Sk, int Hq, int Hkv, int D, int varlen,
                                  int deterministic, size_t *dvec_off, size_t *lse2_off,
                                  size_t *dqacc_off, size_t *rows) {
    Layout L;
    if (!head_dims_ok(D, 0)) return FA_ERR_UNSUPPORTED;
    if (!plan(B, Sq, Sk, Hq, Hkv, D, varlen, deterministic, &L)) return FA_ERR_INVALID_ARG;
    if (dvec_off) *dvec_off = L.dvec / 4;
    if (lse2_off) *lse2_off = L.lse2 / 4;
    if (dqacc_off) *dqacc_off = L.dqacc / 4;
    if (rows) *rows = (size_t)L.rows;
    return FA_OK;
}

fa_status fa_bwd_workspace_sync_layout(int B, int Sq, int Sk, int Hq, int Hkv, int D, int varlen,
                                       int deterministic, size_t *err_off, size_t *sem_off,
                                       size_t *n_sem) {
    Layout L;
    if (!head_dims_ok(D, 0)) return FA_ERR_UNSUPPORTED;
    if (!plan(B, Sq, Sk, Hq, Hkv, D, varlen, deterministic, &L)) return FA_ERR_INVALID_ARG;
    if (err_off) *err_off = L.err;
    if (sem_off) *sem_off = deterministic ? L.sem : 0;
    if (n_sem) *n_sem = deterministic ? (size_t)(L.rows / 64) : 0;
    return FA_OK;
}

fa_status fa_bwd_preprocess(const void *o, const void *dout, const float *lse, int B, int Sq,
                            int Sk, int Hq, int Hkv, int D, const int *cu_seqlens_q,
                            const int *cu_seqlens_k, int deterministic, fa_dtype dtype,
                            void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!o || !dout || !lse) return FA_ERR_INVALID_ARG;
    Prepared P;
    fa_status st = prepare(nullptr, nullptr, nullptr, o, dout, lse, nullptr, nullptr, nullptr, B,
                           Sq, Sk, Hq, Hkv, D, 1.f, 0, cu_seqlens_q, cu_seqlens_k, deterministic,
                           dtype, workspace, workspace_bytes, stream, &P);
    if (st != FA_OK) return st;
    return run_preprocess(P, dtype, stream);
}

fa_status fa_bwd_main(const void *q, const void *k, const void *v, const void *dout, void *dk,
                      void *dv, int B, int Sq, int Sk, int Hq, int Hkv, int D,
                      float softmax_scale, int causal, const int *cu_seqlens_q,
                      const int *cu_seqlens_k, int deterministic, fa_dtype dtype,
                      void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!q || !k || !v || !dout || !dk || !dv) return FA_ERR_INVALID_ARG;
    Prepared P;
    fa_status st = prepare(q, k, v, nullptr, dout, nullptr, nullptr, dk, dv, B, Sq, Sk, Hq, Hkv,
                           D, softmax_scale, causal, cu_seqlens_q, cu_seqlens_k, deterministic,
                           dtype, workspace, workspace_bytes, stream, &P);
    if (st != FA_OK) return st;
    return run_main(P, dtype, stream);
}

fa_status fa_bwd_postprocess(void *dq, int B, int Sq, int Sk, int Hq, int Hkv, int D,
                             float softmax_scale, const int *cu_seqlens_q,
                             const int *cu_seqlens_k, int deterministic, fa_dtype dtype,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!dq) return FA_ERR_INVALID_ARG;
    Prepared P;
    fa_status st = prepare(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, dq, nullptr,
                           nullptr, B, Sq, Sk, Hq, Hkv, D, softmax_scale, 0, cu_seqlens_q,
                           cu_seqlens_k, deterministic, dtype, workspace, workspace_bytes, stream,
                           &P);
    if (st != FA_OK) return st;
    return run_postprocess(P, dtype, stream);
}

fa_status fa_bwd_with_workspace(const void *q, const void *k, const void *v, const void *o,
                                const void *dout, const float *lse, void *dq, void *dk, void *dv,
                                int B, int Sq, int Sk, int Hq, int Hkv, int D,
                                float softmax_scale, int causal, const int *cu_seqlens_q,
                                const int *cu_seqlens_k, int deterministic, fa_dtype dtype,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!workspace) return FA_ERR_INVALID_ARG;   // (fa_bwd_ext would take the library's)
    return fa_bwd_ext(q, k, v, o, dout, lse, dq, dk, dv, B, Sq, Sk, Hq, Hkv, D, softmax_scale,
                      causal, cu_seqlens_q, cu_seqlens_k, nullptr, deterministic, dtype,
                      workspace, workspace_bytes, stream);
}

fa_status fa_bwd_ext(const void *q, const void *k, const void *v, const void *o,
                     const void *dout, const float *lse, void *dq, void *dk, void *dv, int B,
                     int Sq, int Sk, int Hq, int Hkv, int D, float softmax_scale, int causal,
                     const int *cu_seqlens_q, const int *cu_seqlens_k, const fa_ext *ext,
                     int deterministic, fa_dtype dtype, void *workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
    if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
    fa_status st;
    CallWorkspace own;
    if (!workspace) {
        st = check_shape(B, Sq, Sk, Hq, Hkv, D, dtype, cu_seqlens_q, cu_seqlens_k);
        if (st != FA_OK) return st;
        workspace_bytes = fa_bwd_workspace_bytes(B, Sq, Sk, Hq, Hkv, D,
                                                 cu_seqlens_q != nullptr, deterministic);
        if (workspace_bytes == 0) return FA_ERR_INVALID_ARG;
        if ((st = own.take(workspace_bytes, stream)) != FA_OK) return st;
        workspace = own.ptr;
    }
    Prepared P;
    st = prepare(q, k, v, o, dout, lse, dq, dk, dv, B, Sq, Sk, Hq, Hkv, D, softmax_scale, causal,
                 cu_seqlens_q, cu_seqlens_k, deterministic, dtype, workspace, workspace_bytes,
                 stream, &P, ext);
    if (st != FA_OK) return st;
    if (own.ptr && !deterministic) {
        // errors go where fa_device_status finds them once the workspace is gone
        P.p.err = fa::fwd_error_word();
        if (!P.p.err) return FA_ERR_CUDA;
        P.p.err_shared = 1;
    }
    if ((st = run_preprocess(P, dtype, stream)) != FA_OK) return st;
    if (P.p.dbias && (st = zero_dbias(P, stream)) != FA_OK) return st;
    if ((st = run_main(P, dtype, stream)) != FA_OK) return st;
    if ((st = run_postprocess(P, dtype, stream)) != FA_OK) return st;
    if (!deterministic) return FA_OK;
    st = read_error_word(P.p.err, stream, false);
    if (own.ptr && st != FA_OK && st != FA_ERR_CUDA) {
        int *word = fa::fwd_error_word();
        if (!word || fa::launch_error_or(P.p.err, word, stream) != cudaSuccess) return FA_ERR_CUDA;
    }
    return st;
}

fa_status fa_bwd_stages_ext(int stages, const void *q, const void *k, const void *v,
                            const void *o, const void *dout, const float *lse, void *dq,
                            void *dk, void *dv, int B, int Sq, int Sk, int Hq, int Hkv, int D,
                            float softmax_scale, int causal, const int *cu_seqlens_q,
                            const int *cu_seqlens_k, const fa_ext *ext, int deterministic,
                            fa_dtype dtype, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
    const int all = FA_STAGE_PRE | FA_STAGE_MAIN | FA_STAGE_POST;
    if (stages <= 0 || (stages & ~all) || !workspace) return FA_ERR_INVALID_ARG;
    Prepared P;
    fa_status st = prepare(q, k, v, o, dout, lse, dq, dk, dv, B, Sq, Sk, Hq, Hkv, D, softmax_scale,
                           causal, cu_seqlens_q, cu_seqlens_k, deterministic, dtype, workspace,
                           workspace_bytes, stream, &P, ext);
    if (st != FA_OK) return st;
    if ((stages & FA_STAGE_PRE) && (st = run_preprocess(P, dtype, stream)) != FA_OK) return st;
    if (stages & FA_STAGE_MAIN) {
        if (P.p.dbias && (st = zero_dbias(P, stream)) != FA_OK) return st;
        if ((st = run_main(P, dtype, stream)) != FA_OK) return st;
    }
    if ((stages & FA_STAGE_POST) && (st = run_postprocess(P, dtype, stream)) != FA_OK) return st;
    return FA_OK;
}

fa_status fa_bwd(const void *q, const void *k, const void *v, const void *o, const void *dout,
                 const float *lse, void *dq, void *dk, void *dv, int B, int Sq, int Sk, int Hq,
                 int Hkv, int D, float softmax_scale, int causal, const int *cu_seqlens_q,
                 const int *cu_seqlens_k, int deterministic, fa_dtype dtype,
                 cudaStream_t stream) {
    return fa_bwd_ext(q, k, v, o, dout, lse, dq, dk, dv, B, Sq, Sk, Hq, Hkv, D, softmax_scale, causal,
                      cu_seqlens_q, cu_seqlens_k, nullptr, deterministic, dtype, nullptr, 0, stream);
}

fa_status fa_device_status(void *workspace, cudaStream_t stream) {
    int *word = workspace ? static_cast<int *>(workspace) : fa::fwd_error_word();
    if (!word) return FA_ERR_CUDA;
    return read_error_word(word, stream, true);
}

namespace {

// The cache's host-visible fields; fills the kernels' parameter block.
fa_status check_kv_cache(const fa_kv_cache *c, int B, fa_dtype dtype, fa::KvCacheParams *p) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table) return FA_ERR_INVALID_ARG;
    if (B <= 0 || c->num_pages <= 0 || c->page_size <= 0 || c->max_pages <= 0 || c->Hkv <= 0)
        return FA_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) ||
        (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) || (reinterpret_cast<uintptr_t>(c->block_table) & 3u))
        return FA_ERR_INVALID_ARG;
    if (c->page_size % 16 != 0 || c->page_size > 128) return FA_ERR_UNSUPPORTED;
    if (c->D != 64 && c->D != 128) return FA_ERR_UNSUPPORTED;
    if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
    if ((long long)c->max_pages * c->page_size > 0x7fffffffLL - 128) return FA_ERR_INVALID_ARG;   // token indices
    p->k = static_cast<uint8_t *>(c->k);
    p->v = static_cast<uint8_t *>(c->v);
    p->k_scale = c->k_scale;
    p->v_scale = c->v_scale;
    p->table = c->block_table;
    p->num_pages = c->num_pages;
    p->page = c->page_size;
    p->max_pages = c->max_pages;
    p->Hkv = c->Hkv;
    return FA_OK;
}

}  // namespace

fa_status fa_kvcache_append(const fa_kv_cache *cache, const int *cache_len, const void *k_new, const void *v_new,
                            const int *cu_new, int rows, int B, int max_new, fa_dtype dtype,
                            cudaStream_t stream) {
    fa::KvAppendParams p;
    std::memset(&p, 0, sizeof(p));
    fa_status st = check_kv_cache(cache, B, dtype, &p.c);
    if (st != FA_OK) return st;
    if (!cache_len || !k_new || !v_new || rows <= 0 || max_new <= 0) return FA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || (reinterpret_cast<uintptr_t>(cache_len) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu_new) & 3u))
        return FA_ERR_INVALID_ARG;
    if ((long long)B * max_new > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    if (!cu_new && rows != B * max_new) return FA_ERR_INVALID_ARG;
    if (cache->Hkv > 65535) return FA_ERR_UNSUPPORTED;   // grid columns
    if ((st = check_device()) != FA_OK) return st;
    p.c.err = fa::fwd_error_word();
    if (!p.c.err) return FA_ERR_CUDA;
    p.len = cache_len;
    p.cu = cu_new;
    p.k = k_new;
    p.v = v_new;
    p.rows = rows;
    p.B = B;
    p.max_new = max_new;
    return cuda_status(fa::launch_kv_append(p, cache->D, dtype == FA_BF16, stream));
}

size_t fa_fwd_kvcache_workspace_bytes(int D) { return (D == 64 || D == 128) ? fa::kv_workspace_bytes(D) : 0; }

fa_status fa_fwd_kvcache(const void *q, const fa_kv_cache *cache, const int *cache_len, void *o, float *lse, int B,
                         int Sq, int Hq, float softmax_scale, float softcap, int window_left, fa_dtype dtype,
                         void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    fa::KvAttnParams p;
    std::memset(&p, 0, sizeof(p));
    fa_status st = check_kv_cache(cache, B, dtype, &p.c);
    if (st != FA_OK) return st;
    if (!q || !o || !cache_len || !workspace || Sq <= 0 || Hq <= 0 || Hq % cache->Hkv != 0)
        return FA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
        (reinterpret_cast<uintptr_t>(cache_len) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(softmax_scale) && softmax_scale > 0.f) || window_left < -1) return FA_ERR_INVALID_ARG;
    if (softcap != 0.f && !(softcap >= kMinSoftcap && softcap <= kMaxSoftcap)) return FA_ERR_INVALID_ARG;
    if (B > fa::kKvMaxSeqs) return FA_ERR_UNSUPPORTED;
    if ((long long)Sq * Hq > (1 << 24)) return FA_ERR_UNSUPPORTED;
    p.scale_log2 = softmax_scale * kLog2e;
    if (softcap != 0.f) {
        p.cap_log2 = softcap * kLog2e;
        p.cap_k = 2.f * p.scale_log2 / softcap;
        if (!std::isfinite(p.cap_k)) return FA_ERR_INVALID_ARG;
    }
    const size_t need = fa_fwd_kvcache_workspace_bytes(cache->D);
    if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
    p.len = cache_len;
    p.q = q;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.Sq = Sq;
    p.Hq = Hq;
    p.G = Hq / cache->Hkv;
    // tiles of all sequences, heads and row groups are counted in 32 bits
    const long long groups = ((long long)p.G * Sq + 7) / 8;
    const long long tiles = 2 * ((long long)cache->max_pages * cache->page_size / 64 + 3);   // in halves
    if (tiles * B > 0x7fffffffLL / ((long long)cache->Hkv * groups)) return FA_ERR_UNSUPPORTED;
    // rows of V as the tensor loads see it
    if ((long long)cache->num_pages * cache->Hkv * cache->D > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    p.window = std::min(window_left, 1 << 30);   // positions stay inside 32 bits
    if ((st = check_device()) != FA_OK) return st;
    p.c.err = fa::fwd_error_word();
    if (!p.c.err) return FA_ERR_CUDA;
    const size_t n = (size_t)fa::kKvSms * fa::kv_max_warps(cache->D);
    uint8_t *w = static_cast<uint8_t *>(workspace);
    p.acc = reinterpret_cast<float *>(w);
    p.stat = reinterpret_cast<float4 *>(w + n * 2 * 16 * cache->D * sizeof(float));
    p.meta = reinterpret_cast<int4 *>(w + fa::kv_pieces_bytes(n, cache->D));
    p.budget_ns = g_budget_ns.load();
    const int ps = cache->page_size;
    p.v_block = ps % 64 == 0 ? 64 : ps % 32 == 0 ? 32 : 16;
    // pads that spread the blocks of a lane's four rows over the banks; tensor
    // loads (a block narrower than its page) need 128-byte destinations
    p.v_pad = p.v_block != ps || ps == 64 ? 0 : ps == 32 ? 64 : 32;
    CUtensorMap mv;
    if (!encode_v_map(&mv, cache->v, ps, (long long)cache->num_pages * cache->Hkv * cache->D, p.v_block, cache->D))
        return FA_ERR_CUDA;
    return cuda_status(fa::launch_kv_attn(p, mv, cache->D, dtype == FA_BF16, sm_count(), stream));
}

size_t fa_ext_bytes(void) { return sizeof(fa_ext); }

size_t fa_mask_ranges_bytes(int B, int S) {
    if (B <= 0 || S <= 0 || S > fa::kMaxRangeSeq || (long long)B * S > (1LL << 31) - 1) return 0;
    return fa::range_tables(nullptr, B, S).bytes;
}

fa_status fa_mask_ranges(const int *doc_ids, const int *prefix_len, int prefix_per_token, int B, int S,
                         int causal, int window_left, int window_right, void *ranges, size_t ranges_bytes,
                         cudaStream_t stream) {
    const size_t need = fa_mask_ranges_bytes(B, S);
    if (need == 0 || !ranges || (reinterpret_cast<uintptr_t>(ranges) & 255u) || ranges_bytes < need)
        return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(doc_ids) & 3u) || (reinterpret_cast<uintptr_t>(prefix_len) & 3u))
        return FA_ERR_INVALID_ARG;
    if (window_left < -1 || window_right < -1) return FA_ERR_INVALID_ARG;
    // a prefix joined to a window, or to rows that see all keys anyway, is not
    // one interval / has no effect
    if (prefix_len && (!causal || window_left != -1 || window_right != -1)) return FA_ERR_INVALID_ARG;
    if (B > 65535) return FA_ERR_UNSUPPORTED;   // grid rows
    fa_status st = check_device();
    if (st != FA_OK) return st;
    if (causal) window_right = 0;
    const fa::RangeTables t = fa::range_tables(ranges, B, S);
    return cuda_status(fa::launch_mask_ranges(doc_ids, prefix_len, prefix_per_token ? 1 : 0, B, S, window_left,
                                              window_right, t, stream));
}

fa_status fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Sq,
                 int Sk, int Hq, int Hkv, int D, float softmax_scale, int causal,
                 const int *cu_seqlens_q, const int *cu_seqlens_k, fa_dtype dtype,
                 cudaStream_t stream) {
    return fa_fwd_ext(q, k, v, o, lse, B, Sq, Sk, Hq, Hkv, D, softmax_scale, causal, cu_seqlens_q,
                      cu_seqlens_k, nullptr, dtype, stream);
}

fa_status fa_fwd_ext(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                     int Sq, int Sk, int Hq, int Hkv, int D, float softmax_scale, int causal,
                     const int *cu_seqlens_q, const int *cu_seqlens_k, const fa_ext *ext,
                     fa_dtype dtype, cudaStream_t stream) {
    if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
    fa_status st = check_shape(B, Sq, Sk, Hq, Hkv, D, dtype, cu_seqlens_q, cu_seqlens_k);
    if (st != FA_OK) return st;
    if (!(std::isfinite(softmax_scale) && softmax_scale > 0.f)) return FA_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, o, lse};
    for (const void *ptr : ptrs)
        if (!aligned16(ptr)) return FA_ERR_INVALID_ARG;
    fa::BwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = q; p.k = k; p.v = v;
    p.B = B; p.Sq = Sq; p.Sk = Sk; p.Hq = Hq; p.Hkv = Hkv; p.D = pad_d(D); p.Dh = D;
    p.G = Hq / Hkv;
    p.scale = softmax_scale;
    p.scale_log2 = softmax_scale * kLog2e;
    p.causal = causal ? 1 : 0;
    p.varlen = cu_seqlens_q != nullptr;
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    if ((st = apply_ext(p, causal, ext)) != FA_OK) return st;
    if ((st = check_ext_totals(ext, p.varlen, B, Sq, Sk)) != FA_OK) return st;
    if ((st = apply_strides(p, ext, Sq, Sk)) != FA_OK) return st;
    if ((st = check_device()) != FA_OK) return st;
    p.err = fa::fwd_error_word();
    if (!p.err) return FA_ERR_CUDA;
    p.budget_ns = g_budget_ns.load();
    long long rq = Sq, rk = Sk;
    if (p.varlen) {
        st = packed_totals(ext, cu_seqlens_q, cu_seqlens_k, B, Sq, Sk, stream, &rq, &rk);
        if (st != FA_OK) return st;
        p.total_q = rq;
        p.total_k = rk;
        if (rq == 0) return FA_OK;
    }
    // a map needs at least one row; with no keys at all no K/V tile is loaded
    rk = std::max<long long>(rk, 1);
    if (p.varlen && (st = apply_strides(p, ext, rq, rk)) != FA_OK) return st;
    const int bf16 = dtype == FA_BF16;
    const int nb = p.varlen ? 1 : B;
    CUtensorMap mq, mk, mv;
    const int bn = fa::fwd_block_n(p, sm_count());
    if (!encode_rows_map(&mq, q, D, Hq, rq, nb, fa::fwd_block_m(), bf16, p.sq) ||
        !encode_rows_map(&mk, k, D, Hkv, rk, nb, bn, bf16, p.sk) ||
        !encode_rows_map(&mv, v, p.Dhv, Hkv, rk, nb, bn, bf16, p.sv))
        return FA_ERR_CUDA;
    return cuda_status(fa::launch_fwd_tc(p, mq, mk, mv, o, lse, Sq, bf16, sm_count(), stream));
}

}  // extern "C"
