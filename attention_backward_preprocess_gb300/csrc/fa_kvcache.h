// fa_kvcache.h -- parameter blocks of the 8-bit paged key / value cache.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

// The cache: e4m3 values, K as [page][kv head][token][d], V as [page][kv
// head][d][token], one power-of-two scale per (page, kv head).
struct KvCacheParams {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    const int *table;      // [B, max_pages] page numbers
    int num_pages, page, max_pages, Hkv;
    int *err;              // device error word
};

struct KvAppendParams {
    KvCacheParams c;
    const int *len;        // [B] tokens held before the call
    const int *cu;         // [B + 1] rows of the new tokens; null: max_new each
    const void *k, *v;     // [rows, Hkv, D]
    int rows, B, max_new;
};

struct KvAttnParams {
    KvCacheParams c;
    const int *len;        // [B] tokens held, the queries' own among them
    const void *q;         // [B, Sq, Hq, D]
    void *o;
    float *lse;            // [B, Hq, Sq]; null: not written
    int B, Sq, Hq, G;
    int groups;            // row groups (8 or 16 (query, head) rows) per kv head
    int window;            // keys a query sees before its own; < 0: all
    float scale_log2;      // c log2(e)
    float cap_log2, cap_k; // softcap log2(e) and 2 log2(e) c / softcap; 0: no cap
    // workspace: two pieces of up to 16 rows per worker
    float *acc;            // [workers][2] pieces in fragment order
    float4 *stat;          // [workers][2][rows]  (m, l, R, -)
    int4 *meta;            // [workers]  piece 0: segment, sequence, first worker, ends here
    int workers;
    uint32_t page_magic;         // divides by page / 16 (0: by 1)
    // V reaches shared memory in blocks of v_block tokens (64, 32 or 16: the
    // widest that divides a page's tokens), v_pad bytes apart
    int v_block, v_pad;
    long long budget_ns;         // bound of every device-side wait
};

// Workers of the attention kernel at most: kv_max_warps(D) warps of kKvSms CTAs.
// The grid is the device's SM count (152 on GB300), held at kKvSms.
constexpr int kKvSms = 160;
constexpr int kv_max_warps(int D) { return D == 128 ? 8 : 12; }
constexpr int kKvMaxSeqs = 4096;   // sequences whose tile counts fit shared memory
// bytes of two pieces of 16 rows for n holders: fragments, then statistics
inline size_t kv_pieces_bytes(size_t n, int D) { return n * 2 * 16 * (D * sizeof(float) + sizeof(float4)); }
size_t kv_workspace_bytes(int D);

cudaError_t launch_kv_append(const KvAppendParams &p, int D, int bf16, cudaStream_t stream);
cudaError_t launch_kv_attn(const KvAttnParams &p, const CUtensorMap &map_v, int D, int bf16, int sms,
                           cudaStream_t stream);

}  // namespace fa
