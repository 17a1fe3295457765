// fa_kvcache.h -- parameter blocks of the paged key / value caches.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

// The 8-bit cache: e4m3 values, K as [page][kv head][token][d], V as [page][kv
// head][d][token], one power-of-two scale per (page, kv head).
// The 4-bit cache: codes as [page][kv head][token][d / 2] for both, and in place of
// the scales [page][kv head][token][d / 64] words of bf16 (scale, middle).
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

struct KvReadParams {
    KvCacheParams c;
    const int *len, *first, *cu;   // [B] tokens held, [B] first token read (null: 0), [B + 1] rows
    void *k, *v;           // [rows, Hkv, D]
    int rows, B;
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
    int bf16;                    // 4-bit cache: q's and o's type
};

// Has a wait taken more than twice its budget (up to the largest, whose double is out of range)?
#ifdef __CUDACC__
__host__ __device__
#endif
inline bool twice_over(uint64_t waited, long long budget) { return waited / 2 > (uint64_t)budget; }

// Workers of the attention kernel at most: kv_max_warps(D) warps of kKvSms CTAs.
// The grid is the device's SM count (152 on GB300), held at kKvSms.
constexpr int kKvSms = 160;
constexpr int kv_max_warps(int D) { return D == 128 ? 8 : 12; }
constexpr int kKvMaxSeqs = 4096;   // sequences whose tile counts fit shared memory
// bytes of two pieces of 16 rows for n holders: fragments, then statistics
inline size_t kv_pieces_bytes(size_t n, int D) { return n * 2 * 16 * (D * sizeof(float) + sizeof(float4)); }
size_t kv_workspace_bytes(int D);
// Half tiles that opening and closing a segment counts as where work is shared out.
constexpr int kKvOpen = 2, kKv4Open = 4;
// The 4-bit cache's attention has workers of its own number.
constexpr int kKv4MaxWarps = 8;
inline size_t kv4_workers() { return (size_t)kKvSms * kKv4MaxWarps; }

cudaError_t launch_kv_append(const KvAppendParams &p, int D, int bf16, cudaStream_t stream);
cudaError_t launch_kv_attn(const KvAttnParams &p, const CUtensorMap &map_v, int D, int bf16, int sms,
                           cudaStream_t stream);
cudaError_t launch_kv4_append(const KvAppendParams &p, int D, int bf16, int sms, cudaStream_t stream);
cudaError_t launch_kv4_read(const KvReadParams &p, int D, int bf16, int sms, cudaStream_t stream);
cudaError_t launch_kv4_attn(const KvAttnParams &p, const CUtensorMap &map_k, const CUtensorMap &map_v, int D, int sms,
                            cudaStream_t stream);

}  // namespace fa
