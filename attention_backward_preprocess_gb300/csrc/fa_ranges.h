// fa_ranges.h -- the buffer of visible-key intervals that fa_mask_ranges
// fills and the attention kernels read, and its layout.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "fa_params.h"

namespace fa {

// Longest sequence: its rows rounded up to a CTA's, and the search for a document's
// end one step past them (4096 ids), are counted in 32 bits.
constexpr int kMaxRangeSeq = 0x7fffffff - 2 * 4096;

// Per sequence, rows = S rounded up to 128 (rows past S see nothing):
struct RangeTables {
    int rows;
    int2 *row;     // [B][rows]        keys [x, y) the row sees
    int4 *block;   // [B][rows / 64]   over the rows below S of a 64-row block: min lo and
                   //                  max hi of those that see a key (INT_MAX, 0: none);
                   //                  max lo and min hi of all
    int4 *key;     // [B][rows / 128]  row blocks [x, y) the unit of a key block works on, and
                   //                  [z, w) of them whose rows all see the whole key block (a
                   //                  run; the others are tested row by row)
    int *first;    // [B][rows / 64]   first key block whose unit works on the row block
    int *last;     // [B][rows / 64]   running maximum of the last key block (scratch)
    int *order;    // [B][rows / 128]  key blocks, the most row blocks first
    size_t bytes;
};

inline RangeTables range_tables(void *base, int B, int S) {
    RangeTables t;
    const size_t R = ((size_t)S + kRowTile - 1) / kRowTile * kRowTile;
    uint8_t *p = static_cast<uint8_t *>(base);
    size_t off = 0;
    t.rows = (int)R;
    auto take = [&](size_t n) {
        uint8_t *r = base ? p + off : nullptr;
        off = (off + n + 255) / 256 * 256;
        return r;
    };
    t.row = reinterpret_cast<int2 *>(take((size_t)B * R * sizeof(int2)));
    t.block = reinterpret_cast<int4 *>(take((size_t)B * (R / 64) * sizeof(int4)));
    t.key = reinterpret_cast<int4 *>(take((size_t)B * (R / kBlockN) * sizeof(int4)));
    t.first = reinterpret_cast<int *>(take((size_t)B * (R / 64) * sizeof(int)));
    t.last = reinterpret_cast<int *>(take((size_t)B * (R / 64) * sizeof(int)));
    t.order = reinterpret_cast<int *>(take((size_t)B * (R / kBlockN) * sizeof(int)));
    t.bytes = off;
    return t;
}

cudaError_t launch_mask_ranges(const int *doc, const int *prefix, int prefix_per_token, int B, int S, int wl,
                               int wr, const RangeTables &t, cudaStream_t stream);

}  // namespace fa
