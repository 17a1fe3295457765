// fa_rope.h -- parameter block of the rotary-position kernel.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fa {

struct RopeTensor {
    const void *in;
    void *out;
    long long is[3], os[3];   // (batch, row, head) strides in elements
};

struct RopeParams {
    RopeTensor t[2];          // q, k
    int heads[2];             // k: 0 where there is none
    int B, S, D, R;
    const unsigned long long *steps;   // [R / 2] parts of a turn per position, 2^-64ths
    const int *positions;     // [B S]; null: offsets[b] + s
    const int *offsets;       // [B]; null: 0
    float factor;
    int inverse;
    int in_place;             // out is in: the dims behind R stay
    // filled by launch_rope
    int units;                // pieces of a head a thread takes at a time
    int heads_at_once;        // heads whose pieces a CTA's threads cover, in rows
    int step_rows, step_heads;   // and heads beyond them
    int rows_per_cta;
    uint32_t by_units;        // divides a thread's number by units
    int batches;              // sequences with rows apart from each other (1: all rows evenly spaced)
};

cudaError_t launch_rope(RopeParams p, int interleaved, int bf16, int sms, cudaStream_t stream);

}  // namespace fa
