// fa_epilogue.h -- how a unit's dK / dV stores hand the two dS^T tiles on to the
// next unit, in barrier phases.  Plain C++ without CUDA, so that a test on the CPU
// can walk every interleaving of the warps through the very code the kernel runs.
//
// Softmax group g stages its dK or dV in dS^T tile g, in slices of 64 columns: two
// at D = 128, one at D = 64.  Per slice the group's warps arrive on B_EPI_FULL + g,
// its leader stores the tile and arrives on B_EPI_FREE + g once it has been read:
// slices() phases a unit, waited for by the group itself.  The other group must
// not count those (with two per unit the parity behind a unit is the same in every
// unit, so that a wait for it holds back nothing while no slice is out yet): each
// leader also arrives once a unit, after its last slice, on B_EPI_DONE (count 2),
// and every softmax warp waits for that before its first dS^T write of the next
// unit.  A phase of B_EPI_DONE thus cannot complete before every warp has looked
// at the one before it, and one parity bit each is enough.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FA_EPI_FN __host__ __device__ __forceinline__
#else
#define FA_EPI_FN inline
#endif

namespace fa {

struct EpiPhases {
    uint32_t bits = 0;   // bit 0: slices of the own group, bit 1: units with stores (both mod 2)
    static constexpr int slices(int D) { return D / 64; }
    // parity of B_EPI_FULL / B_EPI_FREE (own group) to wait for in the present slice
    FA_EPI_FN uint32_t slice() const { return bits & 1u; }
    FA_EPI_FN void next_slice() { bits ^= 1u; }
    // parity of B_EPI_DONE to wait for before a unit's first dS^T write: the stores
    // of the last unit that had any (before the first one the wait passes)
    FA_EPI_FN uint32_t stored() const { return (bits >> 1 & 1u) ^ 1u; }
    FA_EPI_FN void unit_stored() { bits ^= 2u; }
};

}  // namespace fa
