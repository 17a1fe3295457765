// fa_epilogue.h -- how a unit's dK / dV stores hand the two dS^T tiles on to the
// next unit, in barrier phases.  Plain C++ without CUDA, so that a test on the CPU
// can walk every interleaving of the warps through the very code the kernel runs.
//
// Softmax group g stages its dK or dV in dS^T tile g, in slices of 64 columns: two
// at D = 128, one at D = 64.  Per slice the group's warps arrive on B_EPI_FULL + g
// and its leader stores the tile.  Once the store has read it, the leader arrives
// on B_EPI_FREE + g, for which the group waits before it stages its next slice,
// or after the last slice on B_EPI_DONE (both leaders: count 2), for which every
// softmax warp waits before it begins its next unit with work.  No phase of
// any of them can thus complete before every waiter has looked at the one before
// it, and one parity bit each is enough.  (A group must not look at the other's
// slice barriers: with two phases a unit the parity behind a unit is the same in
// every unit, and a wait for it lets through exactly the group whose other one has
// no slice out yet.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FA_EPI_FN __host__ __device__ __forceinline__
#else
#define FA_EPI_FN inline
#endif

namespace fa {

struct EpiPhases {
    // counts mod 2 -- bit 0: slices of the own group staged, bit 1: units with
    // stores, bit 2: slices of the own group but a unit's last
    uint32_t bits = 0;
    static constexpr int slices(int D) { return D / 64; }
    // parity of the own group's B_EPI_FULL to wait for in the present slice
    FA_EPI_FN uint32_t staged() const { return bits & 1u; }
    FA_EPI_FN void next_staged() { bits ^= 1u; }
    // parity of the own group's B_EPI_FREE to wait for behind a slice but the last
    FA_EPI_FN uint32_t freed() const { return bits >> 2 & 1u; }
    FA_EPI_FN void next_freed() { bits ^= 4u; }
    // parity of B_EPI_DONE to wait for before a unit with work: the stores of the
    // last unit that had any (before the first one the wait passes)
    FA_EPI_FN uint32_t stored() const { return (bits >> 1 & 1u) ^ 1u; }
    FA_EPI_FN void unit_stored() { bits ^= 2u; }
};

}  // namespace fa
