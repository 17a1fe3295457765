// Walks every interleaving of the main backward kernel's softmax warps over the
// hand-off of the two dS^T tiles from one unit's dK / dV stores to the next
// unit's dS^T, with the phase arithmetic of csrc/fa_epilogue.h itself.  Two groups
// of two warps (a leader and another one), three units.  Prints one line:
// "ok <states>" or the first fault found.
//   argv: slices per unit, 3 x (1: the unit stores through the tiles, 0: not), protocol
//   protocol 0: as the kernel runs it
//            1: a wait for the other group's slice barrier behind the unit instead
//            2: no wait at all
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>
#include <vector>

#include "fa_epilogue.h"

namespace {

constexpr int kGroups = 2, kWarps = 2, kUnits = 3;

struct Barrier {   // an mbarrier: arrivals of the phase in progress, phases completed
    uint8_t count, got, done;
    void arrive() {
        if (++got == count) got = 0, ++done;
    }
    bool passed(uint32_t parity) const { return (done & 1u) != parity; }   // try_wait.parity
};
struct Warp {
    uint8_t pc, unit, slice, bits;
};
struct State {
    Warp w[kGroups][kWarps];
    Barrier full[kGroups], free_[kGroups], done;
    uint8_t staged[kGroups];   // the tile holds a slice, or part of one, no store has read
    uint8_t out[kGroups];      // units whose last slice the group's store has read
    uint8_t ds[kUnits];        // warps that wrote their dS^T of the unit
};

int slices, protocol, stores[kUnits];

// One step of a warp: false if it has to wait; *fault: what went wrong.
bool step(State &s, int g, int v, std::string *fault) {
    Warp &w = s.w[g][v];
    fa::EpiPhases epi;
    epi.bits = w.bits;
    auto next_unit = [&] { w.unit++, w.slice = 0, w.pc = 0; };
    switch (w.pc) {
    case 0:   // before the unit
        if (protocol == 0 && !s.done.passed(epi.stored())) return false;
        w.pc = 1;
        break;
    case 1: {   // dS^T lands in either tile
        int before = 0;
        for (int u = 0; u < w.unit; ++u) before += stores[u];
        for (int o = 0; o < kGroups; ++o)
            if (s.staged[o] || s.out[o] < before) *fault = "dS^T of a unit written under a store of the unit before";
        s.ds[w.unit]++;
        if (stores[w.unit]) w.pc = 2;
        else w.pc = 8;
        break;
    }
    case 2:   // the dQ products (and the chunks parked in the tiles) are done with the unit's dS^T
        if (s.ds[w.unit] < kGroups * kWarps) return false;
        w.pc = 3;
        break;
    case 8:   // a unit whose results leave without the tiles
        if (s.ds[w.unit] < kGroups * kWarps) return false;
        next_unit();
        break;
    case 3:   // stage a slice
        if (s.ds[w.unit] < kGroups * kWarps || (w.unit + 1 < kUnits && s.ds[w.unit + 1])) *fault = "a slice staged over dS^T";
        if (s.staged[g] == 2) *fault = "a slice staged under the store of the one before";
        s.staged[g] = 1;
        s.full[g].arrive();
        w.pc = v == 0 ? 4 : 6;
        break;
    case 4:   // the leader issues the store
        if (!s.full[g].passed(epi.staged())) return false;
        s.staged[g] = 2;
        w.pc = 5;
        break;
    case 5:   // the store has read the tile
        s.staged[g] = 0;
        if (w.slice == slices - 1) s.out[g]++;
        if (w.slice == slices - 1) s.done.arrive();
        if (w.slice < slices - 1 || protocol == 1) s.free_[g].arrive();
        w.pc = 6;
        break;
    case 6:
        if (protocol == 1) {   // its slice barrier has a phase for every slice
            if (!s.free_[g].passed(epi.staged())) return false;
        } else if (w.slice < slices - 1) {
            if (!s.free_[g].passed(epi.freed())) return false;
            epi.next_freed();
        }
        epi.next_staged();
        if (++w.slice < slices) {
            w.pc = 3;
            break;
        }
        epi.unit_stored();
        if (protocol == 1) w.pc = 7;
        else next_unit();
        break;
    case 7:
        if (!s.free_[g ^ 1].passed(epi.staged() ^ 1u)) return false;
        next_unit();
        break;
    }
    w.bits = (uint8_t)epi.bits;
    return true;
}

}  // namespace

int main(int argc, char **argv) {
    if (argc != 6) return 2;
    slices = std::atoi(argv[1]);
    for (int u = 0; u < kUnits; ++u) stores[u] = std::atoi(argv[2 + u]);
    protocol = std::atoi(argv[5]);
    State s0;
    std::memset(&s0, 0, sizeof(s0));
    for (int g = 0; g < kGroups; ++g) s0.full[g].count = kWarps, s0.free_[g].count = 1;
    s0.done.count = kGroups;
    auto key = [](const State &s) { return std::string(reinterpret_cast<const char *>(&s), sizeof(s)); };
    std::set<std::string> seen{key(s0)};
    std::vector<State> todo{s0};
    while (!todo.empty()) {
        const State s = todo.back();
        todo.pop_back();
        bool moved = false, left = false;
        for (int g = 0; g < kGroups; ++g)
            for (int v = 0; v < kWarps; ++v) {
                if (s.w[g][v].unit == kUnits) continue;
                left = true;
                State n = s;
                std::string fault;
                if (!step(n, g, v, &fault)) continue;
                moved = true;
                if (!fault.empty()) {
                    std::printf("%s\n", fault.c_str());
                    return 0;
                }
                if (seen.insert(key(n)).second) todo.push_back(n);
            }
        if (left && !moved) {
            std::printf("no warp can go on\n");
            return 0;
        }
    }
    std::printf("ok %zu\n", seen.size());
    return 0;
}
