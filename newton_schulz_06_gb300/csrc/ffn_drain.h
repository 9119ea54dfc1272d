// What a CTA pair of the gated feed-forward kernels still has in flight when a
// wait has run out: plain C++, so that tests/ffn_drain.cpp plays loads and
// aborts through on the CPU.
//
// A step's boxes are asked for by two threads a CTA, and counted on one
// barrier: the leader's of that stage for all four threads, or, where a step
// is short, each CTA's own for its two.  The first of them arms the phase with
// the bytes of all.  A pair that gives up may leave a stage that only some of
// them have asked for: then the phase either expects bytes that never come, or
// is not armed and its barrier says nothing about those under way.
#pragma once

#include <cstdint>

#ifndef MUON_HD
#ifdef __CUDACC__
#define MUON_HD __host__ __device__ __forceinline__
#else
#define MUON_HD inline
#endif
#endif

namespace muon {
namespace ops {

// What a loading thread has asked for.
struct Asked {
    uint32_t steps;          // so many steps, from the first one on
    uint32_t tails, two;     // a bit a stage: its last step was a short one; had two boxes of B
    uint32_t full, tail;     // a bit a stage: whole and short steps it has had, modulo 2
};

// The last of `steps` steps that had the stage: false if none had.
MUON_HD bool last_step(uint32_t steps, uint32_t stage, uint32_t stages, uint32_t* step) {
    if (steps <= stage) return false;
    *step = steps - 1 - (steps - 1 - stage) % stages;
    return true;
}

// What makes the barrier's phase end when the last byte that was asked for is
// there: arm it with these bytes (nobody has), or take these off (they were
// never asked for), and wait for the parity.
struct Settle {
    uint32_t arm, cancel, parity;
    bool wait;
};

// Of one stage's barrier.  by: the threads that load for it, the first of
// which arms it; bytes(i, two): what thread i asks for.  Only the last step
// that any of them asked for can be in flight: a stage is loaded again when its
// products have run.  tail: of the short steps' barrier.
template <typename Bytes>
MUON_HD Settle settle(const Asked* by, int n, uint32_t stage, uint32_t stages, bool tail, Bytes bytes) {
    Settle s{0, 0, 0, false};
    uint32_t step = 0;
    int who = -1;
    for (int i = 0; i < n; ++i) {
        uint32_t at;
        if (last_step(by[i].steps, stage, stages, &at) && (who < 0 || at > step)) {
            step = at;
            who = i;
        }
    }
    if (who < 0 || (by[who].tails >> stage & 1) != (tail ? 1u : 0u)) return s;
    const bool two = by[who].two >> stage & 1;
    uint32_t asked = 0, all = 0;
    for (int i = 0; i < n; ++i) {
        all += bytes(i, two);
        if (by[i].steps > step) asked += bytes(i, two);
    }
    if (by[0].steps > step) s.cancel = all - asked;
    else s.arm = asked;
    s.parity = ((tail ? by[who].tail : by[who].full) >> stage & 1) ^ 1;
    s.wait = true;
    return s;
}

}  // namespace ops
}  // namespace muon
