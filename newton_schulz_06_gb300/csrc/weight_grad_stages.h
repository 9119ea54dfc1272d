// The stages of the weight gradient's rings and which barrier phase a step
// waits for: plain C++, so that tests/weight_grad_stages.cpp plays the waits
// through on the CPU, with loads that arrive in any order.
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

constexpr int W_DEC_GROUPS = 2;      // groups of decoding warps, which take the steps in turn

// Stages of dY (A), of the decoded values (B) and of the 8-bit ones (R).  The
// rings of WIDE are as long as the shared memory allows, and each has its own
// barriers; in the other shape the three share a step's stage and R's loads
// A's barrier, because the decoding warps have no time for more (345 -> 444 us
// with 4096 tokens of 7168 x 8192).
template <bool WIDE>
struct Stages {
    static constexpr int A = WIDE ? 4 : 5, B = WIDE ? 3 : 5, R = WIDE ? 4 : 5;
    static constexpr int AHEAD = R - 2;      // steps that R's loads run ahead of A's (WIDE)
    static_assert(!WIDE || R % W_DEC_GROUPS == 0, "a stage of R is one group's");
};

// The stage of a step in a ring of n, and the parity of the step's phase of
// that stage's barrier.
MUON_HD uint32_t stage_of(uint32_t step, uint32_t n) { return step % n; }
MUON_HD uint32_t parity_of(uint32_t step, uint32_t n) { return step / n & 1; }

// A wait for a parity also returns while the phase before the one that is
// meant has not completed: a group may only wait for a phase of a stage whose
// earlier phases it knows to be over.  Of its own steps it knows; the stage's
// last user may have been the other group's step.  So every step waits for the
// products of the step that last had its stage of B: they read all that was
// loaded and decoded for that step, and those before it ran in order.  It does
// so before anything else unless the stages of R are a group's own.
template <bool WIDE>
MUON_HD bool stage_was_used(uint32_t step) { return step >= uint32_t(Stages<WIDE>::B); }
template <bool WIDE>
MUON_HD uint32_t last_user(uint32_t step) { return step - uint32_t(Stages<WIDE>::B); }

}  // namespace ops
}  // namespace muon
