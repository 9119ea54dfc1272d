// What a CTA pair of the gated feed-forward kernels still has in flight when a
// wait has run out: plain C++, so that tests/ffn_drain.cpp plays loads and
// aborts through on the CPU.
//
// A step's boxes are asked for by two threads a CTA, and counted on one
// barrier: the leader's of that stage for all four threads, or, where the step
// is torn (its last 16 rows are not all the expert's), each CTA's own for its
// two.  Then a warp a CTA asks for zeros over those rows, which count on another
// barrier of the leader's.  The first of each set arms the phase with the bytes of
// all.  A pair that gives up may leave a stage that only some of them have asked
// for: then the phase either expects bytes that never come, or is not armed and
// its barrier says nothing about those under way.
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

constexpr uint32_t DRAIN_BOX = 64 * 64 * 2;      // bytes of a box: 64 rows of 128

// What a loading thread has asked for, or (steps alone) a clearing warp.
struct Asked {
    uint32_t steps;          // so many steps, from the first one on
    uint32_t two;            // a bit a stage: its last step has two boxes of B
    uint32_t torn;           // a bit a stage: its last step is torn,
    uint32_t gaps;           // and has so many rows to clear (four bits a stage)
    uint32_t times;          // a bit a stage: torn steps it has had, modulo 2
};

// n more steps of a tile, the first of them in this stage; gap: the last one's
// (0: it is not torn, or was not asked for).
MUON_HD void ask(Asked& a, uint32_t n, uint32_t stage, uint32_t stages, bool two, uint32_t gap) {
    uint32_t m = n < stages ? ((1u << n) - 1) << stage : ~0u;
    m |= m >> stages;
    a.two = two ? a.two | m : a.two & ~m;
    a.torn &= ~m;
    a.steps += n;
    if (gap) {
        const uint32_t last = (stage + n - 1) % stages;
        a.torn |= 1u << last;
        a.times ^= 1u << last;
        a.gaps = (a.gaps & ~(15u << 4 * last)) | gap << 4 * last;
    }
}

// Bytes that a step takes of a thread for A, for B, of a clearing warp.
MUON_HD uint32_t a_bytes() { return 2 * DRAIN_BOX; }
MUON_HD uint32_t b_bytes(bool two) { return two ? 2 * DRAIN_BOX : DRAIN_BOX; }
MUON_HD uint32_t zero_bytes(uint32_t gap, bool two) { return gap * 128 * (two ? 4 : 3); }

// The last step that any of n threads has asked for in a stage.  No other can
// be in flight: a stage is loaded again when its products have run.
struct Last {
    bool any, two;
    uint32_t step, gap, phase;           // the parity of its phase
};
MUON_HD Last last_of(const Asked* by, int n, uint32_t stage, uint32_t stages) {
    Last l{false, false, 0, 0, 0};
    for (int i = 0; i < n; ++i) {
        const Asked& a = by[i];
        if (a.steps <= stage) continue;
        const uint32_t before = (a.steps - 1 - stage) / stages, step = before * stages + stage;
        if (l.any && step <= l.step) continue;
        // of its stage's steps before, those of its kind
        const uint32_t torn = a.times >> stage & 1;
        if (a.torn >> stage & 1) l = {true, (a.two >> stage & 1) != 0, step, a.gaps >> 4 * stage & 15, torn ^ 1};
        else l = {true, (a.two >> stage & 1) != 0, step, 0, (before ^ torn) & 1};
    }
    return l;
}

// What makes a barrier's phase end when the last byte that was asked for is
// there: arm it with these bytes (nobody has), or take these off (they were
// never asked for), and wait for the parity.
struct Settle {
    uint32_t arm, cancel, parity;
    bool wait;
};
MUON_HD void add(Settle& s, bool asked, bool first, uint32_t bytes, bool& armed) {
    if (first) armed = asked;
    if (asked) {
        s.arm += bytes;
        s.wait = true;
    } else {
        s.cancel += bytes;
    }
}
MUON_HD Settle settled(Settle s, bool armed) {
    if (armed) s.arm = 0;
    else s.cancel = 0;
    return s;
}

// Of a stage's barriers: the leader's of whole steps (by: A and B of the
// leader, then of the other CTA), a CTA's of torn ones (its own A and B), and the
// leader's of the zeros (zeros: both CTAs').
MUON_HD Settle settle_full(const Asked* by, uint32_t stage, uint32_t stages) {
    const Last l = last_of(by, 4, stage, stages);
    Settle s{0, 0, l.phase, false};
    bool armed = false;
    if (l.any && !l.gap)
        for (int i = 0; i < 4; ++i) add(s, by[i].steps > l.step, i == 0, i & 1 ? b_bytes(l.two) : a_bytes(), armed);
    return settled(s, armed);
}
MUON_HD Settle settle_torn(const Asked* by, uint32_t stage, uint32_t stages) {
    const Last l = last_of(by, 2, stage, stages);
    Settle s{0, 0, l.phase, false};
    bool armed = false;
    if (l.any && l.gap)
        for (int i = 0; i < 2; ++i) add(s, by[i].steps > l.step, i == 0, i & 1 ? b_bytes(l.two) : a_bytes(), armed);
    return settled(s, armed);
}
MUON_HD Settle settle_zeros(const Asked* by, const Asked* zeros, uint32_t stage, uint32_t stages) {
    const Last l = last_of(by, 4, stage, stages);
    Settle s{0, 0, l.phase, false};
    bool armed = false;
    if (l.any && l.gap)
        for (int i = 0; i < 2; ++i) add(s, zeros[i].steps > l.step, i == 0, zero_bytes(l.gap, l.two), armed);
    return settled(s, armed);
}

}  // namespace ops
}  // namespace muon
