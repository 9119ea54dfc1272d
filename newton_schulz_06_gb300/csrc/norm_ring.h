// Where a block of the layer norm's ring kernels is in its ring of rows: plain
// C++, so that tests/norm_ring.cpp plays aborts through on the CPU.
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

// A stage and the parity of the phase in which its row's copy lands.
struct RingAt {
    int stage;
    uint32_t phase;
};

// Those of the row d places on (0 <= d <= stages).
MUON_HD RingAt ring_ahead(RingAt at, int stages, int d) {
    at.stage += d;
    if (at.stage >= stages) {
        at.stage -= stages;
        at.phase ^= 1;
    }
    return at;
}

// Whether the copy of the row d places after `row` has been asked for and not
// been waited for, in a block that is at `row` and has not yet asked for what
// follows in that row's stage.
MUON_HD bool ring_in_flight(int64_t rows, int64_t row, int64_t stride, int stages, int d) {
    return d < stages && row + d * stride < rows;
}

}  // namespace ops
}  // namespace muon
