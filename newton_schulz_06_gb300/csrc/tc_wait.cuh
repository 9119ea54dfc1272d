// A bounded wait for phases that are expected within microseconds.
#pragma once

#include "tc_ptx.cuh"

namespace muon {
namespace ops {

// As ptx::wait_bounded, which reads the clock before it looks again: some
// hundred nanoseconds that a phase about to complete should not cost.  Looks
// a few hundred times first.
__device__ __forceinline__ bool wait_soon(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int* err, uint64_t limit_ns) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (ptx::mbar_try_wait(bar, parity)) return true;
    return ptx::wait_bounded(bar, parity, abort_flag, err, limit_ns);
}

}  // namespace ops
}  // namespace muon
