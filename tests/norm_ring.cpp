// Plays the layer norm's ring of rows through on the CPU: a block whose wait
// runs out at any row asks for nothing more, and waits for exactly the copies
// that it has asked for and not waited for.  Prints the number of cases that
// go wrong.
#include <cstdio>
#include <vector>

#include "norm_ring.h"

using namespace muon::ops;

int main() {
    int bad = 0;
    for (int stages = 1; stages <= 8; ++stages)
        for (int stride : {1, 3, 7})
            for (int rows = 1; rows <= 60; ++rows)
                for (int first = 0; first < stride && first < rows; ++first)
                    for (int abort_at = first; abort_at < rows; abort_at += stride) {
                        // phases[s]: copies asked for in stage s; waited[s]: waited for
                        std::vector<int> asked(stages, 0), waited(stages, 0);
                        for (int s = 0; s < stages; ++s) asked[s] += first + s * stride < rows;
                        RingAt at{0, 0};
                        int row = first;
                        bool ok = true;
                        for (; row < rows; row += stride) {
                            // the phase waited for is the one that the last copy lands in
                            ok &= (uint32_t(asked[at.stage] - 1) & 1) == at.phase;
                            if (row == abort_at) break;
                            ++waited[at.stage];
                            ok &= asked[at.stage] == waited[at.stage];
                            asked[at.stage] += row + stages * stride < rows;
                            at = ring_ahead(at, stages, 1);
                        }
                        for (int d = 0; ring_in_flight(rows, row, stride, stages, d); ++d) {
                            const RingAt l = ring_ahead(at, stages, d);
                            ok &= (uint32_t(waited[l.stage]) & 1) == l.phase;
                            ++waited[l.stage];
                        }
                        for (int s = 0; s < stages; ++s) ok &= asked[s] == waited[s];
                        bad += !ok;
                    }
    std::printf("%d\n", bad);
    return 0;
}
