// Plays the loads of a CTA pair of the gated feed-forward kernels through on
// the CPU, with threads of random speed that are stopped at any moment, and
// then what the pair does about its loads in flight (ffn_drain.h).
//
//   ffn_drain <rule>     rule 0: each CTA's first thread waits for the stages
//                        that it has loaded itself (must be found out by the
//                        model); 1: the kernel's
//
// Prints the number of runs in which the pair left with a load in flight, and
// of those in which a wait would not have ended.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "ffn_drain.h"

using namespace muon::ops;

namespace {

// One arrival a phase, and bytes.
struct Bar {
    int pending = 1;
    int64_t bytes = 0;
    uint32_t phase = 0;
    bool over(uint32_t parity) const { return (phase & 1) != parity; }
    void turn() {
        if (pending == 0 && bytes == 0) {
            ++phase;
            pending = 1;
        }
    }
    void arm(int64_t n) {
        bytes += n;
        --pending;
        turn();
    }
    void land(int64_t n) {
        bytes -= n;
        turn();
    }
};

constexpr int STEPS = 60;

struct Step {
    uint32_t gap;
    bool two, ends;          // its tile
};
struct Load {
    Bar* bar;
    int64_t bytes;
};

// bit 0: left with a load in flight; bit 1: a wait that would not end
int plays(std::mt19937& rng, int rule) {
    const uint32_t stages = 5 + rng() % 2;
    std::vector<Step> steps(STEPS);
    for (int i = 0; i < STEPS;) {
        // tiles of one width, of which the last step may be torn
        const int n = 1 + int(rng() % (rng() % 3 ? 4 : 20));
        const bool two = rng() % 3 != 0;
        for (int k = 0; k < n && i < STEPS; ++k, ++i) {
            const bool ends = k == n - 1 || i == STEPS - 1;
            steps[i] = {ends && rng() % 2 ? uint32_t(rng() % 16) : 0u, two, ends};
        }
    }
    std::vector<Bar> full(stages), zero(stages), torn[2];
    torn[0].resize(stages);
    torn[1].resize(stages);
    std::vector<Load> flying;
    Asked by[4] = {}, zeros[2] = {};     // A and B of the leader, of the other CTA
    uint32_t done[4] = {};               // steps of the tile that a thread is in
    uint32_t products = 0;
    const uint32_t moves = rng() % 700, lazy = rng() % 7;
    // (the parity of a step's phase goes by the steps of its kind that its stage had)
    auto parity = [&](uint32_t step) {
        uint32_t n = 0;
        for (uint32_t i = step % stages; i < step; i += stages) n += !steps[i].gap == !steps[step].gap;
        return n & 1;
    };
    auto parts = [&](Bar& bar, int64_t bytes) {
        while (bytes) {
            const int64_t n = bytes < 2048 ? bytes : 1 + int64_t(rng() % bytes);
            flying.push_back({&bar, n});
            bytes -= n;
        }
    };
    for (uint32_t m = 0; m < moves; ++m) {
        const uint32_t what = rng() % 10;
        if (what == lazy && rng() % 8) continue;
        if (what < 4) {
            Asked& me = by[what];
            const uint32_t i = me.steps + done[what], stage = i % stages, rank = what / 2;
            if (i >= STEPS || (i >= stages && products < i - stages + 1)) continue;
            const Step& s = steps[i];
            Bar& bar = s.gap ? torn[rank][stage] : full[stage];
            const int64_t cta = a_bytes() + b_bytes(s.two);
            if (s.gap && what % 2 == 0) bar.arm(cta);
            if (!s.gap && what == 0) bar.arm(2 * cta);
            parts(bar, what % 2 ? b_bytes(s.two) : a_bytes());
            ++done[what];
            if (s.ends) {
                ask(me, done[what], me.steps % stages, stages, s.two, s.gap);
                done[what] = 0;
            }
        } else if (what < 6) {
            const uint32_t rank = what - 4, i = zeros[rank].steps, stage = i % stages;
            if (i >= STEPS) continue;
            const Step& s = steps[i];
            // (the warp goes from torn step to torn step)
            if (s.gap) {
                const uint32_t a = 2 * rank, b = a + 1;
                if (by[a].steps + done[a] <= i || by[b].steps + done[b] <= i || !torn[rank][stage].over(parity(i)))
                    continue;
                if (rank == 0) zero[stage].arm(2 * int64_t(zero_bytes(s.gap, s.two)));
                parts(zero[stage], zero_bytes(s.gap, s.two));
            }
            ++zeros[rank].steps;
        } else if (what < 9) {
            if (flying.empty() || rng() % 3 == 0) continue;
            const size_t at = rng() % flying.size();
            flying[at].bar->land(flying[at].bytes);
            flying.erase(flying.begin() + long(at));
        } else if (products < STEPS) {
            const uint32_t stage = products % stages;
            if ((steps[products].gap ? zero : full)[stage].over(parity(products))) ++products;
        }
    }
    // The pair gives up here, some threads within a tile.
    for (int k = 0; k < 4; ++k)
        if (done[k]) ask(by[k], done[k], by[k].steps % stages, stages, steps[by[k].steps].two, 0);
    struct Wait {
        Bar* bar;
        uint32_t parity;
    };
    std::vector<Wait> waits;
    for (uint32_t s = 0; s < stages; ++s) {
        if (rule == 0) {
            for (int rank = 0; rank < 2; ++rank) {
                const Asked& a = by[2 * rank];
                const Last l = last_of(&a, 1, s, stages);
                if (!l.any) continue;
                if (l.gap) waits.push_back({&torn[rank][s], l.phase});
                else if (rank == 0) waits.push_back({&full[s], l.phase});
            }
            continue;
        }
        auto apply = [&](Bar& bar, const Settle& x) {
            if (!x.wait) return;
            if (x.arm) bar.arm(x.arm);
            if (x.cancel) bar.land(x.cancel);
            waits.push_back({&bar, x.parity});
        };
        for (int rank = 0; rank < 2; ++rank) apply(torn[rank][s], settle_torn(by + 2 * rank, s, stages));
        apply(full[s], settle_full(by, s, stages));
        apply(zero[s], settle_zeros(by, zeros, s, stages));
    }
    // The loads land in any order: when the last wait has ended, all have.
    while (true) {
        bool all = true;
        for (const Wait& w : waits) all &= w.bar->over(w.parity);
        if (all) return flying.empty() ? 0 : 1;
        if (flying.empty()) return 2;
        const size_t at = rng() % flying.size();
        flying[at].bar->land(flying[at].bytes);
        flying.erase(flying.begin() + long(at));
    }
}

}  // namespace

int main(int argc, char** argv) {
    const int rule = argc < 2 ? 1 : std::atoi(argv[1]);
    int left = 0, stuck = 0;
    for (int i = 0; i < 200000; ++i) {
        std::mt19937 rng(1000 + i);
        const int r = plays(rng, rule);
        left += r & 1;
        stuck += r >> 1;
    }
    std::printf("%d %d\n", left, stuck);
    return 0;
}
