// Plays the weight gradient's loads, decoding and products through on the CPU
// with loads and warps of random speed, one barrier phase at a time, from the
// stage numbers and phases that the kernel itself uses.
//
//   weight_grad_stages <guard>     guard 0: without the wait for a stage's
//                                  last user (must be found out by the model)
//
// A barrier counts phases; a wait for a parity returns unless the phase now
// running has that parity.  Prints the number of runs in which a step read or
// overwrote what was another step's, or in which nothing could go on.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "weight_grad_stages.h"

using namespace muon::ops;

namespace {

constexpr int WARPS = 4;             // of a group
constexpr int STEPS = 64;

struct Bar {
    int count, pending;
    uint32_t phase = 0;
    explicit Bar(int n = 1) : count(n), pending(n) {}
    bool over(uint32_t parity) const { return (phase & 1) != parity; }
    // false: more arrivals than the phase takes
    void arrive() {
        if (--pending == 0) {
            ++phase;
            pending = count;
        }
    }
};

// One CTA's decoding of a matrix's steps, and the products that read it (the
// other CTA of the pair changes nothing in these waits).
template <bool WIDE>
bool plays(std::mt19937& rng, bool guard) {
    using S = Stages<WIDE>;
    std::vector<Bar> a(S::A), done(S::A), r(S::R), free_r(S::R, Bar(WARPS)), ready(S::B, Bar(WARPS));
    std::vector<int> has_a(S::A, -1), has_r(S::R, -1);
    std::vector<std::vector<int>> has_b(S::B, std::vector<int>(WARPS, -1));
    struct Load { int step; bool of_r; int left; };
    std::vector<Load> flying;
    uint32_t na = 0, nr = 0, products = 0;
    // a warp's step and what it does next
    struct Warp { uint32_t step; int at = 0; int busy = 0; };
    std::vector<Warp> warps;
    for (int g = 0; g < W_DEC_GROUPS; ++g)
        for (int w = 0; w < WARPS; ++w) warps.push_back({uint32_t(g)});
    // mostly quick loads; now and then one that is much slower than the rest
    auto latency = [&] { return int(rng() % 8 == 0 ? rng() % 400 : rng() % 10); };
    const int slow_group = rng() % 3;
    bool bad = false;
    int idle = 0;
    while (products < STEPS && !bad) {
        bool moved = false;
        // loads issued in order
        if (WIDE && nr < STEPS && nr <= na + S::AHEAD &&
            free_r[stage_of(nr, S::R)].over(parity_of(nr, S::R) ^ 1)) {
            flying.push_back({int(nr), true, latency()});
            ++nr;
            moved = true;
        } else if (na < STEPS && done[stage_of(na, S::A)].over(parity_of(na, S::A) ^ 1) &&
                   (!WIDE || nr > na)) {
            flying.push_back({int(na), false, latency()});
            ++na;
            moved = true;
        }
        // and landing in any
        for (size_t i = 0; i < flying.size();) {
            Load& l = flying[i];
            moved = true;
            if (l.left-- > 0) {
                ++i;
                continue;
            }
            if (l.of_r) {
                has_r[stage_of(l.step, S::R)] = l.step;
                r[stage_of(l.step, S::R)].arrive();
            } else {
                has_a[stage_of(l.step, S::A)] = l.step;
                if (!WIDE) has_r[stage_of(l.step, S::R)] = l.step;
                a[stage_of(l.step, S::A)].arrive();
            }
            flying.erase(flying.begin() + long(i));
        }
        for (size_t i = 0; i < warps.size(); ++i) {
            Warp& w = warps[i];
            if (w.step >= STEPS) continue;
            if (w.busy-- > 0) {
                moved = true;
                continue;
            }
            w.busy = rng() % (int(i) / WARPS == slow_group ? 30 : 3);
            const uint32_t step = w.step, sa = stage_of(step, S::A), sb = stage_of(step, S::B),
                           sr = stage_of(step, S::R);
            const int me = int(i) % WARPS;
            const Bar& in = WIDE ? r[sr] : a[sa];
            const uint32_t last = last_user<WIDE>(step);
            auto used = [&] {                             // the stage's last user
                return !guard || !stage_was_used<WIDE>(step) ||
                       done[stage_of(last, S::A)].over(parity_of(last, S::A));
            };
            auto there = [&] {                            // the 8-bit values
                return in.over(WIDE ? parity_of(step, S::R) : parity_of(step, S::A));
            };
            if (w.at == 0 && (WIDE ? there() : used())) w.at = 1;
            if (w.at == 1) {
                if (!(WIDE ? used() : there())) continue;
                bad |= has_r[sr] != int(step);
                // nothing that the products have not read may be written over
                bad |= has_b[sb][me] >= 0 && uint32_t(has_b[sb][me]) >= products;
                has_b[sb][me] = int(step);
                if (WIDE) free_r[sr].arrive();
                w.at = 2;
            }
            if (w.at == 0) continue;
            if (WIDE && !a[sa].over(parity_of(step, S::A))) continue;
            bad |= has_a[sa] != int(step);
            ready[sb].arrive();
            w.at = 0;
            w.step += W_DEC_GROUPS;
            moved = true;
        }
        // products in order
        if (ready[stage_of(products, S::B)].over(parity_of(products, S::B)) && rng() % 4 == 0) {
            bad |= has_a[stage_of(products, S::A)] != int(products);
            for (int w = 0; w < WARPS; ++w) bad |= has_b[stage_of(products, S::B)][w] != int(products);
            done[stage_of(products, S::A)].arrive();
            ++products;
            moved = true;
        }
        idle = moved ? 0 : idle + 1;
        if (idle > 1000) return false;
    }
    return !bad;
}

template <bool WIDE>
int failures(bool guard, int runs) {
    int n = 0;
    for (int i = 0; i < runs; ++i) {
        std::mt19937 rng(1000 + i);
        n += !plays<WIDE>(rng, guard);
    }
    return n;
}

}  // namespace

int main(int argc, char** argv) {
    const bool guard = argc < 2 || std::atoi(argv[1]) != 0;
    std::printf("%d %d\n", failures<false>(guard, 2000), failures<true>(guard, 2000));
    return 0;
}
