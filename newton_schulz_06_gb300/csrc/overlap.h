// Whether two tensors share memory, from their addresses, sizes and strides:
// host code, which tests/overlap.cpp holds against the sets of their bytes.
#pragma once

#include <cstdint>

namespace muon {
namespace ops {

// Up to three axes of runs of neighbouring bytes.
struct Area {
    __int128 p;
    int64_t run;
    int64_t n[3], stride[3];      // bytes; axes of one place, or of stride 0, are left out
    int axes;
    Area(const void* at, int64_t bytes) : p(reinterpret_cast<uintptr_t>(at)), run(bytes), axes(0) {}
    Area& axis(int64_t count, int64_t bytes) {
        if (count > 1 && bytes != 0) {
            n[axes] = count;
            stride[axes++] = bytes;
        }
        return *this;
    }
    // From the first byte to behind the last one, without the axes whose
    // strides are multiples of `period` (0: with all).
    __int128 span(int64_t period = 0) const {
        __int128 s = run;
        for (int i = 0; i < axes; ++i)
            if (!period || stride[i] % period) s += __int128(n[i] - 1) * stride[i];
        return s;
    }
    Area within(int64_t period) const {
        Area a(nullptr, run);
        a.p = p;
        for (int i = 0; i < axes; ++i)
            if (stride[i] % period) a.axis(n[i], stride[i]);
        return a;
    }
    // Whether places of two indexes may share memory: not where every axis
    // steps over all that the shorter axes hold.
    bool folded() const {
        for (int i = 0; i < axes; ++i) {
            __int128 inner = run;
            for (int j = 0; j < axes; ++j) {
                if (j != i && stride[j] == stride[i]) return true;
                if (stride[j] < stride[i]) inner += __int128(n[j] - 1) * stride[j];
            }
            if (stride[i] < inner) return true;
        }
        return false;
    }
};

// False only where they share nothing.  Tensors that interleave are told apart
// by strides that they have in common (columns of one matrix, matrices of one
// buffer, heads of one row); true, too, for some that interleave otherwise.
inline bool share(const Area& a, const Area& b) {
    if (a.p + a.span() <= b.p || b.p + b.span() <= a.p) return false;
    for (int i = 0; i < a.axes + b.axes; ++i) {
        const int64_t period = i < a.axes ? a.stride[i] : b.stride[i - a.axes];
        if (a.span(period) > period || b.span(period) > period) continue;
        // Without the axes of whole periods b begins `off` behind one of a's
        // places, and so much before the next: those there are of both.
        const int64_t d = static_cast<int64_t>(b.p - a.p);
        const int64_t whole = d / period - (d % period < 0), off = d - whole * period;
        const __int128 last = (a.span() - a.span(period)) / period, first = (b.span(period) - b.span()) / period;
        const Area x = a.within(period);
        Area y = b.within(period), z = y;
        y.p = x.p + off;
        z.p = y.p - period;
        const bool here = first <= whole && whole <= last && share(x, y);
        if (!here && !(first <= whole + 1 && whole + 1 <= last && share(x, z))) return false;
    }
    return true;
}

}  // namespace ops
}  // namespace muon
