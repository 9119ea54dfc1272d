// Rotary positions (muon_rotary): the pairs of a head's values turn by an angle
// that grows with the position,
//     y1 = m (x1 cos - x2 sin),  y2 = m (x2 cos + x1 sin),
// queries and keys in one launch; the gradient is the same with -sin.
//
// Angles.  A pair's frequency is a 64-bit fraction of a turn per position, so
// that position * frequency modulo 2^64 is the angle with whole turns already
// gone, and the product is not rounded (in fp32 it is off by 0.06 radians at
// position 10^6).  What is left is the frequency's own error, made in 64-bit
// floating point: 2^-50 of the whole angle at most, 2e-6 radians at position
// 2^31.  No table of cosines is read: a block makes them for its tokens once, in
// shared memory, and all heads use them.
//
// What bounds it is memory: each value is read and written once (16384 tokens
// of 36 heads of 128 in bf16: 49 us, 6.1 TB/s; 8191 of 65 heads, of which 64 of 192
// values turn: 71 us, 5.8 TB/s; heads off 16 bytes take two to three times as long).
#include "ops_internal.h"

namespace muon {
namespace ops {
namespace {

constexpr int R_THREADS = 256;
constexpr int R_PAIRS = 1024;             // cosines and sines of a block (or one token's)

// u / d for u below 2^31 as a multiplication and a shift ("Division by invariant
// integers using multiplication", Granlund and Montgomery, 1994).
struct Quotient {
    uint32_t d, m, shift;
    void set(int64_t v) {
        d = static_cast<uint32_t>(v);
        int log = 0;
        while ((int64_t(1) << log) < v) ++log;
        m = log ? static_cast<uint32_t>((uint64_t(1) << (31 + log)) / d + 1) : 0;
        shift = log ? log - 1 : 0;
    }
    __device__ __forceinline__ uint32_t of(uint32_t u) const { return d == 1 ? u : __umulhi(u, m) >> shift; }
};

struct RotaryLaunch {
    muon_rotary_tensor t[2];
    const void* positions;
    int64_t stride_pos;
    int64_t offset;
    uint32_t tokens, tokens_block;        // tokens: batch * seq
    uint32_t head;
    Quotient seq, pairs;                  // pairs of a head that turn
    Quotient per_head, per_token;         // units of a head (those that turn, then the rest), of a token
    uint32_t turning, rest;               // how many of each
    int32_t wide_pos;                     // positions are 64-bit
    float scale, sign;
    uint64_t turns[256];
};

// a c + b s, rounded the same way in all kernels.
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
    return __fmaf_rn(a, c, __fmul_rn(b, s));
}

// HALF: pair i is values i and i + pairs of a head; else 2 i and 2 i + 1.  A
// thread's unit is 16 bytes of values, with HALF of both of their halves; of
// a head's rest with HALF as much, from its two halves.  AL: all of these lie on
// 16 bytes; else they are put together from aligned pieces, and across lanes.
template <typename T, bool HALF, bool AL>
__global__ void __launch_bounds__(R_THREADS) rotary_kernel(const __grid_constant__ RotaryLaunch p) {
    extern __shared__ float trig[];       // cosines, then sines, of tokens_block x pairs
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t first = blockIdx.x * p.tokens_block;
    const uint32_t tokens = min(p.tokens_block, p.tokens - first);
    float* const sine = trig + p.tokens_block * p.pairs.d;
    for (uint32_t u = threadIdx.x; u < tokens * p.pairs.d; u += R_THREADS) {
        const uint32_t t = p.pairs.of(u), i = u - t * p.pairs.d;
        const uint32_t b = p.seq.of(first + t), s = first + t - b * p.seq.d;
        int64_t at = s;
        if (p.positions) {
            const int64_t k = int64_t(b) * p.stride_pos + s;
            at = p.wide_pos ? static_cast<const int64_t*>(p.positions)[k]
                            : static_cast<const int32_t*>(p.positions)[k];
        }
        const uint64_t angle = (static_cast<uint64_t>(at) + static_cast<uint64_t>(p.offset)) * p.turns[i];
        // half turns in -1 .. 1
        float c, n;
        sincospif(__ll2float_rn(static_cast<int64_t>(angle)) * 1.0842021724855044e-19f, &n, &c);
        trig[u] = c * p.scale;
        sine[u] = n * p.scale * p.sign;
    }
    __syncthreads();
    const uint32_t q_heads = static_cast<uint32_t>(p.t[0].heads);
    constexpr uint32_t VE = 16 / sizeof(T);
    const uint32_t total = tokens * p.per_token.d;
    // (whole warps: they exchange what lies off 16 bytes)
    for (uint32_t u = threadIdx.x; u - threadIdx.x % 32 < total; u += R_THREADS) {
        const bool live = u < total;
        const uint32_t t = live ? p.per_token.of(u) : 0, in = live ? u - t * p.per_token.d : 0;
        uint32_t h = p.per_head.of(in);
        const uint32_t unit = in - h * p.per_head.d;
        const uint32_t b = p.seq.of(first + t), s = first + t - b * p.seq.d;
        const int which = h >= q_heads;
        if (which) h -= q_heads;
        const muon_rotary_tensor& x = p.t[which];
        const bool turns = unit < p.turning;
        // Where this unit's values are, and how many are left there: those that
        // turn and those that do not are loaded and stored by the same
        // instructions (a branch each took 8191 tokens of 65 heads, 64 of 192
        // values, from 72 to 86 us).
        const uint32_t k = turns ? unit : unit - p.turning;
        const uint32_t from1 = turns ? 0 : 2 * p.pairs.d, from2 = turns ? p.pairs.d : from1 + VE * p.rest;
        const uint32_t to1 = turns ? (HALF ? 1 : 2) * p.pairs.d : HALF ? min(p.head, from2) : p.head;
        const uint32_t to2 = turns ? 2 * p.pairs.d : p.head;
        const int left1 = live ? int(to1) - int(from1 + VE * k) : 0;
        const int left2 = live && HALF ? int(to2) - int(from2 + VE * k) : 0;
        const T* const from = static_cast<const T*>(x.x) + (b * x.x_batch + s * x.x_seq + h * x.x_head + VE * k);
        T* const to = static_cast<T*>(x.y) + (b * x.y_batch + s * x.y_seq + h * x.y_head + VE * k);
        Vec<T, AL> v, w;
        v.load(from + from1, left1);
        if (HALF) w.load(from + from2, left2);
        if (turns) {
            float2 f[VE / 2], g[VE / 2];
            v.get(f);
            if constexpr (HALF) {
                const float* const c = trig + t * p.pairs.d + VE * k;
                const float* const n = sine + t * p.pairs.d + VE * k;
                w.get(g);
#pragma unroll
                for (uint32_t i = 0; i < VE / 2; ++i) {
                    const float2 a = f[i], d = g[i];
                    f[i] = make_float2(turned(a.x, c[2 * i], d.x, -n[2 * i]),
                                       turned(a.y, c[2 * i + 1], d.y, -n[2 * i + 1]));
                    g[i] = make_float2(turned(d.x, c[2 * i], a.x, n[2 * i]),
                                       turned(d.y, c[2 * i + 1], a.y, n[2 * i + 1]));
                }
                w.set(g);
            } else {
                const float* const c = trig + t * p.pairs.d + VE / 2 * k;
                const float* const n = sine + t * p.pairs.d + VE / 2 * k;
#pragma unroll
                for (uint32_t i = 0; i < VE / 2; ++i)
                    f[i] = make_float2(turned(f[i].x, c[i], f[i].y, -n[i]), turned(f[i].y, c[i], f[i].x, n[i]));
            }
            v.set(f);
        }
        v.store(to + from1, left1, k == 0);
        if (HALF) w.store(to + from2, left2, k == 0);
    }
}

// Whether all rows, halves and rests begin and end on 16 bytes.
template <typename T>
bool on_16(const muon_rotary_args& a, bool copy) {
    constexpr int64_t VE = 16 / sizeof(T);
    bool ok = (a.layout == MUON_ROTARY_HALF ? a.pairs : 2 * a.pairs) % VE == 0 && (!copy || a.head % VE == 0);
    const muon_rotary_tensor* const tensors[2] = {&a.q, &a.k};
    for (const muon_rotary_tensor* t : tensors) {
        if (!t->heads) continue;
        ok = ok && reinterpret_cast<uintptr_t>(t->x) % 16 == 0 && reinterpret_cast<uintptr_t>(t->y) % 16 == 0 &&
             (a.batch <= 1 || (t->x_batch % VE == 0 && t->y_batch % VE == 0)) &&
             (a.seq <= 1 || (t->x_seq % VE == 0 && t->y_seq % VE == 0)) &&
             (t->heads <= 1 || (t->x_head % VE == 0 && t->y_head % VE == 0));
    }
    return ok;
}

template <typename T>
cudaError_t launch(RotaryLaunch p, const muon_rotary_args& a, cudaStream_t s) {
    constexpr int64_t VE = 16 / sizeof(T);
    const bool half = a.layout == MUON_ROTARY_HALF;
    const bool rest = a.head > 2 * a.pairs;
    const bool copy = rest && ((a.q.heads && a.q.x != a.q.y) || (a.k.heads && a.k.x != a.k.y));
    p.turning = static_cast<uint32_t>(ceil_div((half ? 1 : 2) * a.pairs, VE));
    p.rest = copy ? static_cast<uint32_t>(ceil_div(a.head - 2 * a.pairs, half ? 2 * VE : VE)) : 0;
    const int64_t per_head = p.turning + p.rest;
    // as many tokens a block as give every thread four units, and no more than
    // leave every SM a block (with eight tokens of 65 heads of 192 a block, so
    // that every thread made a cosine, 8191 tokens took 108 us)
    const int64_t units = (a.q.heads + a.k.heads) * per_head;
    p.per_head.set(per_head);
    p.per_token.set(units);
    int64_t t = ceil_div(4 * R_THREADS, units);
    if (t > R_PAIRS / a.pairs) t = R_PAIRS / a.pairs;
    if (t > ceil_div(p.tokens, 152)) t = ceil_div(p.tokens, 152);
    // (the units of a block are counted in 32 bits)
    if (t > (int64_t(1) << 28) / units) t = (int64_t(1) << 28) / units;
    p.tokens_block = static_cast<uint32_t>(t < 1 ? 1 : t);
    void (*const kernel)(RotaryLaunch) =
        on_16<T>(a, copy) ? (half ? rotary_kernel<T, true, true> : rotary_kernel<T, false, true>)
                          : (half ? rotary_kernel<T, true, false> : rotary_kernel<T, false, false>);
    // (a short last unit reads up to seven cosines and sines too many)
    return launch_kernel(kernel, dim3(static_cast<unsigned>(ceil_div(p.tokens, p.tokens_block))), dim3(R_THREADS),
                         (size_t(2) * p.tokens_block * p.pairs.d + 8) * sizeof(float), s, p);
}

}  // namespace

cudaError_t launch_rotary(const muon_rotary_args& a, cudaStream_t s) {
    RotaryLaunch p = {};
    p.t[0] = a.q;
    p.t[1] = a.k;
    p.positions = a.positions;
    p.wide_pos = a.positions_64;
    p.stride_pos = a.stride_positions;
    p.offset = a.offset;
    p.tokens = static_cast<uint32_t>(a.batch * a.seq);
    p.head = static_cast<uint32_t>(a.head);
    p.seq.set(a.seq);
    p.pairs.set(a.pairs);
    p.scale = a.scale;
    p.sign = a.inverse ? -1.f : 1.f;
    for (int64_t i = 0; i < a.pairs; ++i) p.turns[i] = a.turns[i];
    return a.x_dtype == MUON_F32 ? launch<float>(p, a, s) : launch<__nv_bfloat16>(p, a, s);
}

}  // namespace ops
}  // namespace muon
