// Rotary positions (muon_rotary): the pairs of a head's values turn by an angle
// that grows with the position,
//     y1 = m (x1 cos - x2 sin),  y2 = m (x2 cos + x1 sin),
// queries and keys in one launch; the gradient is the same with -sin.
//
// Angles.  A pair's frequency is a 64-bit fraction of a turn per position, so
// that position * frequency modulo 2^64 is the angle with whole turns already
// gone: exact for every position, where the product in fp32 is off by 0.06
// radians at a million.  No table of cosines is read: a block makes them for
// its tokens once, in shared memory, and all heads use them.
//
// What bounds it is memory: each value is read and written once.
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
    Quotient per_head, per_token;         // units of a head (groups of W pairs, then of W other values), of a token
    int32_t wide_pos, copy;               // positions are 64-bit; the other values are copied
    float scale, sign;
    uint64_t turns[256];
};

// N neighbouring values as they are in memory, W of them an access.
template <typename T, int W, int N>
struct Group {
    struct alignas(sizeof(T) * W) Raw {
        T v[W];
    };
    Raw raw[N / W];
    __device__ __forceinline__ void load(const T* p, int accesses) {
#pragma unroll
        for (int k = 0; k < N / W; ++k)
            if (k < accesses) raw[k] = reinterpret_cast<const Raw*>(p)[k];
    }
    __device__ __forceinline__ void store(T* p, int accesses) const {
#pragma unroll
        for (int k = 0; k < N / W; ++k)
            if (k < accesses) reinterpret_cast<Raw*>(p)[k] = raw[k];
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(raw[i / W].v[i % W]); }
    __device__ __forceinline__ void set(int i, float f) { from_f32(&raw[i / W].v[i % W], f); }
};

// a c + b s, rounded the same way in all kernels.
__device__ __forceinline__ float turned(float a, float c, float b, float s) {
    return __fmaf_rn(a, c, __fmul_rn(b, s));
}

// HALF: pair i is values i and i + pairs of a head; else 2 i and 2 i + 1.
// W: values of a load or store.  A unit of a thread's work is W pairs of HALF,
// or W values (two at least).
template <typename T, int W, bool HALF>
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
        const uint64_t angle = static_cast<uint64_t>(at + p.offset) * p.turns[i];
        // half turns in -1 .. 1
        float c, n;
        sincospif(__ll2float_rn(static_cast<int64_t>(angle)) * 1.0842021724855044e-19f, &n, &c);
        trig[u] = c * p.scale;
        sine[u] = n * p.scale * p.sign;
    }
    __syncthreads();
    const uint32_t q_heads = static_cast<uint32_t>(p.t[0].heads);
    constexpr int N = HALF || W > 1 ? W : 2;              // values of an operand
    constexpr uint32_t PW = HALF ? N : N / 2;             // pairs of a unit
    const uint32_t turning = p.pairs.d / PW;              // units that turn
    for (uint32_t u = threadIdx.x; u < tokens * p.per_token.d; u += R_THREADS) {
        const uint32_t t = p.per_token.of(u), in = u - t * p.per_token.d;
        uint32_t h = p.per_head.of(in);
        const uint32_t unit = in - h * p.per_head.d;
        const uint32_t b = p.seq.of(first + t), s = first + t - b * p.seq.d;
        const int which = h >= q_heads;
        if (which) h -= q_heads;
        const muon_rotary_tensor& x = p.t[which];
        const bool turns = unit < turning;
        // where this unit's values are: those that turn and those that do not
        // are loaded and stored by the same instructions (a branch each took
        // 8191 tokens of 65 heads, 64 of 192 values, from 72 to 86 us)
        const uint32_t rest = 2 * p.pairs.d + (unit - turning) * (HALF ? 2 * W : N);
        const uint32_t at = turns ? unit * N : rest, at2 = turns ? p.pairs.d + unit * N : rest + W;
        const bool second = HALF && (turns || at2 < p.head);
        const int64_t in_x = b * x.x_batch + s * x.x_seq + h * x.x_head;
        const int64_t in_y = b * x.y_batch + s * x.y_seq + h * x.y_head;
        const T* const from = static_cast<const T*>(x.x) + in_x;
        T* const to = static_cast<T*>(x.y) + in_y;
        // (one value at a time, the last of an odd rest is alone)
        const int accesses = N > W && at + 1 == p.head ? 1 : N / W;
        Group<T, W, N> v, w;
        v.load(from + at, accesses);
        if (second) w.load(from + at2, 1);
        if (turns) {
            const float* const c = trig + t * p.pairs.d + unit * PW;
            const float* const n = sine + t * p.pairs.d + unit * PW;
            if constexpr (HALF) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float f = v.get(i), g = w.get(i);
                    v.set(i, turned(f, c[i], g, -n[i]));
                    w.set(i, turned(g, c[i], f, n[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float f = v.get(i), g = v.get(i + 1);
                    v.set(i, turned(f, c[i / 2], g, -n[i / 2]));
                    v.set(i + 1, turned(g, c[i / 2], f, n[i / 2]));
                }
            }
        }
        v.store(to + at, accesses);
        if (second) w.store(to + at2, 1);
    }
}

// The widest group, of up to 16 bytes, in which all rows, halves and rests
// begin and end.
template <typename T>
int group_width(const muon_rotary_args& a, bool copy) {
    int w = 16 / sizeof(T);
    auto fits = [&](int64_t elements) {
        while (w > 1 && elements % w) w >>= 1;
    };
    fits(a.layout == MUON_ROTARY_HALF ? a.pairs : 2 * a.pairs);
    if (copy) fits(a.head);
    const muon_rotary_tensor* const t[2] = {&a.q, &a.k};
    for (int i = 0; i < 2; ++i) {
        if (!t[i]->heads) continue;
        const void* const ptr[2] = {t[i]->x, t[i]->y};
        for (const void* q : ptr)
            while (w > 1 && reinterpret_cast<uintptr_t>(q) % (w * sizeof(T))) w >>= 1;
        if (a.batch > 1) fits(t[i]->x_batch), fits(t[i]->y_batch);
        if (a.seq > 1) fits(t[i]->x_seq), fits(t[i]->y_seq);
        if (t[i]->heads > 1) fits(t[i]->x_head), fits(t[i]->y_head);
    }
    return w;
}

template <typename T, int W>
cudaError_t launch(const RotaryLaunch& p, bool half, cudaStream_t s) {
    const int64_t blocks = ceil_div(p.tokens, p.tokens_block);
    void (*const kernel)(RotaryLaunch) = half ? rotary_kernel<T, W, true> : rotary_kernel<T, W, false>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(R_THREADS),
                         size_t(2) * p.tokens_block * p.pairs.d * sizeof(float), s, p);
}

template <typename T>
cudaError_t launch(RotaryLaunch p, const muon_rotary_args& a, cudaStream_t s) {
    const bool half = a.layout == MUON_ROTARY_HALF;
    const int w = group_width<T>(a, p.copy);
    const int64_t turning = half ? a.pairs / w : a.pairs / (w > 1 ? w / 2 : 1);
    // a unit of the rest is as many values as one of those that turn
    const int64_t values = half ? 2 * w : w > 1 ? w : 2;
    const int64_t per_head = turning + (p.copy ? ceil_div(a.head - 2 * a.pairs, values) : 0);
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
    if constexpr (sizeof(T) == 2)
        if (w == 8) return launch<T, 8>(p, half, s);
    if (w == 4) return launch<T, 4>(p, half, s);
    if (w == 2) return launch<T, 2>(p, half, s);
    return launch<T, 1>(p, half, s);
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
    const bool rest = a.head > 2 * a.pairs;
    p.copy = rest && ((a.q.heads && a.q.x != a.q.y) || (a.k.heads && a.k.x != a.k.y));
    for (int64_t i = 0; i < a.pairs; ++i) p.turns[i] = a.turns[i];
    return a.x_dtype == MUON_F32 ? launch<float>(p, a, s) : launch<__nv_bfloat16>(p, a, s);
}

}  // namespace ops
}  // namespace muon
