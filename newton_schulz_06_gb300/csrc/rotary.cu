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

struct RotaryLaunch {
    muon_rotary_tensor t[2];
    const void* positions;
    int64_t stride_pos;
    int64_t offset;
    uint32_t tokens, seq;                 // tokens: batch * seq
    uint32_t tokens_block;
    uint32_t head, pairs;                 // a head's values, and its pairs that turn
    uint32_t units;                       // of a head: groups of W pairs, then of W other values
    int32_t wide_pos, copy;               // positions are 64-bit; the other values are copied
    float scale, sign;
    uint64_t turns[256];
};

// N neighbouring values, W of them an access.
template <typename T, int W, int N>
struct Group {
    struct alignas(sizeof(T) * W) Raw {
        T v[W];
    };
    static __device__ __forceinline__ void load(const T* p, float (&f)[N]) {
#pragma unroll
        for (int k = 0; k < N / W; ++k) {
            const Raw r = reinterpret_cast<const Raw*>(p)[k];
#pragma unroll
            for (int i = 0; i < W; ++i) f[k * W + i] = to_f32(r.v[i]);
        }
    }
    static __device__ __forceinline__ void store(T* p, const float (&f)[N]) {
#pragma unroll
        for (int k = 0; k < N / W; ++k) {
            Raw r;
#pragma unroll
            for (int i = 0; i < W; ++i) from_f32(&r.v[i], f[k * W + i]);
            reinterpret_cast<Raw*>(p)[k] = r;
        }
    }
};

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
    float* const sine = trig + p.tokens_block * p.pairs;
    for (uint32_t u = threadIdx.x; u < tokens * p.pairs; u += R_THREADS) {
        const uint32_t t = u / p.pairs, i = u - t * p.pairs;
        const uint32_t b = (first + t) / p.seq, s = first + t - b * p.seq;
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
    const uint32_t heads = static_cast<uint32_t>(p.t[0].heads + p.t[1].heads);
    const uint32_t per_token = heads * p.units;
    constexpr int N = HALF || W > 1 ? W : 2;              // values of an operand
    constexpr uint32_t PW = HALF ? N : N / 2;             // pairs of a unit
    const uint32_t turning = p.pairs / PW;                // units that turn
    for (uint32_t u = threadIdx.x; u < tokens * per_token; u += R_THREADS) {
        const uint32_t t = u / per_token, in = u - t * per_token;
        uint32_t h = in / p.units;
        const uint32_t unit = in - h * p.units;
        const int which = h >= p.t[0].heads;
        if (which) h -= static_cast<uint32_t>(p.t[0].heads);
        const muon_rotary_tensor& x = p.t[which];
        const uint32_t b = (first + t) / p.seq, s = first + t - b * p.seq;
        const T* const from = static_cast<const T*>(x.x) + b * x.x_batch + s * x.x_seq + h * x.x_head;
        T* const to = static_cast<T*>(x.y) + b * x.y_batch + s * x.y_seq + h * x.y_head;
        if (unit >= turning) {
            const uint32_t at = 2 * p.pairs + (unit - turning) * W;
            float f[W];
            Group<T, W, W>::load(from + at, f);
            Group<T, W, W>::store(to + at, f);
            continue;
        }
        const float* const c = trig + t * p.pairs + unit * PW;
        const float* const n = sine + t * p.pairs + unit * PW;
        if constexpr (HALF) {
            float a[N], d[N], y[N], z[N];
            Group<T, W, N>::load(from + unit * N, a);
            Group<T, W, N>::load(from + p.pairs + unit * N, d);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                y[i] = a[i] * c[i] - d[i] * n[i];
                z[i] = d[i] * c[i] + a[i] * n[i];
            }
            Group<T, W, N>::store(to + unit * N, y);
            Group<T, W, N>::store(to + p.pairs + unit * N, z);
        } else {
            float a[N], y[N];
            Group<T, W, N>::load(from + unit * N, a);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                y[i] = a[i] * c[i / 2] - a[i + 1] * n[i / 2];
                y[i + 1] = a[i + 1] * c[i / 2] + a[i] * n[i / 2];
            }
            Group<T, W, N>::store(to + unit * N, y);
        }
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
                         size_t(2) * p.tokens_block * p.pairs * sizeof(float), s, p);
}

template <typename T>
cudaError_t launch(RotaryLaunch p, const muon_rotary_args& a, cudaStream_t s) {
    const bool half = a.layout == MUON_ROTARY_HALF;
    const int w = group_width<T>(a, p.copy);
    const int64_t turning = half ? a.pairs / w : a.pairs / (w > 1 ? w / 2 : 1);
    p.units = static_cast<uint32_t>(turning + (p.copy ? (a.head - 2 * a.pairs) / w : 0));
    // as many tokens a block as give every thread four units and a cosine,
    // and no more than leave every SM a block
    const int64_t units = (a.q.heads + a.k.heads) * p.units;
    int64_t t = ceil_div(4 * R_THREADS, units);
    if (t * a.pairs < R_THREADS) t = ceil_div(R_THREADS, a.pairs);
    if (t > R_PAIRS / a.pairs) t = R_PAIRS / a.pairs;
    if (t > ceil_div(p.tokens, 152)) t = ceil_div(p.tokens, 152);
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
    p.seq = static_cast<uint32_t>(a.seq);
    p.head = static_cast<uint32_t>(a.head);
    p.pairs = static_cast<uint32_t>(a.pairs);
    p.scale = a.scale;
    p.sign = a.inverse ? -1.f : 1.f;
    const bool rest = a.head > 2 * a.pairs;
    p.copy = rest && ((a.q.heads && a.q.x != a.q.y) || (a.k.heads && a.k.x != a.k.y));
    for (int64_t i = 0; i < a.pairs; ++i) p.turns[i] = a.turns[i];
    return a.x_dtype == MUON_F32 ? launch<float>(p, a, s) : launch<__nv_bfloat16>(p, a, s);
}

}  // namespace ops
}  // namespace muon
