// The router of a mixture-of-experts block (muon_route, muon_route_grad):
// softmax over the experts, the k largest logits, counts, offsets and the
// balance loss; its gradient.
//
// A token's logits lie in the registers of a warp (of eight lanes up to 32
// experts), in pieces of four neighbouring experts: expert e is value e % 4
// of piece e / 4, and lane l has the pieces l, l + L, ...  The k largest are
// taken from the logits themselves, one after another, so that which experts
// are taken depends on no rounding; a tie goes to the lower index.
//
// Sums of p over the tokens collect in registers, then in one row of partial
// results a block; a cluster of blocks adds these up in order and computes
// offsets and loss.
//
// What bounds the forward pass is the arithmetic of the selection and of the
// exponentials: 32769 tokens of 384 experts, bf16, k = 8: 26 us, 71 % of the
// integer pipe's rate, and 11 us for the second kernel; 262144 tokens 178 us
// (fp32 253 us).  The gradient: 19 us, and 114 us (3.7 TB/s).  200 tokens of
// 128 experts take 5 us in each of the two kernels, a launch's latency.
#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace muon {
namespace ops {
namespace {

constexpr int SMS = 152;
constexpr int JOIN_CTAS = 8;             // the cluster of the second kernel
constexpr int JOIN_THREADS = 512;

template <int V>
__host__ __device__ constexpr int route_threads() { return V <= 16 ? 512 : 256; }

// Values of the L lanes of a token; all lanes of the warp take part.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if constexpr (L == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
template <int L>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
    return ~group_max<L>(~v);
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// e^x for x <= 0 as 2^t (1 + r ln 2), where t is x log2(e) as fp32 holds it and r
// what that leaves: without r the error grows with |x|, to 9e-6 at 100.  Below
// 2^-126 it is 0; a NaN stays one (the limit keeps -infinity out of r).  Two at
// a time it takes the time of the intrinsic without r (262144 tokens of 384
// experts, bf16: 178 us, the gradient 114 and 118 us; 198 and 126 us with expf).
__device__ __forceinline__ float2 exp2_of(float2 x) {
    constexpr float LOG2E = 1.44269502f, REST = 1.92596299e-8f, LN2 = 0.693147181f;
    float2 e;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.x) : "f"(x.x), "f"(-104.f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x.y) : "f"(x.y), "f"(-104.f));
    const float2 t = mul2(x, both(LOG2E));
    const float2 r = fma2(x, both(REST), fma2(x, both(LOG2E), make_float2(-t.x, -t.y)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    return fma2(e, mul2(r, both(LN2)), e);
}
__device__ __forceinline__ float exp_of(float x) {
    constexpr float LOG2E = 1.44269502f, REST = 1.92596299e-8f, LN2 = 0.693147181f;
    float e;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(-104.f));
    const float t = x * LOG2E;
    const float r = fmaf(x, REST, fmaf(x, LOG2E, -t));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return fmaf(e, r * LN2, e);
}
// v = e^(v - top); their sum.  In pairs, but for the forward pass of lanes with
// four values, whose loop over the tokens comes out slower so (2^20 tokens of 8
// experts: 128 us instead of 94; the gradient 59 us, and 61 one at a time).
template <bool PAIRS, int V>
__device__ __forceinline__ float exp_all(float (&v)[V], float top) {
    if constexpr (!PAIRS) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = exp_of(v[i] - top);
            sum += v[i];
        }
        return sum;
    } else {
        float2 sum = both(0.f);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 e = exp2_of(add2(make_float2(v[i], v[i + 1]), both(-top)));
            v[i] = e.x;
            v[i + 1] = e.y;
            sum = add2(sum, e);
        }
        return sum.x + sum.y;
    }
}

// A logit's place in the order of the reals as an unsigned number: never 0,
// which stands for no logit; a NaN is the largest.  Adding 0 makes -0 a 0 and
// every NaN the positive one.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// The V logits of a lane; those past the experts are -infinity.  AL: pieces
// are whole and lie on their size.
template <typename T, int V, int L, bool AL>
struct Logits {
    static constexpr int P = V / 4;
    uint4 raw[P];
    static __device__ __forceinline__ int expert(int i, int lane) { return (i / 4 * L + lane) * 4 + i % 4; }
    __device__ __forceinline__ void load(const T* z, int lane, int experts, bool there) {
        const uint32_t none = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * L + lane) * 4;
            raw[p] = make_uint4(none, none, none, none);
            if (!there || e >= experts) continue;
            if constexpr (AL && sizeof(T) == 4) {
                raw[p] = *reinterpret_cast<const uint4*>(z + e);
            } else if constexpr (AL) {
                const uint2 t = *reinterpret_cast<const uint2*>(z + e);
                raw[p].x = t.x;
                raw[p].y = t.y;
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j] = sizeof(T) == 4 ? 0xff800000u : 0xff80u;
                    if (e + j < experts) {
                        if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(z[e + j]);
                        else w[j] = __bfloat16_as_ushort(z[e + j]);
                    }
                }
                if constexpr (sizeof(T) == 4) {
                    raw[p] = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    raw[p].x = w[0] | w[1] << 16;
                    raw[p].y = w[2] | w[3] << 16;
                }
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if constexpr (sizeof(T) == 4) {
                v[4 * p] = __uint_as_float(raw[p].x);
                v[4 * p + 1] = __uint_as_float(raw[p].y);
                v[4 * p + 2] = __uint_as_float(raw[p].z);
                v[4 * p + 3] = __uint_as_float(raw[p].w);
            } else {
                v[4 * p] = __uint_as_float(raw[p].x << 16);
                v[4 * p + 1] = __uint_as_float(raw[p].x & 0xffff0000u);
                v[4 * p + 2] = __uint_as_float(raw[p].y << 16);
                v[4 * p + 3] = __uint_as_float(raw[p].y & 0xffff0000u);
            }
        }
    }
    static __device__ __forceinline__ void store(T* z, const float (&v)[V], int lane, int experts) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * L + lane) * 4;
            if (e >= experts) continue;
            if constexpr (AL && sizeof(T) == 4) {
                *reinterpret_cast<float4*>(z + e) =
                    make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
            } else if constexpr (AL) {
                const __nv_bfloat162 a = __floats2bfloat162_rn(v[4 * p], v[4 * p + 1]);
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[4 * p + 2], v[4 * p + 3]);
                *reinterpret_cast<uint2*>(z + e) = make_uint2(reinterpret_cast<const uint32_t&>(a),
                                                              reinterpret_cast<const uint32_t&>(b));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (e + j < experts) from_f32(z + e + j, v[4 * p + j]);
            }
        }
    }
};

// The largest logits of a token, one a call.  bf16: a key has the logit's 16
// bits and below them 65535 - expert, so that no two are equal and the next
// one is the largest key below the last.
template <typename T, int V, int L>
struct Selection {
    uint32_t key[V], best;               // best: this lane's largest left
    __device__ __forceinline__ void start(const float (&v)[V], int lane, int experts) {
        best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = Logits<T, V, L, true>::expert(i, lane);
            const uint32_t k = (order_key(v[i]) & 0xffff0000u) | (65535u - e);
            key[i] = e < experts ? k : 0u;
            best = max(best, key[i]);
        }
    }
    __device__ __forceinline__ uint32_t next(int) {
        const uint32_t top = group_max<L>(best);
        // differences wrap: those of keys below top are the larger ones
        uint32_t d = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) d = max(d, key[i] - top);
        best = top + d < top ? top + d : 0u;
        return top;
    }
    static __device__ __forceinline__ float value(uint32_t top) {
        // the index's bits are no part of the logit
        return __uint_as_float(__float_as_uint(key_value(top)) & 0xffff0000u);
    }
    __device__ __forceinline__ int expert(uint32_t top) const { return 65535 - (top & 0xffffu); }
};
// fp32: the key is the whole logit.  A lane knows its largest two and where
// they are; only where both are taken (once a token or so) it looks through
// its keys again, for the largest one after the last in the order by key and
// then by index (262144 tokens of 384 experts: 253 us, and 427 us looking
// after each).
template <int V, int L>
struct Selection<float, V, L> {
    uint32_t key[V], best, second;       // 0: not known
    int at, at2, taken;
    __device__ __forceinline__ void start(const float (&v)[V], int lane, int experts) {
        best = second = 0;
        at = at2 = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = Logits<float, V, L, true>::expert(i, lane) < experts ? order_key(v[i]) : 0u;
            if (key[i] > best) {
                second = best;
                at2 = at;
                best = key[i];
                at = i;
            } else if (key[i] > second) {
                second = key[i];
                at2 = i;
            }
        }
    }
    __device__ __forceinline__ uint32_t next(int lane) {
        const uint32_t top = group_max<L>(best);
        const uint32_t e = ((at >> 2) * L + lane) * 4 + (at & 3);
        taken = static_cast<int>(group_min<L>(best == top ? e : 0xffffffffu));
        const bool mine = top && best == top && static_cast<int>(e) == taken;
        const int last = at;
        if (mine) {
            best = second;
            at = at2;
            second = 0;
        }
        if (__any_sync(0xffffffffu, mine && best == 0u)) {
            if (mine && best == 0u) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i] > best && (key[i] < top || (key[i] == top && i > last))) {
                        best = key[i];
                        at = i;
                    }
            }
        }
        return top;
    }
    static __device__ __forceinline__ float value(uint32_t top) { return key_value(top); }
    __device__ __forceinline__ int expert(uint32_t) const { return taken; }
};

// Partial results of a block: sums of p, then counts, then tokens kept.
__host__ __device__ __forceinline__ int64_t part_words(int64_t experts) { return 2 * experts + 1; }

template <typename T, int V, int L, bool AL>
__global__ void __launch_bounds__(route_threads<V>())
    route_kernel(const __grid_constant__ muon_route_args a, float* part) {
    constexpr int THREADS = route_threads<V>(), WARPS = THREADS / 32, ROWS = THREADS / L;
    extern __shared__ float s_p[];               // WARPS x experts
    __shared__ int s_c[1024];
    __shared__ int s_kept;
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x % L, warp = threadIdx.x >> 5;
    const int E = static_cast<int>(a.experts), K = static_cast<int>(a.k);
    for (int e = threadIdx.x; e < E; e += THREADS) s_c[e] = 0;
    if (threadIdx.x == 0) s_kept = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    int kept = 0;
    const int64_t stride = int64_t(gridDim.x) * ROWS;
    // a block's lanes walk on together: the reductions ask every lane
    const int64_t last = (a.tokens + ROWS - 1) / ROWS * ROWS;
    int64_t t = int64_t(blockIdx.x) * ROWS + threadIdx.x / L;
    Logits<T, V, L, AL> z;
    bool use = false;
    auto fetch = [&](int64_t row) {
        use = row < a.tokens && (!a.mask || a.mask[row]);
        z.load(static_cast<const T*>(a.logits) + row * a.ld_z, lane, E, use);
    };
    fetch(t);
    for (; t < last; t += stride) {
        float v[V];
        z.get(v);
        const bool masked_out = !use;
        fetch(t + stride);                       // ahead of this token's work
        Selection<T, V, L> sel;
        sel.start(v, lane, E);
        uint32_t top = sel.next(lane);
        const float shift = sel.value(top);
        const bool keep = !masked_out && !(shift == -INFINITY);
        const float sum = exp_all<(V > 4)>(v, shift);
        const float inv = 1.f / group_sum<L>(sum);
        if (keep) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
            if (lane == 0) ++kept;
        }
        int my_e = 0;
        uint32_t my_key = 0;
        for (int j = 0;;) {
            if (lane == j) {
                my_key = top;
                my_e = sel.expert(top);
            }
            if (++j == K) break;
            top = sel.next(lane);
        }
        const float my_v = sel.value(my_key);
        const bool mine = keep && lane < K && my_key && !(my_v == -INFINITY);
        float w = mine ? exp_of(my_v - shift) * inv : 0.f;
        if (a.renormalise) {
            const float total = group_sum<L>(w);
            if (mine) w /= total;
        }
        if (lane < K && t < a.tokens) {
            a.indices[t * K + lane] = mine ? my_e : -1;
            a.weights[t * K + lane] = w;
            if (mine) atomicAdd(&s_c[my_e], 1);
        }
    }
    if (kept) atomicAdd(&s_kept, kept);
    // over a warp's tokens (eight lanes each), then the warps' sums in order
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        const int e = Logits<T, V, L, AL>::expert(i, lane);
        if (e < E && (threadIdx.x & 31) < L) s_p[warp * E + e] = acc[i];
    }
    __syncthreads();
    float* out = part + blockIdx.x * part_words(E);
    for (int e = threadIdx.x; e < E; e += THREADS) {
        float p = 0.f;
        for (int w = 0; w < WARPS; ++w) p += s_p[w * E + e];
        out[e] = p;
        reinterpret_cast<int*>(out)[E + e] = s_c[e];
    }
    if (threadIdx.x == 0) reinterpret_cast<int*>(out)[2 * E] = s_kept;
}

// Stores a word to this variable of CTA `rank` of the cluster.
__device__ __forceinline__ void store_to_rank(void* at, uint32_t rank, uint32_t v) {
    const uint32_t addr = ptx::map_to_rank(ptx::smem_u32(at), rank);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// One cluster: each CTA adds up the n partial results of its experts, with as
// many threads an expert as there are (in order within a thread, then the
// threads in order); CTA 0 makes offsets and loss of them.
__global__ void __cluster_dims__(JOIN_CTAS, 1, 1) __launch_bounds__(JOIN_THREADS)
    route_join_kernel(const __grid_constant__ muon_route_args a, const float* part, int n) {
    __shared__ float s_p[JOIN_THREADS];
    __shared__ int s_n[JOIN_THREADS];
    __shared__ int s_count[1024];
    __shared__ float s_term[1024];               // count times sum of p
    __shared__ int s_warp[JOIN_THREADS / 32];
    __shared__ float s_sum[JOIN_THREADS / 32];
    grid_dependency_wait();
    allow_dependent_launch();
    const int E = static_cast<int>(a.experts);
    const int64_t words = part_words(E);
    const int each = (E + JOIN_CTAS - 1) / JOIN_CTAS;        // at most 128
    const int slices = JOIN_THREADS / each;
    const int mine = threadIdx.x % each, slice = threadIdx.x / each;
    const int e = blockIdx.x * each + mine;
    const int* ints = reinterpret_cast<const int*>(part);
    float p = 0.f;
    int c = 0;
    if (e < E && slice < slices)
#pragma unroll 4
        for (int i = slice; i < n; i += slices) {
            p += part[i * words + e];
            c += ints[i * words + E + e];
        }
    s_p[threadIdx.x] = p;
    s_n[threadIdx.x] = c;
    ptx::cluster_sync_all();                              // every CTA runs: its memory can be written
    if (slice == 0 && e < E) {
        for (int s = 1; s < slices; ++s) {
            p += s_p[s * each + mine];
            c += s_n[s * each + mine];
        }
        a.counts[e] = c;
        store_to_rank(&s_count[e], 0, c);
        store_to_rank(&s_term[e], 0, __float_as_uint(static_cast<float>(c) * p));
    }
    ptx::cluster_sync_all();
    if (blockIdx.x != 0) return;
    // two experts a thread: offsets by scanning, the loss's sum, tokens kept
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e0 = 2 * threadIdx.x;
    const int c0 = e0 < E ? s_count[e0] : 0, c1 = e0 + 1 < E ? s_count[e0 + 1] : 0;
    int scan = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
    }
    const float term = warp_sum((e0 < E ? s_term[e0] : 0.f) + (e0 + 1 < E ? s_term[e0 + 1] : 0.f));
    int kept = 0;
    for (int i = threadIdx.x; i < n; i += JOIN_THREADS) kept += ints[i * words + 2 * E];
    kept = __reduce_add_sync(0xffffffffu, kept);
    if (lane == 31) s_warp[warp] = scan;
    if (lane == 0) {
        s_sum[warp] = term;
        s_n[warp] = kept;
    }
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    before += scan - c0 - c1;
    if (e0 < E) a.offsets[e0 + 1] = before + c0;
    if (e0 + 1 < E) a.offsets[e0 + 2] = before + c0 + c1;
    if (threadIdx.x == 0) {
        a.offsets[0] = 0;
        float total = 0.f;
        kept = 0;
        for (int w = 0; w < JOIN_THREADS / 32; ++w) {
            total += s_sum[w];
            kept += s_n[w];
        }
        *a.kept = kept;
        const float t = static_cast<float>(kept);
        *a.loss = kept ? a.coef * static_cast<float>(E) / (static_cast<float>(a.k) * t) * (total / t) : 0.f;
    }
}

// dz = p (h - sum p h), where h is the loss's part, the same for all tokens
// (count times a factor, in registers), and for the taken experts also that
// of their weights: a lane computes theirs again and stores them over the
// others'.  Registers for four blocks an SM: 262144 tokens of 384 experts
// bf16 114 us, fp32 163 us (5.1 TB/s); 126 and 181 us with what the compiler
// takes (79 registers).
template <typename T, int V, int L, bool AL>
__global__ void __launch_bounds__(256, V <= 16 ? 4 : 2)
    route_grad_kernel(const __grid_constant__ muon_route_grad_args a) {
    constexpr int ROWS = 256 / L;
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x % L, base = (threadIdx.x & 31) / L * L;
    const int E = static_cast<int>(a.experts), K = static_cast<int>(a.k);
    const float kept = static_cast<float>(max(1, *a.kept));
    const float factor = (a.dloss ? *a.dloss : 0.f) * a.coef * static_cast<float>(E) /
                         (static_cast<float>(K) * kept) / kept;
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = Logits<T, V, L, AL>::expert(i, lane);
        f[i] = e < E ? factor * static_cast<float>(a.counts[e]) : 0.f;
    }
    const int64_t stride = int64_t(gridDim.x) * ROWS;
    const int64_t last = (a.tokens + ROWS - 1) / ROWS * ROWS;
    int64_t t = int64_t(blockIdx.x) * ROWS + threadIdx.x / L;
    Logits<T, V, L, AL> z;
    int my_e = -1;
    auto fetch = [&](int64_t row) {
        z.load(static_cast<const T*>(a.logits) + row * a.ld_z, lane, E, row < a.tokens);
        my_e = -1;
        if (lane < K && row < a.tokens) my_e = a.indices[row * K + lane];
        if (my_e >= E) my_e = -1;
    };
    fetch(t);
    for (; t < last; t += stride) {
        const int e = my_e;
        const bool row = t < a.tokens;
        float v[V];
        z.get(v);
        float my_z = 0.f, my_w = 0.f, my_d = 0.f, my_f = 0.f;
        if (e >= 0) {
            my_z = to_f32(static_cast<const T*>(a.logits)[t * a.ld_z + e]);
            my_w = a.weights[t * K + lane];
            my_d = a.dweights ? a.dweights[t * a.ld_dw + lane] : 0.f;
            my_f = factor * static_cast<float>(a.counts[e]);
        }
        fetch(t + stride);
        // the first place holds the largest logit, and is empty only if the
        // token takes no part
        const float top = __shfl_sync(0xffffffffu, my_z, base);
        const bool keep = __shfl_sync(0xffffffffu, e, base) >= 0;
        const float sum = exp_all<true>(v, top);
        const float inv = 1.f / group_sum<L>(sum);
        float my_p = e >= 0 ? exp_of(my_z - top) * inv : 0.f;
        if (a.dweights && a.renormalise) {
            const float taken = group_sum<L>(my_p), mean = group_sum<L>(my_w * my_d);
            my_d = e >= 0 ? (my_d - mean) / taken : 0.f;
        }
        float inner = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] *= inv;
            inner = fmaf(v[i], f[i], inner);
        }
        inner = group_sum<L>(fmaf(my_p, my_d, inner));
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = keep ? v[i] * (f[i] - inner) : 0.f;
        T* dz = static_cast<T*>(a.dlogits) + t * a.ld_dz;
        if (row) Logits<T, V, L, AL>::store(dz, v, lane, E);
        __syncwarp();                            // the stores below come after those
        if (row && e >= 0) from_f32(dz + e, my_p * (my_f + my_d - inner));
    }
}

// Rows of a block (of 512 or 256 threads) and how many blocks run.
int route_v(int64_t experts) { return static_cast<int>(ceil_div(experts, 128) * 4); }
// Eight lanes a token, four tokens a warp, where they hold the experts and the
// taken ones (2^20 tokens of 8 experts, k = 2, bf16: 94 us, with a warp a token
// 325; 32 experts, k = 4: 100 and 358 us; the gradient of 8 experts 59 and 237).
bool eight_lanes(int64_t experts, int64_t k) { return experts <= 32 && k <= 8; }
int route_rows(int64_t experts, int64_t k) {
    return eight_lanes(experts, k) ? 64 : route_v(experts) <= 16 ? 16 : 8;
}
int route_parts(const muon_route_args& a) {
    const int64_t g = ceil_div(a.tokens, route_rows(a.experts, a.k));
    return static_cast<int>(g < 1 ? 1 : g > SMS * 2 ? SMS * 2 : g);
}

template <typename T, int V, int L, bool AL>
cudaError_t launch_route_v(const muon_route_args& a, float* part, cudaStream_t s) {
    const size_t smem = size_t(route_threads<V>() / 32) * a.experts * 4;
    return launch_kernel(route_kernel<T, V, L, AL>, dim3(route_parts(a)), dim3(route_threads<V>()), smem,
                         s, a, part);
}
template <typename T, int V, int L, bool AL>
cudaError_t launch_grad_v(const muon_route_grad_args& a, cudaStream_t s) {
    const int64_t g = ceil_div(a.tokens, 256 / L);
    return launch_kernel(route_grad_kernel<T, V, L, AL>,
                         dim3(static_cast<unsigned>(g > SMS * 8 ? SMS * 8 : g)), dim3(256), 0, s, a);
}

template <typename T, bool AL>
cudaError_t route_t(const muon_route_args& a, float* part, cudaStream_t s) {
    if (eight_lanes(a.experts, a.k)) return launch_route_v<T, 4, 8, AL>(a, part, s);
    switch (route_v(a.experts)) {
        case 4: return launch_route_v<T, 4, 32, AL>(a, part, s);
        case 8: return launch_route_v<T, 8, 32, AL>(a, part, s);
        case 12: return launch_route_v<T, 12, 32, AL>(a, part, s);
        case 16: return launch_route_v<T, 16, 32, AL>(a, part, s);
        default: return launch_route_v<T, 32, 32, AL>(a, part, s);
    }
}
template <typename T, bool AL>
cudaError_t route_grad_t(const muon_route_grad_args& a, cudaStream_t s) {
    if (eight_lanes(a.experts, a.k)) return launch_grad_v<T, 4, 8, AL>(a, s);
    switch (route_v(a.experts)) {
        case 4: return launch_grad_v<T, 4, 32, AL>(a, s);
        case 8: return launch_grad_v<T, 8, 32, AL>(a, s);
        case 12: return launch_grad_v<T, 12, 32, AL>(a, s);
        case 16: return launch_grad_v<T, 16, 32, AL>(a, s);
        default: return launch_grad_v<T, 32, 32, AL>(a, s);
    }
}

// Whole pieces of four that lie on their size.
bool whole_pieces(const void* p, int dtype, int64_t rows, int64_t experts, int64_t ld) {
    const int64_t size = dtype == MUON_F32 ? 16 : 8;
    return experts % 4 == 0 && reinterpret_cast<uintptr_t>(p) % size == 0 && (rows <= 1 || ld % 4 == 0);
}

}  // namespace

size_t route_workspace(const muon_route_args& a) {
    return size_t(route_parts(a)) * part_words(a.experts) * 4;
}

cudaError_t launch_route(const muon_route_args& a, void* ws, cudaStream_t s) {
    float* part = static_cast<float*>(ws);
    const bool al = whole_pieces(a.logits, a.z_dtype, a.tokens, a.experts, a.ld_z);
    cudaError_t e;
    if (a.z_dtype == MUON_F32)
        e = al ? route_t<float, true>(a, part, s) : route_t<float, false>(a, part, s);
    else
        e = al ? route_t<__nv_bfloat16, true>(a, part, s) : route_t<__nv_bfloat16, false>(a, part, s);
    if (e != cudaSuccess) return e;
    return launch_kernel(route_join_kernel, dim3(JOIN_CTAS), dim3(JOIN_THREADS), 0, s, a,
                         static_cast<const float*>(part), route_parts(a));
}

cudaError_t launch_route_grad(const muon_route_grad_args& a, cudaStream_t s) {
    if (a.tokens == 0) return cudaSuccess;
    const bool al = whole_pieces(a.logits, a.z_dtype, a.tokens, a.experts, a.ld_z) &&
                    whole_pieces(a.dlogits, a.z_dtype, a.tokens, a.experts, a.ld_dz);
    if (a.z_dtype == MUON_F32)
        return al ? route_grad_t<float, true>(a, s) : route_grad_t<float, false>(a, s);
    return al ? route_grad_t<__nv_bfloat16, true>(a, s) : route_grad_t<__nv_bfloat16, false>(a, s);
}

}  // namespace ops
}  // namespace muon
