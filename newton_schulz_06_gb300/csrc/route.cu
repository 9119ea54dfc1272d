// The router of a mixture-of-experts block (muon_route, muon_route_grad):
// softmax over the experts, the k largest logits, counts, offsets and the
// balance loss; its gradient.
//
// One warp holds a token's logits, expert e in lane e % 32.  The k largest
// are taken from the logits themselves, one after another, so that which
// experts are taken depends on no rounding; a tie goes to the lower index.
#include "ops_internal.h"

namespace muon {
namespace ops {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_PARTS = 304;       // blocks of the first kernel

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A logit's place in the order of the reals as an unsigned number; 0 for
// -infinity, which is never taken, and the largest for a NaN, whose token's
// weights and gradients then show it.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xffffffffu;
    if (v == -INFINITY) return 0u;
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);    // -0 and 0 are equal
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Partial results of a block: sums of p, then counts, then tokens kept.
__host__ __device__ __forceinline__ int64_t part_words(int64_t experts) { return 2 * experts + 1; }

// V: logits a lane holds (experts <= 32 V).
template <typename T, int V>
__global__ void __launch_bounds__(THREADS)
    route_kernel(const __grid_constant__ muon_route_args a, float* part) {
    __shared__ float s_p[1024];
    __shared__ int s_c[1024];
    __shared__ int s_kept;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = static_cast<int>(a.experts), K = static_cast<int>(a.k);
    for (int e = threadIdx.x; e < E; e += THREADS) {
        s_p[e] = 0.f;
        s_c[e] = 0;
    }
    if (threadIdx.x == 0) s_kept = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int64_t t = blockIdx.x * int64_t(WARPS) + warp; t < a.tokens;
         t += int64_t(gridDim.x) * WARPS) {
        const T* z = static_cast<const T*>(a.logits) + t * a.ld_z;
        bool keep = !a.mask || a.mask[t];
        float v[V];
        float top = -INFINITY;
        bool nan = false;
        if (keep) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = i * 32 + lane;
                v[i] = e < E ? to_f32(z[e]) : -INFINITY;
                nan |= v[i] != v[i];
                top = fmaxf(top, v[i]);
            }
            top = warp_max(top);
            nan = __any_sync(0xffffffffu, nan);
            keep = nan || top > -INFINITY;
        }
        int32_t* idx = a.indices + t * K;
        float* wt = a.weights + t * K;
        if (!keep) {
            if (lane < K) {
                idx[lane] = -1;
                wt[lane] = 0.f;
            }
            continue;
        }
        float p[V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = expf(v[i] - top);
            sum += p[i];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] /= sum;
            if (i * 32 + lane < E) acc[i] += p[i];
        }
        uint32_t key[V];
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = order_key(v[i]);
        int my_e = -1;
        float my_w = 0.f, taken = 0.f;
        for (int j = 0; j < K; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) best = max(best, key[i]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best == 0u) break;
            // the lowest index among the equal ones
            int at = 1 << 30;
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
                if (key[i] == best) at = i * 32 + lane;
            at = __reduce_min_sync(0xffffffffu, at);
            float pw = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * 32 + lane == at) {
                    pw = p[i];
                    key[i] = 0u;
                }
            pw = __shfl_sync(0xffffffffu, pw, at & 31);
            taken += pw;
            if (lane == j) {
                my_e = at;
                my_w = pw;
            }
        }
        if (lane < K) {
            idx[lane] = my_e;
            wt[lane] = a.renormalise && my_e >= 0 ? my_w / taken : my_w;
            if (my_e >= 0) atomicAdd(&s_c[my_e], 1);
        }
        if (lane == 0) atomicAdd(&s_kept, 1);
    }
    // sums of p in the order of the warps
    for (int w = 0; w < WARPS; ++w) {
        __syncthreads();
        if (w == warp) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * 32 + lane < E) s_p[i * 32 + lane] += acc[i];
        }
    }
    __syncthreads();
    float* out = part + blockIdx.x * part_words(E);
    for (int e = threadIdx.x; e < E; e += THREADS) {
        out[e] = s_p[e];
        reinterpret_cast<int*>(out)[E + e] = s_c[e];
    }
    if (threadIdx.x == 0) reinterpret_cast<int*>(out)[2 * E] = s_kept;
}

// One block: the partial results in order, offsets, loss.
__global__ void __launch_bounds__(1024)
    route_join_kernel(const __grid_constant__ muon_route_args a, const float* part, int n) {
    __shared__ int s_scan[1024];
    __shared__ float s_sum[32];
    __shared__ int s_kept;
    const int e = threadIdx.x, E = static_cast<int>(a.experts);
    const int64_t words = part_words(E);
    float p = 0.f;
    int c = 0;
    if (e < E)
        for (int i = 0; i < n; ++i) {
            p += part[i * words + e];
            c += reinterpret_cast<const int*>(part)[i * words + E + e];
        }
    if (e == 0) {
        int kept = 0;
        for (int i = 0; i < n; ++i) kept += reinterpret_cast<const int*>(part)[i * words + 2 * E];
        s_kept = kept;
        *a.kept = kept;
    }
    s_scan[e] = c;
    for (int o = 1; o < 1024; o <<= 1) {
        __syncthreads();
        const int add = e >= o ? s_scan[e - o] : 0;
        __syncthreads();
        s_scan[e] += add;
    }
    if (e < E) {
        a.counts[e] = c;
        a.offsets[e + 1] = s_scan[e];
        if (e == 0) a.offsets[0] = 0;
    }
    const float part_sum = warp_sum(e < E ? static_cast<float>(c) * p : 0.f);
    if ((e & 31) == 0) s_sum[e >> 5] = part_sum;
    __syncthreads();
    if (e < 32) {
        const float total = warp_sum(s_sum[e]);
        const float kept = static_cast<float>(s_kept);
        if (e == 0)
            *a.loss = s_kept ? a.coef * static_cast<float>(E) / (static_cast<float>(a.k) * kept) *
                                   (total / kept)
                             : 0.f;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS)
    route_grad_kernel(const __grid_constant__ muon_route_grad_args a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = static_cast<int>(a.experts), K = static_cast<int>(a.k);
    const float kept = static_cast<float>(max(1, *a.kept));
    const float factor = (a.dloss ? *a.dloss : 0.f) * a.coef * static_cast<float>(E) /
                         (static_cast<float>(K) * kept) / kept;
    for (int64_t t = blockIdx.x * int64_t(WARPS) + warp; t < a.tokens;
         t += int64_t(gridDim.x) * WARPS) {
        const T* z = static_cast<const T*>(a.logits) + t * a.ld_z;
        T* dz = static_cast<T*>(a.dlogits) + t * a.ld_dz;
        int my_e = -1;
        float my_w = 0.f, my_d = 0.f;
        if (lane < K) {
            my_e = a.indices[t * K + lane];
            if (my_e >= E) my_e = -1;
            if (my_e >= 0) {
                my_w = a.weights[t * K + lane];
                my_d = a.dweights ? a.dweights[t * a.ld_dw + lane] : 0.f;
            }
        }
        // the first place is empty only if the token takes no part
        if (__shfl_sync(0xffffffffu, my_e, 0) < 0) {
            for (int e = lane; e < E; e += 32) from_f32(dz + e, 0.f);
            continue;
        }
        float p[V], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * 32 + lane;
            p[i] = e < E ? to_f32(z[e]) : -INFINITY;
            top = fmaxf(top, p[i]);
        }
        top = warp_max(top);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = expf(p[i] - top);
            sum += p[i];
        }
        sum = warp_sum(sum);
        float h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * 32 + lane;
            p[i] /= sum;
            h[i] = e < E ? factor * static_cast<float>(a.counts[e]) : 0.f;
        }
        if (a.dweights) {
            if (a.renormalise) {
                float taken = 0.f;
                for (int j = 0; j < K; ++j) {
                    const int e = __shfl_sync(0xffffffffu, my_e, j);
                    float pe = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i * 32 + lane == e) pe = p[i];
                    taken += e >= 0 ? __shfl_sync(0xffffffffu, pe, e & 31) : 0.f;
                }
                const float inner = warp_sum(my_w * my_d);
                my_d = my_e >= 0 ? (my_d - inner) / taken : 0.f;
            }
            for (int j = 0; j < K; ++j) {
                const int e = __shfl_sync(0xffffffffu, my_e, j);
                const float d = __shfl_sync(0xffffffffu, my_d, j);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i * 32 + lane == e) h[i] += d;
            }
        }
        float inner = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) inner = fmaf(p[i], h[i], inner);
        inner = warp_sum(inner);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = i * 32 + lane;
            if (e < E) from_f32(dz + e, p[i] * (h[i] - inner));
        }
    }
}

int route_parts(int64_t tokens) {
    const int64_t g = ceil_div(tokens, WARPS);
    return static_cast<int>(g < 1 ? 1 : g > MAX_PARTS ? MAX_PARTS : g);
}

template <typename T, int V>
cudaError_t route_v(const muon_route_args& a, float* part, cudaStream_t s) {
    const int g = route_parts(a.tokens);
    route_kernel<T, V><<<g, THREADS, 0, s>>>(a, part);
    route_join_kernel<<<1, 1024, 0, s>>>(a, part, g);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t route_grad_v(const muon_route_grad_args& a, cudaStream_t s) {
    const int64_t g = ceil_div(a.tokens, WARPS);
    route_grad_kernel<T, V><<<static_cast<int>(g > 152 * 8 ? 152 * 8 : g), THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t route_t(const muon_route_args& a, float* part, cudaStream_t s) {
    if (a.experts <= 128) return route_v<T, 4>(a, part, s);
    if (a.experts <= 512) return route_v<T, 16>(a, part, s);
    return route_v<T, 32>(a, part, s);
}
template <typename T>
cudaError_t route_grad_t(const muon_route_grad_args& a, cudaStream_t s) {
    if (a.experts <= 128) return route_grad_v<T, 4>(a, s);
    if (a.experts <= 512) return route_grad_v<T, 16>(a, s);
    return route_grad_v<T, 32>(a, s);
}

}  // namespace

size_t route_workspace(const muon_route_args& a) {
    return size_t(route_parts(a.tokens)) * part_words(a.experts) * 4;
}

cudaError_t launch_route(const muon_route_args& a, void* ws, cudaStream_t s) {
    return a.z_dtype == MUON_F32 ? route_t<float>(a, static_cast<float*>(ws), s)
                                 : route_t<__nv_bfloat16>(a, static_cast<float*>(ws), s);
}

cudaError_t launch_route_grad(const muon_route_grad_args& a, cudaStream_t s) {
    if (a.tokens == 0) return cudaSuccess;
    return a.z_dtype == MUON_F32 ? route_grad_t<float>(a, s) : route_grad_t<__nv_bfloat16>(a, s);
}

}  // namespace ops
}  // namespace muon
