// The weight gradient of a product from an 8-bit checkpoint
// (muon_weight_grad): G = dY^T X (+ C), one matrix or one per expert.
#include "ops_internal.h"

namespace muon {
namespace ops {
namespace {

constexpr int TILE = 64;
constexpr int THREADS = 256;

// Rows [begin, end) of matrix e.
__device__ __forceinline__ void segment(const muon_weight_grad_args& a, int64_t e, int64_t* begin,
                                        int64_t* end) {
    *begin = 0;
    *end = a.rows;
    if (a.offsets) {
        *begin = min(max(int64_t(a.offsets[e]), int64_t(0)), a.rows);
        *end = min(max(int64_t(a.offsets[e + 1]), *begin), a.rows);
    }
}

// One 64 x 64 tile of one matrix: 4 x 4 sums a thread.
__global__ void __launch_bounds__(THREADS)
    weight_grad_kernel(const __grid_constant__ muon_weight_grad_args a) {
    __shared__ float s_dy[16][TILE + 1];
    __shared__ float s_h[16][TILE + 1];
    const int64_t j0 = blockIdx.x * int64_t(TILE), i0 = blockIdx.y * int64_t(TILE);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t e = blockIdx.z; e < a.experts; e += gridDim.z) {
        int64_t begin, end;
        segment(a, e, &begin, &end);
        float acc[4][4] = {}, sum[4] = {};
        for (int64_t t0 = begin; t0 < end; t0 += 16) {
            for (int u = threadIdx.x; u < 16 * TILE; u += THREADS) {
                const int64_t t = t0 + u / TILE;
                const int64_t i = i0 + u % TILE, j = j0 + u % TILE;
                s_dy[u / TILE][u % TILE] =
                    t < end && i < a.n
                        ? __bfloat162float(
                              static_cast<const __nv_bfloat16*>(a.dy)[t * a.ld_dy + i])
                        : 0.f;
                s_h[u / TILE][u % TILE] =
                    t < end && j < a.k
                        ? static_cast<float>(a.saved.q[t * a.saved.ld_q + j]) * 0.015625f *
                              scale_pow(a.saved.e[t * a.saved.ld_e + j / CKPT_BLOCK])
                        : 0.f;
            }
            __syncthreads();
            for (int u = 0; u < 16; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float d = s_dy[u][ty * 4 + x];
                    sum[x] += d;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        acc[x][y] = fmaf(d, s_h[u][tx + 16 * y], acc[x][y]);
                }
            __syncthreads();
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int64_t i = i0 + ty * 4 + x, j = j0 + tx + 16 * y;
                if (i >= a.n || j >= a.k) continue;
                float g = acc[x][y];
                if (a.weight) g *= a.weight[j];
                if (a.bias) g = fmaf(a.bias[j], sum[x], g);
                if (a.c) g += load_any(a.c, a.g_dtype, e * a.stride_c + i * a.ld_c + j);
                store_any(a.g, a.g_dtype, e * a.stride_g + i * a.ld_g + j, g);
            }
    }
}

}  // namespace

size_t weight_grad_workspace(const muon_weight_grad_args&) { return 0; }

cudaError_t launch_weight_grad(const muon_weight_grad_args& a, void*, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(ceil_div(a.k, TILE)),
                    static_cast<unsigned>(ceil_div(a.n, TILE)),
                    static_cast<unsigned>(a.experts < 1024 ? a.experts : 1024));
    weight_grad_kernel<<<grid, THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ops
}  // namespace muon
