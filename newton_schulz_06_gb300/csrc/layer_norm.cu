// Layer norm over rows, forward and backward (muon_layer_norm,
// muon_layer_norm_grad).
//
// The variance is taken around the mean in a second sweep (x^2 sums lose it
// when the mean is large), with the first sum's rounding corrected by the sum
// of the deviations.
#include "ops_internal.h"

namespace muon {
namespace ops {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int GRAD_CTAS = 304;      // rows of partial sums of dweight and dbias

// Sums of two values over the block, in a fixed order, returned to all.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* red) {
    a = warp_sum(a);
    b = warp_sum(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = make_float2(0.f, 0.f);
    for (int w = 0; w < WARPS; ++w) {
        t.x += red[w].x;
        t.y += red[w].y;
    }
    return t;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) norm_kernel(const __grid_constant__ muon_layer_norm_args a) {
    __shared__ float2 red[WARPS];
    const float inv_n = 1.f / static_cast<float>(a.cols);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
        T* y = static_cast<T*>(a.y) + r * a.ld_y;
        float s = 0.f;
        for (int64_t c = threadIdx.x; c < a.cols; c += THREADS) s += to_f32(x[c]);
        float mean = block_sum2(s, 0.f, red).x * inv_n;
        float d1 = 0.f, d2 = 0.f;
        for (int64_t c = threadIdx.x; c < a.cols; c += THREADS) {
            const float d = to_f32(x[c]) - mean;
            d1 += d;
            d2 = fmaf(d, d, d2);
        }
        const float2 t = block_sum2(d1, d2, red);
        const float off = t.x * inv_n;
        const float var = fmaxf(fmaf(-off, off, t.y * inv_n), 0.f);
        mean += off;
        const float rstd = 1.f / sqrtf(var + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        const int64_t padded = a.saved.q ? (a.cols + 31) / 32 * 32 : a.cols;
        // whole warps: a warp's 32 columns are one block of the checkpoint
        for (int64_t c = threadIdx.x; c < (padded + 31) / 32 * 32; c += THREADS) {
            float h = 0.f;
            if (c < a.cols) {
                h = (to_f32(x[c]) - mean) * rstd;
                const float w = a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f;
                const float b = a.bias ? load_any(a.bias, a.w_dtype, c) : 0.f;
                from_f32(y + c, fmaf(h, w, b));
            }
            if (a.saved.q) {
                const uint32_t e = scale_byte(__reduce_max_sync(0xffffffffu, mag_bits(h)));
                a.saved.q[r * a.saved.ld_q + c] = static_cast<int8_t>(encode_q(h, e, scale_inv(e)));
                if ((threadIdx.x & 31) == 0)
                    a.saved.e[r * a.saved.ld_e + c / CKPT_BLOCK] = static_cast<uint8_t>(e);
            }
        }
    }
}

// h of column c of row r, from the checkpoint or from x.
template <typename T>
__device__ __forceinline__ float grad_h(const muon_layer_norm_grad_args& a, int64_t r, int64_t c,
                                        float mean, float rstd) {
    if (a.saved.q)
        return static_cast<float>(a.saved.q[r * a.saved.ld_q + c]) * 0.015625f *
               scale_pow(a.saved.e[r * a.saved.ld_e + c / CKPT_BLOCK]);
    return (to_f32(static_cast<const T*>(a.x)[r * a.ld_x + c]) - mean) * rstd;
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
    norm_dx_kernel(const __grid_constant__ muon_layer_norm_grad_args a) {
    __shared__ float2 red[WARPS];
    const float inv_n = 1.f / static_cast<float>(a.cols);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
        T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
        const float rstd = a.rstd[r];
        const float mean = a.saved.q ? 0.f : a.mean[r];
        float s0 = 0.f, s1 = 0.f;
        for (int64_t c = threadIdx.x; c < a.cols; c += THREADS) {
            const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f);
            s0 += g;
            s1 = fmaf(g, grad_h<T>(a, r, c, mean, rstd), s1);
        }
        const float2 t = block_sum2(s0, s1, red);
        const float m0 = t.x * inv_n, m1 = t.y * inv_n;
        for (int64_t c = threadIdx.x; c < a.cols; c += THREADS) {
            const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f);
            from_f32(dx + c, (g - m0 - grad_h<T>(a, r, c, mean, rstd) * m1) * rstd);
        }
    }
}

// Partial column sums: block (x, y) takes columns 256 x .. and every y-th row.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    norm_dw_partial_kernel(const __grid_constant__ muon_layer_norm_grad_args a, float* part) {
    const int64_t c = blockIdx.x * int64_t(THREADS) + threadIdx.x;
    if (c >= a.cols) return;
    float w = 0.f, b = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float dy = to_f32(static_cast<const T*>(a.dy)[r * a.ld_dy + c]);
        const float mean = a.saved.q ? 0.f : a.mean[r];
        b += dy;
        w = fmaf(dy, grad_h<T>(a, r, c, mean, a.rstd[r]), w);
    }
    part[int64_t(2 * blockIdx.y) * a.cols + c] = w;
    part[int64_t(2 * blockIdx.y + 1) * a.cols + c] = b;
}

__global__ void __launch_bounds__(THREADS)
    norm_dw_kernel(const __grid_constant__ muon_layer_norm_grad_args a, const float* part, int n) {
    const int64_t c = blockIdx.x * int64_t(THREADS) + threadIdx.x;
    if (c >= a.cols) return;
    float w = 0.f, b = 0.f;
    for (int i = 0; i < n; ++i) {
        w += part[int64_t(2 * i) * a.cols + c];
        b += part[int64_t(2 * i + 1) * a.cols + c];
    }
    if (a.dweight) store_any(a.dweight, a.w_dtype, c, w);
    if (a.dbias) store_any(a.dbias, a.w_dtype, c, b);
}

int row_grid(int64_t rows) { return static_cast<int>(rows < 152 * 16 ? rows : 152 * 16); }
int grad_parts(int64_t rows) { return static_cast<int>(rows < GRAD_CTAS ? rows : GRAD_CTAS); }

template <typename T>
cudaError_t norm_grad(const muon_layer_norm_grad_args& a, float* part, cudaStream_t s) {
    const int cols = static_cast<int>(ceil_div(a.cols, THREADS));
    if (a.dweight || a.dbias) {
        if (a.rows)
            norm_dw_partial_kernel<T><<<dim3(cols, grad_parts(a.rows)), THREADS, 0, s>>>(a, part);
        norm_dw_kernel<<<cols, THREADS, 0, s>>>(a, part, grad_parts(a.rows));
    }
    // after the sums: dx may be dy
    if (a.rows) norm_dx_kernel<T><<<row_grid(a.rows), THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const muon_layer_norm_args& a, cudaStream_t s) {
    if (a.x_dtype == MUON_F32) norm_kernel<float><<<row_grid(a.rows), THREADS, 0, s>>>(a);
    else norm_kernel<__nv_bfloat16><<<row_grid(a.rows), THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

size_t layer_norm_grad_workspace(const muon_layer_norm_grad_args& a) {
    return (a.dweight || a.dbias) ? size_t(grad_parts(a.rows)) * 2 * size_t(a.cols) * 4 : 0;
}

cudaError_t launch_layer_norm_grad(const muon_layer_norm_grad_args& a, void* ws, cudaStream_t s) {
    return a.x_dtype == MUON_F32 ? norm_grad<float>(a, static_cast<float*>(ws), s)
                                 : norm_grad<__nv_bfloat16>(a, static_cast<float*>(ws), s);
}

}  // namespace ops
}  // namespace muon
