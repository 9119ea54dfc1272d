// Activation checkpoints in 8 bits (muon_ckpt8): blocks of 32 consecutive
// values of a row, value = q * 2^(e - 133).
//
// A power of two as the scale costs up to one bit against max|v| / 127, but
// then q * 2^(e - 133) has at most 7 significant bits and is exact in bf16:
// what reads a checkpoint on the tensor cores rounds nothing again.
#include "ops_internal.h"

namespace muon {
namespace ops {
namespace {

constexpr int THREADS = 256;

// Vector i of rows of `per` vectors: its row and first column.
__device__ __forceinline__ void place(int64_t i, int64_t total, uint32_t per, int ve, int64_t* r, int* c) {
    *r = total <= 0xffffffffll ? static_cast<uint32_t>(i) / per : i / per;
    *c = static_cast<int>(i - *r * per) * ve;
}

// One thread per vector, UNROLL of them in flight.  8192 x 7168 bf16: 35 us,
// 5.1 TB/s of what it reads and writes, fp32 57 us; 7167 columns (vectors put together
// from two) 51 us.
template <typename T, bool AL>
__global__ void __launch_bounds__(THREADS)
    pack_kernel(const T* x, int64_t rows, int64_t cols, int64_t ld_x, muon_ckpt8 out) {
    grid_dependency_wait();
    allow_dependent_launch();
    constexpr int VE = Vec<T, AL>::VE, UNROLL = 4;
    const uint32_t per = static_cast<uint32_t>((cols + CKPT_BLOCK - 1) / CKPT_BLOCK * (CKPT_BLOCK / VE));
    const int64_t total = rows * per;
    const int64_t stride = int64_t(gridDim.x) * THREADS;
    // whole warps walk on together: encode_vec asks every lane
    const int64_t rounded = (total + 31) / 32 * 32;
    for (int64_t i0 = blockIdx.x * int64_t(THREADS) + threadIdx.x; i0 < rounded; i0 += UNROLL * stride) {
        Vec<T, AL> v[UNROLL];
        int64_t r[UNROLL];
        int c[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int64_t i = i0 + u * stride;
            place(i, total, per, VE, &r[u], &c[u]);
            v[u].load(x + r[u] * ld_x + c[u], i < total ? static_cast<int>(cols) - c[u] : 0);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int64_t i = i0 + u * stride;
            if (i >= rounded) break;
            float2 f[VE / 2];
            v[u].get(f);
            encode_vec<VE>(out, r[u], c[u], i < total, f);
        }
    }
}

// The way back: 8192 x 7168 to bf16 34 us, 5.3 TB/s, to fp32 60 us; 7167 columns
// (bf16) 54 us.
template <typename T, bool AL>
__global__ void __launch_bounds__(THREADS)
    unpack_kernel(muon_ckpt8 in, int64_t rows, int64_t cols, T* x, int64_t ld_x) {
    grid_dependency_wait();
    allow_dependent_launch();
    constexpr int VE = Vec<T, AL>::VE;
    const uint32_t per = static_cast<uint32_t>((cols + VE - 1) / VE);
    const int64_t total = rows * per;
    const int64_t rounded = (total + 31) / 32 * 32;
    for (int64_t i = blockIdx.x * int64_t(THREADS) + threadIdx.x; i < rounded;
         i += int64_t(gridDim.x) * THREADS) {
        int64_t r = 0;
        int c = 0;
        Vec<T, AL> v;
        if (i < total) {
            place(i, total, per, VE, &r, &c);
            float2 f[VE / 2];
            decode_vec<VE>(in.q + r * in.ld_q + c, scale_pow(in.e[r * in.ld_e + c / CKPT_BLOCK]), f);
            v.set(f);
        }
        v.store(x + r * ld_x + c, i < total ? static_cast<int>(cols) - c : 0, c == 0);
    }
}

int grid_for(int64_t items) {
    const int64_t g = ceil_div(items, THREADS);
    return static_cast<int>(g < 1 ? 1 : g > 152 * 32 ? 152 * 32 : g);
}

template <typename T>
bool whole(const T* x, int64_t rows, int64_t cols, int64_t ld) {
    return cols % Vec<T, true>::VE == 0 && rows_on_16(x, sizeof(T), rows, ld);
}

template <typename T>
cudaError_t pack(const T* x, int64_t rows, int64_t cols, int64_t ld_x, const muon_ckpt8& saved,
                 cudaStream_t s) {
    const int64_t vectors = rows * ceil_div(cols, CKPT_BLOCK) * (CKPT_BLOCK / Vec<T, true>::VE);
    return launch_kernel(whole(x, rows, cols, ld_x) ? pack_kernel<T, true> : pack_kernel<T, false>,
                         dim3(grid_for(vectors)), dim3(THREADS), 0, s, x, rows, cols, ld_x, saved);
}

template <typename T>
cudaError_t unpack(const muon_ckpt8& saved, int64_t rows, int64_t cols, T* x, int64_t ld_x,
                   cudaStream_t s) {
    return launch_kernel(whole(x, rows, cols, ld_x) ? unpack_kernel<T, true> : unpack_kernel<T, false>,
                         dim3(grid_for(rows * ceil_div(cols, Vec<T, true>::VE))), dim3(THREADS), 0, s,
                         saved, rows, cols, x, ld_x);
}

}  // namespace

cudaError_t launch_ckpt8_pack(const void* x, int x_dtype, int64_t rows, int64_t cols,
                              int64_t ld_x, const muon_ckpt8& saved, cudaStream_t s) {
    return x_dtype == MUON_F32 ? pack(static_cast<const float*>(x), rows, cols, ld_x, saved, s)
                               : pack(static_cast<const __nv_bfloat16*>(x), rows, cols, ld_x, saved, s);
}

cudaError_t launch_ckpt8_unpack(const muon_ckpt8& saved, int64_t rows, int64_t cols, void* x,
                                int x_dtype, int64_t ld_x, cudaStream_t s) {
    return x_dtype == MUON_F32 ? unpack(saved, rows, cols, static_cast<float*>(x), ld_x, s)
                               : unpack(saved, rows, cols, static_cast<__nv_bfloat16*>(x), ld_x, s);
}

}  // namespace ops
}  // namespace muon
