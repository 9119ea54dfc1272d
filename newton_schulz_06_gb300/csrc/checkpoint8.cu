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

// One thread per block of 32.
template <typename T>
__global__ void __launch_bounds__(THREADS)
    pack_kernel(const T* x, int64_t rows, int64_t cols, int64_t ld_x, muon_ckpt8 out) {
    const int64_t nb = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK;
    const int64_t total = rows * nb;
    for (int64_t i = blockIdx.x * int64_t(THREADS) + threadIdx.x; i < total;
         i += int64_t(gridDim.x) * THREADS) {
        const int64_t r = i / nb, b = i % nb;
        const int64_t c0 = b * CKPT_BLOCK;
        const T* src = x + r * ld_x + c0;
        float v[CKPT_BLOCK];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < CKPT_BLOCK; ++j) {
            v[j] = c0 + j < cols ? to_f32(src[j]) : 0.f;
            top = max(top, mag_bits(v[j]));
        }
        const uint32_t e = scale_byte(top);
        const float inv = scale_inv(e);
        int8_t* q = out.q + r * out.ld_q + c0;
#pragma unroll
        for (int j = 0; j < CKPT_BLOCK; ++j) q[j] = static_cast<int8_t>(encode_q(v[j], e, inv));
        out.e[r * out.ld_e + b] = static_cast<uint8_t>(e);
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
    unpack_kernel(muon_ckpt8 in, int64_t rows, int64_t cols, T* x, int64_t ld_x) {
    const int64_t total = rows * cols;
    for (int64_t i = blockIdx.x * int64_t(THREADS) + threadIdx.x; i < total;
         i += int64_t(gridDim.x) * THREADS) {
        const int64_t r = i / cols, c = i % cols;
        const float p = scale_pow(in.e[r * in.ld_e + c / CKPT_BLOCK]);
        from_f32(x + r * ld_x + c, static_cast<float>(in.q[r * in.ld_q + c]) * 0.015625f * p);
    }
}

int grid_for(int64_t items) {
    const int64_t g = ceil_div(items, THREADS);
    return static_cast<int>(g < 1 ? 1 : g > 152 * 32 ? 152 * 32 : g);
}

}  // namespace

cudaError_t launch_ckpt8_pack(const void* x, int x_dtype, int64_t rows, int64_t cols,
                              int64_t ld_x, const muon_ckpt8& saved, cudaStream_t s) {
    const int g = grid_for(rows * ceil_div(cols, CKPT_BLOCK));
    if (x_dtype == MUON_F32)
        pack_kernel<<<g, THREADS, 0, s>>>(static_cast<const float*>(x), rows, cols, ld_x, saved);
    else
        pack_kernel<<<g, THREADS, 0, s>>>(static_cast<const __nv_bfloat16*>(x), rows, cols, ld_x,
                                          saved);
    return cudaGetLastError();
}

cudaError_t launch_ckpt8_unpack(const muon_ckpt8& saved, int64_t rows, int64_t cols, void* x,
                                int x_dtype, int64_t ld_x, cudaStream_t s) {
    const int g = grid_for(rows * cols);
    if (x_dtype == MUON_F32)
        unpack_kernel<<<g, THREADS, 0, s>>>(saved, rows, cols, static_cast<float*>(x), ld_x);
    else
        unpack_kernel<<<g, THREADS, 0, s>>>(saved, rows, cols, static_cast<__nv_bfloat16*>(x),
                                            ld_x);
    return cudaGetLastError();
}

}  // namespace ops
}  // namespace muon
