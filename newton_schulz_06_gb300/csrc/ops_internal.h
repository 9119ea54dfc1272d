// What the operators of a block's training step share: device helpers for
// typed loads and stores, the 8-bit checkpoint's code, reductions, and the
// launch functions behind the C entry points (ops_api.cpp).
#pragma once

#include "../../include/muon.h"
#include "muon_internal.h"

namespace muon {
namespace ops {

constexpr int CKPT_BLOCK = 32;       // values that share one power of two

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Host launch functions.  ws: the workspace of the operator's query.
cudaError_t launch_ckpt8_pack(const void* x, int x_dtype, int64_t rows, int64_t cols,
                              int64_t ld_x, const muon_ckpt8& saved, cudaStream_t s);
cudaError_t launch_ckpt8_unpack(const muon_ckpt8& saved, int64_t rows, int64_t cols, void* x,
                                int x_dtype, int64_t ld_x, cudaStream_t s);
cudaError_t launch_layer_norm(const muon_layer_norm_args& a, cudaStream_t s);
size_t layer_norm_grad_workspace(const muon_layer_norm_grad_args& a);
cudaError_t launch_layer_norm_grad(const muon_layer_norm_grad_args& a, void* ws, cudaStream_t s);
size_t weight_grad_workspace(const muon_weight_grad_args& a);
cudaError_t launch_weight_grad(const muon_weight_grad_args& a, void* ws, cudaStream_t s);
size_t route_workspace(const muon_route_args& a);
cudaError_t launch_route(const muon_route_args& a, void* ws, cudaStream_t s);
cudaError_t launch_route_grad(const muon_route_grad_args& a, cudaStream_t s);
// Waits for the stream; *code: the device error word (DEV_ERR_*), cleared.
cudaError_t ops_status(cudaStream_t s, int* code);

#ifdef __CUDACC__

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Element i of a tensor whose type is known at run time only.
__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
    return dtype == MUON_F32 ? static_cast<const float*>(p)[i]
                             : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float v) {
    if (dtype == MUON_F32) static_cast<float*>(p)[i] = v;
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---- the 8-bit checkpoint's code (muon_ckpt8) ----

// The larger of two magnitudes as bits: sign cleared, so infinities and NaNs
// compare as the largest.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// Scale byte from the largest magnitude's bits: its exponent field (0 below
// 2^-126, 255 for an infinity or a NaN).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) { return top >> 23; }
// 2^(127 - e), by which a block's values are multiplied (then by 64) before
// they are rounded; 0 for e = 255, whose q are written as 0.
__device__ __forceinline__ float scale_inv(uint32_t e) {
    return __uint_as_float(e == 255u ? 0u : e == 254u ? 0x00400000u : (254u - e) << 23);
}
// 2^(e - 127), exact also where it is subnormal; NaN for e = 255.
__device__ __forceinline__ float scale_pow(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
}
// The multiplications by powers of two are exact (the first brings the block
// into [-2, 2]), so this rounds once.
__device__ __forceinline__ int encode_q(float v, uint32_t e, float inv) {
    if (e == 255u) return 0;
    const int q = __float2int_rn(v * inv * 64.f);
    return max(-127, min(127, q));
}

#endif  // __CUDACC__

}  // namespace ops
}  // namespace muon
