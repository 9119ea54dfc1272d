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
size_t gated_ffn_workspace(const muon_gated_ffn_args& a);
cudaError_t launch_gated_ffn(const muon_gated_ffn_args& a, void* ws, cudaStream_t s);
size_t gated_ffn_grad_workspace(const muon_gated_ffn_grad_args& a);
cudaError_t launch_gated_ffn_grad(const muon_gated_ffn_grad_args& a, void* ws, cudaStream_t s);
cudaError_t launch_rotary(const muon_rotary_args& a, cudaStream_t s);
cudaError_t launch_dropout(const muon_dropout_args& a, cudaStream_t s);
// Waits for the stream; *code: the device error word (DEV_ERR_*), cleared.
cudaError_t ops_status(cudaStream_t s, int* code);
// Device addresses of the layer norm's and the feed-forward block's error words.
cudaError_t norm_error_word(void** word);
cudaError_t ffn_error_word(void** word);
// Kernels whose wait nothing satisfies: it runs out after the limit.
cudaError_t launch_ring_timeout(unsigned long long limit_ns, cudaStream_t s);
cudaError_t launch_ffn_timeout(unsigned long long limit_ns, cudaStream_t s);
// Limit of the kernels' waits (MUON_WAIT_LIMIT_MS, else two seconds).
unsigned long long wait_limit_ns();

// Whether every row of a tensor starts on 16 bytes.
inline bool rows_on_16(const void* p, size_t size, int64_t rows, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * size % 16 == 0);
}

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

// Copies `bytes` (a multiple of 16, both addresses on 16) of global memory to
// this CTA's shared memory; completion is counted on the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(__cvta_generic_to_global(src))), "r"(bytes), "r"(bar)
        : "memory");
}

// ---- two floats at a time (one instruction on sm_103a, each rounded as
// its scalar form) ----
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
// Two bf16 numbers of a word.
__device__ __forceinline__ float2 bf16x2_f32(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// ---- 16-byte vectors of VE elements at any alignment ----
//
// A row may start anywhere: a vector that does not lie on 16 bytes is put
// together from the two aligned 16-byte pieces that hold it, so that odd
// widths and odd addresses cost two loads instead of VE.  A kernel adds rows up
// in the same order wherever they lie; which kernel takes them may go by the
// alignment and the number of rows (norm_forward).  Every piece that is read holds at least
// one byte of the row.

// The 16 bytes that start m bytes into lo:hi (0 <= m < 16, a multiple of 2).
__device__ __forceinline__ uint4 shift_bytes(uint4 lo, uint4 hi, uint32_t m) {
    uint32_t w[6] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y};
    if (m & 8) {
        w[0] = w[2];
        w[1] = w[3];
        w[2] = w[4];
        w[3] = w[5];
        w[4] = hi.z;
        w[5] = hi.w;
    }
    if (m & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t b = (m & 2) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], b), __funnelshift_r(w[1], w[2], b),
                      __funnelshift_r(w[2], w[3], b), __funnelshift_r(w[3], w[4], b));
}

//
// AL: every row is known to start on 16 bytes and to hold whole vectors.
template <typename T, bool AL>
struct Vec {
    static constexpr int VE = 16 / sizeof(T);
    uint4 raw;
    // The vector at p, of which the row holds `valid` elements (0 or less:
    // none; those past it are 0).  Shared or global memory.
    __device__ __forceinline__ void load(const T* p, int valid) {
        raw = make_uint4(0u, 0u, 0u, 0u);
        if (valid > 0) load_some(p, valid);
    }
    // The same where the row is known to hold some of it.
    __device__ __forceinline__ void load_some(const T* p, int valid) {
        if (AL) {
            raw = *reinterpret_cast<const uint4*>(p);
            return;
        }
        const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - m);
        raw = q[0];
        if (m) {
            const uint4 hi = valid * int(sizeof(T)) > 16 - int(m) ? q[1] : make_uint4(0u, 0u, 0u, 0u);
            raw = shift_bytes(raw, hi, m);
        }
        if (valid < VE) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (sizeof(T) == 4) {
                    if (i >= valid) w[i] = 0u;
                } else {
                    if (2 * i >= valid) w[i] = 0u;
                    else if (2 * i + 1 >= valid) w[i] &= 0xffffu;
                }
            }
        }
    }
    __device__ __forceinline__ void get(float2 (&f)[VE / 2]) const {
        if constexpr (sizeof(T) == 4) {
            f[0] = make_float2(__uint_as_float(raw.x), __uint_as_float(raw.y));
            f[1] = make_float2(__uint_as_float(raw.z), __uint_as_float(raw.w));
        } else {
            f[0] = bf16x2_f32(raw.x);
            f[1] = bf16x2_f32(raw.y);
            f[2] = bf16x2_f32(raw.z);
            f[3] = bf16x2_f32(raw.w);
        }
    }
    __device__ __forceinline__ void set(const float2 (&f)[VE / 2]) {
        if constexpr (sizeof(T) == 4) {
            raw = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y),
                             __float_as_uint(f[1].x), __float_as_uint(f[1].y));
        } else {
            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[i].x, f[i].y);
        }
    }
    // Element i of 16 bytes.
    static __device__ __forceinline__ void put(T* p, const uint4& r, int i) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        if constexpr (sizeof(T) == 4)
            *p = __uint_as_float(w[i & 3]);
        else
            *reinterpret_cast<unsigned short*>(p) =
                static_cast<unsigned short>(w[(i >> 1) & 3] >> (16 * (i & 1)));
    }
    // Stores the vector at p (`valid` elements, as above).  All lanes of the
    // warp call it, a lane's p one vector past the lane's before it unless it
    // starts a row (row_start).  Off 16 bytes a lane stores the aligned piece
    // that its vector begins in, whose first m bytes come from the lane
    // before, and only the pieces at the ends of the warp or the row go out
    // by elements.
    __device__ __forceinline__ void store(T* p, int valid, bool row_start) const {
        if (AL) {
            if (valid > 0) *reinterpret_cast<uint4*>(p) = raw;
            return;
        }
        const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
        if (__all_sync(0xffffffffu, valid <= 0 || (m == 0 && valid >= VE))) {
            if (valid > 0) *reinterpret_cast<uint4*>(p) = raw;
            return;
        }
        const int lane = threadIdx.x & 31;
        uint4 before;
        before.x = __shfl_up_sync(0xffffffffu, raw.x, 1);
        before.y = __shfl_up_sync(0xffffffffu, raw.y, 1);
        before.z = __shfl_up_sync(0xffffffffu, raw.z, 1);
        before.w = __shfl_up_sync(0xffffffffu, raw.w, 1);
        if (valid <= 0) return;
        const int head = (16 - static_cast<int>(m)) / int(sizeof(T));   // elements in the first piece
        const bool alone = lane == 0 || row_start;
        if (m == 0) {
            if (valid >= VE) {
                *reinterpret_cast<uint4*>(p) = raw;
            } else {
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (i < valid) put(p + i, raw, i);
            }
            return;
        }
        if (!alone && valid >= head) {
            *reinterpret_cast<uint4*>(reinterpret_cast<char*>(p) - m) =
                shift_bytes(before, raw, 16 - m);
        } else {
            if (!alone) {
                // the lane before leaves its last elements to this piece
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (i >= head) put(p + i - VE, before, i);
            }
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (i < head && i < valid) put(p + i, raw, i);
        }
        if (lane == 31 || valid <= VE) {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (i >= head && i < valid) put(p + i, raw, i);
        }
    }
};

// VE elements from column c of a vector of either type (fill where p is
// null), of which `valid` are there; vec: p lies on 16 bytes.
template <int VE>
__device__ __forceinline__ void load_row_vec(const void* p, int dtype, bool vec, int c, int valid,
                                             float fill, float2 (&f)[VE / 2]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) f[i] = both(fill);
    } else if (vec && valid >= VE) {
        if (dtype == MUON_F32) {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
#pragma unroll
            for (int i = 0; i < VE / 4; ++i) {
                const float4 a = q[i];
                f[2 * i] = make_float2(a.x, a.y);
                f[2 * i + 1] = make_float2(a.z, a.w);
            }
        } else {
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + c;
            if constexpr (VE == 8) {
                const uint4 t = *reinterpret_cast<const uint4*>(q);
                f[0] = bf16x2_f32(t.x);
                f[1] = bf16x2_f32(t.y);
                f[2 % (VE / 2)] = bf16x2_f32(t.z);
                f[3 % (VE / 2)] = bf16x2_f32(t.w);
            } else {
                const uint2 t = *reinterpret_cast<const uint2*>(q);
                f[0] = bf16x2_f32(t.x);
                f[1] = bf16x2_f32(t.y);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            f[i] = make_float2(2 * i < valid ? load_any(p, dtype, c + 2 * i) : 0.f,
                               2 * i + 1 < valid ? load_any(p, dtype, c + 2 * i + 1) : 0.f);
    }
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
// v 2^(6 - E) rounded to nearest, ties to even, and limited; 0 where e is
// 255 (inv is 0 then, and the limits' fminf and fmaxf pass a NaN by).  The
// multiplications by powers of two are exact (the first brings the block into
// [-2, 2]); adding 1.5 * 2^23 rounds to whole numbers, which the float's low
// byte then holds.
__device__ __forceinline__ uint32_t encode_q(float v, uint32_t e, float inv) {
    const float x = fmaxf(fminf(v * inv * 64.f, 127.f), -127.f);
    return e == 255u ? 0u : __float_as_uint(x + 12582912.f);
}
// The larger of m and |v|; a NaN wins.
__device__ __forceinline__ float max_mag(float m, float v) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(m), "f"(v));
    return r;
}

// VE values from q, whose block's power of two is p (exact).
template <int VE>
__device__ __forceinline__ void decode_vec(const int8_t* q, float p, float2 (&f)[VE / 2]) {
    const float2 s = both(p * 0.015625f);
    uint32_t w[VE / 4];
    if constexpr (VE == 8) {
        const uint2 t = *reinterpret_cast<const uint2*>(q);
        w[0] = t.x ^ 0x80808080u;
        w[VE / 4 - 1] = t.y ^ 0x80808080u;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(q) ^ 0x80808080u;
    }
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
        // a byte b = q + 128 in the last byte of 2^23 is the float 2^23 + b
        const float2 v = make_float2(
            __uint_as_float(__byte_perm(w[i / 2], 0x4B000000u, 0x7540u + 2 * i % 4)),
            __uint_as_float(__byte_perm(w[i / 2], 0x4B000000u, 0x7541u + 2 * i % 4)));
        f[i] = mul2(add2(v, both(-8388736.f)), s);
    }
}
__device__ __forceinline__ float decode_one(const muon_ckpt8& s, int64_t r, int64_t c) {
    return static_cast<float>(s.q[r * s.ld_q + c]) * 0.015625f *
           scale_pow(s.e[r * s.ld_e + c / CKPT_BLOCK]);
}

// Encodes VE consecutive values of a row whose block of 32 lies in 32 / VE
// neighbouring lanes (values past the row's end given as 0), and writes q at
// column c and the block's scale byte; every lane of the warp calls this, and
// those with !write only take part in the maximum.
template <int VE>
__device__ __forceinline__ void encode_vec(const muon_ckpt8& s, int64_t r, int c, bool write,
                                           const float2 (&f)[VE / 2]) {
    float largest = 0.f;
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) largest = max_mag(max_mag(largest, f[i].x), f[i].y);
    uint32_t top = __float_as_uint(largest);
#pragma unroll
    for (int o = 1; o < CKPT_BLOCK / VE; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t e = scale_byte(top);
    // Blocks of ordinary size whose largest value does not round up to 128:
    // one multiplication and addition rounds (see encode_q).  The others go
    // the longer way.
    const bool plain = e - 7u < 248u - 7u && (top & 0x7fffffu) < 0x7f0000u;
    uint32_t w[VE / 4];
    if (__all_sync(0xffffffffu, plain)) {
        const float2 scale = both(__uint_as_float((260u - e) << 23)), magic = both(12582912.f);
#pragma unroll
        for (int i = 0; i < VE / 4; ++i) {
            const float2 a = fma2(f[2 * i], scale, magic), b = fma2(f[2 * i + 1], scale, magic);
            w[i] = __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                               __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
        }
    } else {
        const float inv = scale_inv(e);
#pragma unroll
        for (int i = 0; i < VE / 4; ++i)
            w[i] = __byte_perm(
                __byte_perm(encode_q(f[2 * i].x, e, inv), encode_q(f[2 * i].y, e, inv), 0x0040),
                __byte_perm(encode_q(f[2 * i + 1].x, e, inv), encode_q(f[2 * i + 1].y, e, inv), 0x0040),
                0x5410);
    }
    if (!write) return;
    int8_t* q = s.q + r * s.ld_q + c;
    if constexpr (VE == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[VE / 4 - 1]);
    else *reinterpret_cast<uint32_t*>(q) = w[0];
    if ((c & (CKPT_BLOCK - 1)) == 0) s.e[r * s.ld_e + c / CKPT_BLOCK] = static_cast<uint8_t>(e);
}

#endif  // __CUDACC__

}  // namespace ops
}  // namespace muon
