// Layer norm over rows, forward and backward (muon_layer_norm,
// muon_layer_norm_grad).
//
// Forward.  A row is read once, in 16-byte vectors (at any alignment: see
// Vec) that stay in registers, by a warp (up to 128 vectors) or a block.  The variance is taken around the
// mean in a second sum over the registers (sums of x^2 lose it when the mean
// is large), with the first sum's rounding corrected by the sum of the
// deviations.  The checkpoint of h is written from the same registers.
//
// Backward.  Blocks stay for many rows, so that the column sums of dweight
// and dbias collect in registers: a thread has the same columns in every row.
// Each block leaves one row of partial sums, which a second kernel adds up in
// order.
#include "ops_internal.h"
#include "tc_ptx.cuh"

namespace muon {
namespace ops {
namespace {

constexpr int SMS = 152;
__device__ int g_norm_err;             // DEV_ERR_TIMEOUT once a bounded wait ran out

// Sums of two values over a row's threads, in a fixed order, returned to all
// of them: a warp, or a block (buf alternates between two, so that one
// barrier a sum is enough).
template <bool WARP>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* buf) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 t = lane < static_cast<int>(blockDim.x >> 5) ? buf[lane] : make_float2(0.f, 0.f);
        a = warp_sum(t.x);
        b = warp_sum(t.y);
    }
    return make_float2(a, b);
}

// ------------------------------------------------------------------ forward

struct NormLaunch {
    muon_layer_norm_args a;
    int32_t w_vec;           // weight and bias allow 16-byte loads
};

// A row in the registers of a warp (WARP; blockDim.y rows a block) or of a
// block: NV vectors a thread.
template <typename T, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
    norm_kernel(const __grid_constant__ NormLaunch p) {
    constexpr int VE = Vec<T>::VE;
    __shared__ float2 red[2][32];
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_args& a = p.a;
    const int64_t r = WARP ? blockIdx.x * int64_t(blockDim.y) + threadIdx.y : int64_t(blockIdx.x);
    if (WARP && r >= a.rows) return;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.f / static_cast<float>(cols);
    const int step = (WARP ? 32 : blockDim.x) * VE;
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    Vec<T> v[NV];
    const int c0 = threadIdx.x * VE;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i].load(x + c0 + i * step, cols - c0 - i * step);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[VE];
        v[i].get(f);
#pragma unroll
        for (int j = 0; j < VE; ++j) s += f[j];
    }
    float mean = row_sum2<WARP>(s, 0.f, red[0]).x * inv_n;
    float d1 = 0.f, d2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int valid = cols - c0 - i * step;
        float f[VE];
        v[i].get(f);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            const float d = j < valid ? f[j] - mean : 0.f;
            d1 += d;
            d2 = fmaf(d, d, d2);
        }
    }
    const float2 t = row_sum2<WARP>(d1, d2, red[1]);
    const float off = t.x * inv_n;
    const float var = fmaxf(fmaf(-off, off, t.y * inv_n), 0.f) + (t.y != t.y ? t.y : 0.f);
    mean += off;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
    T* y = static_cast<T*>(a.y) + r * a.ld_y;
    const int padded = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step, valid = cols - c;
        float h[VE];
        v[i].get(h);
#pragma unroll
        for (int j = 0; j < VE; ++j) h[j] = j < valid ? (h[j] - mean) * rstd : 0.f;
        if (a.saved.q) encode_vec<VE>(a.saved, r, c, c < padded, h);
        if (valid > 0) {
            float w[VE], b[VE];
            load_row_vec<VE>(a.weight, a.w_dtype, p.w_vec, c, valid, 1.f, w);
            load_row_vec<VE>(a.bias, a.w_dtype, p.w_vec, c, valid, 0.f, b);
#pragma unroll
            for (int j = 0; j < VE; ++j) h[j] = fmaf(h[j], w[j], b[j]);
            v[i].set(h);
        }
        v[i].store(y + c, valid, c == 0);
    }
}

// Rows that do not fit a block's registers: three sweeps over the row.
template <typename T>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormLaunch p) {
    __shared__ float2 red[2][32];
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_args& a = p.a;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.f / static_cast<float>(cols);
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    T* y = static_cast<T*>(a.y) + r * a.ld_y;
    float s = 0.f;
    for (int c = threadIdx.x; c < cols; c += 1024) s += to_f32(x[c]);
    float mean = row_sum2<false>(s, 0.f, red[0]).x * inv_n;
    float d1 = 0.f, d2 = 0.f;
    for (int c = threadIdx.x; c < cols; c += 1024) {
        const float d = to_f32(x[c]) - mean;
        d1 += d;
        d2 = fmaf(d, d, d2);
    }
    const float2 t = row_sum2<false>(d1, d2, red[1]);
    const float off = t.x * inv_n;
    const float var = fmaxf(fmaf(-off, off, t.y * inv_n), 0.f) + (t.y != t.y ? t.y : 0.f);
    mean += off;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
    const int padded = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    for (int c = threadIdx.x; c < padded; c += 1024) {
        float h[1] = {c < cols ? (to_f32(x[c]) - mean) * rstd : 0.f};
        if (c < cols) {
            const float w = a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f;
            const float b = a.bias ? load_any(a.bias, a.w_dtype, c) : 0.f;
            from_f32(y + c, fmaf(h[0], w, b));
        }
        if (a.saved.q) encode_vec<1>(a.saved, r, c, true, h);
    }
}

// A row's vectors over threads: a warp up to 4 vectors a lane, then blocks
// with as few vectors a thread as keep them at `best` threads.
struct RowShape {
    bool warp = false;
    int nv = 1, threads = 32;
};
RowShape row_shape(int64_t vectors, int max_nv, int best) {
    RowShape s;
    if (vectors <= 32 * 4) {
        s.warp = true;
        s.nv = vectors <= 32 ? 1 : vectors <= 64 ? 2 : 4;
        return s;
    }
    while (s.nv < max_nv && ceil_div(vectors, s.nv) > best) s.nv *= 2;
    s.threads = static_cast<int>(ceil_div(ceil_div(vectors, s.nv), 32) * 32);
    return s;
}

template <typename T>
cudaError_t norm_forward(NormLaunch& p, cudaStream_t s) {
    p.w_vec = rows_on_16(p.a.weight, 1, 1, 0) && rows_on_16(p.a.bias, 1, 1, 0);
    const unsigned rows = static_cast<unsigned>(p.a.rows);
    const RowShape sh = row_shape(ceil_div(p.a.cols, Vec<T>::VE), 8, 512);
    if (sh.warp) {
        const dim3 grid((rows + 7) / 8), block(32, 8);
        if (sh.nv == 1) return launch_kernel(norm_kernel<T, 1, true>, grid, block, 0, s, p);
        if (sh.nv == 2) return launch_kernel(norm_kernel<T, 2, true>, grid, block, 0, s, p);
        return launch_kernel(norm_kernel<T, 4, true>, grid, block, 0, s, p);
    }
    if (sh.threads > 1024) return launch_kernel(norm_long_kernel<T>, dim3(rows), dim3(1024), 0, s, p);
    const dim3 grid(rows), block(sh.threads);
    if (sh.nv == 1) return launch_kernel(norm_kernel<T, 1, false>, grid, block, 0, s, p);
    if (sh.nv == 2) return launch_kernel(norm_kernel<T, 2, false>, grid, block, 0, s, p);
    if (sh.nv == 4) return launch_kernel(norm_kernel<T, 4, false>, grid, block, 0, s, p);
    return launch_kernel(norm_kernel<T, 8, false>, grid, block, 0, s, p);
}

// ----------------------------------------------------------------- backward

struct GradLaunch {
    muon_layer_norm_grad_args a;
    float* part;             // parts x 2 x cols partial sums of dweight, dbias (or null)
    int32_t w_vec;
    int32_t parts;           // blocks (rows of partial sums)
    int32_t stages;          // rows of the ring in shared memory (norm_grad_ring_kernel)
    uint32_t x_off, stage_bytes;   // of a ring's row: where x (or q) is, and its size
    uint32_t w_bytes;        // the weight's room in shared memory, before the ring
    int64_t ld_part;         // cols rounded up to 4
    unsigned long long wait_limit_ns;
};

// The aligned 16-byte pieces that hold `n` bytes from p.
struct Pieces {
    const char* first;
    uint32_t bytes;
    static __device__ __forceinline__ uint32_t lead(const void* p) {
        return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    }
    __device__ __forceinline__ Pieces(const void* p, uint32_t n)
        : first(static_cast<const char*>(p) - lead(p)), bytes((lead(p) + n + 15u) & ~15u) {}
};

// The partial sums of a block whose threads hold whole columns.
template <int VE, int NV>
__device__ __forceinline__ void store_parts(const GradLaunch& p, int c0, int step,
                                            const float (&dw)[NV * VE], const float (&db)[NV * VE]) {
    const int cols = static_cast<int>(p.a.cols);
    float* w = p.part + int64_t(blockIdx.x) * 2 * p.ld_part;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < VE; j += 4) {
            const int c = c0 + i * step + j;
            if (c >= cols) break;
            const int u = i * VE + j;
            *reinterpret_cast<float4*>(w + c) = make_float4(dw[u], dw[u + 1], dw[u + 2], dw[u + 3]);
            *reinterpret_cast<float4*>(w + p.ld_part + c) =
                make_float4(db[u], db[u + 1], db[u + 2], db[u + 3]);
        }
    }
}

// One vector: dy, h and g = dy * w, from the row's vectors of dy and x (or q
// and its scale).  CKPT: x is the checkpoint's row.
template <typename T, bool CKPT>
struct GradVec {
    static constexpr int VE = Vec<T>::VE;
    float dy[VE], h[VE], g[VE];
    __device__ __forceinline__ void make(const GradLaunch& p, const Vec<T>& dyv, const Vec<T>& xv,
                                         const int8_t* q, uint32_t e, float mean, float rstd,
                                         const void* weight, bool w_vec, int c, int valid) {
        dyv.get(dy);
        if constexpr (CKPT) {
            decode_vec<VE>(q, scale_pow(e), h);
        } else {
            xv.get(h);
#pragma unroll
            for (int j = 0; j < VE; ++j) h[j] = (h[j] - mean) * rstd;
        }
        load_row_vec<VE>(weight, p.a.w_dtype, w_vec, c, valid, 1.f, g);
#pragma unroll
        for (int j = 0; j < VE; ++j) g[j] *= dy[j];
    }
};

// Short rows: a warp has rows of its own (eight warps a block) and reads them
// straight from memory.
template <typename T, int NV, bool CKPT>
__global__ void __launch_bounds__(256) norm_grad_kernel(const __grid_constant__ GradLaunch p) {
    constexpr int VE = Vec<T>::VE;
    extern __shared__ float sums[];               // 2 x cols
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_grad_args& a = p.a;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.f / static_cast<float>(cols);
    constexpr int step = 32 * VE;
    const int c0 = threadIdx.x * VE;
    float dw[NV * VE], db[NV * VE];
#pragma unroll
    for (int i = 0; i < NV * VE; ++i) dw[i] = db[i] = 0.f;
    for (int64_t r = blockIdx.x * 8 + threadIdx.y; r < a.rows; r += gridDim.x * 8) {
        const T* dyp = static_cast<const T*>(a.dy) + r * a.ld_dy;
        Vec<T> dyv[NV], xv[NV];
        uint32_t e[NV];
        const int8_t* q = CKPT ? a.saved.q + r * a.saved.ld_q : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            dyv[i].load(dyp + c, cols - c);
            if constexpr (CKPT) {
                e[i] = c < cols ? a.saved.e[r * a.saved.ld_e + c / CKPT_BLOCK] : 0u;
            } else {
                xv[i].load(static_cast<const T*>(a.x) + r * a.ld_x + c, cols - c);
                e[i] = 0u;
            }
        }
        const float rstd = a.rstd[r];
        const float mean = CKPT ? 0.f : a.mean[r];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c >= cols) break;
            GradVec<T, CKPT> v;
            v.make(p, dyv[i], xv[i], q + c, e[i], mean, rstd, a.weight, p.w_vec, c, cols - c);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                dw[i * VE + j] = fmaf(v.dy[j], v.h[j], dw[i * VE + j]);
                db[i * VE + j] += v.dy[j];
                s0 += v.g[j];
                s1 = fmaf(v.g[j], v.h[j], s1);
            }
        }
        const float2 t = row_sum2<true>(s0, s1, nullptr);
        const float m0 = t.x * inv_n, m1 = t.y * inv_n;
        T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            if (c < cols) {
                GradVec<T, CKPT> v;
                v.make(p, dyv[i], xv[i], q + c, e[i], mean, rstd, a.weight, p.w_vec, c, cols - c);
#pragma unroll
                for (int j = 0; j < VE; ++j) v.g[j] = (v.g[j] - m0 - v.h[j] * m1) * rstd;
                dyv[i].set(v.g);
            }
            dyv[i].store(dx + c, cols - c, c == 0);
        }
    }
    if (!p.part) return;
    // the eight warps' sums, in order
#pragma unroll 1
    for (int w = 0; w < 8; ++w) {
        if (w == static_cast<int>(threadIdx.y)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * step;
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    if (c + j >= cols) break;
                    sums[c + j] = dw[i * VE + j] + (w ? sums[c + j] : 0.f);
                    sums[cols + c + j] = db[i * VE + j] + (w ? sums[cols + c + j] : 0.f);
                }
            }
        }
        __syncthreads();
    }
    float* out = p.part + int64_t(blockIdx.x) * 2 * p.ld_part;
    for (int c = threadIdx.y * 32 + threadIdx.x; c < cols; c += 256) {
        out[c] = sums[c];
        out[p.ld_part + c] = sums[cols + c];
    }
}

// Longer rows, one at a time in a block: dy and x (or q) come through a ring
// of `stages` rows in shared memory, filled by bulk copies of the aligned
// 16-byte pieces that hold a row, so that memory is kept busy whatever the
// registers hold.  With more than one vector a thread, the second sweep takes
// a row from the ring again instead of keeping it in registers.
template <typename T>
constexpr int ring_threads(int nv) { return nv < 4 ? 512 : sizeof(T) == 4 ? 1024 : 512; }
template <typename T, int NV, bool CKPT>
__global__ void __launch_bounds__(ring_threads<T>(NV), NV < 4 ? 2 : 1)
    norm_grad_ring_kernel(const __grid_constant__ GradLaunch p) {
    constexpr int VE = Vec<T>::VE;
    constexpr bool KEEP = NV == 1;
    extern __shared__ __align__(128) uint8_t shared[];
    uint8_t* const ring = shared + p.w_bytes;
    __shared__ float2 red[2][32];
    __shared__ uint64_t full[8];
    __shared__ int abort_flag;
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_grad_args& a = p.a;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.f / static_cast<float>(cols);
    const int step = blockDim.x * VE;
    const int c0 = threadIdx.x * VE;
    const int stages = p.stages;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // the weight, which every row needs twice (the ring leaves L1 no room)
    const void* w_row = a.weight ? shared : nullptr;
    if (a.weight)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            if (a.w_dtype == MUON_F32)
                reinterpret_cast<float*>(shared)[c] = static_cast<const float*>(a.weight)[c];
            else
                reinterpret_cast<__nv_bfloat16*>(shared)[c] =
                    static_cast<const __nv_bfloat16*>(a.weight)[c];
        }
    __syncthreads();
    const T* dy0 = static_cast<const T*>(a.dy);
    const T* x0 = static_cast<const T*>(a.x);
    auto load = [&](int64_t r, int s) {
        if (r >= a.rows) return;
        const uint32_t bar = ptx::smem_u32(&full[s]);
        const uint32_t dst = ptx::smem_u32(ring) + s * p.stage_bytes;
        const Pieces dy(dy0 + r * a.ld_dy, cols * sizeof(T));
        const Pieces x = CKPT ? Pieces(a.saved.q + r * a.saved.ld_q, cols)
                              : Pieces(x0 + r * a.ld_x, cols * sizeof(T));
        ptx::mbar_expect_tx(bar, dy.bytes + x.bytes);
        bulk_load(dst, dy.first, dy.bytes, bar);
        bulk_load(dst + p.x_off, x.first, x.bytes, bar);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < stages; ++s) load(blockIdx.x + int64_t(s) * gridDim.x, s);
    float dw[NV * VE], db[NV * VE];
#pragma unroll
    for (int i = 0; i < NV * VE; ++i) dw[i] = db[i] = 0.f;
    int odd = 0, stage = 0;
    uint32_t phase = 0;
    uint32_t e_next[NV];
    float rstd_next = 0.f, mean_next = 0.f;
    auto fetch = [&](int64_t r) {
        if (r >= a.rows) return;
        rstd_next = a.rstd[r];
        if constexpr (CKPT) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (c0 + i * step < cols)
                    e_next[i] = a.saved.e[r * a.saved.ld_e + (c0 + i * step) / CKPT_BLOCK];
        } else {
            mean_next = a.mean[r];
        }
    };
    fetch(blockIdx.x);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, odd ^= 1) {
        const float rstd = rstd_next, mean = mean_next;
        uint32_t e[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) e[i] = CKPT ? e_next[i] : 0u;
        fetch(r + gridDim.x);
        // a wait that runs out raises the flag, which ends the later ones at
        // once; the rows that follow hold nothing of use then
        ptx::wait_bounded(ptx::smem_u32(&full[stage]), phase, &abort_flag, &g_norm_err,
                          p.wait_limit_ns);
        const uint8_t* at = ring + stage * p.stage_bytes;
        const T* dy_row = reinterpret_cast<const T*>(at + Pieces::lead(dy0 + r * a.ld_dy));
        const T* x_row = reinterpret_cast<const T*>(at + p.x_off + (CKPT ? 0 : Pieces::lead(x0 + r * a.ld_x)));
        const int8_t* q_row = reinterpret_cast<const int8_t*>(at + p.x_off);
        auto vec = [&](int i, GradVec<T, CKPT>& v) {
            const int c = c0 + i * step;
            Vec<T> dyv, xv;
            dyv.load(dy_row + c, cols - c);
            if constexpr (!CKPT) xv.load(x_row + c, cols - c);
            v.make(p, dyv, xv, q_row + c, e[i], mean, rstd, w_row, true, c, VE);
        };
        GradVec<T, CKPT> kept;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (c0 + i * step >= cols) break;
            GradVec<T, CKPT> v;
            vec(i, v);
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                dw[i * VE + j] = fmaf(v.dy[j], v.h[j], dw[i * VE + j]);
                db[i * VE + j] += v.dy[j];
                s0 += v.g[j];
                s1 = fmaf(v.g[j], v.h[j], s1);
            }
            if constexpr (KEEP) kept = v;
        }
        const float2 t = row_sum2<false>(s0, s1, red[odd]);
        // its barrier says that every thread has read the stage
        if (KEEP && threadIdx.x == 0) load(r + int64_t(stages) * gridDim.x, stage);
        const float m0 = t.x * inv_n, m1 = t.y * inv_n;
        T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            Vec<T> out;
            out.raw = make_uint4(0u, 0u, 0u, 0u);
            if (c < cols) {
                GradVec<T, CKPT> v;
                if constexpr (KEEP) v = kept;
                else vec(i, v);
#pragma unroll
                for (int j = 0; j < VE; ++j) v.g[j] = (v.g[j] - m0 - v.h[j] * m1) * rstd;
                out.set(v.g);
            }
            out.store(dx + c, cols - c, c == 0);
        }
        if (!KEEP) {
            __syncthreads();
            if (threadIdx.x == 0) load(r + int64_t(stages) * gridDim.x, stage);
        }
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (p.part) store_parts<VE, NV>(p, c0, step, dw, db);
    __syncthreads();
    if (abort_flag && threadIdx.x == 0) {
        // copies still in flight must land before the block leaves
        const int64_t mine = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x;
        for (int s = 0; s < stages && s < mine; ++s)
            ptx::wait_quiet(ptx::smem_u32(&full[s]),
                            static_cast<uint32_t>((mine - s + stages - 1) / stages - 1) & 1u,
                            p.wait_limit_ns);
    }
}

// The partial sums of 32 columns in a block, 32 of them at a time.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const __grid_constant__ GradLaunch p) {
    __shared__ float red[2][32][33];
    grid_dependency_wait();
    allow_dependent_launch();
    const int cols = static_cast<int>(p.a.cols);
    const int c = blockIdx.x * 32 + threadIdx.x;
    float w = 0.f, b = 0.f;
    if (c < cols)
        for (int i = threadIdx.y; i < p.parts; i += 32) {
            w += p.part[2 * i * p.ld_part + c];
            b += p.part[(2 * i + 1) * p.ld_part + c];
        }
    red[0][threadIdx.y][threadIdx.x] = w;
    red[1][threadIdx.y][threadIdx.x] = b;
    __syncthreads();
    if (threadIdx.y < 2) {
        float s = 0.f;
        for (int i = 0; i < 32; ++i) s += red[threadIdx.y][i][threadIdx.x];
        void* out = threadIdx.y ? p.a.dbias : p.a.dweight;
        if (c < cols && out) store_any(out, p.a.w_dtype, c, s);
    }
}

// Rows that do not fit a block's registers: dx by rows in two sweeps, the
// column sums on their own (before dx, which may be dy).
template <typename T>
__device__ __forceinline__ float long_h(const muon_layer_norm_grad_args& a, int64_t r, int c,
                                        float mean, float rstd) {
    if (a.saved.q) {
        float h[1];
        decode_vec<1>(a.saved.q + r * a.saved.ld_q + c,
                      scale_pow(a.saved.e[r * a.saved.ld_e + c / CKPT_BLOCK]), h);
        return h[0];
    }
    return (to_f32(static_cast<const T*>(a.x)[r * a.ld_x + c]) - mean) * rstd;
}
template <typename T>
__global__ void __launch_bounds__(1024) norm_long_dx_kernel(const __grid_constant__ GradLaunch p) {
    __shared__ float2 red[32];
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_grad_args& a = p.a;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.f / static_cast<float>(cols);
    const int64_t r = blockIdx.x;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
    T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
    const float rstd = a.rstd[r], mean = a.saved.q ? 0.f : a.mean[r];
    float s0 = 0.f, s1 = 0.f;
    for (int c = threadIdx.x; c < cols; c += 1024) {
        const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f);
        s0 += g;
        s1 = fmaf(g, long_h<T>(a, r, c, mean, rstd), s1);
    }
    const float2 t = row_sum2<false>(s0, s1, red);
    const float m0 = t.x * inv_n, m1 = t.y * inv_n;
    for (int c = threadIdx.x; c < cols; c += 1024) {
        const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f);
        from_f32(dx + c, (g - m0 - long_h<T>(a, r, c, mean, rstd) * m1) * rstd);
    }
}
template <typename T>
__global__ void __launch_bounds__(256) norm_long_dw_kernel(const __grid_constant__ GradLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_grad_args& a = p.a;
    const int cols = static_cast<int>(a.cols);
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    float w = 0.f, b = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float dy = to_f32(static_cast<const T*>(a.dy)[r * a.ld_dy + c]);
        b += dy;
        w = fmaf(dy, long_h<T>(a, r, c, a.saved.q ? 0.f : a.mean[r], a.rstd[r]), w);
    }
    float* out = p.part + int64_t(blockIdx.y) * 2 * p.ld_part;
    out[c] = w;
    out[p.ld_part + c] = b;
}

// How a gradient is computed; the same for every alignment.
struct GradPlan {
    RowShape shape;
    int stages = 0;          // > 0: through the ring; 0 and no warp: long rows
    uint32_t x_off = 0, stage_bytes = 0, w_bytes = 0;
    size_t smem = 0;
    int parts = 1;
};
GradPlan grad_plan(const muon_layer_norm_grad_args& a) {
    GradPlan g;
    const int64_t size = a.x_dtype == MUON_F32 ? 4 : 2;
    g.shape = row_shape(ceil_div(a.cols, 16 / size), 4, 512);
    int64_t parts;
    if (g.shape.warp) {
        g.smem = size_t(2) * a.cols * 4;
        parts = ceil_div(a.rows, 8);
        if (parts > SMS * 4) parts = SMS * 4;
    } else {
        // room for a row that starts 14 bytes into its first piece
        const int64_t dy = ceil_div(a.cols * size + 14, 16) * 16;
        const int64_t row = dy + (a.saved.q ? ceil_div(a.cols, 16) * 16 : dy);
        const int most = g.shape.nv < 4 || size == 2 ? 512 : 1024;
        const int per_sm = g.shape.nv < 4 ? 2 : 1;
        // the vectors read whole: room to the end of the last one
        const int64_t w = a.weight ? ceil_div(a.cols, 8) * 8 * (a.w_dtype == MUON_F32 ? 4 : 2) : 0;
        const int64_t w_bytes = ceil_div(w, 128) * 128;
        int64_t stages = ((per_sm == 2 ? 112 : 224) * 1024 - w_bytes) / row;
        if (stages > 8) stages = 8;
        if (g.shape.threads <= most && stages >= 1) {
            g.stages = static_cast<int>(stages);
            g.x_off = static_cast<uint32_t>(dy);
            g.stage_bytes = static_cast<uint32_t>(row);
            g.w_bytes = static_cast<uint32_t>(w_bytes);
            g.smem = size_t(w_bytes) + size_t(row) * stages;
            parts = SMS * per_sm;
        } else {
            parts = 64;
        }
        if (parts > a.rows) parts = a.rows;
    }
    g.parts = static_cast<int>(parts);
    return g;
}

template <void (*KERN)(GradLaunch)>
cudaError_t launch_grad(const GradPlan& g, dim3 block, const GradLaunch& p, cudaStream_t s) {
    if (g.smem > 40 * 1024) {          // with the static arrays, above the default
        static int set[64] = {0};      // the most asked for so far, by device
        int dev = 0;
        cudaGetDevice(&dev);
        const int bytes = static_cast<int>(g.smem);
        if (dev < 0 || dev >= 64 || set[dev] < bytes) {
            const cudaError_t e =
                cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) set[dev] = bytes;
        }
    }
    return launch_kernel(KERN, dim3(g.parts), block, g.smem, s, p);
}

template <typename T, bool CKPT>
cudaError_t grad_rows(const GradPlan& g, const GradLaunch& p, cudaStream_t s) {
    const RowShape& sh = g.shape;
    if (sh.warp) {
        const dim3 block(32, 8);
        if (sh.nv == 1) return launch_grad<norm_grad_kernel<T, 1, CKPT>>(g, block, p, s);
        if (sh.nv == 2) return launch_grad<norm_grad_kernel<T, 2, CKPT>>(g, block, p, s);
        return launch_grad<norm_grad_kernel<T, 4, CKPT>>(g, block, p, s);
    }
    const dim3 block(sh.threads);
    if (sh.nv == 1) return launch_grad<norm_grad_ring_kernel<T, 1, CKPT>>(g, block, p, s);
    if (sh.nv == 2) return launch_grad<norm_grad_ring_kernel<T, 2, CKPT>>(g, block, p, s);
    return launch_grad<norm_grad_ring_kernel<T, 4, CKPT>>(g, block, p, s);
}

template <typename T>
cudaError_t norm_backward(GradLaunch& p, cudaStream_t s) {
    const muon_layer_norm_grad_args& a = p.a;
    const GradPlan g = grad_plan(a);
    const unsigned cols = static_cast<unsigned>(a.cols);
    const bool in_rows = g.shape.warp || g.stages;
    cudaError_t e = cudaSuccess;
    p.parts = g.parts;
    p.stages = g.stages;
    p.x_off = g.x_off;
    p.stage_bytes = g.stage_bytes;
    p.w_bytes = g.w_bytes;
    p.ld_part = ceil_div(a.cols, 4) * 4;
    p.w_vec = rows_on_16(a.weight, 1, 1, 0);
    p.wait_limit_ns = wait_limit_ns();
    if (a.rows == 0) {
        p.parts = 0;
    } else if (in_rows) {
        e = a.saved.q ? grad_rows<T, true>(g, p, s) : grad_rows<T, false>(g, p, s);
    } else if (p.part) {
        e = launch_kernel(norm_long_dw_kernel<T>, dim3((cols + 255) / 256, g.parts), dim3(256), 0, s, p);
    }
    if (e == cudaSuccess && p.part)
        e = launch_kernel(norm_dw_kernel, dim3((cols + 31) / 32), dim3(32, 32), 0, s, p);
    if (e == cudaSuccess && a.rows && !in_rows)
        e = launch_kernel(norm_long_dx_kernel<T>, dim3(static_cast<unsigned>(a.rows)), dim3(1024), 0,
                          s, p);
    return e;
}

}  // namespace

cudaError_t norm_error_word(void** word) { return cudaGetSymbolAddress(word, g_norm_err); }

cudaError_t launch_layer_norm(const muon_layer_norm_args& a, cudaStream_t s) {
    NormLaunch p = {};
    p.a = a;
    return a.x_dtype == MUON_F32 ? norm_forward<float>(p, s) : norm_forward<__nv_bfloat16>(p, s);
}

size_t layer_norm_grad_workspace(const muon_layer_norm_grad_args& a) {
    if (!a.dweight && !a.dbias) return 0;
    const size_t n = size_t(grad_plan(a).parts) * 2 * size_t(ceil_div(a.cols, 4) * 4) * 4;
    return n ? n : 4;        // never NULL: the launch tells by the pointer
}

cudaError_t launch_layer_norm_grad(const muon_layer_norm_grad_args& a, void* ws, cudaStream_t s) {
    GradLaunch p = {};
    p.a = a;
    if (a.dweight || a.dbias) p.part = static_cast<float*>(ws);
    return a.x_dtype == MUON_F32 ? norm_backward<float>(p, s) : norm_backward<__nv_bfloat16>(p, s);
}

}  // namespace ops
}  // namespace muon
