// Layer norm over rows, forward and backward (muon_layer_norm,
// muon_layer_norm_grad).
//
// Forward.  A row is read once, in 16-byte vectors (at any alignment: see
// Vec) that stay in registers, by 8 to 32 lanes of a warp or by a block.  The
// variance is taken around the mean in a second sum over the registers (sums
// of x^2 lose it when the mean is large), which also corrects the rounding of a
// large mean (settle).  The checkpoint of h is written from
// the same registers.
//
// Backward.  Blocks stay for many rows, so that the column sums of dweight
// and dbias collect in registers: a thread has the same columns in every row.
// Each block leaves one row of partial sums, which a second kernel adds up in
// order.
#include <atomic>

#include "norm_ring.h"
#include "ops_internal.h"
#include "tc_wait.cuh"

namespace muon {
namespace ops {
namespace {

constexpr int SMS = 152;
__device__ int g_norm_err;             // DEV_ERR_TIMEOUT once a bounded wait ran out

// Sums of two values over a block, in a fixed order, returned to all threads;
// buf alternates between two, so that one barrier a sum is enough.  Up to 16
// warps, half the lanes add up one value and half the other, which halves the
// shuffles (they were a quarter of the backward kernel's instructions).
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* buf) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool hi = lane & 16;
    float v = hi ? b : a;
    v += __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    float* flat = reinterpret_cast<float*>(buf);
    if ((lane & 15) == 0) flat[2 * (threadIdx.x >> 5) + (lane >> 4)] = v;
    __syncthreads();
    if (warps <= 16) {
        float t = (lane & 15) < warps ? flat[2 * (lane & 15) + (lane >> 4)] : 0.f;
#pragma unroll
        for (int o = 8; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        return make_float2(__shfl_sync(0xffffffffu, t, 0), __shfl_sync(0xffffffffu, t, 16));
    }
    const float2 t = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(t.x), warp_sum(t.y));
}
__device__ __forceinline__ float block_sum(float a, float2* buf) {
    const int lane = threadIdx.x & 31;
    a = warp_sum(a);
    float* flat = reinterpret_cast<float*>(buf);
    if (lane == 0) flat[threadIdx.x >> 5] = a;
    __syncthreads();
    return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? flat[lane] : 0.f);
}
// The same over the L threads of a row: neighbouring lanes (L = 8, 16, 32),
// or the block (L = 0).
template <int L>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* buf) {
    if constexpr (L == 0) {
        return block_sum2(a, b, buf);
    } else {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        return make_float2(a, b);
    }
}

// The variance of a row from the sums of d = x - mean and of d^2; the mean is
// corrected by that of d where it helps.  That sum carries the rounding of every
// d, about 2e-8 of the deviation, the first sum about 6e-8 of the mean: a mean
// above the deviation gains two or three times its error, a smaller one would
// lose (7168 columns of bf16 about 0: 6e-8 of itself became 1.5e-6).
__device__ __forceinline__ float settle(float& mean, float2 sums, float inv_n) {
    const float off = sums.x * inv_n;
    const float var = fmaxf(fmaf(-off, off, sums.y * inv_n), 0.f) + (sums.y != sums.y ? sums.y : 0.f);
    if (mean * mean > var) mean += off;
    return var;
}

// ------------------------------------------------------------------ forward

struct NormLaunch {
    muon_layer_norm_args a;
    int32_t w_vec;           // weight and bias allow 16-byte loads
    int32_t stages;          // rows of the ring in shared memory (norm_ring_kernel)
    uint32_t stage_bytes;
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

// Waits until the ring's stage is full.  A wait that runs out raises the
// flag.  Every thread reads it behind the barrier that follows, where it can
// no longer change, so that the whole block leaves the loop at the same row:
// a stage whose copy has not landed is never asked for again.
__device__ __forceinline__ void ring_wait(uint64_t* bar, uint32_t phase, volatile int* abort_flag,
                                          unsigned long long limit_ns) {
    wait_soon(ptx::smem_u32(bar), phase, abort_flag, &g_norm_err, limit_ns);
}
// After an abort at the row that `at` stands for: the copies still in flight
// must land before the block leaves.
__device__ __forceinline__ void ring_drain(uint64_t* full, RingAt at, int stages, int64_t rows,
                                           int64_t row, unsigned long long limit_ns) {
    for (int d = 0; ring_in_flight(rows, row, gridDim.x, stages, d); ++d) {
        const RingAt l = ring_ahead(at, stages, d);
        ptx::wait_quiet(ptx::smem_u32(&full[l.stage]), l.phase, limit_ns);
    }
}
constexpr int RING_MAX = 8;
// Threads that a block of the ring kernels may have.
template <typename T>
constexpr int ring_threads(int nv) { return nv == 4 && sizeof(T) == 4 ? 1024 : 512; }
// Blocks of that size an SM holds: 64 registers a thread, 128 with four
// vectors of bf16.
constexpr int ring_blocks(int nv) { return nv < 4 ? 2 : 1; }

// Blocks of 256 lanes that an SM is to hold: the rows in flight count for
// more than a few spilled registers (65536 x 768 bf16: 44 us with 5, 50 with
// 3; 65536 x 2048: 99 with 4, 103 with 3; 65536 x 512: 30 with 6, 34 where the
// compiler takes the registers it likes, 41 with 8).
template <typename T>
constexpr int lane_blocks(int nv) { return nv < 4 ? 6 : nv == 4 ? 5 : sizeof(T) == 2 ? 4 : 2; }

// A row in the registers of L lanes (256 / L rows a block) or of a block
// (L = 0): NV vectors a thread.  Lanes need no barrier and few instructions a
// row, and what bounds them is memory: 65536 x 2048 bf16 99 us (5.4 TB/s),
// 65536 x 768 fp32 68 us (5.9 TB/s).  One block a row is for few rows: 64 x
// 2048 4.4 us, which is the latency of the load and of two sums.
template <typename T, bool AL, int NV, int L>
__global__ void __launch_bounds__(L ? 256 : 1024, L ? lane_blocks<T>(NV) : 1)
    norm_kernel(const __grid_constant__ NormLaunch p) {
    constexpr int VE = Vec<T, AL>::VE, F2 = VE / 2;
    __shared__ float2 red[2][32];
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_args& a = p.a;
    const int64_t r = L ? int64_t(blockIdx.x) * (256 / (L ? L : 1)) + threadIdx.x / (L ? L : 1)
                        : int64_t(blockIdx.x);
    // lanes whose row is not there walk along with nothing in it
    const int cols = !L || r < a.rows ? static_cast<int>(a.cols) : 0;
    const float inv_n = 1.f / static_cast<float>(a.cols);
    const int step = (L ? L : blockDim.x) * VE;
    const int c0 = (L ? threadIdx.x % (L ? L : 1) : threadIdx.x) * VE;
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    Vec<T, AL> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i].load(x + c0 + i * step, cols - c0 - i * step);
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float2 v[F2];
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < F2; ++j) s = add2(s, v[j]);
    }
    float mean = (L ? row_sum2<L>(s.x + s.y, 0.f, nullptr).x : block_sum(s.x + s.y, red[0])) * inv_n;
    float2 d1 = both(0.f), d2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int valid = cols - c0 - i * step;
        if (valid <= 0) break;
        float2 v[F2];
        raw[i].get(v);
#pragma unroll
        for (int j = 0; j < F2; ++j) {
            float2 d = add2(v[j], both(-mean));
            if (!AL) {
                if (2 * j >= valid) d.x = 0.f;
                if (2 * j + 1 >= valid) d.y = 0.f;
            }
            d1 = add2(d1, d);
            d2 = fma2(d, d, d2);
        }
    }
    const float2 t = row_sum2<L>(d1.x + d1.y, d2.x + d2.y, red[1]);
    const float rstd = 1.f / sqrtf(settle(mean, t, inv_n) + a.eps);
    if (c0 == 0 && cols) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
    T* y = static_cast<T*>(a.y) + r * a.ld_y;
    const int padded = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step, valid = cols - c;
        float2 h[F2];
        raw[i].get(h);
#pragma unroll
        for (int j = 0; j < F2; ++j) h[j] = mul2(add2(h[j], both(-mean)), both(rstd));
        if (a.saved.q) {
            // past the row's end the checkpoint holds zeros
#pragma unroll
            for (int j = 0; j < F2; ++j) {
                if (AL ? valid <= 0 : 2 * j >= valid) h[j].x = 0.f;
                if (AL ? valid <= 0 : 2 * j + 1 >= valid) h[j].y = 0.f;
            }
            encode_vec<VE>(a.saved, r, c, c < padded, h);
        }
        if (valid > 0) {
            float2 w[F2], b[F2];
            load_row_vec<VE>(a.weight, a.w_dtype, p.w_vec, c, AL ? VE : valid, 1.f, w);
            load_row_vec<VE>(a.bias, a.w_dtype, p.w_vec, c, AL ? VE : valid, 0.f, b);
#pragma unroll
            for (int j = 0; j < F2; ++j) h[j] = fma2(h[j], w[j], b[j]);
            raw[i].set(h);
        }
        raw[i].store(y + c, valid, c == 0);
    }
}

// Many longer rows: blocks that stay, with the weight and the bias of their
// threads' columns in registers and a ring of rows in shared memory that bulk
// copies fill ahead of them.  8192 x 7168 bf16: 51 us (4.6 TB/s), with the
// checkpoint 69 us; 16384 x 4096 fp32 92 us (5.8 TB/s), with it 110 us.  bf16 is bound by the
// instructions of the two sums (59 % of the issue slots, and what waits for
// their shuffles and barriers).  With one vector a thread instead of two, 8192
// x 7168 takes 75 us; rows off 16 bytes take 95 us (8192 x 7167), for their
// vectors are put together from two.
template <typename T, bool AL, int NV, bool CKPT>
__global__ void __launch_bounds__(ring_threads<T>(NV), ring_blocks(NV))
    norm_ring_kernel(const __grid_constant__ NormLaunch p) {
    constexpr int VE = Vec<T, AL>::VE, F2 = VE / 2;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float2 red[2][32];
    __shared__ uint64_t full[RING_MAX];
    __shared__ volatile int abort_flag;
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_args& a = p.a;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.f / static_cast<float>(cols);
    const int step = blockDim.x * VE;
    const int c0 = threadIdx.x * VE;
    const int stages = p.stages;
    const T* x0 = static_cast<const T*>(a.x);
    auto load = [&](int64_t r, int s) {
        if (r >= a.rows) return;
        const Pieces x(x0 + r * a.ld_x, cols * sizeof(T));
        ptx::mbar_expect_tx(ptx::smem_u32(&full[s]), x.bytes);
        bulk_load(ptx::smem_u32(ring) + s * p.stage_bytes, x.first, x.bytes, ptx::smem_u32(&full[s]));
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int s = 0; s < stages; ++s) load(blockIdx.x + int64_t(s) * gridDim.x, s);
    }
    float2 w[NV][F2], b[NV][F2];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step;
        load_row_vec<VE>(a.weight, a.w_dtype, p.w_vec, c, cols - c, 1.f, w[i]);
        load_row_vec<VE>(a.bias, a.w_dtype, p.w_vec, c, cols - c, 0.f, b[i]);
    }
    const int padded = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    __syncthreads();
    RingAt at{0, 0};
    bool aborted = false;
    T* y = static_cast<T*>(a.y) + blockIdx.x * a.ld_y + c0;
    const int64_t y_step = gridDim.x * a.ld_y;
    int64_t r = blockIdx.x;
    for (; r < a.rows; r += gridDim.x, y += y_step) {
        ring_wait(&full[at.stage], at.phase, &abort_flag, p.wait_limit_ns);
        const T* x = reinterpret_cast<const T*>(ring + at.stage * p.stage_bytes +
                                                (AL ? 0 : Pieces::lead(x0 + r * a.ld_x)));
        float2 v[NV][F2];
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<T, AL> raw;
            const int valid = cols - c0 - i * step;
            if (AL && !CKPT) {
                if (valid <= 0) break;
                raw.load_some(x + c0 + i * step, valid);
            } else {
                raw.load(x + c0 + i * step, valid);
            }
            raw.get(v[i]);
#pragma unroll
            for (int j = 0; j < F2; ++j) s = add2(s, v[i][j]);
        }
        float mean = block_sum(s.x + s.y, red[0]) * inv_n;
        // its barrier says that every thread has read the stage; a later row's
        // wait is behind the next barrier
        if ((aborted = abort_flag)) break;
        if (threadIdx.x == 0) load(r + int64_t(stages) * gridDim.x, at.stage);
        float2 d1 = both(0.f), d2 = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int valid = cols - c0 - i * step;
            if (valid <= 0) break;
#pragma unroll
            for (int j = 0; j < F2; ++j) {
                float2 d = add2(v[i][j], both(-mean));
                if (!AL) {
                    if (2 * j >= valid) d.x = 0.f;
                    if (2 * j + 1 >= valid) d.y = 0.f;
                }
                d1 = add2(d1, d);
                d2 = fma2(d, d, d2);
            }
        }
        const float2 t = block_sum2(d1.x + d1.y, d2.x + d2.y, red[1]);
        const float rstd = 1.f / sqrtf(settle(mean, t, inv_n) + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step, valid = cols - c;
            if (AL && !CKPT && valid <= 0) break;
            float2 h[F2];
#pragma unroll
            for (int j = 0; j < F2; ++j) h[j] = mul2(add2(v[i][j], both(-mean)), both(rstd));
            if constexpr (CKPT) {
                if (padded != cols || valid <= 0) {
                    // past the row's end the checkpoint holds zeros
#pragma unroll
                    for (int j = 0; j < F2; ++j) {
                        if (2 * j >= valid) h[j].x = 0.f;
                        if (2 * j + 1 >= valid) h[j].y = 0.f;
                    }
                }
                encode_vec<VE>(a.saved, r, c, c < padded, h);
            }
#pragma unroll
            for (int j = 0; j < F2; ++j) h[j] = fma2(h[j], w[i][j], b[i][j]);
            Vec<T, AL> out;
            out.set(h);
            out.store(y + i * step, valid, c == 0);
        }
        at = ring_ahead(at, stages, 1);
    }
    if (aborted && threadIdx.x == 0) ring_drain(full, at, stages, a.rows, r, p.wait_limit_ns);
}

// Rows that do not fit a block's registers (more than 65536 columns of bf16,
// 32768 of fp32): three sweeps over the row, of which L2 serves two, element by
// element (1024 x 70000 bf16: 269 us, 1.1 TB/s; 1024 x 40000 fp32 169 us; 1024 x
// 65536 bf16 in registers 87 us).
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
    float mean = block_sum2(s, 0.f, red[0]).x * inv_n;
    float d1 = 0.f, d2 = 0.f;
    for (int c = threadIdx.x; c < cols; c += 1024) {
        const float d = to_f32(x[c]) - mean;
        d1 += d;
        d2 = fmaf(d, d, d2);
    }
    const float2 t = block_sum2(d1, d2, red[1]);
    const float rstd = 1.f / sqrtf(settle(mean, t, inv_n) + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
    const int padded = (cols + CKPT_BLOCK - 1) / CKPT_BLOCK * CKPT_BLOCK;
    for (int c = threadIdx.x; c < padded; c += 1024) {
        const float h = c < cols ? (to_f32(x[c]) - mean) * rstd : 0.f;
        if (c < cols) {
            const float w = a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f;
            const float b = a.bias ? load_any(a.bias, a.w_dtype, c) : 0.f;
            from_f32(y + c, fmaf(h, w, b));
        }
        if (a.saved.q) {
            // a warp's 32 columns are one block
            const uint32_t e = scale_byte(__reduce_max_sync(0xffffffffu, mag_bits(h)));
            a.saved.q[r * a.saved.ld_q + c] = static_cast<int8_t>(encode_q(h, e, scale_inv(e)));
            if ((c & 31) == 0) a.saved.e[r * a.saved.ld_e + c / CKPT_BLOCK] = static_cast<uint8_t>(e);
        }
    }
}

// A row's vectors over threads: lanes of a warp up to most_lanes vectors,
// then blocks with as few vectors a thread as keep them at 512 threads.
struct RowShape {
    int lanes = 0;           // 8, 16 or 32; 0: the block
    int nv = 1, threads = 256;
};
RowShape row_shape(int64_t vectors, int most_lanes, int max_nv) {
    RowShape s;
    if (vectors <= most_lanes) {
        s.lanes = vectors <= 8 ? 8 : vectors <= 16 ? 16 : 32;
        s.nv = vectors <= 32 ? 1 : vectors <= 64 ? 2 : vectors <= 128 ? 4 : vectors <= 256 ? 8 : 16;
        return s;
    }
    while (s.nv < max_nv && ceil_div(vectors, s.nv) > 512) s.nv *= 2;
    s.threads = static_cast<int>(ceil_div(ceil_div(vectors, s.nv), 32) * 32);
    return s;
}

// Vectors up to which a row's lanes of a warp are better than blocks.  Rows
// off 16 bytes: 128 (16384 x 2047 bf16: 60 us by blocks, 91 by lanes).  Rows
// on 16 bytes, of which every SM has two rounds: 256 of bf16 and 512 of fp32
// (65536 x 2048 bf16: 99 us by lanes, 140 by blocks; 16384 x 2048: 31 and 40;
// 65536 x 4096: 268 and 270; 16384 x 2048 fp32: 52 and 62).  Fewer rows are
// done sooner by blocks, which spread a row over more warps: 512 x 2048 bf16
// 4.7 us and 12.3 by lanes, 2048 x 2048 9.5 and 13, 8192 x 2048 23 and 25.
template <typename T, bool AL>
int most_lanes(int64_t rows) {
    return !AL || rows < 64 * SMS ? 128 : sizeof(T) == 4 ? 512 : 256;
}

// The most dynamic shared memory that the ring kernels ask for, of all blocks
// of an SM together.
constexpr int64_t RING_SMEM = 224 * 1024;

// Lets a kernel have its dynamic shared memory.  What is set is the same for
// every size, so that calls from several threads cannot leave less than one
// of them needs.
template <auto KERN>
cudaError_t allow_smem(size_t bytes) {
    if (bytes <= 40 * 1024) return cudaSuccess;   // with the static arrays, below the default
    static std::atomic<bool> done[64];           // by device
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(RING_SMEM));
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <void (*KERN)(NormLaunch)>
cudaError_t launch_norm_ring(int grid, int threads, size_t smem, const NormLaunch& p, cudaStream_t s) {
    const cudaError_t e = allow_smem<KERN>(smem);
    return e != cudaSuccess ? e : launch_kernel(KERN, dim3(grid), dim3(threads), smem, s, p);
}

// Rows for which blocks that stay pay: two a block and more (8192 x 7168 bf16
// 51 us, 74 with a block a row; 16384 x 4096 fp32 92 and 109 us; 2048 x 7168
// 17 and 18 us; below that both are bound by the launch).
template <typename T, bool AL>
cudaError_t norm_forward_ring(NormLaunch& p, cudaStream_t s, bool* done) {
    const RowShape sh = row_shape(ceil_div(p.a.cols, Vec<T, AL>::VE), most_lanes<T, AL>(p.a.rows), 4);
    *done = false;
    if (sh.lanes || sh.threads > ring_threads<T>(sh.nv)) return cudaSuccess;
    int per_sm = sh.nv < 4 ? 1024 / sh.threads : 1;
    if (per_sm > 8) per_sm = 8;
    if (p.a.rows < 2 * SMS * per_sm) return cudaSuccess;
    p.stage_bytes = static_cast<uint32_t>(ceil_div(p.a.cols * int64_t(sizeof(T)) + 14, 16) * 16);
    int64_t stages = (RING_SMEM / per_sm - 2048) / p.stage_bytes;
    p.stages = static_cast<int32_t>(stages > RING_MAX ? RING_MAX : stages);
    if (p.stages < 2) return cudaSuccess;
    p.wait_limit_ns = wait_limit_ns();
    *done = true;
    const size_t smem = size_t(p.stage_bytes) * p.stages;
    const int grid = SMS * per_sm;
    if (p.a.saved.q) {
        if (sh.nv == 1) return launch_norm_ring<norm_ring_kernel<T, AL, 1, true>>(grid, sh.threads, smem, p, s);
        if (sh.nv == 2) return launch_norm_ring<norm_ring_kernel<T, AL, 2, true>>(grid, sh.threads, smem, p, s);
        return launch_norm_ring<norm_ring_kernel<T, AL, 4, true>>(grid, sh.threads, smem, p, s);
    }
    if (sh.nv == 1) return launch_norm_ring<norm_ring_kernel<T, AL, 1, false>>(grid, sh.threads, smem, p, s);
    if (sh.nv == 2) return launch_norm_ring<norm_ring_kernel<T, AL, 2, false>>(grid, sh.threads, smem, p, s);
    return launch_norm_ring<norm_ring_kernel<T, AL, 4, false>>(grid, sh.threads, smem, p, s);
}

template <typename T, bool AL>
cudaError_t norm_forward(NormLaunch& p, cudaStream_t s) {
    bool done;
    const cudaError_t e = norm_forward_ring<T, AL>(p, s, &done);
    if (done || e != cudaSuccess) return e;
    const RowShape sh = row_shape(ceil_div(p.a.cols, Vec<T, AL>::VE), most_lanes<T, AL>(p.a.rows), 8);
    const unsigned rows = static_cast<unsigned>(p.a.rows);
    const dim3 block(sh.threads);
    if (sh.lanes) {
        const dim3 grid((rows + 256 / sh.lanes - 1) / (256 / sh.lanes));
        if (sh.lanes == 8) return launch_kernel(norm_kernel<T, AL, 1, 8>, grid, block, 0, s, p);
        if (sh.lanes == 16) return launch_kernel(norm_kernel<T, AL, 1, 16>, grid, block, 0, s, p);
        if (sh.nv == 1) return launch_kernel(norm_kernel<T, AL, 1, 32>, grid, block, 0, s, p);
        if (sh.nv == 2) return launch_kernel(norm_kernel<T, AL, 2, 32>, grid, block, 0, s, p);
        if constexpr (AL) {
            if (sh.nv == 8) return launch_kernel(norm_kernel<T, AL, 8, 32>, grid, block, 0, s, p);
            if constexpr (sizeof(T) == 4)
                if (sh.nv == 16) return launch_kernel(norm_kernel<T, AL, 16, 32>, grid, block, 0, s, p);
        }
        return launch_kernel(norm_kernel<T, AL, 4, 32>, grid, block, 0, s, p);
    }
    const dim3 grid(rows);
    if (sh.threads > 1024) return launch_kernel(norm_long_kernel<T>, grid, dim3(1024), 0, s, p);
    if (sh.nv == 1) return launch_kernel(norm_kernel<T, AL, 1, 0>, grid, block, 0, s, p);
    if (sh.nv == 2) return launch_kernel(norm_kernel<T, AL, 2, 0>, grid, block, 0, s, p);
    if (sh.nv == 4) return launch_kernel(norm_kernel<T, AL, 4, 0>, grid, block, 0, s, p);
    return launch_kernel(norm_kernel<T, AL, 8, 0>, grid, block, 0, s, p);
}

template <typename T>
cudaError_t norm_forward_t(NormLaunch& p, cudaStream_t s) {
    const muon_layer_norm_args& a = p.a;
    p.w_vec = rows_on_16(a.weight, 1, 1, 0) && rows_on_16(a.bias, 1, 1, 0);
    const bool al = a.cols % Vec<T, true>::VE == 0 && rows_on_16(a.x, sizeof(T), a.rows, a.ld_x) &&
                    rows_on_16(a.y, sizeof(T), a.rows, a.ld_y);
    return al ? norm_forward<T, true>(p, s) : norm_forward<T, false>(p, s);
}

// ----------------------------------------------------------------- backward

struct GradLaunch {
    muon_layer_norm_grad_args a;
    float* part;             // parts x 2 x ld_part partial sums of dweight, dbias (or null)
    int64_t ld_part;         // cols rounded up to 4
    int32_t w_vec;
    int32_t parts;           // blocks (rows of partial sums)
    int32_t stages;          // rows of the ring in shared memory (norm_grad_ring_kernel)
    uint32_t x_off, stage_bytes;   // of a ring's row: where x (or q) is, and its size
    uint32_t w_bytes;        // the weight's room in shared memory, before the ring
    unsigned long long wait_limit_ns;
};

// One vector of a row: dy, h and g = dy * weight (the caller puts the weight
// into g).  CKPT: h comes from q and
// its scale byte e, else from x as the forward pass makes it, (x - mean) * rstd
// (x * rstd - mean * rstd would save an instruction for two values, and loses
// the digits that x and the mean share; minus = -mean).
template <typename T, bool AL, bool CKPT>
struct GradVec {
    static constexpr int VE = Vec<T, AL>::VE, F2 = VE / 2;
    float2 dy[F2], h[F2], g[F2];
    __device__ __forceinline__ void make(const Vec<T, AL>& dyv, const Vec<T, AL>& xv, const int8_t* q,
                                         uint32_t e, float rstd, float minus) {
        dyv.get(dy);
        if constexpr (CKPT) {
            decode_vec<VE>(q, scale_pow(e), h);
        } else {
            xv.get(h);
#pragma unroll
            for (int j = 0; j < F2; ++j) h[j] = mul2(add2(h[j], both(minus)), both(rstd));
        }
        // g holds the weight's vector
#pragma unroll
        for (int j = 0; j < F2; ++j) g[j] = mul2(g[j], dy[j]);
    }
    // The columns' and the row's sums.
    __device__ __forceinline__ void add(float2* dw, float2* db, float2& s0, float2& s1) const {
#pragma unroll
        for (int j = 0; j < F2; ++j) {
            dw[j] = fma2(dy[j], h[j], dw[j]);
            db[j] = add2(db[j], dy[j]);
            s0 = add2(s0, g[j]);
            s1 = fma2(g[j], h[j], s1);
        }
    }
    // rstd (g - m0 - h m1), with m0 and m1 times -rstd in n0 and n1.
    __device__ __forceinline__ void finish(float rstd, float n0, float n1, Vec<T, AL>& out) const {
        float2 d[F2];
#pragma unroll
        for (int j = 0; j < F2; ++j) d[j] = fma2(h[j], both(n1), fma2(g[j], both(rstd), both(n0)));
        out.set(d);
    }
};

// Short rows: L lanes have rows of their own (256 / L a block at a time) and
// read them straight from memory, one row ahead.  What bounds it is how many
// rows are in flight: with the registers for four blocks an SM, which stay for
// all rows, 262144 x 128 of bf16 take 47 us (4.2 TB/s), with three 67 us.
template <typename T, bool AL, int L, bool CKPT>
__global__ void __launch_bounds__(256, 4) norm_grad_kernel(const __grid_constant__ GradLaunch p) {
    constexpr int VE = Vec<T, AL>::VE, F2 = VE / 2, ROWS = 256 / L;
    __shared__ float sums[2][32 * VE];
    grid_dependency_wait();
    allow_dependent_launch();
    const muon_layer_norm_grad_args& a = p.a;
    const int cols = static_cast<int>(a.cols);
    const float inv_n = 1.f / static_cast<float>(cols);
    const int c = (threadIdx.x % L) * VE;
    float2 dw[F2], db[F2];
#pragma unroll
    for (int j = 0; j < F2; ++j) dw[j] = db[j] = both(0.f);
    Vec<T, AL> dyv, xv;
    uint2 q8 = make_uint2(0u, 0u);
    uint32_t e = 0;
    float rstd = 0.f, minus = 0.f;
    auto fetch = [&](int64_t r) {
        const int valid = r < a.rows ? cols - c : 0;
        dyv.load(static_cast<const T*>(a.dy) + r * a.ld_dy + c, valid);
        if constexpr (CKPT) {
            if (valid > 0) {
                const int8_t* q = a.saved.q + r * a.saved.ld_q + c;
                if (VE == 8) q8 = *reinterpret_cast<const uint2*>(q);
                else q8.x = *reinterpret_cast<const uint32_t*>(q);
                e = a.saved.e[r * a.saved.ld_e + c / CKPT_BLOCK];
            }
        } else {
            xv.load(static_cast<const T*>(a.x) + r * a.ld_x + c, valid);
        }
        if (r < a.rows) {
            rstd = a.rstd[r];
            minus = CKPT ? 0.f : -a.mean[r];
        }
    };
    const int64_t stride = int64_t(gridDim.x) * ROWS;
    // a block's lanes walk on together: shuffles ask every lane
    const int64_t last = (a.rows + ROWS - 1) / ROWS * ROWS;
    int64_t r = int64_t(blockIdx.x) * ROWS + threadIdx.x / L;
    fetch(r);
    for (; r < last; r += stride) {
        const int valid = r < a.rows ? cols - c : 0;
        const float rs = rstd;
        GradVec<T, AL, CKPT> v;
        float2 s0 = both(0.f), s1 = both(0.f);
        if (valid > 0) {
            load_row_vec<VE>(a.weight, a.w_dtype, p.w_vec, c, AL ? VE : valid, 1.f, v.g);
            v.make(dyv, xv, reinterpret_cast<const int8_t*>(&q8), e, rstd, minus);
            v.add(dw, db, s0, s1);
        }
        fetch(r + stride);
        const float2 t = row_sum2<L>(s0.x + s0.y, s1.x + s1.y, nullptr);
        Vec<T, AL> out;
        if (valid > 0) v.finish(rs, -t.x * inv_n * rs, -t.y * inv_n * rs, out);
        out.store(static_cast<T*>(a.dx) + r * a.ld_dx + c, valid, c == 0);
    }
    if (!p.part) return;
    // over the warp's rows, then the eight warps' sums, in order
#pragma unroll
    for (int o = L; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < F2; ++j) {
            dw[j].x += __shfl_xor_sync(0xffffffffu, dw[j].x, o);
            dw[j].y += __shfl_xor_sync(0xffffffffu, dw[j].y, o);
            db[j].x += __shfl_xor_sync(0xffffffffu, db[j].x, o);
            db[j].y += __shfl_xor_sync(0xffffffffu, db[j].y, o);
        }
    const int warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int w = 0; w < 8; ++w) {
        if (w == warp && (threadIdx.x & 31) < L) {
#pragma unroll
            for (int j = 0; j < F2; ++j) {
                sums[0][c + 2 * j] = dw[j].x + (w ? sums[0][c + 2 * j] : 0.f);
                sums[0][c + 2 * j + 1] = dw[j].y + (w ? sums[0][c + 2 * j + 1] : 0.f);
                sums[1][c + 2 * j] = db[j].x + (w ? sums[1][c + 2 * j] : 0.f);
                sums[1][c + 2 * j + 1] = db[j].y + (w ? sums[1][c + 2 * j + 1] : 0.f);
            }
        }
        __syncthreads();
    }
    float* out = p.part + int64_t(blockIdx.x) * 2 * p.ld_part;
    if (static_cast<int>(threadIdx.x) < cols) {
        out[threadIdx.x] = sums[0][threadIdx.x];
        out[p.ld_part + threadIdx.x] = sums[1][threadIdx.x];
    }
}

// Longer rows, one at a time in a block: dy and x (or q) come through a ring
// of `stages` rows in shared memory, filled by bulk copies of the aligned
// 16-byte pieces that hold a row, so that memory is kept busy whatever the
// registers hold.  With more than one vector a thread, the second sweep takes
// a row from the ring again instead of keeping it in registers.  8192 x 7168
// bf16: 80 us (4.4 TB/s), from the checkpoint 80 us (3.7 TB/s); 16384 x 4096
// fp32 136 us (5.9 TB/s), from it 103 us.  bf16 is bound by instructions and their latency at
// 64 registers a thread: 896 threads of one vector take 91 us, blocks of
// several rows that share the weight 82, a bf16 weight in shared memory 89;
// rows off 16 bytes 169 us (8192 x 7167).
template <typename T, bool AL, int NV, bool CKPT>
__global__ void __launch_bounds__(ring_threads<T>(NV), ring_blocks(NV))
    norm_grad_ring_kernel(const __grid_constant__ GradLaunch p) {
    constexpr int VE = Vec<T, AL>::VE, F2 = VE / 2;
    constexpr bool KEEP = NV == 1;
    extern __shared__ __align__(128) uint8_t shared[];
    uint8_t* const ring = shared + p.w_bytes;
    __shared__ float2 red[2][32];
    __shared__ uint64_t full[RING_MAX];
    __shared__ volatile int abort_flag[2];   // of even and of odd rows
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
        abort_flag[0] = abort_flag[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // the weight in fp32, which every row needs (the ring leaves L1 no room),
    // with zeros to the end of its last vector; beside bf16 rows in two
    // planes, the first and the last four values of the vectors, so that
    // neighbouring threads read neighbouring 16 bytes
    const int w_vecs = (cols + VE - 1) / VE;
    for (int c = threadIdx.x; c < w_vecs * VE; c += blockDim.x) {
        const int plane = VE == 8 ? c / 4 % 2 : 0;
        reinterpret_cast<float*>(shared)[(plane * w_vecs + c / VE) * 4 + c % 4] =
            c >= cols ? 0.f : a.weight ? load_any(a.weight, a.w_dtype, c) : 1.f;
    }
    auto w_vec = [&](int v, float2 (&w)[F2]) {
#pragma unroll
        for (int h = 0; h < VE / 4; ++h) {
            const float4 f = reinterpret_cast<const float4*>(shared)[h * w_vecs + v];
            w[2 * h] = make_float2(f.x, f.y);
            w[2 * h + 1] = make_float2(f.z, f.w);
        }
    };
    __syncthreads();
    const T* dy0 = static_cast<const T*>(a.dy);
    const T* x0 = static_cast<const T*>(a.x);
    auto load = [&](uint32_t r, int s) {
        if (r >= static_cast<uint32_t>(a.rows)) return;
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
        for (int s = 0; s < stages; ++s) load(blockIdx.x + s * gridDim.x, s);
    float2 dw[NV * F2], db[NV * F2];
#pragma unroll
    for (int i = 0; i < NV * F2; ++i) dw[i] = db[i] = both(0.f);
    int odd = 0;
    RingAt at{0, 0};
    bool aborted = false;
    uint32_t e_next[NV];
    float rstd_next = 0.f, mean_next = 0.f;
    auto fetch = [&](uint32_t row) {
        rstd_next = a.rstd[row];
        if constexpr (CKPT) {
            const uint8_t* at = a.saved.e + row * a.saved.ld_e + c0 / CKPT_BLOCK;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (c0 + i * step < cols) e_next[i] = at[i * (step / CKPT_BLOCK)];
        } else {
            mean_next = a.mean[row];
        }
    };
    // rows are below 2^31, and a block's stride is small
    const uint32_t rows = static_cast<uint32_t>(a.rows);
    uint32_t r = blockIdx.x;
    fetch(r);
    for (; r < rows; r += gridDim.x, odd ^= 1) {
        const float rstd = rstd_next, minus = -mean_next;
        uint32_t e[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) e[i] = CKPT ? e_next[i] : 0u;
        if (r + gridDim.x < rows) fetch(r + gridDim.x);
        ring_wait(&full[at.stage], at.phase, &abort_flag[odd], p.wait_limit_ns);
        const uint8_t* here = ring + at.stage * p.stage_bytes;
        const T* dy_row = reinterpret_cast<const T*>(here + (AL ? 0 : Pieces::lead(dy0 + r * a.ld_dy)));
        const T* x_row = reinterpret_cast<const T*>(
            here + p.x_off + (AL || CKPT ? 0 : Pieces::lead(x0 + r * a.ld_x)));
        const int8_t* q_row = reinterpret_cast<const int8_t*>(here + p.x_off);
        auto vec = [&](int i, GradVec<T, AL, CKPT>& v) {
            const int c = c0 + i * step;
            Vec<T, AL> dyv, xv;
            dyv.load_some(dy_row + c, cols - c);
            if constexpr (!CKPT) xv.load_some(x_row + c, cols - c);
            w_vec(threadIdx.x + i * blockDim.x, v.g);
            v.make(dyv, xv, q_row + c, e[i], rstd, minus);
        };
        GradVec<T, AL, CKPT> kept;
        float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (c0 + i * step >= cols) break;
            GradVec<T, AL, CKPT> v;
            vec(i, v);
            v.add(dw + i * F2, db + i * F2, s0, s1);
            if constexpr (KEEP) kept = v;
        }
        const float2 t = block_sum2(s0.x + s0.y, s1.x + s1.y, red[odd]);
        // its barrier says that every thread has read the stage; a wait that
        // raises this flag again is two barriers on
        if ((aborted = abort_flag[odd])) break;
        if (KEEP && threadIdx.x == 0) load(r + stages * gridDim.x, at.stage);
        const float n0 = -t.x * inv_n * rstd, n1 = -t.y * inv_n * rstd;
        T* const dx = static_cast<T*>(a.dx) + r * a.ld_dx + c0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * step;
            Vec<T, AL> out;
            if (AL && c >= cols) break;
            if (AL || c < cols) {
                if constexpr (KEEP) {
                    kept.finish(rstd, n0, n1, out);
                } else {
                    GradVec<T, AL, CKPT> v;
                    vec(i, v);
                    v.finish(rstd, n0, n1, out);
                }
            }
            out.store(dx + i * step, AL ? VE : cols - c, c == 0);
        }
        if (!KEEP) {
            __syncthreads();
            if (threadIdx.x == 0) load(r + stages * gridDim.x, at.stage);
        }
        at = ring_ahead(at, stages, 1);
    }
    if (p.part) {
        float* w = p.part + int64_t(blockIdx.x) * 2 * p.ld_part;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < F2; j += 2) {
                const int c = c0 + i * step + 2 * j, u = i * F2 + j;
                if (c >= cols) break;
                *reinterpret_cast<float4*>(w + c) = make_float4(dw[u].x, dw[u].y, dw[u + 1].x, dw[u + 1].y);
                *reinterpret_cast<float4*>(w + p.ld_part + c) =
                    make_float4(db[u].x, db[u].y, db[u + 1].x, db[u + 1].y);
            }
    }
    if (aborted && threadIdx.x == 0) ring_drain(full, at, stages, rows, r, p.wait_limit_ns);
}

// The partial sums of 32 columns in a block, 32 of them at a time (304 of 7168
// columns 7 us, 1216 of 768 columns 13 us).
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
    if (a.saved.q) return decode_one(a.saved, r, c);
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
    const float2 t = block_sum2(s0, s1, red);
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
    int stages = 0;          // > 0: through the ring; 0 and no lanes: long rows
    uint32_t x_off = 0, stage_bytes = 0, w_bytes = 0;
    size_t smem = 0;
    int parts = 1;
};
GradPlan grad_plan(const muon_layer_norm_grad_args& a) {
    GradPlan g;
    const int64_t size = a.x_dtype == MUON_F32 ? 4 : 2;
    g.shape = row_shape(ceil_div(a.cols, 16 / size), 32, 4);
    int64_t parts;
    if (g.shape.lanes) {
        parts = ceil_div(a.rows, 256 / g.shape.lanes);
        if (parts > SMS * 4) parts = SMS * 4;
    } else {
        // room for a row that starts 14 bytes into its first piece
        const int64_t dy = ceil_div(a.cols * size + 14, 16) * 16;
        const int64_t row = dy + (a.saved.q ? ceil_div(a.cols, 16) * 16 : dy);
        // the weight's vectors are read whole: room to the end of the last one
        const int64_t w_bytes = ceil_div(a.cols, 32) * 32 * 4;
        const int most = size == 4 ? ring_threads<float>(g.shape.nv) : ring_threads<__nv_bfloat16>(g.shape.nv);
        // blocks an SM: about 1024 threads, of the 64 registers that leaves
        int64_t per_sm = g.shape.nv < 4 ? 1024 / g.shape.threads : 1;
        if (per_sm > 8) per_sm = 8;
        int64_t stages = (RING_SMEM / per_sm - 2048 - w_bytes) / row;
        if (stages > RING_MAX) stages = RING_MAX;
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
    const cudaError_t e = allow_smem<KERN>(g.smem);
    return e != cudaSuccess ? e : launch_kernel(KERN, dim3(g.parts), block, g.smem, s, p);
}

template <typename T, bool AL, bool CKPT>
cudaError_t grad_rows(const GradPlan& g, const GradLaunch& p, cudaStream_t s) {
    const RowShape& sh = g.shape;
    const dim3 block(sh.threads);
    if (sh.lanes == 8) return launch_grad<norm_grad_kernel<T, AL, 8, CKPT>>(g, block, p, s);
    if (sh.lanes == 16) return launch_grad<norm_grad_kernel<T, AL, 16, CKPT>>(g, block, p, s);
    if (sh.lanes == 32) return launch_grad<norm_grad_kernel<T, AL, 32, CKPT>>(g, block, p, s);
    if (sh.nv == 1) return launch_grad<norm_grad_ring_kernel<T, AL, 1, CKPT>>(g, block, p, s);
    if (sh.nv == 2) return launch_grad<norm_grad_ring_kernel<T, AL, 2, CKPT>>(g, block, p, s);
    return launch_grad<norm_grad_ring_kernel<T, AL, 4, CKPT>>(g, block, p, s);
}

template <typename T>
cudaError_t norm_backward(GradLaunch& p, cudaStream_t s) {
    const muon_layer_norm_grad_args& a = p.a;
    const GradPlan g = grad_plan(a);
    const unsigned cols = static_cast<unsigned>(a.cols);
    const bool in_rows = g.shape.lanes || g.stages;
    const bool al = a.cols % Vec<T, true>::VE == 0 && rows_on_16(a.dy, sizeof(T), a.rows, a.ld_dy) &&
                    rows_on_16(a.dx, sizeof(T), a.rows, a.ld_dx) &&
                    (a.saved.q || rows_on_16(a.x, sizeof(T), a.rows, a.ld_x));
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
        if (al) e = a.saved.q ? grad_rows<T, true, true>(g, p, s) : grad_rows<T, true, false>(g, p, s);
        else e = a.saved.q ? grad_rows<T, false, true>(g, p, s) : grad_rows<T, false, false>(g, p, s);
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

// A wait that nothing satisfies, as the rings wait.
__global__ void __launch_bounds__(32) ring_timeout_kernel(unsigned long long limit_ns) {
    __shared__ uint64_t bar;
    __shared__ volatile int abort_flag;
    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_u32(&bar), 1);
        abort_flag = 0;
    }
    __syncthreads();
    ring_wait(&bar, 0, &abort_flag, limit_ns);
}

}  // namespace

cudaError_t launch_ring_timeout(unsigned long long limit_ns, cudaStream_t s) {
    return launch_kernel(ring_timeout_kernel, dim3(1), dim3(32), 0, s, limit_ns);
}

cudaError_t norm_error_word(void** word) { return cudaGetSymbolAddress(word, g_norm_err); }

cudaError_t launch_layer_norm(const muon_layer_norm_args& a, cudaStream_t s) {
    NormLaunch p = {};
    p.a = a;
    return a.x_dtype == MUON_F32 ? norm_forward_t<float>(p, s) : norm_forward_t<__nv_bfloat16>(p, s);
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
