// Dropout whose mask is never stored (muon_dropout): y = residual + keep x scale.
//
// Whether element i = row * cols + col is kept is a 16-bit number of a
// counter-based generator, Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): its block i / 8, under
// the counter (i / 8, offset) and the key seed, has eight of them.  The
// backward pass makes the same numbers again.  They go by the element's place,
// not by the memory layout, the grid or the type.
//
// Sixteen bits an element, not 32: a block of ten rounds costs about 60
// instructions, and at 15 an element they, not memory, would bound bf16 rows.
// p is therefore a multiple of 2^-16 (the nearest), and the scale is that of
// the multiple, so that the mean of y is that of x.
#include "ops_internal.h"

namespace muon {
namespace ops {
namespace {

struct DropLaunch {
    const void *x, *r;
    void* y;
    int64_t rows, cols, ld_x, ld_r, ld_y;
    int64_t n;                     // elements
    const int64_t* counter;        // added to the offset, or null
    uint64_t seed, offset;
    uint32_t limit;                // numbers below it drop their element
    float scale;
};

// The eight numbers of a block, two a word, the low half first.
__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
    uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32);
    uint32_t c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ k0;
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ k1;
        c3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ bool kept(const uint4& z, int i, uint32_t limit) {
    const uint32_t w[4] = {z.x, z.y, z.z, z.w};
    return (i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu) >= limit;
}

// Eight neighbouring elements on 16 bytes.
template <typename T>
struct Eight {
    uint4 raw[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T) / 2); ++i) raw[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = sizeof(T) == 4 ? __uint_as_float(w[i % (2 * sizeof(T))])
                                  : __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    static __device__ __forceinline__ void put(T* p, const float (&f)[8]) {
        if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
            __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
        } else {
            uint4 q;
            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            __stcs(reinterpret_cast<uint4*>(p), q);
        }
    }
};

// One element.  A dropped one is 0 whatever x holds there.
template <typename T>
__device__ __forceinline__ void one(const DropLaunch& p, const uint4& z, int i, int64_t row, int64_t col) {
    const float x = to_f32(static_cast<const T*>(p.x)[row * p.ld_x + col]);
    const float r = p.r ? to_f32(static_cast<const T*>(p.r)[row * p.ld_r + col]) : 0.f;
    from_f32(static_cast<T*>(p.y) + row * p.ld_y + col, kept(z, i, p.limit) ? __fmaf_rn(x, p.scale, r) : r);
}

// Blocks whose eight elements are neighbours on 16 bytes: rows of a multiple
// of eight, or dense tensors taken as one row (whose last block may be short).
template <typename T, bool RES>
__global__ void __launch_bounds__(256) dropout_vec_kernel(const __grid_constant__ DropLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const uint64_t offset = p.offset + (p.counter ? static_cast<uint64_t>(*p.counter) : 0u);
    const int64_t blocks = (p.n + 7) / 8;
    const int64_t per_row = (p.cols + 7) / 8;
    const int64_t b = blockIdx.x * int64_t(256) + threadIdx.x;
    if (b >= blocks) return;
    const int64_t row = p.rows == 1 ? 0 : b / per_row, col = (b - row * per_row) * 8;
    if (p.n - b * 8 < 8) {
        const uint4 z = philox(b, offset, p.seed);
        for (int i = 0; i < p.n - b * 8; ++i) one<T>(p, z, i, row, col + i);
        return;
    }
    Eight<T> x, r;
    x.load(static_cast<const T*>(p.x) + row * p.ld_x + col);
    if (RES) r.load(static_cast<const T*>(p.r) + row * p.ld_r + col);
    const uint4 z = philox(b, offset, p.seed);
    float f[8], g[8];
    x.get(f);
    if (RES) r.get(g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float b = RES ? g[i] : 0.f;
        f[i] = kept(z, i, p.limit) ? __fmaf_rn(f[i], p.scale, b) : b;
    }
    Eight<T>::put(static_cast<T*>(p.y) + row * p.ld_y + col, f);
}

// Any rows: a block's elements one by one, also over the ends of rows.
template <typename T>
__global__ void __launch_bounds__(256) dropout_any_kernel(const __grid_constant__ DropLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const uint64_t offset = p.offset + (p.counter ? static_cast<uint64_t>(*p.counter) : 0u);
    const int64_t b = blockIdx.x * int64_t(256) + threadIdx.x;
    if (b * 8 >= p.n) return;
    const uint4 z = philox(b, offset, p.seed);
    int64_t row = b * 8 / p.cols, col = b * 8 - row * p.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (b * 8 + i >= p.n) break;
        one<T>(p, z, i, row, col);
        if (++col == p.cols) {
            col = 0;
            ++row;
        }
    }
}

template <typename T>
cudaError_t launch(DropLaunch p, cudaStream_t s) {
    const bool dense = p.rows == 1 || (p.ld_x == p.cols && p.ld_y == p.cols && (!p.r || p.ld_r == p.cols));
    auto on16 = [&](const void* q, int64_t ld) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && (dense || ld * int64_t(sizeof(T)) % 16 == 0);
    };
    const bool vec = (dense || p.cols % 8 == 0) && on16(p.x, p.ld_x) && on16(p.y, p.ld_y) &&
                     (!p.r || on16(p.r, p.ld_r));
    if (vec && dense) {
        p.rows = 1;
        p.cols = p.n;
    }
    const int64_t blocks = ceil_div(ceil_div(p.n, 8), 256);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    void (*const kernel)(DropLaunch) = !vec  ? dropout_any_kernel<T>
                                       : p.r ? dropout_vec_kernel<T, true>
                                             : dropout_vec_kernel<T, false>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_dropout(const muon_dropout_args& a, cudaStream_t s) {
    DropLaunch p = {};
    p.x = a.x;
    p.r = a.residual;
    p.y = a.y;
    p.rows = a.rows;
    p.cols = a.cols;
    p.ld_x = a.ld_x;
    p.ld_r = a.ld_r;
    p.ld_y = a.ld_y;
    p.n = a.rows * a.cols;
    p.counter = a.counter;
    p.seed = a.seed;
    p.offset = a.offset;
    p.limit = static_cast<uint32_t>(a.p * 65536.0 + 0.5);
    p.scale = p.limit < 65536u ? static_cast<float>(65536.0 / (65536.0 - p.limit)) : 0.f;
    return a.x_dtype == MUON_F32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}

}  // namespace ops
}  // namespace muon
