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
// instructions, and at 15 an element they, not memory, would bound bf16 rows
// (with 8 they still do without a residual: 16384 x 7168 in 90 us, 70 by the
// bytes; with one 108 us, 6.5 TB/s).  p is therefore a multiple of 2^-16 (the nearest), and the scale is that of
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
    uint64_t offset;
    uint32_t key[2][10];           // the rounds'
    uint32_t limit;                // numbers below it drop their element; times 2^16,
    int32_t all;                   // or all are dropped
    float scale;
};

// The eight numbers of a block, two a word, the low half first.
__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t offset, const DropLaunch& p) {
    uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32);
    uint32_t c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ p.key[0][r];
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ p.key[1][r];
        c3 = uint32_t(a);
    }
    // (no number is as large as the limit of all)
    return p.all ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(c0, c1, c2, c3);
}

// A high half is compared in its place, with what is below it: that decides
// nothing.
__device__ __forceinline__ bool kept(const uint4& z, int i, uint32_t limit) {
    const uint32_t w[4] = {z.x, z.y, z.z, z.w};
    return (i & 1 ? w[i / 2] : w[i / 2] << 16) >= limit;
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
// U: blocks a thread takes, whose loads are all out before the first numbers
// are made.
template <typename T, bool RES, int U>
__global__ void __launch_bounds__(256) dropout_vec_kernel(const __grid_constant__ DropLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const uint64_t offset = p.offset + (p.counter ? static_cast<uint64_t>(*p.counter) : 0u);
    const int64_t per_row = (p.cols + 7) / 8;
    const int64_t first = blockIdx.x * int64_t(256 * U) + threadIdx.x;
    Eight<T> x[U], r[U];
    int64_t row[U], col[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t b = first + 256 * k;
        row[k] = p.rows == 1 ? 0 : b / per_row;
        col[k] = (b - row[k] * per_row) * 8;
        if (p.n - b * 8 >= 8) {
            x[k].load(static_cast<const T*>(p.x) + row[k] * p.ld_x + col[k]);
            if (RES) r[k].load(static_cast<const T*>(p.r) + row[k] * p.ld_r + col[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t b = first + 256 * k, left = p.n - b * 8;
        if (left <= 0) return;
        const uint4 z = philox(b, offset, p);
        if (left < 8) {
            for (int i = 0; i < left; ++i) one<T>(p, z, i, row[k], col[k] + i);
            return;
        }
        float f[8], g[8];
        x[k].get(f);
        if (RES) r[k].get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = RES ? g[i] : 0.f;
            f[i] = kept(z, i, p.limit) ? __fmaf_rn(f[i], p.scale, o) : o;
        }
        Eight<T>::put(static_cast<T*>(p.y) + row[k] * p.ld_y + col[k], f);
    }
}

// Any rows: a block's elements one by one, also over the ends of rows.
template <typename T>
__global__ void __launch_bounds__(256) dropout_any_kernel(const __grid_constant__ DropLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const uint64_t offset = p.offset + (p.counter ? static_cast<uint64_t>(*p.counter) : 0u);
    const int64_t b = blockIdx.x * int64_t(256) + threadIdx.x;
    if (b * 8 >= p.n) return;
    const uint4 z = philox(b, offset, p);
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
    // two blocks a thread where that leaves every SM two blocks of threads
    // (16384 x 7168 bf16: 90 us, with a residual 108; one a thread 99 and 115,
    // four 92 and 110)
    const int64_t blocks = ceil_div(ceil_div(p.n, 8), 256);
    const int u = vec && blocks >= 2 * 2 * 152 ? 2 : 1;
    const int64_t grid = ceil_div(blocks, u);
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    void (*const kernel)(DropLaunch) =
        !vec     ? dropout_any_kernel<T>
        : u == 2 ? (p.r ? dropout_vec_kernel<T, true, 2> : dropout_vec_kernel<T, false, 2>)
                 : (p.r ? dropout_vec_kernel<T, true, 1> : dropout_vec_kernel<T, false, 1>);
    return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p);
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
    p.offset = a.offset;
    for (uint32_t i = 0; i < 10; ++i) {
        p.key[0][i] = static_cast<uint32_t>(a.seed) + i * 0x9E3779B9u;
        p.key[1][i] = static_cast<uint32_t>(a.seed >> 32) + i * 0xBB67AE85u;
    }
    const uint32_t limit = static_cast<uint32_t>(a.p * 65536.0 + 0.5);
    p.all = limit == 65536u;
    p.limit = p.all ? 0xffffffffu : limit << 16;
    p.scale = p.all ? 0.f : static_cast<float>(65536.0 / (65536.0 - limit));
    return a.x_dtype == MUON_F32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}

}  // namespace ops
}  // namespace muon
