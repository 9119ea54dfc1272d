// The weight gradient of a product from an 8-bit checkpoint
// (muon_weight_grad): G = dY^T X (+ C), one matrix or one per expert.
//
// Both operands have their long axis, the tokens, as rows: dY is tokens x n
// and the checkpoint tokens x k, so the tensor cores read both as MN-major
// operands and no transpose is made.  A CTA pair (tcgen05 cta_group::2)
// computes a 256 x 256 tile of G (or a 512 x 256 one: WIDE), 64 tokens a step:
// each CTA loads its 128 columns of dY (bf16) and of the checkpoint (8 bits)
// with TMA, four warps turn the latter into bf16 in the tensor cores' swizzled
// layout, and the leader issues the products.  A checkpoint's value
// q 2^(e - 133) is exact in bf16, so the operands are exact and the sums fp32;
// the norm's weight and bias act on the sums, in the epilogue:
//     sum_t dy[t][i] (h[t][j] w[j] + b[j]) = w[j] G0[i][j] + b[j] sum_t dy[t][i].
//
// Roles in a CTA: warp 0 loads, warp 1 issues the products (leader only),
// warps 2-9 write tiles out, warps 10-17 decode, in two groups of four that
// take the steps in turn.  Two accumulators in tensor memory, so that a tile
// is written out while the next one's products run; a WIDE tile has both, one
// for each of its halves.  Pairs walk the tiles in turn; how many tokens a
// tile has is read from the offsets on the device, and every role finds the
// same number.
//
// What bounds it is the tensor cores where the tiles are WIDE (16384 tokens,
// 7168 x 8192, bf16: 1040 us, 1.85 PFLOP/s), and else the decoding warps: at
// 4096 tokens and 256 x 256 tiles 345 us, 310 without the products and 274
// without the decoding.  Four warps a group and two groups beat 2 x 8 warps
// and 4 x 4 (69, 90 and 95 us with 512 tokens of 7168 x 8192), and eight warps
// that write out beat four (their stores of 64-byte rows, 94 us with TMA
// stores and 107 with 32-byte ones straight from registers).
//
// Every wait is bounded; one that runs out raises g_ops_err (muon_ops_sync).
#include <cstdlib>

#include <cudaTypedefs.h>

#include "ops_internal.h"
#include "tc_wait.cuh"
#include "weight_grad_stages.h"

namespace muon {
namespace ops {
namespace {

using namespace ptx;

constexpr int W_TOK = 64;                          // tokens a step
constexpr int W_BOX = W_TOK * 64 * 2;              // 64 bf16 columns of a step
constexpr int W_RBOX = W_TOK * 64;                 // 64 columns of a step in 8 bits
constexpr int W_B_BYTES = 2 * W_BOX;
constexpr int W_R_BYTES = 2 * W_RBOX;
constexpr int W_EPI_WARPS = 8;                     // two for 32 rows of the tile
constexpr int W_DEC_WARPS = 4;                     // that decode one step
constexpr int W_DEC_BLOCKS = 8 / W_DEC_WARPS;      // blocks of 32 values a thread decodes
constexpr int W_DEC_WARP0 = 2 + W_EPI_WARPS;
constexpr int W_THREADS = 32 * (W_DEC_WARP0 + W_DEC_GROUPS * W_DEC_WARPS);
constexpr int W_EPI_BYTES = 32 * 64;               // a warp's staged block: 32 rows of 64 bytes
constexpr int W_ORDER = 512;                       // experts that are taken by their size
constexpr int W_TMEM_COLS = 512;
constexpr int W_PAIRS = 76;                        // a pair per two of the 152 SMs
// A tile's 256-row halves and the rings of stages in shared memory.
template <bool WIDE>
struct Shape {
    static constexpr int HALVES = WIDE ? 2 : 1;
    static constexpr int A_STAGES = Stages<WIDE>::A, B_STAGES = Stages<WIDE>::B, R_STAGES = Stages<WIDE>::R;
    static constexpr int AHEAD = Stages<WIDE>::AHEAD;
    static constexpr int A_BYTES = HALVES * 2 * W_BOX;
    static constexpr int B_OFF = A_STAGES * A_BYTES, R_OFF = B_OFF + B_STAGES * W_B_BYTES;
    static constexpr int BAR_OFF = R_OFF + R_STAGES * W_R_BYTES;
    static constexpr int EPI_OFF = BAR_OFF + 1024;
    static constexpr int ORDER_OFF = EPI_OFF + W_EPI_WARPS * W_EPI_BYTES;
    static constexpr int SMEM = ORDER_OFF + W_ORDER * 2 + 1024;
    static_assert(SMEM <= 232448, "shared memory per CTA");
};
constexpr int COLSUM_PARTS = 32;      // of one matrix's tokens (experts: one part each)
constexpr int BAND = 8;
// The tensor cores cut a running sum off at its last place, twice a product of
// 16 tokens, so that it shrinks: sums of one sign by 9e-7 of themselves after 64
// products and by 4e-5 after 1024, sums of both signs by 1.7e-7 after 64
// (measured).  After this many steps of four products a sum is added to one
// that is rounded to nearest.  fp32 results: 16 (4096 tokens of 7168 x 8192: 380
// us, 363 with one sum, whose error is 1.8e-6 instead of 4e-7).  bf16 results,
// whose rounding is 2e-3: 256, or 16384 tokens, so that what is lost stays at a
// fiftieth of that however many there are (65536 tokens of 7168 x 8192: 4242
// us, and 3980 with one sum, which loses 1e-3 of 200000 tokens).
constexpr int CHUNK_F32 = 16, CHUNK_BF16 = 256;

__device__ int g_ops_err;

struct WgLaunch {
    CUtensorMap tm_dy;       // dY: dims {n, rows}, box {64, 64}, 128-byte swizzle
    CUtensorMap tm_q;        // q: dims {k, rows}, box {64, 64}, 64-byte swizzle
    int32_t vec;             // G's and C's rows lie on 16 bytes
    int32_t sorted;          // experts are taken by their size
    int32_t chunk;           // steps that one accumulator sums
    muon_weight_grad_args a;
    const float *weight, *bias;    // a's, or their fp32 copies
    const float* colsum;     // parts x experts x n sums of dY's columns (bias), or null
    int32_t colsum_parts;
    float* part;             // splits > 1: splits x experts x n x ld_part partial sums
    int64_t ld_part;
    int32_t splits;
    float4* held;            // WIDE: a tile's sums while its next chunk runs
    int32_t tiles_n, tiles_k;
    int32_t items;
    unsigned long long wait_limit_ns;
};

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

// One tile of one matrix over one part of its tokens.
struct Item {
    int32_t e, split;
    int32_t n0, k0;          // first row and column of the tile
    int32_t t0, steps;       // first token, steps of 64 tokens
    int32_t end;             // the matrix's tokens end here
};
// order: the experts by their size (or null: as they are).
template <bool WIDE>
__device__ __forceinline__ Item item_at(const WgLaunch& p, const uint16_t* order, int32_t it) {
    const uint32_t per = static_cast<uint32_t>(p.tiles_n) * p.tiles_k;
    const uint32_t es = static_cast<uint32_t>(it) / per;
    const uint32_t w = it - es * per;
    Item x;
    x.e = static_cast<int32_t>(es / p.splits);
    x.split = static_cast<int32_t>(es - uint32_t(x.e) * p.splits);
    // bands of 2048 rows, column by column: the tiles that run together
    // share their rows of dY and of the checkpoint in L2
    constexpr int HIGH = BAND / Shape<WIDE>::HALVES;
    const uint32_t band = w / (HIGH * p.tiles_k);
    const uint32_t high = min(HIGH, p.tiles_n - static_cast<int>(band) * HIGH);
    const uint32_t in = w - band * HIGH * p.tiles_k;
    x.k0 = static_cast<int32_t>(in / high) * 256;
    x.n0 = static_cast<int32_t>(band * HIGH + in % high) * 256 * Shape<WIDE>::HALVES;
    int64_t begin, end;
    if (order) x.e = order[x.e];
    segment(p.a, x.e, &begin, &end);
    const int64_t steps = (end - begin + W_TOK - 1) / W_TOK;
    int64_t s0 = 0, s1 = steps;
    if (p.splits > 1) {
        s0 = steps * x.split / p.splits;
        s1 = steps * (x.split + 1) / p.splits;
    }
    x.t0 = static_cast<int32_t>(begin + s0 * W_TOK);
    x.steps = static_cast<int32_t>(s1 - s0);
    x.end = static_cast<int32_t>(end);
    return x;
}

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_pair_multicast(uint32_t bar) {
    const uint16_t mask = 0x3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster."
        "multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(mask)
        : "memory");
}
__device__ __forceinline__ void commit_pair_local(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}
// Arrive on a barrier of the pair's leader.  What the waiter's products read
// are this CTA's own writes to its shared memory, ordered before the arrival
// by the fence to the async proxy; a release over the whole cluster would
// wait for every load in flight (the decoding warps' scale loads: 4096 tokens
// of 4096 x 2048 took 256 us instead of 116 at the time).
__device__ __forceinline__ void arrive_leader(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// 16 fp32 columns of this warp's TMEM lanes (asked for; there after
// tmem_ld_wait).
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// The way back; complete on return.
__device__ __forceinline__ void tmem_st16(uint32_t to, const uint32_t (&a)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(to),
        "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7]), "r"(a[8]),
        "r"(a[9]), "r"(a[10]), "r"(a[11]), "r"(a[12]), "r"(a[13]), "r"(a[14]), "r"(a[15])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Those at `to` plus those at `from`, to `to`.
__device__ __forceinline__ void tmem_add16(uint32_t to, uint32_t from) {
    uint32_t a[16], b[16];
    tmem_ld16(to, a);
    tmem_ld16(from, b);
    tmem_ld_wait();
#pragma unroll
    for (int u = 0; u < 16; ++u) a[u] = __float_as_uint(__uint_as_float(a[u]) + __uint_as_float(b[u]));
    tmem_st16(to, a);
}

// 16 columns of an accumulator, with the sums that wait in memory for them
// (this lane's pieces lie 32 apart) added if `more`: to memory, or back.
template <bool BACK>
__device__ __forceinline__ void hold16(float4* held, uint32_t at, bool more) {
    uint32_t raw[16];
    tmem_ld16(at, raw);
    tmem_ld_wait();
    float4 f[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = more ? held[32 * q] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[q].x += __uint_as_float(raw[4 * q]);
        f[q].y += __uint_as_float(raw[4 * q + 1]);
        f[q].z += __uint_as_float(raw[4 * q + 2]);
        f[q].w += __uint_as_float(raw[4 * q + 3]);
        if constexpr (BACK) {
            raw[4 * q] = __float_as_uint(f[q].x);
            raw[4 * q + 1] = __float_as_uint(f[q].y);
            raw[4 * q + 2] = __float_as_uint(f[q].z);
            raw[4 * q + 3] = __float_as_uint(f[q].w);
        } else {
            held[32 * q] = f[q];
        }
    }
    if constexpr (BACK) tmem_st16(at, raw);
}

// The decoding of a block's values.  With b = q + 128 as the last byte of a
// float of exponent field e + 17, the float is 2^(e - 110) + b 2^(e - 133);
// less the same with b = 128 it is q 2^(e - 133), exact, which bf16 holds
// exactly too: a byte shuffle a value, and one addition and one conversion a
// pair.  (In bf16 arithmetic the same took half as many instructions again,
// and the decoding warps' arithmetic is what the tensor cores wait for.)
struct BlockScale {
    uint32_t base;           // the exponent field in its place
    float up;                // 2^64 for the blocks that need it, else 1
};
// A token or column that is not there: its values become 0.
constexpr uint32_t NO_SCALE = 256;
// Blocks above 2^110 or so have no exponent field 17 further up: theirs are
// 64 lower, and what comes out is multiplied (scale_is_high).
__device__ __forceinline__ bool scale_is_high(uint32_t e) { return e >= 238u && e < 255u; }
__device__ __forceinline__ BlockScale block_scale(uint32_t e) {
    BlockScale s;
    s.up = scale_is_high(e) ? 18446744073709551616.f : 1.f;
    // NaN: an infinity's exponent, less a NaN; none: so small that bf16
    // rounds it to 0
    s.base = e == NO_SCALE ? 1u << 23 : e == 255u ? 255u << 23 : (e + 17u - (scale_is_high(e) ? 64u : 0u)) << 23;
    return s;
}
template <bool HIGH>
__device__ __forceinline__ uint2 decode4(uint32_t w, BlockScale s) {
    const uint32_t x = w ^ 0x80808080u;
    const float2 zero = both(-__uint_as_float(s.base | 128u));
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 f = add2(make_float2(__uint_as_float(__byte_perm(x, s.base, 0x7650u + 2 * i)),
                                    __uint_as_float(__byte_perm(x, s.base, 0x7651u + 2 * i))), zero);
        if (HIGH) f = mul2(f, both(s.up));
        const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
        r[i] = reinterpret_cast<const uint32_t&>(v);
    }
    return make_uint2(r[0], r[1]);
}
// 32 values of a block to their places in the tensor cores' layout.
template <bool HIGH>
__device__ __forceinline__ void decode_block(const uint4 (&q)[2], BlockScale s, uint8_t* to, int blk,
                                             uint32_t sw) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint2 v0 = decode4<HIGH>(q[h].x, s), v1 = decode4<HIGH>(q[h].y, s);
        const uint2 v2 = decode4<HIGH>(q[h].z, s), v3 = decode4<HIGH>(q[h].w, s);
        *reinterpret_cast<uint4*>(to + (((blk * 4 + h * 2) ^ sw) << 4)) = make_uint4(v0.x, v0.y, v1.x, v1.y);
        *reinterpret_cast<uint4*>(to + (((blk * 4 + h * 2 + 1) ^ sw) << 4)) =
            make_uint4(v2.x, v2.y, v3.x, v3.y);
    }
}

// What becomes of a sum of row i and column j of matrix e: the norm's weight
// and bias, C, and the store.
__device__ __forceinline__ void finish(const muon_weight_grad_args& a, int64_t e, int64_t i,
                                       int64_t j, float g, float w, float b, float sum) {
    g = fmaf(b, sum, g * w);
    if (a.c) g += load_any(a.c, a.g_dtype, e * a.stride_c + i * a.ld_c + j);
    store_any(a.g, a.g_dtype, e * a.stride_g + i * a.ld_g + j, g);
}

__device__ __forceinline__ float column_sum(const WgLaunch& p, int64_t e, int64_t i) {
    float s = 0.f;
    if (p.colsum_parts == 1) return p.colsum[e * p.a.n + i];
#pragma unroll
    for (int q = 0; q < COLSUM_PARTS; ++q) s += p.colsum[q * p.a.n + i];
    return s;
}

// v += 16 neighbouring elements of a bf16 gradient that lie on 16 bytes.
__device__ __forceinline__ void add16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float f[8];
        load8_bf16(p + 8 * q, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[8 * q + u] += f[u];
    }
}

// 16 columns of 32 sums, staged with the columns XORed with the row, to a
// gradient element by element (rows off 16 bytes, a row's last columns): two
// rows at a time.  `left`: the columns there are; sum: of dY's column `lane`.
// (4096 tokens of 7168 x 8191, bf16: 422 us; 8192 columns, by rows: 287 us.)
__device__ __noinline__ void store_elements(const float* f, void* g, int g_type, int64_t at, int64_t ld,
                                            const void* add, int64_t c_at, int64_t ld_c, int rows,
                                            int left, const float* weight, const float* bias, float sum) {
    const int lane = threadIdx.x & 31, col = lane & 15, two = lane >> 4;
    const bool there = col < left;
    const float w = weight && there ? weight[col] : 1.f, b = bias && there ? bias[col] : 0.f;
    at += two * ld + col;
    c_at += two * ld_c + col;
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + two;
        const float s = __shfl_sync(0xffffffffu, sum, r);
        if (there && r < rows) {
            float t = fmaf(b, s, f[r * 16 + (col ^ (r & 15))] * w);
            if (add) t += load_any(add, g_type, c_at);
            store_any(g, g_type, at, t);
        }
        at += 2 * ld;
        c_at += 2 * ld_c;
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Place of 16-byte piece q of row r in a staged block of 32 rows of 64 bytes.
__device__ __forceinline__ int staged(int r, int q) { return r * 4 + (q ^ ((r >> 1) & 3)); }

// A staged block to a gradient, eight rows a store.
__device__ __forceinline__ void store_rows(const uint4* blk, char* to, int64_t pitch, int rows, int lane) {
    const int piece = lane & 3, sub = lane >> 2;
    to += sub * pitch + piece * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + sub;
        if (r < rows) *reinterpret_cast<uint4*>(to) = blk[staged(r, piece)];
        to += 8 * pitch;
    }
}

// As store_rows, of fp32 and with the epilogue on the way: a thread has the
// same four columns of all its rows, so that w and b are asked for once a
// block; sum is the sum of dY's column `lane`.
__device__ __forceinline__ void finish_rows(const uint4* blk, float* g, int64_t ld, const float* c, int64_t ld_c,
                                            const float* weight, const float* bias, float sum, int rows,
                                            int lane) {
    const int piece = lane & 3, sub = lane >> 2;
    float w[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        w[u] = weight ? weight[piece * 4 + u] : 1.f;
        b[u] = bias ? bias[piece * 4 + u] : 0.f;
    }
    g += sub * ld + piece * 4;
    // C's rows before the first store: C may be G, so that the compiler must
    // keep a load behind the stores before it
    float4 f[4];
    if (c) {
        c += sub * ld_c + piece * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (8 * i + sub < rows) f[i] = *reinterpret_cast<const float4*>(c + 8 * i * ld_c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + sub;
        const float s = __shfl_sync(0xffffffffu, sum, r);
        if (r < rows) {
            const uint4 u = blk[staged(r, piece)];
            float4 v = make_float4(fmaf(b[0], s, __uint_as_float(u.x) * w[0]),
                                   fmaf(b[1], s, __uint_as_float(u.y) * w[1]),
                                   fmaf(b[2], s, __uint_as_float(u.z) * w[2]),
                                   fmaf(b[3], s, __uint_as_float(u.w) * w[3]));
            if (c) {
                v.x += f[i].x;
                v.y += f[i].y;
                v.z += f[i].z;
                v.w += f[i].w;
            }
            *reinterpret_cast<float4*>(g) = v;
        }
        g += 8 * ld;
    }
}

// The steps of a pair's tiles, one after the other.
template <bool WIDE>
struct Steps {
    const WgLaunch& p;
    const uint16_t* order;
    int32_t it, by;
    Item x;
    int s = -1;
    bool more;
    __device__ __forceinline__ Steps(const WgLaunch& l, const uint16_t* o, int first, int stride)
        : p(l), order(o), it(first), by(stride), more(first < l.items) {
        if (more) x = item_at<WIDE>(p, order, it);
        next();
    }
    __device__ __forceinline__ void next() {
        if (!more || ++s < x.steps) return;
        s = 0;
        do {
            it += by;
            more = it < p.items;
            if (more) x = item_at<WIDE>(p, order, it);
        } while (more && x.steps == 0);
    }
};

// F32: what is stored is fp32 (G, or the sums of a part of a split).
template <bool F32, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(W_THREADS, 1)
    weight_grad_kernel(const __grid_constant__ WgLaunch p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using S = Shape<WIDE>;
    uint8_t* sA = smem;
    uint8_t* sB = smem + S::B_OFF;
    uint8_t* sR = smem + S::R_OFF;
    uint64_t* a_bar = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);   // this CTA's dY of a step
    uint64_t* done_bar = a_bar + S::A_STAGES;       // the products of a step have run
    uint64_t* r_bar = done_bar + S::A_STAGES;       // this CTA's 8-bit values
    uint64_t* free_bar = r_bar + S::R_STAGES;       // and they have been read
    uint64_t* ready_bar = free_bar + S::R_STAGES;   // both CTAs' operands (leader's)
    uint64_t* tfull_bar = ready_bar + S::B_STAGES;
    uint64_t* tempty_bar = tfull_bar + 2;
    uint64_t* drain_bar = tempty_bar + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::A_STAGES; ++s) {
            mbar_init(smem_u32(&a_bar[s]), 1);
            mbar_init(smem_u32(&done_bar[s]), 1);
        }
        for (int s = 0; s < S::R_STAGES; ++s) {
            mbar_init(smem_u32(&r_bar[s]), 1);
            mbar_init(smem_u32(&free_bar[s]), W_DEC_WARPS);
        }
        for (int s = 0; s < S::B_STAGES; ++s) mbar_init(smem_u32(&ready_bar[s]), 2 * W_DEC_WARPS);
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull_bar[a]), 1);
            mbar_init(smem_u32(&tempty_bar[a]), 2 * W_EPI_WARPS);
        }
        mbar_init(smem_u32(drain_bar), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile(
            "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                smem_u32(tmem_slot)),
            "r"(W_TMEM_COLS)
            : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    allow_dependent_launch();
    // Experts by their size, the largest first: with tiles dealt out in turn,
    // no pair then has more than about one tile's steps above another.  Sizes
    // that fall as 1 / rank: 128 experts of 768 x 2048 302 us instead of 319,
    // 16 of 2048 x 2048 147 instead of 166; even sizes: no difference.
    uint16_t* order = nullptr;
    if (p.sorted) {
        order = reinterpret_cast<uint16_t*>(smem + S::ORDER_OFF);
        const int experts = static_cast<int>(p.a.experts);
        int64_t* size = reinterpret_cast<int64_t*>(smem);    // the stages are not in use yet
        for (int e = threadIdx.x; e < experts; e += W_THREADS) {
            int64_t begin, end;
            segment(p.a, e, &begin, &end);
            size[e] = end - begin;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < experts; e += W_THREADS) {
            const int64_t mine = size[e];
            int rank_of = 0;
            for (int o = 0; o < experts; ++o)
                rank_of += size[o] > mine || (size[o] == mine && o < e);
            order[rank_of] = static_cast<uint16_t>(e);
        }
        // before the stages' first loads (they are written by another proxy)
        fence_proxy_async_smem();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t limit = p.wait_limit_ns;

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        // WIDE: the 8-bit values some steps ahead, as they are decoded
        // meanwhile; else both operands of a step on one barrier.
        if (lane == 0) {
            Steps<WIDE> ra(p, order, pair, npairs), aa = ra;
            uint32_t nr = 0, na = 0;      // steps issued
            bool ok = true;
            auto load_r = [&](const Steps<WIDE>& at, uint32_t n, uint32_t bar) {
                const uint32_t dst = smem_u32(sR + stage_of(n, S::R_STAGES) * W_R_BYTES);
                const int b0 = at.x.k0 + static_cast<int>(rank) * 128, t = at.x.t0 + at.s * W_TOK;
                tma_load_2d(dst, &p.tm_q, bar, b0, t);
                tma_load_2d(dst + W_RBOX, &p.tm_q, bar, b0 + 64, t);
            };
            while (ok && aa.more) {
                if constexpr (WIDE)
                    for (; ra.more && nr <= na + S::AHEAD; ++nr, ra.next()) {
                        const uint32_t slot = stage_of(nr, S::R_STAGES), rb = smem_u32(&r_bar[slot]);
                        ok = wait_soon(smem_u32(&free_bar[slot]), parity_of(nr, S::R_STAGES) ^ 1, abort_flag,
                                       &g_ops_err, limit);
                        if (!ok) break;
                        mbar_expect_tx(rb, W_R_BYTES);
                        load_r(ra, nr, rb);
                    }
                const uint32_t slot = stage_of(na, S::A_STAGES), ab = smem_u32(&a_bar[slot]);
                ok = ok && wait_soon(smem_u32(&done_bar[slot]), parity_of(na, S::A_STAGES) ^ 1, abort_flag,
                                     &g_ops_err, limit);
                if (!ok) break;
                mbar_expect_tx(ab, S::A_BYTES + (WIDE ? 0 : W_R_BYTES));
                if constexpr (!WIDE) load_r(aa, na, ab);
                const uint32_t dst = smem_u32(sA + slot * S::A_BYTES);
                const int a0 = aa.x.n0 + static_cast<int>(rank) * 128, t = aa.x.t0 + aa.s * W_TOK;
#pragma unroll
                for (int h = 0; h < S::HALVES; ++h) {
                    tma_load_2d(dst + 2 * h * W_BOX, &p.tm_dy, ab, a0 + 256 * h, t);
                    tma_load_2d(dst + (2 * h + 1) * W_BOX, &p.tm_dy, ab, a0 + 256 * h + 64, t);
                }
                ++na;
                aa.next();
            }
            if (!ok) {
                // the last load of each stage
                for (uint32_t i = nr - min(nr, uint32_t(S::R_STAGES)); i < nr; ++i)
                    wait_quiet(smem_u32(&r_bar[stage_of(i, S::R_STAGES)]), parity_of(i, S::R_STAGES), limit);
                for (uint32_t i = na - min(na, uint32_t(S::A_STAGES)); i < na; ++i)
                    wait_quiet(smem_u32(&a_bar[stage_of(i, S::A_STAGES)]), parity_of(i, S::A_STAGES), limit);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------- products (leader)
        if (lane == 0 && rank == 0) {
            uint32_t step = 0;
            uint32_t uses[2] = {0, 0};    // of each accumulator
            uint32_t first = 0;           // the one that the tile starts in
            bool ok = true, any = false;
            // both operands MN-major: two 64-wide halves W_BOX apart, token
            // rows of 128 bytes, 16 of them (2048 bytes) a product
            const uint64_t a_desc = smem_desc(smem_u32(sA), W_BOX, 1024);
            const uint64_t b_desc = smem_desc(smem_u32(sB), W_BOX, 1024);
            const uint32_t idesc = instr_desc(256, 256, 1) | (1u << 15);
            // an accumulator that has been written out
            auto take = [&](uint32_t acc) {
                const uint32_t use = acc ? uses[1]++ : uses[0]++;
                const bool got = wait_soon(smem_u32(&tempty_bar[acc]), (use & 1) ^ 1, abort_flag,
                                           &g_ops_err, limit);
                tc_fence_after();
                return got;
            };
            // the products of a step and of the tile's half h
            auto products = [&](uint32_t acc, int h, bool fresh) {
                const uint64_t ad = a_desc + (stage_of(step, S::A_STAGES) * S::A_BYTES + h * 2 * W_BOX >> 4);
                const uint64_t bd = b_desc + (stage_of(step, S::B_STAGES) * W_B_BYTES >> 4);
#pragma unroll
                for (int kk = 0; kk < W_TOK / 16; ++kk)
                    mma_pair(tmem_base + acc * 256, ad + static_cast<uint64_t>(kk * (2048 >> 4)),
                             bd + static_cast<uint64_t>(kk * (2048 >> 4)), idesc,
                             (fresh && kk == 0) ? 0u : 1u);
            };
            for (int32_t it = pair; ok && it < p.items; it += npairs) {
                const Item x = item_at<WIDE>(p, order, it);
                if (x.steps == 0) continue;
                for (int s0 = 0; ok && s0 < x.steps; s0 += p.chunk) {
                    const uint32_t acc = WIDE ? 0u : s0 ? first ^ 1 : first;
                    if (!take(acc)) {
                        ok = false;
                        break;
                    }
                    const int s1 = min(s0 + p.chunk, x.steps);
                    for (int s = s0; s < s1; ++s, ++step) {
                        if (!wait_soon(smem_u32(&ready_bar[stage_of(step, S::B_STAGES)]),
                                       parity_of(step, S::B_STAGES), abort_flag, &g_ops_err, limit)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        products(acc, 0, s == s0);
                        any = true;
                        if (WIDE) {
                            if (s == s0 && !take(1)) {
                                ok = false;
                                break;
                            }
                            products(1, 1, s == s0);
                        }
                        commit_pair_multicast(smem_u32(&done_bar[stage_of(step, S::A_STAGES)]));
                    }
                    if (ok) commit_pair_multicast(smem_u32(&tfull_bar[acc]));
                }
                first ^= 1;
            }
            if (!ok && any) {
                commit_pair_local(smem_u32(drain_bar));
                wait_quiet(smem_u32(drain_bar), 0, limit);
            }
        }
    } else if (warp >= W_DEC_WARP0) {
        // ----------------------------------------------------------- decode
        // Two groups of warps take the steps in turn.  A thread turns blocks of
        // 32 values: 16 tokens and the two blocks of a 64-wide box in a warp at
        // a time, so that eight lanes' 16-byte accesses fall
        // on all banks in both swizzles.
        const int group = (warp - W_DEC_WARP0) / W_DEC_WARPS;
        const int dw = (warp - W_DEC_WARP0) % W_DEC_WARPS;
        const int box = dw & 1;
        const int row = (dw >> 1) * 16 * W_DEC_BLOCKS + (lane >> 1);   // and 16 rows on, ...
        const int blk = lane & 1;
        const uint32_t src = box * W_RBOX + row * 64;
        const uint32_t src_sw = (row >> 1) & 3;
        const uint32_t dst = box * W_BOX + row * 128;
        const uint32_t dst_sw = row & 7;
        const int nblk = static_cast<int>((p.a.k + CKPT_BLOCK - 1) / CKPT_BLOCK);
        const uint32_t ready_leader = map_to_rank(smem_u32(ready_bar), 0);
        uint32_t before = 0;          // steps of the tiles before this one
        uint32_t step = group;
        bool ok = true;
        // the scale bytes come four of this group's steps at a time, one
        // round ahead, also across tiles
        uint32_t nxt[4][W_DEC_BLOCKS];
        auto fetch = [&](const Item& x, int s) {
            const int eb = (x.k0 + static_cast<int>(rank) * 128) / CKPT_BLOCK + box * 2 + blk;
            const uint8_t* ep = p.a.saved.e + eb;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int su = s + u * W_DEC_GROUPS;
#pragma unroll
                for (int i = 0; i < W_DEC_BLOCKS; ++i) {
                    const int64_t t = int64_t(x.t0) + su * W_TOK + row + 16 * i;
                    nxt[u][i] =
                        (eb < nblk && su < x.steps && t < x.end) ? ep[t * p.a.saved.ld_e] : NO_SCALE;
                }
            }
        };
        Item x, y{};
        int32_t it = pair;
        if (it < p.items) {
            x = item_at<WIDE>(p, order, it);
            fetch(x, group);
        }
        for (; ok && it < p.items; it += npairs, x = y) {
            const int first = (group - static_cast<int>(before)) & (W_DEC_GROUPS - 1);
            before += x.steps;
            const int y_first = (group - static_cast<int>(before)) & (W_DEC_GROUPS - 1);
            const bool more = it + npairs < p.items;
            if (more) y = item_at<WIDE>(p, order, it + npairs);
            if (first >= x.steps && more) fetch(y, y_first);
            for (int s = first; ok && s < x.steps; s += 4 * W_DEC_GROUPS) {
                uint32_t cur[4][W_DEC_BLOCKS];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int i = 0; i < W_DEC_BLOCKS; ++i) cur[u][i] = nxt[u][i];
                if (s + 4 * W_DEC_GROUPS < x.steps) fetch(x, s + 4 * W_DEC_GROUPS);
                else if (more) fetch(y, y_first);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int su = s + u * W_DEC_GROUPS;
                    if (su >= x.steps) break;
                    const uint32_t sa = stage_of(step, S::A_STAGES), sb = stage_of(step, S::B_STAGES),
                                   sr = stage_of(step, S::R_STAGES);
                    // the step that had the stage of B before, which may have
                    // been the other group's: without this wait, a load of
                    // that step's that is slow to land makes a wait for both
                    // operands return too soon (weight_grad_stages.h).  WIDE:
                    // the 8-bit values have a stage whose users are all this
                    // group's, and are asked for first (16384 tokens: 1038 us,
                    // 1061 the other way round)
                    const uint32_t last = last_user<WIDE>(step);
                    const auto used = [&] {
                        return !stage_was_used<WIDE>(step) ||
                               wait_soon(smem_u32(&done_bar[stage_of(last, S::A_STAGES)]),
                                         parity_of(last, S::A_STAGES), abort_flag, &g_ops_err, limit);
                    };
                    const auto there = [&] {
                        return wait_soon(smem_u32(WIDE ? &r_bar[sr] : &a_bar[sa]),
                                         parity_of(step, WIDE ? S::R_STAGES : S::A_STAGES), abort_flag,
                                         &g_ops_err, limit);
                    };
                    const bool got = WIDE ? there() && used() : used() && there();
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    bool high = false;
                    uint4 q[W_DEC_BLOCKS][2];
#pragma unroll
                    for (int i = 0; i < W_DEC_BLOCKS; ++i) {
                        // 16 rows on, the swizzles are the same
                        const uint8_t* r = sR + sr * W_R_BYTES + src + i * 16 * 64;
                        q[i][0] = *reinterpret_cast<const uint4*>(r + (((blk * 2) ^ src_sw) << 4));
                        q[i][1] = *reinterpret_cast<const uint4*>(r + (((blk * 2 + 1) ^ src_sw) << 4));
                        high |= scale_is_high(cur[u][i]);
                    }
                    uint8_t* const to = sB + sb * W_B_BYTES + dst;
                    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
                        for (int i = 0; i < W_DEC_BLOCKS; ++i)
                            decode_block<true>(q[i], block_scale(cur[u][i]), to + i * 16 * 128, blk, dst_sw);
                    } else {
#pragma unroll
                        for (int i = 0; i < W_DEC_BLOCKS; ++i)
                            decode_block<false>(q[i], block_scale(cur[u][i]), to + i * 16 * 128, blk, dst_sw);
                    }
                    if constexpr (WIDE) {
                        // the values have been used, so their loads are done
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&free_bar[sr]));
                        // dY has to be there too
                        const bool in = wait_soon(smem_u32(&a_bar[sa]), parity_of(step, S::A_STAGES),
                                                  abort_flag, &g_ops_err, limit);
                        if (!__all_sync(0xffffffffu, in)) {
                            ok = false;
                            break;
                        }
                    }
                    const int left = x.end - (x.t0 + su * W_TOK);
                    if (left < W_TOK) {
                        // tokens of the next matrix in dY's stage: 0 times a
                        // NaN of theirs would be a NaN here
                        uint8_t* a = sA + sa * S::A_BYTES;
                        constexpr int BOXES = 2 * S::HALVES;
                        for (int c = dw * 32 + lane; c < (W_TOK - left) * 8 * BOXES; c += W_DEC_WARPS * 32)
                            *reinterpret_cast<uint4*>(a + (c >> 3) % BOXES * W_BOX +
                                                      (left + (c >> 3) / BOXES) * 128 + (c & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_leader(ready_leader + 8 * sb);
                    step += W_DEC_GROUPS;
                }
            }
        }
    } else {
        // --------------------------------------------------------- write out
        const int lg = warp & 3;                    // this warp's 32 TMEM lanes,
        const int c_first = (warp - 2) / 4 * 4;     // and four of its 32-column blocks
        uint4* const blk = reinterpret_cast<uint4*>(smem + S::EPI_OFF + (warp - 2) * W_EPI_BYTES);
        const uint32_t tempty_leader = map_to_rank(smem_u32(tempty_bar), 0);
        // WIDE: this lane's places, 16 columns in four pieces 32 apart
        float4* const held = p.held + ((int64_t(blockIdx.x) * W_EPI_WARPS + warp - 2) * 16) * 128 + lane;
        uint32_t uses[2] = {0, 0};
        uint32_t first = 0;
        bool ok = true;
        auto wait_full = [&](uint32_t acc) {
            const uint32_t use = acc ? uses[1]++ : uses[0]++;
            const bool got = wait_soon(smem_u32(&tfull_bar[acc]), use & 1, abort_flag, &g_ops_err,
                                       limit);
            if (!__all_sync(0xffffffffu, got)) return false;
            tc_fence_after();
            return true;
        };
        auto release = [&](uint32_t acc) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * acc);
        };
        for (int32_t it = pair; ok && it < p.items; it += npairs) {
            const Item x = item_at<WIDE>(p, order, it);
            const uint32_t tlane = tmem_base + (static_cast<uint32_t>(lg * 32) << 16);
            if (F32 && p.a.c && p.splits == 1) {
                // C on its way to L2 while the products run
                constexpr int size = F32 ? 4 : 2;
#pragma unroll 1
                for (int h = 0; h < S::HALVES; ++h) {
                    const int64_t i = x.n0 + 256 * h + static_cast<int>(rank) * 128 + lg * 32 + lane;
                    const int64_t j0 = x.k0 + 32 * c_first, j1 = min(p.a.k, j0 + 128);
                    if (i < p.a.n)
                        for (int64_t j = j0; j < j1; j += 128 / size)
                            prefetch_l2(static_cast<const char*>(p.a.c) +
                                        (x.e * p.a.stride_c + i * p.a.ld_c + j) * size);
                }
            }
            if (x.steps) {
                if (!wait_full(first)) {
                    ok = false;
                    break;
                }
                // later chunks of the tokens: added up in fp32, rounded to
                // nearest
                for (int s0 = p.chunk; s0 < x.steps; s0 += p.chunk) {
                    if constexpr (WIDE) {
                        // both accumulators are in use: the sums so far wait
                        // in memory (L2 holds all pairs')
#pragma unroll 1
                        for (int c = 0; c < 16; ++c) {
                            hold16<false>(held + c * 128, tlane + c / 8 * 256 + 32 * c_first + 16 * (c & 7),
                                          s0 > p.chunk);
                            if (c == 7) release(0);
                        }
                        release(1);
                    }
                    if (!wait_full(WIDE ? 0 : first ^ 1)) {
                        ok = false;
                        break;
                    }
                    if constexpr (WIDE) continue;
#pragma unroll 1
                    for (int c = 2 * c_first; c < 2 * (c_first + 4); ++c)
                        tmem_add16(tlane + first * 256 + 16 * c, tlane + (first ^ 1) * 256 + 16 * c);
                    release(first ^ 1);
                }
                if (!ok) break;
                if (WIDE && x.steps > p.chunk)
#pragma unroll 1
                    for (int c = 0; c < 16; ++c)
                        hold16<true>(held + c * 128, tlane + c / 8 * 256 + 32 * c_first + 16 * (c & 7), true);
            }
#pragma unroll 1
            for (int h = 0; h < S::HALVES; ++h) {
                const uint32_t acc = WIDE ? h : first;
                const uint32_t taddr = tlane + acc * 256;
                const int r0 = x.n0 + 256 * h + static_cast<int>(rank) * 128 + lg * 32;
                const int n = static_cast<int>(p.a.n), k = static_cast<int>(p.a.k);
                const int rows = min(32, n - r0);
                // a part of a split leaves its sums as they are
                const bool apply = p.splits == 1;
                const float sum = (apply && p.colsum && lane < rows) ? column_sum(p, x.e, r0 + lane) : 0.f;
                const int64_t ld = apply ? p.a.ld_g : p.ld_part;
                const int64_t g0 = apply ? x.e * p.a.stride_g + r0 * ld
                                         : ((int64_t(x.split) * p.a.experts + x.e) * n + r0) * ld;
                const int64_t c0 = x.e * p.a.stride_c + r0 * p.a.ld_c;
                void* const g = apply ? p.a.g : p.part;
                // a matrix without tokens is 0 whatever its weights are
                const bool affine = apply && x.steps && (p.weight || p.bias);
                const void* const add = apply ? p.a.c : nullptr;
                constexpr int size = F32 ? 4 : 2;
                if (rows > 0) {
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        const int j0 = x.k0 + 32 * c_first + 16 * c;
                        if (j0 >= k) break;
                        // Staged, and stored as rows of 64 bytes (lanes that
                        // store their own rows straight from registers touch 32
                        // lines a store): 16 columns of fp32, or 32 of bf16
                        // from two rounds.  fp32 sums are finished on the way
                        // out of the stage, bf16 ones before they are rounded
                        // into it.
                        const int odd = F32 ? 0 : c & 1;
                        const int row0 = j0 - 16 * odd;
                        const bool whole = p.vec && row0 + (F32 ? 16 : 32) <= k;
                        uint32_t raw[16];
                        if (x.steps) {
                            tmem_ld16(taddr + 32 * c_first + 16 * c, raw);
                            tmem_ld_wait();
                        } else {
#pragma unroll
                            for (int u = 0; u < 16; ++u) raw[u] = 0;
                        }
                        const float* const weight = affine && p.weight ? p.weight + j0 : nullptr;
                        const float* const bias = affine && p.bias ? p.bias + j0 : nullptr;
                        if (F32 && whole) {
                            __syncwarp();      // the last rows have been read
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                blk[staged(lane, q)] =
                                    make_uint4(raw[4 * q], raw[4 * q + 1], raw[4 * q + 2], raw[4 * q + 3]);
                            __syncwarp();
                            float* const to = static_cast<float*>(g) + g0 + j0;
                            if (affine || add)
                                finish_rows(blk, to, ld,
                                            add ? static_cast<const float*>(add) + c0 + j0 : nullptr,
                                            p.a.ld_c, weight, bias, sum, rows, lane);
                            else
                                store_rows(blk, reinterpret_cast<char*>(to), ld * size, rows, lane);
                            continue;
                        }
                        if (whole) {
                            float v[16];
#pragma unroll
                            for (int u = 0; u < 16; ++u) v[u] = __uint_as_float(raw[u]);
                            if (affine) {
                                const float wl = weight ? weight[lane & 15] : 1.f;
                                const float bl = bias ? bias[lane & 15] : 0.f;
#pragma unroll
                                for (int u = 0; u < 16; ++u)
                                    v[u] = fmaf(__shfl_sync(0xffffffffu, bl, u), sum,
                                                v[u] * __shfl_sync(0xffffffffu, wl, u));
                            }
                            if (!odd) __syncwarp();
                            if (add && lane < rows)
                                add16(static_cast<const __nv_bfloat16*>(add) + c0 + lane * p.a.ld_c + j0, v);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                float t[8];
#pragma unroll
                                for (int u = 0; u < 8; ++u) t[u] = v[8 * q + u];
                                store8_bf16(reinterpret_cast<__nv_bfloat16*>(&blk[staged(lane, q + 2 * odd)]),
                                            t);
                            }
                            if (!odd) continue;
                            __syncwarp();
                            store_rows(blk, static_cast<char*>(g) + (g0 + row0) * size, ld * size, rows, lane);
                            continue;
                        }
                        float* const f = reinterpret_cast<float*>(blk);
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            f[lane * 16 + (u ^ (lane & 15))] = __uint_as_float(raw[u]);
                        __syncwarp();
                        store_elements(f, g, F32 ? MUON_F32 : MUON_BF16, g0 + j0, ld, add, c0 + j0,
                                       p.a.ld_c, rows, k - j0, weight, bias, sum);
                        __syncwarp();
                    }
                }
                if (x.steps) release(acc);
            }
            if (!WIDE && x.steps) first ^= 1;
        }
    }

    tc_fence_before();
    cluster_sync_all();      // no CTA leaves while its pair may still touch it
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(W_TMEM_COLS)
                     : "memory");
    }
}

// The splits' partial sums in order, then the epilogue: a block has 1024
// columns of a row, four neighbouring ones a thread.
__global__ void __launch_bounds__(256) weight_grad_join_kernel(const __grid_constant__ WgLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int k = static_cast<int>(p.a.k), j = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (j >= k) return;
    const int64_t rows = p.a.experts * p.a.n;
    const int64_t size = rows * p.ld_part;
    float w[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        w[u] = p.weight && j + u < k ? p.weight[j + u] : 1.f;
        b[u] = p.bias && j + u < k ? p.bias[j + u] : 0.f;
    }
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const int64_t e = p.a.experts == 1 ? 0 : row / p.a.n, i = row - e * p.a.n;
        const float* part = p.part + row * p.ld_part + j;
        float g[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            const float4 f = *reinterpret_cast<const float4*>(part + s * size);
            g[0] += f.x;
            g[1] += f.y;
            g[2] += f.z;
            g[3] += f.w;
        }
        const float sum = p.colsum ? column_sum(p, e, i) : 0.f;
        int64_t begin, end;
        segment(p.a, e, &begin, &end);
        const bool some = end > begin;           // else 0 whatever the weights are
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (j + u < k) finish(p.a, e, i, j + u, g[u], some ? w[u] : 1.f, some ? b[u] : 0.f, sum);
    }
}

// Sums of dY's columns over each matrix's tokens (gridDim.z parts of them):
// 256 columns and 8 rows at a time in a block.  It waits for its loads: 32
// parts of one matrix's tokens keep more of them in flight than 16 (4097
// tokens of 4096 columns, with the product behind it: 82 and 97 us; 64 parts
// are no better).
__global__ void __launch_bounds__(256)
    colsum_kernel(const __grid_constant__ muon_weight_grad_args a, float* out) {
    __shared__ float red[8][256];
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 256 + lane * 8;
    const int n = static_cast<int>(a.n);
    const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(a.dy) + i;
    for (int64_t e = blockIdx.y; e < a.experts; e += gridDim.y) {
        int64_t begin, end;
        segment(a, e, &begin, &end);
        const int64_t len = end - begin;
        const int64_t t0 = begin + len * blockIdx.z / gridDim.z;
        const int64_t t1 = begin + len * (blockIdx.z + 1) / gridDim.z;
        float2 s[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll 8
        for (int64_t t = t0 + warp; t < t1; t += 8) {
            Vec<__nv_bfloat16, false> v;
            float2 f[4];
            v.load(dy + t * a.ld_dy, n - i);
            v.get(f);
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] = add2(s[u], f[u]);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u)
            *reinterpret_cast<float2*>(&red[warp][lane * 8 + 2 * u]) = s[u];
        __syncthreads();
        const int col = blockIdx.x * 256 + threadIdx.x;
        if (col < n) {
            float sum = 0.f;
            for (int w = 0; w < 8; ++w) sum += red[w][threadIdx.x];
            out[(blockIdx.z * a.experts + e) * a.n + col] = sum;
        }
    }
}

// The norm's weight and bias, where they are bf16, as the write-out reads them.
__global__ void __launch_bounds__(256)
    widen_kernel(const __nv_bfloat16* weight, const __nv_bfloat16* bias, int k, float* w, float* b) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= k) return;
    if (weight) w[j] = __bfloat162float(weight[j]);
    if (bias) b[j] = __bfloat162float(bias[j]);
}

// dY with rows that TMA can read: dense rows of ld elements (a multiple of 8).
__global__ void __launch_bounds__(256)
    align_kernel(const __nv_bfloat16* src, int64_t rows, int64_t n, int64_t ld_src,
                 __nv_bfloat16* dst, int64_t ld) {
    grid_dependency_wait();
    allow_dependent_launch();
    for (int64_t u = blockIdx.x * int64_t(256) + threadIdx.x; u < rows * n;
         u += int64_t(gridDim.x) * 256) {
        const int64_t r = u / n, c = u % n;
        dst[r * ld + c] = src[r * ld_src + c];
    }
}

// ------------------------------------------------------------------- host

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

bool dy_aligned(const muon_weight_grad_args& a) {
    return reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 &&
           (a.rows <= 1 || (a.ld_dy % 8 == 0 && a.ld_dy >= a.n));
}

int64_t tiles(const muon_weight_grad_args& a) {
    return a.experts * ceil_div(a.n, 256) * ceil_div(a.k, 256);
}

// Parts that the tokens are split into: as many as give every pair a tile,
// each of eight steps or more on average (8192 tokens of 512 x 2048: 30 us in
// four parts, 55 in one; 300 tokens: 16 and 15 us, not split).
int split_count(const muon_weight_grad_args& a) {
    const int64_t steps = ceil_div(ceil_div(a.rows, a.experts), W_TOK);
    int64_t s = W_PAIRS / tiles(a);
    if (s > steps / 8) s = steps / 8;
    return static_cast<int>(s < 1 ? 1 : s);
}

// Tiles of 512 x 256 instead of 256 x 256.  A decoded value then serves twice
// the products, but there is one accumulator, so that a tile's writing out is
// not hidden, and the last round of tiles is coarser.  In units of 0.21 us a
// pair takes 3 a step + 34 for a wide tile and 2 a step + 10 for another
// (measured with 7168 x 8192 from 300 to 4096 tokens; us, wide and not: 512
// tokens 78 and 68, 1024 108 and 106, 2048 165 and 182, 4096 286 and 345,
// 16384 1040 and 1452).  fp32 sums are added up in both accumulators.
bool is_wide(const muon_weight_grad_args& a, int splits) {
    if (a.g_dtype != MUON_BF16 || splits > 1) return false;
    const int64_t steps = ceil_div(ceil_div(a.rows, a.experts), W_TOK);
    const int64_t tall = a.experts * ceil_div(a.n, 512) * ceil_div(a.k, 256);
    return ceil_div(tall, W_PAIRS) * (3 * steps + 34) < ceil_div(tiles(a), W_PAIRS) * (2 * steps + 10);
}

int grid_for(int64_t items) {
    const int64_t g = ceil_div(items, 256);
    return static_cast<int>(g < 1 ? 1 : g > 152 * 8 ? 152 * 8 : g);
}

struct Layout {
    size_t colsum = 0, dy = 0, part = 0, held = 0, weight = 0, bias = 0, bytes = 0;
    int colsum_parts = 0, splits = 1;
    bool wide = false;
    int64_t ld_dy = 0, ld_part = 0;
};
Layout layout(const muon_weight_grad_args& a) {
    Layout l;
    l.splits = split_count(a);
    if (a.bias) {
        l.colsum = l.bytes;
        l.colsum_parts = a.experts == 1 ? COLSUM_PARTS : 1;
        l.bytes += align256(size_t(l.colsum_parts) * a.experts * a.n * 4);
    }
    if (a.rows && !dy_aligned(a)) {
        l.dy = l.bytes;
        l.ld_dy = ceil_div(a.n, 8) * 8;
        l.bytes += align256(size_t(a.rows) * l.ld_dy * 2);
    }
    if (l.splits > 1) {
        l.part = l.bytes;
        l.ld_part = ceil_div(a.k, 8) * 8;
        l.bytes += align256(size_t(l.splits) * a.experts * a.n * l.ld_part * 4);
    }
    if (a.w_dtype == MUON_BF16) {
        const size_t each = align256(size_t(a.k) * 4);
        l.weight = l.bytes;
        if (a.weight) l.bytes += each;
        l.bias = l.bytes;
        if (a.bias) l.bytes += each;
    }
    l.wide = is_wide(a, l.splits);
    if (l.wide && ceil_div(a.rows, W_TOK) > CHUNK_BF16) {
        // a tile may have more than one chunk
        l.held = l.bytes;
        l.bytes += size_t(W_PAIRS) * 512 * 256 * 4;
    }
    return l;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// A {64, 64}-box map of rows x cols elements; zeros come back past its ends.
bool encode_map(CUtensorMap* tm, CUtensorMapDataType type, size_t size, const void* base,
                int64_t rows, int64_t cols, int64_t ld, CUtensorMapSwizzle sw) {
    if (!encoder()) return false;
    cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    cuuint64_t strides[1] = {cuuint64_t(ld) * size};
    cuuint32_t box[2] = {64, 64}, el[2] = {1, 1};
    return encoder()(tm, type, 2, const_cast<void*>(base), dims, strides, box, el,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether a gradient's rows lie on `bytes`.
bool rows_on(int64_t bytes, const void* p, int64_t size, const muon_weight_grad_args& a, int64_t ld,
             int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (a.n <= 1 || ld * size % bytes == 0) &&
           (a.experts <= 1 || stride * size % bytes == 0);
}

}  // namespace

unsigned long long wait_limit_ns() {
    static const unsigned long long v = [] {
        const char* s = std::getenv("MUON_WAIT_LIMIT_MS");
        const long long ms = s ? std::atoll(s) : 0;
        return (ms > 0 ? static_cast<unsigned long long>(ms) : 2000ull) * 1000000ull;
    }();
    return v;
}

size_t weight_grad_workspace(const muon_weight_grad_args& a) { return layout(a).bytes; }

cudaError_t launch_weight_grad(const muon_weight_grad_args& a, void* ws, cudaStream_t s) {
    const Layout l = layout(a);
    char* base = static_cast<char*>(ws);
    WgLaunch p = {};
    p.a = a;
    p.splits = l.splits;
    const bool wide = l.wide;
    p.tiles_n = static_cast<int32_t>(ceil_div(a.n, wide ? 512 : 256));
    p.tiles_k = static_cast<int32_t>(ceil_div(a.k, 256));
    p.items = static_cast<int32_t>(a.experts * p.tiles_n * p.tiles_k * l.splits);
    p.wait_limit_ns = wait_limit_ns();
    const int64_t size = a.g_dtype == MUON_F32 ? 4 : 2;
    p.chunk = a.g_dtype == MUON_F32 ? CHUNK_F32 : CHUNK_BF16;
    p.held = reinterpret_cast<float4*>(base + l.held);
    p.sorted = a.experts > 1 && a.experts <= W_ORDER;
    if (l.splits > 1) {
        p.part = reinterpret_cast<float*>(base + l.part);
        p.ld_part = l.ld_part;
        p.vec = 1;
    } else {
        auto on = [&](int64_t bytes) {
            return rows_on(bytes, a.g, size, a, a.ld_g, a.stride_g) &&
                   (!a.c || rows_on(bytes, a.c, size, a, a.ld_c, a.stride_c));
        };
        p.vec = on(16);
    }
    cudaError_t e;
    if (a.w_dtype == MUON_BF16 && (a.weight || a.bias)) {
        auto* w = reinterpret_cast<float*>(base + l.weight);
        auto* b = reinterpret_cast<float*>(base + l.bias);
        e = launch_kernel(widen_kernel, dim3(static_cast<unsigned>(ceil_div(a.k, 256))), dim3(256), 0, s,
                          static_cast<const __nv_bfloat16*>(a.weight),
                          static_cast<const __nv_bfloat16*>(a.bias), static_cast<int>(a.k), w, b);
        if (e != cudaSuccess) return e;
        p.weight = a.weight ? w : nullptr;
        p.bias = a.bias ? b : nullptr;
    } else {
        p.weight = static_cast<const float*>(a.weight);
        p.bias = static_cast<const float*>(a.bias);
    }
    if (a.bias) {
        p.colsum = reinterpret_cast<float*>(base + l.colsum);
        p.colsum_parts = l.colsum_parts;
        e = launch_kernel(colsum_kernel,
                          dim3(static_cast<unsigned>(ceil_div(a.n, 256)),
                               static_cast<unsigned>(a.experts < 32768 ? a.experts : 32768),
                               static_cast<unsigned>(l.colsum_parts)),
                          dim3(256), 0, s, a, reinterpret_cast<float*>(base + l.colsum));
        if (e != cudaSuccess) return e;
    }
    if (a.rows) {
        const void* dy = a.dy;
        int64_t ld = a.rows > 1 ? a.ld_dy : ceil_div(a.n, 8) * 8;
        if (!dy_aligned(a)) {
            auto* to = reinterpret_cast<__nv_bfloat16*>(base + l.dy);
            e = launch_kernel(align_kernel, dim3(grid_for(a.rows * a.n)), dim3(256), 0, s,
                              static_cast<const __nv_bfloat16*>(a.dy), a.rows, a.n, a.ld_dy, to,
                              l.ld_dy);
            if (e != cudaSuccess) return e;
            dy = to;
            ld = l.ld_dy;
        }
        const int64_t ld_q = a.rows > 1 ? a.saved.ld_q : ceil_div(a.k, 32) * 32;
        if (!encode_map(&p.tm_dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dy, a.rows, a.n, ld,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_map(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.saved.q, a.rows, a.k, ld_q,
                        CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    }
    const int pairs = p.items < W_PAIRS ? p.items : W_PAIRS;
    const bool f32 = l.splits > 1 || a.g_dtype == MUON_F32;
    const int size_of[3] = {Shape<false>::SMEM, Shape<false>::SMEM, Shape<true>::SMEM};
    void (*const kernel[3])(WgLaunch) = {weight_grad_kernel<false, false>, weight_grad_kernel<true, false>,
                                         weight_grad_kernel<false, true>};
    static int attr_done[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        for (int i = 0; i < 3; ++i) {
            e = cudaFuncSetAttribute(kernel[i], cudaFuncAttributeMaxDynamicSharedMemorySize, size_of[i]);
            if (e != cudaSuccess) return e;
        }
        if (dev >= 0 && dev < 64) attr_done[dev] = 1;
    }
    const int which = wide ? 2 : f32 ? 1 : 0;
    e = launch_kernel(kernel[which], dim3(2 * pairs), dim3(W_THREADS), size_of[which], s, p);
    if (e != cudaSuccess || l.splits == 1) return e;
    const int64_t rows = a.experts * a.n, across = ceil_div(a.k, 1024);
    const int64_t down = ceil_div(152 * 8, across);
    return launch_kernel(weight_grad_join_kernel,
                         dim3(static_cast<unsigned>(across),
                              static_cast<unsigned>(rows < down ? rows : down)),
                         dim3(256), 0, s, p);
}

cudaError_t ops_status(cudaStream_t s, int* code) {
    *code = 0;
    void* words[2];
    cudaError_t e = cudaGetSymbolAddress(&words[0], g_ops_err);
    if (e == cudaSuccess) e = norm_error_word(&words[1]);
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
        int c = 0;
        e = cudaMemcpyAsync(&c, words[i], sizeof(int), cudaMemcpyDeviceToHost, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e == cudaSuccess && c) {
            *code = c;
            e = cudaMemsetAsync(words[i], 0, sizeof(int), s);
            if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        }
    }
    return e;
}

}  // namespace ops
}  // namespace muon
