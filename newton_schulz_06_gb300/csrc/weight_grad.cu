// The weight gradient of a product from an 8-bit checkpoint
// (muon_weight_grad): G = dY^T X (+ C), one matrix or one per expert.
//
// Both operands have their long axis, the tokens, as rows: dY is tokens x n
// and the checkpoint tokens x k, so the tensor cores read both as MN-major
// operands and no transpose is made.  A CTA pair (tcgen05 cta_group::2)
// computes a 256 x 256 tile of G, 64 tokens a step: each CTA loads its 128
// columns of dY (bf16) and of the checkpoint (8 bits) with TMA, eight warps
// turn the latter into bf16 in the tensor cores' swizzled layout, and the
// leader issues the products.  A checkpoint's value q 2^(e - 133) is exact in
// bf16, so the operands are exact and the sums fp32; the norm's weight and
// bias act on the sums, in the epilogue:
//     sum_t dy[t][i] (h[t][j] w[j] + b[j]) = w[j] G0[i][j] + b[j] sum_t dy[t][i].
//
// Roles in a CTA: warp 0 loads, warp 1 issues the products (leader only),
// warps 2-5 write tiles out, warps 6-13 decode.  Two accumulators in tensor
// memory, so a tile is written out while the next one's products run.  Pairs
// walk the tiles in turn; how many tokens a tile has is read from the offsets
// on the device, and every role finds the same number.
//
// Every wait is bounded; one that runs out raises g_ops_err (muon_ops_sync).
#include <cstdlib>

#include <cudaTypedefs.h>

#include "ops_internal.h"
#include "tc_wait.cuh"

namespace muon {
namespace ops {
namespace {

using namespace ptx;

constexpr int W_STAGES = 5;
constexpr int W_TOK = 64;                          // tokens a step
constexpr int W_BOX = W_TOK * 64 * 2;              // 64 bf16 columns of a step
constexpr int W_RBOX = W_TOK * 64;                 // 64 columns of a step in 8 bits
constexpr int W_A_BYTES = 2 * W_BOX;
constexpr int W_B_BYTES = 2 * W_BOX;
constexpr int W_R_BYTES = 2 * W_RBOX;
constexpr int W_TX = W_A_BYTES + W_R_BYTES;
constexpr int W_EPI_WARPS = 4;
constexpr int W_DEC_WARPS = 8;                     // that decode one step
constexpr int W_DEC_GROUPS = 2;                    // steps in turn
constexpr int W_DEC_WARP0 = 2 + W_EPI_WARPS;
constexpr int W_THREADS = 32 * (W_DEC_WARP0 + W_DEC_GROUPS * W_DEC_WARPS);
constexpr int W_BLK = 32 * 64;                     // a staged block: 32 rows of 64 bytes
constexpr int W_EPI_BYTES = 2 * W_BLK;             // two of them a warp
constexpr int W_TMEM_COLS = 512;
constexpr int W_PAIRS = 76;                        // a pair per two of the 152 SMs
constexpr int W_EPI_OFF = W_STAGES * (W_A_BYTES + W_B_BYTES + W_R_BYTES) + 1024;
constexpr int W_SMEM = W_EPI_OFF + W_EPI_WARPS * W_EPI_BYTES + 1024;
static_assert(W_SMEM <= 232448, "shared memory per CTA");
constexpr int COLSUM_PARTS = 16;
constexpr int BAND = 8;
// fp32 results: the tensor cores cut a running sum off at its last place, so
// that it shrinks by about 7e-9 of itself a product of 16 tokens (measured);
// after this many steps it is added to a sum that is rounded to nearest.
constexpr int CHUNK_STEPS = 16;

__device__ int g_ops_err;

struct WgLaunch {
    CUtensorMap tm_dy;       // dY: dims {n, rows}, box {64, 64}, 128-byte swizzle
    CUtensorMap tm_q;        // q: dims {k, rows}, box {64, 64}, 64-byte swizzle
    // where tiles go, if TMA can store there (tma_out): G, or the partial
    // sums of a split; boxes of 32 rows of 64 bytes, 64-byte swizzle
    CUtensorMap tm_out;
    int32_t tma_out;
    int32_t c_vec;           // C's rows allow 16-byte loads
    int32_t chunk;           // steps that one accumulator sums (0: all of a tile's)
    muon_weight_grad_args a;
    const float* colsum;     // parts x experts x n sums of dY's columns (bias), or null
    int32_t colsum_parts;
    float* part;             // splits > 1: splits x experts x n x ld_part partial sums
    int64_t ld_part;
    int32_t splits;
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
__device__ __forceinline__ Item item_at(const WgLaunch& p, int32_t it) {
    const uint32_t per = static_cast<uint32_t>(p.tiles_n) * p.tiles_k;
    const uint32_t es = static_cast<uint32_t>(it) / per;
    const uint32_t w = it - es * per;
    Item x;
    x.e = static_cast<int32_t>(es / p.splits);
    x.split = static_cast<int32_t>(es - uint32_t(x.e) * p.splits);
    // bands of 8 tiles of n, column by column: the tiles that run together
    // share their rows of dY and of the checkpoint in L2
    const uint32_t band = w / (BAND * p.tiles_k);
    const uint32_t high = min(BAND, p.tiles_n - static_cast<int>(band) * BAND);
    const uint32_t in = w - band * BAND * p.tiles_k;
    x.k0 = static_cast<int32_t>(in / high) * 256;
    x.n0 = static_cast<int32_t>(band * BAND + in % high) * 256;
    int64_t begin, end;
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
// wait for every load in flight (measured: the decoding warps' scale loads,
// a third of the kernel's time).
__device__ __forceinline__ void arrive_leader(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Four 8-bit values of a word as bf16 pairs, times s (a power of two in both
// halves), all exact.  0x4300 | (q & 127) is the bf16 number 128 + (q & 127),
// and 0x4300 | (q & 128) is 128 or, where q is negative, 256: their
// difference is q.
__device__ __forceinline__ uint2 decode4(uint32_t w, __nv_bfloat162 s) {
    const uint32_t mag = w & 0x7f7f7f7fu, neg = w & 0x80808080u;
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t m = __byte_perm(mag, 0x43434343u, i ? 0x4342u : 0x4140u);
        const uint32_t c = __byte_perm(neg, 0x43434343u, i ? 0x4342u : 0x4140u);
        const __nv_bfloat162 v = __hmul2(__hsub2(reinterpret_cast<const __nv_bfloat162&>(m),
                                                 reinterpret_cast<const __nv_bfloat162&>(c)), s);
        r[i] = reinterpret_cast<const uint32_t&>(v);
    }
    return make_uint2(r[0], r[1]);
}
// 2^(e - 133) in bf16 (subnormal below e = 7), NaN for e = 255; 0 for
// NO_SCALE, the mark of a token or column that is not there.
constexpr uint32_t NO_SCALE = 256;
__device__ __forceinline__ __nv_bfloat162 scale_bf16x2(uint32_t e) {
    const uint32_t b = e == NO_SCALE ? 0u
                       : e == 255u   ? 0x7fc0u
                       : e >= 7u     ? (e - 6u) << 7
                                     : 1u << e;
    const uint32_t both = b | b << 16;
    return reinterpret_cast<const __nv_bfloat162&>(both);
}

__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(tmap)),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
}
// Byte offset of 16-byte chunk q of row r in a staged block (TMA's 64-byte
// swizzle).
__device__ __forceinline__ uint32_t sw64(int r, int q) {
    return static_cast<uint32_t>(r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
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
    for (int q = 0; q < p.colsum_parts; ++q)
        s += p.colsum[(int64_t(q) * p.a.experts + e) * p.a.n + i];
    return s;
}

// v += C[at .. at + 31], of which `left` are in the row.
__device__ __forceinline__ void add_c(const WgLaunch& p, int64_t at, int left, float (&v)[32]) {
    if (left >= 32 && p.c_vec) {
        if (p.a.g_dtype == MUON_F32) {
            const float4* c = reinterpret_cast<const float4*>(static_cast<const float*>(p.a.c) + at);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 f = c[q];
                v[4 * q] += f.x;
                v[4 * q + 1] += f.y;
                v[4 * q + 2] += f.z;
                v[4 * q + 3] += f.w;
            }
        } else {
            const __nv_bfloat16* c = static_cast<const __nv_bfloat16*>(p.a.c) + at;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f[8];
                load8_bf16(c + 8 * q, f);
#pragma unroll
                for (int u = 0; u < 8; ++u) v[8 * q + u] += f[u];
            }
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < 32; ++u)
        if (u < left) v[u] += load_any(p.a.c, p.a.g_dtype, at + u);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(W_THREADS, 1)
    weight_grad_kernel(const __grid_constant__ WgLaunch p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + W_STAGES * W_A_BYTES;
    uint8_t* sR = sB + W_STAGES * W_B_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sR + W_STAGES * W_R_BYTES);
    uint64_t* full_bar = bars;                      // this CTA's loads of a stage
    uint64_t* ready_bar = bars + W_STAGES;          // both CTAs' decoded stage (leader's)
    uint64_t* empty_bar = bars + 2 * W_STAGES;      // the products have read a stage
    uint64_t* tfull_bar = bars + 3 * W_STAGES;
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
        for (int s = 0; s < W_STAGES; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&ready_bar[s]), 2 * W_DEC_WARPS);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
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
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    grid_dependency_wait();
    allow_dependent_launch();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t limit = p.wait_limit_ns;

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued[W_STAGES];
            for (int s = 0; s < W_STAGES; ++s) issued[s] = 0;
            bool ok = true;
            for (int32_t it = pair; ok && it < p.items; it += npairs) {
                const Item x = item_at(p, it);
                const int a0 = x.n0 + static_cast<int>(rank) * 128;
                const int b0 = x.k0 + static_cast<int>(rank) * 128;
                for (int s = 0; s < x.steps; ++s) {
                    if (!wait_soon(smem_u32(&empty_bar[stage]), phase ^ 1, abort_flag, &g_ops_err,
                                   limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full_bar[stage]);
                    const int t = x.t0 + s * W_TOK;
                    mbar_expect_tx(fb, W_TX);
                    const uint32_t a_dst = smem_u32(sA + stage * W_A_BYTES);
                    const uint32_t r_dst = smem_u32(sR + stage * W_R_BYTES);
                    tma_load_2d(r_dst, &p.tm_q, fb, b0, t);
                    tma_load_2d(r_dst + W_RBOX, &p.tm_q, fb, b0 + 64, t);
                    tma_load_2d(a_dst, &p.tm_dy, fb, a0, t);
                    tma_load_2d(a_dst + W_BOX, &p.tm_dy, fb, a0 + 64, t);
                    issued[stage] = static_cast<int>(phase) + 1;
                    if (++stage == W_STAGES) { stage = 0; phase ^= 1; }
                }
            }
            if (!ok)
                for (int s = 0; s < W_STAGES; ++s)
                    if (issued[s])
                        wait_quiet(smem_u32(&full_bar[s]), static_cast<uint32_t>(issued[s] - 1),
                                   limit);
        }
    } else if (warp == 1) {
        // ------------------------------------------------- products (leader)
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            uint32_t uses[2] = {0, 0};    // of each accumulator
            uint32_t first = 0;           // the one that the tile starts in
            bool ok = true, any = false;
            // both operands MN-major: two 64-wide halves W_BOX apart, token
            // rows of 128 bytes, 16 of them (2048 bytes) a product
            const uint64_t a_desc = smem_desc(smem_u32(sA), W_BOX, 1024);
            const uint64_t b_desc = smem_desc(smem_u32(sB), W_BOX, 1024);
            const uint32_t idesc = instr_desc(256, 256, 1) | (1u << 15);
            for (int32_t it = pair; ok && it < p.items; it += npairs) {
                const Item x = item_at(p, it);
                if (x.steps == 0) continue;
                const int chunk = p.chunk ? p.chunk : x.steps;
                for (int s0 = 0; ok && s0 < x.steps; s0 += chunk) {
                    const uint32_t acc = s0 ? first ^ 1 : first;
                    const uint32_t use = acc ? uses[1]++ : uses[0]++;
                    if (!wait_soon(smem_u32(&tempty_bar[acc]), (use & 1) ^ 1, abort_flag, &g_ops_err,
                                   limit)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + acc * 256;
                    const int s1 = min(s0 + chunk, x.steps);
                    for (int s = s0; s < s1; ++s) {
                        if (!wait_soon(smem_u32(&ready_bar[stage]), phase, abort_flag, &g_ops_err,
                                       limit)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = a_desc + static_cast<uint64_t>(stage) * (W_A_BYTES >> 4);
                        const uint64_t bd = b_desc + static_cast<uint64_t>(stage) * (W_B_BYTES >> 4);
#pragma unroll
                        for (int kk = 0; kk < W_TOK / 16; ++kk)
                            mma_pair(d_tmem, ad + static_cast<uint64_t>(kk * (2048 >> 4)),
                                     bd + static_cast<uint64_t>(kk * (2048 >> 4)), idesc,
                                     (s > s0 || kk > 0) ? 1u : 0u);
                        any = true;
                        commit_pair_multicast(smem_u32(&empty_bar[stage]));
                        if (++stage == W_STAGES) { stage = 0; phase ^= 1; }
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
        // Two groups of warps take the steps in turn.  A thread turns one
        // block of 32 values of one token: 16 tokens and the two blocks of a
        // 64-wide box in a warp, so that eight lanes' 16-byte accesses fall
        // on all banks in both swizzles.
        const int group = (warp - W_DEC_WARP0) / W_DEC_WARPS;
        const int dw = (warp - W_DEC_WARP0) % W_DEC_WARPS;
        const int box = dw & 1;
        const int row = (dw >> 1) * 16 + (lane >> 1);
        const int blk = lane & 1;
        const uint32_t src = box * W_RBOX + row * 64;
        const uint32_t src_sw = (row >> 1) & 3;
        const uint32_t dst = box * W_BOX + row * 128;
        const uint32_t dst_sw = row & 7;
        const int nblk = static_cast<int>((p.a.k + CKPT_BLOCK - 1) / CKPT_BLOCK);
        const uint32_t ready_leader = map_to_rank(smem_u32(ready_bar), 0);
        uint32_t before = 0;          // steps of the tiles before this one
        int stage = group;
        uint32_t phase = 0;
        bool ok = true;
        for (int32_t it = pair; ok && it < p.items; it += npairs) {
            const Item x = item_at(p, it);
            const int eb = (x.k0 + static_cast<int>(rank) * 128) / CKPT_BLOCK + box * 2 + blk;
            const uint8_t* ep = p.a.saved.e + eb;
            const bool col_ok = eb < nblk;
            const int first = (group - static_cast<int>(before)) & (W_DEC_GROUPS - 1);
            before += x.steps;
            // the scale bytes come four of this group's steps at a time, one
            // round ahead
            uint32_t nxt[4];
            auto fetch = [&](int s) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int su = s + u * W_DEC_GROUPS;
                    const int64_t t = int64_t(x.t0) + su * W_TOK + row;
                    nxt[u] = (col_ok && su < x.steps && t < x.end) ? ep[t * p.a.saved.ld_e] : NO_SCALE;
                }
            };
            fetch(first);
            for (int s = first; ok && s < x.steps; s += 4 * W_DEC_GROUPS) {
                uint32_t cur[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) cur[u] = nxt[u];
                fetch(s + 4 * W_DEC_GROUPS);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int su = s + u * W_DEC_GROUPS;
                    if (su >= x.steps) break;
                    const uint32_t fb = smem_u32(&full_bar[stage]);
                    const bool got = wait_soon(fb, phase, abort_flag, &g_ops_err, limit);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    const __nv_bfloat162 sc = scale_bf16x2(cur[u]);
                    const uint8_t* r = sR + stage * W_R_BYTES + src;
                    uint8_t* b = sB + stage * W_B_BYTES + dst;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 q = *reinterpret_cast<const uint4*>(
                            r + (((blk * 2 + h) ^ src_sw) << 4));
                        const uint2 v0 = decode4(q.x, sc), v1 = decode4(q.y, sc);
                        const uint2 v2 = decode4(q.z, sc), v3 = decode4(q.w, sc);
                        *reinterpret_cast<uint4*>(b + (((blk * 4 + h * 2) ^ dst_sw) << 4)) =
                            make_uint4(v0.x, v0.y, v1.x, v1.y);
                        *reinterpret_cast<uint4*>(b + (((blk * 4 + h * 2 + 1) ^ dst_sw) << 4)) =
                            make_uint4(v2.x, v2.y, v3.x, v3.y);
                    }
                    const int left = x.end - (x.t0 + su * W_TOK);
                    if (left < W_TOK) {
                        // tokens of the next matrix in dY's stage: 0 times a
                        // NaN of theirs would be a NaN here
                        uint8_t* a = sA + stage * W_A_BYTES;
                        for (int c = dw * 32 + lane; c < (W_TOK - left) * 16; c += W_DEC_WARPS * 32)
                            *reinterpret_cast<uint4*>(a + (c >> 3 & 1) * W_BOX +
                                                      (left + (c >> 4)) * 128 + (c & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_leader(ready_leader + 8 * stage);
                    stage += W_DEC_GROUPS;
                    if (stage >= W_STAGES) { stage -= W_STAGES; phase ^= 1; }
                }
            }
        }
    } else {
        // --------------------------------------------------------- write out
        const int lg = warp & 3;                    // this warp's 32 TMEM lanes
        uint8_t* const stage0 = smem + W_EPI_OFF + (warp - 2) * W_EPI_BYTES;
        const uint32_t tempty_leader = map_to_rank(smem_u32(tempty_bar), 0);
        const bool f32_out = p.splits > 1 || p.a.g_dtype == MUON_F32;
        uint32_t stores = 0;
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
        // the next of the warp's two staging blocks, once its last TMA store
        // has read it
        auto next_block = [&]() {
            if (lane == 0) bulk_wait_read1();
            __syncwarp();
            return stage0 + (stores++ & 1u) * W_BLK;
        };
        auto store_block = [&](uint8_t* blk, int x, int y, int z) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&p.tm_out, smem_u32(blk), x, y, z);
                bulk_commit();
            }
        };
        for (int32_t it = pair; ok && it < p.items; it += npairs) {
            const Item x = item_at(p, it);
            const uint32_t tlane = tmem_base + (static_cast<uint32_t>(lg * 32) << 16);
            const uint32_t taddr = tlane + first * 256;
            if (x.steps) {
                if (!wait_full(first)) {
                    ok = false;
                    break;
                }
                // later chunks of the tokens: added up in fp32, rounded to
                // nearest
                const int chunk = p.chunk ? p.chunk : x.steps;
                for (int s0 = chunk; s0 < x.steps; s0 += chunk) {
                    if (!wait_full(first ^ 1)) {
                        ok = false;
                        break;
                    }
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        float v[32], w[32];
                        tmem_ld32(taddr + 32 * c, v);
                        tmem_ld32(tlane + (first ^ 1) * 256 + 32 * c, w);
#pragma unroll
                        for (int u = 0; u < 32; ++u) v[u] += w[u];
                        tmem_st32(taddr + 32 * c, v);
                    }
                    release(first ^ 1);
                }
                if (!ok) break;
            }
            const int r0 = x.n0 + static_cast<int>(rank) * 128 + lg * 32;
            const int n = static_cast<int>(p.a.n), k = static_cast<int>(p.a.k);
            const int rows = min(32, n - r0);
            const bool apply = p.splits == 1;
            const float sum = (apply && p.colsum && lane < rows) ? column_sum(p, x.e, r0 + lane) : 0.f;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                const int j0 = x.k0 + 32 * c;
                if (rows <= 0 || j0 >= k) break;
                float v[32];
                if (x.steps) {
                    tmem_ld32(taddr + 32 * c, v);
                } else {
#pragma unroll
                    for (int u = 0; u < 32; ++u) v[u] = 0.f;
                }
                if (apply && (p.a.weight || p.a.bias)) {
                    const float wl = p.a.weight && j0 + lane < k ? p.a.weight[j0 + lane] : 1.f;
                    const float bl = p.a.bias && j0 + lane < k ? p.a.bias[j0 + lane] : 0.f;
#pragma unroll
                    for (int u = 0; u < 32; ++u)
                        v[u] = fmaf(__shfl_sync(0xffffffffu, bl, u), sum,
                                    v[u] * __shfl_sync(0xffffffffu, wl, u));
                }
                if (p.tma_out) {
                    if (apply && p.a.c && lane < rows) {
                        const int64_t at = x.e * p.a.stride_c + int64_t(r0 + lane) * p.a.ld_c + j0;
                        add_c(p, at, k - j0, v);
                    }
                    const int z = apply ? x.e : static_cast<int>(x.split * p.a.experts + x.e);
                    if (f32_out) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (j0 + 16 * h >= k) break;
                            uint8_t* blk = next_block();
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                *reinterpret_cast<float4*>(blk + sw64(lane, q)) =
                                    make_float4(v[16 * h + 4 * q], v[16 * h + 4 * q + 1],
                                                v[16 * h + 4 * q + 2], v[16 * h + 4 * q + 3]);
                            store_block(blk, j0 + 16 * h, r0, z);
                        }
                    } else {
                        uint8_t* blk = next_block();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float t[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) t[u] = v[8 * q + u];
                            store8_bf16(reinterpret_cast<__nv_bfloat16*>(blk + sw64(lane, q)), t);
                        }
                        store_block(blk, j0, r0, z);
                    }
                    continue;
                }
                // rows that TMA cannot store to: turned in shared memory, then
                // row by row
                float* blk = reinterpret_cast<float*>(stage0);
#pragma unroll
                for (int u = 0; u < 32; ++u) blk[lane * 32 + (u ^ lane)] = v[u];
                __syncwarp();
                if (j0 + lane < k) {
                    int64_t g_at = x.e * p.a.stride_g + int64_t(r0) * p.a.ld_g + j0 + lane;
                    int64_t c_at = x.e * p.a.stride_c + int64_t(r0) * p.a.ld_c + j0 + lane;
#pragma unroll 4
                    for (int r = 0; r < rows; ++r) {
                        float g = blk[r * 32 + (lane ^ r)];
                        if (p.a.c) g += load_any(p.a.c, p.a.g_dtype, c_at);
                        store_any(p.a.g, p.a.g_dtype, g_at, g);
                        g_at += p.a.ld_g;
                        c_at += p.a.ld_c;
                    }
                }
                __syncwarp();
            }
            if (x.steps) {
                release(first);
                first ^= 1;
            }
        }
        if (lane == 0) bulk_wait_all0();
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

// The splits' partial sums in order, then the epilogue.
__global__ void __launch_bounds__(256) weight_grad_join_kernel(const __grid_constant__ WgLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t n = p.a.n, k = p.a.k, size = p.a.experts * n * k;
    for (int64_t u = blockIdx.x * int64_t(256) + threadIdx.x; u < size; u += int64_t(gridDim.x) * 256) {
        const int64_t j = u % k, i = u / k % n, e = u / (n * k);
        float g = 0.f;
        const int64_t at = (e * n + i) * p.ld_part + j;
        for (int s = 0; s < p.splits; ++s) g += p.part[s * p.a.experts * n * p.ld_part + at];
        finish(p.a, e, i, j, g, p.a.weight ? p.a.weight[j] : 1.f, p.a.bias ? p.a.bias[j] : 0.f,
               p.colsum ? column_sum(p, e, i) : 0.f);
    }
}

// Sums of dY's columns over each matrix's tokens (gridDim.z parts of them):
// 64 columns and 4 rows at a time in a block.
__global__ void __launch_bounds__(256)
    colsum_kernel(const __grid_constant__ muon_weight_grad_args a, float* out) {
    __shared__ float red[256];
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t i = blockIdx.x * int64_t(64) + (threadIdx.x & 63);
    for (int64_t e = blockIdx.y; e < a.experts; e += gridDim.y) {
        int64_t begin, end;
        segment(a, e, &begin, &end);
        const int64_t len = end - begin;
        const int64_t t0 = begin + len * blockIdx.z / gridDim.z;
        const int64_t t1 = begin + len * (blockIdx.z + 1) / gridDim.z;
        float s = 0.f;
        if (i < a.n)
            for (int64_t t = t0 + (threadIdx.x >> 6); t < t1; t += 4)
                s += __bfloat162float(static_cast<const __nv_bfloat16*>(a.dy)[t * a.ld_dy + i]);
        __syncthreads();
        red[threadIdx.x] = s;
        __syncthreads();
        if (threadIdx.x < 64 && i < a.n)
            out[(blockIdx.z * a.experts + e) * a.n + i] =
                (red[threadIdx.x] + red[threadIdx.x + 64]) +
                (red[threadIdx.x + 128] + red[threadIdx.x + 192]);
    }
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
// each of eight steps or more on average.
int split_count(const muon_weight_grad_args& a) {
    const int64_t steps = ceil_div(ceil_div(a.rows, a.experts), W_TOK);
    int64_t s = W_PAIRS / tiles(a);
    if (s > steps / 8) s = steps / 8;
    return static_cast<int>(s < 1 ? 1 : s);
}

int grid_for(int64_t items) {
    const int64_t g = ceil_div(items, 256);
    return static_cast<int>(g < 1 ? 1 : g > 152 * 8 ? 152 * 8 : g);
}

struct Layout {
    size_t colsum = 0, dy = 0, part = 0, bytes = 0;
    int colsum_parts = 0, splits = 1;
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
        l.ld_part = ceil_div(a.k, 4) * 4;
        l.bytes += align256(size_t(l.splits) * a.experts * a.n * l.ld_part * 4);
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

// A map to store tiles of `count` matrices of n x k with: boxes of 32 rows of
// 64 bytes.
bool encode_out(CUtensorMap* tm, bool f32, void* base, int64_t count, int64_t n, int64_t k,
                int64_t ld, int64_t stride) {
    if (!encoder()) return false;
    const size_t size = f32 ? 4 : 2;
    cuuint64_t dims[3] = {cuuint64_t(k), cuuint64_t(n), cuuint64_t(count)};
    cuuint64_t strides[2] = {cuuint64_t(ld) * size, cuuint64_t(stride) * size};
    cuuint32_t box[3] = {cuuint32_t(64 / size), 32, 1}, el[3] = {1, 1, 1};
    return encoder()(tm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     base, dims, strides, box, el, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether 16-byte accesses and TMA suit a gradient's rows.
bool rows_aligned(const void* p, size_t size, const muon_weight_grad_args& a, int64_t ld,
                  int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.n <= 1 || ld * size % 16 == 0) &&
           (a.experts <= 1 || stride * size % 16 == 0);
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
    p.tiles_n = static_cast<int32_t>(ceil_div(a.n, 256));
    p.tiles_k = static_cast<int32_t>(ceil_div(a.k, 256));
    p.items = static_cast<int32_t>(tiles(a) * l.splits);
    p.wait_limit_ns = wait_limit_ns();
    const size_t size = a.g_dtype == MUON_F32 ? 4 : 2;
    if (a.g_dtype == MUON_F32) p.chunk = CHUNK_STEPS;
    if (a.c) p.c_vec = rows_aligned(a.c, size, a, a.ld_c, a.stride_c);
    if (l.splits > 1) {
        p.part = reinterpret_cast<float*>(base + l.part);
        p.ld_part = l.ld_part;
        p.tma_out = 1;
        if (!encode_out(&p.tm_out, true, p.part, l.splits * a.experts, a.n, a.k, l.ld_part,
                        a.n * l.ld_part))
            return cudaErrorInvalidValue;
    } else if (rows_aligned(a.g, size, a, a.ld_g, a.stride_g)) {
        const int64_t ld = a.n > 1 ? a.ld_g : ceil_div(a.k, 8) * 8;
        p.tma_out = 1;
        if (!encode_out(&p.tm_out, size == 4, a.g, a.experts, a.n, a.k, ld,
                        a.experts > 1 ? a.stride_g : a.n * ld))
            return cudaErrorInvalidValue;
    }
    cudaError_t e;
    if (a.bias) {
        p.colsum = reinterpret_cast<float*>(base + l.colsum);
        p.colsum_parts = l.colsum_parts;
        e = launch_kernel(colsum_kernel,
                          dim3(static_cast<unsigned>(ceil_div(a.n, 64)),
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
    static int attr_done[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(weight_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 W_SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = 1;
    }
    const int pairs = p.items < W_PAIRS ? p.items : W_PAIRS;
    e = launch_kernel(weight_grad_kernel, dim3(2 * pairs), dim3(W_THREADS), W_SMEM, s, p);
    if (e != cudaSuccess || l.splits == 1) return e;
    return launch_kernel(weight_grad_join_kernel, dim3(grid_for(a.experts * a.n * a.k)), dim3(256),
                         0, s, p);
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
