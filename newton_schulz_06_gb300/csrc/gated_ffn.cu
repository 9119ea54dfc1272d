// The gated feed-forward block and its gradient (muon_gated_ffn,
// muon_gated_ffn_grad): five grouped products, one kernel each, over all
// experts' rows at once.
//
//   UP      h = act(x Wg^T) * (x Wu^T)  (g and u kept if asked for)
//   DOWN    y = h Wd^T
//   DHIDDEN dh = dy Wd, at once turned into dg, du and h
//   DX      dx = dg Wg + du Wu, one sum over both products
//   DW      dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//
// All are out[n][m] = sum over k of B[n][k] A[m][k].  A CTA pair (tcgen05
// cta_group::2) computes 256 m x up to 256 n: the matrices of an expert are the
// instruction's M side and its rows (tokens) the N side, because N may be any
// multiple of 32 while M is always 256: an expert's last rows then cost what
// they are, where a last tile of 256 tokens costs 256 (128 experts of about 500
// tokens would waste a quarter).  UP takes 64 rows of Wg and the same 64 of Wu
// as a CTA's 128 rows, so that a tile has both factors of its h.
//
// TMEM holds m in lanes and n in columns, memory wants m along rows.  Sums that
// leave as bf16 (DOWN, DX, DW) are turned by stmatrix, 32 columns at a time;
// those that something is still done to (UP, DHIDDEN, fp32 or added gradients,
// parts of a split) go through shared memory in fp32, 16 columns at a time, after
// which a thread has eight neighbours of an output row, reads what it needs
// beside them, and stores 16 bytes.
//
// Roles in a CTA: warps 0 and 11 load (TMA), warp 1 issues the products (the
// pair's leader only), warps 2-9 are the epilogue, in two teams of four that
// take a tile's columns in turn, warp 10 lays zeros over what DW loads past an
// expert's last token, warp 12 finds the tiles.  Two accumulators, so that a tile
// is written out while the next one's products run.  Pairs walk the tiles in turn.
//
// What bounds it (times in loops of 10 to 30 ms, over several boxes).  Long sums:
// the tensor cores, at the rate that the power limit leaves the library's product
// too (8192 tokens of 4096 x 11008: forward 1219 to 1249 us, 1.79 PFLOP/s; DX 824 to
// 851, 1.76; DW, both of whose operands have k as rows, 1278 to 1369, 1.68; DHIDDEN
// 496 to 504, 1.48, whose write-out reads two and writes three values a sum).
// 128 experts of 2048 x 768 over 65536 rows: forward 411 to 435 us and DX 287 to
// 315, the loads of tiles that are not full and the ends of tiles of 12 to 32
// steps; DHIDDEN 203 to 215, memory (5.6 TB/s); DW 491 to 533, tiles of eight
// steps whose 1.2 GB of results leave meanwhile (442 us without storing them, where
// it took 510).  In longer loops the power limit brings the clocks from 1.9 to 1.48
// GHz, and that forward takes 480 to 495.  Three teams that write out instead of
// two made no difference.
//
// Every wait is bounded; one that runs out raises g_ffn_err (muon_ops_sync).
#include <algorithm>

#include <cudaTypedefs.h>

#include "ffn_drain.h"
#include "ops_internal.h"
#include "tc_wait.cuh"

namespace muon {
namespace ops {
namespace {

using namespace ptx;

constexpr int F_K = 64;                            // of the sums, a step
constexpr int F_BOX = 64 * 64 * 2;                 // a TMA box: 64 rows of 64 bf16
constexpr int F_OP_BYTES = 2 * F_BOX;              // an operand's part of a CTA, a step
constexpr int F_STAGE_BYTES = 2 * F_OP_BYTES;
static_assert(F_BOX == DRAIN_BOX, "what the drain counts");
constexpr int F_EXPERTS = 1024;
constexpr int F_COLS = 16;                         // columns that are turned at a time in fp32
constexpr int F_ROW = 132;                         // floats of a turned row: 128 and a gap
constexpr int F_COLS16 = 32;                       // and in bf16
constexpr int F_ROW16 = 136;
constexpr int F_TURN_BYTES = F_COLS16 * F_ROW16 * 2;
static_assert(F_TURN_BYTES >= F_COLS * F_ROW * 4 && F_TURN_BYTES % 16 == 0, "a team's buffer");
constexpr int F_KEPT_BYTES = 2 * 4 * 128 * 16;     // a team's g and u of 16 columns, twice (DHIDDEN)
constexpr int F_EPI_WARPS = 8;
constexpr int F_CLEAR_WARP = 2 + F_EPI_WARPS;
constexpr int F_LOAD_B_WARP = F_CLEAR_WARP + 1;
constexpr int F_TILE_WARP = F_LOAD_B_WARP + 1;
constexpr int F_THREADS = 32 * (F_TILE_WARP + 1);
constexpr int F_ITEMS = 4;                         // tiles found ahead
constexpr int F_TMEM_COLS = 512;
constexpr int F_PAIRS = 76;                        // a pair per two of the 152 SMs
constexpr int F_BAND = 8;
// DW's sums are as long as an expert has tokens, and the tensor cores cut a
// running sum off at its last place, so that sums of one sign shrink, by 7.6e-8 a
// product of 16 tokens (200003 of them in one sum lose 1.14e-3).  Two cuts of a
// whole place each are the most, 2^-23 of a sum that is on average 0.375 of its
// end's place: 9e-8 a product.  After this many steps of four products a tile's
// sums are added up to nearest, so that at most 4.6e-5 is lost of a bf16 result,
// a fortieth of its own rounding, and 2.3e-5 of an fp32 one, about what the
// rounding of dg, du and h leaves in a sum of 4096.  Whole gradient: 65536
// tokens of 4096 x 4096, bf16 8040 -> 8280 us, fp32 8370 -> 8680; 4097 of 7168 x
// 2048, fp32 441 -> 462, and 477 with the sums so far fetched only when added.
constexpr int F_CHUNK_BF16 = 128, F_CHUNK_F32 = 64;

__device__ int g_ffn_err;

enum Op { UP, DOWN, DHIDDEN, DX, DW };

// Where things are in shared memory.
template <int OP>
struct Space {
    static constexpr int STAGES = OP == DHIDDEN ? 5 : 6;
    static constexpr int BARS = STAGES * F_STAGE_BYTES;
    static constexpr int ASKED = BARS + 320;                 // loads asked for, for an abort
    static constexpr int ITEMS = BARS + 384;                 // tiles handed out
    static constexpr int TURN = ITEMS + 256;
    static constexpr int KEPT = TURN + 2 * F_TURN_BYTES;     // two teams'
    static constexpr int TABLE = KEPT + (OP == DHIDDEN ? 2 * F_KEPT_BYTES : 0);
    static constexpr int BYTES = TABLE + 2 * (F_EXPERTS + 1) * 4 + 1024;
    static_assert(BYTES <= 232448, "shared memory per CTA");
    static_assert(8 * (4 * STAGES + 5 + 2 * F_ITEMS) + 8 <= 320 && 3 * sizeof(Asked) <= 64, "barriers and counts");
};

// One output matrix (or as many as there are experts).
struct Out {
    void* p;
    int64_t ld, stride;
    int32_t vec;             // rows lie on 16 bytes
};

// Zeros come by maps of one row, from rows past it: nothing is read.
constexpr int F_NO_ROW = 64;

// One of the sums' operand pairs: a is M's side, b is N's (b64: in boxes of 64,
// for the tiles that have no more a CTA).  wide_a, wide_b: a box has 128
// columns of an operand whose rows are k (blocks()).
struct Maps {
    CUtensorMap a, b, b64;
    int32_t wide_a, wide_b;
};

struct FfnLaunch {
    Maps maps[3];            // UP: Wg with x, Wu; DX: Wg with dg, Wu with du; DW: its three products
    CUtensorMap zeros[4];    // DW: boxes of 1, 2, 4 and 8 rows of 64
    Out out[3];              // UP: h, g, u; DHIDDEN: dg, du, h; DW: dWg, dWu, dWd
    const void *gate, *up;   // DHIDDEN reads them
    int64_t ld_kept;
    int32_t vec;             // UP, DHIDDEN: rows of all that is read and written here lie on 16 bytes
    const int32_t* offsets;
    int64_t rows;
    int32_t experts;
    int32_t m[2], k;         // extents; DW: m[0] is hidden, m[1] inner; else m[0]
    int32_t a_by_expert[3];  // an expert's own matrix, or one for all
    int32_t products;        // DW: which of them, as bits
    int32_t tile_n;          // rows of N a tile, a multiple of 32
    int32_t splits;          // parts of the sums that tiles of their own take
    int32_t chunk;           // DW: steps that one accumulator sums
    float4* held;            // a tile's sums while its next chunk runs
    float* part;             // splits > 1: their sums, split by split,
    int64_t part_stride;
    int64_t part_ld[2];      // in rows of these lengths (by m's extent; UP: g, then u),
    int64_t part_at[3];      // DW: a product's after another's
    int32_t act;
    int32_t out_f32, accumulate;
    unsigned long long wait_limit_ns;
};

// x / d by d's reciprocal, a sixth of the time of a division.
struct Divisor {
    uint32_t d;
    float inv;
    __device__ __forceinline__ void set(uint32_t v) {
        d = v;
        inv = __frcp_rn(__uint2float_rn(v));
    }
    __device__ __forceinline__ uint32_t of(uint32_t x) const {
        uint32_t q = __float2uint_rz(__uint2float_rz(x) * inv);
        int32_t r = static_cast<int32_t>(x - q * d);
        while (r < 0) {
            --q;
            r += d;
        }
        while (r >= static_cast<int32_t>(d)) {
            ++q;
            r -= d;
        }
        return q;
    }
};

// A tile.
struct alignas(16) Item {
    int32_t e, j;            // expert (below 0: there is no more), product (DW)
    int32_t m0, n0;          // its first m (UP: of h), its first row of N
    int32_t n_end;           // its rows of N end here
    int32_t n;               // the instruction's N
    int32_t steps;           // of 64,
    int32_t s0, split;       // from this one of the whole sum on; which part of it that is
    int32_t t0;              // DW: the first token
    int32_t tail;            // DW: tokens of the last step, if not 64
    // DW: the rows of the last step's last product that are not this expert's
    // (0: the step is not torn)
    __device__ __forceinline__ uint32_t gap() const { return -tail & 15; }
    int32_t chunk;           // DW: which end of a long sum this is (FIRST, LAST)
};
constexpr int FIRST = 1, LAST = 2;
static_assert(F_ITEMS * sizeof(Item) <= 256, "tiles handed out");

// The tiles' places.
template <int OP>
struct Tiles {
    const FfnLaunch& p;
    const int32_t *begin, *first;            // experts' first rows, and first rows of tiles
    int32_t total, steps;
    Divisor whole;                           // tiles of the whole sums
    Divisor tiles_m, band;                   // tiles across M, and in a band
    Divisor per, across[2], bands[2];        // DW: a matrix's tiles; by product (2: the last one)
    int32_t base[2];                         // the second and third product's first tile
    __device__ __forceinline__ Tiles(const FfnLaunch& l, const int32_t* table) : p(l) {
        begin = table;
        first = begin + p.experts + 1;
        if constexpr (OP == DW) {
            uint32_t all = 0;
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const int32_t m = (p.m[j == 2] + 255) / 256, n = (p.m[j != 2] + 255) / 256;
                if (j) base[j - 1] = all;
                all += p.products >> j & 1 ? m * n : 0;
            }
            per.set(all);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                across[i].set((p.m[i] + 255) / 256);
                bands[i].set(F_BAND * across[i].d);
            }
            whole.set(all * p.experts);
        } else {
            tiles_m.set((p.m[0] + (OP == UP ? 127 : 255)) / (OP == UP ? 128 : 256));
            band.set(F_BAND * tiles_m.d);
            whole.set(first[p.experts] * tiles_m.d);
            steps = (p.k + F_K - 1) / F_K * (OP == DX ? 2 : 1);
        }
        total = whole.d * p.splits;
    }
    __device__ __forceinline__ Item at(int32_t it) const {
        Item x;
        x.tail = 0;
        x.j = 0;
        x.chunk = FIRST | LAST;
        x.split = p.splits > 1 ? whole.of(it) : 0;
        it -= x.split * whole.d;
        int32_t in, tn, size, end, all;
        Divisor tm, b;
        if constexpr (OP == DW) {
            x.e = per.of(it);
            in = it - x.e * per.d;
            x.j = in < base[0] ? 0 : in < base[1] ? 1 : 2;
            in -= x.j == 0 ? 0 : x.j == 1 ? base[0] : base[1];
            tm = x.j == 2 ? across[1] : across[0];
            b = x.j == 2 ? bands[1] : bands[0];
            end = p.m[x.j != 2];
            size = 256;
            tn = x.j == 2 ? across[0].d : across[1].d;
            x.t0 = begin[x.e];
            const int32_t len = begin[x.e + 1] - x.t0;
            all = (len + F_K - 1) / F_K;
            x.tail = len % F_K;
        } else {
            // the expert whose tiles these are
            int32_t lo = 0, hi = p.experts;
            const int32_t row = tiles_m.of(it);
            while (hi - lo > 1) {
                const int32_t mid = (lo + hi) >> 1;
                if (first[mid] <= row) lo = mid;
                else hi = mid;
            }
            x.e = lo;
            in = it - first[lo] * tiles_m.d;
            tm = tiles_m;
            b = band;
            tn = first[lo + 1] - first[lo];
            size = p.tile_n;
            end = begin[lo + 1];
            x.t0 = 0;
            all = steps;
        }
        x.s0 = 0;
        x.steps = all;
        if (p.splits > 1) {
            x.s0 = static_cast<int32_t>(int64_t(all) * x.split / p.splits);
            const int32_t s1 = static_cast<int32_t>(int64_t(all) * (x.split + 1) / p.splits);
            x.steps = s1 - x.s0;
            x.t0 += x.s0 * F_K;
            if (s1 < all) x.tail = 0;
        }
        // bands of eight tiles of N, column by column: the tiles that run
        // together share their operands in L2 (8192 tokens of 4096 x 11008, DX:
        // 850 us; bands of four 879, of sixteen 880, of 32 923)
        const int32_t nb = b.of(in), rows = min(F_BAND, tn - nb * F_BAND);
        in -= nb * b.d;
        // in / rows, exact: in is at most 8 x 2048 (tiles across 262144)
        const int32_t m = rows == F_BAND ? in >> 3 : static_cast<int32_t>(__fdividef(in + 0.5f, rows));
        const int32_t n = nb * F_BAND + in - m * rows;
        x.m0 = m * (OP == UP ? 128 : 256);
        x.n0 = (OP == DW ? 0 : begin[x.e]) + n * size;
        x.n_end = min(end, x.n0 + size);
        x.n = (x.n_end - x.n0 + 31) & ~31;
        return x;
    }
};

__device__ __forceinline__ void load_box(uint32_t dst, const void* tmap, uint32_t cluster_bar, int x, int y,
                                         int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::"
        "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
        : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const void* tmap, uint32_t cluster_bar, int x, int y,
                                         int block, int z) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::"
        "complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(block), "r"(z), "r"(cluster_bar)
        : "memory");
}
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void read_cluster(void* to, uint32_t cluster_addr, uint32_t bytes) {
#pragma unroll 1
    for (uint32_t i = 0; i < bytes / 4; ++i)
        asm volatile("ld.shared::cluster.u32 %0, [%1];"
                     : "=r"(static_cast<uint32_t*>(to)[i])
                     : "r"(cluster_addr + 4 * i)
                     : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
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
// 16 fp32 columns of this warp's TMEM lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// 16 columns of 32 lanes as bf16 pairs of neighbouring columns, in the layout
// that stmatrix takes: r[j][i] is of columns 8 j .. 8 j + 7 and lanes 8 i .. 8 i + 7.
__device__ __forceinline__ void tmem_ld_frag(uint32_t addr, uint32_t (&r)[2][4]) {
    uint32_t v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(v[h][0]), "=r"(v[h][1]), "=r"(v[h][2]), "=r"(v[h][3]), "=r"(v[h][4]), "=r"(v[h][5]),
              "=r"(v[h][6]), "=r"(v[h][7])
            : "r"(addr + (static_cast<uint32_t>(16 * h) << 16)));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t* const p = &v[i / 2][4 * j + i % 2 * 2];
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(p[0]), __uint_as_float(p[1]));
            r[j][i] = reinterpret_cast<const uint32_t&>(b);
        }
}
// Four 8 x 8 matrices, turned: lanes 8 i .. 8 i + 7 give the places of matrix
// i's eight columns.
__device__ __forceinline__ void store_turned(uint32_t to, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
// A wait that has gone on for a while.  Where it runs out, the other CTA of the
// pair learns of it, too.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    if (wait_bounded(bar, parity, abort_flag, &g_ffn_err, limit)) return true;
    store_cluster(map_to_rank(smem_u32(const_cast<int*>(abort_flag)), cluster_rank() ^ 1), 1u);
    return false;
}
// As wait_soon, in a pair.
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_long(bar, parity, abort_flag, limit);
}
// The tiles as one warp finds them for all others: finding a tile takes 500 to
// 1200 cycles, in which a role that did it itself kept the tensor cores waiting
// (of 5000 a tile that has eight steps).
struct Feed {
    const Item* items;
    uint32_t full, empty;
    uint32_t n = 0;
    __device__ __forceinline__ Feed(const void* at, uint32_t bars)
        : items(static_cast<const Item*>(at)), full(bars), empty(bars + 8 * F_ITEMS) {}
    // The next tile, for a thread or a whole warp: false where the wait ran
    // out.
    template <bool WARP>
    __device__ __forceinline__ bool next(Item& x, volatile int* abort_flag, uint64_t limit) {
        const uint32_t slot = n % F_ITEMS;
        bool got = wait_pair(full + 8 * slot, n / F_ITEMS & 1, abort_flag, limit);
        if (WARP) got = __all_sync(0xffffffffu, got);
        if (!got) return false;
        x = items[slot];
        if (WARP) __syncwarp();
        if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(empty + 8 * slot);
        ++n;
        return true;
    }
};

// Whether a barrier's phase is over, without waiting.  Asked of the next step's
// barrier before this step's work is issued, the answer's 220 cycles are hidden
// behind it (the products' thread took 590 cycles a step otherwise, of 512 that
// the products take).
__device__ __forceinline__ bool is_over(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The same, and a wait, for a whole warp, whose lanes agree.
__device__ __forceinline__ bool is_over_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, is_over(bar, parity));
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    return __all_sync(0xffffffffu, wait_pair(bar, parity, abort_flag, limit));
}
// One lane of a whole warp.
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "elect.sync _|P, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(p));
    return p != 0;
}
// 16 bytes to shared memory, and a wait for all of this thread's.
__device__ __forceinline__ void copy16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// A barrier of one team's 128 threads.
__device__ __forceinline__ void team_sync(int team) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + team) : "memory");
}

// 1 / (1 + e^-v).  The exponential is off by 2 + 1.2 |v| units of 2^-23 and the
// quotient by 2: 3e-6 at -20, where the bf16 rounding behind them is 4e-3; below
// -87 it is 0.  (With a reciprocal rounded to nearest, UP's write-out took 1550
// cycles for 16 columns, not 600.)
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// Phi(g) = erfc(-g / sqrt(2)) / 2, where e is exp(-g^2 / 2).  With z = |g| / sqrt(2),
// erfc(z) / e is smooth: t P(t) of t = 1 / (1 + 0.43 z), where P, of degree 7, is
// fitted to a relative error of 1e-7 over 0 <= z <= 10 (where e ends).  The lower
// tail keeps all of its digits, of which (1 + erf) / 2 has lost 4 % at -5 and
// everything below -5.6, and there is no second exponential: 128 experts with
// GELU, kept and back, take 437 and 1027 us, by erff 436 and 1043, by erfcf 456
// and 1085.
__device__ __forceinline__ float normal_below(float g, float e) {
    const float t = __fdividef(1.f, fmaf(0.30405592f, fabsf(g), 1.f));
    float p = 0.036572915f;
    p = fmaf(p, t, -0.154047829f);
    p = fmaf(p, t, 0.189943648f);
    p = fmaf(p, t, -0.0411521562f);
    p = fmaf(p, t, 0.122540339f);
    p = fmaf(p, t, 0.102736251f);
    p = fmaf(p, t, 0.122146916f);
    p = fmaf(p, t, 0.12125991f);
    const float tail = p * t * e;
    return g < 0.f ? tail : 1.f - tail;
}

// a = act(g) and d = act'(g), eight at a time.
__device__ __forceinline__ void activate8(int act, const float (&g)[8], float (&a)[8], float (&d)[8]) {
    if (act == MUON_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = logistic(g[i]);
            a[i] = g[i] * s;
            d[i] = fmaf(a[i], 1.f - s, s);
        }
    } else if (act == MUON_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = __expf(-0.5f * g[i] * g[i]), c = normal_below(g[i], e);
            a[i] = g[i] * c;
            d[i] = fmaf(g[i] * 0.39894228f, e, c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // (1 + tanh z) / 2 is the logistic function of 2 z, which is 0 or 1
            // long before the limit on g^2 (no infinity to multiply by 0)
            const float q = fminf(g[i] * g[i], 1000.f), s = logistic(g[i] * fmaf(0.071354816f, q, 1.5957691f));
            a[i] = g[i] * s;
            d[i] = fmaf(a[i] * (1.f - s), fmaf(0.21406445f, q, 1.5957691f), s);
        }
    }
}

// Eight neighbours of a turned row.  The two halves are read in an order that
// lets eight threads' 16 bytes fall on all banks.
__device__ __forceinline__ void turned8(const float* row, int group, float (&v)[8]) {
    const int swap = group >> 2 & 1;
    const float4 a = *reinterpret_cast<const float4*>(row + 8 * group + 4 * swap);
    const float4 b = *reinterpret_cast<const float4*>(row + 8 * group + 4 * (swap ^ 1));
    const float4 lo = swap ? b : a, hi = swap ? a : b;
    v[0] = lo.x;
    v[1] = lo.y;
    v[2] = lo.z;
    v[3] = lo.w;
    v[4] = hi.x;
    v[5] = hi.y;
    v[6] = hi.z;
    v[7] = hi.w;
}

// Eight neighbours of a bf16 row, of which `left` (0 or less: none) are there.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, int left) {
    Vec<__nv_bfloat16, false> v;
    v.load(p, left);
    return v.raw;
}
__device__ __forceinline__ void widen8(const uint4& q, float (&v)[8]) {
    const float2 f[4] = {bf16x2_f32(q.x), bf16x2_f32(q.y), bf16x2_f32(q.z), bf16x2_f32(q.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = f[i].x;
        v[2 * i + 1] = f[i].y;
    }
}
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
    uint4 q;
    __nv_bfloat162* const h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    return q;
}
// Eight neighbours of a bf16 row to any address.  All lanes of a warp call
// this, each eight past the lane before it or at the start of a run; valid:
// what of the run is left (0 or less: nothing).
__device__ __forceinline__ void put8(const Out& o, int64_t at, int valid, bool start, const uint4& q) {
    Vec<__nv_bfloat16, false> v;
    v.raw = q;
    v.store(static_cast<__nv_bfloat16*>(o.p) + at, valid, start);
}
// A weight gradient's eight, of which `left` are there, added to what is there
// if asked for.
__device__ __forceinline__ void put8_f32(const Out& o, int64_t at, int left, bool add, const float (&v)[8]) {
    float* const p = static_cast<float*>(o.p) + at;
    if (o.vec && left >= 8) {
        float4* const q = reinterpret_cast<float4*>(p);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4 f = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            if (add) {
                const float4 c = q[h];
                f = make_float4(f.x + c.x, f.y + c.y, f.z + c.z, f.w + c.w);
            }
            q[h] = f;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = add ? p[i] + v[i] : v[i];
}

// 16 turned columns (rows of the outputs from n0 on) in UP, DHIDDEN and, with
// sums that stay fp32, DW.  WHOLE: all of their rows and columns are there and
// on 16 bytes, so that nothing keeps one unit's instructions from the other's.
// g8, u8: DHIDDEN's g and u.
template <int OP>
struct Units {
    static constexpr int GROUPS = OP == UP ? 8 : 16;      // of eight outputs of a row
    static constexpr int N = F_COLS * GROUPS / 128;       // a thread's
};

// Eight neighbours of an output row: v are their sums (UP: g's, and w u's).
// What leaves is rounded once, from fp32, to bf16: h, dg, du and h again, because
// the next product reads bf16 (a pass from given operands is then off by 2.3e-3 of
// its norm, 1.7e-3 of which is its own result's rounding); g and u, because they
// are what a block keeps for its backward pass, whose gradients are then off by
// 3.5e-3.  In fp32 they would take twice the memory and DHIDDEN's reads.
// valid, start: as put8 has them; left: of the eight that are there.  All lanes
// of a warp call this; WHOLE: all eight are there, on 16 bytes.
template <int OP, bool WHOLE>
__device__ __forceinline__ void finish8(const FfnLaunch& p, int e, int j, int row, int m, int valid, bool start,
                                        float (&v)[8], float (&w)[8], const uint4& g8, const uint4& u8) {
    auto put = [&](const Out& o, const float (&f)[8]) {
        const int64_t at = row * o.ld + m;
        if (WHOLE) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o.p) + at) = narrow8(f);
        else put8(o, at, valid, start, narrow8(f));
    };
    float a[8], d[8];
    if constexpr (OP == UP) {
        activate8(p.act, v, a, d);
#pragma unroll
        for (int q = 0; q < 8; ++q) a[q] *= w[q];
        put(p.out[0], a);
        if (p.out[1].p) {
            put(p.out[1], v);
            put(p.out[2], w);
        }
    } else if constexpr (OP == DHIDDEN) {
        float g[8];
        widen8(g8, g);
        widen8(u8, w);
        activate8(p.act, g, a, d);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            // (dh u may be past the largest number where act'(g) is 0)
            d[q] = d[q] * w[q] * v[q];
            v[q] *= a[q];
            a[q] *= w[q];
        }
        put(p.out[0], d);
        put(p.out[1], v);
        if (p.out[2].p) put(p.out[2], a);
    } else if constexpr (OP == DW) {
        const Out& o = p.out[j];
        const int64_t at = e * o.stride + row * o.ld + m;
        const int left = min(valid, 8);
        if (p.out_f32) {
            put8_f32(o, at, left, p.accumulate, v);
            return;
        }
        if (p.accumulate) {
            float c[8];
            widen8(load8(static_cast<const __nv_bfloat16*>(o.p) + at, left), c);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += c[i];
        }
        put8(o, at, valid, start, narrow8(v));
    } else {
        put(p.out[0], v);
    }
}

// DHIDDEN's g and u of eight places, of which `left` are there.
__device__ __forceinline__ void load_kept(const FfnLaunch& p, int row, int m, int left, uint4& g8, uint4& u8) {
    const int64_t at = row * p.ld_kept + m;
    g8 = load8(static_cast<const __nv_bfloat16*>(p.gate) + at, left);
    u8 = load8(static_cast<const __nv_bfloat16*>(p.up) + at, left);
}

template <int OP, bool WHOLE>
__device__ __forceinline__ void finish_turned(const FfnLaunch& p, const Item& x, const float* turn, int n0, int m0,
                                              int m_end, int tid, const uint4 (&g8)[Units<OP>::N],
                                              const uint4 (&u8)[Units<OP>::N]) {
    constexpr int GROUPS = Units<OP>::GROUPS;
#pragma unroll
    for (int i = 0; i < Units<OP>::N; ++i) {
        const int r = (tid + 128 * i) / GROUPS, group = tid % GROUPS;
        const int row = n0 + r, m = m0 + group * 8;
        const int valid = row < x.n_end ? min(m_end - m, 8 * (GROUPS - group)) : 0;
        float v[8], w[8];
        turned8(turn + r * F_ROW, group, v);
        if (OP == UP) turned8(turn + r * F_ROW, 8 + group, w);
        finish8<OP, WHOLE>(p, x.e, x.j, row, m, valid, group == 0, v, w, g8[i], u8[i]);
    }
}

// The sums of a part, as they are (rows of whole groups of eight).
template <int OP>
__device__ __forceinline__ void store_part(const FfnLaunch& p, const Item& x, const float* turn, int n0, int m0,
                                           int m_end, int tid) {
    constexpr int GROUPS = Units<OP>::GROUPS;
    const int64_t ld = p.part_ld[OP == DW && x.j == 2];
    float* const to = p.part + x.split * p.part_stride + (OP == DW ? p.part_at[x.j] : 0);
#pragma unroll
    for (int i = 0; i < Units<OP>::N; ++i) {
        const int r = (tid + 128 * i) / GROUPS, group = tid % GROUPS;
        const int row = n0 + r, m = m0 + group * 8;
        if (row >= x.n_end || m >= m_end) continue;
#pragma unroll
        for (int h = 0; h < (OP == UP ? 2 : 1); ++h) {
            float v[8];
            turned8(turn + r * F_ROW, 8 * h + group, v);
            float4* const q = reinterpret_cast<float4*>(to + row * ld + h * (ld / 2) + m);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

// DW's sums of the chunks before, 16 columns of them, of which a thread reads
// back what it has written: asked for 16 columns ahead of their use.
struct Held {
    float4 f[Units<DW>::N][2];
    static __device__ __forceinline__ float4* at(const FfnLaunch& p, int c, int i, int tid) {
        return p.held + ((int64_t(blockIdx.x) * (256 / F_COLS) + c) * Units<DW>::N + i) * 256 + tid;
    }
    __device__ __forceinline__ void fetch(const FfnLaunch& p, int c, int tid) {
#pragma unroll
        for (int i = 0; i < Units<DW>::N; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) f[i][h] = at(p, c, i, tid)[128 * h];
    }
    // This chunk's added to them: to memory, or, of the last, to their places.
    __device__ __forceinline__ void add(const FfnLaunch& p, const Item& x, float* turn, int c, int tid) const {
        constexpr int GROUPS = Units<DW>::GROUPS;
#pragma unroll
        for (int i = 0; i < Units<DW>::N; ++i) {
            float* const mine = turn + (tid + 128 * i) / GROUPS * F_ROW + tid % GROUPS * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 v = *reinterpret_cast<const float4*>(mine + 4 * h);
                if (!(x.chunk & FIRST)) {
                    const float4 g = f[i][h];
                    v = make_float4(v.x + g.x, v.y + g.y, v.z + g.z, v.w + g.w);
                }
                if (x.chunk & LAST) *reinterpret_cast<float4*>(mine + 4 * h) = v;
                else at(p, c, i, tid)[128 * h] = v;
            }
        }
    }
};

// The loads of one operand: a thread of its own each, because issuing them
// costs a thread about 100 cycles a box, and products wait for nothing else
// where the sums are long (8192 tokens of 4096 x 11008 and all four boxes of a
// step from one thread: 735 cycles a step, of 512 that the products take).
template <int OP, bool A>
__device__ __forceinline__ void load_operand(const FfnLaunch& p, Feed feed, uint8_t* smem, uint32_t rank,
                                             volatile int* abort_flag) {
    constexpr bool A_MN = OP == DHIDDEN || OP == DX || OP == DW, B_MN = OP == DW;
    constexpr int STAGES = Space<OP>::STAGES;
    const uint32_t full = smem_u32(smem + Space<OP>::BARS), empty = full + 8 * STAGES, torn = empty + 8 * STAGES;
    const uint32_t full_leader = map_to_rank(full, 0), torn_own = map_to_rank(torn, rank);
    const uint32_t stage0 = smem_u32(smem) + (A ? 0 : F_OP_BYTES);
    uint32_t slot = 0, parity = 1;
    Asked asked = {};
    bool ok = true, free_next = false;
    for (Item x; ok;) {
        ok = feed.next<false>(x, abort_flag, p.wait_limit_ns);
        if (!ok || x.e < 0) break;
        const int boxes = (x.n / 2 + 63) / 64;
        const uint32_t bytes = F_OP_BYTES + boxes * F_BOX;
        const int m0 = x.m0 + static_cast<int>(rank) * (OP == UP ? 64 : 128);
        const int n0 = x.n0 + static_cast<int>(rank) * (x.n / 2);
        int s = x.s0;
        const uint32_t first = slot;
        const int stop = x.s0 + x.steps, half = (p.k + F_K - 1) / F_K;
        // DX has two sums' worth of steps, of one operand pair each
#pragma unroll 1
        for (int part = OP == DX && s >= half; ok && s < stop; ++part) {
            const int j = OP == DW ? x.j : part;
            const int end = OP == DX && part == 0 ? min(half, stop) : stop;
            const Maps& m = p.maps[j];
            const int z = p.a_by_expert[j] ? x.e : 0, z1 = p.a_by_expert[1] ? x.e : 0;
            const CUtensorMap* const tb = boxes > 1 ? &m.b : &m.b64;
            int k0 = OP == DW ? x.t0 : (OP == DX ? s - part * half : s) * F_K;
#pragma unroll 1
            for (; s < end; ++s, k0 += F_K) {
                if (!free_next && !wait_pair(empty + 8 * slot, parity, abort_flag, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t ahead = slot + 1 == STAGES ? 0 : slot + 1;
                free_next = is_over(empty + 8 * ahead, ahead ? parity : parity ^ 1);
                uint32_t bar = full_leader + 8 * slot;
                if (OP == DW && s == stop - 1 && x.gap()) {
                    if (A) mbar_expect_tx(torn + 8 * slot, bytes);
                    bar = torn_own + 8 * slot;
                } else {
                    if (A && rank == 0) mbar_expect_tx(full + 8 * slot, 2 * bytes);
                }
                const uint32_t to = stage0 + slot * F_STAGE_BYTES;
                if constexpr (A) {
                    if constexpr (OP == UP) {
                        load_box(to, &m.a, bar, k0, m0, z);
                        load_box(to + F_BOX, &p.maps[1].a, bar, k0, m0, z1);
                    } else if constexpr (A_MN) {
                        if (m.wide_a) {
                            load_box(to, &m.a, bar, 0, k0, m0 / 64, z);
                        } else {
                            load_box(to, &m.a, bar, m0, k0, 0, z);
                            load_box(to + F_BOX, &m.a, bar, m0 + 64, k0, 0, z);
                        }
                    } else {
                        load_box(to, &m.a, bar, k0, m0, z);
                    }
                } else if constexpr (B_MN) {
                    if (m.wide_b && x.n == 256) {
                        load_box(to, &m.b, bar, 0, k0, n0 / 64, 0);
                    } else {
                        load_box(to, &m.b64, bar, n0, k0, 0, 0);
                        if (boxes > 1) load_box(to + F_BOX, &m.b64, bar, n0 + 64, k0, 0, 0);
                    }
                } else {
                    load_box(to, tb, bar, k0, n0, 0);
                }
                if (++slot == STAGES) {
                    slot = 0;
                    parity ^= 1;
                }
            }
        }
        ask(asked, s - x.s0, first, STAGES, boxes > 1, OP == DW && ok ? x.gap() : 0);
    }
    reinterpret_cast<Asked*>(smem + Space<OP>::ASKED)[A ? 0 : 1] = asked;
}

// Waits, no longer than the limit for all of them, for the loads that a pair
// which has given up still has in flight: this CTA's of torn steps, and, where
// the leader does it, what else both CTAs asked for.  No thread asks for more.
template <int OP>
__device__ void drain_loads(uint8_t* smem, uint32_t rank, uint64_t limit) {
    constexpr int STAGES = Space<OP>::STAGES;
    const uint32_t full = smem_u32(smem + Space<OP>::BARS), torn = full + 16 * STAGES, zero = torn + 8 * STAGES;
    // both CTAs' counts, this one's first, where the write-out has ended
    const uint32_t own = smem_u32(smem + Space<OP>::ASKED);
    Asked* const by = reinterpret_cast<Asked*>(smem + Space<OP>::TURN);
    Asked* const zeros = by + 4;
    for (uint32_t r = 0; r < 2; ++r) {
        const uint32_t from = map_to_rank(own, rank ^ r);
        read_cluster(&by[2 * r], from, 2 * sizeof(Asked));
        read_cluster(&zeros[r], from + 2 * sizeof(Asked), sizeof(Asked));
    }
    const uint64_t t0 = global_ns();
    const auto ends = [&](uint32_t bar, const Settle& s) {
        if (!s.wait) return true;
        if (s.arm) mbar_expect_tx(bar, s.arm);
        if (s.cancel) mbar_complete_tx(bar, s.cancel);
        while (!mbar_try_wait(bar, s.parity))
            if (global_ns() - t0 > limit) return false;
        return true;
    };
#pragma unroll 1
    for (uint32_t i = 0; i < STAGES; ++i) {
        if (OP == DW && !ends(torn + 8 * i, settle_torn(by, i, STAGES))) return;
        if (rank != 0) continue;
        if (!ends(full + 8 * i, settle_full(by, i, STAGES))) return;
        if (OP == DW && !ends(zero + 8 * i, settle_zeros(by, zeros, i, STAGES))) return;
    }
}

// What warps 0 and 1 of a pair that has given up do between the CTAs' meeting and
// their end: the others have left.  issued: this warp has issued products.  (Out of
// line, as what a wait that runs out does: at the kernels' ends the same code cost
// every launch 0.1 to 0.45 us.)
template <int OP>
__device__ __noinline__ void give_up(uint8_t* smem, uint32_t drain_bar, bool issued, uint32_t rank, uint64_t limit) {
    if (threadIdx.x == 0) drain_loads<OP>(smem, rank, limit);
    // (the lane that issued the products: elections of one mask agree)
    if (issued && elected()) {
        commit_pair_local(drain_bar);
        wait_quiet(drain_bar, 0, limit);
    }
    __syncwarp();
    cluster_sync_all();
}

template <int OP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(F_THREADS, 1)
    gated_ffn_kernel(const __grid_constant__ FfnLaunch p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using S = Space<OP>;
    constexpr int STAGES = S::STAGES;
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + S::BARS);   // a step's loads (leader's)
    uint64_t* empty_bar = full_bar + STAGES;      // its products have run
    uint64_t* torn_bar = empty_bar + STAGES;      // DW: this CTA's loads of a torn step
    uint64_t* zero_bar = torn_bar + STAGES;       // and both CTAs' zeros over it (leader's)
    uint64_t* tfull_bar = zero_bar + STAGES;
    uint64_t* tempty_bar = tfull_bar + 2;
    uint64_t* drain_bar = tempty_bar + 2;
    uint64_t* item_bar = drain_bar + 1;             // a tile is there; its place is free
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_bar + 2 * F_ITEMS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* const table = reinterpret_cast<int32_t*>(smem + S::TABLE);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;
    constexpr bool A_MN = OP == DHIDDEN || OP == DX || OP == DW, B_MN = OP == DW;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
            mbar_init(smem_u32(&torn_bar[s]), 1);
            mbar_init(smem_u32(&zero_bar[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull_bar[a]), 1);
            mbar_init(smem_u32(&tempty_bar[a]), 2 * F_EPI_WARPS);
        }
        mbar_init(smem_u32(drain_bar), 1);
        for (int i = 0; i < F_ITEMS; ++i) {
            mbar_init(smem_u32(&item_bar[i]), 1);
            // both loading threads, the products' thread, the epilogue's warps, and DW's clearing warp
            mbar_init(smem_u32(&item_bar[F_ITEMS + i]), 3 + F_EPI_WARPS + (OP == DW));
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile(
            "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                smem_u32(tmem_slot)),
            "r"(F_TMEM_COLS)
            : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 2) {
        // the experts' first rows (rising, within the rows there are) and
        // their first rows of tiles
        int32_t rows = 0, tiles = 0;
        for (int e0 = 0; e0 <= p.experts; e0 += 32) {
            const int e = e0 + lane;
            int32_t b = e <= p.experts ? (p.offsets ? p.offsets[e] : e ? int32_t(p.rows) : 0) : 0;
            b = min(max(b, 0), int32_t(p.rows));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, b, o);
                if (lane >= o) b = max(b, v);
            }
            b = max(b, rows);
            const int32_t before = __shfl_up_sync(0xffffffffu, b, 1);
            // tiles of the expert before e
            const int32_t len = e ? b - (lane ? before : rows) : 0;
            int32_t n = (len + p.tile_n - 1) / p.tile_n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, n, o);
                if (lane >= o) n += v;
            }
            n += tiles;
            if (e <= p.experts) {
                table[e] = b;
                table[p.experts + 1 + e] = n;
            }
            rows = __shfl_sync(0xffffffffu, b, 31);
            tiles = __shfl_sync(0xffffffffu, n, 31);
        }
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint64_t limit = p.wait_limit_ns;
    Feed feed(smem + S::ITEMS, smem_u32(item_bar));
    bool any = false;        // products have been issued

    if (warp == 0) {
        // ------------------------------------------------------ loads of A, of B
        if (lane == 0) load_operand<OP, true>(p, feed, smem, rank, abort_flag);
    } else if (warp == F_LOAD_B_WARP) {
        if (lane == 0) load_operand<OP, false>(p, feed, smem, rank, abort_flag);
    } else if (warp == 1) {
        // ------------------------------------------------- products (leader)
        if (lane == 0 && rank != 0) {
            // the other CTA's thread lets its tiles pass
            for (Item x; feed.next<false>(x, abort_flag, limit) && x.e >= 0;) {
            }
        } else if (rank == 0) {
            uint32_t slot = 0;
            uint32_t full_phase = 0, zero_phase = 0;        // a bit a stage
            uint32_t uses[2] = {0, 0};
            uint32_t acc = 0;
            const uint64_t a_desc = smem_desc(smem_u32(smem), A_MN ? F_BOX : 16, 1024);
            const uint64_t b_desc = smem_desc(smem_u32(smem + F_OP_BYTES), B_MN ? F_BOX : 16, 1024);
            const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar);
            uint32_t idesc = 0, d_tmem = 0;
            auto products = [&](uint32_t fresh, int count) {
                const uint64_t ad = a_desc + (slot * F_STAGE_BYTES >> 4);
                const uint64_t bd = b_desc + (slot * F_STAGE_BYTES >> 4);
                if (elected()) {
#pragma unroll
                    for (int kk = 0; kk < F_K / 16; ++kk)
                        if (kk < count)
                            mma_pair(d_tmem, ad + uint64_t(kk * (A_MN ? 2048 : 32) >> 4),
                                     bd + uint64_t(kk * (B_MN ? 2048 : 32) >> 4), idesc, kk ? 1u : fresh);
                    commit_pair_multicast(empty0 + 8 * slot);
                }
                __syncwarp();
            };
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return wait_warp(bar, parity, abort_flag, limit);
            };
            // The next tile and its accumulator are asked for while this one's
            // products run: one after the other they took 800 cycles between
            // two tiles.  The loop over steps has nothing in it that it could do
            // without, and all lanes run it, so that one of them issues products from
            // values the whole warp shares: the products wait for this loop
            // where the sums are long (8192 tokens of 4096 x 11008, forward: 1400 us
            // with the short step and the tile's end in the loop, 1297
            // without, 1250 with the whole warp).
            Item x, y;
            y.e = -1;
            bool there = false, free_acc = false;
            bool ok = feed.next<true>(x, abort_flag, limit);
            while (ok && x.e >= 0) {
                if (x.steps == 0) {
                    ok = feed.next<true>(x, abort_flag, limit);
                    continue;
                }
                const uint32_t use = acc ? uses[1]++ : uses[0]++;
                if (!free_acc && !wait(smem_u32(&tempty_bar[acc]), (use & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                idesc = instr_desc(256, x.n, B_MN) | (A_MN ? 1u << 15 : 0u);
                d_tmem = tmem_base + acc * 256;
                uint32_t fresh = 0;
                any = true;
#pragma unroll 1
                for (int s = x.steps - 1; s > 0; --s) {
                    if (!there && !wait(full0 + 8 * slot, full_phase >> slot & 1)) {
                        ok = false;
                        break;
                    }
                    full_phase ^= 1u << slot;
                    const uint32_t next = slot + 1 == STAGES ? 0 : slot + 1;
                    there = is_over_warp(full0 + 8 * next, full_phase >> next & 1);
                    products(fresh, F_K / 16);
                    fresh = 1;
                    slot = next;
                }
                if (!ok || !(ok = feed.next<true>(y, abort_flag, limit))) break;
                // the last step, which DW's may be a short or a torn one: its
                // products go no further than the expert's tokens
                if (OP == DW && x.gap()) {
                    if (!wait(smem_u32(&zero_bar[slot]), zero_phase >> slot & 1)) {
                        ok = false;
                        break;
                    }
                    zero_phase ^= 1u << slot;
                } else {
                    if (!there && !wait(full0 + 8 * slot, full_phase >> slot & 1)) {
                        ok = false;
                        break;
                    }
                    full_phase ^= 1u << slot;
                }
                free_acc = is_over_warp(smem_u32(&tempty_bar[acc ^ 1]), ((acc ? uses[0] : uses[1]) & 1) ^ 1);
                products(fresh, OP == DW && x.tail ? (x.tail + 15) / 16 : F_K / 16);
                slot = slot + 1 == STAGES ? 0 : slot + 1;
                if (elected()) commit_pair_multicast(smem_u32(&tfull_bar[acc]));
                __syncwarp();
                there = false;
                acc ^= 1;
                x = y;
            }
        }
    } else if (warp == F_TILE_WARP) {
        // ------------------------------------------------------------ tiles
        if (lane == 0) {
            const Tiles<OP> tiles(p, table);
            Item* const items = reinterpret_cast<Item*>(smem + S::ITEMS);
            int32_t it = pair, left = 0, tail = 0;
            Item x{};
            for (uint32_t n = 0;; ++n) {
                // (a tile's chunks follow one another, of about one length)
                if (left == 0) {
                    x.e = -1;
                    if (it < tiles.total) x = tiles.at(it);
                    it += npairs;
                    left = x.e < 0 ? 0 : x.steps;
                    tail = x.tail;
                    x.chunk = FIRST;
                } else {
                    x.t0 += x.steps * F_K;
                    x.chunk = 0;
                }
                if (x.e >= 0) {
                    x.steps = left;
                    if (OP == DW && left > p.chunk) {
                        const int32_t chunks = (left + p.chunk - 1) / p.chunk;
                        x.steps = (left + chunks - 1) / chunks;
                    }
                    left -= x.steps;
                    x.tail = left ? 0 : tail;
                    x.chunk |= left ? 0 : LAST;
                }
                const uint32_t slot = n % F_ITEMS;
                if (!wait_pair(smem_u32(&item_bar[F_ITEMS + slot]), (n / F_ITEMS & 1) ^ 1, abort_flag, limit))
                    break;
                items[slot] = x;
                mbar_arrive(smem_u32(&item_bar[slot]));
                if (x.e < 0) break;
            }
        }
    } else if (warp == F_CLEAR_WARP) {
        // ----------------------------------------------------- torn steps of DW
        if constexpr (OP == DW) {
            // Tokens of the next expert, or of none: 0 times a NaN of theirs would
            // be a NaN here, so both operands' rows are cleared up to the next
            // 16, which a product takes.  The zeros come as loads do, a box a lane,
            // and like them count on the leader's barrier, so that the products
            // read nothing that a thread of the other CTA has written: that
            // took stores, a fence and a release to the whole cluster, with
            // which 128 experts' DW takes 552 to 579 us, not 517 to 533.
            Asked zeros = {};
            uint32_t phase = 0;
            const uint32_t leader = map_to_rank(smem_u32(zero_bar), 0);
            const uint32_t box = lane >> 2, bit = lane & 3;
            for (Item x; feed.next<true>(x, abort_flag, limit) && x.e >= 0;) {
                const uint32_t step = zeros.steps + x.steps, gap = x.gap();
                if (x.steps && gap) {
                    const uint32_t slot = (step - 1) % STAGES;
                    if (!wait_warp(smem_u32(&torn_bar[slot]), phase >> slot & 1, abort_flag, limit)) break;
                    phase ^= 1u << slot;
                    const bool two = x.n > 128;
                    if (lane == 0 && rank == 0) mbar_expect_tx(smem_u32(&zero_bar[slot]), 2 * zero_bytes(gap, two));
                    if (box < (two ? 4 : 3) && gap >> bit & 1)
                        load_box(smem_u32(smem) + slot * F_STAGE_BYTES + box * F_BOX +
                                     (x.tail + (gap & ((1u << bit) - 1))) * 128,
                                 &p.zeros[bit], leader + 8 * slot, 0, F_NO_ROW, 0);
                    __syncwarp();
                }
                zeros.steps = step;
            }
            if (lane == 0) reinterpret_cast<Asked*>(smem + S::ASKED)[2] = zeros;
        }
    } else {
        // --------------------------------------------------------- write out
        const int lg = warp & 3;                    // this warp's 32 TMEM lanes
        const int team = (warp - 2) / 4;
        const int tid = (warp - 2) % 4 * 32 + lane;
        uint8_t* const turn_at = smem + S::TURN + team * F_TURN_BYTES;
        float* const turn = reinterpret_cast<float*>(turn_at);
        const uint32_t tempty_leader = map_to_rank(smem_u32(tempty_bar), 0);
        uint32_t uses[2] = {0, 0};
        uint32_t acc = 0;
        // what DHIDDEN reads beside the sums comes 16 columns ahead of its use
        // by asynchronous copies (loads to registers made what the thread then
        // reads from shared memory wait for them too: 1950 cycles for 16
        // columns, not 1150), to the place that was not read last
        constexpr int UNITS = Units<OP>::N;
        uint4* const kept = reinterpret_cast<uint4*>(smem + S::KEPT + team * F_KEPT_BYTES) + tid;
        int place = 0;
        auto fetch = [&](const Item& x, int c) {
            const int row0 = x.n0 + c * F_COLS + tid / 16, m = x.m0 + static_cast<int>(rank) * 128 + tid % 16 * 8;
            const int64_t at = row0 * p.ld_kept + m;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                if (p.vec && row0 + 8 * i < x.n_end && m + 8 <= p.m[0]) {
                    copy16(kept + 512 * place + 256 * i, static_cast<const __nv_bfloat16*>(p.gate) + at + 8 * i * p.ld_kept);
                    copy16(kept + 512 * place + 256 * i + 128, static_cast<const __nv_bfloat16*>(p.up) + at + 8 * i * p.ld_kept);
                }
            }
        };
        Held held;
        for (Item x;;) {
            bool got = feed.next<true>(x, abort_flag, limit);
            if (got && x.e >= 0) {
                if (OP == DHIDDEN && p.splits == 1) fetch(x, team);
                if (OP == DW && !(x.chunk & FIRST)) held.fetch(p, team, tid);
                if (x.steps) {
                    const uint32_t use = acc ? uses[1]++ : uses[0]++;
                    got = wait_pair(smem_u32(&tfull_bar[acc]), use & 1, abort_flag, limit);
                }
            }
            // the team's barriers need all four warps: a wait that ran out for
            // one leaves them all
            int bad = !got;
            asm volatile(
                "{\n\t.reg .pred a, b;\n\t"
                "setp.ne.s32 a, %0, 0;\n\t"
                "barrier.red.or.pred b, %1, 128, a;\n\t"
                "selp.s32 %0, 1, 0, b;\n\t}"
                : "+r"(bad)
                : "r"(1 + team)
                : "memory");
            if (bad || x.e < 0) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + acc * 256 + (static_cast<uint32_t>(lg * 32) << 16);
            const int n_real = x.n_end - x.n0;
            const int m0 = x.m0 + static_cast<int>(rank) * (OP == UP ? 64 : 128);
            const int m_end = OP == DW ? p.m[x.j == 2] : p.m[0];
            auto release = [&] {
                if (!x.steps) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * acc);
            };
            // the teams take blocks of columns in turn; this one's last
            const bool flat = (OP == DOWN || OP == DX || (OP == DW && !p.out_f32 && !p.accumulate)) && p.splits == 1 &&
                              x.chunk == (FIRST | LAST);
            int last = (n_real - 1) / (flat ? F_COLS16 : F_COLS);
            if ((last & 1) != team) --last;
            if (last < 0) release();
            if constexpr (OP == DOWN || OP == DX || OP == DW) {
                if (flat) {
                    const Out& o = p.out[OP == DW ? x.j : 0];
                    const uint32_t mine = smem_u32(turn_at) + (lane % 8 * F_ROW16 + lg * 32 + lane / 8 * 8) * 2;
                    for (int c = team; c <= last; c += 2) {
                        team_sync(team);          // the last columns have been read
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r[2][4];
                            if (x.steps) {
                                tmem_ld_frag(taddr + c * F_COLS16 + 16 * h, r);
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i) r[i / 4][i % 4] = 0u;
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                store_turned(mine + (16 * h + 8 * j) * F_ROW16 * 2, r[j]);
                        }
                        if (c == last) release();
                        team_sync(team);
                        const int m = m0 + tid % 16 * 8, row0 = x.n0 + c * F_COLS16 + tid / 16;
                        const int left = min(m_end - m, 8 * (16 - tid % 16));
                        const bool whole = o.vec && m0 + 128 <= m_end;
#pragma unroll
                        for (int i = 0; i < F_COLS16 / 8; ++i) {
                            const uint4 q = *reinterpret_cast<const uint4*>(
                                turn_at + ((tid / 16 + 8 * i) * F_ROW16 + tid % 16 * 8) * 2);
                            const int row = row0 + 8 * i;
                            const int64_t at = (OP == DW ? x.e * o.stride : 0) + row * o.ld + m;
                            if (!whole)
                                put8(o, at, row < x.n_end ? left : 0, tid % 16 == 0, q);
                            else if (row < x.n_end)
                                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o.p) + at) = q;
                        }
                    }
                }
            }
            {
                for (int c = flat ? last + 1 : team; c <= last; c += 2) {
                    const int n0 = x.n0 + c * F_COLS;
                    uint32_t raw[16];
                    if (x.steps) {
                        tmem_ld16(taddr + c * F_COLS, raw);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) raw[i] = 0u;
                    }
                    if (c == last) release();
                    team_sync(team);              // the last columns have been read
#pragma unroll
                    for (int i = 0; i < F_COLS; ++i)
                        turn[i * F_ROW + lg * 32 + lane] = __uint_as_float(raw[i]);
                    team_sync(team);
                    if (OP == DW && x.chunk != (FIRST | LAST)) {
                        held.add(p, x, turn, c, tid);
                        if (!(x.chunk & FIRST) && c < last) held.fetch(p, c + 2, tid);
                    }
                    if (!(x.chunk & LAST)) continue;
                    if (p.splits > 1) {
                        store_part<OP>(p, x, turn, n0, m0, m_end, tid);
                    } else if (OP != DW && p.vec && n0 + F_COLS <= x.n_end && m0 + (OP == UP ? 64 : 128) <= m_end) {
                        uint4 g8[UNITS], u8[UNITS];
                        if constexpr (OP == DHIDDEN) {
                            copies_done();
#pragma unroll
                            for (int i = 0; i < UNITS; ++i) {
                                g8[i] = kept[512 * place + 256 * i];
                                u8[i] = kept[512 * place + 256 * i + 128];
                            }
                            place ^= 1;
                            if (c < last) fetch(x, c + 2);
                        }
                        finish_turned<OP, true>(p, x, turn, n0, m0, m_end, tid, g8, u8);
                    } else {
                        uint4 g8[UNITS], u8[UNITS];
                        if constexpr (OP == DHIDDEN) {
                            copies_done();
#pragma unroll
                            for (int i = 0; i < UNITS; ++i) {
                                const int row = n0 + tid / 16 + 8 * i, m = m0 + tid % 16 * 8;
                                load_kept(p, row, m, row < x.n_end ? m_end - m : 0, g8[i], u8[i]);
                            }
                            place ^= 1;
                            if (c < last) fetch(x, c + 2);
                        }
                        finish_turned<OP, false>(p, x, turn, n0, m0, m_end, tid, g8, u8);
                    }
                }
            }
            if (x.steps) acc ^= 1;
        }
        if (OP == DHIDDEN) copies_done();
    }

    tc_fence_before();
    cluster_sync_all();      // no CTA leaves while its pair may still touch it
    if (warp > 1) return;
    // (a wait that ran out in one CTA is known to both by now, whatever of the
    // pair had done its work before)
    if (*abort_flag) give_up<OP>(smem, smem_u32(drain_bar), any, rank, limit);
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(F_TMEM_COLS)
                     : "memory");
    }
}

// The parts of a split sum in order, and what becomes of it: a thread has
// eight neighbours of an output row.  gridDim.y: DW's products.
template <int OP>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ FfnLaunch p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int j = OP == DW ? blockIdx.y : 0;
    if (OP == DW && !(p.products >> j & 1)) return;    // (a whole block)
    const int m_end = p.m[OP == DW && j == 2];
    const int64_t rows = OP == DW ? p.m[j != 2] : p.rows;
    const int64_t ld = p.part_ld[OP == DW && j == 2];
    const int64_t groups = (m_end + 7) / 8;
    const int64_t u = blockIdx.x * int64_t(128) + threadIdx.x;
    const bool live = u < rows * groups;
    const int row = live ? static_cast<int>(u / groups) : 0, m = live ? static_cast<int>(u - row * groups) * 8 : 0;
    const int left = live ? m_end - m : 0;
    uint4 g8 = make_uint4(0u, 0u, 0u, 0u), u8 = g8;
    if (OP == DHIDDEN) load_kept(p, row, m, left, g8, u8);
    const float* const from = p.part + (OP == DW ? p.part_at[j] : 0) + row * ld + m;
    float v[8] = {}, w[8] = {};
    if (live) {
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            const float4* const q = reinterpret_cast<const float4*>(from + s * p.part_stride);
            const float4 a = q[0], b = q[1];
            const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += f[i];
            if (OP == UP) {
                const float4* const r = reinterpret_cast<const float4*>(from + s * p.part_stride + ld / 2);
                const float4 c = r[0], d = r[1];
                const float g[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] += g[i];
            }
        }
    }
    finish8<OP, false>(p, 0, j, row, m, left, m == 0, v, w, g8, u8);
}

// A tensor that TMA cannot read, to dense rows of ld elements (a multiple of 8,
// what is past a row as zeros): eight of a row a thread, put together from the
// two aligned pieces that hold them.
__global__ void __launch_bounds__(256)
    dense_kernel(const __nv_bfloat16* src, int64_t matrices, int64_t rows, int64_t cols, int64_t ld_src,
                 int64_t stride_src, __nv_bfloat16* dst, int64_t ld) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t groups = ld / 8;
    for (int64_t u = blockIdx.x * int64_t(256) + threadIdx.x; u < matrices * rows * groups;
         u += gridDim.x * int64_t(256)) {
        const int64_t r = u / groups, c = (u - r * groups) * 8, e = r / rows;
        Vec<__nv_bfloat16, false> v;
        v.load(src + e * stride_src + (r - e * rows) * ld_src + c, static_cast<int>(cols - c));
        *reinterpret_cast<uint4*>(dst + r * ld + c) = v.raw;
    }
}

// A wait that nothing satisfies, as the roles wait.
__global__ void __launch_bounds__(32) ffn_timeout_kernel(unsigned long long limit_ns) {
    __shared__ uint64_t bar;
    __shared__ volatile int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort_flag = 0;
    }
    __syncthreads();
    wait_soon(smem_u32(&bar), 0, &abort_flag, &g_ffn_err, limit_ns);
}

// ------------------------------------------------------------------- host

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// An operand as the products read it: its own memory, or a dense copy in the
// workspace.
struct Operand {
    const void* p;
    int64_t matrices, rows, cols, ld, stride;
    size_t copy = 0;         // offset of the copy
    bool copied = false;
};

bool tma_reads(const Operand& o) {
    return reinterpret_cast<uintptr_t>(o.p) % 16 == 0 && (o.rows <= 1 || (o.ld % 8 == 0 && o.ld >= o.cols)) &&
           (o.matrices <= 1 || o.stride % 8 == 0);
}

struct Workspace {
    size_t bytes = 0;
    size_t take(size_t n) {
        const size_t at = bytes;
        bytes += align256(n);
        return at;
    }
    Operand operand(const void* p, int64_t matrices, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
        // one matrix for all experts stays one
        Operand o{p, stride == 0 ? 1 : matrices, rows, cols, ld, stride};
        if (rows && !tma_reads(o)) {
            o.copied = true;
            const int64_t wide = ceil_div(cols, 8) * 8;
            o.copy = take(size_t(o.matrices) * rows * wide * 2);
        }
        return o;
    }
};

cudaError_t settle(Operand& o, char* base, cudaStream_t s) {
    if (!o.copied) return cudaSuccess;
    auto* const to = reinterpret_cast<__nv_bfloat16*>(base + o.copy);
    const int64_t ld = ceil_div(o.cols, 8) * 8, blocks = ceil_div(o.matrices * o.rows * (ld / 8), 256);
    const cudaError_t e =
        launch_kernel(dense_kernel, dim3(static_cast<unsigned>(std::min(blocks, int64_t(152 * 16)))), dim3(256), 0, s,
                      static_cast<const __nv_bfloat16*>(o.p), o.matrices, o.rows, o.cols, o.ld, o.stride, to, ld);
    o.p = to;
    o.ld = ld;
    o.stride = o.rows * ld;
    return e;
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

bool encode(CUtensorMap* tm, const void* base, unsigned rank, const int64_t* dims, const int64_t* strides,
            const unsigned* box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    if (!encoder()) return false;
    cuuint64_t d[4], st[3];
    cuuint32_t bx[4], el[4] = {1, 1, 1, 1};
    for (unsigned i = 0; i < rank; ++i) {
        d[i] = cuuint64_t(dims[i]);
        bx[i] = box[i];
        if (i + 1 < rank) st[i] = cuuint64_t(strides[i]) * 2;
    }
    return encoder()(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, st, bx, el,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
int64_t row_stride(const Operand& o) { return o.rows > 1 ? o.ld : ceil_div(o.cols, 8) * 8; }
int64_t matrix_stride(const Operand& o) { return o.matrices > 1 ? o.stride : o.rows * row_stride(o); }

// An operand whose columns are k, in boxes of `high` rows of 64; zeros come
// back past a matrix's rows and columns.
bool rows_map(CUtensorMap* tm, const Operand& o, unsigned high) {
    const int64_t dims[3] = {o.cols, o.rows, o.matrices}, strides[2] = {row_stride(o), matrix_stride(o)};
    const unsigned box[3] = {64, high, 1};
    return encode(tm, o.p, 3, dims, strides, box);
}
// An operand whose rows are k, in boxes of 64 rows of 64 columns; wide: two of
// those side by side, as blocks of columns, which its columns must be whole
// ones of.
bool boxes_map(CUtensorMap* tm, const Operand& o, bool wide) {
    const int64_t dims[4] = {wide ? 64 : o.cols, o.rows, wide ? o.cols / 64 : 1, o.matrices};
    const int64_t strides[3] = {row_stride(o), wide ? 64 : row_stride(o), matrix_stride(o)};
    const unsigned box[4] = {64, 64, wide ? 2u : 1u, 1};
    return encode(tm, o.p, 4, dims, strides, box);
}
bool columns_map(CUtensorMap* tm, const Operand& o, int32_t* wide) {
    *wide = o.cols % 64 == 0;
    return boxes_map(tm, o, *wide != 0);
}

// Boxes of `high` rows of 64 zeros (from F_NO_ROW on), of an operand's memory.
bool zeros_map(CUtensorMap* tm, const Operand& o, unsigned high) {
    const int64_t dims[3] = {64, 1, 1}, strides[2] = {64, 64};
    const unsigned box[3] = {64, high, 1};
    return encode(tm, o.p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// N's side, whose rows are the operand's.
bool rows_of_n(Maps& m, const Operand& o) { return rows_map(&m.b, o, 128) && rows_map(&m.b64, o, 64); }

Out output(void* p, int64_t ld, int64_t rows, int64_t matrices = 1, int64_t stride = 0, int size = 2) {
    return Out{p, ld, stride,
               reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * size % 16 == 0) &&
                   (matrices <= 1 || stride * size % 16 == 0)};
}

using Kernel = void (*)(FfnLaunch);

cudaError_t launch_op(Op op, const FfnLaunch& p, int64_t items, cudaStream_t s) {
    static const Kernel kernel[5] = {gated_ffn_kernel<UP>, gated_ffn_kernel<DOWN>, gated_ffn_kernel<DHIDDEN>,
                                     gated_ffn_kernel<DX>, gated_ffn_kernel<DW>};
    static const Kernel join[5] = {join_kernel<UP>, join_kernel<DOWN>, join_kernel<DHIDDEN>, join_kernel<DX>,
                                   join_kernel<DW>};
    static const int size[5] = {Space<UP>::BYTES, Space<DOWN>::BYTES, Space<DHIDDEN>::BYTES, Space<DX>::BYTES,
                                Space<DW>::BYTES};
    static int attr_done[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        for (int i = 0; i < 5; ++i) {
            const cudaError_t e =
                cudaFuncSetAttribute(kernel[i], cudaFuncAttributeMaxDynamicSharedMemorySize, size[i]);
            if (e != cudaSuccess) return e;
        }
        if (dev >= 0 && dev < 64) attr_done[dev] = 1;
    }
    items *= p.splits;
    const int pairs = static_cast<int>(items < F_PAIRS ? items : F_PAIRS);
    const cudaError_t e = launch_kernel(kernel[op], dim3(2 * pairs), dim3(F_THREADS), size[op], s, p);
    if (e != cudaSuccess || p.splits == 1) return e;
    int64_t units = p.rows * ceil_div(p.m[0], 8);
    if (op == DW) {
        const int64_t a = int64_t(p.m[1]) * ceil_div(p.m[0], 8), b = int64_t(p.m[0]) * ceil_div(p.m[1], 8);
        units = a > b ? a : b;
    }
    return launch_kernel(join[op], dim3(static_cast<unsigned>(ceil_div(units, 128)), op == DW ? 3 : 1), dim3(128), 0,
                         s, p);
}

// How one dense block's product is cut up.
struct Cut {
    int tile_n = 256, splits = 1;
    int64_t row_tiles = 0;
    int64_t ld[2] = {0, 0}, at[3] = {0, 0, 0}, stride = 0;     // of the parts
    int chunk = 0;
    size_t held = 0, bytes = 0;
};

// Parts that the sums are cut into, so that every pair has a tile, of four
// steps at least.  Joining them costs a launch, 3 us of the caller's time and
// about as much of the GPU's, so that 48 steps (0.2 us each, and more where the
// matrices come from memory) have to be saved: 64 tokens of 7168 x 2048 take 28 us
// forward and 70 back, 41 and 95 unsplit; 5 tokens of 2048 x 768, 28 steps saved
// forward, took 15 us instead of 17, but the caller 26 instead of 23.
int split_count(int64_t tiles, int64_t steps) {
    int64_t s = F_PAIRS / tiles;
    if (s > steps / 4) s = steps / 4;
    return s >= 2 && steps - steps / s >= 48 ? static_cast<int>(s) : 1;
}

// op, for rows x ... of one dense block (experts: a tile's rows go by the
// expert, and nothing is split: one of many has its own tiles).
Cut cut(Op op, bool dense, int64_t rows, int64_t experts, int64_t m, int64_t k) {
    Cut c;
    c.row_tiles = rows / 256 + experts;
    if (!dense || rows == 0) return c;
    // tiles of as many rows as make the pairs' rounds come out best: a round of
    // narrower tiles takes less, though not in proportion, because the
    // matrices' part of the loads stays (4096 rows of 4096 x 4096, DHIDDEN: 19
    // tiles of 224 rows are four rounds and take 105 us, 16 of 256 are four, too,
    // and take 112; 4097 rows of 7168 x 2048 forward: 208 and 216)
    const int64_t across = ceil_div(m, op == UP ? 128 : 256), least = ceil_div(rows, 256);
    int64_t best = -1;
    for (int64_t n = least; n <= least + std::min(least / 2, int64_t(32)); ++n) {
        const int64_t size = ceil_div(ceil_div(rows, n), 32) * 32, tiles = ceil_div(rows, size) * across;
        const int64_t cost = ceil_div(tiles, F_PAIRS) * (256 + size);
        if (best < 0 || cost < best) {
            best = cost;
            c.tile_n = static_cast<int>(size);
            c.row_tiles = ceil_div(rows, size);
        }
    }
    c.splits = split_count(c.row_tiles * across, ceil_div(k, F_K) * (op == DX ? 2 : 1));
    if (c.splits > 1) {
        c.ld[0] = ceil_div(m, 8) * 8 * (op == UP ? 2 : 1);
        c.stride = rows * c.ld[0];
        c.bytes = size_t(c.splits) * c.stride * 4;
    }
    return c;
}
Cut cut_grads(bool dense, int64_t rows, int64_t hidden, int64_t inner, int products, bool f32) {
    Cut c;
    const int64_t steps = ceil_div(rows, F_K);
    if (dense) {
        int64_t tiles = 0;
        c.ld[0] = ceil_div(hidden, 8) * 8;
        c.ld[1] = ceil_div(inner, 8) * 8;
        for (int j = 0; j < 3; ++j) {
            if (!(products >> j & 1)) continue;
            tiles += ceil_div(hidden, 256) * ceil_div(inner, 256);
            c.at[j] = c.stride;
            c.stride += j == 2 ? hidden * c.ld[1] : inner * c.ld[0];
        }
        c.splits = tiles ? split_count(tiles, steps) : 1;
        if (c.splits > 1) c.bytes = align256(size_t(c.splits) * c.stride * 4);
    }
    c.chunk = f32 ? F_CHUNK_F32 : F_CHUNK_BF16;
    if (products && steps > c.chunk) {
        // a tile may have more than one chunk
        c.held = c.bytes;
        c.bytes += size_t(F_PAIRS) * 256 * 256 * 4;
    }
    return c;
}
void apply(FfnLaunch& p, const Cut& c, char* parts) {
    p.tile_n = c.tile_n;
    p.splits = c.splits;
    p.part = reinterpret_cast<float*>(parts);
    p.chunk = c.chunk;
    p.held = reinterpret_cast<float4*>(parts + c.held);
    p.part_stride = c.stride;
    for (int i = 0; i < 2; ++i) p.part_ld[i] = c.ld[i];
    for (int i = 0; i < 3; ++i) p.part_at[i] = c.at[i];
}

FfnLaunch common(const int32_t* offsets, int64_t rows, int64_t experts, int act) {
    FfnLaunch p = {};
    p.offsets = offsets;
    p.rows = rows;
    p.experts = static_cast<int32_t>(experts);
    p.act = act;
    p.wait_limit_ns = wait_limit_ns();
    return p;
}

struct Forward {
    Workspace space;
    Operand x, gate, up, down, h;
    size_t h_at, part_at;
    Cut cut_up, cut_down;
};
Forward plan(const muon_gated_ffn_args& a) {
    Forward f;
    const int64_t ld_h = ceil_div(a.inner, 8) * 8;
    f.h_at = f.space.take(size_t(a.rows) * ld_h * 2);
    f.h = Operand{nullptr, 1, a.rows, a.inner, ld_h, 0};
    f.x = f.space.operand(a.x, 1, a.rows, a.hidden, a.ld_x, 0);
    f.gate = f.space.operand(a.w_gate, a.experts, a.inner, a.hidden, a.ld_gate, a.stride_gate);
    f.up = f.space.operand(a.w_up, a.experts, a.inner, a.hidden, a.ld_up, a.stride_up);
    f.down = f.space.operand(a.w_down, a.experts, a.hidden, a.inner, a.ld_down, a.stride_down);
    f.cut_up = cut(UP, !a.offsets, a.rows, a.experts, a.inner, a.hidden);
    f.cut_down = cut(DOWN, !a.offsets, a.rows, a.experts, a.hidden, a.inner);
    f.part_at = f.space.take(std::max(f.cut_up.bytes, f.cut_down.bytes));
    return f;
}

struct Backward {
    Workspace space;
    Operand dy, x, gate, up, down, dg, du, h;
    size_t d_at[3] = {0, 0, 0};      // dg, du, h where the caller gives none
    bool own[3] = {false, false, false};
    size_t part_at;
    Cut cut_dh, cut_dx, cut_dw;
};
Backward plan(const muon_gated_ffn_grad_args& a) {
    Backward b;
    const int64_t ld = ceil_div(a.inner, 8) * 8;
    void* const given[3] = {a.dgate, a.dup, a.h};
    Operand* const d[3] = {&b.dg, &b.du, &b.h};
    for (int i = 0; i < 3; ++i) {
        const bool needed = i < 2 || a.dw_down;
        b.own[i] = !given[i] && needed;
        if (b.own[i]) {
            b.d_at[i] = b.space.take(size_t(a.rows) * ld * 2);
            *d[i] = Operand{nullptr, 1, a.rows, a.inner, ld, 0};
        } else {
            // copied after DHIDDEN has written it
            const bool read = i == 2 ? a.dw_down != nullptr : a.dx || (i ? a.dw_up : a.dw_gate);
            if (read) *d[i] = b.space.operand(given[i], 1, a.rows, a.inner, a.ld_d, 0);
            else *d[i] = Operand{given[i], 1, a.rows, a.inner, a.ld_d, 0};
        }
    }
    b.dy = b.space.operand(a.dy, 1, a.rows, a.hidden, a.ld_dy, 0);
    if (a.dw_gate || a.dw_up) b.x = b.space.operand(a.x, 1, a.rows, a.hidden, a.ld_x, 0);
    if (a.dx) {
        b.gate = b.space.operand(a.w_gate, a.experts, a.inner, a.hidden, a.ld_gate, a.stride_gate);
        b.up = b.space.operand(a.w_up, a.experts, a.inner, a.hidden, a.ld_up, a.stride_up);
    }
    b.down = b.space.operand(a.w_down, a.experts, a.hidden, a.inner, a.ld_down, a.stride_down);
    b.cut_dh = cut(DHIDDEN, !a.offsets, a.rows, a.experts, a.inner, a.hidden);
    if (a.dx) b.cut_dx = cut(DX, !a.offsets, a.rows, a.experts, a.hidden, a.inner);
    b.cut_dw = cut_grads(!a.offsets, a.rows, a.hidden, a.inner,
                         (a.dw_gate ? 1 : 0) | (a.dw_up ? 2 : 0) | (a.dw_down ? 4 : 0), a.g_dtype == MUON_F32);
    b.part_at = b.space.take(std::max(b.cut_dh.bytes, std::max(b.cut_dx.bytes, b.cut_dw.bytes)));
    return b;
}

#define RETURN_IF_CUDA(expr)                       \
    do {                                           \
        const cudaError_t e_ = (expr);             \
        if (e_ != cudaSuccess) return e_;          \
    } while (0)

}  // namespace

size_t gated_ffn_workspace(const muon_gated_ffn_args& a) { return plan(a).space.bytes; }
size_t gated_ffn_grad_workspace(const muon_gated_ffn_grad_args& a) { return plan(a).space.bytes; }

cudaError_t launch_gated_ffn(const muon_gated_ffn_args& a, void* ws, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    Forward f = plan(a);
    char* const base = static_cast<char*>(ws);
    f.h.p = base + f.h_at;
    for (Operand* o : {&f.x, &f.gate, &f.up, &f.down}) RETURN_IF_CUDA(settle(*o, base, s));
    FfnLaunch p = common(a.offsets, a.rows, a.experts, a.activation);
    p.m[0] = static_cast<int32_t>(a.inner);
    p.k = static_cast<int32_t>(a.hidden);
    p.a_by_expert[0] = f.gate.matrices > 1;
    p.a_by_expert[1] = f.up.matrices > 1;
    p.out[0] = output(base + f.h_at, f.h.ld, a.rows);
    p.out[1] = output(a.gate, a.ld_kept, a.rows);
    p.out[2] = output(a.up, a.ld_kept, a.rows);
    p.vec = p.out[1].vec && p.out[2].vec;
    if (!rows_map(&p.maps[0].a, f.gate, 64) || !rows_map(&p.maps[1].a, f.up, 64) || !rows_of_n(p.maps[0], f.x))
        return cudaErrorInvalidValue;
    apply(p, f.cut_up, base + f.part_at);
    RETURN_IF_CUDA(launch_op(UP, p, f.cut_up.row_tiles * ceil_div(a.inner, 128), s));
    p.m[0] = static_cast<int32_t>(a.hidden);
    p.k = static_cast<int32_t>(a.inner);
    p.a_by_expert[0] = f.down.matrices > 1;
    p.out[0] = output(a.y, a.ld_y, a.rows);
    if (!rows_map(&p.maps[0].a, f.down, 128) || !rows_of_n(p.maps[0], f.h)) return cudaErrorInvalidValue;
    apply(p, f.cut_down, base + f.part_at);
    return launch_op(DOWN, p, f.cut_down.row_tiles * ceil_div(a.hidden, 256), s);
}

cudaError_t launch_gated_ffn_grad(const muon_gated_ffn_grad_args& a, void* ws, cudaStream_t s) {
    Backward b = plan(a);
    char* const base = static_cast<char*>(ws);
    Operand* const d[3] = {&b.dg, &b.du, &b.h};
    const bool grads = a.dw_gate || a.dw_up || a.dw_down;
    FfnLaunch p = common(a.offsets, a.rows, a.experts, a.activation);
    if (a.rows) {
        for (Operand* o : {&b.dy, &b.x, &b.gate, &b.up, &b.down}) RETURN_IF_CUDA(settle(*o, base, s));
        p.m[0] = static_cast<int32_t>(a.inner);
        p.k = static_cast<int32_t>(a.hidden);
        p.a_by_expert[0] = b.down.matrices > 1;
        p.gate = a.gate;
        p.up = a.up;
        p.ld_kept = a.ld_kept;
        p.vec = output(const_cast<void*>(a.gate), a.ld_kept, a.rows).vec &&
                output(const_cast<void*>(a.up), a.ld_kept, a.rows).vec;
        for (int i = 0; i < 3; ++i) {
            if (b.own[i]) d[i]->p = base + b.d_at[i];
            p.out[i] = output(const_cast<void*>(d[i]->p), d[i]->ld, a.rows);
            p.vec = p.vec && p.out[i].vec;
        }
        if (!columns_map(&p.maps[0].a, b.down, &p.maps[0].wide_a) || !rows_of_n(p.maps[0], b.dy)) return cudaErrorInvalidValue;
        apply(p, b.cut_dh, base + b.part_at);
        RETURN_IF_CUDA(launch_op(DHIDDEN, p, b.cut_dh.row_tiles * ceil_div(a.inner, 256), s));
        for (Operand* o : d) RETURN_IF_CUDA(settle(*o, base, s));
        if (a.dx) {
            p.m[0] = static_cast<int32_t>(a.hidden);
            p.k = static_cast<int32_t>(a.inner);
            p.a_by_expert[0] = b.gate.matrices > 1;
            p.a_by_expert[1] = b.up.matrices > 1;
            p.out[0] = output(a.dx, a.ld_dx, a.rows);
            if (!columns_map(&p.maps[0].a, b.gate, &p.maps[0].wide_a) ||
                !columns_map(&p.maps[1].a, b.up, &p.maps[1].wide_a) || !rows_of_n(p.maps[0], b.dg) ||
                !rows_of_n(p.maps[1], b.du))
                return cudaErrorInvalidValue;
            apply(p, b.cut_dx, base + b.part_at);
            RETURN_IF_CUDA(launch_op(DX, p, b.cut_dx.row_tiles * ceil_div(a.hidden, 256), s));
        }
    }
    if (!grads) return cudaSuccess;
    p.m[0] = static_cast<int32_t>(a.hidden);
    p.m[1] = static_cast<int32_t>(a.inner);
    p.out_f32 = a.g_dtype == MUON_F32;
    p.accumulate = a.accumulate;
    const int size = p.out_f32 ? 4 : 2;
    p.out[0] = output(a.dw_gate, a.ld_dw_gate, a.inner, a.experts, a.stride_dw_gate, size);
    p.out[1] = output(a.dw_up, a.ld_dw_up, a.inner, a.experts, a.stride_dw_up, size);
    p.out[2] = output(a.dw_down, a.ld_dw_down, a.hidden, a.experts, a.stride_dw_down, size);
    int64_t items = 0;
    const Operand* const left[3] = {&b.x, &b.x, &b.h};
    const Operand* const right[3] = {&b.dg, &b.du, &b.dy};
    for (int j = 0; j < 3; ++j) {
        p.a_by_expert[j] = 0;
        if (!p.out[j].p) continue;
        p.products |= 1 << j;
        const int64_t m = j == 2 ? a.inner : a.hidden, n = j == 2 ? a.hidden : a.inner;
        items += a.experts * ceil_div(m, 256) * ceil_div(n, 256);
        Maps& of = p.maps[j];
        if (a.rows && (!columns_map(&of.a, *left[j], &of.wide_a) || !columns_map(&of.b, *right[j], &of.wide_b) ||
                       !boxes_map(&of.b64, *right[j], false)))
            return cudaErrorInvalidValue;
    }
    for (int i = 0; a.rows && i < 4; ++i)
        if (!zeros_map(&p.zeros[i], b.dy, 1u << i)) return cudaErrorInvalidValue;
    apply(p, b.cut_dw, base + b.part_at);
    return launch_op(DW, p, items, s);
}

cudaError_t launch_ffn_timeout(unsigned long long limit_ns, cudaStream_t s) {
    return launch_kernel(ffn_timeout_kernel, dim3(1), dim3(32), 0, s, limit_ns);
}

cudaError_t ffn_error_word(void** word) { return cudaGetSymbolAddress(word, g_ffn_err); }

}  // namespace ops
}  // namespace muon
