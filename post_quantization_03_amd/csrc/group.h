// Products grouped by expert on the tiles of tile.h (grouped.hip, i8.hip). Not part of the C ABI.
//
// The rows of A are sorted by expert: expert k owns rows begin_k .. end_k - 1 and meets rows k o .. k o + o - 1 of
// the stacked B. The offsets stay on the device, so the host launches as many work-groups as any distribution
// of the n rows can need, and every wavefront finds its own expert and tile from the offsets: 64 at a time, a
// running maximum (which makes any contents of the array a partition of rows inside 0 .. n) and a running sum of tiles.
// Work-groups past the last tile end at once.
#pragma once

#include "tile.h"

namespace kq {

struct Group {
    const int32_t* off;      // experts + 1 offsets
    int experts;
    int n;                   // rows of A: offsets are clamped to 0 .. n
    int o;                   // rows of B an expert
};
constexpr int64_t GROUP_MAX = 4096, GROUP_ROWS_MAX = (1LL << 31) - 512;    // rows and a tile's more fit in 32 bits

__device__ __forceinline__ int clamp_row(int v, int n) { return v < 0 ? 0 : v < n ? v : n; }

// 64 experts from k0 on, one a lane: their rows, and the tiles of `size` rows up to the lane's expert.
struct GroupLanes {
    int begin, rows;
    unsigned own, sum;
};
__device__ __forceinline__ GroupLanes group_lanes(const Group& g, int k0, int before, int size) {
    const int lane = threadIdx.x & 63, k = k0 + lane;
    int end = k < g.experts ? clamp_row(g.off[k + 1], g.n) : 0;
    end = end > before ? end : before;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(end, d);
        if (lane >= d && o > end) end = o;
    }
    const int up = __shfl_up(end, 1);
    GroupLanes l;
    l.begin = lane ? up : before;
    l.rows = end - l.begin;
    l.own = l.sum = (unsigned)(((int64_t)l.rows + size - 1) / size);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const unsigned o = __shfl_up(l.sum, d);
        if (lane >= d) l.sum += o;
    }
    return l;
}
__device__ __forceinline__ int group_first(const Group& g) { return clamp_row(g.off[0], g.n); }
__device__ __forceinline__ int last_row(const GroupLanes& l) { return __builtin_amdgcn_readlane(l.begin + l.rows, 63); }
__device__ __forceinline__ unsigned last_sum(const GroupLanes& l) { return (unsigned)__builtin_amdgcn_readlane((int)l.sum, 63); }

// Tiles of `size` rows of all experts, given the lanes of the first 64.
__device__ __forceinline__ unsigned group_tiles(const Group& g, GroupLanes l, int size) {
    unsigned tiles = last_sum(l);
    for (int k0 = 64; k0 < g.experts; k0 += 64) {
        l = group_lanes(g, k0, last_row(l), size);
        tiles += last_sum(l);
    }
    return tiles;
}

// Expert and rows of tile `id` (`nx` tiles a tile row), and the tile's place among the expert's own; rows = 0 if there is none.
struct GroupAt {
    int k, begin, rows, id;
};
__device__ __forceinline__ GroupAt group_tile(const Group& g, GroupLanes l, unsigned id, int size, unsigned nx) {
    unsigned tiles = 0;                          // of the experts before lane 0's
    for (int k0 = 0;;) {
        const uint64_t hit = __ballot((tiles + l.sum) * nx > id);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            return GroupAt{k0 + at, __builtin_amdgcn_readlane(l.begin, at), __builtin_amdgcn_readlane(l.rows, at),
                           (int)(id - (tiles + (unsigned)__builtin_amdgcn_readlane((int)(l.sum - l.own), at)) * nx)};
        }
        k0 += 64;
        if (k0 >= g.experts) return GroupAt{0, 0, 0, 0};
        tiles += last_sum(l);
        l = group_lanes(g, k0, last_row(l), size);
    }
}

// The rows of expert k.
__device__ __forceinline__ void group_rows(const Group& g, int k, int& begin, int& rows) {
    const int lane = threadIdx.x & 63;
    int b = 0;                                   // largest offset up to k
    for (int j = lane; j <= k; j += 64) {
        const int v = clamp_row(g.off[j], g.n);
        b = v > b ? v : b;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_xor(b, d);
        b = o > b ? o : b;
    }
    const int e = clamp_row(g.off[k + 1], g.n);
    begin = __builtin_amdgcn_readfirstlane(b);
    rows = __builtin_amdgcn_readfirstlane(e > b ? e - b : 0);
}

__device__ __forceinline__ void* rows_on(void* p, int64_t values, int dt) {
    return p ? static_cast<char*>(p) + values * (dt == KQ_BF16 ? 2 : 4) : nullptr;
}

// A product's operands moved to those of the expert at `at`.
template <int E, int MODE>
__device__ __forceinline__ void group_operands(TileArgs& g, const Group& gr, const GroupAt& at) {
    const int64_t begin = at.begin, w0 = (int64_t)at.k * gr.o;
    g.M = at.rows;
    g.A += begin * g.lda;
    g.B += w0 * g.ldb;
    if (MODE == TP_GRAD_X) g.A2 += begin * g.lda2;
    if (MODE == TP_GATED || MODE == TP_GRAD_X) g.B2 += w0 * g.ldb2;
    if (E == EL_I8) {
        g.fA += begin;
        g.fB += w0;
        if (MODE == TP_GATED) g.fB2 += w0;
    }
    g.Y = rows_on(g.Y, begin * g.ldy, g.dt);
    if (MODE == TP_GATED) {
        g.Y2 = rows_on(g.Y2, begin * g.ldy2, g.dt);
        g.Y3 = rows_on(g.Y3, begin * g.ldy3, g.dt);
    }
}

// Place of the expert's tile at.id.
template <typename C>
__device__ __forceinline__ void group_place(TileAt& t, const GroupAt& at, int nx) {
    tile_place(t, at.id, (at.rows + C::TM - 1) / C::TM, nx);
    t.tm = __builtin_amdgcn_readfirstlane(t.tm);
    t.tn = __builtin_amdgcn_readfirstlane(t.tn);
}

// The tiles behind the last full turn of the GPU would keep it waiting a whole turn for few of them, so their K is split as
// tile_plan splits it, by the count that the device finds. The host makes the choice for the counts there can be; both
// kernels of a product look it up.
constexpr int GROUP_COUNTS = 256;        // entries of the table: counts up to a turn's tiles, in steps of group_step
template <typename C>
constexpr unsigned group_step() { return 512 / (C::TM * C::DEEP); }      // work-groups a compute unit
struct GroupCuts {
    uint32_t at[GROUP_COUNTS + 1];       // splits (1: not cut) | slabs of a split << 8
};
struct GroupCut {
    unsigned whole, rest;    // tiles that take all of K, tiles that are cut
    int splits, sper;
};
template <typename C>
__device__ __forceinline__ GroupCut group_cut(const GroupCuts& t, unsigned tiles) {
    constexpr unsigned STEP = group_step<C>(), TURN = GROUP_COUNTS * STEP;
    GroupCut c;
    c.rest = tiles % TURN;
    const uint32_t v = t.at[(c.rest + STEP - 1) / STEP];
    c.splits = (int)(v & 255u);
    c.sper = (int)(v >> 8);
    if (c.splits == 1) c.rest = 0;
    c.whole = tiles - c.rest;
    return c;
}

// Products whose output rows are the tokens: Y = X W^T (plain, gated, int8) and dX = dY W. Bound by what bounds the tiles
// (tile_body), and by ragged counts: tiles have 256 rows, so that an expert adds half a tile row on average. MI355X: 16384 rows of 8
// experts, 4096 x 11008 bf16 1187 us (1.24 PFLOP/s; 68 tile rows for the 64 that the tokens would fill), int8 gated 1376 x 4096 172 to 182 us
// (2.0 to 2.1 POP/s); dX of two products, 8192 rows of 8 experts 11008 x 4096, 1207 us (1.22 PFLOP/s). An int8 gated tile takes 57 us for its 32
// slabs, 7 of them the activations of its 256 x 128 results and 5 the launch, the offsets and the first slab.
template <int E, int MODE, typename C>
__device__ __forceinline__ void group_tile_body(TileArgs g, const Group& gr, const GroupCuts& cuts, unsigned id) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN;
    const int nx = (int)((g.N + TN_OUT - 1) / TN_OUT);
    const GroupLanes l = group_lanes(gr, 0, group_first(gr), C::TM);
    TileAt t;
    t.cut = -1;
    t.split = t.pair = 0;
    const GroupCut c = group_cut<C>(cuts, group_tiles(gr, l, C::TM) * (unsigned)nx);
    if (id < c.whole) {
        // each turn's work-groups, dealt to the 8 XCDs one by one, take tiles XCD by XCD: neighbours in one L2 share their panels
        constexpr unsigned TURN = GROUP_COUNTS * group_step<C>();
        const unsigned first = id / TURN * TURN, left = c.whole - first;
        id = first + (unsigned)xcd_range((int)(id - first), (int)(left < TURN ? left : TURN));
    } else {
        if (c.rest == 0 || id >= c.whole + c.rest * (unsigned)c.splits) return;
        t.split = __builtin_amdgcn_readfirstlane((int)((id - c.whole) / c.rest));
        t.cut = (int)(id - c.whole - (unsigned)t.split * c.rest);
        id = c.whole + (unsigned)t.cut;
        g.splits = c.splits;
        g.sper = c.sper;
    }
    const GroupAt at = group_tile(gr, l, id, C::TM, (unsigned)nx);
    if (at.rows == 0) return;
    group_operands<E, MODE>(g, gr, at);
    group_place<C>(t, at, nx);
    tile_body<E, MODE, C>(g, t);
}
template <int E, int MODE, typename C>
__global__ __launch_bounds__(C::THREADS, C::EU) void group_tile_kernel(TileArgs g, Group gr, GroupCuts cuts) {
    group_tile_body<E, MODE, C>(g, gr, cuts, blockIdx.x);
}

// The sums of the cut tiles' splits, in split order, and the epilogue: bound by the last-level cache, which the sums come from (64 MiB of
// them 12 us), or by latency (4 us where nothing is cut). A few work-groups walk over the pieces, since most counts leave few.
template <int E, int MODE, typename C>
__global__ __launch_bounds__(256) void group_reduce_kernel(TileArgs g0, Group gr, GroupCuts cuts) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN, PER = C::TM * TN_OUT / 1024;
    const int nx = (int)((g0.N + TN_OUT - 1) / TN_OUT);
    const GroupLanes l = group_lanes(gr, 0, group_first(gr), C::TM);
    const GroupCut c = group_cut<C>(cuts, group_tiles(gr, l, C::TM) * (unsigned)nx);
    for (unsigned b = blockIdx.x; b < c.rest * PER; b += gridDim.x) {
        TileArgs g = g0;
        TileAt t;
        t.cut = (int)(b / PER);
        t.split = t.pair = 0;
        const GroupAt at = group_tile(gr, l, c.whole + (unsigned)t.cut, C::TM, (unsigned)nx);
        g.splits = c.splits;
        g.sper = c.sper;
        group_operands<E, MODE>(g, gr, at);
        group_place<C>(t, at, nx);
        tile_reduce<MODE, C, E == EL_I8 ? EL_I8 : EL_F32>(g, t, (int)(b % PER));
    }
}

// dW = dY^T X over each expert's rows, zeros for one without any: `per` tiles an expert (of both gradients), g.splits work-groups a
// tile, each a part of the expert's rows (whose number the device finds: a split may be left without any). Both gradients of 8192 rows of 8
// experts, 11008 x 4096 bf16, take 1355 us (1.09 PFLOP/s): tiles of 16 slabs take 32 us, 23 for their products, 5 to write 128 KiB and 4 to start.
template <int E, typename C>
__device__ __forceinline__ void group_grad_operands(TileArgs& g, const Group& gr, int k) {
    int begin, rows;
    group_rows(gr, k, begin, rows);
    constexpr int BK = 8 * el_chunk<E>();
    g.K = rows;
    g.sper = ((rows + BK - 1) / BK + g.splits - 1) / g.splits;
    g.A += begin * g.lda;
    g.A2 += begin * g.lda2;
    g.B += begin * g.ldb;
    g.Y = rows_on(g.Y, (int64_t)k * gr.o * g.ldy, g.dt);
    g.Y2 = rows_on(g.Y2, (int64_t)k * gr.o * g.ldy2, g.dt);
}
template <typename C>
__device__ __forceinline__ void group_grad_place(TileAt& t, const TileArgs& g, int id, int per) {
    const int ny = (int)((g.M + C::TM - 1) / C::TM), nx = (int)((g.N + C::TN - 1) / C::TN), j = xcd_range(id, per);
    t.pair = __builtin_amdgcn_readfirstlane(j / (ny * nx));
    tile_place(t, j % (ny * nx), ny, nx);
    t.tm = __builtin_amdgcn_readfirstlane(t.tm);
    t.tn = __builtin_amdgcn_readfirstlane(t.tn);
}
template <int E, typename C>
__device__ __forceinline__ void group_grad_body(TileArgs g, const Group& gr, int per, unsigned block) {
    const unsigned each = (unsigned)per * (unsigned)g.splits;
    const int k = (int)(block / each), in = (int)(block - (unsigned)k * each), id = in % per;
    group_grad_operands<E, C>(g, gr, k);
    TileAt t;
    t.split = __builtin_amdgcn_readfirstlane(in / per);
    t.cut = g.splits > 1 ? __builtin_amdgcn_readfirstlane(k * per + id) : -1;
    group_grad_place<C>(t, g, id, per);
    tile_body<E, TP_GRAD_W, C>(g, t);
}
template <int E, typename C>
__global__ __launch_bounds__(C::THREADS, C::EU) void group_grad_kernel(TileArgs g, Group gr, int per) {
    group_grad_body<E, C>(g, gr, per, blockIdx.x);
}
// the sums of the splits
template <int E, typename C>
__global__ __launch_bounds__(256) void group_grad_reduce_kernel(TileArgs g0, Group gr, int per) {
    constexpr int PER = C::TM * C::TN / 1024;
    const unsigned pieces = (unsigned)per * (unsigned)gr.experts * PER;
    for (unsigned b = blockIdx.x; b < pieces; b += gridDim.x) {
        TileArgs g = g0;
        TileAt t;
        t.cut = (int)(b / PER);
        t.split = 0;
        group_grad_operands<E, C>(g, gr, t.cut / per);
        group_grad_place<C>(t, g, t.cut % per, per);
        tile_reduce<TP_GRAD_W, C>(g, t, (int)(b % PER));
    }
}

// dX and dW side by side, `first` work-groups for dX, for small products: each leaves compute units idle that the other fills
// (517 rows of 5 experts 1376 x 1000 fp32: a call of 50 us one after the other, 41 together).
template <int E, int MODE, typename C>
__global__ __launch_bounds__(C::THREADS, C::EU) void group_grads_kernel(TileArgs x, TileArgs w, Group gr, GroupCuts cuts, int per, unsigned first) {
    if (blockIdx.x < first) group_tile_body<E, MODE, C>(x, gr, cuts, blockIdx.x);
    else group_grad_body<E, C>(w, gr, per, blockIdx.x - first);
}

// Few rows an expert: a work-group for 16 NB of them and 16 rows of B. Bound by the stream of the weights: 64 rows of 16 experts, gated
// 1376 x 4096 bf16, 62 us for 361 MB (5.8 TB/s, part of them from the last-level cache). Of an expert with more, the weights come from HBM for the
// work-group that is first and from a cache for the others.
template <int E, bool GATED, int NB>
__global__ __launch_bounds__(FEW_THREADS) void group_few_kernel(FewArgs g, Group gr, int blocks) {
    constexpr int ROWS = 16 * NB;
    const GroupAt at = group_tile(gr, group_lanes(gr, 0, group_first(gr), ROWS), blockIdx.x, ROWS, (unsigned)blocks);
    if (at.rows == 0) return;
    const int first = at.id / blocks * ROWS;
    const int64_t begin = at.begin + first, w0 = (int64_t)at.k * gr.o;
    g.n = at.rows - first < ROWS ? at.rows - first : ROWS;
    g.A += begin * g.lda;
    g.B += w0 * g.ldb;
    if (GATED) g.B2 += w0 * g.ldb2;
    if (E == EL_I8) {
        g.fA += begin;
        g.fB += w0;
        if (GATED) g.fB2 += w0;
    }
    g.Y = rows_on(g.Y, begin * g.ldy, g.dt);
    if (GATED) {
        g.Y2 = rows_on(g.Y2, begin * g.ldy2, g.dt);
        g.Y3 = rows_on(g.Y3, begin * g.ldy3, g.dt);
    }
    few_body<E, GATED, NB, true>(g, at.id % blocks);
}

// ------------------------------------------------------------------------------------------ launches
// Tiles of `size` rows that n rows of `experts` experts take at most: every expert with a row may add a partial one.
inline int64_t group_tiles_max(int64_t n, int64_t experts, int64_t size) {
    const int64_t some = experts < n ? experts : n;
    return (n - some) / size + some;
}

// Whether n rows of `experts` experts run as few tokens each. The counts are not known here; the rule takes their mean. MI355X, us as
// few tokens / as tiles, o x i weights an expert, at a mean of
//   4   bf16 8 x 4096 x 11008: 111 / 113, gated 16 x 1376 x 4096: 67 / 70, 4 x 4096 x 4096: 26 / 29; int8 8 x 4096 x 11008: 58 / 64
//   8   the same: 142 / 132, 81 / 74, 31 / 31; 74 / 73, int8 gated 16 x 1376 x 4096 44 / 41, 12 x 2500 x 4096 31 / 33
//   12  178 / 146, 92 / 78, 36 / 31; 93 / 81
// and fp32 (32 rows a work-group from a mean of 9 on, so that experts of more read their weights twice), plain, and gated after the comma:
//   16  5 x 1376 x 1000: 11.9 / 17.9, 18.7 / 23.2; 8 x 1376 x 4096: 54 / 58, 102 / 112; 8 x 4096 x 11008: 413 / 413, 715 / 782
//   24  the same: 12.5 / 18.2, 19.2 / 23.1; 61 / 58, 107 / 113; 477 / 421, 766 / 787
//   32  15.8 / 18.6, 25.5 / 23.1; 89 / 59, 140 / 116; 627 / 426, 1036 / 793
template <int E>
bool group_few(int64_t n, int64_t experts) {
    return n <= (E == EL_F32 ? 24 : 6) * (experts < n ? experts : n);
}

// Estimated time, us, of work-groups of `per` slabs of tile shape h, with the constants of tile_plan but for fp32's w: 0.44 is what its matrix cores
// take, and what side by side launches of dX and dW are weighed by; tile_plan's 0.2 ranks the cuts of one product.
template <int E>
inline double group_time(int h, int64_t wgs, int64_t per) {
    constexpr int occ_log2[5] = {0, 1, 2, 0, 1};
    constexpr double lat[5] = {1.4, 0.9, 0.75, 0.45, 0.2}, fix[5] = {10.0, 4.0, 1.7, 5.5, 3.0}, w[5] = {1.55, 0.5, E == EL_F32 ? 0.44 : 0.38, 0.45, 0.19};
    const int64_t percu = (wgs + 255) >> 8, rounds = (percu + (1 << occ_log2[h]) - 1) >> occ_log2[h];
    const double by_lat = (double)rounds * lat[h], by_w = (double)percu * w[h];
    return (double)per * (by_lat > by_w ? by_lat : by_w) + (double)rounds * fix[h];
}

// How the weight gradients (o x i, an expert) are cut: tile shape and splits of an expert's rows, for rows dealt evenly. One plan for one
// gradient and for two, so that each has the same bits either way.
struct GradPlan {
    int shape, splits;
};
template <int E>
GradPlan group_grad_plan(int64_t n, int64_t experts, int64_t o, int64_t i) {
    constexpr int size[3] = {256, 128, 64}, BK = 8 * el_chunk<E>(), CUTS = 8, cuts[CUTS] = {1, 2, 3, 4, 6, 8, 12, 16};
    const int64_t slabs = ((n + experts - 1) / experts + BK - 1) / BK;
    GradPlan best{2, 1};
    double least = 0.0;
    for (int h = E == EL_F32 ? 2 : 0; h < 3; h++) {
        const int64_t tiles = experts * ((o + size[h] - 1) / size[h]) * ((i + size[h] - 1) / size[h]);
        for (int c = 0; c < CUTS; c++) {
            const int64_t wgs = tiles * cuts[c], per = (slabs + cuts[c] - 1) / cuts[c];
            if (c && (wgs > 512 << h || per * (cuts[c] - 1) >= slabs)) break;    // two turns at most, and no split empty
            double t = group_time<E>(h, wgs, per);
            if (c) t += 4.0 + (double)wgs * (size[h] * size[h] * 8 / 3.5e6);
            if (least == 0.0 || t < least) {
                least = t;
                best = GradPlan{h, cuts[c]};
            }
        }
    }
    return best;
}

// Whether the weight gradients run beside dX where its tiles are S.
template <int E>
bool group_grad_side(int64_t n, int64_t experts, int64_t o, int64_t i) {
    const GradPlan p = group_grad_plan<E>(n, experts, o, i);
    return p.shape == 2 && p.splits == 1;
}

// Whether a product may take tiles with more slabs in LDS. MI355X, us without / with them, bf16: 500 rows of 4 experts 1376 x 4096 30.6 / 17.6,
// 2000 of 8 64 / 33.7, 300 of 2 4096 x 11008 104 / 75; dX and dW, 2222 rows of 3 experts 5263 x 1251 109 / 91. Slower by up to 7 % where
// few rows leave the weights' stream to bound it: 100 rows of 2 experts 4096 x 11008 52.4 / 55.9. Weight gradients have short sums.
template <int E, int MODE>
constexpr bool group_deep() { return E != EL_F32 && MODE != TP_GRAD_W; }

// Tile shape of a grouped product, for rows dealt evenly (and cut, if that pays: 300 rows of 2 experts 4096 x 11008 bf16 98.7 -> 75.3 us).
template <int E, int MODE>
int group_shape(int64_t n, int64_t experts, int64_t N, int64_t K) {
    if (E == EL_F32) return 2;
    constexpr int size[5] = {256, 128, 64, 128, 64}, BK = 8 * el_chunk<E>();
    const int64_t some = experts < n ? experts : n;
    const int64_t each = some ? (n + some - 1) / some : 0;
    int best = 2;
    double least = 0.0;
    for (int h = 0; h < (group_deep<E, MODE>() ? 5 : 3); h++) {
        const int64_t tn = MODE == TP_GATED ? size[h] / 2 : size[h];
        // small products run side by side, in S tiles (300 rows of 8 experts 1376 x 1000, two products: 28.4 / 41.4 apart, with SD for dX)
        if (h == 3 && tp_grad_x(MODE) && best == 2 && group_grad_side<E>(n, experts, K, N)) break;
        // MD and SD: one turn, however the rows are dealt
        if (h > 2 && group_tiles_max(n, experts, size[h]) * ((N + tn - 1) / tn) > (h == 3 ? 256 : 512)) continue;
        const int64_t tiles = some * ((each + size[h] - 1) / size[h]) * ((N + tn - 1) / tn);
        const int64_t slabs = (K + BK - 1) / BK * (MODE == TP_GRAD_X ? 2 : 1);
        double t = group_time<E>(h, tiles, slabs);
        if constexpr (!tp_grad_x(MODE)) {
            // what the cuts of group_cuts would gain
            const int64_t turn = h > 2 ? 512 >> (4 - h) : 256 << h;
            double cut = t;
            for (int c : {2, 3, 4, 6, 8, 12, 16}) {
                if (tiles >= turn || c > slabs || tiles * c > (h > 2 ? turn : 2 * turn)) break;
                const double us = group_time<E>(h, tiles * c, (slabs + c - 1) / c) + 4.0 + (double)(tiles * c) * (size[h] * size[h] * 8 / 3.5e6);
                cut = us < cut ? us : cut;
            }
            if (cut < t - 5.0) t = cut;
        }
        if (h == 0 || t < least) {
            least = t;
            best = h;
        }
    }
    return best;
}

// How the tiles behind the last full turn are cut, for each number of them, and the most split sums (of a tile) that can make. Split
// sums are written and read once at 3.5 TB/s, by a second launch, which is left out (and nothing cut) where it would not pay: where
// cutting gains less than 5 us on average over the tile counts that n rows may make.
template <int E, int MODE, typename C>
int64_t group_cuts(GroupCuts& t, int64_t n, int64_t experts, int64_t N, int64_t K) {
    constexpr int h = (C::TM == 256 ? 0 : C::TM == 128 ? 1 : 2) + (C::DEEP > 2 ? 2 : 0), BK = 8 * el_chunk<E>(), TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN;
    constexpr int64_t STEP = group_step<C>(), TURN = GROUP_COUNTS * STEP;
    constexpr int products = MODE == TP_GRAD_X ? 2 : 1;
    const int64_t slabs = (K + BK - 1) / BK, nx = (N + TN_OUT - 1) / TN_OUT, most = group_tiles_max(n, experts, C::TM) * nx;
    constexpr int CUTS = 7, cuts[CUTS] = {2, 3, 4, 6, 8, 12, 16};
    int64_t per[CUTS], splits[CUTS];
    for (int c = 0; c < CUTS; c++) {
        per[c] = (slabs + cuts[c] - 1) / cuts[c];
        splits[c] = (slabs + per[c] - 1) / per[c];
    }
    // the cut for k * STEP tiles, and what it gains
    auto choose = [&](int k) {
        t.at[k] = 1u;
        const int64_t rest = k * STEP;
        if (rest == 0 || rest >= TURN || rest >= most + STEP) return 0.0;
        const double whole = group_time<E>(h, rest, slabs * products);
        double least = whole;
        for (int c = 0; c < CUTS; c++) {
            const int64_t wgs = rest * splits[c];
            if (wgs > (C::DEEP > 2 ? 1 : 2) * TURN || per[c] >= 1 << 24) break;
            const double us = group_time<E>(h, wgs, per[c] * products) + 4.0 + (double)wgs * (C::TM * C::TN * 8 / 3.5e6);
            if (us < least) {
                least = us;
                t.at[k] = splits[c] > 1 ? (uint32_t)splits[c] | (uint32_t)per[c] << 8 : 1u;
            }
        }
        return whole - least;
    };
    if constexpr (tp_grad_x(MODE) && C::TM == 64) {
        // dX of small products runs beside dW, which fills what a long K leaves idle: nothing is cut unless K is much longer than both
        // take together (517 rows of 5 experts 1376 x 1000 fp32, us with dX cut / whole: 43.8 / 41.0; 100 rows, two products: 42 / 61; 300
        // rows of 8 experts bf16, two products: 34.6 / 28.9). Also where dX is asked for alone, so that it has the same bits.
        const int64_t each = (n + experts - 1) / experts;
        const int64_t dw = experts * ((K + 63) / 64) * ((N + 63) / 64) * products * ((each + BK - 1) / BK);
        const double both = (double)(most * slabs * products + dw) * (E == EL_F32 ? 0.44 : 0.38) / 256.0;
        if ((double)(slabs * products) * 0.75 < 1.5 * both + 10.0) return 0;
    }
    // tile rows: a whole one for every C::TM rows, and up to one more an expert
    const int64_t some = experts < n ? experts : n, least = (n + C::TM - 1) / C::TM > some ? (n + C::TM - 1) / C::TM : some;
    double sum = 0.0;
    for (int k = 0; k <= 16; k++)
        sum += choose((int)(((least * nx + (most - least * nx) * k / 16) % TURN + STEP - 1) / STEP));
    if (sum < 5.0 * 17) return 0;
    for (int k = 0; k <= GROUP_COUNTS; k++) choose(k);
    int64_t sums = 0;
    for (int k = 0; k <= GROUP_COUNTS && (k - 1) * STEP < most; k++) {
        const int64_t m = (t.at[k] & 255u) > 1 ? k * STEP * (int64_t)(t.at[k] & 255u) : 0;
        sums = m > sums ? m : sums;
    }
    return sums;
}

// f(tile shape) for 0 L, 1 M, 2 S, 3 MD, 4 SD; fp32 has S alone
template <int E, int MODE, typename F>
kq_status with_shape(int shape, F&& f) {
    if constexpr (E != EL_F32) {
        if (shape == 0) return f(TileL{});
        if (shape == 1) return f(TileM{});
    }
    if constexpr (group_deep<E, MODE>()) {
        if (shape == 3) return f(TileMD{});
        if (shape == 4) return f(TileSD{});
    }
    return f(TileS{});
}

// Workspace of a product whose tiles may be cut.
template <int E, int MODE>
size_t group_ws(int64_t n, int64_t experts, int64_t N, int64_t K) {
    size_t bytes = 0;
    if (n > 0)
        with_shape<E, MODE>(group_shape<E, MODE>(n, experts, N, K), [&](auto shape) {
            typedef decltype(shape) C;
            GroupCuts cuts;
            bytes = (size_t)group_cuts<E, MODE, C>(cuts, n, experts, N, K) * C::TM * C::TN * sizeof(float);
            return KQ_OK;
        });
    return bytes;
}

// Work-groups of a product, after its cuts are chosen and its workspace checked.
template <int E, int MODE, typename C>
kq_status group_prepare(GroupCuts& cuts, int64_t& wgs, int64_t& sums, TileArgs& g, const Group& gr, void* ws, size_t ws_bytes, const char* who) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN;
    sums = group_cuts<E, MODE, C>(cuts, gr.n, gr.experts, g.N, g.K);
    if (sums && (!ws || !aligned16(ws) || ws_bytes < (size_t)sums * C::TM * C::TN * sizeof(float)))
        return fail(KQ_EWORKSPACE, "%s: workspace too small or not aligned to 16 bytes", who);
    if (!sums)
        for (uint32_t& c : cuts.at) c = 1u;
    g.part = static_cast<float*>(ws);
    wgs = group_tiles_max(gr.n, gr.experts, C::TM) * ((g.N + TN_OUT - 1) / TN_OUT) + sums;
    return grid_ok(wgs, C::THREADS) ? KQ_OK : fail(KQ_ESHAPE, "%s: too many tiles for a launch", who);
}
template <int E, int MODE, typename C>
kq_status group_sums_launch(const TileArgs& g, const Group& gr, const GroupCuts& cuts, int64_t sums, hipStream_t st, const char* who) {
    constexpr int PER = C::TM * (MODE == TP_GATED ? C::TN / 2 : C::TN) / 1024;
    if (!sums) return KQ_OK;
    const int64_t pieces = sums * PER;
    hipLaunchKernelGGL((group_reduce_kernel<E, MODE, C>), dim3((unsigned)(pieces < 2048 ? pieces : 2048)), dim3(256), 0, st, g, gr, cuts);
    return check_launch(who);
}

template <int E, int MODE>
kq_status group_launch(TileArgs g, const Group& gr, void* ws, size_t ws_bytes, hipStream_t st, const char* who) {
    return with_shape<E, MODE>(group_shape<E, MODE>(gr.n, gr.experts, g.N, g.K), [&](auto shape) {
        typedef decltype(shape) C;
        GroupCuts cuts;
        int64_t wgs, sums;
        KQ_TRY((group_prepare<E, MODE, C>(cuts, wgs, sums, g, gr, ws, ws_bytes, who)));
        static std::atomic<uint64_t> allowed{0};
        KQ_TRY(allow_lds(reinterpret_cast<const void*>(&group_tile_kernel<E, MODE, C>), C::SMEM, allowed, who));
        hipLaunchKernelGGL((group_tile_kernel<E, MODE, C>), dim3((unsigned)wgs), dim3(C::THREADS), C::SMEM, st, g, gr, cuts);
        KQ_TRY(check_launch(who));
        return group_sums_launch<E, MODE, C>(g, gr, cuts, sums, st, who);
    });
}

// Floats of the weight gradients' split sums.
inline size_t group_grad_sums(const GradPlan& p, int64_t experts, int64_t o, int64_t i, int pairs) {
    const int64_t size = 256 >> p.shape, tiles = experts * ((o + size - 1) / size) * ((i + size - 1) / size) * pairs;
    return p.splits > 1 ? (size_t)(tiles * p.splits * size * size) : 0;
}
template <int E>
size_t group_grad_ws(int64_t n, int64_t experts, int64_t o, int64_t i, int pairs) {
    if (n <= 0) return 0;
    return sizeof(float) * group_grad_sums(group_grad_plan<E>(n, experts, o, i), experts, o, i, pairs);
}

// The plan of the weight gradients, its workspace and launch checked: before anything of the call is enqueued.
template <int E>
kq_status group_grad_prepare(GradPlan& plan, const TileArgs& g, const Group& gr, int pairs, const void* ws, size_t ws_bytes, const char* who) {
    plan = group_grad_plan<E>(gr.n, gr.experts, g.M, g.N);
    const size_t need = gr.n ? sizeof(float) * group_grad_sums(plan, gr.experts, g.M, g.N, pairs) : 0;
    if (need && (!ws || !aligned16(ws) || ws_bytes < need)) return fail(KQ_EWORKSPACE, "%s: workspace too small or not aligned to 16 bytes", who);
    return with_shape<E, TP_GRAD_W>(plan.shape, [&](auto shape) {
        typedef decltype(shape) C;
        const int64_t per = ((g.M + C::TM - 1) / C::TM) * ((g.N + C::TN - 1) / C::TN) * pairs;
        return grid_ok(per * gr.experts * plan.splits, C::THREADS) ? KQ_OK : fail(KQ_ESHAPE, "%s: too many tiles for a launch", who);
    });
}
template <int E>
kq_status group_grad_launch(TileArgs g, const GradPlan& plan, const Group& gr, int pairs, void* ws, hipStream_t st, const char* who) {
    g.part = static_cast<float*>(ws);
    g.splits = plan.splits;
    return with_shape<E, TP_GRAD_W>(plan.shape, [&](auto shape) {
        typedef decltype(shape) C;
        const int64_t per = ((g.M + C::TM - 1) / C::TM) * ((g.N + C::TN - 1) / C::TN) * pairs, wgs = per * gr.experts * plan.splits;
        static std::atomic<uint64_t> allowed{0};
        KQ_TRY(allow_lds(reinterpret_cast<const void*>(&group_grad_kernel<E, C>), C::SMEM, allowed, who));
        hipLaunchKernelGGL((group_grad_kernel<E, C>), dim3((unsigned)wgs), dim3(C::THREADS), C::SMEM, st, g, gr, (int)per);
        KQ_TRY(check_launch(who));
        if (plan.splits > 1) {
            const int64_t pieces = per * gr.experts * (C::TM * C::TN / 1024);
            hipLaunchKernelGGL((group_grad_reduce_kernel<E, C>), dim3((unsigned)(pieces < 4096 ? pieces : 4096)), dim3(256), 0, st, g, gr,
                               (int)per);
            KQ_TRY(check_launch(who));
        }
        return KQ_OK;
    });
}

// Both gradients where both are cut into the smallest tiles.
template <int E, int MODE>
bool group_grads_together(const TileArgs& x, const TileArgs& w, const Group& gr) {
    return gr.n && group_shape<E, MODE>(gr.n, gr.experts, x.N, x.K) == 2 && group_grad_side<E>(gr.n, gr.experts, w.M, w.N);
}
template <int E, int MODE>
kq_status group_grads_launch(TileArgs x, TileArgs w, const Group& gr, int pairs, void* ws, size_t ws_bytes, hipStream_t st,
                             const char* who) {
    typedef TileS C;
    GroupCuts cuts;
    int64_t wgs, sums;
    KQ_TRY((group_prepare<E, MODE, C>(cuts, wgs, sums, x, gr, ws, ws_bytes, who)));
    w.splits = 1;
    const int64_t per = ((w.M + C::TM - 1) / C::TM) * ((w.N + C::TN - 1) / C::TN) * pairs;
    if (!grid_ok(wgs + per * gr.experts, C::THREADS)) return fail(KQ_ESHAPE, "%s: too many tiles for a launch", who);
    hipLaunchKernelGGL((group_grads_kernel<E, MODE, C>), dim3((unsigned)(wgs + per * gr.experts)), dim3(C::THREADS), C::SMEM, st, x, w, gr,
                       cuts, (int)per, (unsigned)wgs);
    KQ_TRY(check_launch(who));
    return group_sums_launch<E, MODE, C>(x, gr, cuts, sums, st, who);
}

template <int E, bool GATED>
kq_status group_few_launch(const FewArgs& g, const Group& gr, hipStream_t st, const char* who) {
    const int64_t blocks = (g.o + 15) / 16;
    auto run = [&](auto nb) {
        constexpr int NB = decltype(nb)::value;          // 16 rows each
        const int64_t wgs = blocks * group_tiles_max(gr.n, gr.experts, 16 * NB);
        if (!grid_ok(wgs, FEW_THREADS)) return fail(KQ_ESHAPE, "%s: too many rows", who);
        const size_t sums = (size_t)FEW_WAVES * (GATED ? 2 : 1) * NB * 1024;
        hipLaunchKernelGGL((group_few_kernel<E, GATED, NB>), dim3((unsigned)wgs), dim3(FEW_THREADS), sums, st, g, gr, (int)blocks);
        return check_launch(who);
    };
    if constexpr (E == EL_F32) {
        if (gr.n > 8 * (int64_t)gr.experts) return run(std::integral_constant<int, 2>{});
    }
    return run(std::integral_constant<int, 1>{});
}

// ------------------------------------------------------------------------------------------- checks
inline kq_status group_check(const char* who, const int32_t* offsets, int64_t experts, int64_t n, int64_t o) {
    if (!offsets) return fail(KQ_EINVAL, "%s: null offsets", who);
    if (reinterpret_cast<uintptr_t>(offsets) % 4) return fail(KQ_EINVAL, "%s: offsets must be aligned to 4 bytes", who);
    if (experts <= 0 || experts > GROUP_MAX) return fail(KQ_ESHAPE, "%s: 1 to %lld experts", who, (long long)GROUP_MAX);
    if (n > GROUP_ROWS_MAX || o > TL_ROWS_MAX / experts) return fail(KQ_ESHAPE, "%s: too many rows", who);
    return KQ_OK;
}

}  // namespace kq
