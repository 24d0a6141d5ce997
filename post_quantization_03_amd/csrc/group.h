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
constexpr int64_t GROUP_MAX = 4096, GROUP_ROWS_MAX = (1LL << 31) - 1;

// Expert, its rows, and the tile (of `size` rows, `nx` tiles a tile row) among its own; rows = 0 if there is none.
struct GroupAt {
    int k, begin, rows, id;
};
__device__ __forceinline__ int clamp_row(int v, int n) { return v < 0 ? 0 : v < n ? v : n; }

__device__ __forceinline__ GroupAt group_tile(const Group& g, unsigned id, int size, unsigned nx) {
    const int lane = threadIdx.x & 63;
    int before = clamp_row(g.off[0], g.n);       // end of the expert before lane 0's
    unsigned tiles = 0;                          // of the experts before lane 0's
    for (int k0 = 0; k0 < g.experts; k0 += 64) {
        const int k = k0 + lane;
        int end = k < g.experts ? clamp_row(g.off[k + 1], g.n) : 0;
        end = end > before ? end : before;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(end, d);
            if (lane >= d && o > end) end = o;
        }
        const int up = __shfl_up(end, 1), begin = lane ? up : before, rows = end - begin;
        const unsigned own = (unsigned)(((int64_t)rows + size - 1) / size);
        unsigned sum = own;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const unsigned o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        const uint64_t hit = __ballot((tiles + sum) * nx > id);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            GroupAt at;
            at.k = k0 + l;
            at.begin = __builtin_amdgcn_readlane(begin, l);
            at.rows = __builtin_amdgcn_readlane(rows, l);
            at.id = (int)(id - (tiles + (unsigned)__builtin_amdgcn_readlane((int)(sum - own), l)) * nx);
            return at;
        }
        before = __builtin_amdgcn_readlane(end, 63);
        tiles += (unsigned)__builtin_amdgcn_readlane((int)sum, 63);
    }
    return GroupAt{0, 0, 0, 0};
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

// Products whose output rows are the tokens: Y = X W^T (plain, gated, int8) and dX = dY W. Experts take work-groups in
// turn, each one's tiles dealt to the XCDs by themselves: experts of unequal size then load all XCDs alike.
template <int E, int MODE, typename C>
__global__ __launch_bounds__(C::THREADS, C::EU) void group_tile_kernel(TileArgs g, Group gr) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN;
    const int nx = (int)((g.N + TN_OUT - 1) / TN_OUT);
    const GroupAt at = group_tile(gr, blockIdx.x, C::TM, (unsigned)nx);
    if (at.rows == 0) return;
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
    TileAt t;
    t.cut = -1;
    t.split = t.pair = 0;
    const int ny = (at.rows + C::TM - 1) / C::TM;
    tile_place(t, xcd_range(at.id, ny * nx), ny, nx);
    t.tm = __builtin_amdgcn_readfirstlane(t.tm);
    t.tn = __builtin_amdgcn_readfirstlane(t.tn);
    tile_body<E, MODE, C>(g, t);
}

// dW = dY^T X over each expert's rows, zeros for one without any: `per` tiles an expert (of both gradients).
template <int E, typename C>
__global__ __launch_bounds__(C::THREADS, C::EU) void group_grad_kernel(TileArgs g, Group gr, int per) {
    const int k = (int)(blockIdx.x / (unsigned)per), id = (int)(blockIdx.x - (unsigned)k * (unsigned)per);
    int begin, rows;
    group_rows(gr, k, begin, rows);
    g.K = rows;
    g.A += begin * g.lda;
    g.A2 += begin * g.lda2;
    g.B += begin * g.ldb;
    g.Y = rows_on(g.Y, (int64_t)k * gr.o * g.ldy, g.dt);
    g.Y2 = rows_on(g.Y2, (int64_t)k * gr.o * g.ldy2, g.dt);
    TileAt t;
    t.cut = -1;
    t.split = 0;
    const int ny = (int)((g.M + C::TM - 1) / C::TM), nx = (int)((g.N + C::TN - 1) / C::TN), j = xcd_range(id, per);
    t.pair = __builtin_amdgcn_readfirstlane(j / (ny * nx));
    tile_place(t, j % (ny * nx), ny, nx);
    t.tm = __builtin_amdgcn_readfirstlane(t.tm);
    t.tn = __builtin_amdgcn_readfirstlane(t.tn);
    tile_body<E, TP_GRAD_W, C>(g, t);
}

// Few rows an expert: work-group (block of 16 rows of B, expert with rows). Its rows go 16 NB at a time, the weights
// from HBM the first time and from a cache after that.
template <int E, bool GATED, int NB>
__global__ __launch_bounds__(FEW_THREADS) void group_few_kernel(FewArgs g, Group gr, int blocks) {
    const GroupAt at = group_tile(gr, blockIdx.x, GROUP_ROWS_MAX, (unsigned)blocks);
    if (at.rows == 0) return;
    const int64_t begin = at.begin, w0 = (int64_t)at.k * gr.o;
    g.n = at.rows;
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
    for (;;) {
        few_body<E, GATED, NB>(g, at.id);
        g.n -= 16 * NB;
        if (g.n <= 0) return;
        __syncthreads();         // the sums in LDS have been read
        g.A += 16 * NB * g.lda;
        if (E == EL_I8) g.fA += 16 * NB;
        g.Y = rows_on(g.Y, 16 * NB * g.ldy, g.dt);
        if (GATED) {
            g.Y2 = rows_on(g.Y2, 16 * NB * g.ldy2, g.dt);
            g.Y3 = rows_on(g.Y3, 16 * NB * g.ldy3, g.dt);
        }
    }
}

// ------------------------------------------------------------------------------------------ launches
// Tiles of `size` rows that n rows of `experts` experts take at most: every expert with a row may add a partial one.
inline int64_t group_tiles_max(int64_t n, int64_t experts, int64_t size) {
    const int64_t some = experts < n ? experts : n;
    return (n - some) / size + some;
}

// Whether n rows of `experts` experts run as few tokens each. The counts are not known here; the rule takes their mean.
template <int E>
bool group_few(int64_t n, int64_t experts) {
    const int64_t some = experts < n ? experts : n;
    return n <= 16 * some;
}

// Tile shape of a grouped product, from the times that tile_plan takes and rows dealt evenly.
template <int E, int MODE>
int group_shape(int64_t n, int64_t experts, int64_t N, int64_t K) {
    if (E == EL_F32) return 2;
    constexpr int size[3] = {256, 128, 64}, occ[3] = {1, 2, 4}, BK = 8 * el_chunk<E>();
    constexpr double lat[3] = {1.4, 0.9, 0.75}, fix[3] = {10.0, 4.0, 1.7}, w[3] = {1.55, 0.5, 0.38};
    const int64_t some = experts < n ? experts : n;
    const int64_t each = some ? (n + some - 1) / some : 0;
    int best = 2;
    double least = 0.0;
    for (int h = 0; h < 3; h++) {
        const int64_t tn = MODE == TP_GATED ? size[h] / 2 : size[h];
        int64_t tiles, slabs;
        if (MODE == TP_GRAD_W) {         // N: rows of dW, K: its columns
            tiles = experts * ((N + size[h] - 1) / size[h]) * ((K + size[h] - 1) / size[h]);
            slabs = (each + BK - 1) / BK;
        } else {
            tiles = some * ((each + size[h] - 1) / size[h]) * ((N + tn - 1) / tn);
            slabs = (K + BK - 1) / BK * (MODE == TP_GRAD_X ? 2 : 1);
        }
        const int64_t percu = (tiles + 255) / 256, rounds = (percu + occ[h] - 1) / occ[h];
        const double by_lat = (double)rounds * lat[h], by_w = (double)percu * w[h];
        const double t = (double)slabs * (by_lat > by_w ? by_lat : by_w) + (double)rounds * fix[h];
        if (h == 0 || t < least) {
            least = t;
            best = h;
        }
    }
    return best;
}

// f(tile shape) for 0 L, 1 M, 2 S; fp32 has S alone
template <int E, typename F>
kq_status with_shape(int shape, F&& f) {
    if constexpr (E != EL_F32) {
        if (shape == 0) return f(TileL{});
        if (shape == 1) return f(TileM{});
    }
    return f(TileS{});
}

template <int E, int MODE>
kq_status group_launch(const TileArgs& g, const Group& gr, hipStream_t st, const char* who) {
    return with_shape<E>(group_shape<E, MODE>(gr.n, gr.experts, g.N, g.K), [&](auto shape) {
        typedef decltype(shape) C;
        constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN;
        const int64_t wgs = group_tiles_max(gr.n, gr.experts, C::TM) * ((g.N + TN_OUT - 1) / TN_OUT);
        if (!grid_ok(wgs, C::THREADS)) return fail(KQ_ESHAPE, "%s: too many tiles for a launch", who);
        static std::atomic<uint64_t> allowed{0};
        KQ_TRY(allow_lds(reinterpret_cast<const void*>(&group_tile_kernel<E, MODE, C>), C::SMEM, allowed, who));
        hipLaunchKernelGGL((group_tile_kernel<E, MODE, C>), dim3((unsigned)wgs), dim3(C::THREADS), C::SMEM, st, g, gr);
        return check_launch(who);
    });
}

template <int E>
kq_status group_grad_launch(TileArgs g, const Group& gr, int pairs, hipStream_t st, const char* who) {
    return with_shape<E>(group_shape<E, TP_GRAD_W>(gr.n, gr.experts, g.M, g.N), [&](auto shape) {
        typedef decltype(shape) C;
        const int64_t per = ((g.M + C::TM - 1) / C::TM) * ((g.N + C::TN - 1) / C::TN) * pairs;
        if (!grid_ok(per * gr.experts, C::THREADS)) return fail(KQ_ESHAPE, "%s: too many tiles for a launch", who);
        static std::atomic<uint64_t> allowed{0};
        KQ_TRY(allow_lds(reinterpret_cast<const void*>(&group_grad_kernel<E, C>), C::SMEM, allowed, who));
        hipLaunchKernelGGL((group_grad_kernel<E, C>), dim3((unsigned)(per * gr.experts)), dim3(C::THREADS), C::SMEM, st, g, gr,
                           (int)per);
        return check_launch(who);
    });
}

template <int E, bool GATED>
kq_status group_few_launch(const FewArgs& g, const Group& gr, hipStream_t st, const char* who) {
    const int64_t blocks = (g.o + 15) / 16, wgs = blocks * (gr.experts < gr.n ? gr.experts : gr.n);
    if (!grid_ok(wgs, FEW_THREADS)) return fail(KQ_ESHAPE, "%s: too many rows", who);
    const size_t sums = (size_t)FEW_WAVES * (GATED ? 2 : 1) * 1024;
    hipLaunchKernelGGL((group_few_kernel<E, GATED, 1>), dim3((unsigned)wgs), dim3(FEW_THREADS), sums, st, g, gr, (int)blocks);
    return check_launch(who);
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
