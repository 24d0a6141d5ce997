// Matrix-core products shared by the microscaled 4-bit operators (mx.hip), the gated feed-forward block (gated.hip),
// the 8-bit integer products (i8.hip) and the products grouped by expert (grouped.hip). Not part of the C ABI.
//
// Every operand is handled in 16-byte chunks along its rows: 4 fp32, 8 bf16, 16 int8 or 32 E2M1 values (one
// microscaled block). A lane of an MFMA operand holds exactly one chunk, lane group g = lane / 16
// owning chunk g of four, so one step of four chunks is
//   fp32   four v_mfma_f32_16x16x4_f32          (16 columns of K; element e of every chunk pairs up)
//   bf16   one  v_mfma_f32_16x16x32_bf16        (32 columns)
//   int8   one  v_mfma_i32_16x16x64_i8          (64 columns, int32 sums)
//   E2M1   one  v_mfma_scale_f32_16x16x128      (128 columns, one E8M0 scale byte per lane)
// and one slab of 128 bytes a row is two steps whatever the type: the staging, the LDS layout and the
// loops below are written once for the four.
#pragma once

#include <atomic>
#include <type_traits>

#include "kq_internal.h"

namespace kq {

typedef float tl_f4 __attribute__((ext_vector_type(4)));
typedef int tl_i4 __attribute__((ext_vector_type(4)));
typedef int tl_i8 __attribute__((ext_vector_type(8)));
typedef short tl_s4 __attribute__((ext_vector_type(4)));
typedef __bf16 tl_b8 __attribute__((ext_vector_type(8)));

enum { EL_F32 = 0, EL_BF16 = 1, EL_MX = 2, EL_I8 = 3 };
template <int E>
constexpr int el_chunk() { return E == EL_F32 ? 4 : E == EL_BF16 ? 8 : E == EL_I8 ? 16 : 32; }   // values in 16 bytes
template <int E>
using el_sums = std::conditional_t<E == EL_I8, tl_i4, tl_f4>;                  // four sums of a lane

// A 16-byte chunk of which only the first `part` values count, the others made zero.
template <int E>
__device__ __forceinline__ tl_i4 chunk_head(tl_i4 v, int part) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
        if constexpr (E == EL_F32) v[e] = e < part ? v[e] : 0;
        else if constexpr (E == EL_BF16) v[e] = 2 * e + 1 < part ? v[e] : 2 * e < part ? v[e] & 0xFFFF : 0;
        else v[e] = 4 * e + 3 < part ? v[e] : 4 * e < part ? v[e] & ((1 << 8 * (part - 4 * e)) - 1) : 0;
    }
    return v;
}

// ------------------------------------------------------------------------------------ conversions
__device__ __forceinline__ uint16_t to_bf16(float v) {   // nearest even, NaN stays NaN
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ float from_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// N consecutive values (N a multiple of 4) to dst[0 .. N-1] of row-major out, those below `left` only. dst is
// aligned to min(4 N, 16) bytes for fp32 and to min(2 N, 16) for bf16 when left >= N.
template <int N>
__device__ __forceinline__ void store_run(void* out, int dt, int64_t off, const float (&v)[N], int64_t left) {
    if (dt == KQ_BF16) {
        uint16_t* p = static_cast<uint16_t*>(out) + off;
        if (left >= N) {
            uint32_t w[N / 2];
#pragma unroll
            for (int e = 0; e < N / 2; e++) w[e] = (uint32_t)to_bf16(v[2 * e]) | ((uint32_t)to_bf16(v[2 * e + 1]) << 16);
            if constexpr (N % 8 == 0) {
#pragma unroll
                for (int e = 0; e < N / 8; e++)
                    reinterpret_cast<uint4*>(p)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < N / 4; e++) reinterpret_cast<uint2*>(p)[e] = make_uint2(w[2 * e], w[2 * e + 1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; e++)
                if (e < left) p[e] = to_bf16(v[e]);
        }
    } else {
        float* p = static_cast<float*>(out) + off;
        if (left >= N) {
#pragma unroll
            for (int e = 0; e < N / 4; e++)
                reinterpret_cast<float4*>(p)[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < N; e++)
                if (e < left) p[e] = v[e];
        }
    }
}

// ------------------------------------------------------------------------------------- activations
// gate = act(a) / a, the factor in 0..1 that multiplies a (of max(a, 0): its derivative, 0 at 0). The logistic gates take
// the hardware's exp2 and reciprocal (both within an ulp): the argument's rounding, |a| 2^-24 relative, is of the same order.
__device__ __forceinline__ float logistic(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}
template <int ACT>
__device__ __forceinline__ float act_gate(float a) {
    if constexpr (ACT == KQ_ACT_SILU) return logistic(a);
    else if constexpr (ACT == KQ_ACT_GELU) return 0.5f * erfcf(-0.70710678118654752f * a);
    else if constexpr (ACT == KQ_ACT_GELU_TANH) return logistic(1.5957691216057308f * (a + 0.044715f * a * a * a));
    else return a > 0.0f ? 1.0f : (a == a ? 0.0f : a);
}

// act(a) for its gate p: max(a, 0) by choice, since the product is not 0 at -infinity
template <int ACT>
__device__ __forceinline__ float act_value(float a, float p) {
    if constexpr (ACT == KQ_ACT_RELU) return a > 0.0f ? a : p;
    else return a * p;
}

// act(a) and act'(a)
template <int ACT>
__device__ __forceinline__ void act_both(float a, float& f, float& df) {
    const float p = act_gate<ACT>(a);
    f = act_value<ACT>(a, p);
    if constexpr (ACT == KQ_ACT_SILU) df = p * (1.0f + a * (1.0f - p));
    else if constexpr (ACT == KQ_ACT_GELU) df = p + a * __builtin_amdgcn_exp2f(-0.72134752044448170f * a * a) * 0.39894228040143268f;
    else if constexpr (ACT == KQ_ACT_GELU_TANH)
        // beyond 16 the gate is 0 or 1 to the last bit, and a * a may not be finite
        df = fabsf(a) > 16.0f ? p : p + a * p * (1.0f - p) * 1.5957691216057308f * (1.0f + 0.134145f * a * a);
    else df = p;
}

// f(ACT) for the activation given at run time: one branch around a whole run of values
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case KQ_ACT_SILU: f(std::integral_constant<int, KQ_ACT_SILU>{}); return;
        case KQ_ACT_GELU: f(std::integral_constant<int, KQ_ACT_GELU>{}); return;
        case KQ_ACT_GELU_TANH: f(std::integral_constant<int, KQ_ACT_GELU_TANH>{}); return;
        default: f(std::integral_constant<int, KQ_ACT_RELU>{});
    }
}

// h = act(a) * b
template <int N>
__device__ __forceinline__ void act_times(float (&h)[N], const float (&a)[N], const float (&b)[N], int act) {
    with_act(act, [&](auto A) {
#pragma unroll
        for (int e = 0; e < N; e++) h[e] = act_value<A.value>(a[e], act_gate<A.value>(a[e])) * b[e];
    });
}

// --------------------------------------------------------------------------------------- products
template <int OA, int OB>
__device__ __forceinline__ tl_f4 mma_mx(tl_i4 a, tl_i4 b, tl_f4 c, int sa, int sb) {
    const tl_i8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, OA, sa, OB, sb);
}

// c += a b over one step; for E2M1 byte oa of sa and byte ob of sb are the lane's block scales
// (oa and ob are constants after unrolling)
template <int E>
__device__ __forceinline__ el_sums<E> mma_step(tl_i4 a, tl_i4 b, el_sums<E> c, int sa, int oa, int sb, int ob) {
    if constexpr (E == EL_I8) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    } else if constexpr (E == EL_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(tl_b8, a), __builtin_bit_cast(tl_b8, b), c, 0, 0, 0);
    } else if constexpr (E == EL_F32) {
#pragma unroll
        for (int e = 0; e < 4; e++)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[e]), __int_as_float(b[e]), c, 0, 0, 0);
        return c;
    } else {
        switch (4 * oa + ob) {
            case 0: return mma_mx<0, 0>(a, b, c, sa, sb);
            case 1: return mma_mx<0, 1>(a, b, c, sa, sb);
            case 2: return mma_mx<0, 2>(a, b, c, sa, sb);
            case 3: return mma_mx<0, 3>(a, b, c, sa, sb);
            case 4: return mma_mx<1, 0>(a, b, c, sa, sb);
            case 5: return mma_mx<1, 1>(a, b, c, sa, sb);
            case 6: return mma_mx<1, 2>(a, b, c, sa, sb);
            case 7: return mma_mx<1, 3>(a, b, c, sa, sb);
            case 8: return mma_mx<2, 0>(a, b, c, sa, sb);
            case 9: return mma_mx<2, 1>(a, b, c, sa, sb);
            case 10: return mma_mx<2, 2>(a, b, c, sa, sb);
            case 11: return mma_mx<2, 3>(a, b, c, sa, sb);
            case 12: return mma_mx<3, 0>(a, b, c, sa, sb);
            case 13: return mma_mx<3, 1>(a, b, c, sa, sb);
            case 14: return mma_mx<3, 2>(a, b, c, sa, sb);
            default: return mma_mx<3, 3>(a, b, c, sa, sb);
        }
    }
}

// ------------------------------------------------------------------------------------------ tiles
// What a tile product computes:
//   TP_PLAIN   Y = A B^T                        A: M x K, B: N x K
//   TP_GATED   Y = act(A B^T) * (A B2^T), optionally the two products themselves
//   TP_GRAD_X  Y = A B + A2 B2                  A: M x K, B: K x N
//   TP_GRAD_X1 Y = A B                          A: M x K, B: K x N
//   TP_GRAD_W  Y = A^T B, Y2 = A2^T B           A: K x M, B: K x N
enum { TP_PLAIN = 0, TP_GATED = 1, TP_GRAD_X = 2, TP_GRAD_W = 3, TP_GRAD_X1 = 4 };
constexpr bool tp_grad_x(int mode) { return mode == TP_GRAD_X || mode == TP_GRAD_X1; }

struct TileArgs {
    int64_t M, N, K;                     // K in values
    const char *A, *A2, *B, *B2;
    int64_t lda, lda2, ldb, ldb2;        // bytes
    const uint32_t *sA, *sB;             // E2M1, shapes L, M: scales laid out by mx_layout (ksteps dwords x 64 lanes a group)
    int64_t ksteps;                      // steps of 128 values (an even number)
    const uint8_t *rA, *rB, *rB2;        // E2M1, shape S: the scale bytes themselves, rows of ldr* bytes
    int64_t ldrA, ldrB, ldrB2;
    void *Y, *Y2, *Y3;
    int64_t ldy, ldy2, ldy3;             // values
    int dt;                              // type of the outputs
    int act;
    int pairs;                           // TP_GRAD_W: products (2, or 1 when one gradient is wanted)
    int whole;                           // the first `whole` tiles (of each pair) take all of K, one work-group each;
    int splits, sper;                    // the others are cut into `splits` work-groups of `sper` slabs, whose sums go
    float* part;                         // to part + (cut tile * splits + split) * TM * TN, rows of TN (int8: int32 sums)
    const float *fA, *fB, *fB2;          // int8: the scales of the rows
};

// Tile shapes: TM rows of A by TN rows of B (half gate, half up when gated), WM x WN wavefronts.
// DEEP: slabs in LDS, a power of two. Two as a rule: while one is multiplied the next arrives.
template <int TM_, int TN_, int WM_, int WN_, int OCC, int DEEP_ = 2>
struct TileShape {
    typedef TileShape<TM_, TN_, WM_, WN_, OCC> Shallow;
    static constexpr int DEEP = DEEP_;
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, W = WM_ * WN_, THREADS = 64 * W, EU = OCC;
    static constexpr int FM = TM / WM / 16, FN = TN / WN / 16;           // 16 x 16 fragments of a wavefront
    static constexpr int OPA = TM * 128, BUF = (TM + TN) * 128;          // bytes of A's slab, of both
    static constexpr int QA = TM / 8 / W, QB = TN / 8 / W;               // loads of 1 KiB a wavefront and slab
    static constexpr size_t SMEM = DEEP * BUF;
    static constexpr bool LAID = TM >= 128;                              // E2M1: scales laid out ahead
};
typedef TileShape<256, 256, 2, 4, 2> TileL;      // one work-group a compute unit
typedef TileShape<128, 128, 2, 2, 2> TileM;      // two
typedef TileShape<64, 64, 2, 2, 4> TileS;        // four
// The same tiles for grids that leave a compute unit with one work-group (MD) or two (SD). Such a grid waits for its loads: with one slab
// in flight a slab takes as long as its load (0.4 to 0.9 us), its products a quarter of that. The LDS of the work-groups that are not there
// holds two more slabs; sums are the same, in the same order. MI355X, int8, us with two slabs / with four, each with its best cut: 64 tokens 4096 x 11008
// 16.0 / 14.6, 256 27.4 / 21.6, 1024 59.8 / 46.9; 700 tokens 1376 x 4096 16.8 / 10.4. Of more than one turn they are slower, since fewer
// are resident: 2000 tokens 4096 x 4096 M 34.3, MD 43.2. Taken by the int8 products and by grouped products and dX in bf16; fp32 is
// bound by its matrix cores (300 rows of 5 experts gated 1376 x 1000: 37.9 / 38.9).
typedef TileShape<128, 128, 2, 2, 2, 4> TileMD;
typedef TileShape<64, 64, 2, 2, 4, 4> TileSD;
constexpr int TL_ROWS = 256;                     // rows of the largest tile: padding of mx_layout's groups
// Offsets inside a tile's 256 rows (or 64 K rows) are 32-bit, everything else 64-bit: rows of at most 4 MiB.
constexpr int64_t TL_LD_MAX = 4 << 20, TL_ROWS_MAX = 1LL << 31;
// Results of at most 2^44 values (dozens of times the memory), which keeps the plan's counts in 64 bits.
inline bool tile_sizes_ok(int64_t M, int64_t N) { return M <= TL_ROWS_MAX && N <= TL_ROWS_MAX && M * N <= (1LL << 44); }
// A launch takes fewer than 2^32 threads.
inline bool grid_ok(int64_t groups, int64_t threads) { return groups <= 0xFFFFFFFFLL / threads; }

// Work-groups are dealt to the 8 XCDs in turn, so a range of L of them is remapped to give each XCD one
// contiguous part of it.
__device__ __forceinline__ int xcd_range(int id, int L) {
    const int per = L / 8, rem = L % 8, x = id % 8;
    return x * per + (x < rem ? x : rem) + id / 8;
}

// Tile of a work-group, and its split of K. Tiles run in groups of TL_GROUP tile rows, column by column, so that a
// group's panels of A and B stay in its XCD's L2.
constexpr int TL_GROUP = 8;
struct TileAt {
    int cut, split, pair, tm, tn;        // cut: index among the cut tiles, -1 for a whole one
};
// tile `lid` of a pair
__device__ __forceinline__ void tile_place(TileAt& t, int lid, int ny, int nx) {
    const int grp = lid / (TL_GROUP * nx), r0 = grp * TL_GROUP;
    const int rows = ny - r0 < TL_GROUP ? ny - r0 : TL_GROUP;
    const int in = lid - grp * TL_GROUP * nx;
    t.tm = r0 + in % rows;
    t.tn = in / rows;
}
__device__ __forceinline__ void cut_place(TileAt& t, int j, int ny, int nx, int whole) {
    const int per = nx * ny - whole;     // cut tiles of a pair
    t.cut = j;
    t.pair = j / per;
    tile_place(t, whole + j % per, ny, nx);
}
__device__ __forceinline__ TileAt tile_of(int id, int ny, int nx, const TileArgs& g) {
    TileAt t;
    const int w = g.whole * g.pairs;
    if (id < w) {
        const int j = xcd_range(id, w);
        t.cut = -1;
        t.split = 0;
        t.pair = j / g.whole;
        tile_place(t, j % g.whole, ny, nx);
    } else {
        const int n = nx * ny * g.pairs - w, k = id - w;
        t.split = k / n;
        cut_place(t, xcd_range(k % n, n), ny, nx, g.whole);
    }
    // the same in every lane, but divided in vector registers
    t.cut = __builtin_amdgcn_readfirstlane(t.cut);
    t.split = __builtin_amdgcn_readfirstlane(t.split);
    t.pair = __builtin_amdgcn_readfirstlane(t.pair);
    t.tm = __builtin_amdgcn_readfirstlane(t.tm);
    t.tn = __builtin_amdgcn_readfirstlane(t.tn);
    return t;
}

// Rows of B go to wavefronts in groups of four fragments: 64 rows, or 32 gate rows and the same 32 up rows
// (GF = 4 or 2 fragments). Index x of fragment f of a group holds the group's row b_row<GF>(f, x). A lane of the
// result holds rows 4 g .. 4 g + 3 of every fragment, so with this order neighbouring fragments are
// neighbouring columns: 16-byte stores, and row segments of whole cache lines a group.
template <int GF>
__device__ __forceinline__ int b_row(int f, int x) { return (x >> 2) * (4 * GF) + 4 * f + (x & 3); }

// LDS, operand contiguous along K: rows of 128 bytes, chunk c of row r at position c ^ key(r). The 16 rows
// of a fragment then spread over the banks. For A fragments hold consecutive rows; for B the rows of b_row.
__device__ __forceinline__ int key_a(int r) { return r & 7; }
template <int GF>
__device__ __forceinline__ int key_b(int r) { return (r & 3) | (((r / (4 * GF)) & 1) << 2); }

// LDS, operand contiguous along M or N ("transposed"): rows of K, each of the tile's T values. A fragment reads
// 16 columns of 16 K rows at once, U = 32 (bf16) or 64 (fp32) bytes of each; unit u of K row k lies at
// position u ^ key_t(k), so the rows' units spread over the banks (bf16: 16 rows k & 3, k >> 3 of a
// transposing read; fp32: 4 rows k >> 2).
template <int E, int T>
__device__ __forceinline__ int key_t(int k) {
    if constexpr (E == EL_BF16) return ((k & 3) | (((k >> 3) & 3) << 2)) & (T / 16 - 1);
    else return (k >> 2) & 3;
}

typedef __attribute__((address_space(3))) void* lds_ptr;

// 16 bytes a lane from base + off straight to LDS (lds + 16 lane; base and lds are the wavefront's). HIDDEN:
// the compiler takes a transposing LDS read to depend on every load to LDS in flight and would wait for
// the slab just requested, so beside such reads the load is written out, and where more slabs are in flight than one. It has
// no output register, and landed waits for it. It leaves its LDS base in m0, which nothing else in those kernels uses.
template <bool HIDDEN>
__device__ __forceinline__ void dma16(const char* base, uint32_t off, char* lds) {
    if constexpr (HIDDEN) {
        const tl_i4 rsrc = {(int)(uintptr_t)base, (int)((uintptr_t)base >> 32) & 0xFFFF, -1, 0x00020000};
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                     :: "v"(off), "s"(rsrc), "s"((uint32_t)(uintptr_t)(lds_ptr)lds) : "memory");
    } else {
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0xFFFFFFFF, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)lds, 16, (int)off, 0, 0, 0);
    }
}

// Waits for a wavefront's loads to LDS, but for the last LATER of them.
template <int LATER = 0>
__device__ __forceinline__ void landed() {
    static_assert(LATER < 64, "the counter's six bits");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (LATER & 15) | (LATER >> 4) << 14);      // vmcnt(LATER) alone
}
// Barrier at which every wavefront's loads to LDS have landed. The wait is written out: a barrier by itself
// orders ordinary LDS and global accesses, not the loads that write LDS.
__device__ __forceinline__ void landed_barrier() {
    landed();
    __syncthreads();
}

// One tile, or one split of it. Large products are bound by feeding the matrix cores: at 8192 tokens of 4096 x 11008
// weights (MI355X) the bf16 gated block takes 1110 us (1.33 PFLOP/s, matrix cores busy 66 % of the time at a clock of
// 1.7 GHz), dX 1045 us (1.42 PFLOP/s), both weight gradients 1140 us (1.30 PFLOP/s), the 4-bit product 157 us (4.7
// PFLOP/s, 60 % busy at 1.9 GHz), the 4-bit gated block 350 us (4.2 PFLOP/s, 53 %: its tiles have 16 slabs between
// their first loads and their activations). With their operands in registers the same instructions run at 2.1 (bf16) and
// 7.4 PFLOP/s (E2M1), all the time busy at 2.06 GHz: the LDS reads and the loads cost clock as well as time. A slab of
// shape L has 192 KiB read from LDS, 771 clocks by its counter (255 bytes a clock), beside the 2048 of its matrix instructions (64 a
// wavefront, two wavefronts a SIMD, 16 clocks each): LDS is not the bound. With every load a hit in L2 (all of them of one and the same
// slab) bf16 products take 12 % less and int8 ones 7 %: the loads' latency, of which half a slab's products to a whole one's cover what
// they can. Neither bringing later slabs' lines into L2 by loads of 4 bytes a line (28 to 40 % slower: 64 requests a load) nor four wavefronts of
// 128 x 128 with their sums pinned in accumulation registers (weight gradients 14 % slower: nothing runs beside a barrier) helped. The
// 32 x 32 instructions, by themselves, are slower (1.9 and 6.7 PFLOP/s). No LDS bank conflicts in any of them. A
// work-group that walks over its tiles and loads the next one's first slab before the epilogue changed none of these by
// more than 2 %; four wavefronts of 128 x 128 instead of eight of 128 x 64 read a third less LDS but no longer fit
// their sums and fragments into registers (4-bit product 222 -> 276 us at the time). Grids of about one work-group a
// compute unit are bound by the latency of a slab instead: at 1024 tokens of 4096 x 11008 4-bit weights 256 work-groups of
// shape M walk 43 slabs each in 34 us, 0.79 us a slab whose matrix instructions take 0.25 (32 a wavefront, one wavefront a SIMD),
// since one slab's products are all that covers the next but one's loads.
template <int E, int MODE, typename C>
__device__ __forceinline__ void tile_body(const TileArgs& g, const TileAt& at) {
    extern __shared__ __align__(16) char tl_sm[];
    constexpr bool TA = MODE == TP_GRAD_W, TB = tp_grad_x(MODE) || MODE == TP_GRAD_W, GATED = MODE == TP_GATED;
    static_assert(!TB || (E != EL_MX && E != EL_I8), "blocks of E2M1 lie along K; int8 has no gradients");
    constexpr bool HID = (TB && E == EL_BF16) || C::DEEP > 2;
    static_assert(C::DEEP == 2 || E != EL_MX, "the scales' loads would be waited for with the slabs behind them");
    constexpr int EPC = el_chunk<E>(), BK = 8 * EPC, ES = 16 / (E == EL_MX ? 16 : EPC);   // ES: bytes of a dense value
    constexpr int FM = C::FM, FN = C::FN, QA = C::QA, QB = C::QB;
    constexpr int GF = GATED ? 2 : 4, GW = GATED ? 32 : 64;              // a group's fragments and columns (of a half)
    constexpr int FW = GATED ? FN / 2 : FN, SUB = GF / FW;               // fragments a half of a wavefront, wavefronts a group
    constexpr int TN_OUT = GATED ? C::TN / 2 : C::TN;                    // output columns of a tile
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int x16 = lane & 15, g4 = lane >> 4;
    const int wm = wave / C::WN, wn = wave % C::WN, grp = wn / SUB, sub = wn % SUB;
    const int64_t m0 = (int64_t)at.tm * C::TM, n0 = (int64_t)at.tn * TN_OUT;
    const int mlast = (int)(g.M - 1 - m0 < C::TM - 1 ? g.M - 1 - m0 : C::TM - 1);          // last row inside
    const int nlast = (int)(g.N - 1 - n0 < TN_OUT - 1 ? g.N - 1 - n0 : TN_OUT - 1);
    const bool cut = at.cut >= 0;
    const int wpair = MODE == TP_GRAD_W ? at.pair : 0;

    // ---- staging: loads of 16 bytes a lane; load q of a wavefront fills KiB q * W + wave of its operand
    const int r8 = lane >> 3, pos = lane & 7;
    // chunk of a K-contiguous operand that the lane loads (the same in all loads: they are a multiple of 32 rows apart)
    const int cA = pos ^ r8, cB = pos ^ key_b<GF>(wave * 8 + r8);
    // K row of a transposed operand (in load 0), and the chunk of it that the lane loads
    constexpr int LA = C::TM * ES / 16, LB = C::TN * ES / 16;            // lanes (chunks) a K row
    constexpr int UC = E == EL_BF16 ? 2 : 4;                             // chunks a unit
    auto tchunk = [&](int k, int p, int key, int last) {
        const int c = ((p / UC) ^ key) * UC + p % UC;
        return c * EPC <= last ? c : last / EPC;
    };
    const char *pA, *pB, *pB2 = nullptr;
    int64_t stepA, stepB;
    uint32_t offA[QA], offB[QB];
    auto operands = [&](const char* A, int64_t lda, const char* B, int64_t ldb) {
        pA = A + (TA ? m0 * ES : m0 * lda);
        pB = B + (TB ? n0 * ES : n0 * ldb);
        if (GATED) pB2 = g.B2 + n0 * g.ldb2;
        stepA = TA ? BK * lda : 128;
        stepB = TB ? BK * ldb : 128;
#pragma unroll
        for (int q = 0; q < QA; q++) {
            if constexpr (TA) {
                const int k = (q * C::W + wave) * (64 / LA) + lane / LA;
                offA[q] = (uint32_t)k * (uint32_t)lda + tchunk(k, lane % LA, key_t<E, C::TM>(k), mlast) * 16;
            } else {
                const int r = (q * C::W + wave) * 8 + r8;
                offA[q] = (uint32_t)(r < mlast ? r : mlast) * (uint32_t)lda + cA * 16;
            }
        }
#pragma unroll
        for (int q = 0; q < QB; q++) {
            if constexpr (TB) {
                const int k = (q * C::W + wave) * (64 / LB) + lane / LB;
                offB[q] = (uint32_t)k * (uint32_t)ldb + tchunk(k, lane % LB, key_t<E, C::TN>(k), nlast) * 16;
            } else {
                // gated: the first half of the slab's rows are gate rows, the second up rows
                const int r = (q * C::W + wave) * 8 + r8, rb = GATED ? r & (C::TN / 2 - 1) : r;
                offB[q] = (uint32_t)(rb < nlast ? rb : nlast) * (uint32_t)(GATED && q >= QB / 2 ? g.ldb2 : ldb) + cB * 16;
            }
        }
    };
    const int64_t nch = (g.K + EPC - 1) / EPC;           // chunks of K, the last one possibly partial
    const int part = E == EL_MX ? 0 : (int)(g.K % EPC);  // values in a partial last chunk (E2M1 blocks are whole)
    const int slabsK = (int)((g.K + BK - 1) / BK);
    const int whole = (int)(g.K / BK);                   // slabs that lie inside K
    const int s0 = cut ? at.split * g.sper : 0;          // this work-group's slabs
    const int slabs = cut && slabsK - s0 > g.sper ? g.sper : slabsK - s0;
    int ts = 0;                                          // slab to be staged next

    // Staging of slab ts into buffer buf, load by load (A's, then B's) for a slab inside K. E2M1: also for the last slab, where
    // a chunk past K is replaced by the last one; its scales are zero on both sides, so its products vanish.
    constexpr int LOADS = QA + QB;
    auto load_one = [&](int buf, int d) {
        char* la = tl_sm + buf * C::BUF + wave * 1024;
        int backA = 0, backB = 0;
        if constexpr (E == EL_MX) {
            const int left = (int)nch - 1 - ts * 8;      // the last chunk's place from this slab's first
            backA = left < cA ? (left - cA) * 16 : 0;
            backB = left < cB ? (left - cB) * 16 : 0;
        }
        if (d < QA) dma16<HID>(pA, offA[d < QA ? d : 0] + backA, la + d * (C::W * 1024));
        else dma16<HID>(GATED && d - QA >= QB / 2 ? pB2 : pB, offB[d >= QA ? d - QA : 0] + backB, la + C::OPA + (d - QA) * (C::W * 1024));
    };
    auto staged = [&]() {
        ts++;
        pA += stepA;
        pB += stepB;
        if (GATED) pB2 += 128;
    };
    // The whole of slab ts at once, also one that K ends in. K-contiguous operands: chunks past K become zero.
    // Transposed ones: K rows past K become zero. (Rows and columns past M and N repeat the last one and are never stored.)
    auto stage = [&](int buf) {
        if (E == EL_MX || ts < whole) {
#pragma unroll
            for (int d = 0; d < LOADS; d++) load_one(buf, d);
        } else {
            char* la = tl_sm + buf * C::BUF + wave * 1024;
            char* lb = la + C::OPA;
            constexpr int Q = C::W * 1024;
            const tl_i4 zero = {0, 0, 0, 0};
            const int left = (int)(nch - (int64_t)ts * 8), krows = (int)(g.K - (int64_t)ts * BK);
#pragma unroll
            for (int q = 0; q < QA; q++) {
                const bool in = TA ? (q * C::W + wave) * (64 / LA) + lane / LA < krows : cA < left;
                if (in) dma16<HID>(pA, offA[q], la + q * Q);
                else *reinterpret_cast<tl_i4*>(la + q * Q + lane * 16) = zero;
            }
#pragma unroll
            for (int q = 0; q < QB; q++) {
                const char* b = GATED && q >= QB / 2 ? pB2 : pB;
                const bool in = TB ? (q * C::W + wave) * (64 / LB) + lane / LB < krows : cB < left;
                if (in) dma16<HID>(b, offB[q], lb + q * Q);
                else *reinterpret_cast<tl_i4*>(lb + q * Q + lane * 16) = zero;
            }
        }
        staged();
    };
    // values past K of a partial last chunk, once it has landed: each lane clears its own chunks
    auto clear_part = [&](int t, int buf) {
        if (s0 + t != slabsK - 1) return;
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0) alone
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        char* la = tl_sm + buf * C::BUF + wave * 1024 + lane * 16;
        auto cut = [&](char* p) { *reinterpret_cast<tl_i4*>(p) = chunk_head<E>(*reinterpret_cast<tl_i4*>(p), part); };
        const int last = (int)((nch - 1) & 7);           // the chunk's place in the slab
        if (!TA && cA == last)
            for (int q = 0; q < QA; q++) cut(la + q * C::W * 1024);
        if (!TB && cB == last)
            for (int q = 0; q < QB; q++) cut(la + C::OPA + q * C::W * 1024);
    };

    el_sums<E> acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) acc[i][j] = el_sums<E>{0, 0, 0, 0};

    // Scales of a slab's two steps (E2M1). Shapes L and M take them laid out, a dword of a lane for four fragments
    // (64 rows). Shape S reads 8 bytes (a slab) of the row of each of its 4 fragments, which saves the
    // launch ahead of the product; with M's 8 fragments these loads, 16 rows each, cost more than it
    // (2048 x 11008 x 4096: 123 us, laid out 67; S at 333 x 1376 x 1000: 5.2 us, laid out 10.4).
    constexpr bool LAID = C::LAID;
    constexpr int SA = LAID ? FM / 4 : FM, SB = LAID ? 1 : FN;
    uint32_t scA[SA][2], scB[SB][2], nxA[SA][2], nxB[SB][2];
    const uint32_t *qA = nullptr, *qB = nullptr;         // L, M: step 0 of the slab whose scales are loaded next (uniform)
    const uint8_t *sa = nullptr, *sb = nullptr, *sb2 = nullptr;
    uint32_t soA[SA], soB[SB];
    if constexpr (E == EL_MX && LAID) {
        qA = g.sA + ((m0 + wm * FM * 16) / 64 * g.ksteps + 2 * s0) * 64;
        qB = g.sB + ((n0 / GW + grp) * g.ksteps + 2 * s0) * 64;
    }
    if constexpr (E == EL_MX && !LAID) {
        sa = g.rA + m0 * g.ldrA + s0 * 8;
        sb = g.rB + n0 * g.ldrB + s0 * 8;
        if (GATED) sb2 = g.rB2 + n0 * g.ldrB2 + s0 * 8;
#pragma unroll
        for (int i = 0; i < FM; i++) {
            const int r = wm * FM * 16 + 16 * i + x16;
            soA[i] = (uint32_t)(r < mlast ? r : mlast) * (uint32_t)g.ldrA;
        }
#pragma unroll
        for (int j = 0; j < FN; j++) {
            const int r = grp * GW + b_row<GF>(sub * FW + j % FW, x16);
            soB[j] = (uint32_t)(r < nlast ? r : nlast) * (uint32_t)(j >= FW ? g.ldrB2 : g.ldrB);
        }
    }
    // L, M: step s of the next slab, over the register that its last use has left. Buffer loads: a uniform base and one
    // lane offset, where plain ones would hold a 64-bit address for each of the three.
    auto load_laid = [&](int s) {
        auto word = [&](const uint32_t* p) {
            const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t*>(p), 0, 0xFFFFFFFF, 0x00020000);
            return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, lane * 4, 0, 0);
        };
#pragma unroll
        for (int a = 0; a < SA; a++) scA[a][s] = word(qA + (a * g.ksteps + s) * 64);
        scB[0][s] = word(qB + s * 64);
        if (s == 1) {
            qA += 128;
            qB += 128;
        }
    };
    // S: both steps of slab t (of this work-group), to be taken when its products begin
    auto load_raw = [&](int t) {
        const int left = (int)nch - (s0 + t) * 8;        // blocks from the slab's first
        auto at = [&](int f) { return f < FM ? sa + soA[f < FM ? f : 0] : (f - FM >= FW ? sb2 : sb) + soB[f < FM ? 0 : f - FM]; };
        if (left >= 8) {
#pragma unroll
            for (int f = 0; f < FM + FN; f++) {
                const uint32_t* q = reinterpret_cast<const uint32_t*>(at(f));
                uint32_t* v = f < FM ? nxA[f < FM ? f : 0] : nxB[f < FM ? 0 : f - FM];
                v[0] = q[0];
                v[1] = q[1];
            }
        } else {
            // blocks past K: the smallest scale on both sides, whose products vanish
#pragma unroll
            for (int f = 0; f < FM + FN; f++) {
                const uint32_t* q = reinterpret_cast<const uint32_t*>(at(f));
                uint32_t* v = f < FM ? nxA[f < FM ? f : 0] : nxB[f < FM ? 0 : f - FM];
                const uint32_t lo = q[0], hi = left > 4 ? q[1] : 0u;
                v[0] = g4 < left ? lo : 0u;
                v[1] = 4 + g4 < left ? hi : 0u;
            }
        }
        sa += 8;
        sb += 8;
        if (GATED) sb2 += 8;
    };
    auto take_raw = [&]() {
#pragma unroll
        for (int s = 0; s < 2; s++) {
#pragma unroll
            for (int i = 0; i < FM; i++) scA[i][s] = nxA[i][s] >> (8 * g4);
#pragma unroll
            for (int j = 0; j < FN; j++) scB[j][s] = nxB[j][s] >> (8 * g4);
        }
    };

    // fragment i of A (j of B) for step s of the slab at LDS offset `at`. Transposed: lane x16 of group g4 ends with
    // the K rows of its chunk of column 16 i + x16 (bf16: 8 rows from two transposing reads of 4; fp32: 4 rows);
    // the key of those rows depends on the lane alone, so i enters the address by one exclusive or.
    const int lfA = !TA ? (wm * FM * 16 + x16) * 128 + ((g4 ^ key_a(x16)) << 4)
                  : E == EL_BF16 ? (8 * g4 + (x16 >> 2)) * (C::TM * 2) +
                                   ((wm * FM) ^ key_t<E, C::TM>(8 * g4 + (x16 >> 2))) * 32 + (x16 & 3) * 8
                                 : 4 * g4 * (C::TM * 4) + ((wm * FM) ^ g4) * 64 + x16 * 4;
    const int rB0 = grp * GW + b_row<GF>(sub * FW, x16);
    const int lfB = !TB ? rB0 * 128 + ((g4 ^ key_b<GF>(rB0)) << 4)
                  : E == EL_BF16 ? (8 * g4 + (x16 >> 2)) * (C::TN * 2) +
                                   ((wn * FN) ^ key_t<E, C::TN>(8 * g4 + (x16 >> 2))) * 32 + (x16 & 3) * 8
                                 : 4 * g4 * (C::TN * 4) + ((wn * FN) ^ g4) * 64 + x16 * 4;
    auto tr_frag = [&](int off, int f, int s, int T) -> tl_i4 {
        tl_i4 r;
        if constexpr (E == EL_BF16) {
            const char* p = tl_sm + (off ^ (f * 32)) + s * 32 * T * 2;
            const tl_s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tl_s4*)p);
            const tl_s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) tl_s4*)(p + 8 * T));
            reinterpret_cast<tl_s4*>(&r)[0] = lo;
            reinterpret_cast<tl_s4*>(&r)[1] = hi;
        } else {
            const char* p = tl_sm + (off ^ (f * 64)) + s * 16 * T * 4;
#pragma unroll
            for (int e = 0; e < 4; e++) r[e] = *reinterpret_cast<const int*>(p + e * T * 4);
        }
        return r;
    };
    auto fragA = [&](int at, int i, int s) -> tl_i4 {
        if constexpr (TA) return tr_frag(at + lfA, i, s, C::TM);
        else return *reinterpret_cast<const tl_i4*>(tl_sm + ((at + lfA) ^ (s * 64)) + i * 2048);
    };
    auto fragB = [&](int at, int j, int s) -> tl_i4 {
        at += C::OPA;
        if constexpr (TB) return tr_frag(at + lfB, j, s, C::TN);
        else return *reinterpret_cast<const tl_i4*>(tl_sm + ((at + lfB) ^ (s * 64)) + (j / FW) * (C::TN / 2 * 128) + (j % FW) * 512);
    };

    // The loop is software-pipelined by half a slab: while one step's products run, the next step's fragments
    // come from LDS, and the barrier stands between the two steps of a slab. At the barrier every wavefront
    // has all of slab t in registers or accumulators, so its buffer takes slab t + 2, and slab t + 1 has had
    // a whole slab's products to arrive in. Registers: a fragment of A is overwritten in place by the next
    // step's once its products are issued, except that the first step's last ones are kept beside the second
    // step's (fx), whose loads would otherwise be waited for at the barrier.
    constexpr int KEEP = FM / 4, INPL = FM - KEEP;
    tl_i4 fa[FM], fx[KEEP ? KEEP : 1], fb[2][FN];
    auto slab_at = [&](int t) { return (t & (C::DEEP - 1)) * C::BUF; };
    auto products = [&](int i, int s, tl_i4 a) {
#pragma unroll
        for (int j = 0; j < FN; j++) {
            // rows of the result are B's rows (output columns), columns are A's rows
            if constexpr (E == EL_MX && LAID)
                acc[i][j] = mma_step<E>(fb[s][j], a, acc[i][j], (int)scB[0][s], j, (int)scA[i / 4][s], i & 3);
            else if constexpr (E == EL_MX)
                acc[i][j] = mma_step<E>(fb[s][j], a, acc[i][j], (int)scB[j][s], 0, (int)scA[i][s], 0);
            else
                acc[i][j] = mma_step<E>(fb[s][j], a, acc[i][j], 0, 0, 0, 0);
        }
    };
    // One step: the products of A's fragment i with all of B's, then the reads that replace what they used and
    // (LOAD) loads of the slab after the next into buffer buf, spread over the step: a burst of either holds up the
    // products (8192 tokens, loads spread instead of issued at once: bf16 gated block 1165 -> 1108 us, weight
    // gradients 1270 -> 1145 us, 4-bit product 182 -> 167 us; over half the step: 1 to 8 % slower than over all of it; two
    // of eight put off to the next step: bf16 3 to 5 % slower, they land late). The reads end two rows of products
    // before the step does, so that the barrier finds them done (weight gradients 1157 -> 1138 us).
    auto step = [&](int s, int at, auto READ, auto LOAD, int buf) {
        const int nx = s ^ 1;            // the step whose fragments are read (slab at `at`), unless there is none
#pragma unroll
        for (int i = 0; i < FM; i++) {
            products(i, s, s == 1 && i >= INPL ? fx[i >= INPL ? i - INPL : 0] : fa[i]);
            if constexpr (LOAD.value) {
#pragma unroll
                for (int d = i * LOADS / FM; d < (i + 1) * LOADS / FM; d++) load_one(buf, d);
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (READ.value) {
                if (i < INPL) fa[i] = fragA(at, i, nx);
                if (i < KEEP) {
                    if (s == 0) fx[i] = fragA(at, INPL + i, nx);
                    else fa[INPL + i] = fragA(at, INPL + i, nx);
                }
                if (i < FN) fb[nx][i] = fragB(at, i, nx);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    operands(MODE == TP_GRAD_W && wpair ? g.A2 : g.A, MODE == TP_GRAD_W && wpair ? g.lda2 : g.lda, g.B, g.ldb);
    for (int pair = 0; pair < (MODE == TP_GRAD_X ? 2 : 1); pair++) {
        if (MODE == TP_GRAD_X && pair) operands(g.A2, g.lda2, g.B2, g.ldb2);     // into the same sums
        ts = s0;
        pA += s0 * stepA;
        pB += s0 * stepB;
        if (GATED) pB2 += s0 * 128;
        const int inside = E == EL_MX || whole - s0 > slabs ? slabs : whole - s0;
        // With four slabs in LDS: the barrier in slab t leaves those behind t + 1 in flight, of whole slabs alone (whose loads are always
        // the same in number; the loads of the slab that K ends in, if they are there, are the last ones and only make the wait longer).
        auto deep_barrier = [&](int t) {
            const int last = t + C::DEEP - 1 < inside - 1 ? t + C::DEEP - 1 : inside - 1, later = last - (t + 1);
            if (later >= 2) landed<2 * LOADS>();
            else if (later == 1) landed<LOADS>();
            else landed();
            __syncthreads();
        };
        stage(0);
        if constexpr (C::DEEP == 2) {
            if (part && (!TA || !TB)) clear_part(0, 0);
            if constexpr (E == EL_MX && LAID) load_laid(0);
            if constexpr (E == EL_MX && !LAID) load_raw(0);
            landed_barrier();
            if (slabs > 1) stage(1);
        } else {
            static_assert(C::DEEP == 4, "waits are written for four slabs");
#pragma unroll
            for (int b = 1; b < C::DEEP; b++)
                if (b < slabs) stage(b);
            if (part && (!TA || !TB)) clear_part(0, 0);
            deep_barrier(-1);
        }
#pragma unroll
        for (int j = 0; j < FN; j++) fb[0][j] = fragB(0, j, 0);
#pragma unroll
        for (int i = 0; i < FM; i++) fa[i] = fragA(0, i, 0);
        // LOAD: slab t + 2 (t + DEEP) exists and lies inside K; TAIL: it exists and K ends in it; NEXT: slab t + 1 exists. Constants, so
        // that the loads of a turn of the main loop are always the same in number and the wait for the
        // scales leaves the slab's loads in flight.
        typedef std::true_type Y1;
        typedef std::false_type N0;
        auto turn = [&](int t, auto LOAD, auto TAIL, auto NEXT) {
            if constexpr (E == EL_MX && LAID) load_laid(1);
            if constexpr (E == EL_MX && !LAID) take_raw();
            step(0, slab_at(t), Y1{}, N0{}, 0);
            if constexpr (NEXT.value) {
                if (part && (!TA || !TB)) clear_part(t + 1, (t + 1) & (C::DEEP - 1));
                // slab t + 1 has landed, and every wavefront holds the rest of slab t
                if constexpr (C::DEEP == 2) landed_barrier();
                else deep_barrier(t);
                if constexpr (E == EL_MX && LAID) load_laid(0);      // ahead of the slab's loads
                if constexpr (E == EL_MX && !LAID) load_raw(t + 1);
                if constexpr (TAIL.value) stage(t & (C::DEEP - 1));
            }
            __builtin_amdgcn_sched_barrier(0);
            step(1, slab_at(t + 1), NEXT, LOAD, t & (C::DEEP - 1));
            if constexpr (LOAD.value) staged();
        };
        int t = 0;
        for (; t + C::DEEP < inside; t++) turn(t, Y1{}, N0{}, Y1{});
        if constexpr (E != EL_MX) {
            if (t + C::DEEP < slabs) turn(t++, N0{}, Y1{}, Y1{});
        }
        if constexpr (C::DEEP == 2) {
            if (t + 1 < slabs) turn(t++, N0{}, N0{}, Y1{});
        } else {
            while (t + 1 < slabs) turn(t++, N0{}, N0{}, Y1{});
        }
        turn(t, N0{}, N0{}, N0{});
        // the next pair's first slab overwrites the buffers only once every wavefront has read its last fragments
        if (MODE == TP_GRAD_X && pair == 0) __syncthreads();
    }

    // ---- epilogue: lane holds output row x16 of fragment row i and runs of neighbouring columns
    const bool w2 = MODE == TP_GRAD_W && wpair;
    // split sums: the tile's own rows and columns, kept apart from its place in the result
    float* pt = cut ? g.part + ((int64_t)at.cut * g.splits + at.split) * (C::TM * C::TN) - (m0 * C::TN + n0) : nullptr;
    void* Y = cut ? pt : w2 ? g.Y2 : g.Y;
    const int64_t ldY = cut ? C::TN : w2 ? g.ldy2 : g.ldy;
    const int dt = cut ? KQ_F32 : g.dt;
    const int64_t nrun = n0 + grp * GW + g4 * (4 * GF) + 4 * sub * FW;
    // int8: a sum times the scales of its two rows, their product first (a token's large scale and a weight's small one
    // cancel); a cut tile keeps the whole numbers
    float cs[E == EL_I8 ? 4 * FW : 1], cs2[E == EL_I8 && GATED ? 4 * FW : 1];
    if constexpr (E == EL_I8) {
        if (!cut) {
#pragma unroll
            for (int e = 0; e < 4 * FW; e++) {
                const int64_t n = nrun + e < g.N ? nrun + e : g.N - 1;
                cs[e] = g.fB[n];
                if constexpr (GATED) cs2[e] = g.fB2[n];
            }
        }
    }
    auto value = [&](auto sum, float sa, float sb) {
        if constexpr (E == EL_I8) return cut ? __int_as_float(sum) : (float)sum * (sa * sb);
        else return sum;
    };
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const int64_t m = m0 + wm * FM * 16 + 16 * i + x16;
        if (m >= g.M) continue;
        if (TB && E == EL_BF16 && !cut) {
            // two fragments at a time: lane groups exchange halves, so that each has 8 columns of one of them and a row is written in
            // 64 bytes
#pragma unroll
            for (int j = 0; j < FN; j += 2) {
                uint32_t p[2][2];
#pragma unroll
                for (int h = 0; h < 2; h++) {
#pragma unroll
                    for (int f = 0; f < 2; f++)
                        p[f][h] = (uint32_t)to_bf16((float)acc[i][j + f][2 * h]) | (uint32_t)to_bf16((float)acc[i][j + f][2 * h + 1]) << 16;
                    const auto q = __builtin_amdgcn_permlane16_swap(p[0][h], p[1][h], false, false);
                    p[0][h] = q[0];
                    p[1][h] = q[1];
                }
                const int64_t n = n0 + wn * FN * 16 + 16 * (j + (g4 & 1)) + 8 * (g4 >> 1);
                uint16_t* out = static_cast<uint16_t*>(Y) + m * ldY + n;
                if (n + 8 <= g.N) {
                    *reinterpret_cast<uint4*>(out) = make_uint4(p[0][0], p[0][1], p[1][0], p[1][1]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (n + e < g.N) out[e] = (uint16_t)(p[e / 4][e / 2 % 2] >> (16 * (e % 2)));
                }
            }
        } else if constexpr (TB) {
#pragma unroll
            for (int j = 0; j < FN; j++) {
                const int64_t n = n0 + wn * FN * 16 + 16 * j + 4 * g4;
                const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                store_run<4>(Y, dt, m * ldY + n, v, g.N - n);
            }
        } else {
            const float rs = E == EL_I8 && !cut ? g.fA[m] : 0.0f;
            float a[4 * FW];
#pragma unroll
            for (int j = 0; j < FW; j++)
#pragma unroll
                for (int r = 0; r < 4; r++) a[4 * j + r] = value(acc[i][j][r], rs, cs[E == EL_I8 ? 4 * j + r : 0]);
            if constexpr (!GATED) {
                store_run<4 * FW>(Y, dt, m * ldY + nrun, a, g.N - nrun);
            } else {
                float h[4 * FW], b[4 * FW];
#pragma unroll
                for (int j = 0; j < FW; j++)
#pragma unroll
                    for (int r = 0; r < 4; r++) b[4 * j + r] = value(acc[i][j + FW][r], rs, cs2[E == EL_I8 && GATED ? 4 * j + r : 0]);
                if (cut) {
                    store_run<4 * FW>(pt, KQ_F32, m * C::TN + nrun, a, g.N - nrun);
                    store_run<4 * FW>(pt, KQ_F32, m * C::TN + C::TN / 2 + nrun, b, g.N - nrun);
                } else {
                    act_times(h, a, b, g.act);
                    store_run<4 * FW>(Y, dt, m * ldY + nrun, h, g.N - nrun);
                    if (g.Y2) store_run<4 * FW>(g.Y2, dt, m * g.ldy2 + nrun, a, g.N - nrun);
                    if (g.Y3) store_run<4 * FW>(g.Y3, dt, m * g.ldy3 + nrun, b, g.N - nrun);
                }
            }
        }
    }
}

// the tile of work-group `id` of a whole product
template <int MODE, typename C>
__device__ __forceinline__ TileAt tile_at(const TileArgs& g, int id) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN;
    return tile_of(id, (int)((g.M + C::TM - 1) / C::TM), (int)((g.N + TN_OUT - 1) / TN_OUT), g);
}

template <int E, int MODE, typename C>
__global__ __launch_bounds__(C::THREADS, C::EU) void tile_kernel(TileArgs g) {
    tile_body<E, MODE, C>(g, tile_at<MODE, C>(g, (int)blockIdx.x));
}

// dX and the weight gradients side by side: `first` work-groups for dX, the rest for the others. For small products, which
// leave compute units idle, and whose launches cost as much as they do (61 tokens of 1376 x 1000 fp32: 14.4 us, one
// after the other 9.5 and 9.1 and a launch between; the whole call 22.9 -> 19.3 us).
template <int E, typename C>
__global__ __launch_bounds__(C::THREADS, C::EU) void tile_grads_kernel(TileArgs x, TileArgs w, int first) {
    if ((int)blockIdx.x < first) tile_body<E, TP_GRAD_X, C>(x, tile_at<TP_GRAD_X, C>(x, (int)blockIdx.x));
    else tile_body<E, TP_GRAD_W, C>(w, tile_at<TP_GRAD_W, C>(w, (int)blockIdx.x - first));
}

// Sums of the splits, in split order, and the epilogue: 4 columns a thread, TM * TN_OUT / 1024 work-groups a tile.
// HBM-bound, or latency (96 L tiles in two splits, the tail of the weight gradients at 8192 tokens: 10.6 us, 5.9 TB/s;
// 16 S tiles in 15: 4 us). Splits are not added by atomics: their order would change the sums.
// Piece `piece` of them, of the cut tile `at`:
template <int MODE, typename C, int E = EL_F32>
__device__ __forceinline__ void tile_reduce(const TileArgs& g, const TileAt& at, int piece) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN;
    const int e = piece * 256 + threadIdx.x, r = e / (TN_OUT / 4), c = e % (TN_OUT / 4) * 4;
    const int64_t m = (int64_t)at.tm * C::TM + r, n = (int64_t)at.tn * TN_OUT + c;
    if (m >= g.M || n >= g.N) return;
    const float* p = g.part + (int64_t)at.cut * g.splits * (C::TM * C::TN) + r * C::TN + c;
    auto sum = [&](const float* q, const float* scales, float (&v)[4]) {
        auto load = [&](int k) { return *reinterpret_cast<const el_sums<E>*>(q + (int64_t)k * (C::TM * C::TN)); };
        el_sums<E> s = load(0);
        auto add = [&](const el_sums<E>& t) {
#pragma unroll
            for (int r = 0; r < 4; r++) s[r] += t[r];
        };
        int k = 1;
        for (; k + 4 <= g.splits; k += 4) {      // four loads in flight, added in order
            const el_sums<E> t0 = load(k), t1 = load(k + 1), t2 = load(k + 2), t3 = load(k + 3);
            add(t0); add(t1); add(t2); add(t3);
        }
        for (; k < g.splits; k++) add(load(k));
#pragma unroll
        for (int r = 0; r < 4; r++) {
            if constexpr (E == EL_I8) v[r] = (float)s[r] * (g.fA[m] * scales[n + r < g.N ? n + r : g.N - 1]);
            else v[r] = s[r];
        }
    };
    float a[4];
    sum(p, g.fB, a);
    if constexpr (MODE == TP_GATED) {
        float b[4], h[4];
        sum(p + C::TN / 2, g.fB2, b);
        act_times(h, a, b, g.act);
        store_run<4>(g.Y, g.dt, m * g.ldy + n, h, g.N - n);
        if (g.Y2) store_run<4>(g.Y2, g.dt, m * g.ldy2 + n, a, g.N - n);
        if (g.Y3) store_run<4>(g.Y3, g.dt, m * g.ldy3 + n, b, g.N - n);
    } else {
        const bool w2 = MODE == TP_GRAD_W && at.pair;
        store_run<4>(w2 ? g.Y2 : g.Y, g.dt, m * (w2 ? g.ldy2 : g.ldy) + n, a, g.N - n);
    }
}

// the piece of work-group `block` of a whole product
template <int MODE, typename C, int E = EL_F32>
__device__ __forceinline__ void tile_reduce(const TileArgs& g, int block) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN, PER = C::TM * TN_OUT / 1024;
    TileAt at;
    cut_place(at, block / PER, (int)((g.M + C::TM - 1) / C::TM), (int)((g.N + TN_OUT - 1) / TN_OUT), g.whole);
    tile_reduce<MODE, C, E>(g, at, block % PER);
}

template <int MODE, typename C, int E>
__global__ __launch_bounds__(256) void tile_reduce_kernel(TileArgs g) {
    tile_reduce<MODE, C, E>(g, (int)blockIdx.x);
}

template <typename C>
__global__ __launch_bounds__(256) void tile_reduce_grads_kernel(TileArgs x, TileArgs w, int first) {
    if ((int)blockIdx.x < first) tile_reduce<TP_GRAD_X, C>(x, (int)blockIdx.x);
    else tile_reduce<TP_GRAD_W, C>(w, (int)blockIdx.x - first);
}

// How a product is cut: tile shape (0 L, 1 M, 2 S, 3 MD, 4 SD) and the tiles whose K is split, by the estimated time of each choice.
// A slab of a tile takes `lat` us by itself on a compute unit and `w` us of a busy one's matrix cores, a tile
// `fix` more for its first loads and its epilogue; split sums are written and read once at 3.5 TB/s by a
// second launch (4 us), and E2M1 scales laid out by one of 3 us. The constants are fitted to measurements of 8
// products at 15 sizes each, all shapes and 1 to 16 splits (MI355X); when they were, the choice was within 2 % of
// the fastest on average and 14 % at worst. They rank choices and do not foretell times: fp32's w of 0.2 is less than half of
// the 0.44 us that its matrix cores take for a slab of a tile.
// fp32 products are bound by the matrix cores in every shape and always take the small one, which leaves
// the fewest of them idle. MD and SD (int8 only) are fitted to 21 int8 products, all shapes and cuts: 8 % from the fastest at worst, with
// one turn of work-groups at most. Some times, us (bf16 gated block, n x o x i): 65 x 11008 x 4096 L 87, M 46, S 39; 2048 x 11008 x 4096
// L 320, M 399, S 638; 512 x 4096 x 11008 M 122, M in two splits 93, L in four 96.
struct TilePlan {
    int shape, whole, splits, sper;
    size_t part;         // floats of split sums
};

template <int E, int MODE>
TilePlan tile_plan(int64_t M, int64_t N, int64_t K) {
    // both weight gradients' plan also where one is wanted, so that it is the same bits either way
    constexpr int pairs = MODE == TP_GRAD_W ? 2 : 1;
    constexpr int BK = 8 * el_chunk<E>();
    constexpr int size[5] = {256, 128, 64, 128, 64}, occ[5] = {1, 2, 4, 1, 2}, cuts[8] = {1, 2, 3, 4, 6, 8, 12, 16};
    constexpr double lat[5] = {1.4, 0.9, E == EL_MX ? 0.9 : 0.75, 0.45, 0.2}, fix[5] = {10.0, 4.0, 1.7, 5.5, 3.0};
    constexpr double w[5] = {1.55, 0.5, E == EL_F32 ? 0.2 : E == EL_MX ? 0.68 : 0.38, 0.45, 0.19};
    const int64_t slabs = (K + BK - 1) / BK;
    TilePlan best{};
    double least = 0.0;
    for (int h = E == EL_F32 ? 2 : 0; h < (E == EL_I8 ? 5 : 3); h++) {
        const int64_t tn = MODE == TP_GATED ? size[h] / 2 : size[h];
        const int64_t tiles = ((M + size[h] - 1) / size[h]) * ((N + tn - 1) / tn) * pairs, turn = 256 * occ[h];    // turn: even
        auto time = [&](int64_t wgs, int64_t per) {
            const int64_t percu = (wgs + 255) / 256, rounds = (percu + occ[h] - 1) / occ[h];
            const double by_lat = (double)rounds * lat[h], by_w = (double)percu * w[h];
            return (double)(per * (MODE == TP_GRAD_X ? 2 : 1)) * (by_lat > by_w ? by_lat : by_w) + (double)rounds * fix[h];
        };
        for (int tail = 0; tail < 2; tail++) {
            // all tiles cut alike, or only those behind the last full turn of the GPU's compute units
            const int64_t whole = tail ? tiles / turn * turn : 0, cut = tiles - whole;
            if (tail && (whole == 0 || cut == 0)) continue;
            for (int c = tail; c < 8; c++) {
                const int64_t sper = (slabs + cuts[c] - 1) / cuts[c], splits = (slabs + sper - 1) / sper;
                if (c && splits <= cuts[c - 1]) continue;        // another choice has these, or nearly
                if (h > 2 && tiles * splits > turn) break;       // MD and SD: one turn
                const size_t part = splits > 1 ? (size_t)(cut * splits * size[h] * size[h]) : 0;
                double t = (whole ? time(whole, slabs) : 0.0) + time(cut * splits, sper);
                if (part) t += 4.0 + 8.0 * (double)part / 3.5e6;
                if (E == EL_MX && h < 2) t += 3.0;
                if (best.splits == 0 || t < least) {
                    least = t;
                    best = TilePlan{h, (int)((splits > 1 ? whole : tiles) / pairs), (int)splits, (int)sper, part};
                }
            }
        }
    }
    return best;
}

// Work-groups of a product and of its split sums, after setting the plan's fields of g.
struct TileGrids {
    int64_t tiles, sums;
};
template <int MODE, typename C>
kq_status tile_grids(TileGrids& n, TileArgs& g, const TilePlan& p, const char* who) {
    constexpr int TN_OUT = MODE == TP_GATED ? C::TN / 2 : C::TN, PER = C::TM * TN_OUT / 1024;
    const int64_t tiles = ((g.M + C::TM - 1) / C::TM) * ((g.N + TN_OUT - 1) / TN_OUT);       // of a pair
    const int64_t cut = (tiles - p.whole) * g.pairs;
    n.tiles = (int64_t)p.whole * g.pairs + cut * p.splits;
    n.sums = cut * PER;
    if (!grid_ok(n.tiles, C::THREADS) || !grid_ok(n.sums, 256)) return fail(KQ_ESHAPE, "%s: too many tiles for a launch", who);
    g.whole = p.whole;
    g.splits = p.splits;
    g.sper = p.sper;
    return KQ_OK;
}

// The allowance for dynamic LDS belongs to a device's copy of a kernel: asked for once a device.
inline kq_status allow_lds(const void* kernel, size_t bytes, std::atomic<uint64_t>& allowed, const char* who) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return fail(KQ_EHIP, "%s: no current device", who);
    const uint64_t bit = 1ull << (dev & 63);
    if (dev > 63 || !(allowed.load(std::memory_order_relaxed) & bit)) {
        const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != hipSuccess) return fail(KQ_EHIP, "%s: %s", who, hipGetErrorString(e));
        if (dev <= 63) allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    return KQ_OK;
}

template <int E, int MODE, typename C>
kq_status tile_launch_shape(TileArgs g, const TilePlan& p, hipStream_t st, const char* who) {
    TileGrids n;
    KQ_TRY((tile_grids<MODE, C>(n, g, p, who)));
    static std::atomic<uint64_t> allowed{0};
    KQ_TRY(allow_lds(reinterpret_cast<const void*>(&tile_kernel<E, MODE, C>), C::SMEM, allowed, who));
    hipLaunchKernelGGL((tile_kernel<E, MODE, C>), dim3((unsigned)n.tiles), dim3(C::THREADS), C::SMEM, st, g);
    KQ_TRY(check_launch(who));
    if (n.sums) {
        hipLaunchKernelGGL((tile_reduce_kernel<MODE, typename C::Shallow, E == EL_I8 ? EL_I8 : EL_F32>), dim3((unsigned)n.sums), dim3(256), 0, st, g);
        KQ_TRY(check_launch(who));
    }
    return KQ_OK;
}

// Both gradient products in one launch where both are cut into S tiles.
inline bool grads_together(const TilePlan& x, const TilePlan& w) { return x.shape == 2 && w.shape == 2; }
template <int E>
kq_status tile_launch_grads(TileArgs x, const TilePlan& px, TileArgs w, const TilePlan& pw, hipStream_t st, const char* who) {
    typedef TileS C;
    TileGrids nx, nw;
    KQ_TRY((tile_grids<TP_GRAD_X, C>(nx, x, px, who)));
    KQ_TRY((tile_grids<TP_GRAD_W, C>(nw, w, pw, who)));
    if (!grid_ok(nx.tiles + nw.tiles, C::THREADS) || !grid_ok(nx.sums + nw.sums, 256))
        return fail(KQ_ESHAPE, "%s: too many tiles for a launch", who);
    hipLaunchKernelGGL((tile_grads_kernel<E, C>), dim3((unsigned)(nx.tiles + nw.tiles)), dim3(C::THREADS), C::SMEM, st, x, w,
                       (int)nx.tiles);
    KQ_TRY(check_launch(who));
    if (nx.sums + nw.sums) {
        hipLaunchKernelGGL((tile_reduce_grads_kernel<C>), dim3((unsigned)(nx.sums + nw.sums)), dim3(256), 0, st, x, w, (int)nx.sums);
        KQ_TRY(check_launch(who));
    }
    return KQ_OK;
}

// p: tile_plan<E, MODE>(M, N, K); part: workspace of p.part floats
template <int E, int MODE>
kq_status tile_launch(TileArgs g, const TilePlan& p, int pairs, float* part, hipStream_t st, const char* who) {
    g.pairs = pairs;
    g.part = part;
    if (p.part && !part) return fail(KQ_EWORKSPACE, "%s: workspace too small", who);
    if constexpr (E != EL_F32) {
        if (p.shape == 0) return tile_launch_shape<E, MODE, TileL>(g, p, st, who);
        if (p.shape == 1) return tile_launch_shape<E, MODE, TileM>(g, p, st, who);
    }
    if constexpr (E == EL_I8) {
        if (p.shape == 3) return tile_launch_shape<E, MODE, TileMD>(g, p, st, who);
        if (p.shape == 4) return tile_launch_shape<E, MODE, TileSD>(g, p, st, who);
    }
    return tile_launch_shape<E, MODE, TileS>(g, p, st, who);
}

// ------------------------------------------------------------------------------------- few tokens
// Y (or the gated block) for the few tokens of few_tokens: the weights are read once, straight into registers,
// and that stream is what bounds the call. A work-group owns 16 rows of B (and of B2); its 8 wavefronts take
// the 128-byte slabs of K in turn and their sums meet in LDS, in wavefront order. The rows of A (tokens)
// are few and come from L2. All work-groups of the usual widths are resident at once, and a wavefront has all its loads
// of one or two slabs in flight, so what is left above the stream is one launch and one latency. MI355X, the kernel
// alone, on weights that the last-level cache holds from call to call and (second) on weights rotated past it: 4096 x 11008
// E2M1, one token 6.0 and 8.5 us (4.0 and 2.8 TB/s); gated 11008 x 4096 E2M1, four tokens 13.0 and 15.7 us (3.7
// and 3.1 TB/s); gated bf16, one token 31.4 and 38.1 us (5.7 and 4.7 TB/s, the latter the rate of a copy of 4 GiB). From 9
// tokens on the rows of A cost as well: every work-group reads all of them for its 16 rows of B, at 32 tokens twice the
// bytes of its weights, from L2 (4096 x 11008 E2M1: 7.8 us at 16 tokens, 10.7 at 32).
struct FewArgs {
    int64_t n, o, K;                      // tokens, rows of B, values of K
    const char *A, *B, *B2;
    int64_t lda, ldb, ldb2;               // bytes
    const uint8_t *sA, *sB, *sB2;         // E2M1: E8M0 bytes, rows of lds* bytes
    int64_t ldsa, ldsb, ldsb2;
    void *Y, *Y2, *Y3;
    int64_t ldy, ldy2, ldy3;
    int dt, act;
    const float *fA, *fB, *fB2;           // int8: the scales of the rows
};

constexpr int FEW_WAVES = 8, FEW_THREADS = 64 * FEW_WAVES;

// Whether n tokens run here rather than as tiles. Measured on MI355X, us here / as tiles, o x i weights:
//   E2M1  11008 x 4096: 8.3 / 11.2 at 1 token, 15.4 / 16.1 at 32, 22.2 / 16.1 at 33; 4096 x 11008: 11.8 / 14.8
//         at 32, 14.6 / 14.3 at 33
//   int8  weights from HBM; 4096 x 11008: 11.2 / 14.1 at 1, 13.0 / 14.7 at 16, 20.6 / 15.0 at 24; 16384 x 4096: 15.7 / 17.2 at 8, 19.4 / 17.5
//         at 16; 4096 x 4096: 10.1 / 11.8 at 32; gated (o is then 2 x 11008) 11008 x 4096: 20.5 / 23.2 at 1, 24.1 / 21.8 at 16; gated 1376 x
//         4096: 11.5 / 11.8 at 32; gated 5504 x 8192 is better as tiles from one token on, 23.7 / 21.8
//   bf16  gated 11008 x 4096: 34.1 / 34.7 at 8, 36.2 / 34.4 at 16; 1376 x 1000: 6.7 / 9.2 at 48
//   fp32  gated 11008 x 4096: 104 / 135 at 32, 173 / 134 at 33; 1376 x 1000: 10.0 / 15.4 at 32, 16.6 / 15.6 at 33
template <int E>
bool few_tokens(int64_t n, int64_t o, int64_t i) {
    if (E == EL_I8) return n <= 8 || (n <= 16 && o <= 8192) || (n <= 32 && o * i <= (1 << 24));
    if (E != EL_BF16) return n <= 32;
    return n <= 8 || (n <= 48 && o * i <= (1 << 22));
}

template <int E>
struct FewFrag {
    tl_i4 c[2];       // chunks g4 and 4 + g4 of a slab
    uint32_t s[2];    // E2M1: the scale bytes of the two
};

// Chunks of one row's slab s. `whole`: all eight chunks are full.
template <int E>
__device__ __forceinline__ void few_load(FewFrag<E>& f, const char* row, const uint8_t* srow, int64_t s, int g4,
                                         bool whole, int64_t nch, int part) {
    const char* p = row + s * 128 + g4 * 16;
    if (whole) {
        f.c[0] = *reinterpret_cast<const tl_i4*>(p);
        f.c[1] = *reinterpret_cast<const tl_i4*>(p + 64);
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int64_t c = s * 8 + 4 * h + g4;
            tl_i4 v = {0, 0, 0, 0};
            if (c < nch) v = *reinterpret_cast<const tl_i4*>(p + 64 * h);
            if (E != EL_MX && part && c == nch - 1) v = chunk_head<E>(v, part);
            f.c[h] = v;
        }
    }
    if constexpr (E == EL_MX) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(srow + s * 8);
        if (whole) {
            f.s[0] = q[0] >> (8 * g4);
            f.s[1] = q[1] >> (8 * g4);
        } else {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t b = s * 8 + 4 * h;     // scale rows are read four bytes at a time
                const uint32_t w = b < nch ? q[h] : 0u;
                f.s[h] = b + g4 < nch ? w >> (8 * g4) : 0u;
            }
        }
    }
}

// rows 16 block .. of B, the first 16 NB rows of A. SPREAD: where rows begin at multiples of 128 bytes, a wavefront takes neighbouring slabs of
// K, from a place that differs from block to block. In turns, all work-groups walk along K together and their reads meet in the same memory
// channels, most of all where rows lie a multiple of 4 KiB apart. MI355X, us in turns / spread, weights from HBM: int8, one token 4096 x 11008 13.3 / 11.2, 16384 x 4096 16.2 /
// 14.0; 8 rows of 8 experts 4096 x 11008 bf16 89 / 78, int8 50 / 40. Other rows' slabs share a cache line with the next wavefront's (16 rows of
// 8 experts gated 2000 x 2000 bf16 18.7 / 21.4), and from two blocks of tokens on it costs more reads of A (24 tokens gated 1376 x 4096 int8
// 10.8 / 12.3). Not for the other products of one matrix, which keep the order of their sums; int8's are exact in any.
template <int E, bool GATED, int NB, bool SPREAD>
__device__ __forceinline__ void few_body(const FewArgs& g, int64_t block) {
    extern __shared__ __align__(16) float few_sm[];       // [wave][matrix][token block][lane][4]
    constexpr int EPC = el_chunk<E>(), MATS = GATED ? 2 : 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int x16 = lane & 15, g4 = lane >> 4;
    const int64_t f0 = block * 16;
    const int64_t row = f0 + x16 < g.o ? f0 + x16 : g.o - 1;
    const char* rB = g.B + row * g.ldb;
    const char* rB2 = GATED ? g.B2 + row * g.ldb2 : nullptr;
    const uint8_t* qB = E == EL_MX ? g.sB + row * g.ldsb : nullptr;
    const uint8_t* qB2 = E == EL_MX && GATED ? g.sB2 + row * g.ldsb2 : nullptr;
    const char* rA[NB];
    const uint8_t* qA[NB];
#pragma unroll
    for (int b = 0; b < NB; b++) {
        const int64_t t = 16 * b + x16 < g.n ? 16 * b + x16 : g.n - 1;
        rA[b] = g.A + t * g.lda;
        qA[b] = E == EL_MX ? g.sA + t * g.ldsa : nullptr;
    }
    const int64_t nch = (g.K + EPC - 1) / EPC, slabs = (nch + 7) / 8;
    const int part = (int)(g.K % EPC);
    const int64_t full = E == EL_MX ? nch / 8 : g.K / (8 * EPC);      // slabs whose chunks are all whole

    typedef el_sums<E> Sums;
    Sums acc[MATS][NB];
#pragma unroll
    for (int m = 0; m < MATS; m++)
#pragma unroll
        for (int b = 0; b < NB; b++) acc[m][b] = Sums{0, 0, 0, 0};
    // U slabs at a time: all their loads are in flight before the first product (dense types with two are slower)
    auto batch = [&](int64_t s, auto UC, bool whole) {
        constexpr int U = UC.value;
        FewFrag<E> w[U][MATS], a[U][NB];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t su = s + u * FEW_WAVES;
            few_load<E>(w[u][0], rB, qB, su, g4, whole, nch, part);
            if constexpr (GATED) few_load<E>(w[u][1], rB2, qB2, su, g4, whole, nch, part);
#pragma unroll
            for (int b = 0; b < NB; b++) few_load<E>(a[u][b], rA[b], qA[b], su, g4, whole, nch, part);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int m = 0; m < MATS; m++)
#pragma unroll
                    for (int b = 0; b < NB; b++)
                        acc[m][b] = mma_step<E>(w[u][m].c[h], a[u][b].c[h], acc[m][b], (int)w[u][m].s[h], 0, (int)a[u][b].s[h], 0);
    };
    constexpr int U = E == EL_MX && NB < 4 ? 2 : 1;
    int64_t s = wave;
    if constexpr (SPREAD && NB == 1) {
        static_assert(U == 1, "one slab at a time");
        if (g.ldb % 128 == 0) {
            const int64_t first = full * wave / FEW_WAVES, last = full * (wave + 1) / FEW_WAVES;
            const int64_t from = last > first ? first + (unsigned)block % (unsigned)(last - first) : first;
            for (int64_t t = from; t < last; t++) batch(t, std::integral_constant<int, 1>{}, true);
            for (int64_t t = first; t < from; t++) batch(t, std::integral_constant<int, 1>{}, true);
            s = full;
        }
    }
    for (; s + (U - 1) * FEW_WAVES < full; s += U * FEW_WAVES) batch(s, std::integral_constant<int, U>{}, true);
    if (U > 1 && s < full) batch(s, std::integral_constant<int, 1>{}, true);
    if (full < slabs && wave == (int)(full % FEW_WAVES)) batch(full, std::integral_constant<int, 1>{}, false);

#pragma unroll
    for (int m = 0; m < MATS; m++)
#pragma unroll
        for (int b = 0; b < NB; b++)
            reinterpret_cast<Sums*>(few_sm)[((wave * MATS + m) * NB + b) * 64 + lane] = acc[m][b];
    __syncthreads();
    if (wave >= NB) return;
    // wavefront b finishes token block b: lane holds token x16 and rows f0 + 4 g4 .. + 3
    Sums sum[MATS];
#pragma unroll
    for (int m = 0; m < MATS; m++) {
        sum[m] = Sums{0, 0, 0, 0};
        for (int w = 0; w < FEW_WAVES; w++) {
            const Sums v = reinterpret_cast<const Sums*>(few_sm)[((w * MATS + m) * NB + wave) * 64 + lane];
#pragma unroll
            for (int r = 0; r < 4; r++) sum[m][r] += v[r];
        }
    }
    const int64_t t = 16 * wave + x16, n = f0 + 4 * g4;
    if (t >= g.n) return;
    float v[MATS][4];
#pragma unroll
    for (int m = 0; m < MATS; m++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            if constexpr (E == EL_I8) v[m][r] = (float)sum[m][r] * (g.fA[t] * (m ? g.fB2 : g.fB)[n + r < g.o ? n + r : g.o - 1]);
            else v[m][r] = sum[m][r];
        }
    if constexpr (GATED) {
        float y[4];
        act_times(y, v[0], v[1], g.act);
        store_run<4>(g.Y, g.dt, t * g.ldy + n, y, g.o - n);
        if (g.Y2) store_run<4>(g.Y2, g.dt, t * g.ldy2 + n, v[0], g.o - n);
        if (g.Y3) store_run<4>(g.Y3, g.dt, t * g.ldy3 + n, v[1], g.o - n);
    } else {
        store_run<4>(g.Y, g.dt, t * g.ldy + n, v[0], g.o - n);
    }
}

template <int E, bool GATED, int NB>
__global__ __launch_bounds__(FEW_THREADS) void few_kernel(FewArgs g) {
    few_body<E, GATED, NB, E == EL_I8>(g, (int64_t)blockIdx.x);
}

template <int E, bool GATED>
kq_status few_launch(const FewArgs& g, hipStream_t st, const char* who) {
    const int64_t wgs = (g.o + 15) / 16;
    if (!grid_ok(wgs, FEW_THREADS)) return fail(KQ_ESHAPE, "%s: too many rows", who);
    const dim3 grid((unsigned)wgs);
    const size_t one = (size_t)FEW_WAVES * (GATED ? 2 : 1) * 1024;
    if (g.n <= 16) {
        hipLaunchKernelGGL((few_kernel<E, GATED, 1>), grid, dim3(FEW_THREADS), one, st, g);
    } else if (g.n <= 32) {
        hipLaunchKernelGGL((few_kernel<E, GATED, 2>), grid, dim3(FEW_THREADS), 2 * one, st, g);
    } else if constexpr (E == EL_BF16) {                 // the others have 32 tokens at most
        hipLaunchKernelGGL((few_kernel<E, GATED, 4>), grid, dim3(FEW_THREADS), 4 * one, st, g);
    }
    return check_launch(who);
}

}  // namespace kq
