// Microscaled 4-bit floating point (KronQ review page, Limitations (3): the stored weights are multiplied at
// inference time; OCP Microscaling Formats, MXFP4): blocks of 32 consecutive columns of a row share one
// power-of-two scale 2^(s - 127) (an E8M0 byte s; 255 stands for NaN), and every element is one of
// 0, 1/2, 1, 3/2, 2, 3, 4, 6 with a sign (E2M1), two a byte.
//
// Quantisation of a block with largest magnitude a: s - 127 = floor(log2 a) - 2 (2 is the exponent of the
// largest element, 6 = 1.5 * 2^2), not below -127; elements are x / 2^(s - 127) rounded to the nearest
// value, ties to the even code, and magnitudes past 6 (a / scale lies in [4, 8)) become 6. An all-zero
// block has s = 0. A block that holds an infinity or NaN gets s = 255 and zero codes, so that it reads as
// NaN instead of as some finite value. Division by the scale is exact, so the codes are the exact result.
#include "tile.h"

namespace kq {

// ----------------------------------------------------------------------------------- quantisation
// One lane takes 8 consecutive columns (a quarter block): the four lanes of a block exchange their largest
// magnitude as bit patterns (which order like the magnitudes, infinities and NaN last) and each
// converts its 8 values with the packed conversion instructions into one dword of codes. The pass is bound
// by HBM: each input value is read once and 17 bytes a block are written. MI355X: 8192 x 4096 bf16 15.4 us, 5.5
// TB/s (85 MB in all, less than the last-level cache holds); 5120 x 13824 fp32 75 us, 4.3 TB/s, where a copy of 4 GiB runs at 4.7.
template <bool BF>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                          int64_t ldx, uint8_t* __restrict__ codes, int64_t ldc,
                                                          uint8_t* __restrict__ scales, int64_t lds, int64_t nblk) {
    const int64_t per = nblk * 4, total = rows * per;
    const int64_t step = (int64_t)gridDim.x * 256;       // a multiple of 4: a block's lanes stay together
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += step) {
        const int64_t r = e / per, q = e - r * per, c = q * 8;
        float v[8];
        if constexpr (BF) {
            const uint16_t* p = static_cast<const uint16_t*>(X) + r * ldx + c;
            if (c + 8 <= cols) {
                const uint4 w = *reinterpret_cast<const uint4*>(p);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    v[2 * k] = __uint_as_float(u[k] << 16);
                    v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; k++) v[k] = c + k < cols ? from_bf16(p[k]) : 0.0f;
            }
        } else {
            const float* p = static_cast<const float*>(X) + r * ldx + c;
            if (c + 8 <= cols) {
                const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
                v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
            } else {
#pragma unroll
                for (int k = 0; k < 8; k++) v[k] = c + k < cols ? p[k] : 0.0f;
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const uint32_t b = __float_as_uint(v[k]) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
        // lanes 4 b .. 4 b + 3 hold block b
        uint32_t o = __builtin_amdgcn_update_dpp(0, top, 0xB1, 0xF, 0xF, false);   // lane ^ 1
        top = o > top ? o : top;
        o = __builtin_amdgcn_update_dpp(0, top, 0x4E, 0xF, 0xF, false);            // lane ^ 2
        top = o > top ? o : top;
        const bool bad = top >= 0x7F800000u;
        const int ex = (int)(top >> 23);                 // biased exponent; 0 and 1 clamp to the smallest scale
        const int s = bad ? 255 : ex > 2 ? ex - 2 : 0;
        const float sc = __uint_as_float(s ? (uint32_t)s << 23 : 0x00400000u);     // 2^(s - 127)
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
        *reinterpret_cast<uint32_t*>(codes + r * ldc + q * 4) = bad ? 0u : w;
        if ((q & 3) == 0) scales[r * lds + (q >> 2)] = (uint8_t)s;
    }
}

// One lane expands 8 codes (bf16) or 4 (fp32), 16 bytes of output, so that a wavefront's store is one run of
// 1 KiB; the pass is bound by HBM writes (MI355X: 8192 x 4096 bf16 16 us, 5.3 TB/s; 5120 x 13824 fp32 72 us, 4.5
// TB/s, and 81 us with 8 codes a lane, whose two 16-byte stores are 32 bytes apart from lane to lane). The products with the scale are exact (two significant bits), so both
// types hold them exactly unless they leave the type's range.
template <bool BF>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ldc,
                                                            const uint8_t* __restrict__ scales, int64_t lds,
                                                            int64_t rows, int64_t cols, void* __restrict__ Y, int64_t ldy) {
    constexpr int V = BF ? 8 : 4;
    typedef float f2 __attribute__((ext_vector_type(2)));
    const int64_t per = (cols + V - 1) / V, total = rows * per;
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += step) {
        const int64_t r = e / per, q = e - r * per, c = q * V;
        const uint8_t* p = codes + r * ldc + q * (V / 2);
        const uint32_t w = BF ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
        const uint32_t s = scales[r * lds + c / 32];
        const float sc = s == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(s ? s << 23 : 0x00400000u);
        float v[V];
        const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
        v[0] = a[0] * sc; v[1] = a[1] * sc; v[2] = b[0] * sc; v[3] = b[1] * sc;
        if constexpr (BF) {
            const f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
            v[4] = d[0] * sc; v[5] = d[1] * sc; v[6] = f[0] * sc; v[7] = f[1] * sc;
        }
        store_run<V>(Y, BF ? KQ_BF16 : KQ_F32, r * ldy + c, v, cols - c);
    }
}

// -------------------------------------------------------------------------- scales for large tiles
// A lane of the two larger tile shapes (x16, g4) needs, for step k of 128 columns and each of its fragments, the scale byte
// of one row's block 4 k + g4. This pass gathers them so that one coalesced dword a lane holds four
// fragments' bytes: out[(group * ksteps + k) * 64 + lane], group = 64 rows. Blocks past the last column get
// byte 0 (2^-127), on both operands: the product of two such blocks is below the smallest fp32, zero.
//   KIND 0  A: fragment f holds rows 64 group + 16 f + x16
//   KIND 1  B: rows 64 group + b_row<4>(f, x16)
//   KIND 2  gated: fragments 0, 1 are gate rows 32 group + b_row<2>(f, x16), 2 and 3 up rows
struct MxBytes16 {       // scale rows are aligned to 4 bytes
    uint32_t w[4];
};
struct MxLayout {
    const uint8_t *s, *s2;
    int64_t lds, lds2, rows, groups;
    uint32_t* out;
};

// A lane reads 16 bytes (four steps) of each of its four rows and stores four dwords. Some 5 MB for 8192 tokens: its
// 5 to 7 us are latency, 2 to 4 % of the product behind it.
template <int KIND>
__device__ __forceinline__ void mx_layout_group(const MxLayout& L, int64_t group, int nblk, int ksteps) {
    const int lane = threadIdx.x & 63, x16 = lane & 15, g4 = lane >> 4;
    const uint8_t* row[4];
    uint32_t keep[4];
#pragma unroll
    for (int f = 0; f < 4; f++) {
        const int64_t r = KIND == 0 ? 64 * group + 16 * f + x16
                        : KIND == 1 ? 64 * group + b_row<4>(f, x16) : 32 * group + b_row<2>(f & 1, x16);
        const bool in = r < L.rows;
        keep[f] = in ? 0xFFu : 0u;
        row[f] = KIND == 2 && f >= 2 ? L.s2 + (in ? r : 0) * L.lds2 : L.s + (in ? r : 0) * L.lds;
    }
    for (int k = (threadIdx.x >> 6) * 4; k < ksteps; k += 16) {
        uint32_t v[4][4];                        // [row][step]
#pragma unroll
        for (int f = 0; f < 4; f++) {
            if (16 + 4 * k <= nblk) {
                const MxBytes16 t = *reinterpret_cast<const MxBytes16*>(row[f] + 4 * k);
#pragma unroll
                for (int e = 0; e < 4; e++) v[f][e] = t.w[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++) v[f][e] = 4 * (k + e) < nblk ? *reinterpret_cast<const uint32_t*>(row[f] + 4 * (k + e)) : 0u;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            uint32_t w = 0;
#pragma unroll
            for (int f = 0; f < 4; f++) w |= ((v[f][e] >> (8 * g4)) & keep[f]) << (8 * f);
            if (4 * (k + e) + g4 >= nblk) w = 0;
            if (k + e < ksteps) L.out[(group * ksteps + k + e) * 64 + lane] = w;
        }
    }
}

// one work-group of 4 wavefronts a group of 64 rows, A's groups first
template <bool GATED>
__global__ __launch_bounds__(256) void mx_layout_kernel(MxLayout a, MxLayout b, int nblk, int ksteps) {
    const int64_t group = blockIdx.x;
    if (group < a.groups) mx_layout_group<0>(a, group, nblk, ksteps);
    else mx_layout_group<GATED ? 2 : 1>(b, group - a.groups, nblk, ksteps);
}

// 64-row groups of the laid-out scales: whole tiles, so that every wavefront of the last one reads inside
static int64_t mx_groups_a(int64_t n) { return (n + TL_ROWS - 1) / TL_ROWS * (TL_ROWS / 64); }
static int64_t mx_groups_b(int64_t o, bool gated) { return mx_groups_a(gated ? 2 * o : o); }
static int64_t mx_ksteps(int64_t i) { return (i + 255) / 256 * 2; }

static TilePlan mx_plan(int64_t n, int64_t o, int64_t i, bool gated) {
    return gated ? tile_plan<EL_MX, TP_GATED>(n, o, i) : tile_plan<EL_MX, TP_PLAIN>(n, o, i);
}

struct MxOperand {
    const uint8_t* c;
    int64_t ldc;
    const uint8_t* s;
    int64_t lds;
};

static kq_status mx_check(const char* who, const char* what, const MxOperand& m, int64_t rows, int64_t cols) {
    const int64_t nblk = (cols + 31) / 32;
    if (!m.c || !m.s) return fail(KQ_EINVAL, "%s: null %s", who, what);
    if (m.ldc < 16 * nblk || m.lds < nblk) return fail(KQ_ESHAPE, "%s: leading dimension of %s too small", who, what);
    if (!aligned16(m.c) || m.ldc % 16 || reinterpret_cast<uintptr_t>(m.s) % 4 || m.lds % 4)
        return fail(KQ_EINVAL, "%s: %s codes must be aligned to 16 bytes and scales to 4, rows likewise", who, what);
    if (m.ldc > TL_LD_MAX || m.lds > TL_LD_MAX || rows > TL_ROWS_MAX) return fail(KQ_ESHAPE, "%s: %s too large", who, what);
    return KQ_OK;
}

static kq_status mx_out_check(const char* who, const void* Y, kq_dtype dt, int64_t ldy, int64_t cols) {
    if (!Y) return fail(KQ_EINVAL, "%s: null output", who);
    if (dt != KQ_F32 && dt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (ldy < cols) return fail(KQ_ESHAPE, "%s: leading dimension of the output too small", who);
    if (!aligned16(Y) || ldy % (dt == KQ_BF16 ? 8 : 4)) return fail(KQ_EINVAL, "%s: output rows must be 16-byte aligned", who);
    return KQ_OK;
}

// Y = A B^T, or the gated block when U is given
static kq_status mx_product(const char* who, const MxOperand& A, const MxOperand& B, const MxOperand* U, int64_t n,
                            int64_t o, int64_t i, int act, void* Y, kq_dtype dt, int64_t ldy, void* ws, size_t ws_bytes,
                            hipStream_t st) {
    if (!tile_sizes_ok(n, o)) return fail(KQ_ESHAPE, "%s: result too large", who);
    if (few_tokens<EL_MX>(n, o, i)) {
        FewArgs f{};
        f.n = n; f.o = o; f.K = i;
        f.A = reinterpret_cast<const char*>(A.c); f.lda = A.ldc; f.sA = A.s; f.ldsa = A.lds;
        f.B = reinterpret_cast<const char*>(B.c); f.ldb = B.ldc; f.sB = B.s; f.ldsb = B.lds;
        if (U) { f.B2 = reinterpret_cast<const char*>(U->c); f.ldb2 = U->ldc; f.sB2 = U->s; f.ldsb2 = U->lds; }
        f.Y = Y; f.ldy = ldy; f.dt = dt; f.act = act;
        return U ? few_launch<EL_MX, true>(f, st, who) : few_launch<EL_MX, false>(f, st, who);
    }
    const TilePlan plan = mx_plan(n, o, i, U != nullptr);
    Arena ar(ws, ws_bytes);
    TileArgs g{};
    g.M = n; g.N = o; g.K = i;
    g.A = reinterpret_cast<const char*>(A.c); g.lda = A.ldc;
    g.B = reinterpret_cast<const char*>(B.c); g.ldb = B.ldc;
    g.rA = A.s; g.ldrA = A.lds; g.rB = B.s; g.ldrB = B.lds;
    if (U) {
        g.B2 = reinterpret_cast<const char*>(U->c); g.ldb2 = U->ldc;
        g.rB2 = U->s; g.ldrB2 = U->lds;
    }
    g.Y = Y; g.ldy = ldy; g.dt = dt; g.act = act;
    g.ksteps = mx_ksteps(i);
    const int64_t ga = mx_groups_a(n), gb = mx_groups_b(o, U != nullptr);
    if (plan.shape < 2 && !grid_ok(ga + gb, 256)) return fail(KQ_ESHAPE, "%s: too many rows for a launch", who);
    uint32_t* la = plan.shape < 2 ? ar.take<uint32_t>((size_t)(ga * g.ksteps * 64)) : nullptr;
    uint32_t* lb = plan.shape < 2 ? ar.take<uint32_t>((size_t)(gb * g.ksteps * 64)) : nullptr;
    float* part = plan.part ? ar.take<float>(plan.part) : nullptr;
    if ((plan.shape < 2 || plan.part) && (!ws || !aligned16(ws) || !ar.ok()))
        return fail(KQ_EWORKSPACE, "%s: workspace too small or not aligned to 16 bytes", who);
    if (plan.shape < 2) {
        g.sA = la;
        g.sB = lb;
        const MxLayout a{A.s, nullptr, A.lds, 0, n, ga, la};
        const MxLayout b{B.s, U ? U->s : nullptr, B.lds, U ? U->lds : 0, o, gb, lb};
        const dim3 grid((unsigned)(ga + gb));
        const int nblk = (int)((i + 31) / 32);
        if (U) hipLaunchKernelGGL((mx_layout_kernel<true>), grid, dim3(256), 0, st, a, b, nblk, (int)g.ksteps);
        else hipLaunchKernelGGL((mx_layout_kernel<false>), grid, dim3(256), 0, st, a, b, nblk, (int)g.ksteps);
        KQ_TRY(check_launch(who));
    }
    return U ? tile_launch<EL_MX, TP_GATED>(g, plan, 1, part, st, who) : tile_launch<EL_MX, TP_PLAIN>(g, plan, 1, part, st, who);
}

}  // namespace kq

using namespace kq;

size_t mx_product_ws(int64_t o, int64_t i, int64_t n, bool gated) {
    if (n <= 0 || o <= 0 || i <= 0 || !tile_sizes_ok(n, o) || few_tokens<EL_MX>(n, o, i)) return 0;
    const TilePlan plan = mx_plan(n, o, i, gated);
    Sizer s;
    if (plan.shape < 2) {
        s.take<uint32_t>((size_t)(mx_groups_a(n) * mx_ksteps(i) * 64));
        s.take<uint32_t>((size_t)(mx_groups_b(o, gated) * mx_ksteps(i) * 64));
    }
    if (plan.part) s.take<float>(plan.part);
    return s.used;
}

extern "C" kq_status kq_mx_quantize(const void* X, kq_dtype xdt, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes,
                                    int64_t ldc, uint8_t* scales, int64_t lds, kq_stream stream) {
    const char* who = "kq_mx_quantize";
    if (rows < 0 || cols <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (xdt != KQ_F32 && xdt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (rows == 0) return KQ_OK;
    if (!X) return fail(KQ_EINVAL, "%s: null X", who);
    if (ldx < cols) return fail(KQ_ESHAPE, "%s: ldx < cols", who);
    if (!aligned16(X) || ldx % (xdt == KQ_BF16 ? 8 : 4))
        return fail(KQ_EINVAL, "%s: X must be 16-byte aligned with ldx a multiple of 16 bytes", who);
    KQ_TRY(mx_check(who, "output", MxOperand{codes, ldc, scales, lds}, rows, cols));
    const int64_t nblk = (cols + 31) / 32, total = rows * nblk * 4;
    const unsigned grid = (unsigned)((total + 255) / 256 < 65536 ? (total + 255) / 256 : 65536);
    if (xdt == KQ_BF16)
        hipLaunchKernelGGL((mx_quantize_kernel<true>), dim3(grid), dim3(256), 0, hs(stream), X, rows, cols, ldx, codes, ldc,
                           scales, lds, nblk);
    else
        hipLaunchKernelGGL((mx_quantize_kernel<false>), dim3(grid), dim3(256), 0, hs(stream), X, rows, cols, ldx, codes,
                           ldc, scales, lds, nblk);
    return check_launch(who);
}

extern "C" kq_status kq_mx_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows,
                                      int64_t cols, void* Y, kq_dtype ydt, int64_t ldy, kq_stream stream) {
    const char* who = "kq_mx_dequantize";
    if (rows < 0 || cols <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (ydt != KQ_F32 && ydt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (rows == 0) return KQ_OK;
    KQ_TRY(mx_check(who, "input", MxOperand{codes, ldc, scales, lds}, rows, cols));
    KQ_TRY(mx_out_check(who, Y, ydt, ldy, cols));
    const int64_t v = ydt == KQ_BF16 ? 8 : 4, total = rows * ((cols + v - 1) / v);
    const unsigned grid = (unsigned)((total + 255) / 256 < 65536 ? (total + 255) / 256 : 65536);
    if (ydt == KQ_BF16)
        hipLaunchKernelGGL((mx_dequantize_kernel<true>), dim3(grid), dim3(256), 0, hs(stream), codes, ldc, scales, lds,
                           rows, cols, Y, ldy);
    else
        hipLaunchKernelGGL((mx_dequantize_kernel<false>), dim3(grid), dim3(256), 0, hs(stream), codes, ldc, scales, lds,
                           rows, cols, Y, ldy);
    return check_launch(who);
}

extern "C" kq_status kq_mx_gemm(const uint8_t* Ac, int64_t ldac, const uint8_t* As, int64_t ldas, const uint8_t* Bc,
                                int64_t ldbc, const uint8_t* Bs, int64_t ldbs, int64_t n, int64_t o, int64_t i, void* Y,
                                kq_dtype ydt, int64_t ldy, void* ws, size_t ws_bytes, kq_stream stream) {
    const char* who = "kq_mx_gemm";
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (ydt != KQ_F32 && ydt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (n == 0) return KQ_OK;
    const MxOperand A{Ac, ldac, As, ldas}, B{Bc, ldbc, Bs, ldbs};
    KQ_TRY(mx_check(who, "A", A, n, i));
    KQ_TRY(mx_check(who, "B", B, o, i));
    KQ_TRY(mx_out_check(who, Y, ydt, ldy, o));
    return mx_product(who, A, B, nullptr, n, o, i, 0, Y, ydt, ldy, ws, ws_bytes, hs(stream));
}

extern "C" kq_status kq_mx_gated(const uint8_t* Xc, int64_t ldxc, const uint8_t* Xs, int64_t ldxs, const uint8_t* Gc,
                                 int64_t ldgc, const uint8_t* Gs, int64_t ldgs, const uint8_t* Uc, int64_t lduc,
                                 const uint8_t* Us, int64_t ldus, int64_t n, int64_t o, int64_t i, kq_act act, void* H,
                                 kq_dtype hdt, int64_t ldh, void* ws, size_t ws_bytes, kq_stream stream) {
    const char* who = "kq_mx_gated";
    if (n < 0 || o <= 0 || i <= 0) return fail(KQ_ESHAPE, "%s: bad sizes", who);
    if (hdt != KQ_F32 && hdt != KQ_BF16) return fail(KQ_EINVAL, "%s: bad dtype", who);
    if (act < KQ_ACT_SILU || act > KQ_ACT_RELU) return fail(KQ_EINVAL, "%s: bad activation", who);
    if (n == 0) return KQ_OK;
    const MxOperand X{Xc, ldxc, Xs, ldxs}, G{Gc, ldgc, Gs, ldgs}, U{Uc, lduc, Us, ldus};
    KQ_TRY(mx_check(who, "X", X, n, i));
    KQ_TRY(mx_check(who, "gate weights", G, o, i));
    KQ_TRY(mx_check(who, "up weights", U, o, i));
    KQ_TRY(mx_out_check(who, H, hdt, ldh, o));
    return mx_product(who, X, G, &U, n, o, i, act, H, hdt, ldh, ws, ws_bytes, hs(stream));
}
