// bsp_mxgemm.hip -- grouped expert products of operands in MX formats (32
// values share one power-of-two scale): MXFP4 x MXFP4, MXFP8 x MXFP4 and, for
// the gated block, MXFP8 x MXFP8; and the gated feed-forward block on them.
//
// MXFP4 x MXFP4: gfx950's block-scaled matrix instruction
// V_MFMA_SCALE_F32_32X32X64_F8F6F4 takes codes and E8M0 scales as they are
// stored.  Lane l supplies row l % 32 of its operand, the 32 values of K block
// l / 32 (16 bytes) and that block's scale.  Its sums of MXFP4 products carry
// f32's own rounding alone.
// MXFP8 tokens: that instruction would drop what lies far below its largest
// product (64 values with blocks 2^5 apart: up to 1e-4 of sum |a b|), so their
// products are V_MFMA_F32_32X32X16_BF16's, on values times scales, which bf16
// holds exactly (to_bf16): a row's sums are the same to f32's rounding whatever
// form its batch takes.  At a quarter of the MXFP4 rate, near what the card's
// power sustains in bf16 (8192^3 by the library 1203 TFLOP/s), they bound large
// calls: the gated block of 8192 tokens takes 468 us, 297 by the scaled
// instruction.  The lanes hold the same 32-value block of both operands here too
// and multiply it eight values at a time.
//
// The weights are the instruction's first operand and the tokens the second,
// so a lane ends with one token and 16 of 32 consecutive columns of C (lane
// l: columns 8 q + 4 (l / 32) + 0..3, q = 0..3; two exchanges with lane l ^ 32
// make them 16 neighbours).  Whatever follows the product then stays in
// registers: rounding and whole stores of C, or silu(gate) * up, the maximum
// of a block of 32 and its codes.
#include "bsp_dma.hpp"
#include "bsp_moe.hpp"

namespace bsp {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int i32v4 __attribute__((ext_vector_type(4)));

enum { EPI_BF16 = 0, EPI_F32 = 1, EPI_GATED = 2, EPI_GATED_BWD = 3 };

struct MxArgs {
    const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;
    const int32_t *gather;
    const int64_t *off;
    int32_t G, M, N, K, a_rows;   // rows of C, rows of B per group (gated: 2 I), reduction length
    // C
    void *c;
    int64_t ldc;
    // gated block
    const float *row_weights;
    uint16_t *h;
    uint8_t *h_codes, *h_scales, *ckpt_codes, *ckpt_scales;
    int32_t h_fmt, I;
    uint16_t *dh13;
    float *part;                  // [M][parts]: sums of dh * act * up over 64 columns
    int32_t parts;
    // tiled form: tables and scale planes in the workspace (k_mx_prep)
    i32v4 *tiles;                 // row-grouped: per row tile its group, the group's rows and first tile (find_tile);
                                  // weight gradient: [8][G] per XCD the group, its columns [x, y) and first stage
    int32_t *count;               // listed row tiles (weight gradient: [8] groups of the XCDs)
    uint8_t *a_plane, *b_plane;
    int32_t ntm, ntn, stages;     // row tiles (bound; weight gradient: of M), column tiles, stages of K
};

template <int V>
struct IC {
    static constexpr int v = V;
};

// acc += N block x T block of one 64-value step, both MXFP4; the scales are byte ON of sn and byte OT of st.
template <int ON, int OT>
__device__ __forceinline__ v16f mma(v8i n, v8i t, v16f acc, int sn, int st) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(n, t, acc, 4, 4, ON, sn, OT, st);
}

// Values 8 q .. 8 q + 7 of a lane's block times its scale (byte `at` of `scale`) in bf16, exactly down to 2^-133, for
// scale codes up to 246 (MXFP8) and 252 (MXFP4), the quantizers' largest.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
template <int F>
__device__ __forceinline__ v8bf to_bf16(v8i c, int q, uint32_t scale, int at) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(((scale >> (8 * at)) & 255u) << 23);   // the exponent alone counts; 0 is 2^-127
    v2bf r[4];
    if constexpr (F == 4) {
        const uint32_t x = (uint32_t)c[q];
        r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 0);
        r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 1);
        r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 2);
        r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, s, 3);
    } else {
        const uint32_t x = (uint32_t)c[2 * q], y = (uint32_t)c[2 * q + 1];
        r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, false);
        r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, s, true);
        r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, s, false);
        r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, s, true);
    }
    return v8bf{r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------

// Upper half of a and lower half of b change places.
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// Maximum, and sum, of both halves' values of a token.
__device__ __forceinline__ float both_max(float v) {
    uint32_t a = __float_as_uint(v), b = a;
    swap32(a, b);
    return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float both_sum(float v) {
    uint32_t a = __float_as_uint(v), b = a;
    swap32(a, b);
    return __uint_as_float(a) + __uint_as_float(b);
}

// A lane's 16 values of a 32-column block, as the product left them, in memory at `row`; `left` columns of the block
// exist.  Each store instruction covers 32 contiguous bytes of a row: f32 as the values lie, bf16 after exchanging
// quads 1 with 0 and 3 with 2 between the halves.
__device__ __forceinline__ void bf16_pieces(const uint32_t (&v)[8], u32v4 (&o)[2]) {   // 8 values at 16 i + 8 (l / 32)
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = v[i];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        swap32(q[j], q[2 + j]);
        swap32(q[4 + j], q[6 + j]);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) o[i] = (u32v4){q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]};
}
__device__ __forceinline__ void bf16_pieces(const float (&v)[16], u32v4 (&o)[2]) {
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = bf16x2(v[2 * i], v[2 * i + 1]);
    bf16_pieces(q, o);
}
template <typename V>   // 16 f32, or eight pairs of bf16
__device__ __forceinline__ void store_block(uint16_t *row, const V &v, int lh, int left, bool vec) {
    u32v4 o[2];
    bf16_pieces(v, o);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int c = 16 * i + 8 * lh;
        const u32v4 w = o[i];
        if (vec && c + 8 <= left) {
            st4w<false>(row + c, (u32v4){w[0], w[1], w[2], w[3]});
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (c + j < left) row[c + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
}
__device__ __forceinline__ void store_block(float *row, const float (&v)[16], int lh, int left, bool vec) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int c = 8 * i + 4 * lh;
        if (vec && c + 4 <= left) {
            st4w<false>(row + c, (u32v4){__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                         __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])});
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (c + j < left) row[c + j] = v[4 * i + j];
        }
    }
}

// A 32-value block held by a token's two lanes as MXFP8 (16 bytes of codes at 16 (l / 32)) or MXFP4 (8 bytes at
// 8 (l / 32)); returns the scale code.
__device__ __forceinline__ float block_max(const float (&v)[16]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) a = fmaxf(a, fabsf(v[i]));
    return both_max(a);
}
// The conversions divide by the block's scale themselves: the same codes as from x * 2^-k (tested at every border
// between two codes and its f32 neighbours, for a dozen exponents).  V_CVT_SCALEF32_PK_FP8_F32 does not saturate: values past
// 448 * 2^k, as blocks past the largest exponent have, are clamped before it.  A NaN becomes the NaN code on either path
// (V_MED3_F32 would make it -TOP, in whatever wavefronts clamp).
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d, float scale) {
    typedef short s2 __attribute__((ext_vector_type(2)));
    s2 o = {0, 0};
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, false);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, c, d, scale, true);
    return __builtin_bit_cast(uint32_t, o);
}
__device__ __forceinline__ uint32_t mx8_block(const float (&v)[16], u32v4 &codes) {
    constexpr float TOP = 448.0f * 0x1p119f;
    const float top = block_max(v);
    const int k = mx_block_exponent(top);
    const float s = e8m0_value((uint32_t)(k + 127));
    uint32_t d[4];
    if (__any(top > TOP)) {
        float c[16];
#pragma unroll
        for (int e = 0; e < 16; e++) c[e] = v[e] != v[e] ? v[e] : __builtin_amdgcn_fmed3f(v[e], -TOP, TOP);
#pragma unroll
        for (int q = 0; q < 4; q++) d[q] = fp8x4(c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3], s);
    } else {
#pragma unroll
        for (int q = 0; q < 4; q++) d[q] = fp8x4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3], s);
    }
    swap32(d[0], d[2]);
    swap32(d[1], d[3]);
    codes = (u32v4){d[0], d[2], d[1], d[3]};
    return (uint32_t)(k + 127);
}
__device__ __forceinline__ uint32_t mx4_block(const float (&v)[16], uint2 &codes) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) top = max_nan(top, fabsf(v[i]));
    uint32_t a = __float_as_uint(top), b = a;
    swap32(a, b);
    top = max_nan(__uint_as_float(a), __uint_as_float(b));
    const int k = mx4_block_exponent(top);
    const float s = e8m0_value((uint32_t)(k + 127));
    uint32_t d[4];
#pragma unroll
    for (int q = 0; q < 4; q++) {
        d[q] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[4 * q], v[4 * q + 1], s, 0);
        d[q] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d[q], v[4 * q + 2], v[4 * q + 3], s, 1) & 0xFFFFu;
    }
    swap32(d[0], d[2]);
    swap32(d[1], d[3]);
    codes = make_uint2(d[0] | (d[2] << 16), d[1] | (d[3] << 16));
    return mx4_scale(top, k);
}
__device__ __forceinline__ void store_mx(const float (&v)[16], int fmt, uint8_t *codes, uint8_t *scale, int lh) {
    uint32_t k;
    if (fmt == BSP_FMT_MXFP8) {
        u32v4 c;
        k = mx8_block(v, c);
        st4w<false>(codes + 16 * lh, c);
    } else {
        uint2 c;
        k = mx4_block(v, c);
        st2<false>(codes + 8 * lh, c);
    }
    if (lh == 0) *scale = (uint8_t)k;
}

// Four E4M3 codes times s.
__device__ __forceinline__ void values4(uint32_t c, float s, float *v) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    v[0] = lo.x * s;
    v[1] = lo.y * s;
    v[2] = hi.x * s;
    v[3] = hi.y * s;
}

// The checkpoint of 32 columns of a token: 16 bytes of each half per lane, exchanged into the product's order.
struct Ckpt {
    u32v4 gate, up;
    uint32_t sg, su;
};
__device__ __forceinline__ Ckpt load_ckpt(const MxArgs &p, int r, int col, int lh) {
    Ckpt k;
    const bool in = r >= 0 && col < p.I;
    const int64_t at = in ? (int64_t)r * 2 * p.I + col : 0;   // loaded in any case, dropped later
    k.gate = ld4w<false>(p.ckpt_codes + at + 16 * lh);
    k.up = ld4w<false>(p.ckpt_codes + at + p.I + 16 * lh);
    k.sg = p.ckpt_scales[at / 32];
    k.su = p.ckpt_scales[(at + p.I) / 32];
    return k;
}

// Gradients of gate and up of 32 columns from dh, and h, as pairs of bf16 (pair 2 q + j: columns 8 q + 4 (l / 32) + 2 j
// and the next); returns the lane's part of sum dh act up.  Four columns at a time: 32-column arrays of f32 would not
// fit the registers beside the accumulators.
__device__ __forceinline__ float gated_backward(const Ckpt &k, const v16f &acc, bool ok, float w, uint32_t (&dg)[8],
                                                uint32_t (&du)[8], uint32_t (&h)[8]) {
    uint32_t gc[4] = {k.gate[0], k.gate[2], k.gate[1], k.gate[3]}, uc[4] = {k.up[0], k.up[2], k.up[1], k.up[3]};
    swap32(gc[0], gc[2]);
    swap32(gc[1], gc[3]);
    swap32(uc[0], uc[2]);
    swap32(uc[1], uc[3]);
    const float sg = e8m0_value(k.sg), su = e8m0_value(k.su);
    float dw = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; q++) {
        float gate[4], up[4], s[4], rest[4], x[4], y[4], z[4];
        values4(gc[q], sg, gate);
        values4(uc[q], su, up);
        sigmoid<true>(gate, s, rest);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float dh = ok ? acc[4 * q + e] : 0.0f, act = gate[e] * s[e], d = w * dh, au = act * up[e];
            dw += dh * au;
            z[e] = w * au;
            y[e] = d * act;
            x[e] = d * up[e] * (s[e] + act * (1.0f - s[e]));
        }
#pragma unroll
        for (int j = 0; j < 2; j++) {
            dg[2 * q + j] = bf16x2(x[2 * j], x[2 * j + 1]);
            du[2 * q + j] = bf16x2(y[2 * j], y[2 * j + 1]);
            h[2 * q + j] = bf16x2(z[2 * j], z[2 * j + 1]);
        }
        // one after the other, for the registers' sake
        asm volatile("" : "+v"(dw), "+v"(dg[2 * q]), "+v"(du[2 * q]), "+v"(h[2 * q]));
        __builtin_amdgcn_sched_barrier(0);
    }
    return dw;
}

// What follows the product of 32 tokens with 64 rows of B in the form for few rows, the backward pass apart: acc[j] is
// block j of them.  Lane l has token row r of C (r < 0: none).  ok: the row's source exists (else it counts as zeros);
// w: its weight.  col: first column (gated: of the 32 columns of h, acc[0] gate and acc[1] up).
template <int EPI>
__device__ __forceinline__ void epilogue(const MxArgs &p, v16f (&acc)[2], int r, bool ok, float w, int col, int lh) {
    float v[2][16];
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) v[j][e] = ok ? acc[j][e] : 0.0f;
    if constexpr (EPI == EPI_BF16 || EPI == EPI_F32) {
        const int64_t at = (int64_t)(r < 0 ? 0 : r) * p.ldc + col;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int left = r < 0 ? 0 : p.N - (col + 32 * j);   // both lanes of a token exchange in any case
            if constexpr (EPI == EPI_BF16)
                store_block(reinterpret_cast<uint16_t *>(p.c) + at + 32 * j, v[j], lh, left, (p.ldc & 7) == 0);
            else
                store_block(reinterpret_cast<float *>(p.c) + at + 32 * j, v[j], lh, left, (p.ldc & 3) == 0);
        }
    } else {
        if (r < 0 || col >= p.I) return;   // a token's lanes agree
        if (p.ckpt_codes) {
            const int64_t at = (int64_t)r * 2 * p.I + col;
            store_mx(v[0], BSP_FMT_MXFP8, p.ckpt_codes + at, p.ckpt_scales + at / 32, lh);
            store_mx(v[1], BSP_FMT_MXFP8, p.ckpt_codes + at + p.I, p.ckpt_scales + (at + p.I) / 32, lh);
        }
        float h[16], s[16], rest[16];
        sigmoid<true>(v[0], s, rest);   // h is rounded once, to 3 bits or to bf16, from f32
#pragma unroll
        for (int e = 0; e < 16; e++) h[e] = w * (v[0][e] * s[e] * v[1][e]);
        const int64_t at = (int64_t)r * p.I + col;
        if (p.h_fmt >= 0) {
            uint8_t *codes = p.h_codes + (p.h_fmt == BSP_FMT_MXFP8 ? at : at / 2);
            store_mx(h, p.h_fmt, codes, p.h_scales + at / 32, lh);
        }
        if (p.h) store_block(p.h + at, h, lh, 32, true);
    }
}

// B row of tile row `i` of a 64-row block: the gated block pairs 32 rows of the gate with the 32 of up that share
// their columns.
template <int EPI>
__device__ __forceinline__ int b_row(const MxArgs &p, int col, int i) {
    if (EPI == EPI_GATED) {
        const int c = col + (i & 31);
        return (i & 32 ? p.I : 0) + (c < p.I ? c : p.I - 1);
    }
    return col + i < p.N ? col + i : p.N - 1;
}

// Row tile y of 2^LB rows among the groups' tiles in order: its group, the group's rows [lo, hi) (at most M) and first
// tile.  All NT threads call it.
template <int LB, int NT>
__device__ __forceinline__ bool find_tile(const int64_t *off, int G, int M, int y, i32v4 &tile) {
    __shared__ int found[4];
    __shared__ int wsum[NT / 64];
    const int t = threadIdx.x, lane = t & 63;
    int carry = 0;
    for (int base = 0; base < G; base += NT) {
        const int i = base + t;
        int64_t lo = 0, hi = 0;
        if (i < G) {
            lo = off[i];
            hi = off[i + 1];
            lo = lo < M ? lo : M;
            hi = hi < M ? hi : M;
        }
        const int cnt = hi > lo ? (int)((hi - lo + (1 << LB) - 1) >> LB) : 0;
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(incl, o, 64);
            if (lane >= o) incl += u;
        }
        if (lane == 63) wsum[t >> 6] = incl;
        __syncthreads();
        int first = carry + incl - cnt;
#pragma unroll
        for (int w = 0; w < NT / 64; w++) {
            if (w < t >> 6) first += wsum[w];
            carry += wsum[w];
        }
        if (y >= first && y < first + cnt) {
            found[0] = i;
            found[1] = (int)lo;
            found[2] = (int)hi;
            found[3] = first;
        }
        __syncthreads();
        if (y < carry) {
            tile.x = __builtin_amdgcn_readfirstlane(found[0]);
            tile.y = __builtin_amdgcn_readfirstlane(found[1]);
            tile.z = __builtin_amdgcn_readfirstlane(found[2]);
            tile.w = __builtin_amdgcn_readfirstlane(found[3]);
            return true;
        }
    }
    return false;
}

}  // namespace

// ---------------------------------------------------------------------------
// Few rows (serving): no staging, K split over the workgroup.
// ---------------------------------------------------------------------------
// A workgroup has 32 tokens and 64 rows of B; its eight wavefronts take every
// eighth chunk of 256 K values, straight from global memory into registers,
// and their sums meet in LDS.  The weights are read once and are what bounds
// this form: a chunk's loads are all issued before its first product.
template <int FT, int FN, int EPI>
__global__ __launch_bounds__(512) void k_mx_few(MxArgs p) {
    __shared__ float part[8][32][64];
    const int t = threadIdx.x, l = t & 63, lr = l & 31, lh = l >> 5;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    i32v4 tile;
    if (!find_tile<5, 512>(p.off, p.G, p.M, blockIdx.y, tile)) return;
    const int g = tile.x, row0 = tile.y + 32 * ((int)blockIdx.y - tile.w), row1 = tile.z;
    const int col = blockIdx.x * (EPI == EPI_GATED ? 32 : 64);
    const int r = row0 + lr < row1 ? row0 + lr : -1;
    int src = r;
    if (r >= 0 && p.gather) src = p.gather[r];
    const bool ok = src >= 0 && src < p.a_rows;

    const uint32_t ldt = FT == 4 ? p.K / 2 : p.K, ldn = FN == 4 ? p.K / 2 : p.K;
    const int nblk = p.K / 32;
    const uint8_t *tc = p.a_codes + (size_t)(ok ? src : 0) * ldt, *ts = p.a_scales + (size_t)(ok ? src : 0) * nblk;
    const uint8_t *nc[2], *ns[2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const size_t n = (size_t)g * p.N + b_row<EPI>(p, col, 32 * j + lr);
        nc[j] = p.b_codes + n * ldn;
        ns[j] = p.b_scales + n * nblk;
    }
    v16f acc[2];
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[j][e] = 0.0f;

    // the scale bytes of eight K blocks from block b on, those of this lane's half in bytes 0 and 2 of two words
    auto scales = [&](const uint8_t *s, int b, uint32_t (&o)[2]) __attribute__((always_inline)) {
        uint64_t v = 0;
        if (b + 8 <= nblk) {
            __builtin_memcpy(&v, s + b, 8);
        } else {
            for (int i = 0; i < nblk - b; i++) v |= (uint64_t)s[b + i] << (8 * i);
        }
        v >>= 8 * lh;
        o[0] = (uint32_t)v;
        o[1] = (uint32_t)(v >> 32);
    };
    // this lane's codes of the 64-value step at k0 (zeros past K)
    auto codes = [&](auto F, const uint8_t *c, int k0) __attribute__((always_inline)) -> v8i {
        constexpr int f = decltype(F)::v;
        v8i v = {0, 0, 0, 0, 0, 0, 0, 0};
        if constexpr (f == 4) {
            if (k0 + 32 * lh < p.K) {
                const u32v4 x = ld4w<false>(c + k0 / 2 + 16 * lh);
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] = (int)x[i];
            }
        } else {
            if (k0 + 32 * lh < p.K) {
                const u32v4 x = ld4w<false>(c + k0 + 32 * lh), y = ld4w<false>(c + k0 + 32 * lh + 16);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    v[i] = (int)x[i];
                    v[4 + i] = (int)y[i];
                }
            }
        }
        return v;
    };
    for (int k0 = 256 * w; k0 < p.K; k0 += 8 * 256) {
        uint32_t st[2], sn[2][2];
        v8i a[4], b[4][2];
        scales(ts, k0 / 32, st);
#pragma unroll
        for (int j = 0; j < 2; j++) scales(ns[j], k0 / 32, sn[j]);
#pragma unroll
        for (int s = 0; s < 4; s++) {
            if (k0 + 64 * s < p.K) {
                a[s] = codes(IC<FT>{}, tc, k0 + 64 * s);
#pragma unroll
                for (int j = 0; j < 2; j++) b[s][j] = codes(IC<FN>{}, nc[j], k0 + 64 * s);
            }
        }
        auto step = [&](auto S) __attribute__((always_inline)) {
            constexpr int s = decltype(S)::v;
            if (k0 + 64 * s < p.K) {
                if constexpr (FT == 4) {
#pragma unroll
                    for (int j = 0; j < 2; j++)
                        acc[j] = mma<2 * (s & 1), 2 * (s & 1)>(b[s][j], a[s], acc[j], (int)sn[j][s >> 1], (int)st[s >> 1]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const v8bf t = to_bf16<FT>(a[s], q, st[s >> 1], 2 * (s & 1));
#pragma unroll
                        for (int j = 0; j < 2; j++)
                            acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                to_bf16<FN>(b[s][j], q, sn[j][s >> 1], 2 * (s & 1)), t, acc[j], 0, 0, 0);
                    }
                }
            }
        };
        step(IC<0>{});
        step(IC<1>{});
        step(IC<2>{});
        step(IC<3>{});
    }
    // eight partial sums of each value, in a fixed order: each wavefront adds up four of a lane's 32
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) part[w][16 * j + e][l] = acc[j][e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float s = part[0][4 * w + i][l];
#pragma unroll
        for (int q = 1; q < 8; q++) s += part[q][4 * w + i][l];
        part[0][4 * w + i][l] = s;
    }
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[j][e] = part[0][16 * j + e][l];
    const float rw = r >= 0 && p.row_weights ? p.row_weights[r] : 1.0f;
    if constexpr (EPI == EPI_GATED_BWD) {
        float dw = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int c = col + 32 * j;
            const Ckpt k = load_ckpt(p, r, c, lh);
            uint32_t dg[8], du[8], h[8];
            const float sum = gated_backward(k, acc[j], ok, rw, dg, du, h);
            if (r < 0 || c >= p.I) continue;   // a token's lanes agree
            dw += sum;
            const int64_t at = (int64_t)r * 2 * p.I + c;
            store_block(p.dh13 + at, dg, lh, 32, true);
            store_block(p.dh13 + at + p.I, du, lh, 32, true);
            if (p.h) store_block(p.h + (int64_t)r * p.I + c, h, lh, 32, true);
        }
        dw = both_sum(dw);
        if (p.part && r >= 0 && lh == 0) p.part[(int64_t)r * p.parts + col / 64] = dw;
    } else {
        epilogue<EPI>(p, acc, r, ok, rw, col, lh);
    }
}

// d_row_weights: a row's sums over 64 columns, in order.
__global__ __launch_bounds__(256) void k_row_sums(const float *__restrict__ part, int parts, int M,
                                                  const int64_t *__restrict__ off, int G, float *__restrict__ out) {
    const int64_t r = grid_index() * 256 + threadIdx.x;
    if (r >= M || r >= off[G] || r < off[0]) return;
    float s = 0.0f;
    for (int i = 0; i < parts; i++) s += part[r * parts + i];
    out[r] = s;
}

// ---------------------------------------------------------------------------
// Tiled form.
// ---------------------------------------------------------------------------
// A workgroup computes TB tokens x NB rows of B (gated: NB / 2 columns of h) by
// 2 x WN wavefronts, each TI blocks of 32 tokens x 64.  Stages of both operands
// stream into a ring in LDS, in whole 128-byte lines of every row where the
// format allows: pieces of 64 bytes reach half the rate (17.7 against 33 TB/s
// from the L2).
//   128 x 256: eight wavefronts, one workgroup per compute unit.  256 x 256
//     with a ring of two was faster where the output bounds it (65536 x 768 x
//     2048 by 128 experts: 117 against 133 us) and slower for experts of some
//     hundred rows (36864 x 7168 x 4096 by 257: 1430 against 1240 us).
//   64 x 128, for groups of few rows: four wavefronts, two workgroups per unit
//     (1218 rows of 60 experts, backward: 28 us against 31 of 64 x 256).
template <int FT, int FN, int TB_>
struct MxGeo {
    static constexpr bool BIG = TB_ == 128;
    static constexpr int TB = TB_, NB = BIG ? 256 : 128, WN = NB / 64, NW = 2 * WN, NT = 64 * NW;
    static constexpr int TI = TB / 64;                            // blocks of 32 tokens of a wavefront
    static constexpr int BK = FT == 4 && FN == 4 ? 256 : 128;     // K values of a stage
    static constexpr int SUB = BK / 64, U = BK / 64;              // 64-value steps; scale bytes of a row and lane half
    static constexpr int SPS = 2 * U;                             // scales of a row per stage
    static constexpr int RT = BK * FT / 8, RN = BK * FN / 8;      // code bytes of a row per stage
    static constexpr int CT = TB * RT, CN = NB * RN;              // of an operand
    static constexpr int LT = CT / 1024 / NW, LN = CN / 1024 / NW;   // 1 KB loads per wavefront
    static constexpr int ST = CT + CN, SN = ST + TB * SPS;        // scales of T and N in the stage
    static constexpr int BYTES = SN + NB * SPS;
    static constexpr int LEAST = BIG ? 50688 : 25344, SLOT = BYTES > LEAST ? BYTES : LEAST;   // also the epilogue's (finish)
    static constexpr int NS = 3;                                  // stages in the ring
    static constexpr int SW = NB * SPS > 1024 ? 3 : 2;            // wavefronts that load scales
    static constexpr int OPS = LT + LN;                           // loads per wavefront and stage, scales apart
    static_assert(NS * SLOT + 20 * TB + 128 <= (BIG ? 160 : 80) * 1024, "workgroups per compute unit");
    // a lane's scales of a stage lie together: U bytes of each of its blocks, TI for T and two for N
    static constexpr int TCH = TI * U, NCH = 2 * U;
};

// Where the U scale bytes of row r (of a tile of T or N) and lane half h lie in a stage's scales.
template <typename Geo>
__device__ __forceinline__ int t_chunk(int r, int h) {
    const int blk = r >> 5;
    return (((blk / Geo::TI) * 32 + (r & 31)) * 2 + h) * Geo::TCH + (blk % Geo::TI) * Geo::U;
}
template <typename Geo>
__device__ __forceinline__ int n_chunk(int r, int h) {
    return (((r >> 6) * 32 + (r & 31)) * 2 + h) * Geo::NCH + ((r >> 5) & 1) * Geo::U;
}

// Eight scale bytes of one row from block b on, zeros from block `end` on.
__device__ __forceinline__ uint64_t eight_scales(const uint8_t *row, int64_t b, int64_t end) {
    uint64_t v = 0;
    if (b + 8 <= end) {
        __builtin_memcpy(&v, row + b, 8);
    } else {
        for (int i = 0; i < 8; i++)
            if (b + i < end) v |= (uint64_t)row[b + i] << (8 * i);
    }
    return v;
}
// Bytes 0, 2, 4, 6 (h = 0) or 1, 3, 5, 7 of them: a lane half's blocks of the 64-value steps.
__device__ __forceinline__ uint32_t half_scales(uint64_t v, int h) {
    return __builtin_amdgcn_perm((uint32_t)(v >> 32), (uint32_t)v, h ? 0x07050301u : 0x06040200u);
}

// One launch before the product: the row-tile list and its length, and the scales of both operands tile by tile and
// stage by stage in the order the product reads them (as they are stored, a stage's bytes of each row are a cache
// line apart).
// Row-grouped: workgroups below ntm have a row tile each, the others 256 rows of a group's B.
template <int FT, int FN, int EPI, int TB>
__global__ __launch_bounds__(256) void k_mx_prep(MxArgs p) {
    using Geo = MxGeo<FT, FN, TB>;
    constexpr int U = Geo::U, SPS = Geo::SPS, W = 8 / SPS;   // stages in eight scales
    constexpr int PASS = 4 * W;                              // stages staged at a time (32 scales of a row)
    constexpr int PER = 256 / Geo::NB;                       // column tiles of a workgroup
    __shared__ __attribute__((aligned(16))) uint8_t buf[256 * 32];
    const int t = threadIdx.x, nblk = p.K / 32;
    const uint8_t *row = nullptr;
    uint8_t *out = nullptr;
    const bool tokens = (int)blockIdx.x < p.ntm;
    const int rows = tokens ? TB : Geo::NB, half = tokens ? 0 : t / Geo::NB, i = t - half * Geo::NB;
    if (tokens) {
        constexpr int LB = TB == 128 ? 7 : 6;
        const int y = blockIdx.x;
        i32v4 tile;
        // the listed tiles are the first `count`: the workgroup of the first one that is not listed writes the length
        if (!find_tile<LB, 256>(p.off, p.G, p.M, y, tile)) {
            if (y == 0 || find_tile<LB, 256>(p.off, p.G, p.M, y - 1, tile)) {
                if (t == 0) *p.count = y;
            }
            return;
        }
        const int r = tile.y + TB * (y - tile.w) + i;
        if (t == 0) p.tiles[y] = tile;
        if (y == p.ntm - 1 && t == 0) *p.count = p.ntm;
        if (i < TB && r < tile.z) {
            const int src = p.gather ? p.gather[r] : r;
            if (src >= 0 && src < p.a_rows) row = p.a_scales + (size_t)src * nblk;
        }
        out = p.a_plane + (size_t)y * p.stages * TB * SPS;
    } else {
        const int runs = (p.ntn + PER - 1) / PER, b = blockIdx.x - p.ntm, g = b / runs, nt = PER * (b - g * runs) + half;
        if (p.off[g + 1] <= p.off[g]) return;
        const int col = EPI == EPI_GATED ? Geo::NB / 2 * nt + 32 * (i >> 6) : Geo::NB * nt + (i & ~63);
        if (nt < p.ntn) {
            row = p.b_scales + ((size_t)g * p.N + b_row<EPI>(p, col, i & 63)) * nblk;
            out = p.b_plane + ((size_t)g * p.ntn + nt) * p.stages * Geo::NB * SPS;
        }
    }
    const int pitch = rows * SPS;   // bytes of a stage
    uint8_t *mine = buf + half * Geo::NB * 32;
    for (int s0 = 0; s0 < p.stages; s0 += PASS) {
        if (out && i < rows) {
            uint64_t v[4];
#pragma unroll
            for (int q = 0; q < 4; q++) v[q] = row ? eight_scales(row, (int64_t)s0 * SPS + 8 * q, nblk) : 0;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int at = tokens ? t_chunk<Geo>(i, h) : n_chunk<Geo>(i, h);
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const uint32_t x = half_scales(v[q], h);
#pragma unroll
                    for (int k = 0; k < W; k++) {
                        const uint32_t y = x >> (8 * U * k);
                        __builtin_memcpy(mine + (W * q + k) * pitch + at, &y, U);
                    }
                }
            }
        }
        __syncthreads();
        const int n = (p.stages - s0 < PASS ? p.stages - s0 : PASS) * pitch;
        if (out)
            for (int k = 16 * i; k < n; k += tokens ? 4096 : 16 * Geo::NB)
                *reinterpret_cast<uint4 *>(out + (size_t)s0 * pitch + k) = *reinterpret_cast<const uint4 *>(mine + k);
        __syncthreads();
    }
}

// Weight gradient: stage slot y is stage s of group g, all groups' stages in order; the scales of a run of rows of both
// operands for it.  The first workgroup lists each XCD's groups, the largest first: up to 512
// groups each goes to the XCD with the least work so far (128 experts of 142 to 7300 rows: 39 stages of K at most where
// dealing them out in alternating direction left 52 and a third of the chip idle), more are dealt out.
constexpr int kWgradRows = 512;
template <int FT, int FN>
__global__ __launch_bounds__(256) void k_mx_prep_wgrad(MxArgs p) {
    using Geo = MxGeo<FT, FN, 128>;
    constexpr int U = Geo::U, SPS = Geo::SPS;
    const bool list = blockIdx.x == 0;   // it takes longest
    const int t = threadIdx.x, y = list ? 0x7fffffff : (int)blockIdx.x - 1;
    if (list && blockIdx.y) return;
    __shared__ int64_t wsum[4];
    __shared__ int64_t found[2];
    constexpr int MANY = 512;
    __shared__ i32v4 sorted[MANY];
    __shared__ int place[MANY], many[8];
    const bool greedy = p.G <= MANY;
    if (list && greedy) {
        for (int g = t; g < p.G; g += 256) place[g] = (int)(p.off[g + 1] - p.off[g]);
        __syncthreads();
    }
    int64_t carry = 0, pcarry = 0;
    for (int b = 0; b < p.G; b += 256) {
        const int g = b + t;
        int64_t n = 0;
        if (g < p.G) n = (p.off[g + 1] - p.off[g] + 31) / 32 * 32;
        const int64_t cnt = (n + Geo::BK - 1) / Geo::BK;
        int64_t total, ptotal;
        const int64_t at = carry + block256_excl_scan(cnt, wsum, total);
        const int64_t c0 = pcarry + block256_excl_scan(n, wsum, ptotal), c1 = c0 + n;
        const int beg = (int)(c0 < p.K ? c0 : p.K), end = (int)(c1 < p.K ? c1 : p.K);   // never past the copies' width
        if (list && g < p.G) {
            // rank by counting; past 4096 groups the order stays as it is
            int rank = g;
            if (greedy) {
                const int m = place[g];
                rank = 0;
                for (int h = 0; h < p.G; h++) rank += place[h] > m || (place[h] == m && h < g);
            } else if (p.G <= 4096) {
                const int64_t m = p.off[g + 1] - p.off[g];
                rank = 0;
                for (int h = 0; h < p.G; h++) {
                    const int64_t o = p.off[h + 1] - p.off[h];
                    rank += o > m || (o == m && h < g);
                }
            }
            const i32v4 e = {g, beg, end, (int)at};
            const int q = rank / 8;
            if (greedy) sorted[rank] = e;
            else p.tiles[(int64_t)(q & 1 ? 7 - rank % 8 : rank % 8) * p.G + q] = e;
        }
        if (y >= at && y < at + cnt) {
            found[0] = beg + (y - at) * Geo::BK;
            found[1] = end;
        }
        __syncthreads();
        carry += total;
        pcarry += ptotal;
        if (y < carry) break;
    }
    if (list) {
        if (greedy) {
            __syncthreads();
            if (t == 0) {
                int load[8] = {0, 0, 0, 0, 0, 0, 0, 0}, of[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                int next = sorted[0].z - sorted[0].y;
                for (int r = 0; r < p.G; r++) {
                    const int len = next;
                    if (r + 1 < p.G) next = sorted[r + 1].z - sorted[r + 1].y;
                    const int work = (len + Geo::BK - 1) / Geo::BK + 2;   // its stages, and two for the outputs
                    // the least of the eight, as keys 8 load + XCD
                    int m[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) m[k] = min(8 * load[k] + k, 8 * load[k + 4] + k + 4);
                    const int x = min(min(m[0], m[1]), min(m[2], m[3])) & 7;
                    int at = 0;
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        at = k == x ? of[k] : at;
                        load[k] += k == x ? work : 0;
                        of[k] += k == x;
                    }
                    place[r] = x * p.G + at;
                }
#pragma unroll
                for (int k = 0; k < 8; k++) many[k] = of[k];
            }
            __syncthreads();
            for (int r = t; r < p.G; r += 256) p.tiles[place[r]] = sorted[r];
            if (t < 8) p.count[t] = many[t];
        } else if (t < 8) {
            const int q = p.G / 8, i = q & 1 ? 7 - t : t;   // its place in the last round
            p.count[t] = q + (i < p.G % 8);
        }
        return;
    }
    if (y >= carry) return;
    const int64_t b0 = found[0] / 32, end = found[1] / 32 < b0 + SPS ? found[1] / 32 : b0 + SPS, sr = p.K / 32;
    const int mt = p.ntm * Geo::TB, nt = p.ntn * Geo::NB;
#pragma unroll
    for (int k = 0; k < kWgradRows / 256; k++) {
        const int r = blockIdx.y * kWgradRows + 256 * k + t;
        if (r >= mt + nt) break;
        const bool n = r >= mt;
        const int i = n ? r - mt : r;
        uint64_t v = 0;
        if (i < (n ? p.N : p.M)) v = eight_scales((n ? p.b_scales : p.a_scales) + (size_t)i * sr, b0, end);
        uint8_t *out = n ? p.b_plane + ((size_t)y * p.ntn + i / Geo::NB) * Geo::NB * SPS
                         : p.a_plane + ((size_t)y * p.ntm + i / Geo::TB) * Geo::TB * SPS;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t x = half_scales(v, h);
            __builtin_memcpy(out + (n ? n_chunk<Geo>(i % Geo::NB, h) : t_chunk<Geo>(i % Geo::TB, h)), &x, U);
        }
    }
}

// Chunk c of row r of a stage lies at c ^ swizzle(r).  A fragment's read takes one chunk of 32 rows; in groups of 16 of
// them the chunks fill all 64 banks once.
template <int CH>
__device__ __forceinline__ int swizzle(int r) {
    return CH == 8 ? (r >> 1) & 7 : (r >> 2) & 3;
}

// One output tile: group, rows [row0, row1), column tile, columns [beg, end) of the copies and their stages.
struct MxTile {
    int g, row0, row1, ct, beg, end, nk;
    int slot;   // row tile in the list; weight gradient: first stage slot
    int tm;     // row tile of the matrix (weight gradient)
};

// Persistent workgroups: each walks its tiles, and the ring runs on across
// them, so a tile's first stages are on their way while the one before is
// finished and written.  What a tile's loads need, its list entry, row indices
// and weights, is fetched when the tile before begins to load.  Row-grouped:
// XCD-contiguous runs of the tile order, in which a group's row tiles of one
// column tile are neighbours (they share the weights in that XCD's L2).
// Weight gradient: a group's tiles are one XCD's (k_mx_prep_wgrad).
template <int FT, int FN, int EPI, bool WG, int TB>
__global__ __launch_bounds__((MxGeo<FT, FN, TB>::NT), 2) void k_mx_tile(MxArgs p) {
    using Geo = MxGeo<FT, FN, TB>;
    constexpr int NS = Geo::NS, SPS = Geo::SPS, SUB = Geo::SUB, TI = Geo::TI, U = Geo::U;
    constexpr int CHT = Geo::RT / 16, CHN = Geo::RN / 16;
    __shared__ __attribute__((aligned(16))) uint8_t ring[NS * Geo::SLOT];
    // of the last four tiles that were begun (the loads of a tile begin at most two stages, hence tiles, before its
    // products): what the epilogue needs, and each row's weight and whether it has a source
    __shared__ int info[4][8];
    __shared__ float row_w[WG ? 1 : 4][Geo::TB];
    __shared__ uint8_t row_ok[WG ? 1 : 4][Geo::TB];
    const int t = threadIdx.x, l = t & 63, lr = l & 31, lh = l >> 5;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6), wt = w / Geo::WN, wn = w % Geo::WN;   // along the tokens and along B
    const uint32_t ring_lds = lds_addr(ring);
    const uint32_t ldt = FT == 4 ? p.K / 2 : p.K, ldn = FN == 4 ? p.K / 2 : p.K;

    // ---- this workgroup's tiles: first, first + stride, .. below last ----
    const int x = blockIdx.x & 7, stride = gridDim.x >> 3, per = p.ntm * p.ntn;
    int first, last;
    if (WG) {
        first = blockIdx.x >> 3;
        last = p.count[x] * per;
    } else {
        const int total = *p.count * p.ntn, chunk = (total + 7) / 8;
        first = x * chunk + (blockIdx.x >> 3);
        last = (x + 1) * chunk < total ? (x + 1) * chunk : total;
    }
    // the list entry of tile `lin`, and the tile
    auto entry = [&](int lin) __attribute__((always_inline)) -> i32v4 {
        return sload(p.tiles, WG ? (int64_t)x * p.G + lin / per : (int64_t)(lin / p.ntn));
    };
    auto decode = [&](int lin, i32v4 e) __attribute__((always_inline)) -> MxTile {
        MxTile T;
        T.g = e.x;
        if (WG) {
            const int i = lin % per;
            T.tm = i % p.ntm;
            T.ct = i / p.ntm;
            T.row0 = T.tm * Geo::TB;
            T.row1 = p.M;
            T.beg = e.y;
            T.end = e.z;
            T.slot = e.w;
        } else {
            const int nt = (e.z - e.y + Geo::TB - 1) / Geo::TB, local = lin - e.w * p.ntn;
            T.slot = e.w + local % nt;
            T.ct = local / nt;
            T.row0 = e.y + (local % nt) * Geo::TB;
            T.row1 = e.z;
            T.beg = 0;
            T.end = p.K;
        }
        T.nk = T.end > T.beg ? (T.end - T.beg + Geo::BK - 1) / Geo::BK : 0;
        return T;
    };

    // ---- producer: stages into the ring ----
    // P: the tile whose stages are loaded; Q: the next one, with its row indices and weights on their way; E: the list
    // entry of the one after
    int q_lin = first, p_kt = 0, p_ord = -1;
    bool more = first < last;   // Q is a tile
    MxTile P, Q;
    P.nk = 0;
    i32v4 E = {0, 0, 0, 0};
    int q_src[Geo::LT], q_row = 0;
    float q_w = 1.0f;
    uint32_t ot[Geo::LT], on[Geo::LN];   // this lane's pieces: unit u = 64 (w L + j) + l is chunk u % CH of row u / CH
    const uint8_t *ca = nullptr, *cb = nullptr, *pa = nullptr, *pb = nullptr;
    const size_t pitch_a = (size_t)(WG ? p.ntm : 1) * Geo::TB * SPS, pitch_b = (size_t)(WG ? p.ntn : 1) * Geo::NB * SPS;
    // Q from E; tiles without K work (groups without tokens) are left out
    auto look_ahead = [&]() __attribute__((always_inline)) {
        for (;; E = entry(q_lin)) {
            Q = decode(q_lin, E);
            if (Q.nk > 0) break;
            q_lin += stride;
            if (q_lin >= last) {
                more = false;
                return;
            }
        }
        if constexpr (!WG) {
#pragma unroll
            for (int j = 0; j < Geo::LT; j++) {
                const int i = (64 * (w * Geo::LT + j) + l) / CHT;
                const int r = Q.row0 + i < Q.row1 ? Q.row0 + i : Q.row0;
                q_src[j] = p.gather ? p.gather[r] : r;
            }
            const int r = Q.row0 + (t & (Geo::TB - 1)) < Q.row1 ? Q.row0 + (t & (Geo::TB - 1)) : Q.row0;
            q_row = p.gather ? p.gather[r] : r;
            if (EPI >= EPI_GATED) q_w = p.row_weights ? p.row_weights[r] : 1.0f;
        }
        const int n = q_lin + stride;
        if (n < last) E = entry(n);
    };
    // begin Q
    auto advance = [&]() __attribute__((always_inline)) {
        P = Q;
        p_kt = 0;
        p_ord = (p_ord + 1) & 3;
#pragma unroll
        for (int j = 0; j < Geo::LT; j++) {
            const int u = 64 * (w * Geo::LT + j) + l, i = u / CHT, c = (u % CHT) ^ swizzle<CHT>(i);
            int src;
            if (WG) src = P.row0 + i < P.row1 ? P.row0 + i : P.row0;
            else src = q_src[j] >= 0 && q_src[j] < p.a_rows ? q_src[j] : 0;   // counted as zeros in the epilogue
            ot[j] = (uint32_t)src * ldt + 16 * c;
        }
#pragma unroll
        for (int j = 0; j < Geo::LN; j++) {
            const int u = 64 * (w * Geo::LN + j) + l, i = u / CHN, c = (u % CHN) ^ swizzle<CHN>(i);
            const int col = EPI == EPI_GATED ? Geo::NB / 2 * P.ct + 32 * (i >> 6) : Geo::NB * P.ct + (i & ~63);
            on[j] = (uint32_t)b_row<EPI>(p, col, i & 63) * ldn + 16 * c;
        }
        if (!WG && t < Geo::TB) {
            row_ok[WG ? 0 : p_ord][t] = q_row >= 0 && q_row < p.a_rows;
            if (EPI >= EPI_GATED) row_w[WG ? 0 : p_ord][t] = q_w;
        }
        if (t == 0) {
            int *o = info[p_ord];
            o[0] = P.g; o[1] = P.row0; o[2] = P.row1; o[3] = P.ct; o[4] = P.nk;
        }
        ca = uniform_ptr(p.a_codes + (WG ? (size_t)P.beg * FT / 8 : 0));
        cb = uniform_ptr(p.b_codes + (WG ? (size_t)P.beg * FN / 8 : (size_t)P.g * p.N * ldn));
        if (WG) {
            pa = uniform_ptr(p.a_plane + ((size_t)P.slot * p.ntm + P.tm) * Geo::TB * SPS);
            pb = uniform_ptr(p.b_plane + ((size_t)P.slot * p.ntn + P.ct) * Geo::NB * SPS);
        } else {
            pa = uniform_ptr(p.a_plane + (size_t)P.slot * p.stages * Geo::TB * SPS);
            pb = uniform_ptr(p.b_plane + ((size_t)P.g * p.ntn + P.ct) * p.stages * Geo::NB * SPS);
        }
        q_lin += stride;
        more = q_lin < last;
        if (more) look_ahead();
    };
    // Loads of the next stage (`begin` first) into the ring at byte `at`, part q of SUB of them: issued all at once they
    // held the wavefronts up for two thirds of the stage's products' time, so each step of the products issues a part.
    bool loading = false;
    int left = 0;
    uint32_t l_m0 = 0;
    const uint8_t *l_a = nullptr, *l_b = nullptr;
    auto begin = [&](uint32_t at) __attribute__((always_inline)) {
        loading = p_kt < P.nk || more;
        if (!loading) return;
        if (p_kt == P.nk) advance();
        l_m0 = ring_lds + at;
        left = P.end - P.beg - p_kt * Geo::BK;
        l_a = ca + (size_t)p_kt * Geo::RT;
        l_b = cb + (size_t)p_kt * Geo::RN;
    };
    auto issue = [&](auto Q) __attribute__((always_inline)) {
        constexpr int q = decltype(Q)::v;
        if (!loading) return;
        uint32_t m0 = l_m0;
        asm volatile("" : "+s"(m0));   // opaque: hoisted, the destinations of all loads would each hold a register
        if (left >= Geo::BK) {
#pragma unroll
            for (int j = 0; j < Geo::LT; j++)
                if (j * SUB / Geo::LT == q) dma16(l_a, ot[j], m0 + (w * Geo::LT + j) * 1024);
#pragma unroll
            for (int j = 0; j < Geo::LN; j++)
                if (j * SUB / Geo::LN == q) dma16(l_b, on[j], m0 + Geo::CT + (w * Geo::LN + j) * 1024);
        } else {
            // chunks past the end are zeros (so are their scales)
#pragma unroll
            for (int j = 0; j < Geo::LT; j++) {
                const int u = 64 * (w * Geo::LT + j) + l, c = (u % CHT) ^ swizzle<CHT>(u / CHT);
                if (j * SUB / Geo::LT == q)
                    dma16v(c * (128 / FT) >= left ? kZeroChunk : l_a + ot[j], m0 + (w * Geo::LT + j) * 1024);
            }
#pragma unroll
            for (int j = 0; j < Geo::LN; j++) {
                const int u = 64 * (w * Geo::LN + j) + l, c = (u % CHN) ^ swizzle<CHN>(u / CHN);
                if (j * SUB / Geo::LN == q)
                    dma16v(c * (128 / FN) >= left ? kZeroChunk : l_b + on[j], m0 + Geo::CT + (w * Geo::LN + j) * 1024);
            }
        }
        // scales: T by wavefront 0, N by wavefront 1, a second KB of N's by wavefront 2
        if (q == SUB - 1) {
            if (w == 0) {
                if (l < Geo::TB * SPS / 16) dma16(pa + p_kt * pitch_a, 16 * l, m0 + Geo::ST);
            } else if (w == 1) {
                if (l < Geo::NB * SPS / 16) dma16(pb + p_kt * pitch_b, 16 * l, m0 + Geo::SN);
            } else if (Geo::NB * SPS > 1024 && w == 2) {
                dma16(pb + p_kt * pitch_b, 1024 + 16 * l, m0 + Geo::SN + 1024);
            }
            p_kt++;
        }
    };

    // ---- fragments ----
    // rows 32 apart share the swizzle
    uint32_t ft[SUB][FT == 8 ? 2 : 1], fn[SUB][FN == 8 ? 2 : 1];
#pragma unroll
    for (int s = 0; s < SUB; s++) {
        const int rn = 64 * wn + lr, rt = 32 * TI * wt + lr;
        if constexpr (FT == 4) {
            ft[s][0] = rt * Geo::RT + 16 * ((2 * s + lh) ^ swizzle<CHT>(rt));
        } else {
            ft[s][0] = rt * Geo::RT + 16 * ((4 * s + 2 * lh) ^ swizzle<CHT>(rt));
            ft[s][1] = rt * Geo::RT + 16 * ((4 * s + 2 * lh + 1) ^ swizzle<CHT>(rt));
        }
        if constexpr (FN == 4) {
            fn[s][0] = Geo::CT + rn * Geo::RN + 16 * ((2 * s + lh) ^ swizzle<CHN>(rn));
        } else {
            fn[s][0] = Geo::CT + rn * Geo::RN + 16 * ((4 * s + 2 * lh) ^ swizzle<CHN>(rn));
            fn[s][1] = Geo::CT + rn * Geo::RN + 16 * ((4 * s + 2 * lh + 1) ^ swizzle<CHN>(rn));
        }
    }
    const uint32_t st = Geo::ST + ((wt * 32 + lr) * 2 + lh) * Geo::TCH, sn = Geo::SN + ((wn * 32 + lr) * 2 + lh) * Geo::NCH;

    v16f acc[TI][2];
    int nv = 0, most = 0;   // blocks of 32 tokens in use: of this wavefront, of the fullest
    auto frag = [&](auto F, const uint8_t *s, const uint32_t *at, uint32_t off) __attribute__((always_inline)) -> v8i {
        constexpr int f = decltype(F)::v;
        v8i v = {0, 0, 0, 0, 0, 0, 0, 0};
        const uint4 a = *reinterpret_cast<const uint4 *>(s + at[0] + off);
        v[0] = (int)a.x; v[1] = (int)a.y; v[2] = (int)a.z; v[3] = (int)a.w;
        if constexpr (f == 8) {
            const uint4 b = *reinterpret_cast<const uint4 *>(s + at[1] + off);
            v[4] = (int)b.x; v[5] = (int)b.y; v[6] = (int)b.z; v[7] = (int)b.w;
        }
        return v;
    };
    // a lane's scale bytes of a stage (4, 8 or 16 of T; 2, 4 or 8 of N) as words
    auto chunk = [&](auto B, const uint8_t *s, uint32_t (&o)[4]) __attribute__((always_inline)) {
        constexpr int n = decltype(B)::v;
        if constexpr (n == 16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(s);
            o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
        } else if constexpr (n == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(s);
            o[0] = v.x; o[1] = v.y;
        } else if constexpr (n == 4) {
            o[0] = *reinterpret_cast<const uint32_t *>(s);
        } else {
            o[0] = *reinterpret_cast<const uint16_t *>(s);
        }
    };
    // Products of the stage in the ring at byte `so`, and a part of the next stage's loads with each step.  Blocks behind
    // the last row are multiplied too, whatever the ring holds there: a token's sums are its own, and theirs are not
    // written.  (Skipping them took two forms of this run, whose accumulators the compiler then moved back and forth.)
    auto compute = [&](uint32_t so) __attribute__((always_inline)) {
        const uint8_t *s = ring + so;
        uint32_t sa[4], sb[4];
        chunk(IC<Geo::TCH>{}, s + st, sa);
        chunk(IC<Geo::NCH>{}, s + sn, sb);
        constexpr int PRE = FT == 4 ? 2 : 1;   // steps whose fragments are held
        v8i n[PRE][2], a[PRE][TI];
        auto load = [&](int q) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; j++) n[q & (PRE - 1)][j] = frag(IC<FN>{}, s, fn[q], 32 * Geo::RN * j);
#pragma unroll
            for (int i = 0; i < TI; i++) a[q & (PRE - 1)][i] = frag(IC<FT>{}, s, ft[q], 32 * Geo::RT * i);
        };
        auto two = [&](auto Q, auto I) __attribute__((always_inline)) {
            // byte 4 d + o of a chunk is byte o of word d
            constexpr int q = decltype(Q)::v, i = decltype(I)::v, bt = i * U + q;
            constexpr int h = q & (PRE - 1);
            acc[i][0] = mma<q & 3, bt & 3>(n[h][0], a[h][i], acc[i][0], (int)sb[q >> 2], (int)sa[bt >> 2]);
            acc[i][1] = mma<(U + q) & 3, bt & 3>(n[h][1], a[h][i], acc[i][1], (int)sb[(U + q) >> 2], (int)sa[bt >> 2]);
        };
        // The same in bf16, eight values of each lane's block at a time.
        auto exact = [&](auto Q) __attribute__((always_inline)) {
            constexpr int q = decltype(Q)::v;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const v8bf n0 = to_bf16<FN>(n[0][0], e, sb[0], q), n1 = to_bf16<FN>(n[0][1], e, sb[0], U + q);
#pragma unroll
                for (int i = 0; i < TI; i++) {
                    const v8bf x = to_bf16<FT>(a[0][i], e, sa[0], i * U + q);
                    acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(n0, x, acc[i][0], 0, 0, 0);
                    acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(n1, x, acc[i][1], 0, 0, 0);
                }
            }
        };
        auto step = [&](auto Q) __attribute__((always_inline)) {
            constexpr int q = decltype(Q)::v;
            if constexpr (q < SUB) {
                // the next step's fragments (with MXFP8 tokens the bf16 products bound the step: read when it begins)
                if constexpr (FT == 4 && q + 1 < SUB) load(q + 1);
                if constexpr (FT == 8 && q > 0) load(q);
                issue(Q);
                if constexpr (FT == 4) {
                    two(Q, IC<0>{});
                    if constexpr (TI > 1) two(Q, IC<1>{});
                } else {
                    static_assert(FT == 4 || Geo::TCH <= 4, "a lane's scales in one word");
                    exact(Q);
                }
                asm volatile("" ::: "memory");   // no fragments further ahead: they would not fit the registers
            }
        };
        load(0);
        step(IC<0>{});
        step(IC<1>{});
        step(IC<2>{});
        step(IC<3>{});
    };
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TI; i++)
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
    };
    auto blocks_of = [&](const MxTile &T) __attribute__((always_inline)) {
        const int n = (T.row1 - T.row0 + 31) >> 5, left = n - TI * wt;
        most = n < TI ? n : TI;
        nv = left < 0 ? 0 : left < TI ? left : TI;
    };
    // The tile's outputs go through the ring stage that was multiplied last (`patch`), so that stores cover whole runs
    // of 64 or 128 bytes of a row: left as the lanes have them, 16-byte pieces of 32 rows, each piece was a write
    // request of its own and the L2 took 4 TB/s of them.  16-byte pieces of a staged row are swizzled against bank
    // conflicts.  The stores are non-temporal: kept in the L2, the outputs displaced the operands that other workgroups
    // were about to read (128 weight gradients of 1536 x 2048: 459 against 371 us).
    auto finish = [&](const MxTile &T, int ord, uint8_t *patch) __attribute__((always_inline)) {
        const int col = EPI == EPI_GATED ? Geo::NB / 2 * T.ct + 32 * wn : Geo::NB * T.ct + 64 * wn;   // of this wavefront
        const int row0 = T.row0 + 32 * TI * wt, tr = 32 * TI * wt;   // its tokens, and their place in the tile
        // opaque: offsets that follow from the lane, hoisted out of the tile loop, would hold registers in the product
        int l = threadIdx.x & 63;
        asm volatile("" : "+v"(l));
        const int lr = l & 31, lh = l >> 5;
        waitcnt<63, 0>();
        barrier();   // every wavefront is done with the stage
        if constexpr (EPI == EPI_BF16 || EPI == EPI_F32) {
            // a wavefront's own patch: 32 rows of 128 bytes, 64 columns of bf16 or 32 of f32
            uint8_t *mine = patch + w * 4096;
            constexpr int ESZ = EPI == EPI_BF16 ? 2 : 4, VEC = 16 / ESZ, NJ = EPI == EPI_BF16 ? 2 : 1;
            const bool vec = (p.ldc & (VEC - 1)) == 0;
            const int64_t base = WG ? (int64_t)T.g * p.M : 0;
#pragma unroll
            for (int i = 0; i < TI; i++) {
                if (i >= nv) break;
                const bool ok = WG || row_ok[WG ? 0 : ord][tr + 32 * i + lr];
#pragma unroll
                for (int j0 = 0; j0 < 2; j0 += NJ) {
#pragma unroll
                    for (int jj = 0; jj < NJ; jj++) {
                        float v[16];
#pragma unroll
                        for (int e = 0; e < 16; e++) v[e] = ok ? acc[i][j0 + jj][e] : 0.0f;
                        if constexpr (EPI == EPI_BF16) {
                            u32v4 o[2];
                            bf16_pieces(v, o);
#pragma unroll
                            for (int q = 0; q < 2; q++)
                                *reinterpret_cast<u32v4 *>(mine + lr * 128 + 16 * ((4 * jj + 2 * q + lh) ^ (lr & 7))) = o[q];
                        } else {
#pragma unroll
                            for (int q = 0; q < 4; q++)
                                *reinterpret_cast<u32v4 *>(mine + lr * 128 + 16 * ((2 * q + lh) ^ (lr & 7))) =
                                    (u32v4){__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                            __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])};
                        }
                    }
                    __builtin_amdgcn_wave_barrier();   // the patch is this wavefront's
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const int row = 8 * q + (l >> 3), ch = l & 7, r = row0 + 32 * i + row;
                        const int c = col + 32 * j0 + VEC * ch;
                        const u32v4 v = *reinterpret_cast<const u32v4 *>(mine + row * 128 + 16 * (ch ^ (row & 7)));
                        if (r >= T.row1 || c >= p.N) continue;
                        char *dst = reinterpret_cast<char *>(p.c) + ((base + r) * p.ldc + c) * ESZ;
                        if (vec && c + VEC <= p.N) {
                            st4w<true>(dst, v);
                        } else {
#pragma unroll
                            for (int e = 0; e < VEC; e++) {
                                if (c + e >= p.N) break;
                                if (ESZ == 2) reinterpret_cast<uint16_t *>(dst)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
                                else reinterpret_cast<uint32_t *>(dst)[e] = v[e & 3];
                            }
                        }
                    }
                    __builtin_amdgcn_wave_barrier();
                }
            }
        } else if constexpr (EPI == EPI_GATED) {
            // a patch of the WN wavefronts that share 32 rows, for their columns: codes of gate, up and h (32 WN bytes of a
            // row each; MXFP4 half of it), then the WN scales of a row of each; two patches in turn
            constexpr int WN = Geo::WN, CH = 2 * WN, ARR = 1024 * WN, SCL = 3 * ARR, HALF = SCL + 3 * 32 * WN;
            static_assert((TI > 1 ? 4 : 2) * HALF <= Geo::SLOT, "two patches for each run of tokens in a ring stage");
            const int t = 64 * wn + l, row = t / CH, ch = t % CH, c = 32 * WN * T.ct + 16 * ch;   // in the stores
            const int blocks = p.I / 32;
#pragma unroll
            for (int i = 0; i < TI; i++) {
                if (i >= most) break;   // the same for the whole workgroup, for the barriers
                uint8_t *half = patch + (2 * (i & 1) + wt) * HALF;
                const bool ok = row_ok[ord][tr + 32 * i + lr];
                const float rw = row_w[ord][tr + 32 * i + lr];
                float v[2][16], h[16];
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int e = 0; e < 16; e++) v[j][e] = acc[i][j][e];
                if (!__all(ok)) {
#pragma unroll
                    for (int j = 0; j < 2; j++)
#pragma unroll
                        for (int e = 0; e < 16; e++) v[j][e] = ok ? v[j][e] : 0.0f;
                }
                const int sw8 = 16 * ((2 * wn + lh) ^ swizzle<CH>(lr));
                if (p.ckpt_codes) {
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        u32v4 o;
                        const uint32_t k = mx8_block(v[j], o);
                        *reinterpret_cast<u32v4 *>(half + j * ARR + lr * 32 * WN + sw8) = o;
                        if (lh == 0) half[SCL + (32 * j + lr) * WN + wn] = (uint8_t)k;
                    }
                }
                {
                    float s[16], rest[16];
                    sigmoid<true>(v[0], s, rest);   // h is rounded once, to 3 bits or to bf16, from f32
#pragma unroll
                    for (int e = 0; e < 16; e++) h[e] = rw * (v[0][e] * s[e] * v[1][e]);
                }
                if (p.h_fmt >= 0) {
                    uint32_t k;
                    if (p.h_fmt == BSP_FMT_MXFP8) {
                        u32v4 o;
                        k = mx8_block(h, o);
                        *reinterpret_cast<u32v4 *>(half + 2 * ARR + lr * 32 * WN + sw8) = o;
                    } else {
                        uint2 o;
                        k = mx4_block(h, o);
                        *reinterpret_cast<uint2 *>(half + 2 * ARR + lr * 16 * WN + sw8 / 2) = o;
                    }
                    if (lh == 0) half[SCL + (64 + lr) * WN + wn] = (uint8_t)k;
                }
                waitcnt<63, 0>();
                barrier();
                const int64_t r = row0 + 32 * i + row;
                const int sw = 16 * (ch ^ swizzle<CH>(row));
                if (r < T.row1 && c < p.I) {
                    if (p.ckpt_codes) {
#pragma unroll
                        for (int j = 0; j < 2; j++)
                            st4w<true>(p.ckpt_codes + r * 2 * p.I + j * p.I + c,
                                        *reinterpret_cast<const u32v4 *>(half + j * ARR + row * 32 * WN + sw));
                    }
                    if (p.h_fmt == BSP_FMT_MXFP8)
                        st4w<true>(p.h_codes + r * p.I + c,
                                    *reinterpret_cast<const u32v4 *>(half + 2 * ARR + row * 32 * WN + sw));
                    else if (p.h_fmt == BSP_FMT_MXFP4)
                        st2<true>(p.h_codes + (r * p.I + c) / 2,
                                   *reinterpret_cast<const uint2 *>(half + 2 * ARR + row * 16 * WN + sw / 2));
                }
                // scales: a row's WN of each
                if (t < 96) {
                    const int a = t >> 5, sr = t & 31;
                    const int64_t rs = row0 + 32 * i + sr;
                    uint32_t k = 0;
                    __builtin_memcpy(&k, half + SCL + t * WN, WN);
                    if (rs < T.row1 && (a < 2 ? p.ckpt_codes != nullptr : p.h_fmt >= 0)) {
                        uint8_t *d = a < 2 ? p.ckpt_scales + rs * 2 * blocks + a * blocks : p.h_scales + rs * blocks;
                        d += WN * T.ct;
                        const int some = blocks - WN * T.ct;
                        if (some >= WN) {
                            __builtin_memcpy(d, &k, WN);
                        } else {
                            for (int e = 0; e < some; e++) d[e] = (uint8_t)(k >> (8 * e));
                        }
                    }
                }
                if (p.h) {   // bf16 h: 64 WN bytes of a row, in the same patch
                    constexpr int HC = 4 * WN;
                    waitcnt<63, 0>();
                    barrier();
                    u32v4 o[2];
                    bf16_pieces(h, o);
#pragma unroll
                    for (int q = 0; q < 2; q++)
                        *reinterpret_cast<u32v4 *>(half + lr * 64 * WN + 16 * ((4 * wn + 2 * q + lh) ^ (lr & (HC - 1)))) = o[q];
                    waitcnt<63, 0>();
                    barrier();
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        const int hr = 16 * q + t / HC, hc = t % HC;
                        const int64_t rr = row0 + 32 * i + hr;
                        if (rr < T.row1 && 32 * WN * T.ct + 8 * hc < p.I)
                            st4w<true>(p.h + rr * p.I + 32 * WN * T.ct + 8 * hc,
                                        *reinterpret_cast<const u32v4 *>(half + hr * 64 * WN + 16 * (hc ^ (hr & (HC - 1)))));
                    }
                }
            }
        } else {
            // a wavefront's own patch: three arrays of 32 rows of 64 bytes (32 columns of bf16)
            uint8_t *mine = patch + w * 6144;
            static_assert(Geo::NW * 6144 <= Geo::SLOT, "a patch for each wavefront in a ring stage");
            // the next block's checkpoint is on its way before this one's stores
            Ckpt k = load_ckpt(p, row0 + lr < T.row1 ? row0 + lr : -1, col, lh);
            float dw = 0.0f;
#pragma unroll
            for (int b = 0; b < 2 * TI; b++) {
                const int i = b >> 1, j = b & 1, c = col + 32 * j;
                if (i >= nv) break;
                const Ckpt now = k;
                asm volatile("" ::: "memory");
                if (b + 1 < 2 * TI) {
                    const int rn = row0 + 32 * ((b + 1) >> 1) + lr;
                    k = load_ckpt(p, rn < T.row1 ? rn : -1, col + 32 * ((b + 1) & 1), lh);
                }
                uint32_t v[3][8];
                const float part = gated_backward(now, acc[i][j], row_ok[ord][tr + 32 * i + lr], row_w[ord][tr + 32 * i + lr],
                                                  v[0], v[1], v[2]);
                dw = (j == 0 ? 0.0f : dw) + (c < p.I ? part : 0.0f);
#pragma unroll
                for (int a = 0; a < 3; a++) {
                    u32v4 o[2];
                    bf16_pieces(v[a], o);
#pragma unroll
                    for (int q = 0; q < 2; q++)
                        *reinterpret_cast<u32v4 *>(mine + a * 2048 + lr * 64 + 16 * ((2 * q + lh) ^ ((lr >> 2) & 3))) = o[q];
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int a = 0; a < 3; a++) {
                    if (a == 2 && !p.h) break;
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        const int row = 16 * q + (l >> 2), ch = l & 3;
                        const int64_t r = row0 + 32 * i + row;
                        const u32v4 o = *reinterpret_cast<const u32v4 *>(mine + a * 2048 + row * 64 +
                                                                         16 * (ch ^ ((row >> 2) & 3)));
                        if (r < T.row1 && c < p.I)
                            st4w<true>((a == 2 ? p.h + r * p.I : p.dh13 + (2 * r + a) * p.I) + c + 8 * ch, o);
                    }
                }
                __builtin_amdgcn_wave_barrier();
                if (j == 1 && p.part && col < p.I) {
                    const float sum = both_sum(dw);
                    const int r = row0 + 32 * i + lr;
                    if (r < T.row1 && lh == 0) p.part[(int64_t)r * p.parts + col / 64] = sum;
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // ---- tiles ----
    int queued = 0, landed = 0;           // stages loaded and not yet multiplied, and those known to be there
    uint32_t rd = 0, wr = 0, done = 0;    // ring: next stage to multiply, next to fill, multiplied last
    auto next = [&](uint32_t at) __attribute__((always_inline)) -> uint32_t {
        return at + Geo::SLOT == NS * Geo::SLOT ? 0 : at + Geo::SLOT;
    };
    if (more) {
        E = entry(q_lin);
        look_ahead();
    }
    for (int s = 0; s < NS - 1; s++) {
        begin(wr);
        if (!loading) break;
        issue(IC<0>{});
        issue(IC<1>{});
        if constexpr (SUB > 2) {
            issue(IC<2>{});
            issue(IC<3>{});
        }
        queued++;
        wr = next(wr);
    }
    waitcnt<63, 0>();
    barrier();   // the first tile's info
    for (int ord = 0; queued > 0; ord = (ord + 1) & 3) {
        MxTile T;
        T.g = __builtin_amdgcn_readfirstlane(info[ord][0]);
        T.row0 = __builtin_amdgcn_readfirstlane(info[ord][1]);
        T.row1 = __builtin_amdgcn_readfirstlane(info[ord][2]);
        T.ct = __builtin_amdgcn_readfirstlane(info[ord][3]);
        T.nk = __builtin_amdgcn_readfirstlane(info[ord][4]);
        blocks_of(T);
        clear();
        for (int kt = 0; kt < T.nk; kt++) {
            // the oldest stage has landed once at most the queued - 1 behind it are on their way
            if (landed > 0) {
                landed--;
                waitcnt<63, 0>();   // what `begin` and `finish` left in LDS
            } else {
                wait_stage_w<Geo::OPS>(queued - 1, w < Geo::SW);
            }
            barrier();   // for every wavefront; and the ring stage multiplied last is free
            begin(wr);
            compute(rd);   // a wavefront without rows too: it loads its share
            if (loading) {
                queued++;
                wr = next(wr);
            }
            queued--;
            done = rd;
            rd = next(rd);
        }
        // The next tile's first stages, under way since the last products, have landed before this tile's stores join
        // the queue: its first step then waits for none of them.
        waitcnt<0, 0>();
        landed = queued;
        finish(T, ord, ring + done);
    }
    if constexpr (WG) {
        // gradients of groups without tokens are zeros: the last by size, if they are listed so
        clear();
        const int n = last > first ? (last - first + stride - 1) / stride : 0;
        for (int k = n - 1; k >= 0; k--) {
            const int lin = first + k * stride;
            const MxTile T = decode(lin, entry(lin));
            if (T.nk > 0 && p.G <= 4096) break;
            if (T.nk > 0) continue;
            blocks_of(T);
            finish(T, 0, ring);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
static int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Rows of a row tile: 64 for groups of few rows, where the larger tile's products are mostly of rows that are not there.
// us of 64 / 128, by rows of each of 128 groups of 1536 x 2048 (captured calls; the device alone knows how even the
// groups are):
//                          80           96         112         128         160         192
//   MXFP4  product       80 / 75     84 / 83     89 / 85     97 / 86    111 / 96    126 / 100
//          gated         82 / 82     86 / 93     91 / 95     99 / 96    116 / 109   131 / 114
//          backward      72 / 71     75 / 87     84 / 91     90 / 92    101 / 99    116 / 105
//   MXFP8  product      124 / 137   137 / 151   146 / 158   163 / 165   191 / 181   226 / 194
//   tokens gated        128 / 140   143 / 166   152 / 168   167 / 173   200 / 198   238 / 205
//          backward      94 / 97    100 / 128   109 / 130   122 / 131   135 / 136   158 / 147
// and with 143 rows of each of 257 groups of 4096 x 7168, gated, 1542 / 1317 (MXFP4) and 3241 / 3071 (MXFP8 x MXFP4).
static int tile_rows(int fmt, bool wgrad, bool gated, int64_t M, int64_t G) {
    return wgrad || M / G >= (fmt == BSP_FMT_MXFP4 && !gated ? 80 : 128) ? 128 : 64;
}

// Workspace: the d_row_weights parts, then the tiled form's tables and planes, each on a 256-byte boundary.
struct MxLayout {
    int64_t part, tiles, a_plane, b_plane, total;
    int64_t ntm, ntn, stages;
    int tb;
};
// gated: the gated block or its backward pass.
static MxLayout layout(int fmt, bool wgrad, bool gated, int64_t M, int64_t N, int64_t K, int64_t G, int64_t parts,
                       bool few) {
    MxLayout L = {};
    L.tb = tile_rows(fmt, wgrad, gated, M, G);
    const int64_t bk = fmt == BSP_FMT_MXFP4 ? 256 : 128, sps = bk / 32, nb = L.tb == 128 ? 256 : 128;
    L.tiles = L.a_plane = L.b_plane = L.total = up(M * parts * 4, 256);
    L.ntn = (N + nb - 1) / nb;
    if (few) return L;
    if (wgrad) {
        L.ntm = (M + 127) / 128;
        L.stages = K / bk + G;   // of all groups: each has at most one that is not full
        L.a_plane = L.tiles + up(8 * G * 16 + 8 * 4, 256);
        L.b_plane = L.a_plane + up(L.stages * L.ntm * 128 * sps, 256);
        L.total = L.b_plane + up(L.stages * L.ntn * nb * sps, 256);
    } else {
        L.ntm = M / L.tb + (G < M ? G : M);   // as many as there can be
        L.stages = (K + bk - 1) / bk;
        L.a_plane = L.tiles + up(L.ntm * 16 + 4, 256);
        L.b_plane = L.a_plane + up(L.ntm * L.stages * L.tb * sps, 256);
        L.total = L.b_plane + up(G * L.ntn * L.stages * nb * sps, 256);
    }
    return L;
}
// Up to 64 rows the form without staging, which needs no workspace and one launch.  us of it / of the tiles, by rows of
// 128 groups of 1536 x 2048 (captured calls):
//                          1          16          32          48          64          96         128
//   MXFP4, gated       12 / 18     16 / 19     20 / 21     22 / 22     26 / 24     30 / 30     35 / 32
//   MXFP8 x MXFP4      17 / 26     20 / 26     25 / 30     28 / 31     33 / 32     40 / 39     47 / 43
//   MXFP8              18 / 26     25 / 27     32 / 30     37 / 34     48 / 38     58 / 50     69 / 55
// (products as the gated block; the backward pass 21 / 24, 25 / 30 and 31 / 32 at 64 rows, 27 / 28, 31 / 36 and 44 / 38
// at 128).  From about 50 rows, of MXFP8 weights from 24, the tiles are faster where memory for them is at hand; the
// bound is one for all, so that a serving loop's calls need no workspace.
static bool few_rows(int mode, int64_t M, int tile) {
    return mode != BSP_GEMM_WGRAD && (tile == 32 || (tile == 0 && M <= BSP_FEW_ROWS));
}

int64_t mx_gemm_workspace_bytes(int fmt, int mode, int64_t M, int64_t N, int64_t K, int64_t G, int tile) {
    return layout(fmt, mode == BSP_GEMM_WGRAD, false, M, N, K, G, 0, few_rows(mode, M, tile)).total;
}
int64_t mx_gated_workspace_bytes(int fmt, int64_t R, int64_t I, int64_t K, int64_t G, int tile) {
    return layout(fmt, false, true, R, 2 * I, K, G, 0, few_rows(BSP_GEMM_FPROP, R, tile)).total;
}
int64_t mx_gated_bwd_workspace_bytes(int fmt, int64_t R, int64_t I, int64_t K, int64_t G, bool sums, int tile) {
    return layout(fmt, false, true, R, I, K, G, sums ? (I + 63) / 64 : 0, few_rows(BSP_GEMM_FPROP, R, tile)).total;
}

template <int FT, int FN, int EPI>
static void launch_few(const MxArgs &p, hipStream_t s) {
    const int cols = EPI == EPI_GATED ? 32 : 64, n = EPI == EPI_GATED ? p.I : p.N;
    // every group with rows has a tile, and every 32 rows at most one more
    const int64_t tiles = (int64_t)p.M / 32 + (p.G < p.M ? p.G : p.M);
    k_mx_few<FT, FN, EPI><<<dim3((unsigned)((n + cols - 1) / cols), (unsigned)tiles), 512, 0, s>>>(p);
}

template <int FT, int FN, int EPI, bool WG, int TB>
static void launch_tiles(MxArgs p, const MxLayout &L, uint8_t *ws, hipStream_t s) {
    using Geo = MxGeo<FT, FN, TB>;
    p.ntm = (int32_t)L.ntm; p.ntn = (int32_t)L.ntn; p.stages = (int32_t)L.stages;
    p.a_plane = ws + L.a_plane;
    p.b_plane = ws + L.b_plane;
    p.tiles = reinterpret_cast<i32v4 *>(ws + L.tiles);
    p.count = reinterpret_cast<int32_t *>(p.tiles + (WG ? 8 * (int64_t)p.G : L.ntm));
    if constexpr (WG) {
        const int64_t rows = 128 * L.ntm + 256 * L.ntn;
        k_mx_prep_wgrad<FT, FN><<<dim3((unsigned)(L.stages + 1), (unsigned)((rows + kWgradRows - 1) / kWgradRows)), 256, 0, s>>>(
            p);
    } else {
        k_mx_prep<FT, FN, EPI, TB><<<(unsigned)(L.ntm + p.G * ((L.ntn * Geo::NB + 255) / 256)), 256, 0, s>>>(p);
    }
    // persistent workgroups to an XCD, which has 32 compute units
    const int64_t per_xcd = WG ? p.G * L.ntm * L.ntn : (L.ntm * L.ntn + 7) / 8, most = Geo::BIG ? 32 : 64;
    k_mx_tile<FT, FN, EPI, WG, TB><<<(unsigned)(8 * (per_xcd < most ? per_xcd : most)), Geo::NT, 0, s>>>(p);
}

template <int FT, int FN, int EPI>
static void launch_form(const MxArgs &p, bool few, const MxLayout &L, uint8_t *ws, hipStream_t s) {
    if (few) launch_few<FT, FN, EPI>(p, s);
    else if (L.tb == 128) launch_tiles<FT, FN, EPI, false, 128>(p, L, ws, s);
    else launch_tiles<FT, FN, EPI, false, 64>(p, L, ws, s);
}

template <int EPI>
static void launch_gemm_epi(int fmt, bool wgrad, const MxArgs &p, bool few, const MxLayout &L, uint8_t *ws,
                            hipStream_t s) {
    if (fmt == BSP_FMT_MXFP4) {
        if (wgrad) launch_tiles<4, 4, EPI, true, 128>(p, L, ws, s);
        else launch_form<4, 4, EPI>(p, few, L, ws, s);
    } else {
        if (wgrad) launch_tiles<8, 4, EPI, true, 128>(p, L, ws, s);
        else launch_form<8, 4, EPI>(p, few, L, ws, s);
    }
}

static MxArgs operands(const uint8_t *a_codes, const uint8_t *a_scales, const int32_t *gather, int64_t a_rows,
                       const int64_t *off, int64_t G, int64_t M, int64_t N, int64_t K, const uint8_t *b_codes,
                       const uint8_t *b_scales) {
    MxArgs p = {};
    p.a_codes = a_codes; p.a_scales = a_scales; p.b_codes = b_codes; p.b_scales = b_scales;
    p.gather = gather; p.off = off;
    p.G = (int32_t)G; p.M = (int32_t)M; p.N = (int32_t)N; p.K = (int32_t)K; p.a_rows = (int32_t)a_rows;
    return p;
}

hipError_t launch_mx_gemm(int fmt, int mode, const uint8_t *a_codes, const uint8_t *a_scales, const int32_t *gather,
                          int64_t a_rows, const int64_t *off, int64_t G, int64_t M, int64_t N, int64_t K,
                          const uint8_t *b_codes, const uint8_t *b_scales, void *c, int c_dtype, int64_t ldc,
                          void *workspace, int tile, hipStream_t s) {
    MxArgs p = operands(a_codes, a_scales, gather, a_rows, off, G, M, N, K, b_codes, b_scales);
    p.c = c; p.ldc = ldc;
    const bool wgrad = mode == BSP_GEMM_WGRAD, few = few_rows(mode, M, tile);
    const MxLayout L = layout(fmt, wgrad, false, M, N, K, G, 0, few);
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    if (c_dtype == BSP_DTYPE_BF16) launch_gemm_epi<EPI_BF16>(fmt, wgrad, p, few, L, ws, s);
    else launch_gemm_epi<EPI_F32>(fmt, wgrad, p, few, L, ws, s);
    return hipGetLastError();
}

template <int EPI>
static hipError_t launch_gated_epi(int fmt, const MxArgs &p, bool few, const MxLayout &L, uint8_t *ws, hipStream_t s) {
    if (fmt == BSP_FMT_MXFP4) launch_form<4, 4, EPI>(p, few, L, ws, s);
    else if (fmt == BSP_FMT_MXFP8_MXFP4) launch_form<8, 4, EPI>(p, few, L, ws, s);
    else launch_form<8, 8, EPI>(p, few, L, ws, s);
    return hipGetLastError();
}

hipError_t launch_moe_gated(int fmt, const uint8_t *a_codes, const uint8_t *a_scales, const int32_t *gather,
                            int64_t a_rows, const int64_t *off, int64_t G, int64_t R, int64_t I, int64_t K,
                            const uint8_t *b_codes, const uint8_t *b_scales, const float *row_weights, uint16_t *h,
                            int h_fmt, uint8_t *h_codes, uint8_t *h_scales, uint8_t *ckpt_codes, uint8_t *ckpt_scales,
                            void *workspace, int tile, hipStream_t s) {
    MxArgs p = operands(a_codes, a_scales, gather, a_rows, off, G, R, 2 * I, K, b_codes, b_scales);
    p.row_weights = row_weights; p.h = h; p.h_fmt = h_fmt; p.h_codes = h_codes; p.h_scales = h_scales;
    p.ckpt_codes = ckpt_codes; p.ckpt_scales = ckpt_scales; p.I = (int32_t)I;
    const bool few = few_rows(BSP_GEMM_FPROP, R, tile);
    return launch_gated_epi<EPI_GATED>(fmt, p, few, layout(fmt, false, true, R, 2 * I, K, G, 0, few),
                                       reinterpret_cast<uint8_t *>(workspace), s);
}

hipError_t launch_moe_gated_backward(int fmt, const uint8_t *dy_codes, const uint8_t *dy_scales, const int32_t *gather,
                                     int64_t dy_rows, const int64_t *off, int64_t G, int64_t R, int64_t I, int64_t K,
                                     const uint8_t *b_codes, const uint8_t *b_scales, const uint8_t *ckpt_codes,
                                     const uint8_t *ckpt_scales, const float *row_weights, uint16_t *dh13, uint16_t *h,
                                     float *d_row_weights, void *workspace, int tile, hipStream_t s) {
    MxArgs p = operands(dy_codes, dy_scales, gather, dy_rows, off, G, R, I, K, b_codes, b_scales);
    p.row_weights = row_weights; p.h = h; p.dh13 = dh13; p.I = (int32_t)I;
    p.ckpt_codes = const_cast<uint8_t *>(ckpt_codes); p.ckpt_scales = const_cast<uint8_t *>(ckpt_scales);
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    const int64_t parts = d_row_weights ? (I + 63) / 64 : 0;
    const bool few = few_rows(BSP_GEMM_FPROP, R, tile);
    const MxLayout L = layout(fmt, false, true, R, I, K, G, parts, few);
    p.parts = (int32_t)parts;
    p.part = d_row_weights ? reinterpret_cast<float *>(ws) : nullptr;
    const hipError_t e = launch_gated_epi<EPI_GATED_BWD>(fmt, p, few, L, ws, s);
    if (e != hipSuccess || !d_row_weights) return e;
    k_row_sums<<<grid_of((R + 255) / 256), 256, 0, s>>>(p.part, p.parts, (int)R, off, (int)G, d_row_weights);
    return hipGetLastError();
}

}  // namespace bsp
