// bsp_checkpoint.hip -- SwiGLU whose input is kept for the backward pass as
// MXFP8, and its gradient from that 8-bit checkpoint.
//
//   forward:  h = w silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g));
//             checkpoint = MXFP8([g u]), blocks of 32 along the row
//   backward: du = w dh g s,  dg = w dh u s (1 + g (1 - s)),
//             dw = sum_i dh_i g_i s_i u_i,  h again
// Both are bound by HBM: per h element the forward moves 2 s + 2 + 2.06 bytes
// (s = 4 or 2 for f32 or bf16 h13) and the backward 3 s + 2.06 + 2, each input
// read and each output written once.
//
// A lane takes 16 bytes of h13 (VE = 8 bf16 or 4 f32 values) of the gate and
// the same of the up half, so every load and store of a wavefront is one
// contiguous run, and a block of 32 values lies on 32 / VE neighbouring lanes:
// its maximum is two or three DPP steps.
//
// Cache policy, which decides between 5.1 and 6.7 TB/s here.  Inputs are loaded
// nontemporally (read once; forward 65536 x 768 bf16 74.6 -> 62 us), and of the
// outputs the larger part is stored nontemporally: dh13, and the checkpoint,
// which nobody reads before the backward pass.  h, the next product's operand,
// stays in the 256 MiB last-level cache where it fits there beside what that
// product reads, and is nontemporal past 128 MiB, where it would push itself
// out.  Backward 65536 x 768 (h 96 MiB): all cached 99.6 us, all nontemporal 86,
// h cached 76 (6.6 TB/s); 36864 x 2048 (h 144 MiB): 138, 130, 135.
// Keeping more than one piece per lane in flight changed nothing for bf16 and
// cost f32 3 to 10 %.
// Rows from n_rows on are not loaded: with 20000 of 65536 x 768 unused the
// forward takes 57.6 us instead of 61.3 and the backward 67.6 instead of 75.7;
// with all in use the condition costs 0.5 %.
#include <type_traits>

#include "bsp_moe.hpp"

namespace bsp {

namespace {

template <int CTRL>
__device__ __forceinline__ float lane_perm(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

template <typename T>
constexpr int kVE = 16 / (int)sizeof(T);

// 16 bytes of T as f32.
__device__ __forceinline__ void ld(const float *p, float (&v)[4]) {
    const u32v4 x = ld4w<true>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __uint_as_float(x[i]);
}
__device__ __forceinline__ void ld(const uint16_t *p, float (&v)[8]) { ld8<true>(p, v); }
__device__ __forceinline__ void st_nt(float *p, const float (&v)[4]) {
    st4w<true>(p, (u32v4){__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
}
__device__ __forceinline__ void st_nt(uint16_t *p, const float (&v)[8]) { st8<true>(p, v); }
// h: bf16
template <bool NT>
__device__ __forceinline__ void st_h(uint16_t *p, const float (&v)[4]) {
    st2<NT>(p, make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3])));
}
template <bool NT>
__device__ __forceinline__ void st_h(uint16_t *p, const float (&v)[8]) { st8<NT>(p, v); }
constexpr int64_t kCachedH = 128ll << 20;   // bytes of h kept in the last-level cache

// The E4M3 codes of VE values.
template <int VE>
struct Codes {
    uint32_t q[VE / 4];
};
template <bool NT>
__device__ __forceinline__ void st_codes(uint8_t *p, const Codes<8> &c) { st2<NT>(p, make_uint2(c.q[0], c.q[1])); }
template <bool NT>
__device__ __forceinline__ void st_codes(uint8_t *p, const Codes<4> &c) {
    if (NT) __builtin_nontemporal_store(c.q[0], reinterpret_cast<uint32_t *>(p));
    else *reinterpret_cast<uint32_t *>(p) = c.q[0];
}
__device__ __forceinline__ void ld_codes(const uint8_t *p, Codes<8> &c) {
    const uint2 v = ld2<true>(p);
    c.q[0] = v.x;
    c.q[1] = v.y;
}
__device__ __forceinline__ void ld_codes(const uint8_t *p, Codes<4> &c) {
    c.q[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(p));
}

// MXFP8 of a block held by 32 / VE neighbouring lanes: this lane's codes;
// returns the scale code.
template <int VE>
__device__ __forceinline__ uint32_t mx_block(const float (&v)[VE], Codes<VE> &c) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < VE; i++) a = fmaxf(a, fabsf(v[i]));
    a = fmaxf(a, lane_perm<0xB1>(a));                 // lanes 1 0 3 2
    a = fmaxf(a, lane_perm<0x4E>(a));                 // lanes 2 3 0 1
    if (VE == 4) a = fmaxf(a, lane_perm<0x141>(a));   // lanes 7 .. 0 of each eight
    const int k = mx_block_exponent(a);
    const float inv = exp2i(-k);
#pragma unroll
    for (int i = 0; i < VE; i += 4) c.q[i / 4] = e4m3x4_hw(v[i] * inv, v[i + 1] * inv, v[i + 2] * inv, v[i + 3] * inv);
    return (uint32_t)(k + 127);
}

// The values of VE codes; sc: the block's scale code.
template <int VE>
__device__ __forceinline__ void mx_values(const Codes<VE> &c, uint32_t sc, float (&v)[VE]) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(sc ? sc << 23 : 0x00400000u);   // 2^-127 is a subnormal f32
#pragma unroll
    for (int i = 0; i < VE; i += 4) {
        const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.q[i / 4], false);
        const f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.q[i / 4], true);
        v[i] = lo.x * s;
        v[i + 1] = lo.y * s;
        v[i + 2] = hi.x * s;
        v[i + 3] = hi.y * s;
    }
}

// s = 1 / (1 + e), e = exp(-z), and (FULL) c = 1 - s = e s, of VE values.
// FULL, for f32 results: e = 2^t (1 + d), t = -z log2(e) rounded and d what the
// rounding left out; without d the error of e grows with |z| (2.8 units of 2^-24
// at 4, 60 at 80).  With it s is within 6 + 0.05 |z| units and c, which 1 - s
// would cancel, within 10 + 0.1 |z|.  The forward's h is rounded to bf16 and does
// without.  Past |z| = 87 2^t, the reciprocal (V_RCP_F32 flushes results below
// 2^-126) and d run out of range; a wavefront that has such a value takes exp(z)
// for s there, scaled by 2^64 until the end: subnormal from -87.3, 0 below -104.
template <bool FULL, int VE>
__device__ __forceinline__ void sigmoid(const float (&z)[VE], float (&s)[VE], float (&c)[VE]) {
    constexpr float L2E = 1.44269504088896341f, LN2 = 0.693147180559945309f, FAR = 87.0f;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < VE; i++) {
        const float t = z[i] * -L2E;
        float e = __builtin_amdgcn_exp2f(t);
        if (FULL) e = fmaf(e, fmaf(-t, LN2, -z[i]), e);
        s[i] = __builtin_amdgcn_rcpf(1.0f + e);
        c[i] = e * s[i];
        top = fmaxf(top, fabsf(z[i]));
    }
    if (__any(top > FAR)) {
#pragma unroll
        for (int i = 0; i < VE; i++) {
            const float x = fmaxf(z[i], -110.0f), t = x * L2E;
            const float e = __builtin_amdgcn_exp2f(t + 64.0f);
            if (z[i] < -FAR) {
                s[i] = fmaf(e, fmaf(-t, LN2, x), e) * 0x1p-64f;
                c[i] = 1.0f;
            } else if (z[i] > FAR) {
                s[i] = 1.0f;
                c[i] = 0.0f;
            }
        }
    }
}

// Sum over LPR neighbouring lanes, the same bits on each.
template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

}  // namespace

// LPR lanes to a row.
template <typename T, int LPR, bool HNT>
__global__ __launch_bounds__(256, 8) void k_swiglu_ckpt(const T *__restrict__ h13, int64_t R, int64_t I,
                                                     const float *__restrict__ row_weights,
                                                     const int64_t *__restrict__ n_rows, uint16_t *__restrict__ h_out,
                                                     uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                     uint8_t *__restrict__ ckpt_codes,
                                                     uint8_t *__restrict__ ckpt_scales) {
    constexpr int VE = kVE<T>;
    const int lane = threadIdx.x & (LPR - 1);
    const int64_t r = grid_index() * (256 / LPR) + threadIdx.x / LPR;
    if (r >= R) return;
    const bool used = !n_rows || r < *n_rows;
    const float w = used && row_weights ? row_weights[r] : 1.0f;
    const T *gp = h13 + r * 2 * I;
    for (int64_t c = lane * VE; c < I; c += LPR * VE) {
        float g[VE], u[VE], h[VE];
        if (used) {
            ld(gp + c, g);
            ld(gp + I + c, u);
        } else {
#pragma unroll
            for (int i = 0; i < VE; i++) g[i] = u[i] = 0.0f;
        }
        const int64_t at = r * 2 * I + c;
        Codes<VE> qg, qu;
        const uint32_t sg = mx_block<VE>(g, qg), su = mx_block<VE>(u, qu);
        st_codes<true>(ckpt_codes + at, qg);
        st_codes<true>(ckpt_codes + at + I, qu);
        if ((c & 31) == 0) {
            ckpt_scales[at / 32] = (uint8_t)sg;
            ckpt_scales[(at + I) / 32] = (uint8_t)su;
        }
        float sig[VE], rest[VE];
        sigmoid<false>(g, sig, rest);
#pragma unroll
        for (int i = 0; i < VE; i++) h[i] = w * (g[i] * sig[i] * u[i]);
        if (h_out) st_h<HNT>(h_out + r * I + c, h);
        if (codes) {
#pragma unroll
            for (int i = 0; i < VE; i++) h[i] = __uint_as_float(bf16x2(0.0f, h[i]) & 0xFFFF0000u);
            Codes<VE> q;
            const uint32_t s = mx_block<VE>(h, q);
            st_codes<false>(codes + r * I + c, q);
            if ((c & 31) == 0) scales[(r * I + c) / 32] = (uint8_t)s;
        }
    }
}

template <typename T, int LPR, bool HNT>
__global__ __launch_bounds__(256, 8) void k_swiglu_ckpt_bwd(const T *__restrict__ dh, int64_t R, int64_t I,
                                                         const uint8_t *__restrict__ ckpt_codes,
                                                         const uint8_t *__restrict__ ckpt_scales,
                                                         const float *__restrict__ row_weights,
                                                         const int64_t *__restrict__ n_rows, T *__restrict__ dh13,
                                                         uint16_t *__restrict__ h_out,
                                                         float *__restrict__ d_row_weights) {
    constexpr int VE = kVE<T>;
    const int lane = threadIdx.x & (LPR - 1);
    const int64_t r = grid_index() * (256 / LPR) + threadIdx.x / LPR;
    if (r >= R) return;
    const bool used = !n_rows || r < *n_rows;
    const float w = used && row_weights ? row_weights[r] : 1.0f;
    float dw = 0.0f;
    for (int64_t c = lane * VE; c < I; c += LPR * VE) {
        const int64_t at = r * 2 * I + c;
        float d[VE], g[VE], u[VE], dg[VE], du[VE], h[VE];
        if (used) {
            Codes<VE> qg, qu;
            ld(dh + r * I + c, d);
            ld_codes(ckpt_codes + at, qg);
            ld_codes(ckpt_codes + at + I, qu);
            mx_values<VE>(qg, ckpt_scales[at / 32], g);
            mx_values<VE>(qu, ckpt_scales[(at + I) / 32], u);
        } else {
#pragma unroll
            for (int i = 0; i < VE; i++) d[i] = g[i] = u[i] = 0.0f;
        }
        float s[VE], rest[VE];
        sigmoid<true>(g, s, rest);
#pragma unroll
        for (int i = 0; i < VE; i++) {
            const float a = g[i] * s[i], da = w * d[i], au = a * u[i];
            dw += d[i] * au;
            h[i] = w * au;
            du[i] = da * a;
            // bf16: 1 - s cancels far below its rounding, and rest costs registers that spill
            dg[i] = da * u[i] * (s[i] + a * (VE == 4 ? rest[i] : 1.0f - s[i]));
        }
        st_nt(dh13 + at, dg);
        st_nt(dh13 + at + I, du);
        if (h_out) st_h<HNT>(h_out + r * I + c, h);
    }
    if (d_row_weights) {
        dw = lanes_sum<LPR>(dw);
        if (lane == 0) d_row_weights[r] = dw;
    }
}

// Lanes to a row: a row of up to 64 pieces in one step, longer rows 64 at a
// time (200000 x 160 bf16, 20 pieces, backward: 53 us with 32 lanes, 84 with 64
// and 80 with 8, the fewest idle).
template <typename T, typename F>
static void with_lanes(int64_t R, int64_t I, F f) {
    const int64_t n = I / kVE<T>;
    auto lanes = [&](auto nt) {
        if (n > 32) f(std::integral_constant<int, 64>(), nt);
        else if (n > 16) f(std::integral_constant<int, 32>(), nt);
        else if (n > 8) f(std::integral_constant<int, 16>(), nt);
        else f(std::integral_constant<int, 8>(), nt);
    };
    if (R * I * 2 > kCachedH) lanes(std::true_type());
    else lanes(std::false_type());
}

template <typename T>
static void ckpt_launch(const void *h13, int64_t R, int64_t I, const float *row_weights, const int64_t *n_rows,
                        uint16_t *h_out, uint8_t *codes, uint8_t *scales, uint8_t *ckpt_codes, uint8_t *ckpt_scales,
                        hipStream_t s) {
    with_lanes<T>(R, I, [&](auto l, auto nt) {
        constexpr int LPR = decltype(l)::value, RW = 256 / LPR;
        k_swiglu_ckpt<T, LPR, decltype(nt)::value><<<grid_of((R + RW - 1) / RW), 256, 0, s>>>(
            reinterpret_cast<const T *>(h13), R, I, row_weights, n_rows, h_out, codes, scales, ckpt_codes, ckpt_scales);
    });
}

template <typename T>
static void ckpt_bwd_launch(const void *dh, int64_t R, int64_t I, const uint8_t *ckpt_codes,
                            const uint8_t *ckpt_scales, const float *row_weights, const int64_t *n_rows, void *dh13,
                            uint16_t *h_out, float *d_row_weights, hipStream_t s) {
    with_lanes<T>(R, I, [&](auto l, auto nt) {
        constexpr int LPR = decltype(l)::value, RW = 256 / LPR;
        k_swiglu_ckpt_bwd<T, LPR, decltype(nt)::value><<<grid_of((R + RW - 1) / RW), 256, 0, s>>>(
            reinterpret_cast<const T *>(dh), R, I, ckpt_codes, ckpt_scales, row_weights, n_rows,
            reinterpret_cast<T *>(dh13), h_out, d_row_weights);
    });
}

hipError_t launch_swiglu_checkpoint(const void *h13, int in_dtype, int64_t R, int64_t I, const float *row_weights,
                                    const int64_t *n_rows, uint16_t *h_out, uint8_t *codes, uint8_t *scales,
                                    uint8_t *ckpt_codes, uint8_t *ckpt_scales, hipStream_t s) {
    auto launch = in_dtype == BSP_DTYPE_BF16 ? ckpt_launch<uint16_t> : ckpt_launch<float>;
    launch(h13, R, I, row_weights, n_rows, h_out, codes, scales, ckpt_codes, ckpt_scales, s);
    return hipGetLastError();
}

hipError_t launch_swiglu_checkpoint_backward(const void *dh, int dtype, int64_t R, int64_t I,
                                             const uint8_t *ckpt_codes, const uint8_t *ckpt_scales,
                                             const float *row_weights, const int64_t *n_rows, void *dh13,
                                             uint16_t *h_out, float *d_row_weights, hipStream_t s) {
    auto launch = dtype == BSP_DTYPE_BF16 ? ckpt_bwd_launch<uint16_t> : ckpt_bwd_launch<float>;
    launch(dh, R, I, ckpt_codes, ckpt_scales, row_weights, n_rows, dh13, h_out, d_row_weights, s);
    return hipGetLastError();
}

}  // namespace bsp
