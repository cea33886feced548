// bsp_checkpoint.hip -- SwiGLU whose input is kept for the backward pass as
// MXFP8, and its gradient from that 8-bit checkpoint.
//
//   forward:  h = w silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g));
//             checkpoint = MXFP8([g u]), blocks of 32 along the row
//   backward: du = w dh g s,  dg = w dh u s (1 + g (1 - s)),
//             dw = sum_i dh_i g_i s_i u_i,  h again
// Both are bound by HBM: per h element the forward moves 2 s + 2 + 2.06 bytes
// (s = 4 or 2 for f32 or bf16 h13) and the backward 3 s + 2.06 + 2.
#include "bsp_moe.hpp"

namespace bsp {

namespace {

template <int CTRL>
__device__ __forceinline__ float quad_perm(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// MXFP8 of a block of 32 held as 8 values on each of 4 neighbouring lanes:
// this lane's codes; returns the scale code.
__device__ __forceinline__ uint32_t mx_quad(const float (&v)[8], uint2 &q) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) a = fmaxf(a, fabsf(v[i]));
    a = fmaxf(a, quad_perm<0xB1>(a));   // lanes 1 0 3 2
    a = fmaxf(a, quad_perm<0x4E>(a));   // lanes 2 3 0 1
    const int k = mx_block_exponent(a);
    const float inv = exp2i(-k);
    q.x = e4m3x4_hw(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    q.y = e4m3x4_hw(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    return (uint32_t)(k + 127);
}

// Eight MXFP8 values; sc: the block's scale code.
__device__ __forceinline__ void mx_value8(uint2 q, uint32_t sc, float (&v)[8]) {
    const float s = __uint_as_float(sc ? sc << 23 : 0x00400000u);   // 2^-127 is a subnormal f32
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[i] = e4m3_decode((q.x >> (8 * i)) & 0xFFu) * s;
        v[4 + i] = e4m3_decode((q.y >> (8 * i)) & 0xFFu) * s;
    }
}

// 1 / (1 + exp(-z)).  Evaluated as 2^-32 / (2^-32 + 2^(-z log2(e) - 32)):
// V_RCP_F32 flushes results below 2^-126 to zero, which the plain form meets
// from z < -87.3 while z s is still above the smallest bf16 values; the factor
// keeps its argument and result normal down to z = -110.
__device__ __forceinline__ float sigmoid(float z) {
    const float e = __builtin_amdgcn_exp2f(fmaf(z, -1.44269504088896341f, -32.0f));
    return __builtin_amdgcn_rcpf(0x1p-32f + e) * 0x1p-32f;
}

}  // namespace

// One wavefront per row, eight columns per lane.
template <typename T>
__global__ __launch_bounds__(256) void k_swiglu_ckpt(const T *__restrict__ h13, int64_t R, int64_t I,
                                                     const float *__restrict__ row_weights,
                                                     const int64_t *__restrict__ n_rows, uint16_t *__restrict__ h_out,
                                                     uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                     uint8_t *__restrict__ ckpt_codes,
                                                     uint8_t *__restrict__ ckpt_scales) {
    const int lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= R) return;
    const bool used = !n_rows || r < *n_rows;
    const float w = used && row_weights ? row_weights[r] : 1.0f;
    const T *gp = h13 + r * 2 * I;
    for (int64_t c = lane * 8; c < I; c += 512) {
        float g[8], u[8], h[8];
#pragma unroll
        for (int i = 0; i < 8; i++) g[i] = u[i] = 0.0f;
        if (used) {
            ld8(gp + c, g);
            ld8(gp + I + c, u);
        }
        uint2 qg, qu;
        const uint32_t sg = mx_quad(g, qg), su = mx_quad(u, qu);
        *reinterpret_cast<uint2 *>(ckpt_codes + r * 2 * I + c) = qg;
        *reinterpret_cast<uint2 *>(ckpt_codes + r * 2 * I + I + c) = qu;
        if ((lane & 3) == 0) {
            ckpt_scales[(r * 2 * I + c) / 32] = (uint8_t)sg;
            ckpt_scales[(r * 2 * I + I + c) / 32] = (uint8_t)su;
        }
#pragma unroll
        for (int i = 0; i < 8; i++)
            h[i] = __uint_as_float(f32_to_bf16(w * (g[i] * sigmoid(g[i]) * u[i])) << 16);
        if (h_out) st8(h_out + r * I + c, h);
        if (codes) {
            uint2 q;
            const uint32_t s = mx_quad(h, q);
            *reinterpret_cast<uint2 *>(codes + r * I + c) = q;
            if ((lane & 3) == 0) scales[(r * I + c) / 32] = (uint8_t)s;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_swiglu_ckpt_bwd(const T *__restrict__ dh, int64_t R, int64_t I,
                                                         const uint8_t *__restrict__ ckpt_codes,
                                                         const uint8_t *__restrict__ ckpt_scales,
                                                         const float *__restrict__ row_weights,
                                                         const int64_t *__restrict__ n_rows, T *__restrict__ dh13,
                                                         uint16_t *__restrict__ h_out,
                                                         float *__restrict__ d_row_weights) {
    const int lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= R) return;
    const bool used = !n_rows || r < *n_rows;
    const float w = used && row_weights ? row_weights[r] : 1.0f;
    float dw = 0.0f;
    for (int64_t c = lane * 8; c < I; c += 512) {
        float d[8], g[8], u[8], dg[8], du[8], h[8];
#pragma unroll
        for (int i = 0; i < 8; i++) d[i] = g[i] = u[i] = 0.0f;
        if (used) {
            const int64_t at = r * 2 * I + c;
            ld8(dh + r * I + c, d);
            mx_value8(*reinterpret_cast<const uint2 *>(ckpt_codes + at), ckpt_scales[at / 32], g);
            mx_value8(*reinterpret_cast<const uint2 *>(ckpt_codes + at + I), ckpt_scales[(at + I) / 32], u);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float s = sigmoid(g[i]), a = g[i] * s, da = w * d[i], au = a * u[i];
            dw += d[i] * au;
            h[i] = w * au;
            du[i] = da * a;
            dg[i] = da * u[i] * (s + a * (1.0f - s));
        }
        st8(dh13 + r * 2 * I + c, dg);
        st8(dh13 + r * 2 * I + I + c, du);
        if (h_out) st8(h_out + r * I + c, h);
    }
    if (d_row_weights) {
        dw = wave_sum(dw);
        if (lane == 0) d_row_weights[r] = dw;
    }
}

hipError_t launch_swiglu_checkpoint(const void *h13, int in_dtype, int64_t R, int64_t I, const float *row_weights,
                                    const int64_t *n_rows, uint16_t *h_out, uint8_t *codes, uint8_t *scales,
                                    uint8_t *ckpt_codes, uint8_t *ckpt_scales, hipStream_t s) {
    const unsigned grid = (unsigned)((R + 3) / 4);
    if (in_dtype == BSP_DTYPE_BF16)
        k_swiglu_ckpt<uint16_t><<<grid, 256, 0, s>>>(reinterpret_cast<const uint16_t *>(h13), R, I, row_weights, n_rows,
                                                     h_out, codes, scales, ckpt_codes, ckpt_scales);
    else
        k_swiglu_ckpt<float><<<grid, 256, 0, s>>>(reinterpret_cast<const float *>(h13), R, I, row_weights, n_rows,
                                                  h_out, codes, scales, ckpt_codes, ckpt_scales);
    return hipGetLastError();
}

hipError_t launch_swiglu_checkpoint_backward(const void *dh, int dtype, int64_t R, int64_t I,
                                             const uint8_t *ckpt_codes, const uint8_t *ckpt_scales,
                                             const float *row_weights, const int64_t *n_rows, void *dh13,
                                             uint16_t *h_out, float *d_row_weights, hipStream_t s) {
    const unsigned grid = (unsigned)((R + 3) / 4);
    if (dtype == BSP_DTYPE_BF16)
        k_swiglu_ckpt_bwd<uint16_t><<<grid, 256, 0, s>>>(reinterpret_cast<const uint16_t *>(dh), R, I, ckpt_codes,
                                                         ckpt_scales, row_weights, n_rows,
                                                         reinterpret_cast<uint16_t *>(dh13), h_out, d_row_weights);
    else
        k_swiglu_ckpt_bwd<float><<<grid, 256, 0, s>>>(reinterpret_cast<const float *>(dh), R, I, ckpt_codes,
                                                      ckpt_scales, row_weights, n_rows,
                                                      reinterpret_cast<float *>(dh13), h_out, d_row_weights);
    return hipGetLastError();
}

}  // namespace bsp
