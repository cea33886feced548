// bsp_moe.hpp -- launch entry points of the routing, SwiGLU-checkpoint and
// combine kernels, shared between their files and the C ABI shim (which
// validates the arguments first), and device helpers those kernels share.
#pragma once

#include "bsp_device.hpp"
#include "bsp_internal.hpp"

namespace bsp {

int64_t route_workspace_bytes(int64_t T, int64_t E, int64_t k, int64_t shared);
hipError_t launch_route(const void *logits, int dtype, int64_t T, int64_t E, int64_t ldl, const uint8_t *mask,
                        int64_t k, int64_t shared, int32_t *experts, float *weights, int32_t *counts, int64_t *off,
                        int32_t *src, int32_t *pos, float *row_weights, float *prob_sum, float *loss, bool norm,
                        void *workspace, hipStream_t s);
hipError_t launch_route_backward(const void *logits, int dtype, int64_t T, int64_t E, int64_t ldl,
                                 const uint8_t *mask, int64_t k, int64_t shared, const int32_t *experts,
                                 const int32_t *pos, const int32_t *counts, const float *d_weights,
                                 const float *d_loss, void *d_logits, int64_t ldd, bool norm, hipStream_t s);
hipError_t launch_combine(const void *y, int in_dtype, int64_t rows, int64_t H, int64_t ldy, const int32_t *pos,
                          const float *weights, int64_t T, int64_t kk, void *out, int out_dtype, int64_t ldo,
                          hipStream_t s);
hipError_t launch_swiglu_checkpoint(const void *h13, int in_dtype, int64_t R, int64_t I, const float *row_weights,
                                    const int64_t *n_rows, uint16_t *h_out, uint8_t *codes, uint8_t *scales,
                                    uint8_t *ckpt_codes, uint8_t *ckpt_scales, hipStream_t s);
hipError_t launch_swiglu_checkpoint_backward(const void *dh, int dtype, int64_t R, int64_t I,
                                             const uint8_t *ckpt_codes, const uint8_t *ckpt_scales,
                                             const float *row_weights, const int64_t *n_rows, void *dh13,
                                             uint16_t *h_out, float *d_row_weights, hipStream_t s);

hipError_t launch_quantize_mxfp4(const uint16_t *x, int64_t x_rows, int64_t K, int64_t ldx, const int32_t *gather,
                                 int64_t M, uint8_t *codes_row, uint8_t *scales_row, uint8_t *codes_colT,
                                 uint8_t *scales_colT, int64_t ld, const int64_t *off, int64_t G, int64_t batch,
                                 bool sr, uint64_t seed, hipStream_t s);
hipError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K, void *out,
                                   bool bf16, hipStream_t s);

// Grouped products of MX operands and the gated block.  tile: 0 (by size), 32 (few rows) or 128 (tiled).
int64_t mx_gemm_workspace_bytes(int fmt, int mode, int64_t M, int64_t N, int64_t K, int64_t G, int tile);
int64_t mx_gated_workspace_bytes(int fmt, int64_t R, int64_t I, int64_t K, int64_t G, int tile);
int64_t mx_gated_bwd_workspace_bytes(int fmt, int64_t R, int64_t I, int64_t K, int64_t G, bool sums, int tile);
hipError_t launch_mx_gemm(int fmt, int mode, const uint8_t *a_codes, const uint8_t *a_scales, const int32_t *gather,
                          int64_t a_rows, const int64_t *off, int64_t G, int64_t M, int64_t N, int64_t K,
                          const uint8_t *b_codes, const uint8_t *b_scales, void *c, int c_dtype, int64_t ldc,
                          void *workspace, int tile, hipStream_t s);
hipError_t launch_moe_gated(int fmt, const uint8_t *a_codes, const uint8_t *a_scales, const int32_t *gather,
                            int64_t a_rows, const int64_t *off, int64_t G, int64_t R, int64_t I, int64_t K,
                            const uint8_t *b_codes, const uint8_t *b_scales, const float *row_weights, uint16_t *h,
                            int h_fmt, uint8_t *h_codes, uint8_t *h_scales, uint8_t *ckpt_codes, uint8_t *ckpt_scales,
                            void *workspace, int tile, hipStream_t s);
hipError_t launch_moe_gated_backward(int fmt, const uint8_t *dy_codes, const uint8_t *dy_scales, const int32_t *gather,
                                     int64_t dy_rows, const int64_t *off, int64_t G, int64_t R, int64_t I, int64_t K,
                                     const uint8_t *b_codes, const uint8_t *b_scales, const uint8_t *ckpt_codes,
                                     const uint8_t *ckpt_scales, const float *row_weights, uint16_t *dh13, uint16_t *h,
                                     float *d_row_weights, void *workspace, int tile, hipStream_t s);

// A row of n workgroups as a grid: a grid dimension holds fewer than 2^32
// threads, so longer rows go on over y; the last may be partly past n.
constexpr int64_t kGridX = 1ll << 23;   // of at most 256 threads
inline dim3 grid_of(int64_t n) {
    return n <= kGridX ? dim3((unsigned)n) : dim3((unsigned)kGridX, (unsigned)((n + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t grid_index() { return blockIdx.y * kGridX + blockIdx.x; }

// ---- device helpers shared by the kernels of these entry points ----

// Sum over the 64 lanes, the same bits on every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Two bf16 (a in the low half), nearest even, by V_CVT_PK_BF16_F32.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}

// Loads and stores of 16 and 8 bytes; NT: nontemporal (data used once).
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32v2 __attribute__((ext_vector_type(2)));
template <bool NT>
__device__ __forceinline__ u32v4 ld4w(const void *p) {
    const u32v4 *q = reinterpret_cast<const u32v4 *>(p);
    return NT ? __builtin_nontemporal_load(q) : *q;
}
template <bool NT>
__device__ __forceinline__ void st4w(void *p, u32v4 v) {
    u32v4 *q = reinterpret_cast<u32v4 *>(p);
    if (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
}
template <bool NT>
__device__ __forceinline__ uint2 ld2(const void *p) {
    const u32v2 *q = reinterpret_cast<const u32v2 *>(p);
    const u32v2 v = NT ? __builtin_nontemporal_load(q) : *q;
    return make_uint2(v.x, v.y);
}
template <bool NT>
__device__ __forceinline__ void st2(void *p, uint2 v) {
    u32v2 *q = reinterpret_cast<u32v2 *>(p);
    if (NT) __builtin_nontemporal_store((u32v2){v.x, v.y}, q);
    else *q = (u32v2){v.x, v.y};
}

// Eight consecutive values (16-byte aligned) as f32, and back (bf16: nearest even).
template <bool NT>
__device__ __forceinline__ void ld8(const float *p, float (&v)[8]) {
    const u32v4 x = ld4w<NT>(p), y = ld4w<NT>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[i] = __uint_as_float(x[i]);
        v[4 + i] = __uint_as_float(y[i]);
    }
}
template <bool NT>
__device__ __forceinline__ void ld8(const uint16_t *p, float (&v)[8]) {
    const u32v4 u = ld4w<NT>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16_lo(u[i]);
        v[2 * i + 1] = bf16_hi(u[i]);
    }
}
template <bool NT>
__device__ __forceinline__ void st8(float *p, const float (&v)[8]) {
    st4w<NT>(p, (u32v4){__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
    st4w<NT>(p + 4, (u32v4){__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
}
template <bool NT>
__device__ __forceinline__ void st8(uint16_t *p, const float (&v)[8]) {
    st4w<NT>(p, (u32v4){bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])});
}

// s = 1 / (1 + e), e = exp(-z), and (FULL) c = 1 - s = e s, of VE values.
// FULL, for f32 results and for codes that are rounded from them: e = 2^t (1 + d), t = -z log2(e) rounded and d what the
// rounding left out; without d the error of e grows with |z| (2.8 units of 2^-24
// at 4, 60 at 80).  With it s is within 6 + 0.05 |z| units and c, which 1 - s
// would cancel, within 10 + 0.1 |z|.  swiglu_checkpoint's h is rounded to bf16
// first and does without.  Past |z| = 87 2^t, the reciprocal (V_RCP_F32 flushes results below
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

}  // namespace bsp
