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

}  // namespace bsp
