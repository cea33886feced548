// bsp_mxfp4.hip -- MXFP4: 32 consecutive E2M1 values share one power-of-two
// (E8M0) scale.  Quantization of bf16, rowwise and columnwise, to nearest or
// stochastically, and the values again.
//
//   k = smallest integer with amax <= 6 * 2^k (never clips), in [-127, 125]
//   code = E2M1(x * 2^-k): x * 2^-k is exact in f32 (0 far below the grid), so each value is rounded once
//   a block with a NaN: scale 255, with which the conversions and the matrix instructions give NaN for any code
//
// HBM bounds: 2 bytes in and 17/32 bytes out per value and copy.  8192 x 2048
// takes 10 us rowwise (42 MB, 4.2 TB/s) and 15 in both copies (51 MB, 3.4 TB/s),
// 65536 x 1536 by groups and rounded
// stochastically 147 us (302 MB, 2.1 TB/s): there the generator's vector
// instructions bound it, as they do every stochastic rounding here.
#include "bsp_moe.hpp"

namespace bsp {

namespace {

// Eight codes (element 2j in the low nibble of byte j) of eight values scaled to the grid by r = 2^-k.
__device__ __forceinline__ uint32_t pack8_nearest(const float (&x)[8], float r) {
    uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0] * r, x[1] * r, 1.0f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2] * r, x[3] * r, 1.0f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4] * r, x[5] * r, 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6] * r, x[7] * r, 1.0f, 3);
}

// The same rounded stochastically with the eight 16-bit draws of Philox block `blk` (word 2 of the counter: copy).
__device__ __forceinline__ uint32_t pack8_stochastic(const float (&x)[8], float r, uint64_t blk, uint32_t copy,
                                                     uint32_t key0, uint32_t key1) {
    uint32_t c[4] = {(uint32_t)blk, (uint32_t)(blk >> 32), copy, 0u};
    philox4x32_10(c, key0, key1);
    // packed by funnel shifts, last element first
    uint32_t q = e2m1_sr_code_hi<true>(x[7], r, ~c[3]) >> 28;
#pragma unroll
    for (int w = 3; w >= 0; w--) {
        if (w < 3) q = __builtin_amdgcn_alignbit(q, e2m1_sr_code_hi<true>(x[2 * w + 1], r, ~c[w]), 28);
        q = __builtin_amdgcn_alignbit(q, e2m1_sr_code_hi<false>(x[2 * w], r, ~c[w]), 28);
    }
    return q;
}

__device__ __forceinline__ void unpack8(uint4 raw, float (&x)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
    }
}

__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) a = max_nan(a, fabsf(x[j]));
    return a;
}

// Eight values of a row whose 32-value block lies on four neighbouring lanes: this lane's codes and the scale code.
template <bool SR>
__device__ __forceinline__ uint32_t row_codes(const float (&x)[8], uint64_t blk, uint32_t key0, uint32_t key1,
                                              uint32_t &scale) {
    float a = amax8(x);
    a = max_nan(a, __shfl_xor(a, 1, 64));
    a = max_nan(a, __shfl_xor(a, 2, 64));
    const int k = mx4_block_exponent(a);
    scale = mx4_scale(a, k);
    const float r = exp2i(-k);
    return SR ? pack8_stochastic(x, r, blk, 0u, key0, key1) : pack8_nearest(x, r);
}

}  // namespace

// Rowwise only: eight values per lane.  A stack of matrices is one matrix of rows rows here.
template <bool SR>
__global__ __launch_bounds__(256) void k_mxfp4_row(const uint16_t *__restrict__ x, int64_t rows, int64_t K,
                                                   int64_t ldx, uint8_t *__restrict__ codes,
                                                   uint8_t *__restrict__ scales, const int32_t *__restrict__ gather,
                                                   int64_t x_rows, uint32_t key0, uint32_t key1) {
    const int64_t per = K / 8, i = grid_index() * 256 + threadIdx.x;
    const bool in = i < rows * per;   // K % 32 == 0: the four lanes of a block agree
    const int64_t r = in ? i / per : 0, c = in ? i - r * per : 0;
    int64_t xr = r;
    if (gather) {
        xr = gather[r];
        if (xr < 0 || xr >= x_rows) xr = -1;
    }
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (in && xr >= 0) raw = *reinterpret_cast<const uint4 *>(x + xr * ldx + 8 * c);
    float v[8];
    unpack8(raw, v);
    uint32_t sc;
    const uint32_t q = row_codes<SR>(v, (uint64_t)i, key0, key1, sc);
    if (!in) return;
    reinterpret_cast<uint32_t *>(codes)[i] = q;
    if ((c & 3) == 0) scales[i / 4] = (uint8_t)sc;
}

constexpr int M4_TR = 128, M4_TC = 128;

// One 128 x 128 tile from a single read of x: rowwise blocks straight from
// registers, columnwise blocks (32 along the rows) through LDS.
// GROUPED: tile rows live in the padded row space, where group g starts at
// P[g], the running sum of the group sizes rounded up to 32, and row p of it
// is source row off[g] + (p - P[g]) (zeros past the group); a workgroup finds
// its four 32-row blocks by a scan over the groups.
template <bool ROW, bool GROUPED, bool SR>
__global__ __launch_bounds__(256) void k_mxfp4_tile(const uint16_t *__restrict__ x, int64_t M, int64_t K, int64_t ldx,
                                                    uint8_t *__restrict__ codes_row, uint8_t *__restrict__ scales_row,
                                                    uint8_t *__restrict__ codes_colT,
                                                    uint8_t *__restrict__ scales_colT, int64_t ld,
                                                    const int64_t *__restrict__ off, int G,
                                                    const int32_t *__restrict__ gather, int64_t x_rows, uint32_t key0,
                                                    uint32_t key1) {
    __shared__ __attribute__((aligned(16))) uint16_t tile[M4_TR][M4_TC];
    __shared__ int64_t rdst[M4_TR], xsrc[M4_TR];   // row of the row copy (-1: none) and of x (-1: zeros)
    __shared__ int64_t blk0[M4_TR / 32], blk1[M4_TR / 32], wsum[4];
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
    const int64_t gx = (K + M4_TC - 1) / M4_TC, gy = ((GROUPED ? ld : M) + M4_TR - 1) / M4_TR, n = gx * gy;
    // workgroup L runs tile (L % 8) chunk + L / 8 of the column-major order: each XCD its own run of column tiles,
    // whose rows of a gathered x it finds in its L2
    const int64_t L = grid_index(), chunk = (n + 7) / 8, v = (L % 8) * chunk + L / 8;
    if (v >= n || L / 8 >= chunk) return;
    const int64_t k0 = (v / gy) * M4_TC, p0 = (v % gy) * M4_TR;
    int64_t ptotal = M;
    uint64_t rowel = 0, colel = 0;   // elements before this matrix of a stack, for the random draws
    if (!GROUPED && gridDim.z > 1) {
        const int64_t b = blockIdx.z;
        x += b * x_rows * ldx;
        rowel = (uint64_t)(b * M * K);
        colel = (uint64_t)(b * K * ld);
        if (ROW) {
            codes_row += b * M * (K / 2);
            scales_row += b * M * (K / 32);
        }
        codes_colT += b * K * (ld / 2);
        scales_colT += b * K * (ld / 32);
    }
    if constexpr (GROUPED) {
        const int per = (G + 255) / 256, g0 = t * per, g1 = g0 + per < G ? g0 + per : G;
        int64_t local = 0;
        for (int g = g0; g < g1; g++) local += (off[g + 1] - off[g] + 31) / 32 * 32;
        if (t < M4_TR / 32) blk0[t] = blk1[t] = 0;
        int64_t run = block256_excl_scan(local, wsum, ptotal);
        if (local > 0 && run < p0 + M4_TR && run + local > p0) {
            for (int g = g0; g < g1; g++) {
                const int64_t o0 = off[g], o1 = off[g + 1], pn = (o1 - o0 + 31) / 32 * 32;
#pragma unroll
                for (int b = 0; b < M4_TR / 32; b++) {
                    const int64_t pb = p0 + 32 * b;
                    if (pb >= run && pb < run + pn) {
                        blk0[b] = o0 + (pb - run);
                        blk1[b] = o1 < M ? o1 : M;   // offsets past M are never read
                    }
                }
                run += pn;
            }
        }
        __syncthreads();
        if (p0 >= ptotal) return;
    }
    if (t < M4_TR) {
        int64_t src = p0 + t < M ? p0 + t : -1;
        if (GROUPED) {
            const int64_t s = blk0[t >> 5] + (t & 31);
            src = p0 + t < ptotal && s >= 0 && s < blk1[t >> 5] ? s : -1;
        }
        rdst[t] = src;
        if (src >= 0 && gather) {
            src = gather[src];
            if (src < 0 || src >= x_rows) src = -1;
        }
        xsrc[t] = src;
    }
    __syncthreads();

    // rows: lane l of wavefront w takes 16-byte piece l % 16 of tile rows 32 w + 4 i + l / 16
    const int ch = lane & 15, rq = lane >> 4;
    const int64_t kc = k0 + 8 * ch;
    const bool col_ok = kc < K;
    uint4 raw[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t xr = xsrc[32 * wv + 4 * i + rq];
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (xr >= 0 && col_ok) raw[i] = *reinterpret_cast<const uint4 *>(x + xr * ldx + kc);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int row = 32 * wv + 4 * i + rq;
        if constexpr (ROW) {
            float f[8];
            unpack8(raw[i], f);
            const int64_t dr = rdst[row];
            uint32_t sc;
            const uint32_t q = row_codes<SR>(f, (rowel + (uint64_t)(dr * K + kc)) / 8, key0, key1, sc);
            if (dr >= 0 && col_ok) {
                *reinterpret_cast<uint32_t *>(codes_row + dr * (K / 2) + kc / 2) = q;
                if ((ch & 3) == 0) scales_row[dr * (K / 32) + kc / 32] = (uint8_t)sc;
            }
        }
        *reinterpret_cast<uint4 *>(&tile[row][8 * ch]) = raw[i];
    }
    __syncthreads();

    // columns: thread t owns column t % 128 and two 32-row blocks
    const int c = t & 127, rh = t >> 7;
    const int64_t kcol = k0 + c;
    uint4 q[2];
#pragma unroll
    for (int b = 0; b < 2; b++) {
        const int64_t pb = p0 + 64 * rh + 32 * b;
        float f[4][8], a = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i++) f[i >> 3][i & 7] = __uint_as_float((uint32_t)tile[64 * rh + 32 * b + i][c] << 16);
#pragma unroll
        for (int i = 0; i < 4; i++) a = max_nan(a, amax8(f[i]));
        const int k = mx4_block_exponent(a);
        const float r = exp2i(-k);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = SR ? pack8_stochastic(f[i], r, (colel + (uint64_t)(kcol * ld + pb)) / 8 + i, 1u, key0, key1)
                      : pack8_nearest(f[i], r);
        q[b] = make_uint4(w[0], w[1], w[2], w[3]);
        if (kcol < K && pb < ptotal) scales_colT[kcol * (ld / 32) + pb / 32] = (uint8_t)mx4_scale(a, k);
    }
    __syncthreads();   // the input tile is no longer read

    // codes through LDS, so that a store covers whole 64-byte pieces of rows (four lanes each)
    uint8_t *stage = reinterpret_cast<uint8_t *>(&tile[0][0]);
#pragma unroll
    for (int b = 0; b < 2; b++) *reinterpret_cast<uint4 *>(stage + c * 80 + 16 * (2 * rh + b)) = q[b];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int id = 256 * i + t, r = id >> 2, piece = id & 3;
        if (k0 + r < K && p0 + 32 * piece < ptotal)
            *reinterpret_cast<uint4 *>(codes_colT + (k0 + r) * (ld / 2) + p0 / 2 + 16 * piece) =
                *reinterpret_cast<const uint4 *>(stage + r * 80 + 16 * piece);
    }
}

// Eight values per lane.
template <bool BF16>
__global__ __launch_bounds__(256) void k_dequant_mxfp4(const uint8_t *__restrict__ codes,
                                                       const uint8_t *__restrict__ scales, int64_t n8,
                                                       void *__restrict__ out) {
    const int64_t i = grid_index() * 256 + threadIdx.x;
    if (i >= n8) return;
    const uint32_t c = reinterpret_cast<const uint32_t *>(codes)[i];
    const float s = __uint_as_float((uint32_t)scales[i / 4] << 23);   // its exponent alone counts: 0 is 2^-127, 255 NaN
    const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    const float y[8] = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
    if (BF16) st8<true>(reinterpret_cast<uint16_t *>(out) + 8 * i, y);
    else st8<true>(reinterpret_cast<float *>(out) + 8 * i, y);
}

hipError_t launch_quantize_mxfp4(const uint16_t *x, int64_t x_rows, int64_t K, int64_t ldx, const int32_t *gather,
                                 int64_t M, uint8_t *codes_row, uint8_t *scales_row, uint8_t *codes_colT,
                                 uint8_t *scales_colT, int64_t ld, const int64_t *off, int64_t G, int64_t batch,
                                 bool sr, uint64_t seed, hipStream_t s) {
    const uint32_t key0 = (uint32_t)seed, key1 = (uint32_t)(seed >> 32);
    if (!codes_colT) {
        auto k = sr ? k_mxfp4_row<true> : k_mxfp4_row<false>;
        k<<<grid_of((M * batch * (K / 8) + 255) / 256), 256, 0, s>>>(x, M * batch, K, ldx, codes_row, scales_row,
                                                                     gather, x_rows, key0, key1);
        return hipGetLastError();
    }
    const int64_t tiles = (K + M4_TC - 1) / M4_TC * (((off ? ld : M) + M4_TR - 1) / M4_TR);
    dim3 grid = grid_of(8 * ((tiles + 7) / 8));
    grid.z = (unsigned)batch;
    auto go = [&](auto kern) {
        kern<<<grid, 256, 0, s>>>(x, M, K, ldx, codes_row, scales_row, codes_colT, scales_colT, ld, off, (int)G,
                                  gather, x_rows, key0, key1);
    };
    const bool row = codes_row != nullptr;
    if (off) {
        if (row) go(sr ? k_mxfp4_tile<true, true, true> : k_mxfp4_tile<true, true, false>);
        else go(sr ? k_mxfp4_tile<false, true, true> : k_mxfp4_tile<false, true, false>);
    } else {
        if (row) go(sr ? k_mxfp4_tile<true, false, true> : k_mxfp4_tile<true, false, false>);
        else go(sr ? k_mxfp4_tile<false, false, true> : k_mxfp4_tile<false, false, false>);
    }
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t M, int64_t K, void *out,
                                   bool bf16, hipStream_t s) {
    const int64_t n8 = M * K / 8;
    auto k = bf16 ? k_dequant_mxfp4<true> : k_dequant_mxfp4<false>;
    k<<<grid_of((n8 + 255) / 256), 256, 0, s>>>(codes, scales, n8, out);
    return hipGetLastError();
}

}  // namespace bsp
