// bsp_route.hip -- MoE routing: expert choice, counts, grouped-row map and
// load-balance loss from router logits, the gradient to the logits, and the
// sum of every token's grouped rows.
//
// Routing mathematics.  Per token, p = softmax(l) over the experts whose
// logit is above -inf, the k largest logits (ties to the lower index) with
// weights p (or p over its sum on the choice), and over the batch
//   loss = E / (k n^2) sum_e c_e Q_e,   c_e the rows of expert e,
//   Q_e = sum_t p_te, n the routed tokens.
// The choice compares logits, not probabilities: it is then independent of
// how the exponential is evaluated.
#include "bsp_moe.hpp"

namespace bsp {

// exp(x) for x <= 0, within 3 + 0.05 |x| units of 2^-24: 2^t (1 + d), t = x log2(e)
// and d what its rounding left out; without d the error grows with |x| (63 units
// at 80).  The factor for t is 2^-22 above log2(e), so that d >= 0 and an
// instruction's clamp to [0, 1] leaves it alone but makes the NaN of x = -inf a 0.
// V_EXP_F32 flushes results below 2^-126, from x < -87.3, to 0.  NaN stays NaN.
// Choice and placing of 100003 x 96 take 23.0 us instead of 22.5 for it.
template <bool FULL = true>
__device__ __forceinline__ float exp_f32(float x) {
    constexpr float L2E = 1.44269504088896341f * (1.0f + 0x1p-22f), LN2 = 0.693147180559945309f;
    if (!FULL) return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
    const float t = x * L2E, e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, __builtin_amdgcn_fmed3f(fmaf(-t, LN2, x), 0.0f, 1.0f), e);
}
template <bool FULL>
__device__ __forceinline__ float recip(float x) { return FULL ? 1.0f / x : __builtin_amdgcn_rcpf(x); }
// From about here on fewer lanes to a token pay: choice of 16384 f32 tokens 5.9 us
// (with more lanes 6.0) for 64 experts, 7.4 (6.7) for 128 and 10.5 (10.9) for 256,
// 24000 x 256 11.9 (14.0), 131072 x 256 34.8 (52.1); below, 4096 x 128 6.8 (5.3).
constexpr int64_t kManyTokens = 16384;
// Gradient: three workgroups to a compute unit, as the registers of the widest
// form allow (65537 x 256 bf16: 19.9 us, with 1536 23.4).
constexpr int64_t kBwdWorkgroups = 768;
// Batches that one workgroup finishes in one launch: of 256 threads, or of 1024
// for up to 256 experts and k <= 8 (128 tokens, 128 experts: 10.5 us a call
// instead of 15.3 with two launches; 256 tokens: 14.5, and 24 with 256 experts).
constexpr int64_t kOneSmallTokens = 64, kOneLargeTokens = 128;
constexpr int kMaxShared = 64;
constexpr int kMaxGroups = 1024 + kMaxShared;
constexpr int kFewGroups = kMaxGroups / 2;   // placing: groups of the smaller rank table
constexpr int kSums = 8, kMaxSlice = 1024 / 4 / kSums;   // workgroups that sum the probabilities, their quads of experts

// Lane exchanges within a row of 16 by DPP.  A token's L lanes (4, 8, 16 or 32)
// reduce over xor 1, xor 2, mirror(8), mirror(16), each step joining two
// disjoint sets of lanes; L = 32 ends with the other row of 16.
enum { DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_MIRROR16 = 0x140, DPP_MIRROR8 = 0x141, DPP_ROR4 = 0x124, DPP_ROR8 = 0x128 };
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// All-reduce over the L lanes that share a token.  The sums add the same two
// values on both sides of every step, so all lanes hold the same bits.
template <int L>
__device__ __forceinline__ float group_max(float v) {
    if (L == 32) v = fmaxf(v, __shfl_xor(v, 16, 64));
    if (L >= 16) v = fmaxf(v, dpp<DPP_MIRROR16>(v));
    if (L >= 8) v = fmaxf(v, dpp<DPP_MIRROR8>(v));
    v = fmaxf(v, dpp<DPP_XOR2>(v));
    return fmaxf(v, dpp<DPP_XOR1>(v));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    v += dpp<DPP_XOR1>(v);
    v += dpp<DPP_XOR2>(v);
    if (L >= 8) v += dpp<DPP_MIRROR8>(v);
    if (L >= 16) v += dpp<DPP_MIRROR16>(v);
    if (L == 32) v += __shfl_xor(v, 16, 64);
    return v;
}
// The order of a token's sums is that of 8 lanes for up to 128 logits and of 16
// for more, also on half as many lanes, which long batches use: a lane then holds
// two lanes' parts, of the even and of the odd pieces, and adds their sums as the
// last step would have.  A token's weights and gradient do not depend, to the
// bit, on the size of its batch.
template <int L, int V>
constexpr int kParts = (L * V <= 128 ? 8 : 16) == 2 * L ? 2 : 1;
template <int L, int P>
__device__ __forceinline__ float parts_sum(const float (&s)[P]) {
    float v = group_sum<L>(s[0]);
    if constexpr (P == 2) v += group_sum<L>(s[1]);
    return v;
}

// A token's logits on its L lanes, V to a lane in 16-byte pieces of Q values:
// piece j of lane l is experts [(j L + l) Q, +Q), so a load covers 16 L
// contiguous bytes of each row.
template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);
template <typename T, int L>
__device__ __forceinline__ int expert_of(int lane, int i) {
    constexpr int Q = kPiece<T>;
    return ((i / Q) * L + lane) * Q + i % Q;
}
__device__ __forceinline__ float elem(const float *p) { return *p; }
__device__ __forceinline__ float elem(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) { *p = (uint16_t)bf16x2(v, 0.0f); }
__device__ __forceinline__ void st16(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st16(uint16_t *p, const float *v) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                                               bf16x2(v[6], v[7]));
}
// A row's V logits as loaded.  Every load is issued, those past E from the
// row's start, and what is not wanted becomes -inf afterwards: a load under a
// condition would be waited for before the next.  VEC: rows start on 16 bytes
// and E is a multiple of Q, so a piece is whole or absent.
template <typename T, int L, int V, bool VEC>
struct RowLoad {
    static constexpr int Q = kPiece<T>;
    uint4 r[VEC ? V / Q : 1];
    T x[VEC ? 1 : V];
    __device__ __forceinline__ void load(const T *row, int lane, int E) {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < V / Q; j++) {
                const int e = expert_of<T, L>(lane, j * Q);
                r[j] = *reinterpret_cast<const uint4 *>(row + (e < E ? e : 0));
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int e = expert_of<T, L>(lane, i);
                x[i] = row[e < E ? e : 0];
            }
        }
    }
    __device__ __forceinline__ void get(int lane, int E, bool keep, float (&v)[V]) const {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < V / Q; j++) {
                const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if constexpr (Q == 4) {
                        v[j * Q + i] = __uint_as_float(w[i]);
                    } else {
                        v[j * Q + 2 * i] = bf16_lo(w[i]);
                        v[j * Q + 2 * i + 1] = bf16_hi(w[i]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = elem(&x[i]);
        }
        if (E < L * V || !keep) {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = keep && expert_of<T, L>(lane, i) < E ? v[i] : -INFINITY;
        }
    }
};
template <typename T, int L, int V, bool VEC>
__device__ __forceinline__ void store_logits(T *row, int lane, int E, const float (&v)[V]) {
    constexpr int Q = kPiece<T>;
#pragma unroll
    for (int i = 0; i < V; i += Q) {
        const int e = expert_of<T, L>(lane, i);
        if (VEC) {
            if (e < E) st16(row + e, v + i);
        } else {
#pragma unroll
            for (int q = 0; q < Q; q++)
                if (e + q < E) put(row + e + q, v[i + q]);
        }
    }
}

// Softmax of a token whose largest logit is known: v becomes exp(v - m), 0 for
// -inf; returns the sum over the token.  It is 0 where no logit is above -inf
// and NaN where one is NaN or +inf.
template <typename T, int L, bool FULL, int V>
__device__ __forceinline__ float exp_sum(float (&v)[V], float m) {
    constexpr int P = kParts<L, V>;
    float s[P] = {};
#pragma unroll
    for (int i = 0; i < V; i++) {
        v[i] = exp_f32<FULL>(v[i] - m);
        s[i / kPiece<T> % P] += v[i];
    }
    return parts_sum<L, P>(s);
}

// ---------------------------------------------------------------------------
// The k <= N largest logits of a token by merging sorted lists
// ---------------------------------------------------------------------------
//
// A logit and its expert are one binary64: the high word is the logit's f32
// bits (every f32 up to infinity is a finite binary64 there, in the same
// order), the low word the complement of the expert's index, negated in turn
// for negative logits; -0 becomes +0.  A larger key is a larger logit or, among
// equal ones, a lower index, and no two keys are equal.  One V_MAX_F64 and one
// V_MIN_F64 (they issue at the rate of the f32 ones) are then a
// compare-exchange that carries the index along: half the operations of
// comparing and selecting value and index apart.  Each lane sorts its V keys
// and keeps N; a step across lanes takes the other lane's list in reverse
// (max(a_i, b_{N-1-i}) are the N largest of both) and sorts that bitonic list
// in log2(N) rounds.
__device__ __forceinline__ double make_key(uint32_t hi, uint32_t lo) {
    return __longlong_as_double(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ uint32_t key_hi(double k) { return (uint32_t)((uint64_t)__double_as_longlong(k) >> 32); }
__device__ __forceinline__ uint32_t key_lo(double k) { return (uint32_t)(uint64_t)__double_as_longlong(k); }
__device__ __forceinline__ double logit_key(float v, uint32_t rank) {
    const int32_t b = __float_as_int(v + 0.0f);
    return make_key((uint32_t)b, rank ^ (uint32_t)(b >> 31));
}
__device__ __forceinline__ float key_logit(double k) { return __uint_as_float(key_hi(k)); }
__device__ __forceinline__ int key_expert(double k) {
    return (int)(1023u - ((key_lo(k) ^ (uint32_t)((int32_t)key_hi(k) >> 31)) & 1023u));
}
constexpr uint32_t kNoKey = 0xFFA00000u;   // high word of a key below that of -inf; a NaN as a logit
__device__ __forceinline__ void order2(double &a, double &b) {   // a >= b
    const double x = __builtin_fmax(a, b), y = __builtin_fmin(a, b);
    a = x;
    b = y;
}

// Batcher's odd-even merge sort, descending.
template <int N>
__device__ __forceinline__ void sort_desc(double (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int h = p; h >= 1; h /= 2)
#pragma unroll
            for (int j = h % p; j + h < N; j += 2 * h)
#pragma unroll
                for (int i = 0; i < h; i++)
                    if (j + i + h < N && (j + i) / (2 * p) == (j + i + h) / (2 * p)) order2(k[j + i], k[j + i + h]);
}
// Sorts a bitonic list, descending.
template <int N>
__device__ __forceinline__ void bitonic_desc(double (&k)[N]) {
#pragma unroll
    for (int h = N / 2; h >= 1; h /= 2)
#pragma unroll
        for (int i = 0; i < N; i++)
            if (!(i & h)) order2(k[i], k[i + h]);
}
template <int N>
__device__ __forceinline__ void merge_desc(double (&a)[N], const double (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) a[i] = __builtin_fmax(a[i], b[N - 1 - i]);
    bitonic_desc<N>(a);
}
template <int N, int CTRL>
__device__ __forceinline__ void merge_dpp(double (&a)[N]) {
    double b[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        b[i] = make_key((uint32_t)__builtin_amdgcn_mov_dpp((int)key_hi(a[i]), CTRL, 0xF, 0xF, true),
                        (uint32_t)__builtin_amdgcn_mov_dpp((int)key_lo(a[i]), CTRL, 0xF, 0xF, true));
    }
    merge_desc<N>(a, b);
}

// The N largest of a token's L V logits, descending, on every of its lanes.
template <typename T, int L, int V, int N>
__device__ __forceinline__ void top_keys(const float (&v)[V], int lane, double (&top)[N]) {
    constexpr int M = V < N ? V : N;
#pragma unroll
    for (int c = 0; c < V; c += M) {
        double x[M], part[N];
#pragma unroll
        for (int i = 0; i < M; i++)   // with the last lane's index: the other lanes' bits follow below
            x[i] = logit_key(v[c + i], (uint32_t)(1023 - expert_of<T, L>(L - 1, c + i)));
        sort_desc<M>(x);
#pragma unroll
        for (int i = 0; i < N; i++) part[i] = i < M ? x[i] : make_key(kNoKey, 0);
        if (c == 0) {
#pragma unroll
            for (int i = 0; i < N; i++) top[i] = part[i];
        } else {
            merge_desc<N>(top, part);
        }
    }
    // (piece, lane, element) are bit fields of the index
    const uint32_t mine = (uint32_t)((L - 1 - lane) * kPiece<T>);
#pragma unroll
    for (int i = 0; i < N; i++) top[i] = make_key(key_hi(top[i]), key_lo(top[i]) ^ mine);
    if (L == 32) {
        double b[N];
#pragma unroll
        for (int i = 0; i < N; i++) b[i] = __shfl_xor(top[i], 16, 64);
        merge_desc<N>(top, b);
    }
    if (L >= 16) merge_dpp<N, DPP_MIRROR16>(top);
    if (L >= 8) merge_dpp<N, DPP_MIRROR8>(top);
    merge_dpp<N, DPP_XOR2>(top);
    merge_dpp<N, DPP_XOR1>(top);
}

struct RouteArgs {
    const void *logits;
    const uint8_t *mask;
    int64_t T, ldl;
    int32_t E, k, kk, G;
    bool norm;
    int32_t *experts, *counts, *src, *pos;
    float *weights, *row_weights, *prob_sum, *loss;
    int64_t *off;
    // workspace, one entry per workgroup (a run of CT consecutive tokens)
    int32_t CT, nwg, ldh, lde;
    void *hist;       // rows of each group, then routed tokens: [G + 1][ldh], u8 or (CT > 255) u16 to a run
    float *part;      // [nwg][lde]: sums of probabilities, zeros
    int32_t slice;    // quads of experts whose sums over the runs one workgroup takes: 1, 2, .. 32
    uint64_t *loss_sum;   // see route_sums
};

// Choice, weights, histogram and probability sums of tokens [t0, t1) by one
// workgroup of BT threads, L lanes to a token and k <= N.  hist: LDS [G + 1],
// left with this workgroup's counts; psum: LDS [kSumRows<L, BT>][E], the first
// row left with its probability sums.
template <int L, int BT>
constexpr int kSumRows = BT / (L < 16 ? 16 : L);
template <typename T, int L, int V, int N, int BT, bool VEC>
__device__ __forceinline__ void route_select(const RouteArgs &a, int64_t t0, int64_t t1, int32_t *hist, float *psum) {
    constexpr int KS = N / L > 0 ? N / L : 1;   // choices a lane writes
    constexpr int P = kParts<L, V> < KS ? kParts<L, V> : KS;
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    const bool aux = a.prob_sum != nullptr;
    for (int i = tid; i <= a.G; i += BT) hist[i] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    for (int64_t t = t0 + grp; t < t1; t += BT / L) {
        RowLoad<T, L, V, VEC> in;
        in.load(reinterpret_cast<const T *>(a.logits) + t * a.ldl, lane, a.E);
        const bool keep = !a.mask || a.mask[t];
        float v[V];
        in.get(lane, a.E, keep, v);
        double top[N];
        top_keys<T, L, V, N>(v, lane, top);
        const float best = key_logit(top[0]), m = best > -INFINITY ? best : 0.0f;
        const float sum = exp_sum<T, L, true>(v, m), inv = 1.0f / sum;   // sum >= 1 where routed
        const bool routed = sum > 0.0f, bad = sum != sum;
        if (aux && sum != 0.0f) {             // NaN in a bad row reaches prob_sum and loss
#pragma unroll
            for (int i = 0; i < V; i++) acc[i] = fmaf(v[i], inv, acc[i]);
        }
        int sel[KS];
        float val[KS], part[P] = {};
#pragma unroll
        for (int q = 0; q < KS; q++) {        // choice j = q L + lane
            double mine = top[q * L];
#pragma unroll
            for (int j = 1; j < L; j++)
                if (q * L + j < N) mine = lane == j ? top[q * L + j] : mine;
            const float x = key_logit(mine);
            const bool ok = q * L + lane < a.k && routed && x > -INFINITY;
            sel[q] = ok ? key_expert(mine) : -1;
            val[q] = ok ? exp_f32(x - m) : 0.0f;
            part[q % P] += val[q];
        }
        const float total = parts_sum<L, P>(part);
        const float scale = bad ? sum : !routed ? 0.0f : a.norm ? 1.0f / total : inv;
#pragma unroll
        for (int q = 0; q < KS; q++) {
            const int j = q * L + lane;
            if (j < a.k) {
                a.experts[t * a.kk + j] = sel[q];
                a.weights[t * a.kk + j] = bad ? scale : val[q] * scale;
                if (sel[q] >= 0) atomicAdd(&hist[sel[q]], 1);
            }
        }
        for (int j = a.k + lane; j < a.kk; j += L) {
            const int g = a.E + j - a.k;
            a.experts[t * a.kk + j] = routed ? g : -1;
            a.weights[t * a.kk + j] = routed ? 1.0f : 0.0f;
            if (routed) atomicAdd(&hist[g], 1);
        }
        if (lane == 0 && routed) atomicAdd(&hist[a.G], 1);
    }
    if (aux) {
        // tokens' sums in a fixed order: the lane groups of a row of 16, then rows
#pragma unroll
        for (int i = 0; i < V; i++) {
            if (L < 16) acc[i] += dpp<DPP_ROR8>(acc[i]);
            if (L < 8) acc[i] += dpp<DPP_ROR4>(acc[i]);
        }
        constexpr int W = L < 16 ? 16 : L;    // lanes to a row of psum
        constexpr int Q = kPiece<T>;
        if ((tid & (W - 1)) < L) {
#pragma unroll
            for (int i = 0; i < V; i += Q) {
                const int e = expert_of<T, L>(lane, i);
                if (VEC) {
                    if (e < a.E)
#pragma unroll
                        for (int q = 0; q < Q; q += 4)
                            *reinterpret_cast<float4 *>(psum + tid / W * a.E + e + q) =
                                make_float4(acc[i + q], acc[i + q + 1], acc[i + q + 2], acc[i + q + 3]);
                } else {
#pragma unroll
                    for (int q = 0; q < Q; q++)
                        if (e + q < a.E) psum[tid / W * a.E + e + q] = acc[i + q];
                }
            }
        }
        __syncthreads();
        // the rows in `parts` interleaved shares, then the shares
        const int parts = BT / a.E < 1 ? 1 : BT / a.E < 8 ? BT / a.E : 8;
        float s[BT < L * V ? L * V / BT : 1];
#pragma unroll
        for (int c = 0; c < (BT < L * V ? L * V / BT : 1); c++) {
            const int i = c * BT + tid, q = i / a.E, e = i - q * a.E;
            s[c] = 0.0f;
            if (q < parts)
                for (int w = q; w < kSumRows<L, BT>; w += parts) s[c] += psum[w * a.E + e];
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < (BT < L * V ? L * V / BT : 1); c++)
            if (c * BT + tid < parts * a.E) psum[c * BT + tid] = s[c];
        __syncthreads();
        if (parts > 1 && tid < a.E) {
            for (int q = 1; q < parts; q++) s[0] += psum[q * a.E + tid];
            psum[tid] = s[0];
        }
    }
    __syncthreads();
}

// Expert e's part of the loss but for the factor E / k: (c_e / n) (Q_e / n).
// n = 0: nothing was routed; 0, or NaN if that was for bad rows.
__device__ __forceinline__ float loss_term(int32_t c, float q, int32_t n) {
    return n == 0 ? q : ((float)c / (float)n) * (q / (float)n);
}
// Loss from the batch's counts and probability sums (LDS), by one wavefront.
__device__ void route_loss(const RouteArgs &a, const int32_t *tot, const float *q) {
    const int lane = threadIdx.x & 63;
    float s = 0.0f;
    for (int e = lane; e < a.E; e += 64) s += loss_term(tot[e], q[e], tot[a.G]);
    s = wave_sum(s);
    if (lane == 0) *a.loss = s * ((float)a.E / (float)a.k);
}

// Inclusive sum over the lanes up to this one, by DPP: within rows of 16, then
// the rows' totals to the rows after them.
__device__ __forceinline__ int32_t wave_scan(int32_t v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);    // row_shr 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // lane 15 of a row to the next row
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // lane 31 to the upper rows
    return v;
}

// Exclusive scan of in[0, n) (LDS, n <= kMaxGroups) by a workgroup of NT threads:
// f(i, sum of the entries before i) for every i; returns the total.  f may
// store to in.  One wavefront alone, with up to 17 entries to a lane, took 1400
// cycles for 256 entries, 2300 for 512 and 4900 for 1000; this takes 1100 to 1400.
template <int NT, typename F>
__device__ __forceinline__ int32_t exclusive_scan(const int32_t *in, int n, F f) {
    constexpr int PER = (kMaxGroups + NT - 1) / NT, WAVES = NT / 64;
    __shared__ int32_t wave_total[WAVES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = (n + NT - 1) / NT, i0 = threadIdx.x * per;
    int32_t v[PER], sum = 0;
#pragma unroll
    for (int q = 0; q < PER; q++) {
        v[q] = q < per && i0 + q < n ? in[i0 + q] : 0;
        sum += v[q];
    }
    const int32_t incl = wave_scan(sum);
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    const int32_t upto = wave_scan(lane < WAVES ? wave_total[lane] : 0);
    int32_t run = incl - sum + (wave > 0 ? __builtin_amdgcn_readlane(upto, wave - 1) : 0);
#pragma unroll
    for (int q = 0; q < PER; q++) {
        if (q < per && i0 + q < n) f(i0 + q, run);
        run += v[q];
    }
    return __builtin_amdgcn_readlane(upto, WAVES - 1);
}

// Rows of tokens [t0, t1): base[g] is the first row of group g's choices in
// this run (LDS, advanced here).  Every (group, token) is one bit of an LDS
// table, W words of 32 tokens to a group, so a choice's rank among the run's
// is a population count: rows come out ordered by token whatever the order of
// execution.  A thread holds H choices; the first pass's are loaded ahead of
// the caller's other work.
//
// Longer runs (W >= 8) keep the ranks of the words' first bits beside the
// table (adding up to 16 words for every choice took longer than the rest), and
// put the rows in order in LDS to write them group by group: a scattered
// 4-byte store is an L2 request of its own, and at 600018 choices those of src
// and row_weights took 3 of 13.5 us; in runs of several rows to a group
// neighbouring lanes share requests.
template <int H, int NT>
struct Choices {
    int g[H];
    float w[H];
    __device__ __forceinline__ void load(const RouteArgs &a, int64_t s0, int n) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int h = 0; h < H; h++) {
            g[h] = -1;
            w[h] = 0.0f;
            if (h * NT < n) {
                const int i = h * NT + tid;
                const int64_t c = s0 * a.kk + (i < n ? i : 0);
                g[h] = a.experts[c];   // not looked at here: that would wait for it
                w[h] = a.weights[c];
            }
        }
    }
    // group of choice h of a pass of n, -1 for none
    __device__ __forceinline__ int group(int h, int n) const {
        return h * NT + (int)threadIdx.x < n ? g[h] : -1;
    }
};
template <int H, int NT, int W, int GROUPS>
struct PlaceTable {
    static constexpr bool LONG = W >= 8;
    // Strides: rows of 16 bytes' alignment that start at 16 different banks, an
    // odd multiple of four words.  With rows of 16 words the choices of a
    // wavefront, random groups and one word of each, met at four banks: placing
    // 131072 x 256, top-8, took 14.4 us instead of 13.4.
    static constexpr int BS = LONG ? W + 4 : W, RS = W % 16 == 0 ? W + 8 : W;
    __attribute__((aligned(16))) uint32_t bits[GROUPS * BS];
    __attribute__((aligned(16))) uint16_t rank[LONG ? GROUPS * RS : 8];   // of a word's first bit
    int32_t first[LONG ? GROUPS + 1 : 1];                               // of a group, in the order of rows
    int32_t row[LONG ? H * NT : 1], token[LONG ? H * NT : 1];
    float weight[LONG ? H * NT : 1];
    // tokens of one pass: as many as the threads hold choices of and the table has bits for
    __device__ static __forceinline__ int step(const RouteArgs &a) {
        const int held = H * NT / a.kk;
        return held < 32 * W ? held : 32 * W;
    }
    __device__ __forceinline__ void clear(const RouteArgs &a) {
        for (int i = threadIdx.x; i < a.G * BS; i += NT) bits[i] = 0;
    }
};
// The table has been cleared, and a barrier passed since.
template <int H, int NT, int W, int GROUPS>
__device__ __forceinline__ void route_place(const RouteArgs &a, int64_t t0, int64_t t1, int32_t *base,
                                            PlaceTable<H, NT, W, GROUPS> &tab, Choices<H, NT> &c) {
    constexpr bool LONG = W >= 8;
    constexpr int BS = PlaceTable<H, NT, W, GROUPS>::BS, RS = PlaceTable<H, NT, W, GROUPS>::RS;
    const int tid = threadIdx.x;
    const int step = tab.step(a);
    const int dq = NT / a.kk, dr = NT - dq * a.kk;
    for (int64_t s0 = t0;;) {
        const int n = (int)(t1 - s0 < step ? t1 - s0 : step) * a.kk;
        int tok[H];                                  // token (of the pass) of choice h NT + tid
        {
            int t = tid / a.kk, r = tid - t * a.kk;
#pragma unroll
            for (int h = 0; h < H; h++) {
                tok[h] = t;
                const int g = c.group(h, n);
                if (g >= 0) atomicOr(&tab.bits[g * BS + (t >> 5)], 1u << (t & 31));
                t += dq + (r + dr >= a.kk ? 1 : 0);
                r += dr - (r + dr >= a.kk ? a.kk : 0);
            }
        }
        // All loads have arrived: below, waiting for one would wait for the stores before it as well.
#pragma unroll
        for (int h = 0; h < H; h++) asm volatile("" : "+v"(c.w[h]));
        __syncthreads();
        if constexpr (LONG) {
            for (int g = tid; g < a.G; g += NT) {
                uint32_t k = 0;
#pragma unroll
                for (int x = 0; x < W; x += 8) {
                    const uint4 lo = *reinterpret_cast<const uint4 *>(tab.bits + g * BS + x);
                    const uint4 hi = *reinterpret_cast<const uint4 *>(tab.bits + g * BS + x + 4);
                    const uint32_t b[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    uint32_t r[4];
#pragma unroll
                    for (int y = 0; y < 8; y += 2) {
                        const uint32_t k1 = k + __popc(b[y]);
                        r[y / 2] = k | (k1 << 16);
                        k = k1 + __popc(b[y + 1]);
                    }
                    *reinterpret_cast<uint4 *>(tab.rank + g * RS + x) = make_uint4(r[0], r[1], r[2], r[3]);
                }
                tab.first[g] = (int32_t)k;
            }
            __syncthreads();
            const int32_t rows = exclusive_scan<NT>(tab.first, a.G, [&](int g, int32_t sum) { tab.first[g] = sum; });
            if (tid == 0) tab.first[a.G] = rows;
            __syncthreads();
        }
#pragma unroll
        for (int h = 0; h < H; h++) {
            const int i = h * NT + tid, g = c.group(h, n), t = tok[h];
            int32_t p = -1;
            if (g >= 0) {
                const uint32_t *b = tab.bits + g * BS;
                int rank = __popc(b[t >> 5] & ((1u << (t & 31)) - 1u));
                if constexpr (LONG) {
                    rank += tab.rank[g * RS + (t >> 5)];
                } else {
                    for (int x = 0; x < W - 1; x++) rank += x < t >> 5 ? __popc(b[x]) : 0;
                }
                p = base[g] + rank;
                if constexpr (LONG) {
                    const int slot = tab.first[g] + rank;
                    tab.row[slot] = p;
                    tab.token[slot] = (int32_t)(s0 + t);
                    tab.weight[slot] = c.w[h];
                } else {
                    a.src[p] = (int32_t)(s0 + t);
                    a.row_weights[p] = c.w[h];
                }
            }
            if (i < n) a.pos[s0 * a.kk + i] = p;
        }
        const bool more = s0 + step < t1;
        if (more) c.load(a, s0 + step, (int)(t1 - s0 - step < step ? t1 - s0 - step : step) * a.kk);
        if constexpr (LONG) {
            __syncthreads();
            for (int i = tid; i < tab.first[a.G]; i += NT) {
                const int32_t p = tab.row[i];
                a.src[p] = tab.token[i];
                a.row_weights[p] = tab.weight[i];
            }
        }
        if (!more) return;
        s0 += step;
        __syncthreads();
        for (int i = tid; i < a.G; i += NT)
            for (int x = 0; x < W; x++) base[i] += __popc(tab.bits[i * BS + x]);
        __syncthreads();
        tab.clear(a);
        __syncthreads();
    }
}

__device__ void route_tail(const RouteArgs &a, int64_t used, int64_t i0, int64_t step) {
    for (int64_t r = used + i0; r < a.T * a.kk; r += step) {
        a.src[r] = -1;
        a.row_weights[r] = 0.0f;
    }
}

// Where the groups start, from the totals tot (LDS): counts and offsets for the
// caller if `publish`, base[g] the start plus before[g] (LDS); returns the rows
// in use.  The caller synchronizes.
template <int NT>
__device__ __forceinline__ int64_t route_offsets(const RouteArgs &a, const int32_t *tot, const int32_t *before,
                                                 int32_t *base, bool publish) {
    const int32_t used = exclusive_scan<NT>(tot, a.G, [&](int g, int32_t start) {
        base[g] = start + (before ? before[g] : 0);
        if (publish) {
            a.counts[g] = tot[g];
            a.off[g] = start;
        }
    });
    if (publish && threadIdx.x == 0) {
        a.counts[a.G] = tot[a.G];
        a.off[a.G] = used;
    }
    return used;
}

// Sum over four or eight neighbouring lanes, on all of them.
template <int L>
__device__ __forceinline__ int32_t lanes_sum(int32_t v) {
    if (L == 8) v += __builtin_amdgcn_mov_dpp(v, DPP_MIRROR8, 0xF, 0xF, true);
    v += __builtin_amdgcn_mov_dpp(v, DPP_XOR2, 0xF, 0xF, true);
    return v + __builtin_amdgcn_mov_dpp(v, DPP_XOR1, 0xF, 0xF, true);
}

// First launch, bound by the vector units (8192 x 128 5.6 us, 100003 x 96 15.4 us,
// of which 8.7 are the issue of its vector instructions).  A batch of one run of at most ONE tokens is finished here, by
// its one workgroup (ONE = 0: there are more runs).
template <typename T, int L, int V, int N, int BT, int ONE, bool VEC>
__global__ __launch_bounds__(BT) void k_route_select(RouteArgs a) {
    __shared__ int32_t hist[L * V + kMaxShared + 1];
    __shared__ __attribute__((aligned(16))) float psum[kSumRows<L, BT> * L * V];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * a.CT, t1 = t0 + a.CT < a.T ? t0 + a.CT : a.T;
    route_select<T, L, V, N, BT, VEC>(a, t0, t1, hist, psum);
    if constexpr (ONE > 0) {
        constexpr int H = 4;
        __shared__ int32_t base[L * V + kMaxShared];
        __shared__ PlaceTable<H, BT, ONE / 32, L * V + kMaxShared> tab;
        Choices<H, BT> c;
        const int step = tab.step(a);
        c.load(a, 0, (int)(a.T < step ? a.T : step) * a.kk);
        tab.clear(a);
        if (a.prob_sum) {
            for (int e = tid; e < a.E; e += BT) a.prob_sum[e] = psum[e];
            if (tid < 64) route_loss(a, hist, psum);
        }
        const int64_t used = route_offsets<BT>(a, hist, nullptr, base, true);
        __syncthreads();
        route_place(a, 0, a.T, base, tab, c);
        route_tail(a, used, tid, BT);
    } else {
        for (int i = tid; i <= a.G; i += BT) {
            const int64_t at = (int64_t)i * a.ldh + blockIdx.x;
            if (a.CT > 255) reinterpret_cast<uint16_t *>(a.hist)[at] = (uint16_t)hist[i];
            else reinterpret_cast<uint8_t *>(a.hist)[at] = (uint8_t)hist[i];
        }
        if (a.prob_sum) {
            if (blockIdx.x == 0 && tid == 0) *a.loss_sum = 0;
            for (int e = tid; e < a.lde; e += BT)
                a.part[(int64_t)blockIdx.x * a.lde + e] = e < a.E ? psum[e] : 0.0f;
        }
    }
}

// Sums over all runs, and over the runs before run b, of the histograms'
// columns [c0, c0 + n) and G into tot and before (LDS [n + 1]).  Four (u16: eight) lanes take a
// column, 256 runs of it in flight (a batch has no more up to 16.7 million
// tokens) and the next column's behind them.  A word of a column is four (u16: two) runs, so one dot
// product adds them to the total and one, with weights that end at run b, to
// what precedes it: 2 instructions for 4 counts.  With the columns of a run side
// by side, masked and added as pairs of 16 bits (10 instructions for 4 counts),
// the sums took 7100 cycles for 257 columns and 10900 for 513.
template <typename HT, int NT>
__device__ __forceinline__ void route_totals(const RouteArgs &a, int b, int c0, int n, int32_t *tot, int32_t *before) {
    constexpr int SZ = (int)sizeof(HT), PW = 4 / SZ, L = 4 * SZ, U = 4, RUNS = 256;
    const auto weights = [](int n) -> uint32_t {   // 1 for the first n runs of a word
        const uint32_t one = SZ == 1 ? 0x01010101u : 0x00010001u;
        return n <= 0 ? 0u : n >= PW ? one : one & ((1u << (8 * SZ * n)) - 1u);
    };
    const auto dot = [](uint32_t x, uint32_t w, uint32_t s) -> uint32_t {
        if constexpr (SZ == 1) {
            return __builtin_amdgcn_udot4(x, w, s, false);
        } else {
            typedef unsigned short u16v2 __attribute__((ext_vector_type(2)));
            return __builtin_amdgcn_udot2(__builtin_bit_cast(u16v2, x), __builtin_bit_cast(u16v2, w), s, false);
        }
    };
    const int lane = threadIdx.x & (L - 1), q0 = threadIdx.x / L;
    const auto pass = [&](int r0) {
        uint32_t all[4 * U], pre[4 * U];
#pragma unroll
        for (int i = 0; i < 4 * U; i++) {
            const int r = r0 + ((i / 4) * L + lane) * 4 * PW + i % 4 * PW;
            all[i] = weights(a.nwg - r);
            pre[i] = weights(b - r);
        }
        const auto load = [&](int q, uint4 (&h)[U]) {
            const uint4 *x = reinterpret_cast<const uint4 *>(
                reinterpret_cast<const HT *>(a.hist) + (int64_t)(q < n ? c0 + q : a.G) * a.ldh + r0) + lane;
#pragma unroll
            for (int u = 0; u < U; u++) h[u] = x[r0 + 64 * u < a.ldh ? L * u : 0];
        };
        uint4 next[U];
        load(q0, next);
        for (int q = q0; q <= n; q += NT / L) {
            uint4 h[U];
#pragma unroll
            for (int u = 0; u < U; u++) h[u] = next[u];
            if (q + NT / L <= n) load(q + NT / L, next);
            uint32_t s[4] = {0, 0, 0, 0}, sb[4] = {0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < U; u++) {
                const uint32_t w[4] = {h[u].x, h[u].y, h[u].z, h[u].w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    s[i] = dot(w[i], all[4 * u + i], s[i]);
                    sb[i] = dot(w[i], pre[4 * u + i], sb[i]);
                }
            }
            const int32_t v = lanes_sum<L>((int32_t)(s[0] + s[1] + s[2] + s[3]));
            const int32_t vb = lanes_sum<L>((int32_t)(sb[0] + sb[1] + sb[2] + sb[3]));
            if (lane == 0) tot[q] = (r0 ? tot[q] : 0) + v;
            if (lane == 1) before[q] = (r0 ? before[q] : 0) + vb;
        }
    };
    pass(0);   // out of the loop, whose head would wait for the caller's loads
    for (int r0 = RUNS; r0 < a.nwg; r0 += RUNS) pass(r0);
    __syncthreads();
}

// The sums of the probabilities over the runs and the loss.  Workgroup i takes
// the quads of experts [i S, +S), S = a.slice; 64 / S runs are on a wavefront.
// Eight workgroups, beside those that place the rows: one alone was the last to
// finish by 3.4 us for 256 runs of 256 experts and by 16 for 1000.  Their parts
// of the loss, at most 1 together, meet in one 64-bit integer: 56 bits of the
// sum in units of 2^-54, then how many parts are NaN, then how many have been
// added, 4 bits each.  An integer sum has no order, and whoever's addition is
// the last has the whole loss in hand without reading what others stored
// (storing the parts and counting them with release and acquire took 3.5 us).
// The sum is at least 1 / E^2 (a token's largest probability is at least 1 / E),
// so eight parts rounded to 2^-54 are finer than f32.  tot, scratch: LDS
// [4 S + 1]; red: LDS [NT / 64][S].
template <typename HT, int NT>
__device__ __forceinline__ void route_sums(const RouteArgs &a, int i, int32_t *tot, int32_t *scratch, float4 *red) {
    constexpr int U = 4;
    const int S = a.slice, quads = a.lde / 4, q0 = i * S;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = threadIdx.x & (S - 1), q = q0 + col < quads ? q0 + col : 0;
    const float4 *x = reinterpret_cast<const float4 *>(a.part) + q;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int w = threadIdx.x / S; w < a.nwg; w += U * (NT / S)) {
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; u++) v[u] = x[(int64_t)(w + u * (NT / S) < a.nwg ? w + u * (NT / S) : 0) * quads];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const bool in = w + u * (NT / S) < a.nwg;
            s.x += in ? v[u].x : 0.0f;
            s.y += in ? v[u].y : 0.0f;
            s.z += in ? v[u].z : 0.0f;
            s.w += in ? v[u].w : 0.0f;
        }
    }
    for (int o = 32; o >= S; o >>= 1) {
        s.x += __shfl_xor(s.x, o, 64);
        s.y += __shfl_xor(s.y, o, 64);
        s.z += __shfl_xor(s.z, o, 64);
        s.w += __shfl_xor(s.w, o, 64);
    }
    if (lane < S) red[wave * S + lane] = s;
    const int n = a.E - 4 * q0 < 4 * S ? a.E - 4 * q0 : 4 * S;   // experts
    route_totals<HT, NT>(a, 0, 4 * q0, n, tot, scratch);
    if (wave != 0) return;
    float loss = 0.0f;
    if (4 * lane < n) {
        s = red[lane];
        for (int w = 1; w < NT / 64; w++) {
            const float4 v = red[w * S + lane];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int e = 4 * (q0 + lane) + j;
            if (e < a.E) {
                a.prob_sum[e] = v[j];
                loss += loss_term(tot[4 * lane + j], v[j], tot[n]);
            }
        }
    }
    loss = wave_sum(loss);
    if (lane != 0) return;
    const uint64_t mine = (1ull << 60) | (loss == loss ? (uint64_t)(loss * 0x1p54f) : 1ull << 56);
    const uint64_t all =
        mine + __hip_atomic_fetch_add(a.loss_sum, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((int)(all >> 60) != (quads + S - 1) / S) return;
    const float sum = (float)(all & ((1ull << 56) - 1)) * 0x1p-54f;
    *a.loss = (all >> 56) & 15 ? NAN : sum * ((float)a.E / (float)a.k);
}

// Second launch: workgroup b < nwg places the rows of its run, those after them
// sum the probabilities.  Every workgroup adds up the histograms of all runs by
// itself (what precedes its run, and the totals): about 256 bytes or 2-byte
// words for each of G + 1 columns from L2, which is less than a third launch
// costs.  Bound by the latency of its phases: 8192 x 128 5.8 us, 8192 x 512 6.6,
// 100003 x 96 8.6, of which the histograms' round trip and sums are about 2.
template <int NT, int W, int GROUPS>   // wavefronts per SIMD: the largest table leaves room for one workgroup of 512
constexpr int kPlaceWaves = NT == 512 && W == 8 && GROUPS == kMaxGroups ? 2 : 4;
template <typename HT, int NT, int W, int GROUPS>
__global__ __launch_bounds__(NT, (kPlaceWaves<NT, W, GROUPS>)) void k_route_place(RouteArgs a) {
    constexpr int H = 4;
    __shared__ int32_t tot[GROUPS + 1], before[GROUPS + 1], base[GROUPS];
    __shared__ PlaceTable<H, NT, W, GROUPS> tab;
    const int tid = threadIdx.x, b = blockIdx.x;
    if (b >= a.nwg) {
        __shared__ float4 red[NT / 64 * kMaxSlice];
        route_sums<HT, NT>(a, b - a.nwg, tot, before, red);
        return;
    }
    const int64_t t0 = (int64_t)b * a.CT, t1 = t0 + a.CT < a.T ? t0 + a.CT : a.T;
    Choices<H, NT> c;
    const int step = tab.step(a);
    c.load(a, t0, (int)(t1 - t0 < step ? t1 - t0 : step) * a.kk);
    tab.clear(a);
    route_totals<HT, NT>(a, b, 0, a.G, tot, before);
    const int64_t used = route_offsets<NT>(a, tot, before, base, b == 0);
    __syncthreads();
    route_place(a, t0, t1, base, tab, c);
    route_tail(a, used, (int64_t)b * NT + tid, (int64_t)a.nwg * NT);
}

static int32_t round_up(int64_t n, int64_t m) { return (int32_t)((n + m - 1) / m * m); }

// Runs of whole words of tokens, about one to a compute unit (the placing reads
// every run's histogram in every workgroup), with counts below 2^16.  Where a
// compute unit holds one workgroup of the placing, eight are left to the sums.
static void route_runs(int64_t T, int64_t E, int64_t k, int64_t shared, int32_t &CT, int32_t &nwg) {
    const int64_t one = k <= 8 && E <= 256 ? kOneLargeTokens : kOneSmallTokens;
    CT = T <= one ? (int32_t)one : T >= 248 * 65504ll ? 65504 : round_up((T + 255) / 256, 32);
    if (T > one && T < 248 * 65504ll && (CT > 255 || (CT > 32 && E + shared > kFewGroups)))
        CT = round_up((T + 255 - kSums) / (256 - kSums), 32);
    nwg = (int32_t)((T + CT - 1) / CT);
}

// Runs from one column of the histograms to the next: what four lanes (of two
// bytes: eight) load at a time.
static int32_t hist_stride(int32_t nwg) { return round_up(nwg, 64); }

int64_t route_workspace_bytes(int64_t T, int64_t E, int64_t k, int64_t shared) {
    int32_t CT, nwg;
    route_runs(T, E, k, shared, CT, nwg);
    if (nwg == 1) return 0;
    return (E + shared + 1) * hist_stride(nwg) * (CT > 255 ? 2 : 1) + 4ll * nwg * round_up(E, 4) + 8;
}

template <typename T, int L, int V, int N, bool VEC>
static void route_launch_few(const RouteArgs &a, hipStream_t s) {
    // threads: 8192 x 512 12.0 us with 256, 11.1 with 512, 65536 x 512 52.0 and 42.7 (8192 x 128, whose runs
    // fill 256, 5.4 and 5.6); the longer lists need the registers
    constexpr int B = N == 8 ? 512 : 256;
    if (a.T <= kOneSmallTokens) {
        k_route_select<T, L, V, N, 256, kOneSmallTokens, VEC><<<1, 256, 0, s>>>(a);
    } else if (a.nwg > 1) {
        k_route_select<T, L, V, N, B, 0, VEC><<<a.nwg, B, 0, s>>>(a);
    } else {
        constexpr int B1 = VEC ? 1024 : 512;   // what the registers allow
        if constexpr (N == 8 && L * V <= 256) k_route_select<T, L, V, N, B1, kOneLargeTokens, VEC><<<1, B1, 0, s>>>(a);
    }
}
template <typename T, int L, int V, bool VEC>
static void route_few(const RouteArgs &a, hipStream_t s) {
    if (a.k <= 8) route_launch_few<T, L, V, 8, VEC>(a, s);
    else if (a.k <= 16) route_launch_few<T, L, V, 16, VEC>(a, s);
    else route_launch_few<T, L, V, 32, VEC>(a, s);
}
// Lanes and logits to a lane, f32, choice of 8192 tokens: 64 experts 4.9 us with
// 8 x 8 and 5.6 with 16 x 4; 128: 5.6 with 8 x 16, 6.0 with 16 x 8; 256: 7.1 with
// 16 x 16, 9.0 with 32 x 8; 512: 11.1 with 16 x 32, 11.9 with 32 x 16 (65536
// tokens: 42.7 and 59.6).
template <typename T, bool VEC>
static void route_few_experts(const RouteArgs &a, hipStream_t s) {
    if (a.E <= 64) route_few<T, 8, 8, VEC>(a, s);
    else if (a.E <= 128) route_few<T, 8, 16, VEC>(a, s);
    else if (a.E <= 256) route_few<T, 16, 16, VEC>(a, s);
    else if (a.E <= 512) route_few<T, 16, 32, VEC>(a, s);
    else route_few<T, 32, 32, VEC>(a, s);
}

// Many tokens: four or eight lanes to a token, with as many logits each as the
// experts need (in eights), so that a wavefront's instructions cover 16 or 8
// tokens and the lists cross two or three steps between lanes.  Measured at
// 100003 x 96: choice 15.4 us with 4 lanes of 24 logits, 18.4 with 4 of 32, 20.9
// with 8 of 16 and 29.7 with 16 of 8; at 8192 x 128, where the wavefronts are
// too few to fill the GPU, 8 lanes take 5.6 us and 4 lanes 7.1.
constexpr int kManyThreads = 768;
template <typename T, int L, int V>
static void route_many(const RouteArgs &a, hipStream_t s) {
    k_route_select<T, L, V, 8, kManyThreads, 0, true><<<a.nwg, kManyThreads, 0, s>>>(a);
}
template <typename T>
static void route_dispatch(const RouteArgs &a, bool vec, hipStream_t s) {
    if (a.T >= kManyTokens && a.k <= 8 && a.E <= 256 && vec) {
        if (a.E <= 32) route_many<T, 4, 8>(a, s);
        else if (a.E <= 64) route_many<T, 4, 16>(a, s);
        else if (a.E <= 96) route_many<T, 4, 24>(a, s);
        else if (a.E <= 128) route_many<T, 4, 32>(a, s);
        else if (a.E <= 192) route_many<T, 8, 24>(a, s);
        else route_many<T, 8, 32>(a, s);
    } else if (vec) {
        route_few_experts<T, true>(a, s);
    } else {
        route_few_experts<T, false>(a, s);
    }
    if (a.nwg == 1) return;
    const unsigned grid = (unsigned)(a.nwg + (a.prob_sum ? (a.lde / 4 + a.slice - 1) / a.slice : 0));
    if (a.CT > 255) {
        if (a.G <= kFewGroups) k_route_place<uint16_t, 1024, 16, kFewGroups><<<grid, 1024, 0, s>>>(a);
        else k_route_place<uint16_t, 1024, 8, kMaxGroups><<<grid, 1024, 0, s>>>(a);
    } else if (a.CT > 32) {
        if (a.G <= kFewGroups) k_route_place<uint8_t, 512, 8, kFewGroups><<<grid, 512, 0, s>>>(a);
        else k_route_place<uint8_t, 512, 8, kMaxGroups><<<grid, 512, 0, s>>>(a);
    } else {
        k_route_place<uint8_t, 512, 1, kMaxGroups><<<grid, 512, 0, s>>>(a);
    }
}

// Whole 16-byte pieces: pointers are 16-byte aligned (checked at the C ABI).
static bool whole_pieces(int64_t E, int64_t ld, int dtype) {
    const int64_t Q = dtype == BSP_DTYPE_BF16 ? 8 : 4;
    return ld % Q == 0 && E % Q == 0;
}

hipError_t launch_route(const void *logits, int dtype, int64_t T, int64_t E, int64_t ldl, const uint8_t *mask,
                        int64_t k, int64_t shared, int32_t *experts, float *weights, int32_t *counts, int64_t *off,
                        int32_t *src, int32_t *pos, float *row_weights, float *prob_sum, float *loss, bool norm,
                        void *workspace, hipStream_t s) {
    RouteArgs a;
    a.logits = logits; a.mask = mask; a.T = T; a.ldl = ldl;
    a.E = (int32_t)E; a.k = (int32_t)k; a.kk = (int32_t)(k + shared); a.G = (int32_t)(E + shared);
    a.norm = norm;
    const bool vec = whole_pieces(E, ldl, dtype);
    a.experts = experts; a.counts = counts; a.src = src; a.pos = pos;
    a.weights = weights; a.row_weights = row_weights; a.prob_sum = prob_sum; a.loss = loss; a.off = off;
    route_runs(T, E, k, shared, a.CT, a.nwg);
    a.ldh = hist_stride(a.nwg);
    a.lde = round_up(E, 4);
    a.hist = workspace;
    a.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) +
                                       (int64_t)(a.G + 1) * a.ldh * (a.CT > 255 ? 2 : 1));
    a.loss_sum = reinterpret_cast<uint64_t *>(a.part + (int64_t)a.nwg * a.lde);
    a.slice = 1;
    while (a.slice * kSums < a.lde / 4) a.slice *= 2;
    if (dtype == BSP_DTYPE_BF16) route_dispatch<uint16_t>(a, vec, s);
    else route_dispatch<float>(a, vec, s);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Gradient to the logits
// ---------------------------------------------------------------------------
//
// With p recomputed: the loss gives d_loss E / (k n^2) p (c - sum_e c_e p_e);
// the weights' gradient dw_j at the chosen experts gives w_j (dw_j -
// sum_i w_i dw_i) there (renormalised), or p (dw - sum_j p_j dw_j) with dw = 0
// elsewhere.
struct RouteBwdArgs {
    const void *logits;
    const uint8_t *mask;
    void *d_logits;
    int64_t T, ldl, ldd, rows;
    int32_t E, k, kk, G;
    bool norm;
    const int32_t *experts, *pos, *counts;
    const float *d_weights, *d_loss;
};

// Bound by HBM, every logit read and written once (8192 x 128 f32 4.9 us; 65537 x
// 256 bf16 19.9 us, 3.7 TB/s): a wavefront's loads of a token's logits and choices
// go out together, then the gathers by the choice, and loading the next token's
// ahead of them gained nothing.  Per element the terms that every expert has are
// one multiply-add of the count and one product, e (c1 f - c2); the k chosen
// experts' own terms are added by the lane that holds the choice: it evaluates
// its logit again and stores over the row's element (the same wavefront's store,
// issued later).
template <typename T, int L, int V, bool VEC>
__global__ __launch_bounds__(256) void k_route_bwd(RouteBwdArgs a) {
    constexpr int KS = 32 / L;                // choices per lane, k <= 32
    constexpr int P = kParts<L, V>;
    constexpr bool kFull = sizeof(T) == 4;    // a bf16 gradient's rounding hides the difference
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    const int32_t n = a.counts[a.G];
    const float rn = 1.0f / (n > 0 ? (float)n : 1.0f);
    const float coef = a.d_loss ? *a.d_loss * ((float)a.E / (float)a.k) * rn : 0.0f;
    float f[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = expert_of<T, L>(lane, i);
        f[i] = (float)a.counts[e < a.E ? e : 0] * rn;
    }
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + grp; t < a.T; t += (int64_t)gridDim.x * (256 / L)) {
        const T *in = reinterpret_cast<const T *>(a.logits) + t * a.ldl;
        T *out = reinterpret_cast<T *>(a.d_logits) + t * a.ldd;
        RowLoad<T, L, V, VEC> rows;
        rows.load(in, lane, a.E);
        const bool keep = !a.mask || a.mask[t];
        // choice j = q L + lane: expert, then its logit, count and gradient
        int ex[KS], cnt[KS];
        float x[KS], dw[KS];
#pragma unroll
        for (int q = 0; q < KS; q++) {
            ex[q] = -1;
            x[q] = -INFINITY;
            dw[q] = 0.0f;
            cnt[q] = 0;
            if (a.d_weights && q * L < a.k) {
                const int j = q * L + lane;
                const int64_t c = t * a.kk + (j < a.k ? j : 0);
                const int e = a.experts[c], r = a.pos[c];
                const bool ok = j < a.k && keep && e >= 0 && e < a.E && r >= 0 && r < a.rows;
                const float l = elem(in + (ok ? e : 0)), g = a.d_weights[ok ? r : 0];
                cnt[q] = a.counts[ok ? e : 0];
                ex[q] = ok ? e : -1;
                x[q] = ok ? l : -INFINITY;
                dw[q] = ok ? g : 0.0f;
            }
        }
        float v[V];
        rows.get(lane, a.E, keep, v);
        float m = v[0];
#pragma unroll
        for (int i = 1; i < V; i++) m = fmaxf(m, v[i]);
        m = group_max<L>(m);
        m = m > -INFINITY ? m : 0.0f;
        const float sum = exp_sum<T, L, kFull>(v, m), inv = sum == 0.0f ? 0.0f : recip<kFull>(sum);
        float dots[P] = {}, sums[P] = {}, grads[P] = {};
#pragma unroll
        for (int i = 0; i < V; i++) dots[i / kPiece<T> % P] = fmaf(v[i], f[i], dots[i / kPiece<T> % P]);
#pragma unroll
        for (int q = 0; q < KS; q++) {
            x[q] = exp_f32<kFull>(x[q] - m);
            sums[q % P] += x[q];
            grads[q % P] = fmaf(x[q], dw[q], grads[q % P]);
        }
        const float dot = parts_sum<L, P>(dots) * inv, ps = parts_sum<L, P>(sums), pd = parts_sum<L, P>(grads);
        // renormalised: chosen p / ps; else p itself, whose sum of p dw every expert feels
        const float scale = a.norm ? (ps > 0.0f ? recip<kFull>(ps) : 0.0f) : inv;
        const float c1 = coef * inv, c2 = c1 * dot + (a.norm ? 0.0f : inv * inv * pd);
#pragma unroll
        for (int i = 0; i < V; i++) v[i] *= fmaf(c1, f[i], -c2);
        store_logits<T, L, V, VEC>(out, lane, a.E, v);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < KS; q++)
            if (ex[q] >= 0) {
                const float fe = (float)cnt[q] * rn;
                put(out + ex[q], x[q] * (fmaf(c1, fe, -c2) + scale * (dw[q] - (a.norm ? pd * scale : 0.0f))));
            }
    }
}

template <typename T, int L, int V, bool VEC>
static void route_bwd_launch(const RouteBwdArgs &a, hipStream_t s) {
    const int64_t wgs = (a.T + 256 / L - 1) / (256 / L);
    const unsigned grid = (unsigned)(wgs < kBwdWorkgroups ? wgs : kBwdWorkgroups);
    k_route_bwd<T, L, V, VEC><<<grid, 256, 0, s>>>(a);
}
// Lanes and logits to a lane: 128 experts 8 x 16 (65536 tokens f32: 16.2 us, 16 x 8
// 18.0, 4 x 32 19.9; 32768 bf16: 9.1, 10.6, 9.5); 256 experts 16 x 16, in bf16 and
// with many tokens 8 x 32 (65537 bf16: 19.9 instead of 21.4; but 20000 f32 12.7
// instead of 12.2, and 4096 f32 5.7 instead of 5.1); 512 experts 32 x 16 (65536
// f32: 54.0, 16 x 32 58.6).
template <typename T, bool VEC>
static void route_bwd_dispatch(const RouteBwdArgs &a, hipStream_t s) {
    constexpr int Q = kPiece<T>;
    const bool many = Q == 8 && a.T >= kManyTokens;
    if (a.E <= 64) route_bwd_launch<T, 64 / Q, Q, VEC>(a, s);
    else if (a.E <= 128) route_bwd_launch<T, 8, 16, VEC>(a, s);
    else if (a.E <= 256 && many) route_bwd_launch<T, Q == 8 ? 8 : 16, Q == 8 ? 32 : 16, VEC>(a, s);
    else if (a.E <= 256) route_bwd_launch<T, 16, 16, VEC>(a, s);
    else if (a.E <= 512) route_bwd_launch<T, 32, 16, VEC>(a, s);
    else route_bwd_launch<T, 32, 32, VEC>(a, s);
}

hipError_t launch_route_backward(const void *logits, int dtype, int64_t T, int64_t E, int64_t ldl,
                                 const uint8_t *mask, int64_t k, int64_t shared, const int32_t *experts,
                                 const int32_t *pos, const int32_t *counts, const float *d_weights,
                                 const float *d_loss, void *d_logits, int64_t ldd, bool norm, hipStream_t s) {
    RouteBwdArgs a;
    a.logits = logits; a.mask = mask; a.d_logits = d_logits; a.T = T; a.ldl = ldl; a.ldd = ldd;
    a.E = (int32_t)E; a.k = (int32_t)k; a.kk = (int32_t)(k + shared); a.G = (int32_t)(E + shared);
    a.rows = T * (k + shared);
    a.norm = norm;
    const bool vec = whole_pieces(E, ldl, dtype) && whole_pieces(E, ldd, dtype);
    a.experts = experts; a.pos = pos; a.counts = counts; a.d_weights = d_weights; a.d_loss = d_loss;
    if (dtype == BSP_DTYPE_BF16 && vec) route_bwd_dispatch<uint16_t, true>(a, s);
    else if (dtype == BSP_DTYPE_BF16) route_bwd_dispatch<uint16_t, false>(a, s);
    else if (vec) route_bwd_dispatch<float, true>(a, s);
    else route_bwd_dispatch<float, false>(a, s);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Sum of a token's grouped rows
// ---------------------------------------------------------------------------

// Bound by HBM: every row once.  One thread per token and 16 bytes of a row of
// y, U rows' pieces in flight: batches of four, then two and one, so that no
// load is wasted (with a fixed batch of eight, 16384 x 2 rows of 4096 took 126
// us instead of 68).  An index without a row loads row 0, a line that stays in
// the cache, and counts as zeros.  Rows are loaded and results stored
// nontemporally, neither is used again here: 4096 x 9 rows of 7168 bf16 (a
// tenth dropped) 117 us cached, 99 with such loads, 93 with both (6.3 TB/s).
template <typename TI, int VE, int U>
__device__ __forceinline__ void combine_rows(const TI *__restrict__ y, int64_t rows, int64_t ldy,
                                             const int32_t *__restrict__ pos, const float *__restrict__ weights,
                                             float (&acc)[VE]) {
    u32v4 v[U];
    float w[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int32_t r = pos[u];
        ok[u] = r >= 0 && r < rows;
        v[u] = ld4w<true>(y + (ok[u] ? (int64_t)r * ldy : 0));
        w[u] = weights ? weights[u] : 1.0f;
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        w[u] = ok[u] ? w[u] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) v[u][i] = ok[u] ? v[u][i] : 0u;
#pragma unroll
        for (int q = 0; q < VE; q++) {
            const float x = VE == 4 ? __uint_as_float(v[u][q % 4])
                                    : q % 2 ? bf16_hi(v[u][q / 2 % 4]) : bf16_lo(v[u][q / 2 % 4]);
            acc[q] += w[u] * x;
        }
    }
}
template <typename TI, typename TO>
__global__ __launch_bounds__(256) void k_combine(const TI *__restrict__ y, int64_t rows, int64_t ldy,
                                                 const int32_t *__restrict__ pos, const float *__restrict__ weights,
                                                 int64_t T, int kk, int nc, TO *__restrict__ out, int64_t ldo) {
    constexpr int VE = 16 / (int)sizeof(TI);
    const int64_t i = grid_index() * 256 + threadIdx.x;
    const int64_t t = i / nc;
    if (t >= T) return;
    const int c = (int)(i - t * nc) * VE;
    float acc[VE];
#pragma unroll
    for (int q = 0; q < VE; q++) acc[q] = 0.0f;
    const int32_t *p = pos + t * kk;
    const float *w = weights ? weights + t * kk : nullptr;
    int j = 0;
#pragma unroll 1
    for (; j + 4 <= kk; j += 4) combine_rows<TI, VE, 4>(y + c, rows, ldy, p + j, w ? w + j : nullptr, acc);
    if (kk & 2) {
        combine_rows<TI, VE, 2>(y + c, rows, ldy, p + j, w ? w + j : nullptr, acc);
        j += 2;
    }
    if (kk & 1) combine_rows<TI, VE, 1>(y + c, rows, ldy, p + j, w ? w + j : nullptr, acc);
    TO *o = out + t * ldo + c;
    if constexpr (VE == 8) {
        st8<true>(o, acc);
    } else if constexpr (sizeof(TO) == 4) {
        st4w<true>(o, (u32v4){__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                              __float_as_uint(acc[3])});
    } else {
        st2<true>(o, make_uint2(bf16x2(acc[0], acc[1]), bf16x2(acc[2], acc[3])));
    }
}

template <typename TI, typename TO>
static void combine_launch(const void *y, int64_t rows, int64_t H, int64_t ldy, const int32_t *pos,
                           const float *weights, int64_t T, int64_t kk, void *out, int64_t ldo, hipStream_t s) {
    const int64_t nc = H * (int64_t)sizeof(TI) / 16, n = T * nc;
    k_combine<TI, TO><<<grid_of((n + 255) / 256), 256, 0, s>>>(reinterpret_cast<const TI *>(y), rows, ldy, pos,
                                                                 weights, T, (int)kk, (int)nc,
                                                                 reinterpret_cast<TO *>(out), ldo);
}

hipError_t launch_combine(const void *y, int in_dtype, int64_t rows, int64_t H, int64_t ldy, const int32_t *pos,
                          const float *weights, int64_t T, int64_t kk, void *out, int out_dtype, int64_t ldo,
                          hipStream_t s) {
    const bool bi = in_dtype == BSP_DTYPE_BF16, bo = out_dtype == BSP_DTYPE_BF16;
    if (bi && bo) combine_launch<uint16_t, uint16_t>(y, rows, H, ldy, pos, weights, T, kk, out, ldo, s);
    else if (bi) combine_launch<uint16_t, float>(y, rows, H, ldy, pos, weights, T, kk, out, ldo, s);
    else if (bo) combine_launch<float, uint16_t>(y, rows, H, ldy, pos, weights, T, kk, out, ldo, s);
    else combine_launch<float, float>(y, rows, H, ldy, pos, weights, T, kk, out, ldo, s);
    return hipGetLastError();
}

}  // namespace bsp
