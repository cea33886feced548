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

constexpr float kLog2e = 1.44269504088896341f;
constexpr int64_t kManyTokens = 32768;
constexpr int64_t kBwdWorkgroups = 1280;
constexpr int kRouteThreads = 512;   // workgroup of the placing
constexpr int kWords = 8;            // placing: tokens ranked at a time, in words of 32
constexpr int64_t kOneWorkgroupTokens = 64;
constexpr int kMaxShared = 64;
constexpr int kMaxGroups = 1024 + kMaxShared;

// Lane exchanges within a row of 16 by DPP.  A token's L lanes (4, 8, 16 or 32)
// reduce over mirror(16), mirror(8), xor 2, xor 1, each step joining two
// disjoint sets of lanes; L = 32 starts with the other row of 16.
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
    if (L == 32) v += __shfl_xor(v, 16, 64);
    if (L >= 16) v += dpp<DPP_MIRROR16>(v);
    if (L >= 8) v += dpp<DPP_MIRROR8>(v);
    v += dpp<DPP_XOR2>(v);
    return v + dpp<DPP_XOR1>(v);
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
__device__ __forceinline__ void ld16(const float *p, float *v) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
__device__ __forceinline__ void ld16(const uint16_t *p, float *v) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ void st16(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st16(uint16_t *p, const float *v) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                                               bf16x2(v[6], v[7]));
}
// -inf past E.  VEC: rows start on 16 bytes and E is a multiple of Q, so a
// piece is whole or absent.
template <typename T, int L, int V, bool VEC>
__device__ __forceinline__ void load_logits(const T *row, int lane, int E, float (&v)[V]) {
    constexpr int Q = kPiece<T>;
#pragma unroll
    for (int i = 0; i < V; i += Q) {
        const int e = expert_of<T, L>(lane, i);
        if (VEC && e < E) {
            ld16(row + e, v + i);
        } else {
#pragma unroll
            for (int q = 0; q < Q; q++) v[i + q] = !VEC && e + q < E ? elem(row + e + q) : -INFINITY;
        }
    }
}
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
template <int L, int V>
__device__ __forceinline__ float exp_sum(float (&v)[V], float m) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i++) {
        v[i] = __builtin_amdgcn_exp2f((v[i] - m) * kLog2e);
        s += v[i];
    }
    return group_sum<L>(s);
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
    int32_t *hist;    // [nwg][ldh]: rows of each group, routed tokens, zeros
    float *part;      // [nwg][lde]: sums of probabilities, zeros
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
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    const bool aux = a.prob_sum != nullptr;
    for (int i = tid; i <= a.G; i += BT) hist[i] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    for (int64_t t = t0 + grp; t < t1; t += BT / L) {
        float v[V];
        if (!a.mask || a.mask[t]) {
            load_logits<T, L, V, VEC>(reinterpret_cast<const T *>(a.logits) + t * a.ldl, lane, a.E, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = -INFINITY;
        }
        double top[N];
        top_keys<T, L, V, N>(v, lane, top);
        const float best = key_logit(top[0]), m = best > -INFINITY ? best : 0.0f;
        const float sum = exp_sum<L>(v, m), inv = 1.0f / sum;
        const bool routed = sum > 0.0f, bad = sum != sum;
        if (aux && sum != 0.0f) {             // NaN in a bad row reaches prob_sum and loss
#pragma unroll
            for (int i = 0; i < V; i++) acc[i] = fmaf(v[i], inv, acc[i]);
        }
        int sel[KS];
        float val[KS], total = 0.0f;
#pragma unroll
        for (int q = 0; q < KS; q++) {        // choice j = q L + lane
            double mine = top[q * L];
#pragma unroll
            for (int j = 1; j < L; j++)
                if (q * L + j < N) mine = lane == j ? top[q * L + j] : mine;
            const float x = key_logit(mine);
            const bool ok = q * L + lane < a.k && routed && x > -INFINITY;
            sel[q] = ok ? key_expert(mine) : -1;
            val[q] = ok ? __builtin_amdgcn_exp2f((x - m) * kLog2e) : 0.0f;
            total += val[q];
        }
        total = group_sum<L>(total);
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
        for (int e = tid; e < a.E; e += BT) {
            float s = 0.0f;
#pragma unroll 8
            for (int w = 0; w < kSumRows<L, BT>; w++) s += psum[w * a.E + e];
            psum[e] = s;
        }
    }
    __syncthreads();
}

// Loss from the batch's counts and probability sums (LDS), by one wavefront.
__device__ void route_loss(const RouteArgs &a, const int32_t *tot, const float *q) {
    const int lane = threadIdx.x & 63;
    float s = 0.0f;
    const float n = (float)tot[a.G];
    for (int e = lane; e < a.E; e += 64) s += ((float)tot[e] / n) * (q[e] / n);
    s = wave_sum(s);
    // n = 0: nothing was routed; 0, or NaN if that was for bad rows
    if (lane == 0) {
        float bad = 0.0f;
        if (tot[a.G] == 0) {
            for (int e = 0; e < a.E; e++) bad += q[e];
        }
        *a.loss = tot[a.G] == 0 ? bad : s * ((float)a.E / (float)a.k);
    }
}

// Group starts: exclusive scan of tot[0, G) into base (LDS), by the first
// wavefront; base[G] is the rows in use.
__device__ void route_starts(const RouteArgs &a, const int32_t *tot, int32_t *base) {
    if (threadIdx.x >= 64) return;
    const int lane = threadIdx.x;
    int32_t carry = 0;
    for (int g0 = 0; g0 <= a.G; g0 += 64) {
        const int g = g0 + lane;
        const int32_t c = g < a.G ? tot[g] : 0;
        int32_t v = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int32_t u = __shfl_up(v, o, 64);
            if (lane >= o) v += u;
        }
        if (g <= a.G) base[g] = carry + v - c;
        carry += __shfl(v, 63, 64);
    }
}

// Rows of tokens [t0, t1): base[g] is the first row of group g's choices in
// this run (LDS, advanced here).  Every (group, token) is one bit of an LDS
// table of 32 W tokens, so a choice's rank among the run's is a population
// count: rows come out ordered by token whatever the order of execution.
template <int W>
__device__ __forceinline__ void route_place(const RouteArgs &a, int64_t t0, int64_t t1, int32_t *base,
                                            uint32_t (*bits)[W]) {
    constexpr int H = 4;                      // choices a thread holds between the two passes
    const int tid = threadIdx.x, nt = blockDim.x;
    const int step = H * nt / a.kk < 32 * W ? H * nt / a.kk : 32 * W;
    int tok[H];                               // token (of the pass) of choice h nt + tid
    {
        const int dq = nt / a.kk, dr = nt - dq * a.kk;
        int q = tid / a.kk, r = tid - q * a.kk;
#pragma unroll
        for (int h = 0; h < H; h++) {
            tok[h] = q;
            r += dr;
            q += dq + (r >= a.kk ? 1 : 0);
            r -= r >= a.kk ? a.kk : 0;
        }
    }
    for (int64_t s0 = t0; s0 < t1; s0 += step) {
        const int n = (int)(t1 - s0 < step ? t1 - s0 : step) * a.kk;
        int g[H];
        float w[H];
#pragma unroll
        for (int h = 0; h < H; h++) {
            const int i = h * nt + tid;
            g[h] = i < n ? a.experts[s0 * a.kk + i] : -1;
            w[h] = i < n ? a.weights[s0 * a.kk + i] : 0.0f;
        }
        for (int i = tid; i < a.G * W; i += nt) bits[0][i] = 0;
        __syncthreads();
#pragma unroll
        for (int h = 0; h < H; h++) {
            if (g[h] >= 0) atomicOr(&bits[g[h]][tok[h] >> 5], 1u << (tok[h] & 31));
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < H; h++) {
            const int i = h * nt + tid, t = tok[h];
            int32_t p = -1;
            if (g[h] >= 0) {
                p = base[g[h]];
#pragma unroll
                for (int x = 0; x < W; x++) {
                    const uint32_t b = bits[g[h]][x];
                    p += __popc(x < t >> 5 ? b : x == t >> 5 ? b & ((1u << (t & 31)) - 1u) : 0u);
                }
                a.src[p] = (int32_t)(s0 + t);
                a.row_weights[p] = w[h];
            }
            if (i < n) a.pos[s0 * a.kk + i] = p;
        }
        if (s0 + step >= t1) return;
        __syncthreads();
        for (int i = tid; i < a.G; i += nt) {
#pragma unroll
            for (int x = 0; x < W; x++) base[i] += __popc(bits[i][x]);
        }
        __syncthreads();
    }
}

__device__ void route_tail(const RouteArgs &a, int64_t used, int64_t i0, int64_t step) {
    for (int64_t r = used + i0; r < a.T * a.kk; r += step) {
        a.src[r] = -1;
        a.row_weights[r] = 0.0f;
    }
}

__device__ __forceinline__ void route_counts(const RouteArgs &a, const int32_t *tot, const int32_t *base) {
    for (int i = threadIdx.x; i <= a.G; i += blockDim.x) {
        a.counts[i] = tot[i];
        a.off[i] = base[i];
    }
}

// First launch.  A batch of one run (T <= kOneWorkgroupTokens) is finished
// here, by its one workgroup (ONE).
template <typename T, int L, int V, int N, int BT, bool ONE, bool VEC>
__global__ __launch_bounds__(BT) void k_route_select(RouteArgs a) {
    constexpr int WORDS = kOneWorkgroupTokens / 32;
    constexpr int PSUM = kSumRows<L, BT> * L * V, BITS = ONE ? (L * V + kMaxShared) * WORDS : 0;
    __shared__ int32_t hist[L * V + kMaxShared + 1];
    __shared__ __attribute__((aligned(16))) uint32_t buf[PSUM > BITS ? PSUM : BITS];
    const int tid = threadIdx.x;
    float *psum = reinterpret_cast<float *>(buf);
    const int64_t t0 = (int64_t)blockIdx.x * a.CT, t1 = t0 + a.CT < a.T ? t0 + a.CT : a.T;
    route_select<T, L, V, N, BT, VEC>(a, t0, t1, hist, psum);
    if constexpr (ONE) {
        __shared__ int32_t base[L * V + kMaxShared + 1];
        if (a.prob_sum) {
            for (int e = tid; e < a.E; e += BT) a.prob_sum[e] = psum[e];
            if (tid < 64) route_loss(a, hist, psum);
        }
        route_starts(a, hist, base);
        __syncthreads();
        route_counts(a, hist, base);
        const int64_t used = base[a.G];
        __syncthreads();
        route_place<WORDS>(a, 0, a.T, base, reinterpret_cast<uint32_t(*)[WORDS]>(buf));
        route_tail(a, used, tid, BT);
    } else {
        for (int i = tid; i < a.ldh; i += BT) a.hist[(int64_t)blockIdx.x * a.ldh + i] = i <= a.G ? hist[i] : 0;
        if (a.prob_sum)
            for (int e = tid; e < a.lde; e += BT)
                a.part[(int64_t)blockIdx.x * a.lde + e] = e < a.E ? psum[e] : 0.0f;
    }
}

// Column sums of an [n, ld] array by one workgroup, four columns and every
// parts-th row to a thread with eight rows in flight: f(w, v) sees each
// 16-byte piece; `quads` = ld / 4.
template <typename V4, typename F>
__device__ __forceinline__ void column_pieces(const V4 *__restrict__ x, int n, int quads, int part, int parts, int q,
                                              F f) {
    int w = part;
    for (; w + 7 * parts < n; w += 8 * parts) {
        V4 v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = x[(int64_t)(w + i * parts) * quads + q];
#pragma unroll
        for (int i = 0; i < 8; i++) f(w + i * parts, v[i]);
    }
    for (; w < n; w += parts) f(w, x[(int64_t)w * quads + q]);
}

// Second launch: workgroup b < nwg places the rows of its run; workgroup nwg
// sums the probabilities.  Every workgroup adds up the histograms of all runs
// by itself (what precedes its run, and the totals): at most 512 rows of
// 4 (G + 1) bytes from L2, which is less than a third launch costs.
__global__ __launch_bounds__(kRouteThreads) void k_route_place(RouteArgs a) {
    __shared__ int32_t tot[kMaxGroups + 4], before[kMaxGroups + 4], base[kMaxGroups + 1];
    __shared__ __attribute__((aligned(16))) uint32_t bits[kMaxGroups][kWords];
    const int tid = threadIdx.x, b = blockIdx.x;
    for (int i = tid; i < a.ldh; i += kRouteThreads) tot[i] = before[i] = 0;
    __syncthreads();
    {
        const int quads = a.ldh / 4, parts = kRouteThreads / quads, part = tid / quads, q = tid % quads;
        if (part < parts) {
            int s[4] = {0, 0, 0, 0}, sb[4] = {0, 0, 0, 0};
            column_pieces(reinterpret_cast<const int4 *>(a.hist), a.nwg, quads, part, parts, q, [&](int w, int4 h) {
                const int m = w < b ? -1 : 0, v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    s[i] += v[i];
                    sb[i] += v[i] & m;
                }
            });
#pragma unroll
            for (int i = 0; i < 4; i++) {
                atomicAdd(&tot[4 * q + i], s[i]);
                atomicAdd(&before[4 * q + i], sb[i]);
            }
        }
    }
    __syncthreads();
    if (b == a.nwg) {                       // the loss's workgroup
        float *red = reinterpret_cast<float *>(bits);   // [parts][lde], at most 4 floats per thread
        const int quads = a.lde / 4, parts = kRouteThreads / quads, part = tid / quads, q = tid % quads;
        if (part < parts) {
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            column_pieces(reinterpret_cast<const float4 *>(a.part), a.nwg, quads, part, parts, q, [&](int, float4 v) {
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            });
            reinterpret_cast<float4 *>(red)[part * quads + q] = s;
        }
        __syncthreads();
        float *sum = red + 4 * kRouteThreads;
        for (int e = tid; e < a.E; e += kRouteThreads) {
            float s = 0.0f;
            for (int w = 0; w < parts; w++) s += red[w * a.lde + e];
            sum[e] = s;
            a.prob_sum[e] = s;
        }
        __syncthreads();
        if (tid < 64) route_loss(a, tot, sum);
        return;
    }
    route_starts(a, tot, base);
    __syncthreads();
    const int64_t used = base[a.G];
    if (b == 0) {
        route_counts(a, tot, base);
        __syncthreads();
    }
    for (int i = tid; i < a.G; i += kRouteThreads) base[i] += before[i];
    __syncthreads();
    const int64_t t0 = (int64_t)b * a.CT, t1 = t0 + a.CT < a.T ? t0 + a.CT : a.T;
    route_place<kWords>(a, t0, t1, base, bits);
    route_tail(a, used, (int64_t)b * kRouteThreads + tid, (int64_t)a.nwg * kRouteThreads);
}

static int32_t round4(int64_t n) { return (int32_t)((n + 3) / 4 * 4); }

// Runs of whole words of tokens, at most 256 of them once a run is 256 tokens
// long (its workgroup then has 1024 threads).
static void route_runs(int64_t T, int32_t &CT, int32_t &nwg) {
    CT = (int32_t)(((T + 255) / 256 + 31) / 32 * 32);
    if (T <= kOneWorkgroupTokens) CT = (int32_t)kOneWorkgroupTokens;
    nwg = (int32_t)((T + CT - 1) / CT);
}

int64_t route_workspace_bytes(int64_t T, int64_t E, int64_t shared) {
    int32_t CT, nwg;
    route_runs(T, CT, nwg);
    return nwg == 1 ? 0 : (int64_t)nwg * 4 * (round4(E + shared + 1) + round4(E));
}

template <typename T, int L, int V, int N, bool VEC>
static void route_launch_few(const RouteArgs &a, hipStream_t s) {
    if (a.nwg == 1) k_route_select<T, L, V, N, 256, true, VEC><<<1, 256, 0, s>>>(a);
    else k_route_select<T, L, V, N, 256, false, VEC><<<a.nwg, 256, 0, s>>>(a);
}
template <typename T, int L, int V, bool VEC>
static void route_few(const RouteArgs &a, hipStream_t s) {
    if (a.k <= 8) route_launch_few<T, L, V, 8, VEC>(a, s);
    else if (a.k <= 16) route_launch_few<T, L, V, 16, VEC>(a, s);
    else route_launch_few<T, L, V, 32, VEC>(a, s);
}
template <typename T, bool VEC>
static void route_few_experts(const RouteArgs &a, hipStream_t s) {
    constexpr int Q = kPiece<T>;
    if (a.E <= 64) route_few<T, 64 / Q, Q, VEC>(a, s);
    else if (a.E <= 128) route_few<T, 16, 8, VEC>(a, s);
    else if (a.E <= 256) route_few<T, 16, 16, VEC>(a, s);
    else if (a.E <= 512) route_few<T, 32, 16, VEC>(a, s);
    else route_few<T, 32, 32, VEC>(a, s);
}

constexpr int kManyThreads = 512;
template <typename T>
static void route_dispatch(const RouteArgs &a, bool vec, hipStream_t s) {
    if (a.T >= kManyTokens && a.k <= 8 && a.E <= 256 && vec) {
        constexpr int B = kManyThreads;
        if (a.E <= 64) k_route_select<T, 4, 16, 8, B, false, true><<<a.nwg, B, 0, s>>>(a);
        else if (a.E <= 128) k_route_select<T, 4, 32, 8, B, false, true><<<a.nwg, B, 0, s>>>(a);
        else k_route_select<T, 8, 32, 8, B, false, true><<<a.nwg, B, 0, s>>>(a);
    } else if (vec) {
        route_few_experts<T, true>(a, s);
    } else {
        route_few_experts<T, false>(a, s);
    }
    if (a.nwg > 1) k_route_place<<<a.nwg + (a.prob_sum ? 1 : 0), kRouteThreads, 0, s>>>(a);
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
    route_runs(T, a.CT, a.nwg);
    a.ldh = round4(E + shared + 1);
    a.lde = round4(E);
    a.hist = reinterpret_cast<int32_t *>(workspace);
    a.part = reinterpret_cast<float *>(a.hist + (int64_t)a.nwg * a.ldh);
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

// Per element the terms that every expert has are one multiply-add of the
// count and one product, e (c1 f - c2); the k chosen experts' own terms are
// added by the lane that holds the choice: it evaluates its logit again and
// stores over the row's element (the same wavefront's store, issued later).
template <typename T, int L, int V, bool VEC>
__global__ __launch_bounds__(256) void k_route_bwd(RouteBwdArgs a) {
    constexpr int KS = 32 / L;                // choices per lane, k <= 32
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    float f[V], coef = 0.0f, rn = 0.0f;
    if (a.d_loss) {
        const int32_t n = a.counts[a.G];
        rn = 1.0f / (n > 0 ? (float)n : 1.0f);
        coef = *a.d_loss * ((float)a.E / (float)a.k) * rn;
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = expert_of<T, L>(lane, i);
        f[i] = a.d_loss && e < a.E ? (float)a.counts[e] * rn : 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + grp; t < a.T; t += (int64_t)gridDim.x * (256 / L)) {
        const T *in = reinterpret_cast<const T *>(a.logits) + t * a.ldl;
        T *out = reinterpret_cast<T *>(a.d_logits) + t * a.ldd;
        float v[V];
        if (a.mask && !a.mask[t]) {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = 0.0f;
            store_logits<T, L, V, VEC>(out, lane, a.E, v);
            continue;
        }
        load_logits<T, L, V, VEC>(in, lane, a.E, v);
        int ex[KS];
        float x[KS], dw[KS];
#pragma unroll
        for (int q = 0; q < KS; q++) {
            const int j = q * L + lane;
            ex[q] = -1;
            x[q] = -INFINITY;
            dw[q] = 0.0f;
            if (a.d_weights && j < a.k) {
                const int e = a.experts[t * a.kk + j];
                const int32_t r = a.pos[t * a.kk + j];
                if (e >= 0 && e < a.E && r >= 0 && r < a.rows) {
                    ex[q] = e;
                    x[q] = elem(in + e);
                    dw[q] = a.d_weights[r];
                }
            }
        }
        float m = v[0];
#pragma unroll
        for (int i = 1; i < V; i++) m = fmaxf(m, v[i]);
        m = group_max<L>(m);
        m = m > -INFINITY ? m : 0.0f;
        const float sum = exp_sum<L>(v, m), inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        float dot = 0.0f, ps = 0.0f, pd = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) dot = fmaf(v[i], f[i], dot);
#pragma unroll
        for (int q = 0; q < KS; q++) {
            x[q] = __builtin_amdgcn_exp2f((x[q] - m) * kLog2e);
            ps += x[q];
            pd = fmaf(x[q], dw[q], pd);
        }
        dot = group_sum<L>(dot) * inv;
        ps = group_sum<L>(ps);
        pd = group_sum<L>(pd);
        // renormalised: chosen p / ps; else p itself, whose sum of p dw every expert feels
        const float scale = a.norm ? (ps > 0.0f ? 1.0f / ps : 0.0f) : inv;
        const float c1 = coef * inv, c2 = c1 * dot + (a.norm ? 0.0f : inv * inv * pd);
#pragma unroll
        for (int i = 0; i < V; i++) v[i] *= fmaf(c1, f[i], -c2);
        store_logits<T, L, V, VEC>(out, lane, a.E, v);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < KS; q++)
            if (ex[q] >= 0) {
                const float fe = a.d_loss ? (float)a.counts[ex[q]] * rn : 0.0f;
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
template <typename T, bool VEC>
static void route_bwd_dispatch(const RouteBwdArgs &a, hipStream_t s) {
    constexpr int Q = kPiece<T>;
    const bool many = a.T >= kManyTokens;
    if (a.E <= 64) route_bwd_launch<T, 64 / Q, Q, VEC>(a, s);
    else if (a.E <= 128 && many) route_bwd_launch<T, 4, 32, VEC>(a, s);
    else if (a.E <= 128) route_bwd_launch<T, 16, 8, VEC>(a, s);
    else if (a.E <= 256 && many) route_bwd_launch<T, 8, 32, VEC>(a, s);
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

// One thread per token and eight columns.
template <typename TI, typename TO>
__global__ __launch_bounds__(256) void k_combine(const TI *__restrict__ y, int64_t rows, int64_t ldy,
                                                 const int32_t *__restrict__ pos, const float *__restrict__ weights,
                                                 int64_t T, int kk, int nc, TO *__restrict__ out, int64_t ldo) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / nc;
    if (t >= T) return;
    const int c = (int)(i - t * nc) * 8;
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < kk; j++) {
        const int32_t r = pos[t * kk + j];
        if (r < 0 || r >= rows) continue;
        const float w = weights ? weights[t * kk + j] : 1.0f;
        float v[8];
        ld8(y + (int64_t)r * ldy + c, v);
#pragma unroll
        for (int q = 0; q < 8; q++) acc[q] += w * v[q];
    }
    st8(out + t * ldo + c, acc);
}

template <typename TI, typename TO>
static void combine_launch(const void *y, int64_t rows, int64_t H, int64_t ldy, const int32_t *pos,
                           const float *weights, int64_t T, int64_t kk, void *out, int64_t ldo, hipStream_t s) {
    const int64_t n = T * (H / 8);
    k_combine<TI, TO><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(reinterpret_cast<const TI *>(y), rows, ldy, pos,
                                                                 weights, T, (int)kk, (int)(H / 8),
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
