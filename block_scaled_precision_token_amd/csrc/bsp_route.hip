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
constexpr int kRouteThreads = 512;
constexpr int kSub = 256;            // tokens ranked at a time (one bit each per group)
constexpr int kMaxGroups = 1024 + 64;

// LDS accesses of one wavefront exchanged between its lanes: ordered by the
// hardware, fenced for the compiler.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Rotation within each row of 16 lanes (DPP row_ror).
template <int N>
__device__ __forceinline__ float row_ror(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xF, 0xF, false));
}

// All-reduce over the L lanes that share a token (L = 16 or 64).  The sums add
// the same two values on both sides of every step, so all lanes hold the
// same bits.
template <int L>
__device__ __forceinline__ float group_max(float v) {
    v = fmaxf(v, row_ror<8>(v));
    v = fmaxf(v, row_ror<4>(v));
    v = fmaxf(v, row_ror<2>(v));
    v = fmaxf(v, row_ror<1>(v));
    if (L == 64) {
        v = fmaxf(v, __shfl_xor(v, 16, 64));
        v = fmaxf(v, __shfl_xor(v, 32, 64));
    }
    return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    v += row_ror<8>(v);
    v += row_ror<4>(v);
    v += row_ror<2>(v);
    v += row_ror<1>(v);
    if (L == 64) {
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
    }
    return v;
}

__device__ __forceinline__ float elem(const float *p) { return *p; }
__device__ __forceinline__ float elem(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

// V consecutive logits from e0 on, -inf past E.  vec: rows start on 16 bytes.
template <int V>
__device__ __forceinline__ void load_logits(const float *row, int e0, int E, bool vec, float (&v)[V]) {
    if (vec && e0 + V <= E) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(row + e0 + i);
            v[i] = f.x;
            v[i + 1] = f.y;
            v[i + 2] = f.z;
            v[i + 3] = f.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; i++) v[i] = e0 + i < E ? row[e0 + i] : -INFINITY;
}
template <int V>
__device__ __forceinline__ void load_logits(const uint16_t *row, int e0, int E, bool vec, float (&v)[V]) {
    if (vec && e0 + V <= E) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const uint2 u = *reinterpret_cast<const uint2 *>(row + e0 + i);
            v[i] = bf16_lo(u.x);
            v[i + 1] = bf16_hi(u.x);
            v[i + 2] = bf16_lo(u.y);
            v[i + 3] = bf16_hi(u.y);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; i++) v[i] = e0 + i < E ? elem(row + e0 + i) : -INFINITY;
}
template <int V>
__device__ __forceinline__ void store_logits(float *row, int e0, int E, bool vec, const float (&v)[V]) {
    if (vec && e0 + V <= E) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(row + e0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; i++)
        if (e0 + i < E) row[e0 + i] = v[i];
}
template <int V>
__device__ __forceinline__ void store_logits(uint16_t *row, int e0, int E, bool vec, const float (&v)[V]) {
    if (vec && e0 + V <= E) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<uint2 *>(row + e0 + i) =
                make_uint2(f32_to_bf16(v[i]) | (f32_to_bf16(v[i + 1]) << 16),
                           f32_to_bf16(v[i + 2]) | (f32_to_bf16(v[i + 3]) << 16));
        return;
    }
#pragma unroll
    for (int i = 0; i < V; i++)
        if (e0 + i < E) row[e0 + i] = (uint16_t)f32_to_bf16(v[i]);
}

// Softmax of a token held as V logits on each of L lanes: e_i = exp(l_i - m)
// (0 for -inf), the maximum and the sum.  routed: some logit is above -inf
// and none is NaN or +inf; such a logit makes the sum NaN.
template <int L, int V>
struct Softmax {
    float e[V], m, sum;
    bool routed;
    __device__ __forceinline__ explicit Softmax(const float (&v)[V]) {
        float mx = v[0];
#pragma unroll
        for (int i = 1; i < V; i++) mx = fmaxf(mx, v[i]);
        mx = group_max<L>(mx);
        m = mx > -INFINITY ? mx : 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            e[i] = __builtin_amdgcn_exp2f((v[i] - m) * kLog2e);
            s += e[i];
        }
        sum = group_sum<L>(s);
        routed = sum > 0.0f;
    }
};

struct RouteArgs {
    const void *logits;
    const uint8_t *mask;
    int64_t T, ldl;
    int32_t E, k, kk, G;
    bool norm, vec;
    int32_t *experts, *counts, *src, *pos;
    float *weights, *row_weights, *prob_sum, *loss;
    int64_t *off;
    // workspace, one entry per workgroup (a run of CT consecutive tokens)
    int32_t CT, nwg;
    int32_t *hist;    // [nwg][G + 1]: rows of each group, routed tokens
    float *part;      // [nwg][E]: sums of probabilities
};

// Choice, weights, histogram and probability sums of tokens [t0, t1) by one
// workgroup; L lanes share a token, lane l holds experts [l V, l V + V).
// hist: LDS [G + 1], left with this workgroup's counts; psum: LDS
// [kRouteThreads / 64][E], the first row left with its probability sums.
template <typename T, int L, int V>
__device__ void route_select(const RouteArgs &a, int64_t t0, int64_t t1, int32_t *hist, float *psum) {
    constexpr int KS = L == 16 ? 2 : 1;   // choices a lane keeps (k <= 32)
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    const int first = tid & 63 & ~(L - 1);   // first lane of this token's group
    const int e0 = lane * V;
    const bool aux = a.prob_sum != nullptr;
    for (int i = tid; i <= a.G; i += kRouteThreads) hist[i] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    for (int64_t t = t0 + grp; t < t1; t += kRouteThreads / L) {
        float v[V];
        if (!a.mask || a.mask[t]) {
            load_logits<V>(reinterpret_cast<const T *>(a.logits) + t * a.ldl, e0, a.E, a.vec, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = -INFINITY;
        }
        const Softmax<L, V> s(v);
        const float inv = 1.0f / s.sum;
        if (aux && s.sum != 0.0f) {           // NaN in a bad row reaches prob_sum and loss
#pragma unroll
            for (int i = 0; i < V; i++) acc[i] += s.e[i] * inv;
        }
        // k times: the largest logit left, its lowest index, out of the race
        int sel[KS];
        float val[KS], total = 0.0f;
#pragma unroll
        for (int q = 0; q < KS; q++) {
            sel[q] = -1;
            val[q] = 0.0f;
        }
        for (int j = 0; j < a.k; j++) {
            float lm = v[0];
#pragma unroll
            for (int i = 1; i < V; i++) lm = fmaxf(lm, v[i]);
            const float best = group_max<L>(lm);
            const uint64_t eq = __ballot(lm == best) >> first;
            const int lead = __ffsll((unsigned long long)(L == 64 ? eq : eq & 0xFFFFull)) - 1;
            int at = 0;
#pragma unroll
            for (int i = V - 1; i >= 0; i--)
                if (v[i] == best) at = i;
            const bool mine = lane == lead;
#pragma unroll
            for (int i = 0; i < V; i++)
                if (mine && i == at) v[i] = -INFINITY;
            const int idx = __shfl(e0 + at, first + (lead < 0 ? 0 : lead), 64);
            const bool ok = s.routed && best > -INFINITY;
            const float ex = ok ? __builtin_amdgcn_exp2f((best - s.m) * kLog2e) : 0.0f;
            total += ex;
            if (lane == (j & (L - 1)) && ok) {
#pragma unroll
                for (int q = 0; q < KS; q++)
                    if (q == j / L) {
                        sel[q] = idx;
                        val[q] = ex;
                    }
            }
        }
        const bool bad = s.sum != s.sum;
        const float scale = bad ? s.sum : !s.routed ? 0.0f : a.norm ? 1.0f / total : inv;
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
            a.experts[t * a.kk + j] = s.routed ? g : -1;
            a.weights[t * a.kk + j] = s.routed ? 1.0f : 0.0f;
            if (s.routed) atomicAdd(&hist[g], 1);
        }
        if (lane == 0 && s.routed) atomicAdd(&hist[a.G], 1);
    }
    if (aux) {
        // tokens' sums in a fixed order: lane groups of a wavefront, then wavefronts
        if (L == 16) {
#pragma unroll
            for (int i = 0; i < V; i++) {
                acc[i] += __shfl_xor(acc[i], 16, 64);
                acc[i] += __shfl_xor(acc[i], 32, 64);
            }
        }
        const int wv = tid >> 6;
        if ((tid & 63) < L) {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (e0 + i < a.E) psum[wv * a.E + e0 + i] = acc[i];
        }
        __syncthreads();
        for (int e = tid; e < a.E; e += kRouteThreads) {
            float s = 0.0f;
            for (int w = 0; w < kRouteThreads / 64; w++) s += psum[w * a.E + e];
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
// table of kSub tokens, so a choice's rank among the run's is a population
// count: rows come out ordered by token whatever the order of execution.
__device__ void route_place(const RouteArgs &a, int64_t t0, int64_t t1, int32_t *base, uint32_t (*bits)[kSub / 32]) {
    const int tid = threadIdx.x;
    for (int64_t s0 = t0; s0 < t1; s0 += kSub) {
        const int n = (int)(t1 - s0 < kSub ? t1 - s0 : kSub) * a.kk;
        for (int g = tid; g < a.G; g += kRouteThreads)
#pragma unroll
            for (int w = 0; w < kSub / 32; w++) bits[g][w] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kRouteThreads) {
            const int g = a.experts[s0 * a.kk + i], t = i / a.kk;
            if (g >= 0) atomicOr(&bits[g][t >> 5], 1u << (t & 31));
        }
        __syncthreads();
        for (int i = tid; i < n; i += kRouteThreads) {
            const int64_t c = s0 * a.kk + i;
            const int g = a.experts[c], t = i / a.kk;
            int32_t p = -1;
            if (g >= 0) {
                p = base[g] + __popc(bits[g][t >> 5] & ((1u << (t & 31)) - 1u));
                for (int w = 0; w < t >> 5; w++) p += __popc(bits[g][w]);
                a.src[p] = (int32_t)(s0 + t);
                a.row_weights[p] = a.weights[c];
            }
            a.pos[c] = p;
        }
        __syncthreads();
        for (int g = tid; g < a.G; g += kRouteThreads)
#pragma unroll
            for (int w = 0; w < kSub / 32; w++) base[g] += __popc(bits[g][w]);
    }
}

__device__ void route_tail(const RouteArgs &a, int64_t used, int64_t i0, int64_t step) {
    for (int64_t r = used + i0; r < a.T * a.kk; r += step) {
        a.src[r] = -1;
        a.row_weights[r] = 0.0f;
    }
}

template <typename T, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void k_route_select(RouteArgs a) {
    __shared__ int32_t hist[kMaxGroups + 1];
    __shared__ float psum[(kRouteThreads / 64) * L * V];
    const int64_t t0 = (int64_t)blockIdx.x * a.CT, t1 = t0 + a.CT < a.T ? t0 + a.CT : a.T;
    route_select<T, L, V>(a, t0, t1, hist, psum);
    for (int i = threadIdx.x; i <= a.G; i += kRouteThreads)
        a.hist[(int64_t)blockIdx.x * (a.G + 1) + i] = hist[i];
    if (a.prob_sum)
        for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.part[(int64_t)blockIdx.x * a.E + e] = psum[e];
}

// Second launch: workgroup b < nwg places the rows of its run, from the
// histograms of all runs; workgroup nwg sums the probabilities.
__global__ __launch_bounds__(kRouteThreads) void k_route_place(RouteArgs a) {
    __shared__ int32_t tot[kMaxGroups + 1], before[kMaxGroups + 1], base[kMaxGroups + 1];
    __shared__ uint32_t bits[kMaxGroups][kSub / 32];
    const int tid = threadIdx.x, b = blockIdx.x, C = a.G + 1;
    for (int i = tid; i < C; i += kRouteThreads) tot[i] = before[i] = 0;
    __syncthreads();
    // threads in `parts` rows of C columns (or one row striding over them)
    const int width = C < kRouteThreads ? (C + 63) & ~63 : kRouteThreads, parts = kRouteThreads / width;
    const int part = tid / width;
    if (part < parts) {
        for (int g = tid % width; g < C; g += width) {
            int32_t s = 0, sb = 0;
            for (int w = part; w < a.nwg; w += parts) {
                const int32_t h = a.hist[(int64_t)w * C + g];
                s += h;
                sb += w < b ? h : 0;
            }
            atomicAdd(&tot[g], s);
            atomicAdd(&before[g], sb);
        }
    }
    __syncthreads();
    if (b == a.nwg) {                       // the loss's workgroup
        float *q = reinterpret_cast<float *>(bits);
        for (int e = tid; e < a.E; e += kRouteThreads) {
            float s = 0.0f;
            for (int w = 0; w < a.nwg; w++) s += a.part[(int64_t)w * a.E + e];
            q[e] = s;
            a.prob_sum[e] = s;
        }
        __syncthreads();
        if (tid < 64) route_loss(a, tot, q);
        return;
    }
    route_starts(a, tot, base);
    __syncthreads();
    const int64_t used = base[a.G];
    if (b == 0) {
        for (int i = tid; i < C; i += kRouteThreads) {
            a.counts[i] = tot[i];
            a.off[i] = base[i];
        }
        __syncthreads();
    }
    for (int i = tid; i < a.G; i += kRouteThreads) base[i] += before[i];
    __syncthreads();
    const int64_t t0 = (int64_t)b * a.CT, t1 = t0 + a.CT < a.T ? t0 + a.CT : a.T;
    route_place(a, t0, t1, base, bits);
    route_tail(a, used, (int64_t)b * kRouteThreads + tid, (int64_t)a.nwg * kRouteThreads);
}

// A small batch in one workgroup and one launch.
template <typename T, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void k_route_one(RouteArgs a) {
    __shared__ int32_t tot[kMaxGroups + 1], base[kMaxGroups + 1];
    __shared__ uint32_t bits[kMaxGroups][kSub / 32];
    __shared__ float psum[(kRouteThreads / 64) * L * V];
    const int tid = threadIdx.x;
    route_select<T, L, V>(a, 0, a.T, tot, psum);
    if (a.prob_sum) {
        for (int e = tid; e < a.E; e += kRouteThreads) a.prob_sum[e] = psum[e];
        if (tid < 64) route_loss(a, tot, psum);
    }
    route_starts(a, tot, base);
    __syncthreads();
    for (int i = tid; i <= a.G; i += kRouteThreads) {
        a.counts[i] = tot[i];
        a.off[i] = base[i];
    }
    const int64_t used = base[a.G];
    __syncthreads();
    route_place(a, 0, a.T, base, bits);
    route_tail(a, used, tid, kRouteThreads);
}

constexpr int64_t kOneWorkgroupTokens = 64;

static void route_runs(int64_t T, int32_t &CT, int32_t &nwg) {
    // runs of whole 32-token words, at most 512 of them
    CT = (int32_t)(((T + 511) / 512 + 31) / 32 * 32);
    nwg = (int32_t)((T + CT - 1) / CT);
}

int64_t route_workspace_bytes(int64_t T, int64_t E, int64_t shared) {
    if (T <= kOneWorkgroupTokens) return 0;
    int32_t CT, nwg;
    route_runs(T, CT, nwg);
    const int64_t hist = ((int64_t)nwg * (E + shared + 1) * 4 + 255) / 256 * 256;
    return hist + (int64_t)nwg * E * 4;
}

template <typename T, int L, int V>
static void route_launch(const RouteArgs &a, hipStream_t s) {
    if (a.T <= kOneWorkgroupTokens) {
        k_route_one<T, L, V><<<1, kRouteThreads, 0, s>>>(a);
        return;
    }
    k_route_select<T, L, V><<<a.nwg, kRouteThreads, 0, s>>>(a);
    k_route_place<<<a.nwg + (a.prob_sum ? 1 : 0), kRouteThreads, 0, s>>>(a);
}

template <typename T>
static void route_dispatch(const RouteArgs &a, hipStream_t s) {
    if (a.E <= 64) route_launch<T, 16, 4>(a, s);
    else if (a.E <= 128) route_launch<T, 16, 8>(a, s);
    else if (a.E <= 256) route_launch<T, 16, 16>(a, s);
    else if (a.E <= 512) route_launch<T, 64, 8>(a, s);
    else route_launch<T, 64, 16>(a, s);
}

static bool rows16(const void *p, int64_t ld, int dtype) {
    const int64_t row = ld * (dtype == BSP_DTYPE_BF16 ? 2 : 4);
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && row % 16 == 0;
}

hipError_t launch_route(const void *logits, int dtype, int64_t T, int64_t E, int64_t ldl, const uint8_t *mask,
                        int64_t k, int64_t shared, int32_t *experts, float *weights, int32_t *counts, int64_t *off,
                        int32_t *src, int32_t *pos, float *row_weights, float *prob_sum, float *loss, bool norm,
                        void *workspace, hipStream_t s) {
    RouteArgs a;
    a.logits = logits; a.mask = mask; a.T = T; a.ldl = ldl;
    a.E = (int32_t)E; a.k = (int32_t)k; a.kk = (int32_t)(k + shared); a.G = (int32_t)(E + shared);
    a.norm = norm; a.vec = rows16(logits, ldl, dtype);
    a.experts = experts; a.counts = counts; a.src = src; a.pos = pos;
    a.weights = weights; a.row_weights = row_weights; a.prob_sum = prob_sum; a.loss = loss; a.off = off;
    route_runs(T, a.CT, a.nwg);
    a.hist = reinterpret_cast<int32_t *>(workspace);
    a.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) +
                                       ((int64_t)a.nwg * (a.G + 1) * 4 + 255) / 256 * 256);
    if (dtype == BSP_DTYPE_BF16) route_dispatch<uint16_t>(a, s);
    else route_dispatch<float>(a, s);
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
    bool norm, vec, vecd;
    const int32_t *experts, *pos, *counts;
    const float *d_weights, *d_loss;
};

template <typename T, int L, int V>
__global__ __launch_bounds__(256) void k_route_bwd(RouteBwdArgs a) {
    constexpr int KS = L == 16 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float buf[256 / L][L * V];
    const int tid = threadIdx.x, lane = tid & (L - 1), grp = tid / L;
    const int e0 = lane * V;
    float *row = buf[grp];
    float f[V], coef = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = 0.0f;
    if (a.d_loss) {
        const int32_t ni = a.counts[a.G];
        const float n = ni > 0 ? (float)ni : 1.0f;
        coef = *a.d_loss * ((float)a.E / (float)a.k) / n;
#pragma unroll
        for (int i = 0; i < V; i++) f[i] = e0 + i < a.E ? (float)a.counts[e0 + i] / n : 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + grp; t < a.T; t += (int64_t)gridDim.x * (256 / L)) {
        T *out = reinterpret_cast<T *>(a.d_logits) + t * a.ldd;
        float v[V], d[V];
        if (a.mask && !a.mask[t]) {
#pragma unroll
            for (int i = 0; i < V; i++) d[i] = 0.0f;
            store_logits<V>(out, e0, a.E, a.vecd, d);
            continue;
        }
        load_logits<V>(reinterpret_cast<const T *>(a.logits) + t * a.ldl, e0, a.E, a.vec, v);
        const Softmax<L, V> s(v);
        const float inv = s.sum == 0.0f ? 0.0f : 1.0f / s.sum;
        float p[V], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            p[i] = s.e[i] * inv;
            dot += p[i] * f[i];
        }
        dot = group_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < V; i++) d[i] = coef * (p[i] * (f[i] - dot));
        if (a.d_weights) {
#pragma unroll
            for (int i = 0; i < V; i++) row[e0 + i] = p[i];
            wave_lds_sync();
            int ex[KS];
            float pj[KS], dw[KS], ps = 0.0f, pd = 0.0f;
#pragma unroll
            for (int q = 0; q < KS; q++) {
                const int j = q * L + lane;
                ex[q] = -1;
                pj[q] = dw[q] = 0.0f;
                if (j < a.k) {
                    ex[q] = a.experts[t * a.kk + j];
                    const int32_t r = a.pos[t * a.kk + j];
                    if (ex[q] >= a.E) ex[q] = -1;
                    if (ex[q] >= 0 && r >= 0 && r < a.rows) {
                        pj[q] = row[ex[q]];
                        dw[q] = a.d_weights[r];
                    }
                }
                ps += pj[q];
                pd += pj[q] * dw[q];
            }
            ps = group_sum<L>(ps);
            pd = group_sum<L>(pd);
            wave_lds_sync();
#pragma unroll
            for (int i = 0; i < V; i++) row[e0 + i] = 0.0f;
            wave_lds_sync();
            const float ips = ps > 0.0f ? 1.0f / ps : 0.0f;
#pragma unroll
            for (int q = 0; q < KS; q++)
                if (ex[q] >= 0) row[ex[q]] = a.norm ? pj[q] * ips * (dw[q] - pd * ips) : pj[q] * dw[q];
            wave_lds_sync();
#pragma unroll
            for (int i = 0; i < V; i++) d[i] += row[e0 + i] - (a.norm ? 0.0f : p[i] * pd);
            wave_lds_sync();
        }
        store_logits<V>(out, e0, a.E, a.vecd, d);
    }
}

template <typename T>
static void route_bwd_dispatch(const RouteBwdArgs &a, hipStream_t s) {
    const int L = a.E <= 256 ? 16 : 64;
    const int64_t wgs = (a.T + 256 / L - 1) / (256 / L);
    const unsigned grid = (unsigned)(wgs < 4096 ? wgs : 4096);
    if (a.E <= 64) k_route_bwd<T, 16, 4><<<grid, 256, 0, s>>>(a);
    else if (a.E <= 128) k_route_bwd<T, 16, 8><<<grid, 256, 0, s>>>(a);
    else if (a.E <= 256) k_route_bwd<T, 16, 16><<<grid, 256, 0, s>>>(a);
    else if (a.E <= 512) k_route_bwd<T, 64, 8><<<grid, 256, 0, s>>>(a);
    else k_route_bwd<T, 64, 16><<<grid, 256, 0, s>>>(a);
}

hipError_t launch_route_backward(const void *logits, int dtype, int64_t T, int64_t E, int64_t ldl,
                                 const uint8_t *mask, int64_t k, int64_t shared, const int32_t *experts,
                                 const int32_t *pos, const int32_t *counts, const float *d_weights,
                                 const float *d_loss, void *d_logits, int64_t ldd, bool norm, hipStream_t s) {
    RouteBwdArgs a;
    a.logits = logits; a.mask = mask; a.d_logits = d_logits; a.T = T; a.ldl = ldl; a.ldd = ldd;
    a.E = (int32_t)E; a.k = (int32_t)k; a.kk = (int32_t)(k + shared); a.G = (int32_t)(E + shared);
    a.rows = T * (k + shared);
    a.norm = norm; a.vec = rows16(logits, ldl, dtype); a.vecd = rows16(d_logits, ldd, dtype);
    a.experts = experts; a.pos = pos; a.counts = counts; a.d_weights = d_weights; a.d_loss = d_loss;
    if (dtype == BSP_DTYPE_BF16) route_bwd_dispatch<uint16_t>(a, s);
    else route_bwd_dispatch<float>(a, s);
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
