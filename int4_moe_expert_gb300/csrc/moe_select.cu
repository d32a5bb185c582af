// The choice of a router from its logits, and the gradient of the logits from that of the weights.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_elem.h"
#include "moe_internal.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Choice.  score: sigma(l) = 1 / (1 + exp(-l)) or softmax(l); key: sigma(l) + bias, or the logit itself
// where that gives the same order; the K largest keys, the lower expert among equals.  LPT lanes a
// token, J experts a lane.  The K-th largest of the lanes' maxima is at most the K-th largest key, so
// the experts at or above it (8.9 on average for 8 of 256 in 32 lanes, 10.4 in 16) contain the choice:
// one sort of LPT maxima and one ranking of at most LPT candidates instead of K rounds over all
// experts.  Maxima and candidates go by a fast sigmoid less a margin for its error; the candidates'
// keys are computed again, one a lane.  The order is that of the float64 keys: where two neighbours of the
// ranking are nearer than float32 tells, the whole warp ranks them in float64, and so the groups whose scores
// are that near; with more candidates than lanes it ranks them, with more than 32 it does the row over (in float32
// where ties are of the same logit and bias).
// Bound by the instructions of a token and their latency (67 % of the issue slots with 45 % of the warps, half of the
// ALU's; about 600 instructions for the two tokens of a
// warp, of which 200 for scores, 180 for candidates and their keys, 160 for sort and ranking): 65536 x 256 float32
// 27 us (10.5 to move the bytes), 16381 x 256 bf16 in 8 groups 14 us, 32768 x 64 bf16 softmax 12 us.  More blocks
// an SM with fewer registers, logits loaded a round ahead and K rounds over all experts are slower.
// ---------------------------------------------------------------------------

constexpr int kRouteWarps = 4;
constexpr int kRouteThreads = 32 * kRouteWarps;

struct RouteArgs {
    const void *logits;
    long long ld;
    int dtype;
    const float *bias;       // [E] or NULL
    const uint8_t *mask;     // [T] or NULL
    int *idx;                // [T, K]
    float *w;                // [T, K]
    int T, E, K, groups, kept, per_group;
    unsigned group_of;       // e / per_group = e * group_of >> 20
    int sub;                 // log2 of the lanes that look at a group
    int softmax, renorm;
    float scale;
};

// Errors of a key v = s + bias, s = sigmoid(l), in float32, in units u = 2^-24: the exponent's two roundings 2 |l| u
// and the exponential's 2^-22 make (0.224 x 2 + 0.25 x 4) u, since |l| s (1 - s) < 0.224 and s (1 - s) <= 1/4 is the
// derivative by the exponential's relative error; the sum s, the reciprocal 2 s, the bias |v|: 5 + |v|.
constexpr float kUnit = 1.0f / (1 << 24);
__device__ __forceinline__ float key_error(float v) { return kUnit * (5.0f + fabsf(v)); }
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.0f + ex2_fast(x * -1.44269504f)); }
// the same to 2^-20 of its value (of those that are no subnormals): the exponent with its rounding's remainder
__device__ __forceinline__ float sigmoid(float x) {
    const float hi = x * -1.44269504f, lo = fmaf(x, -1.44269504f, -hi) + x * -1.92596299e-8f;      // log2(e) in two parts
    const float t = ex2_fast(hi);
    return rcp_fast(1.0f + (fabsf(x) < 88.0f ? fmaf(t, lo * 0.693147181f, t) : t));      // beyond, t may be infinite, and the result is 1 or 0
}
__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// calls f with a value of the type that `dtype` names; element e of a row of that type
template <typename F>
__device__ __forceinline__ void by_type(int dtype, F &&f) {
    if (dtype == MOE_DTYPE_F32) f(float{});
    else if (dtype == MOE_DTYPE_BF16) f(__nv_bfloat16{});
    else f(__half{});
}
__device__ __forceinline__ float load_el(const char *row, int dtype, int e) {
    if (dtype == MOE_DTYPE_F32) return load_in(reinterpret_cast<const float *>(row) + e);
    const unsigned short v = load_in(reinterpret_cast<const unsigned short *>(row) + e);
    return dtype == MOE_DTYPE_BF16 ? __uint_as_float((unsigned)v << 16) : __half2float(__ushort_as_half(v));
}

// A place of a token's ranking.
struct __align__(16) Chosen {
    int e;
    float x, key, bias;      // logit, key, bias
};

// One token by a whole warp in float64: keys of all experts in shared memory, the groups, K rounds.
// (Its arguments one by one: the address of the kernel's parameters would have them copied to local memory.)
__device__ __noinline__ void choose64(const char *row, int dtype, const float *bias, int E, int K, int groups, int kept, unsigned group_of, double *key,
                                      Chosen *out) {
    const int lane = threadIdx.x & 31, per_group = E / groups;
    const bool biased = bias != nullptr;
    unsigned on = 0xffffffffu;
    if (groups > 1) {
        for (int e = lane; e < E; e += 32) key[e] = sigmoid64((double)load_el(row, dtype, e)) + (biased ? (double)load_in(bias + e) : 0.0);
        __syncwarp();
        double best = -INFINITY;       // of group `lane`: the sum of its two best, or its one
        if (lane < groups) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int i = 0; i < per_group; i++) {
                const double v = key[lane * per_group + i];
                if (v > b1) {
                    b2 = b1;
                    b1 = v;
                } else if (v > b2) {
                    b2 = v;
                }
            }
            best = per_group > 1 ? b1 + b2 : b1;
            if (isnan(best)) best = -INFINITY;
        }
        int rank = 0;
        for (int g = 0; g < groups; g++) {
            const double v = __shfl_sync(0xffffffffu, best, g);
            rank += v > best || (v == best && g < lane) ? 1 : 0;
        }
        on = __ballot_sync(0xffffffffu, lane < groups && rank < kept);
    }
    for (int e = lane; e < E; e += 32) {
        const float x = load_el(row, dtype, e);
        double v = biased ? (groups > 1 ? key[e] : sigmoid64((double)x) + (double)load_in(bias + e)) : (double)x;
        if (isnan(v) || (groups > 1 && !(on >> ((unsigned)e * group_of >> 20) & 1u))) v = -INFINITY;
        key[e] = v;
    }
    __syncwarp();
    for (int k = 0; k < K; k++) {
        double best = -INFINITY;
        int at = 0x7fffffff;
        for (int e = lane; e < E; e += 32)
            if (key[e] > best || (key[e] == best && e < at)) {       // what was taken is NaN
                best = key[e];
                at = e;
            }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double v = __shfl_xor_sync(0xffffffffu, best, d);
            const int e = __shfl_xor_sync(0xffffffffu, at, d);
            if (v > best || (v == best && e < at)) {
                best = v;
                at = e;
            }
        }
        if (lane == 0) {
            key[at] = __longlong_as_double(0x7ff8000000000000ll);
            out[k] = {at, load_el(row, dtype, at), 0.0f, 0.0f};
        }
        __syncwarp();
    }
}

// The same in float32, K rounds over the order of the keys as integers: for rows with too many candidates, most of them
// equal.  `kept`: a bit for each group's first lane (1 << sub lanes a group).  False: the choice hangs on neighbours
// that float32 does not tell apart and that are not the same logit and bias, or a kept group has a NaN.
__device__ __noinline__ bool choose32(const char *row, int dtype, const float *bias, int E, int K, unsigned kept, unsigned group_of, int sub, float *x,
                                      unsigned *order, Chosen *out) {
    const int lane = threadIdx.x & 31;
    bool unsure = false;
    auto key_of = [](unsigned o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); };
    for (int e = lane; e < E; e += 32) {
        x[e] = load_el(row, dtype, e);
        float v = (bias ? sigmoid_fast(x[e]) + bias[e] : x[e]) + 0.0f;
        const bool in = kept >> (((unsigned)e * group_of >> 20) << sub) & 1u;
        unsure |= isnan(v) && in && kept != ~0u;       // its group was chosen with a score that is not the formula's
        if (isnan(v) || !in) v = -INFINITY;
        const unsigned bits = __float_as_uint(v);
        order[e] = bits ^ ((unsigned)((int)bits >> 31) | 0x80000000u);
    }
    __syncwarp();
    // not surely below u, and neither both infinite nor the same
    auto near = [&](float u, float v, int a, int b) {
        return !(u - v > 2.0f * key_error(u)) && !(u == v && isinf(u)) && !(x[a] == x[b] && bias[a] == bias[b]);
    };
    float last = 0.0f;
    int last_at = -1;
    for (int k = 0; k < K; k++) {
        unsigned best = 0;
        int at = 0x7fffffff;
        for (int e = lane; e < E; e += 32)
            if (order[e] > best) {       // what was taken is 0
                best = order[e];
                at = e;
            }
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        at = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
        const float v = key_of(top);
        if (bias && k > 0) unsure |= near(last, v, last_at, at);
        last = v;
        last_at = at;
        if (lane == 0) out[k] = {at, x[at], v, bias ? bias[at] : 0.0f};
        if (lane == (at & 31)) order[at] = 0;
        __syncwarp();
    }
    if (bias)
        for (int e = lane; e < E; e += 32) unsure |= order[e] != 0 && near(last, key_of(order[e]), last_at, e);
    return !__any_sync(0xffffffffu, unsure);
}

// J experts a lane in runs of V, LPT lanes a token; BIAS: keys sigmoid(l) + bias, else the logits
template <bool BIAS_, int J_, int LPT_, int V_, bool FULL_ = false>
struct RouteLay {
    static constexpr bool BIAS = BIAS_;
    static constexpr int J = J_, LPT = LPT_, V = V_, G = 32 / LPT;
    static constexpr bool FULL = FULL_;      // E = J LPT
    static constexpr int PER_SM = J >= 32 ? 4 : 8;      // blocks
};

template <class L>
__global__ void __launch_bounds__(kRouteThreads, L::PER_SM) route_kernel(const RouteArgs p) {
    constexpr bool BIAS = L::BIAS;
    constexpr int J = L::J, LPT = L::LPT, V = L::V, G = L::G;
    extern __shared__ __align__(16) double route_sm[];                  // [warps][E + 32]: float64 keys; or scores [G][E + 2 LPT] float32; then the bias
    __shared__ Chosen s_sel[kRouteWarps][G][LPT + 1];
    __shared__ short s_cand[kRouteWarps][G][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPT, g = lane / LPT;
    const unsigned lanes = LPT == 32 ? 0xffffffffu : (1u << LPT) - 1u;
    double *key64 = route_sm + (size_t)warp * (p.E + 32);
    float *score = reinterpret_cast<float *>(key64) + (size_t)g * (p.E + 2 * LPT);
    float *bias = reinterpret_cast<float *>(route_sm + (size_t)kRouteWarps * (p.E + 32));
    auto expert = [&](int j) { return V * (l + LPT * (j / V)) + j % V; };
    auto group_at = [&](int j) { return (unsigned)expert(j) * p.group_of >> 20; };
    auto within = [&](int j) { return L::FULL || expert(j) < p.E; };
    auto row_of = [&](long long t) { return static_cast<const char *>(p.logits) + t * p.ld * (p.dtype == MOE_DTYPE_F32 ? 4 : 2); };
    wait_for_stream();
    if constexpr (BIAS) {
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) bias[e] = load_in(p.bias + e);
        __syncthreads();
    }
    const long long step = (long long)gridDim.x * kRouteWarps * G;
    long long t0 = ((long long)blockIdx.x * kRouteWarps + warp) * G;
    for (; t0 < p.T; t0 += step) {
        const long long t = t0 + g;
        const bool here = t < p.T;
        const bool on = here && (!p.mask || load_in(p.mask + t));      // what is ranked for others is not written
        const char *row = row_of(here ? t : p.T - 1);
        float a[J];
        auto logits = [&] {       // -infinity beyond E
            by_type(p.dtype, [&](auto el) {
                using T = decltype(el);
#pragma unroll
                for (int j = 0; j < J; j += V) {
                    Vec<T, V> v;
                    if constexpr (!L::FULL) v.zero();
                    if (within(j)) v.load(reinterpret_cast<const T *>(row) + expert(j));
                    v.get(&a[j]);
                }
            });
            if constexpr (!L::FULL) {
#pragma unroll
                for (int j = 0; j < J; j++) a[j] = within(j) ? a[j] : -INFINITY;
            }
        };
        logits();
        const bool scores = BIAS || p.groups > 1;
        bool slow = false, hard = false;      // rows done over: in float32, or at once in float64
        unsigned kept = ~0u;
        if (scores) {
#pragma unroll
            for (int j = 0; j < J; j += V) {
                float b[V] = {};
                if constexpr (BIAS) {
                    if (within(j)) {
                        Vec<float, V> v;
                        v.load(bias + expert(j));
                        v.get(b);
                    }
                }
#pragma unroll
                for (int i = 0; i < V; i++) a[j + i] = within(j) ? sigmoid_fast(a[j + i]) + b[i] : -INFINITY;
            }
        }
        if (p.groups > 1) {
            // 2^sub lanes a group
            const int gr = l >> p.sub, part = l & ((1 << p.sub) - 1);
            const bool valid = gr < p.groups;
            float best = -INFINITY, err = 0.0f, b1 = -INFINITY, b2 = -INFINITY;
            auto join = [&](float v1, float v2) {      // the two best of b1 >= b2 and v1 >= v2
                b2 = fmaxf(fmaxf(b2, v2), fminf(b1, v1));
                b1 = fmaxf(b1, v1);
            };
            // a group's scores 2^sub places apart from the next one's, for the banks
            if (V > 1 && p.per_group % V == 0) {
                // the two best of every run, then of a group's runs
                float2 *two = reinterpret_cast<float2 *>(score);
#pragma unroll
                for (int j = 0; j + V <= J; j += V) {
                    if (!within(j)) continue;
                    float h = fmaxf(a[j], a[j + V / 2]), low = fminf(a[j], a[j + V / 2]);
                    if constexpr (V == 4) {
                        const float h2 = fmaxf(a[j + 1], a[j + 3]), l2 = fminf(a[j + 1], a[j + 3]);
                        low = fmaxf(fminf(h, h2), fmaxf(low, l2));
                        h = fmaxf(h, h2);
                    }
                    two[expert(j) / V + (group_at(j) << p.sub)] = make_float2(h, low);
                }
                __syncwarp();
                const int runs = p.per_group / V;
                if (valid)
                    for (int i = part; i < runs; i += 1 << p.sub) {
                        const float2 v = two[gr * (runs + (1 << p.sub)) + i];
                        join(v.x, v.y);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < J; j++)
                    if (within(j)) score[expert(j) + (group_at(j) << p.sub)] = a[j];
                __syncwarp();
                if (valid)
                    for (int i = part; i < p.per_group; i += 1 << p.sub) join(score[gr * (p.per_group + (1 << p.sub)) + i], -INFINITY);
            }
            for (int d = 1 << p.sub >> 1; d; d >>= 1) {
                const float v1 = __shfl_xor_sync(0xffffffffu, b1, d), v2 = __shfl_xor_sync(0xffffffffu, b2, d);
                join(v1, v2);
            }
            if (valid) {
                best = p.per_group > 1 ? b1 + b2 : b1;
                err = kUnit * (5.0f + fabsf(b1) + (p.per_group > 1 ? 5.0f + fabsf(b2) + fabsf(best) : 0.0f));
            }
            int rank = 0;
            for (int i = 0; i < p.groups; i++) {
                const float v = __shfl_sync(0xffffffffu, best, i << p.sub, LPT);
                rank += v > best || (v == best && i < gr) ? 1 : 0;
            }
            bool keep = valid && rank < p.kept;
            float lo = keep ? best - err : INFINITY, hi = valid && !keep ? best + err : -INFINITY;
#pragma unroll
            for (int d = LPT / 2; d; d >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
            }
            // a group's NaN or infinite score: the whole row in float64
            const bool odd = valid && !(fabsf(best) + err < INFINITY);
            hard = (__ballot_sync(0xffffffffu, odd) >> (g * LPT) & lanes) != 0;
            slow = hard;
            // between the last kept and the first other: those groups' sums in float64, by all lanes
            const bool doubt = p.kept < p.groups && !slow && on && lo <= hi && valid && part == 0 && best + err >= lo && best - err <= hi;
            unsigned doubts = __ballot_sync(0xffffffffu, doubt);
            if (doubts) {
                double sum = 0.0;
                for (unsigned left = doubts; left; left &= left - 1) {
                    const int who = __ffs(left) - 1, group = who % LPT >> p.sub;
                    const char *other = row_of(t0 + who / LPT);
                    double b1 = -INFINITY, b2 = -INFINITY;
                    for (int i = lane; i < p.per_group; i += 32) {
                        const int e = group * p.per_group + i;
                        const double v = sigmoid64((double)load_el(other, p.dtype, e)) + (BIAS ? (double)bias[e] : 0.0);
                        b2 = fmax(b2, fmin(b1, v));
                        b1 = fmax(b1, v);
                    }
#pragma unroll
                    for (int d = 16; d; d >>= 1) {
                        const double v1 = __shfl_xor_sync(0xffffffffu, b1, d), v2 = __shfl_xor_sync(0xffffffffu, b2, d);
                        b2 = fmax(fmax(b2, v2), fmin(b1, v1));
                        b1 = fmax(b1, v1);
                    }
                    if (lane == who) sum = p.per_group > 1 ? b1 + b2 : b1;
                }
                const unsigned mine = doubts >> (g * LPT) & lanes;
                const int places = __popc((__ballot_sync(0xffffffffu, keep) >> (g * LPT) & lanes) & mine);
                int ahead = 0;
                for (int i = 0; i < p.groups; i++) {
                    const double v = __shfl_sync(0xffffffffu, sum, i << p.sub, LPT);
                    if (mine >> (i << p.sub) & 1u) ahead += v > sum || (v == sum && i < gr) ? 1 : 0;
                }
                if (doubt) keep = ahead < places;
            }
            kept = __ballot_sync(0xffffffffu, keep) >> (g * LPT) & lanes;      // a group's first lane counts
            if constexpr (!BIAS) logits();
            if (V > 1 && p.per_group % V == 0) {
#pragma unroll
                for (int j = 0; j + V <= J; j += V) {
                    const bool in = within(j) && (kept >> (group_at(j) << p.sub) & 1u);
#pragma unroll
                    for (int i = 0; i < V; i++) a[j + i] = in ? a[j + i] : -INFINITY;
                }
            } else {
#pragma unroll
                for (int j = 0; j < J; j++) {
                    const bool in = within(j) && (kept >> (group_at(j) << p.sub) & 1u);
                    a[j] = in ? a[j] : -INFINITY;
                }
            }
            __syncwarp();
        }
        // the K-th largest of the lanes' maxima
        float m = -INFINITY;       // a NaN is passed over
#pragma unroll
        for (int j = 0; j < J; j++) m = fmaxf(m, a[j]);
#pragma unroll
        for (int k = 2; k <= LPT; k *= 2)
#pragma unroll
            for (int d = k / 2; d; d /= 2) {
                const float o = __shfl_xor_sync(0xffffffffu, m, d);
                m = ((l & k) == 0) == ((l & d) == 0) ? fmaxf(m, o) : fminf(m, o);
            }
        const float kth = __shfl_sync(0xffffffffu, m, p.K - 1, LPT);
        const float least = BIAS ? kth - 2.0f * kUnit * (5.0f + fabsf(kth)) : kth;
        slow |= !(least > -INFINITY);
        // bit J - 1 - j: a_j is not below (a NaN neither: it is found among the candidates; 0 - least: -0 is not below +0)
        const float up = 0.0f - least;
        unsigned mine = 0;
#pragma unroll
        for (int j = 0; j < J; j++) mine = __funnelshift_l(__float_as_uint(a[j] + up), mine, 1);
        mine = ~mine & (J == 32 ? 0xffffffffu : (1u << J % 32) - 1u);
        const int own = __popc(mine);
        int at = own;      // the candidates of this lane and those before it
#pragma unroll
        for (int d = 1; d < LPT; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, at, d, LPT);
            if (l >= d) at += o;
        }
        const int n = __shfl_sync(0xffffffffu, at, LPT - 1, LPT);
        slow |= n > 32;
        at -= own;
        if (slow) mine = 0;
        auto next = [&] {
            const int bit = 31 - __clz(mine), j = J - 1 - bit;
            if (mine != 0) s_cand[warp][g][at] = (short)(V * l + j + (LPT - 1) * V * (j / V));
            at++;
            mine &= ~(1u << (bit & 31));
        };
#pragma unroll
        for (int i = 0; i < (J < 3 ? J : 3); i++) next();
        if (J > 3)
            while (__any_sync(0xffffffffu, mine != 0)) next();
        const bool many = on && !slow && n > LPT;
        unsigned again = LPT < 32 ? __ballot_sync(0xffffffffu, many) : 0u;
        __syncwarp();
        // candidates: their keys, their ranks
        const bool one = on && !slow && !many && l < n;
        const int e = one ? s_cand[warp][g][l] : -1;
        const float xe = one ? load_el(row, p.dtype, e) : 0.0f;
        float be = 0.0f, key = xe;
        if constexpr (BIAS) {
            be = one ? bias[e] : 0.0f;
            key = sigmoid_fast(xe) + be;
        }
        key += 0.0f;       // no zero but +0
        slow |= (__ballot_sync(0xffffffffu, one && isnan(key)) >> (g * LPT) & lanes) != 0;
        const unsigned bits = __float_as_uint(key);
        const unsigned order = one ? bits ^ ((unsigned)((int)bits >> 31) | 0x80000000u) : 0u;
        int most = min(n, LPT);
#pragma unroll
        for (int d = LPT; d < 32; d *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        int rank = 0;
        constexpr int kUsual = LPT < 12 ? LPT : 12;       // places without a candidate have the order 0
#pragma unroll
        for (int c = 0; c < kUsual; c++) rank += __shfl_sync(0xffffffffu, order, c, LPT) > order ? 1 : 0;
        for (int c = kUsual; c < most; c++) rank += __shfl_sync(0xffffffffu, order, c, LPT) > order ? 1 : 0;
        if (one) s_sel[warp][g][rank] = {e, xe, key, be};
        __syncwarp();
        // equal keys meet in one place: the lower expert first
        const bool met = one && s_sel[warp][g][rank].e != e;
        if (__any_sync(0xffffffffu, met)) {
            for (int c = 0; c < most; c++) {
                const unsigned o = __shfl_sync(0xffffffffu, order, c, LPT);
                const int oe = __shfl_sync(0xffffffffu, e, c, LPT);
                rank += one && o == order && oe < e ? 1 : 0;
            }
            if (one) s_sel[warp][g][rank] = {e, xe, key, be};
            __syncwarp();
        }
        Chosen c = s_sel[warp][g][l];
        if constexpr (BIAS) {
            // neighbours that float32 does not tell apart, down to the last that is that near to the K-th; the same logit and
            // bias are equal
            const float below = __shfl_down_sync(0xffffffffu, c.key, 1, LPT), last = __shfl_sync(0xffffffffu, c.key, p.K - 1, LPT);
            const float margin = 2.0f * key_error(c.key);
            const bool tight = one && l + 1 < n && !(c.key - below > margin) && (l < p.K || !(last - c.key > margin));
            if (__any_sync(0xffffffffu, tight)) {
                const float x = __shfl_down_sync(0xffffffffu, c.x, 1, LPT), b = __shfl_down_sync(0xffffffffu, c.bias, 1, LPT);
                again |= __ballot_sync(0xffffffffu, tight && !(c.x == x && c.bias == b));
            }
        }
        const bool redo = (again | __ballot_sync(0xffffffffu, slow && on)) != 0;
        __syncwarp();
        // those tokens' candidates by all lanes: in float32 if there were too many of them, in float64 if near
        while (again) {
            const int r = (__ffs(again) - 1) / LPT, count = __shfl_sync(0xffffffffu, n, r * LPT);
            again &= r + 1 < G ? ~0u << ((r + 1) * LPT % 32) : 0u;
            const bool in = lane < count;
            const int ec = in ? s_cand[warp][r][lane] : -1;
            const float xc = in ? load_el(row_of(t0 + r), p.dtype, ec) : -INFINITY, bc = BIAS && in ? bias[ec] : 0.0f;
            const float kc = BIAS ? sigmoid_fast(xc) + bc : xc;
            if (__any_sync(0xffffffffu, in && isnan(kc))) {
                slow |= g == r;
                continue;
            }
            int place = 0;
            bool near = false;      // to one of the first K: more than the ranking needs, but rare
            for (int c = 0; c < count; c++) {
                const float v = __shfl_sync(0xffffffffu, kc, c), x = __shfl_sync(0xffffffffu, xc, c), bb = __shfl_sync(0xffffffffu, bc, c);
                const int o = __shfl_sync(0xffffffffu, ec, c);
                place += v > kc || (v == kc && o < ec) ? 1 : 0;
                if (BIAS) near |= !(fabsf(v - kc) > key_error(v) + key_error(kc)) && !(x == xc && bb == bc);
            }
            if (BIAS && __any_sync(0xffffffffu, in && near && place <= p.K)) {
                const double k64 = in ? sigmoid64((double)xc) + (double)bc : 0.0;
                place = 0;
                for (int c = 0; c < count; c++) {
                    const double v = __shfl_sync(0xffffffffu, k64, c);
                    const int o = __shfl_sync(0xffffffffu, ec, c);
                    place += v > k64 || (v == k64 && o < ec) ? 1 : 0;
                }
            }
            if (in && place < p.K) s_sel[warp][r][place] = {ec, xc, kc, bc};
            __syncwarp();
        }
        again = __ballot_sync(0xffffffffu, slow && on && l == 0);
        while (again) {
            const int first = __ffs(again) - 1, r = first / LPT;
            again &= again - 1;
            const unsigned groups_kept = __shfl_sync(0xffffffffu, kept, first);
            const bool at_once = __shfl_sync(0xffffffffu, (int)hard, first) != 0;
            const char *other = row_of(t0 + r);
            float *x = reinterpret_cast<float *>(key64);
            if (at_once || !choose32(other, p.dtype, BIAS ? bias : nullptr, p.E, p.K, groups_kept, p.groups > 1 ? p.group_of : 0u, p.sub, x,
                                     reinterpret_cast<unsigned *>(x + p.E), s_sel[warp][r])) {
                __syncwarp();
                choose64(other, p.dtype, BIAS ? bias : nullptr, p.E, p.K, p.groups, p.kept, p.group_of, key64, s_sel[warp][r]);
            }
            __syncwarp();
        }
        if (redo) c = s_sel[warp][g][l];
        // weights: lane k of the token its k-th choice
        const bool out = on && l < p.K;
        if (!out) c = {-1, -INFINITY, 0.0f, 0.0f};
        float pr, w, z;
        if (!BIAS && p.softmax) {
            const float top = __shfl_sync(0xffffffffu, c.x, 0, LPT), base = top == -INFINITY ? 0.0f : top;
            pr = out ? expf(c.x - base) : 0.0f;
            z = 0.0f;
            if (p.renorm) {
                z = pr;
            } else {
#pragma unroll
                for (int j = 0; j < J; j++) z += expf(a[j] - base);
            }
        } else {
            pr = out ? sigmoid(c.x) : 0.0f;
            z = pr;
        }
        const bool soft = !BIAS && p.softmax;
        if (soft || p.renorm) {
            if (LPT == 32 || (soft && !p.renorm)) {
#pragma unroll
                for (int d = LPT / 2; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            } else {      // K is at most half the lanes
#pragma unroll
                for (int d = LPT / 4; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            }
            w = p.scale * (soft ? (z == 0.0f ? 0.0f : __fdividef(pr, z)) : __fdividef(pr, z + 1e-20f));
        } else {
            w = p.scale * pr;
        }
        if (here && l < p.K) {
            p.idx[t * p.K + l] = c.e;
            p.w[t * p.K + l] = on ? w : 0.0f;
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// Gradient.  With p_k the chosen scores, D = sum p_k + 1e-20 and d_k the weights' gradient:
//   sigmoid, renormalised   dl_k = s / D (d_k - sum_j d_j p_j / D) p_k (1 - p_k)
//   sigmoid                 dl_k = s d_k p_k (1 - p_k)
//   softmax, renormalised   dl_k = q_k s (d_k - sum_j d_j q_j), q = softmax over the chosen logits
//   softmax                 dl_e = p_e s (d_e - sum_j d_j p_j), d_e = 0 for the others
// An expert that is named twice gets the sum of its gradients.  All but the last read the chosen logits
// alone: a batch of KP lanes a token computes them, the warp fills its tokens' rows with zeros and the
// lanes write their values over them (the same warp's stores, in order).
// Bound by the latency of the loads that hang on one another, index and logit (DRAM at 39 %, a quarter of the issue slots):
// 65536 x 256 float32, K = 8: 20 us; 10.5 for the row of zeros and the indices, 16 with the 64 bytes that each
// scattered logit takes from memory.  32768 x 64 bf16 softmax: 6 us, two thirds of the issue slots.
// ---------------------------------------------------------------------------

struct RouteGradArgs {
    const void *logits;
    long long ld;
    const int *idx;
    const float *dw;
    void *out;
    long long ldd;
    int T, E, K, softmax, renorm, add;
    float scale;
};

constexpr int kGradWarps = 8;

// the sum of v over the lanes of `same` that hold the same expert, in lane order
__device__ __forceinline__ float sum_over(float v, unsigned same) {
    float s = 0.0f;
#pragma unroll 1
    for (int i = 0; i < 32; i++) {
        const float o = __shfl_sync(0xffffffffu, v, i);
        if (same >> i & 1u) s += o;
    }
    return s;
}

// Whether the lane's expert e (any of its token's others) stands twice in the row: each lane leaves its number
// in the expert's byte of the token's E and looks whether it is still there.
__device__ __forceinline__ bool repeated(uint8_t *row, int e, bool used, int k) {
    if (used) row[e] = (uint8_t)k;
    __syncwarp();
    return __any_sync(0xffffffffu, used && row[e] != (uint8_t)k);
}

template <typename T, int KP, int V>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_kernel(const RouteGradArgs p) {
    constexpr int G = 32 / KP;
    extern __shared__ uint8_t route_seen[];      // [warps][G][E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = lane % KP, g = lane / KP;
    uint8_t *seen = route_seen + (size_t)(warp * G + g) * p.E;
    wait_for_stream();
    const long long step = (long long)gridDim.x * kGradWarps * G;
    for (long long t0 = ((long long)blockIdx.x * kGradWarps + warp) * G; t0 < p.T; t0 += step) {
        const long long t = t0 + g;
        const bool on = t < p.T && k < p.K;
        const int e = on ? load_in(p.idx + t * p.K + k) : -1;
        const bool used = (unsigned)e < (unsigned)p.E;
        const float d = used ? load_in(p.dw + t * p.K + k) : 0.0f;
        const float x = used ? to_float(load_in(static_cast<const T *>(p.logits) + t * p.ld + e)) : -INFINITY;
        T *out = static_cast<T *>(p.out);
        if (!p.add) {      // the rows of the warp's tokens
            Vec<T, V> z;
            z.zero();
            const int rows = (int)min((long long)G, p.T - t0), runs = p.E / V;
            T *first = out + t0 * p.ldd;
            if (p.ldd == p.E) {
#pragma unroll 4
                for (int c = lane; c < rows * runs; c += 32) z.store(first + c * V);
            } else {
                for (int r = 0; r < rows; r++)
                    for (int c = lane; c < runs; c += 32) z.store(first + r * p.ldd + c * V);
            }
        }
        auto sum = [](float v) {
#pragma unroll
            for (int i = KP / 2; i; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
            return v;
        };
        float v;
        if (p.softmax) {
            float m = x;
#pragma unroll
            for (int i = KP / 2; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
            if (m == -INFINITY) m = 0.0f;
            const float pr = used ? expf(x - m) : 0.0f, z = sum(pr), q = z == 0.0f ? 0.0f : __fdividef(pr, z);
            v = q * p.scale * (d - sum(d * q));
        } else {
            const float tt = expf(-fabsf(x)), r = __fdividef(1.0f, 1.0f + tt);
            const float pr = used ? (x >= 0.0f ? r : tt * r) : 0.0f, c1 = x >= 0.0f ? tt * r : r;
            if (p.renorm) {
                const float q = __fdividef(pr, sum(pr) + 1e-20f);
                v = q * p.scale * (d - sum(d * q)) * c1;
            } else {
                v = p.scale * d * pr * c1;
            }
        }
        // an expert twice: the first of its lanes writes the sum
        bool writes = used;
        if (repeated(seen, e, used, k)) {
            const unsigned same = __match_any_sync(0xffffffffu, used ? (g << 16 | e) : (int)(0x80000000u | lane));
            v = sum_over(v, same);
            writes = used && lane == __ffs(same) - 1;
        }
        __syncwarp();
        if (writes) {
            T *at = out + t * p.ldd + e;
            if (p.add) v += to_float(*at);
            *at = from_float<T>(v);
        }
    }
}

// softmax without renormalisation: every logit has a gradient; LPT lanes a token, its logits in registers
template <typename T, int J, int LPT, int V>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_dense_kernel(const RouteGradArgs p) {
    constexpr int G = 32 / LPT;
    extern __shared__ uint8_t route_seen[];      // [warps][G][E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPT, g = lane / LPT;
    uint8_t *seen = route_seen + (size_t)(warp * G + g) * p.E;
    auto expert = [&](int j) { return V * (l + LPT * (j / V)) + j % V; };
    auto sum = [](float v) {
#pragma unroll
        for (int i = LPT / 2; i; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
        return v;
    };
    wait_for_stream();
    const long long step = (long long)gridDim.x * kGradWarps * G;
    for (long long t0 = ((long long)blockIdx.x * kGradWarps + warp) * G; t0 < p.T; t0 += step) {
        const long long t = t0 + g;
        const bool here = t < p.T;
        const int e = here && l < p.K ? load_in(p.idx + t * p.K + l) : -1;
        const bool used = (unsigned)e < (unsigned)p.E;
        const unsigned group = LPT == 32 ? 0xffffffffu : ((1u << LPT % 32) - 1u) << (g * LPT);
        const bool any = (__ballot_sync(0xffffffffu, used) & group) != 0;       // a masked token: zeros, whatever its logits hold
        const T *row = static_cast<const T *>(p.logits) + t * p.ld;
        T *out = static_cast<T *>(p.out) + t * p.ldd;
        float x[J];
#pragma unroll
        for (int j = 0; j < J; j += V) {
            if (any && expert(j) < p.E) {
                Vec<T, V> v;
                v.load(row + expert(j));
                v.get(&x[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; i++) x[j + i] = -INFINITY;
            }
        }
        const float xe = used ? to_float(load_in(row + e)) : -INFINITY, d = used ? load_in(p.dw + t * p.K + l) : 0.0f;
        float m = -INFINITY, z = 0.0f;
#pragma unroll
        for (int j = 0; j < J; j++) m = fmaxf(m, x[j]);
#pragma unroll
        for (int i = LPT / 2; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
        if (m == -INFINITY) m = 0.0f;
#pragma unroll
        for (int j = 0; j < J; j++) {
            x[j] = expf(x[j] - m);
            z += x[j];
        }
        z = sum(z);
        const float inv = z == 0.0f ? 0.0f : __fdividef(1.0f, z), pe = used ? expf(xe - m) * inv : 0.0f;
        const float dot = sum(d * pe);
        float de = d;
        bool writes = used;
        if (repeated(seen, e, used, l)) {
            const unsigned same = __match_any_sync(0xffffffffu, used ? (g << 16 | e) : (int)(0x80000000u | lane));
            de = sum_over(d, same);
            writes = used && lane == __ffs(same) - 1;
        }
        float v = pe * p.scale * (de - dot);
        if (writes && p.add) v += to_float(out[e]);
        __syncwarp();
        if (here && (any || !p.add)) {
            const float up = -dot * p.scale * inv;
#pragma unroll
            for (int j = 0; j < J; j += V) {
                if (expert(j) < p.E) {
                    Vec<T, V> o;
                    float u[V];
                    if (p.add) {
                        o.load(out + expert(j));
                        o.get(u);
                    }
#pragma unroll
                    for (int i = 0; i < V; i++) u[i] = any ? x[j + i] * up + (p.add ? u[i] : 0.0f) : 0.0f;
                    o.set(u);
                    o.store(out + expert(j));
                }
            }
        }
        __syncwarp();
        if (writes) out[e] = from_float<T>(v);
    }
}

// V elements together: E and the rows' strides multiples of V, the rows on V elements' boundary
bool rows_of(const void *x, long long ld, int el, int E, int V) {
    return E % V == 0 && ld % V == 0 && reinterpret_cast<uintptr_t>(x) % (uintptr_t)(V * el) == 0;
}

}  // namespace

cudaError_t launch_route_forward(const void *logits, int dtype, long long ld, int T, int E, const float *bias, int K, int softmax,
                                 int groups, int kept, int renorm, float scale, const uint8_t *mask, int *idx, float *w, cudaStream_t st) {
    RouteArgs p = {logits, ld, dtype, bias, mask, idx, w, T, E, K, groups, kept, E / groups, 0, 0, softmax, renorm, scale};
    p.group_of = ((1u << 20) + p.per_group - 1) / p.per_group;
    auto go = [&](auto lay) {
        using L = decltype(lay);
        auto smem = [](int e) { return (size_t)kRouteWarps * (e + 32) * sizeof(double) + (size_t)e * sizeof(float); };
        const cudaError_t e = allow_smem<route_kernel<L>>(smem(1024));
        if (e != cudaSuccess) return e;
        while (groups > 1 && groups << (p.sub + 1) <= L::LPT) p.sub++;
        const long long need = ((long long)T + kRouteWarps * L::G - 1) / (kRouteWarps * L::G), most = (long long)sm_count() * L::PER_SM;
        return launch_early(route_kernel<L>, (unsigned)(need < most ? need : most), kRouteThreads, smem(E), st, 1, p);
    };
    const int el = dtype == MOE_DTYPE_F32 ? 4 : 2;
    const bool quads = rows_of(logits, ld, el, E, 4), pairs = rows_of(logits, ld, el, E, 2) && p.per_group % 2 == 0;
    auto by_size = [&](auto bias_) {
        constexpr bool B = decltype(bias_)::value;
        // Four tokens a warp for few choices of few experts, two while at most half of the lanes' maxima are wanted.
        // With groups the kept ones may share lanes, which leaves more candidates: two tokens where each group covers
        // all their lanes (in runs of two logits 32 experts, one by one 16), or where enough lanes are left in any
        // case (16381 x 256 in 8 groups of which 4: one token in runs of four 19.5 us, two in runs of two 13.9).
        // Experts that are as many as a layout holds in runs (E = J LPT) need no bounds: 65536 x 128 23.1 us, with them
        // 24.2; x 256 26.0 and 28.3, x 512 48 and 53, x 1024 77 and 84.  64 or fewer take runs of four only where these
        // fill the lanes: among fewer lanes more experts are candidates (65536 x 48: 22.0 us, one by one 19.8).
        auto runs = [&](auto j, auto lpt, auto v) {
            constexpr int J = decltype(j)::value, LPT = decltype(lpt)::value, V = decltype(v)::value;
            return E == J * LPT ? go(RouteLay<B, J, LPT, V, true>{}) : go(RouteLay<B, J, LPT, V>{});
        };
        std::integral_constant<int, 2> two;
        std::integral_constant<int, 4> four;
        std::integral_constant<int, 8> eight;
        std::integral_constant<int, 16> sixteen;
        std::integral_constant<int, 32> all;
        if (K <= 4 && groups == 1 && E <= 64) return E <= 16 ? go(RouteLay<B, 2, 8, 1>{}) : go(RouteLay<B, 8, 8, 1>{});
        if (groups > 1 && K <= 8 && groups <= 16 && p.per_group >= 16 && E > 32 && E <= 256) {
            if (E <= 64) return go(RouteLay<B, 4, 16, 1>{});
            if (E <= 128) return go(RouteLay<B, 8, 16, 1>{});
            return pairs && p.per_group >= 32 ? runs(sixteen, sixteen, two) : go(RouteLay<B, 16, 16, 1>{});
        }
        if (K <= 8 && groups <= 16 && kept * 8 >= groups * K) {
            if (E <= 32) return go(RouteLay<B, 2, 16, 1>{});
            if (E <= 64) return E == 4 * 16 && quads ? go(RouteLay<B, 4, 16, 4, true>{}) : go(RouteLay<B, 4, 16, 1>{});
            if (E <= 128) return quads ? runs(eight, sixteen, four) : go(RouteLay<B, 8, 16, 1>{});
            if (E <= 256) return quads ? runs(sixteen, sixteen, four) : go(RouteLay<B, 16, 16, 1>{});
        } else {
            if (E <= 64) return go(RouteLay<B, 2, 32, 1>{});
            if (E <= 256) return quads && E >= 128 ? runs(eight, all, four) : go(RouteLay<B, 8, 32, 1>{});
        }
        if (E <= 512) return quads ? runs(sixteen, all, four) : go(RouteLay<B, 16, 32, 1>{});
        return quads ? runs(all, all, four) : go(RouteLay<B, 32, 32, 1>{});
    };
    return bias && !softmax ? by_size(std::true_type{}) : by_size(std::false_type{});
}

cudaError_t launch_route_backward(const void *logits, int dtype, long long ld, int T, int E, const int *idx, int K, int softmax, int renorm,
                                  float scale, const float *dw, void *out, long long ldd, bool add, cudaStream_t st) {
    const RouteGradArgs p = {logits, ld, idx, dw, out, ldd, T, E, K, softmax, renorm, add, scale};
    return by_dtype(dtype, [&](auto t) {
        using El = decltype(t);
        const int el = (int)sizeof(El);
        auto run = [&](auto kernel, int tokens) {      // of a warp
            const long long per = kGradWarps * tokens, need = (T + per - 1) / per, most = (long long)sm_count() * 8;
            return launch_early(kernel, (unsigned)(need < most ? need : most), 32 * kGradWarps, (size_t)kGradWarps * tokens * E, st, 1, p);
        };
        if (softmax && !renorm) {
            const bool quads = rows_of(logits, ld, el, E, 4) && rows_of(out, ldd, el, E, 4);
            if (K <= 16 && E <= 64) return quads ? run(route_grad_dense_kernel<El, 4, 16, 4>, 2) : run(route_grad_dense_kernel<El, 4, 16, 1>, 2);
            if (K <= 16 && E <= 256) return quads ? run(route_grad_dense_kernel<El, 16, 16, 4>, 2) : run(route_grad_dense_kernel<El, 16, 16, 1>, 2);
            return quads ? run(route_grad_dense_kernel<El, 32, 32, 4>, 1) : run(route_grad_dense_kernel<El, 32, 32, 1>, 1);
        }
        constexpr int V = 16 / (int)sizeof(El);
        const bool wide = rows_of(out, ldd, el, E, V);
        if (K <= 8) return wide ? run(route_grad_kernel<El, 8, V>, 4) : run(route_grad_kernel<El, 8, 1>, 4);
        return wide ? run(route_grad_kernel<El, 32, V>, 1) : run(route_grad_kernel<El, 32, 1>, 1);
    });
}

}  // namespace moe
