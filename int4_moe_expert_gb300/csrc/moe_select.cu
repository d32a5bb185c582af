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
// ranking are nearer than float32 tells, or there are more candidates than lanes, the whole warp ranks them in
// float64; where two groups' scores are that near, or more than 32 candidates, it does the row over.
// ---------------------------------------------------------------------------

constexpr int kRouteWarps = 4;
constexpr int kRouteThreads = 32 * kRouteWarps;

struct RouteArgs {
    const void *logits;
    long long ld;
    const float *bias;       // [E] or NULL
    const uint8_t *mask;     // [T] or NULL
    int *idx;                // [T, K]
    float *w;                // [T, K]
    int T, E, K, groups, kept, per_group;
    unsigned group_of;       // e / per_group = e * group_of >> 20
    int softmax, renorm;
    float scale;
};

// Errors of a key v = sigmoid + bias in float32, in units u = 2^-24.  exp(-l) to 2 ulp: at most 1 u of the
// sigmoid (its derivative by the relative error is s (1 - s) <= 1/4); the sum, the quotient and the
// sum with the bias: s, s and |v|.  So 3 + |v| in all.  The fast exp is documented to (2 + 1.173 |l|) ulp:
// (0.5 + 0.263) 2 u since |l| s (1 - s) < 0.2240; the sum s, the fast quotient 2 ulp, 4 s, the bias |v|: below 7 + |v|.
constexpr float kUnit = 1.0f / (1 << 24);
__device__ __forceinline__ float key_error(float v) { return kUnit * (3.0f + fabsf(v)); }
__device__ __forceinline__ float fast_error(float v) { return kUnit * (7.0f + fabsf(v)); }

__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }
__device__ __forceinline__ float sigmoid(float x) {
    const float t = expf(-fabsf(x)), r = 1.0f / (1.0f + t);
    return x >= 0.0f ? r : t * r;      // a NaN stays one
}
__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

template <typename T>
__device__ __forceinline__ float logit(const RouteArgs &p, long long t, int e) {
    return to_float(load_in(static_cast<const T *>(p.logits) + t * p.ld + e));
}

// What a token's choice leaves for the weights: expert, logit.
struct Chosen {
    int e;
    float x;
};

// One token by a whole warp in float64: keys of all experts in shared memory, the groups, K rounds.
template <typename T>
__device__ __noinline__ void choose64(const RouteArgs &p, long long t, double *key, Chosen *out) {
    const int lane = threadIdx.x & 31;
    const bool biased = !p.softmax && p.bias;
    unsigned on = 0xffffffffu;
    if (p.groups > 1) {
        for (int e = lane; e < p.E; e += 32) key[e] = sigmoid64((double)logit<T>(p, t, e)) + (biased ? (double)load_in(p.bias + e) : 0.0);
        __syncwarp();
        double best = -INFINITY;       // of group `lane`: the sum of its two best, or its one
        if (lane < p.groups) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int i = 0; i < p.per_group; i++) {
                const double v = key[lane * p.per_group + i];
                if (v > b1) {
                    b2 = b1;
                    b1 = v;
                } else if (v > b2) {
                    b2 = v;
                }
            }
            best = p.per_group > 1 ? b1 + b2 : b1;
            if (isnan(best)) best = -INFINITY;
        }
        int rank = 0;
        for (int g = 0; g < p.groups; g++) {
            const double v = __shfl_sync(0xffffffffu, best, g);
            rank += v > best || (v == best && g < lane) ? 1 : 0;
        }
        on = __ballot_sync(0xffffffffu, lane < p.groups && rank < p.kept);
    }
    for (int e = lane; e < p.E; e += 32) {
        const float x = logit<T>(p, t, e);
        double v = biased ? (p.groups > 1 ? key[e] : sigmoid64((double)x) + (double)load_in(p.bias + e)) : (double)x;
        if (isnan(v) || (p.groups > 1 && !(on >> ((unsigned)e * p.group_of >> 20) & 1u))) v = -INFINITY;
        key[e] = v;
    }
    __syncwarp();
    for (int k = 0; k < p.K; k++) {
        double best = -INFINITY;
        int at = 0x7fffffff;
        for (int e = lane; e < p.E; e += 32)
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
            out[k] = {at, logit<T>(p, t, at)};
        }
        __syncwarp();
    }
}

template <typename T_, int J_, int LPT_, int V_>
struct RouteLay {
    using T = T_;
    static constexpr int J = J_, LPT = LPT_, V = V_, G = 32 / LPT;
    static constexpr int PER_SM = J >= 32 ? 4 : J >= 16 ? 6 : 8;      // blocks
};

template <class L>
__global__ void __launch_bounds__(kRouteThreads, L::PER_SM) route_kernel(const RouteArgs p) {
    using T = typename L::T;
    constexpr int J = L::J, LPT = L::LPT, V = L::V, G = L::G;
    extern __shared__ double route_sm[];                  // [warps][E]: float64 keys; or scores [G][E] float32
    __shared__ Chosen s_sel[kRouteWarps][G][LPT + 1];
    __shared__ float s_key[kRouteWarps][G][LPT + 1];
    __shared__ short s_cand[kRouteWarps][G][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPT, g = lane / LPT;
    const unsigned lanes = LPT == 32 ? 0xffffffffu : (1u << LPT) - 1u;
    double *key64 = route_sm + (size_t)warp * p.E;
    float *score = reinterpret_cast<float *>(key64) + (size_t)g * p.E;
    auto expert = [&](int j) { return V * (l + LPT * (j / V)) + j % V; };
    const bool biased = !p.softmax && p.bias;
    wait_for_stream();
    float b[J];
#pragma unroll
    for (int j = 0; j < J; j++) b[j] = biased && expert(j) < p.E ? load_in(p.bias + expert(j)) : 0.0f;
    const long long step = (long long)gridDim.x * kRouteWarps * G;
    for (long long t0 = ((long long)blockIdx.x * kRouteWarps + warp) * G; t0 < p.T; t0 += step) {
        const long long t = t0 + g;
        const bool here = t < p.T, on = here && (!p.mask || load_in(p.mask + t));
        const T *row = static_cast<const T *>(p.logits) + t * p.ld;
        float x[J], a[J];
#pragma unroll
        for (int j = 0; j < J; j += V) {
            if (on && expert(j) < p.E) {
                Vec<T, V> v;
                v.load(row + expert(j));
                v.get(&x[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; i++) x[j + i] = -INFINITY;
            }
        }
        bool slow = false;
        if (biased || p.groups > 1) {
#pragma unroll
            for (int j = 0; j < J; j++) a[j] = expert(j) < p.E ? sigmoid_fast(x[j]) + b[j] : -INFINITY;
        }
        if (p.groups > 1) {
#pragma unroll
            for (int j = 0; j < J; j++)
                if (expert(j) < p.E) score[expert(j)] = a[j];
            __syncwarp();
            float best = -INFINITY, err = 0.0f;
            if (l < p.groups) {
                float b1 = -INFINITY, b2 = -INFINITY;
                const float *s = score + l * p.per_group;
                int i = l % p.per_group;           // lanes begin at different banks
                for (int n = 0; n < p.per_group; n++) {
                    const float v = s[i];
                    b2 = fmaxf(b2, fminf(b1, v));
                    b1 = fmaxf(b1, v);
                    if (++i == p.per_group) i = 0;
                }
                best = p.per_group > 1 ? b1 + b2 : b1;
                err = p.per_group > 1 ? fast_error(b1) + fast_error(b2) + kUnit * fabsf(best) : fast_error(b1);
            }
            int rank = 0;
            for (int i = 0; i < p.groups; i++) {
                const float v = __shfl_sync(0xffffffffu, best, i, LPT);
                rank += v > best || (v == best && i < l) ? 1 : 0;
            }
            const bool keep = l < p.groups && rank < p.kept;
            float lo = keep ? best - err : INFINITY, hi = l < p.groups && !keep ? best + err : -INFINITY;
#pragma unroll
            for (int d = LPT / 2; d; d >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
            }
            // near ones, and a group's NaN or infinite score: float64 decides
            if (p.kept < p.groups) slow = !(lo > hi);
            slow |= __ballot_sync(0xffffffffu, isnan(best) || isnan(err)) != 0;
            const unsigned kept = __ballot_sync(0xffffffffu, keep) >> (g * LPT) & lanes;
#pragma unroll
            for (int j = 0; j < J; j++) {
                const bool in = expert(j) < p.E && (kept >> ((unsigned)expert(j) * p.group_of >> 20) & 1u);
                a[j] = in ? (biased ? a[j] : x[j]) : -INFINITY;
            }
            __syncwarp();
        } else if (!biased) {
#pragma unroll
            for (int j = 0; j < J; j++) a[j] = x[j];
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
        const float least = biased ? kth - 2.0f * fast_error(kth) : kth;
        slow |= !(least > -INFINITY);
        unsigned mine = 0;
#pragma unroll
        for (int j = 0; j < J; j++) mine |= a[j] >= least ? 1u << j : 0u;
        if (slow) mine = 0;
        const int own = __popc(mine);
        int at = own;      // the candidates of this lane and those before it
#pragma unroll
        for (int d = 1; d < LPT; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, at, d, LPT);
            if (l >= d) at += o;
        }
        const int n = __shfl_sync(0xffffffffu, at, LPT - 1, LPT);
        at -= own;
        while (mine != 0 && at < 32) {
            const int j = __ffs(mine) - 1;
            mine &= mine - 1;
            s_cand[warp][g][at++] = (short)(V * (l + LPT * (j / V)) + j % V);
        }
        slow |= n > 32;
        const bool many = on && !slow && n > LPT;
        unsigned again = LPT < 32 ? __ballot_sync(0xffffffffu, many) : 0u;
        __syncwarp();
        // candidates: their keys, their ranks
        const bool one = on && !slow && !many && l < n;
        const int e = one ? s_cand[warp][g][l] : -1;
        const float xe = one ? to_float(load_in(row + e)) : 0.0f;
        const float be = one && biased ? load_in(p.bias + e) : 0.0f;
        const float key = (biased ? sigmoid(xe) + be : xe) + 0.0f;       // no zero but +0
        const unsigned bits = __float_as_uint(key);
        const unsigned hi = one ? bits ^ ((unsigned)((int)bits >> 31) | 0x80000000u) : 0u, lo = one ? ~(unsigned)e : 0u;
        const unsigned long long code = (unsigned long long)hi << 32 | lo;
        int most = n;
#pragma unroll
        for (int d = LPT; d < 32; d *= 2) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        most = min(most, LPT);
        int rank = 0;
        for (int c = 0; c < most; c++) {
            const unsigned h = __shfl_sync(0xffffffffu, hi, c, LPT), lw = __shfl_sync(0xffffffffu, lo, c, LPT);
            rank += ((unsigned long long)h << 32 | lw) > code ? 1 : 0;
        }
        if (one) {
            s_sel[warp][g][rank] = {e, xe};
            s_key[warp][g][rank] = key;
        }
        __syncwarp();
        if (biased) {
            // neighbours that float32 does not tell apart; the same logit and bias are equal
            bool near = false;
            if (one && l < p.K && l + 1 < n) {
                const Chosen u = s_sel[warp][g][l], v = s_sel[warp][g][l + 1];
                const float ku = s_key[warp][g][l], kv = s_key[warp][g][l + 1];
                near = !(ku - kv > 2.0f * key_error(ku)) && !(u.x == v.x && load_in(p.bias + u.e) == load_in(p.bias + v.e));
            }
            again |= __ballot_sync(0xffffffffu, near);
            __syncwarp();
        }
        // those tokens' candidates by all lanes, in float64
        while (again) {
            const int r = (__ffs(again) - 1) / LPT, count = __shfl_sync(0xffffffffu, n, r * LPT);
            again &= r + 1 < G ? ~0u << ((r + 1) * LPT % 32) : 0u;
            const int ec = lane < count ? s_cand[warp][r][lane] : -1;
            const float xc = lane < count ? logit<T>(p, t0 + r, ec) : 0.0f;
            const double k64 = biased && lane < count ? sigmoid64((double)xc) + (double)load_in(p.bias + ec) : (double)xc;
            int r64 = 0;
            for (int c = 0; c < count; c++) {
                const double v = __shfl_sync(0xffffffffu, k64, c);
                const int o = __shfl_sync(0xffffffffu, ec, c);
                r64 += v > k64 || (v == k64 && o < ec) ? 1 : 0;
            }
            if (lane < count && r64 < p.K) s_sel[warp][r][r64] = {ec, xc};
            __syncwarp();
        }
        again = __ballot_sync(0xffffffffu, slow && on && l == 0);
        while (again) {
            const int r = (__ffs(again) - 1) / LPT;
            again &= again - 1;
            choose64<T>(p, t0 + r, key64, s_sel[warp][r]);
            __syncwarp();
        }
        // weights: lane k of the token its k-th choice
        const bool out = on && l < p.K;
        const Chosen c = out ? s_sel[warp][g][l] : Chosen{-1, -INFINITY};
        float pr, w;
        if (p.softmax) {
            const float top = __shfl_sync(0xffffffffu, c.x, 0, LPT), base = top == -INFINITY ? 0.0f : top;
            pr = out ? expf(c.x - base) : 0.0f;
            float z = 0.0f;
            if (p.renorm) {
                z = pr;
            } else {
#pragma unroll
                for (int j = 0; j < J; j++) z += expf(x[j] - base);
            }
#pragma unroll
            for (int d = LPT / 2; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            w = p.scale * (z == 0.0f ? 0.0f : pr / z);
        } else {
            pr = out ? sigmoid(c.x) : 0.0f;
            float z = pr;
#pragma unroll
            for (int d = LPT / 2; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            w = p.scale * (p.renorm ? pr / (z + 1e-20f) : pr);
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

template <typename T, int KP, int V>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_kernel(const RouteGradArgs p) {
    constexpr int G = 32 / KP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = lane % KP, g = lane / KP;
    wait_for_stream();
    const long long step = (long long)gridDim.x * kGradWarps * G;
    for (long long t0 = ((long long)blockIdx.x * kGradWarps + warp) * G; t0 < p.T; t0 += step) {
        const long long t = t0 + g;
        const bool on = t < p.T && k < p.K;
        int e = on ? load_in(p.idx + t * p.K + k) : -1;
        const bool used = (unsigned)e < (unsigned)p.E;
        const float d = used ? load_in(p.dw + t * p.K + k) : 0.0f;
        const float x = used ? to_float(load_in(static_cast<const T *>(p.logits) + t * p.ld + e)) : -INFINITY;
        T *out = static_cast<T *>(p.out);
        if (!p.add) {      // the rows of the warp's tokens
            Vec<T, V> z;
            z.zero();
            const int quads = p.E / V;
            for (int r = 0; r < G && t0 + r < p.T; r++)
                for (int c = lane; c < quads; c += 32) z.store(out + (t0 + r) * p.ldd + (long long)c * V);
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
            const float pr = used ? expf(x - m) : 0.0f, z = sum(pr), q = z == 0.0f ? 0.0f : pr / z;
            v = q * p.scale * (d - sum(d * q));
        } else {
            const float tt = expf(-fabsf(x)), r = 1.0f / (1.0f + tt);
            const float pr = used ? (x >= 0.0f ? r : tt * r) : 0.0f, c1 = x >= 0.0f ? tt * r : r;
            if (p.renorm) {
                const float inv = 1.0f / (sum(pr) + 1e-20f), q = pr * inv;
                v = q * p.scale * (d - sum(d * q)) * c1;
            } else {
                v = p.scale * d * pr * c1;
            }
        }
        // an expert twice: the first of its lanes writes the sum
        const unsigned same = __match_any_sync(0xffffffffu, used ? (g << 16 | e) : (int)(0x80000000u | lane));
        if (__ballot_sync(0xffffffffu, (same & (same - 1u)) != 0)) v = sum_over(v, same);
        __syncwarp();
        if (used && lane == __ffs(same) - 1) {
            T *at = out + t * p.ldd + e;
            if (p.add) v += to_float(*at);
            *at = from_float<T>(v);
        }
    }
}

// softmax without renormalisation: every logit has a gradient; a warp a token, its logits in registers
template <typename T, int J, int V>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_dense_kernel(const RouteGradArgs p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto expert = [&](int j) { return V * (lane + 32 * (j / V)) + j % V; };
    wait_for_stream();
    const long long step = (long long)gridDim.x * kGradWarps;
    for (long long t = (long long)blockIdx.x * kGradWarps + warp; t < p.T; t += step) {
        const int e = lane < p.K ? load_in(p.idx + t * p.K + lane) : -1;
        const bool used = (unsigned)e < (unsigned)p.E;
        const bool any = __any_sync(0xffffffffu, used);       // a masked token: zeros, whatever its logits hold
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
        const float xe = used ? to_float(load_in(row + e)) : -INFINITY, d = used ? load_in(p.dw + t * p.K + lane) : 0.0f;
        float m = -INFINITY, z = 0.0f;
#pragma unroll
        for (int j = 0; j < J; j++) m = fmaxf(m, x[j]);
#pragma unroll
        for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
        if (m == -INFINITY) m = 0.0f;
#pragma unroll
        for (int j = 0; j < J; j++) {
            x[j] = expf(x[j] - m);
            z += x[j];
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
        const float inv = z == 0.0f ? 0.0f : 1.0f / z, pe = used ? expf(xe - m) * inv : 0.0f;
        float dot = d * pe;
#pragma unroll
        for (int i = 16; i; i >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, i);
        const unsigned same = __match_any_sync(0xffffffffu, used ? e : (int)(0x80000000u | lane));
        float de = d;
        if (__ballot_sync(0xffffffffu, (same & (same - 1u)) != 0)) de = sum_over(d, same);
        const bool writes = used && lane == __ffs(same) - 1;
        float v = pe * p.scale * (de - dot);
        if (writes && p.add) v += to_float(out[e]);
        __syncwarp();
        if (any || !p.add) {
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
    RouteArgs p = {logits, ld, bias, mask, idx, w, T, E, K, groups, kept, E / groups, 0, softmax, renorm, scale};
    p.group_of = ((1u << 20) + p.per_group - 1) / p.per_group;
    return by_dtype(dtype, [&](auto t) {
        using El = decltype(t);
        auto go = [&](auto lay) {
            using L = decltype(lay);
            const size_t smem = (size_t)kRouteWarps * E * sizeof(double);
            const cudaError_t e = allow_smem<route_kernel<L>>((size_t)kRouteWarps * 1024 * sizeof(double));
            if (e != cudaSuccess) return e;
            const long long need = ((long long)T + kRouteWarps * L::G - 1) / (kRouteWarps * L::G), most = (long long)sm_count() * L::PER_SM;
            return launch_early(route_kernel<L>, (unsigned)(need < most ? need : most), kRouteThreads, smem, st, 1, p);
        };
        const bool quads = rows_of(logits, ld, sizeof(El), E, 4);
        if (K <= 8 && groups <= 16) {
            if (E <= 32) return go(RouteLay<El, 2, 16, 1>{});
            if (E <= 64) return quads && E == 64 ? go(RouteLay<El, 4, 16, 4>{}) : go(RouteLay<El, 4, 16, 1>{});
            if (E <= 128) return quads ? go(RouteLay<El, 8, 16, 4>{}) : go(RouteLay<El, 8, 16, 1>{});
            if (E <= 256) return quads ? go(RouteLay<El, 16, 16, 4>{}) : go(RouteLay<El, 16, 16, 1>{});
        } else {
            if (E <= 64) return go(RouteLay<El, 2, 32, 1>{});
            if (E <= 256) return quads && E >= 128 ? go(RouteLay<El, 8, 32, 4>{}) : go(RouteLay<El, 8, 32, 1>{});
        }
        return quads ? go(RouteLay<El, 32, 32, 4>{}) : go(RouteLay<El, 32, 32, 1>{});
    });
}

cudaError_t launch_route_backward(const void *logits, int dtype, long long ld, int T, int E, const int *idx, int K, int softmax, int renorm,
                                  float scale, const float *dw, void *out, long long ldd, bool add, cudaStream_t st) {
    const RouteGradArgs p = {logits, ld, idx, dw, out, ldd, T, E, K, softmax, renorm, add, scale};
    return by_dtype(dtype, [&](auto t) {
        using El = decltype(t);
        const int el = (int)sizeof(El);
        const long long most = (long long)sm_count() * 8;
        auto blocks = [&](long long per) {
            const long long need = (T + per - 1) / per;
            return (unsigned)(need < most ? need : most);
        };
        if (softmax && !renorm) {
            auto go = [&](auto kernel) { return launch_early(kernel, blocks(kGradWarps), 32 * kGradWarps, 0, st, 1, p); };
            const bool quads = rows_of(logits, ld, el, E, 4) && rows_of(out, ldd, el, E, 4);
            if (E <= 64) return go(route_grad_dense_kernel<El, 2, 1>);
            if (E <= 256) return quads ? go(route_grad_dense_kernel<El, 8, 4>) : go(route_grad_dense_kernel<El, 8, 1>);
            return quads ? go(route_grad_dense_kernel<El, 32, 4>) : go(route_grad_dense_kernel<El, 32, 1>);
        }
        constexpr int V = 16 / (int)sizeof(El);
        auto go = [&](auto wide, auto narrow, int kp) {
            return launch_early(rows_of(out, ldd, el, E, V) ? wide : narrow, blocks(kGradWarps * (32 / kp)), 32 * kGradWarps, 0, st, 1, p);
        };
        if (K <= 8) return go(route_grad_kernel<El, 8, V>, route_grad_kernel<El, 8, 1>, 8);
        return go(route_grad_kernel<El, 32, V>, route_grad_kernel<El, 32, 1>, 32);
    });
}

}  // namespace moe
