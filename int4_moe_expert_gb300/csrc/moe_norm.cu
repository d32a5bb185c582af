// Root-mean-square norm of a residual stream, with the addition before it and e4m3 output, and its
// gradient.  Bound by memory, or by latency for a few tokens.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_elem.h"
#include "moe_internal.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Norm.  h = x + residual (rounded to the stream's type), r = 1 / sqrt(mean h^2 + eps), y = h r w.  A
// row's elements stay in registers between the sum and the outputs: each thread holds N of them in runs of
// V neighbours, V the most that the rows' alignment allows.  A block a row, or for short rows a warp.
// The e4m3 codes are those of y; with 8 neighbours a lane, 16 lanes hold a 1 x 128 block.  A block's scale steps where its
// largest magnitude passes 448 times a power of two: a row with a block that is nearer to that than
// float32's error has its sum of squares done over in float64, so the scales are those of the formula.
// ---------------------------------------------------------------------------

struct NormArgs {
    const void *x, *res, *w;
    long long ldx, ldr, ldh, ldy;
    void *h, *y;
    float *rstd;
    uint8_t *codes;
    float *scales;         // [blocks(H), T]
    int T, H, w_dtype;
    double eps;
};

constexpr int kWarpRows = 4;       // rows of a block whose warps take a row each

// w's elements c .. c + V - 1 (float32, or the type T of x), as loaded
template <typename T, int V>
struct Weights {
    uint32_t w[V];
    __device__ __forceinline__ void load(const void *p, int w_dtype, int c) {
        if (w_dtype == MOE_DTYPE_F32) {
            Vec<float, V> u;
            u.load(static_cast<const float *>(p) + c);
#pragma unroll
            for (int i = 0; i < V; i++) w[i] = u.w[i];
        } else {
            Vec<T, V> u;
            u.load(static_cast<const T *>(p) + c);
#pragma unroll
            for (int i = 0; i < Vec<T, V>::W; i++) w[i] = u.w[i];
        }
    }
    __device__ __forceinline__ void get(int w_dtype, float *v) const {
        if (w_dtype == MOE_DTYPE_F32) {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = __uint_as_float(w[i]);
        } else {
            Vec<T, V> u;
#pragma unroll
            for (int i = 0; i < Vec<T, V>::W; i++) u.w[i] = w[i];
            u.get(v);
        }
    }
};

// 448 = 1.75 x 2^8: a magnitude (its bits) within 64 units of the step of its block's scale.  float32's
// error: 32 and 10 additions, half of it behind the root, and three more roundings, 24 units at most.
__device__ __forceinline__ bool at_border(unsigned m) { return (unsigned)(abs((int)(m & 0x7FFFFFu) - 0x600000)) <= 64u && m < 0x7F800000u; }

// S: the stream's type (T or float); N elements a thread
template <typename T, typename S, int V, int N, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024) norm_kernel(const NormArgs p) {
    constexpr int C = N / V;
    __shared__ float s_sum[2][32];
    __shared__ double s_sum64[32];
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int per = WARP ? kWarpRows : 1;
    wait_for_stream();
    int turn = 0;
    for (long long t = (long long)blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0); t < p.T; t += (long long)gridDim.x * per) {
        float v[N];
        Weights<T, V> wt[C];       // on their way during the sum
        {
            Vec<T, V> a[C];
            Vec<S, V> b[C];
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                a[i].zero();
                b[i].zero();
                if (c < p.H) {
                    a[i].load(static_cast<const T *>(p.x) + t * p.ldx + c);
                    if (p.res) b[i].load(static_cast<const S *>(p.res) + t * p.ldr + c);
                    if (p.w) wt[i].load(p.w, p.w_dtype, c);
                }
            }
#pragma unroll
            for (int i = 0; i < C; i++) {
                a[i].get(&v[V * i]);
                if (p.res) {
                    float u[V];
                    b[i].get(u);
#pragma unroll
                    for (int k = 0; k < V; k++) u[k] += v[V * i + k];
                    b[i].set(u);
                    b[i].get(&v[V * i]);
                    const int c = V * (tid + nt * i);
                    if (c < p.H) b[i].store(static_cast<S *>(p.h) + t * p.ldh + c);
                }
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < N; i++) ss = fmaf(v[i], v[i], ss);
        ss = sum_all<WARP>(ss, s_sum[turn]);
        turn ^= 1;
        const float r = 1.0f / sqrtf(ss / (float)p.H + (float)p.eps);
        if (tid == 0 && p.rstd) p.rstd[t] = r;
        // y in place of h
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            float w[V] = {};
            if (p.w && c < p.H) wt[i].get(p.w_dtype, w);
#pragma unroll
            for (int k = 0; k < V; k++) v[V * i + k] = p.w ? v[V * i + k] * r * w[k] : v[V * i + k] * r;
            if (p.y && c < p.H) {
                Vec<T, V> o;
                o.set(&v[V * i]);
                o.store(static_cast<T *>(p.y) + t * p.ldy + c);
            }
        }
        if constexpr (V == 8) {
            if (!p.codes) continue;
            unsigned most[C];
            bool near = false;
#pragma unroll
            for (int i = 0; i < C; i++) {
                unsigned m = 0;
#pragma unroll
                for (int k = 0; k < V; k++) m = max(m, abs_bits(v[V * i + k]));
#pragma unroll
                for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
                most[i] = m;
                near |= at_border(m);
            }
            if (WARP ? __any_sync(0xffffffffu, near) : __syncthreads_or(near)) {
                // the thread's own elements of h once more: as it wrote them, or x
                auto again = [&](int c, double (&u)[V]) {
                    float f[V];
                    if (p.res) {
                        Vec<S, V> b;
                        b.load(static_cast<const S *>(p.h) + t * p.ldh + c);
                        b.get(f);
                    } else {
                        Vec<T, V> a;
                        a.load(static_cast<const T *>(p.x) + t * p.ldx + c);
                        a.get(f);
                    }
#pragma unroll
                    for (int k = 0; k < V; k++) u[k] = (double)f[k];
                };
                double s = 0.0;
#pragma unroll 1
                for (int i = 0; i < C; i++) {
                    const int c = V * (tid + nt * i);
                    double u[V];
                    if (c >= p.H) break;
                    again(c, u);
#pragma unroll
                    for (int k = 0; k < V; k++) s = fma(u[k], u[k], s);
                }
                s = sum_all<WARP>(s, s_sum64);
                const double r64 = 1.0 / sqrt(s / (double)p.H + p.eps);
#pragma unroll
                for (int i = 0; i < C; i++) {
                    const int c = V * (tid + nt * i);
                    double m = 0.0;
                    if (c < p.H) {
                        double u[V];
                        float w[V];
                        again(c, u);
                        if (p.w) wt[i].get(p.w_dtype, w);
#pragma unroll
                        for (int k = 0; k < V; k++) m = fmax(m, fabs(p.w ? u[k] * (double)w[k] : u[k]));
                    }
#pragma unroll
                    for (int d = 8; d; d >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, d));
                    if (at_border(most[i])) {      // on the side that float64 says
                        const unsigned at = (most[i] & 0x7F800000u) | 0x600000u;
                        most[i] = m * r64 > (double)__uint_as_float(at) ? at + 1 : at;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                float inv;
                const float s = block_scale(most[i], inv);
                if (c < p.H) {
                    uint2 o;
                    const float *u = &v[V * i];
                    o.x = codes2(u[0] * inv, u[1] * inv) | codes2(u[2] * inv, u[3] * inv) << 16;
                    o.y = codes2(u[4] * inv, u[5] * inv) | codes2(u[6] * inv, u[7] * inv) << 16;
                    *reinterpret_cast<uint2 *>(p.codes + (size_t)t * p.H + c) = o;
                    if (c % 128 == 0) p.scales[(size_t)(c / 128) * p.T + t] = s;
                }
            }
        }
    }
}

// Gradient.  n = h r, d = dy w: dh = (d - n mean(d n)) r + grad_h, dw = sum over the tokens of dy n.
// Blocks stay and take every gridDim-th row; a thread's columns are the same in each, so its part of dw
// stays in registers, and a second kernel adds the blocks' parts in block order.
struct NormGradArgs {
    const void *dy, *h, *w, *gh;
    const float *rstd;
    long long lddy, ldh, ldg, ldo;
    void *out;
    float *part;           // [blocks][H] or NULL: no dw
    int T, H, w_dtype;
};

template <typename T, typename S, int V, int N, int THREADS, int PER_SM, bool WARP>
__global__ void __launch_bounds__(THREADS, PER_SM) norm_grad_kernel(const NormGradArgs p) {
    constexpr int C = N / V;
    extern __shared__ float norm_sm[];      // WARP: [warps][H]
    __shared__ float s_sum[2][32];
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int per = WARP ? kWarpRows : 1;
    wait_for_stream();
    float acc[N];
    Weights<T, V> wt[C];
#pragma unroll
    for (int i = 0; i < N; i++) acc[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < C; i++)
        if (p.w && V * (tid + nt * i) < p.H) wt[i].load(p.w, p.w_dtype, V * (tid + nt * i));
    int turn = 0;
    for (long long t = (long long)blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0); t < p.T; t += (long long)gridDim.x * per) {
        Vec<T, V> a[C];
        Vec<S, V> b[C], g[C];
        const float r = load_in(p.rstd + t);
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            a[i].zero();
            b[i].zero();
            g[i].zero();
            if (c < p.H) {
                a[i].load(static_cast<const T *>(p.dy) + t * p.lddy + c);
                b[i].load(static_cast<const S *>(p.h) + t * p.ldh + c);
                if (p.gh) g[i].load(static_cast<const S *>(p.gh) + t * p.ldg + c);
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < C; i++) {
            float d[V], n[V], w[V] = {};
            a[i].get(d);
            b[i].get(n);
            if (p.w && V * (tid + nt * i) < p.H) wt[i].get(p.w_dtype, w);
#pragma unroll
            for (int k = 0; k < V; k++) {
                const float dn = d[k] * (n[k] * r);
                acc[V * i + k] += dn;
                dot = p.w ? fmaf(dn, w[k], dot) : dot + dn;
            }
        }
        dot = sum_all<WARP>(dot, s_sum[turn]) / (float)p.H;
        turn ^= 1;
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            if (c >= p.H) continue;
            float d[V], n[V], w[V], u[V];
            a[i].get(d);
            b[i].get(n);
            g[i].get(u);
            if (p.w) wt[i].get(p.w_dtype, w);
#pragma unroll
            for (int k = 0; k < V; k++) u[k] = fmaf((p.w ? d[k] * w[k] : d[k]) - n[k] * r * dot, r, u[k]);
            g[i].set(u);
            g[i].store(static_cast<S *>(p.out) + t * p.ldo + c);
        }
    }
    if (!p.part) return;
    if constexpr (WARP) {
        float *mine = norm_sm + (size_t)(threadIdx.x >> 5) * p.H;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int c = V * (tid + nt * (i / V)) + i % V;
            if (c < p.H) mine[c] = acc[i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
            float s = norm_sm[c];
#pragma unroll
            for (int k = 1; k < kWarpRows; k++) s += norm_sm[(size_t)k * p.H + c];
            p.part[(size_t)blockIdx.x * p.H + c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            if (c >= p.H) continue;
#pragma unroll
            for (int k = 0; k < V; k++) p.part[(size_t)blockIdx.x * p.H + c + k] = acc[V * i + k];
        }
    }
}

// dw: 32 columns a block, its warps strands of the parts
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *part, int n, int H, float *dw) {
    __shared__ float s[32][33];
    wait_for_stream();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < H)
#pragma unroll 8
        for (int i = warp; i < n; i += 32) v += load_in(part + (size_t)i * H + c);
    s[warp][lane] = v;
    __syncthreads();
    v = s[lane][warp];          // the strands of column `warp`
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int col = (int)blockIdx.x * 32 + warp;
    if (lane == 0 && col < H) dw[col] = v;
}

}  // namespace

// 16 elements a thread in blocks that leave it 85 registers (8 up to 256, a warp a row, and from 6145 to 8192)
struct GradShape {
    int threads, per_sm;
};
static GradShape norm_grad_shape(int H) {
    if (H <= 256) return {32 * kWarpRows, 8};
    const int n = H > 6144 && H <= 8192 ? 8 : 16, threads = ((H + n - 1) / n + 31) / 32 * 32;
    return {threads, threads <= 128 ? 6 : threads <= 256 ? 3 : threads <= 384 ? 2 : 1};
}
int norm_grad_blocks(int T, int H) {
    if (T <= 0) return 0;
    const long long per = H <= 256 ? kWarpRows : 1, most = (long long)sm_count() * norm_grad_shape(H).per_sm, need = (T + per - 1) / per;
    return (int)(need < most ? need : most);
}
size_t norm_grad_workspace(int T, int H) { return (size_t)norm_grad_blocks(T, H) * H * sizeof(float); }

cudaError_t launch_norm_forward(const void *x, int dtype, long long ldx, const void *res, int s_dtype, long long ldr, const void *w, int w_dtype,
                                int T, int H, double eps, void *h, long long ldh, void *y, long long ldy, float *rstd, uint8_t *codes,
                                float *scales, cudaStream_t st) {
    const NormArgs p = {x, res, w, ldx, ldr, ldh, ldy, h, y, rstd, codes, scales, T, H, w_dtype, eps};
    auto go = [&](auto xt, auto stt) {
        using X = decltype(xt);
        using S = decltype(stt);
        // V neighbours of every tensor's rows together
        auto fits = [&](int v) {
            return H % v == 0 && runs_of(x, ldx, sizeof(X), min(16, v * (int)sizeof(X))) && (!res || (runs_of(res, ldr, sizeof(S), min(16, v * (int)sizeof(S))) && runs_of(h, ldh, sizeof(S), min(16, v * (int)sizeof(S))))) &&
                   (!y || runs_of(y, ldy, sizeof(X), min(16, v * (int)sizeof(X)))) && (!w || runs_of(w, 0, 4, min(16, v * (w_dtype == MOE_DTYPE_F32 ? 4 : 2))));
        };
        auto run = [&](auto kernel, int n, bool warp) {
            if (warp) return launch_early(kernel, (unsigned)((T + kWarpRows - 1) / kWarpRows), 32 * kWarpRows, 0, st, 1, p);
            const int threads = ((H + n - 1) / n + 31) / 32 * 32;
            return launch_early(kernel, (unsigned)T, threads, 0, st, 1, p);
        };
        // 8 elements a thread where that makes the block for few rows, 16 otherwise
        const bool few = T < 2 * sm_count() && H <= 8192;
        auto by_run = [&](auto v) {
            constexpr int V = decltype(v)::value;
            if (H <= 256) return run(norm_kernel<X, S, V, 8, true>, 8, true);
            if (few) return run(norm_kernel<X, S, V, 8, false>, 8, false);
            if (H <= 512) return run(norm_kernel<X, S, V, 16, true>, 16, true);
            return run(norm_kernel<X, S, V, 16, false>, 16, false);
        };
        if (fits(8)) return by_run(std::integral_constant<int, 8>{});
        if (fits(2)) return by_run(std::integral_constant<int, 2>{});
        return by_run(std::integral_constant<int, 1>{});
    };
    return by_dtype(dtype, [&](auto xt) {
        if (s_dtype == MOE_DTYPE_F32) return go(xt, float{});
        return go(xt, xt);
    });
}

cudaError_t launch_norm_backward(const void *dy, int dtype, long long lddy, const void *h, int s_dtype, long long ldh, const float *rstd, const void *w,
                                 int w_dtype, const void *gh, long long ldg, int T, int H, void *out, long long ldo, float *dw, void *ws,
                                 cudaStream_t st) {
    const NormGradArgs p = {dy, h, w, gh, rstd, lddy, ldh, ldg, ldo, out, dw ? static_cast<float *>(ws) : nullptr, T, H, w_dtype};
    const int blocks = norm_grad_blocks(T, H);
    auto go = [&](auto xt, auto stt) {
        using X = decltype(xt);
        using S = decltype(stt);
        auto fits = [&](int v) {
            const int bx = min(16, v * (int)sizeof(X)), bs = min(16, v * (int)sizeof(S));
            return H % v == 0 && runs_of(dy, lddy, sizeof(X), bx) && runs_of(h, ldh, sizeof(S), bs) && runs_of(out, ldo, sizeof(S), bs) &&
                   (!gh || runs_of(gh, ldg, sizeof(S), bs)) && (!w || runs_of(w, 0, 4, min(16, v * (w_dtype == MOE_DTYPE_F32 ? 4 : 2))));
        };
        const int threads = norm_grad_shape(H).threads;
        auto by_run = [&](auto v) {
            constexpr int V = decltype(v)::value;
            if (H <= 256)
                return launch_early(norm_grad_kernel<X, S, V, 8, 32 * kWarpRows, 8, true>, blocks, threads, dw ? (size_t)kWarpRows * H * sizeof(float) : 0, st, 1, p);
            if (threads <= 128) return launch_early(norm_grad_kernel<X, S, V, 16, 128, 6, false>, blocks, threads, 0, st, 1, p);
            if (threads <= 256) return launch_early(norm_grad_kernel<X, S, V, 16, 256, 3, false>, blocks, threads, 0, st, 1, p);
            if (threads <= 384) return launch_early(norm_grad_kernel<X, S, V, 16, 384, 2, false>, blocks, threads, 0, st, 1, p);
            if (H <= 8192) return launch_early(norm_grad_kernel<X, S, V, 8, 1024, 1, false>, blocks, threads, 0, st, 1, p);
            return launch_early(norm_grad_kernel<X, S, V, 16, 1024, 1, false>, blocks, threads, 0, st, 1, p);
        };
        if (fits(8)) return by_run(std::integral_constant<int, 8>{});
        if (fits(2)) return by_run(std::integral_constant<int, 2>{});
        return by_run(std::integral_constant<int, 1>{});
    };
    const cudaError_t e = by_dtype(dtype, [&](auto xt) {
        if (s_dtype == MOE_DTYPE_F32) return go(xt, float{});
        return go(xt, xt);
    });
    if (e != cudaSuccess || !dw) return e;
    return launch_early(norm_dw_kernel, (unsigned)((H + 31) / 32), 1024, 0, st, 1, p.part, blocks, H, dw);
}

}  // namespace moe
