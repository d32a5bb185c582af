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
// V neighbours.  A block a row, or for short rows a warp.
// The e4m3 codes are those of y; with 8 neighbours a lane, 16 lanes hold a 1 x 128 block.  A block's scale steps where its
// largest magnitude passes 448 times a power of two: a row with a block that is nearer to that than
// float32's error has its sum of squares done over in float64, so the scales are those of the formula.  A row whose
// squares leave float32's range is squared once more behind a power of two.
// 32768 x 2048 bf16 on a float32 stream: 117 us at the copy rate; 16381 x 6144 bf16 with values and codes 142 us of
// 134 (59 % of the issue slots: codes and scales).  Rows of odd widths go element by element: 8192 x 4095 bf16
// 58 us of 40, f32 82 us of 79.
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
    float per_h, per_h_rest, eps32, eps_rest, eps_root;      // 1 / H and eps in two parts, the square root of eps
};

constexpr int kWarpRows = 4;       // rows of a block whose warps take a row each
extern __shared__ uint4 norm_shared[];

// A thread's weights (float32, or the type T of x) as loaded: C runs of V, nt V apart.  Every condition that all
// elements share stands outside the loops over them: rows of single elements would be branches otherwise.
template <typename T, int V, int C>
struct Weights {
    uint32_t w[C * V];
    __device__ __forceinline__ void load(const void *p, int w_dtype, int tid, int nt, int H) {
        if (w_dtype == MOE_DTYPE_F32) load_as(static_cast<const float *>(p), tid, nt, H);
        else load_as(static_cast<const T *>(p), tid, nt, H);
    }
    // f(i, weights of run i as float32) for every run
    template <typename F>
    __device__ __forceinline__ void each(int w_dtype, F &&f) const {
        if (w_dtype == MOE_DTYPE_F32) each_as<float>(f);
        else each_as<T>(f);
    }

private:
    template <typename E>
    __device__ __forceinline__ void load_as(const E *p, int tid, int nt, int H) {
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            Vec<E, V> u;
            u.zero();
            if (c < H) u.load(p + c);
#pragma unroll
            for (int k = 0; k < Vec<E, V>::W; k++) w[V * i + k] = u.w[k];
        }
    }
    template <typename E, typename F>
    __device__ __forceinline__ void each_as(F &&f) const {
#pragma unroll
        for (int i = 0; i < C; i++) {
            Vec<E, V> u;
            float v[V];
#pragma unroll
            for (int k = 0; k < Vec<E, V>::W; k++) u.w[k] = w[V * i + k];
            u.get(v);
            f(i, v);
        }
    }
};

// the larger magnitude; a NaN is the largest
__device__ __forceinline__ float larger(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// 448 = 1.75 x 2^8: a magnitude (its bits) within 64 units of the step of its block's scale.  float32's
// error: 32 and 10 additions, half of it behind the root, and three more roundings, 24 units at most.
__device__ __forceinline__ bool at_border(unsigned m) { return (unsigned)(abs((int)(m & 0x7FFFFFu) - 0x600000)) <= 64u && m < 0x7F800000u; }

// The thread's elements of h (v) become y, codes and scales; S: the stream's type (T or float), V neighbours
// together, N elements a thread.
template <typename T, typename S, int V, int N>
__device__ __forceinline__ void norm_outputs(const NormArgs &p, long long t, int tid, int nt, float (&v)[N], float r, const Weights<T, V, N / V> &wt) {
    constexpr int C = N / V;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] *= r;
    if (p.w)
        wt.each(p.w_dtype, [&](int i, const float *w) {
#pragma unroll
            for (int k = 0; k < V; k++) v[V * i + k] *= w[k];
        });
    if (p.y) {
        T *y = static_cast<T *>(p.y) + t * p.ldy;
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            Vec<T, V> o;
            o.set(&v[V * i]);
            if (c < p.H) o.store(y + c);
        }
    }
    if constexpr (V == 8) {
        if (!p.codes) return;
        // The largest magnitude of a run's 1 x 128 block, over its 16 lanes.  Two runs meet in one butterfly: the lanes'
        // upper half ends with the second's.
        static_assert(C == 1 || C == 2, "");
        const bool upper = C == 2 && (threadIdx.x & 8);
        float m[C];
#pragma unroll
        for (int i = 0; i < C; i++) {
            m[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < V; k++) m[i] = larger(m[i], v[V * i + k]);
        }
        float mine = upper ? m[C - 1] : m[0];
        mine = larger(mine, __shfl_xor_sync(0xffffffffu, C == 2 && !upper ? m[C - 1] : m[0], 8));
#pragma unroll
        for (int d = 4; d; d >>= 1) mine = larger(mine, __shfl_xor_sync(0xffffffffu, mine, d));
        unsigned most = __float_as_uint(mine);
        const bool near = at_border(most);
        if (__any_sync(0xffffffffu, near)) {
            // h once more, as it was written, or x: the row's sum by this warp alone
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
            for (int c = V * (threadIdx.x & 31); c < p.H; c += 32 * V) {
                double u[V];
                again(c, u);
#pragma unroll
                for (int k = 0; k < V; k++) s = fma(u[k], u[k], s);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            const double r64 = 1.0 / sqrt(s / (double)p.H + p.eps);
            double m64[C];
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                m64[i] = 0.0;
                if (c < p.H) {
                    double u[V];
                    float w[V];
                    again(c, u);
#pragma unroll
                    for (int k = 0; k < V; k++) w[k] = 1.0f;
                    if (p.w && p.w_dtype == MOE_DTYPE_F32) {
                        Vec<float, V> q;
                        q.load(static_cast<const float *>(p.w) + c);
                        q.get(w);
                    } else if (p.w) {
                        Vec<T, V> q;
                        q.load(static_cast<const T *>(p.w) + c);
                        q.get(w);
                    }
#pragma unroll
                    for (int k = 0; k < V; k++) m64[i] = fmax(m64[i], fabs(u[k] * (double)w[k]));
                }
#pragma unroll
                for (int d = 8; d; d >>= 1) m64[i] = fmax(m64[i], __shfl_xor_sync(0xffffffffu, m64[i], d));
            }
            if (near) {      // on the side that float64 says
                const unsigned at = (most & 0x7F800000u) | 0x600000u;
                most = (upper ? m64[C - 1] : m64[0]) * r64 > (double)__uint_as_float(at) ? at + 1 : at;
            }
        }
        float inv_mine;
        const float scale = block_scale(most, inv_mine);
        const float inv_other = C == 2 ? __shfl_xor_sync(0xffffffffu, inv_mine, 8) : inv_mine;
        {      // the first lane of a run's 16, and for the second run the first of the upper half
            const int c = V * ((tid & ~8) + (upper ? nt : 0));
            if ((threadIdx.x & 7) == 0 && (C == 2 || !(threadIdx.x & 8)) && c < p.H) p.scales[(size_t)(c / 128) * p.T + t] = scale;
        }
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            const float inv = upper == (i == 1) ? inv_mine : inv_other;
            if (c < p.H) {
                uint2 o;
                const float *u = &v[V * i];
                o.x = codes2(u[0] * inv, u[1] * inv) | codes2(u[2] * inv, u[3] * inv) << 16;
                o.y = codes2(u[4] * inv, u[5] * inv) | codes2(u[6] * inv, u[7] * inv) << 16;
                *reinterpret_cast<uint2 *>(p.codes + (size_t)t * p.H + c) = o;
            }
        }
    }
}

// 1 / sqrt(s) of s = mean + eps with little more than its last rounding: the mean and the sum in two parts each, and one
// step of Newton's from the function's value.  (An error here is one of the whole row, and of its codes near a rounding.)
__device__ __forceinline__ float norm_rstd(const NormArgs &p, float ss, float mean, float s, float eps, float eps_rest) {
    const float back = s - mean;
    const float rest = fmaf(ss, p.per_h, -mean) + fmaf(ss, p.per_h_rest, eps_rest) + ((mean - (s - back)) + (eps - back));
    const float r = rsqrtf(s), q = s * r;
    return fmaf(0.5f * r, fmaf(-q, r, 1.0f) - fmaf(rest, r, fmaf(s, r, -q)) * r, r);
}

template <typename T, typename S, int V, int N, int THREADS, int PER_SM, bool WARP>
__global__ void __launch_bounds__(THREADS, PER_SM) norm_kernel(const NormArgs p) {
    constexpr int C = N / V;
    // weights on their way during the sum; not beside four bytes an element of x (8192 x 6144 f32: 125 us so, 118 behind it)
    constexpr bool EARLY = sizeof(T) == 2;
    __shared__ float s_sum[2][32];
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : V < 8 && N == 16 ? THREADS : blockDim.x;
    const int per = WARP ? kWarpRows : 1;
    wait_for_stream();
    const long long t = (long long)blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0);
    if (t >= p.T) return;      // a warp without a row
    float v[N];
    Weights<T, V, C> wt;
    {
        Vec<T, V> a[C];
        const T *x = static_cast<const T *>(p.x) + t * p.ldx;
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            a[i].zero();
            if (c < p.H) a[i].load(x + c);
        }
        if (EARLY && p.w) wt.load(p.w, p.w_dtype, tid, nt, p.H);
        if (p.res) {
            Vec<S, V> b[C];
            const S *res = static_cast<const S *>(p.res) + t * p.ldr;
            S *h = static_cast<S *>(p.h) + t * p.ldh;
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                b[i].zero();
                if (c < p.H) b[i].load(res + c);
            }
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                float u[V];
                a[i].get(&v[V * i]);
                b[i].get(u);
#pragma unroll
                for (int k = 0; k < V; k++) u[k] += v[V * i + k];
                b[i].set(u);
                b[i].get(&v[V * i]);
                if (c < p.H) b[i].store(h + c);
            }
        } else {
#pragma unroll
            for (int i = 0; i < C; i++) a[i].get(&v[V * i]);
        }
    }
    // Squares that leave float32's range are taken again behind a power of two.  A mean between 2^-100 and 2^100 is
    // none of them: the row's sum is below 2^114, and what a square below 2^-126 loses, 2^-150, is nothing.  Scaled
    // ones are between 2^-98 and 2^114.  Small rows stay scaled (no element is past 2^-43), so that y is right where
    // rstd is more than float32 holds; large ones would lose small elements.
    float r, up = 1.0f, down = 1.0f, eps = p.eps32, eps_rest = p.eps_rest;
    for (int turn = 0;; turn++) {
        float ss = 0.0f;
        if (down == 1.0f) {
#pragma unroll
            for (int i = 0; i < N; i++) ss = fmaf(v[i], v[i], ss);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) ss = fmaf(v[i] * down, v[i] * down, ss);
        }
        ss = sum_all<WARP>(ss, s_sum[turn]);       // alike in all threads of the row
        const float mean = ss * p.per_h, s = mean + eps;
        if (s > 0x1p-100f && s < 0x1p100f) {
            r = norm_rstd(p, ss, mean, s, eps, eps_rest) * down;
            break;
        }
        if (turn == 1) {       // zeros, or an infinity or a NaN
            r = rsqrtf(s);
            break;
        }
        if (s < 1.0f) {
            up = 0x1p100f;
#pragma unroll
            for (int i = 0; i < N; i++) v[i] *= up;
        } else {
            down = 0x1p-80f;
        }
        const float root = p.eps_root * (up * down);
        eps = root * root;
        eps_rest = 0.0f;
    }
    if (WARP) __syncwarp();      // the row's h is written, for all lanes
    if (!EARLY && p.w) wt.load(p.w, p.w_dtype, tid, nt, p.H);
    if (tid == 0 && p.rstd) p.rstd[t] = r * up;
    norm_outputs<T, S, V, N>(p, t, tid, nt, v, r, wt);
}

// Gradient.  n = h r, d = dy w: dh = (d - n mean(d n)) r + grad_h, dw = sum over the tokens of dy n.  n comes first
// everywhere: d h leaves float32's range where d n does not.
// Blocks stay and take every gridDim-th row; a thread's columns are the same in each, so its part of dw
// stays in registers, and a second kernel adds the blocks' parts in block order.  Bound by memory up to 6144 columns
// (32768 x 2048 bf16 on float32 144 us of 139, 8192 x 6144 f32 131 of 119); beyond, an SM has one block of a float32
// stream, whose loads wait for its row's sum (8192 x 8192 f32 189 us of 158, bf16 on float32 208 of 139).
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
    float *norm_sm = reinterpret_cast<float *>(norm_shared);      // WARP: [warps][H]
    __shared__ float s_sum[2][32];
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : V == 1 ? THREADS : blockDim.x;
    const int per = WARP ? kWarpRows : 1;
    wait_for_stream();
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; i++) acc[i] = 0.0f;
    int turn = 0;
    for (long long t = (long long)blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0); t < p.T; t += (long long)gridDim.x * per) {
        Vec<T, V> a[C];
        Vec<S, V> b[C], g[C];
        const float r = load_in(p.rstd + t);
        const T *dy = static_cast<const T *>(p.dy) + t * p.lddy;
        const S *h = static_cast<const S *>(p.h) + t * p.ldh, *gh = static_cast<const S *>(p.gh) + t * p.ldg;
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = V * (tid + nt * i);
            a[i].zero();
            b[i].zero();
            g[i].zero();
            if (c < p.H) {
                a[i].load(dy + c);
                b[i].load(h + c);
            }
        }
        if (p.gh) {
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                if (c < p.H) g[i].load(gh + c);
            }
        }
        S *out = static_cast<S *>(p.out) + t * p.ldo;
        float dot = 0.0f;
        if constexpr (V == 8) {
            // dy w run by run, before the sum and behind it: its registers are worth more than the loads from L1
            // (32768 x 2048, bf16 on float32: 145 us, kept in registers 155)
            auto weight = [&](int c, float *w) {
                if (p.w_dtype == MOE_DTYPE_F32) {
                    Vec<float, V> q;
                    q.load(static_cast<const float *>(p.w) + c);
                    q.get(w);
                } else {
                    Vec<T, V> q;
                    q.load(static_cast<const T *>(p.w) + c);
                    q.get(w);
                }
            };
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                float d[V], n[V], w[V] = {};
                a[i].get(d);
                b[i].get(n);
                if (p.w && c < p.H) weight(c, w);
#pragma unroll
                for (int k = 0; k < V; k++) {
                    const float dn = d[k] * (n[k] * r);
                    acc[V * i + k] += dn;
                    dot = p.w ? fmaf(dn, w[k], dot) : dot + dn;
                }
            }
            dot = sum_all<WARP>(dot, s_sum[turn]) / (float)p.H;
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                if (c >= p.H) continue;
                float d[V], n[V], w[V], u[V];
                a[i].get(d);
                b[i].get(n);
                g[i].get(u);
                if (p.w) weight(c, w);
#pragma unroll
                for (int k = 0; k < V; k++) u[k] = fmaf((p.w ? d[k] * w[k] : d[k]) - n[k] * r * dot, r, u[k]);
                g[i].set(u);
                g[i].store(out + c);
            }
        } else {
            float d[N], n[N];      // d: dy w
#pragma unroll
            for (int i = 0; i < C; i++) {
                a[i].get(&d[V * i]);
                b[i].get(&n[V * i]);
            }
#pragma unroll
            for (int i = 0; i < N; i++) {
                n[i] *= r;
                acc[i] = fmaf(d[i], n[i], acc[i]);
            }
            if (p.w) {
                Weights<T, V, C> wt;
                wt.load(p.w, p.w_dtype, tid, nt, p.H);
                wt.each(p.w_dtype, [&](int i, const float *w) {
#pragma unroll
                    for (int k = 0; k < V; k++) d[V * i + k] *= w[k];
                });
            }
#pragma unroll
            for (int i = 0; i < N; i++) dot = fmaf(d[i], n[i], dot);
            const float back = -sum_all<WARP>(dot, s_sum[turn]) / (float)p.H;
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = V * (tid + nt * i);
                float u[V];
                g[i].get(u);
#pragma unroll
                for (int k = 0; k < V; k++) u[k] = fmaf(fmaf(n[V * i + k], back, d[V * i + k]), r, u[k]);
                g[i].set(u);
                if (c < p.H) g[i].store(out + c);
            }
        }
        turn ^= 1;
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

// 16-bit streams: every thread copies its own elements of the next D - 1 rows to shared memory while it works on
// one (asynchronous copies of 16 bytes, which no other thread waits for), so that the bytes in flight do not
// depend on the registers (16384 x 2048 bf16: 60 us without, 53 us with; 16381 x 6144 170 and 145 us).  Float32
// streams do without: the copies fill the shared memory that their warps would need (32768 x 2048, bf16 on
// float32: 146 and 213 us).
__device__ __forceinline__ void async_copy(uint4 *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void async_wait_all_but(int n) {      // groups: 0, 1 or 2
    if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
constexpr int kRingN = 16;      // elements a thread

// unit u of the thread in a ring of units
__device__ __forceinline__ uint4 *ring_unit(int u) { return norm_shared + (size_t)u * blockDim.x + threadIdx.x; }
template <typename T>
__device__ __forceinline__ void ring_fetch(int u, const T *src) {      // 8 elements
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) async_copy(ring_unit(u + i), reinterpret_cast<const uint4 *>(src) + i);
}
template <typename T>
__device__ __forceinline__ Vec<T, 8> ring_get(int u) {
    Vec<T, 8> v;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) {
        const uint4 q = *ring_unit(u + i);
        v.w[4 * i] = q.x;
        v.w[4 * i + 1] = q.y;
        v.w[4 * i + 2] = q.z;
        v.w[4 * i + 3] = q.w;
    }
    return v;
}
constexpr int ring_units(int n, int t, int s, int streams, int d) { return (n / 8) * d * (t / 2 + streams * (s / 2)); }

// The same through a ring of D rows of dy, h and grad_h.
template <typename T, typename S, int THREADS, int PER_SM, bool WARP>
__global__ void __launch_bounds__(THREADS, PER_SM) norm_grad_ring_kernel(const NormGradArgs p, const int D) {
    constexpr int N = kRingN, C = N / 8, UX = sizeof(T) / 2, US = sizeof(S) / 2, STAGE = C * (UX + 2 * US);
    __shared__ float s_sum[2][32];
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int per = WARP ? kWarpRows : 1;
    const long long first = (long long)blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0), step = (long long)gridDim.x * per;
    wait_for_stream();
    auto fetch = [&](long long t, int stage) {
        if (t < p.T) {
#pragma unroll
            for (int i = 0; i < C; i++) {
                const int c = 8 * (tid + nt * i), u = stage * STAGE;
                if (c < p.H) {
                    ring_fetch(u + i * UX, static_cast<const T *>(p.dy) + t * p.lddy + c);
                    ring_fetch(u + C * UX + i * US, static_cast<const S *>(p.h) + t * p.ldh + c);
                    if (p.gh) ring_fetch(u + C * (UX + US) + i * US, static_cast<const S *>(p.gh) + t * p.ldg + c);
                }
            }
        }
        async_commit();
    };
    float r_next = first < p.T ? load_in(p.rstd + first) : 0.0f;
    for (int d = 0; d < D - 1; d++) fetch(first + d * step, d);
    float acc[N], w[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        acc[i] = 0.0f;
        w[i] = 1.0f;
    }
    if (p.w) {
        Weights<T, 8, C> q;
        q.load(p.w, p.w_dtype, tid, nt, p.H);
        q.each(p.w_dtype, [&](int i, const float *f) {
#pragma unroll
            for (int k = 0; k < 8; k++) w[8 * i + k] = f[k];
        });
    }
    int turn = 0, stage = 0;
    for (long long t = first; t < p.T; t += step) {
        fetch(t + (D - 1) * step, stage == 0 ? D - 1 : stage - 1);
        const float r = r_next;
        if (t + step < p.T) r_next = load_in(p.rstd + t + step);
        async_wait_all_but(D - 1);
        const int u = stage * STAGE;
        float d[N], n[N], dot = 0.0f;      // d = dy w
#pragma unroll
        for (int i = 0; i < C; i++) {
            if (8 * (tid + nt * i) >= p.H) continue;
            ring_get<T>(u + i * UX).get(&d[8 * i]);
            ring_get<S>(u + C * UX + i * US).get(&n[8 * i]);
#pragma unroll
            for (int k = 8 * i; k < 8 * i + 8; k++) {
                n[k] *= r;
                acc[k] = fmaf(d[k], n[k], acc[k]);
                d[k] *= w[k];
                dot = fmaf(d[k], n[k], dot);
            }
        }
        const float back = -sum_all<WARP>(dot, s_sum[turn]) / (float)p.H;
        turn ^= 1;
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = 8 * (tid + nt * i);
            if (c >= p.H) continue;
            float o[8] = {};
            Vec<S, 8> q;
            if (p.gh) {
                q = ring_get<S>(u + C * (UX + US) + i * US);
                q.get(o);
            }
#pragma unroll
            for (int k = 0; k < 8; k++) o[k] = fmaf(fmaf(n[8 * i + k], back, d[8 * i + k]), r, o[k]);
            q.set(o);
            q.store(static_cast<S *>(p.out) + t * p.ldo + c);
        }
        stage = stage == D - 1 ? 0 : stage + 1;
    }
    async_wait_all_but(0);
    if (!p.part) return;
    if constexpr (WARP) {      // the warps' parts, in order, through the ring
        float *sums = reinterpret_cast<float *>(norm_shared);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int c = 8 * (tid + nt * (i / 8)) + i % 8;
            if (c < p.H) sums[(threadIdx.x >> 5) * p.H + c] = acc[i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
            float s = sums[c];
#pragma unroll
            for (int k = 1; k < kWarpRows; k++) s += sums[k * p.H + c];
            p.part[(size_t)blockIdx.x * p.H + c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; i++) {
            const int c = 8 * (tid + nt * i);
            if (c >= p.H) continue;
#pragma unroll
            for (int k = 0; k < 2; k++)
                *reinterpret_cast<float4 *>(p.part + (size_t)blockIdx.x * p.H + c + 4 * k) = make_float4(acc[8 * i + 4 * k], acc[8 * i + 4 * k + 1], acc[8 * i + 4 * k + 2], acc[8 * i + 4 * k + 3]);
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

// A ring kernel's shape: 16 elements a thread, a warp a row up to 512, blocks that leave a thread 80 registers (64 in
// blocks of more than 384), rings of three rows where an SM holds them for its blocks, else of two, else of two for fewer
// blocks; none (depth 0) for rows that are too long.
struct RingShape {
    int threads, depth, per_sm;
    size_t smem;
};
constexpr size_t kRingSmem = 220 * 1024;       // of an SM
static int ring_threads(int H) { return H <= 32 * kRingN ? 32 * kWarpRows : ((H + kRingN - 1) / kRingN + 31) / 32 * 32; }
static int ring_per_sm(int threads) { return threads <= 128 ? 768 / threads : threads <= 256 ? 3 : threads <= 512 ? 2 : 1; }
static RingShape ring_shape(int H, int t, int s, int streams) {
    RingShape r = {ring_threads(H), 0, 0, 0};
    const int want = ring_per_sm(r.threads);
    for (int per_sm = want; per_sm >= 1; per_sm--)
        for (int d = per_sm == want ? 3 : 2; d >= 2; d--) {
            const size_t bytes = (size_t)ring_units(kRingN, t, s, streams, d) * r.threads * 16;
            if (per_sm * (bytes + 1536) <= kRingSmem) return {r.threads, d, per_sm, bytes};
        }
    return r;
}
static int norm_blocks(int T, int per, int per_sm) {      // per: rows of a block
    const long long most = (long long)sm_count() * per_sm, need = ((long long)T + per - 1) / per;
    return (int)(need < most ? need : most);
}
// f(kernel's threads, blocks of an SM, a warp a row): the class of a ring kernel
template <typename F>
static cudaError_t ring_class(int H, int threads, F &&f) {
    using std::integral_constant;
    if (H <= 32 * kRingN) return f(integral_constant<int, 128>{}, integral_constant<int, 6>{}, std::true_type{});
    if (threads <= 128) return f(integral_constant<int, 128>{}, integral_constant<int, 6>{}, std::false_type{});
    if (threads <= 256) return f(integral_constant<int, 256>{}, integral_constant<int, 3>{}, std::false_type{});
    if (threads <= 384) return f(integral_constant<int, 384>{}, integral_constant<int, 2>{}, std::false_type{});
    if (threads <= 512) return f(integral_constant<int, 512>{}, integral_constant<int, 2>{}, std::false_type{});
    return f(integral_constant<int, 1024>{}, integral_constant<int, 1>{}, std::false_type{});
}
// threads and blocks of an SM of the kernel that reads straight from memory: 16 elements a thread, a warp a row up to 256
static int direct_threads(int H) { return H <= 256 ? 32 * kWarpRows : ((H + 15) / 16 + 31) / 32 * 32; }
static int direct_per_sm(int H, int threads) { return H <= 256 ? 6 : threads <= 128 ? 640 / threads : threads <= 256 ? 3 : threads <= 384 ? 2 : 1; }
// at most, whatever the types and alignment
int norm_grad_blocks(int T, int H) {
    if (T <= 0) return 0;
    const int a = norm_blocks(T, H <= 32 * kRingN ? kWarpRows : 1, ring_per_sm(ring_threads(H))), b = norm_blocks(T, H <= 256 ? kWarpRows : 1, direct_per_sm(H, direct_threads(H)));
    return a > b ? a : b;
}
size_t norm_grad_workspace(int T, int H) { return (size_t)norm_grad_blocks(T, H) * H * sizeof(float); }

cudaError_t launch_norm_forward(const void *x, int dtype, long long ldx, const void *res, int s_dtype, long long ldr, const void *w, int w_dtype,
                                int T, int H, double eps, void *h, long long ldh, void *y, long long ldy, float *rstd, uint8_t *codes,
                                float *scales, cudaStream_t st) {
    const NormArgs p = {x, res, w, ldx, ldr, ldh, ldy, h, y, rstd, codes, scales, T, H, w_dtype, eps, (float)(1.0 / H), (float)(1.0 / H - (float)(1.0 / H)), (float)eps, (float)(eps - (float)eps), (float)sqrt(eps)};
    auto go = [&](auto xt, auto stt) {
        using X = decltype(xt);
        using S = decltype(stt);
        // V neighbours of every tensor's rows together
        auto fits = [&](int v) {
            return H % v == 0 && runs_of(x, ldx, sizeof(X), min(16, v * (int)sizeof(X))) && (!res || (runs_of(res, ldr, sizeof(S), min(16, v * (int)sizeof(S))) && runs_of(h, ldh, sizeof(S), min(16, v * (int)sizeof(S))))) &&
                   (!y || runs_of(y, ldy, sizeof(X), min(16, v * (int)sizeof(X)))) && (!w || runs_of(w, 0, 4, min(16, v * (w_dtype == MOE_DTYPE_F32 ? 4 : 2))));
        };
        auto run = [&](auto kernel, int threads, int rows) {
            return launch_early(kernel, (unsigned)(((long long)T + rows - 1) / rows), threads, 0, st, 1, p);
        };
        auto up = [](int n) { return (n + 31) / 32 * 32; };
        const int few = up((H + 7) / 8), threads = up((H + 15) / 16);      // with 8 and 16 elements a thread
        auto by_run = [&](auto v) {
            constexpr int V = decltype(v)::value;
            if (H <= 256) return run(norm_kernel<X, S, V, 8, 32 * kWarpRows, 8, true>, 32 * kWarpRows, kWarpRows);
            if (T < 2 * sm_count() && H <= 8192) return run(norm_kernel<X, S, V, 8, 1024, 1, false>, few, 1);
            // 64 registers a thread, 56 for 384 threads (three blocks: 16381 x 6144 bf16 with codes 155 us, with two 165).
            // Single elements and pairs take every thread of their class, whose number is a constant then: elements that
            // a number known at run time lies between have an address each (8192 x 4095 bf16: 110 us, 60 so).
            constexpr bool WHOLE = V < 8;
            if constexpr (WHOLE) {
                if (threads <= 32) return run(norm_kernel<X, S, V, 16, 32, 32, false>, 32, 1);
                if (threads <= 64) return run(norm_kernel<X, S, V, 16, 64, 16, false>, 64, 1);
            }
            if (threads <= 128) return run(norm_kernel<X, S, V, 16, 128, 8, false>, WHOLE ? 128 : threads, 1);
            if (threads <= 256) return run(norm_kernel<X, S, V, 16, 256, 4, false>, WHOLE ? 256 : threads, 1);
            if (threads <= 384) return run(norm_kernel<X, S, V, 16, 384, WHOLE ? 2 : 3, false>, WHOLE ? 384 : threads, 1);
            if (threads <= 512) return run(norm_kernel<X, S, V, 16, 512, 2, false>, WHOLE ? 512 : threads, 1);
            return run(norm_kernel<X, S, V, 16, 1024, 1, false>, WHOLE ? 1024 : threads, 1);
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
    int blocks = 0;
    auto go = [&](auto xt, auto stt) {
        using X = decltype(xt);
        using S = decltype(stt);
        auto fits = [&](int v) {
            const int bx = min(16, v * (int)sizeof(X)), bs = min(16, v * (int)sizeof(S));
            return H % v == 0 && runs_of(dy, lddy, sizeof(X), bx) && runs_of(h, ldh, sizeof(S), bs) && runs_of(out, ldo, sizeof(S), bs) &&
                   (!gh || runs_of(gh, ldg, sizeof(S), bs)) && (!w || runs_of(w, 0, 4, min(16, v * (w_dtype == MOE_DTYPE_F32 ? 4 : 2))));
        };
        const bool eights = fits(8);
        if constexpr (sizeof(S) == 2) {
            const RingShape r = ring_shape(H, sizeof(X), sizeof(S), 2);
            if (eights && r.depth) {
                blocks = norm_blocks(T, H <= 32 * kRingN ? kWarpRows : 1, r.per_sm);
                return ring_class(H, r.threads, [&](auto th, auto per, auto warp) {
                    constexpr auto kernel = norm_grad_ring_kernel<X, S, decltype(th)::value, decltype(per)::value, decltype(warp)::value>;
                    const cudaError_t e = allow_smem<kernel>(kRingSmem);
                    return e != cudaSuccess ? e : launch_early(kernel, blocks, r.threads, r.smem, st, 1, p, r.depth);
                });
            }
        }
        auto by_run = [&](auto v) {
            constexpr int V = decltype(v)::value;
            // single elements take every thread of their class, as in the forward pass (8192 x 4095 bf16: 127 us, 85 so);
            // pairs gain less and lose beyond 8192 (4096 x 9002 bf16: 117 us, 138 so)
            constexpr bool WHOLE = V == 1;
            const int own = direct_threads(H);
            const int threads = !WHOLE || H <= 256 ? own : own <= 32 ? 32 : own <= 64 ? 64 : own <= 128 ? 128 : own <= 256 ? 256 : own <= 384 ? 384 : own <= 512 ? 512 : own <= 768 ? 768 : 1024;
            blocks = norm_blocks(T, H <= 256 ? kWarpRows : 1, direct_per_sm(H, threads));
            if (H <= 256)
                return launch_early(norm_grad_kernel<X, S, V, 8, 32 * kWarpRows, 6, true>, blocks, threads, dw ? (size_t)kWarpRows * H * sizeof(float) : 0, st, 1, p);
            if constexpr (WHOLE) {
                if (threads <= 32) return launch_early(norm_grad_kernel<X, S, V, 16, 32, 20, false>, blocks, threads, 0, st, 1, p);
                if (threads <= 64) return launch_early(norm_grad_kernel<X, S, V, 16, 64, 10, false>, blocks, threads, 0, st, 1, p);
            }
            if (threads <= 128) return launch_early(norm_grad_kernel<X, S, V, 16, 128, 5, false>, blocks, threads, 0, st, 1, p);
            if (threads <= 256) return launch_early(norm_grad_kernel<X, S, V, 16, 256, 3, false>, blocks, threads, 0, st, 1, p);
            if (threads <= 384) return launch_early(norm_grad_kernel<X, S, V, 16, 384, 2, false>, blocks, threads, 0, st, 1, p);
            if (threads <= 512) return launch_early(norm_grad_kernel<X, S, V, 16, 512, 1, false>, blocks, threads, 0, st, 1, p);
            // 80 registers (4096 x 10240 f32 131 us, 9002 bf16 96 us; with the last class's 64: 162 and 131)
            if (threads <= 768) return launch_early(norm_grad_kernel<X, S, V, 16, 768, 1, false>, blocks, threads, 0, st, 1, p);
            return launch_early(norm_grad_kernel<X, S, V, 16, 1024, 1, false>, blocks, threads, 0, st, 1, p);
        };
        if (eights) return by_run(std::integral_constant<int, 8>{});
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
