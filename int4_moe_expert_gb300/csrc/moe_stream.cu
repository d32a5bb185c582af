// The weighted sum of a token's rows behind the experts with its gradient, and the norm and clipping of
// all gradients.  Bound by memory, or by latency for few tokens.  No float atomics: results are the same
// bits every run.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_elem.h"
#include "moe_internal.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Weighted sum of a token's rows: y_t = sum_k w_tk rows[pos_tk] (+ add_t), in float32, in the order of
// k; pairs without a row (pos outside [0, R)) are left out.  A warp a token and 32 runs of its columns,
// four pairs' loads in flight.  Bound by memory: 16384 x 8 rows of 2048 bf16 88 us, at the copy rate.
// ---------------------------------------------------------------------------

constexpr int kCombWarps = 8, kPieceLanes = 31;

struct CombineArgs {
    const void *rows;
    long long ld, ldadd, ldy;
    const int *pos;
    const float *w;          // [T, K] or NULL: 1
    const void *add;
    void *y;
    long long R;
    int T, K, N, parts;      // parts: warps of a token
};

template <typename T, typename Y>
__global__ void __launch_bounds__(32 * kCombWarps) combine_kernel(const CombineArgs p) {
    constexpr int V = 8;
    const int lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kCombWarps + (threadIdx.x >> 5);
    wait_for_stream();
    const long long t = job / p.parts;
    if (t >= p.T) return;
    const int c = ((int)(job - t * p.parts) * 32 + lane) * V;
    int pos = lane < p.K ? load_in(p.pos + t * p.K + lane) : -1;
    const float wt = lane < p.K ? (p.w ? load_in(p.w + t * p.K + lane) : 1.0f) : 0.0f;
    if (pos >= p.R) pos = -1;
    float acc[V] = {};
    constexpr int U = 4;       // pairs in flight
    for (int k0 = 0; k0 < p.K; k0 += U) {
        Vec<T, V> r[U];
        float w[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k = min(k0 + u, 31), at = __shfl_sync(0xffffffffu, pos, k);
            w[u] = __shfl_sync(0xffffffffu, wt, k);
            on[u] = k0 + u < p.K && at >= 0;
            if (on[u] && c < p.N) r[u].load(static_cast<const T *>(p.rows) + at * p.ld + c);
            else r[u].zero();
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (!on[u]) continue;
            float v[V];
            r[u].get(v);
#pragma unroll
            for (int k = 0; k < V; k++) acc[k] = fmaf(w[u], v[k], acc[k]);
        }
    }
    if (c >= p.N) return;
    Vec<Y, V> o;
    if (p.add) {
        float v[V];
        o.load(static_cast<const Y *>(p.add) + t * p.ldadd + c);
        o.get(v);
#pragma unroll
        for (int k = 0; k < V; k++) acc[k] += v[k];
    }
    o.set(acc);
    o.store(static_cast<Y *>(p.y) + t * p.ldy + c);
}

// E elements of a row from column c on, whatever the boundary: the 16-byte pieces that hold them, shifted to their
// place when they are used.  Columns outside [0, N) are anything.  Pieces that are not all of the tensor
// [first, end) are read element by element.
struct Extent {
    uintptr_t first, end;
};
template <typename T, int E, bool ALIGNED = false>
struct Pieces {
    static constexpr int W = E * (int)sizeof(T) / 4, P = W / 4 + (ALIGNED ? 0 : 1);
    uint32_t w[4 * P];
    unsigned s;        // bytes before the first element
    __device__ __forceinline__ void load(const T *row, int c, int N, const Extent x) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row) + (intptr_t)c * (int)sizeof(T);
        s = ALIGNED ? 0u : (unsigned)at & 15u;
        const uintptr_t q = at - s;
        if (q >= x.first && q + 16 * (W / 4 + (s ? 1 : 0)) <= x.end) {
#pragma unroll
            for (int i = 0; i < P; i++) {
                if (i == W / 4 && s == 0) break;
                const uint4 v = load_in(reinterpret_cast<const uint4 *>(q) + i);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else {
            s = 0;
            constexpr int PER = 4 / (int)sizeof(T);
#pragma unroll
            for (int i = 0; i < W; i++) {
                w[i] = 0;
#pragma unroll
                for (int h = 0; h < PER; h++) {
                    const int col = c + PER * i + h;
                    if (col < 0 || col >= N) continue;
                    if constexpr (PER == 2) w[i] |= (unsigned)load_in(reinterpret_cast<const unsigned short *>(row) + col) << (16 * h);
                    else w[i] = load_in(reinterpret_cast<const unsigned *>(row) + col);
                }
            }
        }
    }
    __device__ __forceinline__ void get(float *v) const {
        Vec<T, E> o;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < W; i++) o.w[i] = w[i];
        } else {
            uint32_t b[W + 2];
#pragma unroll
            for (int i = 0; i < W + 2; i++) b[i] = s & 8u ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < W + 1; i++) b[i] = s & 4u ? b[i + 1] : b[i];
#pragma unroll
            for (int i = 0; i < W; i++) o.w[i] = sizeof(T) == 4 ? b[i] : __funnelshift_r(b[i], b[i + 1], 8u * (s & 2u));
        }
        o.get(v);
    }
};
// the columns of v[E] from c on that the row has; c's address on a 16-byte boundary
template <typename T, int E>
__device__ __forceinline__ void store_run(T *row, int c, int N, const float *v) {
    Vec<T, E> o;
    o.set(v);
    if (c >= 0 && c + E <= N) {
        o.store(row + c);
    } else {
#pragma unroll
        for (int i = 0; i < E; i++)
            if (c + i >= 0 && c + i < N) row[c + i] = from_float<T>(v[i]);
    }
}
template <typename T>
__device__ __forceinline__ int off_boundary(const T *p) {      // elements since the last 16-byte boundary
    return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}
template <typename T>
__device__ __forceinline__ Extent extent(const void *x, long long rows, long long ld, int N) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(x);
    return {at, at + (uintptr_t)(((rows - 1) * ld + N) * (long long)sizeof(T))};
}

// Rows that start off 16-byte boundaries or end off a run: the same, in runs that begin on the boundaries of y.  A lane
// loads the 8-byte pieces that begin in its run and takes the words behind from the next lane, so that 31 lanes have a
// run; what is left of the shift is a word and a half.  8192 x 8 rows of 2047 bf16: 66 us (16-byte pieces, whose words
// are three selections from their place, 76; single elements 153).
template <typename T, typename Y>
__global__ void __launch_bounds__(32 * kCombWarps, sizeof(T) > sizeof(Y) ? 4 : 5) combine_pieces_kernel(const CombineArgs p) {
    constexpr int E = sizeof(T) == 4 && sizeof(Y) == 4 ? 4 : 8, W = E * (int)sizeof(T) / 4;
    constexpr int U = 4;       // pairs in flight
    const int lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kCombWarps + (threadIdx.x >> 5);
    wait_for_stream();
    const long long t = job / p.parts;
    if (t >= p.T) return;
    Y *y = static_cast<Y *>(p.y) + t * p.ldy;
    const int c = ((int)(job - t * p.parts) * kPieceLanes + lane) * E - off_boundary(y);
    const int pos = lane < p.K ? load_in(p.pos + t * p.K + lane) : -1;
    const float wt = lane < p.K ? (p.w ? load_in(p.w + t * p.K + lane) : 1.0f) : 0.0f;
    const bool has = pos >= 0 && pos < p.R;
    const unsigned on = __ballot_sync(0xffffffffu, has);
    const unsigned long long row = (unsigned long long)reinterpret_cast<uintptr_t>(static_cast<const T *>(p.rows) + (has ? pos : 0) * p.ld);
    // rows next to the tensor's ends, where pieces may lie partly outside it
    const bool ends = __any_sync(0xffffffffu, has && (pos * p.ld < 64 || (p.R - 1 - pos) * p.ld < 64));
    const Extent x = extent<T>(p.rows, p.R, p.ld, p.N);
    const bool wanted = c - E < p.N;
    const int by = c * (int)sizeof(T);
    float acc[E] = {};
    for (int k0 = 0; k0 < p.K; k0 += U) {
        uint32_t r[U][W];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uintptr_t q = (uintptr_t)(__shfl_sync(0xffffffffu, row, k0 + u) + by) & ~(uintptr_t)7;
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                uint2 v = make_uint2(0, 0);
                if (wanted && on >> (k0 + u) & 1u && (!ends || (q + 4 * i >= x.first && q + 4 * i + 8 <= x.end)))
                    v = load_in(reinterpret_cast<const uint2 *>(q) + i / 2);
                r[u][i] = v.x;
                r[u][i + 1] = v.y;
            }
        }
        if (ends) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                const uintptr_t q = (uintptr_t)(__shfl_sync(0xffffffffu, row, k0 + u) + by) & ~(uintptr_t)7;
                if (!wanted || !(on >> (k0 + u) & 1u)) continue;
#pragma unroll
                for (int i = 0; i < 4 * W; i += (int)sizeof(T)) {
                    const uintptr_t at = q + i, piece = q + (i & ~7);
                    if (at < x.first || at >= x.end || (piece >= x.first && piece + 8 <= x.end)) continue;
                    if constexpr (sizeof(T) == 2) r[u][i / 4] |= (unsigned)load_in(reinterpret_cast<const unsigned short *>(at)) << (8 * (i & 2));
                    else r[u][i / 4] = load_in(reinterpret_cast<const unsigned *>(at));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (!(on >> (k0 + u) & 1u)) continue;
            const float w = __shfl_sync(0xffffffffu, wt, k0 + u);
            const unsigned s = (unsigned)__shfl_sync(0xffffffffu, (unsigned)row, k0 + u) + (unsigned)by;      // the same boundary in all lanes
            const uint32_t next = __shfl_down_sync(0xffffffffu, r[u][0], 1), after = sizeof(T) == 2 ? __shfl_down_sync(0xffffffffu, r[u][1], 1) : 0u;
            uint32_t b[W + 1];
#pragma unroll
            for (int i = 0; i <= W; i++) {
                const uint32_t here = i < W ? r[u][i] : next, behind = i + 1 < W ? r[u][i + 1] : i + 1 == W ? next : after;
                b[i] = s & 4u ? behind : here;
            }
            Vec<T, E> o;
            float v[E];
#pragma unroll
            for (int i = 0; i < W; i++) o.w[i] = sizeof(T) == 4 ? b[i] : __funnelshift_r(b[i], b[i + 1], 8u * (s & 2u));
            o.get(v);
#pragma unroll
            for (int i = 0; i < E; i++) acc[i] = fmaf(w, v[i], acc[i]);
        }
    }
    if (lane >= kPieceLanes || c >= p.N) return;
    if (p.add) {
        Pieces<Y, E> o;
        float v[E];
        o.load(static_cast<const Y *>(p.add) + t * p.ldadd, c, p.N, extent<Y>(p.add, p.T, p.ldadd, p.N));
        o.get(v);
#pragma unroll
        for (int k = 0; k < E; k++) acc[k] += v[k];
    }
    store_run<Y, E>(y, c, p.N, acc);
}

// Gradients: drows[r] = w_tk dy_t for the pair of token t = tokens[r] whose row r is (the sum of the
// weights if the token names r more than once), zeros for rows that no pair of their token names;
// dw_tk = rows[pos_tk] . dy_t.  Blocks of tokens read each row once and write its gradient beside it;
// further blocks look for rows without a pair, 32 a warp, and fill them.  Bound by memory: 16384 x 8 rows of 2048 bf16
// 185 us, 94 % of the copy rate.
struct CombineGradArgs {
    const void *dy, *rows;
    long long lddy, ld, ldd;
    const int *pos, *tokens;
    const float *w;
    void *drows;
    float *dw;
    long long R;
    int T, K, N, token_blocks;
};

constexpr int kCombGradThreads = 128, kCombGradWarps = kCombGradThreads / 32;

// the rows without a pair among the block's: f(row) by whole warps
template <typename F>
__device__ __forceinline__ void empty_rows(const CombineGradArgs &p, F &&f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long r = ((long long)((int)blockIdx.x - p.token_blocks) * kCombGradWarps + warp) * 32 + lane;
    bool empty = r < p.R;
    if (empty) {
        const int t = load_in(p.tokens + r);
        if ((unsigned)t < (unsigned)p.T)
            for (int k = 0; k < p.K && empty; k++) empty = load_in(p.pos + (long long)t * p.K + k) != r;
    }
    unsigned todo = __ballot_sync(0xffffffffu, empty);
    while (todo) {
        f(r - lane + __ffs(todo) - 1);
        todo &= todo - 1;
    }
}

// Token t's pairs by one warp: row (-1: none), whether the pair writes its row's gradient, and with which weight.
struct Pairs {
    int pos[32], write[32];
    float w[32];
};
__device__ __forceinline__ void token_pairs(const CombineGradArgs &p, long long t, int lane, Pairs &s) {
    int pos = lane < p.K ? load_in(p.pos + t * p.K + lane) : -1;
    if (pos >= p.R) pos = -1;
    float w = lane < p.K ? (p.w ? load_in(p.w + t * p.K + lane) : 1.0f) : 0.0f;
    const bool ours = pos >= 0 && load_in(p.tokens + pos) == t;
    // a row that the token names twice: its first pair writes, with the sum of the weights
    const unsigned same = __match_any_sync(0xffffffffu, pos >= 0 ? pos : (int)(0x80000000u | lane));
    if (__ballot_sync(0xffffffffu, (same & (same - 1u)) != 0)) {
        float sum = 0.0f;
        for (int i = 0; i < 32; i++) {
            const float o = __shfl_sync(0xffffffffu, w, i);
            if (same >> i & 1u) sum += o;
        }
        w = sum;
    }
    s.pos[lane] = pos;
    s.write[lane] = ours && lane == __ffs(same) - 1;
    s.w[lane] = w;
}

// Warps hide the loads: the pairs' rows and weights stay in shared memory, since in registers they cost half the
// warps and as much of the speed (8192 x 8 rows of 2048 bf16: 104 us of 89).
template <typename T>
__global__ void __launch_bounds__(kCombGradThreads) combine_grad_kernel(const CombineGradArgs p) {
    constexpr int V = 8;
    constexpr int NW = kCombGradWarps, U = 8;
    __shared__ Pairs s;
    __shared__ float s_part[NW][U];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    wait_for_stream();
    T *drows = static_cast<T *>(p.drows);
    if ((int)blockIdx.x >= p.token_blocks) {
        Vec<T, V> z;
        z.zero();
        empty_rows(p, [&](long long r) {
            for (int c = V * lane; c < p.N; c += 32 * V) z.store(drows + r * p.ldd + c);
        });
        return;
    }
    const long long t = blockIdx.x;
    if (warp == 0) token_pairs(p, t, lane, s);
    __syncthreads();
    const T *dy = static_cast<const T *>(p.dy) + t * p.lddy, *rows = static_cast<const T *>(p.rows);
    for (int k0 = 0; k0 < p.K; k0 += U) {
        float dot[U] = {};
        for (int c = V * tid; c < p.N; c += V * kCombGradThreads) {
            Vec<T, V> g, r[U];
            float d[V];
            g.load(dy + c);
            if (p.dw) {
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int at = k0 + u < p.K ? s.pos[k0 + u] : -1;
                    if (at >= 0) r[u].load(rows + at * p.ld + c);
                    else r[u].zero();
                }
            }
            g.get(d);
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (k0 + u >= p.K || s.pos[k0 + u] < 0) continue;
                float v[V];
                if (p.dw) {
                    r[u].get(v);
#pragma unroll
                    for (int k = 0; k < V; k++) dot[u] = fmaf(v[k], d[k], dot[u]);
                }
                if (p.drows && s.write[k0 + u]) {
                    const float w = s.w[k0 + u];
#pragma unroll
                    for (int k = 0; k < V; k++) v[k] = w * d[k];
                    r[u].set(v);
                    r[u].store(drows + s.pos[k0 + u] * p.ldd + c);
                }
            }
        }
        if (p.dw) {
#pragma unroll
            for (int u = 0; u < U; u++) {
#pragma unroll
                for (int i = 16; i; i >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], i);
                if (lane == 0) s_part[warp][u] = dot[u];
            }
            __syncthreads();
            if (tid < U && k0 + tid < p.K) {
                float sum = s_part[0][tid];
#pragma unroll
                for (int i = 1; i < NW; i++) sum += s_part[i][tid];
                p.dw[t * p.K + k0 + tid] = s.pos[k0 + tid] >= 0 ? sum : 0.0f;
            }
            __syncthreads();
        }
    }
}

// The same for rows off 16-byte boundaries, each on its own: a warp a pair, in runs that begin on the boundaries of the
// gradient's row (of the row where there is no gradient); ALIGNED: the row has the same.  8192 x 8 rows of 2047 bf16:
// 135 us (one element at a time 243; the runs inside the rows on a path of their own, with the shift as a constant, 144).
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kCombGradThreads) combine_grad_pieces_kernel(const CombineGradArgs p) {
    constexpr int E = 16 / (int)sizeof(T), C = 4;      // runs in flight
    __shared__ Pairs s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_for_stream();
    T *drows = static_cast<T *>(p.drows);
    if ((int)blockIdx.x >= p.token_blocks) {
        empty_rows(p, [&](long long r) {
            const float zero[E] = {};
            T *d = drows + r * p.ldd;
            for (int c = E * lane - off_boundary(d); c < p.N; c += 32 * E) store_run<T, E>(d, c, p.N, zero);
        });
        return;
    }
    const long long t = blockIdx.x;
    if (warp == 0) token_pairs(p, t, lane, s);
    __syncthreads();
    const T *dy = static_cast<const T *>(p.dy) + t * p.lddy;
    const Extent in = extent<T>(p.dy, p.T, p.lddy, p.N), of_rows = extent<T>(p.rows, p.R, p.ld, p.N);
    for (int k = warp; k < p.K; k += kCombGradWarps) {
        const long long at = s.pos[k];
        const bool write = drows && at >= 0 && s.write[k];
        float dot = 0.0f;
        if (at >= 0 && (write || p.dw)) {
            const T *row = static_cast<const T *>(p.rows) + at * p.ld;
            T *d = drows + at * p.ldd;
            const float w = s.w[k];
            for (int c0 = E * lane - (drows ? off_boundary(d) : off_boundary(row)); c0 < p.N; c0 += 32 * E * C) {
                Pieces<T, E, ALIGNED> r[C];
                if (p.dw) {
#pragma unroll
                    for (int i = 0; i < C; i++)
                        if (c0 + 32 * E * i < p.N) r[i].load(row, c0 + 32 * E * i, p.N, of_rows);
                }
#pragma unroll
                for (int i = 0; i < C; i++) {
                    const int c = c0 + 32 * E * i;
                    if (c >= p.N) break;
                    Pieces<T, E> g;
                    float x[E], v[E];
                    g.load(dy, c, p.N, in);
                    g.get(x);
                    if (p.dw) {
                        r[i].get(v);
                        const bool inside = c >= 0 && c + E <= p.N;
                        float sum = 0.0f;       // of the run: few roundings on the way
#pragma unroll
                        for (int j = 0; j < E; j++)
                            if (inside || (c + j >= 0 && c + j < p.N)) sum = fmaf(v[j], x[j], sum);
                        dot += sum;
                    }
                    if (write) {
#pragma unroll
                        for (int j = 0; j < E; j++) v[j] = w * x[j];
                        store_run<T, E>(d, c, p.N, v);
                    }
                }
            }
        }
        if (p.dw) {
#pragma unroll
            for (int i = 16; i; i >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, i);
            if (lane == 0) p.dw[t * p.K + k] = dot;
        }
    }
}

// ---------------------------------------------------------------------------
// Norm of all gradients together, and clipping.  The tensors' addresses come as kernel parameters (no
// table to upload, nothing to keep while a captured call lives).  A chunk is a power of two of elements of one
// tensor, 32768 or as many as give every block one; blocks take every gridDim-th chunk.  Squares are added in float32 over a thread's batch, which
// is added to a float64 sum; a batch whose largest magnitude's square would leave float32's normal range
// (2^-50, 2^56) is squared in float64.  Clipping takes the chunks from the last to the first: what the
// norm read last is still in L2.
// Bound by memory: 700 million values (2.35 GB read twice and written once) 1.06 ms, 98 % of the copy
// rate; 1.5 million 11 us, three launches' latency and a float64 sum.
// ---------------------------------------------------------------------------

constexpr int kChunkMost = 15, kChunkLeast = 11;       // log2 of a chunk's elements
constexpr int kClipThreads = 256;
constexpr int kClipFew = 64, kClipMany = 512;      // tensors of a launch: 2 and 18 KB of parameters
constexpr int kSquaresPerSm = 5, kClipPerSm = 4;       // blocks, all resident

struct ClipTensor {
    const void *in;
    void *out;
    long long n;
    int dtype;
};
template <int MOST>
struct ClipTable {
    unsigned first[MOST + 1];       // first chunk of every tensor
    int count, chunk;               // tensors, log2 of a chunk's elements
    ClipTensor tensor[MOST];
};

// The tensor that holds a chunk, by all threads of the block: the parameters' first reads come from far, and a
// search by one thread would wait for several of them one after another.
template <int MOST>
__device__ __forceinline__ int tensor_of(const ClipTable<MOST> &p, unsigned chunk) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < MOST; i += kClipThreads) {
        const int k = i + (int)threadIdx.x;
        n += __syncthreads_count(k < p.count && p.first[k < MOST ? k : 0] <= chunk);
    }
    return n - 1;
}

// 16 bytes that are read once
template <typename T>
__device__ __forceinline__ void load_once(Vec<T, 16 / (int)sizeof(T)> &v, const T *p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "l"(p));
}

// squares of a batch of magnitudes' float32 values
template <int N>
__device__ __forceinline__ double squares(const float (&v)[N]) {
    float s = 0.0f, m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) {
        s = fmaf(v[i], v[i], s);
        m = fmaxf(m, fabsf(v[i]));
    }
    if (m == 0.0f || (m > 8.8817842e-16f && m < 7.2057594e16f)) return (double)s;
    double d = 0.0;
#pragma unroll      // (a loop would index v, and have it in local memory on the usual way too: half the rate)
    for (int i = 0; i < N; i++) d = fma((double)v[i], (double)v[i], d);
    return d;
}

// f(first element, elements) of a chunk by 16-byte runs, or elements where it begins or ends inside one
template <typename T, typename HEAD, typename BODY>
__device__ __forceinline__ void over_chunk(const T *p, int n, HEAD &&one, BODY &&run) {
    constexpr int V = 16 / (int)sizeof(T);
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T)), head = min(n, off ? V - off : 0);
    const int body = (n - head) / V, tail = n - head - body * V;
    if ((int)threadIdx.x < head) one(threadIdx.x);
    if ((int)threadIdx.x >= 32 && (int)threadIdx.x - 32 < tail) one(head + body * V + (int)threadIdx.x - 32);
    run(head, body);
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int n) {
    constexpr int V = 16 / (int)sizeof(T), U = 4;
    double sum = 0.0;
    over_chunk<T>(
        p, n,
        [&](int i) {
            const double v = (double)to_float(load_in(p + i));
            sum += v * v;
        },
        [&](int head, int body) {
            for (int i = threadIdx.x; i < body; i += U * kClipThreads) {
                Vec<T, V> r[U];
                float v[U * V];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (i + u * kClipThreads < body) load_once(r[u], p + head + (long long)(i + u * kClipThreads) * V);
                    else r[u].zero();
                }
#pragma unroll
                for (int u = 0; u < U; u++) r[u].get(&v[u * V]);
                sum += squares(v);
            }
        });
    return sum;
}

// The sum over the block, in thread 0: by one warp, since float64 additions of all warps would queue for an SM's
// two float64 lanes (738 blocks of 2048 elements: 10.0 us with every warp's shuffles, 6.1 so).
__device__ __forceinline__ double sum64(double v) {
    __shared__ double s_sum[kClipThreads];
    s_sum[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = s_sum[threadIdx.x];
#pragma unroll
        for (int i = 32; i < kClipThreads; i += 32) v += s_sum[threadIdx.x + i];
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    }
    return v;
}

template <int MOST>
__global__ void __launch_bounds__(kClipThreads, kSquaresPerSm) grad_squares_kernel(const __grid_constant__ ClipTable<MOST> p, double *part) {
    wait_for_stream();
    double sum = 0.0;
    for (unsigned c = blockIdx.x; c < p.first[p.count]; c += gridDim.x) {
        const int k = tensor_of(p, c);
        const ClipTensor q = p.tensor[k];
        const long long at = (long long)(c - p.first[k]) << p.chunk;
        const int n = (int)min(1ll << p.chunk, q.n - at);
        if (q.dtype == MOE_DTYPE_F32) sum += chunk_squares(static_cast<const float *>(q.in) + at, n);
        else if (q.dtype == MOE_DTYPE_BF16) sum += chunk_squares(static_cast<const __nv_bfloat16 *>(q.in) + at, n);
        else sum += chunk_squares(static_cast<const __half *>(q.in) + at, n);
    }
    sum = sum64(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_kernel(const double *part, int n, float *norm) {
    wait_for_stream();
    double v = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kClipThreads) v += load_in(part + i);
    v = sum64(v);
    if (threadIdx.x == 0) *norm = (float)sqrt(v);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *out, int n, float c) {
    constexpr int V = 16 / (int)sizeof(T), U = 4;
    if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15u) {      // runs of one are no runs of the other
        for (int i = threadIdx.x; i < n; i += kClipThreads) out[i] = from_float<T>(to_float(load_in(p + i)) * c);
        return;
    }
    over_chunk<T>(
        p, n, [&](int i) { out[i] = from_float<T>(to_float(load_in(p + i)) * c); },
        [&](int head, int body) {
            for (int i = threadIdx.x; i < body; i += U * kClipThreads) {
                Vec<T, V> r[U];
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (i + u * kClipThreads < body) load_once(r[u], p + head + (long long)(i + u * kClipThreads) * V);
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (i + u * kClipThreads >= body) continue;
                    float v[V];
                    r[u].get(v);
#pragma unroll
                    for (int k = 0; k < V; k++) v[k] *= c;
                    r[u].set(v);
                    r[u].store(out + head + (long long)(i + u * kClipThreads) * V);
                }
            }
        });
}

template <int MOST>
__global__ void __launch_bounds__(kClipThreads, kClipPerSm) grad_clip_kernel(const __grid_constant__ ClipTable<MOST> p, const float *norm, float most) {
    wait_for_stream();
    const float ratio = most / (load_in(norm) + 1e-6f), c = ratio >= 1.0f ? 1.0f : ratio;      // a NaN stays one
    const unsigned chunks = p.first[p.count];
    for (unsigned i = blockIdx.x; i < chunks; i += gridDim.x) {
        const unsigned ch = chunks - 1 - i;
        const int k = tensor_of(p, ch);
        const ClipTensor q = p.tensor[k];
        if (c == 1.0f && q.in == q.out) continue;      // as they are
        const long long at = (long long)(ch - p.first[k]) << p.chunk;
        const int n = (int)min(1ll << p.chunk, q.n - at);
        if (q.dtype == MOE_DTYPE_F32) chunk_scale(static_cast<const float *>(q.in) + at, static_cast<float *>(q.out) + at, n, c);
        else if (q.dtype == MOE_DTYPE_BF16)
            chunk_scale(static_cast<const __nv_bfloat16 *>(q.in) + at, static_cast<__nv_bfloat16 *>(q.out) + at, n, c);
        else chunk_scale(static_cast<const __half *>(q.in) + at, static_cast<__half *>(q.out) + at, n, c);
    }
}

// f(table, blocks) for tables of up to MOST tensors (2^45 elements in all at most: chunks are 32-bit)
template <int MOST, typename F>
cudaError_t by_tables(int count, const void *const *in, void *const *out, const int32_t *dtype, const int64_t *n, int per_sm, F &&f) {
    ClipTable<MOST> p;
    const unsigned most = (unsigned)sm_count() * per_sm;
    unsigned long long all = 0;
    for (int i = 0; i < count; i++) all += (unsigned long long)n[i];
    p.chunk = kChunkMost;
    while (p.chunk > kChunkLeast && all >> p.chunk < most) p.chunk--;
    for (int i = 0; i < count;) {
        p.count = 0;
        unsigned chunks = 0;
        for (; i < count && p.count < MOST; i++) {
            if (n[i] == 0) continue;
            p.tensor[p.count] = {in[i], out ? out[i] : nullptr, (long long)n[i], dtype[i]};
            p.first[p.count++] = chunks;
            chunks += (unsigned)((n[i] + (1ll << p.chunk) - 1) >> p.chunk);
        }
        if (p.count == 0) break;
        p.first[p.count] = chunks;
        const cudaError_t e = f(p, chunks < most ? chunks : most);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_combine_forward(const void *rows, int dtype, long long ld, long long R, int N, const int *pos, int T, int K, const float *w,
                                   const void *add, long long ldadd, void *y, int y_dtype, long long ldy, cudaStream_t st) {
    CombineArgs p = {rows, ld, ldadd, ldy, pos, w, add, y, R, T, K, N, 1};
    return by_dtype(dtype, [&](auto rt) {
        using X = decltype(rt);
        return by_dtype(y_dtype, [&](auto yt) {
            using Y = decltype(yt);
            auto go = [&](auto kernel, int columns, int each) {       // columns of a warp
                p.parts = (columns + each - 1) / each;
                const long long blocks = ((long long)T * p.parts + kCombWarps - 1) / kCombWarps;
                return launch_early(kernel, (unsigned)blocks, 32 * kCombWarps, 0, st, 1, p);
            };
            if (N % 8 == 0 && runs_of(rows, ld, sizeof(X), 16) && runs_of(y, ldy, sizeof(Y), 16) && (!add || runs_of(add, ldadd, sizeof(Y), 16)))
                return go(combine_kernel<X, Y>, N, 8 * 32);
            return go(combine_pieces_kernel<X, Y>, N + 16 / (int)sizeof(Y) - 1, (sizeof(X) == 4 && sizeof(Y) == 4 ? 4 : 8) * kPieceLanes);
        });
    });
}

cudaError_t launch_combine_backward(const void *dy, int dtype, long long lddy, const void *rows, long long ld, long long R, int N, const int *pos,
                                    int T, int K, const int *tokens, const float *w, void *drows, long long ldd, float *dw, cudaStream_t st) {
    CombineGradArgs p = {dy, rows, lddy, ld, ldd, pos, tokens, w, drows, dw, R, T, K, N, T};
    const long long more = drows ? (R + kCombGradThreads - 1) / kCombGradThreads : 0;
    return by_dtype(dtype, [&](auto t) {
        using X = decltype(t);
        constexpr int el = (int)sizeof(X);
        auto go = [&](auto kernel) { return launch_early(kernel, (unsigned)(T + more), kCombGradThreads, 0, st, 1, p); };
        if (N % 8 == 0 && runs_of(dy, lddy, el, 16) && (!dw || runs_of(rows, ld, el, 16)) && (!drows || runs_of(drows, ldd, el, 16)))
            return go(combine_grad_kernel<X>);
        const bool alike = !drows || !dw || ((reinterpret_cast<uintptr_t>(rows) - reinterpret_cast<uintptr_t>(drows)) % 16 == 0 && (ld - ldd) * el % 16 == 0);
        return alike ? go(combine_grad_pieces_kernel<X, true>) : go(combine_grad_pieces_kernel<X, false>);
    });
}

size_t grad_norm_workspace(int count) {
    const size_t tables = count <= kClipFew ? 1 : ((size_t)count + kClipMany - 1) / kClipMany;
    return tables * sm_count() * kSquaresPerSm * sizeof(double);
}

cudaError_t launch_grad_norm(int count, const void *const *grads, const int32_t *dtype, const int64_t *n, float *norm, void *ws, cudaStream_t st) {
    double *part = static_cast<double *>(ws);
    int parts = 0;
    auto go = [&](auto &table, unsigned blocks) {
        constexpr int MOST = sizeof(table.tensor) / sizeof(ClipTensor);
        const cudaError_t e = launch_early(grad_squares_kernel<MOST>, blocks, kClipThreads, 0, st, 1, table, part + parts);
        parts += (int)blocks;
        return e;
    };
    const cudaError_t e = count <= kClipFew ? by_tables<kClipFew>(count, grads, nullptr, dtype, n, kSquaresPerSm, go)
                                        : by_tables<kClipMany>(count, grads, nullptr, dtype, n, kSquaresPerSm, go);
    if (e != cudaSuccess) return e;
    return launch_early(grad_norm_kernel, 1, kClipThreads, 0, st, 1, part, parts, norm);
}

cudaError_t launch_grad_clip(int count, const void *const *grads, const int32_t *dtype, const int64_t *n, const float *norm, float most,
                             void *const *out, cudaStream_t st) {
    auto go = [&](auto &table, unsigned blocks) {
        constexpr int MOST = sizeof(table.tensor) / sizeof(ClipTensor);
        return launch_early(grad_clip_kernel<MOST>, blocks, kClipThreads, 0, st, 1, table, norm, most);
    };
    return count <= kClipFew ? by_tables<kClipFew>(count, grads, out, dtype, n, kClipPerSm, go) : by_tables<kClipMany>(count, grads, out, dtype, n, kClipPerSm, go);
}

}  // namespace moe
