// Router operators around a choice of experts: token lists per expert, and the balance loss with
// its gradient.  No per-call state outside the caller's buffers, no atomics on floats: results are
// the same bits every run.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moe_internal.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Token lists.  A stable counting sort of the pairs (t, k) by expert: every block owns a contiguous
// range of pairs, every warp of a block a contiguous part of it, so that a pair's place is its
// expert's offset + the expert's pairs in earlier blocks + in earlier warps + earlier in the warp.
// Bound by latency (one launch for up to kListsOne pairs, else two: every block adds up the other
// blocks' counts from L2 itself, which costs less than a third launch).
// ---------------------------------------------------------------------------

constexpr int kListThreads = 1024;
constexpr int kListWarps = kListThreads / 32;
constexpr int kListsOne = 8192;         // pairs that one block sorts alone
constexpr int kListsMin = 2048;         // pairs per block otherwise, at least
constexpr int kListsBlocks = 148;       // blocks, at most
constexpr int kAhead = 4;               // 32-pair loads of a warp in flight

struct ListArgs {
    const int *idx;
    int *counts, *offsets, *rows, *pos;
    int *hist;          // [blocks][E] (more than one block)
    long long pairs, room;
    int K, E, align, chunk, blocks;
};

__device__ __forceinline__ int pair_expert(const ListArgs &p, long long i, long long end) {
    const int e = i < end ? load_in(p.idx + i) : -1;
    return (unsigned)e < (unsigned)p.E ? e : -1;
}

__global__ void __launch_bounds__(kListThreads) lists_count_kernel(const ListArgs p) {
    extern __shared__ int h[];
    for (int e = threadIdx.x; e < p.E; e += kListThreads) h[e] = 0;
    __syncthreads();
    wait_for_stream();
    const long long lo = (long long)blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.pairs);
#pragma unroll 4
    for (long long i = lo + threadIdx.x; i < hi; i += kListThreads) {
        const int e = pair_expert(p, i, hi);
        if (e >= 0) atomicAdd(&h[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kListThreads) p.hist[(size_t)blockIdx.x * p.E + e] = h[e];
}

__global__ void __launch_bounds__(kListThreads, 1) lists_kernel(const ListArgs p) {
    extern __shared__ int sm[];
    int *h = sm;                              // [warps][E] pairs of each warp, then each warp's next place
    int *off = sm + kListWarps * p.E;         // [E + 1]
    int *before = off + p.E + 1;              // [E] this expert's pairs in earlier blocks
    int *total = before + p.E;                // [E]
    __shared__ int s_warp[kListWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool one = p.blocks == 1;
    const int part = max(((p.chunk + kListWarps - 1) / kListWarps + 31) & ~31, 32);   // pairs of a warp
    const int nw = min((p.chunk + part - 1) / part, kListWarps);                      // warps with pairs
    for (int i = tid; i < nw * p.E; i += kListThreads) h[i] = 0;
    for (int e = tid; e < p.E; e += kListThreads) before[e] = total[e] = 0;
    __syncthreads();
    wait_for_stream();
    const long long lo = (long long)blockIdx.x * p.chunk, hi = min(lo + p.chunk, p.pairs);
    const long long wlo = lo + (long long)warp * part, whi = min(wlo + part, hi);
    int *hw = h + warp * p.E;
    // kAhead x 32 pairs' experts at once: the loads are what the warp waits for
    int ex[kAhead];
    auto load = [&](long long i) {
#pragma unroll
        for (int k = 0; k < kAhead; k++) ex[k] = pair_expert(p, i + 32 * k + lane, whi);
    };
    for (long long i = wlo; i < whi; i += 32 * kAhead) {
        load(i);
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int e = ex[k];
            const unsigned same = __match_any_sync(0xffffffffu, e);
            if (e >= 0 && lane == __ffs(same) - 1) hw[e] += __popc(same);
            __syncwarp();
        }
    }
    if (!one && p.E % 4 == 0) {
        // counts of the other blocks: thread = (four experts, part of the blocks)
        const int quads = p.E / 4, groups = kListThreads / quads;
        const int q = tid % quads, g = tid / quads;
        if (g < groups) {
            int4 b4 = make_int4(0, 0, 0, 0), all = b4;
#pragma unroll 8
            for (int b = g; b < p.blocks; b += groups) {
                const int4 v = load_in(reinterpret_cast<const int4 *>(p.hist + (size_t)b * p.E) + q);
                all = make_int4(all.x + v.x, all.y + v.y, all.z + v.z, all.w + v.w);
                if (b < (int)blockIdx.x) b4 = make_int4(b4.x + v.x, b4.y + v.y, b4.z + v.z, b4.w + v.w);
            }
            const int bv[4] = {b4.x, b4.y, b4.z, b4.w}, av[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (bv[k]) atomicAdd(&before[4 * q + k], bv[k]);
                if (av[k]) atomicAdd(&total[4 * q + k], av[k]);
            }
        }
    } else if (!one) {
        const int groups = p.E >= kListThreads ? 1 : kListThreads / p.E;
        for (int i = tid; i < groups * p.E; i += kListThreads) {
            const int e = i % p.E, g = i / p.E;
            int b4 = 0, all = 0;
#pragma unroll 16
            for (int b = g; b < p.blocks; b += groups) {
                const int v = load_in(p.hist + (size_t)b * p.E + e);
                all += v;
                b4 += b < (int)blockIdx.x ? v : 0;
            }
            if (b4) atomicAdd(&before[e], b4);
            if (all) atomicAdd(&total[e], all);
        }
    }
    __syncthreads();
    // thread = expert (E <= threads): the warps' counts become each warp's first place within this
    // block's pairs of the expert; then the running sum of the padded counts over the experts
    int mine = 0, place = 0, n = 0, padded = 0;
    if (tid < p.E) {
        int at = before[tid];
        for (int w0 = 0; w0 < nw; w0 += 8) {
            int c[8];
#pragma unroll
            for (int w = 0; w < 8; w++) c[w] = w0 + w < nw ? h[(w0 + w) * p.E + tid] : 0;
#pragma unroll
            for (int w = 0; w < 8; w++) {
                if (w0 + w < nw) h[(w0 + w) * p.E + tid] = at;
                at += c[w];
            }
        }
        n = one ? at : total[tid];
        if (one) total[tid] = n;
        padded = (n + p.align - 1) / p.align * p.align;
        mine = padded;
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, mine, d);
        if (lane >= d) mine += u;
    }
    if (lane == 31) s_warp[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        int v = s_warp[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        s_warp[lane] = v;
    }
    __syncthreads();
    place = mine - padded + (warp ? s_warp[warp - 1] : 0);
    if (tid < p.E) {
        off[tid] = place;
        if (tid == p.E - 1) off[p.E] = place + padded;
        if (blockIdx.x == 0) {
            p.counts[tid] = n;
            p.offsets[tid] = place;
            if (tid == p.E - 1) p.offsets[p.E] = place + padded;
        }
    }
    __syncthreads();
    const bool kept = whi - wlo <= 32 * kAhead;      // the experts are still in registers
    for (long long i = wlo; i < whi; i += 32 * kAhead) {
        if (!kept) load(i);
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int e = ex[k];
            const long long j = i + 32 * k + lane;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const int leader = __ffs(same) - 1;
            int at = 0;
            if (e >= 0 && lane == leader) {
                at = hw[e];
                hw[e] = at + __popc(same);
            }
            at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1u));
            if (j < whi) {
                if (e >= 0) at += off[e];
                p.pos[j] = e >= 0 ? at : -1;
                if (e >= 0) p.rows[at] = (int)((unsigned)j / (unsigned)p.K);      // below 2^31, as the rows are
            }
            __syncwarp();
        }
    }
    // rows without a token: behind each expert's pairs (its block's warps) and behind the last segment
    for (int e = (int)blockIdx.x * kListWarps + warp; e < p.E; e += p.blocks * kListWarps)
        for (long long r = (long long)off[e] + total[e] + lane; r < off[e + 1]; r += 32) p.rows[r] = -1;      // may step past 2^31
    for (long long r = off[p.E] + (long long)blockIdx.x * kListThreads + tid; r < p.room; r += (long long)p.blocks * kListThreads)
        p.rows[r] = -1;
}

// ---------------------------------------------------------------------------
// Balance loss.  For the segment (sequence) s of n_s unmasked tokens, with p_te the router's
// normalised score (softmax(l), or sigma(l) / (sum_e sigma(l) + 1e-20)) and c_se the number of the
// segment's choices that fell on expert e:
//     L = coef / S  sum_s  E / (K n_s^2)  sum_e c_se sum_t p_te
//     dL / dl_te = coef E / (S K n_s^2) p_te (c_se - sum_j p_tj c_sj)  [x (1 - sigma_te), sigmoid]
// (the counts are constants).  The forward reads the logits once, keeps each block's sums per expert in
// registers and adds the blocks' sums in block order; the gradient needs every count first, so it reads
// the logits again and writes.  A block of tokens b that meets segment s leaves its sums in slot b + s:
// both only grow along the tokens, so slots never meet.  Long batches are bound by the instructions of
// the scores and their latency (131072 x 64 bf16, softmax: forward 15.2 us, gradient 12.9 us; 59 % of the
// issue slots while active, 44 and 47 % over the launches; their bytes alone would take 3 and 5 us), short
// ones by launches and dependent loads.
// ---------------------------------------------------------------------------

constexpr int kBalThreads = 256;
constexpr int kBalWarps = kBalThreads / 32;

struct BalArgs {
    const void *logits;
    long long ld, ldd;
    const int *idx;
    const int *seq;            // [S + 1] or NULL: one segment of all tokens
    const uint8_t *mask;       // [T] or NULL
    const float *grad;         // upstream gradient, or NULL: 1
    float *loss;
    int *counts, *tokens;      // [S, E], [S]
    float *sums;               // [S, E]
    void *dlogits;
    int2 *part;                // [slots][E]: sum (float32 bits) and count of a block's tokens of one segment
    int *part_tokens;          // [slots]
    float *part_loss;          // [S][groups of EB experts]
    float scale;               // coef E / (K S)
    int T, E, K, S, per_block, softmax, zero_rest;
};

template <typename T>
__device__ __forceinline__ float ld1(const T *p);
template <>
__device__ __forceinline__ float ld1<float>(const float *p) { return load_in(p); }
template <>
__device__ __forceinline__ float ld1<__nv_bfloat16>(const __nv_bfloat16 *p) {
    return __uint_as_float((uint32_t)load_in(reinterpret_cast<const unsigned short *>(p)) << 16);
}
template <>
__device__ __forceinline__ float ld1<__half>(const __half *p) { return __half2float(load_in(p)); }
template <typename T>
__device__ __forceinline__ T cast1(float v);
template <>
__device__ __forceinline__ float cast1<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 cast1<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half cast1<__half>(float v) { return __float2half_rn(v); }
// four neighbours
__device__ __forceinline__ void ld4(const float *p, float *v) {
    const float4 f = load_in(reinterpret_cast<const float4 *>(p));
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
}
__device__ __forceinline__ void ld4(const __nv_bfloat16 *p, float *v) {
    const uint2 f = load_in(reinterpret_cast<const uint2 *>(p));
    v[0] = __uint_as_float(f.x << 16);
    v[1] = __uint_as_float(f.x & 0xFFFF0000u);
    v[2] = __uint_as_float(f.y << 16);
    v[3] = __uint_as_float(f.y & 0xFFFF0000u);
}
__device__ __forceinline__ void ld4(const __half *p, float *v) {
    const uint2 f = load_in(reinterpret_cast<const uint2 *>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&f.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&f.y));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}
__device__ __forceinline__ void st4(float *p, const float *v) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
template <typename T>
__device__ __forceinline__ void st4(T *p, const float *v) {
    const T t[4] = {cast1<T>(v[0]), cast1<T>(v[1]), cast1<T>(v[2]), cast1<T>(v[3])};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(t);
}

// How a warp holds tokens: LPT lanes a token (32 / LPT tokens at once), J experts a lane; with VEC
// (E a multiple of 4, rows aligned) quads of neighbouring experts, else every LPT-th expert.
template <typename T_, int J_, int LPT_, bool VEC_>
struct Lay {
    using T = T_;
    static constexpr int J = J_, LPT = LPT_, G = 32 / LPT;
    static constexpr bool VEC = VEC_;
    static constexpr int U = J <= 8 ? 2 : 1;      // tokens in flight for every group of lanes
    __device__ __forceinline__ static int expert(int l, int j) { return VEC ? 4 * (l + LPT * (j / 4)) + j % 4 : l + LPT * j; }
    // a token's logits; -infinity (a score of 0) outside E and, without `on`, everywhere
    __device__ __forceinline__ static void load(const T *row, int E, int l, bool on, float (&x)[J]) {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < J; j += 4) {
                if (on && expert(l, j) < E) ld4(row + expert(l, j), &x[j]);
                else x[j] = x[j + 1] = x[j + 2] = x[j + 3] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int j = 0; j < J; j++) x[j] = on && expert(l, j) < E ? ld1(row + expert(l, j)) : -INFINITY;
        }
    }
    __device__ __forceinline__ static void store(T *row, int E, int l, const float (&x)[J]) {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < J; j += 4)
                if (expert(l, j) < E) st4(row + expert(l, j), &x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < J; j++)
                if (expert(l, j) < E) row[expert(l, j)] = cast1<T>(x[j]);
        }
    }
    __device__ __forceinline__ static float add(float v) {
#pragma unroll
        for (int d = LPT / 2; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    }
    __device__ __forceinline__ static float most(float v) {   // a NaN may be passed over: the sum carries it
#pragma unroll
        for (int d = LPT / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
};
// The segments' offsets, in shared memory where they fit: a chain of dependent loads costs a
// microsecond a step.  Clamped to [0, T].
constexpr int kSegs = 512;
struct Segs {
    const int *g, *sm;
    int T, S;
    // all threads of the block; ends with a barrier
    __device__ __forceinline__ Segs(const BalArgs &p, int *buf) : g(p.seq), sm(p.seq && p.S < kSegs ? buf : nullptr), T(p.T), S(p.S) {
        if (sm)
            for (int i = threadIdx.x; i <= S; i += blockDim.x) buf[i] = min(max(load_in(g + i), 0), T);
        __syncthreads();
    }
    __device__ __forceinline__ int at(int s) const { return sm ? sm[s] : g ? min(max(load_in(g + s), 0), T) : (s ? T : 0); }
    // first segment that ends after token t (S when none does)
    __device__ __forceinline__ int of(int t) const {
        int lo = 0, hi = S;
        while (lo < hi) {
            const int m = (lo + hi) >> 1;
            if (at(m + 1) > t) hi = m;
            else lo = m + 1;
        }
        return lo;
    }
};
// a token's scores (0 where the logit is -infinity) and one over their sum, which normalises them;
// c1: 1 - sigma (sigmoid only)
template <class L>
__device__ __forceinline__ float scores(const float (&x)[L::J], int softmax, float (&pr)[L::J], float (&c1)[L::J]) {
    constexpr int J = L::J;
    float z = 0.0f;
    if (softmax) {
        float m = x[0];
#pragma unroll
        for (int j = 1; j < J; j++) m = fmaxf(m, x[j]);
        m = L::most(m);
        if (m == -INFINITY) m = 0.0f;      // no expert left: every probability 0 (below)
#pragma unroll
        for (int j = 0; j < J; j++) {
            pr[j] = expf(x[j] - m);
            z += pr[j];
        }
        z = L::add(z);
        z = z == 0.0f ? 1.0f : z;
    } else {
#pragma unroll
        for (int j = 0; j < J; j++) {
            const float t = expf(-fabsf(x[j])), r = __fdividef(1.0f, 1.0f + t);
            pr[j] = x[j] >= 0.0f ? r : t * r;      // a NaN stays one
            c1[j] = x[j] >= 0.0f ? t * r : r;
            z += pr[j];
        }
        z = L::add(z) + 1e-20f;
    }
    return 1.0f / z;
}

// Five blocks an SM where the scores leave registers for it (131072 x 64: 15.2 us, unbounded 15.6, six
// 16.0; the gradient spills then: 12.9 us unbounded, 14.4 with five).
template <class L>
__global__ void __launch_bounds__(kBalThreads, L::J <= 8 ? 5 : 1) balance_part_kernel(const BalArgs p) {
    constexpr int J = L::J, U = L::U, G = L::G;
    extern __shared__ float bsm[];
    float *ws = bsm;                                                 // [warps * G][E]
    int *cnt = reinterpret_cast<int *>(bsm + kBalWarps * G * p.E);   // [E]
    __shared__ int s_n, s_seg[kSegs];
    wait_for_stream();
    const Segs seg(p, s_seg);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % L::LPT, g = lane / L::LPT;
    const int t0 = (int)blockIdx.x * p.per_block, t1 = min(t0 + p.per_block, p.T);
    const typename L::T *logits = static_cast<const typename L::T *>(p.logits);
    for (int s = seg.of(t0); s < p.S && seg.at(s) < t1; s++) {
        const int a = max(seg.at(s), t0), b = min(seg.at(s + 1), t1);
        if (a >= b) continue;
        for (int e = tid; e < p.E; e += kBalThreads) cnt[e] = 0;
        if (tid == 0) s_n = 0;
        __syncthreads();
        const int *idx = p.idx + (long long)a * p.K;
        const int n_idx = (b - a) * p.K;                         // at most 128 tokens' choices
        constexpr int UI = 4;                                    // choices in flight
        for (int i = tid; i < n_idx; i += UI * kBalThreads) {
            int e[UI];
#pragma unroll
            for (int u = 0; u < UI; u++) {
                const int k = i + u * kBalThreads;
                e[u] = k < n_idx && (!p.mask || load_in(p.mask + a + k / p.K)) ? load_in(idx + k) : -1;
            }
#pragma unroll
            for (int u = 0; u < UI; u++)
                if ((unsigned)e[u] < (unsigned)p.E) atomicAdd(&cnt[e[u]], 1);
        }
        float sum[J];
#pragma unroll
        for (int j = 0; j < J; j++) sum[j] = 0.0f;
        int n = 0;
        for (int t = a + warp * G; t < b; t += U * kBalWarps * G) {      // the warp's lanes together
            float x[U][J];
            bool on[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int tt = t + u * kBalWarps * G + g;
                on[u] = tt < b && (!p.mask || p.mask[tt]);
                L::load(logits + (long long)tt * p.ld, p.E, l, on[u], x[u]);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                float pr[J], c1[J];
                const float inv = scores<L>(x[u], p.softmax, pr, c1);
#pragma unroll
                for (int j = 0; j < J; j++) sum[j] = fmaf(pr[j], inv, sum[j]);
                n += on[u] ? 1 : 0;
            }
        }
#pragma unroll
        for (int j = 0; j < J; j++)
            if (L::expert(l, j) < p.E) ws[(warp * G + g) * p.E + L::expert(l, j)] = sum[j];
        if (l == 0) atomicAdd(&s_n, n);
        __syncthreads();
        const size_t slot = (size_t)blockIdx.x + s;
        for (int e = tid; e < p.E; e += kBalThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kBalWarps * G; w++) v += ws[w * p.E + e];
            p.part[slot * p.E + e] = make_int2(__float_as_int(v), cnt[e]);
        }
        if (tid == 0) p.part_tokens[slot] = s_n;
        __syncthreads();
    }
}

// One block per (segment, EB experts): the slots' sums in a fixed order (strands of slots, then the
// strands), then the block's part of the loss.  Bound by latency: few loads a thread, all in flight.
constexpr int kSumE = 8;           // the least EB: the most parts of the loss
constexpr int kLossThreads = 1024;
template <int EB, int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) balance_sum_kernel(const BalArgs p) {
    constexpr int STRANDS = THREADS / EB, WARPS = THREADS / 32, LE = EB < 32 ? EB : 32, ROWS = STRANDS * LE / 32;
    static_assert(WARPS <= 32 && (EB < 32 ? ROWS == WARPS && ROWS % (32 / EB) == 0 : EB % 32 == 0), "");
    __shared__ float s_sum[ROWS][EB], s_part[(EB + 31) / 32];
    __shared__ int s_cnt[ROWS][EB], s_tok[WARPS];
    wait_for_stream();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s = (int)blockIdx.x, g = (int)blockIdx.y, G = (int)gridDim.y, e = EB * g + tid % EB;
    const int a = p.seq ? min(max(load_in(p.seq + s), 0), p.T) : 0, b = p.seq ? min(max(load_in(p.seq + s + 1), 0), p.T) : p.T;
    float sum = 0.0f;
    int cnt = 0, tok = 0;
    if (b > a) {
        const int b0 = a / p.per_block, b1 = (b - 1) / p.per_block;
        if (e < p.E) {
#pragma unroll 8
            for (int k = b0 + tid / EB; k <= b1; k += STRANDS) {
                const int2 v = load_in(p.part + ((size_t)k + s) * p.E + e);
                sum += __int_as_float(v.x);
                cnt += v.y;
            }
        }
        for (int k = b0 + tid; k <= b1; k += THREADS) tok += p.part_tokens[(size_t)k + s];
    }
#pragma unroll
    for (int d = LE; d < 32; d *= 2) {
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
        cnt += __shfl_xor_sync(0xffffffffu, cnt, d);
    }
    tok = __reduce_add_sync(0xffffffffu, tok);
    if (lane < LE) {
        s_sum[EB < 32 ? warp : tid / EB][tid % EB] = sum;
        s_cnt[EB < 32 ? warp : tid / EB][tid % EB] = cnt;
    }
    if (lane == 0) s_tok[warp] = tok;
    __syncthreads();
    // the first warps: a lane an expert (EB < 32: of every (32 / EB)-th row, then the lanes' sums)
    constexpr int STEP = 32 / LE;
    if (warp < (EB + 31) / 32) {
        sum = 0.0f;
        cnt = 0;
#pragma unroll
        for (int i = 0; i < ROWS / STEP; i++) {
            sum += s_sum[lane / LE + i * STEP][tid % EB];
            cnt += s_cnt[lane / LE + i * STEP][tid % EB];
        }
#pragma unroll
        for (int d = LE; d < 32; d *= 2) {
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
            cnt += __shfl_xor_sync(0xffffffffu, cnt, d);
        }
        if (lane < LE && e < p.E) {
            p.sums[(size_t)s * p.E + e] = sum;
            p.counts[(size_t)s * p.E + e] = cnt;
        }
        float l = e < p.E ? sum * (float)cnt : 0.0f;
#pragma unroll
        for (int d = LE / 2; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (EB > 32 && lane == 0) s_part[warp] = l;
        sum = l;
    }
    if (EB > 32) __syncthreads();
    if (warp == 0) {
        if (EB > 32) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EB / 32; i++) sum += s_part[i];
        }
        tok = __reduce_add_sync(0xffffffffu, lane < WARPS ? s_tok[lane] : 0);
        if (lane == 0) {
            if (g == 0) p.tokens[s] = tok;
            const float n = (float)max(tok, 1);
            p.part_loss[(size_t)s * G + g] = p.scale / n * (sum / n);
        }
    }
}

// The parts of the loss, in a fixed order.  A launch of its own costs less than a count of the blocks
// that are done, for the last of them to add up (9 sequences of 4099 tokens, 256 experts: 11.1 and
// 11.7 us of the forward; 128 sequences of 32768: 48 and 56 us, every block's count at one address).
__global__ void __launch_bounds__(kLossThreads) balance_loss_kernel(const float *part, int n, float *loss) {
    __shared__ float s_part[32];
    wait_for_stream();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float l = 0.0f;
#pragma unroll 8
    for (int i = tid; i < n; i += kLossThreads) l += load_in(part + i);
#pragma unroll
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) s_part[warp] = l;
    __syncthreads();
    if (warp == 0) {
        l = s_part[lane];
#pragma unroll
        for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0) *loss = l;
    }
}

// Every warp a run of tokens; a segment's counts stay in registers.
template <class L>
__global__ void __launch_bounds__(kBalThreads) balance_grad_kernel(const BalArgs p) {
    constexpr int J = L::J, U = L::U, G = L::G;
    __shared__ int s_seg[kSegs];
    wait_for_stream();
    const Segs seg(p, s_seg);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L::LPT, k = lane / L::LPT;
    const int each = p.per_block / kBalWarps;
    const int ta = ((int)blockIdx.x * kBalWarps + warp) * each, tb = min(ta + each, p.T);
    const typename L::T *logits = static_cast<const typename L::T *>(p.logits);
    typename L::T *out = static_cast<typename L::T *>(p.dlogits);
    const float g = (p.grad ? load_in(p.grad) : 1.0f) * p.scale;
    int done = ta;      // the run's tokens before it are written, or outside every segment and to be kept
    auto zeros = [&](int end) {
        const float z[J] = {};
        for (int t = done + k; p.zero_rest && t < end; t += G) L::store(out + (long long)t * p.ldd, p.E, l, z);
    };
    for (int s = ta < tb ? seg.of(ta) : p.S; s < p.S && seg.at(s) < tb; s++) {
        const int a = max(seg.at(s), ta), b = min(seg.at(s + 1), tb);
        if (a >= b) continue;
        zeros(a);
        done = b;
        const float n = (float)max(load_in(p.tokens + s), 1), up = g / n / n;
        float c[J];
#pragma unroll
        for (int j = 0; j < J; j++) c[j] = L::expert(l, j) < p.E ? (float)load_in(p.counts + (size_t)s * p.E + L::expert(l, j)) * up : 0.0f;
        for (int t = a; t < b; t += U * G) {
            float x[U][J];
            bool on[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int tt = t + u * G + k;
                on[u] = tt < b && (!p.mask || p.mask[tt]);
                L::load(logits + (long long)tt * p.ld, p.E, l, on[u], x[u]);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int tt = t + u * G + k;
                float pr[J], c1[J], dot = 0.0f;
                const float inv = scores<L>(x[u], p.softmax, pr, c1);
                if (!p.softmax) {      // normalised first: sigmoids can all be so small that their sum with c underflows
#pragma unroll
                    for (int j = 0; j < J; j++) pr[j] *= inv;
                }
#pragma unroll
                for (int j = 0; j < J; j++) dot = fmaf(pr[j], c[j], dot);
                dot = L::add(dot);
                if (p.softmax) {
                    dot *= inv;
#pragma unroll
                    for (int j = 0; j < J; j++) x[u][j] = pr[j] * inv * (c[j] - dot);
                } else {
#pragma unroll
                    for (int j = 0; j < J; j++) x[u][j] = pr[j] * (c[j] - dot) * c1[j];
                }
                if (p.mask && !on[u]) {      // zeros whatever the counts are multiplied by: 0 times an infinite gradient is none
#pragma unroll
                    for (int j = 0; j < J; j++) x[u][j] = 0.0f;
                }
                if (tt < b) L::store(out + (long long)tt * p.ldd, p.E, l, x[u]);
            }
        }
    }
    zeros(tb);
}

template <bool VEC, typename F>
cudaError_t by_layout(int dtype, int E, F &&f) {
#define MOE_BAL_E(T)                                         \
    do {                                                     \
        if (E <= 32) return f(Lay<T, 4, 8, VEC>{});          \
        if (E <= 64) return f(Lay<T, 8, 8, VEC>{});          \
        if (E <= 128) return f(Lay<T, 8, 16, VEC>{});        \
        if (E <= 256) return f(Lay<T, 8, 32, VEC>{});        \
        if (E <= 512) return f(Lay<T, 16, 32, VEC>{});       \
        return f(Lay<T, 32, 32, VEC>{});                     \
    } while (0)
    if (dtype == MOE_DTYPE_F32) MOE_BAL_E(float);
    if (dtype == MOE_DTYPE_BF16) MOE_BAL_E(__nv_bfloat16);
    MOE_BAL_E(__half);
#undef MOE_BAL_E
}
// quads: E and the rows' strides multiples of four, the rows on four elements' boundary
bool quads(const void *x, long long ld, int dtype, int E) {
    const int el = dtype == MOE_DTYPE_F32 ? 4 : 2;
    return E % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(x) & (uintptr_t)(4 * el - 1)) == 0;
}

// tokens of a block: enough blocks to cover the card four times, at most 128 tokens each (fewer slots
// for the sums to read; the kernels step up to a block past T in 32 bits: MOE_BALANCE_MAX_TOKENS)
int tokens_per_block(int T) {
    int n = 128;
    while (n > kBalWarps && (T + n - 1) / n < 4 * 152) n /= 2;
    return n;
}
size_t balance_slots(int T, int S) {
    const int per = tokens_per_block(T);
    return (size_t)((T + per - 1) / per) + (size_t)S;
}
size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace

int lists_blocks(long long pairs) {
    if (pairs <= kListsOne) return 1;
    const long long b = (pairs + kListsMin - 1) / kListsMin;
    return (int)(b < kListsBlocks ? b : kListsBlocks);
}

size_t lists_workspace(long long pairs, int E) {
    const int b = lists_blocks(pairs);
    return b == 1 ? 0 : (size_t)b * E * sizeof(int);
}

cudaError_t launch_lists(const int *idx, int T, int K, int E, int align, long long room, int *counts, int *offsets, int *rows,
                         int *pos, void *ws, cudaStream_t st) {
    ListArgs p = {idx, counts, offsets, rows, pos, static_cast<int *>(ws), (long long)T * K, room, K, E, align, 0, 1};
    p.blocks = lists_blocks(p.pairs);
    p.chunk = (int)((p.pairs + p.blocks - 1) / p.blocks);
    if (p.blocks > 1) {
        const cudaError_t e = launch_early(lists_count_kernel, p.blocks, kListThreads, E * sizeof(int), st, 1, p);
        if (e != cudaSuccess) return e;
    }
    auto smem = [](size_t e) { return (kListWarps * e + 3 * e + 1) * sizeof(int); };
    const cudaError_t e = allow_smem<lists_kernel>(smem(1024));
    if (e != cudaSuccess) return e;
    return launch_early(lists_kernel, p.blocks, kListThreads, smem((size_t)E), st, 1, p);
}

size_t balance_workspace(int T, int E, int S) {
    const size_t slots = balance_slots(T, S);
    return up16(slots * E * 8) + up16(slots * 4) + up16((size_t)S * ((E + kSumE - 1) / kSumE) * 4);
}

cudaError_t launch_balance_forward(const void *logits, int dtype, long long ld, int T, int E, const int *idx, int K, int softmax,
                                   float coef, const int *seq, int S, const uint8_t *mask, float *loss, int *counts, float *sums,
                                   int *tokens, void *ws, cudaStream_t st) {
    BalArgs p = {};
    p.logits = logits;
    p.ld = ld;
    p.idx = idx;
    p.seq = seq;
    p.mask = mask;
    p.loss = loss;
    p.counts = counts;
    p.tokens = tokens;
    p.sums = sums;
    p.scale = (float)((double)coef * E / ((double)K * S));
    p.T = T;
    p.E = E;
    p.K = K;
    p.S = S;
    p.softmax = softmax;
    p.per_block = tokens_per_block(T);
    const size_t slots = balance_slots(T, S);
    char *w = static_cast<char *>(ws);
    p.part = reinterpret_cast<int2 *>(w);
    w += up16(slots * E * 8);
    p.part_tokens = reinterpret_cast<int *>(w);
    w += up16(slots * 4);
    p.part_loss = reinterpret_cast<float *>(w);
    auto go = [&](auto lay) {
        using L = decltype(lay);
        const int blocks = T > 0 ? (T + p.per_block - 1) / p.per_block : 1;
        return launch_early(balance_part_kernel<L>, blocks, kBalThreads, ((size_t)kBalWarps * L::G + 1) * E * sizeof(float), st, 1, p);
    };
    const cudaError_t e = quads(logits, ld, dtype, E) ? by_layout<true>(dtype, E, go) : by_layout<false>(dtype, E, go);
    if (e != cudaSuccess) return e;
    auto add_up = [&](auto kernel, int eb, int threads) {
        const int groups = (E + eb - 1) / eb;
        const cudaError_t er = launch_early(kernel, dim3(S, groups), threads, 0, st, 1, p);
        if (er != cudaSuccess) return er;
        return launch_early(balance_loss_kernel, 1, kLossThreads, 0, st, 1, p.part_loss, S * groups, loss);
    };
    // By the slots of a sequence on average (the offsets are on the device): many strands for many of
    // them, else few blocks.  The forward of 32768
    // x 256 scores, 1024 slots, by 8 experts x 128 strands / 32 x 8 / 256 x 1: 1 sequence 17 / 28 / 91 us,
    // 9 18 / 22 / 43, 32 24 / 19 / 28, 128 48 / 21 / 23, 500 133 / 29 / 24, 4000 901 / 87 / 49.
    const size_t each = slots / S;
    if (each >= 48) return add_up(balance_sum_kernel<8, 1024>, 8, 1024);
    if (each >= 5) return add_up(balance_sum_kernel<32, 256>, 32, 256);
    return add_up(balance_sum_kernel<256, 256>, 256, 256);
}

cudaError_t launch_balance_backward(const void *logits, int dtype, long long ld, int T, int E, int K, int softmax, float coef,
                                    const int *counts, const int *tokens, const int *seq, int S, const uint8_t *mask,
                                    const float *grad, void *dlogits, long long ldd, bool zero_rest, cudaStream_t st) {
    BalArgs p = {};
    p.logits = logits;
    p.ld = ld;
    p.ldd = ldd;
    p.seq = seq;
    p.mask = mask;
    p.grad = grad;
    p.counts = const_cast<int *>(counts);
    p.tokens = const_cast<int *>(tokens);
    p.dlogits = dlogits;
    p.scale = (float)((double)coef * E / ((double)K * S));
    p.T = T;
    p.E = E;
    p.K = K;
    p.S = S;
    p.softmax = softmax;
    p.zero_rest = zero_rest && seq;
    p.per_block = tokens_per_block(T);
    auto go = [&](auto lay) {
        return launch_early(balance_grad_kernel<decltype(lay)>, (T + p.per_block - 1) / p.per_block, kBalThreads, 0, st, 1, p);
    };
    return quads(logits, ld, dtype, E) && quads(dlogits, ldd, dtype, E) ? by_layout<true>(dtype, E, go) : by_layout<false>(dtype, E, go);
}

}  // namespace moe
