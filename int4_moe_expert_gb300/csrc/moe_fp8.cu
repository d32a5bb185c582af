// Block-scaled e4m3 products on the 5th-generation tensor cores.
//
// One kernel serves three products (a "column" is a row of the B operand, a "lane" a row of A):
//   matmul  y[r, n]     = sum_kb xs[kb, r] ws[e, n / 128, kb] sum_{k in kb} x[r, k] w[e][n, k]
//           A = the weights (lanes n), B = the activations (columns r), e = the expert whose
//           offsets hold r; without offsets one weight matrix
//   dgrad   the same call with the transposed weights
//   wgrad   dw[e][n, k] = sum_kb dys[kb, n] xs[kb, k] sum_{r in kb} dy[n, r] x[k, r]
//           A = the column-quantised x (lanes k), B = the column-quantised dy (columns n),
//           kb over the 128-row blocks of expert e
// always out[column][lane], so a warp stores 32 neighbouring values of one output row.
//
// The scales are general float32, so a block's product cannot stay in the tensor core's
// accumulator: each 128-element block of the inner axis is one stage (128 bytes a row, exactly
// one 128-byte swizzle atom), its four MMAs (K 32) write a fresh accumulator of a small ring in
// tensor memory, and eight (four for narrow tiles) warps add it, times its scales, to the float32
// sums in their registers.  All sums over blocks are float32 in block order.
//
// Warp roles: epilogue warps (tcgen05.ld, two-wide fused multiply-adds, the stores), one warp of
// tensor copies, one MMA-issuing warp, one warp that multiplies and stages the scales.  mbarrier
// rings connect them; every wait is bounded, and a block that gives up sets the error word, waits
// (bounded) for its copies and MMAs and frees its tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

#include "moe_internal.h"
#include "moe_ptx.h"

// device error word of the handle-less products (moe_fp8_device_error)
static __device__ unsigned g_fp8_err;

namespace moe {
namespace {

constexpr int kKB = 128;                 // inner elements per stage and per scale
constexpr int kARows = 128;              // lanes of a tile
constexpr int kABytes = kARows * kKB;    // A bytes of a stage

struct GemmArgs {
    const float *sa;        // block scales [E][ceil(na / 128)][nkb], or (wgrad) row scales [nkb][na]
    const float *sb;        // column scales [nkb][nb]
    const int *offsets;     // [E + 1] or NULL
    void *out;
    long long ldo;          // elements between columns of out
    long long out_stride;   // elements between experts of out (wgrad)
    int na, nb;             // rows of A (of one expert), rows of B
    int nkb;                // 128-blocks of the inner axis (wgrad: of all experts' rows)
    int E;
    int out_dtype;
    unsigned *err;
};

template <int BT_, int CH_, bool WG_, bool SPLIT_, int STAGES_>
struct Cfg {
    static constexpr int BT = BT_;           // columns of a tile
    static constexpr int CH = CH_;           // column parts, four epilogue warps each
    static constexpr bool WG = WG_;          // wgrad: per-lane A scales, inner range per expert
    static constexpr bool SPLIT = SPLIT_;    // a cluster shares one tile, each block part of the inner axis
    static constexpr int S = STAGES_;
    static constexpr int EW = 4 * CH;        // epilogue warps
    static constexpr int THREADS = 32 * (EW + 4);
    static constexpr int NT = (512 / BT < 4) ? 512 / BT : 4;   // accumulator ring
    static constexpr int TCOLS = NT * BT < 32 ? 32 : NT * BT;
    static constexpr int BBYTES = BT * kKB;
    static constexpr int STAGE = kABytes + BBYTES;
    static constexpr int SS = 4;             // scale ring
    static constexpr int SF = BT + (WG ? kARows : 0);   // floats of a scale slot
    static constexpr int CW = BT / CH;       // columns of an epilogue thread
    static constexpr int LD = CW < 32 || CW > 32 ? 16 : 32;   // columns of one tcgen05.ld
    static constexpr int PER_SM = CH == 1 ? 2 : 1;   // blocks an SM holds
    static constexpr size_t SMEM = (size_t)S * STAGE + 1024;
    static constexpr bool BIGREG = CW > 64;
    static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BT >> 3) << 17) | ((128u >> 4) << 24);
    static_assert(!SPLIT || (size_t)kARows * BT * 4 <= (size_t)S * STAGE, "partial sums reuse the stage ring");
};

constexpr int kMaxExperts = 1024;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// K-major operand with the 128-byte swizzle: groups of 8 rows 1024 bytes apart
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
template <int N>
__device__ __forceinline__ void tc_ld(uint32_t taddr, uint32_t (&r)[N]) {
    static_assert(N == 16 || N == 32, "columns of a load");
    if constexpr (N == 32) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                     "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                       "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                       "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                     : "r"(taddr));
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr));
    }
}
// waits for this warp's tensor-memory loads; names the registers so that no use of them moves above it
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 16) {
        if (i == 0)
            asm volatile("tcgen05.wait::ld.sync.aligned;"
                         : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                           "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                         :: "memory");
        else
            asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                              "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                              "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15]) :: "memory");
    }
}
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    uint32_t x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ void lds_2x64(uint32_t addr, uint64_t &a, uint64_t &b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half to_out<__half>(float v) { return __float2half_rn(v); }
__device__ __forceinline__ void store_out(void *out, long long i, float v, int dtype) {
    if (dtype == MOE_DTYPE_F32) static_cast<float *>(out)[i] = v;
    else if (dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16 *>(out)[i] = to_out<__nv_bfloat16>(v);
    else static_cast<__half *>(out)[i] = to_out<__half>(v);
}
// the first `n` of a thread's column sums, columns ldo elements apart
template <typename T, int N2>
__device__ __forceinline__ void store_columns(void *out, long long i, long long ldo, const uint64_t (&acc)[N2], int n) {
    T *o = static_cast<T *>(out) + i;
#pragma unroll
    for (int k = 0; k < N2; k++) {
        float x, y;
        unpack2(acc[k], x, y);
        if (2 * k < n) *o = to_out<T>(x);
        o += ldo;
        if (2 * k + 1 < n) *o = to_out<T>(y);
        o += ldo;
    }
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float ld_peer(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// One tile of the product: lanes a0.., columns b0..bend, inner blocks [k0, k1) of expert e.
struct Tile {
    int e, a0, b0, bend, k0, k1;
};

// Walks the tiles in order of the expert, the column tile and the lane tile (lane tiles fastest:
// the blocks that run together share their columns, and the weights stay in L2).
template <class C>
struct Walk {
    const GemmArgs &p;
    const int *first;   // shared memory, [E + 1]: column tiles before each expert (matmul with offsets)
    int nat, e;
    __device__ Walk(const GemmArgs &p_, const int *first_) : p(p_), first(first_), nat((p_.na + kARows - 1) / kARows), e(0) {}
    __device__ __forceinline__ int total() const {
        if (C::WG) return p.E * nat * ((p.nb + C::BT - 1) / C::BT);
        return nat * (p.offsets ? first[p.E] : (p.nb + C::BT - 1) / C::BT);
    }
    __device__ __forceinline__ Tile at(int t) {
        Tile r;
        const int j = t / nat;
        r.a0 = (t - j * nat) * kARows;
        if (C::WG) {
            const int nbt = (p.nb + C::BT - 1) / C::BT;
            r.e = j / nbt;
            r.b0 = (j - r.e * nbt) * C::BT;
            r.bend = p.nb;
            if (p.offsets) {
                r.k0 = min(max(p.offsets[r.e], 0) / kKB, p.nkb);
                r.k1 = min(max(p.offsets[r.e + 1] / kKB, r.k0), p.nkb);
            } else {
                r.k0 = 0;
                r.k1 = p.nkb;
            }
        } else {
            r.k0 = 0;
            r.k1 = p.nkb;
            if (p.offsets) {
                while (first[e + 1] <= j) e++;
                const int a = min(max(p.offsets[e], 0), p.nb);
                r.e = e;
                r.b0 = a + (j - first[e]) * C::BT;
                r.bend = min(max(p.offsets[e + 1], a), p.nb);
            } else {
                r.e = 0;
                r.b0 = j * C::BT;
                r.bend = p.nb;
            }
        }
        return r;
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM) fp8_gemm_kernel(const __grid_constant__ CUtensorMap amap,
                                                                 const __grid_constant__ CUtensorMap bmap,
                                                                 const GemmArgs p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long s_full[C::S], s_empty[C::S];
    __shared__ __align__(8) unsigned long long s_tfull[C::NT], s_tempty[C::NT];
    __shared__ __align__(8) unsigned long long s_sfull[C::SS], s_sempty[C::SS];
    __shared__ __align__(8) unsigned long long s_drain;
    __shared__ __align__(16) float s_scale[C::SS][C::SF];
    __shared__ int s_first[C::WG ? 1 : kMaxExperts + 1];
    __shared__ uint32_t s_taddr;
    __shared__ int s_fail, s_issued;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;

    if (tid == 0) {
        s_fail = 0;
        s_issued = 0;
        for (int i = 0; i < C::S; i++) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&s_empty[i]), 1);
        }
        for (int i = 0; i < C::NT; i++) {
            mbar_init(smem_u32(&s_tfull[i]), 1);
            mbar_init(smem_u32(&s_tempty[i]), C::EW);
        }
        for (int i = 0; i < C::SS; i++) {
            mbar_init(smem_u32(&s_sfull[i]), 32);
            mbar_init(smem_u32(&s_sempty[i]), C::EW);
        }
        mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::EW + 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_taddr)), "n"(C::TCOLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (!C::WG && p.offsets) {
        // column tiles of every expert; the running sum by one warp
        for (int e = tid; e < p.E; e += C::THREADS) {
            const int a = min(max(p.offsets[e], 0), p.nb), b = min(max(p.offsets[e + 1], a), p.nb);
            s_first[e + 1] = (b - a + C::BT - 1) / C::BT;
        }
        __syncthreads();
        if (warp == 0) {
            int run = 0;
            for (int e0 = 0; e0 < p.E; e0 += 32) {
                int v = e0 + lane < p.E ? s_first[e0 + lane + 1] : 0;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int u = __shfl_up_sync(0xffffffffu, v, d);
                    if (lane >= d) v += u;
                }
                if (e0 + lane < p.E) s_first[e0 + lane + 1] = run + v;
                run += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0) s_first[0] = 0;
        }
    }
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t taddr = s_taddr;
    volatile int *fail = &s_fail;

    const uint32_t crank = C::SPLIT ? cluster_rank() : 0u, csize = C::SPLIT ? cluster_size() : 1u;
    const int t0 = C::SPLIT ? (int)(blockIdx.x / csize) : (int)blockIdx.x;
    Walk<C> walk(p, s_first);
    const int total = walk.total();
    const int tstep = C::SPLIT ? (1 << 30) : (int)gridDim.x;
    // this block's share of a tile's inner blocks
    auto part = [&](Tile &t) {
        if (C::SPLIT) {
            const int n = t.k1 - t.k0;
            const int lo = t.k0 + (int)((long long)n * crank / csize), hi = t.k0 + (int)((long long)n * (crank + 1) / csize);
            t.k0 = lo;
            t.k1 = hi;
        }
    };

    if (warp < C::EW) {
        // 384 threads x 168 registers at launch = 256 x 216 + 128 x 72
        if constexpr (C::BIGREG) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // epilogue: lane quarter warp % 4, columns of part warp / 4
        const int q4 = warp & 3, part_c = (warp >> 2) * C::CW;
        const uint32_t trow = taddr + ((uint32_t)(32 * q4) << 16) + (uint32_t)part_c;
        int it = 0;
        bool ok = true;
        for (int t = t0; t < total && ok; t += tstep) {
            Tile ti = walk.at(t);
            part(ti);
            uint64_t acc[C::CW / 2];
#pragma unroll
            for (int i = 0; i < C::CW / 2; i++) acc[i] = 0ull;
            for (int kb = ti.k0; kb < ti.k1; kb++, it++) {
                const int q = it % C::NT, s = it % C::SS;
                const bool w = !*fail && mbar_wait(smem_u32(&s_sfull[s]), (uint32_t)(it / C::SS) & 1u) &&
                               mbar_wait(smem_u32(&s_tfull[q]), (uint32_t)(it / C::NT) & 1u);
                if (!__all_sync(0xffffffffu, w)) {
                    *fail = 1;
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sc = smem_u32(&s_scale[s][part_c]);
                uint64_t la = 0;
                if (C::WG) {
                    const uint32_t f = __float_as_uint(s_scale[s][C::BT + 32 * q4 + lane]);
                    la = pack2(f, f);
                }
                constexpr int NL = C::CW / C::LD;
                uint32_t r[2][C::LD];
                tc_ld<C::LD>(trow + (uint32_t)(q * C::BT), r[0]);
#pragma unroll
                for (int l = 0; l < NL; l++) {
                    tc_wait_ld(r[l & 1]);
                    if (l + 1 < NL) tc_ld<C::LD>(trow + (uint32_t)(q * C::BT + (l + 1) * C::LD), r[(l + 1) & 1]);
                    if (l + 1 == NL) {
                        // the accumulator is in registers: the slot may be written again
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        if (lane == 0) mbar_arrive(smem_u32(&s_tempty[q]));
                    }
#pragma unroll
                    for (int i = 0; i < C::LD; i += 4) {
                        uint64_t s0, s1;
                        lds_2x64(sc + (uint32_t)(l * C::LD + i) * 4u, s0, s1);
                        if (C::WG) {
                            s0 = mul2(s0, la);
                            s1 = mul2(s1, la);
                        }
                        const int o = (l * C::LD + i) / 2;
                        acc[o] = fma2(pack2(r[l & 1][i], r[l & 1][i + 1]), s0, acc[o]);
                        acc[o + 1] = fma2(pack2(r[l & 1][i + 2], r[l & 1][i + 3]), s1, acc[o + 1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s_sempty[s]));
            }
            if (!ok) break;
            const int n = ti.a0 + 32 * q4 + lane;
            if (C::SPLIT) {
                // partial sums [column][lane] over the stage ring: every copy into it was consumed
                float *ps = reinterpret_cast<float *>(smem_raw + (ring - smem_u32(smem_raw)));
#pragma unroll
                for (int i = 0; i < C::CW / 2; i++) {
                    float x, y;
                    unpack2(acc[i], x, y);
                    ps[(part_c + 2 * i) * kARows + 32 * q4 + lane] = x;
                    ps[(part_c + 2 * i + 1) * kARows + 32 * q4 + lane] = y;
                }
            } else if (n < p.na) {
                const int c = ti.b0 + part_c, cols = ti.bend - c;
                const long long at = (C::WG ? (long long)ti.e * p.out_stride : 0ll) + (long long)c * p.ldo + n;
                if (p.out_dtype == MOE_DTYPE_F32) store_columns<float>(p.out, at, p.ldo, acc, cols);
                else if (p.out_dtype == MOE_DTYPE_BF16) store_columns<__nv_bfloat16>(p.out, at, p.ldo, acc, cols);
                else store_columns<__half>(p.out, at, p.ldo, acc, cols);
            }
        }
    } else {
        if constexpr (C::BIGREG) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == C::EW) {
            // tensor copies
            if (lane == 0) {
                int it = 0;
                for (int t = t0; t < total; t += tstep) {
                    Tile ti = walk.at(t);
                    part(ti);
                    bool ok = true;
                    for (int kb = ti.k0; kb < ti.k1; kb++, it++) {
                        const int j = it % C::S;
                        if (*fail || (it >= C::S && !mbar_wait(smem_u32(&s_empty[j]), (uint32_t)(it / C::S + 1) & 1u))) {
                            *fail = 1;
                            ok = false;
                            break;
                        }
                        const uint32_t bar = smem_u32(&s_full[j]), dst = ring + (uint32_t)(j * C::STAGE);
                        mbar_expect_tx(bar, C::STAGE);
                        tma_load_3d(dst, &amap, kb * kKB, ti.a0, C::WG ? 0 : ti.e, bar);
                        tma_load_2d(dst + kABytes, &bmap, kb * kKB, ti.b0, bar);
                        s_issued = it + 1;
                    }
                    if (!ok) break;
                }
            }
        } else if (warp == C::EW + 1) {
            // MMA issue: one fresh accumulator of the ring per stage
            if (lane == 0) {
                int it = 0;
                bool ok = true;
                const uint64_t ad0 = sw128_desc(ring), bd0 = sw128_desc(ring + kABytes);
                for (int t = t0; t < total && ok; t += tstep) {
                    Tile ti = walk.at(t);
                    part(ti);
                    for (int kb = ti.k0; kb < ti.k1; kb++, it++) {
                        const int j = it % C::S, q = it % C::NT;
                        if (*fail || (it >= C::NT && !mbar_wait(smem_u32(&s_tempty[q]), (uint32_t)(it / C::NT + 1) & 1u)) ||
                            !mbar_wait(smem_u32(&s_full[j]), (uint32_t)(it / C::S) & 1u)) {
                            *fail = 1;
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint64_t off = (uint64_t)((j * C::STAGE) >> 4);
                        const uint32_t d = taddr + (uint32_t)(q * C::BT);
    #pragma unroll
                        for (int ks = 0; ks < 4; ks++)
                            mma_f8(d, ad0 + off + 2 * ks, bd0 + off + 2 * ks, C::IDESC, ks > 0);
                        tc_commit(smem_u32(&s_empty[j]));
                        tc_commit(smem_u32(&s_tfull[q]));
                    }
                }
                if (it > 0 || !ok) {
                    tc_commit(smem_u32(&s_drain));
                    if (!mbar_wait(smem_u32(&s_drain), 0u)) *fail = 1;
                }
            }
        } else if (warp == C::EW + 2) {
            // scales: column scales (times the weight block's scale) of every stage, four stages' loads at once
            int it = 0;
            bool ok = true;
            constexpr int PB = (C::BT + 31) / 32, U = PB > 4 ? 2 : 4;
            for (int t = t0; t < total && ok; t += tstep) {
                Tile ti = walk.at(t);
                part(ti);
                const float *sa = C::WG ? p.sa : p.sa + ((size_t)ti.e * ((p.na + kARows - 1) / kARows) + ti.a0 / kARows) * p.nkb;
                for (int kb0 = ti.k0; kb0 < ti.k1 && ok; kb0 += U) {
                    float v[U][PB], a[U][C::WG ? 4 : 1];
    #pragma unroll
                    for (int u = 0; u < U; u++) {
                        const bool in = kb0 + u < ti.k1;
                        const float *sb = p.sb + (size_t)(kb0 + u) * p.nb;
    #pragma unroll
                        for (int i = 0; i < PB; i++) {
                            const int c = 32 * i + lane;
                            v[u][i] = in && (C::BT >= 32 || c < C::BT) && ti.b0 + c < ti.bend ? __ldg(sb + ti.b0 + c) : 0.0f;
                        }
                        if (C::WG) {
    #pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const int c = ti.a0 + 32 * i + lane;
                                a[u][i] = in && c < p.na ? __ldg(p.sa + (size_t)(kb0 + u) * p.na + c) : 0.0f;
                            }
                        } else {
                            a[u][0] = in ? __ldg(sa + kb0 + u) : 0.0f;
                        }
                    }
    #pragma unroll
                    for (int u = 0; u < U; u++) {
                        if (kb0 + u >= ti.k1) break;
                        const int q = it % C::SS;
                        const bool w = it < C::SS || mbar_wait(smem_u32(&s_sempty[q]), (uint32_t)(it / C::SS + 1) & 1u);
                        if (!__all_sync(0xffffffffu, w && !*fail)) {
                            *fail = 1;
                            ok = false;
                            break;
                        }
    #pragma unroll
                        for (int i = 0; i < PB; i++)
                            if (C::BT >= 32 || lane < C::BT) s_scale[q][32 * i + lane] = C::WG ? v[u][i] : v[u][i] * a[u][0];
                        if (C::WG) {
    #pragma unroll
                            for (int i = 0; i < 4; i++) s_scale[q][C::BT + 32 * i + lane] = a[u][i];
                        }
                        mbar_arrive(smem_u32(&s_sfull[q]));
                        it++;
                    }
                }
            }
        }
    }
    __syncthreads();
    if (s_fail && tid == 0) {
        // after a wait that ran out: copies still in flight land before the shared memory is released
        // (bounded; the MMA thread waited for its own MMAs)
        for (int i = max(0, s_issued - C::S); i < s_issued; i++)
            mbar_wait(smem_u32(&s_full[i % C::S]), (uint32_t)(i / C::S) & 1u);
        atomicOr(p.err, MOE_DEVICE_ERR_TC);
    }
    if (C::SPLIT) {
        // sums of all blocks of the cluster, in block order: block r adds columns r, r + csize, ...
        cluster_sync_all();
        if (t0 < total) {
            const Tile ti = walk.at(t0);
            for (int c = (int)crank + (int)csize * (tid >> 7); c < C::BT; c += (int)csize * (C::THREADS >> 7)) {
                const int l = tid & 127, n = ti.a0 + l;
                float v = 0.0f;
                for (uint32_t r = 0; r < csize; r++) v += ld_peer(ring + (uint32_t)(c * kARows + l) * 4u, r);
                if (n < p.na && ti.b0 + c < ti.bend) store_out(p.out, (long long)(ti.b0 + c) * p.ldo + n, v, p.out_dtype);
            }
        }
        cluster_sync_all();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == C::EW + 3) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(C::TCOLS) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Quantisers.  A block's scale is a power of two, so that x / s is exact and the only rounding is
// the one to e4m3 (nearest, ties to even): every orientation and every implementation agrees bit
// for bit.  Memory-bound: each element is read once and its codes are written once.
// ---------------------------------------------------------------------------

constexpr int kQThreads = 256;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half *p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ unsigned max_bits(float4 v) {
    return max(max(abs_bits(v.x), abs_bits(v.y)), max(abs_bits(v.z), abs_bits(v.w)));
}
// The least power of two s >= 2^-126 with largest / s <= 448 = 1.75 x 2^8 (1 for a block of zeros,
// NaN for one with a NaN or an infinity) and 1 / s, from the largest magnitude's bits.
__device__ __forceinline__ float block_scale(unsigned largest, float &inv) {
    if (largest >= 0x7F800000u) {
        inv = __uint_as_float(0x7FC00000u);
        return inv;
    }
    if (largest == 0) {
        inv = 1.0f;
        return 1.0f;
    }
    const int j = max((int)(largest >> 23) - 127 - 8 + ((largest & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
    inv = __uint_as_float((unsigned)(127 - j) << 23);
    return __uint_as_float((unsigned)(127 + j) << 23);
}
__device__ __forceinline__ uint32_t codes2(float a, float b) {   // a in the low byte
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t codes4(float4 v, float inv) {
    return codes2(v.x * inv, v.y * inv) | (codes2(v.z * inv, v.w * inv) << 16);
}
__device__ __forceinline__ int src_row(const int *rows, int r, int R, int n_src) {
    if (r >= R) return -1;
    if (!rows) return r;
    const int s = __ldg(rows + r);
    return (s >= 0 && s < n_src) ? s : -1;
}

struct QuantArgs {
    const void *x;
    long long ld;        // elements between rows of x
    const int *rows;     // [R] source rows, negative: zeros; or NULL
    uint8_t *codes;      // [R, width]
    float *scales;       // [blocks(width), R]
    uint8_t *codes_t;    // [width, 128 blocks(R)] or NULL
    float *scales_t;     // [blocks(R), width]
    int n_src, R, width;
};

// Rows only: a warp per 1 x 128 block (four elements a lane), KG blocks of RW rows each.
template <typename T, int RW, int KG>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const QuantArgs p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = (int)blockIdx.x * (kQThreads / 32 * RW) + warp, kb0 = (int)blockIdx.y * KG;
    const T *x = static_cast<const T *>(p.x);
    float4 v[RW][KG];
#pragma unroll
    for (int i = 0; i < RW; i++) {
        const int r = r0 + i * (kQThreads / 32), s = src_row(p.rows, r, p.R, p.n_src);
#pragma unroll
        for (int g = 0; g < KG; g++) {
            const int c = (kb0 + g) * kKB + 4 * lane;
            v[i][g] = s >= 0 && c < p.width ? load4(x + (long long)s * p.ld + c) : make_float4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < RW; i++) {
        const int r = r0 + i * (kQThreads / 32);
#pragma unroll
        for (int g = 0; g < KG; g++) {
            const int kb = kb0 + g, c = kb * kKB + 4 * lane;
            float inv;
            const float s = block_scale(__reduce_max_sync(0xffffffffu, max_bits(v[i][g])), inv);
            if (r < p.R && c < p.width) {
                *reinterpret_cast<uint32_t *>(p.codes + (size_t)r * p.width + c) = codes4(v[i][g], inv);
                if (lane == 0) p.scales[(size_t)kb * p.R + r] = s;
            }
        }
    }
}

// element (r, c) of a 128 x 128 tile in shared memory: 16-byte chunks of a row permuted by the
// row's group of 16, so that rows are written and columns read without bank conflicts
__device__ __forceinline__ int tile_at(int r, int c) { return r * kKB + (c ^ ((r >> 4) << 2)); }

// Rows and columns of a 128 x 128 tile, or (WT) one scale for the whole tile of a weight matrix:
// x is read once, the transposed codes leave shared memory 16 rows a lane.
template <typename T, bool WT>
__global__ void __launch_bounds__(kQThreads) quantize_tile_kernel(const QuantArgs p) {
    extern __shared__ __align__(16) float tile[];
    __shared__ unsigned s_max[kQThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = (int)blockIdx.y * kKB, kb = (int)blockIdx.x, e = (int)blockIdx.z;
    const int c = kb * kKB + 4 * lane;
    const T *x = static_cast<const T *>(p.x) + (WT ? (size_t)e * p.R * p.ld : 0);
    uint8_t *codes = p.codes + (WT ? (size_t)e * p.R * p.width : 0);
    const int ldt = WT ? p.R : ((p.R + kKB - 1) / kKB) * kKB;   // bytes between rows of codes_t
    uint8_t *codes_t = p.codes_t + (WT ? (size_t)e * p.R * p.width : 0);
    const int nrb = (p.R + kKB - 1) / kKB, nkb = (p.width + kKB - 1) / kKB;
    float wscale = 0.0f, winv = 0.0f;
    constexpr int U = 8;
    unsigned most = 0;
    for (int i0 = warp; i0 < kKB; i0 += U * (kQThreads / 32)) {
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * (kQThreads / 32), s = src_row(p.rows, r0 + i, p.R, p.n_src);
            v[u] = s >= 0 && c < p.width ? load4(x + (long long)s * p.ld + c) : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * (kQThreads / 32), r = r0 + i;
            *reinterpret_cast<float4 *>(&tile[tile_at(i, 4 * lane)]) = v[u];
            const unsigned m = max_bits(v[u]);
            if (WT) {
                most = max(most, m);
            } else {
                float inv;
                const float s = block_scale(__reduce_max_sync(0xffffffffu, m), inv);
                if (r < p.R && c < p.width) {
                    *reinterpret_cast<uint32_t *>(codes + (size_t)r * p.width + c) = codes4(v[u], inv);
                    if (lane == 0) p.scales[(size_t)kb * p.R + r] = s;
                }
            }
        }
    }
    if (WT) {
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) s_max[warp] = most;
    }
    __syncthreads();
    if (WT) {
        for (int i = 0; i < kQThreads / 32; i++) most = max(most, s_max[i]);
        wscale = block_scale(most, winv);
        if (threadIdx.x == 0) {
            p.scales[((size_t)e * nrb + blockIdx.y) * nkb + kb] = wscale;
            if (p.codes_t) p.scales_t[((size_t)e * nkb + kb) * nrb + blockIdx.y] = wscale;
        }
        for (int i = warp; i < kKB; i += kQThreads / 32)
            if (r0 + i < p.R && c < p.width)
                *reinterpret_cast<uint32_t *>(codes + (size_t)(r0 + i) * p.width + c) =
                    codes4(*reinterpret_cast<const float4 *>(&tile[tile_at(i, 4 * lane)]), winv);
        if (!p.codes_t) return;
    }
    // columns: lane = 16-row chunk (lane & 7) of column 4 j + (lane >> 3)
    const int ch = lane & 7;
    for (int j = warp; j < kKB / 4; j += kQThreads / 32) {
        const int cc = 4 * j + (lane >> 3), col = kb * kKB + cc;
        float v[16];
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            v[i] = tile[tile_at(16 * ch + i, cc)];
            m = max(m, abs_bits(v[i]));
        }
        float s = wscale, inv = winv;
        if (!WT) {
#pragma unroll
            for (int d = 1; d < 8; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
            s = block_scale(m, inv);
        }
        if (col >= p.width) continue;
        if (!WT && ch == 0) p.scales_t[(size_t)blockIdx.y * p.width + col] = s;
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; i++) q[i] = codes4(make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]), inv);
        uint8_t *o = codes_t + (size_t)col * ldt + r0 + 16 * ch;
        if (!WT || (p.R % 16 == 0 && r0 + 16 * ch < p.R)) {
            *reinterpret_cast<uint4 *>(o) = make_uint4(q[0], q[1], q[2], q[3]);
        } else if constexpr (WT) {
            for (int i = 0; i < 16; i++)
                if (r0 + 16 * ch + i < p.R) o[i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
        }
    }
}

int sm_count() {
    static int n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    if (!n[dev]) cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev);
    return n[dev] > 0 ? n[dev] : 152;
}

}  // namespace

cudaError_t launch_quantize(const void *x, int dtype, long long ld, int n_src, int width, const int *rows, int R,
                            uint8_t *codes, float *scales, uint8_t *codes_t, float *scales_t, cudaStream_t st) {
    const QuantArgs p = {x, ld, rows, codes, scales, codes_t, scales_t, n_src, R, width};
    const int nkb = (width + kKB - 1) / kKB;
    if (codes_t) {
        const dim3 grid(nkb, (R + kKB - 1) / kKB);
        constexpr int smem = kKB * kKB * 4;
        auto go = [&](auto kernel) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess) {
                kernel<<<grid, kQThreads, smem, st>>>(p);
                e = cudaGetLastError();
            }
            return e;
        };
        if (dtype == MOE_DTYPE_F32) return go(quantize_tile_kernel<float, false>);
        if (dtype == MOE_DTYPE_BF16) return go(quantize_tile_kernel<__nv_bfloat16, false>);
        return go(quantize_tile_kernel<__half, false>);
    }
    // few rows: one block a warp, so that the blocks cover the card; many: four rows of four blocks
    const bool few = (long long)R * nkb < 16ll * 8 * 4 * sm_count();
    const int rw = few ? 1 : 4, kg = few ? 1 : 4;
    const dim3 grid((R + 8 * rw - 1) / (8 * rw), (nkb + kg - 1) / kg);
    if (dtype == MOE_DTYPE_F32) {
        if (few) quantize_rows_kernel<float, 1, 1><<<grid, kQThreads, 0, st>>>(p);
        else quantize_rows_kernel<float, 4, 4><<<grid, kQThreads, 0, st>>>(p);
    } else if (dtype == MOE_DTYPE_BF16) {
        if (few) quantize_rows_kernel<__nv_bfloat16, 1, 1><<<grid, kQThreads, 0, st>>>(p);
        else quantize_rows_kernel<__nv_bfloat16, 4, 4><<<grid, kQThreads, 0, st>>>(p);
    } else {
        if (few) quantize_rows_kernel<__half, 1, 1><<<grid, kQThreads, 0, st>>>(p);
        else quantize_rows_kernel<__half, 4, 4><<<grid, kQThreads, 0, st>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_quantize_weights(const void *w, int dtype, int E, int N, int K, uint8_t *codes, float *scales,
                                    uint8_t *codes_t, float *scales_t, cudaStream_t st) {
    const QuantArgs p = {w, K, nullptr, codes, scales, codes_t, scales_t, N, N, K};
    const dim3 grid((K + kKB - 1) / kKB, (N + kKB - 1) / kKB, E);
    constexpr int smem = kKB * kKB * 4;
    auto go = [&](auto kernel) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) {
            kernel<<<grid, kQThreads, smem, st>>>(p);
            e = cudaGetLastError();
        }
        return e;
    };
    if (dtype == MOE_DTYPE_F32) return go(quantize_tile_kernel<float, true>);
    if (dtype == MOE_DTYPE_BF16) return go(quantize_tile_kernel<__nv_bfloat16, true>);
    return go(quantize_tile_kernel<__half, true>);
}

// ---------------------------------------------------------------------------
// Product launches
// ---------------------------------------------------------------------------

namespace {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 f = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    return f;
}

// codes [n2][rows][cols] as boxes of 128 bytes x box_rows, 128-byte swizzle; outside: zeros
bool tmap(CUtensorMap *m, int rank, const void *base, uint64_t cols, uint64_t rows, uint64_t n2, int box_rows) {
    const cuuint64_t dims[3] = {cols, rows, n2};
    const cuuint64_t strides[2] = {cols, cols * rows};
    const cuuint32_t box[3] = {(cuuint32_t)kKB, (cuuint32_t)box_rows, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    std::memset(m, 0, sizeof(*m));
    return tmap_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void *>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t error_word(unsigned **err) {
    static unsigned *word[64] = {};
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!word[dev]) {
        void *ptr = nullptr;
        e = cudaGetSymbolAddress(&ptr, g_fp8_err);
        if (e != cudaSuccess) return e;
        word[dev] = static_cast<unsigned *>(ptr);
    }
    *err = word[dev];
    return cudaSuccess;
}

// grid: blocks (of clusters of `cluster`); the B map's box is the tile's columns
template <class C>
cudaError_t launch_gemm(const GemmArgs &p, const CUtensorMap &am, const uint8_t *b, uint64_t b_cols, uint64_t b_rows,
                        long long tiles, int per_sm, int cluster, cudaStream_t st) {
    CUtensorMap bm;
    if (!tmap(&bm, 2, b, b_cols, b_rows, 1, C::BT)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(fp8_gemm_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const long long most = (long long)sm_count() * per_sm;
    cfg.gridDim = dim3((unsigned)(C::SPLIT ? tiles * cluster : (tiles < most ? tiles : most)));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    if (C::SPLIT) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)cluster;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<C>, am, bm, p);
}

}  // namespace

cudaError_t launch_fp8_matmul(const uint8_t *x, const float *xs, int R, const uint8_t *w, const float *ws, int E, int N, int K,
                              const int *offsets, void *y, int y_dtype, long long ldy, cudaStream_t st) {
    if (!tmap_encoder()) return cudaErrorNotSupported;
    GemmArgs p = {};
    p.sa = ws;
    p.sb = xs;
    p.offsets = offsets;
    p.out = y;
    p.ldo = ldy;
    p.na = N;
    p.nb = R;
    p.nkb = (K + kKB - 1) / kKB;
    p.E = E;
    p.out_dtype = y_dtype;
    cudaError_t e = error_word(&p.err);
    if (e != cudaSuccess) return e;
    CUtensorMap am;
    if (!tmap(&am, 3, w, K, N, E, kARows)) return cudaErrorInvalidValue;
    const long long nat = (N + kARows - 1) / kARows;
    const int used = offsets ? (E < R ? E : R) : 1;      // weight matrices that rows can belong to
    const int each = (R + used - 1) / used;
    auto tiles = [&](int bt) { return nat * (offsets ? (long long)R / bt + used : ((long long)R + bt - 1) / bt); };
    auto go = [&](auto c, int per_sm) {
        using C = decltype(c);
        return launch_gemm<C>(p, am, x, K, R, tiles(C::BT), per_sm, 1, st);
    };
    auto go_split = [&](auto c) {
        using C = decltype(c);
        int cs = 8;
        while (cs > 1 && (cs > p.nkb || tiles(C::BT) * cs > 4ll * sm_count())) cs /= 2;
        return launch_gemm<C>(p, am, x, K, R, tiles(C::BT), 2, cs, st);
    };
    if (each <= 16) {
        if (tiles(16) <= 2 * sm_count()) return go_split(Cfg<16, 1, false, true, 5>{});
        return go(Cfg<16, 1, false, false, 5>{}, 2);
    }
    if (each <= 64) {
        if (tiles(64) <= 2 * sm_count()) return go_split(Cfg<64, 1, false, true, 4>{});
        return go(Cfg<64, 1, false, false, 4>{}, 2);
    }
    if (each <= 256) return go(Cfg<128, 2, false, false, 6>{}, 1);
    return go(Cfg<256, 2, false, false, 4>{}, 1);
}

cudaError_t launch_fp8_wgrad(const uint8_t *xt, const float *xs, const uint8_t *dyt, const float *dys, int R, int N, int K, int E,
                             const int *offsets, void *dw, int dw_dtype, cudaStream_t st) {
    if (!tmap_encoder()) return cudaErrorNotSupported;
    GemmArgs p = {};
    p.sa = xs;
    p.sb = dys;
    p.offsets = offsets;
    p.out = dw;
    p.ldo = K;
    p.out_stride = (long long)N * K;
    p.na = K;
    p.nb = N;
    p.nkb = R / kKB;
    p.E = E;
    p.out_dtype = dw_dtype;
    cudaError_t e = error_word(&p.err);
    if (e != cudaSuccess) return e;
    CUtensorMap am;
    if (!tmap(&am, 3, xt, R, K, 1, kARows)) return cudaErrorInvalidValue;
    using C = Cfg<128, 2, true, false, 6>;
    const long long tiles = (long long)E * ((K + kARows - 1) / kARows) * ((N + C::BT - 1) / C::BT);
    return launch_gemm<C>(p, am, dyt, R, N, tiles, 1, 1, st);
}

cudaError_t fp8_error_read(unsigned *flags) {
    unsigned *word = nullptr;
    cudaError_t e = error_word(&word);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(flags, word, sizeof(unsigned), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && *flags) e = cudaMemset(word, 0, sizeof(unsigned));
    return e;
}

}  // namespace moe
