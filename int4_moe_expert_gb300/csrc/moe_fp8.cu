// Block-scaled e4m3 quantisers and products on the 5th-generation tensor cores.
//
//   matmul  y[r, n]     = sum_kb xs[kb, r] ws[e, n / 128, kb] sum_{k in kb} x[r, k] w[e][n, k]
//           (e: the expert whose offsets hold r; without offsets one weight matrix).  The gradient
//           of x is the same product with the transposed weights.
//   wgrad   dw[e][n, k] = sum_kb dys[kb, n] xs[kb, k] sum_{r in kb} dy[n, r] x[k, r]
//           over the 128-row blocks kb of expert e
//
// Every 128-element block of the inner axis is one stage of a shared-memory ring: 128 bytes a row,
// exactly one 128-byte swizzle atom, four MMAs of K 32.  The matmul's scales are general float32, so
// a block's product cannot stay in the tensor core's accumulator: its MMAs write a fresh one, and
// the epilogue warps add that, times its scales, to float32 sums in their registers, in block order.
// The wgrad's scales are powers of two and the tensor core applies them.
//
// Two kernels.  fp8_narrow_kernel: 16 rows or fewer of a weight matrix, weights as lanes (M 128),
// rows as columns (N 16), bound by the weights' bytes.  fp8_wide_kernel: rows as lanes, contiguous
// outputs as columns, tiles of 128 x 128, 128 x 256, or 256 x 256 by a pair of blocks.
//
// Warp roles: epilogue warps (tcgen05.ld, two-wide fused multiply-adds, the stores), one warp of
// tensor copies, one MMA-issuing warp, one or two warps of scales.  mbarrier rings connect them;
// every wait is bounded, and a block that gives up sets the error word, waits (bounded) for its
// copies and MMAs and frees its tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>
#include <cstring>
#include <type_traits>

#include "moe_internal.h"
#include "moe_ptx.h"

// device error word of the handle-less products (moe_fp8_device_error)
static __device__ unsigned g_fp8_err;

namespace moe {
namespace {

constexpr int kKB = 128;                 // inner elements per stage and per scale
constexpr int kARows = 128;              // lanes of a tile
constexpr int kABytes = kARows * kKB;    // A bytes of a stage

struct NarrowArgs {
    const float *sa;        // weights' block scales [E][ceil(na / 128)][nkb]
    const float *sb;        // rows' scales [nkb][nb]
    const int *offsets;     // [E + 1] or NULL
    void *out;
    long long ldo;          // elements between rows of out
    int na, nb;             // weight rows (of one expert), rows of x
    int nkb;                // 128-blocks of the inner axis
    int E;
    int out_dtype;
    unsigned *err;
    int stall, stall_block;       // testing: this block of every tile's stops copying after `stall` stages
};

template <bool SPLIT_>
struct NarrowCfg {
    static constexpr int BT = 16;            // rows of x of a tile, the MMA's columns
    static constexpr bool SPLIT = SPLIT_;    // a cluster shares one tile, each block part of the inner axis
    static constexpr int S = 5;              // stages: two blocks an SM keep 180 KB of weights in flight
    static constexpr int EW = 4;             // epilogue warps
    static constexpr int THREADS = 32 * (EW + 4);
    static constexpr int NT = 4;             // accumulator ring
    static constexpr int TCOLS = NT * BT;
    static constexpr int STAGE = kABytes + BT * kKB;
    static constexpr int SS = 8;             // scale ring
    static constexpr int PER_SM = 2;         // blocks an SM holds
    static constexpr size_t SMEM = (size_t)S * STAGE + 1024;
    // f8f6f4: D f32 at bit 4, A and B e4m3 (0), N / 8 at bit 17, M / 16 at bit 24
    static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BT >> 3) << 17) | ((128u >> 4) << 24);
    static_assert(!SPLIT || (size_t)kARows * BT * 4 <= (size_t)S * STAGE, "partial sums reuse the stage ring");
    static_assert(PER_SM * (SMEM + 6 * 1024) <= 227 * 1024, "two blocks fit an SM");
};

constexpr int kMaxExperts = 1024;
constexpr uint32_t kMaxSplit = 8;        // blocks of a cluster that share a tile

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
__device__ __forceinline__ void prefetch_map(const void *map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }
// K-major operand with the 128-byte swizzle: groups of 8 rows 1024 bytes apart
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// N columns of this lane from tensor memory, and the wait for them: one block of code, so that the
// registers are not named before they are filled (a separate wait that names them costs a move each)
template <int N>
__device__ __forceinline__ void tc_ld(uint32_t taddr, uint32_t (&r)[N]) {
    static_assert(N == 16 || N == 64, "columns of a load");
    if constexpr (N == 64) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
                     "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                     "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
                     "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
                     "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                       "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                       "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
                       "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
                       "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
                       "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
                       "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
                     : "r"(taddr) : "memory");
    } else {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
                     "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr) : "memory");
    }
}
// one lane of a converged warp, chosen so that the compiler keeps the warp's values in uniform
// registers: the tensor copies and MMAs take their operands there, and a branch on the lane number
// costs ~100 cycles for each of them (measured: 980 cycles a stage in the issuing thread, 512 of
// tensor work)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// mbar_try that also acquires what the other block of a cluster released to the barrier
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// mbar_wait that also gives up once another role of the block has
template <bool CLUSTER = false>
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, const volatile int *fail) {
    auto passed = [&] { return CLUSTER ? mbar_try_cluster(bar, parity) : mbar_try(bar, parity); };
    if (passed()) return true;
    const unsigned long long t0 = tc_now();
    for (;;) {
        for (int i = 0; i < 64; i++)
            if (passed()) return true;
        if (*fail || tc_now() - t0 > kTcWaitNs) return false;
    }
}
// slot and phase of a ring of N, counted without divisions
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1u;
        }
    }
};
// 4-byte asynchronous copy global -> shared; !in: zeros
__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// this thread's arrival, once its asynchronous copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The two scales of a block's sum, whose product may lie outside float32's normal range although the
// scaled sum lies inside: the sum times f, times p, times q, of which f keeps the mantissas, so that
// only the last product can overflow or lose bits.
struct FarScale {
    float f, p, q;
    __device__ __forceinline__ FarScale(float a, float b) {
        int e = 0;
        f = mantissa(a, e) * mantissa(b, e);
        e = min(max(e, -250), 250);      // beyond it any sum but 0 leaves float32 (they lie between 2^-18 and 2^25)
        p = __uint_as_float((unsigned)(127 + e / 2) << 23);
        q = __uint_as_float((unsigned)(127 + e - e / 2) << 23);
    }
    // v / 2^e in [1, 2), e added to `e`; 0, infinities and NaN as they are
    static __device__ __forceinline__ float mantissa(float v, int &e) {
        if (fabsf(v) < 0x1p-126f) {
            v *= 0x1p24f;
            e -= 24;
        }
        const uint32_t u = __float_as_uint(v);
        if (v == 0.0f || (u & 0x7F800000u) == 0x7F800000u) return v;
        e += (int)((u >> 23) & 0xFFu) - 127;
        return __uint_as_float((u & 0x807FFFFFu) | 0x3F800000u);
    }
    __device__ __forceinline__ uint32_t times(uint32_t sum) const { return __float_as_uint(__uint_as_float(sum) * f * p * q); }
};
__device__ __forceinline__ bool is_finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }
// kFar or more: not a normal number
constexpr uint32_t kFar = 0xFE000000u;
__device__ __forceinline__ uint32_t farness(float product) { return 2u * __float_as_uint(product) - 0x01000000u; }
// the product of two numbers overflows, or loses bits below the normal range (that of powers of two hardly does)
__device__ __forceinline__ bool far_scales(float a, float b) {
    const float f = a * b;
    return farness(f) >= kFar && a != 0.0f && b != 0.0f && is_finite(a) && is_finite(b) && (!is_finite(f) || a * 0x1p48f * b != f * 0x1p48f);
}
// c and the products of four e4m3 codes
__device__ __forceinline__ float dot4(uint32_t a, uint32_t b, float c) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
        uint32_t u, v;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(u) : "h"((uint16_t)(a >> (16 * i))));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"((uint16_t)(b >> (16 * i))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u)), g = __half22float2(*reinterpret_cast<const __half2 *>(&v));
        c = fmaf(f.x, g.x, fmaf(f.y, g.y, c));
    }
    return c;
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
// Arrives once this thread's reads of its cluster's memory are done.  Relaxed, since the arrival hands
// over no data and a release costs 0.5 us; what orders it behind the reads is that it depends on them:
// `zero` is 0, but only the values that were read, masked by a run-time 0, say so.
__device__ __forceinline__ void cluster_done_reading(uint32_t zero) {
    if (zero == 0) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_peer(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// counts `bytes` as copied on this block's barrier
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
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
    const NarrowArgs &p;
    const int *first;   // shared memory, [E + 1]: column tiles before each expert (matmul with offsets)
    int nat, e;
    __device__ Walk(const NarrowArgs &p_, const int *first_) : p(p_), first(first_), nat((p_.na + kARows - 1) / kARows), e(0) {}
    __device__ __forceinline__ int total() const { return nat * (p.offsets ? first[p.E] : (p.nb + C::BT - 1) / C::BT); }
    __device__ __forceinline__ Tile at(int t) {
        Tile r;
        const int j = t / nat;
        r.a0 = (t - j * nat) * kARows;
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
        return r;
    }
};

// first[e + 1] holds expert e's tiles: makes it the tiles of experts 0..e (one warp)
__device__ __forceinline__ void prefix_tiles(int *first, int E, int lane) {
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        int v = e0 + lane < E ? first[e0 + lane + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        if (e0 + lane < E) first[e0 + lane + 1] = run + v;
        run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) first[0] = 0;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM) fp8_narrow_kernel(const __grid_constant__ CUtensorMap amap,
                                                                           const __grid_constant__ CUtensorMap bmap,
                                                                           const NarrowArgs p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long s_full[C::S], s_empty[C::S];
    __shared__ __align__(8) unsigned long long s_tfull[C::NT], s_tempty[C::NT];
    __shared__ __align__(8) unsigned long long s_sfull[C::SS], s_sempty[C::SS];
    __shared__ __align__(8) unsigned long long s_drain;
    __shared__ __align__(16) float s_scale[C::SS][C::BT];
    __shared__ float s_wscale[C::SS];
    __shared__ int s_first[kMaxExperts + 1];
    __shared__ uint32_t s_taddr;
    __shared__ int s_fail, s_issued;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;

    if (tid == 0) {
        prefetch_map(&amap);
        prefetch_map(&bmap);
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
    wait_for_stream();
    if (p.offsets) {
        // column tiles of every expert; the running sum by one warp
        for (int e = tid; e < p.E; e += C::THREADS) {
            const int a = min(max(p.offsets[e], 0), p.nb), b = min(max(p.offsets[e + 1], a), p.nb);
            s_first[e + 1] = (b - a + C::BT - 1) / C::BT;
        }
        __syncthreads();
        if (warp == 0) prefix_tiles(s_first, p.E, lane);
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
        // epilogue: lane quarter warp % 4
        const int q4 = warp & 3;
        const uint32_t trow = taddr + ((uint32_t)(32 * q4) << 16);
        Ring<C::NT> tq;
        Ring<C::SS> ts;
        bool ok = true;
        for (int t = t0; t < total && ok; t += tstep) {
            Tile ti = walk.at(t);
            part(ti);
            uint64_t acc[C::BT / 2];
#pragma unroll
            for (int i = 0; i < C::BT / 2; i++) acc[i] = 0ull;
            for (int kb = ti.k0; kb < ti.k1; kb++) {
                const int q = tq.slot, s = ts.slot;
                if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_sfull[s]), ts.phase, fail) &&
                                                 ring_wait(smem_u32(&s_tfull[q]), tq.phase, fail))) {
                    *fail = 1;
                    ok = false;
                    break;
                }
                tq.next();
                ts.next();
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t sc = smem_u32(&s_scale[s][0]), f = __float_as_uint(s_wscale[s]);
                const uint64_t ws = pack2(f, f);
                uint32_t r[C::BT];
                tc_ld<C::BT>(trow + (uint32_t)(q * C::BT), r);
                // the accumulator is in registers: the slot may be written again
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                if (lane == 0) mbar_arrive(smem_u32(&s_tempty[q]));
                const float mine = s_scale[s][lane % C::BT], wscale = __uint_as_float(f);
                if (__any_sync(0xffffffffu, farness(mine * wscale) >= kFar && mine != 0.0f && wscale != 0.0f)) {
#pragma unroll
                    for (int i = 0; i < C::BT; i += 2) {
                        const FarScale a(s_scale[s][i], wscale), b(s_scale[s][i + 1], wscale);
                        acc[i / 2] = add2(acc[i / 2], pack2(a.times(r[i]), b.times(r[i + 1])));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C::BT; i += 4) {
                        uint64_t s0, s1;
                        lds_2x64(sc + 4u * i, s0, s1);
                        acc[i / 2] = fma2(pack2(r[i], r[i + 1]), mul2(s0, ws), acc[i / 2]);
                        acc[i / 2 + 1] = fma2(pack2(r[i + 2], r[i + 3]), mul2(s1, ws), acc[i / 2 + 1]);
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
                for (int i = 0; i < C::BT / 2; i++) {
                    float x, y;
                    unpack2(acc[i], x, y);
                    ps[2 * i * kARows + 32 * q4 + lane] = x;
                    ps[(2 * i + 1) * kARows + 32 * q4 + lane] = y;
                }
            } else if (n < p.na) {
                const int cols = ti.bend - ti.b0;
                const long long at = (long long)ti.b0 * p.ldo + n;
                if (p.out_dtype == MOE_DTYPE_F32) store_columns<float>(p.out, at, p.ldo, acc, cols);
                else if (p.out_dtype == MOE_DTYPE_BF16) store_columns<__nv_bfloat16>(p.out, at, p.ldo, acc, cols);
                else store_columns<__half>(p.out, at, p.ldo, acc, cols);
            }
        }
    } else {
        if (warp == C::EW) {
            // tensor copies
            Ring<C::S> r;
            bool ok = true, stalled = false;
            int n = 0;
            const int most = (int)crank == p.stall_block ? p.stall : INT_MAX;
            for (int t = t0; t < total && ok && !stalled; t += tstep) {
                Tile ti = walk.at(t);
                part(ti);
                stalled = ti.k1 - ti.k0 > most - n;
                if (stalled) ti.k1 = ti.k0 + most - n;
                for (int kb = ti.k0; kb < ti.k1; kb++) {
                    // a fresh ring's slots pass: the phase before the first is over
                    if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_empty[r.slot]), r.phase ^ 1u, fail))) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t bar = smem_u32(&s_full[r.slot]), dst = ring + (uint32_t)(r.slot * C::STAGE);
                        mbar_expect_tx(bar, C::STAGE);
                        tma_load_3d(dst, &amap, kb * kKB, ti.a0, ti.e, bar);
                        tma_load_2d(dst + kABytes, &bmap, kb * kKB, ti.b0, bar);
                    }
                    r.next();
                    n++;
                }
            }
            if (lane == 0) s_issued = n;
            if (!ok) *fail = 1;
        } else if (warp == C::EW + 1) {
            // MMA issue: one fresh accumulator of the ring per stage
            Ring<C::S> r;
            Ring<C::NT> q;
            bool ok = true, any = false;
            const uint64_t ad0 = sw128_desc(ring), bd0 = sw128_desc(ring + kABytes);
            for (int t = t0; t < total && ok; t += tstep) {
                Tile ti = walk.at(t);
                part(ti);
                for (int kb = ti.k0; kb < ti.k1; kb++) {
                    if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_full[r.slot]), r.phase, fail) &&
                                                     ring_wait(smem_u32(&s_tempty[q.slot]), q.phase ^ 1u, fail))) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (elect_one()) {
                        const uint64_t off = (uint64_t)((r.slot * C::STAGE) >> 4);
                        const uint32_t d = taddr + (uint32_t)(q.slot * C::BT);
#pragma unroll
                        for (int ks = 0; ks < 4; ks++)
                            mma_f8(d, ad0 + off + 2 * ks, bd0 + off + 2 * ks, C::IDESC, ks > 0);
                        tc_commit(smem_u32(&s_empty[r.slot]));
                        tc_commit(smem_u32(&s_tfull[q.slot]));
                    }
                    r.next();
                    q.next();
                    any = true;
                }
            }
            if (!ok) *fail = 1;
            if (any) {
                // every MMA is done before the shared memory and the tensor memory go (bounded)
                __syncwarp();
                if (elect_one()) tc_commit(smem_u32(&s_drain));
                if (!mbar_wait(smem_u32(&s_drain), 0u)) *fail = 1;
            }
        } else if (warp == C::EW + 2) {
            // scales: the columns' and the weight block's, copied asynchronously up to SS stages ahead
            Ring<C::SS> s;
            bool ok = true;
            for (int t = t0; t < total && ok; t += tstep) {
                Tile ti = walk.at(t);
                part(ti);
                const float *sa = p.sa + ((size_t)ti.e * walk.nat + ti.a0 / kARows) * p.nkb;
                for (int kb = ti.k0; kb < ti.k1; kb++) {
                    const int q = s.slot;
                    if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_sempty[q]), s.phase ^ 1u, fail))) {
                        *fail = 1;
                        ok = false;
                        break;
                    }
                    s.next();
                    const float *sb = p.sb + (size_t)kb * p.nb;
                    const bool in = ti.b0 + lane < ti.bend;
                    if (lane < C::BT) cp_async4(smem_u32(&s_scale[q][lane]), in ? sb + ti.b0 + lane : p.sb, in);
                    if (lane == 0) cp_async4(smem_u32(&s_wscale[q]), sa + kb, true);
                    cp_async_arrive(smem_u32(&s_sfull[q]));
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
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
        // sums of all blocks of the cluster, in block order: block r adds columns r, r + csize, ...;
        // every block's value of a column in flight at once
        cluster_sync_all();
        uint32_t zero = 0;
        if (t0 < total) {
            const Tile ti = walk.at(t0);
            uint32_t peer[kMaxSplit];
#pragma unroll
            for (uint32_t r = 0; r < kMaxSplit; r++) peer[r] = peer_addr(ring, r < csize ? r : 0u);
            const int l = tid & 127, n = ti.a0 + l;
            for (int c = (int)crank + (int)csize * (tid >> 7); c < C::BT; c += (int)csize * (C::THREADS >> 7)) {
                float v[kMaxSplit], sum = 0.0f;
#pragma unroll
                for (uint32_t r = 0; r < kMaxSplit; r++) v[r] = r < csize ? ld_peer(peer[r] + (uint32_t)(c * kARows + l) * 4u) : 0.0f;
#pragma unroll
                for (uint32_t r = 0; r < kMaxSplit; r++) sum += v[r];
                zero |= __float_as_uint(sum) & (uint32_t)(p.E >> 31);      // E is positive
                if (n < p.na && ti.b0 + c < ti.bend) store_out(p.out, (long long)(ti.b0 + c) * p.ldo + n, sum, p.out_dtype);
            }
        }
        cluster_done_reading(zero);
        cluster_wait();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == C::EW + 3) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(C::TCOLS) : "memory");
    }
}

// ---------------------------------------------------------------------------
// Wide tiles: lanes are the rows of the output, columns its contiguous elements.  PAIR: a cluster of
// two blocks shares a tile of 256 x 256 (cta_group::2: one MMA of M 256 over both SMs' tensor cores),
// each block copying its own 128 rows of A and half of B: 32 KB for 128 x 256 x 128 products instead
// of 48 KB, which is what an SM's path from L2 carries at the tensor cores' e4m3 rate (512 cycles a
// stage x 64 bytes).
//   matmul  A = x (lanes: rows r), B = w (columns n): a lane's scale is one number per block and 128
//           columns, so adding a block's product costs one two-wide fma per two elements.  Bound by
//           that: MMAs into one of two accumulators (512 cycles), the commit's way to the epilogue
//           warps (~280), their 2 x 64 columns out of tensor memory and into the sums (~380), the
//           release's way back (~400; from the other block through its shared memory) make ~840 cycles
//           a stage where the tensor cores need 512: 16381 x 4096 x 6144 273-276 us, 3.0 PFLOP/s.
//           A pair's full warps store by tensor copies, so that the next tile's sums do not wait for
//           the stores (with two more staging buffers and a stage less, against the others' path: 275
//           and 278 us; 65536 x 2048 x 2048 200 and 213 us; 64 experts of it 250 and 250 us).
//           Measured and not kept: accumulators of 128 columns (298-359 us: twice the waits), 32-column
//           loads, pipelined or not (420-444 us: each costs its latency), 16 warps (no registers), an MMA
//           a block with B copied to both (no way between the blocks, but 48 KB into each SM: 295 us).
//   wgrad   (MX) A = dy, B = x, both column-quantised.  Their scales are powers of two, so the tensor
//           core applies them itself (kind::mxf8f6f4; the float32's exponent byte is the ue8m0 scale)
//           and sums stay in tensor memory for kFlush blocks: 273 ns a stage, the tensor cores' rate
//           (3.2 PFLOP/s on 2048 x 2048 from 65536 rows).  64 experts' 2048 x 2048 float32 outputs:
//           277 us, bound by memory traffic (1.07 GB of stores alone take 188 us in this pattern, a
//           fill 143 us); stores by tensor copies, whose staging takes a stage: 292 us, one long sum 193
//           for 171 us; prefetching operands, mixing experts' tiles, streaming stores, 6 stages:
//           no gain or slower.
// ---------------------------------------------------------------------------

template <bool PAIR_, bool MX_, int BN_ = 256, bool SPLIT_ = false>
struct WideCfg {
    static constexpr bool PAIR = PAIR_, MX = MX_;
    static constexpr bool SPLIT = SPLIT_;                     // a cluster shares a tile, each block part of the inner axis
    static constexpr int BN = BN_;                            // columns of a tile
    static constexpr int ROWS = PAIR ? 256 : 128;             // rows of a tile
    static constexpr int BROWS = PAIR ? BN / 2 : BN;          // rows of B that one block copies
    static constexpr int STAGE = kABytes + BROWS * kKB;
    static constexpr int S = STAGE > 32768 ? 3 : (PAIR && !MX) ? 4 : 5;
    static constexpr bool TST = PAIR && !MX;                  // full warps store by tensor copies
    static constexpr int EW = 8;                              // epilogue warps: a lane quarter, half of the columns each
    static constexpr int WC = BN / 2;
    static constexpr int THREADS = 32 * (EW + 4);
    static constexpr bool BIGREG = WC > 64;
    static constexpr int SS = 8;                              // scale ring (matmul)
    [[maybe_unused]] static constexpr int RS = 8;                              // ring of scales as loaded (MX), in stages
    [[maybe_unused]] static constexpr int SG = 4, SB = 3;                      // ring of staged scales (MX): SB batches of SG stages
    [[maybe_unused]] static constexpr int SG0 = SG - 2;                        // the first batch starts there: two stages, ready sooner
    [[maybe_unused]] static constexpr int SFBYTES = 512 + 4 * BN;              // staged scales of a stage (MX): 128 + BN words
    [[maybe_unused]] static constexpr int SFCOLS = 4 + BN / 32;                // their tensor-memory columns
    static constexpr int OUTB = TST ? 8192 : 4096;            // staging of an epilogue warp: (two times) 32 rows x 128 bytes
    static constexpr int NT = MX ? 2 : 512 / BN;              // accumulators: of tiles (MX), of stages
    [[maybe_unused]] static constexpr int ACC1 = MX && 2 * BN + SFCOLS * S > 512 ? 512 - SFCOLS * S - BN : BN;   // from one to the next (MX: may overlap)
    [[maybe_unused]] static constexpr int PLD = BN + 4;                        // floats of a row of partial sums (SPLIT)
    static constexpr size_t SMEM = 1024 + (size_t)S * STAGE + EW * OUTB + (MX ? (SB * SG + RS) * SFBYTES : 0);
    // f8f6f4: D f32 at bit 4; mxf8f6f4: ue8m0 scales at bit 23
    static constexpr uint32_t IDESC = (MX ? 1u << 23 : 1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(ROWS >> 4) << 24);
    static_assert(!SPLIT || (!PAIR && 128 * PLD * 4 <= S * STAGE), "partial sums reuse the stage ring");
    static_assert(SMEM + (MX ? 2 : 16) * 1024 <= 227 * 1024, "the rings and the static arrays fit one block's shared memory");
};

// address of this shared variable in the cluster's first block
__device__ __forceinline__ uint32_t in_leader(uint32_t saddr) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(saddr));
    return a;
}
// arrival on a barrier of the other block that hands over tensor memory alone (tcgen05.fence orders
// it): no cluster-wide release, which costs a memory barrier of about a microsecond
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t caddr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}
// the same after ordinary stores to shared memory, which an operation that the other block issues reads
__device__ __forceinline__ void mbar_release_cluster(uint32_t caddr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void wide_load(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                     ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
    else
        tma_load_3d(dst, map, x, y, z, bar);
}
template <bool PAIR>
__device__ __forceinline__ void wide_commit(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(bar), "h"((uint16_t)3) : "memory");
    else
        tc_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void wide_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
    else
        mma_f8(d, a, b, idesc, acc);
}
template <bool PAIR>
__device__ __forceinline__ void wide_mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc) : "memory");
}
// 32 rows x 16 bytes of shared memory -> 4 columns of tensor memory, in all four lane quarters
template <bool PAIR>
__device__ __forceinline__ void wide_cp_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// MX: blocks of the inner axis that the tensor core adds up before the registers take the sum over.  Its
// additions truncate, so an error grows with the length (2-norm against 64 bits, float32 outputs from
// 32768 rows: 6.5e-6 in one go).
constexpr int kFlush = 16;

struct WideArgs {
    const uint8_t *a, *b;   // matmul: the codes [na][K], [E][nb][K]
    int K;
    const float *sa;        // row scales of A [nkb][na] (wgrad: power of two)
    const float *sb;        // matmul: block scales of B [E][ceil(nb / 128)][nkb]; wgrad: row scales [nkb][nb]
    const int *offsets;     // [E + 1] or NULL
    void *out;
    long long ldo, out_stride;
    int na, nb, nkb, E, out_dtype;
    int vec;                              // every output row starts on a 16-byte boundary (2: and the tensor copies can take it)
    unsigned *err;
    int stall, stall_block;               // as in NarrowArgs
};

// rows [r0, rend) (this block's 128), columns c0.., inner blocks [k0, k1) of expert e
struct WideTile {
    int e, r0, rend, c0, k0, k1;
};

template <class C>
struct WideWalk {
    const WideArgs &p;
    const int *first;    // matmul with offsets: row tiles before each expert
    int nct, nrt, e, rank;
    __device__ WideWalk(const WideArgs &p_, const int *first_, int rank_)
        : p(p_), first(first_), nct((p_.nb + C::BN - 1) / C::BN), nrt((p_.na + C::ROWS - 1) / C::ROWS), e(0), rank(rank_) {}
    __device__ __forceinline__ int total() const { return nct * (C::MX ? p.E * nrt : (p.offsets ? first[p.E] : nrt)); }
    __device__ __forceinline__ WideTile at(int t) {
        WideTile r;
        const int j = t / nct;
        r.c0 = (t - j * nct) * C::BN;
        r.k0 = 0;
        r.k1 = p.nkb;
        r.e = 0;
        r.rend = p.na;
        if (C::MX) {
            r.e = j / nrt;
            r.r0 = (j - r.e * nrt) * C::ROWS;
            if (p.offsets) {
                r.k0 = min(max(p.offsets[r.e], 0) / kKB, p.nkb);
                r.k1 = min(max(p.offsets[r.e + 1] / kKB, r.k0), p.nkb);
            }
        } else if (p.offsets) {
            while (first[e + 1] <= j) e++;
            const int a = min(max(p.offsets[e], 0), p.na);
            r.e = e;
            r.r0 = a + (j - first[e]) * C::ROWS;
            r.rend = min(max(p.offsets[e + 1], a), p.na);
        } else {
            r.r0 = j * C::ROWS;
        }
        r.r0 += 128 * rank;
        return r;
    }
};

// A warp's 32 rows x 32 float32 (64 16-bit) columns: packed values through shared memory (16-byte
// chunks permuted by the row against bank conflicts) to full 128-byte stores; rows from `rows` on
// and columns from `cols` on are not written.
template <typename T>
__device__ __forceinline__ void store_chunk(const uint4 (&v)[8], uint32_t stage, T *out, long long ldo, int rows, int cols, bool vec, int lane) {
    constexpr int PER = 16 / (int)sizeof(T);       // elements of 16 bytes
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i++)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + (uint32_t)(lane * 128 + ((i ^ (lane & 7)) << 4))), "r"(v[i].x),
                     "r"(v[i].y), "r"(v[i].z), "r"(v[i].w) : "memory");
    __syncwarp();
    if (vec && cols >= 8 * PER) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int r = 4 * i + (lane >> 3), k = lane & 7;
            uint4 u;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                         : "r"(stage + (uint32_t)(r * 128 + ((k ^ (r & 7)) << 4))) : "memory");
            if (r < rows) *reinterpret_cast<uint4 *>(out + (long long)r * ldo + k * PER) = u;
        }
    } else {
        for (int r = 0; r < min(rows, 32); r++)
            for (int c = lane; c < min(cols, 8 * PER); c += 32) {
                const uint32_t a = stage + (uint32_t)(r * 128 + (((c / PER) ^ (r & 7)) << 4) + (c % PER) * (int)sizeof(T));
                if constexpr (sizeof(T) == 4) {
                    uint32_t u;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(a) : "memory");
                    reinterpret_cast<uint32_t *>(out)[(long long)r * ldo + c] = u;
                } else {
                    uint16_t u;
                    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(u) : "r"(a) : "memory");
                    reinterpret_cast<uint16_t *>(out)[(long long)r * ldo + c] = u;
                }
            }
    }
}
template <typename T>
__device__ __forceinline__ uint32_t pack16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// 64 columns' sums of a lane's row (two neighbours in each element of v)
template <typename T>
__device__ __forceinline__ void store_64(const uint64_t *v, uint32_t stage, void *out, long long at, long long ldo, int rows, int cols, bool vec, int lane) {
    T *o = static_cast<T *>(out) + at;
    uint4 q[8];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                float a, b, c, d;
                unpack2(v[16 * h + 2 * i], a, b);
                unpack2(v[16 * h + 2 * i + 1], c, d);
                q[i] = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
            }
            if (cols > 32 * h) store_chunk<T>(q, stage, o + 32 * h, ldo, rows, cols - 32 * h, vec, lane);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float a, b;
                unpack2(v[4 * i + k], a, b);
                w[k] = pack16<T>(a, b);
            }
            q[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (cols > 0) store_chunk<T>(q, stage, o, ldo, rows, cols, vec, lane);
    }
}
__device__ __forceinline__ void store_cols(const uint64_t *v, uint32_t stage, const WideArgs &p, long long at, int rows, int cols, int lane) {
    if (p.out_dtype == MOE_DTYPE_F32) store_64<float>(v, stage, p.out, at, p.ldo, rows, cols, p.vec, lane);
    else if (p.out_dtype == MOE_DTYPE_BF16) store_64<__nv_bfloat16>(v, stage, p.out, at, p.ldo, rows, cols, p.vec, lane);
    else store_64<__half>(v, stage, p.out, at, p.ldo, rows, cols, p.vec, lane);
}

// 64 columns' partial sums of a row to shared memory
__device__ __forceinline__ void partial_64(const uint64_t *v, uint32_t at) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at + 8u * i), "l"(v[i]), "l"(v[i + 1]) : "memory");
}

// A warp's full 32 rows x 128 columns from row `row`, column c0 on, by tensor copies from two staged
// chunks of 32 x 128 bytes (the copy's swizzle is store_chunk's permutation).  All of them inside the
// matrix: at its edge a copy writes whole 16-byte pieces, past a width that does not end with one.
// The registers are free once the chunks are staged.
template <typename T>
__device__ __forceinline__ void store_async(const uint64_t (&v)[64], uint32_t stage, const void *map, int row, int c0, int lane) {
    constexpr int PER = 128 / (int)sizeof(T), NCH = 128 / PER;      // columns of a chunk, chunks
#pragma unroll
    for (int c = 0; c < NCH; c++) {
        if (c % 2 == 0) {      // both buffers have been read
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
        }
        const uint32_t buf = stage + (uint32_t)((c & 1) * 4096);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            uint32_t w[4];
            if constexpr (sizeof(T) == 4) {
                float f[4];
                unpack2(v[c * 16 + 2 * i], f[0], f[1]);
                unpack2(v[c * 16 + 2 * i + 1], f[2], f[3]);
#pragma unroll
                for (int k = 0; k < 4; k++) w[k] = __float_as_uint(f[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    float a, b;
                    unpack2(v[c * 32 + 4 * i + k], a, b);
                    w[k] = pack16<T>(a, b);
                }
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + (uint32_t)(lane * 128 + ((i ^ (lane & 7)) << 4))), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(c0 + c * PER), "r"(row), "r"(buf) : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
}

// The outputs of those of a warp's 32 rows that have far scales, once more: each block's sum in float32 by
// ordinary instructions, scaled without an intermediate value that leaves float32's range.  Such scales
// are rare (gradients next to either end of the range), and a second way through the loop over the blocks
// costs the usual one moves of its sums: 16381 x 4096 x 6144 281 -> 345 us, against no more time for
// one maximum of the products' farness in the loop.  Called once no other role waits for this warp.
// x, xs: the first row's codes and scale (block kb's at xs + kb na); w, ws: the first column's
__device__ __noinline__ void far_rows(const uint8_t *x, const float *xs, int na, const uint8_t *w, const float *ws, int K, int k0, int k1, int rows,
                                      int cols, void *out, long long ldo, int dtype, int lane) {
    bool mine = false;
#pragma unroll 4
    for (int kb = k0; kb < (lane < rows ? k1 : k0); kb++) mine |= far_scales(load_in(xs + (size_t)kb * na + lane), load_in(ws + kb));
    for (unsigned todo = __ballot_sync(0xffffffffu, mine); todo; todo &= todo - 1) {
        const int r = __ffs(todo) - 1;
        for (int c = lane; c < cols; c += 32) {
            float sum = 0.0f;
            for (int kb = k0; kb < k1; kb++) {
                float s = 0.0f;
                for (int k = kb * kKB; k < min((kb + 1) * kKB, K); k += 16) {
                    const uint4 a = load_in(reinterpret_cast<const uint4 *>(x + (size_t)r * K + k)), b = load_in(reinterpret_cast<const uint4 *>(w + (size_t)c * K + k));
                    s = dot4(a.x, b.x, dot4(a.y, b.y, dot4(a.z, b.z, dot4(a.w, b.w, s))));
                }
                sum += __uint_as_float(FarScale(load_in(xs + (size_t)kb * na + r), load_in(ws + kb)).times(__float_as_uint(s)));
            }
            store_out(out, (long long)r * ldo + c, sum, dtype);
        }
    }
    __syncwarp();
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) fp8_wide_kernel(const __grid_constant__ CUtensorMap amap,
                                                                 const __grid_constant__ CUtensorMap bmap,
                                                                 const __grid_constant__ CUtensorMap omap, const WideArgs p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long s_full[C::S], s_empty[C::S];
    __shared__ __align__(8) unsigned long long s_tfull[C::NT], s_tempty[C::NT];
    __shared__ __align__(8) unsigned long long s_sfull[C::SS], s_sempty[C::SS];   // MX: by batch of stages
    __shared__ __align__(8) unsigned long long s_drain;
    __shared__ float s_scale[C::MX ? 1 : C::SS][128], s_wscale[C::MX ? 1 : C::SS][2];   // matmul: rows', weight blocks'
    __shared__ int s_first[C::MX ? 1 : kMaxExperts + 1];
    __shared__ uint32_t s_taddr;
    __shared__ int s_fail, s_issued, s_peer_issued;
    __shared__ __align__(8) unsigned long long s_rfull[C::MX ? C::RS : 1], s_rempty[C::MX ? C::RS : 1];
    static_assert(C::SB <= C::SS, "barriers for every batch of scales");
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t staging = ring + (uint32_t)(C::S * C::STAGE), sfring = staging + (uint32_t)(C::EW * C::OUTB);
    const int rank = C::PAIR ? (int)cluster_rank() : 0;
    constexpr int NB = C::PAIR ? 2 : 1;      // blocks of a tile

    if (tid == 0) {
        prefetch_map(&amap);
        prefetch_map(&bmap);
        s_fail = 0;
        s_issued = 0;
        for (int i = 0; i < C::S; i++) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&s_empty[i]), 1);
        }
        for (int i = 0; i < C::NT; i++) {
            mbar_init(smem_u32(&s_tfull[i]), 1);
            mbar_init(smem_u32(&s_tempty[i]), NB * C::EW);
        }
        for (int i = 0; i < C::SS; i++) {
            mbar_init(smem_u32(&s_sfull[i]), C::MX ? NB : 32);
            mbar_init(smem_u32(&s_sempty[i]), C::MX ? 1 : C::EW);
        }
        for (int i = 0; C::MX && i < C::RS; i++) {
            mbar_init(smem_u32(&s_rfull[i]), 32);
            mbar_init(smem_u32(&s_rempty[i]), 1);
        }
        mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::EW + 3) {
        if constexpr (C::PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_taddr)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_taddr)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    wait_for_stream();
    if (!C::MX && p.offsets) {
        for (int e = tid; e < p.E; e += C::THREADS) {
            const int a = min(max(p.offsets[e], 0), p.na), b = min(max(p.offsets[e + 1], a), p.na);
            s_first[e + 1] = (b - a + C::ROWS - 1) / C::ROWS;
        }
        __syncthreads();
        if (warp == 0) prefix_tiles(s_first, p.E, lane);
    }
    __syncthreads();
    if (C::PAIR) cluster_sync_all();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t taddr = s_taddr;
    volatile int *fail = &s_fail;
    WideWalk<C> walk(p, s_first, rank);
    const int crank = C::SPLIT ? (int)cluster_rank() : 0, csize = C::SPLIT ? (int)cluster_size() : 1;
    const int total = walk.total(), t0 = (int)blockIdx.x / (C::SPLIT ? csize : NB), tstep = C::SPLIT ? 1 << 30 : (int)gridDim.x / NB;
    auto tile_at = [&](int t) {
        WideTile r = walk.at(t);
        if (C::SPLIT) {      // this block's part of the inner axis
            const int n = r.k1 - r.k0, lo = r.k0 + (int)((long long)n * crank / csize);
            r.k1 = r.k0 + (int)((long long)n * (crank + 1) / csize);
            r.k0 = lo;
        }
        return r;
    };
    // MX: stages the exponent bytes of the scales of this block's 128 rows of A and of all columns of B from
    // the float32 values that another warp copied, in batches of SG stages.  A pair's tensor copies of
    // them are issued by its first block, so that the second's stores need a release and an acquire for
    // the whole cluster.  The release takes 1.4 us, a stage 0.27: hence one for a batch, by a warp that waits
    // for no loads, and in the second block two such warps (`which` 0 and 1) that take the batches in turn.
    // 2048 x 2048 from 65536 rows: a release for every stage 424 us, batches of 3 / 4 / 6 with as many
    // batches as fit 182 / 173 / 191, one warp for loads and stores 208.
    [[maybe_unused]] constexpr int NV = 4 + C::BN / 32;      // values a lane: 128 rows of A, the tile's of B
    [[maybe_unused]] const uint32_t raw = sfring + (uint32_t)(C::SB * C::SG * C::SFBYTES);
    [[maybe_unused]] auto stage_scales = [&](int which) {
        Ring<C::RS> q;
        Ring<C::SB> sb;
        int sg = C::SG0;
        bool ok = true, any = false, mine = which == 0;
        auto hand_over = [&] {      // the batch so far
            if (mine) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (rank) mbar_release_cluster(in_leader(smem_u32(&s_sfull[sb.slot])));
                    else mbar_arrive(smem_u32(&s_sfull[sb.slot]));
                }
            }
            if (rank) mine = !mine;
            sb.next();
            sg = 0;
        };
        for (int t = t0; t < total && ok; t += tstep) {
            const WideTile ti = tile_at(t);
            for (int kb = ti.k0; kb < ti.k1; kb++) {
                if (mine) {
                    if (!__all_sync(0xffffffffu, (sg > 0 || ring_wait(smem_u32(&s_sempty[sb.slot]), sb.phase ^ 1u, fail)) &&
                                                     ring_wait(smem_u32(&s_rfull[q.slot]), q.phase, fail))) {
                        ok = false;
                        break;
                    }
                    const uint32_t src = raw + (uint32_t)(q.slot * C::SFBYTES + lane * 4);
                    // word of row r: 16-byte line r % 32, its (r / 32) % 4-th word, 512 bytes per 128 rows
                    const uint32_t sf = sfring + (uint32_t)((sb.slot * C::SG + sg) * C::SFBYTES + lane * 16);
                    uint32_t w[NV];
#pragma unroll
                    for (int i = 0; i < NV; i++) {
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[i]) : "r"(src + 128u * i) : "memory");
                        w[i] = ((w[i] >> 23) & 0xFFu) * 0x01010101u;
                    }
#pragma unroll
                    for (int i = 0; i < NV; i += 4)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sf + 128u * i), "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]) : "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_rempty[q.slot]));
                }
                q.next();
                any = true;
                if (++sg == C::SG) hand_over();
            }
        }
        if (ok && any && sg > 0) hand_over();
        // the arrivals that free the last batches are in before this block ends
        for (int i = 0; i < C::SB && ok; i++) {
            ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&s_sempty[sb.slot]), sb.phase ^ 1u, fail));
            sb.next();
        }
        if (!ok) *fail = 1;
    };

    if (warp < C::EW) {
        // 384 threads x 168 registers at launch = 256 x 216 + 128 x 72
        if constexpr (C::BIGREG) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int q4 = warp & 3, half = warp >> 2;          // lane quarter, half of the columns
        const uint32_t trow = taddr + ((uint32_t)(32 * q4) << 16);
        const uint32_t stage = staging + (uint32_t)(warp * C::OUTB);
        const uint32_t te0 = C::PAIR ? in_leader(smem_u32(&s_tempty[0])) : smem_u32(&s_tempty[0]);
        auto release = [&](int q) {      // tensor-memory part q of this tile is in registers
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            if (lane == 0) {
                if (C::PAIR) mbar_arrive_cluster(te0 + 8u * q);
                else mbar_arrive(te0 + 8u * q);
            }
        };
        [[maybe_unused]] auto w_scales = [&](const WideTile &ti, int c0) { return p.sb + ((size_t)ti.e * ((p.nb + kKB - 1) / kKB) + c0 / kKB) * p.nkb; };
        [[maybe_unused]] float *ring_out = reinterpret_cast<float *>(smem_raw + (ring - smem_u32(smem_raw)));
        Ring<C::NT> tq;
        Ring<C::SS> ts;
        int done = 0;
        bool ok = true, far = false;      // far: of a row of this lane's (matmul)
        for (int t = t0; t < total && ok; t += tstep) {
            const WideTile ti = tile_at(t);
            const int row = ti.r0 + 32 * q4, rows = ti.rend - row, c0 = ti.c0 + C::WC * half, cols = p.nb - c0;
            const long long at = (C::MX ? (long long)ti.e * p.out_stride : 0ll) + (long long)row * p.ldo + c0;
            if constexpr (C::MX) {
                // every kFlush blocks the registers take the sums over from tensor memory (none: zeros)
                uint64_t acc[C::WC / 64][32];
#pragma unroll
                for (int l = 0; l < C::WC / 64; l++)
#pragma unroll
                    for (int i = 0; i < 32; i++) acc[l][i] = 0ull;
                for (int kc = ti.k0; kc < ti.k1; kc += kFlush) {
                    const int q = done & 1;
                    if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_tfull[q]), (uint32_t)(done >> 1) & 1u, fail))) {
                        *fail = 1;
                        ok = false;
                        break;
                    }
                    done++;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t base = trow + (uint32_t)((q ? C::ACC1 : 0) + C::WC * half);
#pragma unroll
                    for (int l = 0; l < C::WC / 64; l++) {
                        uint32_t r[64];
                        tc_ld<64>(base + 64u * l, r);
                        if (l + 1 == C::WC / 64) release(0);      // the next sums may start (the accumulators overlap)
#pragma unroll
                        for (int i = 0; i < 32; i++) acc[l][i] = add2(acc[l][i], pack2(r[2 * i], r[2 * i + 1]));
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int l = 0; l < C::WC / 64; l++) {
                    if constexpr (C::SPLIT) partial_64(acc[l], ring + (uint32_t)((32 * q4 + lane) * C::PLD + C::WC * half) * 4u);
                    else if (rows > 0) store_cols(acc[l], stage, p, at + 64 * l, rows, cols - 64 * l, lane);
                }
            } else {
                uint64_t acc[C::WC / 2];
                uint32_t worst = 0;      // farness of the scales
#pragma unroll
                for (int i = 0; i < C::WC / 2; i++) acc[i] = 0ull;
                for (int kb = ti.k0; kb < ti.k1; kb++) {
                    const int q = tq.slot, s = ts.slot;
                    if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_sfull[s]), ts.phase, fail) &&
                                                     ring_wait(smem_u32(&s_tfull[q]), tq.phase, fail))) {
                        *fail = 1;
                        ok = false;
                        break;
                    }
                    tq.next();
                    ts.next();
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const float xscale = s_scale[s][32 * q4 + lane], wscale = s_wscale[s][C::WC * half / kKB];
                    const uint32_t f = __float_as_uint(xscale * wscale);
                    const uint64_t sc = pack2(f, f);
                    worst = max(worst, farness(__uint_as_float(f)));
                    const uint32_t base = trow + (uint32_t)(C::BN * q + C::WC * half);
#pragma unroll
                    for (int l = 0; l < C::WC / 64; l++) {
                        uint32_t r[64];
                        tc_ld<64>(base + (uint32_t)(64 * l), r);
                        if (l + 1 == C::WC / 64) release(q);
#pragma unroll
                        for (int i = 0; i < 32; i++) acc[32 * l + i] = fma2(pack2(r[2 * i], r[2 * i + 1]), sc, acc[32 * l + i]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_sempty[s]));
                }
                if (!ok) break;
                far |= worst >= kFar && lane < rows && cols > 0;
                if constexpr (C::SPLIT) {
                    // partial sums [row][column] over the stage ring: every copy into it was consumed
                    partial_64(acc, ring + (uint32_t)((32 * q4 + lane) * C::PLD + C::WC * half) * 4u);
                    __syncwarp();
                    if (__any_sync(0xffffffffu, far))
                        far_rows(p.a + (size_t)row * p.K, p.sa + row, p.na, p.b + ((size_t)ti.e * p.nb + c0) * p.K, w_scales(ti, c0), p.K, ti.k0, ti.k1,
                                 rows, min(cols, C::WC), ring_out + (32 * q4) * C::PLD + C::WC * half, C::PLD, MOE_DTYPE_F32, lane);
                } else if (C::TST && p.vec == 2 && rows >= 32 && cols >= 128) {
                    if constexpr (C::TST) {
                        if (p.out_dtype == MOE_DTYPE_F32) store_async<float>(acc, stage, &omap, row, c0, lane);
                        else if (p.out_dtype == MOE_DTYPE_BF16) store_async<__nv_bfloat16>(acc, stage, &omap, row, c0, lane);
                        else store_async<__half>(acc, stage, &omap, row, c0, lane);
                    }
                } else if (rows > 0) {
                    if constexpr (C::TST) {      // an earlier tile's copies may still read the staging
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        __syncwarp();
                    }
#pragma unroll
                    for (int l = 0; l < C::WC / 64; l++) store_cols(acc + 32 * l, stage, p, at + 64 * l, rows, cols - 64 * l, lane);
                }
            }
        }
        if (C::TST && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (!C::MX && !C::SPLIT && ok && __any_sync(0xffffffffu, far)) {
            // once no other role waits for this one
            __syncwarp();
            walk.e = 0;
            for (int t = t0; t < total; t += tstep) {
                const WideTile ti = tile_at(t);
                const int row = ti.r0 + 32 * q4, rows = ti.rend - row, c0 = ti.c0 + C::WC * half, cols = p.nb - c0;
                if (rows > 0 && cols > 0)
                    far_rows(p.a + (size_t)row * p.K, p.sa + row, p.na, p.b + ((size_t)ti.e * p.nb + c0) * p.K, w_scales(ti, c0), p.K, ti.k0, ti.k1,
                             rows, min(cols, C::WC), static_cast<char *>(p.out) + ((long long)row * p.ldo + c0) * (p.out_dtype == MOE_DTYPE_F32 ? 4 : 2), p.ldo,
                             p.out_dtype, lane);
            }
        }
    } else {
        if constexpr (C::BIGREG) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == C::EW) {
            // tensor copies: this block's rows of A and its part of B
            Ring<C::S> r;
            bool ok = true, stalled = false;
            int n = 0;
            const int most = rank + crank == p.stall_block ? p.stall : INT_MAX;
            const uint32_t full0 = C::PAIR ? in_leader(smem_u32(&s_full[0])) : smem_u32(&s_full[0]);
            for (int t = t0; t < total && ok && !stalled; t += tstep) {
                WideTile ti = tile_at(t);
                stalled = ti.k1 - ti.k0 > most - n;
                if (stalled) ti.k1 = ti.k0 + most - n;
                for (int kb = ti.k0; kb < ti.k1; kb++) {
                    // a fresh ring's slots pass: the phase before the first is over
                    if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_empty[r.slot]), r.phase ^ 1u, fail))) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t bar = full0 + 8u * (uint32_t)r.slot, dst = ring + (uint32_t)(r.slot * C::STAGE);
                        if (rank == 0) mbar_expect_tx(smem_u32(&s_full[r.slot]), NB * C::STAGE);
                        wide_load<C::PAIR>(dst, &amap, kb * kKB, ti.r0, 0, bar);
                        wide_load<C::PAIR>(dst + kABytes, &bmap, kb * kKB, ti.c0 + rank * C::BROWS, C::MX ? 0 : ti.e, bar);
                    }
                    r.next();
                    n++;
                }
            }
            if (lane == 0) s_issued = n;
            if (C::PAIR && ok && !stalled) {
                // the first block's MMAs free this block's slots too: the last of those arrivals are in
                // before this block ends
                for (int i = 0; i < C::S && ok; i++) {
                    ok = __all_sync(0xffffffffu, ring_wait(smem_u32(&s_empty[r.slot]), r.phase ^ 1u, fail));
                    r.next();
                }
            }
            if (!ok) *fail = 1;
        } else if (warp == C::EW + 1) {
            // MMA issue (by the tile's first block)
            if (rank == 0) {
                Ring<C::S> r;
                Ring<C::NT> q;  // matmul: accumulator of the stage; MX: of the tile
                Ring<C::SB> sb; // MX: batch of scales, the stage's number in it
                int sg = C::SG0;
                int sums = 0;   // MX: accumulators begun
                bool ok = true, any = false;
                const uint64_t ad0 = sw128_desc(ring), bd0 = sw128_desc(ring + kABytes);
                // shared-memory operand of the scale copies: 8-row groups of 16 bytes 128 bytes apart, no swizzle
                const uint64_t sd0 = (uint64_t)((sfring >> 4) & 0x3FFF) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
                for (int t = t0; t < total && ok; t += tstep) {
                    const WideTile ti = tile_at(t);
                    const int k1 = ti.k1;
                    for (int kb = ti.k0; kb < k1; kb++) {
                        const bool fresh = C::MX && (kb - ti.k0) % kFlush == 0;
                        // MX: the previous sums, whose columns overlap these, are in registers (and so those
                        // before them, which used this accumulator)
                        if (fresh && sums > 0 && !__all_sync(0xffffffffu, ring_wait(smem_u32(&s_tempty[0]), (uint32_t)(sums - 1) & 1u, fail))) {
                            ok = false;
                            break;
                        }
                        const bool last = C::MX && (kb + 1 == k1 || (kb + 1 - ti.k0) % kFlush == 0);
                        // the operands first: they are there early, the accumulator comes back last
                        const bool w = ring_wait(smem_u32(&s_full[r.slot]), r.phase, fail) &&
                                       (C::MX ? (sg > 0 && any) || ring_wait<C::PAIR>(smem_u32(&s_sfull[sb.slot]), sb.phase, fail)
                                              : ring_wait(smem_u32(&s_tempty[q.slot]), q.phase ^ 1u, fail));
                        if (!__all_sync(0xffffffffu, w)) {
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        if (elect_one()) {
                            const uint64_t off = (uint64_t)((r.slot * C::STAGE) >> 4);
                            if constexpr (C::MX) {
                                const uint32_t tsf = taddr + (uint32_t)(512 - C::SFCOLS * (C::S - r.slot));
                                const uint64_t sd = sd0 + (uint64_t)(((sb.slot * C::SG + sg) * C::SFBYTES) >> 4);
#pragma unroll
                                for (int i = 0; i < 1 + C::BN / 128; i++) wide_cp_scales<C::PAIR>(tsf + 4 * i, sd + (uint64_t)(i * (512 >> 4)));
                                const uint32_t d = taddr + (uint32_t)(q.slot ? C::ACC1 : 0);
#pragma unroll
                                for (int ks = 0; ks < 4; ks++)
                                    wide_mma_mx<C::PAIR>(d, ad0 + off + 2 * ks, bd0 + off + 2 * ks, C::IDESC, tsf, tsf + 4, !fresh || ks > 0);
                            } else {
                                const uint32_t d = taddr + (uint32_t)(C::BN * q.slot);
#pragma unroll
                                for (int ks = 0; ks < 4; ks++) wide_mma<C::PAIR>(d, ad0 + off + 2 * ks, bd0 + off + 2 * ks, C::IDESC, ks > 0);
                            }
                            wide_commit<C::PAIR>(smem_u32(&s_empty[r.slot]));
                            if (C::MX && sg + 1 == C::SG) wide_commit<C::PAIR>(smem_u32(&s_sempty[sb.slot]));
                            if (!C::MX || last) wide_commit<C::PAIR>(smem_u32(&s_tfull[q.slot]));
                        }
                        r.next();
                        if (!C::MX || last) q.next();
                        if (last) sums++;
                        if (C::MX && ++sg == C::SG) {
                            sg = 0;
                            sb.next();
                        }
                        any = true;
                    }
                }
                if (!ok) *fail = 1;
                if (any) {
                    // every MMA is done before the shared memory and the tensor memory go (bounded)
                    __syncwarp();
                    if (elect_one()) {
                        if (C::MX && sg > 0) wide_commit<C::PAIR>(smem_u32(&s_sempty[sb.slot]));
                        if constexpr (C::PAIR)
                            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&s_drain)) : "memory");
                        else
                            tc_commit(smem_u32(&s_drain));
                    }
                    if (!mbar_wait(smem_u32(&s_drain), 0u)) *fail = 1;
                }
            } else if constexpr (C::MX) {
                stage_scales(0);
            }
        } else if constexpr (!C::MX) {
            if (warp == C::EW + 2) {
                // scales: the rows' and the two weight blocks', copied asynchronously up to SS stages ahead
                Ring<C::SS> r;
                bool ok = true;
                const int nbb = (p.nb + kKB - 1) / kKB;
                for (int t = t0; t < total && ok; t += tstep) {
                    const WideTile ti = tile_at(t);
                    const float *sw = p.sb + ((size_t)ti.e * nbb + ti.c0 / kKB + (lane & 1)) * p.nkb;
                    const bool in_w = ti.c0 + kKB * (lane & 1) < p.nb && kKB * (lane & 1) < C::BN;
                    for (int kb = ti.k0; kb < ti.k1; kb++) {
                        const int s = r.slot;
                        if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_sempty[s]), r.phase ^ 1u, fail))) {
                            *fail = 1;
                            ok = false;
                            break;
                        }
                        r.next();
                        const float *sr = p.sa + (size_t)kb * p.na;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int r = ti.r0 + 32 * i + lane;
                            cp_async4(smem_u32(&s_scale[s][32 * i + lane]), r < p.na ? sr + r : p.sa, r < p.na);
                        }
                        if (lane < 2) cp_async4(smem_u32(&s_wscale[s][lane]), in_w ? sw + kb : p.sb, in_w);
                        cp_async_arrive(smem_u32(&s_sfull[s]));
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
        } else {
            if (warp == C::EW + 2) {
                // the scales' float32 values, copied asynchronously up to RS stages ahead
                Ring<C::RS> q;
                bool ok = true;
                for (int t = t0; t < total && ok; t += tstep) {
                    const WideTile ti = tile_at(t);
                    for (int kb = ti.k0; kb < ti.k1; kb++) {
                        if (!__all_sync(0xffffffffu, ring_wait(smem_u32(&s_rempty[q.slot]), q.phase ^ 1u, fail))) {
                            *fail = 1;
                            ok = false;
                            break;
                        }
                        const uint32_t dst = raw + (uint32_t)(q.slot * C::SFBYTES + lane * 4);
                        const float *a = p.sa + (size_t)kb * p.na, *b = p.sb + (size_t)kb * p.nb;
#pragma unroll
                        for (int i = 0; i < NV; i++) {
                            const int r = (i < 4 ? ti.r0 : ti.c0 - 128) + 32 * i + lane;
                            const bool in = r < (i < 4 ? p.na : p.nb);
                            cp_async4(dst + 128u * i, in ? (i < 4 ? a : b) + r : p.sa, in);
                        }
                        cp_async_arrive(smem_u32(&s_rfull[q.slot]));
                        q.next();
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
            } else {
                stage_scales(rank);
            }
        }
    }
    __syncthreads();
    if (s_fail && tid == 0) {
        if (C::PAIR) {      // the other block gives up too (below)
            st_peer(peer_addr(smem_u32(&s_fail), (uint32_t)(rank ^ 1)), 1);
        } else {
            // after a wait that ran out: copies still in flight land before the shared memory goes (bounded)
            for (int i = max(0, s_issued - C::S); i < s_issued; i++) mbar_wait(smem_u32(&s_full[i % C::S]), (uint32_t)(i / C::S) & 1u);
            atomicOr(p.err, MOE_DEVICE_ERR_TC);
        }
    }
    if constexpr (C::SPLIT) {
        // sums of all blocks of the cluster, in block order: block r adds rows r, r + csize, ..., a warp a
        // row, every block's value in flight at once
        cluster_sync_all();
        uint32_t zero = 0;
        if (t0 < total) {
            const WideTile ti = walk.at(t0);
            uint32_t peer[kMaxSplit];
#pragma unroll
            for (uint32_t r = 0; r < kMaxSplit; r++) peer[r] = peer_addr(ring, (int)r < csize ? r : 0u);
            for (int row = crank + csize * warp; row < 128; row += csize * (C::THREADS / 32)) {
                if (ti.r0 + row >= ti.rend) break;
                float4 v[kMaxSplit], sum = make_float4(0, 0, 0, 0);
                const uint32_t off = (uint32_t)(row * C::PLD + 4 * lane) * 4u;
#pragma unroll
                for (int r = 0; r < (int)kMaxSplit; r++) v[r] = r < csize ? ld_peer4(peer[r] + off) : make_float4(0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < (int)kMaxSplit; r++) sum = make_float4(sum.x + v[r].x, sum.y + v[r].y, sum.z + v[r].z, sum.w + v[r].w);
                zero |= (__float_as_uint(sum.x) | __float_as_uint(sum.y) | __float_as_uint(sum.z) | __float_as_uint(sum.w)) & (uint32_t)(p.E >> 31);
                const int c = ti.c0 + 4 * lane;
                const long long at = (C::MX ? (long long)ti.e * p.out_stride : 0ll) + (long long)(ti.r0 + row) * p.ldo + c;
                if (p.vec && c + 4 <= p.nb) {
                    if (p.out_dtype == MOE_DTYPE_F32)
                        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = sum;
                    else if (p.out_dtype == MOE_DTYPE_BF16)
                        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) = make_uint2(pack16<__nv_bfloat16>(sum.x, sum.y), pack16<__nv_bfloat16>(sum.z, sum.w));
                    else
                        *reinterpret_cast<uint2 *>(static_cast<__half *>(p.out) + at) = make_uint2(pack16<__half>(sum.x, sum.y), pack16<__half>(sum.z, sum.w));
                } else {
                    const float f[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (c + k < p.nb) store_out(p.out, at + k, f[k], p.out_dtype);
                }
            }
        }
        cluster_done_reading(zero);
        cluster_wait();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (C::PAIR) {
        cluster_sync_all();     // the other block's MMAs, copies and arrivals reach into this one's memory
        if (s_fail) {
            // A wait ran out.  Both blocks' copies in flight land before the shared memory goes (bounded): they
            // count on the first block's barriers, which makes up for the stages that one block alone began
            if (rank == 1 && tid == 0) st_peer(peer_addr(smem_u32(&s_peer_issued), 0u), s_issued);
            cluster_sync_all();
            if (rank == 0 && tid == 0) {
                const int lo = min(s_issued, s_peer_issued), hi = max(s_issued, s_peer_issued);
                for (int i = lo; i < hi; i++) {
                    if (hi == s_issued) mbar_complete_tx(smem_u32(&s_full[i % C::S]), C::STAGE);
                    else mbar_expect_tx(smem_u32(&s_full[i % C::S]), C::STAGE);
                }
                for (int i = max(0, hi - C::S); i < hi; i++) mbar_wait(smem_u32(&s_full[i % C::S]), (uint32_t)(i / C::S) & 1u);
                atomicOr(p.err, MOE_DEVICE_ERR_TC);
            }
            cluster_sync_all();
        }
    }
    if (warp == C::EW + 3) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (C::PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
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
__device__ __forceinline__ float4 load4<float>(const float *p) { return load_in(reinterpret_cast<const float4 *>(p)); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 v = load_in(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half *p) {
    const uint2 v = load_in(reinterpret_cast<const uint2 *>(p));
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
    const int s = load_in(rows + r);
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

// Few rows: a warp per 1 x 128 block (four elements a lane), so that the blocks cover the card.
// Bound by latency.
template <typename T>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const QuantArgs p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = (int)blockIdx.x * (kQThreads / 32) + warp, kb = (int)blockIdx.y, c = kb * kKB + 4 * lane;
    wait_for_stream();
    const int s = src_row(p.rows, r, p.R, p.n_src);
    const float4 v = s >= 0 && c < p.width ? load4(static_cast<const T *>(p.x) + (long long)s * p.ld + c) : make_float4(0, 0, 0, 0);
    float inv;
    const float scale = block_scale(__reduce_max_sync(0xffffffffu, max_bits(v)), inv);
    if (r < p.R && c < p.width) {
        *reinterpret_cast<uint32_t *>(p.codes + (size_t)r * p.width + c) = codes4(v, inv);
        if (lane == 0) p.scales[(size_t)kb * p.R + r] = scale;
    }
}

// the larger magnitudes of two packed pairs (a NaN is the largest)
template <typename T>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t word_max<__nv_bfloat16>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <>
__device__ __forceinline__ uint32_t word_max<__half>(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <>
__device__ __forceinline__ uint32_t word_max<float>(uint32_t a, uint32_t b) { return max(a, b); }   // bits of magnitudes

// A lane's eight neighbouring elements of a row, as loaded (32-bit words of one or two elements).
// Maxima are kept in the same form: words of magnitudes, one 16-bit magnitude m(k) per column.
template <typename T>
struct Oct {
    static constexpr int W = 8 * (int)sizeof(T) / 4;
    static constexpr uint32_t ABS = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = load_in(reinterpret_cast<const uint4 *>(p) + i / 4);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; i++) w[i] = 0;
    }
    // elements 2 k and 2 k + 1
    __device__ __forceinline__ uint64_t pair(int k) const {
        if constexpr (sizeof(T) == 4) return pack2(w[2 * k], w[2 * k + 1]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value) return pack2(w[k] << 16, w[k] & 0xFFFF0000u);
        else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            return pack2(__float_as_uint(f.x), __float_as_uint(f.y));
        }
    }
    // float32 bits of the larger magnitude in a word of maxima
    static __device__ __forceinline__ unsigned bits(uint32_t m) {
        if constexpr (sizeof(T) == 4) return m;
        const unsigned h = max(m >> 16, m & 0xFFFFu);
        return std::is_same<T, __nv_bfloat16>::value ? h << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
    }
};
__device__ __forceinline__ uint32_t codes4(uint64_t ab, uint64_t cd) {
    float a, b, c, d;
    unpack2(ab, a, b);
    unpack2(cd, c, d);
    return __byte_perm(codes2(a, b), codes2(c, d), 0x5410);
}

// The 1 x 128 blocks of a 128 x 128 tile, along the rows (kRows) or both ways (kBoth), or one scale for
// the whole tile of a weight matrix (kWeights).
// x is read once and stays in registers: a warp holds 16 rows, a half-warp one row at a time, a lane
// eight neighbouring columns of eight neighbouring rows, so that a lane's codes of a column are eight
// neighbouring bytes of the transposed output; only codes and the columns' maxima pass through shared
// memory.  Bound by instruction issue, then by memory: the row maxima meet in one transposing
// butterfly (a lane ends with one row), a row's scale is computed once.
enum QuantMode { kRows, kBoth, kWeights };
template <typename T, QuantMode MODE>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 4 ? 2 : 4) quantize_tile_kernel(const QuantArgs p) {
    constexpr bool WT = MODE == kWeights, COLS = MODE != kRows;
    constexpr int NW = kQThreads / 32, W = Oct<T>::W;
    __shared__ __align__(16) uint8_t s_codes[COLS ? kKB * kKB : 16];
    __shared__ __align__(16) uint32_t s_col[COLS ? NW : 1][16 * W];         // column maxima of every warp's rows
    __shared__ __align__(16) float s_inv[kKB];                   // 1 / scale of every column
    __shared__ unsigned s_max[NW];
    static_assert(NW == 8, "16 rows a warp");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = lane >> 4, l16 = lane & 15;
    const int r0 = (int)blockIdx.y * kKB, kb = (int)blockIdx.x, e = (int)blockIdx.z;
    const int c = kb * kKB + 8 * l16, rw = r0 + 16 * warp;
    const T *x = static_cast<const T *>(p.x) + (WT ? (size_t)e * p.R * p.ld : 0);
    uint8_t *codes = p.codes + (WT ? (size_t)e * p.R * p.width : 0);
    const int ldt = WT ? p.R : ((p.R + kKB - 1) / kKB) * kKB;    // bytes between rows of codes_t
    uint8_t *codes_t = p.codes_t + (WT ? (size_t)e * p.R * p.width : 0);
    const int nrb = (p.R + kKB - 1) / kKB, nkb = (p.width + kKB - 1) / kKB;
    const bool in = c < p.width;

    wait_for_stream();
    const int src = src_row(p.rows, rw + l16, p.R, p.n_src);
    Oct<T> v[8];
    if (__all_sync(0xffffffffu, src >= 0 && in)) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i].load(x + (long long)__shfl_sync(0xffffffffu, src, 8 * half + i) * p.ld + c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int s = __shfl_sync(0xffffffffu, src, 8 * half + i);
            if (s >= 0 && in) v[i].load(x + (long long)s * p.ld + c);
            else v[i].zero();
        }
    }
    uint32_t cm[W], rm[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
#pragma unroll
        for (int k = 0; k < W; k++) {
            const uint32_t a = v[i].w[k] & Oct<T>::ABS;
            cm[k] = i ? word_max<T>(cm[k], a) : a;
            rm[i] = k ? word_max<T>(rm[i], a) : a;
        }
    }
    // lane ends with the maximum of row 8 half + (l16 >> 1)
#pragma unroll
    for (int d = 8; d > 1; d >>= 1) {
#pragma unroll
        for (int i = 0; i < d / 2; i++) {
            const uint32_t give = (lane & d) ? rm[i] : rm[i + d / 2], keep = (lane & d) ? rm[i + d / 2] : rm[i];
            rm[i] = word_max<T>(keep, __shfl_xor_sync(0xffffffffu, give, d));
        }
    }
    const unsigned mine = Oct<T>::bits(word_max<T>(rm[0], __shfl_xor_sync(0xffffffffu, rm[0], 1)));
    float rinv;
    if (WT) {
        const unsigned m = __reduce_max_sync(0xffffffffu, mine);
        if (lane == 0) s_max[warp] = m;
        __syncthreads();
        unsigned most = 0;
#pragma unroll
        for (int i = 0; i < NW; i++) most = max(most, s_max[i]);
        const float s = block_scale(most, rinv);
        if (tid == 0) {
            p.scales[((size_t)e * nrb + blockIdx.y) * nkb + kb] = s;
            if (p.codes_t) p.scales_t[((size_t)e * nkb + kb) * nrb + blockIdx.y] = s;
        }
    } else {
        const float s = block_scale(mine, rinv);
        const int r = rw + (lane >> 1);
        if (!(lane & 1) && r < p.R) p.scales[(size_t)kb * p.R + r] = s;
        if constexpr (COLS) {
#pragma unroll
            for (int k = 0; k < W; k++) cm[k] = word_max<T>(cm[k], __shfl_xor_sync(0xffffffffu, cm[k], 16));
            if (half == 0) {
#pragma unroll
                for (int k = 0; k < W; k += 4) *reinterpret_cast<uint4 *>(&s_col[warp][l16 * W + k]) = make_uint4(cm[k], cm[k + 1], cm[k + 2], cm[k + 3]);
            }
            __syncthreads();
            if (tid < kKB) {
                // column tid: its 16-bit half of the word that two columns share, or its own word
                constexpr bool wide = sizeof(T) == 4;
                uint32_t m = 0;
#pragma unroll
                for (int w = 0; w < NW; w++) m = word_max<T>(m, s_col[w][wide ? tid : tid >> 1]);
                float ci;
                const float t = block_scale(Oct<T>::bits(wide ? m : (tid & 1) ? m & 0xFFFF0000u : m & 0xFFFFu), ci);
                s_inv[tid] = ci;
                if (kb * kKB + tid < p.width) p.scales_t[(size_t)blockIdx.y * p.width + kb * kKB + tid] = t;
            }
            __syncthreads();
        }
    }
    uint64_t cs[4] = {};
    if (MODE == kBoth) {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            const float4 f = *reinterpret_cast<const float4 *>(&s_inv[8 * l16 + 2 * k]);
            cs[k] = pack2(__float_as_uint(f.x), __float_as_uint(f.y));
            cs[k + 1] = pack2(__float_as_uint(f.z), __float_as_uint(f.w));
        }
    }
    // codes of two rows at a time, both orientations from the same float32 values; q: this lane's
    // eight bytes of each of its columns
    const int ra = rw + 8 * half;
    uint8_t *o = codes + (size_t)ra * p.width + c;
    uint32_t q[8][2];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint64_t f[2][4];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t r = __float_as_uint(WT ? rinv : __shfl_sync(0xffffffffu, rinv, 16 * half + 2 * (i + h)));
            const uint64_t rr = pack2(r, r);
            uint64_t a[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const uint64_t u = v[i + h].pair(k);
                a[k] = mul2(u, rr);
                f[h][k] = MODE == kBoth ? mul2(u, cs[k]) : a[k];
            }
            if (in && ra + i + h < p.R)
                *reinterpret_cast<uint2 *>(o + (size_t)((i + h) * p.width)) = make_uint2(codes4(a[0], a[1]), codes4(a[2], a[3]));
        }
        if constexpr (COLS) {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float a0, a1, b0, b1;
                unpack2(f[0][k], a0, b0);
                unpack2(f[1][k], a1, b1);
                const uint32_t x0 = codes2(a0, a1), x1 = codes2(b0, b1);
                if (i % 4 == 0) {
                    q[2 * k][i / 4] = x0;
                    q[2 * k + 1][i / 4] = x1;
                } else {
                    q[2 * k][i / 4] = __byte_perm(q[2 * k][i / 4], x0, 0x5410);
                    q[2 * k + 1][i / 4] = __byte_perm(q[2 * k + 1][i / 4], x1, 0x5410);
                }
            }
        }
    }
    if constexpr (!COLS) return;
    if (WT && !p.codes_t) return;
    // 16-byte chunk `warp` of column 8 l16 + k, at chunk position warp ^ (l16 & 7) of that column's 128 bytes
#pragma unroll
    for (int k = 0; k < 8; k++)
        *reinterpret_cast<uint2 *>(&s_codes[(8 * l16 + k) * kKB + 16 * (warp ^ (l16 & 7)) + 8 * half]) = make_uint2(q[k][0], q[k][1]);
    __syncthreads();
    for (int i = tid; i < kKB * 8; i += kQThreads) {
        const int cc = i >> 3, ch = i & 7, col = kb * kKB + cc, r = r0 + 16 * ch;
        if (col >= p.width) continue;
        const uint4 u = *reinterpret_cast<const uint4 *>(&s_codes[cc * kKB + 16 * (ch ^ ((cc >> 3) & 7))]);
        uint8_t *t = codes_t + (size_t)col * ldt + r;
        if (!WT || (p.R % 16 == 0 && r < p.R)) {
            *reinterpret_cast<uint4 *>(t) = u;
        } else if constexpr (WT) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            for (int k = 0; k < 16; k++)
                if (r + k < p.R) t[k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
        }
    }
}

int sm_count() {
    static std::atomic<int> n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    int v = n[dev].load(std::memory_order_relaxed);
    if (!v && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) n[dev].store(v, std::memory_order_relaxed);
    return v > 0 ? v : 152;
}

}  // namespace

cudaError_t launch_quantize(const void *x, int dtype, long long ld, int n_src, int width, const int *rows, int R,
                            uint8_t *codes, float *scales, uint8_t *codes_t, float *scales_t, cudaStream_t st) {
    const QuantArgs p = {x, ld, rows, codes, scales, codes_t, scales_t, n_src, R, width};
    const int nkb = (width + kKB - 1) / kKB;
    if (codes_t) {
        const dim3 grid(nkb, (R + kKB - 1) / kKB);
        if (dtype == MOE_DTYPE_F32) return launch_early(quantize_tile_kernel<float, kBoth>, grid, kQThreads, 0, st, 1, p);
        if (dtype == MOE_DTYPE_BF16) return launch_early(quantize_tile_kernel<__nv_bfloat16, kBoth>, grid, kQThreads, 0, st, 1, p);
        return launch_early(quantize_tile_kernel<__half, kBoth>, grid, kQThreads, 0, st, 1, p);
    }
    // tiles where they cover two thirds of the card, else a block a warp (bf16, width 2048: 1024 rows 2.7 us
    // in tiles, 3.2 us by warps; 512 rows 2.7 and 2.5 us; 65536 rows 59 us, 0.99 of the copy rate, and 122 us)
    const dim3 tiles(nkb, (R + kKB - 1) / kKB), grid((R + 7) / 8, nkb);
    const bool few = (long long)tiles.x * tiles.y * 3 < 2 * sm_count();
    auto go = [&](auto t) {
        using T = decltype(t);
        if (few) return launch_early(quantize_rows_kernel<T>, grid, kQThreads, 0, st, 1, p);
        return launch_early(quantize_tile_kernel<T, kRows>, tiles, kQThreads, 0, st, 1, p);
    };
    if (dtype == MOE_DTYPE_F32) return go(float{});
    if (dtype == MOE_DTYPE_BF16) return go(__nv_bfloat16{});
    return go(__half{});
}

cudaError_t launch_quantize_weights(const void *w, int dtype, int E, int N, int K, uint8_t *codes, float *scales,
                                    uint8_t *codes_t, float *scales_t, cudaStream_t st) {
    const QuantArgs p = {w, K, nullptr, codes, scales, codes_t, scales_t, N, N, K};
    const dim3 grid((K + kKB - 1) / kKB, (N + kKB - 1) / kKB, E);
    if (dtype == MOE_DTYPE_F32) return launch_early(quantize_tile_kernel<float, kWeights>, grid, kQThreads, 0, st, 1, p);
    if (dtype == MOE_DTYPE_BF16) return launch_early(quantize_tile_kernel<__nv_bfloat16, kWeights>, grid, kQThreads, 0, st, 1, p);
    return launch_early(quantize_tile_kernel<__half, kWeights>, grid, kQThreads, 0, st, 1, p);
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
    static std::atomic<unsigned *> word[64] = {};
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    *err = word[dev].load(std::memory_order_relaxed);
    if (*err) return cudaSuccess;
    void *ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_fp8_err);
    if (e != cudaSuccess) return e;
    *err = static_cast<unsigned *>(ptr);
    word[dev].store(*err, std::memory_order_relaxed);
    return cudaSuccess;
}

// what moe_fp8_debug_stall_next_call asked of this thread's next product
struct Stall {
    int stages, block;
};
constexpr Stall kNoStall = {INT_MAX, 0};
thread_local Stall t_stall = kNoStall;
template <class Args>
void take_stall(Args &p) {
    p.stall = t_stall.stages;
    p.stall_block = t_stall.block;
    t_stall = kNoStall;
}

// grid: blocks (of clusters of `cluster`); the B map's box is the tile's columns
template <class C>
cudaError_t launch_narrow(const NarrowArgs &p, const CUtensorMap &am, const uint8_t *b, uint64_t b_cols, uint64_t b_rows,
                        long long tiles, int per_sm, int cluster, cudaStream_t st) {
    CUtensorMap bm;
    if (!tmap(&bm, 2, b, b_cols, b_rows, 1, C::BT)) return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<fp8_narrow_kernel<C>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const long long most = (long long)sm_count() * per_sm;
    const dim3 grid((unsigned)(C::SPLIT ? tiles * cluster : (tiles < most ? tiles : most)));
    return launch_early(fp8_narrow_kernel<C>, grid, C::THREADS, C::SMEM, st, C::SPLIT ? (unsigned)cluster : 1u, am, bm, p);
}

// y [nb columns, na rows] as boxes of 128 bytes x 32 rows for the stores; rows on 16-byte boundaries
// (no: a stride that the tensor copies cannot take)
bool out_tmap(CUtensorMap *m, const WideArgs &p) {
    const int el = p.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)p.nb, (cuuint64_t)p.na}, strides[1] = {(cuuint64_t)p.ldo * el};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / el), 32}, es[2] = {1, 1};
    const CUtensorMapDataType type = p.out_dtype == MOE_DTYPE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : p.out_dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    std::memset(m, 0, sizeof(*m));
    return tmap_encoder()(m, type, 2, p.out, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch_wide(WideArgs p, const uint8_t *a, uint64_t a_cols, const uint8_t *b, uint64_t b_cols, uint64_t b_mats,
                        long long tiles, int cluster, cudaStream_t st) {
    CUtensorMap am, bm;
    if (!tmap(&am, 3, a, a_cols, p.na, 1, 128) || !tmap(&bm, 3, b, b_cols, p.nb, b_mats, C::BROWS)) return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<fp8_wide_kernel<C>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const long long nb = C::PAIR ? 2 : 1, most = sm_count() / nb;
    const long long blocks = C::SPLIT ? tiles * cluster : nb * (tiles < most ? tiles : most);
    CUtensorMap om = {};
    if (C::TST && p.vec && out_tmap(&om, p)) p.vec = 2;
    return launch_early(fp8_wide_kernel<C>, dim3((unsigned)blocks), C::THREADS, C::SMEM, st, (unsigned)(C::SPLIT ? cluster : nb), am, bm, om, p);
}

bool rows_aligned(const void *out, long long ldo, int dtype) {
    const int el = dtype == MOE_DTYPE_F32 ? 4 : 2;
    return (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && ldo * el % 16 == 0;
}

}  // namespace

cudaError_t launch_fp8_matmul(const uint8_t *x, const float *xs, int R, const uint8_t *w, const float *ws, int E, int N, int K,
                              const int *offsets, void *y, int y_dtype, long long ldy, cudaStream_t st) {
    if (!tmap_encoder()) return cudaErrorNotSupported;
    NarrowArgs p = {};
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
    take_stall(p);
    const long long nat = (N + kARows - 1) / kARows;
    const int used = offsets ? (E < R ? E : R) : 1;      // weight matrices that rows can belong to
    const int each = (R + used - 1) / used;              // rows of one on average: the offsets are on the device
    if (each <= 16) {
        // few rows of every weight matrix: weights as lanes, 16 rows as columns, two blocks an SM; bound by
        // the weights' bytes.  Up to eight blocks share a tile's inner axis while all fit at once.
        const long long most = nat * (offsets ? (long long)R / 16 + used : ((long long)R + 15) / 16);
        int cs = (int)kMaxSplit;
        while (cs > 1 && (cs > p.nkb || most * cs > 2ll * sm_count())) cs /= 2;
        if (cs > 1) return launch_narrow<NarrowCfg<true>>(p, am, x, K, R, most, 2, cs, st);
        return launch_narrow<NarrowCfg<false>>(p, am, x, K, R, most, 2, 1, st);
    }
    WideArgs q = {};
    q.a = x;
    q.b = w;
    q.K = K;
    q.sa = xs;
    q.sb = ws;
    q.offsets = offsets;
    q.out = y;
    q.ldo = ldy;
    q.na = R;
    q.nb = N;
    q.nkb = p.nkb;
    q.E = E;
    q.out_dtype = y_dtype;
    q.vec = rows_aligned(y, ldy, y_dtype);
    q.err = p.err;
    q.stall = p.stall;
    q.stall_block = p.stall_block;
    auto wide_tiles = [&](int rows, int bn, int per_expert) {      // at most (2) or expected (1: half a tile more an expert)
        return (long long)((N + bn - 1) / bn) * (offsets ? (long long)R / rows + (used * per_expert + 1) / 2 : ((long long)R + rows - 1) / rows);
    };
    auto wide = [&](auto c, int cluster) {
        using C = decltype(c);
        return launch_wide<C>(q, x, K, w, K, E, wide_tiles(C::ROWS, C::BN, 2), cluster, st);
    };
    // The tile with the least estimated time: rounds over the card's SMs x (inner blocks x the time of
    // one + the time to store a tile), in us.  Measured a block (a stage) and a tile: 128 x 128 0.30 and
    // 0.5, 128 x 256 0.43 and 0.8, a pair's 256 x 256 0.385 and 1.4; sharing a tile's inner axis costs
    // 2.2.  (N 4096, K 6144: 512 rows 20.2 / 24.7 / 24.2 us, 16381 rows 410 / 299 / 277 us; 128 rows
    // 19.1 us alone, 11.7 us with four blocks a tile.  64 experts, N = K = 2048, 8192 rows: 66 / 62 / 71 us.)
    const long long sms = sm_count();
    auto rounds = [&](int rows, int bn, long long at_once) { return (double)((wide_tiles(rows, bn, 1) + at_once - 1) / at_once); };
    const double mid = rounds(128, 128, sms) * (0.30 * p.nkb + 0.5), one = rounds(128, 256, sms) * (0.43 * p.nkb + 0.8),
                 pair = rounds(256, 256, sms / 2) * (0.385 * p.nkb + 1.4);
    int split = 1;
    for (int cs = 2; cs <= 4; cs *= 2)      // clusters that all fit at once: a second round would start from nothing
        if (wide_tiles(128, 128, 2) * cs <= sms - 4 && p.nkb >= 2 * cs) split = cs;
    if (split > 1 && 2.2 + 0.30 * p.nkb / split < (mid < one ? mid : one)) return wide(WideCfg<false, false, 128, true>{}, split);
    if (mid <= one && mid <= pair) return wide(WideCfg<false, false, 128>{}, 1);
    if (one <= pair) return wide(WideCfg<false, false>{}, 1);
    return wide(WideCfg<true, false>{}, 1);
}

cudaError_t launch_fp8_wgrad(const uint8_t *xt, const float *xs, const uint8_t *dyt, const float *dys, int R, int N, int K, int E,
                             const int *offsets, void *dw, int dw_dtype, cudaStream_t st) {
    if (!tmap_encoder()) return cudaErrorNotSupported;
    WideArgs p = {};
    p.sa = dys;
    p.sb = xs;
    p.offsets = offsets;
    p.out = dw;
    p.ldo = K;
    p.out_stride = (long long)N * K;
    p.na = N;
    p.nb = K;
    p.nkb = R / kKB;
    p.E = E;
    p.out_dtype = dw_dtype;
    p.vec = rows_aligned(dw, K, dw_dtype);
    const cudaError_t e = error_word(&p.err);
    if (e != cudaSuccess) return e;
    take_stall(p);
    auto tiles = [&](int rows, int bn) { return (long long)E * ((N + rows - 1) / rows) * ((K + bn - 1) / bn); };
    // Few outputs from many rows: 128 x 128 tiles, whose inner range a cluster shares, all at once (clusters
    // of eight fit about 14 times); else a pair's 256 x 256 tiles.  Estimated in us from measurements: a
    // pair's block 0.273 and tile 1.2, a cluster's block 0.31 and its exchange 2.5 more (512 x 512 from
    // 32768 rows: 76 us by pairs, 28 us by four blocks a tile; from 256 rows 8.3 and 8.4 us).
    const long long sms = sm_count();
    const double per = (double)p.nkb / E;
    const double pair = (double)((tiles(256, 256) + sms / 2 - 1) / (sms / 2)) * (0.273 * per + 1.2);
    int split = 1;
    for (int cs = 2; cs <= (int)kMaxSplit; cs *= 2)
        if (tiles(128, 128) * cs <= sms - (cs > 4 ? 40 : 4) && per >= 2 * cs) split = cs;
    auto go = [&](auto c, int cluster) {
        using C = decltype(c);
        return launch_wide<C>(p, dyt, R, xt, R, 1, tiles(C::ROWS, C::BN), cluster, st);
    };
    if (split > 1 && 0.31 * per / split + 2.5 < pair) return go(WideCfg<false, true, 128, true>{}, split);
    return go(WideCfg<true, true>{}, 1);
}

void fp8_stall_next(int stages, int block) { t_stall = {stages, block}; }

cudaError_t fp8_error_read(unsigned *flags) {
    unsigned *word = nullptr;
    cudaError_t e = error_word(&word);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(flags, word, sizeof(unsigned), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && *flags) e = cudaMemset(word, 0, sizeof(unsigned));
    return e;
}

}  // namespace moe
