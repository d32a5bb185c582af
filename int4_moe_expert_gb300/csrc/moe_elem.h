// Elements of the handle-less operators: loads and stores of neighbouring float32, float16 or bfloat16
// values, sums over a block, and the e4m3 block scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "moe_internal.h"

namespace moe {

__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
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

// 2^x to a relative 2^-22 and 1 / x to 2^-23 (the documented errors), subnormals as zeros
__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// two neighbours of one 32-bit word, and back (rounded to nearest even)
template <typename T>
__device__ __forceinline__ void from_word(uint32_t w, float &a, float &b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        a = f.x;
        b = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint32_t to_word(float a, float b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
template <typename T>
__device__ __forceinline__ float to_float(T v) {
    if constexpr (std::is_same<T, float>::value) return v;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __bfloat162float(v);
    else return __half2float(v);
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
    if constexpr (std::is_same<T, float>::value) return v;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(v);
    else return __float2half_rn(v);
}

// V neighbours as the 32-bit words that hold them (one element in the low half for V = 1 of a 16-bit
// type); p on V elements' boundary, 16 bytes at most
template <typename T, int V>
struct Vec {
    static constexpr int BYTES = V * (int)sizeof(T), W = (BYTES + 3) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 v = load_in(reinterpret_cast<const uint4 *>(p) + i / 4);
                w[i] = v.x;
                w[i + 1] = v.y;
                w[i + 2] = v.z;
                w[i + 3] = v.w;
            }
        } else if constexpr (BYTES == 8) {
            const uint2 v = load_in(reinterpret_cast<const uint2 *>(p));
            w[0] = v.x;
            w[1] = v.y;
        } else if constexpr (BYTES == 4) {
            w[0] = load_in(reinterpret_cast<const uint32_t *>(p));
        } else {
            w[0] = load_in(reinterpret_cast<const unsigned short *>(p));
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < W; i += 4) reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (BYTES == 4) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else {
            *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; i++) w[i] = 0;
    }
    __device__ __forceinline__ void get(float *v) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = __uint_as_float(w[i]);
        } else if constexpr (V == 1) {
            float other;
            from_word<T>(w[0], v[0], other);
        } else {
#pragma unroll
            for (int i = 0; i < W; i++) from_word<T>(w[i], v[2 * i], v[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void set(const float *v) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; i++) w[i] = __float_as_uint(v[i]);
        } else if constexpr (V == 1) {
            w[0] = to_word<T>(v[0], 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < W; i++) w[i] = to_word<T>(v[2 * i], v[2 * i + 1]);
        }
    }
};

// The sum of v over the threads of a block (or, WARP, of a warp), in every one of them and in the same
// order each time.  buf: a word for each warp, free again after the next barrier of the block.
template <bool WARP, typename V>
__device__ __forceinline__ V sum_all(V v, V *buf) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31, nw = (int)blockDim.x >> 5;
        if (lane == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < nw ? buf[lane] : (V)0;
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    }
    return v;
}

// every row of x (el bytes an element, ld elements apart) on a boundary of `bytes`
inline bool runs_of(const void *x, long long ld, int el, int bytes) {
    return reinterpret_cast<uintptr_t>(x) % (uintptr_t)bytes == 0 && ld * el % bytes == 0;
}

// calls f with a value of the type that `dtype` (MOE_DTYPE_*) names
template <typename F>
cudaError_t by_dtype(int dtype, F &&f) {
    if (dtype == MOE_DTYPE_F32) return f(float{});
    if (dtype == MOE_DTYPE_BF16) return f(__nv_bfloat16{});
    return f(__half{});
}

int sm_count();      // of the current device (moe_fp8.cu)

}  // namespace moe
