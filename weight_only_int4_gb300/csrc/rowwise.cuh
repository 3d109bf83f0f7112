// Helpers of the kernels that own whole rows: 8-element vectors in their own
// type, sums and maxima over a thread block, and the int8 codes of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace w4a16 {
namespace rowwise {

enum : int { kF16 = 0, kBf16 = 1, kF32 = 2 };

template <int kType>
constexpr int kBytes = kType == kF32 ? 4 : 2;

// Eight consecutive elements in their own type: 16 bytes, or 32 for FP32.
template <int kType>
struct Vec8 {
    static constexpr int kQuads = kType == kF32 ? 2 : 1;
    uint4 v[kQuads];
    static __device__ const uint4* place(const void* x, long long elem) {
        return reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + elem * kBytes<kType>);
    }
    __device__ void zero() {
#pragma unroll
        for (auto& q : v) q = make_uint4(0, 0, 0, 0);
    }
    // read once: not kept in L1
    __device__ void load_stream(const void* x, long long elem) {
        const uint4* p = place(x, elem);
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                         : "l"(p + i));
    }
    // read again by other rows: kept
    __device__ void load_shared(const void* x, long long elem) {
        const uint4* p = place(x, elem);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) v[i] = __ldg(p + i);
    }
    __device__ void store(void* x, long long elem) const {
        uint4* p = const_cast<uint4*>(place(x, elem));
#pragma unroll
        for (int i = 0; i < kQuads; ++i) p[i] = v[i];
    }
    __device__ void widen(float (&f)[8]) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
        if constexpr (kType == kF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kType == kBf16) {
                    f[2 * i] = __uint_as_float(w[i] << 16);
                    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                } else {
                    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    f[2 * i] = t.x;
                    f[2 * i + 1] = t.y;
                }
            }
        }
    }
    __device__ void round(const float (&f)[8]) {
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
        if constexpr (kType == kF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kType == kBf16) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
    }
};

// Largest magnitude as FP32 bits: the order of the bits is the order of the
// magnitudes, infinity and NaN above every finite value.
__device__ __forceinline__ uint32_t magnitude(const float (&f)[8], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return m;
}

// As two packed 16-bit magnitudes.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Running maximum of a row in its own type, and that as FP32 bits.
template <int kType>
__device__ __forceinline__ uint32_t raw_magnitude(const Vec8<kType>& x, uint32_t m) {
    if constexpr (kType == kF32) {
        float f[8];
        x.widen(f);
        return magnitude(f, m);
    } else {
        const uint4 q = x.v[0];
        return max_u16x2(m, max_u16x2(max_u16x2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                                      max_u16x2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu)));
    }
}
template <int kType>
__device__ __forceinline__ uint32_t raw_to_f32(uint32_t m) {
    if constexpr (kType == kF32) return m;
    const uint32_t v = max(m & 0xFFFFu, m >> 16);
    if constexpr (kType == kBf16) return v << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(v))));
}

// How rows of `vecs` vectors are laid over threads: x threads hold a row, `per`
// vectors each; rows that one warp holds come y to a block (no barriers).
struct Layout {
    int per, x, y;
};
// Up to `most` vectors per thread (a power of two), no more threads than they need.
inline Layout layout_of(long long vecs, int most) {
    int per = 1;
    while (per < most && vecs > 32ll * per) per *= 2;
    const long long x = ((vecs + per - 1) / per + 31) / 32 * 32;
    return {per, static_cast<int>(x), x == 32 ? 4 : 1};
}

// Sum / maximum over the threads of a row (the block, or a warp of its own), the
// same in every thread, the sum in a fixed order. `scratch`: 32 words that no other
// reduction of the row uses. Every thread calls it.
__device__ __forceinline__ float block_sum(float v, float* scratch) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? scratch[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* scratch) {
    v = __reduce_max_sync(0xffffffffu, v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < warps ? scratch[threadIdx.x & 31] : 0u);
}

// int8 codes of a row with largest magnitude amax,
//
//     c = RN(127 v / amax), ties to even,   scale = RN(amax / 127),
//
// decided exactly. q = v * (127 / amax) is off by at most 2^-16 (two roundings
// of relative size 2^-24 at |q| <= 127), so the nearest whole number is right
// unless q lies within 2^-15 of a half; there 254 |v| is compared with
// (2 k + 1) amax, k the whole number below, each product held as a rounded value
// and its exact remainder. Rows far from 1 are moved there by a power of two,
// so neither 127 / amax nor a product leaves the FP32 range.
struct RowCodes {
    float amax;     // after the power of two
    float factor;   // 127 / amax; 0 for a row of zeros or with an infinity or NaN
    float move;
    float scale;    // NaN for a row with an infinity or NaN

    __device__ explicit RowCodes(uint32_t amax_bits) {
        const float a = __uint_as_float(amax_bits);
        const bool plain = amax_bits != 0u && amax_bits < 0x7F800000u;
        move = a > 0x1p100f ? 0x1p-64f : a < 0x1p-64f ? 0x1p64f : 1.f;
        amax = a * move;
        factor = plain ? __fdiv_rn(127.f, amax) : 0.f;
        scale = plain ? __fdiv_rn(a, 127.f) : amax_bits ? __uint_as_float(0x7FC00000u) : 0.f;
    }
    static constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to a whole number in the low bits

    // The code of v where q is next to a half: k is the lower of the two whole numbers around |q|.
    __device__ float decide(float v) const {
        const float a = fabsf(v), n = __fmaf_rn(a, factor, kMagic) - kMagic;
        const float k = n - (__fmaf_rn(a, factor, -n) < 0.f ? 1.f : 0.f), m = 2.f * k + 1.f;
        const float p = 254.f * a, pe = __fmaf_rn(254.f, a, -p);
        const float r = m * amax, re = __fmaf_rn(m, amax, -r);
        const float over = p != r ? p - r : pe - re;   // rounding keeps the order, so p != r decides
        const bool odd = static_cast<int>(k) & 1;
        return copysignf(over > 0.f || (over == 0.f && odd) ? k + 1.f : k, v);
    }

    // Eight codes, one per byte. A factor of 0 gives zeros even for an infinity or NaN.
    __device__ uint2 operator()(const float (&x)[8]) const {
        if (factor == 0.f) return make_uint2(0u, 0u);
        float v[8], f[8], worst = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = x[i];
            if (move != 1.f) v[i] *= move;
            f[i] = __fmaf_rn(v[i], factor, kMagic);
            worst = fmaxf(worst, fabsf(__fmaf_rn(v[i], factor, kMagic - f[i])));
        }
        if (worst > 0.5f - 0x1p-15f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (fabsf(__fmaf_rn(v[i], factor, kMagic - f[i])) > 0.5f - 0x1p-15f) f[i] = kMagic + decide(v[i]);
            }
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
        return make_uint2(prmt(prmt(w[0], w[1], 0x0040u), prmt(w[2], w[3], 0x0040u), 0x5410u),
                          prmt(prmt(w[4], w[5], 0x0040u), prmt(w[6], w[7], 0x0040u), 0x5410u));
    }
};

}  // namespace rowwise
}  // namespace w4a16
