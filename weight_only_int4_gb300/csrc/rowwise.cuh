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

// Two FP32 values in a 64-bit register, two operations per instruction, each
// rounded as alone: what bounds these kernels next to the memory is the
// instructions they issue.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ float2 parts(Pair p) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(p));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Eight consecutive elements in their own type: 16 bytes, or 32 for FP32.
template <int kType>
struct Vec8 {
    static constexpr int kQuads = kType == kF32 ? 2 : 1;
    uint4 v[kQuads];
    // `at`: the thread's byte in the array, the vector's first
    __device__ void zero() {
#pragma unroll
        for (auto& q : v) q = make_uint4(0, 0, 0, 0);
    }
    // read once: not kept in L1
    __device__ void load_stream(const void* at) {
        const uint4* p = static_cast<const uint4*>(at);
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                         : "l"(p + i));
    }
    // read again by other rows: kept
    __device__ void load_shared(const void* at) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) v[i] = __ldg(static_cast<const uint4*>(at) + i);
    }
    __device__ void store(void* at) const {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) static_cast<uint4*>(at)[i] = v[i];
    }
    __device__ void widen(Pair (&f)[4]) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kType == kF32) f[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
            if constexpr (kType == kBf16)
                f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
            if constexpr (kType == kF16) {
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[i] = pair(h.x, h.y);
            }
        }
    }
    __device__ void round(const Pair (&f)[4]) {
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = parts(f[i]);
            if constexpr (kType == kF32) {
                w[2 * i] = __float_as_uint(t.x);
                w[2 * i + 1] = __float_as_uint(t.y);
            } else if constexpr (kType == kBf16) {
                const __nv_bfloat162 h = __float22bfloat162_rn(t);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __float22half2_rn(t);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
};

// Sum of squares of eight values onto two sums: of 16-bit values without widening
// them first, each square exact.
template <int kType>
__device__ __forceinline__ float2 add_squares(const Vec8<kType>& x, float2 sum) {
    if constexpr (kType == kF32) {
        Pair f[4], s = pair(sum.x, sum.y);
        x.widen(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma2(f[i], f[i], s);
        return parts(s);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(x.v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum.x = fma_mixed<kType == kBf16, 0, 0>(w[i], w[i], sum.x);
            sum.y = fma_mixed<kType == kBf16, 1, 1>(w[i], w[i], sum.y);
        }
        return sum;
    }
}

// Larger of a running magnitude and those of eight values, as FP32 bits; a NaN
// stays one, so infinity and NaN end up above every finite value.
__device__ __forceinline__ uint32_t magnitude(const Pair (&f)[4], uint32_t m) {
    float v = __uint_as_float(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = parts(f[i]);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(fabsf(t.x)));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(fabsf(t.y)));
    }
    return __float_as_uint(v);
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
        Pair f[4];
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

// Sum / maximum over the threads of a row (the block, or with kWarps a warp), the
// same in every thread, the sum in a fixed order. `scratch`: 32 words, 16-byte aligned, that no other
// reduction of the row uses. Every thread calls it.
template <bool kWarps>
__device__ __forceinline__ float block_sum(float v, float* scratch) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (kWarps) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    if (threadIdx.x < 32 && threadIdx.x >= warps) scratch[threadIdx.x] = 0.f;
    __syncthreads();
    const float4* four = reinterpret_cast<const float4*>(scratch);
    float4 s = four[0];
#pragma unroll 4
    for (int w = 4; w < warps; w += 4) {
        const float4 t = four[w >> 2];
        s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
    }
    return (s.x + s.y) + (s.z + s.w);
}
template <bool kWarps>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* scratch) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (kWarps) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < warps ? scratch[threadIdx.x & 31] : 0u);
}

// int8 codes of a row with largest magnitude amax,
//
//     c = RN(127 v / amax), ties to even,   scale = RN(amax / 127),
//
// decided exactly. f = 127 / amax is off by a relative 2^-23 at most and the product
// v f enters a fused addition, so the nearest whole number is right unless
// 127 v / amax lies within 2^-16 of a half.
//
// FP32 values: there 254 |v| is compared with (2 k + 1) amax, k the whole number
// below, each product held as a rounded value and its exact remainder.
//
// 16-bit values: v and amax have at most 11 bits, X and A as whole numbers. With
// q = 127 X / (A 2^j), what is not a half is at least 1 / (2 A 2^j) >= 2^-20 q away
// from it, more than the error: only halves themselves matter. They are the
// solutions of 254 X = (2 k + 1) A 2^j. Where 127 does not divide A, the odd part of A
// divides X and 2 k + 1 = 127: v is half of amax, q = 63.5, and f rounded up takes
// it to 64, the even one. Where 127 divides A, f is exact for A = 127 2^i (bfloat16
// has no other such A) and the fused addition rounds halves to even itself; else the row is
// compared as above.
//
// Rows far from 1 are moved there by a power of two, so neither f nor a product
// leaves the FP32 range.
template <int kType>
struct RowCodes {
    float amax;     // after the power of two
    float factor;   // 127 / amax, rounded up; 0 for a row of zeros or with an infinity or NaN
    float move;
    float scale;    // NaN for a row with an infinity or NaN
    bool compare;

    __device__ explicit RowCodes(uint32_t amax_bits) {
        const float a = __uint_as_float(amax_bits);
        const bool plain = amax_bits != 0u && amax_bits < 0x7F800000u;
        move = a > 0x1p100f ? 0x1p-64f : a < 0x1p-64f ? 0x1p64f : 1.f;
        amax = a * move;
        factor = __fdiv_rn(127.f, amax);
        const float below = __fmaf_rn(factor, amax, -127.f);   // exact
        if (below < 0.f) factor = __uint_as_float(__float_as_uint(factor) + 1u);
        if (!plain) factor = 0.f;
        scale = plain ? __fdiv_rn(a, 127.f) : amax_bits ? __uint_as_float(0x7FC00000u) : 0.f;
        compare = kType == kF32 ||
                  (kType == kF16 && ((__float_as_uint(amax) & 0x7FFFFFu) | 0x800000u) % 127u == 0u && below != 0.f);
    }
    static constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to a whole number in the low bits
    static constexpr float kNear = 0.5f - 0x1p-15f;

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
    __device__ uint2 operator()(Pair (&v)[4]) const {
        if (factor == 0.f) return make_uint2(0u, 0u);
        if (move != 1.f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(move));
        }
        Pair f[4];
        const Pair by = both(factor), magic = both(kMagic);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = fma2(v[i], by, magic);
        if (compare) {
            const Pair minus_by = both(-factor), minus_magic = both(-kMagic);
            Pair d[4];   // minus what the code is off by
            float worst = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[i] = fma2(v[i], minus_by, add2(f[i], minus_magic));
                const float2 t = parts(d[i]);
                worst = fmaxf(worst, fmaxf(fabsf(t.x), fabsf(t.y)));
            }
            if (worst > kNear) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 t = parts(d[i]), x = parts(v[i]);
                    float2 c = parts(f[i]);
                    if (fabsf(t.x) > kNear) c.x = kMagic + decide(x.x);
                    if (fabsf(t.y) > kNear) c.y = kMagic + decide(x.y);
                    f[i] = pair(c.x, c.y);
                }
            }
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = parts(f[i]);
            w[i] = prmt(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040u);
        }
        return make_uint2(prmt(w[0], w[1], 0x5410u), prmt(w[2], w[3], 0x5410u));
    }
};

}  // namespace rowwise
}  // namespace w4a16
