// Quantisation to MXFP4 and the row layout's way back.
//
// A block is 32 consecutive elements along the axis that a product will
// contract. With amax its largest magnitude,
//
//     e = max(floor(log2(amax)) - 2 + 127, 0),   c = RN_E2M1(v * 2^(127 - e)),
//
// so the largest magnitude lands in [4, 8); E2M1 ends at 6 and what lies above
// becomes 6. An all-zero block has e = 0; a block that holds an infinity or a
// NaN has e = 255 (every value of it reads as NaN) and codes 0. floor(log2) is
// the FP32 exponent field of amax (an FP32 subnormal amax clamps to e = 0 like
// every amax below 2^-125), and 2^(127 - e) is a normal FP32 number for every
// e in 0..252, so the product v * 2^(127 - e) is exact unless it is subnormal,
// far below the first rounding boundary 0.25: each code is rounded once.
//
// Everything here streams its operands once and is bound by HBM bandwidth
// (2.53 bytes per element for 16-bit inputs) or, for small inputs, by the
// launch.
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace w4a16 {
namespace {

constexpr int kThreads = 256;

enum : int { kF16 = 0, kBf16 = 1, kF32 = 2 };

// Eight consecutive elements in their own type: 16 bytes, or 32 for FP32.
template <int kType>
struct Octet {
    uint4 v[kType == kF32 ? 2 : 1];
    __device__ void zero() {
#pragma unroll
        for (auto& q : v) q = make_uint4(0, 0, 0, 0);
    }
    __device__ void load(const void* x, long long elem) {
        const uint8_t* at = static_cast<const uint8_t*>(x) + elem * (kType == kF32 ? 4 : 2);
        const uint4* p = reinterpret_cast<const uint4*>(at);
#pragma unroll
        for (int i = 0; i < (kType == kF32 ? 2 : 1); ++i)
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                         : "l"(p + i));
    }
    __device__ void widen(float (&f)[8]) const {
        if constexpr (kType == kF32) {
            const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
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
};

// Largest magnitude of a block, as FP32 bits (NaN and infinity compare above
// every finite value), to its exponent byte and the factor 2^(127 - e).
__device__ __forceinline__ uint32_t block_exponent(uint32_t amax_bits) {
    const uint32_t E = amax_bits >> 23;
    return E == 255u ? 255u : E < 2u ? 0u : E - 2u;
}
__device__ __forceinline__ float block_factor(uint32_t e) {
    return __uint_as_float(e == 255u ? 0u : (254u - e) << 23);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// FP32 bits of the larger magnitude of two packed 16-bit ones.
template <int kType>
__device__ __forceinline__ uint32_t wide_magnitude(uint32_t m) {
    const uint32_t v = max(m & 0xFFFFu, m >> 16);
    if constexpr (kType == kBf16) return v << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(v))));
}

// Eight scaled values to a word, the first in the lowest four bits. The
// conversion rounds to nearest even and saturates at 6.
__device__ __forceinline__ uint32_t to_codes(const float (&f)[8], float s) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(f[0] * s), "f"(f[1] * s), "f"(f[2] * s), "f"(f[3] * s), "f"(f[4] * s), "f"(f[5] * s), "f"(f[6] * s),
          "f"(f[7] * s));
    return w;
}

// Byte offset of the scale word (four consecutive blocks) of row r, block
// group kg, in tiles of 128 rows x 4 blocks: within a tile, row r sits at
// (r % 32) * 16 + (r / 32 % 4) * 4, the order in which the tensor cores take
// the scales of 128 operand rows.
__device__ __forceinline__ long long scale_word(long long r, long long kg, long long groups) {
    const int ri = static_cast<int>(r & 127);
    return ((r >> 7) * groups + kg) * 512 + (ri & 31) * 16 + (ri >> 5) * 4;
}

// Rows: sixteen lanes take 128 elements of a row (four blocks, eight elements
// a lane: 16-byte loads, 4-byte stores, both coalesced); lanes past the row's
// end write the zero bytes that pad its last exponent word. kUnroll groups a
// half-warp are in flight together. What bounds it for 16-bit inputs is
// instructions per element: magnitudes are compared as packed 16-bit integers
// (the order of the bits is the order of the magnitudes) and a group's place is
// stepped, not divided for (101 us without either): 8192 x 21504 bf16 87.0 us
// (5.12 TB/s); FP32, with twice the bytes per instruction, 8192 x 8192 48.1 us
// (6.33).
template <int kType, int kUnroll, typename Index>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const void* __restrict__ x, uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ es, Index items, Index groups,
                                                              int K) {
    const int sub = threadIdx.x & 15;
    const Index half = static_cast<Index>((blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x) >> 4);
    const Index halves = static_cast<Index>((static_cast<long long>(gridDim.x) * kThreads) >> 4);
    const Index step_rows = halves / groups, step_groups = halves - step_rows * groups;
    const int words = K >> 3;
    Index next_row = half / groups, next_kg = half - next_row * groups;
    // the trip count is the same for both half-warps of a warp: the shuffles below name all lanes
    const Index first = half & ~static_cast<Index>(1);
    for (Index base = 0; first + base < items; base += halves * kUnroll) {
        Octet<kType> v[kUnroll];
        Index row[kUnroll], kg[kUnroll];
        bool valid[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            row[u] = next_row;
            kg[u] = next_kg;
            next_row += step_rows;
            next_kg += step_groups;
            if (next_kg >= groups) next_kg -= groups, ++next_row;
            valid[u] = half + base + halves * u < items && static_cast<int>(kg[u]) * 16 + sub < words;
            v[u].zero();
            if (valid[u])
                v[u].load(x, static_cast<long long>(row[u]) * K + static_cast<long long>(kg[u]) * 128 + sub * 8);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            uint32_t amax;
            if constexpr (kType == kF32) {
                float f[8];
                v[u].widen(f);
                amax = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(f[i]) & 0x7FFFFFFFu);
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            } else {
                const uint4 q = v[u].v[0];
                uint32_t m = max_u16x2(max_u16x2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                                       max_u16x2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
                m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
                amax = wide_magnitude<kType>(m);
            }
            const uint32_t e = block_exponent(amax);
            if (valid[u]) {
                float f[8];
                v[u].widen(f);
                codes[static_cast<long long>(row[u]) * words + static_cast<long long>(kg[u]) * 16 + sub] =
                    e == 255u ? 0u : to_codes(f, block_factor(e));
            }
            if ((sub & 3) == 0 && half + base + halves * u < items)
                es[scale_word(row[u], kg[u], groups) + (sub >> 2)] = static_cast<uint8_t>(e);
        }
    }
}

// Columns: a thread owns the 32 rows of one block of kCols adjacent columns
// (8-byte loads; a warp reads 256 consecutive bytes of each row): all 32 loads
// are in flight before the first is used.
// 5376 x 43008: 89.1 us (6.57 TB/s) from 16 bits, 157.2 us (6.67) from FP32.
template <int kType, typename Index>
__global__ void __launch_bounds__(kThreads) quant_cols_kernel(const void* __restrict__ x, uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ es, Index items, int N) {
    constexpr int kCols = kType == kF32 ? 2 : 4;
    const Index per_block = static_cast<Index>(N / kCols);
    for (Index it = static_cast<Index>(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x); it < items;
         it += static_cast<Index>(static_cast<long long>(gridDim.x) * kThreads)) {
        const long long blk = it / per_block;
        const int c = static_cast<int>(it - static_cast<Index>(blk) * per_block) * kCols;
        const uint8_t* src = static_cast<const uint8_t*>(x) + (blk * 32 * N + c) * (kType == kF32 ? 4 : 2);
        const long long pitch = static_cast<long long>(N) * (kType == kF32 ? 4 : 2);
        uint2 v[32];
#pragma unroll
        for (int r = 0; r < 32; ++r)
            asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                         : "=r"(v[r].x), "=r"(v[r].y)
                         : "l"(src + r * pitch));
        // element of row r, column j of the thread's
        auto elem = [&](int r, int j) -> float {
            if constexpr (kType == kF32) return __uint_as_float(j ? v[r].y : v[r].x);
            const uint32_t w = j < 2 ? v[r].x : v[r].y;
            if constexpr (kType == kBf16) return __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
            return __half2float(__ushort_as_half(static_cast<unsigned short>((j & 1) ? (w >> 16) : (w & 0xFFFFu))));
        };
        uint32_t word[4][kCols], ebytes = 0;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            uint32_t amax = 0;
#pragma unroll
            for (int r = 0; r < 32; ++r) amax = max(amax, __float_as_uint(elem(r, j)) & 0x7FFFFFFFu);
            const uint32_t e = block_exponent(amax);
            ebytes |= e << (8 * j);
            const float s = block_factor(e);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = elem(8 * w + i, j);
                word[w][j] = e == 255u ? 0u : to_codes(f, s);
            }
        }
        uint32_t* dst = codes + blk * 4 * N + c;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if constexpr (kCols == 4)
                *reinterpret_cast<uint4*>(dst + static_cast<long long>(w) * N) =
                    make_uint4(word[w][0], word[w][1], word[w][2], word[w][3]);
            else
                *reinterpret_cast<uint2*>(dst + static_cast<long long>(w) * N) = make_uint2(word[w][0], word[w][1]);
        }
        if constexpr (kCols == 4)
            *reinterpret_cast<uint32_t*>(es + blk * N + c) = ebytes;
        else
            *reinterpret_cast<uint16_t*>(es + blk * N + c) = static_cast<uint16_t>(ebytes);
    }
}

// Row layout to bf16 values: a thread takes one word (eight codes) to one
// 16-byte store. Exact, as the column layout's dense copy is.
// 8192 x 21504 80 us (5.58 TB/s), 2048 x 5376 6.8 us.
template <typename Index>
__global__ void __launch_bounds__(kThreads) dequant_rows_kernel(const uint32_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ es,
                                                                uint16_t* __restrict__ w, Index items, Index words,
                                                                Index groups) {
    constexpr int kUnroll = 4;
    const Index step = static_cast<Index>(static_cast<long long>(gridDim.x) * kThreads);
    for (Index i0 = static_cast<Index>(blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x); i0 < items;
         i0 += step * kUnroll) {
        uint32_t q[kUnroll], e[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const Index i = i0 + step * u;
            q[u] = e[u] = 0;
            if (i < items) {
                const Index row = i / words, k8 = i - row * words;
                q[u] = __ldg(codes + i);
                e[u] = __ldg(es + scale_word(row, k8 >> 4, groups) + ((k8 >> 2) & 3));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const Index i = i0 + step * u;
            if (i >= items) break;
            uint32_t fa, fb, o[4];
            mx::pair_factors(e[u], e[u], fa, fb);
            const uint32_t q4 = q[u] >> 4;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t h = prmt(q[u], q4, static_cast<uint32_t>(b | ((4 + b) << 8))) & 0x000F000Fu;
                o[b] = mx::mul_bf16x2(mx::mul_bf16x2(mx::e2m1x2_scaled(h), fa), fb);
            }
            reinterpret_cast<uint4*>(w)[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Plain scale bytes [rows, K/32] to tiles; the bytes past a row's end are zero.
// For load time: byte loads, 43008 x 5376 13.1 us (1.1 TB/s), 2048 x 5376 2.3 us.
__global__ void __launch_bounds__(kThreads) tile_scales_kernel(const uint8_t* __restrict__ src,
                                                               uint8_t* __restrict__ dst, long long items,
                                                               long long groups, long long blocks) {
    for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < items;
         i += static_cast<long long>(gridDim.x) * kThreads) {
        const long long row = i / groups, kg = i - row * groups;
        uint32_t b = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * kg + j < blocks) b |= static_cast<uint32_t>(__ldg(src + row * blocks + 4 * kg + j)) << (8 * j);
        *reinterpret_cast<uint32_t*>(dst + scale_word(row, kg, groups)) = b;
    }
}

// An ordinary launch (see launch_rows in mx_matmul.cu).
template <typename... Params, typename... Args>
cudaError_t launch(void (*kern)(Params...), long long blocks, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

// 32-bit indices (a division per item) wherever every index the kernel forms,
// one grid stride past the end included, fits them.
constexpr long long kIndexLimit = (1ll << 31) - (1ll << 26);

template <int kType>
cudaError_t quant_rows(const void* x, uint32_t* codes, uint8_t* es, long long M, long long K, const DeviceProps& dp,
                       cudaStream_t s) {
    const long long groups = (K + 127) / 128, items = M * groups;
    constexpr int kHalves = kThreads / 16;
    // one group per half-warp while the grid has room, then two at a time (three and four: the same; eight: 15 %
    // slower, registers cost more warps than the loads in flight gain)
    constexpr int kDeep = 2;
    const long long one = (items + kHalves - 1) / kHalves;
    const long long cap = static_cast<long long>(dp.sms) * 32;
    if (one <= cap)
        return launch(quant_rows_kernel<kType, 1, unsigned>, one, s, x, codes, es, items, groups, K);
    const long long grid = std::min(cap, (one + kDeep - 1) / kDeep);
    if (items < kIndexLimit)
        return launch(quant_rows_kernel<kType, kDeep, unsigned>, grid, s, x, codes, es, items, groups, K);
    return launch(quant_rows_kernel<kType, kDeep, unsigned long long>, grid, s, x, codes, es, items, groups, K);
}

template <int kType>
cudaError_t quant_cols(const void* x, uint32_t* codes, uint8_t* es, long long K, long long N, const DeviceProps& dp,
                       cudaStream_t s) {
    const long long items = (K / 32) * (N / (kType == kF32 ? 2 : 4));
    const long long grid = std::min<long long>((items + kThreads - 1) / kThreads, static_cast<long long>(dp.sms) * 16);
    if (items < kIndexLimit) return launch(quant_cols_kernel<kType, unsigned>, grid, s, x, codes, es, items, N);
    return launch(quant_cols_kernel<kType, unsigned long long>, grid, s, x, codes, es, items, N);
}

}  // namespace

cudaError_t launch_mx_quantize(const void* x, uint32_t* codes, uint8_t* es, int64_t rows, int64_t cols, int dim,
                               int type, const DeviceProps& dp, cudaStream_t s) {
    if (dim == 0) {
        if (type == kF16) return quant_cols<kF16>(x, codes, es, rows, cols, dp, s);
        if (type == kBf16) return quant_cols<kBf16>(x, codes, es, rows, cols, dp, s);
        return quant_cols<kF32>(x, codes, es, rows, cols, dp, s);
    }
    if (type == kF16) return quant_rows<kF16>(x, codes, es, rows, cols, dp, s);
    if (type == kBf16) return quant_rows<kBf16>(x, codes, es, rows, cols, dp, s);
    return quant_rows<kF32>(x, codes, es, rows, cols, dp, s);
}

cudaError_t launch_mx_dequant_rows(const uint32_t* codes, const uint8_t* es, void* w, int64_t rows, int64_t cols,
                                   const DeviceProps& dp, cudaStream_t s) {
    const long long words = cols / 8, items = rows * words, groups = (cols + 127) / 128;
    const long long grid =
        std::min<long long>((items + kThreads - 1) / kThreads, static_cast<long long>(dp.sms) * 8);
    if (items < kIndexLimit)
        return launch(dequant_rows_kernel<unsigned>, grid, s, codes, es, static_cast<uint16_t*>(w), items, words,
                          groups);
    return launch(dequant_rows_kernel<unsigned long long>, grid, s, codes, es, static_cast<uint16_t*>(w), items,
                      words, groups);
}

cudaError_t launch_mx_tile_scales(const uint8_t* src, uint8_t* dst, int64_t rows, int64_t cols, const DeviceProps& dp,
                                  cudaStream_t s) {
    const long long groups = (cols + 127) / 128, items = rows * groups;
    const long long grid =
        std::min<long long>((items + kThreads - 1) / kThreads, static_cast<long long>(dp.sms) * 8);
    return launch(tile_scales_kernel, grid, s, src, dst, items, groups, cols / 32);
}

}  // namespace w4a16
