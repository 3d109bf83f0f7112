// Rows of int8 codes with one FP32 scale each, and the way back.
//
//     s[r] = RN(amax / 127),   c[r, k] = RN(127 x[r, k] / amax),   amax = max_k |x[r, k]|
//
// codes decided exactly (rowwise.cuh), ties to even. A row of zeros has scale 0
// and codes 0; a row with an infinity or a NaN has scale NaN and codes 0, so
// every value of it reads as NaN. Each operand is streamed once; bound by HBM
// bandwidth or, for few rows, by the launch.
#include "internal.h"
#include "rowwise.cuh"

#include <algorithm>

namespace w4a16 {
namespace {

using namespace rowwise;

// A thread block takes a row (kWarps: each of its warps one): each thread holds
// kPer vectors of 8 elements in their own type between the maximum and the codes,
// so the row is read once. 43008 x 5376 bf16 99.0 us (7.0 TB/s; 203 with one vector
// per thread, 130 with four), FP32 162.9 (7.1); 2048 x 5376 bf16 7.2 us, 1 x 5376 1.5.
template <int kType, int kPer, int kMaxThreads, bool kWarps = false>
__global__ void __launch_bounds__(kMaxThreads) quant_row_kernel(const void* __restrict__ x, int8_t* __restrict__ codes,
                                                                float* __restrict__ scales, long long rows, int K) {
    __shared__ uint32_t scratch[32];
    const long long row = kWarps ? blockIdx.x * static_cast<long long>(blockDim.y) + threadIdx.y : blockIdx.x;
    if (kWarps && row >= rows) return;
    const int vecs = K >> 3;
    const uint8_t* from = static_cast<const uint8_t*>(x) + row * K * kBytes<kType>;
    int8_t* to = codes + row * K;
    Vec8<kType> v[kPer];
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const uint32_t c = p * blockDim.x + threadIdx.x;
        v[p].zero();
        if (c < vecs) v[p].load_stream(from + c * (8u * kBytes<kType>));
    }
#pragma unroll
    for (int p = 0; p < kPer; ++p) m = raw_magnitude(v[p], m);
    const RowCodes<kType> code(block_max<kWarps>(raw_to_f32<kType>(m), scratch));
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const uint32_t c = p * blockDim.x + threadIdx.x;
        if (c >= vecs) break;
        Pair f[4];
        v[p].widen(f);
        *reinterpret_cast<uint2*>(to + 8u * c) = code(f);
    }
    if (threadIdx.x == 0) scales[row] = code.scale;
}

// Rows longer than a block holds (65536 elements of 16 bits, 32768 of 32): read
// twice, the second time mostly from L2. 2048 x 65552 bf16 103 us (3.9 TB/s; 77 at 65536,
// held in registers), 2048 x 131056 212, FP32 385 (3.5).
template <int kType>
__global__ void __launch_bounds__(1024) quant_long_kernel(const void* __restrict__ x, int8_t* __restrict__ codes,
                                                          float* __restrict__ scales, int K) {
    __shared__ uint32_t scratch[32];
    const long long row = blockIdx.x;
    const int vecs = K >> 3;
    const uint8_t* from = static_cast<const uint8_t*>(x) + row * K * kBytes<kType>;
    uint32_t m = 0;
#pragma unroll 4
    for (int c = threadIdx.x; c < vecs; c += 1024) {
        Vec8<kType> v;
        v.load_stream(from + 8ll * kBytes<kType> * c);
        m = raw_magnitude(v, m);
    }
    const RowCodes<kType> code(block_max<false>(raw_to_f32<kType>(m), scratch));
#pragma unroll 4
    for (int c = threadIdx.x; c < vecs; c += 1024) {
        Pair f[4];
        Vec8<kType> v;
        v.load_stream(from + 8ll * kBytes<kType> * c);
        v.widen(f);
        *reinterpret_cast<uint2*>(codes + row * K + 8ll * c) = code(f);
    }
    if (threadIdx.x == 0) scales[row] = code.scale;
}

// A thread takes 8 codes at a time, four such loads in flight: c * s in FP32,
// rounded to the output type. 43008 x 5376 to bf16 or fp16 112 us (6.2 TB/s), to FP32 265
// (4.4).
template <int kType, typename Index>
__global__ void __launch_bounds__(256) dequant_kernel(const int8_t* __restrict__ codes,
                                                      const float* __restrict__ scales, void* __restrict__ y,
                                                      Index items, Index vecs) {
    constexpr int kUnroll = 4;
    const Index step = static_cast<Index>(static_cast<long long>(gridDim.x) * 256);
    for (Index i0 = static_cast<Index>(blockIdx.x * 256ll + threadIdx.x); i0 < items; i0 += step * kUnroll) {
        uint2 q[kUnroll];
        float s[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const Index i = i0 + step * u;
            if (i < items) {
                q[u] = __ldg(reinterpret_cast<const uint2*>(codes) + i);
                s[u] = __ldg(scales + i / vecs);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const Index i = i0 + step * u;
            if (i >= items) break;
            Pair f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = (j < 2 ? q[u].x : q[u].y) >> (16 * (j & 1));
                f[j] = mul2(pair(static_cast<float>(static_cast<int8_t>(w)),
                                 static_cast<float>(static_cast<int8_t>(w >> 8))), both(s[u]));
            }
            Vec8<kType> o;
            o.round(f);
            o.store(static_cast<uint8_t*>(y) + 8ll * kBytes<kType> * i);
        }
    }
}

// Ordinary launches, as in mx_quant.cu.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kern)(Params...), long long blocks, dim3 threads, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = threads;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

template <int kType>
cudaError_t quantize(const void* x, int8_t* codes, float* scales, long long rows, long long K, const DeviceProps& dp,
                     cudaStream_t s) {
    constexpr int kMost = kType == kF32 ? 4 : 8;   // vectors of 32 registers in all
    const long long vecs = K / 8;
    if (vecs > 1024 * kMost) return launch(quant_long_kernel<kType>, rows, dim3(1024), s, x, codes, scales, K);
    Layout l = layout_of(vecs, kMost);
    if (rows <= 2ll * dp.sms) {   // the latency of a row is what counts: as many threads as there are
        l.per = vecs <= 1024 ? 1 : vecs <= 2048 ? std::min(4, kMost) : l.per;
        l.x = static_cast<int>(((vecs + l.per - 1) / l.per + 31) / 32 * 32);
        l.y = 1;
    }
    const dim3 threads(static_cast<unsigned>(l.x), static_cast<unsigned>(l.y));
    const long long blocks = (rows + l.y - 1) / l.y;
    if (l.per == kMost && l.x > 512) {   // long rows: twice the vectors
        const dim3 half(static_cast<unsigned>((vecs + 2 * kMost - 1) / (2 * kMost) + 31) / 32 * 32);
        return launch(quant_row_kernel<kType, 2 * kMost, 512>, blocks, half, s, x, codes, scales, rows, K);
    }
    if (l.y > 1)
        switch (l.per) {
            case 1: return launch(quant_row_kernel<kType, 1, 128, true>, blocks, threads, s, x, codes, scales, rows, K);
            case 2: return launch(quant_row_kernel<kType, 2, 128, true>, blocks, threads, s, x, codes, scales, rows, K);
            case 4: return launch(quant_row_kernel<kType, 4, 128, true>, blocks, threads, s, x, codes, scales, rows, K);
            default:
                return launch(quant_row_kernel<kType, kMost, 128, true>, blocks, threads, s, x, codes, scales, rows, K);
        }
    if constexpr (kMost == 8)
        if (l.per == 8) return launch(quant_row_kernel<kType, 8, 512>, blocks, threads, s, x, codes, scales, rows, K);
    if (l.per == 1) return launch(quant_row_kernel<kType, 1, 1024>, blocks, threads, s, x, codes, scales, rows, K);
    return launch(quant_row_kernel<kType, 4, 512>, blocks, threads, s, x, codes, scales, rows, K);
}

template <int kType>
cudaError_t dequantize(const int8_t* codes, const float* scales, void* y, long long rows, long long K,
                       const DeviceProps& dp, cudaStream_t s) {
    const long long vecs = K / 8, items = rows * vecs;
    const long long grid = std::min<long long>((items + 255) / 256, static_cast<long long>(dp.sms) * 16);
    if (items < (1ll << 31) - (1ll << 26))
        return launch(dequant_kernel<kType, unsigned>, grid, dim3(256), s, codes, scales, y, items, vecs);
    return launch(dequant_kernel<kType, unsigned long long>, grid, dim3(256), s, codes, scales, y, items, vecs);
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int8_t* codes, float* scales, int64_t rows, int64_t cols, int type,
                                 const DeviceProps& dp, cudaStream_t s) {
    if (type == kF16) return quantize<kF16>(x, codes, scales, rows, cols, dp, s);
    if (type == kBf16) return quantize<kBf16>(x, codes, scales, rows, cols, dp, s);
    return quantize<kF32>(x, codes, scales, rows, cols, dp, s);
}

cudaError_t launch_int8_dequant(const int8_t* codes, const float* scales, void* y, int64_t rows, int64_t cols,
                                int type, const DeviceProps& dp, cudaStream_t s) {
    if (type == kF16) return dequantize<kF16>(codes, scales, y, rows, cols, dp, s);
    if (type == kBf16) return dequantize<kBf16>(codes, scales, y, rows, cols, dp, s);
    return dequantize<kF32>(codes, scales, y, rows, cols, dp, s);
}

}  // namespace w4a16
