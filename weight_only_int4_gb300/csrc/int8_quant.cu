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

// A thread block takes a row: each thread holds kPer vectors of 8 elements in
// their own type between the maximum and the codes, so the row is read once.
template <int kType, int kPer>
__global__ void __launch_bounds__(1024) quant_row_kernel(const void* __restrict__ x, int8_t* __restrict__ codes,
                                                         float* __restrict__ scales, int K) {
    __shared__ uint32_t scratch[32];
    const long long row = blockIdx.x;
    const int vecs = K >> 3;
    Vec8<kType> v[kPer];
    float f[8];
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int c = p * blockDim.x + threadIdx.x;
        v[p].zero();
        if (c < vecs) v[p].load_stream(x, row * K + 8ll * c);
    }
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        v[p].widen(f);
        m = magnitude(f, m);
    }
    const RowCodes code(block_max(m, scratch));
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int c = p * blockDim.x + threadIdx.x;
        if (c >= vecs) break;
        v[p].widen(f);
        *reinterpret_cast<uint2*>(codes + row * K + 8ll * c) = code(f);
    }
    if (threadIdx.x == 0) scales[row] = code.scale;
}

// Rows longer than a block holds: read twice, the second time mostly from L2.
template <int kType>
__global__ void __launch_bounds__(1024) quant_long_kernel(const void* __restrict__ x, int8_t* __restrict__ codes,
                                                          float* __restrict__ scales, int K) {
    __shared__ uint32_t scratch[32];
    const long long row = blockIdx.x;
    const int vecs = K >> 3;
    float f[8];
    uint32_t m = 0;
#pragma unroll 4
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
        Vec8<kType> v;
        v.load_stream(x, row * K + 8ll * c);
        v.widen(f);
        m = magnitude(f, m);
    }
    const RowCodes code(block_max(m, scratch));
#pragma unroll 4
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
        Vec8<kType> v;
        v.load_stream(x, row * K + 8ll * c);
        v.widen(f);
        *reinterpret_cast<uint2*>(codes + row * K + 8ll * c) = code(f);
    }
    if (threadIdx.x == 0) scales[row] = code.scale;
}

// A thread takes 8 codes: c * s in FP32, rounded to the output type.
template <int kType, typename Index>
__global__ void __launch_bounds__(256) dequant_kernel(const int8_t* __restrict__ codes,
                                                      const float* __restrict__ scales, void* __restrict__ y,
                                                      Index items, Index vecs) {
    const Index step = static_cast<Index>(static_cast<long long>(gridDim.x) * 256);
    for (Index i = static_cast<Index>(blockIdx.x * 256ll + threadIdx.x); i < items; i += step) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(codes) + i);
        const float s = __ldg(scales + i / vecs);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3)))) * s;
        Vec8<kType> o;
        o.round(f);
        o.store(y, 8ll * i);
    }
}

// Ordinary launches, as in mx_quant.cu.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kern)(Params...), long long blocks, int threads, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

template <int kType>
cudaError_t quantize(const void* x, int8_t* codes, float* scales, long long rows, long long K, cudaStream_t s) {
    const long long vecs = K / 8;
    auto threads = [&](int per) { return static_cast<int>(((vecs + per - 1) / per + 31) / 32 * 32); };
    if (vecs <= 1024) return launch(quant_row_kernel<kType, 1>, rows, threads(1), s, x, codes, scales, K);
    if (vecs <= 2048) return launch(quant_row_kernel<kType, 2>, rows, threads(2), s, x, codes, scales, K);
    if (vecs <= 4096) return launch(quant_row_kernel<kType, 4>, rows, threads(4), s, x, codes, scales, K);
    return launch(quant_long_kernel<kType>, rows, 1024, s, x, codes, scales, K);
}

template <int kType>
cudaError_t dequantize(const int8_t* codes, const float* scales, void* y, long long rows, long long K,
                       const DeviceProps& dp, cudaStream_t s) {
    const long long vecs = K / 8, items = rows * vecs;
    const long long grid = std::min<long long>((items + 255) / 256, static_cast<long long>(dp.sms) * 32);
    if (items < (1ll << 31) - (1ll << 26))
        return launch(dequant_kernel<kType, unsigned>, grid, 256, s, codes, scales, y, items, vecs);
    return launch(dequant_kernel<kType, unsigned long long>, grid, 256, s, codes, scales, y, items, vecs);
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int8_t* codes, float* scales, int64_t rows, int64_t cols, int type,
                                 cudaStream_t s) {
    if (type == kF16) return quantize<kF16>(x, codes, scales, rows, cols, s);
    if (type == kBf16) return quantize<kBf16>(x, codes, scales, rows, cols, s);
    return quantize<kF32>(x, codes, scales, rows, cols, s);
}

cudaError_t launch_int8_dequant(const int8_t* codes, const float* scales, void* y, int64_t rows, int64_t cols,
                                int type, const DeviceProps& dp, cudaStream_t s) {
    if (type == kF16) return dequantize<kF16>(codes, scales, y, rows, cols, dp, s);
    if (type == kBf16) return dequantize<kBf16>(codes, scales, y, rows, cols, dp, s);
    return dequantize<kF32>(codes, scales, y, rows, cols, dp, s);
}

}  // namespace w4a16
