// Product of int8 operands with a scale per row of each,
//
//     y[m, n] = (sum_k a[m, k] b[n, k]) * sa[m] * sb[n].
//
// Rows kernel: four 8-bit products and their 32-bit sum per instruction
// (dp4a), exact.
#include "internal.h"
#include "rowwise.cuh"

#include <algorithm>

namespace w4a16 {
namespace {

enum : int { kF16 = 0, kBf16 = 1, kF32 = 2 };

template <int kOut>
__device__ __forceinline__ void store1(void* y, size_t at, float v) {
    if constexpr (kOut == kF32) static_cast<float*>(y)[at] = v;
    if constexpr (kOut == kBf16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    if constexpr (kOut == kF16) static_cast<__half*>(y)[at] = __float2half_rn(v);
}

__device__ __forceinline__ uint4 load_weights(const int8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ int dot16(uint4 a, uint4 b, int acc) {
    acc = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), acc);
    acc = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), acc);
    acc = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), acc);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), acc);
}

// A warp takes four rows of b and MT of a; each lane 16 bytes of K at a time.
constexpr int kWarps = 8, kRows = 4;

template <int kOut, int MT>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const int8_t* __restrict__ a, const float* __restrict__ sa,
                                                           const int8_t* __restrict__ b, const float* __restrict__ sb,
                                                           void* __restrict__ y, int M, int N, int K) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n0 = (blockIdx.x * static_cast<long long>(kWarps) + warp) * kRows;
    if (n0 >= N) return;
    for (int m0 = blockIdx.y * MT; m0 < M; m0 += gridDim.y * MT) {
        int acc[MT][kRows] = {};
#pragma unroll 2
        for (int k = lane * 16; k < K; k += 512) {
            uint4 w[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) w[r] = load_weights(b + (n0 + r) * K + k);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(a + static_cast<long long>(min(m0 + m, M - 1)) * K + k));
#pragma unroll
                for (int r = 0; r < kRows; ++r) acc[m][r] = dot16(v, w[r], acc[m][r]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int sum = __reduce_add_sync(0xffffffffu, acc[m][r]);
                if (lane == r && m0 + m < M)
                    store1<kOut>(y, static_cast<size_t>(m0 + m) * N + n0 + r,
                                 static_cast<float>(sum) * __ldg(sa + m0 + m) * __ldg(sb + n0 + r));
            }
    }
}

template <int kOut, int MT>
cudaError_t launch_rows(const Int8MatmulArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const long long rows = kWarps * kRows;
    cfg.gridDim = dim3(static_cast<unsigned>((a.N + rows - 1) / rows),
                       static_cast<unsigned>(std::min<long long>((a.M + MT - 1) / MT, 65535)));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, rows_kernel<kOut, MT>, a.a, a.sa, a.b, a.sb, a.y, a.M, a.N, a.K);
}

template <int kOut>
cudaError_t launch_typed(const Int8MatmulArgs& a, cudaStream_t s) {
    if (a.M == 1) return launch_rows<kOut, 1>(a, s);
    if (a.M == 2) return launch_rows<kOut, 2>(a, s);
    if (a.M <= 4) return launch_rows<kOut, 4>(a, s);
    return launch_rows<kOut, 8>(a, s);
}

}  // namespace

size_t int8_matmul_workspace_bytes(int64_t, int64_t, int64_t, const DeviceProps&) { return 0; }

cudaError_t launch_int8_matmul(const Int8MatmulArgs& a, int out_type, void*, const DeviceProps&, cudaStream_t s) {
    if (out_type == kF16) return launch_typed<kF16>(a, s);
    if (out_type == kBf16) return launch_typed<kBf16>(a, s);
    return launch_typed<kF32>(a, s);
}

}  // namespace w4a16
