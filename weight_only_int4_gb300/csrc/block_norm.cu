// The step between two blocks of a transformer, in one pass over its rows:
//
//     u  = h * rsqrt(mean(h^2) + eps) * after        (u = h without `after`)
//     r' = r + scale * gate * u
//     y  = r' * rsqrt(mean(r'^2) + eps) * weight     dense, or int8 codes with a scale per row
//
// A thread block takes a row; each thread holds its elements in registers from
// the first load to the last store, so h and r are read once and r' and y
// written once. All arithmetic is FP32: u and the r' that is normalised are not
// rounded in between; r', y and the scale are rounded once, when they are
// stored. Two or three reductions separate the passes over the registers.
// Bound by HBM bandwidth or, for few rows, by the launch and the reductions.
#include "internal.h"
#include "rowwise.cuh"

namespace w4a16 {
namespace {

using namespace rowwise;

template <int kAct, int kRes, int kPer, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const BlockNormArgs a) {
    __shared__ float scratch[3][32];
    const long long row = blockIdx.x * static_cast<long long>(blockDim.y) + threadIdx.y;
    if (row >= a.T) return;
    const int H = static_cast<int>(a.H), vecs = H >> 3;
    const float inv_h = 1.f / static_cast<float>(H);
    Vec8<kRes> rv[kPer];
    Vec8<kAct> hv[kPer];
    float f[8];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int c = p * blockDim.x + threadIdx.x;
        rv[p].zero();
        hv[p].zero();
        if (c < vecs) {
            rv[p].load_stream(a.residual, row * H + 8ll * c);
            if (a.h) hv[p].load_stream(a.h, row * H + 8ll * c);
        }
    }
    float norm_h = 1.f;
    if (a.after) {
        float sum = 0.f;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            hv[p].widen(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __fmaf_rn(f[i], f[i], sum);
        }
        norm_h = rsqrtf(block_sum(sum, scratch[0]) * inv_h + a.eps);
    }
    float r[kPer][8], sum = 0.f;
    float row_gate = a.scale;
    if (a.gate && a.gate_kind == kGateToken) {
        const uint16_t* p16 = static_cast<const uint16_t*>(a.gate) + row;
        if constexpr (kAct == kF32) row_gate *= __ldg(static_cast<const float*>(a.gate) + row);
        else if constexpr (kAct == kBf16) row_gate *= __uint_as_float(static_cast<uint32_t>(__ldg(p16)) << 16);
        else row_gate *= __half2float(__ushort_as_half(__ldg(p16)));
    }
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int c = p * blockDim.x + threadIdx.x;
        rv[p].widen(r[p]);
        if (c >= vecs || !a.h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __fmaf_rn(r[p][i], r[p][i], sum);
            continue;
        }
        float u[8];
        hv[p].widen(u);
        if (a.after) {
            Vec8<kAct> w;
            w.load_shared(a.after, 8ll * c);
            w.widen(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] *= norm_h * f[i];
        }
        if (a.gate && a.gate_kind != kGateToken) {
            Vec8<kAct> g;
            if (a.gate_kind == kGateChannel) g.load_shared(a.gate, 8ll * c);
            else g.load_stream(a.gate, row * H + 8ll * c);
            g.widen(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[p][i] = __fmaf_rn(row_gate, u[i], r[p][i]);
            sum = __fmaf_rn(r[p][i], r[p][i], sum);
        }
        rv[p].round(r[p]);
        rv[p].store(a.residual_out, row * H + 8ll * c);
    }
    if (!a.weight) return;
    const float norm_r = rsqrtf(block_sum(sum, scratch[1]) * inv_h + a.eps);
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int c = p * blockDim.x + threadIdx.x;
        if (c >= vecs) break;
        Vec8<kAct> w;
        w.load_shared(a.weight, 8ll * c);
        w.widen(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[p][i] *= norm_r * f[i];
        if (a.codes) {
            m = magnitude(r[p], m);
        } else {
            w.round(r[p]);
            w.store(a.y, row * H + 8ll * c);
        }
    }
    if (!a.codes) return;
    const RowCodes code(block_max(m, reinterpret_cast<uint32_t*>(scratch[2])));
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int c = p * blockDim.x + threadIdx.x;
        if (c >= vecs) break;
        *reinterpret_cast<uint2*>(a.codes + row * H + 8ll * c) = code(r[p]);
    }
    if (threadIdx.x == 0) a.code_scales[row] = code.scale;
}

template <int kAct, int kRes>
cudaError_t launch_typed(const BlockNormArgs& a, cudaStream_t s) {
    const Layout l = layout_of(a.H / 8, 4);   // by H alone: a row's sums do not depend on the number of rows
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + l.y - 1) / l.y));
    cfg.blockDim = dim3(static_cast<unsigned>(l.x), static_cast<unsigned>(l.y));
    cfg.stream = s;
    switch (l.per) {
        case 1: return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 1, 1024>, a);
        case 2: return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 2, 1024>, a);
        default: return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 4, 512>, a);
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int act, int res, cudaStream_t s) {
    if (act == kF32) return launch_typed<kF32, kF32>(a, s);
    if (act == kBf16) return res == kF32 ? launch_typed<kBf16, kF32>(a, s) : launch_typed<kBf16, kBf16>(a, s);
    return res == kF32 ? launch_typed<kF16, kF32>(a, s) : launch_typed<kF16, kF16>(a, s);
}

}  // namespace w4a16
