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
// stored. Both norms are formed in the order written: h * after or rsqrt * weight
// first would leave the FP32 range where the formula does not (zero rows under
// large weights would give NaN). Up to three reductions separate the passes over the registers.
//
// What bounds it: HBM for many rows (8192 x 5376, bf16, norms on both sides and a
// gate: 56.1 us, 6.3 TB/s; 8192 x 5376 with an FP32 residual 83.5 us, 6.3). In between,
// latencies and issue slots: blocks start together, wait for their loads together and then
// compute together (2048 x 5376 to int8 17.4 us where the bytes take 11.5, some 26
// instructions an element). One row: 3.4 us, launch and three reductions. Bulk copies of
// the next rows into a ring of shared memory by persistent blocks were slower, 80 us
// instead of 59 then: they take registers, and so rows in flight.
#include "internal.h"
#include "rowwise.cuh"

namespace w4a16 {
namespace {

using namespace rowwise;

// A row per block, or (kWarps) per warp, blockDim.y rows to a block. Vectors per thread, and threads x blocks per SM that
// the registers are held to (us, bf16, 44 M elements):
//   bf16 residual, norms on both sides and a gate: 3 vectors, 384 x 3 (56 registers): 56.3 at H = 5120, 57.8 at 8192, 60.5 at
//     9040; 3 vectors, 512 x 2 (58): 57.2, 66.2, 66.0; 4 vectors, 512 x 2 (64): 59.8, 60.6, 65.7; with 2 vectors 67.5 at
//     5376, with 1 88.8. Rows of more than 9216: 3 vectors, 512 x 2, 59.9 at 12288, 4 65.8;
//   FP32 residual, the same / to int8: 2 vectors 82.0 / 79.0 at 4096, 92.6 / 91.9 at 6912, 117 / 121 at 11008; 3 vectors 87.1 /
//     78.5, 89.0 / 79.6, 95.4 / 86.9. Rows of more than 12288: 4 vectors, 512 x 2 (64, 212 bytes of spills) 125 / 107 at 12304,
//     112 / 100 at 16384; without spills 4 vectors, 512 x 1 (114) 129 / 130, 120 / 117; 3 vectors, 704 x 1 (74) 127 / 126, 115 /
//     116; 2 vectors, 1024 (60) 129 / 130, 117 / 119. One row of 16384 alone 7.0 us; 6.1, 6.1, 6.4 in the others.
//   FP32 activations: 2 vectors, up to 1024 threads; 8192 x 8192 199 us, 498 x 13568 to int8 27.5.
// Kernels held to 56 registers spill 8 bytes (bf16 residual) or 28 (FP32), 4 vectors with a 16-bit residual 20.
template <int kAct, int kRes, int kPer, int kMaxThreads, int kBlocks, bool kWarps>
__global__ void __launch_bounds__(kMaxThreads, kBlocks)
block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
    __shared__ __align__(16) float scratch[3][32];
    const long long row = kWarps ? blockIdx.x * static_cast<long long>(blockDim.y) + threadIdx.y : blockIdx.x;
    if (kWarps && row >= a.T) return;
    const int H = static_cast<int>(a.H);
    const uint32_t vecs = static_cast<uint32_t>(H) >> 3;
    const float inv_h = 1.f / static_cast<float>(H);
    constexpr uint32_t kActVec = 8 * kBytes<kAct>, kResVec = 8 * kBytes<kRes>;
    auto bytes = [](const void* p) { return static_cast<const uint8_t*>(p); };
    const uint8_t* h_row = bytes(a.h) + row * H * kBytes<kAct>;
    const uint8_t* r_row = bytes(a.residual) + row * H * kBytes<kRes>;
    uint8_t* out_row = static_cast<uint8_t*>(a.residual_out) + row * H * kBytes<kRes>;
    // A thread past the row's end holds zeros, which change neither a sum nor the largest magnitude; it reads vectors that
    // exist and stores nothing.
    uint32_t at[kPer];
    bool mine[kPer];
    Vec8<kRes> rv[kPer];
    Vec8<kAct> hv[kPer];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const uint32_t c = p * blockDim.x + threadIdx.x;
        mine[p] = c < vecs;
        at[p] = min(c, vecs - 1u);
        rv[p].zero();
        hv[p].zero();
        if (mine[p]) {
            rv[p].load_stream(r_row + at[p] * kResVec);
            if (a.h) hv[p].load_stream(h_row + at[p] * kActVec);
        }
    }
    Pair r[kPer][4];   // u, then r', then y
    if (a.h) {
        Pair by_gate = both(a.scale);
        if (a.after) {
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < kPer; ++p) sum = add_squares(hv[p], sum);
            const Pair by_h = both(rsqrtf(block_sum<kWarps>(sum.x + sum.y, scratch[0]) * inv_h + a.eps));
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
                Vec8<kAct> w;
                w.load_shared(bytes(a.after) + at[p] * kActVec);
                Pair f[4];
                hv[p].widen(r[p]);
                w.widen(f);
#pragma unroll
                for (int i = 0; i < 4; ++i) r[p][i] = mul2(mul2(r[p][i], by_h), f[i]);
            }
        } else {
#pragma unroll
            for (int p = 0; p < kPer; ++p) hv[p].widen(r[p]);
        }
        if (a.gate) {
            if (a.gate_kind == kGateToken) {
                float g;
                const uint16_t* p16 = static_cast<const uint16_t*>(a.gate) + row;
                if constexpr (kAct == kF32) g = __ldg(static_cast<const float*>(a.gate) + row);
                else if constexpr (kAct == kBf16) g = __uint_as_float(static_cast<uint32_t>(__ldg(p16)) << 16);
                else g = __half2float(__ushort_as_half(__ldg(p16)));
                by_gate = both(a.scale * g);
            } else {
                const uint8_t* gate_row = bytes(a.gate) + (a.gate_kind == kGateElement ? row * H * kBytes<kAct> : 0);
#pragma unroll
                for (int p = 0; p < kPer; ++p) {
                    Vec8<kAct> g;
                    Pair f[4];
                    g.load_shared(gate_row + at[p] * kActVec);
                    g.widen(f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[p][i] = mul2(r[p][i], f[i]);
                }
            }
        }
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            Pair f[4];
            rv[p].widen(f);
#pragma unroll
            for (int i = 0; i < 4; ++i) r[p][i] = fma2(by_gate, r[p][i], f[i]);
            rv[p].round(r[p]);
            if (mine[p]) rv[p].store(out_row + at[p] * kResVec);
        }
    } else {
#pragma unroll
        for (int p = 0; p < kPer; ++p) rv[p].widen(r[p]);
    }
    if (!a.weight) return;
    Pair sum = both(0.f);
#pragma unroll
    for (int p = 0; p < kPer; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma2(r[p][i], r[p][i], sum);
    const float2 t = parts(sum);
    const Pair by_r = both(rsqrtf(block_sum<kWarps>(t.x + t.y, scratch[1]) * inv_h + a.eps));
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        Vec8<kAct> w;
        Pair f[4];
        w.load_shared(bytes(a.weight) + at[p] * kActVec);
        w.widen(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[p][i] = mul2(mul2(r[p][i], by_r), f[i]);
    }
    if (!a.codes) {
        uint8_t* y_row = static_cast<uint8_t*>(a.y) + row * H * kBytes<kAct>;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            Vec8<kAct> w;
            w.round(r[p]);
            if (mine[p]) w.store(y_row + at[p] * kActVec);
        }
        return;
    }
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < kPer; ++p) m = magnitude(r[p], m);
    int8_t* codes_row = a.codes + row * H;
    const RowCodes<kF32> code(block_max<kWarps>(m, reinterpret_cast<uint32_t*>(scratch[2])));
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const uint2 c = code(r[p]);
        if (mine[p]) *reinterpret_cast<uint2*>(codes_row + 8u * at[p]) = c;
    }
    if (threadIdx.x == 0) a.code_scales[row] = code.scale;
}

template <int kAct, int kRes>
cudaError_t launch_typed(const BlockNormArgs& a, cudaStream_t s) {
    // by H alone: a row's sums do not depend on the number of rows
    const long long vecs = a.H / 8;
    const Layout l = layout_of(vecs, kRes == kF32 ? 2 : 4);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + l.y - 1) / l.y));
    cfg.blockDim = dim3(static_cast<unsigned>(l.x), static_cast<unsigned>(l.y));
    cfg.stream = s;
    if (l.y > 1) {
        if (l.per == 1) return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 1, 128, 0, true>, a);
        if (l.per == 2) return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 2, 128, 0, true>, a);
        if constexpr (kRes != kF32) return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 4, 128, 0, true>, a);
    }
    [[maybe_unused]] auto threads = [&](int per) { return static_cast<unsigned>((vecs + per - 1) / per + 31) / 32 * 32; };
    if constexpr (kRes == kF32) {
        if (kAct == kF32 || a.H < 6144)
            return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 2, 1024, 0, false>, a);
    }
    if constexpr (kAct != kF32) {
        if (a.H > 12288) {
            cfg.blockDim.x = threads(4);
            return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 4, 512, 2, false>, a);
        }
        cfg.blockDim.x = threads(3);
        if (cfg.blockDim.x > 384) return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 3, 512, 2, false>, a);
        return cudaLaunchKernelEx(&cfg, block_norm_kernel<kAct, kRes, 3, 384, 3, false>, a);
    }
    return cudaErrorInvalidValue;   // not reached
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int act, int res, cudaStream_t s) {
    if (act == kF32) return launch_typed<kF32, kF32>(a, s);
    if (act == kBf16) return res == kF32 ? launch_typed<kBf16, kF32>(a, s) : launch_typed<kBf16, kBf16>(a, s);
    return res == kF32 ? launch_typed<kF16, kF32>(a, s) : launch_typed<kF16, kF16>(a, s);
}

}  // namespace w4a16
