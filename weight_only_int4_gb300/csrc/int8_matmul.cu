// Product of int8 operands with a scale per row of each,
//
//     y[m, n] = (sum_k a[m, k] b[n, k]) * sa[m] * sb[n].
//
// sm_103a's tcgen05.mma has no integer kind, and its warp-level int8 product
// (mma.sync) runs at 158 Top/s, a quarter of the warp-level fp16 one's 604
// (measured), so the codes go through the fp16 tcgen05.mma: a code is a whole number of at most 8 bits, exact in
// fp16, a product exact in FP32, and the FP32 sum exact while every partial sum
// stays within 2^24. The weights b, which every call streams, are widened on the way from
// shared memory to tensor memory, where the MMA takes its first operand from:
// they cross HBM, L2 and shared memory as single bytes. The activations a are
// widened in the kernel too (tiles of up to 64 rows) or to fp16 in the workspace by a
// kernel of their own before it.
//
// Three kernels:
//   rows    few rows of a: dot products of four bytes (dp4a), exact in 32 bits;
//           streams b. The instruction's rate (about 18 lanes a cycle and SM, measured)
//           bounds it from four rows on.
//   tiles   128 rows of b against 16..128 rows of a per tile; whole tiles, a cluster
//           per tile, or tiles shared between CTAs by (tile, K step) units.
//   pair    256 rows of b against up to 256 rows of a on CTA pairs (cta_group::2).
//
// Every mbarrier wait is bounded (about two seconds). On expiry the kernel
// records the timeout in a device word, raises the abort flag, every role
// stops, copies and MMAs in flight are waited for (bounded), tensor memory is
// freed and the kernel returns.
#include "internal.h"
#include "rowwise.cuh"
#include "tmap.h"

#include <algorithm>
#include <atomic>

namespace w4a16 {

__device__ unsigned int g_int8_matmul_error = 0;

namespace {

enum : int { kF16 = 0, kBf16 = 1, kF32 = 2 };

constexpr int kStepK = 128;                  // elements of K per step: one 128-byte-swizzled row of codes
constexpr uint32_t kOpCols = kStepK / 2;     // tensor-memory columns of a step's widened weights
constexpr int kEpiWarp0 = 4;
constexpr unsigned long long kWaitLimitCycles = 4000000000ull;   // ~2 s at 2 GHz
constexpr unsigned int kErrTimeout = 9u;

// Abort flag of this CTA; in a pair a timeout raises the peer's flag too.
struct Abort {
    volatile int* flag;
    uint32_t addr;
    uint32_t peer;   // cluster rank of the peer, or ~0
};

__device__ __noinline__ bool give_up(const Abort& ab) {
    *ab.flag = 1;
    if (ab.peer != ~0u) st_cluster_u32(ab.addr, ab.peer, 1u);
    atomicOr(&g_int8_matmul_error, 1u << kErrTimeout);
    return false;
}

// kRelaxed: the phase is completed by relaxed arrivals from the pair's CTAs.
template <bool kRelaxed = false>
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
    return kRelaxed ? mbar_try_wait_relaxed(bar, parity) : mbar_try_wait(bar, parity);
}

template <bool kRelaxed = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Abort& ab) {
    if (try_bar<kRelaxed>(bar, parity)) return true;
    const unsigned long long t0 = clock64();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (try_bar<kRelaxed>(bar, parity)) return true;
        if (*ab.flag) return false;
        if (clock64() - t0 > kWaitLimitCycles) return give_up(ab);
    }
}

// For a converged warp that goes on together: one lane polls and a vote spreads
// the verdict, so the operands of the tensor-core instructions that follow stay
// in uniform registers.
template <bool kRelaxed = false>
__device__ __forceinline__ bool uniform_wait_bar(uint32_t bar, uint32_t parity, const Abort& ab, bool leader) {
    bool done = true;
    if (leader) done = try_bar<kRelaxed>(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    bool ok = true;
    if (leader) ok = wait_bar<kRelaxed>(bar, parity, ab);
    return __all_sync(0xffffffffu, ok);
}

// Several warps go on together once their first thread has seen up to three
// phases complete, in this order: named barrier `id` spreads its verdict and orders
// the others' accesses after its acquires. One thread polls, not one per warp: polls
// take issue slots and shared-memory cycles from the warps at work (128-row tiles, 16
// rows of a, steps of K measured at 0.47 us with 24 warps polling, 0.39 us so).
__device__ __forceinline__ bool group_wait(int id, int threads, bool first, const Abort& ab, uint32_t bar0,
                                           uint32_t parity0, uint32_t bar1 = 0u, uint32_t parity1 = 0u,
                                           uint32_t bar2 = 0u, uint32_t parity2 = 0u) {
    int ok = 1;
    if (first)
        ok = wait_bar(bar0, parity0, ab) && (bar1 == 0u || wait_bar(bar1, parity1, ab)) &&
             (bar2 == 0u || wait_bar(bar2, parity2, ab));
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %0, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "+r"(ok)
        : "r"(id), "r"(threads)
        : "memory");
    return ok != 0;
}

template <int kOut>
__device__ __forceinline__ void store1(void* y, size_t at, float v) {
    if constexpr (kOut == kF32) static_cast<float*>(y)[at] = v;
    if constexpr (kOut == kBf16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    if constexpr (kOut == kF16) static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// Four codes (offset by 128: bytes 0..255) to two pairs of fp16 values: 1024 + u
// is the fp16 bit pattern 0x6400 | u, and the subtraction of 1152 is exact.
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = codes ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(prmt(u, 0x64646464u, 0x4140u)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(prmt(u, 0x64646464u, 0x4342u)), "r"(0x64806480u));
}

// Half a row (64 codes) of a 128-byte-swizzled tile of codes, widened, to 32 columns of tensor memory.
__device__ __forceinline__ void widen_half_row(uint32_t tile, int row, int half, uint32_t taddr) {
    uint32_t o[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t at = tile + row * 128 + (((4 * half + i) ^ (row & 7)) << 4);
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
#pragma unroll
        for (int j = 0; j < 4; ++j) widen4(w[j], o[8 * i + 2 * j], o[8 * i + 2 * j + 1]);
    }
    tmem_st_32x32b_x32(taddr, o);
}

// 16 codes of a 128-byte-swizzled tile [rows x 128] widened to the fp16 operand tile: two boxes of 64 columns, `box`
// bytes each, 128-byte swizzle. Piece i of the tile's 8 per row: eight lanes take half a row each of two neighbours, so
// that their stores reach different banks (their loads collide in pairs).
__device__ __forceinline__ void widen_piece(uint32_t codes, uint32_t wide, uint32_t box, int i) {
    const int c = i & 3, half = (i >> 3) & 1, r = ((i >> 4) << 1) | ((i >> 2) & 1);
    uint32_t w[4], o[8];
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(codes + r * 128 + (((4 * half + c) ^ (r & 7)) << 4)));
#pragma unroll
    for (int j = 0; j < 4; ++j) widen4(w[j], o[2 * j], o[2 * j + 1]);
    const uint32_t row = wide + half * box + r * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row + (((2 * c + h) ^ (r & 7)) << 4)), "r"(o[4 * h]),
                     "r"(o[4 * h + 1]), "r"(o[4 * h + 2]), "r"(o[4 * h + 3])
                     : "memory");
}

// MMAs (16 deep) of a K step.
__device__ __forceinline__ int step_mmas(int K, int kt) { return min(kStepK / 16, (K - kt * kStepK + 15) >> 4); }

// ---------------------------------------------------------------------------
// activations to fp16
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) widen_kernel(const int8_t* __restrict__ a, __half* __restrict__ out,
                                                    long long items) {
    const long long step = gridDim.x * 256ll;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < items; i += step) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(a) + i);
        uint4 o;
        widen4(q.x, o.x, o.y);
        widen4(q.y, o.z, o.w);
        reinterpret_cast<uint4*>(out)[i] = o;
    }
}

// ---------------------------------------------------------------------------
// few rows of a
// ---------------------------------------------------------------------------
namespace rows {

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

// A warp takes kRows rows of b and MT of a, each lane 16 bytes of K at a time,
// the loads of kDeep such chunks in flight. Blocks are small and many, so that the last
// ones leave few SMs idle; registers are left to the loads (one resident block
// asked for: with the compiler's own choice 39.1 us instead of 34.6 at
// 1 x 43008 x 5376, less in flight).
// 1 x 43008 x 5376 34.5 us (6.7 TB/s), 4 rows 39.3; 1 x 2048 x 2048 1.9; 1 x 4096 x 131056 80.2 (6.7 TB/s). With few
// rows of b a warp still walks all of K: 8 x 264 x 8208 9.9 us, 4 x 264 x 131056 99 (the bytes take 5).
constexpr int kWarps = 4;

template <int kOut, int MT, int kRows, int kDeep>
__global__ void __launch_bounds__(kWarps * 32, 1) rows_kernel(const int8_t* __restrict__ a, const float* __restrict__ sa,
                                                              const int8_t* __restrict__ b, const float* __restrict__ sb,
                                                              void* __restrict__ y, int M, int N, int K) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n0 = (blockIdx.x * static_cast<long long>(kWarps) + warp) * kRows;
    if (n0 >= N) return;
    const int m0 = blockIdx.y * MT;
    int acc[MT][kRows] = {};
#pragma unroll kDeep
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

template <int kOut, int MT, int kRows, int kDeep>
cudaError_t launch_mt(const Int8MatmulArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    constexpr long long kBlock = kWarps * kRows;
    cfg.gridDim = dim3(static_cast<unsigned>((a.N + kBlock - 1) / kBlock), static_cast<unsigned>((a.M + MT - 1) / MT));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, rows_kernel<kOut, MT, kRows, kDeep>, a.a, a.sa, a.b, a.sb, a.y, a.M, a.N, a.K);
}

// Rows of b per warp and chunks in flight (us, 1 x 43008 x 5376, 1 x 5376 x 21504 / 2 and 4 x 43008 x 5376): 2 rows, 4
// chunks 34.5, 18.1 / 38.9, 53.7; 4 rows, 2 chunks 34.4, 20.1 / 35.5, 38.7.
template <int kOut>
cudaError_t launch(const Int8MatmulArgs& a, cudaStream_t s) {
    switch (a.M) {
        case 1: return launch_mt<kOut, 1, 2, 4>(a, s);
        case 2: return launch_mt<kOut, 2, 4, 2>(a, s);
        case 3: return launch_mt<kOut, 3, 4, 2>(a, s);
        case 4: return launch_mt<kOut, 4, 4, 2>(a, s);
        case 5:
        case 6: return launch_mt<kOut, 6, 4, 2>(a, s);
        default: return launch_mt<kOut, 8, 4, 2>(a, s);
    }
}

}  // namespace rows

// ---------------------------------------------------------------------------
// 128 rows of b against 16..128 rows of a
// ---------------------------------------------------------------------------
// Warp roles, one CTA per SM:
//   warps 0, 3   producers: per K step TMA brings the tile's codes [128 x 128]
//                and MP rows of a, as codes (up to 64 rows, beside them) or
//                widened before (128 rows: in two 64-column boxes, warp 3), all with
//                the 128-byte swizzle
//   warps 12..27 four groups, steps in turn, widen the codes of b into an operand
//                stage of tensor memory (thread = row of b = lane) and those of a
//                into an operand tile in shared memory
//   warp 1       issues the step's MMAs (M = 128, N = MP, A from tensor memory)
//                into one of two accumulators
//   warps 4..11  epilogue, two warps per lane quarter, half the rows of a each
//   warp 2       tensor memory
// Three ways to hand out the work:
//   whole tiles, one or more per CTA;
//   split > 1: a cluster of `split` CTAs per tile, each a part of K; the parts are
//     added from the CTAs' shared memory, in the order of K;
//   share: with more tiles than CTAs, equal ranges of (tile, K step) units, tile by
//     tile. A tile that lies in two CTAs' ranges is finished by the later of them,
//     which adds the two FP32 parts from global memory, the lower CTA's first.
// All three are deterministic.
//
// 64 x 16384 x 5376 23.4 us, 16 x 43008 x 5376 44.5, 64 rows 52.4, 128 60.9; K of any length:
// 64 x 4096 x 65536 60.4. From K = 2688 to 21504, a step and what does not go with K take
//   one tile to a CTA (N = 16384)    0.37 to 0.41 us and 5 to 7 us with 16 rows, 0.39 to 0.41 and 6 to 7 with 64;
//   units shared (N = 43008)         0.36 to 0.38 and 9 to 12 with 16 rows, 0.37 to 0.39 and 11 to 15 with 32, 0.40 to
//                                    0.43 and 12 to 16 with 64, 0.41 to 0.44 and 18 to 23 with 128, the kernel that
//                                    widens them included.
// HBM alone: 0.37 us a step for 152 CTAs, 0.31 for the 128 that N = 16384 gives a tile. Sharing costs some 5 us over whole
// tiles, parts in global memory and their joins, and more with more rows. 72 registers a thread, 4 to 12 bytes of spills
// with 32 rows and more.
namespace tiles {

constexpr int BN = 128;
constexpr int kThreads = 896;
constexpr int kEpiWarps = 8, kWidenWarp0 = 12, kGroups = 4, kGroupWarps = 4;
constexpr size_t kSlotFloats = 128 * 128;   // partial tile, [row of a][row of b]
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxSplit = 8;

template <int MP>
struct Cfg {
    // Up to 64 rows of a are widened here, by every CTA for itself: no kernel before this one, and half the bytes from
    // L2. With 128 rows shared memory would have to carry more than the step's loads leave it time for.
    static constexpr bool kInline = MP <= 64;
    // Rows of a that are widened here share the stages of b's codes; those that came widened have stages of their own that go
    // by the operand's and are refilled from L2.
    static constexpr int kStages = MP == 16 ? 11 : MP == 32 ? 9 : 6;
    static constexpr int kOpStages = 4, kXStages = kInline ? kStages : kOpStages;
    static constexpr uint32_t kWBytes = BN * kStepK;
    static constexpr uint32_t kXBytes = MP * kStepK * (kInline ? 1 : 2);   // rows of a as they are loaded
    static constexpr uint32_t kWideBytes = MP * kStepK * 2, kBox = kWideBytes / 2;
    static constexpr uint32_t kXAt = kStages * kWBytes, kWideAt = kXAt + kXStages * kXBytes;
    static constexpr uint32_t kRingBytes = kWideAt + (kInline ? kOpStages * kWideBytes : 0);
    static constexpr uint32_t kAccCols = MP < 32 ? 32 : MP;   // the epilogue reads up to 32 columns at a time
    static constexpr uint32_t kOpCol0 = 2 * kAccCols;
    static_assert(kOpCol0 + kOpStages * kOpCols <= kTmemCols, "tensor memory budget");
    // A group takes codes from stages that other groups used in between. It waits for its operand stage first: then the
    // MMAs of kOpStages steps before have retired, every step up to there had been widened, and the phase of the code
    // stage that it skipped is complete.
    static_assert(kStages >= kOpStages && kOpStages % kGroups == 0, "no group waits past an open phase");
    static_assert(kXBytes % 1024 == 0 && kWideBytes % 1024 == 0, "operand tiles stay 1024-byte aligned");
};

template <int MP>
struct __align__(8) Barriers {
    uint64_t full[Cfg<MP>::kStages];        // codes landed (kInline: of both)
    uint64_t empty[Cfg<MP>::kStages];       // widened
    uint64_t xfull[Cfg<MP>::kOpStages];     // rows of a that came widened landed; free with the operand stage
    uint64_t afull[Cfg<MP>::kOpStages];     // operand stage written
    uint64_t aempty[Cfg<MP>::kOpStages];    // MMAs that read it retired
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int last[2];
};
template <int MP>
constexpr size_t smem_bytes() {
    return 1024 + Cfg<MP>::kRingBytes + sizeof(Barriers<MP>);
}

struct Work {
    int split;       // CTAs of a cluster per tile
    int share;       // units shared
    int each, more;  // units (share) or tiles per CTA, and how many of the first CTAs take one more
};

template <int kOut, int MP>
__global__ void __launch_bounds__(kThreads, 1)
tiles_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
             const float* __restrict__ sa, const float* __restrict__ sb, void* __restrict__ y, int M, int N, int K,
             int ld, const Work work, float* __restrict__ partials, uint32_t* __restrict__ tickets) {
    using C = Cfg<MP>;
    constexpr int S = C::kStages, A = C::kOpStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Barriers<MP>* bars = reinterpret_cast<Barriers<MP>*>(smem + C::kRingBytes);
    const uint32_t base = smem_u32(smem);
    auto st_w = [&](int s) { return base + s * C::kWBytes; };
    auto st_x = [&](int s) { return base + C::kXAt + s * C::kXBytes; };
    auto st_wide = [&](int s) { return base + C::kWideAt + s * C::kWideBytes; };   // kInline

    // split > 1: this CTA's part, [row of a][128], once the ring is idle
    float* parts = reinterpret_cast<float*>(smem);
    static_assert(MP * 128 * 4 <= C::kRingBytes, "a part fits the ring");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_m = (M + MP - 1) / MP;
    const int kt_total = (K + kStepK - 1) / kStepK;
    // this CTA's units
    const int split = work.split, share = work.share, b = blockIdx.x;
    const int part_k = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    int u_begin, u_end;
    if (split > 1) {
        const int first = b / split * kt_total;
        u_begin = first + part_k * kt_total / split;
        u_end = first + (part_k + 1) * kt_total / split;
    } else {
        const int scale = share ? 1 : kt_total;
        u_begin = (b * work.each + min(b, work.more)) * scale;
        u_end = u_begin + (work.each + (b < work.more ? 1 : 0)) * scale;
    }
    const int t_begin = u_begin / kt_total, k_begin = u_begin - t_begin * kt_total, steps = u_end - u_begin;
    const Abort ab{&bars->abort, 0u, ~0u};

    // A producer's place, kept from step to step: its divisions would be on the way of every refill.
    int at_k = k_begin, at_t = t_begin, at_m = t_begin % num_m * MP, at_n = t_begin / num_m * BN;
    auto advance = [&]() {
        if (++at_k < kt_total) return;
        at_k = 0;
        ++at_t;
        at_m = at_t % num_m * MP;
        at_n = at_t / num_m * BN;
    };
    auto feed = [&](int s) {
        const uint32_t fb = smem_u32(&bars->full[s]);
        mbar_arrive_expect_tx(fb, C::kWBytes + (C::kInline ? C::kXBytes : 0u));
        tma_load_2d(st_w(s), &tw, at_k * kStepK, at_n, fb);
        if (C::kInline) tma_load_2d(st_x(s), &tx, at_k * kStepK, at_m, fb);
        advance();
    };
    auto feed_wide = [&](int s) {
        const uint32_t fb = smem_u32(&bars->xfull[s]);
        mbar_arrive_expect_tx(fb, C::kXBytes);
        tma_load_2d(st_x(s), &tx, at_k * kStepK, at_m, fb);
        tma_load_2d(st_x(s) + C::kBox, &tx, at_k * kStepK + 64, at_m, fb);
        advance();
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), kGroupWarps);
        }
        for (int s = 0; s < A; ++s) {
            mbar_init(smem_u32(&bars->xfull[s]), 1);
            mbar_init(smem_u32(&bars->afull[s]), kGroupWarps);
            mbar_init(smem_u32(&bars->aempty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&bars->tfull[a]), 1);
            mbar_init(smem_u32(&bars->tempty[a]), kEpiWarps);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
        fence_proxy_async_smem();   // this thread's copies complete on the barriers before any other synchronisation
        // the rings are filled before the other warps are ready
        for (int s = 0; s < min(S, steps); ++s) feed(s);
    }
    if (warp == 2) tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 0 || (!C::kInline && warp == 3)) {
        // ------------------------------------------------------------ producers: codes (warp 0), widened rows (warp 3)
        if (lane == 0) {
            const bool wide = warp == 3;
            const int ring = wide ? A : S;
            const uint32_t free = smem_u32(wide ? &bars->aempty[0] : &bars->empty[0]);
            uint32_t parity = wide ? 1u : 0u;
            int s = 0, i = wide ? 0 : S;   // codes: the ring has been filled
            for (; i < steps; ++i) {
                if (!wait_bar(free + 8 * s, parity, ab)) break;
                if (wide) feed_wide(s);
                else feed(s);
                if (++s == ring) s = 0, parity ^= 1u;
            }
            drain_ring(wide ? bars->xfull : bars->full, ring, min(i, steps));
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t kIdesc = umma_idesc_f16(BN, MP, false);
        const bool leader = elect_one();
        const uint64_t desc_x = sw128_kmajor_desc(C::kInline ? st_wide(0) : st_x(0));
        const uint32_t bar_afull = smem_u32(&bars->afull[0]), bar_aempty = smem_u32(&bars->aempty[0]);
        int seg = 0;
        uint32_t committed = 0;   // steps
        bool ok = true;
        for (int u = u_begin, k0 = k_begin; u < u_end && ok; ++seg, k0 = 0) {
            const int k1 = min(kt_total, k0 + (u_end - u));
            const int acc = seg & 1;
            if (!uniform_wait_bar(smem_u32(&bars->tempty[acc]), ((seg >> 1) & 1) ^ 1, ab, leader)) {
                ok = false;
                break;
            }
            const uint32_t d = tmem + acc * C::kAccCols;
            for (int kt = k0; kt < k1; ++kt) {
                // the group that wrote the stage had waited for the step's rows of a too
                const uint32_t as = committed % A;
                if (!uniform_wait_bar(bar_afull + 8 * as, committed / A & 1u, ab, leader)) { ok = false; break; }
                tc_fence_after();
                const uint64_t x = desc_x + static_cast<uint64_t>(as) * (C::kWideBytes >> 4);
                const uint32_t a = tmem + C::kOpCol0 + as * kOpCols;
                const int nk = step_mmas(K, kt);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kStepK / 16; ++kk)
                        if (kk < nk)
                            umma_f16_ta(d, a + 8 * kk, x + (kk >> 2) * (C::kBox >> 4) + 2 * (kk & 3), kIdesc,
                                        kt != k0 || kk);
                    umma_commit(bar_aempty + 8 * as);
                }
                ++committed;
                __syncwarp();
            }
            if (!ok) break;
            if (leader) umma_commit(smem_u32(&bars->tfull[acc]));
            __syncwarp();
            u += k1 - k0;
        }
        if (leader) {
            umma_commit(smem_u32(&bars->drain));
            drain_ring(&bars->drain, 1, 1);
            drain_ring(bars->aempty, A, committed);
        }
    } else if (warp >= kWidenWarp0) {
        // ------------------------------------------------------------ codes to operands
        const int group = (warp - kWidenWarp0) / kGroupWarps, in_group = (warp - kWidenWarp0) % kGroupWarps;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t op = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kOpCol0;
        const uint32_t bar_free = smem_u32(&bars->aempty[0]), bar_full = smem_u32(&bars->full[0]),
                       bar_x = smem_u32(&bars->xfull[0]);
        int s = group, as = group;
        uint32_t parity = 0, aparity = 0;
        for (int j = group; j < steps; j += kGroups) {
            if (!group_wait(1 + group, kGroupWarps * 32, in_group == 0 && lane == 0, ab, bar_free + 8 * as, aparity ^ 1u,
                            bar_full + 8 * s, parity, C::kInline ? 0u : bar_x + 8 * as, aparity))
                break;
            tc_fence_after();
            widen_half_row(st_w(s), row, 0, op + as * kOpCols);
            widen_half_row(st_w(s), row, 1, op + as * kOpCols + 32);
            if constexpr (C::kInline) {
#pragma unroll
                for (int i = in_group * 32 + lane; i < MP * 8; i += kGroupWarps * 32)
                    widen_piece(st_x(s), st_wide(as), C::kBox, i);
                fence_proxy_async_smem();   // the MMAs read these stores
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->empty[s]));   // every lane's loads have returned
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->afull[as]));
            if ((s += kGroups) >= S) s -= S, parity ^= 1u;
            if ((as += kGroups) >= A) as -= A, aparity ^= 1u;
        }
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, side = (warp - kEpiWarp0) >> 2;
        constexpr int kCols = MP < 64 ? 16 : 32, kSide = MP / 2 < 16 ? 16 : MP / 2;   // rows of a at a time, per warp
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        int seg = 0;
        for (int u = u_begin, t = t_begin, k0 = k_begin; u < u_end; ++seg, ++t, k0 = 0) {
            const int k1 = min(kt_total, k0 + (u_end - u));
            u += k1 - k0;
            const int acc = seg & 1;
            const int m0 = t % num_m * MP, mc = min(MP, M - m0);
            const int n = t / num_m * BN + q * 32 + lane;
            const float tn = n < N ? __ldg(sb + n) : 0.f;
            if (!group_wait(8, kEpiWarps * 32, threadIdx.x == kEpiWarp0 * 32, ab, smem_u32(&bars->tfull[acc]), (seg >> 1) & 1)) {
                // up to two commits may be on their way
                if (threadIdx.x == kEpiWarp0 * 32) drain_ring(bars->tfull, 2, seg + 2);
                break;
            }
            tc_fence_after();
            const bool whole = k0 == 0 && k1 == kt_total;
            // slot 1: the tile begins here; slot 0: an earlier CTA began it
            float* part =
                partials + (static_cast<size_t>(blockIdx.x) * 2 + (k0 == 0 ? 1 : 0)) * kSlotFloats + q * 32 + lane;
#pragma unroll 1
            for (int c = side * kSide; c < min(mc, (side + 1) * kSide); c += kCols) {
                uint32_t r[kCols];
                if constexpr (kCols == 32) tmem_ld_32x32b_x32(tmem + lanes + acc * C::kAccCols + c, r);
                else tmem_ld_32x32b_x16(tmem + lanes + acc * C::kAccCols + c, r);
                tmem_wait_ld();
                if (split > 1) {
                    // the ring is idle: this CTA's copies have landed and its MMAs have read them
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        if (c + i < mc) parts[(c + i) * 128 + q * 32 + lane] = __uint_as_float(r[i]);
                } else if (whole) {
                    if (n < N) {
#pragma unroll
                        for (int i = 0; i < kCols; ++i)
                            if (c + i < mc)
                                store1<kOut>(y, static_cast<size_t>(m0 + c + i) * ld + n,
                                             __uint_as_float(r[i]) * __ldg(sa + m0 + c + i) * tn);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        if (c + i < mc) __stcg(part + (c + i) * 128, __uint_as_float(r[i]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->tempty[acc]));
        }
    }

    __syncwarp();
    tc_fence_before();
    if (split > 1) {
        cluster_sync();   // every part of the tile is in its CTA's shared memory
        const int t = b / split, m0 = t % num_m * MP, mc = min(MP, M - m0);
        const int col = threadIdx.x & 127, n = t / num_m * BN + col;
        const float tn = n < N ? __ldg(sb + n) : 0.f;
        const uint32_t at = smem_u32(parts) + 4u * col;
        for (int m = kThreads / 128 * part_k + (threadIdx.x >> 7); m < mc; m += kThreads / 128 * split) {
            float v[kMaxSplit], sum = 0.f;
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c) v[c] = c < split ? ld_cluster_f32(at + 512u * m, c) : 0.f;
#pragma unroll
            for (int c = 0; c < kMaxSplit; ++c)
                if (c < split) sum += v[c];
            if (n < N) store1<kOut>(y, static_cast<size_t>(m0 + m) * ld + n, sum * __ldg(sa + m0 + m) * tn);
        }
        cluster_sync();   // no CTA leaves while another may read its part
    } else {
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (!share) return;

    // Shared tiles: the one that this CTA's range begins inside of and the one that it ends inside of. Every range is
    // at least a tile long, so no tile lies in three.
    const bool head = k_begin != 0;
    const int t_end = u_end / kt_total;
    const bool tail = u_end != t_end * kt_total;
    if (threadIdx.x < 2) {
        int last = 0;
        if (threadIdx.x == 0 ? head : tail) {
            uint32_t* ticket = tickets + (threadIdx.x == 0 ? b - 1 : b);   // the lower CTA's
            __threadfence();   // the parts that this CTA's epilogue wrote before the barrier
            last = atomicAdd(ticket, 1u) == 1u;
            if (last) {
                *ticket = 0u;
                __threadfence();
            }
        }
        bars->last[threadIdx.x] = last;
    }
    __syncthreads();
    // half the threads for either tile
    const int which = threadIdx.x >= kThreads / 2, thread = threadIdx.x - which * (kThreads / 2);
    constexpr int kRowsAtOnce = kThreads / 2 / 128, kBatch = MP >= 64 ? 8 : MP >= 32 ? 4 : 2;
    if (!bars->last[which] || thread >= kRowsAtOnce * 128) return;
    const int t = which ? t_end : t_begin, lower = which ? b : b - 1;
    const int m0 = t % num_m * MP, mc = min(MP, M - m0);
    const int col = thread & 127, n = t / num_m * BN + col;
    if (n >= N) return;
    const float tn = __ldg(sb + n);
    const float* lo = partials + (static_cast<size_t>(lower) * 2 + 1) * kSlotFloats + col;
    const float* hi = partials + (static_cast<size_t>(lower) * 2 + 2) * kSlotFloats + col;
    for (int c = thread >> 7; c < mc; c += kRowsAtOnce * kBatch) {
        float p[kBatch], v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int m = min(c + j * kRowsAtOnce, mc - 1);
            p[j] = __ldcg(lo + m * 128);
            v[j] = __ldcg(hi + m * 128);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int m = c + j * kRowsAtOnce;
            if (m < mc) store1<kOut>(y, static_cast<size_t>(m0 + m) * ld + n, (p[j] + v[j]) * __ldg(sa + m0 + m) * tn);
        }
    }
}

}  // namespace tiles

// ---------------------------------------------------------------------------
// CTA pairs: 256 rows of b against bm (a multiple of 32, up to 256) rows of a
// ---------------------------------------------------------------------------
// CTA r of the pair holds rows [128 r, 128 r + 128) of the tile's block of b (its
// tensor-memory lanes) and bm / 2 rows of its block of a (its half of the MMA's
// second operand). Per K step an SM receives 16 KB of codes and, with bm = 256, 32 KB
// of fp16 rows of a for 16.8 MFLOP.
//
//   warp 3       both: TMA of the CTA's codes (a ring of its own)
//   warp 0       both: TMA of the CTA's rows of a, complete on the even CTA's barrier
//   warps 12..19 both: two groups of four on alternate steps widen the codes into
//                an operand stage of the CTA's tensor memory and arrive on the
//                even CTA's barrier
//   warp 1       even: issues the pair's MMAs; its commits free the stages in both
//   warps 4..11  both: epilogue, two warps per lane quarter, bm / 2 columns each
//   warp 2       tensor memory
//
// What the odd CTA's widening warps publish lies in tensor memory alone: they wait
// for their stores, fence (tcgen05.fence::before_thread_sync) and arrive on the even
// CTA's barrier relaxed, which costs them nothing; the MMA thread waits relaxed and
// fences after. Rows of a are published by the copies themselves.
//
// Tensor memory: one accumulator of up to 256 columns and four operand stages of 64.
// The epilogue takes the accumulator into registers, scaled and rounded to 16
// bits, and lets the next tile's MMAs start before it stores (FP32 results are
// stored first: twice the registers). Two accumulators for bm <= 128 were no faster
// (2048 x 16384 x 512 42 us instead of 34 with bm = 256), nor was sharing K steps
// between pairs: the FP32 parts of a tile are 256 KB (512 x 5376 x 5376 44 us instead of 33).
//
// 2048 x 43008 x 5376 458 us in a burst, 2.07 PFLOP/s: at the rate of the fp16 MMAs (a
// K step's eight take about 0.6 us, its 48 KB of loads 0.58 at 82 KB a us and SM). In a
// loop the power limit decides, and with it the codes: 463 to 483 us with uniform ones, 449
// to 464 as activations and weights have them. FP32 results, twice the bytes, stored before
// the next tile's MMAs start: 517 us; 4096 x 4096 x 4096 96 (bf16 82), 2048 x 16384 x 1024 75
// (51). 2048 x 4096 x 65536 632. 96 registers a thread; 24 bytes of spills with 16-bit results.
namespace pair {

constexpr int BN = 256, CM = 128, CN = 128;   // CM: rows of a per CTA at most
constexpr int kThreads = 640;
constexpr int kEpiWarps = 8, kWidenWarp0 = 12, kGroups = 2, kGroupWarps = 4;
constexpr int kStages = 4, kWStages = 5;     // of a and operands; of codes
constexpr uint32_t kXBytes = CM * kStepK * 2, kWBytes = CN * kStepK;
constexpr uint32_t kOpCol0 = 256, kTmemCols = 512;
static_assert(kOpCol0 + kStages * kOpCols == kTmemCols, "tensor memory budget");
static_assert(kStages % kGroups == 0, "each group owns whole operand stages");
// A group takes codes from stages that the other group used in between. It waits
// for the operand stage first: then the MMAs of four steps before have retired,
// so every step up to there, the one that last used this stage of codes among
// them, had been widened and its barrier's phase is complete.
static_assert(kWStages > kStages, "a skipped phase of a code stage is complete");

struct __align__(8) Barriers {
    uint64_t wfull[kWStages];    // this CTA's codes landed
    uint64_t wempty[kWStages];   // widened
    uint64_t xfull[kStages];     // even CTA: both CTAs' rows of a landed
    uint64_t afull[kStages];     // even CTA: both CTAs' operand stages written
    uint64_t empty[kStages];     // both: the step's MMAs retired
    uint64_t tfull;              // both: accumulator complete
    uint64_t tempty;             // even CTA: accumulator read by the pair's epilogue warps
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
constexpr size_t kScaleBytes = kEpiWarps * 128 * 4;
constexpr size_t kSmemBytes = 1024 + kStages * kXBytes + kWStages * kWBytes + kScaleBytes + sizeof(Barriers);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

// Tiles in groups of eight along M, then along N: what runs together shares its
// rows of a and its codes in L2.
struct Place {
    int m, n;
};
__device__ __forceinline__ Place place_of(long long t, int num_m, int num_n) {
    constexpr int kBand = 8;
    const int band = static_cast<int>(t / (static_cast<long long>(kBand) * num_n));
    const int rows = min(kBand, num_m - band * kBand);
    const int in = static_cast<int>(t - static_cast<long long>(band) * kBand * num_n);
    return {band * kBand + in % rows, in / rows};
}

// Two 16-bit values to the next two rows of a column, where `left` rows are left. In one piece: the compiler otherwise
// holds the addresses of all 128 rows of a tile at once.
__device__ __forceinline__ void store_two_rows(uint16_t*& dst, long long pitch, uint32_t v, int left) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
        "setp.gt.s32 p, %3, 0;\n\tsetp.gt.s32 q, %3, 1;\n\t"
        "@p st.global.b16 [%0], lo;\n\tadd.s64 %0, %0, %2;\n\t"
        "@q st.global.b16 [%0], hi;\n\tadd.s64 %0, %0, %2;\n\t}"
        : "+l"(dst)
        : "r"(v), "l"(pitch), "r"(left)
        : "memory");
}

template <int kOut>
__global__ void __launch_bounds__(kThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
            const float* __restrict__ sa, const float* __restrict__ sb, void* __restrict__ y, int M, int N, int K,
            int ld, int bm) {
    extern __shared__ uint8_t smem_raw[];
    // the same layout in both CTAs: the MMA addresses the peer's rows of a at this CTA's offsets
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scales = reinterpret_cast<float*>(smem + kStages * kXBytes + kWStages * kWBytes);
    Barriers* bars = reinterpret_cast<Barriers*>(smem + kStages * kXBytes + kWStages * kWBytes + kScaleBytes);
    const uint32_t base = smem_u32(smem);
    auto st_x = [&](int s) { return base + s * kXBytes; };
    auto st_w = [&](int s) { return base + kStages * kXBytes + s * kWBytes; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int pair_id = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int half = bm / 2, num_m = (M + bm - 1) / bm, num_n = (N + BN - 1) / BN;
    const long long tiles = static_cast<long long>(num_m) * num_n;
    const int kt_total = (K + kStepK - 1) / kStepK;
    const Abort ab{&bars->abort, smem_u32(&bars->abort), static_cast<uint32_t>(rank ^ 1)};

    if (threadIdx.x == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(smem_u32(&bars->wfull[s]), 1);
            mbar_init(smem_u32(&bars->wempty[s]), kGroupWarps);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bars->xfull[s]), 1);
            mbar_init(smem_u32(&bars->afull[s]), 2 * kGroupWarps);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->tfull), 1);
        mbar_init(smem_u32(&bars->tempty), 2 * kEpiWarps);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tw);
        tma_prefetch_desc(&tx);
    }
    if (warp == 2) tmem_alloc_pair(smem_u32(&bars->tmem_base), kTmemCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------------ producers: rows of a (warp 0), codes (warp 3)
        if (lane == 0) {
            const bool codes = warp == 3;
            const int S = codes ? kWStages : kStages;
            const uint32_t bar_empty = smem_u32(codes ? &bars->wempty[0] : &bars->empty[0]);
            const uint32_t even = map_to_cta(smem_u32(&bars->xfull[0]), 0);
            int s = 0;
            long long steps = 0;
            uint32_t parity = 1u;
            bool ok = true;
            for (long long t = pair_id; t < tiles && ok; t += npairs) {
                const Place at = place_of(t, num_m, num_n);
                const int m0 = at.m * bm + rank * half, n0 = at.n * BN + rank * CN;
                for (int kt = 0; kt < kt_total; ++kt) {
                    if (!wait_bar(bar_empty + 8 * s, parity, ab)) { ok = false; break; }
                    if (codes) {
                        const uint32_t fb = smem_u32(&bars->wfull[s]);
                        mbar_arrive_expect_tx(fb, kWBytes);
                        tma_load_2d(st_w(s), &tw, kt * kStepK, n0, fb);
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars->xfull[s]), bm * kStepK * 2);
                        tma_load_2d_pair(st_x(s), &tx, kt * kStepK, m0, even + 8u * s);
                        tma_load_2d_pair(st_x(s) + kXBytes / 2, &tx, kt * kStepK + 64, m0, even + 8u * s);
                    }
                    ++steps;
                    if (++s == S) s = 0, parity ^= 1u;
                }
            }
            // copies and commits in flight arrive before the pair leaves
            if (codes) {
                drain_ring(bars->wfull, kWStages, steps);
            } else {
                if (rank == 0) drain_ring(bars->xfull, kStages, steps);
                drain_ring(bars->empty, kStages, steps);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs (even CTA)
        if (rank == 0) {
            const uint32_t idesc = umma_idesc_f16(BN, bm, false);
            constexpr uint16_t kPair = 0x3;
            const bool leader = elect_one();
            const uint64_t desc_x = sw128_kmajor_desc(st_x(0));
            const uint32_t bar_x = smem_u32(&bars->xfull[0]), bar_a = smem_u32(&bars->afull[0]),
                           bar_empty = smem_u32(&bars->empty[0]);
            int s = 0, it = 0;
            uint32_t parity = 0;
            bool ok = true;
            for (long long t = pair_id; t < tiles && ok; t += npairs, ++it) {
                if (!uniform_wait_bar<true>(smem_u32(&bars->tempty), (it & 1) ^ 1, ab, leader)) { ok = false; break; }
                tc_fence_after();
                for (int kt = 0; kt < kt_total; ++kt) {
                    if (!uniform_wait_bar(bar_x + 8 * s, parity, ab, leader) ||
                        !uniform_wait_bar<true>(bar_a + 8 * s, parity, ab, leader)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t x = desc_x + static_cast<uint64_t>(s) * (kXBytes >> 4);
                    const uint32_t a = tmem + kOpCol0 + s * kOpCols;
                    const int nk = step_mmas(K, kt);
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kStepK / 16; ++kk)
                            if (kk < nk)
                                umma_f16_ta_pair(tmem, a + 8 * kk, x + (kk >> 2) * (kXBytes >> 5) + 2 * (kk & 3), idesc,
                                                 kt || kk);
                        umma_commit_pair_mc(bar_empty + 8 * s, kPair);
                    }
                    __syncwarp();
                    if (++s == kStages) s = 0, parity ^= 1u;
                }
                if (!ok) break;
                if (leader) umma_commit_pair_mc(smem_u32(&bars->tfull), kPair);
                __syncwarp();
            }
            if (leader) {
                umma_commit_pair(smem_u32(&bars->drain));
                drain_ring(&bars->drain, 1, 1);
            }
        }
    } else if (warp >= kWidenWarp0) {
        // ------------------------------------------------------------ codes to tensor memory
        const int group = (warp - kWidenWarp0) / kGroupWarps, in_group = (warp - kWidenWarp0) % kGroupWarps;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t op = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kOpCol0;
        const long long mine = pair_id < tiles ? (tiles - 1 - pair_id) / npairs + 1 : 0;
        const long long steps = mine * kt_total;
        int s = group, ws = group;
        uint32_t parity = 1u, wparity = 0;
        for (long long j = group; j < steps; j += kGroups) {
            if (!group_wait(1 + group, kGroupWarps * 32, in_group == 0 && lane == 0, ab, smem_u32(&bars->empty[s]), parity,
                            smem_u32(&bars->wfull[ws]), wparity))
                break;
            tc_fence_after();
            widen_half_row(st_w(ws), row, 0, op + s * kOpCols);
            widen_half_row(st_w(ws), row, 1, op + s * kOpCols + 32);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->wempty[ws]));   // every lane's loads have returned
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(smem_u32(&bars->afull[s]), 0);
            if ((s += kGroups) >= kStages) s -= kStages, parity ^= 1u;
            if ((ws += kGroups) >= kWStages) ws -= kWStages, wparity ^= 1u;
        }
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, side = (warp - kEpiWarp0) >> 2;
        const uint32_t d = tmem + (static_cast<uint32_t>(q * 32) << 16) + side * half;
        float* mine = scales + (warp - kEpiWarp0) * 128;
        int it = 0;
        for (long long t = pair_id; t < tiles; t += npairs, ++it) {
            const Place at = place_of(t, num_m, num_n);
            const int n = at.n * BN + rank * CN + q * 32 + lane;
            const int m0 = at.m * bm + side * half, mc = min(half, M - m0);
            const float tn = n < N ? __ldg(sb + n) : 0.f;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[32 * i + lane] = 32 * i + lane < mc ? __ldg(sa + m0 + 32 * i + lane) : 0.f;
            __syncwarp();
            if (!group_wait(8, kEpiWarps * 32, threadIdx.x == kEpiWarp0 * 32, ab, smem_u32(&bars->tfull), it & 1)) {
                // one commit at most is on its way to this CTA
                if (threadIdx.x == kEpiWarp0 * 32) drain_ring(&bars->tfull, 1, it + 1);
                break;
            }
            tc_fence_after();
            if constexpr (kOut == kF32) {
#pragma unroll 1
                for (int ch = 0; ch * 32 < half; ++ch) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(d + ch * 32, r);
                    tmem_wait_ld();
                    if (n < N) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (ch * 32 + i < mc)
                                store1<kOut>(y, static_cast<size_t>(m0 + ch * 32 + i) * ld + n,
                                             __uint_as_float(r[i]) * mine[ch * 32 + i] * tn);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(smem_u32(&bars->tempty), 0);
            } else {
                uint32_t o[64];   // of lower tiles the last are not stored
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(d + ch * 16, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = *reinterpret_cast<const float2*>(mine + ch * 16 + 2 * i);
                        const float lo = __uint_as_float(r[2 * i]) * f.x * tn, hi = __uint_as_float(r[2 * i + 1]) * f.y * tn;
                        if constexpr (kOut == kBf16) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                            o[8 * ch + i] = *reinterpret_cast<const uint32_t*>(&h);
                        } else {
                            const __half2 h = __floats2half2_rn(lo, hi);
                            o[8 * ch + i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(smem_u32(&bars->tempty), 0);
                // no branch around the stores: the roundings above would be put off into it, and the raw sums, twice the
                // registers, kept until then
                uint16_t* dst = static_cast<uint16_t*>(y) + static_cast<size_t>(m0) * ld + n;
                const long long pitch = 2ll * ld;
                const int left = n < N ? mc : 0;
#pragma unroll
                for (int i = 0; i < 64; ++i) store_two_rows(dst, pitch, o[i], left - 2 * i);
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync();   // neither CTA leaves while the pair's copies, MMAs or arrivals may touch it
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

}  // namespace pair

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Ticket words (one per CTA of the tiles kernel) at the start of the workspace.
constexpr size_t kControlBytes = 4096;
constexpr int kMaxCtas = static_cast<int>(kControlBytes / 4);
// Rows of a that are widened at a time: bounds the workspace, and keeps them in L2. More rows are cut into equal chunks.
constexpr long long kChunkRows = 8192;
long long chunk_rows(long long M) {
    const long long chunks = (M + kChunkRows - 1) / kChunkRows;
    return chunks == 1 ? M : ((M + chunks - 1) / chunks + 255) / 256 * 256;
}

// Rows of a per tile of the pairs, and the columns of y that the pairs take: all of them, or those of whole waves, the rest
// going to 128-row tiles in a second kernel, in clusters of up to 8. By an estimate in hundredths of a microsecond:
// a K step of a pair takes 0.38 us with up to 128 rows, 0.44, 0.46, 0.51 and 0.58 with 160, 192, 224 and 256 (two tiles
// along M; 0.47 to 0.58 with one, bound by HBM); one on 128-row tiles 0.5, the second kernel 6 us besides. Clusters count as 4
// at most: with all 8 counted the rest is chosen where it loses (201 x 10936 x 11536 52.8 us, then 61.9; 343 x 13488 x 10320
// 81.4 / 88.5; 2351 x 1808 x 13088 97.9 / 94.1), with 4 launched it takes longer (353 x 13032 x 21312 155 / 164). With tiles of
// 256 rows / so (us): 600 x 4096 x 4096 27.2 / 22.0, 300 x 16384 x 1024 23.4 / 17.3, 420 x 5944 x 16944 81.9 / 64.7,
// 4096 x 4096 x 4096 90.1 / 81.6. All columns on pairs of 256 rows / whole waves and the rest: 436 x 10672 x 13200 (84 tiles
// on 76 pairs) 124.5 / 85.2, 1024 x 5120 x 5376 (80) 58.3 / 45.8.
struct PairPlan {
    int bm;
    long long columns, cost;
};
PairPlan pair_plan(long long M, long long N, long long K, int sms, long long pairs) {
    const long long num_n = (N + pair::BN - 1) / pair::BN, steps = (K + kStepK - 1) / kStepK;
    PairPlan best{0, 0, 1ll << 62};
    for (long long parts = (M + 255) / 256; parts <= (M + 127) / 128; ++parts) {
        const long long bm = ((M + parts - 1) / parts + 31) / 32 * 32, num_m = (M + bm - 1) / bm, tiles = num_m * num_n;
        const long long step = 38 + std::max(0ll, bm - 128) * 5 / 32, all = (tiles + pairs - 1) / pairs * steps * step;
        if (all < best.cost) best = {static_cast<int>(bm), N, all};
        const long long waves = tiles / pairs, cut = waves * pairs / num_m;   // whole waves, columns of tiles in them
        if (cut < 1 || cut >= num_n) continue;
        const long long rest = ((M + 127) / 128) * ((N - cut * pair::BN + tiles::BN - 1) / tiles::BN);
        if (rest > sms) continue;
        const long long split = std::min<long long>({4, sms / rest, std::max<long long>(1, steps / 2)});
        const long long both = waves * steps * step + 50 * ((steps + split - 1) / split) + 600;
        if (both < best.cost) best = {static_cast<int>(bm), cut * pair::BN, both};
    }
    return best;
}

struct Plan {
    int mp;       // rows of a per tile of the tiles kernel; 0: CTA pairs; -1: the rows kernel
    bool split;   // tiles kernel: a cluster per tile, where the clusters are resident at once
    bool share;   // tiles kernel: units shared between CTAs
    bool widen;   // rows of a widened by a kernel before
};
// CTAs of a cluster per tile: the largest that `sms` SMs have room for, from 6 saved steps on.
long long cluster_of(long long tiles, long long steps, long long sms) {
    const long long split = std::min<long long>({tiles::kMaxSplit, sms / tiles, steps / 2});
    return split > 1 && steps - steps / split >= 6 ? split : 1;
}
// Measured on 152 SMs (us a call):
//   rows / tiles kernel: 4 x 43008 x 5376 39.3 / 42.5, 8 x 8192 x 4096 12.0 / 12.2, 5 x 8192 x 8192 17.9 / 17.5, 8 x
//     43008 x 5376 63.9 / 43.4, 16 x 4096 x 2048 7.4 / 7.6, 16 x 4096 x 4096 11.0 / 9.7; by the sums per warp, of which
//     each lane's part is added at the end: 8 x 8192 x 1024 5.5 / 7.3, 8 x 16384 x 512 8.0 / 6.3, 16 x 32024 x 144
//     21.3 / 6.6;
//   128-row tiles / pairs: whole, one wave, 4190 x 424 x 8720 57.3 / 49.2, 231 x 7352 x 4272 23.5 / 21.1, 512 x 4096 x
//     4096 20.9 / 20.5, 128 x 19456 x 12288 58.5 / 53.1; a cluster per tile, 256 x 4096 x 14336 35.1 / 50.0; two
//     waves 256 x 16384 x 5376 43.9 / 33.1: pairs but where a cluster works on a tile;
//   whole tiles / shared units: 16 x 20480 x 5376 (160 tiles) 33.9 / 24.9, 30720 columns (240) 35.0 / 33.8, 36864
//     (288) 35.8 / 39.5, 43008 (336) 50.4 / 44.6; 64 rows 40.0 / 31.1, 41.0 / 41.1, 41.7 / 47.4, 58.1 / 52.5: shared
//     where the last wave leaves a fifth of all SM time idle;
//   whole tiles / a cluster per tile: 16 x 8192 x 5376 17.9 / 13.5 (2 CTAs), 64 x 4096 x 4096 17.7 / 11.3 (4), 16 x 4096
//     x 1024 7.2 / 6.4 (4: 6 steps saved), 128 x 8192 x 2048 15.2 / 15.7 (2: 8 saved), 16 x 2048 x 512 5.7 / 6.3 (2: 2
//     saved): from 6 saved steps on;
//   fewer rows per tile than there are (128 / 64 / 32), where the tiles still fit one wave: up to 64 rows are widened in
//     the kernel, and more SMs take part: 300 x 2600 x 2080 16.4 / 11.9 / 15.9, 668 x 24 x 16352 22.0 / 15.2 / 13.4,
//     7200 x 96 x 5920 42.9 / 24.0 / 32.1, 200 x 2048 x 2048 11.7 / 11.3 / 10.0, 256 x 4096 x 4096 19.7 / 17.9 / 26.7,
//     80 x 5376 x 5376 17.0 / 21.6 / 19.1, 128 x 8192 x 5376 22.0 / 22.0 / 34.0. By an estimate, within 2 us of these
//     times: the steps of a CTA, what a tile takes besides, 2 us to add the parts of a cluster, the widening kernel's
//     launch and bytes.
Plan plan(long long M, long long N, long long K, int sms) {
    const long long weights = N * K;
    if (M <= 4 || (M * N <= 3ll << 15 && weights <= (M <= 8 ? 1ll << 25 : M <= 16 ? 1ll << 23 : 0)))
        return {-1, false, false, false};
    const long long cols = (N + tiles::BN - 1) / tiles::BN, steps = (K + kStepK - 1) / kStepK;
    const int most = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    int mp = most;
    if (M > 128 || cols <= sms) {
        // in hundredths of a microsecond
        const long long widen = 400 + M * K * 3 / 70000;   // the launch, and the kernel's bytes
        long long least = 1ll << 62;
        if (M > 64) least = pair_plan(M, N, K, sms, std::max(1, sms / 2)).cost + 400 + widen, mp = 0;
        for (int rows = most; rows >= 16; rows /= 2) {
            const long long tiles = ((M + rows - 1) / rows) * cols;
            if (tiles > sms || rows < std::min(32, most)) break;
            const long long split = cluster_of(tiles, steps, sms);
            if (rows == 128 && split == 1) continue;
            const long long step = rows == 128 ? 48 : rows == 64 ? 40 : 39;
            const long long fixed = rows == 128 ? 600 : rows == 64 ? 500 : 400;
            const long long estimate =
                (steps + split - 1) / split * step + fixed + (split > 1 ? 200 : 0) + (rows == 128 ? widen : 0);
            if (estimate < least) least = estimate, mp = rows;
        }
        if (!mp) return {0, false, false, true};
    }
    const long long tiles = ((M + mp - 1) / mp) * cols, waves = (tiles + sms - 1) / sms;
    return {mp, 2 * tiles <= sms, tiles > sms && waves * sms * 4 > tiles * 5, mp > 64};
}

size_t partial_bytes(const DeviceProps& dp) {
    return static_cast<size_t>(dp.sms) * 2 * tiles::kSlotFloats * sizeof(float);
}

bool encode_codes(CUtensorMap* map, const int8_t* codes, int rows, int K, int box_rows) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, static_cast<uint64_t>(K), static_cast<uint64_t>(rows),
                     static_cast<uint64_t>(K), kStepK, static_cast<uint32_t>(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}
bool encode_wide(CUtensorMap* map, const __half* a, int rows, int K, int box_rows) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a, static_cast<uint64_t>(K), static_cast<uint64_t>(rows),
                     static_cast<uint64_t>(K) * 2, 64, static_cast<uint32_t>(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

// Clusters of `size` CTAs of a kernel (one CTA per SM) that can be resident at once on the device, asked for once.
int resident(const void* kern, const DeviceProps& dp, int size, int threads, size_t smem, std::atomic<int>* cache) {
    std::atomic<int>& known = cache[dp.device & 63];
    if (const int n = known.load(std::memory_order_relaxed)) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size * (dp.sms / size)));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
        (void)cudaGetLastError();
        n = dp.sms / size;
    }
    known.store(n, std::memory_order_relaxed);
    return n;
}
template <int kOut>
int resident_pairs(const DeviceProps& dp) {
    static std::atomic<int> cache[64];
    return resident(reinterpret_cast<const void*>(pair::pair_kernel<kOut>), dp, 2, pair::kThreads, pair::kSmemBytes, cache);
}
template <int kOut, int MP>
int resident_clusters(const DeviceProps& dp, int size) {
    static std::atomic<int> cache[tiles::kMaxSplit + 1][64];
    return resident(reinterpret_cast<const void*>(tiles::tiles_kernel<kOut, MP>), dp, size, tiles::kThreads,
                    tiles::smem_bytes<MP>(), cache[size]);
}

// Kernels that use tensor memory are launched without programmatic
// serialization, as those of mx_matmul.cu.
template <int kOut>
cudaError_t launch_pair(const Int8MatmulArgs& a, int bm, const __half* wide, const DeviceProps& dp, cudaStream_t s) {
    auto kern = pair::pair_kernel<kOut>;
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), dp.device, pair::kSmemBytes);
        e != cudaSuccess)
        return e;
    CUtensorMap tw, tx;
    if (!encode_codes(&tw, a.b, a.N, a.K, pair::CN) || !encode_wide(&tx, wide, a.M, a.K, bm / 2))
        return cudaErrorInvalidValue;
    const long long tiles = static_cast<long long>((a.M + bm - 1) / bm) * ((a.N + pair::BN - 1) / pair::BN);
    const long long pairs = std::max<long long>(1, std::min<long long>(tiles, resident_pairs<kOut>(dp)));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(pair::kThreads);
    cfg.dynamicSmemBytes = pair::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tw, tx, a.sa, a.sb, a.y, a.M, a.N, a.K, a.ld, bm);
}

template <int kOut, int MP>
cudaError_t launch_tiles(const Int8MatmulArgs& a, const Plan& pl, const __half* wide, float* partials, uint32_t* tickets,
                         const DeviceProps& dp, cudaStream_t s) {
    using C = tiles::Cfg<MP>;
    auto kern = tiles::tiles_kernel<kOut, MP>;
    constexpr size_t kSmem = tiles::smem_bytes<MP>();
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), dp.device, kSmem); e != cudaSuccess)
        return e;
    CUtensorMap tw, tx;
    if (!encode_codes(&tw, a.b, a.N, a.K, tiles::BN) ||
        !(C::kInline ? encode_codes(&tx, a.a, a.M, a.K, MP) : encode_wide(&tx, wide, a.M, a.K, MP)))
        return cudaErrorInvalidValue;
    const long long tiles = static_cast<long long>((a.M + MP - 1) / MP) * ((a.N + tiles::BN - 1) / tiles::BN);
    const long long steps = (a.K + kStepK - 1) / kStepK, units = tiles * steps;
    if (units >= 1ll << 31) return cudaErrorInvalidValue;   // 35 TB of codes
    int split = 1;
    if (pl.split) {
        split = static_cast<int>(cluster_of(tiles, steps, dp.sms));
        // all of them resident at once (50 tiles at 64 x 6400 x 5376: clusters of 3 are not, 25.8 us instead of 17.6
        // with 2, on an earlier kernel)
        while (split > 1 && tiles > resident_clusters<kOut, MP>(dp, split)) --split;
        if (split > 1 && steps - steps / split < 6) split = 1;
    }
    const long long grid = split > 1 ? tiles * split : std::min<long long>({tiles, dp.sms, kMaxCtas});
    const long long items = pl.share ? units : tiles;
    const tiles::Work work{split, pl.share ? 1 : 0, static_cast<int>(items / grid), static_cast<int>(items % grid)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(tiles::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (split > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(split);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kern, tw, tx, a.sa, a.sb, a.y, a.M, a.N, a.K, a.ld, work, partials, tickets);
}

template <int kOut>
cudaError_t launch_pairs(const Int8MatmulArgs& all, const __half* wide, const DeviceProps& dp, cudaStream_t s) {
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(pair::pair_kernel<kOut>), dp.device,
                                            pair::kSmemBytes);
        e != cudaSuccess)
        return e;
    const PairPlan pl = pair_plan(all.M, all.N, all.K, dp.sms, resident_pairs<kOut>(dp));
    const long long cut = pl.columns;
    Int8MatmulArgs a = all;
    a.N = static_cast<int>(cut);
    const cudaError_t e = launch_pair<kOut>(a, pl.bm, wide, dp, s);
    if (e != cudaSuccess || cut == all.N) return e;
    a.N = static_cast<int>(all.N - cut);
    a.b += cut * all.K;
    a.sb += cut;
    a.y = static_cast<uint8_t*>(all.y) + cut * (kOut == kF32 ? 4 : 2);
    return launch_tiles<kOut, 128>(a, {128, true, false, true}, wide, nullptr, nullptr, dp, s);
}

template <int kOut>
cudaError_t launch_typed(const Int8MatmulArgs& all, void* workspace, const DeviceProps& dp, cudaStream_t s) {
    const Plan pl = plan(all.M, all.N, all.K, dp.sms);
    if (pl.mp < 0) return rows::launch<kOut>(all, s);
    uint32_t* tickets = static_cast<uint32_t*>(workspace);
    uint8_t* at = static_cast<uint8_t*>(workspace) + kControlBytes;
    float* partials = reinterpret_cast<float*>(at);
    __half* wide = reinterpret_cast<__half*>(at + (pl.share ? partial_bytes(dp) : 0));
    const long long chunk = pl.widen ? chunk_rows(all.M) : all.M;
    for (long long m0 = 0; m0 < all.M; m0 += chunk) {
        Int8MatmulArgs a = all;
        a.M = static_cast<int>(std::min(chunk, all.M - m0));
        a.a += m0 * all.K;
        a.sa += m0;
        a.y = static_cast<uint8_t*>(all.y) + m0 * all.N * (kOut == kF32 ? 4 : 2);
        cudaError_t e = cudaSuccess;
        if (pl.widen) {
            const long long items = static_cast<long long>(a.M) * a.K / 8;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>((items + 255) / 256, dp.sms * 16ll)));
            cfg.blockDim = dim3(256);
            cfg.stream = s;
            if ((e = cudaLaunchKernelEx(&cfg, widen_kernel, a.a, wide, items)) != cudaSuccess) return e;
        }
        switch (pl.mp) {
            case 0: e = launch_pairs<kOut>(a, wide, dp, s); break;
            case 16: e = launch_tiles<kOut, 16>(a, pl, wide, partials, tickets, dp, s); break;
            case 32: e = launch_tiles<kOut, 32>(a, pl, wide, partials, tickets, dp, s); break;
            case 64: e = launch_tiles<kOut, 64>(a, pl, wide, partials, tickets, dp, s); break;
            default: e = launch_tiles<kOut, 128>(a, pl, wide, partials, tickets, dp, s); break;
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

size_t int8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, const DeviceProps& dp) {
    const Plan pl = plan(M, N, K, dp.sms);
    const size_t wide = pl.widen ? static_cast<size_t>(chunk_rows(M)) * static_cast<size_t>(K) * 2 : 0;
    const size_t parts = pl.share ? partial_bytes(dp) : 0;
    return wide + parts ? kControlBytes + parts + wide : 0;
}

void int8_matmul_plan(int64_t M, int64_t N, int64_t K, int sms, int (&out)[5]) {
    const Plan pl = plan(M, N, K, sms);
    const long long rows = pl.widen ? std::min<long long>(M, chunk_rows(M)) : M;
    long long mp = pl.mp, columns = N;
    out[0] = pl.mp, out[1] = 1, out[2] = pl.share, out[3] = 0, out[4] = 0;
    if (pl.mp == 0) {
        const PairPlan pp = pair_plan(rows, N, K, sms, std::max(1, sms / 2));
        out[3] = pp.bm, out[4] = static_cast<int>(pp.columns);
        mp = 128, columns = N - pp.columns;   // the rest
    }
    if (columns && (pl.split || pl.mp == 0))
        out[1] = static_cast<int>(cluster_of((rows + mp - 1) / mp * ((columns + tiles::BN - 1) / tiles::BN),
                                             (K + kStepK - 1) / kStepK, sms));
}

cudaError_t launch_int8_matmul(const Int8MatmulArgs& a, int out_type, void* workspace, const DeviceProps& dp,
                               cudaStream_t s) {
    if (out_type == kF16) return launch_typed<kF16>(a, workspace, dp, s);
    if (out_type == kBf16) return launch_typed<kBf16>(a, workspace, dp, s);
    return launch_typed<kF32>(a, workspace, dp, s);
}

cudaError_t read_and_clear_int8_matmul_error(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_int8_matmul_error, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_int8_matmul_error, &zero, sizeof(zero));
    }
    *out = v;
    return e;
}

}  // namespace w4a16
