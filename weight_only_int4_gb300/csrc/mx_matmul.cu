// Product of two MXFP4 operands on the 5th-generation tensor cores,
//
//     y[m, n] = sum_k A[m, k] B[n, k],   A = a * 2^(ea - 127) per 32 elements of K, B alike,
//
// both in the row layout (codes along K, exponent bytes in tiles of 128 rows x
// 4 blocks). tcgen05.mma kind::mxf4 multiplies the codes as they are, applies
// both rows' exponents to every 32-deep partial product and accumulates in
// FP32, so nothing is decoded: codes and exponent tiles go from global memory
// to shared memory by TMA, the exponents on to tensor memory by tcgen05.cp.
// FP32 sums are rounded once to the output type.
//
// A K step is 256 deep: 128 bytes of codes per row, the width of one
// 128-byte-swizzled row, four MMAs of 64, two exponent tiles per 128 rows.
// Codes past K are zero-filled by TMA and their exponent bytes are zero
// (2^-127), so the tail of a block group adds nothing.
//
// Two kernels:
//   pair_kernel  CTA pairs own 256 x 256 tiles of y (cta_group::2).
//   rows_kernel  128 rows of B against 16..128 rows of A per CTA: what has few
//                tiles of that size. K is split over a cluster, or the (tile, K
//                step) units over all CTAs, where whole tiles would leave SMs
//                idle.
//
// Every mbarrier wait is bounded (about two seconds). On expiry the kernel
// records the timeout in a device word, raises the abort flag, every role
// stops, copies and MMAs in flight are waited for (bounded), tensor memory is
// freed and the kernel returns.
#include "internal.h"
#include "ptx.cuh"
#include "tmap.h"

#include <algorithm>
#include <mutex>

namespace w4a16 {

__device__ unsigned int g_mx_matmul_error = 0;

namespace {

constexpr int kStepK = 256;                 // elements of K per step
constexpr uint32_t kRowBytes = kStepK / 2;  // codes of one row of a step
constexpr uint32_t kScaleTile = 512;        // exponent bytes of 128 rows x 128 elements
constexpr int kThreads = 256;
constexpr int kEpiWarp0 = 4;                // warps 4..7: one tensor-memory lane quarter each
constexpr unsigned long long kWaitLimitCycles = 4000000000ull;   // ~2 s at 2 GHz
constexpr unsigned int kErrTimeout = 9u;

enum : int { kF16 = 0, kBf16 = 1, kF32 = 2 };

// Abort flag of this CTA; in a pair a timeout raises the peer's flag too.
struct Abort {
    volatile int* flag;
    uint32_t addr;
    uint32_t peer;   // cluster rank of the peer, or ~0
};

__device__ __noinline__ bool give_up(const Abort& ab) {
    *ab.flag = 1;
    if (ab.peer != ~0u) st_cluster_u32(ab.addr, ab.peer, 1u);
    atomicOr(&g_mx_matmul_error, 1u << kErrTimeout);
    return false;
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Abort& ab) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = clock64();
    for (;;) {
        // a few polls between looks at the clock; a thread suspended in its wait wakes up late
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*ab.flag) return false;
        if (clock64() - t0 > kWaitLimitCycles) return give_up(ab);
    }
}

// The same for a converged warp that goes on together: one lane polls and a vote
// spreads the verdict, which the compiler knows to be uniform. The warp that
// issues tensor-core instructions waits this way, so that their operands stay in
// uniform registers: under a single-lane branch every instruction moves its
// operands there first, 65 cycles each (measured), more than the copies and
// MMAs themselves take.
__device__ __forceinline__ bool uniform_wait_bar(uint32_t bar, uint32_t parity, const Abort& ab, bool leader) {
    bool done = true;
    if (leader) done = mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    bool ok = true;
    if (leader) ok = wait_bar(bar, parity, ab);
    return __all_sync(0xffffffffu, ok);
}

// Lane 0 waits; the shuffle orders the other lanes' accesses after its acquire.
__device__ __forceinline__ bool warp_wait_bar(uint32_t bar, uint32_t parity, const Abort& ab, int lane) {
    int ok = 1;
    if (lane == 0) ok = wait_bar(bar, parity, ab) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// Bounded wait for the last phase of each ring barrier that `steps` steps have
// used, before the ring's shared memory is given back: no copy, and no arrival
// of a tensor-core commit, may be in flight to a CTA that has left (the next
// kernel's CTA, started early, keeps its own barriers there).
__device__ __forceinline__ void drain_ring(const uint64_t* bars, int stages, long long steps) {
    const unsigned long long t0 = clock64();
    for (long long i = steps > stages ? steps - stages : 0; i < steps; ++i)
        while (!mbar_try_wait(smem_u32(bars + i % stages), static_cast<uint32_t>(i / stages) & 1u) &&
               clock64() - t0 < kWaitLimitCycles) {
        }
}

template <int kOut>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (kOut == kBf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <int kOut>
__device__ __forceinline__ void store1(void* y, size_t at, float v) {
    if constexpr (kOut == kF32) static_cast<float*>(y)[at] = v;
    if constexpr (kOut == kBf16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    if constexpr (kOut == kF16) static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// 32 consecutive columns of one row, in groups of 8 (N % 8 == 0).
template <int kOut>
__device__ __forceinline__ void store_row32(void* y, size_t row_at, int n, int N, const uint32_t (&r)[32]) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (n + 8 * v >= N) break;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[8 * v + i]);
        if constexpr (kOut == kF32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(y) + row_at + n + 8 * v);
            dst[0] = make_float4(f[0], f[1], f[2], f[3]);
            dst[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + row_at + n + 8 * v) =
                make_uint4(pack2<kOut>(f[0], f[1]), pack2<kOut>(f[2], f[3]), pack2<kOut>(f[4], f[5]),
                           pack2<kOut>(f[6], f[7]));
        }
    }
}

// MMAs (64 deep) of a K step.
__device__ __forceinline__ int step_mmas(int K, int kt) { return min(4, (K - kt * kStepK + 63) >> 6); }

// ---------------------------------------------------------------------------
// CTA pairs, 256 x 256 tiles
// ---------------------------------------------------------------------------
// CTA r of the pair holds rows [128r, 128r + 128) of the tile's A block and of
// its B block, the exponents of those A rows and of all 256 B rows. Per K step
// an SM receives 35 KB for 16.8 MFLOP. All loads of both CTAs complete on the
// even CTA's barrier; its MMA thread copies the exponents to tensor memory in
// both CTAs and issues the pair's MMAs.
//
// Tensor memory (512 columns): two 256-column accumulators that overlap by 96
// columns, [0, 256) and [160, 416), and four exponent buffers of 24 columns.
// The epilogue reads the shared 96 columns first and then lets the next tile's
// MMAs start into the other accumulator, so only that read, not the whole
// epilogue, separates two tiles' MMAs.
//
// The MMAs of a step take about 220 ns (measured with the copies left out);
// what the warps that feed them do per step has to stay below that, so codes
// and exponents have a producer thread each, no thread divides, and the MMA warp
// stays converged (uniform_wait_bar).
namespace pair {

constexpr int BM = 256, BN = 256, CM = 128, CN = 128;
constexpr int kStages = 6;
constexpr uint32_t kABytes = CM * kRowBytes, kBBytes = CN * kRowBytes;
constexpr uint32_t kSfaBytes = 2 * kScaleTile, kSfbBytes = 4 * kScaleTile;
constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
static_assert(kStageBytes % 1024 == 0, "operand tiles stay 1024-byte aligned");
constexpr uint32_t kAcc1 = 160, kScaleCol = kAcc1 + 256, kScaleCols = 24;
constexpr int kScaleBufs = 4;
constexpr int kShared = (256 - kAcc1) / 32;   // 32-column chunks of an accumulator that the other one overlaps
constexpr uint32_t kTmemCols = 512;
static_assert(kScaleCol + kScaleBufs * kScaleCols == kTmemCols, "tensor memory budget");
static_assert(kStages > kScaleBufs, "a stage's barrier turns once between the uses of an exponent buffer");

struct __align__(8) Barriers {
    uint64_t full[kStages];     // even CTA: both CTAs' copies landed
    uint64_t empty[kStages];    // both: the step's MMAs retired
    uint64_t tfull[2];          // both: accumulator complete
    uint64_t tempty;            // even CTA: the shared columns were read (one arrival per epilogue warp of the pair)
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + sizeof(Barriers);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

template <int kOut>
__global__ void __launch_bounds__(kThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
            const __grid_constant__ CUtensorMap tsa, const __grid_constant__ CUtensorMap tsb, void* __restrict__ y,
            int M, int N, int K) {
    extern __shared__ uint8_t smem_raw[];
    // the same layout in both CTAs: the MMA and the exponent copies address the peer's at this CTA's offsets
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Barriers* bars = reinterpret_cast<Barriers*>(smem + kStages * kStageBytes);
    const uint32_t base = smem_u32(smem);
    auto st_a = [&](int s) { return base + s * kStageBytes; };
    auto st_b = [&](int s) { return base + s * kStageBytes + kABytes; };
    auto st_sfa = [&](int s) { return base + s * kStageBytes + kABytes + kBBytes; };
    auto st_sfb = [&](int s) { return base + s * kStageBytes + kABytes + kBBytes + kSfaBytes; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair_id = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int num_m = (M + BM - 1) / BM, num_n = (N + BN - 1) / BN;
    const long long tiles = static_cast<long long>(num_m) * num_n;
    const int kt_total = (K + kStepK - 1) / kStepK;
    const Abort ab{&bars->abort, smem_u32(&bars->abort), rank ^ 1u};

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->tfull[0]), 1);
        mbar_init(smem_u32(&bars->tfull[1]), 1);
        mbar_init(smem_u32(&bars->tempty), 2 * 4);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&ta);
        tma_prefetch_desc(&tb);
        tma_prefetch_desc(&tsa);
        tma_prefetch_desc(&tsb);
    }
    if (warp == 2) tmem_alloc_pair(smem_u32(&bars->tmem_base), kTmemCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------------ producers: codes (warp 0), exponents (warp 3)
        if (lane == 0) {
            const int r = static_cast<int>(rank);
            const uint32_t even = map_to_cta(smem_u32(&bars->full[0]), 0);
            int s = 0, steps = 0;
            uint32_t parity = 1u;
            bool ok = true;
            for (long long t = pair_id; t < tiles && ok; t += npairs) {
                const int m_blk = static_cast<int>(t % num_m), n_blk = static_cast<int>(t / num_m);
                const int m0 = m_blk * BM + r * CM, n0 = n_blk * BN + r * CN;
                for (int kt = 0; kt < kt_total; ++kt) {
                    if (!wait_bar(smem_u32(&bars->empty[s]), parity, ab)) { ok = false; break; }
                    const uint32_t bar = even + 8u * s;
                    if (warp == 0) {
                        if (r == 0) mbar_arrive_expect_tx(smem_u32(&bars->full[s]), 2 * kStageBytes);
                        tma_load_2d_pair(st_a(s), &ta, kt * static_cast<int>(kRowBytes), m0, bar);
                        tma_load_2d_pair(st_b(s), &tb, kt * static_cast<int>(kRowBytes), n0, bar);
                    } else {
                        tma_load_3d_pair(st_sfa(s), &tsa, 0, 2 * kt, m_blk * 2 + r, bar);
                        tma_load_3d_pair(st_sfb(s), &tsb, 0, 2 * kt, n_blk * 2, bar);
                    }
                    ++steps;
                    if (++s == kStages) s = 0, parity ^= 1u;
                }
            }
            // every step's copies (counted in the even CTA) and commits have arrived
            if (rank == 0) drain_ring(bars->full, kStages, steps);
            drain_ring(bars->empty, kStages, steps);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ exponent copies and MMAs (even CTA)
        if (rank == 0) {
            constexpr uint32_t kIdesc0 = umma_idesc_mxf4(BM, BN, 0), kIdesc1 = umma_idesc_mxf4(BM, BN, 1);
            constexpr uint16_t kPair = 0x3;
            const bool leader = elect_one();
            const uint64_t desc_a = sw128_kmajor_desc(st_a(0)), desc_b = sw128_kmajor_desc(st_b(0));
            const uint64_t desc_sf = scale_copy_desc(st_sfa(0));
            const uint32_t bar_full = smem_u32(&bars->full[0]), bar_empty = smem_u32(&bars->empty[0]);
            int s = 0, buf = 0, behind = 0, it = 0;   // behind: the stage used kScaleBufs steps ago
            uint32_t parity = 0, behind_parity = 0, steps = 0;
            bool ok = true;
            for (long long t = pair_id; t < tiles && ok; t += npairs, ++it) {
                if (it > 0 && !uniform_wait_bar(smem_u32(&bars->tempty), (it - 1) & 1, ab, leader)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + ((it & 1) ? kAcc1 : 0u);
                for (int kt = 0; kt < kt_total; ++kt) {
                    // the MMAs that read this exponent buffer before have retired
                    if (steps >= kScaleBufs) {
                        if (!uniform_wait_bar(bar_empty + 8 * behind, behind_parity, ab, leader)) { ok = false; break; }
                        if (++behind == kStages) behind = 0, behind_parity ^= 1u;
                    } else {
                        ++steps;
                    }
                    if (!uniform_wait_bar(bar_full + 8 * s, parity, ab, leader)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sfa = tmem + kScaleCol + buf * kScaleCols, sfb = sfa + 8;
                    const uint64_t off = static_cast<uint64_t>(s) * (kStageBytes >> 4);
                    const uint64_t a = desc_a + off, b = desc_b + off, sf = desc_sf + off;
                    // exponent tiles of a stage: A's two groups of 128 along K, then the groups of B's rows 0..127
                    // and 128..255
                    constexpr uint32_t kTile = kScaleTile >> 4;
                    const int nk = step_mmas(K, kt);
                    if (leader) {
                        tmem_cp_scales_pair(sfa, sf);
                        tmem_cp_scales_pair(sfb, sf + 2 * kTile);
                        tmem_cp_scales_pair(sfb + 4, sf + 4 * kTile);
                        if (nk > 2) {
                            tmem_cp_scales_pair(sfa + 4, sf + kTile);
                            tmem_cp_scales_pair(sfb + 8, sf + 3 * kTile);
                            tmem_cp_scales_pair(sfb + 12, sf + 5 * kTile);
                        }
                        // 64 elements (32 bytes) further along K inside the swizzle atom
                        umma_mxf4_pair(d, a, b, kIdesc0, sfa, sfb, kt != 0);
                        if (nk > 1) umma_mxf4_pair(d, a + 2, b + 2, kIdesc1, sfa, sfb, 1);
                        if (nk > 2) umma_mxf4_pair(d, a + 4, b + 4, kIdesc0, sfa + 4, sfb + 8, 1);
                        if (nk > 3) umma_mxf4_pair(d, a + 6, b + 6, kIdesc1, sfa + 4, sfb + 8, 1);
                        umma_commit_pair_mc(bar_empty + 8 * s, kPair);
                    }
                    __syncwarp();
                    if (++s == kStages) s = 0, parity ^= 1u;
                    if (++buf == kScaleBufs) buf = 0;
                }
                if (!ok) break;
                if (leader) umma_commit_pair_mc(smem_u32(&bars->tfull[it & 1]), kPair);
                __syncwarp();
            }
            if (leader) {
                umma_commit_pair(smem_u32(&bars->drain));
                drain_ring(&bars->drain, 1, 1);
            }
        }
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        int it = 0;
        for (long long t = pair_id; t < tiles; t += npairs, ++it) {
            const int m_blk = static_cast<int>(t % num_m), n_blk = static_cast<int>(t / num_m);
            if (!warp_wait_bar(smem_u32(&bars->tfull[it & 1]), (it >> 1) & 1, ab, lane)) break;
            tc_fence_after();
            const uint32_t d = tmem + lanes + ((it & 1) ? kAcc1 : 0u);
            const int m = m_blk * BM + static_cast<int>(rank) * CM + q * 32 + lane;
            const size_t row_at = static_cast<size_t>(m) * N;
            const int n0 = n_blk * BN;
            // columns shared with the other accumulator first: the last of the even one, the first of the odd
            const int c0 = (it & 1) ? 0 : 8 - kShared;
            {
                uint32_t r[kShared][32];
#pragma unroll
                for (int i = 0; i < kShared; ++i) tmem_ld_32x32b_x32(d + (c0 + i) * 32, r[i]);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(smem_u32(&bars->tempty), 0);
                if (m < M) {
#pragma unroll
                    for (int i = 0; i < kShared; ++i) store_row32<kOut>(y, row_at, n0 + (c0 + i) * 32, N, r[i]);
                }
            }
#pragma unroll 1
            for (int i = 0; i < 8 - kShared; ++i) {
                const int ch = (it & 1) ? i + kShared : i;
                uint32_t r[32];
                tmem_ld_32x32b_x32(d + ch * 32, r);
                tmem_wait_ld();
                if (m < M) store_row32<kOut>(y, row_at, n0 + ch * 32, N, r);
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
// few rows of A: 128 rows of B per tile, stream-K
// ---------------------------------------------------------------------------
// The tile's 128 rows of B are the MMA's M, MP rows of A its N: with few rows
// of A the kernel streams B and is bound by HBM bandwidth, or by the latency of
// a tile's K steps (about 0.29 us each, with a ring of 6..10 steps) where few
// tiles leave SMs idle. Three ways to hand out the work:
//   whole tiles, one or more per CTA;
//   split > 1: a cluster of `split` CTAs per tile, each a part of K; the parts
//     are added from the CTAs' shared memory, in the order of K;
//   share: equal ranges of (tile, K step) units; a tile shared by several CTAs
//     is finished by the last of them (a ticket per tile and epilogue warp),
//     which adds their FP32 parts from global memory in ascending CTA order.
// All three are deterministic.
namespace rows {

constexpr int BN = 128;
constexpr size_t kSlotFloats = 128 * 128;   // partial tile, [row of A][row of B]

template <int MP>
struct Cfg {
    static constexpr int kStages = MP == 128 ? 6 : MP == 64 ? 8 : 10;
    static constexpr uint32_t kABytes = BN * kRowBytes;   // the MMA's A: rows of B
    static constexpr uint32_t kXBytes = MP * kRowBytes;
    static constexpr uint32_t kStageBytes = kABytes + kXBytes + 4 * kScaleTile;
    static_assert(kStageBytes % 1024 == 0, "operand tiles stay 1024-byte aligned");
    static constexpr uint32_t kAccCols = MP < 32 ? 32 : MP;   // the epilogue reads 32 columns at a time
    static constexpr uint32_t kScaleCol = 2 * kAccCols;       // 16 columns of exponents per stage
    static constexpr uint32_t kTmemCols = kScaleCol + 16 * kStages <= 256 ? 256 : 512;
    static_assert(kScaleCol + 16 * kStages <= 512, "tensor memory budget");
    // What plan() never gives a template is not compiled into it: 128-row tiles are taken where more than half of the
    // SMs have one, and tiles are shared only for one row tile.
    static constexpr bool kSplits = MP < 128, kShares = MP <= kMxMatmulSharedMaxM;
};

template <int MP>
struct __align__(8) Barriers {
    uint64_t full[Cfg<MP>::kStages];
    uint64_t empty[Cfg<MP>::kStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
template <int MP>
constexpr size_t smem_bytes() {
    return 1024 + Cfg<MP>::kStages * Cfg<MP>::kStageBytes + sizeof(Barriers<MP>);
}

// CTA b of G owns units [b U / G, (b + 1) U / G) (tiles where none are shared); the owner of unit u.
__device__ __forceinline__ long long first_unit(long long b, long long U, int G) { return b * U / G; }
__device__ __forceinline__ int unit_owner(long long u, long long U, int G) {
    return static_cast<int>(((u + 1) * G - 1) / U);
}

template <int kOut, int MP>
__global__ void __launch_bounds__(kThreads, 1)
rows_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
            const uint8_t* __restrict__ ew, const uint8_t* __restrict__ ex, void* __restrict__ y,
            int M, int N, int K, int split_by, int shared_units, float* __restrict__ partials,
            uint32_t* __restrict__ tickets) {
    using C = Cfg<MP>;
    constexpr int S = C::kStages;
    const int split = C::kSplits ? split_by : 1;
    const bool share = C::kShares && shared_units;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Barriers<MP>* bars = reinterpret_cast<Barriers<MP>*>(smem + S * C::kStageBytes);
    const uint32_t base = smem_u32(smem);
    auto st_w = [&](int s) { return base + s * C::kStageBytes; };
    auto st_x = [&](int s) { return base + s * C::kStageBytes + C::kABytes; };
    auto st_sw = [&](int s) { return base + s * C::kStageBytes + C::kABytes + C::kXBytes; };
    auto st_sx = [&](int s) { return st_sw(s) + 2 * kScaleTile; };
    // split > 1: this CTA's part, [row of A][128], once the ring is idle
    float* parts = reinterpret_cast<float*>(smem);
    static_assert(MP * 128 * 4 <= S * C::kStageBytes, "a part fits the ring");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_m = (M + MP - 1) / MP, num_n = (N + BN - 1) / BN;
    const int kt_total = (K + kStepK - 1) / kStepK, groups = (K + 127) >> 7;
    const int G = gridDim.x;
    const long long T = static_cast<long long>(num_m) * num_n, U = T * kt_total;
    const int part_k = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    long long u_begin, u_end;
    if (split > 1) {
        const long long first = static_cast<long long>(blockIdx.x / split) * kt_total;
        u_begin = first + static_cast<long long>(part_k) * kt_total / split;
        u_end = first + static_cast<long long>(part_k + 1) * kt_total / split;
    } else {
        u_begin = share ? first_unit(blockIdx.x, U, G) : first_unit(blockIdx.x, T, G) * kt_total;
        u_end = share ? first_unit(blockIdx.x + 1ll, U, G) : first_unit(blockIdx.x + 1ll, T, G) * kt_total;
    }
    const Abort ab{&bars->abort, 0u, ~0u};

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&bars->tfull[a]), 1);
            mbar_init(smem_u32(&bars->tempty[a]), 4);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tw);
        tma_prefetch_desc(&tx);
    }
    if (warp == 2) tmem_alloc(smem_u32(&bars->tmem_base), C::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int s = 0, steps = 0;
            uint32_t parity = 1u;
            bool ok = true;
            for (long long u = u_begin; u < u_end && ok;) {
                const long long t = u / kt_total;
                const int k0 = static_cast<int>(u - t * kt_total);
                const int k1 = static_cast<int>(std::min<long long>(kt_total, k0 + (u_end - u)));
                const int m_blk = static_cast<int>(t % num_m), n_blk = static_cast<int>(t / num_m);
                for (int kt = k0; kt < k1; ++kt) {
                    if (!wait_bar(smem_u32(&bars->empty[s]), parity, ab)) { ok = false; break; }
                    const uint32_t fb = smem_u32(&bars->full[s]);
                    // the exponent tiles of a row tile lie one after the other along K
                    const uint32_t sf = min(2, groups - 2 * kt) * kScaleTile;
                    mbar_arrive_expect_tx(fb, C::kABytes + C::kXBytes + 2 * sf);
                    tma_load_2d(st_w(s), &tw, kt * static_cast<int>(kRowBytes), n_blk * BN, fb);
                    tma_load_2d(st_x(s), &tx, kt * static_cast<int>(kRowBytes), m_blk * MP, fb);
                    bulk_load(st_sw(s), ew + (static_cast<size_t>(n_blk) * groups + 2 * kt) * kScaleTile, sf, fb);
                    bulk_load(st_sx(s), ex + (static_cast<size_t>(m_blk * MP / 128) * groups + 2 * kt) * kScaleTile, sf,
                              fb);
                    ++steps;
                    if (++s == S) s = 0, parity ^= 1u;
                }
                u += k1 - k0;
            }
            drain_ring(bars->full, S, steps);
            drain_ring(bars->empty, S, steps);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ exponent copies and MMAs
        constexpr uint32_t kIdesc0 = umma_idesc_mxf4(BN, MP, 0), kIdesc1 = umma_idesc_mxf4(BN, MP, 1);
        const bool leader = elect_one();
        const uint64_t desc_w = sw128_kmajor_desc(st_w(0)), desc_x = sw128_kmajor_desc(st_x(0));
        const uint64_t desc_sf = scale_copy_desc(st_sw(0));
        const uint32_t bar_full = smem_u32(&bars->full[0]), bar_empty = smem_u32(&bars->empty[0]);
        int s = 0, seg = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (long long u = u_begin; u < u_end && ok; ++seg) {
            const int k0 = static_cast<int>(u % kt_total);
            const int k1 = static_cast<int>(std::min<long long>(kt_total, k0 + (u_end - u)));
            const int acc = seg & 1;
            if (!uniform_wait_bar(smem_u32(&bars->tempty[acc]), ((seg >> 1) & 1) ^ 1, ab, leader)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + acc * C::kAccCols;
            // exponents of 32 rows per column: where the tile's rows begin in their 128-row exponent tile (fewer
            // than 32 rows of A per tile only come as the first)
            const uint32_t x_col = static_cast<uint32_t>(u / kt_total % num_m) * MP % 128 / 32;
            for (int kt = k0; kt < k1; ++kt) {
                if (!uniform_wait_bar(bar_full + 8 * s, parity, ab, leader)) { ok = false; break; }
                tc_fence_after();
                // one exponent buffer per stage: the MMAs that read it retired before the stage was refilled
                const uint32_t sfw = tmem + C::kScaleCol + 16 * s, sfx = sfw + 8;
                const uint64_t off = static_cast<uint64_t>(s) * (C::kStageBytes >> 4);
                const uint64_t w = desc_w + off, x = desc_x + off, sf = desc_sf + off;
                constexpr uint32_t kTile = kScaleTile >> 4;
                const int nk = step_mmas(K, kt);
                if (leader) {
                    tmem_cp_scales(sfw, sf);
                    tmem_cp_scales(sfx, sf + 2 * kTile);
                    if (nk > 2) {
                        tmem_cp_scales(sfw + 4, sf + kTile);
                        tmem_cp_scales(sfx + 4, sf + 3 * kTile);
                    }
                    const uint32_t x0 = sfx + x_col, x1 = x0 + 4;
                    umma_mxf4(d, w, x, kIdesc0, sfw, x0, kt != k0);
                    if (nk > 1) umma_mxf4(d, w + 2, x + 2, kIdesc1, sfw, x0, 1);
                    if (nk > 2) umma_mxf4(d, w + 4, x + 4, kIdesc0, sfw + 4, x1, 1);
                    if (nk > 3) umma_mxf4(d, w + 6, x + 6, kIdesc1, sfw + 4, x1, 1);
                    umma_commit(bar_empty + 8 * s);
                }
                __syncwarp();
                if (++s == S) s = 0, parity ^= 1u;
            }
            if (!ok) break;
            if (leader) umma_commit(smem_u32(&bars->tfull[acc]));
            __syncwarp();
            u += k1 - k0;
        }
        if (leader) {
            umma_commit(smem_u32(&bars->drain));
            drain_ring(&bars->drain, 1, 1);
        }
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        int seg = 0;
        for (long long u = u_begin; u < u_end; ++seg) {
            const long long t = u / kt_total;
            const int k0 = static_cast<int>(u - t * kt_total);
            const int k1 = static_cast<int>(std::min<long long>(kt_total, k0 + (u_end - u)));
            u += k1 - k0;
            const int acc = seg & 1;
            if (!warp_wait_bar(smem_u32(&bars->tfull[acc]), (seg >> 1) & 1, ab, lane)) break;
            tc_fence_after();
            const int m0 = static_cast<int>(t % num_m) * MP;
            const int mc = min(MP, M - m0);                              // rows of A of this tile
            const int n = static_cast<int>(t / num_m) * BN + q * 32 + lane;
            const bool whole = !C::kShares || (k0 == 0 && k1 == kt_total);
            // slot 1: the tile begins here; slot 0: an earlier CTA began it
            float* part =
                partials + (static_cast<size_t>(blockIdx.x) * 2 + (k0 == 0 ? 1 : 0)) * kSlotFloats + q * 32 + lane;
#pragma unroll 1
            for (int ch = 0; ch * 32 < mc; ++ch) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tmem + lanes + acc * C::kAccCols + ch * 32, r);
                tmem_wait_ld();
                if (split > 1) {
                    // the ring is idle: this CTA's copies have landed and its MMAs have read them
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (ch * 32 + i < mc) parts[(ch * 32 + i) * 128 + q * 32 + lane] = __uint_as_float(r[i]);
                } else if (whole) {
                    if (n < N) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (ch * 32 + i < mc)
                                store1<kOut>(y, static_cast<size_t>(m0 + ch * 32 + i) * N + n, __uint_as_float(r[i]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (ch * 32 + i < mc) __stcg(part + (ch * 32 + i) * 128, __uint_as_float(r[i]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->tempty[acc]));
            if (whole || split > 1) continue;
            const long long first = t * kt_total;
            const int b_lo = unit_owner(first, U, G), b_hi = unit_owner(first + kt_total - 1, U, G);
            __threadfence();
            __syncwarp();
            uint32_t last = 0;
            if (lane == 0) last = atomicAdd(tickets + 4 * t + q, 1u) == static_cast<unsigned>(b_hi - b_lo);
            last = __shfl_sync(0xffffffffu, last, 0);
            if (!last) continue;
            __threadfence();
            if (n < N) {
                const float* lo = partials + (static_cast<size_t>(b_lo) * 2 + 1) * kSlotFloats + q * 32 + lane;
                for (int c = 0; c < mc; c += 16) {
                    float sum[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[i] = c + i < mc ? __ldcg(lo + (c + i) * 128) : 0.f;
                    for (int b = b_lo + 1; b <= b_hi; ++b) {
                        const float* src = partials + static_cast<size_t>(b) * 2 * kSlotFloats + q * 32 + lane;
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = c + i < mc ? __ldcg(src + (c + i) * 128) : 0.f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[i] += v[i];
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < mc) store1<kOut>(y, static_cast<size_t>(m0 + c + i) * N + n, sum[i]);
                }
            }
            if (lane == 0) tickets[4 * t + q] = 0u;
        }
    }

    __syncwarp();
    tc_fence_before();
    if (split > 1) {
        cluster_sync();   // every part of the tile is in its CTA's shared memory
        const long long t = blockIdx.x / split;
        const int m0 = static_cast<int>(t % num_m) * MP, mc = min(MP, M - m0);
        const int col = threadIdx.x & 127, n = static_cast<int>(t / num_m) * BN + col;
        const uint32_t at = smem_u32(parts) + 4u * col;
        for (int m = 2 * part_k + (threadIdx.x >> 7); m < mc; m += 2 * split) {
            float v[8], sum = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = c < split ? ld_cluster_f32(at + 512u * m, c) : 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < split) sum += v[c];
            if (n < N) store1<kOut>(y, static_cast<size_t>(m0 + m) * N + n, sum);
        }
        cluster_sync();   // no CTA leaves while another may read its part
    } else {
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace rows

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Codes [rows, K/2 bytes]: boxes of one K step by `box_rows` rows.
bool encode_codes(CUtensorMap* map, const uint32_t* codes, int rows, int K, int box_rows) {
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, static_cast<uint64_t>(K / 2),
                     static_cast<uint64_t>(rows), static_cast<uint64_t>(K / 2), kRowBytes,
                     static_cast<uint32_t>(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}
// Exponent tiles [row tile, group of 128 along K, 128 words]: boxes of one K step (two groups) by `tiles` row tiles.
bool encode_scales(CUtensorMap* map, const uint8_t* es, int rows, int K, int tiles) {
    const uint64_t groups = static_cast<uint64_t>((K + 127) / 128);
    return encode_3d(map, CU_TENSOR_MAP_DATA_TYPE_INT32, es, 128, groups, static_cast<uint64_t>((rows + 127) / 128),
                     kScaleTile, groups * kScaleTile, 128, 2, static_cast<uint32_t>(tiles), CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct Plan {
    int mp;       // rows of A per tile; 0: the pair kernel
    int split;    // CTAs of a cluster per tile
    bool share;   // tiles split between CTAs by units
};

// Measured on 152 SMs (us a call, whole tiles unless said):
//   pair kernel against 128-row tiles: 1024 x 2560 x 5376 (160 tiles) 13.7 / 19.0, 200 x 16384 x 5376 (256) 16.2 /
//     20.2, 512 x 4096 x 4096 (128) 11.7 / 11.1, 700 x 2560 x 5376 (120) 14.0 / 12.6: the pair kernel where 128-row
//     tiles need a second wave;
//   64-row against 128-row tiles: 300 x 2600 x 2080 (63 tiles of 128) 7.9 / 9.1, 128 x 6144 x 2048 (48) 7.8 / 8.7,
//     512 x 4096 x 4096 (128) 15.0 / 11.1: 64 where both kinds fit one wave;
//   shared units against whole tiles: 16 x 43008 x 5376 (336 tiles) 27.1 / 29.5, 32 rows 29.2 / 29.7, but 64 rows
//     32.9 / 29.9 and what fits one wave slower (16 x 16384 x 5376 15.0 / 12.3): up to 32 rows, where the last wave
//     is mostly idle.
Plan plan(long long M, long long N, long long K, int sms) {
    const long long cols = (N + rows::BN - 1) / rows::BN, steps = (K + kStepK - 1) / kStepK;
    const long long tiles128 = ((M + 127) / 128) * cols;
    if (M > 128 && tiles128 > sms) return {0, 1, false};
    const int mp = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 || 2 * tiles128 <= sms ? 64 : 128;
    const long long tiles = ((M + mp - 1) / mp) * cols;
    // A step saved is worth 0.3 us; a cluster's sum costs 1 to 1.5 us with up to 32 rows and 2 with 64. Whole / split:
    // 1 x 2048 x 4096 10.2 / 5.8 (6 CTAs a tile), 1 x 5376 x 21504 30.2 / 15.3 (3), 100 x 1288 x 9120 15.8 / 8.7 (6),
    // 16 x 5376 x 2048 7.4 / 6.6 (3: 6 steps saved), 16 x 8192 x 2048 7.5 / 7.6 (2: 4 saved), 64 x 5376 x 2048 7.7 /
    // 8.4 (3: 6 saved). Clusters of 7 and 8 do not all fit at once: 16 x 2048 x 8192 7.8 with 6, 13.2 with 7, 12.3
    // with 8.
    const long long split = std::min<long long>({6, sms / tiles, steps / 2});
    if (split > 1 && steps - steps / split >= (mp <= 32 ? 5 : 8)) return {mp, static_cast<int>(split), false};
    const long long waves = (tiles + sms - 1) / sms;
    return {mp, 1, M <= kMxMatmulSharedMaxM && tiles > sms && waves * sms * 100 > tiles * 115};
}

template <int kOut>
int resident_pairs(const DeviceProps& dp) {
    static std::mutex mu;
    static int cached[64] = {0};
    const int dev = (dp.device >= 0 && dp.device < 64) ? dp.device : 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!cached[dev]) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (dp.sms / 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = pair::kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, pair::pair_kernel<kOut>, &cfg) != cudaSuccess || n <= 0) {
            (void)cudaGetLastError();
            n = dp.sms / 2;
        }
        cached[dev] = n;
    }
    return cached[dev];
}

template <int kOut>
cudaError_t launch_pair(const MxMatmulArgs& a, const DeviceProps& dp, cudaStream_t s) {
    auto kern = pair::pair_kernel<kOut>;
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), dp.device, pair::kSmemBytes);
        e != cudaSuccess)
        return e;
    CUtensorMap ta, tb, tsa, tsb;
    if (!encode_codes(&ta, a.a, a.M, a.K, pair::CM) || !encode_codes(&tb, a.b, a.N, a.K, pair::CN) ||
        !encode_scales(&tsa, a.ea, a.M, a.K, 1) || !encode_scales(&tsb, a.eb, a.N, a.K, 2))
        return cudaErrorInvalidValue;
    const long long tiles = static_cast<long long>((a.M + pair::BM - 1) / pair::BM) * ((a.N + pair::BN - 1) / pair::BN);
    cudaLaunchConfig_t cfg = {};
    const long long pairs = std::max<long long>(1, std::min<long long>(tiles, resident_pairs<kOut>(dp)));
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = pair::kSmemBytes;
    cfg.stream = s;
    // no programmatic serialization: see launch_rows
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, ta, tb, tsa, tsb, a.y, a.M, a.N, a.K);
}

template <int kOut, int MP>
cudaError_t launch_rows(const MxMatmulArgs& a, const Plan& pl, float* partials, uint32_t* tickets,
                        const DeviceProps& dp, cudaStream_t s) {
    auto kern = rows::rows_kernel<kOut, MP>;
    constexpr size_t kSmem = rows::smem_bytes<MP>();
    static_assert(kSmem <= 227 * 1024, "shared memory budget");
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), dp.device, kSmem); e != cudaSuccess)
        return e;
    CUtensorMap tw, tx;
    if (!encode_codes(&tw, a.b, a.N, a.K, rows::BN) || !encode_codes(&tx, a.a, a.M, a.K, MP))
        return cudaErrorInvalidValue;
    const long long tiles = static_cast<long long>((a.M + MP - 1) / MP) * ((a.N + rows::BN - 1) / rows::BN);
    const long long units = tiles * ((a.K + kStepK - 1) / kStepK);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pl.split > 1 ? tiles * pl.split
                                                          : std::min<long long>(pl.share ? units : tiles, dp.sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    // No kernel of this file or of mx_quant.cu is launched with programmatic
    // serialization. With it on the quantisation and on the pair kernel, a queue of
    // about a hundred calls stopped making progress; the calls were right one at a
    // time, and reading gave no cause: every grid waits for earlier grids only, no
    // two of these CTAs with tensor memory fit one SM, and the ring barriers are
    // drained before a CTA leaves. What such a CTA does before its dependency wait
    // is not bounded by a time limit either (tensor-memory allocation, the cluster
    // barrier, the wait itself). So what follows one of these kernels starts when it
    // has completed.
    cudaLaunchAttribute attr[1];
    if (pl.split > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(pl.split);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kern, tw, tx, a.eb, a.ea, a.y, a.M, a.N, a.K, pl.split, pl.share ? 1 : 0,
                              partials, tickets);
}

size_t partial_bytes(const DeviceProps& dp) {
    return static_cast<size_t>(dp.sms) * 2 * rows::kSlotFloats * sizeof(float);
}

template <int kOut>
cudaError_t launch_typed(const MxMatmulArgs& a, void* workspace, const DeviceProps& dp, cudaStream_t s) {
    const Plan pl = plan(a.M, a.N, a.K, dp.sms);
    float* partials = static_cast<float*>(workspace);
    uint32_t* tickets = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + partial_bytes(dp));
    switch (pl.mp) {
        case 0: return launch_pair<kOut>(a, dp, s);
        case 16: return launch_rows<kOut, 16>(a, pl, partials, tickets, dp, s);
        case 32: return launch_rows<kOut, 32>(a, pl, partials, tickets, dp, s);
        case 64: return launch_rows<kOut, 64>(a, pl, partials, tickets, dp, s);
        default: return launch_rows<kOut, 128>(a, pl, partials, tickets, dp, s);
    }
}

}  // namespace

void mx_matmul_plan(int64_t M, int64_t N, int64_t K, int sms, int (&out)[3]) {
    const Plan pl = plan(M, N, K, sms);
    out[0] = pl.mp, out[1] = pl.split, out[2] = pl.share ? 1 : 0;
}

size_t mx_matmul_workspace_bytes(int64_t M, int64_t N, const DeviceProps& dp) {
    if (M > kMxMatmulSharedMaxM) return 0;
    const size_t cols = static_cast<size_t>((N + rows::BN - 1) / rows::BN);
    return partial_bytes(dp) + ((cols * 4 * sizeof(uint32_t) + 255) & ~size_t(255));
}

cudaError_t launch_mx_matmul(const MxMatmulArgs& a, int out_type, void* workspace, const DeviceProps& dp,
                             cudaStream_t s) {
    if (out_type == kF16) return launch_typed<kF16>(a, workspace, dp, s);
    if (out_type == kBf16) return launch_typed<kBf16>(a, workspace, dp, s);
    return launch_typed<kF32>(a, workspace, dp, s);
}

cudaError_t read_and_clear_mx_matmul_error(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_mx_matmul_error, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_mx_matmul_error, &zero, sizeof(zero));
    }
    *out = v;
    return e;
}

}  // namespace w4a16
