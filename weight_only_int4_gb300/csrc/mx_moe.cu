// A whole mixture-of-experts layer for a few tokens, in one kernel:
//
//     p    = softmax(x R^T), the k largest of each token (ties to the lower index)
//     h_e  = silu(x W1_e) * (x W3_e)            for the chosen experts e
//     y    = sum_e p_e (h_e W2_e)
//
// W13_e = [W1_e | W3_e] and W2_e are MXFP4 in the weight layout (codes along K,
// one exponent byte per 32 rows of a column). With few tokens every chosen
// expert's weights are read once and used for a handful of rows, so the layer is
// bound by HBM bandwidth; small calls by the latency of their four dependent
// phases, which is why they share one launch:
//
//   0  router logits (warp-level bf16 MMAs, 16 experts x 8 tokens a CTA) and x
//      as fp16 with one power-of-two factor per token
//      -- grid barrier --
//   1  every CTA picks the experts itself (a warp per token) and lists the
//      tokens of each expert in groups of up to 16
//   2  items (group, 32 gate columns and their 32 up columns): products, SwiGLU,
//      h as fp16 with one power of two per 32 columns
//      -- grid barrier (the first weights of phase 3 are already on their way) --
//   3  items (group, 64 columns of y): products; the last of a token's k experts
//      to finish a column block adds the k parts in order: deterministic
//
// A CTA is one producer warp and sixteen consumer warps around a ring of
// stages. A stage is 256 rows of K by 64 columns of codes (two TMA boxes of 32
// columns, 128-byte swizzle), their exponent bytes and the same 256 elements of
// the group's activation rows. Two sets of eight warps, each with a ring of its
// own, take alternate stages of an item (which set takes the first depends on
// the column block alone, so a token's sums are formed in the same order
// whatever else the call holds); a warp converts one 32-row block: a lane's 16-byte load holds eight consecutive
// codes of each of four columns, which become fp16 pairs by the hardware's
// exact conversion and serve as the A operand of warp-level MMAs (columns of W
// as MMA rows, tokens as MMA columns), x as B; K is permuted alike on both
// sides, so neither needs a shuffle. The block's FP32 products are scaled by
// the columns' 2^(e - 127) as they are added up. The sixteen warps' sums meet
// in shared memory once per item.
//
// Activations in fp16: a token's x is multiplied by the power of two that
// brings its largest magnitude just below 2^15, a run of 32 h values likewise
// (then aligned to the run with the largest magnitude of its row, again by a
// power of two). Values within 2^-29 of the largest convert exactly or, for h,
// with fp16's 11 bits; smaller ones lose at most 2^-39 of the largest.
//
// Waits are bounded (about two seconds); on expiry the kernel records the
// timeout in a device word, every role stops, copies in flight are waited for
// (bounded) and the kernel returns.
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include "tmap.h"

#include <algorithm>

namespace w4a16 {

__device__ unsigned int g_mx_moe_error = 0;

namespace {

constexpr int kConsumerWarps = 16;
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kSetStages = 3;            // ring of each set of warps
constexpr int kStages = 2 * kSetStages;
constexpr int kStepK = 256;              // rows of K per stage: one 32-row block per warp of a set
constexpr int kBlocks = kStepK / 32;
constexpr int kGroup = 16;               // tokens of an expert taken together
constexpr int kMaxExperts = kMoeMaxExperts;
constexpr int kMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
constexpr uint32_t kBoxBytes = 32 * 128;             // 32 word rows x 32 columns
constexpr uint32_t kScaleBoxBytes = kBlocks * 32;
constexpr uint32_t kXStride = 704;       // 8 records of 80 bytes, padded so that two rows' 64 bytes hit different banks
constexpr uint32_t kStageBytes = 2 * kBoxBytes + 2 * kScaleBoxBytes + kGroup * kXStride;
static_assert(kStageBytes % 128 == 0, "stages stay 128-byte aligned");
constexpr uint32_t kStagePitch = (kStageBytes + 1023) & ~1023u;   // swizzled boxes start 1024-byte aligned
constexpr int kRedPitch = 33;            // floats per slot of a warp's partial sums
constexpr int kRedSlots = 32;            // [token parity of an 8-token tile, tile][box][column % 4]
constexpr uint32_t kSuspendNs = 20000;
constexpr unsigned long long kWaitLimitCycles = 4000000000ull;   // ~2 s at 2 GHz
constexpr unsigned int kErrTimeout = 9u;
constexpr int kHRecord = 80;             // 32 fp16 values, the run's shift, padding to 16 bytes

struct __align__(16) Shared {
    float red[kConsumerWarps][kRedSlots][kRedPitch];
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t phase3;                     // h of every CTA is visible
    unsigned long long mask[kMaxExperts];
    float weight[kMaxSlots];             // of slot t * k + j
    uint32_t group[kMaxSlots];           // expert | count << 16
    uint16_t first[kMaxSlots];           // the group's first entry in `list`
    uint16_t list[kMaxSlots];            // slots, ordered by expert, then token
    uint16_t ids[kMaxSlots];             // expert of slot t * k + j
    uint16_t offset[kMaxExperts], goffset[kMaxExperts];
    int groups;
    uint32_t generation;
    int abort;
};
constexpr size_t kSmemBytes = 1024 + kStages * kStagePitch + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct Params {
    const uint16_t* x;
    const uint16_t* router;
    uint16_t* y;
    uint32_t* control;     // barrier count, barrier generation, then tickets
    float* logits;         // [T, E]
    uint16_t* x16;         // [T, H]
    float* xfactor;        // [T]
    int* hshift;           // [T k], smallest shift of the slot's runs
    uint8_t* h;            // [T k, I / 32] records
    float* part;           // [T k, H]
    int T, E, k, H, I;
    int renormalize;
};

__device__ __forceinline__ void fail(Shared* sm) {
    *reinterpret_cast<volatile int*>(&sm->abort) = 1;
    atomicOr(&g_mx_moe_error, 1u << kErrTimeout);
}

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Shared* sm) {
    const uint32_t b = smem_u32(bar);
    const unsigned long long t0 = clock64();
    for (;;) {
        if (mbar_try_wait_suspend(b, parity, kSuspendNs)) return true;
        if (*reinterpret_cast<volatile int*>(&sm->abort)) return false;
        if (clock64() - t0 > kWaitLimitCycles) {
            fail(sm);
            return false;
        }
    }
}
__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity, Shared* sm, int lane) {
    int ok = 1;
    if (lane == 0) ok = wait_bar(bar, parity, sm) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Grid barrier in two halves. control[0] counts arrivals, control[1] is the
// generation; the last CTA to arrive resets the count and then advances it.
__device__ __forceinline__ void grid_arrive(uint32_t* control) {
    __threadfence();
    if (atomicAdd(control, 1u) == gridDim.x - 1) {
        control[0] = 0u;
        __threadfence();
        atomicAdd(control + 1, 1u);
    }
}
__device__ __forceinline__ bool grid_wait(const uint32_t* control, uint32_t generation, Shared* sm) {
    const unsigned long long t0 = clock64();
    while (ld_acquire(control + 1) != generation) {
        if (*reinterpret_cast<volatile int*>(&sm->abort)) return false;
        if (clock64() - t0 > kWaitLimitCycles) {
            fail(sm);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// Untiled copy of `bytes` (a multiple of 16), global to shared.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// D = A * B on fp16 (FP32 result), accumulators starting at zero or at D.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// fp16 2^d in both halves, d <= 0; zero below the fp16 subnormals.
__device__ __forceinline__ uint32_t pow2_f16x2(int d) {
    const uint32_t h = d >= -14 ? static_cast<uint32_t>(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u;
    return h * 0x10001u;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// ---------------------------------------------------------------------------
// phase 0
// ---------------------------------------------------------------------------
// Logits of 16 experts x 8 tokens: the consumer warps take 32-element blocks of
// H in turn and their sums meet in shared memory.
__device__ void router_tile(const Params& p, Shared* sm, int e0, int t0, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int blocks = p.H >> 5;
    const bool ok0 = e0 + g < p.E, ok1 = e0 + g + 8 < p.E, okx = t0 + g < p.T;
    const uint4* r0 = reinterpret_cast<const uint4*>(p.router + static_cast<size_t>(ok0 ? e0 + g : 0) * p.H) + t;
    const uint4* r1 = reinterpret_cast<const uint4*>(p.router + static_cast<size_t>(ok1 ? e0 + g + 8 : 0) * p.H) + t;
    const uint4* xr = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(okx ? t0 + g : 0) * p.H) + t;
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int kBatch = 4;
    for (int b = warp; b < blocks; b += kConsumerWarps * kBatch) {
        uint4 a0[kBatch], a1[kBatch], xb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int c = b + i * kConsumerWarps;
            const uint4 z = make_uint4(0, 0, 0, 0);
            const bool in = c < blocks;
            a0[i] = in && ok0 ? __ldg(r0 + c * 4) : z;
            a1[i] = in && ok1 ? __ldg(r1 + c * 4) : z;
            xb[i] = in && okx ? __ldg(xr + c * 4) : z;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            mma_m16n8k16<true>(d, a0[i].x, a1[i].x, a0[i].y, a1[i].y, xb[i].x, xb[i].y);
            mma_m16n8k16<true>(d, a0[i].z, a1[i].z, a0[i].w, a1[i].w, xb[i].z, xb[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sm->red[warp][i][lane] = d[i];
    consumer_sync();
    const int i = warp;   // 4 warps finish one register of the fragment each
    if (i < 4) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) s += sm->red[w][i][lane];
        const int e = e0 + g + (i >> 1) * 8, tok = t0 + 2 * t + (i & 1);
        if (e < p.E && tok < p.T) __stcg(p.logits + static_cast<size_t>(tok) * p.E + e, s);
    }
    consumer_sync();
}

// One token's x as fp16, scaled by a power of two.
__device__ void convert_token(const Params& p, Shared* sm, int tok, int warp, int lane) {
    const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(tok) * p.H);
    const int n = p.H >> 3, tid = warp * 32 + lane;
    uint32_t m = 0;
    for (int i = tid; i < n; i += kConsumers) {
        const uint4 v = __ldg(src + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, max((w[j] >> 7) & 0xFFu, (w[j] >> 23) & 0xFFu));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) sm->red[warp][0][0] = __uint_as_float(m);
    consumer_sync();
    for (int w = 0; w < kConsumerWarps; ++w) m = max(m, __float_as_uint(sm->red[w][0][0]));
    const int c = mx::x_shift(m);
    uint4* dst = reinterpret_cast<uint4*>(p.x16 + static_cast<size_t>(tok) * p.H);
    for (int i = tid; i < n; i += kConsumers) {
        const uint4 v = __ldg(src + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = mx::x_to_f16(static_cast<uint16_t>(w[j]), c) |
                   static_cast<uint32_t>(mx::x_to_f16(static_cast<uint16_t>(w[j] >> 16), c)) << 16;
        __stcg(dst + i, make_uint4(o[0], o[1], o[2], o[3]));
    }
    if (tid == 0) __stcg(p.xfactor + tok, mx::x_unshift(c));
    for (int j = tid; j < p.k; j += kConsumers) __stcg(p.hshift + tok * p.k + j, 127);
    consumer_sync();
}

// ---------------------------------------------------------------------------
// phase 1
// ---------------------------------------------------------------------------
// One token's experts, by one warp: k rounds of a warp-wide maximum. Every
// round takes an expert not taken before whatever the logits hold (NaN too).
__device__ void pick_experts(const Params& p, Shared* sm, int tok, int lane) {
    constexpr int kPer = kMaxExperts / 32;
    const float* row = p.logits + static_cast<size_t>(tok) * p.E;
    float v[kPer];
    uint32_t key[kPer];   // ordered as the logits are; 0: absent or taken
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < p.E ? __ldcg(row + e) : 0.f;
        const uint32_t b = __float_as_uint(v[i] == 0.f ? 0.f : v[i]);   // -0 equals 0
        key[i] = e < p.E ? max((b >> 31) ? ~b : (b | 0x80000000u), 1u) : 0u;
    }
    float top = 0.f, sum = 0.f, mine = 0.f;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t high = __reduce_max_sync(0xffffffffu, best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == high ? static_cast<uint32_t>(lane + 32 * at) : ~0u);
        float l = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (e == static_cast<uint32_t>(lane + 32 * i)) {
                l = v[i];
                key[i] = 0;
            }
        l = __shfl_sync(0xffffffffu, l, e & 31);
        if (j == 0) top = l;
        const float ex = expf(l - top);
        sum += ex;
        if (lane == j) mine = ex;
        if (lane == 0) {
            sm->ids[tok * p.k + j] = static_cast<uint16_t>(e);
            atomicOr(&sm->mask[e], 1ull << tok);
        }
    }
    if (!p.renormalize) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < p.E) sum += expf(v[i] - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < p.k) sm->weight[tok * p.k + lane] = mine / sum;
}

// Prefix sums over the experts of their tokens and groups (one warp).
__device__ void number_groups(const Params& p, Shared* sm, int lane) {
    constexpr int kPer = kMaxExperts / 32;
    int n[kPer], tokens = 0, groups = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane * kPer + i;
        n[i] = e < p.E ? __popcll(sm->mask[e]) : 0;
        tokens += n[i];
        groups += (n[i] + kGroup - 1) / kGroup;
    }
    int at = tokens, ga = groups;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, at, o), b = __shfl_up_sync(0xffffffffu, ga, o);
        if (lane >= o) at += a, ga += b;
    }
    if (lane == 31) sm->groups = ga;
    at -= tokens;
    ga -= groups;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane * kPer + i;
        if (e < p.E) {
            sm->offset[e] = static_cast<uint16_t>(at);
            for (int q = 0; q < n[i]; q += kGroup, ++ga) {
                sm->group[ga] = static_cast<uint32_t>(e) | static_cast<uint32_t>(min(kGroup, n[i] - q)) << 16;
                sm->first[ga] = static_cast<uint16_t>(at + q);
            }
        }
        at += n[i];
    }
}

// ---------------------------------------------------------------------------
// phases 2 and 3: the stream of stages
// ---------------------------------------------------------------------------
// A 32-row block of 64 columns against the group's rows, added to acc
// [8-token tile][16-column tile][fragment]. kH: the rows are runs of h with
// shifts of their own, `align` holds the rows' common shift.
template <bool kH>
__device__ __forceinline__ void block_products(float (&acc)[2][4][4], uint32_t stage, int c, bool two, int g, int t,
                                               const int (&align)[2]) {
    const int row = 4 * c + t;
    const uint32_t chunk = static_cast<uint32_t>((g >> 1) | ((g & 1) << 2));
    const uint32_t waddr = stage + row * 128 + ((chunk ^ (row & 7)) << 4);
    const uint32_t saddr = stage + 2 * kBoxBytes + c * 32 + chunk * 4;
    const uint32_t xaddr = stage + 2 * kBoxBytes + 2 * kScaleBoxBytes + g * kXStride + c * (kH ? kHRecord : 64) + t * 16;
    uint32_t b[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        if (n == 1 && !two) break;
        const uint4 v = ld_shared_v4(xaddr + n * 8 * kXStride);
        b[n][0] = v.x, b[n][1] = v.y, b[n][2] = v.z, b[n][3] = v.w;
        if constexpr (kH) {
            const int shift = static_cast<int>(ld_shared_u32(xaddr + n * 8 * kXStride - t * 16 + 64));
            const uint32_t f = pow2_f16x2(min(align[n] - shift, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i) b[n][i] = hmul2(b[n][i], f);
        }
    }
#pragma unroll
    for (int box = 0; box < 2; ++box) {
        const uint4 w = ld_shared_v4(waddr + box * kBoxBytes);
        const uint32_t e4 = ld_shared_u32(saddr + box * kScaleBoxBytes);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t lo[4], hi[4];
            mx::e2m1x8_to_f16x2(words[2 * m], lo);
            mx::e2m1x8_to_f16x2(words[2 * m + 1], hi);
            const float s0 = mx::scale_f32((e4 >> (16 * m)) & 0xFFu), s1 = mx::scale_f32((e4 >> (16 * m + 8)) & 0xFFu);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if (n == 1 && !two) break;
                float d[4];
                mma_f16_zero(d, lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
                mma_m16n8k16<false>(d, lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
                float(&a)[4] = acc[n][2 * box + m];
                a[0] = fmaf(d[0], s0, a[0]);
                a[1] = fmaf(d[1], s0, a[1]);
                a[2] = fmaf(d[2], s1, a[2]);
                a[3] = fmaf(d[3], s1, a[3]);
            }
        }
    }
}

// A warp's sums to shared memory: slot [tile][token parity][box][column % 4],
// at the lane that holds them.
__device__ __forceinline__ void store_sums(Shared* sm, const float (&acc)[2][4][4], bool two, int warp, int lane) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        if (n == 1 && !two) break;
#pragma unroll
        for (int q = 0; q < 4; ++q)       // 16-column tile: box q >> 1, columns 2 (q & 1) and + 1 of every four
#pragma unroll
            for (int i = 0; i < 4; ++i)   // fragment: column i >> 1, token parity i & 1
                sm->red[warp][n * 16 + (i & 1) * 8 + (q >> 1) * 4 + (q & 1) * 2 + (i >> 1)][lane] = acc[n][q][i];
    }
}

// The sum over the warps of token n, column `col` (0..31) of box `box`.
__device__ __forceinline__ float load_sum(const Shared* sm, int n, int box, int col) {
    const int chunk = col >> 2;
    const int g = ((chunk & 3) << 1) | (chunk >> 2);
    const int slot = (n >> 3) * 16 + (n & 1) * 8 + box * 4 + (col & 3);
    const int at = g * 4 + ((n & 7) >> 1);
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w) s += sm->red[w][slot][at];
    return s;
}

__global__ void __launch_bounds__(kThreads, 1)
moe_kernel(const __grid_constant__ CUtensorMap tw13, const __grid_constant__ CUtensorMap te13,
           const __grid_constant__ CUtensorMap tw2, const __grid_constant__ CUtensorMap te2, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared* sm = reinterpret_cast<Shared*>(ring + kStages * kStagePitch);
    const uint32_t ring_base = smem_u32(ring);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grid = gridDim.x, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&sm->full[s]), 1);
            mbar_init(smem_u32(&sm->empty[s]), kConsumerWarps / 2);
        }
        mbar_init(smem_u32(&sm->phase3), 1);
        sm->abort = 0;
        sm->generation = ld_acquire(p.control + 1);
        fence_mbar_init();
        tma_prefetch_desc(&tw13);
        tma_prefetch_desc(&te13);
        tma_prefetch_desc(&tw2);
        tma_prefetch_desc(&te2);
    }
    for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) sm->mask[e] = 0ull;
    __syncthreads();

    // ---------------------------------------------------------------- phase 0
    if (warp < kConsumerWarps) {
        const int etiles = (p.E + 15) >> 4, tiles = etiles * ((p.T + 7) >> 3);
        for (int u = cta; u < tiles + p.T; u += grid) {
            if (u < tiles)
                router_tile(p, sm, (u % etiles) * 16, (u / etiles) * 8, warp, lane);
            else
                convert_token(p, sm, u - tiles, warp, lane);
        }
        fence_proxy_async_global();   // x16 is read by bulk copies
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        grid_arrive(p.control);
        grid_wait(p.control, sm->generation + 1, sm);
    }
    __syncthreads();

    // ---------------------------------------------------------------- phase 1
    const bool alive = *reinterpret_cast<volatile int*>(&sm->abort) == 0;
    if (alive) {
        for (int tok = warp; tok < p.T; tok += kThreads / 32) pick_experts(p, sm, tok, lane);
        __syncthreads();
        if (warp == 0) number_groups(p, sm, lane);
        __syncthreads();
        for (int s = threadIdx.x; s < p.T * p.k; s += kThreads) {
            const int e = sm->ids[s];
            sm->list[sm->offset[e] + __popcll(sm->mask[e] & ((1ull << (s / p.k)) - 1))] = static_cast<uint16_t>(s);
        }
        __syncthreads();
    }
    const int groups = alive ? sm->groups : 0;
    const int items2 = groups * (p.I >> 5), items3 = groups * ((p.H + 63) >> 6);
    const int blocks2 = p.H >> 5, blocks3 = p.I >> 5;                    // 32-row blocks of K
    const int steps2 = (blocks2 + kBlocks - 1) / kBlocks, steps3 = (blocks3 + kBlocks - 1) / kBlocks;

    if (warp == kConsumerWarps) {
        // ------------------------------------------------------------ producer
        fence_proxy_async_global();
        bool ok = true;
        // the CTA's stages of a phase in order, and how many each set's ring has seen
        struct Cursor {
            int item, ks;
            uint32_t used[2];
        };
        auto set_of = [&](const Cursor& u) { return (u.ks + u.item / groups) & 1; };
        auto slot_of = [&](const Cursor& u) {
            const int q = set_of(u);
            return q * kSetStages + static_cast<int>(u.used[q] % kSetStages);
        };
        auto advance = [&](Cursor& u, int steps) {
            ++u.used[set_of(u)];
            if (++u.ks == steps) u.ks = 0, u.item += grid;
        };
        // weights of one stage (lane 0; waits for the stage to be free and announces all its bytes)
        auto weights = [&](bool second, const Cursor& u) {
            const int s = slot_of(u);
            if (!warp_wait_bar(&sm->empty[s], (u.used[set_of(u)] / kSetStages & 1u) ^ 1u, sm, lane)) return false;
            if (lane == 0) {
                const uint32_t gr = sm->group[u.item % groups];
                const int e = gr & 0xFFFFu, n = gr >> 16, cb = u.item / groups;
                const int nb = min(kBlocks, (second ? blocks3 : blocks2) - u.ks * kBlocks);
                const uint32_t bar = smem_u32(&sm->full[s]), dst = ring_base + s * kStagePitch;
                mbar_arrive_expect_tx(bar, 2 * kBoxBytes + 2 * kScaleBoxBytes + n * nb * (second ? kHRecord : 64));
                const int c0 = second ? cb * 64 : cb * 32, c1 = second ? cb * 64 + 32 : p.I + cb * 32;
                const int kb = e * (second ? blocks3 : blocks2) + u.ks * kBlocks;   // 32-row block of the stack
                const CUtensorMap* tw = second ? &tw2 : &tw13;
                const CUtensorMap* te = second ? &te2 : &te13;
                tma_load_2d(dst, tw, c0, kb * 4, bar);
                tma_load_2d(dst + kBoxBytes, tw, c1, kb * 4, bar);
                tma_load_2d(dst + 2 * kBoxBytes, te, c0, kb, bar);
                tma_load_2d(dst + 2 * kBoxBytes + kScaleBoxBytes, te, c1, kb, bar);
            }
            return true;
        };
        // activation rows of the stage, one copy per lane
        auto rows = [&](bool second, const Cursor& u) {
            const int s = slot_of(u), gi = u.item % groups;
            if (lane < static_cast<int>(sm->group[gi] >> 16)) {
                const int slot = sm->list[sm->first[gi] + lane];
                const int nb = min(kBlocks, (second ? blocks3 : blocks2) - u.ks * kBlocks);
                const uint32_t dst =
                    ring_base + s * kStagePitch + 2 * kBoxBytes + 2 * kScaleBoxBytes + lane * kXStride;
                if (second)
                    bulk_load(dst, p.h + (static_cast<size_t>(slot) * blocks3 + u.ks * kBlocks) * kHRecord,
                              nb * kHRecord, smem_u32(&sm->full[s]));
                else
                    bulk_load(dst, p.x16 + static_cast<size_t>(slot / p.k) * p.H + u.ks * kStepK, nb * 64,
                              smem_u32(&sm->full[s]));
            }
        };
        Cursor u{cta, 0, {0u, 0u}};
        while (u.item < items2 && ok) {
            ok = weights(false, u);
            if (!ok) break;
            rows(false, u);
            advance(u, steps2);
        }
        // the rings' worth of phase 3 weights before the barrier, their rows after it
        u.item = cta;
        u.ks = 0;
        const Cursor start = u;
        while (u.item < items3 && ok) {
            const int q = set_of(u);
            if (u.used[q] - start.used[q] == kSetStages) break;
            ok = weights(true, u);
            if (ok) advance(u, steps3);
        }
        if (ok && alive) {
            int go = 1;
            if (lane == 0) go = grid_wait(p.control, sm->generation + 2, sm) ? 1 : 0;
            go = __shfl_sync(0xffffffffu, go, 0);
            __syncwarp();
            ok = go != 0;
            fence_proxy_async_global();
            if (lane == 0 && ok) mbar_arrive(smem_u32(&sm->phase3));
        }
        if (ok)
            for (Cursor v = start; v.item != u.item || v.ks != u.ks; advance(v, steps3)) rows(true, v);
        while (u.item < items3 && ok) {
            ok = weights(true, u);
            if (!ok) break;
            rows(true, u);
            advance(u, steps3);
        }
        // copies in flight land before the CTA's shared memory is given back
        if (lane == 0) {
            const unsigned long long t0 = clock64();
            for (int q = 0; q < 2; ++q)
                for (uint32_t i = u.used[q] > kSetStages ? u.used[q] - kSetStages : 0; i < u.used[q]; ++i)
                    while (!mbar_try_wait(smem_u32(&sm->full[q * kSetStages + i % kSetStages]), i / kSetStages & 1u) &&
                           clock64() - t0 < kWaitLimitCycles) {
                    }
        }
    } else {
        // ------------------------------------------------------------ consumers
        const int g = lane >> 2, t = lane & 3;
        const int set = warp >> 3, c = warp & 7;
        uint32_t used = 0;   // stages of the set's ring so far
        bool ok = alive;
        const int no_align[2] = {0, 0};

        // ---- phase 2
        for (int item = cta; item < items2; item += grid) {
            const int gi = item % groups, cb = item / groups;
            const int n = sm->group[gi] >> 16;
            float acc[2][4][4];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][b][i] = 0.f;
            for (int ks = (cb ^ set) & 1; ks < steps2; ks += 2, ++used) {
                const int s = set * kSetStages + static_cast<int>(used % kSetStages);
                if (!ok || !warp_wait_bar(&sm->full[s], used / kSetStages & 1u, sm, lane)) {
                    ok = false;
                    continue;
                }
                if (ks * kBlocks + c < blocks2)
                    block_products<false>(acc, ring_base + s * kStagePitch, c, n > 8, g, t, no_align);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm->empty[s]));
            }
            consumer_sync();   // the previous item's sums have been read
            store_sums(sm, acc, n > 8, warp, lane);
            consumer_sync();
            if (warp < n && ok) {
                const int slot = sm->list[sm->first[gi] + warp];
                const float f = __ldcg(p.xfactor + slot / p.k);
                const float gate = load_sum(sm, warp, 0, lane) * f, up = load_sum(sm, warp, 1, lane) * f;
                const float h = silu(gate) * up;
                const int shift = mx::x_shift(__reduce_max_sync(0xffffffffu, (__float_as_uint(h) >> 23) & 0xFFu));
                uint8_t* rec = p.h + (static_cast<size_t>(slot) * blocks3 + cb) * kHRecord;
                const float scaled = h * __uint_as_float(static_cast<uint32_t>(shift + 127) << 23);
                __stcg(reinterpret_cast<unsigned short*>(rec) + lane, __half_as_ushort(__float2half_rn(scaled)));
                if (lane == 0) {
                    __stcg(reinterpret_cast<int*>(rec + 64), shift);
                    atomicMin(p.hshift + slot, shift);
                }
            }
        }
        fence_proxy_async_global();   // h is read by bulk copies
        consumer_sync();
        if (threadIdx.x == 0 && alive) grid_arrive(p.control);

        // ---- phase 3
        if (ok) ok = warp_wait_bar(&sm->phase3, 0, sm, lane);
        for (int item = cta; item < items3; item += grid) {
            const int gi = item % groups, cb = item / groups;
            const int n = sm->group[gi] >> 16;
            int align[2] = {0, 0};
#pragma unroll
            for (int a = 0; a < 2; ++a)
                if (ok && g + 8 * a < n) align[a] = __ldcg(p.hshift + sm->list[sm->first[gi] + g + 8 * a]);
            float acc[2][4][4];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][b][i] = 0.f;
            for (int ks = (cb ^ set) & 1; ks < steps3; ks += 2, ++used) {
                const int s = set * kSetStages + static_cast<int>(used % kSetStages);
                if (!ok || !warp_wait_bar(&sm->full[s], used / kSetStages & 1u, sm, lane)) {
                    ok = false;
                    continue;
                }
                if (ks * kBlocks + c < blocks3)
                    block_products<true>(acc, ring_base + s * kStagePitch, c, n > 8, g, t, align);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm->empty[s]));
            }
            consumer_sync();
            store_sums(sm, acc, n > 8, warp, lane);
            consumer_sync();
            if (warp < n && ok) {
                const int slot = sm->list[sm->first[gi] + warp], tok = slot / p.k;
                const float f = mx::x_unshift(__ldcg(p.hshift + slot)), pw = sm->weight[slot];
                float* part = p.part + static_cast<size_t>(slot) * p.H + cb * 64;
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (cb * 64 + b * 32 < p.H)
                        __stcg(part + b * 32 + lane, load_sum(sm, warp, b, lane) * f * pw);
                __threadfence();
                __syncwarp();
                uint32_t* ticket = p.control + 2 + static_cast<size_t>(cb) * kMoeMaxTokens + tok;
                uint32_t last = 0;
                if (lane == 0) last = atomicAdd(ticket, 1u) == static_cast<uint32_t>(p.k - 1);
                last = __shfl_sync(0xffffffffu, last, 0);
                if (last) {
                    __threadfence();
                    const float* src = p.part + static_cast<size_t>(tok) * p.k * p.H + cb * 64 + lane;
                    float sum[2] = {0.f, 0.f};
                    for (int q = 0; q < p.k; ++q)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            if (cb * 64 + b * 32 < p.H) sum[b] += __ldcg(src + static_cast<size_t>(q) * p.H + b * 32);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (cb * 64 + b * 32 < p.H)
                            p.y[static_cast<size_t>(tok) * p.H + cb * 64 + b * 32 + lane] =
                                __bfloat16_as_ushort(__float2bfloat16_rn(sum[b]));
                    if (lane == 0) *ticket = 0u;
                }
            }
        }
    }
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

struct Layout {
    size_t logits, x16, xfactor, hshift, h, part, total;
};
Layout layout(int T, int E, int k, int H, int I) {
    Layout l;
    size_t at = kMoeControlBytes;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    const size_t slots = static_cast<size_t>(T) * k;
    l.logits = take(static_cast<size_t>(T) * E * 4);
    l.x16 = take(static_cast<size_t>(T) * H * 2);
    l.xfactor = take(static_cast<size_t>(T) * 4);
    l.hshift = take(slots * 4);
    l.h = take(slots * (I / 32) * kHRecord);
    l.part = take(slots * H * 4);
    l.total = at;
    return l;
}

}  // namespace

size_t mx_moe_workspace_bytes(int T, int E, int k, int H, int I) { return layout(T, E, k, H, I).total; }

cudaError_t launch_mx_moe(const MxMoeArgs& a, void* workspace, const DeviceProps& dp, cudaStream_t s) {
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(moe_kernel), dp.device, kSmemBytes);
        e != cudaSuccess)
        return e;
    CUtensorMap tw13, te13, tw2, te2;
    const uint64_t E = a.E, H = a.H, I = a.I;
    if (!encode_2d(&tw13, CU_TENSOR_MAP_DATA_TYPE_INT32, a.w13, 2 * I, E * (H / 8), 2 * I * 4, 32, kStepK / 8,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&te13, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.e13, 2 * I, E * (H / 32), 2 * I, 32, kBlocks,
                   CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_2d(&tw2, CU_TENSOR_MAP_DATA_TYPE_INT32, a.w2, H, E * (I / 8), H * 4, 32, kStepK / 8,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&te2, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.e2, H, E * (I / 32), H, 32, kBlocks,
                   CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Layout l = layout(a.T, a.E, a.k, a.H, a.I);
    Params p;
    p.x = static_cast<const uint16_t*>(a.x);
    p.router = static_cast<const uint16_t*>(a.router);
    p.y = static_cast<uint16_t*>(a.y);
    p.control = reinterpret_cast<uint32_t*>(ws);
    p.logits = reinterpret_cast<float*>(ws + l.logits);
    p.x16 = reinterpret_cast<uint16_t*>(ws + l.x16);
    p.xfactor = reinterpret_cast<float*>(ws + l.xfactor);
    p.hshift = reinterpret_cast<int*>(ws + l.hshift);
    p.h = ws + l.h;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.T = a.T;
    p.E = a.E;
    p.k = a.k;
    p.H = a.H;
    p.I = a.I;
    p.renormalize = a.renormalize ? 1 : 0;
    // no more CTAs than the larger of the two expert phases can use
    const long long slots = static_cast<long long>(a.T) * a.k;
    const long long want = slots * std::max<long long>(a.I / 32, (a.H + 63) / 64);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max<long long>(1, std::min<long long>(want, dp.sms))));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    // the CTAs wait for one another at the grid barriers: all of them are resident together or the launch fails
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_kernel, tw13, te13, tw2, te2, p);
}

cudaError_t read_and_clear_mx_moe_error(uint32_t* out) {
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_mx_moe_error, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_mx_moe_error, &zero, sizeof(zero));
    }
    *out = v;
    return e;
}

}  // namespace w4a16
