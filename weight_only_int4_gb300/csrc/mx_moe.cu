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
//   0  router logits (warp-level bf16 MMAs, 16 experts x 8 tokens and a part of
//      H a CTA) and x as fp16 with one power-of-two factor per token
//      -- grid barrier --
//   1  every CTA picks the experts itself (a warp per token) and lists the
//      tokens of each expert in groups of up to 8
//   2  items (group, 32 gate columns and their 32 up columns): products, SwiGLU,
//      h as fp16 with one power of two per 32 columns
//      -- grid barrier (weights of phase 3 are already on their way) --
//   3  items (group, 64 columns of y): products, each token's part from each of
//      its k experts to global memory (L2)
//      -- grid barrier --
//   4  the k parts of every y added in order: deterministic
//
// A CTA is two producer warps, sixteen consumer warps and two epilogue warps
// around a ring of stages. A stage is 512 rows of K by 64 columns of codes (two
// TMA boxes of 32 columns, 128-byte swizzle), their exponent bytes and the same
// 512 elements of the group's activation rows. Two sets of eight consumer
// warps, each with a producer and half of the ring, take alternate stages of the
// CTA's items; an item's parts are added from the set of its first stage on, so a
// token's sums are formed in the same order whatever else the call holds. A warp
// converts four 32-row blocks of one box: a lane's 16-byte load holds eight
// consecutive codes of each of four columns, which become fp16 pairs by the
// hardware's exact conversion and serve as the A operand of warp-level MMAs
// (columns of W as MMA rows, tokens as MMA columns), x as B; K is permuted alike
// on both sides, so neither needs a shuffle. A block's FP32 products are scaled
// by the columns' 2^(e - 127) as they are added up. At the end of an item the
// warps leave their sums in a buffer and go on; the epilogue warps, two tokens
// each at a time, add the eight parts in order and finish the item beside the
// next ones.
//
// Measured in a graph of calls on operands larger than L2: 1 token, 4 of 32
// experts of 2048 x 1024 14.5..17.0 us; 16 tokens, 8 of 64 of 4096 x 1024 80..82
// (the weights' bytes take 56 at the copy bandwidth); 64 tokens, 8 of 128 of
// 2048 x 1024 102..105 (63). What bounds the last one: 18.6 us are everything but the
// items (barriers, router, top-k, the last sums). Without the products the call
// takes 87 us, without the loads as long as with them, without loads and epilogue
// 84: the consumer warps' instructions, and the epilogue warps' beside them. More
// warps lose more by their smaller share of the registers than they win: a third
// set of consumers at 72 registers took 119..124 us against 109, four epilogue
// warps at 80 registers 111..113 against 102.
//
// Activations in fp16: a token's x, and every run of 32 values of h, is
// multiplied by the power of two that brings its largest magnitude just below
// 2^15; the inverse goes into the FP32 scaling (per token at the end, per run
// with the block's). Values within 2^-29 of the largest convert exactly or, for
// h, with fp16's 11 bits; smaller ones lose at most 2^-39 of the largest.
//
// The gate and up sums are kept without the token's factor as long as every
// exponent byte is in 64..191: below 2^(23 + 64 + 11), they cannot overflow
// whatever the factor is. From the first other byte on a warp keeps its sums of
// the item in true units, factor and exponent applied to each block's products
// in the order that stays in range, and marks them for the epilogue.
//
// Waits are bounded (about two seconds); on expiry the kernel records the
// timeout in a device word, every role stops, copies in flight are waited for
// (bounded) and the kernel returns.
#include "internal.h"
#include "mxfp4.cuh"
#include "ptx.cuh"
#include "tmap.h"

#include <algorithm>
#include <type_traits>

namespace w4a16 {

__device__ unsigned int g_mx_moe_error = 0;

namespace {

constexpr int kConsumerWarps = 16, kEpilogues = 2, kProducers = 2;
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kThreads = kConsumers + (kEpilogues + kProducers) * 32;
constexpr int kStepK = 512;              // rows of K per stage
constexpr int kBlocks = kStepK / 32;
constexpr int kWarpBlocks = 4;           // consecutive 32-row blocks of a box that a warp converts
constexpr int kSlices = kBlocks / kWarpBlocks;
constexpr int kMaxExperts = kMoeMaxExperts;
constexpr int kMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
static_assert(kMaxSlots <= 1 << 10 && kMoeMaxTokens <= 1 << 6, "a list entry's 16 bits");
constexpr uint32_t kBoxBytes = kStepK / 8 * 128;     // 64 word rows x 32 columns
constexpr uint32_t kScaleBoxBytes = kBlocks * 32;
constexpr uint32_t kWeightBytes = 2 * kBoxBytes + 2 * kScaleBoxBytes;
static_assert(kWeightBytes % 1024 == 0, "swizzled boxes start 1024-byte aligned");
// A run of h: 32 fp16 values, then the FP32 factor 2^-shift four times: lanes that read the factors of rows 0, 2, 4, 6
// (or 1, 3, 5, 7), whose strides share a bank, take a copy each.
constexpr uint32_t kHRecord = 80;
constexpr uint32_t kXStride = kBlocks * kHRecord + 64;   // a row of a stage; two rows' 64 bytes hit different banks
constexpr int kRedPitch = 33;            // floats per slot of a warp's partial sums
constexpr unsigned long long kWaitLimitCycles = 4000000000ull;   // ~2 s at 2 GHz
constexpr unsigned int kErrTimeout = 9u;

// Tokens of an expert taken together: one MMA's columns. With groups of 16 the
// ring falls from six stages to four and the accumulators spill: 64 tokens of
// 2048 x 1024 took 174 us against 108 with 4 tokens per expert on average, 86
// against 76 with 16 and 76 against 71 with 32, where the further groups' weights
// come from L2.
constexpr int kGroup = 8;
constexpr int kRedSlots = 8;                     // [token parity][column % 4]
constexpr int kBuffers = 2;                      // of partial sums
constexpr int kSetStages = 3;                    // half of the ring
constexpr int kStages = 2 * kSetStages;
constexpr uint32_t kRowBytes = kGroup * kXStride;

struct __align__(16) Shared {
    float red[kBuffers][kConsumerWarps][kRedSlots][kRedPitch];
    uint32_t factored[kBuffers][4];   // byte w: warp w's gate and up sums hold the token's factor
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t sums[kBuffers];          // a buffer of partial sums is complete
    uint64_t taken[kBuffers];         // ... and has been read
    uint64_t phase3;                     // h of every CTA is visible
    uint64_t phase4;                     // the parts of y are
    uint32_t mask[kMaxExperts][2];       // tokens of each expert
    float weight[kMaxSlots];             // of slot t * k + j
    uint32_t group[kMaxSlots];           // expert | count << 16
    uint16_t first[kMaxSlots];           // the group's first entry in `list`
    uint16_t list[kMaxSlots];            // slot | token << 10, ordered by expert, then token
    float xfactor[kMoeMaxTokens];
    uint16_t ids[kMaxSlots];             // expert of slot t * k + j
    uint16_t offset[kMaxExperts];
    uint32_t scan[kMaxExperts / 32];
    int groups;
    uint32_t epoch;
    int abort;
};
constexpr size_t kSmemBytes = 1024 + kStages * (kWeightBytes + kRowBytes) + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct Params {
    const uint16_t* x;
    const uint16_t* router;
    uint16_t* y;
    uint32_t* control;     // epoch, then two sets of barrier counts
    float* logits;         // [splits, T, E], the parts of H in order
    uint16_t* x16;         // [T, H]
    float* xfactor;        // [T]
    uint8_t* h;            // [T k, I / 32] records
    float* part;           // [T k, H]
    int T, E, k, H, I;
    int splits;            // parts of H in the router product
    int renormalize;
};
constexpr int kBarriers = 3;
constexpr int kMaxSplits = 4;
constexpr int kRouterDepth = 1024;   // elements of H in a part of the router product

__device__ __forceinline__ void fail(volatile int* abort) {
    *abort = 1;
    atomicOr(&g_mx_moe_error, 1u << kErrTimeout);
}

// A poll takes 111 cycles (measured, phase complete). With one lane polling and
// a shuffle of its verdict a wait took 266; the whole warp polling in one
// instruction and voting takes 131.
__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
    const uint32_t b = smem_u32(bar);
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    const unsigned long long t0 = clock64();
    for (;;) {
        // a few polls between looks at the clock
        for (int i = 0; i < 32; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
        if (__any_sync(0xffffffffu, clock64() - t0 > kWaitLimitCycles)) {
            fail(abort);
            return false;
        }
    }
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Grid barriers. A call uses one of two sets of counts, by the parity of the
// call's epoch, and zeroes the other set (the previous call's); the epoch
// advances once every CTA has passed the first barrier, so all have read it.
__device__ __forceinline__ void grid_arrive(uint32_t* count) {
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
}
__device__ __forceinline__ bool grid_wait(const uint32_t* count, volatile int* abort) {
    const unsigned long long t0 = clock64();
    while (ld_acquire(count) != gridDim.x) {
        if (*abort) return false;
        if (clock64() - t0 > kWaitLimitCycles) {
            fail(abort);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// D = A * B on fp16 (FP32 result), accumulators starting at zero or at D.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// g / (1 + exp(-g)), with the numerator and denominator multiplied by exp(g)
// where g is negative: the divisor stays in [1, 2] (or NaN), where the fast
// division is within 2 units in the last place. It has no branch, so that the
// epilogue's two tokens overlap.
__device__ __forceinline__ float silu(float g) {
    const float t = expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * t : g, 1.f + t);
}

// ---------------------------------------------------------------------------
// phase 0
// ---------------------------------------------------------------------------
// Logits of 16 experts x 8 tokens over part `part` of H: the consumer warps take
// 32-element blocks in turn and their sums meet in shared memory. Parts of 1024
// (up to four): 16 tokens, 64 experts of 4096 x 1024 take 79.2 us against 79.8 in
// parts of 2048 (undivided it cost 2 us more), 4 tokens, 128 experts of
// 2048 x 768 32.7 against 33.6; only 64 tokens with 128 experts, whose tiles alone
// fill the GPU, pay for it (103.1 against 102.3; 105.0 in parts of 512).
__device__ void router_tile(const Params& p, float (*scratch)[4][32], int e0, int t0, int part, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int all = p.H >> 5, first = all * part / p.splits, blocks = all * (part + 1) / p.splits;
    const bool ok0 = e0 + g < p.E, ok1 = e0 + g + 8 < p.E, okx = t0 + g < p.T;
    const uint4* r0 = reinterpret_cast<const uint4*>(p.router + static_cast<size_t>(ok0 ? e0 + g : 0) * p.H) + t;
    const uint4* r1 = reinterpret_cast<const uint4*>(p.router + static_cast<size_t>(ok1 ? e0 + g + 8 : 0) * p.H) + t;
    const uint4* xr = reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(okx ? t0 + g : 0) * p.H) + t;
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    constexpr int kBatch = 4;
    for (int b = first + warp; b < blocks; b += kConsumerWarps * kBatch) {
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
    for (int i = 0; i < 4; ++i) scratch[warp][i][lane] = d[i];
    consumer_sync();
    const int i = warp;   // 4 warps finish one register of the fragment each
    if (i < 4) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumerWarps; ++w) s += scratch[w][i][lane];
        const int e = e0 + g + (i >> 1) * 8, tok = t0 + 2 * t + (i & 1);
        if (e < p.E && tok < p.T) __stcg(p.logits + (static_cast<size_t>(part) * p.T + tok) * p.E + e, s);
    }
    consumer_sync();
}

// One token's x as fp16, scaled by a power of two.
__device__ void convert_token(const Params& p, float (*scratch)[4][32], int tok, int warp, int lane) {
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
    if (lane == 0) scratch[warp][0][0] = __uint_as_float(m);
    consumer_sync();
    for (int w = 0; w < kConsumerWarps; ++w) m = max(m, __float_as_uint(scratch[w][0][0]));
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
    consumer_sync();
}

// ---------------------------------------------------------------------------
// phase 1
// ---------------------------------------------------------------------------
// FP32 to unsigned keys of the same order, never 0, and back. (-0 counts as 0;
// a NaN sorts above every number or below, by its sign.)
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
    return max((b >> 31) ? ~b : (b | 0x80000000u), 1u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

// One token's experts, by one warp. Each lane sorts the logits it holds (experts
// lane, lane + 32, ...), then k rounds take the largest head of the 32 lists,
// the lower expert where heads are equal. Every round takes an expert that was
// not taken before, whatever the logits hold.
template <int kPer>
__device__ __forceinline__ void pick_experts(const Params& p, Shared* sm, int tok, int lane) {
    const float* row = p.logits + static_cast<size_t>(tok) * p.E;
    uint32_t key[kPer], id[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        id[i] = lane + 32 * i;
        key[i] = 0u;   // absent
        if (id[i] < static_cast<uint32_t>(p.E)) {
            float v = __ldcg(row + id[i]);
            if (p.splits > 1) {
                float part[kMaxSplits - 1];
#pragma unroll
                for (int q = 1; q < kMaxSplits; ++q)
                    part[q - 1] = q < p.splits ? __ldcg(row + static_cast<size_t>(q) * p.T * p.E + id[i]) : 0.f;
#pragma unroll
                for (int q = 1; q < kMaxSplits; ++q) v += part[q - 1];
            }
            key[i] = order_key(v);
        }
    }
    float total = 0.f;
    if (!p.renormalize) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) m = max(m, key[i]);
        const float top = key_value(__reduce_max_sync(0xffffffffu, m));
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i]) total += expf(key_value(key[i]) - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    // neighbours exchange only where the later one is larger: equal keys keep their order
#pragma unroll
    for (int r = 0; r < kPer; ++r)
#pragma unroll
        for (int i = r & 1; i + 1 < kPer; i += 2) {
            const bool swap = key[i + 1] > key[i];
            const uint32_t k0 = key[i], i0 = id[i];
            key[i] = swap ? key[i + 1] : k0;
            id[i] = swap ? id[i + 1] : i0;
            key[i + 1] = swap ? k0 : key[i + 1];
            id[i + 1] = swap ? i0 : id[i + 1];
        }
    uint32_t won = 0, expert = 0;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t high = __reduce_max_sync(0xffffffffu, key[0]);
        const bool tied = key[0] == high;
        const uint32_t who = __ballot_sync(0xffffffffu, tied);
        uint32_t e = __shfl_sync(0xffffffffu, id[0], __ffs(who) - 1);
        if (who & (who - 1)) e = __reduce_min_sync(0xffffffffu, tied ? id[0] : ~0u);
        if (tied && id[0] == e) {
#pragma unroll
            for (int i = 0; i + 1 < kPer; ++i) key[i] = key[i + 1], id[i] = id[i + 1];
            key[kPer - 1] = 0;
        }
        if (lane == j) won = high, expert = e;
    }
    // lane j holds the token's j-th choice
    const float top = __shfl_sync(0xffffffffu, key_value(won), 0);
    const float ex = lane < p.k ? expf(key_value(won) - top) : 0.f;
    float sum = ex;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < p.k) {
        sm->weight[tok * p.k + lane] = ex / (p.renormalize ? sum : total);
        sm->ids[tok * p.k + lane] = static_cast<uint16_t>(expert);
        atomicOr(&sm->mask[expert][tok >> 5], 1u << (tok & 31));
    }
}

// Tokens and groups of every expert, numbered in the experts' order: one thread
// per expert, prefix sums over packed counts (tokens | groups << 16). All
// threads of the CTA.
__device__ __forceinline__ void number_groups(const Params& p, Shared* sm) {
    const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
    int n = 0;
    uint32_t own = 0, at = 0;
    if (e < kMaxExperts) {
        n = e < p.E ? __popc(sm->mask[e][0]) + __popc(sm->mask[e][1]) : 0;
        own = at = static_cast<uint32_t>(n) | static_cast<uint32_t>((n + kGroup - 1) / kGroup) << 16;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += v;
        }
        if (lane == 31) sm->scan[warp] = at;
    }
    __syncthreads();
    if (e < kMaxExperts) {
#pragma unroll
        for (int w = 0; w < kMaxExperts / 32; ++w)
            if (w < warp) at += sm->scan[w];
        if (e == kMaxExperts - 1) sm->groups = static_cast<int>(at >> 16);
        at -= own;
        sm->offset[e] = static_cast<uint16_t>(at & 0xFFFFu);
        int gi = static_cast<int>(at >> 16);
        for (int q = 0; q < n; q += kGroup, ++gi) {
            sm->group[gi] = static_cast<uint32_t>(e) | static_cast<uint32_t>(min(kGroup, n - q)) << 16;
            sm->first[gi] = static_cast<uint16_t>((at & 0xFFFFu) + q);
        }
    }
    __syncthreads();
    // a slot's place among its expert's: the tokens before it
    for (int s = threadIdx.x; s < p.T * p.k; s += kThreads) {
        const int ex = sm->ids[s], tok = s / p.k;
        const unsigned long long m = sm->mask[ex][0] | static_cast<unsigned long long>(sm->mask[ex][1]) << 32;
        sm->list[sm->offset[ex] + __popcll(m & ((1ull << tok) - 1))] = static_cast<uint16_t>(s | tok << 10);
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// phases 2 and 3
// ---------------------------------------------------------------------------
// A CTA's items, every grid-th: group and column block without a division each.
struct Walk {
    int group, column, groups, columns, cols;
    __device__ __forceinline__ Walk(int item, int grid, int cols)
        : group(item / cols), column(item - group * cols), groups(grid / cols), columns(grid - groups * cols),
          cols(cols) {}
    __device__ __forceinline__ void next() {
        group += groups;
        column += columns;
        if (column >= cols) column -= cols, ++group;
    }
};

// What a lane takes of kCount 32-row blocks of one box of a stage, from block
// c + first on: words of codes, the 16 bytes of its row of activations at `rows`
// and, where the rows are records of h (kH), the factors of its tokens 2 t and
// 2 t + 1 at `factors`.
template <bool kH, int kCount>
struct Operands {
    uint4 w[kCount], x[kCount];
    float f0[kCount], f1[kCount];
    __device__ __forceinline__ void load(uint32_t box, uint32_t rows, uint32_t factors, int c, int first, int g,
                                         int t) {
        const uint32_t chunk = static_cast<uint32_t>((g >> 1) | ((g & 1) << 2));   // quarter-warps hit every bank once
        constexpr uint32_t kRec = kH ? kHRecord : 64;
#pragma unroll
        for (int j = 0; j < kCount; ++j) {
            const int row = 4 * (c + first + j) + t;
            w[j] = ld_shared_v4(box + row * 128 + ((chunk ^ (row & 7)) << 4));
            x[j] = ld_shared_v4(rows + (first + j) * kRec);
            if constexpr (kH) {
                f0[j] = __uint_as_float(ld_shared_u32(factors + (first + j) * kRec));
                f1[j] = __uint_as_float(ld_shared_u32(factors + (first + j) * kRec + kXStride));
            }
        }
    }
};

// d f s: what rounds or leaves the range in between does so in the result. A
// factor above 1 belongs to large activations, one up to 1 to small ones.
__device__ __forceinline__ float scaled_sum(float d, float f, float s, float acc) {
    const bool large = f > 1.f;
    return fmaf(d * (large ? s : f), large ? f : s, acc);
}

// Their products added to acc [16-column tile][fragment]. kEdge: any exponent
// byte may be among e4, and f0 and f1 are factors of tokens 2 t and 2 t + 1 (1
// where the sums are kept without them).
template <bool kEdge, bool kH, int kCount>
__device__ __forceinline__ void add_products(float (&acc)[2][4], const Operands<kH, kCount>& o,
                                             const uint32_t (&e4)[4], int first, float f0 = 1.f, float f1 = 1.f) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
        const uint32_t words[4] = {o.w[j].x, o.w[j].y, o.w[j].z, o.w[j].w}, e = e4[first + j];
        // 2^(e - 127): the byte as an FP32 exponent field, right for 1..254
        float scale[4];
        if constexpr (kEdge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) scale[i] = mx::scale_f32((e >> (8 * i)) & 0xFFu);
        } else {
            scale[0] = __uint_as_float((e & 0xFFu) << 23);
            scale[1] = __uint_as_float((e & 0xFF00u) << 15);
            scale[2] = __uint_as_float((e & 0xFF0000u) << 7);
            scale[3] = __uint_as_float((e >> 24) << 23);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t lo[4], hi[4];
            mx::e2m1x8_to_f16x2(words[2 * m], lo);
            mx::e2m1x8_to_f16x2(words[2 * m + 1], hi);
            float d[4];
            mma_f16_zero(d, lo[0], hi[0], lo[1], hi[1], o.x[j].x, o.x[j].y);
            mma_m16n8k16<false>(d, lo[2], hi[2], lo[3], hi[3], o.x[j].z, o.x[j].w);
            float(&a)[4] = acc[m];
            if constexpr (kH && kEdge) {
                a[0] = scaled_sum(d[0], o.f0[j], scale[2 * m], a[0]);
                a[1] = scaled_sum(d[1], o.f1[j], scale[2 * m], a[1]);
                a[2] = scaled_sum(d[2], o.f0[j], scale[2 * m + 1], a[2]);
                a[3] = scaled_sum(d[3], o.f1[j], scale[2 * m + 1], a[3]);
            } else if constexpr (kH) {
                // with a usual exponent d scale is in range, whatever the factor is
                a[0] = fmaf(d[0] * scale[2 * m], o.f0[j], a[0]);
                a[1] = fmaf(d[1] * scale[2 * m], o.f1[j], a[1]);
                a[2] = fmaf(d[2] * scale[2 * m + 1], o.f0[j], a[2]);
                a[3] = fmaf(d[3] * scale[2 * m + 1], o.f1[j], a[3]);
            } else if constexpr (kEdge) {
                a[0] = scaled_sum(d[0], f0, scale[2 * m], a[0]);
                a[1] = scaled_sum(d[1], f1, scale[2 * m], a[1]);
                a[2] = scaled_sum(d[2], f0, scale[2 * m + 1], a[2]);
                a[3] = scaled_sum(d[3], f1, scale[2 * m + 1], a[3]);
            } else {
                a[0] = fmaf(d[0], scale[2 * m], a[0]);
                a[1] = fmaf(d[1], scale[2 * m], a[1]);
                a[2] = fmaf(d[2], scale[2 * m + 1], a[2]);
                a[3] = fmaf(d[3], scale[2 * m + 1], a[3]);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
moe_kernel(const __grid_constant__ CUtensorMap tw13, const __grid_constant__ CUtensorMap te13,
           const __grid_constant__ CUtensorMap tw2, const __grid_constant__ CUtensorMap te2, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring_base = smem_u32(ring), rows_base = ring_base + kStages * kWeightBytes;
    Shared* sm = reinterpret_cast<Shared*>(ring + kStages * (kWeightBytes + kRowBytes));
    volatile int* abort = &sm->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grid = gridDim.x, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&sm->full[s]), 1);
            mbar_init(smem_u32(&sm->empty[s]), kConsumerWarps / 2);
        }
        for (int b = 0; b < kBuffers; ++b) {
            mbar_init(smem_u32(&sm->sums[b]), kConsumerWarps);
            mbar_init(smem_u32(&sm->taken[b]), kEpilogues);
        }
        mbar_init(smem_u32(&sm->phase3), 1);
        mbar_init(smem_u32(&sm->phase4), 1);
        *abort = 0;
        for (int b = 0; b < kBuffers; ++b)
            for (int i = 0; i < 4; ++i) sm->factored[b][i] = 0u;
        sm->epoch = ld_acquire(p.control);
        fence_mbar_init();
        tma_prefetch_desc(&tw13);
        tma_prefetch_desc(&te13);
        tma_prefetch_desc(&tw2);
        tma_prefetch_desc(&te2);
    }
    if (threadIdx.x < kMaxExperts) sm->mask[threadIdx.x][0] = sm->mask[threadIdx.x][1] = 0u;
    __syncthreads();
    uint32_t* counts = p.control + 1 + kBarriers * (sm->epoch & 1u);

    // ---------------------------------------------------------------- phase 0
    if (warp < kConsumerWarps) {
        float(*scratch)[4][32] = reinterpret_cast<float(*)[4][32]>(&sm->red[0][0][0][0]);
        const int etiles = (p.E + 15) >> 4, tiles = etiles * ((p.T + 7) >> 3), units = tiles * p.splits;
        for (int u = cta; u < units + p.T; u += grid) {
            const int tile = u % tiles;
            if (u < units)
                router_tile(p, scratch, (tile % etiles) * 16, (tile / etiles) * 8, u / tiles, warp, lane);
            else
                convert_token(p, scratch, u - units, warp, lane);
        }
        fence_proxy_async_global();   // x16 is read by bulk copies
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        grid_arrive(counts);
        grid_wait(counts, abort);
        if (cta == 0) {
            uint32_t* other = p.control + 1 + kBarriers * ((sm->epoch & 1u) ^ 1u);
            for (int i = 0; i < kBarriers; ++i) other[i] = 0u;
            p.control[0] = sm->epoch + 1u;
        }
    }
    __syncthreads();

    // ---------------------------------------------------------------- phase 1
    const bool alive = *abort == 0;
    if (alive) {
        if (threadIdx.x < p.T) sm->xfactor[threadIdx.x] = __ldcg(p.xfactor + threadIdx.x);
        for (int tok = warp; tok < p.T; tok += kThreads / 32) {
            if (p.E <= 64)
                pick_experts<2>(p, sm, tok, lane);
            else if (p.E <= 128)
                pick_experts<4>(p, sm, tok, lane);
            else
                pick_experts<kMaxExperts / 32>(p, sm, tok, lane);
        }
        __syncthreads();
        number_groups(p, sm);
    }
    // Items, column blocks fastest: CTAs next to one another read neighbouring columns of an expert
    const int groups = alive ? sm->groups : 0;
    const int cols2 = p.I >> 5, cols3 = (p.H + 63) >> 6;                 // column blocks
    const int items2 = groups * cols2, items3 = groups * cols3;
    const int blocks2 = p.H >> 5, blocks3 = p.I >> 5;                    // 32-row blocks of K
    const int steps2 = (blocks2 + kBlocks - 1) / kBlocks, steps3 = (blocks3 + kBlocks - 1) / kBlocks;

    if (warp >= kConsumerWarps + kEpilogues) {
        // ------------------------------------------------------------ producers, one per set
        const int set = warp - kConsumerWarps - kEpilogues;
        int slot = 0, seen = 0;
        uint32_t base = 0;   // the item's first stage among all of the CTA's
        uint32_t parity = 1u;
        bool ok = alive;
        fence_proxy_async_global();
        auto phase = [&](auto second) {
            constexpr bool kH = decltype(second)::value;
            constexpr uint32_t kRec = kH ? kHRecord : 64;
            const int items = kH ? items3 : items2, cols = kH ? cols3 : cols2;
            const int blocks = kH ? blocks3 : blocks2, steps = kH ? steps3 : steps2;
            const CUtensorMap* tw = kH ? &tw2 : &tw13;
            const CUtensorMap* te = kH ? &te2 : &te13;
            // Phase 3's first stages get their weights before h is complete and their rows after it.
            bool open = !kH;
            int held = 0, held_slot[kSetStages] = {};
            uint32_t held_bytes[kSetStages] = {};
            const uint8_t* held_src[kSetStages] = {};
            auto rows = [&](int s, const uint8_t* src, uint32_t bytes) {   // one row per lane
                if (src) bulk_load(rows_base + s * kRowBytes + lane * kXStride, src, bytes, smem_u32(&sm->full[s]));
            };
            auto release = [&] {
                ok = ok && warp_wait_bar(&sm->phase3, 0, abort);
                fence_proxy_async_global();
#pragma unroll
                for (int i = 0; i < kSetStages; ++i)
                    if (ok && i < held) rows(held_slot[i], held_src[i], held_bytes[i]);
                open = true;
            };
            Walk at(cta, grid, cols);
            for (int item = cta; item < items && ok; item += grid, at.next(), base += steps) {
                const int gi = at.group, cb = at.column;
                const uint32_t gr = sm->group[gi];
                const int n = gr >> 16, kb0 = static_cast<int>(gr & 0xFFFFu) * blocks;   // 32-row block of the stack
                const int c0 = kH ? cb * 64 : cb * 32, c1 = kH ? c0 + 32 : p.I + c0;
                const uint8_t* src = nullptr;
                if (lane < n) {
                    const uint32_t sl = sm->list[sm->first[gi] + lane];
                    src = kH ? p.h + static_cast<size_t>(sl & 1023u) * blocks * kHRecord
                             : reinterpret_cast<const uint8_t*>(p.x16 + static_cast<size_t>(sl >> 10) * p.H);
                }
                for (int ks = (base ^ set) & 1; ks < steps; ks += 2) {
                    const int s = set * kSetStages + slot, kb = kb0 + ks * kBlocks;
                    if (!warp_wait_bar(&sm->empty[s], parity, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bytes = min(kBlocks, blocks - ks * kBlocks) * kRec;
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(&sm->full[s]), dst = ring_base + s * kWeightBytes;
                        mbar_arrive_expect_tx(bar, kWeightBytes + n * bytes);
                        tma_load_2d(dst, tw, c0, kb * 4, bar);
                        tma_load_2d(dst + kBoxBytes, tw, c1, kb * 4, bar);
                        tma_load_2d(dst + 2 * kBoxBytes, te, c0, kb, bar);
                        tma_load_2d(dst + 2 * kBoxBytes + kScaleBoxBytes, te, c1, kb, bar);
                    }
                    __syncwarp();
                    const uint8_t* from = src ? src + static_cast<size_t>(ks) * kBlocks * kRec : nullptr;
                    if (open) {
                        rows(s, from, bytes);
                    } else {
#pragma unroll
                        for (int i = 0; i < kSetStages; ++i)
                            if (i == held) held_slot[i] = s, held_src[i] = from, held_bytes[i] = bytes;
                        if (++held == kSetStages) release();
                    }
                    ++seen;
                    if (++slot == kSetStages) slot = 0, parity ^= 1u;
                }
            }
            if (!open) release();
        };
        phase(std::false_type{});
        phase(std::true_type{});
        // copies in flight land before the CTA's shared memory is given back
        if (lane == 0) {
            const unsigned long long t0 = clock64();
            for (int i = max(0, seen - kSetStages); i < seen; ++i)
                while (!mbar_try_wait(smem_u32(&sm->full[set * kSetStages + i % kSetStages]), i / kSetStages & 1) &&
                       clock64() - t0 < kWaitLimitCycles) {
                }
        }
    } else if (warp < kConsumerWarps) {
        // ------------------------------------------------------------ consumers
        const int g = lane >> 2, t = lane & 3;
        const int set = warp >> 3, box = (warp >> 2) & 1, c0 = (warp & 3) * kWarpBlocks;
        uint32_t base = 0;    // the item's first stage among all of the CTA's: stage q is set q % 2's
        uint32_t count = 0;   // items so far
        uint32_t parity = 0;  // of the set's next stage
        int slot = 0;         // ... its place in the set's half of the ring
        bool ever = false;    // the warp has marked a buffer
        bool ok = alive, next = false;   // next: it was complete when looked at beside the last one's products
        auto phase = [&](auto second) {
            constexpr bool kH = decltype(second)::value;
            constexpr uint32_t kRec = kH ? kHRecord : 64;
            const int items = kH ? items3 : items2;
            const int blocks = kH ? blocks3 : blocks2, steps = kH ? steps3 : steps2;
            for (int item = cta; item < items; item += grid, ++count, base += steps) {
                uint32_t plain = 0x80808080u;   // 0: the sums hold the tokens' factors
                float acc[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
                const int b = static_cast<int>(count % kBuffers);
                const uint32_t turn = (count / kBuffers & 1u) ^ 1u;
                bool room = mbar_test_wait(smem_u32(&sm->taken[b]), turn);
                for (int ks = (base ^ set) & 1; ks < steps; ks += 2) {
                    const int here = blocks - ks * kBlocks - c0;   // of the warp's blocks, those that exist
                    const int s = set * kSetStages + slot;
                    if (!ok || !(__all_sync(0xffffffffu, next) || warp_wait_bar(&sm->full[s], parity, abort))) {
                        ok = false;
                        continue;
                    }
                    const uint32_t stage = ring_base + s * kWeightBytes, weights = stage + box * kBoxBytes;
                    const uint32_t in = rows_base + s * kRowBytes + c0 * kRec;
                    const uint32_t rows = in + g * kXStride + t * 16, factors = in + 2 * t * kXStride + 64 + 4 * t;
                    uint32_t e4[kWarpBlocks];
#pragma unroll
                    for (int i = 0; i < kWarpBlocks; ++i)
                        e4[i] = ld_shared_u32(stage + 2 * kBoxBytes + box * kScaleBoxBytes + (c0 + i) * 32 +
                                              ((g >> 1) | ((g & 1) << 2)) * 4);
                    if (++slot == kSetStages) slot = 0, parity ^= 1u;
                    const uint32_t empty = smem_u32(&sm->empty[s]);
                    const uint32_t after = smem_u32(&sm->full[set * kSetStages + slot]);
                    // An unusual exponent byte: the sums take on the tokens' factors, if they have not yet
                    auto use_factors = [&](float& f0, float& f1) {
                        const int gi = item / cols2, n = sm->group[gi] >> 16;
                        const uint16_t* list = sm->list + sm->first[gi];
                        if (2 * t < n) f0 = sm->xfactor[list[2 * t] >> 10];
                        if (2 * t + 1 < n) f1 = sm->xfactor[list[2 * t + 1] >> 10];
                        if (!plain) return;
#pragma unroll
                        for (int m = 0; m < 2; ++m) acc[m][0] *= f0, acc[m][1] *= f1, acc[m][2] *= f0, acc[m][3] *= f1;
                        plain = 0u;
                        ever = true;
                    };
                    // The usual stage: all four blocks, which then overlap; it goes back to the producer once the
                    // operands are in registers. Every exponent byte in 64..191 (bits 7 and 6 differ; scales
                    // 2^-63..2^64): none is 0 or 255. A stage that ends early: one block at a time.
                    if (here >= kWarpBlocks) {
                        uint32_t usual = plain;
#pragma unroll
                        for (int i = 0; i < kWarpBlocks; ++i) usual &= e4[i] ^ (e4[i] << 1);
                        Operands<kH, kWarpBlocks> o;
                        o.load(weights, rows, factors, c0, 0, g, t);
                        next = mbar_test_wait(after, parity);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(empty);
                        if (__all_sync(0xffffffffu, usual == 0x80808080u)) {
                            add_products<false>(acc, o, e4, 0);
                        } else {
                            float f0 = 1.f, f1 = 1.f;
                            if constexpr (!kH) use_factors(f0, f1);
                            add_products<true>(acc, o, e4, 0, f0, f1);
                        }
                    } else {
                        float f0 = 1.f, f1 = 1.f;
                        if constexpr (!kH) {
                            uint32_t usual = plain;
#pragma unroll
                            for (int i = 0; i < kWarpBlocks - 1; ++i)
                                if (i < here) usual &= e4[i] ^ (e4[i] << 1);
                            if (!__all_sync(0xffffffffu, usual == 0x80808080u)) use_factors(f0, f1);
                        }
#pragma unroll
                        for (int i = 0; i < kWarpBlocks - 1; ++i)
                            if (i < here) {
                                Operands<kH, 1> o;
                                o.load(weights, rows, factors, c0, i, g, t);
                                add_products<true>(acc, o, e4, i, f0, f1);
                            }
                        next = mbar_test_wait(after, parity);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(empty);
                    }
                }
                // sums to the item's buffer: slot [token parity][column % 4], at the lane that holds them
                if (ok) ok = __all_sync(0xffffffffu, room) || warp_wait_bar(&sm->taken[b], turn, abort);
#pragma unroll
                for (int m = 0; m < 2; ++m)       // columns 2 m and 2 m + 1 of every four
#pragma unroll
                    for (int i = 0; i < 4; ++i)   // fragment: column i >> 1, token parity i & 1
                        sm->red[b][warp][(i & 1) * 4 + m * 2 + (i >> 1)][lane] = acc[m][i];
                if (!kH && ever && lane == 0) reinterpret_cast<volatile uint8_t*>(sm->factored[b])[warp] = plain ? 0 : 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm->sums[b]));
            }
        };
        phase(std::false_type{});
        phase(std::true_type{});
    } else {
        // ------------------------------------------------------------ epilogue
        const int half = warp - kConsumerWarps;   // tokens 4 i + 2 half and the next of a group
        uint32_t count = 0;
        bool ok = alive;
        uint32_t base = 0;
        // token n of the group, column `lane`: warp w's part of it
        auto part_of = [&](int b, int n, int w) {
            const int chunk = lane >> 2, slot = (n & 1) * 4 + (lane & 3);
            const int from = (((chunk & 3) << 1) | (chunk >> 2)) * 4 + (n >> 1);
            return &sm->red[b][w][slot][from];
        };
        // and the sum of a box's parts, from the set of the item's first stage on: the same order whichever set that is
        auto total = [&](int b, int n, int box, int start) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int w = 0; w < kSlices; ++w) s += *part_of(b, n, (q ^ start) * 8 + box * 4 + w);
            return s;
        };
        Walk at(cta, grid, cols2);
        for (int item = cta; item < items2; item += grid, at.next(), ++count, base += steps2) {
            const int gi = at.group, cb = at.column, n = sm->group[gi] >> 16;
            const int b = static_cast<int>(count % kBuffers), start = static_cast<int>(base & 1u);
            int slot = 0;
            float f = 0.f;
            if (lane < n) {
                const uint32_t sl = sm->list[sm->first[gi] + lane];
                slot = sl & 1023u;
                f = sm->xfactor[sl >> 10];
            }
            if (!ok || !warp_wait_bar(&sm->sums[b], count / kBuffers & 1u, abort)) {
                ok = false;
                continue;
            }
            const uint32_t* has = sm->factored[b];
            if (has[0] | has[1] | has[2] | has[3]) {
                // some parts hold the factors: the others get them in place, by the lanes that will add them up
                for (int n0 = 2 * half; n0 < n; n0 += (n0 & 1) ? 2 * kEpilogues - 1 : 1) {
                    const float fi = __shfl_sync(0xffffffffu, f, n0);
                    for (int w = 0; w < kConsumerWarps; ++w)
                        if (!((has[w >> 2] >> (8 * (w & 3))) & 0xFFu)) *part_of(b, n0, w) *= fi;
                }
                f = 1.f;
            }
            float back = 0.f;   // lane i: token i's factor 2^-shift
            for (int i0 = 2 * half; i0 < n; i0 += 2 * kEpilogues) {
                float h[2];
                int sh[2];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const float fi = __shfl_sync(0xffffffffu, f, i0 + d);   // 0 past the last token
                    const float gate = total(b, i0 + d, 0, start) * fi, up = total(b, i0 + d, 1, start) * fi;
                    h[d] = silu(gate) * up;
                }
#pragma unroll
                for (int d = 0; d < 2; ++d)
                    sh[d] = mx::x_shift(__reduce_max_sync(0xffffffffu, (__float_as_uint(h[d]) >> 23) & 0xFFu));
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int si = __shfl_sync(0xffffffffu, slot, i0 + d);
                    const float scaled = h[d] * __uint_as_float(static_cast<uint32_t>(sh[d] + 127) << 23);
                    if (i0 + d < n)
                        __stcg(reinterpret_cast<unsigned short*>(
                                   p.h + (static_cast<size_t>(si) * blocks3 + cb) * kHRecord) + lane,
                               __half_as_ushort(__float2half_rn(scaled)));
                    if (lane == i0 + d) back = mx::x_unshift(sh[d]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm->taken[b]));
            if (lane < n && ((lane >> 1) & 1) == half)
                __stcg(reinterpret_cast<float4*>(p.h + (static_cast<size_t>(slot) * blocks3 + cb) * kHRecord + 64),
                       make_float4(back, back, back, back));
        }
        fence_proxy_async_global();   // h is read by bulk copies
        auto epilogue_sync = [] { asm volatile("bar.sync 2, %0;" ::"n"(kEpilogues * 32) : "memory"); };
        epilogue_sync();
        if (half == 0 && lane == 0 && alive) {
            grid_arrive(counts + 1);
            if (grid_wait(counts + 1, abort)) mbar_arrive(smem_u32(&sm->phase3));
        }
        __syncwarp();

        at = Walk(cta, grid, cols3);
        for (int item = cta; item < items3; item += grid, at.next(), ++count, base += steps3) {
            const int gi = at.group, cb = at.column, n = sm->group[gi] >> 16;
            const int b = static_cast<int>(count % kBuffers), start = static_cast<int>(base & 1u);
            const int slot = lane < n ? sm->list[sm->first[gi] + lane] & 1023 : 0;
            const float pw = lane < n ? sm->weight[slot] : 0.f;
            if (!ok || !warp_wait_bar(&sm->sums[b], count / kBuffers & 1u, abort)) {
                ok = false;
                continue;
            }
            const bool right = cb * 64 + 32 < p.H;   // H % 64 may be 32
            for (int i0 = 2 * half; i0 < n; i0 += 2 * kEpilogues) {
                float sums[2][2];
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int box = 0; box < 2; ++box) sums[d][box] = total(b, i0 + d, box, start);
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const int si = __shfl_sync(0xffffffffu, slot, i0 + d);
                    const float wi = __shfl_sync(0xffffffffu, pw, i0 + d);
                    if (i0 + d < n) {
                        float* part = p.part + static_cast<size_t>(si) * p.H + cb * 64 + lane;
                        __stcg(part, sums[d][0] * wi);
                        if (right) __stcg(part + 32, sums[d][1] * wi);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm->taken[b]));
        }
        epilogue_sync();
        if (half == 0 && lane == 0 && alive) {
            grid_arrive(counts + 2);
            if (grid_wait(counts + 2, abort)) mbar_arrive(smem_u32(&sm->phase4));
        }
    }

    // ---------------------------------------------------------------- phase 4
    __syncwarp();   // single-lane roles rejoin their warp
    if (!alive || !warp_wait_bar(&sm->phase4, 0, abort)) return;
    const int quads = p.H >> 2;
    for (int i = cta * kThreads + static_cast<int>(threadIdx.x); i < p.T * quads; i += grid * kThreads) {
        const int tok = i / quads, col = (i - tok * quads) * 4;
        const float* src = p.part + static_cast<size_t>(tok) * p.k * p.H + col;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q0 = 0; q0 < p.k; q0 += 8) {
            float4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = q0 + q < p.k ? __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(q0 + q) * p.H))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 8; ++q) s.x += v[q].x, s.y += v[q].y, s.z += v[q].z, s.w += v[q].w;
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
        *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(tok) * p.H + col) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

struct Layout {
    size_t logits, x16, xfactor, h, part, total;
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
    l.logits = take(static_cast<size_t>(kMaxSplits) * T * E * 4);
    l.x16 = take(static_cast<size_t>(T) * H * 2);
    l.xfactor = take(static_cast<size_t>(T) * 4);
    l.h = take(slots * (I / 32) * kHRecord);
    l.part = take(slots * H * 4);
    l.total = at;
    return l;
}

cudaError_t launch_kernel(const CUtensorMap (&maps)[4], Params p, const DeviceProps& dp, cudaStream_t s) {
    if (cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(moe_kernel), dp.device, kSmemBytes);
        e != cudaSuccess)
        return e;
    // no more CTAs than the larger of the two expert phases can use
    const long long slots = static_cast<long long>(p.T) * p.k;
    const long long want = slots * std::max<long long>(p.I / 32, (p.H + 63) / 64);
    cudaLaunchConfig_t cfg = {};
    const int grid = static_cast<int>(std::min<long long>(want, dp.sms));
    // The number of parts depends on H alone, and with it the order of a logit's sum: the other tokens of a call change
    // nothing.
    p.splits = std::min(kMaxSplits, (p.H + kRouterDepth - 1) / kRouterDepth);
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    // the CTAs wait for one another at the grid barriers: all of them are resident together or the launch fails
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_kernel, maps[0], maps[1], maps[2], maps[3], p);
}

}  // namespace

size_t mx_moe_workspace_bytes(int T, int E, int k, int H, int I) { return layout(T, E, k, H, I).total; }

cudaError_t launch_mx_moe(const MxMoeArgs& a, void* workspace, const DeviceProps& dp, cudaStream_t s) {
    CUtensorMap maps[4];
    const uint64_t E = a.E, H = a.H, I = a.I;
    if (!encode_2d(&maps[0], CU_TENSOR_MAP_DATA_TYPE_INT32, a.w13, 2 * I, E * (H / 8), 2 * I * 4, 32, kStepK / 8,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&maps[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.e13, 2 * I, E * (H / 32), 2 * I, 32, kBlocks,
                   CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_2d(&maps[2], CU_TENSOR_MAP_DATA_TYPE_INT32, a.w2, H, E * (I / 8), H * 4, 32, kStepK / 8,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&maps[3], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.e2, H, E * (I / 32), H, 32, kBlocks,
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
    p.h = ws + l.h;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.T = a.T;
    p.E = a.E;
    p.k = a.k;
    p.H = a.H;
    p.I = a.I;
    p.renormalize = a.renormalize ? 1 : 0;
    return launch_kernel(maps, p, dp, s);
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
