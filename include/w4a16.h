/*
 * w4a16.h -- C ABI of libw4a16, the W4A16 group-quantized linear layer for
 * NVIDIA GB300 (sm_103a).
 *
 * The layer (one weight-only int4 linear layer, activations in fp16/bf16):
 *
 *     y[m, n] = sum_k x[m, k] * (q[k, n] - z[k / g, n]) * s[k / g, n]
 *
 *   x   [M, K]    activations, fp16 or bf16, row-major
 *   q   [K, N]    4-bit weight codes 0..15, stored packed (see qweight)
 *   s   [K/g, N]  one scale per group of g rows of K and per column, same
 *                 dtype as x
 *   z   [K/g, N]  4-bit zero-points 0..15, stored packed (see qzeros); the
 *                 symmetric layer has no zero-point tensor and uses z = 8,
 *                 the "code - 8" recentring described on "qsa_prompt_attn:
 *                 Q4_0 KV on tensor cores" (section "What")
 *   y   [M, N]    output, same dtype as x, rounded to nearest-even from an
 *                 FP32 accumulator
 *
 * Packed layouts (words are read as uint32 bit patterns):
 *   qweight int32 [K/8, N]    nibble j (bits 4j..4j+3) of word [w, n] holds
 *                             q[8w + j, n]
 *   qzeros  int32 [K/g, N/8]  the zero-point of column n sits in word
 *                             [t, n/8] at bits 4*(n%8). This is the packed
 *                             zero-point layout of "Keep W4A16 zero-points
 *                             packed at 4 bits instead of expanding to 2
 *                             bytes" (section "Change"); that page's point is
 *                             that the kernel reads zero-points in this form,
 *                             0.5 byte per group and column, and never an
 *                             expanded activation-dtype copy of them.
 *
 * Conventions for every entry point below:
 *   - Every tensor pointer is a DEVICE pointer owned by the caller; tensors
 *     are dense and row-major. The library never allocates or frees device
 *     memory and never synchronises, except w4a16_device_status, which
 *     synchronises the given stream.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *   - All argument checks run on the host BEFORE anything is launched; a
 *     failed check returns an error status and launches nothing.
 *   - A launch error is returned as W4A16_ERR_CUDA. The library does not
 *     clear CUDA's sticky error state.
 *   - The library runs only on compute capability 10.3 (GB300); any other
 *     device gives W4A16_ERR_DEVICE.
 *   - Shape limits: N % 8 == 0, K % g == 0, g in {32, 64, 128, 256}, all
 *     dimensions > 0 and < 2^31 (at most 2^31 - 512 in the layers and products,
 *     whose tiles are counted in 32 bits), base pointers 16-byte aligned. Products of
 *     dimensions are not limited: every offset is computed in 64 bits, so
 *     tensors past 2^32 elements or 4 GiB are fine.
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define W4A16_ABI_VERSION 1

typedef enum {
    W4A16_OK = 0,
    W4A16_ERR_NULL = 1,        /* a required pointer is NULL                          */
    W4A16_ERR_SHAPE = 2,       /* a dimension is out of range or inconsistent         */
    W4A16_ERR_DTYPE = 3,       /* unknown activation dtype                            */
    W4A16_ERR_ALIGN = 4,       /* a base pointer is not 16-byte aligned               */
    W4A16_ERR_UNSUPPORTED = 5, /* valid request this build does not implement         */
    W4A16_ERR_DEVICE = 6,      /* no CUDA device, or not compute capability 10.3      */
    W4A16_ERR_WORKSPACE = 7,   /* workspace missing or smaller than required          */
    W4A16_ERR_CUDA = 8,        /* a CUDA runtime call or a launch failed              */
    W4A16_ERR_TIMEOUT = 9      /* a device-side pipeline wait ran out (see below)     */
} w4a16_status;

typedef enum {
    W4A16_F16 = 0,
    W4A16_BF16 = 1,
    W4A16_F32 = 2 /* only where an entry point says so; the layers take F16 and BF16 */
} w4a16_dtype;

/* Same type as cudaStream_t; declared here so the header needs no CUDA include. */
typedef struct CUstream_st* w4a16_stream;

/* Which kernel a workspace query is for. */
typedef enum {
    W4A16_OP_GEMV = 0,
    W4A16_OP_GEMM = 1,
    W4A16_OP_MXFP4_MATMUL = 2
} w4a16_op;

/*
 * w4a16_pack -- pack 4-bit codes eight to a 32-bit word.
 *
 * src  uint8 [rows, cols]; only the low 4 bits of each byte are used.
 * dim  0: pack along rows -> dst int32 [rows/8, cols]; nibble j of word
 *         [w, c] is src[8w + j, c] (the qweight layout, rows = K);
 *      1: pack along cols -> dst int32 [rows, cols/8]; column c goes to word
 *         [r, c/8] at bits 4*(c%8) (the qzeros layout of "Keep W4A16
 *         zero-points packed at 4 bits instead of expanding to 2 bytes",
 *         section "Change", rows = K/g, cols = N).
 * The packed dimension must be a multiple of 8. Bit-exact; deterministic.
 * Errors: NULL, SHAPE (non-positive or not a multiple of 8), ALIGN (either
 * pointer not 16-byte aligned), DEVICE, CUDA.
 */
w4a16_status w4a16_pack(const uint8_t* src, int32_t* dst, int64_t rows, int64_t cols, int dim,
                        w4a16_stream stream);

/*
 * w4a16_unpack -- inverse of w4a16_pack. `rows`, `cols` and `dim` describe the
 * UNPACKED tensor dst uint8 [rows, cols] (values 0..15); src is the packed
 * int32 tensor of w4a16_pack's output shape. This is the inverse that the
 * zero-point page names as unpacking along the packed dimension. Errors as
 * for w4a16_pack.
 */
w4a16_status w4a16_unpack(const int32_t* src, uint8_t* dst, int64_t rows, int64_t cols, int dim,
                          w4a16_stream stream);

/*
 * w4a16_workspace_bytes -- bytes of device workspace `op` needs for this shape
 * on the current device. For the GEMV: the FP32 partial-sum slots of the
 * GEMV kernel (8 KB per SM), then those of the few-row tensor-core kernel
 * that w4a16_mxfp4_gemv runs for 5..16 rows of large layers (128 KB per SM;
 * both sizes depend only on the device), then the ticket words of whichever
 * kernel needs more for this shape (one per column block, or four per 128
 * columns; rounded up to 256 bytes). For the GEMM
 * with M <= 128: FP32 partial slots of 128 KB per SM, followed by four 32-bit
 * tickets per 128 columns (rounded up to 256 bytes); 0 for the GEMM with
 * M > 128. The same sizes serve w4a16_mxfp4_gemv and w4a16_mxfp4_gemm with
 * g = 32. For the MXFP4 product (g = 32) with M <= 32: FP32 partial tiles of
 * 128 KB per SM, then four 32-bit tickets per 128 columns of y (rounded up to
 * 256 bytes); 0 for the product with M > 32.
 * Returns 0 for shapes the op rejects and when no GB300 is current.
 */
size_t w4a16_workspace_bytes(w4a16_op op, int64_t M, int64_t N, int64_t K, int64_t g);

/*
 * w4a16_capture_id -- 0 while `stream` is not being captured into a CUDA graph,
 * else a number that no other capture of the process has. (No counterpart on
 * the pages this library follows.)
 *
 * A workspace has to be zero before the first kernel that uses it runs. A
 * zero fill made while a stream is captured becomes a node of that graph and
 * runs with it alone, so a workspace filled in one capture must not serve a
 * second one: the second graph may be replayed first. Graphs that may run at
 * the same time must not share a workspace either. With this number a caller
 * that keeps workspaces gives each capture its own. Touches no device memory;
 * 0 also where the query fails (such a stream takes no launch either).
 */
uint64_t w4a16_capture_id(w4a16_stream stream);

/*
 * w4a16_gemv -- decode path, 1 <= M <= 16.
 *
 * One row (and two rows of a layer of at most 4 * 2^20 weights) is
 * converted with FP32 FMAs; 2..16 rows otherwise go through warp-level
 * m16n8k16 tensor-core MMAs: (q - z) formed exactly in 16 bits as the A
 * operand, x as B, FP32 accumulators scaled once per 32-row chunk (measured
 * at N = 43008, K = 5376: 39.3 us at M = 4 against 58.9 us with FMAs, 59 us
 * at M = 16 against 67.5 us on the few-row tensor-core kernel of w4a16_gemm).
 *
 * Streams qweight, scales and qzeros once with 128-bit coalesced loads; the
 * loads of the next 32-row chunk of K are in flight while the current one is
 * converted, which is the overlap whose absence the zero-point page blames for
 * its batch-4, g=128 regression (section "Known regression"). A persistent
 * grid (one CTA per SM at most) takes equal shares of (column block, K chunk)
 * items, so every SM streams the same bytes (for small layers, a whole number
 * of CTAs per column block when that is cheaper); a column block shared by several CTAs is finished by the last of
 * them to arrive, which sums the partial vectors in ascending CTA order: the
 * result is deterministic.
 *
 * The kernel is launched with programmatic stream serialization. Its prologue
 * (barrier setup and an L2 prefetch of its first weight chunks, a cache hint
 * that delivers no data to the kernel) may overlap the end of the preceding
 * kernel on `stream`; every read of x, qweight, scales, qzeros and the
 * workspace, and every write, happens after that kernel has completed and
 * its memory operations are visible, exactly as for an ordinary launch.
 *
 * x        [M, K] dtype `dt`
 * qweight  int32 [K/8, N]
 * scales   [K/g, N] dtype `dt`
 * qzeros   int32 [K/g, N/8], or NULL for the symmetric layer (z = 8)
 * y        [M, N] dtype `dt`, written (not accumulated into)
 * workspace, workspace_bytes   device scratch of at least
 *          w4a16_workspace_bytes(W4A16_OP_GEMV, M, N, K, g) bytes, 16-byte
 *          aligned, owned by the caller. It must be zero-filled before its
 *          first use; every call leaves its ticket words at zero again and
 *          writes partial sums only below the ticket region, so one
 *          workspace sized for the largest N serves any later call of any
 *          shape. Two calls that may run at the same time (different
 *          streams) must not share a workspace, and the GEMV and the GEMM
 *          must not share one: the GEMM's partial-sum region covers the
 *          GEMV's ticket words (the MXFP4 GEMV and GEMM use the same layouts
 *          as these two and may share with them respectively).
 * Errors: NULL, SHAPE (M outside 1..16, N % 8, K % g), UNSUPPORTED (g not in
 * {32, 64, 128, 256}), DTYPE, ALIGN, WORKSPACE (NULL, unaligned or too small),
 * DEVICE, CUDA.
 */
w4a16_status w4a16_gemv(const void* x, const int32_t* qweight, const void* scales,
                        const int32_t* qzeros, void* y, int64_t M, int64_t N, int64_t K,
                        int64_t g, w4a16_dtype dt, void* workspace, size_t workspace_bytes,
                        w4a16_stream stream);

/*
 * w4a16_gemv_noalloc -- w4a16_gemv for callers that cannot allocate device
 * memory. (No counterpart on the pages this library follows.)
 *
 * Some callers have no way to obtain scratch memory: a plugin loaded into a
 * host program that owns every device allocation and hands plugins no
 * allocator; a serving process that has already reserved all device memory
 * for its own pools; a latency-critical loop where cudaMalloc, which can
 * synchronise the device and take unbounded time, is not allowed. This entry
 * point takes the same arguments as w4a16_gemv minus the workspace and uses a
 * fixed 4 MiB scratch array compiled into the library instead. It calls no
 * cudaMalloc, cudaFree or other allocating routine.
 *
 * - The array lives in every GPU that loads the library, until the process
 *   exits.
 * - The first call on a device looks up the array's device address once
 *   (cudaGetSymbolAddress, with that device current); make that first call
 *   before any stream capture on the device. A first call made while `stream`
 *   is being captured does not look the address up: it returns
 *   W4A16_ERR_CUDA and enqueues nothing.
 * - Every call on a device uses the same array and clears its ticket words
 *   (an asynchronous memset on `stream`) before the kernel. Two calls that can
 *   run at the same time on one device (different streams) race on the array
 *   and give wrong results: serialise them.
 * - A shape whose scratch (w4a16_workspace_bytes(W4A16_OP_GEMV, ...)) exceeds
 *   4 MiB is rejected with W4A16_ERR_WORKSPACE; the partial-sum region takes
 *   8 KB per SM and each column block a 4-byte ticket (column blocks are at
 *   least 64 columns wide), so on a 152-SM GB300 every N up to about 47
 *   million columns fits.
 * It runs the same kernel and plan as w4a16_gemv, so its results are
 * identical to w4a16_gemv's. Other errors as for w4a16_gemv.
 */
w4a16_status w4a16_gemv_noalloc(const void* x, const int32_t* qweight, const void* scales,
                                const int32_t* qzeros, void* y, int64_t M, int64_t N, int64_t K,
                                int64_t g, w4a16_dtype dt, w4a16_stream stream);

/*
 * w4a16_gemm -- prefill path, any M >= 1.
 *
 * M <= 128 runs an operand-swapped kernel: 128 weight columns per tile, the
 * dequantised weight tile as the MMA's 128-row operand and x (padded to 32,
 * 64 or 128 rows) as the other, so no MMA work is spent on 256-row tiles. The
 * dequantised tile is written straight into tensor memory and the MMA reads
 * it there. Its (column block, K step) pairs (256 deep up to 64 padded rows of
 * x, 128 above) are split into equal contiguous ranges,
 * one per SM (stream-K); a column block split between CTAs is finished by the
 * last of them, which sums their FP32 partials from the workspace in
 * ascending CTA order (deterministic). This path needs a workspace of
 * w4a16_workspace_bytes(W4A16_OP_GEMM, M, N, K, g) bytes with the GEMV's
 * ownership and zero-fill rules (W4A16_ERR_WORKSPACE otherwise); after a
 * W4A16_ERR_TIMEOUT reported by w4a16_device_status, zero it again. It is
 * launched with programmatic stream serialization like w4a16_gemv: its
 * prologue (barrier setup, tensor-memory allocation, tensor-map prefetch) may
 * overlap the end of the preceding kernel on `stream`, and every read and
 * write of caller memory follows that kernel's completion.
 * Larger M runs the kernel described next and needs no workspace.
 *
 * Clusters of two CTAs (one per SM) own 256 x 256 output tiles of a
 * persistent grid. Per 64-deep K step each CTA brings its 128 rows of x and
 * the packed weights of its 128 columns into shared memory with TMA, sixteen
 * warps dequantise the weight tile ONCE into a shared bf16/fp16 operand tile
 * that every MMA of the tile consumes (the cooperative shared tile of "ROCm
 * KQuantGemmKWmmaQ4K/Q6K: redesign around a cooperative shared tile",
 * section "Confirmed mechanism"), and one thread issues
 * tcgen05.mma.cta_group::2 (M=256, N=256) over both CTAs' operands with the
 * FP32 accumulator in tensor memory. M and N tails are handled by TMA zero
 * fill on loads and predicated stores. The dequantised weight is (q - z) * s
 * rounded once to the activation dtype.
 *
 * Arguments and errors as w4a16_gemv, except M >= 1 with no upper limit.
 * W4A16_ERR_TIMEOUT is never returned here; a pipeline wait that runs out
 * sets a device flag that w4a16_device_status reports.
 */
w4a16_status w4a16_gemm(const void* x, const int32_t* qweight, const void* scales,
                        const int32_t* qzeros, void* y, int64_t M, int64_t N, int64_t K,
                        int64_t g, w4a16_dtype dt, void* workspace, size_t workspace_bytes,
                        w4a16_stream stream);

/*
 * w4a16_dequant -- dense dequantised copy of the packed weights:
 *
 *     w[k, n] = RN((q[k, n] - z[k / g, n]) * s[k / g, n])
 *
 * in dtype `dt`, row-major [K, N]: the dense dequantised weight copy that
 * "Keep W4A16 zero-points packed at 4 bits instead of expanding to 2 bytes"
 * (section "Change") builds at load time beside the skinny GEMM. (q - z) is exact in 16-bit
 * arithmetic and the product is rounded once, so the result is bit-exact.
 *
 * qweight  int32 [K/8, N]; scales [K/g, N] dtype `dt`; qzeros int32
 *          [K/g, N/8] or NULL (symmetric, z = 8)
 * w        [K, N] dtype `dt`, written (device memory owned by the caller)
 * Errors: NULL, SHAPE (N % 8, K % g, non-positive), UNSUPPORTED (g), DTYPE,
 * ALIGN, DEVICE, CUDA. Streams each operand once; bound by HBM bandwidth.
 */
w4a16_status w4a16_dequant(const int32_t* qweight, const void* scales, const int32_t* qzeros, void* w, int64_t N,
                           int64_t K, int64_t g, w4a16_dtype dt, w4a16_stream stream);

/*
 * MXFP4 weights -- "Add BF16xFP4 MoE GEMM stage1 kernel" (section "Technical
 * Details"): bf16 activations, weights stored as 4-bit E2M1 codes with one
 * E8M0 exponent byte e per 32 consecutive K rows of a column, decoded in
 * software to bf16 before the contraction, FP32 accumulation. The weight is
 *
 *     W[k, n] = RN_bf16( E2M1(q[k, n]) * 2^(e[k / 32, n] - 127) )
 *
 * where code q has the sign in bit 3, a 2-bit exponent field E (bias 1) in
 * bits 2..1 and a mantissa bit m in bit 0 (E = 0: m / 2, otherwise
 * 2^(E - 1) (1 + m/2)): magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6. Byte 0 means
 * 2^-127 and byte 255 NaN (every weight of that block is NaN). Every W is
 * exact in bf16 except where it exceeds the bf16 range (+-inf).
 *
 * qweight  int32 [K/8, N], the W4A16 word layout: nibble j of word [w, n] is
 *          the code of row 8w + j
 * escale   uint8 [K/32, N]: exponent byte of block b, column n at b * N + n
 * x        bf16 [M, K]; y bf16 [M, N], written (not accumulated into)
 * Shapes: N % 16 == 0 (each exponent row starts 16-byte aligned), K % 32 == 0.
 * Every pointer 16-byte aligned device memory owned by the caller.
 * Errors: NULL, SHAPE, ALIGN, DEVICE, CUDA, WORKSPACE (GEMV only).
 */

/*
 * w4a16_mxfp4_dequant -- dense bf16 copy W [K, N] (row-major) of MXFP4
 * weights. Bit-exact. Streams each operand once; bound by HBM bandwidth.
 */
w4a16_status w4a16_mxfp4_dequant(const int32_t* qweight, const uint8_t* escale, void* w, int64_t N, int64_t K,
                                 w4a16_stream stream);

/*
 * w4a16_mxfp4_gemv -- decode path for MXFP4 weights, 1 <= M <= 16: the
 * w4a16_gemv kernel with the E2M1 decode in place of the 4-bit integer one
 * (each 32-row chunk is one exponent block; its scale 2^(e - 127) is applied
 * in FP32 once per chunk). Same persistent grid, deterministic fix-up and
 * programmatic launch, and the same conversion choice: FP32 FMAs for one row
 * (and two rows of a layer of at most 4 * 2^20 weights), warp-level
 * tensor-core MMAs on fp16 operands otherwise (each chunk's x rows are first
 * rescaled to fp16 by a power of two per row, undone in FP32). 9..16 rows of
 * a layer with at least 48 * 2^20 weights run the few-row tensor-core kernel
 * of w4a16_mxfp4_gemm instead, where the 16-row rescale costs more than the
 * MMAs save (43008 x 5376, M = 12: 110.5 against 77.3 us; M = 8 stays on the
 * GEMV: 59.4 against 77.1 us).
 * Workspace: at least w4a16_workspace_bytes(W4A16_OP_GEMV, M, N, K, 32) bytes,
 * with the same ownership and zero-fill rules as for w4a16_gemv.
 */
w4a16_status w4a16_mxfp4_gemv(const void* x, const int32_t* qweight, const uint8_t* escale, void* y, int64_t M,
                              int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                              w4a16_stream stream);

/*
 * w4a16_mxfp4_gemm -- prefill path for MXFP4 weights, any M >= 1: the
 * w4a16_gemm kernels (operand-swapped and stream-K for M <= 128, CTA pairs
 * above) with the E2M1 decode writing the bf16 operand tile. Workspace as for
 * w4a16_gemm (needed for M <= 128, sized by w4a16_workspace_bytes(
 * W4A16_OP_GEMM, M, N, K, 32)). A pipeline wait that runs out sets the device
 * flag that w4a16_device_status reports.
 */
w4a16_status w4a16_mxfp4_gemm(const void* x, const int32_t* qweight, const uint8_t* escale, void* y, int64_t M,
                              int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                              w4a16_stream stream);

/*
 * MXFP4 in the row layout, and quantisation to MXFP4. (No counterpart on the
 * pages this library follows: they take quantised weights as given.)
 *
 * The layout above keeps the eight codes of a word along K of a [K, N] weight
 * (dim 0 of w4a16_pack). The row layout keeps them along the rows of a matrix
 * [R, K] whose rows are contracted (dim 1): activations, or a weight stored
 * one output feature per row.
 *   codes   int32 [R, K/8]: nibble j of word [r, w] is the code of element
 *           [r, 8w + j]
 *   escale  uint8 [ceil(R/128), ceil(K/128), 32, 4, 4]: tiles of 128 rows x 4
 *           blocks (a block is 32 consecutive elements of a row), 512 bytes a
 *           tile. The byte of row r, block b has index [r/128, b/4, r%32,
 *           (r/32)%4, b%4], the order in which the tensor cores take the
 *           scales of 128 operand rows. Bytes of blocks past the row's end are
 *           zero; bytes of rows past R are never used for a result.
 */

/*
 * w4a16_mxfp4_quantize -- codes and exponent bytes of x [rows, cols], dtype
 * `dt` (F16, BF16 or F32), row-major. Blocks run along `dim`:
 *   dim 0  blocks of 32 rows of a column -> codes int32 [rows/8, cols], escale
 *          uint8 [rows/32, cols]: the weight layout of w4a16_mxfp4_gemv,
 *          w4a16_mxfp4_gemm and w4a16_mxfp4_moe. rows % 32 == 0, cols % 16 == 0.
 *   dim 1  blocks of 32 columns of a row -> the row layout. cols % 32 == 0.
 *
 * With amax the largest magnitude of a block,
 *
 *     e = max(floor(log2(amax)) - 2 + 127, 0)
 *     c = E2M1(v * 2^(127 - e)), to nearest, ties to the code with bit 0 clear;
 *         magnitudes above 6 become 6
 *
 * so the largest magnitude is scaled into [4, 8). A block of zeros has e = 0.
 * A block that holds an infinity or a NaN has e = 255 and codes 0: each of its
 * values reads as NaN. Values that MXFP4 represents exactly are kept exactly,
 * so quantising a dense copy gives its values back. Bit-exact; deterministic.
 * Streams each operand once. An ordinary launch (no programmatic serialization).
 * Errors: NULL, DTYPE, SHAPE (non-positive, not a multiple as above, dim),
 * ALIGN (a pointer not 16-byte aligned), DEVICE, CUDA.
 */
w4a16_status w4a16_mxfp4_quantize(const void* x, int32_t* codes, uint8_t* escale, int64_t rows, int64_t cols, int dim,
                                  w4a16_dtype dt, w4a16_stream stream);

/*
 * w4a16_mxfp4_dequant_rows -- dense bf16 copy [rows, cols] (row-major) of the
 * row layout. Bit-exact. Errors: NULL, SHAPE (non-positive, cols % 32), ALIGN,
 * DEVICE, CUDA.
 */
w4a16_status w4a16_mxfp4_dequant_rows(const int32_t* codes, const uint8_t* escale, void* w, int64_t rows, int64_t cols,
                                      w4a16_stream stream);

/*
 * w4a16_mxfp4_tile_scales -- exponent bytes stored one row after the other,
 * src uint8 [rows, cols/32], to the tiles of the row layout (for operands
 * quantised elsewhere). dst must not overlap src. Errors: NULL, SHAPE
 * (non-positive, cols % 32), ALIGN (dst not 16-byte aligned), DEVICE, CUDA.
 */
w4a16_status w4a16_mxfp4_tile_scales(const uint8_t* src, uint8_t* dst, int64_t rows, int64_t cols,
                                     w4a16_stream stream);

/*
 * w4a16_mxfp4_matmul -- product of two MXFP4 operands in the row layout,
 *
 *     y[m, n] = sum_k A[m, k] * B[n, k]
 *
 * A [M, K] (codes `a`, exponent tiles `ea`), B [N, K] (`b`, `eb`): activations
 * quantised by w4a16_mxfp4_quantize(dim 1) against a weight quantised once, one
 * output feature per row. The tensor cores multiply the 4-bit codes
 * themselves, apply both exponents per 32 elements of K and accumulate in
 * FP32; the sum is rounded once to `dt` (F16, BF16 or F32). An exponent byte of
 * 255 makes every y of its row (of A) or column (of B) NaN. Exponents whose
 * product leaves the FP32 range overflow to infinity or flush to zero.
 *
 * Large products run on CTA pairs (256 x 256 tiles); the others (always for
 * M <= 128) on a kernel with 128 rows of B per tile, whose CTAs may split a
 * tile's K among them. With M <= 32 it takes a workspace of
 * w4a16_workspace_bytes(W4A16_OP_MXFP4_MATMUL, M, N, K, 32) bytes, with the
 * ownership and zero-fill rules of w4a16_gemv's (one sized for the largest N
 * serves every shape); a workspace of this op serves this op only. With M > 32 it
 * uses none. Split tiles are summed in a fixed order: the result is
 * deterministic. After a W4A16_ERR_TIMEOUT reported by w4a16_device_status, zero
 * the workspace again.
 *
 * M >= 1, N % 8 == 0, K % 32 == 0. An ordinary launch (no programmatic
 * serialization).
 * Errors: NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, DEVICE, CUDA.
 */
w4a16_status w4a16_mxfp4_matmul(const int32_t* a, const uint8_t* ea, const int32_t* b, const uint8_t* eb, void* y,
                                int64_t M, int64_t N, int64_t K, w4a16_dtype dt, void* workspace,
                                size_t workspace_bytes, w4a16_stream stream);

/*
 * w4a16_mxfp4_moe -- a mixture-of-experts layer with MXFP4 expert weights for
 * 1..64 tokens, in one kernel. ("Add BF16xFP4 MoE GEMM stage1 kernel" is the
 * gate/up product alone, with the routing done outside.)
 *
 *     p[t, :]   = softmax(x[t, :] . router^T) over the E experts
 *     chosen(t) = the top_k experts of largest logit, ties to the lower index;
 *                 with `renormalize` their p is divided by its sum
 *     h_e[t, :] = silu(x W1_e) * (x W3_e),     silu(v) = v / (1 + exp(-v))
 *     y[t, :]   = sum over chosen e of p[t, e] * (h_e[t, :] W2_e)
 *
 * x       bf16 [T, H]; router bf16 [E, H], one expert per row
 * w13     int32 [E, H/8, 2 I], e13 uint8 [E, H/32, 2 I]: every expert's
 *         [W1 | W3] in the weight layout above, gate columns [0, I), up
 *         columns [I, 2 I) (w4a16_mxfp4_quantize with dim 0 on the stack
 *         [E * H, 2 I])
 * w2      int32 [E, I/8, H], e2 uint8 [E, I/32, H]
 * y       bf16 [T, H], written (not accumulated into)
 *
 * Logits, softmax, the products' sums and the weighted sum are FP32. x and h
 * enter the products as fp16 scaled by powers of two (x per token, h per 32
 * columns): x converts exactly where it is within 2^-29 of its token's largest
 * magnitude, h is rounded to 11 bits. Weights of a chosen expert are read once
 * per 8 tokens that chose it (again mostly from L2); experts nobody chose are not
 * read. A token's y does not depend on the other tokens, bit for bit, and the
 * result is deterministic. A token with an infinity or NaN in x or in a chosen
 * expert's block yields NaN there and leaves other tokens alone.
 *
 * workspace: at least w4a16_mxfp4_moe_workspace_bytes(...) bytes with the
 * ownership and zero-fill rules of w4a16_gemv's (what must start at zero are
 * barrier words in its first 256 bytes, which every call leaves as the next
 * needs them: one workspace serves calls of any shape it is large enough for,
 * and is not zeroed again between them). Two calls that
 * may run at the same time must not share one. After a W4A16_ERR_TIMEOUT
 * reported by w4a16_device_status, zero it again.
 *
 * Launched cooperatively (its thread blocks wait for one another at three
 * points); it can be captured in a CUDA graph.
 * Limits: 1 <= T <= 64, 1 <= E <= 256, 1 <= top_k <= min(E, 16), H and I
 * multiples of 32, H <= 65536.
 * Errors: NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, CUDA.
 */
w4a16_status w4a16_mxfp4_moe(const void* x, const void* router, const int32_t* w13, const uint8_t* e13,
                             const int32_t* w2, const uint8_t* e2, void* y, int64_t T, int64_t E, int64_t top_k,
                             int64_t H, int64_t I, int renormalize, void* workspace, size_t workspace_bytes,
                             w4a16_stream stream);

/* Bytes of workspace w4a16_mxfp4_moe needs; 0 for shapes it rejects. */
size_t w4a16_mxfp4_moe_workspace_bytes(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t I);

/*
 * 8-bit integer operands: rows of int8 codes with one FP32 scale per row, the
 * value of an element being code * scale. (No counterpart on the pages this
 * library follows.) Activations have a row per token, weights a row per output
 * channel: [N, K] as they are stored before any packing.
 *   codes   int8 [R, K]
 *   scale   float [R]
 */

/*
 * w4a16_int8_quantize -- codes and scales of the rows of x [rows, cols], dtype
 * `dt` (F16, BF16 or F32), row-major. With amax the largest magnitude of a row,
 *
 *     scale = RN(amax / 127),   code = RN(127 x / amax), ties to even
 *
 * Both are decided exactly (the quotient is not rounded before the code is).
 * Codes lie in -127..127. A row of zeros has scale 0 and codes 0. A row that
 * holds an infinity or a NaN has scale NaN and codes 0: each of its values reads
 * as NaN. Rows whose amax / 127 is below 2^-126 have a subnormal scale, with fewer
 * bits. cols % 16 == 0. Bit-exact; deterministic.
 * Errors: NULL, DTYPE, SHAPE (non-positive, cols % 16), ALIGN (a pointer not
 * 16-byte aligned), DEVICE, CUDA.
 */
w4a16_status w4a16_int8_quantize(const void* x, int8_t* codes, float* scale, int64_t rows, int64_t cols,
                                 w4a16_dtype dt, w4a16_stream stream);

/*
 * w4a16_int8_dequant -- dense copy y [rows, cols] of dtype `dt` (F16, BF16 or
 * F32): code * scale in FP32, rounded to `dt`. Errors as w4a16_int8_quantize.
 */
w4a16_status w4a16_int8_dequant(const int8_t* codes, const float* scale, void* y, int64_t rows, int64_t cols,
                                w4a16_dtype dt, w4a16_stream stream);

/*
 * w4a16_int8_matmul -- product of two int8 operands with a scale per row of each,
 *
 *     y[m, n] = (sum_k a[m, k] * b[n, k]) * a_scale[m] * b_scale[n]
 *
 * A [M, K]: activations quantised by w4a16_int8_quantize, a scale per token.
 * B [N, K]: a weight quantised once, a scale per output channel. Any int8 value
 * may occur, -128 too. A sum is exact where none of its partial sums exceeds 2^24 in
 * magnitude: wherever sum |a b| does not, so for K <= 1024 always, and beyond that
 * for a mean |a b| of up to 2^24 / K (780 at K = 21504). Past it, few rows (up to 4,
 * up to 16 of a small layer and output) are still summed in 32-bit integers and
 * rounded once, more are summed in FP32 with an error of up to
 * (K / 16 + 256) 2^-23 sum |a b|: there y of a row may depend on M. Both scales are
 * applied in FP32, a_scale first, and the result is rounded once to `dt` (F16,
 * BF16 or F32). A NaN scale makes every y of its row or column NaN.
 *
 * workspace: w4a16_int8_matmul_workspace_bytes(M, N, K) bytes with the ownership
 * and zero-fill rules of w4a16_gemv's (what must start at zero are ticket words in
 * its first 4096 bytes, which every call leaves at zero: one workspace serves calls
 * of any shape it is large enough for). NULL where that is 0. Two calls that may run
 * at the same time must not share one. After a W4A16_ERR_TIMEOUT reported by
 * w4a16_device_status, zero it again.
 *
 * Deterministic. M >= 1, N % 8 == 0, K % 16 == 0, K <= 131056.
 * Errors: NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, DEVICE, CUDA.
 */
w4a16_status w4a16_int8_matmul(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale, void* y,
                               int64_t M, int64_t N, int64_t K, w4a16_dtype dt, void* workspace,
                               size_t workspace_bytes, w4a16_stream stream);

/*
 * Bytes of workspace w4a16_int8_matmul needs on the current device; 0 where it
 * needs none, for shapes it rejects, and when no GB300 is current.
 */
size_t w4a16_int8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* What the gate of w4a16_block_norm is given for. */
typedef enum {
    W4A16_GATE_CHANNEL = 0, /* [H]    */
    W4A16_GATE_TOKEN = 1,   /* [T]    */
    W4A16_GATE_ELEMENT = 2  /* [T, H] */
} w4a16_gate;

/*
 * w4a16_block_norm -- the step between two blocks of a transformer: the norm
 * after a block, its gate and the residual's scale, the residual update, the norm
 * before the next block and, where asked for, its quantisation. (No counterpart on
 * the pages this library follows.)
 *
 *     u  = h * rsqrt(mean(h^2) + eps) * after     (u = h where `after` is NULL)
 *     r' = residual + scale * gate * u            (gate 1 where NULL; r' = residual where h is NULL)
 *     y  = r' * rsqrt(mean(r'^2) + eps) * weight
 *
 * with the means over the H elements of a row. All in FP32; r' is normalised as
 * it is before it is rounded to be stored.
 *
 * residual [T, H] dtype `residual_dt`; h, gate, after [H], weight [H], y [T, H]
 * dtype `dt`. residual_dt is dt or F32.
 *   residual_out  [T, H] dtype residual_dt, r'; may be `residual` itself. Required
 *                 with h, NULL without (nothing would change).
 *   weight        NULL: no norm before the next block; y, codes and code_scale
 *                 are then NULL.
 *   y             [T, H] dtype dt, or NULL:
 *   codes         int8 [T, H] with code_scale float [T], y as w4a16_int8_quantize
 *                 makes it of the unrounded y.
 * One of h and weight at least; after and gate only with h. Outputs other than
 * residual_out must not overlap the inputs or one another.
 * scale finite, eps positive and finite (UNSUPPORTED otherwise). H % 16 == 0, H <= 16384.
 * u and y are formed in the order written; scale, gate and u are multiplied in any
 * order. Rows whose sum of squares leaves the FP32 range are normalised to zero, as
 * the formula in FP32 gives it. A row with an infinity or a NaN yields NaN in that
 * row (codes 0, scale NaN) and leaves other rows alone. Deterministic; a row does
 * not depend on the others. An ordinary launch (no programmatic serialization).
 * Errors: NULL (residual, or a pointer that another one asks for), DTYPE, SHAPE
 * (T, H, the gate kind, a pointer given that must be NULL), UNSUPPORTED, ALIGN,
 * DEVICE, CUDA.
 */
w4a16_status w4a16_block_norm(const void* residual, w4a16_dtype residual_dt, const void* h, const void* after,
                              const void* gate, w4a16_gate gate_kind, float scale, void* residual_out,
                              const void* weight, float eps, void* y, int8_t* codes, float* code_scale, int64_t T,
                              int64_t H, w4a16_dtype dt, w4a16_stream stream);

/*
 * w4a16_device_status -- synchronise `stream`, then read and clear the
 * device-side error word of the current device. Every wait on an mbarrier
 * inside the GEMM pipeline gives up after about two seconds; the kernel then
 * records W4A16_ERR_TIMEOUT there, drains its own copies in flight, frees its
 * tensor memory and returns, so the CUDA context stays usable. Returns
 * W4A16_OK when nothing was recorded, W4A16_ERR_CUDA if synchronisation
 * failed.
 */
w4a16_status w4a16_device_status(w4a16_stream stream);

/*
 * w4a16_selftest_wait_timeout -- exercise the device-side failure path. (No
 * counterpart on the pages this library follows.)
 *
 * Launches, asynchronously on `stream`, one warp that waits on an mbarrier
 * nothing will complete, with the same bounded wait the GEMV uses. After about
 * two seconds the wait gives up, records W4A16_ERR_TIMEOUT in the device error
 * word and the kernel exits normally, so the CUDA context stays usable; a
 * following w4a16_device_status(stream) returns W4A16_ERR_TIMEOUT (and clears
 * the word). Touches no caller memory. Errors: DEVICE, CUDA (launch failed).
 */
w4a16_status w4a16_selftest_wait_timeout(w4a16_stream stream);

/*
 * w4a16_selftest_mxfp4_matmul_plan -- how w4a16_mxfp4_matmul would run a shape
 * on a device of `sms` SMs, for tests that have to reach each way of running
 * it. Host only. (No counterpart on the pages this library follows.)
 * plan[0]  rows of A per tile (16, 32, 64 or 128), or 0: 256 x 256 tiles on CTA
 *          pairs
 * plan[1]  CTAs of a cluster that split a tile's K (1: not split)
 * plan[2]  1 if tiles are shared between CTAs through the workspace
 * Errors: NULL, SHAPE.
 */
w4a16_status w4a16_selftest_mxfp4_matmul_plan(int64_t M, int64_t N, int64_t K, int sms, int* plan);

/*
 * w4a16_selftest_int8_matmul_plan -- how w4a16_int8_matmul would run a shape (its
 * first rows, where they are cut into chunks) on a device of `sms` SMs, all
 * clusters resident, for tests that have to reach each way of running it. Host
 * only. (No counterpart on the pages this library follows.)
 * plan[0]  rows of A per tile of 128 rows of B (16, 32, 64 or 128), 0: CTA pairs,
 *          -1: dot products
 * plan[1]  CTAs of a cluster that split a tile's K (1: not split); with pairs, a
 *          tile of the columns that they leave
 * plan[2]  1 if tiles are shared between CTAs through the workspace
 * plan[3]  rows of A per tile of the pairs, 0 without pairs
 * plan[4]  columns of y that the pairs take, 0 without pairs
 * Errors: NULL, SHAPE.
 */
w4a16_status w4a16_selftest_int8_matmul_plan(int64_t M, int64_t N, int64_t K, int sms, int* plan);

/* Human-readable name of a status code (static storage, never NULL). */
const char* w4a16_status_string(w4a16_status status);

/* W4A16_ABI_VERSION of the compiled library. */
int w4a16_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */
