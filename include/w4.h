/*
 * w4.h -- C ABI of libw4: weight-only INT4 (group 128) matrix-vector product
 * y = W x on one NVIDIA GB300 (sm_103a).
 *
 * What is computed.  W is N x K.  Each weight is stored as a 4-bit unsigned
 * integer q in 0..15; every group of 128 consecutive weights of a row along K
 * has one fp16 scale s and one zero point z in 0..15, and the weight's value is
 * w = (q - z) * s.  Activations x are bfloat16, M = 1..8 token rows; the
 * product is y[m][n] = sum_k w[n][k] * x[m][k], accumulated in fp32.
 *   Sources (page title, section): group-wise INT4 weights with one fp16 scale
 *   per 128 weights of an output row -- "Building an LLM Inference Runtime: A
 *   Deep Dive into Qwen2.5-Coder-7B on NVIDIA H100", section "The Stack
 *   Architecture: A One-Page Overview"; a zero point per group applied as
 *   (q - z) * s -- "Custom AWQ Dequantization Kernel", section "Dead ends in
 *   profiling"; dequantisation fused into the matrix-vector kernel, no fp16 W
 *   materialised -- "CodeAlign-Runtime", section "Level 3 -- INT4 Quantization
 *   + Fused Kernel"; 1..8 rows (plain decode and a speculative-verify batch)
 *   with identical per-row results -- "qengine", section "How it works".
 *
 * Canonical layout (what callers hold; row-major, contiguous):
 *   qweight uint32 [N][K/8]: nibble j (bits 4j..4j+3) of word w is k = 8w + j
 *   scales  uint16 [N][K/128]: binary16 bit patterns
 *   zeros   uint8  [N][K/128]: values 0..15
 *   x       uint16 [M][K]: bfloat16 bit patterns
 *   y       uint16 [M][N] (bfloat16, round-to-nearest-even) or float [M][N]
 *
 * Conventions for every call:
 *   - Pointers named device are CUDA device pointers; the caller owns all
 *     memory.  The library never allocates device or pinned memory.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *     stream) and is asynchronous unless stated otherwise.
 *   - Errors are returned, never aborted on.  Argument checks happen on the
 *     host before anything is enqueued; a failed launch returns W4_ERR_CUDA.
 *   - K must be a positive multiple of 128, N positive, 1 <= M <= 8.
 */
#ifndef W4_H
#define W4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
/* The same object as cudaStream_t. */
typedef struct CUstream_st *w4_stream_t;

typedef enum w4_status {
    W4_OK = 0,
    W4_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, zero point > 15 */
    W4_ERR_UNSUPPORTED = 2,   /* M outside 1..8, or a call not allowed in stream capture */
    W4_ERR_LAYOUT = 3,        /* repacked buffer header does not match */
    W4_ERR_CUDA = 4,          /* a CUDA runtime call or kernel launch failed */
    W4_ERR_SCRATCH_LIMIT = 5  /* needs more than W4_STATIC_SCRATCH_BYTES of scratch */
} w4_status;

#define W4_GROUP_SIZE 128
#define W4_MAX_TOKENS 8
#define W4_LAYOUT_ID 1
#define W4_LAYOUT_ID_SWIGLU 2      /* gate/up-interleaved layout (w4_repack_swiglu) */
#define W4_LAYOUT_VERSION 4
#define W4_HEADER_BYTES 128
/* Size of the static device array behind w4_gemv_ws_static (4 MiB). */
#define W4_STATIC_SCRATCH_BYTES (4u * 1024u * 1024u)

/* Human-readable name of a status code (static string, never NULL). */
const char *w4_status_string(w4_status status);

/* Library version as major * 10000 + minor * 100 + patch. */
int w4_version(void);

/*
 * Sizes in bytes of the three buffers that w4_repack writes for an N x K
 * weight (the kernel layout): with NB = ceil(N / 128) row blocks and
 * G = K / 128 groups, qweight = W4_HEADER_BYTES + NB*G*8192, scales =
 * NB*G*256, zeros = NB*G*64.  The qweight buffer starts with a header
 * (layout id, version, K, N, error words).  Rows are padded to a multiple of
 * 128 with zero weights; the padding is never written back as output.
 * Errors: W4_ERR_INVALID_ARG for bad K/N or a NULL output pointer.
 */
w4_status w4_repacked_sizes(int K, int N, size_t *qweight_bytes,
                            size_t *scales_bytes, size_t *zeros_bytes);

/*
 * Offline, once per weight matrix: canonical layout -> kernel layout.
 * The offline packing step of "Building an LLM Inference Runtime ...",
 * sections "The Stack Architecture" and "Bug #3" (the runtime consumes one
 * fixed nibble interleave and refuses any other layout id).
 *
 *   qweight, scales, zeros : device, canonical layout (see top); qweight 16-byte
 *                            aligned, scales 2-byte aligned
 *   qweight_out, scales_out, zeros_out : device, sizes from w4_repacked_sizes,
 *                            each 16-byte aligned
 *
 * Validates every zero point on the device (must be <= 15) and therefore
 * synchronises `stream` before returning: not capturable into a CUDA graph
 * (returns W4_ERR_UNSUPPORTED if `stream` is capturing).
 * Errors: W4_ERR_INVALID_ARG (bad sizes/pointers, or a zero point > 15 -- the
 * outputs are then unspecified), W4_ERR_CUDA.
 */
w4_status w4_repack(const uint32_t *qweight, const uint16_t *scales,
                    const uint8_t *zeros, int K, int N, void *qweight_out,
                    void *scales_out, void *zeros_out, w4_stream_t stream);

/*
 * Host-side check of a repacked qweight buffer's header.  `header` is a host
 * copy of its first W4_HEADER_BYTES bytes.  Returns W4_OK when the magic,
 * layout id and version are this library's and K, N match; W4_ERR_LAYOUT
 * otherwise; W4_ERR_CUDA if a w4_gemv on this weight recorded that it gave up
 * waiting for its own copies (see w4_gemv); W4_ERR_INVALID_ARG for NULL.
 */
w4_status w4_check_header(const void *header, int K, int N);

/*
 * Weights to fp16, for checking: w_out[n][k] = fp16((q - z) * s), the exact
 * product rounded once to nearest-even.  Takes the canonical layout.
 * The "one thread per packed word, read once, unpack all eight" dequantiser of
 * "Custom AWQ Dequantization Kernel", section "Kernel versions" (v2).
 *
 *   qweight, scales, zeros : device, canonical; qweight 16-byte aligned
 *   w_out                  : device, uint16 [N][K] binary16 bits, 16-byte aligned
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_CUDA.  Zero points > 15 are used as given.
 */
w4_status w4_dequant(const uint32_t *qweight, const uint16_t *scales,
                     const uint8_t *zeros, int K, int N, uint16_t *w_out,
                     w4_stream_t stream);

/*
 * The hot path: y = W x with W in the kernel layout written by w4_repack.
 * Dequantisation happens in registers; fp32 accumulation; deterministic (the
 * same inputs give bit-identical y on every call) and batch-invariant (row m
 * of y does not depend on M or on the other rows of x).  Graph-capturable:
 * no synchronisation, allocation or host read.
 * Fused dequantise-and-multiply GEMV of "CodeAlign-Runtime", section "Level 3",
 * and "qengine", section "How it works" (4-bit matrix-vector kernel, partial
 * sums added in a fixed order).
 *
 *   qweight, scales, zeros : device, the three buffers of w4_repack, each
 *                            16-byte aligned
 *   x                      : device, bfloat16 [M][K], 16-byte aligned
 *   y                      : device, bfloat16 [M][N], 2-byte aligned
 * The header is not read here (that would need a device read); check it once
 * with w4_check_header.  Every wait inside the kernel is bounded: a block that
 * gives up (about 2 s without progress -- never in normal operation) sets the
 * header's error word, which w4_check_header then reports, and leaves its
 * outputs unwritten.  So although qweight is passed as const, its buffer must
 * be writable device memory: the kernel may write that one 32-bit word of the
 * header (byte offset 28) and nothing else of it.  Weights, scales and zeros
 * must not be written by work still running on the device when w4_gemv is
 * enqueued.  The kernel writes no memory beyond y except that error word.
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (M outside 1..8), W4_ERR_CUDA.
 */
w4_status w4_gemv(const void *qweight, const void *scales, const void *zeros,
                  const uint16_t *x, uint16_t *y, int M, int K, int N,
                  w4_stream_t stream);

/* Same as w4_gemv but writes the fp32 result before the bfloat16 cast
 * (y: device float [M][N], 4-byte aligned).  For checking. */
w4_status w4_gemv_f32(const void *qweight, const void *scales, const void *zeros,
                      const uint16_t *x, float *y, int M, int K, int N,
                      w4_stream_t stream);

/*
 * The product for any number of tokens M >= 1.  Up to 16 tokens it is w4_gemv
 * in passes of at most 8 tokens (one or two passes over the weight; row m is
 * bit-identical to w4_gemv on that token alone).  For more tokens the weight
 * is read once, in one pass on the tensor cores, where passes of 8 tokens
 * ("qengine", section "How the numbers were measured") would stream it once
 * per pass: a thread block owns a 128-row block of W and a tile of up to 128
 * tokens; per 128-k group it unpacks (q - z) exactly to bf16 into tensor
 * memory, multiplies it by the tile's x on the tensor cores with fp32
 * accumulation, and adds s times the group's sum into the token's fp32
 * result, group by group in order (the arithmetic of the GEMV's exact path).
 * There a token's result does not depend on M (> 16) or on which tokens share
 * its tile, and repeated calls give the same bits; its rows are not
 * bit-identical to w4_gemv's (different summation order inside a group), both
 * lying within the stated tolerances of the oracle.  Long K with few row
 * blocks is split over up to 8 blocks of a thread-block cluster, combined in
 * a fixed order.
 *   qweight, scales, zeros, y [M][N], stream : as for w4_gemv
 *   x [M][K]  : as for w4_gemv; for M > 16 read with tensor copies, so its
 *               address must be 16-byte aligned
 * The kernels may write the header's error word (byte offset 28), as w4_gemv.
 * For M > 16 every thread block takes all of its SM's tensor memory while it
 * runs: a kernel on another stream holding tensor memory on the same SM
 * delays it until that memory is freed.
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (M < 1, or for M > 16:
 * M * K >= 2^40, more than 65535 tiles of 128 tokens, or a weight of 2^25 or
 * more 128 x 128 records), W4_ERR_CUDA; in passes, the first error stops the
 * rest.
 */
w4_status w4_gemm(const void *qweight, const void *scales, const void *zeros, const uint16_t *x,
                  uint16_t *y, int M, int K, int N, w4_stream_t stream);

/* w4_gemm writing the fp32 result before the bfloat16 cast (y: float [M][N]). */
w4_status w4_gemm_f32(const void *qweight, const void *scales, const void *zeros,
                      const uint16_t *x, float *y, int M, int K, int N, w4_stream_t stream);

/*
 * Workspace for w4_gemv_ws on the current device, in bytes (depends on K, N
 * and the SM count only).  Errors: W4_ERR_INVALID_ARG, W4_ERR_CUDA (no device).
 */
w4_status w4_gemv_workspace_bytes(int K, int N, size_t *bytes);

/*
 * The same product as w4_gemv, split evenly over one wave of thread blocks
 * (three per SM): every block streams an equal contiguous run of the weight's
 * 128-row x 128-k records, and the row blocks that fall between two blocks
 * are combined through `workspace` by the last block to finish its part, in a
 * fixed order (deterministic, no float atomics, no block ever waits for
 * another).  It needs no thread-block clusters and never launches more than
 * three blocks per SM, for callers that want that footprint; on the shapes
 * measured on GB300, w4_gemv is faster.  Same result for a token whatever M
 * is; bit-identical across calls.
 *
 *   qweight, scales, zeros, x, y : as for w4_gemv
 *   workspace       : device, 256-byte aligned, at least
 *                     w4_gemv_workspace_bytes(K, N) bytes, all zero before its
 *                     first use.  It starts with one 32-bit counter per
 *                     128-row block (padded to a multiple of 256 bytes), which
 *                     every completed call leaves at zero again; the rest holds
 *                     the partial sums of the last call.  So one workspace
 *                     serves any number of calls in a row, but calls that
 *                     share it must not overlap on the device; after a call
 *                     that reported a kernel error, zero it again.
 * Errors: W4_ERR_INVALID_ARG (also for a short or misaligned workspace),
 * W4_ERR_UNSUPPORTED (M outside 1..8), W4_ERR_CUDA.
 */
w4_status w4_gemv_ws(const void *qweight, const void *scales, const void *zeros,
                     const uint16_t *x, uint16_t *y, int M, int K, int N, void *workspace,
                     size_t workspace_bytes, w4_stream_t stream);

/* w4_gemv_ws writing the fp32 result before the bfloat16 cast (y: device
 * float [M][N], 4-byte aligned).  For checking. */
w4_status w4_gemv_ws_f32(const void *qweight, const void *scales, const void *zeros,
                         const uint16_t *x, float *y, int M, int K, int N, void *workspace,
                         size_t workspace_bytes, w4_stream_t stream);

/*
 * w4_gemv_ws without a caller workspace: the scratch lives in a static device
 * array of W4_STATIC_SCRATCH_BYTES inside the library, and this call allocates
 * nothing (no cudaMalloc, no cudaFree, no allocating library routine).  The
 * paper has no counterpart of this entry point; it is here for callers that
 * cannot allocate device memory where they call the GEMV -- code running
 * inside an allocator or memory-pool callback (an allocation there would
 * re-enter the allocator), a plug-in of a host program that has reserved all
 * device memory up front and hands out only the buffers it manages, or a
 * latency-bound path that must not take the device-wide synchronisation and
 * the failure mode of cudaMalloc.
 *
 *   qweight, scales, zeros, x, y, M, K, N, stream : as for w4_gemv
 *
 * The array costs W4_STATIC_SCRATCH_BYTES on every GPU that loads libw4,
 * held until the process exits.  The first call on a device (the current one)
 * looks up the array's device address; make that first call before any
 * stream capture.  Every call on a device uses the same array, which keeps
 * the last call's contents: each call clears the row-block counters it uses
 * (an asynchronous memset on `stream`) and overwrites the partial sums before
 * reading them, so consecutive calls are independent, but calls that overlap
 * on the GPU (other streams, other host threads) race and give wrong results.
 * A product needs w4_gemv_workspace_bytes(K, N) bytes of scratch; more than
 * W4_STATIC_SCRATCH_BYTES is refused with W4_ERR_SCRATCH_LIMIT before
 * anything else is checked or enqueued.  That need depends on the SM count:
 * with NB = ceil(N / 128) row blocks and W = NB * K / 128 records, it is
 * round_up(4 * NB, 256) bytes of counters plus 2 * min(W, 3 * SMs) * 4096
 * bytes of partial sums.  On a 152-SM GB300 the partial sums take at most
 * 3.56 MiB, which leaves room for about 114,000 row blocks (14.6 M output
 * rows); on a GPU with 171 or more SMs the partial sums alone exceed the
 * array for every product of at least 3 * SMs records.
 * Errors: W4_ERR_SCRATCH_LIMIT, W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (M
 * outside 1..8), W4_ERR_CUDA (no device, or the array could not be found).
 */
w4_status w4_gemv_ws_static(const void *qweight, const void *scales, const void *zeros,
                            const uint16_t *x, uint16_t *y, int M, int K, int N,
                            w4_stream_t stream);

/*
 * Gated MLP input projection with the SwiGLU activation fused into the
 * product ("qengine", section "How it works": gate and up projections
 * interleaved so that SwiGLU runs in registers).  The weight is the fused
 * [2I][K] matrix of the gate projection (rows 0..I-1) and the up projection
 * (rows I..2I-1), canonical layout as above; the result is
 *   y[m][j] = silu(g) * u,  g = sum_k Wgate[j][k] x[m][k],
 *   u = sum_k Wup[j][k] x[m][k],  silu(g) = g / (1 + exp(-g)),
 * with g and u accumulated exactly as by w4_gemv_f32 and the activation and
 * product in fp32.
 *
 * w4_repacked_sizes_swiglu: byte sizes of the three buffers of the
 *   interleaved layout for I outputs (16 * ceil(I / 8) kernel rows).
 * w4_repack_swiglu: as w4_repack, for the fused [2I][K] weight (qweight
 *   uint32 [2I][K/8], scales [2I][K/128], zeros [2I][K/128]); the header
 *   records layout W4_LAYOUT_ID_SWIGLU and N = I.  Synchronises; refuses
 *   stream capture (W4_ERR_UNSUPPORTED); zero points > 15 -> W4_ERR_INVALID_ARG.
 * w4_check_header_swiglu: as w4_check_header for that layout and I.
 * w4_gemv_swiglu: y bfloat16 [M][I] (round to nearest even); arguments as
 *   for w4_gemv with N replaced by I; the weight buffers must come from
 *   w4_repack_swiglu.  w4_gemv_swiglu_f32: the fp32 result.
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (M outside 1..8),
 * W4_ERR_CUDA.
 */
w4_status w4_repacked_sizes_swiglu(int K, int I, size_t *qweight_bytes, size_t *scales_bytes,
                                   size_t *zeros_bytes);
w4_status w4_repack_swiglu(const uint32_t *qweight, const uint16_t *scales, const uint8_t *zeros,
                           int K, int I, void *qweight_out, void *scales_out, void *zeros_out,
                           w4_stream_t stream);
w4_status w4_check_header_swiglu(const void *header, int K, int I);
w4_status w4_gemv_swiglu(const void *qweight, const void *scales, const void *zeros,
                         const uint16_t *x, uint16_t *y, int M, int K, int I,
                         w4_stream_t stream);
w4_status w4_gemv_swiglu_f32(const void *qweight, const void *scales, const void *zeros,
                             const uint16_t *x, float *y, int M, int K, int I,
                             w4_stream_t stream);

/* Quantisation rules for w4_quantize. */
#define W4_QUANT_ASYMMETRIC 0
#define W4_QUANT_SYMMETRIC 1

/*
 * Quantise binary16 weights to the canonical layout, per row and group of
 * 128 consecutive weights along K, computing in fp32 from the exact binary16
 * values with every operation rounded to nearest (ties to even); the codes
 * are taken against the stored fp16 scale, so (q - z) * s is the value the
 * product uses:
 *   W4_QUANT_ASYMMETRIC: lo = min(0, min w), hi = max(0, max w),
 *     s = fp16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15),
 *     q = clamp(rint(w / s) + z, 0, 15)  (round to nearest with a zero point
 *     per group: the storage format of this library);
 *   W4_QUANT_SYMMETRIC: s = fp16(max |w| / 7), z = 8,
 *     q = clamp(rint(w / s), -8, 7) + 8  (the pages' scheme: scale = absmax
 *     / 7, "Building an LLM Inference Runtime ...", section "The Stack
 *     Architecture: A One-Page Overview"; values in [-8, 7],
 *     "CodeAlign-Runtime", section "Level 3 -- INT4 Quantization + Fused
 *     Kernel"; stored with the fixed zero point 8).
 * A group whose scale rounds to 0 stores s = 0 and q = z.
 *
 *   w       : device, binary16 bit patterns [N][K], 16-byte aligned; finite
 *   mode    : W4_QUANT_ASYMMETRIC or W4_QUANT_SYMMETRIC
 *   qweight : device, uint32 [N][K/8] (canonical nibble order), 4-byte aligned
 *   scales  : device, binary16 [N][K/128], 2-byte aligned
 *   zeros   : device, uint8 [N][K/128]
 * Outputs are written completely; w4_repack then gives the kernel layout.
 * Errors: W4_ERR_INVALID_ARG (bad pointers, sizes or mode), W4_ERR_CUDA.
 */
w4_status w4_quantize(const uint16_t *w, int K, int N, int mode, uint32_t *qweight,
                      uint16_t *scales, uint8_t *zeros, w4_stream_t stream);

/*
 * The launch shape w4_gemv uses for an N x K weight on the current device:
 * 16-row tiles per thread block, the number of K splits (thread blocks of
 * one cluster that each reduce a slice of K and combine in a fixed order),
 * and whether the zero point is folded out of the inner product (1: fp16
 * operands 1024 + q and 1024 + 16 q with x scaled per token into fp16
 * range, the zero point removed once per group and output through the
 * group's half sums of x, chosen when a block streams at least 8 groups;
 * 0: the bf16 tensor-core operand is q - z, exactly).  Both are the same sum
 * up to fp32 rounding.  Depends on K and N only, never on M.  Outputs may be
 * NULL.
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_CUDA (no device).
 */
w4_status w4_gemv_config(int K, int N, int *tiles_per_block, int *k_splits,
                         int *zero_point_folded);

/* How w4_gemv launches a product (filled by w4_gemv_plan). */
typedef struct w4_gemv_launch_info {
    int k_splits;            /* thread blocks per cluster, each reducing a slice of K */
    int zero_point_folded;   /* 1: fp16 operands, zero point folded out; 0: exact q - z */
    int grid_x, grid_y;      /* launch grid: row blocks (or persistent slots) x K splits */
    int persistent;          /* 1: each block takes row blocks in turn */
    int overlap;             /* 1: launched with programmatic dependent launch (starts
                                while the previous kernel in the stream finishes) */
    int capped;              /* 1: shared memory padded so that at most the needed
                                number of blocks share an SM */
    int ring_stages;         /* depth of the shared-memory weight ring */
    int wide_prologue;       /* 1: folded x prologue spread over (group, token) pairs */
    int blocks_per_sm_max;   /* blocks per SM the kernel instance is built for */
    size_t smem_bytes;       /* dynamic shared memory per block */
} w4_gemv_launch_info;

/*
 * Diagnostic with no counterpart in the pages: the launch w4_gemv makes for
 * M tokens of an N x K weight on the current device (split, arithmetic, grid,
 * residency, overlap), so that callers and tests can see which kernel path a
 * shape takes.  Computes the same plan w4_gemv computes before each launch;
 * launches nothing.
 *   info : host, written on success
 * Errors: W4_ERR_INVALID_ARG (bad K/N, NULL info), W4_ERR_UNSUPPORTED (M
 * outside 1..8, or no launch shape fits), W4_ERR_CUDA (no device).
 */
w4_status w4_gemv_plan(int M, int K, int N, w4_gemv_launch_info *info);

/*
 * Diagnostic with no counterpart in the pages: runs, in one thread of one
 * block, the bounded mbarrier wait the GEMV kernels use on a barrier that
 * nothing ever completes, and stores into *status (device, 4-byte aligned)
 * 1 if the wait gave up after its limit (about 2 s of clock cycles, the
 * expected outcome) or 0 if it wrongly returned success.  Shows on a real
 * GPU that a wait which can never finish ends, reports, and leaves the
 * context usable.  Asynchronous on `stream`; takes about 2 s on the GPU.
 * Errors: W4_ERR_INVALID_ARG (status NULL or misaligned), W4_ERR_CUDA.
 */
w4_status w4_selftest_bounded_wait(uint32_t *status, w4_stream_t stream);

/* Modes of w4_stream_read. */
#define W4_STREAM_READ_RING 0
#define W4_STREAM_READ_LD128 1

/*
 * Diagnostic: reads `bytes` of device memory once and folds them into one
 * word, to measure the read-only bandwidth a kernel gets on this GPU -- the
 * ceiling a memory-bound GEMV is judged against ("qengine", section
 * "Learnings": measure your own ceiling with a plain read benchmark; a copy
 * also writes, and the data sheet is a peak no kernel reaches).
 *   W4_STREAM_READ_RING : the GEMV's own method -- contiguous shares of the
 *     buffer moved in 8 KB cp.async.bulk records through a 12-stage
 *     shared-memory ring, two blocks per SM; `bytes` a multiple of 8192.
 *   W4_STREAM_READ_LD128: 16-byte streaming loads in a grid-stride loop, four
 *     blocks of 512 threads per SM; `bytes` a multiple of 16.
 *   src : device, 16-byte aligned
 *   out : device uint32 [2]; out[0] is xor-ed with the folded word, out[1]
 *         gets bit 0 if a bounded wait gave up (never in normal operation)
 * Asynchronous on `stream`; time it with events around the call.
 * Errors: W4_ERR_INVALID_ARG (pointers, alignment, size, mode), W4_ERR_CUDA.
 */
w4_status w4_stream_read(const void *src, size_t bytes, int mode, uint32_t *out,
                         w4_stream_t stream);

/* ======================================================================
 * Rotary positions, a paged key-value cache and attention over it: what a
 * decoder layer does between its qkv product and its o product.  (The paged
 * cache and its decode attention: "Building an LLM Inference Runtime ...",
 * section "The Stack Architecture: A One-Page Overview"; partial results over
 * pieces of the length, joined by their log-sum-exp: "CodeAlign-Runtime",
 * section "Level 4"; 1..8 new tokens: "qengine", section "How it works".)
 *
 * Like the products, every call below enqueues work on `stream`, allocates
 * nothing, checks its arguments on the host and can be captured in a CUDA
 * graph.  The structures are host memory, read during the call.  Positions,
 * lengths and block tables are device memory and are checked by the kernels:
 * what is out of range is left out and recorded in the caller's error word
 * (device uint32, may be NULL; the kernels only ever set bits of it):
 */
#define W4_KV_ERR_POSITION 1u    /* a position past the rotation table or the block table */
#define W4_KV_ERR_PAGE 2u        /* a page number outside the pool */
#define W4_KV_ERR_SEQUENCE 4u    /* a sequence number outside the block table */
#define W4_KV_ERR_LENGTH 8u      /* a length past the block table (it is cut to it) */
#define W4_KV_ERR_WAIT 16u       /* a kernel gave up waiting for its own copies */
#define W4_KV_ERR_BLOCK 32u      /* a listed block outside its sequence, or out of order */

/* A bfloat16 tensor [tokens][heads][head_dim] whose last dimension is
 * contiguous; strides in elements (may be those of a slice of a wider row,
 * such as the q heads of a fused qkv product). */
typedef struct w4_heads {
    void *data;                  /* device; only read where the call takes it as an input */
    int64_t token_stride;
    int64_t head_stride;
} w4_heads;

/* Which values of a head form a pair: i and i + rotary_dim/2, or 2i and 2i+1. */
#define W4_ROPE_HALF 0
#define W4_ROPE_INTERLEAVED 1

/* A table of rotations: (cos, sin) pairs, float [rows][rotary_dim/2][2], row p
 * for position p.  Filled by w4_rope_table, or by the caller. */
typedef struct w4_rotation {
    const float *table;          /* device, 16-byte aligned */
    int rows;
    int rotary_dim;              /* even; the first rotary_dim values of a head are rotated */
    int layout;                  /* W4_ROPE_HALF or W4_ROPE_INTERLEAVED */
} w4_rotation;

/* How frequencies are scaled for contexts longer than the trained one. */
#define W4_ROPE_SCALE_NONE 0     /* f_i = base^(-2i/rotary_dim) */
#define W4_ROPE_SCALE_LINEAR 1   /* f_i / factor */
#define W4_ROPE_SCALE_BASE 2     /* base * factor^(rotary_dim/(rotary_dim-2)) instead of base */
#define W4_ROPE_SCALE_PARTS 3    /* between f_i / factor, for pairs that make at most low_turns
                                    turns in original_context positions, and f_i, for those that
                                    make at least high_turns; linear in the turns between.  (A
                                    model whose table is linear in the pair's index i instead,
                                    between two whole indices, brings its own table.) */
typedef struct w4_rope_spec {
    int rotary_dim;              /* even, 2..512 */
    int scaling;
    double base;                 /* > 0 */
    double factor;               /* > 0 (ignored by W4_ROPE_SCALE_NONE) */
    double original_context;     /* W4_ROPE_SCALE_PARTS: > 0 */
    double low_turns;            /* W4_ROPE_SCALE_PARTS: low_turns < high_turns */
    double high_turns;
    double amplitude;            /* cos and sin are multiplied by it (1: a plain rotation) */
} w4_rope_spec;

/*
 * Fills rows 0..rows-1 of a rotation table: amplitude * (cos, sin)(p * f_i).
 * The angle p * f_i is reduced to a fraction of a turn in 64-bit integers, so
 * whole turns drop out exactly: the angle is within p * f_i * 2^-52 of that of
 * the double-precision f_i, and the entry is that angle's within 1 ulp.
 *   table : device, float [rows][rotary_dim/2][2], 16-byte aligned
 * Errors: W4_ERR_INVALID_ARG (a base or frequency that comes out infinite
 * too), W4_ERR_CUDA.
 */
w4_status w4_rope_table(const w4_rope_spec *spec, int rows, float *table, w4_stream_t stream);

/*
 * y[t][h] = x[t][h] with its first rotary_dim values rotated by the table's
 * row positions[t]; for a pair (a, b): (a c - b s, b c + a s), every operation
 * rounded to fp32 once, the results rounded to bfloat16 once; the other
 * values of the head are copied.  A negative position -p rotates back by row
 * p: that is the transposed map, so it turns gradients of y into gradients
 * of x.
 *   x, y      : device, 2-byte aligned.  y may be x (same strides); otherwise
 *               they must not overlap.  Rows that are 16-byte aligned (data,
 *               strides, rotary_dim a multiple of 16) go by 16-byte accesses.
 *   tokens    : >= 0 (0: nothing is done);  heads >= 1
 *   head_dim  : 1..1024, at least rotary_dim
 *   positions : device int32 [tokens]; a token whose |position| is not a row
 *               of the table is left out (W4_KV_ERR_POSITION)
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (2^31 or more blocks of
 * work), W4_ERR_CUDA.
 */
w4_status w4_rope(const w4_heads *x, const w4_heads *y, int tokens, int heads, int head_dim,
                  const int32_t *positions, const w4_rotation *rotation, uint32_t *error,
                  w4_stream_t stream);

/* Storage formats of a paged cache. */
#define W4_KV_BF16 0
#define W4_KV_INT8 1
#define W4_KV_INT4 2

/*
 * Paged key-value cache.  The pool is an array of records; a record holds the
 * keys and values of 16 consecutive tokens of one key/value head:
 *   record of (page p, head h, tokens 16i..16i+15 of the page) =
 *     number (p * kv_heads + h) * (page_tokens / 16) + i
 * so the record of 16 tokens is one contiguous copy, whatever the page size.
 * With D = head_dim and r = 0..15 a token of the record, its bytes are
 *   keys    16 rows of D values, row r for token r
 *     bf16: 2D bytes a row; the 16-byte piece c of a row is stored as piece c ^ (r & 7)
 *     int8: D bytes a row; for D = 128, piece c is stored as piece c ^ (4 * (r & 1))
 *     int4: D/2 bytes a row; value d is nibble d & 1 of byte d / 2
 *   values
 *     bf16: as the keys
 *     int8: value d of token r is byte d/32 * 512 + L * 16 + (d/8 % 4) * 4 + B
 *     int4: value d of token r is nibble (d/8 & 1) of byte
 *           d/64 * 512 + L * 16 + (d/16 % 4) * 4 + B
 *           with L = 4 * (d & 7) + (r & 7) / 2 and B = 2 * (r & 1) + r / 8:
 *           the order in which the tensor cores' lanes take them
 *   int8, int4: then 16 key and 16 value descriptors, uint32: binary16 scale
 *           s | zero point z << 16
 * for 64 D bytes (bf16), 32 D + 128 (int8) or 16 D + 128 (int4) in all.
 * A token's key (value) of a head is one group, quantised with a zero point to
 * Q = 255 or 15 levels, in fp32, each operation rounded to nearest even:
 * lo = min(0, min x), hi = max(0, max x), s = binary16((hi - lo) * r) with r the
 * fp32 value of 1 / Q (s at most 65504), z = clamp(rint(-lo / s), 0, Q),
 * q = clamp(rint(x / s) + z, 0, Q), read back as (q - z) * s; s = 0 stores
 * z = q = 0.  An infinite value is held as the largest that the scale reaches,
 * NaN as 0; bf16 caches keep both.
 */
typedef struct w4_kv_cache {
    void *pool;                  /* device, 128-byte aligned, w4_kv_pool_bytes() bytes */
    int format;                  /* W4_KV_* */
    int kv_heads;                /* >= 1 */
    int head_dim;                /* 64 or 128 */
    int page_tokens;             /* a multiple of 16 */
    int pages;                   /* >= 1 */
    uint32_t *error;             /* device error word, 4-byte aligned, or NULL */
} w4_kv_cache;

/* Block table: pages[b * stride + i] is the page with tokens i * page_tokens ..
 * (i+1) * page_tokens - 1 of sequence b. */
typedef struct w4_block_table {
    const int32_t *pages;        /* device int32 */
    int seqs;                    /* rows, >= 1 */
    int width;                   /* pages a row, >= 1 */
    int64_t stride;              /* row stride, >= width */
} w4_block_table;

/* Bytes of a pool (pool, error and block contents are not looked at).
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (head_dim). */
w4_status w4_kv_pool_bytes(const w4_kv_cache *cache, size_t *bytes);

/*
 * Writes new tokens into the cache, rotating q (into q_out) and k on the way:
 * the one launch between the qkv product and the attention.  Token t is at
 * positions[t] of sequence seq_ids[t]; no two tokens of a call may name the
 * same place, and other tokens of the records that are touched stay as they
 * are.  k is rotated in fp32 and quantised from there; v is taken as it is.
 *   k, v      : device [tokens][kv_heads][head_dim], rows 16-byte aligned
 *   q, q_out  : device [tokens][q_heads][head_dim], rows 16-byte aligned, or
 *               both NULL; q_out may be q; without a rotation q is copied
 *   positions : device int32 [tokens]; a negative one marks padding: the token
 *               is left out
 *   seq_ids   : device int32 [tokens], or NULL: tokens is a multiple of
 *               table->seqs and every sequence has tokens / seqs consecutive ones
 *   rotation  : NULL for none; rotary_dim a multiple of 16, at most head_dim
 * A token that is out of range (position, sequence, page) is left out whole,
 * its q too, and recorded in cache->error.
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (head_dim; 2^27 or more
 * tokens x heads of k, v and q), W4_ERR_CUDA.
 */
w4_status w4_kv_append(const w4_kv_cache *cache, const w4_heads *k, const w4_heads *v,
                       const w4_heads *q, const w4_heads *q_out, int q_heads, int tokens,
                       const int32_t *positions, const int32_t *seq_ids,
                       const w4_block_table *table, const w4_rotation *rotation,
                       w4_stream_t stream);

/*
 * Reads tokens back, in any order: k_out[t], v_out[t] = the cached key and
 * value of positions[t] of sequence seq_ids[t], (q - z) * s rounded once to
 * bfloat16.  Tokens that are negative or out of range are left out as above.
 * Arguments as for w4_kv_append; k_out or v_out may be NULL.
 */
w4_status w4_kv_read(const w4_kv_cache *cache, const w4_heads *k_out, const w4_heads *v_out,
                     int tokens, const int32_t *positions, const int32_t *seq_ids,
                     const w4_block_table *table, w4_stream_t stream);

/* Bytes of workspace for w4_paged_attn on the current device: it depends on
 * head_dim and the SM count only.  Errors: W4_ERR_INVALID_ARG,
 * W4_ERR_UNSUPPORTED, W4_ERR_CUDA. */
w4_status w4_paged_attn_workspace_bytes(const w4_kv_cache *cache, size_t *bytes);

/*
 * Attention of the last `tokens` tokens of every sequence over its cache.
 * lens[b] counts the cached tokens of sequence b, the new ones included: new
 * token i is at position p = lens[b] - tokens + i and sees the keys
 * j <= p, and j > p - window where window > 0.  With the row of q of token
 * b * tokens + i and head h, and the key/value head h / (q_heads / kv_heads):
 *   out = sum_j softmax_j(scale * q . k_j) v_j,
 *   lse = ln sum_j exp(scale * q . k_j)
 * A row that sees no key (lens[b] = 0, or p < 0) gives out = 0, lse = -inf.
 * What the pool holds past lens[b] is never looked at (it may be NaN).
 * Products on the tensor cores: bf16 operands for a bf16 cache, exact codes
 * against fp16 for the quantised ones; scores, maxima, sums and outputs are
 * fp32; probabilities enter the second product in two bf16 parts (16 bits in
 * all), against codes as fp16.  The sums' order depends on the lengths, the
 * window and the device only, never on which block finishes first: repeated
 * calls give the same bits.
 *   q      : device [seqs * tokens][q_heads][head_dim] bf16, rows 16-byte aligned
 *   out    : device [seqs * tokens][q_heads][head_dim] bf16, rows 16-byte aligned
 *            (w4_paged_attn_f32: float, rows 16-byte aligned)
 *   lse    : device float [seqs * tokens][q_heads], or NULL
 *   tokens : 1..8;  q_heads : a multiple of kv_heads, at most 4096 times it
 *   lens   : device int32 [table->seqs]; negative counts as 0
 *   scale  : finite; usually head_dim^-0.5
 *   window : >= 0; 0, or as many as the table has room for, leave nothing out
 *   workspace : device, 256-byte aligned; calls that overlap on the device must
 *            not share one; what it holds between calls does not matter
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (tokens, head_dim, a table with
 * room for more than 2^31 - 256 tokens a sequence, or one that with the heads
 * allows 2^31 or more visits of records), W4_ERR_CUDA.
 */
w4_status w4_paged_attn(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                        int q_heads, int tokens, const int32_t *lens,
                        const w4_block_table *table, float scale, int window, float *lse,
                        void *workspace, size_t workspace_bytes, w4_stream_t stream);
w4_status w4_paged_attn_f32(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                            int q_heads, int tokens, const int32_t *lens,
                            const w4_block_table *table, float scale, int window, float *lse,
                            void *workspace, size_t workspace_bytes, w4_stream_t stream);

/* ======================================================================
 * Long contexts: attention over the blocks of a cache that a cheap score
 * selects, and eviction of the tokens that got little attention.  A block is a
 * page of the cache: block n of a sequence is its tokens n * page_tokens ..
 * (n+1) * page_tokens - 1.  (None of the pages has them; they work on the cache
 * above, in its manner: lengths and lists are device memory, checked by the
 * kernels.)
 *
 * A decode step that reads a part of the cache:
 *   w4_kv_append, w4_key_bounds (the blocks that got new keys), w4_block_scores,
 *   w4_select (unit = page_tokens), w4_sparse_attn.  New tokens see themselves and
 *   one another where their blocks are listed: 1 + (tokens + page_tokens - 2) /
 *   page_tokens last ones hold them.
 * Cutting a cache down to `count` tokens a head:
 *   w4_paged_attn, w4_attn_weights over the steps, then w4_select (unit = 1),
 *   w4_kv_gather into other pages; its counts are the sequences' new lengths.
 *   Kept keys stay rotated by the positions that they had.  A token that is
 *   appended later goes to the place after the kept ones, while its rotation
 *   goes by its position in the text: w4_rope, then w4_kv_append without a
 *   rotation.
 * ====================================================================== */

/*
 * Bounds of the keys of blocks: for every sequence, those that its last `tokens`
 * tokens lie in (after a decode step one or two, after a prompt all of it), and
 * every key/value head:
 *   bounds[page][head][0][d] = max, bounds[page][head][1][d] = min
 * over the block's tokens j < lens[b] of value d of key j, as w4_kv_read returns
 * it; if one of them is NaN, both are.  They go by page: a page that several
 * sequences share has to hold as many tokens in each of them (a full one does).
 * Otherwise every value is that of any one of them, and the bounds may hold for
 * none.
 *   bounds : device, bfloat16 [pages][kv_heads][2][head_dim], 16-byte aligned
 *   tokens : >= 1
 *   lens   : device int32 [table->seqs]; negative counts as 0
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (head_dim; a table with room for
 * more than 2^31 - 2^21 tokens a sequence, or for 2^31 or more records of 16
 * tokens, those of every head), W4_ERR_CUDA.
 */
w4_status w4_key_bounds(const w4_kv_cache *cache, uint16_t *bounds, int tokens,
                        const int32_t *lens, const w4_block_table *table, w4_stream_t stream);

/*
 * How large q . k can be in a block, from its bounds:
 *   scores[b][h][n] = max over the rows of sum_d (q_d >= 0 ? q_d hi_d : q_d lo_d)
 * the rows being the new tokens of sequence b (at positions lens[b] - tokens + i
 * >= 0) in the q_heads / kv_heads query heads of h; bf16 products summed in fp32.
 * One that is not finite (bounds or queries that are not) counts as +infinity, a
 * block whose page is not in the pool as -infinity.  Blocks from lens[b] on are
 * left as they were.  New tokens of one call share their scores: a call for
 * single tokens, or a table with a row for each, keeps them apart.
 *   bounds  : as w4_key_bounds fills it
 *   q       : device [seqs * tokens][q_heads][head_dim] bf16, rows 16-byte aligned
 *   tokens  : 1..8;  q_heads : a multiple of kv_heads, at most 4096 times it
 *   scores  : device float [seqs][kv_heads][columns]
 *   columns : >= table->width
 * The pool is not looked at.
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (tokens, head_dim, sizes as
 * above), W4_ERR_CUDA.
 */
w4_status w4_block_scores(const w4_kv_cache *cache, const uint16_t *bounds, const w4_heads *q,
                          int q_heads, int tokens, const int32_t *lens,
                          const w4_block_table *table, float *scores, int columns,
                          w4_stream_t stream);

/*
 * The best `count` items of every row, in ascending order: row (b, h) has
 * n = ceil(lens[b] / unit) items (`columns` at most) with a score each.  The first
 * `first` and the last `last` items are always chosen, then those with the
 * largest scores, of equal ones (0 and -0 are) the first; NaN counts as larger
 * than any number.  With n <= count all are chosen.
 *   index[b][h][i], i < counts[b] = min(n, count): the chosen items
 * Entries from counts[b] on are left as they were.
 *   scores : device float [seqs][heads][columns]
 *   lens   : device int32 [seqs]; negative counts as 0
 *   unit   : >= 1: page_tokens where items are blocks, 1 where they are tokens
 *   first, last : >= 0;  count : >= 1, at least first + last
 *   index  : device int32 [seqs][heads][count];  counts : device int32 [seqs]
 * index and counts must not overlap what is read.
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (2^27 or more rows, 2^30 or
 * more columns), W4_ERR_CUDA.
 */
w4_status w4_select(const float *scores, int seqs, int heads, int columns, const int32_t *lens,
                    int unit, int first, int last, int count, int32_t *index, int32_t *counts,
                    w4_stream_t stream);

/*
 * w4_paged_attn over listed blocks only: new token i sees the keys of the blocks
 * blocks[b][h][0 .. counts[b] - 1] at its own position p = lens[b] - tokens + i
 * and before.  All of them ascending, it gives what w4_paged_attn gives, up to
 * the order of sums.  The sums' order depends on the lengths, the lists and the
 * device only.
 *   blocks : device int32 [seqs][kv_heads][most], ascending; an entry that is not
 *            above the one before it, or no block of the sequence, is left out
 *            (W4_KV_ERR_BLOCK; a block that a list out of order names again later
 *            counts again)
 *   counts : device int32 [seqs]; taken as 0 below it, as most above it
 *   most   : >= 1
 * The other arguments, a row that sees no key, and the errors are those of
 * w4_paged_attn, the workspace too.
 */
w4_status w4_sparse_attn(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                         int q_heads, int tokens, const int32_t *lens,
                         const w4_block_table *table, const int32_t *blocks,
                         const int32_t *counts, int most, float scale, float *lse,
                         void *workspace, size_t workspace_bytes, w4_stream_t stream);
w4_status w4_sparse_attn_f32(const w4_kv_cache *cache, const w4_heads *q, const w4_heads *out,
                             int q_heads, int tokens, const int32_t *lens,
                             const w4_block_table *table, const int32_t *blocks,
                             const int32_t *counts, int most, float scale, float *lse,
                             void *workspace, size_t workspace_bytes, w4_stream_t stream);

/*
 * What the cached tokens get of the new tokens' attention, added to what they had:
 *   weights[b][h][j] = (j < lens[b] - tokens ? decay * before[b][h][j] : 0)
 *                      + sum over the rows that see key j of exp(scale q . k_j - lse)
 * for j < lens[b], the rows being those of w4_paged_attn (new tokens x query heads
 * of h) with its window, and lse what it returned for them (not w4_sparse_attn, which
 * leaves keys out): each row adds 1 in all.
 * The new tokens' own places start at 0, so weights need not be cleared.  Entries
 * from lens[b] on are left as they were.  A row whose lse is infinite gives
 * nothing; a key that no row sees, or whose page is not in the pool, gets nothing.
 * Sums are fp32, in an order that depends on the sizes alone.
 *   q       : as for w4_paged_attn
 *   lse     : device float [seqs * tokens][q_heads]
 *   before  : device float [seqs][kv_heads][columns], or NULL: 0; not read where
 *             decay is 0; may be weights, otherwise must not overlap it
 *   decay   : finite
 *   weights : device float [seqs][kv_heads][columns]
 *   columns : >= 1; a longer sequence is cut to it (W4_KV_ERR_LENGTH)
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (tokens, head_dim, sizes as for
 * w4_key_bounds), W4_ERR_CUDA.
 */
w4_status w4_attn_weights(const w4_kv_cache *cache, const w4_heads *q, const float *lse,
                          int q_heads, int tokens, const int32_t *lens,
                          const w4_block_table *table, float scale, int window,
                          const float *before, float decay, float *weights, int columns,
                          w4_stream_t stream);

/*
 * Moves listed tokens to other pages, as they are held, every key/value head its
 * own ones: place i of sequence b in the table `to` gets token index[b][h][i] of
 * the table `table`, for i < counts[b]; and their weights with them:
 *   weights_out[b][h][i] = weights[b][h][index[b][h][i]]
 * Indices may be in any order and repeat.  A place whose index is negative, or no
 * token of the sequence (W4_KV_ERR_POSITION), stays as it was, and so do other
 * places of the records that are touched.  With the lists of w4_select, counts are
 * the new lengths; the old pages are free afterwards.  (The new pages' keys have no
 * bounds yet: w4_key_bounds, with as many tokens.)
 *   table, to : of the same cache, with as many sequences.  No page that is
 *             written may be one that is read (two tables at one address are
 *             refused)
 *   lens    : device int32 [table->seqs], of `table`
 *   index   : device int32 [seqs][kv_heads][most]
 *   counts  : device int32 [seqs]; taken as 0 below it; above most or the room of
 *             `to` cut (W4_KV_ERR_LENGTH)
 *   weights : device float [seqs][kv_heads][columns], tokens from columns on are
 *             not there; weights_out : device float [seqs][kv_heads][columns_out],
 *             columns_out >= most, must not overlap it; or both NULL
 * Errors: W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED (head_dim, sizes as for
 * w4_key_bounds), W4_ERR_CUDA.
 */
w4_status w4_kv_gather(const w4_kv_cache *cache, const w4_block_table *table,
                       const int32_t *lens, const int32_t *index, const int32_t *counts, int most,
                       const w4_block_table *to, const float *weights, int columns,
                       float *weights_out, int columns_out, w4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W4_H */
