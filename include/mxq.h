/*
 * mxq.h -- C ABI of the GB300 MX block-quantization library (libmxq.so).
 *
 * Plain pointers and sizes only.  Every data pointer is a DEVICE pointer that
 * the caller owns (allocated, for example, with torch or cudaMalloc); the
 * library never allocates, never frees and never synchronizes inside these
 * calls.  Work is enqueued on the caller's `stream` (0 = legacy default
 * stream), so every call can be captured in a CUDA graph and ordered with the
 * caller's own work.  Kernels are launched with programmatic dependent launch:
 * one may be scheduled, and run its shared-memory set-up, while the previous
 * kernel on the stream is still running, but it touches no global memory
 * before that kernel has completed, so stream order is kept exactly.
 *
 * Return value: MXQ_OK (0) when the work was enqueued, a negative MXQ_E* code
 * when an argument was rejected (nothing is enqueued and no byte of any output
 * is touched) or when the launch failed.  Argument checks run on the host and
 * make no CUDA call, so a rejected call is safe on any thread and any device.
 * The library never aborts, throws or raises a device trap.
 *
 * Checks that need device data (the group offsets of mxq_quantize_2d_dual) are
 * made by the kernel itself: on failure it writes nothing and sets a bit in
 * the device status word of the current device (mxq_device_status).
 *
 * Sources for the operations (page title, section):
 *   [AO]  pytorch/ao PR #4995 "Fused dual-axis MXFP8 quantization with correct
 *         metadata" -- description and review replies.
 *   [MX9] AMD-AGI/ALTO PR #33 "mx9: add fused MX9 quantization kernel with
 *         pack/unpack" -- Summary, "Key design choices", review thread.
 */
#ifndef MXQ_H_
#define MXQ_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as the CUDA runtime's cudaStream_t (a repeated identical typedef
   is legal in C11 and C++). */
typedef struct CUstream_st *cudaStream_t;

/* ---- status codes ------------------------------------------------------ */
#define MXQ_OK 0
#define MXQ_EBADSHAPE (-1) /* a size is negative, too large, or violates the method's multiples */
#define MXQ_EBADDTYPE (-2) /* dtype code is not MXQ_F32 / MXQ_BF16 */
#define MXQ_EBADOFFS (-3)  /* group count out of range, or offs/G inconsistent */
#define MXQ_EALIGN (-4)    /* a pointer is not 16-byte aligned (offs: 4-byte) */
#define MXQ_EOVERLAP (-5)  /* two buffers' byte ranges overlap (or one wraps past the top of memory) */
#define MXQ_ECUDA (-6)     /* the CUDA runtime refused the launch */
#define MXQ_ENULL (-7)     /* a required pointer is NULL */
#define MXQ_ESCRATCH (-8)  /* needs more than the static scratch of the no-allocation call */

/* ---- dtype codes ------------------------------------------------------- */
#define MXQ_F32 0
#define MXQ_BF16 1

/* ---- limits ------------------------------------------------------------ */
#define MXQ_MAX_GROUPS 1024 /* largest G accepted by mxq_quantize_2d_dual */

/* ---- device status word bits (see mxq_device_status) ------------------- */
#define MXQ_DEV_BADOFFS 0x1u /* offs failed the device-side check: no output written */
#define MXQ_DEV_TIMEOUT 0x2u /* an internal pipeline wait gave up: outputs incomplete */
#define MXQ_DEV_OOB 0x4u     /* checked build only: a store out of its buffer was skipped */
#define MXQ_DEV_BADINDEX 0x8u /* an expert, row or table index was out of range and left out */

/*
 * Dual-axis MXFP8 quantization of one bf16 matrix, reading it once.
 * [AO] description: one read of x emits four outputs -- E4M3 data cast in 1x32
 * blocks along N (rowwise) and in 32x1 blocks along M (colwise), and the two
 * E8M0 "rceil" scale tensors already in the blocked layout that block-scaled
 * MMA consumes, with the colwise scales grouped by the K-group offsets and
 * zeroed for the uncovered tail past offs[G-1].
 *
 *   x      bf16 [M, N] row-major (2*M*N bytes), 16-byte aligned.
 *   M, N   multiples of 128, >= 0 (the [AO] description requires both sizes and
 *          every group size to be multiples of 128).  M == 0 or N == 0 is a
 *          no-op.
 *   offs   device int32 [G]: cumulative group ends, non-decreasing, each a
 *          multiple of 128, offs[G-1] <= M (empty groups allowed); 4-byte
 *          aligned.  NULL selects dense placement (one group [0, M)); then G
 *          must be 0.  1 <= G <= MXQ_MAX_GROUPS otherwise.
 *   q_row  E4M3 [M*N]: q_row[m*N + n]; 16-byte aligned.
 *   s_row  E8M0 [M*N/32]: the [M, N/32] scale matrix in the 128x4 blocked
 *          layout: scale (r, c) at ((r/128)*(C/4) + c/4)*512 + (r%32)*16 +
 *          ((r%128)/32)*4 + c%4 with C = N/32.
 *   q_col  E4M3 [N*M]: q_col[n*M + m], i.e. [N, M] row-major ("logically
 *          transposed colwise store").
 *   s_col  E8M0 [N*M/32]: group g = [lo, hi) owns bytes [N*lo/32, N*hi/32),
 *          its [N, (hi-lo)/32] colwise scale matrix in the same blocked
 *          layout; bytes from N*offs[G-1]/32 to the end are written as 0.
 *          Rows in the tail are still quantized in q_row, s_row and q_col.
 *   stream CUDA stream for the launch.
 * Scale and data rules ([AO] description, "Bug-compatible" list): the scale
 * byte is the smallest s with amax <= 448*2^(s-127); data is x*2^(127-s) cast
 * to E4M3 with round-to-nearest-even; a block with any NaN gets scale 255 and
 * all-NaN (0x7F) data on both axes; a block with +-Inf and no NaN gets scale
 * 255 and 0x7F data rowwise, and scale 254 with +-Inf saturated to +-448
 * colwise.
 * Buffers must not overlap one another, x or offs.  Every byte of every output
 * is written (for valid offs); outputs need no initialisation.
 */
int mxq_quantize_2d_dual(const void *x, int64_t M, int64_t N, const int32_t *offs, int32_t G,
                         uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                         cudaStream_t stream);

/*
 * The same cast on a band of rows [row0, row0 + rows) of a full [M, N] tensor,
 * for data-parallel shards along M.  The pages' tiles and blocks are
 * independent, so the band's outputs are exactly the full call's bytes at the
 * band's places; only s_col needs the band's position, because a group's slab
 * offset and width come from the full tensor's offs.
 *
 *   x      bf16 [rows, N]: the band (row0 .. row0+rows-1 of the full tensor).
 *   rows, row0, M, N   multiples of 128 with row0 + rows <= M; rows == 0 is a
 *          no-op.
 *   offs, G  the full tensor's K-group offsets (as for mxq_quantize_2d_dual,
 *          checked on the device against M); NULL and 0 for dense.
 *   q_row  E4M3 [rows*N]: rows row0.. of the full q_row.
 *   s_row  E8M0 [rows*N/32]: bytes [row0*N/32, (row0+rows)*N/32) of the full
 *          s_row (the blocked layout keeps a band of 128-row blocks together).
 *   q_col  E4M3 [N*rows]: [N, rows] row-major, columns row0.. of the full q_col.
 *   s_col  E8M0 [N*M/32]: the FULL colwise scale buffer; the call writes the
 *          512-byte atoms of its rows (and the zero atoms of its tail rows) and
 *          leaves every other byte alone, so bands that cover [0, M) once write
 *          every byte once, with no exchange between them.
 * Errors and device status as for mxq_quantize_2d_dual; MXQ_EBADSHAPE also for
 * a band outside [0, M).
 */
int mxq_quantize_2d_dual_rows(const void *x, int64_t rows, int64_t N, int64_t row0, int64_t M,
                              const int32_t *offs, int32_t G, uint8_t *q_row, uint8_t *s_row,
                              uint8_t *q_col, uint8_t *s_col, cudaStream_t stream);

/*
 * MX9 pack.  [MX9] Summary / "Key design choices": blocks of 16 consecutive
 * elements along the last axis (block b = r*(cols/16) + j); per block a
 * shared exponent E = max over the block of the element exponents taken from
 * the native bits (biased exponent field - 127: fp32 bits 30..23, bf16 bits
 * 14..7), stored as max_exp[b] = E + 127; per pair p of elements (2p, 2p+1) a
 * prime bit (bit p of prime[b], LSB = pair 0) set when the pair's exponent is
 * below E; scale exponent k_p = max(E - 6 - prime_p, -126); data
 * q = clamp(round_half_even(x / 2^k_p), -127, 127).  NaN packs to 0, +-Inf to
 * +-127 (max_exp 255).
 *
 *   x        fp32 or bf16 [rows, cols] row-major, 16-byte aligned.
 *   dtype    MXQ_F32 or MXQ_BF16 (type of x).
 *   rows, cols  rows >= 0, cols >= 0 and cols % 16 == 0.
 *   q        int8 [n_blocks, 16], n_blocks = rows*cols/16; 16-byte aligned.
 *   max_exp  uint8 [n_blocks].
 *   prime    uint8 [n_blocks] (the page's [n_blocks, 1]).
 * Buffers must not overlap.  9 bits per element in total.
 */
int mx9_pack(const void *x, int dtype, int64_t rows, int64_t cols, int8_t *q, uint8_t *max_exp,
             uint8_t *prime, cudaStream_t stream);

/*
 * MX9 unpack: y = q * 2^k_p with k_p rebuilt from max_exp and prime as in
 * mx9_pack ([MX9] Summary: the packed form is dequantized back to fp32/bf16;
 * the caller passes the shape back because it is not stored).  The result is
 * exact in fp32 and bf16; a block with max_exp 255 can give +-Inf.
 *
 *   q, max_exp, prime  as produced by mx9_pack (q 16-byte aligned).
 *   y        fp32 or bf16 [rows, cols] row-major output, 16-byte aligned.
 *   dtype    MXQ_F32 or MXQ_BF16 (type of y).
 */
int mx9_unpack(const int8_t *q, const uint8_t *max_exp, const uint8_t *prime, void *y, int dtype,
               int64_t rows, int64_t cols, cudaStream_t stream);

/*
 * MX9 and MX6 in one packed uint8 tensor ([MX9] commits: MX9 packed into one
 * uint8 tensor with MX6 and MX9 sent to the packed kernels, and strided inputs
 * accepted; the suite's axis, non-contiguous and padding tests).  One record per 16-element block, [exponent byte, prime
 * byte, data] (the review excerpt stores the exponent at the record start):
 *   MXQ_FMT_MX9: data = 16 int8 q as in mx9_pack; 18-byte records, 9 bits/elem.
 *   MXQ_FMT_MX6: the same rule with 4 magnitude bits, k = max(E - 3 - prime,
 *     -126), q clamped to [-15, 15], stored as sixteen 5-bit two's-complement
 *     codes (element i at bits 5i..5i+4 of the 10 data bytes read as one
 *     little-endian number); 12-byte records, 6 bits/elem.
 * The 2-D tensor has `rows` x `cols` elements, element (r, c) at x[r*ld + c]
 * (ld >= cols, any element-aligned x: strided views are accepted).  Blocks
 * run along `axis`: 1 = along each row, block b = r*ceil(cols/16) + j over
 * columns 16j..16j+15; 0 = down each column, b = c*ceil(rows/16) + j over rows
 * 16j..16j+15 (the tensor with the blocked axis moved last).  A partial last
 * block is zero-padded and then follows the normal rule; unpack writes only
 * the tensor's own elements.  packed: n_blocks * record bytes, 2-byte (MX9) or
 * 4-byte (MX6) aligned.  Any allowed alignment gives the same bytes; 16-byte
 * aligned packed, x and row pitch (ld * element size) select the faster
 * kernels.  Shape and axis are not stored: the caller passes them back to
 * unpack.  Errors: MXQ_EBADDTYPE (dtype or fmt), MXQ_EBADSHAPE (negative
 * sizes, ld < cols, axis not 0/1), MXQ_ENULL, MXQ_EALIGN (x not element-
 * aligned, packed below the sizes above), MXQ_EOVERLAP, MXQ_ECUDA.
 */
#define MXQ_FMT_MX9 9
#define MXQ_FMT_MX6 6
#define MXQ_MX9_RECORD_BYTES 18
#define MXQ_MX6_RECORD_BYTES 12
int mx_pack_packed(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ld, int axis,
                   int fmt, uint8_t *packed, cudaStream_t stream);
int mx_unpack_packed(const uint8_t *packed, int fmt, void *y, int dtype, int64_t rows,
                     int64_t cols, int64_t ld, int axis, cudaStream_t stream);

/*
 * The three-pass composition that the fused cast replaces ([AO] description,
 * first paragraph: a 1x32 cast along N, a 32x1 cast along M and a standalone
 * K-groups swizzle of the colwise scales, reading x twice).  Kept so that the
 * fused kernel can be measured against it and for callers that want one axis.
 *
 * mxq_quantize_1x32: q_row and s_row exactly as mxq_quantize_2d_dual writes
 *   them.  Arguments as there.
 * mxq_quantize_32x1: q_col as mxq_quantize_2d_dual writes it, and the colwise
 *   scales as a plain row-major [N, M/32] matrix s_rm (byte n*(M/32) + i for
 *   the 32x1 block of rows 32i..32i+31 of column n).  Its block rule is the
 *   separate 32x1 cast's ([AO] description, NaN paragraph): the amax skips NaN
 *   (an all-NaN block takes scale 0), +-Inf gives scale 254 and +-448 data,
 *   a NaN element stays a NaN byte.  So it differs from the fused cast only in
 *   blocks that hold NaN.
 * mxq_swizzle_kgroups: s_rm [N, M/32] -> s_col in the fused cast's layout:
 *   per-group blocked slabs, zeros from N*offs[G-1]/32 on (offs/G as for
 *   mxq_quantize_2d_dual; invalid offs are detected on the device, nothing is
 *   written and MXQ_DEV_BADOFFS is set).
 * mxq_quantize_2d_dual_3pass: the three launches in order on `stream`, with
 *   the caller's `workspace` (>= N*M/32 bytes, 16-byte aligned, not
 *   overlapping any other buffer; returns MXQ_EBADSHAPE if too small) holding
 *   s_rm between the second and third.
 * All pointers are device pointers; 16-byte alignment as for the fused cast.
 */
int mxq_quantize_1x32(const void *x, int64_t M, int64_t N, uint8_t *q_row, uint8_t *s_row,
                      cudaStream_t stream);
int mxq_quantize_32x1(const void *x, int64_t M, int64_t N, uint8_t *q_col, uint8_t *s_rm,
                      cudaStream_t stream);
int mxq_swizzle_kgroups(const uint8_t *s_rm, int64_t N, int64_t M, const int32_t *offs, int32_t G,
                        uint8_t *s_col, cudaStream_t stream);
int mxq_quantize_2d_dual_3pass(const void *x, int64_t M, int64_t N, const int32_t *offs, int32_t G,
                               uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                               uint8_t *workspace, int64_t workspace_bytes, cudaStream_t stream);

/*
 * mxq_quantize_2d_dual_3pass without any allocation.  The pages have no
 * counterpart: this is a library convenience.  It is for callers that cannot
 * allocate device memory when they need the cast -- work recorded into a CUDA
 * graph in global capture mode (allocation is illegal there), latency-critical
 * paths where cudaMalloc/cudaFree can synchronize the device, and plugins inside
 * a framework that owns all device memory through an allocator they cannot
 * reach.  The three passes' workspace is a static device array of
 * MXQ_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads the
 * library holds until the process exits; the call makes no cudaMalloc or
 * cudaFree and calls no allocating routine.
 *   Arguments, outputs and errors as mxq_quantize_2d_dual_3pass minus the
 *   workspace; returns MXQ_ESCRATCH, enqueuing nothing, when M*N/32 exceeds
 *   MXQ_NOALLOC_SCRATCH_BYTES (16 MiB: M*N up to 2^29 elements).
 *   The first call on a device looks up the array's device address with that
 *   device current; make that first call before any stream capture.  The
 *   address is looked up again when the current context changes (after a
 *   device reset, say), so the first call in a new context also belongs
 *   before any capture.
 *   All calls share the one array and each overwrites the part it uses before
 *   reading it: calls that may overlap on the GPU (different streams without
 *   ordering between them) race on it and must be serialized by the caller.
 */
#define MXQ_NOALLOC_SCRATCH_BYTES (16u << 20)
int mxq_quantize_2d_dual_3pass_noalloc(const void *x, int64_t M, int64_t N, const int32_t *offs,
                                       int32_t G, uint8_t *q_row, uint8_t *s_row, uint8_t *q_col,
                                       uint8_t *s_col, cudaStream_t stream);

/*
 * Block-scaled MXFP8 matrix product on the tensor cores, reading E4M3 rows and
 * E8M0 scale matrices exactly as mxq_quantize_2d_dual stores them: the consumer
 * check of the layouts ([AO] description, first paragraph: the scales are
 * written in the blocked form the block-scaled MMA reads; "Uncovered tail"
 * paragraph: one slab per K-group).  tcgen05.mma of kind mxf8f6f4 with one
 * E8M0 scale per 32 K elements; a checking tool, not a tuned GEMM (one CTA per
 * 128x128 output tile, no overlap of loads and MMAs).
 *   D[i, j] = sum_k A(i, k) * 2^(sa(i, k/32) - 127) * B(j, k) * 2^(sb(j, k/32) - 127)
 *   a      E4M3 [Ma, K], row i at a + i*lda (K contiguous bytes); e.g. q_row
 *          (lda = N), or a K-group's columns of q_col (a = q_col + lo, lda = M).
 *   sa     E8M0 [Ma, K/32] in the 128x4 blocked layout (s_row, or the group's
 *          s_col slab at s_col + N*lo/32).
 *   b, ldb, sb   likewise for B [Nb, K].
 *   d      fp32 [Ma, Nb] row-major.
 *   Ma, Nb, K    multiples of 128, at most 2^24 (Ma == 0 or Nb == 0: no-op;
 *          K == 0 with Ma, Nb > 0: MXQ_EBADSHAPE); lda, ldb >= K, multiples of 16
 *          and at most 2^40; every pointer 16-byte aligned; d must not overlap an
 *          input.
 * Every internal wait is bounded (MXQ_DEV_TIMEOUT in the status word).
 */
int mxq_mxfp8_scaled_mm(const uint8_t *a, int64_t lda, const uint8_t *sa, const uint8_t *b,
                        int64_t ldb, const uint8_t *sb, float *d, int64_t Ma, int64_t Nb, int64_t K,
                        cudaStream_t stream);

/* ======================================================================== *
 * Operators of a mixture-of-experts training step around the cast.
 *
 * Types are MXQ_F32 or MXQ_BF16; sums, softmax statistics and norms are fp32
 * and every result is rounded once.  Matrices are row-major with `ld`
 * elements between their rows (ld >= the row's length, at most 2^31 - 1);
 * pointers need the alignment of their elements only, and accesses widen to 16
 * bytes where every pitch and address allows it.  `workspace` is device memory
 * (16-byte aligned) that a call uses and leaves: at least the bytes that the
 * matching _workspace() call returns (a host computation; negative: MXQ_E*;
 * 0: none, the pointer may be NULL).
 * A too small one is refused with MXQ_EBADSHAPE.  Results have the same bits in
 * every run: no sum depends on the order in which blocks run.
 * ======================================================================== */

/*
 * Routing of `tokens` tokens to k of `experts` experts, with the balance loss.
 *   logits   [tokens, experts], rows ld elements apart.
 *   k        1 .. min(experts, 32); experts 1 .. MXQ_MAX_GROUPS.
 *   mask     uint8 [tokens], 0 leaves the token out, or NULL.
 *   ids      int32 [tokens, k]: the experts with the k largest logits, largest
 *            first, ties to the lowest index.  A logit of -inf (or NaN) is never
 *            chosen: where fewer than k are left the rest of the row is -1.
 *   weights  fp32 [tokens, k]: p = softmax(logits) at the ids (renorm 0), or p
 *            over the sum of the chosen (renorm 1); 0 beside an id of -1.
 *   counts   int32 [experts]: tokens that chose each expert.
 *   loss     fp32: E/(k n^2) * sum_e counts_e * sum_t p_te over the n = *routed
 *            tokens that are not masked and have a logit other than -inf; 0 for
 *            n == 0.  Tokens that are not counted have ids -1 and weights 0.
 * A row with NaN or +inf has NaN probabilities (and makes the loss NaN).
 *
 * mxq_moe_route_backward: the logits' gradient from those of the weights and of
 * the loss (each may be NULL: zero), with the choice held fixed; rows of tokens
 * that are not counted are written as 0.  ids, counts and routed are the
 * forward call's.  dlogits has the logits' type, rows ldd elements apart.
 */
int64_t mxq_moe_route_workspace(int64_t tokens, int32_t experts);
int mxq_moe_route(const void *logits, int dtype, int64_t tokens, int32_t experts, int64_t ld,
                  int32_t k, const uint8_t *mask, int renorm, float *weights, int32_t *ids,
                  int32_t *counts, float *loss, int32_t *routed, uint8_t *workspace,
                  int64_t workspace_bytes, cudaStream_t stream);
int mxq_moe_route_backward(const void *logits, int dtype, int64_t tokens, int32_t experts,
                           int64_t ld, int32_t k, const uint8_t *mask, int renorm,
                           const int32_t *ids, const int32_t *counts, const int32_t *routed,
                           const float *dweights, const float *dloss, void *dlogits, int64_t ldd,
                           cudaStream_t stream);

/*
 * Routing by scores with a bias, among the best groups of experts.  As mxq_moe_route but
 * for these:
 *   scores   s = 1 / (1 + e^-logit) (MXQ_SCORES_SIGMOID) or softmax(logits)
 *            (MXQ_SCORES_SOFTMAX).
 *   bias     fp32 [experts] or NULL: experts are chosen by s + bias, and their weights
 *            are of s alone.  An expert whose s + bias is -inf or NaN is never chosen.
 *   groups, best   the experts lie in `groups` (1 .. 32, a divisor of experts) equal
 *            groups of consecutive ones; a group's value is the sum of its two largest
 *            s + bias (of one where there is one), and the k experts are chosen among those
 *            of the `best` groups with the largest values, ties to the lowest index.
 *            k at most experts / groups * best.
 *   ids      int32 [tokens, k]: the chosen experts, largest s + bias first, ties to the
 *            lowest index.  The choice is that of 64-bit sums: near ties are computed so.
 *   weights  fp32 [tokens, k]: scale * s at the ids (renorm 0), or scale * s over the sum
 *            of the chosen s (renorm 1; 0 where that sum is 0).  An s below 2^-126 is 0.
 *   loss     as there, with p = s / sum_e s_e (0 where that sum is 0).
 * workspace: of mxq_moe_route_workspace.
 *
 * mxq_moe_route_groups_backward: the logits' gradient, the choice held fixed.  The bias
 * has none: it moves by the counts.
 */
#define MXQ_SCORES_SIGMOID 0
#define MXQ_SCORES_SOFTMAX 1
int mxq_moe_route_groups(const void *logits, int dtype, int64_t tokens, int32_t experts, int64_t ld,
                         int32_t k, const float *bias, int scores, int32_t groups, int32_t best,
                         const uint8_t *mask, int renorm, float scale, float *weights, int32_t *ids,
                         int32_t *counts, float *loss, int32_t *routed, uint8_t *workspace,
                         int64_t workspace_bytes, cudaStream_t stream);
int mxq_moe_route_groups_backward(const void *logits, int dtype, int64_t tokens, int32_t experts,
                                  int64_t ld, int32_t k, int scores, const uint8_t *mask,
                                  int renorm, float scale, const int32_t *ids, const int32_t *counts,
                                  const int32_t *routed, const float *dweights, const float *dloss,
                                  void *dlogits, int64_t ldd, cudaStream_t stream);

/*
 * The exchange of rows between tokens and expert groups.  Assignment
 * i = token*k + j takes row slots[i] of a matrix of M rows in which the groups
 * follow one another, each in token order and filled up to a multiple of 128
 * rows: the matrix and the offs that mxq_quantize_2d_dual takes.
 *   mxq_moe_rows       the rows that hold every routing of these sizes, a
 *                      multiple of 128 (a host computation; negative: MXQ_E*).
 *   mxq_moe_plan       from ids int32 [tokens, k] (-1: not routed; an id outside
 *                      [0, experts) also sets MXQ_DEV_BADINDEX): offs int32
 *                      [experts] (cumulative ends), slots int32 [tokens, k] (-1:
 *                      none), source int32 [M] (the assignment of each row, or -1).
 *                      M >= mxq_moe_rows(), a multiple of 128.
 *   mxq_moe_dispatch   rows[slots[i]] = x[i / k]; rows without an assignment 0.
 *   mxq_moe_combine    y[t] = sum_j w[t, j] * rows[slots[t, j]], j ascending; w =
 *                      1 for weights NULL, which is the gradient of dispatch.
 *   mxq_moe_combine_backward   drows[slots[i]] = w_i * dy[i / k], other rows 0;
 *                      dweights[i] = <dy[i / k], rows[slots[i]]>, 0 without a slot.
 * x, y, dy are [tokens, D], rows and drows [M, D], all of one type; weights and
 * dweights fp32 [tokens, k].  A slot outside [0, M) is left out and sets
 * MXQ_DEV_BADINDEX.
 */
int64_t mxq_moe_rows(int64_t tokens, int32_t k, int32_t experts);
int64_t mxq_moe_plan_workspace(int64_t tokens, int32_t k, int32_t experts);
int mxq_moe_plan(const int32_t *ids, int64_t tokens, int32_t k, int32_t experts, int64_t M,
                 int32_t *offs, int32_t *slots, int32_t *source, uint8_t *workspace,
                 int64_t workspace_bytes, cudaStream_t stream);
int mxq_moe_dispatch(const void *x, int dtype, int64_t tokens, int64_t D, int64_t ldx, int32_t k,
                     const int32_t *slots, const int32_t *source, int64_t M, void *rows,
                     int64_t ldr, cudaStream_t stream);
int mxq_moe_combine(const void *rows, int dtype, int64_t M, int64_t D, int64_t ldr, int64_t tokens,
                    int32_t k, const int32_t *slots, const float *weights, void *y, int64_t ldy,
                    cudaStream_t stream);
int mxq_moe_combine_backward(const void *dy, int dtype, int64_t tokens, int64_t D, int64_t ldy,
                             const void *rows, int64_t ldr, int64_t M, int32_t k,
                             const int32_t *slots, const int32_t *source, const float *weights,
                             void *drows, int64_t ldd, float *dweights, cudaStream_t stream);

/*
 * The experts' products on the cast's bytes, block-scaled MXFP8 on the tensor cores
 * (tcgen05), and the gradients around them.  Rows lie in groups that end at offs
 * (int32 [G] on the device, as for mxq_quantize_2d_dual; NULL and G 0: one group of
 * all M rows, and one matrix of everything below that has G); M, N and K are
 * multiples of 128, at most 2^24.
 *   mxq_moe_linear   z[m, n] = sum_k x[m, k] w[e, n, k] + bias[e, n],
 *                    y = act(z) + residual, e the group of row m; rows behind the
 *                    last group are written as 0 in y and z.
 *     x, sx     E4M3 [M, K], rows ldx bytes apart, and its blocked E8M0 scales
 *               [M*K/32]: q_row and s_row of the cast.
 *     w, sw     E4M3 [G, N, K], rows ldw and matrices stride_w bytes apart, and the
 *               matrices' blocked scales one after another [G*N*K/32]: of one cast of
 *               [G*N, K] q_row and s_row; for the rows' gradient (x = the cast dz
 *               [M, N], K the weights' N) its q_col, with ldw = G*N and stride_w = N,
 *               and the s_col of a cast with offs N, 2N, ..., G*N.  Pitches are
 *               multiples of 16.
 *     bias      [G, N] of type bias_dtype, or NULL.
 *     activation  MXQ_ACT_NONE, _RELU, _SILU (z / (1 + e^-z)) or _GELU (the tanh form,
 *               0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))).
 *     residual  [M, N] of the output's type, rows ldr apart, or NULL; may be y itself.
 *     y, z      [M, N] of type dtype, each rounded once from fp32; z may be NULL.
 *   mxq_moe_weight_gradient   dw[e, n, k] = sum over the rows m of group e of
 *               a[n, m] b[k, m], added to what dw holds with `accumulate` (in fp32; the
 *               addition to an fp32 dw takes subnormal numbers for 0); a group without
 *               rows gives 0 (or leaves dw).
 *     a, sa     q_col [N, M] and s_col [N*M/32] of the cast dz; b, sb of the cast x.
 *     dw        [G, N, K] of type dtype, rows ldd and matrices stride_d apart.
 *   mxq_moe_linear_backward   dz = dy act'(z) (rows behind the last group: 0) and
 *               dbias[e, n] = the sum of dz (in fp32, before its rounding) over the
 *               rows of group e.  dy, z, dz [M, N] of type dtype; dz may be dy itself;
 *               dz or dbias (fp32 [G, N]) may be NULL, z with MXQ_ACT_NONE.
 * Sums are fp32.  Scale byte 255 is NaN.  Invalid offs are detected on the device:
 * nothing is written and MXQ_DEV_BADOFFS is set.  Every internal wait is bounded
 * (MXQ_DEV_TIMEOUT in the status word).
 */
#define MXQ_ACT_NONE 0
#define MXQ_ACT_RELU 1
#define MXQ_ACT_SILU 2
#define MXQ_ACT_GELU 3
int mxq_moe_linear(const uint8_t *x, int64_t ldx, const uint8_t *sx, const uint8_t *w, int64_t ldw,
                   int64_t stride_w, const uint8_t *sw, const int32_t *offs, int32_t G, int64_t M,
                   int64_t N, int64_t K, const void *bias, int bias_dtype, int activation,
                   const void *residual, int64_t ldr, int dtype, void *y, int64_t ldy, void *z,
                   int64_t ldz, cudaStream_t stream);
int mxq_moe_weight_gradient(const uint8_t *a, int64_t lda, const uint8_t *sa, const uint8_t *b,
                            int64_t ldb, const uint8_t *sb, const int32_t *offs, int32_t G,
                            int64_t M, int64_t N, int64_t K, int accumulate, int dtype, void *dw,
                            int64_t ldd, int64_t stride_d, cudaStream_t stream);
int64_t mxq_moe_linear_backward_workspace(int64_t M, int64_t N);
int mxq_moe_linear_backward(const void *dy, int dtype, int64_t ld_dy, const void *z, int64_t ldz,
                            int activation, const int32_t *offs, int32_t G, int64_t M, int64_t N,
                            void *dz, int64_t ld_dz, float *dbias, uint8_t *workspace,
                            int64_t workspace_bytes, cudaStream_t stream);

/*
 * Scaled lookup in a table [rows, D], and the table's gradient.
 *   ids      int32 or int64 (ids_bytes 4 or 8, else MXQ_EBADDTYPE) [tokens].  An id
 *            outside [0, rows) gives a row of zeros, adds to no gradient and sets
 *            MXQ_DEV_BADINDEX.
 *   mxq_embedding            y[t] = scale * table[ids[t]], types dtype -> out_dtype.
 *   mxq_embedding_backward   dtable[v] = scale * sum of dy[t] over ids[t] == v, in
 *            a fixed order; every row is written, 0 where no token has it.  Tokens
 *            whose id is `padding` are left out (-1: none).  dy has type dtype,
 *            dtable out_dtype.
 * tokens at most 2^29 - 1.
 */
int mxq_embedding(const void *ids, int ids_bytes, int64_t tokens, const void *table, int dtype,
                  int64_t rows, int64_t D, int64_t ldw, float scale, void *y, int out_dtype,
                  int64_t ldy, cudaStream_t stream);
int64_t mxq_embedding_backward_workspace(int64_t tokens, int64_t rows, int64_t D);
int mxq_embedding_backward(const void *ids, int ids_bytes, int64_t tokens, const void *dy,
                           int dtype, int64_t D, int64_t ldd, int64_t rows, int64_t padding,
                           float scale, void *dtable, int out_dtype, int64_t ldw,
                           uint8_t *workspace, int64_t workspace_bytes, cudaStream_t stream);

/*
 * An AdamW step over many tensors in one launch, in place:
 *   g = grad * grad_scale;  m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2;
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 *   tensors   host array of `count` (at most MXQ_ADAMW_TENSORS) entries, read during the
 *             call: n contiguous elements p of type dtype, their gradient of type
 *             grad_dtype, a bf16 copy that the new values are also rounded to (or NULL),
 *             and `start`, the place of its moments in m and v, a multiple of 128.
 *             Nothing is done for n == 0.  A bf16 p is rounded to nearest.
 *   bits      32: m and v fp32 [total].  8: m and the root of v as E4M3 [total] with E8M0
 *             scales m_scale and v_scale [total/32], one for 32 elements by the cast's
 *             rule; rounded at random from (seed, t, place), m and the root with their
 *             exact value as mean (v, the square, gains the roundings' variance, some
 *             percent), a root that is not 0 never to 0 (elements below 2^-17 of the
 *             largest of their 32 take smaller steps); a block with a value that is not
 *             finite becomes NaN.  All bytes of a tensor's last 32 are written, 0 behind its
 *             end.  total is a multiple of 128; m and v 16-byte aligned.
 *   t         *step_at (device memory) or, with step_at NULL, step; at least 1.
 *   lr        *lr_at (device memory) or, with lr_at NULL, lr.
 *   grad_scale  device memory, or NULL: 1.
 *   beta1, beta2 in [0, 1), eps >= 0.
 * No two outputs may overlap, nor an output and an input.
 *
 * mxq_adamw_check: the checks of a longer list (at most 2^24 entries), which takes several
 * calls, before the first of them: types, sizes, places and overlaps among all of its
 * buffers.  It launches nothing and needs no device.
 */
#define MXQ_ADAMW_TENSORS 512
typedef struct mxq_adamw_tensor {
  void *p;
  const void *grad;
  void *copy;
  int64_t n, start;
  int32_t dtype, grad_dtype;
} mxq_adamw_tensor;
int mxq_adamw(const mxq_adamw_tensor *tensors, int32_t count, int32_t bits, void *m, void *v,
              uint8_t *m_scale, uint8_t *v_scale, int64_t total, int64_t step,
              const int64_t *step_at, double lr, const float *lr_at, double beta1, double beta2,
              double eps, double weight_decay, const float *grad_scale, uint64_t seed,
              cudaStream_t stream);
int mxq_adamw_check(const mxq_adamw_tensor *tensors, int64_t count, int32_t bits, const void *m,
                    const void *v, const uint8_t *m_scale, const uint8_t *v_scale, int64_t total,
                    const int64_t *step_at, const float *lr_at, const float *grad_scale);

/*
 * Newton-Schulz orthogonalisation of a momentum matrix, or of a stack of them:
 *   X = g / (|g|_F + eps);  `steps` times  X <- (aI + bA + cA^2) X, A = X X^T
 *   (X (aI + bA + cA^2), A = X^T X, for m > n: the same matrix);  out = scale * X.
 *   g        [batch, m, n], rows ld and matrices `stride` elements apart.
 *   out      bf16 [batch, m, n], rows ldo and matrices stride_o elements apart.
 *   steps    1 .. 64; a, b, c finite; eps >= 0.  m, n at most 2^20, batch at
 *            most 65535.
 * The products take fp16 operands and accumulate in fp32 (tcgen05): an error of
 * about 1e-3 (Frobenius, of the result's norm) for five steps of the usual
 * coefficients, beside the 1.7e-3 of the rounding to bf16; sides up to 64 carry
 * pairs of fp16 and are exact to the rounding.  The norm is right for any finite g (its
 * squares are summed in three ranges of fp32), and X has the same relative error where
 * |g| is far below eps; a matrix of zeros gives 0, or NaN with eps == 0.  The iterates are taken to stay within |X| <= 1.5 in the spectral norm,
 * as they do for the usual coefficients (3.4445, -4.775, 2.0315); beyond eight
 * times that fp16 overflows.  Directions in which g is zero, or below 2^-12 of
 * its norm, carry rounding noise that the iteration magnifies up to a^steps.
 * Every internal wait is bounded (MXQ_DEV_TIMEOUT in the status word).
 */
int64_t mxq_orthogonalize_workspace(int64_t batch, int64_t m, int64_t n);
int mxq_orthogonalize(const void *g, int dtype, int64_t batch, int64_t m, int64_t n, int64_t ld,
                      int64_t stride, int32_t steps, float a, float b, float c, float eps,
                      float scale, void *out, int64_t ldo, int64_t stride_o, uint8_t *workspace,
                      int64_t workspace_bytes, cudaStream_t stream);

/*
 * Device status word of the current device: a sticky OR of MXQ_DEV_* bits set
 * by kernels since the last clear.  Writes it to *out and clears it when
 * `clear` is non-zero.  This call synchronizes the device (it reads device
 * memory); use it for diagnostics and tests, not inside captured work.
 * Returns MXQ_OK, MXQ_ENULL or MXQ_ECUDA.
 * mxq_last_device_status is the same call under the boundary's other name: the
 * word lives in device memory and is read by a copy (hence the synchronization)
 * instead of in a library-owned pinned host flag, so that no compute call
 * needs an allocation.
 */
int mxq_device_status(uint32_t *out, int clear);
int mxq_last_device_status(uint32_t *out, int clear);

/*
 * Self-test of failure detection, on the GPU and without a fault: launches one
 * warp that waits, with the same bounded wait the pipelines use, on an
 * mbarrier nothing ever completes.  The wait gives up after `limit_ns`
 * nanoseconds (1e6 .. 4e9, else MXQ_EBADSHAPE), the kernel records
 * MXQ_DEV_TIMEOUT in the device status word and returns, and the context stays
 * usable.  The production kernels use a 4 s limit per wait.
 */
int mxq_selftest_wait_timeout(uint64_t limit_ns, cudaStream_t stream);

/*
 * Checked builds.  A library compiled with MXQ_DEBUG_BOUNDS=1 (the
 * package's build step makes it as libmxq_checked.so beside libmxq.so)
 * tests the byte range of every global store its kernels make outside the
 * TMA tensor stores (whose bounds the tensor maps enforce) against the
 * output buffer it belongs to; a range that would leave the buffer is not
 * written and MXQ_DEV_OOB is set in the device status word.  Results are
 * otherwise identical.  mxq_debug_bounds() returns 1 in a checked build and
 * 0 in a release build.  mxq_selftest_bounds() launches one thread that
 * tests a range lying past a 64-byte dummy buffer, without any access: a
 * checked build records MXQ_DEV_OOB, a release build records nothing.
 * Returns MXQ_OK or MXQ_ECUDA.
 * mxq_selftest_watch() makes a checked build count every access of the
 * training operators' kernels that touches `address` (device memory; NULL: no
 * address) as one outside its buffer, which is left out and recorded, so that
 * a test can see that an access is checked; a release build takes the call and
 * does nothing.  It waits for the device.
 */
int mxq_debug_bounds(void);
int mxq_selftest_bounds(cudaStream_t stream);
int mxq_selftest_watch(const void *address);

/* Static description of a status code (never NULL). */
const char *mxq_status_string(int status);

/* Library ABI version, (major << 16) | minor. */
int mxq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_H_ */
