/*
 * mxfp8_partial.h -- C ABI of the GB300 partial MXFP8 cast of master weights.
 *
 * The operation is the distributed master-weight writeback described on the page
 * "Support row-only MXFP8 distributed master-weight casts" (TransformerEngine
 * pull request 3488), sections "Changes" and the flow diagram: each rank holds a
 * contiguous fragment of a flattened rows x cols FP32 (or BF16) master weight;
 *   1. partial amax   -- 1x32 row-block and 32x1 column-block maxima of |x| over
 *                        the fragment, for the directions the weight has;
 *   2. packed MAX reduce of those amaxes over all ranks (here: over shard slots
 *                        of one device buffer);
 *   3. scale update   -- E8M0 block scales from the reduced amaxes;
 *   4. partial cast   -- master -> BF16 (nearest-even) -> E4M3 (nearest-even,
 *                        saturating at 448), written in place into the rowwise and,
 *                        when present, columnwise outputs.
 * Scale convention (the pages print none): scale exponent
 * e = floor(log2(amax)) - 8, clamped to [-127, 127], amax 0 -> -127; the stored
 * E8M0 byte is e + 127 (0xFF for a NaN/infinite amax).  Data byte =
 * E4M3(bf16(x) * 2^-e).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every pointer inside an mxfp8_tensor is a DEVICE pointer (global memory of
 *   the current CUDA device), or page-locked host memory that the device can
 *   address directly (see mxfp8_device_can_access).  The caller owns all memory;
 *   the library never allocates, frees or keeps a pointer after the call returns.
 * - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL = the
 *   legacy default stream).  A return of 0 means "validated and launched".
 *   Kernels are launched as programmatic dependents of the kernel before them in
 *   the stream: they may be scheduled while that kernel's last blocks run, but
 *   read and write nothing until it has completed, so stream order holds.
 * - Tensors are dense and row-major: a 2-D tensor's row stride is shape[1].
 * - An EMPTY handle (data == NULL, or any shape entry == 0, or a NULL handle
 *   pointer) means "this direction is absent" (section "Changes": omission uses
 *   empty tensor handles, not a magic shape).
 * - Return status: 0 ok; 1 invalid argument; 2 shape/padding mismatch;
 *   3 dtype mismatch; 4 missing required tensor; 6 CUDA launch error.
 *   (5, non-contiguous, is raised by language bindings that can see strides.)
 *   mxfp8_last_error() gives a message for the calling thread's last failure.
 * - Thread safety: entry points may be called concurrently from several host
 *   threads; results written by two launches to the same buffer race.
 */
#ifndef MXFP8_PARTIAL_H_
#define MXFP8_PARTIAL_H_

#include <stdint.h>

/* Every entry point below is exported; everything else in the library is hidden. */
#if defined(__GNUC__)
#define MXFP8_API __attribute__((visibility("default")))
#else
#define MXFP8_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MXFP8_DTYPE_F32 = 0,  /* float                              */
  MXFP8_DTYPE_BF16 = 1, /* bfloat16 (16-bit patterns)         */
  MXFP8_DTYPE_U8 = 2    /* uint8: E8M0 scales and E4M3 data   */
} mxfp8_dtype;

typedef struct {
  void* data;       /* device pointer, element-aligned; NULL => empty      */
  int32_t dtype;    /* mxfp8_dtype                                         */
  int32_t ndim;     /* 1 or 2                                              */
  int64_t shape[2]; /* shape[1] ignored when ndim == 1                     */
} mxfp8_tensor;

/* Size limits of every entry point taking rows x cols: 1 <= cols <= 2^37 and
 * rows * cols <= 2^40 elements; outside them the call returns MXFP8_ERR_INVALID. */
enum {
  MXFP8_OK = 0,
  MXFP8_ERR_INVALID = 1,
  MXFP8_ERR_SHAPE = 2,
  MXFP8_ERR_DTYPE = 3,
  MXFP8_ERR_MISSING = 4,
  MXFP8_ERR_NONCONTIGUOUS = 5,
  MXFP8_ERR_CUDA = 6
};

/*
 * Partial amax (page "Support row-only MXFP8 distributed master-weight casts",
 * review thread: documentation of the partial amax entry point).
 *
 * input         [in]     fragment: numel(input) = len contiguous F32 or BF16
 *                        values, element k of the fragment is element
 *                        start_offset + k of the flattened rows x cols weight.
 * amax_rowwise  [in,out] REQUIRED, 2-D [>= rows][>= ceil(cols/32)], dtype of the
 *                        input.  Entry (i, b) = max |x| over the fragment's
 *                        elements of row i, columns [32b, 32b+32).
 * amax_colwise  [in,out] OPTIONAL (empty => the columnwise direction is skipped
 *                        entirely, at compile time in the kernel), 2-D
 *                        [>= ceil(rows/32)][>= cols], dtype of the input.
 *                        Entry (c, j) = max |x| over the fragment's elements of
 *                        column j, rows [32c, 32c+32).
 * Only entries of blocks that contain at least one fragment element are written
 * (overwritten, not max-accumulated); every other entry keeps its value, so a
 * caller that reduces across fragments zeroes its buffers first.  An empty
 * fragment (len 0) writes nothing and returns 0.  NaN members make the entry NaN,
 * stored as the canonical quiet NaN (F32 0x7FC00000, BF16 0x7FC0) whatever their
 * NaN patterns.
 * Errors: 1 if start_offset < 0, rows/cols out of the size limits, start_offset + len > rows*cols,
 * or a pointer is not element-aligned; 2 on a too-small amax shape;
 * 3 if an amax dtype differs from the input dtype or the input is not F32/BF16;
 * 4 if amax_rowwise is empty (and len > 0).
 */
MXFP8_API int mxfp8_partial_amax(const mxfp8_tensor* input, mxfp8_tensor* amax_rowwise,
                       mxfp8_tensor* amax_colwise, int64_t rows, int64_t cols,
                       int64_t start_offset, void* stream);

/*
 * Packed MAX reduction (page "Support row-only MXFP8 distributed master-weight
 * casts", section "Changes": one packed-amax MAX all-reduce; here the ranks are
 * emulated as slots of one device buffer).
 *
 * slots  [in]  2-D [S][E] F32 or BF16: S packed amax buffers of E entries each.
 * out    [out] E entries (any shape with numel == E), same dtype.
 * out[k] = max over s of |slots[s][k]|; NaN propagates as the canonical quiet NaN
 * (F32 0x7FC00000, BF16 0x7FC0).  S == 1 copies |.|.
 * out may not overlap slots.  Errors: 2 numel mismatch, 3 dtype, 4 empty out.
 */
MXFP8_API int mxfp8_amax_max_reduce(const mxfp8_tensor* slots, mxfp8_tensor* out, void* stream);

/*
 * Scale update (page "Support row-only MXFP8 distributed master-weight casts",
 * flow diagram: "update scales for present directions").
 *
 * amax_rowwise      [in]  REQUIRED, [>= rows][>= ceil(cols/32)], F32 or BF16.
 * amax_colwise      [in]  OPTIONAL, [>= ceil(rows/32)][>= cols], same dtype;
 *                         empty => no columnwise scales are computed.
 * scale_inv_rowwise [out] REQUIRED, U8 [>= rows][>= ceil(cols/32)].
 * scale_inv_colwise [out] U8 [>= ceil(rows/32)][>= cols]; required iff
 *                         amax_colwise is present, ignored otherwise.
 * Writes the E8M0 byte of every entry of the compact block grid
 * (rows x ceil(cols/32) and ceil(rows/32) x cols); padding is left untouched.
 */
MXFP8_API int mxfp8_update_scales(const mxfp8_tensor* amax_rowwise, const mxfp8_tensor* amax_colwise,
                        mxfp8_tensor* scale_inv_rowwise, mxfp8_tensor* scale_inv_colwise,
                        int64_t rows, int64_t cols, void* stream);

/*
 * Partial cast (page "Support row-only MXFP8 distributed master-weight casts",
 * sections "Changes" and the review thread's documentation of the partial cast:
 * rowwise outputs are required; columnwise scales are required when the
 * columnwise output is present and ignored when it is omitted).
 *
 * input             [in]  fragment as for mxfp8_partial_amax.
 * scale_inv_rowwise [in]  REQUIRED U8 [>= rows][>= ceil(cols/32)] E8M0 bytes.
 * scale_inv_colwise [in]  U8 [>= ceil(rows/32)][>= cols]; required iff
 *                         output_colwise is present, ignored otherwise.
 * output_rowwise    [out] REQUIRED U8, numel >= out_offset + len.
 * output_colwise    [out] OPTIONAL U8 (empty => no columnwise reads or writes),
 *                         numel >= out_offset + len.
 * For fragment element k (weight element (i, j)): y = BF16 rounding of x
 * (identity for BF16 input); output_rowwise[out_offset + k] = E4M3(y * 2^-e_r),
 * e_r from scale_inv_rowwise[i][j/32]; output_colwise likewise with
 * scale_inv_colwise[i/32][j].  Outputs hold E4M3 bytes in the weight's own
 * row-major layout (the columnwise copy is not transposed).  out_offset =
 * start_offset writes into a full-size rows*cols output in place; out_offset = 0
 * writes a fragment-sized output.  Bytes outside the fragment are not touched.
 * Errors: 1 bad offsets/sizes; 2 output or scale too small; 3 dtype;
 * 4 rowwise scale/output missing, or columnwise output without columnwise scales.
 */
MXFP8_API int mxfp8_partial_cast(const mxfp8_tensor* input, const mxfp8_tensor* scale_inv_rowwise,
                       const mxfp8_tensor* scale_inv_colwise, mxfp8_tensor* output_rowwise,
                       mxfp8_tensor* output_colwise, int64_t rows, int64_t cols,
                       int64_t start_offset, int64_t out_offset, void* stream);

/*
 * Batched entry points: many fragments (of one or several weights) per call, e.g. all
 * fragments a rank holds for a batch of weights (page "Support row-only MXFP8
 * distributed master-weight casts", section "Changes": mixed row-only and
 * bidirectional batches).  Each job means exactly what the single-fragment call with
 * the same arguments means; the jobs are validated first (a failure launches nothing
 * and names the job), then run as few kernels as possible: jobs that share the input
 * dtype, the model dtype and (cast) whether the outputs allow word stores go into one
 * launch (at most 64 jobs each; row-only and bidirectional jobs, and fragments whose
 * virtual base is or is not 16-byte aligned, together, each tile taking its job's
 * specialisation), with the tiles of all jobs scheduled together.  Jobs may run concurrently:
 * jobs whose written entries overlap (two fragments of one weight writing the SAME
 * amax buffer, whose boundary blocks both jobs overwrite) race -- give each fragment
 * its own amax buffer, as a packed per-rank slot does.  Fragments of one weight write
 * disjoint output bytes and may share the outputs.  F32 and BF16 jobs may be mixed
 * in one call.  njobs may be 0; jobs with empty fragments are skipped.
 */
typedef struct {
  mxfp8_tensor input;
  mxfp8_tensor amax_rowwise;
  mxfp8_tensor amax_colwise; /* empty => row-only */
  int64_t rows, cols, start_offset;
} mxfp8_amax_job;

/* Model dtype the master values are rounded through before quantisation ("rounding
 * through the model dtype", section "Changes").  The single-fragment entry points
 * use BF16; jobs carry the choice (a zero-initialised job means BF16). */
enum { MXFP8_MODEL_BF16 = 0, MXFP8_MODEL_F16 = 1 };

typedef struct {
  mxfp8_tensor input;
  mxfp8_tensor scale_inv_rowwise;
  mxfp8_tensor scale_inv_colwise;
  mxfp8_tensor output_rowwise;
  mxfp8_tensor output_colwise; /* empty => row-only */
  int64_t rows, cols, start_offset, out_offset;
  int32_t model_dtype;         /* MXFP8_MODEL_BF16 (0) or MXFP8_MODEL_F16 */
} mxfp8_cast_job;

typedef struct {
  mxfp8_tensor amax_rowwise;
  mxfp8_tensor amax_colwise; /* empty => row-only */
  mxfp8_tensor scale_inv_rowwise;
  mxfp8_tensor scale_inv_colwise;
  int64_t rows, cols;
} mxfp8_scale_job;

MXFP8_API int mxfp8_partial_amax_batched(const mxfp8_amax_job* jobs, int32_t njobs, void* stream);
MXFP8_API int mxfp8_update_scales_batched(const mxfp8_scale_job* jobs, int32_t njobs, void* stream);

/*
 * Packed MAX reduction fused with the scale update (the reduction of
 * mxfp8_amax_max_reduce and the scale update of mxfp8_update_scales_batched in one
 * pass over the packed buffer, for the slots of ranks emulated on one GPU).
 *
 * slots   [in]  2-D [S][P] F32 or BF16 packed amax buffers.
 * reduced [out] P entries, same dtype.
 * jobs    [in]  njobs scale jobs (see mxfp8_scale_job) whose amax grids are views
 *               INTO `reduced`; entry (r, c) of such a view at reduced offset o is
 *               reduced[o] = max_s |slots[s][o]|, and its E8M0 byte goes to the job's
 *               scale grid.  Entries of `reduced` outside every view are not written.
 * Results equal mxfp8_amax_max_reduce followed by mxfp8_update_scales_batched.
 * Errors: as those two; 1 if a view does not lie inside `reduced`.
 */
MXFP8_API int mxfp8_amax_max_reduce_update_scales(const mxfp8_tensor* slots, mxfp8_tensor* reduced,
                                        const mxfp8_scale_job* jobs, int32_t njobs,
                                        void* stream);

/*
 * The same reduction when each slot holds amaxes only where its rank's fragments are.
 * A rank's partial amax writes exactly the entries of the blocks its fragments touch;
 * every other entry of its slot is never written.  Rather than zeroing those entries
 * before every step and reading them back in the reduction, the caller names, per slot,
 * the packed entries it holds, and the reduction reads only those (the emulated MAX
 * all-reduce of section "Changes" then moves only the bytes the ranks produced).
 *
 * slot_ranges [in] nranges triples (slot, begin, end): slot `slot` (< S <= 64) holds
 *                  valid amaxes for packed entries [begin, end) (0 <= begin <= end <= P).
 *                  Entries of a slot outside all of its ranges count as zero and are
 *                  not read (their contents are irrelevant); an entry no slot holds
 *                  reduces to +0.  Ranges of one slot may touch or overlap.
 * nranges == 0 (slot_ranges may be NULL): every slot holds every entry, exactly as
 * mxfp8_amax_max_reduce_update_scales.
 * Other arguments, results and errors as mxfp8_amax_max_reduce_update_scales; 1 also
 * for a malformed range or more than 64 slots with ranges.
 */
MXFP8_API int mxfp8_amax_max_reduce_update_scales_ranged(const mxfp8_tensor* slots,
                                               mxfp8_tensor* reduced,
                                               const mxfp8_scale_job* jobs, int32_t njobs,
                                               const int64_t* slot_ranges, int32_t nranges,
                                               void* stream);

MXFP8_API int mxfp8_partial_cast_batched(const mxfp8_cast_job* jobs, int32_t njobs, void* stream);

/*
 * One-pass quantisation of a fragment made of WHOLE blocks.  When every row block
 * (and, with a columnwise output, every column block) that the fragment touches lies
 * wholly inside it -- a rank that owns whole weights or whole 32-row bands, or a
 * single rank -- no cross-rank MAX reduction is needed (the MAX over one rank is the
 * identity), and amax, scale update and cast of the page "Support row-only MXFP8
 * distributed master-weight casts" (flow diagram) run as ONE kernel that reads the
 * input from HBM once.  Results are bit-identical to mxfp8_partial_amax ->
 * mxfp8_update_scales -> mxfp8_partial_cast on the same fragment.
 *
 * input, output_rowwise, output_colwise, rows, cols, start_offset, out_offset: as for
 *                   mxfp8_partial_cast; the columnwise direction is present iff
 *                   output_colwise is.
 * amax_rowwise / amax_colwise [out] OPTIONAL grids as for mxfp8_partial_amax; when
 *                   given, the block maxima are stored too (a columnwise amax grid is
 *                   ignored without a columnwise output).
 * scale_inv_rowwise [out] REQUIRED; scale_inv_colwise [out] required iff
 *                   output_colwise is present.  Entries of blocks the fragment touches
 *                   are written; others are left untouched.
 * Precondition (status 1 otherwise): start_offset % cols and (start_offset + len) %
 * cols are multiples of 32, and with a columnwise output start_offset and
 * start_offset + len are multiples of 32*cols (the end may also be rows*cols).
 */
MXFP8_API int mxfp8_quantize_whole_blocks(const mxfp8_tensor* input, mxfp8_tensor* amax_rowwise,
                                mxfp8_tensor* amax_colwise, mxfp8_tensor* scale_inv_rowwise,
                                mxfp8_tensor* scale_inv_colwise, mxfp8_tensor* output_rowwise,
                                mxfp8_tensor* output_colwise, int64_t rows, int64_t cols,
                                int64_t start_offset, int64_t out_offset, void* stream);

typedef struct {
  mxfp8_tensor input;
  mxfp8_tensor amax_rowwise;      /* optional */
  mxfp8_tensor amax_colwise;      /* optional */
  mxfp8_tensor scale_inv_rowwise;
  mxfp8_tensor scale_inv_colwise;
  mxfp8_tensor output_rowwise;
  mxfp8_tensor output_colwise;    /* empty => row-only */
  int64_t rows, cols, start_offset, out_offset;
  int32_t model_dtype;            /* MXFP8_MODEL_BF16 (0) or MXFP8_MODEL_F16 */
} mxfp8_quantize_job;

/* Batched form of mxfp8_quantize_whole_blocks, with the conventions of the other
 * batched entry points. */
MXFP8_API int mxfp8_quantize_whole_blocks_batched(const mxfp8_quantize_job* jobs, int32_t njobs,
                                        void* stream);

/*
 * Scale layout for GEMM consumers.  Rearranges a compact E8M0 grid into the layout in
 * which block-scaled tensor-core GEMMs read scale factors: the logical matrix L (the
 * grid when transpose == 0; its transpose when transpose == 1, e.g. a columnwise
 * [ceil(rows/32)][cols] grid consumed as [cols][ceil(rows/32)]) is padded with zero
 * bytes to multiples of 128 rows and 4 columns and cut into 128x4 tiles, stored in
 * row-major tile order, 512 bytes each; inside a tile element (r, c) sits at byte
 * (r % 32) * 16 + (r / 32) * 4 + c.  (An output format next to the path: the pages
 * only require padded scale grids.)
 *
 * scale_inv [in]  U8 2-D [>= nrows][>= ncols] (row stride shape[1]).
 * out       [out] U8, numel >= mxfp8_swizzled_scales_size(nrows, ncols, transpose).
 * Errors: 1 bad sizes or transpose flag, 2 out too small, 3 dtype, 4 missing tensor.
 */
MXFP8_API int mxfp8_swizzle_scales(const mxfp8_tensor* scale_inv, mxfp8_tensor* out, int64_t nrows,
                         int64_t ncols, int32_t transpose, void* stream);

/* Bytes of the GEMM layout of an nrows x ncols grid (transpose as above). */
MXFP8_API int64_t mxfp8_swizzled_scales_size(int64_t nrows, int64_t ncols, int32_t transpose);

/*
 * Host memory.  Every entry point takes device-accessible pointers.  On this platform
 * (unified virtual addressing; Grace-Blackwell's coherent CPU-GPU link) page-locked
 * host memory from cudaHostAlloc / cudaHostRegister is device-accessible through the
 * same pointer, so the kernels can read master weights from, and write E4M3 data to,
 * host memory directly.  mxfp8_device_can_access returns 1 when the current device can
 * dereference [ptr, ptr + bytes) (device, managed, or mapped page-locked host memory)
 * and 0 otherwise (e.g. pageable host memory); language bindings check host buffers
 * with it before passing them.  It enqueues nothing.
 */
MXFP8_API int mxfp8_device_can_access(const void* ptr, int64_t bytes);

/*
 * Sharded update of one weight without any device allocation.  The source pages have
 * no counterpart of this entry point.
 *
 * It is for callers that cannot allocate device memory at the moment they need the
 * update -- a memory-pool allocator running its own maintenance, a framework that has
 * reserved all device memory up front, or code where a cudaMalloc would synchronise
 * the device.  The update needs working memory for one amax slot per fragment and for
 * the reduced amax; here that memory is one file-scope device array of 64 MiB, which
 * every GPU that loads this library holds until the process exits.
 *
 * fragments[f]      [in]  fragment f of the rows x cols weight (F32 or BF16, one dtype
 *                         for all; empty fragments are skipped), starting at flat
 *                         element start_offsets[f].  Fragments must not overlap
 *                         (status 1 when two non-empty fragments do).
 * scale_inv_rowwise [out] REQUIRED U8 [>= rows][>= ceil(cols/32)].
 * scale_inv_colwise [out] U8 [>= ceil(rows/32)][>= cols]; required iff output_colwise.
 * output_rowwise    [out] REQUIRED U8, full size (rows*cols), written where the
 *                         fragments are.
 * output_colwise    [out] OPTIONAL U8 full size; empty => row-only.
 * Results equal mxfp8_partial_amax of every fragment into its own zeroed slot,
 * mxfp8_amax_max_reduce over the slots, mxfp8_update_scales and mxfp8_partial_cast of
 * every fragment (it runs exactly those entry points), with BF16 as the model dtype.
 * Limits: 1..64 fragments and (nfrags + 1) amax slots of rows*ceil(cols/32) (+
 * ceil(rows/32)*cols when columnwise) entries, each rounded up to 256 bytes, within
 * the 64 MiB; a larger request fails with status 2 and a message giving the bytes
 * needed.  Every argument is checked before anything is launched: a non-zero status
 * leaves every caller buffer untouched.  The first call on a device looks up the
 * array's device address (with that device current); make that first call before any
 * stream capture.  Every call uses
 * the same array and leaves its contents behind (slots are cleared at the start of
 * each call); calls that overlap on the GPU -- on different streams or from
 * different threads -- race on it.
 */
MXFP8_API int mxfp8_sharded_update_noalloc(const mxfp8_tensor* fragments, const int64_t* start_offsets,
                                 int32_t nfrags, mxfp8_tensor* scale_inv_rowwise,
                                 mxfp8_tensor* scale_inv_colwise, mxfp8_tensor* output_rowwise,
                                 mxfp8_tensor* output_colwise, int64_t rows, int64_t cols,
                                 void* stream);

/*
 * NVFP4 partial cast.  The same distributed steps as the MXFP8 entry points above (partial
 * amax of a fragment, MAX reduction of the packed amaxes over ranks with
 * mxfp8_amax_max_reduce on F32 slots, scale update, partial cast in place) for the NVFP4
 * format.  The page "Support row-only MXFP8 distributed master-weight casts" leaves NVFP4
 * out of its scope (section "Scope") and gives no rule for it; the convention is:
 *   blocks   1x16 along rows (rowwise), 16x1 along columns (columnwise);
 *   G        tensor amax: max |x| over the whole weight, F32;
 *   S        tensor encode scale 2688 / G in F32 (448 * 6); 1 when G == 0; the largest
 *            finite float when the quotient overflows;
 *   s        block scale byte: E4M3(fp32(fp32(A / 6) * S)), A the block amax
 *            (nearest-even, saturating at 448);
 *   data     E2M1(fp32(y * fp32(S / decode(s)))) (0 when s decodes to 0), y = x rounded
 *            to BF16 (nearest-even; identity for BF16 input); E2M1 has magnitudes 0,
 *            0.5, 1, 1.5, 2, 3, 4, 6 (codes 0-7, sign in bit 3), nearest-even,
 *            saturating at 6.  Two codes per byte: element at nibble position p sits in
 *            byte p / 2, the low nibble holding even p.
 * Each F32 step is one correctly rounded operation.  Non-finite inputs are outside the
 * convention (E2M1 has no NaN or infinity): their codes are unspecified.  A consumer
 * dequantises a code q of block scale s as decode(q) * decode(s) / S.
 */

/*
 * input         [in]     fragment as for mxfp8_partial_amax (F32 or BF16).
 * amax_rowwise  [in,out] REQUIRED F32 [>= rows][>= ceil(cols/16)]: entry (i, b) = max |x|
 *                        over the fragment's elements of row i, columns [16b, 16b+16).
 * amax_colwise  [in,out] OPTIONAL F32 [>= ceil(rows/16)][>= cols]: entry (c, j) over
 *                        rows [16c, 16c+16) of column j; empty => row-only.
 * amax_tensor   [in,out] REQUIRED F32, at least 1 element: element 0 is max-accumulated
 *                        with the fragment's largest |x| (it must hold +0 or a previous
 *                        maximum: initialise it to +0 before the first fragment).
 * Entries of blocks the fragment touches are overwritten, others untouched; NaN
 * members give the canonical quiet NaN.  Errors as mxfp8_partial_amax; 4 also for a
 * missing amax_tensor; 3 if an amax tensor is not F32.
 */
MXFP8_API int nvfp4_partial_amax(const mxfp8_tensor* input, mxfp8_tensor* amax_rowwise,
                       mxfp8_tensor* amax_colwise, mxfp8_tensor* amax_tensor, int64_t rows,
                       int64_t cols, int64_t start_offset, void* stream);

/*
 * amax_rowwise [in] REQUIRED F32 [>= rows][>= ceil(cols/16)] (reduced over ranks);
 * amax_colwise [in] OPTIONAL F32 [>= ceil(rows/16)][>= cols]; empty => no columnwise scales;
 * amax_tensor  [in] REQUIRED F32: element 0 is G;
 * scale_rowwise [out] REQUIRED U8 [>= rows][>= ceil(cols/16)] E4M3 block scales;
 * scale_colwise [out] U8 [>= ceil(rows/16)][>= cols]; required iff amax_colwise present.
 * Writes every entry of the compact grids; padding untouched.
 */
MXFP8_API int nvfp4_update_scales(const mxfp8_tensor* amax_rowwise, const mxfp8_tensor* amax_colwise,
                        const mxfp8_tensor* amax_tensor, mxfp8_tensor* scale_rowwise,
                        mxfp8_tensor* scale_colwise, int64_t rows, int64_t cols, void* stream);

/*
 * input          [in]  fragment as for mxfp8_partial_cast.
 * scale_rowwise  [in]  REQUIRED U8 [>= rows][>= ceil(cols/16)].
 * scale_colwise  [in]  U8 [>= ceil(rows/16)][>= cols]; required iff output_colwise.
 * amax_tensor    [in]  REQUIRED F32: element 0 is G (the same G the scales came from).
 * output_rowwise [out] REQUIRED U8 packed codes, numel >= (out_offset + len) / 2.
 * output_colwise [out] OPTIONAL U8 packed codes (empty => row-only), same size rule.
 * Element k of the fragment goes to nibble position out_offset + k (out_offset =
 * start_offset: full-size output of ceil(rows*cols/2) bytes, in place; 0: fragment-
 * size output).  Two codes share a byte, so cols, start_offset, the fragment length and
 * out_offset must be even (status 1 otherwise); then every byte a fragment writes
 * belongs to it alone.  Other errors as mxfp8_partial_cast.
 */
MXFP8_API int nvfp4_partial_cast(const mxfp8_tensor* input, const mxfp8_tensor* scale_rowwise,
                       const mxfp8_tensor* scale_colwise, const mxfp8_tensor* amax_tensor,
                       mxfp8_tensor* output_rowwise, mxfp8_tensor* output_colwise, int64_t rows,
                       int64_t cols, int64_t start_offset, int64_t out_offset, void* stream);

/*
 * Training operators around the MXFP8 weights: 8-bit activation checkpoints, the
 * block-scaled matrix product that reads them and the cast's outputs, and layer norm.
 * (No counterpart in the source pages, which end at the weights.)
 *
 * Conventions of these entry points, besides the ones at the top of this file:
 * - A matrix argument is 2-D [>= rows][>= cols] with row stride shape[1] (a padded or a
 *   larger buffer's rows), or 1-D and dense.  A vector argument has numel >= its length.
 * - Scales in the GEMM layout: the 128x4-tile layout of mxfp8_swizzle_scales, at least
 *   mxfp8_swizzled_scales_size bytes, 16-byte aligned.
 * - Outputs must not overlap inputs, unless an argument says so.
 * - A call with no elements to write returns 0 and launches nothing.
 * - The first product or layer norm on a device loads its kernels and looks up a device address:
 *   make one such call before a stream capture.
 */

/*
 * 8-bit activation checkpoint: E4M3 codes of an activation (or of a gradient) with one E8M0
 * scale per 128 values, along its rows and/or along its columns, from one read of the input.
 * The scale convention is the one at the top of this file with blocks of 128 (the last block
 * of a row or column may be shorter) and without the rounding through BF16:
 * code = E4M3(x * 2^-e), one rounding.  A block that holds a NaN or an infinity has the scale
 * byte 0xFF and NaN codes.
 *
 * input          [in]  F32 or BF16 matrix rows x cols.
 * codes_rowwise  [out] OPTIONAL U8 matrix rows x cols, in blocks of 1x128.
 * scale_rowwise  [out] required iff codes_rowwise: its scale grid [rows][ceil(cols/128)] in the
 *                      GEMM layout (transpose 0), padding entries written as zeros.
 * codes_colwise  [out] OPTIONAL U8 matrix rows x cols (not transposed), in blocks of 128x1.
 * scale_colwise  [out] required iff codes_colwise: its scale grid [ceil(rows/128)][cols] in the
 *                      GEMM layout with transpose 1, padding entries written as zeros.
 * Errors: 1 bad sizes or a scale buffer that is not 16-byte aligned; 2 a buffer too small;
 * 3 dtype; 4 a missing input or scale buffer, or neither direction present.
 */
MXFP8_API int mxfp8_checkpoint_save(const mxfp8_tensor* input, mxfp8_tensor* codes_rowwise,
                          mxfp8_tensor* scale_rowwise, mxfp8_tensor* codes_colwise,
                          mxfp8_tensor* scale_colwise, int64_t rows, int64_t cols, void* stream);

/*
 * The values that one copy of a checkpoint stands for: output = decode(code) * 2^(s - 127).
 *
 * codes   [in]  U8 matrix rows x cols;  scale [in] its scales as mxfp8_checkpoint_save wrote
 *               them;  colwise 1 for the columnwise copy, 0 for the rowwise one.
 * output  [out] F32 or BF16 matrix rows x cols (exact in both, BF16 subnormals rounded to
 *               nearest-even).  Errors as above; 1 also for another colwise.
 */
MXFP8_API int mxfp8_checkpoint_restore(const mxfp8_tensor* codes, const mxfp8_tensor* scale,
                             mxfp8_tensor* output, int64_t rows, int64_t cols, int32_t colwise,
                             void* stream);

/*
 * Matrix product of two block-scaled 8-bit operands,
 *   out[i][j] = sum_p A(i, p) * B(j, p) (+ addend[i][j]),   i < m, j < n, p < k,
 * A(i, p) = decode(code) * 2^(s - 127), s the scale of the block of p; likewise B.  Products
 * are exact and summed in F32 by the matrix instruction, whose additions are coarser than one rounding to
 * nearest each (k = 8192: a relative error of 5e-7 over the matrix, 1.2e-7 with F32 products of the decoded
 * values); the addend joins in F32 and the result is rounded once.
 *
 * a, b               [in] U8 E4M3 codes.  Rowwise (colwise flag 0): the matrix m x k (n x k), the
 *                         contraction along its rows.  Columnwise (flag 1): the matrix k x m
 *                         (k x n), the contraction along its columns -- the columnwise copy of
 *                         a checkpoint or of a weight, read as it lies.
 * a_scale, b_scale   [in] the operand's scales in the GEMM layout, logical grid
 *                         [m][ceil(k/block)] ([n][...]): transpose 0 of a rowwise grid,
 *                         transpose 1 of a columnwise one.  Padding entries must not be 0xFF.
 * a_block, b_block        values per scale along the contraction: 128 (checkpoints) or 32
 *                         (weights of mxfp8_partial_cast).
 * addend             [in] OPTIONAL F32 matrix m x n; may be the same matrix as an F32 out (the
 *                         product is then added to it).
 * out               [out] F32 or BF16 matrix m x n.
 * With y = x W^T, W [outs][ins]: output y: a = x rowwise, b = W rowwise; input gradient
 * dx = dy W: a = dy rowwise, b = W columnwise; weight gradient dW = dy^T x: a = dy columnwise,
 * b = x columnwise.  k may be 0 (operands and scales may then be empty): out = addend or 0.
 * Operands whose base and row stride are multiples of 16 bytes are fetched as they lie; others
 * are realigned on the way, which takes longer.
 * Results do not depend on the run: no atomics, one fixed order of sums per shape, alignment and number of
 * the GPU's SMs.
 * Errors: 1 bad sizes (m, n, k <= 2^31 - 1024), flags or blocks, unaligned scales, or an addend
 * that overlaps out without being the same matrix; 2 a buffer too small; 3 dtype; 4 missing.
 */
MXFP8_API int mxfp8_gemm(const mxfp8_tensor* a, const mxfp8_tensor* a_scale, const mxfp8_tensor* b,
               const mxfp8_tensor* b_scale, const mxfp8_tensor* addend, mxfp8_tensor* out, int64_t m,
               int64_t n, int64_t k, int32_t a_colwise, int32_t b_colwise, int32_t a_block,
               int32_t b_block, void* stream);

/*
 * Health of the operators' kernels: waits for `stream`, then returns 0, or MXFP8_ERR_CUDA when
 * a product or a layer norm on the current device gave up a wait on its own copies or
 * tensor-core work (every wait inside these kernels ends after about two seconds; the outputs of such a call
 * are invalid).  Each such kernel is reported once, by the first call that sees it; those on other streams
 * than `stream` once they have completed.  Not for use during stream capture.
 */
MXFP8_API int mxfp8_device_status(void* stream);

/*
 * Layer norm of each row: output = (x - mean) * rstd * weight + bias, mean and rstd =
 * 1 / sqrt(var + eps) over the row's cols values (var: the mean squared deviation), in F32,
 * rounded once.
 *
 * input   [in]  F32 or BF16 matrix rows x cols;  output [out] same dtype; may be the input.
 * weight  [in]  F32 or BF16 vector of cols;  bias [in] OPTIONAL, weight's dtype.
 * mean, rstd [out] F32 vectors of rows.
 * Errors: 1 bad sizes (cols <= 2^31 - 1024) or eps < 0 or NaN; 2 too small; 3 dtype; 4 missing.
 */
MXFP8_API int mxfp8_layer_norm_forward(const mxfp8_tensor* input, const mxfp8_tensor* weight,
                             const mxfp8_tensor* bias, mxfp8_tensor* output, mxfp8_tensor* mean,
                             mxfp8_tensor* rstd, int64_t rows, int64_t cols, float eps, void* stream);

/*
 * Gradients of layer norm.  With xh = (x - mean) * rstd and g = grad_output * weight:
 *   grad_input  = rstd * (g - mean_cols(g) - xh * mean_cols(g * xh))
 *   grad_weight = sum_rows grad_output * xh,   grad_bias = sum_rows grad_output.
 *
 * grad_output [in]  F32 or BF16 matrix rows x cols.
 * input       [in]  the forward pass's input: the dtype of grad_output, or U8: the rowwise copy of
 *                   its checkpoint, with input_scale its scales (input_scale is empty otherwise).
 * weight      [in]  F32 or BF16 vector;  mean, rstd [in] F32, as the forward pass left them.
 * grad_input  [out] dtype of grad_output; may be grad_output itself.
 * grad_weight [out] F32 vector of cols;  grad_bias [out] OPTIONAL F32 vector of cols.
 * workspace   [out] at least mxfp8_layer_norm_workspace_size(rows, cols) bytes (U8), 16-byte
 *                   aligned; its contents before the call do not matter and after it mean
 *                   nothing.  Calls that overlap on the GPU need workspaces of their own.
 * The sums have one fixed order for a shape and the alignment of the arguments: results do not
 * depend on the run.
 * rows == 0: the gradients of weight and bias are set to zero.
 * Errors: 1 bad sizes, unaligned scales or workspace; 2 too small; 3 dtype; 4 missing.
 */
MXFP8_API int mxfp8_layer_norm_backward(const mxfp8_tensor* grad_output, const mxfp8_tensor* input,
                              const mxfp8_tensor* input_scale, const mxfp8_tensor* weight,
                              const mxfp8_tensor* mean, const mxfp8_tensor* rstd,
                              mxfp8_tensor* grad_input, mxfp8_tensor* grad_weight,
                              mxfp8_tensor* grad_bias, mxfp8_tensor* workspace, int64_t rows,
                              int64_t cols, void* stream);

/* Bytes of workspace of mxfp8_layer_norm_backward on any device (-1 for bad sizes). */
MXFP8_API int64_t mxfp8_layer_norm_workspace_size(int64_t rows, int64_t cols);

/* Message describing the calling thread's most recent non-zero status ("" if none). */
MXFP8_API const char* mxfp8_last_error(void);

/* Library version as major*10000 + minor*100 + patch. */
MXFP8_API int mxfp8_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_PARTIAL_H_ */
