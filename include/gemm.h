/*
 * gemm.h -- C ABI of libgemm: dense C = A*B on one GB300 GPU (sm_103a).
 *
 * The operation.  With A of size M x K, B of size K x N and C of size M x N,
 *     C_ij = sum over k = 0 .. K-1 of A_ik * B_kj
 * ("Shared Memory Tiling for Matrix Multiplication", opening formula).  All
 * three matrices are dense and row-major with no leading-dimension argument:
 * A_ik is A[i*K + k], B_kj is B[k*N + j], C_ij is C[i*N + j] ("Matrix
 * Multiplication -- Naive to Tiled", section 02).  C is overwritten, as that
 * page's kernels store the finished sum; it is never read.
 *
 * Argument order (M, K, N) follows the kernel signature of that same section.
 *
 * Every pointer is a DEVICE pointer on the calling thread's current CUDA
 * device; the caller owns all buffers and the stream, and the library frees
 * nothing it did not allocate.  Every call is asynchronous: it validates its
 * arguments on the host, enqueues its kernels on `stream` and returns.  Device
 * errors of an earlier call surface through gemm_debug_status() or the
 * caller's own synchronisation.  No call exits the process or traps the GPU.
 *
 * `stream` is a cudaStream_t (the pointer type is declared here so this header
 * needs no CUDA header); NULL means the legacy default stream.
 *
 * Environment (testing and tuning only; read once per process): with
 * GEMM_FORCE_CONFIG=single_cta the tensor-core modes use the 1-SM kernel even
 * where 2-SM clusters fit; =b_boxes_2d makes them load B by 2-D boxes per
 * column block even where the atom-ordered 4-D form applies (same results,
 * bit for bit); =ffma_small / =ffma_tiles128 make every GEMM_FP32 product
 * take the 32 x 32-tile or the 128 x 128-tile FFMA kernel instead of the one
 * chosen by shape; =ffma_no_stream keeps GEMM_FP32 products of a quarter of a
 * wave to two waves of tiles off the stream-K form.  Results stay within each mode's
 * tolerance.
 */
#ifndef LIBGEMM_GEMM_H
#define LIBGEMM_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* the type behind cudaStream_t */

#if defined(__GNUC__)
#define GEMM_API __attribute__((visibility("default")))
#else
#define GEMM_API
#endif

/* precision_mode values */
enum gemm_mode {
    /* A, B: const float*.  Exact binary32 arithmetic on the CUDA cores: every
     * product-accumulate is one fused multiply-add rounded to nearest, k
     * ascending for each C_ij.  When the output tiles do not fill the GPU
     * and K is long, the library cuts K into consecutive ranges, runs the
     * chain over each range and adds the range sums in range order (binary32
     * adds): the same result on every run of the same shape. */
    GEMM_FP32 = 0,
    /* A, B: const float*.  Tensor cores (tcgen05, kind::tf32): the inputs are
     * read as TF32 (sign, 8-bit exponent, top 10 fraction bits of each
     * binary32), products are accumulated in binary32. */
    GEMM_TF32 = 1,
    /* A, B: const uint16_t* holding bfloat16 values (the caller rounds its
     * data to bfloat16).  Tensor cores (tcgen05, kind::f16 with BF16
     * inputs), binary32 accumulation. */
    GEMM_BF16 = 2,
    /* A, B: const uint16_t* holding IEEE binary16 values.  Tensor cores
     * (tcgen05, kind::f16 with F16 inputs), binary32 accumulation -- the
     * FP16-input, FP32-accumulate product the first page's "Further
     * Optimisation Ideas" names for tensor cores. */
    GEMM_FP16 = 3,
    /* A, B: const float*.  The library rounds them to bfloat16 (to nearest,
     * ties to even) in a conversion pass, then multiplies as GEMM_BF16:
     * BF16 tensor-core speed for float data, at BF16 input precision.  The
     * result equals GEMM_BF16 on the caller-rounded operands, bit for bit. */
    GEMM_FP32_VIA_BF16 = 4,
    /* A, B: const float*.  As GEMM_TF32, but the library first rounds each
     * input to the nearest TF32 value (ties away from zero) in a conversion
     * pass, instead of letting the tensor cores drop the 13 low fraction
     * bits: the rounding errors of the inputs then have no sign bias, at the
     * cost of the pass (scratch for the rounded copies of A and B).  The
     * result equals GEMM_TF32 on the caller-rounded operands, bit for bit. */
    GEMM_TF32_RN = 5
};

/* Status codes returned by every entry point (0 = success). */
enum gemm_status {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1,        /* NULL pointer with a non-empty matrix, negative
                                        dimension, unknown mode, C overlapping A or B,
                                        or a size whose element count overflows int64 */
    GEMM_ERR_MISALIGNED = 2,         /* pointer not aligned to its element size
                                        (4 bytes for float, 2 for bfloat16/binary16) */
    GEMM_ERR_CUDA = 3,               /* a CUDA runtime call or kernel launch failed */
    GEMM_ERR_NO_MEMORY = 4,          /* the stream-ordered scratch allocation failed */
    GEMM_ERR_UNSUPPORTED_DEVICE = 5, /* the current device is not compute capability 10.3 */
    GEMM_ERR_TIMEOUT = 6,            /* a bounded wait inside a kernel expired; the kernel
                                        stopped early and its output is not valid */
    GEMM_ERR_SCRATCH_LIMIT = 7,      /* gemm_tf32_noalloc: the product needs more scratch
                                        than GEMM_NOALLOC_SCRATCH_BYTES */
    GEMM_ERR_BOUNDS = 8,             /* debug build only (gemm_debug_build() == 1): a kernel
                                        computed a global-memory access outside the buffer
                                        it belongs to; the access was skipped and the
                                        output is not valid */
    GEMM_ERR_INDEX = 9               /* reported by gemm_debug_status(): a kernel met a page
                                        number, a position or a row offset outside the cache,
                                        the page table or the rows of its call; it skipped
                                        that part, whose output is not valid */
};

/*
 * C = A*B.
 *   A               device pointer to M*K elements (float; bfloat16 in GEMM_BF16;
 *                   binary16 in GEMM_FP16)
 *   B               device pointer to K*N elements (same element type as A)
 *   C               device pointer to M*N floats; overwritten; must not overlap A or B
 *   M, K, N         dimensions, each >= 0.  M == 0 or N == 0: nothing is done.
 *                   K == 0: C is set to 0 (the empty sum).
 *   precision_mode  one of enum gemm_mode
 *   stream          stream to enqueue on
 * GEMM_FP32_VIA_BF16 and GEMM_TF32_RN take scratch for the rounded copies of A
 * and B, from the same stream-ordered allocator.
 * Any alignment of element size or more is accepted.  When a tensor-core mode
 * meets a row stride that is not a multiple of 16 bytes, or a base address
 * that is not 16-byte aligned, the operand is first copied into a scratch
 * buffer with a padded row stride; that buffer is taken from and returned to
 * CUDA's stream-ordered allocator on `stream` inside the call.  GEMM_FP32
 * does the same for B (K * roundup(N, 4) floats) when B's rows are not
 * 16-byte aligned and M >= 1024, so that B can be read 16 bytes at a time;
 * the K-split forms of both paths take workspace from the same allocator.
 * Returns GEMM_OK or an enum gemm_status code; on an error nothing is enqueued.
 */
GEMM_API int gemm(const void* A, const void* B, float* C, int64_t M, int64_t K, int64_t N,
         int precision_mode, struct CUstream_st* stream);

/*
 * C = alpha*A*B + beta*C -- the generalised product of the cuBLAS call that
 * "Matrix Multiplication -- Naive to Tiled" (section 07, Further Optimisation
 * Ideas) uses as its yardstick, for the same row-major operands as gemm().
 *   alpha, beta     binary32 scalars (host values)
 *   other arguments as for gemm(); C is read as well as written when beta != 0
 * Each C_ij is computed from the mode's sum acc_ij as fma(beta, C_ij, alpha *
 * acc_ij), the product alpha * acc_ij rounded to binary32 first and the fused
 * multiply-add rounded once.  Conventions of the BLAS, where the page is
 * silent:
 *   beta == 0       C is not read (NaN or garbage in C does not propagate);
 *                   each C_ij := alpha * acc_ij.
 *   alpha == 0, or K == 0   A and B are not read and no product is formed;
 *                   C := beta * C (each element rounded once), C := 0 when
 *                   beta == 0 as well, and nothing is enqueued when beta == 1.
 *   alpha == 1, beta == 0   identical to gemm(), bit for bit.
 * Validation, status codes, scratch use and asynchrony are those of gemm().
 */
GEMM_API int gemm_ex(const void* A, const void* B, float* C, int64_t M, int64_t K, int64_t N,
                     float alpha, float beta, int precision_mode, struct CUstream_st* stream);

/* Static, human-readable name of a status code ("unknown status" otherwise). */
GEMM_API const char* gemm_status_string(int status);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word, which kernels set when a bounded wait expires or an index that they
 * read is out of range, and, in the debug build, the bounds-check flags.
 * Returns GEMM_OK, GEMM_ERR_TIMEOUT, GEMM_ERR_BOUNDS (debug build),
 * GEMM_ERR_INDEX (the first of these where several happened), or
 * GEMM_ERR_CUDA if the synchronisation itself failed.
 */
GEMM_API int gemm_debug_status(struct CUstream_st* stream);

/*
 * 1 when this library was built with device-side bounds checks (compiled
 * with GEMM_DEBUG: every kernel checks each global access against the extent
 * of the buffer it belongs to, skips one that falls outside and records it
 * for gemm_debug_status), 0 for the release build, whose kernels carry no
 * checks.  The checks stand in for a memory checker where none can run.
 */
GEMM_API int gemm_debug_build(void);

/* Library version as major*10000 + minor*100 + patch. */
GEMM_API int gemm_version(void);

/*
 * Number of kernels this library has launched in this process, all devices
 * and streams together.  Lets a benchmark count the launches in a timed
 * region.
 */
GEMM_API int64_t gemm_launch_count(void);

/*
 * Self-test of the bounded wait used by the tensor-core kernel's pipeline:
 * launches one block that waits on a barrier nothing will ever complete,
 * giving up after `timeout_ns` nanoseconds (clamped to 1 us .. 2 s), and
 * synchronises.  Returns GEMM_ERR_TIMEOUT when the wait expired and was
 * reported as it should be, GEMM_OK if it was not (a defect), or a launch
 * error.  Clears the error word before returning.  The GPU stays usable.
 */
GEMM_API int gemm_selftest_bounded_wait(int64_t timeout_ns, struct CUstream_st* stream);

/*
 * gemm_tf32_noalloc -- the GEMM_TF32 product without allocating device memory.
 *
 * The pages have no counterpart for this entry point; it is a service of this
 * library.  gemm() in GEMM_TF32 sometimes needs scratch memory -- a copy of A
 * or B with 16-byte row strides when TMA cannot read them in place (K or N
 * not a multiple of 4, or a base not 16-byte aligned), and the workspace of
 * a K split (products with few output tiles and a long K, or a partial last
 * round of tiles, e.g. 4096^3) -- and takes it from CUDA's stream-ordered
 * allocator.  Some callers cannot allow that: a host application that has
 * reserved the device memory for its own pool, so an allocation would fail
 * or eat into its budget; or a latency-critical loop where an allocation may
 * stall or fail at a bad moment.  This entry point uses instead one static
 * device buffer of GEMM_NOALLOC_SCRATCH_BYTES, compiled into the library: it
 * never calls cudaMalloc, cudaMallocAsync, cudaFree or any allocating
 * routine.
 *
 * Arguments and results are those of gemm() with precision_mode GEMM_TF32:
 * A, B, C device pointers (float, 4-byte aligned), row-major, C overwritten,
 * asynchronous on `stream`.  The product is planned exactly as gemm() plans
 * it (the same kernels, the same K split, the same order of summation), so
 * C equals gemm()'s C bit for bit.  K == 0 gives C = 0.
 *
 * Limit: the scratch gemm() would take for the product -- 4 * M * roundup(K, 32)
 * bytes for a re-strided A, 4 * K * roundup(N, 32) for a re-strided B, and
 * 256 KB per split piece of the K split, each rounded up to 256 bytes -- must
 * not exceed GEMM_NOALLOC_SCRATCH_BYTES (64 MiB).  Aligned products with
 * K, N multiples of 4 need at most the split workspace (14.7 MB at 4096^3,
 * 18.5 MB at 256 x 65536 x 256).  A product that needs more returns
 * GEMM_ERR_SCRATCH_LIMIT and enqueues nothing.
 *
 * Set-up and memory: the first call on a device (that device current) does
 * the library's per-device set-up and looks up the buffer's device address,
 * which loads this part of the library's device code, the 64 MiB buffer
 * with it, onto the device.  Make that first call before the application
 * reserves the rest of the device memory for itself, and before any stream
 * capture; later calls allocate nothing.  With CUDA's lazy module loading
 * (the default) only devices on which this entry point has been called hold
 * the buffer; with CUDA_MODULE_LOADING=EAGER every device on which the
 * process uses this library holds it.  It stays until the process exits.
 *
 * Sharing: every call on a device uses the same buffer, which keeps the last
 * call's contents (nothing in it needs to start at zero: every byte a call
 * reads was written earlier in that call).  Calls whose kernels overlap on
 * the GPU -- on different streams, or from different threads -- race on the
 * buffer and give wrong results: order them on one stream, or synchronise
 * between them.
 */
#define GEMM_NOALLOC_SCRATCH_BYTES (64ll * 1024 * 1024)

GEMM_API int gemm_tf32_noalloc(const float* A, const float* B, float* C, int64_t M, int64_t K,
                               int64_t N, struct CUstream_st* stream);

/*
 * ---- operands held in few bits ------------------------------------------
 *
 * The products of a decoding step, in which one operand is kept in 4 or 8
 * bits with scales: C = X*W with a 4-bit W for a few rows X, and attention
 * (two products with a softmax between them) over a paged cache of keys and
 * values in 8 or 4 bits.  The rules above hold: device pointers, asynchronous on
 * `stream`, status codes, nothing enqueued on an error, scratch from the
 * library's stream-ordered pool, safe under stream capture after the first
 * call on a device.  Indices that live in device memory (page numbers,
 * positions, row offsets) are checked by the kernels: one outside its range
 * is skipped and reported by gemm_debug_status() as GEMM_ERR_INDEX.
 */

/* Element types of the 16- and 32-bit operands. */
enum gemm_type { GEMM_TYPE_F32 = 0, GEMM_TYPE_BF16 = 1, GEMM_TYPE_F16 = 2 };

/*
 * 4-bit weights.  W stands for the K x N matrix q_kn * s_gn, q in [-7, 7],
 * with one bfloat16 scale s for each column n and each `group` consecutive
 * rows g = k / group (group: 32, 64 or 128; the last group may be short).
 * C_mn = sum over k of X_mk * q_kn * s_(k/group)n.
 *
 * Layout.  Codes: u = q + 8, in blocks of 16 columns x 64 rows of 512 bytes;
 * block (n / 16, k / 64) is number (n / 16) * ceil(K / 64) + k / 64.  In a
 * block, the 32-bit word 4 * (4 * (n % 8) + k % 32 / 8) + 2 * (k % 64 / 32)
 * + k % 8 / 4 holds the element in bits 4i .. 4i + 3 with i = 4 * (k % 2) +
 * 2 * (k % 4 / 2) + n % 16 / 8: what one lane of a warp needs for a matrix
 * instruction is one 16-byte load.  Scales: element
 * (((n / 16) * ceil(K / group) + k / group) * 8 + n % 8) * 2 + n % 16 / 8.
 * gemm_w4_quantize writes q = 0 and s = 0 where the blocks reach past K or N.
 */

/* Bytes of the codes and of the scales of a K x N matrix (both 0 when K or N
 * is 0); GEMM_ERR_INVALID_ARG for a group that is not 32, 64 or 128 or sizes
 * out of range. */
GEMM_API int gemm_w4_sizes(int64_t K, int64_t N, int group, int64_t* code_bytes,
                           int64_t* scale_bytes);

/*
 * B (K x N, row stride ldb >= N elements, of `type`) to codes and scales:
 * s = max|b| * (1 / 7) over the group's rows of the column (one binary32
 * product with the binary32 1 / 7), rounded to bfloat16, q = b / s rounded to the nearest integer (ties to even) and held to
 * [-7, 7].  A group whose s is under 2^-126 becomes zeros; one that holds a
 * NaN or an infinity gets s = NaN, so that every product with it is NaN.
 * codes and scales: 16-byte aligned, here and below.
 */
GEMM_API int gemm_w4_quantize(const void* B, int64_t ldb, int type, int64_t K, int64_t N,
                              int group, void* codes, void* scales, struct CUstream_st* stream);

/* The values q * s (formed in binary32, rounded once to `type`) into B. */
GEMM_API int gemm_w4_dequantize(const void* codes, const void* scales, int64_t K, int64_t N,
                                int group, void* B, int64_t ldb, int type,
                                struct CUstream_st* stream);

/*
 * C = X*W.  X: M x K, row stride ldx elements, bfloat16 or binary16
 * (x_type); C: M x N, row stride ldc, of x_type or float (c_type),
 * overwritten, not overlapping the inputs.  Made for few rows: up to 32 rows
 * read W once, and each further 32 read it again.  Products q * x are exact,
 * summed in binary32 over a group (or a part of one) and scaled there; C is
 * rounded once.  The order of the sums depends on the sizes alone.  K == 0
 * gives 0.
 */
GEMM_API int gemm_w4(const void* X, int64_t ldx, int x_type, const void* codes,
                     const void* scales, void* C, int64_t ldc, int c_type, int64_t M, int64_t K,
                     int64_t N, int group, struct CUstream_st* stream);

/*
 * A paged cache of keys and values in 8 bits.  A page holds page_tokens
 * consecutive tokens (16, 32, 64 or 128) of one sequence for every head;
 * element d of token t, head h of page p is code (((p * heads + h) *
 * page_tokens + t) * head_dim + d), an unsigned byte c + 128 with c in
 * [-127, 127], and stands for c * scale[p * heads + h] (binary32 scales, one
 * for the page's keys and one for its values, >= 0 or NaN).  head_dim: 64 or
 * 128.  Codes are 16-byte aligned.  The caller owns all of it; a page needs
 * no initial contents.
 */
typedef struct gemm_kv_cache {
    void* k_codes;
    void* v_codes;
    float* k_scales;
    float* v_scales;
    int64_t pages;
    int32_t heads, page_tokens, head_dim;
} gemm_kv_cache;

/*
 * What the calls on a cache share: a batch of sequences with their rows of
 * new tokens (or queries) one after another.
 *   page_table  int32[sequences][table_width]: the page that holds a
 *               sequence's tokens page_tokens * i ... in column i
 *               (table_width * page_tokens <= 2^31 - 1024)
 *   starts      int32[sequences + 1]: sequence b's rows are starts[b] ..
 *               starts[b + 1] - 1 (ascending; starts[0] = 0, the last one
 *               = tokens); a sequence may have none
 *   tokens      the number of rows; it and `sequences` are host values
 * These arrays are on the device, 4-byte aligned.
 */

/*
 * Writes new keys and values: row starts[b] + i becomes token first[b] + i of
 * sequence b.  K and V: rows of heads x head_dim elements of `type`, element
 * (row, h, d) at row * row_stride + h * head_stride + d (strides in
 * elements, >= 0).  For each page, head and operand that gets new tokens,
 *     s' = max(s, max|x| * (1 / 127))   (s = 0 if token 0 of the page is new)
 * over its new elements x; new codes are x * (1 / s') rounded to the nearest
 * integer (ties to even) and held to [-127, 127]; if s' > s the page's older
 * codes c (its tokens before the first new one) become c * (s * (1 / s'))
 * rounded alike.  Each of these steps is one binary32 operation.  With
 * s' < 2^-126 they are all 0; a NaN or an infinity makes s' NaN, so that the
 * page's tokens read as NaN for that head until its token 0 is written again.
 * Tokens after the last new one are left as they are.  No page may belong to
 * two of the sequences that are written in one call.
 */
GEMM_API int gemm_kv_append(const gemm_kv_cache* cache, const void* K, int64_t k_row_stride,
                            int64_t k_head_stride, const void* V, int64_t v_row_stride,
                            int64_t v_head_stride, int type, const int32_t* page_table,
                            int64_t table_width, const int32_t* starts, const int32_t* first,
                            int64_t tokens, int64_t sequences, struct CUstream_st* stream);

/*
 * Reads tokens back: rows starts[b] + i of K and V (dense, tokens x heads x
 * head_dim, of `type`, 16-byte aligned) become the values of token
 * first[b] + i of sequence b: c * s in binary32, rounded once.
 */
GEMM_API int gemm_kv_read(const gemm_kv_cache* cache, void* K, void* V, int type,
                          const int32_t* page_table, int64_t table_width, const int32_t* starts,
                          const int32_t* first, int64_t tokens, int64_t sequences,
                          struct CUstream_st* stream);

/*
 * Attention of ragged queries over the cache.  Sequence b has lengths[b]
 * tokens in the cache and T = starts[b + 1] - starts[b] queries, which stand
 * at its last T positions: query i at p = lengths[b] - T + i.  For query
 * head h (of q_heads, a multiple of the cache's heads; it reads head
 * h / (q_heads / heads))
 *     O = sum over j of softmax_j(scale * Q . K_j) V_j
 * over the tokens 0 <= j < lengths[b], with causal != 0 only j <= p, and with
 * window > 0 (causal only) only j > p - window.  A query that sees no token
 * (p < 0, or an empty cache) gets 0.  Pages wholly before every query's window
 * are not looked up: their entries of the table may be anything.  Q and O:
 * rows of q_heads x head_dim elements of `type` (bfloat16 or binary16), strides
 * as above; O must not overlap the inputs, nor its rows and heads one another.
 * Softmax statistics and sums are binary32 (a weight under 2^-126 of the row's
 * largest counts as 0); a weight times its page's value scale enters the second
 * product as binary16 relative to the largest that the row sees, O is rounded
 * once.  The order of the sums depends on the sizes, the lengths and the page
 * table's width alone.
 */
GEMM_API int gemm_kv_attention(const gemm_kv_cache* cache, const void* Q, int64_t q_row_stride,
                               int64_t q_head_stride, void* O, int64_t o_row_stride,
                               int64_t o_head_stride, int type, int32_t q_heads, float scale,
                               int causal, int64_t window, const int32_t* page_table,
                               int64_t table_width, const int32_t* starts,
                               const int32_t* lengths, int64_t tokens, int64_t sequences,
                               struct CUstream_st* stream);

/*
 * A paged cache of keys and values in 4 bits.  Pages are as above (page_tokens
 * tokens of one sequence for every head); what differs is that every token and
 * head has scales of its own, one for its keys and one for its values, so that a
 * token is written without a change to any other.  Keys and values of a page and
 * head are one record of page_tokens * (head_dim + 4) bytes, number p * heads + h:
 *     key codes     page_tokens * head_dim / 2 bytes
 *     value codes   the same
 *     key scales, value scales   bfloat16[page_tokens] each, >= 0 or NaN
 * A code is a nibble u = c + 8, c in [-7, 7], and stands for c * its scale.  Key
 * codes: element d of token t is nibble d % 2 (0: the low one) of byte t *
 * head_dim / 2 + d % 32 / 8 * (head_dim / 8) + d / 32 * 4 + d % 8 / 2.  Value
 * codes, in blocks of 16 tokens: nibble d % 2 of byte t / 16 * (8 * head_dim) +
 * t % 16 / 8 * (4 * head_dim) + (4 * (d % 64 / 8) + t % 8 / 2) * (head_dim / 8)
 * + d / 64 * 8 + d % 8 / 4 * 4 + t % 2 * 2 + d % 4 / 2.  What one lane of a warp
 * needs of 16 tokens for its matrix instructions is one 16-byte load of each 8
 * tokens (8-byte with head_dim 64).  `data` is 16-byte aligned; a page needs no initial
 * contents.  page_tokens and head_dim as above.
 */
typedef struct gemm_kv4_cache {
    void* data;
    int64_t pages;
    int32_t heads, page_tokens, head_dim;
} gemm_kv4_cache;

/*
 * As gemm_kv_append, into a cache of 4 bits.  Each row's head_dim elements x of a
 * head get s = max|x| * (1 / 7) (one binary32 product with the binary32 1 / 7),
 * rounded to bfloat16, and c = x / s rounded to the nearest integer (ties to even)
 * and held to [-7, 7].  With s under 2^-126 they are zeros (c = 0, s = 0); a
 * NaN or an infinity makes s NaN, so that this token reads as NaN for that head.
 * Nothing else of the cache is written: a page may belong to two sequences, as
 * long as no token of it is written twice in one call.
 */
GEMM_API int gemm_kv4_append(const gemm_kv4_cache* cache, const void* K, int64_t k_row_stride,
                             int64_t k_head_stride, const void* V, int64_t v_row_stride,
                             int64_t v_head_stride, int type, const int32_t* page_table,
                             int64_t table_width, const int32_t* starts, const int32_t* first,
                             int64_t tokens, int64_t sequences, struct CUstream_st* stream);

/* As gemm_kv_read, from a cache of 4 bits. */
GEMM_API int gemm_kv4_read(const gemm_kv4_cache* cache, void* K, void* V, int type,
                           const int32_t* page_table, int64_t table_width, const int32_t* starts,
                           const int32_t* first, int64_t tokens, int64_t sequences,
                           struct CUstream_st* stream);

/*
 * As gemm_kv_attention, over a cache of 4 bits.  A query's row is brought to binary16
 * by a power of two (exact, but for elements under 2^-14 of the row's largest).  A
 * weight times its token's value scale, or where a sequence and head has many rows
 * the largest value scale of its 16 tokens, enters the second product as binary16
 * relative to the largest such product that the row sees.
 */
GEMM_API int gemm_kv4_attention(const gemm_kv4_cache* cache, const void* Q, int64_t q_row_stride,
                                int64_t q_head_stride, void* O, int64_t o_row_stride,
                                int64_t o_head_stride, int type, int32_t q_heads, float scale,
                                int causal, int64_t window, const int32_t* page_table,
                                int64_t table_width, const int32_t* starts,
                                const int32_t* lengths, int64_t tokens, int64_t sequences,
                                struct CUstream_st* stream);

/*
 * ---- what a batch of sequences needs around a cache ----------------------
 */

/*
 * The plan of a step, made on the device from what is there: row offsets,
 * positions and slots of the new tokens, and the pages that they need.
 *   lengths         int32[sequences]: tokens that each sequence has in the cache
 *   counts          int32[sequences]: how many it gets (0: it rests)
 *   free_pages      int32[free_capacity]: a stack of free pages, of which the
 *                   first available[0] are on it
 *   page_table      as above; its columns up to a sequence's present length
 *                   name its pages, the others are written here
 * and it writes
 *   starts          int32[sequences + 1]: exclusive sums of the counts
 *   first           int32[sequences]: the lengths as they were
 *   new_lengths     int32[sequences]: lengths + counts; may be `lengths`
 *   page_table      the pages that the new tokens begin: taken off the stack's
 *                   top in the order of sequences and tokens
 *   heights         int32[sequences + 1]: the stack's height before each sequence
 *                   takes its pages, and after the last one (under 0: so many
 *                   were missing)
 *   left            int32[1]: what is left on the stack; may be `available`
 *   positions       int32[tokens]: first[b] + i in row starts[b] + i
 *   slots           int64[tokens]: page * page_tokens + position % page_tokens of
 *                   that token's page, -1 where it has none
 * `tokens` is the room that positions and slots have; rows past starts[sequences]
 * get -1 in both (gemm_rotary leaves such rows as they are; so do the calls on a
 * cache, which report offsets that end before the last row).  page_tokens is a
 * power of 2 up to 2^20.  Reported as GEMM_ERR_INDEX: a negative length or count
 * (taken for 0), counts whose sum is over `tokens` (sequences get the rows that
 * there is room for, in their order, and starts, lengths and pages go by those
 * alone), a sequence longer than the table is wide or a stack that runs
 * out (the tokens without a page have -1 in slots, and, inside the table, in
 * page_table), a height over free_capacity.
 * The arrays do not overlap but where said.  Calls that take from one stack are one
 * after another.  A sequence that ends gives its pages back by their numbers written
 * to free_pages from available[0] on, which then counts them.
 */
GEMM_API int gemm_kv_plan(int32_t* page_table, int64_t table_width, const int32_t* lengths,
                          const int32_t* counts, const int32_t* free_pages,
                          int64_t free_capacity, const int32_t* available, int32_t page_tokens,
                          int64_t tokens, int64_t sequences, int32_t* starts, int32_t* first,
                          int32_t* new_lengths, int32_t* heights, int32_t* left,
                          int32_t* positions, int64_t* slots, struct CUstream_st* stream);

/* How the elements of a head pair up: i with i + rotary_dim / 2, or 2i with 2i + 1. */
enum gemm_rotary_layout { GEMM_ROTARY_HALF = 0, GEMM_ROTARY_INTERLEAVED = 1 };

/*
 * Rotary positions.  Pair i (i < rotary_dim / 2) of every head in row r, the
 * elements (a, b), becomes
 *     magnitude * (a cos x - b sin x),  magnitude * (b cos x + a sin x)
 * with x = positions[r] * frequency i; with inverse != 0 by -x, which is the
 * transposed map: the gradient's way back.  Elements from rotary_dim on are
 * copied.  A row with a negative position is left as it is (its results are not
 * written).
 *   Q, K      rows of q_heads and k_heads heads of head_dim elements of `type`
 *             (strides in elements, >= 0); K may be NULL with k_heads 0
 *   Q_out, K_out  the results, likewise; each may be its input (same address and
 *             strides) and must not overlap anything else.  Slices of one array do not
 *             overlap where rows or heads of one lie between those of the other.
 *   head_dim  up to 1024; rotary_dim: even, 2 .. head_dim
 *   positions int32[rows], on the device
 *   turns     uint64[rotary_dim / 2], on the device: frequency i in turns
 *             (radians / 2 pi) a position, times 2^64, rounded.  The angle is the
 *             product's fraction of a turn, exact for every position; what it is past
 *             the nearest quarter turn is rounded to binary32.
 * Sines and cosines (to some 2^-24 of themselves, next to their zeros too), products
 * and sums are binary32; a result is rounded once.
 */
GEMM_API int gemm_rotary(const void* Q, int64_t q_row_stride, int64_t q_head_stride, void* Q_out,
                         int64_t q_out_row_stride, int64_t q_out_head_stride, int32_t q_heads,
                         const void* K, int64_t k_row_stride, int64_t k_head_stride, void* K_out,
                         int64_t k_out_row_stride, int64_t k_out_head_stride, int32_t k_heads,
                         int type, int64_t rows, int32_t head_dim, int32_t rotary_dim, int layout,
                         const int32_t* positions, const uint64_t* turns, float magnitude,
                         int inverse, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBGEMM_GEMM_H */
