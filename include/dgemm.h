/*
 * dgemm.h -- C ABI of libdgemm.so: tiled dense GEMM C = A x B on MI355X (gfx950).
 *
 * Operation.  Every entry point computes C = A x B, C_ij = sum_k A_ik * B_kj,
 * 2*M*N*K flops ("Optimizing GEMM in HIP", ROCm optimization guide, section
 * "GEMM fundamentals"), with products and sums in FP32 (FP32 accumulation for
 * every input format) and one conversion of each FP32 result to the output
 * format with round-to-nearest-even.  C is overwritten (no alpha/beta).
 *
 * Layouts (leading dimensions are in ELEMENTS):
 *   DGEMM_NN  A is M x K row-major       A(i,k) = A[i*lda + k],  lda >= K
 *             B is K x N row-major       B(k,j) = B[k*ldb + j],  ldb >= N
 *             C is M x N row-major       C(i,j) = C[i*ldc + j],  ldc >= N
 *   DGEMM_TN  the pairing named TN in "FP16 GEMM Optimization on AMD RDNA 3
 *             and RDNA 4", section "What We Are Computing": both operands
 *             contiguous along K, C column-major.
 *             A is M x K row-major       A(i,k) = A[i*lda + k],  lda >= K
 *             B is K x N column-major    B(k,j) = B[j*ldb + k],  ldb >= K
 *             C is M x N column-major    C(i,j) = C[j*ldc + i],  ldc >= M
 *
 * Formats: FP32 = IEEE binary32; FP16 = IEEE binary16 bits; BF16 = bfloat16
 * bits; FP8 = OCP E4M3 ("E4M3FN": bias 7, max 448, no infinity) bytes, used
 * raw with no scale factors ("FP8 GEMM Optimization on AMD RDNA 4", section
 * "What Changes at FP8"), producing FP32 output.
 *
 * Memory and ownership.  A, B and C are DEVICE pointers owned by the caller;
 * the library never allocates, frees or retains them and keeps no mutable
 * global state (beyond two thread-local diagnostics: the last HIP error code
 * and the clock-trace buffer set with dgemm_trace_clock), so calls are
 * reentrant.
 * A and B must not overlap C, and must be readable over whole rows of
 * their pitch: A over M*lda elements, B over K*ldb (NN) or N*ldb (TN); the
 * kernels copy 16-byte pieces and may read the padding of the last row.
 * Alignment: A and B must be 16-byte aligned and lda*elem, ldb*elem must be
 * multiples of 16 bytes (elem = bytes per input element); C needs only its
 * element alignment (wider stores are used when C and ldc allow them).
 * Size limits: the bytes one block tile addresses in an operand must stay
 * below 2^31 (for a K-contiguous operand: 256 rows * ld * elem; for the NN
 * B operand: K * ldb * elem), and the tiles of C have to fit a launch (fewer
 * than 2^32 work-items: they do while the product of M and N, both rounded up
 * to multiples of 32, is below 2^32); beyond that the call returns
 * DGEMM_ERR_UNSUPPORTED.
 *
 * Streams.  The work is enqueued on `stream` (a hipStream_t; NULL = the null
 * stream) and the call returns without synchronising.  Faults inside the
 * kernel surface at the caller's next synchronisation.
 *
 * Errors.  Each call returns a dgemm_status and never prints or aborts; the
 * code of the last HIP failure is kept per thread (dgemm_last_hip_error).
 * Checks, in this order: layout -> DGEMM_ERR_INVALID_LAYOUT; any of M, N, K
 * negative -> DGEMM_ERR_INVALID_DIM; M == 0 or N == 0 -> DGEMM_OK with no
 * work; a NULL A or B (when K > 0) or NULL C -> DGEMM_ERR_NULL_POINTER; a
 * leading dimension below its minimum -> DGEMM_ERR_INVALID_LD; misaligned A
 * or B base or pitch -> DGEMM_ERR_MISALIGNED; size limits ->
 * DGEMM_ERR_UNSUPPORTED; a HIP launch error -> DGEMM_ERR_HIP.
 * K == 0 is valid: C is filled with zeros (the empty sum).
 */
#ifndef DGEMM_H
#define DGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { DGEMM_NN = 0, DGEMM_TN = 1 } dgemm_layout;

typedef enum {
  DGEMM_OK = 0,
  DGEMM_ERR_INVALID_DIM = 1,
  DGEMM_ERR_NULL_POINTER = 2,
  DGEMM_ERR_INVALID_LD = 3,
  DGEMM_ERR_INVALID_LAYOUT = 4,
  DGEMM_ERR_MISALIGNED = 5,
  DGEMM_ERR_UNSUPPORTED = 6,
  DGEMM_ERR_HIP = 7,
  DGEMM_ERR_INVALID_TYPE = 8
} dgemm_status;

/* Element types of the operators that take more than one. */
typedef enum { DGEMM_F32 = 0, DGEMM_F16 = 1, DGEMM_BF16 = 2 } dgemm_type;

/* FP32 x FP32 -> FP32. */
int gemm_f32(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
             const float* B, int64_t ldb, float* C, int64_t ldc, int layout, void* stream);

/* FP16 x FP16 -> FP16 (binary16 bit patterns), FP32 accumulation. */
int gemm_f16(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda,
             const uint16_t* B, int64_t ldb, uint16_t* C, int64_t ldc, int layout, void* stream);

/* BF16 x BF16 -> BF16 (bfloat16 bit patterns), FP32 accumulation. */
int gemm_bf16(int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda,
              const uint16_t* B, int64_t ldb, uint16_t* C, int64_t ldc, int layout, void* stream);

/* OCP FP8 E4M3 x E4M3 -> FP32, FP32 accumulation, no scale factors. */
int gemm_fp8(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
             const uint8_t* B, int64_t ldb, float* C, int64_t ldc, int layout, void* stream);

/*
 * OCP FP8 E4M3 x E4M3 -> FP32 with scale factors, the per-tensor or per-row
 * factors a quantized kernel carries on top of the raw FP8 product ("FP8
 * GEMM Optimization on AMD RDNA 4", section "What Changes at FP8"):
 *   C_ij = (sum_k A_ik * B_kj) * (sa_i * sb_j)
 * with the sum accumulated in FP32 as in gemm_fp8 and each of the two
 * products rounded to FP32 (round-to-nearest-even); IEEE rules apply to
 * zero, infinite and NaN factors (K == 0 gives 0 * sa_i * sb_j).
 * scale_a: DEVICE pointer to n_scale_a FP32 values, n_scale_a = 1 (sa_i =
 *          scale_a[0] for every i) or M (sa_i = scale_a[i], one per row of A);
 * scale_b: DEVICE pointer to n_scale_b FP32 values, 1 or N (one per column
 *          of B, whatever the layout).
 * Both are read by the kernel at run time (stream-ordered like A and B), must
 * be 4-byte aligned, and are owned by the caller.  Other arguments, layouts
 * and checks as gemm_fp8; additionally a count other than those above ->
 * DGEMM_ERR_INVALID_DIM (checked with the dimensions), a NULL factor pointer
 * -> DGEMM_ERR_NULL_POINTER, a misaligned one -> DGEMM_ERR_MISALIGNED.
 */
int gemm_fp8_scaled(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
                    const uint8_t* B, int64_t ldb, float* C, int64_t ldc,
                    const float* scale_a, int64_t n_scale_a, const float* scale_b, int64_t n_scale_b,
                    int layout, void* stream);

/*
 * MXFP8: OCP E4M3 x E4M3 -> FP32 with one E8M0 scale per 32 consecutive k of
 * each row of A and of each column of B (the block scales of the OCP
 * Microscaling (MX) format, fed to the scale operands of the gfx950 MFMA;
 * the scaled successor that "FP8 GEMM Optimization on AMD RDNA 4", section
 * "What Changes at FP8", leaves for later work):
 *   C_ij = sum over blocks b of 2^(sa_ib - 127) * 2^(sb_jb - 127)
 *          * sum_{k = 32b}^{32b + 31} A_ik * B_kj
 * accumulated in FP32.  K must be a multiple of 32 (else
 * DGEMM_ERR_INVALID_DIM, checked with the dimensions).
 * scale_a: DEVICE pointer to M*ldsa bytes; sa_ib is scale_a[i*ldsa + b],
 *          ldsa >= K/32 (the kernels read whole 16-byte groups of a row).
 * scale_b: DEVICE pointer to N*ldsb bytes; sb_jb is scale_b[j*ldsb + b],
 *          ldsb >= K/32 (one row of scales per column j of B, in either
 *          layout).  With K == 0 neither is read (and may be NULL).
 * Both must be 16-byte aligned with ldsa, ldsb multiples of 16
 * (else DGEMM_ERR_MISALIGNED); an ld below K/32 -> DGEMM_ERR_INVALID_LD;
 * 256*ldsa or 256*ldsb at or above 2^31 -> DGEMM_ERR_UNSUPPORTED.  The scale
 * byte 255 (NaN in the format) is not supported: its result is unspecified.
 * Other arguments, layouts and checks as gemm_fp8.
 */
int gemm_mxfp8(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
               const uint8_t* B, int64_t ldb, float* C, int64_t ldc,
               const uint8_t* scale_a, int64_t ldsa, const uint8_t* scale_b, int64_t ldsb,
               int layout, void* stream);

/*
 * int8 x int8 -> FP32, FP16 or BF16 with scale factors (a linear layer
 * quantized symmetrically, one factor per token and per output channel):
 *   C_ij = (sum_k A_ik * B_kj) * (sa_i * sb_j)
 * The sum is exact in 32-bit integers (all 256 values of a byte are allowed),
 * converted to FP32 (one rounding), multiplied in FP32 as in gemm_fp8_scaled
 * and rounded once more to c_type (a dgemm_type; ldc counts elements of it).
 * K above 131071, where a sum could leave 32 bits, -> DGEMM_ERR_UNSUPPORTED.
 * A c_type that is none -> DGEMM_ERR_INVALID_TYPE (checked after the layout).
 * Factors and all other arguments and checks as gemm_fp8_scaled.
 */
int gemm_i8_scaled(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                   const int8_t* B, int64_t ldb, void* C, int64_t ldc, int c_type,
                   const float* scale_a, int64_t n_scale_a, const float* scale_b, int64_t n_scale_b,
                   int layout, void* stream);

/*
 * The int8 products of a mixture of experts: `rows` tokens sorted by group
 * (expert), group e's at rows offsets[e] .. offsets[e + 1] - 1 of C, each
 * multiplied with its group's weights.  All row-major:
 *   C[n*ldc + j] = (sum_k A[r*lda + k] * B[e*group_b + j*ldb + k]) * (sa_r * sb_ej)
 * with r = n, or r = row_index[n] where row_index is given (rows of A in
 * another order, each as often as wanted).  Sums, factors, rounding and
 * c_type as gemm_i8_scaled.
 * A: rows_a x K, lda >= K.  B: `groups` matrices of N x K, ldb >= K, group_b
 * elements apart (0: one matrix for every group).  C: rows x N, ldc >= N.
 * offsets: DEVICE pointer to groups + 1 values, ascending, within 0 .. rows
 * (read by the kernel; values outside are clamped).  Rows of C before the
 * first and behind the last group are left as they were, a group may be empty.
 * row_index: DEVICE pointer to `rows` values or NULL (then rows_a >= rows is
 * required); a row whose index is outside 0 .. rows_a - 1 counts as zeros
 * with the factor 0.
 * scale_a: n_scale_a = 1 or rows_a values; scale_b: n_scale_b = 1 or
 * groups*N values, scale_b[e*N + j].
 * A and B must be 16-byte aligned with lda, ldb and group_b multiples of 16,
 * A readable over rows_a*lda and B over (groups - 1)*group_b + N*ldb bytes;
 * offsets, row_index and the factors 4-byte, C element-aligned.
 * Checks, in this order: c_type; negative extents or group_b ->
 * DGEMM_ERR_INVALID_DIM; groups above 2^20, N or groups*N above 2^31 - 1 ->
 * DGEMM_ERR_UNSUPPORTED; factor counts, rows_a against rows ->
 * DGEMM_ERR_INVALID_DIM; rows == 0, N == 0 or groups == 0 -> DGEMM_OK with no
 * work; NULL pointers (A and B may be NULL if K == 0, A and scale_a if
 * rows_a == 0); leading dimensions; alignment; limits ->
 * DGEMM_ERR_UNSUPPORTED: K above 131071; 256*lda, 256*ldb, 4*rows, 4*rows_a,
 * 4*N or (with row_index) rows_a*lda at or above 2^31; more tiles than a launch
 * holds (never while N, rounded up to a multiple of 32, times rows + 15*groups
 * is below 2^32).
 */
int gemm_i8_grouped(int64_t groups, int64_t rows, int64_t N, int64_t K, const int8_t* A, int64_t rows_a, int64_t lda,
                    const int32_t* row_index, const int8_t* B, int64_t ldb, int64_t group_b, void* C, int64_t ldc,
                    int c_type, const float* scale_a, int64_t n_scale_a, const float* scale_b, int64_t n_scale_b,
                    const int32_t* offsets, void* stream);

/*
 * Rows to int8 with one factor per row, as the products above take them:
 *   scale[i] = fl(max_k |x_ik| / 127),  Q_ik = round(x_ik / scale[i])
 * with the quotient taken exactly and rounded to nearest-even, in -127 .. 127.
 * A row of zeros (or one so small that scale[i] rounds to 0) gets scale 0
 * and zeros; a row that holds an infinity or NaN gets that as its scale and
 * zeros, so that its products are NaN.  K == 0: scale 0.
 * X: rows x K row-major of type x_type, ldx >= K; Q: ldq >= K.  No alignment
 * beyond that of the elements; elements of Q past K in a row are left.
 * Checks: x_type; negative sizes -> DGEMM_ERR_INVALID_DIM; rows == 0 ->
 * DGEMM_OK; NULL pointers (X and Q may be NULL if K == 0); leading
 * dimensions; alignment; rows or K above 2^31 - 1 -> DGEMM_ERR_UNSUPPORTED.
 */
int quantize_i8(int64_t rows, int64_t K, const void* X, int64_t ldx, int x_type, int8_t* Q, int64_t ldq,
                float* scale, void* stream);

/*
 * Tokens sorted by expert and back (mixture of experts).  A pair (t, j) is
 * choice j of token t; `tokens` x k of them, numbered t*k + j.
 *
 * expert_sort: a stable counting sort of the pairs by ids[t*k + j] (64- or
 * 32-bit integers, id_bytes = 8 or 4).  A pair whose id is outside 0 ..
 * experts - 1 is dropped.  Writes
 *   offsets[e]      number of pairs of experts below e; experts + 1 values
 *   slot[t*k + j]   the pair's place in the sorted order, -1 if dropped
 *   pair[n]         the pair at place n, -1 behind the last one
 *   token[n]        its token, pair[n] / k, -1 behind the last one (may be
 *                   NULL: not wanted; the row_index of gemm_i8_grouped)
 * all DEVICE arrays of 32-bit integers.  The order within an expert is that
 * of the pairs.  workspace: expert_sort_workspace(tokens, k, experts) bytes
 * of DEVICE memory (0: may be NULL), 4-byte aligned, free again once the call's
 * work on the stream is done; too few bytes -> DGEMM_ERR_INVALID_DIM.
 * experts <= 1024 and tokens*k <= 2^31 - 1, else DGEMM_ERR_UNSUPPORTED (the
 * workspace query then returns -1).
 *
 * expert_dispatch: Y[slot[t*k + j]] = X[t] for every pair (rows of H values);
 * rows of Y that no slot names are left as they were.
 * expert_combine: O[t] = sum_j w[t*k + j] * Y[slot[t*k + j]], in the order of
 * j in FP32 and rounded once; weights == NULL: all 1, which is the gradient
 * of expert_dispatch.  A token with no pair gets zeros.
 * expert_combine_grad, the gradients of expert_combine:
 *   dY[slot[t*k + j]] = w[t*k + j] * dO[t],  dW[t*k + j] = dO[t] . Y[slot[t*k + j]]
 * (FP32, 0 for a dropped pair); rows of dY that no slot names are left.
 * weights == NULL: all 1; dW == NULL: not wanted (Y is then not read and may
 * be NULL); dY == NULL likewise.  With rows == 0 or H == 0 neither dO nor Y is
 * read (both may be NULL) and dW is zeros.
 * What a call writes must not overlap what it reads.
 * In all three a slot outside 0 .. rows - 1 (rows: of Y and dY) counts as
 * dropped; a slot must not occur twice where rows are written.  `type` is the
 * dgemm_type of every row matrix; pitches are in elements, at least H; no
 * alignment beyond that of the elements.  Every result is the same from run
 * to run.
 * Checks: type (id_bytes); negative sizes -> DGEMM_ERR_INVALID_DIM; nothing
 * to do -> DGEMM_OK; NULL pointers; leading dimensions; alignment; limits
 * (tokens*k, rows or H above 2^31 - 1 -> DGEMM_ERR_UNSUPPORTED).
 */
int64_t expert_sort_workspace(int64_t tokens, int64_t k, int64_t experts);
int expert_sort(int64_t tokens, int64_t k, int64_t experts, const void* ids, int id_bytes, int32_t* offsets,
                int32_t* slot, int32_t* pair, int32_t* token, void* workspace, int64_t workspace_bytes,
                void* stream);
int expert_dispatch(int64_t tokens, int64_t k, int64_t H, int type, const void* X, int64_t ldx, const int32_t* slot,
                    void* Y, int64_t rows, int64_t ldy, void* stream);
int expert_combine(int64_t tokens, int64_t k, int64_t H, int type, const void* Y, int64_t rows, int64_t ldy,
                   const int32_t* slot, const float* weights, void* O, int64_t ldo, void* stream);
int expert_combine_grad(int64_t tokens, int64_t k, int64_t H, int type, const void* dO, int64_t ldo, const void* Y,
                        int64_t rows, int64_t ldy, const int32_t* slot, const float* weights, void* dY, int64_t lddy,
                        float* dW, void* stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* gemm_strerror(int status);

/*
 * dgemm_last_hip_error: the hipError_t code behind the calling thread's most
 * recent DGEMM_ERR_HIP (0 if there was none); dgemm_hip_error_string: HIP's
 * static description of such a code.  For diagnostics only.
 */
int dgemm_last_hip_error(void);
const char* dgemm_hip_error_string(int code);

/*
 * Host-side introspection (no GPU work; used by host-only tests and reports).
 *
 * dgemm_tile_map: the block -> output-tile mapping the kernels use, for a grid
 * of tiles_p x tiles_q tiles, grouping `group` tiles along p ("FP16 GEMM
 * Optimization on AMD RDNA 3 and RDNA 4", section "Step 6: Block Scheduling
 * for Cache Reuse") after spreading consecutive tiles over the 8 XCDs.
 * Writes the tile coordinates of block `pid`; returns 0, or -1 for pid out of
 * range or non-positive sizes.
 *
 * dgemm_lds_bytes: LDS footprint (BM + BN) * (BK * elem + pad_bytes) * buffers
 * of a block tile, the sizing rule behind the LDS tables of "FP16 GEMM
 * Optimization on AMD RDNA 3 and RDNA 4" (Step 5, Table 9) and "FP8 GEMM
 * Optimization on AMD RDNA 4" (Configs 1-4).  Returns -1 for negative inputs.
 *
 * dgemm_kernel_config: writes a one-line description (kernel name, tile, wave
 * grid, LDS bytes, grid size) of the kernel a call with these arguments would
 * launch into buf (at most len bytes, NUL-terminated).  dtype: 0 f32, 1 f16,
 * 2 bf16, 3 fp8, 4 fp8 with scale factors, 5 MXFP8, 6 / 7 / 8 int8 with
 * FP32 / FP16 / BF16 results.  Returns 0, or a
 * dgemm_status for invalid arguments.
 *
 * dgemm_grouped_config: the same for gemm_i8_grouped with results of c_type
 * (a dgemm_type), with (gather != 0) or without a row_index.
 */
/*
 * dgemm_trace_clock (diagnostics, used to report the engine clock the GEMM
 * itself ran at): while `buf` is set, every launch of the four-wave kernels
 * made by later calls from the calling thread records, for each workgroup
 * w < n_workgroups, four 64-bit values at buf[4w .. 4w + 3]: the core clock
 * counter and the 100 MHz real-time counter when the workgroup started, and
 * both again when it finished.  Engine clock in Hz over the workgroup =
 * (buf[4w+2] - buf[4w]) / (buf[4w+3] - buf[4w+1]) * 1e8 (the counters of
 * different XCDs have different origins: compare stamps of one workgroup
 * only).  `buf` is a DEVICE pointer to 4*n_workgroups values owned by the
 * caller, written asynchronously on the call's stream; later launches
 * overwrite it.  NULL turns the trace off.  Only the main launch of a call
 * is traced (not the second launch of a split call); other kernels (FP32,
 * skinny, ragged K) ignore it.  Returns DGEMM_ERR_INVALID_DIM for n_workgroups < 0.
 */
int dgemm_trace_clock(unsigned long long* buf, int64_t n_workgroups);

int dgemm_tile_map(int64_t tiles_p, int64_t tiles_q, int64_t group, int64_t pid,
                   int64_t* tile_p, int64_t* tile_q);
int64_t dgemm_lds_bytes(int bm, int bn, int bk, int elem, int pad_bytes, int buffers);
int dgemm_kernel_config(int dtype, int layout, int64_t M, int64_t N, int64_t K, char* buf, int64_t len);
int dgemm_grouped_config(int c_type, int gather, int64_t groups, int64_t rows, int64_t N, int64_t K, char* buf,
                         int64_t len);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_H */
