/*
 * swizzled_gemm.h -- C ABI of libswizzled_gemm.so, an MI355X (gfx950) GEMM
 * whose operand tiles are staged in LDS under an XOR swizzle.
 *
 * Operation.  D = A*B (+C): a tiled matrix multiply-accumulate with 16-bit
 * inputs and fp32 accumulation -- the tensor-core operation D = A*B + C of
 * "Tensor Cores, layouts, and swizzling" (opening section), computed by the
 * sample tiled matmul of "Swizzling explained properly" (section "Sample
 * swizzled matmul") with tiles staged in on-chip memory under the swizzle
 * f(r, c) = (r, c XOR r) of that page (section "What does swizzling do?").
 * Passing C = NULL computes D = A*B, the "enable-input-d = false" form of
 * "06 Blackwell Tensor Core - tcgen05 MMA" (operand table); a non-NULL C is
 * the accumulate form D = A*B + C.
 *
 * Conventions shared by every entry point:
 *  - All pointers named A, B, C, D, SFA, SFB are DEVICE pointers of the
 *    current HIP device; m_offsets is a HOST pointer.  The caller owns every
 *    buffer; the library never allocates, frees or synchronises.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  A
 *    call enqueues its kernels on that stream and returns at once; results
 *    are visible after the stream is synchronised.
 *  - Matrices are dense and row-major with no padding: a "K-major" operand
 *    is stored [rows][K] (K contiguous), an "MN-major" one [K][rows].
 *    A: K-major [M][K] or MN-major [K][M].  B: K-major [N][K] (B transposed)
 *    or MN-major [K][N].  C and D: [M][N].
 *  - Every pointer must be 16-byte aligned and every row pitch (contiguous
 *    extent x element size) a multiple of 16 bytes, the 16-byte atom rule of
 *    both swizzle pages ("LBO, SBO and SWZ", section 1; "Swizzling explained
 *    properly", section "What about base?") and of the TMA stride rule in
 *    "Tensor Cores, layouts, and swizzling".  Violations return
 *    SG_ERR_ALIGN.  M, N and K themselves may be ragged (not multiples of
 *    the tile); M = 0 or N = 0 is a no-op; K = 0 gives D = C (or 0).
 *  - Return value: SG_OK (0) or a negative SG_ERR_* code; on error nothing is
 *    enqueued and gemm_last_error() describes the failure (thread-local).
 */
#ifndef SWIZZLED_GEMM_H
#define SWIZZLED_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define SG_OK 0
#define SG_ERR_NULL (-1)   /* a required pointer is NULL */
#define SG_ERR_ALIGN (-2)  /* pointer not 16-byte aligned, or row pitch not a multiple of 16 B */
#define SG_ERR_SHAPE (-3)  /* negative size, or beyond the supported extent */
#define SG_ERR_DTYPE (-4)  /* unsupported element type combination */
#define SG_ERR_MAJOR (-5)  /* majorness not SG_K_MAJOR / SG_MN_MAJOR */
#define SG_ERR_GROUPS (-6) /* bad group count or offsets */
#define SG_ERR_HIP (-7)    /* a HIP call failed; see gemm_last_error() */

/* Element types. */
#define SG_NONE 0
#define SG_F16 1  /* IEEE binary16 */
#define SG_BF16 2 /* bfloat16 */
#define SG_F32 3  /* IEEE binary32 */
#define SG_E4M3 4 /* OCP FP8 E4M3 (bias 7, max 448, no infinity) */
#define SG_E8M0 5 /* OCP E8M0 scale, value 2^(e-127) */
#define SG_E2M1 6 /* OCP FP4 E2M1 (bias 1, max 6, two elements per byte) */
#define SG_E2M3 7 /* OCP FP6 E2M3 (bias 1, max 7.5, no infinity or NaN) */
#define SG_E3M2 8 /* OCP FP6 E3M2 (bias 3, max 28, no infinity or NaN) */

#define SG_I32 9  /* 32-bit and 64-bit integers (targets of the cross entropy) */
#define SG_I64 10

/* Layouts of the e8m0 scale arrays of the block-scaled GEMMs. */
#define SG_SF_ROWS 0   /* [rows][K/32]: row r's byte b at r * (K/32) + b */
#define SG_SF_BLOCKS 1 /* 1 KiB blocks of 64 rows x 16 bytes, see mx_scales_to_blocks */

/* Operand majorness. */
#define SG_K_MAJOR 0  /* K is the contiguous dimension */
#define SG_MN_MAJOR 1 /* M (for A) or N (for B) is the contiguous dimension */

/* Largest group count grouped_gemm_run accepts. */
#define SG_MAX_GROUPS 256

/*
 * gemm_run -- D = A*B (+C), fp32 accumulation.
 *   M, N, K    problem sizes (>= 0).
 *   A          ab_dtype, K-major [M][K] or MN-major [K][M] (a_major).
 *   B          ab_dtype, K-major [N][K] or MN-major [K][N] (b_major).
 *   ab_dtype   SG_F16 or SG_BF16.
 *   C          NULL (treated as zero) or [M][N] of c_dtype (SG_F32, SG_BF16,
 *              SG_F16).  C may equal D (in-place accumulate) when c_dtype ==
 *              d_dtype; any other overlap of C or D with inputs is undefined.
 *   D          [M][N] of d_dtype: SG_F32, SG_BF16 or SG_F16 (the fp32
 *              accumulator is rounded to nearest even).
 * Errors: SG_ERR_NULL (A, B or D NULL with M, N > 0 -- A/B may be NULL when
 * K = 0), SG_ERR_ALIGN, SG_ERR_SHAPE (a size < 0, or a per-tile operand
 * extent of 2^31 bytes or more), SG_ERR_DTYPE, SG_ERR_MAJOR, SG_ERR_HIP.
 */
int gemm_run(int64_t M, int64_t N, int64_t K, const void* A, int a_major,
             const void* B, int b_major, int ab_dtype, const void* C,
             int c_dtype, void* D, int d_dtype, void* stream);

/*
 * gemm_strided_run -- D = alpha * A*B + beta * C with leading dimensions,
 * fp32 accumulation.  Operands are addressed as "Tensor Cores, layouts, and
 * swizzling" describes its tensor-memory tile copies (section on the Tensor
 * Memory Accelerator): by dimensions and row strides that are multiples of
 * 16 bytes, with elements past the edges read as zero.
 *   alpha, beta  fp32 scalars.  D = round(alpha * acc + beta * C) with acc the
 *                fp32 sum over K; alpha = beta = 1 gives gemm_run's result
 *                bit for bit.  alpha == 0: A and B are not read (D = beta*C);
 *                beta == 0 or C == NULL: C is not read.
 *   A   K-major: element (m, k) at A[m*lda + k], lda >= K;
 *       MN-major: element (m, k) at A[k*lda + m], lda >= M.
 *   B   K-major: element (k, n) at B[n*ldb + k], ldb >= K;
 *       MN-major: element (k, n) at B[k*ldb + n], ldb >= N.
 *   C   element (m, n) at C[m*ldc + n], ldc >= N; D at D[m*ldd + n], ldd >= N.
 *   Leading dimensions are in elements; every row pitch (ld * element size)
 *   must be a multiple of 16 bytes and every pointer 16-byte aligned.  C may
 *   equal D when c_dtype == d_dtype and ldc == ldd.  The other arguments and
 *   the errors are gemm_run's, plus SG_ERR_SHAPE for a leading dimension below
 *   its minimum, an N that is not a multiple of 4 (the epilogue writes D
 *   four columns at a time; gemm_run's packed rows already imply it), or a
 *   K that is not a multiple of 8 while A or B is K-major (the loaders move
 *   whole 16-byte chunks of a row, so the elements past K inside the last
 *   chunk would be read from the row's padding; gemm_run's packed K-major
 *   rows already imply K % 8 == 0 through the 16-byte pitch rule).
 */
int gemm_strided_run(int64_t M, int64_t N, int64_t K, float alpha, const void* A,
                     int64_t lda, int a_major, const void* B, int64_t ldb, int b_major,
                     int ab_dtype, float beta, const void* C, int64_t ldc, int c_dtype,
                     void* D, int64_t ldd, int d_dtype, void* stream);

/*
 * grouped_gemm_run -- for each group g in [0, G):
 *   D[off_g : off_{g+1}] = A[off_g : off_{g+1}] * B_g,
 * the grouped GEMM named in "LBO, SBO and SWZ for a tcgen05 tile"
 * (introduction); the pages give no further definition, so each group is the
 * plain dense GEMM on its row range.  Groups share N and K.
 *   G          number of groups, 1..SG_MAX_GROUPS.
 *   m_offsets  HOST array of G+1 row offsets: m_offsets[0] = 0, non-
 *              decreasing; group g owns rows [m_offsets[g], m_offsets[g+1]).
 *              Empty groups are allowed.  Read during the call only.
 *   A          ab_dtype, K-major [m_offsets[G]][K].
 *   B          ab_dtype, G contiguous blocks, each K-major [N][K]
 *              (b_major must be SG_K_MAJOR).
 *   D          [m_offsets[G]][N] of d_dtype (SG_F32, SG_BF16, SG_F16).
 * Errors: as gemm_run, plus SG_ERR_GROUPS (G out of range, m_offsets[0] != 0
 * or decreasing offsets).
 */
int grouped_gemm_run(int G, const int64_t* m_offsets, int64_t N, int64_t K,
                     const void* A, int a_major, const void* B, int b_major,
                     int ab_dtype, void* D, int d_dtype, void* stream);

/*
 * mx_gemm_run -- block-scaled (MXFP8) GEMM:
 *   D[m][n] = sum_blk 2^(SFA[m][blk]-127) * 2^(SFB[n][blk]-127)
 *             * sum_{k in blk} A[m][k] * B[n][k],
 * with 32-element K blocks: output (m, n) uses SFA[m, sfk] for A and
 * SFB[n, sfk] for B ("06 Blackwell Tensor Core - tcgen05 MMA", section
 * "Block-Scaled MMA").  fp32 accumulation.
 *   A    e4m3 K-major [M][K];  SFA  e8m0 [M][K/32].
 *   B    e4m3 K-major [N][K];  SFB  e8m0 [N][K/32].
 *   D    [M][N] of d_dtype (SG_F32 or SG_BF16).
 *   K    must be a multiple of 128 (four scale blocks per 16-byte row chunk
 *        pair); M and N may be ragged.
 * Scale byte 255 (NaN) propagates NaN.
 * Errors: SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE (K % 128 != 0 or extents),
 * SG_ERR_DTYPE, SG_ERR_HIP.
 */
int mx_gemm_run(int64_t M, int64_t N, int64_t K, const void* A,
                const void* SFA, const void* B, const void* SFB, void* D,
                int d_dtype, void* stream);

/*
 * mxfp4_gemm_run -- the block-scaled GEMM of mx_gemm_run with OCP FP4 E2M1
 * elements (MXFP4): 1 sign, 2 exponent bits (bias 1), 1 fraction bit,
 * values +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}; two elements per byte, element 2i
 * in the low nibble of byte i.  The scale rule is mx_gemm_run's ("06
 * Blackwell Tensor Core - tcgen05 MMA", section "Block-Scaled MMA"); the
 * 32-element block and e8m0 scales as there.  fp32 accumulation.
 *   A    e2m1 K-major [M][K/2] bytes;  SFA  e8m0 [M][K/32].
 *   B    e2m1 K-major [N][K/2] bytes;  SFB  e8m0 [N][K/32].
 *   D    [M][N] of d_dtype (SG_F32 or SG_BF16).
 *   K    must be a multiple of 256 (one 128-byte row chunk per K tile);
 *        M and N may be ragged.
 * Errors: SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE (K % 256 != 0 or
 * extents), SG_ERR_DTYPE, SG_ERR_HIP.
 */
int mxfp4_gemm_run(int64_t M, int64_t N, int64_t K, const void* A,
                   const void* SFA, const void* B, const void* SFB, void* D,
                   int d_dtype, void* stream);

/*
 * mxfp6_gemm_run -- the block-scaled GEMM of mx_gemm_run with OCP FP6
 * elements (MXFP6): fmt SG_E2M3 (1 sign, 2 exponent bits with bias 1, 3
 * fraction bits; largest magnitude 7.5, smallest 0.125) or SG_E3M2 (1 sign,
 * 3 exponent bits with bias 3, 2 fraction bits; largest 28, smallest
 * 0.0625); neither has infinity or NaN.  A row is a 6-bit stream: element k
 * at bits [6k, 6k+6) of the row's bytes, little endian (four elements in
 * three bytes).  The scale rule is mx_gemm_run's ("06 Blackwell Tensor Core
 * - tcgen05 MMA", section "Block-Scaled MMA"); the 32-element block and
 * e8m0 scales as there.  fp32 accumulation.
 *   A    fp6 K-major [M][3K/4] bytes;  SFA  e8m0 [M][K/32].
 *   B    fp6 K-major [N][3K/4] bytes;  SFB  e8m0 [N][K/32].
 *   D    [M][N] of d_dtype (SG_F32 or SG_BF16).
 *   K    must be a multiple of 128 (96 bytes of every row per K tile);
 *        M and N may be ragged.  No read leaves the M*3K/4 bytes of A, the
 *        N*3K/4 bytes of B or the scale arrays.
 * Errors: SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE (K % 128 != 0 or
 * extents), SG_ERR_DTYPE (fmt or d_dtype), SG_ERR_HIP.
 */
int mxfp6_gemm_run(int fmt, int64_t M, int64_t N, int64_t K, const void* A,
                   const void* SFA, const void* B, const void* SFB, void* D,
                   int d_dtype, void* stream);

/*
 * mx_scales_blocks_bytes -- the size in bytes of an e8m0 scale array of
 * `rows` rows and K/32 blocks in the SG_SF_BLOCKS layout (host-side, no GPU
 * needed): ceil(rows/64) * ceil(K/512) * 1024.  Returns SG_ERR_SHAPE
 * (negative) for rows < 0, K < 0 or K not a multiple of 32.
 */
int64_t mx_scales_blocks_bytes(int64_t rows, int64_t K);

/*
 * mx_scales_to_blocks -- rearranges e8m0 scales SF [rows][K/32] (SG_SF_ROWS,
 * the layout of "06 Blackwell Tensor Core - tcgen05 MMA", section
 * "Block-Scaled MMA": SFA(M, SFK), SFB(N, SFK)) into `out`, SG_SF_BLOCKS:
 * row r's scale byte b (32-element block b of K) goes to byte
 *   ((r / 64) * G + b / 16) * 1024 + (r % 64) * 16 + 8 * (b % 2) + (b % 16) / 2,
 * G = ceil(K/512): the 16 bytes of one group of 16 blocks for 64 consecutive
 * rows are one contiguous KiB, and a row's 16 bytes hold the group's 8 even
 * blocks, then its 8 odd ones.  Bytes for rows past `rows` (up to the next
 * multiple of 64) and blocks past K/32 are written as zero.  The scaled
 * MFMA's two lane halves scale the even and the odd blocks of a 64-wide K
 * step, so the block-scaled GEMMs load a row's group as one 8-byte half per
 * lane, with no rearranging after the load; from SG_SF_BLOCKS a wave's load
 * of 32 rows covers 4 cache lines instead of the 32 (one per row) of
 * SG_SF_ROWS.  SF: DEVICE memory, 4-byte aligned; out: DEVICE memory of
 * mx_scales_blocks_bytes(rows, K) bytes, 16-byte aligned (caller-owned).
 * Asynchronous on `stream` (a hipStream_t, NULL for the default stream).
 * Errors: SG_ERR_SHAPE (K not a multiple of 128, negative sizes, 2^31 or
 * more blocks of 64 rows, K past 2^29), SG_ERR_NULL, SG_ERR_ALIGN,
 * SG_ERR_HIP.
 */
int mx_scales_to_blocks(const void* SF, int64_t rows, int64_t K, void* out, void* stream);

/*
 * mx_gemm_blocks_run -- the block-scaled GEMM of mx_gemm_run (fmt SG_E4M3),
 * mxfp4_gemm_run (SG_E2M1) or mxfp6_gemm_run (SG_E2M3, SG_E3M2), with SFA
 * and SFB in the SG_SF_BLOCKS layout (mx_scales_to_blocks), 16-byte aligned.
 * The layout's padding (rows past M or N in the last 64 rows, blocks past
 * K/32 in the last group) is never used and may hold anything.  Every other
 * argument, requirement and result is that entry point's; the D it computes
 * is bit-identical.  Errors: theirs, and SG_ERR_DTYPE for
 * another fmt.
 */
int mx_gemm_blocks_run(int fmt, int64_t M, int64_t N, int64_t K, const void* A,
                       const void* SFA, const void* B, const void* SFB, void* D,
                       int d_dtype, void* stream);

/*
 * gemm_layout_run -- the bf16 GEMM with A and B K-major (and optional C) on
 * 256x256 tiles of the 8-wave ping-pong kernel with 32x32x16 MFMAs (the
 * 16x16x32 variant of gemm_run reads fragments in another lane pattern), with
 * a chosen LDS operand layout: the layout experiment of "Swizzling explained
 * properly" (sections "Why swizzle?" and "Results") on gfx950.
 *   swz_units  16: the library's layout (the 16-byte unit index XORed with
 *              the 256-byte bank-line index: ds_read_b128 reads 64 banks of
 *              4 bytes); 8: the same XOR over 128-byte lines; 0: no swizzle.
 * Every layout gives the same D; only LDS bank conflicts and speed differ.
 * The other arguments are gemm_run's (ab_dtype = SG_BF16, both operands
 * SG_K_MAJOR).  Errors: as gemm_run, and SG_ERR_SHAPE for swz_units not in
 * {0, 8, 16}.
 */
int gemm_layout_run(int swz_units, int64_t M, int64_t N, int64_t K, const void* A,
                    const void* B, const void* C, int c_dtype, void* D, int d_dtype,
                    void* stream);

/*
 * gemm_layout_io_run -- the input/output half of the layout experiment of
 * "Swizzling explained properly" (section "Results": swizzling the input
 * tiles against swizzling only the output tile), on gemm_run's own 256x256
 * kernel (8 waves, 16x16x32 MFMAs) for bf16 K-major A and B and a 16-bit D,
 * which that kernel stages in LDS (with a 16-bit C brought in by its last
 * loads).  operand_swz: 16 = the library's operand layout (16-byte units
 * XORed with the 256-byte bank-line index), 0 = no swizzle.  output_swz: 1 =
 * the C and D staging areas use their XOR keys (the library), 0 = logical
 * chunk order.  Every combination gives the same D bit for bit; only LDS
 * bank conflicts and speed differ.  The other arguments are gemm_run's, with
 * C NULL or 16-bit and d_dtype SG_BF16 or SG_F16.  Errors: as gemm_run, and
 * SG_ERR_SHAPE for another operand_swz or output_swz, SG_ERR_DTYPE for a
 * 32-bit C or D.
 */
int gemm_layout_io_run(int operand_swz, int output_swz, int64_t M, int64_t N, int64_t K,
                       const void* A, const void* B, const void* C, int c_dtype, void* D,
                       int d_dtype, void* stream);

/*
 * gemm_layout128_run -- gemm_layout_run on 128x128 tiles of the 4-wave
 * kernel (the 32x32x16 MFMA), where a padded layout also fits in LDS: the
 * padding alternative to swizzling weighed in "Swizzling explained properly"
 * (sections "Why swizzle?" and "Results").
 *   layout  16, 8 or 0 as gemm_layout_run's swz_units, or SG_LAYOUT_PAD16:
 *           no XOR, each 128-byte LDS row followed by 16 bytes of padding
 *           (loaded through registers, since padded rows do not tile the
 *           direct-to-LDS path's 1 KiB regions).
 * Every layout gives the same D.  Errors: as gemm_layout_run, SG_ERR_SHAPE
 * for another layout value.
 */
#define SG_LAYOUT_PAD16 (-1)
int gemm_layout128_run(int layout, int64_t M, int64_t N, int64_t K, const void* A,
                       const void* B, const void* C, int c_dtype, void* D, int d_dtype,
                       void* stream);

/*
 * i8_gemm_run -- the product of 8-bit integer matrices with one scale per row
 * of A (token) and per row of B (output channel):
 *   D[m][n] = SA[m] * SB[n] * sum_k A[m][k] * B[n][k].
 * The sum is exact (32-bit integers); it is converted to fp32 and multiplied
 * by SA[m], then by SB[n], one rounding each, then rounded to d_dtype.
 *   A   int8 [M][lda], K codes a row;  SA  fp32 [M].
 *   B   int8 [N][ldb], K codes a row;  SB  fp32 [N].
 *   D   [M][ldd] of d_dtype (SG_F32, SG_BF16, SG_F16), N values a row.  N and
 *       ldd may be any; D is aligned to its elements (rows that are 16-byte
 *       aligned are written fastest).
 *   K   a multiple of 16 (i8_quant_run pads with zeros), at most 131056, for
 *       which the sum cannot overflow.  K = 0 gives D = 0.
 *   lda, ldb are multiples of 16, A and B 16-byte aligned.
 * Codes are any of -128 .. 127.  A NaN scale makes its row or column NaN.
 * Here and in the calls below no output may overlap an input or another output.
 * Errors: SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE (also a leading dimension
 * below its minimum, a tile's panel of 2^31 bytes or more, or 2^23 tiles or
 * more: the tiles are 16 to 64 columns wide for up to 64 rows, 64 x 64 to 256 x
 * 256 beyond), SG_ERR_DTYPE, SG_ERR_HIP.
 */
int i8_gemm_run(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* SA,
                const void* B, int64_t ldb, const float* SB, void* D, int64_t ldd, int d_dtype,
                void* stream);

/*
 * i8_grouped_gemm_run -- i8_gemm_run for G experts, whose row ranges are in
 * DEVICE memory (moe_plan_run writes them), so that no copy to the host stands
 * between routing and the product:
 *   D[r] = the 8-bit product of A's row a(r) with B_g, for offsets[g] <= r <
 *   offsets[g+1], a(r) = rows[r], or r without `rows`.
 *   R        rows of D.  Rows at and behind offsets[G] are left as they were.
 *   offsets  DEVICE int32 [G+1], not decreasing, within [0, R].  The device
 *            clamps them: offsets that break this rule give undefined values
 *            in D, and no access outside the buffers.
 *   rows     DEVICE int32 [R], or NULL.  An index outside [0, a_rows) makes
 *            its row of D zero.
 *   A        int8 [a_rows][lda] (a_rows >= R without `rows`);  SA [a_rows].
 *   B        int8, G blocks [N][K], packed;  SB  fp32 [G][N].
 * G is 1..SG_MAX_GROUPS.  The kernel is chosen from R / G, not from the
 * offsets.  Everything else is i8_gemm_run's.  Errors: its, SG_ERR_GROUPS (G),
 * and SG_ERR_SHAPE for a gathered A of 2^31 bytes or more.
 */
int i8_grouped_gemm_run(int G, int64_t R, int64_t N, int64_t K, const int32_t* offsets,
                        const void* A, int64_t lda, int64_t a_rows, const int32_t* rows,
                        const float* SA, const void* B, const float* SB, void* D, int64_t ldd,
                        int d_dtype, void* stream);

/*
 * i8_quant_run -- rows of X to 8-bit codes with one scale per row, for the
 * operands of the 8-bit products (activations at every call, weights once):
 *   a = max_k |X[r][k]|,  S[r] = max(a, 2^-100) / 127,
 *   Q[r][k] = round(X[r][k] * (127 / max(a, 2^-100))),
 * each step rounded once to fp32 and the codes to nearest even: |Q| <= 127.  A
 * row that holds an infinity or a NaN has S[r] = NaN and codes 0, so that a
 * product with it is NaN.
 *   X   [R][ldx] of x_dtype (SG_F32, SG_BF16, SG_F16), K values a row; any
 *       ldx >= K and any alignment of its elements (16-byte aligned rows of a
 *       multiple of 8 values are read fastest).
 *   Q   int8 [R][ldq], 16-byte aligned, ldq a multiple of 16.  Columns K up to
 *       the next multiple of 16 are written as zero; those behind are left.
 *   S   fp32 [R].
 * K = 0 writes S only.  Errors: SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE,
 * SG_ERR_DTYPE, SG_ERR_HIP.
 */
int i8_quant_run(int64_t R, int64_t K, const void* X, int64_t ldx, int x_dtype, void* Q,
                 int64_t ldq, float* S, void* stream);

/* Expert routing. */
#define SG_SCORE_SOFTMAX 0
#define SG_SCORE_SIGMOID 1
#define SG_GROUP_MAX 0  /* a group scores its largest key */
#define SG_GROUP_TOP2 1 /* the sum of its two largest keys */
#define SG_MAX_TOP_K 32
#define SG_MAX_ROUTE_GROUPS 32

/*
 * moe_route_run -- chooses top_k of E experts for each of T tokens and their
 * weights.
 *   scores   s[e] = softmax over the token's logits, or sigmoid of each.  A
 *            logit of -inf or NaN is masked: it scores 0, takes no part in the
 *            softmax and is never chosen.  A logit of +inf counts as the largest
 *            finite fp32 value (two of them, or one and that value, are equal).
 *   keys     s[e] + bias[e] evaluated in 64 bits.  Without a bias (and without
 *            SG_GROUP_TOP2 groups) the experts are ordered by their logits,
 *            which is the exact order of their scores.  A key of -inf or NaN
 *            masks the expert too.
 *   groups   with n_groups > 1 (dividing E) the experts form n_groups equal
 *            runs; only those of the top_groups best groups can be chosen.
 *   ids      int32 [T][top_k]: the experts by falling key; among equal keys
 *            (and equal groups) the lowest index comes first.  -1 where no
 *            expert is left (a fully masked token has -1 throughout).
 *   weights  fp32 [T][top_k]: s[id] (without the bias), with renorm divided by
 *            their sum (by 2^-126 where the sum is smaller), times scale; 0
 *            where the id is -1.
 *   logits   [T][ldl] of dtype (SG_F32, SG_BF16, SG_F16), any ldl >= E;
 *   bias     fp32 [E] or NULL.
 * E is 1..SG_MAX_GROUPS, top_k 1..SG_MAX_TOP_K and at most the experts that
 * can be chosen, n_groups at most SG_MAX_ROUTE_GROUPS.  Errors: SG_ERR_NULL,
 * SG_ERR_ALIGN, SG_ERR_SHAPE, SG_ERR_DTYPE, SG_ERR_GROUPS, SG_ERR_HIP.
 */
int moe_route_run(int64_t T, int E, int top_k, const void* logits, int64_t ldl, int dtype,
                  const float* bias, int score, int n_groups, int top_groups, int group_score,
                  int renorm, float scale, float* weights, int32_t* ids, void* stream);

/*
 * moe_route_backward_run -- the gradient of the logits from the gradient of
 * moe_route_run's weights, the choice of experts held fixed.
 *   dweights  fp32 [T][top_k];  ids  int32 [T][top_k] as moe_route_run wrote
 *             them (ids outside [0, E) carry no gradient; an id that appears
 *             twice counts twice).
 *   dlogits   [T][lddl] of the logits' type, E values a row: all written, zero
 *             for masked logits.
 * score, renorm and scale are the forward call's.  Errors as there.
 */
int moe_route_backward_run(int64_t T, int E, int top_k, const float* dweights, const void* logits,
                           int64_t ldl, int dtype, const int32_t* ids, int score, int renorm,
                           float scale, void* dlogits, int64_t lddl, void* stream);

/*
 * moe_plan_run -- sorts the T * top_k (token, expert) pairs by expert, stably
 * and without a copy to the host:
 *   offsets  int32 [E+1]: expert e's pairs are the sorted rows [offsets[e],
 *            offsets[e+1]); offsets[E] is the number of valid pairs.
 *   rows     int32 [T*top_k]: the token of each sorted row (the row index that
 *            i8_grouped_gemm_run gathers by); -1 behind offsets[E].
 *   slots    int32 [T][top_k]: the sorted row of each pair, -1 where its id is
 *            outside [0, E).
 *   ids      int32 [T][top_k].
 *   workspace  DEVICE, moe_plan_workspace_bytes(T * top_k, E) bytes, 4-byte
 *            aligned (0 bytes up to 16384 pairs: may be NULL).  It holds nothing
 *            between calls; calls that may run at the same time need their own.
 * T = 0 writes offsets only.  Errors: SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE,
 * SG_ERR_HIP.
 */
int moe_plan_run(int64_t T, int E, int top_k, const int32_t* ids, int32_t* offsets, int32_t* rows,
                 int32_t* slots, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that moe_plan_run needs for P pairs (host only), or
 * SG_ERR_SHAPE (negative). */
int64_t moe_plan_workspace_bytes(int64_t P, int E);

/*
 * moe_balance_run -- how evenly a router spreads its tokens over its experts
 * (the auxiliary loss of its training), and the tokens of each expert:
 *   share[t][e] = s[t][e] / sum_e s[t][e],  s the scores of moe_route_run (a
 *                 masked logit scores 0; the sum is at least 2^-126),
 *   counts[e]   = the pairs of ids that name e,
 *   loss        = sum_e (E * counts[e] / sum counts) * (1/n) sum_t share[t][e],
 * n the tokens with a logit that is not masked.  1 for an even load, E where all
 * goes to one expert; 0 without a token or a pair.
 *   logits   [T][ldl] of dtype (SG_F32, SG_BF16, SG_F16), any ldl >= E.
 *   ids      int32 [T][top_k] as moe_route_run writes them; those outside
 *            [0, E) are not counted.
 *   loss     fp32 [1];  counts  int32 [E];  tokens  int32 [1]: n.
 *   workspace  DEVICE, moe_balance_workspace_bytes(T, E) bytes, 16-byte aligned
 *            (0 bytes up to 256 tokens: may be NULL).  It holds nothing between
 *            calls; calls that may run at the same time need their own.
 * Sums are added in a fixed order.  T = 0 writes zeros.  E is 1..SG_MAX_GROUPS,
 * top_k 1..min(E, SG_MAX_TOP_K), T * top_k below 2^31.  Errors: SG_ERR_NULL,
 * SG_ERR_ALIGN, SG_ERR_SHAPE, SG_ERR_DTYPE, SG_ERR_HIP.
 */
int moe_balance_run(int64_t T, int E, int top_k, const void* logits, int64_t ldl, int dtype,
                    const int32_t* ids, int score, float* loss, int32_t* counts,
                    int32_t* tokens, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that moe_balance_run needs (host only), or SG_ERR_SHAPE. */
int64_t moe_balance_workspace_bytes(int64_t T, int E);

/*
 * moe_balance_backward_run -- the gradient of the logits from that of
 * moe_balance_run's loss, the counts held fixed.
 *   dloss    DEVICE fp32 [1];  counts, tokens  as moe_balance_run wrote them
 *            (counts added up over several calls, with their tokens, give the
 *            gradient of the loss over all of them).
 *   dlogits  [T][lddl] of the logits' type, E values a row: all written, zero
 *            for masked logits.
 * score is the forward call's.  Errors as there.
 */
int moe_balance_backward_run(int64_t T, int E, const float* dloss, const void* logits,
                             int64_t ldl, int dtype, const int32_t* counts,
                             const int32_t* tokens, int score, void* dlogits, int64_t lddl,
                             void* stream);

/*
 * gemm_xent_run -- softmax cross entropy over a vocabulary of N words for M
 * tokens, without keeping the logits z = alpha * A*B:
 *   z[m][n] = alpha * sum_k A[m][k] * B[n][k]  (fp32 accumulation),
 *   lse[m]  = log sum_n exp z[m][n],
 *   loss[m] = lse[m] - z[m][targets[m]], or 0 where targets[m] lies outside
 *             [0, N) (a token without a target: padding, a prompt).
 * A token with a logit of NaN or +inf has lse = loss = NaN (0 without a
 * target); logits of -inf count as probability 0.  N = 0 gives lse = -inf.
 *   A        ab_dtype (SG_F16, SG_BF16) [M][lda], K values a row.
 *   B        ab_dtype [N][ldb], K values a row: a word each.
 *   targets  [M] of target_dtype (SG_I32, SG_I64).
 *   loss, lse  fp32 [M].
 *   K        a multiple of 8; lda, ldb multiples of 8 below 2^22; A and B
 *            16-byte aligned.  N and M may be any.
 *   workspace  DEVICE, gemm_xent_workspace_bytes(M, N, K) bytes, 16-byte
 *            aligned: two floats for each token and column tile (8192 tokens,
 *            131072 words: 34 MB, where the logits would be 4.3 GB).  It holds
 *            nothing between calls; calls that may run at the same time need
 *            their own.
 * The result depends on nothing but the arguments (no atomics).  Errors:
 * SG_ERR_NULL, SG_ERR_ALIGN (also an output or the workspace that overlaps
 * another argument), SG_ERR_SHAPE (also 2^23 tiles or more), SG_ERR_DTYPE,
 * SG_ERR_HIP.
 */
int gemm_xent_run(int64_t M, int64_t N, int64_t K, float alpha, const void* A, int64_t lda,
                  const void* B, int64_t ldb, int ab_dtype, const void* targets, int target_dtype,
                  float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                  void* stream);

/* Bytes of workspace that gemm_xent_run needs (host only), or SG_ERR_SHAPE. */
int64_t gemm_xent_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * gemm_xent_backward_run -- the gradients of A and B from those of
 * gemm_xent_run's loss and lse:
 *   g[m][n] = alpha * ((dl[m] + dlse[m]) * exp(z[m][n] - lse[m])
 *                      - (n == targets[m] ? dl[m] : 0)),
 *   dA = g*B,  dB = g^T*A,
 * dl = dloss, or 0 for a token without a target; g is 0 for a token whose dl and
 * dlse are 0, whatever its A holds (its row of dA is 0; dB adds 0 * A, so that A
 * has to be finite there).  The logits are computed again, a run of words at a
 * time.  g is rounded to ab_dtype, up to 64 tokens to twice as many bits; the sums
 * are fp32, the results are rounded once.  For that the terms of both types are
 * scaled by a power of two over the largest |dl| (of those that, with dlse, are
 * numbers): that weight and its equals become the power of two, the others take
 * one rounding of fp32 each, and in fp16 what is below 2^-38 of the largest is
 * lost.  Error over the norm of dA and dB, beyond 64 tokens: 0.0017 to 0.0019 in
 * bf16 with equal weights, 0.0023 with random ones (0.00166 is the rounding of
 * the results), 0.00025 and 0.00029 in fp16 (0.00021).
 *   dloss    fp32 [M];  dlse  fp32 [M] or NULL (zero).
 *   lse      fp32 [M] as gemm_xent_run wrote it for the same A, B and alpha.
 *   dA       ab_dtype [M][ldda], or NULL: not wanted;  dB  ab_dtype [N][lddb],
 *            or NULL.  16-byte aligned, row pitches too.  Both are overwritten
 *            whole (zeros where M or N is 0).  Neither may overlap an input, so
 *            neither gradient replaces its operand (SG_ERR_ALIGN); rows of one
 *            pitch may lie side by side.
 *   workspace  DEVICE, gemm_xent_backward_workspace_bytes(M, N, K, ldb) bytes,
 *            16-byte aligned; as above.  Beside 16 bytes a token it holds g of
 *            one run, 2 * M bytes a word (4 * M up to 64 tokens), at most 512 MB
 *            or 256 words; with several runs 4 * M * K bytes; where dA has few
 *            tiles 4 * M * K for each of up to 32 shares of the words, so many
 *            that they fill the CUs.  Up to 64 tokens there is always a share,
 *            each is 8 * M * K, and a second copy of A takes 4 * M * K.
 * M is below 2^22, and with dB the rows of A span less than 2^31 bytes.  The
 * other arguments and the errors are gemm_xent_run's.
 */
int gemm_xent_backward_run(int64_t M, int64_t N, int64_t K, float alpha, const float* dloss,
                           const float* dlse, const void* A, int64_t lda, const void* B,
                           int64_t ldb, int ab_dtype, const void* targets, int target_dtype,
                           const float* lse, void* dA, int64_t ldda, void* dB, int64_t lddb,
                           void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that gemm_xent_backward_run needs (host only), or
 * SG_ERR_SHAPE. */
int64_t gemm_xent_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t ldb);

/* Thread-local text of the last failing call ("" if none).  Never NULL. */
const char* gemm_last_error(void);

/* Library version and build description.  Never NULL. */
const char* gemm_version(void);

/*
 * gemm_lds_layout -- the LDS byte map the kernels use for a K-major operand
 * tile (host-side, no GPU needed).  Writes out[r * (row_bytes/16) + c] = the
 * byte offset within one LDS stage of logical 16-byte chunk c of tile row r,
 * for r < rows.  row_bytes is 64, 128 or 256; rows a positive multiple of 8.
 * The map is the XOR swizzle of "Swizzling explained properly" applied to
 * (bank line, 16-byte unit within the line), never splitting a 16-byte atom.
 * Returns SG_OK, SG_ERR_NULL or SG_ERR_SHAPE.
 */
int gemm_lds_layout(int rows, int row_bytes, int32_t* out);

/*
 * gemm_lds_layout_mxfp6 -- the LDS byte map of mxfp6_gemm_run's operand
 * tiles (host-side, no GPU needed).  Writes out[r * 12 + q] = the byte
 * offset within one LDS stage of bytes [8q, 8q + 8) of the 96 bytes of tile
 * row r, for r < rows.  The map is gemm_lds_layout's XOR swizzle for
 * 128-byte rows with every odd row displaced by 8 bytes, except the rows at
 * block position `unshifted` (row % 32 == unshifted; 32 for none), which the
 * kernel uses for the tile holding the operand's last row.  The displacement
 * lets 8-byte reads of 32 rows, which the XOR of 16-byte units alone maps
 * to 16 bank slots, reach all 32 ("Swizzling explained properly", section
 * "Why swizzle?": the bank arithmetic).  rows is a positive multiple of 32.
 * Returns SG_OK, SG_ERR_NULL or SG_ERR_SHAPE.
 */
int gemm_lds_layout_mxfp6(int rows, int unshifted, int32_t* out);

/*
 * gemm_lds_layout_cblock -- where the 256x256 bf16/fp16 kernel keeps a
 * 16-bit C in LDS for its epilogue (host-side, no GPU needed).  That kernel
 * reads C (the "+C" of the GEMM) through the loads of its last two K tiles,
 * which would otherwise fetch zeros past K, into the four half-tile ring
 * slots those loads fill.  Writes out[(w * 128 + r) * 8 + c], for wave
 * w < 4 of a 128-row group, row r < 128 and 16-byte chunk c < 8 of that
 * wave's 128 x 64 block of C: quarter r / 32 (which slot) times 16384 plus
 * the byte offset inside the slot's 16 KiB half.  The placement is an XOR
 * of the chunk index with a row key, the same construction as the operand
 * swizzle ("Swizzling explained properly", section "What does swizzling
 * do?"), chosen for 8-byte epilogue reads.  Returns SG_OK or SG_ERR_NULL.
 */
int gemm_lds_layout_cblock(int32_t* out);

/*
 * gemm_lds_image -- runs the kernels' global->LDS loader once for one operand
 * tile and copies the LDS stage out byte for byte, unswizzled by nothing.
 *   X         device operand, K-major [rows_total][K] of elem_bytes-sized
 *             elements (2 for f16/bf16, 1 for e4m3).
 *   tile_rows 128 or 256; the tile covers rows [row0, row0 + tile_rows)
 *             and the 128-byte K slice starting at element k0 (k0 * elem_bytes
 *             a multiple of 128).  Rows >= rows_total and k >= K read as zero.
 *   out       device buffer of tile_rows * 128 bytes.
 * Returns SG_OK or an SG_ERR_* code.
 */
int gemm_lds_image(const void* X, int64_t rows_total, int64_t K, int elem_bytes,
                   int64_t row0, int64_t k0, int tile_rows, void* out,
                   void* stream);

/*
 * Measurement support (not part of any GEMM call).
 *
 * gemm_clock_trace -- turns the clock trace of this thread's later launches
 * on (buf non-NULL) or off (buf NULL).  While on, every kernel of a gemm_run,
 * gemm_strided_run, gemm_layout_run, gemm_layout128_run, grouped_gemm_run,
 * mx_gemm_run, mxfp4_gemm_run, mxfp6_gemm_run, i8_gemm_run or
 * i8_grouped_gemm_run call (of the last, the workgroups that have a tile)
 * records, for each workgroup b < slots, buf[4b .. 4b+3] = {shader-clock counter at its start,
 * the same at the end of its first wave, real-time counter at the start, the
 * same at the end}.  The shader-clock counter (s_memtime) advances once per
 * core clock; the real-time counter (s_memrealtime) at the constant rate
 * written to *wall_khz (kHz, the device attribute; NULL skips it).  So
 * (t_end - t_start) / (rt_end - rt_start) * wall_khz is the clock in kHz
 * that workgroup ran at: the clock the GEMM itself held, which sets its
 * clock-adjusted MFMA peak.  buf: DEVICE memory of 4 * slots uint64_t,
 * 8-byte aligned, alive while the trace is on.  The kernels only test the
 * pointer when the trace is off.  Errors: SG_ERR_SHAPE (slots < 0),
 * SG_ERR_ALIGN, SG_ERR_HIP.
 */
int gemm_clock_trace(void* buf, int64_t slots, int* wall_khz);

/*
 * gemm_clock_probe -- a kernel of W = gemm_clock_probe_waves() waves, one
 * workgroup of eight waves per CU of 256 CUs (two waves per SIMD, as the
 * 256x256 GEMM runs), each issuing `iters` rounds of 8 independent
 * v_mfma_f32_16x16x32_bf16 (16 cycles each) on random bf16 register
 * operands.  Wave w writes out[4w .. 4w+3] = {shader-clock counter at the
 * start of its loop, at the end, real-time counter at the start, at the end}
 * and out[4W + w] = bits of its fp32 accumulator sum.  Over a CU's eight
 * waves, 16 * 2 * 8 * iters cycles (the MFMAs of one SIMD) per real-time
 * span is the clock under a full MFMA load, and the shader-clock span over
 * the same real-time span shows whether the counter counts core clocks.
 * out: DEVICE memory of 5 * W uint64_t.  iters in [1, 2^24].  Errors:
 * SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE, SG_ERR_HIP.
 */
int gemm_clock_probe(int64_t iters, void* out, void* stream);
int gemm_clock_probe_waves(void);

/*
 * gemm_last_kernel -- the kernel instantiation the last call on this thread
 * that launched one enqueued, as "name<parameters>" (for example
 * "pingpong16_gemm_kernel<bf16,k,k,swz16>"); "" before any launch.  Calls
 * that launch nothing (an error, an empty problem) leave it unchanged.
 * Thread-local; never NULL.
 */
const char* gemm_last_kernel(void);

/*
 * gemm_lds_image_tile -- runs one loader of the 256x256 kernels once, as the
 * first group of four waves of a workgroup issues it, and copies the LDS it
 * filled to `out` byte for byte, so that tests can hold the loaded image
 * against the byte map the fragment reads use ("Swizzling explained
 * properly", section "Sample swizzled matmul": the stores into the swizzled
 * tile and the reads out of it must use one map).
 *   X        DEVICE rows of `row_bytes` bytes (a multiple of 16), `rows` of
 *            them, 16-byte aligned; bytes past a row or rows past `rows`
 *            read as zero where the loader zero-fills.
 *   kind     SG_IMG_HALF / SG_IMG_HALF_KEXACT: a K-major 16-bit operand; the
 *              half tile of rows [row0, row0 + 128) and bytes [byte0, byte0
 *              + 128) (byte0 % 128 == 0) through the loader that checks K
 *              per load / the K-exact loader (row_bytes % 128 == 0).  The
 *              image is 16384 bytes laid out by gemm_lds_layout(128, 128).
 *            SG_IMG_MN256: an MN-major 16-bit operand [K = rows][row_bytes/2];
 *              k rows [row0, row0 + 64) (row0 % 64 == 0), columns [byte0/2,
 *              byte0/2 + 128) (byte0 % 256 == 0).  16384 bytes: byte b of
 *              k row r at 256 r + 32 ((b / 32) XOR key(r)) + b mod 32,
 *              key(r) = (r mod 4) + 4 (bit 3 of r).
 *            SG_IMG_FP6: an MXFP6 operand (row_bytes = 3K/4, a multiple of
 *              96); rows [row0, row0 + 128) of the 256-row tile at row0
 *              (row0 % 256 == 0), the K tile of bytes [byte0, byte0 + 96)
 *              (byte0 % 96 == 0).  16384 bytes laid out by
 *              gemm_lds_layout_mxfp6(128, u) with u the block position of
 *              the operand's last row if that row lies in this 256-row tile,
 *              else 32.
 *            SG_IMG_CBLOCK: a 16-bit C [rows][row_bytes/2]; the first 128
 *              rows of the 256 x 256 output tile at (row0, byte0/2) (row0 %
 *              256 == 0, byte0 % 512 == 0).  65536 bytes: the four
 *              quarters of gemm_lds_layout_cblock(), quarter Q at 16384 Q.
 *   out      DEVICE buffer of 16384 (65536 for SG_IMG_CBLOCK) bytes.
 * Errors: SG_ERR_NULL, SG_ERR_ALIGN, SG_ERR_SHAPE (origin not on the grid,
 * or outside the operand), SG_ERR_DTYPE (unknown kind), SG_ERR_HIP.
 */
#define SG_IMG_HALF 1
#define SG_IMG_HALF_KEXACT 2
#define SG_IMG_MN256 3
#define SG_IMG_FP6 4
#define SG_IMG_CBLOCK 5
int gemm_lds_image_tile(int kind, const void* X, int64_t rows, int64_t row_bytes,
                        int64_t row0, int64_t byte0, void* out, void* stream);

/*
 * gemm_mfma_scale_probe -- one v_mfma_scale_f32_32x32x64_f8f6f4 of one wave
 * with the format code fmt for both operands (0 e4m3, 2 e2m3, 3 e3m2, 4
 * e2m1), accumulating from zero: lane l (0..63) passes a[32 l .. 32 l + 31]
 * as its first source operand, b[32 l ..] as its second, and scale bytes
 * sa[l], sb[l] (byte 0 of each scale register).  out[16 l + r] receives
 * accumulator register r of lane l.  It exposes the scaled MFMA's operand
 * and scale layout -- which K element and which 32-element block each lane
 * and byte feed ("06 Blackwell Tensor Core - tcgen05 MMA", section
 * "Block-Scaled MMA", defines that placement for its own hardware) -- to
 * tests with one-hot operands.  a, b: DEVICE, 2048 bytes each; sa, sb: 64
 * bytes each; out: 4096 bytes (fp32).
 * Errors: SG_ERR_NULL, SG_ERR_ALIGN (a, b, out not 16-byte aligned),
 * SG_ERR_DTYPE (fmt), SG_ERR_HIP.
 */
int gemm_mfma_scale_probe(int fmt, const void* a, const void* b, const void* sa,
                          const void* sb, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SWIZZLED_GEMM_H */
