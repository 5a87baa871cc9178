/*
 * mx.h -- C ABI of the GB300 (sm_103a) block-scaled quantization and GEMM library
 * (libmxgb.so).
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are CALLER-OWNED DEVICE memory.  No call allocates or frees.
 *  - Every call is asynchronous on `stream` (a cudaStream_t passed as void*; NULL is the
 *    legacy default stream).  No call synchronizes the host.  Kernels are launched with
 *    programmatic dependent launch: one may be scheduled while the previous kernel on the
 *    stream finishes, but it reads no memory before that kernel has completed, so stream
 *    order holds for every input, whichever kernel wrote it.
 *  - Matrices are row-major.  A GEMM computes C[m][n] = sum_k A[m][k] * B[n][k]: both code
 *    operands are K-contiguous ("TN" in column-major BLAS terms).  Column-wise quantized
 *    copies are stored physically transposed, so fprop, dgrad and wgrad all run as this one
 *    product:  fprop  Y  = X W^T : A = X row-wise,   B = W row-wise
 *              dgrad dX  = G W   : A = G row-wise,   B = W column-wise (W^T)
 *              wgrad dW  = G^T X : A = G column-wise, B = X column-wise
 *  - Arguments are validated on the host before anything is launched.  A null pointer, a
 *    shape that is not a multiple of the tile, a misaligned pointer or a bad enum value
 *    returns MX_ERR_INVALID_ARG; a valid but unimplemented combination returns
 *    MX_ERR_UNSUPPORTED; a launch failure returns MX_ERR_CUDA.  The quantizers take at most
 *    65535 tiles of 128 columns (cols <= 8388480); wider inputs return MX_ERR_INVALID_ARG.
 *  - Device-side waits are bounded.  A wait that runs out sets a device error word instead of
 *    hanging; mx_check() reports it as MX_ERR_TIMEOUT.
 *
 * Scale-factor layouts ("GEMM layout", written by the quantizers, read by the GEMMs)
 *  - MX, E8M0, one scale per 32 consecutive elements along K.  For a code matrix Q[R][K]
 *    (R % 128 == 0, K % 128 == 0) the R*K/32 scale bytes form 512-byte chunks, one per
 *    128 rows x 128 elements of K.  Chunk (rb, kc), rb < R/128, kc < K/128, starts at byte
 *    (rb * (K/128) + kc) * 512.  Inside it, the scale of row 128*rb + i and of 32-block
 *    4*kc + j is at byte (i % 32) * 16 + (i / 32) * 4 + j.
 *  - NVFP4, E4M3, one scale per 16 consecutive elements along K: the same 512-byte chunk
 *    shape, but a chunk covers 128 rows x 64 elements of K (4 blocks of 16); chunk (rb, kc),
 *    kc < K/64, starts at byte (rb * (K/64) + kc) * 512, in-chunk offset as above.
 *  - DeepSeek FP32 scales: 1x128 activation tiles are stored k-block-major, s[K/128][R]
 *    (float), so one k-block's scales for consecutive rows are contiguous; 128x128 weight
 *    blocks are stored s[R/128][K/128] (float).
 *  - Packed FP4: element 2i of a row in the low nibble of byte i, element 2i+1 in the high
 *    nibble.
 *
 * Sources (page title and section):
 *  [MX]  "MXFP8 on SM120: software support" (xuesongtap.github.io): sec 0.1 MX block format,
 *        E8M0 scale, q = Q_FP8(x / s); sec 0.3 block-scaled dot product; sec 1.1-1.2 TN/NN/NT
 *        and the fprop/dgrad/wgrad GEMM trio; sec 1.2 row-wise vs column-wise blocks.
 *  [DS]  "Why FP8 training is stable" (magicnetworld.com): sec 4 s = amax/MAX; sec 5 1x128
 *        activation tiles and 128x128 weight blocks; sec 6.3 FP32 promotion every N_C = 128.
 *  [NV]  "NVFP4: high accuracy with 4 bits" (theluyuan.com): sec 5.4 two-level scales;
 *        sec 5.6 worked example; sec 7.3-7.4 block scale outside the sum, global scale in the
 *        epilogue.
 */
#ifndef MXGB_MX_H_
#define MXGB_MX_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MX_OK = 0,
  MX_ERR_INVALID_ARG = 1,
  MX_ERR_UNSUPPORTED = 2,
  MX_ERR_CUDA = 3,
  MX_ERR_TIMEOUT = 4
} mx_status;

typedef enum { MX_E4M3 = 0, MX_E5M2 = 1, MX_E2M1 = 2 } mx_elem;
typedef enum { MX_SCALE_E8M0 = 0, MX_SCALE_UE4M3 = 1, MX_SCALE_FP32 = 2, MX_SCALE_FP32_POW2 = 3 } mx_scale_fmt;
typedef enum { MX_ROWWISE = 1, MX_COLWISE = 2, MX_BOTH = 3 } mx_layout;
typedef enum { MX_OUT_F32 = 0, MX_OUT_BF16 = 1 } mx_out;
typedef enum { MX_HALF_BF16 = 0, MX_HALF_F16 = 1 } mx_half;

/* Version of this ABI (bumped on any signature or layout change). */
int mx_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* mx_status_string(mx_status s);

/*
 * mx_quantize -- block quantization of a bf16 matrix.  [MX] sec 0.1, [DS] sec 4-5.
 *
 * x[rows][cols]: bf16, row-major, 16-byte aligned.  Blocks run along cols (the reduction
 * axis of the consuming GEMM) for the row-wise copy and along rows for the column-wise copy.
 *
 * Supported combinations (anything else returns MX_ERR_UNSUPPORTED):
 *  1. MX: block = 32, block_rows = 1, elem = MX_E4M3 or MX_E5M2 (MXFP8) or MX_E2M1
 *     (MXFP4, [NV] sec 5.5), sfmt = MX_SCALE_E8M0, layout = ROWWISE, COLWISE or BOTH;
 *     rows % 128 == 0, cols % 128 == 0.
 *     Per block: amax = max |x|; k = clamp(floor(log2 amax) - emax, -127, 127) with emax 8
 *     (E4M3), 15 (E5M2) or 2 (E2M1), k = -127 when amax == 0; scale byte = k + 127;
 *     q = RNE-satfinite(x * 2^-k).  A NaN or Inf in a block gives scale 0xFF and all codes
 *     0x7F (E2M1: 0x7).  With BOTH, both copies come from one read of x.
 *       q_row[rows][cols] u8, s_row: rows*cols/32 bytes in the MX GEMM layout;
 *       q_col[cols][rows] u8 (transposed), s_col: the MX GEMM layout of that [cols][rows]
 *       matrix.  Pointers of a copy that is not requested may be NULL.
 *       MXFP4 codes are packed two per byte, element 2i in the low nibble:
 *       q_row[rows][cols/2], q_col[cols][rows/2].
 *  1b. MX with 2-D weight blocks: block = 32, block_rows = 32, elem = MX_E4M3 or MX_E5M2,
 *     sfmt = MX_SCALE_E8M0 ([MX] sec 1.3): one scale per 32x32 block of x by the rule of 1
 *     over the whole block, stored expanded exactly as in 1 (every 1x32 block of a row-wise
 *     row and of a column-wise row carries its 32x32 block's scale), so mx_gemm consumes it
 *     unchanged; the column-wise codes are the transpose of the row-wise ones.
 *  2. DeepSeek activations: block = 128, block_rows = 1, elem = MX_E4M3,
 *     sfmt = MX_SCALE_FP32, layout = ROWWISE; rows % 128 == 0, cols % 128 == 0.
 *     s = fl32(amax / 448) (1.0 when amax == 0); q = RNE-satfinite(fl32(x / s)).
 *       q_row[rows][cols] u8, s_row float[cols/128][rows].
 *  3. DeepSeek weights: block = 128, block_rows = 128, otherwise as 2.
 *  2/3 with sfmt = MX_SCALE_FP32_POW2: Float8BlockScaling with power-of-two scales ([MX]
 *     sec 1.3): s = 2^k with k the smallest integer such that 448 * 2^k >= amax (clamped to
 *     [-127, 127]; s = 1 when amax == 0), q = RNE-satfinite(x * 2^-k); same layouts as 2/3.
 *     mx_scales_from_fp32_blocks turns these scales into MX scales for mx_gemm.
 *       q_row[rows][cols] u8, s_row float[rows/128][cols/128].
 *     Inputs for 2 and 3 must be finite.
 */
mx_status mx_quantize(const void* x, int64_t rows, int64_t cols, int block, int block_rows,
                      mx_elem elem, mx_scale_fmt sfmt, mx_layout layout,
                      void* q_row, void* s_row, void* q_col, void* s_col, void* stream);

/*
 * mx_quantize_dual -- MX quantization of one bf16 matrix into both element formats at once:
 * E4M3 and E5M2 codes with their E8M0 scales, row-wise and/or column-wise, from a single read of
 * x.  Each output is exactly what mx_quantize (block = 32, MX_SCALE_E8M0) writes for that format.
 * [MX] sec 0.1 (block format; E4M3 and E5M2 are both MXFP8 element encodings) and sec 1.2
 * (row-wise and column-wise copies).  Shapes, alignment and layouts as in mx_quantize; the eight
 * output pointers of the requested copies must be non-NULL.
 */
mx_status mx_quantize_dual(const void* x, int64_t rows, int64_t cols, mx_layout layout,
                           void* q_row_e4m3, void* s_row_e4m3, void* q_col_e4m3, void* s_col_e4m3,
                           void* q_row_e5m2, void* s_row_e5m2, void* q_col_e5m2, void* s_col_e5m2,
                           void* stream);

/*
 * mx_gemm -- MX block-scaled GEMM (MXFP8, MXFP4).  [MX] sec 0.3, [NV] sec 5.5:
 *   C[m][n] = sum_b sA[m][b] sB[n][b] sum_{i<32} qA[m][32b+i] qB[n][32b+i], FP32 accumulate.
 *
 * qa[M][K], qb[N][K]: E4M3 or E5M2 codes (ea, eb), 16-byte aligned; sa, sb: E8M0 scales in
 * the MX GEMM layout.  out: M rows of ldc elements (ldc >= N, ldc % 8 == 0), FP32 or bf16
 * (RNE).  M % 128 == 0, N % 128 == 0, K % 128 == 0.
 * MXFP4: ea = eb = MX_E2M1, qa[M][K/2], qb[N][K/2] packed (element 2i in the low nibble, as
 * mx_quantize writes them), K % 256 == 0.  An E2M1 operand with an FP8 one returns
 * MX_ERR_UNSUPPORTED.
 */
mx_status mx_gemm(const void* qa, const void* sa, mx_elem ea,
                  const void* qb, const void* sb, mx_elem eb,
                  int64_t M, int64_t N, int64_t K,
                  void* out, mx_out out_dtype, int64_t ldc, void* stream);

/*
 * nvfp4_quantize_ex -- NVFP4 with the training options of [DS] sec 13 and [NV] sec 3.2.
 *
 * Same arguments, layouts and limits as nvfp4_quantize, plus:
 *   use_rht = 1: every 1x16 block along cols is first replaced by 0.25 * H16 * (d .* x), H16
 *     the 16x16 Sylvester Hadamard matrix and d_i = -1 where bit i of rht_signs is set (the
 *     random signs are an input; rht_signs <= 0xFFFF).  Computed in FP32 with butterflies in
 *     the order h = 1, 2, 4, 8; the global maximum, block scales and codes are those of the
 *     transformed values.  Operands transformed with the same signs multiply to the same
 *     product (0.25 H16 is orthogonal and symmetric).
 *   rbits != NULL: stochastic rounding of the element codes.  rbits[rows][cols] (u8, 16-byte
 *     aligned) holds one random byte r per element; with y = fl32(x / s_hat), |y| < 6 lying
 *     between E2M1 values lo <= |y| < hi, the code rounds up iff r < floor(256 (|y| - lo) /
 *     (hi - lo)); |y| >= 6 gives 6.  NULL: round to nearest even as nvfp4_quantize.
 * use_rht not 0/1 or rht_signs > 0xFFFF: MX_ERR_INVALID_ARG.
 */
mx_status nvfp4_quantize_ex(const void* x, int64_t rows, int64_t cols, int use_rht, uint32_t rht_signs,
                            const void* rbits, void* q_packed, void* s_ue4m3, float* gscale, void* workspace,
                            void* stream);

/*
 * nvfp4_quantize_2d -- NVFP4 with 16x16 2-D blocks (weights, [DS] sec 13).
 *
 * One E4M3 block scale per 16x16 block of x (the recipe of nvfp4_quantize with the block maximum
 * over 256 elements; same global scale), written for both orientations: q_row[rows][cols/2] and
 * s_row (the NVFP4 GEMM layout of [rows][cols/16]) as nvfp4_quantize writes them, and
 * q_col[cols][rows/2], s_col (the layout of [cols][rows/16]) for the transposed matrix; the two
 * hold the same codes and scales.  rows % 128 == 0, cols % 128 == 0; workspace as for
 * nvfp4_quantize.
 */
mx_status nvfp4_quantize_2d(const void* x, int64_t rows, int64_t cols, void* q_row, void* s_row, void* q_col,
                            void* s_col, float* gscale, void* workspace, void* stream);

/*
 * mx_scales_from_fp32_blocks -- Float8BlockScaling scales in MX form.  [MX] sec 1.3.
 *
 * s: power-of-two FP32 block scales as mx_quantize(block = 128, sfmt = MX_SCALE_FP32_POW2)
 * writes them: block_rows = 1 -> float[cols/128][rows] (1x128 tiles of a [rows][cols] code
 * matrix), block_rows = 128 -> float[rows/128][cols/128] (128x128 blocks); 4-byte aligned.
 * s_e8m0: rows*cols/32 bytes (16-byte aligned), written in the MX GEMM layout of the
 * [rows][cols] code matrix: each 1x32 block gets its 128-block's scale 2^k as the E8M0 code
 * k + 127; a scale that is not exactly 2^k with -127 <= k <= 127 becomes the E8M0 NaN code 0xFF
 * (products that use it are NaN).  The E4M3 codes are passed to mx_gemm as they are.
 * rows % 128 == 0, cols % 128 == 0, block_rows 1 or 128, else MX_ERR_INVALID_ARG.
 */
mx_status mx_scales_from_fp32_blocks(const float* s, int64_t rows, int64_t cols, int block_rows, void* s_e8m0,
                                     void* stream);

/*
 * mx_selftest_wait_timeout -- exercises the failure path of the device-side waits.  Launches one
 * CTA that waits on an mbarrier nothing ever arrives on, through the same bounded wait the GEMM
 * kernels use, with a budget of budget_us microseconds (1 .. 1000000) instead of the kernels'
 * 2 s.  The wait runs out, records its site in the device error word and the kernel returns; the
 * next mx_check() on the stream reports MX_ERR_TIMEOUT (and clears the word).  Nothing faults
 * and the context stays usable.  Returns MX_ERR_INVALID_ARG for a budget out of range.
 */
mx_status mx_selftest_wait_timeout(int64_t budget_us, void* stream);

/*
 * mx_unswizzle_scales / mx_swizzle_scales -- byte permutations between the GEMM scale layout
 * (the chunked layout described at the top of this header, as the quantizers write it and the
 * GEMMs read it) and a plain row-major matrix s_plain[rows][nblocks], one byte per block:
 * nblocks = K/32 for MX (E8M0) scales and K/16 for NVFP4 (E4M3) scales of a [rows][K] code
 * matrix.  For inspecting scales, comparing them with another implementation, or bringing in
 * scales computed elsewhere.  Both buffers are device memory of rows*nblocks bytes and must not
 * overlap; the chunked one 16-byte aligned, the plain one 4-byte aligned.
 * rows % 128 == 0, nblocks % 4 == 0, else MX_ERR_INVALID_ARG.  No arithmetic: bytes move as
 * they are.
 */
mx_status mx_unswizzle_scales(const void* s_gemm, int64_t rows, int64_t nblocks, void* s_plain, void* stream);
mx_status mx_swizzle_scales(const void* s_plain, int64_t rows, int64_t nblocks, void* s_gemm, void* stream);

/*
 * mx_gemm_mxout -- MXFP8 GEMM whose epilogue quantizes its own results for the next product
 * (producer-side fusion of the MX quantization; [MX] sec 0.1 rule, [DS] sec 9 quantizes the
 * activations that feed the next FP8 product before they leave).
 *
 * The product of mx_gemm (same operands, formats and FP32 accumulation), then per 1x32 block of
 * each output row the MX quantization of the FP32 results into out_elem (MX_E4M3 or MX_E5M2):
 * scale byte max(exp(amax) - emax, 0) (0xFF and codes 0x7F when a result is Inf or NaN), codes
 * RNE-satfinite(y * 2^-k).  q_out[M][ldq] u8 codes (ldq >= N, ldq % 16 == 0), s_out: M*N/32
 * bytes in the MX GEMM layout of [M][N] -- exactly the A operand of a following mx_gemm.
 * No bf16 / FP32 output is written.  M % 256 == 0, N % 256 == 0, K % 128 == 0.
 */
mx_status mx_gemm_mxout(const void* qa, const void* sa, mx_elem ea, const void* qb, const void* sb, mx_elem eb,
                        int64_t M, int64_t N, int64_t K, mx_elem out_elem, void* q_out, void* s_out, int64_t ldq,
                        void* stream);

/*
 * mx_gemm_mxout_ex -- mx_gemm_mxout with the copies a training step needs ([MX] sec 1.2: a
 * transpose needs its own blocks, scales and codes): layout MX_ROWWISE writes the row-wise copy
 * exactly as mx_gemm_mxout (q_row[M][ldq_row], s_row in the MX GEMM layout of [M][N]);
 * MX_COLWISE writes the column-wise copy -- 32x1 blocks down each column of the result, stored
 * transposed like mx_quantize's column-wise output: q_col[N][ldq_col] codes (ldq_col >= M,
 * ldq_col % 16 == 0) and s_col: M*N/32 bytes in the MX GEMM layout of [N][M], i.e. the operand of
 * a following product that reduces over M; MX_BOTH writes both from the same FP32 results.  Same
 * scale and code rule as mx_gemm_mxout per block.  Pointers of a copy not requested may be NULL.
 * M % 256 == 0, N % 256 == 0, K % 128 == 0.
 */
mx_status mx_gemm_mxout_ex(const void* qa, const void* sa, mx_elem ea, const void* qb, const void* sb, mx_elem eb,
                           int64_t M, int64_t N, int64_t K, mx_elem out_elem, mx_layout layout, void* q_row,
                           void* s_row, int64_t ldq_row, void* q_col, void* s_col, int64_t ldq_col, void* stream);

/*
 * mx_gemm_grouped -- MXFP8 expert GEMMs of a mixture-of-experts layer in one launch.  [MX]
 * sec 1.2 (grouped GEMM is its own entry point besides the single GEMMs).
 *
 * groups G (1..1024); group g multiplies rows off[g] .. off[g+1]-1 of A by the g-th block of B:
 *   C[m][n] = sum_b sA[m][b] sB[gN + n][b] sum_{i<32} qA[m][32b+i] qB[gN + n][32b+i]
 * for off[g] <= m < off[g+1], with the block scaling of mx_gemm.
 * qa[M][K] (all groups' rows stacked), sa its E8M0 scales in the MX GEMM layout of [M][K];
 * qb[G*N][K] (block g = rows gN .. gN+N-1), sb the layout of [G*N][K]; out M rows of ldc
 * elements.  group_offsets: device int64[G + 1], 8-byte aligned, read by the kernel (so the
 * expert sizes can come from device-side routing without a host round trip); they must satisfy
 * off[0] = 0, off[G] = M, off[g] <= off[g+1] and off[g] % 128 == 0 (an empty group is allowed).
 * Offsets that break this make the call do nothing and mx_check return MX_ERR_INVALID_ARG.
 * M % 128 == 0, N % 256 == 0, K % 128 == 0, element formats as mx_gemm: MXFP8 (E4M3 / E5M2) or
 * MXFP4 (both MX_E2M1, codes packed as mx_quantize writes them, K % 256 == 0).
 */
mx_status mx_gemm_grouped(const void* qa, const void* sa, mx_elem ea, const void* qb, const void* sb, mx_elem eb,
                          const int64_t* group_offsets, int64_t groups, int64_t M, int64_t N, int64_t K, void* out,
                          mx_out out_dtype, int64_t ldc, void* stream);

/*
 * nvfp4_gemm_grouped -- NVFP4 expert GEMMs in one launch: group g computes, for its rows
 * off[g] <= m < off[g+1],  C[m][n] = s_gA * s_gB[g] * sum_b sA[m][b] sB[gN + n][b] sum_{i<16} qA qB
 * ([NV] sec 7.3-7.4; each expert's weights are quantized as their own tensor, so each has its own
 * global scale).  qa[M][K/2] packed E2M1 with sa in the NVFP4 GEMM layout of [M][K] and one global
 * scale ga (device float); qb[G*N][K/2] with sb the layout of [G*N][K] and gb: device float[G].
 * group_offsets as mx_gemm_grouped.  M % 128 == 0, N % 256 == 0, K % 256 == 0.
 */
mx_status nvfp4_gemm_grouped(const void* qa, const void* sa, const float* ga, const void* qb, const void* sb,
                             const float* gb, const int64_t* group_offsets, int64_t groups, int64_t M, int64_t N,
                             int64_t K, void* out, mx_out out_dtype, int64_t ldc, void* stream);

/*
 * nvfp4_gemm_grouped_ex -- nvfp4_gemm_grouped with, when ga_per_group == 1, one global scale of A
 * per group: ga is then a device float[G] and group g's results are scaled by ga[g] * gb[g] (the
 * tokens routed to each expert quantized as a tensor of their own, e.g. by nvfp4_quantize_grouped
 * with the same offsets).  ga_per_group == 0 is nvfp4_gemm_grouped; any other value returns
 * MX_ERR_INVALID_ARG.
 */
mx_status nvfp4_gemm_grouped_ex(const void* qa, const void* sa, const float* ga, int ga_per_group, const void* qb,
                                const void* sb, const float* gb, const int64_t* group_offsets, int64_t groups,
                                int64_t M, int64_t N, int64_t K, void* out, mx_out out_dtype, int64_t ldc,
                                void* stream);

/*
 * fp8_blockwise_gemm_grouped -- the DeepSeek FP8 expert GEMMs of a mixture-of-experts layer in one
 * launch ([DS] sec 5, 6.3; group layout as mx_gemm_grouped): group g computes, for its rows
 * off[g] <= m < off[g+1], C[m][n] = sum_kb sA[kb][m] sB[gN/128 + n/128][kb] P_kb[m][n], with P_kb
 * the exact FP32 sum of qA qB over k-block kb (promotion every 128 of K, as fp8_blockwise_gemm).
 * qa[M][K] E4M3 with sa float[K/128][M] (1x128 tiles); qb[G*N][K] E4M3, the experts' [N][K]
 * weights stacked, with sb float[G*N/128][K/128] (their 128x128 blocks stacked the same way, as
 * one mx_quantize(block=128, block_rows=128) of the stacked weights gives).  group_offsets as
 * mx_gemm_grouped.  M % 128 == 0, N % 256 == 0, K % 128 == 0, 1 <= G <= 1024; out as for mx_gemm.
 */
mx_status fp8_blockwise_gemm_grouped(const void* qa, const float* sa, const void* qb, const float* sb,
                                     const int64_t* group_offsets, int64_t groups, int64_t M, int64_t N, int64_t K,
                                     void* out, mx_out out_dtype, int64_t ldc, void* stream);

/* Bytes of caller-owned device workspace nvfp4_quantize needs (>= 16). */
size_t nvfp4_workspace_bytes(int64_t rows, int64_t cols);

/*
 * nvfp4_quantize -- NVFP4 two-level quantization.  [NV] sec 5.4, 5.6.
 *   pass 1: amax over the whole tensor; s_g = fl32(amax / 2688) (1.0 if amax == 0),
 *           written to *gscale (device float).
 *   pass 2: per 16 consecutive elements along cols: t = fl32(fl32(bamax / 6) / s_g);
 *           c = E4M3 RNE-satfinite(t); s_hat = fl32(dec(c) * s_g);
 *           q = E2M1 RNE-satfinite(fl32(x / s_hat)) (0 when s_hat == 0).
 * x[rows][cols] bf16 (finite); q_packed[rows][cols/2] u8; s_ue4m3: rows*cols/16 bytes in the
 * NVFP4 GEMM layout; workspace: nvfp4_workspace_bytes() bytes, 16-byte aligned, contents
 * need not be initialised (the call clears it on `stream`).  rows % 128 == 0,
 * cols % 64 == 0.
 */
mx_status nvfp4_quantize(const void* x, int64_t rows, int64_t cols,
                         void* q_packed, void* s_ue4m3, float* gscale,
                         void* workspace, void* stream);

/*
 * nvfp4_quantize_grouped -- NVFP4 quantization of G row groups of one bf16 matrix, each group a
 * tensor of its own (the weights or tokens of MoE experts; [NV] sec 5.4 applied per group): group
 * g, rows off[g] <= r < off[g+1], gets its own amax and global scale gscale[g].  The results equal
 * G calls of nvfp4_quantize on the groups' row slices, bit for bit: q_packed and s_ue4m3 hold the
 * codes and scale chunks of the whole [rows][cols] matrix in the NVFP4 GEMM layout, group g's in
 * its own rows (the layout nvfp4_gemm_grouped reads for B, whose gb is this gscale).
 * group_offsets: device int64[G + 1], 0 = off[0] <= off[1] <= ... <= off[G] = rows, all multiples
 * of 128; an empty group gets gscale 1.0.  Offsets that break this contract make the next
 * mx_check() report MX_ERR_INVALID_ARG; the outputs are then unspecified, but no access leaves
 * the caller's buffers.  gscale: device float[G]; workspace: 4 * G bytes (at least 16), 16-byte
 * aligned, cleared by the call on `stream`.  1 <= G <= 1024, rows % 128 == 0, cols % 64 == 0.
 */
mx_status nvfp4_quantize_grouped(const void* x, int64_t rows, int64_t cols, const int64_t* group_offsets,
                                 int64_t groups, void* q_packed, void* s_ue4m3, float* gscale, void* workspace,
                                 void* stream);

/*
 * nvfp4_gemm -- NVFP4 block-scaled GEMM.  [NV] sec 7.3-7.4:
 *   C[m][n] = gA * gB * sum_b sA[m][b] sB[n][b] sum_{i<16} qA qB, FP32 accumulate; the two
 *   global scales (device floats written by nvfp4_quantize) are applied in the epilogue.
 * qa[M][K/2], qb[N][K/2] packed E2M1; sa, sb in the NVFP4 GEMM layout.
 * M % 128 == 0, N % 128 == 0, K % 256 == 0; out as for mx_gemm.
 */
mx_status nvfp4_gemm(const void* qa, const void* sa, const float* ga,
                     const void* qb, const void* sb, const float* gb,
                     int64_t M, int64_t N, int64_t K,
                     void* out, mx_out out_dtype, int64_t ldc, void* stream);

/*
 * fp8_blockwise_gemm -- DeepSeek-style FP8 GEMM with FP32 promotion.  [DS] sec 6.3:
 *   for every 128-wide k-block kb: P = sum_{k in kb} qA[m][k] qB[n][k] (tensor cores, FP32),
 *   acc += sA[kb][m] * sB[n/128][kb] * P in FP32 registers.
 * qa[M][K], qb[N][K] E4M3; sa float[K/128][M] (1x128 tiles, k-block-major);
 * sb float[N/128][K/128] (128x128 blocks).  M % 128 == 0, N % 128 == 0, K % 128 == 0.
 */
mx_status fp8_blockwise_gemm(const void* qa, const float* sa,
                             const void* qb, const float* sb,
                             int64_t M, int64_t N, int64_t K,
                             void* out, mx_out out_dtype, int64_t ldc, void* stream);

/*
 * nvfp4_quantize_noalloc -- the same NVFP4 quantization as nvfp4_quantize, for callers that
 * cannot allocate device memory (for example a plug-in inside a host whose allocator owns all of
 * the GPU's memory, or a launch path that must never call cudaMalloc because it synchronizes the
 * device).  It takes no workspace and allocates nothing: its scratch is a 64 KB array inside
 * libmxgb.so that every GPU which loads the library keeps until the process exits.  The pages
 * have no counterpart to this entry point; it exists only for such callers.
 *
 * Arguments and results are those of nvfp4_quantize (identical codes, scales and gscale).
 * Limit: rows <= 262144 (the array holds one partial maximum per 16 rows); larger inputs return
 * MX_ERR_INVALID_ARG.  The first call on each device looks up the array's device address (with
 * that device current); make that first call before any stream capture.  The address is cached
 * per device ordinal, so the library assumes that every call on a device runs in the CUDA
 * runtime's primary context of that device (the context the runtime API and PyTorch use); a
 * caller that makes its own driver-API contexts must not call this entry point from them.  All
 * calls share the one array: calls that overlap on the GPU (different streams, or different host
 * threads, without ordering between them) race and may produce wrong results.  Each call writes every scratch slot
 * it reads before reading it, so nothing left by an earlier call needs clearing.
 */
mx_status nvfp4_quantize_noalloc(const void* x, int64_t rows, int64_t cols,
                                 void* q_packed, void* s_ue4m3, float* gscale, void* stream);

/* Bytes of the scale tensor mx_quantize / nvfp4_quantize write for a [rows][cols] input:
 * block 32 + E8M0 -> rows*cols/32 (block_rows 1, and 32: 2-D blocks are stored expanded);
 * block 16 + UE4M3 -> rows*cols/16; block 128 + FP32 or FP32_POW2 -> 4*rows*cols/128
 * (block_rows 1) or 4*(rows/128)*(cols/128) (block_rows 128).  0 if the combination is not
 * supported. */
size_t mx_scale_bytes(int64_t rows, int64_t cols, int block, int block_rows, mx_scale_fmt sfmt);

/*
 * 8-bit key/value cache.
 *
 * A cache keeps the keys and values of many requests in blocks of P = block_tokens tokens
 * (16, 32, 64 or 128), as 8-bit codes with one FP32 scale for each block and kv head:
 *   k_codes, v_codes  u8 [num_blocks][kv_heads][P][head_dim], E4M3 or E5M2, 16-byte aligned;
 *   k_scale, v_scale  float [num_blocks][kv_heads]; a token's value is code * scale.
 * Scales are 0 or between 2^-48 and 2^48 (kv_cache_append writes powers of two of that range); a block of
 * scale 0 holds zeros, whatever its codes.  Any other scale breaks the contract (below), and so does a block
 * number out of range: attention gives NaN in the rows that see the block, and only there.
 * head_dim is 64 or 128, kv_heads at most 1024, and num_blocks * kv_heads * P at most 2^31 - 1.
 * A request's tokens are in the blocks that its row of block_tables[requests][max_blocks] (int32)
 * names, P by P; entries past its length are not read, nor by kv_attention those that lie in front of
 * every row's window (a caller may have given such blocks back).  requests is at most 16384,
 * max_blocks * P and the tokens of a call at most 2^30.  Lengths, block numbers and slots are on the
 * device and the host cannot see them: where they break their contract nothing is read or written out
 * of range, and mx_check returns MX_ERR_INVALID_ARG.
 */

/*
 * kv_block_tables -- gives requests their cache blocks and new tokens their places.
 *
 * len_before[r] tokens are held by the first ceil(len_before / P) entries of request r's table row;
 * len_after[r] are to be held.  A request that shrinks (rewound, or finished with len_after = 0)
 * puts entries ceil(len_after / P) .. on the free stack, in order; then requests that grow take
 * blocks off its top, in request order.  free_list[free_capacity] holds the stack, free_count[1] its
 * height.  Tables and free_list are updated in place (entries that a request gave back stay in its
 * row, unread); free_count is only read: info[0] is the new height.
 * The new tokens are those of requests that grow: q_start[requests + 1] their numbering, and for
 * each, positions[num_tokens] its place in the request and slot_map[num_tokens] (int64) its slot
 * block * P + position % P.  num_tokens may exceed their number: the rest is -1.
 * If the stack has too few blocks nothing is moved, info[1] is how many are missing (0 otherwise),
 * info[0] is free_count, and all slots and positions are -1.
 * The step has to stop there (q_start numbers the tokens all the same, and the tables have no blocks for them):
 * look at info[1] on the host before kv_attention.
 * Contract: 0 <= lengths <= max_blocks * P; the stack stays within its capacity; new tokens at most
 * num_tokens; no block is held twice.  Where lengths or counts break it nothing is moved and q_start is 0.
 * Block numbers are moved as they are; one below 0 that is moved or that a new token's place needs is reported,
 * and the token's slot is -1.
 * One launch; the same inputs give the same outputs, and the same call again changes nothing.
 */
mx_status kv_block_tables(int32_t* block_tables, int64_t requests, int64_t max_blocks, const int32_t* len_before,
                          const int32_t* len_after, int32_t* free_list, int64_t free_capacity,
                          const int32_t* free_count, int block_tokens, int64_t num_tokens, int32_t* q_start,
                          int64_t* slot_map, int32_t* positions, int32_t* info, void* stream);

/*
 * kv_cache_append -- writes new keys and values into the cache, quantizing them.
 *
 * k, v: num_tokens tokens of kv_heads heads of head_dim elements, bf16 or fp16, 16-byte aligned,
 * elements contiguous, token and head strides (in elements) multiples of 8: slices of a fused
 * projection will do.  Token t goes to slot_map[t] = block * P + offset; -1 leaves it out.
 * Tokens that follow each other in one block are a run; a block has at most one run in a call.
 * Scales are powers of two: 2^k, k the smallest in [-48, 48] with MAX * 2^k >= amax over the finite
 * values (MAX 448 or 57344; 1 if amax = 0), q = RNE-satfinite(x / scale), NaN -> 0x7F.  A run that
 * starts at offset 0 sets its block's scale from its own values.  One that starts later keeps the
 * block's scale or, where its values need a larger one, raises it, and the codes at the offsets in
 * front of it are rounded again to the new scale; a scale of 0 becomes the run's own (the tokens in front are zeros),
 * and where the block's scale is out of range the run is left out.
 */
mx_status kv_cache_append(const void* k, const void* v, mx_half type, int64_t num_tokens, int64_t k_stride_token,
                          int64_t k_stride_head, int64_t v_stride_token, int64_t v_stride_head,
                          const int64_t* slot_map, void* k_codes, void* v_codes, float* k_scale, float* v_scale,
                          mx_elem elem, int64_t num_blocks, int64_t kv_heads, int block_tokens, int head_dim,
                          void* stream);

/* Bytes of workspace kv_attention needs for these sizes (0 if they are not supported). */
size_t kv_attention_workspace_bytes(int64_t num_tokens, int64_t requests, int64_t max_q_len, int64_t heads,
                                    int64_t kv_heads, int head_dim);

/*
 * kv_attention -- attention of new queries over the cache.
 *
 * q: num_tokens rows of heads x head_dim, bf16 or fp16, 16-byte aligned, strides as in
 * kv_cache_append; rows q_start[r] .. q_start[r + 1] are request r's, the last of its lengths[r]
 * cached tokens (so append first).  heads is a multiple of kv_heads; query heads g * heads / kv_heads
 * and up share kv head g.  Row i of n stands at position p = lengths[r] - n + i and sees the tokens
 * j < lengths[r] with j <= p if causal and j > p - window if window > 0.  No request has more than
 * max_q_len rows (itself at most num_tokens).  softmax_scale is positive and at most 1e30.
 *   out[num_tokens][heads][head_dim] (q's type, 32-byte aligned) = softmax(softmax_scale * q k_j) v_j,
 *   lse[num_tokens][heads] (float) = log sum_j exp(softmax_scale * q k_j).
 * Rows that see no token, and rows from q_start[requests] on, give 0 and -inf.  Rows of a request whose
 * length or rows break their contract, and rows in front of q_start[0], are not written.  NaN in tokens
 * that a row does not see does not reach it, nor does the scale of a block that it does not see.
 * Infinities in the cache (E5M2; append writes none) may come out as NaN.  workspace:
 * kv_attention_workspace_bytes bytes, 32-byte aligned; its first 4096 bytes are zero before its first
 * use and are left zero, so that the next call can use it, for whatever sizes it is large enough (after
 * MX_ERR_TIMEOUT they are to be cleared again); calls that may overlap need one each.  Calls from
 * several host threads on one stream do not overlap, and may share one.
 * Sums and softmax statistics are FP32.  For the second product each token's weight, times its block's V scale, is
 * rounded to FP16 beside the row's largest: below 2^-14 of it bits are lost, from 2^-25 on it is 0.
 */
mx_status kv_attention(const void* q, mx_half type, int64_t num_tokens, int64_t heads, int64_t q_stride_token,
                       int64_t q_stride_head, const void* k_codes, const void* v_codes, const float* k_scale,
                       const float* v_scale, mx_elem elem, int64_t num_blocks, int64_t kv_heads, int block_tokens,
                       int head_dim, const int32_t* block_tables, int64_t max_blocks, const int32_t* lengths,
                       const int32_t* q_start, int64_t requests, int64_t max_q_len, float softmax_scale, int causal,
                       int64_t window, void* out, float* lse, void* workspace, void* stream);

/*
 * Norm and rotation of queries and keys.
 *
 * qk_norm_rope -- RMS norm of each head with weights and rotation to its token's position, in one pass:
 *   y = R(p) (x r * w),  r = (mean_i x_i^2 + eps)^(-1/2)  over the head's head_dim values, in FP32, rounded once.
 * q, k: num_tokens tokens of heads (kv_heads) heads of head_dim values, bf16 or fp16, 16-byte aligned, values
 * contiguous, token and head strides (in elements) multiples of 8: slices of a fused projection will do.  kv_heads may
 * be 0 (k, k_weight and k_out NULL then).  num_tokens (heads + kv_heads) is at most 2^31 - 1.  head_dim is a multiple of 8, at most 256.  Outputs have strides of their own
 * and may be the inputs themselves (q_out q, k_out k: same address and strides); otherwise they may not overlap an input,
 * each other or themselves (slices of one buffer do not).
 * q_weight, k_weight [head_dim], 16-byte aligned: x's type, or FP32 with weight_f32 = 1.
 * cos_sin float [max_positions][rot_dim], 16-byte aligned: rot_dim / 2 cosines of a position's angles, then their sines.
 * R turns the first rot_dim values of a head (a multiple of 16; 0: none, and cos_sin may be NULL), as pairs
 * (i, rot_dim / 2 + i), or (2i, 2i + 1) with interleaved = 1: (a, b) -> (a cos - b sin, b cos + a sin).
 * positions int32 [num_tokens] (may be NULL with rot_dim 0); -1 leaves a token out: its rows are not written.  Any
 * other position out of range is left out and reported by mx_check.  0 <= eps <= 1.
 */
mx_status qk_norm_rope(const void* q, const void* k, mx_half type, int64_t num_tokens, int64_t heads, int64_t kv_heads,
                       int head_dim, int64_t q_stride_token, int64_t q_stride_head, int64_t k_stride_token,
                       int64_t k_stride_head, const void* q_weight, const void* k_weight, int weight_f32,
                       const float* cos_sin, int64_t max_positions, int rot_dim, const int32_t* positions, float eps,
                       int interleaved, void* q_out, void* k_out, int64_t q_out_stride_token, int64_t q_out_stride_head,
                       int64_t k_out_stride_token, int64_t k_out_stride_head, void* stream);

/* Bytes of workspace qk_norm_rope_backward needs (0 if head_dim is not supported). */
size_t qk_norm_rope_workspace_bytes(int head_dim);

/*
 * qk_norm_rope_backward -- gradients of qk_norm_rope with respect to q, k and the weights.  With g = R(p)^T dy, xh = x r:
 *   dx = r (w g - xh mean(w g xh)),   dw = sum over tokens and heads of g xh.
 * dq_out, dk_out: the results' gradients; q, k: the forward pass's inputs (not its results); all as there, with their
 * own strides.  dq, dk may be dq_out, dk_out themselves, or q, k; otherwise no output, nor the workspace, may overlap
 * an input, another output or itself.  A token that the forward pass left out gets zeros in dq and dk and adds nothing
 * to the weights' gradients, dq_weight and dk_weight, float [head_dim], which are written, not added to, in an order of
 * sums that depends on the sizes alone.  workspace: qk_norm_rope_workspace_bytes bytes, 16-byte aligned, contents need
 * not be initialised; calls that may overlap need one each.  Calls from several host threads on one stream do not
 * overlap, and may share one.
 */
mx_status qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q, const void* k, mx_half type,
                                int64_t num_tokens, int64_t heads, int64_t kv_heads, int head_dim,
                                int64_t dq_out_stride_token, int64_t dq_out_stride_head, int64_t dk_out_stride_token,
                                int64_t dk_out_stride_head, int64_t q_stride_token, int64_t q_stride_head,
                                int64_t k_stride_token, int64_t k_stride_head, const void* q_weight, const void* k_weight,
                                int weight_f32, const float* cos_sin, int64_t max_positions, int rot_dim,
                                const int32_t* positions, float eps, int interleaved, void* dq, void* dk,
                                int64_t dq_stride_token, int64_t dq_stride_head, int64_t dk_stride_token,
                                int64_t dk_stride_head, float* dq_weight, float* dk_weight, void* workspace, void* stream);

/*
 * Trees of drafted tokens.
 *
 * A step may run a tree of tokens for each request: row q_start[r] + i is node i of request r's tree, of at most
 * max_q_len <= 1024 nodes.  Node 0 is the root: the last token that the request has for certain.  A node's parent has
 * a smaller number; parents[] are numbers within the request, -1 has none.  Nodes are cached in order, node i at place
 * lengths[r] - n + i of the request (n its nodes; lengths[r] counts them), which kv_block_tables gives slots for; the
 * position that a node stands for is lengths[r] - n + its depth.  q_start and lengths break their contract as for
 * kv_attention: such a request is left out and reported by mx_check.
 */

/*
 * kv_draft_trees -- what each node sees, and where it stands.
 *   tree_mask[num_tokens][mask_words]: bit j % 64 of word j / 64 is set for the node itself and its ancestors j, with a
 *   window > 0 only for those at a depth greater than its own less the window;
 *   positions[num_tokens] = lengths[r] - n + depth (a node without parent has depth 0).
 * 64 mask_words >= max_q_len, mask_words <= 16.  A request with a parent out of range gets masks of 0 and positions -1,
 * and is reported.  Rows from q_start[requests] on get the same; rows of requests that are left out are not written.
 * Outputs may not overlap inputs or each other, here and in kv_verify_drafts.
 */
mx_status kv_draft_trees(const int32_t* parents, int64_t num_tokens, const int32_t* lengths, const int32_t* q_start,
                         int64_t requests, int64_t max_q_len, int64_t window, int64_t* tree_mask, int64_t mask_words,
                         int32_t* positions, void* stream);

/*
 * kv_tree_attention -- kv_attention of a tree's queries over the cache and over the nodes that they see.
 *
 * As kv_attention, but that of a request's n newest tokens, its nodes, row i sees those whose bits tree_mask has in row
 * q_start[r] + i (kv_draft_trees gives one; any other does, and bits from n on are not looked at), and of the
 * lengths[r] - n tokens in front of them all, or those j > positions[q_start[r] + i] - window with a window > 0.  The
 * nodes follow the mask alone.  positions is read only with a window (NULL will do without) and lies in
 * [lengths[r] - n, lengths[r]); one that does not is reported, and taken as the nearest that does.  A request whose
 * length is less than n breaks its contract.  max_q_len <= 1024, 64 mask_words >= max_q_len, mask_words <= 16.
 * workspace: as for kv_attention, and the same one will do.
 */
mx_status kv_tree_attention(const void* q, mx_half type, int64_t num_tokens, int64_t heads, int64_t q_stride_token,
                            int64_t q_stride_head, const void* k_codes, const void* v_codes, const float* k_scale,
                            const float* v_scale, mx_elem elem, int64_t num_blocks, int64_t kv_heads, int block_tokens,
                            int head_dim, const int32_t* block_tables, int64_t max_blocks, const int32_t* lengths,
                            const int32_t* q_start, int64_t requests, int64_t max_q_len, const int64_t* tree_mask,
                            int64_t mask_words, const int32_t* positions, float softmax_scale, int64_t window, void* out,
                            float* lse, void* workspace, void* stream);

/*
 * kv_verify_drafts -- which drafts stay, and the token behind them.
 *
 * target_probs[num_tokens] are rows of vocab probabilities (FP32, rows target_stride apart): row q_start[r] + i is the
 * target model's distribution of the token that follows node i.  drafts[num_tokens] are the nodes' tokens (the root's is
 * not read).  With draft_probs (rows draft_stride apart) the children of node i were drawn from row i of it, one after
 * the other and independently; without (NULL) they are certain: some tokens, each different from its siblings.
 * From the root on, the children of the last accepted node u are tried in order.  With P = target(u), Z = 1, W = 0,
 * child x (accept_random its number) is accepted if accept_random q(x) Z < P(x), where q = draft(u), and then its
 * children are tried; else W += Z, P = max(target(u) - W q, 0), Z = sum P.  Certain drafts have q(x) = 1: accepted if
 * accept_random Z < P(x), else P(x) = 0 and Z -= P(x).  Behind the last accepted node the next token is the first whose
 * running sum of P is above sample_random[r] sum P; where nothing is left of P (all of it rounds to 0, below), target(u)
 * is drawn from instead.
 * For each request, at its rows from q_start[r] on:
 *   counts[r] = accepted nodes, the root among them (0 for a request without rows);
 *   path[..] = the accepted nodes, the root first, then -1;
 *   tokens[..] = the accepted drafts and then the next token, counts[r] of them, then -1.
 * Rows from q_start[requests] on get -1.  Sums are of whole multiples of 2^-44, to which each P is rounded: no order
 * changes them, and they are within 1.2 vocab 2^-45 of the exact ones (an entry below 2^-46 is never drawn).  Random
 * numbers are in [0, 1).  A probability or random number that is negative, NaN or 2 and above counts as 0 and is reported.
 * A request with a token or parent out of range gets counts 0 and -1, and is reported; one whose P and target are all 0
 * gets -1 as its next token, and is reported.  A sum of P that is 2 or more is reported (its row is no distribution): Z is
 * then just below 2, and from 4096 on the next token is -1.  Requests with broken starts get counts 0.
 * vocab is at most 2^20, probabilities need 4-byte alignment.
 */
mx_status kv_verify_drafts(const float* target_probs, int64_t target_stride, const float* draft_probs, int64_t draft_stride,
                           int64_t vocab, const int32_t* drafts, const int32_t* parents, int64_t num_tokens,
                           const int32_t* q_start, int64_t requests, int64_t max_q_len, const float* accept_random,
                           const float* sample_random, int32_t* path, int32_t* tokens, int32_t* counts, void* stream);

/*
 * kv_cache_compact -- moves the accepted nodes' keys and values together, in place.
 *
 * Node path[q_start[r] + i] of request r, i < counts[r], moves to place lengths[r] - n + i; kept_lengths[r] becomes
 * lengths[r] - n + counts[r], the request's length from then on (give it to kv_block_tables, which takes the blocks
 * behind it back).  path rises and counts[r] <= n <= 1024 (as kv_verify_drafts gives them).  What moves into one block
 * is a run: the block keeps its scale or, where a value would not fit (|value| > MAX scale), raises it to the smallest
 * 2^k that does, and the codes in front of the run are rounded again, as kv_cache_append does; codes whose block has
 * the same scale move as they are.  A block of scale 0 takes the run's own.  Codes from kept_lengths[r] on are left as
 * they were.  A request whose path, counts, blocks, length or starts break their contract is left as it is, keeps
 * lengths[r] and is reported.  Tokens of a block whose scale is out of range become NaN, and have no part in the scale
 * of the block that they move to; a run into such a block is left out; both are reported.  No two requests have a block
 * that is written to in common.  kept_lengths and the keys', values' and scales' tensors may not overlap each other or
 * an input.
 */
mx_status kv_cache_compact(const int32_t* path, const int32_t* counts, int64_t num_tokens, const int32_t* lengths,
                           const int32_t* q_start, int64_t requests, const int32_t* block_tables, int64_t max_blocks,
                           void* k_codes, void* v_codes, float* k_scale, float* v_scale, mx_elem elem, int64_t num_blocks,
                           int64_t kv_heads, int block_tokens, int head_dim, int32_t* kept_lengths, void* stream);

/*
 * mx_check -- synchronizes `stream`, then reads and clears the library's device error word.
 * Returns MX_ERR_TIMEOUT if a kernel's bounded wait ran out since the last check,
 * MX_ERR_INVALID_ARG if the only events were device inputs that broke their contract (a grouped GEMM's
 * offsets, a key/value cache's lengths, query starts, blocks, slots or scales), MX_ERR_CUDA on a pending CUDA error, MX_OK
 * otherwise.  This is the only call that synchronizes.
 */
mx_status mx_check(void* stream);

/* Number of SMs the GEMM kernels size their persistent grids for (0 before the first call
 * that launches a GEMM on the current device). */
int mx_num_sms(void);

#ifdef __cplusplus
}
#endif

#endif /* MXGB_MX_H_ */
