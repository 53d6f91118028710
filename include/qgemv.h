/*
 * qgemv.h -- few-row quantized GEMV for AMD Instinct MI355X (gfx950).
 *
 *   y[M,N] = x[M,K] . dequant(W[N,K])^T,   1 <= M <= 16
 *
 * The verify step of speculative / multi-token-prediction decoding runs a
 * weight matrix against a handful of activation rows ("metal : few-row MMA
 * mat-mul and batched copies for speculative decoding", Overview: 2..16 src1
 * rows; "MLX quantized_matmul small-M verify kernels", Facts: the M=2..12
 * window between qmv and qmm).  This library reads and dequantizes every
 * weight group once per call and reuses it for all M rows, instead of
 * streaming the weights once per row.
 *
 * Weight format (affine group quantization, the "affine" mode of the MLX
 * page's Facts on qmv_wide; 4 B of fp16 scale+bias per group, Facts: the
 * group-size mechanism):
 *   w[n,k] = s[n, k/gs] * q[n,k] + b[n, k/gs]
 *   codes   uint8 [N][K*bits/8], row-major, no padding between rows.
 *           bits = 4: two codes per byte, column k in bits 4*(k%2).. (low
 *           nibble first).  bits = 2: four codes per byte, column k in bits
 *           2*(k%4).. (lowest crumb first).  bits = 8: one code per byte,
 *           the unsigned byte (the int8 affine mode of qmv_wide, MLX page,
 *           Facts: the int8 M=8 speedup).
 *   scales  IEEE fp16 bit patterns [N][K/gs], row-major.
 *   biases  IEEE fp16 bit patterns [N][K/gs], row-major.
 * Activations x: bfloat16 bit patterns [M][K], row-major (weights are stored
 * [out,in], so the product is x @ W^T; MLX page, Facts: (M,5120)@(17408,5120)^T).
 * Output y: fp32 [M][N], row-major, overwritten (no accumulate).
 *
 * Conventions for every entry point:
 *   - All buffer pointers are DEVICE pointers on the current HIP device.  The
 *     caller owns every buffer; the library allocates no device memory,
 *     keeps no mutable state between calls and never synchronizes the host.
 *   - `stream` is a hipStream_t passed as void*; NULL means the null stream.
 *     Work is enqueued asynchronously on it.
 *   - Arguments are validated on the host before anything is launched; on
 *     failure a negative status is returned and nothing is enqueued.
 *   - A kernel launch error reported by the HIP runtime returns QGEMV_EHIP.
 *   - Errors inside a running kernel cannot happen for validated arguments
 *     (all accesses are bounded by M, N, K).
 *   - Calls are reentrant and may run concurrently on different streams.
 */
#ifndef QGEMV_H
#define QGEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define QGEMV_OK 0
#define QGEMV_EINVAL (-1)       /* bad shape / bits / group size / null pointer   */
#define QGEMV_EUNSUPPORTED (-2) /* valid format, but the requested path cannot run it */
#define QGEMV_EALIGN (-3)       /* a buffer pointer is not 16-byte aligned            */
#define QGEMV_EHIP (-4)         /* the HIP runtime rejected a launch                  */

/* Kernel paths. */
#define QGEMV_PATH_AUTO 0 /* let qgemv_select choose                                 */
#define QGEMV_PATH_DOT 1  /* multi-row dot path: one wave per row tile, lanes split K */
#define QGEMV_PATH_MFMA 2 /* split-K bf16 MFMA path: waves split K, LDS reduction    */

/* Limits checked by validation. */
#define QGEMV_MAX_M 16
#define QGEMV_MAX_K 131072
#define QGEMV_MAX_N 4194304
#define QGEMV_MAX_EXPERTS 4096 /* experts per qgemv_gather call */
#define QGEMV_MAX_PAIRS 256    /* (row, expert) pairs per qgemv_gather call */

/*
 * qgemv_small -- y = x . dequant(W)^T for 1 <= M <= 16, path chosen by
 * qgemv_select.
 *
 * Requirements (else QGEMV_EINVAL / QGEMV_EALIGN):
 *   bits in {2, 4, 8}; group_size in {32, 64, 128}; 1 <= M <= 16;
 *   1 <= N <= QGEMV_MAX_N; 64 <= K <= QGEMV_MAX_K; K % 64 == 0;
 *   K % group_size == 0; codes, scales, biases, x, y non-NULL and each
 *   16-byte aligned (every device allocation is).
 * Numerics: products of bf16 activations with exact integer codes are
 * accumulated in fp32 per group; the per-group scale is applied once to the
 * group's partial dot product and the bias once to the group's activation sum
 * (scale hoisted out of the inner loop, MLX page, Facts: the qmv_wide tuning
 * bullet).  Result within 1e-3 * sum_k |x_k w_k| + 1e-6 of the exact value.
 * An output column n whose dequantized weights w[n][*] are all exactly zero
 * gives exactly 0 (exactly r with the residual sum).
 * Results are deterministic (where the MFMA path splits K over two
 * workgroups, y receives exactly two float additions onto zero, which
 * commute bit for bit).  Within one path, row m of an M-row call equals
 * (bitwise) the M=1 call on x[m] whenever both calls run the same kernel
 * configuration, whose per-row accumulation order depends on the shape
 * alone.  One case depends on M: on the MFMA path, with more 16-column
 * tiles than compute units and K too long for the register-resident
 * persistent kernel (K > 4096 for 4-bit codes in groups of 32 or 64, K >
 * 6144 otherwise), the long-K kernel takes its phase count and
 * blocks per wave from an LDS budget that grows with M, and the single-pass
 * kernel runs beyond the largest M that budget holds.  Rows of calls on
 * different sides of such a threshold agree within the tolerance above, not
 * bit for bit (K = 17408, N = 5120, 4-bit, group size 128: M = 1..7, 8..14
 * and 15..16 are three configurations).
 */
int qgemv_small(const uint8_t *codes, const uint16_t *scales, const uint16_t *biases,
                const uint16_t *x, float *y, int M, int N, int K, int bits, int group_size,
                void *stream);

/*
 * qgemv_small_add -- the fused residual sum: y = x . dequant(W)^T + residual,
 * for 1 <= M <= 16, path chosen by qgemv_select (the MUL_MAT + ADD fusion of
 * "metal : few-row MMA mat-mul and batched copies for speculative decoding",
 * Overview: the residual sum is written from the mat-mul's store, saving the
 * separate ADD launch and its read and write of y).
 *
 * residual: fp32 [M][N], row-major, the output's layout; DEVICE pointer,
 * 16-byte aligned, read only.  It may be y itself (in place: y += x W^T);
 * otherwise it must not overlap y (QGEMV_EINVAL).  NULL -> QGEMV_EINVAL.
 * Other arguments, requirements and errors as qgemv_small.
 * Numerics: y[m,n] is the fp32 product that qgemv_small would store for this
 * path, plus residual[m,n] rounded once in fp32 -- bit for bit qgemv_small
 * followed by a separate fp32 add -- except for an in-place call on a shape
 * where the MFMA path splits K across workgroups: that call runs the unsplit
 * kernel (the split needs y prefilled), whose product may differ from the
 * split one in the last bits.  Tolerance against the exact value:
 * 1e-3 * sum_k |x_k w_k| + 1e-6 + 2^-23 * (|r| + sum_k |x_k w_k|).
 * Row m still equals (bitwise) the M=1 call on x[m] and residual[m].
 */
int qgemv_small_add(const uint8_t *codes, const uint16_t *scales, const uint16_t *biases,
                    const uint16_t *x, const float *residual, float *y, int M, int N, int K,
                    int bits, int group_size, void *stream);

/*
 * qgemv_run_path_add -- qgemv_small_add with an explicit path (as
 * qgemv_run_path).
 */
int qgemv_run_path_add(int path, const uint8_t *codes, const uint16_t *scales,
                       const uint16_t *biases, const uint16_t *x, const float *residual, float *y,
                       int M, int N, int K, int bits, int group_size, void *stream);

/*
 * qgemv_select -- the path qgemv_small takes for this shape: QGEMV_PATH_DOT or
 * QGEMV_PATH_MFMA, or a negative status if the shape is invalid.  The choice
 * comes from a crossover table measured on MI355X (which rows of a shape
 * family favour the MFMA path), in the spirit of the per-type start rows of
 * the few-row MMA PR (Overview) and MLX's per-shape qmv batch limit (MLX page,
 * Facts: get_qmv_batch_limit), but calibrated on CDNA4.  Pure host function;
 * touches no device.
 */
int qgemv_select(int M, int N, int K, int bits, int group_size);

/*
 * qgemv_run_path -- qgemv_small with an explicit path (QGEMV_PATH_AUTO,
 * QGEMV_PATH_DOT or QGEMV_PATH_MFMA), for forced-path sweeps and tests (the
 * pages' A/B knobs: the specgate-metal README's GGML_METAL_NO_MV_EXT /
 * GGML_METAL_MM_MIN; MLX page, Facts: forced qmv vs qmm sweeps).
 * Returns QGEMV_EUNSUPPORTED if the path cannot run the shape (the MFMA path
 * needs K to be a multiple of 256 (2-bit) / 128 (4-bit) / 64 (8-bit), and
 * group_size >= 64 for 2-bit codes; K a multiple of 4*group_size, or for 2-
 * and 4-bit codes at least 4 groups, the remainder then running as a partial
 * last block of the single-pass MFMA kernel).  Other arguments as
 * qgemv_small.
 */
int qgemv_run_path(int path, const uint8_t *codes, const uint16_t *scales,
                   const uint16_t *biases, const uint16_t *x, float *y, int M, int N, int K,
                   int bits, int group_size, void *stream);

/*
 * qgemv_path_supported -- 1 if `path` can run this shape, 0 if not, negative
 * status if the shape itself is invalid.  Host only.
 */
int qgemv_path_supported(int path, int M, int N, int K, int bits, int group_size);

/*
 * qgemv_unpack_probe -- writes the integer codes exactly as a path's kernels
 * decode them: q_out[n][k] (uint8, [N][K], row-major) for every n < N, k < K.
 * The kernels turn codes into exact bf16 values q in registers; this probe
 * runs the same device routines (same loads, lane exchanges and conversions;
 * on the MFMA path both of its load forms, which must agree) and writes back
 * q, so the decoded codes can be compared bit-exactly with the format's
 * definition.  path: QGEMV_PATH_DOT or QGEMV_PATH_MFMA (the two
 * paths pair codes differently).  Requirements as qgemv_run_path for that
 * path (group_size only selects the MFMA layout, pass the one you will use);
 * q_out non-NULL.
 */
int qgemv_unpack_probe(int path, const uint8_t *codes, uint8_t *q_out, int N, int K, int bits,
                       int group_size, void *stream);

/*
 * qgemv_stream_probe -- read-only streaming kernel over `nbytes` bytes of
 * `buf` (16-byte aligned, nbytes a multiple of 16): every byte is loaded once
 * with non-temporal 128-bit loads (1 KiB contiguous per wave instruction,
 * `loads_per_thread` loads in flight per thread: 1, 2, 4, 8 or 16), folded with
 * XOR, and one uint32 per 256-thread workgroup is written to
 * out[0 .. qgemv_stream_probe_blocks(nbytes)-1] (enough for every setting;
 * the XOR of all of them is the XOR of the buffer's 32-bit words).
 * layout 0: a thread's loads are one grid-width apart; layout 1: they are
 * 1 KiB apart, so that each wave reads loads_per_thread KiB in one piece.
 * The fastest setting at a byte count is the bandwidth ceiling a pure read of
 * that many bytes reaches, measured the same way as the GEMV kernels.
 * EINVAL for another loads_per_thread or layout.
 */
int qgemv_stream_probe(const uint8_t *buf, size_t nbytes, uint32_t *out, int loads_per_thread,
                       int layout, void *stream);
int qgemv_stream_probe_blocks(size_t nbytes);

/*
 * ---------------------------------------------------------------- FP block formats
 *
 * The block-scaled floating-point modes of qmv_wide (MLX page, Facts: qmv_wide
 * covers affine, nvfp4, mxfp4 and mxfp8, with their M=8 speedups on the
 * Gemma-4-12B gate/up shape).  Element and scale encodings follow the OCP
 * Microscaling Formats (MX) v1.0 specification:
 *   QGEMV_FMT_MXFP4  FP4 E2M1 elements, two per byte (low nibble first);
 *                    one E8M0 scale byte (2^(e-127)) per 32 elements.
 *   QGEMV_FMT_NVFP4  FP4 E2M1 elements as above; one FP8 E4M3 scale byte per
 *                    16 elements (no per-tensor scale: a constant factor the
 *                    caller can apply to y).
 *   QGEMV_FMT_MXFP8  FP8 E4M3 elements (OCP: bias 7, no infinities, S.1111.111
 *                    NaN), one per byte; one E8M0 scale byte per 32 elements.
 * w[n,k] = scale[n, k/block] * element[n,k]; no bias.
 *   codes   uint8 [N][K*bits/8] (bits = 4 or 8), row-major, 16-byte aligned.
 *   scales  uint8 [N][K/block], row-major, 16-byte aligned.
 *   x       bf16 [M][K]; y fp32 [M][N] as for qgemv_small.
 *   residual  NULL for the plain product, else fp32 [M][N] added in the
 *           store exactly as qgemv_small_add (may be y itself, else must not
 *           overlap it).
 * Requirements (else QGEMV_EINVAL / QGEMV_EALIGN): format one of the three;
 * 1 <= M <= 16; 1 <= N <= QGEMV_MAX_N; 64 <= K <= QGEMV_MAX_K, K % 64 == 0.
 * The MFMA path needs K % 128 == 0.  Elements are decoded exactly (every E2M1
 * and E4M3 value is a bf16 value); each block's scale is applied once in fp32
 * to the block's partial dot product, except on the MFMA path for nvfp4, where
 * each element is multiplied by its E4M3 block scale before the product (the
 * product of an E4M3 and an E2M1 value is itself exact in bf16).  Tolerance
 * and row invariance as qgemv_small.
 */
#define QGEMV_FMT_MXFP4 1
#define QGEMV_FMT_NVFP4 2
#define QGEMV_FMT_MXFP8 3

int qgemv_small_fp(const uint8_t *codes, const uint8_t *scales, const uint16_t *x,
                   const float *residual, float *y, int M, int N, int K, int format,
                   void *stream);

/* qgemv_run_path_fp -- qgemv_small_fp with an explicit path (as qgemv_run_path). */
int qgemv_run_path_fp(int path, const uint8_t *codes, const uint8_t *scales, const uint16_t *x,
                      const float *residual, float *y, int M, int N, int K, int format,
                      void *stream);

/* qgemv_select_fp / qgemv_path_supported_fp -- as qgemv_select /
 * qgemv_path_supported, for an FP format.  Host only. */
int qgemv_select_fp(int M, int N, int K, int format);
int qgemv_path_supported_fp(int path, int M, int N, int K, int format);

/*
 * qgemv_unpack_probe_fp -- writes the element values exactly as a path's
 * kernels decode them, as bf16 bit patterns: out[n][k] (uint16, [N][K]), before
 * the block scale is applied, for the bit-exact test of the decoding.
 */
int qgemv_unpack_probe_fp(int path, const uint8_t *codes, uint16_t *out, int N, int K, int format,
                          void *stream);

/*
 * qgemv_gather -- gathered (MoE) verify over (activation row, expert) pairs:
 *
 *   y[p] = x[x_idx[p]] . dequant(W[e_idx[p]])^T,   0 <= p < P
 *
 * the MoE form of the verify product (MLX page, Facts: dense and MoE
 * gather_qmm verify; the expert-union cost per verify row).  Every expert in
 * the union of e_idx is read and dequantized once per call for all the pairs
 * routed to it, instead of once per pair.
 *   codes   uint8 [E][N][K*bits/8]; scales, biases fp16 [E][N][K/group_size]:
 *           E matrices in the affine format of qgemv_small, one after another.
 *   x       bf16 [X][K] activation rows.
 *   x_idx, e_idx  int32 [P], DEVICE arrays (the routing stays on the device):
 *           the activation row and the expert of each pair.
 *   y       fp32 [P][N], row p written for every valid pair.
 * A pair whose x_idx is outside [0, X) or e_idx outside [0, E) is skipped and
 * its row of y is left unchanged (the indices are read on the device; the
 * host cannot check them without a synchronization).
 * Requirements (else QGEMV_EINVAL / QGEMV_EALIGN / QGEMV_EUNSUPPORTED):
 * shape and format as qgemv_run_path with the MFMA path (bits, group_size, N,
 * K, and the MFMA path's K requirements); 1 <= P <= QGEMV_MAX_PAIRS;
 * 1 <= E <= QGEMV_MAX_EXPERTS; X >= 1; pointers non-NULL, codes, scales,
 * biases, x and y 16-byte aligned, x_idx and e_idx 4-byte aligned.
 * Runs on an MFMA kernel (any number of pairs per expert, 16 rows at a
 * time): the single-pass one for X <= 2, the persistent one for X >= 3 where
 * the shape fits it.  Each pair's row has the numerics of the MFMA path
 * (within the tolerance of qgemv_small; its K split over waves is the
 * kernel's own, so it may differ from a dense call, and between the two
 * kernels, in the last bits), is deterministic, and does not depend on the
 * other pairs of the call (bitwise the same as a call with the same x and X
 * and that pair alone).
 */
int qgemv_gather(const uint8_t *codes, const uint16_t *scales, const uint16_t *biases,
                 const uint16_t *x, const int32_t *x_idx, const int32_t *e_idx, float *y, int P,
                 int X, int E, int N, int K, int bits, int group_size, void *stream);

/*
 * ---------------------------------------------------------------- verify step around the products
 *
 * What a verify step does between the quantized products: append the new
 * rows' keys and values to a paged cache, attend from those rows over the
 * cache, and accept or refuse the drafted tokens.
 *
 * Rows of several sequences lie one after another: sequence b owns the rows
 * start[b] .. start[b+1]-1 of T (its last accepted token and the drafts after
 * it), and len[b] counts its tokens, those rows included, so that row t is
 * the token at position len[b] - (start[b+1] - t).  start (int32 [B+1],
 * ascending) and len (int32 [B]) are DEVICE arrays: the host reads neither,
 * and every value that comes from them or from the page table is checked on
 * the device before it forms an address.  A length below 0 counts as 0, one
 * past QGEMV_MAX_CONTEXT as that; a start below 0 as 0, one past T as T, in
 * every call alike.  Where starts descend, it is not defined which sequence has
 * the rows between them; the append stores none of them.
 *
 * Element types of these entry points.
 */
#define QGEMV_F32 0
#define QGEMV_BF16 1
#define QGEMV_F16 2
#define QGEMV_E4M3 3 /* OCP FP8 E4M3, no infinity */

#define QGEMV_MAX_GROUP 64         /* query heads on one key-value head          */
#define QGEMV_MAX_CONTEXT (1 << 30) /* tokens of one sequence (page * width)      */
#define QGEMV_MAX_VOCABULARY (1 << 24)

/*
 * A paged cache: page p holds `page` slots, each with a key and a value of
 * `dim` elements for each of `heads` heads.  The token at position j of
 * sequence b lies in slot j % page of page table[b * width + j / page].
 * Slot s, head h of page p starts at byte p * stride_page + s * stride_slot +
 * h * stride_head of k and of v (the same strides for both), so a cache
 * [page][slot][head][dim] and one [page][head][slot][dim] are both described.
 *   dtype    QGEMV_BF16, QGEMV_F16, or QGEMV_E4M3 with k_scale and v_scale
 *            (fp32 [heads], DEVICE; the key is the stored value times its
 *            head's scale; NULL otherwise).
 *   Requirements (else QGEMV_EINVAL / QGEMV_EALIGN): dim 64, 128 or 256;
 *   heads, pages, page, width and batch at least 1; page * width at most
 *   QGEMV_MAX_CONTEXT; strides positive multiples of 16; k and v 16-byte,
 *   table and scales 4-byte aligned.
 * A table entry outside [0, pages) is a page that is not there: a row
 * appended to it is dropped, and its tokens are seen by no row.  A token past
 * the table's width is treated alike: where a sequence's length passes the
 * table, its rows keep their positions, those past the table's end are not
 * stored and see what of their range is there.
 */
typedef struct qgemv_kv_cache {
  void *k, *v;
  const int32_t *table;
  const float *k_scale, *v_scale;
  int64_t stride_page, stride_slot, stride_head;
  int32_t pages, page, width, batch, heads, dim, dtype;
} qgemv_kv_cache;

/*
 * qgemv_kv_append -- K[slot of row t][h] = cast(new_k[t][h]), and V alike, for
 * the T rows of all sequences.
 *   new_k, new_v  [T][heads][dim] of src_dtype (QGEMV_F32, QGEMV_BF16 or
 *           QGEMV_F16; the products' fp32 output can be passed as it is);
 *           row and head strides in elements, dim contiguous.
 * A value is rounded once, to nearest even.  For an E4M3 cache it is divided
 * by its head's scale (one fp32 rounding) and limited to +-448 first.  NaN
 * stays NaN.  Rows with a negative position are dropped.  Two rows that are
 * given the same slot leave either's value there.
 * T = 0 does nothing; 2^24 rows and more, or more than 2^30 values of a row's
 * keys, are too many (QGEMV_EUNSUPPORTED).
 * Strides must be multiples of 16 bytes and pointers 16-byte aligned
 * (QGEMV_EALIGN).
 */
int qgemv_kv_append(const qgemv_kv_cache *cache, const void *new_k, int64_t k_row, int64_t k_head,
                    const void *new_v, int64_t v_row, int64_t v_head, int src_dtype,
                    const int32_t *start, const int32_t *len, int T, void *stream);

/*
 * qgemv_kv_attend -- attention of the T new rows over the cache, for
 * q_heads = G * heads query heads (query head hq reads key-value head hq / G):
 *
 *   s_j = scale * (q . k_j),  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j)
 *
 * over the tokens j that the row at position pos sees: j <= pos, and where
 * window > 0 also j > pos - window or j < sinks.  window = 0: all of them.
 * A row that sees nothing gives 0 and -inf.  What an unseen slot holds (NaN
 * and infinities too) does not reach a result.
 *   q, out  [T][q_heads][dim] of q_dtype (QGEMV_BF16 or QGEMV_F16; a 16-bit
 *           cache has the same type), row and head strides in elements, dim
 *           contiguous, strides multiples of 16 bytes, 16-byte aligned.
 *   lse     fp32 [T][q_heads] (natural logarithm), or NULL.
 *   M       the largest number of rows of a sequence, 1..QGEMV_MAX_M (a
 *           sequence's rows past M are left unwritten).
 *   workspace  qgemv_kv_attend_workspace bytes, 16-byte aligned, contents
 *           free; not shared by calls that may run at the same time.  The size
 *           for M rows is enough for every smaller M and every window over the
 *           same cache.
 * Scores, softmax statistics and sums are fp32.  The weights exp(s_j - ..) are
 * rounded to q_dtype for the product with the values, after their fp32 sum has
 * taken them: half a step each, relative to the weight; in fp16, weights below
 * 2^-21 of the largest lose further bits, and those below 2^-32 count as 0
 * beside the values.  Results are deterministic.
 * The launch follows from the sizes alone (page * width, the window, M, the
 * batch), since lengths are on the device: over a table much wider than the
 * sequences a call costs a few us more than over one as wide as the longest.
 * 2^24 items (sequences times key-value heads times groups of 64..256 rows) or
 * 2^30 pieces of work, counted as if every sequence filled the table, are too
 * many (QGEMV_EUNSUPPORTED).
 */
int64_t qgemv_kv_attend_workspace(const qgemv_kv_cache *cache, int M, int q_heads, int T);
int qgemv_kv_attend(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head,
                    void *out, int64_t out_row, int64_t out_head, int q_dtype, float *lse,
                    const int32_t *start, const int32_t *len, int T, int M, int q_heads, int window,
                    int sinks, float scale, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * qgemv_kv_attend_shared -- qgemv_kv_attend for sequences that begin with the
 * same tokens in the same pages (a common prompt), whose keys and values are
 * read once for all of them.
 *   shared  int32 [1], DEVICE: how many tokens the sequences have in common.
 *           Its whole pages, at most all of the table's but the last column,
 *           are read through the first sequence's table row; the caller has
 *           them in every row alike.  0 or less: none.  A length may end before
 *           them.
 * Other arguments, requirements and results as qgemv_kv_attend; rows of no
 * sequence are left unwritten.  The two ways to compute a row agree within the
 * roundings named there, not bit for bit.
 *   workspace  qgemv_kv_attend_shared_workspace bytes: enough for every smaller
 *           M and T and every window over the same cache.
 * Besides the limits there, 2^30 rows times query heads on a key-value head and
 * 2^30 pieces of the common part are too many (QGEMV_EUNSUPPORTED).
 */
int64_t qgemv_kv_attend_shared_workspace(const qgemv_kv_cache *cache, int M, int q_heads, int T);
int qgemv_kv_attend_shared(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head,
                           void *out, int64_t out_row, int64_t out_head, int q_dtype, float *lse,
                           const int32_t *start, const int32_t *len, const int32_t *shared, int T, int M,
                           int q_heads, int window, int sinks, float scale, void *workspace,
                           int64_t workspace_bytes, void *stream);

/*
 * qgemv_kv_append_rotated -- qgemv_kv_append with the rotation of positions on
 * the way, and the queries rotated for the attention after it:
 *
 *   angle(t, i) = p(t, axis(i)) * freq[i]                       0 <= i < pairs
 *   (a, b) -> (a cos angle - b sin angle, a sin angle + b cos angle)
 *
 * of the pairs of each query and key: values i and pairs + i of a head, or with
 * interleaved 2 i and 2 i + 1; a head's values from 2 * pairs on, and all of
 * new_v, stay.
 *   q       [T][q_heads][dim] of src_dtype; out the same of out_dtype
 *           (QGEMV_BF16 or QGEMV_F16), its values all in places of their own:
 *           q itself (same type and strides), or apart from it, and apart from
 *           new_k and new_v: before or after them, or other columns, first to
 *           last, of rows as many bytes apart, or of heads where those of all
 *           rows are equally far apart (QGEMV_EINVAL).  Rows of no sequence are
 *           left unwritten.
 *   freq    fp32 [pairs], DEVICE; pairs a multiple of 8, at most dim / 2.
 *   position  int32 [axes][T], DEVICE, axes position_axis elements apart: the
 *           rows' positions on each axis; NULL: one axis, a row's place in its
 *           sequence.
 *   axis    int32 [pairs], DEVICE, limited to 0 .. axes - 1: the axis of each
 *           pair; NULL: the first.  NULL where position is.
 * cos and sin are fp32, within 2^-22 where |p(t, i) * freq[i]| < 2^40; a rotated
 * value is rounded to fp32 and then once to its type.  Other arguments,
 * requirements and errors as qgemv_kv_append.
 */
int qgemv_kv_append_rotated(const qgemv_kv_cache *cache, const void *q, int64_t q_row, int64_t q_head, int q_heads,
                            void *out, int64_t out_row, int64_t out_head, int out_dtype, const void *new_k,
                            int64_t k_row, int64_t k_head, const void *new_v, int64_t v_row, int64_t v_head,
                            int src_dtype, const int32_t *start, const int32_t *len, int T, const float *freq,
                            int pairs, const int32_t *position, int64_t position_axis, int axes,
                            const int32_t *axis, int interleaved, void *stream);

/*
 * qgemv_route -- the experts of each row and their weights; experts [T * k] is
 * what qgemv_gather takes as e_idx.
 *
 *   score_e  = exp(x_e) / sum exp(x)  (QGEMV_SOFTMAX)  or  1 / (1 + exp(-x_e))
 *   choice_e = score_e + bias_e
 *
 * The E experts make `groups` groups of neighbours.  Of these the `keep` whose
 * `best` (1 or 2) greatest choices have the greatest sum remain, and of their
 * experts the k of greatest choice, in that order; equal ones by their number.
 * weights are scale times the scores (without the bias), with renormalise over
 * their sum (0 where that is 0).
 *   logits  [T][E] of QGEMV_F32, QGEMV_BF16 or QGEMV_F16, row stride `row`
 *           elements.  An expert whose logit is -inf or NaN, or whose choice
 *           is, is not there: it has no part in the softmax (its logit) and is
 *           not chosen, nor is a group of such.  Where fewer than k are there,
 *           the list ends with -1 (which qgemv_gather skips) and weight 0.  A
 *           logit of +inf leaves a row's softmax without values: weights NaN
 *           where the logits choose (below), no expert where the scores do.
 *   bias    fp32 [E], DEVICE, or NULL.
 * Scores and choices are fp64; without a bias and with best = 1 the choice is
 * by the logits themselves, which their scores' order is.  Choices count as
 * equal within 2^-48 of their value.  Deterministic.
 * At most QGEMV_MAX_ROUTED experts, QGEMV_MAX_GROUPS groups, k of
 * QGEMV_MAX_CHOSEN (QGEMV_EUNSUPPORTED) and of the experts of `keep` groups
 * (QGEMV_EINVAL); 2^24 rows are too many.
 */
#define QGEMV_SOFTMAX 0
#define QGEMV_SIGMOID 1
#define QGEMV_MAX_ROUTED 1024
#define QGEMV_MAX_GROUPS 64
#define QGEMV_MAX_CHOSEN 64
int qgemv_route(const void *logits, int64_t row, int dtype, const float *bias, int32_t *experts, float *weights,
                int T, int E, int k, int score, int groups, int keep, int best, int renormalise, float scale,
                void *stream);

/*
 * qgemv_adapt -- low-rank adapters of many requests beside a shared projection:
 *
 *   out[t] = y[t] + scales[a] * B[a] (A[a] x[t]),   a = adapter[t]
 *
 *   y, out  fp32 [T][N], row strides in elements, 4-byte aligned: a product's
 *           output, or columns of it.  out may be y itself (rows without an
 *           adapter are then not touched), otherwise it must not overlap it:
 *           before or after it, or other columns of rows as far apart.
 *   x       [T][K] of QGEMV_BF16 or QGEMV_F16, the product's activations, row
 *           stride a multiple of 8 elements.
 *   a, b    [n][r][K] and [n][N][r] of the same type, packed: the adapters.  K
 *           and r multiples of 8, r at most QGEMV_MAX_RANK; an adapter of
 *           lower rank is one with rows and columns of zeros.
 *   adapter int32 [T], DEVICE: each row's, or none where outside [0, n).
 *   scales  fp32 [n], DEVICE, or NULL: 1.
 *   workspace  qgemv_adapt_workspace bytes, 16-byte aligned, contents free;
 *           enough for every smaller T and r; not shared by calls that may run
 *           at the same time.
 * x, a, b 16-byte aligned.  Products of 16-bit values are summed in fp32; the
 * rank's sums enter the second product in 16-bit parts that have their 24 bits
 * (in fp16 22 bits of the row's largest).  Deterministic, and
 * a row's result does not depend on the other rows' values.  2^24 rows are
 * too many.
 */
#define QGEMV_MAX_RANK 256
int64_t qgemv_adapt_workspace(int T, int r);
int qgemv_adapt(const float *y, int64_t y_row, float *out, int64_t out_row, const void *x, int64_t x_row,
                const void *a, const void *b, int dtype, const int32_t *adapter, const float *scales, int T, int n,
                int r, int K, int N, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * qgemv_verify_drafts -- which drafted tokens of each sequence are accepted,
 * and the token after them.
 *   p       [T][V] target probabilities after row t (QGEMV_F32, QGEMV_BF16 or
 *           QGEMV_F16), row stride p_row elements;
 *   q       the draft model's probabilities the draft of row t was drawn
 *           from, same type, row stride q_row; NULL where drafts have none
 *           (each then counts as drawn with probability 1).
 *   tokens  int32 [T], the token fed at row t: the draft checked against row
 *           t is tokens[t+1] of the same sequence.
 *   u       fp32 [T], uniform in [0, 1): row t's number decides on its draft,
 *           the last row's draws the token.
 * The draft d of row t is accepted while u[t] * q[t][d] < p[t][d].  At the
 * first refusal, row r, weights are w = max(p[r] - q[r], 0) (q NULL: p[r]
 * with the refused token's set to 0), or p[r] where those sum to 0; without a
 * refusal w = p of the last row.  The token is the first i whose running sum
 * w[0] + .. + w[i] exceeds u[last row] * sum(w); V - 1 where none does, 0
 * where that product is NaN.  Products and sums are fp64; where their rounding
 * decides, the token is a neighbour that has a weight, never one without.
 *   out     int32 [T]: the accepted drafts of each sequence, the drawn token,
 *           then -1; count int32 [B]: accepted drafts + 1 (0 for a sequence
 *           without rows).
 *   M       the largest number of rows of a sequence, 1..QGEMV_MAX_M (rows
 *           past M are not looked at and left unwritten).
 *   workspace  qgemv_verify_drafts_workspace bytes, 16-byte aligned, filled
 *           with zeros once before its first use (every call leaves it fit
 *           for the next, of any size that it has the bytes for); not shared
 *           by calls that may run at the same time.
 * A draft outside [0, V) is refused.  Deterministic; a sequence's answer does
 * not depend on the others.  2^24 sequences and more are too many
 * (QGEMV_EUNSUPPORTED).
 */
int64_t qgemv_verify_drafts_workspace(int B, int V);
int qgemv_verify_drafts(const void *p, int64_t p_row, const void *q, int64_t q_row, int dtype,
                        const int32_t *tokens, const float *u, const int32_t *start, int32_t *out,
                        int32_t *count, int B, int T, int M, int V, void *workspace,
                        int64_t workspace_bytes, void *stream);

/* qgemv_strerror -- static description of a status code. */
const char *qgemv_strerror(int status);

/* qgemv_version -- library ABI version (major*10000 + minor*100 + patch). */
int qgemv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_H */
