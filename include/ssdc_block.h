/*
 * ssdc_block.h -- C ABI of the operators around the scan, in libssdc.so: what a
 * block needs before and after its recurrence, in training and in serving.
 *
 *   gated scan      the real-valued sibling of the complex scan: one gated
 *                   linear recurrence per channel, forward, one token at a
 *                   time, and the gradients
 *   residual norm   residual addition and root-mean-square norm, with an output
 *                   in 8 bits and a scale for each 128 features; the gradients
 *   8-bit product   C = A B^T from e4m3 values with a scale for each group or
 *                   block of 128, and the quantisers that make its operands
 *
 * Conventions are those of ssdc.h: status codes, no aborts, argument errors
 * found on the host before anything is enqueued, the caller owns every buffer,
 * work is enqueued on `stream`. All pointers are device pointers, aligned to
 * their element (the state, scale and weight arrays are float). A stride that is
 * never taken (of a single row, token or batch row) may be anything. Types:
 */
#ifndef SSDC_BLOCK_H
#define SSDC_BLOCK_H

#include "ssdc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_TYPE_F32 0
#define SSD_TYPE_BF16 1
#define SSD_TYPE_E4M3 2 /* 8 bits: sign, 4 exponent, 3 mantissa bits; largest value 448 */

/* Values that share a scale in the 8-bit layouts. */
#define SSD_FP8_GROUP 128

/*
 * Gated scan. For every batch row b and channel d, independently:
 *
 *   a_t = sigmoid(f_t)
 *   c_t = a_t, or 0 where reset[b, t] is not zero (the first token of a document
 *         in a packed row: nothing is carried into it)
 *   v_t = sigmoid(i_t) x_t, or (1 - a_t) x_t without an input gate
 *   h_t = c_t h_{t-1} + v_t,   h_{-1} = h0 (zero without one)
 *
 * x, f, i, h and the gradients hold `type` (F32 or BF16) values; gates, sums and
 * states are fp32. A sequence array is given by its first element and the
 * element strides of batch rows and tokens; channels are contiguous. So the
 * three inputs may be column slices of one projection's output, and either
 * order of batch and time works. Input strides may be zero (broadcast rows); a
 * token stride of 2^31 bytes or more is SSDC_ERR_UNSUPPORTED. Fastest are arrays
 * whose rows, strides and first elements are whole 16-byte units and whose batch
 * rows are further apart than their tokens.
 */
typedef struct {
    const void *p;
    int64_t stride_b, stride_t;
} ssd_seq_in;
typedef struct {
    void *p;
    int64_t stride_b, stride_t;
} ssd_seq_out;
typedef struct {
    int64_t B, T, D; /* batch rows, tokens, channels; B D up to 2^31 - 1 */
    int32_t type;    /* SSD_TYPE_F32 or SSD_TYPE_BF16 */
} ssd_gated_dims;

/*
 * Forward pass.
 *   x, f      inputs;  i: input gate, or i.p NULL (coupled gates)
 *   h0        (B, D) dense fp32, or NULL: zero
 *   reset     (B, T) dense bytes, or NULL
 *   h         output;  it must not overlap an input
 *   h_last    output (B, D) fp32, the state after the last token; it may be h0
 *   states    output for the backward pass, or NULL:
 *             ssd_gated_scan_states_bytes() bytes, the state entering every
 *             SSD_GATED_STATE_TOKENS-th token, (B, ceil(T / that), D) fp32
 *   status    a device word, or NULL. The CTAs of a cluster wait for one another for
 *             two seconds at most; a wait that gives up sets the word to
 *             SSDC_ERR_TIMEOUT, and the results are NaN. The caller zeroes it once
 *             (ssd_complex_status() reads it)
 * One launch. Results do not depend on timing: sums run in a fixed order.
 *
 * ssd_gated_scan_fwd_ws: the same with a workspace of ssd_gated_scan_workspace_bytes() (16-byte
 * aligned; its contents need not be kept). Where sequences are long and too few for the GPU,
 * those are cut into segments that are walked at the same time, in two launches; elsewhere the
 * size is 0, and the call is the one above.
 */
#define SSD_GATED_STATE_TOKENS 64
size_t ssd_gated_scan_states_bytes(ssd_gated_dims dims);
int ssd_gated_scan_fwd(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float *h0, const uint8_t *reset,
                       ssd_gated_dims dims, ssd_seq_out h, float *h_last, float *states, int32_t *status,
                       cudaStream_t stream);

size_t ssd_gated_scan_workspace_bytes(ssd_gated_dims dims);
int ssd_gated_scan_fwd_ws(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float *h0, const uint8_t *reset,
                          ssd_gated_dims dims, ssd_seq_out h, float *h_last, float *states, int32_t *status,
                          void *workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * One token for every batch row (the forward pass at T = 1, for generation):
 * state_out = c state_in + v, h = state_out in `type`. state_out may be state_in.
 * The token strides of the sequences are not used. One launch.
 */
int ssd_gated_scan_step(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float *state_in, int64_t B, int64_t D,
                        int32_t type, ssd_seq_out h, float *state_out, cudaStream_t stream);

/*
 * Backward pass: with g_t the gradient of h_t after all later tokens,
 *   g_t = dh_t + c_{t+1} g_{t+1}   (dh_last added at the last token)
 *   dx_t = s g_t (s the input's factor: sigmoid(i_t), or 1 - a_t)
 *   df_t = a_t (1 - a_t) g_t h_{t-1} (0 at a reset), and - a_t (1 - a_t) g_t x_t
 *          more without an input gate
 *   di_t = x_t s (1 - s) g_t,   dh0 = c_0 g_0
 *   states    what the forward pass kept for the same inputs (h0 is in it)
 *   dh        gradient of h;  dh_last (B, D) fp32, or NULL: zero
 *   di        given exactly with i;  dh0: (B, D) fp32, or NULL: not written; it
 *             may be dh_last;  status: as for the forward pass
 * The states inside a chunk are recomputed in fp32 from `states`. One launch.
 */
int ssd_gated_scan_bwd(ssd_seq_in x, ssd_seq_in f, ssd_seq_in i, const float *states, const uint8_t *reset,
                       ssd_seq_in dh, const float *dh_last, ssd_gated_dims dims, ssd_seq_out dx, ssd_seq_out df,
                       ssd_seq_out di, float *dh0, int32_t *status, cudaStream_t stream);

/*
 * Residual norm over M rows of D features:
 *   r = x + residual (r = x without one),  rstd = 1 / sqrt(mean(r^2) + eps),
 *   y = r rstd w
 * in fp32; r is rounded to `type` when it is written, y is made from the
 * unrounded sum.
 *   x, residual   rows of `type` values, ld elements apart; residual.p may be NULL
 *   w             (D) fp32, or NULL: ones
 *   r             output rows of `type`, or p NULL: not written. It may be x or
 *                 residual itself
 *   y             output rows of `out_type`: F32, BF16, or E4M3: then
 *                   scale[g * M + m] = max(max |y| over the group, 2^-100) / 448
 *                   q = y / scale, rounded to nearest, ties to even
 *                 for the group g of features 128 g .. 128 g + 127 of row m, the
 *                 layout that ssd_fp8_matmul reads. A row that holds an infinity
 *                 or a NaN gives NaN where its values do
 *   rstd          output (M) fp32, or NULL
 * D up to 32768. One launch.
 */
typedef struct {
    const void *p;
    int64_t ld;
} ssd_rows_in;
typedef struct {
    void *p;
    int64_t ld;
} ssd_rows_out;
int ssd_residual_norm_fwd(ssd_rows_in x, ssd_rows_in residual, const float *w, float eps, int64_t M, int64_t D,
                          int32_t type, ssd_rows_out r, int32_t out_type, ssd_rows_out y, float *scale,
                          float *rstd, cudaStream_t stream);

/*
 * Its gradients. With xh = r rstd and gy = dy w:
 *   dx = dr + rstd (gy - xh mean(gy xh))   (the gradient of x and of residual)
 *   dw = sum over rows of dy xh
 *   dy, dr, r   rows of `type`; dr.p may be NULL (zero). r: what the forward pass
 *               wrote;  rstd (M) fp32 likewise
 *   dx          output rows of `type`; it may be dy or dr itself
 *   dw          output (D) fp32, or NULL
 *   workspace   ssd_residual_norm_bwd_workspace_bytes(M, D) bytes, 256-byte
 *               aligned, no initialisation needed (NULL without dw)
 * dw is summed in a fixed order. One launch, and one more for dw.
 */
size_t ssd_residual_norm_bwd_workspace_bytes(int64_t M, int64_t D);
int ssd_residual_norm_bwd(ssd_rows_in dy, ssd_rows_in dr, ssd_rows_in r, const float *w, const float *rstd,
                          int64_t M, int64_t D, int32_t type, ssd_rows_out dx, float *dw, void *workspace,
                          size_t ws_bytes, cudaStream_t stream);

/*
 * 8-bit layouts. An operand of R rows and C columns is held as e4m3 values in
 * rows of ld bytes (ld a multiple of 16, at least C; the bytes past C are never
 * read) and fp32 scales; an element's value is its e4m3 value times its scale:
 *   SSD_SCALE_ROWS    scale[g * R + r] for the columns 128 g .. of row r
 *   SSD_SCALE_BLOCKS  scale[(r / 128) * ceil(C / 128) + c / 128]
 *
 * ssd_fp8_quantize makes them from x, M rows of K values of `type`. The scale of a
 * group or block is max(max |x|, 2^-100) / 448; the e4m3 value is x / scale
 * rounded to nearest, ties to even. q is the operand (M, K), qt the transposed one
 * (K, M) with its groups along M (for SSD_SCALE_BLOCKS its values are those of q);
 * either may have p NULL. One launch; x is read once.
 */
#define SSD_SCALE_ROWS 0
#define SSD_SCALE_BLOCKS 1
int ssd_fp8_quantize(ssd_rows_in x, int64_t M, int64_t K, int32_t type, int32_t scales, ssd_rows_out q,
                     float *scale, ssd_rows_out qt, float *scale_t, cudaStream_t stream);

/*
 * C[m, n] = sum_k A[m, k] B[n, k] over the operands' values: the e4m3 products
 * of 128 columns are summed on the tensor cores, then scaled and added in fp32.
 *   a, a_scale   (M, K), SSD_SCALE_ROWS
 *   b, b_scale   (N, K), b_scales = SSD_SCALE_BLOCKS (weights) or SSD_SCALE_ROWS
 *   c            output rows of `out_type` (F32 or BF16), ld elements apart; what
 *                lies between its rows is not written
 *   workspace    ssd_fp8_matmul_workspace_bytes() bytes, 256-byte aligned, for one
 *                call at a time. Its first word is a status that a wait that gave
 *                up sets (ssd_complex_status() reads it); C is then incomplete. The
 *                caller zeroes its first SSD_FP8_MATMUL_ZEROED bytes, or all of it
 *                if it has fewer, once, before the first call, and again after such
 *                a status
 * a.p and b.p are 16-byte aligned. Where CTAs share tiles (the workspace is then
 * larger than SSD_FP8_MATMUL_ZEROED) all of them have to run at the same time: the
 * call is SSDC_ERR_CUDA where the device's SMs are not all there for it.
 */
#define SSD_FP8_MATMUL_ZEROED 16384
size_t ssd_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K);
int ssd_fp8_matmul(ssd_rows_in a, const float *a_scale, ssd_rows_in b, const float *b_scale, int32_t b_scales,
                   int64_t M, int64_t N, int64_t K, int32_t out_type, ssd_rows_out c, void *workspace,
                   size_t ws_bytes, cudaStream_t stream);

/*
 * Any of the calls above that launch work, from its arguments as 64-bit words: in
 * order, structures member by member, integers sign-extended, eps as the bits of a
 * float in the low half. For bindings in which passing twenty arguments takes
 * longer than launching the kernel. The checks and results are those of the call;
 * an unknown call is SSDC_ERR_INVALID.
 */
#define SSD_CALL_GATED_SCAN_FWD 0      /* 21 words */
#define SSD_CALL_GATED_SCAN_STEP 1     /* 17 words */
#define SSD_CALL_GATED_SCAN_BWD 2      /* 30 words */
#define SSD_CALL_RESIDUAL_NORM_FWD 3   /* 16 words */
#define SSD_CALL_RESIDUAL_NORM_BWD 4   /* 16 words */
#define SSD_CALL_FP8_QUANTIZE 5        /* 12 words */
#define SSD_CALL_FP8_MATMUL 6          /* 15 words */
#define SSD_CALL_GATED_SCAN_FWD_WS 7   /* 23 words */
int ssd_block_call(int32_t call, const int64_t *words, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SSDC_BLOCK_H */
