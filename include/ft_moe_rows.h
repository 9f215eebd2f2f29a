/*
 * ft_moe_rows.h -- rows around the expert FFN of ft_moe.h: activations in 8-bit floating point with a
 * scale per 128 values, their products with block-scaled 8-bit weights (dense, or one matrix per
 * expert), and what a training step needs of the routing: token rows in expert order with their
 * gradient, and the gradient of the weighted combine down to the router's logits.
 *
 * The FP8 block linear and the expert banks in FP8 blocks are named by the FreeToken walk-through
 * "深入FreeToken架构：从HTTP API到CUDA内核的本地MoE推理引擎全链路剖析" (yfxerp.com), sections 五 and 六; the
 * expert dispatch in section 一.
 *
 * Every convention of ft_moe.h holds here: device pointers, 16-byte aligned, dense row-major arrays,
 * caller-owned buffers, enqueue-only on `stream`, FT_OK or a status with ft_moe_last_error(), calls
 * reentrant and capturable into a graph.  No call here needs a workspace or keeps any state, and no
 * result depends on the order in which blocks or atomics run: the same inputs give the same bits.
 * Outputs must not overlap inputs or each other.  Sizes of 0 rows or tokens are no-ops.  Sizes that one launch
 * cannot count are refused with FT_E_UNSUPPORTED: more than 2^29 - 32 scales, 2^26 - 4 pieces of 1024 values of token
 * rows, 2^24 - 1 tokens (ft_moe_combine_grad), 2^23 - 8 tiles of a product.
 *
 * 8-bit rows.  A row of K values (K % 16 == 0) is K e4m3fn codes and S = ft_moe_fp8_scale_cols(K) fp32
 * scales: scale b covers values 128 b .. 128 b + 127 (the last block may be shorter) and the columns
 * from ceil(K / 128) on are 0.  value = scale * code, with
 *   top   = max(largest magnitude of the block, 2^-100)
 *   scale = top / 448 rounded to fp32
 *   code  = the e4m3 value nearest to 448 * x / top, ties to even (bf16 inputs: exactly; fp32 and SwiGLU
 *           inputs: nearest to that quotient formed in fp32, which is off by up to 3 * 2^-24 of itself)
 * A block that holds a NaN or an infinity gets a NaN scale and NaN codes.
 */
#ifndef FT_MOE_ROWS_H
#define FT_MOE_ROWS_H

#include "ft_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flag of the row calls: rows are fp32 instead of bf16 (inputs, and the outputs of their type). */
#define FT_ROWS_F32 0x20

/* Scale columns of an 8-bit row of K values: one per 128, rounded up to a multiple of 4 (rows of scales
 * stay 16-byte aligned); 0 when K <= 0. */
int ft_moe_fp8_scale_cols(int K);

/*
 * Rows to 8-bit rows.  x bf16 (FT_ROWS_F32: fp32) [rows][K] -> codes [rows][K], scales fp32 [rows][S].
 */
int ft_moe_quant_fp8(const void* x, int rows, int K, uint8_t* codes, float* scales, int flags, hipStream_t stream);

/*
 * The 8-bit rows of h = SiLU(g) * u, SiLU(g) = g / (1 + e^-g), computed and quantised in fp32 (h is not
 * rounded to bf16 in between).  gu bf16 [rows][2 I]: gate columns 0 .. I-1, up columns I .. 2I-1
 * (what ft_moe_fp8_grouped_matmul gives for W13 rows [gate ; up]) -> codes [rows][I], scales [rows][S].
 * SiLU(g) u is off by up to about (|g| + 10) * 2^-24 of itself (the GPU's exp2 and reciprocal instructions), and
 * 1 / (1 + e^-g) under 2^-126 (g < -87.3) may count as 0.
 */
int ft_moe_swiglu_fp8(const uint16_t* gu, int rows, int I, uint8_t* codes, float* scales, hipStream_t stream);

/*
 * Token rows in expert order.  For every pair (t, j) that has a row: x_sorted[inv[t*k+j]] = x[t].
 * ids, inv as ft_moe_route and ft_moe_permute give them.  A pair has a row when ids[t*k+j] lies in [0, E),
 * inv[t*k+j] in [0, T*k), and slot_of_expert (int32 [E]; NULL: every expert counts) is not negative for
 * its expert, nor past the bank where the flags hold FT_N_SLOTS(n); rows of other pairs are left as they were.
 * (ft_moe_permute gives every pair a place of its own; a place that several pairs name holds parts of any of their
 * rows.)  x, x_sorted bf16 (FT_ROWS_F32: fp32), d % 8 == 0.  (This call, ft_moe_dispatch_fp8, ft_moe_dispatch_grad and
 * ft_moe_combine_grad read the same table: beside ft_moe_fp8_grouped_matmul, which skips slots outside its n_slots,
 * give them its n_slots, so that rows it left alone are not read.)
 */
int ft_moe_dispatch(const void* x, const int32_t* ids, const int32_t* inv, const int32_t* slot_of_expert, int T,
                    int E, int k, int d, void* x_sorted, int flags, hipStream_t stream);

/*
 * The same with 8-bit rows out: the 8-bit row of x[t] (ft_moe_quant_fp8) at every row inv[t*k+j] of token t.
 * codes [T*k][d], scales [T*k][S], d % 16 == 0.
 */
int ft_moe_dispatch_fp8(const void* x, const int32_t* ids, const int32_t* inv, const int32_t* slot_of_expert, int T,
                        int E, int k, int d, uint8_t* codes, float* scales, int flags, hipStream_t stream);

/*
 * Gradient of ft_moe_dispatch: dx[t] = sum over j ascending of dx_sorted[inv[t*k+j]] over the pairs that have a
 * row, summed in fp32 and rounded once (0 for a token without any).
 */
int ft_moe_dispatch_grad(const void* dx_sorted, const int32_t* ids, const int32_t* inv, const int32_t* slot_of_expert,
                         int T, int E, int k, int d, void* dx, int flags, hipStream_t stream);

/*
 * Gradient of ft_moe_combine, and of ft_moe_route's weights, for a gradient dout of its `out`
 * (fp32 [T][d], or bf16 with FT_OUT_BF16).  For every pair that has a row r = inv[t*k+j] (as above):
 *   dy_sorted[r] = w[t][j] * dout[t], rounded to bf16          (rows of other pairs are left as they were)
 *   dw[t][j]     = sum_c dout[t][c] * y_sorted[r][c] in fp32   (0 for other pairs)
 * and, when dlogits is not NULL, for every token
 *   dlogits[t][e] = sum over j with ids[t][j] == e of w_j * (dw_j - sum_i w_i dw_i), else 0:
 * the gradient through w = softmax of the k chosen logits; the choice itself has none.
 * y_sorted bf16 [T*k][d], dw fp32 [T][k], dlogits fp32 [T][E]; d % 8 == 0.  The gradient of y_shared is
 * dout itself.
 */
int ft_moe_combine_grad(const void* dout, const uint16_t* y_sorted, const int32_t* ids, const float* w,
                        const int32_t* inv, const int32_t* slot_of_expert, int T, int E, int k, int d,
                        uint16_t* dy_sorted, float* dw, float* dlogits, int flags, hipStream_t stream);

/*
 * Product of 8-bit rows with a block-scaled 8-bit matrix:
 *   out[m][n] = sum over blocks b of 128 along K of
 *               a_scales[m][b] * w_scales[n / 128][b] * (sum over k in block b of a[m][k] * w[n][k])
 * a codes [M][K] with scales [M][S]; w e4m3fn codes [N][K] with fp32 scales [ceil(N/128)][ceil(K/128)]: the
 * canonical FT_W_FP8_B128 matrix (not the interleaved bank).  out fp32 [M][N], or bf16 with FT_OUT_BF16 (rounded
 * once).  K % 16 == 0, K <= 2^20; M and N are any.  Block sums are multiplied with the product of their two
 * scales, itself formed in fp32 (scales whose product leaves fp32's range lose the block), and added in fp32.
 * With fp32 results the code products of a block are exact and are added in fp32.  With FT_OUT_BF16 and more than
 * a few rows (the sizes decide) they are added by the 8-bit matrix instructions, which cut each product in a group of
 * 8 at 2^-13 of the group's largest before adding: off by at most 7 * 2^-13 of the sum of the products'
 * magnitudes, by about 1.3e-5 of the result's norm for normally distributed values.  Where products cancel to a small
 * result, that can be more than the 2^-8 of itself that bf16 rounds to: ask for fp32 results there.
 * The kernel, and with it the order of the sums, is chosen by the sizes: a row's last bits depend on how many other
 * rows are in the call.
 * A gradient with respect to the rows is the same call with the transposed codes and scales.
 */
int ft_moe_fp8_matmul(const uint8_t* a, const float* a_scales, int M, const uint8_t* w, const float* w_scales, int N,
                      int K, void* out, int flags, hipStream_t stream);

/*
 * The same with one matrix per expert: rows offsets[e] .. offsets[e+1]-1 of the P rows (offsets int32 [E+1]
 * from ft_moe_permute; entries are taken as if clipped to [0, P]) are multiplied with the matrix in slot
 * slot_of_expert[e] of w [n_slots][N][K], w_scales [n_slots][ceil(N/128)][ceil(K/128)].  Rows of experts
 * without a slot in [0, n_slots), and rows that belong to no expert, are left as they were; a row that a table
 * which does not ascend gives to several experts gets the result of one of them.
 * 1 <= E <= 1024.
 */
int ft_moe_fp8_grouped_matmul(const uint8_t* a, const float* a_scales, int P, const uint8_t* w, const float* w_scales,
                              int n_slots, int N, int K, const int32_t* offsets, const int32_t* slot_of_expert, int E,
                              void* out, int flags, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* FT_MOE_ROWS_H */
