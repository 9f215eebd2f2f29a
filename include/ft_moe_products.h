/*
 * ft_moe_products.h -- bf16 products of token rows with one matrix per expert and their gradients, SwiGLU
 * rows with their gradient, and low-rank adapters of many requests beside a shared projection.
 *
 * With ft_moe_dispatch, ft_moe_combine and their gradients (ft_moe_rows.h) the products and SwiGLU make up
 * a training step of the routed-expert FFN; the adapters stand beside ft_moe_fp8_matmul or any other
 * projection whose result is in memory.  The expert groups are those of the FreeToken walk-through
 * "深入FreeToken架构：从HTTP API到CUDA内核的本地MoE推理引擎全链路剖析" (yfxerp.com), section 五.
 *
 * Every convention of ft_moe.h holds here: device pointers, 16-byte aligned, dense row-major arrays,
 * caller-owned buffers, enqueue-only on `stream`, FT_OK or a status with ft_moe_last_error(), calls
 * reentrant and capturable into a graph.  No call keeps any state, and no result depends on the order in which
 * blocks run: the same inputs give the same bits.  Only rows that tables name more than once are excepted (several
 * experts' in offsets that do not ascend, twice in gather): which of their results remains may differ from call to call.
 * Workspaces' contents do not matter; calls that may overlap, and graphs that may, need their own.  Outputs must not
 * overlap inputs or each other, except where said.  Sizes of 0 rows are no-ops, except where said.
 *
 * Rows of an expert.  offsets int32 [E+1] as from ft_moe_permute: expert e has rows offsets[e] .. offsets[e+1]-1
 * of the P rows (entries are taken as if clipped to [0, P]; 1 <= E <= 1024).  slot_of_expert int32 [E] names
 * the expert's matrix; NULL: expert e has matrix e (E <= n_slots).  Experts without a slot in [0, n_slots) are
 * skipped.  Several experts may name one matrix.
 *
 * Sums are fp32 sums of exact products of bf16 values, rounded once to the output's type.  Their order, and with it a
 * result's last bits, depends on the sizes of the call and, for the rows, on the slot of their matrix; for a matrix's
 * gradient, on the number of rows its expert has.
 */
#ifndef FT_MOE_PRODUCTS_H
#define FT_MOE_PRODUCTS_H

#include "ft_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flag of ft_moe_grouped_matmul_wgrad: dw += the gradient (fp32 dw). */
#define FT_ADD_TO_OUT 0x40

/*
 * out[p][n] = sum_k a[p][k] * w[slot][n][k] for the rows p of every expert.
 * a bf16 [P][K], w bf16 [n_slots][N][K], out fp32 [P][N], or bf16 with FT_OUT_BF16.  N % 8 == 0, K % 8 == 0, both at
 * most 2^20.  Rows that belong to no expert with a slot are left as they were; each value of a row that a table which
 * does not ascend gives to several experts is the result of one or another of them.
 */
int ft_moe_grouped_matmul(const uint16_t* a, int P, const uint16_t* w, int n_slots, int N, int K, const int32_t* offsets,
                          const int32_t* slot_of_expert, int E, void* out, int flags, hipStream_t stream);

/*
 * The gradient of its rows: da[p][k] = sum_n dout[p][n] * w[slot][n][k].  dout bf16 [P][N], da fp32 [P][K], or
 * bf16 with FT_OUT_BF16; everything else as above.
 */
int ft_moe_grouped_matmul_grad(const uint16_t* dout, int P, const uint16_t* w, int n_slots, int N, int K,
                               const int32_t* offsets, const int32_t* slot_of_expert, int E, void* da, int flags,
                               hipStream_t stream);

/*
 * The gradient of its matrices, by expert: dw[e][n][k] = sum over the expert's rows p of dout[p][n] * a[p][k].
 * dout bf16 [P][N], a bf16 [P][K], dw fp32 [E][N][K] (with FT_ADD_TO_OUT: dw += the gradient), or bf16 with
 * FT_OUT_BF16.  An expert without rows gets zeros (with FT_ADD_TO_OUT: keeps what it has), also where P == 0.
 * slot_of_expert here only says which experts count (NULL: all): where an entry is negative, or not below n with
 * FT_N_SLOTS(n), the expert's part of dw is left as it was.  (A matrix that several experts name has the sum of their
 * parts as its gradient; the caller adds them.)
 * ws: ft_moe_grouped_matmul_wgrad_workspace(N, K, E) bytes of device memory (0 for few tiles: then ws may be NULL).
 */
size_t ft_moe_grouped_matmul_wgrad_workspace(int N, int K, int E);
int ft_moe_grouped_matmul_wgrad(const uint16_t* dout, const uint16_t* a, int P, int N, int K, const int32_t* offsets,
                                const int32_t* slot_of_expert, int E, void* dw, void* ws, size_t ws_bytes, int flags,
                                hipStream_t stream);

/*
 * h = SiLU(g) * u, SiLU(g) = g / (1 + e^-g), formed in fp32 and rounded once.  gu bf16 [rows][2 I]: gate columns
 * 0 .. I-1, up columns I .. 2I-1 (what ft_moe_grouped_matmul gives for W13 rows [gate ; up]) -> h bf16 [rows][I].
 * I % 8 == 0, I <= 2^20.  SiLU(g) u is off by up to about (|g| + 10) * 2^-24 of itself before it is rounded (the GPU's
 * exp2 and reciprocal instructions), and 1 / (1 + e^-g) under 2^-126 (g < -87.3) may count as 0.
 */
int ft_moe_swiglu(const uint16_t* gu, int rows, int I, uint16_t* h, hipStream_t stream);

/*
 * Its gradient for dh bf16 [rows][I]: dgu bf16 [rows][2 I] with s = 1 / (1 + e^-g) and
 *   dg = dh * u * s * (1 + g * (1 - s)),   du = dh * g * s.
 * dgu may be gu itself.
 */
int ft_moe_swiglu_grad(const uint16_t* gu, const uint16_t* dh, int rows, int I, uint16_t* dgu, hipStream_t stream);

/*
 * Low-rank adapters: for every row t of T with an adapter
 *   out[t][n] = base[t][n] + scale[slot] * sum_j (sum_k x[t][k] a[slot][j][k]) * b[slot][n][j]
 * and out[t] = base[t] for the others.  x bf16 [T][K], a bf16 [n_slots][r][K], b bf16 [n_slots][N][r], scale fp32
 * [n_slots] (NULL: 1), base and out fp32 [T][N], or bf16 with FT_OUT_BF16; out may be base itself.
 * The rows of adapter i of E are gather[offsets[i]] .. gather[offsets[i+1]-1], as ft_moe_permute gives them for the
 * rows' adapters (k = 1); rows without an adapter are given number E there (and E + 1 experts), or an adapter
 * without a slot in [0, n_slots).  slot_of_adapter NULL: adapter i is in slot i (E <= n_slots).  Positions before
 * offsets[0] and from offsets[E] on count as rows without an adapter; entries of gather outside [0, T) are skipped; a row that gather
 * does not name is left as it was, one that it names twice is formed twice (with out == base: added twice or once),
 * and rows that a table which does not ascend gives to several adapters get values of no use.
 * r % 8 == 0, r <= 256 (adapters of smaller rank: zeros behind), N % 8 == 0, K % 8 == 0, both at most 2^20, T < 2^24;
 * sizes whose tiles an int cannot count, whatever offsets holds, are refused with FT_E_UNSUPPORTED.
 * The inner sums are held in fp32 and enter the outer ones as bf16 terms: two for bf16 results, within 2^-16 of themselves,
 * three for fp32 ones, all of them.  The terms have the sum's sign and none is 0 beside a sum that is not: infinities and NaN of x, a, b
 * and scale give what the formula gives.
 * ws: ft_moe_lora_workspace(T, E, r, N, K) bytes of device memory (0 for few rows: then ws may be NULL).
 */
size_t ft_moe_lora_workspace(int T, int E, int r, int N, int K);
int ft_moe_lora(const void* base, const uint16_t* x, int T, const uint16_t* a, const uint16_t* b, const float* scale,
                int n_slots, int r, int N, int K, const int32_t* offsets, const int32_t* gather,
                const int32_t* slot_of_adapter, int E, void* out, void* ws, size_t ws_bytes, int flags, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* FT_MOE_PRODUCTS_H */
