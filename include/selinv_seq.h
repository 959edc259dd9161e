/*
 * selinv_seq.h -- C ABI of the sequence-mixer operators of the library:
 * recurrences over a chain of tokens instead of a symmetric chain of blocks.
 *
 *   selinv_conv_*   short causal convolution of every channel
 *   selinv_scan_*   selective state space scan (a lower-bidiagonal chain whose
 *                   coupling is one scalar per head and token)
 *   selinv_qkrot_*  norm of every query and key head with the rotation by
 *                   position
 *
 * Each comes as the forward call, as its reverse mode (_vjp) and, where a state
 * is carried, as the call for one token per sequence (_step), which updates a
 * pool of states in place.
 *
 * Conventions, beyond those of selinv.h (device pointers, caller-owned memory
 * and workspace, work enqueued on `stream`, synchronous status):
 *   - The suffix names the element type of the token arrays: _f32, _f16,
 *     _bf16.  Parameters (weights, biases, A, D, dt_bias, rotation tables),
 *     their gradients and the scan's states are always float32.  Sums, norms
 *     and states are held in float32 or more, and enter the scan's products
 *     with 24 bits at least; an output is rounded to its type once.
 *   - The arguments are passed in a struct; a pointer marked "opt" may be
 *     NULL.  Strides are in elements, the innermost dimension is contiguous;
 *     an array without stride fields is contiguous.  Any alignment of the
 *     element type is accepted; 16-byte aligned rows are the fast case.
 *   - `lengths` (opt, int32 [B]): row r holds lengths[r] tokens (clamped to
 *     0..T) of the padded T.  What lies past them has no effect (of the scan's
 *     dt it may be read and dropped, all else is not read); outputs and
 *     gradients there are written as zero, and the state handed on is the one
 *     after the last token (the initial state for a row of length zero).
 *   - `slots` (opt, int32 [B], the _step calls): row r uses state
 *     slots[r] of the pool of n_slots; NULL = its own index.  A row whose slot
 *     is outside 0..n_slots-1 (-1 marks an idle row) gets zero outputs and
 *     touches no state.  Slots of one call must differ from each other.
 *   - Results do not depend on timing: no atomics, sums in a fixed order.
 *   - Outputs must not alias inputs or each other (the _step state excepted).
 *   - An empty batch or length (B = 0, T = 0) is valid: the states and
 *     gradients that exist are written.
 *   - Sizes: B (T + 128) and B (T + 128) C / 16 at most 2^30, C at most 2^27;
 *     B T at most 2^26 - 4 for selinv_qkrot_*; B H at most 2^20 and B (T + 128)
 *     H / 64 at most 2^30 for selinv_scan_*; the chunks of selinv_scan_vjp_*, B
 *     G times T over 64 (bfloat16) or 32 rounded up, below 2^23.  Larger calls
 *     are refused.
 *   - Return: SELINV_OK, SELINV_ERR_INVALID_ARG or SELINV_ERR_HIP.
 */
#ifndef SELINV_SEQ_H
#define SELINV_SEQ_H

#include "selinv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------ short convolution
 * With the row's past written before it, whole = [state, x] (zeros if state
 * is NULL),
 *   v[t][c] = bias[c] + sum_j weight[c][j] whole[t + j][c],   j = 0..W-1,
 *   y = silu ? v / (1 + exp(-v)) : v,
 *   state_out = the last W-1 tokens of whole.
 *   x [B][T][C] (strides), weight [C][W], bias [C] opt, state [B][W-1][C] opt;
 *   y [B][T][C], state_out [B][W-1][C] opt.
 *   vjp: y_bar [B][T][C] (strides), state_out_bar [B][W-1][C] opt ->
 *   x_bar [B][T][C], weight_bar [C][W], bias_bar [C] opt,
 *   state_bar [B][W-1][C] opt.
 *   step: x, y [B][C] (x with its stride x_sb), state [n_slots][W-1][C]
 *   updated in place.
 * C >= 1, 1 <= W <= SELINV_CONV_MAX_W. */
#define SELINV_CONV_MAX_W 8

typedef struct selinv_conv_args {
  int64_t B, T, n_slots; /* n_slots: step only */
  int64_t x_sb, x_st;    /* strides of x */
  int64_t yb_sb, yb_st;  /* strides of y_bar (vjp) */
  int32_t C, W, silu, reserved;
  const void *x;
  const float *weight;
  const float *bias;      /* opt */
  const void *state;      /* opt; step: the pool, written */
  const int32_t *lengths; /* opt; forward and vjp */
  const int32_t *slots;   /* opt; step */
  void *y;                /* forward and step */
  void *state_out;        /* opt; forward */
  const void *y_bar;      /* vjp, as are all below */
  const void *state_out_bar; /* opt */
  void *x_bar;
  float *weight_bar;
  float *bias_bar;        /* opt */
  void *state_bar;        /* opt */
} selinv_conv_args;

SELINV_API int selinv_conv_f32(const selinv_conv_args *a, void *stream);
SELINV_API int selinv_conv_f16(const selinv_conv_args *a, void *stream);
SELINV_API int selinv_conv_bf16(const selinv_conv_args *a, void *stream);
SELINV_API int selinv_conv_step_f32(const selinv_conv_args *a, void *stream);
SELINV_API int selinv_conv_step_f16(const selinv_conv_args *a, void *stream);
SELINV_API int selinv_conv_step_bf16(const selinv_conv_args *a, void *stream);
SELINV_API size_t selinv_conv_vjp_workspace_bytes(int64_t B, int64_t T, int32_t C, int32_t W);
SELINV_API int selinv_conv_vjp_f32(const selinv_conv_args *a, void *workspace,
                                   size_t workspace_bytes, void *stream);
SELINV_API int selinv_conv_vjp_f16(const selinv_conv_args *a, void *workspace,
                                   size_t workspace_bytes, void *stream);
SELINV_API int selinv_conv_vjp_bf16(const selinv_conv_args *a, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* ------------------------------------------------- head norm and rotation
 * For every token and every head u of q or k, with its weight w [D]:
 *   r = 1 / sqrt(mean(u^2) + eps),  v = u r w,
 * then for i < R/2, with c = cos[pos][i], s = sin[pos][i] and the pair
 * (a, b) = (v_i, v_{i+R/2}), or (v_{2i}, v_{2i+1}) if interleaved,
 *   (a, b) -> (a c - b s, b c + a s);
 * the elements from R on are left as they are.
 *   q [B][T][Hq][D], k [B][T][Hk][D] (strides), q_weight, k_weight [D],
 *   cos, sin [table_rows][R/2], positions [B][T] (strides; int32, or int64 if
 *   positions_64); q_out, k_out contiguous.  A token whose position is outside
 *   0..table_rows-1 gets NaN.
 *   vjp: q_bar, k_bar (cotangents of q_out, k_out; strides) -> q_grad
 *   [B][T][Hq][D], k_grad [B][T][Hk][D], q_weight_grad, k_weight_grad [D].
 * Hq >= 1, Hk >= 0 (0: queries alone; the k arrays may be NULL, and
 * k_weight_grad is written as zero where given), 1 <= D <=
 * SELINV_QKROT_MAX_D, 0 <= R <= D, R even. */
#define SELINV_QKROT_MAX_D 512

typedef struct selinv_qkrot_args {
  int64_t B, T, table_rows;
  int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh;         /* strides of q, k */
  int64_t qb_sb, qb_st, qb_sh, kb_sb, kb_st, kb_sh;   /* of q_bar, k_bar (vjp) */
  int64_t pos_sb, pos_st;                             /* of positions */
  int32_t Hq, Hk, D, R, interleaved, positions_64;
  float eps;
  int32_t reserved;
  const void *q, *k;
  const float *q_weight, *k_weight;
  const float *cos_table, *sin_table; /* NULL only if R == 0 */
  const void *positions;              /* NULL only if R == 0 */
  void *q_out, *k_out;                /* forward */
  const void *q_bar, *k_bar;          /* vjp, as are all below */
  void *q_grad, *k_grad;
  float *q_weight_grad, *k_weight_grad;
} selinv_qkrot_args;

SELINV_API int selinv_qkrot_f32(const selinv_qkrot_args *a, void *stream);
SELINV_API int selinv_qkrot_f16(const selinv_qkrot_args *a, void *stream);
SELINV_API int selinv_qkrot_bf16(const selinv_qkrot_args *a, void *stream);
SELINV_API size_t selinv_qkrot_vjp_workspace_bytes(int64_t B, int64_t T, int32_t D);
SELINV_API int selinv_qkrot_vjp_f32(const selinv_qkrot_args *a, void *workspace,
                                    size_t workspace_bytes, void *stream);
SELINV_API int selinv_qkrot_vjp_f16(const selinv_qkrot_args *a, void *workspace,
                                    size_t workspace_bytes, void *stream);
SELINV_API int selinv_qkrot_vjp_bf16(const selinv_qkrot_args *a, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* --------------------------------------------------------- selective scan
 * Per row and head h (of group g = h / (H / G)), with the state S a P x N
 * matrix:
 *   d_t = softplus ? log(1 + exp(dt_t + dt_bias)) : dt_t + dt_bias,
 *   S_t = exp(d_t A) S_{t-1} + d_t x_t B_t^T,
 *   y_t = S_t C_t + D x_t.
 *   x [B][T][H][P], dt [B][T][H], Bm, Cm [B][T][G][N] (strides), A [H],
 *   D [H] opt, dt_bias [H] opt, state [B][H][P][N] opt (float32);
 *   y [B][T][H][P], state_out [B][H][P][N] opt (float32).
 *   vjp: y_bar (strides), state_out_bar [B][H][P][N] opt (float32) -> x_bar,
 *   dt_bar, B_bar, C_bar (contiguous), A_bar [H], D_bar [H] opt,
 *   dt_bias_bar [H] opt, state_bar [B][H][P][N] opt.
 *   step: x, y [B][H][P], dt [B][H], Bm, Cm [B][G][N] (their batch and head
 *   strides), state [n_slots][H][P][N] updated in place.
 * H a multiple of G, 1 <= P <= SELINV_SCAN_MAX_P, 1 <= N <=
 * SELINV_SCAN_MAX_N.  Token inputs and d_t A have to be finite inside a row's
 * length: a token's values may reach the 63 tokens before it as 0 * inf. */
#define SELINV_SCAN_MAX_P 256
#define SELINV_SCAN_MAX_N 128

typedef struct selinv_scan_args {
  int64_t B, T, n_slots; /* n_slots: step only */
  int64_t x_sb, x_st, x_sh, dt_sb, dt_st, b_sb, b_st, b_sg, c_sb, c_st, c_sg; /* strides */
  int64_t yb_sb, yb_st, yb_sh; /* strides of y_bar (vjp) */
  int32_t H, P, G, N, softplus, reserved;
  const void *x, *dt, *Bm, *Cm;
  const float *A;
  const float *D;       /* opt */
  const float *dt_bias; /* opt */
  const float *state;   /* opt; step: the pool, written */
  const int32_t *lengths; /* opt; forward and vjp */
  const int32_t *slots;   /* opt; step */
  void *y;                /* forward and step */
  float *state_out;       /* opt; forward */
  const void *y_bar;      /* vjp, as are all below */
  const float *state_out_bar; /* opt */
  void *x_bar, *dt_bar, *B_bar, *C_bar;
  float *A_bar;
  float *D_bar;       /* opt */
  float *dt_bias_bar; /* opt */
  float *state_bar;   /* opt */
} selinv_scan_args;

SELINV_API size_t selinv_scan_workspace_bytes(int dtype_bytes, int64_t B, int64_t T, int32_t H,
                                              int32_t P, int32_t N);
SELINV_API int selinv_scan_f32(const selinv_scan_args *a, void *workspace,
                               size_t workspace_bytes, void *stream);
SELINV_API int selinv_scan_f16(const selinv_scan_args *a, void *workspace,
                               size_t workspace_bytes, void *stream);
SELINV_API int selinv_scan_bf16(const selinv_scan_args *a, void *workspace,
                                size_t workspace_bytes, void *stream);
SELINV_API int selinv_scan_step_f32(const selinv_scan_args *a, void *stream);
SELINV_API int selinv_scan_step_f16(const selinv_scan_args *a, void *stream);
SELINV_API int selinv_scan_step_bf16(const selinv_scan_args *a, void *stream);
/* Two float32 states a head and chunk of 32 tokens, which is enough for every
 * type of dtype_bytes; the chunks of bfloat16 are of 64, and its calls need no
 * more than the second query says. */
SELINV_API size_t selinv_scan_vjp_workspace_bytes(int dtype_bytes, int64_t B, int64_t T, int32_t H,
                                                  int32_t P, int32_t G, int32_t N);
SELINV_API size_t selinv_scan_vjp_bf16_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t P,
                                                       int32_t G, int32_t N);
SELINV_API int selinv_scan_vjp_f32(const selinv_scan_args *a, void *workspace,
                                   size_t workspace_bytes, void *stream);
SELINV_API int selinv_scan_vjp_f16(const selinv_scan_args *a, void *workspace,
                                   size_t workspace_bytes, void *stream);
SELINV_API int selinv_scan_vjp_bf16(const selinv_scan_args *a, void *workspace,
                                    size_t workspace_bytes, void *stream);

#ifdef __cplusplus
} /* extern "C" */
#endif
#endif /* SELINV_SEQ_H */
