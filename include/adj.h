/*
 * adj.h -- C ABI of libadj.so, the GB300 (sm_103a) adjoint-sharding gradient path
 * for residual stacks of diagonal selective state-space layers.
 *
 * Source of the operations: the review page "Adjoint sharding for very long
 * context training of state space models" (pith.science), cited as [AS].
 *
 * Layer model ([AS] Assumptions: Sec. 3.1 SSM dynamics h_t = A_t h_{t-1} + B_t x_t,
 * y_t = C_t h_t; Sec. 3.2 residual structure y^K = y^0 + sum_k ytilde^k), in the
 * diagonal selective form A_t = diag(a_t), B_t xhat_t = u_t, C_t = W_o^T diag(c_t):
 *     a_t = sigmoid(xhat_t W_a + b_a),  u_t = xhat_t W_B,  c_t = xhat_t W_c,
 *     h_t = a_t . h_{t-1} + u_t  (h_0 = 0),   y_t = xhat_t + (c_t . h_t) W_o.
 *
 * Conventions shared by every call:
 *  - Arrays are row-major and token-major: [B,T,P] and [B,T,N] with the last
 *    index contiguous.  Every array pointer is a DEVICE pointer owned by the
 *    caller; the library never allocates, frees or keeps a pointer after a call.
 *  - Every pointer must be 16-byte aligned; P and N must be multiples of 8;
 *    B, T >= 0 are arbitrary (B*T == 0 launches nothing and returns ADJ_OK).
 *  - `ws` is caller-owned device scratch of at least adj_workspace_bytes() bytes,
 *    256-byte aligned.  Its first 256 bytes hold the sticky device status word
 *    read by adj_stream_status(); zero them once (cudaMemset) before first use.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Calls are asynchronous on that stream.  Calls sharing one `ws` must be
 *    ordered on one stream.  A call enqueues only kernels and memsets on the
 *    stream (no allocation, no host synchronisation), so a sequence of calls can
 *    be captured into a CUDA graph and replayed; the graph keeps the pointers
 *    and sizes it was captured with.
 *  - Every argument is validated on the host before anything is launched; on an
 *    error nothing is launched and nothing is written.  Launch failures return
 *    ADJ_ECUDA.  Bounded device-side waits that give up record ADJ_ETIMEOUT in
 *    the workspace status word and return without hanging; read it with
 *    adj_stream_status().  Nothing throws, traps or exits.
 */
#ifndef ADJ_H_
#define ADJ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ADJ_OK = 0,
    ADJ_EINVAL = 1,      /* null pointer, bad enum, bad window */
    ADJ_ESHAPE = 2,      /* negative or unsupported sizes */
    ADJ_EALIGN = 3,      /* a pointer not 16-byte aligned (ws: 256-byte) */
    ADJ_EDTYPE = 4,      /* unsupported dtype combination */
    ADJ_EWORKSPACE = 5,  /* ws_bytes below adj_workspace_bytes() */
    ADJ_ECUDA = 6,       /* a CUDA launch or runtime call failed */
    ADJ_ETIMEOUT = 7     /* a bounded device wait gave up (see adj_stream_status) */
} adj_status;

typedef enum { ADJ_F32 = 0, ADJ_BF16 = 1 } adj_dtype;

/* Problem sizes and storage types of one layer call.
 * x_dtype: storage of the GEMM operands xhat, W_in, W_o (and of y_x below).
 * d_dtype: storage of the VJP factors D_a, D_u, D_c and of E. */
typedef struct {
    int64_t B, T;
    int32_t P, N;
    int32_t x_dtype, d_dtype;
} adj_dims;

/* Layer weights (device pointers).
 * W_in [P,3N] x_dtype: column blocks [W_a | W_B | W_c].
 * b_a  [N]   fp32.
 * W_o  [N,P] x_dtype. */
typedef struct {
    const void *W_in;
    const float *b_a;
    const void *W_o;
} adj_weights;

enum {
    ADJ_OP_FWD = 0, ADJ_OP_BWD_FULL = 1, ADJ_OP_BWD_TRUNC = 2, ADJ_OP_PARAM = 3, ADJ_OP_LOSS = 4,
    ADJ_OP_SEL_FWD = 5, ADJ_OP_SEL_BWD = 6, ADJ_OP_SEL_PARAM = 7,  /* the general selective layer (below) */
    ADJ_OP_LIN_FWD = 8, ADJ_OP_LIN_BWD = 9,                        /* adj_lin_workspace_bytes only */
    ADJ_OP_SSM_FWD = 10, ADJ_OP_SSM_BWD = 11                       /* adj_ssm_workspace_bytes only */
};

/* Workspace bytes that call `op` needs for these sizes (Tbar: the window of
 * ADJ_OP_BWD_TRUNC and ADJ_OP_SEL_BWD, ignored otherwise).  One workspace of the maximum over the
 * ops used serves them all.  Returns 0 for invalid sizes. */
size_t adj_workspace_bytes(const adj_dims *dims, int op, int64_t Tbar);

/* Forward pass of one layer storing the states the adjoint needs
 * ([AS] Referee Report, comment on Algorithm 1: per-token, per-layer states are
 * kept; here a_t, c_t and h_t, the layer input being the caller's xhat).
 *   xhat [B,T,P] x_dtype  layer input as GEMM operand
 *   xres [B,T,P] fp32     residual input; NULL = use xhat's values
 *   a, c, h [B,T,N] fp32  stored gate, output gate and state (written)
 *   y    [B,T,P] fp32     layer output xres + (c . h) W_o (written; NULL to skip)
 *   y_x  [B,T,P] x_dtype  y rounded to x_dtype for the next layer's xhat
 *                         (written; NULL to skip; must be NULL if x_dtype is fp32) */
adj_status adj_fwd_scan(const adj_dims *dims, const adj_weights *w, const void *xhat,
                        const float *xres, float *a, float *c, float *h, float *y, void *y_x,
                        void *ws, size_t ws_bytes, void *stream);

/* Loss of the last layer and its cotangent: L = sum_{b,t} 1/2 ||y_t - target_t||^2,
 * gy = y - target.  y, target, gy [B,T,P] fp32 (gy written; may alias y);
 * gy_x [B,T,P] bf16: gy rounded to bf16 (written; NULL to skip; needs gy), the operand the
 * bf16 layers' backward GEMMs read (see gy_x of adj_bwd_* and adj_param_grad);
 * loss: one device double (written; NULL to skip).  Uses dims->B, T, P only. */
adj_status adj_loss_mse(const adj_dims *dims, const float *y, const float *target, float *gy,
                        void *gy_x, double *loss, void *ws, size_t ws_bytes, void *stream);

/* Adjoint pass of one layer, full window ([AS] Core claim, Proposition 2, with
 * lambda_{t,i} = C_t prod_{j=i+1..t} A_j; the sum over t of dl_t/dy_t lambda_{t,i}
 * is the reverse recurrence of [AS] What carries the argument, Proposition 1).
 * With g_t = gy_t W_o^T and mu_i = sum_{t>=i} g_t . c_t . prod_{j=i+1..t} a_j it
 * writes the per-token VJP seeds
 *   D_a = mu_i . h_{i-1} . a_i (1 - a_i)   (vjp^{A_i}),   D_u = mu_i   (vjp^{B_i}),
 *   D_c = g_t . h_t,  E = c_t . h_t        (vjp^{C_t}),
 * all [B,T,N] in d_dtype.  a, c, h [B,T,N] fp32 from adj_fwd_scan; gy [B,T,P]
 * fp32 = dL/dy of this layer (the total cotangent).  gy_x [B,T,P] bf16 (NULL to skip;
 * bf16 layers only): gy rounded to bf16, read in place of gy by the product g = gy W_o^T
 * (which rounds gy to bf16 in bf16 layers anyway).
 * dz [B*T, ceil(N/128)] fp32 (NULL to skip; needs w->b_a): per token and group of 128
 * channels, the sum of D_a z_a + D_u u + D_c c over the group, with the seeds as stored,
 * z_a = logit(a_t) - b_a = xhat_t W_a and u_t = h_t - a_t h_{t-1} = xhat_t W_B.  Summed
 * over the groups this is D_t . (xhat_t W_in) = xhat_t . dxhat_t, the row dot product
 * that adj_param_grad needs for a normalised layer input (see r and dz there). */
adj_status adj_bwd_full(const adj_dims *dims, const adj_weights *w, const float *a,
                        const float *c, const float *h, const float *gy, const void *gy_x, void *D_a,
                        void *D_u, void *D_c, void *E, float *dz, void *ws, size_t ws_bytes, void *stream);

/* As adj_bwd_full, truncated to the window Tbar ([AS] Core claim, last sentence;
 * Referee Report on Section 4.3): mu_i sums only t with t - i < Tbar.  Tbar >= 1;
 * Tbar >= T gives the full result. */
adj_status adj_bwd_trunc(const adj_dims *dims, const adj_weights *w, const float *a,
                         const float *c, const float *h, const float *gy, const void *gy_x, void *D_a,
                         void *D_u, void *D_c, void *E, float *dz, int64_t Tbar, void *ws, size_t ws_bytes,
                         void *stream);

/* Parameter gradients as reductions over all tokens ([AS] Core claim: the sum over
 * t and i of the VJPs, applied once per token to the summed seeds):
 *   dW_in [P,3N] = xhat^T [D_a | D_u | D_c],  db_a [N] = sum_t D_a,
 *   dW_o  [N,P]  = E^T gy,
 * fp32, overwritten (accumulate = 0) or added to (accumulate = 1).
 * The cotangent of the layer input, at most one of (NULL to skip):
 *   gy_prev [B,T,P] fp32 = gy + [D_a | D_u | D_c] W_in^T: the total cotangent of the
 *           layer below when that layer's output is this layer's input unchanged
 *           ([AS] residual identity; Proposition 3);
 *           with r and dz (both or neither): the layer input is the normalised residual
 *           stream xhat = y / r of adj_rms_norm, and gy_prev = gy + (dxhat - xhat m / P) / r
 *           with dxhat = [D_a | D_u | D_c] W_in^T and m = sum of dz's groups, the
 *           cotangent of y through the normalisation ([AS] Load-bearing premise); r [B,T]
 *           fp32 from adj_rms_norm, dz from adj_bwd_*, xhat as passed above;
 *   dxhat   [B,T,P] fp32 = [D_a | D_u | D_c] W_in^T alone (for adj_rms_norm_bwd).
 * bf16 layers only (NULL to skip): gy_x [B,T,P] bf16, gy rounded to bf16, read in place of
 * gy by the dW_o product; gy_prev_x [B,T,P] bf16, gy_prev rounded to bf16 (written; needs
 * gy_prev), the next layer's gy_x. */
adj_status adj_param_grad(const adj_dims *dims, const adj_weights *w, const void *xhat,
                          const void *D_a, const void *D_u, const void *D_c, const void *E,
                          const float *gy, const void *gy_x, float *dW_in, float *db_a, float *dW_o,
                          float *gy_prev, void *gy_prev_x, float *dxhat, const float *r, const float *dz,
                          int accumulate, void *ws, size_t ws_bytes, void *stream);

/* Normalised layer input of a stacked layer ([AS] Load-bearing premise: the layers
 * read "normalized inputs"): per token, xhat = y / r with
 * r = sqrt(mean_p y_p^2 + ADJ_NORM_EPS).  y [B,T,P] fp32 (the residual stream y^{k-1});
 * xhat [B,T,P] in dims->x_dtype and r [B,T] fp32 are written.  No workspace. */
#define ADJ_NORM_EPS 1e-6f
adj_status adj_rms_norm(const adj_dims *dims, const float *y, void *xhat, float *r, void *stream);

/* Cotangent through the normalisation: gy_prev = gy + (dxhat - xhat mean_p(xhat dxhat)) / r,
 * xhat = y / r recomputed from y [B,T,P] fp32 and r [B,T] from adj_rms_norm.
 * gy_prev [B,T,P] fp32 may alias dxhat or gy. */
adj_status adj_rms_norm_bwd(const adj_dims *dims, const float *y, const float *r, const float *dxhat,
                            const float *gy, float *gy_prev, void *stream);

/* ---------------------------------------------------------------------------
 * The general selective layer.  The pages give the layer only in its general form
 * h_t = A_t h_{t-1} + B_t xhat_t, y_t = C_t h_t with A_t, B_t, C_t functions of the token
 * ([AS] Circularity Check, assumptions); these calls take its selective reading, per
 * channel p < P and state n < N (N = 8 or 16):
 *     z_t = xhat_t W_in                      W_in [P, P+2N] = [W_dt | W_B | W_C]
 *     dt_t,p = softplus(z_t,p + b_dt,p),  B_t,n = z_t,P+n,  C_t,n = z_t,P+N+n
 *     Abar_t,pn = exp(dt_t,p A_pn)            A [P,N], the continuous-time decay
 *     h_t,pn = Abar_t,pn h_t-1,pn + dt_t,p B_t,n xhat_t,p   (h_-1 = 0)
 *     y_t,p = xres_t,p + sum_n C_t,n h_t,pn   (the residual identity; xres = xhat
 *                                             for a lone layer)
 * i.e. a PN-dimensional state with A_t = diag(Abar_t) and the full P x PN output map
 * C_t[p, (p,n)] = C_t,n.  Its gradient is the same sum over token pairs of independent
 * VJPs as the diagonal layer's ([AS] Core claim, Proposition 2), full or truncated to a
 * window.  Sizes: adj_dims with N = 8 or 16, P a multiple of 8, B <= 65535; x_dtype is
 * the storage of xhat and W_in, d_dtype that of dz.  h is [B,T,P,N] fp32 (state index
 * last).  No call waits on another CTA; adj_sel_bwd's waits for its own bulk copies are
 * bounded and record ADJ_ETIMEOUT in the workspace if one gives up.
 *
 * Stacks ([AS] What carries the argument: y^K = y^0 + sum_k ytilde^k; Load-bearing
 * premise: normalised inputs): layer 1 reads the input, layer k >= 2 reads the residual
 * stream y^{k-1} normalised per token, xhat^k = y^{k-1} / r (adj_rms_norm), with
 * xres = y^{k-1}.  Its input path then passes the cotangent down:
 *     gy^{k-1} = gy^k + (dxhat - xhat (xhat . dxhat) / P) / r,
 *     dxhat_t,p = (dz_t W_in^T)_p + dt_t,p sum_n mu_t,pn B_t,n
 * (the projection and the input term of the step), computed by adj_sel_bwd (r, gadd,
 * rowdot) and adj_sel_param_grad (gy_prev).
 * ------------------------------------------------------------------------- */
typedef struct {
    const void *W_in;    /* [P, P+2N] x_dtype */
    const float *b_dt;   /* [P] */
    const float *A;      /* [P, N] */
} adj_sel_weights;

/* Forward pass storing what the adjoint needs ([AS] Referee Report on Algorithm 1: the
 * per-token states are kept):
 *   xhat [B,T,P] x_dtype    layer input
 *   xres [B,T,P] fp32       residual input (NULL: xhat's values; a stacked layer passes
 *                           the residual stream y^{k-1} it normalised into xhat)
 *   z    [B,T,P+2N] fp32    xhat W_in, without b_dt (written)
 *   h    [B,T,P,N] fp32     states (written)
 *   y    [B,T,P] fp32       layer output (written; may not alias xres) */
adj_status adj_sel_fwd(const adj_dims *dims, const adj_sel_weights *w, const void *xhat, const float *xres,
                       float *z, float *h, float *y, void *ws, size_t ws_bytes, void *stream);

/* Columns of adj_sel_bwd's rowdot for these sizes (0 for sizes the selective calls reject). */
size_t adj_sel_rowdot_cols(const adj_dims *dims);

/* Adjoint of one selective layer for the cotangent gy = dL/dy [B,T,P] fp32: the window
 * sums mu_i = sum_{t=i}^{min(T-1, i+Tbar-1)} gy_t^T C_t prod_{j=i+1..t} A_j (all t >= i when
 * Tbar <= 0 or Tbar >= T; otherwise Tbar must be a multiple of 16), and the VJP of every
 * token's step and output map ([AS] Core claim, Proposition 2; last sentence: truncation):
 *   dz [B,T,P+2N] d_dtype   cotangent of z (written): columns p < P: the step's
 *                           (sum_n mu_pn (A_pn Abar_pn h_{t-1},pn + B_n xhat_p)) sigmoid(z_p + b_dt,p);
 *                           columns P+n: sum_p mu_pn dt_p xhat_p (B_t); P+N+n: sum_p gy_p h_t,pn (C_t)
 *   dA [P,N] fp32           sum_t mu_pn dt_p Abar_pn h_{t-1},pn (written)
 * xhat, z, h as written by adj_sel_fwd.
 * The input path of a stacked layer (all three or none; NULL for a lone layer or layer 1):
 *   r      [B,T] fp32                   the rms from adj_rms_norm (xhat = y^{k-1} / r)
 *   gadd   [B,T,P] fp32 (written)       gy + dt sum_n mu B / r, the input term's share
 *   rowdot [B*T, adj_sel_rowdot_cols] fp32 (written)  partial sums of xhat . dxhat, the
 *                                       projection's share taken as dz . z (z = xhat W_in,
 *                                       dz as stored), which adj_sel_param_grad sums
 * gadd may not alias gy. */
adj_status adj_sel_bwd(const adj_dims *dims, const adj_sel_weights *w, const void *xhat, const float *z,
                       const float *h, const float *gy, int64_t Tbar, void *dz, float *dA, const float *r,
                       float *gadd, float *rowdot, void *ws, size_t ws_bytes, void *stream);

/* Parameter gradients from dz ([AS] Core claim: the sum over tokens of the VJPs):
 *   dW_in [P, P+2N] fp32 = sum_t xhat_t^T dz_t,   db_dt [P] fp32 = sum_t dz_t[:P].
 * accumulate (0 or 1) adds into the outputs instead of overwriting them.
 * With the input path (r, gadd, rowdot from adj_sel_bwd and gy_prev, all or none; w->W_in
 * then required, w may be NULL otherwise): gy_prev [B,T,P] fp32 (written) =
 * gadd + (dz W_in^T - xhat m / P) / r with m the sum of rowdot's columns, the cotangent
 * of the residual stream y^{k-1} below. */
adj_status adj_sel_param_grad(const adj_dims *dims, const adj_sel_weights *w, const void *xhat, const void *dz,
                              float *dW_in, float *db_dt, const float *r, const float *gadd, const float *rowdot,
                              float *gy_prev, int accumulate, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * Operators of a language model built of such layers (library facilities; the pages
 * describe the gradient path only).
 *
 * Linear attention with a decay for each head: the selective recurrence with a matrix
 * state per head.  Per head h of H, with q and k of head h / (H / Hk):
 *     S_t = exp(g_t) S_{t-1} + k_t v_t^T        S_t [Dk, Dv]
 *     o_t = scale * q_t S_t
 * Arrays (ld*: elements from one token to the next, so q, k and v may be column slices
 * of one projection; sequences follow each other at T * ld*):
 *   q [B,T,Hk,Dk], k [B,T,Hk,Dk], v [B,T,H,Dv], o [B,T,H,Dv]   x_dtype
 *   g [B,T,H] fp32 (dense): the logarithm of the decay, expected <= 0.  exp(g) is taken as
 *     zero below -104 (minus infinity included): the state starts afresh at that token, and
 *     what came before leaves no trace in it, which packs several documents into one row
 *   s0, s1 [B,H,Dk,Dv] fp32 (dense): the states before the first and after the last token
 * A value that is not finite spreads to the outputs of its chunk of 128 tokens and onwards.
 * Sizes: Dk and Dv multiples of 8 from 8 to 128; Hk divides H; H, B <= 65535; every ld* at
 * least its row's heads times width and a multiple of 16 bytes.  x_dtype fp32: products in
 * fp32.  x_dtype bf16: fp32 sums of products of bf16 operands, in which every value between is a
 * sum of two or three bf16; states are fp32.  o, dq, dk and dv have their own rounding alone; s1, ds0
 * and dg are fp32 sums on tensor cores, off by 4e-7, 6e-7 and 7e-7 (2-norm) the largest seen.
 * ------------------------------------------------------------------------- */
typedef struct {
    int64_t B, T;
    int32_t H, Hk, Dk, Dv;
    int32_t x_dtype;
    float scale;
    int64_t ldq, ldk, ldv, ldo;
} adj_lin_dims;

/* Workspace bytes of ADJ_OP_LIN_FWD or ADJ_OP_LIN_BWD (0 for sizes the calls reject). */
size_t adj_lin_workspace_bytes(const adj_lin_dims *dims, int op);

/* Chunked form over T tokens.  s0 NULL: a state of zeros; s1 NULL: not written.  o may not
 * alias an input.  B*T = 0 copies s0 (or zeros) to s1. */
adj_status adj_lin_fwd(const adj_lin_dims *dims, const void *q, const void *k, const void *v, const float *g,
                       const float *s0, void *o, float *s1, void *ws, size_t ws_bytes, void *stream);

/* Gradients for the cotangents go [B,T,H,Dv] of o (x_dtype, pitch ldo) and ds1 of s1 (NULL:
 * zeros).  dq, dk, dv have the layout of q, k, v; dg [B,T,H] and ds0 fp32 (ds0 NULL: not
 * written).  q and k shared by several heads receive the sum over them, taken in a fixed
 * order.  dg is zero where exp(g) is taken as zero.  No output may alias an input. */
adj_status adj_lin_bwd(const adj_lin_dims *dims, const void *q, const void *k, const void *v, const float *g,
                       const float *s0, const void *go, const float *ds1, void *dq, void *dk, void *dv, float *dg,
                       float *ds0, void *ws, size_t ws_bytes, void *stream);

/* One token for each of B sequences (dims->T is not read; ld* are the distances between
 * sequences): state [n_slots,H,Dk,Dv] fp32 is updated in place, sequence b's in slot
 * slots[b] (slots NULL: slot b, needs n_slots >= B).  A slot outside [0, n_slots) leaves
 * the pool untouched and gives a row of zeros (the padding of a batch); a slot given twice is
 * a race.  No workspace. */
adj_status adj_lin_step(const adj_lin_dims *dims, const void *q, const void *k, const void *v, const float *g,
                        float *state, int64_t n_slots, const int32_t *slots, void *o, void *stream);

/* Log probabilities of given tokens.  Per row x = logits[n, :V] with lse = log sum_j e^x_j and
 * p_j = e^(x_j - lse):
 *   lse      [N] fp32
 *   logp     [N] fp32 = x_target - lse; a target outside [0, V) is not scored: 0, no gradient
 *   entropy  [N] fp32 = -sum_j p_j log p_j
 *   top_id   [N,top] int32, top_logp [N,top] fp32: the `top` largest, largest first, equal
 *            ones by the lower index (NaN counts as largest)
 *   dlogits  [N,V] x_dtype (row pitch ldd) = glp_n (1[j = target] - p_j)
 *                                            - gent_n p_j (log p_j + entropy_n),
 *            the gradient for given cotangents glp of logp and gent of entropy [N] fp32
 * Minus infinity in x is a masked token (p = 0, dlogits = 0, or glp_n where it is the target), and so in
 * effect is any value far below the row's largest; every finite value of the type is in range.  A row of
 * minus infinity alone has lse = -inf, logp = -inf, entropy = 0 and dlogits = 0; a row of one
 * finite value, however low, is uniform.  A NaN or +inf makes its row NaN.  Cotangents of the
 * entropy up to 7e32 leave masked tokens without a gradient.
 * Any output may be NULL (top_id and top_logp both or neither; top = 0 for neither); dlogits
 * needs glp or gent (a NULL one counts as zeros) and may be the logits array itself when
 * ldd = ld.  logits and dlogits need only their type's alignment, ld, ldd >= V.  top <= V and
 * top <= ADJ_LOGPROB_MAX_TOP; N < 2^28, V < 2^31.  One launch, no workspace. */
typedef struct {
    int64_t N, V, ld, ldd;
    int32_t x_dtype, top;
} adj_logprob_dims;
#define ADJ_LOGPROB_MAX_TOP 32
adj_status adj_logprob(const adj_logprob_dims *dims, const void *logits, const int64_t *targets, float *logp,
                       float *entropy, float *lse, int32_t *top_id, float *top_logp, const float *glp,
                       const float *gent, void *dlogits, void *stream);

/* Clipping gradients by their global norm: over all n values x of all tensors
 *   norm = sqrt(sum x^2),  coef = min(1, max_norm / (norm + ADJ_CLIP_EPS)),  dst = coef * src.
 * segs is a HOST array (copied at the call) of nseg tensors: src and dst device pointers of
 * n values of `dtype`, aligned to that type; dst = src clips in place (and with coef = 1
 * nothing is written then), any other overlap is an error of the caller; dst NULL: the tensor
 * counts in the norm only.  out: two device floats, norm and coef.  Sums are fp32: squares past
 * 3.4e38 make the norm infinite.  An infinite norm gives
 * coef 0, a NaN gives NaN (and NaN gradients): no call hides a step that has to be skipped.
 * Sums are in a fixed order: the same inputs give the same bits.  Up to 1000 tensors the blocks wait
 * for one another, with a limit: past it the status word is set, norm and coef are NaN, and what
 * has not been scaled stays as it was.  The first 256 bytes of ws have to be zero before the first
 * call, and before the next one after ADJ_ETIMEOUT. */
typedef struct {
    const void *src;
    void *dst;
    int64_t n;           /* below 2^40 */
    int32_t dtype;
    int32_t reserved;    /* zero */
} adj_grad_seg;
#define ADJ_CLIP_EPS 1e-6f
size_t adj_clip_workspace_bytes(void);
adj_status adj_grad_clip(const adj_grad_seg *segs, int64_t nseg, float max_norm, float *out, void *ws,
                         size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * What stands around a selective recurrence in such a model: a short causal convolution
 * before it, and the recurrence itself with states that come in and go out.
 *
 * Sequences.  packed = 0: B sequences of T tokens, one behind the other (arrays [B,T,..]).
 * packed = 1: B sequences of any lengths in T tokens together (arrays [T,..]); `offsets`
 * [B+1] int64 on the DEVICE, 0 <= offsets[0] <= .. <= offsets[B] <= T: sequence b is the
 * tokens offsets[b] to offsets[b+1], none if they are equal.  Tokens before offsets[0] and
 * from offsets[B] on belong to no sequence: their inputs count for nothing, and their rows of
 * the outputs stay as they were.  Offsets that break this rule give unspecified values, but
 * no access out of bounds.  A sequence without tokens passes its state through.  Nothing
 * reaches from one sequence into another, values that are not finite included (but for
 * gradients of parameters, which sum over all).
 * ld*: elements from one token to the next (so that arrays may be column slices of one
 * projection), multiples of 16 bytes.  No output may overlap an input (s1 with s0, ds0
 * with ds1, a step's y with what it reads) or another output; an input's address as an output is refused.  A pool of states has n_slots entries; slots [B] int32
 * gives the entry of each sequence (NULL: entry b, needs n_slots >= B).  A slot outside
 * [0, n_slots) leaves the pool untouched and gives a row of zeros (the padding of a batch; a pool without
 * entries may be NULL); a slot given twice is a race.
 * ------------------------------------------------------------------------- */

/* Short causal convolution, each channel with its own W taps.  With the list
 * c = s0[b,0..W-1), x_0, x_1, .. of a sequence:
 *     p_t = bias + sum_j w[p,j] c_{t+j},    y_t = p_t, or p_t sigmoid(p_t) with act = 1
 *   x, y [rows,P] x_dtype; w [P,W], bias [P] fp32 (bias NULL: zeros)
 *   s0, s1 [B,W-1,P] x_dtype: the last W-1 entries of the list before and after the tokens
 * P a multiple of 8, W 2 to 4; sums in fp32. */
typedef struct {
    int64_t B, T;
    int64_t ldx, ldy;
    int32_t P, W;
    int32_t x_dtype, packed, act;
    int32_t reserved;            /* zero */
} adj_conv_dims;

/* s0 NULL: zeros; s1 NULL: not written.  No workspace. */
adj_status adj_conv_fwd(const adj_conv_dims *dims, const void *x, const float *w, const float *bias, const void *s0,
                        const int64_t *offsets, void *y, void *s1, void *stream);

/* Workspace bytes of adj_conv_bwd (0 for sizes it rejects). */
size_t adj_conv_workspace_bytes(const adj_conv_dims *dims);

/* Gradients for the cotangents go [rows,P] of y (pitch ldy) and ds1 [B,W-1,P] of s1 (both
 * x_dtype; ds1 NULL: zeros): dx (pitch ldx), dw [P,W] fp32, dbias [P] fp32 (NULL: not written),
 * ds0 [B,W-1,P] x_dtype (NULL: not written).  Sums in a fixed order. */
adj_status adj_conv_bwd(const adj_conv_dims *dims, const void *x, const float *w, const float *bias, const void *s0,
                        const int64_t *offsets, const void *go, const void *ds1, void *dx, float *dw, float *dbias,
                        void *ds0, void *ws, size_t ws_bytes, void *stream);

/* One token for each of B sequences (dims->T and packed are not read; ld* are the distances
 * between sequences): state [n_slots,W-1,P] x_dtype is updated in place.  No workspace. */
adj_status adj_conv_step(const adj_conv_dims *dims, const void *x, const float *w, const float *bias, void *state,
                         int64_t n_slots, const int32_t *slots, void *y, void *stream);

/* Selective scan, per channel p and state n:
 *     d_t = softplus(dt_t + dt_bias),   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t
 *     v_t = sum_n C_t h_t + D x_t,      y_t = v_t, or v_t z_t sigmoid(z_t) with z
 *   x, dt, z, y [rows,P], Bm, Cm [rows,N] x_dtype; A [P,N], D, dt_bias [P] fp32
 *   s0, s1 [B,P,N] fp32: the states before the first and after the last token
 * A is expected <= 0; larger ones are allowed as long as products of exp(d A) over a sequence stay
 * finite.  dt of minus infinity is a step of zero: a token of finite x and B leaves the state as it is.
 * P a multiple of 8; N 8, 16, 32 or 64; states and sums in fp32. */
typedef struct {
    int64_t B, T;
    int64_t ldx, lddt, ldz, ldB, ldC, ldy;
    int32_t P, N;
    int32_t x_dtype, packed;
} adj_ssm_dims;

/* Workspace bytes of ADJ_OP_SSM_FWD or ADJ_OP_SSM_BWD (0 for sizes the calls reject). */
size_t adj_ssm_workspace_bytes(const adj_ssm_dims *dims, int op);

/* D, z, dt_bias, s0 NULL: zeros (z: no gate); s1 NULL: not written. */
adj_status adj_ssm_fwd(const adj_ssm_dims *dims, const void *x, const void *dt, const float *A, const void *Bm,
                       const void *Cm, const float *D, const void *z, const float *dt_bias, const float *s0,
                       const int64_t *offsets, void *y, float *s1, void *ws, size_t ws_bytes, void *stream);

/* Gradients for the cotangents go [rows,P] of y (x_dtype, pitch ldy) and ds1 of s1 (NULL: zeros).
 * dx, ddt, dz, dB, dC have the type and pitch of x, dt, z, Bm, Cm; dA, dD, ddt_bias, ds0 are fp32.
 * dD, ddt_bias, ds0 NULL: not written; dz is needed where z is given, and NULL without.  Sums in a
 * fixed order. */
adj_status adj_ssm_bwd(const adj_ssm_dims *dims, const void *x, const void *dt, const float *A, const void *Bm,
                       const void *Cm, const float *D, const void *z, const float *dt_bias, const float *s0,
                       const int64_t *offsets, const void *go, const float *ds1, void *dx, void *ddt, float *dA,
                       void *dB, void *dC, float *dD, void *dz, float *ddt_bias, float *ds0, void *ws,
                       size_t ws_bytes, void *stream);

/* One token for each of B sequences (dims->T and packed are not read; ld* are the distances
 * between sequences): state [n_slots,P,N] fp32 is updated in place.  No workspace. */
adj_status adj_ssm_step(const adj_ssm_dims *dims, const void *x, const void *dt, const float *A, const void *Bm,
                        const void *Cm, const float *D, const void *z, const float *dt_bias, float *state,
                        int64_t n_slots, const int32_t *slots, void *y, void *stream);

/* Sampling a token from logits, by given random numbers.  Per row x = logits[n, :V] with its largest
 * value m, and the row's settings (fp32, top_k int32; a NULL array: the value in brackets):
 *   weights   w_i = round(2^40 e^((x_i - m) / temperature)), whole numbers  [1]
 *   kept      a prefix of the order by x descending, then i ascending: those with
 *             w_i >= min_p 2^40 [0], of these the first top_k (<= 0: all) [0], of these the
 *             shortest prefix that holds at least top_p of their weight, and one at least [1]
 *   token     the first kept j, by index, with sum of the kept w_i, i <= j, > u[n] * their total
 *   logp      log(w_j / total), from (x_j - m) / temperature itself
 * u [N] fp32 in [0, 1) (others are taken as the nearest such number, NaN as 0).  Temperature 0 takes
 * the largest logit, the lowest index first; top_p >= 1 and min_p <= 0 keep all, min_p > 1 is taken as 1
 * (the weights of 2^40, equals of the largest logit among them), top_p <= 0 keeps the first alone.  Minus infinity
 * is a masked token, and so is one whose distance from m is beyond fp32.  Weights are off by one unit at most; as they
 * are whole numbers the result does not depend on the order of sums, and equal rows give equal tokens.
 * token [N] int64 and logp [N] fp32 (NULL: not written).  Without a finite value a row gives token -1 and
 * logp -inf; with a NaN or +inf in it, or a setting that is NaN or a negative temperature, token -1 and
 * logp NaN.  logits need only their type's alignment, ld >= V; N < 2^28, 1 <= V <= ADJ_SAMPLE_MAX_V.  One
 * launch, no workspace. */
#define ADJ_SAMPLE_MAX_V 393216
typedef struct {
    int64_t N, V, ld;
    int32_t x_dtype;
    int32_t reserved;            /* zero */
} adj_sample_dims;
adj_status adj_sample(const adj_sample_dims *dims, const void *logits, const float *u, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, int64_t *token, float *logp,
                      void *stream);

/* Synchronise `stream`, return and clear the sticky device status of `ws`
 * (ADJ_OK or ADJ_ETIMEOUT); ADJ_ECUDA if the stream reports an error. */
adj_status adj_stream_status(void *ws, void *stream);

/* Static description of a status code. */
const char *adj_status_str(adj_status s);

/* The forward pass of adj_fwd_scan for callers that cannot allocate device memory
 * (the paper has no counterpart: it concerns how scratch memory is obtained).
 * Scratch comes from a 32 MiB array inside the library, which every GPU that loads
 * the library holds until the process exits, so no workspace is passed.  Inputs and
 * outputs are as in adj_fwd_scan.  Problems whose adj_workspace_bytes(dims,
 * ADJ_OP_FWD, 0) exceeds 32 MiB are rejected with ADJ_EWORKSPACE before anything is
 * launched.  `status` (device pointer to one unsigned, NULL to skip) receives the
 * call's device status word after the launches (non-zero: a bounded wait gave up).
 * The first call on a device looks up the array's device address and must come
 * before any stream capture.  All calls share the array: calls that overlap on the
 * GPU race.  Allocates nothing (no cudaMalloc/cudaFree). */
adj_status adj_fwd_scan_noalloc(const adj_dims *dims, const adj_weights *w, const void *xhat,
                                const float *xres, float *a, float *c, float *h, float *y, void *y_x,
                                unsigned *status, void *stream);

/* Failure-path self test (a library facility with no counterpart on the pages): runs
 * the bounded device waits the kernels rely on against objects that are never released.
 *   which & 1: the scans' decoupled look-back -- the forward state scan kernel runs over a
 *              small problem held in ws whose first chunk is never launched, so every
 *              other chunk waits for a predecessor that never publishes (a few seconds);
 *   which & 2: an mbarrier wait (TMA staging, GEMM pipeline) on a barrier that is never
 *              arrived on (about 2 s).
 * Each wait gives up after its limit, records the timeout in ws's status word and returns;
 * adj_stream_status(ws) then reports ADJ_ETIMEOUT.  ws: device memory, 256-byte aligned,
 * at least adj_selftest_ws_bytes() bytes, status word zero before the call. */
size_t adj_selftest_ws_bytes(void);
adj_status adj_selftest_waits(void *ws, size_t ws_bytes, int which, void *stream);

/* 1 if this process's GEMMs may take the four-CTA layout, whose loads are multicast inside the
 * cluster: in a process that is no rank of several (WORLD_SIZE unset or 1) and sees one GPU at most,
 * unless ADJ_GEMM_QUAD=0.  Read once a process. */
int adj_gemm_multicast(void);

/* ---- Launch accounting and per-kernel timing (a library facility; the pages
 * describe no implementation, so these have no counterpart there).
 * adj_launch_count: kernels launched by this library since it was loaded.
 * adj_profile_enable(1): from now on every launch is bracketed by CUDA events
 *   on its stream; adj_profile_read(id, &n, &ms) synchronises on those events and
 *   returns the launch count and summed device time of kernel kind `id`
 *   (0 <= id < adj_profile_kernels(), named by adj_profile_name(id));
 *   adj_profile_reset() forgets all records.  Host-thread safe. */
unsigned long long adj_launch_count(void);
void adj_profile_enable(int on);
void adj_profile_reset(void);
int adj_profile_kernels(void);
const char *adj_profile_name(int id);
adj_status adj_profile_read(int id, int64_t *launches, double *total_ms);

#ifdef __cplusplus
}
#endif
#endif /* ADJ_H_ */
