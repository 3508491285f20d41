/*
 * mlp_ops.h -- the individual operations of the MLP training step, callable
 * on caller-owned device buffers.  They run the same kernels mlp_train_step
 * runs; they exist so that each step of the path can be checked and timed on
 * its own at full size.
 *
 * Common conventions: device pointers on the current CUDA device; dense
 * row-major layouts with explicit leading dimensions (`ld*`, in elements);
 * dtype MLP_F32 (float) or MLP_BF16 (bfloat16 bits); `stream` is a
 * cudaStream_t.  Every call validates its arguments and returns before
 * enqueuing anything when they are invalid; it returns once its kernels are
 * enqueued.  Device-side conditions (label range, wait timeouts) are OR-ed
 * into `err_dev` (a device uint32, nullable) with the bits
 *   1 = label or index outside its range, 2 = non-finite loss, 4 = bounded wait gave up.
 * For MLP_BF16 the GEMM operands are read by TMA: every operand base must be
 * 16-byte aligned and every leading dimension a multiple of 8 elements.
 * The GEMM entry points (linear_act, dgrad, wgrad) also take MLP_F32X3:
 * every matrix argument that is fp32 under MLP_F32 (X, W, H, dY, dX) is then
 * three bf16 planes [3][rows][ld] (mlp.h), produced by mlp_op_split3; the
 * bias, dW and db stay fp32; S is read from its first (hi) plane only, so
 * only ReLU / no activation are accepted; the TMA rules of MLP_BF16 apply.
 */
#ifndef MLP_OPS_H_
#define MLP_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* LinearAct forward (noeira.ai "Neural networks", "The design in one page":
 * MatMul+Bias+Activation as one kernel, bias and activation in the GEMM
 * epilogue):  u = X W^T + b,  H = act(u),  U = u (optional, nullable).
 *   X [M, K] (ldx), W [N, K] (ldw), b fp32 [N], H [M, N] (ldh), U [M, N] (ldu).
 * Accumulation is fp32; H and U are rounded to the dtype. */
mlp_status mlp_op_linear_act(int dtype, int act, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                             const void* W, int64_t ldw, const float* b, void* H, int64_t ldh, void* U, int64_t ldu,
                             uint32_t* err_dev, void* stream);

/* dgrad with the activation VJP fused (noeira "The design in one page":
 * vjp per module):  dX = (dY W) * act'(S)
 *   dY [M, N] (ldy), W [N, K] (ldw), S [M, K] (lds) = what the forward of the
 *   layer below stored: h for ReLU (mask h > 0), u for GELU, unused for
 *   MLP_ACT_NONE (nullable); dX [M, K] (ldx). */
mlp_status mlp_op_dgrad(int dtype, int act, int64_t M, int64_t N, int64_t K, const void* dY, int64_t ldy,
                        const void* W, int64_t ldw, const void* S, int64_t lds, void* dX, int64_t ldx,
                        uint32_t* err_dev, void* stream);

/* The three bf16 planes of an fp32 matrix X [rows, cols] (ldx):
 * P [3][rows][ldp] with P[0] = bf16(X), P[1] = bf16(X - P[0]),
 * P[2] = bf16(X - P[0] - P[1]) (the MLP_F32X3 encoding, mlp.h). */
mlp_status mlp_op_split3(int64_t rows, int64_t cols, const float* X, int64_t ldx, void* P, int64_t ldp,
                         void* stream);

/* Workspace bytes mlp_op_wgrad needs for this shape (0 if none). */
size_t mlp_op_wgrad_workspace_bytes(int dtype, int64_t N, int64_t K, int64_t B);

/* wgrad with the bias gradient fused:  dW = dY^T X (fp32 [N, K], lddw),
 * db = sum over rows of dY (fp32 [N], nullable).
 *   dY [B, N] (ldy), X [B, K] (ldx).  The reduction over B may be split;
 *   partial sums go to `workspace` (device, ws_bytes >= the size above) and
 *   are added in a fixed order, so results are deterministic. */
mlp_status mlp_op_wgrad(int dtype, int64_t N, int64_t K, int64_t B, const void* dY, int64_t ldy, const void* X,
                        int64_t ldx, float* dW, int64_t lddw, float* db, void* workspace, size_t ws_bytes,
                        uint32_t* err_dev, void* stream);

/* mlp_op_wgrad without a workspace argument (the pages have no counterpart:
 * this is a convenience of this library).  Some callers cannot call
 * cudaMalloc: an application whose device memory belongs to another
 * allocator (a framework's caching pool, a fixed up-front reservation) has
 * no extra buffer to pass, and a latency-critical loop must not allocate,
 * since cudaMalloc/cudaFree can synchronise the device and fail under memory
 * pressure.  This entry point allocates nothing: the split-K partial sums go
 * to a built-in device array of 16 MiB, which every GPU that loads the
 * library holds until the process exits.
 *   Same arguments, layouts and results as mlp_op_wgrad, for every dtype it
 *   takes (MLP_F32, MLP_BF16, MLP_F32X3).  Returns MLP_ERR_SHAPE, before
 *   enqueuing anything, when the shape needs more than 16 MiB of scratch
 *   (mlp_op_wgrad_workspace_bytes tells how much).
 *   The array's device address is looked up (cudaGetSymbolAddress, with the
 *   device current) by the first call on a device, which should come before
 *   any stream capture; later calls look it up again unless their stream is
 *   capturing, so a cudaDeviceReset between calls leaves no stale address.
 *   Every call shares the one array per device: calls whose kernels overlap
 *   on the GPU (other streams, other threads) race on it and must be
 *   serialised by the caller.  Each call writes every scratch element it
 *   later reads, so nothing is carried over from a previous call. */
mlp_status mlp_op_wgrad_noalloc(int dtype, int64_t N, int64_t K, int64_t B, const void* dY, int64_t ldy,
                                const void* X, int64_t ldx, float* dW, int64_t lddw, float* db, uint32_t* err_dev,
                                void* stream);

/* Softmax cross-entropy, forward and backward in one pass over each row
 * (devpost "Orthon", "Selected Orthon vs. PyTorch results": one kernel reads
 * the logits once):  loss_rows[i] = logsumexp(z_i) - z_i[y_i] (fp32),
 * dz_i = (softmax(z_i) - onehot(y_i)) * grad_scale (dtype; grad_scale = 1/B
 * gives the gradient of the batch-mean loss).
 *   z [B, C] (ldz), labels int32 [B], dz [B, C] (lddz). */
mlp_status mlp_op_softmax_ce(int dtype, int64_t B, int64_t C, const void* z, int64_t ldz, const int32_t* labels,
                             float grad_scale, void* dz, int64_t lddz, float* loss_rows, uint32_t* err_dev,
                             void* stream);

/* Squared error of outputs z [B, C] (ldz, dtype) against fp32 targets t
 * [B, C] (ldt), the MSE loss (pypi "munet-nn", "Python training":
 * mse_loss):  loss_rows[i] = sum_j (z_ij - t_ij)^2 (fp32), dz_ij = (z_ij -
 * t_ij) * grad_scale (dtype; grad_scale = 2 / (B C) gives the gradient of
 * the mean over all elements, the loss being sum(loss_rows) / (B C)). */
mlp_status mlp_op_mse(int dtype, int64_t B, int64_t C, const void* z, int64_t ldz, const float* t, int64_t ldt,
                      float grad_scale, void* dz, int64_t lddz, float* loss_rows, void* stream);

/* A bf16 output layer fused with softmax cross-entropy, its VJPs included
 * (the softmax-CE-in-GEMM path of MLP_OPT_CE_GEMM): for h [B, K] (ldh, bf16),
 * W [C, K] (bf16, row pitch K), bias [C] (fp32) and labels int32 [B]:
 *   z = h W^T + bias, stored bf16 in z [B, C] (ldz);
 *   loss_rows[i] = logsumexp(z_i) - z_i[y_i] (fp32, from the stored logits);
 *   dX = (dz W) * act'(aux) [B, K] (ldx, bf16; act of the layer below: aux is
 *     its stored h for ReLU, u for GELU; MLP_ACT_NONE: aux unused), and
 *   dW = dz^T h (fp32 [C, K], lddw), db = sum_rows dz (fp32 [C]),
 * with dz = (softmax(z) - onehot(y)) / B formed on the fly from the stored
 * logits and never written.  C > 128; K and the pitches multiples of 8; ws
 * (device, 16-byte aligned) of mlp_op_linear_ce_workspace_bytes(B, C, K)
 * bytes.  Launches the forward GEMM, the statistics combine, the dgrad and
 * the wgrad (+ its split-K reduce).  A label outside [0, C) sets the error
 * bit in err_dev (its loss row is 0). */
size_t mlp_op_linear_ce_workspace_bytes(int64_t B, int64_t C, int64_t K);
mlp_status mlp_op_linear_ce(int64_t B, int64_t C, int64_t K, const void* h, int64_t ldh, const void* W,
                            const float* bias, const int32_t* labels, int act, const void* aux, int64_t ld_aux,
                            void* z, int64_t ldz, float* loss_rows, void* dX, int64_t ldx, float* dW, int64_t lddw,
                            float* db, void* ws, size_t ws_bytes, uint32_t* err_dev, void* stream);

/* loss = mean(loss_rows[0..B)) summed in a fixed order (device float). */
mlp_status mlp_op_loss_mean(int64_t B, const float* loss_rows, float* loss, uint32_t* err_dev, void* stream);

/* AdamW at step t >= 1 over flat fp32 planes p, g, m, v of n elements
 * (MuNet "What runs today": AdamW; noeira "The design in one page": moments
 * co-located per parameter):  m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2;
 * p = p - lr (m/(1-b1^t) / (sqrt(v/(1-b2^t)) + eps) + wd p).  w16 (nullable)
 * receives bf16(p) after the update.  Planes 16-byte aligned, w16 8-byte. */
mlp_status mlp_op_adamw(int64_t n, float* p, const float* g, float* m, float* v, void* w16, int64_t t, float lr,
                        float beta1, float beta2, float eps, float wd, void* stream);

/* One update of rule `kind` (MLP_OPTIM_ADAMW / _ADAM / _SGD of mlp.h, same
 * formulas) over flat fp32 planes of n elements, with global-norm clipping
 * when max_norm > 0: g is scaled by min(1, max_norm / (||g||_2 + 1e-6))
 * before the update (g itself is not changed) and ||g|| goes to norm_dev
 * (device float, nullable).  ws_dev (device, 16-byte aligned, at least
 * MLP_OPTIM_WS_FLOATS floats) holds per-block partial sums of squares; it is
 * needed only when clipping.  t >= 1 for the Adam rules (bias correction);
 * SGD ignores t, beta2, eps and v.  w16 (nullable) receives bf16(p).
 * Clipping launches two kernels (norm, then update), otherwise one. */
enum { MLP_OPTIM_WS_FLOATS = 1216 };
mlp_status mlp_op_optim(int kind, int64_t n, float* p, float* g, float* m, float* v, void* w16, int64_t t, float lr,
                        float beta1, float beta2, float eps, float wd, float max_norm, float* ws_dev,
                        float* norm_dev, void* stream);

/* The error path of the device waits, exercised without a fault: one thread
 * waits, through the same bounded wait every tensor-core kernel uses for its
 * pipeline barriers, for an mbarrier phase that nothing completes; after
 * limit_ns (at most 1 s) it gives up, sets the timeout bit (1 << 2, the bit
 * behind MLP_ERR_TIMEOUT) in err_dev and the kernel returns normally, so the
 * context stays usable. */
mlp_status mlp_op_wait_timeout_check(uint64_t limit_ns, uint32_t* err_dev, void* stream);

/* Row argmax of z [B, C] (ldz) into int32 out [B]; lowest index on ties. */
mlp_status mlp_op_argmax(int dtype, int64_t B, int64_t C, const void* z, int64_t ldz, int32_t* out, void* stream);

/* The k largest entries of every row of z [B, C] (ldz; MLP_F32 or MLP_BF16),
 * descending, the lowest column first among equals; NaN is below everything
 * and -0 equals +0:
 *   values fp32 [B, k] (ldv), indices int32 [B, k] (ldi),
 *   lse[i] = log sum_c exp(z_ic / T)  (fp32 [B], nullable),
 *   tail[i] the same over the columns not among the k  (fp32 [B], nullable;
 *   -infinity where nothing is left), as mlp_op_distill takes it.
 * 1 <= k <= 256, k <= C <= 384000; T = temperature, 1e-6 to 1e6 (it changes the two sums
 * alone).  Entries of -infinity are taken like others, last.  Where a row holds NaN or
 * +infinity its lse is NaN, and its tail NaN or +infinity unless only the k entries hold
 * it.  Any base and pitch.  Nothing written may overlap anything read. */
enum { MLP_TOPK_MAX = 256, MLP_TOPK_MAX_COLUMNS = 384000 };
mlp_status mlp_op_topk(int dtype, int64_t B, int64_t C, int64_t k, const void* z, int64_t ldz, float temperature,
                       float* values, int64_t ldv, int32_t* indices, int64_t ldi, float* lse, float* tail,
                       void* stream);

/* Distillation from a teacher's top logits: softmax cross-entropy's soft
 * sibling, forward and backward in one pass over each row of the student's
 * logits z [B, C] (ldz).  The teacher's row is k logits t_values fp32 [B, k]
 * (ldtv) at columns t_indices int32 [B, k] (ldti; distinct; -1: unused entry) and
 * t_tail fp32 [B] (nullable: -infinity), the log of what its other columns
 * add up to at temperature T (mlp_op_topk's tail).  With
 *   p_j = e^(t_j / T) / (sum_j e^(t_j / T) + e^tail),  p_r = 1 - sum_j p_j,
 *   q = softmax(z / T),  R = the sum of q over the columns not given:
 *   KD = sum_j p_j log(p_j / q_j) + p_r log(p_r / R)   (0 log 0 = 0),
 *   CE = logsumexp(z) - z_y   (labels int32 [B]; nullable where ce_weight is 0, not
 *   read then),
 *   loss_rows = w (ce_weight CE + kd_weight KD)   (fp32 [B]),
 *   dz = w grad_scale (ce_weight (softmax(z) - onehot(y)) + kd_weight / T g)
 *   (dtype, lddz; nullable: the loss alone; may be z with z's pitch),
 *   g = q_j - p_j at the teacher's columns, q (1 - p_r / R) at the others.
 * Without a tail that is the teacher's top renormalised (p_r = 0).  kd_weight = T^2
 * keeps the gradient's size over T.  w = row_weights fp32 [B] (nullable: 1); where
 * it is 0, loss and gradient are 0 whatever the row, its label and its teacher
 * hold.  A teacher's row with nothing in it (no entry above -infinity, no tail)
 * has KD 0.  A label or column out of range, or a column given twice, sets bit 1 of
 * err_dev, and that row's loss and gradient are 0.  A teacher that gives weight
 * (p_j that fp32 holds) where the student has none (z = -infinity) has an infinite loss;
 * a row of z that holds NaN or +infinity, or nothing but -infinity, gives NaN.
 * A row counts by its logits' differences: shifted as a whole it gives the same.
 * Shares are fp32's, each right to a few 2^-22 of itself and, beside a tail, to half a step of the
 * tail in fp32.  Where teacher and student are close, loss and gradient are what such shares leave:
 * at a high T, p and q differ by about |t - z| / T of themselves, and with a tail near 10 the loss is off
 * by about 2e-7 T of itself and the gradient by 1e-7 T of its largest entry (1e-4 at T = 1000; little
 * is left of either at 1e6).
 * 1 <= k <= 256, k <= C <= 384000; T from 1e-6 to 1e6.  Any base and pitch; rows of dz with
 * another address modulo 16 than z's are written element by element.  But for dz in z's
 * place, nothing written may overlap anything read. */
mlp_status mlp_op_distill(int dtype, int64_t B, int64_t C, int64_t k, const void* z, int64_t ldz,
                          const float* t_values, int64_t ldtv, const int32_t* t_indices, int64_t ldti,
                          const float* t_tail, const int32_t* labels, const float* row_weights, float temperature,
                          float ce_weight, float kd_weight, float grad_scale, void* dz, int64_t lddz,
                          float* loss_rows, uint32_t* err_dev, void* stream);

/* Beam search's step: of every batch entry's beams x C pairs (beam, token) the m
 * best, best first, by
 *   total(w, c) = scores[w] + z_wc - logsumexp(z_w),
 * z [batch * beams, C] (ldz; MLP_F32 or MLP_BF16), scores fp32 [batch, beams] the beams'
 * log-probabilities so far.  A finished beam (done uint8 [batch, beams] not 0;
 * nullable: none) offers token eos at total scores[w] and every other at -infinity,
 * and its logits are not read.
 *   scores_out fp32, parents int32 (the beam), tokens int32 [batch, m]; done_out
 *   uint8 [batch, m] (nullable): the parent was finished or the token is eos (eos
 *   may be -1, no end token, where done is null).
 * Totals are formed and compared in 64 bits from each row's logsumexp, whose sum is fp32's (off
 * by about 3e-7): a beam's own tokens are in the order of their logits, and pairs of different
 * beams whose totals are closer than that may come in either order.  Equal totals go by beam,
 * then by logit and token (by token alone where a beam's logits are not read).  A beam of score
 * -infinity, finished or not, has every total -infinity (a search starts with scores
 * 0, -infinity, ...), and so has a row of nothing but -infinity; one whose score is NaN or
 * +infinity or whose row holds NaN or +infinity has NaN, below everything.
 * beams <= 32, m <= 64, m <= beams * C, C <= 384000.  With m = beams, scores_out may be scores
 * and done_out may be done (refused with another m); nothing else written may overlap anything
 * read.  workspace: 8-byte aligned, at least the bytes below (0: a shape that is refused);
 * workspaces of calls that may overlap must not. */
size_t mlp_op_beam_select_workspace_bytes(int dtype, int64_t batch, int64_t beams, int64_t C, int64_t m);
mlp_status mlp_op_beam_select(int dtype, int64_t batch, int64_t beams, int64_t C, int64_t m, const void* z,
                              int64_t ldz, const float* scores, const uint8_t* done, int32_t eos, float* scores_out,
                              int32_t* parents, int32_t* tokens, uint8_t* done_out, void* workspace, size_t ws_bytes,
                              void* stream);

/* The states that go with the beams (keys and values, recurrent states, token
 * histories), after a selection: for every plane p (a layer's tensor), batch entry b
 * and new beam i
 *   dst(p, b, i) = src(p, b, parents[b, i]),
 * rows of row_bytes bytes at src + p src_plane + (b beams_in + beam) src_pitch, likewise
 * dst (pitches and planes in bytes), parents int32 [batch, beams_out] (ldp: a
 * selection's m entries of which beams_out are taken).  dst may be src with the
 * same layout: rows that stay where they are are not touched then.  Otherwise
 * nothing written may overlap anything read.  A parent outside [0, beams_in) sets bit 1 of
 * err_dev and leaves its row as it was.  beams <= 32; moved in units of 16 bytes (8 for more
 * than 8 beams, 4 for more than 16) where bases, pitches and row_bytes allow it, else
 * of 4, 2 or 1. */
mlp_status mlp_op_beam_reorder(int64_t planes, int64_t batch, int64_t beams_in, int64_t beams_out, int64_t row_bytes,
                               const void* src, int64_t src_pitch, int64_t src_plane, const int32_t* parents,
                               int64_t ldp, void* dst, int64_t dst_pitch, int64_t dst_plane, uint32_t* err_dev,
                               void* stream);

/* Layer norm over the rows of X [M, D] (ldx; MLP_F32 or MLP_BF16), the norm
 * in front of a feed-forward block:
 *   mean_i = sum_j X_ij / D,  rstd_i = 1 / sqrt(sum_j (X_ij - mean_i)^2 / D
 *   + eps),  Y_ij = (X_ij - mean_i) rstd_i gamma_j + beta_j.
 *   gamma, beta fp32 [D] (nullable: 1 and 0); Y [M, D] (ldy, dtype; may be
 *   X with X's pitch); mean, rstd fp32 [M] (nullable: not kept).  eps >= 0 and finite.
 * Any D up to 65535 * 256 and any pitch.  Rows move 16 bytes at a time where D,
 * base and pitch allow it, else 4 bytes, else an element.  Statistics are
 * fp32, from the elements as stored: squares of differences from the mean
 * leave fp32 above 1e19 (rstd 0) and lose bits below 1e-19.  A row that holds
 * NaN or an infinity has y and rstd NaN. */
mlp_status mlp_op_layernorm(int dtype, int64_t M, int64_t D, const void* X, int64_t ldx, const float* gamma,
                            const float* beta, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
                            void* stream);

/* Its vector-Jacobian product: with xh = (X - mean) rstd and w = gamma dY,
 *   dX = rstd (w - mean_j(w) - xh mean_j(w xh))   (dtype, lddx; may be dY with
 *   dY's pitch),
 *   dgamma_j = sum_i dY_ij xh_ij,  dbeta_j = sum_i dY_ij  (fp32 [D], nullable).
 * X, mean and rstd are what the forward read and kept.  workspace (device, at
 * least the bytes below for this shape) holds per-block partial sums of
 * dgamma and dbeta, added in a fixed order; it is not needed where both are
 * null.  Workspaces of calls that may overlap must not. */
size_t mlp_op_layernorm_backward_workspace_bytes(int dtype, int64_t M, int64_t D);
mlp_status mlp_op_layernorm_backward(int dtype, int64_t M, int64_t D, const void* dY, int64_t lddy, const void* X,
                                     int64_t ldx, const float* gamma, const float* mean, const float* rstd, void* dX,
                                     int64_t lddx, float* dgamma, float* dbeta, void* workspace, size_t ws_bytes,
                                     void* stream);

/* Activation checkpoints in 8 bits: a matrix kept between the forward and the
 * backward pass as e4m3 codes with one scale per row and 32 columns (about
 * half the bytes of bf16).  For a block of 32 columns with amax its largest
 * finite magnitude, k is the smallest exponent >= -120 with amax <= 448 2^k;
 * E holds k + 127, Q the values X 2^-k rounded to e4m3 (to nearest, ties to
 * even).  A code stands for e4m3 * 2^k, exact in fp32 and in bf16, off by at
 * most 2^-4 of the value, or 2^(k - 10) where that is more: 2^-17.8 of the
 * block's amax, but 2^-130 where amax is below 224 * 2^-120 and k stays at -120.
 * Infinities and NaN are kept as NaN; a magnitude of 2^128 (1 - 2^-5) or more
 * reads back as infinite.  Read back, E may hold any byte: 255, which stands for
 * no k, makes its block's values NaN.
 *   X, Y [rows, cols] (ldx, ldy; MLP_F32 or MLP_BF16), Q uint8 [rows, cols]
 *   (ldq), E uint8 [rows, ceil(cols / 32)] (lde).
 * Any pitch; 16-byte aligned rows of X / Y with 8-byte aligned rows of Q move
 * by wide accesses.  Nothing written may overlap anything read. */
mlp_status mlp_op_quant8(int dtype, int64_t rows, int64_t cols, const void* X, int64_t ldx, uint8_t* Q, int64_t ldq,
                         uint8_t* E, int64_t lde, void* stream);
mlp_status mlp_op_dequant8(int dtype, int64_t rows, int64_t cols, const uint8_t* Q, int64_t ldq, const uint8_t* E,
                           int64_t lde, void* Y, int64_t ldy, void* stream);

/* The gated feed-forward projection of a language-model block: both
 * projections, the activation and the product in one kernel,
 *   s = X W^T + b,  g = s[:, :F],  u = s[:, F:],  H = act(g) * u.
 *   X [M, K] (ldx); W [2F, K] (ldw), the gate's F rows and then the up
 *   projection's; b fp32 [2F], nullable; H [M, F] (ldh).
 *   act: MLP_ACT_NONE, _RELU, _GELU_TANH or MLP_ACT_SILU (g / (1 + e^-g)).
 * s is kept for the backward when S is set: in the dtype, S [M, 2F] (lds); or
 * with SE set as an 8-bit checkpoint (mlp_op_quant8), S uint8 [M, 2F] the
 * codes and SE uint8 [M, 2 ceil(F / 32)] (ldse) the scales, the gate's blocks
 * first (gate and up half each as one matrix of F columns).  H comes from the
 * fp32 sums, before s is rounded; a gate that is NaN gives NaN with every act.  MLP_F32 or MLP_BF16; MLP_BF16 takes K, F
 * and the leading dimensions (but ldse) in multiples of 8 and 16-byte aligned
 * matrices (S codes: 8-byte).  M from one token on (MLP_F32: to 65535 * 128).
 * Nothing written may overlap anything read. */
enum { MLP_ACT_SILU = 3 };   /* the gated operations only */
mlp_status mlp_op_gated_linear(int dtype, int act, int64_t M, int64_t F, int64_t K, const void* X, int64_t ldx,
                               const void* W, int64_t ldw, const float* b, void* H, int64_t ldh, void* S, int64_t lds,
                               uint8_t* SE, int64_t ldse, uint32_t* err_dev, void* stream);

/* Its vector-Jacobian product, through the down projection Y = H Wd^T that
 * follows it (mlp_op_dgrad with the gate in the epilogue):
 *   dH = dY Wd,  dS = [dH * u * act'(g) | dH * act(g)],  H = act(g) * u.
 *   dY [M, N] (lddy); Wd [N, F] (ldw); S (lds), SE (ldse) what the forward
 *   kept; dS [M, 2F] (ldds); H [M, F] (ldh), nullable: formed again from s,
 *   so that it need not be kept for dWd = dY^T H.
 * dX and the projections' gradients are mlp_op_dgrad(MLP_ACT_NONE) and
 * mlp_op_wgrad (or _wgrad8) of dS and W with 2F output columns.  ReLU's
 * derivative at 0 is 0.  Types and alignment as above, N a multiple of 8;
 * nothing written may overlap anything read. */
mlp_status mlp_op_gated_dgrad(int dtype, int act, int64_t M, int64_t N, int64_t F, const void* dY, int64_t lddy,
                              const void* Wd, int64_t ldw, const void* S, int64_t lds, const uint8_t* SE, int64_t ldse,
                              void* dS, int64_t ldds, void* H, int64_t ldh, uint32_t* err_dev, void* stream);

/* mlp_op_wgrad with the layer's input kept as an 8-bit checkpoint:
 *   dW = dY^T X (fp32 [N, K], lddw), db = sum over rows of dY (nullable),
 *   dY [B, N] (ldy; MLP_F32 or MLP_BF16), X [B, K] the values of Q (ldq), E
 *   (lde).  The values are read back into the workspace (16-byte aligned, at
 *   least the bytes below; the dtype holds them exactly): the result is that
 *   of mlp_op_wgrad on them up to the order of its sums (bf16: none of them over
 *   more than 2048 rows on the tensor cores).  MLP_BF16 takes K and
 *   lddw in multiples of 4, ldy of 8 and 16-byte aligned dY and dW.
 *   Workspaces of calls that may overlap must not. */
size_t mlp_op_wgrad8_workspace_bytes(int dtype, int64_t N, int64_t K, int64_t B);
mlp_status mlp_op_wgrad8(int dtype, int64_t N, int64_t K, int64_t B, const void* dY, int64_t ldy, const uint8_t* Q,
                         int64_t ldq, const uint8_t* E, int64_t lde, float* dW, int64_t lddw, float* db,
                         void* workspace, size_t ws_bytes, uint32_t* err_dev, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MLP_OPS_H_ */
