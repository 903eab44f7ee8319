/*
 * mlstm_block.h -- C ABI of the operators that stand around the recurrence of
 * mlstm.h in a model: the short causal convolution before it, the selective
 * state space scan beside it, and the group norm with an activation or an
 * output gate after it.
 *
 * Conventions of mlstm.h hold: the caller owns every buffer, calls only
 * enqueue work on `stream`, nothing is allocated or synchronised, no state is
 * kept between calls, argument errors are found on the host before any launch
 * (MLSTM_ERR_INVALID, MLSTM_ERR_UNSUPPORTED, MLSTM_ERR_WORKSPACE), and a
 * failed launch is MLSTM_ERR_CUDA.  The calls run on the current device, may
 * be captured into graphs, and may run at the same time on several streams if
 * each has its own workspace.  Results do not depend on scheduling: sums over
 * tokens, channels and batches are taken in a fixed order, and atomics only
 * hand out work.  Some kernels wait, bounded, for another CTA's part of the
 * same launch; a wait that was given up is reported by mlstm_device_status.
 * A launch behind a failed one runs normally, and so does every replay of a
 * captured one: what a failure leaves for its own launch to see lies in the
 * workspace and is cleared when the launch starts, and each failure is counted.
 *
 * Sizes.  B T < 2^30, NH d <= 2^24, B NH d < 2^31, B T NH d < 2^40, and what the
 * operators say; other values return MLSTM_ERR_UNSUPPORTED.
 *
 * Types.  Activations and their gradients are in the one I/O dtype
 * (MLSTM_BF16 or MLSTM_FP32); parameters, their gradients and the scan's
 * states are fp32.  All arithmetic is fp32, rounded once to the I/O dtype; sums
 * over tokens are fp32 too, of partial sums over some hundred tokens each.
 * Exponentials are the hardware's (relative error 2^-22) of an argument
 * rounded to fp32: a decay of the scan, exp(delta A), is good to
 * (1 + 2 |delta A|) 2^-22.
 *
 * Strided tensors.  Activations are passed with their strides, so a slice of
 * a projection or a head-major tensor is read or written in place.  The last
 * dimension has stride 1; pointers are aligned to their element.  Where every
 * pointer and stride is a multiple of 16 bytes and the channel counts are
 * multiples of 8 the kernels use 16-byte accesses, else element accesses; the
 * results agree.  Outputs must not overlap inputs except where said.
 */
#ifndef MLSTM_BLOCK_H
#define MLSTM_BLOCK_H

#include <stddef.h>

#include "mlstm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A tensor of the I/O dtype: element (b, t, g, j) at
 * data[b batch + t token + g head + j], strides in elements. */
typedef struct {
  void* data;
  long long batch, token, head;
} mlstm_rows_t;

typedef enum { MLSTM_ACT_NONE = 0, MLSTM_ACT_SILU = 1, MLSTM_ACT_SIGMOID = 2 } mlstm_act_t;
typedef enum { MLSTM_SCOPE_TOKEN = 0, MLSTM_SCOPE_SEQUENCE = 1 } mlstm_scope_t;

/* ---------------------------------------------------------------------------
 * Short causal convolution, one filter of W taps per channel (D = NH d
 * channels), 2 <= W <= 4, act MLSTM_ACT_NONE or MLSTM_ACT_SILU:
 *
 *   pre[b, t, c] = bias[c] + sum_{j < W} weight[c, j] x[b, t - (W - 1) + j, c]
 *   y = act(pre)
 *
 * x [B, T, D]; weight [D, W]; bias [D] or NULL; y as [B, T, NH, d] with a head
 * stride, so that it can be written head-major for the recurrence (x.head is
 * ignored: x's channels are contiguous).
 *   state_in   [B, W - 1, D] contiguous, I/O dtype: the inputs before the first
 *              token, oldest first; NULL: zeros.
 *   state_out  the last W - 1 inputs, same layout; NULL: not wanted.  Must not
 *              overlap state_in.
 * ------------------------------------------------------------------------- */
int mlstm_conv_fwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                   const void* state_in, const mlstm_rows_t* y, void* state_out, int B, int T,
                   int NH, int d, int W, int act, int dtype, void* stream);

/* Bytes of workspace mlstm_conv_bwd needs (0 on an argument error). */
size_t mlstm_conv_bwd_workspace_size(int B, int T, int NH, int d, int W, int dtype);

/* Gradients of sum(dy y) + sum(dstate_out state_out): dx [B, T, D] (strided),
 * dweight [D, W], dbias [D] (NULL: not wanted) and dstate_in [B, W - 1, D]
 * (NULL: not wanted).  dy is laid out like y.  dstate_out NULL: none. */
int mlstm_conv_bwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                   const void* state_in, const mlstm_rows_t* dy, const void* dstate_out,
                   const mlstm_rows_t* dx, float* dweight, float* dbias, void* dstate_in,
                   void* workspace, size_t workspace_bytes, int B, int T, int NH, int d, int W,
                   int act, int dtype, void* stream);

/* One token: x [B, D] and y [B, NH, d] (their token strides are ignored).
 * Reads state_in, writes state_out (both required); they may be the same
 * buffer, but must not overlap otherwise. */
int mlstm_conv_step(const mlstm_rows_t* x, const float* weight, const float* bias,
                    const void* state_in, const mlstm_rows_t* y, void* state_out, int B, int NH,
                    int d, int W, int act, int dtype, void* stream);

/* ---------------------------------------------------------------------------
 * Selective state space scan: N states per channel with a diagonal
 * transition, 1 <= N <= 64, D channels in G groups (G divides D) that share B
 * and C:
 *
 *   delta = softplus(dt + dt_bias)      (or dt + dt_bias with softplus == 0)
 *   s[n] <- exp(delta A[c, n]) s[n] + delta x B[n]
 *   y    = (sum_n C[n] s[n] + skip[c] x) silu(z)
 *
 * x, dt, z, y [B, T, D] (head strides ignored); b, c [B, T, G, N] (head: the
 * stride between groups); a [D, N]; skip, dt_bias [D] or NULL (zeros); z.data
 * NULL: no gate.  state_in, state_out [B, D, N] fp32 contiguous, the state
 * before the first and after the last token; NULL: zeros / not wanted.  States,
 * saved and workspaces are 16-byte aligned.
 * a may be -infinity: a decay of 0.  Infinite and NaN inputs reach y and the
 * states as the formula in fp32 has them; gradients that the formula makes
 * infinite may be NaN.
 * ------------------------------------------------------------------------- */
typedef struct {
  mlstm_rows_t x, dt, z, b, c;
  const float *a, *skip, *dt_bias;
  const float* state_in;
  int B, T, D, G, N, softplus, dtype;
} mlstm_scan_t;

/* Bytes of `saved` that mlstm_scan_fwd fills and mlstm_scan_bwd reads: the
 * states entering every eighth token, fp32, N rounded up to 8, 16, 32 or 64
 * (0 on an argument error). */
size_t mlstm_scan_saved_size(int B, int T, int D, int G, int N, int dtype);

/* Bytes of workspace mlstm_scan_fwd needs; may be 0, and then the workspace
 * may be NULL (0 on an argument error too).  Few long sequences are cut into
 * segments that are scanned at once, whose states lie there. */
size_t mlstm_scan_fwd_workspace_size(int B, int T, int D, int G, int N, int dtype);

/* Forward.  saved NULL: no backward will follow.  state_out must not overlap
 * state_in.  T = 0 copies state_in (or zeros) to state_out. */
int mlstm_scan_fwd(const mlstm_scan_t* p, const mlstm_rows_t* y, void* saved, float* state_out,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace mlstm_scan_bwd needs (0 on an argument error).  Most of
 * it holds shares of db and dc, one for each tile of 64 channels (128, 32 and 16
 * for up to 8, 32 and 64 states): 8 bytes for each token, tile and rounded-up
 * state, 268 MB at B8 T4096 D4096 N16. */
size_t mlstm_scan_bwd_workspace_size(int B, int T, int D, int G, int N, int dtype);

/* Gradients of the scan; NULL data: that output is not wanted, except dx, ddt,
 * db, dc and da, which are always written. */
typedef struct {
  mlstm_rows_t dx, ddt, dz; /* [B, T, D]; dz is required when z is given */
  mlstm_rows_t db, dc;      /* [B, T, G, N] */
  float *da;                /* [D, N] */
  float *dskip, *ddt_bias;  /* [D] */
  float* dstate_in;         /* [B, D, N]; must not overlap dstate_out */
} mlstm_scan_grads_t;

/* Backward of sum(dy y) + sum(dstate_out state_out), dy [B, T, D], dstate_out
 * [B, D, N] or NULL; `saved` from the forward of the same inputs. */
int mlstm_scan_bwd(const mlstm_scan_t* p, const mlstm_rows_t* dy, const void* saved,
                   const float* dstate_out, const mlstm_scan_grads_t* grads, void* workspace,
                   size_t workspace_bytes, void* stream);

/* One token (p->T is ignored and taken as 1): reads p->state_in, writes
 * state_out (both required; they may be the same buffer, but must not overlap
 * otherwise). */
int mlstm_scan_step(const mlstm_scan_t* p, const mlstm_rows_t* y, float* state_out, void* stream);

/* ---------------------------------------------------------------------------
 * Group norm with an activation or an output gate.  x as [B, T, NH, d] (any
 * batch, token and head strides: channels last, or head-major as mlstm_fwd
 * writes it), groups = heads of d channels.  Statistics over the d channels of
 * one token (MLSTM_SCOPE_TOKEN, d <= 512) or over the T d values of a sequence
 * (MLSTM_SCOPE_SEQUENCE):
 *
 *   n = (x - mean) / sqrt(var + eps) weight + bias
 *   y = act(n)                 gate->data NULL
 *   y = n act(gate)            otherwise
 *
 * weight, bias [NH d] or NULL (1 / 0).  eps > 0.  stats: fp32 pairs (mean,
 * 1 / sqrt(var + eps)), [B, T, NH, 2] or [B, NH, 2], written by the forward
 * (NULL: not wanted) and read by the backward; T = 0 leaves them as they were.
 * Over a sequence a variance beyond fp32's range gives 1 / sqrt(var) = 0.
 * ------------------------------------------------------------------------- */
size_t mlstm_group_norm_stats_size(int B, int T, int NH, int d, int scope);

/* Workspace of the forward (backward == 0) or backward pass, in bytes; may be
 * 0, and then the workspace may be NULL. */
size_t mlstm_group_norm_workspace_size(int B, int T, int NH, int d, int scope, int dtype,
                                       int backward);

int mlstm_group_norm_fwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                         const mlstm_rows_t* gate, const mlstm_rows_t* y, float* stats,
                         void* workspace, size_t workspace_bytes, int B, int T, int NH, int d,
                         int scope, int act, float eps, int dtype, void* stream);

/* dgate is required when gate is given; dweight and dbias [NH d] may be NULL. */
int mlstm_group_norm_bwd(const mlstm_rows_t* x, const float* weight, const float* bias,
                         const mlstm_rows_t* gate, const mlstm_rows_t* dy, const float* stats,
                         const mlstm_rows_t* dx, const mlstm_rows_t* dgate, float* dweight,
                         float* dbias, void* workspace, size_t workspace_bytes, int B, int T,
                         int NH, int d, int scope, int act, int dtype, void* stream);

/* Self-test of the failure report, as mlstm_selftest_timeout: enqueue one tiny
 * kernel that waits as the kernels of `family` do, on a word that nothing
 * raises, gives up after 2 s and returns.  The next mlstm_device_status
 * returns MLSTM_ERR_TIMEOUT.  workspace: 8 bytes at least. */
typedef enum {
  MLSTM_WAITS_SCAN_FWD = 0,
  MLSTM_WAITS_SCAN_BWD = 1,
  MLSTM_WAITS_NORM = 2
} mlstm_block_waits_t;
int mlstm_block_selftest_timeout(int family, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLSTM_BLOCK_H */
