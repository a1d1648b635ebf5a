/*
 * moe.h -- C ABI of libmoe: one mixture-of-experts layer on one GPU: its
 * forward pass (router -> token dispatch -> grouped SwiGLU experts ->
 * combine), its backward pass, the clipping of gradients by their norm, and
 * what a training step does next: AdamW and the update of a balance bias.
 *
 * Sources, by page title and section:
 *   [EP]       Transformers docs, "Expert parallelism" (intro): a router sends
 *              each token to a few experts and gathers the results.
 *   [EP-add]   same page, "Adding an implementation": the expert call takes
 *              (hidden_states, top_k_index, top_k_weights), runs the experts
 *              through experts_forward(tokens, expert_ids, weights), and
 *              returns each token's weighted expert output.
 *   [EP-disp]  same page, "Token dispatch": each (token, expert) pair goes to
 *              its expert, the experts run on what arrives, and the results
 *              are combined with the routing weights.
 *   [EP-impl]  same page, "Choosing an implementation": a path without host
 *              synchronisation can be captured in a CUDA graph.
 *   [TP-pack]  Transformers docs, "Tensor parallelism for inference",
 *              "Packed strategies": gate_up_proj is (num_experts, hidden,
 *              2*expert_dim), applied with a batched matmul and split with
 *              chunk(2, dim=-1) into (gate, up).
 *
 * Notation: T tokens, d hidden size, E experts, k experts per token, f expert
 * FFN width, P = T*k routed (token, expert) pairs.
 *
 * Conventions shared by every entry point:
 *   - All tensors are dense, row-major, and live in DEVICE memory unless an
 *     argument says "host".  The caller allocates and owns every buffer,
 *     including the workspace; the library never allocates or frees memory.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream) and never synchronises with the host, so a
 *     sequence of calls can be captured in a CUDA graph [EP-impl].
 *     moe_last_device_error() is the one call that synchronises.
 *   - Calls with buffers and workspaces of their own may be queued on several
 *     streams.  But order bf16 calls of moe_forward, moe_route and
 *     moe_grouped_swiglu, of their _scored forms and of their gradients by
 *     events where E >= 64 or 64 <= P / E < 512, as the Python layer does, so
 *     that no other of these runs beside them: two side by side have, seldom,
 *     not ended, for a cause that is not known.
 *   - Arguments are checked on the host before anything is launched; a
 *     failed check launches nothing and returns the status.  Returned
 *     statuses describe launch-time problems; problems found by a kernel
 *     (an expert id out of range, a bounded wait that ran out) are recorded
 *     in a device error word read by moe_last_device_error().
 *   - T == 0 is legal: the call returns MOE_OK and launches nothing.
 *   - An expert may receive zero pairs.
 *   - Activation dtype (x, expert weights, x_perm, h_perm, y_perm, out):
 *     MOE_BF16 (fp32 accumulation everywhere) or MOE_F32.  The router weight,
 *     logits and routing weights are always fp32.
 *   - Alignment: every pointer 16-byte aligned; d and f multiples of 8.
 *   - Limits: 1 <= k <= min(E, 32), E <= 1024, P < 2^31.
 *   - Device: the current CUDA device must be an sm_103 GPU (GB300); the
 *     library carries code for that architecture only.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,    /* null pointer, bad size, misalignment */
    MOE_ERR_UNSUPPORTED = -2,    /* shape/dtype outside the limits above, or no sm_103 device */
    MOE_ERR_WORKSPACE = -3,      /* ws_bytes smaller than the call needs */
    MOE_ERR_CUDA = -4,           /* a CUDA runtime/driver call failed */
    MOE_ERR_DEVICE_TIMEOUT = -5, /* a kernel's bounded wait ran out (device error word) */
    MOE_ERR_BAD_ROUTING = -6     /* a kernel met an expert id outside [0, E) (device error word) */
} moe_status_t;

typedef enum {
    MOE_F32 = 0,
    MOE_BF16 = 1,
    MOE_E4M3 = 2 /* states of moe_adamw_step only */
} moe_dtype_t;

typedef struct {
    int64_t T;           /* tokens in the batch (>= 0) */
    int32_t d;           /* hidden size */
    int32_t E;           /* number of experts */
    int32_t k;           /* experts per token */
    int32_t f;           /* expert FFN width (gate and up each have f columns) */
    int32_t act_dtype;   /* moe_dtype_t */
    int32_t renormalize; /* 1: divide the chosen k softmax weights by their sum; 0: keep them */
    int32_t scale_inputs;  /* 0: routing weights scale the expert outputs in the combine;
                              1: they scale the expert inputs in the dispatch and the
                              combine sums unweighted (experts that receive tokens already
                              scaled by the router score [EP]; with k == E every expert
                              sees every token: the form with nothing to dispatch) */
} moe_config_t;

/* Human-readable name of a status.  Never NULL; the string is static. */
const char *moe_status_string(moe_status_t status);

/* Detail of the last failed call on this host thread (empty if none). */
const char *moe_last_error_message(void);

/*
 * Bytes of workspace moe_forward needs for `cfg` (0 when T == 0).  The same
 * buffer also satisfies moe_route and moe_dispatch.  The workspace holds the
 * router logits and scratch, routing, dispatch arrays and the permuted
 * activations h_perm, y_perm and, where moe_forward uses it, x_perm (see
 * moe_workspace_layout).  The
 * router's share depends on the current device's SM count (its K splits
 * fill one wave); with no usable device it is sized for 152 SMs.
 */
size_t moe_workspace_size(const moe_config_t *cfg);

/*
 * Where moe_forward keeps its intermediates inside its workspace: byte
 * offsets from the start of the buffer (each 256-byte aligned).  After a
 * moe_forward call has completed, these regions hold that call's router
 * logits, routing, dispatch arrays and permuted activations, so a caller can
 * read, for instance, the chosen experts and weights of every token.
 *   logits    float [T][E]   (including logit_bias)
 *   topk_idx  int32 [T][k],  topk_w float [T][k]
 *   counts    int32 [E],     offsets int32 [E+1]
 *   pos       int32 [P],     src_token int32 [P]   (as moe_dispatch defines them)
 *   x_perm    act [P][d],    h_perm act [P][f],    y_perm act [P][d]
 *   total     = moe_workspace_size(cfg)
 * Any other bytes of the workspace are library scratch.  x_perm is
 * MOE_WS_ABSENT (no such region: the workspace is that much smaller) when
 * moe_forward does not form the permuted rows: with k == E the experts read
 * x directly, and where the first grouped GEMM gathers its rows from x it
 * reads them through src_token (see moe_forward).  T == 0 gives all zeros.  Returns MOE_ERR_INVALID_ARG /
 * MOE_ERR_UNSUPPORTED for a config moe_forward would reject, or a NULL
 * `layout`.  Launches nothing (it only queries the current device's SM
 * count, as moe_workspace_size does).
 */
#define MOE_WS_ABSENT ((size_t)-1)
typedef struct {
    size_t logits, topk_idx, topk_w, counts, offsets, pos, src_token;
    size_t x_perm, h_perm, y_perm;
    size_t total;
} moe_workspace_layout_t;

moe_status_t moe_workspace_layout(const moe_config_t *cfg, moe_workspace_layout_t *layout);

/* Bytes of workspace moe_dispatch needs for `cfg`: the per-chunk expert
 * count matrix (E x chunks int32) and a 16-byte ticket counter. */
size_t moe_dispatch_workspace_size(const moe_config_t *cfg);

/*
 * Number of kernel launches one moe_forward call makes for `cfg`: the router
 * (1 to 3 launches, by path), the dispatch (2; 1 when k == E, except for
 * fp32 with scale_inputs, and 1 when it copies unscaled rows with E <= 16
 * and P <= 16384 as described at moe_dispatch), the two grouped GEMMs (2, or
 * 4 when bf16 experts average 64 to 511 rows each and are split between two
 * tile shapes) and the combine (1).  0 when T == 0; -1 for an invalid
 * configuration.  Makes no CUDA call.
 */
int moe_forward_kernel_launches(const moe_config_t *cfg);

/*
 * Bytes of workspace moe_route needs for `cfg`: 0 when the logits are
 * computed on the CUDA cores (fp32 activations, E < 64 or E > 256, E not a
 * multiple of 16, or d not a multiple of 64); otherwise the three-term bf16
 * split of Wr (E * 3d * 2 bytes) and fp32 partial logits of the K splits.
 */
size_t moe_route_workspace_size(const moe_config_t *cfg);

/*
 * Router [EP-add: the router yields top_k_index and top_k_weights].
 *   logits[t][e] = sum_i x[t][i] * Wr[e][i] + (logit_bias ? logit_bias[e] : 0),
 *     computed in fp32 and written to `logits`;
 *   topk_idx[t][j]: the j-th largest logit of row t; equal logits go to the
 *     lower expert id (+0.0 and -0.0 are equal); a NaN ranks below every
 *     number;
 *   topk_w[t][j] = p_e / (renormalize ? sum of p over the chosen k : 1) with
 *     p = softmax over all E logits of row t.
 * x          [T][d]  act dtype
 * Wr         [E][d]  fp32 (nn.Linear layout)
 * logit_bias [E]     fp32 or NULL: an additive per-expert logit offset
 * logits     [T][E]  fp32, written
 * topk_idx   [T][k]  int32, written; topk_w [T][k] fp32, written
 * ws         at least moe_route_workspace_size(cfg) bytes, 256-byte aligned
 *            (may be NULL when that size is 0)
 * The selection is made on exactly the fp32 values written to `logits`.
 * For bf16 x, d % 64 == 0 and either 64 <= E <= 256 or (8 <= E < 64 and
 * T >= 1024), with E % 8 == 0, the products are formed on the tensor cores:
 * Wr is split into three bf16 terms
 * (w = w1 + w2 + w3, ~2^-25 relative), each product with the exact bf16 x is
 * exact, and accumulation is fp32; otherwise fp32 FMAs on the CUDA cores.
 */
moe_status_t moe_route(const moe_config_t *cfg, const void *x, const float *Wr,
                       const float *logit_bias, float *logits, int32_t *topk_idx,
                       float *topk_w, void *ws, size_t ws_bytes, void *stream);

/*
 * The selection and weights of moe_route on a GIVEN fp32 logit buffer
 * [T][E] (read only).  Writes topk_idx [T][k] and topk_w [T][k].
 */
moe_status_t moe_route_from_logits(const moe_config_t *cfg, const float *logits,
                                   int32_t *topk_idx, float *topk_w, void *stream);

/*
 * Token dispatch, single-device form [EP-disp]: every (token, slot) pair is
 * given a row of the expert-contiguous order.
 *   counts[e]     = number of pairs with topk_idx == e                 [E]
 *   offsets[e]    = sum_{e' < e} counts[e'];  offsets[E] = P            [E+1]
 *   pos[t*k+j]    = row of pair (t, j): offsets[e] + the number of pairs
 *                   (t', j') with topk_idx == e and t' < t (stable, so
 *                   rows of one expert are in ascending token order)    [P]
 *   src_token[r]  = token of row r (src_token[pos[q]] == q / k)         [P]
 *   x_perm[r][:]  = x[src_token[r]][:]                                  [P][d] act dtype
 *                   (scale_inputs: topk_w[q] * x[t][:], formed in fp32 and
 *                   rounded once to the act dtype, for the pair q of row r)
 * topk_idx is [T][k] int32; each entry must lie in [0, E) -- an entry outside
 * sets MOE_ERR_BAD_ROUTING in the device error word and that pair is dropped.
 * topk_w [T][k] fp32: read only when cfg->scale_inputs (may be NULL otherwise).
 * ws: at least moe_dispatch_workspace_size(cfg) bytes, 256-byte aligned.
 * Two launches: a rank kernel (per-chunk counts, stable ranks, and, in its
 * last block, the scan that yields counts and offsets) and a kernel that
 * places every pair's row and copies it.  The rank kernel's ticket counter
 * in ws is cleared first with a 4-byte cudaMemsetAsync on `stream`.
 * One launch, with ws not touched and no memset, when E <= 16, P <= 16384,
 * the rows are not scaled and a row is k KB to 16 KB (d * element size):
 * every block of that launch counts all P ids itself and places its own
 * tokens' pairs.
 */
moe_status_t moe_dispatch(const moe_config_t *cfg, const int32_t *topk_idx,
                          const float *topk_w, const void *x, int32_t *counts,
                          int32_t *offsets, int32_t *pos, int32_t *src_token,
                          void *x_perm, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_dispatch without a caller workspace.  (The pages have no counterpart:
 * this is a deployment variant of the same dispatch.)
 *
 * For callers that cannot allocate device memory for scratch: a plugin whose
 * host framework owns all device memory and passes only the layer's inputs
 * and outputs, or a service that must not call cudaMalloc after start-up.
 * The scratch moe_dispatch would take from `ws` (its count matrix and ticket
 * counter) lives instead in a fixed 1 MiB array inside the library.  Results are
 * identical to moe_dispatch.  This call allocates nothing and calls no
 * allocating routine.
 * The array belongs to the library's device code.  With CUDA's lazy module
 * loading (the default), that code, and with it the array's 1 MiB, may be
 * loaded onto a device only when the library first uses the device; from
 * then on the device holds it until the process exits.  A service that must
 * not commit device memory once it is serving should therefore make one
 * call (any T > 0) on each device at start-up.
 *
 * Limit: moe_dispatch_workspace_size(cfg) must be <= 1 MiB (E times the
 * number of 2048-pair chunks <= 262,140: any P for E <= 256; P <= 522,240
 * for E = 1024); larger sizes return MOE_ERR_UNSUPPORTED and launch nothing.
 * Set-up: the first call with T > 0 on a device looks up the array's device
 * address (cudaGetSymbolAddress) with that device current, once, and keeps
 * it; make that first call before any stream capture.  The kept address is
 * not refreshed, so a device reset (cudaDeviceReset, or a teardown and
 * re-creation of the primary context) after the first call is not
 * supported.  All calls on a device share the array, so calls whose kernels
 * overlap on the GPU race: serialise them.
 * Other arguments, errors and outputs are as for moe_dispatch.
 */
moe_status_t moe_dispatch_noalloc(const moe_config_t *cfg, const int32_t *topk_idx,
                                  const float *topk_w, const void *x, int32_t *counts,
                                  int32_t *offsets, int32_t *pos, int32_t *src_token,
                                  void *x_perm, void *stream);

/*
 * Grouped SwiGLU experts [EP-add: experts_forward; TP-pack]: for every expert
 * e and every row r in [offsets[e], offsets[e+1]):
 *   gu        = x_perm[r] @ W_gate_up[e]        (W_gate_up: [E][d][2f])
 *   h_perm[r] = silu(gu[0:f]) * gu[f:2f],  silu(z) = z / (1 + exp(-z))
 *   y_perm[r] = h_perm[r] @ W_down[e]           (W_down: [E][f][d])
 * x_perm [P][d], h_perm [P][f] (written), y_perm [P][d] (written), all in the
 * act dtype; offsets [E+1] int32 as written by moe_dispatch (P = offsets[E]).
 * bf16: fp32 accumulation on the tensor cores, h_perm and y_perm rounded to
 * bf16.  The second product reads the bf16 h_perm.
 */
moe_status_t moe_grouped_swiglu(const moe_config_t *cfg, const void *x_perm,
                                const int32_t *offsets, const void *W_gate_up,
                                const void *W_down, void *h_perm, void *y_perm,
                                void *stream);

/*
 * Weighted combine [EP-add: the weighted expert output of each token;
 * EP-disp: combined with the routing weights]:
 *   out[t][:] = sum_{j=0}^{k-1} topk_w[t][j] * y_perm[pos[t*k+j]][:]
 * summed in slot order in fp32, then rounded to the act dtype.  With
 * cfg->scale_inputs the weights were applied at dispatch: the rows are summed
 * unweighted and topk_w is not read (may be NULL).
 * y_perm [P][d], pos [P] int32, topk_w [T][k] fp32, out [T][d] (written).
 */
moe_status_t moe_combine(const moe_config_t *cfg, const void *y_perm,
                         const int32_t *pos, const float *topk_w, void *out,
                         void *stream);

/*
 * The whole layer, one stream, no host synchronisation: moe_route,
 * moe_dispatch, moe_grouped_swiglu, moe_combine.
 * When k == E every expert receives every token, so there is nothing to
 * permute [EP]: expert e's segment is rows e*T .. e*T + T-1 in token order,
 * the dispatch only writes counts, offsets, pos and src_token, and the first
 * grouped GEMM reads the rows of x itself instead of x_perm (for fp32 with
 * the weights on the inputs, the scaled rows are copied instead).
 * Otherwise, for bf16 activations with d a multiple of 64 and f <= 3072, the
 * permuted copy of x is not formed either: the dispatch writes counts,
 * offsets, pos and src_token, and the first grouped GEMM gathers row r of
 * the segments from x[src_token[r]] itself (measured faster there than
 * writing and reading x_perm; with the weights on the outputs the results
 * are bit-identical to the copying path).
 * On both paths, weights on the inputs (scale_inputs != 0, bf16) are
 * applied by the first grouped GEMM: row r's gate and up products are
 * multiplied by its pair's weight in fp32 before the SwiGLU, (w x) W =
 * w (x W), where the copying path rounds w x to bf16 first.
 * x [T][d], Wr [E][d] fp32, logit_bias [E] fp32 or NULL,
 * W_gate_up [E][d][2f], W_down [E][f][d], out [T][d] (written).
 * ws: at least moe_workspace_size(cfg) bytes, 256-byte aligned; its
 * contents after the call are the intermediates (layout internal).
 */
moe_status_t moe_forward(const moe_config_t *cfg, const void *x, const float *Wr,
                         const float *logit_bias, const void *W_gate_up,
                         const void *W_down, void *out, void *ws, size_t ws_bytes,
                         void *stream);

/*
 * moe_forward with the activations in HOST memory: copies x_host -> x_dev,
 * runs the layer into out_dev, copies out_dev -> out_host, all enqueued on
 * `stream`.  x_host / out_host ([T][d], act dtype) should be pinned for the
 * copies to be asynchronous; the caller synchronises `stream` before reading
 * out_host.  x_dev / out_dev are caller device buffers of the same size.
 */
moe_status_t moe_forward_host(const moe_config_t *cfg, const void *x_host,
                              const float *Wr, const float *logit_bias,
                              const void *W_gate_up, const void *W_down,
                              void *out_host, void *x_dev, void *out_dev,
                              void *ws, size_t ws_bytes, void *stream);

/* ------------------------------ backward pass ------------------------------
 *
 * The gradients of the four steps above and of the whole layer, for a caller
 * that trains it.  Conventions as above, and:
 *   - gradients of activations and expert weights have the act dtype, those
 *     of routing weights, logits, the router weight and bias are fp32; every
 *     sum is fp32 in an order fixed by the sizes, so results repeat bit for
 *     bit; each output is rounded once at its end (see
 *     moe_grouped_swiglu_backward for its one rounded intermediate);
 *   - outputs are written, not added to; an output may not overlap an input
 *     unless the entry says so;
 *   - T == 0 launches no kernel, but weight gradients (sums over no rows) are
 *     cleared: their buffers are set to zero on `stream`;
 *   - a pair dropped by the dispatch (pos == -1) contributes nothing and has
 *     a zero weight gradient.
 */

/*
 * Gradient of moe_combine:
 *   dy_perm[pos[t*k+j]][:] = topk_w[t][j] * dout[t][:]
 *   dtopk_w[t][j]          = <dout[t], y_perm[pos[t*k+j]]>
 * With cfg->scale_inputs the combine sums unweighted: dy_perm's rows are
 * dout's, and y_perm, topk_w and dtopk_w are not used (may be NULL; the
 * weights' gradient then comes from moe_dispatch_backward).
 * dout [T][d], y_perm [P][d], pos [P], topk_w [T][k]; dy_perm [P][d] and
 * dtopk_w [T][k] written.
 */
moe_status_t moe_combine_backward(const moe_config_t *cfg, const void *dout, const void *y_perm,
                                  const int32_t *pos, const float *topk_w, void *dy_perm,
                                  float *dtopk_w, void *stream);

/*
 * Gradient of moe_dispatch's rows:
 *   dx[t][:] = sum_j dx_perm[pos[t*k+j]][:]
 * summed in slot order.  With cfg->scale_inputs
 *   dx[t][:]      = sum_j topk_w[t][j] * dx_perm[pos[t*k+j]][:]
 *   dtopk_w[t][j] = <x[t], dx_perm[pos[t*k+j]]>
 * else topk_w, x and dtopk_w are not used (may be NULL).
 * dx_perm [P][d], pos [P], topk_w [T][k], x [T][d]; dx [T][d] and dtopk_w
 * [T][k] written.
 */
moe_status_t moe_dispatch_backward(const moe_config_t *cfg, const void *dx_perm,
                                   const int32_t *pos, const float *topk_w, const void *x,
                                   void *dx, float *dtopk_w, void *stream);

/* Bytes of workspace moe_grouped_swiglu_backward needs for `cfg`. */
size_t moe_grouped_swiglu_backward_workspace_size(const moe_config_t *cfg);

/*
 * Gradient of moe_grouped_swiglu.  For expert e and row r of its segment,
 * with the gate and up products (g, u) = x_perm[r] @ W_gate_up[e] formed
 * again (the forward pass does not keep them), s = 1 / (1 + exp(-g)) and
 * dh = dy_perm[r] @ W_down[e]^T:
 *   dgu          = [ dh u s (1 + g (1 - s)),  dh g s ]                   [2f]
 *   dx_perm[r]   = dgu @ W_gate_up[e]^T
 *   dW_gate_up[e] = sum over the segment's rows of x_perm[r]^T dgu[r]
 *   dW_down[e]    = sum over the segment's rows of h_perm[r]^T dy_perm[r]
 * An expert without rows has zero weight gradients.
 * x_perm, h_perm, offsets: as the forward pass left them.  bf16: fp32
 * accumulation on the tensor cores; g, u and dh stay fp32, and dgu is rounded
 * to bf16 where it becomes an operand of the last products.
 * x_perm [P][d], offsets [E+1], W_gate_up [E][d][2f], W_down [E][f][d],
 * h_perm [P][f], dy_perm [P][d]; dx_perm [P][d], dW_gate_up [E][d][2f] and
 * dW_down [E][f][d] written (rows of dx_perm past offsets[E] are not).
 * ws: at least moe_grouped_swiglu_backward_workspace_size(cfg) bytes, 256-byte
 * aligned.
 */
moe_status_t moe_grouped_swiglu_backward(const moe_config_t *cfg, const void *x_perm,
                                         const int32_t *offsets, const void *W_gate_up,
                                         const void *W_down, const void *h_perm,
                                         const void *dy_perm, void *dx_perm, void *dW_gate_up,
                                         void *dW_down, void *ws, size_t ws_bytes, void *stream);

/* Bytes of workspace moe_route_backward needs for `cfg`. */
size_t moe_route_backward_workspace_size(const moe_config_t *cfg);

/*
 * Gradient of moe_route.  With S = sum_j topk_w[t][j] dtopk_w[t][j]:
 *   renormalize: the weights are a softmax over the chosen logits alone:
 *     dlogits[t][topk_idx[t][j]] = topk_w[t][j] (dtopk_w[t][j] - S), 0 elsewhere;
 *   else, with p = softmax over all E logits of row t and g[e] = dtopk_w[t][j]
 *     where e = topk_idx[t][j], 0 elsewhere:
 *     dlogits[t][e] = p[e] (g[e] - S);
 *   dWr         = dlogits^T @ x,   dlogit_bias = column sums of dlogits
 *   dx          = dx_in + dlogits @ Wr     (dx_in NULL: no first term)
 * The selection itself has no gradient.  logits (read only without
 * renormalize; NULL allowed with it), topk_idx and topk_w: as moe_route wrote
 * them.  An expert id outside [0, E) sets MOE_ERR_BAD_ROUTING in the device
 * error word and that slot contributes nothing.
 * x [T][d] act dtype, Wr [E][d], logits [T][E], topk_idx, topk_w, dtopk_w
 * [T][k], dx_in [T][d] act dtype or NULL (may be dx itself); dlogits [T][E],
 * dWr [E][d], dlogit_bias [E] (or NULL), dx [T][d] written.
 * ws: at least moe_route_backward_workspace_size(cfg) bytes, 256-byte aligned.
 */
moe_status_t moe_route_backward(const moe_config_t *cfg, const void *x, const float *Wr,
                                const float *logits, const int32_t *topk_idx,
                                const float *topk_w, const float *dtopk_w, const void *dx_in,
                                float *dlogits, float *dWr, float *dlogit_bias, void *dx, void *ws,
                                size_t ws_bytes, void *stream);

/* Bytes of workspace moe_backward needs for `cfg` (0 when T == 0). */
size_t moe_backward_workspace_size(const moe_config_t *cfg);

/*
 * The whole layer's gradient, one stream, no host synchronisation: from dout
 * = dLoss/dout to the gradients of x and of every parameter, by the four
 * entries above.  fwd_ws is the workspace of the moe_forward call whose
 * gradient is taken, with the same cfg, x and weights, unchanged since (its
 * routing, h_perm and y_perm are read; where moe_forward formed no permuted
 * copy of x, the rows are copied here into ws).
 * x, dout, dx [T][d]; Wr, dWr [E][d]; W_gate_up, dW_gate_up [E][d][2f];
 * W_down, dW_down [E][f][d]; dlogit_bias [E] or NULL.
 * ws: at least moe_backward_workspace_size(cfg) bytes, 256-byte aligned, not
 * fwd_ws.
 */
moe_status_t moe_backward(const moe_config_t *cfg, const void *x, const float *Wr,
                          const void *W_gate_up, const void *W_down, const void *fwd_ws,
                          size_t fwd_ws_bytes, const void *dout, void *dx, float *dWr,
                          float *dlogit_bias, void *dW_gate_up, void *dW_down, void *ws,
                          size_t ws_bytes, void *stream);

/* One gradient tensor of moe_clip_grad_norm. */
typedef struct {
    const void *grad;  /* numel elements, aligned to its element size */
    void *out;         /* clipped copy, same type; may be grad itself; NULL: norm only */
    int64_t numel;     /* >= 0 */
    int32_t dtype;     /* moe_dtype_t */
    int32_t reserved;  /* 0 */
} moe_grad_t;

/* Bytes of workspace moe_clip_grad_norm needs, for any list. */
size_t moe_clip_grad_norm_workspace_size(void);

/*
 * The global 2-norm of n gradient tensors, and the tensors scaled so that it
 * is at most max_norm (no counterpart on the pages: the step between a
 * layer's gradients and its optimizer):
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   out  = g * min(1, max_norm / (norm + 1e-6)),  rounded once
 * A thread sums 64 of 16384 elements' squares in fp32, scaled by a power of two
 * where they would leave its range; beyond that sums are fp64, in a fixed
 * order.  So the norm is within a few fp32 roundings for any finite
 * gradients, as long as it is a finite float itself.  It never leaves the device.
 * A NaN or infinite gradient gives a NaN or infinite norm, finite gradients
 * whose norm is past 3.4e38 an infinite one, and the scale follows the formula
 * (an infinite norm scales finite gradients to 0): a caller that wants to skip
 * such a step reads `norm`.
 * grads: HOST array of n >= 0 entries, read before the call returns; `norm`:
 * one float on the device, written (0 for no elements).  max_norm >= 0.
 * ws: at least moe_clip_grad_norm_workspace_size() bytes, 256-byte aligned.
 * Tensors may overlap only where out == grad.
 */
moe_status_t moe_clip_grad_norm(const moe_grad_t *grads, int64_t n, float max_norm, float *norm,
                                void *ws, size_t ws_bytes, void *stream);

/* ------------------------- routing by other scores -------------------------
 *
 * The router of a layer that is balanced by a bias instead of a loss, and whose
 * experts come in groups (no counterpart on the pages).  With L a token's
 * logits (including logit_bias) and b the balance bias:
 *   s_e = exp(L_e) / sum_i exp(L_i)     (MOE_SCORE_SOFTMAX)
 *       = 1 / (1 + exp(-L_e))           (MOE_SCORE_SIGMOID)
 *   q_e = s_e + b_e
 *   the E experts form `groups` groups of E / groups consecutive ones; the
 *     topk_groups groups with the largest u_g stay, u_g = the largest q of the
 *     group (MOE_GROUP_MAX) or the sum of its two largest (MOE_GROUP_TOP2; a
 *     group of one expert: its q); equal u go to the lower group;
 *   topk_idx[t][j]: the j-th largest q among the experts that stay; equal q go
 *     to the lower id;
 *   topk_w[t][j] = weight_scale * s_e / (cfg->renormalize ? sum of s over the
 *     chosen k : 1),  e = topk_idx[t][j].
 * The bias moves the choice and not the weights, and has no gradient:
 * moe_update_balance_bias trains it.  Without a bias the experts are ordered by
 * their logits (the order of s as real numbers).  With one, and for sums of two, q
 * and u are compared as 64-bit values, however near they are in fp32.
 * Edges: a NaN q or u ranks below every number (a NaN logit makes all of a
 * softmax row NaN, and all of its weights).  A logit of -inf has a score of 0, and still a q of b_e: to
 * exclude an expert from every choice give it a bias of -inf.  A row of -inf alone
 * has scores of 0.  Where all chosen scores are 0 their renormalised weights are
 * 0; scores that fp32 cannot hold keep their shares.  A logit of +inf is not
 * supported with softmax scores.
 * Limits: 1 <= groups <= 32, E a multiple of groups, 1 <= topk_groups <=
 * groups, k <= topk_groups * E / groups, 2^-100 <= weight_scale <= 2^100.
 */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_score_t;

typedef struct {
    int32_t score;       /* moe_score_t */
    int32_t groups;      /* 1: no groups */
    int32_t topk_groups;
    int32_t group_score; /* moe_group_score_t */
    float weight_scale;  /* factor on the routing weights */
    int32_t reserved;    /* 0 */
} moe_router_t;

/*
 * moe_route with the scores of `router`.  balance_bias [E] fp32 or NULL; the
 * other arguments, and the workspace, are moe_route's.
 */
moe_status_t moe_route_scored(const moe_config_t *cfg, const moe_router_t *router, const void *x,
                              const float *Wr, const float *logit_bias, const float *balance_bias,
                              float *logits, int32_t *topk_idx, float *topk_w, void *ws,
                              size_t ws_bytes, void *stream);

/* The same selection and weights on a GIVEN fp32 logit buffer [T][E] (read
 * only); cfg's d, f and act_dtype are checked but not used. */
moe_status_t moe_route_scored_from_logits(const moe_config_t *cfg, const moe_router_t *router,
                                          const float *logits, const float *balance_bias,
                                          int32_t *topk_idx, float *topk_w, void *stream);

/*
 * Gradient of the weights above with respect to the logits, with
 * S = sum_j topk_w[t][j] dtopk_w[t][j], c = weight_scale, w and d for
 * topk_w[t][j] and dtopk_w[t][j], e = topk_idx[t][j]:
 *   softmax, renormalize: dlogits[t][e] = w (d - S / c), 0 elsewhere;
 *   softmax:              dlogits[t][i] = s_i (c g_i - S), g_e = d, 0 elsewhere;
 *   sigmoid, renormalize: dlogits[t][e] = w (d - S / c) (1 - s_e), 0 elsewhere;
 *   sigmoid:              dlogits[t][e] = w d (1 - s_e), 0 elsewhere.
 * The choice itself has no gradient, and groups play no part.  logits, topk_idx
 * (a token's ids distinct) and topk_w as the route wrote them (logits may be
 * NULL for softmax with renormalize).  An id outside [0, E) sets
 * MOE_ERR_BAD_ROUTING in the device error word and contributes nothing.
 * dlogits [T][E] written.
 */
moe_status_t moe_route_scored_from_logits_backward(const moe_config_t *cfg,
                                                   const moe_router_t *router,
                                                   const float *logits, const int32_t *topk_idx,
                                                   const float *topk_w, const float *dtopk_w,
                                                   float *dlogits, void *stream);

/* Bytes of workspace moe_route_scored_backward needs. */
size_t moe_route_scored_backward_workspace_size(const moe_config_t *cfg,
                                                const moe_router_t *router);

/* moe_route_backward with these dlogits: the same arguments, sums and edges. */
moe_status_t moe_route_scored_backward(const moe_config_t *cfg, const moe_router_t *router,
                                       const void *x, const float *Wr, const float *logits,
                                       const int32_t *topk_idx, const float *topk_w,
                                       const float *dtopk_w, const void *dx_in, float *dlogits,
                                       float *dWr, float *dlogit_bias, void *dx, void *ws,
                                       size_t ws_bytes, void *stream);

/*
 * The whole layer and its gradient with such a router: moe_forward and
 * moe_backward but for the routing (the same workspace layout and size for the
 * forward pass; one launch more than moe_forward_kernel_launches says where
 * E <= 32 and the logits are formed on the CUDA cores).
 */
moe_status_t moe_forward_scored(const moe_config_t *cfg, const moe_router_t *router, const void *x,
                                const float *Wr, const float *logit_bias,
                                const float *balance_bias, const void *W_gate_up,
                                const void *W_down, void *out, void *ws, size_t ws_bytes,
                                void *stream);

/* Bytes of workspace moe_backward_scored needs (0 when T == 0). */
size_t moe_backward_scored_workspace_size(const moe_config_t *cfg, const moe_router_t *router);

moe_status_t moe_backward_scored(const moe_config_t *cfg, const moe_router_t *router,
                                 const void *x, const float *Wr, const void *W_gate_up,
                                 const void *W_down, const void *fwd_ws, size_t fwd_ws_bytes,
                                 const void *dout, void *dx, float *dWr, float *dlogit_bias,
                                 void *dW_gate_up, void *dW_down, void *ws, size_t ws_bytes,
                                 void *stream);

/*
 * One step of the balance bias of `layers` layers: with n the pairs that each
 * expert of a layer received (moe_dispatch's counts, or their sums over several
 * batches),
 *   balance_bias[l][e] += rate * sign(sum_i n[l][i] - E n[l][e])
 *   imbalance[l]        = E max_e n[l][e] / sum_e n[l][e]   (0 without pairs)
 * An expert whose load is the mean keeps its bias; counts are compared as
 * whole numbers.
 * counts [layers][E] int32 >= 0, balance_bias [layers][E] fp32 (updated),
 * imbalance [layers] fp32 (written) or NULL: element-aligned pointers.
 * layers >= 0 (0 launches nothing), 1 <= E <= 1024, rate finite.
 */
moe_status_t moe_update_balance_bias(const int32_t *counts, int64_t layers, int32_t E, float rate,
                                     float *balance_bias, float *imbalance, void *stream);

/* --------------------------------- AdamW -----------------------------------
 *
 * One AdamW step over many parameter tensors at once, in place (no counterpart
 * on the pages: the step after moe_clip_grad_norm).  With g a gradient, t the
 * step's number, counted from 1:
 *   g' = g * min(1, max_norm / (norm + 1e-6))      (norm given; else g' = g)
 *   m  = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *   p  = p (1 - lr weight_decay)
 *        - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32, from the new m and v before they are rounded to their storage.  With
 * moe_clip_grad_norm's `norm` (its out = NULL) the clipped gradients are never
 * written.
 *
 * Storage.  A parameter is fp32 or bf16, and so is its gradient.  A bf16
 * parameter may have an fp32 master copy: then the master is stepped and the
 * parameter is its rounding.  Without one, `stochastic` rounds the new bf16
 * value to one of its two neighbours, with the probabilities that keep it right
 * on average (rounding to the nearest loses every update below 2^-9 of the
 * value); 0 rounds to the nearest.
 * States are fp32 (m and v), or 8 bits (MOE_E4M3): m and r = sqrt(v) in blocks
 * of 256 consecutive elements, each an e4m3 value times the block's scale, a
 * power of two 2^(e - 7) with 2^e <= the block's largest magnitude < 2^(e + 1)
 * (at least 2^-126).  They are rounded stochastically: a state's change of a few
 * percent of itself, or less, is far below a step of e4m3, and would be lost
 * whole by rounding to the nearest.  An r above 0 is stored as at least the
 * smallest code, so that no later step divides by eps alone (a v below 2^-126
 * counts as 0, and eps = 0 then divides by 0).  (Zeros in all bytes and scales are
 * valid initial states of either kind.)
 * An element whose m or v is a NaN or infinite costs the others of its block
 * nothing: the scales are those of the largest finite magnitudes.  A NaN is
 * stored as NaN, an infinite m as the format's largest value, an infinite v as a
 * negative NaN of r, which the next step reads as infinite (so, as with fp32
 * states, a gradient whose square overflows leaves its parameter to the decay).
 *
 * Random numbers: 32 bits of every element, a function of `seed` (a caller takes
 * another each step), the number of its block of 256 elements counted over the
 * whole list, and its place in the block.  So a step repeats bit for bit.
 */
typedef struct {
    void *param;       /* updated */
    const void *grad;
    void *exp_avg;     /* m; updated */
    void *exp_avg_sq;  /* v (fp32 states) or r = sqrt(v) (8-bit states); updated */
    float *exp_avg_scale;     /* 8-bit states: [ceil(numel / 256)], updated; else NULL */
    float *exp_avg_sq_scale;  /* the same */
    float *master;     /* bf16 parameters: fp32 copy, updated, or NULL; fp32: NULL */
    int64_t numel;     /* >= 0 */
    int32_t param_dtype, grad_dtype; /* MOE_F32 or MOE_BF16 */
    int32_t state_dtype;             /* MOE_F32 or MOE_E4M3 */
    float weight_decay;
} moe_adamw_tensor_t;

typedef struct {
    double lr, beta1, beta2, eps;  /* lr >= 0; 0 <= beta < 1; eps 0 or >= 2^-126 */
    int64_t step;                  /* >= 1 */
    uint64_t seed;
    float max_norm;                /* >= 0; read when `norm` is given */
    int32_t stochastic;            /* bf16 parameters without a master copy */
    int32_t skip_nonfinite;        /* 1: a NaN or infinite `norm` leaves everything as it was */
    int32_t reserved;              /* 0 */
} moe_adamw_hyper_t;

/* What changes from step to step, for a call that is captured in a graph. */
typedef struct {
    float lr;
    float step_size;    /* lr / (1 - beta1^t) */
    float inv_sqrt_bc2; /* 1 / sqrt(1 - beta2^t) */
    uint32_t seed_lo, seed_hi;
    uint32_t reserved[3];
} moe_adamw_scalars_t;

/* Fills *out from hyper's lr, betas, step and seed (on the host). */
moe_status_t moe_adamw_scalars(const moe_adamw_hyper_t *hyper, moe_adamw_scalars_t *out);

/*
 * tensors: HOST array of n >= 0 entries, read before the call returns; pointers
 * element-aligned (the fastest path wants 16 bytes), tensors that do not
 * overlap.  norm: one float on the device or NULL.  scalars: NULL, or 16-byte
 * aligned device memory that the kernels read lr, step and seed from instead of
 * `hyper`: a captured graph is replayed after a copy of new moe_adamw_scalars.
 * No workspace.
 */
moe_status_t moe_adamw_step(const moe_adamw_tensor_t *tensors, int64_t n,
                            const moe_adamw_hyper_t *hyper, const float *norm,
                            const moe_adamw_scalars_t *scalars, void *stream);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word.  Returns MOE_OK, MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_BAD_ROUTING, or
 * MOE_ERR_CUDA if the synchronisation itself failed.
 */
moe_status_t moe_last_device_error(void *stream);

/*
 * Limit, in nanoseconds, on every bounded device-side wait of later launches
 * from this process (default 2e9 = 2 s; 0 restores the default).  A wait
 * that runs out records MOE_ERR_DEVICE_TIMEOUT and the kernel returns.
 * Limits below 10 ms are raised to 10 ms (unless the test hook
 * moe_debug_inject_wait_timeout is on): a CTA pair that gave up within one
 * pipeline stage could otherwise leave a copy in flight that no barrier of
 * its pair expects.
 */
void moe_set_wait_limit_ns(uint64_t ns);

/* The wait limit later launches will use, after the 10 ms floor. */
uint64_t moe_wait_limit_ns(void);

/*
 * Test hook for the failure path (no counterpart on the pages).  While
 * enabled (non-zero), every later tensor-core grouped GEMM launch first waits
 * on a barrier that nothing signals, so that wait runs out after the wait
 * limit: the kernel records MOE_ERR_DEVICE_TIMEOUT, drains its in-flight
 * copies, frees its tensor memory and returns without computing.  The
 * outputs of such a call are undefined.  Off by default.
 */
void moe_debug_inject_wait_timeout(int enable);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
