// kernels.h -- host-side launchers of the libmoe kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "moe.h"

namespace moe {

struct Shape {
    int64_t T;
    int d, E, k, f;
    bool bf16;    // activation dtype: bf16 (else fp32)
    bool renorm;  // renormalise the chosen k weights
    bool scale_inputs;  // routing weights scale expert inputs (dispatch), not outputs
    int64_t P() const { return T * (int64_t)k; }
};

// Router: logits[T][E] = x @ Wr^T (+ bias), fp32 accumulation.  When
// router_selects_in_logits(s) and idx/w are given, the same launch also
// writes the top-k selection and weights (no separate top-k launch).
// zero_word (optional, for the selecting launches here and below): a word
// the launch sets to 0, so a later kernel in the stream finds it cleared
// (the dispatch's ticket counter).
cudaError_t launch_router_logits(const Shape &s, const void *x, const float *Wr,
                                 const float *bias, float *logits, cudaStream_t st,
                                 int32_t *idx = nullptr, float *w = nullptr,
                                 unsigned *zero_word = nullptr);
bool router_selects_in_logits(const Shape &s);
// Top-k selection and softmax weights on a given fp32 logit buffer.
cudaError_t launch_topk(const Shape &s, const float *logits, int32_t *idx, float *w,
                        cudaStream_t st, unsigned *zero_word = nullptr);
// Top-k on logits formed as sum of `splits` partial buffers [splits][T][E]
// (added in split order) plus bias; the logits are written to `logits`.
cudaError_t launch_topk_partials(const Shape &s, const float *partial, int splits,
                                 const float *bias, float *logits, int32_t *idx, float *w,
                                 cudaStream_t st, unsigned *zero_word = nullptr);

// Router logits on the tensor cores (bf16 x, fp32 Wr split into 3 bf16 terms).
struct RouterTcPlan {
    int ctas;          // 2: CTA pairs on 256-token tiles; 1: single CTAs on 128-token tiles
    int ks_total;      // pipeline stages of a row tile: d / 64 (three W' tiles each) or 3d / 64
    int ks_per_split;  // stages per CTA
    int splits;        // K splits (blockIdx.y)
};
bool router_tc_eligible(const Shape &s);
RouterTcPlan router_tc_plan(const Shape &s);
size_t router_tc_scratch_bytes(const Shape &s);  // split weight + partial logits
cudaError_t launch_router_logits_tc(const Shape &s, const void *x, const float *Wr, void *scratch,
                                    float **partial_out, int *splits_out, const DevStatus &ds,
                                    cudaStream_t st);

// Dispatch: chunking of the P pairs over the rank kernel's blocks.
struct DispatchGrid {
    int chunk;  // pairs per block (a multiple of 256)
    int blocks;  // number of blocks (>= 1 when P > 0)
};
DispatchGrid dispatch_grid(int64_t P, int E);
// A dispatch that copies unscaled rows runs as one launch (no count matrix,
// no ticket) when E <= 16, P <= 16384 and a row is k KB to 16 KB.
bool dispatch_fits_one_launch(const Shape &s);
size_t dispatch_scratch_bytes(const Shape &s);  // count matrix [E][chunks] + ticket
// The ticket counter inside the dispatch scratch `hist` (must be 0 when the
// dispatch's first launch starts; the dispatch leaves it 0).
unsigned *dispatch_ticket(const Shape &s, int32_t *hist);
// x_perm == nullptr: counts, offsets, pos and src_token only (no row gather).
// scale != nullptr: each gathered row is multiplied by its pair's weight;
// without x_perm, row_scale[row] = scale[pair] instead (if row_scale).
// in_forward: the dispatch runs inside moe_forward, after the route, whose
// last launch cleared the ticket; its launches overlap the route's by
// programmatic dependent launch.  Otherwise (a standalone call) the ticket is
// cleared here with a 4-byte cudaMemsetAsync, after which the first launch
// starts only once all earlier work in the stream is done.
cudaError_t launch_dispatch(const Shape &s, const int32_t *idx, const void *x, int32_t *counts,
                            int32_t *offsets, int32_t *pos, int32_t *src_token, void *x_perm,
                            int32_t *hist, const DevStatus &ds, cudaStream_t st,
                            const float *scale = nullptr, bool in_forward = false,
                            float *row_scale = nullptr);

// Grouped SwiGLU experts.  bf16: tcgen05 tensor-core path; fp32: SIMT path.
// Kernel launches of one launch_grouped_swiglu_tc call (2, or 4 when the
// experts are split between CTA-pair and single-CTA tiles).
int grouped_swiglu_tc_launches(const Shape &s);
// Whether launch_grouped_swiglu_tc can gather G1's rows (src_token) for s,
// and whether doing so is measured faster than reading a permuted copy.
bool grouped_swiglu_tc_gathers(const Shape &s);
bool grouped_swiglu_tc_gather_pays(const Shape &s);
// a_local: x_perm is the T token rows x, and row r of expert e's segment
// reads row r - offsets[e] (every expert receives every token, in order).
// src_token (not null): x_perm is the T token rows x, and G1 gathers row r
// of the segments from row src_token[r] (d a multiple of 64, no a_local).
// row_scale (not null): G1 multiplies row r's gate and up accumulators by
// row_scale[r] (the routing weight on the expert's input, applied after the
// product instead of to the rows).
cudaError_t launch_grouped_swiglu_tc(const Shape &s, const void *x_perm, const int32_t *offsets,
                                     const void *Wgu, const void *Wd, void *h_perm, void *y_perm,
                                     const DevStatus &ds, cudaStream_t st, bool a_local = false,
                                     const int32_t *src_token = nullptr,
                                     const float *row_scale = nullptr);
cudaError_t launch_grouped_swiglu_f32(const Shape &s, const float *x_perm, const int32_t *offsets,
                                      const float *Wgu, const float *Wd, float *h_perm,
                                      float *y_perm, cudaStream_t st, bool a_local = false);

// Dispatch when every token picks every expert (k == E): counts[e] = T,
// offsets[e] = e*T, pos[t*E+j] = idx[t][j]*T + t, src_token[e*T + t] = t.
// No rows are copied (the experts read x with a_local).  One launch.
// w, row_scale (both or neither): row_scale[idx[t][j]*T + t] = w[t][j].
cudaError_t launch_dispatch_all_experts(const Shape &s, const int32_t *idx, int32_t *counts,
                                        int32_t *offsets, int32_t *pos, int32_t *src_token,
                                        const DevStatus &ds, cudaStream_t st,
                                        const float *w = nullptr, float *row_scale = nullptr);

// Weighted combine of the expert rows back into token order (w == nullptr:
// unweighted sum).
cudaError_t launch_combine(const Shape &s, const void *y_perm, const int32_t *pos, const float *w,
                           void *out, cudaStream_t st);

// ------------------------------ backward pass ------------------------------
// dst[pos[q]] = w[q] * src[q / k] for every pair q (w == nullptr: unscaled),
// and with dw (not null) dw[q] = <src[q / k], y_perm[pos[q]]>: the gradient of
// the combine (src = dout), or the permuted copy of x (dw == nullptr).
cudaError_t launch_scatter_rows(const Shape &s, const void *src, const void *y_perm,
                                const int32_t *pos, const float *w, void *dst, float *dw,
                                cudaStream_t st);
// dx[t] = sum_j dx_perm[pos[t*k+j]] (w == nullptr), or weighted by w with
// dw[t*k+j] = <x[t], dx_perm[pos[t*k+j]]>.
cudaError_t launch_dispatch_backward(const Shape &s, const void *dx_perm, const int32_t *pos,
                                     const float *w, const void *x, void *dx, float *dw,
                                     cudaStream_t st);

// fp32: out[t] = add[t] (if given; may be out) + sum_j w[t*k+j] rows[idx[t*k+j]].
cudaError_t launch_gather_sum_f32(const Shape &s, const float *rows, const int32_t *idx,
                                  const float *w, const float *add, float *out, cudaStream_t st);

// Operands of the grouped SwiGLU's gradient (see moe_grouped_swiglu_backward).
struct ExpertsBwd {
    const void *x_perm;
    const int32_t *offsets;
    const void *Wgu, *Wd, *h_perm, *dy_perm;
    void *dx_perm, *dWgu, *dWd, *ws;
};
cudaError_t launch_experts_backward_f32(const Shape &s, const ExpertsBwd &a, cudaStream_t st);
// bf16: tcgen05 tensor cores.
size_t experts_backward_tc_scratch_bytes(const Shape &s);
cudaError_t launch_experts_backward_tc(const Shape &s, const ExpertsBwd &a, const DevStatus &ds,
                                       cudaStream_t st);

// How the routing weights' gradient becomes the logits' (route_scored.cu has the
// formulas): the chosen logits alone, or (dense: softmax scores that are not
// renormalised) every logit's.
struct ScoreGrad {
    int sigmoid, dense;
    float scale;  // the factor on the weights
    float share;  // of the weighted sum S that a chosen logit loses: 1/scale if renormalised, or 0
    // dl of a chosen logit L (read for sigmoid scores only), with weight w and dLoss/dw d
    __device__ __forceinline__ float chosen(float w, float d, float S, float L) const {
        const float t = w * (share != 0.f ? d - S * share : d);
        return sigmoid ? t * (1.f / (1.f + expf(L))) : t;
    }
};

// Operands of the router's gradient (see moe_route_backward).
struct RouteBwd {
    const void *x;
    const float *Wr, *logits;
    const int32_t *idx;
    const float *w, *dw;
    const void *dx_in;
    float *dlogits, *dWr, *dbias;
    void *dx, *ws;
    ScoreGrad f;
};
size_t route_backward_scratch_bytes(const Shape &s);
// The router gradient's products on the tensor cores (bf16 x), over operands
// that route_bwd.cu split into bf16 terms: dx = dx_in + dl_x W with dl_x
// [T][K] and W [K][d], and part[s] [K][d] = the sum over split s's tokens of
// dl_w[t]^T x[t], dl_w [T][K]; rows of dl_x and dl_w are ld elements apart.
struct RouteProducts {
    const void *x, *dl_x, *dl_w, *W, *dx_in;
    int K, n_splits;
    int64_t ld;
    const int32_t *all, *splits;  // {0, T} and the n_splits + 1 split boundaries
    void *dx;
    float *part;
};
int route_backward_splits(int64_t T, int d, int cols);
cudaError_t launch_route_backward_tc(const Shape &s, const RouteProducts &r, const DevStatus &ds,
                                     cudaStream_t st);
cudaError_t launch_route_backward(const Shape &s, const RouteBwd &a, const DevStatus &ds,
                                  cudaStream_t st);

// ------------------------- scored routing (route_scored.cu) -------------------------
struct Router {
    bool sigmoid, top2;
    int G, Gk;
    float scale;
};
// Selection and weights by r's scores, on given logits (nparts == 0) or on the
// sum of nparts partial buffers plus logit_bias, which is written to `logits`.
// bias: the balance bias, or null.  zero_word: as for launch_topk.
cudaError_t launch_select(const Shape &s, const Router &r, float *logits, const float *partial,
                          int nparts, const float *logit_bias, const float *bias, int32_t *idx,
                          float *w, cudaStream_t st, unsigned *zero_word = nullptr);
cudaError_t launch_logits_grad(const Shape &s, const ScoreGrad &f, const float *logits,
                               const int32_t *idx, const float *w, const float *dw, float *dlogits,
                               const DevStatus &ds, cudaStream_t st);
cudaError_t launch_balance(const int32_t *counts, int64_t layers, int E, float rate, float *bias,
                           float *imbalance, cudaStream_t st);

// ------------------------------ AdamW (adamw.cu) ------------------------------
int64_t adamw_chunk();  // elements per unit of work (the limit is 2^30 units)
cudaError_t launch_adamw(const moe_adamw_tensor_t *t, int64_t n, const moe_adamw_scalars_t &sc,
                         const moe_adamw_scalars_t *dev, const moe_adamw_hyper_t &h,
                         const float *norm, cudaStream_t st);

// Global norm of n gradient tensors and their clipped copies.
size_t clip_scratch_bytes();
int64_t clip_chunk();  // elements per unit of work (the library's limit is 2^31 units)
cudaError_t launch_clip(const moe_grad_t *g, int64_t n, float max_norm, float *norm, void *ws,
                        cudaStream_t st);

// Streaming multiprocessors of the current device (queried once per device).
// Without a usable device (sizing a workspace on a host with no GPU) it is
// 152, a GB300's count; a launch always plans with the real device's count,
// and a workspace sized for fewer SMs than the device has is then reported
// as too small (MOE_ERR_WORKSPACE), never overrun.
int device_sm_count();

// Last detailed message set by a launcher (thread-local; empty if none).
void set_error_message(const char *fmt, ...);
const char *error_message();

}  // namespace moe
