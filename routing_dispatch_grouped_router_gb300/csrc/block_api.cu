// C ABI of the operators around the layer (declared in include/mok.h): the
// residual addition with RMS norm, the router's auxiliary losses, the dense
// product, dropout, the norms after and before a block and the products grouped
// by expert.  Argument checks and the order of kernels; nothing is enqueued
// before every argument has been checked.
#include <cuda_runtime.h>

#include "mok_internal.h"

using namespace mok;

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool elem_ok(int32_t e) { return e == MOK_ELEM_BF16 || e == MOK_ELEM_F32; }
size_t elem_size(int32_t e) { return e == MOK_ELEM_F32 ? 4 : 2; }
// (a refused launch also stays as the thread's last error, which the next call of
// another library would take for its own)
mok_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOK_OK;
  cudaGetLastError();
  return MOK_ERR_CUDA;
}

// A row stride: 0 stands for `cols`; less than a row is wrong.
bool stride(int64_t* ld, int64_t cols) {
  if (*ld == 0) *ld = cols;
  return *ld >= cols && *ld <= (1LL << 40);
}

mok_status norm_desc(const mok_rmsnorm_desc* desc, mok_rmsnorm_desc* D) {
  if (!desc) return MOK_ERR_INVALID_ARG;
  *D = *desc;
  if (D->rows < 0 || D->d <= 0 || !(D->eps >= 0.f)) return MOK_ERR_INVALID_ARG;
  if (D->rows >= (1LL << 31) || D->d > 16384) return MOK_ERR_UNSUPPORTED;
  if (!elem_ok(D->x_elem) || !elem_ok(D->s_elem) || !elem_ok(D->weight_elem))
    return MOK_ERR_UNSUPPORTED;
  if (D->reserved != 0) return MOK_ERR_UNSUPPORTED;
  if (!stride(&D->ld_x, D->d) || !stride(&D->ld_res, D->d) || !stride(&D->ld_s, D->d) ||
      !stride(&D->ld_y, D->d))
    return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}

mok_status balance_desc(const mok_balance_desc* desc, mok_balance_desc* D) {
  if (!desc) return MOK_ERR_INVALID_ARG;
  *D = *desc;
  if (D->T < 0 || D->E <= 0 || D->k <= 0) return MOK_ERR_INVALID_ARG;
  if (D->E > kMaxExperts || D->k > kMaxTopK || D->k > D->E) return MOK_ERR_UNSUPPORTED;
  if (D->T >= (1LL << 30) / D->k) return MOK_ERR_UNSUPPORTED;
  if (!stride(&D->ld_logits, D->E)) return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}

mok_status linear_desc(const mok_linear_desc* desc, mok_linear_desc* D) {
  if (!desc) return MOK_ERR_INVALID_ARG;
  *D = *desc;
  if (D->M < 0 || D->N <= 0 || D->K <= 0) return MOK_ERR_INVALID_ARG;
  if (D->M > (1 << 24) || D->N > (1 << 24) || D->K > (1 << 24) || D->K % 8)
    return MOK_ERR_UNSUPPORTED;
  if (D->act < MOK_ACT_NONE || D->act > MOK_ACT_GELU) return MOK_ERR_UNSUPPORTED;
  if (!elem_ok(D->y_elem) || !elem_ok(D->dx_elem)) return MOK_ERR_UNSUPPORTED;
  if (D->accumulate & ~(MOK_ADD_DX | MOK_ADD_DW)) return MOK_ERR_UNSUPPORTED;
  if (!stride(&D->ld_x, D->K)) return MOK_ERR_INVALID_ARG;
  if (D->ld_x % 8) return MOK_ERR_UNSUPPORTED;
  return MOK_OK;
}

mok_status dropout_desc(const mok_dropout_desc* desc, mok_dropout_desc* D) {
  if (!desc) return MOK_ERR_INVALID_ARG;
  *D = *desc;
  if (D->rows < 0 || D->d <= 0 || !(D->p >= 0.0 && D->p <= 1.0)) return MOK_ERR_INVALID_ARG;
  if (D->rows >= (1LL << 31) || D->d >= (1LL << 31)) return MOK_ERR_UNSUPPORTED;
  if (!elem_ok(D->x_elem) || !elem_ok(D->y_elem) || D->reserved != 0) return MOK_ERR_UNSUPPORTED;
  if (!stride(&D->ld_x, D->d) || !stride(&D->ld_res, D->d) || !stride(&D->ld_y, D->d))
    return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}

mok_status dropout(const mok_dropout_desc* desc, const void* x, const void* residual,
                   const int64_t* rng, void* y, void* stream) {
  mok_dropout_desc D;
  mok_status st = dropout_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!rng || (D.rows > 0 && (!x || !y))) return MOK_ERR_INVALID_ARG;
  const size_t ye = elem_size(D.y_elem);
  if (!aligned(x, elem_size(D.x_elem)) || !aligned(residual, ye) || !aligned(y, ye) ||
      !aligned(rng, 8))
    return MOK_ERR_INVALID_ARG;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_dropout(D, x, residual, rng, y, static_cast<cudaStream_t>(stream)));
}

mok_status post_pre_desc(const mok_post_pre_desc* desc, mok_post_pre_desc* D) {
  if (!desc) return MOK_ERR_INVALID_ARG;
  *D = *desc;
  if (D->rows < 0 || D->d <= 0 || !(D->eps >= 0.f)) return MOK_ERR_INVALID_ARG;
  if (D->rows >= (1LL << 31) || D->d > 16384) return MOK_ERR_UNSUPPORTED;
  if (!elem_ok(D->x_elem) || !elem_ok(D->s_elem) || !elem_ok(D->weight_elem) ||
      !elem_ok(D->gate_elem) || !elem_ok(D->y_elem) || !elem_ok(D->dx_elem))
    return MOK_ERR_UNSUPPORTED;
  if (D->gate < MOK_GATE_NONE || D->gate > MOK_GATE_TOKEN) return MOK_ERR_UNSUPPORTED;
  if (!stride(&D->ld_x, D->d) || !stride(&D->ld_res, D->d) || !stride(&D->ld_s, D->d) ||
      !stride(&D->ld_y, D->d) || !stride(&D->ld_dx, D->d) || !stride(&D->ld_dr, D->d))
    return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}

// Whether there is a gate where the descriptor has one.  Without rows a token's gate is
// empty and may be NULL; a channel's is [d], and the sums read it.
bool gate_fits(const mok_post_pre_desc& D, const void* gate) {
  if (D.rows == 0) return gate || D.gate != MOK_GATE_CHANNEL;
  return (gate != nullptr) == (D.gate != MOK_GATE_NONE);
}

mok_status grouped_desc(const mok_grouped_desc* desc, mok_grouped_desc* D) {
  if (!desc) return MOK_ERR_INVALID_ARG;
  *D = *desc;
  if (D->rows < 0 || D->N <= 0 || D->K <= 0 || D->E <= 0) return MOK_ERR_INVALID_ARG;
  if (D->rows > (1 << 24) || D->N > (1 << 20) || D->K > (1 << 20) || D->N % 8 || D->K % 8 ||
      D->E > kMaxExperts)
    return MOK_ERR_UNSUPPORTED;
  if (!elem_ok(D->y_elem) || !elem_ok(D->dx_elem)) return MOK_ERR_UNSUPPORTED;
  if (D->accumulate & ~MOK_ADD_DW) return MOK_ERR_UNSUPPORTED;
  if (!stride(&D->ld_x, D->K) || !stride(&D->ld_y, D->N) || !stride(&D->ld_dx, D->K))
    return MOK_ERR_INVALID_ARG;
  // (the TMA's strides end below 2^40 bytes)
  if (D->ld_x % 8 || D->ld_y % 8 || D->ld_dx % 8 || D->ld_x >= (1LL << 37) ||
      D->ld_y >= (1LL << 37) || D->ld_dx >= (1LL << 37))
    return MOK_ERR_UNSUPPORTED;
  return MOK_OK;
}

}  // namespace

extern "C" {

mok_status mok_add_rmsnorm_forward(const mok_rmsnorm_desc* desc, const void* x,
                                   const void* residual, const void* weight, void* s, void* y,
                                   void* values, uint8_t* codes, uint8_t* scales, void* stream) {
  mok_rmsnorm_desc D;
  mok_status st = norm_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!weight || (codes == nullptr) != (scales == nullptr)) return MOK_ERR_INVALID_ARG;
  if (D.rows > 0 && (!x || (residual && !s) || (!y && !values && !codes)))
    return MOK_ERR_INVALID_ARG;
  if (!residual && D.x_elem != D.s_elem) return MOK_ERR_UNSUPPORTED;
  if ((values || codes) && D.d % 32) return MOK_ERR_UNSUPPORTED;
  const size_t se = elem_size(D.s_elem);
  if (!aligned(x, elem_size(D.x_elem)) || !aligned(residual, se) || !aligned(s, se) ||
      !aligned(weight, elem_size(D.weight_elem)) || !aligned(y, 2) || !aligned(values, 2))
    return MOK_ERR_INVALID_ARG;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_add_rmsnorm(D, x, residual, weight, s, y, values, codes, scales,
                                        static_cast<cudaStream_t>(stream)));
}

mok_status mok_add_rmsnorm_workspace_size(const mok_rmsnorm_desc* desc, size_t* bytes) {
  mok_rmsnorm_desc D;
  const mok_status st = norm_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!bytes) return MOK_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(norm_bwd_blocks(D)) * static_cast<size_t>(D.d) * 4;
  return MOK_OK;
}

mok_status mok_add_rmsnorm_backward(const mok_rmsnorm_desc* desc, const void* dy, const void* s,
                                    const void* weight, const void* ds, void* dx,
                                    float* dweight, void* workspace, size_t ws_bytes,
                                    int32_t* status, void* stream) {
  mok_rmsnorm_desc D;
  mok_status st = norm_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!weight || (D.rows > 0 && (!dy || !s || !dx))) return MOK_ERR_INVALID_ARG;
  const size_t se = elem_size(D.s_elem);
  if (!aligned(dy, elem_size(D.x_elem)) || !aligned(s, se) || !aligned(ds, se) ||
      !aligned(dx, se) || !aligned(weight, elem_size(D.weight_elem)) || !aligned(dweight, 4) ||
      !aligned(status, 4))
    return MOK_ERR_INVALID_ARG;
  if (dweight && D.rows > 0) {
    if (!workspace || !aligned(workspace, 16)) return MOK_ERR_INVALID_ARG;
    size_t need = 0;
    mok_add_rmsnorm_workspace_size(&D, &need);
    if (ws_bytes < need) return MOK_ERR_WORKSPACE;
  }
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_add_rmsnorm_bwd(D, dy, s, weight, ds, dx, dweight,
                                            static_cast<float*>(workspace), status,
                                            static_cast<cudaStream_t>(stream)));
}

mok_status mok_router_balance_workspace_size(const mok_balance_desc* desc, size_t* bytes) {
  mok_balance_desc D;
  const mok_status st = balance_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!bytes) return MOK_ERR_INVALID_ARG;
  BalanceWs W;
  balance_layout(D, &W);
  *bytes = W.total;
  return MOK_OK;
}

mok_status mok_router_balance_forward(const mok_balance_desc* desc, const float* logits,
                                      const int32_t* topk_idx, const uint8_t* mask, float* loss,
                                      int32_t* counts, float* prob, float* lse, int32_t* n_valid,
                                      void* workspace, size_t ws_bytes, int32_t* status,
                                      void* stream) {
  mok_balance_desc D;
  mok_status st = balance_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!loss || !counts || !prob || !n_valid) return MOK_ERR_INVALID_ARG;
  if (D.T > 0 && (!logits || !topk_idx || !lse)) return MOK_ERR_INVALID_ARG;
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(loss, 4) || !aligned(counts, 4) ||
      !aligned(prob, 4) || !aligned(lse, 4) || !aligned(n_valid, 4) || !aligned(status, 4) ||
      !aligned(workspace, 16))
    return MOK_ERR_INVALID_ARG;
  BalanceWs W;
  balance_layout(D, &W);
  if (W.total > 0 && !workspace) return MOK_ERR_INVALID_ARG;
  if (ws_bytes < W.total) return MOK_ERR_WORKSPACE;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_balance_fwd(D, logits, topk_idx, mask, loss, counts, prob, lse,
                                        n_valid, workspace, status,
                                        static_cast<cudaStream_t>(stream)));
}

mok_status mok_router_balance_backward(const mok_balance_desc* desc, const float* dloss,
                                       const float* logits, const float* lse,
                                       const int32_t* counts, const int32_t* n_valid,
                                       const uint8_t* mask, float* dlogits, void* stream) {
  mok_balance_desc D;
  mok_status st = balance_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!dloss || !counts || !n_valid) return MOK_ERR_INVALID_ARG;
  if (D.T > 0 && (!logits || !lse || !dlogits)) return MOK_ERR_INVALID_ARG;
  if (!aligned(dloss, 4) || !aligned(logits, 4) || !aligned(lse, 4) || !aligned(counts, 4) ||
      !aligned(n_valid, 4) || !aligned(dlogits, 4))
    return MOK_ERR_INVALID_ARG;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_balance_bwd(D, dloss, logits, lse, counts, n_valid, mask, dlogits,
                                        static_cast<cudaStream_t>(stream)));
}

mok_status mok_linear_forward(const mok_linear_desc* desc, const void* x, const void* w,
                              const float* bias, const void* residual, void* y, void* z,
                              void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  mok_linear_desc D;
  mok_status st = linear_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!w || (D.M > 0 && (!x || !y))) return MOK_ERR_INVALID_ARG;
  const size_t ye = elem_size(D.y_elem);
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 4) || !aligned(residual, ye) ||
      !aligned(y, ye) || !aligned(z, ye) || !aligned(status, 4) || !aligned(workspace, 16))
    return MOK_ERR_INVALID_ARG;
  const size_t need = linear_fwd_bytes(D);
  if (need > 0 && !workspace) return MOK_ERR_INVALID_ARG;
  if (ws_bytes < need) return MOK_ERR_WORKSPACE;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_linear(D, x, w, bias, residual, y, z, workspace, status,
                                   static_cast<cudaStream_t>(stream)));
}

mok_status mok_linear_workspace_size(const mok_linear_desc* desc, int backward, size_t* bytes) {
  mok_linear_desc D;
  const mok_status st = linear_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!bytes) return MOK_ERR_INVALID_ARG;
  if (!backward) {
    *bytes = linear_fwd_bytes(D);
    return MOK_OK;
  }
  LinearWs W;
  linear_layout(D, backward == 2 && linear_dz_is_dy(D, nullptr), &W);
  *bytes = W.total;
  return MOK_OK;
}

mok_status mok_linear_backward(const mok_linear_desc* desc, const void* dy, const void* x,
                               const void* w, const void* z, void* dx, float* dw, float* dbias,
                               void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  mok_linear_desc D;
  mok_status st = linear_desc(desc, &D);
  if (st != MOK_OK) return st;
  if ((D.accumulate & MOK_ADD_DX) && dx && D.dx_elem != MOK_ELEM_F32)
    return MOK_ERR_UNSUPPORTED;
  if (D.M > 0 && (!dy || (dw && !x) || (dx && !w))) return MOK_ERR_INVALID_ARG;
  if (D.M > 0 && D.act != MOK_ACT_NONE && !z) return MOK_ERR_INVALID_ARG;
  const size_t ye = elem_size(D.y_elem);
  if (!aligned(dy, ye) || !aligned(z, ye) || !aligned(x, 16) || !aligned(w, 16) ||
      !aligned(dx, 16) || !aligned(dw, 16) || !aligned(dbias, 4) || !aligned(workspace, 16) ||
      !aligned(status, 4))
    return MOK_ERR_INVALID_ARG;
  LinearWs W;
  linear_layout(D, linear_dz_is_dy(D, dy), &W);
  if (D.M > 0 && W.total > 0 && !workspace) return MOK_ERR_INVALID_ARG;
  if (D.M > 0 && ws_bytes < W.total) return MOK_ERR_WORKSPACE;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_linear_bwd(D, dy, x, w, z, dx, dw, dbias, workspace, status,
                                       static_cast<cudaStream_t>(stream)));
}

mok_status mok_dropout_forward(const mok_dropout_desc* desc, const void* x, const void* residual,
                               const int64_t* rng, void* y, void* stream) {
  return dropout(desc, x, residual, rng, y, stream);
}

mok_status mok_dropout_backward(const mok_dropout_desc* desc, const void* dy, const int64_t* rng,
                                void* dx, void* stream) {
  return dropout(desc, dy, nullptr, rng, dx, stream);
}

mok_status mok_post_pre_rmsnorm_forward(const mok_post_pre_desc* desc, const void* x,
                                        const void* residual, const void* post_weight,
                                        const void* pre_weight, const void* gate, void* s,
                                        void* y, int32_t* status, void* stream) {
  mok_post_pre_desc D;
  mok_status st = post_pre_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!post_weight || !pre_weight || (D.rows > 0 && (!x || !residual || !s || !y)))
    return MOK_ERR_INVALID_ARG;
  if (!gate_fits(D, gate)) return MOK_ERR_INVALID_ARG;
  const size_t se = elem_size(D.s_elem), we = elem_size(D.weight_elem);
  if (!aligned(x, elem_size(D.x_elem)) || !aligned(residual, se) || !aligned(s, se) ||
      !aligned(y, 2) || !aligned(post_weight, we) || !aligned(pre_weight, we) ||
      !aligned(gate, elem_size(D.gate_elem)) || !aligned(status, 4))
    return MOK_ERR_INVALID_ARG;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_post_pre(D, x, residual, post_weight, pre_weight, gate, s, y,
                                     status, static_cast<cudaStream_t>(stream)));
}

mok_status mok_post_pre_rmsnorm_workspace_size(const mok_post_pre_desc* desc, size_t* bytes) {
  mok_post_pre_desc D;
  const mok_status st = post_pre_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!bytes) return MOK_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(post_pre_bwd_blocks(D)) * static_cast<size_t>(D.d) * 8;
  return MOK_OK;
}

mok_status mok_post_pre_rmsnorm_backward(const mok_post_pre_desc* desc, const void* dy,
                                         const void* x, const void* s, const void* post_weight,
                                         const void* pre_weight, const void* gate,
                                         const void* ds, void* dx, void* dresidual, float* dpost,
                                         float* dpre, float* dgate, void* workspace,
                                         size_t ws_bytes, int32_t* status, void* stream) {
  mok_post_pre_desc D;
  mok_status st = post_pre_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!post_weight || !pre_weight || (D.rows > 0 && (!dy || !x || !s || !dx || !dresidual)))
    return MOK_ERR_INVALID_ARG;
  if (!gate_fits(D, gate)) return MOK_ERR_INVALID_ARG;
  if (dgate && D.gate == MOK_GATE_NONE) return MOK_ERR_INVALID_ARG;
  const size_t se = elem_size(D.s_elem), we = elem_size(D.weight_elem);
  if (!aligned(dy, elem_size(D.y_elem)) || !aligned(x, elem_size(D.x_elem)) || !aligned(s, se) ||
      !aligned(ds, se) || !aligned(dresidual, se) || !aligned(dx, elem_size(D.dx_elem)) ||
      !aligned(post_weight, we) || !aligned(pre_weight, we) ||
      !aligned(gate, elem_size(D.gate_elem)) || !aligned(dpost, 4) || !aligned(dpre, 4) ||
      !aligned(dgate, 4) || !aligned(status, 4))
    return MOK_ERR_INVALID_ARG;
  if (D.rows > 0 && (dpost || dpre || (dgate && D.gate == MOK_GATE_CHANNEL))) {
    if (!workspace || !aligned(workspace, 16)) return MOK_ERR_INVALID_ARG;
    size_t need = 0;
    mok_post_pre_rmsnorm_workspace_size(&D, &need);
    if (ws_bytes < need) return MOK_ERR_WORKSPACE;
  }
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(launch_post_pre_bwd(D, dy, x, s, post_weight, pre_weight, gate, ds, dx,
                                         dresidual, dpost, dpre, dgate,
                                         static_cast<float*>(workspace), status,
                                         static_cast<cudaStream_t>(stream)));
}

mok_status mok_grouped_linear_forward(const mok_grouped_desc* desc, const void* x, const void* w,
                                      const int32_t* offsets, void* y, int32_t* status,
                                      void* stream) {
  mok_grouped_desc D;
  mok_status st = grouped_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!w || !offsets || (D.rows > 0 && (!x || !y))) return MOK_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(offsets, 4) ||
      !aligned(status, 4))
    return MOK_ERR_INVALID_ARG;
  st = mok_check_device();
  if (st != MOK_OK) return st;
  return cuda_status(
      launch_grouped_fwd(D, x, w, offsets, y, status, static_cast<cudaStream_t>(stream)));
}

mok_status mok_grouped_linear_workspace_size(const mok_grouped_desc* desc, size_t* bytes) {
  mok_grouped_desc D;
  const mok_status st = grouped_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (!bytes) return MOK_ERR_INVALID_ARG;
  *bytes = grouped_ws_bytes(D);
  return MOK_OK;
}

mok_status mok_grouped_linear_backward(const mok_grouped_desc* desc, const void* dy,
                                       const void* x, const void* w, const int32_t* offsets,
                                       void* dx, float* dw, void* workspace, size_t ws_bytes,
                                       int32_t* status, void* stream) {
  mok_grouped_desc D;
  mok_status st = grouped_desc(desc, &D);
  if (st != MOK_OK) return st;
  if (D.y_elem != MOK_ELEM_BF16) return MOK_ERR_UNSUPPORTED;
  if (!offsets || (dx && !w) || (D.rows > 0 && (!dy || (dw && !x)))) return MOK_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(w, 16) || !aligned(dx, 16) ||
      !aligned(dw, 16) || !aligned(offsets, 4) || !aligned(workspace, 16) || !aligned(status, 4))
    return MOK_ERR_INVALID_ARG;
  if (dw) {
    const size_t need = grouped_ws_bytes(D);
    if (need > 0 && !workspace) return MOK_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOK_ERR_WORKSPACE;
  }
  st = mok_check_device();
  if (st != MOK_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dx) st = cuda_status(launch_grouped_dx(D, dy, w, offsets, dx, status, s));
  if (st == MOK_OK && dw) st = cuda_status(launch_grouped_dw(D, dy, x, offsets, dw, workspace, status, s));
  return st;
}

}  // extern "C"
