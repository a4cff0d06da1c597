// layer_api.cu -- the extern "C" boundary of the layer function's operators
// (layer norm, gated feed-forward block): argument validation and launches.
// No entry point allocates, synchronises or keeps state between calls.
#include <math.h>

#include "mhc_common.cuh"
#include "mhc_dispatch.h"

namespace {

constexpr int64_t kMaxTokens = (int64_t)0x7fffffffLL - 256;  // 32-bit tile coordinates
constexpr int64_t kMaxWidth = (int64_t)1 << 24;

mhc_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA; }

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool width_ok(int64_t c) { return c >= 8 && c % 8 == 0 && c <= kMaxWidth; }

size_t elem(int dtype) { return dtype == MHC_DTYPE_BF16 ? 2 : 4; }

mhc_status check(const mhc_norm_params* p) {
  if (!p || p->T < 1 || p->T > kMaxTokens || !width_ok(p->C)) return MHC_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || !isfinite(p->eps)) return MHC_ERR_INVALID_ARG;
  if (p->dtype != MHC_DTYPE_F32 && p->dtype != MHC_DTYPE_BF16) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

mhc_status check(const mhc_ffn_params* p) {
  if (!p || p->T < 1 || p->T > kMaxTokens || !width_ok(p->C) || !width_ok(p->F) || p->wait_ns < 0)
    return MHC_ERR_INVALID_ARG;
  if (p->dtype != MHC_DTYPE_F32 && p->dtype != MHC_DTYPE_BF16) return MHC_ERR_UNSUPPORTED;
  if (p->act != MHC_ACT_SILU && p->act != MHC_ACT_GELU) return MHC_ERR_UNSUPPORTED;
  return MHC_OK;
}

// One array argument: where it lies and how long it is.  p == nullptr marks an
// optional array that was left out.
struct Span {
  const void* p;
  size_t bytes;
  bool out;
};

// Every array 16-byte aligned, and no output over another array.
template <int K>
mhc_status check_spans(const Span (&a)[K]) {
  for (int i = 0; i < K; ++i)
    if (((uintptr_t)a[i].p & 15u) != 0) return MHC_ERR_INVALID_ARG;
  for (int i = 0; i < K; ++i)
    for (int j = 0; j < i; ++j) {
      if ((!a[i].out && !a[j].out) || !a[i].p || !a[j].p) continue;
      const uintptr_t pi = (uintptr_t)a[i].p, pj = (uintptr_t)a[j].p;
      if (pi < pj + a[j].bytes && pj < pi + a[i].bytes) return MHC_ERR_INVALID_ARG;
    }
  return MHC_OK;
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws != nullptr && bytes >= need && ((uintptr_t)ws & 255u) == 0);
}

}  // namespace

extern "C" {

mhc_status mhc_layer_norm(const mhc_norm_params* p, const void* x, const float* weight,
                          const float* bias, void* y, int* dev_status, mhc_stream_t stream) {
  mhc_status st = check(p);
  if (st != MHC_OK) return st;
  if (!x || !weight || !y) return MHC_ERR_INVALID_ARG;
  const size_t act = (size_t)p->T * p->C * elem(p->dtype), row = (size_t)p->C * 4;
  const Span a[] = {{x, act, false}, {weight, row, false}, {bias, row, false}, {y, act, true}};
  st = check_spans(a);
  if (st != MHC_OK) return st;
  return from_cuda(mhc::norm_fwd_dispatch(p->dtype, p->T, p->C, p->eps, x, weight, bias, y,
                                          dev_status, (cudaStream_t)stream));
}

size_t mhc_layer_norm_backward_workspace_size(const mhc_norm_params* p) {
  if (check(p) != MHC_OK) return 0;
  return round_up(mhc::norm_bwd_workspace_bytes(p->T, p->C, p->dtype), 256);
}

mhc_status mhc_layer_norm_backward(const mhc_norm_params* p, const void* x, const float* weight,
                                   const void* grad_y, void* grad_x, float* grad_weight,
                                   float* grad_bias, void* workspace, size_t workspace_bytes,
                                   int* dev_status, mhc_stream_t stream) {
  mhc_status st = check(p);
  if (st != MHC_OK) return st;
  if (!x || !weight || !grad_y || !grad_x || !grad_weight) return MHC_ERR_INVALID_ARG;
  const size_t need = mhc_layer_norm_backward_workspace_size(p);
  if (!workspace_ok(workspace, workspace_bytes, need)) return MHC_ERR_WORKSPACE;
  const size_t act = (size_t)p->T * p->C * elem(p->dtype), row = (size_t)p->C * 4;
  const Span a[] = {{x, act, false},          {weight, row, false},   {grad_y, act, false},
                    {grad_x, act, true},      {grad_weight, row, true}, {grad_bias, row, true},
                    {workspace, need, true}};
  st = check_spans(a);
  if (st != MHC_OK) return st;
  return from_cuda(mhc::norm_bwd_dispatch(p->dtype, p->T, p->C, p->eps, x, weight, grad_y, grad_x,
                                          grad_weight, grad_bias, workspace, dev_status,
                                          (cudaStream_t)stream));
}

size_t mhc_ffn_workspace_size(const mhc_ffn_params* p) {
  if (check(p) != MHC_OK) return 0;
  return round_up(mhc::ffn_fwd_workspace_bytes(p->dtype, p->T, p->C, p->F), 256);
}

mhc_status mhc_ffn(const mhc_ffn_params* p, const void* x, const void* w_gate, const void* w_up,
                   const void* w_down, void* y, void* workspace, size_t workspace_bytes,
                   int* dev_status, mhc_stream_t stream) {
  mhc_status st = check(p);
  if (st != MHC_OK) return st;
  if (!x || !w_gate || !w_up || !w_down || !y) return MHC_ERR_INVALID_ARG;
  const size_t need = mhc_ffn_workspace_size(p);
  if (!workspace_ok(workspace, workspace_bytes, need)) return MHC_ERR_WORKSPACE;
  const size_t act = (size_t)p->T * p->C * elem(p->dtype);
  const size_t wt = (size_t)p->F * p->C * elem(p->dtype);
  const Span a[] = {{x, act, false},     {w_gate, wt, false}, {w_up, wt, false},
                    {w_down, wt, false}, {y, act, true},      {workspace, need, true}};
  st = check_spans(a);
  if (st != MHC_OK) return st;
  return from_cuda(mhc::ffn_fwd_dispatch(p->dtype, p->act, p->T, p->C, p->F, x, w_gate, w_up,
                                         w_down, y, workspace, dev_status, p->wait_ns,
                                         (cudaStream_t)stream));
}

size_t mhc_ffn_backward_workspace_size(const mhc_ffn_params* p) {
  if (check(p) != MHC_OK) return 0;
  return round_up(mhc::ffn_bwd_workspace_bytes(p->dtype, p->T, p->C, p->F), 256);
}

mhc_status mhc_ffn_backward(const mhc_ffn_params* p, const void* x, const void* w_gate,
                            const void* w_up, const void* w_down, const void* grad_y, void* grad_x,
                            void* grad_w_gate, void* grad_w_up, void* grad_w_down, void* workspace,
                            size_t workspace_bytes, int* dev_status, mhc_stream_t stream) {
  mhc_status st = check(p);
  if (st != MHC_OK) return st;
  if (!x || !w_gate || !w_up || !w_down || !grad_y || !grad_x || !grad_w_gate || !grad_w_up ||
      !grad_w_down)
    return MHC_ERR_INVALID_ARG;
  const size_t need = mhc_ffn_backward_workspace_size(p);
  if (!workspace_ok(workspace, workspace_bytes, need)) return MHC_ERR_WORKSPACE;
  const size_t act = (size_t)p->T * p->C * elem(p->dtype);
  const size_t wt = (size_t)p->F * p->C * elem(p->dtype);
  const Span a[] = {{x, act, false},          {w_gate, wt, false},   {w_up, wt, false},
                    {w_down, wt, false},      {grad_y, act, false},  {grad_x, act, true},
                    {grad_w_gate, wt, true},  {grad_w_up, wt, true}, {grad_w_down, wt, true},
                    {workspace, need, true}};
  st = check_spans(a);
  if (st != MHC_OK) return st;
  return from_cuda(mhc::ffn_bwd_dispatch(p->dtype, p->act, p->T, p->C, p->F, x, w_gate, w_up,
                                         w_down, grad_y, grad_x, grad_w_gate, grad_w_up,
                                         grad_w_down, workspace, dev_status, p->wait_ns,
                                         (cudaStream_t)stream));
}

}  // extern "C"
