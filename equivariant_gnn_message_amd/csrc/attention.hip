// Entry points of attention among the nodes of each graph (contract in e3conv.h): argument
// checks, and the parameters of the kernels in attention_fwd.hip and attention_bwd.hip.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <string>

#include "attention_tile.h"
#include "e3conv.h"
#include "kernels.h"

namespace e3c {
namespace {

using attn::kMaxDim;

e3conv_status bad(const char* what) { return api_fail(E3CONV_ERR_INVALID_ARGUMENT, what); }

// Sizes, dtype, scale and strides; E3CONV_OK leaves the error detail as it is.
e3conv_status check_sizes(const e3conv_attention_args* a) {
  if (!a) return bad("args is NULL");
  if (a->dtype != E3CONV_F32 && a->dtype != E3CONV_BF16) return bad("bad dtype");
  if (a->num_graphs < 0 || a->num_q < 0 || a->num_k < 0) return bad("negative size");
  if (a->num_graphs == 0 && (a->num_q > 0 || a->num_k > 0)) return bad("rows without a graph");
  if (a->heads_q <= 0 || a->heads_kv <= 0 || a->heads_q % a->heads_kv != 0)
    return bad("heads_q must be a positive multiple of heads_kv");
  if (a->dim_qk < 1 || a->dim_qk > kMaxDim || a->dim_v < 1 || a->dim_v > kMaxDim)
    return bad("dim_qk and dim_v must be in [1, 128]");
  const int64_t most = ((int64_t)1 << 31) - ((int64_t)1 << 20);
  if (a->num_q >= most / a->heads_q || a->num_k >= most / a->heads_kv || a->num_graphs >= (1 << 20))
    return bad("sizes must fit int32 indices");
  if (!std::isfinite(a->scale)) return bad("scale must be finite");
  return E3CONV_OK;
}

e3conv_status check_args(const e3conv_attention_args* a) {
  const e3conv_status st = check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (a->q_row < 0 || a->q_head < 0 || a->k_row < 0 || a->k_head < 0 || a->v_row < 0 || a->v_head < 0)
    return bad("negative stride");
  if (a->num_graphs > 0 && (!a->q_ptr || !a->k_ptr)) return bad("NULL device pointer");
  if (a->num_q > 0 && !a->q) return bad("NULL device pointer");
  if (a->num_k > 0 && (!a->k || !a->v)) return bad("NULL device pointer");
  return E3CONV_OK;
}

// Whether 16-byte loads of whole units of eight elements reach no further than the rows.
bool vector_rows(const void* p, int64_t row, int64_t head, int dim, int size) {
  const int64_t unit = 16 / size;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % unit == 0 && head % unit == 0 && dim % 8 == 0;
}
// Elements of the rows' aligned stores: 8 of bf16, 4, or 0.
int vector_stores(const void* p, int64_t row, int64_t head, int dim, int size) {
  const auto aligned = [&](int n) {
    return reinterpret_cast<uintptr_t>(p) % (n * size) == 0 && row % n == 0 && head % n == 0;
  };
  return size == 2 && dim % 8 == 0 && aligned(8) ? 8 : aligned(4) ? 4 : 0;
}

attn::Params params(const e3conv_attention_args& a) {
  attn::Params p{};
  p.a = a;
  p.group = a.heads_q / a.heads_kv;
  const attn::GroupDiv by = attn::group_div(p.group);
  p.magic = by.magic;
  p.shift = by.shift;
  p.group_log2 = by.log2;
  p.negate = a.scale < 0.0f;
  // a zero scale: logits far below one unit of the sums' rounding, infinities as they are
  p.c = std::fabs(a.scale) * attn::kLog2e;
  if (p.c < FLT_MIN) p.c = FLT_MIN;
  const int size = a.dtype == E3CONV_F32 ? 4 : 2;
  p.vec = vector_rows(a.q, a.q_row, a.q_head, a.dim_qk, size) && vector_rows(a.k, a.k_row, a.k_head, a.dim_qk, size) &&
          vector_rows(a.v, a.v_row, a.v_head, a.dim_v, size);
  p.full = a.dim_qk == a.dim_v && a.dim_qk == attn::padded(a.dim_qk);
  return p;
}

}  // namespace
}  // namespace e3c

extern "C" {

e3conv_status e3conv_attention_workspace_size(const e3conv_attention_args* a, int backward, size_t* bytes) {
  const e3conv_status st = e3c::check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (!bytes) return e3c::bad("bytes is NULL");
  *bytes = backward ? e3c::attn::backward_workspace(*a) : e3c::attn::forward_workspace(*a);
  return e3c::api_ok();
}

e3conv_status e3conv_attention(const e3conv_attention_args* a, void* out, int64_t out_row, int64_t out_head,
                               float* lse, void* workspace, size_t bytes, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (a->num_q == 0) return e3c::api_ok();
  if (!out) return e3c::bad("NULL device pointer");
  if (out_row < 0 || out_head < 0) return e3c::bad("negative stride");
  const size_t need = e3c::attn::forward_workspace(*a);
  if (bytes < need || (need > 0 && !workspace))
    return e3c::api_fail(E3CONV_ERR_WORKSPACE, "attention needs " + std::to_string(need) + " bytes");
  e3c::attn::Params p = e3c::params(*a);
  p.out = out;
  p.out_row = out_row;
  p.out_head = out_head;
  p.vec_st = e3c::vector_stores(out, out_row, out_head, a->dim_v, a->dtype == E3CONV_F32 ? 4 : 2);
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  const hipError_t err = e3c::attn::launch_forward(p, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) return e3c::api_hip_fail(err, "attention launch");
  return e3c::api_ok();
}

e3conv_status e3conv_attention_backward(const e3conv_attention_args* a, const void* out, const float* lse,
                                        const void* grad_out, void* grad_q, void* grad_k, void* grad_v,
                                        const int64_t strides[10], void* workspace, size_t bytes,
                                        void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (!strides) return e3c::bad("strides is NULL");
  for (int i = 0; i < 10; ++i)
    if (strides[i] < 0) return e3c::bad("negative stride");
  if (a->num_q == 0 && a->num_k == 0) return e3c::api_ok();
  if (a->num_q > 0 && (!out || !lse || !grad_out || !grad_q)) return e3c::bad("NULL device pointer");
  if (a->num_k > 0 && (!grad_k || !grad_v)) return e3c::bad("NULL device pointer");
  const size_t need = e3c::attn::backward_workspace(*a);
  if (bytes < need || (need > 0 && !workspace))
    return e3c::api_fail(E3CONV_ERR_WORKSPACE, "attention backward needs " + std::to_string(need) + " bytes");
  e3c::attn::Params p = e3c::params(*a);
  p.out = const_cast<void*>(out);
  p.lse = const_cast<float*>(lse);
  p.go = grad_out;
  p.gq = grad_q;
  p.gk = grad_k;
  p.gv = grad_v;
  long* const at[10] = {&p.out_row, &p.out_head, &p.go_row, &p.go_head, &p.gq_row,
                        &p.gq_head, &p.gk_row, &p.gk_head, &p.gv_row, &p.gv_head};
  for (int i = 0; i < 10; ++i) *at[i] = strides[i];
  const int size = a->dtype == E3CONV_F32 ? 4 : 2;
  p.vec = p.vec && e3c::vector_rows(out, p.out_row, p.out_head, a->dim_v, size) &&
          e3c::vector_rows(grad_out, p.go_row, p.go_head, a->dim_v, size);
  p.vec_st = std::min({e3c::vector_stores(grad_q, p.gq_row, p.gq_head, a->dim_qk, size),
                       e3c::vector_stores(grad_k, p.gk_row, p.gk_head, a->dim_qk, size),
                       e3c::vector_stores(grad_v, p.gv_row, p.gv_head, a->dim_v, size)});
  p.delta = static_cast<float*>(workspace);
  const hipError_t err = e3c::attn::launch_backward(p, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) return e3c::api_hip_fail(err, "attention backward launch");
  return e3c::api_ok();
}

}  // extern "C"
