// Attention among the nodes of each graph, and its reverse pass (contract in e3conv.h).
//
// One wave per row: S = scale <q, k> of 64 keys at a time (a lane each), the
// running maximum and sum of the softmax, then out with the lanes across the
// value dimensions.  The reverse pass forms P = exp(S - lse) again, once per
// query row (grad_q, which also leaves delta) and once per key row (grad_k, grad_v).
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "e3conv.h"
#include "kernels.h"

namespace e3c {
namespace {

constexpr int kMaxDim = 128;

struct AttnParams {
  e3conv_attention_args a;
  int group;                       // query heads per kv head
  void* out;
  long out_row, out_head;
  float* lse;
  const void* go;
  long go_row, go_head;
  void *gq, *gk, *gv;
  long gq_row, gq_head, gk_row, gk_head, gv_row, gv_head;
  float* delta;                    // (num_q, heads_q), reverse pass
};

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __bf16* p) { return (float)*p; }

__device__ __forceinline__ float wave_max(float v) {
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Offset i of a segment table, kept inside [0, n] whatever the table holds.
__device__ __forceinline__ int offset(const int* ptr, int i, int n) {
  const int v = ptr[i];
  return v < 0 ? 0 : (v > n ? n : v);
}

// The graph whose segment holds row i.
__device__ __forceinline__ int graph_of(const int* ptr, int graphs, int i) {
  int lo = 0, hi = graphs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ptr[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <class T>
__device__ __forceinline__ float dot(const T* a, const T* b, int n) {
  float s = 0.0f;
  for (int d = 0; d < n; ++d) s = fmaf(load(a + d), load(b + d), s);
  return s;
}

template <class T>
__global__ void __launch_bounds__(64) attn_fwd(AttnParams p) {
  const e3conv_attention_args& a = p.a;
  const int h = blockIdx.x % a.heads_q, i = blockIdx.x / a.heads_q, c = h / p.group, lane = threadIdx.x;
  const int g = graph_of(a.q_ptr, a.num_graphs, i);
  const T* q = (const T*)a.q + i * a.q_row + h * a.q_head;
  const T* k = (const T*)a.k + c * a.k_head;
  const T* v = (const T*)a.v + c * a.v_head;
  int k0 = offset(a.k_ptr, g, (int)a.num_k);
  const int k1 = offset(a.k_ptr, g + 1, (int)a.num_k);
  if (a.q_mask && !a.q_mask[i]) k0 = k1;
  float m = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f;
  for (; k0 < k1; k0 += 64) {
    const int j = k0 + lane;
    const bool seen = j < k1 && (!a.k_mask || a.k_mask[j]);
    const float s = seen ? a.scale * dot(q, k + j * a.k_row, a.dim_qk) : -INFINITY;
    const unsigned long any = __ballot(seen);
    if (!any) continue;
    const float mn = fmaxf(m, wave_max(s));
    const float base = mn == -INFINITY ? 0.0f : mn;
    const float r = expf(m - base), e = seen ? expf(s - base) : 0.0f;
    l = l * r + wave_sum(e);
    o0 *= r;
    o1 *= r;
    m = mn;
    for (int t = 0; t < 64; ++t) {
      if (!(any >> t & 1)) continue;
      const float w = __shfl(e, t);
      const T* vr = v + (k0 + t) * a.v_row;
      if (lane < a.dim_v) o0 = fmaf(w, load(vr + lane), o0);
      if (lane + 64 < a.dim_v) o1 = fmaf(w, load(vr + lane + 64), o1);
    }
  }
  T* out = (T*)p.out + i * p.out_row + h * p.out_head;
  const float inv = m == -INFINITY && l == 0.0f ? 0.0f : 1.0f / l;
  if (lane < a.dim_v) out[lane] = (T)(o0 * inv);
  if (lane + 64 < a.dim_v) out[lane + 64] = (T)(o1 * inv);
  if (lane == 0 && p.lse) p.lse[(long)i * a.heads_q + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <class T>
__global__ void __launch_bounds__(64) attn_bwd_q(AttnParams p) {
  const e3conv_attention_args& a = p.a;
  const int h = blockIdx.x % a.heads_q, i = blockIdx.x / a.heads_q, c = h / p.group, lane = threadIdx.x;
  const int g = graph_of(a.q_ptr, a.num_graphs, i);
  const T* q = (const T*)a.q + i * a.q_row + h * a.q_head;
  const T* go = (const T*)p.go + i * p.go_row + h * p.go_head;
  const T* out = (const T*)p.out + i * p.out_row + h * p.out_head;
  const T* k = (const T*)a.k + c * a.k_head;
  const T* v = (const T*)a.v + c * a.v_head;
  int k0 = offset(a.k_ptr, g, (int)a.num_k);
  const int k1 = offset(a.k_ptr, g + 1, (int)a.num_k);
  const float lse = p.lse[(long)i * a.heads_q + h];
  if ((a.q_mask && !a.q_mask[i]) || lse == -INFINITY) k0 = k1;
  float delta = 0.0f, g0 = 0.0f, g1 = 0.0f;
  if (k0 < k1) {
    if (lane < a.dim_v) delta += load(go + lane) * load(out + lane);
    if (lane + 64 < a.dim_v) delta += load(go + lane + 64) * load(out + lane + 64);
    delta = wave_sum(delta);
  }
  if (lane == 0) p.delta[(long)i * a.heads_q + h] = delta;
  for (; k0 < k1; k0 += 64) {
    const int j = k0 + lane;
    const bool seen = j < k1 && (!a.k_mask || a.k_mask[j]);
    float ds = 0.0f;
    if (seen) {
      const float w = expf(a.scale * dot(q, k + j * a.k_row, a.dim_qk) - lse);
      ds = a.scale * w * (dot(go, v + j * a.v_row, a.dim_v) - delta);
    }
    const unsigned long any = __ballot(seen);
    for (int t = 0; t < 64; ++t) {
      if (!(any >> t & 1)) continue;
      const float w = __shfl(ds, t);
      const T* kr = k + (k0 + t) * a.k_row;
      if (lane < a.dim_qk) g0 = fmaf(w, load(kr + lane), g0);
      if (lane + 64 < a.dim_qk) g1 = fmaf(w, load(kr + lane + 64), g1);
    }
  }
  T* gq = (T*)p.gq + i * p.gq_row + h * p.gq_head;
  if (lane < a.dim_qk) gq[lane] = (T)g0;
  if (lane + 64 < a.dim_qk) gq[lane + 64] = (T)g1;
}

template <class T>
__global__ void __launch_bounds__(64) attn_bwd_kv(AttnParams p) {
  const e3conv_attention_args& a = p.a;
  const int c = blockIdx.x % a.heads_kv, j = blockIdx.x / a.heads_kv, lane = threadIdx.x;
  const int g = graph_of(a.k_ptr, a.num_graphs, j);
  const T* k = (const T*)a.k + j * a.k_row + c * a.k_head;
  const T* v = (const T*)a.v + j * a.v_row + c * a.v_head;
  const int q0 = offset(a.q_ptr, g, (int)a.num_q);
  int rows = (offset(a.q_ptr, g + 1, (int)a.num_q) - q0) * p.group;    // (query, head of the group)
  if (a.k_mask && !a.k_mask[j]) rows = 0;
  float k0 = 0.0f, k1 = 0.0f, v0 = 0.0f, v1 = 0.0f;
  for (int r0 = 0; r0 < rows; r0 += 64) {
    const int r = r0 + lane;
    bool sees = r < rows;
    float w = 0.0f, ds = 0.0f;
    if (sees) {
      const int i = q0 + r / p.group, h = c * p.group + r % p.group;
      const float lse = p.lse[(long)i * a.heads_q + h];
      sees = lse != -INFINITY && (!a.q_mask || a.q_mask[i]);
      if (sees) {
        w = expf(a.scale * dot((const T*)a.q + i * a.q_row + h * a.q_head, k, a.dim_qk) - lse);
        const float dp = dot((const T*)p.go + i * p.go_row + h * p.go_head, v, a.dim_v);
        ds = a.scale * w * (dp - p.delta[(long)i * a.heads_q + h]);
      }
    }
    const unsigned long any = __ballot(sees);
    for (int t = 0; t < 64; ++t) {
      if (!(any >> t & 1)) continue;
      const int i = q0 + (r0 + t) / p.group, h = c * p.group + (r0 + t) % p.group;
      const float wt = __shfl(w, t), dt = __shfl(ds, t);
      const T* q = (const T*)a.q + i * a.q_row + h * a.q_head;
      const T* go = (const T*)p.go + i * p.go_row + h * p.go_head;
      if (lane < a.dim_qk) k0 = fmaf(dt, load(q + lane), k0);
      if (lane + 64 < a.dim_qk) k1 = fmaf(dt, load(q + lane + 64), k1);
      if (lane < a.dim_v) v0 = fmaf(wt, load(go + lane), v0);
      if (lane + 64 < a.dim_v) v1 = fmaf(wt, load(go + lane + 64), v1);
    }
  }
  T* gk = (T*)p.gk + j * p.gk_row + c * p.gk_head;
  T* gv = (T*)p.gv + j * p.gv_row + c * p.gv_head;
  if (lane < a.dim_qk) gk[lane] = (T)k0;
  if (lane + 64 < a.dim_qk) gk[lane + 64] = (T)k1;
  if (lane < a.dim_v) gv[lane] = (T)v0;
  if (lane + 64 < a.dim_v) gv[lane + 64] = (T)v1;
}

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

size_t workspace_bytes(const e3conv_attention_args& a, int backward) {
  return backward ? ((size_t)a.num_q * a.heads_q * sizeof(float) + 15) / 16 * 16 : 0;
}

}  // namespace
}  // namespace e3c

extern "C" {

e3conv_status e3conv_attention_workspace_size(const e3conv_attention_args* a, int backward, size_t* bytes) {
  const e3conv_status st = e3c::check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (!bytes) return e3c::bad("bytes is NULL");
  *bytes = e3c::workspace_bytes(*a, backward);
  return e3c::api_ok();
}

e3conv_status e3conv_attention(const e3conv_attention_args* a, void* out, int64_t out_row, int64_t out_head,
                               float* lse, void* workspace, size_t bytes, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (a->num_q == 0) return e3c::api_ok();
  if (!out) return e3c::bad("NULL device pointer");
  if (out_row < 0 || out_head < 0) return e3c::bad("negative stride");
  e3c::AttnParams p{};
  p.a = *a;
  p.group = a->heads_q / a->heads_kv;
  p.out = out;
  p.out_row = out_row;
  p.out_head = out_head;
  p.lse = lse;
  const dim3 grid((unsigned)(a->num_q * a->heads_q));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a->dtype == E3CONV_F32) hipLaunchKernelGGL(e3c::attn_fwd<float>, grid, dim3(64), 0, s, p);
  else hipLaunchKernelGGL(e3c::attn_fwd<__bf16>, grid, dim3(64), 0, s, p);
  const hipError_t err = hipGetLastError();
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
  const size_t need = e3c::workspace_bytes(*a, 1);
  if (bytes < need || (need > 0 && !workspace))
    return e3c::api_fail(E3CONV_ERR_WORKSPACE, "attention backward needs " + std::to_string(need) + " bytes");
  e3c::AttnParams p{};
  p.a = *a;
  p.group = a->heads_q / a->heads_kv;
  p.out = const_cast<void*>(out);
  p.lse = const_cast<float*>(lse);
  p.go = grad_out;
  p.gq = grad_q;
  p.gk = grad_k;
  p.gv = grad_v;
  long* const at[10] = {&p.out_row, &p.out_head, &p.go_row, &p.go_head, &p.gq_row,
                        &p.gq_head, &p.gk_row, &p.gk_head, &p.gv_row, &p.gv_head};
  for (int i = 0; i < 10; ++i) *at[i] = strides[i];
  p.delta = static_cast<float*>(workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 gq((unsigned)(a->num_q * a->heads_q)), gk((unsigned)(a->num_k * a->heads_kv));
  if (a->num_q > 0) {
    if (a->dtype == E3CONV_F32) hipLaunchKernelGGL(e3c::attn_bwd_q<float>, gq, dim3(64), 0, s, p);
    else hipLaunchKernelGGL(e3c::attn_bwd_q<__bf16>, gq, dim3(64), 0, s, p);
  }
  if (a->num_k > 0) {
    if (a->dtype == E3CONV_F32) hipLaunchKernelGGL(e3c::attn_bwd_kv<float>, gk, dim3(64), 0, s, p);
    else hipLaunchKernelGGL(e3c::attn_bwd_kv<__bf16>, gk, dim3(64), 0, s, p);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return e3c::api_hip_fail(err, "attention backward launch");
  return e3c::api_ok();
}

}  // extern "C"
