// Group norm with an activation over the rows of each graph, channels last, and its
// reverse pass (contract in e3conv.h).
//
// One work-group per (graph, group): mean, then the variance about it, then
// the rows.  The reverse pass takes the two means of a group the same way; the
// weight and bias gradients are sums over all rows, one work-group per channel.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "e3conv.h"
#include "kernels.h"

namespace e3c {
namespace {

constexpr int kMaxChannels = 4096;

struct NormParams {
  e3conv_group_norm_args a;
  int gc;                          // channels of a group
  void* y;
  long y_row;
  float *mean, *rstd;
  const void* gy;
  long gy_row;
  void* gx;
  long gx_row;
  float *gw, *gb;
};

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __bf16* p) { return (float)*p; }

__device__ __forceinline__ int offset(const int* ptr, int i, int n) {
  const int v = ptr[i];
  return v < 0 ? 0 : (v > n ? n : v);
}

__device__ __forceinline__ int graph_of(const int* ptr, int graphs, int i) {
  int lo = 0, hi = graphs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ptr[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sum over the 256 threads of a work-group, in every thread.
__device__ float block_sum(float v) {
  __shared__ float part[4];
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case E3CONV_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case E3CONV_ACT_SILU: return z / (1.0f + expf(-z));
    case E3CONV_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    default: return z;
  }
}

__device__ __forceinline__ float activate_grad(float z, int act) {
  switch (act) {
    case E3CONV_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case E3CONV_ACT_SILU: {
      const float e = 1.0f / (1.0f + expf(-z));
      return e * (1.0f + z * (1.0f - e));
    }
    case E3CONV_ACT_GELU:
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * 0.39894228040143268f * expf(-0.5f * z * z);
    default: return 1.0f;
  }
}

template <class T>
__global__ void __launch_bounds__(256) norm_fwd(NormParams p) {
  const e3conv_group_norm_args& a = p.a;
  const int b = blockIdx.x / a.groups, grp = blockIdx.x % a.groups, gc = p.gc, c0 = grp * gc;
  const int r0 = offset(a.row_ptr, b, (int)a.num_rows), r1 = offset(a.row_ptr, b + 1, (int)a.num_rows);
  const T* x = (const T*)a.x + c0;
  const long n = (long)(r1 > r0 ? r1 - r0 : 0) * gc;
  float s = 0.0f, cnt = 0.0f;
  for (long t = threadIdx.x; t < n; t += 256) {
    const long r = r0 + t / gc;
    if (a.row_mask && !a.row_mask[r]) continue;
    s += load(x + r * a.x_row + t % gc);
    cnt += 1.0f;
  }
  cnt = block_sum(cnt);
  const float mean = cnt > 0.0f ? block_sum(s) / cnt : (block_sum(s), 0.0f);
  float v = 0.0f;
  for (long t = threadIdx.x; t < n; t += 256) {
    const long r = r0 + t / gc;
    if (a.row_mask && !a.row_mask[r]) continue;
    const float d = load(x + r * a.x_row + t % gc) - mean;
    v = fmaf(d, d, v);
  }
  v = block_sum(v);
  const float rstd = 1.0f / sqrtf((cnt > 0.0f ? v / cnt : 0.0f) + a.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[b * a.groups + grp] = mean;
    if (p.rstd) p.rstd[b * a.groups + grp] = rstd;
  }
  for (long t = threadIdx.x; t < n; t += 256) {
    const long r = r0 + t / gc;
    const int c = (int)(t % gc);
    float y = 0.0f;
    if (!a.row_mask || a.row_mask[r]) {
      const float xh = (load(x + r * a.x_row + c) - mean) * rstd;
      y = activate(fmaf(xh, a.weight ? a.weight[c0 + c] : 1.0f, a.bias ? a.bias[c0 + c] : 0.0f), a.activation);
    }
    ((T*)p.y)[r * p.y_row + c0 + c] = (T)y;
  }
}

// dz of row r, channel c and its xhat.
template <class T>
__device__ __forceinline__ float dz_of(const NormParams& p, long r, int c, float mean, float rstd, float& xh) {
  const e3conv_group_norm_args& a = p.a;
  xh = (load((const T*)a.x + r * a.x_row + c) - mean) * rstd;
  const float z = fmaf(xh, a.weight ? a.weight[c] : 1.0f, a.bias ? a.bias[c] : 0.0f);
  return load((const T*)p.gy + r * p.gy_row + c) * activate_grad(z, a.activation);
}

// Before norm_bwd_x, which may write grad_x over grad_y.
template <class T>
__global__ void __launch_bounds__(256) norm_bwd_w(NormParams p) {
  const e3conv_group_norm_args& a = p.a;
  const int c = blockIdx.x, grp = c / p.gc;
  float w = 0.0f, b = 0.0f;
  for (long r = threadIdx.x; r < a.num_rows; r += 256) {
    if (a.row_mask && !a.row_mask[r]) continue;
    const int g = graph_of(a.row_ptr, a.num_graphs, (int)r) * a.groups + grp;
    float xh;
    const float dz = dz_of<T>(p, r, c, p.mean[g], p.rstd[g], xh);
    w = fmaf(dz, xh, w);
    b += dz;
  }
  w = block_sum(w);
  b = block_sum(b);
  if (threadIdx.x == 0) {
    if (p.gw) p.gw[c] = w;
    if (p.gb) p.gb[c] = b;
  }
}

template <class T>
__global__ void __launch_bounds__(256) norm_bwd_x(NormParams p) {
  const e3conv_group_norm_args& a = p.a;
  const int b = blockIdx.x / a.groups, grp = blockIdx.x % a.groups, gc = p.gc, c0 = grp * gc;
  const int r0 = offset(a.row_ptr, b, (int)a.num_rows), r1 = offset(a.row_ptr, b + 1, (int)a.num_rows);
  const long n = (long)(r1 > r0 ? r1 - r0 : 0) * gc;
  const float mean = p.mean[b * a.groups + grp], rstd = p.rstd[b * a.groups + grp];
  float s1 = 0.0f, s2 = 0.0f, cnt = 0.0f;
  for (long t = threadIdx.x; t < n; t += 256) {
    const long r = r0 + t / gc;
    if (a.row_mask && !a.row_mask[r]) continue;
    const int c = c0 + (int)(t % gc);
    float xh;
    const float dn = dz_of<T>(p, r, c, mean, rstd, xh) * (a.weight ? a.weight[c] : 1.0f);
    s1 += dn;
    s2 = fmaf(dn, xh, s2);
    cnt += 1.0f;
  }
  cnt = fmaxf(block_sum(cnt), 1.0f);
  const float m1 = block_sum(s1) / cnt, m2 = block_sum(s2) / cnt;
  for (long t = threadIdx.x; t < n; t += 256) {
    const long r = r0 + t / gc;
    const int c = c0 + (int)(t % gc);
    float dx = 0.0f;
    if (!a.row_mask || a.row_mask[r]) {
      float xh;
      const float dn = dz_of<T>(p, r, c, mean, rstd, xh) * (a.weight ? a.weight[c] : 1.0f);
      dx = rstd * (dn - m1 - xh * m2);
    }
    ((T*)p.gx)[r * p.gx_row + c] = (T)dx;
  }
}

e3conv_status bad(const char* what) { return api_fail(E3CONV_ERR_INVALID_ARGUMENT, what); }

e3conv_status check_sizes(const e3conv_group_norm_args* a) {
  if (!a) return bad("args is NULL");
  if (a->dtype != E3CONV_F32 && a->dtype != E3CONV_BF16) return bad("bad dtype");
  if (a->num_graphs < 0 || a->num_rows < 0) return bad("negative size");
  if (a->num_graphs == 0 && a->num_rows > 0) return bad("rows without a graph");
  if (a->channels < 1 || a->channels > kMaxChannels || a->groups < 1 || a->channels % a->groups != 0)
    return bad("channels must be in [1, 4096] and a multiple of groups");
  if (a->num_rows + a->num_graphs >= ((int64_t)1 << 31) - ((int64_t)1 << 20))
    return bad("sizes must fit int32 indices");
  if ((int)a->activation < E3CONV_ACT_NONE || (int)a->activation > E3CONV_ACT_GELU) return bad("unknown activation");
  if (!(a->eps > 0.0f) || !std::isfinite(a->eps)) return bad("eps must be positive");
  return E3CONV_OK;
}

e3conv_status check_args(const e3conv_group_norm_args* a) {
  const e3conv_status st = check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (a->x_row < 0) return bad("negative stride");
  if (a->num_graphs > 0 && !a->row_ptr) return bad("NULL device pointer");
  if (a->num_rows > 0 && !a->x) return bad("NULL device pointer");
  return E3CONV_OK;
}

}  // namespace
}  // namespace e3c

extern "C" {

e3conv_status e3conv_group_norm_workspace_size(const e3conv_group_norm_args* a, int backward, size_t* bytes) {
  const e3conv_status st = e3c::check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (!bytes) return e3c::bad("bytes is NULL");
  *bytes = 0;
  return e3c::api_ok();
}

e3conv_status e3conv_group_norm(const e3conv_group_norm_args* a, void* y, int64_t y_row, float* mean, float* rstd,
                                void* workspace, size_t bytes, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (y_row < 0) return e3c::bad("negative stride");
  if (a->num_graphs == 0) return e3c::api_ok();
  if (a->num_rows > 0 && !y) return e3c::bad("NULL device pointer");
  e3c::NormParams p{};
  p.a = *a;
  p.gc = a->channels / a->groups;
  p.y = y;
  p.y_row = y_row;
  p.mean = mean;
  p.rstd = rstd;
  const dim3 grid((unsigned)((long)a->num_graphs * a->groups));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a->dtype == E3CONV_F32) hipLaunchKernelGGL(e3c::norm_fwd<float>, grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(e3c::norm_fwd<__bf16>, grid, dim3(256), 0, s, p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return e3c::api_hip_fail(err, "group norm launch");
  return e3c::api_ok();
}

e3conv_status e3conv_group_norm_backward(const e3conv_group_norm_args* a, const float* mean, const float* rstd,
                                         const void* grad_y, int64_t grad_y_row, void* grad_x,
                                         int64_t grad_x_row, float* grad_weight, float* grad_bias,
                                         void* workspace, size_t bytes, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (grad_y_row < 0 || grad_x_row < 0) return e3c::bad("negative stride");
  if (a->num_graphs > 0 && (!mean || !rstd)) return e3c::bad("NULL device pointer");
  if (a->num_rows > 0 && (!grad_y || !grad_x)) return e3c::bad("NULL device pointer");
  e3c::NormParams p{};
  p.a = *a;
  p.gc = a->channels / a->groups;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.gy = grad_y;
  p.gy_row = grad_y_row;
  p.gx = grad_x;
  p.gx_row = grad_x_row;
  p.gw = grad_weight;
  p.gb = grad_bias;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (grad_weight || grad_bias) {
    const dim3 grid((unsigned)a->channels);
    if (a->dtype == E3CONV_F32) hipLaunchKernelGGL(e3c::norm_bwd_w<float>, grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(e3c::norm_bwd_w<__bf16>, grid, dim3(256), 0, s, p);
  }
  if (a->num_rows > 0) {
    const dim3 grid((unsigned)((long)a->num_graphs * a->groups));
    if (a->dtype == E3CONV_F32) hipLaunchKernelGGL(e3c::norm_bwd_x<float>, grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(e3c::norm_bwd_x<__bf16>, grid, dim3(256), 0, s, p);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return e3c::api_hip_fail(err, "group norm backward launch");
  return e3c::api_ok();
}

}  // extern "C"
