// Root-mean-square norm of rows, or of each of their groups of channels, with a residual's
// addition, and its reverse pass (contract in e3conv.h).
//
// With s = x + residual and size channels a group,
//     rstd = 1 / sqrt(sum s^2 / size + eps),   y = weight s rstd,
// and with xhat = s rstd and dn = weight grad_y
//     grad_s = rstd (dn - xhat sum(dn xhat) / size) + grad_total,   grad_weight = sum grad_y xhat.
// A team of threads takes an item (a group of a row), each thread every team-th run of 16 bytes; the row stays
// in registers between its statistics and its result, so everything is read once and written once.  Memory
// bound: 100 000 rows of 512 channels in bf16, each of four heads by itself, take the kernel 33 us for 205 MB (6.1 TB/s, a
// stream copy's rate; 40 us a call among others), the reverse pass with a residual 73 us for 410 MB (5.6 TB/s) and
// 5 us for the join (76 us a call).  In the reverse pass a team takes many items, always of the same weights, and keeps
// its part of their gradient in registers; parts are joined within the work-group, then by a second launch, in a fixed
// order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <numeric>
#include <string>

#include "e3conv.h"
#include "kernels.h"
#include "row_units.h"

namespace e3c {
namespace {

using namespace rows;

constexpr int NT = 256;               // threads of a work-group
constexpr int kMaxSize = 16383, kMaxChannels = 65536;   // 2 NT threads hold 32 values each; the contract ends below 16 384
constexpr int kWide = 8192;           // groups beyond it take work-groups of 2 NT threads

struct RmsParams {
  e3conv_rms_norm_args a;
  int size;                           // channels of a group
  int units;                          // runs of V channels of a group
  int team, team_log2;                // threads of an item, a power of two
  Div by_groups, by_period;
  int items;                          // rows x groups
  int vec_weight;                     // the weight is 16-byte aligned
  void* y;
  long y_row;
  void* total;
  long total_row;
  float* rstd;
  const void* gy;
  long gy_row;
  const void* gt;
  long gt_row;
  void* gx;
  long gx_row;
  float* gw;
  // reverse pass: items of a team lie `stride` apart, a multiple of `residues`, so that all of them meet
  // the weights of group (first item) % residues
  int residues, used, stride, blocks;
  float* part;                        // (blocks used / residues, residues size)
  int part_rows;
};

// Sum over the threads of a team; every thread has it.  WAVES: those of the one team of a work-group, or 0 where
// the teams are parts of waves.
template <int WAVES>
__device__ __forceinline__ float team_sum(float v, int team, float* red) {
  if constexpr (WAVES > 0) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (red[0] + red[1]) + (red[2] + red[3]);
    return WAVES == 4 ? v : v + ((red[4] + red[5]) + (red[6] + red[7]));
  } else {
    for (int o = team >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
  }
}

// The weights of V channels from channel c of a row on.
template <int V>
__device__ __forceinline__ void weights(const RmsParams& p, int c, float (&w)[V]) {
  if (!p.a.weight) {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = 1.0f;
    return;
  }
  const int at = c - p.by_period.of(c) * p.by_period.d;
  if (V > 1 && p.vec_weight) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p.a.weight + at + i);
      w[i] = f.x;
      w[i + 1] = f.y;
      w[i + 2] = f.z;
      w[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = p.a.weight[at + i];
  }
}

constexpr int threads_of(int waves) { return waves == 8 ? 2 * NT : NT; }

// U: runs of a thread.  WAVES: as above.  A team takes items that meet the same weights, and the
// next one's loads are issued before this one is used: all of an item's together, the mask's byte too; runs
// beyond the group read its first, and what does not count is cleared afterwards.  (Not with 8 waves: the next item's
// loads would take the registers of the second work-group.)
template <class T, int V, int U, int WAVES>
__global__ void __launch_bounds__(threads_of(WAVES)) rms_norm(RmsParams p) {
  constexpr bool BIG = WAVES > 0, AHEAD = WAVES < 8;
  __shared__ float red[8];
  const e3conv_rms_norm_args& a = p.a;
  const int t = BIG ? threadIdx.x : threadIdx.x & (p.team - 1), mine = BIG ? 0 : threadIdx.x >> p.team_log2;
  const long first_item = (long)blockIdx.x * p.used + mine;
  if (mine >= p.used || first_item >= p.items) return;      // whole teams; a team that is a work-group meets at barriers
  float w[U][V];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int u = t + k * p.team, g = (int)(first_item % p.residues);
    weights<V>(p, g * p.size + (u < p.units ? u * V : 0), w[k]);
  }
  struct Item {
    typename Run<T, V>::type x[U], r[U];
    unsigned char mask;
  };
  const auto load = [&](long at, Item& to) {
    const int item = (int)at, row = p.by_groups.of(item), c0 = (item - row * a.groups) * p.size;
    const T* x = (const T*)a.x + row * a.x_row + c0;
    to.mask = a.row_mask ? a.row_mask[row] : 1;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * p.team;
      to.x[k] = read<T, V>(x + (u < p.units ? u * V : 0));
    }
    if (a.residual) {
      const T* res = (const T*)a.residual + row * a.residual_row + c0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = t + k * p.team;
        to.r[k] = read<T, V>(res + (u < p.units ? u * V : 0));
      }
    }
  };
  Item next;
  if (AHEAD) load(first_item, next);
  for (long at = first_item; at < p.items; at += p.stride) {
    Item now = next;
    if (!AHEAD) load(at, now);
    else if (at + p.stride < p.items) load(at + p.stride, next);
    const int item = (int)at, row = p.by_groups.of(item), c0 = (item - row * a.groups) * p.size;
    float s[U][V], sum = 0.0f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const bool on = now.mask && t + k * p.team < p.units;
      widen<T, V>(now.x[k], s[k]);
      if (a.residual) {
        float r[V];
        widen<T, V>(now.r[k], r);
#pragma unroll
        for (int i = 0; i < V; ++i) s[k][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[k][i] = on ? s[k][i] : 0.0f;
        sum = fmaf(s[k][i], s[k][i], sum);
      }
    }
    sum = team_sum<WAVES>(sum, p.team, red);
    const float rstd = 1.0f / sqrtf(sum / (float)p.size + a.eps);
    if (t == 0 && p.rstd) p.rstd[item] = rstd;
    T* y = (T*)p.y + row * p.y_row + c0;
    T* total = p.total ? (T*)p.total + row * p.total_row + c0 : nullptr;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * p.team;
      if (u >= p.units) break;
      if (total) store<T, V>(total + u * V, s[k]);
      float v[V];      // y from the unrounded sum
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = w[k][i] * (s[k][i] * rstd);
      store<T, V>(y + u * V, v);
    }
  }
}

template <class T, int V, int U, int WAVES>
__global__ void __launch_bounds__(threads_of(WAVES)) rms_norm_grad(RmsParams p) {
  constexpr bool BIG = WAVES > 0, AHEAD = WAVES < 8;
  __shared__ float red[8];
  __shared__ float parts[BIG ? 1 : NT * V * U];
  const e3conv_rms_norm_args& a = p.a;
  const int t = BIG ? threadIdx.x : threadIdx.x & (p.team - 1), mine = BIG ? 0 : threadIdx.x >> p.team_log2;
  const long first_item = (long)blockIdx.x * p.used + mine;
  float gw[U][V], w[U][V];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int u = t + k * p.team, g = (int)(first_item % p.residues);
    weights<V>(p, g * p.size + (u < p.units ? u * V : 0), w[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) gw[k][i] = 0.0f;
  }
  // an item's loads; the next one's are issued before this one is used
  struct Item {
    typename Run<T, V>::type x[U], g[U], t[U];
    float rstd;
    unsigned char mask;
  };
  const auto load = [&](long at, Item& to) {
    const int item = (int)at, row = p.by_groups.of(item), c0 = (item - row * a.groups) * p.size;
    const T *x = (const T*)a.x + row * a.x_row + c0, *g = (const T*)p.gy + row * p.gy_row + c0;
    to.mask = a.row_mask ? a.row_mask[row] : 1;
    to.rstd = p.rstd[item];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * p.team, e = u < p.units ? u * V : 0;
      to.x[k] = read<T, V>(x + e);
      to.g[k] = read<T, V>(g + e);
    }
    if (p.gt) {
      const T* gt = (const T*)p.gt + row * p.gt_row + c0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = t + k * p.team;
        to.t[k] = read<T, V>(gt + (u < p.units ? u * V : 0));
      }
    }
  };
  Item next;
  if (AHEAD && mine < p.used && first_item < p.items) load(first_item, next);
  if (mine < p.used)
    for (long at = first_item; at < p.items; at += p.stride) {
      Item now = next;
      if (!AHEAD) load(at, now);
      else if (at + p.stride < p.items) load(at + p.stride, next);
      const int item = (int)at, row = p.by_groups.of(item), c0 = (item - row * a.groups) * p.size;
      const float rstd = now.mask ? now.rstd : 0.0f;
      float xh[U][V], dn[U][V], dot = 0.0f;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool on = now.mask && t + k * p.team < p.units;
        float g[V];
        widen<T, V>(now.x[k], xh[k]);
        widen<T, V>(now.g[k], g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xh[k][i] = on ? xh[k][i] * rstd : 0.0f;
          g[i] = on ? g[i] : 0.0f;
          gw[k][i] = fmaf(g[i], xh[k][i], gw[k][i]);
          dn[k][i] = w[k][i] * g[i];
          dot = fmaf(dn[k][i], xh[k][i], dot);
        }
      }
      dot = team_sum<WAVES>(dot, p.team, red) / (float)p.size;
      T* gx = (T*)p.gx + row * p.gx_row + c0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = t + k * p.team;
        if (u >= p.units) break;
        float v[V];
        widen<T, V>(now.t[k], v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = rstd * fmaf(-xh[k][i], dot, dn[k][i]);
          v[i] = !now.mask ? 0.0f : p.gt ? v[i] + d : d;
        }
        store<T, V>(gx + u * V, v);
      }
    }
  if (!p.gw) return;
  // parts of the teams that meet the same weights, joined; a row of `size` values for each residue
  const int teams = BIG ? 1 : p.used;
  const long first = (long)blockIdx.x * p.part_rows;
  if constexpr (!BIG) {
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) parts[(mine * U + k) * p.team * V + i * p.team + t] = gw[k][i];
    __syncthreads();
    for (int e = threadIdx.x; e < p.part_rows * U * p.team * V; e += NT) {
      const int r = e / (U * p.team * V), j = e - r * (U * p.team * V);
      float v = 0.0f;
      for (int m = r; m < teams; m += p.part_rows) v += parts[m * (U * p.team * V) + j];
      const int k = j / (p.team * V), i = (j - k * (p.team * V)) / p.team, c = (j & (p.team - 1)) + k * p.team;
      if (c < p.units) p.part[(first + r) * p.size + c * V + i] = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * p.team;
      if (u < p.units)
#pragma unroll
        for (int i = 0; i < V; ++i) p.part[first * p.size + u * V + i] = gw[k][i];
    }
  }
}

// grad_weight[w] = the sum over the rows of `part` (width values each) of their values w, w + period, ...
// Sixteen columns to a work-group, sixteen threads each.
__global__ void __launch_bounds__(NT) rms_norm_join(const float* part, long rows, int width, int period, float* gw) {
  __shared__ float red[16][17];
  const int col = threadIdx.x & 15, lane = threadIdx.x >> 4, w = blockIdx.x * 16 + col;
  float v = 0.0f;
  if (w < period)
    for (int c = w; c < width; c += period)
#pragma unroll 8
      for (long r = lane; r < rows; r += 16) v += part[r * width + c];
  red[lane][col] = v;
  __syncthreads();
  if (threadIdx.x < 16 && w < period) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += red[i][col];
    gw[w] = v;
  }
}

// --------------------------------------------------------------- launches ---

int vector_width(const e3conv_rms_norm_args& a) { return a.dtype == E3CONV_F32 ? 4 : 8; }

// Teams: the threads of one wave or fewer up to 256 runs, else the work-group, of twice the threads beyond kWide channels
// (their values are 64 registers' worth and more in 256).
struct Shape {
  int units, team, team_log2, runs;
  bool big;
};
Shape shape_of(int size, int v) {
  Shape s{};
  s.units = (size + v - 1) / v;
  s.big = s.units > 256;
  while (!s.big && s.team_log2 < 6 && (1 << s.team_log2) < s.units) ++s.team_log2;
  if (s.big) s.team_log2 = size > kWide ? 9 : 8;
  s.team = 1 << s.team_log2;
  s.runs = (s.units + s.team - 1) / s.team;
  return s;
}

// How the reverse pass shares items among teams.
struct Sharing {
  int residues, used, part_rows;
  int64_t blocks;
};
Sharing sharing_of(const e3conv_rms_norm_args& a, const Shape& s, bool back) {
  Sharing h;
  const int size = a.channels / a.groups, teams = std::max(1, NT >> s.team_log2);
  h.residues = a.weight_channels / std::gcd(a.weight_channels, size);
  h.used = h.residues <= teams ? teams / h.residues * h.residues : teams;
  h.part_rows = std::min(h.residues, h.used);
  const int64_t items = a.num_rows * a.groups;
  // work-groups: their teams' number is a multiple of `residues`
  const int whole = h.residues <= teams ? 1 : h.residues / std::gcd(h.residues, teams);
  int64_t n = std::min<int64_t>((items + h.used - 1) / h.used, back ? 512 : 2048);
  h.blocks = (std::max<int64_t>(n, 1) + whole - 1) / whole * whole;
  return h;
}

size_t workspace_bytes(const e3conv_rms_norm_args& a) {
  // the element-wise form has the most parts a work-group; either may run
  size_t most = 0;
  for (int v : {1, vector_width(a)}) {
    const Sharing h = sharing_of(a, shape_of(a.channels / a.groups, v), true);
    most = std::max(most, (size_t)h.blocks * h.part_rows * (a.channels / a.groups) * sizeof(float));
  }
  return (most + 15) / 16 * 16;
}

template <class T, int V, int U, int WAVES>
hipError_t run(const RmsParams& p, bool back, hipStream_t s) {
  if (back) {
    hipLaunchKernelGGL((rms_norm_grad<T, V, U, WAVES>), dim3(p.blocks), dim3(threads_of(WAVES)), 0, s, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || !p.gw) return err;
    const long rows = (long)p.blocks * p.part_rows / p.residues;
    hipLaunchKernelGGL(rms_norm_join, dim3((p.a.weight_channels + 15) / 16), dim3(NT), 0, s, p.part, rows,
                       p.residues * p.size, p.a.weight_channels, p.gw);
  } else {
    hipLaunchKernelGGL((rms_norm<T, V, U, WAVES>), dim3(p.blocks), dim3(threads_of(WAVES)), 0, s, p);
  }
  return hipGetLastError();
}
template <class T, int V>
hipError_t by_runs(const RmsParams& p, const Shape& sh, bool back, hipStream_t s) {
  if (!sh.big) return sh.runs == 1 ? run<T, V, 1, 0>(p, back, s)
                    : sh.runs == 2 ? run<T, V, 2, 0>(p, back, s) : run<T, V, 4, 0>(p, back, s);
  if (sh.team > NT) return run<T, V, 32 / V, 8>(p, back, s);
  if (sh.runs <= 2) return run<T, V, 2, 4>(p, back, s);
  if constexpr (V == 8) {
    return run<T, V, 4, 4>(p, back, s);
  } else {
    if (sh.runs <= 4) return run<T, V, 4, 4>(p, back, s);
    if (V == 4 || sh.runs <= 8) return run<T, V, 8, 4>(p, back, s);
    return run<T, V, V == 1 ? 32 : 8, 4>(p, back, s);
  }
}

hipError_t launch(RmsParams p, bool back, bool vec, void* workspace, hipStream_t s) {
  const e3conv_rms_norm_args& a = p.a;
  const bool f32 = a.dtype == E3CONV_F32;
  const int v = vector_width(a);
  p.size = a.channels / a.groups;
  if (p.size % v != 0 || a.weight_channels % v != 0) vec = false;
  const Shape sh = shape_of(p.size, vec ? v : 1);
  p.units = sh.units;
  p.team = sh.team;
  p.team_log2 = sh.team_log2;
  p.by_groups = div_by(a.groups);
  p.by_period = div_by(a.weight_channels);
  p.items = (int)(a.num_rows * a.groups);
  p.vec_weight = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  const Sharing h = sharing_of(a, sh, back);
  p.residues = h.residues;
  p.used = h.used;
  p.blocks = (int)h.blocks;
  p.stride = (int)h.blocks * h.used;
  p.part_rows = h.part_rows;
  p.part = static_cast<float*>(workspace);
  if (f32) return vec ? by_runs<float, 4>(p, sh, back, s) : by_runs<float, 1>(p, sh, back, s);
  return vec ? by_runs<__bf16, 8>(p, sh, back, s) : by_runs<__bf16, 1>(p, sh, back, s);
}

e3conv_status bad(const char* what) { return api_fail(E3CONV_ERR_INVALID_ARGUMENT, what); }

e3conv_status check_sizes(const e3conv_rms_norm_args* a) {
  if (!a) return bad("args is NULL");
  if (a->dtype != E3CONV_F32 && a->dtype != E3CONV_BF16) return bad("bad dtype");
  if (a->num_rows < 0) return bad("negative size");
  if (a->channels < 1 || a->channels > kMaxChannels || a->groups < 1 || a->channels % a->groups != 0 ||
      a->channels / a->groups > kMaxSize)
    return bad("channels must be in [1, 65536] and a multiple of groups, with fewer than 16384 in a group");
  if (a->weight_channels < 1 || a->channels % a->weight_channels != 0)
    return bad("channels must be a multiple of weight_channels");
  if (a->num_rows >= (((int64_t)1 << 31) - ((int64_t)1 << 20)) / a->groups) return bad("sizes must fit int32 indices");
  if (!(a->eps > 0.0f) || !std::isfinite(a->eps)) return bad("eps must be positive");
  return E3CONV_OK;
}

e3conv_status check_args(const e3conv_rms_norm_args* a) {
  const e3conv_status st = check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (a->x_row < 0 || a->residual_row < 0) return bad("negative stride");
  if (a->num_rows > 0 && !a->x) return bad("NULL device pointer");
  return E3CONV_OK;
}

}  // namespace
}  // namespace e3c

extern "C" {

e3conv_status e3conv_rms_norm(const e3conv_rms_norm_args* a, void* y, int64_t y_row, void* total, int64_t total_row,
                              float* rstd, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (y_row < 0 || total_row < 0) return e3c::bad("negative stride");
  if (a->num_rows == 0) return e3c::api_ok();
  if (!y) return e3c::bad("NULL device pointer");
  if (y == total) return e3c::bad("y and total are one array");
  e3c::RmsParams p{};
  p.a = *a;
  p.y = y;
  p.y_row = y_row;
  p.total = total;
  p.total_row = total_row;
  p.rstd = rstd;
  const int v = e3c::vector_width(*a);
  const bool vec = e3c::aligned(a->x, a->x_row, v) && e3c::aligned(y, y_row, v) &&
                   (!a->residual || e3c::aligned(a->residual, a->residual_row, v)) &&
                   (!total || e3c::aligned(total, total_row, v));
  const hipError_t err = e3c::launch(p, false, vec, nullptr, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) return e3c::api_hip_fail(err, "rms norm launch");
  return e3c::api_ok();
}

e3conv_status e3conv_rms_norm_workspace_size(const e3conv_rms_norm_args* a, size_t* bytes) {
  const e3conv_status st = e3c::check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (!bytes) return e3c::bad("bytes is NULL");
  *bytes = e3c::workspace_bytes(*a);
  return e3c::api_ok();
}

e3conv_status e3conv_rms_norm_backward(const e3conv_rms_norm_args* a, const float* rstd, const void* grad_y,
                                       int64_t grad_y_row, const void* grad_total, int64_t grad_total_row,
                                       void* grad_x, int64_t grad_x_row, float* grad_weight, void* workspace,
                                       size_t bytes, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (a->residual) return e3c::bad("the reverse pass takes the sum as x, and no residual");
  if (grad_y_row < 0 || grad_total_row < 0 || grad_x_row < 0) return e3c::bad("negative stride");
  if (a->num_rows == 0) {
    if (!grad_weight) return e3c::api_ok();
    const hipError_t e = e3c::launch_fill_zero(grad_weight, (size_t)a->weight_channels, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? e3c::api_ok() : e3c::api_hip_fail(e, "fill launch");
  }
  if (!rstd || !grad_y || !grad_x) return e3c::bad("NULL device pointer");
  const size_t need = grad_weight ? e3c::workspace_bytes(*a) : 0;
  if (bytes < need || (need > 0 && !workspace))
    return e3c::api_fail(E3CONV_ERR_WORKSPACE, "rms norm backward needs " + std::to_string(need) + " bytes");
  e3c::RmsParams p{};
  p.a = *a;
  p.rstd = const_cast<float*>(rstd);
  p.gy = grad_y;
  p.gy_row = grad_y_row;
  p.gt = grad_total;
  p.gt_row = grad_total_row;
  p.gx = grad_x;
  p.gx_row = grad_x_row;
  p.gw = grad_weight;
  const int v = e3c::vector_width(*a);
  const bool vec = e3c::aligned(a->x, a->x_row, v) && e3c::aligned(grad_y, grad_y_row, v) &&
                   e3c::aligned(grad_x, grad_x_row, v) &&
                   (!grad_total || e3c::aligned(grad_total, grad_total_row, v));
  const hipError_t err = e3c::launch(p, true, vec, workspace, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) return e3c::api_hip_fail(err, "rms norm backward launch");
  return e3c::api_ok();
}

}  // extern "C"
