// Rotary positions over several axes, and their reverse pass (contract in e3conv.h).
//
// Pair p of every head of row i is turned by angle[i, p] = sum_a positions[i, a] waves[p, a]:
//     (u, v) -> (u cos - v sin, u sin + v cos).
// The reverse pass turns the gradient back, (gu, gv); with d_angle[i, p] = sum over heads of (u gv - v gu),
//     grad_positions[i, a] = sum_p d_angle waves[p, a],   grad_waves[p, a] = sum_i d_angle positions[i, a].
// A work-group takes tiles of whole rows.  The tile's cosines and sines are formed once for all heads, the
// angle in 64 bits and in turns (of a position of 10^4 wave lengths 32 bits leave three digits), and stand in
// LDS; the rows then pass through registers in runs of 16 bytes, whatever their heads.  In the reverse pass
// each pair's d_angle goes to LDS and is summed over the heads in order.  Memory bound: 100 000 rows of 12 heads of 64
// in bf16 take the kernel 49 us for 307 MB (6.2 TB/s, the rate of a stream copy; 55.6 us a call among others); the reverse
// pass of 20 000 rows of 8 heads of 32 in fp32 15 us for 62 MB, where the chain of a work-group's few tiles shows, and
// 4 us to join grad_waves (18.3 us a call).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "e3conv.h"
#include "kernels.h"
#include "row_units.h"

namespace e3c {
namespace {

using namespace rows;

constexpr int NT = 256;               // threads of a work-group
constexpr int kMaxDim = 256, kMaxAxes = 4;
constexpr int kTile = 8192;           // elements of a tile, or one row's: the forward kernel's loop takes any number of them
constexpr int kGradTile = 4096;       // the same of the reverse pass, which keeps half as many values in LDS: a row's heads
                                      // go in parts if they have more
constexpr int kTileRows = 128;        // a tile has at most NT angles: each thread forms one
constexpr int kTable = 512;           // and its rows in the table are whole runs: 128 rows of 4 at most, or 256 + 85 3

struct RotaryParams {
  e3conv_rotary_args a;
  int units;                          // runs of a head: of V elements, or turned pairs of V and then V elements
  int turning;                        // units that hold pairs
  int stride;                         // pairs of a row of the table, whole runs
  int tile_rows;
  int tile_heads;                     // reverse pass
  int tiles, blocks;
  Div by_units, by_heads, by_pairs, by_axes, by_values;
  float sign;
  unsigned x_row, x_head;             // strides in elements
  void* out;
  unsigned out_row, out_head;
  const void* g;                      // reverse pass: the gradient, turned back
  unsigned g_row, g_head;
  float* gp;
  float* gw;
  double* part;                       // (blocks, pairs axes)
};

// Where a unit of a row's head lies: its first elements, its second ones, and its first pair.
template <int V, bool ADJACENT>
struct Unit {
  int u, v, pair;
  bool turns;
  __device__ __forceinline__ Unit(const RotaryParams& p, int k) {
    turns = k < p.turning;
    if constexpr (ADJACENT && V > 1) {            // V / 2 pairs in a run
      u = v = k * V;
      pair = k * (V / 2);
    } else if (ADJACENT) {                        // one pair
      u = turns ? 2 * k : k + p.turning;
      v = u + 1;
      pair = k;
    } else {
      u = turns ? k * V : k * V + p.turning * V;  // beyond the pairs' second halves
      v = u + p.a.pairs;
      pair = k * V;
    }
  }
};

// cos and sin of 2 pi t, |t| <= 1/2, within 1.5 2^-24 and within 2 2^-24 of their own size.  The nearest quarter turn leaves
// |x| <= pi / 4 in 64 bits, of which 32 go on with the rest, lo.  (The rounding of t to 32 bits would be 2^-26 of a turn,
// 1.6 2^-24 of the angle, for all heads of a row alike, whose sums make the angles' gradients; the series in 64 bits
// too gives no digit more and costs heads that are alone in their rows 8 % in place of 3.)  The Taylor series to x^9
// and x^10 err by less than 2^-28; the last sum adds a term of at most 0.31 to x or 1.
__device__ __forceinline__ float2 cos_sin(double t) {
  const double quarter = rint(4.0 * t), wide = 6.283185307179586477 * fma(-0.25, quarter, t);
  const float x = (float)wide, lo = (float)(wide - (double)x), y = x * x;
  float s = fmaf(y, 1.0f / 362880, -1.0f / 5040), c = fmaf(y, -1.0f / 3628800, 1.0f / 40320);
  s = fmaf(y, s, 1.0f / 120);
  c = fmaf(y, c, -1.0f / 720);
  s = fmaf(y, s, -1.0f / 6);
  c = fmaf(y, c, 1.0f / 24);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, -x * lo);
  s = x + fmaf(x * y, s, fmaf(lo, c, lo));
  c = 1.0f + c;
  const int q = (int)quarter;
  const float a = q & 1 ? s : c, b = q & 1 ? c : s;
  return make_float2(((q + 1) & 2) ? -a : a, (q & 2) ? -b : b);
}

// The cosine and sine that this thread forms for the tile.  begin() starts its loads, ahead of the rows' own (loads
// arrive in order), all of them without a branch; finish() leaves it in LDS.
struct Angle {
  float x[kMaxAxes], w[kMaxAxes];
  unsigned char live;
  int r, k;
  __device__ __forceinline__ void begin(const RotaryParams& p, long row0, int nrows) {
    const e3conv_rotary_args& a = p.a;
    const int e = min((int)threadIdx.x, nrows * a.pairs - 1);
    r = p.by_pairs.of(e);
    k = e - r * a.pairs;
    const float *at = a.positions + (row0 + r) * a.position_row, *wave = a.waves + k * a.axes;
    live = a.row_mask ? a.row_mask[row0 + r] : 1;
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i) {
      const int j = min(i, a.axes - 1);
      x[i] = at[j];
      w[i] = wave[j];
    }
  }
  // lives: which rows count.
  __device__ __forceinline__ void finish(const RotaryParams& p, int nrows, float2* table, unsigned char* lives) const {
    const e3conv_rotary_args& a = p.a;
    double angle = 0.0;
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i) angle = fma((double)x[i], i < a.axes ? (double)w[i] : 0.0, angle);
    const double turns = angle * 0.15915494309189533577;
    float2 cs = cos_sin(turns - rint(turns));
    cs.y *= p.sign;
    if ((int)threadIdx.x < nrows * a.pairs) {
      // a masked row's position may be anything
      table[r * p.stride + k] = live ? cs : make_float2(1.0f, 0.0f);
      if (k == 0) lives[r] = live;
    }
  }
};

// A unit's elements in registers.
template <class T, int V, bool ADJACENT>
struct Held {
  typename Run<T, V>::type a, b;
  static constexpr bool TWO = !ADJACENT || V == 1;     // second elements of the pairs apart from the first
  __device__ __forceinline__ void load(const T* head, const Unit<V, ADJACENT>& at) {
    a = read<T, V>(head + at.u);
    if (TWO && at.turns) b = read<T, V>(head + at.v);
  }
  __device__ __forceinline__ void clear() {
    a = typename Run<T, V>::type{};
    b = typename Run<T, V>::type{};
  }
};

// Turns the pairs of a unit: x holds its run, or x the first elements of its pairs and y the second ones.  cs: its row
// of the table.
template <int V, bool ADJACENT>
__device__ __forceinline__ void turn(const float2* cs, const RotaryParams& p, const Unit<V, ADJACENT>& at, float (&x)[V],
                                     float (&y)[V]) {
  if constexpr (ADJACENT && V > 1) {
    float4 t[V / 4];
    const float4* from = reinterpret_cast<const float4*>(cs + (at.pair < p.stride ? at.pair : 0));
#pragma unroll
    for (int i = 0; i < V / 4; ++i) t[i] = from[i];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {            // chosen, not branched around: a run may end beyond the pairs
      const float c = i & 1 ? t[i / 2].z : t[i / 2].x, s = i & 1 ? t[i / 2].w : t[i / 2].y;
      const float u = x[2 * i], v = x[2 * i + 1], a = fmaf(u, c, -(v * s)), b = fmaf(u, s, v * c);
      const bool on = at.pair + i < p.a.pairs;
      x[2 * i] = on ? a : u;
      x[2 * i + 1] = on ? b : v;
    }
  } else if (at.turns) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 t = cs[at.pair + i];
      const float u = x[i], v = y[i];
      x[i] = fmaf(u, t.x, -(v * t.y));
      y[i] = fmaf(u, t.y, v * t.x);
    }
  }
}

// Row r and head h of a tensor of which `first` is the tile's first row.
template <class T>
__device__ __forceinline__ T* place(T* first, unsigned row, unsigned head, int r, int h) {
  return first + ((uint64_t)row * (unsigned)r + (uint64_t)head * (unsigned)h);
}

template <class T, int V, bool ADJACENT>
__global__ void __launch_bounds__(NT) rotary(RotaryParams p) {
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  __shared__ unsigned char live[kTileRows];
  const e3conv_rotary_args& a = p.a;
  const long tile = block_index();
  if (tile >= p.tiles) return;
  const long row0 = tile * p.tile_rows;
  const int nrows = (int)min((long)p.tile_rows, a.num_rows - row0);
  const T* const from = (const T*)a.x + row0 * p.x_row;
  T* const to = (T*)p.out + row0 * p.out_row;
  const int n = nrows * a.heads * p.units;
  constexpr int N = 4;
  Angle angle;
  angle.begin(p, row0, nrows);
  for (int e0 = threadIdx.x; e0 - (int)threadIdx.x < n; e0 += N * NT) {
    Held<T, V, ADJACENT> held[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = min(e0 + i * NT, n - 1), rh = p.by_units.of(e), r = p.by_heads.of(rh);
      held[i].load(place(from, p.x_row, p.x_head, r, rh - r * a.heads), Unit<V, ADJACENT>(p, e - rh * p.units));
    }
    if (e0 == (int)threadIdx.x) {                // while the first loads are on their way
      angle.finish(p, nrows, table, live);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = e0 + i * NT;
      if (e >= n) break;
      const int rh = p.by_units.of(e), r = p.by_heads.of(rh);
      const Unit<V, ADJACENT> at(p, e - rh * p.units);
      if (!live[r]) held[i].clear();
      float x[V], y[V];
      widen<T, V>(held[i].a, x);
      widen<T, V>(held[i].b, y);
      turn<V, ADJACENT>(table + r * p.stride, p, at, x, y);
      T* head = place(to, p.out_row, p.out_head, r, rh - r * a.heads);
      store<T, V>(head + at.u, x);
      if (Held<T, V, ADJACENT>::TWO && at.turns) store<T, V>(head + at.v, y);
    }
  }
}

// With the gradients of positions or waves: turns back g and forms d_angle.  A work-group takes every
// blocks-th tile and keeps its part of grad_waves: a thread has one value of it (or two) and one of the rows in turn.
template <class T, int V, bool ADJACENT>
__global__ void __launch_bounds__(NT) rotary_grad(RotaryParams p) {
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  __shared__ float angles[kGradTile / 2];      // (row, head, pair)
  __shared__ float sums[NT];                   // (row, pair), over the heads
  __shared__ float waves[kMaxDim / 2 * kMaxAxes], places[kTileRows * kMaxAxes];
  __shared__ unsigned char live[kTileRows];
  const e3conv_rotary_args& a = p.a;
  constexpr int N = 2, W = kMaxDim / 2 * kMaxAxes / NT;
  const int values = a.pairs * a.axes;
  for (int e = threadIdx.x; e < values; e += NT) waves[e] = a.waves[e];
  const int lanes = values <= NT ? p.by_values.of(NT) : 1;                  // rows in turn for each value
  const int lane = values <= NT ? p.by_values.of(threadIdx.x) : 0;
  double gw[W];
#pragma unroll
  for (int i = 0; i < W; ++i) gw[i] = 0.0;
  for (long tile = blockIdx.x; tile < p.tiles; tile += p.blocks) {
    const long row0 = tile * p.tile_rows;
    const int nrows = (int)min((long)p.tile_rows, a.num_rows - row0);
    const int sum_r = p.by_pairs.of(threadIdx.x), sum_k = threadIdx.x - sum_r * a.pairs;   // this thread's (row, pair)
    float sum = 0.0f;
    Angle angle;
    angle.begin(p, row0, nrows);
    for (int h0 = 0; h0 < a.heads; h0 += p.tile_heads) {      // more than one part: the tile is one row
      const int heads = min(p.tile_heads, a.heads - h0), n = nrows * heads * p.units;
      for (int e0 = threadIdx.x; e0 - (int)threadIdx.x < n; e0 += N * NT) {
        Held<T, V, ADJACENT> hg[N], hx[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int e = min(e0 + i * NT, n - 1), rh = p.by_units.of(e), r = nrows == 1 ? 0 : p.by_heads.of(rh);
          const int h = h0 + rh - r * heads;
          const Unit<V, ADJACENT> at(p, e - rh * p.units);
          hg[i].load(place((const T*)p.g + row0 * p.g_row, p.g_row, p.g_head, r, h), at);
          hx[i].load(place((const T*)a.x + row0 * p.x_row, p.x_row, p.x_head, r, h), at);
        }
        if (h0 == 0 && e0 == (int)threadIdx.x) {              // while the first loads are on their way
          __syncthreads();                                    // the last tile's sums and places are read
          angle.finish(p, nrows, table, live);
          for (int e = threadIdx.x; e < nrows * a.axes; e += NT) {
            const int r = p.by_axes.of(e);
            places[e] = a.positions[(row0 + r) * a.position_row + (e - r * a.axes)];
          }
          __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int e = e0 + i * NT;
          if (e >= n) break;
          const int rh = p.by_units.of(e), r = nrows == 1 ? 0 : p.by_heads.of(rh), h = rh - r * heads;
          const Unit<V, ADJACENT> at(p, e - rh * p.units);
          if (!live[r]) {
            hg[i].clear();
            hx[i].clear();
          }
          float gu[V], gv[V], u[V], v[V];
          widen<T, V>(hg[i].a, gu);
          widen<T, V>(hg[i].b, gv);
          widen<T, V>(hx[i].a, u);
          widen<T, V>(hx[i].b, v);
          turn<V, ADJACENT>(table + r * p.stride, p, at, gu, gv);
          T* to = place((T*)p.out + row0 * p.out_row, p.out_row, p.out_head, r, h0 + h);
          store<T, V>(to + at.u, gu);
          if (Held<T, V, ADJACENT>::TWO && at.turns) store<T, V>(to + at.v, gv);
          float* d = angles + (r * heads + h) * a.pairs + at.pair;
          if constexpr (ADJACENT && V > 1) {
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
              if (at.pair + j < a.pairs) d[j] = fmaf(u[2 * j], gu[2 * j + 1], -(u[2 * j + 1] * gu[2 * j]));
          } else if (at.turns) {
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = fmaf(u[j], gv[j], -(v[j] * gu[j]));
          }
        }
      }
      __syncthreads();
      if (sum_r < nrows)
#pragma unroll 4
        for (int h = 0; h < heads; ++h) sum += angles[(sum_r * heads + h) * a.pairs + sum_k];
      if (h0 + p.tile_heads < a.heads) __syncthreads();
    }
    sums[threadIdx.x] = sum;
    __syncthreads();
    if (p.gp)
      for (int e = threadIdx.x; e < nrows * a.axes; e += NT) {
        const int r = p.by_axes.of(e), x = e - r * a.axes;
        float s = 0.0f;
#pragma unroll 4
        for (int k = 0; k < a.pairs; ++k) s = fmaf(sums[r * a.pairs + k], waves[k * a.axes + x], s);
        p.gp[row0 * a.axes + e] = s;
      }
    if (p.gw && lane < lanes) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int e = threadIdx.x - lane * values + i * NT;
        if (e >= values) break;
        const int k = p.by_axes.of(e), x = e - k * a.axes;
#pragma unroll 4
        for (int r = lane; r < nrows; r += lanes) {
          const float d = sums[r * a.pairs + k];
          // a masked row's position may be anything
          if (live[r]) gw[i] = fma((double)d, (double)places[r * a.axes + x], gw[i]);
        }
      }
    }
  }
  if (!p.gw) return;
  if (lanes > 1) {                             // the parts of a value's rows, in order
    double* parts = reinterpret_cast<double*>(table);
    __syncthreads();
    parts[threadIdx.x] = gw[0];
    __syncthreads();
    if (threadIdx.x < (unsigned)values) {
      double v = parts[threadIdx.x];
      for (int i = 1; i < lanes; ++i) v += parts[threadIdx.x + i * values];
      p.part[(long)blockIdx.x * values + threadIdx.x] = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int e = threadIdx.x + i * NT;
    if (e < values) p.part[(long)blockIdx.x * values + e] = gw[i];
  }
}

// grad_waves: the sum of the work-groups' parts.  Eight values to a work-group, whole 64-byte lines of the parts, and
// 32 threads for each.
__global__ void __launch_bounds__(NT) rotary_join(const double* part, int blocks, int n, float* gw) {
  __shared__ double red[32][9];
  const int col = threadIdx.x & 7, lane = threadIdx.x >> 3, at = blockIdx.x * 8 + col;
  double v = 0.0;
  if (at < n)
#pragma unroll 8
    for (int b = lane; b < blocks; b += 32) v += part[(long)b * n + at];
  red[lane][col] = v;
  __syncthreads();
  if (threadIdx.x < 8 && at < n) {
    v = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += red[i][col];
    gw[at] = (float)v;
  }
}

// --------------------------------------------------------------- launches ---

// Rows of a tile: about four tiles to a compute unit, as far as the angles' threads and LDS have room.
void tiles_of(const e3conv_rotary_args& a, bool grad, RotaryParams& p) {
  const int most = grad ? kGradTile : kTile, width = a.heads * a.dim;
  p.tile_heads = std::min<int>(a.heads, std::max(1, most / a.dim));
  int64_t rows = (a.num_rows + 1023) / 1024;
  rows = std::min<int64_t>(rows, std::min({most / width, NT / a.pairs, kTileRows}));
  p.tile_rows = (int)std::max<int64_t>(rows, 1);
  p.tiles = (int)((a.num_rows + p.tile_rows - 1) / p.tile_rows);
  p.blocks = std::min(p.tiles, 1024);
}

template <class T, int V, bool ADJACENT>
hipError_t run(const RotaryParams& p, hipStream_t s) {
  if (!p.gp && !p.gw) {
    hipLaunchKernelGGL((rotary<T, V, ADJACENT>), grid_of(p.tiles), dim3(NT), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((rotary_grad<T, V, ADJACENT>), dim3(p.blocks), dim3(NT), 0, s, p);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.gw) return err;
  const int n = p.a.pairs * p.a.axes;
  hipLaunchKernelGGL(rotary_join, dim3((n + 7) / 8), dim3(NT), 0, s, p.part, p.blocks, n, p.gw);
  return hipGetLastError();
}

// vec: rows and heads of all tensors are 16-byte aligned.
hipError_t launch(RotaryParams p, bool vec, hipStream_t s) {
  const e3conv_rotary_args& a = p.a;
  const bool f32 = a.dtype == E3CONV_F32, adjacent = a.layout == E3CONV_ROTARY_ADJACENT;
  const int v = f32 ? 4 : 8;
  p.x_row = (unsigned)a.x_row;
  p.x_head = (unsigned)a.x_head;
  // whole runs, and in halves no run that holds both pairs and elements beyond them
  vec = vec && a.dim % v == 0 && (adjacent || a.pairs % v == 0);
  const int n = vec ? v : 1;
  if (adjacent && vec) {
    p.units = a.dim / n;
    p.turning = p.units;
  } else {
    p.turning = a.pairs / n;
    p.units = p.turning + (a.dim - 2 * a.pairs) / n;
  }
  tiles_of(a, p.gp || p.gw, p);
  const int whole = adjacent && vec ? v / 2 : 1;
  p.stride = (a.pairs + whole - 1) / whole * whole;
  p.by_units = div_by(p.units);
  p.by_heads = div_by(a.heads);
  p.by_pairs = div_by(a.pairs);
  p.by_axes = div_by(a.axes);
  p.by_values = div_by(a.pairs * a.axes);
  if (f32) {
    if (!vec) return adjacent ? run<float, 1, true>(p, s) : run<float, 1, false>(p, s);
    return adjacent ? run<float, 4, true>(p, s) : run<float, 4, false>(p, s);
  }
  if (!vec) return adjacent ? run<__bf16, 1, true>(p, s) : run<__bf16, 1, false>(p, s);
  return adjacent ? run<__bf16, 8, true>(p, s) : run<__bf16, 8, false>(p, s);
}

size_t workspace_bytes(const e3conv_rotary_args& a) {
  RotaryParams p{};
  tiles_of(a, true, p);
  return ((size_t)p.blocks * a.pairs * a.axes * sizeof(double) + 15) / 16 * 16;
}

// Row and head strides are kept in 32 bits.
bool strides(int64_t row, int64_t head) { return row >= 0 && row <= 0xffffffffL && head >= 0 && head <= 0xffffffffL; }
constexpr const char* kStrides = "strides must be in [0, 2^32)";

bool aligned(const void* p, int64_t row, int64_t head, int dtype) {
  const int v = dtype == E3CONV_F32 ? 4 : 8;
  return rows::aligned(p, row, v) && head % v == 0;
}

e3conv_status bad(const char* what) { return api_fail(E3CONV_ERR_INVALID_ARGUMENT, what); }

e3conv_status check_sizes(const e3conv_rotary_args* a) {
  if (!a) return bad("args is NULL");
  if (a->dtype != E3CONV_F32 && a->dtype != E3CONV_BF16) return bad("bad dtype");
  if (a->layout != E3CONV_ROTARY_ADJACENT && a->layout != E3CONV_ROTARY_HALVES) return bad("unknown layout");
  if (a->num_rows < 0) return bad("negative size");
  if (a->dim < 1 || a->dim > kMaxDim) return bad("dim must be in [1, 256]");
  if (a->heads < 1 || a->heads > 65536) return bad("heads must be in [1, 65536]");
  if (a->pairs < 1 || a->pairs > a->dim / 2) return bad("pairs must be in [1, dim / 2]");
  if (a->axes < 1 || a->axes > kMaxAxes) return bad("axes must be in [1, 4]");
  if (a->num_rows >= ((int64_t)1 << 31) - ((int64_t)1 << 20)) return bad("sizes must fit int32 indices");
  return E3CONV_OK;
}

e3conv_status check_args(const e3conv_rotary_args* a) {
  const e3conv_status st = check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (!strides(a->x_row, a->x_head)) return bad(kStrides);
  if (a->position_row < 0) return bad("negative stride");
  if (!a->waves) return bad("NULL device pointer");
  if (a->num_rows > 0 && (!a->x || !a->positions)) return bad("NULL device pointer");
  return E3CONV_OK;
}

}  // namespace
}  // namespace e3c

extern "C" {

e3conv_status e3conv_rotary(const e3conv_rotary_args* a, void* out, int64_t out_row, int64_t out_head, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (!e3c::strides(out_row, out_head)) return e3c::bad(e3c::kStrides);
  if (a->num_rows == 0) return e3c::api_ok();
  if (!out) return e3c::bad("NULL device pointer");
  e3c::RotaryParams p{};
  p.a = *a;
  p.sign = 1.0f;
  p.out = out;
  p.out_row = (unsigned)out_row;
  p.out_head = (unsigned)out_head;
  const bool vec = e3c::aligned(a->x, a->x_row, a->x_head, a->dtype) && e3c::aligned(out, out_row, out_head, a->dtype);
  const hipError_t err = e3c::launch(p, vec, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) return e3c::api_hip_fail(err, "rotary launch");
  return e3c::api_ok();
}

e3conv_status e3conv_rotary_workspace_size(const e3conv_rotary_args* a, size_t* bytes) {
  const e3conv_status st = e3c::check_sizes(a);
  if (st != E3CONV_OK) return st;
  if (!bytes) return e3c::bad("bytes is NULL");
  *bytes = e3c::workspace_bytes(*a);
  return e3c::api_ok();
}

e3conv_status e3conv_rotary_backward(const e3conv_rotary_args* a, const void* grad_out, int64_t grad_out_row,
                                     int64_t grad_out_head, void* grad_x, int64_t grad_x_row, int64_t grad_x_head,
                                     float* grad_positions, float* grad_waves, void* workspace, size_t bytes,
                                     void* stream) {
  const bool angles = grad_positions || grad_waves;
  e3conv_rotary_args args = a ? *a : e3conv_rotary_args{};
  if (a && !angles && !args.x) args.x = grad_out;      // the features enter the angles' gradients alone
  const e3conv_status st = e3c::check_args(a ? &args : nullptr);
  if (st != E3CONV_OK) return st;
  if (!e3c::strides(grad_out_row, grad_out_head) || !e3c::strides(grad_x_row, grad_x_head)) return e3c::bad(e3c::kStrides);
  if (a->num_rows == 0) {
    if (!grad_waves) return e3c::api_ok();
    const hipError_t e = e3c::launch_fill_zero(grad_waves, (size_t)a->pairs * a->axes, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? e3c::api_ok() : e3c::api_hip_fail(e, "fill launch");
  }
  if (!grad_out || !grad_x) return e3c::bad("NULL device pointer");
  const size_t need = grad_waves ? e3c::workspace_bytes(*a) : 0;
  if (bytes < need || (need > 0 && !workspace))
    return e3c::api_fail(E3CONV_ERR_WORKSPACE, "rotary backward needs " + std::to_string(need) + " bytes");
  e3c::RotaryParams p{};
  p.a = args;
  p.sign = -1.0f;
  p.out = grad_x;
  p.out_row = (unsigned)grad_x_row;
  p.out_head = (unsigned)grad_x_head;
  bool vec = e3c::aligned(grad_out, grad_out_row, grad_out_head, a->dtype) &&
             e3c::aligned(grad_x, grad_x_row, grad_x_head, a->dtype);
  if (angles) {
    vec = vec && e3c::aligned(a->x, a->x_row, a->x_head, a->dtype);
    p.g = grad_out;
    p.g_row = (unsigned)grad_out_row;
    p.g_head = (unsigned)grad_out_head;
    p.gp = grad_positions;
    p.gw = grad_waves;
    p.part = static_cast<double*>(workspace);
  } else {                                             // the forward kernel turns grad_out back
    p.a.x = grad_out;
    p.a.x_row = grad_out_row;
    p.a.x_head = grad_out_head;
  }
  const hipError_t err = e3c::launch(p, vec, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) return e3c::api_hip_fail(err, "rotary backward launch");
  return e3c::api_ok();
}

}  // extern "C"
