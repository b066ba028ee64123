// Group norm with an activation over the rows of each graph, channels last, and its
// reverse pass (contract in e3conv.h).
//
// The rows of a graph are cut into chunks of p.chunk rows, one work-group each; a thread
// keeps one run of V channels (16 bytes) and strides over the rows, so loads are whole
// lines and per-channel values stay in registers.  A graph of one chunk is finished by the
// work-group that read it, its rows still in cache; graphs of more chunks take further
// launches:
//   sums    per chunk and channel: mean and squared deviations (forward), or
//           sum dz and sum dz xhat (reverse), to the workspace;
//   finish  per graph and group: mean and rstd, or the two means of the reverse pass,
//           from its chunks in chunk order (where graphs have few chunks, every
//           work-group of the next launch does this for its graph instead);
//   apply   per chunk: the rows; and in the reverse pass the weight and bias gradients.
// Variances are squared deviations from the mean of the rows before, joined by counts and means
// (Chan, Golub and LeVeque 1979), so neither a mean far from zero nor an outlying row costs digits.
// Memory bound: the rows are read twice and written once where a graph has more than one
// chunk (the second time from cache where the tensor fits it), else once and once: 1M rows of
// 64 channels bf16 in 84 us, 128 MB read in 24 us, read again and written in 52.  Calls of some MB are bound by
// the latency of a work-group (finding its graph, constants, a few rows, the sums) and the
// launches: reverse pass of 20 000 x 128 fp32 in 19 us, 100 000 x 64 bf16 in 29 us.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "e3conv.h"
#include "kernels.h"

namespace e3c {
namespace {

constexpr int kMaxChannels = 4096;
constexpr int NT = 256;            // threads of a work-group

// n / d for 0 <= n < 2^31 by a product: ceil(2^(31 + l) / d) with 2^l >= d.  The runtime divisions
// of a work-group's start cost as much as its loads where a chunk is a few rows a thread.
struct Div {
  int d;
  unsigned magic;
  int shift;
  __device__ __forceinline__ int of(int n) const { return d == 1 ? n : (int)(__umulhi((unsigned)n, magic) >> shift); }
};
Div div_by(int d) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  return {d, l > 0 ? (unsigned)((((uint64_t)1 << (31 + l)) + d - 1) / d) : 0, l > 0 ? l - 1 : 0};
}

struct NormParams {
  e3conv_group_norm_args a;
  int gc;                          // channels of a group
  int units;                       // runs of V channels in a row
  Div by_gc, by_width;             // by gc, and by min(units, NT)
  int chunk_log2, chunk;           // rows of a work-group, a power of two
  int slots;                       // chunk slots: rows / chunk + graphs
  int inline_finish;               // 1: finish within apply
  int vec_affine;                  // weight and bias are 16-byte aligned
  void* y;
  long y_row;
  float *mean, *rstd;
  const void* gy;
  long gy_row;
  void* gx;
  long gx_row;
  float *gw, *gb;
  float2* sums;                    // (slots, channels) of the chunks
  float* counts;                   // (slots) counted rows
  float2* stats;                   // (graphs, groups): mean and rstd, or the reverse pass's means
};

// ------------------------------------------------------------- work-groups ---

// n work-groups for each of the columns.  A launch takes less than 2^32 threads along an axis, so
// more than 2^20 work-groups go on along z.
constexpr unsigned kAlongX = 1u << 20;
dim3 grid_of(int64_t n, unsigned columns) {
  if (n <= kAlongX) return dim3((unsigned)n, columns);
  return dim3(kAlongX, columns, (unsigned)((n + kAlongX - 1) / kAlongX));
}
// Which of the n this one is; there may be some more.
__device__ __forceinline__ unsigned block_index() { return blockIdx.z * kAlongX + blockIdx.x; }

// ------------------------------------------------------------------ graphs ---

__device__ __forceinline__ int clamp_row(int v, long n) { return v < 0 ? 0 : (v > n ? (int)n : v); }
__device__ __forceinline__ int offset(const NormParams& p, int g) {
  return clamp_row(p.a.row_ptr[g], p.a.num_rows);
}

// Chunks of graph g take the slots first / chunk + g and on, first being its first row:
// enough for ceil(rows / chunk) of them, and one at least.
__device__ __forceinline__ int first_slot(const NormParams& p, int g) { return (offset(p, g) >> p.chunk_log2) + g; }

// The chunk of a slot: rows [begin, end) of graph g.
struct Chunk {
  int g, begin, end;
  bool first;      // the graph's first chunk
  bool only;       // and its only one
  bool none;       // a slot without a chunk
};
// The graph of a slot is the last whose first slot is not beyond it; 256 offsets are tried at a time.
__device__ __forceinline__ Chunk chunk_of(const NormParams& p, int slot) {
  const int lane = threadIdx.x & 63;
  int lo = 0, count = p.a.num_graphs;
  while (count > 1) {
    const int step = (count + 255) >> 8;
    int at[4], hits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) at[k] = p.a.row_ptr[lo + min((4 * lane + k) * step, count - 1)];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = (4 * lane + k) * step;
      hits += __popcll(__ballot(i < count && (clamp_row(at[k], p.a.num_rows) >> p.chunk_log2) + lo + i <= slot));
    }
    hits = max(hits, 1);
    lo += (hits - 1) * step;
    count = min(step, count - (hits - 1) * step);
  }
  Chunk c;
  c.g = __builtin_amdgcn_readfirstlane(lo);
  const int r0 = offset(p, c.g), r1 = max(r0, offset(p, c.g + 1));
  const int k = slot - ((r0 >> p.chunk_log2) + c.g);
  c.first = k == 0;
  c.only = c.first && r1 - r0 <= p.chunk && p.units <= NT;
  c.none = k < 0 || (k > 0 && ((long)k << p.chunk_log2) >= r1 - r0);
  c.begin = c.none ? r0 : r0 + (k << p.chunk_log2);
  c.end = (int)min((long)r1, (long)c.begin + p.chunk);
  return c;
}

// --------------------------------------------------------------- elements ---

template <class T, int V>
struct Run {
  typedef T type __attribute__((ext_vector_type(V)));
};
template <class T>
struct Run<T, 1> {
  typedef T type;
};
template <class T, int V>
__device__ __forceinline__ typename Run<T, V>::type read(const T* p) {
  return *reinterpret_cast<const typename Run<T, V>::type*>(p);
}
template <class T, int V>
__device__ __forceinline__ void widen(const typename Run<T, V>::type& r, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = (float)r;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)r[i];
  }
}
// v, or 0 where keep is 0 (else all ones), whatever v is.
__device__ __forceinline__ float kept(float v, uint32_t keep) { return __uint_as_float(__float_as_uint(v) & keep); }
// PAST: results go past the L2s.
template <class T, int V, bool PAST>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
  typename Run<T, V>::type r;
  if constexpr (V == 1) {
    r = (T)v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = (T)v[i];
  }
  typename Run<T, V>::type* to = reinterpret_cast<typename Run<T, V>::type*>(p);
  if constexpr (PAST) __builtin_nontemporal_store(r, to);
  else *to = r;
}

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == E3CONV_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if (ACT == E3CONV_ACT_SILU) return z * sigmoid(z);
  if (ACT == E3CONV_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  return z;
}
template <int ACT>
__device__ __forceinline__ float activate_grad(float z) {
  if (ACT == E3CONV_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if (ACT == E3CONV_ACT_SILU) {
    const float e = sigmoid(z);
    return e * fmaf(z, 1.0f - e, 1.0f);
  }
  if (ACT == E3CONV_ACT_GELU)
    return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
           z * 0.39894228040143268f * __builtin_amdgcn_exp2f(z * z * -0.72134752044448170368f);
  return 1.0f;
}

// ---------------------------------------------------------------- threads ---

// Thread -> run of channels and row of each pass.  units > NT: blockIdx.y picks NT of them.
struct Place {
  int unit, row, step;     // step: rows of a pass
  int width;               // units of this work-group
  int col;                 // unit within them
  bool on;
};
__device__ __forceinline__ Place place(const NormParams& p) {
  Place q;
  const int from = blockIdx.y * NT;
  q.width = min(p.units - from, NT);
  const bool usual = q.width == p.by_width.d;
  q.step = usual ? p.by_width.of(NT) : NT / q.width;
  q.row = usual ? p.by_width.of(threadIdx.x) : (int)threadIdx.x / q.width;
  q.col = threadIdx.x - q.row * q.width;
  q.unit = from + q.col;
  q.on = q.row < q.step;
  return q;
}

// s1 and s2 of two threads of one unit: their sums, or
struct Add {
  static constexpr bool COUNTED = false;
  template <int V>
  static __device__ __forceinline__ void join(float&, float, float (&s1)[V], float (&s2)[V], const float (&t1)[V],
                                              const float (&t2)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s1[i] += t1[i];
      s2[i] += t2[i];
    }
  }
};
// mean and squared deviations of n and of k values, of them all: a sum of terms that are not
// negative, so no cancellation wherever the means lie.
struct Moments {
  static constexpr bool COUNTED = true;
  template <int V>
  static __device__ __forceinline__ void join(float& n, float k, float (&s1)[V], float (&s2)[V], const float (&t1)[V],
                                              const float (&t2)[V]) {
    const float all = n + k, f = all > 0.0f ? k * __builtin_amdgcn_rcpf(all) : 0.0f, g = n * f;
    n = all;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = t1[i] - s1[i];
      s1[i] = fmaf(d, f, s1[i]);
      s2[i] += fmaf(d * d, g, t2[i]);
    }
  }
};
// Joins n, s1 and s2 over the threads of one unit; the result is in those of row 0.  Threads of a
// row have the same n.
template <class Join, int V>
__device__ void join_rows(const Place& q, float2* red, float n, float (&s1)[V], float (&s2)[V]) {
  __shared__ float counts[Join::COUNTED ? NT : 1];
  int rows = q.step, row = q.row;
  bool on = q.on;
  float k = 0.0f, t1[V], t2[V];
  if (64 % q.width == 0) {     // within a wave first
    for (int o = 32; o >= q.width; o >>= 1) {
      if (Join::COUNTED) k = __shfl_xor(n, o);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t1[i] = __shfl_xor(s1[i], o);
        t2[i] = __shfl_xor(s2[i], o);
      }
      Join::template join<V>(n, k, s1, s2, t1, t2);
    }
    rows = NT / 64;
    row = threadIdx.x >> 6;
    on = (threadIdx.x & 63) < q.width;
  }
  int half = 1;
  while (half < rows) half <<= 1;
  const int unit = q.col;
  for (half >>= 1; half > 0; half >>= 1) {
    if (on && row >= half && row < rows) {
      if (Join::COUNTED) counts[row - half] = n;
#pragma unroll
      for (int i = 0; i < V; ++i) red[((row - half) * V + i) * q.width + unit] = make_float2(s1[i], s2[i]);
    }
    __syncthreads();
    if (on && row < half && row + half < rows) {
      if (Join::COUNTED) k = counts[row];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 r = red[(row * V + i) * q.width + unit];
        t1[i] = r.x;
        t2[i] = r.y;
      }
      Join::template join<V>(n, k, s1, s2, t1, t2);
    }
    __syncthreads();
    rows = min(rows, half);
  }
}
template <int V>
__device__ __forceinline__ void add_rows(const Place& q, float2* red, float (&s1)[V], float (&s2)[V]) {
  join_rows<Add, V>(q, red, 0.0f, s1, s2);
}

// Counted rows of a chunk (in every thread), and the first of them (end if none).
__device__ int count_rows(const NormParams& p, const Chunk& c, int* first) {
  *first = c.begin;
  if (!p.a.row_mask) return c.end - c.begin;
  __shared__ int part[NT / 64], low[NT / 64];
  int n = 0, f = c.end;
  for (int r = c.begin + (int)threadIdx.x; r < c.end; r += NT)
    if (p.a.row_mask[r]) {
      ++n;
      f = min(f, r);
    }
  for (int o = 32; o > 0; o >>= 1) {
    n += __shfl_xor(n, o);
    f = min(f, __shfl_xor(f, o));
  }
  if ((threadIdx.x & 63) == 0) {
    part[threadIdx.x >> 6] = n;
    low[threadIdx.x >> 6] = f;
  }
  __syncthreads();
  *first = min(min(low[0], low[1]), min(low[2], low[3]));
  return part[0] + part[1] + part[2] + part[3];
}

// For this thread's rows of the chunk, N at a time: load(i, row) of all of them, then use(i, row,
// keep), keep all ones for a row that counts and else 0, then done().  Rows that do not count are computed
// and their results cleared: a choice by condition becomes a branch for each element (reverse
// pass of 100 000 masked rows of 64 channels bf16: 30.4 against 28.7 us).
template <int N, bool MASK, class L, class F, class D>
__device__ __forceinline__ void rows_of(const NormParams& p, const Chunk& c, const Place& q, L load, F use, D done) {
  for (int r = c.begin + q.row; r < c.end; r += N * q.step) {
    uint32_t keep[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = min(r + i * q.step, c.end - 1);
      load(i, (long)at);
      keep[i] = MASK ? p.a.row_mask[at] : 1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (r + i * q.step < c.end) use(i, (long)(r + i * q.step), !MASK || keep[i] ? ~0u : 0u);
    done();
  }
}
template <int N, class L, class F, class D>
__device__ __forceinline__ void each_row(const NormParams& p, const Chunk& c, const Place& q, L load, F use, D done) {
  if (!q.on) return;
  if (p.a.row_mask) rows_of<N, true>(p, c, q, load, use, done);
  else rows_of<N, false>(p, c, q, load, use, done);
}
template <int N, class L, class F>
__device__ __forceinline__ void each_row(const NormParams& p, const Chunk& c, const Place& q, L load, F use) {
  each_row<N>(p, c, q, load, use, [] {});
}

// Calls use(i, group) for the V channels from c0 on.
template <int V, class F>
__device__ __forceinline__ void each_group(const NormParams& p, int c0, F use) {
  const int gc = p.gc;
  int g = p.by_gc.of(c0), left = (g + 1) * gc - c0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (left == 0) {
      ++g;
      left = gc;
    }
    --left;
    use(i, g);
  }
}

// Per-channel constants of a thread's run.
template <int V>
struct Channels {
  float w[V], b[V], mean[V], rstd[V];
  // Few and wide loads: one of four bytes for each channel and constant cost a chunk of a few
  // rows a thread more than its rows.
  __device__ __forceinline__ void affine(const NormParams& p, int c0) {
    read(p.a.weight, c0, p.vec_affine, 1.0f, w);
    read(p.a.bias, c0, p.vec_affine, 0.0f, b);
  }
  static __device__ __forceinline__ void read(const float* from, int c0, int vec, float none, float (&v)[V]) {
    if (!from) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = none;
    } else if (V % 4 == 0 && vec) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 x = reinterpret_cast<const float4*>(from + c0)[i];
        v[4 * i] = x.x;
        v[4 * i + 1] = x.y;
        v[4 * i + 2] = x.z;
        v[4 * i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = from[c0 + i];
    }
  }
  __device__ __forceinline__ void moments(const NormParams& p, int g, int c0) {
    int have = -1;
    float m = 0.0f, r = 0.0f;
    each_group<V>(p, c0, [&](int i, int grp) {
      if (grp != have) {
        have = grp;
        m = p.mean[g * p.a.groups + grp];
        r = p.rstd[g * p.a.groups + grp];
      }
      mean[i] = m;
      rstd[i] = r;
    });
  }
};

// Sum over the threads of a work-group, in every thread.
__device__ float block_sum(float v) {
  __shared__ float part[NT / 64];
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// The V sums from c0 on of a slot.
template <int V>
__device__ __forceinline__ void read_sums(const NormParams& p, long slot, int c0, float (&s1)[V], float (&s2)[V]) {
  const float2* at = p.sums + slot * p.a.channels + c0;
  if constexpr (V == 1) {
    s1[0] = at[0].x;
    s2[0] = at[0].y;
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float4 x = reinterpret_cast<const float4*>(at)[i];
      s1[2 * i] = x.x;
      s2[2 * i] = x.y;
      s1[2 * i + 1] = x.z;
      s2[2 * i + 1] = x.w;
    }
  }
}
template <int V>
__device__ __forceinline__ void write_sums(const NormParams& p, long slot, int c0, const float (&s1)[V],
                                           const float (&s2)[V]) {
  float2* at = p.sums + slot * p.a.channels + c0;
  if constexpr (V == 1) {
    at[0] = make_float2(s1[0], s2[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      reinterpret_cast<float4*>(at)[i] = make_float4(s1[2 * i], s2[2 * i], s1[2 * i + 1], s2[2 * i + 1]);
  }
}

// The slots of a graph's chunks.
struct Slots {
  int first, count;
};
__device__ __forceinline__ Slots slots_of(const NormParams& p, int g) {
  const int r0 = offset(p, g), rows = offset(p, g + 1) - r0;
  return {(r0 >> p.chunk_log2) + g, max((int)(((long)rows + p.chunk - 1) >> p.chunk_log2), 1)};
}

// ---------------------------------------------------------------- forward ---

template <class T, int V, int ACT, bool S>
__device__ __forceinline__ void write_rows(const NormParams& p, const Chunk& c, const Place& q,
                                           const Channels<V>& k) {
  const T* x = (const T*)p.a.x + q.unit * V;
  T* y = (T*)p.y + q.unit * V;
  typename Run<T, V>::type raw[4];
  each_row<4>(p, c, q, [&](int j, long r) { raw[j] = read<T, V>(x + r * p.a.x_row); },
              [&](int j, long r, uint32_t keep) {
    float v[V];
    widen<T, V>(raw[j], v);
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = kept(activate<ACT>(fmaf((v[i] - k.mean[i]) * k.rstd[i], k.w[i], k.b[i])), keep);
    store<T, V, S>(y + r * p.y_row, v);
  });
}

// Seven waves a SIMD: one register more than 72 costs one of them (4096 graphs of 20 rows of 32
// channels bf16: 49 us with six, 46 with seven).
template <class T, int V, int ACT, bool S>
__global__ void __launch_bounds__(NT, 7) norm_sums(NormParams p) {
  const unsigned slot = block_index();
  if (slot >= (unsigned)p.slots) return;
  const Chunk c = chunk_of(p, (int)slot);
  if (c.none) return;
  const Place q = place(p);
  const T* x = (const T*)p.a.x + q.unit * V;
  int first;
  const int n = count_rows(p, c, &first);
  // Mean and squared deviations of the rows so far.  A batch of four rows is summed about the mean
  // before it (the first about the chunk's first counted row), and at most the batch's share
  // of the rows is subtracted from its squares: an outlier costs no digits, whichever row it
  // is.  (With all rows about the first one: rstd off by 1e-3 where that one is a master
  // node's, 10 000 times the others, in a chunk of 30 000.)
  float at[V], mean[V], s2[V], d1[V], d2[V], count = 0.0f, batch = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) at[i] = s2[i] = d1[i] = d2[i] = 0.0f;
  if (q.on && n > 0) widen<T, V>(read<T, V>(x + first * p.a.x_row), at);
#pragma unroll
  for (int i = 0; i < V; ++i) mean[i] = at[i];
  typename Run<T, V>::type raw[4];
  each_row<4>(p, c, q, [&](int j, long r) { raw[j] = read<T, V>(x + r * p.a.x_row); },
              [&](int j, long, uint32_t keep) {
    float v[V];
    widen<T, V>(raw[j], v);
    batch += kept(1.0f, keep);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = kept(v[i] - mean[i], keep);
      d1[i] += d;
      d2[i] = fmaf(d, d, d2[i]);
    }
  }, [&] {
    count += batch;
    const float inv = count > 0.0f ? __builtin_amdgcn_rcpf(count) : 0.0f;
    batch = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = d1[i] * inv;
      s2[i] += fmaf(-d, d1[i], d2[i]);
      mean[i] += d;
      d1[i] = d2[i] = 0.0f;
    }
  });
  // of the chunk, per channel, the mean less `at`
  float s1[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s1[i] = mean[i] - at[i];
  __shared__ float2 red[NT * V];
  join_rows<Moments, V>(q, red, q.on ? count : 0.0f, s1, s2);
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s2[i] = fmaxf(s2[i], 0.0f);
    s1[i] += at[i];
  }
  const int c0 = q.unit * V;
  if (!c.only) {
    if (threadIdx.x < q.width) write_sums<V>(p, slot, c0, s1, s2);
    if (threadIdx.x == 0 && blockIdx.y == 0) p.counts[slot] = (float)n;
    return;
  }
  // the graph's only chunk: its groups here, each by every thread that has one of its channels,
  // in channel order
  if (threadIdx.x < q.width)
#pragma unroll
    for (int i = 0; i < V; ++i) red[c0 + i] = make_float2(s1[i], s2[i]);
  __syncthreads();
  Channels<V> k;
  k.affine(p, c0);
  int have = -1;
  float m = 0.0f, rs = 0.0f;
  each_group<V>(p, c0, [&](int i, int g) {
    if (g != have) {
      have = g;
      const float2* of = red + g * p.gc;
      m = 0.0f;
      for (int j = 0; j < p.gc; ++j) m += of[j].x - of[0].x;
      m = n > 0 ? of[0].x + m / (float)p.gc : 0.0f;
      float v = 0.0f;
      for (int j = 0; j < p.gc; ++j) {
        const float d = of[j].x - m;
        v += fmaf((float)n * d, d, of[j].y);
      }
      rs = 1.0f / sqrtf(v * (inv / (float)p.gc) + p.a.eps);
    }
    k.mean[i] = m;
    k.rstd[i] = rs;
    if (threadIdx.x < q.width && (c0 + i) == g * p.gc) {
      if (p.mean) p.mean[c.g * p.a.groups + g] = m;
      if (p.rstd) p.rstd[c.g * p.a.groups + g] = rs;
    }
  });
  write_rows<T, V, ACT, S>(p, c, q, k);
}

// One work-group per (graph, group): joins the chunks about the common mean.
__global__ void __launch_bounds__(NT) norm_finish(NormParams p) {
  const unsigned pair = block_index();
  if (pair >= (unsigned)p.a.num_graphs * (unsigned)p.a.groups) return;
  const int g = (int)(pair / p.a.groups), grp = (int)(pair % p.a.groups);
  const Slots s = slots_of(p, g);
  if (s.count == 1 && p.units <= NT) return;
  const int total = s.count * p.gc;
  const float2* sums = p.sums + (long)s.first * p.a.channels + grp * p.gc;
  const float base = sums[0].x;
  float n = 0.0f, m = 0.0f, v = 0.0f;
#pragma unroll 4
  for (int t = threadIdx.x; t < total; t += NT) {
    const float k = p.counts[s.first + p.by_gc.of(t)];
    n += k;
    m = fmaf(k, sums[(long)p.by_gc.of(t) * p.a.channels + (t - p.by_gc.of(t) * p.gc)].x - base, m);
  }
  n = block_sum(n);
  m = block_sum(m);
  m = n > 0.0f ? base + m / n : 0.0f;
#pragma unroll 4
  for (int t = threadIdx.x; t < total; t += NT) {
    const float2 x = sums[(long)p.by_gc.of(t) * p.a.channels + (t - p.by_gc.of(t) * p.gc)];
    const float d = x.x - m;
    v += fmaf(p.counts[s.first + p.by_gc.of(t)] * d, d, x.y);
  }
  v = block_sum(v);
  const float rs = 1.0f / sqrtf((n > 0.0f ? v / n : 0.0f) + p.a.eps);
  if (threadIdx.x == 0) {
    p.stats[pair] = make_float2(m, rs);
    if (p.mean) p.mean[pair] = m;
    if (p.rstd) p.rstd[pair] = rs;
  }
}

// The same for all groups of a graph by one work-group (units <= NT): each thread joins its
// channels over its share of the chunks, then the shares and the channels of a group are
// joined.  In chunk order, so every work-group of the graph gets the same bits.
template <int V>
__device__ void finish_here(const NormParams& p, const Chunk& c, const Place& q, float2* red, Channels<V>& k) {
  const Slots s = slots_of(p, c.g);
  const int c0 = q.unit * V;
  int some = 0;      // means are joined less that of the first chunk with a counted row
  while (some + 1 < s.count && p.counts[s.first + some] == 0.0f) ++some;
  float n = 0.0f, base[V], s1[V], s2[V];
  read_sums<V>(p, s.first + some, c0, base, s1);
#pragma unroll
  for (int i = 0; i < V; ++i) s1[i] = s2[i] = 0.0f;
  if (q.on)
#pragma unroll 2
    for (int j = q.row; j < s.count; j += q.step) {
      float m1[V], m2[V];
      read_sums<V>(p, s.first + j, c0, m1, m2);
#pragma unroll
      for (int i = 0; i < V; ++i) m1[i] -= base[i];
      Moments::join<V>(n, p.counts[s.first + j], s1, s2, m1, m2);
    }
  join_rows<Moments, V>(q, red, n, s1, s2);
  n = block_sum(q.on && q.col == 0 ? n : 0.0f);
  const float inv = n > 0.0f ? 1.0f / n : 0.0f;
  if (threadIdx.x < q.width)
#pragma unroll
    for (int i = 0; i < V; ++i) red[c0 + i] = make_float2(base[i] + s1[i], s2[i]);
  __syncthreads();
  int have = -1;
  float m = 0.0f, rs = 0.0f;
  each_group<V>(p, c0, [&](int i, int g) {
    if (g != have) {
      have = g;
      const float2* of = red + g * p.gc;
      m = 0.0f;
      for (int j = 0; j < p.gc; ++j) m += of[j].x - of[0].x;
      m = n > 0.0f ? of[0].x + m / (float)p.gc : 0.0f;
      float v = 0.0f;
      for (int j = 0; j < p.gc; ++j) {
        const float d = of[j].x - m;
        v += fmaf(n * d, d, of[j].y);
      }
      rs = 1.0f / sqrtf(v * (inv / (float)p.gc) + p.a.eps);
    }
    k.mean[i] = m;
    k.rstd[i] = rs;
    if (c.first && threadIdx.x < q.width && c0 + i == g * p.gc) {
      if (p.mean) p.mean[c.g * p.a.groups + g] = m;
      if (p.rstd) p.rstd[c.g * p.a.groups + g] = rs;
    }
  });
}

template <class T, int V, int ACT, bool HERE, bool S>
__global__ void __launch_bounds__(NT) norm_apply(NormParams p) {
  const unsigned slot = block_index();
  if (slot >= (unsigned)p.slots) return;
  const Chunk c = chunk_of(p, (int)slot);
  if (c.none || c.only) return;
  const Place q = place(p);
  const int c0 = q.unit * V;
  Channels<V> k;
  k.affine(p, c0);
  if (HERE) {
    __shared__ float2 red[NT * V];
    finish_here<V>(p, c, q, red, k);
  } else {
    int have = -1;
    float2 s = make_float2(0.0f, 0.0f);
    each_group<V>(p, c0, [&](int i, int g) {
      if (g != have) {
        have = g;
        s = p.stats[c.g * p.a.groups + g];
      }
      k.mean[i] = s.x;
      k.rstd[i] = s.y;
    });
  }
  write_rows<T, V, ACT, S>(p, c, q, k);
}

// ---------------------------------------------------------------- reverse ---

// Rows of x and grad_y of a thread's run of channels.
template <class T, int V>
struct RowPair {
  typename Run<T, V>::type x, gy;
  __device__ __forceinline__ void load(const NormParams& p, long r, int c0) {
    x = read<T, V>((const T*)p.a.x + r * p.a.x_row + c0);
    gy = read<T, V>((const T*)p.gy + r * p.gy_row + c0);
  }
  // dz and xhat
  template <int ACT>
  __device__ __forceinline__ void grad(const Channels<V>& k, uint32_t keep, float (&dz)[V], float (&xh)[V]) const {
    widen<T, V>(x, xh);
    widen<T, V>(gy, dz);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float h = (xh[i] - k.mean[i]) * k.rstd[i];
      dz[i] = kept(dz[i] * activate_grad<ACT>(fmaf(h, k.w[i], k.b[i])), keep);
      xh[i] = kept(h, keep);
    }
  }
};

template <class T, int V, int ACT, bool S>
__device__ __forceinline__ void write_grads(const NormParams& p, const Chunk& c, const Place& q,
                                            const Channels<V>& k, const float (&m1)[V], const float (&m2)[V]) {
  T* gx = (T*)p.gx + q.unit * V;
  RowPair<T, V> row[4];
  each_row<4>(p, c, q, [&](int j, long r) { row[j].load(p, r, q.unit * V); },
              [&](int j, long r, uint32_t keep) {
    float dz[V], xh[V];
    row[j].template grad<ACT>(k, ~0u, dz, xh);
#pragma unroll
    for (int i = 0; i < V; ++i)
      dz[i] = kept(k.rstd[i] * (fmaf(dz[i], k.w[i], -m1[i]) - xh[i] * m2[i]), keep);
    store<T, V, S>(gx + r * p.gx_row, dz);
  });
}

// Means of w dz and w dz xhat of the groups of a thread's channels, from their sums over n rows.
template <int V>
__device__ void group_means(const NormParams& p, const Place& q, const Channels<V>& k, float n, float2* red,
                            const float (&s1)[V], const float (&s2)[V], float (&m1)[V], float (&m2)[V]) {
  const int c0 = q.unit * V;
  if (threadIdx.x < q.width)
#pragma unroll
    for (int i = 0; i < V; ++i) red[c0 + i] = make_float2(s1[i] * k.w[i], s2[i] * k.w[i]);
  __syncthreads();
  const float inv = n > 0.0f ? 1.0f / (n * (float)p.gc) : 0.0f;
  int have = -1;
  float a = 0.0f, b = 0.0f;
  each_group<V>(p, c0, [&](int i, int g) {
    if (g != have) {
      have = g;
      a = b = 0.0f;
      for (int j = 0; j < p.gc; ++j) {
        a += red[g * p.gc + j].x;
        b += red[g * p.gc + j].y;
      }
    }
    m1[i] = a * inv;
    m2[i] = b * inv;
  });
}

template <class T, int V, int ACT, bool S>
__global__ void __launch_bounds__(NT) norm_grad_sums(NormParams p) {
  const unsigned slot = block_index();
  if (slot >= (unsigned)p.slots) return;
  const Chunk c = chunk_of(p, (int)slot);
  const Place q = place(p);
  const int c0 = q.unit * V;
  float s1[V], s2[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s1[i] = s2[i] = 0.0f;
  if (c.none) {     // the weight gradient sums over all slots
    if (threadIdx.x < q.width) write_sums<V>(p, slot, c0, s1, s2);
    return;
  }
  Channels<V> k;
  k.affine(p, c0);
  k.moments(p, c.g, c0);
  float n = 0.0f;
  RowPair<T, V> row[4];
  each_row<4>(p, c, q, [&](int j, long r) { row[j].load(p, r, c0); },
              [&](int j, long, uint32_t keep) {
    float dz[V], xh[V];
    row[j].template grad<ACT>(k, keep, dz, xh);
    n += keep ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s1[i] += dz[i];
      s2[i] = fmaf(dz[i], xh[i], s2[i]);
    }
  });
  __shared__ float2 red[NT * V];
  add_rows<V>(q, red, s1, s2);
  n = block_sum(q.on && q.col == 0 ? n : 0.0f);
  if (threadIdx.x < q.width) write_sums<V>(p, slot, c0, s1, s2);
  if (threadIdx.x == 0 && blockIdx.y == 0) p.counts[slot] = n;
  if (!c.only) return;
  float m1[V], m2[V];
  group_means<V>(p, q, k, n, red, s1, s2, m1, m2);
  write_grads<T, V, ACT, S>(p, c, q, k, m1, m2);
}

// One work-group per (graph, group).
__global__ void __launch_bounds__(NT) norm_grad_finish(NormParams p) {
  const unsigned pair = block_index();
  if (pair >= (unsigned)p.a.num_graphs * (unsigned)p.a.groups) return;
  const int g = (int)(pair / p.a.groups), grp = (int)(pair % p.a.groups);
  const Slots s = slots_of(p, g);
  if (s.count == 1 && p.units <= NT) return;
  const int total = s.count * p.gc;
  float n = 0.0f, m1 = 0.0f, m2 = 0.0f;
#pragma unroll 4
  for (int t = threadIdx.x; t < total; t += NT) {
    const int ch = grp * p.gc + t - p.by_gc.of(t) * p.gc;
    const float2 x = p.sums[(long)(s.first + p.by_gc.of(t)) * p.a.channels + ch];
    const float w = p.a.weight ? p.a.weight[ch] : 1.0f;
    n += p.counts[s.first + p.by_gc.of(t)];
    m1 = fmaf(w, x.x, m1);
    m2 = fmaf(w, x.y, m2);
  }
  n = fmaxf(block_sum(n), 1.0f);
  m1 = block_sum(m1) / n;
  m2 = block_sum(m2) / n;
  if (threadIdx.x == 0) p.stats[pair] = make_float2(m1, m2);
}

// Weight and bias gradients of four channels: 64 threads each over the slots.
__device__ void affine_grads(const NormParams& p, int c0, float2* red) {
  const int c = c0 + (threadIdx.x & 3);
  float w = 0.0f, b = 0.0f;
  if (c < p.a.channels)
#pragma unroll 8
    for (int s = threadIdx.x >> 2; s < p.slots; s += NT / 4) {
      const float2 v = p.sums[(long)s * p.a.channels + c];
      b += v.x;
      w += v.y;
    }
  red[threadIdx.x] = make_float2(b, w);
  __syncthreads();
  for (int o = NT / 2; o >= 4; o >>= 1) {
    if ((int)threadIdx.x < o) {
      red[threadIdx.x].x += red[threadIdx.x + o].x;
      red[threadIdx.x].y += red[threadIdx.x + o].y;
    }
    __syncthreads();
  }
  if (threadIdx.x < 4 && c < p.a.channels) {
    if (p.gb) p.gb[c] = red[threadIdx.x].x;
    if (p.gw) p.gw[c] = red[threadIdx.x].y;
  }
}

// Work-groups from p.slots on take the weight and bias gradients.
template <class T, int V, int ACT, bool HERE, bool S>
__global__ void __launch_bounds__(NT) norm_grad_apply(NormParams p) {
  __shared__ float2 red[NT * V];
  const unsigned slot = block_index();
  if (slot >= (unsigned)p.slots) {
    const unsigned c = (slot - p.slots) * 4;
    if (blockIdx.y == 0 && c < (unsigned)p.a.channels) affine_grads(p, (int)c, red);
    return;
  }
  const Chunk c = chunk_of(p, (int)slot);
  if (c.none || c.only) return;
  const Place q = place(p);
  const int c0 = q.unit * V;
  Channels<V> k;
  k.affine(p, c0);
  k.moments(p, c.g, c0);
  float m1[V], m2[V];
  if (HERE) {
    const Slots s = slots_of(p, c.g);
    float n = 0.0f, s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s1[i] = s2[i] = 0.0f;
    if (q.on)
#pragma unroll 2
      for (int j = q.row; j < s.count; j += q.step) {
        n += p.counts[s.first + j];
        float a1[V], a2[V];
        read_sums<V>(p, s.first + j, c0, a1, a2);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s1[i] += a1[i];
          s2[i] += a2[i];
        }
      }
    add_rows<V>(q, red, s1, s2);
    n = block_sum(q.on && q.col == 0 ? n : 0.0f);
    group_means<V>(p, q, k, n, red, s1, s2, m1, m2);
  } else {
    int have = -1;
    float2 s = make_float2(0.0f, 0.0f);
    each_group<V>(p, c0, [&](int i, int g) {
      if (g != have) {
        have = g;
        s = p.stats[c.g * p.a.groups + g];
      }
      m1[i] = s.x;
      m2[i] = s.y;
    });
  }
  write_grads<T, V, ACT, S>(p, c, q, k, m1, m2);
}

// --------------------------------------------------------------- launches ---

template <class T, int V, int ACT, bool S>
hipError_t forward(const NormParams& p, bool one, hipStream_t s) {
  const dim3 grid = grid_of(p.slots, (unsigned)((p.units + NT - 1) / NT));
  hipLaunchKernelGGL((norm_sums<T, V, ACT, S>), grid, dim3(NT), 0, s, p);
  if (one) return hipGetLastError();
  if (p.inline_finish) {
    hipLaunchKernelGGL((norm_apply<T, V, ACT, true, S>), grid, dim3(NT), 0, s, p);
  } else {
    hipLaunchKernelGGL(norm_finish, grid_of((int64_t)p.a.num_graphs * p.a.groups, 1), dim3(NT), 0, s, p);
    hipLaunchKernelGGL((norm_apply<T, V, ACT, false, S>), grid, dim3(NT), 0, s, p);
  }
  return hipGetLastError();
}

template <class T, int V, int ACT, bool S>
hipError_t backward(const NormParams& p, bool one, hipStream_t s) {
  const unsigned columns = (unsigned)((p.units + NT - 1) / NT);
  const unsigned affine = p.gw || p.gb ? (unsigned)((p.a.channels + 3) / 4) : 0;
  hipLaunchKernelGGL((norm_grad_sums<T, V, ACT, S>), grid_of(p.slots, columns), dim3(NT), 0, s, p);
  if (one && affine == 0) return hipGetLastError();
  const dim3 grid = grid_of((int64_t)p.slots + affine, columns);
  if (p.inline_finish || one) {
    hipLaunchKernelGGL((norm_grad_apply<T, V, ACT, true, S>), grid, dim3(NT), 0, s, p);
  } else {
    hipLaunchKernelGGL(norm_grad_finish, grid_of((int64_t)p.a.num_graphs * p.a.groups, 1), dim3(NT), 0, s, p);
    hipLaunchKernelGGL((norm_grad_apply<T, V, ACT, false, S>), grid, dim3(NT), 0, s, p);
  }
  return hipGetLastError();
}

template <class T, int V, bool S>
hipError_t by_activation(const NormParams& p, bool back, bool one, hipStream_t s) {
  switch (p.a.activation) {
    case E3CONV_ACT_RELU:
      return back ? backward<T, V, E3CONV_ACT_RELU, S>(p, one, s) : forward<T, V, E3CONV_ACT_RELU, S>(p, one, s);
    case E3CONV_ACT_SILU:
      return back ? backward<T, V, E3CONV_ACT_SILU, S>(p, one, s) : forward<T, V, E3CONV_ACT_SILU, S>(p, one, s);
    case E3CONV_ACT_GELU:
      return back ? backward<T, V, E3CONV_ACT_GELU, S>(p, one, s) : forward<T, V, E3CONV_ACT_GELU, S>(p, one, s);
    default:
      return back ? backward<T, V, E3CONV_ACT_NONE, S>(p, one, s) : forward<T, V, E3CONV_ACT_NONE, S>(p, one, s);
  }
}

// Rows of a chunk, as a power of two: all of them where the call is small and has many graphs (then
// every graph is one chunk and one launch does it; a graph with all 2^18 elements to itself
// takes its work-group some 50 us), else about four work-groups per compute unit, 16 KiB
// each at least.
int chunk_rows_log2(const e3conv_group_norm_args& a) {
  const int64_t row = (int64_t)a.channels * (a.dtype == E3CONV_F32 ? 4 : 2), all = a.num_rows * a.channels;
  int64_t rows = (a.num_rows + 1023) / 1024;
  if (rows * row < 16384) rows = (16384 + row - 1) / row;
  if (all <= 1 << 18 && all <= (int64_t)16384 * a.num_graphs) rows = a.num_rows;
  int l = 0;
  while (((int64_t)1 << l) < rows) ++l;
  return l < 30 ? l : 30;
}
int chunk_slots(const e3conv_group_norm_args& a) { return (int)((a.num_rows >> chunk_rows_log2(a)) + a.num_graphs); }

// sums (slots, channels), stats (graphs, groups), counts (slots); none for a forward of one launch.
size_t workspace_bytes(const e3conv_group_norm_args& a, bool back) {
  if (!back && a.channels <= NT && a.num_rows <= (int64_t)1 << chunk_rows_log2(a)) return 0;
  const size_t slots = (size_t)chunk_slots(a);
  return (slots * a.channels + (size_t)a.num_graphs * a.groups) * sizeof(float2) + (slots * sizeof(float) + 15) / 16 * 16;
}

// Whether 16-byte runs of channels are aligned in a tensor.
bool aligned(const void* p, int64_t row, int v) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % v == 0; }

hipError_t launch(NormParams p, bool back, bool vec, void* workspace, hipStream_t s) {
  const bool f32 = p.a.dtype == E3CONV_F32;
  const int v = f32 ? 4 : 8;
  if (p.a.channels % v != 0) vec = false;
  p.gc = p.a.channels / p.a.groups;
  p.units = vec ? p.a.channels / v : p.a.channels;
  p.by_gc = div_by(p.gc);
  p.by_width = div_by(p.units < NT ? p.units : NT);
  p.chunk_log2 = chunk_rows_log2(p.a);
  p.chunk = 1 << p.chunk_log2;
  // results larger than the L2s go past them: the rows that are read again stay there (1M rows of
  // 64 channels bf16: 84 against 97 us); smaller ones stay for the operator that reads them next
  const bool past = p.a.num_rows * p.a.channels * (f32 ? 4 : 2) > (int64_t)32 << 20;
  p.vec_affine = (reinterpret_cast<uintptr_t>(p.a.weight) | reinterpret_cast<uintptr_t>(p.a.bias)) % 16 == 0;
  p.slots = chunk_slots(p.a);
  p.sums = static_cast<float2*>(workspace);
  p.stats = p.sums + (size_t)p.slots * p.a.channels;
  p.counts = reinterpret_cast<float*>(p.stats + (size_t)p.a.num_graphs * p.a.groups);
  const bool one = p.a.num_rows <= p.chunk && p.units <= NT;
  // with few chunks a graph, joining them in every work-group of the graph costs less than a launch
  p.inline_finish = p.units <= NT && p.a.num_rows / p.chunk <= (int64_t)16 * p.a.num_graphs;
  if (f32 && !vec) return by_activation<float, 1, false>(p, back, one, s);
  if (!vec) return by_activation<__bf16, 1, false>(p, back, one, s);
  if (f32 && past) return by_activation<float, 4, true>(p, back, one, s);
  if (f32) return by_activation<float, 4, false>(p, back, one, s);
  if (past) return by_activation<__bf16, 8, true>(p, back, one, s);
  return by_activation<__bf16, 8, false>(p, back, one, s);
}

e3conv_status bad(const char* what) { return api_fail(E3CONV_ERR_INVALID_ARGUMENT, what); }

e3conv_status check_sizes(const e3conv_group_norm_args* a) {
  if (!a) return bad("args is NULL");
  if (a->dtype != E3CONV_F32 && a->dtype != E3CONV_BF16) return bad("bad dtype");
  if (a->num_graphs < 0 || a->num_rows < 0) return bad("negative size");
  if (a->num_graphs == 0 && a->num_rows > 0) return bad("rows without a graph");
  if (a->channels < 1 || a->channels > kMaxChannels || a->groups < 1 || a->channels % a->groups != 0)
    return bad("channels must be in [1, 4096] and a multiple of groups");
  if (a->num_rows + a->num_graphs >= ((int64_t)1 << 31) - ((int64_t)1 << 20) ||
      (int64_t)a->num_graphs * a->groups >= ((int64_t)1 << 31) - ((int64_t)1 << 20))
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
  *bytes = e3c::workspace_bytes(*a, backward != 0);
  return e3c::api_ok();
}

e3conv_status e3conv_group_norm(const e3conv_group_norm_args* a, void* y, int64_t y_row, float* mean, float* rstd,
                                void* workspace, size_t bytes, void* stream) {
  const e3conv_status st = e3c::check_args(a);
  if (st != E3CONV_OK) return st;
  if (y_row < 0) return e3c::bad("negative stride");
  if (a->num_graphs == 0) return e3c::api_ok();
  if (a->num_rows > 0 && !y) return e3c::bad("NULL device pointer");
  const size_t need = e3c::workspace_bytes(*a, false);
  if (bytes < need || (need > 0 && !workspace))
    return e3c::api_fail(E3CONV_ERR_WORKSPACE, "group norm needs " + std::to_string(need) + " bytes");
  e3c::NormParams p{};
  p.a = *a;
  p.y = y;
  p.y_row = y_row;
  p.mean = mean;
  p.rstd = rstd;
  const int v = a->dtype == E3CONV_F32 ? 4 : 8;
  const hipError_t err =
      e3c::launch(p, false, e3c::aligned(a->x, a->x_row, v) && e3c::aligned(y, y_row, v), workspace,
                  static_cast<hipStream_t>(stream));
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
  if (a->num_graphs == 0) {
    hipError_t e = hipSuccess;
    for (float* g : {grad_weight, grad_bias})
      if (g && e == hipSuccess) e = e3c::launch_fill_zero(g, (size_t)a->channels, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return e3c::api_hip_fail(e, "fill launch");
    return e3c::api_ok();
  }
  const size_t need = e3c::workspace_bytes(*a, true);
  if (bytes < need || !workspace)
    return e3c::api_fail(E3CONV_ERR_WORKSPACE, "group norm backward needs " + std::to_string(need) + " bytes");
  e3c::NormParams p{};
  p.a = *a;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.gy = grad_y;
  p.gy_row = grad_y_row;
  p.gx = grad_x;
  p.gx_row = grad_x_row;
  p.gw = grad_weight;
  p.gb = grad_bias;
  const int v = a->dtype == E3CONV_F32 ? 4 : 8;
  const bool vec = e3c::aligned(a->x, a->x_row, v) && e3c::aligned(grad_y, grad_y_row, v) &&
                   e3c::aligned(grad_x, grad_x_row, v);
  const hipError_t err = e3c::launch(p, true, vec, workspace, static_cast<hipStream_t>(stream));
  if (err != hipSuccess) return e3c::api_hip_fail(err, "group norm backward launch");
  return e3c::api_ok();
}

}  // extern "C"
