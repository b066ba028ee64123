// Differential attention, forward, on the matrix cores (contract in e3conv.h, tiles in attention_tile.h).
//
//     out = softmax(scale q1 k1^T) v - lambda softmax(scale q2 k2^T) v
//
// As the plain attention's forward, a wave owns 32 rows and walks over the keys, rows along the columns:
//     S1^T = K1 Q1^T,  S2^T = K2 Q2^T,   O1^T += V^T P1^T,  O2^T += V^T P2^T,
// each map with a running maximum and sum of its own, in one pass.  Each transposed operand of V is read from LDS
// once for both maps' products.  (The difference of the maps could be taken before one product with V, but needs
// both sums first: a second pass over all logits, whose products and exponentials cost as much as that product
// saves with dim_v = 2 dim_qk.)
#include "attention_diff_tile.h"
#include "kernels.h"

namespace e3c {
namespace attn {
namespace {

template <class T, int D, int RW, int TK, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? diff_waves_fwd(sizeof(T) == 4, D) : 1) diff_fwd(DiffParams p) {
  constexpr int P = planes<T>(), KS = D / 32, NB = TK / 32, W = P == 1 ? 4 : 2;   // W: operands read ahead
  struct Buffer {
    Tile<P, TK, D> k, v;
    float bias[TK];
  };
  static_assert(BUF == 2 || !(sizeof(T) == 2 && LOAD != kElements), "loads straight to LDS need the other buffer");
  __shared__ __attribute__((aligned(16))) Buffer first, second;
  const e3conv_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 31, h = lane >> 5;

  const long block = block_index();
  if (block >= p.blocks) return;
  const Where place = where((int)block, p.blocks, p.slots, p.splits);
  const int split = place.split, slot = place.slot, c = place.c;
  constexpr int BM = 32 * RW;
  const int g = graph_of_slot(a.q_ptr, a.num_graphs, a.num_q, p.group, BM, slot);
  const int q0 = offset(a.q_ptr, g, a.num_q);
  const int nrows = (offset(a.q_ptr, g + 1, a.num_q) - q0) * p.group;
  const int r0 = tile_start(slot, first_slot(a.q_ptr, g, a.num_q, p.group, BM), BM, nrows);
  if (r0 < 0) return;

  const int r = r0 + 32 * w + n;
  const bool row = r < nrows, idle = r0 + 32 * w >= nrows;   // idle: a wave without rows only loads
  const int qi = q0 + (row ? query_of(p, r) : 0), head = c * p.group + (row ? r - (qi - q0) * p.group : 0);
  const bool live = row && (!a.q_mask || a.q_mask[qi]);

  // this split's keys: whole tiles of the graph's
  const int kb = offset(a.k_ptr, g, a.num_k), ke = offset(a.k_ptr, g + 1, a.num_k);
  const int tiles = ke > kb ? (ke - kb + TK - 1) / TK : 0, per = (tiles + p.splits - 1) / p.splits;
  const int k0 = kb + min(split * per, tiles) * TK;
  const int k1 = min(ke, kb + min((split + 1) * per, tiles) * TK);

  Keys<T, D, TK, 64 * RW, LOAD, 2> keys;
  keys.begin(p, c, k0, k1);
  keys.pair.clear(a.dim_qk, a.dim_v, first.k, first.v);
  if (BUF == 2) keys.pair.clear(a.dim_qk, a.dim_v, second.k, second.v);
  if (k0 < k1) keys.issue(p, first.k, first.v);

  Frag<P> q[2][KS];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    row_operand<T, D / 2, LOAD>((const T*)a.q + qi * a.q_row + (2 * head + x) * a.q_head, a.dim_qk, live, q[x]);
    if (p.negate)
#pragma unroll
      for (int t = 0; t < KS; ++t) flip_sign(q[x][t]);
  }

  f32x16 o[2][D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) o[0][dt] = o[1][dt] = f32x16{};
  // of the logits in units of log 2; l: this half's keys, too large by `over` (compensated from tile to tile)
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, over[2] = {0.0f, 0.0f};

  const auto use = [&](Buffer& now, int from, Buffer& next) {
    Tile<P, TK, D>&kt = now.k, &vt = now.v;
    if (BUF == 1) __syncthreads();
    keys.finish(p, from, kt, vt, now.bias);
    __syncthreads();
    if (from + TK < k1) keys.issue(p, next.k, next.v);
    if (idle) return;

    Frag<P> f[2][2 * NB];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      f32x16 s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) s[b] = by_row(now.bias + 32 * b, lane);
      ahead<NB * KS, W, Frag<P>>([&](int i) { return kt.rows(32 * (i % NB), x * KS + i / NB, lane); },
                                 [&](int i, const Frag<P>& y) { s[i % NB] = mma(y, q[x][i / NB], s[i % NB]); });
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
      top = fmaxf(top, other_half(top)) * p.c;
      // m is the maximum only to within 2^kSlack, so that o and l are scaled again in few tiles
      constexpr float kSlack = 8.0f;
      if (__ballot(top > m[x] + kSlack)) {
        const float mn = fmaxf(m[x], top), base = mn == -INFINITY ? 0.0f : mn;
        const float by = __builtin_amdgcn_exp2f(m[x] - base);
        m[x] = mn;
        l[x] *= by;
        over[x] *= by;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[x][dt][i] *= by;
      }
      const float base = m[x] == -INFINITY ? 0.0f : m[x];
      float sum = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            e[i] = __builtin_amdgcn_exp2f(fmaf(s[b][8 * t + i], p.c, -base));
            sum += e[i];
          }
          // bf16: P rounded for its product, the sum from the unrounded values
          to_frag(e, f[x][2 * b + t]);
        }
      sum -= over[x];
      const float both = l[x] + sum;
      over[x] = (both - l[x]) - sum;
      l[x] = both;
    }
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
      ahead<D / 32, W, Frag<P>>([&](int dt) { return vt.columns(16 * t, dt, lane); },
                                [&](int dt, const Frag<P>& y) {
                                  o[0][dt] = mma(y, f[0][t], o[0][dt]);
                                  o[1][dt] = mma(y, f[1][t], o[1][dt]);
                                });
  };
  if constexpr (BUF == 2) walk<2, TK>(k0, k1, first, second, use);
  else walk<1, TK>(k0, k1, first, first, use);

#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] -= over[x];
    l[x] += other_half(l[x]);
  }
  if (!row) return;
  const long at = (long)qi * a.heads_q + head;
  if (!live) {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
  }
  if (p.splits > 1) {
    const long rows = 2 * a.num_q * a.heads_q;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const long i = split * rows + 2 * at + x;
      store_row(p.part + i * a.dim_v, o[x], a.dim_v, 1.0f, true, a.dim_v % 4 == 0);
      if (h == 0) reinterpret_cast<float2*>(p.part_ml)[i] = make_float2(m[x], l[x]);
    }
    return;
  }
  const float inv0 = l[0] == 0.0f ? 0.0f : 1.0f / l[0], inv1 = l[1] == 0.0f ? 0.0f : 1.0f / l[1];
  const float lam = p.lam[head];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      o[1][dt][i] *= inv1;
      o[0][dt][i] = fmaf(-lam, o[1][dt][i], o[0][dt][i] * inv0);
    }
  store_row((T*)p.out + qi * p.out_row + head * p.out_head, o[0], a.dim_v, 1.0f, live, p.vec_st);
  if (p.second)
    store_row((T*)p.second + qi * p.second_row + head * p.second_head, o[1], a.dim_v, 1.0f, live, p.vec_st);
  if (h == 0 && p.lse) {
    const auto lse = [](float m, float l) { return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2; };
    reinterpret_cast<float2*>(p.lse)[at] = make_float2(lse(m[0], l[0]), lse(m[1], l[1]));
  }
}

// Joins the splits of one row: each map's o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, and their difference.
// Sixteen waves take the splits of one map, then of the other, in turn.
constexpr int kJoinWaves = 16;
template <class T>
__global__ void __launch_bounds__(64 * kJoinWaves) diff_join(DiffParams p) {
  const e3conv_attention_args& a = p.a;
  __shared__ float weight[kMaxSplits], sum[kJoinWaves][kMaxDim], red[2][kJoinWaves];
  const long rows = 2 * a.num_q * a.heads_q, at = block_index();
  if (2 * at >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  float result[2], lse[2];
  for (int x = 0; x < 2; ++x) {
    float m = -INFINITY, l = 0.0f;
    if (tid < p.splits) {
      const float2 ml = reinterpret_cast<const float2*>(p.part_ml)[tid * rows + 2 * at + x];
      m = ml.x;
      l = ml.y;
    }
    const float* part = p.part + (2 * at + x) * a.dim_v;
    constexpr int N = kMaxSplits / kJoinWaves;
    float v0[N], v1[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = w + i * kJoinWaves;
      const float* o = part + s * rows * a.dim_v;
      v0[i] = s < p.splits && lane < a.dim_v ? o[lane] : 0.0f;
      v1[i] = s < p.splits && lane + 64 < a.dim_v ? o[lane + 64] : 0.0f;
    }
    float top = m;
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) red[0][w] = top;
    __syncthreads();
    top = red[0][0];
#pragma unroll
    for (int i = 1; i < kJoinWaves; ++i) top = fmaxf(top, red[0][i]);
    const float base = top == -INFINITY ? 0.0f : top, f = __builtin_amdgcn_exp2f(m - base);
    if (tid < kMaxSplits) weight[tid] = f;
    l *= f;
    for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
    if (lane == 0) red[1][w] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinWaves; ++i) l += red[1][i];
    float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float by = weight[w + i * kJoinWaves];
      a0 = fmaf(by, v0[i], a0);
      a1 = fmaf(by, v1[i], a1);
    }
    sum[w][lane] = a0;
    sum[w][lane + 64] = a1;
    __syncthreads();
    float v = 0.0f;
    if (tid < a.dim_v)
#pragma unroll
      for (int i = 0; i < kJoinWaves; ++i) v += sum[i][tid];
    result[x] = l == 0.0f ? 0.0f : v / l;
    lse[x] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
    __syncthreads();
  }
  const int head = (int)(at % a.heads_q);
  const long qi = at / a.heads_q;
  if (tid < a.dim_v) {
    ((T*)p.out)[qi * p.out_row + head * p.out_head + tid] = (T)fmaf(-p.lam[head], result[1], result[0]);
    if (p.second) ((T*)p.second)[qi * p.second_row + head * p.second_head + tid] = (T)result[1];
  }
  if (tid == 0 && p.lse) reinterpret_cast<float2*>(p.lse)[at] = make_float2(lse[0], lse[1]);
}

// The same for many rows of few splits: a thread for each element, consecutive ones side by side.
constexpr int kFewSplits = 32;
template <class T>
__global__ void __launch_bounds__(256) diff_join_rows(DiffParams p) {
  const e3conv_attention_args& a = p.a;
  const long rows = 2 * a.num_q * a.heads_q, i = block_index() * 256 + threadIdx.x, at = i / a.dim_v;
  if (2 * at >= rows) return;
  const int d = (int)(i - at * a.dim_v);
  float result[2], lse[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + 2 * at + x;
    const float* part = p.part + (2 * at + x) * a.dim_v + d;
    float top = -INFINITY, l = 0.0f, v = 0.0f;
    for (int s = 0; s < p.splits; ++s) top = fmaxf(top, ml[s * rows].x);
    const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      const float2 y = ml[s * rows];
      const float f = __builtin_amdgcn_exp2f(y.x - base);
      l = fmaf(f, y.y, l);
      v = fmaf(f, part[s * rows * a.dim_v], v);
    }
    result[x] = l == 0.0f ? 0.0f : v / l;
    lse[x] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
  }
  const long qi = at / a.heads_q;
  const int head = (int)(at - qi * a.heads_q);
  ((T*)p.out)[qi * p.out_row + head * p.out_head + d] = (T)fmaf(-p.lam[head], result[1], result[0]);
  if (p.second) ((T*)p.second)[qi * p.second_row + head * p.second_head + d] = (T)result[1];
  if (d == 0 && p.lse) reinterpret_cast<float2*>(p.lse)[at] = make_float2(lse[0], lse[1]);
}

Shape shape_of(const e3conv_attention_args& a) {
  const bool f32 = a.dtype == E3CONV_F32;
  const int width = diff_width(a);
  return choose(a.num_q * (a.heads_q / a.heads_kv), a.num_k, a.num_graphs, a.heads_kv, diff_waves_fwd(f32, width),
                diff_unit_us(f32, width, false), 2 * a.dim_v);
}

// LDS: the tiles of both buffers, at most 64 KiB (two work-groups of a compute unit).
template <class T, int D, int LOAD>
void launch(const DiffParams& p, int rw, hipStream_t s) {
  constexpr int TK4 = sizeof(T) == 4 && D == 128 ? 32 : 64, TILE = planes<T>() * D * 2 * 2;
  constexpr int BUF4 = 2 * TK4 * TILE <= 65536 ? 2 : 1, BUF1 = sizeof(T) == 2 && LOAD != kElements ? 2 : 1;
  if (rw == 4) hipLaunchKernelGGL((diff_fwd<T, D, 4, TK4, BUF4, LOAD>), grid_of(p.blocks), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((diff_fwd<T, D, 1, 32, BUF1, LOAD>), grid_of(p.blocks), dim3(64), 0, s, p);
}
template <class T, int D>
void launch(const DiffParams& p, int rw, hipStream_t s) {
  if (!p.vec) launch<T, D, kElements>(p, rw, s);
  else if (sizeof(T) == 2 && p.full) launch<T, D, sizeof(T) == 2 ? kFull : kUnits>(p, rw, s);
  else launch<T, D, kUnits>(p, rw, s);
}

template <class T>
hipError_t forward(const DiffParams& p, int rw, hipStream_t s) {
  if (diff_width(p.a) == 64) launch<T, 64>(p, rw, s);
  else launch<T, 128>(p, rw, s);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.splits == 1) return err;
  if (p.splits <= kFewSplits) {
    const long blocks = ((long)p.a.num_q * p.a.heads_q * p.a.dim_v + 255) / 256;
    hipLaunchKernelGGL(diff_join_rows<T>, grid_of(blocks), dim3(256), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(diff_join<T>, grid_of(p.a.num_q * p.a.heads_q), dim3(64 * kJoinWaves), 0, s, p);
  return hipGetLastError();
}

}  // namespace

// Maximum and sum of n partial rows, then (16-byte aligned) the rows.
static size_t ml_floats(size_t n) { return (2 * n + 3) / 4 * 4; }

size_t diff_forward_workspace(const e3conv_attention_args& a) {
  const Shape sh = shape_of(a);
  const size_t n = (size_t)sh.splits * 2 * a.num_q * a.heads_q;
  return sh.splits > 1 ? (ml_floats(n) + n * a.dim_v) * sizeof(float) : 0;
}

hipError_t launch_diff_forward(const DiffParams& given, hipStream_t s) {
  DiffParams p = given;
  const Shape sh = shape_of(p.a);
  p.slots = sh.slots;
  p.splits = sh.splits;
  p.part_ml = p.part;
  p.part += ml_floats((size_t)sh.splits * 2 * p.a.num_q * p.a.heads_q);
  const long grid = (long)sh.slots * sh.splits * p.a.heads_kv;
  if (grid > 0x7fffffffL) return hipErrorInvalidValue;
  p.blocks = (int)grid;
  return p.a.dtype == E3CONV_F32 ? forward<float>(p, sh.rw, s) : forward<__bf16>(p, sh.rw, s);
}

}  // namespace attn
}  // namespace e3c
