// Differential attention, forward, on the matrix cores (contract in e3conv.h, tiles in attention_tile.h).
//
//     out = softmax(scale q1 k1^T) v - lambda softmax(scale q2 k2^T) v
//
// As the plain attention's forward, a wave owns 32 rows and walks over the keys, rows along the columns, but of one
// map: two waves share 32 rows,
//     S_m^T = K_m Q_m^T,   O_m^T += V^T P_m^T,
// each with a running maximum and sum of its own, in one pass, and the second map's wave hands its result to the
// first's through LDS at the end.  (Both maps in one wave read each operand of V once, but their sums are 128
// registers with dim_v = 128, and the whole spills: 1200 us for 100 000 ragged nodes.  The difference of the maps
// could be taken before one product with V, but needs both sums first: a second pass over all logits, whose
// products and exponentials cost as much as that product saves with dim_v = 2 dim_qk.)
// 100 000 nodes in ragged graphs, four heads of two maps of 64 over two kv heads, dim_v 128, bf16: 477 us, 675 TFLOP/s
// of products (both results take two with V: 252 us at a library product's rate).  Vector instructions take 55 % and
// products 33 % of the SIMD cycles, LDS has no conflicts, and neither fewer LDS reads nor fewer vector instructions
// change the time: no unit bounds it.  Every tile of 32 keys ends in a wait for all of its loads and a barrier, one
// tile is in flight, and two to three waves a SIMD are too few to cover that and the chain logits - exponentials - product.
#include "attention_diff_tile.h"
#include "kernels.h"

namespace e3c {
namespace attn {
namespace {

// RB: blocks of 32 rows of a work-group, a pair of waves each.
template <class T, int D, int RB, int LOAD>
__global__ void __launch_bounds__(128 * RB, RB > 1 ? diff_waves_fwd(sizeof(T) == 4) : 1) diff_fwd(DiffParams p) {
  constexpr int P = planes<T>(), KS = D / 32, TK = 32, BUF = P == 1 ? 2 : 1, W = P == 1 ? 4 : 2;   // W: operands read ahead
  struct Buffer {
    Tile<P, TK, D> k, v;
    float bias[TK];
  };
  static_assert(sizeof(Buffer) * BUF >= 128u * D * RB && RB <= 2, "room for the second map's results");
  __shared__ __attribute__((aligned(16))) Buffer first, second;
  const e3conv_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 31, h = lane >> 5;
  const int map = w & 1, block = w >> 1;

  const long index = block_index();
  if (index >= p.blocks) return;
  const Where place = where<kRun>((int)index, p.blocks, p.slots, p.splits);
  const int split = place.split, slot = place.slot, c = place.c;
  constexpr int BM = 32 * RB;
  const int g = graph_of_slot(a.q_ptr, a.num_graphs, a.num_q, p.group, BM, slot);
  const int q0 = offset(a.q_ptr, g, a.num_q);
  const int nrows = (offset(a.q_ptr, g + 1, a.num_q) - q0) * p.group;
  const int r0 = tile_start(slot, first_slot(a.q_ptr, g, a.num_q, p.group, BM), BM, nrows);
  if (r0 < 0) return;

  const int r = r0 + 32 * block + n;
  const bool row = r < nrows, idle = r0 + 32 * block >= nrows;   // idle: a wave without rows only loads
  const int qi = q0 + (row ? query_of(p, r) : 0), head = c * p.group + (row ? r - (qi - q0) * p.group : 0);
  const bool live = row && (!a.q_mask || a.q_mask[qi]);

  // this split's keys: whole tiles of the graph's
  const int kb = offset(a.k_ptr, g, a.num_k), ke = offset(a.k_ptr, g + 1, a.num_k);
  const int tiles = ke > kb ? (ke - kb + TK - 1) / TK : 0, per = (tiles + p.splits - 1) / p.splits;
  const int k0 = kb + min(split * per, tiles) * TK;
  const int k1 = min(ke, kb + min((split + 1) * per, tiles) * TK);

  DiffKeys<T, D, TK, 128 * RB, LOAD> keys;
  keys.begin(p, c, k0, k1);
  keys.pair.clear(a.dim_qk, a.dim_v, first.k, first.v);
  if (BUF == 2) keys.pair.clear(a.dim_qk, a.dim_v, second.k, second.v);
  if (k0 < k1) keys.issue(p, first.k, first.v);

  Frag<P> q[KS];
  row_operand<T, D / 2, LOAD>((const T*)a.q + qi * a.q_row + (2 * head + map) * a.q_head, a.dim_qk, live, q);
  if (p.negate)
#pragma unroll
    for (int t = 0; t < KS; ++t) flip_sign(q[t]);

  f32x16 o[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) o[dt] = f32x16{};
  // of the logits in units of log 2; l: this half's keys, too large by `over` (compensated from tile to tile)
  float m = -INFINITY, l = 0.0f, over = 0.0f;

  const auto use = [&](Buffer& now, int from, Buffer& next) {
    Tile<P, TK, D>&kt = now.k, &vt = now.v;
    if (BUF == 1) __syncthreads();
    keys.finish(p, from, kt, vt, now.bias);
    __syncthreads();
    if (from + TK < k1) keys.issue(p, next.k, next.v);
    if (idle) return;

    f32x16 s = by_row(now.bias, lane);
    ahead<KS, W, Frag<P>>([&](int i) { return kt.rows(0, map * KS + i, lane); },
                          [&](int i, const Frag<P>& x) { s = mma(x, q[i], s); });
    // the first operands of V come while the softmax is formed
    Ahead<D / 16, W, Frag<P>> values;
    const auto load = [&](int i) { return vt.columns(16 * (i / (D / 32)), i % (D / 32), lane); };
    values.start(load);
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    top = fmaxf(top, other_half(top)) * p.c;
    // m is the maximum only to within 2^kSlack, so that o and l are scaled again in few tiles
    constexpr float kSlack = 8.0f;
    if (__ballot(top > m + kSlack)) {
      const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.0f : mn;
      const float f = __builtin_amdgcn_exp2f(m - base);
      m = mn;
      l *= f;
      over *= f;
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] *= f;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f;
    Frag<P> f[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(fmaf(s[8 * t + i], p.c, -base));
        sum += e[i];
      }
      // bf16: P rounded for its product, the sum from the unrounded values
      to_frag(e, f[t]);
    }
    values.run(load, [&](int i, const Frag<P>& x) {
      const int dt = i % (D / 32);
      o[dt] = mma(x, f[i / (D / 32)], o[dt]);
    });
    sum -= over;
    const float both = l + sum;
    over = (both - l) - sum;
    l = both;
  };
  if constexpr (BUF == 2) walk<2, TK>(k0, k1, first, second, use);
  else walk<1, TK>(k0, k1, first, first, use);

  l -= over;
  l += other_half(l);
  const long at = (long)qi * a.heads_q + head;
  if (!live) {
    m = -INFINITY;
    l = 0.0f;
  }
  if (p.splits > 1) {
    if (!row) return;
    const long i = split * (2 * a.num_q * a.heads_q) + 2 * at + map;
    store_row(p.part + i * a.dim_v, o, a.dim_v, 1.0f, true, a.dim_v % 4 == 0);
    if (h == 0) reinterpret_cast<float2*>(p.part_ml)[i] = make_float2(m, l);
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] *= inv;
  // the second map's result, register by register
  float* const hand = reinterpret_cast<float*>(BUF == 2 && block == 1 ? &second : &first) +
                      (BUF == 2 ? 0 : block * 32 * D) + lane;
  __syncthreads();
  if (map == 1)
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) hand[(16 * dt + i) * 64] = o[dt][i];
  __syncthreads();
  if (!row) return;
  if (map == 0) {
    const float lam = p.lam[head];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[dt][i] = fmaf(-lam, hand[(16 * dt + i) * 64], o[dt][i]);
    store_row((T*)p.out + qi * p.out_row + head * p.out_head, o, a.dim_v, 1.0f, live, p.vec_st);
  } else if (p.second) {
    store_row((T*)p.second + qi * p.second_row + head * p.second_head, o, a.dim_v, 1.0f, live, p.vec_st);
  }
  if (h == 0 && p.lse) p.lse[2 * at + map] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Joins the splits of 32 elements of one row: each map's o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, and
// their difference.  32 threads take the splits of an element and map in turn, all their loads in flight at once
// (a work-group for all of a row's elements, one map after the other: 32 us for 461 splits of four rows).
constexpr int kJoinLanes = 32;
template <class T>
__global__ void __launch_bounds__(32 * kJoinLanes) diff_join(DiffParams p) {
  const e3conv_attention_args& a = p.a;
  constexpr int N = kMaxSplits / kJoinLanes, WAVES = kJoinLanes / 2;
  __shared__ float weight[2][kMaxSplits], red[4][WAVES], sum[2][WAVES][32];
  const int columns = (a.dim_v + 31) / 32;
  const long rows = 2 * a.num_q * a.heads_q, index = block_index(), at = index / columns;
  if (2 * at >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, first = tid >> 5;
  const int d = (int)(index - at * columns) * 32 + (tid & 31);
  float4 ml = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);       // maximum and sum of both maps
  if (tid < p.splits) ml = *reinterpret_cast<const float4*>(p.part_ml + 2 * (tid * rows + 2 * at));
  float v[2][N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int s = first + i * kJoinLanes;
    const float* o = p.part + (s * rows + 2 * at) * a.dim_v + d;
    const bool on = s < p.splits && d < a.dim_v;
    v[0][i] = on ? o[0] : 0.0f;
    v[1][i] = on ? o[a.dim_v] : 0.0f;
  }
  float m[2] = {ml.x, ml.z}, l[2] = {ml.y, ml.w}, top[2] = {ml.x, ml.z};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    for (int o = 32; o > 0; o >>= 1) top[x] = fmaxf(top[x], __shfl_xor(top[x], o));
    if (lane == 0) red[x][w] = top[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    top[x] = red[x][0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) top[x] = fmaxf(top[x], red[x][i]);
    const float f = __builtin_amdgcn_exp2f(m[x] - (top[x] == -INFINITY ? 0.0f : top[x]));
    if (tid < kMaxSplits) weight[x][tid] = f;
    l[x] *= f;
    for (int o = 32; o > 0; o >>= 1) l[x] += __shfl_xor(l[x], o);
    if (lane == 0) red[2 + x][w] = l[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(weight[x][first + i * kJoinLanes], v[x][i], s);
    s += __shfl_xor(s, 32);
    if (lane < 32) sum[x][w][lane] = s;
  }
  __syncthreads();
  if (tid >= 32 || d >= a.dim_v) return;
  float result[2], lse[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float s = 0.0f, all = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      s += sum[x][i][tid];
      all += red[2 + x][i];
    }
    result[x] = all == 0.0f ? 0.0f : s / all;
    lse[x] = all == 0.0f ? -INFINITY : (top[x] + __builtin_amdgcn_logf(all)) * kLn2;
  }
  const int head = (int)(at % a.heads_q);
  const long qi = at / a.heads_q;
  ((T*)p.out)[qi * p.out_row + head * p.out_head + d] = (T)fmaf(-p.lam[head], result[1], result[0]);
  if (p.second) ((T*)p.second)[qi * p.second_row + head * p.second_head + d] = (T)result[1];
  if (d == 0 && p.lse) reinterpret_cast<float2*>(p.lse)[at] = make_float2(lse[0], lse[1]);
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

// Blocks of 32 rows of a work-group where graphs have more than 64 rows.
constexpr int kBlocks = 2;

Shape shape_of(const e3conv_attention_args& a) {
  const bool f32 = a.dtype == E3CONV_F32;
  return choose(a.num_q * (a.heads_q / a.heads_kv), a.num_k, a.num_graphs, a.heads_kv, diff_waves_fwd(f32),
                diff_unit_us(f32, diff_width(a), false) / 2, 2 * a.dim_v, kBlocks);
}

template <class T, int D, int LOAD>
void launch(const DiffParams& p, int rw, hipStream_t s) {
  if (rw == kBlocks) hipLaunchKernelGGL((diff_fwd<T, D, kBlocks, LOAD>), grid_of(p.blocks), dim3(128 * kBlocks), 0, s, p);
  else hipLaunchKernelGGL((diff_fwd<T, D, 1, LOAD>), grid_of(p.blocks), dim3(128), 0, s, p);
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
  const long blocks = (long)p.a.num_q * p.a.heads_q * ((p.a.dim_v + 31) / 32);
  hipLaunchKernelGGL(diff_join<T>, grid_of(blocks), dim3(32 * kJoinLanes), 0, s, p);
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
