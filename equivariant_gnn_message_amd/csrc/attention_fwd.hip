// Attention forward on the matrix cores (contract in e3conv.h, tiles in attention_tile.h).
//
// A wave owns 32 rows (a row is one query of one of the query heads that share a
// kv head) and walks over the graph's keys in tiles that its work-group holds in
// LDS.  With the rows along the columns of both products,
//     S^T (keys x rows) = K Q^T,     out^T (dim x rows) += V^T P^T,
// a lane keeps one row: maximum and sum of its softmax are sums within the lane
// and one exchange with the other half of the wave, and P^T is the second
// product's operand where the first one left it.  One pass over the keys with the running
// maximum and sum (online softmax, Milakov and Gimelshein 2018; rescaled only when the maximum
// has grown by more than a threshold, published as conditional rescaling); the sum over tiles
// is compensated (Kahan 1965).  The next tile is on its way while the current one is used.
//
// What bounds it (100 000 nodes in ragged graphs, 8 / 2 heads of 64, bf16: 309 us,
// 695 TFLOP/s): vector instructions beside the products.  A tile of 64 keys costs a wave
// 16 products (512 cycles) and 217 vector instructions (counted, start and end of a
// work-group among them); scale, exponential, sum, maximum and packing of its 32 logits a
// lane are about 130 of these.  The vector ALU is busy in 68 % of the SIMD cycles and the matrix
// cores in 35 %.  In loops of nothing else, two waves of a SIMD took the sum of both times for
// multiply-adds beside products, and 0.86 of it for exponentials.
// LDS conflicts are none (the tiles' permutation); reads are a third of its rate.
// fp32 has the same form with six products for one; with few rows (one query against 100 000
// keys, 17.3 us) it is bound by the keys' bytes and the join of the splits.
#include "attention_tile.h"
#include "kernels.h"

namespace e3c {
namespace attn {
namespace {

template <class T, int D, int RW, int TK, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? waves_fwd(sizeof(T) == 4, D) : 1) attn_fwd(Params p) {
  constexpr int P = planes<T>(), KS = D / 16, W = P == 1 ? 4 : 2;   // W: operands read ahead
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

  Keys<T, D, TK, 64 * RW, LOAD> keys;
  keys.begin(p, c, k0, k1);
  keys.pair.clear(a.dim_qk, a.dim_v, first.k, first.v);
  if (BUF == 2) keys.pair.clear(a.dim_qk, a.dim_v, second.k, second.v);
  if (k0 < k1) keys.issue(p, first.k, first.v);

  Frag<P> q[KS];
  row_operand<T, D, LOAD>((const T*)a.q + qi * a.q_row + head * a.q_head, a.dim_qk, live, q);
  if (p.negate)
#pragma unroll
    for (int t = 0; t < KS; ++t) flip_sign(q[t]);

  f32x16 o[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) o[dt] = f32x16{};
  // of the logits in units of log 2; l: this half's keys, too large by `over`.  A tile's
  // exponentials are summed by themselves and added with compensation: keys of few kinds give equal terms, whose
  // roundings all have one sign (100 000 keys of two kinds: lse off by 3.1e-4 with l += e key by key).
  float m = -INFINITY, l = 0.0f, over = 0.0f;

  const auto use = [&](Buffer& now, int from, Buffer& next) {
    Tile<P, TK, D>&kt = now.k, &vt = now.v;
    if (BUF == 1) __syncthreads();
    keys.finish(p, from, kt, vt, now.bias);
    __syncthreads();
    if (from + TK < k1) keys.issue(p, next.k, next.v);
    if (idle) return;

    f32x16 s[TK / 32];
    constexpr int NB = TK / 32;
#pragma unroll
    for (int b = 0; b < NB; ++b) s[b] = by_row(now.bias + 32 * b, lane);
    ahead<NB * KS, W, Frag<P>>([&](int i) { return kt.rows(32 * (i % NB), i / NB, lane); },
                               [&](int i, const Frag<P>& x) { s[i % NB] = mma(x, q[i / NB], s[i % NB]); });
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < TK / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    top = fmaxf(top, other_half(top)) * p.c;
    // m is the maximum only to within 2^kSlack: P and l may grow to 2^kSlack, and o and l
    // are scaled again in few tiles (in the first sixteen, some row of 32 has a new maximum
    // nearly always)
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
#pragma unroll
    for (int b = 0; b < TK / 32; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_amdgcn_exp2f(fmaf(s[b][8 * t + i], p.c, -base));
          sum += e[i];
        }
        // bf16: P rounded for its product, the sum from the unrounded values
        Frag<P> f;
        to_frag(e, f);
        ahead<D / 32, W, Frag<P>>([&](int dt) { return vt.columns(32 * b + 16 * t, dt, lane); },
                                  [&](int dt, const Frag<P>& x) { o[dt] = mma(x, f, o[dt]); });
      }
    sum -= over;
    const float both = l + sum;
    over = (both - l) - sum;
    l = both;
  };
  if constexpr (BUF == 2) walk<2, TK>(k0, k1, first, second, use);
  else walk<1, TK>(k0, k1, first, first, use);

  l -= over;
  l += other_half(l);
  if (!row) return;
  const long at = (long)qi * a.heads_q + head;
  if (!live) {
    m = -INFINITY;
    l = 0.0f;
  }
  if (p.splits > 1) {
    const long rows = a.num_q * a.heads_q, i = split * rows + at;
    float* to = p.part + i * a.dim_v;
    store_row(to, o, a.dim_v, 1.0f, true, a.dim_v % 4 == 0);
    if (h == 0) reinterpret_cast<float2*>(p.part_ml)[i] = make_float2(m, l);
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  store_row((T*)p.out + qi * p.out_row + head * p.out_head, o, a.dim_v, inv, live, p.vec_st);
  if (h == 0 && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// Joins the splits of one row: out = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s.  Sixteen
// waves take the splits in turn, so that their rows are all in flight at once: the time is
// that of a few dependent reads (the loop of one wave over 64 splits took 20 us).
constexpr int kJoinWaves = 16;
template <class T>
__global__ void __launch_bounds__(64 * kJoinWaves) attn_join(Params p) {
  const e3conv_attention_args& a = p.a;
  __shared__ float weight[kMaxSplits], sum[kJoinWaves][kMaxDim], red[2][kJoinWaves];
  const long rows = a.num_q * a.heads_q, at = block_index();
  if (at >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  float m = -INFINITY, l = 0.0f;
  if (tid < p.splits) {
    const float2 ml = reinterpret_cast<const float2*>(p.part_ml)[tid * rows + at];
    m = ml.x;
    l = ml.y;
  }
  const float* part = p.part + at * a.dim_v;
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
    const float f = weight[w + i * kJoinWaves];
    a0 = fmaf(f, v0[i], a0);
    a1 = fmaf(f, v1[i], a1);
  }
  sum[w][lane] = a0;
  sum[w][lane + 64] = a1;
  __syncthreads();
  const int head = (int)(at % a.heads_q);
  const long qi = at / a.heads_q;
  if (tid < a.dim_v) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinWaves; ++i) v += sum[i][tid];
    ((T*)p.out)[qi * p.out_row + head * p.out_head + tid] = (T)(l == 0.0f ? 0.0f : v / l);
  }
  if (tid == 0 && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
}

// The same for many rows of few splits: a thread for each element, consecutive ones side by side.
// (By 16 waves a row, 36 000 rows of 3 splits took 0.6 ms.)
constexpr int kFewSplits = 32;
template <class T>
__global__ void __launch_bounds__(256) attn_join_rows(Params p) {
  const e3conv_attention_args& a = p.a;
  const long rows = a.num_q * a.heads_q, i = block_index() * 256 + threadIdx.x, at = i / a.dim_v;
  if (at >= rows) return;
  const int d = (int)(i - at * a.dim_v);
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + at;
  const float* part = p.part + at * a.dim_v + d;
  float top = -INFINITY, l = 0.0f, v = 0.0f;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, ml[s * rows].x);
  const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float2 x = ml[s * rows];
    const float f = __builtin_amdgcn_exp2f(x.x - base);
    l = fmaf(f, x.y, l);
    v = fmaf(f, part[s * rows * a.dim_v], v);
  }
  const long qi = at / a.heads_q;
  const int head = (int)(at - qi * a.heads_q);
  ((T*)p.out)[qi * p.out_row + head * p.out_head + d] = (T)(l == 0.0f ? 0.0f : v / l);
  if (d == 0 && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
}

Shape shape_of(const e3conv_attention_args& a) {
  const bool f32 = a.dtype == E3CONV_F32;
  const int dim = a.dim_qk > a.dim_v ? a.dim_qk : a.dim_v;
  return choose(a.num_q * (a.heads_q / a.heads_kv), a.num_k, a.num_graphs, a.heads_kv,
                waves_fwd(f32, padded(dim)), unit_us(f32, dim, false), a.dim_v);
}

// LDS: the tiles of both buffers, at most 64 KiB (two work-groups of a compute unit).
template <class T, int D, int LOAD>
void launch(const Params& p, int rw, hipStream_t s) {
  constexpr int TK4 = sizeof(T) == 4 && D == 128 ? 32 : 64, TILE = planes<T>() * D * 2 * 2;
  constexpr int BUF4 = 2 * TK4 * TILE <= 65536 ? 2 : 1, BUF1 = sizeof(T) == 2 && LOAD != kElements ? 2 : 1;
  if (rw == 4) hipLaunchKernelGGL((attn_fwd<T, D, 4, TK4, BUF4, LOAD>), grid_of(p.blocks), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((attn_fwd<T, D, 1, 32, BUF1, LOAD>), grid_of(p.blocks), dim3(64), 0, s, p);
}
template <class T, int D>
void launch(const Params& p, int rw, hipStream_t s) {
  if (!p.vec) launch<T, D, kElements>(p, rw, s);
  else if (sizeof(T) == 2 && p.full) launch<T, D, sizeof(T) == 2 ? kFull : kUnits>(p, rw, s);
  else launch<T, D, kUnits>(p, rw, s);
}

template <class T>
hipError_t forward(const Params& p, int rw, hipStream_t s) {
  const int dim = p.a.dim_qk > p.a.dim_v ? p.a.dim_qk : p.a.dim_v;
  if (dim <= 32) launch<T, 32>(p, rw, s);
  else if (dim <= 64) launch<T, 64>(p, rw, s);
  else launch<T, 128>(p, rw, s);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.splits == 1) return err;
  if (p.splits <= kFewSplits) {
    const long blocks = ((long)p.a.num_q * p.a.heads_q * p.a.dim_v + 255) / 256;
    hipLaunchKernelGGL(attn_join_rows<T>, grid_of(blocks), dim3(256), 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(attn_join<T>, grid_of(p.a.num_q * p.a.heads_q), dim3(64 * kJoinWaves), 0, s, p);
  return hipGetLastError();
}

}  // namespace

// Maximum and sum of n partial rows, then (16-byte aligned) the rows.
static size_t ml_floats(size_t n) { return (2 * n + 3) / 4 * 4; }

size_t forward_workspace(const e3conv_attention_args& a) {
  const Shape sh = shape_of(a);
  const size_t n = (size_t)sh.splits * a.num_q * a.heads_q;
  return sh.splits > 1 ? (ml_floats(n) + n * a.dim_v) * sizeof(float) : 0;
}

hipError_t launch_forward(const Params& given, hipStream_t s) {
  Params p = given;
  const Shape sh = shape_of(p.a);
  p.slots = sh.slots;
  p.splits = sh.splits;
  p.part_ml = p.part;
  p.part += ml_floats((size_t)sh.splits * p.a.num_q * p.a.heads_q);
  const long grid = (long)sh.slots * sh.splits * p.a.heads_kv;
  if (grid > 0x7fffffffL) return hipErrorInvalidValue;
  p.blocks = (int)grid;
  return p.a.dtype == E3CONV_F32 ? forward<float>(p, sh.rw, s) : forward<__bf16>(p, sh.rw, s);
}

}  // namespace attn
}  // namespace e3c
