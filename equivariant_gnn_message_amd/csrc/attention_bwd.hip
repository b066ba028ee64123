// Reverse pass of attention on the matrix cores (contract in e3conv.h, tiles in
// attention_tile.h).  Two kernels, each forming P = exp(S - lse) again, none with atomics:
//
// attn_bwd_q   a wave owns 32 rows and walks over the keys.  Rows along the columns:
//                S^T = K Q^T,  dP^T = V G^T,  dS^T = P^T (dP^T - delta),  dQ^T += K^T dS^T;
//              it also forms delta = <grad_out, out> of its rows and leaves it for
// attn_bwd_kv  a wave owns 32 keys and walks over the rows of all query heads that
//              share its kv head.  Keys along the columns:
//                S = Q K^T,  dP = G V^T,  dV^T += G^T P,  dK^T += Q^T dS.
// Seven products instead of the five of a single kernel that adds dQ by atomics: the
// result is the same bits every time, and nothing but delta passes through memory.
// Where the work-groups are few both run in one launch (attn_bwd_both), the second forming
// delta itself: there the launches are the time (16 us as two, 12 as one for 64 graphs of
// 64 nodes).
//
// What bounds them: for fp32 (20 000 nodes, 4 heads of 32, 3.57 ms: 1.5 + 2.0) the products,
// six bf16 ones for each, 58 % of the SIMD cycles, and the splitting of P and dS into their parts,
// 41 %; for bf16 with 128 dimensions (50 000 ragged nodes, 548 us: 0.22 +
// 0.33 ms) the latency of LDS and barriers at one wave a SIMD for grad_k and grad_v, whose
// operands and sums fill 371 registers; with few rows (4 queries against 12 500 keys, 89 us)
// the bytes of k, v and their gradients.
#include "attention_tile.h"
#include "kernels.h"

namespace e3c {
namespace attn {
namespace {

// A tile of keys, and one of rows, in LDS.
template <class T, int D, int ROWS>
struct KeyBuffer {
  Tile<planes<T>(), ROWS, D> k, v;
  float bias[ROWS];
};
template <class T, int D, int ROWS>
struct RowBuffer {
  Tile<planes<T>(), ROWS, D> q, g;
  float lse[ROWS], delta[ROWS];
};

template <class T, int D, int RW, int TK, int BUF, int LOAD>
__device__ __forceinline__ void bwd_q(const Params& p, const Where& place, KeyBuffer<T, D, TK>& first,
                                      KeyBuffer<T, D, TK>& second) {
  typedef KeyBuffer<T, D, TK> Buffer;
  static_assert(BUF == 2 || !(sizeof(T) == 2 && LOAD != kElements), "loads straight to LDS need the other buffer");
  constexpr int P = planes<T>(), KS = D / 16, W = P == 1 ? 4 : 2;   // W: operands read ahead
  const e3conv_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 31, h = lane >> 5;

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
  const long at = (long)qi * a.heads_q + head;
  float lse = p.lse[at];
  const bool live = row && (!a.q_mask || a.q_mask[qi]) && lse != -INFINITY;
  lse = live ? lse * kLog2e : 0.0f;

  const int kb = offset(a.k_ptr, g, a.num_k), ke = offset(a.k_ptr, g + 1, a.num_k);
  const int tiles = ke > kb ? (ke - kb + TK - 1) / TK : 0, per = (tiles + p.splits - 1) / p.splits;
  const int k0 = kb + min(split * per, tiles) * TK;
  const int k1 = min(ke, kb + min((split + 1) * per, tiles) * TK);

  Keys<T, D, TK, 64 * RW, LOAD> keys;
  keys.begin(p, c, k0, k1);
  keys.pair.clear(a.dim_qk, a.dim_v, first.k, first.v);
  if (BUF == 2) keys.pair.clear(a.dim_qk, a.dim_v, second.k, second.v);
  if (k0 < k1) keys.issue(p, first.k, first.v);

  Frag<P> q[KS], go[KS];
  const T* gp = (const T*)p.go + qi * p.go_row + head * p.go_head;
  const T* op = (const T*)p.out + qi * p.out_row + head * p.out_head;
  row_operand<T, D, LOAD>((const T*)a.q + qi * a.q_row + head * a.q_head, a.dim_qk, live, q);
  row_operand<T, D, LOAD>(gp, a.dim_v, live, go);
  float delta = 0.0f;
#pragma unroll
  for (int t = 0; t < KS; ++t) {
    const int d = 16 * t + 8 * h;
    const Raw<T> gr = fetch8<LOAD != kElements>(gp, d, a.dim_v), orow = fetch8<LOAD != kElements>(op, d, a.dim_v);
    if (p.negate) flip_sign(q[t]);
#pragma unroll
    for (int i = 0; i < 8; ++i) delta = d < a.dim_v ? fmaf(gr.at(i), orow.at(i), delta) : delta;
  }
  delta = live ? delta + other_half(delta) : 0.0f;
  if (p.delta && row && h == 0 && split == 0) p.delta[at] = delta;

  // dP - delta from the start: -delta is the accumulator's first value (where its 16
  // registers do not cost a wave)
  constexpr bool FOLD = D < 128;
  f32x16 less_delta;
#pragma unroll
  for (int i = 0; i < 16; ++i) less_delta[i] = -delta;
  f32x16 dq[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) dq[dt] = f32x16{};

  const auto use = [&](Buffer& now, int from, Buffer& next) {
    Tile<P, TK, D>&kt = now.k, &vt = now.v;
    if (BUF == 1) __syncthreads();
    keys.finish(p, from, kt, vt, now.bias);
    __syncthreads();
    if (from + TK < k1) keys.issue(p, next.k, next.v);
    if (idle) return;

#pragma unroll
    for (int b = 0; b < TK / 32; ++b) {
      if (b > 0 && from + 32 * b >= k1) break;
      f32x16 s = by_row(now.bias + 32 * b, lane), dp = FOLD ? less_delta : f32x16{};
      ahead<2 * KS, W, Frag<P>>(
          [&](int i) { return i & 1 ? vt.rows(32 * b, i >> 1, lane) : kt.rows(32 * b, i >> 1, lane); },
          [&](int i, const Frag<P>& x) {
            if (i & 1) dp = mma(x, go[i >> 1], dp);
            else s = mma(x, q[i >> 1], s);
          });
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], p.c, -lse));
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = s[8 * t + i] * (FOLD ? dp[8 * t + i] : dp[8 * t + i] - delta);
        Frag<P> f;   // bf16: dS rounded for its product
        to_frag(e, f);
        ahead<D / 32, W, Frag<P>>([&](int dt) { return kt.columns(32 * b + 16 * t, dt, lane); },
                                  [&](int dt, const Frag<P>& x) { dq[dt] = mma(x, f, dq[dt]); });
      }
    }
  };
  if constexpr (BUF == 2) walk<2, TK>(k0, k1, first, second, use);
  else walk<1, TK>(k0, k1, first, first, use);

  if (!row) return;
  if (p.splits > 1) {
    store_row(p.part + (split * (a.num_q * a.heads_q) + at) * a.dim_qk, dq, a.dim_qk, 1.0f, live, a.dim_qk % 4 == 0);
    return;
  }
  store_row((T*)p.gq + qi * p.gq_row + head * p.gq_head, dq, a.dim_qk, a.scale, live, p.vec_st);
}

template <class T, int D, int RW, int TQ, int BUF, int LOAD, bool OWN>
__device__ __forceinline__ void bwd_kv(const Params& p, const Where& place, RowBuffer<T, D, TQ>& first,
                                       RowBuffer<T, D, TQ>& second) {
  typedef RowBuffer<T, D, TQ> Buffer;
  static_assert(BUF == 2 || !(sizeof(T) == 2 && LOAD != kElements), "loads straight to LDS need the other buffer");
  constexpr int P = planes<T>(), KS = D / 16, W = P == 1 ? 4 : 2;   // W: operands read ahead
  const e3conv_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 31;

  const int split = place.split, slot = place.slot, c = place.c;
  constexpr int BN = 32 * RW;
  const int g = graph_of_slot(a.k_ptr, a.num_graphs, a.num_k, 1, BN, slot);
  const int kb = offset(a.k_ptr, g, a.num_k), ke = offset(a.k_ptr, g + 1, a.num_k);
  const int first_key = tile_start(slot, first_slot(a.k_ptr, g, a.num_k, 1, BN), BN, ke - kb);
  if (first_key < 0) return;
  const int j0 = kb + first_key;

  const int j = j0 + 32 * w + n;
  const bool key = j < ke, idle = j0 + 32 * w >= ke;   // idle: a wave without keys only loads
  const bool live = key && (!a.k_mask || a.k_mask[j]);

  // this split's rows: whole tiles of the graph's
  const int q0 = offset(a.q_ptr, g, a.num_q);
  const int nrows = (offset(a.q_ptr, g + 1, a.num_q) - q0) * p.group;
  const int tiles = nrows > 0 ? (nrows + TQ - 1) / TQ : 0, per = (tiles + p.splits_kv - 1) / p.splits_kv;
  const int r0 = min(split * per, tiles) * TQ;
  const int r1 = min(nrows, min((split + 1) * per, tiles) * TQ);

  Rows<T, D, TQ, 64 * RW, LOAD, OWN> rows;
  rows.begin(p, c, q0, r0, r1);
  rows.pair.clear(a.dim_qk, a.dim_v, first.q, first.g);
  if (BUF == 2) rows.pair.clear(a.dim_qk, a.dim_v, second.q, second.g);
  if (r0 < r1) rows.issue(p, first.q, first.g);

  Frag<P> k[KS], v[KS];
  const int jr = key ? j : j0;
  row_operand<T, D, LOAD>((const T*)a.k + jr * a.k_row + c * a.k_head, a.dim_qk, live, k);
  row_operand<T, D, LOAD>((const T*)a.v + jr * a.v_row + c * a.v_head, a.dim_v, live, v);
  if (p.negate)
#pragma unroll
    for (int t = 0; t < KS; ++t) flip_sign(k[t]);

  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) dk[dt] = dv[dt] = f32x16{};

  const auto use = [&](Buffer& now, int from, Buffer& next) {
    Tile<P, TQ, D>&qt = now.q, &gt = now.g;
    if (BUF == 1) __syncthreads();
    rows.finish(p, from, qt, gt, now.lse, now.delta);
    __syncthreads();
    if (from + TQ < r1) rows.issue(p, next.q, next.g);
    if (idle) return;

#pragma unroll
    for (int b = 0; b < TQ / 32; ++b) {
      if (b > 0 && from + 32 * b >= r1) break;
      // dP - delta from the start: the rows' -delta are the accumulator's first values
      f32x16 s = f32x16{}, dp = by_row(now.delta + 32 * b, lane);
      ahead<2 * KS, W, Frag<P>>(
          [&](int i) { return i & 1 ? gt.rows(32 * b, i >> 1, lane) : qt.rows(32 * b, i >> 1, lane); },
          [&](int i, const Frag<P>& x) {
            if (i & 1) dp = mma(x, v[i >> 1], dp);
            else s = mma(x, k[i >> 1], s);
          });
      const f32x16 ls = by_row(now.lse + 32 * b, lane);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], p.c, -ls[i]));
        dp[i] *= s[i];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float e[8];
        Frag<P> f[2];   // bf16: P and dS rounded for their products
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = s[8 * t + i];
        to_frag(e, f[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = dp[8 * t + i];
        to_frag(e, f[1]);
        ahead<D / 16, W, Frag<P>>(
            [&](int i) {
              return i & 1 ? qt.columns(32 * b + 16 * t, i >> 1, lane) : gt.columns(32 * b + 16 * t, i >> 1, lane);
            },
            [&](int i, const Frag<P>& x) {
              if (i & 1) dk[i >> 1] = mma(x, f[1], dk[i >> 1]);
              else dv[i >> 1] = mma(x, f[0], dv[i >> 1]);
            });
      }
    }
  };
  if constexpr (BUF == 2) walk<2, TQ>(r0, r1, first, second, use);
  else walk<1, TQ>(r0, r1, first, first, use);

  if (!key) return;
  if (p.splits_kv > 1) {
    const int width = a.dim_qk + a.dim_v;
    float* to = p.part_kv + (split * (a.num_k * a.heads_kv) + (long)j * a.heads_kv + c) * width;
    const bool vec = a.dim_qk % 4 == 0 && a.dim_v % 4 == 0;
    store_row(to, dk, a.dim_qk, 1.0f, live, vec);
    store_row(to + a.dim_qk, dv, a.dim_v, 1.0f, live, vec);
    return;
  }
  store_row((T*)p.gk + j * p.gk_row + c * p.gk_head, dk, a.dim_qk, a.scale, live, p.vec_st);
  store_row((T*)p.gv + j * p.gv_row + c * p.gv_head, dv, a.dim_v, 1.0f, live, p.vec_st);
}

template <class T, int D, int RW, int TK, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? waves_bwd(sizeof(T) == 4, D) : 1) attn_bwd_q(Params p) {
  __shared__ __attribute__((aligned(16))) KeyBuffer<T, D, TK> first, second;
  const long b = block_index();
  if (b < p.blocks) bwd_q<T, D, RW, TK, BUF, LOAD>(p, where((int)b, p.blocks, p.slots, p.splits), first, second);
}
template <class T, int D, int RW, int TQ, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? waves_kv(sizeof(T) == 4, D) : 1) attn_bwd_kv(Params p) {
  __shared__ __attribute__((aligned(16))) RowBuffer<T, D, TQ> first, second;
  const long b = block_index();
  if (b < p.blocks)
    bwd_kv<T, D, RW, TQ, BUF, LOAD, false>(p, where((int)b, p.blocks, p.slots_kv, p.splits_kv), first, second);
}
template <class T, int D, int RW, int ROWS, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? waves_kv(sizeof(T) == 4, D) : 1) attn_bwd_both(Params p) {
  union Buffer {
    KeyBuffer<T, D, ROWS> keys;
    RowBuffer<T, D, ROWS> rows;
  };
  __shared__ __attribute__((aligned(16))) Buffer first, second;
  const long at = block_index();
  if (at >= p.blocks) return;
  const int b = (int)at, n = p.first_blocks;
  if (b < n)
    bwd_q<T, D, RW, ROWS, BUF, LOAD>(p, where(b, n, p.slots, p.splits), first.keys, second.keys);
  else
    bwd_kv<T, D, RW, ROWS, BUF, LOAD, true>(p, where(b - n, p.blocks - n, p.slots_kv, p.splits_kv), first.rows,
                                           second.rows);
}

// Sums the splits of all three gradients.  `each` elements to a work-group: 256, a thread each,
// or 64, and four waves share each one's splits, eight at a time.
struct Sum {
  const float* part;
  long rows;            // (i, head)
  int width, from, dim; // elements from .. from + dim - 1 of `width`
  int heads, splits, each;
  long blocks;
  float factor;
  void* out;
  long out_row, out_head;
};
struct Sums {
  Sum of[3];
};
template <class T>
__global__ void __launch_bounds__(256) attn_sum(Sums all) {
  __shared__ float red[4][64];
  long b = block_index();
  int which = 0;
  while (which < 2 && b >= all.of[which].blocks) b -= all.of[which++].blocks;
  const Sum& m = all.of[which];
  if (b >= m.blocks) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const bool wide = m.each == 256;
  const long i = b * m.each + (wide ? (int)threadIdx.x : lane), at = i / m.dim;
  const int d = (int)(i - at * m.dim);
  const float* q = m.part + at * m.width + m.from + d;
  const long step = m.rows * m.width;
  float v = 0.0f;
  if (at < m.rows) {
    if (wide) {
#pragma unroll 4
      for (int s = 0; s < m.splits; ++s) v += q[s * step];
    } else {
      int s = w;
      for (; s + 28 < m.splits; s += 32) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = q[(s + 4 * k) * step];
#pragma unroll
        for (int k = 0; k < 8; ++k) v += x[k];
      }
      for (; s < m.splits; s += 4) v += q[s * step];
    }
  }
  if (!wide) {
    red[w][lane] = v;
    __syncthreads();
    if (w > 0) return;
    v = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
  }
  if (at < m.rows)
    ((T*)m.out)[at / m.heads * m.out_row + at % m.heads * m.out_head + d] = (T)(v * m.factor);
}

// The sums that p's splits ask for; none (blocks 0) where there is one split.
Sum sum_of(const float* part, long rows, int width, int from, int dim, int heads, int splits, float factor, void* out,
           long row, long head) {
  Sum m{part, rows, width, from, dim, heads, splits, splits <= 8 ? 256 : 64, 0, factor, out, row, head};
  if (splits > 1) m.blocks = (rows * dim + m.each - 1) / m.each;
  return m;
}
template <class T>
hipError_t sums(const Params& p, hipStream_t s) {
  const e3conv_attention_args& a = p.a;
  const long nq = a.num_q * a.heads_q, nk = a.num_k * a.heads_kv;
  const int width = a.dim_qk + a.dim_v;
  const Sums all{{sum_of(p.part, nq, a.dim_qk, 0, a.dim_qk, a.heads_q, p.splits, a.scale, p.gq, p.gq_row, p.gq_head),
                  sum_of(p.part_kv, nk, width, 0, a.dim_qk, a.heads_kv, p.splits_kv, a.scale, p.gk, p.gk_row, p.gk_head),
                  sum_of(p.part_kv, nk, width, a.dim_qk, a.dim_v, a.heads_kv, p.splits_kv, 1.0f, p.gv, p.gv_row,
                         p.gv_head)}};
  const long blocks = all.of[0].blocks + all.of[1].blocks + all.of[2].blocks;
  if (blocks > 0) hipLaunchKernelGGL(attn_sum<T>, grid_of(blocks), dim3(256), 0, s, all);
  return hipGetLastError();
}

Shape shape_q(const e3conv_attention_args& a) {
  const bool f32 = a.dtype == E3CONV_F32;
  const int dim = a.dim_qk > a.dim_v ? a.dim_qk : a.dim_v;
  return choose(a.num_q * (a.heads_q / a.heads_kv), a.num_k, a.num_graphs, a.heads_kv,
                waves_bwd(f32, padded(dim)), unit_us(f32, dim, true), a.dim_qk);
}
Shape shape_kv(const e3conv_attention_args& a) {
  const bool f32 = a.dtype == E3CONV_F32;
  const int dim = a.dim_qk > a.dim_v ? a.dim_qk : a.dim_v;
  return choose(a.num_k, a.num_q * (a.heads_q / a.heads_kv), a.num_graphs, a.heads_kv,
                waves_kv(f32, padded(dim)), unit_us(f32, dim, true), a.dim_qk + a.dim_v);
}

// Rows of a tile and buffers: 64 and two where they fit 64 KiB of LDS and the registers of two
// waves a SIMD.
template <class T, int D, int LOAD>
struct Tiling {
  static constexpr int ROWS = D == 128 ? 32 : 64;
  static constexpr int BUF4 = 2 * ROWS * planes<T>() * D * 2 * 2 <= 65536 ? 2 : 1;
  static constexpr int BUF1 = sizeof(T) == 2 && LOAD != kElements ? 2 : 1;
};
template <class T, int D, int LOAD>
void launch_q(const Params& p, int rw, hipStream_t s) {
  typedef Tiling<T, D, LOAD> L;
  if (rw == 4) hipLaunchKernelGGL((attn_bwd_q<T, D, 4, L::ROWS, L::BUF4, LOAD>), grid_of(p.blocks), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((attn_bwd_q<T, D, 1, 32, L::BUF1, LOAD>), grid_of(p.blocks), dim3(64), 0, s, p);
}
template <class T, int D, int LOAD>
void launch_kv(const Params& p, int rw, hipStream_t s) {
  typedef Tiling<T, D, LOAD> L;
  constexpr int ROWS = sizeof(T) == 2 ? 64 : L::ROWS;
  if (rw == 4) hipLaunchKernelGGL((attn_bwd_kv<T, D, 4, ROWS, L::BUF4, LOAD>), grid_of(p.blocks), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((attn_bwd_kv<T, D, 1, 32, L::BUF1, LOAD>), grid_of(p.blocks), dim3(64), 0, s, p);
}
template <class T, int D>
void launch_q(const Params& p, int rw, hipStream_t s) {
  if (!p.vec) launch_q<T, D, kElements>(p, rw, s);
  else if (sizeof(T) == 2 && p.full) launch_q<T, D, sizeof(T) == 2 ? kFull : kUnits>(p, rw, s);
  else launch_q<T, D, kUnits>(p, rw, s);
}
template <class T, int D>
void launch_kv(const Params& p, int rw, hipStream_t s) {
  if (!p.vec) launch_kv<T, D, kElements>(p, rw, s);
  else if (sizeof(T) == 2 && p.full) launch_kv<T, D, sizeof(T) == 2 ? kFull : kUnits>(p, rw, s);
  else launch_kv<T, D, kUnits>(p, rw, s);
}

template <class T, int D, int LOAD>
void launch_both(const Params& p, int rw, hipStream_t s) {
  typedef Tiling<T, D, LOAD> L;
  if (rw == 4) hipLaunchKernelGGL((attn_bwd_both<T, D, 4, L::ROWS, L::BUF4, LOAD>), grid_of(p.blocks), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((attn_bwd_both<T, D, 1, 32, L::BUF1, LOAD>), grid_of(p.blocks), dim3(64), 0, s, p);
}
template <class T, int D>
void launch_both(const Params& p, int rw, hipStream_t s) {
  if (!p.vec) launch_both<T, D, kElements>(p, rw, s);
  else if (sizeof(T) == 2 && p.full) launch_both<T, D, sizeof(T) == 2 ? kFull : kUnits>(p, rw, s);
  else launch_both<T, D, kUnits>(p, rw, s);
}

// Whether both kernels go in one launch: work-groups of one size, and either of one wave without
// splits (small graphs), or not more of them than places.
bool together(const e3conv_attention_args& a, const Shape& q, const Shape& kv) {
  if (q.rw != kv.rw) return false;
  const long blocks = ((long)q.slots * q.splits + (long)kv.slots * kv.splits) * a.heads_kv;
  if (q.rw == 1 && q.splits == 1 && kv.splits == 1) return blocks <= 0x7fffffffL;
  const int dim = a.dim_qk > a.dim_v ? a.dim_qk : a.dim_v;
  return blocks <= 256 * (q.rw == 1 ? 4 : waves_kv(a.dtype == E3CONV_F32, padded(dim)));
}

template <class T>
hipError_t backward(Params p, const Shape& q, const Shape& kv, hipStream_t s) {
  const e3conv_attention_args& a = p.a;
  const int dim = a.dim_qk > a.dim_v ? a.dim_qk : a.dim_v;
  p.slots = q.slots;
  p.splits = q.splits;
  p.slots_kv = kv.slots;
  p.splits_kv = kv.splits;
  const long nq = (long)q.slots * q.splits * a.heads_kv, nk = (long)kv.slots * kv.splits * a.heads_kv;
  if (nq > 0x7fffffffL || nk > 0x7fffffffL) return hipErrorInvalidValue;
  if (together(a, q, kv)) {
    p.delta = nullptr;
    p.first_blocks = (int)nq;
    p.blocks = (int)(nq + nk);
    if (dim <= 32) launch_both<T, 32>(p, q.rw, s);
    else if (dim <= 64) launch_both<T, 64>(p, q.rw, s);
    else launch_both<T, 128>(p, q.rw, s);
  } else {
    if (a.num_q > 0) {
      p.blocks = (int)nq;
      if (dim <= 32) launch_q<T, 32>(p, q.rw, s);
      else if (dim <= 64) launch_q<T, 64>(p, q.rw, s);
      else launch_q<T, 128>(p, q.rw, s);
    }
    if (a.num_k > 0) {
      p.blocks = (int)nk;
      if (dim <= 32) launch_kv<T, 32>(p, kv.rw, s);
      else if (dim <= 64) launch_kv<T, 64>(p, kv.rw, s);
      else launch_kv<T, 128>(p, kv.rw, s);
    }
  }
  const hipError_t err = hipGetLastError();
  return err != hipSuccess ? err : sums<T>(p, s);
}

// Floats of the workspace: delta (where the kernels are two), and the partial results.
struct Space {
  size_t delta, q, kv;
};
Space space(const e3conv_attention_args& a, const Shape& q, const Shape& kv) {
  const size_t nq = (size_t)a.num_q * a.heads_q, nk = (size_t)a.num_k * a.heads_kv;
  const auto aligned = [](size_t n) { return (n + 3) / 4 * 4; };
  return {together(a, q, kv) ? 0 : aligned(nq), q.splits > 1 ? aligned(q.splits * nq * a.dim_qk) : 0,
          kv.splits > 1 ? aligned(kv.splits * nk * (a.dim_qk + a.dim_v)) : 0};
}

}  // namespace

size_t backward_workspace(const e3conv_attention_args& a) {
  const Space n = space(a, shape_q(a), shape_kv(a));
  return (n.delta + n.q + n.kv) * sizeof(float);
}

hipError_t launch_backward(const Params& given, hipStream_t s) {
  Params p = given;
  const Shape q = shape_q(p.a), kv = shape_kv(p.a);
  const Space n = space(p.a, q, kv);
  p.part = p.delta + n.delta;
  p.part_kv = p.part + n.q;
  return p.a.dtype == E3CONV_F32 ? backward<float>(p, q, kv, s) : backward<__bf16>(p, q, kv, s);
}

}  // namespace attn
}  // namespace e3c
