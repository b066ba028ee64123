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
// Where graphs have at most 64 rows and keys both run in one launch (attn_bwd_small), the
// second forming delta itself: there the launches are the time (16 us as two, 12 as one
// for 64 graphs of 64 nodes).
#include "attention_tile.h"
#include "kernels.h"

namespace e3c {
namespace attn {
namespace {

template <class T, int D, int RW, int TK, int BUF, bool VEC>
__device__ __forceinline__ void bwd_q(const Params& p, const Where& place) {
  constexpr int P = planes<T>(), KS = D / 16, W = P == 1 ? 4 : 2;   // W: operands read ahead
  struct Buffer {
    Tile<P, TK, D> k, v;
    float bias[TK];
  };
  static_assert(BUF == 2 || !(sizeof(T) == 2 && VEC), "loads straight to LDS need the other buffer");
  __shared__ __attribute__((aligned(16))) Buffer first, second;
  const e3conv_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 31, h = lane >> 5;

  const int split = place.split, slot = place.slot, c = place.c;
  constexpr int BM = 32 * RW;
  const int g = graph_of_slot(a.q_ptr, a.num_graphs, a.num_q, p.group, BM, slot);
  const int q0 = offset(a.q_ptr, g, a.num_q);
  const int nrows = (offset(a.q_ptr, g + 1, a.num_q) - q0) * p.group;
  const int r0 = (slot - first_slot(a.q_ptr, g, a.num_q, p.group, BM)) * BM;
  if (r0 >= nrows) return;

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

  Keys<T, D, TK, 64 * RW, VEC> keys;
  keys.begin(p, c, k0, k1);
  if (k0 < k1) keys.issue(p, first.k, first.v);

  Frag<P> q[KS], go[KS];
  const T* gp = (const T*)p.go + qi * p.go_row + head * p.go_head;
  const T* op = (const T*)p.out + qi * p.out_row + head * p.out_head;
  row_operand<T, D, VEC>((const T*)a.q + qi * a.q_row + head * a.q_head, a.dim_qk, live, q);
  row_operand<T, D, VEC>(gp, a.dim_v, live, go);
  float delta = 0.0f;
#pragma unroll
  for (int t = 0; t < KS; ++t) {
    const int d = 16 * t + 8 * h;
    const Raw<T> gr = fetch8<VEC>(gp, d, a.dim_v), orow = fetch8<VEC>(op, d, a.dim_v);
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
    float* to = p.part + (split * (a.num_q * a.heads_q) + at) * a.dim_qk;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float v[4] = {dq[dt][4 * b], dq[dt][4 * b + 1], dq[dt][4 * b + 2], dq[dt][4 * b + 3]};
        store4(to, 32 * dt + 8 * b + 4 * h, a.dim_qk, v, a.dim_qk % 4 == 0);
      }
    return;
  }
  T* to = (T*)p.gq + qi * p.gq_row + head * p.gq_head;
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = live ? dq[dt][4 * b + i] * a.scale : 0.0f;
      store4(to, 32 * dt + 8 * b + 4 * h, a.dim_qk, v, p.vec_st);
    }
}

template <class T, int D, int RW, int TQ, int BUF, bool VEC, bool OWN>
__device__ __forceinline__ void bwd_kv(const Params& p, const Where& place) {
  constexpr int P = planes<T>(), KS = D / 16, W = P == 1 ? 4 : 2;   // W: operands read ahead
  struct Buffer {
    Tile<P, TQ, D> q, g;
    float lse[TQ], delta[TQ];
  };
  static_assert(BUF == 2 || !(sizeof(T) == 2 && VEC), "loads straight to LDS need the other buffer");
  __shared__ __attribute__((aligned(16))) Buffer first, second;
  const e3conv_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 31, h = lane >> 5;

  const int split = place.split, slot = place.slot, c = place.c;
  constexpr int BN = 32 * RW;
  const int g = graph_of_slot(a.k_ptr, a.num_graphs, a.num_k, 1, BN, slot);
  const int kb = offset(a.k_ptr, g, a.num_k), ke = offset(a.k_ptr, g + 1, a.num_k);
  const int j0 = kb + (slot - first_slot(a.k_ptr, g, a.num_k, 1, BN)) * BN;
  if (j0 >= ke) return;

  const int j = j0 + 32 * w + n;
  const bool key = j < ke, idle = j0 + 32 * w >= ke;   // idle: a wave without keys only loads
  const bool live = key && (!a.k_mask || a.k_mask[j]);

  // this split's rows: whole tiles of the graph's
  const int q0 = offset(a.q_ptr, g, a.num_q);
  const int nrows = (offset(a.q_ptr, g + 1, a.num_q) - q0) * p.group;
  const int tiles = nrows > 0 ? (nrows + TQ - 1) / TQ : 0, per = (tiles + p.splits - 1) / p.splits;
  const int r0 = min(split * per, tiles) * TQ;
  const int r1 = min(nrows, min((split + 1) * per, tiles) * TQ);

  Rows<T, D, TQ, 64 * RW, VEC, OWN> rows;
  rows.begin(p, c, q0, r0, r1);
  if (r0 < r1) rows.issue(p, first.q, first.g);

  Frag<P> k[KS], v[KS];
  const int jr = key ? j : j0;
  row_operand<T, D, VEC>((const T*)a.k + jr * a.k_row + c * a.k_head, a.dim_qk, live, k);
  row_operand<T, D, VEC>((const T*)a.v + jr * a.v_row + c * a.v_head, a.dim_v, live, v);
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
  if (p.splits > 1) {
    const int width = a.dim_qk + a.dim_v;
    float* to = p.part + (split * (a.num_k * a.heads_kv) + (long)j * a.heads_kv + c) * width;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = live ? dk[dt][4 * b + i] : 0.0f;
          y[i] = live ? dv[dt][4 * b + i] : 0.0f;
        }
        const bool vec = a.dim_qk % 4 == 0 && a.dim_v % 4 == 0;
        store4(to, 32 * dt + 8 * b + 4 * h, a.dim_qk, x, vec);
        store4(to + a.dim_qk, 32 * dt + 8 * b + 4 * h, a.dim_v, y, vec);
      }
    return;
  }
  T* tk = (T*)p.gk + j * p.gk_row + c * p.gk_head;
  T* tv = (T*)p.gv + j * p.gv_row + c * p.gv_head;
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = live ? dk[dt][4 * b + i] * a.scale : 0.0f;
        y[i] = live ? dv[dt][4 * b + i] : 0.0f;
      }
      store4(tk, 32 * dt + 8 * b + 4 * h, a.dim_qk, x, p.vec_st);
      store4(tv, 32 * dt + 8 * b + 4 * h, a.dim_v, y, p.vec_st);
    }
}

template <class T, int D, int RW, int TK, int BUF, bool VEC>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? waves_bwd(sizeof(T) == 4, D) : 1) attn_bwd_q(Params p) {
  bwd_q<T, D, RW, TK, BUF, VEC>(p, where(blockIdx.x, gridDim.x, p.slots, p.splits));
}
template <class T, int D, int RW, int TQ, int BUF, bool VEC>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? waves_kv(sizeof(T) == 4, D) : 1) attn_bwd_kv(Params p) {
  bwd_kv<T, D, RW, TQ, BUF, VEC, false>(p, where(blockIdx.x, gridDim.x, p.slots, p.splits));
}
template <class T, int D, bool VEC>
__global__ void __launch_bounds__(64) attn_bwd_small(Params p) {
  constexpr int BUF = sizeof(T) == 2 && VEC ? 2 : 1;
  const int b = blockIdx.x, n = p.first_blocks;
  if (b < n) bwd_q<T, D, 1, 32, BUF, VEC>(p, where(b, n, p.slots, 1));
  else bwd_kv<T, D, 1, 32, BUF, VEC, true>(p, where(b - n, gridDim.x - n, p.slots_kv, 1));
}

// Sums the splits: element d < dim of row (i, head) of `width` floats, times factor.  Four
// waves of a work-group take 64 elements, each a quarter of the splits, eight at a time.
template <class T>
__global__ void __launch_bounds__(256) attn_sum(const float* part, long rows, int width, int from, int dim, int heads,
                                                int splits, float factor, T* out, long out_row, long out_head) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long i = (long)blockIdx.x * 64 + lane;
  const long at = i / dim;
  const int d = (int)(i - at * dim);
  const float* q = part + at * width + from + d;
  float v = 0.0f;
  if (at < rows) {
    int s = w;
    for (; s + 28 < splits; s += 32) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = q[(s + 4 * k) * rows * width];
#pragma unroll
      for (int k = 0; k < 8; ++k) v += x[k];
    }
    for (; s < splits; s += 4) v += q[s * rows * width];
  }
  red[w][lane] = v;
  __syncthreads();
  if (w == 0 && at < rows) {
    v = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
    out[at / heads * out_row + at % heads * out_head + d] = (T)(v * factor);
  }
}

template <class T>
hipError_t sum(const Params& p, long rows, int width, int from, int dim, int heads, float factor, void* out, long row,
               long head, hipStream_t s) {
  const long blocks = (rows * dim + 63) / 64;
  if (blocks > 0x7fffffffL) return hipErrorInvalidValue;
  if (blocks > 0)
    hipLaunchKernelGGL(attn_sum<T>, dim3((unsigned)blocks), dim3(256), 0, s, p.part, rows, width, from, dim, heads,
                       p.splits, factor, (T*)out, row, head);
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

size_t delta_bytes(const e3conv_attention_args& a) {
  return ((size_t)a.num_q * a.heads_q * sizeof(float) + 15) / 16 * 16;
}

// Rows of a tile and buffers: 64 and two where they fit 64 KiB of LDS and the registers of two
// waves a SIMD.
template <class T, int D, bool VEC>
struct Tiling {
  static constexpr int ROWS = D == 128 ? 32 : 64;
  static constexpr int BUF4 = 2 * ROWS * planes<T>() * D * 2 * 2 <= 65536 ? 2 : 1;
  static constexpr int BUF1 = sizeof(T) == 2 && VEC ? 2 : 1;
};
template <class T, int D, bool VEC>
void launch_q(const Params& p, int rw, unsigned grid, hipStream_t s) {
  typedef Tiling<T, D, VEC> L;
  if (rw == 4) hipLaunchKernelGGL((attn_bwd_q<T, D, 4, L::ROWS, L::BUF4, VEC>), dim3(grid), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((attn_bwd_q<T, D, 1, 32, L::BUF1, VEC>), dim3(grid), dim3(64), 0, s, p);
}
template <class T, int D, bool VEC>
void launch_kv(const Params& p, int rw, unsigned grid, hipStream_t s) {
  typedef Tiling<T, D, VEC> L;
  constexpr int ROWS = sizeof(T) == 2 ? 64 : L::ROWS;
  if (rw == 4) hipLaunchKernelGGL((attn_bwd_kv<T, D, 4, ROWS, L::BUF4, VEC>), dim3(grid), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((attn_bwd_kv<T, D, 1, 32, L::BUF1, VEC>), dim3(grid), dim3(64), 0, s, p);
}
template <class T, int D>
void launch_q(const Params& p, int rw, unsigned grid, hipStream_t s) {
  if (p.vec) launch_q<T, D, true>(p, rw, grid, s);
  else launch_q<T, D, false>(p, rw, grid, s);
}
template <class T, int D>
void launch_kv(const Params& p, int rw, unsigned grid, hipStream_t s) {
  if (p.vec) launch_kv<T, D, true>(p, rw, grid, s);
  else launch_kv<T, D, false>(p, rw, grid, s);
}

template <class T, int D>
void launch_small(const Params& p, unsigned grid, hipStream_t s) {
  if (p.vec) hipLaunchKernelGGL((attn_bwd_small<T, D, true>), dim3(grid), dim3(64), 0, s, p);
  else hipLaunchKernelGGL((attn_bwd_small<T, D, false>), dim3(grid), dim3(64), 0, s, p);
}

// Whether both kernels have work-groups of one wave and no splits.
bool small(const e3conv_attention_args& a) {
  const Shape q = shape_q(a), kv = shape_kv(a);
  return q.rw == 1 && kv.rw == 1 && q.splits == 1 && kv.splits == 1 &&
         ((long)q.slots + kv.slots) * a.heads_kv <= 0x7fffffffL;
}

template <class T>
hipError_t backward(Params p, hipStream_t s) {
  const e3conv_attention_args& a = p.a;
  const int dim = a.dim_qk > a.dim_v ? a.dim_qk : a.dim_v;
  if (small(a)) {
    const Shape q = shape_q(a), kv = shape_kv(a);
    p.delta = nullptr;
    p.splits = 1;
    p.slots = q.slots;
    p.slots_kv = kv.slots;
    p.first_blocks = q.slots * a.heads_kv;
    const unsigned grid = (unsigned)(p.first_blocks + kv.slots * a.heads_kv);
    if (dim <= 32) launch_small<T, 32>(p, grid, s);
    else if (dim <= 64) launch_small<T, 64>(p, grid, s);
    else launch_small<T, 128>(p, grid, s);
    return hipGetLastError();
  }
  if (a.num_q > 0) {
    const Shape sh = shape_q(a);
    const long grid = (long)sh.slots * sh.splits * a.heads_kv;
    if (grid > 0x7fffffffL) return hipErrorInvalidValue;
    p.slots = sh.slots;
    p.splits = sh.splits;
    if (dim <= 32) launch_q<T, 32>(p, sh.rw, (unsigned)grid, s);
    else if (dim <= 64) launch_q<T, 64>(p, sh.rw, (unsigned)grid, s);
    else launch_q<T, 128>(p, sh.rw, (unsigned)grid, s);
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && sh.splits > 1)
      err = sum<T>(p, a.num_q * a.heads_q, a.dim_qk, 0, a.dim_qk, a.heads_q, a.scale, p.gq, p.gq_row, p.gq_head, s);
    if (err != hipSuccess) return err;
  }
  if (a.num_k > 0) {
    const Shape sh = shape_kv(a);
    const long grid = (long)sh.slots * sh.splits * a.heads_kv;
    if (grid > 0x7fffffffL) return hipErrorInvalidValue;
    p.slots = sh.slots;
    p.splits = sh.splits;
    if (dim <= 32) launch_kv<T, 32>(p, sh.rw, (unsigned)grid, s);
    else if (dim <= 64) launch_kv<T, 64>(p, sh.rw, (unsigned)grid, s);
    else launch_kv<T, 128>(p, sh.rw, (unsigned)grid, s);
    hipError_t err = hipGetLastError();
    const int width = a.dim_qk + a.dim_v;
    const long rows = a.num_k * a.heads_kv;
    if (err == hipSuccess && sh.splits > 1)
      err = sum<T>(p, rows, width, 0, a.dim_qk, a.heads_kv, a.scale, p.gk, p.gk_row, p.gk_head, s);
    if (err == hipSuccess && sh.splits > 1)
      err = sum<T>(p, rows, width, a.dim_qk, a.dim_v, a.heads_kv, 1.0f, p.gv, p.gv_row, p.gv_head, s);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace

// delta, then one region for the partial results of either kernel in turn.
size_t backward_workspace(const e3conv_attention_args& a) {
  if (small(a)) return 0;
  const Shape sq = shape_q(a), sk = shape_kv(a);
  const size_t q = sq.splits > 1 ? (size_t)sq.splits * a.num_q * a.heads_q * a.dim_qk : 0;
  const size_t k = sk.splits > 1 ? (size_t)sk.splits * a.num_k * a.heads_kv * (a.dim_qk + a.dim_v) : 0;
  return delta_bytes(a) + (q > k ? q : k) * sizeof(float);
}

hipError_t launch_backward(const Params& given, hipStream_t s) {
  Params p = given;
  p.part = p.delta + delta_bytes(p.a) / sizeof(float);
  return p.a.dtype == E3CONV_F32 ? backward<float>(p, s) : backward<__bf16>(p, s);
}

}  // namespace attn
}  // namespace e3c
