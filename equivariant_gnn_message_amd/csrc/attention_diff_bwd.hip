// Reverse pass of differential attention on the matrix cores (contract in e3conv.h, tiles in attention_tile.h).
// With P1 and P2 formed again from the logits and both lse, dP = grad_out v^T and delta_m = <grad_out, O_m>,
//     dS1 = P1 (dP - delta1),   dS2 = -lambda P2 (dP - delta2),   dv = (P1 - lambda P2)^T grad_out,
//     dq_m = scale dS_m k_m,    dk_m = scale dS_m^T q_m,          dlambda = -sum_rows sum_keys P2 dP:
// one product for dP and one for dv serve both maps.  As in the plain attention's reverse pass, two kernels, none
// with atomics:
//
// diff_bwd_q   a wave owns 32 rows (of one map with bf16: its sums and operands leave two waves a SIMD) and walks over
//              the keys, rows along the columns.  It starts from deltas of out and O2 (delta1 = <grad_out, out> +
//              lambda delta2), which are off by the rounding of out and O2: where v and grad_out have means by
//              2^-9 of delta with bf16, and dq, a sum over keys whose dS cancel, by that times sum_j P k_j (a
//              hundredth of dq for 20 000 keys).  So it also sums r_m = sum_j P_m (dP - delta_m), which a true
//              delta makes 0, and B_m = sum_j P_m k_m by one product more for each operand of K, and takes
//                dq_m = scale (sum dS_m k_m - r_m B_m),   delta_m + r_m for diff_bwd_kv,
//                dlambda = -sum over the rows of delta2 + r_2;
//              where the keys are split, diff_join_delta adds the r of a row's splits to its deltas;
// diff_bwd_kv  a wave owns 32 keys and walks over the rows of all query heads that share its kv head.
// In fp32, where the work-groups are few, both run in one launch (diff_bwd_both), the second forming the deltas of out and
// O2 itself: their rounding of 2^-24 is that of dP's own dot product.  With bf16 it is not, so grad_k waits for the deltas:
// with v and grad_out of mean 2 the error of grad_k (rms) is 2.0e-3 instead of 3.8e-3 for 64 graphs of 64 nodes, for 2.6 us
// (21.1 -> 23.7), and 2.3e-3 instead of 3.6e-3 for three rows of 20 011 keys.
// 50 000 nodes in ragged graphs, four heads of two maps of 64 over two kv heads, dim_v 128, bf16: 332 us for grad_q
// (matrix 39 %, vector 46 % of the SIMD cycles) and 469 us for the others (29 % and 41 %); 20 000 nodes in one graph, two
// heads of 32 and 64 in fp32: 1914 and 2292 us, 45 % of the cycles products (six for each of fp32).  With two waves a SIMD
// (one in fp32) the chain of products, exponentials and roundings bounds them.
#include "attention_diff_tile.h"
#include "attention_sum.h"
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
  float values[kRowValues][ROWS];
};

// Sums of the rows' values for each of the query heads that share kv head c; all threads of the work-group
// come here.  Row i of the work-group's rows is head (r0 + i) % group; `block` is this wave's, or -1.
template <int BM, int NT>
__device__ __forceinline__ void sum_lam(const DiffParams& p, float* rows, float value, int block, int r0, float* to) {
  if (block >= 0 && (threadIdx.x & 32) == 0) rows[block * 32 + (threadIdx.x & 31)] = value;
  __syncthreads();
  const int first = r0 - query_of(p, r0) * p.group;
  for (int x = threadIdx.x; x < p.group; x += NT) {
    float v = 0.0f;
    for (int i = x >= first ? x - first : x - first + p.group; i < BM; i += p.group) v += rows[i];
    to[x] = v;
  }
}

// Of P for B alone: its leading part is enough (B is multiplied by r, a rounding error).
template <int P>
__device__ __forceinline__ f32x16 mma_leading(const Frag<P>& a, const Frag<1>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}

template <class T, int D, int RW, int TK, int BUF, int LOAD>
__device__ __forceinline__ void bwd_q(const DiffParams& p, const Where& place, KeyBuffer<T, D, TK>& first,
                                      KeyBuffer<T, D, TK>& second, float* lam_rows) {
  typedef KeyBuffer<T, D, TK> Buffer;
  static_assert(BUF == 2 || !(sizeof(T) == 2 && LOAD != kElements), "loads straight to LDS need the other buffer");
  constexpr int P = planes<T>(), KS = D / 32, VS = D / 16, W = P == 1 ? 4 : 2;   // W: operands read ahead
  constexpr int NM = diff_maps(P == 3, D, RW), DT = D / 64;
  const e3conv_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, n = lane & 31, h = lane >> 5;
  const int map0 = NM == 1 ? w & 1 : 0, block = NM == 1 ? w >> 1 : w;

  const int split = place.split, slot = place.slot, c = place.c;
  constexpr int BM = 32 * RW * NM / 2;
  const int g = graph_of_slot(a.q_ptr, a.num_graphs, a.num_q, p.group, BM, slot);
  const int q0 = offset(a.q_ptr, g, a.num_q);
  const int nrows = (offset(a.q_ptr, g + 1, a.num_q) - q0) * p.group;
  const int r0 = tile_start(slot, first_slot(a.q_ptr, g, a.num_q, p.group, BM), BM, nrows);
  float* const lam_to = p.part_lam + ((long)split * p.slots + slot) * a.heads_q + c * p.group;
  if (r0 < 0) {
    for (int x = threadIdx.x; x < p.group; x += 64 * RW) lam_to[x] = 0.0f;
    return;
  }

  const int r = r0 + 32 * block + n;
  const bool row = r < nrows, idle = r0 + 32 * block >= nrows;   // idle: a wave without rows only loads
  const int qi = q0 + (row ? query_of(p, r) : 0), head = c * p.group + (row ? r - (qi - q0) * p.group : 0);
  const long at = (long)qi * a.heads_q + head;
  const float2 both = reinterpret_cast<const float2*>(p.lse)[at];
  const float lam = p.lam[head];
  const bool live = row && (!a.q_mask || a.q_mask[qi]) && both.x != -INFINITY;

  const int kb = offset(a.k_ptr, g, a.num_k), ke = offset(a.k_ptr, g + 1, a.num_k);
  const int tiles = ke > kb ? (ke - kb + TK - 1) / TK : 0, per = (tiles + p.splits - 1) / p.splits;
  const int k0 = kb + min(split * per, tiles) * TK;
  const int k1 = min(ke, kb + min((split + 1) * per, tiles) * TK);

  DiffKeys<T, D, TK, 64 * RW, LOAD> keys;
  keys.begin(p, c, k0, k1);
  keys.pair.clear(a.dim_qk, a.dim_v, first.k, first.v);
  if (BUF == 2) keys.pair.clear(a.dim_qk, a.dim_v, second.k, second.v);
  if (k0 < k1) keys.issue(p, first.k, first.v);

  Frag<P> q[NM][KS], go[VS];
  const T* gp = (const T*)p.go + qi * p.go_row + head * p.go_head;
  const T* op = (const T*)p.out + qi * p.out_row + head * p.out_head;
  const T* sp = (const T*)p.second + qi * p.second_row + head * p.second_head;
#pragma unroll
  for (int x = 0; x < NM; ++x) {
    row_operand<T, D / 2, LOAD>((const T*)a.q + qi * a.q_row + (2 * head + map0 + x) * a.q_head, a.dim_qk, live, q[x]);
    if (p.negate)
#pragma unroll
      for (int t = 0; t < KS; ++t) flip_sign(q[x][t]);
  }
  row_operand<T, D, LOAD>(gp, a.dim_v, live, go);
  float delta0 = 0.0f, delta1 = 0.0f;
#pragma unroll
  for (int t = 0; t < VS; ++t) {
    const int d = 16 * t + 8 * h;
    const Raw<T> gr = fetch8<LOAD != kElements>(gp, d, a.dim_v), orow = fetch8<LOAD != kElements>(op, d, a.dim_v),
                 srow = fetch8<LOAD != kElements>(sp, d, a.dim_v);
    if (d < a.dim_v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        delta0 = fmaf(gr.at(i), orow.at(i), delta0);
        delta1 = fmaf(gr.at(i), srow.at(i), delta1);
      }
  }
  delta1 = live ? delta1 + other_half(delta1) : 0.0f;
  delta0 = live ? fmaf(lam, delta1, delta0 + other_half(delta0)) : 0.0f;
  float lse[NM], delta[NM], rest[NM];
#pragma unroll
  for (int x = 0; x < NM; ++x) {
    lse[x] = !live ? 0.0f : (map0 + x == 0 ? both.x : both.y) * kLog2e;
    delta[x] = map0 + x == 0 ? delta0 : delta1;
    rest[x] = 0.0f;
  }

  f32x16 dq[NM][DT], bar[NM][DT];
#pragma unroll
  for (int x = 0; x < NM; ++x)
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) dq[x][dt] = bar[x][dt] = f32x16{};

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
      f32x16 s[NM], dp = f32x16{};
      s[0] = by_row(now.bias + 32 * b, lane);
      if (NM == 2) s[NM - 1] = s[0];
      // operands of K and V in turn; with one map K has half as many
      constexpr int N = NM == 2 ? 2 * VS : VS + KS;
      const auto is_v = [](int i) { return NM == 2 ? i & 1 : i % 3 > 0; };
      const auto index = [](int i) { return NM == 2 ? i >> 1 : i % 3 > 0 ? i / 3 * 2 + i % 3 - 1 : i / 3; };
      ahead<N, W, Frag<P>>(
          [&](int i) {
            return is_v(i) ? vt.rows(32 * b, index(i), lane) : kt.rows(32 * b, map0 * KS + index(i), lane);
          },
          [&](int i, const Frag<P>& y) {
            const int j = index(i);
            if (is_v(i)) dp = mma(y, go[j], dp);
            else s[j / KS] = mma(y, q[j / KS][j % KS], s[j / KS]);
          });
      // the first operands of K come while dS is formed
      Ahead<2 * NM * DT, W, Frag<P>> keys_of;
      const auto load = [&](int i) {
        return kt.columns(32 * b + 16 * (i / (NM * DT)), map0 * DT + i % (NM * DT), lane);
      };
      keys_of.start(load);
      Frag<P> f[NM][2];   // bf16: dS rounded for its product
      Frag<1> prob[NM][2];
#pragma unroll
      for (int x = 0; x < NM; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float e[8], pr[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int y = 8 * t + i;
            pr[i] = __builtin_amdgcn_exp2f(fmaf(s[x][y], p.c, -lse[x]));
            const float less = dp[y] - delta[x];
            rest[x] = fmaf(pr[i], less, rest[x]);     // explicit: every form of the loads gives the same bits
            e[i] = pr[i] * less;
          }
          to_frag(e, f[x][t]);
          to_frag(pr, prob[x][t]);
        }
      keys_of.run(load, [&](int i, const Frag<P>& y) {
        const int t = i / (NM * DT), dt = i % (NM * DT), x = dt / DT, d = dt % DT;
        dq[x][d] = mma(y, f[x][t], dq[x][d]);
        bar[x][d] = mma_leading(y, prob[x][t], bar[x][d]);
      });
    }
  };
  if constexpr (BUF == 2) walk<2, TK>(k0, k1, first, second, use);
  else walk<1, TK>(k0, k1, first, first, use);

#pragma unroll
  for (int x = 0; x < NM; ++x) rest[x] += other_half(rest[x]);
  const float of_lam = split == 0 ? delta[NM - 1] + rest[NM - 1] : rest[NM - 1];
  sum_lam<BM, 64 * RW>(p, lam_rows, live ? of_lam : 0.0f, map0 + NM == 2 ? block : -1, r0, lam_to);
  if (!row) return;
#pragma unroll
  for (int x = 0; x < NM; ++x) {
    const int m = map0 + x;
    const float factor = m == 0 ? 1.0f : -lam;      // dS2 without its -lambda above
    // a split's r is not the row's: the joins take the row's off, of grad_q and of the deltas
    if (p.delta && h == 0 && split == 0) p.delta[2 * at + m] = p.splits > 1 || !live ? delta[x] : delta[x] + rest[x];
    if (p.splits > 1) {
      const long i = (split * (a.num_q * a.heads_q) + at) * 2 + m;
      float* to = p.part + i * 2 * a.dim_qk;
      store_row(to, dq[x], a.dim_qk, factor, live, a.dim_qk % 4 == 0);
      store_row(to + a.dim_qk, bar[x], a.dim_qk, factor, live, a.dim_qk % 4 == 0);
      if (h == 0) p.part_rest[i] = live ? rest[x] : 0.0f;
    } else {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[x][dt][i] = fmaf(-rest[x], bar[x][dt][i], dq[x][dt][i]);
      store_row((T*)p.gq + qi * p.gq_row + (2 * head + m) * p.gq_head, dq[x], a.dim_qk, a.scale * factor, live, p.vec_st);
    }
  }
}

// What a work-group forms of its keys: both gradients, or one of them (the products with q, and the exponentials,
// are then formed twice).
enum Role { kBothGrads, kGradK, kGradV };
template <class T, int D, int RW, int TQ, int BUF, int LOAD, bool OWN, Role ROLE>
__device__ __forceinline__ void bwd_kv(const DiffParams& p, const Where& place, RowBuffer<T, D, TQ>& first,
                                       RowBuffer<T, D, TQ>& second) {
  typedef RowBuffer<T, D, TQ> Buffer;
  static_assert(BUF == 2 || !(sizeof(T) == 2 && LOAD != kElements), "loads straight to LDS need the other buffer");
  constexpr int P = planes<T>(), KS = D / 32, VS = D / 16, W = P == 1 ? 4 : 2;   // W: operands read ahead
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

  DiffRows<T, D, TQ, 64 * RW, LOAD, OWN> rows;
  rows.begin(p, c, q0, r0, r1);
  rows.pair.clear(a.dim_qk, a.dim_v, first.q, first.g);
  if (BUF == 2) rows.pair.clear(a.dim_qk, a.dim_v, second.q, second.g);
  if (r0 < r1) rows.issue(p, first.q, first.g);

  Frag<P> k[2][KS], v[VS];
  const int jr = key ? j : j0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    row_operand<T, D / 2, LOAD>((const T*)a.k + jr * a.k_row + (2 * c + x) * a.k_head, a.dim_qk, live, k[x]);
    if (p.negate)
#pragma unroll
      for (int t = 0; t < KS; ++t) flip_sign(k[x][t]);
  }
  if (ROLE != kGradV) row_operand<T, D, LOAD>((const T*)a.v + jr * a.v_row + c * a.v_head, a.dim_v, live, v);

  f32x16 dk[2][D / 64], dv[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 64; ++dt) dk[0][dt] = dk[1][dt] = f32x16{};
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) dv[dt] = f32x16{};

  const auto use = [&](Buffer& now, int from, Buffer& next) {
    Tile<P, TQ, D>&qt = now.q, &gt = now.g;
    if (BUF == 1) __syncthreads();
    rows.finish(p, from, qt, gt, now.values);
    __syncthreads();
    if (from + TQ < r1) rows.issue(p, next.q, next.g);
    if (idle) return;

#pragma unroll
    for (int b = 0; b < TQ / 32; ++b) {
      if (b > 0 && from + 32 * b >= r1) break;
      // dP - delta1 from the start: the rows' -delta1 are the accumulator's first values
      f32x16 s[2], dp;
      s[0] = s[1] = f32x16{};
      if constexpr (ROLE == kGradV) {
        ahead<VS, W, Frag<P>>([&](int i) { return qt.rows(32 * b, (i & 1) * KS + (i >> 1), lane); },
                              [&](int i, const Frag<P>& y) { s[i & 1] = mma(y, k[i & 1][i >> 1], s[i & 1]); });
      } else {
        dp = by_row(now.values[kDelta] + 32 * b, lane);
        ahead<2 * VS, W, Frag<P>>(
            [&](int i) { return i & 1 ? gt.rows(32 * b, i >> 1, lane) : qt.rows(32 * b, i >> 1, lane); },
            [&](int i, const Frag<P>& y) {
              const int x = i >> 1;
              if (i & 1) dp = mma(y, v[x], dp);
              else s[x / KS] = mma(y, k[x / KS][x % KS], s[x / KS]);
            });
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float e[3][8], lse0[8], lse1[8], lam[8], less[8];
        Frag<P> f[3];   // bf16: both dS and P1 - lambda P2 rounded for their products
        by_half(now.values[kLse0] + 32 * b, t, lane, lse0);
        by_half(now.values[kLse1] + 32 * b, t, lane, lse1);
        by_half(now.values[kLam] + 32 * b, t, lane, lam);
        if (ROLE != kGradV) by_half(now.values[kLess] + 32 * b, t, lane, less);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int y = 8 * t + i;
          const float p0 = __builtin_amdgcn_exp2f(fmaf(s[0][y], p.c, -lse0[i]));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(s[1][y], p.c, -lse1[i]));
          if (ROLE != kGradV) {
            e[0][i] = p0 * dp[y];
            e[1][i] = p1 * lam[i] * (dp[y] + less[i]);
          }
          if (ROLE != kGradK) e[2][i] = fmaf(p1, lam[i], p0);
        }
#pragma unroll
        for (int x = 0; x < 3; ++x)
          if (x < 2 ? ROLE != kGradV : ROLE != kGradK) to_frag(e[x], f[x]);
        const auto add_k = [&](int dt, const Frag<P>& y) {
          const int x = dt / (D / 64), d = dt % (D / 64);
          dk[x][d] = mma(y, f[x], dk[x][d]);
        };
        const auto add_v = [&](int dt, const Frag<P>& y) { dv[dt] = mma(y, f[2], dv[dt]); };
        const auto of_q = [&](int dt) { return qt.columns(32 * b + 16 * t, dt, lane); };
        const auto of_g = [&](int dt) { return gt.columns(32 * b + 16 * t, dt, lane); };
        if constexpr (ROLE == kGradK) ahead<D / 32, W, Frag<P>>(of_q, add_k);
        else if constexpr (ROLE == kGradV) ahead<D / 32, W, Frag<P>>(of_g, add_v);
        else
          ahead<D / 16, W, Frag<P>>([&](int i) { return i & 1 ? of_q(i >> 1) : of_g(i >> 1); },
                                    [&](int i, const Frag<P>& y) {
                                      if (i & 1) add_k(i >> 1, y);
                                      else add_v(i >> 1, y);
                                    });
      }
    }
  };
  if constexpr (BUF == 2) walk<2, TQ>(r0, r1, first, second, use);
  else walk<1, TQ>(r0, r1, first, first, use);

  if (!key) return;
  if (p.splits_kv > 1) {
    const int width = 2 * a.dim_qk + a.dim_v;
    float* to = p.part_kv + (split * (a.num_k * a.heads_kv) + (long)j * a.heads_kv + c) * width;
    const bool vec = a.dim_qk % 4 == 0 && a.dim_v % 4 == 0;
    if (ROLE != kGradV) {
      store_row(to, dk[0], a.dim_qk, 1.0f, live, vec);
      store_row(to + a.dim_qk, dk[1], a.dim_qk, 1.0f, live, vec);
    }
    if (ROLE != kGradK) store_row(to + 2 * a.dim_qk, dv, a.dim_v, 1.0f, live, vec);
    return;
  }
  if (ROLE != kGradV)
#pragma unroll
    for (int x = 0; x < 2; ++x)
      store_row((T*)p.gk + j * p.gk_row + (2 * c + x) * p.gk_head, dk[x], a.dim_qk, a.scale, live, p.vec_st);
  if (ROLE != kGradK) store_row((T*)p.gv + j * p.gv_row + c * p.gv_head, dv, a.dim_v, 1.0f, live, p.vec_st);
}

template <class T, int D, int RW, int TK, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? diff_waves_q(sizeof(T) == 4, D) : 1) diff_bwd_q(DiffParams p) {
  __shared__ __attribute__((aligned(16))) KeyBuffer<T, D, TK> first, second;
  __shared__ float lam_rows[32 * RW];
  const long b = block_index();
  if (b < p.blocks)
    bwd_q<T, D, RW, TK, BUF, LOAD>(p, where<kRun>((int)b, p.blocks, p.slots, p.splits), first, second, lam_rows);
}
template <class T, int D, int RW, int TQ, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, RW == 4 ? diff_waves_kv(sizeof(T) == 4, D) : 1) diff_bwd_kv(DiffParams p) {
  __shared__ __attribute__((aligned(16))) RowBuffer<T, D, TQ> first, second;
  const long b = block_index();
  if (b >= p.blocks) return;
  if constexpr (diff_two_roles(sizeof(T) == 4, D, RW)) {
    const int n = p.blocks / 2;
    if (b < n)
      bwd_kv<T, D, RW, TQ, BUF, LOAD, false, kGradK>(p, where<kRun>((int)b, n, p.slots_kv, p.splits_kv), first, second);
    else
      bwd_kv<T, D, RW, TQ, BUF, LOAD, false, kGradV>(p, where<kRun>((int)b - n, n, p.slots_kv, p.splits_kv), first, second);
  } else {
    bwd_kv<T, D, RW, TQ, BUF, LOAD, false, kBothGrads>(p, where<kRun>((int)b, p.blocks, p.slots_kv, p.splits_kv), first, second);
  }
}
// delta + r of each row and map whose keys are split, the splits' r in a fixed order: as many threads to a value as it
// has splits, up to a wave (80 000 values of four splits: 15.4 us with a wave each, 4.6 so).
inline int join_threads_log2(int splits) {
  int n = 0;
  while (n < 6 && (1 << n) < splits) ++n;
  return n;
}
__global__ void __launch_bounds__(256) diff_join_delta(DiffParams p, int threads_log2) {
  const int threads = 1 << threads_log2, lane = threadIdx.x & (threads - 1);
  const long n = 2 * p.a.num_q * p.a.heads_q, i = (block_index() * 256 + threadIdx.x) >> threads_log2;
  if (i >= n) return;
  float r = 0.0f;
#pragma unroll 4
  for (int s = lane; s < p.splits; s += threads) r += p.part_rest[s * n + i];
  for (int o = threads >> 1; o > 0; o >>= 1) r += __shfl_xor(r, o);
  if (lane == 0) p.delta[i] += r;
}
template <class T, int D, int RW, int ROWS, int BUF, int LOAD>
__global__ void __launch_bounds__(64 * RW, 1) diff_bwd_both(DiffParams p) {
  union Buffer {
    KeyBuffer<T, D, ROWS> keys;
    RowBuffer<T, D, ROWS> rows;
  };
  __shared__ __attribute__((aligned(16))) Buffer first, second;
  __shared__ float lam_rows[32 * RW];
  const long at = block_index();
  if (at >= p.blocks) return;
  const int b = (int)at, n = p.first_blocks;
  if (b < n)
    bwd_q<T, D, RW, ROWS, BUF, LOAD>(p, where<kRun>(b, n, p.slots, p.splits), first.keys, second.keys, lam_rows);
  else
    bwd_kv<T, D, RW, ROWS, BUF, LOAD, true, kBothGrads>(p, where<kRun>(b - n, p.blocks - n, p.slots_kv, p.splits_kv),
                                                        first.rows, second.rows);
}

template <class T>
hipError_t sums(const DiffParams& p, hipStream_t s) {
  const e3conv_attention_args& a = p.a;
  const long nq = a.num_q * a.heads_q, nk = a.num_k * a.heads_kv;
  const int width = 2 * a.dim_qk + a.dim_v;
  Sums all{{sum_of(p.part, 2 * nq, 2 * a.dim_qk, 0, a.dim_qk, 1, 2 * a.heads_q, p.splits, a.scale, p.gq, p.gq_row,
                   p.gq_head, p.part_rest),
            sum_of(p.part_kv, nk, width, 0, 2 * a.dim_qk, 2, a.heads_kv, p.splits_kv, a.scale, p.gk, p.gk_row, p.gk_head),
            sum_of(p.part_kv, nk, width, 2 * a.dim_qk, a.dim_v, 1, a.heads_kv, p.splits_kv, 1.0f, p.gv, p.gv_row,
                   p.gv_head)}};
  long blocks = all.of[0].blocks + all.of[1].blocks + all.of[2].blocks;
  if (p.glam) {
    all.lam = p.part_lam;
    all.lams = a.num_q > 0 ? p.slots * p.splits : 0;
    all.heads = a.heads_q;
    all.glam = p.glam;
    blocks += all.heads;
  }
  if (blocks > 0) hipLaunchKernelGGL(attn_sum<T>, grid_of(blocks), dim3(256), 0, s, all);
  return hipGetLastError();
}

// Small graphs leave most of the chip idle, and a launch that adds parts (lambda's) follows in any case: the other axis
// is split down to its tiles of 32 while all work-groups of both kernels find a place (64 graphs of 64 nodes, fp32:
// 17.8 -> 14.6 us).
Shape split_small(Shape s, long others, int graphs, int heads) {
  const long g = graphs > 0 ? graphs : 1, tiles = ((others + g - 1) / g + 31) / 32;
  if (s.rw == 1 && s.splits == 1)
    while (2 * s.splits <= tiles && 2l * s.splits * s.slots * heads <= 512) s.splits *= 2;
  return s;
}
Shape shape_q(const e3conv_attention_args& a) {
  const bool f32 = a.dtype == E3CONV_F32;
  const int width = diff_width(a), wide = 2 * diff_maps(f32, width, 4);    // blocks of 32 rows of four waves
  const Shape s = choose(a.num_q * (a.heads_q / a.heads_kv), a.num_k, a.num_graphs, a.heads_kv, diff_waves_q(f32, width),
                         diff_unit_us(f32, width, true) * wide / 4, 4 * a.dim_qk, wide);
  // with bf16 split keys would ask for one launch more, diff_join_delta (64 graphs of 64 nodes 23.7 -> 26.8 us)
  return f32 ? split_small(s, a.num_k, a.num_graphs, a.heads_kv) : s;
}
Shape shape_kv(const e3conv_attention_args& a) {
  const bool f32 = a.dtype == E3CONV_F32;
  const int width = diff_width(a);
  const long rows = a.num_q * (a.heads_q / a.heads_kv);
  return split_small(choose(a.num_k, rows, a.num_graphs, a.heads_kv, diff_waves_kv(f32, width),
                            diff_unit_us(f32, width, true), 2 * a.dim_qk + a.dim_v), rows, a.num_graphs, a.heads_kv);
}

// Rows of a tile and buffers: 64 and two where they fit 64 KiB of LDS and the registers.
template <class T, int D, int LOAD>
struct Tiling {
  static constexpr int ROWS = D == 128 ? 32 : 64;
  static constexpr int BUF4 = 2 * ROWS * planes<T>() * D * 2 * 2 <= 65536 ? 2 : 1;
  static constexpr int BUF1 = sizeof(T) == 2 && LOAD != kElements ? 2 : 1;
  static constexpr int LEAST = diff_maps(sizeof(T) == 4, D, 2) == 1 ? 2 : 1;   // waves of 32 rows
};
enum Which { kQ, kKv, kBoth };
template <class T, int D, int LOAD>
void launch(const DiffParams& p, Which which, int rw, hipStream_t s) {
  typedef Tiling<T, D, LOAD> L;
  const dim3 grid = grid_of(p.blocks);
  if (which == kQ) {
    if (rw == 4) hipLaunchKernelGGL((diff_bwd_q<T, D, 4, L::ROWS, L::BUF4, LOAD>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((diff_bwd_q<T, D, L::LEAST, 32, L::BUF1, LOAD>), grid, dim3(64 * L::LEAST), 0, s, p);
  } else if (which == kKv) {
    if (rw == 4) hipLaunchKernelGGL((diff_bwd_kv<T, D, 4, L::ROWS, L::BUF4, LOAD>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((diff_bwd_kv<T, D, 1, 32, L::BUF1, LOAD>), grid, dim3(64), 0, s, p);
  } else if constexpr (sizeof(T) == 4) {
    if (rw == 4) hipLaunchKernelGGL((diff_bwd_both<T, D, 4, L::ROWS, L::BUF4, LOAD>), grid, dim3(256), 0, s, p);
    else if constexpr (L::LEAST == 1)
      hipLaunchKernelGGL((diff_bwd_both<T, D, 1, 32, L::BUF1, LOAD>), grid, dim3(64), 0, s, p);
  }
}
template <class T, int D>
void by_load(const DiffParams& p, Which which, int rw, hipStream_t s) {
  if (!p.vec) launch<T, D, kElements>(p, which, rw, s);
  else if (sizeof(T) == 2 && p.full) launch<T, D, sizeof(T) == 2 ? kFull : kUnits>(p, which, rw, s);
  else launch<T, D, kUnits>(p, which, rw, s);
}
template <class T>
void by_width(const DiffParams& p, Which which, int rw, hipStream_t s) {
  if (diff_width(p.a) == 64) by_load<T, 64>(p, which, rw, s);
  else by_load<T, 128>(p, which, rw, s);
}

// Whether both kernels go in one launch: fp32, work-groups of one size, and either of one wave without
// splits (small graphs), or not more of them than places.
bool together(const e3conv_attention_args& a, const Shape& q, const Shape& kv) {
  if (a.dtype != E3CONV_F32 || (q.rw == 1) != (kv.rw == 1)) return false;
  if (q.rw == 1 && diff_maps(true, diff_width(a), 2) == 1) return false;
  const long blocks = ((long)q.slots * q.splits + (long)kv.slots * kv.splits) * a.heads_kv;
  if (q.rw == 1 && q.splits == 1 && kv.splits == 1) return blocks <= 0x7fffffffL;
  return blocks <= 256 * (q.rw == 1 ? 4 : 1);
}

template <class T>
hipError_t backward(DiffParams p, const Shape& q, const Shape& kv, hipStream_t s) {
  const e3conv_attention_args& a = p.a;
  p.slots = q.slots;
  p.splits = q.splits;
  p.slots_kv = kv.slots;
  p.splits_kv = kv.splits;
  const long nq = (long)q.slots * q.splits * a.heads_kv, nk = (long)kv.slots * kv.splits * a.heads_kv;
  if (nq > 0x7fffffffL || nk > 0x3fffffffL) return hipErrorInvalidValue;
  if (together(a, q, kv)) {
    p.delta = nullptr;
    p.first_blocks = (int)nq;
    p.blocks = (int)(nq + nk);
    if (p.blocks > 0) by_width<T>(p, kBoth, kv.rw, s);     // none without graphs
  } else {
    if (a.num_q > 0) {
      p.blocks = (int)nq;
      by_width<T>(p, kQ, q.rw == 1 ? 1 : 4, s);
      if (q.splits > 1 && a.num_k > 0) {
        const int threads_log2 = join_threads_log2(q.splits);
        hipLaunchKernelGGL(diff_join_delta, grid_of((((2l * a.num_q * a.heads_q) << threads_log2) + 255) / 256), dim3(256),
                           0, s, p, threads_log2);
      }
    }
    if (a.num_k > 0) {
      p.blocks = (int)nk * (diff_two_roles(sizeof(T) == 4, diff_width(a), kv.rw) ? 2 : 1);
      by_width<T>(p, kKv, kv.rw, s);
    }
  }
  const hipError_t err = hipGetLastError();
  return err != hipSuccess ? err : sums<T>(p, s);
}

// Floats of the workspace: the deltas (where the kernels are two), the partial results, and lambda's.
struct Space {
  size_t delta, q, rest, kv, lam;
};
Space space(const e3conv_attention_args& a, const Shape& q, const Shape& kv) {
  const size_t nq = (size_t)a.num_q * a.heads_q, nk = (size_t)a.num_k * a.heads_kv;
  const auto aligned = [](size_t n) { return (n + 3) / 4 * 4; };
  return {together(a, q, kv) ? 0 : aligned(2 * nq), q.splits > 1 ? aligned(q.splits * nq * 4 * a.dim_qk) : 0,
          q.splits > 1 ? aligned(q.splits * nq * 2) : 0,
          kv.splits > 1 ? aligned(kv.splits * nk * (2 * a.dim_qk + a.dim_v)) : 0,
          aligned((size_t)q.slots * q.splits * a.heads_q)};
}

}  // namespace

size_t diff_backward_workspace(const e3conv_attention_args& a) {
  const Space n = space(a, shape_q(a), shape_kv(a));
  return (n.delta + n.q + n.rest + n.kv + n.lam) * sizeof(float);
}

hipError_t launch_diff_backward(const DiffParams& given, hipStream_t s) {
  DiffParams p = given;
  const Shape q = shape_q(p.a), kv = shape_kv(p.a);
  const Space n = space(p.a, q, kv);
  p.part = p.delta + n.delta;
  p.part_rest = p.part + n.q;
  p.part_kv = p.part_rest + n.rest;
  p.part_lam = p.part_kv + n.kv;
  return p.a.dtype == E3CONV_F32 ? backward<float>(p, q, kv, s) : backward<__bf16>(p, q, kv, s);
}

}  // namespace attn
}  // namespace e3c
