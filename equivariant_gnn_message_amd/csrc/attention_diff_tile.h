// What the kernels of differential attention share: their parameters, the rows that the reverse pass walks over,
// and the launch shapes.  Tiles, loads and products are those of attention_tile.h; a row of q or k there is two
// heads side by side, the operands of the two softmax maps, D / 2 elements each.
#pragma once

#include "attention_tile.h"

namespace e3c {
namespace attn {

// heads_q, heads_kv: pairs of maps.  dim_qk: of one map.
struct DiffParams : Params {
  const float* lam;                // (heads_q)
  void* second;                    // the second map's result, or NULL
  long second_row, second_head;
  float* glam;                     // (heads_q)
  float* part_lam;                 // (splits slots, heads_q), their sum is -glam
};

// Elements of a pair of maps' operands, or of a row of v: the tile's width.
inline int diff_width(const e3conv_attention_args& a) { return 2 * a.dim_qk <= 64 && a.dim_v <= 64 ? 64 : 128; }

// The tiles of the rows that a work-group of the reverse pass walks over, and for each row the lse of both maps
// (base 2), -delta of the first map, the first's delta less the second's, and -lambda.  A row that sees no key
// or lies beyond the end has lse = +infinity, which makes its P zero.  OWN: the deltas are formed
// here, else they were left in memory.
enum { kLse0, kLse1, kDelta, kLess, kLam, kRowValues };
template <class T, int D, int ROWS, int NT, int LOAD, bool OWN>
struct DiffRows {
  typedef Pair<T, D, ROWS, NT, LOAD, 2> PairT;
  typedef typename PairT::TileT TileT;
  PairT pair;
  float lse0, lse1, delta0, delta1, lam;
  unsigned char m;
  const T *qb, *gb;      // the kv head's first row of the graph
  long at0;              // of the statistics
  int q0, h0, next, end;

  __device__ __forceinline__ void begin(const DiffParams& p, int c, int first_query, int r0, int r1) {
    const e3conv_attention_args& a = p.a;
    q0 = first_query;
    h0 = c * p.group;
    qb = (const T*)a.q + q0 * a.q_row + 2 * h0 * a.q_head;
    gb = (const T*)p.go + q0 * p.go_row + h0 * p.go_head;
    at0 = (long)q0 * a.heads_q + h0;
    next = r0;
    end = r1;
  }
  __device__ __forceinline__ void issue(const DiffParams& p, TileT& qt, TileT& gt) {
    const e3conv_attention_args& a = p.a;
#pragma unroll
    for (int e = 0; e < PairT::E; ++e) {
      const int r = min(next + PairT::row(e), end - 1), i = query_of(p, r), x = r - i * p.group;
      pair.issue(e, qb + i * a.q_row + 2 * x * a.q_head + PairT::first_x(e, a.dim_qk, a.q_head),
                 gb + i * p.go_row + x * p.go_head + PairT::first(e, a.dim_v), a.dim_qk, a.dim_v, qt, gt);
    }
    const int r = min(next + (int)(threadIdx.x & 63), end - 1), i = query_of(p, r), x = r - i * p.group;
    const long at = at0 + (long)i * a.heads_q + x;
    const float2 both = reinterpret_cast<const float2*>(p.lse)[at];
    lse0 = both.x;
    lse1 = both.y;
    lam = p.lam[h0 + x];
    if constexpr (OWN) {
      const T* g = gb + i * p.go_row + x * p.go_head;
      const T* o = (const T*)p.out + (long)(q0 + i) * p.out_row + (h0 + x) * p.out_head;
      const T* o2 = (const T*)p.second + (long)(q0 + i) * p.second_row + (h0 + x) * p.second_head;
      delta0 = delta1 = 0.0f;
      for (int d = 0; d < a.dim_v; d += 8) {
        const Raw<T> u = fetch8<PairT::VEC>(g, d, a.dim_v), v = fetch8<PairT::VEC>(o, d, a.dim_v),
                     w = fetch8<PairT::VEC>(o2, d, a.dim_v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          delta0 = fmaf(u.at(j), v.at(j), delta0);
          delta1 = fmaf(u.at(j), w.at(j), delta1);
        }
      }
      delta0 = fmaf(lam, delta1, delta0);
    } else {
      const float2 d = reinterpret_cast<const float2*>(p.delta)[at];
      delta0 = d.x;
      delta1 = d.y;
    }
    if (a.q_mask) m = a.q_mask[q0 + i];
    next += ROWS;
  }
  // r0: the first row of the issued tile.
  __device__ __forceinline__ void finish(const DiffParams& p, int r0, TileT& qt, TileT& gt,
                                         float (&values)[kRowValues][ROWS]) const {
    const int lane = threadIdx.x & 63;
    const bool sees = lane < ROWS && r0 + lane < end && lse0 != -INFINITY && (!p.a.q_mask || m);
    if (threadIdx.x < ROWS) {
      values[kLse0][lane] = sees ? lse0 * kLog2e : INFINITY;
      values[kLse1][lane] = sees ? lse1 * kLog2e : INFINITY;
      values[kDelta][lane] = sees ? -delta0 : 0.0f;
      values[kLess][lane] = sees ? delta0 - delta1 : 0.0f;
      values[kLam][lane] = sees ? -lam : 0.0f;
    }
    pair.finish(__ballot(sees), p.a.dim_qk, p.a.dim_v, qt, gt);
  }
};

// Half of by_row's values: those of accumulator registers 8 t .. 8 t + 7.
__device__ __forceinline__ void by_half(const float* rows, int t, int lane, float (&v)[8]) {
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const f32x4 r = *reinterpret_cast<const f32x4*>(rows + 8 * (2 * t + x) + 4 * (lane >> 5));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * x + i] = r[i];
  }
}

// Waves of a SIMD that the registers are kept to: forward, grad_q, grad_k with grad_v.
constexpr int diff_waves_fwd(bool f32) { return f32 ? 2 : 3; }
constexpr int diff_waves_q(bool f32, int d) { return f32 ? 1 : 2; }
constexpr int diff_waves_kv(bool f32, int d) { return f32 ? 1 : (d == 64 ? 2 : 1); }

// us of a work-group of four waves for one key or row (as unit_us): two maps beside one product with v.
inline double diff_unit_us(bool f32, int width, bool backward) { return 1.6 * unit_us(f32, width, backward); }

// Launchers.
hipError_t launch_diff_forward(const DiffParams& p, hipStream_t s);
hipError_t launch_diff_backward(const DiffParams& p, hipStream_t s);
size_t diff_forward_workspace(const e3conv_attention_args& a);
size_t diff_backward_workspace(const e3conv_attention_args& a);

}  // namespace attn
}  // namespace e3c
