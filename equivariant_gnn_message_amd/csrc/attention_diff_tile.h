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
  float* part_rest;                // (splits, num_q, heads_q, 2): r of the splits
  float* part_lam;                 // (splits slots, heads_q), their sum is -glam
};

// Elements of a pair of maps' operands, or of a row of v: the tile's width.
inline int diff_width(const e3conv_attention_args& a) { return 2 * a.dim_qk <= 64 && a.dim_v <= 64 ? 64 : 128; }

// Loads of a tile's rows of the two operands.  A tile lies at a base that the whole wave shares and advances by scalar
// instructions; a lane adds the offset of its unit of its rows, 32 bits wide and the same for every tile (the
// 64-bit addresses of a tile's loads were a third of the loop's vector instructions).  The last tile's rows,
// and all rows where they lie too far apart (element-wise loads), are addressed one by one.
template <class T, int D, int ROWS, int NT, int LOAD>
struct DiffPair : Pair<T, D, ROWS, NT, LOAD, 2> {
  typedef Pair<T, D, ROWS, NT, LOAD, 2> Base;
  typedef typename Base::TileT TileT;
  static constexpr int E = Base::E, KEPT = Base::SAME ? 1 : E;
  static constexpr bool NEAR = LOAD != kElements;
  unsigned xo[KEPT], yo[KEPT];     // bytes

  __device__ __forceinline__ void offset(int e, long x, long y) {
    if (e < KEPT) {
      xo[e] = (unsigned)(x * (long)sizeof(T));
      yo[e] = (unsigned)(y * (long)sizeof(T));
    }
  }
  // xb, yb: the tile's base.  x_step, y_step: elements between two rows of a thread where it has the same unit of all.
  __device__ __forceinline__ void issue_near(const T* xb, const T* yb, long x_step, long y_step, int dim_x, int dim_y,
                                             TileT& xt, TileT& yt) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = Base::SAME ? 0 : e;
      const char* x = reinterpret_cast<const char*>(xb + (Base::SAME ? e * x_step : 0));
      const char* y = reinterpret_cast<const char*>(yb + (Base::SAME ? e * y_step : 0));
      this->issue(e, reinterpret_cast<const T*>(x + xo[i]), reinterpret_cast<const T*>(y + yo[i]), dim_x, dim_y, xt, yt);
    }
    asm volatile("");      // or the compiler joins these loads with those of the other branch, by 64-bit addresses
  }
};

// Whether rows that 16-byte loads reach lie near enough for those offsets: a tile's rows within 4 GiB.
inline bool near_rows(int64_t row, int64_t head, int size) { return (64 * row + 256 * head) * size < (int64_t)1 << 32 &&
                                                                     row < (int64_t)1 << 32 && head < (int64_t)1 << 32; }

// The tiles of the keys of one kv head, and the starting value of each key's logits: 0, or -infinity for a key that
// is not seen.  Rows beyond the last key read the last one.
template <class T, int D, int ROWS, int NT, int LOAD>
struct DiffKeys {
  typedef DiffPair<T, D, ROWS, NT, LOAD> PairT;
  typedef typename PairT::TileT TileT;
  PairT pair;
  unsigned char m;
  const T *kb, *vb;      // the next tile's first key
  int next, end;         // keys of this work-group not yet loaded

  __device__ __forceinline__ void begin(const Params& p, int c, int k0, int k1) {
    const e3conv_attention_args& a = p.a;
    kb = (const T*)a.k + 2 * c * a.k_head + k0 * a.k_row;
    vb = (const T*)a.v + c * a.v_head + k0 * a.v_row;
#pragma unroll
    for (int e = 0; e < PairT::E; ++e)
      pair.offset(e, PairT::row(e) * a.k_row + PairT::first_x(e, a.dim_qk, a.k_head),
                  PairT::row(e) * a.v_row + PairT::first(e, a.dim_v));
    next = k0;
    end = k1;
  }
  __device__ __forceinline__ void issue(const Params& p, TileT& kt, TileT& vt) {
    const e3conv_attention_args& a = p.a;
    if (PairT::NEAR && next + ROWS <= end) {
      pair.issue_near(kb, vb, PairT::STEP * a.k_row, PairT::STEP * a.v_row, a.dim_qk, a.dim_v, kt, vt);
    } else {
#pragma unroll
      for (int e = 0; e < PairT::E; ++e) {
        const long r = min(end - 1 - next, PairT::row(e));
        pair.issue(e, kb + r * a.k_row + PairT::first_x(e, a.dim_qk, a.k_head), vb + r * a.v_row + PairT::first(e, a.dim_v),
                   a.dim_qk, a.dim_v, kt, vt);
      }
    }
    if (a.k_mask) m = a.k_mask[min(next + (int)(threadIdx.x & 63), end - 1)];
    kb += ROWS * a.k_row;
    vb += ROWS * a.v_row;
    next += ROWS;
  }
  // k0: the first key of the issued tile.
  __device__ __forceinline__ void finish(const Params& p, int k0, TileT& kt, TileT& vt, float* bias) const {
    const int lane = threadIdx.x & 63;
    const bool sees = lane < ROWS && k0 + lane < end && (!p.a.k_mask || m);
    if (threadIdx.x < ROWS) bias[lane] = sees ? 0.0f : -INFINITY;
    pair.finish(__ballot(sees), p.a.dim_qk, p.a.dim_v, kt, vt);
  }
};

// The tiles of the rows that a work-group of the reverse pass walks over, and for each row the lse of both maps
// (base 2), -delta of the first map, the first's delta less the second's, and -lambda.  A row that sees no key
// or lies beyond the end has lse = +infinity, which makes its P zero.  OWN: the deltas are formed
// here, else they were left in memory.
enum { kLse0, kLse1, kDelta, kLess, kLam, kRowValues };
template <class T, int D, int ROWS, int NT, int LOAD, bool OWN>
struct DiffRows {
  typedef DiffPair<T, D, ROWS, NT, LOAD> PairT;
  typedef typename PairT::TileT TileT;
  PairT pair;
  float2 lse, delta;
  float lam;
  unsigned char m;
  const T *qb, *gb;      // the kv head's first row of the next tile's first query (of the graph's first, unless `whole`)
  long at0;              // of the statistics
  int q0, h0, next, end, i0;   // i0: the next tile's first query in the graph
  bool whole;            // tiles hold whole queries: every tile's rows lie alike

  __device__ __forceinline__ void begin(const DiffParams& p, int c, int first_query, int r0, int r1) {
    const e3conv_attention_args& a = p.a;
    q0 = first_query;
    h0 = c * p.group;
    whole = PairT::NEAR && ROWS >> p.group_log2 << p.group_log2 == ROWS;
    i0 = whole ? r0 >> p.group_log2 : 0;
    qb = (const T*)a.q + (long)(q0 + i0) * a.q_row + 2 * h0 * a.q_head;
    gb = (const T*)p.go + (long)(q0 + i0) * p.go_row + h0 * p.go_head;
    at0 = (long)q0 * a.heads_q + h0;
    next = r0;
    end = r1;
#pragma unroll
    for (int e = 0; e < PairT::E; ++e) {
      const int r = PairT::row(e), i = query_of(p, r), x = r - i * p.group;
      pair.offset(e, i * a.q_row + 2 * x * a.q_head + PairT::first_x(e, a.dim_qk, a.q_head),
                  i * p.go_row + x * p.go_head + PairT::first(e, a.dim_v));
    }
  }
  __device__ __forceinline__ void issue(const DiffParams& p, TileT& qt, TileT& gt) {
    const e3conv_attention_args& a = p.a;
    // STEP rows on lie STEP / group queries on where the heads of a group divide STEP
    const int by = PairT::STEP >> p.group_log2;
    if (whole && next + ROWS <= end && (!PairT::SAME || by << p.group_log2 == PairT::STEP)) {
      pair.issue_near(qb, gb, by * a.q_row, by * p.go_row, a.dim_qk, a.dim_v, qt, gt);
    } else {
#pragma unroll
      for (int e = 0; e < PairT::E; ++e) {
        const int r = min(next + PairT::row(e), end - 1), i = query_of(p, r), x = r - i * p.group;
        pair.issue(e, qb + (i - i0) * a.q_row + 2 * x * a.q_head + PairT::first_x(e, a.dim_qk, a.q_head),
                   gb + (i - i0) * p.go_row + x * p.go_head + PairT::first(e, a.dim_v), a.dim_qk, a.dim_v, qt, gt);
      }
    }
    const int r = min(next + (int)(threadIdx.x & 63), end - 1), i = query_of(p, r), x = r - i * p.group;
    const int at = i * a.heads_q + x;                 // below 2^31: all rows and heads are
    lse = reinterpret_cast<const float2*>(p.lse)[at0 + at];
    lam = p.lam[h0 + x];
    if constexpr (OWN) {
      const T* g = (const T*)p.go + (long)(q0 + i) * p.go_row + (h0 + x) * p.go_head;
      const T* o = (const T*)p.out + (long)(q0 + i) * p.out_row + (h0 + x) * p.out_head;
      const T* o2 = (const T*)p.second + (long)(q0 + i) * p.second_row + (h0 + x) * p.second_head;
      delta = make_float2(0.0f, 0.0f);
#pragma unroll 4
      for (int d = 0; d < a.dim_v; d += 8) {
        const Raw<T> u = fetch8<PairT::VEC>(g, d, a.dim_v), v = fetch8<PairT::VEC>(o, d, a.dim_v),
                     w = fetch8<PairT::VEC>(o2, d, a.dim_v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          delta.x = fmaf(u.at(j), v.at(j), delta.x);
          delta.y = fmaf(u.at(j), w.at(j), delta.y);
        }
      }
      delta.x = fmaf(lam, delta.y, delta.x);
    } else {
      delta = reinterpret_cast<const float2*>(p.delta)[at0 + at];
    }
    if (a.q_mask) m = a.q_mask[q0 + i];
    next += ROWS;
    if (whole) {
      const int on = ROWS >> p.group_log2;
      i0 += on;
      qb += on * a.q_row;
      gb += on * p.go_row;
    }
  }
  // r0: the first row of the issued tile.
  __device__ __forceinline__ void finish(const DiffParams& p, int r0, TileT& qt, TileT& gt,
                                         float (&values)[kRowValues][ROWS]) const {
    const int lane = threadIdx.x & 63;
    const bool sees = lane < ROWS && r0 + lane < end && lse.x != -INFINITY && (!p.a.q_mask || m);
    if (threadIdx.x < ROWS) {
      values[kLse0][lane] = sees ? lse.x * kLog2e : INFINITY;
      values[kLse1][lane] = sees ? lse.y * kLog2e : INFINITY;
      values[kDelta][lane] = sees ? -delta.x : 0.0f;
      values[kLess][lane] = sees ? delta.x - delta.y : 0.0f;
      values[kLam][lane] = sees ? -lam : 0.0f;
    }
    pair.finish(__ballot(sees), p.a.dim_qk, p.a.dim_v, qt, gt);
  }
};

// As ahead(), in two parts: the first loads are started before work that needs none of them (a softmax's
// exponentials), and in the second part each operand's successor is loaded as it is used.
template <int N, int W, class F>
struct Ahead {
  F ring[W];
  template <class Load>
  __device__ __forceinline__ void start(Load load) {
#pragma unroll
    for (int i = 0; i < W && i < N; ++i) ring[i] = load(i);
    __builtin_amdgcn_sched_barrier(0x6);
  }
  template <class Load, class Use>
  __device__ __forceinline__ void run(Load load, Use use) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      __builtin_amdgcn_sched_barrier(0x6);
      use(i, ring[i % W]);
      if (i + W < N) ring[i % W] = load(i + W);
    }
    __builtin_amdgcn_sched_barrier(0x6);
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

// Work-groups of neighbouring tiles on one die (where()): of 32, 8 and 1 places, 8 serve both the forward (472, 474,
// 479 us for 100 000 ragged nodes) and the reverse pass (771, 760, 776 us for 50 000), whose work-groups are few.
constexpr int kRun = 8;

// Waves of a SIMD that the registers are kept to: forward, grad_q, grad_k with grad_v.  The bf16 forward's three
// spill 30 registers with 128 dimensions and are faster than two all the same (473 against 495 us for 100 000 ragged nodes);
// two of the fp32 reverse pass need a map, or a gradient, to a wave and lose (20 000 nodes: grad_q 4285 -> 4530 us for
// the whole, grad_k and grad_v 5040).
constexpr int diff_waves_fwd(bool f32) { return f32 ? 2 : 3; }
constexpr int diff_waves_q(bool f32, int d) { return f32 ? 1 : 2; }
constexpr int diff_waves_kv(bool f32, int d) { return f32 ? 1 : 2; }
// Maps of a wave of diff_bwd_q: with one, two waves share 32 rows.  Sums and operands of two maps do not fit the
// registers of two waves a SIMD with bf16, nor those of one with fp32 and 128 dimensions (all others: 64 dimensions in fp32
// take 4285 us for 20 000 nodes with two, 4530 with one).
constexpr int diff_maps(bool f32, int d, int rw) { return rw > 1 && (f32 ? d == 128 : rw == 4) ? 1 : 2; }
// Whether work-groups of four waves form grad_k or grad_v, not both: sums and operands of both fit one wave a SIMD alone
// with 128 dimensions in bf16 (reverse of 50 000 ragged nodes 799 us, by roles 760).
constexpr bool diff_two_roles(bool f32, int d, int rw) { return !f32 && d == 128 && rw == 4; }

// us of a work-group of four waves for one key or row (as unit_us): two maps beside one product with v.
inline double diff_unit_us(bool f32, int width, bool backward) { return 1.6 * unit_us(f32, width, backward); }

// Launchers.
hipError_t launch_diff_forward(const DiffParams& p, hipStream_t s);
hipError_t launch_diff_backward(const DiffParams& p, hipStream_t s);
size_t diff_forward_workspace(const e3conv_attention_args& a);
size_t diff_backward_workspace(const e3conv_attention_args& a);

}  // namespace attn
}  // namespace e3c
