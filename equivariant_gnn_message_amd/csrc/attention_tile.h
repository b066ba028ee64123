// Tiles of the attention kernels: rows of q, k, v and grad_out in LDS, operands of
// v_mfma_f32_32x32x16_bf16, and the map from work-groups to graphs.
//
// The instruction computes C (32 x 32) += A (32 x 16) B (16 x 32).  Lane l = 32 h + n
// holds A[n][8 h + j], B[8 h + j][n] (j = 0..7) and, in accumulator register i,
// C[8 (i / 4) + 4 h + i % 4][n].  The contraction may run through its 16 slots
// in any order, so registers 8 t .. 8 t + 7 of an accumulator are, as they lie, the
// B operand of a product over the accumulator's rows: slot (h, j) is row
// 16 t + 8 (j / 4) + 4 h + j % 4.  Probabilities go from the product that forms
// their logits to the product that uses them without leaving their lane.
#pragma once

#include <hip/hip_runtime.h>

#include "attention_slots.h"
#include "e3conv.h"

namespace e3c {
namespace attn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxDim = 128;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct Params {
  e3conv_attention_args a;
  int group;                       // query heads per kv head
  unsigned magic;                  // r / group = (r magic) >> 32 >> shift for 0 <= r < 2^31, group > 1
  int shift;
  int group_log2;                  // of a power of two, else 31
  float c;                         // |scale| log2(e), at least the smallest normal number
  int negate;                      // scale < 0: q enters with its sign changed
  int vec;                         // 16-byte loads of q, k, v, grad_out (and out) rows
  int full;                        // dim_qk and dim_v are both 32, 64 or 128
  int vec_st;                      // elements of the outputs' aligned stores: 8 (bf16), 4 or 0
  int slots;                       // work-group slots of the row (or key) tiles
  int splits;                      // ranges of the other axis, joined by a second kernel
  int blocks;                      // work-groups of the launch
  int first_blocks;                // reverse pass in one launch: its work-groups for grad_q,
  int slots_kv, splits_kv;         // and the slots and splits of the others
  void* out;
  long out_row, out_head;
  float* lse;
  const void* go;
  long go_row, go_head;
  void *gq, *gk, *gv;
  long gq_row, gq_head, gk_row, gk_head, gv_row, gv_head;
  float* delta;                    // (num_q, heads_q), reverse pass
  float* part;                     // partial results of the splits
  float* part_kv;                  // and those of grad_k and grad_v
  float* part_ml;                  // and their softmax maximum and sum
};

// An fp32 operand is the sum of three bf16 parts (24 significant bits), a bf16
// operand is one.  P planes of eight elements.
template <int P>
struct Frag {
  bf16x8 p[P];
};

template <class T>
constexpr int planes() {
  return sizeof(T) == 4 ? 3 : 1;
}

// Products of order up to 2^-16 of the leading one; those left out are below 2^-24.
__device__ __forceinline__ f32x16 mma(const Frag<1>& a, const Frag<1>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<3>& a, const Frag<3>& b, f32x16 c) {
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[2], b.p[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[2], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[1], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}

// Eight fp32 values as an operand: rounded to bf16 (one plane), or split in three parts
// v0 = bf16(v), v1 = bf16(v - v0), v2 = bf16(v - v0 - v1).  The differences are exact, so the
// two-term dot product with (-1, 0) or (0, -1) gives them without unpacking v0: seven
// instructions a pair instead of eleven.
__device__ __forceinline__ bf16x2 round2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_convertvector((f32x2{a, b}), bf16x2);
}
__device__ __forceinline__ void to_frag(const float (&v)[8], Frag<1>& f) {
  union {
    bf16x2 two[4];
    bf16x8 all;
  } r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.two[i] = round2(v[2 * i], v[2 * i + 1]);
  f.p[0] = r.all;
}
__device__ __forceinline__ void to_frag(const float (&v)[8], Frag<3>& f) {
  // in registers: as an immediate operand the pair would be read as one 32-bit float
  unsigned first = 0x0000bf80u, second = 0xbf800000u;
  asm("" : "+s"(first));
  asm("" : "+s"(second));
  const bf16x2 lo = __builtin_bit_cast(bf16x2, first), hi = __builtin_bit_cast(bf16x2, second);
  union {
    bf16x2 two[4];
    bf16x8 all;
  } r[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
    r[0].two[i] = round2(a, b);
    a = __builtin_amdgcn_fdot2_f32_bf16(r[0].two[i], lo, a, false);
    b = __builtin_amdgcn_fdot2_f32_bf16(r[0].two[i], hi, b, false);
    r[1].two[i] = round2(a, b);
    a = __builtin_amdgcn_fdot2_f32_bf16(r[1].two[i], lo, a, false);
    b = __builtin_amdgcn_fdot2_f32_bf16(r[1].two[i], hi, b, false);
    r[2].two[i] = round2(a, b);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) f.p[k] = r[k].all;
}

// Eight consecutive elements of a row as they lie in memory.
template <class T>
struct Raw;
template <>
struct Raw<__bf16> {
  bf16x8 v;
  __device__ __forceinline__ float at(int i) const { return (float)v[i]; }
};
template <>
struct Raw<float> {
  f32x4 a, b;
  __device__ __forceinline__ float at(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};

// Eight elements of a row from element d on, of dim.  VEC: rows are 16-byte aligned and
// dim is a multiple of 8; a unit beyond dim reads the row's first one (the caller drops
// it).  Else element by element, zeros beyond dim.
template <bool VEC>
__device__ __forceinline__ Raw<__bf16> fetch8(const __bf16* row, int d, int dim) {
  Raw<__bf16> r;
  if (VEC) {
    r.v = *reinterpret_cast<const bf16x8*>(row + (d < dim ? d : 0));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = d + i < dim ? row[d + i] : (__bf16)0.0f;
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ Raw<float> fetch8(const float* row, int d, int dim) {
  Raw<float> r;
  if (VEC) {
    const float* p = row + (d < dim ? d : 0);
    r.a = *reinterpret_cast<const f32x4*>(p);
    r.b = *reinterpret_cast<const f32x4*>(p + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = d + i < dim ? row[d + i] : 0.0f;
      r.b[i] = d + i + 4 < dim ? row[d + i + 4] : 0.0f;
    }
  }
  return r;
}

// keep = false: zeros, whatever r holds (NaN too).
__device__ __forceinline__ Frag<1> frag_of(const Raw<__bf16>& r, bool keep) {
  Frag<1> f;
  f.p[0] = keep ? r.v : bf16x8{};
  return f;
}
__device__ __forceinline__ Frag<3> frag_of(const Raw<float>& r, bool keep) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = keep ? r.at(i) : 0.0f;
  Frag<3> f;
  to_frag(v, f);
  return f;
}
template <int P>
__device__ __forceinline__ void flip_sign(Frag<P>& f) {
#pragma unroll
  for (int k = 0; k < P; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) f.p[k][i] = -f.p[k][i];
}

// ROWS x D elements in LDS, units of eight elements (16 bytes).  Units of a row are
// permuted by its number so that the two ways of reading meet no bank twice: 16
// consecutive rows at one unit (row operand), and four consecutive rows (from a
// multiple of 4) at four consecutive units (column operand).
template <int P, int ROWS, int D>
struct Tile {
  static constexpr int U = D / 8;
  bf16x8 u[P][ROWS * U];

  static __device__ __forceinline__ int swizzle(int row) {
    if (D == 32) return (row >> 2) & 3;
    if (D == 64) return ((row >> 1) & 1) << 2 | ((row >> 2) & 3);
    return (row & 3) << 2 | ((row >> 2) & 3);
  }
  static __device__ __forceinline__ int at(int row, int unit) { return row * U + (unit ^ swizzle(row)); }

  __device__ __forceinline__ void store(int row, int unit, const Frag<P>& f) {
#pragma unroll
    for (int k = 0; k < P; ++k) u[k][at(row, unit)] = f.p[k];
  }
  // A operand: rows row0 + n, elements 16 step + 8 h + j.
  __device__ __forceinline__ Frag<P> rows(int row0, int step, int lane) const {
    Frag<P> f;
    const int i = at(row0 + (lane & 31), 2 * step + (lane >> 5));
#pragma unroll
    for (int k = 0; k < P; ++k) f.p[k] = u[k][i];
    return f;
  }
  // A operand of the transposed tile: element column 32 dt + n, and along the slots the
  // rows row0 + 8 (j / 4) + 4 h + j % 4 (row0 a multiple of 16).  ds_read_b64_tr_b16:
  // of 16 lanes, lane i gives the address of columns 4 (i % 4) .. + 3 of row i / 4 and
  // receives the four rows of column i.
  __device__ __forceinline__ Frag<P> columns(int row0, int dt, int lane) const {
    const int i = lane & 15, block = lane >> 4;
    const int unit = 4 * dt + 2 * (block & 1) + ((i >> 1) & 1);
    const int row = row0 + 4 * (block >> 1) + (i >> 2);
    Frag<P> f;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const s16x4 lo = tr(&u[k][at(row, unit)], i & 1), hi = tr(&u[k][at(row + 8, unit)], i & 1);
      union {
        s16x4 s[2];
        bf16x8 b;
      } both = {{lo, hi}};
      f.p[k] = both.b;
    }
    return f;
  }
  static __device__ __forceinline__ s16x4 tr(const bf16x8* p, int half) {
    typedef __attribute__((address_space(3))) s16x4* lds;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(reinterpret_cast<const s16x4*>(p) + half));
  }
};

// n work-groups.  A launch takes less than 2^32 threads along an axis, so more than 2^20 work-groups go
// on along y.
constexpr unsigned kAlongX = 1u << 20;
inline dim3 grid_of(long n) {
  return n <= kAlongX ? dim3((unsigned)n) : dim3(kAlongX, (unsigned)((n + kAlongX - 1) / kAlongX));
}
// Which of the n this one is; there may be some more.
__device__ __forceinline__ long block_index() { return (long)blockIdx.y * kAlongX + blockIdx.x; }

// Work-group -> (split, slot, kv head).  Work-groups go to the eight dies in turn, each with
// an L2 of its own: runs of 32 consecutive places, which share a graph's keys (or rows),
// are put on one die.
struct Where {
  int split, slot, c;
};
__device__ __forceinline__ Where where(int b, int blocks, int slots, int splits) {
  constexpr int DIES = 8, RUN = 32;
  const int whole = blocks / (DIES * RUN) * (DIES * RUN);
  if (b < whole) {
    const int r = b % (DIES * RUN);
    b = b - r + r % DIES * RUN + r / DIES;
  }
  Where w;
  w.slot = b % slots;
  b /= slots;
  w.split = b % splits;
  w.c = b / splits;
  return w;
}

// Value of the lane with the other h.
__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

__device__ __forceinline__ int offset(const int* ptr, int i, long n) { return clamp_offset(ptr[i], n); }
__device__ __forceinline__ int first_slot(const int* ptr, int g, long n, int mult, int tile) {
  return slot_at(offset(ptr, g, n), g, mult, tile);
}
__device__ __forceinline__ int graph_of_slot(const int* ptr, int graphs, long n, int mult, int tile, int slot) {
  const int lane = threadIdx.x & 63;
  return __builtin_amdgcn_readfirstlane(search_graph(graphs, [&](int lo, int step, int count) {
    const int i = lane * step;
    bool before = false;
    if (i < count) before = first_slot(ptr, lo + i, n, mult, tile) <= slot;
    return __popcll(__ballot(before));
  }));
}

// Row r of a graph's rows is head r % group of query r / group.
__device__ __forceinline__ int query_of(const Params& p, int r) { return div_group(r, p.group, p.magic, p.shift); }

// How a kernel loads rows: element by element, in whole units of eight elements, or (bf16) in
// whole units that fill the tile.
constexpr int kElements = 0, kUnits = 1, kFull = 2;

// A work-group's loads of a tile of ROWS rows of two operands that share their row order (k and
// v, or q and grad_out): issue() starts them, finish() leaves the tile in LDS, with zeros
// in place of the rows that do not count, whatever memory holds there (the caller
// waits at a barrier after it).  bf16 rows of whole units go from memory to LDS by
// themselves, the lane's unit chosen so that the tile's permutation comes out; lanes of
// units beyond dim load nothing and leave the zeros that clear() has put there (an infinity
// would be NaN against the other operand's zeros; clearing them after each tile's loads took
// 10 % with 96 dimensions).  Others pass through registers: fp32 is split on the way.
template <class T, int D, int ROWS, int NT, int LOAD>
struct Pair {
  static constexpr int P = planes<T>(), U = D / 8, E = ROWS * U / NT, STEP = NT / U;
  static constexpr bool VEC = LOAD != kElements, DMA = sizeof(T) == 2 && VEC, SPARE = LOAD != kFull;
  typedef Tile<P, ROWS, D> TileT;
  static_assert(ROWS * U % NT == 0 && ROWS <= 64, "");
  Raw<T> x[DMA ? 1 : E], y[DMA ? 1 : E];

  static __device__ __forceinline__ int row(int e) { return (int)threadIdx.x / U + e * STEP; }
  static __device__ __forceinline__ int unit(int e) {
    const int slot = threadIdx.x % U;
    return DMA ? slot ^ TileT::swizzle(row(e)) : slot;
  }
  // Zeros in this thread's units beyond dim.
  static __device__ __forceinline__ void clear(int dim_x, int dim_y, TileT& xt, TileT& yt) {
    if constexpr (DMA && SPARE)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (unit(e) * 8 >= dim_x) xt.u[0][e * NT + threadIdx.x] = bf16x8{};
        if (unit(e) * 8 >= dim_y) yt.u[0][e * NT + threadIdx.x] = bf16x8{};
      }
  }
  // First element of this thread's unit of row e, as far as the row has it.
  static __device__ __forceinline__ int first(int e, int dim) {
    const int d = unit(e) * 8;
    return DMA && SPARE && d >= dim ? 0 : d;
  }
  // Whether all rows of a thread have the same unit (their numbers differ by multiples of 16).
  static constexpr bool SAME = !DMA || STEP % 16 == 0;
  // xp and yp: this thread's unit of its row e.
  __device__ __forceinline__ void issue(int e, const T* xp, const T* yp, int dim_x, int dim_y, TileT& xt, TileT& yt) {
    if constexpr (DMA) {
      typedef const __attribute__((address_space(1))) void* from;
      typedef __attribute__((address_space(3))) void* to;
      const int at = e * NT + __builtin_amdgcn_readfirstlane(threadIdx.x & ~63);   // the wave's first unit
      if (!SPARE || unit(e) * 8 < dim_x) __builtin_amdgcn_global_load_lds((from)xp, (to)&xt.u[0][at], 16, 0, 0);
      if (!SPARE || unit(e) * 8 < dim_y) __builtin_amdgcn_global_load_lds((from)yp, (to)&yt.u[0][at], 16, 0, 0);
    } else {
      const int d = unit(e) * 8;
      x[e] = fetch8<VEC>(xp - d, d, dim_x);
      y[e] = fetch8<VEC>(yp - d, d, dim_y);
    }
  }
  // seen: a bit for each row of the tile that counts.
  __device__ __forceinline__ void finish(unsigned long seen, int dim_x, int dim_y, TileT& xt, TileT& yt) const {
    const bool whole = seen == (ROWS == 64 ? ~0ul : (1ul << (ROWS & 63)) - 1);
    if constexpr (DMA) {
      arrive();
      if (!whole) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!(seen >> row(e) & 1)) {      // a unit that this thread has loaded itself
            xt.u[0][e * NT + threadIdx.x] = bf16x8{};
            yt.u[0][e * NT + threadIdx.x] = bf16x8{};
          }
      }
    } else if (whole && (!VEC || (dim_x == D && dim_y == D))) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xt.store(row(e), unit(e), frag_of(x[e], true));
        yt.store(row(e), unit(e), frag_of(y[e], true));
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool keep = seen >> row(e) & 1;
        xt.store(row(e), unit(e), frag_of(x[e], keep && unit(e) * 8 < dim_x));
        yt.store(row(e), unit(e), frag_of(y[e], keep && unit(e) * 8 < dim_y));
      }
    }
  }
  // Waits until all loads that this wave has issued are there.
  static __device__ __forceinline__ void arrive() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)
};

// The tiles of the keys of one kv head, and the starting value of each key's logits: 0, or
// -infinity for a key that is not seen.  Rows beyond the last key read the last one.
template <class T, int D, int ROWS, int NT, int LOAD>
struct Keys {
  typedef Pair<T, D, ROWS, NT, LOAD> PairT;
  typedef typename PairT::TileT TileT;
  PairT pair;
  unsigned char m;
  const T *kp, *vp;      // this thread's unit of its first row of the next tile
  int next, end;         // keys of this work-group not yet loaded

  __device__ __forceinline__ void begin(const Params& p, int c, int k0, int k1) {
    const e3conv_attention_args& a = p.a;
    const long j = k0 + PairT::row(0);
    kp = (const T*)a.k + c * a.k_head + j * a.k_row + PairT::first(0, a.dim_qk);
    vp = (const T*)a.v + c * a.v_head + j * a.v_row + PairT::first(0, a.dim_v);
    next = k0;
    end = k1;
  }
  static __device__ __forceinline__ int shift(int e, int dim) {
    return PairT::SAME ? 0 : PairT::first(e, dim) - PairT::first(0, dim);
  }
  __device__ __forceinline__ void issue(const Params& p, TileT& kt, TileT& vt) {
    const e3conv_attention_args& a = p.a;
    if (next + ROWS <= end) {
#pragma unroll
      for (int e = 0; e < PairT::E; ++e)
        pair.issue(e, kp + (e * PairT::STEP * a.k_row + shift(e, a.dim_qk)),
                   vp + (e * PairT::STEP * a.v_row + shift(e, a.dim_v)), a.dim_qk, a.dim_v, kt, vt);
    } else {
#pragma unroll
      for (int e = 0; e < PairT::E; ++e) {
        const int back = min(end - 1 - (next + PairT::row(0)), e * PairT::STEP);
        pair.issue(e, kp + (back * a.k_row + shift(e, a.dim_qk)), vp + (back * a.v_row + shift(e, a.dim_v)), a.dim_qk,
                   a.dim_v, kt, vt);
      }
    }
    if (a.k_mask) m = a.k_mask[min(next + (int)(threadIdx.x & 63), end - 1)];
    kp += ROWS * a.k_row;
    vp += ROWS * a.v_row;
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

// The tiles of the rows (queries and their heads of one kv head) that a work-group of the
// reverse pass walks over, and each row's lse (base 2) and -delta.  A row that sees no key
// or lies beyond the end has lse = +infinity, which makes its P zero.  OWN: delta is formed
// here, else it was left in memory.
template <class T, int D, int ROWS, int NT, int LOAD, bool OWN>
struct Rows {
  typedef Pair<T, D, ROWS, NT, LOAD> PairT;
  typedef typename PairT::TileT TileT;
  PairT pair;
  float lse, delta;
  unsigned char m;
  const T *qb, *gb;      // the kv head's first row of the graph
  const T *qp, *gp;      // this thread's unit of its first row of the next tile
  long at0;              // of lse and delta
  int q0, next, end;

  __device__ __forceinline__ void begin(const Params& p, int c, int first_query, int r0, int r1) {
    const e3conv_attention_args& a = p.a;
    q0 = first_query;
    qb = (const T*)a.q + q0 * a.q_row + c * p.group * a.q_head;
    gb = (const T*)p.go + q0 * p.go_row + c * p.group * p.go_head;
    at0 = (long)q0 * a.heads_q + c * p.group;
    next = r0;
    end = r1;
    const int r = r0 + PairT::row(0), i = query_of(p, r), x = r - i * p.group;
    qp = qb + i * a.q_row + x * a.q_head + PairT::first(0, a.dim_qk);
    gp = gb + i * p.go_row + x * p.go_head + PairT::first(0, a.dim_v);
  }
  static __device__ __forceinline__ int shift(int e, int dim) {
    return PairT::SAME ? 0 : PairT::first(e, dim) - PairT::first(0, dim);
  }
  __device__ __forceinline__ void issue(const Params& p, TileT& qt, TileT& gt) {
    const e3conv_attention_args& a = p.a;
    // STEP rows on lie STEP / group queries on where the heads of a group divide STEP
    const int by = PairT::STEP >> p.group_log2;
    if (next + ROWS <= end && by << p.group_log2 == PairT::STEP) {
#pragma unroll
      for (int e = 0; e < PairT::E; ++e)
        pair.issue(e, qp + (e * by * a.q_row + shift(e, a.dim_qk)), gp + (e * by * p.go_row + shift(e, a.dim_v)),
                   a.dim_qk, a.dim_v, qt, gt);
      qp += PairT::E * by * a.q_row;
      gp += PairT::E * by * p.go_row;
    } else {
#pragma unroll
      for (int e = 0; e < PairT::E; ++e) {
        const int r = min(next + PairT::row(e), end - 1), i = query_of(p, r), x = r - i * p.group;
        pair.issue(e, qb + i * a.q_row + x * a.q_head + PairT::first(e, a.dim_qk),
                   gb + i * p.go_row + x * p.go_head + PairT::first(e, a.dim_v), a.dim_qk, a.dim_v, qt, gt);
      }
    }
    const int r = min(next + (int)(threadIdx.x & 63), end - 1), i = query_of(p, r);
    const long at = at0 + (long)i * (a.heads_q - p.group) + r;
    lse = p.lse[at];
    if constexpr (OWN) {
      const int x = r - i * p.group;
      const T* g = gb + i * p.go_row + x * p.go_head;
      const T* o = (const T*)p.out + (q0 + i) * p.out_row + ((at0 - (long)q0 * a.heads_q) + x) * p.out_head;
      delta = 0.0f;
      for (int d = 0; d < a.dim_v; d += 8) {
        const Raw<T> u = fetch8<PairT::VEC>(g, d, a.dim_v), v = fetch8<PairT::VEC>(o, d, a.dim_v);
#pragma unroll
        for (int j = 0; j < 8; ++j) delta = fmaf(u.at(j), v.at(j), delta);
      }
    } else {
      delta = p.delta[at];
    }
    if (a.q_mask) m = a.q_mask[q0 + i];
    next += ROWS;
  }
  // r0: the first row of the issued tile.
  __device__ __forceinline__ void finish(const Params& p, int r0, TileT& qt, TileT& gt, float* lse_of,
                                         float* delta_of) const {
    const int lane = threadIdx.x & 63;
    const bool sees = lane < ROWS && r0 + lane < end && lse != -INFINITY && (!p.a.q_mask || m);
    if (threadIdx.x < ROWS) {
      lse_of[lane] = sees ? lse * kLog2e : INFINITY;
      delta_of[lane] = sees ? -delta : 0.0f;
    }
    pair.finish(__ballot(sees), p.a.dim_qk, p.a.dim_v, qt, gt);
  }
};

// Walks over the tiles of [from, to), STEP rows each: start(buffer) issues a tile's loads,
// use(buffer, first row, next buffer) has it finished and used; the next tile's loads are
// issued after the barrier that follows finish.  Two buffers need one barrier a tile; they
// are separate variables, so that the compiler knows the loads in flight from the
// reads of the other one.
template <int BUF, int STEP, class Buffer, class Use>
__device__ __forceinline__ void walk(int from, int to, Buffer& a, Buffer& b, Use use) {
  while (from < to) {
    use(a, from, b);
    from += STEP;
    if (BUF == 2) {
      if (from >= to) break;
      use(b, from, a);
      from += STEP;
    }
  }
}

// Values of 32 rows from LDS where an accumulator has them: register i is row 8 (i / 4) +
// 4 h + i % 4.
__device__ __forceinline__ f32x16 by_row(const float* rows, int lane) {
  f32x16 r;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(rows + 8 * x + 4 * (lane >> 5));
#pragma unroll
    for (int i = 0; i < 4; ++i) r[4 * x + i] = v[i];
  }
  return r;
}

// The B operands of one row (lane n's, k = 16 t + 8 h + j) from memory; zeros unless live.
template <class T, int D, int LOAD>
__device__ __forceinline__ void row_operand(const T* row, int dim, bool live, Frag<planes<T>()> (&f)[D / 16]) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int t = 0; t < D / 16; ++t) {
    const int d = 16 * t + 8 * h;
    f[t] = frag_of(fetch8<LOAD != kElements>(row, d, dim), live && d < dim);
  }
}

// Four consecutive elements d .. d + 3 of a row with dim elements.
template <class T>
__device__ __forceinline__ void store4(T* p, int d, int dim, const float (&v)[4], bool vec) {
  if (vec && d + 4 <= dim) {
    typedef T V __attribute__((ext_vector_type(4)));
    V o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (T)v[i];
    *reinterpret_cast<V*>(p + d) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < dim) p[d + i] = (T)v[i];
  }
}

// use(i, load(i)) for i < N, the loads W steps ahead of their use.  The fences keep loads
// and products in this order (vector instructions may pass): left alone, the compiler
// puts each LDS read right before its product, and every product waits for its read.
template <int N, int W, class F, class Load, class Use>
__device__ __forceinline__ void ahead(Load load, Use use) {
  F ring[W];
#pragma unroll
  for (int i = 0; i < W && i < N; ++i) ring[i] = load(i);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_barrier(0x6);
    use(i, ring[i % W]);
    if (i + W < N) ring[i % W] = load(i + W);
  }
  __builtin_amdgcn_sched_barrier(0x6);
}

// Stores a wave's transposed result: lane (h, n) has elements 32 dt + 8 b + 4 h + 0 .. 3 of row
// `to`, in o[dt][4 b ..]; zeros unless live.  bf16 with 16-byte rows: the halves of the wave
// exchange every other group of four, so that each lane stores eight in a row.
template <class T, int N>
__device__ __forceinline__ void store_row(T* to, const f32x16 (&o)[N], int dim, float factor, bool live, int vec) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int dt = 0; dt < N; ++dt) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = live ? o[dt][i] * factor : 0.0f;
    if (sizeof(T) == 2 && vec == 8) {
#pragma unroll
      for (int b = 0; b < 4; b += 2) {
        const auto pair = [&](int i) { return __builtin_bit_cast(unsigned, round2(v[i], v[i + 1])); };
        const auto r0 = __builtin_amdgcn_permlane32_swap(pair(4 * b), pair(4 * b + 4), false, false);
        const auto r1 = __builtin_amdgcn_permlane32_swap(pair(4 * b + 2), pair(4 * b + 6), false, false);
        const int d = 32 * dt + 8 * (b + h);
        if (d < dim) *reinterpret_cast<uint4*>(to + d) = make_uint4(r0[0], r1[0], r0[1], r1[1]);
      }
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float x[4] = {v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]};
        store4(to, 32 * dt + 8 * b + 4 * h, dim, x, vec != 0);
      }
    }
  }
}

// ------------------------------------------------------------ launch shapes ---

// Waves of a SIMD that the registers are kept to: with one, nothing covers the latency of LDS
// and the barriers (grad_q with 128 dimensions, bf16: 322 us with one, 255 with two).
// Forward, grad_q, and grad_k with grad_v, whose 128-wide bf16 form spills 40 registers when
// kept to two (628 against 470 us).
constexpr int waves_fwd(bool f32, int d) { return f32 ? (d == 32 ? 3 : d == 64 ? 2 : 1) : (d == 32 ? 4 : d == 64 ? 3 : 2); }
constexpr int waves_bwd(bool f32, int d) { return f32 ? (d == 32 ? 2 : 1) : (d == 32 ? 3 : 2); }
constexpr int waves_kv(bool f32, int d) { return f32 ? (d == 32 ? 2 : 1) : (d == 32 ? 3 : d == 64 ? 2 : 1); }

constexpr int kMaxSplits = 512;
inline int padded(int dim) { return dim <= 32 ? 32 : dim <= 64 ? 64 : 128; }   // of the tiles

struct Shape {
  int rw;        // waves of a work-group, 32 rows each
  int slots;     // its row tiles: rows / (32 rw) + graphs
  int splits;    // ranges of the other axis
};

// Work-groups of four waves share each tile of the other axis where a graph has more than 64
// rows (of a graph of 64 rows two of the four would idle), else of one wave.  The other
// axis is split where the row tiles leave compute units idle, in the first filling of the
// chip or the last (628 work-groups on 512 places are 2 fillings; split in four, 5 of a
// quarter each: 4.3 against 3.7 ms for the reverse pass of 20 000 nodes).  The choice minimises
// an estimate from `unit`, the us of one work-group for one row of the other axis (below),
// and the partial results' bytes.  Lengths are on the device: averages stand for them.
inline Shape choose(long rows, long others, int graphs, int heads, int waves, double unit, int width) {
  const long g = graphs > 0 ? graphs : 1, avg = (rows + g - 1) / g, avg_o = (others + g - 1) / g;
  Shape s;
  s.rw = avg > 64 ? 4 : 1;
  s.slots = (int)(rows / (32 * s.rw) + graphs);
  const long n = g * ((avg + 32 * s.rw - 1) / (32 * s.rw)) * heads;
  const long places = 256 * (s.rw == 4 ? waves : 4);
  long most = (avg_o + 127) / 128;
  if (most > kMaxSplits) most = kMaxSplits;
  double best = 1e30;
  s.splits = 1;
  for (long k = 1; k <= most; k += k < 16 ? 1 : k / 8) {
    const long fillings = (n * k + places - 1) / places;
    const double join = k > 1 ? 5.0 + (double)k * rows * heads * width * 8e-6 / 3.0 : 0.0;
    const double us = fillings * (double)avg_o / k * unit + join;
    if (us < 0.95 * best) {
      best = us;
      s.splits = (int)k;
    }
  }
  return s;
}
// us of a work-group of four waves for one key or row, with its neighbours on the compute unit.
// Measured: forward in bf16 with 64 dimensions, 309 us for 8.2 fillings of the chip over 1000 keys; the
// others in proportion to their own measurements.  It decides between splits only.
inline double unit_us(bool f32, int dim, bool backward) {
  return 0.04 * (dim <= 32 ? 0.7 : dim <= 64 ? 1.0 : 2.0) * (f32 ? 1.7 : 1.0) * (backward ? 1.5 : 1.0);
}

// Launchers.
hipError_t launch_forward(const Params& p, hipStream_t s);
hipError_t launch_backward(const Params& p, hipStream_t s);
size_t forward_workspace(const e3conv_attention_args& a);
size_t backward_workspace(const e3conv_attention_args& a);

}  // namespace attn
}  // namespace e3c
