// Joins what the work-groups of the attention kernels' reverse passes leave: the splits of the three gradients, and
// the parts of lambda's.
#pragma once

#include "attention_tile.h"

namespace e3c {
namespace attn {
namespace {

// Sums the splits of a gradient.  `each` elements to a work-group: 256, a thread each,
// or 64, and four waves share each one's splits, eight at a time.
struct Sum {
  const float* part;
  long rows;            // (i, head)
  int width, from, dim; // elements from .. from + dim - 1 of `width`
  int maps, heads, splits, each;   // maps: heads of dim / maps elements side by side in a row
  long blocks;
  float factor;
  void* out;
  long out_row, out_head;
  const float* rest;    // or NULL: (splits, rows), whose sum times that of the elements `dim` on is taken off
};
struct Sums {
  Sum of[3];
  const float* lam;     // (lams, heads): the last `heads` work-groups add -glam
  int lams, heads;
  float* glam;
};
template <class T>
__global__ void __launch_bounds__(256) attn_sum(Sums all) {
  __shared__ float red[4][64];
  long b = block_index();
  int which = 0;
  while (which < 2 && b >= all.of[which].blocks) b -= all.of[which++].blocks;
  const Sum& m = all.of[which];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (b >= m.blocks) {
    b -= m.blocks;
    if (b >= all.heads) return;
    float v = 0.0f;
#pragma unroll 8
    for (int i = threadIdx.x; i < all.lams; i += 256) v += all.lam[(long)i * all.heads + b];
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if (lane == 0) red[w][0] = v;
    __syncthreads();
    if (threadIdx.x == 0) all.glam[b] = -((red[0][0] + red[1][0]) + (red[2][0] + red[3][0]));
    return;
  }
  const bool wide = m.each == 256;
  const long i = b * m.each + (wide ? (int)threadIdx.x : lane), at = i / m.dim;
  const int d = (int)(i - at * m.dim);
  const float* q = m.part + at * m.width + m.from + d;
  const long step = m.rows * m.width;
  float v = 0.0f, bar = 0.0f, rest = 0.0f;
  if (at < m.rows) {
    int s = wide ? 0 : w;
    const int by = wide ? 1 : 4;
    for (; s + 7 * by < m.splits; s += 8 * by) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = q[(s + k * by) * step];
#pragma unroll
      for (int k = 0; k < 8; ++k) v += x[k];
    }
    for (; s < m.splits; s += by) v += q[s * step];
    if (m.rest)
#pragma unroll 4
      for (s = wide ? 0 : w; s < m.splits; s += by) {
        bar += q[s * step + m.dim];
        rest += m.rest[s * m.rows + at];
      }
  }
  if (!wide) {
    const auto of_waves = [&](float x) {
      red[w][lane] = x;
      __syncthreads();
      x = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
      __syncthreads();
      return x;
    };
    v = of_waves(v);
    if (m.rest) {
      bar = of_waves(bar);
      rest = of_waves(rest);
    }
    if (w > 0) return;
  }
  if (m.rest) v = fmaf(-rest, bar, v);
  if (at < m.rows) {
    const int second = m.maps == 2 && d >= m.dim / 2;
    ((T*)m.out)[at / m.heads * m.out_row + (at % m.heads * m.maps + second) * m.out_head + d - second * (m.dim / 2)] =
        (T)(v * m.factor);
  }
}

// The sums that a gradient's splits ask for; none (blocks 0) where there is one split.
Sum sum_of(const float* part, long rows, int width, int from, int dim, int maps, int heads, int splits, float factor,
           void* out, long row, long head, const float* rest = nullptr) {
  Sum m{part, rows, width, from, dim, maps, heads, splits, splits <= 8 ? 256 : 64, 0, factor, out, row, head, rest};
  if (splits > 1) m.blocks = (rows * dim + m.each - 1) / m.each;
  return m;
}

}  // namespace
}  // namespace attn
}  // namespace e3c
