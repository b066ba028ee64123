// Rows read in runs of elements: what the kernels of the root-mean-square norm and of rotary positions share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace e3c {
namespace rows {

// n / d for 0 <= n < 2^31 by a product: ceil(2^(31 + l) / d) with 2^l >= d.
struct Div {
  int d;
  unsigned magic;
  int shift;
  __device__ __forceinline__ int of(int n) const { return d == 1 ? n : (int)(__umulhi((unsigned)n, magic) >> shift); }
};
inline Div div_by(int d) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  return {d, l > 0 ? (unsigned)((((uint64_t)1 << (31 + l)) + d - 1) / d) : 0, l > 0 ? l - 1 : 0};
}

// n work-groups.  A launch takes less than 2^32 threads along an axis, so more than 2^20 work-groups go
// on along y.
constexpr unsigned kAlongX = 1u << 20;
inline dim3 grid_of(int64_t n) {
  return n <= kAlongX ? dim3((unsigned)n) : dim3(kAlongX, (unsigned)((n + kAlongX - 1) / kAlongX));
}
// Which of the n this one is; there may be some more.
__device__ __forceinline__ long block_index() { return (long)blockIdx.y * kAlongX + blockIdx.x; }

template <class T, int V>
struct Run {
  typedef T type __attribute__((ext_vector_type(V)));
};
template <class T>
struct Run<T, 1> {
  typedef T type;
};
template <class T, int V>
__device__ __forceinline__ typename Run<T, V>::type read(const T* p) {
  return *reinterpret_cast<const typename Run<T, V>::type*>(p);
}
template <class T, int V>
__device__ __forceinline__ void widen(const typename Run<T, V>::type& r, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = (float)r;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)r[i];
  }
}
template <class T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
  typename Run<T, V>::type r;
  if constexpr (V == 1) {
    r = (T)v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = (T)v[i];
  }
  *reinterpret_cast<typename Run<T, V>::type*>(p) = r;
}

// Whether runs of 16 bytes (v elements) are aligned in rows of this stride.
inline bool aligned(const void* p, int64_t row, int v) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % v == 0;
}

}  // namespace rows
}  // namespace e3c
