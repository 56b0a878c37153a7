// Row pieces of the block operators: V consecutive elements of one row held
// in float32 registers, moved by one access of up to 16 bytes.
#pragma once

#include "common.cuh"

namespace ret {

// V elements of T, V * sizeof(T) bytes (2, 4, 8 or 16) and aligned to that.
template <typename T, int V> struct alignas(V * sizeof(T)) Pack {
  T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_pack(const T* p, float (&x)[V]) {
  const Pack<T, V> u = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = Elem<T>::ld(&u.e[i]);
}

// One rounding (to nearest even) of the float32 value to the storage type.
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float (&x)[V]) {
  Pack<T, V> u;
#pragma unroll
  for (int i = 0; i < V; ++i) Elem<T>::st(&u.e[i], x[i]);
  *reinterpret_cast<Pack<T, V>*>(p) = u;
}

// sigmoid(x); e^-x overflowing to inf gives 0.
__device__ __forceinline__ float sigmoidf(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// swish(x) = x sigmoid(x) and its derivative sigmoid(x) (1 + x (1 - sigmoid(x))).
__device__ __forceinline__ void swish_grad(float x, float* swish, float* slope) {
  const float s = sigmoidf(x);
  *swish = x * s;
  *slope = s * fmaf(x, 1.0f - s, 1.0f);
}

inline bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Multiprocessors of the current device.
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    n = 148;
  return n;
}

}  // namespace ret
