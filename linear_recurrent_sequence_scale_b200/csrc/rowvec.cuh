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

// One rounding (to nearest even) of the float32 value to the storage type;
// two bf16 in one conversion.
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float (&x)[V]) {
  Pack<T, V> u;
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      *reinterpret_cast<__nv_bfloat162*>(&u.e[i]) = __floats2bfloat162_rn(x[i], x[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) Elem<T>::st(&u.e[i], x[i]);
  }
  *reinterpret_cast<Pack<T, V>*>(p) = u;
}

template <typename T> struct Type { using type = T; };
template <int I> struct Int { static constexpr int value = I; };

// n values computed together; two go through the paired float32 instructions.
// At 6.5 TB/s an SM has about 31 instruction slots per lane for an element of
// which 6 bytes move: the kernels below stay under that only with pairs and
// with the plain hardware exponential and reciprocal.
// A pair is one 64-bit register.
template <int n> struct Vec;
template <> struct Vec<1> {
  float a;
  __device__ __forceinline__ float operator[](int) const { return a; }
};
template <> struct Vec<2> {
  unsigned long long ab;
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(static_cast<uint32_t>(i ? ab >> 32 : ab));
  }
};
__device__ __forceinline__ Vec<2> two(float a, float b) {
  Vec<2> r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.ab) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Vec<1> vec(const float (&x)[1]) { return {x[0]}; }
__device__ __forceinline__ Vec<2> vec(const float (&x)[2]) { return two(x[0], x[1]); }
template <int n> __device__ __forceinline__ Vec<n> all(float x) {
  float v[n];
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = x;
  return vec(v);
}
__device__ __forceinline__ Vec<1> fma(Vec<1> a, Vec<1> b, Vec<1> c) {
  return {fmaf(a.a, b.a, c.a)};
}
__device__ __forceinline__ Vec<2> fma(Vec<2> a, Vec<2> b, Vec<2> c) {
  Vec<2> r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.ab) : "l"(a.ab), "l"(b.ab), "l"(c.ab));
  return r;
}
__device__ __forceinline__ Vec<1> add(Vec<1> a, Vec<1> b) { return {a.a + b.a}; }
__device__ __forceinline__ Vec<2> add(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.ab) : "l"(a.ab), "l"(b.ab));
  return r;
}
__device__ __forceinline__ Vec<1> mul(Vec<1> a, Vec<1> b) { return {a.a * b.a}; }
__device__ __forceinline__ Vec<2> mul(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.ab) : "l"(a.ab), "l"(b.ab));
  return r;
}

// 2^x and 1/x by the hardware's approximations (2 and 1 units in the last
// place); 1/x of an infinity is 0.
template <int n> __device__ __forceinline__ Vec<n> exp2v(Vec<n> x) {
  float y[n];
#pragma unroll
  for (int i = 0; i < n; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y[i]) : "f"(x[i]));
  return vec(y);
}
template <int n> __device__ __forceinline__ Vec<n> rcpv(Vec<n> x) {
  float y[n];
#pragma unroll
  for (int i = 0; i < n; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y[i]) : "f"(x[i]));
  return vec(y);
}
constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(g) = 1 / (1 + e^-g), an overflow of e^-g giving 0, and swish(g).
template <int n> __device__ __forceinline__ Vec<n> sigmoid(Vec<n> g) {
  return rcpv(add(exp2v(mul(g, all<n>(-kLog2e))), all<n>(1.0f)));
}
template <int n> __device__ __forceinline__ Vec<n> swish(Vec<n> g) { return mul(g, sigmoid(g)); }

// swish(g) and its derivative sigmoid(g) + swish(g) (1 - sigmoid(g)).
template <int n>
__device__ __forceinline__ void swish_grad(Vec<n> g, Vec<n>* sw, Vec<n>* slope) {
  const Vec<n> s = sigmoid(g);
  *sw = mul(g, s);
  *slope = fma(*sw, fma(s, all<n>(-1.0f), all<n>(1.0f)), s);
}

__device__ __forceinline__ float total(Vec<2> x) { return x[0] + x[1]; }

// One thread's part of a row of d = nv V elements: CH accesses of V elements,
// TPR threads apart.  Elements past d are zeros.  FULL: there are none (d =
// CH V TPR, and the row exists), which spares the zeros and the comparisons.
template <typename T, int V, int CH, int TPR, bool FULL = false> struct RowPart {
  static constexpr int E = CH * V, P = E / 2;
  static_assert(E % 2 == 0, "handled in pairs");
  Vec<2> p[P];
  __device__ __forceinline__ float get(int e) const { return p[e / 2][e % 2]; }
  __device__ __forceinline__ void put(int e, float x) {
    p[e / 2] = e % 2 ? two(p[e / 2][0], x) : two(x, p[e / 2][1]);
  }
  // `nv` is 0 for a thread whose row does not exist
  __device__ __forceinline__ void load(const T* from, int lane, int nv) {
    float v[E];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = c * TPR + lane;
      float x[V];
      if (FULL || i < nv) {
        load_pack<T, V>(from + i * V, x);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < V; ++k) v[c * V + k] = x[k];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = two(v[2 * i], v[2 * i + 1]);
  }
  template <typename S>  // stores to another element type share the layout
  __device__ __forceinline__ void store(S* to, int lane, int nv) const {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = c * TPR + lane;
      float x[V];
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = get(c * V + k);
      if (FULL || i < nv) store_pack<S, V>(to + i * V, x);
    }
  }
  // Zeros past d again.
  __device__ __forceinline__ void clear_rest(int lane, int nv) {
    if constexpr (!FULL) {
      if (nv == CH * TPR) return;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (c * TPR + lane >= nv) {
#pragma unroll
          for (int k = 0; k < V; ++k) put(c * V + k, 0.0f);
        }
    }
  }
  // v <- (v - [mean]) r, r = 1 / sqrt(mean square + eps); returns r.  sum(x)
  // adds x over the row's threads.  A row that does not exist gets r = 0.
  template <typename Sum>
  __device__ __forceinline__ float normalise(int lane, int nv, bool layer, float eps, float inv_d,
                                             Sum sum) {
    if (layer) {
      Vec<2> s = all<2>(0.0f);
#pragma unroll
      for (int i = 0; i < P; ++i) s = add(s, p[i]);
      const Vec<2> less = all<2>(-sum(total(s), 0) * inv_d);
#pragma unroll
      for (int i = 0; i < P; ++i) p[i] = add(p[i], less);
      clear_rest(lane, nv);
    }
    Vec<2> q = all<2>(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) q = fma(p[i], p[i], q);
    const float square = sum(total(q), 1);
    const float r = FULL || nv > 0 ? rsqrtf(fmaf(square, inv_d, eps)) : 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = mul(p[i], all<2>(r));
    return r;
  }
};

inline bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace ret
