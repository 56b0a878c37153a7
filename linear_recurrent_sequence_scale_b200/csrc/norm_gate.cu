// Per-head norm and output gate as a pass of its own, and its backward.
//
// One row is the d_v outputs of one (batch, head, token).  With
//     z = (y - mean) r,  r = 1 / sqrt(var + eps)      (GroupNorm, biased)
//     z = y r,           r = 1 / sqrt(mean(y^2) + eps)  (RMS)
// the forward writes o = swish(g) (.) z ("RetNet - Retentive Network - A
// Successor to Transformer for LLMs", core components, item 4: GroupNorm with
// swish gating), and the backward, with dz = do (.) swish(g),
//     dg = do (.) z (.) swish'(g)
//     dy = r (dz - [mean(dz)] - z mean(dz (.) z))    ([] for GroupNorm only).
//
// Bound by HBM: every element is read once and written once.  A row stays in
// the registers of TPR threads of one warp (16 bytes per access, CH accesses
// per tensor), so its sums are warp shuffles and the variance is taken about
// the mean, not as a difference of moments.  y and dy are head-major, as
// retention writes and reads them; g, o, do and dg may be token-major, as the
// projections around the layer want them: a row is one contiguous piece of
// d_v elements either way, so the change of layout costs nothing.
#include "common.cuh"
#include "kernels.h"
#include "rowvec.cuh"

namespace ret {
namespace ng {

constexpr int kThreads = 256;

// Sum over the TPR lanes that share a row.
template <int TPR> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Where row n of (batch, head) bh begins: head-major, or token-major with ld
// elements between tokens.
__device__ __forceinline__ long long row_at(int bh, int n, int H, int N, int dv, bool token_major,
                                            long long ld) {
  if (!token_major) return ((long long)bh * N + n) * dv;
  const int b = bh / H;
  return ((long long)b * N + n) * ld + (long long)(bh - b * H) * dv;
}

template <typename T, int CH, int TPR, bool GATE>
struct Row {
  static constexpr int V = 16 / sizeof(T);
  float v[CH][V];
  // elements past dv read as zero, so that they add nothing to a sum
  __device__ __forceinline__ void load(const T* p, int lane, int nv) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = c * TPR + lane;
      if (i < nv) {
        load_pack<T, V>(p + (long long)i * V, v[c]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) v[c][k] = 0.0f;
      }
    }
  }
  __device__ __forceinline__ void store(T* p, int lane, int nv) const {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = c * TPR + lane;
      if (i < nv) store_pack<T, V>(p + (long long)i * V, v[c]);
    }
  }
  // v <- z, the normalised row; returns r.  Elements past dv stay zero.
  __device__ __forceinline__ float normalise(int lane, int nv, bool layer, float eps, float inv_d) {
    if (layer) {
      float s = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int k = 0; k < V; ++k) s += v[c][k];
      const float mean = row_sum<TPR>(s) * inv_d;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if (c * TPR + lane < nv) {
#pragma unroll
          for (int k = 0; k < V; ++k) v[c][k] -= mean;
        }
    }
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < V; ++k) q = fmaf(v[c][k], v[c][k], q);
    const float r = rsqrtf(fmaf(row_sum<TPR>(q), inv_d, eps));
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < V; ++k) v[c][k] *= r;
    return r;
  }
};

template <typename T, int CH, int TPR, bool GATE>
__global__ void __launch_bounds__(kThreads)
norm_gate_rows(const T* y, const T* gate, T* o, int H, int N, int dv, bool layer, float eps,
               bool token_major, long long ldg, long long ldo) {
  using R = Row<T, CH, TPR, GATE>;
  constexpr int V = R::V;
  const int lane = threadIdx.x % TPR, bh = blockIdx.y, nv = dv / V;
  const int n = blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const int take = n < N ? nv : 0;  // threads past the last row take part in the shuffles only
  const int row = min(n, N - 1);
  R z, g;
  z.load(y + ((long long)bh * N + row) * dv, lane, take);
  if constexpr (GATE) g.load(gate + row_at(bh, row, H, N, dv, token_major, ldg), lane, take);
  z.normalise(lane, take, layer, eps, 1.0f / dv);
  if constexpr (GATE) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < V; ++k) z.v[c][k] *= g.v[c][k] * sigmoidf(g.v[c][k]);
  }
  z.store(o + row_at(bh, row, H, N, dv, token_major, ldo), lane, take);
}

template <typename T, int CH, int TPR, bool GATE>
__global__ void __launch_bounds__(kThreads)
norm_gate_rows_backward(const T* y, const T* gate, const T* d_o, T* grad_y, T* grad_gate, int H,
                        int N, int dv, bool layer, float eps, bool token_major, long long ldg,
                        long long lddo, long long ldgg) {
  using R = Row<T, CH, TPR, GATE>;
  constexpr int V = R::V;
  const int lane = threadIdx.x % TPR, bh = blockIdx.y, nv = dv / V;
  const int n = blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const int take = n < N ? nv : 0;
  const int row = min(n, N - 1);
  const float inv_d = 1.0f / dv;
  R z, g, d;
  z.load(y + ((long long)bh * N + row) * dv, lane, take);
  d.load(d_o + row_at(bh, row, H, N, dv, token_major, lddo), lane, take);
  if constexpr (GATE) g.load(gate + row_at(bh, row, H, N, dv, token_major, ldg), lane, take);
  const float r = z.normalise(lane, take, layer, eps, inv_d);
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if constexpr (GATE) {
        float sw, slope;
        swish_grad(g.v[c][k], &sw, &slope);
        g.v[c][k] = d.v[c][k] * z.v[c][k] * slope;
        d.v[c][k] *= sw;
      }
      s1 += d.v[c][k];
      s2 = fmaf(d.v[c][k], z.v[c][k], s2);
    }
  if constexpr (GATE) g.store(grad_gate + row_at(bh, row, H, N, dv, token_major, ldgg), lane, take);
  s1 = layer ? row_sum<TPR>(s1) * inv_d : 0.0f;
  s2 = row_sum<TPR>(s2) * inv_d;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int k = 0; k < V; ++k) z.v[c][k] = r * (d.v[c][k] - s1 - z.v[c][k] * s2);
  z.store(grad_y + ((long long)bh * N + row) * dv, lane, take);
}

template <int I> struct Int { static constexpr int value = I; };

// The fewest lanes whose 16-byte accesses cover a row; rows longer than a
// warp's take more accesses per lane.
template <typename Fn> cudaError_t by_width(int nv, Fn fn) {
  if (nv <= 4) return fn(Int<1>(), Int<4>());
  if (nv <= 8) return fn(Int<1>(), Int<8>());
  if (nv <= 16) return fn(Int<1>(), Int<16>());
  if (nv <= 32) return fn(Int<1>(), Int<32>());
  if (nv <= 64) return fn(Int<2>(), Int<32>());
  if (nv <= 128) return fn(Int<4>(), Int<32>());
  return fn(Int<8>(), Int<32>());
}

template <typename T, bool GATE> cudaError_t forward_t(const NormGateArgs& a, cudaStream_t st) {
  return by_width(a.dv * (int)sizeof(T) / 16, [&](auto ch, auto tpr) {
    constexpr int CH = decltype(ch)::value, TPR = decltype(tpr)::value;
    const dim3 grid(cdiv(a.N, kThreads / TPR), a.B * a.H);
    norm_gate_rows<T, CH, TPR, GATE><<<grid, kThreads, 0, st>>>(
        static_cast<const T*>(a.y), static_cast<const T*>(a.gate), static_cast<T*>(a.o), a.H, a.N,
        a.dv, a.norm == RET_NORM_LAYER, a.eps, a.token_major != 0, a.ldg, a.ldo);
    return cudaPeekAtLastError();
  });
}

template <typename T, bool GATE> cudaError_t backward_t(const NormGateArgs& a, cudaStream_t st) {
  return by_width(a.dv * (int)sizeof(T) / 16, [&](auto ch, auto tpr) {
    constexpr int CH = decltype(ch)::value, TPR = decltype(tpr)::value;
    const dim3 grid(cdiv(a.N, kThreads / TPR), a.B * a.H);
    norm_gate_rows_backward<T, CH, TPR, GATE><<<grid, kThreads, 0, st>>>(
        static_cast<const T*>(a.y), static_cast<const T*>(a.gate), static_cast<const T*>(a.d_o),
        static_cast<T*>(a.grad_y), static_cast<T*>(a.grad_gate), a.H, a.N, a.dv,
        a.norm == RET_NORM_LAYER, a.eps, a.token_major != 0, a.ldg, a.ldo, a.ldgg);
    return cudaPeekAtLastError();
  });
}

}  // namespace ng

cudaError_t launch_norm_gate(const NormGateArgs& a, cudaStream_t st) {
  if (a.dtype == RET_BF16)
    return a.gate ? ng::forward_t<__nv_bfloat16, true>(a, st)
                  : ng::forward_t<__nv_bfloat16, false>(a, st);
  return a.gate ? ng::forward_t<float, true>(a, st) : ng::forward_t<float, false>(a, st);
}

cudaError_t launch_norm_gate_backward(const NormGateArgs& a, cudaStream_t st) {
  if (a.dtype == RET_BF16)
    return a.gate ? ng::backward_t<__nv_bfloat16, true>(a, st)
                  : ng::backward_t<__nv_bfloat16, false>(a, st);
  return a.gate ? ng::backward_t<float, true>(a, st) : ng::backward_t<float, false>(a, st);
}

}  // namespace ret
