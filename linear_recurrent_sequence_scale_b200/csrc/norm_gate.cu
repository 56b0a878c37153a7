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

// Blocks of four warps: 8 x 8 x 16384 x 256 backward takes 426 us, 460 with
// eight (three such blocks fit an SM at 78 registers, and wait for their
// slowest warp).
constexpr int kThreads = 128;

// Sum over the TPR lanes that share a row.
template <int TPR> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The rows of a block: kTurns times kThreads / TPR tokens of one (batch, head).
// Heads run fastest over the grid, so that the blocks at work together cover
// whole tokens of the token-major arrays: with tokens fastest they would all
// be in one head and touch one piece of d_v elements in every H (8 x 16 x 8192
// x 512 in bf16: 656 against 641 us).  Several turns share the block's place
// in the arrays, whose computation would otherwise cost as much as a row.
constexpr int kTurns = 4;
struct Where {
  int b, h, n0;
  __device__ __forceinline__ Where(int H, int N, int rows) {
    const int blocks = cdiv(N, rows);
    const unsigned rest = blockIdx.x / H;
    h = blockIdx.x - rest * H;
    b = rest / blocks;
    n0 = (rest - b * blocks) * rows;
  }
  // Where row n begins: head-major, or token-major with ld elements between tokens.
  __device__ __forceinline__ long long head_major(int n, int H, int N, int dv) const {
    return (((long long)b * H + h) * N + n) * dv;
  }
  __device__ __forceinline__ long long at(int n, int H, int N, int dv, bool token_major,
                                          long long ld) const {
    return token_major ? ((long long)b * N + n) * ld + (long long)h * dv
                       : head_major(n, H, N, dv);
  }
};

template <typename T, int CH, int TPR, bool GATE>
__global__ void __launch_bounds__(kThreads)
norm_gate_rows(const T* y, const T* gate, T* o, int H, int N, int dv, bool layer, float eps,
               bool token_major, long long ldg, long long ldo) {
  using R = RowPart<T, 16 / sizeof(T), CH, TPR>;
  constexpr int kRows = kThreads / TPR;
  const Where w(H, N, kTurns * kRows);
  const int lane = threadIdx.x % TPR, nv = dv / (16 / (int)sizeof(T));
  const float inv_d = 1.0f / dv;
  int n = w.n0 + threadIdx.x / TPR;
  y += w.head_major(n, H, N, dv);
  if constexpr (GATE) gate += w.at(n, H, N, dv, token_major, ldg);
  o += w.at(n, H, N, dv, token_major, ldo);
  const long long step = (long long)kRows * dv, step_g = token_major ? kRows * ldg : step,
                  step_o = token_major ? kRows * ldo : step;
#pragma unroll 1
  for (int i = 0; i < kTurns && w.n0 + i * kRows < N; ++i, n += kRows) {
    const int take = n < N ? nv : 0;  // threads past the last row only join the shuffles
    R z, g;
    z.load(y, lane, take);
    if constexpr (GATE) g.load(gate, lane, take);
    z.normalise(lane, take, layer, eps, inv_d, [](float x, int) { return row_sum<TPR>(x); });
    if constexpr (GATE) {
#pragma unroll
      for (int k = 0; k < R::P; ++k) z.p[k] = mul(z.p[k], swish(g.p[k]));
    }
    z.store(o, lane, take);
    y += step, o += step_o;
    if constexpr (GATE) gate += step_g;
  }
}

template <typename T, int CH, int TPR, bool GATE>
__global__ void __launch_bounds__(kThreads)
norm_gate_rows_backward(const T* y, const T* gate, const T* d_o, T* grad_y, T* grad_gate, int H,
                        int N, int dv, bool layer, float eps, bool token_major, long long ldg,
                        long long lddo, long long ldgg) {
  using R = RowPart<T, 16 / sizeof(T), CH, TPR>;
  constexpr int kRows = kThreads / TPR;
  const Where w(H, N, kTurns * kRows);
  const int lane = threadIdx.x % TPR, nv = dv / (16 / (int)sizeof(T));
  const float inv_d = 1.0f / dv;
  int n = w.n0 + threadIdx.x / TPR;
  y += w.head_major(n, H, N, dv);
  grad_y += w.head_major(n, H, N, dv);
  d_o += w.at(n, H, N, dv, token_major, lddo);
  if constexpr (GATE) {
    gate += w.at(n, H, N, dv, token_major, ldg);
    grad_gate += w.at(n, H, N, dv, token_major, ldgg);
  }
  const long long step = (long long)kRows * dv, step_g = token_major ? kRows * ldg : step,
                  step_o = token_major ? kRows * lddo : step,
                  step_gg = token_major ? kRows * ldgg : step;
#pragma unroll 1
  for (int i = 0; i < kTurns && w.n0 + i * kRows < N; ++i, n += kRows) {
    const int take = n < N ? nv : 0;
    R z, g, d;
    z.load(y, lane, take);
    d.load(d_o, lane, take);
    if constexpr (GATE) g.load(gate, lane, take);
    const float r = z.normalise(lane, take, layer, eps, inv_d,
                                [](float x, int) { return row_sum<TPR>(x); });
    Vec<2> p1 = all<2>(0.0f), p2 = p1;
#pragma unroll
    for (int k = 0; k < R::P; ++k) {
      Vec<2> dk = d.p[k];
      const Vec<2> zk = z.p[k];
      if constexpr (GATE) {
        Vec<2> sw, slope;
        swish_grad(g.p[k], &sw, &slope);
        g.p[k] = mul(mul(dk, zk), slope);
        dk = mul(dk, sw);
        d.p[k] = dk;
      }
      p1 = add(p1, dk);
      p2 = fma(dk, zk, p2);
    }
    if constexpr (GATE) g.store(grad_gate, lane, take);
    const float s1 = layer ? row_sum<TPR>(total(p1)) * -inv_d : 0.0f;
    const float s2 = row_sum<TPR>(total(p2)) * -inv_d;
#pragma unroll
    for (int k = 0; k < R::P; ++k)
      z.p[k] = mul(all<2>(r), fma(z.p[k], all<2>(s2), add(d.p[k], all<2>(s1))));
    z.store(grad_y, lane, take);
    y += step, grad_y += step, d_o += step_o;
    if constexpr (GATE) gate += step_g, grad_gate += step_gg;
  }
}

// Two 16-byte accesses per lane and tensor, so that a row's sums cost few
// shuffles per element (8 x 8 x 2048 x 256 backward: 74 us with one access
// and twice the lanes, 65 with two); rows longer than a warp's take more.
template <typename Fn> cudaError_t by_width(int nv, Fn fn) {
  if (nv <= 8) return fn(Int<2>(), Int<4>());
  if (nv <= 16) return fn(Int<2>(), Int<8>());
  if (nv <= 32) return fn(Int<2>(), Int<16>());
  if (nv <= 64) return fn(Int<2>(), Int<32>());
  if (nv <= 128) return fn(Int<4>(), Int<32>());
  return fn(Int<8>(), Int<32>());
}

template <typename T, bool GATE> cudaError_t forward_t(const NormGateArgs& a, cudaStream_t st) {
  return by_width(a.dv * (int)sizeof(T) / 16, [&](auto ch, auto tpr) {
    constexpr int CH = decltype(ch)::value, TPR = decltype(tpr)::value;
    const unsigned grid = (unsigned)cdiv(a.N, kTurns * (kThreads / TPR)) * a.B * a.H;
    norm_gate_rows<T, CH, TPR, GATE><<<grid, kThreads, 0, st>>>(
        static_cast<const T*>(a.y), static_cast<const T*>(a.gate), static_cast<T*>(a.o), a.H, a.N,
        a.dv, a.norm == RET_NORM_LAYER, a.eps, a.token_major != 0, a.ldg, a.ldo);
    return cudaPeekAtLastError();
  });
}

template <typename T, bool GATE> cudaError_t backward_t(const NormGateArgs& a, cudaStream_t st) {
  return by_width(a.dv * (int)sizeof(T) / 16, [&](auto ch, auto tpr) {
    constexpr int CH = decltype(ch)::value, TPR = decltype(tpr)::value;
    const unsigned grid = (unsigned)cdiv(a.N, kTurns * (kThreads / TPR)) * a.B * a.H;
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
