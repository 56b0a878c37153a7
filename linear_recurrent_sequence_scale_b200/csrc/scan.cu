// Gated linear recurrence: a decay per channel and token.
//
// Per channel, with a_t the decay and c_t = 1 - a_t its complement,
//     LOGIT   a_t = sigmoid(f_t),  h_t = a_t h_{t-1} + c_t x_t
//     LOG     a_t = exp(f_t),      h_t = a_t h_{t-1} + x_t
// and y_t = h_t, or swish(g_t) h_t with an output gate.  It is the recurrent
// form of retention ("RetNet - Retentive Network - A Successor to
// Transformer for LLMs", Key Equations, Recurrent Form) with the fixed gamma
// replaced by a gate of the input and the d_k x d_v state by one value per
// channel.
//
// The decay is kept as its complement and applied as h - c h: a decay close
// to 1 rounded to float32 would be off by up to 2^-25 every token, the same
// way each time where the gate is steady, while c carries full relative
// precision.  fma(-c, h, h) is exactly 0 at c = 1, so a token with a zero
// decay drops all that was before it.
#include "common.cuh"
#include "kernels.h"
#include "rowvec.cuh"

namespace ret {
namespace scan {

// 1 - a.  LOGIT: sigmoid(-f) from e^-|f|, which cannot overflow.  LOG:
// 1 - e^f, by the Taylor series of e^f - 1 where the difference would cancel
// (|f| < 1/4: seven terms leave 5e-8 of the value).
template <int FORM>
__device__ __forceinline__ float complement(float f) {
  if constexpr (FORM == RET_SCAN_LOGIT) {
    const float e = __expf(-fabsf(f));
    const float r = __fdividef(1.0f, 1.0f + e);
    return f >= 0.0f ? e * r : r;
  } else {
    float s = fmaf(f, 1.0f / 720.0f, 1.0f / 120.0f);
    s = fmaf(f, s, 1.0f / 24.0f);
    s = fmaf(f, s, 1.0f / 6.0f);
    s = fmaf(f, s, 0.5f);
    s = fmaf(f, s, 1.0f);
    return fabsf(f) < 0.25f ? -f * s : 1.0f - __expf(f);
  }
}

// h_t from h_{t-1}, the complement c and the input x.
template <int FORM>
__device__ __forceinline__ float advance(float h, float c, float x) {
  const float kept = fmaf(-c, h, h);
  return FORM == RET_SCAN_LOGIT ? fmaf(c, x, kept) : kept + x;
}

constexpr int kThreads = 128;

// Where element (b, t, d) of an operand lies.
template <typename T>
__device__ __forceinline__ T* at(const Operand& o, long long b, long long t, long long d) {
  return static_cast<T*>(o.p) + b * o.batch + t * o.token + d;
}

// One thread per (batch, channel), token after token.
template <typename T, int FORM, bool GATE>
__global__ void __launch_bounds__(kThreads) scan_channels(const ScanArgs a) {
  const long long ch = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (ch >= (long long)a.B * a.D) return;
  const long long b = ch / a.D, d = ch % a.D;
  const long long nc = cdiv(a.N, RET_SCAN_CHUNK);
  float h = a.state_in ? a.state_in[ch] : 0.0f;
  for (int t = 0; t < a.N; ++t) {
    if (a.chunk_states && t % RET_SCAN_CHUNK == 0)
      a.chunk_states[(b * nc + t / RET_SCAN_CHUNK) * a.D + d] = h;
    h = advance<FORM>(h, complement<FORM>(Elem<T>::ld(at<T>(a.f, b, t, d))),
                      Elem<T>::ld(at<T>(a.x, b, t, d)));
    float out = h;
    if constexpr (GATE) {
      const float g = Elem<T>::ld(at<T>(a.gate, b, t, d));
      out *= g * sigmoidf(g);
    }
    Elem<T>::st(at<T>(a.y, b, t, d), out);
  }
  if (a.state_out) a.state_out[ch] = h;
}

// Backward.  With G_t the gradient that reaches h_t from y_t and from
// everything after it,
//     G_t = dh_t + a_{t+1} G_{t+1},   a_N G_N := d state_out,
//     dh_t = dy_t, or dy_t swish(g_t) with a gate,
//     LOGIT  dx_t = c_t G_t,   df_t = (h_{t-1} - x_t) a_t c_t G_t
//     LOG    dx_t = G_t,       df_t = h_{t-1} a_t G_t
//     dg_t = dy_t h_t swish'(g_t),   d state_in = a_0 G_0.
// One thread per (batch, channel) walks the chunks backwards, recomputing
// each chunk's h from the state that entered it.
template <typename T, int FORM, bool GATE>
__global__ void __launch_bounds__(kThreads) scan_channels_backward(const ScanArgs a) {
  const long long ch = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (ch >= (long long)a.B * a.D) return;
  const long long b = ch / a.D, d = ch % a.D;
  const int nc = cdiv(a.N, RET_SCAN_CHUNK);
  float flow = a.d_state_out ? a.d_state_out[ch] : 0.0f;  // a_{t+1} G_{t+1}
  for (int i = nc - 1; i >= 0; --i) {
    float before[RET_SCAN_CHUNK];
    const int t0 = i * RET_SCAN_CHUNK, L = min(RET_SCAN_CHUNK, a.N - t0);
    float h = a.chunk_states[(b * nc + i) * a.D + d];
    for (int j = 0; j < L; ++j) {
      before[j] = h;
      h = advance<FORM>(h, complement<FORM>(Elem<T>::ld(at<T>(a.f, b, t0 + j, d))),
                        Elem<T>::ld(at<T>(a.x, b, t0 + j, d)));
    }
    for (int j = L - 1; j >= 0; --j) {
      const int t = t0 + j;
      const float c = complement<FORM>(Elem<T>::ld(at<T>(a.f, b, t, d)));
      const float x = Elem<T>::ld(at<T>(a.x, b, t, d));
      float dh = Elem<T>::ld(at<T>(a.d_y, b, t, d));
      if constexpr (GATE) {
        float sw, slope;
        swish_grad(Elem<T>::ld(at<T>(a.gate, b, t, d)), &sw, &slope);
        Elem<T>::st(at<T>(a.grad_gate, b, t, d), dh * advance<FORM>(before[j], c, x) * slope);
        dh *= sw;
      }
      const float G = dh + flow;
      flow = fmaf(-c, G, G);
      Elem<T>::st(at<T>(a.grad_x, b, t, d), FORM == RET_SCAN_LOGIT ? c * G : G);
      Elem<T>::st(at<T>(a.grad_f, b, t, d),
                  FORM == RET_SCAN_LOGIT ? (before[j] - x) * c * flow : before[j] * flow);
    }
  }
  if (a.d_state_in) a.d_state_in[ch] = flow;
}

// One token: h = a h + ..., y = h or swish(g) h.  A thread owns V channels of
// one batch row; the float32 state is read and written once, so HBM bounds it
// at large batches and the launch at small ones.
template <typename T, int FORM, bool GATE, int V>
__global__ void __launch_bounds__(kThreads) scan_token(const ScanArgs a) {
  const int per_row = a.D / V;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)a.B * per_row) return;
  const long long b = i / per_row, d = (i - b * per_row) * V;
  float h[V], f[V], x[V], g[V];
  load_pack<float, V>(a.state_in + b * a.D + d, h);
  load_pack<T, V>(at<T>(a.f, b, 0, d), f);
  load_pack<T, V>(at<T>(a.x, b, 0, d), x);
  if constexpr (GATE) load_pack<T, V>(at<T>(a.gate, b, 0, d), g);
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = advance<FORM>(h[v], complement<FORM>(f[v]), x[v]);
  store_pack<float, V>(a.state_out + b * a.D + d, h);
  if constexpr (GATE) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] *= g[v] * sigmoidf(g[v]);
  }
  store_pack<T, V>(at<T>(a.y, b, 0, d), h);
}

// Calls fn with the element type, the form and whether there is a gate as
// compile-time values.
template <typename T> struct Type { using type = T; };
template <int I> struct Int { static constexpr int value = I; };
template <typename Fn>
cudaError_t dispatch(int dtype, int form, bool gate, Fn fn) {
  auto with_form = [&](auto t) {
    if (form == RET_SCAN_LOGIT)
      return gate ? fn(t, Int<RET_SCAN_LOGIT>(), Int<1>()) : fn(t, Int<RET_SCAN_LOGIT>(), Int<0>());
    return gate ? fn(t, Int<RET_SCAN_LOG>(), Int<1>()) : fn(t, Int<RET_SCAN_LOG>(), Int<0>());
  };
  return dtype == RET_BF16 ? with_form(Type<__nv_bfloat16>()) : with_form(Type<float>());
}

}  // namespace scan

size_t scan_workspace_bytes(int, int, int, int) { return 0; }

cudaError_t launch_scan(const ScanArgs& a, cudaStream_t st) {
  return scan::dispatch(a.dtype, a.form, a.gate.p != nullptr, [&](auto t, auto form, auto gate) {
    using T = typename decltype(t)::type;
    const unsigned grid =
        static_cast<unsigned>(((long long)a.B * a.D + scan::kThreads - 1) / scan::kThreads);
    scan::scan_channels<T, decltype(form)::value, decltype(gate)::value != 0>
        <<<grid, scan::kThreads, 0, st>>>(a);
    return cudaPeekAtLastError();
  });
}

cudaError_t launch_scan_backward(const ScanArgs& a, cudaStream_t st) {
  return scan::dispatch(a.dtype, a.form, a.gate.p != nullptr, [&](auto t, auto form, auto gate) {
    using T = typename decltype(t)::type;
    const unsigned grid =
        static_cast<unsigned>(((long long)a.B * a.D + scan::kThreads - 1) / scan::kThreads);
    scan::scan_channels_backward<T, decltype(form)::value, decltype(gate)::value != 0>
        <<<grid, scan::kThreads, 0, st>>>(a);
    return cudaPeekAtLastError();
  });
}

cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t st) {
  // four channels per thread where every row splits into aligned groups of four
  const size_t es = a.dtype == RET_BF16 ? 2 : 4;
  const auto fits = [&](const Operand& o) {
    return !o.p || (aligned_to(o.p, 4 * es) && (a.B == 1 || o.batch % 4 == 0));
  };
  const bool wide = a.D % 4 == 0 && fits(a.x) && fits(a.f) && fits(a.gate) && fits(a.y) &&
                    aligned_to(a.state_in, 16) && aligned_to(a.state_out, 16);
  return scan::dispatch(a.dtype, a.form, a.gate.p != nullptr, [&](auto t, auto form, auto gate) {
    using T = typename decltype(t)::type;
    constexpr int F = decltype(form)::value;
    constexpr bool G = decltype(gate)::value != 0;
    const long long threads = (long long)a.B * (wide ? a.D / 4 : a.D);
    const unsigned grid = static_cast<unsigned>((threads + scan::kThreads - 1) / scan::kThreads);
    if (wide)
      scan::scan_token<T, F, G, 4><<<grid, scan::kThreads, 0, st>>>(a);
    else
      scan::scan_token<T, F, G, 1><<<grid, scan::kThreads, 0, st>>>(a);
    return cudaPeekAtLastError();
  });
}

}  // namespace ret
