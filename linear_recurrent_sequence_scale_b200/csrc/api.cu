// C ABI of libretention.so: argument checks and kernel dispatch.
//
// Every check runs on the host before anything is launched, so a non-zero
// status means no kernel ran and no memory was touched.
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "retention.h"

namespace {

thread_local int g_last_cuda_error = 0;

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return RET_OK;
  g_last_cuda_error = static_cast<int>(e);
  return RET_ECUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool valid_dtype(int dt) { return dt == RET_F32 || dt == RET_BF16; }

// Sizes shared by the sequence forms.  dk, dv: multiples of 8 in [8, 512].
int check_seq_dims(int B, int H, int N, int dk, int dv, int dtype) {
  if (B < 1 || H < 1 || N < 0 || dk < 8 || dv < 8) return RET_EINVAL;
  if (dk % 8 || dv % 8) return RET_EINVAL;
  if (!valid_dtype(dtype)) return RET_EINVAL;
  if ((int64_t)B * H > 65535) return RET_EUNSUPPORTED;
  if (dk > 512 || dv > 512) return RET_EUNSUPPORTED;
  if ((int64_t)B * H * N * (dk > dv ? dk : dv) > ((int64_t)1 << 40)) return RET_EUNSUPPORTED;
  return RET_OK;
}

int check_eps(float eps) { return isnan(eps) ? RET_EINVAL : RET_OK; }

bool pow2_in(int x, int lo, int hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }

// Shapes the tensor-core kernels handle (bf16 only).
bool tc_dims(int dk, int dv) { return pow2_in(dk, 64, 256) && pow2_in(dv, 64, 512); }
bool tc_chunk(int chunk) { return pow2_in(chunk, 64, 512); }
// The chunk length the tensor-core kernels work in.  Their row tiles hold 128
// query rows, so a 64-token chunk runs as 128-token chunks: every chunk
// length gives the same output and final state in exact arithmetic (the
// chunkwise form regroups one sum), and this moves only where the bf16
// copies of the carried state are rounded, every 128 tokens instead of 64.
int tc_tile(int chunk) { return chunk < 128 ? 128 : chunk; }

size_t tc_workspace_bytes(int B, int H, int N, int dk, int dv, int chunk) {
  const size_t nc = (size_t)((N + chunk - 1) / chunk);
  return 2 * (size_t)B * H * nc * dk * dv;
}

}  // namespace

extern "C" {

const char* ret_status_string(int status) {
  switch (status) {
    case RET_OK: return "ok";
    case RET_EINVAL: return "invalid argument";
    case RET_EUNSUPPORTED: return "unsupported configuration";
    case RET_ECUDA: return "CUDA runtime error";
    case RET_EWORKSPACE: return "workspace too small";
    default: return "unknown status";
  }
}

int ret_last_cuda_error(void) { return g_last_cuda_error; }

const char* ret_version(void) { return "retention-b200 0.1 (sm_100a)"; }

int ret_device_error(void) {
  const int a = ret::tc_state_device_error();
  const int b = ret::tc_out_device_error();
  const int c = ret::selftest_device_error();
  const int d = ret::scan_device_error();
  const int e = ret::add_norm_device_error();
  if (a < 0 || b < 0 || c < 0 || d < 0 || e < 0) return -1;
  return a ? a : (b ? b : (c ? c : (d ? d : e)));
}

int ret_selftest_bounded_wait(int limit_ms, void* stream) {
  if (limit_ms < 1 || limit_ms > 10000) return RET_EINVAL;
  return cuda_status(
      ret::launch_bounded_wait_selftest(limit_ms, static_cast<cudaStream_t>(stream)));
}

int ret_selftest_scan_wait(int limit_ms, void* workspace, size_t workspace_bytes, void* stream) {
  if (limit_ms < 1 || limit_ms > 10000) return RET_EINVAL;
  if (!workspace || workspace_bytes < ret::kSelftestBytes) return RET_EWORKSPACE;
  if (!aligned16(workspace)) return RET_EINVAL;
  return cuda_status(ret::launch_scan_wait_selftest(limit_ms, workspace,
                                                    static_cast<cudaStream_t>(stream)));
}

int ret_parallel_gated(const void* q, const void* k, const void* v, const float* gammas,
                       const void* gate, void* o, int B, int H, int N, int dk, int dv, int dtype,
                       float gn_eps, void* stream) {
  int s = check_seq_dims(B, H, N, dk, dv, dtype);
  if (s) return s;
  if ((s = check_eps(gn_eps))) return s;
  if (N == 0) return RET_OK;
  if (!q || !k || !v || !o || !gammas) return RET_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return RET_EINVAL;
  if (gate && !aligned16(gate)) return RET_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == RET_BF16 && tc_dims(dk, dv)) {
    if ((int64_t)((N + 127) / 128) > 65535) return RET_EUNSUPPORTED;
    return cuda_status(ret::launch_tc_out(q, k, v, gammas, 0, nullptr, 0, gate, o, B, H, N, dk,
                                          dv, gn_eps, 1, 0, st));
  }
  return cuda_status(ret::launch_simt_parallel(q, k, v, gammas, gate, o, B, H, N, dk, dv, dtype,
                                               gn_eps, st));
}

int ret_parallel(const void* q, const void* k, const void* v, const float* gammas, void* o,
                 int B, int H, int N, int dk, int dv, int dtype, float gn_eps, void* stream) {
  return ret_parallel_gated(q, k, v, gammas, nullptr, o, B, H, N, dk, dv, dtype, gn_eps, stream);
}

size_t ret_chunkwise_workspace(int B, int H, int N, int dk, int dv, int chunk, int dtype) {
  if (check_seq_dims(B, H, N, dk, dv, dtype) != RET_OK || chunk < 1) return 0;
  if (N == 0) return 0;
  if (dtype == RET_BF16 && tc_dims(dk, dv) && tc_chunk(chunk))
    return tc_workspace_bytes(B, H, N, dk, dv, tc_tile(chunk));
  return ret::simt_workspace_bytes(B, H, N, dk, dv, chunk);
}

}  // extern "C"

namespace {

bool tc_config(int dtype, int dk, int dv, int chunk) {
  return dtype == RET_BF16 && tc_dims(dk, dv) && tc_chunk(chunk);
}

// Checks shared by the chunkwise entry points (everything but the pointers
// that only one phase reads).
int check_chunkwise(int B, int H, int N, int dk, int dv, int dtype, int chunk,
                    const float* gammas, const void* workspace, size_t workspace_bytes) {
  int s = check_seq_dims(B, H, N, dk, dv, dtype);
  if (s) return s;
  if (chunk < 1 || !gammas) return RET_EINVAL;
  if (N == 0) return RET_OK;
  const size_t need = ret_chunkwise_workspace(B, H, N, dk, dv, chunk, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return RET_EWORKSPACE;
  if (workspace && !aligned16(workspace)) return RET_EINVAL;
  if (tc_config(dtype, dk, dv, chunk)) {
    const int c = tc_tile(chunk);
    const int nc = (N + c - 1) / c;
    if ((int64_t)nc * (c / 128) > 65535) return RET_EUNSUPPORTED;
  }
  return RET_OK;
}

}  // namespace

extern "C" {

int ret_chunkwise_states(const void* k, const void* v, const float* gammas, int chunk,
                         const float* state_in, float* state_out, int B, int H, int N, int dk,
                         int dv, int dtype, void* workspace, size_t workspace_bytes,
                         void* stream) {
  int s = check_chunkwise(B, H, N, dk, dv, dtype, chunk, gammas, workspace, workspace_bytes);
  if (s) return s;
  if ((state_in && !aligned16(state_in)) || (state_out && !aligned16(state_out)))
    return RET_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    // No tokens: the final state is the initial one.
    if (!state_out || state_in == state_out) return RET_OK;
    const size_t state_bytes = sizeof(float) * (size_t)B * H * dk * dv;
    if (state_in)
      return cuda_status(
          cudaMemcpyAsync(state_out, state_in, state_bytes, cudaMemcpyDeviceToDevice, st));
    return cuda_status(cudaMemsetAsync(state_out, 0, state_bytes, st));
  }
  if (!k || !v || !aligned16(k) || !aligned16(v)) return RET_EINVAL;
  if (tc_config(dtype, dk, dv, chunk)) {
    // Needed whenever a state enters, crosses a chunk boundary or is
    // returned; the incoming state is also stored in workspace slot 0.
    const int c = tc_tile(chunk);
    const int nc = (N + c - 1) / c;
    if (nc == 1 && !state_out && !state_in) return RET_OK;
    return cuda_status(ret::launch_tc_state(k, v, gammas, c, state_in, state_out, workspace,
                                            state_in != nullptr, B, H, N, dk, dv, st));
  }
  return cuda_status(ret::launch_simt_states(k, v, gammas, chunk, state_in, state_out, B, H, N,
                                             dk, dv, dtype, workspace, st));
}

}  // extern "C"

namespace {

// The output phase; after_states: the states phase of the same call was
// launched just before it on the stream (programmatic dependent launch).
int chunkwise_output_impl(const void* q, const void* k, const void* v, const float* gammas,
                          int chunk, int has_state_in, const void* gate, void* o, int B, int H,
                          int N, int dk, int dv, int dtype, float gn_eps, const void* workspace,
                          size_t workspace_bytes, void* stream, bool after_states) {
  int s = check_chunkwise(B, H, N, dk, dv, dtype, chunk, gammas, workspace, workspace_bytes);
  if (s) return s;
  if ((s = check_eps(gn_eps))) return s;
  if (N == 0) return RET_OK;
  if (!q || !k || !v || !o) return RET_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return RET_EINVAL;
  if (gate && !aligned16(gate)) return RET_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tc_config(dtype, dk, dv, chunk))
    return cuda_status(ret::launch_tc_out(q, k, v, gammas, tc_tile(chunk), workspace,
                                          has_state_in != 0, gate, o, B, H, N, dk, dv, gn_eps, 0,
                                          after_states, st));
  return cuda_status(ret::launch_simt_output(q, k, v, gammas, chunk, gate, o, B, H, N, dk, dv,
                                             dtype, gn_eps, workspace, st));
}

}  // namespace

extern "C" {

int ret_chunkwise_output_gated(const void* q, const void* k, const void* v, const float* gammas,
                               int chunk, int has_state_in, const void* gate, void* o, int B,
                               int H, int N, int dk, int dv, int dtype, float gn_eps,
                               const void* workspace, size_t workspace_bytes, void* stream) {
  return chunkwise_output_impl(q, k, v, gammas, chunk, has_state_in, gate, o, B, H, N, dk, dv,
                               dtype, gn_eps, workspace, workspace_bytes, stream, false);
}

int ret_chunkwise_output(const void* q, const void* k, const void* v, const float* gammas,
                         int chunk, int has_state_in, void* o, int B, int H, int N, int dk, int dv,
                         int dtype, float gn_eps, const void* workspace, size_t workspace_bytes,
                         void* stream) {
  return ret_chunkwise_output_gated(q, k, v, gammas, chunk, has_state_in, nullptr, o, B, H, N, dk,
                                    dv, dtype, gn_eps, workspace, workspace_bytes, stream);
}

int ret_chunkwise_gated(const void* q, const void* k, const void* v, const float* gammas,
                        int chunk, const float* state_in, float* state_out, const void* gate,
                        void* o, int B, int H, int N, int dk, int dv, int dtype, float gn_eps,
                        void* workspace, size_t workspace_bytes, void* stream) {
  // Every check of both phases runs before the first launch.
  int s = check_chunkwise(B, H, N, dk, dv, dtype, chunk, gammas, workspace, workspace_bytes);
  if (s) return s;
  if ((s = check_eps(gn_eps))) return s;
  if (N > 0) {
    if (!q || !k || !v || !o) return RET_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return RET_EINVAL;
    if (gate && !aligned16(gate)) return RET_EINVAL;
  }
  if ((state_in && !aligned16(state_in)) || (state_out && !aligned16(state_out)))
    return RET_EINVAL;
  s = ret_chunkwise_states(k, v, gammas, chunk, state_in, state_out, B, H, N, dk, dv, dtype,
                           workspace, workspace_bytes, stream);
  if (s) return s;
  // the states kernel ran (and may still be draining) unless nothing needed it
  const bool scanned = tc_config(dtype, dk, dv, chunk) &&
                       ((N + tc_tile(chunk) - 1) / tc_tile(chunk) > 1 || state_out || state_in);
  return chunkwise_output_impl(q, k, v, gammas, chunk, state_in != nullptr, gate, o, B, H, N, dk,
                               dv, dtype, gn_eps, workspace, workspace_bytes, stream, scanned);
}

int ret_chunkwise(const void* q, const void* k, const void* v, const float* gammas, int chunk,
                  const float* state_in, float* state_out, void* o, int B, int H, int N, int dk,
                  int dv, int dtype, float gn_eps, void* workspace, size_t workspace_bytes,
                  void* stream) {
  return ret_chunkwise_gated(q, k, v, gammas, chunk, state_in, state_out, nullptr, o, B, H, N, dk,
                             dv, dtype, gn_eps, workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace {

// The bf16 backward as three forward calls (backward_tc.cu): reversed copies
// of q, k, v and dO, the prepared states, then the forward calls' workspace.
struct BwdTcLayout {
  size_t qr, kr, vr, dor, sin_t, dso_t, dso, g0, fws, fws_bytes, total;
};

bool bwd_tc(int dtype, int chunk) { return dtype == RET_BF16 && tc_chunk(chunk); }

BwdTcLayout bwd_tc_layout(int B, int H, int N, int dk, int dv, int chunk) {
  auto al = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t BH = (size_t)B * H;
  const size_t rk = al(BH * N * dk * 2), rv = al(BH * N * dv * 2), st = al(BH * dk * dv * 4);
  BwdTcLayout L;
  L.qr = 0;
  L.kr = L.qr + rk;
  L.vr = L.kr + rk;
  L.dor = L.vr + rv;
  L.sin_t = L.dor + rv;
  L.dso_t = L.sin_t + st;
  L.dso = L.dso_t + st;
  L.g0 = L.dso + st;
  L.fws = L.g0 + st;
  const size_t a = ret_chunkwise_workspace(B, H, N, dv, dk, chunk, RET_BF16);  // dq, dk calls
  const size_t b = ret_chunkwise_workspace(B, H, N, dk, dv, chunk, RET_BF16);  // the dv call
  L.fws_bytes = al(a > b ? a : b);
  L.total = L.fws + L.fws_bytes;
  return L;
}

}  // namespace

extern "C" {

size_t ret_chunkwise_backward_workspace(int B, int H, int N, int dk, int dv, int chunk,
                                        int dtype) {
  if (check_seq_dims(B, H, N, dk, dv, dtype) != RET_OK || chunk < 1 || N == 0) return 0;
  if (bwd_tc(dtype, chunk)) return bwd_tc_layout(B, H, N, dk, dv, chunk).total;
  return ret::backward_workspace_bytes(B, H, N, dk, dv, chunk);
}

int ret_chunkwise_backward(const void* q, const void* k, const void* v, const float* gammas,
                           int chunk, const float* state_in, const void* d_o,
                           const float* d_state_out, void* dq, void* dk_, void* dv_,
                           float* d_state_in, int B, int H, int N, int dk, int dv, int dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int s = check_seq_dims(B, H, N, dk, dv, dtype);
  if (s) return s;
  if (chunk < 1 || !gammas) return RET_EINVAL;
  if ((state_in && !aligned16(state_in)) || (d_state_out && !aligned16(d_state_out)) ||
      (d_state_in && !aligned16(d_state_in)))
    return RET_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t state_bytes = sizeof(float) * (size_t)B * H * dk * dv;
  if (N == 0) {
    // No tokens: the final state is the initial one, so their gradients are equal.
    if (!d_state_in) return RET_OK;
    if (d_state_out)
      return cuda_status(cudaMemcpyAsync(d_state_in, d_state_out, state_bytes,
                                         cudaMemcpyDeviceToDevice, st));
    return cuda_status(cudaMemsetAsync(d_state_in, 0, state_bytes, st));
  }
  if (!q || !k || !v || !d_o || !dq || !dk_ || !dv_) return RET_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(d_o) || !aligned16(dq) ||
      !aligned16(dk_) || !aligned16(dv_))
    return RET_EINVAL;
  const size_t need = ret_chunkwise_backward_workspace(B, H, N, dk, dv, chunk, dtype);
  if (!workspace || workspace_bytes < need) return RET_EWORKSPACE;
  if (!aligned16(workspace)) return RET_EINVAL;
  if (!bwd_tc(dtype, chunk))
    return cuda_status(ret::launch_chunkwise_backward(q, k, v, gammas, chunk, state_in, d_o,
                                                      d_state_out, dq, dk_, dv_, d_state_in, B,
                                                      H, N, dk, dv, dtype, workspace, st));
  // bf16: each gradient is the forward chunkwise form of permuted inputs
  // (backward_tc.cu states the identities), run by the forward's kernels.
  const BwdTcLayout L = bwd_tc_layout(B, H, N, dk, dv, chunk);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  void *qr = w + L.qr, *kr = w + L.kr, *vr = w + L.vr, *dor = w + L.dor;
  float* sin_t = reinterpret_cast<float*>(w + L.sin_t);
  float* dso_t = reinterpret_cast<float*>(w + L.dso_t);
  float* dso = reinterpret_cast<float*>(w + L.dso);
  float* g0 = reinterpret_cast<float*>(w + L.g0);
  void* fws = w + L.fws;
  const int BH = B * H;
  cudaError_t e;
#define RET_TRY(call)                            \
  do {                                           \
    if ((e = (call)) != cudaSuccess) return cuda_status(e); \
  } while (0)
#define RET_TRY_STATUS(call)                     \
  do {                                           \
    const int s2 = (call);                       \
    if (s2 != RET_OK) return s2;                 \
  } while (0)
  // the forward calls' own checks (e.g. the chunk-count limit) before any
  // launch, so that a failing status still means nothing ran
  RET_TRY_STATUS(check_chunkwise(B, H, N, dv, dk, RET_BF16, chunk, gammas, fws, L.fws_bytes));
  RET_TRY_STATUS(check_chunkwise(B, H, N, dk, dv, RET_BF16, chunk, gammas, fws, L.fws_bytes));
  RET_TRY(ret::launch_reverse_rows(q, qr, BH, N, dk, st));
  RET_TRY(ret::launch_reverse_rows(k, kr, BH, N, dk, st));
  RET_TRY(ret::launch_reverse_rows(v, vr, BH, N, dv, st));
  RET_TRY(ret::launch_reverse_rows(d_o, dor, BH, N, dv, st));
  if (state_in) RET_TRY(ret::launch_prep_state(state_in, sin_t, gammas, BH, H, dk, dv, 1, 0, 0, st));
  if (d_state_out) {
    RET_TRY(ret::launch_prep_state(d_state_out, dso_t, gammas, BH, H, dk, dv, 1, 1, 0, st));
    RET_TRY(ret::launch_prep_state(d_state_out, dso, gammas, BH, H, dk, dv, 0, 1, 0, st));
  }
  // dq = forward(dO, V, K; S_in^T)
  RET_TRY_STATUS(ret_chunkwise(d_o, v, k, gammas, chunk, state_in ? sin_t : nullptr, nullptr, dq,
                               B, H, N, dv, dk, RET_BF16, -1.f, fws, L.fws_bytes, stream));
  // dk, reversed = forward(V', dO', Q'; dS_out^T / gamma)
  RET_TRY_STATUS(ret_chunkwise(vr, dor, qr, gammas, chunk, d_state_out ? dso_t : nullptr, nullptr,
                               dk_, B, H, N, dv, dk, RET_BF16, -1.f, fws, L.fws_bytes, stream));
  // dv, reversed = forward(K', Q', dO'; dS_out / gamma), final state G_0
  RET_TRY_STATUS(ret_chunkwise(kr, qr, dor, gammas, chunk, d_state_out ? dso : nullptr,
                               d_state_in ? g0 : nullptr, dv_, B, H, N, dk, dv, RET_BF16, -1.f,
                               fws, L.fws_bytes, stream));
  RET_TRY(ret::launch_reverse_rows(dk_, dk_, BH, N, dk, st));
  RET_TRY(ret::launch_reverse_rows(dv_, dv_, BH, N, dv, st));
  if (d_state_in) RET_TRY(ret::launch_prep_state(g0, d_state_in, gammas, BH, H, dk, dv, 0, 0, 1, st));
  if (d_state_out)
    RET_TRY(ret::launch_gamma_zero_last_token(k, v, d_state_out, gammas, dk_, dv_, BH, H, N, dk,
                                              dv, st));
#undef RET_TRY
#undef RET_TRY_STATUS
  return RET_OK;
}

int ret_state_combine(const float* locals, const int* spans, int r, const float* gammas,
                      const float* state0, float* state_in, int B, int H, int dk, int dv,
                      void* stream) {
  if (B < 1 || H < 1 || dk < 8 || dv < 8 || dk % 8 || dv % 8) return RET_EINVAL;
  if (r < 0 || (r > 0 && (!locals || !spans)) || !gammas || !state_in) return RET_EINVAL;
  if (r > ret::kMaxSpans) return RET_EUNSUPPORTED;
  if ((int64_t)B * H * dk * dv > ((int64_t)1 << 40)) return RET_EUNSUPPORTED;
  for (int g = 0; g < r; ++g)
    if (spans[g] < 0) return RET_EINVAL;
  if ((locals && !aligned16(locals)) || (state0 && !aligned16(state0)) || !aligned16(state_in))
    return RET_EINVAL;
  return cuda_status(ret::launch_state_combine(locals, spans, r, gammas, state0, state_in, B, H,
                                               dk, dv, static_cast<cudaStream_t>(stream)));
}

int ret_step_rotated(const void* q, const void* k, const void* v, const float* gammas,
                     const float* theta, long long pos, float* state, const void* gate, void* o,
                     int B, int H, int dk, int dv, int dtype, float gn_eps, void* stream) {
  if (B < 1 || H < 1 || dk < 8 || dv < 8 || dk % 8 || dv % 8) return RET_EINVAL;
  if (!valid_dtype(dtype)) return RET_EINVAL;
  int s = check_eps(gn_eps);
  if (s) return s;
  if (dk > 4096 || dv > 1024 || (int64_t)B * H > 65535) return RET_EUNSUPPORTED;
  if (!q || !k || !v || !gammas || !state || !o) return RET_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state) || !aligned16(o))
    return RET_EINVAL;
  if (gate && !aligned16(gate)) return RET_EINVAL;
  if (theta && (pos < 0 || pos > ((long long)1 << 53))) return RET_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_status(ret::launch_step(q, k, v, gammas, state, gate, o, B, H, dk, dv, dtype, gn_eps,
                                      theta, theta ? pos : 0, st));
}

int ret_step_gated(const void* q, const void* k, const void* v, const float* gammas,
                   float* state, const void* gate, void* o, int B, int H, int dk, int dv,
                   int dtype, float gn_eps, void* stream) {
  return ret_step_rotated(q, k, v, gammas, nullptr, 0, state, gate, o, B, H, dk, dv, dtype,
                          gn_eps, stream);
}

int ret_step(const void* q, const void* k, const void* v, const float* gammas, float* state,
             void* o, int B, int H, int dk, int dv, int dtype, float gn_eps, void* stream) {
  return ret_step_gated(q, k, v, gammas, state, nullptr, o, B, H, dk, dv, dtype, gn_eps, stream);
}

int ret_rotate(const void* x, void* y, const float* theta, long long pos0, int B, int H, int N,
               int d, int dtype, void* stream) {
  if (B < 1 || H < 1 || N < 0 || d < 2 || d % 2) return RET_EINVAL;
  if (!valid_dtype(dtype)) return RET_EINVAL;
  if (pos0 < 0 || pos0 > ((long long)1 << 53) - N) return RET_EINVAL;
  if (N == 0) return RET_OK;  // nothing to read or write; x, y, theta may be NULL
  if (!x || !y || !theta) return RET_EINVAL;
  if (!aligned16(x) || !aligned16(y)) return RET_EINVAL;
  if ((int64_t)B * H > INT32_MAX || (int64_t)N * d > ((int64_t)1 << 38) ||
      (int64_t)B * H * N * d > ((int64_t)1 << 40))
    return RET_EUNSUPPORTED;
  const uintptr_t bytes = (uintptr_t)((int64_t)B * H * N * d * (dtype == RET_BF16 ? 2 : 4));
  const uintptr_t xs = reinterpret_cast<uintptr_t>(x), ys = reinterpret_cast<uintptr_t>(y);
  if (xs != ys && xs < ys + bytes && ys < xs + bytes) return RET_EINVAL;  // partial overlap
  return cuda_status(ret::launch_rotate(x, y, theta, pos0, B, H, N, d, dtype,
                                        static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// A [batches][rows] lattice of `width`-byte pieces.
struct Extent {
  const void* p;
  int64_t batches, batch, rows, row, width;
};

Extent flat(const void* p, int64_t bytes) { return {p, 1, bytes, 1, bytes, bytes}; }

// Whether pieces of wa and wb bytes that repeat every `period` bytes, `off`
// bytes from one to the other, leave each other alone.
bool apart(int64_t off, int64_t period, int64_t wa, int64_t wb) {
  if (period < 1) return false;
  off %= period;
  if (off < 0) off += period;
  return off >= wa && period - off >= wb;
}

int64_t reach(const Extent& e) {
  return (e.batches - 1) * e.batch + (e.rows - 1) * e.row + e.width;
}

// Whether two arrays share a byte.  Slices of one buffer interleave without
// sharing: channels of each token, or spans of each batch row's tokens (equal
// pitches).  Other lattices whose ranges meet count as sharing.
bool overlap(const Extent& a, const Extent& b) {
  if (!a.p || !b.p || a.width < 1 || b.width < 1) return false;
  const intptr_t pa = reinterpret_cast<intptr_t>(a.p), pb = reinterpret_cast<intptr_t>(b.p);
  if (pa + reach(a) <= pb || pb + reach(b) <= pa) return false;
  const int64_t off = pb - pa;
  const bool one = a.batches == 1 && b.batches == 1;
  if (!one && (a.batches != b.batches || a.batch != b.batch)) return true;
  const int64_t wa = (a.rows - 1) * a.row + a.width, wb = (b.rows - 1) * b.row + b.width;
  if (!one && a.batch > 0 && apart(off, a.batch, wa, wb)) return false;
  if (a.rows != b.rows || a.row != b.row || a.rows == 1) return true;
  // every piece starts at a multiple of the smaller pitch, if that divides the larger
  int64_t period = a.row;
  if (!one) {
    const int64_t large = a.batch > a.row ? a.batch : a.row;
    period = a.batch > a.row ? a.row : a.batch;
    if (period < 1 || large % period) return true;
  }
  return !apart(off, period, a.width, b.width);
}

bool same(const Extent& a, const Extent& b) {
  return a.p == b.p && a.batches == b.batches && a.rows == b.rows && a.width == b.width &&
         (a.batches == 1 || a.batch == b.batch) && (a.rows == 1 || a.row == b.row);
}

// The outputs against the inputs and one another; aliasing(o, i) says whether
// output o may be the very array that input i is.
template <typename May>
bool clash(const Extent* out, int n_out, const Extent* in, int n_in, May may) {
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (overlap(out[o], in[i]) && !(may(o, i) && same(out[o], in[i]))) return true;
    for (int q = 0; q < o; ++q)
      if (overlap(out[o], out[q])) return true;
  }
  return false;
}

bool aligned_elem(const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == RET_BF16 ? 1u : 3u)) == 0;
}

int64_t elem_bytes(int dtype) { return dtype == RET_BF16 ? 2 : 4; }

int check_scan(int B, int N, int D, int form, int dtype) {
  if (B < 1 || N < 0 || D < 1 || !valid_dtype(dtype)) return RET_EINVAL;
  if (form != RET_SCAN_LOGIT && form != RET_SCAN_LOG) return RET_EINVAL;
  const int64_t channels = (int64_t)B * D;
  // places up to an item past the end are computed in an int
  if (channels > INT32_MAX - 4096 || N > INT32_MAX - 4096) return RET_EUNSUPPORTED;
  if (N > 0 && channels > ((int64_t)1 << 40) / N) return RET_EUNSUPPORTED;
  // items of 64 tokens x 32 channels are counted in an int
  const int64_t items = (int64_t)B * ((D + 31) / 32) * (((int64_t)N + 63) / 64);
  if (items > ((int64_t)1 << 30)) return RET_EUNSUPPORTED;
  return RET_OK;
}

// An operand of the recurrence.  Rows must not share elements: batch rows
// follow one another (batch pitch past the last token's row) or lie between
// two tokens (time-major).
int check_operand(const ret::Operand& o, int B, int N, int D, int dtype) {
  constexpr int64_t kMost = (int64_t)1 << 44;
  if (!o.p || !aligned_elem(o.p, dtype)) return RET_EINVAL;
  if ((N > 1 && o.token < D) || (B > 1 && o.batch < D)) return RET_EINVAL;
  if ((N > 1 && o.token > kMost / N) || (B > 1 && o.batch > kMost / B)) return RET_EUNSUPPORTED;
  if (B > 1 && N > 1 && o.batch < (N - 1) * o.token + D && o.token < (B - 1) * o.batch + D)
    return RET_EINVAL;
  return RET_OK;
}

// Operand k of a call: its pitches in elements from the host array, or dense.
// A single token has no pitch to the next: whatever is given for it (a span of
// one token of a longer sequence, say) does not reach the kernels, which
// address rows behind the last one by it and count on its alignment.
ret::Operand operand(const void* p, const long long* pitches, int k, int N, int D) {
  ret::Operand o = {const_cast<void*>(p), (long long)N * D, D};
  if (pitches) o.batch = pitches[2 * k];
  if (pitches && N > 1) o.token = pitches[2 * k + 1];
  return o;
}

Extent extent(const ret::Operand& o, int B, int N, int D, int dtype) {
  const int64_t es = elem_bytes(dtype);
  return {o.p, B, (B > 1 ? o.batch : 0) * es, N, (N > 1 ? o.token : 0) * es, D * es};
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The final state of an empty sequence is the initial one.
int pass_state(const float* in, float* out, int64_t n, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!out || in == out) return RET_OK;
  const size_t bytes = sizeof(float) * (size_t)n;
  return cuda_status(in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, st)
                        : cudaMemsetAsync(out, 0, bytes, st));
}

}  // namespace

extern "C" {

size_t ret_scan_workspace(int B, int N, int D, int dtype) {
  if (check_scan(B, N, D, RET_SCAN_LOGIT, dtype) != RET_OK || N == 0) return 0;
  return ret::scan_workspace_bytes(B, N, D, dtype);
}

int ret_scan(const void* x, const void* f, const void* gate, const float* state_in,
             float* state_out, float* chunk_states, void* y, const long long* pitches, int B,
             int N, int D, int form, int dtype, void* workspace, size_t workspace_bytes,
             void* stream) {
  int s = check_scan(B, N, D, form, dtype);
  if (s) return s;
  if (!aligned4(state_in) || !aligned4(state_out) || !aligned4(chunk_states)) return RET_EINVAL;
  const int64_t state_bytes = 4 * (int64_t)B * D;
  const Extent si = flat(state_in, state_bytes), so = flat(state_out, state_bytes);
  if (overlap(si, so) && !same(si, so)) return RET_EINVAL;
  if (N == 0) return pass_state(state_in, state_out, (int64_t)B * D, stream);
  ret::ScanArgs a = {};
  a.x = operand(x, pitches, 0, N, D), a.f = operand(f, pitches, 1, N, D);
  a.gate = operand(gate, pitches, 2, N, D), a.y = operand(y, pitches, 3, N, D);
  for (const ret::Operand* o : {&a.x, &a.f, &a.gate, &a.y})
    if ((o != &a.gate || gate) && (s = check_operand(*o, B, N, D, dtype))) return s;
  const size_t need = ret_scan_workspace(B, N, D, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return RET_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return RET_EINVAL;
  const int64_t chunks = (N + RET_SCAN_CHUNK - 1) / RET_SCAN_CHUNK;
  const Extent in[] = {extent(a.x, B, N, D, dtype), extent(a.f, B, N, D, dtype),
                       extent(a.gate, B, N, D, dtype), si};
  const Extent out[] = {extent(a.y, B, N, D, dtype), so,
                        flat(chunk_states, state_bytes * chunks), flat(workspace, (int64_t)need)};
  if (clash(out, 4, in, 4, [](int o, int i) { return o == 1 && i == 3; })) return RET_EINVAL;
  a.state_in = state_in, a.state_out = state_out, a.chunk_states = chunk_states;
  a.B = B, a.N = N, a.D = D, a.form = form, a.dtype = dtype, a.workspace = workspace;
  return cuda_status(ret::launch_scan(a, static_cast<cudaStream_t>(stream)));
}

int ret_scan_step(const void* x, const void* f, const void* gate, const float* state_in,
                  float* state_out, void* y, const long long* pitches, int B, int D, int form,
                  int dtype, void* stream) {
  int s = check_scan(B, 1, D, form, dtype);
  if (s) return s;
  ret::ScanArgs a = {};
  a.x = {const_cast<void*>(x), pitches ? pitches[0] : D, D};
  a.f = {const_cast<void*>(f), pitches ? pitches[1] : D, D};
  a.gate = {const_cast<void*>(gate), pitches ? pitches[2] : D, D};
  a.y = {y, pitches ? pitches[3] : D, D};
  for (const ret::Operand* o : {&a.x, &a.f, &a.gate, &a.y})
    if ((o != &a.gate || gate) && (s = check_operand(*o, B, 1, D, dtype))) return s;
  if (!state_in || !state_out || !aligned4(state_in) || !aligned4(state_out)) return RET_EINVAL;
  const int64_t state_bytes = 4 * (int64_t)B * D;
  const Extent in[] = {extent(a.x, B, 1, D, dtype), extent(a.f, B, 1, D, dtype),
                       extent(a.gate, B, 1, D, dtype), flat(state_in, state_bytes)};
  const Extent out[] = {extent(a.y, B, 1, D, dtype), flat(state_out, state_bytes)};
  if (clash(out, 2, in, 4, [](int o, int i) { return o == 1 && i == 3; })) return RET_EINVAL;
  a.state_in = state_in, a.state_out = state_out;
  a.B = B, a.N = 1, a.D = D, a.form = form, a.dtype = dtype;
  return cuda_status(ret::launch_scan_step(a, static_cast<cudaStream_t>(stream)));
}

int ret_scan_backward(const void* x, const void* f, const void* gate, const float* chunk_states,
                      const void* d_y, const float* d_state_out, void* grad_x, void* grad_f,
                      void* grad_gate, float* d_state_in, const long long* pitches, int B, int N,
                      int D, int form, int dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int s = check_scan(B, N, D, form, dtype);
  if (s) return s;
  if (!aligned4(chunk_states) || !aligned4(d_state_out) || !aligned4(d_state_in))
    return RET_EINVAL;
  const int64_t state_bytes = 4 * (int64_t)B * D;
  const Extent si = flat(d_state_out, state_bytes), so = flat(d_state_in, state_bytes);
  if (overlap(si, so) && !same(si, so)) return RET_EINVAL;
  if (N == 0) return pass_state(d_state_out, d_state_in, (int64_t)B * D, stream);
  if (!gate) grad_gate = nullptr;
  ret::ScanArgs a = {};
  a.x = operand(x, pitches, 0, N, D), a.f = operand(f, pitches, 1, N, D);
  a.gate = operand(gate, pitches, 2, N, D), a.d_y = operand(d_y, pitches, 3, N, D);
  a.grad_x = operand(grad_x, pitches, 4, N, D), a.grad_f = operand(grad_f, pitches, 5, N, D);
  a.grad_gate = operand(grad_gate, pitches, 6, N, D);
  for (const ret::Operand* o :
       {&a.x, &a.f, &a.gate, &a.d_y, &a.grad_x, &a.grad_f, &a.grad_gate})
    if (((o != &a.gate && o != &a.grad_gate) || gate) &&
        (s = check_operand(*o, B, N, D, dtype)))
      return s;
  if (!chunk_states) return RET_EINVAL;
  const size_t need = ret_scan_workspace(B, N, D, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return RET_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return RET_EINVAL;
  const int64_t chunks = (N + RET_SCAN_CHUNK - 1) / RET_SCAN_CHUNK;
  const Extent in[] = {extent(a.x, B, N, D, dtype), extent(a.f, B, N, D, dtype),
                       extent(a.gate, B, N, D, dtype), extent(a.d_y, B, N, D, dtype),
                       si, flat(chunk_states, state_bytes * chunks)};
  const Extent out[] = {extent(a.grad_x, B, N, D, dtype), extent(a.grad_f, B, N, D, dtype),
                        extent(a.grad_gate, B, N, D, dtype), so,
                        flat(workspace, (int64_t)need)};
  if (clash(out, 5, in, 6, [](int o, int i) { return o == 3 && i == 4; })) return RET_EINVAL;
  a.chunk_states = const_cast<float*>(chunk_states);
  a.d_state_out = d_state_out, a.d_state_in = d_state_in;
  a.B = B, a.N = N, a.D = D, a.form = form, a.dtype = dtype, a.workspace = workspace;
  return cuda_status(ret::launch_scan_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

bool norm_kind(int norm) { return norm == RET_NORM_LAYER || norm == RET_NORM_RMS; }

// Sizes of the norm-and-gate calls; a pitch of 0 becomes the dense one.
int check_norm_gate(int B, int H, int N, int dv, int norm, float eps, int token_major, int dtype,
                    long long** pitches, int n_pitches) {
  if (B < 1 || H < 1 || N < 0 || dv < 8 || dv % 8 || !valid_dtype(dtype)) return RET_EINVAL;
  if (!norm_kind(norm) || !(eps >= 0.0f) || isinf(eps)) return RET_EINVAL;
  if (dv > 1024 || (int64_t)B * H > 65535 || N > INT32_MAX - 4096) return RET_EUNSUPPORTED;
  // blocks of at least eight rows are counted in an int
  if ((int64_t)B * H * (((int64_t)N + 7) / 8) > INT32_MAX) return RET_EUNSUPPORTED;
  if ((int64_t)B * H * N * dv > ((int64_t)1 << 40)) return RET_EUNSUPPORTED;
  const int64_t dense = (int64_t)H * dv;
  for (int i = 0; i < n_pitches; ++i) {
    if (!token_major || *pitches[i] == 0) *pitches[i] = dense;
    if (*pitches[i] < dense || *pitches[i] % 8) return RET_EINVAL;
    if (N > 0 && *pitches[i] > ((int64_t)1 << 44) / ((int64_t)B * N)) return RET_EUNSUPPORTED;
  }
  return RET_OK;
}

}  // namespace

extern "C" {

int ret_norm_gate(const void* y, const void* gate, void* o, int B, int H, int N, int dv, int norm,
                  float eps, int token_major, long long ldg, long long ldo, int dtype,
                  void* stream) {
  long long* pitches[] = {&ldg, &ldo};
  int s = check_norm_gate(B, H, N, dv, norm, eps, token_major, dtype, pitches, 2);
  if (s) return s;
  if (N == 0) return RET_OK;
  if (!y || !o || !aligned16(y) || !aligned16(o) || !aligned16(gate)) return RET_EINVAL;
  const int64_t rows = (int64_t)B * N, es = elem_bytes(dtype), w = (int64_t)H * dv * es;
  // head-major arrays, and token-major ones of one head, have y's layout
  const bool like_y = !token_major || H == 1;
  const Extent in[] = {{y, 1, 0, rows, w, w}, {gate, 1, 0, rows, ldg * es, w}};
  const Extent out[] = {{o, 1, 0, rows, ldo * es, w}};
  if (clash(out, 1, in, 2, [&](int, int i) { return i == 1 || like_y; })) return RET_EINVAL;
  ret::NormGateArgs a = {};
  a.y = y, a.gate = gate, a.o = o, a.ldg = ldg, a.ldo = ldo;
  a.B = B, a.H = H, a.N = N, a.dv = dv, a.norm = norm, a.token_major = token_major != 0;
  a.dtype = dtype, a.eps = eps;
  return cuda_status(ret::launch_norm_gate(a, static_cast<cudaStream_t>(stream)));
}

int ret_norm_gate_backward(const void* y, const void* gate, const void* d_o, void* grad_y,
                           void* grad_gate, int B, int H, int N, int dv, int norm, float eps,
                           int token_major, long long ldg, long long lddo, long long ldgg,
                           int dtype, void* stream) {
  long long* pitches[] = {&ldg, &lddo, &ldgg};
  int s = check_norm_gate(B, H, N, dv, norm, eps, token_major, dtype, pitches, 3);
  if (s) return s;
  if (N == 0) return RET_OK;
  if (!gate) grad_gate = nullptr;
  if (!y || !d_o || !grad_y || (gate && !grad_gate)) return RET_EINVAL;
  if (!aligned16(y) || !aligned16(gate) || !aligned16(d_o) || !aligned16(grad_y) ||
      !aligned16(grad_gate))
    return RET_EINVAL;
  const int64_t rows = (int64_t)B * N, es = elem_bytes(dtype), w = (int64_t)H * dv * es;
  const Extent in[] = {{y, 1, 0, rows, w, w},
                       {gate, 1, 0, rows, ldg * es, w},
                       {d_o, 1, 0, rows, lddo * es, w}};
  const Extent out[] = {{grad_y, 1, 0, rows, w, w}, {grad_gate, 1, 0, rows, ldgg * es, w}};
  if (clash(out, 2, in, 3, [](int o, int i) { return o == 0 ? i == 0 : i > 0; }))
    return RET_EINVAL;
  ret::NormGateArgs a = {};
  a.y = y, a.gate = gate, a.d_o = d_o, a.grad_y = grad_y, a.grad_gate = grad_gate;
  a.ldg = ldg, a.ldo = lddo, a.ldgg = ldgg;
  a.B = B, a.H = H, a.N = N, a.dv = dv, a.norm = norm, a.token_major = token_major != 0;
  a.dtype = dtype, a.eps = eps;
  return cuda_status(ret::launch_norm_gate_backward(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

int check_add_norm(long long rows, int d, int post_norm, int norm, float alpha, float beta,
                   float eps, int dtype, const float* w_post, const float* w) {
  if (rows < 0 || d < 1 || !valid_dtype(dtype)) return RET_EINVAL;
  if (!norm_kind(norm) || (post_norm != RET_NORM_NONE && !norm_kind(post_norm)))
    return RET_EINVAL;
  if (!(eps >= 0.0f) || isinf(eps) || !isfinite(alpha) || !isfinite(beta)) return RET_EINVAL;
  if (!aligned16(w_post) || !aligned16(w)) return RET_EINVAL;
  if (d > 16384 || rows > INT32_MAX || rows > ((int64_t)1 << 40) / d) return RET_EUNSUPPORTED;
  return RET_OK;
}

}  // namespace

extern "C" {

int ret_add_norm(const void* x, const void* residual, const float* w_post, const float* w,
                 void* res_out, void* y, long long rows, int d, int post_norm, int norm,
                 float alpha, float beta, float eps, int dtype, void* stream) {
  int s = check_add_norm(rows, d, post_norm, norm, alpha, beta, eps, dtype, w_post, w);
  if (s) return s;
  if (rows == 0) return RET_OK;
  if (!x || !res_out || !y) return RET_EINVAL;
  for (const void* p : {x, residual, (const void*)res_out, (const void*)y})
    if (!aligned_elem(p, dtype)) return RET_EINVAL;
  const int64_t bytes = rows * d * elem_bytes(dtype);
  const Extent in[] = {flat(x, bytes), flat(residual, bytes), flat(w_post, 4 * (int64_t)d),
                       flat(w, 4 * (int64_t)d)};
  const Extent out[] = {flat(res_out, bytes), flat(y, bytes)};
  if (clash(out, 2, in, 4, [](int, int i) { return i < 2; })) return RET_EINVAL;
  ret::AddNormArgs a = {};
  a.x = x, a.residual = residual, a.w_post = w_post, a.w = w, a.res_out = res_out, a.y = y;
  a.rows = rows, a.d = d, a.post_norm = post_norm, a.norm = norm, a.dtype = dtype;
  a.alpha = alpha, a.beta = beta, a.eps = eps;
  return cuda_status(ret::launch_add_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t ret_add_norm_backward_workspace(long long rows, int d) {
  if (check_add_norm(rows, d, RET_NORM_NONE, RET_NORM_RMS, 1.0f, 1.0f, 0.0f, RET_F32, nullptr,
                     nullptr) != RET_OK)
    return 0;
  return ret::add_norm_backward_workspace_bytes(rows, d);
}

int ret_add_norm_backward(const void* x, const void* res_out, const float* w_post, const float* w,
                          const void* d_y, const void* d_res_out, void* grad_x,
                          void* grad_residual, float* grad_w, float* grad_w_post, long long rows,
                          int d, int post_norm, int norm, float alpha, float beta, float eps,
                          int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int s = check_add_norm(rows, d, post_norm, norm, alpha, beta, eps, dtype, w_post, w);
  if (s) return s;
  if (!aligned4(grad_w) || !aligned4(grad_w_post)) return RET_EINVAL;
  const int64_t bytes = rows * d * elem_bytes(dtype), wbytes = 4 * (int64_t)d;
  if (grad_w && overlap(flat(grad_w, wbytes), flat(grad_w_post, wbytes))) return RET_EINVAL;
  if (rows == 0) {
    s = pass_state(nullptr, grad_w, d, stream);
    return s ? s : pass_state(nullptr, grad_w_post, d, stream);
  }
  const bool need_x = post_norm != RET_NORM_NONE || grad_w_post;
  if (!need_x) x = nullptr;
  if (!res_out || !d_y || (need_x && !x)) return RET_EINVAL;
  for (const void* p : {x, res_out, d_y, d_res_out, (const void*)grad_x,
                        (const void*)grad_residual})
    if (!aligned_elem(p, dtype)) return RET_EINVAL;
  const size_t need = grad_w || grad_w_post ? ret_add_norm_backward_workspace(rows, d) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return RET_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return RET_EINVAL;
  const Extent in[] = {flat(x, bytes),         flat(res_out, bytes),  flat(d_y, bytes),
                       flat(d_res_out, bytes), flat(w_post, wbytes), flat(w, wbytes)};
  const Extent out[] = {flat(grad_x, bytes), flat(grad_residual, bytes), flat(grad_w, wbytes),
                        flat(grad_w_post, wbytes), flat(workspace, (int64_t)need)};
  if (clash(out, 5, in, 6, [](int o, int i) { return o < 2 && i < 4; })) return RET_EINVAL;
  ret::AddNormArgs a = {};
  a.x = x, a.w_post = w_post, a.w = w, a.res_out = const_cast<void*>(res_out), a.d_y = d_y;
  a.d_res_out = d_res_out, a.grad_x = grad_x, a.grad_residual = grad_residual;
  a.grad_w = grad_w, a.grad_w_post = grad_w_post;
  a.rows = rows, a.d = d, a.post_norm = post_norm, a.norm = norm, a.dtype = dtype;
  a.alpha = alpha, a.beta = beta, a.eps = eps;
  return cuda_status(ret::launch_add_norm_backward(a, static_cast<float*>(workspace),
                                                   static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
