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
#include "sm100.cuh"

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

constexpr int kThreads = 128;  // of the single-token kernel

// Where element (b, t, d) of an operand lies.
template <typename T>
__device__ __forceinline__ T* at(const Operand& o, long long b, long long t, long long d) {
  return static_cast<T*>(o.p) + b * o.batch + t * o.token + d;
}

// ---- sequence form ------------------------------------------------------------
//
// The recurrence composes: a span of tokens turns the state s before it into
// H + s - C s, where H is its end state from zero and 1 - C the product of
// its decays (kept as C for the reason above: C <- C + c (1 - C) per token).
// The sequence is cut into items of kTok tokens x one 128-byte piece of
// channels.  A block keeps a ring of items in shared memory (loads of the
// next ones run while one is computed), and per item
//   1. each of 8 warps scans its own kTok/8 tokens from zero, channels across
//      lanes (4 bytes of them each), and leaves (C, H) in shared memory;
//   2. warp 0 folds the eight, publishes the item's (C, H), looks back over
//      the previous items of the same channels until it meets one whose end
//      state is published, folds forward from there, and publishes its own
//      end state;
//   3. every warp runs its tokens again from the state that enters them and
//      writes y.
// So every element crosses HBM once, and neither few channels nor long
// sequences leave SMs idle.
//
// Items are taken from a counter in time order: an item's predecessors are
// held by blocks that already run, and each block works through its items in
// the order it took them, so waiting for them always ends, whatever else the
// GPU runs.  The wait is bounded in time all the same.  A published word is
// its own flag (every word of the workspace starts as kEmpty, which no
// result of arithmetic is), so no fence or lock is needed, and folding from
// any published end state gives the same bits: the end state of an item is
// itself the fold of its (C, H) over the one before.
constexpr int kWarps = 8;
constexpr int kBlock = 32 * kWarps;
constexpr int kPiece = 128;                // bytes of one row of an item
constexpr uint32_t kEmpty = 0xffffffffu;   // a NaN that arithmetic never returns
constexpr int kWindow = 4;                 // predecessors looked at together
constexpr int kSiteForward = 801, kSiteBackward = 802;

struct Plan {
  int* ticket;     // starts at -1 (all bits set, like the rest of the workspace)
  float* end;      // [tile][B][blocks][channels]: end states
  float2* span;    // same: (C, H)
  int blocks;      // pieces of channels per batch row
  int tiles;       // items per piece
  int items;
};

__device__ __forceinline__ float word(float x) {
  return __float_as_uint(x) == kEmpty ? __uint_as_float(0x7fffffffu) : x;
}
__device__ __forceinline__ bool written(float x) { return __float_as_uint(x) != kEmpty; }
__device__ __forceinline__ float ld_word(const float* p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_words(const float2* p) {
  float2 v;
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_word(float* p, float v) {
  asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(word(v)) : "memory");
}
__device__ __forceinline__ void st_words(float2* p, float x, float y) {
  asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(word(x)),
               "f"(word(y))
               : "memory");
}

// The state after a span (C, H) entered with s.
__device__ __forceinline__ float fold(float s, float C, float H) { return fmaf(-C, s, s) + H; }

// The state that enters item `tile` (> 0) of a channel: `at` points at the
// channel's words of that item, `pitch` words from one tile to the next.
__device__ __forceinline__ float look_back(const Plan& p, size_t at, size_t pitch, int tile,
                                           int site) {
  float s = 0.0f;
  bool found = false;
  uint64_t t0 = 0;
  int tries = 0;
  while (true) {
    float e[kWindow];
    float2 g[kWindow];
#pragma unroll
    for (int i = 0; i < kWindow; ++i) {
      e[i] = __uint_as_float(kEmpty);
      if (tile - 1 - i >= 0) {
        e[i] = ld_word(p.end + at - (i + 1) * pitch);
        if (i + 1 < kWindow) g[i] = ld_words(p.span + at - (i + 1) * pitch);
      }
    }
    // the nearest published end state, if every span after it is published
    if (!found) {
      bool whole = true;
#pragma unroll
      for (int i = 0; i < kWindow; ++i) {
        if (!found && whole && written(e[i])) {
          s = e[i];
          found = true;
#pragma unroll
          for (int k = i - 1; k >= 0; --k) s = fold(s, g[k].x, g[k].y);
        }
        if (i + 1 < kWindow && tile - 1 - i >= 0)
          whole = whole && written(g[i].x) && written(g[i].y);
      }
    }
    if (__all_sync(0xffffffffu, found)) return s;
    if (++tries % 64 == 0) {
      const uint64_t now = sm100::globaltimer();
      if (t0 == 0) t0 = now;
      // out of time, or another wait was: the whole warp gives up together
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&g_device_error) != 0 ||
                                      now - t0 > sm100::kWaitLimitNs)) {
        sm100::record_error(site);
        return __uint_as_float(0x7fffffffu);
      }
    }
  }
}

// ---- moving an item into shared memory ------------------------------------------
template <int W> __device__ __forceinline__ void cp_async(uint32_t dst, const char* src, bool ok) {
  const int n = ok ? W : 0;  // 0: writes zeros, reads nothing
  if constexpr (W == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// kTok rows of kPiece bytes: rows past `rows` and bytes past `bytes` become
// zeros.  W: bytes per access; 2 (rows aligned to a bf16 only) has no
// asynchronous form and goes through registers.
template <int W, int TOK>
__device__ __forceinline__ void copy_item(char* dst, const char* src, long long pitch, int rows,
                                          int bytes) {
  if constexpr (W >= 4) {
    constexpr int kPer = kPiece / W, kStep = kBlock / kPer;
    const int col = (threadIdx.x % kPer) * W;
    const uint32_t d = sm100::smem_u32(dst) + col;
#pragma unroll
    for (int i = 0; i < TOK / kStep; ++i) {
      const int r = i * kStep + threadIdx.x / kPer;
      const bool ok = r < rows && col < bytes;
      cp_async<W>(d + r * kPiece, ok ? src + r * pitch + col : src, ok);
    }
  } else {
    const int col = (threadIdx.x % 32) * 4;
#pragma unroll 8
    for (int i = 0; i < TOK / kWarps; ++i) {
      const int r = i * kWarps + threadIdx.x / 32;
      uint32_t v = 0;
      if (r < rows) {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(src + r * pitch + col);
        if (col < bytes) v = q[0];
        if (col + 2 < bytes) v |= (uint32_t)q[1] << 16;
      }
      *reinterpret_cast<uint32_t*>(dst + r * kPiece + col) = v;
    }
  }
}

// The channels of one lane: 4 bytes of a row.
template <typename T> struct Lane {
  static constexpr int n = 4 / sizeof(T);
  float v[n];
  __device__ __forceinline__ void get(const char* row) {
    load_pack<T, n>(reinterpret_cast<const T*>(row) + (threadIdx.x % 32) * n, v);
  }
  // `left`: channels of the piece that exist from this lane's first one on
  template <bool PAIR> __device__ __forceinline__ void put(T* p, int left) const {
    if (PAIR || n == 1) {
      if (left > 0) store_pack<T, n>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (i < left) Elem<T>::st(p + i, v[i]);
    }
  }
};

constexpr int kTokForward = 128, kTokBackward = RET_SCAN_CHUNK;
static_assert(kTokForward % RET_SCAN_CHUNK == 0, "chunk states are kept at warp boundaries");
static_assert((kTokForward / kWarps) * (RET_SCAN_CHUNK / (kTokForward / kWarps)) == RET_SCAN_CHUNK,
              "a chunk is a whole number of warps' tokens");

template <int OPERANDS, int TOK> struct Ring {
  static constexpr int kOperand = TOK * kPiece;
  static constexpr int kStage = OPERANDS * kOperand + 256;  // + one float per channel
  static constexpr int kStages = kStage <= 36 * 1024 ? 3 : 2;
  static constexpr int kBytes = kStages * kStage;  // two blocks per SM
};

// Item bookkeeping shared by the two directions: slot s of the ring holds item
// take[s]; one thread takes the next while the block computes.
template <int STAGES> struct Items {
  int take[STAGES];
};

template <typename T, int FORM, bool GATE, int W>
__global__ void __launch_bounds__(kBlock, 2) scan_items(const ScanArgs a, const Plan p) {
  using L = Lane<T>;
  using R = Ring<GATE ? 3 : 2, kTokForward>;
  constexpr int n = L::n, kTok = kTokForward, S = kTok / kWarps, C = 32 * n;
  extern __shared__ __align__(128) char ring[];
  __shared__ Items<R::kStages> items;
  __shared__ float agg_c[kWarps][C], agg_h[kWarps][C], enter[C];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const size_t pitch = (size_t)a.B * p.blocks * C;
  const int pieces = a.B * p.blocks;

  const auto load = [&](int slot) {
    const int item = items.take[slot];
    if (item < p.items) {
      const int tile = item / pieces, rest = item - tile * pieces;
      const int b = rest / p.blocks, d = (rest - b * p.blocks) * C;
      const int t = tile * kTok, rows = a.N - t, bytes = (a.D - d) * (int)sizeof(T);
      char* s = ring + slot * R::kStage;
      copy_item<W, kTok>(s, (const char*)at<const T>(a.f, b, t, d), a.f.token * sizeof(T), rows,
                         bytes);
      copy_item<W, kTok>(s + R::kOperand, (const char*)at<const T>(a.x, b, t, d),
                         a.x.token * sizeof(T), rows, bytes);
      if constexpr (GATE)
        copy_item<W, kTok>(s + 2 * R::kOperand, (const char*)at<const T>(a.gate, b, t, d),
                           a.gate.token * sizeof(T), rows, bytes);
    }
    cp_commit();
  };

  if (threadIdx.x == 0)
    for (int s = 0; s < R::kStages; ++s)
      items.take[s] = p.ticket ? atomicAdd(p.ticket, 1) + 1 : (int)(blockIdx.x + s * gridDim.x);
  __syncthreads();
  for (int s = 0; s < R::kStages; ++s) load(s);

  for (int k = 0, slot = 0;; ++k, slot = slot + 1 == R::kStages ? 0 : slot + 1) {
    const int item = items.take[slot];
    if (item >= p.items) break;
    const int tile = item / pieces, rest = item - tile * pieces;
    const int b = rest / p.blocks, d0 = (rest - b * p.blocks) * C;
    const int rows = min(kTok, a.N - tile * kTok);
    const int d = d0 + lane * n, left = a.D - d;
    const size_t words = (size_t)tile * pitch + (size_t)rest * C + lane * n;
    int next = 0;
    if (threadIdx.x == 0)
      next = p.ticket ? atomicAdd(p.ticket, 1) + 1
                      : (int)(blockIdx.x + (k + R::kStages) * gridDim.x);
    cp_wait<R::kStages - 1>();
    __syncthreads();
    const char* f = ring + slot * R::kStage + warp * S * kPiece;
    const char* x = f + R::kOperand;

    // 1. this warp's tokens from zero; tokens past the end change nothing
    float c[S][n], C_w[n], H_w[n];
#pragma unroll
    for (int i = 0; i < n; ++i) C_w[i] = H_w[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < S; ++j) {
      L fv, xv;
      fv.get(f + j * kPiece);
      xv.get(x + j * kPiece);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        c[j][i] = warp * S + j < rows ? complement<FORM>(fv.v[i]) : 0.0f;
        H_w[i] = advance<FORM>(H_w[i], c[j][i], xv.v[i]);
        C_w[i] = fmaf(c[j][i], 1.0f - C_w[i], C_w[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      agg_c[warp][lane * n + i] = C_w[i];
      agg_h[warp][lane * n + i] = H_w[i];
    }
    __syncthreads();

    // 2. the state that enters the item
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        float C_t = 0.0f, H_t = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float cw = agg_c[w][lane * n + i];
          H_t = fold(H_t, cw, agg_h[w][lane * n + i]);
          C_t = fmaf(cw, 1.0f - C_t, C_t);
        }
        C_w[i] = C_t, H_w[i] = H_t;
        if (tile > 0 && tile + 1 < p.tiles) st_words(p.span + words + i, C_t, H_t);
      }
#pragma unroll
      for (int i = 0; i < n; ++i) {
        float s;
        if (tile > 0)
          s = look_back(p, words + i, pitch, tile, kSiteForward);
        else
          s = a.state_in && i < left ? a.state_in[(size_t)b * a.D + d + i] : 0.0f;
        if (tile + 1 < p.tiles) st_word(p.end + words + i, fold(s, C_w[i], H_w[i]));
        enter[lane * n + i] = s;
      }
    }
    __syncthreads();

    // 3. the same tokens from the state that enters them
    float h[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
      h[i] = enter[lane * n + i];
      for (int w = 0; w < warp; ++w)
        h[i] = fold(h[i], agg_c[w][lane * n + i], agg_h[w][lane * n + i]);
    }
    const int t0 = tile * kTok + warp * S, mine = min(S, a.N - t0);
    if (a.chunk_states && t0 % RET_SCAN_CHUNK == 0 && mine > 0) {
      float* keep = a.chunk_states +
                    ((size_t)b * cdiv(a.N, RET_SCAN_CHUNK) + t0 / RET_SCAN_CHUNK) * a.D + d;
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (i < left) keep[i] = h[i];
    }
    T* y = at<T>(a.y, b, t0, d);
#pragma unroll
    for (int j = 0; j < S; ++j) {
      if (j < mine) {
        L xv, out;
        xv.get(x + j * kPiece);
#pragma unroll
        for (int i = 0; i < n; ++i) out.v[i] = h[i] = advance<FORM>(h[i], c[j][i], xv.v[i]);
        if constexpr (GATE) {
          L g;
          g.get(f + 2 * R::kOperand + j * kPiece);
#pragma unroll
          for (int i = 0; i < n; ++i) out.v[i] *= g.v[i] * sigmoidf(g.v[i]);
        }
        out.template put<(W >= 4)>(y, left);
        y += a.y.token;
      }
    }
    if (a.state_out && mine > 0 && t0 + mine == a.N) {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (i < left) a.state_out[(size_t)b * a.D + d + i] = h[i];
    }
    if (threadIdx.x == 0) items.take[slot] = next;
    __syncthreads();
    load(slot);
  }
  cp_wait<0>();
}

// Backward.  With G_t the gradient that reaches h_t from y_t and from
// everything after it,
//     G_t = dh_t + a_{t+1} G_{t+1},   a_N G_N := d state_out,
//     dh_t = dy_t, or dy_t swish(g_t) with a gate,
//     LOGIT  dx_t = c_t G_t,   df_t = (h_{t-1} - x_t) a_t c_t G_t
//     LOG    dx_t = G_t,       df_t = h_{t-1} a_t G_t
//     dg_t = dy_t h_t swish'(g_t),   d state_in = a_0 G_0.
// What flows to the token before, E_t = a_t G_t, obeys the same kind of
// recurrence in reversed time: a span turns the flow e behind it into
// E + e - C e with the same C.  So the items are taken from the end of the
// sequence, of one chunk each: the state that enters the chunk comes from the
// forward call, h is recomputed in float32 inside it, and the flow is looked
// for in the items after it as the forward does in those before.
template <typename T, int FORM, bool GATE, int W>
__global__ void __launch_bounds__(kBlock, 2) scan_items_backward(const ScanArgs a, const Plan p) {
  using L = Lane<T>;
  using R = Ring<GATE ? 4 : 3, kTokBackward>;
  constexpr int n = L::n, kTok = kTokBackward, S = kTok / kWarps, C = 32 * n;
  constexpr int kX = R::kOperand, kDy = 2 * R::kOperand, kGate = 3 * R::kOperand;
  constexpr int kState = (GATE ? 4 : 3) * R::kOperand;
  extern __shared__ __align__(128) char ring[];
  __shared__ Items<R::kStages> items;
  __shared__ float agg_c[kWarps][C], agg_h[kWarps][C], agg_e[kWarps][C], leave[C];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const size_t pitch = (size_t)a.B * p.blocks * C;
  const int pieces = a.B * p.blocks;

  const auto load = [&](int slot) {
    const int item = items.take[slot];
    if (item < p.items) {
      const int turn = item / pieces, rest = item - turn * pieces, tile = p.tiles - 1 - turn;
      const int b = rest / p.blocks, d = (rest - b * p.blocks) * C;
      const int t = tile * kTok, rows = a.N - t, bytes = (a.D - d) * (int)sizeof(T);
      char* s = ring + slot * R::kStage;
      copy_item<W, kTok>(s, (const char*)at<const T>(a.f, b, t, d), a.f.token * sizeof(T), rows,
                         bytes);
      copy_item<W, kTok>(s + kX, (const char*)at<const T>(a.x, b, t, d), a.x.token * sizeof(T),
                         rows, bytes);
      copy_item<W, kTok>(s + kDy, (const char*)at<const T>(a.d_y, b, t, d),
                         a.d_y.token * sizeof(T), rows, bytes);
      if constexpr (GATE)
        copy_item<W, kTok>(s + kGate, (const char*)at<const T>(a.gate, b, t, d),
                           a.gate.token * sizeof(T), rows, bytes);
      if (threadIdx.x < C) {
        const bool ok = d + (int)threadIdx.x < a.D;
        const float* st = a.chunk_states + ((size_t)b * p.tiles + tile) * a.D + d;
        cp_async<4>(sm100::smem_u32(s + kState) + threadIdx.x * 4,
                    (const char*)(st + (ok ? threadIdx.x : 0)), ok);
      }
    }
    cp_commit();
  };

  if (threadIdx.x == 0)
    for (int s = 0; s < R::kStages; ++s)
      items.take[s] = p.ticket ? atomicAdd(p.ticket, 1) + 1 : (int)(blockIdx.x + s * gridDim.x);
  __syncthreads();
  for (int s = 0; s < R::kStages; ++s) load(s);

  for (int k = 0, slot = 0;; ++k, slot = slot + 1 == R::kStages ? 0 : slot + 1) {
    const int item = items.take[slot];
    if (item >= p.items) break;
    const int turn = item / pieces, rest = item - turn * pieces, tile = p.tiles - 1 - turn;
    const int b = rest / p.blocks, d0 = (rest - b * p.blocks) * C;
    const int rows = min(kTok, a.N - tile * kTok);
    const int d = d0 + lane * n, left = a.D - d;
    const size_t words = (size_t)turn * pitch + (size_t)rest * C + lane * n;
    int next = 0;
    if (threadIdx.x == 0)
      next = p.ticket ? atomicAdd(p.ticket, 1) + 1
                      : (int)(blockIdx.x + (k + R::kStages) * gridDim.x);
    cp_wait<R::kStages - 1>();
    __syncthreads();
    const char* stage = ring + slot * R::kStage;
    const char* f = stage + warp * S * kPiece;

    // 1. this warp's tokens: forwards from a zero state, backwards from a zero flow
    float c[S][n], dh[S][n], slope[GATE ? S : 1][n], C_w[n], H_w[n], E_w[n];
#pragma unroll
    for (int i = 0; i < n; ++i) C_w[i] = H_w[i] = E_w[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < S; ++j) {
      L fv, xv, dv;
      fv.get(f + j * kPiece);
      xv.get(f + kX + j * kPiece);
      dv.get(f + kDy + j * kPiece);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        c[j][i] = warp * S + j < rows ? complement<FORM>(fv.v[i]) : 0.0f;
        H_w[i] = advance<FORM>(H_w[i], c[j][i], xv.v[i]);
        C_w[i] = fmaf(c[j][i], 1.0f - C_w[i], C_w[i]);
        dh[j][i] = dv.v[i];
      }
      if constexpr (GATE) {
        L g;
        g.get(f + kGate + j * kPiece);
#pragma unroll
        for (int i = 0; i < n; ++i) {
          float sw, sl;
          swish_grad(g.v[i], &sw, &sl);
          slope[j][i] = dh[j][i] * sl;
          dh[j][i] *= sw;
        }
      }
    }
#pragma unroll
    for (int j = S - 1; j >= 0; --j)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float G = dh[j][i] + E_w[i];
        E_w[i] = fmaf(-c[j][i], G, G);
      }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      agg_c[warp][lane * n + i] = C_w[i];
      agg_h[warp][lane * n + i] = H_w[i];
      agg_e[warp][lane * n + i] = E_w[i];
    }
    __syncthreads();

    // 2. the flow that reaches the item from behind
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        float C_t = 0.0f, E_t = 0.0f;
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
          const float cw = agg_c[w][lane * n + i];
          E_t = fold(E_t, cw, agg_e[w][lane * n + i]);
          C_t = fmaf(cw, 1.0f - C_t, C_t);
        }
        C_w[i] = C_t, E_w[i] = E_t;
        if (turn > 0 && turn + 1 < p.tiles) st_words(p.span + words + i, C_t, E_t);
      }
#pragma unroll
      for (int i = 0; i < n; ++i) {
        float s;
        if (turn > 0)
          s = look_back(p, words + i, pitch, turn, kSiteBackward);
        else
          s = a.d_state_out && i < left ? a.d_state_out[(size_t)b * a.D + d + i] : 0.0f;
        if (turn + 1 < p.tiles) st_word(p.end + words + i, fold(s, C_w[i], E_w[i]));
        leave[lane * n + i] = s;
      }
    }
    __syncthreads();

    // 3. h forwards from the state that enters, then the gradients backwards
    const int t0 = tile * kTok + warp * S, mine = min(S, a.N - t0);
    float h[n], before[S][n], flow[n];
    const float* state = reinterpret_cast<const float*>(stage + kState);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      h[i] = state[lane * n + i];
      for (int w = 0; w < warp; ++w)
        h[i] = fold(h[i], agg_c[w][lane * n + i], agg_h[w][lane * n + i]);
      flow[i] = leave[lane * n + i];
      for (int w = kWarps - 1; w > warp; --w)
        flow[i] = fold(flow[i], agg_c[w][lane * n + i], agg_e[w][lane * n + i]);
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      L xv, dg;
      xv.get(f + kX + j * kPiece);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        before[j][i] = h[i];
        h[i] = advance<FORM>(h[i], c[j][i], xv.v[i]);
        if constexpr (GATE) dg.v[i] = h[i] * slope[j][i];
      }
      if constexpr (GATE)
        if (j < mine) dg.template put<(W >= 4)>(at<T>(a.grad_gate, b, t0 + j, d), left);
    }
#pragma unroll
    for (int j = S - 1; j >= 0; --j) {
      L xv, dx, df;
      xv.get(f + kX + j * kPiece);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float G = dh[j][i] + flow[i];
        flow[i] = fmaf(-c[j][i], G, G);
        dx.v[i] = FORM == RET_SCAN_LOGIT ? c[j][i] * G : G;
        df.v[i] = FORM == RET_SCAN_LOGIT ? (before[j][i] - xv.v[i]) * c[j][i] * flow[i]
                                         : before[j][i] * flow[i];
      }
      if (j < mine) {
        dx.template put<(W >= 4)>(at<T>(a.grad_x, b, t0 + j, d), left);
        df.template put<(W >= 4)>(at<T>(a.grad_f, b, t0 + j, d), left);
      }
    }
    if (a.d_state_in && tile == 0 && warp == 0) {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (i < left) a.d_state_in[(size_t)b * a.D + d + i] = flow[i];
    }
    if (threadIdx.x == 0) items.take[slot] = next;
    __syncthreads();
    load(slot);
  }
  cp_wait<0>();
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

namespace scan {

constexpr size_t kHead = 256;  // the ticket's place at the front of the workspace

int channels_per_piece(int dtype) { return kPiece / (dtype == RET_BF16 ? 2 : 4); }

// Words of one kind (end states; half of the spans) that `tiles` items per
// piece need.
size_t words(int B, int D, int dtype, int tiles) {
  const int C = channels_per_piece(dtype);
  return (size_t)tiles * B * cdiv(D, C) * C;
}

Plan plan(const ScanArgs& a, int tok) {
  Plan p = {};
  p.blocks = cdiv(a.D, channels_per_piece(a.dtype));
  p.tiles = cdiv(a.N, tok);
  p.items = a.B * p.blocks * p.tiles;
  if (p.tiles > 1) {
    char* ws = static_cast<char*>(a.workspace);
    const size_t n = words(a.B, a.D, a.dtype, p.tiles);
    p.ticket = reinterpret_cast<int*>(ws);
    p.span = reinterpret_cast<float2*>(ws + kHead);
    p.end = reinterpret_cast<float*>(ws + kHead + n * sizeof(float2));
  }
  return p;
}

// Bytes per access of the loads: what every row of every operand is aligned
// to.  Stores take a lane's 4 bytes at once from 4 on.
int access(const ScanArgs& a) {
  const int es = a.dtype == RET_BF16 ? 2 : 4;
  size_t bits = (size_t)a.D * es;
  for (const Operand* o :
       {&a.x, &a.f, &a.gate, &a.y, &a.d_y, &a.grad_x, &a.grad_f, &a.grad_gate}) {
    if (!o->p) continue;
    bits |= reinterpret_cast<size_t>(o->p);
    if (a.B > 1) bits |= (size_t)o->batch * es;
    if (a.N > 1) bits |= (size_t)o->token * es;
  }
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

template <typename Kernel>
cudaError_t run(Kernel kernel, const ScanArgs& a, const Plan& p, int smem, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (p.ticket) {
    const size_t bytes = kHead + 12 * words(a.B, a.D, a.dtype, p.tiles);
    if ((e = cudaMemsetAsync(a.workspace, 0xff, bytes, st)) != cudaSuccess) return e;
  }
  const int most = 2 * sm_count();
  kernel<<<p.items < most ? p.items : most, kBlock, smem, st>>>(a, p);
  return cudaPeekAtLastError();
}

}  // namespace scan

int scan_device_error() { return read_clear_device_error(); }

// For either direction: the backward's items are the shorter ones.  A
// sequence of one item needs none.
size_t scan_workspace_bytes(int B, int N, int D, int dtype) {
  const int tiles = cdiv(N, scan::kTokBackward);
  return tiles > 1 ? scan::kHead + 12 * scan::words(B, D, dtype, tiles) : 0;
}

cudaError_t launch_scan(const ScanArgs& a, cudaStream_t st) {
  const scan::Plan p = scan::plan(a, scan::kTokForward);
  const int w = scan::access(a);
  return scan::dispatch(a.dtype, a.form, a.gate.p != nullptr, [&](auto t, auto form, auto gate) {
    using T = typename decltype(t)::type;
    constexpr int F = decltype(form)::value;
    constexpr bool G = decltype(gate)::value != 0;
    constexpr int smem = scan::Ring<G ? 3 : 2, scan::kTokForward>::kBytes;
    if (w == 16) return scan::run(scan::scan_items<T, F, G, 16>, a, p, smem, st);
    if (sizeof(T) == 4 || w == 4) return scan::run(scan::scan_items<T, F, G, 4>, a, p, smem, st);
    if constexpr (sizeof(T) == 2)
      return scan::run(scan::scan_items<T, F, G, 2>, a, p, smem, st);
    return cudaErrorInvalidValue;
  });
}

cudaError_t launch_scan_backward(const ScanArgs& a, cudaStream_t st) {
  const scan::Plan p = scan::plan(a, scan::kTokBackward);
  const int w = scan::access(a);
  return scan::dispatch(a.dtype, a.form, a.gate.p != nullptr, [&](auto t, auto form, auto gate) {
    using T = typename decltype(t)::type;
    constexpr int F = decltype(form)::value;
    constexpr bool G = decltype(gate)::value != 0;
    constexpr int smem = scan::Ring<G ? 4 : 3, scan::kTokBackward>::kBytes;
    if (w == 16) return scan::run(scan::scan_items_backward<T, F, G, 16>, a, p, smem, st);
    if (sizeof(T) == 4 || w == 4)
      return scan::run(scan::scan_items_backward<T, F, G, 4>, a, p, smem, st);
    if constexpr (sizeof(T) == 2)
      return scan::run(scan::scan_items_backward<T, F, G, 2>, a, p, smem, st);
    return cudaErrorInvalidValue;
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
