// Residual sum with the norms around it, and its backward.
//
// One row is the d features of one token.  With N(v) = (v - mean) r,
// r = 1 / sqrt(var + eps) (layer) or N(v) = v r, r = 1 / sqrt(mean(v^2) + eps)
// (RMS), the forward computes
//     u  = w_post (.) N_post(x)          norm after the block (optional)
//     r' = alpha residual + beta u       the residual stream
//     y  = w (.) N(r')                   norm before the next block
// ("RetNet - Retentive Network - A Successor to Transformer for LLMs",
// framework graph: norm and residual around each sub-layer), and the backward, with
// h = N(r') and hx = N_post(x),
//     dr' = r (w dy - [mean(w dy)] - h mean(w dy (.) h)) + d res_out
//     d residual = alpha dr',   dw = sum over rows of dy (.) h
//     du = beta dr',   dw_post = sum over rows of du (.) hx
//     dx = rx (w_post du - [mean(w_post du)] - hx mean(w_post du (.) hx)),
// dx = w_post du without the norm after the block ([] for layer norms only).
//
// Bound by HBM: x, the residual and both outputs cross it once.  A row stays
// in the registers of TPR threads, and its sums go through warp shuffles and,
// for rows longer than a warp's, shared memory.  y is computed from r' before
// its rounding to the storage type, so y carries one rounding only; the
// backward starts from the stored r'.
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "rowvec.cuh"
#include "sm100.cuh"

namespace ret {
namespace an {

// Sums of a and b over the TPR threads of a row.  `slot` (two floats per
// warp) may be used again once every thread has passed another sum's barrier.
template <int TPR> __device__ __forceinline__ void row_sum2(float& a, float& b, float2* slot) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    if (threadIdx.x % 32 == 0) slot[threadIdx.x / 32] = make_float2(a, b);
    asm volatile("bar.sync 1, %0;" ::"n"(TPR) : "memory");
    a = 0.0f, b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) a += slot[w].x, b += slot[w].y;
  }
}
template <int TPR> __device__ __forceinline__ float row_sum(float a, float2* slot) {
  float b = 0.0f;
  row_sum2<TPR>(a, b, slot);
  return a;
}

// Row geometry: CH accesses of V elements per thread and tensor.
template <typename T, int V, int CH, int TPR, bool FULL = false> struct Geo {
  using type = T;
  using Full = Geo<T, V, CH, TPR, true>;  // for rows of exactly CH V TPR elements
  static constexpr bool kFull = FULL;
  static constexpr int kV = V, kCH = CH, kTPR = TPR;
  static constexpr int kThreads = TPR < 64 ? 128 : TPR;  // several short rows per block
  static constexpr int kRows = kThreads / TPR;
};

template <typename G>
struct Row : RowPart<typename G::type, G::kV, G::kCH, G::kTPR, G::kFull> {
  static constexpr int V = G::kV, CH = G::kCH, TPR = G::kTPR;
  using Base = RowPart<typename G::type, V, CH, TPR, G::kFull>;
  using Base::P;
  using Base::p;
  // v <- v (.) w
  __device__ __forceinline__ void scale(const float* w, int lane, int nv) {
    constexpr int Q = V < 4 ? V : 4;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = c * TPR + lane;
      if (i < nv) {
#pragma unroll
        for (int j = 0; j < V; j += Q) {
          float f[Q];
          load_pack<float, Q>(w + (long long)i * V + j, f);
#pragma unroll
          for (int k = 0; k < Q; ++k) this->put(c * V + j + k, this->get(c * V + j + k) * f[k]);
        }
      }
    }
  }
  // v <- N(v); returns r.  slots: two of row_sum2's
  __device__ __forceinline__ float norm(int lane, int nv, bool layer, float eps, float inv_d,
                                        float2* slots) {
    return this->normalise(lane, nv, layer, eps, inv_d, [&](float x, int which) {
      return row_sum<TPR>(x, slots + 32 * which);
    });
  }
  // v <- r (v - [mean(v)] - h mean(v (.) h)), the norm's backward
  __device__ __forceinline__ void norm_backward(const Row& h, float r, int lane, int nv, bool layer,
                                                float inv_d, float2* slot) {
    Vec<2> p1 = all<2>(0.0f), p2 = p1;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      p1 = add(p1, p[i]);
      p2 = fma(p[i], h.p[i], p2);
    }
    float s1 = total(p1), s2 = total(p2);
    row_sum2<TPR>(s1, s2, slot);
    s1 = layer ? s1 * -inv_d : 0.0f;
    s2 *= -inv_d;
#pragma unroll
    for (int i = 0; i < P; ++i)
      p[i] = mul(all<2>(r), fma(h.p[i], all<2>(s2), add(p[i], all<2>(s1))));
    if (layer) this->clear_rest(lane, nv);
  }
  // v <- v + a (.) b
  __device__ __forceinline__ void add_product(const Row& a, const Row& b) {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = fma(a.p[i], b.p[i], p[i]);
  }
  __device__ __forceinline__ void times(float f) {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = mul(p[i], all<2>(f));
  }
};

template <typename G>
__global__ void __launch_bounds__(G::kThreads)
add_norm_rows(AddNormArgs a) {
  using T = typename G::type;
  using R = Row<G>;
  __shared__ float2 slots[4 * 32];
  const int lane = threadIdx.x % G::kTPR, nv = a.d / G::kV;
  const long long n = (long long)blockIdx.x * G::kRows + threadIdx.x / G::kTPR;
  const int take = n < a.rows ? nv : 0;  // threads past the last row only join the sums
  const long long at = min(n, a.rows - 1) * a.d;
  const float inv_d = 1.0f / a.d;
  R u, s;
  u.load(static_cast<const T*>(a.x) + at, lane, take);
  if (a.residual) s.load(static_cast<const T*>(a.residual) + at, lane, take);
  if (a.post_norm != RET_NORM_NONE)
    u.norm(lane, take, a.post_norm == RET_NORM_LAYER, a.eps, inv_d, slots);
  if (a.w_post) u.scale(a.w_post, lane, take);
  u.times(a.beta);
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < R::P; ++i)
      u.p[i] = fma(all<2>(a.alpha), s.p[i], u.p[i]);
  }
  u.store(static_cast<T*>(a.res_out) + at, lane, take);
  u.norm(lane, take, a.norm == RET_NORM_LAYER, a.eps, inv_d, slots + 64);
  if (a.w) u.scale(a.w, lane, take);
  u.store(static_cast<T*>(a.y) + at, lane, take);
}

// A block's sums of the weight gradients, one partial row of the workspace for
// each of the rows that it works on at a time.
template <typename G>
__device__ __forceinline__ void put_partials(const AddNormArgs& a, int lane, int nv, long long part,
                                             const Row<G>& acc_w, const Row<G>& acc_post,
                                             float* part_w, float* part_post) {
  constexpr int Q = G::kV < 4 ? G::kV : 4;
#pragma unroll
  for (int c = 0; c < G::kCH; ++c) {
    const int i = c * G::kTPR + lane;
    if (i >= nv) continue;
#pragma unroll
    for (int k = 0; k < G::kV; k += Q) {
      float f[Q];
      const long long to = part * a.d + (long long)i * G::kV + k;
      if (part_w) {
#pragma unroll
        for (int j = 0; j < Q; ++j) f[j] = acc_w.get(c * G::kV + k + j);
        store_pack<float, Q>(part_w + to, f);
      }
      if (part_post) {
#pragma unroll
        for (int j = 0; j < Q; ++j) f[j] = acc_post.get(c * G::kV + k + j);
        store_pack<float, Q>(part_post + to, f);
      }
    }
  }
}

// Persistent over rows, loads straight into registers: rows under 512 bytes
// (several per block), and those that the ring below cannot hold, wider than
// 16 KB (8192 elements where they do not split into 16-byte pieces).
template <typename G>
__global__ void __launch_bounds__(G::kThreads)
add_norm_rows_backward(AddNormArgs a, float* part_w, float* part_post) {
  using T = typename G::type;
  using R = Row<G>;
  __shared__ float2 slots[6 * 32];
  const int lane = threadIdx.x % G::kTPR, nv = a.d / G::kV;
  const float inv_d = 1.0f / a.d;
  const bool post = a.post_norm != RET_NORM_NONE;
  R acc_w, acc_post;
#pragma unroll
  for (int i = 0; i < R::P; ++i) acc_w.p[i] = acc_post.p[i] = all<2>(0.0f);
  const long long groups = (a.rows + G::kRows - 1) / G::kRows;
  for (long long g = blockIdx.x; g < groups; g += gridDim.x) {
    const long long n = g * G::kRows + threadIdx.x / G::kTPR;
    const int take = n < a.rows ? nv : 0;
    const long long at = min(n, a.rows - 1) * a.d;
    R h, d, s, x;
    h.load(static_cast<const T*>(a.res_out) + at, lane, take);
    d.load(static_cast<const T*>(a.d_y) + at, lane, take);
    if (a.d_res_out) s.load(static_cast<const T*>(a.d_res_out) + at, lane, take);
    if (post || part_post) x.load(static_cast<const T*>(a.x) + at, lane, take);
    const float r = h.norm(lane, take, a.norm == RET_NORM_LAYER, a.eps, inv_d, slots);
    if (part_w) acc_w.add_product(d, h);
    if (a.w) d.scale(a.w, lane, take);
    d.norm_backward(h, r, lane, take, a.norm == RET_NORM_LAYER, inv_d, slots + 64);
    if (a.d_res_out) {
#pragma unroll
      for (int i = 0; i < R::P; ++i) d.p[i] = add(d.p[i], s.p[i]);
    }
    if (a.grad_residual) {
      s = d;
      s.times(a.alpha);
      s.store(static_cast<T*>(a.grad_residual) + at, lane, take);
    }
    d.times(a.beta);
    float rx = 1.0f;
    if (post) rx = x.norm(lane, take, a.post_norm == RET_NORM_LAYER, a.eps, inv_d, slots + 96);
    if (part_post) acc_post.add_product(d, x);
    if (a.grad_x) {
      if (a.w_post) d.scale(a.w_post, lane, take);
      if (post)
        d.norm_backward(x, rx, lane, take, a.post_norm == RET_NORM_LAYER, inv_d, slots + 160);
      d.store(static_cast<T*>(a.grad_x) + at, lane, take);
    }
  }
  put_partials<G>(a, lane, nv, (long long)blockIdx.x * G::kRows + threadIdx.x / G::kTPR, acc_w,
                  acc_post, part_w, part_post);
}

// The same with the rows coming through a ring in shared memory.  A block is
// as many groups of TPR threads as an SM holds, each working on a row of its
// own with the next ones on their way (its first thread copies whole rows, each
// tensor's being one contiguous piece): while one group waits for its row's
// sums another computes.  A thread has 32 elements of a row, so the
// sums cost few instructions per element; both norms' moments cross the group
// in one exchange, each warp taking its own about its own mean and the group
// joining them (Chan, Golub and LeVeque's pairwise variance); and the weights
// wait in shared memory.  65536 x 4096 in bf16, both norms and both weights:
// 1027 us with loads in registers and five exchanges, 670 through rings of
// two blocks per SM with 16 elements per thread, 600 with three groups of
// 128 threads.
constexpr int kSiteRing = 811;
constexpr int kMaxStages = 4;
// The same serves rows that are not 16-byte aligned: they come as the granules
// that cover them (the bytes before a row lie in its own first 16 bytes of
// memory; none behind it is read), and threads take single elements.  16384 x
// 4095 in bf16, an RMS and a layer norm: 824 us with single elements from HBM,
// 399 so.
constexpr int kGranuleStages = 2;
constexpr int kRingWarps = 12;  // three on each scheduler: 168 registers a thread
constexpr int kRingBytes = 225 * 1024;  // beside 1 KB of barriers and sums

// Bytes of the ring for a row of `bytes`.
__host__ __device__ constexpr int ring_row(int bytes, bool whole) {
  return whole ? bytes : (bytes + 14 + 15) / 16 * 16;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, uintptr_t src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

__device__ __forceinline__ Vec<2> warp_sum(Vec<2> x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = add(x, two(__shfl_xor_sync(0xffffffffu, x[0], o),
                   __shfl_xor_sync(0xffffffffu, x[1], o)));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A row's mean (0 for RMS) and 1 / spread.
struct Moments {
  float mean, r;
};

template <typename G> struct Block {
  static constexpr int W = G::kTPR / 32;
  static constexpr int kLane = G::kCH * G::kV;  // elements of a thread in a full row
  // The group's barrier; a warp by itself needs its memory ordered only.
  static __device__ __forceinline__ void sync(int group) {
    if constexpr (W == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(G::kTPR) : "memory");
  }
  // Elements of the row that warp w holds.
  static __device__ __forceinline__ int held(int w, int nv) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < G::kCH; ++c) n += min(max(nv - (c * G::kTPR + w * 32), 0), 32);
    return n * G::kV;
  }
  // One warp's mean (layer) and sum of squares about it.
  static __device__ __forceinline__ float2 own(const Row<G>& v, bool layer, int lane, int nv) {
    using R = Row<G>;
    float mean = 0.0f;
    if (layer) {
      Vec<2> s = all<2>(0.0f);
#pragma unroll
      for (int i = 0; i < R::P; ++i) s = add(s, v.p[i]);
      const int n = G::kFull ? 32 * kLane : held(lane / 32, nv);
      const float sum = warp_sum(total(s));
      mean = n > 0 ? __fdividef(sum, (float)n) : 0.0f;
    }
    Vec<2> q = all<2>(0.0f);
    if (layer) {
      R t = v;
#pragma unroll
      for (int i = 0; i < R::P; ++i) t.p[i] = add(t.p[i], all<2>(-mean));
      t.clear_rest(lane, nv);
#pragma unroll
      for (int i = 0; i < R::P; ++i) q = fma(t.p[i], t.p[i], q);
    } else {
#pragma unroll
      for (int i = 0; i < R::P; ++i) q = fma(v.p[i], v.p[i], q);
    }
    return make_float2(mean, total(q));  // the squares still spread over the lanes
  }
  // The row's moments from the warps' (.x mean, .y sum of squares about it).
  template <typename Get>
  static __device__ __forceinline__ Moments join(Get get, bool layer, float eps, float inv_d,
                                                 int nv) {
    float mean = 0.0f, m2 = 0.0f;
    if (!layer) {
#pragma unroll
      for (int w = 0; w < W; ++w) m2 += get(w).y;
    } else if (G::kFull) {  // every warp holds as much
      float apart = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) mean += get(w).x;
      mean *= 1.0f / W;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 g = get(w);
        m2 += g.y;
        apart = fmaf(g.x - mean, g.x - mean, apart);
      }
      m2 = fmaf(apart, 32.0f * kLane, m2);
    } else {
      for (int w = 0; w < W; ++w) mean = fmaf(get(w).x, held(w, nv) * inv_d, mean);
      for (int w = 0; w < W; ++w) {
        const float2 g = get(w);
        m2 += fmaf((g.x - mean) * (g.x - mean), (float)held(w, nv), g.y);
      }
    }
    return {mean, rsqrtf(fmaf(m2, inv_d, eps))};
  }
  // Both sums over the group.
  static __device__ __forceinline__ Vec<2> sum(Vec<2> x, float2* slot, int group, int lane) {
    x = warp_sum(x);
    if constexpr (W > 1) {
      if (lane % 32 == 0) slot[lane / 32] = make_float2(x[0], x[1]);
      sync(group);
      x = all<2>(0.0f);
#pragma unroll
      for (int w = 0; w < W; w += 2) {
        const float4 f = *reinterpret_cast<const float4*>(slot + w);
        x = add(x, add(two(f.x, f.y), two(f.z, f.w)));
      }
    }
    return x;
  }
  // v <- (v - mean) r
  static __device__ __forceinline__ void apply(Row<G>& v, Moments m, bool layer, int lane,
                                               int nv) {
#pragma unroll
    for (int i = 0; i < Row<G>::P; ++i)
      v.p[i] = fma(v.p[i], all<2>(m.r), all<2>(-m.mean * m.r));
    if (layer) v.clear_rest(lane, nv);
  }
  // d <- r (d - [mean(d)] - h mean(d (.) h))
  static __device__ __forceinline__ void back(Row<G>& d, const Row<G>& h, float r, bool layer,
                                              float inv_d, float2* slot, int group, int lane,
                                              int nv) {
    using R = Row<G>;
    Vec<2> p1 = all<2>(0.0f), p2 = p1;
#pragma unroll
    for (int i = 0; i < R::P; ++i) {
      p1 = add(p1, d.p[i]);
      p2 = fma(d.p[i], h.p[i], p2);
    }
    const Vec<2> s = sum(two(total(p1), total(p2)), slot, group, lane);
    const float s1 = layer ? s[0] * -inv_d : 0.0f, s2 = s[1] * -inv_d;
#pragma unroll
    for (int i = 0; i < R::P; ++i)
      d.p[i] = mul(all<2>(r), fma(h.p[i], all<2>(s2), add(d.p[i], all<2>(s1))));
    if (layer) d.clear_rest(lane, nv);
  }
  // v <- v (.) w
  static __device__ __forceinline__ void scale(Row<G>& v, const float* w, int lane, int nv) {
    if constexpr (G::kV == 1) {
#pragma unroll
      for (int i = 0; i < Row<G>::P; ++i) {
        const int c0 = 2 * i * G::kTPR + lane, c1 = c0 + G::kTPR;
        v.p[i] = mul(v.p[i], two(c0 < nv ? w[c0] : 0.0f, c1 < nv ? w[c1] : 0.0f));
      }
    } else {
#pragma unroll
      for (int c = 0; c < G::kCH; ++c) {
        const int i = c * G::kTPR + lane;
        if (G::kFull || i < nv) {
#pragma unroll
          for (int j = 0; j < G::kV; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(w + i * G::kV + j);
            const int k = (c * G::kV + j) / 2;
            v.p[k] = mul(v.p[k], two(f.x, f.y));
            v.p[k + 1] = mul(v.p[k + 1], two(f.z, f.w));
          }
        }
      }
    }
  }
};

template <typename G>
__global__ void __launch_bounds__(32 * kRingWarps, 1)
add_norm_ring_backward(AddNormArgs a, float* part_w, float* part_post, int groups, int stages) {
  using T = typename G::type;
  using R = Row<G>;
  using B = Block<G>;
  constexpr int kMaxGroups = kRingWarps / B::W;
  extern __shared__ __align__(128) char ring[];
  __shared__ float4 moments[kMaxGroups][B::W];
  __shared__ __align__(16) float2 slots[kMaxGroups][2][B::W];
  __shared__ uint64_t full[kMaxGroups][kMaxStages];
  const bool post = a.post_norm != RET_NORM_NONE, need_x = post || part_post;
  const bool layer = a.norm == RET_NORM_LAYER, layer_post = a.post_norm == RET_NORM_LAYER;
  // a row's place in the ring: its bytes, or the 16-byte granules that cover it
  constexpr bool kWhole = G::kV > 1;
  const uint32_t row = ring_row(a.d * (int)sizeof(T), kWhole);
  const uint32_t stage = row * (2 + (a.d_res_out ? 1 : 0) + (need_x ? 1 : 0));
  // behind the groups' rings, the weights
  float* w = reinterpret_cast<float*>(ring + groups * stages * stage);
  float* w_post = w + (a.w ? a.d : 0);
  if (threadIdx.x == 0) {
    for (int g = 0; g < groups; ++g)
      for (int s = 0; s < stages; ++s) sm100::mbar_init(&full[g][s], 1);
    sm100::fence_mbar_init();
  }
  for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
    if (a.w) w[i] = a.w[i];
    if (a.w_post) w_post[i] = a.w_post[i];
  }
  __syncthreads();
  const int group = threadIdx.x / G::kTPR, lane = threadIdx.x % G::kTPR, nv = a.d / G::kV;
  const long long first = (long long)blockIdx.x * groups, step = (long long)gridDim.x * groups;
  R acc_w, acc_post;
#pragma unroll
  for (int i = 0; i < R::P; ++i) acc_w.p[i] = acc_post.p[i] = all<2>(0.0f);
  int fetched = 0;  // rows, by the group's first thread
  // Row n into stage s: by the group's first thread, as bulk copies; rows that
  // are not 16-byte aligned by all of its threads, granule by granule.
  const auto fetch = [&](long long n, int s) {
    if constexpr (!kWhole) {
      if (n < a.rows) {
        const uint32_t to = sm100::smem_u32(ring + (group * stages + s) * stage);
        const auto copy = [&](const void* p, uint32_t place) {
          const uintptr_t start = reinterpret_cast<uintptr_t>(static_cast<const T*>(p) + n * a.d);
          const uintptr_t end = start + a.d * sizeof(T);
          for (uint32_t at = lane * 16; at < row; at += G::kTPR * 16) {
            const uintptr_t granule = (start & ~(uintptr_t)15) + at;
            if (granule < end)
              cp_async16(to + place + at, granule, end - granule < 16 ? (int)(end - granule) : 16);
          }
        };
        copy(a.res_out, 0);
        copy(a.d_y, row);
        if (a.d_res_out) copy(a.d_res_out, 2 * row);
        if (need_x) copy(a.x, stage - row);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return;
    }
    if (lane != 0 || n >= a.rows) return;
    char* to = ring + (group * stages + s) * stage;
    const auto load = [&](const void* p, uint32_t place) {
      sm100::bulk_load(to + place, static_cast<const T*>(p) + n * a.d, row, &full[group][s]);
    };
    ++fetched;
    sm100::mbar_arrive_expect_tx(&full[group][s], stage);
    load(a.res_out, 0);
    load(a.d_y, row);
    if (a.d_res_out) load(a.d_res_out, 2 * row);
    if (need_x) load(a.x, stage - row);
  };
  for (int s = 0; s < stages; ++s) fetch(first + group + s * step, s);
  const float inv_d = 1.0f / a.d;
  int s = 0, phase = 0;
  bool ok = true;  // every row waited for has landed
  for (long long n = first + group; n < a.rows; n += step) {
    if constexpr (kWhole) {
      ok = sm100::mbar_wait(&full[group][s], phase, kSiteRing + 1) && ok;
    } else {
      asm volatile("cp.async.wait_group %0;" ::"n"(kGranuleStages - 1) : "memory");
      B::sync(group);
    }
    const char* here = ring + (group * stages + s) * stage;
    const long long at = n * a.d;
    const auto load = [&](R& part, uint32_t place, const void* p) {
      const uint32_t off =
          kWhole ? 0 : (uint32_t) reinterpret_cast<uintptr_t>(static_cast<const T*>(p) + at) & 15;
      part.load(reinterpret_cast<const T*>(here + place + off), lane, nv);
    };
    R h, d;
    // both norms' moments
    float2 mine_x = make_float2(0.0f, 0.0f);
    if (post) {
      load(d, stage - row, a.x);
      mine_x = B::own(d, layer_post, lane, nv);
    }
    load(h, 0, a.res_out);
    const float2 mine_h = B::own(h, layer, lane, nv);
    const Vec<2> m2 = warp_sum(two(mine_h.y, mine_x.y));
    if (lane % 32 == 0)
      moments[group][lane / 32] = make_float4(mine_h.x, m2[0], mine_x.x, m2[1]);
    B::sync(group);
    const Moments mh = B::join(
        [&](int i) { return make_float2(moments[group][i].x, moments[group][i].y); }, layer,
        a.eps, inv_d, nv);
    Moments mx = {0.0f, 1.0f};
    if (post)
      mx = B::join([&](int i) { return make_float2(moments[group][i].z, moments[group][i].w); },
                   layer_post, a.eps, inv_d, nv);
    if (B::W == 1) __syncwarp();  // read before the next row's are written
    // through the norm before the next block
    B::apply(h, mh, layer, lane, nv);
    load(d, row, a.d_y);
    if (part_w) acc_w.add_product(d, h);
    if (a.w) B::scale(d, w, lane, nv);
    B::back(d, h, mh.r, layer, inv_d, slots[group][0], group, lane, nv);
    if (a.d_res_out) {
      load(h, 2 * row, a.d_res_out);
#pragma unroll
      for (int i = 0; i < R::P; ++i) d.p[i] = add(d.p[i], h.p[i]);
    }
    if (a.grad_residual) {
      h = d;
      h.times(a.alpha);
      h.store(static_cast<T*>(a.grad_residual) + at, lane, nv);
    }
    d.times(a.beta);
    // and through the one after the block
    if (need_x) load(h, stage - row, a.x);
    B::sync(group);  // the stage has been read
    if (ok) fetch(n + stages * step, s);  // after a wait gave up a copy may be under way
    if (post) B::apply(h, mx, layer_post, lane, nv);
    if (part_post) acc_post.add_product(d, h);
    if (a.grad_x) {
      if (a.w_post) B::scale(d, w_post, lane, nv);
      if (post) B::back(d, h, mx.r, layer_post, inv_d, slots[group][1], group, lane, nv);
      d.store(static_cast<T*>(a.grad_x) + at, lane, nv);
    }
    if (++s == stages) s = 0, phase ^= 1;
  }
  // and they end before the block does
  if (kWhole && lane == 0 && !ok)
    for (int i = 0; i < stages; ++i)
      if (fetched > i) sm100::mbar_drain(&full[group][i], ((fetched - 1 - i) / stages) % 2);
  if constexpr (!kWhole) asm volatile("cp.async.wait_group 0;" ::: "memory");
  // the groups' sums, through the place of their rings, in the groups' order
  float* sums = reinterpret_cast<float*>(ring);
  for (int which = 0; which < 2; ++which) {
    float* part = which ? part_post : part_w;
    if (!part) continue;
    __syncthreads();
    put_partials<G>(a, lane, nv, group, which ? acc_post : acc_w, acc_w, sums, nullptr);
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
      float s = sums[i];
      for (int g = 1; g < groups; ++g) s += sums[(long long)g * a.d + i];
      part[(long long)blockIdx.x * a.d + i] = s;
    }
  }
}

// grad[c] = sum of the partial rows, in a fixed order: 8 warps take every
// eighth row of 32 columns, then their sums are added in order.
constexpr int kReduceWarps = 8;
__global__ void __launch_bounds__(32 * kReduceWarps)
sum_partials(const float* __restrict__ part_w, const float* __restrict__ part_post,
             float* __restrict__ grad_w, float* __restrict__ grad_post, int parts, int d) {
  __shared__ float s[kReduceWarps][32];
  const float* part = blockIdx.y ? part_post : part_w;
  float* grad = blockIdx.y ? grad_post : grad_w;
  if (!part) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < d)
    for (int p = warp; p < parts; p += kReduceWarps) sum += part[(long long)p * d + col];
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < d) {
    for (int w = 1; w < kReduceWarps; ++w) sum += s[w][lane];
    grad[col] = sum;
  }
}

// Whether every row of every tensor splits into 16-byte pieces.
bool vectored(const AddNormArgs& a) {
  const int es = a.dtype == RET_BF16 ? 2 : 4;
  if ((long long)a.d * es % 16) return false;
  for (const void* p : {a.x, a.residual, (const void*)a.res_out, (const void*)a.y, a.d_y,
                        a.d_res_out, (const void*)a.grad_x, (const void*)a.grad_residual})
    if (p && !aligned_to(p, 16)) return false;
  return true;
}

template <typename T, int V, int CH, typename Fn> cudaError_t by_threads(int nv, Fn fn) {
  if (nv <= 32 * CH) return fn(Geo<T, V, CH, 32>());
  if (nv <= 64 * CH) return fn(Geo<T, V, CH, 64>());
  if (nv <= 128 * CH) return fn(Geo<T, V, CH, 128>());
  if (nv <= 256 * CH) return fn(Geo<T, V, CH, 256>());
  if (nv <= 512 * CH) return fn(Geo<T, V, CH, 512>());
  return fn(Geo<T, V, CH, 1024>());
}

// Calls fn with the row geometry for these sizes; d <= 16384.
template <typename Fn> cudaError_t by_geometry(const AddNormArgs& a, Fn fn) {
  const bool bf16 = a.dtype == RET_BF16;
  if (vectored(a)) {
    if (bf16) return by_threads<__nv_bfloat16, 8, 2>(a.d / 8, fn);
    return a.d <= 8192 ? by_threads<float, 4, 2>(a.d / 4, fn) : fn(Geo<float, 4, 4, 1024>());
  }
  if (bf16)
    return a.d <= 8192 ? by_threads<__nv_bfloat16, 1, 8>(a.d, fn)
                       : fn(Geo<__nv_bfloat16, 1, 16, 1024>());
  return a.d <= 8192 ? by_threads<float, 1, 8>(a.d, fn) : fn(Geo<float, 1, 16, 1024>());
}

// Blocks of the backward.  A fixed count, so that the order of the weight
// gradients' sums does not depend on the device.
constexpr int kMaxBlocks = 592;   // four per SM
constexpr int kRingBlocks = 148;  // one per SM

}  // namespace an

size_t add_norm_backward_workspace_bytes(long long rows, int d) {
  // a block leaves one partial row per weight, or one for each of its four
  // rows where rows are short enough for a warp (512 elements at most)
  const long long per_block = d <= 512 ? 4 : 1;
  const long long parts =
      per_block * (rows < an::kMaxBlocks ? (rows > 0 ? rows : 0) : an::kMaxBlocks);
  return sizeof(float) * 2 * (size_t)parts * d;
}

cudaError_t launch_add_norm(const AddNormArgs& a, cudaStream_t st) {
  return an::by_geometry(a, [&](auto geo) {
    using G = decltype(geo);
    const unsigned grid = static_cast<unsigned>((a.rows + G::kRows - 1) / G::kRows);
    an::add_norm_rows<G><<<grid, G::kThreads, 0, st>>>(a);
    return cudaPeekAtLastError();
  });
}

namespace an {

constexpr int kMaxDevices = 64;

// Shape of the ring kernel's blocks for rows of this size.
struct RingPlan {
  int groups = 0, stages = 0, smem = 0;  // no groups: it does not serve
};
template <typename G> RingPlan ring_plan(const AddNormArgs& a) {
  RingPlan p;
  const int tensors = 2 + (a.d_res_out ? 1 : 0) +
                      (a.post_norm != RET_NORM_NONE || a.grad_w_post ? 1 : 0);
  const int stage = tensors * ring_row(a.d * (int)sizeof(typename G::type), G::kV > 1);
  // (an odd width leaves the second weight's row unaligned: only single elements read it)
  const int weights = a.d * 4 * ((a.w ? 1 : 0) + (a.w_post ? 1 : 0));
  const int fit = (kRingBytes - weights) / (2 * stage), most = kRingWarps / (G::kTPR / 32);
  p.groups = fit < most ? fit : most;
  if (p.groups < 1) return RingPlan();
  p.stages = (kRingBytes - weights) / (p.groups * stage);
  const int most_stages = G::kV > 1 ? kMaxStages : kGranuleStages;
  if (p.stages > most_stages) p.stages = most_stages;
  p.smem = p.groups * p.stages * stage + weights;
  return p;
}

template <typename G>
cudaError_t run_ring(const AddNormArgs& a, float* ws, int* parts, cudaStream_t st) {
  const RingPlan p = ring_plan<G>(a);
  *parts = 0;
  if (!p.groups) return cudaSuccess;
  const long long want = (a.rows + p.groups - 1) / p.groups;
  const int grid = static_cast<int>(want < kRingBlocks ? want : kRingBlocks);
  const bool exact = a.d == G::kCH * G::kV * G::kTPR;
  const auto kernel = exact ? add_norm_ring_backward<typename G::Full> : add_norm_ring_backward<G>;
  // the permission for the shared memory is asked for once per kernel and device
  static std::atomic<bool> allowed[2][kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !allowed[exact][dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) allowed[exact][dev].store(true);
  }
  kernel<<<grid, p.groups * G::kTPR, p.smem, st>>>(
      a, a.grad_w ? ws : nullptr,
      a.grad_w_post ? ws + (a.grad_w ? (size_t)grid * a.d : (size_t)0) : nullptr, p.groups,
      p.stages);
  *parts = grid;
  return cudaPeekAtLastError();
}

template <typename T>
cudaError_t by_elements(const AddNormArgs& a, float* ws, int* parts, cudaStream_t st) {
  if (a.d <= 256) return run_ring<Geo<T, 1, 8, 32>>(a, ws, parts, st);
  if (a.d <= 512) return run_ring<Geo<T, 1, 16, 32>>(a, ws, parts, st);
  if (a.d <= 1024) return run_ring<Geo<T, 1, 32, 32>>(a, ws, parts, st);
  if (a.d <= 2048) return run_ring<Geo<T, 1, 32, 64>>(a, ws, parts, st);
  if (a.d <= 4096) return run_ring<Geo<T, 1, 32, 128>>(a, ws, parts, st);
  if (a.d <= 8192) return run_ring<Geo<T, 1, 32, 256>>(a, ws, parts, st);
  return cudaSuccess;
}

// Rows of at least 512 bytes, if two of them fit; *parts stays 0 where the ring
// does not serve.
cudaError_t through_ring(const AddNormArgs& a, float* ws, int* parts, cudaStream_t st) {
  using bf16 = __nv_bfloat16;
  *parts = 0;
  const bool half = a.dtype == RET_BF16;
  if (a.d * (half ? 2 : 4) < 512) return cudaSuccess;
  if (!vectored(a)) return half ? by_elements<bf16>(a, ws, parts, st)
                                : by_elements<float>(a, ws, parts, st);
  const int nv = a.d * (half ? 2 : 4) / 16;
  if (nv > 1024) return cudaSuccess;
  if (half) {
    if (nv <= 64) return run_ring<Geo<bf16, 8, 2, 32>>(a, ws, parts, st);
    if (nv <= 128) return run_ring<Geo<bf16, 8, 4, 32>>(a, ws, parts, st);
    if (nv <= 256) return run_ring<Geo<bf16, 8, 4, 64>>(a, ws, parts, st);
    if (nv <= 512) return run_ring<Geo<bf16, 8, 4, 128>>(a, ws, parts, st);
    return run_ring<Geo<bf16, 8, 4, 256>>(a, ws, parts, st);
  }
  if (nv <= 128) return run_ring<Geo<float, 4, 4, 32>>(a, ws, parts, st);
  if (nv <= 256) return run_ring<Geo<float, 4, 8, 32>>(a, ws, parts, st);
  if (nv <= 512) return run_ring<Geo<float, 4, 8, 64>>(a, ws, parts, st);
  return run_ring<Geo<float, 4, 8, 128>>(a, ws, parts, st);
}

}  // namespace an

int add_norm_device_error() { return read_clear_device_error(); }

cudaError_t launch_add_norm_backward(const AddNormArgs& a, float* ws, cudaStream_t st) {
  int parts = 0;
  cudaError_t e = an::through_ring(a, ws, &parts, st);
  if (e != cudaSuccess) return e;
  if (!parts) {
    e = an::by_geometry(a, [&](auto geo) {
      using G = decltype(geo);
      const long long groups = (a.rows + G::kRows - 1) / G::kRows;
      const int grid = static_cast<int>(groups < an::kMaxBlocks ? groups : an::kMaxBlocks);
      parts = grid * G::kRows;
      float* part_post =
          a.grad_w_post ? ws + (a.grad_w ? (size_t)parts * a.d : (size_t)0) : nullptr;
      an::add_norm_rows_backward<G>
          <<<grid, G::kThreads, 0, st>>>(a, a.grad_w ? ws : nullptr, part_post);
      return cudaPeekAtLastError();
    });
  }
  if (e != cudaSuccess || !(a.grad_w || a.grad_w_post)) return e;
  const float* part_post = ws + (a.grad_w ? (size_t)parts * a.d : (size_t)0);
  an::sum_partials<<<dim3(cdiv(a.d, 32), 2), 32 * an::kReduceWarps, 0, st>>>(
      a.grad_w ? ws : nullptr, a.grad_w_post ? part_post : nullptr, a.grad_w, a.grad_w_post, parts,
      a.d);
  return cudaPeekAtLastError();
}

}  // namespace ret
