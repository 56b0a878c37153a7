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
// A decay is kept as one float32 m with its full relative precision at both
// ends of its range:
//     m < 0    a = 1 + m     (rounded as a, a decay close to 1 would be off by
//                            up to 2^-25 every token, the same way each time
//                            where the gate is steady)
//     m >= 0   a = m         (held as a - 1, a decay close to 0 would be off by
//                            2^-25 of 1: by 0.1 to 0.9% at e^-12, all of it at
//                            e^-18, and with it the gradient of f)
// and a decay of exactly 1 as -2^-126, so that the sign tells the two apart
// (every part of 1 down to 2^-126 is kept).  With c = 1 where m < 0 and 0
// elsewhere, a z = m z + c z; a token with a zero decay drops all that was
// before it.  The state itself is carried as z = h (LOG) or z = -h (LOGIT),
// so that its input is q x with q = a - 1 and no negation.
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "rowvec.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace ret {
namespace scan {

constexpr float kLeast = 1.17549435e-38f;  // 2^-126

// c: 1 where the decay is 1 + m, 0 where it is m.  By a multiplication that
// saturates (m below 0 is at most -2^-126), which leaves the integer pipe to the
// conversions (65536 x 4096 in bf16: 306 us by comparison, 300 so), and again
// where it is needed, as the tokens' c would fill the registers.
template <int n> __device__ __forceinline__ Vec<n> near_one(Vec<n> m) {
  float c[n];
#pragma unroll
  for (int i = 0; i < n; ++i)
    asm volatile("mul.sat.f32 %0, %1, 0fff000000;" : "=f"(c[i]) : "f"(m[i]));  // -2^127
  return vec(c);
}

// A token's decay, from its f.
//     LOGIT  q = a - 1 = -1 / (1 + e^f), of full relative precision for every f
//            (an overflow of e^f gives 0); a = -q e^f
//     LOG    a = e^f; a - 1 by its Taylor series from f = -1/4 on (six terms
//            leave 5e-8 of the value)
template <int n> struct Decay {
  Vec<n> m, a;
  Vec<n> q;  // LOGIT only
};
template <int FORM, int n> __device__ __forceinline__ Decay<n> decay(Vec<n> f) {
  Decay<n> r;
  const Vec<n> e = exp2v(mul(f, all<n>(kLog2e)));
  float pick[n], c[n];
  if constexpr (FORM == RET_SCAN_LOGIT) {
    r.q = rcpv(fma(e, all<n>(-1.0f), all<n>(-1.0f)));
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool near = f[i] > 0.0f;
      pick[i] = near ? 1.0f : -e[i];
      c[i] = near ? 1.0f : 0.0f;
    }
    r.m = mul(add(r.q, all<n>(-kLeast)), vec(pick));
    r.a = add(r.m, vec(c));
  } else {
    Vec<n> s = fma(f, all<n>(1.0f / 720.0f), all<n>(1.0f / 120.0f));
    s = fma(f, s, all<n>(1.0f / 24.0f));
    s = fma(f, s, all<n>(1.0f / 6.0f));
    s = fma(f, s, all<n>(0.5f));
    s = fma(f, s, all<n>(1.0f));
    s = fma(f, s, all<n>(-kLeast));
#pragma unroll  // (-1/4 < f <= -0 in one comparison of their bits)
    for (int i = 0; i < n; ++i)
      pick[i] = __float_as_int(f[i]) < __float_as_int(-0.25f) ? s[i] : e[i];
    r.m = vec(pick);
    r.a = add(r.m, near_one(r.m));
  }
  return r;
}
// q from m and c; 0 again where the decay is exactly 1.
template <int n> __device__ __forceinline__ Vec<n> less_one(Vec<n> m, Vec<n> c) {
  return add(fma(c, all<n>(kLeast), m), add(c, all<n>(-1.0f)));
}
// a z, and a z + more.
template <int n> __device__ __forceinline__ Vec<n> decayed(Vec<n> z, Vec<n> m, Vec<n> c) {
  return fma(m, z, mul(c, z));
}
template <int n>
__device__ __forceinline__ Vec<n> decayed(Vec<n> z, Vec<n> m, Vec<n> c, Vec<n> more) {
  return fma(m, z, fma(c, z, more));
}

// z from the state h and back.
template <int FORM> __device__ __forceinline__ float turn(float h) {
  return FORM == RET_SCAN_LOGIT ? -h : h;
}

// What a token with input x adds to z.
template <int FORM, int n> __device__ __forceinline__ Vec<n> drive(Vec<n> q, Vec<n> x) {
  if constexpr (FORM == RET_SCAN_LOGIT) return mul(q, x);
  return x;
}

constexpr int kThreads = 128;  // of the single-token kernel

// Where element (b, t, d) of an operand lies.
template <typename T>
__device__ __forceinline__ T* at(const Operand& o, long long b, long long t, long long d) {
  return static_cast<T*>(o.p) + b * o.batch + t * o.token + d;
}

// ---- sequence form ------------------------------------------------------------
//
// The recurrence composes: a span of tokens turns the z before it into
// Z + A z, where Z is its end from zero and A the product of its decays, held
// as one number M like a single decay, and for the same reasons.  (Z itself is
// taken with the decays rounded as a: over the 32 tokens of a warp that adds
// up to no more than their other roundings, and saves an operation each.)
// The sequence is cut into items of kTok tokens x one 128-byte piece of
// channels.  A block keeps a ring of items in shared memory (loads of the
// next ones run while one is computed), and per item
//   1. each of 8 warps scans its own kTok/8 tokens from zero, channels across
//      lanes (4 bytes of them each), and leaves (M, Z) in shared memory;
//   2. every warp folds the spans of the warps before it; the last one so has
//      the item's (M, Z) and publishes it;
//   3. every warp runs its tokens again from the z that enters them and
//      writes y; the last one publishes the item's end.
// What enters the item is found meanwhile by a ninth warp, the scout: it looks
// back over the previous items of the same channels until it meets one whose
// end is published, and folds forward from there over the published spans.
// So every element crosses HBM once, and neither few channels nor long
// sequences leave SMs idle: the single-pass prefix scan with decoupled
// look-back (Merrill and Garland, 2016).  (With the look-back done by one of the eight
// warps between 2 and 3, the others waited for it 60% of the time: 556 us
// instead of 401 us for 65536 x 4096 in bf16.)
//
// Block k of G takes items k, k + G, k + 2 G ... of the order in time, and the
// launch is cooperative: every block of it runs, or none, so an item's
// predecessors are always being worked on and waiting for them ends, whatever
// else the GPU runs.  The wait is bounded in time all the same.  (Items taken
// from a counter instead, three ahead for the ring, end up in clumps: a block
// that was held up takes its next ones in one burst, and its neighbours in
// time then wait for one another: 651 us where this order takes 401.)  A
// published word is
// its own flag (every word of the workspace starts as kEmpty, which no
// result of arithmetic is), so no fence or lock is needed, and folding from
// any published end gives the same bits: the end of an item is itself the fold
// of its (M, Z) over the one before.
constexpr int kWarps = 8;
constexpr int kCompute = 32 * kWarps;
constexpr int kPiece = 128;                // bytes of one row of an item
constexpr uint32_t kEmpty = 0xffffffffu;   // a NaN that arithmetic never returns
constexpr int kSiteForward = 801, kSiteBackward = 802;

struct Plan {
  float* end;      // [tile][B][blocks][channels]: what leaves an item
  float* span;     // same, two words per channel: a lane's M's, then its Z's
  int blocks;      // pieces of channels per batch row
  int pieces;      // of all batch rows
  int tiles;       // items per piece
  int items;
  int window;      // predecessors looked at together
  int skip_turns, skip_rest;  // from one of a block's items to its next: the grid
                              // in whole turns, and the rest of it
  int first;       // turn of the first block's first item (not 0 in the self-test)
  uint64_t limit;  // of every wait, ns
  // words from one turn to the next, and where a lane's begin (n channels per lane)
  __device__ __forceinline__ size_t pitch(int n) const { return (size_t)pieces * 32 * n; }
  template <typename Item>
  __device__ __forceinline__ size_t words(const Item& it, int n, int lane) const {
    return ((size_t)it.turn * pieces + it.rest) * 32 * n + lane * n;
  }
};

__device__ __forceinline__ float word(float x) {
  return __float_as_uint(x) == kEmpty ? __uint_as_float(0x7fffffffu) : x;
}
template <int n> __device__ __forceinline__ bool written(const Vec<n>& x) {
  bool r = true;
#pragma unroll
  for (int i = 0; i < n; ++i) r = r && __float_as_uint(x[i]) != kEmpty;
  return r;
}
// Words are read and written one by one as far as their meaning goes; the
// vector forms only save instructions.
__device__ __forceinline__ void ld_words(const float* p, Vec<1>& a) {
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(a.a) : "l"(p) : "memory");
}
__device__ __forceinline__ void ld_words(const float* p, Vec<2>& a) {
  float x, y;
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];"
               : "=f"(x), "=f"(y)
               : "l"(p)
               : "memory");
  a = two(x, y);
}
__device__ __forceinline__ void ld_words(const float* p, Vec<1>& a, Vec<1>& b) {
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];"
               : "=f"(a.a), "=f"(b.a)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void ld_words(const float* p, Vec<2>& a, Vec<2>& b) {
  float x, y, z, w;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x), "=f"(y), "=f"(z), "=f"(w)
               : "l"(p)
               : "memory");
  a = two(x, y), b = two(z, w);
}
__device__ __forceinline__ void st_words(float* p, Vec<1> a) {
  asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(word(a.a)) : "memory");
}
__device__ __forceinline__ void st_words(float* p, Vec<2> a) {
  asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(word(a[0])),
               "f"(word(a[1]))
               : "memory");
}
__device__ __forceinline__ void st_words(float* p, Vec<1> a, Vec<1> b) {
  asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(word(a.a)),
               "f"(word(b.a))
               : "memory");
}
__device__ __forceinline__ void st_words(float* p, Vec<2> a, Vec<2> b) {
  asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(word(a[0])),
               "f"(word(a[1])), "f"(word(b[0])), "f"(word(b[1]))
               : "memory");
}

// z after a span (M, Z) entered with z.
template <int n> __device__ __forceinline__ Vec<n> fold(Vec<n> z, Vec<n> M, Vec<n> Z) {
  return decayed(z, M, near_one(M), Z);
}

// No more than the largest float32 (a NaN stays one): a product of decays above
// 1 that no float32 holds leaves a zero state zero then, and ends at a decay of 0.
template <int FORM, int n> __device__ __forceinline__ Vec<n> bounded(Vec<n> p) {
  if constexpr (FORM == RET_SCAN_LOGIT) {
    return p;
  } else {
    float v[n];
#pragma unroll
    for (int i = 0; i < n; ++i)
      asm("min.NaN.f32 %0, %1, 0f7f7fffff;" : "=f"(v[i]) : "f"(p[i]));
    return vec(v);
  }
}

// A product of decays, P, and its difference from 1, Q: each is exact where
// the other is not, and the product is held by Q from P = 5/8 on (of LOGIT's
// decays none at or below 1/2 is in it then).
template <int FORM, int n> struct Product {
  Vec<n> P = all<n>(1.0f), Q = all<n>(0.0f);
  __device__ __forceinline__ void take(Vec<n> m) {  // one more span
    const Vec<n> c = near_one(m);
    Q = fma(less_one(m, c), P, Q);
    P = bounded<FORM>(mul(P, add(m, c)));
  }
  __device__ __forceinline__ Vec<n> held() const {
    float m[n];
#pragma unroll
    for (int i = 0; i < n; ++i) m[i] = P[i] > 0.625f && Q[i] < 0.0f ? Q[i] : P[i];
    return vec(m);
  }
};

// The product of a warp's tokens.  LOG: e to the sum of their f, in four parts.
template <int FORM, int n> struct Tokens : Product<FORM, n> {
  using Product<FORM, n>::P;
  using Product<FORM, n>::Q;
  Vec<n> part[4] = {all<n>(0.0f), all<n>(0.0f), all<n>(0.0f), all<n>(0.0f)};
  __device__ __forceinline__ void take(int j, Vec<n> f, const Decay<n>& a) {
    if constexpr (FORM == RET_SCAN_LOGIT)
      Q = fma(a.q, P, Q);
    else
      part[j % 4] = add(part[j % 4], f);
    P = bounded<FORM>(mul(P, a.a));  // (LOG: for the backward's flow alone)
  }
  __device__ __forceinline__ Vec<n> held() const {
    if constexpr (FORM == RET_SCAN_LOGIT) return Product<FORM, n>::held();
    const Vec<n> f = add(add(part[0], part[1]), add(part[2], part[3]));
    float below[n];  // a sum of 0 is held as a difference from 1, too
#pragma unroll
    for (int i = 0; i < n; ++i) below[i] = f[i] == 0.0f ? -0.0f : f[i];
    return bounded<FORM>(decay<FORM>(vec(below)).m);
  }
};

// What enters item `tile` (> 0) of a lane's channels: `at` points at their
// words of that item, `pitch` words from one tile to the next.
template <int kWindow, int n>
__device__ __forceinline__ Vec<n> look_back(const Plan& p, size_t at, size_t pitch, int tile,
                                            int site) {
  Vec<n> z = all<n>(0.0f);
  bool found = false;
  uint64_t t0 = 0;
  int tries = 0;
  while (true) {
    Vec<n> e[kWindow], M[kWindow], Z[kWindow];
#pragma unroll
    for (int i = 0; i < kWindow; ++i) {
      e[i] = all<n>(__uint_as_float(kEmpty));
      if (tile - 1 - i >= 0) {
        ld_words(p.end + at - (i + 1) * pitch, e[i]);
        if (i + 1 < kWindow) ld_words(p.span + 2 * (at - (i + 1) * pitch), M[i], Z[i]);
      }
    }
    // the nearest published end state, if every span after it is published
    if (!found) {
      bool whole = true;
#pragma unroll
      for (int i = 0; i < kWindow; ++i) {
        if (!found && whole && written(e[i])) {
          z = e[i];
          found = true;
#pragma unroll
          for (int k = i - 1; k >= 0; --k) z = fold(z, M[k], Z[k]);
        }
        if (i + 1 < kWindow && tile - 1 - i >= 0) whole = whole && written(M[i]) && written(Z[i]);
      }
    }
    if (__all_sync(0xffffffffu, found)) return z;
    if (++tries % 64 == 0) {
      const uint64_t now = sm100::globaltimer();
      if (t0 == 0) t0 = now;
      // out of time, or another wait was: the whole warp gives up together
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&g_device_error) != 0 ||
                                      now - t0 > p.limit)) {
        sm100::record_error(site);
        return all<n>(__uint_as_float(0x7fffffffu));
      }
    }
  }
}

// ---- moving an item into shared memory ------------------------------------------
// 16 bytes, of which the first n are read and the others become zeros.
__device__ __forceinline__ void cp_async(uint32_t dst, const char* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows that are not 16-byte aligned are copied as the 16-byte granules that
// cover them, nine for a piece, and read from where they begin in the first:
// a granule's bytes before the row are read along (they lie in the row's own
// 16 bytes of memory), those behind the piece or the row's end are not.
// Copied 4 bytes at a time, 8 x 2048 x 2046 in bf16 took 122 us gated and 222
// backward, and with a bf16's alignment (2047), through registers, 427 and
// 557; in granules 103 and 189, 117 and 186.
constexpr int kGranules = kPiece / 16 + 1;
template <int W> constexpr int kRow = W == 16 ? kPiece : 16 * kGranules;  // in shared memory

// TOK rows of kPiece bytes: rows past `rows` and bytes past `width` become zeros.
// The width is the piece's own (an int holds no row's bytes: D may pass 2^30).
template <int TOK>
__device__ __forceinline__ void copy_item(char* dst, const char* src, long long pitch, int rows,
                                          int width) {
  const uint32_t to = sm100::smem_u32(dst);
#pragma unroll
  for (int k = 0; k < (TOK * kGranules + kCompute - 1) / kCompute; ++k) {
    const int i = k * kCompute + threadIdx.x;
    if ((k + 1) * kCompute > TOK * kGranules && i >= TOK * kGranules) break;
    const int r = i / kGranules, g = i - r * kGranules;
    const uintptr_t start = reinterpret_cast<uintptr_t>(src) + r * pitch;
    const uintptr_t granule = (start & ~(uintptr_t)15) + 16 * g;
    const int n = r < rows ? max(0, min(16, (int)(start + width - granule))) : 0;
    cp_async(to + i * 16, reinterpret_cast<const char*>(n > 0 ? granule : start & ~(uintptr_t)15),
             n);
  }
}

// Barrier of the eight computing warps.
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kCompute) : "memory");
}

// The channels of one lane: 4 bytes of a row.
template <typename T> constexpr int kLane = 4 / sizeof(T);
// One operand's rows of a warp's tokens in shared memory: where the first one's
// granules begin, and the low bits of its address and pitch in memory.
struct Rows {
  char* p;
  uint32_t low, pitch;
};
template <typename T> __device__ __forceinline__ Vec<kLane<T>> get(const char* row) {
  float r[kLane<T>];
  load_pack<T, kLane<T>>(reinterpret_cast<const T*>(row) + (threadIdx.x % 32) * kLane<T>, r);
  return vec(r);
}
template <typename T, int n> __device__ __forceinline__ void set(char* row, const Vec<n>& x) {
  float v[n];
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = x[i];
  store_pack<T, n>(reinterpret_cast<T*>(row) + (threadIdx.x % 32) * n, v);
}
template <typename T, int W>
__device__ __forceinline__ Vec<kLane<T>> get(const Rows& rows, int j) {
  if constexpr (W == 16) {
    return get<T>(rows.p + j * kRow<W>);
  } else {
    const char* row = rows.p + j * kRow<W> + ((rows.low + j * rows.pitch) & 15);
    if constexpr (W >= 4) {
      return get<T>(row);
    } else {
      const T* q = reinterpret_cast<const T*>(row) + (threadIdx.x % 32) * kLane<T>;
      float r[kLane<T>];
#pragma unroll
      for (int i = 0; i < kLane<T>; ++i) r[i] = Elem<T>::ld(q + i);
      return vec(r);
    }
  }
}
// `left`: channels of the piece that exist from this lane's first one on.
template <typename T, bool PAIR, int n>
__device__ __forceinline__ void put(T* p, const Vec<n>& x, int left) {
  float v[n];
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = x[i];
  if (PAIR || n == 1) {
    if (left > 0) store_pack<T, n>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (i < left) Elem<T>::st(p + i, v[i]);
  }
}
template <int n> __device__ __forceinline__ Vec<n> get_state(const float* p, int left) {
  float r[n];
#pragma unroll
  for (int i = 0; i < n; ++i) r[i] = p && i < left ? p[i] : 0.0f;
  return vec(r);
}
template <int n> __device__ __forceinline__ void put_state(float* p, const Vec<n>& x, int left) {
#pragma unroll
  for (int i = 0; i < n; ++i)
    if (i < left) p[i] = x[i];
}
template <int FORM, int n> __device__ __forceinline__ Vec<n> turn(Vec<n> h) {
  float r[n];
#pragma unroll
  for (int i = 0; i < n; ++i) r[i] = turn<FORM>(h[i]);
  return vec(r);
}

// Shape of the work: one block per SM with long items.  That makes a warp's
// work large against its share of the folds, barriers and look-back: with two
// blocks of half as many tokens each 65536 x 4096 in bf16 takes 371 us instead
// of 293, and 8 x 2048 x 2048 gated 65 instead of 63.
constexpr int kTokForward = 256, kTokBackward = 128;
constexpr int kTokLeast = 64;  // of any item

// SUMS: span sums that the warps exchange beside the ring, 4 KB each.
template <int OPERANDS, int SUMS, int TOK, int W> struct Ring {
  static constexpr int kOperand = TOK * kRow<W>;
  static constexpr int kStage = OPERANDS * kOperand;
  static constexpr int kRoom = 227 * 1024 - 1024 * (4 * SUMS + 1);
  static constexpr int kFit = kRoom / kStage;
  static constexpr int kStages = kFit < 4 ? kFit : 4;
  static constexpr int kBytes = kStages * kStage;
  static_assert(kStages >= 2 && TOK >= kTokLeast && TOK % RET_SCAN_CHUNK == 0 &&
                    RET_SCAN_CHUNK % (TOK / kWarps) == 0,
                "chunk states are kept and read where a warp's tokens begin");
};

// The items of a block, one after another: dealt in the order in time, or,
// where the block keeps whole pieces, each piece from its first turn to its
// last.
template <bool WHOLE> struct Walk {
  int turn;  // place in the order that state flows: 0 has no predecessor
  int rest;  // batch row and piece of its channels in one
  __device__ __forceinline__ Walk(const Plan& p)
      : turn(WHOLE ? 0 : p.first + blockIdx.x / p.pieces),
        rest(WHOLE ? blockIdx.x : blockIdx.x % p.pieces) {}
  __device__ __forceinline__ void next(const Plan& p) {
    if constexpr (WHOLE) {
      if (++turn == p.tiles) turn = 0, rest += gridDim.x;
    } else {
      turn += p.skip_turns;
      rest += p.skip_rest;
      if (rest >= p.pieces) rest -= p.pieces, ++turn;
    }
  }
  __device__ __forceinline__ bool ends(const Plan& p) const {
    return WHOLE ? rest >= p.pieces : turn >= p.tiles;
  }
};

// What the scout hands to the computing warps: what enters the item of round
// k, in enter[k % 2]; and the ring's barriers where TMA fills and empties it.
template <int STAGES, int n> struct Desk {
  Vec<n> enter[2][32];
  uint64_t full[2], free[2];
  uint64_t loaded[STAGES], done[STAGES];
};

// By the whole block, before anything else.
template <int STAGES, int n> __device__ __forceinline__ void open_desk(Desk<STAGES, n>& desk) {
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&desk.full[i], 1);
      sm100::mbar_init(&desk.free[i], kWarps);
    }
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      sm100::mbar_init(&desk.loaded[i], 1);
      sm100::mbar_init(&desk.done[i], kWarps);
    }
    sm100::fence_mbar_init();
  }
  __syncthreads();
}

// The scout's rounds.  first(rest): what enters a turn 0 item.
template <bool WHOLE, int STAGES, int n, typename First>
__device__ __forceinline__ void scout(Desk<STAGES, n>& desk, const Plan& p, int site,
                                      First first) {
  const int lane = threadIdx.x % 32;
  Walk<WHOLE> w(p);
  if constexpr (WHOLE) {  // the last computing warp hands each end on by itself
    if (!w.ends(p)) desk.enter[0][lane] = first(w.rest);
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&desk.full[0]);
  } else {
    for (int k = 0; !w.ends(p); ++k, w.next(p)) {
      Vec<n> z;
      if (w.turn == 0) {
        z = first(w.rest);
      } else {
        const size_t words = p.words(w, n, lane);
        z = p.window <= 2   ? look_back<2, n>(p, words, p.pitch(n), w.turn, site)
            : p.window <= 4 ? look_back<4, n>(p, words, p.pitch(n), w.turn, site)
                            : look_back<8, n>(p, words, p.pitch(n), w.turn, site);
      }
      // the slot's previous contents (round k - 2) have been read
      if (k >= 2) sm100::mbar_wait(&desk.free[k % 2], (k / 2 - 1) % 2, site + 2, p.limit);
      desk.enter[k % 2][lane] = z;
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&desk.full[k % 2]);
    }
  }
}

// By the computing warps: what enters the item of round k.  Where the block
// keeps whole pieces it was put there in round k - 1, on the far side of this
// round's barrier (only round 0 has it from the scout).
template <bool WHOLE, int STAGES, int n>
__device__ __forceinline__ Vec<n> entering(Desk<STAGES, n>& desk, const Plan& p, int k,
                                           int site) {
  const int lane = threadIdx.x % 32;
  if constexpr (WHOLE) {
    if (k == 0) sm100::mbar_wait(&desk.full[0], 0, site + 4, p.limit);
    return desk.enter[k % 2][lane];
  } else {
    sm100::mbar_wait(&desk.full[k % 2], (k / 2) % 2, site + 4, p.limit);
    const Vec<n> z = desk.enter[k % 2][lane];
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&desk.free[k % 2]);
    return z;
  }
}

// An operand as TMA sees it: [D] x the pitch that is smaller x the larger one.
struct Mapped {
  CUtensorMap map;
  int time_major;  // the batch pitch is the smaller one
};
__device__ __forceinline__ void tma_load(void* dst, const Mapped& m, uint64_t* bar, int d, int t,
                                         int b) {
  sm100::tma_load_3d(dst, &m.map, bar, d, m.time_major ? b : t, m.time_major ? t : b);
}
__device__ __forceinline__ void tma_store(const Mapped& m, const void* src, int d, int t, int b) {
  sm100::tma_store_3d(&m.map, sm100::smem_u32(src), d, m.time_major ? b : t,
                      m.time_major ? t : b);
}

// One thread's rounds where TMA moves the items: operands 0 .. IN-1 of an item
// are loaded to its slot, and once the computing warps have put results in
// place of some of them, those are stored and the slot is filled again.  Rows
// and channels past the end read as zeros and are not written.  tile(turn):
// place in time.  out[i]: the operand whose place result i has taken.
template <bool WHOLE, typename R, int IN, int OUT, int TOK, int STAGES, int n, typename Tile>
__device__ __forceinline__ void mover(Desk<STAGES, n>& desk, char* ring, const Plan& p,
                                      const Mapped* in, const Mapped* out, const int (&place)[OUT],
                                      int site, Tile tile) {
  constexpr int C = 32 * n;
  Walk<WHOLE> ahead(p), w(p);
  int loads[STAGES];
#pragma unroll
  for (int s = 0; s < STAGES; ++s) loads[s] = 0;
  const auto load = [&](int slot) {
    const int b = ahead.rest / p.blocks, d = (ahead.rest - b * p.blocks) * C;
    const int t = tile(ahead.turn) * TOK;
    sm100::mbar_arrive_expect_tx(&desk.loaded[slot], R::kStage);
#pragma unroll
    for (int i = 0; i < IN; ++i)
      tma_load(ring + slot * R::kStage + i * R::kOperand, in[i], &desk.loaded[slot], d, t, b);
    ahead.next(p);
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s)
    if (!ahead.ends(p)) load(s), ++loads[s];
  bool ok = true;
  for (int k = 0; ok && !w.ends(p);) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s, ++k) {
      if (!ok || w.ends(p)) break;
      // The computing warps say done after a wait that gave up as well: the slot is
      // touched again only once its own load has landed.
      ok = sm100::mbar_wait(&desk.done[s], (k / STAGES) % 2, site + 6, p.limit) &&
           sm100::mbar_wait(&desk.loaded[s], (k / STAGES) % 2, site + 6, p.limit);
      if (!ok) break;
      const int b = w.rest / p.blocks, d = (w.rest - b * p.blocks) * C;
      const int t = tile(w.turn) * TOK;
#pragma unroll
      for (int i = 0; i < OUT; ++i)
        tma_store(out[i], ring + s * R::kStage + place[i] * R::kOperand, d, t, b);
      sm100::bulk_commit();
      w.next(p);
      if (!ahead.ends(p)) {
        sm100::bulk_wait_read0();
        load(s), ++loads[s];
      }
    }
  }
  sm100::bulk_wait0();
  if (!ok) {  // some wait gave up: the loads under way still end before the block does
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
      if (loads[s] > 0) sm100::mbar_drain(&desk.loaded[s], (loads[s] - 1) % 2);
  }
}

// Threads of a block: the computing warps, the scout, and the mover.
template <int W> constexpr int kBlockOf = kCompute + 32 + (W == 16 ? 32 : 0);

template <int OPERANDS, int W> struct Maps {
  Mapped m[OPERANDS];
};
template <int OPERANDS> struct Maps<OPERANDS, 4> {};
template <int OPERANDS> struct Maps<OPERANDS, 2> {};

// The f of a token that is not there: a decay of 1 and, its x being zero, no
// input (LOG: its f is a zero as well).
template <int FORM, int n> __device__ __forceinline__ void mask(Vec<n>& f, bool there) {
  if (FORM == RET_SCAN_LOGIT && !there) f = all<n>(__uint_as_float(0x7f800000u));
}

// W: bytes that every row of every operand is aligned to (16, 4 or 2).  With
// 16, TMA moves the items: the loads cost the computing warps nothing, and y
// leaves from the place of f without an address or a bound being computed.
// Otherwise the computing warps copy, and store y themselves.
template <typename T, int FORM, bool GATE, int W, bool WHOLE>
__global__ void __launch_bounds__(kBlockOf<W>, 1)
scan_items(const ScanArgs a, const Plan p, const __grid_constant__ Maps<GATE ? 4 : 3, W> maps) {
  constexpr int IN = GATE ? 3 : 2;  // f, x, gate
  using R = Ring<IN, 2, kTokForward, W>;
  constexpr int n = kLane<T>, kTok = kTokForward, S = kTok / kWarps, C = 32 * n;
  constexpr int ST = R::kStages, kX = R::kOperand, kGate = 2 * R::kOperand;
  constexpr bool kTma = W == 16;
  using V = Vec<n>;
  extern __shared__ __align__(128) char ring[];
  __shared__ Desk<ST, n> desk;
  __shared__ V agg_m[2][kWarps][32], agg_z[2][kWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  const auto first = [&](int rest) {  // z before a sequence
    const int b = rest / p.blocks, d = (rest - b * p.blocks) * C + lane * n;
    return turn<FORM>(
        get_state<n>(a.state_in && rest < p.pieces ? a.state_in + (size_t)b * a.D + d : nullptr,
                     a.D - d));
  };
  open_desk(desk);
  if (warp == kWarps) {
    scout<WHOLE>(desk, p, kSiteForward, first);
    return;
  }
  if constexpr (kTma) {
    if (warp > kWarps) {
      if (lane == 0)
        mover<WHOLE, R, IN, 1, kTok>(desk, ring, p, maps.m, maps.m + IN, {0}, kSiteForward,
                           [](int turn) { return turn; });
      return;
    }
  }

  Walk<WHOLE> ahead(p), w(p);
  const auto load = [&](int slot) {
    if (!ahead.ends(p)) {
      const int b = ahead.rest / p.blocks, d = (ahead.rest - b * p.blocks) * C;
      const int t = ahead.turn * kTok, rows = a.N - t, width = min(a.D - d, C) * (int)sizeof(T);
      char* s = ring + slot * R::kStage;
      copy_item<kTok>(s, (const char*)at<const T>(a.f, b, t, d), a.f.token * sizeof(T), rows,
                         width);
      copy_item<kTok>(s + kX, (const char*)at<const T>(a.x, b, t, d), a.x.token * sizeof(T),
                         rows, width);
      if constexpr (GATE)
        copy_item<kTok>(s + kGate, (const char*)at<const T>(a.gate, b, t, d),
                           a.gate.token * sizeof(T), rows, width);
      ahead.next(p);
    }
    cp_commit();
  };
  if constexpr (!kTma)
    for (int s = 0; s + 1 < ST; ++s) load(s);

  for (int k = 0, slot = 0, phase = 0; !w.ends(p); ++k, w.next(p)) {
    const int b = w.rest / p.blocks, d = (w.rest - b * p.blocks) * C + lane * n, left = a.D - d;
    const int t0 = w.turn * kTok + warp * S, mine = min(S, a.N - t0);
    if constexpr (kTma) {
      sm100::mbar_wait(&desk.loaded[slot], phase, kSiteForward + 8, p.limit);
    } else {
      cp_wait<ST - 2>();
      compute_sync();  // the item is here, and the previous one's slot is free
      load(slot == 0 ? ST - 1 : slot - 1);
    }
    const auto rows = [&](const Operand& o, int place) {
      Rows r = {ring + slot * R::kStage + place + warp * S * kRow<W>, 0, 0};
      if constexpr (!kTma) {
        r.low = (uint32_t) reinterpret_cast<uintptr_t>(at<const T>(o, b, t0, d - lane * n));
        r.pitch = (uint32_t)o.token * sizeof(T);
      }
      return r;
    };
    const Rows f = rows(a.f, 0), x = rows(a.x, kX);

    // 1. this warp's tokens from zero; u, what a token adds, stays in registers
    // where those suffice (8 x 2048 x 2047 gated: 144 us with it, 119 without)
    constexpr bool kKeep = W == 16 || !GATE;
    V m[S], u[kKeep ? S : 1], Z = all<n>(0.0f);
    Tokens<FORM, n> product;
    const auto from_zero = [&](auto whole) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        V ft = get<T, W>(f, j);
        if (!decltype(whole)::value) mask<FORM>(ft, j < mine);
        const Decay<n> token = decay<FORM>(ft);
        m[j] = token.m;
        const V more = drive<FORM>(token.q, get<T, W>(x, j));
        if constexpr (kKeep) u[j] = more;
        Z = fma(token.a, Z, more);
        product.take(j, ft, token);
      }
    };
    if (mine == S)
      from_zero(Int<1>());
    else
      from_zero(Int<0>());
    V M = product.held();
    agg_m[k % 2][warp][lane] = M;
    agg_z[k % 2][warp][lane] = Z;
    compute_sync();

    // 2. the span of the warps before, and of the item
    Product<FORM, n> behind;
    V Zb = all<n>(0.0f);
#pragma unroll
    for (int v = 0; v < kWarps - 1; ++v) {
      if (v >= warp) break;
      Zb = fold(Zb, agg_m[k % 2][v][lane], agg_z[k % 2][v][lane]);
      behind.take(agg_m[k % 2][v][lane]);
    }
    const V Mb = behind.held();
    const bool publish = warp == kWarps - 1 && w.turn + 1 < p.tiles;
    if (warp == kWarps - 1) {
      Z = fold(Zb, M, Z);
      behind.take(M);
      M = behind.held();
      if (publish && !WHOLE) st_words(p.span + 2 * p.words(w, n, lane), M, Z);
    }
    V z = entering<WHOLE>(desk, p, k, kSiteForward);
    if (warp == kWarps - 1) {
      if constexpr (WHOLE)
        desk.enter[(k + 1) % 2][lane] = publish ? fold(z, M, Z) : first(w.rest + gridDim.x);
      else if (publish)
        st_words(p.end + p.words(w, n, lane), fold(z, M, Z));
    }
    z = fold(z, Mb, Zb);

    // 3. the same tokens from the z that enters them
    if (a.chunk_states && t0 % RET_SCAN_CHUNK == 0 && mine > 0)
      put_state(a.chunk_states +
                    ((size_t)b * cdiv(a.N, RET_SCAN_CHUNK) + t0 / RET_SCAN_CHUNK) * a.D + d,
                turn<FORM>(z), left);
    T* y = kTma ? nullptr : at<T>(a.y, b, t0, d);
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const V c = near_one(m[j]);
      if constexpr (kKeep)
        z = decayed(z, m[j], c, u[j]);
      else
        z = decayed(z, m[j], c, drive<FORM>(less_one(m[j], c), get<T, W>(x, j)));
      V out = turn<FORM>(z);
      if constexpr (GATE) out = mul(out, swish(get<T, W>(rows(a.gate, kGate), j)));
      if constexpr (kTma) {
        set<T>(f.p + j * kRow<W>, out);
      } else {
        if (j < mine) put<T, (W >= 4)>(y, out, left);
        y += a.y.token;
      }
    }
    if (a.state_out && mine > 0 && t0 + mine == a.N)
      put_state(a.state_out + (size_t)b * a.D + d, turn<FORM>(z), left);
    if constexpr (kTma) {
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&desk.done[slot]);
    }
    if (++slot == ST) slot = 0, phase ^= 1;
  }
  if constexpr (!kTma) cp_wait<0>();
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
// E + A e with the same A.  So the items are taken from the end of the
// sequence: the state that enters a chunk comes from the
// forward call, h is recomputed in float32 inside it, and the flow is looked
// for in the items after it as the forward does in those before.
template <typename T, int FORM, bool GATE, int W, bool WHOLE>
__global__ void __launch_bounds__(kBlockOf<W>, 1)
scan_items_backward(const ScanArgs a, const Plan p,
                    const __grid_constant__ Maps<GATE ? 7 : 5, W> maps) {
  constexpr int IN = GATE ? 4 : 3;  // f, x, d_y, gate; grad_f, grad_x and grad_gate in their place
  using R = Ring<IN, 3, kTokBackward, W>;
  constexpr int n = kLane<T>, kTok = kTokBackward, S = kTok / kWarps, C = 32 * n;
  constexpr int ST = R::kStages, kX = R::kOperand, kDy = 2 * R::kOperand, kGate = 3 * R::kOperand;
  constexpr bool kTma = W == 16;
  using V = Vec<n>;
  extern __shared__ __align__(128) char ring[];
  __shared__ Desk<ST, n> desk;
  __shared__ V agg_m[2][kWarps][32], agg_z[2][kWarps][32], agg_e[2][kWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  const auto first = [&](int rest) {  // the flow behind a sequence
    const int b = rest / p.blocks, d = (rest - b * p.blocks) * C + lane * n;
    return get_state<n>(
        a.d_state_out && rest < p.pieces ? a.d_state_out + (size_t)b * a.D + d : nullptr, a.D - d);
  };
  open_desk(desk);
  if (warp == kWarps) {
    scout<WHOLE>(desk, p, kSiteBackward, first);
    return;
  }
  if constexpr (kTma) {
    if (warp > kWarps) {
      const auto tile = [&](int turn) { return p.tiles - 1 - turn; };
      if (lane == 0) {
        if constexpr (GATE)
          mover<WHOLE, R, IN, 3, kTok>(desk, ring, p, maps.m, maps.m + IN, {0, 1, 3},
                                       kSiteBackward, tile);
        else
          mover<WHOLE, R, IN, 2, kTok>(desk, ring, p, maps.m, maps.m + IN, {0, 1},
                                       kSiteBackward, tile);
      }
      return;
    }
  }

  Walk<WHOLE> ahead(p), w(p);
  const auto load = [&](int slot) {
    if (!ahead.ends(p)) {
      const int b = ahead.rest / p.blocks, d = (ahead.rest - b * p.blocks) * C;
      const int t = (p.tiles - 1 - ahead.turn) * kTok;
      const int rows = a.N - t, width = min(a.D - d, C) * (int)sizeof(T);
      char* s = ring + slot * R::kStage;
      copy_item<kTok>(s, (const char*)at<const T>(a.f, b, t, d), a.f.token * sizeof(T), rows,
                         width);
      copy_item<kTok>(s + kX, (const char*)at<const T>(a.x, b, t, d), a.x.token * sizeof(T),
                         rows, width);
      copy_item<kTok>(s + kDy, (const char*)at<const T>(a.d_y, b, t, d),
                         a.d_y.token * sizeof(T), rows, width);
      if constexpr (GATE)
        copy_item<kTok>(s + kGate, (const char*)at<const T>(a.gate, b, t, d),
                           a.gate.token * sizeof(T), rows, width);
      ahead.next(p);
    }
    cp_commit();
  };
  if constexpr (!kTma)
    for (int s = 0; s + 1 < ST; ++s) load(s);

  for (int k = 0, slot = 0, phase = 0; !w.ends(p); ++k, w.next(p)) {
    const int b = w.rest / p.blocks, d = (w.rest - b * p.blocks) * C + lane * n, left = a.D - d;
    const int tile = p.tiles - 1 - w.turn, t0 = tile * kTok + warp * S, mine = min(S, a.N - t0);
    // what enters the chunk of this warp's tokens: read here, needed after 1
    const int chunk = t0 / RET_SCAN_CHUNK, head = warp - t0 % RET_SCAN_CHUNK / S;
    V z = get_state<n>(
        mine > 0 ? a.chunk_states + ((size_t)b * cdiv(a.N, RET_SCAN_CHUNK) + chunk) * a.D + d
                 : nullptr,
        left);
    if constexpr (kTma) {
      sm100::mbar_wait(&desk.loaded[slot], phase, kSiteBackward + 8, p.limit);
    } else {
      cp_wait<ST - 2>();
      compute_sync();
      load(slot == 0 ? ST - 1 : slot - 1);
    }
    const auto rows = [&](const Operand& o, int place) {
      Rows r = {ring + slot * R::kStage + place + warp * S * kRow<W>, 0, 0};
      if constexpr (!kTma) {
        r.low = (uint32_t) reinterpret_cast<uintptr_t>(at<const T>(o, b, t0, d - lane * n));
        r.pitch = (uint32_t)o.token * sizeof(T);
      }
      return r;
    };
    const Rows f = rows(a.f, 0), x = rows(a.x, kX), dy = rows(a.d_y, kDy);
    Rows g = {};
    if constexpr (GATE) g = rows(a.gate, kGate);

    // 1. this warp's tokens: forwards from a zero state, and what flows out of
    // them backwards from a zero flow, the sum of a_0 ... a_j dh_j
    constexpr bool kKeep = kTma;  // (8 x 2048 x 2047 gated: 194 us with it, 184 without)
    V m[S], before[S], dh[S], slope[GATE ? S : 1], Z = all<n>(0.0f), E = Z;
    Tokens<FORM, n> product;
    const auto from_zero = [&](auto whole) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        V ft = get<T, W>(f, j);
        if (!decltype(whole)::value) mask<FORM>(ft, j < mine);
        const Decay<n> token = decay<FORM>(ft);
        m[j] = token.m;
        const V more = drive<FORM>(token.q, get<T, W>(x, j));
        if constexpr (kKeep) before[j] = more;  // for now: what a token adds
        Z = fma(token.a, Z, more);
        product.take(j, ft, token);
        dh[j] = get<T, W>(dy, j);
        if constexpr (GATE) {
          V sw, sl;
          swish_grad(get<T, W>(g, j), &sw, &sl);
          slope[j] = turn<FORM>(mul(dh[j], sl));  // with the sign of z
          dh[j] = mul(dh[j], sw);
        }
        E = fma(product.P, dh[j], E);
      }
    };
    if (mine == S)
      from_zero(Int<1>());
    else
      from_zero(Int<0>());
    V M = product.held();
    agg_m[k % 2][warp][lane] = M;
    agg_z[k % 2][warp][lane] = Z;
    agg_e[k % 2][warp][lane] = E;
    compute_sync();

    // 2. the span of the warps behind, and of the item
    Product<FORM, n> behind;
    V Eb = all<n>(0.0f);
#pragma unroll
    for (int v = kWarps - 1; v > 0; --v) {
      if (v <= warp) break;
      Eb = fold(Eb, agg_m[k % 2][v][lane], agg_e[k % 2][v][lane]);
      behind.take(agg_m[k % 2][v][lane]);
    }
    const V Mb = behind.held();
    const bool publish = warp == 0 && w.turn + 1 < p.tiles;
    if (warp == 0) {
      E = fold(Eb, M, E);
      behind.take(M);
      M = behind.held();
      if (publish && !WHOLE) st_words(p.span + 2 * p.words(w, n, lane), M, E);
    }
    // z forwards from the state that enters the chunk
    z = turn<FORM>(z);
    for (int v = head; v < warp; ++v) z = fold(z, agg_m[k % 2][v][lane], agg_z[k % 2][v][lane]);
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const V c = near_one(m[j]);
      V more = before[j];
      if constexpr (!kKeep) more = drive<FORM>(less_one(m[j], c), get<T, W>(x, j));
      before[j] = z;
      z = decayed(z, m[j], c, more);
      if constexpr (GATE) {
        if constexpr (kTma)
          set<T>(g.p + j * kRow<W>, mul(z, slope[j]));
        else if (j < mine)
          put<T, (W >= 4)>(at<T>(a.grad_gate, b, t0 + j, d), mul(z, slope[j]), left);
      }
    }

    // 3. the gradients, backwards
    V flow = entering<WHOLE>(desk, p, k, kSiteBackward);
    if (warp == 0) {
      if constexpr (WHOLE)
        desk.enter[(k + 1) % 2][lane] = publish ? fold(flow, M, E) : first(w.rest + gridDim.x);
      else if (publish)
        st_words(p.end + p.words(w, n, lane), fold(flow, M, E));
    }
    flow = fold(flow, Mb, Eb);
#pragma unroll
    for (int j = S - 1; j >= 0; --j) {
      const V G = add(dh[j], flow);
      const V c = near_one(m[j]);
      flow = decayed(G, m[j], c);
      V dx = G, df = mul(before[j], flow);
      if (FORM == RET_SCAN_LOGIT) {
        const V q = less_one(m[j], c);
        dx = turn<FORM>(mul(q, G));
        df = mul(mul(add(before[j], get<T, W>(x, j)), q), flow);
      }
      if constexpr (kTma) {
        set<T>(x.p + j * kRow<W>, dx);
        set<T>(f.p + j * kRow<W>, df);
      } else if (j < mine) {
        put<T, (W >= 4)>(at<T>(a.grad_x, b, t0 + j, d), dx, left);
        put<T, (W >= 4)>(at<T>(a.grad_f, b, t0 + j, d), df, left);
      }
    }
    if (a.d_state_in && tile == 0 && warp == 0)
      put_state(a.d_state_in + (size_t)b * a.D + d, flow, left);
    if constexpr (kTma) {
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&desk.done[slot]);
    }
    if (++slot == ST) slot = 0, phase ^= 1;
  }
  if constexpr (!kTma) cp_wait<0>();
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
  float z[V], f[V], x[V], g[V];
  load_pack<float, V>(a.state_in + b * a.D + d, z);
  load_pack<T, V>(at<T>(a.f, b, 0, d), f);
  load_pack<T, V>(at<T>(a.x, b, 0, d), x);
  if constexpr (GATE) load_pack<T, V>(at<T>(a.gate, b, 0, d), g);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Decay<1> token = decay<FORM>(Vec<1>{f[v]});
    z[v] = turn<FORM>(decayed(Vec<1>{turn<FORM>(z[v])}, token.m, near_one(token.m),
                              drive<FORM>(token.q, Vec<1>{x[v]})).a);
  }
  store_pack<float, V>(a.state_out + b * a.D + d, z);
  if constexpr (GATE) {
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] *= swish(Vec<1>{g[v]}).a;
  }
  store_pack<T, V>(at<T>(a.y, b, 0, d), z);
}

// Calls fn with the element type, the form and whether there is a gate as
// compile-time values.
template <typename Fn>
cudaError_t dispatch(int dtype, int form, bool gate, Fn fn) {
  auto with_form = [&](auto t) {
    if (form == RET_SCAN_LOGIT)
      return gate ? fn(t, Int<RET_SCAN_LOGIT>(), Int<1>()) : fn(t, Int<RET_SCAN_LOGIT>(), Int<0>());
    return gate ? fn(t, Int<RET_SCAN_LOG>(), Int<1>()) : fn(t, Int<RET_SCAN_LOG>(), Int<0>());
  };
  return dtype == RET_BF16 ? with_form(Type<__nv_bfloat16>()) : with_form(Type<float>());
}

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
  p.pieces = a.B * p.blocks;
  p.items = p.pieces * p.tiles;
  p.limit = sm100::kWaitLimitNs;
  if (p.tiles > 1) {
    const size_t n = words(a.B, a.D, a.dtype, p.tiles);
    p.span = static_cast<float*>(a.workspace);
    p.end = p.span + 2 * n;
  }
  return p;
}

// Whether TMA can move an operand: 16-byte aligned rows, and pitches that its
// maps can hold.
bool mappable(const Operand& o, const ScanArgs& a, int es) {
  const uint64_t row = (uint64_t)a.D * es, token = a.N > 1 ? (uint64_t)o.token * es : row;
  const uint64_t batch = a.B > 1 ? (uint64_t)o.batch * es : token;
  const uint64_t small = token < batch ? token : batch, large = token < batch ? batch : token;
  return aligned_to(o.p, 16) && (row | token | batch) % 16 == 0 && large < ((uint64_t)1 << 40) &&
         large % small == 0;
}

// What every row of every operand is aligned to, up to TMA's needs.
int alignment(const ScanArgs& a) {
  const int es = a.dtype == RET_BF16 ? 2 : 4;
  uint64_t bits = (uint64_t)a.D * es;
  bool all = true;
  for (const Operand* o :
       {&a.x, &a.f, &a.gate, &a.y, &a.d_y, &a.grad_x, &a.grad_f, &a.grad_gate}) {
    if (!o->p) continue;
    bits |= reinterpret_cast<uint64_t>(o->p);
    if (a.B > 1) bits |= (uint64_t)o->batch * es;
    if (a.N > 1) bits |= (uint64_t)o->token * es;
    all = all && mappable(*o, a, es);
  }
  return all ? 16 : bits % 4 == 0 ? 4 : 2;
}

cudaError_t map_operand(Mapped* m, const Operand& o, const ScanArgs& a, int tok) {
  const int es = a.dtype == RET_BF16 ? 2 : 4;
  const uint64_t row = (uint64_t)a.D * es, token = a.N > 1 ? (uint64_t)o.token * es : row;
  const uint64_t batch = a.B > 1 ? (uint64_t)o.batch * es : token;
  m->time_major = batch < token;
  const uint32_t box = kPiece / es;
  return m->time_major
             ? make_tmap_rows(&m->map, o.p, es, a.D, a.B, a.N, batch, token, box, 1, tok)
             : make_tmap_rows(&m->map, o.p, es, a.D, a.N, a.B, token, batch, box, tok, 1);
}

// Whether blocks keep whole pieces, of `most` that run at once: then neither
// the workspace nor a cooperative launch is needed, but a block's rounds follow
// one another, and are as many as the fullest block's.  Dealing the items
// instead costs as much as two to four rounds (of the backward's shorter ones,
// four to seven): in bf16, pieces x tokens, 148 x 4096 gated, 16 rounds either
// way, 61 us in whole pieces and 66 dealt; 128 x 8192, 32 rounds or 27.7, 79 us
// both ways; 160 x 2048, 16 or 8.6, 43 and 33.  And it costs a call 2 us on the
// host, as much as a few rounds: 32 x 1024 in float32, 4 rounds or 0.9, 17 and
// 20 us a call, 64 x 2048, 8 or 3.5, 18 and 20; in bf16, whose rounds are
// longer, 32 x 2048, 8 or 1.7, 23 and 20.
constexpr int kFewRounds = 10;
bool keeps_whole(const Plan& p, int most) {
  const int64_t rounds = (int64_t)p.tiles * ((p.pieces + most - 1) / most);
  return rounds <= kFewRounds || rounds - 3 <= p.items / most;
}

// Sizes whose calls keep whole pieces on any device: they need no workspace.
bool always_whole(int pieces, int N) {
  return cdiv(N, kTokLeast) <= kFewRounds && pieces <= 128;
}

// What a kernel needs from the runtime, asked once per device: the permission
// for its shared memory, and how many of its blocks run at once.
constexpr int kMaxDevices = 64;
using Known = std::atomic<int>[kMaxDevices];  // blocks, 0 until asked

template <typename Kernel>
cudaError_t resident(Kernel dealt, Kernel whole, int threads, int smem, Known& known,
                     int* blocks) {
  int dev = 0, per_sm = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && (*blocks = known[dev].load()) > 0) return cudaSuccess;
  for (Kernel k : {dealt, whole})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, dealt, threads, smem);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *blocks = per_sm * sms;
  if (e != cudaSuccess) return e;
  if (*blocks < 1) return cudaErrorInvalidConfiguration;
  if (dev < kMaxDevices) known[dev].store(*blocks);
  return cudaSuccess;
}

// tok: tokens of an item; ops: the kernel's operands in the order of its maps.
template <int W, int OPERANDS>
cudaError_t run(void (*dealt)(ScanArgs, Plan, Maps<OPERANDS, W>),
                void (*whole)(ScanArgs, Plan, Maps<OPERANDS, W>), const ScanArgs& a, int tok,
                int smem, const Operand* const (&ops)[OPERANDS], Known& known, cudaStream_t st) {
  int most = 0;
  cudaError_t e = resident(dealt, whole, kBlockOf<W>, smem, known, &most);
  if (e != cudaSuccess) return e;
  Plan p = plan(a, tok);
  const bool keep = always_whole(p.pieces, a.N) || keeps_whole(p, most);
  const auto kernel = keep ? whole : dealt;
  const int units = keep ? p.pieces : p.items, grid = units < most ? units : most;
  p.skip_turns = grid / p.pieces, p.skip_rest = grid % p.pieces;
  // More words polled delay the ones that matter, fewer make more hops of a
  // chain: by how many predecessors are at work at once.  65536 x 4096 in bf16,
  // 2.3 of them: 280 us looking at two, 298 at four; 65536 x 1024, 9.2: 155 at
  // two, 107 at four, 112 at eight; 65536 x 64, 148: 81 at four, 58 at eight.
  p.window = p.skip_turns <= 2 ? 2 : p.skip_turns <= 16 ? 4 : 8;
  Maps<OPERANDS, W> maps;
  if constexpr (W == 16)
    for (int i = 0; i < OPERANDS; ++i)
      if ((e = map_operand(&maps.m[i], *ops[i], a, tok)) != cudaSuccess) return e;
  if (keep) {  // nothing to wait for
    kernel<<<grid, kBlockOf<W>, smem, st>>>(a, p, maps);
    return cudaPeekAtLastError();
  }
  e = cudaMemsetAsync(a.workspace, 0xff, 12 * words(a.B, a.D, a.dtype, p.tiles), st);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3(kBlockOf<W>);
  cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, p, maps);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <typename T, int F, bool G, int W>
cudaError_t forward(const ScanArgs& a, cudaStream_t st) {
  static Known known;
  constexpr int smem = Ring<G ? 3 : 2, 2, kTokForward, W>::kBytes;
  if constexpr (G) {
    const Operand* const ops[] = {&a.f, &a.x, &a.gate, &a.y};
    return run<W>(scan_items<T, F, G, W, false>, scan_items<T, F, G, W, true>, a, kTokForward,
                  smem, ops, known, st);
  } else {
    const Operand* const ops[] = {&a.f, &a.x, &a.y};
    return run<W>(scan_items<T, F, G, W, false>, scan_items<T, F, G, W, true>, a, kTokForward,
                  smem, ops, known, st);
  }
}

template <typename T, int F, bool G, int W>
cudaError_t backward(const ScanArgs& a, cudaStream_t st) {
  static Known known;
  constexpr int smem = Ring<G ? 4 : 3, 3, kTokBackward, W>::kBytes;
  if constexpr (G) {
    const Operand* const ops[] = {&a.f,      &a.x,      &a.d_y,      &a.gate,
                                  &a.grad_f, &a.grad_x, &a.grad_gate};
    return run<W>(scan_items_backward<T, F, G, W, false>, scan_items_backward<T, F, G, W, true>, a,
                  kTokBackward, smem, ops, known, st);
  } else {
    const Operand* const ops[] = {&a.f, &a.x, &a.d_y, &a.grad_f, &a.grad_x};
    return run<W>(scan_items_backward<T, F, G, W, false>, scan_items_backward<T, F, G, W, true>, a,
                  kTokBackward, smem, ops, known, st);
  }
}

// The second of two items whose predecessor no block works on.
cudaError_t lone_item(void* ws, uint64_t limit, cudaStream_t st) {
  constexpr int D = 32, N = 2 * kTokForward;
  char* rows = static_cast<char*>(ws) + kSelftestRows;
  ScanArgs a = {};
  Operand* const ops[] = {&a.f, &a.x, &a.y};
  for (int i = 0; i < 3; ++i) *ops[i] = {rows + i * sizeof(float) * N * D, N * D, D};
  a.B = 1, a.N = N, a.D = D, a.form = RET_SCAN_LOG, a.dtype = RET_F32, a.workspace = ws;
  const auto kernel = scan_items<float, RET_SCAN_LOG, false, 16, false>;
  constexpr int smem = Ring<2, 2, kTokForward, 16>::kBytes;
  Plan p = plan(a, kTokForward);
  p.skip_turns = 1, p.window = 2, p.first = 1, p.limit = limit;
  Maps<3, 16> maps;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  for (int i = 0; i < 3 && e == cudaSuccess; ++i)
    e = map_operand(&maps.m[i], *ops[i], a, kTokForward);
  if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0xff, kSelftestRows, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(rows, 0, kSelftestBytes - kSelftestRows, st);
  if (e != cudaSuccess) return e;
  kernel<<<1, kBlockOf<16>, smem, st>>>(a, p, maps);
  return cudaPeekAtLastError();
}

}  // namespace scan

int scan_device_error() { return read_clear_device_error(); }

cudaError_t launch_scan_wait_selftest(int limit_ms, void* ws, cudaStream_t st) {
  constexpr size_t operand = sizeof(float) * 2 * scan::kTokForward * 32;
  static_assert(kSelftestRows >= 12 * 2 * 32 && kSelftestBytes >= kSelftestRows + 3 * operand,
                "two items of 32 float32 channels");
  return scan::lone_item(ws, static_cast<uint64_t>(limit_ms) * 1000000ull, st);
}

// For either direction and any alignment: as many items as the shortest make.
size_t scan_workspace_bytes(int B, int N, int D, int dtype) {
  const int tiles = cdiv(N, scan::kTokLeast);
  if (tiles == 1 || scan::always_whole(B * cdiv(D, scan::channels_per_piece(dtype)), N)) return 0;
  return 12 * scan::words(B, D, dtype, tiles);
}

cudaError_t launch_scan(const ScanArgs& a, cudaStream_t st) {
  const int w = scan::alignment(a);
  return scan::dispatch(a.dtype, a.form, a.gate.p != nullptr, [&](auto t, auto form, auto gate) {
    using T = typename decltype(t)::type;
    constexpr int F = decltype(form)::value;
    constexpr bool G = decltype(gate)::value != 0;
    if (w == 16) return scan::forward<T, F, G, 16>(a, st);
    if constexpr (sizeof(T) == 2)
      if (w == 2) return scan::forward<T, F, G, 2>(a, st);
    return scan::forward<T, F, G, 4>(a, st);
  });
}

cudaError_t launch_scan_backward(const ScanArgs& a, cudaStream_t st) {
  const int w = scan::alignment(a);
  return scan::dispatch(a.dtype, a.form, a.gate.p != nullptr, [&](auto t, auto form, auto gate) {
    using T = typename decltype(t)::type;
    constexpr int F = decltype(form)::value;
    constexpr bool G = decltype(gate)::value != 0;
    if (w == 16) return scan::backward<T, F, G, 16>(a, st);
    if constexpr (sizeof(T) == 2)
      if (w == 2) return scan::backward<T, F, G, 2>(a, st);
    return scan::backward<T, F, G, 4>(a, st);
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
