// token_logprobs.cu - log probability and rank of given tokens, entropy and the
// most probable tokens of their rows (sm_103a).
//
//   lse = m + ln sum exp(x_v - m),   logprob = x_tok - lse,
//   entropy = ln l - (sum e_v z_v) / l   with z = x - m, e = exp(z), l = sum e,
//   rank = number of tokens ahead of tok in the order (value down, index up).
//
// The logits are read once, and no unit binds alone: of the 59 us of 3001 rows of 50021 bf16 logits (K = 5, a tenth of the rows has no
// token) the bytes need 40, 10 instructions a logit 36 and the exponentials 28; K = 0 and all rows take 54. A thread takes 16-byte pieces at a stride of the CTA; packed fp32 and bf16 instructions handle two
// logits at once. fp32 sums: a thread adds 530 values at most one after the other
// and folds such sums of longer rows (up to 128); a tree adds the threads'.
//
// The K largest come almost for free: the threads' maxima are known, and with T the K-th largest of the maxima of 32 or 64 groups
// of threads at least K values are >= T, and few more in a row without order. Only threads with a maximum >= T are looked
// at again, out of L2 and by the whole CTA; what is >= T is ranked by counting (a key is value and index in 64 bits).
// Lists of a cluster's CTAs are merged by its first. A row is shared by a cluster of up to 8 CTAs where rows are few: 64 rows of
// 131072 fp32 logits take 11.6 us with K = 20, 8.2 with K = 0. Many short rows have a warp each: 42046 rows of 1559 bf16 logits 117 us with K = 20.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fd.h"
#include "ptx.cuh"
#include "step.h"

namespace fd {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCtas = 8;
constexpr int kMaxKeys = 256;  // values >= T that are sorted at once (at least the threads of a CTA)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Whole numbers in the order of the floats (-0 with 0; NaN below -inf).
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// A list's key: value first, then the lower index. 0: no entry.
typedef unsigned long long Key;
__device__ __forceinline__ Key key_of(float x, int v) {
  const uint32_t o = ordered(x);
  return o ? static_cast<Key>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(v)) : 0ull;
}

// A new key into a warp's list (lane i holds the i-th largest).
__device__ __forceinline__ void insert(Key &mine, Key k) {
  const int lane = threadIdx.x & 31;
  const int at = __popc(__ballot_sync(0xffffffffu, mine > k));
  const Key up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane > at) mine = up;
  else if (lane == at) mine = k;
}

// The 32 largest of two sorted lists, sorted: b is read backwards, the larger of
// each pair is a bitonic sequence of them.
__device__ __forceinline__ Key merge(Key a, Key b_reversed) {
  Key x = a > b_reversed ? a : b_reversed;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key y = __shfl_xor_sync(0xffffffffu, x, o);
    const bool low = (lane & o) == 0;
    x = low == (x > y) ? x : y;
  }
  return x;
}

// Sums of a part of a row, relative to one of its logits m (0 in place of -inf): l = sum e,
// w = sum e z (z in units of ln 2), n = tokens ahead of the given one.
struct Part {
  float m, l, w;
  int n;
};

__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

// (from - to) in units of ln 2 for sums that go from one reference to a larger one; -1000 at least, where all of a sum is
// 0 (a difference that overflows would make 0 times it NaN). A sum relative to -inf is 0 and stays.
__device__ __forceinline__ float shift_of(float from, float to) {
  return from == -INFINITY ? 0.f : fmaxf((from - base_of(to)) * kLog2e, -1000.f);
}

// The sums relative to the maximum `top` >= p.m.
__device__ __forceinline__ void rebase(Part &p, float top) {
  const float d = shift_of(p.m, top), f = exp2f(d);
  p.w = f * (p.w + d * p.l);
  p.l *= f;
  p.m = top;
}

template <bool F32>
struct Row {
  static constexpr int kVec = F32 ? 4 : 8;  // values of a piece
  const char *base;                         // the row's first value, rounded down to 16 bytes
  int lead, V;                              // values of the first piece ahead of the row

  __device__ __forceinline__ int pieces() const { return (lead + V + kVec - 1) / kVec; }
  __device__ __forceinline__ bool whole(int c) const { return c * kVec >= lead && (c + 1) * kVec <= lead + V; }
  // Piece c, all of it in the row.
  __device__ __forceinline__ uint4 fetch(int c) const { return __ldg(reinterpret_cast<const uint4 *>(base) + c); }
  // Piece c; places outside the row read -inf.
  __device__ __forceinline__ uint4 load(int c) const {
    if (whole(c)) return fetch(c);
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = F32 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = c * kVec - lead + i;
      if (v >= 0 && v < V) {
        if constexpr (F32) {
          u[i] = reinterpret_cast<const uint32_t *>(base)[lead + v];
        } else {
          const uint32_t x = reinterpret_cast<const unsigned short *>(base)[lead + v];
          u[i / 2] = i & 1 ? (u[i / 2] & 0xffffu) | x << 16 : (u[i / 2] & 0xffff0000u) | x;
        }
      }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  static __device__ __forceinline__ float value(const uint4 &w, int i) {  // value i of a piece
    const int at = F32 ? i : i >> 1;
    const uint32_t u = at & 2 ? (at & 1 ? w.w : w.z) : (at & 1 ? w.y : w.x);
    return __uint_as_float(F32 || (i & 1) ? (F32 ? u : u & 0xffff0000u) : u << 16);
  }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[kVec]) {
    if constexpr (F32) {
      x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};

// Pairs of fp32 (one instruction for both on sm_100 and later).
typedef unsigned long long F2;
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(F2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The smallest number of the logits' type above x (NaN above +inf: nothing is).
template <bool F32>
__device__ __forceinline__ float next_above(float x) {
  const uint32_t u = __float_as_uint(x), one = F32 ? 1u : 0x10000u;
  if (x == 0.f) return __uint_as_float(one);
  return __uint_as_float(u & 0x80000000u ? u - one : u + one);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t both(float x) {  // a bf16 value twice
  const uint32_t u = __float_as_uint(x);
  return u >> 16 | (u & 0xffff0000u);
}
// What a thread sums over its pieces of a row.
//
// Sums are relative to `base`, the largest logit of its first pieces, until one exceeds that by 40: 2^24 exponentials up to
// e^40 stay in range, and rescaling at every new maximum would cost a warp as much as the rest (some lane has one at
// nearly every piece). z = x - base is kept above -inf, which would make e z NaN where e is 0 (a NaN stays): fp32 at -160
// ln 2, bf16 by raising x to a bf16 value `least` about 120 below base, two at once.
//
// Tokens ahead of the given one are counted by the sign of x - t (one shift-and-add a logit): `less` of them are below t. That
// misses where t is no finite number or not above every `least` that logits were raised to (the last one, or, of pieces of -inf ahead
// of the first number, -120), and where logits are NaN or +inf (l is NaN then): there the pieces are counted again.
template <bool F32, bool HALVES, bool LONG>
struct Stream {
  static constexpr int kVec = Row<F32>::kVec;
  float base = -INFINITY, high = -INFINITY;
  float most = -INFINITY, odd = -INFINITY;                     // the maxima: of all, or (HALVES) of even and odd places
  float minus = 0.f;                                           // -base (0 while that is -inf)
  F2 l2, w2;                                                   // sums (LONG: since the last fold)
  float folded_l = 0.f, folded_w = 0.f;                        // LONG: sums ahead of it
  unsigned less = 0;
  uint32_t least = 0xc2f0c2f0u;                                // bf16: -120 while base is -inf
  bool blank = false;                                          // bf16: pieces were added while base was -inf

  // Below about -3.33e38 (bf16) there is no finite `least`: z is 0 or far below, so w is 0 whatever the -inf made of it.
  __device__ __forceinline__ bool lowest() const { return !F32 && base < -3.3e38f && base != -INFINITY; }
  __device__ __forceinline__ void sums(float &l, float &w) const {
    float l0, l1, w0, w1;
    split(l2, l0, l1);
    split(w2, w0, w1);
    l = l0 + l1;
    w = w0 + w1;
    if constexpr (LONG) l += folded_l, w += folded_w;
    if (lowest()) w = 0.f;
  }
  __device__ __forceinline__ void fold() {
    float l, w;
    sums(l, w);
    folded_l = l, folded_w = w;
    l2 = w2 = pair(0.f, 0.f);
  }
  __device__ __forceinline__ void rebase_to(float top) {
    float l, w;
    sums(l, w);
    const float d = shift_of(base, top), f = exp2f(d);
    w = f * (w + d * l);
    l *= f;
    if constexpr (LONG) folded_l = l, folded_w = w, l = w = 0.f;
    l2 = pair(l, 0.f);
    w2 = pair(w, 0.f);
    base = top;
    high = top + 40.f;
    minus = -base_of(base);
    if constexpr (!F32) least = both(__bfloat162float(__float2bfloat16_rd(-minus - fmaxf(120.f, fabsf(minus) * 0x1p-6f))));
  }
  // The values of N pieces; t: what the values of a piece are compared with.
  template <int N>
  __device__ __forceinline__ void add(const uint4 (&u)[N], const float (&t)[N]) {
    float even, top;
    if constexpr (F32) {
      even = top = -INFINITY;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        even = fmaxf(even, fmaxf(__uint_as_float(u[k].x), __uint_as_float(u[k].z)));
        top = fmaxf(top, fmaxf(__uint_as_float(u[k].y), __uint_as_float(u[k].w)));
      }
    } else {
      uint32_t x = 0xff80ff80u;
#pragma unroll
      for (int k = 0; k < N; ++k) x = max_bf16x2(x, max_bf16x2(max_bf16x2(u[k].x, u[k].y), max_bf16x2(u[k].z, u[k].w)));
      even = __uint_as_float(x << 16), top = __uint_as_float(x & 0xffff0000u);
    }
    if constexpr (HALVES) most = fmaxf(most, even), odd = fmaxf(odd, top);
    top = fmaxf(even, top);
    if constexpr (!HALVES) most = fmaxf(most, top);
    if (top > high) rebase_to(top);
    if constexpr (!F32) blank |= base == -INFINITY;
    const F2 minus2 = pair(minus, minus), log2e = pair(kLog2e, kLog2e);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t x[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      const F2 minus_t = pair(-t[k], -t[k]);
#pragma unroll
      for (int i = 0; i < kVec / 2; ++i) {
        F2 v;
        if constexpr (F32) {
          v = pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
        } else {
          const uint32_t y = max_nan_bf16x2(x[i], least);
          v = pair(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
        }
        F2 z = mul2(add2(v, minus2), log2e);
        float z0, z1, d0, d1;
        split(z, z0, z1);
        if constexpr (F32) {
          z0 = max_nan(z0, -160.f), z1 = max_nan(z1, -160.f);
          z = pair(z0, z1);
        }
        const F2 e = pair(fast_exp2(z0), fast_exp2(z1));
        l2 = add2(l2, e);
        w2 = fma2(e, z, w2);
        split(add2(v, minus_t), d0, d1);
        less += __float_as_uint(d0) >> 31;
        less += __float_as_uint(d1) >> 31;
      }
    }
  }
  // Whether `less` may be wrong, t the smallest number that was compared with.
  __device__ __forceinline__ bool recount(float t, float l) const {
    return !(fabsf(t) < INFINITY) || l != l || (!F32 && (t <= __uint_as_float(least << 16) || (blank && t <= -120.f)));
  }
};

// LONG: rows of which a thread takes more than kThreadValues logits, half of them in each sum of a pair.
constexpr int kThreadValues = 1024;

template <bool F32, int kThreads, bool LONG>
__global__ void __launch_bounds__(kThreads, LONG || kThreads == 256 ? 1024 / kThreads : (kThreads == 32 ? 32 : 1280 / kThreads))
    fd_token_logprobs_kernel(const __grid_constant__ LogprobsParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kVec = Row<F32>::kVec;
  constexpr int kPieces = kThreads == 256 ? 4 : 3;  // pieces a thread has in flight
  constexpr int kFold = kThreadValues / kVec * kThreads;  // pieces of so many after which a CTA's threads fold their sums
  __shared__ Part parts[kWarps];
  __shared__ Part cta_part;            // read by the cluster's first CTA
  __shared__ uint32_t maxima[kThreads];
  __shared__ unsigned short flagged[kThreads];
  __shared__ Key keys[kMaxKeys];
  __shared__ int num_flagged, num_keys;
  __shared__ Key cta_list[32];         // read by the cluster's first CTA
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = p.ctas, rank = ctas > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int64_t r = blockIdx.x / ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) num_flagged = num_keys = 0;
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  const long long tok = p.tok64 ? static_cast<const long long *>(p.tokens)[r * p.t_s]
                                : static_cast<const int *>(p.tokens)[r * p.t_s];
  if (tok < 0 || tok >= p.V) {  // no token: the row is not read (every CTA of the cluster returns)
    if (rank != 0) return;
    if (tok >= p.V && tid == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_BAD_TOKEN);
    if (tid == 0) {
      p.logprobs[r] = 0.f;
      if (p.ranks) p.ranks[r] = -1;
      if (p.entropy) p.entropy[r] = 0.f;
    }
    if (tid < p.K) p.top_ids[r * p.ti_s + tid] = -1, p.top_logprobs[r * p.tl_s + tid] = 0.f;
    return;
  }
  Row<F32> row;
  {
    const char *first = static_cast<const char *>(p.logits) + r * p.l_s * (F32 ? 4 : 2);
    row.base = reinterpret_cast<const char *>(reinterpret_cast<uintptr_t>(first) & ~static_cast<uintptr_t>(15));
    row.lead = static_cast<int>(first - row.base) / (F32 ? 4 : 2);
    row.V = p.V;
  }
  float xt;
  if constexpr (F32) xt = reinterpret_cast<const float *>(row.base)[row.lead + tok];
  else xt = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row.base)[row.lead + tok]);
  // this CTA's pieces
  const int total = row.pieces(), per = (total + ctas - 1) / ctas;
  const int p0 = min(total, rank * per), p1 = min(total, p0 + per);

  // ---- the stream
  // Ahead of the token an equal logit counts too (to a difference from -0 both zeros are +0); behind it x > xt is x >= the
  // next number above.
  const float xt_here = xt == 0.f ? -0.f : xt;
  const float xt_above = next_above<F32>(xt);
  const int tok_piece = (static_cast<int>(tok) + row.lead) / kVec;
  Stream<F32, kWarps == 1, LONG> sum;
  sum.l2 = sum.w2 = pair(0.f, 0.f);
  int n = 0;
  // Tokens ahead of the given one in a piece, one by one.
  auto exact = [&](int c, const uint4 &u) {
    float x[kVec];
    row.unpack(u, x);
    int count = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = c * kVec - row.lead + i;
      count += v >= 0 && v < row.V && (x[i] > xt || (x[i] == xt && v < tok));
    }
    return count;
  };
  // Where the row's first and last piece are partial, their threads take them apart from the stream.
  auto partial = [&](int c) {
    const uint4 u[1] = {row.load(c)};
    const float t[1] = {0.f};
    const unsigned less = sum.less;
    sum.add(u, t);
    sum.less = less;
    n += exact(c, u[0]);
  };
  {
    const bool head = p0 + tid == 0 && row.lead != 0;
    const bool tail = (row.lead + row.V) % kVec != 0 && p0 < p1 && p1 == total && (total - 1 - p0) % kThreads == tid;
    const int c1 = p1 - (tail ? 1 : 0);
    int c = p0 + tid;
    if (head && c < c1) {
      partial(c);
      c += kThreads;
    }
    const int c_first = c;
    for (; c + (kPieces - 1) * kThreads < c1; c += kPieces * kThreads) {
      uint4 u[kPieces];
      float t[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) u[k] = row.fetch(c + k * kThreads);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) t[k] = c + k * kThreads < tok_piece ? xt_here : xt_above;
      sum.add(u, t);
      if constexpr (LONG)
        if ((c ^ (c + kPieces * kThreads)) & -kFold) sum.fold();
    }
    uint4 left[kPieces - 1];
#pragma unroll
    for (int k = 0; k < kPieces - 1; ++k)
      if (c + k * kThreads < c1) left[k] = row.fetch(c + k * kThreads);
#pragma unroll
    for (int k = 0; k < kPieces - 1; ++k) {
      if (c + k * kThreads < c1) {
        const uint4 u[1] = {left[k]};
        const float t[1] = {c + k * kThreads < tok_piece ? xt_here : xt_above};
        sum.add(u, t);
      }
    }
    if (tail) partial(total - 1);
    // whole pieces: c_first, c_first + kThreads, ..
    const int pieces = c_first < c1 ? (c1 - c_first + kThreads - 1) / kThreads : 0;
    float l, w;
    sum.sums(l, w);
    if (sum.recount(xt, l)) {
      for (int i = 0; i < pieces; ++i) n += exact(c_first + i * kThreads, row.load(c_first + i * kThreads));
    } else {
      n += pieces * kVec - static_cast<int>(sum.less);
      if (tok_piece >= c_first && tok_piece < c1 && (tok_piece - p0) % kThreads == tid) {
        // (the token's own piece was compared as one behind it)
        float x[kVec];
        row.unpack(row.fetch(tok_piece), x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) n += x[i] == xt && tok_piece * kVec - row.lead + i < tok;
      }
    }
  }
  Part mine;
  sum.sums(mine.l, mine.w);
  mine.m = sum.base;
  mine.n = n;

  // ---- the CTA's maximum (over the threads' maxima, which the search for the K largest needs too)
  const uint32_t mo = p0 + tid < p1 ? ordered(fmaxf(sum.most, sum.odd)) : 0u;
  maxima[tid] = mo;
  __syncthreads();
  uint32_t all[kWarps], top_o = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    all[i] = maxima[32 * i + lane];
    top_o = max(top_o, all[i]);
  }
  top_o = __reduce_max_sync(0xffffffffu, top_o);
  rebase(mine, top_o ? value_of(top_o) : -INFINITY);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mine.l += __shfl_xor_sync(0xffffffffu, mine.l, o);
    mine.w += __shfl_xor_sync(0xffffffffu, mine.w, o);
  }
  mine.n = __reduce_add_sync(0xffffffffu, mine.n);
  if (lane == 0) parts[warp] = mine;

  // ---- the K largest of this CTA's pieces
  if (p.K > 0) {
    // T: the K-th largest of the maxima of 32 (K up to 8) or 64 groups (those of a lane in all warps, or in the even and the
    // odd ones; of a single warp its lanes' even and odd places), its upper 18 bits, bit by bit. At least K values are >= T,
    // and of a row without order up to 9 or 44 (a little more for the cut bits). 0 where fewer groups have a piece.
    uint32_t g0 = 0, g1 = 0;
    if constexpr (kWarps == 1) {
      if (mo != 0) g0 = ordered(sum.most), g1 = ordered(sum.odd);
    } else {
#pragma unroll
      for (int i = 0; i < kWarps; i += 2) g0 = max(g0, all[i]), g1 = max(g1, all[i + 1]);
    }
    if (p.K <= 8) g0 = max(g0, g1), g1 = 0;
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit >= 14; --bit) {
      const uint32_t to = t | 1u << bit;
      const int count = __popc(__ballot_sync(0xffffffffu, g0 >= to)) + __popc(__ballot_sync(0xffffffffu, g1 >= to));
      if (count >= p.K) t = to;
    }
    const float limit = t > ordered(-INFINITY) ? value_of(t) : -INFINITY;
    // threads with a value >= T are looked at again: their pieces, shared out over the CTA
    if (mo != 0 && mo >= t) flagged[atomicAdd(&num_flagged, 1)] = tid;
    __syncthreads();
    const int pieces = (p1 - p0 + kThreads - 1) / kThreads, items = num_flagged * pieces;
    // Piece of item i: the thread flagged[i / pieces], its piece i % pieces. The quotient in fp32 is right for every number of
    // pieces and threads that V up to 2^24 allows (checked one by one at both ends of every quotient).
    const float inv = 1.f / pieces;
    auto item = [&](int i) {
      const int f = static_cast<int>((i + 0.5f) * inv);
      return p0 + flagged[f] + (i - f * pieces) * kThreads;
    };
    for (int i = tid; i < items; i += kThreads) {
      const int c = item(i);
      if (c < p1) {
        const uint4 u = row.load(c);
        float x[kVec], top = -INFINITY;
        row.unpack(u, x);
#pragma unroll
        for (int v = 0; v < kVec; ++v) top = fmaxf(top, x[v]);
        if (top >= limit) {  // (few)
          unsigned hits = 0;
#pragma unroll
          for (int v = 0; v < kVec; ++v) hits |= static_cast<unsigned>(x[v] >= limit) << v;
          while (hits) {
            const int v = __ffs(hits) - 1, at = c * kVec - row.lead + v;
            hits &= hits - 1;
            if (at >= 0 && at < row.V) {
              const int to = atomicAdd(&num_keys, 1);
              if (to < kMaxKeys) keys[to] = key_of(row.value(u, v), at);
            }
          }
        }
      }
    }
    __syncthreads();
    if (num_keys <= kMaxKeys) {
      // each key's place is the number of larger ones
      const int count = num_keys;
      if (tid < 32 && tid >= count) cta_list[tid] = 0;
      for (int i = tid; i < count; i += kThreads) {
        const Key mine = keys[i];
        int at = 0;
#pragma unroll 4
        for (int j = 0; j < count; ++j) at += keys[j] > mine;
        if (at < 32) cta_list[at] = mine;
      }
      __syncthreads();
    } else {
      // many equal values, or a row that rises along a thread's pieces: each warp keeps a list of its share
      Key best = 0;
      for (int i0 = warp * 32; i0 < items; i0 += kThreads) {
        const int i = i0 + lane, c = i < items ? item(i) : p1;
        float x[kVec];
        if (c < p1) row.unpack(row.load(c), x);
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const int at = c * kVec - row.lead + v;
          Key k = c < p1 && x[v] >= limit && at >= 0 && at < row.V ? key_of(x[v], at) : 0;
          Key worst = __shfl_sync(0xffffffffu, best, p.K - 1);
          unsigned in = __ballot_sync(0xffffffffu, k > worst);
          while (in) {
            const int from = __ffs(in) - 1;
            insert(best, __shfl_sync(0xffffffffu, k, from));
            worst = __shfl_sync(0xffffffffu, best, p.K - 1);
            if (lane == from) k = 0;
            in = __ballot_sync(0xffffffffu, k > worst);
          }
        }
      }
      __syncthreads();  // keys are read
      keys[tid] = best;  // (a list a warp)
      __syncthreads();
      if (warp == 0) {
        for (int i = 1; i < kWarps; ++i) best = merge(best, keys[32 * i + 31 - lane]);
        cta_list[lane] = best;
      }
    }
  }

  // ---- sums
  __syncthreads();
  if (warp == 0) {
    mine = lane < kWarps ? parts[lane] : Part{0.f, 0.f, 0.f, 0};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      mine.l += __shfl_xor_sync(0xffffffffu, mine.l, o);
      mine.w += __shfl_xor_sync(0xffffffffu, mine.w, o);
      mine.n += __shfl_xor_sync(0xffffffffu, mine.n, o);
    }
    if (lane == 0) cta_part = mine;
  }
  if (ctas > 1) cluster.sync();
  if (rank == 0 && warp == 0) {
    __syncwarp();
    Part all = {-INFINITY, 0.f, 0.f, 0};
    if (lane < ctas) all = ctas > 1 ? *cluster.map_shared_rank(&cta_part, lane) : cta_part;
    Key best = 0;
    if (p.K > 0) {
      best = cta_list[lane];
      if (ctas > 1) {
        Key other[kMaxCtas - 1];
#pragma unroll
        for (int c = 1; c < kMaxCtas; ++c) other[c - 1] = c < ctas ? *cluster.map_shared_rank(&cta_list[31 - lane], c) : 0;
#pragma unroll
        for (int c = 1; c < kMaxCtas; ++c)
          if (c < ctas) best = merge(best, other[c - 1]);
      }
    }
    if (ctas > 1) {
      float top = all.m;
#pragma unroll
      for (int o = kMaxCtas / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      rebase(all, top);
#pragma unroll
      for (int o = kMaxCtas / 2; o > 0; o >>= 1) {
        all.l += __shfl_xor_sync(0xffffffffu, all.l, o);
        all.w += __shfl_xor_sync(0xffffffffu, all.w, o);
        all.n += __shfl_xor_sync(0xffffffffu, all.n, o);
      }
    }
    all.m = __shfl_sync(0xffffffffu, all.m, 0);  // (lanes from kMaxCtas on held nothing)
    all.l = __shfl_sync(0xffffffffu, all.l, 0);
    const bool none = all.m == -INFINITY && all.l == 0.f;  // every logit is -inf
    const float log_l = logf(all.l);
    // (x - m) - ln l keeps the last places that m + ln l would lose
    if (lane == 0) {
      p.logprobs[r] = none ? -INFINITY : (xt - all.m) - log_l;
      if (p.ranks) p.ranks[r] = all.n;
      if (p.entropy) p.entropy[r] = none ? 0.f : log_l - all.w / all.l * kLn2;
    }
    if (lane < p.K) {
      const float x = value_of(static_cast<uint32_t>(best >> 32));
      p.top_ids[r * p.ti_s + lane] = best ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
      p.top_logprobs[r * p.tl_s + lane] = none ? -INFINITY : (best ? (x - all.m) - log_l : __uint_as_float(0x7fc00000u));
    }
  }
  if (ctas > 1) cluster.sync();  // the first CTA has read
}

}  // namespace

// Rows that fill the GPU with smaller CTAs: ten an SM (1000 x 50021 bf16 26.4 us, with CTAs twice the size 29.2; 500 x 50021 15.2, 14.5).
constexpr int kManyRows = 900;

cudaError_t launch_token_logprobs(LogprobsParams p, cudaStream_t stream) {
  // CTAs a row: more while all fit the GPU at once (four of 256 threads an SM) with 4096 values each at least.
  p.ctas = 1;
  while (p.ctas < kMaxCtas && 2ll * p.ctas * p.R <= 608 && p.V >= 2 * p.ctas * 4096) p.ctas *= 2;
  // Threads: half as many where rows fill the GPU with CTAs of half the size, and half again for short rows: the parts of a CTA that
  // wait (the token's logit, the K largest) then lie beside the streams of more others. us, K = 5, 64 / 128 / 256 threads: 11120 x
  // 9700 bf16 61 / 73 / 126, 20000 x 6000 77 / 101 / 177, 4000 x 32000 66 / 57 / 70, 3001 x 50021 74 / 63 / 74, 700 x 9700 8.5 / 7.4 / 10.5.
  // A warp a row (no barrier that waits; 32 an SM) where the rows are short and many: us, 32 / 64 threads, 42046 x 1559 bf16: K = 0
  // 61 / 91, K = 5 93 / 139, K = 20 114 / 159; 3000 x 4000 bf16, K = 8: 11.8 / 12.3. A warp looks at up to all of its row again, so
  // with large K in longer rows, or where a second round of rows is not filled, it loses: 20000 x 2000 fp32, K = 20: 70 / 64, 5000 x
  // 4000 bf16, K = 20: 24.8 / 21.5; 5000 x 3900 fp32, K = 8: 32.4 / 24.9.
  const long long bytes = static_cast<long long>(p.V) * (p.f32 ? 4 : 2);
  const bool many = p.R >= kManyRows, brief = p.ctas == 1 && bytes <= 32768;
  const bool single = p.ctas == 1 && (p.K <= 8 ? p.R >= 2432 && bytes <= 8192 : p.R >= 9728 && bytes <= 6400);
  const int threads = single ? 32 : (many && brief ? 64 : (many || brief ? 128 : 256));
  // (rows that take 1024 logits a thread at most need no folds, whose registers cost CTAs an SM: 3001 x 50021 bf16 59 us, with folds
  // 65; 1000 x 262144 bf16 121, without them 116. 64 threads or fewer have such rows only.)
  const bool folds = p.V > static_cast<long long>(kThreadValues) * threads * p.ctas;
  const dim3 grid(static_cast<unsigned>(p.R) * p.ctas);
  auto go = [&](auto f32, auto f16, int n) { return launch_step(p.f32 ? f32 : f16, p, grid, n, 0, n == 256 ? p.ctas : 1, stream); };
  if (threads == 32) return go(fd_token_logprobs_kernel<true, 32, false>, fd_token_logprobs_kernel<false, 32, false>, 32);
  if (threads == 64) return go(fd_token_logprobs_kernel<true, 64, false>, fd_token_logprobs_kernel<false, 64, false>, 64);
  if (threads == 128 && folds) return go(fd_token_logprobs_kernel<true, 128, true>, fd_token_logprobs_kernel<false, 128, true>, 128);
  if (threads == 128) return go(fd_token_logprobs_kernel<true, 128, false>, fd_token_logprobs_kernel<false, 128, false>, 128);
  if (folds) return go(fd_token_logprobs_kernel<true, 256, true>, fd_token_logprobs_kernel<false, 256, true>, 256);
  return go(fd_token_logprobs_kernel<true, 256, false>, fd_token_logprobs_kernel<false, 256, false>, 256);
}

}  // namespace fd
