// cache_append.cu - keys and values of new tokens into the paged cache, and the
// bounds of the pages that change (sm_103a).
//
// bf16 rows are copied. int8 rows get one scale a (token, head), s = max|x| /
// 127, int4 rows one for every 32 channels, s = max|x| / 7 (fp32, rounded to
// nearest); the code is the whole number nearest to x / s, ties to even, decided
// exactly: c = x / s with an approximate reciprocal, rounded, is at most one off; the
// residual x - c s is a multiple of s's last place below 2 s and therefore exact in
// one fused multiply-add, and its comparison with s / 2 says whether c moves by one.
//
// Bounds of a page and head are the smallest and the largest stored value of each
// channel over the page's keys 0 .. the last new one: rounded down and up to
// bf16 where the cache holds codes. They are formed anew from the page's rows
// (not updated), so keys that a refused draft left behind never stay in them.
//
// HBM binds a prompt (rows read once, written once), latency a decode step. The slots of one call come in runs of neighbours
// in one page. A warp (a decode step: a CTA) takes a run and a head: 16-byte pieces of a row by neighbouring lanes, old rows
// from the cache and new ones from the input (with one run a page no thread reads what another one writes in the same call; with
// several a run may read rows that another one is writing, for bounds that are not defined then), and one reduction of both bounds over
// its lanes. 33K tokens x 8 heads of 128 channels: bf16 46 us (6.1 TB/s, 0.9 of the copy rate), int8 and int4 81 and 83
// (27 instructions a value, issue slots 70 % busy, DRAM 26 %; 64 registers a thread, some spilled); a token for each of 64 requests 2.9
// us (int8 5.2), four each into an int4 cache 6.1.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fd.h"
#include "ptx.cuh"
#include "step.h"

namespace fd {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}

// top / TOP rounded to nearest: with y the reciprocal rounded to nearest and q within a place of the quotient, q + (top - q
// TOP) y rounds to it (Markstein); top - q TOP is exact. Below 2^-100 and for no number the division itself.
template <int TOP>
__device__ __forceinline__ float scale_of(float top) {
  constexpr float y = 1.f / TOP;
  const float q = top * y, s = fmaf(fmaf(-q, static_cast<float>(TOP), top), y, q);
  return top >= 0x1p-100f && top < INFINITY ? s : __fdiv_rn(top, static_cast<float>(TOP));
}

__device__ __forceinline__ float reciprocal(float s) {  // within a place
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: whole numbers stand in the low bits of a sum with it

// Codes of eight channels whose scale is s (the largest magnitude over TOP), as whole numbers in fp32.
__device__ __forceinline__ void codes8(float (&x)[8], float s, float (&q)[8]) {
  if (!(s > 0x1p-100f && s < 0x1p100f)) {
    // where 1 / s would overflow or lose places: both times a power of two (x that this takes to 0 are 0 beside s)
    const float f = s < 1.f ? 0x1p110f : 0x1p-110f;
    // no codes for zeros, nor for a row with an infinity or NaN: its scale makes it NaN
    const bool none = !(s > 0.f && s < INFINITY);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = none ? 0.f : x[i] * f;
    s = none ? 1.f : s * f;
  }
  const float inv = reciprocal(s);
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = fmaf(x[i], inv, kWhole) - kWhole;
    off = fmaxf(off, fabsf(fmaf(-q[i], s, x[i])));
  }
  if (off < 0.5f * s) return;
  // a quotient at a half, or next to one and on its other side
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = fmaf(-q[i], s, x[i]), r2 = r + r;
    const bool odd = static_cast<int>(q[i]) & 1;
    if (r2 > s || (r2 == s && odd)) q[i] += 1.f;
    else if (r2 < -s || (r2 == -s && odd)) q[i] -= 1.f;
  }
}

// Running bounds of a lane's eight channels: fp32, or bf16 pairs where the cache holds bf16.
template <int KIND>
struct Bounds {
  float lo[8], hi[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  }
  __device__ __forceinline__ void join(int x) {  // with the lane `x` away
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], x));
      hi[i] = max_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], x));
    }
  }
  __device__ __forceinline__ void rounded(uint4 &down, uint4 &up) const {  // to bf16, outwards
    uint32_t d[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 a = {__float2bfloat16_rd(lo[2 * i]), __float2bfloat16_rd(lo[2 * i + 1])};
      const __nv_bfloat162 b = {__float2bfloat16_ru(hi[2 * i]), __float2bfloat16_ru(hi[2 * i + 1])};
      d[i] = *reinterpret_cast<const uint32_t *>(&a);
      u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    down = make_uint4(d[0], d[1], d[2], d[3]);
    up = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Bounds<KV_BF16> {
  uint32_t lo[4], hi[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) lo[i] = 0x7f807f80u, hi[i] = 0xff80ff80u;
  }
  __device__ __forceinline__ void add(int i, uint32_t x, uint32_t y) {
    asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo[i]) : "r"(x));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi[i]) : "r"(y));
  }
  __device__ __forceinline__ void join(int x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) add(i, __shfl_xor_sync(0xffffffffu, lo[i], x), __shfl_xor_sync(0xffffffffu, hi[i], x));
  }
  __device__ __forceinline__ void rounded(uint4 &down, uint4 &up) const {
    down = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    up = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
};

// What a lane holds of a row of the cache: 8 channels.
template <int KIND>
struct Piece;
template <>
struct Piece<KV_BF16> {
  uint4 w;
};
template <>
struct Piece<KV_I8> {
  uint2 w;
  float s;
};
template <>
struct Piece<KV_I4> {
  uint32_t w;
  float s;
};

template <int KIND>
__device__ __forceinline__ void fold(Bounds<KIND> &b, const Piece<KIND> &r) {
  if constexpr (KIND == KV_BF16) {
    const uint32_t x[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) b.add(i, x[i], x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int c;
      if constexpr (KIND == KV_I8) c = static_cast<int>((i < 4 ? r.w.x : r.w.y) << (24 - 8 * (i & 3))) >> 24;
      else c = static_cast<int>(r.w << (28 - 4 * i)) >> 28;
      const float f = static_cast<float>(c);
      b.lo[i] = min_nan(b.lo[i], __fmul_rd(f, r.s));  // (code times scale has up to 31 bits)
      b.hi[i] = max_nan(b.hi[i], __fmul_ru(f, r.s));
    }
  }
}

// The same from the codes as whole numbers in fp32.
template <int KIND>
__device__ __forceinline__ void fold(Bounds<KIND> &b, const float (&q)[8], float s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    b.lo[i] = min_nan(b.lo[i], __fmul_rd(q[i], s));
    b.hi[i] = max_nan(b.hi[i], __fmul_ru(q[i], s));
  }
}

template <int KIND, int D>
struct Append {
  static constexpr int kLanes = D / 8;  // lanes a row
  static constexpr int kPieceBytes = KIND == KV_BF16 ? 16 : (KIND == KV_I8 ? 8 : 4);

  // Codes of a new row's piece; lanes of one scale agree on it. The bounds take it where `in`.
  static __device__ __forceinline__ Piece<KIND> quantise(const uint4 &w, Bounds<KIND> *bounds, bool in) {
    Piece<KIND> r;
    if constexpr (KIND == KV_BF16) {
      r.w = w;
      if (bounds && in) fold<KIND>(*bounds, r);
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      uint32_t m = 0u;  // the largest magnitudes of even and odd channels
      auto grow = [&](uint32_t x) { asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x)); };
#pragma unroll
      for (int i = 0; i < 4; ++i) grow(u[i] & 0x7fff7fffu);
      constexpr int span = KIND == KV_I8 ? kLanes : 4;
#pragma unroll
      for (int o = 1; o < span; o <<= 1) grow(__shfl_xor_sync(0xffffffffu, m, o));
      constexpr int kTop = KIND == KV_I8 ? 127 : 7;
      r.s = scale_of<kTop>(max_nan(bf16_lo(m), bf16_hi(m)));
      float x[8], q[8];
      unpack8(w, x);
      codes8(x, r.s, q);
      if (bounds && in) fold<KIND>(*bounds, q, r.s);
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(q[i] + kWhole);  // (two's complement in the low bits)
      if constexpr (KIND == KV_I8) {
        r.w.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        r.w.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
      } else {
        r.w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w |= (c[i] & 15u) << (4 * i);
      }
    }
    return r;
  }
};

__device__ __forceinline__ long long slot_at(const CacheAppendParams &p, long long i) {
  long long s = p.slots64 ? static_cast<const long long *>(p.slots)[i * p.s_s]
                          : static_cast<const int *>(p.slots)[i * p.s_s];
  if (s >= p.num_slots) {
    if (p.status) atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
    s = -1;
  }
  return s < 0 ? -1 : s;
}

// WARPS take a run together: 1 (each warp a run of its own, no barrier) where tokens are many and pages small; kWarps where
// each token has a page of its own (a decode step: latency counts) or runs are long. ROWS: rows of the input that a lane has under
// way in each tensor.
template <int KIND, int D, int WARPS, int ROWS>
__global__ void __launch_bounds__(kThreads, KIND != KV_BF16 ? 8 : (ROWS == 8 ? 4 : 6)) fd_cache_append_kernel(const __grid_constant__ CacheAppendParams p) {
  using A = Append<KIND, D>;
  constexpr int kRows = 32 * WARPS / A::kLanes;  // rows at a time
  __shared__ uint4 part[WARPS][2][A::kLanes];
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const int tid = WARPS == 1 ? lane : threadIdx.x;
  const int sub = tid % A::kLanes, group = tid / A::kLanes;
  // a CTA's (or a warp's) head and tokens
  const long long unit = WARPS == 1 ? static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5) : blockIdx.x;
  const int h = static_cast<int>(unit % p.Hkv);
  const long long c0 = unit / p.Hkv * p.chunk;
  const long long c1 = c0 + p.chunk < p.T ? c0 + p.chunk : p.T;
  if (c0 >= p.T) return;
  griddep_wait();  // inputs written by the previous kernel are visible from here on

  auto cache_row = [&](unsigned char *cache, long long slot) {
    return cache + (slot >> p.log2_page) * p.c_sp + (slot & (p.P - 1)) * p.c_ss + h * p.c_sh + sub * A::kPieceBytes;
  };
  auto scale_at = [&](int which, long long slot) {
    return p.scales + which * p.sc_sk + (slot >> p.log2_page) * p.sc_sp + (slot & (p.P - 1)) * p.sc_ss + h * p.sc_sh +
           (KIND == KV_I4 ? sub / 4 : 0);
  };
  auto load = [&](long long slot) {  // a key of the cache
    Piece<KIND> r;
    const unsigned char *at = cache_row(p.k_cache, slot);
    if constexpr (KIND == KV_BF16) r.w = *reinterpret_cast<const uint4 *>(at);
    if constexpr (KIND == KV_I8) r.w = *reinterpret_cast<const uint2 *>(at), r.s = *scale_at(0, slot);
    if constexpr (KIND == KV_I4) r.w = *reinterpret_cast<const uint32_t *>(at), r.s = *scale_at(0, slot);
    return r;
  };
  auto store = [&](int which, long long slot, const Piece<KIND> &r) {
    unsigned char *at = cache_row(which ? p.v_cache : p.k_cache, slot);
    if constexpr (KIND == KV_BF16) *reinterpret_cast<uint4 *>(at) = r.w;
    if constexpr (KIND == KV_I8) *reinterpret_cast<uint2 *>(at) = r.w;
    if constexpr (KIND == KV_I4) *reinterpret_cast<uint32_t *>(at) = r.w;
    if constexpr (KIND != KV_BF16)
      if (sub % (KIND == KV_I8 ? A::kLanes : 4) == 0) *scale_at(which, slot) = r.s;
  };
  constexpr int kUnroll = ROWS;
  struct Rows {
    uint4 k[kUnroll], v[kUnroll];
  };
  auto fetch = [&](long long i, long long t1) {  // rows i, i + kRows, ..
    Rows r;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long t = i + u * kRows;
      r.k[u] = r.v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (t < t1) {
        r.k[u] = __ldcs(reinterpret_cast<const uint4 *>(p.k + t * p.k_st + h * p.k_sh) + sub);
        r.v[u] = __ldcs(reinterpret_cast<const uint4 *>(p.v + t * p.v_st + h * p.v_sh) + sub);
      }
    }
    return r;
  };

  if (!p.bounds) {
    for (long long i = c0 + group; __any_sync(0xffffffffu, i < c1); i += kRows * kUnroll) {
      long long slot[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) slot[u] = i + u * kRows < c1 ? slot_at(p, i + u * kRows) : -1;
      const Rows r = fetch(i, c1);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const Piece<KIND> k = A::quantise(r.k[u], nullptr, false), v = A::quantise(r.v[u], nullptr, false);
        if (slot[u] >= 0) store(0, slot[u], k), store(1, slot[u], v);
      }
    }
    return;
  }
  // Runs that start in these tokens: a slot whose predecessor is not its neighbour, or lies in another page. Lane l looks at
  // token w0 - 1 + l.
  for (long long w0 = c0; w0 < c1; w0 += 31) {
    const long long at = w0 - 1 + lane;
    const long long s = at >= 0 && at < p.T ? slot_at(p, at) : -1;
    const long long ahead = __shfl_up_sync(0xffffffffu, s, 1);
    const bool on = lane > 0 && s >= 0 && ahead >= 0 && ahead + 1 == s && (s & (p.P - 1)) != 0;  // goes on from the token ahead
    const unsigned going = __ballot_sync(0xffffffffu, on);
    unsigned todo = __ballot_sync(0xffffffffu, lane > 0 && s >= 0 && !on && at < c1);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const long long t0 = w0 - 1 + l, first = __shfl_sync(0xffffffffu, s, l);
      const int off = static_cast<int>(first & (p.P - 1)), most = p.P - off;
      // how far the run goes: as far as the window shows, and on from there
      const unsigned rest = l < 31 ? ~(going >> (l + 1)) : 1u;
      int n = l < 31 ? min(31 - l, __ffs(rest) - 1) + 1 : 1;
      if (l + n == 32) {
        while (n < most) {
          const long long j = t0 + n + lane;
          const bool same = n + lane < most && j < p.T && slot_at(p, j) == first + n + lane;
          const unsigned stop = __ballot_sync(0xffffffffu, !same);
          const int more = stop ? __ffs(stop) - 1 : 32;
          n += more;
          if (more < 32) break;
        }
      }
      Bounds<KIND> bounds;
      bounds.clear();
      Rows r = fetch(t0 + group, t0 + n);  // (the first new rows are on their way with the old ones)
      // the keys that the page holds ahead of the run
      constexpr int kOld = KIND == KV_BF16 ? 8 : 4;
      for (int o = group; o < off; o += kRows * kOld) {
        Piece<KIND> old[kOld];
#pragma unroll
        for (int u = 0; u < kOld; ++u)
          if (o + u * kRows < off) old[u] = load(first - off + o + u * kRows);
#pragma unroll
        for (int u = 0; u < kOld; ++u)
          if (o + u * kRows < off) fold<KIND>(bounds, old[u]);
      }
      // the run
      for (int i = group;; ) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const bool in = i + u * kRows < n;
          const Piece<KIND> k = A::quantise(r.k[u], &bounds, in), v = A::quantise(r.v[u], nullptr, false);
          if (in) {
            store(0, first + i + u * kRows, k);
            store(1, first + i + u * kRows, v);
          }
        }
        i += kRows * kUnroll;
        if (!__any_sync(0xffffffffu, i < n)) break;
        r = fetch(t0 + i, t0 + n);
      }
      // over the groups of a warp, then over the warps
#pragma unroll
      for (int x = A::kLanes; x < 32; x <<= 1) bounds.join(x);
      uint4 down, up;
      __nv_bfloat16 *to = p.bounds + (first >> p.log2_page) * p.b_sp + h * p.b_sh;
      bounds.rounded(down, up);
      if constexpr (WARPS == 1) {
        if (lane < A::kLanes) {
          reinterpret_cast<uint4 *>(to)[lane] = down;
          reinterpret_cast<uint4 *>(to + p.b_sm)[lane] = up;
        }
      } else {
        // (rounded outwards each: the smallest of rounded values is the rounded smallest)
        __syncthreads();  // the last run's parts are read
        if (lane < A::kLanes) part[warp][0][lane] = down, part[warp][1][lane] = up;
        __syncthreads();
        if (tid < A::kLanes) {
          Bounds<KV_BF16> all;
          all.clear();
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            const uint4 d = part[w][0][tid], x = part[w][1][tid];
            all.add(0, d.x, x.x), all.add(1, d.y, x.y), all.add(2, d.z, x.z), all.add(3, d.w, x.w);
          }
          all.rounded(down, up);
          reinterpret_cast<uint4 *>(to)[tid] = down;
          reinterpret_cast<uint4 *>(to + p.b_sm)[tid] = up;
        }
      }
    }
  }
}

template <int KIND, int D>
cudaError_t launch(CacheAppendParams p, cudaStream_t stream) {
  auto go = [&](auto kernel, int warps) {
    const long long units = (p.T + p.chunk - 1) / p.chunk * p.Hkv, ctas = warps == 1 ? (units + kWarps - 1) / kWarps : units;
    return launch_step(kernel, p, dim3(static_cast<unsigned>(ctas)), kThreads, 0, 1, stream);
  };
  const long long rows = p.T * p.Hkv;
  // A token and head a CTA up to 2432 of them (a decode step). An SM holds 8, of bf16 caches 6, by their registers, so this is up to two
  // or three rounds. us, bf16, this / the kernels below: pages of 64, 2048 rows 7.7 / 8.5, 2400 rows 8.5 / 9.4; pages of 16, 1200 rows 4.7 /
  // 3.3, 2400 rows 7.0 / 3.9. (Of quantised caches the kernel is the same on both sides.) Else, with the rows that a lane has under way
  // and the registers that this leaves: 33K tokens x 8 heads, pages of 16, bf16 8 rows 46 us (0.9 of the copy rate), 4 rows 65; int8 and
  // int4 2 rows 81 and 83, 4 rows 94 and 106 (more spills).
  p.chunk = 1;
  if (rows <= 152 * 16) return go(fd_cache_append_kernel<KIND, D, kWarps, 1>, kWarps);
  constexpr bool kQuantised = KIND != KV_BF16;
  constexpr int kMany = kQuantised ? 2 : 8;
  p.chunk = static_cast<int>(std::min<long long>(std::max<long long>(rows / (152 * 24), 1), p.P > 32 ? 31 : 16));
  while ((p.T + p.chunk - 1) / p.chunk * p.Hkv > 0x7fffffff) p.chunk *= 2;
  // CTAs a run for large pages, and for few tokens into a quantised cache (us, a CTA / a warp a run: 23K tokens in runs of 193 x 8
  // heads, pages of 256, int4 82 / 202, bf16 46 / 54; 2000 tokens x 8 heads, pages of 16, int4 15 / 24, bf16 9.9 / 7.6). Tokens a
  // CTA or warp: so many that each warp slot of the GPU has some, and up to 16 or, of large pages, 31, which a look at the slots shows
  // (800 x 4: 7.6, with 16 always 11.0).
  constexpr int kLong = kQuantised ? 1 : 4;
  if (p.P > 32 || (kQuantised && rows < 20000)) return go(fd_cache_append_kernel<KIND, D, kWarps, kLong>, kWarps);
  return go(fd_cache_append_kernel<KIND, D, 1, kMany>, 1);
}

template <int KIND>
cudaError_t launch_d(int head_dim, const CacheAppendParams &p, cudaStream_t stream) {
  return head_dim == 64 ? launch<KIND, 64>(p, stream) : launch<KIND, 128>(p, stream);
}

}  // namespace

cudaError_t launch_cache_append(int kind, int head_dim, CacheAppendParams p, cudaStream_t stream) {
  if (kind == KV_BF16) return launch_d<KV_BF16>(head_dim, p, stream);
  if (kind == KV_I8) return launch_d<KV_I8>(head_dim, p, stream);
  return launch_d<KV_I4>(head_dim, p, stream);
}

}  // namespace fd
