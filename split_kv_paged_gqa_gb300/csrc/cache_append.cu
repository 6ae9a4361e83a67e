// cache_append.cu - keys and values of new tokens into the paged cache, and the
// bounds of the pages that change (sm_103a).
//
// bf16 rows are copied. int8 rows get one scale a (token, head), s = max|x| /
// 127, int4 rows one for every 32 channels, s = max|x| / 7 (fp32, rounded to
// nearest); the code is the whole number nearest to x / s, ties to even, decided
// exactly: with c = rint(x * (1 / s)) at most one off, the residual x - c s is a
// multiple of s's last place below 2 s and therefore exact in one fused
// multiply-add, and its comparison with s / 2 says whether c moves by one.
//
// Bounds of a page and head are the smallest and the largest stored value of each
// channel over the page's keys 0 .. the last new one: rounded down and up to
// bf16 where the cache holds codes. They are formed anew from the page's rows
// (not updated), so keys that a refused draft left behind never stay in them.
//
// HBM binds a prompt (rows read once, written once), latency a decode step. The
// slots of one call come in runs of neighbours in one page. A CTA takes a
// run and a head: 16-byte pieces of a row by neighbouring lanes, old rows from
// the cache and new ones from the input (no thread reads what another one
// writes in the same call), and one reduction of both bounds over the CTA.
#include <cuda_runtime.h>
#include <stdint.h>

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

// Codes of eight channels whose scale is s (the largest magnitude over TOP).
template <int TOP>
__device__ __forceinline__ void codes8(const float (&x)[8], float s, int (&c)[8]) {
  // (1 / s overflows below 2^-128, and loses places above 2^126: the quotient itself there)
  const bool plain = s > 0x1p-100f && s < 0x1p100f;
  const float inv = plain ? __frcp_rn(s) : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q = rintf(plain ? x[i] * inv : (s != 0.f ? __fdiv_rn(x[i], s) : 0.f));
    const float r = fmaf(-q, s, x[i]), r2 = r + r;
    const bool odd = static_cast<int>(q) & 1;
    if (r2 > s || (r2 == s && odd)) q += 1.f;
    else if (r2 < -s || (r2 == -s && odd)) q -= 1.f;
    // a row with an infinity or NaN has no codes: its scale makes it NaN
    c[i] = s < INFINITY ? max(-TOP, min(TOP, static_cast<int>(q))) : 0;
    if (s == 0.f) c[i] = 0;
  }
}

// Running bounds of a lane's eight channels.
struct Bounds {
  float lo[8], hi[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  }
  __device__ __forceinline__ void add(int i, float down, float up) {
    lo[i] = min_nan(lo[i], down);
    hi[i] = max_nan(hi[i], up);
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
__device__ __forceinline__ void fold(Bounds &b, const Piece<KIND> &r) {
  if constexpr (KIND == KV_BF16) {
    float x[8];
    unpack8(r.w, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) b.add(i, x[i], x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int c;
      if constexpr (KIND == KV_I8) c = static_cast<int>((i < 4 ? r.w.x : r.w.y) << (24 - 8 * (i & 3))) >> 24;
      else c = static_cast<int>(r.w << (28 - 4 * i)) >> 28;
      const float f = static_cast<float>(c);
      b.add(i, __fmul_rd(f, r.s), __fmul_ru(f, r.s));  // (code times scale has up to 31 bits)
    }
  }
}

template <int KIND, int D>
struct Append {
  static constexpr int kLanes = D / 8;             // lanes a row
  static constexpr int kRows = kThreads / kLanes;  // rows at a time
  static constexpr int kPieceBytes = KIND == KV_BF16 ? 16 : (KIND == KV_I8 ? 8 : 4);

  // Codes of a new row's piece; lanes of one scale agree on it.
  static __device__ __forceinline__ Piece<KIND> quantise(const uint4 &w) {
    Piece<KIND> r;
    if constexpr (KIND == KV_BF16) {
      r.w = w;
    } else {
      float x[8];
      unpack8(w, x);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[i]));
      constexpr int span = KIND == KV_I8 ? kLanes : 4;
#pragma unroll
      for (int o = 1; o < span; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      constexpr int kTop = KIND == KV_I8 ? 127 : 7;
      r.s = __fdiv_rn(top, static_cast<float>(kTop));
      int c[8];
      codes8<kTop>(x, r.s, c);
      if constexpr (KIND == KV_I8) {
        r.w.x = (c[0] & 255) | (c[1] & 255) << 8 | (c[2] & 255) << 16 | static_cast<uint32_t>(c[3]) << 24;
        r.w.y = (c[4] & 255) | (c[5] & 255) << 8 | (c[6] & 255) << 16 | static_cast<uint32_t>(c[7]) << 24;
      } else {
        r.w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w |= static_cast<uint32_t>(c[i] & 15) << (4 * i);
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

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) fd_cache_append_kernel(const __grid_constant__ CacheAppendParams p) {
  using A = Append<KIND, D>;
  __shared__ float part[kWarps][2][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = tid % A::kLanes, group = tid / A::kLanes, h = blockIdx.y;
  const long long c0 = static_cast<long long>(blockIdx.x) * p.chunk;
  const long long c1 = c0 + p.chunk < p.T ? c0 + p.chunk : p.T;
  griddep_wait();  // inputs written by the previous kernel are visible from here on

  auto cache_row = [&](unsigned char *cache, long long slot) {
    return cache + (slot >> p.log2_page) * p.c_sp + (slot & (p.P - 1)) * p.c_ss + h * p.c_sh + sub * A::kPieceBytes;
  };
  auto scale_at = [&](int which, long long slot) {
    return p.scales + which * p.sc_sk + (slot >> p.log2_page) * p.sc_sp + (slot & (p.P - 1)) * p.sc_ss + h * p.sc_sh +
           (KIND == KV_I4 ? sub / 4 : 0);
  };
  auto store = [&](int which, long long slot, const Piece<KIND> &r) {
    unsigned char *at = cache_row(which ? p.v_cache : p.k_cache, slot);
    if constexpr (KIND == KV_BF16) *reinterpret_cast<uint4 *>(at) = r.w;
    if constexpr (KIND == KV_I8) *reinterpret_cast<uint2 *>(at) = r.w;
    if constexpr (KIND == KV_I4) *reinterpret_cast<uint32_t *>(at) = r.w;
    if constexpr (KIND != KV_BF16)
      if (sub % (KIND == KV_I8 ? A::kLanes : 4) == 0) *scale_at(which, slot) = r.s;
  };
  // Rows t0 .. t1 of the input into their slots: first + (t - t0), or each its own (first < 0).
  auto write_rows = [&](long long t0, long long t1, long long first, Bounds *bounds) {
    constexpr int kUnroll = 4;
    for (long long t = t0 + group; __any_sync(0xffffffffu, t < t1); t += A::kRows * kUnroll) {
      uint4 kw[kUnroll], vw[kUnroll];
      long long slot[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const long long i = t + u * A::kRows;
        slot[u] = i < t1 ? (first >= 0 ? first + (i - t0) : slot_at(p, i)) : -1;
        kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (slot[u] >= 0) {
          kw[u] = __ldcs(reinterpret_cast<const uint4 *>(p.k + i * p.k_st + h * p.k_sh) + sub);
          vw[u] = __ldcs(reinterpret_cast<const uint4 *>(p.v + i * p.v_st + h * p.v_sh) + sub);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const Piece<KIND> k = A::quantise(kw[u]), v = A::quantise(vw[u]);
        if (slot[u] >= 0) {
          store(0, slot[u], k);
          store(1, slot[u], v);
          if (bounds) fold<KIND>(*bounds, k);
        }
      }
    }
  };

  if (!p.bounds) {
    write_rows(c0, c1, -1, nullptr);
    return;
  }
  // Runs that start in this CTA's tokens. Lane l looks at token w0 + l: a run starts
  // where the slot ahead is not the neighbour, or lies in another page.
  for (long long w0 = c0; w0 < c1; w0 += 32) {
    const long long i = w0 + lane;
    const long long s = i < c1 ? slot_at(p, i) : -1;
    long long ahead = __shfl_up_sync(0xffffffffu, s, 1);
    if (lane == 0) ahead = w0 > 0 ? slot_at(p, w0 - 1) : -1;
    const bool starts = s >= 0 && (ahead < 0 || ahead + 1 != s || (s & (p.P - 1)) == 0);
    unsigned todo = __ballot_sync(0xffffffffu, starts);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const long long t0 = w0 + l, first = __shfl_sync(0xffffffffu, s, l);
      const int off = static_cast<int>(first & (p.P - 1));
      const int most = p.P - off;
      // how far the run goes
      int n = 1;
      while (n < most) {
        const long long j = t0 + n + lane;
        const bool on = n + lane < most && j < p.T && slot_at(p, j) == first + n + lane;
        const unsigned stop = __ballot_sync(0xffffffffu, !on);
        const int more = stop ? __ffs(stop) - 1 : 32;
        n += more;
        if (more < 32) break;
      }
      Bounds bounds;
      bounds.clear();
      // the keys that the page holds ahead of the run
      constexpr int kUnroll = 8;
      for (int o = group; o < off; o += A::kRows * kUnroll) {
        Piece<KIND> r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int row = o + u * A::kRows;
          if (row < off) {
            const long long slot = first - off + row;
            const unsigned char *at = cache_row(p.k_cache, slot);
            if constexpr (KIND == KV_BF16) r[u].w = *reinterpret_cast<const uint4 *>(at);
            if constexpr (KIND == KV_I8) r[u].w = *reinterpret_cast<const uint2 *>(at), r[u].s = *scale_at(0, slot);
            if constexpr (KIND == KV_I4) r[u].w = *reinterpret_cast<const uint32_t *>(at), r[u].s = *scale_at(0, slot);
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (o + u * A::kRows < off) fold<KIND>(bounds, r[u]);
      }
      write_rows(t0, t0 + n, first, &bounds);
      // over the groups of a warp, then over the warps
#pragma unroll
      for (int x = A::kLanes; x < 32; x <<= 1) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          bounds.lo[c] = min_nan(bounds.lo[c], __shfl_xor_sync(0xffffffffu, bounds.lo[c], x));
          bounds.hi[c] = max_nan(bounds.hi[c], __shfl_xor_sync(0xffffffffu, bounds.hi[c], x));
        }
      }
      __syncthreads();  // the last run's partial bounds are read
      if (lane < A::kLanes) {
#pragma unroll
        for (int c = 0; c < 8; ++c) part[warp][0][8 * lane + c] = bounds.lo[c], part[warp][1][8 * lane + c] = bounds.hi[c];
      }
      __syncthreads();
      __nv_bfloat16 *to = p.bounds + (first >> p.log2_page) * p.b_sp + h * p.b_sh;
      for (int x = tid; x < 2 * D; x += kThreads) {
        const int m = x / D, c = x % D;
        float y = part[0][m][c];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) y = m ? max_nan(y, part[w][m][c]) : min_nan(y, part[w][m][c]);
        to[m * p.b_sm + c] = m ? __float2bfloat16_ru(y) : __float2bfloat16_rd(y);
      }
    }
  }
}

template <int KIND, int D>
cudaError_t launch(CacheAppendParams p, cudaStream_t stream) {
  const long long ctas = (p.T + p.chunk - 1) / p.chunk;
  return launch_step(fd_cache_append_kernel<KIND, D>, p, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(p.Hkv)),
                     kThreads, 0, 1, stream);
}

template <int KIND>
cudaError_t launch_d(int head_dim, const CacheAppendParams &p, cudaStream_t stream) {
  return head_dim == 64 ? launch<KIND, 64>(p, stream) : launch<KIND, 128>(p, stream);
}

}  // namespace

cudaError_t launch_cache_append(int kind, int head_dim, CacheAppendParams p, cudaStream_t stream) {
  // Tokens a CTA: one while all fit the GPU at once (a decode step: each its own
  // page), else 16.
  p.chunk = p.T * p.Hkv <= 152 * 16 ? 1 : 16;
  while ((p.T + p.chunk - 1) / p.chunk > 0x7fffffff) p.chunk *= 2;
  if (kind == KV_BF16) return launch_d<KV_BF16>(head_dim, p, stream);
  if (kind == KV_I8) return launch_d<KV_I8>(head_dim, p, stream);
  return launch_d<KV_I4>(head_dim, p, stream);
}

}  // namespace fd
