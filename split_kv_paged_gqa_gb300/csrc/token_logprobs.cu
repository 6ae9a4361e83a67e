// token_logprobs.cu - log probability and rank of given tokens, entropy and the
// most probable tokens of their rows (sm_103a).
//
//   lse = m + ln sum exp(x_v - m),   logprob = x_tok - lse,
//   entropy = ln l - (sum e_v z_v) / l   with z = x - m, e = exp(z), l = sum e,
//   rank = number of tokens ahead of tok in the order (value down, index up).
//
// The logits are read once, so HBM binds many rows and latency a few. A thread
// takes 16-byte pieces at a stride of the CTA, with its own running maximum, so
// that the stream needs no exchange; the sums of the threads are joined at the end
// (fp32: a thread sums a few hundred values, the tree over the threads the rest).
//
// The K largest come almost for free: with M_t the maxima of the threads (which
// the stream forms anyway) and T the K-th largest of them, at least K values are
// >= T, and all values > T lie with fewer than K threads. Only threads with M_t
// >= T are looked at again, each by its whole warp out of L2, and what is >= T
// goes into a sorted list a warp (lane i holds its i-th best as one 64-bit key of
// value and index). The warps' lists are joined by bitonic merges, the lists of a
// cluster's CTAs by its first. A row is shared by a cluster of up to 8 CTAs where
// rows are few.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fd.h"
#include "ptx.cuh"
#include "step.h"

namespace fd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCtas = 8;
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

// Sums of a part of a row, relative to its maximum m: l = sum e, w = sum e z
// (z in units of ln 2), n = tokens ahead of the given one.
struct Part {
  float m, l, w;
  int n;
};

__device__ __forceinline__ Part join(const Part &a, const Part &b) {
  Part r;
  r.m = fmaxf(a.m, b.m);
  const float base = r.m == -INFINITY ? 0.f : r.m;
  // (a part without values has m = -inf and sums 0; so has one whose values are all -inf)
  const float da = a.m == -INFINITY ? 0.f : (a.m - base) * kLog2e, db = b.m == -INFINITY ? 0.f : (b.m - base) * kLog2e;
  const float ca = exp2f(da), cb = exp2f(db);
  r.l = a.l * ca + b.l * cb;
  r.w = (a.l != 0.f ? ca * (a.w + da * a.l) : 0.f) + (b.l != 0.f ? cb * (b.w + db * b.l) : 0.f);
  r.n = a.n + b.n;
  return r;
}

__device__ __forceinline__ Part shfl_part(const Part &p, int o) {
  return {__shfl_xor_sync(0xffffffffu, p.m, o), __shfl_xor_sync(0xffffffffu, p.l, o),
          __shfl_xor_sync(0xffffffffu, p.w, o), __shfl_xor_sync(0xffffffffu, p.n, o)};
}

template <bool F32>
struct Row {
  static constexpr int kVec = F32 ? 4 : 8;  // values of a piece
  const char *base;                         // the row's first value, rounded down to 16 bytes
  int lead, V;                              // values of the first piece ahead of the row

  __device__ __forceinline__ int pieces() const { return (lead + V + kVec - 1) / kVec; }
  // Piece c; values outside the row are -inf.
  __device__ __forceinline__ void load(int c, float (&x)[kVec]) const {
    const int v0 = c * kVec - lead;
    if (v0 >= 0 && v0 + kVec <= V) {
      const uint4 w = __ldg(reinterpret_cast<const uint4 *>(base) + c);
      unpack(w, x);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int v = v0 + i;
        x[i] = -INFINITY;
        if (v >= 0 && v < V) {
          if constexpr (F32) x[i] = reinterpret_cast<const float *>(base)[lead + v];
          else x[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[lead + v]);
        }
      }
    }
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

template <bool F32>
__global__ void __launch_bounds__(kThreads, 3) fd_token_logprobs_kernel(const __grid_constant__ LogprobsParams p) {
  constexpr int kVec = Row<F32>::kVec;
  constexpr int kPieces = 16 / kVec;  // pieces a step: 16 values a thread
  __shared__ Part parts[kWarps];
  __shared__ Part cta_part;            // read by the cluster's first CTA
  __shared__ Key lists[kWarps][32];
  __shared__ Key cta_list[32];         // read by the cluster's first CTA
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = p.ctas, rank = ctas > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int64_t r = blockIdx.x / ctas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

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
  Part mine = {-INFINITY, 0.f, 0.f, 0};
  auto step = [&](const float (&x)[kVec], int c) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kVec; ++i) top = fmaxf(top, x[i]);
    if (top > mine.m) {  // (rare after the first few)
      const float d = mine.l != 0.f ? (mine.m - top) * kLog2e : 0.f, f = exp2f(d);
      mine.w = f * (mine.w + d * mine.l);
      mine.l *= f;
      mine.m = top;
    }
    const float base = mine.m == -INFINITY ? 0.f : mine.m;
    const int v0 = c * kVec - row.lead;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      // z at least -160: there e is 0, and -inf would make e z NaN (a NaN stays)
      const float z = max_nan((x[i] - base) * kLog2e, -160.f), e = fast_exp2(z);
      mine.l += e;
      mine.w = fmaf(e, z, mine.w);
      // (the index as unsigned: places ahead of the row, which read -inf, come behind)
      mine.n += x[i] > xt || (x[i] == xt && static_cast<unsigned>(v0 + i) < static_cast<unsigned>(tok));
    }
  };
  for (int c = p0 + tid; c < p1; c += kPieces * kThreads) {
    float x[kPieces][kVec];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if (c + k * kThreads < p1) row.load(c + k * kThreads, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if (c + k * kThreads < p1) step(x[k], c + k * kThreads);
    }
  }

  // ---- the K largest of this CTA's pieces
  if (p.K > 0) {
    const uint32_t mo = p0 + tid < p1 ? ordered(mine.m) : 0u;
    // the K-th largest of the threads' maxima (0 where fewer threads have a piece), bit by bit
    uint32_t t = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t to = t | 1u << bit;
      if (__syncthreads_count(mo >= to) >= p.K) t = to;
    }
    const float limit = t ? value_of(t) : -INFINITY;
    Key best = 0;
    unsigned look = __ballot_sync(0xffffffffu, mo != 0 && mo >= t);
    while (look) {
      const int l = __ffs(look) - 1;
      look &= look - 1;
      for (int c0 = p0 + warp * 32 + l; c0 < p1; c0 += 32 * kThreads) {
        const int c = c0 + lane * kThreads;  // 32 pieces of that thread, one a lane
        float x[kVec];
        const bool here = c < p1;
        if (here) row.load(c, x);
        const int v0 = c * kVec - row.lead;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          Key k = 0;
          if (here && x[i] >= limit && v0 + i >= 0 && v0 + i < row.V) k = key_of(x[i], v0 + i);
          Key worst = __shfl_sync(0xffffffffu, best, p.K - 1);
          unsigned in = __ballot_sync(0xffffffffu, k > worst);
          while (in) {
            const int s = __ffs(in) - 1;
            insert(best, __shfl_sync(0xffffffffu, k, s));
            worst = __shfl_sync(0xffffffffu, best, p.K - 1);
            if (lane == s) k = 0;
            in = __ballot_sync(0xffffffffu, k > worst);
          }
        }
      }
    }
    lists[warp][lane] = best;
    __syncthreads();
#pragma unroll 1
    for (int half = kWarps / 2; half > 0; half >>= 1) {
      if (warp < half) {
        best = merge(best, lists[warp + half][31 - lane]);
        __syncwarp();
        lists[warp][lane] = best;
      }
      __syncthreads();
    }
    if (warp == 0) cta_list[lane] = best;
  }

  // ---- sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine = join(mine, shfl_part(mine, o));
  if (lane == 0) parts[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    mine = lane < kWarps ? parts[lane] : Part{-INFINITY, 0.f, 0.f, 0};
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) mine = join(mine, shfl_part(mine, o));
    if (lane == 0) cta_part = mine;
  }
  if (ctas > 1) cluster.sync();
  if (rank == 0 && warp == 0) {
    __syncwarp();
    Part all = cta_part;
    Key best = p.K > 0 ? cta_list[lane] : 0;
    for (int c = 1; c < ctas; ++c) {
      all = join(all, *cluster.map_shared_rank(&cta_part, c));
      if (p.K > 0) best = merge(best, *cluster.map_shared_rank(&cta_list[31 - lane], c));
    }
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

cudaError_t launch_token_logprobs(LogprobsParams p, cudaStream_t stream) {
  // CTAs a row: more while all fit the GPU at once (two an SM) with 4096 values each at least.
  p.ctas = 1;
  while (p.ctas < kMaxCtas && 2ll * p.ctas * p.R <= 304 && p.V >= 2 * p.ctas * 4096) p.ctas *= 2;
  const dim3 grid(static_cast<unsigned>(p.R) * p.ctas);
  return p.f32 ? launch_step(fd_token_logprobs_kernel<true>, p, grid, kThreads, 0, p.ctas, stream)
               : launch_step(fd_token_logprobs_kernel<false>, p, grid, kThreads, 0, p.ctas, stream);
}

}  // namespace fd
