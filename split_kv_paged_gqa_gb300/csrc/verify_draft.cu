// verify_draft.cu - verification of drafted tokens (sm_103a).
//
// Drafted token x_i (i = 0, 1, ...) is accepted while u_i * q_i(x_i) < p_i(x_i),
// p the target's and q the draft's probability. At the first refusal n the step
// ends with a sample from w(v) = max(p_n(v) - q_n(v), 0); with every draft
// accepted it ends with a sample from the target's row behind them. The sample
// is the lowest v whose cumulative weight exceeds u_K times the row's total.
//
// One row of p (and after a refusal one of q) per request is all that has to be
// read, so HBM binds a large batch and latency a small one. A cluster of CTAs
// takes a request, each a contiguous range of the vocabulary: one pass sums the
// range in segments, the CTAs' totals are exchanged through distributed shared
// memory (no workspace, no atomics: a call's result depends on nothing but its
// inputs), and the CTA whose range holds the sample reads the one segment that
// holds it again.
//
// Arithmetic: acceptance compares in 64 bits, where the product of two fp32
// values is exact. A weight p - q with p > q is held as an exact pair of fp32
// values (d = p - q rounded, e = (p - d) - q), and pairs are summed with an
// error-free transformation (Knuth's two-sum, the errors in a second word):
// about 46 bits for 12 fp32 operations a token. The fp64 pipe (about two
// operations a clock and SM) would need 230 us for 256 rows of 131072, and 5 us
// for one prefix sum over 512 threads.
#include <cooperative_groups.h>

#include <type_traits>

#include "fd.h"
#include "latent.h"
#include "ptx.cuh"

namespace fd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kStep = 512;      // tokens that a warp loads at once: four 16-byte loads a lane and row
constexpr int kMaxSegs = 1024;  // segments of a CTA's range

struct Pair {  // an unevaluated sum hi + lo
  float hi, lo;
};

__device__ __forceinline__ Pair add_pair(Pair a, float hi, float lo) {
  const float s = a.hi + hi, b = s - a.hi;
  const float err = (a.hi - (s - b)) + (hi - b);  // a.hi + hi = s + err exactly
  return {s, a.lo + (err + lo)};
}

// a + b with the second word brought below half a unit of the first
__device__ __forceinline__ Pair join(Pair a, Pair b) {
  const Pair t = add_pair(a, b.hi, b.lo);
  const float s = t.hi + t.lo;
  return {s, t.lo - (s - t.hi)};
}

__device__ __forceinline__ bool above(Pair a, Pair b) {  // a > b
  const Pair d = add_pair(a, -b.hi, -b.lo);
  return d.hi + d.lo > 0.f;
}

// a * u to about 47 bits
__device__ __forceinline__ Pair times(Pair a, float u) {
  const float hi = a.hi * u;
  return join({hi, 0.f}, {fmaf(a.hi, u, -hi), a.lo * u});
}

__device__ __forceinline__ bool positive(Pair a) { return a.hi + a.lo > 0.f; }

// max(p - q, 0) exactly; NaN counts as 0
__device__ __forceinline__ Pair weight_of(float p, float q) {
  const bool pos = p > q;
  const float d = p - q, e = (p - d) - q;  // exact for p >= q >= 0
  return {pos ? d : 0.f, pos ? e : 0.f};
}

__device__ __forceinline__ Pair add_weight(Pair a, float p, float q) {
  const Pair w = weight_of(p, q);
  return add_pair(a, w.hi, w.lo);
}

// A weight times a power of two. Down, a bit that would be lost stays: a token with
// any weight can be the sample.
__device__ __forceinline__ Pair scaled(Pair w, float scale) {
  return {w.hi > 0.f ? fmaxf(w.hi * scale, 0x1p-149f) : 0.f, w.lo * scale};
}

__device__ __forceinline__ long long token_at(const VerifyParams &p, int b, int i) {
  const int64_t at = b * p.x_sb + i * p.x_sk;
  return p.tok64 ? static_cast<const long long *>(p.tokens)[at] : static_cast<const int *>(p.tokens)[at];
}

__device__ __forceinline__ Pair shfl_up_pair(Pair v, int o) {
  return {__shfl_up_sync(0xffffffffu, v.hi, o), __shfl_up_sync(0xffffffffu, v.lo, o)};
}

// Inclusive prefix sum over the block's threads; sums: a word per warp, and the
// block's total behind them.
__device__ __forceinline__ Pair block_scan(Pair v, Pair *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair up = shfl_up_pair(v, o);
    if (lane >= o) v = join(up, v);
  }
  __syncthreads();  // earlier readers of sums are through
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    Pair t = lane < kWarps ? sums[lane] : Pair{0.f, 0.f};
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const Pair up = shfl_up_pair(t, o);
      if (lane >= o) t = join(up, t);
    }
    if (lane < kWarps) sums[lane] = t;
  }
  __syncthreads();
  return warp ? join(sums[warp - 1], v) : v;
}

__global__ void __launch_bounds__(kThreads, 2) fd_verify_draft_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ Pair seg_sum[kMaxSegs];
  __shared__ Pair sums[kWarps];
  __shared__ Pair range_total;  // read by the cluster's other CTAs
  __shared__ Pair seg_start;
  __shared__ int accepted, first_seg, last_seg, first_hit, last_positive;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = p.ranks, rank = ranks > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int b = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  griddep_wait();               // inputs written by the previous kernel are visible from here on
  // ---- how many drafted tokens stand: a lane a position, two for K > 32
  if (warp == 0) {
    int count = p.K;
    if (p.num_draft) {
      count = p.num_draft[b * p.n_s];
      if (count < 0 || count > p.K) {
        if (lane == 0 && rank == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_BAD_TOKEN);
        count = count < 0 ? 0 : p.K;
      }
    }
    int n = 0;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      bool good = false, bad_token = false;
      if (i < count) {
        const long long x = token_at(p, b, i);
        bad_token = x < 0 || x >= p.V;
        if (!bad_token) {
          const double u = p.u[b * p.u_sb + i * p.u_sk];
          const double q = p.draft ? static_cast<double>(p.draft[b * p.d_sb + i * p.d_sk + x]) : 1.0;
          good = u * q < static_cast<double>(p.target[b * p.t_sb + i * p.t_sk + x]);
        }
      }
      const unsigned ok = __ballot_sync(0xffffffffu, good), bad = __ballot_sync(0xffffffffu, bad_token);
      const int run = __ffs(~ok) - 1;  // accepted in a row (-1: all 32)
      n = i0 + (run < 0 ? 32 : run);
      // a bad token is recorded where the walk meets it
      if (run >= 0 && ((bad >> run) & 1u) && lane == 0 && rank == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_BAD_TOKEN);
      if (run >= 0) break;
    }
    if (n > count) n = count;
    if (lane == 0) {
      accepted = n | (n < count ? 0x10000 : 0);
      first_seg = first_hit = 0x7fffffff;
      last_seg = last_positive = -1;
    }
  }
  __syncthreads();
  const int n = accepted & 0xffff;
  bool refused = accepted & 0x10000;
  const float *tr = p.target + b * p.t_sb + n * p.t_sk;
  const float *dr = refused && p.draft ? p.draft + b * p.d_sb + n * p.d_sk : nullptr;
  long long gone = -1;  // without draft probabilities: the refused token, which carries no weight
  if (refused && !p.draft) gone = token_at(p, b, n);

  // ---- this CTA's range, in segments
  const int v0 = min(p.V, rank * p.range), v1 = min(p.V, v0 + p.range);
  const int nseg = (v1 - v0 + p.seg - 1) / p.seg;
  int hit = -1;       // the sample, in the CTA that holds it
  bool last_try = !refused;
  // Pairs hold sums from 2^-60 to the largest fp32 number to 46 bits. A row whose
  // sum lies outside is summed again with its weights scaled (exactly, but for
  // bits below 2^-85 beside a sum above 2^127).
  float scale = 1.f;
  enum { kDone, kNone, kScale };  // the sample is found (maybe by another CTA); no weight; a sum to be scaled
  // (Two copies of the pass: a scale that may change costs the usual one 1-2 %.)
  auto pass = [&](auto how) -> int {
    constexpr bool as_is = decltype(how)::value;
    auto weight = [&](int v) {
      const Pair x = v == gone ? Pair{0.f, 0.f} : weight_of(tr[v], dr ? dr[v] : 0.f);
      return as_is ? x : scaled(x, scale);
    };
    const bool vec = (reinterpret_cast<uintptr_t>(tr) & 15) == 0 && (!dr || (reinterpret_cast<uintptr_t>(dr) & 15) == 0);
    for (int s = warp; s < nseg; s += kWarps) {
      const int a = v0 + s * p.seg, z = min(v1, a + p.seg);
      Pair sum = {0.f, 0.f};
      for (int c = a; c < z && as_is; c += kStep) {
        float tv[16], dv[16];
        if (vec && c + kStep <= z) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4 *>(tv + 4 * k) = __ldcs(reinterpret_cast<const float4 *>(tr + c + 128 * k) + lane);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4 *>(dv + 4 * k) =
                dr ? __ldcs(reinterpret_cast<const float4 *>(dr + c + 128 * k) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
          if (gone >= c && gone < c + kStep) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (c + 128 * (k >> 2) + 4 * lane + (k & 3) == gone) tv[k] = 0.f;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int v = c + 32 * k + lane;
            tv[k] = v < z && v != gone ? tr[v] : 0.f;
            dv[k] = dr && v < z ? dr[v] : 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) sum = add_weight(sum, tv[k], dv[k]);
      }
#pragma unroll 1
      for (int v = a + lane; v < z && !as_is; v += 32) {
        const Pair w = weight(v);
        sum = add_pair(sum, w.hi, w.lo);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Pair up = {__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)};
        sum = join(sum, up);
      }
      if (lane == 0) seg_sum[s] = sum;
    }
    __syncthreads();
    // prefix sums of the segments: two a thread
    const Pair none = {0.f, 0.f};
    const Pair s0 = 2 * tid < nseg ? seg_sum[2 * tid] : none, s1 = 2 * tid + 1 < nseg ? seg_sum[2 * tid + 1] : none;
    const Pair two = join(s0, s1);
    Pair incl = block_scan(two, sums);
    Pair before = none, total = sums[kWarps - 1];
    const float u = p.u[b * p.u_sb + p.K * p.u_sk];
    int owner = 0;
    if (ranks > 1) {
      if (tid == 0) range_total = total;
      cluster.sync();
      Pair t[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) t[r] = r < ranks ? *cluster.map_shared_rank(&range_total, r) : none;
      cluster.sync();  // every CTA has read
      total = none;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r == rank) before = total;
        total = join(total, t[r]);
      }
      // The CTA whose range holds the sample: the first whose end exceeds the
      // goal (the last with any weight, should none: u out of [0, 1)). Every CTA
      // finds the same one from the same sums.
      const Pair goal = times(total, u);
      Pair end = none;
      int last = 0;
      owner = -1;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        end = join(end, t[r]);
        if (positive(t[r])) {
          last = r;
          if (owner < 0 && above(end, goal)) owner = r;
        }
      }
      if (owner < 0) owner = last;
    }
    if (as_is) {
      const float t = total.hi + total.lo;
      if (!(t <= 0x1.fffffep127f)) scale = 0x1p-64f;  // (infinite, or NaN from infinities)
      else if (t > 0.f && t < 0x1p-60f) scale = 0x1p64f;
      if (scale != 1.f) return kScale;
    }
    if (!positive(total) && !last_try) return kNone;
    if (positive(total) && owner == rank) {
      // its first segment whose end exceeds the goal (a rounding of the sums may
      // leave none: its last with weight)
      const Pair goal = times(total, u);
      incl = join(before, incl);
      const Pair begin = join(incl, {-two.hi, -two.lo});
      const Pair mid = join(begin, s0);
      if (positive(s0)) {
        atomicMax(&last_seg, 2 * tid);
        if (above(mid, goal)) atomicMin(&first_seg, 2 * tid);
      }
      if (positive(s1)) {
        atomicMax(&last_seg, 2 * tid + 1);
        if (above(incl, goal)) atomicMin(&first_seg, 2 * tid + 1);
      }
      __syncthreads();
      const int f = first_seg != 0x7fffffff ? first_seg : last_seg;
      if (tid == f / 2) seg_start = (f & 1) ? mid : begin;
      // its tokens again: contiguous pieces, one a thread
      const int a = v0 + f * p.seg, z = min(v1, a + p.seg);
      const int piece = (z - a + kThreads - 1) / kThreads, c0 = min(z, a + tid * piece), c1 = min(z, c0 + piece);
      Pair w = none;
      int last = -1;
      for (int v = c0; v < c1; ++v) {
        const Pair x = weight(v);
        w = join(w, x);
        if (x.hi > 0.f) last = v;
      }
      Pair end = block_scan(w, sums);  // (its barriers publish seg_start)
      end = join(seg_start, end);
      if (last >= 0) {
        atomicMax(&last_positive, last);
        if (above(end, goal)) {
          Pair acc = join(end, {-w.hi, -w.lo});
          for (int v = c0; v < c1; ++v) {
            const Pair x = weight(v);
            acc = join(acc, x);
            if (x.hi > 0.f && (above(acc, goal) || v == last)) {
              atomicMin(&first_hit, v);
              break;
            }
          }
        }
      }
      __syncthreads();
      hit = first_hit != 0x7fffffff ? first_hit : last_positive;
    }
    if (!positive(total) && rank == 0) hit = p.V - 1;  // no weight at all
    return kDone;
  };
  while (true) {
    int end = pass(std::true_type{});
    if (end == kScale) end = pass(std::false_type{});
    if (end == kDone) break;
    last_try = true;  // p <= q everywhere: the target's row as it is
    dr = nullptr;
    gone = -1;
    scale = 1.f;
  }
  if (hit < 0) return;
  for (int i = tid; i <= p.K; i += kThreads)
    p.out[b * p.o_sb + i] = i < n ? static_cast<int>(token_at(p, b, i)) : (i == n ? hit : -1);
  if (tid == 0) p.emitted[b] = n + 1;
}

}  // namespace

cudaError_t launch_verify_draft(VerifyParams p, cudaStream_t stream) {
  // CTAs a request, a portable cluster at most: one an SM (152) with 4096 tokens
  // each at least, up to 256 (two an SM) with 32768 each. Measured in loops (us, 1 /
  // 2 / 4 / 8 CTAs): 1 x 32000 8.8 / 8.5 / 7.2 / 7.1, 8 x 131072 20.6 / 14.3 / 10.5 /
  // 8.8, 33 x 50021 14.1 / 11.2 / 9.0 / 10.6, 64 x 131072 23.4 / 15.7 / 15.3 / 21.7,
  // 128 x 131072 27.4 / 23.3 / 29.6 / 41.7, 128 x 32000 9.3 / 11.4 / 17.3 / 30.4, 160
  // x 131072 35.2 / 36.7 / 38.8 / 51.1.
  p.ranks = 1;
  auto fits = [&](int64_t ranks) {
    return (ranks * p.B <= 152 && p.V >= ranks * 4096) || (ranks * p.B <= 256 && p.V >= ranks * 32768);
  };
  while (p.ranks < 8 && fits(2 * p.ranks)) p.ranks *= 2;
  p.range = (p.V + p.ranks - 1) / p.ranks;
  p.range = (p.range + kStep - 1) / kStep * kStep;
  p.seg = ((p.range + kMaxSegs - 1) / kMaxSegs + kStep - 1) / kStep * kStep;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fd_verify_draft_kernel, p);
}

}  // namespace fd
