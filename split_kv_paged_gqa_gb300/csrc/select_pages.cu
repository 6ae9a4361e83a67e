// select_pages.cu - the pages of a paged cache whose bounds allow the largest
// scores, for each query token and KV head (sm_103a).
//
// A key k with lo <= k <= hi in every channel scores q . k <= sum_d max(q_d lo_d,
// q_d hi_d) = q+ . hi + q- . lo with q+ = max(q, 0), q- = min(q, 0); summed over
// the G query heads of a KV head this is Q+ . hi + Q- . lo with Q the sums of the
// heads' parts: 2 D products a page, whatever G.
//
// The choice is the one that 64-bit scores give. Scores are formed in fp32 with a
// bound on their error: the rounding of Q, 8 products with additions a lane and 5
// exchanges are off by at most 14 2^-24 of A = sum_d |Q_d| max|bound_d| (the largest of
// each channel over a warp's pages) and terms of second order; 24 are taken. With T
// the k-th largest fp32 score and E that bound, pages above T + 2 E belong to the
// choice and pages below T - 2 E do not; only those between (mostly none but the
// border page itself) are scored again in fp64 (Q as the sum of two fp32 words, the
// products exact), and ranked, ties to the lowest page. The fp64 pipe (about two
// operations a clock and SM) takes 1.7 ms for all pages of 64 requests of 1024 x 8
// heads; this way it sees a few.
//
// A page's bounds (4 D bytes a head) are read once: HBM binds a batch, latency one
// request. A cluster of CTAs scores one request and head, a warp 8 pages at a time
// (a lane 16 bytes of each), and its first CTA chooses: the scores stand in its
// shared memory, T is found by linear histograms (1024 bins over the range, then
// over the bin that holds it, until 32 scores are left to rank). 64 requests of
// 256-1024 pages x 8 heads take 43 us (4.0 TB/s; the same loads without a product
// 35), one of 2048 pages x 8 heads 9.9 us (launch and first loads 3.2, scores 2.2,
// choice 4.5).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fd.h"
#include "ptx.cuh"
#include "step.h"

namespace fd {
namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 1024;
constexpr int kMaxRanks = 8;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Whole numbers in the order of the values; a NaN above all.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  if (x != x) return ~0ull;
  const unsigned long long u = __double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum over the block, and exclusive prefix sum.
template <int kWarps>
__device__ __forceinline__ int block_sum(int v, int *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < kWarps ? sums[lane] : 0);
}
template <int kWarps>
__device__ __forceinline__ int block_scan(int v, int *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  const int before = __reduce_add_sync(0xffffffffu, lane < warp && lane < kWarps ? sums[lane] : 0);
  return before + incl - v;
}

// Shared memory of a CTA. Behind it, for W pages: keys (64-bit scores of border
// pages), scores, and the border pages' indices.
struct alignas(16) Smem {
  float q[2][128], q_low[2][128];  // Q-, Q+ and what their rounding left
  unsigned hist[kBins];
  int sums[32];
  unsigned lo, hi;           // range of the scores under search, ordered
  int nans, numbers;
  unsigned most;             // A, the largest of the warps'; a NaN is above all (its bits)
  float few[32];
  int count, bin, above, on;
};

constexpr size_t smem_bytes(size_t W) { return (sizeof(Smem) + (8 + 4 + 2) * W + 15) / 16 * 16; }  // key, score, index

template <int D, int kThreads, int kCtas = 1024 / kThreads>
__global__ void __launch_bounds__(kThreads, kCtas) fd_select_pages_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kLanes = D / 4;            // lanes a page: half of them the lower bounds, half the upper
  constexpr int kAt = 32 / kLanes;         // pages a warp loads at once
  constexpr int kUnroll = 8, kPages = kAt * kUnroll;
  extern __shared__ __align__(16) unsigned char raw[];
  Smem &s = *reinterpret_cast<Smem *>(raw);
  static_assert(sizeof(Smem) % 8 == 0, "keys are 8-byte aligned");
  auto *keys = reinterpret_cast<unsigned long long *>(raw + sizeof(Smem));
  float *scores = reinterpret_cast<float *>(keys + p.W);
  auto *border = reinterpret_cast<unsigned short *>(scores + p.W);
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = p.ranks, rank = ranks > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int unit = blockIdx.x / ranks;
  const int t = unit % p.Tq;
  unit /= p.Tq;
  const int h = unit % p.Hkv, b = unit / p.Hkv;
  int *out = p.selected + b * p.s_sb + t * p.s_st + h * p.s_sh;

  griddep_wait();  // inputs written by the previous kernel are visible from here on
  // what the first steps need, all under way at once: the length, the first 8 heads' channel
  int L = p.seqlens[b * p.sl_s];
  const __nv_bfloat16 *qc = p.q + b * p.q_sb + t * p.q_st + static_cast<int64_t>(h) * p.G * p.q_sh + tid % D;
  float heads[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) heads[g] = tid < D && g < p.G ? __bfloat162float(qc[g * p.q_sh]) : 0.f;
  const int *table = p.page_table + b * p.pt_sb + p.first;
  const long long cap = static_cast<long long>(p.W) * p.P;
  if (L < 0 || L > cap) {
    if (tid == 0 && rank == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_SEQLEN_OVERFLOW);
    L = L < 0 ? 0 : static_cast<int>(cap);
  }
  const int visible = max(0, L - (p.Tq - 1) + t), n = (visible + p.P - 1) / p.P;
  if (n <= p.S) {  // no choice (every CTA of the cluster returns)
    if (rank == 0)
      for (int i = tid; i < p.S; i += kThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int first = p.first, m = n - p.first - p.last;  // the pages that are chosen among: first .. first + m
  const int k = p.S - p.first - p.last;                 // how many (k < m)
  if (tid == 0) s.lo = 0xffffffffu, s.hi = 0u, s.nans = s.numbers = s.on = 0, s.most = 0u;
  for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
  if (ranks > 1) cluster.sync();  // the first CTA runs: its shared memory can be written

  if (k > 0) {
    const int per = ((m + ranks - 1) / ranks + kPages - 1) / kPages * kPages;
    const int i0 = min(m, rank * per), i1 = min(m, i0 + per);
    int a = i0 + warp * kPages;
    int next_id = lane < kPages && a + lane < i1 ? table[a + lane] : -1;
    // ---- Q
    if (tid < D) {
      // sums of two words: s + v = t + e exactly (Knuth)
      float hi[2] = {0.f, 0.f}, low[2] = {0.f, 0.f};
      for (int g0 = 0; g0 < p.G; g0 += 8) {
        if (g0 > 0) {
#pragma unroll
          for (int g = 0; g < 8; ++g) heads[g] = g0 + g < p.G ? __bfloat162float(qc[(g0 + g) * p.q_sh]) : 0.f;
        }
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          // (comparisons, so that a NaN query makes NaN sums)
          const float v[2] = {heads[g] > 0.f ? 0.f : heads[g], heads[g] < 0.f ? 0.f : heads[g]};
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float sum = hi[x] + v[x], back = sum - hi[x];
            low[x] += (hi[x] - (sum - back)) + (v[x] - back);
            hi[x] = sum;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float sum = hi[x] + low[x];  // the words' sum rounded, and what that leaves
        s.q[x][tid] = sum;
        s.q_low[x][tid] = low[x] - (sum - hi[x]);
      }
    }
    __syncthreads();
    // ---- scores: a lane's 8 channels of the lower or the upper bounds
    const int side = (lane % kLanes) / (kLanes / 2), sub = lane % (kLanes / 2);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = s.q[side][8 * sub + i];
    float *to = ranks > 1 ? cluster.map_shared_rank(scores, 0) : scores;
    Smem *lead = ranks > 1 ? cluster.map_shared_rank(&s, 0) : &s;
    uint32_t most[4] = {0u, 0u, 0u, 0u};  // largest magnitudes of the channels, bf16 pairs
    const __nv_bfloat16 *bounds = p.bounds + h * p.b_sh + side * p.b_sm + 8 * sub;
    unsigned lo = 0xffffffffu, hi = 0u;
    int nans = 0, numbers = 0;
    for (; a < i1; a += kWarps * kPages) {
      // page ids of these kPages pages, one a lane (-1 past the last: such lanes load nothing, so that A knows this choice's pages only)
      int id = next_id;
      const bool in = lane < kPages && a + lane < i1;
      const int a2 = a + kWarps * kPages;
      next_id = lane < kPages && a2 + lane < i1 ? table[a2 + lane] : -1;
      const bool bad = in && (id < 0 || id >= p.num_pages);
      if (__any_sync(0xffffffffu, bad) && lane == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
      if (bad) id = -1;
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int page = __shfl_sync(0xffffffffu, id, u * kAt + lane / kLanes);
        w[u] = make_uint4(0u, 0u, 0u, 0u);
        if (page >= 0) w[u] = __ldg(reinterpret_cast<const uint4 *>(bounds + page * p.b_sp));
      }
      float v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sum = fmaf(q[2 * c], bf16_lo(x[c]), sum);
          sum = fmaf(q[2 * c + 1], bf16_hi(x[c]), sum);
          asm("{.reg .b32 t;\n\tand.b32 t, %1, 0x7fff7fff;\n\tmax.bf16x2 %0, %0, t;}" : "+r"(most[c]) : "r"(x[c]));
        }
        v[u] = sum;
      }
      // over the lanes of a page: halves of the pages are exchanged, so 8 sums take 7 shuffles, then single ones
#pragma unroll
      for (int o = 4, x = kLanes / 2; o > 0; o >>= 1, x >>= 1) {
        const bool up = lane & x;
#pragma unroll
        for (int u = 0; u < o; ++u) {
          const float give = up ? v[u] : v[u + o], keep = up ? v[u + o] : v[u];
          v[u] = keep + __shfl_xor_sync(0xffffffffu, give, x);
        }
      }
#pragma unroll
      for (int x = kLanes / 16; x > 0; x >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], x);
      // which page this lane holds: bits of the lane from kLanes / 2 down to kLanes / 8
      const int u = (lane & (kLanes / 2) ? 4 : 0) + (lane & (kLanes / 4) ? 2 : 0) + (lane & (kLanes / 8) ? 1 : 0);
      const int i = u * kAt + lane / kLanes;
      const bool gone = __shfl_sync(0xffffffffu, id, i) < 0;
      // (a NaN as +inf, which no number is while A is finite; a page out of range as -inf)
      if (lane % (kLanes / 8) == 0 && a + i < i1) {
        const float x = gone ? -INFINITY : (v[0] == v[0] ? v[0] : INFINITY);
        to[a + i] = x;
        nans += x == INFINITY;
        if (fabsf(x) < INFINITY) {
          ++numbers;
          lo = min(lo, ordered(x));
          hi = max(hi, ordered(x));
        }
      }
    }
    // A: a warp's sum bounds those of its pages. (Rounded upwards, it is 0 only if all products are.)
    float A = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      A = __fmaf_ru(fabsf(q[2 * c]), bf16_lo(most[c]), __fmaf_ru(fabsf(q[2 * c + 1]), bf16_hi(most[c]), A));
#pragma unroll
    for (int x = kLanes / 2; x > 0; x >>= 1) A += __shfl_xor_sync(0xffffffffu, A, x);
    if (kAt > 1) A = max_nan(A, __shfl_xor_sync(0xffffffffu, A, 16));
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    nans = __reduce_add_sync(0xffffffffu, nans);
    numbers = __reduce_add_sync(0xffffffffu, numbers);
    if (lane == 0) {
      atomicMax(&lead->most, __float_as_uint(A) & 0x7fffffffu);  // (A >= 0: its bits are in order, a NaN's the largest)
      atomicMin(&lead->lo, lo);
      atomicMax(&lead->hi, hi);
      if (nans) atomicAdd(&lead->nans, nans);
      atomicAdd(&lead->numbers, numbers);
    }
  }
  if (ranks > 1) {
    cluster.sync();  // the scores stand in the first CTA's shared memory
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  int need = 0;  // how many of the pages marked kMaybe belong to the choice: the first of them
  constexpr float kYes = INFINITY, kMaybe = 0.f, kNo = -INFINITY;
  if (k > 0) {
    const float A = __uint_as_float(s.most);
    const float E2 = 2.f * 24.f * 0x1p-24f * A;
    // else sums may have overflowed, or products lost places below the smallest numbers: all pages in fp64
    const bool finite = A == 0.f || (A < 1e38f && A >= 0x1p-80f);
    // pages by class: +inf stands for a NaN score, -inf for a page id out of range
    const int nans = s.nans, numbers = s.numbers;
    if (finite && (nans >= k || nans + numbers <= k)) {
      // no border among numbers: the first of the NaNs, or all numbers and the first of the pages out of range
      const bool all = nans < k;
      need = all ? k - nans - numbers : k;
      for (int i = tid; i < m; i += kThreads) {
        const float x = scores[i];
        scores[i] = all ? (x == -INFINITY ? kMaybe : kYes) : (x == INFINITY ? kMaybe : kNo);
      }
    } else {
      float T = 0.f;
      if (finite) {
        // ---- the kk-th largest number
        int kk = k - nans;
        for (bool fresh = true;; fresh = false) {
          const float lo = value_of(s.lo), hi = value_of(s.hi);
          T = lo;
          if (lo == hi) break;
          const float scale = kBins / (hi - lo);
          auto bin_of = [&](float x) { return min(kBins - 1, static_cast<int>((x - lo) * scale)); };
          if (!fresh) {  // (the first time the bins are zero from the start)
            for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
            __syncthreads();
          }
          for (int i = tid; i < m; i += kThreads) {
            const float x = scores[i];
            if (x >= lo && x <= hi) atomicAdd(&s.hist[bin_of(x)], 1u);
          }
          __syncthreads();
          // bins from the top: kBins / kThreads neighbours a thread
          constexpr int kMine = kBins / kThreads;
          const int top = kBins - 1 - kMine * tid;
          int sum = 0;
#pragma unroll
          for (int i = 0; i < kMine; ++i) sum += s.hist[top - i];
          int before = block_scan<kWarps>(sum, s.sums);
          if (before < kk && before + sum >= kk) {
            int i = 0;
            while (before + static_cast<int>(s.hist[top - i]) < kk) before += s.hist[top - i++];
            s.bin = top - i;
            s.above = before;
            s.count = 0;
          }
          if (tid == 0) s.lo = 0xffffffffu, s.hi = 0u;  // (read by all ahead of the scan)
          __syncthreads();
          const int bin = s.bin, left = s.hist[bin];
          kk -= s.above;
          if (left <= 32) {  // few enough to rank, by every warp for itself
            for (int i = tid; i < m; i += kThreads) {
              const float x = scores[i];
              if (x >= lo && x <= hi && bin_of(x) == bin) s.few[atomicAdd(&s.count, 1)] = x;
            }
            __syncthreads();
            const float x = lane < left ? s.few[lane] : -INFINITY;
            int ahead = 0;
            for (int j = 0; j < left; ++j) ahead += s.few[j] > x || (s.few[j] == x && j < lane);
            T = __shfl_sync(0xffffffffu, x, __ffs(__ballot_sync(0xffffffffu, lane < left && ahead == kk - 1)) - 1);
            break;
          }
          for (int i = tid; i < m; i += kThreads) {
            const float x = scores[i];
            if (x >= lo && x <= hi && bin_of(x) == bin) atomicMin(&s.lo, ordered(x)), atomicMax(&s.hi, ordered(x));
          }
          __syncthreads();
        }
      }
      // ---- pages above the border, on it and below
      const float up = T + E2, down = T - E2;
      int above = 0;
      for (int i = tid; i < m; i += kThreads) {
        const float x = scores[i];
        if (finite && x > up) {
          ++above;
          scores[i] = kYes;
        } else if (finite && x < down) {
          scores[i] = kNo;
        } else {
          border[atomicAdd(&s.on, 1)] = static_cast<unsigned short>(i);
          scores[i] = kMaybe;
        }
      }
      need = k - block_sum<kWarps>(above, s.sums);
      const int on = s.on;
      if (need < on && A != 0.f) {  // (with A = 0 all scores are 0: the first pages)
        // ---- the border in fp64
        auto q_exact = [&](int side, int d) {
          const float hi = s.q[side][d];
          if (fabsf(hi) < INFINITY) return static_cast<double>(hi) + static_cast<double>(s.q_low[side][d]);
          double sum = 0.0;  // no number, or past fp32
          for (int g = 0; g < p.G; ++g) {
            const float v = __bfloat162float(p.q[b * p.q_sb + t * p.q_st + (static_cast<int64_t>(h) * p.G + g) * p.q_sh + d]);
            sum += side ? (v < 0.f ? 0.f : v) : (v > 0.f ? 0.f : v);
          }
          return sum;
        };
        auto *exact = reinterpret_cast<double *>(s.hist);
        for (int x = tid; x < 2 * D; x += kThreads) exact[x] = q_exact(x / D, x % D);
        __syncthreads();
        for (int e = warp; e < on; e += kWarps) {
          const int id = p.page_table[b * p.pt_sb + first + border[e]];
          const bool bad = id < 0 || id >= p.num_pages;
          double sum = 0.0;
          if (!bad) {
            const __nv_bfloat16 *at = p.bounds + id * p.b_sp + h * p.b_sh;
#pragma unroll
            for (int x = lane; x < 2 * D; x += 32)
              sum = fma(exact[x], static_cast<double>(__bfloat162float(at[(x / D) * p.b_sm + x % D])), sum);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane == 0) keys[e] = bad ? 0ull : ordered(sum);
        }
        __syncthreads();
        if (on > 512) {
          // many (equal pages, no fp32 scores): ranking takes on * on steps, a search for the need-th largest 64 on
          unsigned long long key = 0;
          for (unsigned long long bit = 1ull << 63; bit; bit >>= 1) {
            int at_least = 0;
            for (int e = tid; e < on; e += kThreads) at_least += keys[e] >= (key | bit);
            if (block_sum<kWarps>(at_least, s.sums) >= need) key |= bit;
          }
          above = 0;
          for (int e = tid; e < on; e += kThreads) {
            above += keys[e] > key;
            scores[border[e]] = keys[e] > key ? kYes : (keys[e] == key ? kMaybe : kNo);
          }
          need -= block_sum<kWarps>(above, s.sums);
        } else {
          for (int e = tid; e < on; e += kThreads) {
            const unsigned long long mine = keys[e];
            const int i = border[e];
            int ahead = 0;
            for (int j = 0; j < on; ++j) ahead += keys[j] > mine || (keys[j] == mine && border[j] < i);
            scores[i] = ahead < need ? kYes : kNo;
          }
        }
      }
    }
    __syncthreads();
  }

  // ---- the list, pages upwards: a thread takes neighbours
  for (int i = tid; i < p.first; i += kThreads) out[i] = i;
  for (int i = tid; i < p.last; i += kThreads) out[p.first + k + i] = n - p.last + i;
  if (k > 0) {
    const int per = (m + kThreads - 1) / kThreads, a = min(m, tid * per), z = min(m, a + per);
    int yes = 0, maybe = 0;
    for (int i = a; i < z; ++i) {
      yes += scores[i] == kYes;
      maybe += scores[i] == kMaybe;
    }
    // both counts in one sum (each below 2^15)
    const int ahead = block_scan<kWarps>(yes | maybe << 16, s.sums);
    int maybe_left = max(0, need - (ahead >> 16));  // ties that this thread may still take
    int at = (ahead & 0xffff) + min(ahead >> 16, need);
    for (int i = a; i < z; ++i) {
      const float x = scores[i];
      const bool in = x == kYes || (x == kMaybe && maybe_left-- > 0);
      if (in) out[first + at++] = first + i;
    }
  }
}

template <int D, int kThreads, int kCtas = 1024 / kThreads>
cudaError_t launch(const SelectParams &p, cudaStream_t stream) {
  // the kernel's limit of shared memory, once a device
  static std::atomic<unsigned long long> ready{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (device & 63);
  if (device > 63 || !(ready.load() & bit)) {
    e = cudaFuncSetAttribute(fd_select_pages_kernel<D, kThreads, kCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem_bytes(kSelectMaxPages)));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  return launch_step(fd_select_pages_kernel<D, kThreads, kCtas>, p, dim3(static_cast<unsigned>(p.B) * p.Tq * p.Hkv * p.ranks), kThreads,
                     smem_bytes(p.W), p.ranks, stream);
}

template <int kThreads, int kCtas = 1024 / kThreads>
cudaError_t launch_d(int head_dim, const SelectParams &p, cudaStream_t stream) {
  return head_dim == 64 ? launch<64, kThreads, kCtas>(p, stream) : launch<128, kThreads, kCtas>(p, stream);
}

}  // namespace

cudaError_t launch_select_pages(int head_dim, SelectParams p, cudaStream_t stream) {
  const long long units = static_cast<long long>(p.B) * p.Tq * p.Hkv;
  const size_t held = 228 * 1024 / (smem_bytes(p.W) + 1024);  // CTAs whose shared memory an SM holds
  p.ranks = 1;
  // Choices of which CTAs of 512 threads (two an SM) would not fit the GPU at once: small CTAs, as many an SM as its memory
  // holds, and two a choice while these fit. 64 requests of 256-1024 pages x 8 heads take 42.9 us; one CTA of 128 / 256 / 512
  // threads 51.7 / 45.5 / 46.4, four of 128 46.3. 300 of 2048 pages x 8 heads: 256 threads 338 us, 512 351, 128 390.
  if (units > 304 && held >= 8) {
    if (2 * units <= 1216 && p.W >= 256) p.ranks = 2;
    return launch_d<128>(head_dim, p, stream);
  }
  if (units > 304 && held >= 4) return launch_d<256>(head_dim, p, stream);
  // CTAs of 512 threads, more a choice while all fit at once with 64 pages each at least: 4 x 15360 pages x 8 heads 65.7 us
  // with four, 92 with eight; 512 pages x 8 heads 6.6 with eight, 7.3 with four. One that has an SM to itself may use more
  // registers: 2048 pages x 8 heads 9.9 us, 10.2 without; 64 x 8192 383 us, 475 without, 1113 in CTAs of 128 threads.
  while (p.ranks < kMaxRanks && 2 * p.ranks * units <= (held >= 2 ? 304 : 152) && p.W >= 2 * p.ranks * 64) p.ranks *= 2;
  if (held < 2 || units * p.ranks <= 152) return launch_d<512, 1>(head_dim, p, stream);
  return launch_d<512>(head_dim, p, stream);
}

}  // namespace fd
