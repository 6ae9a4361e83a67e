// append_slots.cu - pages and cache slots of a step's new tokens (sm_103a).
//
// Request b holds L_b keys on ceil(L_b / P) pages and gets n_b more. It needs
//   need_b = ceil((L_b + n_b) / P) - ceil(L_b / P)
// pages; with e_b the sum of need over the requests up to b, it takes the free
// pages e_b - need_b .. e_b - 1 if there are so many, and none otherwise. (Ends
// only grow, so every request behind the first that fails and needs a page fails
// too, and nothing has to be known of one request to serve another.)
//
// A call moves a few words a request and 8 to 12 bytes a token, so launch and
// load latency bind it. Every CTA of 1024 threads forms the prefix sums of all
// requests itself, 1024 at a time (two block scans over what is in L2 after the
// first CTA), and then writes its own 1024 tokens, each found by bisection: one
// launch, no CTA waits for another, and 256 CTAs rescan 500 requests in the time
// that a second launch would take. 64 requests with a token or none take 3.9 us on
// the device, 254K tokens of 500 requests 7.1 us (3.1 MB: 0.45 us at the copy rate).
#include <cuda_runtime.h>
#include <stdint.h>

#include "fd.h"
#include "ptx.cuh"
#include "step.h"

namespace fd {
namespace {

constexpr int kThreads = 1024;
constexpr int kTokens = 1024;  // tokens a CTA

// Inclusive prefix sum over the block; sums[32] is left with the warps' totals' prefix sums.
__device__ __forceinline__ long long block_scan(long long v, long long *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  __syncthreads();  // earlier readers of sums are through
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long t = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += up;
    }
    sums[lane] = t;
  }
  __syncthreads();
  return warp ? v + sums[warp - 1] : v;
}

__device__ __forceinline__ int clamp_int(long long v) { return v > 0x7fffffff ? 0x7fffffff : static_cast<int>(v); }

__global__ void __launch_bounds__(kThreads) fd_append_slots_kernel(const __grid_constant__ SlotsParams p) {
  __shared__ long long sums[32];
  __shared__ int start[kThreads];  // first token of each request
  __shared__ int held[kThreads];   // its keys before
  __shared__ int page0[kThreads];  // free page of table entry j: page0 + j; kNone: not served
  __shared__ int last_end;
  constexpr int kNone = -0x7fffffff - 1;
  const int tid = threadIdx.x;
  const long long t0 = static_cast<long long>(blockIdx.x) * kTokens;
  const long long t1 = t0 + kTokens < p.T ? t0 + kTokens : p.T;
  const int chunks = (p.B + kThreads - 1) / kThreads;
  const int bx = blockIdx.x, grid = gridDim.x;
  const int last_mine = bx < chunks ? bx + (chunks - 1 - bx) / grid * grid : -1;  // last chunk that this CTA writes
  if (tid == 0) last_end = 0;
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  long long n_free = p.num_free ? *p.num_free : p.F;
  if (n_free > p.F) {
    if (bx == 0 && tid == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
    n_free = p.F;
  }
  if (n_free < 0) n_free = 0;

  long long cu0 = 0, pages0 = 0;  // tokens and pages of the requests ahead of the chunk
  for (int c = 0; c < chunks; ++c) {
    const bool mine = c % grid == bx;  // this CTA writes the chunk's per-request outputs
    if (cu0 >= t1 && last_mine < c) break;
    const int b = c * kThreads + tid;
    int L = 0, n = 0;
    bool bad = false;
    if (b < p.B) {
      L = p.seqlens[b * p.sl_s];
      n = p.num_new[b * p.n_s];
      bad = L < 0 || n < 0;
      L = max(L, 0);
      n = max(n, 0);
      bad = bad || static_cast<long long>(L) + n > 0x7fffffff;
    }
    const long long cu_end = cu0 + block_scan(n, sums);
    const long long chunk_tokens = sums[31];
    const int before = L / p.P + (L % p.P != 0);
    const long long end_pos = static_cast<long long>(L) + n;
    const long long after = (end_pos + p.P - 1) / p.P;
    bad = bad || after > p.W || cu_end > p.T;
    const long long need = bad ? 0 : after - before;
    const long long end = pages0 + block_scan(need, sums);
    const bool served = !bad && (need == 0 || end <= n_free);
    start[tid] = clamp_int(cu_end - n);
    held[tid] = L;
    page0[tid] = served ? static_cast<int>(end - need - before) : kNone;
    if (served && need > 0) atomicMax(&last_end, static_cast<int>(end));
    if (b < p.B && mine) {
      p.new_seqlens[b] = served ? L + n : L;
      if (b == 0) p.cu[0] = 0;
      p.cu[b + 1] = clamp_int(cu_end);
      if (p.status && !served) atomicOr(p.status, bad ? FD_DEVSTAT_SEQLEN_OVERFLOW : FD_DEVSTAT_NO_PAGES);
    }
    pages0 += sums[31];
    __syncthreads();
    if (mine && c == chunks - 1 && tid == 0) *p.pages_taken = last_end;
    // this CTA's tokens of the chunk's requests
    const long long a = t0 > cu0 ? t0 : cu0, z = t1 < cu0 + chunk_tokens ? t1 : cu0 + chunk_tokens;
    for (long long i = a + tid; i < z; i += kThreads) {
      int lo = 0, hi = kThreads - 1;  // the last request that starts at or before token i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      const long long pos = held[lo] + (i - start[lo]);
      long long slot = -1;
      if (page0[lo] != kNone) {
        const int j = static_cast<int>(pos) / p.P, off = static_cast<int>(pos) % p.P, L0 = held[lo];
        int *entry = p.page_table + (static_cast<int64_t>(c) * kThreads + lo) * p.pt_sb + j;
        int page;
        if (j < L0 / p.P + (L0 % p.P != 0)) {
          page = *entry;
        } else {
          page = p.free_pages[static_cast<int64_t>(page0[lo] + j) * p.f_s];
          if (off == 0) *entry = page;  // (a new page's first key is always new)
        }
        slot = static_cast<long long>(page) * p.P + off;
        if (page < 0 || (!p.slots64 && slot > 0x7fffffff)) {
          slot = -1;
          if (p.status) atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
        }
      }
      if (p.slots64) static_cast<long long *>(p.slots)[i] = slot;
      else static_cast<int *>(p.slots)[i] = static_cast<int>(slot);
      if (p.positions) p.positions[i] = clamp_int(pos);
    }
    cu0 += chunk_tokens;
  }
  // rows behind the last request's: no token (cu0 is the batch's total where any are left)
  for (long long i = (t0 > cu0 ? t0 : cu0) + tid; i < t1; i += kThreads) {
    if (p.slots64) static_cast<long long *>(p.slots)[i] = -1;
    else static_cast<int *>(p.slots)[i] = -1;
    if (p.positions) p.positions[i] = 0;
  }
}

}  // namespace

cudaError_t launch_append_slots(const SlotsParams &p, cudaStream_t stream) {
  const long long ctas = (p.T + kTokens - 1) / kTokens;
  return launch_step(fd_append_slots_kernel, p, dim3(static_cast<unsigned>(ctas < 1 ? 1 : ctas)), kThreads, 0, 1, stream);
}

}  // namespace fd
