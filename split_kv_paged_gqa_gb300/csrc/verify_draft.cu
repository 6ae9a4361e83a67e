// verify_draft.cu - verification of drafted tokens (sm_103a).
//
// Drafted token x_i (i = 0, 1, ...) is accepted while u_i * q_i(x_i) < p_i(x_i),
// p the target's and q the draft's probability. At the first refusal n the step
// ends with a sample from w(v) = max(p_n(v) - q_n(v), 0); with every draft
// accepted it ends with a sample from the target's row behind them. The sample
// is the lowest v whose cumulative weight exceeds u_K times the row's total.
// One CTA per request; products, sums and comparisons in 64 bits (a product of
// two fp32 values is exact there, so acceptance never depends on a rounding).
#include "fd.h"
#include "latent.h"

namespace fd {
namespace {

constexpr int kThreads = 1024;

__device__ __forceinline__ long long token_at(const VerifyParams &p, int b, int i) {
  const int64_t at = b * p.x_sb + i * p.x_sk;
  return p.tok64 ? static_cast<const long long *>(p.tokens)[at] : static_cast<const int *>(p.tokens)[at];
}

__global__ void __launch_bounds__(kThreads) fd_verify_draft_kernel(const VerifyParams p) {
  __shared__ double part[kThreads];
  __shared__ int found, bad;
  const int b = blockIdx.x, tid = threadIdx.x;
  int count = p.K;
  if (p.num_draft) {
    count = p.num_draft[b * p.n_s];
    if (count < 0 || count > p.K) {
      if (tid == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_BAD_TOKEN);
      count = count < 0 ? 0 : p.K;
    }
  }
  if (tid == 0) found = p.V - 1, bad = 0;
  int n = 0;
  long long x = -1;
  for (; n < count; ++n) {
    x = token_at(p, b, n);
    if (x < 0 || x >= p.V) {
      if (tid == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_BAD_TOKEN);
      break;
    }
    const double q = p.draft ? static_cast<double>(p.draft[b * p.d_sb + n * p.d_sk + x]) : 1.0;
    const double u = p.u[b * p.u_sb + n * p.u_sk];
    if (!(u * q < static_cast<double>(p.target[b * p.t_sb + n * p.t_sk + x]))) break;
  }
  const bool refused = n < count;
  const float *tr = p.target + b * p.t_sb + n * p.t_sk;
  const float *dr = refused && p.draft ? p.draft + b * p.d_sb + n * p.d_sk : nullptr;
  const int seg = (p.V + kThreads - 1) / kThreads;
  const int v0 = min(p.V, tid * seg), v1 = min(p.V, v0 + seg);
  for (int plain = refused ? 0 : 1; plain < 2; ++plain) {  // the residual; without any weight in it, the target's row
    auto weight = [&](int v) -> double {
      double w = tr[v];
      if (!plain) w = dr ? w - static_cast<double>(dr[v]) : (v == x ? 0.0 : w);
      return w > 0.0 ? w : 0.0;
    };
    double sum = 0.0;
    for (int v = v0; v < v1; ++v) sum += weight(v);
    __syncthreads();
    part[tid] = sum;
    __syncthreads();
    if (tid == 0) {
      double acc = 0.0;
      for (int i = 0; i < kThreads; ++i) {
        const double t = part[i];
        part[i] = acc;
        acc += t;
      }
      bad = !(acc > 0.0);
      part[0] = acc;  // its own prefix is 0
    }
    __syncthreads();
    if (bad && !plain) continue;
    const double total = part[0], at = static_cast<double>(p.u[b * p.u_sb + p.K * p.u_sk]) * total;
    double acc = tid ? part[tid] : 0.0;
    for (int v = v0; v < v1; ++v) {
      acc += weight(v);
      if (acc > at) {
        atomicMin(&found, v);
        break;
      }
    }
    break;
  }
  __syncthreads();
  for (int i = tid; i <= p.K; i += kThreads)
    p.out[b * p.o_sb + i] = i < n ? static_cast<int>(token_at(p, b, i)) : (i == n ? found : -1);
  if (tid == 0) p.emitted[b] = n + 1;
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyParams &p, cudaStream_t stream) {
  fd_verify_draft_kernel<<<p.B, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fd
