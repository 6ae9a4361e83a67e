// latent_prefill.cu - expanded latent attention of ragged prompts (sm_103a).
//
// Query i of request b (its q tokens are rows cu_q[b] .. cu_q[b + 1]) sees the
// first i + 1 + (Lk - Lq) of the request's Lk keys. Scores add the head's own
// 128 channels and the 64 rotary channels that all heads share:
//   s_ij = scale * (q_i[0:128] . k_jh + q_i[128:192] . kpe_j),  o_i = sum_j softmax(s_i)_j v_jh.
// One CTA per (16 queries, head, request): each of 8 warps owns two rows; keys
// pass through shared memory in blocks of 32, one per lane for the scores, four
// channels per lane for the sums, with a running maximum and sum in fp32.
#include <math.h>

#include "fd.h"
#include "latent.h"
#include "ptx.cuh"

namespace fd {
namespace {

constexpr int kRows = 16, kKeys = 32, kThreads = 256, kD = kLatNope + kLatR, kPad = kD + 2;

__global__ void __launch_bounds__(kThreads) fd_latent_prefill_kernel(const LatentPrefillParams p) {
  __shared__ float qs[kRows * kD];
  __shared__ __nv_bfloat16 ks[kKeys * kPad];
  __shared__ __nv_bfloat16 vs[kKeys * kLatV];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z, i0 = blockIdx.x * kRows;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], s0 = p.cu_k[b], s1 = p.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > p.Sq || s0 < 0 || s1 < s0 || s1 > p.Sk || q1 - q0 > p.max_q) {
    if (tid == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_SEQLEN_OVERFLOW);
    return;
  }
  const int Lq = q1 - q0, Lk = s1 - s0;
  if (i0 >= Lq) return;
  for (int i = tid; i < kRows * kD; i += kThreads) {
    const int r = i0 + i / kD, c = i % kD;
    qs[i] = r < Lq ? __bfloat162float(p.q[static_cast<int64_t>(q0 + r) * p.q_ss + h * p.q_sh + c]) : 0.f;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][4] = {};
  const int kend = min(Lk, i0 + kRows + Lk - Lq);  // keys that the tile's last row sees
  for (int k0 = 0; k0 < kend; k0 += kKeys) {
    __syncthreads();
    for (int i = tid; i < kKeys * kD; i += kThreads) {
      const int j = i / kD, c = i % kD;
      const int64_t key = s0 + k0 + j;
      __nv_bfloat16 v = __float2bfloat16(0.f);
      if (k0 + j < Lk) v = c < kLatNope ? p.k[key * p.k_ss + h * p.k_sh + c] : p.kpe[key * p.pe_ss + c - kLatNope];
      ks[j * kPad + c] = v;
    }
    for (int i = tid; i < kKeys * kLatV; i += kThreads) {
      const int j = i / kLatV, c = i % kLatV;
      vs[i] = k0 + j < Lk ? p.v[static_cast<int64_t>(s0 + k0 + j) * p.v_ss + h * p.v_sh + c] : __float2bfloat16(0.f);
    }
    __syncthreads();
    for (int i = 0; i < 2; ++i) {
      const int r = warp * 2 + i;
      const int lim = i0 + r < Lq ? i0 + r + 1 + Lk - Lq : 0;
      float s = 0.f;
      for (int c = 0; c < kD; ++c) s = fmaf(qs[r * kD + c], __bfloat162float(ks[lane * kPad + c]), s);
      s = k0 + lane < lim ? s * p.scale_log2 : -INFINITY;
      float mx = s;
      for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
      const float mn = fmaxf(m[i], mx);
      if (mn == -INFINITY) continue;
      const float e = exp2f(s - mn), a = exp2f(m[i] - mn);
      float sum = e;
      for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
      l[i] = l[i] * a + sum;
      m[i] = mn;
      for (int c = 0; c < 4; ++c) o[i][c] *= a;
      for (int j = 0; j < kKeys; ++j) {
        const float pj = __shfl_sync(~0u, e, j);
        if (pj != 0.f)
          for (int c = 0; c < 4; ++c) o[i][c] = fmaf(pj, __bfloat162float(vs[j * kLatV + c * 32 + lane]), o[i][c]);
      }
    }
  }
  for (int i = 0; i < 2; ++i) {
    const int r = i0 + warp * 2 + i;
    if (r >= Lq) continue;
    const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
    for (int c = 0; c < 4; ++c) {
      const int64_t at = static_cast<int64_t>(q0 + r) * p.o_ss + h * p.o_sh + c * 32 + lane;
      if (p.out_f32) static_cast<float *>(p.out)[at] = o[i][c] * inv;
      else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o[i][c] * inv);
    }
    if (lane == 0 && p.lse)
      p.lse[static_cast<int64_t>(q0 + r) * p.l_ss + h * p.l_sh] =
          l[i] > 0.f ? (m[i] + log2f(l[i])) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams &p, cudaStream_t stream) {
  fd_latent_prefill_kernel<<<dim3((p.max_q + kRows - 1) / kRows, p.H, p.B), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fd
