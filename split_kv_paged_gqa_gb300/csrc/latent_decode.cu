// latent_decode.cu - absorbed latent attention over a paged cache (sm_103a).
//
// A token's cache row c_j holds 512 latent and 64 rotary channels. With the
// per-head up-projections absorbed into q, every head attends to the same rows:
//   s_rj = scale * q_r . c_j (576 channels),  o_r = sum_j softmax(s_r)_j c_j[0:512].
// One CTA per (request, tile of 16 query rows): each of 8 warps owns two rows;
// keys pass through shared memory in blocks of 32, one per lane for the scores
// (rows padded to an odd number of words: no bank conflicts), 16 channels per
// lane for the sums, with a running maximum and sum in fp32.
#include <math.h>

#include "fd.h"
#include "latent.h"
#include "ptx.cuh"

namespace fd {
namespace {

constexpr int kRows = 16, kKeys = 32, kThreads = 256, kPad = kLatRow + 2;

__global__ void __launch_bounds__(kThreads) fd_latent_decode_kernel(const LatentDecodeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float *qs = reinterpret_cast<float *>(smem);                                   // [16][576]
  __nv_bfloat16 *ks = reinterpret_cast<__nv_bfloat16 *>(qs + kRows * kLatRow);   // [32][578]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y, row0 = blockIdx.x * kRows;
  const int cap = p.max_pages * p.page_size;
  int L = p.seqlens[b * p.sl_s];
  if (L < 0 || L > cap) {
    if (tid == 0) atomicOr(p.status, FD_DEVSTAT_SEQLEN_OVERFLOW);
    L = L < 0 ? 0 : cap;
  }
  for (int i = tid; i < kRows * kLatRow; i += kThreads) {
    const int r = row0 + i / kLatRow, c = i % kLatRow;
    float v = 0.f;
    if (r < p.R) v = __bfloat162float(p.q[b * p.q_sb + (r / p.H) * p.q_st + (r % p.H) * p.q_sh + c]);
    qs[i] = v;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][16];
  int lim[2];
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + warp * 2 + i;
    lim[i] = r < p.R ? L - (p.Tq - 1) + r / p.H : 0;
    for (int c = 0; c < 16; ++c) o[i][c] = 0.f;
  }
  for (int k0 = 0; k0 < L; k0 += kKeys) {
    __syncthreads();
    for (int i = tid; i < kKeys * (kLatRow / 2); i += kThreads) {
      const int j = i / (kLatRow / 2), c = i % (kLatRow / 2) * 2, key = k0 + j;
      uint32_t v = 0u;
      if (key < L) {
        const int pid = p.page_table[b * p.pt_sb + (key >> p.log2_page)];
        if (pid >= 0 && pid < p.num_pages)
          v = *reinterpret_cast<const uint32_t *>(p.cache + pid * p.c_sp + (key & (p.page_size - 1)) * p.c_ss + c);
        else
          atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
      }
      *reinterpret_cast<uint32_t *>(ks + j * kPad + c) = v;
    }
    __syncthreads();
    for (int i = 0; i < 2; ++i) {
      const float *qr = qs + (warp * 2 + i) * kLatRow;
      float s = 0.f;
      for (int c = 0; c < kLatRow; ++c) s = fmaf(qr[c], __bfloat162float(ks[lane * kPad + c]), s);
      s = k0 + lane < lim[i] ? s * p.scale_log2 : -INFINITY;
      float mx = s;
      for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
      const float mn = fmaxf(m[i], mx);
      if (mn == -INFINITY) continue;
      const float e = exp2f(s - mn), a = exp2f(m[i] - mn);
      float sum = e;
      for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
      l[i] = l[i] * a + sum;
      m[i] = mn;
      for (int c = 0; c < 16; ++c) o[i][c] *= a;
      for (int j = 0; j < kKeys; ++j) {
        const float pj = __shfl_sync(~0u, e, j);
        if (pj != 0.f)
          for (int c = 0; c < 16; ++c) o[i][c] = fmaf(pj, __bfloat162float(ks[j * kPad + c * 32 + lane]), o[i][c]);
      }
    }
  }
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + warp * 2 + i;
    if (r >= p.R) continue;
    const int t = r / p.H, h = r % p.H;
    const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
    for (int c = 0; c < 16; ++c) {
      const int64_t at = b * p.o_sb + t * p.o_st + h * p.o_sh + c * 32 + lane;
      if (p.out_f32) static_cast<float *>(p.out)[at] = o[i][c] * inv;
      else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o[i][c] * inv);
    }
    if (lane == 0 && p.lse)
      p.lse[b * p.l_sb + t * p.l_st + h * p.l_sh] =
          l[i] > 0.f ? (m[i] + log2f(l[i])) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_latent_decode(const LatentDecodeParams &p, cudaStream_t stream) {
  const int bytes = kRows * kLatRow * 4 + kKeys * kPad * 2;
  cudaError_t e = cudaFuncSetAttribute(fd_latent_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  fd_latent_decode_kernel<<<dim3((p.R + kRows - 1) / kRows, p.B), kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fd
