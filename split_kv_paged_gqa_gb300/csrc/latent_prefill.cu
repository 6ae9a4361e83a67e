// latent_prefill.cu - expanded latent attention of ragged prompts on the
// tcgen05 tensor cores (sm_103a).
//
// Query i of request b (its q tokens are rows cu_q[b] .. cu_q[b + 1]) sees the
// first i + 1 + (Lk - Lq) of the request's Lk keys. Scores add the head's own
// 128 channels and the 64 rotary channels that all heads share:
//   s_ij = scale * (q_i[0:128] . k_jh + q_i[128:192] . kpe_j),  o_i = sum_j softmax(s_i)_j v_jh.
// 640 flops a visible (query, key, head): the tensor cores bound it.
//
// One CTA = one head and 256 queries of one request, as two sub-tiles of 128
// rows whose turns on the tensor cores alternate: while the softmax warps of
// one work on its scores, the MMAs of the other run. Key tiles of 128.
//  * producer warp: Q once, then K tiles (three 16 KB blocks of 64 channels:
//    two of k_nope, one of k_pe) and V tiles (two blocks) through a ring of
//    eight 16 KB slots with TMA (128-byte swizzle), in the order in which the
//    MMAs use them: K0 K1 V0 K2 V1 K3 V2 ...
//  * MMA warp, one thread: S = Q K^T (M = 128, N = 128, 12 K steps) into TMEM,
//    O += P V (P from TMEM, V read MN-major, 8 K steps). Per sub-tile in issue
//    order S(0), PV(0), S(1), PV(1), ...: MMAs execute in issue order, so S(j + 1)
//    may overwrite P(j), and the arrival that announces S(j + 1) says that
//    PV(j) is done.
//  * four softmax warps per sub-tile, a row a thread: running maximum moved only
//    when a row outgrows it by 2^8 (then O is rescaled in TMEM), weights
//    rounded to bf16 (the tensor core's operand type; at most 2^-8 of each)
//    over the scores' columns, sums and LSE in fp32 from the unrounded weights.
// TMEM: two score tiles and two output tiles of 128 columns, all 512.
#include <math.h>

#include "fd.h"
#include "latent.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace fd {
namespace {

constexpr int kSub = 128;                        // query rows of a sub-tile
constexpr int kKeys = 128;                       // keys of a tile
constexpr int kSlotBytes = 128 * 128;            // 128 rows x 64 channels
constexpr int kSlots = 8;
constexpr int kQBlocks = 3;                      // (128 + 64) / 64
constexpr int kProducer = 8, kMma = 9, kThreads = 320;
constexpr int kOffRing = 2 * kQBlocks * kSlotBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kBars = 2 * kSlots + 8;            // full, empty, qfull[2], sfull[2], pfull[2], ofull (count 2 commits), vfix
constexpr int kOffMisc = kOffBar + kBars * 8;
constexpr int kSmem = kOffMisc + 16;
constexpr int kSmemAlloc = kSmem + 1024;         // slack to align the base to 1024
static_assert(kSmemAlloc <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kTmO = 256;  // S of sub-tile x at 128 x, O at 256 + 128 x

__device__ unsigned g_status_sink;               // for calls without a status word

// Ring position of the first slot of K tile j (three slots) and V tile j (two).
__device__ __forceinline__ int pos_k(int j) { return j == 0 ? 0 : 5 * j - 2; }
__device__ __forceinline__ int pos_v(int j) { return 5 * j + 6; }

__device__ __forceinline__ bool wait_bar(uint64_t *bar, unsigned parity, unsigned *status, volatile int *abort) {
  if (mbar_test(bar, parity)) return true;
  if (*abort) return false;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, FD_DEVSTAT_WAIT_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_bar_warp(uint64_t *bar, unsigned parity, unsigned *status, volatile int *abort) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, status, abort)) != 0;
}

__global__ void __launch_bounds__(kThreads, 1)
    fd_latent_prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                             const __grid_constant__ CUtensorMap tmpe, const __grid_constant__ CUtensorMap tmv,
                             const __grid_constant__ LatentPrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);
  uint64_t *empty = full + kSlots;
  uint64_t *qfull = empty + kSlots;  // [sub-tile]
  uint64_t *sfull = qfull + 2;       // [sub-tile] scores written (and the PV before them done)
  uint64_t *pfull = sfull + 2;       // [sub-tile] weights written
  uint64_t *ofull = pfull + 2;       // all MMAs done
  uint64_t *vfix = ofull + 1;        // rows of the last V tile past the request's keys are zero
  uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned *status = p.status ? p.status : &g_status_sink;
  // the last queries of a request see the most keys: they start first
  const int h = blockIdx.x % p.H, rest = blockIdx.x / p.H;
  const int b = rest % p.B, i0 = (p.q_tiles - 1 - rest / p.B) * (2 * kSub);
  griddep_wait();
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], s0 = p.cu_k[b], s1 = p.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > p.Sq || s0 < 0 || s1 < s0 || s1 > p.Sk || q1 - q0 > p.max_q) {
    if (threadIdx.x == 0) atomicOr(status, FD_DEVSTAT_SEQLEN_OVERFLOW);
    return;
  }
  const int Lq = q1 - q0, Lk = s1 - s0, ahead = Lk - Lq;
  if (i0 >= Lq) return;
  // key tiles that a sub-tile's last row sees
  auto tiles = [&](int x) {
    const int first = i0 + x * kSub;
    if (first >= Lq) return 0;
    const int see = min(Lq, first + kSub) + ahead;
    return see <= 0 ? 0 : (see + kKeys - 1) / kKeys;
  };
  const int na = tiles(0), nb = tiles(1), nt = max(na, nb);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&qfull[x], 1);
      mbar_init(&sfull[x], 1);
      mbar_init(&pfull[x], 4);
    }
    mbar_init(ofull, 1);
    mbar_init(vfix, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMma) tmem_alloc(tslot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const int last_valid = Lk - (nt - 1) * kKeys;  // keys of the request in the last tile
  const bool fix = nt > 0 && last_valid < kKeys;

  if (warp == kProducer) {
    // ======================= TMA producer =======================
    if (nt > 0) {
      const uint64_t pol = l2_policy_evict_normal();
      bool ok = true;
      int last = -1;  // last ring position filled
      if (elect_one()) {
        for (int x = 0; x < 2; ++x) {
          if (x == 0 ? na == 0 : nb == 0) continue;
          mbar_arrive_expect_tx(&qfull[x], kQBlocks * kSlotBytes);
          for (int c = 0; c < kQBlocks; ++c)
            tma_load_3d(smem + (x * kQBlocks + c) * kSlotBytes, &tmq, c * 64, h, q0 + i0 + x * kSub, &qfull[x], pol);
        }
        auto slot = [&](int pos) -> uint8_t * {  // a free slot's address, its barrier armed
          const int s = pos % kSlots;
          ok = ok && wait_bar(&empty[s], ((pos / kSlots) & 1) ^ 1, status, abort_flag);
          if (!ok) return nullptr;
          mbar_arrive_expect_tx(&full[s], kSlotBytes);
          last = pos;
          return smem + kOffRing + s * kSlotBytes;
        };
        auto load_k = [&](int j) {
          for (int c = 0; c < 3 && ok; ++c) {
            const int pos = pos_k(j) + c;
            uint8_t *dst = slot(pos);
            if (!dst) break;
            if (c < 2) tma_load_3d(dst, &tmk, c * 64, h, s0 + j * kKeys, &full[pos % kSlots], pol);
            else tma_load_2d(dst, &tmpe, 0, s0 + j * kKeys, &full[pos % kSlots], pol);
          }
        };
        load_k(0);
        for (int j = 0; j < nt && ok; ++j) {
          if (j + 1 < nt) load_k(j + 1);
          for (int c = 0; c < 2 && ok; ++c) {
            const int pos = pos_v(j) + c;
            uint8_t *dst = slot(pos);
            if (dst) tma_load_3d(dst, &tmv, c * 64, h, s0 + j * kKeys, &full[pos % kSlots], pol);
          }
        }
        if (!ok)  // given up: the copies in flight land before the CTA ends
          for (int pos = max(0, last - kSlots + 1); pos <= last; ++pos)
            mbar_wait(&full[pos % kSlots], (pos / kSlots) & 1, status);
      }
      __syncwarp();
      if (fix) {
        // Rows of the last V tile past the request's keys belong to nobody here
        // and may hold anything; their weight 0 needs them finite.
        const int pos = pos_v(nt - 1);
        for (int c = 0; c < 2; ++c) {
          const int s = (pos + c) % kSlots;
          if (!wait_bar_warp(&full[s], ((pos + c) / kSlots) & 1, status, abort_flag)) break;
          uint8_t *v = smem + kOffRing + s * kSlotBytes + last_valid * 128;
          for (int i = lane; i < (kKeys - last_valid) * 8; i += 32)
            reinterpret_cast<uint4 *>(v)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(vfix);
      }
    }
  } else if (warp == kMma) {
    // ======================= MMA issuer =======================
    if (nt > 0 && elect_one()) {
      const uint32_t base = smem_u32(smem);
      const uint64_t qd = umma_desc_sw128(base), kd = umma_desc_sw128(base + kOffRing);
      const uint64_t vd = umma_desc_sw128_mn(base + kOffRing, kSlotBytes, 1024);
      constexpr uint32_t id_s = umma_idesc_bf16(128, kKeys, false, false);
      constexpr uint32_t id_o = umma_idesc_bf16(128, 64, false, true);
      bool ok = true;
      int started = 0;  // bit x: sub-tile x has scores issued
      auto scores = [&](int x, int j, bool wait_k) {
        if (!ok) return;
        if (j == 0) ok = wait_bar(&qfull[x], 0, status, abort_flag);
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const int pos = pos_k(j) + c, s = pos % kSlots;
          if (ok && wait_k) ok = wait_bar(&full[s], (pos / kSlots) & 1, status, abort_flag);
          if (!ok) return;
          if (c == 0 || wait_k) tc_fence_after();
          const uint64_t kt = kd + ((s * kSlotBytes) >> 4), qt = qd + (((x * kQBlocks + c) * kSlotBytes) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f16_ss(tmem + x * 128, qt + ((k * 32) >> 4), kt + ((k * 32) >> 4), id_s, (c > 0 || k > 0) ? 1u : 0u);
        }
        started |= 1 << x;
      };
      auto values = [&](int x, int j, bool wait_v) {
        if (ok) ok = wait_bar(&pfull[x], j & 1, status, abort_flag);
        if (!ok) return;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int pos = pos_v(j) + c, s = pos % kSlots;
          if (ok && wait_v) {
            ok = wait_bar(&full[s], (pos / kSlots) & 1, status, abort_flag);
            if (ok && c == 0 && fix && j == nt - 1) ok = wait_bar(vfix, 0, status, abort_flag);
          }
          if (!ok) return;
          tc_fence_after();
          const uint64_t vt = vd + ((s * kSlotBytes) >> 4);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)  // 64 value channels at a time: a slot
            umma_f16_ts(tmem + kTmO + x * 128 + c * 64, tmem + x * 128 + k * 8, vt + ((k * 2048) >> 4), id_o,
                        (j > 0 || k > 0) ? 1u : 0u);
        }
      };
      auto release = [&](int pos, int n) {
        for (int i = 0; i < n; ++i) umma_commit(&empty[(pos + i) % kSlots]);
      };
      if (na > 0) {
        scores(0, 0, true);
        if (ok) umma_commit(&sfull[0]);
      }
      if (nb > 0) {
        scores(1, 0, na == 0);
        if (ok) umma_commit(&sfull[1]);
      }
      if (ok) release(pos_k(0), 3);
      for (int j = 0; j < nt && ok; ++j) {
        // sub-tile 0, then 1: PV(j), S(j + 1); the first to use a tile waits for it, the last frees it
        if (j < na) values(0, j, true);
        if (ok && j < na && j >= nb) release(pos_v(j), 2);
        if (ok && j + 1 < na) {
          scores(0, j + 1, true);
          if (ok) umma_commit(&sfull[0]);
          if (ok && j + 1 >= nb) release(pos_k(j + 1), 3);
        }
        if (j < nb) values(1, j, j >= na);
        if (ok && j < nb) release(pos_v(j), 2);
        if (ok && j + 1 < nb) {
          scores(1, j + 1, j + 1 >= na);
          if (ok) umma_commit(&sfull[1]);
          if (ok) release(pos_k(j + 1), 3);
        }
      }
      if (started) {
        umma_commit(ofull);
        mbar_wait(ofull, 0, status);  // MMAs end before TMEM is released
      }
    }
    __syncwarp();
  } else {
    // ======================= softmax warps =======================
    const int x = warp >> 2, n = x == 0 ? na : nb;
    const int r = (warp & 3) * 32 + lane, i = i0 + x * kSub + r;  // this thread's row: TMEM lane r of its sub-tile
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_base + x * 128, to = tmem + lane_base + kTmO + x * 128;
    const int lim = i < Lq ? min(Lk, max(0, i + 1 + ahead)) : 0;
    const int lim_min = __reduce_min_sync(0xffffffffu, lim);
    float m = -INFINITY, l = 0.f;
    const float2 sc = make_float2(p.scale_log2, p.scale_log2);
    for (int j = 0; j < n; ++j) {
      wait_bar_warp(&sfull[x], j & 1, status, abort_flag);
      tc_fence_after();
      float s[kKeys];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s + 32 * c);
      tmem_wait_ld();
      if ((j + 1) * kKeys > lim_min) {
        const int see = lim - j * kKeys;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) s[c] = c < see ? s[c] : -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < kKeys; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      if (__any_sync(0xffffffffu, top > m + 8.f)) {
        const float mn = fmaxf(m, top), f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
        m = mn;
        l *= f;
        if (j > 0) {  // PV(j - 1) is done: S(j) was issued behind it
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            float o[16];
            tmem_ld16(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] *= f;
            tmem_st16(to + c, o);
          }
        }
      }
      const float u = m == -INFINITY ? 0.f : -m;
      const float2 off = make_float2(u, u);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 a = fma2(make_float2(s[c + 2 * k], s[c + 2 * k + 1]), sc, off);
          const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
          sum = add2(sum, e);
          w[k] = pack_bf16x2(e.x, e.y);
        }
        tmem_st16u(ts + c / 2, w);
      }
      l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull[x]);
    }
    if (n > 0) {
      wait_bar_warp(ofull, 0, status, abort_flag);
      tc_fence_after();
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t at = static_cast<int64_t>(q0 + i) * p.o_ss + h * p.o_sh;
#pragma unroll 1
    for (int c = 0; c < 128; c += 16) {
      float o[16];
      if (n > 0) {
        tmem_ld16(to + c, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = l > 0.f ? o[k] * inv : 0.f;
      if (i >= Lq) continue;
      if (p.out_f32) {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + c);
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      } else {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at + c);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          dst[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                              pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
      }
    }
    if (p.lse && i < Lq)
      p.lse[static_cast<int64_t>(q0 + i) * p.l_ss + h * p.l_sh] =
          l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_latent_prefill(const CUtensorMap (&tm)[4], LatentPrefillParams p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(fd_latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  p.q_tiles = (p.max_q + 2 * kSub - 1) / (2 * kSub);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.q_tiles) * p.H * p.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemAlloc;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fd_latent_prefill_kernel, tm[0], tm[1], tm[2], tm[3], p);
}

}  // namespace fd
