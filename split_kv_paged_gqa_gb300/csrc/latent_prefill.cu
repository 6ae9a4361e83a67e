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
//    MMAs first use and release them: K0 V0 K1 V1 ... (with K1 ahead of V0 each V
//    tile waits for the release of the K tile in use: 1044 us instead of 855 on
//    16K queries x 16 heads).
//  * MMA warp, one thread: S = Q K^T (M = 128, N = 128, 12 K steps) into TMEM,
//    O += P V (P from TMEM, V read MN-major, 8 K steps). Per sub-tile in issue
//    order S(0), PV(0), S(1), PV(1), ...: MMAs execute in issue order, so S(j + 1)
//    may overwrite P(j), and the arrival that announces S(j + 1) says that
//    PV(j) is done.
//  * eight softmax warps per sub-tile, two threads a row (a warp alone on its
//    scheduler takes 1130 clocks for a row of 128, two warps with 64 each 860;
//    the chain S, softmax, PV of a sub-tile sets the pace): running maximum moved
//    only when a row outgrows it by 2^8 (then O is rescaled in TMEM), weights
//    rounded to bf16 (the tensor core's operand type; at most 2^-8 of each)
//    over the scores' columns, sums and LSE in fp32 from the unrounded weights.
// TMEM: two score tiles and two output tiles of 128 columns, all 512.
//
// Few queries behind many keys leave most SMs without a CTA: then a cluster of
// 2, 4 or 8 shares an item, each CTA a run of its key tiles, and joins the fp32
// outputs through distributed shared memory (ranks_of below has the rule).
// Measured in loops: 16384 tokens x 16 heads 835 to 880 us from box to box (1560 to
// 1650 TFLOP/s: the power cap sets the clock; 795 us before it does), 8192 x 16
// 207, 2048 x 16 33, 512 behind 8488 x 16 44, 128 x 16 6.4.
#include <cooperative_groups.h>
#include <math.h>

#include "fd.h"
#include "latent.h"
#include "latent_ptx.cuh"
#include "tc.cuh"

namespace fd {
namespace {

namespace cg = cooperative_groups;

constexpr int kSub = 128;                        // query rows of a sub-tile
constexpr int kKeys = 128;                       // keys of a tile
constexpr int kSlotBytes = 128 * 128;            // 128 rows x 64 channels
constexpr int kSlots = 8;
constexpr int kQBlocks = 3;                      // (128 + 64) / 64
constexpr int kProducer = 16, kMma = 17, kThreads = 18 * 32;
constexpr int kOffRing = 2 * kQBlocks * kSlotBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kBars = kSlots + 13;               // full, kempty[2], vempty[2], qfull[2], sfull[2], pfull[2], ofull[2], vfix
constexpr int kOffMisc = kOffBar + kBars * 8;
constexpr int kOffSwap = kOffMisc + 16;          // float [256]: a row's word between its two threads
constexpr int kOffItem = kOffSwap + 2 * kSub * 4;  // the CTA's Item
constexpr int kOffTaken = kOffItem + 20;
constexpr int kOffDrain = kOffItem + 24;
constexpr int kSmem = kOffDrain + 8;
constexpr int kSmemAlloc = kSmem + 1024;         // slack to align the base to 1024
static_assert(kSmemAlloc <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kTmO = 256;  // S of sub-tile x at 128 x, O at 256 + 128 x

__device__ unsigned g_status_sink;               // for calls without a status word

// Eight words to global memory: one store where the address allows (a row half
// is written by one thread: 32-byte pieces are whole sectors), else two.
__device__ __forceinline__ void store32(void *dst, const uint32_t *v, int wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  else {
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Ring position of the first slot of K tile j (three slots) and V tile j (two).
__device__ __forceinline__ int pos_k(int j) { return 5 * j; }
__device__ __forceinline__ int pos_v(int j) { return 5 * j + 3; }

// Bounded wait that gives up at once when another warp of the CTA has (the
// abort word). After a timeout every warp runs to the end: the softmax warps
// without waiting, and without arriving, so that no MMA starts and no slot is
// refilled on their word; the producer and the MMA warp stop, and wait for what
// they have in flight before the CTA reuses or leaves its memory. SPIN: the MMA thread tests without being suspended (a suspended
// thread wakes later; 966 -> 855 us on 16K queries x 16 heads), with a short
// sleep that leaves the shared-memory pipe to the softmax warps (846 -> 828).
template <bool SPIN = false>
__device__ __forceinline__ bool wait_bar(uint64_t *bar, unsigned parity, unsigned limit_ns, unsigned *status,
                                         volatile int *abort) {
  unsigned long long t0 = 0;
  // (a wait with a limit shorter than a suspension is not suspended)
  for (unsigned spins = 0;
       !(SPIN || limit_ns < kSuspendHintNs ? mbar_test(bar, parity) : mbar_try_wait(bar, parity)); ++spins) {
    if (SPIN && (spins & 255u) != 255u) {
      __nanosleep(20);
      continue;
    }
    if (*abort) return false;
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > limit_ns) {
      atomicOr(status, FD_DEVSTAT_WAIT_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool wait_bar_warp(uint64_t *bar, unsigned parity, unsigned limit_ns, unsigned *status,
                                              volatile int *abort) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, limit_ns, status, abort)) != 0;
}

// 256 queries of a request, from its i0-th on (i0 < 0: nothing to do).
struct Item {
  int i0, q0, Lq, s0, Lk;  // first query; the request's first query row, queries, first key row, keys
};

// Whether query rows [q0, q1) and key rows [s0, s1) of a request lie in the tensors.
__device__ __forceinline__ bool rows_ok(const LatentPrefillParams &p, int q0, int q1, int s0, int s1) {
  return q0 >= 0 && q1 >= q0 && q1 <= p.Sq && s0 >= 0 && s1 >= s0 && s1 <= p.Sk && q1 - q0 <= p.max_q;
}

// The u-th tile of 256 queries: requests in chunks of 32, and within a chunk the
// last queries first (they see the most keys), level by level over its requests.
// A request with bad rows has no tiles, nor one whose rows an earlier one owns.
// Warp-collective. report: looks at all requests and records bad ones. (A CTA
// without a tile costs its SM 0.6 us: 4 x 2500 queries x 32 heads with room for
// 10000 each 242 us without this, 221 with it.)
__device__ __forceinline__ Item find_item(const LatentPrefillParams &p, int u, int lane, bool report, unsigned *status) {
  Item it = {-1, 0, 0, 0, 0};
  int end = 0;  // of the query rows so far
  bool found = false;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B && (report || !found); b0 += 32) {
    const bool in = b0 + lane < p.B;
    const int b = min(b0 + lane, p.B - 1);
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], s0 = p.cu_k[b], s1 = p.cu_k[b + 1];
    bool ok = rows_ok(p, q0, q1, s0, s1);
    int upto = ok ? max(end, q1) : end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) upto = max(upto, __shfl_up_sync(0xffffffffu, upto, o));
    const int before = __shfl_up_sync(0xffffffffu, upto, 1);
    ok = ok && q0 >= (lane ? before : end);
    end = __shfl_sync(0xffffffffu, upto, 31);
    if (report && in && !ok) atomicOr(status, FD_DEVSTAT_SEQLEN_OVERFLOW);
    const int n = in && ok ? (q1 - q0 + 2 * kSub - 1) / (2 * kSub) : 0;
    const int total = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
    if (!found && u < total) {
      found = true;
      int top = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(n)));
      while (true) {  // levels next .. top - 1 have the requests of at least `top` tiles
        const unsigned at = __ballot_sync(0xffffffffu, n >= top);
        const int next = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(n < top ? n : 0)));
        const int c = __popc(at), here = c * (top - next);
        if (u < here) {
          const unsigned mine = __ballot_sync(0xffffffffu, n >= top && __popc(at & ((1u << lane) - 1u)) == u % c);
          const int src = __ffs(mine) - 1;
          it.i0 = (top - 1 - u / c) * (2 * kSub);
          it.q0 = __shfl_sync(0xffffffffu, q0, src);
          it.Lq = __shfl_sync(0xffffffffu, q1 - q0, src);
          it.s0 = __shfl_sync(0xffffffffu, s0, src);
          it.Lk = __shfl_sync(0xffffffffu, s1 - s0, src);
          break;
        }
        u -= here;
        top = next;
      }
    }
    u -= total;
  }
  return it;
}

// The outputs of R ranks for this warp's 16 / R rows from `row0`, joined and
// written: each lane reads one row's maximum or sum of one rank, then four
// channels of eight (row, rank) pairs at a time, so that the reads of the other
// CTAs' shared memory overlap.
template <int R>
__device__ __forceinline__ void join_ranks(cg::cluster_group &cluster, uint8_t *smem, float *stat,
                                           const LatentPrefillParams &p, int row0, int q0, int i0, int Lq, int h,
                                           int lane) {
  constexpr int kRows = 16 / R, kAtOnce = 8 / R;
  const int mine = lane >> 1;  // pair: row mine / R, rank mine % R
  const float st = cluster.map_shared_rank(stat, mine % R)[(lane & 1) * 2 * kSub + row0 + mine / R];
#pragma unroll
  for (int k0 = 0; k0 < kRows; k0 += kAtOnce) {
    if (i0 + row0 + k0 >= Lq) break;
    float4 o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int row = row0 + k0 + u / R;
      o[u] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(smem, u % R) + kOffRing + row * 512 +
                                               ((lane ^ (row & 31)) << 4));
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      float top = -INFINITY, total = 0.f, w[R];
#pragma unroll
      for (int c = 0; c < R; ++c) {
        w[c] = __shfl_sync(0xffffffffu, st, ((k0 + k) * R + c) * 2);
        top = fmaxf(top, w[c]);
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < R; ++c) {
        const float l = __shfl_sync(0xffffffffu, st, ((k0 + k) * R + c) * 2 + 1);
        // A rank that saw nothing is left out (its scores may have been NaN: its sum
        // says so). One whose keys have lost all their weight is not: 0 times NaN.
        const bool seen = w[c] != -INFINITY;
        w[c] = seen ? fast_exp2(w[c] - top) : 0.f;
        total += l * w[c];
        const float4 v = seen ? o[k * R + c] : make_float4(0.f, 0.f, 0.f, 0.f);
        acc.x += v.x * w[c];
        acc.y += v.y * w[c];
        acc.z += v.z * w[c];
        acc.w += v.w * w[c];
      }
      const int i = i0 + row0 + k0 + k;
      if (i >= Lq) break;
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const int64_t at = static_cast<int64_t>(q0 + i) * p.o_ss + h * p.o_sh + lane * 4;
      if (p.out_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (p.lse && lane == 0)
        p.lse[static_cast<int64_t>(q0 + i) * p.l_ss + h * p.l_sh] =
            total == 0.f ? -INFINITY : (top + log2f(total)) * 0.69314718055994531f;
    }
  }
}

// SPLIT: a cluster of p.ranks CTAs shares an item, each a run of its key tiles;
// their outputs are joined through distributed shared memory.
template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    fd_latent_prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                             const __grid_constant__ CUtensorMap tmpe, const __grid_constant__ CUtensorMap tmv,
                             const __grid_constant__ LatentPrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);
  uint64_t *kempty = full + kSlots;  // [2]: K tile j released, on barrier j % 2
  uint64_t *vempty = kempty + 2;     // [2]: V tile j
  uint64_t *qfull = vempty + 2;      // [sub-tile]
  uint64_t *sfull = qfull + 2;       // [sub-tile] scores written (and the PV before them done)
  uint64_t *pfull = sfull + 2;       // [sub-tile] weights written
  uint64_t *ofull = pfull + 2;       // [sub-tile] output complete
  uint64_t *vfix = ofull + 2;        // rows of the last V tile past the request's keys are zero
  uint64_t *drain = reinterpret_cast<uint64_t *>(smem + kOffDrain);  // the MMA thread gave up: its MMAs are done
  uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned *status = p.status ? p.status : &g_status_sink;
  const int unit = SPLIT ? blockIdx.x / p.ranks : blockIdx.x, rank = SPLIT ? blockIdx.x % p.ranks : 0;
  const int h = unit % p.H;
  Item *const item = reinterpret_cast<Item *>(smem + kOffItem);
  volatile int *const taken = reinterpret_cast<volatile int *>(smem + kOffTaken);  // the item's rows are an earlier request's
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  if (warp == 0) {
    const int u = unit / p.H;
    if (p.ragged) {
      const Item it = find_item(p, u, lane, blockIdx.x == 0, status);
      if (lane == 0) {
        *item = it;
        *taken = 0;
      }
    } else if (lane == 0) {  // the same order, with CTAs for tiles that shorter requests lack (0.3 us less)
      const int b = u % p.B, first = (p.tiles / p.B - 1 - u / p.B) * (2 * kSub);
      const int a = p.cu_q[b], e = p.cu_q[b + 1], c = p.cu_k[b], f = p.cu_k[b + 1];
      const bool ok = rows_ok(p, a, e, c, f);
      if (!ok) atomicOr(status, FD_DEVSTAT_SEQLEN_OVERFLOW);
      *item = Item{ok && first < e - a ? first : -1, a, e - a, c, f - c};
      *taken = 0;
    }
  } else if (warp == kProducer) {
    if (lane == 0) {
      for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(&kempty[x], 1);
        mbar_init(&vempty[x], 1);
        mbar_init(&qfull[x], 1);
        mbar_init(&sfull[x], 1);
        mbar_init(&pfull[x], 8);
        mbar_init(&ofull[x], 1);
      }
      mbar_init(vfix, 1);
      mbar_init(drain, 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
  } else if (warp == kMma) {
    tmem_alloc(tslot, kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const int i0 = item->i0, q0 = item->q0, Lq = item->Lq;
  int s0 = item->s0, Lk = item->Lk, ahead = Lk - Lq;
  if (i0 < 0) {  // the same for every thread of a cluster
    if (warp == kMma) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  // key tiles that a sub-tile's last row sees
  auto tiles = [&](int x) {
    const int first = i0 + x * kSub;
    if (first >= Lq) return 0;
    const int see = min(Lq, first + kSub) + ahead;
    return see <= 0 ? 0 : (see + kKeys - 1) / kKeys;
  };
  int na = tiles(0), nb = tiles(1), nt = max(na, nb);
  if (SPLIT) {  // this CTA's run of the item's tiles, as if the keys began there
    const int per = (nt + p.ranks - 1) / p.ranks, t0 = rank * per;
    s0 += t0 * kKeys;
    Lk -= t0 * kKeys;
    ahead -= t0 * kKeys;
    na = min(max(na - t0, 0), per);
    nb = min(max(nb - t0, 0), per);
    nt = max(na, nb);
  }

  const int last_valid = Lk - (nt - 1) * kKeys;  // keys of the request in the last tile
  const bool fix = nt > 0 && last_valid < kKeys;
  float row_m = -INFINITY, row_l = 0.f;  // (SPLIT) the softmax threads' row

  if (warp == kProducer) {
    // ======================= TMA producer =======================
    if (nt > 0) {
      const uint64_t pol = l2_policy_evict_normal();
      bool ok = true;
      int last = -1;  // last ring position filled
      if (elect_one()) {
        auto load_q = [&](int x) {
          if ((x == 0 ? na : nb) == 0) return;
          mbar_arrive_expect_tx(&qfull[x], kQBlocks * kSlotBytes);
          for (int c = 0; c < kQBlocks; ++c)
            tma_load_3d(smem + (x * kQBlocks + c) * kSlotBytes, &tmq, c * 64, h, q0 + i0 + x * kSub, &qfull[x], pol);
        };
        load_q(0);
        auto slot = [&](int pos) -> uint8_t * {  // a free slot's address, its barrier armed
          const int s = pos % kSlots;
          if (pos >= kSlots) {  // the tile that held the slot is released
            const int was = pos - kSlots, j = was / 5;
            ok = ok && wait_bar(was % 5 < 3 ? &kempty[j & 1] : &vempty[j & 1], (j >> 1) & 1, p.wait_ns, status, abort_flag);
          }
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
        for (int j = 0; j < nt && ok; ++j) {
          load_k(j);
          if (j == 0) load_q(1);
          for (int c = 0; c < 2 && ok; ++c) {
            const int pos = pos_v(j) + c;
            uint8_t *dst = slot(pos);
            if (dst) tma_load_3d(dst, &tmv, c * 64, h, s0 + j * kKeys, &full[pos % kSlots], pol);
          }
        }
      }
      __syncwarp();
      if (fix) {
        // Rows of the last V tile past the request's keys belong to nobody here
        // and may hold anything; their weight 0 needs them finite.
        const int pos = pos_v(nt - 1);
        for (int c = 0; c < 2; ++c) {
          const int s = (pos + c) % kSlots;
          if (!wait_bar_warp(&full[s], ((pos + c) / kSlots) & 1, p.wait_ns, status, abort_flag)) break;
          uint8_t *v = smem + kOffRing + s * kSlotBytes + last_valid * 128;
          for (int i = lane; i < (kKeys - last_valid) * 8; i += 32)
            reinterpret_cast<uint4 *>(v)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(vfix);
      }
      // The last copy into each slot lands, and the queries, before the CTA reuses or
      // leaves its memory: nobody else waits for them when another warp has given up.
      if (elect_one()) {  // (the same lane as above)
        for (int pos = max(0, last - kSlots + 1); pos <= last; ++pos)
          mbar_wait(&full[pos % kSlots], (pos / kSlots) & 1, status);
        if (na > 0) mbar_wait(&qfull[0], 0, status);
        if (nb > 0) mbar_wait(&qfull[1], 0, status);
      }
      __syncwarp();
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
      auto scores = [&](int x, int j, bool wait_k) {
        if (!ok) return;
        if (j == 0) ok = wait_bar<true>(&qfull[x], 0, p.wait_ns, status, abort_flag);
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const int pos = pos_k(j) + c, s = pos % kSlots;
          if (ok && wait_k) ok = wait_bar<true>(&full[s], (pos / kSlots) & 1, p.wait_ns, status, abort_flag);
          if (!ok) return;
          if (c == 0 || wait_k) tc_fence_after();
          const uint64_t kt = kd + ((s * kSlotBytes) >> 4), qt = qd + (((x * kQBlocks + c) * kSlotBytes) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f16_ss(tmem + x * 128, qt + ((k * 32) >> 4), kt + ((k * 32) >> 4), id_s, (c > 0 || k > 0) ? 1u : 0u);
        }
      };
      auto values = [&](int x, int j, bool wait_v) {
        if (ok) ok = wait_bar<true>(&pfull[x], j & 1, p.wait_ns, status, abort_flag);
        if (!ok) return;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int pos = pos_v(j) + c, s = pos % kSlots;
          if (ok && wait_v) {
            ok = wait_bar<true>(&full[s], (pos / kSlots) & 1, p.wait_ns, status, abort_flag);
            if (ok && c == 0 && fix && j == nt - 1) ok = wait_bar<true>(vfix, 0, p.wait_ns, status, abort_flag);
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
      // One commit a released tile: commits queue behind the MMAs, and the thread behind them.
      auto release_k = [&](int j) { umma_commit(&kempty[j & 1]); };
      auto release_v = [&](int j) { umma_commit(&vempty[j & 1]); };
      if (na > 0) {
        scores(0, 0, true);
        if (ok) umma_commit(&sfull[0]);
      }
      if (nb > 0) {
        scores(1, 0, na == 0);
        if (ok) umma_commit(&sfull[1]);
      }
      if (ok) release_k(0);
      for (int j = 0; j < nt && ok; ++j) {
        // sub-tile 0, then 1: PV(j), S(j + 1); the first to use a tile waits for it, the last frees it
        if (j < na) values(0, j, true);
        if (ok && j + 1 == na) umma_commit(&ofull[0]);
        if (ok && j < na && j >= nb) release_v(j);
        if (ok && j + 1 < na) {
          scores(0, j + 1, true);
          if (ok) umma_commit(&sfull[0]);
          if (ok && j + 1 >= nb) release_k(j + 1);
        }
        if (j < nb) values(1, j, j >= na);
        if (ok && j + 1 == nb) umma_commit(&ofull[1]);
        if (ok && j < nb) release_v(j);
        if (ok && j + 1 < nb) {
          scores(1, j + 1, j + 1 >= na);
          if (ok) umma_commit(&sfull[1]);
          if (ok) release_k(j + 1);
        }
      }
      // MMAs end before TMEM is released
      if (!ok) umma_commit(drain);
      if (!ok || na > 0) mbar_wait(ok ? &ofull[0] : drain, 0, status);
      if (ok && nb > 0) mbar_wait(&ofull[1], 0, status);
    }
    __syncwarp();
  } else {
    // ======================= softmax warps =======================
    // Sub-tile x, half of the keys (and of the output channels), quarter of the
    // rows; the two warps of a quarter agree on the rows' maxima.
    const int x = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, n = x == 0 ? na : nb;
    // A request that begins before the end of an earlier one with good rows owns
    // none of its own: it is recorded, and nothing is written. (find_item gives it
    // no tiles. Here the loads of the queries and keys hide the look at the earlier
    // requests: in front of the first barrier it cost 4000 prompts of 50 tokens 18 %.)
    if (!p.ragged) {
      const int b = unit / p.H % p.B;
      bool late = false;
#pragma unroll 1
      for (int e0 = threadIdx.x; e0 < b; e0 += 8 * kProducer * 32) {
        int end[8];  // the loads first: behind branches each would wait for the one before
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int e = e0 + k * kProducer * 32;
          end[k] = e < b ? p.cu_q[e + 1] : 0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (end[k] > q0) {
            const int e = e0 + k * kProducer * 32;
            late = late || rows_ok(p, p.cu_q[e], end[k], p.cu_k[e], p.cu_k[e + 1]);
          }
      }
      if (late) {
        *taken = 1;
        atomicOr(status, FD_DEVSTAT_SEQLEN_OVERFLOW);
      }
      if (b > 0) named_barrier(9, kProducer * 32);
    }
    const int pair_bar = 1 + x * 4 + quarter;  // named barrier of the two warps
    const int r = quarter * 32 + lane, i = i0 + x * kSub + r;  // this thread's row: TMEM lane r of its sub-tile
    float *swap = reinterpret_cast<float *>(smem + kOffSwap) + x * kSub + r;
    // op(v, the other thread's v) over the row's two threads, through one word
    auto join = [&](float v, auto op) {
      if (half == 0) *swap = v;
      named_barrier(pair_bar, 64);
      if (half == 1) {
        v = op(v, *swap);
        *swap = v;
      }
      named_barrier(pair_bar, 64);
      if (half == 0) v = *swap;
      return v;
    };
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_base + x * 128, to = tmem + lane_base + kTmO + x * 128 + half * 64;
    // keys that the row sees (a row behind the request's last is never written: no mask)
    const int lim = i < Lq ? max(0, min(Lk, i + 1 + ahead)) : 0x7fffffff;
    const int lim_min = __reduce_min_sync(0xffffffffu, lim);
    constexpr int kCols = kKeys / 2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;  // no wait of this warp has run out
    const float2 sc = make_float2(p.scale_log2, p.scale_log2);
    for (int j = 0; j < n; ++j) {
      ok = ok && wait_bar_warp(&sfull[x], j & 1, p.wait_ns, status, abort_flag);
      tc_fence_after();
      float s[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += 32) tmem_ld32(ts + half * kCols + c, s + c);
      tmem_wait_ld();
      const int key0 = j * kKeys + half * kCols;
      if (key0 + kCols > lim_min) {
        const int see = lim - key0, see_min = lim_min - key0;
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 16)
          if (c0 + 16 > see_min) {
#pragma unroll
            for (int c = c0; c < c0 + 16; ++c) s[c] = c < see ? s[c] : -INFINITY;
          }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 60; c += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], s[c + k], s[c + 4 + k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[60 + k]);
      float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
      // (the vote also keeps either warp's weights off scores the other has yet to read)
      if (bar_red_or(pair_bar, 64, top > m + 8.f)) {
        top = join(top, [](float a, float b) { return fmaxf(a, b); });
        const float mn = fmaxf(m, top), f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
        m = mn;
        l *= f;
        if (j > 0) {  // PV(j - 1) is done: S(j) was issued behind it
#pragma unroll 1
          for (int c = 0; c < 64; c += 8) {
            float o[8];
            tmem_ld8(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] *= f;
            tmem_st8(to + c, o);
          }
        }
      }
      const float u = m == -INFINITY ? 0.f : -m;
      const float2 off = make_float2(u, u);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 a = fma2(make_float2(s[c + 2 * k], s[c + 2 * k + 1]), sc, off);
          const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
          sum[k & 1] = add2(sum[k & 1], e);
          w[k] = pack_bf16x2(e.x, e.y);
        }
        tmem_st8u(ts + (half * kCols + c) / 2, w);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&pfull[x]);
    }
    l = join(l, [](float a, float b) { return a + b; });
    if (n > 0) {
      if (ok) wait_bar_warp(&ofull[x], 0, p.wait_ns, status, abort_flag);
      tc_fence_after();
    }
    if (SPLIT) {
      row_m = m;
      row_l = l;
    } else {
      const bool write = i < Lq && *taken == 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;  // l = 0: no visible key; a NaN stays one
      const int64_t at = static_cast<int64_t>(q0 + i) * p.o_ss + h * p.o_sh + half * 64;
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        float o[16];
        if (n > 0) {
          tmem_ld16(to + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = l == 0.f ? 0.f : o[k] * inv;
        if (!write) continue;
        if (p.out_f32) {
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(o[k]);
          store32(static_cast<float *>(p.out) + at + c, v, p.wide);
          store32(static_cast<float *>(p.out) + at + c + 8, v + 8, p.wide);
        } else {
          uint32_t v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = pack_bf16x2(o[2 * k], o[2 * k + 1]);
          store32(static_cast<__nv_bfloat16 *>(p.out) + at + c, v, p.wide);
        }
      }
      if (p.lse && half == 0 && write)
        p.lse[static_cast<int64_t>(q0 + i) * p.l_ss + h * p.l_sh] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
  if (SPLIT) {
    // ======================= join of the ranks =======================
    // Every MMA of this CTA is done behind the barrier: the ring takes its output
    // (row of 512 bytes, 16-byte chunks XORed with the row), the Q tiles the
    // rows' maxima and sums. Then each rank joins 256 / ranks of the rows.
    cg::cluster_group cluster = cg::this_cluster();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    float *const stat = reinterpret_cast<float *>(smem);  // [256] maxima, [256] sums
    if (warp < kProducer) {
      const int x = warp >> 3, half = (warp >> 2) & 1, row = x * kSub + (warp & 3) * 32 + lane;
      const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kTmO + x * 128 + half * 64;
      const int n = x == 0 ? na : nb;
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        float o[16];
        if (n > 0) {
          tmem_ld16(to + c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int chunk = (half * 16 + c / 4 + k) ^ (row & 31);
          *reinterpret_cast<float4 *>(smem + kOffRing + row * 512 + chunk * 16) =
              n > 0 ? make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      if (half == 0) {
        stat[row] = row_m;
        stat[2 * kSub + row] = row_l;
      }
    }
    cluster.sync();
    if (warp < kProducer && *taken == 0) {
      if (p.ranks == 2)
        join_ranks<2>(cluster, smem, stat, p, rank * 128 + warp * 8, q0, i0, Lq, h, lane);
      else if (p.ranks == 4)
        join_ranks<4>(cluster, smem, stat, p, rank * 64 + warp * 4, q0, i0, Lq, h, lane);
      else
        join_ranks<8>(cluster, smem, stat, p, rank * 32 + warp * 2, q0, i0, Lq, h, lane);
    }
    cluster.sync();  // the other ranks have read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// CTAs that share a tile of 256 queries: as many as end first by a count in key
// tiles (1.6 us each; a CTA costs 3 beside its own, 8 with the join), as long as
// all clusters run at once, one CTA on each of 152 SMs (76, 36 and 15 clusters
// of 2, 4 and 8). Measured, with 1 / 2 / 4 / 8 CTAs: 4 heads x 512 queries x
// 32000 keys 396 / 218 / 116 / 66 us, 16 x 512 x 9000 120 / 71 / 42 / 79,
// 16 x 1 x 8192 100 / 56 / 33 / 39, 16 x 128 x 1024 17 / 16 / 12 / 20, 32 x 1024
// x 16384 213 / 234 / 263 / 354, 16 x 2048 x 2048 33 / 35 / 56 / 118. With more
// items it depends on the lengths, which only the device has: four chunks of 700
// queries behind 6300 keys x 16 heads 192 / 175 / 210 / 306, four of 300-1024
// behind 1000-11000 166 / 183 with 1 / 2. (Sk / B stands for the lengths, which
// only the device has; with padded key tensors, or one long request among short
// ones, the choice is that of other lengths, the result the same.)
int ranks_of(const LatentPrefillParams &p) {
  const int64_t items = static_cast<int64_t>(p.tiles) * p.H;  // at most
  const float tiles = static_cast<float>(p.Sk) / (static_cast<float>(p.B) * kKeys);
  const int clusters[4] = {152, 76, 36, 15};
  int ranks = 1;
  float least = tiles + 3.f;
  for (int k = 1; k < 4 && items <= clusters[k]; ++k) {
    const float cost = tiles / (1 << k) + 8.f;
    if (cost < least) {
      least = cost;
      ranks = 1 << k;
    }
  }
  return ranks;
}

}  // namespace

cudaError_t launch_latent_prefill(const CUtensorMap (&tm)[4], LatentPrefillParams p, cudaStream_t stream) {
  p.ranks = ranks_of(p);
  auto *const kernel = p.ranks > 1 ? fd_latent_prefill_kernel<true> : fd_latent_prefill_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.ranks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles) * p.H * p.ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemAlloc;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = p.ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tm[0], tm[1], tm[2], tm[3], p);
}

}  // namespace fd
