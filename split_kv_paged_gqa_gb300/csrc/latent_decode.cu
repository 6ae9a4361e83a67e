// latent_decode.cu - absorbed latent attention over a paged cache on the
// tcgen05 tensor cores (sm_103a).
//
// A token's cache row c_j holds 512 latent and 64 rotary channels. With the
// per-head up-projections absorbed into q, every head attends to the same rows:
//   s_rj = scale * q_r . c_j (576 channels),  o_r = sum_j softmax(s_r)_j c_j[0:512].
// A request's R = Tq * H query rows share its keys, so a row block loaded once
// is key and value of all of them: 1152 bytes and 2176 R flops a key. HBM binds
// below about 150 rows a request; above, the tensor cores do.
//
// Placement: the batch's keys, cut into tiles of 64, form one line of n tiles
// (request after request). CTA group g of G takes tiles [g per, (g + 1) per),
// per = ceil(n / G), whatever requests they belong to, so every SM gets the
// same work for any mix of lengths; G groups of one CTA per row tile fill the
// SMs once. A CTA's piece of a request is final when it holds the whole
// request; else it is a partial (fp32, with its LSE) and the merge kernel joins
// them. A CTA has at most two partials: one that continues an earlier CTA's
// request (slot 0) and one that starts a request (slot 1).
//
// One CTA = 4 softmax warps, a TMA producer warp and an MMA warp, for at most
// 64 query rows:
//  * K/V tile j lands in one of two 72 KB stages as nine K-major column blocks
//    of 64 channels (128-byte swizzle): five slots with barriers of their own
//    (four of 128 latent channels, one of the 64 rotary ones), so the scores
//    start on the first slot and each slot is refilled as soon as it is free.
//  * scores S = Q K^T: M = 64 rows, N = 64 keys, 36 K steps (fp32 in TMEM, two
//    buffers).
//  * softmax: each warp owns 16 rows (four threads a row). The running maximum
//    moves only when a row outgrows it by 2^8 (lazy rescale); weights are
//    rounded to bf16, the tensor core's operand type beside bf16 values
//    (at most 2^-8 of each weight); their sum and the LSE stay fp32 and use
//    the unrounded weights.
//  * O^T += V^T P^T: the same K tile read MN-major, M = 128 of the 512 value
//    channels at a time, N = the CTA's rows (a multiple of 16): 4 x N columns
//    of TMEM. V is never transposed or copied.
#include <math.h>

#include "fd.h"
#include "latent.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace fd {
namespace {

constexpr int kTile = 64;                      // keys per tile
constexpr int kRows = kLatRowTile;             // query rows per CTA at most
constexpr int kBlock = kTile * 128;            // bytes of one 64-channel column block of a tile
constexpr int kBlocks = kLatRow / 64;          // 9
constexpr int kSlots = 5;                      // barrier slots of a stage: 4 x 128 channels, 1 x 64
constexpr int kStages = 2;
constexpr int kStageBytes = kBlocks * kBlock;  // 73,728
constexpr int kSoftWarps = 4, kProducer = 4, kMma = 5;
constexpr int kThreads = 192;
constexpr int kOffQ = kStages * kStageBytes;
constexpr int kOffP = kOffQ + kBlocks * kRows * 128;
constexpr int kOffRow = kOffP + kRows * kTile * 2;       // int64 [64] output offset of a row (-1: padding)
constexpr int kOffF = kOffRow + kRows * 8;               // float [64] rescale factors, later 1 / sum
constexpr int kOffBar = kOffF + kRows * 4;
constexpr int kBars = 2 * kStages * kSlots + 2 + 3;      // full, empty, sfull[2], pfull, ofull, qfull
constexpr int kOffMisc = kOffBar + kBars * 8;            // TMEM address, abort word
constexpr int kSmem = kOffMisc + 16;
constexpr int kSmemAlloc = kSmem + 1024;                 // slack to align the base to 1024
static_assert(kSmemAlloc <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kTmS = 256;          // O^T: 4 x 64 columns from 0; S: 2 x 64 from 256

__device__ __forceinline__ int load_len(const LatentDecodeParams &p, int b) {
  const int L = ld_cg(p.seqlens + b * p.sl_s), cap = p.max_pages * p.page_size;
  return L < 0 ? 0 : (L > cap ? cap : L);
}

__device__ __forceinline__ int tiles_of(int L) { return (L + kTile - 1) / kTile; }

// Tiles per CTA group of a batch of n tiles.
__device__ __forceinline__ long long tiles_per_group(long long n, int groups) {
  const long long per = (n + groups - 1) / groups;
  return per < 1 ? 1 : per;
}

// A CTA's walk over its pieces: request b, tiles [t0, t1), length L.
struct Piece {
  int b, t0, t1, L;
};

struct Walk {
  int b;           // request of the next piece
  int t0;          // its first tile
  long long left;  // tiles not yet taken
};

// The start of group g's range: total tiles, then the request that holds the
// range's first tile. Warp-collective (all lanes, same arguments). Four
// lengths a lane: one round trip for up to 128 requests.
__device__ __forceinline__ Walk locate(const LatentDecodeParams &p, int g, int lane) {
  int first[4];
  long long n = 0;
  for (int i0 = 0; i0 < p.B; i0 += 128) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + 4 * lane + k;
      const int t = i < p.B ? tiles_of(load_len(p, i)) : 0;
      if (i0 == 0) first[k] = t;
      n += t;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  const long long per = tiles_per_group(n, p.groups);
  const long long start = g * per;
  Walk w;
  w.b = p.B;
  w.t0 = 0;
  w.left = n - start < per ? n - start : per;
  if (w.left <= 0) {
    w.left = 0;
    return w;
  }
  long long base = 0;
  for (int i0 = 0; i0 < p.B; i0 += 128) {
    int t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + 4 * lane + k;
      t[k] = i0 == 0 ? first[k] : (i < p.B ? tiles_of(load_len(p, i)) : 0);
    }
    const long long mine = static_cast<long long>(t[0]) + t[1] + t[2] + t[3];
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > start);
    if (hit) {
      const int src = __ffs(hit) - 1;
      long long at = base + incl - mine;  // tiles before this lane's requests
      int k = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (k == i && at + t[i] <= start) {
          at += t[i];
          ++k;
        }
      w.b = __shfl_sync(0xffffffffu, i0 + 4 * lane + k, src);
      w.t0 = __shfl_sync(0xffffffffu, static_cast<int>(start - at), src);
      return w;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  w.left = 0;
  return w;
}

__device__ __forceinline__ bool next_piece(const LatentDecodeParams &p, Walk &w, Piece &out) {
  if (w.left <= 0) return false;
  for (; w.b < p.B; ++w.b, w.t0 = 0) {
    const int L = load_len(p, w.b), nt = tiles_of(L);
    if (w.t0 >= nt) continue;
    const long long room = nt - w.t0;
    const int take = static_cast<int>(room < w.left ? room : w.left);
    out.b = w.b;
    out.t0 = w.t0;
    out.t1 = w.t0 + take;
    out.L = L;
    w.left -= take;
    ++w.b;
    w.t0 = 0;
    return true;
  }
  return false;
}

// Bounded wait that gives up at once when another warp of the CTA has: after a
// timeout every warp runs to the end without waiting.
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
    fd_latent_decode_kernel(const __grid_constant__ CUtensorMap tmc, const __grid_constant__ LatentDecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  int64_t *row_off = reinterpret_cast<int64_t *>(smem + kOffRow);
  float *factor = reinterpret_cast<float *>(smem + kOffF);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);  // [stage][slot]: the slot's bytes have landed
  uint64_t *empty = full + kStages * kSlots;                      // [stage][slot]: its MMAs are done
  uint64_t *sfull = empty + kStages * kSlots;                     // [2]: scores of tile j in buffer j % 2
  uint64_t *pfull = sfull + 2;                                    // weights of tile j written
  uint64_t *ofull = pfull + 1;                                    // O holds tile j
  uint64_t *qfull = ofull + 1;                                    // queries of the next piece written
  uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = blockIdx.x % p.row_tiles, g = blockIdx.x / p.row_tiles;
  const int row0 = rt * p.rows_per_tile;
  const int nrows = min(p.rows_per_tile, p.R - row0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages * kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&sfull[0], 1);
    mbar_init(&sfull[1], 1);
    mbar_init(pfull, kSoftWarps);
    mbar_init(ofull, 1);
    mbar_init(qfull, kSoftWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  // Requests without keys: zeros, lse -inf; a length out of range is recorded.
  for (int b = g; b < p.B; b += p.groups) {
    const int raw = ld_cg(p.seqlens + b * p.sl_s);
    if (raw > 0) {
      if (threadIdx.x == 0 && raw > p.max_pages * p.page_size) atomicOr(p.status, FD_DEVSTAT_SEQLEN_OVERFLOW);
      continue;
    }
    if (threadIdx.x == 0 && raw < 0) atomicOr(p.status, FD_DEVSTAT_SEQLEN_OVERFLOW);
    for (int i = threadIdx.x; i < nrows * kLatC; i += kThreads) {
      const int rg = row0 + i / kLatC, t = rg / p.H, h = rg - t * p.H;
      const int64_t at = b * p.o_sb + t * p.o_st + h * p.o_sh + i % kLatC;
      if (p.out_f32) static_cast<float *>(p.out)[at] = 0.f;
      else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(0.f);
      if (p.lse && i % kLatC == 0) p.lse[b * p.l_sb + t * p.l_st + h * p.l_sh] = -INFINITY;
    }
  }
  Walk walk = locate(p, g, lane);
  if (walk.left <= 0) return;  // the same for every thread of the CTA
  if (warp == kMma) tmem_alloc(tslot, kTmemCols);
  if (warp < kSoftWarps) {  // padding rows of Q read as zero
    for (int i = threadIdx.x; i < (kRows - nrows) * (kLatRow / 8); i += kSoftWarps * 32) {
      const int r = nrows + i / (kLatRow / 8), c = i % (kLatRow / 8);
      *reinterpret_cast<uint4 *>(smem + kOffQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  if (warp == kProducer) {
    // ======================= TMA producer =======================
    if (lane == 0) tma_prefetch_desc(&tmc);
    // one CTA reads a tile when there is one row tile; else its neighbours do soon
    const uint64_t pol = p.row_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
    const int P = p.page_size;
    const int log2_seg = p.log2_page < 6 ? p.log2_page : 6, seg = 1 << log2_seg;  // keys per TMA box
    const int i = lane & 7, blk = lane >> 3;  // this lane's segment of the tile (at most 8) and block of the slot
    Piece pc;
    int j = 0, last_stage_slot = -1;
    bool ok = true;
    while (ok && next_piece(p, walk, pc)) {
      const int *pt = p.page_table + pc.b * p.pt_sb;
      auto ld_pid = [&](int t) {
        const int key = t * kTile + (i << log2_seg);
        return i < (kTile >> log2_seg) && key < pc.L ? pt[key >> p.log2_page] : 0;
      };
      int pid_next = ld_pid(pc.t0);
      for (int t = pc.t0; ok && t < pc.t1; ++t, ++j) {
        int pid = pid_next;
        if (t + 1 < pc.t1) pid_next = ld_pid(t + 1);
        const int tok0 = t * kTile, nseg = (min(kTile, pc.L - tok0) + seg - 1) >> log2_seg;
        const bool mine = i < nseg;
        const bool bad = mine && (pid < 0 || pid >= p.num_pages);
        if (bad) pid = p.num_pages;  // outside the pool: record, and let TMA zero-fill
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
        const int stage = j % kStages;
        const unsigned ph = (j / kStages) & 1;
#pragma unroll 1
        for (int s = 0; s < kSlots; ++s) {
          uint64_t *fb = &full[stage * kSlots + s];
          if (!wait_bar_warp(&empty[stage * kSlots + s], ph ^ 1, p.status, abort_flag)) {
            ok = false;
            break;
          }
          const int blocks = s < 4 ? 2 : 1;
          if (lane == 0) mbar_arrive_expect_tx(fb, static_cast<unsigned>(blocks * nseg * seg * 128));
          __syncwarp();
          if (mine && blk < blocks) {
            const int c = 2 * s + blk;
            tma_load_3d(smem + stage * kStageBytes + c * kBlock + (i << log2_seg) * 128, &tmc, c * 64,
                        (tok0 + (i << log2_seg)) & (P - 1), pid, fb, pol);
          }
          last_stage_slot = j * kSlots + s;
        }
      }
    }
    if (!ok && lane == 0) {  // given up: the copies in flight land before the CTA ends
      for (int k = max(0, last_stage_slot - kStages * kSlots + 1); k <= last_stage_slot; ++k)
        mbar_wait(&full[(k / kSlots % kStages) * kSlots + k % kSlots], (k / kSlots / kStages) & 1, p.status);
    }
    __syncwarp();
  } else if (warp == kMma) {
    // ======================= MMA issuer =======================
    // Whatever is ready goes first, PV before scores: a PV frees the slots that
    // the producer waits for.
    if (lane == 0) {
      const uint32_t base = smem_u32(smem);
      const uint64_t qd = umma_desc_sw128(base + kOffQ), pd = umma_desc_sw128(base + kOffP);
      const uint64_t kd = umma_desc_sw128(base), vd = umma_desc_sw128_mn(base, kBlock, 1024);
      const uint32_t id_s = umma_idesc_bf16(64, kTile, false, false);
      const uint32_t id_o = umma_idesc_bf16(128, p.rows_per_tile, true, false);
      const int n_tiles = static_cast<int>(walk.left);
      Piece pc;
      next_piece(p, walk, pc);
      int piece_end = pc.t1 - pc.t0;  // the CTA's first tile behind the piece whose scores are being issued
      int jq = 0, slot = 0, piece = 0, jo = 0;
      unsigned starts = 1u;  // bit j % 4: tile j starts a piece
      bool q_ready = false;
      uint64_t *last_bar = nullptr;  // the barrier and phase of the last commit
      unsigned last_par = 0;
      unsigned long long idle = 0;
      while (jo < n_tiles) {
        bool moved = false;
        if (jo < jq && mbar_test(pfull, jo & 1)) {
          tc_fence_after();
          const uint32_t st = ((jo % kStages) * kStageBytes) >> 4;
          const uint32_t fresh = (starts >> (jo & 3)) & 1u;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              umma_f16_ss(tmem + d * kRows, vd + st + ((d * 2 * kBlock + k * 2048) >> 4), pd + ((k * 32) >> 4), id_o,
                          (k > 0 || !fresh) ? 1u : 0u);
            umma_commit(&empty[(jo % kStages) * kSlots + d]);
          }
          umma_commit(ofull);
          last_bar = ofull;
          last_par = jo & 1;
          ++jo;
          moved = true;
        } else if (jq < n_tiles && jq < jo + 2) {
          // scores of tile jq: its buffer was read by the softmax of tile jq - 2,
          // whose weights PV(jq - 2) has taken
          if (!q_ready && mbar_test(qfull, piece & 1)) q_ready = true;
          if (q_ready && mbar_test(&full[(jq % kStages) * kSlots + slot], (jq / kStages) & 1)) {
            tc_fence_after();
            const uint32_t st = ((jq % kStages) * kStageBytes + slot * 2 * kBlock) >> 4;
            const uint32_t dst = tmem + kTmS + (jq & 1) * kTile;
            const uint32_t qs = (slot * 2 * kRows * 128) >> 4;
            if (slot < 4) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_f16_ss(dst, qd + qs + (((k >> 2) * kRows * 128 + (k & 3) * 32) >> 4),
                            kd + st + (((k >> 2) * kBlock + (k & 3) * 32) >> 4), id_s, (slot > 0 || k > 0) ? 1u : 0u);
              ++slot;
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f16_ss(dst, qd + qs + ((k * 32) >> 4), kd + st + ((k * 32) >> 4), id_s, 1u);
              umma_commit(&empty[(jq % kStages) * kSlots + 4]);
              umma_commit(&sfull[jq & 1]);
              last_bar = &sfull[jq & 1];
              last_par = (jq >> 1) & 1;
              slot = 0;
              ++jq;
              starts &= ~(1u << (jq & 3));
              if (jq == piece_end && jq < n_tiles) {
                next_piece(p, walk, pc);
                piece_end += pc.t1 - pc.t0;
                starts |= 1u << (jq & 3);
                ++piece;
                q_ready = false;
              }
            }
            moved = true;
          }
        }
        if (moved) {
          idle = 0;
        } else {
          if (*abort_flag) break;
          const unsigned long long now = globaltimer_ns();
          if (idle == 0) {
            idle = now;
          } else if (now - idle > kWaitLimitNs) {
            atomicOr(p.status, FD_DEVSTAT_WAIT_TIMEOUT);
            *abort_flag = 1;
            break;
          }
        }
      }
      // every MMA issued has completed before TMEM is released
      if (last_bar) mbar_wait(last_bar, last_par, p.status);
    }
    __syncwarp();
  } else {
    // ======================= softmax warps =======================
    const uint32_t to = tmem + (static_cast<uint32_t>(warp * 32) << 16);  // this thread's value channels
    const uint32_t ts = to + kTmS;                                        // this warp's 16 rows of scores
    const bool live = warp * 16 < nrows, ragged = warp * 16 + 16 > nrows;
    const int ra = warp * 16 + (lane >> 2), rb = ra + 8;  // this thread's rows of the tile
    const int qcol = (lane & 3) * 2;
    const int npad = p.rows_per_tile;
    auto load_q = [&](const Piece &pc) {
      for (int i = threadIdx.x; i < nrows * (kLatRow / 8); i += kSoftWarps * 32) {
        const int r = i / (kLatRow / 8), c = i % (kLatRow / 8), rg = row0 + r;
        const int t = rg / p.H, h = rg - t * p.H;
        cp_async_ca<16>(smem + kOffQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                        p.q + pc.b * p.q_sb + t * p.q_st + h * p.q_sh + c * 8);
      }
    };
    auto publish_q = [&] {
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
    };
    Piece pc;
    bool more = next_piece(p, walk, pc);
    load_q(pc);
    publish_q();
    int j = 0;
    while (more) {
      // where this piece's rows go (read in the epilogue)
      const bool whole = pc.t0 == 0 && pc.t1 == tiles_of(pc.L);
      const int64_t part_row = (static_cast<int64_t>(2 * g + (pc.t0 == 0 ? 1 : 0)) * p.row_tiles + rt) * kRows;
      named_barrier(1, kSoftWarps * 32);  // the epilogue before has read factor and row_off
      if (threadIdx.x < kRows) {
        const int r = threadIdx.x, rg = row0 + r, t = rg / p.H, h = rg - t * p.H;
        row_off[r] = r >= nrows ? -1 : whole ? pc.b * p.o_sb + t * p.o_st + h * p.o_sh : (part_row + r) * kLatC;
      }
      const int lima = ra < nrows ? pc.L - (p.Tq - 1) + (row0 + ra) / p.H : 0;
      const int limb = rb < nrows ? pc.L - (p.Tq - 1) + (row0 + rb) / p.H : 0;
      const int limmin = pc.L - (p.Tq - 1) + row0 / p.H;  // the tile's first row sees the fewest keys
      float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
      for (int t = pc.t0; t < pc.t1; ++t, ++j) {
        const int tok0 = t * kTile;
        wait_bar_warp(&sfull[j & 1], (j >> 1) & 1, p.status, abort_flag);
        tc_fence_after();
        float v[32];
        float xa = -INFINITY, xb = -INFINITY;
        if (live) {
          tmem_ld_16x64(ts + (j & 1) * kTile, v);
          tmem_wait_ld();
          if (tok0 + kTile > limmin || ragged) {  // some key is past some row's limit, or a row is padding
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int k0 = tok0 + 8 * c + qcol;
              v[4 * c] = k0 < lima ? v[4 * c] : -INFINITY;
              v[4 * c + 1] = k0 + 1 < lima ? v[4 * c + 1] : -INFINITY;
              v[4 * c + 2] = k0 < limb ? v[4 * c + 2] : -INFINITY;
              v[4 * c + 3] = k0 + 1 < limb ? v[4 * c + 3] : -INFINITY;
            }
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            xa = fmaxf(xa, fmaxf(v[4 * c], v[4 * c + 1]));
            xb = fmaxf(xb, fmaxf(v[4 * c + 2], v[4 * c + 3]));
          }
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2)) * p.scale_log2;
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2)) * p.scale_log2;
        }
        if (bar_red_or(1, kSoftWarps * 32, xa > ma + 8.f || xb > mb + 8.f)) {
          // some row outgrew its maximum by 2^8: every row takes its new one
          const float na = fmaxf(ma, xa), nb = fmaxf(mb, xb);
          const float fa = na == -INFINITY ? 1.f : fast_exp2(ma - na), fb = nb == -INFINITY ? 1.f : fast_exp2(mb - nb);
          ma = na;
          mb = nb;
          la *= fa;
          lb *= fb;
          if (t > pc.t0) {  // scale the sums so far, once PV(j - 1) is in
            if ((lane & 3) == 0) {
              factor[ra] = fa;
              factor[rb] = fb;
            }
            named_barrier(1, kSoftWarps * 32);
            wait_bar_warp(ofull, (j - 1) & 1, p.status, abort_flag);
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < 4; ++d)
#pragma unroll 1
              for (int c = 0; c < npad; c += 16) {
                float o[16];
                tmem_ld16(to + d * kRows + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= factor[c + i];
                tmem_st16(to + d * kRows + c, o);
              }
            tmem_wait_st();
          }
        }
        const float ua = ma == -INFINITY ? 0.f : ma, ub = mb == -INFINITY ? 0.f : mb;
        uint32_t wa[8], wb[8];
        if (live) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float e0 = fast_exp2(fmaf(v[4 * c], p.scale_log2, -ua));
            const float e1 = fast_exp2(fmaf(v[4 * c + 1], p.scale_log2, -ua));
            const float e2 = fast_exp2(fmaf(v[4 * c + 2], p.scale_log2, -ub));
            const float e3 = fast_exp2(fmaf(v[4 * c + 3], p.scale_log2, -ub));
            la += e0 + e1;
            lb += e2 + e3;
            wa[c] = pack_bf16x2(e0, e1);
            wb[c] = pack_bf16x2(e2, e3);
          }
        }
        // the P buffer is free once PV(j - 1) has read it
        if (j > 0) wait_bar_warp(ofull, (j - 1) & 1, p.status, abort_flag);
        if (live) {
          uint8_t *pa = smem + kOffP + ra * 128 + 2 * qcol, *pb = pa + 8 * 128;  // rows 8 apart share the swizzle phase
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            *reinterpret_cast<uint32_t *>(pa + ((c ^ (ra & 7)) << 4)) = wa[c];
            *reinterpret_cast<uint32_t *>(pb + ((c ^ (ra & 7)) << 4)) = wb[c];
          }
        }
        const int valid = pc.L - tok0;
        if (valid < kTile) {  // value rows past the request's keys may hold anything: weight 0 needs them finite
          uint8_t *st = smem + (j % kStages) * kStageBytes;
          for (int i = threadIdx.x; i < (kTile - valid) * 64; i += kSoftWarps * 32)
            *reinterpret_cast<uint4 *>(st + ((i & 63) >> 3) * kBlock + (valid + (i >> 6)) * 128 + ((i & 7) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
      }
      // ---- the next piece's queries are fetched while the last PV runs
      const Piece cur = pc;
      more = next_piece(p, walk, pc);
      if (more) load_q(pc);
      // ---- epilogue: normalise O^T and write this piece's rows
      la += __shfl_xor_sync(0xffffffffu, la, 1);
      lb += __shfl_xor_sync(0xffffffffu, lb, 1);
      la += __shfl_xor_sync(0xffffffffu, la, 2);
      lb += __shfl_xor_sync(0xffffffffu, lb, 2);
      named_barrier(1, kSoftWarps * 32);  // every rescale has read factor
      if ((lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i ? rb : ra;
          const float l = i ? lb : la, m = i ? mb : ma;
          factor[r] = l > 0.f ? 1.f / l : 0.f;
          const float lse = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
          if (r < nrows) {
            const int rg = row0 + r, tq = rg / p.H, h = rg - tq * p.H;
            if (!whole) p.lse_part[part_row + r] = lse;
            else if (p.lse) p.lse[cur.b * p.l_sb + tq * p.l_st + h * p.l_sh] = lse;
          }
        }
      }
      wait_bar_warp(ofull, (j - 1) & 1, p.status, abort_flag);
      tc_fence_after();
      named_barrier(1, kSoftWarps * 32);
      const bool bf = whole && !p.out_f32;
      float *const of = whole ? static_cast<float *>(p.out) : p.o_part;
      __nv_bfloat16 *const ob = static_cast<__nv_bfloat16 *>(p.out);
#pragma unroll 1
      for (int d = 0; d < 4; ++d) {
        const int ch = d * 128 + warp * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < npad; c += 16) {
          float o[16];
          tmem_ld16(to + d * kRows + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int64_t at = row_off[c + i];
            if (at >= 0) {
              const float x = o[i] * factor[c + i];
              if (bf) ob[at + ch] = __float2bfloat16_rn(x);
              else of[at + ch] = x;
            }
          }
        }
      }
      tc_fence_before();  // O is read before the next piece's PV overwrites it
      if (more) publish_q();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of a request's partials: out = sum_c w_c o_c / sum_c w_c with
// w_c = exp(lse_c - max_c lse_c). Threads work in four groups of 128, four
// channels a thread: with many rows each group has a row of its own, with few
// the groups share one row's partials (more loads in flight; joined in shared
// memory). A request that lies in one CTA's range was written by it, one
// without keys too.
constexpr int kMergeThreads = 512, kMergeGroups = kMergeThreads / 128;

__global__ void __launch_bounds__(kMergeThreads) fd_latent_merge_kernel(const __grid_constant__ LatentDecodeParams p) {
  __shared__ float4 acc_s[kMergeGroups][128];
  __shared__ float z_s[kMergeGroups];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const int r = p.merge_rows == 1 ? blockIdx.x : blockIdx.x * kMergeGroups + grp, b = blockIdx.y;
  // The lengths are read before the wait: the decode kernel triggers this grid
  // only after its own dependency wait and does not write them.
  long long n = 0, before = 0;
  for (int i = lane; i < p.B; i += 32) {
    const int t = tiles_of(load_len(p, i));
    n += t;
    before += i < b ? t : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    n += __shfl_xor_sync(0xffffffffu, n, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  const int mine = tiles_of(load_len(p, b));
  const long long per = tiles_per_group(n, p.groups);
  const int c0 = static_cast<int>(before / per), c1 = mine ? static_cast<int>((before + mine - 1) / per) : c0;
  griddep_wait();  // in every CTA: this grid must not end before the decode kernel's
  if (c0 == c1) return;
  const bool one = p.merge_rows == 1;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float Z = 0.f, M = -INFINITY;
  if (r < p.R) {
    const int rt = r / p.rows_per_tile;
    const int64_t row = (static_cast<int64_t>(2 * c0) * p.row_tiles + rt) * kRows + (r - rt * p.rows_per_tile);
    const int64_t stride = static_cast<int64_t>(2 * p.row_tiles) * kRows;  // rows from one CTA group to the next
    const int64_t slot1 = static_cast<int64_t>(p.row_tiles) * kRows;       // slot 1 lies behind slot 0
    const int np = c1 - c0 + 1;
    auto part = [&](int c) { return row + c * stride + (c == 0 ? slot1 : 0); };
    for (int c = lane; c < np; c += 32) M = fmaxf(M, p.lse_part[part(c)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M > -INFINITY) {
      const int step = one ? kMergeGroups : 1;
#pragma unroll 8
      for (int c = one ? grp : 0; c < np; c += step) {
        const float w = expf(p.lse_part[part(c)] - M);  // exp(-inf) = 0; its partial is a finite 0
        const float4 o = *reinterpret_cast<const float4 *>(p.o_part + part(c) * kLatC + tid * 4);
        Z += w;
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
      }
    }
  }
  if (one) {
    acc_s[grp][tid] = acc;
    if (tid == 0) z_s[grp] = Z;
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int k = 1; k < kMergeGroups; ++k) {
      const float4 o = acc_s[k][tid];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
      Z += z_s[k];
    }
  }
  if (r >= p.R) return;
  const float inv = Z > 0.f ? 1.f / Z : 0.f;
  const int t = r / p.H, h = r - t * p.H;
  const int64_t at = b * p.o_sb + t * p.o_st + h * p.o_sh + tid * 4;
  if (p.out_f32)
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (tid == 0 && p.lse) p.lse[b * p.l_sb + t * p.l_st + h * p.l_sh] = Z > 0.f ? M + logf(Z) : -INFINITY;
}

}  // namespace

cudaError_t latent_decode_prepare() {
  return cudaFuncSetAttribute(fd_latent_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
}

cudaError_t launch_latent_decode(const CUtensorMap &tmc, LatentDecodeParams p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.groups * p.row_tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemAlloc;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // rows enough to fill the SMs with one 128-thread group each: a row per group
  p.merge_rows = static_cast<int64_t>(p.B) * p.R > 1216 ? kMergeGroups : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fd_latent_decode_kernel, tmc, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>((p.R + p.merge_rows - 1) / p.merge_rows), static_cast<unsigned>(p.B));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fd_latent_merge_kernel, p);
}

}  // namespace fd
