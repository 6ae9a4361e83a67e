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
// Placement: the batch's keys, cut into tiles of 64, form one line of n places
// (request after request). CTA group g of G takes places [g per, (g + 1) per),
// per = ceil(n / G), whatever requests they belong to, so every SM gets the
// same work for any mix of lengths; G groups of one CTA per row tile fill the
// SMs once. Ahead of each request's tiles the line has p.change places without
// one, for a CTA's change to it (its queries, the pipeline's refill, one more
// epilogue: 4.6 us at 64 rows, tiles 1.6): 1 place at 16 rows, 3 at 64 (64 rows,
// 24 x 4000 keys without 38.9 us, with 36.0; 16 rows, 200 x 300 keys 31.0 and
// 28.0). A CTA's piece of a request is final when it holds the whole request;
// else it is a partial (fp32, with its LSE) and the merge kernel joins them. A CTA has at most two partials: one that continues an earlier CTA's
// request (slot 0) and one that starts a request (slot 1).
//
// One CTA = 8 softmax warps, a TMA producer warp and two MMA warps, for at most
// 64 query rows:
//  * K/V tile j lands in one of two 72 KB stages as nine column blocks of 64
//    channels (128-byte swizzle, atoms of 8 keys). TMA boxes are as large as the
//    layout allows, because a box of one block (8 KB) costs as much issue time
//    as one of three: 8 KB boxes streamed at 6.6 TB/s in a copy loop of this
//    shape, 24 KB boxes at 7.2. A box is three blocks x 64 keys of a page, or x 8
//    keys for pages under 64 (24 x 4000 keys in pages of 8, 16, 32, 64: 39.3, 39.6,
//    39.2, 39.8 us a call). A stage is three slots of three blocks, each with
//    barriers of its own, so the scores start on the first slot and each slot is
//    refilled as soon as it is free.
//  * scores S = Q K^T: M = 64 rows, N = 64 keys, 36 K steps (fp32 in TMEM, two
//    buffers).
//  * softmax: each warp owns 16 rows x 32 keys (four threads a row). The running
//    maximum moves only when a row outgrows it by 2^8 (lazy rescale), so the
//    common tile needs one vote and no exchange of maxima; weights are
//    rounded to bf16, the tensor core's operand type beside bf16 values
//    (at most 2^-8 of each weight); their sum and the LSE stay fp32 and use
//    the unrounded weights.
//  * O^T += V^T P^T: the same K tile read MN-major, M = 128 of the 512 value
//    channels at a time, N = the CTA's rows (a multiple of 16): 4 x N columns
//    of TMEM. V is never transposed or copied.
#include <math.h>

#include <initializer_list>

#include "fd.h"
#include "latent.h"
#include "latent_ptx.cuh"
#include "tc.cuh"

namespace fd {
namespace {

constexpr int kTile = 64;                      // keys per tile
constexpr int kRows = kLatRowTile;             // query rows per CTA at most
constexpr int kBlock = kTile * 128;            // bytes of one 64-channel column block of a tile
constexpr int kBlocks = kLatRow / 64;          // 9
constexpr int kSlots = 3;                      // barrier slots of a stage, three blocks each
constexpr int kStages = 2;
constexpr int kStageBytes = kBlocks * kBlock;  // 73,728
constexpr int kSoftWarps = 8, kProducer = 8, kQk = 9, kPv = 10;
constexpr int kSoftThreads = kSoftWarps * 32, kThreads = kSoftThreads + 96;
constexpr int kOffQ = kStages * kStageBytes;
constexpr int kOffP = kOffQ + kBlocks * kRows * 128;
constexpr int kOffRow = kOffP + kRows * kTile * 2;       // int64 [64] output offset of a row (-1: padding)
constexpr int kOffF = kOffRow + kRows * 8;               // float [64] rescale factors, later 1 / sum
constexpr int kOffRed = kOffF + kRows * 4;                // float [2][64] row maxima or sums of the two key halves
constexpr int kOffBar = kOffRed + 2 * kRows * 4;
constexpr int kBars = 2 * kStages * kSlots + 4 + 3;      // full, empty, sfull[2], sfree[2], pfull, ofull, qfull
constexpr int kOffMisc = kOffBar + kBars * 8;            // TMEM address, abort word
constexpr int kOffDrain = kOffMisc + 16;
constexpr int kSmem = kOffDrain + 16;
constexpr int kSmemAlloc = kSmem + 1024;                 // slack to align the base to 1024
static_assert(kSmemAlloc <= 227 * 1024, "shared memory");
constexpr uint32_t kTmemCols = 512, kTmS = 256;          // O^T: 4 x 64 columns from 0; S: 2 x 64 from 256

__device__ __forceinline__ int load_len(const LatentDecodeParams &p, int b) {
  const int L = ld_cg(p.seqlens + b * p.sl_s), cap = p.max_pages * p.page_size;
  return L < 0 ? 0 : (L > cap ? cap : L);
}

__device__ __forceinline__ int tiles_of(int L) { return (L + kTile - 1) / kTile; }

// A request's places in the line: its tiles, behind p.change places for a CTA's
// change to it.
__device__ __forceinline__ int places_of(const LatentDecodeParams &p, int L) { return L > 0 ? tiles_of(L) + p.change : 0; }

// Places per CTA group of a line of n (n < 2^31: checked by the caller against
// the page table's capacity).
__device__ __forceinline__ int tiles_per_group(int n, int groups) {
  const int per = static_cast<int>((static_cast<unsigned>(n) + groups - 1) / static_cast<unsigned>(groups));
  return per < 1 ? 1 : per;
}

// A CTA's walk over its pieces: request b, tiles [t0, t1), length L.
struct Piece {
  int b, t0, t1, L;
};

struct Walk {
  int b;     // request of the next piece
  int t0;    // its first tile
  int left;  // places not yet taken
  int L;     // length of request b, if known (-1)
};

// The start of group g's range: total places, then the request that holds the
// range's first; left = 0 when no tile lies in the range. Warp-collective (all lanes, same arguments). Four
// lengths a lane: one round trip for up to 128 requests.
__device__ __forceinline__ Walk locate(const LatentDecodeParams &p, int g, int lane) {
  int len[4];
  auto load = [&](int i0) {  // the four loads first: behind branches each would wait for the one before
#pragma unroll
    for (int k = 0; k < 4; ++k) len[k] = load_len(p, min(i0 + 4 * lane + k, p.B - 1));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + 4 * lane + k >= p.B) len[k] = 0;
    return places_of(p, len[0]) + places_of(p, len[1]) + places_of(p, len[2]) + places_of(p, len[3]);
  };
  const int mine0 = load(0);
  int n = mine0;
#pragma unroll 1
  for (int i0 = 128; i0 < p.B; i0 += 128) n += load(i0);
  n = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
  const int per = tiles_per_group(n, p.groups);
  Walk w;
  w.b = p.B;
  w.t0 = 0;
  w.left = 0;
  w.L = -1;
  const long long start_ll = static_cast<long long>(g) * per;
  if (start_ll >= n) return w;
  const int start = static_cast<int>(start_ll);
  w.left = min(per, n - start);
  int base = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < p.B; i0 += 128) {
    const int mine = i0 == 0 && p.B <= 128 ? mine0 : load(i0);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > start);
    if (hit) {
      const int src = __ffs(hit) - 1;
      int at = base + incl - mine, k = 0, L = len[0];  // places before this lane's requests
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (k == i && at + places_of(p, len[i]) <= start) {
          at += places_of(p, len[i]);
          ++k;
          L = len[i + 1];
        }
      w.b = __shfl_sync(0xffffffffu, i0 + 4 * lane + k, src);
      w.t0 = __shfl_sync(0xffffffffu, start - at, src) - p.change;
      w.L = __shfl_sync(0xffffffffu, L, src);
      if (w.t0 < 0) {  // the range starts within the request's change places
        w.left = max(0, w.left + w.t0);
        w.t0 = 0;
      }
      return w;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  w.left = 0;
  return w;
}

__device__ __forceinline__ bool next_piece(const LatentDecodeParams &p, Walk &w, Piece &out) {
  if (w.left <= 0) return false;
#pragma unroll 1
  for (; w.b < p.B; ++w.b, w.t0 = 0, w.L = -1) {
    const int L = w.L >= 0 ? w.L : load_len(p, w.b), nt = tiles_of(L);
    if (w.t0 >= nt) continue;
    const int take = min(nt - w.t0, w.left);
    out.b = w.b;
    out.t0 = w.t0;
    out.t1 = w.t0 + take;
    out.L = L;
    w.left -= take + p.change;
    ++w.b;
    w.t0 = 0;
    w.L = -1;
    return true;
  }
  return false;
}

// Bounded wait that gives up at once when another warp of the CTA has. After a
// timeout every warp runs to the end: the softmax warps without waiting, and
// without arriving, so that no MMA starts and no stage is refilled on their word;
// the producer and the MMA warps stop, and wait for what they have in flight
// before the CTA leaves (their copies and MMAs would write into the next CTA's
// shared and tensor memory).
__device__ __forceinline__ bool wait_bar(uint64_t *bar, unsigned parity, const LatentDecodeParams &p, volatile int *abort) {
  if (mbar_test(bar, parity)) return true;
  if (*abort) return false;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity, p.hint_ns)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > p.wait_ns) {
      atomicOr(p.status, FD_DEVSTAT_WAIT_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_bar_warp(uint64_t *bar, unsigned parity, const LatentDecodeParams &p,
                                              volatile int *abort) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, p, abort)) != 0;
}

// BIG: pages of 64 keys and more (a template parameter, so that the MMA issue
// loop's descriptor offsets are constants: computed ones cost it 35 clocks an MMA).
// AHEAD: tiles are prefetched into L2 (several row tiles, contiguous rows).
template <bool BIG, bool AHEAD>
__global__ void __launch_bounds__(kThreads, 1)
    fd_latent_decode_kernel(const __grid_constant__ CUtensorMap tmc, const __grid_constant__ LatentDecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  int64_t *row_off = reinterpret_cast<int64_t *>(smem + kOffRow);
  float *factor = reinterpret_cast<float *>(smem + kOffF);
  float *red = reinterpret_cast<float *>(smem + kOffRed);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);  // [stage][slot]: the slot's bytes have landed
  uint64_t *empty = full + kStages * kSlots;                      // [stage][slot]: its MMAs are done
  uint64_t *sfull = empty + kStages * kSlots;                     // [2]: scores of tile j in buffer j % 2
  uint64_t *sfree = sfull + 2;                                    // [2]: scores read by the softmax
  uint64_t *pfull = sfree + 2;                                    // weights of tile j written
  uint64_t *ofull = pfull + 1;                                    // O holds tile j
  uint64_t *qfull = ofull + 1;                                    // queries of the next piece written
  uint64_t *drain = reinterpret_cast<uint64_t *>(smem + kOffDrain);  // [2]: an MMA warp that gave up: its MMAs are done
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
    mbar_init(&sfree[0], kSoftWarps);
    mbar_init(&sfree[1], kSoftWarps);
    mbar_init(pfull, kSoftWarps);
    mbar_init(ofull, 1);
    mbar_init(qfull, kSoftWarps);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kQk) tmem_alloc(tslot, kTmemCols);
  if (warp < kSoftWarps) {  // padding rows of Q read as zero
    for (int i = threadIdx.x; i < (kRows - nrows) * (kLatRow / 8); i += kSoftThreads) {
      const int r = nrows + i / (kLatRow / 8), c = i % (kLatRow / 8);
      *reinterpret_cast<uint4 *>(smem + kOffQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // inputs written by the previous kernel are visible from here on
  griddep_launch_dependents();
  Walk walk = locate(p, g, lane);
  if (walk.left <= 0) {  // the same for every thread of the CTA
    if (warp == kQk) tmem_dealloc(*tslot, kTmemCols);
    return;
  }
  const uint32_t tmem = *tslot;
  // Stage layout (byte (key, block) = (key / 8) atom_stride + block blk_stride
  // + (key % 8) 128): pages of 64 keys and more [block][64 keys], smaller ones
  // [8 keys][block][8 keys].
  constexpr uint32_t atom_stride = BIG ? 1024u : kBlocks * 1024u, blk_stride = BIG ? kBlock : 1024u;

  if (warp == kProducer) {
    // ======================= TMA producer =======================
    if (lane == 0) tma_prefetch_desc(&tmc);
    // one CTA reads a tile when there is one row tile; else its neighbours do soon
    const uint64_t pol = p.row_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
    const int P = p.page_size;
    // With several row tiles the tensor cores set the pace and HBM has time: the
    // first of the CTAs that read a tile prefetches the next one into L2, which
    // takes the load's wait off the chain of the two stages (32 x 128 heads x 10000
    // keys 125 -> 113 us a call, 64 x 96 x 20000 418 -> 378, 8 x 512 x 8000 95 -> 89;
    // two to four tiles ahead 114 to 116). With one row tile HBM sets it, and more
    // in flight changes little: 64 x 20000 keys with 16 / 32 / 48 / 64 rows 242 ->
    // 236, 244 -> 240, 246 -> 244, 246 -> 249, 8 x 8000 with 16 22.5 -> 23.3.
    const bool ahead = AHEAD && rt == 0;
    constexpr int log2_seg = BIG ? 6 : 3, seg = 1 << log2_seg;  // keys per TMA box
    const int i = lane & 7;  // the segment of a tile (at most 8) whose page this lane holds
    Piece pc;
    int j = 0, last = -1;
    bool ok = true;
    while (ok && next_piece(p, walk, pc)) {
      const int *pt = p.page_table + pc.b * p.pt_sb;
      auto ld_pid = [&](int t) {
        const int key = t * kTile + (i << log2_seg);
        return i < (kTile >> log2_seg) && key < pc.L ? pt[key >> p.log2_page] : 0;
      };
      // lane k prefetches the tile's rows in its k-th page
      const int log2_part = min(6, p.log2_page);  // keys of a tile in one page
      auto ld_ahead = [&](int t) {
        const int key = t * kTile + (lane << log2_part);
        return lane < (kTile >> log2_part) && t < pc.t1 && key < pc.L ? pt[key >> p.log2_page] : -1;
      };
      int pid_next = ld_pid(pc.t0), pid_ahead = ahead ? ld_ahead(pc.t0 + 1) : -1;
      for (int t = pc.t0; ok && t < pc.t1; ++t, ++j) {
        int pid = pid_next;
        if (t + 1 < pc.t1) pid_next = ld_pid(t + 1);
        const int tok0 = t * kTile, nseg = (min(kTile, pc.L - tok0) + seg - 1) >> log2_seg;
        const bool mine = i < nseg;
        const bool bad = mine && (pid < 0 || pid >= p.num_pages);
        if (bad) pid = p.num_pages;  // outside the pool: record, and let TMA zero-fill
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
        if (ahead) {
          if (pid_ahead >= 0 && pid_ahead < p.num_pages) {
            const int slot = ((t + 1) * kTile + (lane << log2_part)) & (P - 1);
            l2_prefetch_bulk(p.cache + pid_ahead * p.c_sp + slot * kLatRow, static_cast<unsigned>((kLatRow * 2) << log2_part));
          }
          pid_ahead = ld_ahead(t + 2);
        }
        const int stage = j % kStages;
        const unsigned ph = (j / kStages) & 1;
#pragma unroll 1
        for (int s = 0; s < kSlots; ++s) {
          uint64_t *fb = &full[stage * kSlots + s];
          if (!wait_bar_warp(&empty[stage * kSlots + s], ph ^ 1, p, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t *dst = smem + stage * kStageBytes + s * 3 * blk_stride;
          if (elect_one()) mbar_arrive_expect_tx(fb, static_cast<unsigned>(nseg * seg * 128 * (kBlocks / kSlots)));
          for (int k = 0; k < nseg; ++k) {
            const int page = __shfl_sync(0xffffffffu, pid, k), off = k << log2_seg;
            if (elect_one()) tma_load_4d(dst + k * atom_stride, &tmc, 0, (tok0 + off) & (P - 1), 3 * s, page, fb, pol);
          }
          last = j * kSlots + s;
        }
      }
    }
    // The last copy into each slot lands before the CTA ends: nobody else waits for
    // it when another warp has given up.
    if (lane == 0)
      for (int k = max(0, last - kStages * kSlots + 1); k <= last; ++k)
        mbar_wait(&full[(k / kSlots % kStages) * kSlots + k % kSlots], (k / kSlots / kStages) & 1, p.status);
    __syncwarp();
  } else if (warp == kQk) {
    // ======================= score MMAs =======================
    // Two warps issue MMAs, each in its own order, so that neither the scores of
    // the next tile nor the sums of this one wait behind the other's barriers.
    // (One thread that polls for both: 60 to 350 clocks of looking between
    // bursts, more than the three MMAs that the queue holds.)
    if (elect_one()) {
      const uint32_t base = smem_u32(smem);
      const uint64_t qd = umma_desc_sw128(base + kOffQ);
      const uint64_t kd = umma_desc_sw128_mn(base, 16, atom_stride);  // K-major: no second column stride
      constexpr uint32_t idesc = umma_idesc_bf16(64, kTile, false, false);
      constexpr uint32_t kb = blk_stride >> 4;
      Piece pc;
      int j = 0, piece = 0;
      bool ok = true;
      uint64_t *last_bar = nullptr;
      unsigned last_par = 0;
      while (ok && next_piece(p, walk, pc)) {
        ok = wait_bar(qfull, piece & 1, p, abort_flag);
        ++piece;
        for (int t = pc.t0; ok && t < pc.t1; ++t, ++j) {
          // S buffer j % 2: the softmax has read tile j - 2
          if (j >= 2) ok = wait_bar(&sfree[j & 1], ((j >> 1) & 1) ^ 1, p, abort_flag);
          const uint64_t kt = kd + (((j % kStages) * kStageBytes) >> 4);
          const uint32_t dst = tmem + kTmS + (j & 1) * kTile;
#pragma unroll
          for (int s = 0; s < kSlots; ++s) {
            if (ok)
              ok = wait_bar(&full[(j % kStages) * kSlots + s], (j / kStages) & 1, p, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 12 * s; k < 12 * s + 12; ++k)
              umma_f16_ss(dst, qd + (((k >> 2) * kRows * 128 + (k & 3) * 32) >> 4),
                          kt + (k >> 2) * kb + (((k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
          }
          if (!ok) break;  // (scores that lack a slot are not announced)
          umma_commit(&sfull[j & 1]);
          last_bar = &sfull[j & 1];
          last_par = (j >> 1) & 1;
        }
      }
      // MMAs end before TMEM is released. (Given up: the scores two tiles back may
      // be unfinished too, and last_bar's parity does not tell their phase from the last.)
      if (!ok) {
        umma_commit(&drain[0]);
        last_bar = &drain[0];
        last_par = 0;
      }
      if (last_bar) mbar_wait(last_bar, last_par, p.status);
    }
    __syncwarp();
  } else if (warp == kPv) {
    // ======================= value MMAs =======================
    if (elect_one()) {
      const uint32_t base = smem_u32(smem);
      const uint64_t pd = umma_desc_sw128(base + kOffP);
      const uint64_t vd = umma_desc_sw128_mn(base, blk_stride, atom_stride);
      constexpr uint32_t kb = blk_stride >> 4, ka = atom_stride >> 3;  // descriptor steps: a block; 16 keys
      const uint32_t idesc = umma_idesc_bf16(128, p.rows_per_tile, true, false);
      Piece pc;
      int j = 0;
      bool ok = true;
      while (ok && next_piece(p, walk, pc)) {
        for (int t = pc.t0; t < pc.t1; ++t, ++j) {
          ok = wait_bar(pfull, j & 1, p, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vt = vd + (((j % kStages) * kStageBytes) >> 4);
          const uint32_t keep = t > pc.t0 ? 1u : 0u;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              umma_f16_ss(tmem + d * kRows, vt + d * 2 * kb + k * ka, pd + ((k * 32) >> 4), idesc, k > 0 ? 1u : keep);
            // value blocks 2d and 2d + 1 are done: slot 0 (blocks 0-2) after d = 1, slot 1 after d = 2, slot 2
            // after d = 3 (the scores of this tile are complete: the weights came from them)
            if (d > 0) umma_commit(&empty[(j % kStages) * kSlots + d - 1]);
          }
          umma_commit(ofull);
        }
      }
      if (!ok) umma_commit(&drain[1]);
      if (!ok || j > 0) mbar_wait(ok ? ofull : &drain[1], ok ? (j - 1) & 1 : 0, p.status);  // MMAs end before TMEM is released
    }
    __syncwarp();
  } else {
    // ======================= softmax warps =======================
    // Warp w reaches TMEM lanes 32 (w % 4) .. +31: rows 16 (w % 4) .. +15 of the
    // scores, value channels 32 (w % 4) .. +31 of each 128 of O^T. The two warps
    // of a quarter share the keys of a tile, and the four blocks of O^T.
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t to = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t ts = to + kTmS + half * 32;
    const bool live = quarter * 16 < nrows, ragged = quarter * 16 + 16 > nrows;
    const int ra = quarter * 16 + (lane >> 2), rb = ra + 8;  // this thread's rows of the tile
    const int qcol = half * 32 + (lane & 3) * 2;             // its first key of a tile (then every 8th pair)
    const int npad = p.rows_per_tile;
    // The rows' offsets in q are the same for every piece: lane k holds row
    // warp + 8 k's.
    const int qr = row0 + warp + kSoftWarps * (lane & 7), qt = qr / p.H;
    const int64_t q_off = qt * p.q_st + (qr - qt * p.H) * p.q_sh;
    auto load_q = [&](const Piece &pc) {  // a warp a row, 16 bytes a lane
      const __nv_bfloat16 *q = p.q + pc.b * p.q_sb + lane * 8;
      uint8_t *dst = smem + kOffQ + (lane >> 3) * (kRows * 128) + warp * 128 + (((lane & 7) ^ (warp & 7)) << 4);
#pragma unroll
      for (int k = 0; k < kRows / kSoftWarps; ++k) {  // row warp + 8 k: the same swizzle phase
        const __nv_bfloat16 *src = q + __shfl_sync(0xffffffffu, q_off, k);
        if (warp + kSoftWarps * k >= nrows) break;
        uint8_t *d = dst + k * (kSoftWarps * 128);
        cp_async_ca<16>(d, src);
        cp_async_ca<16>(d + 4 * kRows * 128, src + 256);
        if (lane < 8) cp_async_ca<16>(d + 8 * kRows * 128, src + 512);
      }
    };
    bool speak = lane == 0;
    auto publish_q = [&] {
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (speak) mbar_arrive(qfull);
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
      named_barrier(1, kSoftThreads);  // the epilogue before has read factor and row_off
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
        if (!wait_bar_warp(&sfull[j & 1], (j >> 1) & 1, p, abort_flag)) speak = false;
        tc_fence_after();
        float v[16];
        float xa = -INFINITY, xb = -INFINITY;
        if (live) {
          tmem_ld_16x32(ts + (j & 1) * kTile, v);
          tmem_wait_ld();
          tc_fence_before();
        }
        __syncwarp();
        if (speak) mbar_arrive(&sfree[j & 1]);
        if (live) {
          if (tok0 + kTile > limmin || ragged) {  // some key is past some row's limit, or a row is padding
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k0 = tok0 + 8 * c + qcol;
              v[4 * c] = k0 < lima ? v[4 * c] : -INFINITY;
              v[4 * c + 1] = k0 + 1 < lima ? v[4 * c + 1] : -INFINITY;
              v[4 * c + 2] = k0 < limb ? v[4 * c + 2] : -INFINITY;
              v[4 * c + 3] = k0 + 1 < limb ? v[4 * c + 3] : -INFINITY;
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            xa = fmaxf(xa, fmaxf(v[4 * c], v[4 * c + 1]));
            xb = fmaxf(xb, fmaxf(v[4 * c + 2], v[4 * c + 3]));
          }
          xa *= p.scale_log2;
          xb *= p.scale_log2;
        }
        if (bar_red_or(1, kSoftThreads, xa > ma + 8.f || xb > mb + 8.f)) {
          // some row outgrew its maximum by 2^8: every row takes its new one
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
          if ((lane & 3) == 0) {
            red[half * kRows + ra] = xa;
            red[half * kRows + rb] = xb;
          }
          named_barrier(1, kSoftThreads);
          const float na = fmaxf(ma, fmaxf(red[ra], red[kRows + ra])), nb = fmaxf(mb, fmaxf(red[rb], red[kRows + rb]));
          const float fa = na == -INFINITY ? 1.f : fast_exp2(ma - na), fb = nb == -INFINITY ? 1.f : fast_exp2(mb - nb);
          ma = na;
          mb = nb;
          la *= fa;
          lb *= fb;
          if (t > pc.t0) {  // scale the sums so far, once PV(j - 1) is in
            if ((lane & 3) == 0) {  // the two halves write the same values
              factor[ra] = fa;
              factor[rb] = fb;
            }
            named_barrier(1, kSoftThreads);
            if (!wait_bar_warp(ofull, (j - 1) & 1, p, abort_flag)) speak = false;
            tc_fence_after();
#pragma unroll 1
            for (int d = 2 * half; d < 2 * half + 2; ++d)
#pragma unroll 1
              for (int c = 0; c < npad; c += 16) {
                float o[16], f[16];
                tmem_ld16(to + d * kRows + c, o);
#pragma unroll
                for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(f + i) = *reinterpret_cast<float4 *>(factor + c + i);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f[i];
                tmem_st16(to + d * kRows + c, o);
              }
            tmem_wait_st();
          }
        }
        const float ua = ma == -INFINITY ? 0.f : ma, ub = mb == -INFINITY ? 0.f : mb;
        uint32_t wa[4], wb[4];
        if (live) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
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
        if (j > 0 && !wait_bar_warp(ofull, (j - 1) & 1, p, abort_flag)) speak = false;
        if (live) {
          uint8_t *pa = smem + kOffP + ra * 128 + 4 * (lane & 3), *pb = pa + 8 * 128;  // rows 8 apart share the swizzle phase
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int chunk = ((4 * half + c) ^ (ra & 7)) << 4;
            *reinterpret_cast<uint32_t *>(pa + chunk) = wa[c];
            *reinterpret_cast<uint32_t *>(pb + chunk) = wb[c];
          }
        }
        const int valid = pc.L - tok0;
        if (valid < kTile) {  // value rows past the request's keys may hold anything: weight 0 needs them finite
          uint8_t *st = smem + (j % kStages) * kStageBytes;
          for (int i = threadIdx.x; i < (kTile - valid) * 64; i += kSoftThreads) {
            const int key = valid + (i >> 6);
            *reinterpret_cast<uint4 *>(st + ((i & 63) >> 3) * blk_stride + (key >> 3) * atom_stride + (key & 7) * 128 +
                                       ((i & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (speak) mbar_arrive(pfull);
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
      named_barrier(1, kSoftThreads);  // every rescale has read factor and red
      if ((lane & 3) == 0) {
        red[half * kRows + ra] = la;
        red[half * kRows + rb] = lb;
      }
      named_barrier(1, kSoftThreads);
      if ((lane & 3) == 0 && half == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = i ? rb : ra;
          const float l = red[r] + red[kRows + r], m = i ? mb : ma;
          // l = 0: no visible key. A NaN stays one, in the LSE too (a partial with LSE -inf is left out)
          factor[r] = l == 0.f ? 0.f : 1.f / l;
          const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
          if (r < nrows) {
            const int rg = row0 + r, tq = rg / p.H, h = rg - tq * p.H;
            if (!whole) p.lse_part[part_row + r] = lse;
            else if (p.lse) p.lse[cur.b * p.l_sb + tq * p.l_st + h * p.l_sh] = lse;
          }
        }
      }
      if (!wait_bar_warp(ofull, (j - 1) & 1, p, abort_flag)) speak = false;
      tc_fence_after();
      named_barrier(1, kSoftThreads);
      const bool bf = whole && !p.out_f32;
      float *const of = whole ? static_cast<float *>(p.out) : p.o_part;
      __nv_bfloat16 *const ob = static_cast<__nv_bfloat16 *>(p.out);
#pragma unroll 1
      for (int c = 0; c < npad; c += 16) {
        // offsets and factors first: the compiler cannot move shared-memory
        // loads over the stores (110 clocks a store with them in between)
        int64_t at[16];
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2)
          *reinterpret_cast<longlong2 *>(at + i) = *reinterpret_cast<longlong2 *>(row_off + c + i);
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(f + i) = *reinterpret_cast<float4 *>(factor + c + i);
        const int ch = half * 256 + quarter * 32 + lane;
        float o[2][16];
        tmem_ld16(to + 2 * half * kRows + c, o[0]);
        tmem_ld16(to + (2 * half + 1) * kRows + c, o[1]);
        tmem_wait_ld();
        if (bf) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (at[i] >= 0) {
              ob[at[i] + ch] = __float2bfloat16_rn(o[0][i] * f[i]);
              ob[at[i] + ch + 128] = __float2bfloat16_rn(o[1][i] * f[i]);
            }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (at[i] >= 0) {
              of[at[i] + ch] = o[0][i] * f[i];
              of[at[i] + ch + 128] = o[1][i] * f[i];
            }
        }
      }
      tc_fence_before();  // O is read before the next piece's PV overwrites it
      if (more) publish_q();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kQk) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of a request's partials: out = sum_c w_c o_c / sum_c w_c with
// w_c = exp(lse_c - max_c lse_c). A warp takes every `merge_warps`-th partial of
// a row, 16 / N channels a lane, U partials and their LSEs in one round trip; the
// warps of a row are joined in shared memory. A request that lies in one CTA's
// range was written by it; the rows of one without keys are written here.
// Shapes (see launch_latent_decode): W = 16 warps, U = 4 for few rows with many
// partials each, the fewest rows cut into N parts of their channels; W = 8,
// U = 2 (64 registers, four CTAs an SM) for many.
template <int W, int U, int N>
__global__ void __launch_bounds__(W * 32, W == 8 ? 4 : 1)
    fd_latent_merge_kernel(const __grid_constant__ LatentDecodeParams p) {
  constexpr int kCh = kLatC / N, kVec = kCh / 128;  // channels of this CTA; 16-byte words a lane
  __shared__ float acc_s[W][kCh];
  __shared__ float stat_s[W][2];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = p.merge_warps, sub = warp % wpr;
  const int r = blockIdx.x * (W / wpr) + warp / wpr, b = blockIdx.y, ch0 = blockIdx.z * kCh;
  // The lengths are read before the wait: the decode kernel triggers this grid
  // only after its own dependency wait and does not write them.
  int n = 0, before = 0, mine = 0;
  for (int i0 = 0; i0 < p.B; i0 += 64) {
    const int i = i0 + lane, L0 = load_len(p, min(i, p.B - 1)), L1 = load_len(p, min(i + 32, p.B - 1));
    const int n0 = i < p.B ? places_of(p, L0) : 0, n1 = i + 32 < p.B ? places_of(p, L1) : 0;
    n += n0 + n1;
    before += (i < b ? n0 : 0) + (i + 32 < b ? n1 : 0);
    mine += (i == b ? tiles_of(L0) : 0) + (i + 32 == b ? tiles_of(L1) : 0);
  }
  n = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
  before = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(before)));
  mine = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine)));
  const int per = tiles_per_group(n, p.groups);
  const int first = before + p.change, c0 = first / per, c1 = mine ? (first + mine - 1) / per : c0;
  if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) {  // a length out of range is recorded
    const int raw = ld_cg(p.seqlens + b * p.sl_s);
    if (raw < 0 || raw > p.max_pages * p.page_size) atomicOr(p.status, FD_DEVSTAT_SEQLEN_OVERFLOW);
  }
  griddep_wait();  // in every CTA: this grid must not end before the decode kernel's
  if (mine && c0 == c1) return;
  const int np = mine ? c1 - c0 + 1 : 0;  // a request without keys: out = 0, lse = -inf
  float4 acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float Z = 0.f, M = -INFINITY;
  if (r < p.R) {
    const int rt = r / p.rows_per_tile;
    const int64_t row = (static_cast<int64_t>(2 * c0) * p.row_tiles + rt) * kRows + (r - rt * p.rows_per_tile);
    const int64_t stride = static_cast<int64_t>(2 * p.row_tiles) * kRows;  // rows from one CTA group to the next
    const int64_t slot1 = static_cast<int64_t>(p.row_tiles) * kRows;       // slot 1 lies behind slot 0
#pragma unroll 1
    for (int cc = sub; cc < np; cc += U * wpr) {
      float4 o[U][kVec];
      float l[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = cc + u * wpr;
        l[u] = -INFINITY;
        if (c < np) {
          const int64_t at = row + c * stride + (c == 0 ? slot1 : 0);
          l[u] = p.lse_part[at];
          const float4 *src = reinterpret_cast<const float4 *>(p.o_part + at * kLatC + ch0) + lane;
#pragma unroll
          for (int i = 0; i < kVec; ++i) o[u][i] = src[32 * i];
        }
      }
      float top = M;
      bool any = false;  // a partial with visible keys (its LSE may be NaN, which the maximum passes over)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        top = fmaxf(top, l[u]);
        any |= l[u] != -INFINITY;
      }
      if (!any) continue;
      const float keep = expf(M - top);
      M = top;
      Z *= keep;
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = make_float4(acc[i].x * keep, acc[i].y * keep, acc[i].z * keep, acc[i].w * keep);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (l[u] == -INFINITY) continue;  // no partial, or one without visible keys
        const float w = expf(l[u] - top);
        Z += w;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          acc[i].x = fmaf(w, o[u][i].x, acc[i].x);
          acc[i].y = fmaf(w, o[u][i].y, acc[i].y);
          acc[i].z = fmaf(w, o[u][i].z, acc[i].z);
          acc[i].w = fmaf(w, o[u][i].w, acc[i].w);
        }
      }
    }
  }
  const int t = r / p.H, h = r - t * p.H;
  const int64_t out = b * p.o_sb + t * p.o_st + h * p.o_sh + ch0;
  const int64_t lse_at = b * p.l_sb + t * p.l_st + h * p.l_sh;
  auto write4 = [&](int ch, const float4 &v, float f) {
    if (p.out_f32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + out + ch) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + out + ch) =
          make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
  };
  if (wpr == 1) {
    if (r >= p.R) return;
    const float inv = Z == 0.f ? 0.f : 1.f / Z;
#pragma unroll
    for (int i = 0; i < kVec; ++i) write4(i * 128 + lane * 4, acc[i], inv);
    if (lane == 0 && ch0 == 0 && p.lse) p.lse[lse_at] = Z == 0.f ? -INFINITY : M + logf(Z);
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) *reinterpret_cast<float4 *>(&acc_s[warp][i * 128 + lane * 4]) = acc[i];
  if (lane == 0) {
    stat_s[warp][0] = M;
    stat_s[warp][1] = Z;
  }
  __syncthreads();
  if (r >= p.R) return;
  // the row's warps share its channels
  const int w0 = warp - sub;
  float top = -INFINITY, total = 0.f;
  for (int w = w0; w < w0 + wpr; ++w) top = fmaxf(top, stat_s[w][0]);
  for (int w = w0; w < w0 + wpr; ++w) total += stat_s[w][1] == 0.f ? 0.f : stat_s[w][1] * expf(stat_s[w][0] - top);
  const float inv = total == 0.f ? 0.f : 1.f / total;
  for (int ch = (sub * 32 + lane) * 4; ch < kCh; ch += wpr * 128) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = w0; w < w0 + wpr; ++w) {
      if (stat_s[w][1] == 0.f) continue;
      const float f = expf(stat_s[w][0] - top);
      const float4 x = *reinterpret_cast<const float4 *>(&acc_s[w][ch]);
      v.x = fmaf(f, x.x, v.x);
      v.y = fmaf(f, x.y, v.y);
      v.z = fmaf(f, x.z, v.z);
      v.w = fmaf(f, x.w, v.w);
    }
    write4(ch, v, inv);
  }
  if (sub == 0 && lane == 0 && ch0 == 0 && p.lse) p.lse[lse_at] = total == 0.f ? -INFINITY : top + logf(total);
}

}  // namespace

cudaError_t latent_decode_prepare() {
  for (auto *kernel : {fd_latent_decode_kernel<false, false>, fd_latent_decode_kernel<false, true>,
                       fd_latent_decode_kernel<true, false>, fd_latent_decode_kernel<true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
  // Merge warps a row, up to what the SMs hold at once (152 x 32 warps of the
  // 8-warp shape: one wave), and no more than a request's expected partials.
  // Sixteen where a row has that many; then two CTAs a row, half its channels
  // each, while all run at once (us a call back to back with 1 / 2 / 4 parts: 16
  // rows x 200 keys 10.7 / 10.2 / 11.0, x 4000 13.5 / 12.7 / 12.4, x 32768 18.5 /
  // 17.2 / 16.7; 128 rows x 32768 24.7 / 29.5 / 37.7).
  const int64_t rows = static_cast<int64_t>(p.B) * p.R;
  p.merge_warps = 16;
  while (p.merge_warps > 1 && (rows * p.merge_warps > 4864 || p.merge_warps > p.groups / p.B + 1)) p.merge_warps >>= 1;
  auto *const kernel = p.log2_page >= 6
                           ? (p.cache ? fd_latent_decode_kernel<true, true> : fd_latent_decode_kernel<true, false>)
                           : (p.cache ? fd_latent_decode_kernel<false, true> : fd_latent_decode_kernel<false, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tmc, p);
  if (e != cudaSuccess) return e;
  const int warps = p.merge_warps == 16 ? 16 : 8, per_cta = warps / p.merge_warps;
  cfg.gridDim = dim3(static_cast<unsigned>((p.R + per_cta - 1) / per_cta), static_cast<unsigned>(p.B));
  cfg.blockDim = dim3(static_cast<unsigned>(warps * 32));
  cfg.dynamicSmemBytes = 0;
  if (warps == 16 && 2 * rows <= 152) {
    cfg.gridDim.z = 2;
    return cudaLaunchKernelEx(&cfg, fd_latent_merge_kernel<16, 4, 2>, p);
  }
  return warps == 16 ? cudaLaunchKernelEx(&cfg, fd_latent_merge_kernel<16, 4, 1>, p)
                     : cudaLaunchKernelEx(&cfg, fd_latent_merge_kernel<8, 2, 1>, p);
}

}  // namespace fd
