// decode_sparse.cu - grouped-query decode attention over selected pages of a paged
// cache (sm_103a).
//
// For a request, query token and KV head the list names positions of the page
// table; the G query heads attend to the keys of those pages that the token may
// see:  out = sum_j p_j v_j,  p = softmax(scale q . k),  lse = ln sum exp.
//
// HBM binds it: 4 D bytes a key and head (bf16), against 4 G D operations; of a quantised cache, turning its codes into
// operands (1.75 to 2 instructions each) binds as much. A warp works alone: it takes every (4 R)-th tile of 16 keys of the list
// (R CTAs of 4 warps share a list), copies its rows with cp.async into a ring of its own, and keeps a running maximum,
// sum and the outputs in registers (one pass, no barrier inside the loop). Queries are the narrow side of the products: S^T =
// K Q^T and O^T = V^T P^T on mma.m16n8k16 with 16 keys or channels by 8 query rows, so that 8 heads fill it; two such
// tiles for up to 16. Both operands come from row-major rows in shared memory with 16-byte loads: the order of the channels
// inside a k step is free as long as Q and K agree, V's pairs of keys are joined with byte permutes, and P^T is its
// accumulators transposed by movmatrix. At the end the warps' parts are joined through shared memory, those of a cluster's CTAs
// through distributed shared memory: one launch, no workspace, and no atomics in a result. 64 requests x 8 heads of 4096 keys
// take 155-161 us in bf16 (two GPUs; the copy rate), 108 in int8, 104 in int4; 24 requests x 4 tokens of up to 1072 keys 50, 45 and
// 43; one request of 2048 keys 7.4.
//
// The tensor core's operands are bf16, which would round a weight by up to 2^-8 of it, as
// much as the output's own rounding. Weights go in as two words (2^-15 at most), with a second product
// of each tile of values (one word: int8 104 and 42 us, int4 95 and 39, bf16 160 and 49); sums and lse use the unrounded ones.
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

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;      // keys of a tile
constexpr int kMaxRanks = 8;

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t at) { return __uint_as_float(lds32(at)); }

// Two bf16 of the 8-bit codes in bits 0..7 and 16..23: 128 + the low seven bits, less 128 or (negative codes) 256, which is the
// code, exactly.
__device__ __forceinline__ uint32_t byte_pair(uint32_t x) {
  uint32_t d, less;
  asm("lop3.b32 %0, %1, 0x007f007f, 0x43004300, 0xea;" : "=r"(d) : "r"(x));     // (x & mask) | 128
  asm("lop3.b32 %0, %1, 0x00800080, 0x43004300, 0x6a;" : "=r"(less) : "r"(x));  // (x & mask) ^ 128
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&d), *reinterpret_cast<__nv_bfloat162 *>(&less));
  return *reinterpret_cast<const uint32_t *>(&v);
}
// Two bf16 of the 4-bit codes in bits 0..3 and 16..19 (offset by 8): 128 + u, less 136.
__device__ __forceinline__ uint32_t nibble_pair(uint32_t x) {
  uint32_t d;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(d) : "r"(x));
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&d), __float2bfloat162_rn(136.f));
  return *reinterpret_cast<const uint32_t *>(&v);
}

// What the upper 16 bits of a (given as u) leave of it, and 2^-24 of a more, so that it is not 0 (of weights above 2^-109) and an
// infinite value times it no NaN. One rounding.
__device__ __forceinline__ float rest_of(float a, uint32_t u) {
  return fmaf(__uint_as_float(u & 0xffff0000u), -(1.f - 0x1p-24f), a);
}

// A tile in shared memory, and how a thread (g = lane / 4, t = lane % 4) reads its
// fragments: S^T has keys g and 8 + g, O^T += V^T P^T keys 2 t, 2 t + 1, 8 + 2 t, 9 + 2 t
// of thread t. 16-byte pieces of a row of 128 bytes or more are placed by
// the key's low bits, so that both reads hit every bank once.
template <int KIND, int D>
struct Tile {
  static constexpr int kRow = KIND == KV_BF16 ? 2 * D : (KIND == KV_I8 ? D : D / 2);  // bytes of a row
  static constexpr bool kSwizzled = kRow >= 128;
  static constexpr int kStride = kSwizzled ? kRow : kRow + 16;
  static constexpr int kGroups = KIND == KV_I4 ? D / 32 : 1;
  static constexpr int kScaleBytes = KIND == KV_BF16 ? 0 : 4 * kGroups;  // of a row
  static constexpr int kScales = 2 * kTile * kStride;                    // where they begin: K's, then V's
  static constexpr int kBytes = kScales + 2 * kTile * kScaleBytes;
  static constexpr int kStages = KIND == KV_BF16 ? (D == 128 ? 3 : 6) : (KIND == KV_I8 ? 3 : 4);
  static constexpr int kSteps = D / 16;   // k steps of a score
  static constexpr int kMTiles = D / 16;  // m tiles of an output

  static __device__ __forceinline__ uint32_t piece(int key, int c) {  // offset of 16-byte piece c of a key's row
    return key * kStride + ((kSwizzled ? c ^ ((key & 6) ^ ((key & 1) << 2)) : c) << 4);
  }
};

// Channel that row r (0 .. 15) of m tile j of an output is.
template <int KIND, int D>
__device__ __forceinline__ int channel_of(int j, int r) {
  const int g = r & 7, tile = 2 * j + (r >> 3);
  if constexpr (KIND == KV_BF16) return 8 * (g + 8 * (tile / 8)) + tile % 8;
  if constexpr (KIND == KV_I8) return D / 8 * g + tile;
  return 32 * (tile / 4) + 4 * g + tile % 4;
}

// NQ: tiles of 8 query rows (heads).
template <int KIND, int D, int NQ>
__global__ void __launch_bounds__(kThreads, KIND == KV_BF16 ? 2 : (NQ == 1 ? 4 : 3)) fd_decode_sparse_kernel(const __grid_constant__ SparseParams p) {
  using T = Tile<KIND, D>;
  constexpr int kRows = 8 * NQ;
  extern __shared__ __align__(128) unsigned char smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = p.ranks, rank = ranks > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  // unit: row tile, then query token, then head, then request (neighbours share pages in L2)
  int unit = blockIdx.x / ranks;
  const int rt = unit % p.row_tiles;
  unit /= p.row_tiles;
  const int t = unit % p.Tq;
  unit /= p.Tq;
  const int h = unit % p.Hkv, b = unit / p.Hkv;
  const int rows = min(kRows, p.G - rt * kRows), head0 = h * p.G + rt * kRows;

  griddep_wait();  // inputs written by the previous kernel are visible from here on
  int L = p.seqlens[b * p.sl_s];
  const long long cap = static_cast<long long>(p.W) * p.P;
  if (L < 0 || L > cap) {
    if (tid == 0 && rank == 0 && p.status) atomicOr(p.status, FD_DEVSTAT_SEQLEN_OVERFLOW);
    L = L < 0 ? 0 : static_cast<int>(cap);
  }
  const int limit = max(0, L - (p.Tq - 1) + t);  // keys that the token sees

  // ---- Q: rows g and g + 8. Of k step s thread t4 holds the 4 channels that it reads of K there.
  uint32_t q[NQ][T::kSteps][2];
  {
    const __nv_bfloat16 *base = p.q + b * p.q_sb + t * p.q_st;
#pragma unroll
    for (int half = 0; half < NQ; ++half) {
      const bool in = g + 8 * half < rows;
      const __nv_bfloat16 *row = base + static_cast<int64_t>(head0 + (in ? g + 8 * half : 0)) * p.q_sh;
#pragma unroll
      for (int s = 0; s < T::kSteps; ++s) {
        int c;  // first of the 4 channels
        if constexpr (KIND == KV_BF16) c = 8 * (t4 + 4 * (s / 2)) + 4 * (s % 2);
        else if constexpr (KIND == KV_I8 && D == 128) c = 16 * (t4 + 4 * (s / 4)) + 4 * (s % 4);
        else if constexpr (KIND == KV_I8) c = 16 * t4 + 4 * s;
        else c = 32 * (s / 2) + 8 * t4 + 4 * (s % 2);
        uint2 w = make_uint2(0u, 0u);
        if constexpr (KIND == KV_I4) {
          // nibbles i and i + 4 of a word come out together: channels 2 (s % 2) + {0, 4} and {1, 5} of the thread's 8
          const uint32_t *x = reinterpret_cast<const uint32_t *>(row + 32 * (s / 2) + 8 * t4) + s % 2;
          if (in) {
            const uint32_t a = x[0], z = x[2];  // channels (2 j, 2 j + 1) and (2 j + 4, 2 j + 5), j = s % 2
            w = make_uint2(__byte_perm(a, z, 0x5410), __byte_perm(a, z, 0x7632));
          }
          (void)c;
        } else if constexpr (KIND == KV_I8) {
          if (in) {  // bytes 0 and 2, then 1 and 3 of a word of codes come out together
            const uint2 x = *reinterpret_cast<const uint2 *>(row + c);
            w = make_uint2(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632));
          }
        } else {
          if (in) w = *reinterpret_cast<const uint2 *>(row + c);
        }
        q[half][s][0] = w.x;
        q[half][s][1] = w.y;
      }
    }
  }

  // ---- this warp's tiles: tile i of the list for i = warp_at, warp_at + stride, ...
  const int stride = kWarps * ranks, at0 = rank * kWarps + warp;
  const int per_page = p.P / kTile;  // tiles a page (0: a tile holds two pages)
  const int tiles = p.P >= kTile ? p.S * per_page : (p.S + 1) / 2;
  const int mine = at0 < tiles ? (tiles - 1 - at0) / stride + 1 : 0;
  const int *list = p.selected + b * p.s_sb + t * p.s_st + h * p.s_sh;
  const int *table = p.page_table + b * p.pt_sb;
  // Tiles are looked up 32 at a time (of 8-key pages 16), one a lane: page id, first slot, and how many of the tile's slots are
  // visible (of 8-key pages lanes l and 16 + l hold the two pages of a tile). Those without a visible slot are passed over.
  const bool two = per_page == 0;
  const int batch = two ? 16 : 32, log2_tiles = p.log2_page - 4;
  int looked = 0, look_page = 0, look_slot = 0, look_seen = 0;
  unsigned todo = 0;  // of the tiles looked up: with a visible slot, not yet fetched
  auto look_up = [&]() {
    const int n = looked + (two ? lane & 15 : lane), i = at0 + n * stride;
    look_page = look_slot = look_seen = 0;
    if (n < mine) {
      const int e = two ? 2 * i + (lane >> 4) : i >> log2_tiles;
      const int pos = e < p.S ? list[e] : -1;
      look_slot = two ? 0 : (i & (per_page - 1)) * kTile;
      const long long first = static_cast<long long>(pos) * p.P + look_slot;  // the tile's first key
      if (pos >= 0 && first < limit) {
        look_page = table[pos];
        look_seen = static_cast<int>(min(static_cast<long long>(two ? 8 : kTile), limit - first));
        if (look_page < 0 || look_page >= p.num_pages) {
          if (p.status) atomicOr(p.status, FD_DEVSTAT_BAD_PAGE);
          look_page = look_seen = 0;
        }
      }
    }
    looked += batch;
    todo = __ballot_sync(0xffffffffu, look_seen > 0);
    if (two) todo = (todo | todo >> 16) & 0xffffu;
  };

  unsigned char *ring = smem + warp * T::kStages * T::kBytes;
  const uint32_t ring32 = smem_u32(ring);
  // Copies of the next tile into slot `to` of the ring; its rows that are not visible are zeros. Returns the visible rows, a bit
  // each; 0 behind the last tile.
  auto fetch = [&](int slot) -> unsigned {
    while (!todo && looked < mine) look_up();
    unsigned seen = 0;
    if (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int pa = __shfl_sync(0xffffffffu, look_page, l), sa = __shfl_sync(0xffffffffu, look_seen, l);
      const int slot0 = __shfl_sync(0xffffffffu, look_slot, l);
      int pb = pa, sb = 0;
      if (two) {
        pb = __shfl_sync(0xffffffffu, look_page, l + 16);
        sb = __shfl_sync(0xffffffffu, look_seen, l + 16);
      }
      seen = ((1u << sa) - 1) | ((1u << sb) - 1) << 8;
      const uint32_t to = ring32 + slot * T::kBytes;
      constexpr int kPieces = T::kRow / 16, kAt = 32 / kPieces;  // pieces of a row; rows a step
      const int c = lane % kPieces, r0 = lane / kPieces;
      const int64_t in_page = static_cast<int64_t>(slot0 + r0) * p.c_ss + h * p.c_sh + 16 * c;
      const int64_t off_a = pa * p.c_sp + in_page, off_b = pb * p.c_sp + in_page - 8 * p.c_ss;
#pragma unroll
      for (int u = 0; u < kTile / kAt; ++u) {
        const int r = u * kAt + r0;
        const int bytes = (seen >> r) & 1 ? 16 : 0;
        const int64_t off = bytes ? (two && r >= 8 ? off_b : off_a) + u * kAt * p.c_ss : 0;
        cp_async_16(to + T::piece(r, c), p.k_cache + off, bytes);
        cp_async_16(to + kTile * T::kStride + T::piece(r, c), p.v_cache + off, bytes);
      }
      if constexpr (KIND != KV_BF16) {  // lane: row lane % 16 of K's (below 16) or V's scales
        const int r = lane & 15, which = lane >> 4;
        const bool second = two && r >= 8;
        const bool in = (seen >> r) & 1;
        const int64_t off = which * p.sc_sk + static_cast<int64_t>(second ? pb : pa) * p.sc_sp +
                            (slot0 + (second ? r - 8 : r)) * p.sc_ss + h * p.sc_sh;
        const uint32_t dst = to + T::kScales + (which * kTile + r) * T::kScaleBytes;
        if constexpr (T::kScaleBytes == 16) cp_async_16(dst, p.scales + (in ? off : 0), in ? 16 : 0);
        else cp_async_small<T::kScaleBytes>(dst, p.scales + (in ? off : 0), in ? T::kScaleBytes : 0);
      }
    }
    cp_async_commit();
    return seen;
  };

  float o[NQ][T::kMTiles][4];
#pragma unroll
  for (int k = 0; k < NQ; ++k)
#pragma unroll
    for (int j = 0; j < T::kMTiles; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[k][j][i] = 0.f;
  // query rows 8 k + 2 t4 + x (l: of keys g and g + 8 of the tiles only)
  float m[NQ][2], l[NQ][2];
#pragma unroll
  for (int k = 0; k < NQ; ++k)
#pragma unroll
    for (int x = 0; x < 2; ++x) m[k][x] = -INFINITY, l[k][x] = 0.f;

  unsigned ahead[T::kStages - 1];  // visible rows of the tiles on their way
#pragma unroll
  for (int n = 0; n < T::kStages - 1; ++n) ahead[n] = fetch(n);
  int st = 0, into = T::kStages - 1;  // slots of the tile to be read and of the one to be copied
#pragma unroll 1
  while (ahead[0]) {
    {
      // the tile kStages - 1 ahead, into the slot that the last tile left
      const unsigned seen = ahead[0];
#pragma unroll
      for (int i = 0; i < T::kStages - 2; ++i) ahead[i] = ahead[i + 1];
      __syncwarp();
      ahead[T::kStages - 2] = fetch(into);
      cp_async_wait<T::kStages - 1>();
      __syncwarp();
      const uint32_t kt = ring32 + st * T::kBytes, vt = kt + kTile * T::kStride, sc = kt + T::kScales;
      // ---- S^T = K Q^T: keys g, 8 + g by query rows 2 t4, 2 t4 + 1
      float s[NQ][4];
#pragma unroll
      for (int k = 0; k < NQ; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[k][x] = 0.f;
      if constexpr (KIND == KV_BF16) {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 w = lds128(kt + T::piece(g, t4 + 4 * j)), z = lds128(kt + T::piece(8 + g, t4 + 4 * j));
          const uint32_t a0[4] = {w.x, z.x, w.y, z.y}, a1[4] = {w.z, z.z, w.w, z.w};
#pragma unroll
          for (int k = 0; k < NQ; ++k) {
            mma_bf16_16816(s[k], a0, q[k][2 * j][0], q[k][2 * j][1]);
            mma_bf16_16816(s[k], a1, q[k][2 * j + 1][0], q[k][2 * j + 1][1]);
          }
        }
      } else if constexpr (KIND == KV_I8) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint4 w = lds128(kt + T::piece(g, t4 + 4 * j)), z = lds128(kt + T::piece(8 + g, t4 + 4 * j));
          const uint32_t x0[4] = {w.x, w.y, w.z, w.w}, x1[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {  // bytes (0, 2) and (1, 3) of a word
            const uint32_t a[4] = {byte_pair(x0[y]), byte_pair(x1[y]), byte_pair(x0[y] >> 8), byte_pair(x1[y] >> 8)};
#pragma unroll
            for (int k = 0; k < NQ; ++k) mma_bf16_16816(s[k], a, q[k][4 * j + y][0], q[k][4 * j + y][1]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {  // a group of 32 channels has a scale of its own
          const uint32_t w = lds32(kt + g * T::kStride + 16 * j + 4 * t4) ^ 0x88888888u;
          const uint32_t z = lds32(kt + (8 + g) * T::kStride + 16 * j + 4 * t4) ^ 0x88888888u;
          const uint32_t a0[4] = {nibble_pair(w), nibble_pair(z), nibble_pair(w >> 4), nibble_pair(z >> 4)};
          const uint32_t a1[4] = {nibble_pair(w >> 8), nibble_pair(z >> 8), nibble_pair(w >> 12), nibble_pair(z >> 12)};
          const float f0 = lds_f32(sc + g * T::kScaleBytes + 4 * j), f1 = lds_f32(sc + (8 + g) * T::kScaleBytes + 4 * j);
#pragma unroll
          for (int k = 0; k < NQ; ++k) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            mma_bf16_16816(part, a0, q[k][2 * j][0], q[k][2 * j][1]);
            mma_bf16_16816(part, a1, q[k][2 * j + 1][0], q[k][2 * j + 1][1]);
            s[k][0] = fmaf(part[0], f0, s[k][0]);
            s[k][1] = fmaf(part[1], f0, s[k][1]);
            s[k][2] = fmaf(part[2], f1, s[k][2]);
            s[k][3] = fmaf(part[3], f1, s[k][3]);
          }
        }
      }
      // ---- scaled by log2(e) and the softmax scale; keys that are not visible are out
      const bool in0 = (seen >> g) & 1, in1 = (seen >> (8 + g)) & 1;
      float f0 = p.scale_log2, f1 = f0;
      if constexpr (KIND == KV_I8) f0 *= lds_f32(sc + 4 * g), f1 *= lds_f32(sc + 4 * (8 + g));
      float top[NQ][2];
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          s[k][x] = in0 ? s[k][x] * f0 : -INFINITY;
          s[k][2 + x] = in1 ? s[k][2 + x] * f1 : -INFINITY;
          top[k][x] = fmaxf(s[k][x], s[k][2 + x]);
        }
      }
      bool more = false;
#pragma unroll
      for (int k = 0; k < NQ; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) more |= top[k][x] > m[k][x];
      // (m is the same in all lanes of a t4: a new maximum in any lane is found by its own lane)
      if (__any_sync(0xffffffffu, more)) {
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float now = fmaxf(m[k][x], top[k][x]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
            const float f = m[k][x] == now ? 1.f : fast_exp2(m[k][x] - now);  // (0 from -inf)
            m[k][x] = now;
            l[k][x] *= f;
#pragma unroll
            for (int j = 0; j < T::kMTiles; ++j) {
              o[k][j][x] *= f;
              o[k][j][2 + x] *= f;
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float base = m[k][x] == -INFINITY ? 0.f : m[k][x];
          s[k][x] = fast_exp2(s[k][x] - base);
          s[k][2 + x] = fast_exp2(s[k][2 + x] - base);
          l[k][x] += s[k][x] + s[k][2 + x];
        }
      }
      // P^T: weights of keys 2 t4, 2 t4 + 1 and 8 more by query row g (times the values' scales of keys g and 8 + g), in two
      // words: the upper 16 bits, and what they leave, rounded.
      auto weights = [&](int k, float w0, float w1, uint32_t (&w)[2], uint32_t (&low)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float a = s[k][2 * x] * (x ? w1 : w0), b = s[k][2 * x + 1] * (x ? w1 : w0);
          const uint32_t u = __float_as_uint(a), v = __float_as_uint(b);
          w[x] = movmatrix_trans(__byte_perm(u, v, 0x7632));
          low[x] = movmatrix_trans(pack_bf16x2(rest_of(a, u), rest_of(b, v)));
        }
      };
      // ---- O^T += V^T P^T
      const int k0 = 2 * t4;
      if constexpr (KIND == KV_BF16) {
        uint32_t pw[NQ][2], pl[NQ][2];
#pragma unroll
        for (int k = 0; k < NQ; ++k) weights(k, 1.f, 1.f, pw[k], pl[k]);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {  // channels 8 (g + 8 j) .. + 7
          const uint4 w0 = lds128(vt + T::piece(k0, g + 8 * j)), w1 = lds128(vt + T::piece(k0 + 1, g + 8 * j));
          const uint4 w2 = lds128(vt + T::piece(k0 + 8, g + 8 * j)), w3 = lds128(vt + T::piece(k0 + 9, g + 8 * j));
          const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
          const uint32_t x2[4] = {w2.x, w2.y, w2.z, w2.w}, x3[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t a[4] = {__byte_perm(x0[y], x1[y], 0x5410), __byte_perm(x0[y], x1[y], 0x7632),
                                   __byte_perm(x2[y], x3[y], 0x5410), __byte_perm(x2[y], x3[y], 0x7632)};
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
              mma_bf16_16816(o[k][4 * j + y], a, pw[k][0], pw[k][1]);
              mma_bf16_16816(o[k][4 * j + y], a, pl[k][0], pl[k][1]);
            }
          }
        }
      } else if constexpr (KIND == KV_I8) {
        const uint32_t vs = sc + kTile * 4;
        uint32_t pw[NQ][2], pl[NQ][2];
#pragma unroll
        for (int k = 0; k < NQ; ++k) weights(k, lds_f32(vs + 4 * g), lds_f32(vs + 4 * (8 + g)), pw[k], pl[k]);
        uint32_t x[4][4];  // codes of 16 (D 128) or 8 (D 64) channels of the four keys
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int key = k0 + (y & 1) + 8 * (y >> 1);
          if constexpr (D == 128) {
            const uint4 w = lds128(vt + T::piece(key, g));
            x[y][0] = w.x, x[y][1] = w.y, x[y][2] = w.z, x[y][3] = w.w;
          } else {
            const uint2 w = lds64(vt + key * T::kStride + 8 * g);
            x[y][0] = w.x, x[y][1] = w.y;
          }
        }
#pragma unroll
        for (int z = 0; z < D / 32; ++z) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // bytes 2 y and 2 y + 1 of both keys of a pair
            const uint32_t sel = y ? 0x7632 : 0x5410;
            const uint32_t u = __byte_perm(x[0][z], x[1][z], sel), v = __byte_perm(x[2][z], x[3][z], sel);
            const uint32_t a[4] = {byte_pair(u), byte_pair(u >> 8), byte_pair(v), byte_pair(v >> 8)};
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
              mma_bf16_16816(o[k][2 * z + y], a, pw[k][0], pw[k][1]);
              mma_bf16_16816(o[k][2 * z + y], a, pl[k][0], pl[k][1]);
            }
          }
        }
      } else {
        const uint32_t vs = sc + kTile * T::kScaleBytes;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {  // channels 32 j + 4 g .. + 3
          uint32_t pw[NQ][2], pl[NQ][2];
          const float w0 = lds_f32(vs + g * T::kScaleBytes + 4 * j), w1 = lds_f32(vs + (8 + g) * T::kScaleBytes + 4 * j);
#pragma unroll
          for (int k = 0; k < NQ; ++k) weights(k, w0, w1, pw[k], pl[k]);
          const uint32_t col = vt + 16 * j + 2 * g;
          const uint32_t x = (lds16(col + k0 * T::kStride) | lds16(col + (k0 + 1) * T::kStride) << 16) ^ 0x88888888u;
          const uint32_t y = (lds16(col + (k0 + 8) * T::kStride) | lds16(col + (k0 + 9) * T::kStride) << 16) ^ 0x88888888u;
          const uint32_t a0[4] = {nibble_pair(x), nibble_pair(x >> 4), nibble_pair(y), nibble_pair(y >> 4)};
          const uint32_t a1[4] = {nibble_pair(x >> 8), nibble_pair(x >> 12), nibble_pair(y >> 8), nibble_pair(y >> 12)};
#pragma unroll
          for (int k = 0; k < NQ; ++k) {
            mma_bf16_16816(o[k][2 * j], a0, pw[k][0], pw[k][1]);
            mma_bf16_16816(o[k][2 * j + 1], a1, pw[k][0], pw[k][1]);
            mma_bf16_16816(o[k][2 * j], a0, pl[k][0], pl[k][1]);
            mma_bf16_16816(o[k][2 * j + 1], a1, pl[k][0], pl[k][1]);
          }
        }
      }
      into = st;
      st = st + 1 == T::kStages ? 0 : st + 1;
    }
  }
  cp_async_wait<0>();

  // ---- the warps' parts into shared memory: [warp][row][channel], m and l behind them
#pragma unroll
  for (int k = 0; k < NQ; ++k)
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[k][x] += __shfl_xor_sync(0xffffffffu, l[k][x], d);
  __syncthreads();  // the rings are free
  constexpr int kPitch = D + 4;
  float *part_o = reinterpret_cast<float *>(smem);           // [kWarps][kRows][kPitch]
  float *part_m = part_o + kWarps * kRows * kPitch;          // [kWarps][kRows]
  float *part_l = part_m + kWarps * kRows;
  float *cta_m = part_l + kWarps * kRows, *cta_l = cta_m + kRows;  // of the CTA; its outputs in part_o's first rows
#pragma unroll
  for (int k = 0; k < NQ; ++k) {
#pragma unroll
    for (int j = 0; j < T::kMTiles; ++j) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        part_o[(warp * kRows + 8 * k + 2 * t4 + (x & 1)) * kPitch + channel_of<KIND, D>(j, g + 8 * (x >> 1))] = o[k][j][x];
    }
    if (g == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        part_m[warp * kRows + 8 * k + 2 * t4 + x] = m[k][x];
        part_l[warp * kRows + 8 * k + 2 * t4 + x] = l[k][x];
      }
    }
  }
  __syncthreads();
  // joined: a thread takes channels c, c + 1 .. of rows; the CTA's own parts are its alone until the cluster meets
  auto weight = [](float mi, float top) { return mi == -INFINITY ? 0.f : exp2f(mi - top); };
  for (int x = tid; x < kRows * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = 4 * (x % (D / 4));
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w * kRows + r]);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = weight(part_m[w * kRows + r], top);
      const float4 v = *reinterpret_cast<const float4 *>(part_o + (w * kRows + r) * kPitch + c);
      // (a part without weight may hold a NaN times 0: a part that saw no key holds zeros)
      sum.x = fmaf(v.x, f, sum.x), sum.y = fmaf(v.y, f, sum.y), sum.z = fmaf(v.z, f, sum.z), sum.w = fmaf(v.w, f, sum.w);
      total = fmaf(part_l[w * kRows + r], f, total);
    }
    *reinterpret_cast<float4 *>(part_o + r * kPitch + c) = sum;  // (only this thread reads or writes these places)
    if (c == 0) cta_m[r] = top, cta_l[r] = total;
  }
  if (ranks > 1) cluster.sync();
  else __syncthreads();
  // ---- the cluster's parts, and the outputs: each CTA a share of the rows' pieces
  const int quads = rows * (D / 4);
  for (int x = rank * kThreads + tid; x < quads; x += ranks * kThreads) {
    const int r = x / (D / 4), c = 4 * (x % (D / 4));
    float4 sum = *reinterpret_cast<const float4 *>(part_o + r * kPitch + c);
    float top = cta_m[r], total = cta_l[r];
    if (ranks > 1) {
      top = -INFINITY;
      for (int i = 0; i < ranks; ++i) top = fmaxf(top, *cluster.map_shared_rank(cta_m + r, i));
      sum = make_float4(0.f, 0.f, 0.f, 0.f);
      total = 0.f;
      for (int i = 0; i < ranks; ++i) {
        const float f = weight(*cluster.map_shared_rank(cta_m + r, i), top);
        const float4 v = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(part_o + r * kPitch + c, i));
        sum.x = fmaf(v.x, f, sum.x), sum.y = fmaf(v.y, f, sum.y), sum.z = fmaf(v.z, f, sum.z), sum.w = fmaf(v.w, f, sum.w);
        total = fmaf(*cluster.map_shared_rank(cta_l + r, i), f, total);
      }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int64_t at = b * p.o_sb + t * p.o_st + static_cast<int64_t>(head0 + r) * p.o_sh + c;
    if (p.out_f32) {
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
          make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
    } else {
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
          make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
    }
    if (c == 0 && p.lse)
      p.lse[b * p.l_sb + t * p.l_st + static_cast<int64_t>(head0 + r) * p.l_sh] =
          total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
  }
  if (ranks > 1) cluster.sync();  // the others have read this CTA's parts
}

template <int KIND, int D, int NQ>
cudaError_t launch(SparseParams p, cudaStream_t stream) {
  using T = Tile<KIND, D>;
  constexpr size_t kRing = static_cast<size_t>(kWarps) * T::kStages * T::kBytes;
  constexpr size_t kJoin = sizeof(float) * (kWarps * 8 * NQ * (D + 4) + 2 * kWarps * 8 * NQ + 2 * 8 * NQ);
  constexpr size_t kSmem = kRing > kJoin ? kRing : kJoin;
  // the kernel's limit of shared memory, once a device
  static std::atomic<unsigned long long> ready{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (device & 63);
  if (device > 63 || !(ready.load() & bit)) {
    e = cudaFuncSetAttribute(fd_decode_sparse_kernel<KIND, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem));
    if (e == cudaSuccess)  // (several CTAs an SM need all of it)
      e = cudaFuncSetAttribute(fd_decode_sparse_kernel<KIND, D, NQ>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  // CTAs a list: more up to kFit CTAs with a tile for each warp. Of a bf16 cache two an SM, which all fit at once (HBM binds; with two
  // CTAs a list 64 x 8 lists of 4096 keys take 168 us, with one 160; 8 x 8 lists of 2048 keys 22.6 with eight, 16.7 with four).
  // Of a quantised one eight an SM, two rounds of the four (three for 16 query rows) that fit: instructions bind, and in the second round
  // CTAs come and go one by one (int8, 64 x 8 lists of 4096 keys 108 us, with one CTA a list 120; but 16 x 8 of 2048 27.4 with eight, 22.4
  // with four).
  p.row_tiles = (p.G + 8 * NQ - 1) / (8 * NQ);
  constexpr int kFit = KIND == KV_BF16 ? 304 : 1216;
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.Tq * p.row_tiles;
  const long long tiles = (static_cast<long long>(p.S) * p.P + kTile - 1) / kTile;
  p.ranks = 1;
  while (p.ranks < kMaxRanks && 2 * p.ranks * units <= kFit && tiles >= 2 * p.ranks * kWarps) p.ranks *= 2;
  return launch_step(fd_decode_sparse_kernel<KIND, D, NQ>, p, dim3(static_cast<unsigned>(units * p.ranks)), kThreads, kSmem,
                     p.ranks, stream);
}

template <int KIND>
cudaError_t launch_d(int head_dim, const SparseParams &p, cudaStream_t stream) {
  if (p.G <= 8) return head_dim == 64 ? launch<KIND, 64, 1>(p, stream) : launch<KIND, 128, 1>(p, stream);
  return head_dim == 64 ? launch<KIND, 64, 2>(p, stream) : launch<KIND, 128, 2>(p, stream);
}

}  // namespace

cudaError_t launch_decode_sparse(int kind, int head_dim, SparseParams p, cudaStream_t stream) {
  if (kind == KV_BF16) return launch_d<KV_BF16>(head_dim, p, stream);
  if (kind == KV_I8) return launch_d<KV_I8>(head_dim, p, stream);
  return launch_d<KV_I4>(head_dim, p, stream);
}

}  // namespace fd
