// latent.h - host/device interface of latent attention (keys and values from
// one shared latent vector a token) and of draft verification.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fd {

// Widths of the latent-attention operators, in channels.
constexpr int kLatC = 512;             // latent part of a cache row: key and value of every head
constexpr int kLatR = 64;              // rotary part of a key, shared by every head
constexpr int kLatRow = kLatC + kLatR; // a cache row, and a query row of the absorbed form
constexpr int kLatRowTile = 64;        // query rows of a decode CTA at most
constexpr int kLatNope = 128;          // expanded form: per-head key channels without the rotary part
constexpr int kLatV = 128;             // expanded form: value channels of a head

constexpr unsigned kLatWaitNs = 2000000000u;  // limit of a kernel's wait, 2 s
constexpr unsigned kLatHintNs = 10000000u;    // and of a thread's suspension in it, 10 ms

// Absorbed decode over a paged latent cache.
struct LatentDecodeParams {
  const __nv_bfloat16 *cache;  // set when tiles are prefetched into L2, else null
  int64_t c_sp;                // its page stride
  const __nv_bfloat16 *q;      // [B, Tq, H, 576]
  int64_t q_sb, q_st, q_sh;
  const int *page_table;       // [B, W]
  int64_t pt_sb;
  const int *seqlens;          // [B]
  int64_t sl_s;
  int num_pages, page_size, log2_page, max_pages;
  int B, Tq, H, R;             // R = Tq * H query rows share a request's keys
  int row_tiles;               // ceil(R / 64) CTAs share a range of keys
  int rows_per_tile;           // rows of each, a multiple of 16
  int change;                  // places that a change to a request takes in the line of tiles
  int groups;                  // ranges the batch's keys are cut into
  int merge_warps;             // merge warps a row (set by the launcher)
  float scale_log2;            // softmax_scale * log2(e)
  float *o_part;               // [groups][2][row_tiles][64][512] partial outputs
  float *lse_part;             // [groups][2][row_tiles][64] and their LSEs
  void *out;                   // [B, Tq, H, 512]
  int out_f32;
  int64_t o_sb, o_st, o_sh;
  float *lse;                  // [B, Tq, H] or null
  int64_t l_sb, l_st, l_sh;
  unsigned *status;
  unsigned wait_ns, hint_ns;   // limit of a wait, and of a thread's suspension in one
};

cudaError_t latent_decode_prepare();  // raise the kernel's shared-memory limit
cudaError_t launch_latent_decode(const CUtensorMap &tmc, LatentDecodeParams p, cudaStream_t stream);

// Expanded attention of ragged prompts.
struct LatentPrefillParams {
  const int *cu_q, *cu_k;  // [B + 1]
  int B, H, Sq, Sk, max_q;
  int tiles;               // tiles of 256 queries at most
  int ragged;              // 1: fewer than the longest request's for each, found on the device
  int ranks;               // CTAs that share one, each a part of its keys (set by the launcher)
  int wide;                // 1: the rows of out start on 32-byte boundaries
  float scale_log2;        // softmax_scale * log2(e)
  void *out;               // [Sq, H, 128]
  int out_f32;
  int64_t o_ss, o_sh;
  float *lse;              // [Sq, H] or null
  int64_t l_ss, l_sh;
  unsigned *status;        // or null
  unsigned wait_ns;        // limit of a wait
};

// tm: tensor maps of q, k_nope, k_pe, v (64 channels x 128 rows a box).
cudaError_t launch_latent_prefill(const CUtensorMap (&tm)[4], LatentPrefillParams p, cudaStream_t stream);

// Verification of drafted tokens.
struct VerifyParams {
  const float *target;      // [B, K + 1, V]
  int64_t t_sb, t_sk;
  const float *draft;       // [B, K, V] or null
  int64_t d_sb, d_sk;
  const void *tokens;       // [B, K] int32 or int64
  int tok64;
  int64_t x_sb, x_sk;
  const int *num_draft;     // [B] or null
  int64_t n_s;
  const float *u;           // [B, K + 1]
  int64_t u_sb, u_sk;
  int B, K, V;
  int *out;                 // [B, K + 1]
  int64_t o_sb;
  int *emitted;             // [B]
  unsigned *status;         // or null
  int ranks;                // CTAs a request (set by the launcher, as the next two)
  int range, seg;           // tokens a CTA, tokens a segment
};

cudaError_t launch_verify_draft(VerifyParams p, cudaStream_t stream);

}  // namespace fd
