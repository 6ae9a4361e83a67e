// step.h - host/device interface of a decode step over selected pages: slots
// for new tokens, cache writes, page selection, attention over the selected
// pages, log probabilities.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace fd {

// Pages and cache slots of new tokens.
struct SlotsParams {
  const int *seqlens;     // [B] keys before
  int64_t sl_s;
  const int *num_new;     // [B]
  int64_t n_s;
  const int *free_pages;  // [F]
  int64_t f_s;
  int F;
  const int *num_free;    // [1] or null: F
  int B, P, W;
  int64_t T;
  int *page_table;        // [B, W]
  int64_t pt_sb;
  void *slots;            // [T] int32 or int64
  int slots64;
  int *positions;         // [T] or null
  int *new_seqlens;       // [B]
  int *cu;                // [B + 1]
  int *pages_taken;       // [1]
  unsigned *status;       // or null
};

cudaError_t launch_append_slots(const SlotsParams &p, cudaStream_t stream);

// Keys and values of new tokens into the cache, and the bounds of changed pages.
struct CacheAppendParams {
  const __nv_bfloat16 *k, *v;  // [T, Hkv, D]
  int64_t k_st, k_sh, v_st, v_sh;
  const void *slots;           // [T] int32 or int64
  int slots64;
  int64_t s_s;
  int64_t T;
  int Hkv, P, log2_page;
  int64_t num_slots;           // num_pages * P
  unsigned char *k_cache, *v_cache;
  int64_t c_sp, c_ss, c_sh;    // byte strides of page, slot, head
  float *scales;               // [2, num_pages, P, Hkv, n_g] or null
  int64_t sc_sk, sc_sp, sc_ss, sc_sh;
  __nv_bfloat16 *bounds;       // [num_pages, Hkv, 2, D] or null
  int64_t b_sp, b_sh, b_sm;
  int chunk;                   // tokens a CTA (set by the launcher)
  unsigned *status;            // or null
};

cudaError_t launch_cache_append(int kind, int head_dim, CacheAppendParams p, cudaStream_t stream);

// Pages whose bounds allow the largest scores.
struct SelectParams {
  const __nv_bfloat16 *q;       // [B, Tq, Hq, D]
  int64_t q_sb, q_st, q_sh;
  const __nv_bfloat16 *bounds;  // [num_pages, Hkv, 2, D]
  int64_t b_sp, b_sh, b_sm;
  const int *page_table;        // [B, W]
  int64_t pt_sb;
  const int *seqlens;           // [B]
  int64_t sl_s;
  int num_pages, B, Tq, Hkv, G, P, W;
  int S, first, last;
  int *selected;                // [B, Tq, Hkv, S]
  int64_t s_sb, s_st, s_sh;
  unsigned *status;             // or null
  int ranks;                    // CTAs that share a choice (set by the launcher)
};

constexpr int kSelectMaxPages = 15360;  // page-table width that a choice can be made among (shared memory)

cudaError_t launch_select_pages(int head_dim, SelectParams p, cudaStream_t stream);

// Attention over selected pages.
struct SparseParams {
  const __nv_bfloat16 *q;  // [B, Tq, Hq, D]
  int64_t q_sb, q_st, q_sh;
  const unsigned char *k_cache, *v_cache;
  int64_t c_sp, c_ss, c_sh;  // byte strides of page, slot, head
  const float *scales;       // [2, num_pages, P, Hkv, n_g] or null
  int64_t sc_sk, sc_sp, sc_ss, sc_sh;
  const int *page_table;     // [B, W]
  int64_t pt_sb;
  const int *seqlens;        // [B]
  int64_t sl_s;
  const int *selected;       // [B, Tq, Hkv, S]
  int64_t s_sb, s_st, s_sh;
  int num_pages, B, Tq, Hkv, G, P, log2_page, W, S;
  int row_tiles;             // tiles of 8 or 16 query heads (set by the launcher)
  int ranks;                 // CTAs that share a list (set by the launcher)
  float scale_log2;          // softmax_scale * log2(e)
  void *out;                 // [B, Tq, Hq, D]
  int out_f32;
  int64_t o_sb, o_st, o_sh;
  float *lse;                // [B, Tq, Hq] or null
  int64_t l_sb, l_st, l_sh;
  unsigned *status;          // or null
};

cudaError_t launch_decode_sparse(int kind, int head_dim, SparseParams p, cudaStream_t stream);

// Log probabilities of given tokens.
struct LogprobsParams {
  const void *logits;  // [R, V] bf16 or fp32
  int f32;
  int64_t l_s;         // elements
  const void *tokens;  // [R] int32 or int64
  int tok64;
  int64_t t_s;
  int R, V, K;
  float *logprobs;     // [R]
  int *ranks;          // [R] or null
  float *entropy;      // [R] or null
  int *top_ids;        // [R, K] or null
  float *top_logprobs;
  int64_t ti_s, tl_s;
  unsigned *status;    // or null
  int ctas;            // CTAs a row (set by the launcher)
};

constexpr int kMaxTop = 32;

cudaError_t launch_token_logprobs(LogprobsParams p, cudaStream_t stream);

// A launch of clusters of `cluster` CTAs that may start while the kernel ahead
// of it ends (every kernel here waits for that one before its first access).
template <typename Kernel, typename Params>
inline cudaError_t launch_step(Kernel kernel, const Params &p, dim3 grid, int threads, size_t smem, int cluster,
                               cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace fd
