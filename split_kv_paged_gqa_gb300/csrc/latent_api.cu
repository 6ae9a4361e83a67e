// latent_api.cu - the C ABI of latent attention and draft verification:
// descriptor validation and launch. As in the rest of the C ABI a call checks
// its descriptors in O(1), reads no device memory on the host, never
// synchronises or allocates, and can be captured in a CUDA graph.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "checks.h"
#include "fd.h"
#include "latent.h"
#include "plan.h"

using fd::aligned;
using fd::check_tensor;
using fd::fail;

namespace {

thread_local unsigned g_wait_ns = fd::kLatWaitNs;  // fd_selftest_wait_limit

// Rows moved as 16-byte pieces: base and the given outer strides in multiples
// of 16 bytes. es is the element size.
fd_status check_rows16(const fd_tensor *t, const char *name, int es) {
  bool ok = aligned(t->data, 16);
  for (int i = 0; i + 1 < t->ndim; ++i) ok = ok && (t->shape[i] < 2 || (t->stride[i] * es) % 16 == 0);
  return ok ? FD_OK : fail(FD_ERR_UNSUPPORTED, "%s rows must be 16-byte aligned", name);
}

// Operands of TMA: no broadcast or reversed dimension.
fd_status check_tma(const fd_tensor *t, const char *name) {
  FD_TRY(check_rows16(t, name, 2));
  for (int i = 0; i + 1 < t->ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] <= 0)
      return fail(FD_ERR_UNSUPPORTED, "%s must not have a stride of zero or less", name);
  return FD_OK;
}

// Outputs: no two elements in one place (their writes would race).
fd_status check_distinct(const fd_tensor *t, const char *name) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] == 0)
      return fail(FD_ERR_UNSUPPORTED, "%s must not have a broadcast dimension", name);
  return FD_OK;
}

fd_status check_out(const fd_tensor *t, int ndim) {
  FD_TRY(check_tensor(t, "out", ndim));
  FD_TRY(check_distinct(t, "out"));
  if (t->dtype != FD_BF16 && t->dtype != FD_FP32) return fail(FD_ERR_INVALID_ARG, "out must be bf16 or fp32");
  return check_rows16(t, "out", t->dtype == FD_BF16 ? 2 : 4);
}

fd_status check_status(const fd_tensor *t) {
  if (!t || !t->data) return FD_OK;
  FD_TRY(check_tensor(t, "status", 1));
  if (t->dtype != FD_INT32 || t->shape[0] < 1) return fail(FD_ERR_INVALID_ARG, "status must be int32 [1]");
  return FD_OK;
}

// Tensor map of a latent cache, viewed as [page][block of 64 channels][slot][64]:
// boxes of three blocks x 64 slots of one page (8 slots for pages under 64),
// 128-byte swizzle. It depends only on pointer, shape and strides, which
// a serving loop keeps fixed: re-encoded only when they change.
fd_status latent_cache_map(CUtensorMap *map, const fd_tensor *c, fd_plan *pl) {
  fd_plan::MapEntry &e = pl->map_cache[0];
  bool hit = e.valid && e.data == c->data && e.shape[0] == c->shape[0];
  for (int i = 0; hit && i < 2; ++i) hit = e.stride[i] == c->stride[i];
  if (!hit) {
    fd::EncodeTiledFn fn = fd::encode_fn();
    if (!fn) return fail(FD_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    constexpr unsigned kBlocks = fd::kLatRow / 64;
    cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(pl->page), kBlocks, static_cast<cuuint64_t>(c->shape[0])};
    // a one-page pool's page stride is never used; the driver still wants a multiple of 16 bytes
    const int64_t sp = c->shape[0] > 1 ? c->stride[0] : static_cast<int64_t>(pl->page) * fd::kLatRow;
    cuuint64_t strides[3] = {static_cast<cuuint64_t>(c->stride[1] * 2), 128u, static_cast<cuuint64_t>(sp * 2)};
    cuuint32_t box[4] = {64u, pl->page >= 64 ? 64u : 8u, 3u, 1u};
    cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    e.valid = false;
    const CUresult r = fn(reinterpret_cast<CUtensorMap *>(e.map), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, c->data, dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
      return fail(FD_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled rejected the cache layout (%d)", (int)r);
    e.valid = true;
    e.data = c->data;
    e.shape[0] = c->shape[0];
    e.stride[0] = c->stride[0];
    e.stride[1] = c->stride[1];
  }
  std::memcpy(map, e.map, sizeof(CUtensorMap));
  return FD_OK;
}

// Tensor map of a prompt tensor [rows, (heads,) channels]: boxes of 64 channels
// x 128 rows of one head, 128-byte swizzle. Each thread keeps the last map of
// each of a call's tensors, re-encoded when pointer, shape or strides change.
fd_status rows_map(CUtensorMap *map, const fd_tensor *t, int which) {
  struct Entry {
    fd_tensor key;
    bool valid;
    alignas(64) unsigned char map[sizeof(CUtensorMap)];
  };
  static thread_local Entry cache[4];
  Entry &e = cache[which];
  bool hit = e.valid && e.key.data == t->data && e.key.ndim == t->ndim;
  for (int i = 0; hit && i < t->ndim; ++i) hit = e.key.shape[i] == t->shape[i] && e.key.stride[i] == t->stride[i];
  if (!hit) {
    fd::EncodeTiledFn fn = fd::encode_fn();
    if (!fn) return fail(FD_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const int nd = t->ndim;
    cuuint64_t dims[3], strides[2];
    cuuint32_t box[3], estr[3] = {1u, 1u, 1u};
    for (int i = 0; i < nd; ++i) {
      const int a = nd - 1 - i;  // innermost first
      dims[i] = static_cast<cuuint64_t>(t->shape[a]);
      // the stride of a dimension of one is never used; the driver still wants a multiple of 16 bytes
      if (i > 0) strides[i - 1] = t->shape[a] > 1 ? static_cast<cuuint64_t>(t->stride[a]) * 2 : 128u;
      box[i] = i == 0 ? 64u : (i == nd - 1 ? 128u : 1u);
    }
    e.valid = false;
    const CUresult r = fn(reinterpret_cast<CUtensorMap *>(e.map), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          static_cast<cuuint32_t>(nd), t->data, dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
      return fail(FD_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled rejected a prompt tensor's layout (%d)", (int)r);
    e.key = *t;
    e.valid = true;
  }
  std::memcpy(map, e.map, sizeof(CUtensorMap));
  return FD_OK;
}

}  // namespace

extern "C" fd_status fd_latent_plan_create(int device, int max_batch, int max_q_per_req, int num_heads,
                                           int page_size, float softmax_scale, fd_plan **plan) {
  if (!plan) return fail(FD_ERR_INVALID_ARG, "plan out-pointer is NULL");
  *plan = nullptr;
  if (max_batch < 1 || max_batch > 65535)
    return fail(FD_ERR_INVALID_ARG, "max_batch %d not in [1, 65535]", max_batch);
  if (max_q_per_req < 1 || max_q_per_req > 64)
    return fail(FD_ERR_INVALID_ARG, "max_q_per_req %d not in [1, 64]", max_q_per_req);
  if (num_heads < 1 || num_heads > 1024) return fail(FD_ERR_INVALID_ARG, "num_heads %d not in [1, 1024]", num_heads);
  int lp = 3;
  while (lp < 8 && (1 << lp) != page_size) ++lp;
  if ((1 << lp) != page_size)
    return fail(FD_ERR_UNSUPPORTED, "page_size %d must be a power of two in [8, 256]", page_size);
  if (!(softmax_scale > 0.f) || std::isinf(softmax_scale))
    return fail(FD_ERR_INVALID_ARG, "softmax_scale must be finite and > 0 (the absorbed form has no head dim to take it from)");

  fd_plan *pl = new (std::nothrow) fd_plan();
  if (!pl) return fail(FD_ERR_CUDA, "out of host memory");
  pl->latent = true;
  pl->device = device;
  pl->max_batch = max_batch;
  pl->max_q = max_q_per_req;
  pl->hq = num_heads;
  pl->hkv = 1;
  pl->d = fd::kLatC;
  pl->page = page_size;
  pl->log2_page = lp;
  pl->scale = softmax_scale;
  pl->cache_loaded = true;  // no tuning table
  if (device >= 0) {
    fd::DeviceGuard guard(device);
    cudaError_t e = guard.ok ? cudaSuccess : cudaErrorInvalidDevice;
    cudaDeviceProp prop;
    if (e == cudaSuccess) e = cudaGetDeviceProperties(&prop, device);
    if (e == cudaSuccess) {
      pl->num_sms = prop.multiProcessorCount;
      if (prop.major * 10 + prop.minor < 100) e = cudaErrorInvalidDevice;
    }
    const size_t row_tiles = (static_cast<size_t>(num_heads) * max_q_per_req + fd::kLatRowTile - 1) / fd::kLatRowTile;
    pl->ws_rows = 2 * fd::kLatRowTile * std::max<size_t>(pl->num_sms, row_tiles);
    if (e == cudaSuccess) e = cudaMalloc(&pl->o_part, pl->ws_rows * pl->d * sizeof(float));
    if (e == cudaSuccess) e = cudaMalloc(&pl->lse_part, pl->ws_rows * sizeof(float));
    if (e == cudaSuccess) e = fd::latent_decode_prepare();
    if (e == cudaSuccess && !fd::encode_fn()) e = cudaErrorSymbolNotFound;
    if (e == cudaSuccess) e = cudaMalloc(&pl->status, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemset(pl->status, 0, sizeof(unsigned));
    if (e != cudaSuccess) {
      fd_plan_destroy(pl);
      return fail(FD_ERR_CUDA, "plan setup on device %d failed: %s (%d)", device, cudaGetErrorString(e), (int)e);
    }
  }
  *plan = pl;
  return FD_OK;
}

extern "C" fd_status fd_selftest_wait_limit(unsigned limit_ns) {
  if (limit_ns > fd::kLatWaitNs)
    return fail(FD_ERR_INVALID_ARG, "limit %u ns outside [0, %u]", limit_ns, fd::kLatWaitNs);
  g_wait_ns = limit_ns ? limit_ns : fd::kLatWaitNs;
  return FD_OK;
}

extern "C" fd_status fd_decode_latent(const fd_tensor *q, const fd_tensor *kv_cache, const fd_tensor *page_table,
                                      const fd_tensor *cache_seqlens, int q_per_req, fd_tensor *out, fd_tensor *lse,
                                      fd_stream_t stream) {
  fd_plan *pl = fd_get_plan();
  if (!pl) return fail(FD_ERR_NO_PLAN, "no current plan on this thread (call fd_set_plan)");
  if (!pl->latent) return fail(FD_ERR_INVALID_ARG, "the current plan is not a latent plan (fd_latent_plan_create)");
  FD_TRY(check_tensor(q, "q", 4));
  if (q->dtype != FD_BF16) return fail(FD_ERR_INVALID_ARG, "q must be bf16");
  const int64_t B = q->shape[0], Tq = q->shape[1];
  if (q->shape[2] != pl->hq || q->shape[3] != fd::kLatRow)
    return fail(FD_ERR_INVALID_ARG, "q must be [B, Tq, H=%d, %d]", pl->hq, fd::kLatRow);
  if (B < 1 || B > pl->max_batch) return fail(FD_ERR_INVALID_ARG, "batch %lld not in [1, %d]", (long long)B, pl->max_batch);
  if (q_per_req != Tq) return fail(FD_ERR_INVALID_ARG, "q_per_req %d != q.shape[1] %lld", q_per_req, (long long)Tq);
  if (Tq < 1 || Tq > pl->max_q) return fail(FD_ERR_INVALID_ARG, "q_per_req %d not in [1, %d]", q_per_req, pl->max_q);
  FD_TRY(check_rows16(q, "q", 2));
  FD_TRY(check_tensor(kv_cache, "kv_cache", 3));
  if (kv_cache->dtype != FD_BF16) return fail(FD_ERR_INVALID_ARG, "kv_cache must be bf16");
  if (kv_cache->shape[0] < 1 || kv_cache->shape[0] > 0x7fffffff || kv_cache->shape[1] != pl->page ||
      kv_cache->shape[2] != fd::kLatRow)
    return fail(FD_ERR_INVALID_ARG, "kv_cache must be [num_pages, P=%d, %d]", pl->page, fd::kLatRow);
  FD_TRY(check_tma(kv_cache, "kv_cache"));
  FD_TRY(check_tensor(page_table, "page_table", 2));
  if (page_table->dtype != FD_INT32 || page_table->shape[0] != B || page_table->shape[1] < 1)
    return fail(FD_ERR_INVALID_ARG, "page_table must be int32 [B=%lld, W>=1]", (long long)B);
  if (page_table->shape[1] > (0x7fffffff - 255) / pl->page)  // (a length rounded up to tiles stays an int)
    return fail(FD_ERR_UNSUPPORTED, "page_table too wide");
  if (B * ((page_table->shape[1] * pl->page + 63) / 64 + 3) > 0x7fffffff)
    return fail(FD_ERR_UNSUPPORTED, "page_table holds more than 2^31 tiles of 64 keys");
  FD_TRY(check_tensor(cache_seqlens, "cache_seqlens", 1, false));
  if (cache_seqlens->dtype != FD_INT32 || cache_seqlens->shape[0] != B)
    return fail(FD_ERR_INVALID_ARG, "cache_seqlens must be int32 [B=%lld]", (long long)B);
  FD_TRY(check_out(out, 4));
  if (out->shape[0] != B || out->shape[1] != Tq || out->shape[2] != pl->hq || out->shape[3] != fd::kLatC)
    return fail(FD_ERR_INVALID_ARG, "out must be [B, Tq, H, %d]", fd::kLatC);
  if (lse && lse->data) {
    FD_TRY(check_tensor(lse, "lse", 3, false));
    if (lse->dtype != FD_FP32 || lse->shape[0] != B || lse->shape[1] != Tq || lse->shape[2] != pl->hq)
      return fail(FD_ERR_INVALID_ARG, "lse must be fp32 [B, Tq, H]");
    FD_TRY(check_distinct(lse, "lse"));
  }
  if (pl->device < 0) return fail(FD_ERR_WORKSPACE, "host-only plan cannot decode");
  fd::DeviceGuard guard(pl->device);
  if (!guard.ok) return fail(FD_ERR_CUDA, "cannot make device %d current", pl->device);

  fd::LatentDecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16 *>(q->data);
  p.q_sb = q->stride[0];
  p.q_st = q->stride[1];
  p.q_sh = q->stride[2];
  p.page_table = static_cast<const int *>(page_table->data);
  p.pt_sb = page_table->stride[0];
  p.seqlens = static_cast<const int *>(cache_seqlens->data);
  p.sl_s = cache_seqlens->stride[0];
  p.num_pages = static_cast<int>(kv_cache->shape[0]);
  p.page_size = pl->page;
  p.log2_page = pl->log2_page;
  p.max_pages = static_cast<int>(page_table->shape[1]);
  p.B = static_cast<int>(B);
  p.Tq = static_cast<int>(Tq);
  p.H = pl->hq;
  p.R = p.Tq * p.H;
  p.row_tiles = (p.R + fd::kLatRowTile - 1) / fd::kLatRowTile;
  p.rows_per_tile = ((p.R + p.row_tiles - 1) / p.row_tiles + 15) / 16 * 16;
  p.groups = std::max(1, pl->num_sms / p.row_tiles);
  p.change = 1 + p.rows_per_tile / 32;  // (at most 3)
  if (p.row_tiles > 1 && kv_cache->stride[1] == fd::kLatRow) {  // (a page's rows are one run of bytes)
    p.cache = static_cast<const __nv_bfloat16 *>(kv_cache->data);
    p.c_sp = kv_cache->stride[0];
  }
  p.o_part = pl->o_part;
  p.lse_part = pl->lse_part;
  p.scale_log2 = pl->scale * 1.4426950408889634f;
  p.out = out->data;
  p.out_f32 = out->dtype == FD_FP32;
  p.o_sb = out->stride[0];
  p.o_st = out->stride[1];
  p.o_sh = out->stride[2];
  if (lse && lse->data) {
    p.lse = static_cast<float *>(lse->data);
    p.l_sb = lse->stride[0];
    p.l_st = lse->stride[1];
    p.l_sh = lse->stride[2];
  }
  p.status = pl->status;
  p.wait_ns = g_wait_ns;
  p.hint_ns = std::min(p.wait_ns, fd::kLatHintNs);
  CUtensorMap tmc;
  FD_TRY(latent_cache_map(&tmc, kv_cache, pl));
  const cudaError_t e = fd::launch_latent_decode(tmc, p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FD_ERR_CUDA, "latent decode launch failed: %s (%d)", cudaGetErrorString(e), (int)e);
  return FD_OK;
}

extern "C" fd_status fd_prefill_latent(const fd_tensor *q, const fd_tensor *k_nope, const fd_tensor *k_pe,
                                       const fd_tensor *v, const fd_tensor *cu_seqlens_q,
                                       const fd_tensor *cu_seqlens_k, int max_seqlen_q, float softmax_scale,
                                       fd_tensor *out, fd_tensor *lse, fd_tensor *status, fd_stream_t stream) {
  constexpr int64_t kMax = 0x7fffffff;
  FD_TRY(check_tensor(q, "q", 3));
  if (q->dtype != FD_BF16) return fail(FD_ERR_INVALID_ARG, "q must be bf16");
  const int64_t Sq = q->shape[0], H = q->shape[1];
  if (Sq < 1 || Sq > kMax || H < 1 || H > 65535 || q->shape[2] != fd::kLatNope + fd::kLatR)
    return fail(FD_ERR_INVALID_ARG, "q must be [Sq>=1, 1<=H<=65535, %d]", fd::kLatNope + fd::kLatR);
  FD_TRY(check_tma(q, "q"));
  FD_TRY(check_tensor(k_nope, "k_nope", 3));
  const int64_t Sk = k_nope->shape[0];
  if (k_nope->dtype != FD_BF16 || Sk < 1 || Sk > kMax || k_nope->shape[1] != H || k_nope->shape[2] != fd::kLatNope)
    return fail(FD_ERR_INVALID_ARG, "k_nope must be bf16 [Sk>=1, H=%lld, %d]", (long long)H, fd::kLatNope);
  FD_TRY(check_tma(k_nope, "k_nope"));
  FD_TRY(check_tensor(k_pe, "k_pe", 2));
  if (k_pe->dtype != FD_BF16 || k_pe->shape[0] != Sk || k_pe->shape[1] != fd::kLatR)
    return fail(FD_ERR_INVALID_ARG, "k_pe must be bf16 [Sk=%lld, %d]", (long long)Sk, fd::kLatR);
  FD_TRY(check_tma(k_pe, "k_pe"));
  FD_TRY(check_tensor(v, "v", 3));
  if (v->dtype != FD_BF16 || v->shape[0] != Sk || v->shape[1] != H || v->shape[2] != fd::kLatV)
    return fail(FD_ERR_INVALID_ARG, "v must be bf16 [Sk=%lld, H=%lld, %d]", (long long)Sk, (long long)H, fd::kLatV);
  FD_TRY(check_tma(v, "v"));
  FD_TRY(check_tensor(cu_seqlens_q, "cu_seqlens_q", 1));
  const int64_t B = cu_seqlens_q->shape[0] - 1;
  if (cu_seqlens_q->dtype != FD_INT32 || B < 1 || B > 65535)
    return fail(FD_ERR_INVALID_ARG, "cu_seqlens_q must be int32 [B + 1], B in [1, 65535]");
  FD_TRY(check_tensor(cu_seqlens_k, "cu_seqlens_k", 1));
  if (cu_seqlens_k->dtype != FD_INT32 || cu_seqlens_k->shape[0] != B + 1)
    return fail(FD_ERR_INVALID_ARG, "cu_seqlens_k must be int32 [B + 1 = %lld]", (long long)(B + 1));
  if (max_seqlen_q < 1) return fail(FD_ERR_INVALID_ARG, "max_seqlen_q %d < 1", max_seqlen_q);
  if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale))
    return fail(FD_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
  FD_TRY(check_out(out, 3));
  if (out->shape[0] != Sq || out->shape[1] != H || out->shape[2] != fd::kLatV)
    return fail(FD_ERR_INVALID_ARG, "out must be [Sq=%lld, H=%lld, %d]", (long long)Sq, (long long)H, fd::kLatV);
  if (lse && lse->data) {
    FD_TRY(check_tensor(lse, "lse", 2, false));
    if (lse->dtype != FD_FP32 || lse->shape[0] != Sq || lse->shape[1] != H)
      return fail(FD_ERR_INVALID_ARG, "lse must be fp32 [Sq, H]");
    FD_TRY(check_distinct(lse, "lse"));
  }
  FD_TRY(check_status(status));

  fd::LatentPrefillParams p;
  std::memset(&p, 0, sizeof(p));
  p.cu_q = static_cast<const int *>(cu_seqlens_q->data);
  p.cu_k = static_cast<const int *>(cu_seqlens_k->data);
  p.B = static_cast<int>(B);
  p.H = static_cast<int>(H);
  p.Sq = static_cast<int>(Sq);
  p.Sk = static_cast<int>(Sk);
  p.max_q = static_cast<int>(std::min<int64_t>(max_seqlen_q, Sq));
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt(static_cast<float>(fd::kLatNope + fd::kLatR));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out->data;
  p.out_f32 = out->dtype == FD_FP32;
  p.o_ss = out->stride[0];
  p.o_sh = out->stride[1];
  if (lse && lse->data) {
    p.lse = static_cast<float *>(lse->data);
    p.l_ss = lse->stride[0];
    p.l_sh = lse->stride[1];
  }
  p.status = status && status->data ? static_cast<unsigned *>(status->data) : nullptr;
  p.wait_ns = g_wait_ns;
  const int es = p.out_f32 ? 4 : 2;
  p.wide = aligned(out->data, 32) && (p.o_ss * es) % 32 == 0 && (p.o_sh * es) % 32 == 0;
  // Tiles of 256 queries: as many as the longest request has for each, or what Sq
  // rows of B requests can fill where that is less, and by enough: a CTA without a
  // tile costs 0.6 us, and one that finds its tile 0.35 us for each 32 requests
  // ahead of its own (half of B on average).
  const int64_t each = (p.max_q + 255ll) / 256 * B, fill = Sq / 256 + B;
  p.ragged = (each - fill) * 64 * 2 > fill * B;
  const int64_t tiles = p.ragged ? fill : each;
  if (tiles * H > kMax) return fail(FD_ERR_UNSUPPORTED, "too many tiles of 256 queries");
  p.tiles = static_cast<int>(tiles);
  CUtensorMap tm[4];
  FD_TRY(rows_map(&tm[0], q, 0));
  FD_TRY(rows_map(&tm[1], k_nope, 1));
  FD_TRY(rows_map(&tm[2], k_pe, 2));
  FD_TRY(rows_map(&tm[3], v, 3));
  const cudaError_t e = fd::launch_latent_prefill(tm, p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FD_ERR_CUDA, "latent prefill launch failed: %s (%d)", cudaGetErrorString(e), (int)e);
  return FD_OK;
}

extern "C" fd_status fd_verify_draft(const fd_tensor *target_probs, const fd_tensor *draft_probs,
                                     const fd_tensor *draft_tokens, const fd_tensor *num_draft,
                                     const fd_tensor *uniforms, fd_tensor *out_tokens, fd_tensor *num_emitted,
                                     fd_tensor *status, fd_stream_t stream) {
  FD_TRY(check_tensor(target_probs, "target_probs", 3));
  const int64_t B = target_probs->shape[0], K = target_probs->shape[1] - 1, V = target_probs->shape[2];
  if (target_probs->dtype != FD_FP32 || B < 1 || B > 65535 || K < 0 || K > 64 || V < 1 || V > (1 << 24))
    return fail(FD_ERR_INVALID_ARG, "target_probs must be fp32 [1<=B<=65535, 1<=K+1<=65, 1<=V<=2^24]");
  const bool has_draft = draft_probs && draft_probs->data;
  if (has_draft) {
    FD_TRY(check_tensor(draft_probs, "draft_probs", 3));
    if (draft_probs->dtype != FD_FP32 || draft_probs->shape[0] != B || draft_probs->shape[1] != K ||
        draft_probs->shape[2] != V)
      return fail(FD_ERR_INVALID_ARG, "draft_probs must be fp32 [B=%lld, K=%lld, V=%lld]", (long long)B, (long long)K,
                  (long long)V);
  }
  if (K > 0) {
    FD_TRY(check_tensor(draft_tokens, "draft_tokens", 2, false));
    if ((draft_tokens->dtype != FD_INT32 && draft_tokens->dtype != FD_INT64) || draft_tokens->shape[0] != B ||
        draft_tokens->shape[1] != K)
      return fail(FD_ERR_INVALID_ARG, "draft_tokens must be int32 or int64 [B=%lld, K=%lld]", (long long)B, (long long)K);
  }
  const bool has_num = num_draft && num_draft->data;
  if (has_num) {
    FD_TRY(check_tensor(num_draft, "num_draft", 1, false));
    if (num_draft->dtype != FD_INT32 || num_draft->shape[0] != B)
      return fail(FD_ERR_INVALID_ARG, "num_draft must be int32 [B=%lld]", (long long)B);
  }
  FD_TRY(check_tensor(uniforms, "uniforms", 2, false));
  if (uniforms->dtype != FD_FP32 || uniforms->shape[0] != B || uniforms->shape[1] != K + 1)
    return fail(FD_ERR_INVALID_ARG, "uniforms must be fp32 [B=%lld, K+1=%lld]", (long long)B, (long long)(K + 1));
  FD_TRY(check_tensor(out_tokens, "out_tokens", 2));
  if (out_tokens->dtype != FD_INT32 || out_tokens->shape[0] != B || out_tokens->shape[1] != K + 1)
    return fail(FD_ERR_INVALID_ARG, "out_tokens must be int32 [B=%lld, K+1=%lld]", (long long)B, (long long)(K + 1));
  FD_TRY(check_distinct(out_tokens, "out_tokens"));
  FD_TRY(check_tensor(num_emitted, "num_emitted", 1));
  if (num_emitted->dtype != FD_INT32 || num_emitted->shape[0] != B)
    return fail(FD_ERR_INVALID_ARG, "num_emitted must be int32 [B=%lld]", (long long)B);
  FD_TRY(check_status(status));

  fd::VerifyParams p;
  std::memset(&p, 0, sizeof(p));
  p.target = static_cast<const float *>(target_probs->data);
  p.t_sb = target_probs->stride[0];
  p.t_sk = target_probs->stride[1];
  if (has_draft) {
    p.draft = static_cast<const float *>(draft_probs->data);
    p.d_sb = draft_probs->stride[0];
    p.d_sk = draft_probs->stride[1];
  }
  if (K > 0) {
    p.tokens = draft_tokens->data;
    p.tok64 = draft_tokens->dtype == FD_INT64;
    p.x_sb = draft_tokens->stride[0];
    p.x_sk = draft_tokens->stride[1];
  }
  if (has_num) {
    p.num_draft = static_cast<const int *>(num_draft->data);
    p.n_s = num_draft->stride[0];
  }
  p.u = static_cast<const float *>(uniforms->data);
  p.u_sb = uniforms->stride[0];
  p.u_sk = uniforms->stride[1];
  p.B = static_cast<int>(B);
  p.K = static_cast<int>(K);
  p.V = static_cast<int>(V);
  p.out = static_cast<int *>(out_tokens->data);
  p.o_sb = out_tokens->stride[0];
  p.emitted = static_cast<int *>(num_emitted->data);
  p.status = status && status->data ? static_cast<unsigned *>(status->data) : nullptr;
  const cudaError_t e = fd::launch_verify_draft(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(FD_ERR_CUDA, "verify launch failed: %s (%d)", cudaGetErrorString(e), (int)e);
  return FD_OK;
}
