// step_api.cu - the C ABI of a decode step over selected pages: descriptor
// validation and launch. As in the rest of the C ABI a call checks its
// descriptors in O(1), reads no device memory on the host, never synchronises or
// allocates, and can be captured in a CUDA graph.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "checks.h"
#include "fd.h"
#include "plan.h"
#include "step.h"

using fd::aligned;
using fd::check_distinct;
using fd::check_rows16;
using fd::check_status;
using fd::check_tensor;
using fd::fail;

namespace {

constexpr int64_t kInt = 0x7fffffff;

bool given(const fd_tensor *t) { return t && t->data; }

// int32 [n] of any stride (n < 0: any length); outputs are contiguous
fd_status check_ints(const fd_tensor *t, const char *name, int64_t n, bool output) {
  FD_TRY(check_tensor(t, name, 1, output));
  if (t->dtype != FD_INT32 || (n >= 0 && t->shape[0] != n))
    return n < 0 ? fail(FD_ERR_INVALID_ARG, "%s must be an int32 vector", name)
                 : fail(FD_ERR_INVALID_ARG, "%s must be int32 [%lld]", name, (long long)n);
  return FD_OK;
}

// Bytes that a vector spans, from its first element.
int64_t span(const fd_tensor *t, int es) { return t->shape[0] > 0 ? ((t->shape[0] - 1) * t->stride[0] + 1) * es : 0; }

bool overlap(const fd_tensor *a, const fd_tensor *b) {
  const char *x = static_cast<const char *>(a->data), *y = static_cast<const char *>(b->data);
  return x < y + span(b, 4) && y < x + span(a, 4);
}

fd_status check_page_size(int64_t page_size, int *log2_page) {
  int lp = 3;
  while (lp < 8 && (1 << lp) != page_size) ++lp;
  if ((1 << lp) != page_size)
    return fail(FD_ERR_UNSUPPORTED, "page size %lld must be a power of two in [8, 256]", (long long)page_size);
  *log2_page = lp;
  return FD_OK;
}

struct Caches {
  int kind, D, Hkv, P, log2_page, num_pages, es;
};

// k_cache, v_cache and kv_scales of any of the three cache types. (Hkv and D < 0: taken from the cache.)
fd_status check_caches(const fd_tensor *k, const fd_tensor *v, const fd_tensor *scales, int64_t Hkv, int64_t D, Caches *c) {
  FD_TRY(check_tensor(k, "k_cache", 4));
  FD_TRY(check_tensor(v, "v_cache", 4));
  if (k->dtype != FD_BF16 && k->dtype != FD_INT8 && k->dtype != FD_INT4X2)
    return fail(FD_ERR_INVALID_ARG, "k_cache must be bf16, int8 or int4x2");
  c->kind = k->dtype == FD_BF16 ? fd::KV_BF16 : (k->dtype == FD_INT8 ? fd::KV_I8 : fd::KV_I4);
  c->es = k->dtype == FD_BF16 ? 2 : 1;
  if (D != 64 && D != 128) return fail(FD_ERR_UNSUPPORTED, "head_dim %lld must be 64 or 128", (long long)D);
  const int64_t rowe = c->kind == fd::KV_I4 ? D / 2 : D;
  if (k->shape[0] < 1 || k->shape[0] > kInt || k->shape[2] < 1 || (Hkv >= 0 && k->shape[2] != Hkv) || k->shape[3] != rowe)
    return fail(FD_ERR_INVALID_ARG, "k_cache must be [num_pages>=1, P, Hkv, %lld]", (long long)rowe);
  if (v->dtype != k->dtype) return fail(FD_ERR_INVALID_ARG, "v_cache's type differs from k_cache's");
  for (int i = 0; i < 4; ++i) {
    if (v->shape[i] != k->shape[i]) return fail(FD_ERR_INVALID_ARG, "k_cache and v_cache shapes differ");
    if (v->shape[i] > 1 && v->stride[i] != k->stride[i])
      return fail(FD_ERR_UNSUPPORTED, "k_cache and v_cache strides differ");
  }
  FD_TRY(check_rows16(k, "k_cache", c->es));
  FD_TRY(check_rows16(v, "v_cache", c->es));
  FD_TRY(check_page_size(k->shape[1], &c->log2_page));
  c->P = static_cast<int>(k->shape[1]);
  c->D = static_cast<int>(D);
  c->Hkv = static_cast<int>(k->shape[2]);
  c->num_pages = static_cast<int>(k->shape[0]);
  if (c->Hkv > 1024) return fail(FD_ERR_UNSUPPORTED, "more than 1024 KV heads");
  if (c->kind == fd::KV_BF16) {
    if (given(scales)) return fail(FD_ERR_INVALID_ARG, "kv_scales must be NULL for a bf16 cache");
    return FD_OK;
  }
  const int ng = c->kind == fd::KV_I8 ? 1 : c->D / 32;
  FD_TRY(check_tensor(scales, "kv_scales", 5));
  if (scales->dtype != FD_FP32 || scales->shape[0] != 2 || scales->shape[1] != k->shape[0] || scales->shape[2] != c->P ||
      scales->shape[3] != c->Hkv || scales->shape[4] != ng)
    return fail(FD_ERR_INVALID_ARG, "kv_scales must be fp32 [2, %d, %d, %d, %d]", c->num_pages, c->P, c->Hkv, ng);
  bool ok = aligned(scales->data, 4 * ng);
  for (int i = 0; i < 4; ++i) ok = ok && (scales->shape[i] < 2 || scales->stride[i] % ng == 0);
  if (!ok) return fail(FD_ERR_UNSUPPORTED, "kv_scales rows must be %d-byte aligned", 4 * ng);
  return FD_OK;
}

fd_status check_bounds(const fd_tensor *t, int64_t num_pages, int64_t Hkv, int64_t D) {
  FD_TRY(check_tensor(t, "page_bounds", 4));
  if (t->dtype != FD_BF16 || t->shape[0] < 1 || t->shape[0] > kInt || (num_pages >= 0 && t->shape[0] != num_pages) ||
      t->shape[1] < 1 || t->shape[1] > 1024 || (Hkv >= 0 && t->shape[1] != Hkv) || t->shape[2] != 2 || t->shape[3] != D)
    return fail(FD_ERR_INVALID_ARG, "page_bounds must be bf16 [num_pages, Hkv, 2, %lld]", (long long)D);
  return check_rows16(t, "page_bounds", 2);
}

// q, page_table, cache_seqlens of a decode call
fd_status check_query(const fd_tensor *q, const fd_tensor *page_table, const fd_tensor *seqlens, int q_per_req, int64_t Hkv,
                      int page_size) {
  FD_TRY(check_tensor(q, "q", 4));
  if (q->dtype != FD_BF16) return fail(FD_ERR_INVALID_ARG, "q must be bf16");
  const int64_t B = q->shape[0], Tq = q->shape[1], Hq = q->shape[2], D = q->shape[3];
  if (D != 64 && D != 128) return fail(FD_ERR_UNSUPPORTED, "head_dim %lld must be 64 or 128", (long long)D);
  if (B < 1 || B > 65535) return fail(FD_ERR_INVALID_ARG, "batch %lld not in [1, 65535]", (long long)B);
  if (Tq < 1 || Tq > 64) return fail(FD_ERR_INVALID_ARG, "q.shape[1] %lld not in [1, 64]", (long long)Tq);
  if (q_per_req != Tq) return fail(FD_ERR_INVALID_ARG, "q_per_req %d != q.shape[1] %lld", q_per_req, (long long)Tq);
  if (Hq < Hkv || Hq % Hkv || Hq > 4096)
    return fail(FD_ERR_INVALID_ARG, "%lld query heads are no multiple of %lld KV heads in [1, 4096]", (long long)Hq, (long long)Hkv);
  FD_TRY(check_rows16(q, "q", 2));
  FD_TRY(check_tensor(page_table, "page_table", 2));
  if (page_table->dtype != FD_INT32 || page_table->shape[0] != B || page_table->shape[1] < 1)
    return fail(FD_ERR_INVALID_ARG, "page_table must be int32 [B=%lld, W>=1]", (long long)B);
  if (page_table->shape[1] > (kInt - 255) / page_size) return fail(FD_ERR_UNSUPPORTED, "page_table too wide");
  return check_ints(seqlens, "cache_seqlens", B, false);
}

fd_status launched(cudaError_t e, const char *what) {
  if (e != cudaSuccess) return fail(FD_ERR_CUDA, "%s launch failed: %s (%d)", what, cudaGetErrorString(e), (int)e);
  return FD_OK;
}

unsigned *status_word(const fd_tensor *t) { return given(t) ? static_cast<unsigned *>(t->data) : nullptr; }

}  // namespace

extern "C" fd_status fd_append_slots(const fd_tensor *cache_seqlens, const fd_tensor *num_new, const fd_tensor *free_pages,
                                     const fd_tensor *num_free, int page_size, fd_tensor *page_table, fd_tensor *slots,
                                     fd_tensor *positions, fd_tensor *new_seqlens, fd_tensor *cu_seqlens_q,
                                     fd_tensor *pages_taken, fd_tensor *status, fd_stream_t stream) {
  FD_TRY(check_ints(cache_seqlens, "cache_seqlens", -1, false));
  const int64_t B = cache_seqlens->shape[0];
  if (B < 1 || B > 65535) return fail(FD_ERR_INVALID_ARG, "batch %lld not in [1, 65535]", (long long)B);
  FD_TRY(check_ints(num_new, "num_new", B, false));
  FD_TRY(check_ints(free_pages, "free_pages", -1, false));
  if (free_pages->shape[0] < 1 || free_pages->shape[0] > kInt)
    return fail(FD_ERR_INVALID_ARG, "free_pages must hold 1 .. 2^31-1 pages");
  if (given(num_free)) FD_TRY(check_ints(num_free, "num_free", 1, false));
  if (page_size < 1) return fail(FD_ERR_INVALID_ARG, "page_size %d < 1", page_size);
  FD_TRY(check_tensor(page_table, "page_table", 2));
  if (page_table->dtype != FD_INT32 || page_table->shape[0] != B || page_table->shape[1] < 1 || page_table->shape[1] > kInt)
    return fail(FD_ERR_INVALID_ARG, "page_table must be int32 [B=%lld, W>=1]", (long long)B);
  FD_TRY(check_distinct(page_table, "page_table"));
  FD_TRY(check_tensor(slots, "slots", 1));
  const int64_t T = slots->shape[0];
  if ((slots->dtype != FD_INT32 && slots->dtype != FD_INT64) || T < 1 || T > kInt)
    return fail(FD_ERR_INVALID_ARG, "slots must be int32 or int64 [1 .. 2^31-1]");
  if (given(positions)) FD_TRY(check_ints(positions, "positions", T, true));
  FD_TRY(check_ints(new_seqlens, "new_seqlens", B, true));
  FD_TRY(check_ints(cu_seqlens_q, "cu_seqlens_q", B + 1, true));
  FD_TRY(check_ints(pages_taken, "pages_taken", 1, true));
  FD_TRY(check_status(status));
  // (CTAs read the requests' numbers while others write)
  const fd_tensor *ins[4] = {cache_seqlens, num_new, free_pages, given(num_free) ? num_free : nullptr};
  const fd_tensor *outs[3] = {new_seqlens, cu_seqlens_q, pages_taken};
  for (const fd_tensor *a : ins)
    for (const fd_tensor *b : outs)
      if (a && overlap(a, b)) return fail(FD_ERR_UNSUPPORTED, "outputs must not overlap inputs");

  fd::SlotsParams p;
  std::memset(&p, 0, sizeof(p));
  p.seqlens = static_cast<const int *>(cache_seqlens->data);
  p.sl_s = cache_seqlens->stride[0];
  p.num_new = static_cast<const int *>(num_new->data);
  p.n_s = num_new->stride[0];
  p.free_pages = static_cast<const int *>(free_pages->data);
  p.f_s = free_pages->stride[0];
  p.F = static_cast<int>(free_pages->shape[0]);
  p.num_free = given(num_free) ? static_cast<const int *>(num_free->data) : nullptr;
  p.B = static_cast<int>(B);
  p.P = page_size;
  p.W = static_cast<int>(page_table->shape[1]);
  p.T = T;
  p.page_table = static_cast<int *>(page_table->data);
  p.pt_sb = page_table->stride[0];
  p.slots = slots->data;
  p.slots64 = slots->dtype == FD_INT64;
  p.positions = given(positions) ? static_cast<int *>(positions->data) : nullptr;
  p.new_seqlens = static_cast<int *>(new_seqlens->data);
  p.cu = static_cast<int *>(cu_seqlens_q->data);
  p.pages_taken = static_cast<int *>(pages_taken->data);
  p.status = status_word(status);
  return launched(fd::launch_append_slots(p, reinterpret_cast<cudaStream_t>(stream)), "append slots");
}

extern "C" fd_status fd_cache_append(const fd_tensor *k, const fd_tensor *v, const fd_tensor *slots, fd_tensor *k_cache,
                                     fd_tensor *v_cache, fd_tensor *kv_scales, fd_tensor *page_bounds, fd_tensor *status,
                                     fd_stream_t stream) {
  FD_TRY(check_tensor(k, "k", 3));
  FD_TRY(check_tensor(v, "v", 3));
  const int64_t T = k->shape[0], Hkv = k->shape[1], D = k->shape[2];
  if (k->dtype != FD_BF16 || v->dtype != FD_BF16) return fail(FD_ERR_INVALID_ARG, "k and v must be bf16");
  if (T < 1 || T > kInt || Hkv < 1) return fail(FD_ERR_INVALID_ARG, "k must be [1 <= T <= 2^31-1, Hkv>=1, D]");
  for (int i = 0; i < 3; ++i)
    if (v->shape[i] != k->shape[i]) return fail(FD_ERR_INVALID_ARG, "k and v shapes differ");
  FD_TRY(check_rows16(k, "k", 2));
  FD_TRY(check_rows16(v, "v", 2));
  FD_TRY(check_tensor(slots, "slots", 1, false));
  if ((slots->dtype != FD_INT32 && slots->dtype != FD_INT64) || slots->shape[0] != T)
    return fail(FD_ERR_INVALID_ARG, "slots must be int32 or int64 [T=%lld]", (long long)T);
  Caches c;
  FD_TRY(check_caches(k_cache, v_cache, kv_scales, Hkv, D, &c));
  FD_TRY(check_distinct(k_cache, "k_cache"));
  FD_TRY(check_distinct(v_cache, "v_cache"));
  if (c.kind != fd::KV_BF16) FD_TRY(check_distinct(kv_scales, "kv_scales"));
  if (given(page_bounds)) {
    FD_TRY(check_bounds(page_bounds, c.num_pages, Hkv, D));
    FD_TRY(check_distinct(page_bounds, "page_bounds"));
  }
  FD_TRY(check_status(status));

  fd::CacheAppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.k = static_cast<const __nv_bfloat16 *>(k->data);
  p.v = static_cast<const __nv_bfloat16 *>(v->data);
  p.k_st = k->stride[0];
  p.k_sh = k->stride[1];
  p.v_st = v->stride[0];
  p.v_sh = v->stride[1];
  p.slots = slots->data;
  p.slots64 = slots->dtype == FD_INT64;
  p.s_s = slots->stride[0];
  p.T = T;
  p.Hkv = c.Hkv;
  p.P = c.P;
  p.log2_page = c.log2_page;
  p.num_slots = static_cast<int64_t>(c.num_pages) * c.P;
  p.k_cache = static_cast<unsigned char *>(k_cache->data);
  p.v_cache = static_cast<unsigned char *>(v_cache->data);
  p.c_sp = k_cache->stride[0] * c.es;
  p.c_ss = k_cache->stride[1] * c.es;
  p.c_sh = k_cache->stride[2] * c.es;
  if (c.kind != fd::KV_BF16) {
    p.scales = static_cast<float *>(kv_scales->data);
    p.sc_sk = kv_scales->stride[0];
    p.sc_sp = kv_scales->stride[1];
    p.sc_ss = kv_scales->stride[2];
    p.sc_sh = kv_scales->stride[3];
  }
  if (given(page_bounds)) {
    p.bounds = static_cast<__nv_bfloat16 *>(page_bounds->data);
    p.b_sp = page_bounds->stride[0];
    p.b_sh = page_bounds->stride[1];
    p.b_sm = page_bounds->stride[2];
  }
  p.status = status_word(status);
  return launched(fd::launch_cache_append(c.kind, c.D, p, reinterpret_cast<cudaStream_t>(stream)), "cache append");
}

extern "C" fd_status fd_select_pages(const fd_tensor *q, const fd_tensor *page_bounds, const fd_tensor *page_table,
                                     const fd_tensor *cache_seqlens, int q_per_req, int page_size, int num_first, int num_last,
                                     fd_tensor *selected, fd_tensor *status, fd_stream_t stream) {
  FD_TRY(check_tensor(q, "q", 4));
  FD_TRY(check_bounds(page_bounds, -1, -1, q->shape[3]));
  const int64_t Hkv = page_bounds->shape[1];
  int log2_page;
  FD_TRY(check_page_size(page_size, &log2_page));
  FD_TRY(check_query(q, page_table, cache_seqlens, q_per_req, Hkv, page_size));
  const int64_t B = q->shape[0], Tq = q->shape[1];
  if (page_table->shape[1] > fd::kSelectMaxPages)
    return fail(FD_ERR_UNSUPPORTED, "page_table is wider than %d pages", fd::kSelectMaxPages);
  if (B * Tq * Hkv > kInt / 8) return fail(FD_ERR_UNSUPPORTED, "more than 2^28 choices");
  FD_TRY(check_tensor(selected, "selected", 4));
  const int64_t S = selected->shape[3];
  if (selected->dtype != FD_INT32 || selected->shape[0] != B || selected->shape[1] != Tq || selected->shape[2] != Hkv || S < 1 ||
      S > kInt)
    return fail(FD_ERR_INVALID_ARG, "selected must be int32 [B=%lld, Tq=%lld, Hkv=%lld, S>=1]", (long long)B, (long long)Tq,
                (long long)Hkv);
  FD_TRY(check_distinct(selected, "selected"));
  if (num_first < 0 || num_last < 1 || static_cast<int64_t>(num_first) + num_last > S)
    return fail(FD_ERR_INVALID_ARG, "num_first %d >= 0 and num_last %d >= 1 must fit S=%lld pages", num_first, num_last, (long long)S);
  FD_TRY(check_status(status));

  fd::SelectParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16 *>(q->data);
  p.q_sb = q->stride[0];
  p.q_st = q->stride[1];
  p.q_sh = q->stride[2];
  p.bounds = static_cast<const __nv_bfloat16 *>(page_bounds->data);
  p.b_sp = page_bounds->stride[0];
  p.b_sh = page_bounds->stride[1];
  p.b_sm = page_bounds->stride[2];
  p.page_table = static_cast<const int *>(page_table->data);
  p.pt_sb = page_table->stride[0];
  p.seqlens = static_cast<const int *>(cache_seqlens->data);
  p.sl_s = cache_seqlens->stride[0];
  p.num_pages = static_cast<int>(page_bounds->shape[0]);
  p.B = static_cast<int>(B);
  p.Tq = static_cast<int>(Tq);
  p.Hkv = static_cast<int>(Hkv);
  p.G = static_cast<int>(q->shape[2] / Hkv);
  p.P = page_size;
  p.W = static_cast<int>(page_table->shape[1]);
  p.S = static_cast<int>(S);
  p.first = num_first;
  p.last = num_last;
  p.selected = static_cast<int *>(selected->data);
  p.s_sb = selected->stride[0];
  p.s_st = selected->stride[1];
  p.s_sh = selected->stride[2];
  p.status = status_word(status);
  return launched(fd::launch_select_pages(static_cast<int>(q->shape[3]), p, reinterpret_cast<cudaStream_t>(stream)),
                  "page selection");
}

extern "C" fd_status fd_token_logprobs(const fd_tensor *logits, const fd_tensor *tokens, fd_tensor *logprobs, fd_tensor *ranks,
                                       fd_tensor *entropy, fd_tensor *top_ids, fd_tensor *top_logprobs, fd_tensor *status,
                                       fd_stream_t stream) {
  FD_TRY(check_tensor(logits, "logits", 2));
  const int64_t R = logits->shape[0], V = logits->shape[1];
  if (logits->dtype != FD_BF16 && logits->dtype != FD_FP32) return fail(FD_ERR_INVALID_ARG, "logits must be bf16 or fp32");
  if (R < 1 || R > kInt / 8 || V < 1 || V > (1 << 24))
    return fail(FD_ERR_INVALID_ARG, "logits must be [1 <= R < 2^28, 1 <= V <= 2^24]");
  if (!aligned(logits->data, logits->dtype == FD_BF16 ? 2 : 4)) return fail(FD_ERR_UNSUPPORTED, "logits are not aligned to their type");
  FD_TRY(check_tensor(tokens, "tokens", 1, false));
  if ((tokens->dtype != FD_INT32 && tokens->dtype != FD_INT64) || tokens->shape[0] != R)
    return fail(FD_ERR_INVALID_ARG, "tokens must be int32 or int64 [R=%lld]", (long long)R);
  FD_TRY(check_tensor(logprobs, "logprobs", 1));
  if (logprobs->dtype != FD_FP32 || logprobs->shape[0] != R) return fail(FD_ERR_INVALID_ARG, "logprobs must be fp32 [R=%lld]", (long long)R);
  if (given(ranks)) FD_TRY(check_ints(ranks, "ranks", R, true));
  if (given(entropy)) {
    FD_TRY(check_tensor(entropy, "entropy", 1));
    if (entropy->dtype != FD_FP32 || entropy->shape[0] != R) return fail(FD_ERR_INVALID_ARG, "entropy must be fp32 [R=%lld]", (long long)R);
  }
  int64_t K = 0;
  if (given(top_ids) != given(top_logprobs)) return fail(FD_ERR_INVALID_ARG, "top_ids and top_logprobs come together");
  if (given(top_ids)) {
    FD_TRY(check_tensor(top_ids, "top_ids", 2));
    FD_TRY(check_tensor(top_logprobs, "top_logprobs", 2));
    K = top_ids->shape[1];
    if (top_ids->dtype != FD_INT32 || top_ids->shape[0] != R || K < 1 || K > fd::kMaxTop || K > V)
      return fail(FD_ERR_INVALID_ARG, "top_ids must be int32 [R=%lld, 1 <= K <= min(%d, V)]", (long long)R, fd::kMaxTop);
    if (top_logprobs->dtype != FD_FP32 || top_logprobs->shape[0] != R || top_logprobs->shape[1] != K)
      return fail(FD_ERR_INVALID_ARG, "top_logprobs must be fp32 [R=%lld, K=%lld]", (long long)R, (long long)K);
    FD_TRY(check_distinct(top_ids, "top_ids"));
    FD_TRY(check_distinct(top_logprobs, "top_logprobs"));
  }
  FD_TRY(check_status(status));

  fd::LogprobsParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits->data;
  p.f32 = logits->dtype == FD_FP32;
  p.l_s = logits->stride[0];
  p.tokens = tokens->data;
  p.tok64 = tokens->dtype == FD_INT64;
  p.t_s = tokens->stride[0];
  p.R = static_cast<int>(R);
  p.V = static_cast<int>(V);
  p.K = static_cast<int>(K);
  p.logprobs = static_cast<float *>(logprobs->data);
  p.ranks = given(ranks) ? static_cast<int *>(ranks->data) : nullptr;
  p.entropy = given(entropy) ? static_cast<float *>(entropy->data) : nullptr;
  if (K > 0) {
    p.top_ids = static_cast<int *>(top_ids->data);
    p.top_logprobs = static_cast<float *>(top_logprobs->data);
    p.ti_s = top_ids->stride[0];
    p.tl_s = top_logprobs->stride[0];
  }
  p.status = status_word(status);
  return launched(fd::launch_token_logprobs(p, reinterpret_cast<cudaStream_t>(stream)), "log probabilities");
}

extern "C" fd_status fd_decode_sparse(const fd_tensor *q, const fd_tensor *k_cache, const fd_tensor *v_cache,
                                      const fd_tensor *kv_scales, const fd_tensor *page_table, const fd_tensor *cache_seqlens,
                                      const fd_tensor *selected, int q_per_req, float softmax_scale, fd_tensor *out,
                                      fd_tensor *lse, fd_tensor *status, fd_stream_t stream) {
  FD_TRY(check_tensor(q, "q", 4));
  Caches c;
  FD_TRY(check_caches(k_cache, v_cache, kv_scales, -1, q->shape[3], &c));
  FD_TRY(check_query(q, page_table, cache_seqlens, q_per_req, c.Hkv, c.P));
  const int64_t B = q->shape[0], Tq = q->shape[1], Hq = q->shape[2];
  FD_TRY(check_tensor(selected, "selected", 4));
  const int64_t S = selected->shape[3];
  if (selected->dtype != FD_INT32 || selected->shape[0] != B || selected->shape[1] != Tq || selected->shape[2] != c.Hkv || S < 1 ||
      S > kInt / c.P)
    return fail(FD_ERR_INVALID_ARG, "selected must be int32 [B=%lld, Tq=%lld, Hkv=%d, 1 <= S < 2^31 / P]", (long long)B,
                (long long)Tq, c.Hkv);
  if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale))
    return fail(FD_ERR_INVALID_ARG, "softmax_scale must be finite and >= 0");
  if (B * Tq * Hq > kInt / 8) return fail(FD_ERR_UNSUPPORTED, "more than 2^28 query rows");
  FD_TRY(check_tensor(out, "out", 4));
  if (out->dtype != FD_BF16 && out->dtype != FD_FP32) return fail(FD_ERR_INVALID_ARG, "out must be bf16 or fp32");
  for (int i = 0; i < 4; ++i)
    if (out->shape[i] != q->shape[i]) return fail(FD_ERR_INVALID_ARG, "out must have q's shape");
  FD_TRY(check_distinct(out, "out"));
  FD_TRY(check_rows16(out, "out", out->dtype == FD_BF16 ? 2 : 4));
  if (given(lse)) {
    FD_TRY(check_tensor(lse, "lse", 3, false));
    if (lse->dtype != FD_FP32 || lse->shape[0] != B || lse->shape[1] != Tq || lse->shape[2] != Hq)
      return fail(FD_ERR_INVALID_ARG, "lse must be fp32 [B, Tq, Hq]");
    FD_TRY(check_distinct(lse, "lse"));
  }
  FD_TRY(check_status(status));

  fd::SparseParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16 *>(q->data);
  p.q_sb = q->stride[0];
  p.q_st = q->stride[1];
  p.q_sh = q->stride[2];
  p.k_cache = static_cast<const unsigned char *>(k_cache->data);
  p.v_cache = static_cast<const unsigned char *>(v_cache->data);
  p.c_sp = k_cache->stride[0] * c.es;
  p.c_ss = k_cache->stride[1] * c.es;
  p.c_sh = k_cache->stride[2] * c.es;
  if (c.kind != fd::KV_BF16) {
    p.scales = static_cast<const float *>(kv_scales->data);
    p.sc_sk = kv_scales->stride[0];
    p.sc_sp = kv_scales->stride[1];
    p.sc_ss = kv_scales->stride[2];
    p.sc_sh = kv_scales->stride[3];
  }
  p.page_table = static_cast<const int *>(page_table->data);
  p.pt_sb = page_table->stride[0];
  p.seqlens = static_cast<const int *>(cache_seqlens->data);
  p.sl_s = cache_seqlens->stride[0];
  p.selected = static_cast<const int *>(selected->data);
  p.s_sb = selected->stride[0];
  p.s_st = selected->stride[1];
  p.s_sh = selected->stride[2];
  p.num_pages = c.num_pages;
  p.B = static_cast<int>(B);
  p.Tq = static_cast<int>(Tq);
  p.Hkv = c.Hkv;
  p.G = static_cast<int>(Hq / c.Hkv);
  p.P = c.P;
  p.log2_page = c.log2_page;
  p.W = static_cast<int>(page_table->shape[1]);
  p.S = static_cast<int>(S);
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.f / std::sqrt(static_cast<float>(c.D));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out->data;
  p.out_f32 = out->dtype == FD_FP32;
  p.o_sb = out->stride[0];
  p.o_st = out->stride[1];
  p.o_sh = out->stride[2];
  if (given(lse)) {
    p.lse = static_cast<float *>(lse->data);
    p.l_sb = lse->stride[0];
    p.l_st = lse->stride[1];
    p.l_sh = lse->stride[2];
  }
  p.status = status_word(status);
  return launched(fd::launch_decode_sparse(c.kind, c.D, p, reinterpret_cast<cudaStream_t>(stream)), "sparse decode");
}
