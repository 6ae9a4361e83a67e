// autotune.cu - num_splits selection and the startup autotuner.
//
// Follows "feat(autotune): separate general and decode attention warmup"
// (LightLLM PR 1549): decode attention is tuned only at startup, outside CUDA
// graph capture, on representative inputs built for the purpose (section
// "Changes": rebuild_input_func; representative length 32768 by default,
// section "Covered decode kernels"); KV-length run keys are bucketed while a
// call still uses its real lengths; chosen configurations are persisted per
// kernel and reused, and deleting the cache forces a new search (section
// "Changes": decode attention treats FORCE_AUTOTUNE as adaptive tuning, so
// entries already tuned are never searched again); cached nearest-key matches
// are invalidated when a new configuration is saved. The warmup phases of the
// same section (GENERAL, DECODE_ATTENTION; a nestable scope that restores the
// previous phase) decide whether a decode call may tune (autotune_on_call).
//
// Table key: (batch, bucket) with bucket a power of two of the KV length,
// stored as -bucket for the mixed-length table (see tuning_lengths).
// Lookup for a call: the nearest tuned batch (smallest >= B, else the
// largest), then the lookup bucket (exact, else the smallest larger, else the
// largest), memoised until the next save. The lookup bucket is the next power
// of two >= the host-known max length; under the balanced split policy with a
// mean-length hint it is the power of two nearest the mean instead: balanced
// splits give a mixed batch of mean m about the per-CTA work of an
// equal-length batch of length m. When the hints also show a spread (max >=
// 1.25 x mean), the mixed-length table is used: at few splits per request,
// the uneven last splits of a mixed batch leave SMs idle that an equal-length
// batch keeps busy, so the two want different counts. Without any entry a
// heuristic sizes the grid to two CTAs per SM.
#include <nvtx3/nvToolsExt.h>
#include <cuda_runtime.h>
#include <sys/stat.h>

#include <algorithm>
#include <cerrno>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>
#include <vector>

#include "fd.h"
#include "kernels.h"
#include "plan.h"

using fd::fail;

namespace {

thread_local int g_phase = FD_PHASE_NONE;  // the calling thread's warmup phase

int next_pow2(int v) {
  int r = 1;
  while (r < v && r < (1 << 30)) r <<= 1;
  return r;
}

bool is_pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

// The power of two nearest to v on a log scale (the geometric midpoint
// between p / 2 and p decides).
int nearest_pow2(int v) {
  const int p = next_pow2(v);
  return (p > 1 && 2.0 * v * v < static_cast<double>(p) * p) ? p / 2 : p;
}

int heuristic_splits(const fd_plan *pl, int batch, int max_seqlen) {
  const int G = pl->hq / pl->hkv;
  const long ctas = static_cast<long>(batch) * pl->hkv * ((G + 15) / 16);
  const long target = 2L * pl->num_sms;
  int s = 1;
  while (static_cast<long>(s) * ctas < target && s < pl->max_splits) s <<= 1;
  const int L = max_seqlen > 0 ? max_seqlen : 32768;
  while (s > 1 && L / s < 256) s >>= 1;
  return std::min(s, pl->max_splits);
}

// Candidates: powers of two up to max_splits, 3, 6 and 12, plus the split
// counts that fill one or two waves of one CTA per SM for this batch (e.g. 19 for one
// request of 8 KV heads on 152 SMs), where a power of two leaves SMs idle;
// none that cuts the bucket length into splits of fewer than 128 keys (such
// calls take microseconds, and their timing is noise).
std::vector<int> candidate_splits(const fd_plan *pl, int batch, int bucket) {
  const int cap = std::max(1, std::min(pl->max_splits, bucket / 128));
  std::vector<int> c;
  for (int S = 1; S <= cap; S <<= 1) c.push_back(S);
  for (int S = 3; S <= cap && S <= 12; S <<= 1) c.push_back(S);  // 3, 6, 12: between the powers of two
  const int G = pl->hq / pl->hkv;
  const long base = static_cast<long>(batch) * pl->hkv * ((G * pl->max_q + 15) / 16);
  for (int k = 1; k <= 2; ++k) {
    const long sw = k * static_cast<long>(pl->num_sms) / base;
    if (sw >= 2 && sw <= cap && !is_pow2(static_cast<int>(sw))) c.push_back(static_cast<int>(sw));
  }
  std::sort(c.begin(), c.end());
  c.erase(std::unique(c.begin(), c.end()), c.end());
  return c;
}

const char *kv_name(fd_dtype t) {
  return t == FD_BF16 ? "bf16" : t == FD_INT8 ? "int8" : t == FD_INT4X2 ? "int4" : "x";
}

// Request lengths of the tuning inputs for bucket K: all K, or (mixed) spread
// evenly over [K/8, 15K/8], whose mean is K.
std::vector<int> tuning_lengths(int batch, int bucket, bool mixed) {
  std::vector<int> L(batch, bucket);
  if (mixed && batch > 1)
    for (int i = 0; i < batch; ++i)
      L[i] = std::max(1, static_cast<int>(std::lround(bucket * (1.0 + 14.0 * i / (batch - 1)) / 8.0)));
  return L;
}

std::string cache_path(const fd_plan *pl) {
  return pl->cache_dir + "/fd_splits_" + fd::autotune_key(pl) + ".json";
}

// -------------------------------------------------------------- tuning inputs

// Integer mixer ("lowbias32", C. Wellons) for reproducible synthetic fills
// and the tuning inputs' page placement.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  x ^= x >> 16;
  return x;
}

__global__ void fill_bf16_kernel(__nv_bfloat16 *p, size_t n, uint32_t seed) {
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const uint32_t h = mix32(static_cast<uint32_t>(i) * 2654435761u ^ seed ^ static_cast<uint32_t>(i >> 32));
    p[i] = __float2bfloat16_rn((h >> 8) * (2.0f / 16777216.0f) - 1.0f);
  }
}

__global__ void fill_u8_kernel(uint8_t *p, size_t n, uint32_t seed) {
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<size_t>(gridDim.x) * blockDim.x)
    p[i] = static_cast<uint8_t>(mix32(static_cast<uint32_t>(i) ^ seed) >> 24);
}

__global__ void fill_f32_kernel(float *p, size_t n, float v) {
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<size_t>(gridDim.x) * blockDim.x)
    p[i] = v;
}

// Calls in one captured sequence at most (each on pages of its own).
constexpr int kMaxSeq = 64;

struct TuneBuffers {
  void *q = nullptr, *out = nullptr, *k = nullptr, *v = nullptr;
  float *lse = nullptr, *scales = nullptr;
  int *pt = nullptr, *sl = nullptr;
  long pool_pages = 0;
  int width = 0, bmax = 0, tq = 1;
  double l2_bytes = 0.0;
  cudaStream_t ts = nullptr;  // private stream: captured and replayed sequences
  ~TuneBuffers() {
    for (void *p : {q, out, k, v, static_cast<void *>(lse), static_cast<void *>(scales),
                    static_cast<void *>(pt), static_cast<void *>(sl)})
      if (p) cudaFree(p);
    if (ts) cudaStreamDestroy(ts);
  }
};

#define TRY_CUDA(x)                                                                        \
  do {                                                                                     \
    cudaError_t e_ = (x);                                                                  \
    if (e_ != cudaSuccess) return fail(FD_ERR_CUDA, "autotune: %s: %s", #x, cudaGetErrorString(e_)); \
  } while (0)

fd_status tune_alloc(fd_plan *pl, TuneBuffers &tb, int bmax, int max_bucket, cudaStream_t st) {
  int l2 = 0;
  TRY_CUDA(cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, pl->device));
  const int rowe = pl->kv_dtype == FD_INT4X2 ? pl->d / 2 : pl->d;
  const int es = pl->kv_dtype == FD_BF16 ? 2 : 1;
  const int ng = pl->kv_dtype == FD_INT4X2 ? pl->d / 32 : 1;
  const size_t page_bytes = static_cast<size_t>(pl->page) * pl->hkv * rowe * es;
  tb.bmax = bmax;
  tb.tq = pl->max_q;
  tb.width = (2 * max_bucket + pl->page - 1) / pl->page;  // room for mixed lengths up to 15/8 bucket
  // Pool: distinct pages for the largest batch's call and for a sequence of
  // eight one-request calls, at least 4x L2 of K+V, at most a quarter of the
  // free device memory (beyond that, page ids wrap around the pool).
  size_t free_b = 0, total_b = 0;
  TRY_CUDA(cudaMemGetInfo(&free_b, &total_b));
  const size_t kv_page = 2 * page_bytes + (pl->kv_dtype != FD_BF16 ? 2ull * pl->page * pl->hkv * ng * 4 : 0);
  long want = std::max(static_cast<long>(bmax), 8L) * tb.width;
  want = std::max(want, static_cast<long>(4.0 * std::max(l2, 1 << 20) / kv_page) + 1);
  const long mem_cap = static_cast<long>(free_b / 4 / kv_page);
  tb.pool_pages = std::max(1L, std::min(want, mem_cap));
  const size_t qn = static_cast<size_t>(bmax) * tb.tq * pl->hq * pl->d;
  const size_t kvn = static_cast<size_t>(tb.pool_pages) * pl->page * pl->hkv * rowe;
  TRY_CUDA(cudaMalloc(&tb.q, qn * 2));
  TRY_CUDA(cudaMalloc(&tb.out, qn * 2));
  TRY_CUDA(cudaMalloc(&tb.lse, static_cast<size_t>(bmax) * tb.tq * pl->hq * 4));
  TRY_CUDA(cudaMalloc(&tb.k, kvn * es));
  TRY_CUDA(cudaMalloc(&tb.v, kvn * es));
  if (pl->kv_dtype != FD_BF16) {
    const size_t sn = 2ull * tb.pool_pages * pl->page * pl->hkv * ng;
    TRY_CUDA(cudaMalloc(&tb.scales, sn * 4));
    fill_f32_kernel<<<1024, 256, 0, st>>>(tb.scales, sn, 0.02f);
  }
  const size_t pt_rows = static_cast<size_t>(bmax) * kMaxSeq;
  TRY_CUDA(cudaMalloc(&tb.pt, pt_rows * tb.width * 4));
  TRY_CUDA(cudaMalloc(&tb.sl, static_cast<size_t>(bmax) * 4));
  TRY_CUDA(cudaStreamCreateWithFlags(&tb.ts, cudaStreamNonBlocking));
  tb.l2_bytes = static_cast<double>(std::max(l2, 1 << 20));
  fill_bf16_kernel<<<1024, 256, 0, st>>>(static_cast<__nv_bfloat16 *>(tb.q), qn, 17u);
  if (pl->kv_dtype == FD_BF16) {
    fill_bf16_kernel<<<4096, 256, 0, st>>>(static_cast<__nv_bfloat16 *>(tb.k), kvn, 29u);
    fill_bf16_kernel<<<4096, 256, 0, st>>>(static_cast<__nv_bfloat16 *>(tb.v), kvn, 31u);
  } else {
    fill_u8_kernel<<<4096, 256, 0, st>>>(static_cast<uint8_t *>(tb.k), kvn, 29u);
    fill_u8_kernel<<<4096, 256, 0, st>>>(static_cast<uint8_t *>(tb.v), kvn, 31u);
  }
  TRY_CUDA(cudaGetLastError());
  // row r holds pages perm[r * width ...] (mod pool): rows of different calls
  // of a sequence name different pages while the pool lasts, and, as in a
  // serving engine's page pool, a request's pages lie scattered over the pool
  // (a fixed Fisher-Yates shuffle driven by the mixer above, so every tuning
  // run sees the same placement)
  std::vector<int> perm(static_cast<size_t>(tb.pool_pages));
  for (long i = 0; i < tb.pool_pages; ++i) perm[i] = static_cast<int>(i);
  for (long i = tb.pool_pages - 1; i > 0; --i) {
    const uint32_t h = mix32(static_cast<uint32_t>(i) * 2654435761u ^ 0x5bd1e995u);
    std::swap(perm[i], perm[static_cast<long>(h % static_cast<uint32_t>(i + 1))]);
  }
  std::vector<int> pt(pt_rows * tb.width);
  for (size_t r = 0; r < pt_rows; ++r)
    for (int p = 0; p < tb.width; ++p)
      pt[r * tb.width + p] = perm[(static_cast<long>(r) * tb.width + p) % tb.pool_pages];
  TRY_CUDA(cudaMemcpyAsync(tb.pt, pt.data(), pt.size() * 4, cudaMemcpyHostToDevice, st));
  TRY_CUDA(cudaStreamSynchronize(st));
  return FD_OK;
}

void make_desc(fd_tensor &t, void *data, fd_dtype dt, std::initializer_list<int64_t> shape) {
  std::memset(&t, 0, sizeof(t));
  t.data = data;
  t.dtype = dt;
  t.ndim = static_cast<int>(shape.size());
  int i = 0;
  for (int64_t s : shape) t.shape[i++] = s;
  int64_t st = 1;
  for (int k = t.ndim - 1; k >= 0; --k) {
    t.stride[k] = st;
    st *= t.shape[k];
  }
}

// The tuner's scale buffer: logical [2, N, P, Hkv, ng], stored head-major
// within a page ([2, N, Hkv, P, ng] in memory) as the workloads store them, so
// the scales of one (page, head) are contiguous.
void make_scale_desc(fd_tensor &t, void *data, int64_t pool, int page, int hkv, int ng) {
  std::memset(&t, 0, sizeof(t));
  t.data = data;
  t.dtype = FD_FP32;
  t.ndim = 5;
  const int64_t shape[5] = {2, pool, page, hkv, ng};
  const int64_t stride[5] = {pool * hkv * page * ng, static_cast<int64_t>(hkv) * page * ng, ng,
                             static_cast<int64_t>(page) * ng, 1};
  for (int i = 0; i < 5; ++i) {
    t.shape[i] = shape[i];
    t.stride[i] = stride[i];
  }
}

// Device time of one call with `S` splits in the steady state of a decode
// loop: a CUDA graph of n_seq calls, each on pages of its own, replayed back
// to back (each call's start overlaps the previous call's end). The calls of
// a sequence together read at least 4x L2 where the pool allows, so no call
// finds its pages in L2 from the previous replay. Median of five blocks of
// at least sixteen calls (candidates 2 % apart must not swap places by noise).
fd_status tune_time(fd_plan *pl, TuneBuffers &tb, int batch, int bucket, bool mixed, int S, double *ms_out) {
  const int rowe = pl->kv_dtype == FD_INT4X2 ? pl->d / 2 : pl->d;
  const int ng = pl->kv_dtype == FD_INT4X2 ? pl->d / 32 : 1;
  const long call_pages = static_cast<long>(batch) * tb.width;
  const long fit = std::max(1L, tb.pool_pages / call_pages);  // sequences with distinct pages
  const std::vector<int> sl = tuning_lengths(batch, bucket, mixed);
  double keys = 0.0;
  for (int x : sl) keys += x;
  const double call_bytes = keys * pl->hkv * rowe * (pl->kv_dtype == FD_BF16 ? 4.0 : 2.0);
  const long cold = static_cast<long>(std::ceil(4.0 * tb.l2_bytes / std::max(call_bytes, 1.0)));
  const int n_seq = static_cast<int>(std::min<long>({fit, static_cast<long>(kMaxSeq), std::max(1L, cold)}));
  const int reps = std::max(1, (16 + n_seq - 1) / n_seq);  // replays per timed block
  cudaStream_t ts = tb.ts;
  TRY_CUDA(cudaMemcpyAsync(tb.sl, sl.data(), sl.size() * 4, cudaMemcpyHostToDevice, ts));
  TRY_CUDA(cudaStreamSynchronize(ts));
  fd_tensor q, k, v, sc, sq, out, lse;
  make_desc(q, tb.q, FD_BF16, {batch, tb.tq, pl->hq, pl->d});
  make_desc(k, tb.k, pl->kv_dtype, {tb.pool_pages, pl->page, pl->hkv, rowe});
  make_desc(v, tb.v, pl->kv_dtype, {tb.pool_pages, pl->page, pl->hkv, rowe});
  make_scale_desc(sc, tb.scales, tb.pool_pages, pl->page, pl->hkv, ng);
  make_desc(sq, tb.sl, FD_INT32, {batch});
  make_desc(out, tb.out, FD_BF16, {batch, tb.tq, pl->hq, pl->d});
  make_desc(lse, tb.lse, FD_FP32, {batch, tb.tq, pl->hq});
  fd_plan *prev = fd_get_plan();
  fd_set_plan(pl);
  const bool was_profiling = pl->profiling;
  pl->profiling = false;

  fd_status s = FD_OK;
  cudaGraph_t graph = nullptr;
  cudaGraphExec_t exec = nullptr;
  cudaError_t ce = cudaStreamBeginCapture(ts, cudaStreamCaptureModeThreadLocal);
  if (ce != cudaSuccess) s = fail(FD_ERR_CUDA, "autotune: capture failed: %s", cudaGetErrorString(ce));
  for (int i = 0; i < n_seq && s == FD_OK; ++i) {
    fd_tensor pt;
    make_desc(pt, tb.pt + static_cast<size_t>(i) * call_pages, FD_INT32, {batch, tb.width});
    s = fd_decode_paged(&q, &k, &v, tb.scales ? &sc : nullptr, &pt, &sq, tb.tq, S, &out, &lse,
                        reinterpret_cast<fd_stream_t>(ts));
  }
  if (ce == cudaSuccess) {
    const cudaError_t e2 = cudaStreamEndCapture(ts, &graph);
    if (s == FD_OK && e2 != cudaSuccess)
      s = fail(FD_ERR_CUDA, "autotune: capture failed: %s", cudaGetErrorString(e2));
  }
  if (s == FD_OK && cudaGraphInstantiate(&exec, graph, 0) != cudaSuccess)
    s = fail(FD_ERR_CUDA, "autotune: graph instantiation failed");

  cudaEvent_t e0 = nullptr, e1 = nullptr;
  std::vector<float> times;
  if (s == FD_OK) {
    cudaEventCreate(&e0);
    cudaEventCreate(&e1);
    // the first replay uploads the graph and warms up
    if (cudaGraphLaunch(exec, ts) != cudaSuccess) s = fail(FD_ERR_CUDA, "autotune: graph launch failed");
  }
  for (int blk = 0; blk < 5 && s == FD_OK; ++blk) {
    cudaEventRecord(e0, ts);
    for (int r = 0; r < reps && s == FD_OK; ++r)
      if (cudaGraphLaunch(exec, ts) != cudaSuccess) s = fail(FD_ERR_CUDA, "autotune: graph launch failed");
    cudaEventRecord(e1, ts);
    if (s == FD_OK && cudaEventSynchronize(e1) != cudaSuccess) s = fail(FD_ERR_CUDA, "autotune: timing failed");
    float ms = 0.f;
    if (s == FD_OK) cudaEventElapsedTime(&ms, e0, e1);
    times.push_back(ms / (reps * n_seq));
  }
  if (e0) cudaEventDestroy(e0);
  if (e1) cudaEventDestroy(e1);
  if (exec) cudaGraphExecDestroy(exec);
  if (graph) cudaGraphDestroy(graph);
  pl->profiling = was_profiling;
  fd_set_plan(prev);
  if (s != FD_OK) return s;
  std::sort(times.begin(), times.end());
  *ms_out = times[times.size() / 2];
  return FD_OK;
}

}  // namespace

namespace fd {

std::string autotune_key(const fd_plan *pl) {
  std::string g;
  for (char c : pl->gpu_name) g += (isalnum(static_cast<unsigned char>(c)) ? c : '_');
  char buf[256];
  snprintf(buf, sizeof(buf), "%s_%dsm_%s_hq%d_hkv%d_d%d_p%d_tq%d", g.c_str(), pl->num_sms,
           kv_name(pl->kv_dtype), pl->hq, pl->hkv, pl->d, pl->page, pl->max_q);
  return buf;
}

fd_status autotune_load(fd_plan *pl) {
  pl->cache_loaded = true;
  if (pl->cache_dir.empty()) return FD_OK;
  FILE *f = fopen(cache_path(pl).c_str(), "rb");
  if (!f) return FD_OK;  // nothing cached yet
  std::string txt;
  char buf[4096];
  size_t n;
  while ((n = fread(buf, 1, sizeof(buf), f)) > 0) txt.append(buf, n);
  fclose(f);
  const size_t ent = txt.find("\"entries\"");
  if (ent == std::string::npos) return fail(FD_ERR_IO, "autotune cache %s has no entries", cache_path(pl).c_str());
  size_t pos = ent;
  auto field = [](const std::string &obj, const char *name, long *v) {
    const size_t k = obj.find(std::string("\"") + name + "\"");
    if (k == std::string::npos) return false;
    const size_t c = obj.find(':', k);
    if (c == std::string::npos) return false;
    char *end = nullptr;
    *v = strtol(obj.c_str() + c + 1, &end, 10);
    return end != obj.c_str() + c + 1;
  };
  while ((pos = txt.find('{', pos + 1)) != std::string::npos) {
    const size_t close = txt.find('}', pos);
    if (close == std::string::npos) break;
    const std::string obj = txt.substr(pos, close - pos);
    long b, k, s, spread = 0;
    if (!field(obj, "spread", &spread)) spread = 0;
    if (field(obj, "batch", &b) && field(obj, "bucket", &k) && field(obj, "num_splits", &s) && b >= 1 &&
        is_pow2(static_cast<int>(k)) && s >= 1 && s <= pl->max_splits)
      pl->table[{static_cast<int>(b), static_cast<int>(spread ? -k : k)}] = static_cast<int>(s);
    pos = close;
  }
  pl->memo.clear();
  return FD_OK;
}

fd_status autotune_save(fd_plan *pl) {
  pl->memo.clear();  // a new configuration invalidates nearest-key matches
  if (pl->cache_dir.empty()) return FD_OK;
  mkdir(pl->cache_dir.c_str(), 0755);
  const std::string path = cache_path(pl);
  const std::string tmp = path + ".tmp";
  FILE *f = fopen(tmp.c_str(), "wb");
  if (!f) return fail(FD_ERR_IO, "cannot write %s", tmp.c_str());
  fprintf(f, "{\n  \"version\": 1,\n  \"key\": \"%s\",\n  \"entries\": [", autotune_key(pl).c_str());
  bool first = true;
  for (const auto &kv : pl->table) {
    auto t = pl->table_time.find(kv.first);
    fprintf(f, "%s\n    {\"batch\": %d, \"bucket\": %d, \"spread\": %d, \"num_splits\": %d, \"time\": %.6g}",
            first ? "" : ",", kv.first.first, std::abs(kv.first.second), kv.first.second < 0 ? 1 : 0, kv.second,
            t == pl->table_time.end() ? 0.0 : t->second);
    first = false;
  }
  fprintf(f, "\n  ]\n}\n");
  if (fclose(f) != 0 || rename(tmp.c_str(), path.c_str()) != 0)
    return fail(FD_ERR_IO, "cannot write %s", path.c_str());
  return FD_OK;
}

fd_status autotune_on_call(fd_plan *pl, int batch, cudaStream_t stream) {
  if (g_phase != FD_PHASE_DECODE_ATTENTION) return FD_OK;  // only decode attention tunes, only in its phase
  if (!pl->timer) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) return fail(FD_ERR_CUDA, "cudaStreamIsCapturing failed");
    if (cs != cudaStreamCaptureStatusNone) return FD_OK;  // never inside capture: look the table up
  }
  if (!pl->cache_loaded) autotune_load(pl);
  int len = 32768;  // the representative KV length
  if (const char *e = std::getenv("FD_AUTOTUNE_SEQ_LEN")) {
    const int v = atoi(e);
    if (v > 0) len = v;
  }
  const int bucket = next_pow2(len);
  if (pl->table.count({batch, bucket})) return FD_OK;
  return fd_autotune(pl, &batch, 1, bucket, bucket, reinterpret_cast<fd_stream_t>(stream));
}

int choose_splits(fd_plan *pl, int batch, int max_seqlen) {
  const bool by_mean = pl->split_policy == FD_SPLIT_BALANCED && pl->mean_hint > 0;
  if (pl->table.empty()) return heuristic_splits(pl, batch, by_mean ? pl->mean_hint : max_seqlen);
  const int bucket_q = by_mean ? nearest_pow2(pl->mean_hint) : (max_seqlen > 0 ? next_pow2(max_seqlen) : 0);
  bool mixed = by_mean && batch > 1 && 4LL * max_seqlen >= 5LL * pl->mean_hint;
  const int memo_key = mixed ? -bucket_q : bucket_q;
  auto m = pl->memo.find({batch, memo_key});
  if (m != pl->memo.end()) return m->second;
  std::set<int> batches;
  for (const auto &kv : pl->table)
    if ((kv.first.second < 0) == mixed) batches.insert(kv.first.first);
  if (batches.empty()) {  // no mixed-length entries: the equal-length table
    mixed = false;
    for (const auto &kv : pl->table)
      if (kv.first.second > 0) batches.insert(kv.first.first);
  }
  auto bi = batches.lower_bound(batch);
  const int tb = bi != batches.end() ? *bi : *batches.rbegin();
  std::set<int> buckets;  // absolute buckets of the chosen table
  for (const auto &kv : pl->table)
    if (kv.first.first == tb && (kv.first.second < 0) == mixed) buckets.insert(std::abs(kv.first.second));
  int kb;
  if (bucket_q == 0) {
    kb = *buckets.rbegin();
  } else {
    auto ki = buckets.lower_bound(bucket_q);
    kb = ki != buckets.end() ? *ki : *buckets.rbegin();
  }
  const int S = std::min(pl->table[{tb, mixed ? -kb : kb}], pl->max_splits);
  pl->memo[{batch, memo_key}] = S;
  return S;
}

}  // namespace fd

extern "C" {

fd_status fd_query_splits(fd_plan *plan, int batch, int max_seqlen, int *num_splits) {
  if (!plan || !num_splits) return fail(FD_ERR_INVALID_ARG, "NULL argument");
  if (plan->latent) return fail(FD_ERR_UNSUPPORTED, "a latent plan has no tuning table");
  if (batch < 1) return fail(FD_ERR_INVALID_ARG, "batch %d < 1", batch);
  if (max_seqlen < 0) return fail(FD_ERR_INVALID_ARG, "max_seqlen %d < 0", max_seqlen);
  if (!plan->cache_loaded) fd::autotune_load(plan);
  *num_splits = fd::choose_splits(plan, batch, max_seqlen);
  return FD_OK;
}

fd_status fd_autotune_set_timer(fd_plan *plan, fd_timer_fn fn, void *user) {
  if (!plan) return fail(FD_ERR_INVALID_ARG, "plan is NULL");
  if (plan->latent) return fail(FD_ERR_UNSUPPORTED, "a latent plan has no tuning table");
  plan->timer = fn;
  plan->timer_user = user;
  return FD_OK;
}

fd_status fd_autotune_set_input_hook(fd_plan *plan, fd_tune_inputs_fn fn, void *user) {
  if (!plan) return fail(FD_ERR_INVALID_ARG, "plan is NULL");
  if (plan->latent) return fail(FD_ERR_UNSUPPORTED, "a latent plan has no tuning table");
  plan->input_hook = fn;
  plan->input_user = user;
  return FD_OK;
}

fd_status fd_autotune_clear(fd_plan *plan, int remove_file) {
  if (!plan) return fail(FD_ERR_INVALID_ARG, "plan is NULL");
  if (plan->latent) return fail(FD_ERR_UNSUPPORTED, "a latent plan has no tuning table");
  plan->table.clear();
  plan->table_time.clear();
  plan->memo.clear();
  plan->cache_loaded = true;  // do not reload the file being discarded
  if (remove_file && !plan->cache_dir.empty()) {
    if (std::remove(cache_path(plan).c_str()) != 0 && errno != ENOENT)
      return fail(FD_ERR_IO, "cannot remove %s", cache_path(plan).c_str());
  }
  return FD_OK;
}

fd_status fd_warmup_enter(int phase, int *previous) {
  if (phase != FD_PHASE_NONE && phase != FD_PHASE_GENERAL && phase != FD_PHASE_DECODE_ATTENTION)
    return fail(FD_ERR_INVALID_ARG, "warmup phase %d unknown", phase);
  if (previous) *previous = g_phase;
  g_phase = phase;
  return FD_OK;
}

fd_status fd_warmup_exit(int previous) {
  if (previous != FD_PHASE_NONE && previous != FD_PHASE_GENERAL && previous != FD_PHASE_DECODE_ATTENTION)
    return fail(FD_ERR_INVALID_ARG, "warmup phase %d unknown", previous);
  g_phase = previous;
  return FD_OK;
}

int fd_warmup_current(void) { return g_phase; }

fd_status fd_autotune_set_cache_dir(fd_plan *plan, const char *dir) {
  if (!plan) return fail(FD_ERR_INVALID_ARG, "plan is NULL");
  if (plan->latent) return fail(FD_ERR_UNSUPPORTED, "a latent plan has no tuning table");
  plan->cache_dir = dir ? dir : "";
  return fd::autotune_load(plan);
}

fd_status fd_autotune_stats(fd_plan *plan, int *searches, int *cache_hits) {
  if (!plan) return fail(FD_ERR_INVALID_ARG, "plan is NULL");
  if (plan->latent) return fail(FD_ERR_UNSUPPORTED, "a latent plan has no tuning table");
  if (searches) *searches = plan->searches;
  if (cache_hits) *cache_hits = plan->cache_hits;
  return FD_OK;
}

fd_status fd_autotune(fd_plan *plan, const int *batch_sizes, int n_batch, int min_bucket, int max_bucket,
                      fd_stream_t stream) {
  if (!plan) return fail(FD_ERR_INVALID_ARG, "plan is NULL");
  if (plan->latent) return fail(FD_ERR_UNSUPPORTED, "a latent plan has no tuning table");
  if (!batch_sizes || n_batch < 1) return fail(FD_ERR_INVALID_ARG, "no batch sizes");
  for (int i = 0; i < n_batch; ++i)
    if (batch_sizes[i] < 1 || batch_sizes[i] > plan->max_batch)
      return fail(FD_ERR_INVALID_ARG, "batch size %d not in [1, %d]", batch_sizes[i], plan->max_batch);
  if (min_bucket == 0) min_bucket = 1024;
  if (max_bucket == 0) {
    max_bucket = 32768;
    if (const char *e = std::getenv("FD_AUTOTUNE_SEQ_LEN")) {
      const int v = atoi(e);
      if (v > 0) max_bucket = next_pow2(v);
    }
  }
  if (!is_pow2(min_bucket) || !is_pow2(max_bucket) || min_bucket > max_bucket)
    return fail(FD_ERR_INVALID_ARG, "buckets must be powers of two with min <= max");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!plan->timer) {
    if (plan->device < 0) return fail(FD_ERR_WORKSPACE, "host-only plan cannot time kernels");
    fd::DeviceGuard guard(plan->device);
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &cs) != cudaSuccess)
      return fail(FD_ERR_CUDA, "cudaStreamIsCapturing failed");
    if (cs != cudaStreamCaptureStatusNone)
      return fail(FD_ERR_CAPTURING, "autotuning cannot run inside CUDA graph capture");
  }
  if (!plan->cache_loaded) {
    fd_status s = fd::autotune_load(plan);
    if (s != FD_OK) return s;
  }

  // keys (batch, bucket) for equal lengths and (batch, -bucket) for mixed
  // lengths (batches of two or more requests)
  std::vector<std::pair<int, int>> todo;
  for (int i = 0; i < n_batch; ++i)
    for (int k = min_bucket; k <= max_bucket; k <<= 1)
      for (int sign : {1, -1}) {
        if (sign < 0 && batch_sizes[i] < 2) continue;
        const std::pair<int, int> key{batch_sizes[i], sign * k};
        if (plan->table.count(key)) {
          ++plan->cache_hits;
          continue;
        }
        if (std::find(todo.begin(), todo.end(), key) == todo.end()) todo.push_back(key);
      }
  if (todo.empty()) return FD_OK;

  fd::DeviceGuard guard(plan->device);
  TuneBuffers tb;
  if (!plan->timer) {
    int bmax = 0;
    for (auto &k : todo) bmax = std::max(bmax, k.first);
    fd_status s = tune_alloc(plan, tb, bmax, max_bucket, st);
    if (s != FD_OK) return s;
  }
  // NVTX range over the search, one nested range per key (visible to nsys / ncu)
  nvtxRangePushA("fd_autotune");
  struct PopRange {
    ~PopRange() { nvtxRangePop(); }
  } pop_outer;
  for (auto &key : todo) {
    ++plan->searches;
    char label[64];
    std::snprintf(label, sizeof(label), "fd_autotune B=%d K=%d%s", key.first, std::abs(key.second),
                  key.second < 0 ? " mixed" : "");
    nvtxRangePushA(label);
    PopRange pop_key;
    if (!plan->timer && plan->input_hook) {  // representative inputs from the caller
      const int rowe = plan->kv_dtype == FD_INT4X2 ? plan->d / 2 : plan->d;
      const int ng = plan->kv_dtype == FD_INT4X2 ? plan->d / 32 : 1;
      fd_tensor q, k, v, sc;
      make_desc(q, tb.q, FD_BF16, {key.first, tb.tq, plan->hq, plan->d});
      make_desc(k, tb.k, plan->kv_dtype, {tb.pool_pages, plan->page, plan->hkv, rowe});
      make_desc(v, tb.v, plan->kv_dtype, {tb.pool_pages, plan->page, plan->hkv, rowe});
      make_scale_desc(sc, tb.scales, tb.pool_pages, plan->page, plan->hkv, ng);
      fd_status hs = plan->input_hook(plan->input_user, key.first, std::abs(key.second), key.second < 0 ? 1 : 0, &q,
                                      &k, &v, tb.scales ? &sc : nullptr, reinterpret_cast<fd_stream_t>(st));
      if (hs != FD_OK) return fail(hs, "autotune: the input hook returned %d", (int)hs);
      if (cudaStreamSynchronize(st) != cudaSuccess) return fail(FD_ERR_CUDA, "autotune: input hook work failed");
    }
    std::vector<std::pair<int, double>> timed;
    for (int S : candidate_splits(plan, key.first, std::abs(key.second))) {
      double t = 0.0;
      if (plan->timer) {
        t = plan->timer(plan->timer_user, key.first, key.second, S);
      } else {
        fd_status s = tune_time(plan, tb, key.first, std::abs(key.second), key.second < 0, S, &t);
        if (s != FD_OK) return s;
      }
      timed.emplace_back(S, t);
    }
    // the fastest; on an exact tie, the fewer splits
    int best = timed[0].first;
    double best_t = timed[0].second;
    for (auto &c : timed)
      if (c.second < best_t) {
        best = c.first;
        best_t = c.second;
      }
    plan->table[key] = best;
    plan->table_time[key] = best_t;
  }
  return fd::autotune_save(plan);
}

}  // extern "C"
