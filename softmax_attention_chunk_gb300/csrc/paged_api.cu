// C ABI of paged serving: argument validation and dispatch.  Declared in include/path_attn.h.
#include "paged.h"

#include <math.h>

using namespace pathattn;

namespace {

bool aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_cache_sizes(const path_paged_cache_t* c) {
  if (!c) return PATH_ERR_INVALID_ARG;
  if (c->slots <= 0 || c->heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->table_width <= 0 || c->k_pages <= 0 ||
      c->v_pages <= 0)
    return PATH_ERR_INVALID_ARG;
  if (c->cache_dtype != PATH_BF16 && c->cache_dtype != PATH_FP32) return PATH_ERR_INVALID_ARG;
  if (c->head_dim != kHeadDim && c->head_dim != kHeadDimWide) return PATH_ERR_UNSUPPORTED;
  const int P = c->page_size;
  if (P != 16 && P != 32 && P != 64 && P != 128 && P != 256) return PATH_ERR_UNSUPPORTED;
  if (c->slots > 65535 || c->heads > 1024) return PATH_ERR_UNSUPPORTED;
  // positions, tile numbers of a call and row numbers of a pool are 32-bit
  if ((long long)c->table_width * P > (1LL << 30) || (long long)c->slots * c->table_width > (1LL << 26))
    return PATH_ERR_UNSUPPORTED;
  const long long pages = c->k_pages > c->v_pages ? c->k_pages : c->v_pages;
  if (pages * c->heads * P > 0x7fffffffLL) return PATH_ERR_UNSUPPORTED;
  return PATH_OK;
}
int check_cache(const path_paged_cache_t* c) {
  const int rc = check_cache_sizes(c);
  if (rc != PATH_OK) return rc;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || (c->a_pool && !aligned(c->a_pool, 16))) return PATH_ERR_INVALID_ARG;
  if (!aligned(c->k_table, 4) || !aligned(c->v_table, 4) || !aligned(c->seq_len, 4) || !aligned(c->k_ref, 4) ||
      !aligned(c->v_ref, 4) || !aligned(c->status, 4) || (c->extended && !aligned(c->extended, 4)) ||
      (c->a_rest && !aligned(c->a_rest, 16)))
    return PATH_ERR_INVALID_ARG;
  return PATH_OK;
}
int check_paged_desc(const path_paged_cache_t* c, const path_paged_desc_t* d) {
  if (!d) return PATH_ERR_INVALID_ARG;
  if (d->heads_q <= 0 || d->total_tokens < 0 || d->max_new < 0 || d->window < 0 || d->sinks < 0 || d->max_multi < 0 || !isfinite(d->scale))
    return PATH_ERR_INVALID_ARG;
  if (d->heads_q % c->heads != 0) return PATH_ERR_INVALID_ARG;
  if (d->heads_q / c->heads > kPagedMaxGroup) return PATH_ERR_UNSUPPORTED;
  if (d->total_tokens > (1 << 22) || (long long)d->total_tokens * d->heads_q > 0x7fffffffLL / 64) return PATH_ERR_UNSUPPORTED;
  return PATH_OK;
}
PagedArgs paged_args(const path_paged_cache_t* c, const path_paged_desc_t* d) {
  PagedArgs p{};
  p.c = *c;
  p.hq = d->heads_q;
  p.G = d->heads_q / c->heads;
  p.total = d->total_tokens;
  p.max_new = d->max_new < d->total_tokens ? d->max_new : d->total_tokens;
  p.window = d->window;
  p.sinks = d->sinks;
  p.multi = d->max_multi;
  p.scl = d->scale * kLog2e;
  return p;
}
int cuda_status(cudaError_t e) { return e == cudaSuccess ? PATH_OK : PATH_ERR_CUDA; }

// The checks that the page calls share.
int check_pages_call(const path_paged_cache_t* c, const void* ws, size_t ws_bytes) {
  const int rc = check_cache(c);
  if (rc != PATH_OK) return rc;
  if (!aligned(ws, 256)) return PATH_ERR_INVALID_ARG;
  return ws_bytes < pages_ws_bytes(*c) ? PATH_ERR_WORKSPACE : PATH_OK;
}

}  // namespace

#define PATH_API __attribute__((visibility("default")))
extern "C" {

PATH_API size_t path_paged_workspace_size(const path_paged_cache_t* cache, const path_paged_desc_t* desc) {
  if (check_cache_sizes(cache) != PATH_OK || check_paged_desc(cache, desc) != PATH_OK) return 0;
  return paged_ws_bytes(paged_args(cache, desc));
}

PATH_API int path_paged_extend(const path_paged_cache_t* cache, const path_paged_desc_t* desc, const int* q_start,
                               const void* q, const void* k, const void* v, const void* w, const float* beta,
                               const float* log_f, void* o, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc == PATH_OK) rc = check_paged_desc(cache, desc);
  if (rc != PATH_OK) return rc;
  if ((log_f == nullptr) != (cache->a_pool == nullptr)) return PATH_ERR_INVALID_ARG;
  if (q_start ? !aligned(q_start, 4) : desc->total_tokens != cache->slots) return PATH_ERR_INVALID_ARG;
  if (!q_start && desc->max_new < 1) return PATH_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(w, 16) || !aligned(beta, 16) || !aligned(o, 16) ||
      (log_f && !aligned(log_f, 16)))
    return PATH_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return PATH_ERR_INVALID_ARG;
  PagedArgs p = paged_args(cache, desc);
  if (ws_bytes < paged_ws_bytes(p)) return PATH_ERR_WORKSPACE;
  if (desc->total_tokens == 0 || desc->max_new == 0) return PATH_OK;
  p.q_start = q_start;
  p.q = q;
  p.k = k;
  p.v = v;
  p.w = w;
  p.beta = beta;
  p.log_f = log_f;
  p.o = o;
  return cuda_status(launch_paged(p, (char*)ws, (cudaStream_t)stream));
}

PATH_API int path_paged_advance(const path_paged_cache_t* cache, const int* q_start, void* stream) {
  const int rc = check_cache(cache);
  if (rc != PATH_OK) return rc;
  if (q_start && !aligned(q_start, 4)) return PATH_ERR_INVALID_ARG;
  return cuda_status(launch_paged_advance(*cache, q_start, (cudaStream_t)stream));
}

PATH_API int path_paged_status(const path_paged_cache_t* cache, int* code, void* stream) {
  const int rc = check_cache(cache);
  if (rc != PATH_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  int h = 0;
  if (code) *code = 0;
  if (cudaMemcpyAsync(&h, cache->status, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return PATH_ERR_CUDA;
  if (code) *code = h;
  if (h == 0) return PATH_OK;
  if (cudaMemsetAsync(cache->status, 0, sizeof(int), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
    return PATH_ERR_CUDA;
  if (h >= PATH_PAGED_WAIT) return PATH_ERR_INTERNAL;
  return h == PATH_PAGED_CAPACITY || h == PATH_PAGED_NO_PAGES ? PATH_ERR_CAPACITY : PATH_ERR_INVALID_ARG;
}

PATH_API size_t path_pages_workspace_size(const path_paged_cache_t* cache) {
  return check_cache_sizes(cache) == PATH_OK ? pages_ws_bytes(*cache) : 0;
}

PATH_API int path_pages_reserve(const path_paged_cache_t* cache, const int* n_new, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_pages_call(cache, ws, ws_bytes);
  if (rc != PATH_OK) return rc;
  if (n_new && !aligned(n_new, 4)) return PATH_ERR_INVALID_ARG;
  return cuda_status(launch_pages_reserve(*cache, n_new, (char*)ws, (cudaStream_t)stream));
}

PATH_API int path_pages_plan(const path_paged_cache_t* cache, const int* n_new, const int* from_start, int tokens, int* q_start,
                             int* slot, int* position, int* k_row, int* v_row, int* source, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_pages_call(cache, ws, ws_bytes);
  if (rc != PATH_OK) return rc;
  if (tokens < 0 || (n_new && !aligned(n_new, 4)) || !aligned(q_start, 4)) return PATH_ERR_INVALID_ARG;
  if (from_start && !aligned(from_start, 4)) return PATH_ERR_INVALID_ARG;
  if (tokens > 0 && ((from_start == nullptr) != (source == nullptr) || !aligned(slot, 4) || !aligned(position, 4) || !aligned(k_row, 4) || !aligned(v_row, 4) || (source && !aligned(source, 4))))
    return PATH_ERR_INVALID_ARG;
  if (tokens > (1 << 22)) return PATH_ERR_UNSUPPORTED;
  return cuda_status(launch_pages_plan(*cache, n_new, from_start, tokens, q_start, slot, position, k_row, v_row, source, (char*)ws,
                                       (cudaStream_t)stream));
}

PATH_API int path_pages_fork(const path_paged_cache_t* cache, const int* parents, const int* children, int count, void* ws,
                             size_t ws_bytes, void* stream) {
  const int rc = check_pages_call(cache, ws, ws_bytes);
  if (rc != PATH_OK) return rc;
  if (count < 0 || count > cache->slots || !aligned(parents, 4) || !aligned(children, 4)) return PATH_ERR_INVALID_ARG;
  if (count == 0) return PATH_OK;
  return cuda_status(launch_pages_fork(*cache, parents, children, count, (char*)ws, (cudaStream_t)stream));
}

PATH_API int path_pages_free(const path_paged_cache_t* cache, const int* slots, int count, void* ws, size_t ws_bytes,
                             void* stream) {
  const int rc = check_pages_call(cache, ws, ws_bytes);
  if (rc != PATH_OK) return rc;
  if (count < 0 || count > cache->slots || !aligned(slots, 4)) return PATH_ERR_INVALID_ARG;
  if (count == 0) return PATH_OK;
  return cuda_status(launch_pages_free(*cache, slots, count, (char*)ws, (cudaStream_t)stream));
}

PATH_API int path_pages_trim(const path_paged_cache_t* cache, int window, int sinks, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_pages_call(cache, ws, ws_bytes);
  if (rc != PATH_OK) return rc;
  if (window <= 0 || sinks < 0) return PATH_ERR_INVALID_ARG;
  return cuda_status(launch_pages_trim(*cache, window, sinks, (char*)ws, (cudaStream_t)stream));
}

PATH_API int path_pages_compact(const path_paged_cache_t* cache, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_pages_call(cache, ws, ws_bytes);
  if (rc != PATH_OK) return rc;
  return cuda_status(launch_pages_compact(*cache, (char*)ws, (cudaStream_t)stream));
}

}  // extern "C"
