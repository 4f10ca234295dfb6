// C ABI of linear attention: argument validation and dispatch.  Declared in include/path_attn.h.
#include "linear.h"

#include <math.h>

using namespace pathattn;

namespace {

bool aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? PATH_OK : PATH_ERR_CUDA; }

int check_heads(int heads_q, int heads, int head_dim, int dtype, float scale) {
  if (heads <= 0 || heads_q <= 0 || heads_q % heads != 0 || head_dim <= 0 || !isfinite(scale)) return PATH_ERR_INVALID_ARG;
  if (dtype != PATH_BF16 && dtype != PATH_FP32) return PATH_ERR_INVALID_ARG;
  if (head_dim != kHeadDim && head_dim != kHeadDimWide) return PATH_ERR_UNSUPPORTED;
  if (heads > 1024 || heads_q / heads > kPagedMaxGroup) return PATH_ERR_UNSUPPORTED;
  return PATH_OK;
}
int check_desc(const path_linear_desc_t* d) {
  if (!d || d->batch <= 0 || d->seqlen <= 0) return PATH_ERR_INVALID_ARG;
  const int rc = check_heads(d->heads_q, d->heads, d->head_dim, d->dtype, d->scale);
  if (rc != PATH_OK) return rc;
  // sequences are a grid dimension, rows of a tensor are numbered in 32 bits
  if (d->batch > 65535 || (long long)d->batch * d->heads_q * d->seqlen > 0x7fffffffLL) return PATH_ERR_UNSUPPORTED;
  return PATH_OK;
}
int check_cache(const path_linear_cache_t* c) {
  if (!c || c->slots <= 0) return PATH_ERR_INVALID_ARG;
  return c->slots > 65535 ? PATH_ERR_UNSUPPORTED : check_heads(c->heads, c->heads, c->head_dim, c->dtype, 1.f);
}
int check_cache_memory(const path_linear_cache_t* c) {
  const int rc = check_cache(c);
  if (rc != PATH_OK) return rc;
  return aligned(c->state, 16) && aligned(c->status, 4) ? PATH_OK : PATH_ERR_INVALID_ARG;
}
int check_step(const path_linear_cache_t* c, const path_linear_step_t* s) {
  if (!s || s->total_tokens < 0 || s->max_new < 0) return PATH_ERR_INVALID_ARG;
  const int rc = check_heads(s->heads_q, c->heads, c->head_dim, c->dtype, s->scale);
  if (rc != PATH_OK) return rc;
  return s->total_tokens > (1 << 22) || (long long)s->total_tokens * s->heads_q > 0x7fffffffLL / 64 ? PATH_ERR_UNSUPPORTED : PATH_OK;
}

LinArgs dense_args(const path_linear_desc_t* d, int ops) {
  LinArgs p{};
  p.ops = ops;
  p.slots = ops == 1 ? 1 : 2;
  p.D = d->head_dim;
  p.heads = d->heads;
  p.G = d->heads_q / d->heads;
  p.seqs = d->batch;
  p.L = d->seqlen;
  p.scale = d->scale;
  lin_plan(p, d->dtype == PATH_BF16);
  return p;
}
// o = walk of x over y and z; queries: x and o have the query heads (else y and z have them).
LinOp dense_op(const path_linear_desc_t* d, const void* x, const void* y, const void* z, void* o, bool queries, bool reverse) {
  const int G = d->heads_q / d->heads;
  const long long t = d->head_dim, h = t * d->seqlen;
  const long long wide = h * d->heads_q, narrow = h * d->heads;
  return LinOp{x, y, z, o, queries ? G : 1, queries ? 1 : G, reverse, t, h, queries ? wide : narrow, t, h, queries ? narrow : wide};
}
LinArgs packed_args(const path_linear_cache_t* c, const path_linear_step_t* s) {
  LinArgs p{};
  p.ops = p.slots = 1;
  p.D = c->head_dim;
  p.heads = c->heads;
  p.G = s->heads_q / c->heads;
  p.seqs = c->slots;
  p.packed = 1;
  p.total = s->total_tokens;
  p.max_new = s->max_new < s->total_tokens ? s->max_new : s->total_tokens;
  p.min_new = kLinTokenMax + 1;
  p.scale = s->scale;
  p.state = c->state;
  p.update = s->update != 0;
  if (p.max_new > kLinTokenMax) lin_plan(p, c->dtype == PATH_BF16);
  return p;
}
size_t packed_ws(const LinArgs& p) { return p.max_new > kLinTokenMax ? lin_ws_bytes(p) : 256; }

}  // namespace

#define PATH_API __attribute__((visibility("default")))
extern "C" {

PATH_API size_t path_linear_workspace_size(const path_linear_desc_t* desc, int for_backward) {
  return check_desc(desc) == PATH_OK ? lin_ws_bytes(dense_args(desc, for_backward ? 3 : 1)) : 0;
}

PATH_API int path_linear_fwd(const path_linear_desc_t* desc, const void* q, const void* k, const void* v, const float* log_decay,
                             void* o, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_desc(desc);
  if (rc != PATH_OK) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(log_decay, 4) || !aligned(o, 16) || !aligned(ws, 256))
    return PATH_ERR_INVALID_ARG;
  LinArgs p = dense_args(desc, 1);
  if (ws_bytes < lin_ws_bytes(p)) return PATH_ERR_WORKSPACE;
  p.log_decay = log_decay;
  p.err = (int*)ws;
  p.stall_ns = debug_stall_ns();
  p.op[0] = dense_op(desc, q, k, v, o, true, false);
  return cuda_status(launch_linear(p, desc->dtype == PATH_BF16, (char*)ws, (cudaStream_t)stream));
}

PATH_API int path_linear_bwd(const path_linear_desc_t* desc, const void* q, const void* k, const void* v, const float* log_decay,
                             const void* dO, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_desc(desc);
  if (rc != PATH_OK) return rc;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(log_decay, 4) || !aligned(dO, 16) || !aligned(ws, 256) ||
      (!dq && !dk && !dv) || (dq && !aligned(dq, 16)) || (dk && !aligned(dk, 16)) || (dv && !aligned(dv, 16)))
    return PATH_ERR_INVALID_ARG;
  LinArgs p = dense_args(desc, 3);
  if (ws_bytes < lin_ws_bytes(p)) return PATH_ERR_WORKSPACE;
  p.log_decay = log_decay;
  p.err = (int*)ws;
  p.stall_ns = debug_stall_ns();
  p.ops = p.slots = 0;
  if (dq) {
    p.maker[p.slots++] = p.ops;
    p.op[p.ops++] = dense_op(desc, dO, v, k, dq, true, false);
  }
  if (dk || dv) {  // sums of q dO^T over later tokens are dv's states, their transposes dk's
    const int slot = p.slots++;
    p.maker[slot] = p.ops;
    if (dv) p.op[p.ops++] = dense_op(desc, k, q, dO, dv, false, true);
    if (dk) p.op[p.ops++] = dense_op(desc, v, dO, q, dk, false, true);
    for (int i = p.maker[slot]; i < p.ops; ++i) {
      p.op[i].slot = slot;
      p.op[i].turned = i > p.maker[slot];
    }
  }
  return cuda_status(launch_linear(p, desc->dtype == PATH_BF16, (char*)ws, (cudaStream_t)stream));
}

PATH_API int path_linear_workspace_status(const path_linear_desc_t* desc, const void* ws, size_t ws_bytes, int* code, void* stream) {
  const int rc = check_desc(desc);
  if (rc != PATH_OK) return rc;
  if (!aligned(ws, 256)) return PATH_ERR_INVALID_ARG;
  if (ws_bytes < 256) return PATH_ERR_WORKSPACE;
  int h = 0;
  if (code) *code = 0;
  if (desc->dtype != PATH_BF16) return cuda_status(cudaStreamSynchronize((cudaStream_t)stream));  // no kernel that waits
  if (cudaMemcpyAsync(&h, ws, sizeof(int), cudaMemcpyDeviceToHost, (cudaStream_t)stream) != cudaSuccess ||
      cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess)
    return PATH_ERR_CUDA;
  if (code) *code = h;
  return h == 0 ? PATH_OK : PATH_ERR_INTERNAL;
}

PATH_API size_t path_linear_extend_workspace_size(const path_linear_cache_t* cache, const path_linear_step_t* step) {
  if (check_cache(cache) != PATH_OK || check_step(cache, step) != PATH_OK) return 0;
  return packed_ws(packed_args(cache, step));
}

PATH_API int path_linear_extend(const path_linear_cache_t* cache, const path_linear_step_t* step, const int* q_start, const void* q,
                                const void* k, const void* v, const float* log_decay, void* o, void* ws, size_t ws_bytes,
                                void* stream) {
  int rc = check_cache_memory(cache);
  if (rc == PATH_OK) rc = check_step(cache, step);
  if (rc != PATH_OK) return rc;
  if (q_start ? !aligned(q_start, 4) : step->total_tokens != cache->slots || step->max_new < 1) return PATH_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(log_decay, 4) || !aligned(o, 16)) return PATH_ERR_INVALID_ARG;
  LinArgs p = packed_args(cache, step);
  if (p.max_new > kLinTokenMax) {
    if (!aligned(ws, 256)) return PATH_ERR_INVALID_ARG;
    if (ws_bytes < packed_ws(p)) return PATH_ERR_WORKSPACE;
  }
  if (step->total_tokens == 0 || step->max_new == 0) return PATH_OK;
  const long long d = cache->head_dim, tq = d * step->heads_q, tk = d * cache->heads;
  p.q_start = q_start;
  p.log_decay = log_decay;
  p.err = (int*)ws;
  p.stall_ns = debug_stall_ns();
  p.status = cache->status;
  p.op[0] = LinOp{q, k, v, o, p.G, 1, 0, tq, d, 0, tk, d, 0};
  const bool bf16 = cache->dtype == PATH_BF16;
  cudaError_t e = launch_linear_token(p, bf16, (cudaStream_t)stream);
  if (e == cudaSuccess && p.max_new > kLinTokenMax && q_start) e = launch_linear(p, bf16, (char*)ws, (cudaStream_t)stream);
  return cuda_status(e);
}

PATH_API int path_linear_fork(const path_linear_cache_t* cache, const int* parents, const int* children, int count, void* stream) {
  const int rc = check_cache_memory(cache);
  if (rc != PATH_OK) return rc;
  if (count < 0 || count > cache->slots || !aligned(children, 4) || (parents && !aligned(parents, 4))) return PATH_ERR_INVALID_ARG;
  if (count == 0) return PATH_OK;
  return cuda_status(launch_linear_copy(cache->state, cache->status, cache->slots, (size_t)cache->heads * cache->head_dim * cache->head_dim,
                                        parents, children, count, (cudaStream_t)stream));
}

PATH_API int path_linear_status(const path_linear_cache_t* cache, int* code, void* stream) {
  const int rc = check_cache_memory(cache);
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
  return h >= PATH_PAGED_WAIT ? PATH_ERR_INTERNAL : PATH_ERR_INVALID_ARG;
}

}  // extern "C"
