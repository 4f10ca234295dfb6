// Paged serving: declarations shared by its translation units (not part of the ABI).
#pragma once

#include "../../include/path_attn.h"
#include "internal.h"

namespace pathattn {

constexpr int kPagedMaxGroup = 16;   // query heads per key head
constexpr int kPagedChunk = 32;      // new tokens per UT chunk of the CUDA-core kernels

// Slots with several new tokens go through the chunk kernels in rounds of as many slots as this workspace holds (one at
// least).  A call's host side knows neither which slots these are nor, unless it is told, how many: up to half as many as
// there are new tokens, and each may end in a partly filled chunk, block and query pair.  So a workspace for all of them at
// once grows with the slots of the cache (2 tokens of a slot, 8 key and 32 query heads of dim 128: 9 MB; 512 tokens beside 1023
// single ones 9 GiB).  A round more costs its launches and a tail (1024 prompts of 30 tokens, those heads: 5.06 ms in one round,
// 5.55 in three, 6.16 in five of 2 GiB).
constexpr size_t kRoundBytes = size_t(4) << 30;

// What a kernel of path_paged_extend needs of the call, by value.
struct PagedArgs {
  path_paged_cache_t c;
  int hq, G;            // query heads; query heads per key head
  int total, max_new;
  int window, sinks;
  float scl;            // scale * log2(e)
  const int* q_start;   // or null: one token per slot
  const void *q, *k, *v, *w;
  const float *beta, *log_f;
  void* o;
  int min_new;          // more tokens: slots with fewer new ones are left to the streaming kernels
  int multi;            // slots with several new tokens that the caller allows, 0: any number
  int skip;             // prompt chunks: new tokens of each slot that earlier passes have done
};

#ifdef __CUDACC__
#define PATH_HD __host__ __device__ inline
#else
#define PATH_HD inline
#endif

// The most slots with several new tokens that a call may have, and of these those that a round takes: bytes(n) is the
// workspace for n of them.
inline int most_multi(const PagedArgs& p) {
  int n = p.total / 2 < p.c.slots ? p.total / 2 : p.c.slots;
  if (p.multi > 0 && p.multi < n) n = p.multi;
  return n < 1 ? 1 : n;
}
template <typename F>
int round_slots(int most, F bytes) {
  if (bytes(most) <= kRoundBytes) return most;
  int lo = 1, hi = most;  // lo: fits, or is one
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (bytes(mid) <= kRoundBytes) lo = mid; else hi = mid;
  }
  const int rounds = (most + lo - 1) / lo;
  return (most + rounds - 1) / rounds;  // (rounds of like size)
}
// Bytes asked for: those of a round, and with several rounds no less than smaller calls in one round ask for.
inline size_t round_bytes(size_t bytes, bool rounds) { return rounds && bytes < kRoundBytes ? kRoundBytes : bytes; }

// The new tokens of slot b: first packed token and count, and the cached length.  A bad row of q_start, a
// negative or overlong length gives count 0 and its code.
struct SlotSpan {
  int q0, n, t0, code;
};
PATH_HD SlotSpan slot_span_of(int b, const int* q_start, int seq_len, int total, int max_new, int table_width,
                              int page_size) {
  SlotSpan s{0, 0, seq_len, 0};
  int n = 1, q0 = b;
  if (q_start) {
    q0 = q_start[b];
    const long long dn = (long long)q_start[b + 1] - q0;
    if (q0 < 0 || dn < 0 || (long long)q0 + dn > total || dn > max_new) {
      s.code = PATH_PAGED_BAD_START;
      return s;
    }
    n = (int)dn;
    if (n == 0) return s;
    if (seq_len < 0) {
      s.code = PATH_PAGED_BAD_SLOT;
      return s;
    }
  } else if (seq_len < 0) {
    return s;
  }
  if ((long long)seq_len + n > (long long)table_width * page_size) {
    s.code = PATH_PAGED_CAPACITY;
    return s;
  }
  s.q0 = q0;
  s.n = n;
  return s;
}
// Row j of slot b in a pool: its row number for head h, or -1 where the table holds no page of the pool.
PATH_HD long long pool_row(const path_paged_cache_t& c, const int* table, int pages, int b, int h, int j) {
  const int pg = table[(size_t)b * c.table_width + j / c.page_size];
  if ((unsigned)pg >= (unsigned)pages) return -1;
  return ((long long)pg * c.heads + h) * c.page_size + j % c.page_size;
}
// Whether there are pages of both pools for rows t0 .. t0 + n - 1 of slot b, by one thread.
PATH_HD bool rows_there(const path_paged_cache_t& c, int b, int t0, int n) {
  bool ok = true;
  for (int x = t0 / c.page_size; n > 0 && x <= (t0 + n - 1) / c.page_size; ++x) {
    const size_t at = (size_t)b * c.table_width + x;
    ok &= (unsigned)c.k_table[at] < (unsigned)c.k_pages && (unsigned)c.v_table[at] < (unsigned)c.v_pages;
  }
  return ok;
}
// Whether the token at position pq sees row j <= pq (window 0: all).
PATH_HD bool sees(int window, int sinks, int pq, int j) { return window <= 0 || j > pq - window || j < sinks; }

// The cached rows of a sequence that a call works on: rows [0, sinks) (first tokens that stay visible) and
// those its first new token sees, up to t0, cut into tiles of `rows` rows that start at multiples of
// `rows`.  Tile i of the list is tile i < nh ? i : i + skip of the sequence.
struct LiveTiles {
  int nh, skip, count;
};
PATH_HD LiveTiles live_tiles(int t0, int window, int sinks, int rows) {
  LiveTiles l{0, 0, 0};
  const int all = t0 <= 0 ? 0 : (t0 + rows - 1) / rows;
  l.nh = l.count = all;
  if (window <= 0 || all == 0) return l;
  const int head = sinks < t0 ? sinks : t0;
  const int from = t0 - window + 1 > 0 ? t0 - window + 1 : 0;
  const int nh = (head + rows - 1) / rows;
  const int first = from >= t0 ? all : from / rows;
  if (first <= nh) return l;
  l.nh = nh;
  l.skip = first - nh;
  l.count = all - l.skip;
  return l;
}
PATH_HD int live_tile(const LiveTiles& l, int i) { return i < l.nh ? i : i + l.skip; }
// The same from the newest tile to the oldest: with a forget gate the largest scores come first, so the running
// maximum of a softmax hardly moves after the first tile (oldest first it rises at every tile).
PATH_HD int newest_tile(const LiveTiles& l, int i) { return live_tile(l, l.count - 1 - i); }

#ifdef __CUDACC__
__device__ __forceinline__ SlotSpan slot_span(const PagedArgs& p, int b) {
  return slot_span_of(b, p.q_start, p.c.seq_len[b], p.total, p.max_new, p.c.table_width, p.c.page_size);
}
__device__ __forceinline__ void paged_error(int* status, int code) { atomicCAS(status, 0, code); }
// Running sum of log f at a row of the value pool: a pair of fp32 numbers (48 bits) where the cache has a place for the
// rest.  The sums are absolute, so that pages can be shared, and grow with the position: after a million tokens fp32
// alone would lose a log f of 0.01 whole.
__device__ __forceinline__ double load_sum(const path_paged_cache_t& c, long long at) {
  return c.a_rest ? (double)c.a_pool[at] + c.a_rest[at] : c.a_pool[at];
}
__device__ __forceinline__ void store_sum(const path_paged_cache_t& c, long long at, double a) {
  const float hi = (float)a;
  c.a_pool[at] = hi;
  if (c.a_rest) c.a_rest[at] = isfinite(hi) ? (float)(a - hi) : 0.f;
}
__device__ __forceinline__ float sum_rest(const path_paged_cache_t& c, long long at) { return c.a_rest ? c.a_rest[at] : 0.f; }
// Numbers the slots with several new tokens in slot order, by a block of 32 warps, one slot per thread and step: this
// slot's number; `numbered` (the same in all threads) counts on.  multi: 32 ints in shared memory, not written again before
// the block's next barrier.
__device__ __forceinline__ int number_multi(bool have, int* multi, int& numbered) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned some = __ballot_sync(0xffffffffu, have);
  if (lane == 0) multi[warp] = __popc(some);
  __syncthreads();
  const int m = multi[lane];
  const int number = numbered + (int)__reduce_add_sync(0xffffffffu, lane < warp ? m : 0) + __popc(some & ((1u << lane) - 1));
  numbered += (int)__reduce_add_sync(0xffffffffu, m);
  return number;
}
// What a call did with slot b, for path_paged_advance: its new tokens, or -1 where it was left out.
__device__ __forceinline__ void note_extended(const path_paged_cache_t& c, int b, int n) {
  if (c.extended) c.extended[b] = n;
}
// rows_there() by a warp, for as many rows as there may be.
__device__ __forceinline__ bool rows_there_warp(const path_paged_cache_t& c, int b, int t0, int n) {
  bool ok = true;
  for (int x = t0 / c.page_size + (threadIdx.x & 31); x <= (t0 + n - 1) / c.page_size; x += 32) {
    const size_t at = (size_t)b * c.table_width + x;
    ok &= (unsigned)c.k_table[at] < (unsigned)c.k_pages && (unsigned)c.v_table[at] < (unsigned)c.v_pages;
  }
  return __all_sync(0xffffffffu, ok);
}
// The planning kernels' look at a slot with several new tokens, by a whole warp (one slot per lane, s.n > 0 where the lane
// has such a slot): clears s.n where a page for one of all its new tokens (t0, n: of the call) is missing.
__device__ __forceinline__ void leave_out_pageless(const path_paged_cache_t& c, int b, int t0, int n, SlotSpan& s, bool report) {
  unsigned look = __ballot_sync(0xffffffffu, s.n > 0);
  while (look) {
    const int lane = __ffs(look) - 1;
    look &= look - 1;
    const bool ok = rows_there_warp(c, __shfl_sync(0xffffffffu, b, lane), __shfl_sync(0xffffffffu, t0, lane),
                                    __shfl_sync(0xffffffffu, n, lane));
    if (!ok && lane == (int)(threadIdx.x & 31)) {
      s.n = 0;
      s.code = PATH_PAGED_BAD_PAGE;
      if (report) paged_error(c.status, s.code);
    }
  }
}
// Programmatic dependent launch: every kernel of a call begins with chain(), which waits until the kernel before it has
// ended and lets the next one's blocks take their places meanwhile (they wait there).  The first statement of every
// kernel, for all threads: a grid that ended without having waited would end the chain early.  Pointers to what earlier
// kernels write are not __restrict__ and not read with __ldg: such loads may pass the wait or find a line that the kernel
// before has left in the read-only path.
__device__ __forceinline__ void chain() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
#endif

// ---- launchers ----
// path_paged_extend: chooses the kernels of a call.
size_t paged_ws_bytes(const PagedArgs& p);
cudaError_t launch_paged(const PagedArgs& p, char* ws, cudaStream_t st);

size_t paged_chunk_ws_bytes(const PagedArgs& p);
cudaError_t launch_paged_chunk(const PagedArgs& p, char* ws, cudaStream_t st);

// Slots with one new token; where paged_drafts() holds (bf16), all slots of the call.
bool paged_drafts(const PagedArgs& p);
size_t paged_token_ws_bytes(const PagedArgs& p);
cudaError_t launch_paged_token(const PagedArgs& p, char* ws, cudaStream_t st);

// Prompt chunks, bf16.
size_t paged_new_ws_bytes(const PagedArgs& p);
cudaError_t launch_paged_new(const PagedArgs& p, char* ws, cudaStream_t st);

size_t pages_ws_bytes(const path_paged_cache_t& c);
cudaError_t launch_pages_reserve(const path_paged_cache_t& c, const int* n_new, char* ws, cudaStream_t st);
cudaError_t launch_pages_plan(const path_paged_cache_t& c, const int* n_new, const int* from_start, int tokens, int* q_start,
                              int* slot, int* position, int* k_row, int* v_row, int* source, char* ws, cudaStream_t st);
cudaError_t launch_pages_fork(const path_paged_cache_t& c, const int* parents, const int* children, int count, char* ws,
                              cudaStream_t st);
cudaError_t launch_pages_free(const path_paged_cache_t& c, const int* slots, int count, char* ws, cudaStream_t st);
cudaError_t launch_pages_trim(const path_paged_cache_t& c, int window, int sinks, char* ws, cudaStream_t st);
cudaError_t launch_pages_compact(const path_paged_cache_t& c, char* ws, cudaStream_t st);
cudaError_t launch_paged_advance(const path_paged_cache_t& c, const int* q_start, cudaStream_t st);

}  // namespace pathattn
