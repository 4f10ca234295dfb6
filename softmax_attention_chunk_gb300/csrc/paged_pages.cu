// Paged serving: giving out, copying, returning and compacting pages.
//
// The bookkeeping of a call (tables, lengths, reference counts) is done by one block, so that pages are
// given out in a fixed order (lowest free number first) without atomics deciding it; what it finds out
// goes into the workspace as a list of (source, destination) pages, which a second kernel copies with
// the whole GPU.  A call first counts what it needs and looks at every entry of its lists, and only then
// writes; a code in the status word means that nothing was written.
// Bound: the copies (each byte read and written once): compaction that moves 426 MB 148 us, of which the copy 127 (6.7
// TB/s, a plain copy's rate) and the bookkeeping by one block the rest (pieces of 16 KB in place of 8: 147); a fork of
// one short sequence is the latency of its launches.
#include <cooperative_groups.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace pathattn {
namespace {

constexpr int NT = 1024;           // threads of the bookkeeping block
constexpr int NW = NT / 32;
constexpr int CT = 256;            // threads of a copying block
constexpr int kMaxSlots = 65535;   // duplicate check: one bit per slot in shared memory

// Workspace: counts, then the page lists of the two pools (sources, destinations), the per-entry offsets of a
// fork / reserve, and the old -> new map of a compaction.
struct PagesWs {
  size_t head, ksrc, kdst, vsrc, vdst, koff, voff, kmap, vmap, total;
};
PagesWs pages_ws(const path_paged_cache_t& c) {
  PagesWs w{};
  size_t off = 0;
  auto take = [&](size_t n) { size_t o = off; off = align_up(off + n * 4, 256); return o; };
  w.head = take(16);
  w.ksrc = take(c.k_pages);
  w.kdst = take(c.k_pages);
  w.vsrc = take(c.v_pages);
  w.vdst = take(c.v_pages);
  w.koff = take(c.slots);
  w.voff = take(c.slots);
  w.kmap = take(c.k_pages);
  w.vmap = take(c.v_pages);
  w.total = off;
  return w;
}
struct Lists {  // the same, as pointers; head: 0 key copies, 1 value copies, 2 keys in use, 3 values in use
  int *head, *ksrc, *kdst, *vsrc, *vdst, *koff, *voff, *kmap, *vmap;
};
Lists lists(const path_paged_cache_t& c, char* ws) {
  const PagesWs w = pages_ws(c);
  auto at = [&](size_t o) { return (int*)(ws + o); };
  return {at(w.head), at(w.ksrc), at(w.kdst), at(w.vsrc), at(w.vdst), at(w.koff), at(w.voff), at(w.kmap), at(w.vmap)};
}

template <typename I> struct BlockScanOf {
  I sum[NW];
};
using BlockScan = BlockScanOf<int>;
// Exclusive prefix sum of one number per thread over the block; *total gets the sum.
template <typename I> __device__ I block_scan(I x, BlockScanOf<I>& s, I* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  I v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I a = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += a;
  }
  __syncthreads();  // the previous use of s is over
  if (lane == 31) s.sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    I t = s.sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const I a = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += a;
    }
    s.sum[lane] = t;
  }
  __syncthreads();
  *total = s.sum[NW - 1];
  return v - x + (warp > 0 ? s.sum[warp - 1] : 0);
}

// The numbers of the first `need` pages with ref == 0, in rising order, into out; returns how many were
// found (fewer: the pool has no more).  A warp looks at PER rows of 32 neighbouring pages, the next ones on their way.
__device__ int lowest_free(const int* ref, int pages, int need, int* out, BlockScan& s) {
  constexpr int PER = 16;
  const int lane = threadIdx.x & 31, at0 = (threadIdx.x >> 5) * (32 * PER) + lane;
  int have = 0;
  int r[PER], next[PER];
  auto load = [&](int base, int (&x)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = base + at0 + 32 * i < pages ? ref[base + at0 + 32 * i] : 1;
  };
  if (need > 0) load(0, next);
  for (int base = 0; base < pages && have < need; base += NT * PER) {
    unsigned free[PER];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) r[i] = next[i];
    if (base + NT * PER < pages) load(base + NT * PER, next);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      free[i] = __ballot_sync(0xffffffffu, r[i] <= 0);
      mine += __popc(free[i]);
    }
    int tot;
    int at = have + block_scan(lane == 0 ? mine : 0, s, &tot);
    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int mineat = at + __popc(free[i] & ((1u << lane) - 1));
      if ((free[i] >> lane & 1) && mineat < need) out[mineat] = base + at0 + 32 * i;
      at += __popc(free[i]);
    }
    have += tot;
  }
  return have < need ? have : need;
}

// Whether an entry of list[0, count) is no slot, is listed twice, or has not seq_len >= 0 (used) or < 0.
__device__ bool bad_slots(const int* list, int count, const int* seq_len, int slots, bool used,
                          unsigned* seen) {
  for (int i = threadIdx.x; i < (slots + 31) / 32; i += NT) seen[i] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < count; i += NT) {
    const int b = list[i];
    if ((unsigned)b >= (unsigned)slots) {
      bad = true;
      continue;
    }
    if ((seq_len[b] >= 0) != used) bad = true;
    if (atomicOr(&seen[b >> 5], 1u << (b & 31)) >> (b & 31) & 1) bad = true;
  }
  return __syncthreads_or(bad) != 0;
}

// ---------------- reserve, plan ----------------
// Where the packed tokens of a plan go.
struct PlanMaps {
  const int *q_start, *from_start;
  int *slot, *position, *k_row, *v_row, *source;
  int tokens;
};
// Token i's entries; at(b): q_start[b].  What another block may just have written is read past L1.
template <typename At> __device__ __forceinline__ void plan_token(const path_paged_cache_t& c, const PlanMaps& m, At at, int i) {
  int slot = -1, pos = -1, k = -1, v = -1, from = -1;
  if (i < at(c.slots)) {
    int lo = 0, hi = c.slots;  // the last slot that starts at i or before: slots without tokens start where the next one does
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (at(mid) <= i) lo = mid; else hi = mid;
    }
    slot = lo;
    const int len = __ldcg(c.seq_len + slot);
    pos = (len < 0 ? 0 : len) + i - at(slot);  // (below 0: being opened)
    const size_t e = (size_t)slot * c.table_width + pos / c.page_size;
    const int kp = __ldcg(c.k_table + e), vp = __ldcg(c.v_table + e), in = pos % c.page_size;
    k = (unsigned)kp < (unsigned)c.k_pages ? kp * c.page_size + in : -1;
    v = (unsigned)vp < (unsigned)c.v_pages ? vp * c.page_size + in : -1;
    if (m.from_start) from = m.from_start[slot] + i - at(slot);
  }
  m.slot[i] = slot;
  m.position[i] = pos;
  m.k_row[i] = k;
  m.v_row[i] = v;
  if (m.source) m.source[i] = from;
}
constexpr int kPlanStarts = 2048;  // q_start in shared memory, up to so many slots
// Up to so many tokens the planning blocks write the maps themselves: a launch less (4080 tokens: 24.7 us a call in place of 31.3,
// 12.3 us on the GPU either way; 16000 tokens would take them 20.5 us).
constexpr int kPlanInline = 4096;
__global__ void __launch_bounds__(CT) plan_kernel(path_paged_cache_t c, PlanMaps m) {
  chain();
  __shared__ int starts[kPlanStarts + 1];
  const bool copied = c.slots <= kPlanStarts;
  if (copied) {
    for (int b = threadIdx.x; b <= c.slots; b += CT) starts[b] = m.q_start[b];
    __syncthreads();
  }
  const int i = blockIdx.x * CT + threadIdx.x;
  if (i < m.tokens) plan_token(c, m, [&](int b) { return copied ? starts[b] : m.q_start[b]; }, i);
}

// One block for the keys' pool and one for the values' (a cluster): each counts what its table lacks and looks for as many
// free pages; only when both know that nothing is refused do they write.  Slots are taken NT at a time, their columns
// (those behind the last page, up to the page of the last new row) side by side in order.
// q_start (or null): gets the running sums of the slots' new tokens, zeros where the call records a code; more of them than
// m.tokens are one.  inside: writes the maps too.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NT)
    reserve_kernel(path_paged_cache_t c, const int* n_new, Lists w, int* q_start, PlanMaps m, bool inside) {
  chain();
  __shared__ BlockScan s;
  __shared__ BlockScanOf<long long> wide;
  __shared__ int code, first[NT + 1], column[NT];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, P = c.page_size, tokens = m.tokens;
  const bool values = cluster.block_rank() == 1;
  int* table = values ? c.v_table : c.k_table;
  int* ref = values ? c.v_ref : c.k_ref;
  int* list = values ? w.vdst : w.kdst;
  const int pages = values ? c.v_pages : c.k_pages;
  if (tid == 0) code = 0;
  __syncthreads();
  long long all = 0;
  // visit(entry, lacks) for every column of every slot, by the whole block in step; count: the first time
  auto walk = [&](bool count, auto visit) {
    for (int base = 0; base < c.slots; base += NT) {
      const int b = base + tid;
      int cols = 0, n = 0;
      if (b < c.slots) {
        const int len = c.seq_len[b];
        n = n_new ? n_new[b] : (len >= 0 ? 1 : 0);
        n = n < 0 ? 0 : n;
        const long long have = len < 0 ? 0 : len, to = have + n;
        column[tid] = (int)((have + P - 1) / P);
        if (n && to > (long long)c.table_width * P) atomicCAS(&code, 0, PATH_PAGED_CAPACITY);
        else if (n) cols = (int)((to + P - 1) / P) - column[tid];
      }
      if (count && q_start) {
        long long t;
        const long long a = all + block_scan<long long>(n, wide, &t);
        if (!values && b < c.slots) q_start[b] = (int)(a < tokens ? a : tokens);
        all += t;
      }
      int total;
      first[tid] = block_scan(cols, s, &total);
      if (tid == 0) first[NT] = total;
      __syncthreads();
      for (int i0 = 0; i0 < total; i0 += NT) {
        const int i = i0 + tid;
        size_t e = 0;
        bool lacks = false;
        if (i < total) {
          int lo = 0, hi = NT;
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i) lo = mid; else hi = mid;
          }
          e = (size_t)(base + lo) * c.table_width + column[lo] + (i - first[lo]);
          lacks = table[e] < 0;
        }
        visit(e, lacks);
      }
      __syncthreads();
    }
  };
  int need = 0;
  walk(true, [&](size_t, bool lacks) { need += __syncthreads_count(lacks); });
  if (q_start && tid == 0) {
    if (!values) q_start[c.slots] = (int)(all < tokens ? all : tokens);
    if (all > tokens) atomicCAS(&code, 0, PATH_PAGED_BAD_START);
  }
  __syncthreads();
  if (code == 0 && (need > pages || lowest_free(ref, pages, need, list, s) < need) && tid == 0) code = PATH_PAGED_NO_PAGES;
  cluster.sync();
  const int mine = code, other = *cluster.map_shared_rank(&code, values ? 0 : 1);
  cluster.sync();  // (neither block has gone while the other reads, nor writes before both know)
  if (mine || other) {
    if (!values) {
      if (tid == 0) paged_error(c.status, mine ? mine : other);
      if (q_start)
        for (int b = tid; b <= c.slots; b += NT) q_start[b] = 0;
    }
    if (inside)
      for (int i = tid + (values ? NT : 0); i < tokens; i += 2 * NT) {
        m.slot[i] = m.position[i] = m.k_row[i] = m.v_row[i] = -1;
        if (m.source) m.source[i] = -1;
      }
    return;
  }
  int given = 0;
  walk(false, [&](size_t e, bool lacks) {
    int t;
    const int at = given + block_scan<int>(lacks, s, &t);
    if (lacks) {
      const int pg = list[at];
      table[e] = pg;
      ref[pg] = 1;
    }
    given += t;
  });
  if (inside) {  // both tables and q_start stand
    __threadfence();
    cluster.sync();
    const bool copied = c.slots <= NT;
    if (copied) {
      for (int b = tid; b <= c.slots; b += NT) first[b] = __ldcg(q_start + b);
      __syncthreads();
    }
    for (int i = tid + (values ? NT : 0); i < tokens; i += 2 * NT)
      plan_token(c, m, [&](int b) { return copied ? first[b] : __ldcg(q_start + b); }, i);
  }
  if (!values)  // (an empty slot counts as length 0 above, so it does not matter when the other block sees this)
    for (int b = tid; b < c.slots; b += NT)
      if (n_new && n_new[b] > 0 && c.seq_len[b] < 0) {
        c.seq_len[b] = 0;
        note_extended(c, b, 0);
      }
}

// ---------------- fork ----------------
__global__ void __launch_bounds__(NT) fork_kernel(path_paged_cache_t c, const int* parents,
                                                  const int* children, int count, Lists w) {
  chain();
  __shared__ BlockScan s;
  __shared__ unsigned seen[(kMaxSlots + 31) / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = c.page_size;
  if (tid == 0) w.head[0] = w.head[1] = 0;
  const bool bad = bad_slots(children, count, c.seq_len, c.slots, false, seen);
  bool lost = false;
  for (int i = tid; i < count; i += NT) {
    const int b = parents[i];
    if ((unsigned)b >= (unsigned)c.slots || c.seq_len[b] < 0) lost = true;
  }
  if (__syncthreads_or(bad || lost)) {
    if (tid == 0) paged_error(c.status, PATH_PAGED_BAD_SLOT);
    return;
  }
  for (int i = warp; i < count; i += NW) {  // pages each child gets, one warp per child
    const int b = parents[i], len = c.seq_len[b];
    const int ncol = (int)(((long long)len + P - 1) / P);
    int nk = 0, nv = 0;
    bool out = ncol > c.table_width;
    for (int x = lane; x < min(ncol, c.table_width); x += 32) {
      const int kp = c.k_table[(size_t)b * c.table_width + x], vp = c.v_table[(size_t)b * c.table_width + x];
      nk += kp >= 0;
      nv += vp >= 0 && x == ncol - 1 && len % P != 0;
      out |= kp >= c.k_pages || vp >= c.v_pages;
    }
    nk = __reduce_add_sync(0xffffffffu, nk);
    nv = __reduce_add_sync(0xffffffffu, nv);
    lost |= out;
    if (lane == 0) {
      w.koff[i] = nk;
      w.voff[i] = nv;
    }
  }
  if (__syncthreads_or(lost)) {
    if (tid == 0) paged_error(c.status, PATH_PAGED_BAD_PAGE);
    return;
  }
  int needk = 0, needv = 0;  // (at most slots * table_width)
  for (int base = 0; base < count; base += NT) {
    const int i = base + tid;
    int t1, t2;
    const int a = block_scan(i < count ? w.koff[i] : 0, s, &t1);
    if (i < count) w.koff[i] = needk + a;
    const int e = block_scan(i < count ? w.voff[i] : 0, s, &t2);
    if (i < count) w.voff[i] = needv + e;
    needk += t1;
    needv += t2;
  }
  __syncthreads();
  if (needk > c.k_pages || needv > c.v_pages || lowest_free(c.k_ref, c.k_pages, needk, w.kdst, s) < needk ||
      lowest_free(c.v_ref, c.v_pages, needv, w.vdst, s) < needv) {
    if (tid == 0) paged_error(c.status, PATH_PAGED_NO_PAGES);
    return;
  }
  __syncthreads();
  for (int i = warp; i < count; i += NW) {
    const int b = parents[i], ch = children[i], len = c.seq_len[b];
    const int ncol = (int)(((long long)len + P - 1) / P);
    int ak = w.koff[i], av = w.voff[i];
    for (int x0 = 0; x0 < c.table_width; x0 += 32) {
      const int x = x0 + lane;
      int kp = -1, vp = -1;
      if (x < ncol) {
        kp = c.k_table[(size_t)b * c.table_width + x];
        vp = c.v_table[(size_t)b * c.table_width + x];
      }
      const bool ck = kp >= 0, cv = vp >= 0 && x == ncol - 1 && len % P != 0;
      const unsigned mk = __ballot_sync(0xffffffffu, ck), mv = __ballot_sync(0xffffffffu, cv);
      const unsigned below = (1u << lane) - 1;
      if (ck) {
        const int at = ak + __popc(mk & below);
        w.ksrc[at] = kp;
        kp = w.kdst[at];
        c.k_ref[kp] = 1;
      }
      if (cv) {
        const int at = av + __popc(mv & below);
        w.vsrc[at] = vp;
        vp = w.vdst[at];
        c.v_ref[vp] = 1;
      } else if (vp >= 0) {
        atomicAdd(&c.v_ref[vp], 1);
      }
      if (x < c.table_width) {
        c.k_table[(size_t)ch * c.table_width + x] = kp < 0 ? -1 : kp;
        c.v_table[(size_t)ch * c.table_width + x] = vp < 0 ? -1 : vp;
      }
      ak += __popc(mk);
      av += __popc(mv);
    }
    if (lane == 0) {
      c.seq_len[ch] = len;
      note_extended(c, ch, 0);
    }
  }
  if (tid == 0) {
    w.head[0] = needk;
    w.head[1] = needv;
  }
}

// ---------------- free, trim ----------------
// Returns column x of slot b.
__device__ __forceinline__ void drop(const path_paged_cache_t& c, int b, int x) {
  int* kt = c.k_table + (size_t)b * c.table_width + x;
  int* vt = c.v_table + (size_t)b * c.table_width + x;
  const int kp = *kt, vp = *vt;
  if ((unsigned)kp < (unsigned)c.k_pages) c.k_ref[kp] = 0;
  if ((unsigned)vp < (unsigned)c.v_pages) atomicSub(&c.v_ref[vp], 1);
  *kt = -1;
  *vt = -1;
}
__global__ void __launch_bounds__(NT) free_kernel(path_paged_cache_t c, const int* list, int count) {
  chain();
  __shared__ unsigned seen[(kMaxSlots + 31) / 32];
  if (bad_slots(list, count, c.seq_len, c.slots, true, seen)) {
    if (threadIdx.x == 0) paged_error(c.status, PATH_PAGED_BAD_SLOT);
    return;
  }
  for (int i = threadIdx.x >> 5; i < count; i += NW) {
    const int b = list[i];
    for (int x = threadIdx.x & 31; x < c.table_width; x += 32) drop(c, b, x);
    if ((threadIdx.x & 31) == 0) {
      c.seq_len[b] = -1;
      note_extended(c, b, 0);
    }
  }
}
// One block per slot: slots share no table row, and value counts fall by atomics (sums of ones: the order
// does not matter).
__global__ void __launch_bounds__(CT) trim_kernel(path_paged_cache_t c, int window, int sinks) {
  chain();
  const int b = blockIdx.x, P = c.page_size, len = c.seq_len[b];
  if (len <= 0) return;
  // rows j with sinks <= j <= len - window are hidden from position len on
  for (int x = threadIdx.x; x < c.table_width; x += CT) {
    const long long first = (long long)x * P, last = first + P - 1;
    if (first >= sinks && last <= (long long)len - window && last < len - 1) drop(c, b, x);
  }
}

// ---------------- compact ----------------
// Pool by pool: pages in use above the number of used ones, and holes below it, both in rising order.
__device__ int dense_lists(int* ref, int pages, int* src, int* dst, int* map,
                           int* used_out, BlockScan& s) {
  constexpr int PER = 8;
  int used = 0;
  for (int base = 0; base < pages; base += NT * PER) {
    int n = 0, t;
    const int p0 = base + threadIdx.x * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += p0 + i < pages && ref[p0 + i] > 0;
    block_scan(n, s, &t);
    used += t;
  }
  int nd = 0, ns = 0;
  for (int base = 0; base < pages; base += NT * PER) {
    const int p0 = base + threadIdx.x * PER;
    int hole = 0, full = 0, t1, t2;
    unsigned bits = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int pg = p0 + i;
      const bool u = pg < pages && ref[pg] > 0;
      if (u) bits |= 1u << i;
      hole += !u && pg < used;
      full += u && pg >= used;
    }
    int ad = nd + block_scan(hole, s, &t1), as = ns + block_scan(full, s, &t2);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int pg = p0 + i;
      const bool u = bits >> i & 1;
      if (!u && pg < used) dst[ad++] = pg;
      if (!u && pg >= used && pg < pages) map[pg] = pg;  // (named by a table all the same: left)
      if (u && pg >= used) src[as++] = pg;
    }
    nd += t1;
    ns += t2;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ns; i += NT) {
    const int a = src[i], b = dst[i];
    map[a] = b;
    ref[b] = ref[a];
    ref[a] = 0;
  }
  *used_out = used;
  return ns;
}
__global__ void __launch_bounds__(NT) compact_kernel(path_paged_cache_t c, Lists w) {
  chain();
  __shared__ BlockScan s;
  int used;
  if (blockIdx.x == 0) {  // one block per pool
    const int n = dense_lists(c.k_ref, c.k_pages, w.ksrc, w.kdst, w.kmap, &used, s);
    if (threadIdx.x == 0) {
      w.head[0] = n;
      w.head[2] = used;
    }
  } else {
    const int n = dense_lists(c.v_ref, c.v_pages, w.vsrc, w.vdst, w.vmap, &used, s);
    if (threadIdx.x == 0) {
      w.head[1] = n;
      w.head[3] = used;
    }
  }
}

// ---------------- copies ----------------
constexpr int kPiece = 8192;  // bytes of a page that one block copies at a time
// Copies the listed pages; with `map` also rewrites the tables (entries at or above the number of pages
// in use have moved).
__global__ void __launch_bounds__(CT) copy_kernel(path_paged_cache_t c, Lists w, size_t page_bytes, int map) {
  chain();
  const int nk = w.head[0], nv = w.head[1];
  const size_t abytes = c.a_pool ? (size_t)c.heads * c.page_size * 4 : 0;
  const long long pieces = (long long)((page_bytes + kPiece - 1) / kPiece);  // (a piece may be short)
  const long long apieces = (long long)((abytes + kPiece - 1) / kPiece);
  const long long uk = nk * pieces, uv = nv * pieces, ua = nv * apieces, ur = c.a_rest ? ua : 0;
  for (long long u = blockIdx.x; u < uk + uv + ua + ur; u += gridDim.x) {
    char* pool;
    const int *src, *dst;
    size_t size = page_bytes;
    long long x = u, per = pieces;
    if (u < uk) {
      pool = (char*)c.k_pool; src = w.ksrc; dst = w.kdst;
    } else if (u < uk + uv) {
      x = u - uk;
      pool = (char*)c.v_pool; src = w.vsrc; dst = w.vdst;
    } else {
      x = u - uk - uv;
      pool = (char*)c.a_pool; src = w.vsrc; dst = w.vdst;
      if (x >= ua) {
        x -= ua;
        pool = (char*)c.a_rest;
      }
      size = abytes;
      per = apieces;
    }
    const size_t i = x / per, off = (size_t)(x % per) * kPiece;
    const uint4* from = (const uint4*)(pool + (size_t)src[i] * size + off);
    uint4* to = (uint4*)(pool + (size_t)dst[i] * size + off);
    const int n = (int)((size - off < kPiece ? size - off : kPiece) / 16);
    uint4 r[kPiece / 16 / CT];
#pragma unroll
    for (int q = 0; q < kPiece / 16 / CT; ++q) {
      const int e = q * CT + threadIdx.x;
      if (e < n) r[q] = from[e];
    }
#pragma unroll
    for (int q = 0; q < kPiece / 16 / CT; ++q) {
      const int e = q * CT + threadIdx.x;
      if (e < n) to[e] = r[q];
    }
  }
  if (map) {
    const int usedk = w.head[2], usedv = w.head[3];
    const size_t n = (size_t)c.slots * c.table_width;
    for (size_t e = (size_t)blockIdx.x * CT + threadIdx.x; e < n; e += (size_t)gridDim.x * CT) {
      const int kp = c.k_table[e], vp = c.v_table[e];
      if (kp >= usedk && kp < c.k_pages) c.k_table[e] = w.kmap[kp];
      if (vp >= usedv && vp < c.v_pages) c.v_table[e] = w.vmap[vp];
    }
  }
}

__global__ void advance_kernel(path_paged_cache_t c, const int* q_start) {
  chain();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= c.slots) return;
  const int len = c.seq_len[b];
  if (len < 0) return;
  const long long n = q_start ? (long long)q_start[b + 1] - q_start[b] : 1;
  if (n == 0) return;  // (what another call gave the slot keeps waiting)
  const int given = c.extended ? c.extended[b] : 0;
  if (given < 0) {  // left out: extend has recorded why
    c.extended[b] = 0;
    return;
  }
  int code = 0;
  if (n < 0 || (given > 0 && n != given)) code = PATH_PAGED_BAD_START;
  else if (len + n > (long long)c.table_width * c.page_size) code = PATH_PAGED_CAPACITY;
  else if (given == 0 && !rows_there(c, b, len, (int)n)) code = PATH_PAGED_BAD_PAGE;  // (no extend has looked)
  if (code) {
    paged_error(c.status, code);
    return;
  }
  c.seq_len[b] = (int)(len + n);
  note_extended(c, b, 0);
}

size_t page_bytes(const path_paged_cache_t& c) {
  return (size_t)c.heads * c.page_size * c.head_dim * (c.cache_dtype == PATH_BF16 ? 2 : 4);
}
cudaError_t copy_pages(const path_paged_cache_t& c, const Lists& w, int map, cudaStream_t st) {
  return launch_chained(copy_kernel, 152 * 8, CT, 0, st, c, w, page_bytes(c), map);
}

}  // namespace

size_t pages_ws_bytes(const path_paged_cache_t& c) { return pages_ws(c).total; }

cudaError_t launch_pages_reserve(const path_paged_cache_t& c, const int* n_new, char* ws, cudaStream_t st) {
  return launch_chained(reserve_kernel, 2, NT, 0, st, c, n_new, lists(c, ws), nullptr, PlanMaps{}, false);
}
cudaError_t launch_pages_plan(const path_paged_cache_t& c, const int* n_new, const int* from_start, int tokens, int* q_start,
                              int* slot, int* position, int* k_row, int* v_row, int* source, char* ws, cudaStream_t st) {
  const PlanMaps m{q_start, from_start, slot, position, k_row, v_row, source, tokens};
  const bool inside = tokens <= kPlanInline;
  const cudaError_t e = launch_chained(reserve_kernel, 2, NT, 0, st, c, n_new, lists(c, ws), q_start, m, inside);
  if (e != cudaSuccess || inside) return e;
  return launch_chained(plan_kernel, (unsigned)((tokens + CT - 1) / CT), CT, 0, st, c, m);
}
cudaError_t launch_pages_fork(const path_paged_cache_t& c, const int* parents, const int* children, int count, char* ws,
                              cudaStream_t st) {
  const Lists w = lists(c, ws);
  const cudaError_t e = launch_chained(fork_kernel, 1, NT, 0, st, c, parents, children, count, w);
  if (e != cudaSuccess) return e;
  return copy_pages(c, w, 0, st);
}
cudaError_t launch_pages_free(const path_paged_cache_t& c, const int* slots, int count, char*, cudaStream_t st) {
  return launch_chained(free_kernel, 1, NT, 0, st, c, slots, count);
}
cudaError_t launch_pages_trim(const path_paged_cache_t& c, int window, int sinks, char*, cudaStream_t st) {
  return launch_chained(trim_kernel, (unsigned)c.slots, CT, 0, st, c, window, sinks);
}
cudaError_t launch_pages_compact(const path_paged_cache_t& c, char* ws, cudaStream_t st) {
  const Lists w = lists(c, ws);
  const cudaError_t e = launch_chained(compact_kernel, 2, NT, 0, st, c, w);
  if (e != cudaSuccess) return e;
  return copy_pages(c, w, 1, st);
}
cudaError_t launch_paged_advance(const path_paged_cache_t& c, const int* q_start, cudaStream_t st) {
  return launch_chained(advance_kernel, (unsigned)((c.slots + 255) / 256), 256, 0, st, c, q_start);
}

}  // namespace pathattn
