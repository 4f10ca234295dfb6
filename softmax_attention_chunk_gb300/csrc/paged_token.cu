// Paged serving, few new tokens per slot (one token, or, bf16, draft tokens): one pass over the
// cache that reads every key and value once and writes every key once.
//
// Mathematics: as in paged_chunk.cu, with the slot's n <= 16 new tokens as a single chunk.  Per key head
// the n * G transported queries z (G query heads per key head) and the n rows of W meet a cached key k as
//   s = k . z,   c = k W^T,   k <- k - c Y   (Y = U^T W;  n = 1: Y = beta w, z = q - beta (w . q) w).
//
// Bound: HBM (key read, key write, value read: 6 D bytes per cached row and head).  So:
//  * every warp works alone, without barriers, on its share of the call: the (slot, head, 16-row tile) units
//    of all sequences in one list, cut into equal runs, so that ragged lengths load all SMs alike; a run that
//    ends inside a (slot, head) leaves a partial softmax state, merged by a second kernel in a fixed order;
//  * a tile's rows go from global memory straight into the operand registers of 16x8x16 warp MMAs: the
//    operands' summation index may be permuted at will as long as both sides agree, so a lane's 16-byte
//    piece of a key row is two A fragments of K Z^T and of K W^T (keys are the 16 rows, queries and tokens the
//    columns), and its pieces of four value rows, paired by byte permutes, are A fragments of V^T P^T.  The
//    rewritten key leaves in the registers it came in.  tcgen05 would take 64 or 128 rows of queries where there are
//    1 to 32 and a trip through shared memory; here the tensor work stays far below the memory time;
//  * z, P and c are held as bf16 pairs (high + rest, about 16 bits), so that the only rounding to 8 bits is the
//    one that the cache and the output need: the extra MMAs are free under the memory bound.
// Measured: 4 x 32 heads x 32000 rows, head dim 64, 252 us (6.2 TB/s, 93 % of a copy's rate); 48 ragged sequences up
// to 4096 x 8 key heads, head dim 128, 4 heads per key head, 112 us (5.4 TB/s, 80 %: 250 registers leave 8 warps
// per SM, and a warp's loads wait on one another's tiles).  Value and key pieces through a ring in shared memory
// (cp.async, 2 to 4 tiles ahead): 278 us in place of 244 for the former's kernel; not tried at head dim 128, where registers
// are what is short.  16 x 8 heads x 5000 rows, 8 draft tokens of 2 heads, head dim 64: 90 us (floor 37: the preparing and
// merging launches, 12 warps per SM beside 168 registers of operands and accumulators, and the fragments of z, W and Y, read
// again for every tile: 9 KB beside 4 KB of keys and values; DRAM 42 %).
#include "paged.h"
#include "dev_common.cuh"
#include "mma_common.cuh"

namespace pathattn {
namespace {

constexpr int NT = 128, WARPS = NT / 32;
constexpr int RT = 16;             // rows per tile
constexpr int kSmemSlots = 1024;   // slots whose unit list each block builds for itself
constexpr float kTau = 8.f;        // lazy rescale: the reference moves when a score exceeds it by 2^8

struct TokenWs {
  int blocks;              // of the streaming kernel
  int nq;                  // query columns of a (slot, head): 8 NQ8
  size_t ustart;           // int [slots + 1]: first unit of each slot
  size_t m, l, acc;        // partial states [2 * warps][nq](, [D])
  size_t frag;             // draft tokens: per (slot, head) z and W, Y fragments
  size_t sm, sl, sacc;     // draft tokens: the new tokens' own state [slots][H][nq](, [D])
  size_t total;
};

// Blocks per SM: what the registers of the operands in flight (32 at head dim 64, 64 at 128) and of the
// accumulators (D NQ8 / 4) leave without spills.  One token, one query column tile, 4 x 32768 rows: head dim 64 with
// 4 / 3 / 2 blocks 130 / 141 / 172 us, head dim 128 with 2 / 3 blocks 132 / 156 us (floor 120).
constexpr int blocks_per_sm(int D, int nq8) { return D == 64 ? (nq8 == 1 ? 4 : nq8 == 2 ? 3 : 2) : 2; }

// Which slots the kernels here take: by the tokens of a slot.
enum { kOnlyOne = 0, kDrafts = 1 };

template <int D, int NQ8>
__host__ __device__ constexpr int frag_words() {  // uint32 per lane of one (slot, head): z high and rest, W, Y high and rest
  return NQ8 * (D / 8) * 2 + 2 * (D / 8) + 2 * (D / 8) * 2;
}
int token_nq(const PagedArgs& p, int n) {  // query columns for slots of at most n tokens
  const int c = n * p.G;
  return c <= 8 ? 8 : c <= 16 ? 16 : 32;
}
TokenWs token_ws(const PagedArgs& p, int n) {
  TokenWs w{};
  const size_t D = p.c.head_dim;
  w.nq = token_nq(p, n);
  const long long most = (long long)p.c.slots * p.c.heads * (((long long)p.c.table_width * p.c.page_size + RT - 1) / RT);
  const int full = 152 * blocks_per_sm((int)D, w.nq / 8);
  w.blocks = (int)(most < (long long)full * WARPS ? (most + WARPS - 1) / WARPS : full);
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align_up(off + bytes, 256); return o; };
  w.ustart = take((size_t)(p.c.slots + 1) * 4);
  const size_t parts = (size_t)2 * w.blocks * WARPS * w.nq;
  w.m = take(parts * 4);
  w.l = take(parts * 4);
  w.acc = take(parts * D * 4);
  if (n > 1) {
    const size_t items = (size_t)p.c.slots * p.c.heads;
    w.frag = take(items * 32 * 4 * (size_t)((w.nq / 8) * (D / 8) * 2 + 2 * (D / 8) + 2 * (D / 8) * 2));
    w.sm = take(items * w.nq * 4);
    w.sl = take(items * w.nq * 4);
    w.sacc = take(items * w.nq * D * 4);
  }
  w.total = off;
  return w;
}

// Units of a (slot, head), none where the slot is left out (a bad row, no page for one of its at most 16 new tokens):
// kSetup that stand for the time a warp needs to begin it (no work, so that runs over many
// short sequences are not longer than others), then its live tiles, at least one (the new tokens themselves).
constexpr int kSetup = 2;
// Units are numbered with 32 bits.  Slots whose visible rows all lie in key pages of their own have at most 2^31 / 16 (the rows
// of a pool) and 3 * 2^26 for beginnings and new tokens; more than this means that lengths name rows without pages, and the
// call leaves all its slots out.
constexpr long long kMaxUnits = 1 << 30;
__device__ __forceinline__ long long slot_units(const PagedArgs& p, int b, int mode, bool report) {
  const SlotSpan s = slot_span(p, b);
  const bool mine = s.n > 0 && (mode != kOnlyOne || s.n == 1);
  const bool there = !mine || rows_there(p.c, b, s.t0, s.n);
  if (report && (s.code || mine)) {
    if (s.code || !there) paged_error(p.c.status, s.code ? s.code : (int)PATH_PAGED_BAD_PAGE);
    note_extended(p.c, b, s.code || !there ? -1 : s.n);
  }
  if (!mine || !there) return 0;
  const int nt = live_tiles(s.t0, p.window, p.sinks, RT).count;
  return (long long)(kSetup + (nt > 0 ? nt : 1)) * p.c.heads;
}
// First unit of each slot, by the whole block; out may be shared memory.
template <int THREADS>
__device__ void unit_starts(const PagedArgs& p, int mode, bool report, int* out) {
  __shared__ long long wsum[THREADS / 32], carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int base = 0; base < p.c.slots; base += THREADS) {
    const int b = base + tid;
    const long long n = b < p.c.slots ? slot_units(p, b, mode, report) : 0;
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += a;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    long long before = carry;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (b < p.c.slots) out[b] = (int)(before + x - n);
    __syncthreads();
    if (tid == THREADS - 1) carry = before + x;
    __syncthreads();
  }
  if (carry > kMaxUnits) {
    for (int b = tid; b < p.c.slots; b += THREADS) {
      if (report && slot_units(p, b, mode, false) > 0) {
        paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
        note_extended(p.c, b, -1);
      }
      out[b] = 0;
    }
  }
  if (tid == 0) out[p.c.slots] = carry > kMaxUnits ? 0 : (int)carry;
  __syncthreads();
}
__global__ void __launch_bounds__(1024) unit_starts_kernel(PagedArgs p, int mode, int* out) {
  chain();
  unit_starts<1024>(p, mode, true, out);
}
// The first block's list for the merge.
__device__ __forceinline__ void keep_starts(const int* start, int slots, int* out) {
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= slots; b += NT) out[b] = start[b];
}
__device__ __forceinline__ int find_slot(const int* start, int slots, int u) {
  int lo = 0, hi = slots;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}
// Units of a warp's run.
__device__ __forceinline__ int run_length(int units, int warps) { return (units + warps - 1) / warps; }

__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// One warp: the softmax state of the query columns over the rows it has met.
template <int D, int NQ8>
struct State {
  float acc[NQ8][D / 16][4];  // O^T: tile j of column tile q; lane (g, t): d = 64 (j / 4) + 8 g + 2 (j % 4) (+ 1: c2, c3),
                              // columns 2t (c0, c2) and 2t + 1 (c1, c3)
  float m[NQ8][2], l[NQ8][2];  // reference (the same in all lanes of a column), this lane's share of the sum
};

// NT8 = 0: every slot of the list has one token.  Otherwise NT8 tiles of 8 tokens, fragments from draft_prep_kernel.
template <int D, int NQ8, int NT8, bool FOX>
__global__ void __launch_bounds__(NT, blocks_per_sm(D, NQ8)) token_kernel(PagedArgs p, TokenWs w, char* ws) {
  chain();
  __shared__ int s_start[kSmemSlots + 1];
  constexpr bool ONE = NT8 == 0;
  // z in B fragment order: registers where they are few, else one copy per warp in shared memory
  constexpr bool ZS = ONE && (D == 128 || NQ8 > 1);
  __shared__ uint4 s_z[ZS ? WARPS : 1][ZS ? NQ8 * 2 * (D / 32) : 1][32];
  constexpr int KB = D / 32;  // 32-column blocks of a row: a lane holds one 16-byte piece of each
  constexpr int CS = D / 64;  // 64-column blocks: value pieces per row and lane
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warp = blockIdx.x * WARPS + (threadIdx.x >> 5), warps = gridDim.x * WARPS;
  const int H = p.c.heads, G = p.G, P = p.c.page_size;
  const int* start;
  if (p.c.slots <= kSmemSlots) {
    unit_starts<NT>(p, ONE ? kOnlyOne : kDrafts, blockIdx.x == 0, s_start);
    start = s_start;
  } else {
    start = (const int*)(ws + w.ustart);
  }
  const int units = start[p.c.slots];
  const int run = run_length(units, warps);
  const int u0 = warp * run, u1 = min(u0 + run, units);
  // the list for the merge: with drafts here, with one token at the end (each where the registers of the loop do not suffer:
  // 4 x 32000 rows of 32 heads 253 us, with this here 270)
  if (!ONE) {
    if (p.c.slots <= kSmemSlots) keep_starts(start, p.c.slots, (int*)(ws + w.ustart));
    if (u0 >= u1) return;
  }

  const __nv_bfloat16* kpool = (const __nv_bfloat16*)p.c.k_pool;
  const __nv_bfloat16* vpool = (const __nv_bfloat16*)p.c.v_pool;
  int b = u0 < u1 ? find_slot(start, p.c.slots, u0) : 0;
  int u = u0;
  while (u < u1) {
    while (start[b + 1] <= u) ++b;  // slots without units are passed over
    const SlotSpan sp = slot_span(p, b);
    const LiveTiles lt = live_tiles(sp.t0, p.window, p.sinks, RT);
    const int per = kSetup + (lt.count > 0 ? lt.count : 1);
    const int h = (u - start[b]) / per;
    const int s0 = start[b] + h * per + kSetup;  // the item's first unit with work
    const int e0 = s0 + per - kSetup;            // and the one behind it
    if (u < s0) u = s0;
    if (u >= u1) break;
    const int ue = e0 < u1 ? e0 : u1;
    const int n = ONE ? 1 : sp.n;
    const int cols = n * G;
    State<D, NQ8> st;
    uint32_t zh[ZS ? 1 : NQ8][KB][4], zl[ZS ? 1 : NQ8][KB][4];  // ONE: z in B fragment order
    uint32_t wf[KB][4];                          // ONE: the lane's pieces of w
    float beta = 0.f;
    const uint32_t* frag = nullptr;              // drafts: this item's fragments, lane-major words
    // bias of a column's token since t0 (FOX, drafts) and its position
    float cb[NQ8][2];
    int cp[NQ8][2];
#pragma unroll
    for (int q = 0; q < NQ8; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * q + 2 * t + e, i = !ONE && col < cols ? col / G : 0;
        cp[q][e] = sp.t0 + i;
        cb[q][e] = 0.f;
        if (FOX && !ONE)
          for (int x = 0; x <= i; ++x) cb[q][e] += p.log_f[((size_t)sp.q0 + x) * H + h] * kLog2e;
      }
    // forget gate: lanes 0 and 1 of a row's four hold the sums of rows g and g + 8, lanes 2 and 3 what fp32 left of them;
    // they arrive with the tile's keys (24 x 6000..16384 rows under a window of 4096, 16 heads, head dim 64: 117 us, with
    // the values, waited for behind the next keys' loads, 133)
    const float* sums = t < 2 ? p.c.a_pool : p.c.a_rest;
    float last = 0.f;  // the last row's sum, or its rest
    if (FOX && sp.t0 > 0 && sums) {
      const long long r = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 - 1);
      if (r >= 0) last = sums[r];
    }
    const size_t tok = (size_t)sp.q0 * H + h;    // the first new token's row of k, v, w
    if constexpr (ONE) {
      beta = clamp_beta(p.beta[tok]);
      float wd[KB][8];
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        const uint4 r = ld16((const __nv_bfloat16*)p.w + tok * D + 32 * x + 8 * t);
        wf[x][0] = r.x; wf[x][1] = r.y; wf[x][2] = r.z; wf[x][3] = r.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) { wd[x][2 * i] = lo_f(wf[x][i]); wd[x][2 * i + 1] = hi_f(wf[x][i]); }
      }
#pragma unroll
      for (int q = 0; q < NQ8; ++q) {
        const int col = 8 * q + g;
        float qd[KB][8], dot = 0.f, self = 0.f;
#pragma unroll
        for (int x = 0; x < KB; ++x) {
          uint4 r = make_uint4(0, 0, 0, 0);
          if (col < cols) r = ld16((const __nv_bfloat16*)p.q + ((size_t)sp.q0 * p.hq + h * G + col) * D + 32 * x + 8 * t);
          const uint4 kr = ld16((const __nv_bfloat16*)p.k + tok * D + 32 * x + 8 * t);
          const uint32_t rr[4] = {r.x, r.y, r.z, r.w}, kk[4] = {kr.x, kr.y, kr.z, kr.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qd[x][2 * i] = lo_f(rr[i]);
            qd[x][2 * i + 1] = hi_f(rr[i]);
            dot += qd[x][2 * i] * wd[x][2 * i] + qd[x][2 * i + 1] * wd[x][2 * i + 1];
            self += qd[x][2 * i] * lo_f(kk[i]) + qd[x][2 * i + 1] * hi_f(kk[i]);
          }
        }
        dot = group_sum<4>(dot) * beta;
        self = group_sum<4>(self) * p.scl;
#pragma unroll
        for (int x = 0; x < KB; ++x) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            split2(qd[x][2 * i] - dot * wd[x][2 * i], qd[x][2 * i + 1] - dot * wd[x][2 * i + 1], hi[i], lo[i]);
          if constexpr (ZS) {  // (read back by the same lane only)
            s_z[threadIdx.x >> 5][(2 * q) * KB + x][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            s_z[threadIdx.x >> 5][(2 * q + 1) * KB + x][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) { zh[q][x][i] = hi[i]; zl[q][x][i] = lo[i]; }
          }
        }
        // the new token's own score, at the lanes of its column
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float s = __shfl_sync(0xffffffffu, self, (2 * t + e) * 4);
          st.m[q][e] = u == s0 ? s : -INFINITY;
          st.l[q][e] = u == s0 && g == 0 ? 1.f : 0.f;
        }
      }
#pragma unroll
      for (int x = 0; x < CS; ++x) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (u == s0) r = ld16((const __nv_bfloat16*)p.v + tok * D + 64 * x + 8 * g);
        const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 0; q < NQ8; ++q) {
            st.acc[q][4 * x + i][0] = st.acc[q][4 * x + i][1] = lo_f(rr[i]);
            st.acc[q][4 * x + i][2] = st.acc[q][4 * x + i][3] = hi_f(rr[i]);
          }
      }
      if (u == s0) {  // the new row joins the cache
        const long long kr = pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, sp.t0);
        const long long vr = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0);
        if (lane < D / 8) {
          *reinterpret_cast<uint4*>((__nv_bfloat16*)p.c.k_pool + kr * D + lane * 8) = ld16((const __nv_bfloat16*)p.k + tok * D + lane * 8);
          *reinterpret_cast<uint4*>((__nv_bfloat16*)p.c.v_pool + vr * D + lane * 8) = ld16((const __nv_bfloat16*)p.v + tok * D + lane * 8);
        }
        if (FOX) {
          const float rest = __shfl_sync(0xffffffffu, last, 2);
          if (lane == 0) store_sum(p.c, vr, (double)last + rest + p.log_f[tok]);
        }
      }
      if (FOX && t >= 2) last += p.log_f[tok];  // the one token's bias
    } else {
      const size_t item = (size_t)b * H + h;
      frag = (const uint32_t*)(ws + w.frag) + item * 32 * frag_words<D, NQ8>();
      // the item's first run starts from the new tokens' own state
#pragma unroll
      for (int q = 0; q < NQ8; ++q) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const size_t at = item * w.nq + 8 * q + 2 * t + e;
          st.m[q][e] = u == s0 ? ((const float*)(ws + w.sm))[at] : -INFINITY;
          st.l[q][e] = u == s0 && g == 0 ? ((const float*)(ws + w.sl))[at] : 0.f;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            float2 v = make_float2(0.f, 0.f);
            if (u == s0)
              v = *reinterpret_cast<const float2*>((const float*)(ws + w.sacc) + at * D + 64 * (j / 4) + 8 * g + 2 * (j % 4));
            st.acc[q][j][e] = v.x;
            st.acc[q][j][2 + e] = v.y;
          }
        }
      }
    }

    // ---- the cached tiles ----
    const int i0 = u - s0, i1 = lt.count > 0 ? ue - s0 : i0;  // (no cached rows: nothing to stream)
    uint4 kr[2][KB], vr[4][CS];
    float aj = 0.f;  // this lane's part of the tile's sums
    auto page = [&](const int* table, int i) { return table[(size_t)b * p.c.table_width + newest_tile(lt, i) * RT / P]; };
    int kp = -1, vp = -1, kpn = -1, vpn = -1;  // pages of the current and the next tile
    long long krow = 0, vrow = 0;
    auto rows_of = [&](int i, int pk, int pv, long long& rk, long long& rv) {
      const int in = newest_tile(lt, i) * RT % P;
      rk = ((long long)pk * H + h) * P + in;
      rv = ((long long)pv * H + h) * P + in;
    };
    auto good = [&](int pk, int pv) { return (unsigned)pk < (unsigned)p.c.k_pages && (unsigned)pv < (unsigned)p.c.v_pages; };
    auto load_k = [&](long long r) {
      const __nv_bfloat16* at = kpool + r * D + 8 * t;
#pragma unroll
      for (int x = 0; x < KB; ++x) {
        kr[0][x] = ld16(at + (size_t)g * D + 32 * x);
        kr[1][x] = ld16(at + (size_t)(g + 8) * D + 32 * x);
      }
    };
    auto load_v = [&](long long r) {
      const __nv_bfloat16* at = vpool + r * D + 8 * g;
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < CS; ++x) vr[y][x] = ld16(at + (size_t)(2 * t + (y & 1) + 8 * (y >> 1)) * D + 64 * x);
    };
    auto load_a = [&](long long r) {
      if (FOX && sums) aj = sums[r + g + 8 * (t & 1)];
    };
    bool ok = false;
    if (i0 < i1) {
      kp = page(p.c.k_table, i0);
      vp = page(p.c.v_table, i0);
      ok = good(kp, vp);
      if (ok) {
        rows_of(i0, kp, vp, krow, vrow);
        load_k(krow);
        load_a(vrow);
        load_v(vrow);
      }
      if (i0 + 1 < i1) {
        kpn = page(p.c.k_table, i0 + 1);
        vpn = page(p.c.v_table, i0 + 1);
      }
    }
    for (int i = i0; i < i1; ++i) {
      const int j0 = newest_tile(lt, i) * RT;
      const bool cur = ok;
      if (!cur && lane == 0) paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
      float s[NQ8][4], c[ONE ? 1 : NT8][4];
      // whole: every row of the tile is there, seen by every token and kept
      const bool whole = j0 + RT <= sp.t0 && (p.window <= 0 || j0 > sp.t0 + n - p.window || j0 + RT <= p.sinks);
      const long long kat = krow;
      if (cur) {
        // scores and rewriting coefficients; the A fragments are the loaded pieces
#pragma unroll
        for (int q = 0; q < NQ8; ++q) s[q][0] = s[q][1] = s[q][2] = s[q][3] = 0.f;
#pragma unroll
        for (int q = 0; q < (ONE ? 1 : NT8); ++q) c[q][0] = c[q][1] = c[q][2] = c[q][3] = 0.f;
#pragma unroll
        for (int x = 0; x < KB; ++x) {
          const uint32_t r0[4] = {kr[0][x].x, kr[0][x].y, kr[0][x].z, kr[0][x].w};
          const uint32_t r1[4] = {kr[1][x].x, kr[1][x].y, kr[1][x].z, kr[1][x].w};
          uint4 zq[ZS ? NQ8 : 1][2];
          if constexpr (ZS) {
#pragma unroll
            for (int q = 0; q < NQ8; ++q) {
              zq[q][0] = s_z[threadIdx.x >> 5][(2 * q) * KB + x][lane];
              zq[q][1] = s_z[threadIdx.x >> 5][(2 * q + 1) * KB + x][lane];
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t a0 = r0[2 * y], a1 = r1[2 * y], a2 = r0[2 * y + 1], a3 = r1[2 * y + 1];
            if constexpr (ONE) {
#pragma unroll
              for (int q = 0; q < NQ8; ++q) {
                if constexpr (ZS) {
                  mma_bf16(s[q], a0, a1, a2, a3, y ? zq[q][0].z : zq[q][0].x, y ? zq[q][0].w : zq[q][0].y);
                  mma_bf16(s[q], a0, a1, a2, a3, y ? zq[q][1].z : zq[q][1].x, y ? zq[q][1].w : zq[q][1].y);
                } else {
                  mma_bf16(s[q], a0, a1, a2, a3, zh[q][x][2 * y], zh[q][x][2 * y + 1]);
                  mma_bf16(s[q], a0, a1, a2, a3, zl[q][x][2 * y], zl[q][x][2 * y + 1]);
                }
              }
              const uint32_t b0 = g == 0 ? wf[x][2 * y] : 0u, b1 = g == 0 ? wf[x][2 * y + 1] : 0u;
              mma_bf16(c[0], a0, a1, a2, a3, b0, b1);
            } else {
              // words of a fragment: [z: column tile][high, rest][W: token tile], pairs (b0, b1) per (x, y)
              const uint2* f = reinterpret_cast<const uint2*>(frag) + lane;
              const int k = 2 * x + y;
#pragma unroll
              for (int q = 0; q < NQ8; ++q) {
                const uint2 zhv = f[((2 * q) * (D / 16) + k) * 32], zlv = f[((2 * q + 1) * (D / 16) + k) * 32];
                mma_bf16(s[q], a0, a1, a2, a3, zhv.x, zhv.y);
                mma_bf16(s[q], a0, a1, a2, a3, zlv.x, zlv.y);
              }
#pragma unroll
              for (int q = 0; q < NT8; ++q) {
                const uint2 wv = f[((2 * NQ8 + q) * (D / 16) + k) * 32];
                mma_bf16(c[q], a0, a1, a2, a3, wv.x, wv.y);
              }
            }
          }
        }
        // k <- k - c Y, stored where it came from
        bool keep0 = true, keep1 = true;
        if (!whole) {
          keep0 = j0 + g < sp.t0 && sees(p.window, p.sinks, sp.t0 + n, j0 + g);
          keep1 = j0 + g + 8 < sp.t0 && sees(p.window, p.sinks, sp.t0 + n, j0 + g + 8);
        }
        __nv_bfloat16* dst = (__nv_bfloat16*)p.c.k_pool + kat * D + 8 * t;
        if constexpr (ONE) {
          const float c0 = -beta * __shfl_sync(0xffffffffu, c[0][0], lane & 28), c1 = -beta * __shfl_sync(0xffffffffu, c[0][2], lane & 28);
#pragma unroll
          for (int x = 0; x < KB; ++x) {
            uint32_t r0[4] = {kr[0][x].x, kr[0][x].y, kr[0][x].z, kr[0][x].w};
            uint32_t r1[4] = {kr[1][x].x, kr[1][x].y, kr[1][x].z, kr[1][x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float wl = lo_f(wf[x][y]), wh = hi_f(wf[x][y]);
              r0[y] = pack2(fmaf(c0, wl, lo_f(r0[y])), fmaf(c0, wh, hi_f(r0[y])));
              r1[y] = pack2(fmaf(c1, wl, lo_f(r1[y])), fmaf(c1, wh, hi_f(r1[y])));
            }
            if (keep0) *reinterpret_cast<uint4*>(dst + (size_t)g * D + 32 * x) = make_uint4(r0[0], r0[1], r0[2], r0[3]);
            if (keep1) *reinterpret_cast<uint4*>(dst + (size_t)(g + 8) * D + 32 * x) = make_uint4(r1[0], r1[1], r1[2], r1[3]);
          }
        } else {
          // c as A fragments.  16 tokens: high and rest apart, c Y = ch Yh + cl Yh + ch Yl.  8 tokens: the 16
          // columns are high and rest, against Yh twice, and high again against Yl
          uint32_t ah[4], al[4];
          split2(c[0][0], c[0][1], ah[0], al[0]);
          split2(c[0][2], c[0][3], ah[1], al[1]);
          if constexpr (NT8 == 2) {
            split2(c[1][0], c[1][1], ah[2], al[2]);
            split2(c[1][2], c[1][3], ah[3], al[3]);
          }
          const uint2* f = reinterpret_cast<const uint2*>(frag) + (2 * NQ8 + 2) * (D / 16) * 32 + lane;
#pragma unroll
          for (int x = 0; x < KB; ++x) {
            uint32_t r0[4] = {kr[0][x].x, kr[0][x].y, kr[0][x].z, kr[0][x].w};
            uint32_t r1[4] = {kr[1][x].x, kr[1][x].y, kr[1][x].z, kr[1][x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              float k4[4] = {lo_f(r0[y]), hi_f(r0[y]), lo_f(r1[y]), hi_f(r1[y])};
              const uint2 yh = f[(4 * x + y) * 32], yl = f[(D / 8 + 4 * x + y) * 32];  // -Y
              if constexpr (NT8 == 2) {
                mma_bf16(k4, ah[0], ah[1], ah[2], ah[3], yh.x, yh.y);
                mma_bf16(k4, al[0], al[1], al[2], al[3], yh.x, yh.y);
                mma_bf16(k4, ah[0], ah[1], ah[2], ah[3], yl.x, yl.y);
              } else {
                mma_bf16(k4, ah[0], ah[1], al[0], al[1], yh.x, yh.x);
                mma_bf16_k8(k4, ah[0], ah[1], yl.x);
              }
              r0[y] = pack2(k4[0], k4[1]);
              r1[y] = pack2(k4[2], k4[3]);
            }
            if (keep0) *reinterpret_cast<uint4*>(dst + (size_t)g * D + 32 * x) = make_uint4(r0[0], r0[1], r0[2], r0[3]);
            if (keep1) *reinterpret_cast<uint4*>(dst + (size_t)(g + 8) * D + 32 * x) = make_uint4(r1[0], r1[1], r1[2], r1[3]);
          }
        }
      }
      float bias0 = 0.f, bias1 = 0.f;  // a_last - a_j of rows g and g + 8, log2 units
      if (FOX && cur) {
        float x = last - aj;
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        const float y = __shfl_xor_sync(0xffffffffu, x, 1);
        bias0 = (t & 1 ? y : x) * kLog2e;
        bias1 = (t & 1 ? x : y) * kLog2e;
      }
      // the next tile's keys (and sums) set out as soon as this one's registers are free
      long long kn = 0, vn = 0;
      ok = i + 1 < i1 && good(kpn, vpn);
      if (ok) {
        rows_of(i + 1, kpn, vpn, kn, vn);
        load_k(kn);
        load_a(vn);
      }
      krow = kn;
      const long long vnext = vn;
      if (i + 2 < i1) {
        kpn = page(p.c.k_table, i + 2);
        vpn = page(p.c.v_table, i + 2);
      }
      if (cur) {
        bool up = false;
#pragma unroll
        for (int q = 0; q < NQ8; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[q][e] * p.scl;
            if (FOX) x += (e < 2 ? bias0 : bias1) + (ONE ? 0.f : cb[q][e & 1]);
            if (!whole) {
              const int j = j0 + g + (e < 2 ? 0 : 8);
              if (j >= sp.t0 || !sees(p.window, p.sinks, cp[q][e & 1], j)) x = -INFINITY;
            }
            s[q][e] = x;
            up |= x > st.m[q][e & 1] + kTau;
          }
        if (!whole) {  // rows behind the sequence may hold anything: 0 times that has to be 0
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (j0 + 2 * t + (y & 1) + 8 * (y >> 1) >= sp.t0) {
#pragma unroll
              for (int x = 0; x < CS; ++x) vr[y][x] = make_uint4(0, 0, 0, 0);
            }
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int q = 0; q < NQ8; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(s[q][e], s[q][e + 2]);
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              const float mo = st.m[q][e], mn = fmaxf(mo, x);
              const float f = mn == -INFINITY ? 1.f : fast_exp2(mo - mn);
              st.m[q][e] = mn;
              st.l[q][e] *= f;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                st.acc[q][j][e] *= f;
                st.acc[q][j][e + 2] *= f;
              }
            }
        }
        // probabilities as B fragments of V^T P^T: keys become the rows
        uint32_t ph[NQ8][2], pl[NQ8][2];
#pragma unroll
        for (int q = 0; q < NQ8; ++q) {
          const float m0 = st.m[q][0] == -INFINITY ? 0.f : st.m[q][0], m1 = st.m[q][1] == -INFINITY ? 0.f : st.m[q][1];
          const float p0 = fast_exp2(s[q][0] - m0), p1 = fast_exp2(s[q][1] - m1);
          const float p2 = fast_exp2(s[q][2] - m0), p3 = fast_exp2(s[q][3] - m1);
          st.l[q][0] += p0 + p2;
          st.l[q][1] += p1 + p3;
          uint32_t h0, h1, l0, l1;
          split2(p0, p1, h0, l0);
          split2(p2, p3, h1, l1);
          ph[q][0] = transpose8(h0);
          ph[q][1] = transpose8(h1);
          pl[q][0] = transpose8(l0);
          pl[q][1] = transpose8(l1);
        }
#pragma unroll
        for (int x = 0; x < CS; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            auto word = [&](int k) { return y == 0 ? vr[k][x].x : y == 1 ? vr[k][x].y : y == 2 ? vr[k][x].z : vr[k][x].w; };
            const uint32_t a0 = __byte_perm(word(0), word(1), 0x5410), a1 = __byte_perm(word(0), word(1), 0x7632);
            const uint32_t a2 = __byte_perm(word(2), word(3), 0x5410), a3 = __byte_perm(word(2), word(3), 0x7632);
#pragma unroll
            for (int q = 0; q < NQ8; ++q) {
              mma_bf16(st.acc[q][4 * x + y], a0, a1, a2, a3, ph[q][0], ph[q][1]);
              mma_bf16(st.acc[q][4 * x + y], a0, a1, a2, a3, pl[q][0], pl[q][1]);
            }
          }
      }
      if (ok) load_v(vnext);
    }

    // ---- the item's end or the run's: output, or a partial state ----
    const bool complete = u == s0 && ue == e0;
    const size_t slot = ((size_t)2 * warp + (u0 >= s0 - kSetup ? 0 : 1)) * w.nq;  // the run's first item, or its last
#pragma unroll
    for (int q = 0; q < NQ8; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[q][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int col = 8 * q + 2 * t + e;
        if (col >= cols) continue;
        if (complete) {
          const float inv = 1.f / l;
          __nv_bfloat16* o = (__nv_bfloat16*)p.o + (((size_t)sp.q0 + col / G) * p.hq + h * G + col % G) * D + 8 * g;
#pragma unroll
          for (int x = 0; x < CS; ++x) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = pack2(st.acc[q][4 * x + i][e] * inv, st.acc[q][4 * x + i][2 + e] * inv);
            *reinterpret_cast<uint4*>(o + 64 * x) = make_uint4(r[0], r[1], r[2], r[3]);
          }
        } else {
          if (g == 0) {
            ((float*)(ws + w.m))[slot + col] = st.m[q][e];
            ((float*)(ws + w.l))[slot + col] = l;
          }
          float* a = (float*)(ws + w.acc) + (slot + col) * D + 8 * g;
#pragma unroll
          for (int x = 0; x < CS; ++x) {
            *reinterpret_cast<float4*>(a + 64 * x) = make_float4(st.acc[q][4 * x][e], st.acc[q][4 * x][2 + e],
                                                                 st.acc[q][4 * x + 1][e], st.acc[q][4 * x + 1][2 + e]);
            *reinterpret_cast<float4*>(a + 64 * x + 4) = make_float4(st.acc[q][4 * x + 2][e], st.acc[q][4 * x + 2][2 + e],
                                                                     st.acc[q][4 * x + 3][e], st.acc[q][4 * x + 3][2 + e]);
          }
        }
      }
    u = ue;
  }
  if (ONE && p.c.slots <= kSmemSlots) keep_starts(start, p.c.slots, (int*)(ws + w.ustart));
}

// ---- draft tokens: the n <= 16 new tokens of a (slot, head) among themselves ----
// One block each; a few thousand multiply-adds in fp32.  Writes what the streaming warps hold in registers (z, W, -Y
// in the lane order of their B fragments), the new tokens' own softmax state, and the appended rows.
constexpr int DT = 512, DN = 16;  // (128 threads: 19 us for 8 tokens of 16 x 8 slots and heads)
template <int D>
struct DraftSmem {
  float w[DN][D + 4], k[DN][D + 4], v[DN][D + 4], y[DN][D + 4];
  float q[32][D + 4];
  float g[DN][DN + 1], n[DN][DN + 1], u[DN][DN + 1], x[DN][DN + 1];
  float m1[32][DN + 1], a[32][DN + 1], s[32][DN + 1];
  float beta[DN], lf[DN];
  long long kr[DN], vr[DN];  // the appended rows' places
};
template <int D, bool FOX>
__global__ void __launch_bounds__(DT) draft_prep_kernel(PagedArgs p, TokenWs w, char* ws) {
  chain();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  DraftSmem<D>& sm = *reinterpret_cast<DraftSmem<D>*>(smem_raw);
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, H = p.c.heads, G = p.G;
  const SlotSpan sp = slot_span(p, b);
  if (sp.n == 0) return;
  const int n = sp.n, cols = n * G;
  const __nv_bfloat16 *gq = (const __nv_bfloat16*)p.q, *gk = (const __nv_bfloat16*)p.k;
  const __nv_bfloat16 *gv = (const __nv_bfloat16*)p.v, *gw = (const __nv_bfloat16*)p.w;
  auto row8 = [&](float* dst, const __nv_bfloat16* src) {
    const uint4 r = ld16(src);
    const uint32_t rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dst[2 * i] = lo_f(rr[i]);
      dst[2 * i + 1] = hi_f(rr[i]);
    }
  };
  for (int e = tid; e < DN * (D / 8); e += DT) {
    const int r = e / (D / 8), x = e % (D / 8) * 8;
    if (r < n) {
      const size_t at = (((size_t)sp.q0 + r) * H + h) * D + x;
      row8(&sm.w[r][x], gw + at);
      row8(&sm.k[r][x], gk + at);
      row8(&sm.v[r][x], gv + at);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) sm.w[r][x + i] = sm.k[r][x + i] = sm.v[r][x + i] = 0.f;
    }
  }
  for (int e = tid; e < cols * (D / 8); e += DT) {
    const int r = e / (D / 8), x = e % (D / 8) * 8;
    row8(&sm.q[r][x], gq + (((size_t)sp.q0 + r / G) * p.hq + h * G + r % G) * D + x);
  }
  if (tid < DN) {
    sm.beta[tid] = tid < n ? clamp_beta(p.beta[((size_t)sp.q0 + tid) * H + h]) : 0.f;
    float a = 0.f;
    if (FOX)
      for (int i = 0; i <= tid && i < n; ++i) a += p.log_f[((size_t)sp.q0 + i) * H + h];
    sm.lf[tid] = a;
    if (tid < n) {
      sm.kr[tid] = pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, sp.t0 + tid);
      sm.vr[tid] = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 + tid);
    }
  }
  if (__syncthreads_or(tid < n && (sm.kr[tid] < 0 || sm.vr[tid] < 0))) return;  // left out, which the streaming pass reports
  auto dot = [](const float* a, const float* c) {
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll 8
    for (int i = 0; i < D; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(a + i), y = *reinterpret_cast<const float4*>(c + i);
      s0 = fmaf(x.x, y.x, s0);
      s1 = fmaf(x.y, y.y, s1);
      s2 = fmaf(x.z, y.z, s2);
      s3 = fmaf(x.w, y.w, s3);
    }
    return (s0 + s1) + (s2 + s3);
  };
  const int n2 = n * n;
  for (int e = tid; e < 2 * (n2 + cols * n); e += DT) {  // the four kinds of products of rows
    if (e < n2) {
      const int i = e / n, j = e % n;
      sm.g[i][j] = j < i ? dot(sm.w[i], sm.w[j]) : 0.f;
    } else if (e < 2 * n2) {
      const int i = (e - n2) / n, j = (e - n2) % n;
      sm.n[i][j] = j < i ? dot(sm.w[i], sm.k[j]) : 0.f;
    } else {
      const int r = e - 2 * n2, which = r / (cols * n), c = r % (cols * n) / n, j = r % n;
      const bool in = j <= c / G;
      if (which == 0) sm.m1[c][j] = in ? dot(sm.q[c], sm.w[j]) : 0.f;
      else sm.s[c][j] = in ? dot(sm.q[c], sm.k[j]) : 0.f;
    }
  }
  __syncthreads();
  if (tid < DN) {  // U, one column per lane
    for (int i = 0; i < n; ++i) {
      float a = tid == i ? 1.f : 0.f;
      for (int m = tid; m < i; ++m) a -= sm.g[i][m] * sm.u[m][tid];
      sm.u[i][tid] = tid <= i ? sm.beta[i] * a : 0.f;
    }
  }
  __syncthreads();
  for (int e = tid; e < n2 + cols * n; e += DT) {
    if (e < n2) {
      const int i = e / n, j = e % n;
      float a = 0.f;
      for (int m = j + 1; m <= i; ++m) a += sm.u[i][m] * sm.n[m][j];
      sm.x[i][j] = a;
    } else {
      const int c = (e - n2) / n, j = (e - n2) % n;
      float a = 0.f;
      for (int m = j; m < n; ++m) a += sm.m1[c][m] * sm.u[m][j];
      sm.a[c][j] = a;
    }
  }
  __syncthreads();
  const size_t item = (size_t)b * H + h;
  // scores of the new tokens among themselves and their softmax: 4 lanes per column
  {
    const int c = tid >> 2, sub = tid & 3;
    const int i = c < cols ? c / G : 0;
    float s[4], mx = -INFINITY;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = sub + 4 * x;
      s[x] = -INFINITY;
      if (c < cols && j <= i && sees(p.window, p.sinks, sp.t0 + i, sp.t0 + j)) {
        float v = sm.s[c][j];
        for (int m = j + 1; m <= i; ++m) v -= sm.a[c][m] * sm.n[m][j];
        s[x] = v * p.scl + (FOX ? (sm.lf[i] - sm.lf[j]) * kLog2e : 0.f);
      }
      mx = fmaxf(mx, s[x]);
    }
    mx = group_max<4>(mx);
    float l = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float e = s[x] == -INFINITY ? 0.f : fast_exp2(s[x] - mx);
      l += e;
      s[x] = e;
    }
    l = group_sum<4>(l);
    __syncthreads();
    if (c < cols) {
#pragma unroll
      for (int x = 0; x < 4; ++x) sm.s[c][sub + 4 * x] = s[x];
      if (sub == 0) {
        ((float*)(ws + w.sm))[item * w.nq + c] = mx;
        ((float*)(ws + w.sl))[item * w.nq + c] = l;
      }
    }
  }
  // Y = U^T W; z = q - A W over q; the appended keys k - X^T W
  for (int e = tid; e < DN * D; e += DT) {
    const int r = e / D, x = e % D;
    float y = 0.f;
    for (int m = r; m < n; ++m) y += sm.u[m][r] * sm.w[m][x];
    sm.y[r][x] = r < n ? y : 0.f;
    if (r < n) {
      float kx = sm.k[r][x];
      for (int m = r + 1; m < n; ++m) kx -= sm.x[m][r] * sm.w[m][x];
      const long long kr = sm.kr[r], vr = sm.vr[r];
      ((__nv_bfloat16*)p.c.k_pool)[kr * D + x] = __float2bfloat16_rn(kx);
      ((__nv_bfloat16*)p.c.v_pool)[vr * D + x] = __float2bfloat16_rn(sm.v[r][x]);
      if (FOX && x == 0) {
        const long long last = sp.t0 > 0 ? pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 - 1) : -1;
        store_sum(p.c, vr, (last >= 0 ? load_sum(p.c, last) : 0.0) + sm.lf[r]);
      }
    }
  }
  for (int e = tid; e < cols * D; e += DT) {
    const int c = e / D, x = e % D;
    float z = sm.q[c][x];
    for (int m = 0; m <= c / G; ++m) z -= sm.a[c][m] * sm.w[m][x];
    sm.q[c][x] = z;
  }
  __syncthreads();
  float* sacc = (float*)(ws + w.sacc) + item * w.nq * D;
  for (int e = tid; e < w.nq * D; e += DT) {
    const int c = e / D, x = e % D;
    float a = 0.f;
    if (c < cols)
      for (int j = 0; j <= c / G; ++j) a += sm.s[c][j] * sm.v[j][x];
    sacc[e] = a;
  }
  if (tid < w.nq && tid >= cols) {  // columns without a query
    ((float*)(ws + w.sm))[item * w.nq + tid] = -INFINITY;
    ((float*)(ws + w.sl))[item * w.nq + tid] = 0.f;
  }
  // fragments
  const int nq8 = w.nq / 8, words = nq8 * (D / 8) * 2 + 2 * (D / 8) + 2 * (D / 8) * 2;
  uint2* f = reinterpret_cast<uint2*>((uint32_t*)(ws + w.frag) + item * 32 * words);
  const int lane = tid & 31, g = lane >> 2, t = lane & 3;
  for (int k = tid >> 5; k < (nq8 + 2) * (D / 16); k += DT / 32) {
    const int q = k / (D / 16), y = k % (D / 16), d0 = 32 * (y >> 1) + 8 * t + 4 * (y & 1);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (q < nq8) {
      const int c = 8 * q + g;
      if (c < cols)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = sm.q[c][d0 + i];
      uint2 hi, lo;
      split2(v[0], v[1], hi.x, lo.x);
      split2(v[2], v[3], hi.y, lo.y);
      f[((2 * q) * (D / 16) + y) * 32 + lane] = hi;
      f[((2 * q + 1) * (D / 16) + y) * 32 + lane] = lo;
    } else {
      const int r = 8 * (q - nq8) + g;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = sm.w[r][d0 + i];
      f[((2 * nq8 + q - nq8) * (D / 16) + y) * 32 + lane] = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    }
  }
  f += (2 * nq8 + 2) * (D / 16) * 32;
  for (int k = tid >> 5; k < D / 8; k += DT / 32) {
    const int d = 32 * (k >> 2) + 8 * (g >> 1) + 2 * (k & 3) + (g & 1);
    uint2 hi, lo;
    split2(-sm.y[2 * t][d], -sm.y[2 * t + 1][d], hi.x, lo.x);
    split2(-sm.y[2 * t + 8][d], -sm.y[2 * t + 9][d], hi.y, lo.y);
    f[k * 32 + lane] = hi;
    f[(D / 8 + k) * 32 + lane] = lo;
  }
}

// Merge of the partial states: one block per (slot, head, cs query columns).  D / 4 lanes share a column; groups of
// lanes take the columns and, where these are few, share the runs of a column; sums in a fixed order.
constexpr int MT = 256;
constexpr int merge_columns(int D, int cols) {  // a power of two, at most the groups of a block
  int cs = 1;
  while (cs < cols && cs < MT / (D / 4) / 4) cs *= 2;
  return cs;
}
template <typename T, int D>
__global__ void __launch_bounds__(MT) token_merge_kernel(PagedArgs p, TokenWs w, const char* ws, int mode, int warps,
                                                         int cs) {
  chain();
  constexpr int L = D / 4, GR = MT / L;
  __shared__ float4 s_acc[GR][L];
  __shared__ float s_l[GR];
  const int b = blockIdx.x, h = blockIdx.y, gr = threadIdx.x / L, x = threadIdx.x % L;
  const SlotSpan sp = slot_span(p, b);
  const int cols = sp.n * p.G, c0 = blockIdx.z * cs;
  if (sp.n == 0 || (mode == kOnlyOne && sp.n != 1) || c0 >= cols) return;
  const int* start = (const int*)(ws + w.ustart);
  if (start[b + 1] == start[b]) return;  // left out
  const int run = run_length(start[p.c.slots], warps);
  const int kt = live_tiles(sp.t0, p.window, p.sinks, RT).count;
  const int each = kt > 0 ? kt : 1;
  const int s0 = start[b] + h * (kSetup + each) + kSetup, ra = s0 / run, n = (s0 + each - 1) / run - ra + 1;  // the item's runs
  if (n == 1) return;  // written by its run
  const float *gm = (const float*)(ws + w.m), *gl = (const float*)(ws + w.l), *ga = (const float*)(ws + w.acc);
  const int lead = ra * run >= s0 - kSetup ? 0 : 1;  // the place of the first run's part
  {
    const int col = c0 + gr % cs, pg = gr / cs, pn = GR / cs;
    auto at = [&](int r) { return ((size_t)2 * (ra + r) + (r == 0 ? lead : 0)) * w.nq + col; };
    float M = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < cols)
      for (int r = x; r < n; r += L) M = fmaxf(M, gm[at(r)]);
    M = group_max<L>(M);
    if (col < cols) {
#pragma unroll 4
      for (int r = pg; r < n; r += pn) {
        const float ms = gm[at(r)];
        const float f = ms == -INFINITY ? 0.f : fast_exp2(ms - M);
        const float4 v = *reinterpret_cast<const float4*>(ga + at(r) * D + 4 * x);
        l += gl[at(r)] * f;
        a.x += v.x * f;
        a.y += v.y * f;
        a.z += v.z * f;
        a.w += v.w * f;
      }
    }
    s_acc[gr][x] = a;
    if (x == 0) s_l[gr] = l;
    __syncthreads();
    if (pg == 0 && col < cols) {
      for (int y = 1; y < pn; ++y) {
        const float4 v = s_acc[gr + y * cs][x];
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
        l += s_l[gr + y * cs];
      }
      const float inv = 1.f / l;
      T* o = (T*)p.o + (((size_t)sp.q0 + col / p.G) * p.hq + h * p.G + col % p.G) * D + 4 * x;
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(o) = make_uint2(pack2(a.x * inv, a.y * inv), pack2(a.z * inv, a.w * inv));
      else *reinterpret_cast<float4*>(o) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    }
  }
}

// ---- one token per slot, fp32 caches ----
// The same runs of units on the CUDA cores (12 D bytes per cached row and head): D / 4 lanes share a row, 16 bytes each;
// z . k, w . k and the softmax in fp32.  GP: query heads per key head, rounded up to a power of two.
constexpr int blocks32(int D, int gp) { return gp <= 4 ? blocks_per_sm(D, 1) : 2; }
template <int D, int GP, bool FOX>
__global__ void __launch_bounds__(NT, blocks32(D, GP)) token32_kernel(PagedArgs p, TokenWs w, char* ws) {
  chain();
  __shared__ int s_start[kSmemSlots + 1];
  constexpr int L = D / 4, RW = 32 / L, AHEAD = 4;  // lanes of a row, rows side by side, row groups on the way
  const int lane = threadIdx.x & 31, x4 = lane % L * 4, grp = lane / L;
  const int warp = blockIdx.x * WARPS + (threadIdx.x >> 5), warps = gridDim.x * WARPS;
  const int H = p.c.heads, G = p.G, P = p.c.page_size;
  const int* start;
  if (p.c.slots <= kSmemSlots) {
    unit_starts<NT>(p, kOnlyOne, blockIdx.x == 0, s_start);
    start = s_start;
  } else {
    start = (const int*)(ws + w.ustart);
  }
  const int units = start[p.c.slots], run = run_length(units, warps);
  const int u0 = warp * run, u1 = min(u0 + run, units);
  auto ld4 = [](const float* q) { return *reinterpret_cast<const float4*>(q); };
  auto dot4 = [](const float4& a, const float4& c) { return a.x * c.x + a.y * c.y + a.z * c.z + a.w * c.w; };
  float *kpool = (float*)p.c.k_pool, *vpool = (float*)p.c.v_pool;
  int b = u0 < u1 ? find_slot(start, p.c.slots, u0) : 0;
  int u = u0;
  while (u < u1) {
    while (start[b + 1] <= u) ++b;
    const SlotSpan sp = slot_span(p, b);
    const LiveTiles lt = live_tiles(sp.t0, p.window, p.sinks, RT);
    const int per = kSetup + (lt.count > 0 ? lt.count : 1);
    const int h = (u - start[b]) / per;
    const int s0 = start[b] + h * per + kSetup, e0 = s0 + per - kSetup;
    if (u < s0) u = s0;
    if (u >= u1) break;
    const int ue = e0 < u1 ? e0 : u1;
    const bool head = u == s0;  // this run has the item's first unit: the new token itself
    const size_t tok = (size_t)sp.q0 * H + h;
    const float beta = clamp_beta(p.beta[tok]);
    const float4 wv = ld4((const float*)p.w + tok * D + x4), kv = ld4((const float*)p.k + tok * D + x4);
    const float4 vv = ld4((const float*)p.v + tok * D + x4);
    float a_last = 0.f, a_more = 0.f, lf = 0.f;
    if (FOX) {
      lf = p.log_f[tok];
      const long long r = sp.t0 > 0 ? pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 - 1) : -1;
      if (r >= 0) {
        a_last = p.c.a_pool[r];
        a_more = sum_rest(p.c, r);
      }
    }
    float4 z[GP], acc[GP];
    float m[GP], l[GP];
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      const float4 q = g < G ? ld4((const float*)p.q + ((size_t)sp.q0 * p.hq + h * G + g) * D + x4) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float c = beta * group_sum<L>(dot4(q, wv)), s = group_sum<L>(dot4(q, kv)) * p.scl;
      z[g] = make_float4(q.x - c * wv.x, q.y - c * wv.y, q.z - c * wv.z, q.w - c * wv.w);
      const bool mine = head && grp == 0;
      m[g] = mine ? s : -INFINITY;
      l[g] = mine ? 1.f : 0.f;
      acc[g] = mine ? vv : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (head) {
      const long long kr = pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, sp.t0);
      const long long vr = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0);
      if (grp == 0) {
        *reinterpret_cast<float4*>(kpool + kr * D + x4) = kv;
        *reinterpret_cast<float4*>(vpool + vr * D + x4) = vv;
      }
      if (FOX && lane == 0) store_sum(p.c, vr, (double)a_last + a_more + lf);
    }
    const int i0 = u - s0, i1 = lt.count > 0 ? ue - s0 : i0;
    for (int i = i0; i < i1; ++i) {
      const int j0 = newest_tile(lt, i) * RT;
      const int kp = p.c.k_table[(size_t)b * p.c.table_width + j0 / P];
      const int vp = p.c.v_table[(size_t)b * p.c.table_width + j0 / P];
      if ((unsigned)kp >= (unsigned)p.c.k_pages || (unsigned)vp >= (unsigned)p.c.v_pages) {
        if (lane == 0) paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
        continue;
      }
      float* krow = kpool + (((long long)kp * H + h) * P + j0 % P) * D + x4;
      const long long vr0 = ((long long)vp * H + h) * P + j0 % P;
      const float* vrow = vpool + vr0 * D + x4;
#pragma unroll 1
      for (int r0 = 0; r0 < RT; r0 += AHEAD * RW) {
        float4 kk[AHEAD], va[AHEAD];
        float bias[AHEAD];  // a_last - a_j
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
          const int r = r0 + e * RW + grp;
          kk[e] = ld4(krow + (size_t)r * D);
          va[e] = ld4(vrow + (size_t)r * D);
          bias[e] = FOX ? (a_last - p.c.a_pool[vr0 + r]) + (a_more - sum_rest(p.c, vr0 + r)) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
          const int r = r0 + e * RW + grp, j = j0 + r;
          const float c = beta * group_sum<L>(dot4(kk[e], wv));
          float s[GP];
#pragma unroll
          for (int g = 0; g < GP; ++g) s[g] = group_sum<L>(dot4(kk[e], z[g])) * p.scl;
          if (j < sp.t0 && sees(p.window, p.sinks, sp.t0 + 1, j))
            *reinterpret_cast<float4*>(krow + (size_t)r * D) =
                make_float4(kk[e].x - c * wv.x, kk[e].y - c * wv.y, kk[e].z - c * wv.z, kk[e].w - c * wv.w);
          if (j < sp.t0 && sees(p.window, p.sinks, sp.t0, j)) {  // (uniform in the row's lanes)
#pragma unroll
            for (int g = 0; g < GP; ++g) {
              const float v = FOX ? s[g] + (bias[e] + lf) * kLog2e : s[g], mn = fmaxf(m[g], v);
              const float f = fast_exp2(m[g] - mn), pr = fast_exp2(v - mn);
              m[g] = mn;
              l[g] = l[g] * f + pr;
              acc[g] = make_float4(acc[g].x * f + pr * va[e].x, acc[g].y * f + pr * va[e].y, acc[g].z * f + pr * va[e].z,
                                   acc[g].w * f + pr * va[e].w);
            }
          }
        }
      }
    }
    const bool complete = head && ue == e0;
    const size_t slot = ((size_t)2 * warp + (u0 >= s0 - kSetup ? 0 : 1)) * w.nq;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      if (RW == 2) {  // the two rows' states
        const float mo = __shfl_xor_sync(0xffffffffu, m[g], 16), M = fmaxf(m[g], mo);
        const float f = m[g] == -INFINITY ? 0.f : fast_exp2(m[g] - M);
        l[g] *= f;
        acc[g] = make_float4(acc[g].x * f, acc[g].y * f, acc[g].z * f, acc[g].w * f);
        m[g] = M;
        l[g] += __shfl_xor_sync(0xffffffffu, l[g], 16);
        acc[g].x += __shfl_xor_sync(0xffffffffu, acc[g].x, 16);
        acc[g].y += __shfl_xor_sync(0xffffffffu, acc[g].y, 16);
        acc[g].z += __shfl_xor_sync(0xffffffffu, acc[g].z, 16);
        acc[g].w += __shfl_xor_sync(0xffffffffu, acc[g].w, 16);
      }
      if (g >= G || grp != 0) continue;
      if (complete) {
        const float inv = 1.f / l[g];
        *reinterpret_cast<float4*>((float*)p.o + ((size_t)sp.q0 * p.hq + h * G + g) * D + x4) =
            make_float4(acc[g].x * inv, acc[g].y * inv, acc[g].z * inv, acc[g].w * inv);
      } else {
        if (x4 == 0) {
          ((float*)(ws + w.m))[slot + g] = m[g];
          ((float*)(ws + w.l))[slot + g] = l[g];
        }
        *reinterpret_cast<float4*>((float*)(ws + w.acc) + (slot + g) * D + x4) = acc[g];
      }
    }
    u = ue;
  }
  if (p.c.slots <= kSmemSlots) keep_starts(start, p.c.slots, (int*)(ws + w.ustart));
}
template <int D, int GP, bool FOX>
cudaError_t token32_t(const PagedArgs& p, const TokenWs& w, char* ws, cudaStream_t st) {
  cudaError_t e;
  if (p.c.slots > kSmemSlots &&
      (e = launch_chained(unit_starts_kernel, 1, 1024, 0, st, p, (int)kOnlyOne, (int*)(ws + w.ustart))) != cudaSuccess)
    return e;
  const int blocks = w.blocks < 152 * blocks32(D, GP) ? w.blocks : 152 * blocks32(D, GP);
  if ((e = launch_chained(token32_kernel<D, GP, FOX>, blocks, NT, 0, st, p, w, ws)) != cudaSuccess) return e;
  const int cs = merge_columns(D, p.G);
  return launch_chained(token_merge_kernel<float, D>, dim3(p.c.slots, p.c.heads, (p.G + cs - 1) / cs), MT, 0, st, p, w, ws,
                        (int)kOnlyOne, blocks * WARPS, cs);
}
template <int D, bool FOX>
cudaError_t token32_d(const PagedArgs& p, const TokenWs& w, char* ws, cudaStream_t st) {
  if (p.G == 1) return token32_t<D, 1, FOX>(p, w, ws, st);
  if (p.G == 2) return token32_t<D, 2, FOX>(p, w, ws, st);
  if (p.G <= 4) return token32_t<D, 4, FOX>(p, w, ws, st);
  if (p.G <= 8) return token32_t<D, 8, FOX>(p, w, ws, st);
  return token32_t<D, 16, FOX>(p, w, ws, st);
}

template <int D, int NQ8, int NT8, bool FOX>
cudaError_t token_t(const PagedArgs& p, const TokenWs& w, char* ws, cudaStream_t st) {
  constexpr bool ONE = NT8 == 0;
  const int mode = ONE ? kOnlyOne : kDrafts;
  cudaError_t e;
  if (p.c.slots > kSmemSlots &&
      (e = launch_chained(unit_starts_kernel, 1, 1024, 0, st, p, mode, (int*)(ws + w.ustart))) != cudaSuccess)
    return e;
  if (!ONE) {
    auto prep = draft_prep_kernel<D, FOX>;
    if ((e = cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(DraftSmem<D>))) != cudaSuccess ||
        (e = launch_chained(prep, dim3(p.c.slots, p.c.heads), DT, sizeof(DraftSmem<D>), st, p, w, ws)) != cudaSuccess)
      return e;
  }
  if ((e = launch_chained(token_kernel<D, NQ8, NT8, FOX>, w.blocks, NT, 0, st, p, w, ws)) != cudaSuccess) return e;
  const int cols = (ONE ? 1 : p.max_new) * p.G, cs = merge_columns(D, cols);
  return launch_chained(token_merge_kernel<__nv_bfloat16, D>, dim3(p.c.slots, p.c.heads, (cols + cs - 1) / cs), MT, 0, st, p, w, ws, mode,
                        w.blocks * WARPS, cs);
}
template <int D, bool FOX>
cudaError_t token_d(const PagedArgs& p, const TokenWs& w, bool drafts, char* ws, cudaStream_t st) {
  if (!drafts) return w.nq == 8 ? token_t<D, 1, 0, FOX>(p, w, ws, st) : token_t<D, 2, 0, FOX>(p, w, ws, st);
  if (p.max_new <= 8) {
    if (w.nq == 8) return token_t<D, 1, 1, FOX>(p, w, ws, st);
    if (w.nq == 16) return token_t<D, 2, 1, FOX>(p, w, ws, st);
    if constexpr (D == 64) return token_t<D, 4, 1, FOX>(p, w, ws, st);
  }
  return token_t<D, 2, 2, FOX>(p, w, ws, st);
}

}  // namespace

// Drafts go through the streaming pass while their columns' accumulators and fragments leave it fast enough: 16
// columns (8 heads x 16 x 2000..8192 rows, 8 tokens, G = 2: head dim 64 102 us against 137 for the prompt chunk path, 128
// 182 against 216), at head dim 64 up to 8 tokens also 32 (135 against 142).  Beyond that the chunk path's second
// pass over the keys costs less (32 columns, head dim 128: 337 against 227; 16 tokens, head dim 64: 153 against 138).  All of
// these figures are of that one batch; where the two paths meet at other lengths was not measured.
bool paged_drafts(const PagedArgs& p) {
  if (p.c.cache_dtype != PATH_BF16 || p.max_new <= 1 || p.max_new > DN) return false;
  const int cols = p.max_new * p.G;
  return cols <= 16 || (p.c.head_dim == kHeadDim && p.max_new <= 8 && cols <= 32);
}
size_t paged_token_ws_bytes(const PagedArgs& p) { return token_ws(p, paged_drafts(p) ? p.max_new : 1).total; }
cudaError_t launch_paged_token(const PagedArgs& p, char* ws, cudaStream_t st) {
  const bool drafts = paged_drafts(p), fox = p.log_f != nullptr;
  const TokenWs w = token_ws(p, drafts ? p.max_new : 1);
  if (p.c.cache_dtype != PATH_BF16) {
    if (p.c.head_dim == kHeadDim) return fox ? token32_d<kHeadDim, true>(p, w, ws, st) : token32_d<kHeadDim, false>(p, w, ws, st);
    return fox ? token32_d<kHeadDimWide, true>(p, w, ws, st) : token32_d<kHeadDimWide, false>(p, w, ws, st);
  }
  if (p.c.head_dim == kHeadDim)
    return fox ? token_d<kHeadDim, true>(p, w, drafts, ws, st) : token_d<kHeadDim, false>(p, w, drafts, ws, st);
  return fox ? token_d<kHeadDimWide, true>(p, w, drafts, ws, st) : token_d<kHeadDimWide, false>(p, w, drafts, ws, st);
}

}  // namespace pathattn
