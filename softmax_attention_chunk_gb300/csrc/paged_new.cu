// Paged serving of bf16 caches: prompt chunks (slots with more new tokens than the streaming kernels take).
//
// Mathematics (paged_chunk.cu has the formulas): the new tokens of a slot are cut into UT chunks of 64 and blocks
// of 256 (four chunks).  A chain over all earlier chunks per query tile would cost a D x D product per step;
// instead
//  * inside its block a query chunk meets the earlier chunks right to left (at most three steps) and arrives at the
//    block's start: zs, and the softmax state so far;
//  * the keys of a block are carried on: to the block's end, then through every later block,
//    rows <- rows F_block, and a copy is kept at each block start ("version").  For the queries of block b
//    the keys of all earlier blocks, in version b, are plain rows: attention without transport;
//  * rows of the identity carried the same way are the products G_b = F_0 ... F_(b-1), which move zs to the
//    start of the call (z = zs G_b^T, for the cached rows), and at the end M, by which the cached rows are
//    multiplied.
// So all attention but the 256-token diagonal runs in the tensor-core kernel (paged_tc.cu).
//
// Roundings: U W, F, the carried rows and M are held as bf16 pairs (high + rest, about 16 bits; products of three
// terms), and so are z and P within the block, so chains of chunks and blocks do not accumulate 8-bit rounding.  Rounded to bf16
// once, as tensor-core operands: the versions, X (it moves scores inside one chunk only), and z and P for the rows
// of earlier blocks and the cached ones as paged_tc.cu says.  Cached keys are exact as stored.
//
// These kernels are small next to the attention (2048 tokens, 32 heads, D = 128: about 15 of 1200 GFLOP) and bound
// by latency, so they run 16x8x16 warp MMAs on tiles in shared memory, one block per chunk, head and task.  At that
// size, over 32768 cached rows, one after the other: preparation 29 us, carrying in the block 29, queries with the
// carrying on beside them 125 (tensor pipe 41 %, 8 warps per SM), start 23, rewrite 28, merge 34, attention 726; their
// chained launches overlap to 1003 us for the call.  512 tokens x 32 heads over 8000 at D = 64: 20, 10, 30, 5, 20, 16 and 69.
#include "paged_tc.h"
#include "dev_common.cuh"
#include "mma_common.cuh"

namespace pathattn {
namespace {

constexpr int C = 64;            // UT chunk
constexpr int MB = kTcBlockTokens;  // tokens of a block: 256
constexpr int CPB = MB / C;      // chunks of a block

using bf16 = __nv_bfloat16;

// ---- warp tiles ----
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
}
// c[NT][4] (16 x 8 NT) += A (KS fragments of 16 columns) B; B in shared memory as [n][k] rows (T = false) or [k][n]
// rows (T = true) of ld elements.
template <int NT, int KS, bool T>
__device__ __forceinline__ void warp_mm(float (&c)[NT][4], const uint32_t (&a)[KS][4], const bf16* b, int ld) {
  const int lane = threadIdx.x & 31, mat = lane >> 3, row = lane & 7;
#pragma unroll
  for (int k = 0; k < KS; ++k)
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t r[4];
      if (T) ldm4t(r, b + (16 * k + (mat & 1) * 8 + row) * ld + 8 * n + (mat >> 1) * 8);
      else ldm4(r, b + (8 * n + (mat >> 1) * 8 + row) * ld + 16 * k + (mat & 1) * 8);
      mma_bf16(c[n], a[k][0], a[k][1], a[k][2], a[k][3], r[0], r[1]);
      mma_bf16(c[n + 1], a[k][0], a[k][1], a[k][2], a[k][3], r[2], r[3]);
    }
}
// The same with A a pair (high, rest): every fragment of B is fetched once for both.
template <int NT, int KS, bool T>
__device__ __forceinline__ void warp_mm2(float (&c)[NT][4], const uint32_t (&a)[KS][4], const uint32_t (&e)[KS][4], const bf16* b, int ld) {
  const int lane = threadIdx.x & 31, mat = lane >> 3, row = lane & 7;
#pragma unroll
  for (int k = 0; k < KS; ++k)
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t r[4];
      if (T) ldm4t(r, b + (16 * k + (mat & 1) * 8 + row) * ld + 8 * n + (mat >> 1) * 8);
      else ldm4(r, b + (8 * n + (mat >> 1) * 8 + row) * ld + 16 * k + (mat & 1) * 8);
      mma_bf16(c[n], a[k][0], a[k][1], a[k][2], a[k][3], r[0], r[1]);
      mma_bf16(c[n + 1], a[k][0], a[k][1], a[k][2], a[k][3], r[2], r[3]);
      mma_bf16(c[n], e[k][0], e[k][1], e[k][2], e[k][3], r[0], r[1]);
      mma_bf16(c[n + 1], e[k][0], e[k][1], e[k][2], e[k][3], r[2], r[3]);
    }
}
template <int KS>
__device__ __forceinline__ void load_a(uint32_t (&a)[KS][4], const bf16* t, int ld, int m0) {
  const int lane = threadIdx.x & 31, mat = lane >> 3, row = lane & 7;
#pragma unroll
  for (int k = 0; k < KS; ++k) ldm4(a[k], t + (m0 + (mat & 1) * 8 + row) * ld + 16 * k + (mat >> 1) * 8);
}
// Accumulators as A fragments, high + rest.
template <int KS>
__device__ __forceinline__ void to_a2(uint32_t (&hi)[KS][4], uint32_t (&lo)[KS][4], const float (&c)[2 * KS][4]) {
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    split2(c[2 * k][0], c[2 * k][1], hi[k][0], lo[k][0]);
    split2(c[2 * k][2], c[2 * k][3], hi[k][1], lo[k][1]);
    split2(c[2 * k + 1][0], c[2 * k + 1][1], hi[k][2], lo[k][2]);
    split2(c[2 * k + 1][2], c[2 * k + 1][3], hi[k][3], lo[k][3]);
  }
}
// rows x D bf16 from global (row pitch in elements) to shared memory, rows >= `have` zero; asynchronous.
template <int D, int LD, int THREADS>
__device__ __forceinline__ void fetch(bf16* dst, const bf16* src, size_t pitch, int rows, int have) {
  for (int e = threadIdx.x; e < rows * (D / 8); e += THREADS) {
    const int r = e / (D / 8), x = e % (D / 8) * 8;
    const bool ok = r < have;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + r * LD + x)),
                 "l"(src + (ok ? (size_t)r * pitch + x : 0)), "r"(ok ? 16 : 0)
                 : "memory");
  }
}
// Fetches so far form a group; all but the newest N groups have arrived.
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory"); }

// ---- workspace ----
struct NewWs {
  int most, group;         // slots with several new tokens: of any legal call, of a round
  int nch, nblk;           // chunks and blocks of any legal pass of a round
  size_t cstart, bstart, pstart, ustart, vstart, rstart, mstart;  // plan (TcPlan)
  size_t nx, nuw;          // -X [nch][H][64][64], -U W [2][nch][H][64][D] (high, rest)
  size_t kr, f;            // K-> [2][nch][H][64][D], F [2][nch][H][D][D] (high, rest)
  size_t ke, fb;           // keys at their block's end [2][nblk][H][256][D], block products [2][nblk][H][D][D]
  size_t gb, mm;           // G_b [2][nblk][H][D][D], M [2][group][H][D][D]
  size_t ver;              // versions: rows [D]
  size_t cn;               // forget gate: sums since the start of the call [H][nblk * 256]
  size_t zs, z;            // queries at the block's and at the call's start [2][H][pairs][256][D] (rest: TcPlan)
  size_t m, l, acc;        // the diagonal's state [nch][hq][64](, [D])
  size_t pm, pl, pacc;     // parts of the tensor-core attention
  size_t err, total;
  long long ver_rows;
  int pairs;
};
NewWs new_ws(const PagedArgs& p, int group) {  // for rounds of `group` slots
  NewWs w{};
  const size_t D = p.c.head_dim, H = p.c.heads, hq = p.hq;
  const long long live = w.group = group;
  const long long most = p.max_new < kTcPassTokens ? p.max_new : kTcPassTokens;  // new tokens of a slot in a pass
  const long long tokens = p.total < most * live ? p.total : most * live;
  auto parts_of = [&](long long x) { const long long n = (tokens + (x - 1) * live) / x; return n < 1 ? 1LL : n; };
  w.nch = (int)parts_of(C);
  w.nblk = (int)parts_of(MB);
  const long long np = (tokens * p.G + (kTcPair - 1) * live) / kTcPair;
  w.pairs = (int)(np < 1 ? 1 : np);
  const long long blk = (most + MB - 1) / MB;
  w.ver_rows = (long long)H * w.nblk * (blk > 1 ? blk - 1 : 0) * (MB / 2);
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align_up(off + bytes, 256); return o; };
  const size_t S1 = p.c.slots + 1;
  w.cstart = take(S1 * 4);
  w.bstart = take(S1 * 4);
  w.pstart = take(S1 * 4);
  w.rstart = take(S1 * 4);
  w.mstart = take(S1 * 4);
  w.vstart = take(S1 * 8);
  w.ustart = take(S1 * 8);
  w.nx = take((size_t)w.nch * H * C * C * 2);
  w.nuw = take((size_t)2 * w.nch * H * C * D * 2);
  w.kr = take((size_t)2 * w.nch * H * C * D * 2);
  w.f = take((size_t)2 * w.nch * H * D * D * 2);
  w.ke = take((size_t)2 * w.nblk * H * MB * D * 2);
  w.fb = take((size_t)2 * w.nblk * H * D * D * 2);
  w.gb = take((size_t)2 * w.nblk * H * D * D * 2);
  w.mm = take((size_t)2 * group * H * D * D * 2);
  w.ver = take((size_t)w.ver_rows * D * 2);
  w.cn = take((size_t)H * w.nblk * MB * 4);
  w.zs = take((size_t)2 * H * w.pairs * kTcPair * D * 2);
  w.z = take((size_t)2 * H * w.pairs * kTcPair * D * 2);
  w.m = take((size_t)w.nch * hq * C * 4);
  w.l = take((size_t)w.nch * hq * C * 4);
  w.acc = take((size_t)w.nch * hq * C * D * 4);
  const size_t parts = 2 * (size_t)H * w.pairs + kTcBlocks;
  w.pm = take(parts * kTcPair * 4);
  w.pl = take(parts * kTcPair * 4);
  w.pacc = take(parts * kTcPair * D * 4);
  w.err = take(4);
  w.total = off;
  return w;
}

NewWs new_ws(const PagedArgs& p) {
  const int most = most_multi(p);
  NewWs w = new_ws(p, round_slots(most, [&](int n) { return new_ws(p, n).total; }));
  w.most = most;
  return w;
}

// ---- plan ----
// Exclusive prefix sums over the slots, all at once: chunks, blocks, query pairs, rewrite tiles, version rows, units, slots of
// the round.  Slots with several new tokens are numbered in order; the round takes those from number `first` on, and those from number `most` on are left out.
__global__ void __launch_bounds__(1024) plan_kernel(PagedArgs p, TcPlan pl, int first, int most, bool report) {
  chain();
  constexpr int N = 7;
  __shared__ long long wsum[N][32], carry[N];
  __shared__ int multi[32];
  __shared__ unsigned long long tokens;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < N) carry[tid] = 0;
  if (tid == 0) {
    *pl.err = 0;
    tokens = 0;
  }
  int numbered = 0;  // slots with several new tokens so far
  __syncthreads();
  for (int base = 0; base < p.c.slots; base += 1024) {
    const int b = base + tid;
    long long v[N] = {0, 0, 0, 0, 0, 0, 0}, x[N];
    SlotSpan all{};
    int n = 0;
    if (b < p.c.slots) {
      all = slot_span(p, b);
      if (report && all.code) paged_error(p.c.status, all.code);
      if (all.n < p.min_new) all.n = 0;
      n = all.n;
    }
    leave_out_pageless(p.c, b, all.t0, n, all, report);
    const int number = number_multi(all.n > 0, multi, numbered);
    if (all.n > 0) {
      atomicAdd(&tokens, (unsigned long long)all.n);
      if (number >= most) {
        all.n = 0;
        if (report) paged_error(p.c.status, PATH_PAGED_BAD_START);
      }
    }
    if (report && n > 0) note_extended(p.c, b, all.n > 0 ? n : -1);
    if (all.n > 0) {
      const SlotSpan s = pass_part(p, all);
      if (s.n > 0 && number >= first && number - first < pl.group) {
        const long long H = p.c.heads, np = ((long long)s.n * p.G + kTcPair - 1) / kTcPair, nb = (s.n + MB - 1) / MB;
        v[0] = (s.n + C - 1) / C;
        v[1] = nb;
        v[2] = np;
        v[3] = live_tiles(s.t0, p.window, p.sinks, kRewriteRows).count;
        v[4] = H * (MB / 2) * nb * (nb - 1);
        v[5] = H * (np * live_tiles(s.t0, p.window, p.sinks, kTcKeys).count + new_units(np, p.G));
        v[6] = 1;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = v[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x[i], o);
        if (lane >= o) x[i] += a;
      }
      if (lane == 31) wsum[i][warp] = x[i];
    }
    __syncthreads();
    if (warp < N) {  // warp i adds up row i
      long long t = wsum[warp][lane], y = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += a;
      }
      const long long c0 = carry[warp];
      wsum[warp][lane] = c0 + y - t;
      __syncwarp();
      if (lane == 31) carry[warp] = c0 + y;
    }
    __syncthreads();
    if (b < p.c.slots) {
      long long e[N];
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = wsum[i][warp] + x[i] - v[i];
      pl.cstart[b] = (int)e[0];
      pl.bstart[b] = (int)e[1];
      pl.pstart[b] = (int)e[2];
      pl.rstart[b] = (int)e[3];
      pl.vstart[b] = e[4];
      pl.ustart[b] = e[5];
      pl.mstart[b] = (int)e[6];
    }
    __syncthreads();
  }
  const int S = p.c.slots;
  if (tid == 0) {
    pl.cstart[S] = (int)carry[0];
    pl.bstart[S] = (int)carry[1];
    pl.pstart[S] = (int)carry[2];
    pl.rstart[S] = (int)carry[3];
    pl.vstart[S] = carry[4];
    pl.ustart[S] = carry[5];
    pl.mstart[S] = (int)carry[6];
  }
  // rows of q_start that overlap: more tokens than the workspace is for
  if (tokens > (unsigned long long)p.total) {
    if (tid == 0) paged_error(p.c.status, PATH_PAGED_BAD_START);
    __syncthreads();
    for (int b = tid; b <= S; b += 1024) {
      if (report && b < S && slot_span(p, b).n >= p.min_new) note_extended(p.c, b, -1);
      pl.cstart[b] = pl.bstart[b] = pl.pstart[b] = pl.rstart[b] = pl.mstart[b] = 0;
      pl.vstart[b] = pl.ustart[b] = 0;
    }
  }
}
__device__ __forceinline__ int owner(const int* start, int slots, int x) {
  int lo = 0, hi = slots;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// ---- chunk preparation: one block per (chunk, key head) ----
// W and K are bf16 as given, so their products are exact up to the fp32 sums; U, N, X, Y enter later products as pairs.
constexpr int PT = 256;
template <int D>
struct PrepSmem {
  static constexpr int LD = D + 8, LX = C + 8;
  bf16 w[C][LD], k[C][LD];
  union {
    struct { float g[C][C + 1], u[C][C + 1], t[32][33]; };  // until U is split
    struct { bf16 yh[C][LD], yl[C][LD]; };                   // from then on
  };
  bf16 uh[C][LX], ul[C][LX], nh[C][LX], nl[C][LX];           // (X takes the place of N)
  float beta[C];
};
// A fragments of the transpose of a tile stored as [k][m] rows.
template <int KS>
__device__ __forceinline__ void load_at(uint32_t (&a)[KS][4], const bf16* t, int ld, int m0) {
  const int lane = threadIdx.x & 31, mat = lane >> 3, row = lane & 7;
#pragma unroll
  for (int k = 0; k < KS; ++k) ldm4t(a[k], t + (16 * k + (mat >> 1) * 8 + row) * ld + m0 + (mat & 1) * 8);
}
template <int NT>
__device__ __forceinline__ void zero(float (&c)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
}
// Accumulators at (m0, n0) as a pair of bf16 tiles (or, lo null, rounded) with row pitch ld.
template <int NT>
__device__ __forceinline__ void put_pair(const float (&c)[NT][4], bf16* hi, bf16* lo, int ld, int m0, int n0) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t a, e;
      split2(c[n][2 * y], c[n][2 * y + 1], a, e);
      const size_t at = (size_t)(m0 + g + 8 * y) * ld + n0 + 8 * n + 2 * t;
      *reinterpret_cast<uint32_t*>(hi + at) = a;
      if (lo) *reinterpret_cast<uint32_t*>(lo + at) = e;
    }
}
template <int D>
__global__ void __launch_bounds__(PT, 2) prep_kernel(PagedArgs p, NewWs w, TcPlan pl, char* ws) {
  chain();
  extern __shared__ __align__(16) uint8_t smem[];
  using S = PrepSmem<D>;
  S& s = *reinterpret_cast<S*>(smem);
  constexpr int LD = S::LD, LX = S::LX;
  const int c = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = p.c.heads;
  const int g = lane >> 2, t = lane & 3;
  if (c >= pl.cstart[p.c.slots]) return;
  const int b = owner(pl.cstart, p.c.slots, c);
  const SlotSpan sp = pass_span(p, b);
  const int r0 = (c - pl.cstart[b]) * C, rows = min(C, sp.n - r0);
  const size_t tok0 = (size_t)sp.q0 + r0;
  fetch<D, LD, PT>(&s.w[0][0], (const bf16*)p.w + (tok0 * H + h) * D, (size_t)H * D, C, rows);
  fetch<D, LD, PT>(&s.k[0][0], (const bf16*)p.k + (tok0 * H + h) * D, (size_t)H * D, C, rows);
  if (tid < C) s.beta[tid] = tid < rows ? clamp_beta(p.beta[(tok0 + tid) * H + h]) : 0.f;
  for (int e = tid; e < C * C; e += PT) s.u[e / C][e % C] = 0.f;
  fetch_wait();
  __syncthreads();
  const int m0 = (warp & 3) * 16, nh = warp >> 2;  // this warp's 16 rows and column half of a 64-row product
  {
    uint32_t a[D / 16][4];
    float x[4][4], y[4][4];
    load_a(a, &s.w[0][0], LD, m0);
    zero(x);
    zero(y);
    warp_mm<4, D / 16, false>(x, a, &s.w[32 * nh][0], LD);  // W W^T
    warp_mm<4, D / 16, false>(y, a, &s.k[32 * nh][0], LD);  // W K^T
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = m0 + g + (e >> 1) * 8, j = 32 * nh + 8 * n + 2 * t + (e & 1);
        s.g[i][j] = x[n][e];
        if (j >= i) y[n][e] = 0.f;
      }
    put_pair(y, &s.nh[0][0], &s.nl[0][0], LX, m0, 32 * nh);
  }
  __syncthreads();
  // U, block inversion: the two diagonal 32-row blocks by forward substitution (one warp each, one column per
  // lane), then U21 = -U22 G21 U11
  if (tid < 64) {
    const int o = tid & 32, col = tid & 31;
    float u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float a0 = (col == i) ? 1.f : 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) {
        const float x = s.g[o + i][o + m] * u[m];
        if ((m & 3) == 0) a0 -= x;
        else if ((m & 3) == 1) a1 -= x;
        else if ((m & 3) == 2) a2 -= x;
        else a3 -= x;
      }
      u[i] = s.beta[o + i] * ((a0 + a1) + (a2 + a3));
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) s.u[o + i][o + col] = u[i];
  }
  __syncthreads();
  const int i4 = tid >> 3, j4 = (tid & 7) * 4;  // one row, four columns per thread of a 32 x 32 product
  {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int m = 0; m < 32; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = fmaf(s.g[32 + i4][m], s.u[m][j4 + e], a[e]);
#pragma unroll
    for (int e = 0; e < 4; ++e) s.t[i4][j4 + e] = a[e];
  }
  __syncthreads();
  {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int m = 0; m < 32; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = fmaf(s.u[32 + i4][32 + m], s.t[m][j4 + e], a[e]);
#pragma unroll
    for (int e = 0; e < 4; ++e) s.u[32 + i4][j4 + e] = -a[e];
  }
  __syncthreads();
  for (int e = tid; e < C * C / 2; e += PT) {
    const int i = e / (C / 2), j = e % (C / 2) * 2;
    uint32_t hi, lo;
    split2(s.u[i][j], s.u[i][j + 1], hi, lo);
    *reinterpret_cast<uint32_t*>(&s.uh[i][j]) = hi;
    *reinterpret_cast<uint32_t*>(&s.ul[i][j]) = lo;
  }
  __syncthreads();
  const size_t cc = (size_t)c * H + h;
  constexpr int NH = D / 16;  // 8-column tiles of half a row
  {
    uint32_t ah[4][4], al[4][4];
    load_a(ah, &s.uh[0][0], LX, m0);
    load_a(al, &s.ul[0][0], LX, m0);
    float x[4][4];
    zero(x);
    warp_mm2<4, 4, true>(x, ah, al, &s.nh[0][32 * nh], LX);  // X = U N
    warp_mm<4, 4, true>(x, ah, &s.nl[0][32 * nh], LX);
    __syncthreads();  // (every warp has read N)
    put_pair(x, &s.nh[0][0], &s.nl[0][0], LX, m0, 32 * nh);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] = -x[n][e];
    put_pair(x, (bf16*)(ws + w.nx) + cc * C * C, (bf16*)nullptr, C, m0, 32 * nh);
    float y[NH][4];
    zero(y);
    warp_mm2<NH, 4, true>(y, ah, al, &s.w[0][8 * NH * nh], LD);  // U W
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[n][e] = -y[n][e];
    bf16* uw = (bf16*)(ws + w.nuw) + cc * C * D;
    put_pair(y, uw, uw + (size_t)w.nch * H * C * D, D, m0, 8 * NH * nh);
    load_at(ah, &s.uh[0][0], LX, m0);
    load_at(al, &s.ul[0][0], LX, m0);
    zero(y);
    warp_mm2<NH, 4, true>(y, ah, al, &s.w[0][8 * NH * nh], LD);  // Y = U^T W
    put_pair(y, &s.yh[0][0], &s.yl[0][0], LD, m0, 8 * NH * nh);
  }
  __syncthreads();
  {
    uint32_t ah[4][4], al[4][4];
    load_at(ah, &s.nh[0][0], LX, m0);
    load_at(al, &s.nl[0][0], LX, m0);
    float y[NH][4];
    zero(y);
    warp_mm2<NH, 4, true>(y, ah, al, &s.w[0][8 * NH * nh], LD);  // X^T W
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t kk = *reinterpret_cast<const uint32_t*>(&s.k[m0 + g + 8 * v][8 * NH * nh + 8 * n + 2 * t]);
        y[n][2 * v] = lo_f(kk) - y[n][2 * v];
        y[n][2 * v + 1] = hi_f(kk) - y[n][2 * v + 1];
      }
    bf16* kr = (bf16*)(ws + w.kr) + cc * C * D;
    put_pair(y, kr, kr + (size_t)w.nch * H * C * D, D, m0, 8 * NH * nh);
  }
  // F = I - W^T Y: D rows over the warps
  bf16* f = (bf16*)(ws + w.f) + cc * D * D;
  for (int tile = warp; tile < D / 16 * 2; tile += PT / 32) {
    const int fm = tile / 2 * 16, fn = tile % 2;
    uint32_t a[4][4];
    load_at(a, &s.w[0][0], LD, fm);
    float y[NH][4];
    zero(y);
    warp_mm<NH, 4, true>(y, a, &s.yh[0][8 * NH * fn], LD);
    warp_mm<NH, 4, true>(y, a, &s.yl[0][8 * NH * fn], LD);
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = fm + g + (e >> 1) * 8, j = 8 * NH * fn + 8 * n + 2 * t + (e & 1);
        y[n][e] = (i == j ? 1.f : 0.f) - y[n][e];
      }
    put_pair(y, f, f + (size_t)w.nch * H * D * D, D, fm, 8 * NH * fn);
  }
}

// ---- carried rows ----
constexpr int WT = 128;
template <int D>
constexpr size_t carry_smem() { return (size_t)2 * D * (D + 8) * 2; }
// A slab of 64 rows (16 per warp) in fp32 accumulators: rows <- rows F, F as a pair of [D][D] matrices.
template <int D>
struct Slab {
  float c[D / 8][4];
  __device__ __forceinline__ void load(const bf16* hi, const bf16* lo) {  // [64][D]
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, r0 = (threadIdx.x >> 5) * 16 + g;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const size_t at = (size_t)(r0 + 8 * y) * D + 8 * n + 2 * t;
        const uint32_t a = *reinterpret_cast<const uint32_t*>(hi + at), e = *reinterpret_cast<const uint32_t*>(lo + at);
        c[n][2 * y] = lo_f(a) + lo_f(e);
        c[n][2 * y + 1] = hi_f(a) + hi_f(e);
      }
  }
  __device__ __forceinline__ void times(const bf16* fh, const bf16* fl, bf16* sm) {
    constexpr int LD = D + 8;
    bf16 *sh = sm, *sl = sm + D * LD;
    __syncthreads();
    fetch<D, LD, WT>(sh, fh, D, D, D);
    fetch<D, LD, WT>(sl, fl, D, D, D);
    uint32_t ah[D / 16][4], al[D / 16][4];
    to_a2(ah, al, c);
#pragma unroll
    for (int n = 0; n < D / 8; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
    fetch_wait();
    __syncthreads();
    warp_mm2<D / 8, D / 16, true>(c, ah, al, sh, LD);
    warp_mm<D / 8, D / 16, true>(c, ah, sl, LD);
  }
  // rows r of `rows` as a pair, or (lo null) rounded
  __device__ __forceinline__ void store(bf16* hi, bf16* lo, int rows = 64) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, r0 = (threadIdx.x >> 5) * 16 + g;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (r0 + 8 * y >= rows) continue;
        const size_t at = (size_t)(r0 + 8 * y) * D + 8 * n + 2 * t;
        uint32_t a, e;
        split2(c[n][2 * y], c[n][2 * y + 1], a, e);
        *reinterpret_cast<uint32_t*>(hi + at) = a;
        if (lo) *reinterpret_cast<uint32_t*>(lo + at) = e;
      }
  }
};

// Level 1, one block per (block, key head, slab): slabs 0..3 are the block's chunks of keys, carried to the
// block's end; the others rows of the block product.
template <int D>
__device__ void carry_in_block(const PagedArgs& p, const NewWs& w, const TcPlan& pl, char* ws, bf16* sm, int blk, int h, int slab) {
  const int H = p.c.heads;
  const int b = owner(pl.bstart, p.c.slots, blk);
  const SlotSpan sp = pass_span(p, b);
  const int lb = blk - pl.bstart[b], nch = (min(MB, sp.n - lb * MB) + C - 1) / C, c0 = pl.cstart[b] + lb * CPB;
  if (slab < CPB && slab >= nch) return;
  const size_t fstep = (size_t)w.nch * H * D * D, kstep = (size_t)w.nch * H * C * D;
  const bf16 *fh = (const bf16*)(ws + w.f), *kr = (const bf16*)(ws + w.kr);
  Slab<D> s;
  int c = c0;
  if (slab < CPB) {
    c = c0 + slab;
    const bf16* at = kr + ((size_t)c * H + h) * C * D;
    s.load(at, at + kstep);
  } else {
    const bf16* at = fh + ((size_t)c * H + h) * D * D + (size_t)(slab - CPB) * 64 * D;
    s.load(at, at + fstep);
  }
  for (++c; c < c0 + nch; ++c) {
    const bf16* at = fh + ((size_t)c * H + h) * D * D;
    s.times(at, at + fstep, sm);
  }
  const size_t bb = (size_t)blk * H + h;
  if (slab < CPB) {
    bf16* at = (bf16*)(ws + w.ke) + (bb * MB + slab * C) * D;
    s.store(at, at + (size_t)w.nblk * H * MB * D);
  } else {
    bf16* at = (bf16*)(ws + w.fb) + bb * D * D + (size_t)(slab - CPB) * 64 * D;
    s.store(at, at + (size_t)w.nblk * H * D * D);
  }
}

// Level 2: through the later blocks of the slot, a copy at every block start; at the end into the pages, or M.
template <int D>
__device__ void carry_on(const PagedArgs& p, const NewWs& w, const TcPlan& pl, char* ws, bf16* sm, int blk, int h, int slab) {
  const int H = p.c.heads;
  if (blk >= pl.bstart[p.c.slots]) return;
  const int b = owner(pl.bstart, p.c.slots, blk);
  const SlotSpan sp = pass_span(p, b);
  const int b0 = pl.bstart[b], lb = blk - b0, nb = (sp.n + MB - 1) / MB;
  const int rows = slab < CPB ? min(C, sp.n - lb * MB - slab * C) : 64;
  if (rows <= 0 || (slab >= CPB && lb > 0)) return;  // (the slot's first block carries the identity)
  const size_t fstep = (size_t)w.nblk * H * D * D, kstep = (size_t)w.nblk * H * MB * D;
  const size_t bb = (size_t)blk * H + h;
  const int ir = (slab - CPB) * 64;
  Slab<D> s;
  if (slab < CPB) {
    const bf16* at = (const bf16*)(ws + w.ke) + (bb * MB + slab * C) * D;
    s.load(at, at + kstep);
  } else {
    const bf16* at = (const bf16*)(ws + w.fb) + bb * D * D + (size_t)ir * D;
    s.load(at, at + fstep);
  }
  for (int x = lb + 1; x < nb; ++x) {
    // rows at the start of block x
    if (slab < CPB) {
      // versions of a slot: per head, blocks 1..: version x has 256 x rows and lies behind 128 x (x - 1) rows
      const long long v = pl.vstart[b] + (long long)h * (MB / 2) * nb * (nb - 1) + (long long)(MB / 2) * x * (x - 1) + lb * MB + slab * C;
      s.store((bf16*)(ws + w.ver) + v * D, nullptr);
    } else {
      bf16* at = (bf16*)(ws + w.gb) + ((size_t)(b0 + x) * H + h) * D * D + (size_t)ir * D;
      s.store(at, at + fstep);
    }
    const bf16* at = (const bf16*)(ws + w.fb) + ((size_t)(b0 + x) * H + h) * D * D;
    s.times(at, at + fstep, sm);
  }
  if (slab >= CPB) {
    bf16* at = (bf16*)(ws + w.mm) + ((size_t)pl.mstart[b] * H + h) * D * D + (size_t)ir * D;
    s.store(at, at + (size_t)pl.group * H * D * D);
    return;
  }
  // the appended rows
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, r0 = (threadIdx.x >> 5) * 16 + g;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int r = r0 + 8 * y;
    if (r >= rows) continue;
    const long long at = pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, sp.t0 + lb * MB + slab * C + r);
    if (at < 0) {
      paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
      continue;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<uint32_t*>((bf16*)p.c.k_pool + at * D + 8 * n + 2 * t) = pack2(s.c[n][2 * y], s.c[n][2 * y + 1]);
  }
}

// Sums of log f since the start of the pass, and the running sums of the appended rows: one block per (slot of the round,
// head).
__device__ void gate_sums(const PagedArgs& p, const NewWs& w, const TcPlan& pl, char* ws, int m, int h) {
  __shared__ float wsum[WT / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, H = p.c.heads;
  if (m >= pl.mstart[p.c.slots]) return;
  const int b = owner(pl.mstart, p.c.slots, m);
  const SlotSpan sp = pass_span(p, b);
  const long long last = sp.t0 > 0 ? pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 - 1) : -1;
  const double a0 = last >= 0 ? load_sum(p.c, last) : 0.0;
  float* cn = (float*)(ws + w.cn) + ((size_t)h * w.nblk + pl.bstart[b]) * MB;
  double carry = 0.0;
  for (int base = 0; base < sp.n; base += WT) {
    const int r = base + tid;
    const float v = r < sp.n ? p.log_f[((size_t)sp.q0 + r) * H + h] : 0.f;
    float x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float a = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += a;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    float before = 0.f, all = 0.f;
#pragma unroll
    for (int i = 0; i < WT / 32; ++i) {
      if (i < warp) before += wsum[i];
      all += wsum[i];
    }
    if (r < sp.n) {
      const double c = carry + before + x;
      cn[r] = (float)c;
      const long long at = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 + r);
      if (at >= 0) store_sum(p.c, at, a0 + c);
    }
    carry += all;
  }
}

// Blocks: (block, head, slab) of level 1, then (slot of the round, head) of the gate's sums.
template <int D>
__global__ void __launch_bounds__(WT) carry_in_block_kernel(PagedArgs p, NewWs w, TcPlan pl, char* ws) {
  chain();
  extern __shared__ __align__(16) uint8_t smem[];
  const int slabs = CPB + D / 64, H = p.c.heads;
  const int x = blockIdx.x, n1 = w.nblk * H * slabs;
  if (x >= n1) {
    gate_sums(p, w, pl, ws, (x - n1) / H, (x - n1) % H);
    return;
  }
  const int blk = x / (H * slabs), rest = x % (H * slabs);
  if (blk >= pl.bstart[p.c.slots]) return;
  carry_in_block<D>(p, w, pl, ws, (bf16*)smem, blk, rest / slabs, rest % slabs);
}

// ---- queries: diagonal chunk and the earlier chunks of the block; one block per (chunk, query head) ----
template <int D>
struct QSmem {
  static constexpr int LD = D + 8, LX = C + 8, T = C * LD;  // one [64][D] tile
  static constexpr int kQ = 0, kW = T, kK = 2 * T, kV = 3 * T, kUW = 4 * T, kUWl = 5 * T, kX = 6 * T;
  static constexpr int kFh = 2 * T, kFl = kFh + D * LD;     // chain: keys at 0, values at T, F behind them
  static constexpr int end1 = kX + C * LX, end2 = kFl + D * LD;
  static constexpr size_t bytes = (size_t)(end1 > end2 ? end1 : end2) * 2;
};
// Online softmax of the scores of 64 keys (16 rows per warp, log2 domain, hidden ones -inf): p as pairs of A fragments.
__device__ __forceinline__ void softmax64(float (&s)[8][4], float (&m)[2], float (&l)[2], float (&corr)[2], uint32_t (&pa)[4][4],
                                          uint32_t (&pb)[4][4]) {
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    float mx = -INFINITY;
#pragma unroll
    for (int n = 0; n < 8; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * y], s[n][2 * y + 1]));
    mx = group_max<4>(mx);
    const float mn = fmaxf(m[y], mx);
    corr[y] = mn == -INFINITY ? 1.f : fast_exp2(m[y] - mn);
    m[y] = mn;
    const float mu = mn == -INFINITY ? 0.f : mn;
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      s[n][2 * y] = fast_exp2(s[n][2 * y] - mu);
      s[n][2 * y + 1] = fast_exp2(s[n][2 * y + 1] - mu);
      sum += s[n][2 * y] + s[n][2 * y + 1];
    }
    l[y] = l[y] * corr[y] + sum;
  }
  to_a2(pa, pb, s);
}
// The first thread blocks carry keys on (level 2: the longest chains, and independent of the queries).
template <int D, bool FOX>
__global__ void __launch_bounds__(WT, D == 64 ? 3 : 2) query_kernel(PagedArgs p, NewWs w, TcPlan pl, char* ws) {
  chain();
  extern __shared__ __align__(16) uint8_t smem[];
  bf16* sm = (bf16*)smem;
  using S = QSmem<D>;
  constexpr int LD = S::LD, LX = S::LX;
  const int slabs = CPB + D / 64, carries = w.nblk * p.c.heads * slabs;
  if ((int)blockIdx.x < carries) {
    const int x = blockIdx.x;
    // slabs of the identity first, then by block: chains fall in length
    const int per = p.c.heads * slabs;
    carry_on<D>(p, w, pl, ws, sm, x / per, x % per / slabs, slabs - 1 - x % slabs);
    return;
  }
  const int c = (blockIdx.x - carries) / p.hq, qh = (blockIdx.x - carries) % p.hq, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int H = p.c.heads, G = p.G, h = qh / G;
  if (c >= pl.cstart[p.c.slots]) return;
  const int b = owner(pl.cstart, p.c.slots, c);
  const SlotSpan sp = pass_span(p, b);
  const int lc = c - pl.cstart[b], r0 = lc * C, rows = min(C, sp.n - r0);
  const size_t cc = (size_t)c * H + h, tok = (size_t)sp.q0 + r0;
  fetch<D, LD, WT>(sm + S::kQ, (const bf16*)p.q + (tok * p.hq + qh) * D, (size_t)p.hq * D, C, rows);
  fetch<D, LD, WT>(sm + S::kW, (const bf16*)p.w + (tok * H + h) * D, (size_t)H * D, C, rows);
  fetch<D, LD, WT>(sm + S::kK, (const bf16*)p.k + (tok * H + h) * D, (size_t)H * D, C, rows);
  fetch<D, LD, WT>(sm + S::kV, (const bf16*)p.v + (tok * H + h) * D, (size_t)H * D, C, rows);
  fetch<D, LD, WT>(sm + S::kUW, (const bf16*)(ws + w.nuw) + cc * C * D, D, C, C);
  fetch<D, LD, WT>(sm + S::kUWl, (const bf16*)(ws + w.nuw) + ((size_t)w.nch * H + cc) * C * D, D, C, C);
  fetch<C, LX, WT>(sm + S::kX, (const bf16*)(ws + w.nx) + cc * C * C, C, C, C);
  fetch_wait();
  __syncthreads();
  if (qh % G == 0)  // the values join the cache
    for (int e = tid; e < rows * (D / 8); e += WT) {
      const int r = e / (D / 8), x = e % (D / 8) * 8;
      const long long at = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 + r0 + r);
      if (at >= 0) *reinterpret_cast<uint4*>((bf16*)p.c.v_pool + at * D + x) = *reinterpret_cast<const uint4*>(sm + S::kV + r * LD + x);
      else paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
    }
  const int ra = warp * 16 + g;  // this lane's rows: ra, ra + 8
  float ci[2] = {0.f, 0.f};
  const float* cn = (const float*)(ws + w.cn) + ((size_t)h * w.nblk + pl.bstart[b]) * MB;
  if (FOX)
#pragma unroll
    for (int y = 0; y < 2; ++y) ci[y] = ra + 8 * y < rows ? cn[r0 + ra + 8 * y] : 0.f;
  // scores in the log2 domain of the keys of local chunk x, hidden ones -inf
  auto finish = [&](float (&s)[8][4], int x) {
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = r0 + ra + (e >> 1) * 8, j = x * C + 8 * n + 2 * t + (e & 1);
        float v = s[n][e] * p.scl;
        if (FOX && j <= i && j < sp.n) v += (ci[e >> 1] - cn[j]) * kLog2e;
        if (j > i || !sees(p.window, p.sinks, sp.t0 + i, sp.t0 + j)) v = -INFINITY;
        s[n][e] = v;
      }
  };
  float o[D / 8][4], z[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, corr[2];
  uint32_t pa[4][4], pb[4][4];
  {
    uint32_t qa[D / 16][4], mh[4][4], ml[4][4];
    load_a(qa, sm + S::kQ, LD, warp * 16);
    float s1[8][4], s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s1[n][e] = s[n][e] = 0.f;
    warp_mm<8, D / 16, false>(s1, qa, sm + S::kW, LD);
    warp_mm<8, D / 16, false>(s, qa, sm + S::kK, LD);
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (8 * n + 2 * t + (e & 1) > ra + (e >> 1) * 8) s1[n][e] = 0.f;  // lower(Q W^T)
    to_a2(mh, ml, s1);
    warp_mm2<8, 4, true>(s, mh, ml, sm + S::kX, LX);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int y = 0; y < 4; ++y) {  // the fragment's registers as accumulators
        z[2 * k + (y >> 1)][2 * (y & 1)] = lo_f(qa[k][y]);
        z[2 * k + (y >> 1)][2 * (y & 1) + 1] = hi_f(qa[k][y]);
      }
    warp_mm2<D / 8, 4, true>(z, mh, ml, sm + S::kUW, LD);
    warp_mm<D / 8, 4, true>(z, mh, sm + S::kUWl, LD);
    finish(s, lc);
    softmax64(s, m, l, corr, pa, pb);
  }
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  warp_mm2<D / 8, 4, true>(o, pa, pb, sm + S::kV, LD);
  // The earlier chunks of the block: keys and values of the next one are fetched while F is applied, its F while the
  // scores are worked on.
  const int first = lc / CPB * CPB;
  auto fetch_rows = [&](int x) {
    fetch<D, LD, WT>(sm, (const bf16*)(ws + w.kr) + ((size_t)(c - lc + x) * H + h) * C * D, D, C, C);
    fetch<D, LD, WT>(sm + S::T, (const bf16*)p.v + (((size_t)sp.q0 + x * C) * H + h) * D, (size_t)H * D, C, C);
  };
  auto fetch_f = [&](int x) {
    const bf16* fh = (const bf16*)(ws + w.f) + ((size_t)(c - lc + x) * H + h) * D * D;
    fetch<D, LD, WT>(sm + S::kFh, fh, D, D, D);
    fetch<D, LD, WT>(sm + S::kFl, fh + (size_t)w.nch * H * D * D, D, D, D);
  };
  if (lc > first) {
    __syncthreads();
    fetch_rows(lc - 1);
    fetch_commit();
    fetch_f(lc - 1);
    fetch_commit();
  }
  for (int x = lc - 1; x >= first; --x) {
    uint32_t za[D / 16][4], zb[D / 16][4];
    to_a2(za, zb, z);
    fetch_wait_but<1>();
    __syncthreads();
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    warp_mm2<8, D / 16, false>(s, za, zb, sm, LD);
    finish(s, x);
    softmax64(s, m, l, corr, pa, pb);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] *= corr[e >> 1];
    warp_mm2<D / 8, 4, true>(o, pa, pb, sm + S::T, LD);
    __syncthreads();
    if (x > first) fetch_rows(x - 1);
    fetch_commit();
    fetch_wait_but<1>();
    __syncthreads();
#pragma unroll
    for (int n = 0; n < D / 8; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.f;
    warp_mm2<D / 8, D / 16, false>(z, za, zb, sm + S::kFh, LD);
    warp_mm<D / 8, D / 16, false>(z, za, sm + S::kFl, LD);
    if (x > first) {
      __syncthreads();
      fetch_f(x - 1);
    }
    fetch_commit();
  }
  const size_t st = ((size_t)c * p.hq + qh) * C;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int r = ra + 8 * y;
    const float ls = group_sum<4>(l[y]);  // (all lanes: before any leaves)
    if (r >= rows) continue;
    if (t == 0) {
      ((float*)(ws + w.m))[st + r] = m[y];
      ((float*)(ws + w.l))[st + r] = ls;
    }
    float* acc = (float*)(ws + w.acc) + (st + r) * D;
    const int R = (r0 + r) * G + qh % G;
    const size_t zr = (((size_t)h * w.pairs + pl.pstart[b]) * kTcPair + R) * D, zstep = (size_t)H * w.pairs * kTcPair * D;
    const bool rest = D == 64 || sp.n * G - R / kTcPair * kTcPair <= kTcPair / 2;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      *reinterpret_cast<float2*>(acc + 8 * n + 2 * t) = make_float2(o[n][2 * y], o[n][2 * y + 1]);
      uint32_t zz, ze;
      split2(z[n][2 * y], z[n][2 * y + 1], zz, ze);
      const size_t at = zr + 8 * n + 2 * t;
      *reinterpret_cast<uint32_t*>((bf16*)(ws + w.zs) + at) = zz;
      if (lc < CPB) *reinterpret_cast<uint32_t*>((bf16*)(ws + w.z) + at) = zz;
      if (rest) {
        *reinterpret_cast<uint32_t*>((bf16*)(ws + w.zs) + zstep + at) = ze;
        if (lc < CPB) *reinterpret_cast<uint32_t*>((bf16*)(ws + w.z) + zstep + at) = ze;
      }
    }
  }
}

// z = zs G_b^T for the query pairs behind the first block: one block per (64 rows of a pair, head).
template <int D>
__global__ void __launch_bounds__(WT) start_kernel(PagedArgs p, NewWs w, TcPlan pl, char* ws) {
  chain();
  extern __shared__ __align__(16) uint8_t smem[];
  bf16* sm = (bf16*)smem;
  constexpr int LD = D + 8;
  const int pr = blockIdx.x / 4, q = blockIdx.x % 4, h = blockIdx.y, H = p.c.heads;
  if (pr >= pl.pstart[p.c.slots]) return;
  const int b = owner(pl.pstart, p.c.slots, pr);
  const SlotSpan sp = pass_span(p, b);
  const int lp = pr - pl.pstart[b], blk = lp / p.G;
  if (blk == 0 || lp * kTcPair + q * 64 >= sp.n * p.G) return;
  const bf16* gh = (const bf16*)(ws + w.gb) + ((size_t)(pl.bstart[b] + blk) * H + h) * D * D;
  const size_t row = ((size_t)h * w.pairs + pr) * kTcPair + q * 64;
  const size_t zstep = (size_t)H * w.pairs * kTcPair * D;
  const bool rest = D == 64 || sp.n * p.G - lp * kTcPair <= kTcPair / 2;
  bf16 *sz = sm + 2 * D * LD, *se = sz + 64 * LD;
  fetch<D, LD, WT>(sm, gh, D, D, D);
  fetch<D, LD, WT>(sm + D * LD, gh + (size_t)w.nblk * H * D * D, D, D, D);
  fetch<D, LD, WT>(sz, (const bf16*)(ws + w.zs) + row * D, D, 64, 64);
  if (rest) fetch<D, LD, WT>(se, (const bf16*)(ws + w.zs) + zstep + row * D, D, 64, 64);
  fetch_wait();
  __syncthreads();
  uint32_t a[D / 16][4];
  Slab<D> s;
  zero(s.c);
  if (rest) {
    load_a(a, se, LD, (threadIdx.x >> 5) * 16);
    warp_mm<D / 8, D / 16, false>(s.c, a, sm, LD);
  }
  load_a(a, sz, LD, (threadIdx.x >> 5) * 16);
  warp_mm<D / 8, D / 16, false>(s.c, a, sm, LD);
  warp_mm<D / 8, D / 16, false>(s.c, a, sm + D * LD, LD);
  bf16* z = (bf16*)(ws + w.z) + row * D;
  s.store(z, rest ? z + zstep : nullptr);
}

// ---- merge: the diagonal's state, earlier blocks' parts, cached parts; one warp per (token, query head) ----
// Bound: the parts' bytes (2048 tokens x 32 heads at head dim 128: 150 MB, from L2), and where there are few chunks the
// latency of a row's loads.  Rows of a block: a chunk's 64, or 16 below 1024 (chunk, head) pairs (4 x 100 tokens x 8 heads
// 230 -> 220 us for the call; 16 x 1700 x 32, with 13000 pairs, 1810 with 64 and 1923 with 16).
constexpr int GT = 256;
template <int D>
__global__ void __launch_bounds__(GT) merge_kernel(PagedArgs p, NewWs w, TcPlan pl, int GR, const char* ws) {
  chain();
  constexpr int L = D / 4, PG = 32 / L;  // lanes of a row; parts summed side by side
  const int c = blockIdx.x / (C / GR), qh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x4 = lane % L * 4, pg = lane / L;
  if (blockIdx.x == 0 && qh == 0 && threadIdx.x == 0 && *pl.err) paged_error(p.c.status, PATH_PAGED_WAIT + *pl.err);
  if (c >= pl.cstart[p.c.slots]) return;
  const int b = owner(pl.cstart, p.c.slots, c), H = p.c.heads;
  const SlotSpan sp = pass_span(p, b);
  const int lc = c - pl.cstart[b], rows = min(C, sp.n - lc * C), h = qh / p.G, g = qh % p.G;
  const int kt = live_tiles(sp.t0, p.window, p.sinks, kTcKeys).count;
  const int np = pl.pstart[b + 1] - pl.pstart[b];
  const long long per = units_per_block(pl, p.c.slots);
  const long long head = pl.ustart[b] + h * ((long long)np * kt + new_units(np, p.G));
  const float* cn = (const float*)(ws + w.cn) + ((size_t)h * w.nblk + pl.bstart[b]) * MB + lc * C;
  int pair = -1, n1 = 0, n = 0;
  long long from1 = 0, from2 = 0;
#pragma unroll 2
  for (int r = blockIdx.x % (C / GR) * GR + warp, r1 = min(rows, r - warp + GR); r < r1; r += GT / 32) {
    const size_t row = ((size_t)c * p.hq + qh) * C + r;
    const int R = (lc * C + r) * p.G + g;
    const float m0 = ((const float*)(ws + w.m))[row], l0 = ((const float*)(ws + w.l))[row];
    const float4 v0 = *reinterpret_cast<const float4*>((const float*)(ws + w.acc) + row * D + x4);
    const float bias = p.log_f ? cn[r] * kLog2e : 0.f;
    if (R / kTcPair != pair) {  // the pair's units: cached tiles, then those of earlier blocks; their parts
      pair = R / kTcPair;
      const int blk = pair / p.G;
      const long long us = head + (long long)pair * kt + new_units(pair, p.G);
      from1 = from2 = 2 * ((long long)pl.pstart[b] * H + (long long)h * np + pair);
      n1 = n = 0;
      if (kt > 0) {
        const long long f = us / per;
        n = n1 = (int)((us + kt - 1) / per - f + 1);
        from1 += f;
      }
      if (blk > 0) {
        const long long f = (us + kt) / per;
        n += (int)((us + kt + 2 * blk - 1) / per - f + 1);
        from2 += f + 1 - n1;
      }
    }
    auto at = [&](int x) { return (size_t)((x < n1 ? from1 : from2) + x) * kTcPair + R % kTcPair; };
    // maxima and sums of up to 32 parts at a time, one per lane; the first parts' rows set out beside them
    constexpr int AHEAD = 4 / PG;
    float4 v[AHEAD];
#pragma unroll
    for (int y = 0; y < AHEAD; ++y)
      v[y] = y * PG + pg < n ? *reinterpret_cast<const float4*>(pl.acc + at(y * PG + pg) * D + x4) : make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = lane < n ? pl.m[at(lane)] + bias : -INFINITY;
    const float lx = lane < n ? pl.l[at(lane)] : 0.f;
    float M = fmaxf(m0, mx);
    for (int x = lane + 32; x < n; x += 32) M = fmaxf(M, pl.m[at(x)] + bias);
    M = group_max<32>(M);
    const float f0 = fast_exp2(m0 - M);
    float4 a = pg == 0 ? make_float4(v0.x * f0, v0.y * f0, v0.z * f0, v0.w * f0) : make_float4(0.f, 0.f, 0.f, 0.f);
    float fx = mx == -INFINITY ? 0.f : fast_exp2(mx - M);  // (-inf: a part that saw nothing)
    float l = lx * fx;
#pragma unroll
    for (int y = 0; y < AHEAD; ++y) {
      const float f = __shfl_sync(0xffffffffu, fx, y * PG + pg);
      a.x += v[y].x * f;
      a.y += v[y].y * f;
      a.z += v[y].z * f;
      a.w += v[y].w * f;
    }
    for (int x0 = AHEAD * PG; x0 < n; x0 += PG) {
      const int x = x0 + pg;
      float f;
      if (x0 < 32) {
        f = __shfl_sync(0xffffffffu, fx, x);
      } else {
        const float ms = x < n ? pl.m[at(x)] + bias : -INFINITY;
        f = ms == -INFINITY ? 0.f : fast_exp2(ms - M);
        if (lane % L == 0 && x < n) l += pl.l[at(x)] * f;
      }
      if (x < n) {
        const float4 w4 = *reinterpret_cast<const float4*>(pl.acc + at(x) * D + x4);
        a.x += w4.x * f;
        a.y += w4.y * f;
        a.z += w4.z * f;
        a.w += w4.w * f;
      }
    }
    l = group_sum<32>(l) + l0 * f0;
    if (PG == 2) {
      a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
      a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
      a.z += __shfl_xor_sync(0xffffffffu, a.z, 16);
      a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
    }
    if (pg == 0) {
      const float inv = 1.f / l;
      bf16* o = (bf16*)p.o + (((size_t)sp.q0 + lc * C + r) * p.hq + qh) * D + x4;
      *reinterpret_cast<uint2*>(o) = make_uint2(pack2(a.x * inv, a.y * inv), pack2(a.z * inv, a.w * inv));
    }
  }
}

template <int D>
cudaError_t new_t(PagedArgs p, char* ws, cudaStream_t st) {
  const NewWs w = new_ws(p);
  const int H = p.c.heads;
  const bool fox = p.log_f != nullptr;
  cudaError_t e;
  auto prep = prep_kernel<D>;
  auto c1 = carry_in_block_kernel<D>;
  auto qk = fox ? query_kernel<D, true> : query_kernel<D, false>;
  auto sk = start_kernel<D>;
  const size_t s1 = sizeof(PrepSmem<D>), s2 = carry_smem<D>(), s3 = QSmem<D>::bytes;
  const size_t s4 = (size_t)(2 * D + 128) * (D + 8) * 2;
  const auto big = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(prep, big, (int)s1)) != cudaSuccess || (e = cudaFuncSetAttribute(c1, big, (int)s2)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(qk, big, (int)(s3 > s2 ? s3 : s2))) != cudaSuccess ||
      (e = cudaFuncSetAttribute(sk, big, (int)s4)) != cudaSuccess)
    return e;
  TcPlan pl{};
  pl.group = w.group;
  pl.mstart = (int*)(ws + w.mstart);
  pl.pairs = w.pairs;
  pl.blocks = w.nblk;
  pl.cstart = (int*)(ws + w.cstart);
  pl.bstart = (int*)(ws + w.bstart);
  pl.pstart = (int*)(ws + w.pstart);
  pl.rstart = (int*)(ws + w.rstart);
  pl.vstart = (long long*)(ws + w.vstart);
  pl.ustart = (long long*)(ws + w.ustart);
  pl.m = (float*)(ws + w.pm);
  pl.l = (float*)(ws + w.pl);
  pl.acc = (float*)(ws + w.pacc);
  pl.cn = (const float*)(ws + w.cn);
  pl.z = ws + w.z;
  pl.zs = ws + w.zs;
  pl.ver = ws + w.ver;
  pl.ver_rows = w.ver_rows;
  pl.mm = ws + w.mm;
  pl.err = (int*)(ws + w.err);
  const bool many = p.max_new > MB;  // a slot may have a second block
  const unsigned carries = (unsigned)(w.nblk * H * (CPB + D / 64));
  const int gr = (long long)w.nch * p.hq < 1024 ? 16 : C;
  for (int first = 0; first < w.most; first += w.group)
    for (p.skip = 0; p.skip < p.max_new; p.skip += kTcPassTokens) {
      if ((e = launch_chained(plan_kernel, 1, 1024, 0, st, p, pl, first, w.most, first == 0 && p.skip == 0)) != cudaSuccess ||
          (e = launch_chained(prep, dim3(w.nch, H), PT, s1, st, p, w, pl, ws)) != cudaSuccess ||
          (e = launch_chained(c1, carries + (fox ? w.group * H : 0), WT, s2, st, p, w, pl, ws)) != cudaSuccess ||
          (e = launch_chained(qk, carries + w.nch * p.hq, WT, s3 > s2 ? s3 : s2, st, p, w, pl, ws)) != cudaSuccess)
        return e;
      if (many && (e = launch_chained(sk, dim3(w.pairs * 4, H), WT, s4, st, p, w, pl, ws)) != cudaSuccess) return e;
      if ((e = launch_attend_tc(p, pl, st)) != cudaSuccess || (e = launch_rewrite_tc(p, pl, st)) != cudaSuccess ||
          (e = launch_chained(merge_kernel<D>, dim3(w.nch * (C / gr), p.hq), GT, 0, st, p, w, pl, gr, ws)) != cudaSuccess)
        return e;
    }
  return cudaSuccess;
}

}  // namespace

size_t paged_new_ws_bytes(const PagedArgs& p) {
  const NewWs w = new_ws(p);
  return round_bytes(w.total, w.group < w.most);
}
cudaError_t launch_paged_new(const PagedArgs& p, char* ws, cudaStream_t st) {
  return p.c.head_dim == kHeadDim ? new_t<kHeadDim>(p, ws, st) : new_t<kHeadDimWide>(p, ws, st);
}

}  // namespace pathattn
