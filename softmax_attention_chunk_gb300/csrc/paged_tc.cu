// Paged serving of bf16 caches: attention of many queries over cached rows on the tensor cores (tcgen05).
//
// Mathematics: the queries come transported to the start of the call's new tokens (z, paged_chunk.cu), so the
// cached rows need no transport: s = z k~^T, softmax, o = P V, with the running maximum and sum of one pass.
// Row i G + g of a (slot, key head) is head g of new token i: the G query heads that share keys share tiles.
//
// Bound: the tensor cores and the exponentials (4 D flops and one exponential per query-key pair; the keys and
// values of a tile are read once per 256 query rows, from L2 after the first).  So one persistent block per SM with
// two 128-row query tiles: while the softmax threads of one tile work on its scores, the tensor core forms the
// other's.  Per step of 128 keys and tile:
//   S = Z K^T (both operands in shared memory), softmax by one thread per row, P (bf16) over the first half of S in
//   TMEM, O += P V with P as the TMEM operand.
// Warp 8 brings key and value tiles by TMA, one box per page piece (pages of 16 to 256 rows; the 128-byte swizzle
// repeats every 8 rows), into a ring, newest tiles first (with a forget gate the recent keys hold the maximum: oldest
// first, the reference rose at every step, 406 -> 296 us for 2048 tokens over 16384 with the gate).  Warps 9 and 10
// issue the MMAs of one query tile each and clear value rows that hold no cached token (their probabilities are 0,
// but 0 times what lies there has to be 0).  The (slot, head, query pair, key tile) units of a
// call are one list cut into equal runs, one per block; a run's share of a query pair leaves its softmax state in
// a part of the workspace, merged in list order by merge kernel with the new tokens' own state.
//
// Roundings: P to bf16 (its row sums are of the unrounded values), as the MMA takes it beside bf16 values.  z is a
// bf16 pair (rounded, rest; a second product into S) at head dim 64, where the tensor cores have the time (512 tokens over
// 8000 x 32 heads: 171 -> 179 us for the whole call), and at 128 for pairs of up to 128 rows, whose rest lies in the
// second tile's place; else it is rounded once.  With both, what is left of o's error is that of two bf16 roundings.
//
// Measured: 2048 tokens x 32 heads over 32768 rows at head dim 128 (1.1 TFLOP) 726 us, 1.5 PFLOP/s, 78 % of a large
// library product (tensor pipe 60 % of its cycles); 2048 x 32 over 16384 at head dim 64 (275 GFLOP) 370 us, 0.74 PFLOP/s:
// tensor pipe 48 %, exponentials 33 %, issue 39 %, no unit saturated, each tile's chain of score product, softmax and
// value product a latency.  Tried and slower (the 1.1 TFLOP case's whole call, 1003 us): two threads per row 1441,
// maximum first and a second pass for the exponentials 1297, loads of the next scores under way 1020, the second tile
// half a step behind 1064, P as a bf16 pair 1707, key steps of 64 (attention) 1027 against 862 at the time.  Copies at head
// dim 64 without the exponentials, the TMEM loads or nearly all MMAs take 1.05, 1.08 and 0.87 of the time.
#include "paged_tc.h"
#include "dev_common.cuh"
#include "tc_common.cuh"
#include "scan_common.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

namespace pathattn {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {
using namespace tc;

constexpr int KT = kTcKeys;
constexpr int NSOFT = 256, NTHREADS = NSOFT + 64, ATHREADS = NSOFT + 96;  // rewrite; attention
constexpr int NINFO = 8;      // key tiles whose masks and biases are kept: more than the ring runs ahead
constexpr float kTau = 8.f;   // lazy rescale threshold (log2 units)
constexpr uint32_t COL_S = 0, COL_O = 256;  // two tiles each: S 128 columns, O D columns
constexpr uint32_t TILE = 128 * 128;        // bytes of a 128 x 64 bf16 tile

template <int D, bool FOX>
struct __align__(1024) TcSmem {
  static constexpr int X = D / 64;
  static constexpr int NBUF = D == 64 ? 8 : FOX ? 4 : 5;  // what 227 KB hold
  static constexpr int ZT = D == 64 ? 4 : 2;  // query tiles: two, and (D = 64) what rounding left of them
  uint8_t z[ZT][X][TILE];
  uint8_t buf[NBUF][X][TILE];
  float aj[FOX ? NINFO : 1][FOX ? KT : 1];  // forget gate: running sums of the tile's rows
  float ar[FOX ? NINFO : 1][FOX ? KT : 1];  // and what fp32 left of them (cached rows of a cache that keeps it)
  alignas(16) float kbias[FOX ? 2 : 1][FOX ? 2 : 1][FOX ? KT : 4];  // the softmax threads' key biases (log2 units)
  uint32_t okmask[NINFO];       // 16-row groups of the tile that are there
  uint64_t info[NINFO];
  uint64_t full[NBUF], empty[NBUF];
  uint64_t z_full, z_empty, s_full[2], p_ready[2], o_full[2], o_read[2];
  uint32_t tmem_base;
};

// A run's share of one query pair: over cached rows, or over the slot's own earlier blocks.
struct Segment {
  bool own;                 // earlier blocks: keys in the version of the pair's block, values as packed
  int b, h, pair, rows;     // rows of the pair (1..256)
  int i0, i1;               // key tiles
  int t0;                   // rows there are: cached ones, or new ones before the block
  int base;                 // position of row 0: 0, or that of the first new token
  long long item, ver;      // number of the item; own: first row of the version
  SlotSpan sp;
  LiveTiles lt;
};
// The segment that starts at unit u, and the first unit behind it.
__device__ __forceinline__ Segment segment_at(const PagedArgs& p, const TcPlan& pl, long long u, long long u1, long long* next) {
  Segment s;
  int lo = 0, hi = p.c.slots;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.ustart[mid] <= u) lo = mid; else hi = mid;
  }
  s.b = lo;
  s.sp = pass_span(p, s.b);
  s.lt = live_tiles(s.sp.t0, p.window, p.sinks, KT);
  const int np = pl.pstart[s.b + 1] - pl.pstart[s.b], kt = s.lt.count, G = p.G;
  const long long each = (long long)np * kt + new_units(np, G), in = u - pl.ustart[s.b];
  s.h = (int)(in / each);
  long long r = in % each;
  int m = 0;  // the pair's block: its units start behind those of m G pairs
  while ((m + 1) * G < np && (long long)(m + 1) * G * kt + new_units((long long)(m + 1) * G, G) <= r) ++m;
  r -= (long long)m * G * kt + new_units((long long)m * G, G);
  const int of_pair = kt + 2 * m;
  s.pair = m * G + (int)(r / of_pair);
  s.i0 = (int)(r % of_pair);
  s.own = s.i0 >= kt;
  int count = kt;
  if (!s.own) {
    s.t0 = s.sp.t0;
    s.base = 0;
    s.ver = 0;
  } else {
    s.i0 -= kt;
    count = 2 * m;
    s.t0 = m * kTcBlockTokens;
    s.base = s.sp.t0;
    s.lt = LiveTiles{count, 0, count};
    const long long nb = (s.sp.n + kTcBlockTokens - 1) / kTcBlockTokens;
    s.ver = pl.vstart[s.b] + s.h * (kTcBlockTokens / 2) * nb * (nb - 1) + (long long)(kTcBlockTokens / 2) * m * (m - 1);
  }
  const long long left = u1 - u;
  s.i1 = left < count - s.i0 ? s.i0 + (int)left : count;
  s.rows = min(256, s.sp.n * G - s.pair * 256);
  s.item = 2 * ((long long)pl.pstart[s.b] * p.c.heads + (long long)s.h * np + s.pair) + (s.own ? 1 : 0);
  *next = u + (s.i1 - s.i0);
  return s;
}

// A value that is the same in all lanes, in a uniform register (a warp reduction leaves its result in one): the
// MMA takes its descriptors from uniform registers, and what is not known to be uniform is moved there anew for
// every instruction.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
// The tcgen05 instructions of tc_common.cuh issued by one elected lane of a converged warp.
__device__ __forceinline__ void mma_ss_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_elect(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

template <int D, bool FOX>
__global__ void __launch_bounds__(ATHREADS, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_zs,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_ver, const __grid_constant__ CUtensorMap tm_new, const PagedArgs p,
                     const TcPlan pl) {
  chain();
  extern __shared__ uint8_t smem_raw[];
  using Smem = TcSmem<D, FOX>;
  constexpr int X = Smem::X, NBUF = Smem::NBUF;
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long units = pl.ustart[p.c.slots];
  const long long per = units_per_block(pl, p.c.slots);
  const long long u0 = per * blockIdx.x, u1 = u0 + per < units ? u0 + per : units;
  if (u0 >= u1) return;
  if (tid == 0) {
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 2);  // one arrival per query tile
    }
    for (int i = 0; i < NINFO; ++i) mbar_init(&s.info[i], 1);
    mbar_init(&s.z_full, 1);
    mbar_init(&s.z_empty, 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s.s_full[t], 1);
      mbar_init(&s.p_ready[t], 128);
      mbar_init(&s.o_full[t], 1);
      mbar_init(&s.o_read[t], 128);
    }
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(&s.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.tmem_base;
  int* err = pl.err;

  if (warp == 8) {
    // ---------------- producer: Z once per segment, key and value tiles ----------------
    const int P = p.c.page_size, RB = P < KT ? P : KT, nl = KT / RB;
    int n = 0, kk = 0, seg = 0;  // buffers, key tiles and segments so far
    bool ok = true;
    for (long long u = u0; ok && u < u1;) {
      const Segment g = segment_at(p, pl, u, u1, &u);
      if (seg > 0) ok = mbar_wait_lean(&s.z_empty, (seg - 1) & 1, err, 1);
      if (!ok) break;
      if (lane == 0) {
        // rows 0..127, 128..255 and the rests, or (D = 128) of up to 128 rows the rest in the place of the second tile
        const int zr = (g.h * pl.pairs + pl.pstart[g.b] + g.pair) * 256, ze = p.c.heads * pl.pairs * 256 + zr;
        mbar_arrive_expect_tx(&s.z_full, Smem::ZT * X * TILE);
        for (int i = 0; i < Smem::ZT; ++i)
          for (int x = 0; x < X; ++x)
            tma_load_2d(s.z[i][x], g.own ? &tm_zs : &tm_z, 64 * x,
                        D == 64 ? (i < 2 ? zr : ze) + i % 2 * 128 : i == 0 ? zr : g.rows > 128 ? zr + 128 : ze, &s.z_full);
      }
      ++seg;
      // the pair's first token sees the farthest back
      const int p_min = g.sp.t0 + g.pair * 256 / p.G;
      for (int i = g.i0; i < g.i1; ++i, ++kk) {
        const int j0 = newest_tile(g.lt, i) * KT;
        const int j = j0 + 16 * lane;
        int kp = -1, vp = -1;
        bool here = lane < 8 && j < g.t0 &&
                    (p.window <= 0 || g.base + j < p.sinks || g.base + j + 15 > p_min - p.window);
        if (here && !g.own) {
          kp = p.c.k_table[(size_t)g.b * p.c.table_width + j / P];
          vp = p.c.v_table[(size_t)g.b * p.c.table_width + j / P];
          if ((unsigned)kp >= (unsigned)p.c.k_pages || (unsigned)vp >= (unsigned)p.c.v_pages) {
            here = false;
            paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
          }
        }
        const uint32_t groups = __ballot_sync(0xffffffffu, here);
        // lane l brings piece l of the tile: a page's rows (the first group that is there names the page), or the
        // whole tile of an earlier block
        const int pr = g.own ? KT : RB, pieces = g.own ? 1 : nl, sub = pr / 16;
        const uint32_t mine = lane < pieces ? (groups >> (lane * sub)) & ((1u << sub) - 1) : 0u;
        const int from = mine ? lane * sub + __ffs(mine) - 1 : lane;
        kp = __shfl_sync(0xffffffffu, kp, from);
        vp = __shfl_sync(0xffffffffu, vp, from);
        const uint32_t loads = __popc(__ballot_sync(0xffffffffu, mine != 0));
        const int in = (j0 + lane * RB) % P;
        const int kb = n % NBUF, vb = (n + 1) % NBUF, ib = kk % NINFO;
        if (n >= NBUF) ok = ok && mbar_wait_lean(&s.empty[kb], (n / NBUF - 1) & 1, err, 2);
        if (!ok) break;
        if (lane == 0) {
          s.okmask[ib] = groups;
          if (FOX) mbar_arrive_expect_tx(&s.info[ib], loads * pr * (!g.own && p.c.a_rest ? 8 : 4));
          else mbar_arrive(&s.info[ib]);
          mbar_arrive_expect_tx(&s.full[kb], loads * pr * 128 * X);
        }
        __syncwarp();
        if (mine) {
          const int y = g.own ? (int)(g.ver + j0) : (kp * p.c.heads + g.h) * P + in;
          const void* map = g.own ? (const void*)&tm_ver : (const void*)&tm_k;
#pragma unroll
          for (int x = 0; x < X; ++x) tma_load_2d(s.buf[kb][x] + lane * pr * 128, map, 64 * x, y, &s.full[kb]);
          if (FOX) {
            const float* a = g.own ? pl.cn + ((size_t)g.h * pl.blocks + pl.bstart[g.b]) * kTcBlockTokens + j0
                                   : p.c.a_pool + ((size_t)vp * p.c.heads + g.h) * P + in;
            bulk_load(s.aj[ib] + lane * pr, a, pr * 4, &s.info[ib]);
            if (!g.own && p.c.a_rest) bulk_load(s.ar[ib] + lane * pr, p.c.a_rest + (a - p.c.a_pool), pr * 4, &s.info[ib]);
          }
        }
        if (n + 1 >= NBUF) ok = mbar_wait_lean(&s.empty[vb], ((n + 1) / NBUF - 1) & 1, err, 3);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&s.full[vb], loads * pr * 128 * X);
        __syncwarp();
        if (mine) {
          const int y = g.own ? g.sp.q0 + j0 : (vp * p.c.heads + g.h) * P + in;
          const void* map = g.own ? (const void*)&tm_new : (const void*)&tm_v;
          const int x0 = g.own ? g.h * D : 0;
#pragma unroll
          for (int x = 0; x < X; ++x) tma_load_2d(s.buf[vb][x] + lane * pr * 128, map, x0 + 64 * x, y, &s.full[vb]);
        }
        n += 2;
      }
    }
    // after a failure: no copy may land in shared memory once the block has gone (bounded waits)
    if (!ok) {
      if (seg > 0) mbar_wait_ns(&s.z_full, (seg - 1) & 1, nullptr, 0, 1000000ull);
      for (int i = n > NBUF ? n - NBUF : 0; i < n + 2; ++i) mbar_wait_ns(&s.full[i % NBUF], (i / NBUF) & 1, nullptr, 0, 1000000ull);
      for (int i = kk > NINFO ? kk - NINFO : 0; i <= kk; ++i) mbar_wait_ns(&s.info[i % NINFO], (i / NINFO) & 1, nullptr, 0, 1000000ull);
    }
  } else if (warp == 9 || warp == 10) {
    // ---------------- MMA issuer of tile t (a converged warp; one elected lane issues) ----------------
    const int t = warp - 9;
    const uint32_t idesc_s = idesc_bf16(128, KT, 0, 0), idesc_o = idesc_bf16(128, D, 0, 1);
    const uint64_t dz = sdesc_sw128(0, 1024, 16), dv = sdesc_sw128(0, 1024, TILE);
    const uint32_t a_z = uniform(smem_u32(s.z[t][0]) >> 4), a_b = uniform(smem_u32(s.buf[0][0]) >> 4), tbu = uniform(tb);
    const uint32_t d_s = tbu + COL_S + 128 * uniform(t), d_o = tbu + COL_O + D * uniform(t);
    int n = 0, kk = 0, seg = 0, np = 0, os = 0;  // buffers, key tiles, segments; probability tiles and segments of this tile
    bool ok = true;
    auto issue_s = [&](int buf, bool rest) {
      const uint64_t za = dz + a_z, kb = dz + a_b + uniform(buf * X * (TILE / 16));
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss_elect(d_s, za + (uint64_t)(x * (TILE / 16) + 2 * k), kb + (uint64_t)(x * (TILE / 16) + 2 * k), idesc_s, (x | k) ? 1u : 0u);
      if (rest)  // two tiles on, or in the second's place
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss_elect(d_s, za + (uint64_t)((2 + x) * (TILE / 16) + 2 * k), kb + (uint64_t)(x * (TILE / 16) + 2 * k), idesc_s, 1u);
      mma_commit_elect(&s.s_full[t]);
      mma_commit_elect(&s.empty[buf]);
    };
    for (long long u = u0; ok && u < u1; ++seg) {
      const Segment g = segment_at(p, pl, u, u1, &u);
      const int nk = g.i1 - g.i0;
      if (t == 1 && g.rows <= 128) {  // no second tile: the buffers' phases still end with this warp's arrivals
        for (int k = 0; ok && k < 2 * nk; ++k) {
          ok = mbar_wait_lean(&s.full[(n + k) % NBUF], ((n + k) / NBUF) & 1, err, 4);
          if (ok && lane == 0) mbar_arrive(&s.empty[(n + k) % NBUF]);
        }
        if (ok) ok = mbar_wait_lean(&s.z_full, seg & 1, err, 4);
        if (ok && lane == 0) mbar_arrive(&s.z_empty);
        n += 2 * nk;
        kk += nk;
        continue;
      }
      ok = mbar_wait_lean(&s.z_full, seg & 1, err, 4) && mbar_wait_lean(&s.full[n % NBUF], (n / NBUF) & 1, err, 5);
      if (!ok) break;
      tc_fence_after();
      const bool rest = D == 64 || g.rows <= 128;
      issue_s(n % NBUF, rest);
      if (nk == 1) mma_commit_elect(&s.z_empty);
      for (int k = 0; ok && k < nk; ++k, ++kk, n += 2) {
        const int vb = (n + 1) % NBUF, nb = (n + 2) % NBUF;
        ok = mbar_wait_lean(&s.full[vb], ((n + 1) / NBUF) & 1, err, 6);
        if (!ok) break;
        const int j0 = newest_tile(g.lt, g.i0 + k) * KT;
        // (the tile's mask: written by the producer before it arrived for the key buffer, which this warp has
        // waited for)
        const uint32_t groups = *reinterpret_cast<volatile uint32_t*>(&s.okmask[kk % NINFO]);
        if (groups != 0xffu || j0 + KT > g.t0) {  // (both tiles' warps write the same zeros)
          for (int r = lane >> 3; r < KT; r += 4)
            if (!(groups >> (r >> 4) & 1) || j0 + r >= g.t0)
#pragma unroll
              for (int x = 0; x < X; ++x) *reinterpret_cast<uint4*>(s.buf[vb][x] + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (k + 1 < nk) ok = mbar_wait_lean(&s.full[nb], ((n + 2) / NBUF) & 1, err, 9);
        ok = ok && mbar_wait_lean(&s.p_ready[t], np & 1, err, 7);
        if (ok && k == 0 && os > 0) ok = mbar_wait_lean(&s.o_read[t], (os - 1) & 1, err, 8);
        if (!ok) break;
        ++np;
        __syncwarp();
        tc_fence_after();
        const uint64_t vd = dv + a_b + uniform(vb * X * (TILE / 16));
        const uint32_t first = uniform(k == 0 ? 0u : 1u);
#pragma unroll
        for (int y = 0; y < KT / 16; ++y)
          mma_ts_elect(d_o, d_s + 8 * y, vd + (uint64_t)(128 * y), idesc_o, y == 0 ? first : 1u);
        if (k + 1 == nk) mma_commit_elect(&s.o_full[t]);
        if (k + 1 < nk) {
          issue_s(nb, rest);
          if (k + 2 == nk) mma_commit_elect(&s.z_empty);
        }
        mma_commit_elect(&s.empty[vb]);
      }
      ++os;
    }
  } else {
    // ---------------- softmax: thread = row of tile warp / 4 ----------------
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t c_s = tb + lane_off + COL_S + 128 * t, c_o = tb + lane_off + COL_O + D * t;
    int kk = 0, ns = 0, os = 0;
    bool ok = true;
    // (with the forget gate the tile's threads meet at a barrier every step: after a wait has given up they all walk
    // on to the end, without further waits)
    for (long long u = u0; (FOX || ok) && u < u1;) {
      const Segment g = segment_at(p, pl, u, u1, &u);
      const int nk = g.i1 - g.i0;
      if (t == 1 && g.rows <= 128) {  // no second tile
        kk += nk;
        continue;
      }
      const int R = g.pair * 256 + 128 * t + r;
      const int pos = g.sp.t0 + R / p.G;
      // positions of this warp's tile: a tile of keys that all of them see needs no mask
      const int p_max = g.sp.t0 + (g.pair * 256 + 128 * t + 127) / p.G;
      float a_last = 0.f, a_more = 0.f;
      const bool pairs = FOX && !g.own && p.c.a_rest;
      if (FOX && !g.own && g.sp.t0 > 0) {  // (own rows: the sums start at 0)
        const long long row = pool_row(p.c, p.c.v_table, p.c.v_pages, g.b, g.h, g.sp.t0 - 1);
        if (row >= 0) {
          a_last = p.c.a_pool[row];
          a_more = sum_rest(p.c, row);
        }
      }
      float m = -INFINITY, l = 0.f;
      for (int k = 0; (FOX || ok) && k < nk; ++k, ++kk, ++ns) {
        // (the scores first: with them the producer is known to be at most one phase of `info` ahead)
        ok = ok && mbar_wait_lean(&s.s_full[t], ns & 1, err, 10) && mbar_wait_lean(&s.info[kk % NINFO], (kk / NINFO) & 1, err, 11);
        if (!FOX && !ok) break;
        tc_fence_after();
        const int j0 = newest_tile(g.lt, g.i0 + k) * KT;
        const uint32_t groups = s.okmask[kk % NINFO];
        const bool mask = groups != 0xffu || j0 + KT > g.t0 ||
                          (p.window > 0 && g.base + j0 + KT > p.sinks && g.base + j0 <= p_max - p.window);
        // forget gate: the keys' biases, one per thread of the tile, doubly buffered by the barrier of the next step
        float* kb = s.kbias[FOX ? t : 0][FOX ? (ns & 1) : 0];
        if (FOX) {
          kb[r] = ((a_last - s.aj[kk % NINFO][r]) + (pairs ? a_more - s.ar[kk % NINFO][r] : 0.f)) * kLog2e;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
        }
        // bits of the keys 32 q .. 32 q + 31 that the row sees: there, and a first token or in the window
        auto visible = [&](int q) {
          auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
          const int o = j0 + 32 * q;
          uint32_t w = below(g.t0 - o);
          w &= ((groups >> (2 * q) & 1) ? 0xffffu : 0u) | ((groups >> (2 * q + 1) & 1) ? 0xffff0000u : 0u);
          if (p.window > 0) w &= below(p.sinks - (g.base + o)) | ~below(pos - p.window + 1 - (g.base + o));
          return w;
        };
        // One pass over the scores with the reference as it stands: probabilities (kept in registers, the scores stay
        // in TMEM), row sum and maximum.  Where a score exceeds the reference by more than 2^8 (the first tile, and
        // rarely later), the reference moves, O is rescaled and the pass is taken again.  (Two instances: the masks of
        // the rare tiles stay out of the others' instructions.)
        uint32_t pk[64];
        float sum = 0.f;
        auto step = [&](auto masked) {
          constexpr bool MASK = decltype(masked)::value;
          constexpr bool logd = FOX || MASK;  // scores in the log2 domain with biases and hidden ones -inf; else raw
          const float f = logd ? 1.f : p.scl;
          const bool low = !logd && p.scl < 0.f;  // the largest exponent is the smallest score
          for (int pass = 0; pass < 2; ++pass) {
            float e0, e1;
            e0 = e1 = low ? INFINITY : -INFINITY;
            const float mu = m == -INFINITY ? 0.f : m;
            uint64_t acc[2] = {0ull, 0ull};
            const uint64_t nm = f2(-mu, -mu), sc = f2(f, f), scl2 = f2(p.scl, p.scl);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t x[32];
              tmem_ld32(c_s + 32 * q, x);
              tmem_ld_wait();
              if (FOX) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(kb + 32 * q + j);
                  float v0, v1, v2, v3;
                  f2_split(f2_fma(f2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), scl2, bv.x), v0, v1);
                  f2_split(f2_fma(f2(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), scl2, bv.y), v2, v3);
                  x[j] = __float_as_uint(v0);
                  x[j + 1] = __float_as_uint(v1);
                  x[j + 2] = __float_as_uint(v2);
                  x[j + 3] = __float_as_uint(v3);
                }
              } else if (MASK) {
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * p.scl);
              }
              if (MASK) {
                const uint32_t w = visible(q);
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = (w >> j & 1) ? x[j] : 0xff800000u;
              }
              if (low) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  e0 = min3(e0, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                  e1 = min3(e1, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
                }
              } else {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  e0 = max3(e0, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                  e1 = max3(e1, __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
                }
              }
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float a0, a1;
                f2_split(f2_fma(f2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), sc, nm), a0, a1);
                const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
                acc[j & 1] = f2_add(acc[j & 1], f2(p0, p1));
                pk[16 * q + j] = pack_bf16(p0, p1);
              }
            }
            float s0, s1, s2, s3;
            f2_split(acc[0], s0, s1);
            f2_split(acc[1], s2, s3);
            sum = (s0 + s1) + (s2 + s3);
            const float mx = (low ? fminf(e0, e1) : fmaxf(e0, e1)) * f;
            const bool up = mx > m + kTau;
            if (!__any_sync(0xffffffffu, up)) break;
            const float mn = up ? fmaxf(m, mx) : m;
            const float corr = up ? fast_exp2(m - mn) : 1.f;  // (m = -inf at first: 0)
            m = mn;
            l *= corr;
            if (k > 0) {  // (S of this step was issued behind the last P V, which has completed with it)
#pragma unroll
              for (int q = 0; q < D / 32; ++q) {
                uint32_t ob[32];
                tmem_ld32(c_o + 32 * q, ob);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) ob[j] = __float_as_uint(__uint_as_float(ob[j]) * corr);
                tmem_st32(c_o + 32 * q, ob);
              }
            }
          }
        };
        if (mask) step(std::true_type{});
        else step(std::false_type{});
        l += sum;
        tmem_st32(c_s, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));  // over the scores
        tmem_st32(c_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&s.p_ready[t]);
      }
      ok = ok && mbar_wait_lean(&s.o_full[t], os & 1, err, 12);
      ++os;
      if (!FOX && !ok) break;
      tc_fence_after();
      const size_t row = (size_t)(g.item + blockIdx.x) * 256 + 128 * t + r;
      float* dst = pl.acc + row * D;
      const bool real = 128 * t + r < g.rows;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t ob[32];
        tmem_ld32(c_o + 32 * q, ob);
        tmem_ld_wait();
        if (real)
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<uint4*>(dst + 32 * q + j) = make_uint4(ob[j], ob[j + 1], ob[j + 2], ob[j + 3]);
      }
      if (real) {
        pl.m[row] = m;
        pl.l[row] = l;
      }
      tc_fence_before();
      mbar_arrive(&s.o_read[t]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// ---- cached rows: k <- k M ----
// Bound: HBM (each key read and written once, 4 D bytes) against 2 D^2 multiply-adds per row, M being a bf16 pair
// (high + rest: the only rounding left is the stored key's).  As warp MMAs these took 88 us for 8 x 32768 rows at
// head dim 128 where the bytes take 20; tcgen05 has four times their rate.  A persistent block per SM: a tile of 128
// rows by TMA, K M_high + K M_rest into one of two TMEM accumulators, one thread per row rounds and stores.
template <int D>
struct __align__(1024) RewSmem {
  static constexpr int X = D / 64;
  static constexpr int NBUF = D == 64 ? 8 : 4;
  uint8_t m[2][X][D * 128];     // M high, M rest: [D rows][64] per column half
  uint8_t buf[NBUF][X][TILE];
  uint64_t full[NBUF], empty[NBUF], m_full, m_empty, acc_full[2], acc_free[2];
  uint32_t tmem_base;
};
struct RewSegment {
  int b, h, i0, i1;
  SlotSpan sp;
  LiveTiles lt;
};
__device__ __forceinline__ RewSegment rew_segment(const PagedArgs& p, const TcPlan& pl, long long u, long long u1, long long* next) {
  RewSegment s;
  int lo = 0, hi = p.c.slots;
  const int at = (int)(u / p.c.heads);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.rstart[mid] <= at) lo = mid; else hi = mid;
  }
  s.b = lo;
  s.sp = pass_span(p, s.b);
  s.lt = live_tiles(s.sp.t0, p.window, p.sinks, kRewriteRows);
  const long long in = u - (long long)pl.rstart[s.b] * p.c.heads;
  s.h = (int)(in / s.lt.count);
  s.i0 = (int)(in % s.lt.count);
  const long long left = u1 - u;
  s.i1 = left < s.lt.count - s.i0 ? s.i0 + (int)left : s.lt.count;
  *next = u + (s.i1 - s.i0);
  return s;
}
template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
    rewrite_tc_kernel(const __grid_constant__ CUtensorMap tm_m, const __grid_constant__ CUtensorMap tm_k, const PagedArgs p,
                      const TcPlan pl) {
  chain();
  extern __shared__ uint8_t smem_raw[];
  using Smem = RewSmem<D>;
  constexpr int X = Smem::X, NBUF = Smem::NBUF;
  constexpr uint32_t COLS = D == 64 ? 128 : 256;
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = p.c.page_size;
  const long long units = (long long)pl.rstart[p.c.slots] * p.c.heads, per = (units + gridDim.x - 1) / gridDim.x;
  const long long u0 = per * blockIdx.x, u1 = u0 + per < units ? u0 + per : units;
  if (u0 >= u1) return;
  if (tid == 0) {
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.m_full, 1);
    mbar_init(&s.m_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s.acc_full[t], 1);
      mbar_init(&s.acc_free[t], 128);
    }
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(&s.tmem_base, COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.tmem_base;
  int* err = pl.err;
  // whether a later token sees row j of the cached rows
  auto keep = [&](const RewSegment& g, int j) { return j < g.sp.t0 && sees(p.window, p.sinks, g.sp.t0 + g.sp.n, j); };

  if (warp == 8) {
    const int RB = P < KT ? P : KT, nl = KT / RB;
    int n = 0, seg = 0;
    bool ok = true;
    for (long long u = u0; ok && u < u1; ++seg) {
      const RewSegment g = rew_segment(p, pl, u, u1, &u);
      if (seg > 0) ok = mbar_wait_lean(&s.m_empty, (seg - 1) & 1, err, 20);
      if (!ok) break;
      if (lane == 0) {
        const int m = pl.mstart[g.b];
        mbar_arrive_expect_tx(&s.m_full, 2 * X * D * 128);
        for (int v = 0; v < 2; ++v)
          for (int x = 0; x < X; ++x)
            tma_load_2d(s.m[v][x], &tm_m, 64 * x, ((v * pl.group + m) * p.c.heads + g.h) * D, &s.m_full);
      }
      for (int i = g.i0; i < g.i1; ++i, ++n) {
        const int j = live_tile(g.lt, i) * KT + lane * RB;
        // a piece comes if its page is there and a row of it is kept (rows of a piece are neighbours: its first tokens,
        // or its end, are the ones that may still be seen)
        int kp = -1;
        if (lane < nl && j < g.sp.t0 && (keep(g, j) || keep(g, min(j + RB, g.sp.t0) - 1))) {
          kp = p.c.k_table[(size_t)g.b * p.c.table_width + j / P];
          if ((unsigned)kp >= (unsigned)p.c.k_pages) {
            kp = -1;
            paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
          }
        }
        const uint32_t loads = __popc(__ballot_sync(0xffffffffu, kp >= 0));
        const int kb = n % NBUF;
        if (n >= NBUF) ok = mbar_wait_lean(&s.empty[kb], (n / NBUF - 1) & 1, err, 21);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&s.full[kb], loads * RB * 128 * X);
        __syncwarp();
        if (kp >= 0)
#pragma unroll
          for (int x = 0; x < X; ++x)
            tma_load_2d(s.buf[kb][x] + lane * RB * 128, &tm_k, 64 * x, (kp * p.c.heads + g.h) * P + j % P, &s.full[kb]);
      }
    }
    if (!ok) {  // (bounded: no copy may land once the block has gone)
      if (seg > 0) mbar_wait_ns(&s.m_full, (seg - 1) & 1, nullptr, 0, 1000000ull);
      mbar_wait_ns(&s.m_full, seg & 1, nullptr, 0, 1000000ull);
      for (int i = n > NBUF ? n - NBUF : 0; i <= n; ++i) mbar_wait_ns(&s.full[i % NBUF], (i / NBUF) & 1, nullptr, 0, 1000000ull);
    }
  } else if (warp == 9) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, D, 0, 1);
      const uint64_t da = sdesc_sw128(smem_u32(s.buf[0][0]), 1024, 16);
      const uint64_t db = sdesc_sw128(smem_u32(s.m[0][0]), 1024, D * 128);
      int n = 0, seg = 0;
      bool ok = true;
      for (long long u = u0; ok && u < u1; ++seg) {
        const RewSegment g = rew_segment(p, pl, u, u1, &u);
        ok = mbar_wait_lean(&s.m_full, seg & 1, err, 22);
        for (int i = g.i0; ok && i < g.i1; ++i, ++n) {
          const int kb = n % NBUF, t = n & 1;
          ok = mbar_wait_lean(&s.full[kb], (n / NBUF) & 1, err, 23);
          if (ok && n >= 2) ok = mbar_wait_lean(&s.acc_free[t], (n / 2 - 1) & 1, err, 24);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tb + D * t, da + (uint64_t)((kb * X + k / 4) * (TILE / 16) + 2 * (k % 4)),
                     db + (uint64_t)(v * X * (D * 128 / 16) + 128 * k), idesc, (v | k) ? 1u : 0u);
          mma_commit(&s.empty[kb]);
          mma_commit(&s.acc_full[t]);
        }
        if (ok) mma_commit(&s.m_empty);
      }
    }
  } else {
    const int t = warp >> 2, r = tid & 127;
    const uint32_t c_a = tb + ((uint32_t)((warp & 3) * 32) << 16) + D * t;
    int n = 0;
    bool ok = true;
    for (long long u = u0; ok && u < u1;) {
      const RewSegment g = rew_segment(p, pl, u, u1, &u);
      for (int i = g.i0; ok && i < g.i1; ++i, ++n) {
        if ((n & 1) != t) continue;
        const int j = live_tile(g.lt, i) * KT + r;
        __nv_bfloat16* dst = nullptr;
        if (keep(g, j)) {
          const long long at = pool_row(p.c, p.c.k_table, p.c.k_pages, g.b, g.h, j);
          if (at >= 0) dst = (__nv_bfloat16*)p.c.k_pool + at * D;
        }
        ok = mbar_wait_lean(&s.acc_full[t], (n / 2) & 1, err, 25);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t x[32];
          tmem_ld32(c_a + 32 * q, x);
          tmem_ld_wait();
          if (dst)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              *reinterpret_cast<uint4*>(dst + 32 * q + 8 * y) =
                  make_uint4(pack_bf16(__uint_as_float(x[8 * y]), __uint_as_float(x[8 * y + 1])),
                             pack_bf16(__uint_as_float(x[8 * y + 2]), __uint_as_float(x[8 * y + 3])),
                             pack_bf16(__uint_as_float(x[8 * y + 4]), __uint_as_float(x[8 * y + 5])),
                             pack_bf16(__uint_as_float(x[8 * y + 6]), __uint_as_float(x[8 * y + 7])));
        }
        tc_fence_before();
        mbar_arrive(&s.acc_free[t]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tb, COLS);
  }
}

// 2-D map over `rows` rows of `cols` bf16 with 128-byte swizzled boxes of box_rows x 64.
bool make_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FOX>
cudaError_t attend_t(const PagedArgs& p, const TcPlan& pl, cudaStream_t st) {
  CUtensorMap mz, mzs, mk, mv, mver, mnew;
  const int P = p.c.page_size, RB = P < KT ? P : KT;
  const uint64_t zrows = (uint64_t)p.c.heads * pl.pairs * kTcPair;
  const uint64_t zall = 2 * zrows;  // (rounded, rest)
  const bool own = pl.ver_rows > 0;  // (no version rows: no slot has a second block, the maps are not used)
  if (!make_map(&mz, pl.z, D, zall, 128) || !make_map(&mzs, pl.zs, D, zall, 128) ||
      !make_map(&mk, p.c.k_pool, D, (uint64_t)p.c.k_pages * p.c.heads * P, RB) ||
      !make_map(&mv, p.c.v_pool, D, (uint64_t)p.c.v_pages * p.c.heads * P, RB) ||
      !make_map(&mver, own ? pl.ver : pl.z, D, own ? (uint64_t)pl.ver_rows : zrows, KT) ||
      !make_map(&mnew, p.v, (uint64_t)p.c.heads * D, (uint64_t)p.total, KT))
    return cudaErrorInvalidValue;
  auto kern = attend_tc_kernel<D, FOX>;
  const size_t smem = sizeof(TcSmem<D, FOX>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, kTcBlocks, ATHREADS, smem, st, mz, mzs, mk, mv, mver, mnew, p, pl);
}

template <int D>
cudaError_t rewrite_t(const PagedArgs& p, const TcPlan& pl, cudaStream_t st) {
  CUtensorMap mm, mk;
  const int P = p.c.page_size, RB = P < KT ? P : KT;
  if (!make_map(&mm, pl.mm, D, (uint64_t)2 * pl.group * p.c.heads * D, D) ||
      !make_map(&mk, p.c.k_pool, D, (uint64_t)p.c.k_pages * p.c.heads * P, RB))
    return cudaErrorInvalidValue;
  auto kern = rewrite_tc_kernel<D>;
  const size_t smem = sizeof(RewSmem<D>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, kTcBlocks, NTHREADS, smem, st, mm, mk, p, pl);
}

}  // namespace

cudaError_t launch_rewrite_tc(const PagedArgs& p, const TcPlan& pl, cudaStream_t st) {
  return p.c.head_dim == kHeadDim ? rewrite_t<kHeadDim>(p, pl, st) : rewrite_t<kHeadDimWide>(p, pl, st);
}

cudaError_t launch_attend_tc(const PagedArgs& p, const TcPlan& pl, cudaStream_t st) {
  const bool fox = p.log_f != nullptr;
  if (p.c.head_dim == kHeadDim) return fox ? attend_t<kHeadDim, true>(p, pl, st) : attend_t<kHeadDim, false>(p, pl, st);
  return fox ? attend_t<kHeadDimWide, true>(p, pl, st) : attend_t<kHeadDimWide, false>(p, pl, st);
}

}  // namespace pathattn
