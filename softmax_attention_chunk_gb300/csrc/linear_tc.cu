// Linear attention on the tensor cores (bf16): the walk of linear.h in chunks of 128 tokens, one block per key head and segment.
// Of a chunk, with r the row and m the rows that are tokens,
//   S = X Y^T,  O = X State (tcgen05),  P = S masked and weighted with g^(distance), O scaled by g^(distance to the state),
//   O += P Z,  Delta^T = Z^T Y', Y' = Y weighted with g^(distance to the chunk's end),  State = g^m State + Delta.
// State is float32 in registers, transposed (a thread holds a part of a column); the operand of the next chunk is its copy as
// two bf16 numbers.  P goes back to tensor memory over S, Y' to shared memory over Y.
//
// One warp moves tiles (TMA), one issues every product, the others (a row and 32 columns of O per thread) do the rest; they meet
// at mbarriers only.  S of the next chunk is issued as soon as P has been read; the warps whose part of P is all masked weigh Y
// meanwhile.  The chain from chunk to chunk is P, P Z and Delta, State and the product with it.
//
// Roundings beside the output's: P and Y' to bf16, the operands' type (relative 2^-8; what reaches an output is the sum of
// independent ones; of few sequences of one chunk P is two bf16 numbers).  Where the state is an output itself (serving) Y' is
// the sum of three bf16 numbers, as exact as float32.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "dev_common.cuh"
#include "linear.h"
#include "tc_common.cuh"

namespace pathattn {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // fwd_tc.cu

namespace {

using namespace tc;

constexpr int C = 128, TILE = C * 128;
constexpr int COL_S = 0, COL_O = 128;   // tensor memory: S and P, O, then Delta
constexpr int Z0 = 32;                  // zeros before g^0 in the table

struct LinMaps {
  CUtensorMap x[3], y[3], z[3], o[3];
};

template <int D> struct Shape {
  static constexpr int X = D / 64;          // 64-column tiles of a row block
  static constexpr int CG = D / 32;         // column groups: a warp of each to every 32 rows
  static constexpr int WARPS = 4 * CG;      // computing warps; one more issues, one moves tiles
  static constexpr int LIGHT = 2;           // (head dim 64) warps whose part of P is all masked
  static constexpr int NT = 32 * (WARPS + 2);
  static constexpr int BLOCKS = D == 64 ? 2 : 1;  // to an SM
  static constexpr int NO = D == 64 ? 1 : 2;      // buffers of O
  static constexpr int COL_D = COL_O + NO * D, COLS = D == 64 ? 256 : 512;
};
template <int D, int PARTS> struct Smem {
  // Buffers: what the block's share of 227 KB holds.  O leaves through x's place once x has been read; before that the second
  // part of Y' lies there, the third has a place of its own.
  static constexpr int X = D / 64, NX = PARTS == 1 ? 2 : 1, NY = 2, NZ = D == 64 ? 2 : 1, NE = PARTS == 3 ? 1 : 0;
  uint8_t x[NX][X][TILE], y[NY][X][TILE], z[NZ + NE][X][TILE];
  uint8_t sb[2][X][D * 128];                // the state, rows of D columns: rounded, and what that leaves
  float pw[Z0 + C + 4];                     // 0 .., then g^n
  float2 keep[2];                           // g^n of a whole chunk and of the last one
  alignas(16) float colw[32];               // g^n of a 32-column block's columns
  // A wait looks at the parity of a phase: none of these may complete two phases while someone still waits for the first.  So
  // what frees or fills one of several buffers has a barrier for each.
  uint64_t full_x[NX], full_y[NY], full_z[2], yz_free[2], out_full[NX];
  uint64_t clean, s_full, o_full, d_full, t_full, c_full, w_full, p_full, done;
  uint32_t tmem_base;
};

__device__ __forceinline__ uint64_t f2_bits(uint32_t a, uint32_t b) { return (uint64_t)b << 32 | a; }
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) { return pack_bf16(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
// Four products in a row, of operands AS and BS (16-byte units) apart, issued by one elected lane of a converged warp; the
// first adds to D where accumulate is set.
template <int AS, int BS> __device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, %5;\n\tadd.s64 b1, %2, %6;\n\t"
      "add.s64 a2, %1, 2 * %5;\n\tadd.s64 b2, %2, 2 * %6;\n\t"
      "add.s64 a3, %1, 3 * %5;\n\tadd.s64 b3, %2, 3 * %6;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(AS), "n"(BS)
      : "memory");
}
// The same with A in tensor memory, at a0 .. a3.
template <int BS> __device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "add.s64 b1, %5, %8;\n\tadd.s64 b2, %5, 2 * %8;\n\tadd.s64 b3, %5, 3 * %8;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %6, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], b1, %6, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], b2, %6, t;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], b3, %6, t;\n\t}" ::"r"(d),
      "r"(a0), "r"(a1), "r"(a2), "r"(a3), "l"(b), "r"(idesc), "r"(accumulate), "n"(BS)
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// 16 bytes of Y (8 columns of a row), weighted, as a sum of PARTS bf16 numbers.
template <int PARTS> __device__ __forceinline__ void weighted(uint4 y, float w, uint4 (&out)[PARTS]) {
  const uint32_t in[4] = {y.x, y.y, y.z, y.w};
  uint32_t o[PARTS][4];
  const uint64_t ww = f2(w, w), minus = f2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t v = f2_mul(f2_bits(in[i] << 16, in[i] & 0xffff0000u), ww);
#pragma unroll
    for (int t = 0; t < PARTS; ++t) {
      o[t][i] = pack_pair(v);
      if (t + 1 < PARTS) v = f2_fma(f2_bits(o[t][i] << 16, o[t][i] & 0xffff0000u), minus, v);
    }
  }
#pragma unroll
  for (int t = 0; t < PARTS; ++t) out[t] = make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
}

// FINE: P as two bf16 numbers.
template <int D, bool STATES, int PARTS, bool FINE>
__global__ void __launch_bounds__(Shape<D>::NT, Shape<D>::BLOCKS)
    linear_tc_kernel(const __grid_constant__ LinMaps maps, const LinArgs p) {
  chain();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using Sh = Shape<D>;
  using Sm = Smem<D, PARTS>;
  constexpr int X = Sh::X, NX = Sm::NX, NY = Sm::NY, NCT = 32 * Sh::WARPS, COL_D = Sh::COL_D;
  constexpr int NZ = STATES && PARTS == 1 ? 2 : Sm::NZ;  // (states alone: x's place is z's second buffer)
  constexpr int NF = NZ < NY ? NZ : NY;       // of y and z together: the next of the same number waits for the one before
  constexpr int NS = D == 64 ? 16 : 32;       // state elements of a thread
  constexpr int SW = C / Sh::CG, SQ = SW / 32;  // columns of S of a warp
  Sm& s = *reinterpret_cast<Sm*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, cg = warp >> 2;
  const bool lead = warp == Sh::WARPS, mover = warp == Sh::WARPS + 1;
  // At head dim 64 the warps whose part of P is all masked weigh Y while the others make P; else every computing warp does,
  // after P (head dim 128, 4 x 16 x 2048: forward 59 us in place of 70 with six of sixteen warps).
  constexpr bool ALL = STATES || PARTS > 1 || D == 128;
  int blk = blockIdx.x;  // (neighbouring blocks, the gradients of one head, share operands)
  const int kinds = STATES ? p.slots : p.ops, oi = STATES ? p.maker[blk % kinds] : blk % kinds;
  blk /= kinds;
  const int h = blk % p.heads, item = blk / p.heads;
  const LinOp& op = p.op[oi];
  const LinItem it = lin_item(p, item);
  if (it.seg < 0) return;
  if (smem_u32(smem_raw) & 1023) {  // (swizzled tiles begin on 1024 bytes)
    if (tid == 0) {
      atomicCAS(p.err, 0, PATH_PAGED_WAIT + 16);
      if (p.status) paged_error(p.status, PATH_PAGED_WAIT + 16);
    }
    return;
  }
  const bool rev = op.reverse != 0;
  const int gx = op.gx, gy = op.gy, G = STATES || gy > gx ? gy : gx;
  const float l2 = lin_log2(p.log_decay[h]);
  // chunks of the segment: in tokens, segments and chunks begin at multiples of their lengths
  const int nch = (it.n + C - 1) / C, per = p.seg / C, nseg = (nch + per - 1) / per;
  const int c0 = (rev ? nseg - 1 - it.seg : it.seg) * per, count = min(per, nch - c0);
  const int steps = count * G;
  // S of step i: with several y to an x, O's second buffer is S's, and the next S does not wait for P to be read
  const bool two_s = Sh::NO > 1 && gy > 1;
  auto s_col = [&](int i) { return two_s && i % 2 ? COL_O + D : COL_S; };
  auto chunk_of = [&](int k) { return rev ? c0 + count - 1 - k : c0 + k; };
  auto rows_of = [&](int k) { return min(C, it.n - chunk_of(k) * C); };
  auto ragged = [&](int k) { return p.packed && rows_of(k) < C; };  // (the last chunk of a walk onwards)

  if (tid == 0) {
    for (int i = 0; i < NX; ++i) mbar_init(&s.full_x[i], 1);
    for (int i = 0; i < NY; ++i) mbar_init(&s.full_y[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.full_z[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&s.yz_free[i], 1);
    for (int i = 0; i < NX; ++i) mbar_init(&s.out_full[i], Sh::WARPS);
    mbar_init(&s.s_full, 1);
    mbar_init(&s.o_full, 1);
    mbar_init(&s.d_full, 1);
    mbar_init(&s.t_full, 1);
    mbar_init(&s.c_full, 1);
    mbar_init(&s.clean, Sh::WARPS);
    mbar_init(&s.w_full, ALL ? Sh::WARPS : Sh::LIGHT);
    mbar_init(&s.p_full, Sh::WARPS);
    mbar_init(&s.done, Sh::WARPS);
    fence_barrier_init();
  }
  if (lead) tmem_alloc(&s.tmem_base, Sh::COLS);
  if (tid < Z0 + C + 1) s.pw[tid] = tid < Z0 ? 0.f : exp2f(l2 * (tid - Z0));
  if (tid < 32) s.colw[tid] = exp2f(l2 * (rev ? tid : 31 - tid));
  if (tid < 2) s.keep[tid] = lin_decay(p.log_decay[h], tid == 0 ? C : it.n - (nch - 1) * C);
  const size_t dd = (size_t)D * D;
  float* part = p.parts + (((size_t)op.slot * p.items + item) * p.heads + h) * dd;
  float* own = p.state ? p.state + ((size_t)it.seq * p.heads + h) * dd : nullptr;
  const bool split = p.max_new > p.seg;  // the segments' starting states are in parts
  const float* from = STATES ? nullptr : split ? part : own;
  // this thread's part of the state: column sv, rows sk ..
  const int sv = D == 64 ? 16 * quad + (lane & 15) : 32 * quad + lane;
  const int sk = D == 64 ? 32 * (lane >> 4) + 16 * cg : 32 * cg;
  uint64_t st[NS / 2];  // pairs of floats
  auto put_state = [&]() {
    const uint64_t minus = f2(-1.f, -1.f);
#pragma unroll
    for (int e = 0; e < NS; e += 8) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t v = st[e / 2 + j];
        hi[j] = pack_pair(v);
        lo[j] = pack_pair(f2_fma(f2_bits(hi[j] << 16, hi[j] & 0xffff0000u), minus, v));
      }
      const int k = sk + e;
      const uint32_t at = k / 64 * (D * 128) + sw128_offset(sv, k % 64);
      *reinterpret_cast<uint4*>(&s.sb[0][0][0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(&s.sb[1][0][0] + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };
  if (warp < Sh::WARPS) {
#pragma unroll
    for (int e = 0; e < NS; e += 2) {
      const size_t at = op.turned ? (size_t)sv * D + sk + e : (size_t)(sk + e) * D + sv;
      st[e / 2] = from ? f2(from[at], from[at + (op.turned ? 1 : D)]) : 0;
    }
    if (!STATES && from) put_state();
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.tmem_base;
  int* err = p.err;
  bool ok = true;
  if (p.stall_ns) {  // before any copy or product: a wait that nothing arrives at, and the block's end after it
    if (mover && lane == 0) ok = mbar_wait_ns(&s.done, 0, err, PATH_PAGED_WAIT + 35, p.stall_ns);
    if (!ok && p.status) paged_error(p.status, PATH_PAGED_WAIT + 35);
    __syncthreads();
    if (lead) tmem_dealloc(tb, Sh::COLS);
    return;
  }
  auto wait = [&](uint64_t* bar, uint32_t n, int code) {  // for the n-th completion; the whole warp agrees
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_lean(bar, n & 1, err, PATH_PAGED_WAIT + code));
    return ok;
  };

  auto z_buffer = [&](int n) -> uint8_t (*)[TILE] { return STATES && PARTS == 1 && n % NZ ? s.x[0] : s.z[n % Sm::NZ]; };
  if (mover) {
    // ---------------- tiles in and out ----------------
    const int row0 = p.packed ? it.q0 : 0;
    const int px = (p.packed ? 0 : it.seq * p.heads * gx) + h * gx, py = (p.packed ? 0 : it.seq * p.heads * gy) + h * gy;
    auto load = [&](uint8_t (*to)[TILE], const CUtensorMap* map, uint64_t* bar, int k, int plane) {
      if (lane != 0) return;
      mbar_arrive_expect_tx(bar, X * TILE);
#pragma unroll
      for (int j = 0; j < X; ++j) tma_load_3d(to[j], map, 64 * j, row0 + chunk_of(k) * C, plane, bar);
    };
    // the tile after that, into L2: by the time its buffer is free it is near
    auto ahead = [&](const CUtensorMap* map, int k, int plane) {
      if (lane != 0 || k >= count) return;
#pragma unroll
      for (int j = 0; j < X; ++j) tma_prefetch_3d(map, 64 * j, row0 + chunk_of(k) * C, plane);
    };
    int kx = 0, hx = 0, nx = 0, ky = 0, hy = 0, ny = 0, kz = 0, hz = 0, nz = 0;  // (chunk, head, number) of the next load
    auto next_x = [&]() {
      if (kx >= count) return;
      load(s.x[nx % NX], &maps.x[oi], &s.full_x[nx % NX], kx, px + hx);
      ++nx;
      if (++hx >= gx) hx = 0, ++kx;
      ahead(&maps.x[oi], kx, px + hx);
    };
    auto next_y = [&]() {
      if (ky >= count) return;
      load(s.y[ny % NY], &maps.y[oi], &s.full_y[ny % NY], ky, py + hy);
      ++ny;
      if (++hy >= gy) hy = 0, ++ky;
      ahead(&maps.y[oi], ky, py + hy);
    };
    auto next_z = [&]() {
      if (kz >= count) return;
      load(z_buffer(nz), &maps.z[oi], &s.full_z[nz % NZ], kz, py + hz);
      ++nz;
      if (++hz >= gy) hz = 0, ++kz;
      ahead(&maps.z[oi], kz, py + hz);
    };
    next_y();
    if (!STATES) next_x();
    next_z();
    next_y();
    if (!STATES && NX > 1) next_x();
    if (NZ > 1) next_z();
    int g = 0, k = 0, un = 0, xn = 0;
    for (int i = 0; i < steps && ok; ++i) {
      const bool last = g == G - 1;
      if (gy > 1 || last) {  // y and z have been read
        if (!wait(&s.yz_free[un % NF], un / NF, 10)) break;
        ++un;
        next_y();
        next_z();
      }
      if (!STATES && (gx > 1 || last)) {  // o lies in x's place
        if (!wait(&s.out_full[xn % NX], xn / NX, 11)) break;
        if (!ragged(k) && lane == 0)
#pragma unroll
          for (int j = 0; j < X; ++j) tma_store_3d(&maps.o[oi], s.x[xn % NX][j], 64 * j, row0 + chunk_of(k) * C, px + (gx > 1 ? g : 0));
        if (lane == 0) {
          bulk_commit();
          bulk_wait_read0();
        }
        __syncwarp();
        next_x();
        ++xn;
      }
      if (last) g = 0, ++k;
      else ++g;
    }
  } else if (lead) {
    // ---------------- products ----------------
    const uint32_t id_s = idesc_bf16(C, C, 0, 0), id_x = idesc_bf16(C, D, 0, 0), id_o = idesc_bf16(C, D, 0, 1), id_d = idesc_bf16(D, D, 1, 1);
    const uint64_t kd = sdesc_sw128(0, 1024, 16), md = sdesc_sw128(0, 1024, TILE);
    const uint32_t tbu = uniform(tb), base = uniform(smem_u32(smem_raw) >> 4);
    auto at16 = [&](const void* a) { return base + (uint32_t)(((const uint8_t*)a - smem_raw) >> 4); };
    auto buffer = [&](const void* first, int i) { return at16(first) + uniform(i * (X * TILE / 16)); };
    int g = 0, k = 0, yn = 0, xn = 0, un = 0;  // head, chunk; numbers of y (and z) and x; of deltas
    auto operands = [&]() {
      wait(&s.full_y[yn % NY], yn / NY, 17);
      if (STATES) wait(&s.full_z[yn % NZ], yn / NZ, 25);
      else wait(&s.full_x[xn % NX], xn / NX, 18);
      if (ragged(k)) wait(&s.clean, 0, 19);
      tc_fence_after();
    };
    auto issue_s = [&](int i) {  // over P of the step before (two_s: before that one), which has been read
      const uint32_t d_s = tbu + uniform(s_col(i));
      const uint32_t a_x = buffer(s.x, xn % NX), a_y = buffer(s.y, yn % NY);
#pragma unroll
      for (int j = 0; j < X; ++j) mma4_ss<2, 2>(d_s, kd + (a_x + j * (TILE / 16)), kd + (a_y + j * (TILE / 16)), id_s, j ? 1u : 0u);
      commit_elect(&s.s_full);
    };
    auto z_at = [&](int n) { return base + uniform((uint32_t)(&z_buffer(n)[0][0] - smem_raw) >> 4); };
    auto issue_delta = [&](int yn, uint32_t accumulate, bool total) {
      const uint32_t a_z = z_at(yn);
#pragma unroll
      for (int t = 0; t < PARTS; ++t) {
        const uint32_t a_w = t == 0 ? buffer(s.y, yn % NY) : at16(t == 1 ? s.x[0] : s.z[Sm::NZ]);
#pragma unroll
        for (int k = 0; k < 2; ++k) mma4_ss<128, 128>(tbu + COL_D, md + (a_z + 512u * k), md + (a_w + 512u * k), id_d, (t | k) ? 1u : accumulate);
      }
      commit_elect(&s.yz_free[yn % NF]);
      if (STATES || gy > 1) commit_elect(&s.d_full);
      if (total) commit_elect(&s.t_full);
    };
    // O's part from the state, of the x at hand: into the O buffer whose last output has been taken
    int on = 0;
    auto o_at = [&](int n) { return tbu + COL_O + uniform(two_s ? 0 : n % Sh::NO * D); };
    auto issue_inter = [&]() {
      const uint32_t a_x = buffer(s.x, xn % NX), d_o = o_at(on);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < X; ++j) mma4_ss<2, 2>(d_o, kd + (a_x + j * (TILE / 16)), kd + at16(s.sb[t][j]), id_x, (t | j) ? 1u : 0u);
      commit_elect(&s.o_full);
    };
    bool early = false;  // this step's has been issued
    operands();
    if (!STATES && ok) issue_s(0);
    for (int i = 0; i < steps && ok; ++i) {
      const bool last = g == G - 1, update = gy > 1 || last;
      const bool old = from || k > 0;  // there is a state before the chunk
      const uint32_t more = uniform(STATES ? i > 0 : gy > 1 && g > 0);
      if constexpr (!STATES) {
        if (old && (gx > 1 || g == 0) && !early) {
          if (i > 0 && !wait(&s.done, i - 1, 20)) break;
          tc_fence_after();
          issue_inter();
        }
        early = false;
        if (!wait(&s.full_z[yn % NZ], yn / NZ, 25) || !wait(&s.p_full, i, 21)) break;
        tc_fence_after();
        const uint32_t a_z = z_at(yn), first = uniform(old ? 1u : 0u) | more;
        const uint32_t d_s = tbu + uniform(s_col(i));
        auto at_p = [&](int e) { return d_s + 16 * e / SW * SW + 16 * e % SW / 2; };  // of 16 tokens
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          mma4_ts<128>(o_at(on), at_p(e), at_p(e + 1), at_p(e + 2), at_p(e + 3), md + (a_z + 128u * e), id_o, e ? 1u : first);
          constexpr int R = SW / 2;  // what rounding left of P, behind it
          if (FINE) mma4_ts<128>(o_at(on), at_p(e) + R, at_p(e + 1) + R, at_p(e + 2) + R, at_p(e + 3) + R, md + (a_z + 128u * e), id_o, 1u);
        }
        commit_elect(&s.c_full);
      }
      // Delta, and S of the next step; S first where no state waits for Delta
      const int y0 = yn;
      const bool s_first = !STATES && D == 64 && gy > 1 && !last;  // (with one buffer of z its next tile waits for Delta)
      auto delta = [&]() {
        if (!update || !wait(&s.w_full, un++, 22)) return;
        tc_fence_after();
        issue_delta(y0, more, STATES ? i + 1 == steps : last);
      };
      if (!s_first) delta();
      if (gy > 1 || last) ++yn;
      if (gx > 1 || last) ++xn, ++on;
      if (last) g = 0, ++k;
      else ++g;
      if (ok && i + 1 < steps) {
        operands();
        if (!STATES && (two_s ? ok : wait(&s.c_full, i, 24))) {
          tc_fence_after();
          issue_s(i + 1);
          if (Sh::NO > 1 && gx > 1 && g > 0 && old) {  // (the state is the same, and P of this step was made after the last output)
            issue_inter();
            early = true;
          }
        }
      }
      if (s_first && ok) delta();
    }
  } else {
    // ---------------- weights, state, output ----------------
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int r = 32 * quad + lane;  // row of S and O
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const int light = rev ? (cg == 0 ? quad - 2 : -1) : (cg == 1 && quad < 2 ? quad : -1);  // number among them, or below 0
    auto o_col = [&](int n) { return COL_O + (two_s ? 0 : n % Sh::NO * D); };
    int g = 0, k = 0, yn = 0, xn = 0, in = 0;  // in: products with the state
    for (int i = 0; i < steps && ok; ++i) {
      const int m = rows_of(k), yb = yn % NY;
      const bool fresh = gy > 1 || g == 0, last = g == G - 1, update = gy > 1 || last;
      const bool inter = (from || k > 0) && (gx > 1 || g == 0);
      if (fresh && ragged(k)) {  // rows of the next sequence: they may hold anything
        wait(&s.full_y[yb], yn / NY, 32);
        if (!wait(&s.full_z[yn % NZ], yn / NZ, 33)) break;
        uint8_t* z = &z_buffer(yn)[0][0];
        for (int e = tid; e < (C - m) * 8 * X; e += NCT) {
          const uint32_t at = e / ((C - m) * 8) * TILE + (m * 8 + e % ((C - m) * 8)) * 16;
          *reinterpret_cast<uint4*>(&s.y[yb][0][0] + at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(z + at) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        arrive(&s.clean);
      }
      uint32_t a[32];
      if constexpr (!STATES) {
        if (two_s && g > 0 && !wait(&s.c_full, i - 1, 33)) break;  // (its phases one by one)
        if (!wait(&s.s_full, i, 34)) break;
        tc_fence_after();
        // P over S: a warp's columns become half as many of packed pairs, in the place of their first half; FINE: the rest of
        // each in that of the second, once all of S has been read
        uint32_t rest[FINE ? SQ : 1][16];
#pragma unroll
        for (int q = 0; q < SQ; ++q) {
          const int jb = SQ * cg + q;
          uint32_t b[16];
          auto pair = [&](int e, uint64_t v) {
            b[e] = pack_pair(v);
            if (FINE) rest[q][e] = pack_pair(f2_fma(f2_bits(b[e] << 16, b[e] & 0xffff0000u), f2(-1.f, -1.f), v));
          };
          if (jb == quad || (jb < quad) != rev) {
            tmem_ld32(tb + lane_off + s_col(i) + 32 * jb, a);
            if (jb == quad) {
              const float* w = &s.pw[Z0 + (rev ? -lane : lane)];
              tmem_ld_wait();
              if (rev) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) pair(e / 2, f2_mul(f2_bits(a[e], a[e + 1]), f2(w[e], w[e + 1])));
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 2) pair(e / 2, f2_mul(f2_bits(a[e], a[e + 1]), f2(w[-e], w[-e - 1])));
              }
            } else {
              const float w = s.pw[Z0 + (rev ? 32 * jb - r : r - 32 * jb - 31)];
              const uint64_t ww = f2(w, w);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const ulonglong2 cw = *reinterpret_cast<const ulonglong2*>(&s.colw[e]);
                pair(e / 2, f2_mul(f2_mul(f2_bits(a[e], a[e + 1]), cw.x), ww));
                pair(e / 2 + 1, f2_mul(f2_mul(f2_bits(a[e + 2], a[e + 3]), cw.y), ww));
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) pair(e, 0);
          }
          tmem_st16(tb + lane_off + s_col(i) + SW * cg + 16 * q, b);
        }
        if constexpr (FINE)
#pragma unroll
          for (int q = 0; q < SQ; ++q) tmem_st16(tb + lane_off + s_col(i) + SW * cg + SW / 2 + 16 * q, rest[q]);
        if (inter) {  // what lies before the chunk, weighted
          if (!wait(&s.o_full, in, 35)) break;
          ++in;
          tc_fence_after();
          tmem_ld32(tb + lane_off + o_col(xn) + 32 * cg, a);
          const float w = s.pw[Z0 + (rev ? max(m - r, 0) : r + 1)];
          const uint64_t ww = f2(w, w);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t v = f2_mul(f2_bits(a[e], a[e + 1]), ww);
            a[e] = (uint32_t)v, a[e + 1] = (uint32_t)(v >> 32);
          }
          tmem_st32(tb + lane_off + o_col(xn) + 32 * cg, a);
        }
        tmem_st_wait();
        tc_fence_before();
        arrive(&s.p_full);
      }
      if (update) {  // Y' over Y, whose products have been made; rows behind m become 0
        if (STATES && !wait(&s.full_y[yb], yn / NY, 36)) break;
        // (PARTS > 1: the further parts' places have been read)
        if (STATES && PARTS > 1 && i > 0 && !wait(&s.d_full, i - 1, 36)) break;
        // states alone: weighed to the segment's end, so that all deltas add up where they are
        const float ahead = STATES ? exp2f(l2 * (rev ? (chunk_of(k) - c0) * C : min(it.n, (c0 + count) * C) - chunk_of(k) * C - m)) : 1.f;
        if (ALL || light >= 0) {
          constexpr int STEP = 32 * (ALL ? Sh::WARPS : Sh::LIGHT);
#pragma unroll 4
          for (int e = ALL ? tid : 32 * light + lane; e < C * 8 * X; e += STEP) {
            const int row = e / 8 % C;
            const uint32_t at = e / (8 * C) * TILE + (e % (8 * C)) * 16;
            uint8_t* y = &s.y[yb][0][0] + at;
            uint4 w[PARTS], in = *reinterpret_cast<const uint4*>(y);
            if (row >= m) in = make_uint4(0, 0, 0, 0);
            weighted<PARTS>(in, s.pw[Z0 + (rev ? row : max(m - 1 - row, 0))] * ahead, w);
            *reinterpret_cast<uint4*>(y) = w[0];
            if constexpr (PARTS > 1) {
              *reinterpret_cast<uint4*>(&s.x[0][0][0] + at) = w[1];
              *reinterpret_cast<uint4*>(&s.z[Sm::NZ][0][0] + at) = w[2];
            }
          }
          fence_proxy_async_smem();
          // (w_full is one phase ahead at most; with one y to a chunk t_full sees to it)
          if ((gy > 1 || (STATES && PARTS == 1)) && i > 0 && !wait(&s.d_full, i - 1, 37)) break;
          arrive(&s.w_full);
        }
      }
      const bool emit = !STATES && (gx > 1 || last);
      uint32_t out[16];
      auto put_out = [&]() {
        if (!ragged(k)) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(s.x[xn % NX][cg / 2] + sw128_offset(r, cg % 2 * 32 + 8 * j)) = make_uint4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
          fence_proxy_async_smem();
        } else if (r < m) {  // a box would reach into the next sequence
          __nv_bfloat16* o = (__nv_bfloat16*)op.o + ((long long)it.q0 + chunk_of(k) * C + r) * op.xt + (long long)(h * gx + (gx > 1 ? g : 0)) * op.xh + 32 * cg;
#pragma unroll
          for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(o + 8 * j) = make_uint4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
        }
        arrive(&s.out_full[xn % NX]);
      };
      if (emit) {
        if (!wait(&s.c_full, i, 38)) break;
        tc_fence_after();
        tmem_ld32(tb + lane_off + o_col(xn) + 32 * cg, a);
        const uint64_t scale = f2(p.scale, p.scale);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) out[j] = pack_pair(f2_mul(f2_bits(a[2 * j], a[2 * j + 1]), scale));
        if (PARTS == 1) put_out();
      }
      if (STATES ? i + 1 == steps : last) {
        if (!wait(&s.t_full, STATES ? 0 : k, 39)) break;
        tc_fence_after();
        const float2 kept = s.keep[m < C];
        const uint64_t keep = f2(kept.x, kept.x), rest = f2(kept.y, kept.y);
        // The decay's rest where the state is kept for later calls.  Else a walk's chunks are too few for it to show beside bf16 (16384
        // tokens: 2^-17 of the oldest one's weight at most; with it 8 x 32 x 4096 at d 64 391 us forward and backward in place of 389).
        constexpr bool REST = PARTS == 3 && !STATES;
        uint32_t b[NS];
        if constexpr (D == 64) tmem_ld16x2_16(tb + lane_off + COL_D + 16 * cg, b);
        else tmem_ld32(tb + lane_off + COL_D + 32 * cg, b);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < NS; e += 2) {
          const uint64_t add = f2_bits(b[e], b[e + 1]);
          st[e / 2] = f2_fma(st[e / 2], keep, REST ? f2_fma(st[e / 2], rest, add) : add);
        }
        if (!STATES && k + 1 < count) {  // (the last product with the old one is over: P waited for it)
          put_state();
          fence_proxy_async_smem();
        }
      }
      if (emit && PARTS > 1) put_out();  // (x's place holds a part of Y' until now)
      tc_fence_before();
      if (!STATES) arrive(&s.done);
      if (gx > 1 || last) ++xn;
      if (gy > 1 || last) ++yn;
      if (last) g = 0, ++k;
      else ++g;
    }
    float* to = STATES ? part : !split && p.update ? own : nullptr;
    if (ok && to)
#pragma unroll
      for (int e = 0; e < NS; e += 2) {
        float a, b;
        f2_split(st[e / 2], a, b);
        to[(size_t)(sk + e) * D + sv] = a;
        to[(size_t)(sk + e + 1) * D + sv] = b;
      }
  }
  if (!ok && mover && lane == 0) {
    if (p.status) paged_error(p.status, *reinterpret_cast<volatile int*>(err));
    // after a failure: no copy may land in shared memory once the block has gone (bounded waits on whatever is in flight)
    for (int b = 0; b < 2; ++b) {
      for (int j = 0; j < NX; ++j) mbar_wait_ns(&s.full_x[j], b, nullptr, 0, 1000000ull);
      for (int j = 0; j < NY; ++j) mbar_wait_ns(&s.full_y[j], b, nullptr, 0, 1000000ull);
      for (int j = 0; j < NZ; ++j) mbar_wait_ns(&s.full_z[j], b, nullptr, 0, 1000000ull);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (lead) {
    tc_fence_after();
    tmem_dealloc(tb, Sh::COLS);
  }
}

// [planes][rows][D] bf16, `row` and `plane` elements apart, in boxes of 128 rows x 64 columns; rows behind the last read as
// zero and are not written.
bool make_map(CUtensorMap* m, const void* base, int D, long long rows, long long planes, long long row, long long plane) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)planes};
  cuuint64_t strides[2] = {(cuuint64_t)row * 2, (cuuint64_t)plane * 2};
  cuuint32_t box[3] = {64, C, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool STATES, int PARTS, bool FINE = false> cudaError_t launch(const LinMaps& maps, const LinArgs& p, cudaStream_t st) {
  static_assert(Shape<D>::BLOCKS * (sizeof(Smem<D, PARTS>) + 1024) <= 233472, "shared memory of an SM");
  auto kern = linear_tc_kernel<D, STATES, PARTS, FINE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D, PARTS>));
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3((unsigned)((long long)p.items * p.heads * (STATES ? p.slots : p.ops))), Shape<D>::NT, sizeof(Smem<D, PARTS>), st, maps, p);
}

}  // namespace

cudaError_t launch_linear_tc(const LinArgs& p, bool states, cudaStream_t st) {
  LinMaps maps;
  for (int i = 0; i < p.ops; ++i) {
    const LinOp& op = p.op[i];
    const long long rows = p.packed ? p.total : p.L, seqs = p.packed ? 1 : p.seqs;
    const long long nx = seqs * p.heads * op.gx, ny = seqs * p.heads * op.gy;
    // (planes of one sequence follow one another at the heads' distance, and so do sequences)
    if (!make_map(&maps.x[i], op.x, p.D, rows, nx, op.xt, op.xh) || !make_map(&maps.o[i], op.o, p.D, rows, nx, op.xt, op.xh) ||
        !make_map(&maps.y[i], op.y, p.D, rows, ny, op.yt, op.yh) || !make_map(&maps.z[i], op.z, p.D, rows, ny, op.yt, op.yh))
      return cudaErrorInvalidValue;
  }
  // A cache's states (whether or not they are written, for the same outputs) come from the states' pass where there are
  // several segments, else from the walk.
  const bool exact = p.state && (states || p.max_new <= p.seg);
  // Few sequences of one chunk: P's rounding is one of an output's two, and of so few numbers that it need not average out to the
  // other's size (a token alone: up to 2^-8 of its output, beside the output's own).  Free where the blocks are one wave (8 heads x
  // 128: 11.9 us with and without); 64 x 32 x 128 would take 56 us in place of 50.
  const bool fine = p.max_new <= C && (long long)p.items * p.heads * p.ops <= 152 * (p.D == 64 ? Shape<64>::BLOCKS : Shape<128>::BLOCKS);
  if (p.D == 64) {
    if (states) return exact ? launch<64, true, 3>(maps, p, st) : launch<64, true, 1>(maps, p, st);
    if (fine) return exact ? launch<64, false, 3, true>(maps, p, st) : launch<64, false, 1, true>(maps, p, st);
    return exact ? launch<64, false, 3>(maps, p, st) : launch<64, false, 1>(maps, p, st);
  }
  if (states) return exact ? launch<128, true, 3>(maps, p, st) : launch<128, true, 1>(maps, p, st);
  if (fine) return exact ? launch<128, false, 3, true>(maps, p, st) : launch<128, false, 1, true>(maps, p, st);
  return exact ? launch<128, false, 3>(maps, p, st) : launch<128, false, 1>(maps, p, st);
}

}  // namespace pathattn
