// Linear attention on the tensor cores (bf16): the walk of linear.h in chunks of 128 tokens, one block per key head, segment
// and 64 columns of z and o, two blocks to an SM.  Of a chunk, with r the row and m the rows that are tokens,
//   S = X Y^T,  O = X State (tcgen05),  P = S masked and weighted with g^(distance), O scaled by g^(distance to the state),
//   O += P Z,  Delta = Y^T Z', Z' = Z weighted with g^(distance to the chunk's end),  State = g^m State + Delta.
// State is float32 in registers, its bf16 copy in shared memory the operand of the next chunk; P goes back to tensor memory
// over S.  A block's phases follow one another (the state is a chain); the SM's other block fills their gaps.
//
// Roundings beside the output's: P and the state's copy to bf16, the operands' type (relative 2^-8 each; what reaches an
// output is their independent sum).  Z' is the sum of PARTS bf16 numbers: two (2^-16) keep a third such rounding out of the
// outputs, three (2^-24) leave a cache's states, which are outputs themselves, as exact as float32 sums.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "dev_common.cuh"
#include "linear.h"
#include "tc_common.cuh"

namespace pathattn {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // fwd_tc.cu

namespace {

using namespace tc;

constexpr int NT = 256, C = 128, V = 64, TILE = C * 128;
constexpr int COL_S = 0, COL_O = 128, COL_D = 192, COLS = 256;  // tensor memory: S and P, O, Delta
constexpr int Z0 = 32;                                          // zeros before g^0 in the table

struct LinMaps {
  CUtensorMap x[3], y[3], z[3], o[3];
};

template <int D, int PARTS> struct Smem {
  // Tiles of a row block; buffers of y and of z; places for the further parts of Z': what two blocks in 227 KB leave (at head
  // dim 128 the further parts take x's place once x has been read).
  static constexpr int X = D / 64, NY = D == 64 && PARTS == 1 ? 2 : 1, NZ = D == 64 && PARTS < 3 ? 2 : 1, REST = D == 64 ? PARTS - 1 : 0;
  uint8_t x[X][TILE], y[NY][X][TILE], z[NZ][TILE];
  uint8_t zs[1 + REST][TILE];  // Z'; the first, then, O on its way out
  uint8_t sb[D * 128];     // the state in bf16
  float pw[Z0 + C + 8];    // 0 .., then g^n
  alignas(16) float colw[32];  // g^n of a 32-column block's columns
  uint64_t full_x, full_y[NY], full_z[NZ], bar_a, bar_b, bar_c, zfree;
  uint32_t tmem_base;
};

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
// Issued by one elected lane of a converged warp.
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
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 bytes of Z (8 columns of a row), weighted, as a sum of bf16 numbers: parts FROM .. TO - 1 of it.
template <int FROM, int TO> __device__ __forceinline__ void weighted(uint4 z, float w, uint4 (&out)[TO - FROM]) {
  const uint32_t in[4] = {z.x, z.y, z.z, z.w};
  uint32_t o[TO - FROM][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = lo_of(in[i]) * w, b = hi_of(in[i]) * w;
#pragma unroll
    for (int t = 0; t < TO; ++t) {
      const uint32_t x = pack_bf16(a, b);
      if (t >= FROM) o[t - FROM][i] = x;
      a -= lo_of(x), b -= hi_of(x);
    }
  }
#pragma unroll
  for (int t = 0; t < TO - FROM; ++t) out[t] = make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
}

template <int D, bool STATES, int PARTS>
__global__ void __launch_bounds__(NT, 2) linear_tc_kernel(const __grid_constant__ LinMaps maps, const LinArgs p) {
  chain();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using Sm = Smem<D, PARTS>;
  constexpr int X = Sm::X, NY = Sm::NY, NZ = Sm::NZ, NV = D / V;
  // at head dim 128 the further parts of Z' are made after x has been read
  constexpr bool LATE = !STATES && D == 128 && PARTS > 1;
  constexpr int SOON = LATE ? 1 : PARTS;
  constexpr int NS = D == 64 ? 16 : 32;  // state elements of a thread
  Sm& s = *reinterpret_cast<Sm*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
  // neighbouring blocks share operands: the columns of a head, then the gradients of one head
  int blk = blockIdx.x;
  const int v0 = blk % NV * V;
  blk /= NV;
  const int oi = blk % p.ops;
  blk /= p.ops;
  const int h = blk % p.heads, item = blk / p.heads;
  const LinOp& op = p.op[oi];
  const LinItem it = lin_item(p, item);
  if (it.seg < 0) return;
  if (smem_u32(smem_raw) & 1023) {  // (swizzled tiles begin on 1024 bytes)
    if (tid == 0) atomicCAS(p.err, 0, PATH_PAGED_WAIT + 16);
    return;
  }
  const bool rev = op.reverse != 0;
  const int gx = op.gx, gy = op.gy, G = STATES || gy > gx ? gy : gx;
  const float l2 = lin_log2(p.log_decay[h]);
  // chunks of the segment: in tokens, segments and chunks begin at multiples of their lengths
  const int nch = (it.n + C - 1) / C, per = p.seg / C, nseg = (nch + per - 1) / per;
  const int c0 = (rev ? nseg - 1 - it.seg : it.seg) * per, count = min(per, nch - c0);
  auto chunk_at = [&](int k) { return rev ? c0 + count - 1 - k : c0 + k; };
  const int steps = count * G;

  if (tid == 0) {
    mbar_init(&s.full_x, 1);
    for (int i = 0; i < NY; ++i) mbar_init(&s.full_y[i], 1);
    for (int i = 0; i < NZ; ++i) mbar_init(&s.full_z[i], 1);
    mbar_init(&s.bar_a, 1);
    mbar_init(&s.bar_b, 1);
    mbar_init(&s.bar_c, 1);
    mbar_init(&s.zfree, 1);
    fence_barrier_init();
  }
  const int lead = rev ? 3 : 4;  // the warp whose share of P is all masked loads and issues
  if (warp == lead) tmem_alloc(&s.tmem_base, COLS);
  if (tid < Z0 + C + 1) s.pw[tid] = tid < Z0 ? 0.f : exp2f(l2 * (tid - Z0));
  if (tid < 32) s.colw[tid] = exp2f(l2 * (rev ? tid : 31 - tid));
  const size_t dd = (size_t)D * D;
  float* part = p.parts + (((size_t)oi * p.items + item) * p.heads + h) * dd;
  float* own = p.state ? p.state + ((size_t)it.seq * p.heads + h) * dd : nullptr;
  const bool split = p.max_new > p.seg;  // the segments' starting states are in parts
  const float* from = STATES ? nullptr : split ? part : own;
  // this thread's part of the state: row srow, columns scol ..
  const int srow = D == 64 ? 16 * quad + (lane & 15) : 32 * quad + lane;
  const int scol = D == 64 ? 32 * (lane >> 4) + 16 * half : 32 * half;
  float st[NS];
#pragma unroll
  for (int e = 0; e < NS; e += 4) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (from) a = *reinterpret_cast<const float4*>(from + (size_t)srow * D + v0 + scol + e);
    st[e] = a.x, st[e + 1] = a.y, st[e + 2] = a.z, st[e + 3] = a.w;
  }
  auto put_state = [&]() {
#pragma unroll
    for (int e = 0; e < NS; e += 8)
      *reinterpret_cast<uint4*>(s.sb + sw128_offset(srow, scol + e)) =
          make_uint4(pack_bf16(st[e], st[e + 1]), pack_bf16(st[e + 2], st[e + 3]), pack_bf16(st[e + 4], st[e + 5]), pack_bf16(st[e + 6], st[e + 7]));
  };
  if (!STATES && from) put_state();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.tmem_base, lane_off = (uint32_t)(quad * 32) << 16;

  // ---- loads, by the lead warp's first lane: number i of x, of y and of z ----
  const int row0 = p.packed ? it.q0 : 0;
  const int px = (p.packed ? 0 : it.seq * p.heads * gx) + h * gx, py = (p.packed ? 0 : it.seq * p.heads * gy) + h * gy;
  const bool xstep = gx > 1 || LATE;  // x is brought anew for every step (else for every chunk)
  const int nx = STATES ? 0 : xstep ? steps : count, ny = gy > 1 ? steps : count;
  auto load_x = [&](int i) {
    if (lane != 0 || i >= nx) return;
    mbar_arrive_expect_tx(&s.full_x, X * TILE);
    for (int j = 0; j < X; ++j) tma_load_3d(s.x[j], &maps.x[oi], 64 * j, row0 + chunk_at(xstep ? i / G : i) * C, px + i % gx, &s.full_x);
  };
  auto load_y = [&](int i) {
    if (lane != 0 || i >= ny) return;
    mbar_arrive_expect_tx(&s.full_y[i % NY], X * TILE);
    for (int j = 0; j < X; ++j) tma_load_3d(s.y[i % NY][j], &maps.y[oi], 64 * j, row0 + chunk_at(i / gy) * C, py + i % gy, &s.full_y[i % NY]);
  };
  auto load_z = [&](int i) {
    if (lane != 0 || i >= ny) return;
    mbar_arrive_expect_tx(&s.full_z[i % NZ], TILE);
    tma_load_3d(s.z[i % NZ], &maps.z[oi], v0, row0 + chunk_at(i / gy) * C, py + i % gy, &s.full_z[i % NZ]);
  };
  if (warp == lead) {
    load_y(0);
    load_x(0);
    load_z(0);
    if (NY > 1) load_y(1);
    if (NZ > 1) load_z(1);
  }
  __syncwarp();

  const uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, V, 0, 1), id_d = idesc_bf16(D, V, 1, 1);
  const uint64_t kd = sdesc_sw128(0, 1024, 16), md = sdesc_sw128(0, 1024, TILE);
  const uint32_t tbu = uniform(tb);
  auto at16 = [&](const void* a) { return uniform(smem_u32(a) >> 4); };
  const uint32_t a_x = at16(s.x), a_zs = at16(s.zs), a_sb = at16(s.sb);
  auto issue_delta = [&](uint32_t a_y, uint32_t a_w, uint32_t accumulate) {
#pragma unroll
    for (int k = 0; k < C / 16; ++k)
      mma_ss_elect(tbu + COL_D, md + (a_y + 128u * k), md + (a_w + 128u * k), id_d, k ? 1u : accumulate);
  };
  auto rest = [&](int t) { return D == 64 ? s.zs[t] : s.x[t - 1]; };  // part t > 0 of Z'
  bool ok = true;
  int emits = 0;  // tiles of o sent on their way
  bool sent = false;
  for (int i = 0; i < steps; ++i) {
    const int k = i / G, g = i % G, c = chunk_at(k), m = min(C, it.n - c * C);
    const int xn = xstep ? i : k, yn = gy > 1 ? i : k, yb = yn % NY, zb = yn % NZ;
    const bool fresh = gy > 1 || g == 0, last = g == G - 1;
    const bool old = from || k > 0;          // there is a state before the chunk
    const bool inter = old && (gx > 1 || g == 0);
    ok = mbar_wait_lean(&s.full_y[yb], (yn / NY) & 1, p.err, PATH_PAGED_WAIT + 17) && ok;
    if (!STATES && warp == lead) {
      ok = mbar_wait_lean(&s.full_x, xn & 1, p.err, PATH_PAGED_WAIT + 18) && ok;
      __syncwarp();
      tc_fence_after();
      const uint32_t a_y = at16(s.y[yb]);
#pragma unroll
      for (int j = 0; j < X; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_ss_elect(tbu + COL_S, kd + (a_x + j * (TILE / 16) + 2u * e), kd + (a_y + j * (TILE / 16) + 2u * e), id_s, (j | e) ? 1u : 0u);
      if (inter)
#pragma unroll
        for (int j = 0; j < X; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_ss_elect(tbu + COL_O, kd + (a_x + j * (TILE / 16) + 2u * e), md + (a_sb + 128u * (4 * j + e)), id_o, (j | e) ? 1u : 0u);
      commit_elect(&s.bar_a);
      if (sent && lane == 0) {
        bulk_wait_read0();
        mbar_arrive(&s.zfree);
      }
      __syncwarp();
    }
    sent = false;
    if (emits > 0) ok = mbar_wait_lean(&s.zfree, (emits - 1) & 1, p.err, PATH_PAGED_WAIT + 19) && ok;
    if (fresh) {
      ok = mbar_wait_lean(&s.full_z[zb], (yn / NZ) & 1, p.err, PATH_PAGED_WAIT + 20) && ok;
      if (p.packed && m < C) {  // rows of the next sequence: they may hold anything
        for (int r = m + (tid >> 3); r < C; r += NT / 8) {
#pragma unroll
          for (int j = 0; j < X; ++j) *reinterpret_cast<uint4*>(s.y[yb][j] + r * 128 + (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(s.z[zb] + r * 128 + (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < C * 8 / NT; ++j) {  // (weights of rows behind m: of zeros)
        const int r = (tid >> 3) + j * (NT / 8);
        const uint32_t at = r * 128 + (tid & 7) * 16;
        const float w = s.pw[Z0 + (rev ? r : m > r ? m - 1 - r : 0)];
        const uint4 z = *reinterpret_cast<const uint4*>(s.z[zb] + at);
        uint4 out[SOON];
        weighted<0, SOON>(z, w, out);
        *reinterpret_cast<uint4*>(s.zs[0] + at) = out[0];
#pragma unroll
        for (int t = 1; t < SOON; ++t) *reinterpret_cast<uint4*>(rest(t) + at) = out[t];
      }
      fence_proxy_async_smem();
      if (!__syncthreads_and(ok)) break;
      if (warp == lead) {
        tc_fence_after();
        const uint32_t a_y = at16(s.y[yb]);
        issue_delta(a_y, a_zs, gy > 1 && g > 0 ? 1u : 0u);
#pragma unroll
        for (int t = 1; t < SOON; ++t) issue_delta(a_y, at16(rest(t)), 1u);
        if (!LATE) commit_elect(&s.bar_b);
      }
    }
    if constexpr (!STATES) {
      ok = mbar_wait_lean(&s.bar_a, i & 1, p.err, PATH_PAGED_WAIT + 21) && ok;
      tc_fence_after();
      const int r = 32 * quad + lane;
      if (inter) {  // what lies before the chunk, weighted
        uint32_t a[32];
        tmem_ld32(tb + lane_off + COL_O + 32 * half, a);
        tmem_ld_wait();
        const float w = s.pw[Z0 + (rev ? max(m - r, 0) : r + 1)];
#pragma unroll
        for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * w);
        tmem_st32(tb + lane_off + COL_O + 32 * half, a);
      }
      // P over S: a warp's 64 columns become 32 of packed pairs in the place of their first half
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int jb = 2 * half + q;
        uint32_t a[32], b[16];
        if (jb == quad) {
          tmem_ld32(tb + lane_off + COL_S + 32 * jb, a);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int d0 = rev ? e - lane : lane - e, d1 = rev ? d0 + 1 : d0 - 1;
            const float x = __uint_as_float(a[e]) * s.pw[Z0 + d0], y = __uint_as_float(a[e + 1]) * s.pw[Z0 + d1];
            b[e / 2] = pack_bf16(d0 >= 0 ? x : 0.f, d1 >= 0 ? y : 0.f);
          }
        } else if ((jb < quad) != rev) {
          tmem_ld32(tb + lane_off + COL_S + 32 * jb, a);
          tmem_ld_wait();
          const float w = s.pw[Z0 + (rev ? 32 * jb - r : r - 32 * jb - 31)];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 cw = *reinterpret_cast<const float4*>(&s.colw[e]);
            b[e / 2] = pack_bf16(__uint_as_float(a[e]) * (w * cw.x), __uint_as_float(a[e + 1]) * (w * cw.y));
            b[e / 2 + 1] = pack_bf16(__uint_as_float(a[e + 2]) * (w * cw.z), __uint_as_float(a[e + 3]) * (w * cw.w));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) b[e] = 0;
        }
        tmem_st16(tb + lane_off + COL_S + 64 * half + 16 * q, b);
      }
      if constexpr (LATE) {
        if (fresh) {
#pragma unroll
          for (int j = 0; j < C * 8 / NT; ++j) {
            const int row = (tid >> 3) + j * (NT / 8);
            const uint32_t at = row * 128 + (tid & 7) * 16;
            uint4 out[PARTS - 1];
            weighted<1, PARTS>(*reinterpret_cast<const uint4*>(s.z[zb] + at), s.pw[Z0 + (rev ? row : m > row ? m - 1 - row : 0)], out);
#pragma unroll
            for (int t = 1; t < PARTS; ++t) *reinterpret_cast<uint4*>(rest(t) + at) = out[t - 1];
          }
          fence_proxy_async_smem();
        }
      }
      tmem_st_wait();
      tc_fence_before();
      if (!__syncthreads_and(ok)) break;
      if (warp == lead) {
        tc_fence_after();
        const uint32_t a_z = at16(s.z[zb]);
        const uint32_t first = uniform(old || (gy > 1 && g > 0) ? 1u : 0u);
#pragma unroll
        for (int e = 0; e < C / 16; ++e)
          mma_ts_elect(tbu + COL_O, tbu + COL_S + (e < 4 ? 8 * e : 32 + 8 * e), md + (a_z + 128u * e), id_o, e ? 1u : first);
        commit_elect(&s.bar_c);
        if (LATE && fresh) {
#pragma unroll
          for (int t = 1; t < PARTS; ++t) issue_delta(at16(s.y[yb]), at16(rest(t)), 1u);
          commit_elect(&s.bar_b);
        }
        if (!(LATE && fresh) && (xstep || last)) load_x(xn + 1);
      }
    }
    if (fresh || last) ok = mbar_wait_lean(&s.bar_b, yn & 1, p.err, PATH_PAGED_WAIT + 22) && ok;
    if (warp == lead && __all_sync(0xffffffffu, ok)) {
      if (LATE && fresh) load_x(xn + 1);
      if (gy > 1 || last) load_y(yn + NY);
      if (STATES) load_z(yn + NZ);
    }
    if (last) {
      tc_fence_after();
      const float keep = s.pw[Z0 + m];
      uint32_t a[NS];
      if constexpr (D == 64) tmem_ld16x2_16(tb + lane_off + COL_D + 16 * half, a);
      else tmem_ld32(tb + lane_off + COL_D + 32 * half, a);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < NS; ++e) st[e] = st[e] * keep + __uint_as_float(a[e]);
      if (!STATES && k + 1 < count) {
        put_state();
        fence_proxy_async_smem();
      }
    }
    if constexpr (!STATES) {
      ok = mbar_wait_lean(&s.bar_c, i & 1, p.err, PATH_PAGED_WAIT + 23) && ok;
      tc_fence_after();
      if (warp == lead && (gy > 1 || last) && __all_sync(0xffffffffu, ok)) load_z(yn + NZ);
      const bool emit = gx > 1 || last;
      if (emit) {
        uint32_t a[32];
        tmem_ld32(tb + lane_off + COL_O + 32 * half, a);
        tmem_ld_wait();
        const int r = 32 * quad + lane;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = pack_bf16(__uint_as_float(a[e + 2 * j]) * p.scale, __uint_as_float(a[e + 2 * j + 1]) * p.scale);
          *reinterpret_cast<uint4*>(s.zs[0] + sw128_offset(r, 32 * half + e)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      if (!__syncthreads_and(ok)) break;
      if (emit) {
        if (!p.packed || m == C) {
          if (warp == lead && lane == 0) tma_store_3d(&maps.o[oi], s.zs[0], v0, row0 + c * C, px + (gx > 1 ? g : 0));
        } else {  // a box would reach into the next sequence
          __nv_bfloat16* o = (__nv_bfloat16*)op.o + (long long)(it.q0 + c * C) * op.xt + (long long)(h * gx + (gx > 1 ? g : 0)) * op.xh + v0;
          for (int r = tid >> 3; r < m; r += NT / 8)
            *reinterpret_cast<uint4*>(o + r * op.xt + (tid & 7) * 8) = *reinterpret_cast<const uint4*>(s.zs[0] + sw128_offset(r, (tid & 7) * 8));
          __syncthreads();
        }
        if (warp == lead && lane == 0) bulk_commit();
        ++emits;
        sent = true;
      }
    } else {
      tc_fence_before();
    }
  }
  if (ok) {
    float* to = STATES ? part : !split && p.update ? own : nullptr;
    if (to)
#pragma unroll
      for (int e = 0; e < NS; e += 4)
        *reinterpret_cast<float4*>(to + (size_t)srow * D + v0 + scol + e) = make_float4(st[e], st[e + 1], st[e + 2], st[e + 3]);
  } else if (warp == lead && lane == 0) {
    if (p.status) paged_error(p.status, *reinterpret_cast<volatile int*>(p.err));
    // after a failure: no copy may land in shared memory once the block has gone (bounded waits on whatever is in flight)
    for (int b = 0; b < 2; ++b) {
      mbar_wait_ns(&s.full_x, b, nullptr, 0, 1000000ull);
      for (int j = 0; j < NY; ++j) mbar_wait_ns(&s.full_y[j], b, nullptr, 0, 1000000ull);
      for (int j = 0; j < NZ; ++j) mbar_wait_ns(&s.full_z[j], b, nullptr, 0, 1000000ull);
    }
  }
  if (!STATES && warp == lead && lane == 0) bulk_wait_read0();
  tc_fence_before();
  __syncthreads();
  if (warp == lead) {
    tc_fence_after();
    tmem_dealloc(tb, COLS);
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

template <int D, bool STATES, int PARTS> cudaError_t launch(const LinMaps& maps, const LinArgs& p, cudaStream_t st) {
  static_assert(2 * (sizeof(Smem<D, PARTS>) + 1024) <= 233472, "two blocks to an SM");
  auto kern = linear_tc_kernel<D, STATES, PARTS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D, PARTS>));
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3((unsigned)((long long)p.items * p.heads * p.ops * (D / V))), NT, sizeof(Smem<D, PARTS>), st, maps, p);
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
  // (a cache's states: whether or not they are written, for the same outputs)
  if (p.D == 64) {
    if (states) return p.state ? launch<64, true, 3>(maps, p, st) : launch<64, true, 2>(maps, p, st);
    return p.state ? launch<64, false, 3>(maps, p, st) : launch<64, false, 2>(maps, p, st);
  }
  if (states) return p.state ? launch<128, true, 3>(maps, p, st) : launch<128, true, 2>(maps, p, st);
  return p.state ? launch<128, false, 3>(maps, p, st) : launch<128, false, 2>(maps, p, st);
}

}  // namespace pathattn
