// Linear attention on the tensor cores (bf16): the walk of linear.h in chunks of 128 tokens, one block per key head, segment
// and 64 columns of z and o, two blocks to an SM.  Of a chunk, with r the row and m the rows that are tokens,
//   S = X Y^T,  O = X State (tcgen05),  P = S masked and weighted with g^(distance), O scaled by g^(distance to the state),
//   O += P Z,  Delta = Y^T Z', Z' = Z weighted with g^(distance to the chunk's end),  State = g^m State + Delta.
// State is float32 in registers; the operand of the next chunk is its copy as two bf16 numbers.  P goes back to tensor memory
// over S.  A block's phases follow one another (the state is a chain); the SM's other block fills their gaps.
//
// Roundings beside the output's: P and Z' to bf16, the operands' type (relative 2^-8; what reaches an output is the sum of
// independent ones).  Where the state is an output itself (serving) Z' is the sum of three bf16 numbers, as exact as float32.
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
  CUtensorMap x[3], y[3], z[3];
};

template <int D, int PARTS> struct Smem {
  // Tiles of a row block, buffers of y and of z: what two blocks in 227 KB leave.  The second part of Z' takes x's place once
  // x has been read, the third x's second tile or one of its own.
  static constexpr int X = D / 64, NY = D == 64 && PARTS == 1 ? 2 : 1, NZ = D == 64 ? 2 : 1, REST = D == 64 && PARTS == 3 ? 1 : 0;
  uint8_t x[X][TILE], y[NY][X][TILE], z[NZ][TILE];
  uint8_t zs[1 + REST][TILE];  // between chunks what rounding the state left (D rows), in a chunk Z'
  uint8_t sb[D * 128];         // the state in bf16
  float pw[Z0 + C + 8];        // 0 .., then g^n
  alignas(16) float colw[32];  // g^n of a 32-column block's columns
  uint64_t full_x, full_y[NY], full_z[NZ], bar_a, bar_b, bar_c;
  uint32_t tmem_base;
};

__device__ __forceinline__ uint64_t f2_bits(uint32_t a, uint32_t b) { return (uint64_t)b << 32 | a; }
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) { return pack_bf16(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))); }
// 32 bytes of global memory, aligned to them or (wide false) to 16.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
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

// 16 bytes of Z (8 columns of a row), weighted, as a sum of PARTS bf16 numbers.
template <int PARTS> __device__ __forceinline__ void weighted(uint4 z, float w, uint4 (&out)[PARTS]) {
  const uint32_t in[4] = {z.x, z.y, z.z, z.w};
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

template <int D, bool STATES, int PARTS>
__global__ void __launch_bounds__(NT, 2) linear_tc_kernel(const __grid_constant__ LinMaps maps, const LinArgs p) {
  chain();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  using Sm = Smem<D, PARTS>;
  constexpr int X = Sm::X, NY = Sm::NY, NZ = Sm::NZ, NV = D / V;
  constexpr int NS = D == 64 ? 16 : 32;  // state elements of a thread
  constexpr int ZR = C * 8 / NT;         // 16-byte pieces of Z of a thread
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
  const int steps = count * G;

  if (tid == 0) {
    mbar_init(&s.full_x, 1);
    for (int i = 0; i < NY; ++i) mbar_init(&s.full_y[i], 1);
    for (int i = 0; i < NZ; ++i) mbar_init(&s.full_z[i], 1);
    mbar_init(&s.bar_a, 1);
    mbar_init(&s.bar_b, 1);
    mbar_init(&s.bar_c, 1);
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
    for (int e = 0; e < NS; e += 8) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = st[e + 2 * j], b = st[e + 2 * j + 1];
        hi[j] = pack_bf16(a, b);
        lo[j] = pack_bf16(a - lo_of(hi[j]), b - hi_of(hi[j]));
      }
      const uint32_t at = sw128_offset(srow, scol + e);
      *reinterpret_cast<uint4*>(s.sb + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(s.zs[0] + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };
  if (!STATES && from) put_state();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.tmem_base, lane_off = (uint32_t)(quad * 32) << 16;

  // ---- loads, by the lead warp's first lane: of step (chunk k, head g), the n-th of its kind ----
  const int row0 = p.packed ? it.q0 : 0;
  const int px = (p.packed ? 0 : it.seq * p.heads * gx) + h * gx, py = (p.packed ? 0 : it.seq * p.heads * gy) + h * gy;
  auto row_of = [&](int k) { return row0 + (rev ? c0 + count - 1 - k : c0 + k) * C; };
  auto load_x = [&](int k, int g) {
    if (STATES || lane != 0 || k >= count) return;
    mbar_arrive_expect_tx(&s.full_x, X * TILE);
    for (int j = 0; j < X; ++j) tma_load_3d(s.x[j], &maps.x[oi], 64 * j, row_of(k), px + g, &s.full_x);
  };
  auto load_y = [&](int k, int g, int n) {
    if (lane != 0 || k >= count) return;
    mbar_arrive_expect_tx(&s.full_y[n % NY], X * TILE);
    for (int j = 0; j < X; ++j) tma_load_3d(s.y[n % NY][j], &maps.y[oi], 64 * j, row_of(k), py + g, &s.full_y[n % NY]);
  };
  auto load_z = [&](int k, int g, int n) {
    if (lane != 0 || k >= count) return;
    mbar_arrive_expect_tx(&s.full_z[n % NZ], TILE);
    tma_load_3d(s.z[n % NZ], &maps.z[oi], v0, row_of(k), py + g, &s.full_z[n % NZ]);
  };
  int ky = 0, gyn = 0, kz = 0, gzn = 0;  // (chunk, head) of the y and z to load next
  auto next_y = [&](int n) {
    load_y(ky, gyn, n);
    if (++gyn == gy) gyn = 0, ++ky;
  };
  auto next_z = [&](int n) {
    load_z(kz, gzn, n);
    if (++gzn == gy) gzn = 0, ++kz;
  };
  if (warp == lead) {
    next_y(0);
    load_x(0, 0);
    next_z(0);
    if (NY > 1) next_y(1);
    if (NZ > 1) next_z(1);
  }
  __syncwarp();

  const uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, V, 0, 1), id_d = idesc_bf16(D, V, 1, 1);
  const uint64_t kd = sdesc_sw128(0, 1024, 16), md = sdesc_sw128(0, 1024, TILE);
  const uint32_t tbu = uniform(tb), base = uniform(smem_u32(smem_raw) >> 4);
  auto at16 = [&](const void* a) { return base + (uint32_t)(((const uint8_t*)a - smem_raw) >> 4); };
  auto rest = [&](int t) { return t <= X ? s.x[t - 1] : s.zs[t - X]; };  // part t > 0 of Z'
  auto issue_delta = [&](int yb, uint32_t accumulate) {
    const uint32_t a_y = at16(s.y[0]) + yb * (X * TILE / 16);
#pragma unroll
    for (int t = 0; t < PARTS; ++t) {
      const uint32_t a_w = at16(t ? rest(t) : s.zs[0]);
#pragma unroll
      for (int k = 0; k < C / 16; ++k)
        mma_ss_elect(tbu + COL_D, md + (a_y + 128u * k), md + (a_w + 128u * k), id_d, (t | k) ? 1u : accumulate);
    }
    commit_elect(&s.bar_b);
  };
  bool ok = true;
  int g = 0, k = 0, yn = 0, xn = 0, un = 0;  // numbers of the y (and z) and x at hand; states' updates so far
  for (int i = 0; i < steps; ++i) {
    const int c = rev ? c0 + count - 1 - k : c0 + k, m = min(C, it.n - c * C);
    const int yb = yn % NY, zb = yn % NZ;
    const bool fresh = gy > 1 || g == 0, last = g == G - 1;
    const bool update = gy > 1 || last;      // (with several x: once the last has met the old state)
    const bool old = from || k > 0;          // there is a state before the chunk
    const bool inter = old && (gx > 1 || g == 0);
    if (fresh && p.packed && m < C) {  // rows of the next sequence: they may hold anything
      ok = mbar_wait_lean(&s.full_y[yb], (yn / NY) & 1, p.err, PATH_PAGED_WAIT + 17) && ok;
      ok = mbar_wait_lean(&s.full_z[zb], (yn / NZ) & 1, p.err, PATH_PAGED_WAIT + 18) && ok;
      for (int r = m + (tid >> 3); r < C; r += NT / 8) {
#pragma unroll
        for (int j = 0; j < X; ++j) *reinterpret_cast<uint4*>(s.y[yb][j] + r * 128 + (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(s.z[zb] + r * 128 + (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncthreads();
    }
    if (warp == lead) {
      ok = mbar_wait_lean(&s.full_y[yb], (yn / NY) & 1, p.err, PATH_PAGED_WAIT + 19) && ok;
      if constexpr (!STATES) {
        ok = mbar_wait_lean(&s.full_x, xn & 1, p.err, PATH_PAGED_WAIT + 20) && ok;
        __syncwarp();
        tc_fence_after();
        const uint32_t a_x = at16(s.x[0]), a_y = at16(s.y[0]) + yb * (X * TILE / 16);
#pragma unroll
        for (int j = 0; j < X; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_ss_elect(tbu + COL_S, kd + (a_x + j * (TILE / 16) + 2u * e), kd + (a_y + j * (TILE / 16) + 2u * e), id_s, (j | e) ? 1u : 0u);
        if (inter) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < X; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_ss_elect(tbu + COL_O, kd + (a_x + j * (TILE / 16) + 2u * e), md + (at16(t ? s.zs[0] : s.sb) + 128u * (4 * j + e)), id_o,
                             (t | j | e) ? 1u : 0u);
        }
        commit_elect(&s.bar_a);
      }
      __syncwarp();
    }
    ok = mbar_wait_lean(&s.full_z[zb], (yn / NZ) & 1, p.err, PATH_PAGED_WAIT + 21) && ok;
    // Z': computed while the products run, stored once they no longer read what lies in its place
    const int zr0 = tid >> 3;
    const uint32_t zat = zr0 * 128 + (tid & 7) * 16;
    auto piece = [&](int j, uint4 (&out)[PARTS]) {  // (weights of rows behind m: of zeros)
      const int r = zr0 + j * (NT / 8);
      weighted<PARTS>(*reinterpret_cast<const uint4*>(s.z[zb] + zat + j * (NT * 16)), s.pw[Z0 + (rev ? r : max(m - 1 - r, 0))], out);
    };
    uint4 held[PARTS == 1 ? ZR : 1][1];
    if constexpr (PARTS == 1) {
      if (update)
#pragma unroll
        for (int j = 0; j < ZR; ++j) piece(j, held[j]);
    }
    if constexpr (!STATES) {
      ok = mbar_wait_lean(&s.bar_a, i & 1, p.err, PATH_PAGED_WAIT + 22) && ok;
      tc_fence_after();
    }
    if (update) {
#pragma unroll
      for (int j = 0; j < ZR; ++j) {
        if constexpr (PARTS == 1) {
          *reinterpret_cast<uint4*>(s.zs[0] + zat + j * (NT * 16)) = held[j][0];
        } else {
          uint4 out[PARTS];
          piece(j, out);
#pragma unroll
          for (int t = 0; t < PARTS; ++t) *reinterpret_cast<uint4*>((t ? rest(t) : s.zs[0]) + zat + j * (NT * 16)) = out[t];
        }
      }
      fence_proxy_async_smem();
    }
    if constexpr (!STATES) {
      const int r = 32 * quad + lane;
      uint32_t a[32];
      if (inter) {  // what lies before the chunk, weighted
        tmem_ld32(tb + lane_off + COL_O + 32 * half, a);
        const float w = s.pw[Z0 + (rev ? max(m - r, 0) : r + 1)];
        const uint64_t ww = f2(w, w);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t v = f2_mul(f2_bits(a[e], a[e + 1]), ww);
          a[e] = (uint32_t)v, a[e + 1] = (uint32_t)(v >> 32);
        }
        tmem_st32(tb + lane_off + COL_O + 32 * half, a);
      }
      // P over S: a warp's 64 columns become 32 of packed pairs in the place of their first half
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int jb = 2 * half + q;
        uint32_t b[16];
        if (jb == quad || (jb < quad) != rev) {
          tmem_ld32(tb + lane_off + COL_S + 32 * jb, a);
          if (jb == quad) {
            const float* w = &s.pw[Z0 + (rev ? -lane : lane)];
            tmem_ld_wait();
            if (rev) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) b[e / 2] = pack_pair(f2_mul(f2_bits(a[e], a[e + 1]), f2(w[e], w[e + 1])));
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2) b[e / 2] = pack_pair(f2_mul(f2_bits(a[e], a[e + 1]), f2(w[-e], w[-e - 1])));
            }
          } else {
            const float w = s.pw[Z0 + (rev ? 32 * jb - r : r - 32 * jb - 31)];
            const uint64_t ww = f2(w, w);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const ulonglong2 cw = *reinterpret_cast<const ulonglong2*>(&s.colw[e]);
              b[e / 2] = pack_pair(f2_mul(f2_mul(f2_bits(a[e], a[e + 1]), cw.x), ww));
              b[e / 2 + 1] = pack_pair(f2_mul(f2_mul(f2_bits(a[e + 2], a[e + 3]), cw.y), ww));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) b[e] = 0;
        }
        tmem_st16(tb + lane_off + COL_S + 64 * half + 16 * q, b);
      }
      tmem_st_wait();
    }
    tc_fence_before();
    if (!__syncthreads_and(ok)) break;
    if (warp == lead) {
      tc_fence_after();
      if (update) issue_delta(yb, gy > 1 && g > 0 ? 1u : 0u);
      if constexpr (!STATES) {
        const uint32_t a_z = at16(s.z[0]) + zb * (TILE / 16);
        const uint32_t first = uniform(old || (gy > 1 && g > 0) ? 1u : 0u);
#pragma unroll
        for (int e = 0; e < C / 16; ++e)
          mma_ts_elect(tbu + COL_O, tbu + COL_S + (e < 4 ? 8 * e : 32 + 8 * e), md + (a_z + 128u * e), id_o, e ? 1u : first);
        commit_elect(&s.bar_c);
        if ((gx > 1 || last) && !(PARTS > 1 && update)) load_x(last ? k + 1 : k, last || gx == 1 ? 0 : g + 1);
      }
    }
    if (update) {
      ok = mbar_wait_lean(&s.bar_b, un & 1, p.err, PATH_PAGED_WAIT + 23) && ok;
      ++un;
      if (warp == lead && __all_sync(0xffffffffu, ok)) {
        if (PARTS > 1) load_x(k + 1, 0);
        next_y(yn + NY);
        if (STATES) next_z(yn + NZ);
      }
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
      ok = mbar_wait_lean(&s.bar_c, i & 1, p.err, PATH_PAGED_WAIT + 24) && ok;
      tc_fence_after();
      if (warp == lead && update && __all_sync(0xffffffffu, ok)) next_z(yn + NZ);
      const int r = 32 * quad + lane;
      if (gx > 1 || last) {
        uint32_t a[32];
        tmem_ld32(tb + lane_off + COL_O + 32 * half, a);
        __nv_bfloat16* o = (__nv_bfloat16*)op.o + (p.packed ? 0 : it.seq * op.xb) + (long long)(row0 + c * C + r) * op.xt +
                           (long long)(h * gx + (gx > 1 ? g : 0)) * op.xh + v0 + 32 * half;
        const bool wide = (reinterpret_cast<uintptr_t>(op.o) & 31) == 0;
        const uint64_t scale = f2(p.scale, p.scale);
        tmem_ld_wait();
        if (r < m)
#pragma unroll
          for (int e = 0; e < 32; e += 16) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = pack_pair(f2_mul(f2_bits(a[e + 2 * j], a[e + 2 * j + 1]), scale));
            store32(o + e, w, wide);
          }
      }
    }
    tc_fence_before();
    if (!STATES && !__syncthreads_and(ok)) break;
    if (gy > 1 || last) ++yn;
    if (gx > 1 || last) ++xn;
    if (last) g = 0, ++k;
    else ++g;
  }
  if (__syncthreads_and(ok)) {
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
  tc_fence_before();
  __syncthreads();
  if (warp == lead) {
    tc_fence_after();
    tmem_dealloc(tb, COLS);
  }
}

// [planes][rows][D] bf16, `row` and `plane` elements apart, in boxes of 128 rows x 64 columns; rows behind the last read as
// zero.
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
    if (!make_map(&maps.x[i], op.x, p.D, rows, nx, op.xt, op.xh) ||
        !make_map(&maps.y[i], op.y, p.D, rows, ny, op.yt, op.yh) || !make_map(&maps.z[i], op.z, p.D, rows, ny, op.yt, op.yh))
      return cudaErrorInvalidValue;
  }
  // (a cache's states: whether or not they are written, for the same outputs)
  if (p.D == 64) {
    if (states) return p.state ? launch<64, true, 3>(maps, p, st) : launch<64, true, 1>(maps, p, st);
    return p.state ? launch<64, false, 3>(maps, p, st) : launch<64, false, 1>(maps, p, st);
  }
  if (states) return p.state ? launch<128, true, 3>(maps, p, st) : launch<128, true, 1>(maps, p, st);
  return p.state ? launch<128, false, 3>(maps, p, st) : launch<128, false, 1>(maps, p, st);
}

}  // namespace pathattn
