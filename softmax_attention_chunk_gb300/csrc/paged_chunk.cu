// Paged serving: attention of new tokens over a paged cache, CUDA-core kernels in fp32 arithmetic (fp32 caches).
//
// Mathematics (one sequence, one key head; t0 cached rows, n new tokens with rows of W and beta; the UT
// representation of the PaTH reading notes, cc.laoqi.cc/papers/2505.16381, §2.6-§2.8).  The new
// tokens are cut into chunks of B rows.  Per chunk
//   U = (I + strictLower(D W W^T))^-1 D,   X = U strictLower(W K^T),   Y = U^T W,
//   Q<- = Q - lower(Q W^T) U W   (queries at the chunk's start),   K-> = K - X^T W   (keys at its end),
//   F = I - W^T Y = H_first ... H_last,   S_diag = lower(Q K^T) - lower(Q W^T) X.
// A query meets the earlier new chunks right to left, Z <- Z F_c^T, and arrives at the start of the new
// tokens as z; the logit of a cached row is then z . k~ (k~ as the cache holds it).  The new keys walk to
// the end of the call, K->_c F_{c+1} ... F_last, and the cached rows become k~ M, M = F_0 ... F_last.
//
// Six launches: plan (lengths, chunk list), chunk preparation, then one of {query scan, key walk} per
// block, cached attention split over key ranges, cached rewrite, and the merge of the splits.
//
// Bound: fp32 multiply-adds and shared-memory reads of the products on the CUDA cores (operands as three bf16 parts each
// would keep 24 bits on the tensor cores too; not built); products keep
// 2 x 4 results per thread, tiles move 16 bytes at a time, the merge takes a row's ranges side by side (262 -> 184 -> 140 ->
// 116 -> 109 us for 3 slots of 5 to 97 tokens over up to 1500 rows x 8 heads, head dim 64: what is left is a chain of six
// launches with few blocks each, every one a chain of products; attention 25, scan and walk 33, rewrite 17).
#include "paged.h"
#include "dev_common.cuh"

namespace pathattn {
namespace {

constexpr int NT = 256;
constexpr int B = kPagedChunk;
constexpr int KT = 64;  // cached rows per tile

// C = op(A) op(B) of matrices in shared memory, fp32: op(A)(i, k) = TA ? A[k lda + i] : A[i lda + k], op(B)(k, j) = TB ?
// B[j ldb + k] : B[k ldb + j].  2 x 4 results per thread, 16-byte loads along whichever index is contiguous; every
// result goes to epi(i, j, value).
template <int M, int N, int K, bool TA, bool TB, typename Epi>
__device__ __forceinline__ void product(const float* A, int lda, const float* B, int ldb, Epi epi) {
  static_assert(M % 2 == 0 && N % 4 == 0 && K % 4 == 0, "tile shape");
  auto ld4 = [](const float* q) { return *reinterpret_cast<const float4*>(q); };
  auto at = [](const float4& v, int e) { return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w; };
  constexpr int TN = N / 4, TILES = M / 2 * TN;
  for (int tile = threadIdx.x; tile < TILES; tile += NT) {
    // columns of a thread lie TN apart where B is read along k (neighbouring threads then read neighbouring rows)
    const int i0 = tile / TN * 2, jt = tile % TN;
    float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
      float a[2][4];
      if (TA) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = *reinterpret_cast<const float2*>(A + (k + e) * lda + i0);
          a[0][e] = v.x;
          a[1][e] = v.y;
        }
      } else {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float4 v = ld4(A + (i0 + y) * lda + k);
          a[y][0] = v.x; a[y][1] = v.y; a[y][2] = v.z; a[y][3] = v.w;
        }
      }
      if (TB) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 v = ld4(B + (jt + j * TN) * ldb + k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[0][j] = fmaf(a[0][e], at(v, e), c[0][j]);
            c[1][j] = fmaf(a[1][e], at(v, e), c[1][j]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v = ld4(B + (k + e) * ldb + 4 * jt);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            c[0][j] = fmaf(a[0][e], at(v, j), c[0][j]);
            c[1][j] = fmaf(a[1][e], at(v, j), c[1][j]);
          }
        }
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int j = 0; j < 4; ++j) epi(i0 + y, TB ? jt + j * TN : 4 * jt + j, c[y][j]);
  }
}

// Workspace (element offsets are computed on the host and the device from the same sizes).
struct ChunkWs {
  int most, group;     // slots with several new tokens: of any legal call, of a round
  int nch;             // chunk slots: at least the chunks of any legal round
  int nsplit;          // key ranges of the cached attention (range 0 also carries the new tokens' state)
  size_t plan;         // int [3][slots + 1]: first chunk of each slot, first live cached tile, slots of the round before it
  size_t kr, f;        // K-> [nch][H][B][D], F [nch][H][D][D]
  size_t fa, ft;       // forget gate: inclusive sums inside the chunk [nch][H][B], chunk totals [nch][H]
  size_t z, qb;        // Q<-, then z [nch][hq][B][D]; row biases sum of log f since t0 [nch][hq][B]
  size_t m, l, acc;    // softmax states [nsplit][nch][hq][B](, [D])
  size_t mm;           // M [group][H][D][D]
  size_t total;
};
ChunkWs chunk_ws(const PagedArgs& p, int group) {  // for rounds of `group` slots
  ChunkWs w{};
  w.group = group;
  const size_t D = p.c.head_dim, H = p.c.heads, hq = p.hq;
  // every slot may end in a partly filled chunk
  const long long tokens = p.total < (long long)p.max_new * group ? p.total : (long long)p.max_new * group;
  const long long most = (tokens + (long long)(B - 1) * group) / B;
  w.nch = (int)(most < 1 ? 1 : most);
  const long long ctas = (long long)w.nch * p.hq;
  w.nsplit = ctas >= 1216 ? 1 : (int)((1216 + ctas - 1) / ctas);
  if (w.nsplit > 64) w.nsplit = 64;
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align_up(off + bytes, 256); return o; };
  w.plan = take((size_t)3 * (p.c.slots + 1) * 4);
  w.kr = take((size_t)w.nch * H * B * D * 4);
  w.f = take((size_t)w.nch * H * D * D * 4);
  w.fa = take((size_t)w.nch * H * B * 4);
  w.ft = take((size_t)w.nch * H * 4);
  w.z = take((size_t)w.nch * hq * B * D * 4);
  w.qb = take((size_t)w.nch * hq * B * 4);
  w.m = take((size_t)w.nsplit * w.nch * hq * B * 4);
  w.l = take((size_t)w.nsplit * w.nch * hq * B * 4);
  w.acc = take((size_t)w.nsplit * w.nch * hq * B * D * 4);
  w.mm = take((size_t)group * H * D * D * 4);
  w.total = off;
  return w;
}
ChunkWs chunk_ws(const PagedArgs& p) {
  const int most = most_multi(p);
  ChunkWs w = chunk_ws(p, round_slots(most, [&](int n) { return chunk_ws(p, n).total; }));
  w.most = most;
  return w;
}

__device__ __forceinline__ SlotSpan chunk_span(const PagedArgs& p, int b) {
  SlotSpan s = slot_span(p, b);
  if (s.n < p.min_new) s.n = 0;
  return s;
}

// First chunk and first live tile of every slot, and the slots of the round before it (exclusive prefix sums; entry `slots`
// holds the totals).  Slots with several new tokens are numbered in order: the round takes `group` of them from number
// `first` on, and those from number `most` on are left out.
__global__ void __launch_bounds__(1024) plan_kernel(PagedArgs p, int* plan, int first, int group, int most) {
  chain();
  __shared__ int wsum[2][32], multi[32];
  __shared__ int carry[2];
  __shared__ unsigned long long tokens;
  const bool report = first == 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* cstart = plan;
  int* tstart = plan + p.c.slots + 1;
  int* mstart = tstart + p.c.slots + 1;
  if (tid < 2) carry[tid] = 0;
  if (tid == 0) tokens = 0;
  int numbered = 0;  // slots with several new tokens so far
  __syncthreads();
  for (int base = 0; base < p.c.slots; base += 1024) {
    const int b = base + tid;
    int nc = 0, nt = 0;
    SlotSpan s{};
    if (b < p.c.slots) {
      s = chunk_span(p, b);
      if (report && s.code) paged_error(p.c.status, s.code);
    }
    const int n = s.n;
    leave_out_pageless(p.c, b, s.t0, n, s, report);
    const int number = number_multi(s.n > 0, multi, numbered);
    if (s.n > 0) {
      atomicAdd(&tokens, (unsigned long long)s.n);
      if (number >= most) {
        s.n = 0;
        if (report) paged_error(p.c.status, PATH_PAGED_BAD_START);
      }
    }
    if (report && n > 0) note_extended(p.c, b, s.n > 0 ? n : -1);
    const int before = number - first;
    if (s.n > 0 && before >= 0 && before < group) {
      nc = (s.n + B - 1) / B;
      nt = live_tiles(s.t0, p.window, p.sinks, KT).count;
    }
    if (b < p.c.slots) mstart[b] = before < 0 ? 0 : before < group ? before : group;
    int ic = nc, it = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, ic, o), e = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) { ic += a; it += e; }
    }
    if (lane == 31) { wsum[0][warp] = ic; wsum[1][warp] = it; }
    __syncthreads();
    int oc = carry[0], ot = carry[1];
    for (int w = 0; w < warp; ++w) { oc += wsum[0][w]; ot += wsum[1][w]; }
    if (b < p.c.slots) { cstart[b] = oc + ic - nc; tstart[b] = ot + it - nt; }
    __syncthreads();
    if (tid == 1023) { carry[0] = oc + ic; carry[1] = ot + it; }
    __syncthreads();
  }
  if (tid == 0) {
    cstart[p.c.slots] = carry[0];
    tstart[p.c.slots] = carry[1];
    const int left = min(numbered, most) - first;
    mstart[p.c.slots] = left < 0 ? 0 : left < group ? left : group;
  }
  // rows of q_start that overlap: more tokens than the workspace is for
  if (tokens > (unsigned long long)p.total) {
    if (tid == 0) paged_error(p.c.status, PATH_PAGED_BAD_START);
    __syncthreads();
    for (int b = tid; b <= p.c.slots; b += 1024) {
      if (report && b < p.c.slots && chunk_span(p, b).n > 0) note_extended(p.c, b, -1);
      cstart[b] = tstart[b] = mstart[b] = 0;
    }
  }
}

// The slot that owns entry x of a prefix array with x < start[slots].
__device__ __forceinline__ int owner(const int* start, int slots, int x) {
  int lo = 0, hi = slots;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <int D>
struct PrepSmem {
  static constexpr int DS = D + 4, BS = B + 4;
  static constexpr int kW = 0, kK = kW + B * DS, kQ = kK + B * DS, kV = kQ + B * DS, kY = kV + B * DS;
  static constexpr int kU = kY + B * DS, kX = kU + B * BS, kG = kX + B * BS, kN = kG + B * BS;
  static constexpr int kM1 = kN + B * BS, kA = kM1 + B * BS, kS = kA + B * BS;
  static constexpr int kBeta = kS + B * BS, kLf = kBeta + B, total = kLf + B;
};

// One block per (chunk, key head).
template <int D>
__global__ void __launch_bounds__(NT) prep_kernel(PagedArgs p, ChunkWs w, char* ws) {
  chain();
  extern __shared__ float sm[];
  using S = PrepSmem<D>;
  constexpr int DS = S::DS, BS = S::BS;
  float *sW = sm + S::kW, *sK = sm + S::kK, *sQ = sm + S::kQ, *sV = sm + S::kV, *sY = sm + S::kY;
  float *sU = sm + S::kU, *sX = sm + S::kX, *sG = sm + S::kG, *sN = sm + S::kN, *sM1 = sm + S::kM1;
  float *sA = sm + S::kA, *sS = sm + S::kS, *sBeta = sm + S::kBeta, *sLf = sm + S::kLf;
  const int* cstart = (const int*)(ws + w.plan);
  const int c = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, H = p.c.heads;
  if (c >= cstart[p.c.slots]) return;
  const int b = owner(cstart, p.c.slots, c);
  const SlotSpan sp = chunk_span(p, b);
  const int r0 = (c - cstart[b]) * B, rows = min(B, sp.n - r0);
  const float *k = (const float*)p.k, *v = (const float*)p.v, *wv = (const float*)p.w, *q = (const float*)p.q;
  const size_t tok0 = (size_t)sp.q0 + r0;
#pragma unroll
  for (int i = 0; i < B * (D / 4) / NT; ++i) {
    const int e = i * NT + tid, r = e / (D / 4), x = e % (D / 4) * 4;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t at = ((tok0 + (r < rows ? r : 0)) * H + h) * D + x;
    auto get = [&](const float* src) { return r < rows ? *reinterpret_cast<const float4*>(src + at) : none; };
    const float4 w4 = get(wv), k4 = get(k), v4 = get(v);
    *reinterpret_cast<float4*>(sW + r * DS + x) = w4;
    *reinterpret_cast<float4*>(sK + r * DS + x) = k4;
    *reinterpret_cast<float4*>(sV + r * DS + x) = v4;
  }
  if (tid < B) {
    const bool ok = tid < rows;
    sBeta[tid] = ok ? clamp_beta(p.beta[(tok0 + tid) * H + h]) : 0.f;
    float a = ok && p.log_f ? p.log_f[(tok0 + tid) * H + h] : 0.f;  // inclusive sums by a warp scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, a, o);
      if (tid >= o) a += y;
    }
    sLf[tid] = a;
  }
  __syncthreads();
  product<B, B, D, false, true>(sW, DS, sW, DS, [&](int i, int j, float x) { sG[i * BS + j] = j < i ? x : 0.f; });
  product<B, B, D, false, true>(sW, DS, sK, DS, [&](int i, int j, float x) { sN[i * BS + j] = j < i ? x : 0.f; });
  __syncthreads();
  // U by forward substitution, one column per lane: u_i = beta_i (e_i - sum_{m<i} G_im u_m)
  if (tid < 32) {
    float u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float a0 = (tid == i) ? 1.f : 0.f, a1 = 0.f;
#pragma unroll
      for (int m = 0; m + 1 < i; m += 2) {
        a0 -= sG[i * BS + m] * u[m];
        a1 -= sG[i * BS + m + 1] * u[m + 1];
      }
      if (i & 1) a0 -= sG[i * BS + i - 1] * u[i - 1];
      u[i] = sBeta[i] * (a0 + a1);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) sU[i * BS + tid] = u[i];
  }
  __syncthreads();
  product<B, B, B, false, false>(sU, BS, sN, BS, [&](int i, int j, float x) { sX[i * BS + j] = x; });
  product<B, D, B, true, false>(sU, BS, sW, DS, [&](int m, int n, float x) { sY[m * DS + n] = x; });
  __syncthreads();
  {
    float* kr = (float*)(ws + w.kr) + ((size_t)c * H + h) * B * D;
    float* f = (float*)(ws + w.f) + ((size_t)c * H + h) * D * D;
    product<B, D, B, true, false>(sX, BS, sW, DS, [&](int j, int n, float x) { kr[j * D + n] = sK[j * DS + n] - x; });
    product<D, D, B, true, false>(sW, DS, sY, DS, [&](int n, int x, float y) { f[n * D + x] = (n == x ? 1.f : 0.f) - y; });
    if (p.log_f && tid < B) ((float*)(ws + w.fa))[((size_t)c * H + h) * B + tid] = sLf[tid];
    if (p.log_f && tid == 0) ((float*)(ws + w.ft))[(size_t)c * H + h] = sLf[B - 1];
  }
  for (int g = 0; g < p.G; ++g) {
    const int qh = h * p.G + g;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < B * (D / 4) / NT; ++i) {
      const int e = i * NT + tid, r = e / (D / 4), x = e % (D / 4) * 4;
      *reinterpret_cast<float4*>(sQ + r * DS + x) =
          r < rows ? *reinterpret_cast<const float4*>(q + ((tok0 + r) * p.hq + qh) * D + x) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    product<B, B, D, false, true>(sQ, DS, sW, DS, [&](int i, int j, float x) { sM1[i * BS + j] = j <= i ? x : 0.f; });
    product<B, B, D, false, true>(sQ, DS, sK, DS, [&](int i, int j, float x) { sS[i * BS + j] = x; });
    __syncthreads();
    product<B, B, B, false, false>(sM1, BS, sU, BS, [&](int i, int j, float x) { sA[i * BS + j] = x; });
    product<B, B, B, false, false>(sM1, BS, sX, BS, [&](int i, int j, float x) { sS[i * BS + j] -= x; });
    __syncthreads();
    const size_t row = ((size_t)c * p.hq + qh) * B;
    float* z = (float*)(ws + w.z) + row * D;
    product<B, D, B, false, false>(sA, BS, sW, DS, [&](int i, int n, float x) { z[i * D + n] = sQ[i * DS + n] - x; });
    // softmax of the diagonal chunk: 8 threads per row (log2 domain)
    const int r = tid >> 3, sub = tid & 7;
    float mx = -INFINITY;
    for (int j = sub; j < B; j += 8) {
      float s = -INFINITY;
      if (j <= r && r < rows && sees(p.window, p.sinks, sp.t0 + r0 + r, sp.t0 + r0 + j))
        s = sS[r * BS + j] * p.scl + (sLf[r] - sLf[j]) * kLog2e;
      sS[r * BS + j] = s;
      mx = fmaxf(mx, s);
    }
    mx = group_max<8>(mx);
    float l = 0.f;
    for (int j = sub; j < B; j += 8) {
      const float s = sS[r * BS + j];
      const float e = s == -INFINITY ? 0.f : fast_exp2(s - mx);
      sS[r * BS + j] = e;
      l += e;
    }
    l = group_sum<8>(l);
    if (sub == 0) {
      ((float*)(ws + w.m))[row + r] = mx;
      ((float*)(ws + w.l))[row + r] = l;
    }
    __syncthreads();
    float* acc = (float*)(ws + w.acc) + row * D;
    product<B, D, B, false, false>(sS, BS, sV, DS, [&](int i, int n, float x) { acc[i * D + n] = x; });
  }
}

template <int D>
struct ScanSmem {
  static constexpr int DS = D + 4, KS = B + 4;
  static constexpr int kZ = 0, kZn = kZ + B * DS, kK = kZn + B * DS, kV = kK + B * DS, kAcc = kV + B * DS;
  static constexpr int kP = kAcc + B * DS;
  static constexpr int kM = kP + B * KS, kF = kM + B * 3;  // kM: maximum, sum, row bias
};

// R rows of D floats between memory (row pitch in floats) and a tile in shared memory (row pitch ds), 16 bytes at a time.
template <int R, int D>
__device__ __forceinline__ void tile_in(float* dst, int ds, const float* src, size_t pitch) {
#pragma unroll
  for (int i = 0; i < R * (D / 4) / NT; ++i) {
    const int e = i * NT + threadIdx.x, r = e / (D / 4), x = e % (D / 4) * 4;
    *reinterpret_cast<float4*>(dst + r * ds + x) = *reinterpret_cast<const float4*>(src + (size_t)r * pitch + x);
  }
}
template <int R, int D>
__device__ __forceinline__ void tile_out(float* dst, const float* src, int ds) {
#pragma unroll
  for (int i = 0; i < R * (D / 4) / NT; ++i) {
    const int e = i * NT + threadIdx.x, r = e / (D / 4), x = e % (D / 4) * 4;
    *reinterpret_cast<float4*>(dst + (size_t)r * D + x) = *reinterpret_cast<const float4*>(src + r * ds + x);
  }
}

// Online softmax of the score tile sP [B][nk] (already masked, log2 domain): probabilities replace the
// scores, the row's maximum and sum are updated and acc rescaled.  All threads; ends with a barrier.
template <int D>
__device__ __forceinline__ void softmax_step(float* sP, int ps, int nk, float* sM, float* sAcc, int ds) {
  const int r = threadIdx.x >> 3, sub = threadIdx.x & 7;
  float mx = -INFINITY;
  for (int j = sub; j < nk; j += 8) mx = fmaxf(mx, sP[r * ps + j]);
  mx = group_max<8>(mx);
  const float mo = sM[r], mn = fmaxf(mo, mx);
  const float corr = mn == -INFINITY ? 1.f : fast_exp2(mo - mn);
  float l = 0.f;
  for (int j = sub; j < nk; j += 8) {
    const float s = sP[r * ps + j];
    const float e = s == -INFINITY ? 0.f : fast_exp2(s - mn);
    sP[r * ps + j] = e;
    l += e;
  }
  l = group_sum<8>(l);
  for (int x = sub; x < D; x += 8) sAcc[r * ds + x] *= corr;
  __syncwarp();
  if (sub == 0) {
    sM[r] = mn;
    sM[B + r] = sM[B + r] * corr + l;
  }
  __syncthreads();
}

// Query scan over the earlier new chunks of the slot: one block per (chunk, query head).
template <int D>
__device__ void scan_block(const PagedArgs& p, const ChunkWs& w, char* ws, float* sm, int c, int qh) {
  using S = ScanSmem<D>;
  constexpr int DS = S::DS, KS = S::KS;
  float *sZ = sm + S::kZ, *sZn = sm + S::kZn, *sK = sm + S::kK, *sV = sm + S::kV, *sAcc = sm + S::kAcc;
  float *sP = sm + S::kP, *sM = sm + S::kM, *sF = sm + S::kF;
  const int* cstart = (const int*)(ws + w.plan);
  const int tid = threadIdx.x, H = p.c.heads, h = qh / p.G;
  const int b = owner(cstart, p.c.slots, c);
  const SlotSpan sp = chunk_span(p, b);
  const int lc = c - cstart[b], rows = min(B, sp.n - lc * B);
  const size_t row = ((size_t)c * p.hq + qh) * B;
  float* z = (float*)(ws + w.z) + row * D;
  float* acc = (float*)(ws + w.acc) + row * D;
  float *gm = (float*)(ws + w.m) + row, *gl = (float*)(ws + w.l) + row;
  const float* fa = (const float*)(ws + w.fa);
  const float* ft = (const float*)(ws + w.ft);
  if (lc == 0) {  // already at the start of the new tokens
    if (p.log_f && tid < B) ((float*)(ws + w.qb))[row + tid] = fa[((size_t)c * H + h) * B + tid];
    return;
  }
  tile_in<B, D>(sZ, DS, z, D);
  tile_in<B, D>(sAcc, DS, acc, D);
  if (tid < B) {
    sM[tid] = gm[tid];
    sM[B + tid] = gl[tid];
    sM[2 * B + tid] = p.log_f ? fa[((size_t)c * H + h) * B + tid] : 0.f;  // row bias so far
  }
  const float* v = (const float*)p.v;
  for (int c2 = lc - 1; c2 >= 0; --c2) {
    const size_t cc = (size_t)(c - lc + c2) * H + h;
    const float* kr = (const float*)(ws + w.kr) + cc * B * D;
    const float* f = (const float*)(ws + w.f) + cc * D * D;
    const size_t tok = (size_t)sp.q0 + (size_t)c2 * B;
    __syncthreads();
    tile_in<B, D>(sK, DS, kr, D);
    tile_in<B, D>(sV, DS, v + (tok * H + h) * D, (size_t)H * D);  // (an earlier chunk is full)
    tile_in<D, D>(sF, DS, f, D);
    __syncthreads();
    product<B, B, D, false, true>(sZ, DS, sK, DS, [&](int i, int j, float x) {
      float s = -INFINITY;
      const int jn = c2 * B + j, in = lc * B + i;
      if (i < rows && sees(p.window, p.sinks, sp.t0 + in, sp.t0 + jn)) {
        s = x * p.scl;
        if (p.log_f) s += (sM[2 * B + i] + (ft[cc] - fa[cc * B + j])) * kLog2e;
      }
      sP[i * KS + j] = s;
    });
    product<B, D, D, false, true>(sZ, DS, sF, DS, [&](int i, int n, float x) { sZn[i * DS + n] = x; });
    __syncthreads();
    softmax_step<D>(sP, KS, B, sM, sAcc, DS);
    product<B, D, B, false, false>(sP, KS, sV, DS, [&](int i, int n, float x) { sAcc[i * DS + n] += x; });
    if (p.log_f && tid < B) sM[2 * B + tid] += ft[cc];
    float* t = sZ; sZ = sZn; sZn = t;
  }
  __syncthreads();
  tile_out<B, D>(z, sZ, DS);
  tile_out<B, D>(acc, sAcc, DS);
  if (tid < B) {
    gm[tid] = sM[tid];
    gl[tid] = sM[B + tid];
    if (p.log_f) ((float*)(ws + w.qb))[row + tid] = sM[2 * B + tid];
  }
}

// Key walk of one (slot m of the round, key head): the new rows to the end of the call and into the pages, M.
template <int D>
__device__ void walk_block(const PagedArgs& p, const ChunkWs& w, char* ws, float* sm, int m, int h) {
  constexpr int DS = D + 4;
  float *sR = sm, *sF = sR + D * DS, *sK = sF + D * DS;
  const int* cstart = (const int*)(ws + w.plan);
  const int* mstart = cstart + 2 * (p.c.slots + 1);
  const int tid = threadIdx.x, H = p.c.heads;
  if (m >= mstart[p.c.slots]) return;
  const int b = owner(mstart, p.c.slots, m);
  const SlotSpan sp = chunk_span(p, b);
  const int nc = cstart[b + 1] - cstart[b];
  float* kp = (float*)p.c.k_pool;
  float* vp = (float*)p.c.v_pool;
  const float* v = (const float*)p.v;
  // values and running sums
  for (int r = tid >> 4; r < sp.n; r += NT / 16) {
    const long long at = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 + r);
    if (at < 0) {
      paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
      continue;
    }
    for (int x = tid & 15; x < D; x += 16) vp[at * D + x] = v[(((size_t)sp.q0 + r) * H + h) * D + x];
  }
  if (p.log_f) {
    __shared__ float wsum[NT / 32];
    const long long last = sp.t0 > 0 ? pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 - 1) : -1;
    double a = last >= 0 ? load_sum(p.c, last) : 0.0;
    for (int base = 0; base < sp.n; base += NT) {
      const int r = base + tid;
      float x = r < sp.n ? p.log_f[((size_t)sp.q0 + r) * H + h] : 0.f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, x, o);
        if ((tid & 31) >= o) x += y;
      }
      __syncthreads();
      if ((tid & 31) == 31) wsum[tid >> 5] = x;
      __syncthreads();
      float before = 0.f, all = 0.f;
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) {
        if (i < tid >> 5) before += wsum[i];
        all += wsum[i];
      }
      const long long at = r < sp.n ? pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 + r) : -1;
      if (at >= 0) store_sum(p.c, at, a + before + x);
      a += all;
    }
  }
  for (int e = tid; e < D * D; e += NT) sR[(e / D) * DS + e % D] = (e / D == e % D) ? 1.f : 0.f;
  float* mm = (float*)(ws + w.mm) + ((size_t)m * H + h) * D * D;
  for (int lc = nc - 1; lc >= 0; --lc) {
    const size_t cc = (size_t)(cstart[b] + lc) * H + h;
    const float* kr = (const float*)(ws + w.kr) + cc * B * D;
    const float* f = (const float*)(ws + w.f) + cc * D * D;
    const int rows = min(B, sp.n - lc * B);
    __syncthreads();
    tile_in<B, D>(sK, DS, kr, D);
    tile_in<D, D>(sF, DS, f, D);
    __syncthreads();
    product<B, D, D, false, false>(sK, DS, sR, DS, [&](int i, int n, float x) {
      if (i < rows) {
        const long long at = pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, sp.t0 + lc * B + i);
        if (at >= 0) kp[at * D + n] = (lc == nc - 1 ? sK[i * DS + n] : x);
        else paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
      }
    });
    // R <- F_c R, by way of M's place in global memory until every thread has read R
    product<D, D, D, false, false>(sF, DS, sR, DS, [&](int i, int n, float x) { mm[i * D + n] = x; });
    __syncthreads();
    tile_in<D, D>(sR, DS, mm, D);
  }
}

template <int D>
constexpr size_t scan_walk_smem() {
  constexpr size_t scan = (size_t)(ScanSmem<D>::kF + D * (D + 4)) * 4;
  constexpr size_t walk = (size_t)(2 * D + B) * (D + 4) * 4;
  return scan > walk ? scan : walk;
}

// Blocks [0, group * H) walk keys, the others scan queries.
template <int D>
__global__ void __launch_bounds__(NT) scan_walk_kernel(PagedArgs p, ChunkWs w, char* ws) {
  chain();
  extern __shared__ float sm[];
  const int nw = w.group * p.c.heads;
  if ((int)blockIdx.x < nw) {
    walk_block<D>(p, w, ws, sm, blockIdx.x / p.c.heads, blockIdx.x % p.c.heads);
    return;
  }
  const int x = blockIdx.x - nw, c = x / p.hq;
  if (c >= ((const int*)(ws + w.plan))[p.c.slots]) return;
  scan_block<D>(p, w, ws, sm, c, x % p.hq);
}

// Cached attention: one block per (chunk, query head, key range).  A warp owns 8 query rows, its lanes two of a tile's
// 64 keys each: scores, softmax and (by columns) the output stay in registers, and only the probabilities pass through
// shared memory, within the warp.  Keys and values arrive by asynchronous copies behind the other product.  Bound: the
// products' shared-memory reads (per 64 multiply-adds of a thread 10 to 12 reads of 16 bytes, 4 cycles of the SM each for
// a warp): 2 x 150 tokens x 32 heads over 8100 rows, head dim 64 (20 GFLOP), 867 us, 23 TFLOP/s; with 2 x 4 results per
// thread and the softmax in shared memory the smaller case above took 38 us here in place of 25.
constexpr int AT = 128;  // threads
template <int D>
struct AttendSmem {
  static constexpr int DS = D + 4, PS = KT + 4;
  static constexpr int kZ = 0, kK = kZ + B * DS, kV = kK + KT * DS, kP = kV + KT * DS, kBias = kP + B * PS;
  static constexpr int kRow = kBias + 2 * KT, total = kRow + 2 * 2 * 2 * KT;  // places: two 64-bit ones per row and tile
};
template <int D>
__global__ void __launch_bounds__(AT, D == 64 ? 4 : 2) attend_kernel(PagedArgs p, ChunkWs w, char* ws) {
  chain();
  extern __shared__ __align__(16) float sm[];
  using S = AttendSmem<D>;
  constexpr int DS = S::DS, PS = S::PS, V = D / 32;  // V: columns of a lane
  float *sZ = sm + S::kZ, *sK = sm + S::kK, *sV = sm + S::kV, *sP = sm + S::kP;
  const int* cstart = (const int*)(ws + w.plan);
  const int c = blockIdx.x, qh = blockIdx.y, split = blockIdx.z, tid = threadIdx.x, lane = tid & 31, w8 = tid / 32 * 8;
  if (c >= cstart[p.c.slots]) return;
  const int h = qh / p.G, b = owner(cstart, p.c.slots, c);
  const SlotSpan sp = chunk_span(p, b);
  const int r0 = (c - cstart[b]) * B, rows = min(B, sp.n - r0);
  const LiveTiles lt = live_tiles(sp.t0, p.window, p.sinks, KT);
  const int per = (lt.count + w.nsplit - 1) / w.nsplit;
  const int i0 = min(split * per, lt.count), i1 = min(i0 + per, lt.count);
  const size_t row0 = ((size_t)c * p.hq + qh) * B;
  const size_t row = (size_t)split * w.nch * p.hq * B + row0;
  if (split == 0 && i0 >= i1) return;  // the new tokens' state stands
  float* acc_out = (float*)(ws + w.acc) + row * D;
  float *gm = (float*)(ws + w.m) + row, *gl = (float*)(ws + w.l) + row;
  if (i0 >= i1) {
    if (tid < B) {
      gm[tid] = -INFINITY;
      gl[tid] = 0.f;
    }
    return;
  }
  const float *kp = (const float*)p.c.k_pool, *vp = (const float*)p.c.v_pool;
  float a_last = 0.f, a_more = 0.f;  // the last row's sum, a pair
  if (p.log_f) {
    const long long last = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, sp.t0 - 1);
    if (last >= 0) {
      a_last = p.c.a_pool[last];
      a_more = sum_rest(p.c, last);
    }
  }
  long long* place = reinterpret_cast<long long*>(sm + S::kRow);  // [tile parity][key, value][row]: the pools' rows, or -1
  // Places and biases (a_last - a_j; hidden rows -inf) of tile i.  A row that no query of the chunk sees is not looked up
  // (its page may be gone); a row is there only with both its key and its value.
  auto look = [&](int i) {
    if (tid >= KT || i >= i1) return;
    const int j = live_tile(lt, i) * KT + tid, at = (i & 1) * 2 * KT + tid;
    long long ka = -1, va = -1;
    if (j < sp.t0 && sees(p.window, p.sinks, sp.t0 + r0, j)) {
      ka = pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, j);
      va = pool_row(p.c, p.c.v_table, p.c.v_pages, b, h, j);
      if (ka < 0 || va < 0) {
        ka = va = -1;
        paged_error(p.c.status, PATH_PAGED_BAD_PAGE);
      }
    }
    place[at] = ka;
    place[at + KT] = va;
    sm[S::kBias + (i & 1) * KT + tid] = va < 0 ? -INFINITY : p.log_f ? (a_last - p.c.a_pool[va]) + (a_more - sum_rest(p.c, va)) : 0.f;
  };
  auto fetch = [&](float* dst, const float* pool, int i, int value) {
    const long long* from = place + ((i & 1) * 2 + value) * KT;
#pragma unroll
    for (int y = 0; y < KT * (D / 4) / AT; ++y) {
      const int e = y * AT + tid, r = e / (D / 4), x = e % (D / 4) * 4;
      const long long at = from[r];
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + r * DS + x)),
                   "l"(pool + (at >= 0 ? at * D + x : 0)), "r"(at >= 0 ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look(i0);
  __syncthreads();
  fetch(sK, kp, i0, 0);
  fetch(sV, vp, i0, 1);
  look(i0 + 1);
  const float* z = (const float*)(ws + w.z) + row0 * D;
  for (int e = tid; e < B * (D / 4); e += AT) {
    const int r = e / (D / 4), x = e % (D / 4) * 4;
    *reinterpret_cast<float4*>(sZ + r * DS + x) = *reinterpret_cast<const float4*>(z + r * D + x);
  }
  float m[8], l[8], qb[8], acc[8][V];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    m[r] = split == 0 ? gm[w8 + r] : -INFINITY;
    l[r] = split == 0 && lane == 0 ? gl[w8 + r] : 0.f;
    qb[r] = p.log_f ? ((const float*)(ws + w.qb))[row0 + w8 + r] : 0.f;
#pragma unroll
    for (int x = 0; x < V; ++x) acc[r][x] = split == 0 ? acc_out[(w8 + r) * D + lane * V + x] : 0.f;
  }
  auto ld4 = [](const float* q) { return *reinterpret_cast<const float4*>(q); };
  for (int i = i0; i < i1; ++i) {
    const int j0 = live_tile(lt, i) * KT;
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    float s[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r) s[r][0] = s[r][1] = 0.f;
#pragma unroll 2
    for (int k = 0; k < D; k += 4) {
      const float4 k0 = ld4(sK + lane * DS + k), k1 = ld4(sK + (lane + 32) * DS + k);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float4 q = ld4(sZ + (w8 + r) * DS + k);
        s[r][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[r][0]))));
        s[r][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[r][1]))));
      }
    }
    const float* sB = sm + S::kBias + (i & 1) * KT;
    const float b0 = sB[lane], b1 = sB[lane + 32];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int pos = sp.t0 + r0 + w8 + r;
      const float x0 = b0 != -INFINITY && sees(p.window, p.sinks, pos, j0 + lane) ? s[r][0] * p.scl + (b0 + qb[r]) * kLog2e : -INFINITY;
      const float x1 = b1 != -INFINITY && sees(p.window, p.sinks, pos, j0 + lane + 32) ? s[r][1] * p.scl + (b1 + qb[r]) * kLog2e : -INFINITY;
      const float mn = fmaxf(m[r], group_max<32>(fmaxf(x0, x1)));
      const float corr = mn == -INFINITY ? 1.f : fast_exp2(m[r] - mn);
      const float e0 = x0 == -INFINITY ? 0.f : fast_exp2(x0 - mn), e1 = x1 == -INFINITY ? 0.f : fast_exp2(x1 - mn);
      m[r] = mn;
      l[r] = l[r] * corr + e0 + e1;
      sP[(w8 + r) * PS + lane] = e0;
      sP[(w8 + r) * PS + lane + 32] = e1;
#pragma unroll
      for (int x = 0; x < V; ++x) acc[r][x] *= corr;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (i + 1 < i1) fetch(sK, kp, i + 1, 0);
#pragma unroll 2
    for (int k = 0; k < KT; k += 4) {
      float v[4][V];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int x = 0; x < V; x += 2) {
          const float2 y = *reinterpret_cast<const float2*>(sV + (k + e) * DS + lane * V + x);
          v[e][x] = y.x;
          v[e][x + 1] = y.y;
        }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float4 q = ld4(sP + (w8 + r) * PS + k);
#pragma unroll
        for (int x = 0; x < V; ++x) acc[r][x] = fmaf(q.x, v[0][x], fmaf(q.y, v[1][x], fmaf(q.z, v[2][x], fmaf(q.w, v[3][x], acc[r][x]))));
      }
    }
    __syncthreads();
    if (i + 1 < i1) fetch(sV, vp, i + 1, 1);
    look(i + 2);
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const float ls = group_sum<32>(l[r]);
    if (lane == 0) {
      gm[w8 + r] = m[r];
      gl[w8 + r] = ls;
    }
#pragma unroll
    for (int x = 0; x < V; ++x) acc_out[(w8 + r) * D + lane * V + x] = acc[r][x];
  }
}

// k <- k M for the cached rows that a later token sees: blocks take runs of (live tile, head).
template <int D>
__global__ void __launch_bounds__(NT) rewrite_kernel(PagedArgs p, ChunkWs w, const char* ws) {
  chain();
  extern __shared__ float sm[];
  constexpr int DS = D + 4;
  float *sMm = sm, *sK = sMm + D * DS;
  const int* tstart = (const int*)(ws + w.plan) + p.c.slots + 1;
  const int tid = threadIdx.x, H = p.c.heads;
  const long long units = (long long)tstart[p.c.slots] * H;
  const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  float* kp = (float*)p.c.k_pool;
  int have = -1;  // (slot, head) whose M is in shared memory
  for (long long u = u0; u < u1; ++u) {
    // units of a slot: head-major, so that a block keeps its M
    const int b = owner(tstart, p.c.slots, (int)(u / H));
    const int nt = tstart[b + 1] - tstart[b];
    const long long in = u - (long long)tstart[b] * H;
    const int h = (int)(in / nt), i = (int)(in % nt);
    const SlotSpan sp = chunk_span(p, b);
    const LiveTiles lt = live_tiles(sp.t0, p.window, p.sinks, KT);
    const int j0 = live_tile(lt, i) * KT;
    __syncthreads();
    if (have != b * H + h) {
      const int m = tstart[p.c.slots + 1 + b];  // (mstart)
      const float* mm = (const float*)(ws + w.mm) + ((size_t)m * H + h) * D * D;
      tile_in<D, D>(sMm, DS, mm, D);
      have = b * H + h;
    }
    auto keep = [&](int j) { return j < sp.t0 && sees(p.window, p.sinks, sp.t0 + sp.n, j); };
    for (int r = tid >> 3; r < KT; r += NT / 8) {
      const long long at = keep(j0 + r) ? pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, j0 + r) : -1;
#pragma unroll
      for (int x = (tid & 7) * 4; x < D; x += 32)
        *reinterpret_cast<float4*>(sK + r * DS + x) =
            at >= 0 ? *reinterpret_cast<const float4*>(kp + at * D + x) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    product<KT, D, D, false, false>(sK, DS, sMm, DS, [&](int r, int n, float x) {
      if (keep(j0 + r)) {
        const long long at = pool_row(p.c, p.c.k_table, p.c.k_pages, b, h, j0 + r);
        if (at >= 0) kp[at * D + n] = (x);
      }
    });
  }
}

// Merge of the key ranges (at most 64): one warp per (row, query head), 8 rows per block.
template <int D>
__global__ void __launch_bounds__(NT) merge_kernel(PagedArgs p, ChunkWs w, const char* ws) {
  chain();
  constexpr int BR = NT / 32, V = D / 32;
  const int* cstart = (const int*)(ws + w.plan);
  const int c = blockIdx.x / (B / BR), qh = blockIdx.y, lane = threadIdx.x & 31;
  if (c >= cstart[p.c.slots]) return;
  const int b = owner(cstart, p.c.slots, c);
  const SlotSpan sp = chunk_span(p, b);
  const int r0 = (c - cstart[b]) * B, rows = min(B, sp.n - r0), r = blockIdx.x % (B / BR) * BR + (threadIdx.x >> 5);
  if (r >= rows) return;
  const float *gm = (const float*)(ws + w.m), *gl = (const float*)(ws + w.l), *ga = (const float*)(ws + w.acc);
  const size_t stride = (size_t)w.nch * p.hq * B, row = ((size_t)c * p.hq + qh) * B + r;
  // a range's maximum and sum per lane (two where there are more than 32)
  float m[2], f[2], l = 0.f;
#pragma unroll
  for (int y = 0; y < 2; ++y) m[y] = lane + 32 * y < w.nsplit ? gm[(lane + 32 * y) * stride + row] : -INFINITY;
  const float M = group_max<32>(fmaxf(m[0], m[1]));
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    f[y] = m[y] == -INFINITY ? 0.f : fast_exp2(m[y] - M);
    if (m[y] != -INFINITY) l += gl[(lane + 32 * y) * stride + row] * f[y];
  }
  l = group_sum<32>(l);
  float a[V];
#pragma unroll
  for (int x = 0; x < V; ++x) a[x] = 0.f;
#pragma unroll 4
  for (int s = 0; s < w.nsplit; ++s) {
    const float fs = __shfl_sync(0xffffffffu, s < 32 ? f[0] : f[1], s & 31);
#pragma unroll
    for (int x = 0; x < V; ++x) {
      const float v = ga[(s * stride + row) * D + x * 32 + lane];
      a[x] += fs == 0.f ? 0.f : v * fs;  // (a range that saw nothing has written nothing)
    }
  }
  float* o = (float*)p.o + (((size_t)sp.q0 + r0 + r) * p.hq + qh) * D;
  const float inv = 1.f / l;
#pragma unroll
  for (int x = 0; x < V; ++x) o[x * 32 + lane] = a[x] * inv;
}

template <int D>
cudaError_t chunk_t(const PagedArgs& p, char* ws, cudaStream_t st) {
  const ChunkWs w = chunk_ws(p);
  cudaError_t e;
  auto prep = prep_kernel<D>;
  auto scan = scan_walk_kernel<D>;
  auto att = attend_kernel<D>;
  auto rew = rewrite_kernel<D>;
  const size_t s1 = (size_t)PrepSmem<D>::total * 4, s2 = scan_walk_smem<D>();
  const size_t s3 = (size_t)AttendSmem<D>::total * 4, s4 = (size_t)(D + KT) * (D + 4) * 4;
  if ((e = cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s1)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(scan, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s2)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(att, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s3)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(rew, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s4)) != cudaSuccess) return e;
  for (int first = 0; first < w.most; first += w.group)
    if ((e = launch_chained(plan_kernel, 1, 1024, 0, st, p, (int*)(ws + w.plan), first, w.group, w.most)) != cudaSuccess ||
        (e = launch_chained(prep, dim3(w.nch, p.c.heads), NT, s1, st, p, w, ws)) != cudaSuccess ||
        (e = launch_chained(scan, w.group * p.c.heads + w.nch * p.hq, NT, s2, st, p, w, ws)) != cudaSuccess ||
        (e = launch_chained(att, dim3(w.nch, p.hq, w.nsplit), AT, s3, st, p, w, ws)) != cudaSuccess ||
        (e = launch_chained(rew, 608, NT, s4, st, p, w, ws)) != cudaSuccess ||
        (e = launch_chained(merge_kernel<D>, dim3(w.nch * (B / (NT / 32)), p.hq), NT, 0, st, p, w, ws)) != cudaSuccess)
      return e;
  return cudaSuccess;
}

}  // namespace

size_t paged_chunk_ws_bytes(const PagedArgs& p) {
  const ChunkWs w = chunk_ws(p);
  return round_bytes(w.total, w.group < w.most);
}

cudaError_t launch_paged_chunk(const PagedArgs& p, char* ws, cudaStream_t st) {
  return p.c.head_dim == kHeadDim ? chunk_t<kHeadDim>(p, ws, st) : chunk_t<kHeadDimWide>(p, ws, st);
}

size_t paged_ws_bytes(const PagedArgs& p) {
  size_t n = paged_token_ws_bytes(p);
  if (p.max_new > 1 && !paged_drafts(p)) n += p.c.cache_dtype == PATH_BF16 ? paged_new_ws_bytes(p) : paged_chunk_ws_bytes(p);
  return n;
}
cudaError_t launch_paged(const PagedArgs& p, char* ws, cudaStream_t st) {
  const cudaError_t e = launch_paged_token(p, ws, st);
  if (e != cudaSuccess || p.max_new <= 1 || paged_drafts(p)) return e;
  PagedArgs more = p;
  more.min_new = 2;
  char* rest = ws + paged_token_ws_bytes(p);
  return p.c.cache_dtype == PATH_BF16 ? launch_paged_new(more, rest, st) : launch_paged_chunk(more, rest, st);
}

}  // namespace pathattn
