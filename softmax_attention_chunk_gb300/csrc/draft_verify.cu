// Verification of drafted tokens against a target model's probabilities (path_draft_verify): acceptance of the drafts of a slot
// and the draw of the token after them, one cluster of blocks per slot.
//
// Every block of the cluster finds the first draft not kept (a few loads), takes a slice of the one row (target) or two
// (target, draft) that decide the next token, and sums r = max(0, p - q) over it; every warp writes its sum to every block of the
// cluster, and the warp in whose share the running sum passes uniform * total finds the entry.
// Sums: the result is an index, so sums that are only nearly right give wrong answers: the running sum passes its goal at
// another entry with probability (entries) * (error).  Sums are pairs of floats instead, the second what rounding took from the
// first: about 2^-44 of the sum.  double would be as exact and costs 13 us of the GPU's few FP64 units for 64 rows of 131072
// (with double for the warps' totals and the search alone: 25 us a call there, 19 without; of 5 tokens 12 and 8).  The sums of
// two entries at a time by paired arithmetic: 19 -> 16.5 us with the rows in L2.
// Bound: the rows' bytes, behind a chain of dependent loads (q_start, tokens, their probabilities) and before the search.  A
// warp keeps three loads of each row on their way through shared memory (64 rows of 131072 from HBM: 21 -> 17 us; asked for in
// L2 ahead of loads to registers instead: 24).
#include <cooperative_groups.h>

#include "dev_common.cuh"
#include "paged.h"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace pathattn {
namespace {

using namespace tc;

constexpr int NT = 256, NW = NT / 32;
constexpr int STEP = 512;        // entries whose sum a warp keeps apart
constexpr int kMaxSteps = 32;    // steps of a warp: one lane each in the search
constexpr int kMaxCluster = 8;
constexpr int RING = 4;          // loads of a warp in shared memory, all but one on their way

struct VerifyArgs {
  path_verify_desc_t d;
  int slots_cl;                  // blocks of a cluster
  int tile;                      // entries of a warp, a multiple of STEP
  const int *q_start, *tokens;
  const float* uniform;
  const void *target, *draft;
  int *keep, *next, *status;
};

__device__ __forceinline__ float positive(float x) { return x > 0.f ? x : 0.f; }  // (NaN: 0)

// N consecutive probabilities; those at and behind `left` are 0.
template <typename T, int N> __device__ __forceinline__ void load_n(const T* a, int left, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = left > 0 ? positive(to_f<T>(*a)) : 0.f;
  } else {  // 16-byte loads; rows are whole multiples of them
    uint4 x = left > 0 ? *reinterpret_cast<const uint4*>(a) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = positive(__uint_as_float(w[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = positive(__uint_as_float(w[i] << 16));
        v[2 * i + 1] = positive(__uint_as_float(w[i] & 0xffff0000u));
      }
    }
  }
}

// 16 bytes to shared memory, zeros where there are none.
__device__ __forceinline__ void cp_16(void* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Residual max(0, p - q) as an exact pair (hi, lo).
__device__ __forceinline__ float2 residual(float p, float q) {
  q = fminf(p, q);
  const float s = p - q;
  return make_float2(s, (p - s) - q);  // exact: p >= q >= 0
}
// sum (hi, lo) += r: the rounding of hi + r.x is found exactly and kept in lo.
__device__ __forceinline__ void add_pair(float2& sum, float2 r) {
  const float t = sum.x + r.x, b = t - sum.x;
  sum.y += ((sum.x - (t - b)) + (r.x - b)) + r.y;
  sum.x = t;
}
// The residuals of two entries to two sums, by paired arithmetic.
struct TwoSums {
  uint64_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(uint64_t p, uint64_t q) {  // p >= q
    const uint64_t minus = f2(-1.f, -1.f), s = f2_fma(q, minus, p), rest = f2_fma(q, minus, f2_fma(s, minus, p));
    const uint64_t t = f2_add(hi, s), b = f2_fma(hi, minus, t);
    lo = f2_add(lo, f2_add(f2_add(f2_fma(f2_fma(b, minus, t), minus, hi), f2_fma(b, minus, s)), rest));
    hi = t;
  }
  __device__ __forceinline__ float2 sum() const {
    float a, b, c, d;
    f2_split(hi, a, b);
    f2_split(lo, c, d);
    float2 x = make_float2(a, c);
    add_pair(x, make_float2(b, d));
    return x;
  }
};
__device__ __forceinline__ float2 shfl_up_pair(float2 x, int o) {
  return make_float2(__shfl_up_sync(0xffffffffu, x.x, o), __shfl_up_sync(0xffffffffu, x.y, o));
}
__device__ __forceinline__ float2 shfl_pair(float2 x, int l) {
  return make_float2(__shfl_sync(0xffffffffu, x.x, l), __shfl_sync(0xffffffffu, x.y, l));
}
// The lanes' running sums, N of them at once.
template <int N> __device__ __forceinline__ void warp_scan(float2 (&x)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 a = shfl_up_pair(x[j], o);
      if (lane >= o) add_pair(x[j], a);
    }
}
__device__ __forceinline__ bool some(float2 x) { return x.x + x.y > 0.f; }
// Whether a sum passes the goal u * all.
struct Goal {
  float up;    // of a total so small that products would lose bits (under 2^-60): 2^60
  float2 goal;
  __device__ __forceinline__ Goal(float u, float2 all) : up(all.x < 0x1p-60f ? 0x1p60f : 1.f) {
    goal.x = u * (all.x * up);
    goal.y = __fmaf_rn(u, all.x * up, -goal.x) + u * (all.y * up);
  }
  __device__ __forceinline__ bool passed(float2 sum) const {
    float2 d = make_float2(sum.x * up, sum.y * up);
    add_pair(d, make_float2(-goal.x, -goal.y));
    return some(d);
  }
};
// The first lane whose running sum passes the goal, or (rounding) the last with a positive part; -1: none is.
__device__ __forceinline__ int first_past(const Goal& goal, float2 upto, float2 part) {
  const unsigned past = __ballot_sync(0xffffffffu, goal.passed(upto) && some(part)), any = __ballot_sync(0xffffffffu, some(part));
  return past ? __ffs(past) - 1 : any ? 31 - __clz(any) : -1;
}

template <typename T, int N>
__global__ void __launch_bounds__(NT, 4) draft_verify_kernel(const VerifyArgs a) {
  chain();
  constexpr int LOADS = STEP / (32 * N);
  constexpr int PAIR = N > 1 ? 1 : 2;          // loads whose entries are taken in pairs
  constexpr int PER = kMaxCluster * NW / 32;  // warps' sums of the cluster to a lane
  __shared__ float2 warp_sum[2][kMaxCluster * NW];  // of every warp of the cluster; one for each round
  __shared__ int first_bad;
  __shared__ __align__(16) uint8_t ring[N > 1 ? NW : 1][RING][2][32][16];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster.block_rank(), b = blockIdx.x / a.slots_cl;
  int q0 = a.q_start[b], n = 0;
  {
    const long long dn = (long long)a.q_start[b + 1] - q0;
    if (q0 < 0 || dn < 0 || q0 + dn > a.d.total_tokens || dn > a.d.max_new) {
      if (rank == 0 && tid == 0) paged_error(a.status, PATH_PAGED_BAD_START);
    } else {
      n = (int)dn;
    }
  }
  if (n == 0) {  // (the whole cluster)
    if (rank == 0 && tid == 0) a.keep[b] = 0, a.next[b] = -1;
    return;
  }
  auto started = cluster.barrier_arrive();  // (waited for before the others' shared memory is written)
  const T* target = (const T*)a.target;
  const T* draft = (const T*)a.draft;
  const float u = a.uniform[q0];
  if (warp == 0) {
    int bad = n;
    for (int i0 = 1; i0 < n && bad == n; i0 += 32) {
      const int i = i0 + lane;
      bool good = true;
      if (i < n) {
        const int x = a.tokens[q0 + i];
        const float ui = a.uniform[q0 + i];
        good = (unsigned)x < (unsigned)a.d.vocab;
        if (!good && rank == 0) paged_error(a.status, PATH_PAGED_BAD_TOKEN);
        if (good) {
          const float p = positive(to_f<T>(target[(q0 + i - 1) * a.d.target_stride + x]));
          const float q = draft ? positive(to_f<T>(draft[(q0 + i) * a.d.draft_stride + x])) : 1.f;
          good = (double)ui * q < (double)p;
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !good);
      if (no) bad = i0 + __ffs(no) - 1;
    }
    if (lane == 0) {
      first_bad = bad;
      if (rank == 0) a.keep[b] = bad;
    }
  }
  __syncthreads();
  const int bad = first_bad;
  const T* p = target + (q0 + bad - 1) * a.d.target_stride;
  const T* q = draft && bad < n ? draft + (q0 + bad) * a.d.draft_stride : nullptr;
  int out = !draft && bad < n ? a.tokens[q0 + bad] : -1;  // the entry that is left out of p
  const int vocab = a.d.vocab, steps = a.tile / STEP;
  const int v0 = (rank * NW + warp) * a.tile;
  // The warp's next 512 bytes of each row on their way to shared memory: a lane's 16 bytes are its own, nobody else waits.
  int coming = 0;
  const int stop = min(vocab, v0 + a.tile);
  auto fetch = [&](int slot) {
    const int at = min(coming, vocab - N);
    cp_16(ring[warp][slot][0][lane], p + at, coming < stop);
    if (q) cp_16(ring[warp][slot][1][lane], q + at, coming < stop);
    cp_commit();
    coming += 32 * N;
  };
  for (int round = 0; round < 2; ++round) {
    float2 mine = make_float2(0.f, 0.f);  // of step `lane`
    if constexpr (N > 1) {
      coming = v0 + lane * N;
#pragma unroll
      for (int i = 0; i < RING - 1; ++i) fetch(i);
    }
    for (int s = 0; s < steps; ++s) {
      TwoSums sums;
#pragma unroll(N > 1 ? LOADS : 2)
      for (int j = 0; j < LOADS; j += PAIR) {
        float pv[PAIR * N], qv[PAIR * N];
        const int from = v0 + s * STEP + j * 32 * N;
        if constexpr (N > 1) {
          const int i = LOADS % RING ? s * LOADS + j : j;
          cp_wait<RING - 2>();
          load_n<T, N>((const T*)ring[warp][i % RING][0][lane], 1, pv);
          if (q) load_n<T, N>((const T*)ring[warp][i % RING][1][lane], 1, qv);
          fetch((i + RING - 1) % RING);
        } else {
          for (int i = 0; i < PAIR; ++i) {
            const int at = from + 32 * i + lane;
            load_n<T, N>(p + at, vocab - at, *reinterpret_cast<float(*)[N]>(pv + i));
            if (q) load_n<T, N>(q + at, vocab - at, *reinterpret_cast<float(*)[N]>(qv + i));
          }
        }
        if (out >= from && out < from + PAIR * 32 * N)
#pragma unroll
          for (int i = 0; i < PAIR * N; ++i)
            if (from + i / N * 32 * N + lane * N + i % N == out) pv[i] = 0.f;
#pragma unroll
        for (int i = 0; i < PAIR * N; i += 2)
          sums.add(f2(pv[i], pv[i + 1]), q ? f2(fminf(pv[i], qv[i]), fminf(pv[i + 1], qv[i + 1])) : 0);
      }
      float2 sum = sums.sum();
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        add_pair(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, o), __shfl_xor_sync(0xffffffffu, sum.y, o)));
      if (lane == s) mine = sum;
    }
    // The last copies (zeros) too: nothing orders two copies to one place, and the second round's first ones go to theirs.
    if constexpr (N > 1) cp_wait<0>();
    float2 upto[1] = {mine};
    warp_scan(upto);
    const float2 total = shfl_pair(upto[0], 31);
    if (round == 0) cluster.barrier_wait(std::move(started));
    if (lane < a.slots_cl) *cluster.map_shared_rank(&warp_sum[round][rank * NW + warp], lane) = total;
    cluster.sync();  // (the only one of a round: a block that leaves after it has written and been written to)
    // every warp finds the cluster's sum, and whether the goal lies in its own share
    float2 part[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int w = lane * PER + i;
      part[i] = w < a.slots_cl * NW ? warp_sum[round][w] : make_float2(0.f, 0.f);
    }
    float2 lane_sum = part[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) add_pair(lane_sum, part[i]);
    float2 lane_upto[1] = {lane_sum};
    warp_scan(lane_upto);
    const float2 all = shfl_pair(lane_upto[0], 31);
    if (!some(all) && round == 0 && (q || out >= 0)) {
      q = nullptr;  // nothing is left of the target: its own row
      out = -1;
      continue;
    }
    const Goal goal(u, all);
    const int l = first_past(goal, lane_upto[0], lane_sum);
    if (l < 0) {
      if (rank == 0 && tid == 0) a.next[b] = -1;
      return;
    }
    // the first part at which the running sum passes
    float2 run = shfl_up_pair(lane_upto[0], 1);
    if (lane == 0) run = make_float2(0.f, 0.f);
    float2 at_owner = run;
    bool there = false;
    int owner = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float2 old = run;
      add_pair(run, part[i]);
      if (!there && some(part[i])) {
        owner = i;
        at_owner = old;
        there = goal.passed(run);
      }
    }
    owner = __shfl_sync(0xffffffffu, lane * PER + owner, l);
    float2 before = shfl_pair(at_owner, l);
    if (owner != rank * NW + warp) return;
    float2 past = before;
    add_pair(past, upto[0]);
    const int s = first_past(goal, past, mine);
    if (s < 0) {  // (an infinity in the row)
      if (lane == 0) a.next[b] = -1;
      return;
    }
    const float2 prev = shfl_pair(upto[0], s > 0 ? s - 1 : 0);
    if (s > 0) add_pair(before, prev);
    // the step's entries again: 16 to a lane, then those of the lane at which the sum passes, one to a lane
    const int e0 = v0 + s * STEP + lane * (STEP / 32);
    TwoSums sums;
#pragma unroll
    for (int j = 0; j < STEP / 32; j += N < 2 ? 2 : N) {
      float pv[N < 2 ? 2 : N], qv[N < 2 ? 2 : N];
#pragma unroll
      for (int i = 0; i < (N < 2 ? 2 : 1); ++i) {
        load_n<T, N>(p + e0 + j + i, vocab - e0 - j - i, *reinterpret_cast<float(*)[N]>(pv + i));
        if (q) load_n<T, N>(q + e0 + j + i, vocab - e0 - j - i, *reinterpret_cast<float(*)[N]>(qv + i));
      }
#pragma unroll
      for (int i = 0; i < (N < 2 ? 2 : N); i += 2) {
        const float p0 = e0 + j + i == out ? 0.f : pv[i], p1 = e0 + j + i + 1 == out ? 0.f : pv[i + 1];
        sums.add(f2(p0, p1), q ? f2(fminf(p0, qv[i]), fminf(p1, qv[i + 1])) : 0);
      }
    }
    const float2 own = sums.sum();
    float2 own_upto[1] = {own};
    warp_scan(own_upto);
    past = before;
    add_pair(past, own_upto[0]);
    const int w = first_past(goal, past, own);
    int found = -1;
    if (w >= 0) {
      const float2 less = shfl_pair(own_upto[0], w > 0 ? w - 1 : 0);
      if (w > 0) add_pair(before, less);
      const int x = v0 + s * STEP + w * (STEP / 32) + lane, left = lane < STEP / 32 && x != out ? vocab - x : 0;
      float px[1], qx[1] = {0.f};
      load_n<T, 1>(p + x, left, px);
      if (q) load_n<T, 1>(q + x, left, qx);
      const float2 r = residual(px[0], qx[0]);
      float2 r_upto[1] = {r};
      warp_scan(r_upto);
      past = before;
      add_pair(past, r_upto[0]);
      const int i = first_past(goal, past, r);
      if (i >= 0) found = x - lane + i;
    }
    if (lane == 0) a.next[b] = found;
    return;
  }
}

template <typename T, int N> cudaError_t launch(VerifyArgs& a, int slots, cudaStream_t st) {
  // As many blocks to a slot as fill the GPU, each with 4096 entries or more, and few enough steps to a warp.
  int cl = 1;
  while (cl < kMaxCluster && ((long long)slots * cl < 304 || a.d.vocab > cl * NW * STEP * kMaxSteps) && a.d.vocab > cl * 4096) cl *= 2;
  a.slots_cl = cl;
  a.tile = (a.d.vocab + cl * NW * STEP - 1) / (cl * NW * STEP) * STEP;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(slots * cl));
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cl;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, draft_verify_kernel<T, N>, (const VerifyArgs)a);
}

bool aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace pathattn

using namespace pathattn;

extern "C" __attribute__((visibility("default"))) int path_draft_verify(const path_verify_desc_t* desc, const int* q_start,
                                                                         const int* tokens, const float* uniform,
                                                                         const void* target, const void* draft, int* keep,
                                                                         int* next, int* status, void* stream) {
  if (!desc || desc->slots <= 0 || desc->total_tokens < 0 || desc->max_new < 0 || desc->vocab <= 0) return PATH_ERR_INVALID_ARG;
  if (desc->dtype != PATH_BF16 && desc->dtype != PATH_FP32) return PATH_ERR_INVALID_ARG;
  if (desc->target_stride < desc->vocab || (draft && desc->draft_stride < desc->vocab)) return PATH_ERR_INVALID_ARG;
  if (desc->slots > 65535 || desc->vocab > (1 << 20)) return PATH_ERR_UNSUPPORTED;
  const int e = desc->dtype == PATH_BF16 ? 2 : 4;
  if (!aligned(q_start, 4) || !aligned(keep, 4) || !aligned(next, 4) || !aligned(status, 4)) return PATH_ERR_INVALID_ARG;
  if (desc->total_tokens > 0 && (!aligned(tokens, 4) || !aligned(uniform, 4) || !aligned(target, e) || (draft && !aligned(draft, e))))
    return PATH_ERR_INVALID_ARG;
  VerifyArgs a{};
  a.d = *desc;
  a.q_start = q_start;
  a.tokens = tokens;
  a.uniform = uniform;
  a.target = target;
  a.draft = draft;
  a.keep = keep;
  a.next = next;
  a.status = status;
  // 16-byte loads where every row begins on 16 bytes and is a whole number of them, else entry by entry
  const int per = 16 / e;
  const bool wide = aligned(target, 16) && desc->target_stride % per == 0 && desc->vocab % per == 0 &&
                    (!draft || (aligned(draft, 16) && desc->draft_stride % per == 0));
  cudaError_t r;
  if (desc->dtype == PATH_BF16)
    r = wide ? launch<__nv_bfloat16, 8>(a, desc->slots, (cudaStream_t)stream) : launch<__nv_bfloat16, 1>(a, desc->slots, (cudaStream_t)stream);
  else
    r = wide ? launch<float, 4>(a, desc->slots, (cudaStream_t)stream) : launch<float, 1>(a, desc->slots, (cudaStream_t)stream);
  return r == cudaSuccess ? PATH_OK : PATH_ERR_CUDA;
}
