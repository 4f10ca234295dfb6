// Verification of drafted tokens against a target model's probabilities (path_draft_verify): acceptance of the drafts of a slot
// and the draw of the token after them, one cluster of blocks per slot.
//
// Every block of the cluster finds the first draft not kept (a few loads), takes a slice of the one row (target) or two
// (target, draft) that decide the next token, and sums r = max(0, p - q) over it; the slices' sums go round through
// distributed shared memory, and the block in whose slice the running sum passes uniform * total finds the entry.
// Sums: the result is an index, so sums that are only nearly right give wrong answers: the running sum passes its goal at
// another entry with probability (entries) * (error).  double sums would be exact enough and cost 13 us of the GPU's few FP64
// units for 64 rows of 131072; a lane instead adds pairs of floats (p - q and the sum with their rounding errors, exactly),
// about 2^-44 of the sum, and only lanes' totals become doubles.
#include <cooperative_groups.h>

#include "dev_common.cuh"
#include "paged.h"

namespace cg = cooperative_groups;

namespace pathattn {
namespace {

constexpr int NT = 256, NW = NT / 32;
constexpr int STEP = 512;        // entries whose sum a warp keeps apart
constexpr int kMaxSteps = 32;    // steps of a warp: one lane each in the search
constexpr int kMaxCluster = 8;

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

// Residual max(0, p - q) as an exact pair (hi, lo).
__device__ __forceinline__ float2 residual(float p, float q) {
  if (!(p > q)) return make_float2(0.f, 0.f);
  const float s = p - q;
  return make_float2(s, (p - s) - q);  // exact: p >= q >= 0
}
// sum (hi, lo) += r: the rounding of hi + r.x is found exactly and kept in lo.
__device__ __forceinline__ void add_pair(float2& sum, float2 r) {
  const float t = sum.x + r.x, b = t - sum.x;
  sum.y += ((sum.x - (t - b)) + (r.x - b)) + r.y;
  sum.x = t;
}
__device__ __forceinline__ double warp_scan(double x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double a = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += a;
  }
  return x;
}
// The first lane whose running sum passes goal, or (rounding) the last with a positive part; -1: none is.
__device__ __forceinline__ int first_past(double upto, double part, double goal) {
  const unsigned past = __ballot_sync(0xffffffffu, upto > goal && part > 0.0), some = __ballot_sync(0xffffffffu, part > 0.0);
  return past ? __ffs(past) - 1 : some ? 31 - __clz(some) : -1;
}

template <typename T, int N>
__global__ void __launch_bounds__(NT, 4) draft_verify_kernel(const VerifyArgs a) {
  chain();
  constexpr int LOADS = STEP / (32 * N);
  constexpr int PER = kMaxCluster * NW / 32;  // warps' sums of the cluster to a lane
  __shared__ double warp_sum[NW];
  __shared__ int first_bad;
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
  const T* target = (const T*)a.target;
  const T* draft = (const T*)a.draft;
  const double u = a.uniform[q0];
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
  float pv[LOADS][N], qv[LOADS][N];
  auto load = [&](int at0) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int at = at0 + (j * 32 + lane) * N;
      load_n<T, N>(p + at, vocab - at, pv[j]);
      if (q) load_n<T, N>(q + at, vocab - at, qv[j]);
    }
  };
  auto entry = [&](int at0, int j, int i) {
    return residual(at0 + (j * 32 + lane) * N + i == out ? 0.f : pv[j][i], q ? qv[j][i] : 0.f);
  };
  for (int round = 0; round < 2; ++round) {
    double mine = 0;  // of step `lane`
    for (int s = 0; s < steps; ++s) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {  // (in halves: registers for four blocks to an SM, which keep more loads on their way)
        constexpr int H = LOADS / 2;
        float ph[H][N], qh[H][N];
        const int at0 = v0 + s * STEP + half * (STEP / 2) + lane * N;
#pragma unroll
        for (int j = 0; j < H; ++j) {
          load_n<T, N>(p + at0 + j * 32 * N, vocab - at0 - j * 32 * N, ph[j]);
          if (q) load_n<T, N>(q + at0 + j * 32 * N, vocab - at0 - j * 32 * N, qh[j]);
        }
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) add_pair(sum, residual(at0 + j * 32 * N + i == out ? 0.f : ph[j][i], q ? qh[j][i] : 0.f));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        add_pair(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, o), __shfl_xor_sync(0xffffffffu, sum.y, o)));
      if (lane == s) mine = (double)sum.x + (double)sum.y;
    }
    const double upto = warp_scan(mine);
    if (lane == 31) warp_sum[warp] = upto;
    cluster.sync();
    // every warp finds the cluster's sum, and whether the goal lies in its own share
    double part[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int w = lane * PER + i;
      part[i] = w < a.slots_cl * NW ? *cluster.map_shared_rank(&warp_sum[w % NW], w / NW) : 0.0;
    }
    cluster.sync();  // no block leaves, or sums again, while others read its sums
    double lane_sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) lane_sum += part[i];
    const double lane_upto = warp_scan(lane_sum);
    const double all = __shfl_sync(0xffffffffu, lane_upto, 31);
    if (!(all > 0.0) && round == 0 && (q || out >= 0)) {
      q = nullptr;  // nothing is left of the target: its own row
      out = -1;
      continue;
    }
    const double goal = u * all;
    const int l = first_past(lane_upto, lane_sum, goal);
    if (l < 0) {
      if (rank == 0 && tid == 0) a.next[b] = -1;
      return;
    }
    const double before_lane = lane_upto - lane_sum;
    // the first part at which the running sum passes
    double run = before_lane, at_owner = before_lane;
    bool there = false;
    int owner = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!there && part[i] > 0.0) {
        owner = i;
        at_owner = run;
        there = run + part[i] > goal;
      }
      run += part[i];
    }
    owner = __shfl_sync(0xffffffffu, lane * PER + owner, l);
    double before = __shfl_sync(0xffffffffu, at_owner, l);
    if (owner != rank * NW + warp) return;
    const int s = first_past(before + upto, mine, goal);
    if (s < 0) {  // (an infinity in the row)
      if (lane == 0) a.next[b] = -1;
      return;
    }
    const double prev = __shfl_sync(0xffffffffu, upto, s > 0 ? s - 1 : 0);
    if (s > 0) before += prev;
    // the step's entries again, exactly
    load(v0 + s * STEP);
    double sum_j[LOADS], upto_j[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) add_pair(sum, entry(v0 + s * STEP, j, i));
      upto_j[j] = sum_j[j] = (double)sum.x + (double)sum.y;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const double x = __shfl_up_sync(0xffffffffu, upto_j[j], o);
        if (lane >= o) upto_j[j] += x;
      }
    int found = -1;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const unsigned past = __ballot_sync(0xffffffffu, before + upto_j[j] > goal && sum_j[j] > 0.0);
      const unsigned some = __ballot_sync(0xffffffffu, sum_j[j] > 0.0);
      if (some) {
        const int w = past ? __ffs(past) - 1 : 31 - __clz(some);  // (in case rounding lets none pass: the last)
        double at = before + (upto_j[j] - sum_j[j]);
        int x = -1;
        bool passed = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 r = entry(v0 + s * STEP, j, i);
          at += (double)r.x + (double)r.y;
          if (r.x > 0.f && !passed) {
            x = v0 + s * STEP + (j * 32 + lane) * N + i;
            passed = at > goal;
          }
        }
        found = __shfl_sync(0xffffffffu, x, w);
        if (past) break;
      }
      before += __shfl_sync(0xffffffffu, upto_j[j], 31);
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
