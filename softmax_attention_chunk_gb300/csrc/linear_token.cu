// Linear attention of single and draft tokens: the recurrence itself, S <- g S + k v^T, o = scale S^T q, token by token, with
// the state of a slot and key head in one block's registers (float32, read and written once per call).
// Bound: the state's bytes, 8 D^2 per slot and key head (4 D^2 where it is not written back); with several tokens the paired
// multiply-adds (for a row of four columns four to take a token in, two for each query head), which shared memory feeds with k
// and q in float32, each number twice.
#include "dev_common.cuh"
#include "linear.h"
#include "tc_common.cuh"

namespace pathattn {
namespace {

using namespace tc;

constexpr int NT = 256, W = NT / 32;
constexpr int kTokenBytes = 48 << 10;  // tokens in shared memory at once

template <typename T> __device__ __forceinline__ void load4s(const T* a, float (&v)[4]);
template <> __device__ __forceinline__ void load4s<float>(const float* a, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(a);
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
template <> __device__ __forceinline__ void load4s<__nv_bfloat16>(const __nv_bfloat16* a, float (&v)[4]) {
  const uint2 x = *reinterpret_cast<const uint2*>(a);
  v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
}

template <typename T> __device__ __forceinline__ void store4(T* a, const float (&v)[4], float scale);
template <> __device__ __forceinline__ void store4<float>(float* a, const float (&v)[4], float scale) {
  *reinterpret_cast<float4*>(a) = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* a, const float (&v)[4], float scale) {
  *reinterpret_cast<uint2*>(a) = make_uint2(pack_bf16(v[0] * scale, v[1] * scale), pack_bf16(v[2] * scale, v[3] * scale));
}

// Rows of o (token, query head) whose sums the warps join at once; floats of a token in shared memory: k twice, v, q twice;
// tokens there at once.
constexpr int kJoin = 8;
PATH_HD int token_floats(int D, int G) { return (3 + 2 * G) * D; }
PATH_HD int token_batch(int D, int G) { return kTokenBytes / (4 * token_floats(D, G)); }

// Of many slots: whether there is a bad row among all.  (Every block reading all rows before its own: 60000 slots of one head 582 us a
// call, with this pass 341.)
__global__ void __launch_bounds__(NT) linear_rows_kernel(const LinArgs p) {
  chain();
  const int b = blockIdx.x * NT + threadIdx.x;
  if (b >= p.seqs) return;
  const LinSpan s = lin_span(p.q_start, b, p.total, p.max_new);
  if (s.code) paged_error(p.status, s.code);
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, D == 64 ? 4 : 2) linear_token_kernel(const LinArgs p) {
  chain();
  if (p.max_new > kLinTokenMax && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.err = 0;  // (of the kernels that follow)
  constexpr int CG = D / 4;      // lanes of a row, four columns each
  constexpr int RG = NT / CG;    // row groups
  constexpr int RP = D / RG;     // rows of a thread, one behind the other
  constexpr int OB = kJoin;
  extern __shared__ __align__(16) float smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = tid % CG * 4, r0 = tid / CG * RP;
  const int h = blockIdx.x, b = blockIdx.y, G = p.G;
  // Whether the slot may begin before an earlier one's tokens end: only where a row before it ends above its start (a thread each) or,
  // with more slots than threads, where a row is bad, for which linear_rows_kernel has looked at all.  Asked for beside the slot's own
  // row and compared with it: waited for later, or earlier than the state's loads, 4096 slots of 4 heads at d 64 take 110 and 97 us, 95 so.
  const bool here = p.q_start && p.seqs <= NT;
  const int above = here ? p.q_start[min(tid + 1, b)] : tid == 0 ? __ldcg(p.status) : 0;
  const LinSpan sp = lin_span(p.q_start, b, p.total, p.max_new);
  const bool may = here ? above > sp.q0 : p.q_start && above != 0;
  if (sp.code && h == 0 && tid == 0) paged_error(p.status, sp.code);
  const int n = sp.n;
  if (n == 0 || (n > kLinTokenMax && h > 0)) return;
  auto late = [&]() {  // met by the whole block
    if (!__syncthreads_or(may)) return false;
    bool is = false;
    for (int i = tid; i < b; i += NT) {
      const LinSpan e = lin_span(p.q_start, i, p.total, p.max_new);
      is |= e.n > 0 && e.q0 + e.n > sp.q0;
    }
    is = __syncthreads_or(is);
    if (is && h == 0 && tid == 0) paged_error(p.status, PATH_PAGED_BAD_START);
    return is;
  };
  if (n > kLinTokenMax) {  // (reported here, left out by the kernels that follow)
    late();
    return;
  }
  float* own = p.state + (((size_t)b * p.heads + h) * D + r0) * D + c;
  ulonglong2 s[RP];  // pairs of floats
#pragma unroll
  for (int i = 0; i < RP; ++i) s[i] = *reinterpret_cast<const ulonglong2*>(own + i * D);
  const LinOp& op = p.op[0];
  const int per = token_floats(D, G), batch = min(token_batch(D, G), min(p.max_new, kLinTokenMax));
  float* red = smem + batch * per;  // [2][OB][W][D]: the warps' sums
  const float2 g1 = lin_decay(p.log_decay[h], 1);
  // The rest of every token's decay goes to the state at the first one: it is what would add up from call to call.  Inside the call
  // a weight is then off by 15 * 2^-25 at most (at every token: 48 slots of 2..9 drafts 16.8 us in place of 15.3).
  const uint64_t keep = f2(g1.x, g1.x), rest = f2(g1.y * n, g1.y * n);
  int buf = 0;
  for (int t0 = 0; t0 < n; t0 += batch) {
    const int m = min(batch, n - t0);
    __syncthreads();  // the batch before has been read
    // a row (k, v or a head's q of a token) to D / 4 threads
    for (int t = 0, x = tid / CG;; x += RG) {
      while (x >= 2 + G) x -= 2 + G, ++t;
      if (t >= m) break;
      const long long at = sp.q0 + t0 + t;
      float a[4];
      load4s<T>(x == 0 ? (const T*)op.y + at * op.yt + h * op.yh + c
                : x == 1 ? (const T*)op.z + at * op.yt + h * op.yh + c
                         : (const T*)op.x + at * op.xt + (long long)(h * G + x - 2) * op.xh + c,
                a);
      float* to = smem + t * per + (x == 0 ? 2 * c : x == 1 ? 2 * D + c : (2 * x - 1) * D + 2 * c);
      if (x == 1) {
        *reinterpret_cast<float4*>(to) = make_float4(a[0], a[1], a[2], a[3]);
      } else {
        reinterpret_cast<float4*>(to)[0] = make_float4(a[0], a[0], a[1], a[1]);
        reinterpret_cast<float4*>(to)[1] = make_float4(a[2], a[2], a[3], a[3]);
      }
    }
    if (late()) return;  // (at the barrier that the tokens need anyway: one of its own took 64 slots 47 us in place of 43)
    T* o = (T*)op.o + (long long)(sp.q0 + t0) * op.xt + (long long)h * G * op.xh;
    const float* at = smem;
    int g = 0;  // head
    const int rows = m * G;
    for (int i = 0; i < rows; ++i) {
      if (g == 0) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(at + 2 * D + c);
        auto take = [&](auto more) {
#pragma unroll
          for (int j = 0; j < RP; j += 2) {
            const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(at + 2 * (r0 + j));
            s[j].x = f2_fma(s[j].x, keep, more(s[j].x, f2_mul(k.x, v.x)));
            s[j].y = f2_fma(s[j].y, keep, more(s[j].y, f2_mul(k.x, v.y)));
            s[j + 1].x = f2_fma(s[j + 1].x, keep, more(s[j + 1].x, f2_mul(k.y, v.x)));
            s[j + 1].y = f2_fma(s[j + 1].y, keep, more(s[j + 1].y, f2_mul(k.y, v.y)));
          }
        };
        if (t0 + i == 0) take([&](uint64_t old, uint64_t kv) { return f2_fma(old, rest, kv); });
        else take([](uint64_t, uint64_t kv) { return kv; });
      }
      uint64_t o0 = 0, o1 = 0;
      const float* q = at + (3 + 2 * g) * D + 2 * r0;
#pragma unroll
      for (int j = 0; j < RP; j += 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(q + 2 * j);
        o0 = f2_fma(s[j].x, x.x, o0);
        o1 = f2_fma(s[j].y, x.x, o1);
        o0 = f2_fma(s[j + 1].x, x.y, o0);
        o1 = f2_fma(s[j + 1].y, x.y, o1);
      }
      float a[4];
      f2_split(o0, a[0], a[1]);
      f2_split(o1, a[2], a[3]);
      if (CG < 32)  // two row groups to a warp
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] += __shfl_xor_sync(0xffffffffu, a[j], 16);
      if (CG == 32 || lane < CG)
        *reinterpret_cast<float4*>(red + ((buf * OB + i % OB) * W + warp) * D + c) = make_float4(a[0], a[1], a[2], a[3]);
      if (++g == G) g = 0, at += per;
      const int done = i % OB + 1;
      if (done == OB || i + 1 == rows) {
        __syncthreads();  // (the other half of red was read before the block came here)
        const int j = tid / CG;
        if (j < done) {
          const float* from = red + ((buf * OB + j) * W) * D + c;
          float sum[4] = {};
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(from + w * D);
            sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
          }
          const unsigned row = i + 1 - done + j, t = row / (unsigned)G, gr = row % (unsigned)G;
          store4<T>(o + t * op.xt + gr * op.xh + c, sum, p.scale);
        }
        buf ^= 1;
      }
    }
  }
  if (p.update)
#pragma unroll
    for (int i = 0; i < RP; ++i) *reinterpret_cast<ulonglong2*>(own + i * D) = s[i];
}

template <typename T, int D> cudaError_t launch(const LinArgs& p, cudaStream_t st) {
  const int most = p.max_new < kLinTokenMax ? p.max_new : kLinTokenMax, fits = token_batch(D, p.G), batch = most < fits ? most : fits;
  const int rows = most * p.G <= kJoin ? most * p.G : 2 * kJoin;
  const size_t smem = sizeof(float) * (batch * token_floats(D, p.G) + W * D * rows);
  if (smem > 48 << 10) {
    cudaError_t e = cudaFuncSetAttribute(linear_token_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  if (p.q_start && p.seqs > NT) {
    cudaError_t e = launch_chained(linear_rows_kernel, (unsigned)((p.seqs + NT - 1) / NT), NT, 0, st, p);
    if (e != cudaSuccess) return e;
  }
  return launch_chained(linear_token_kernel<T, D>, dim3(p.heads, p.seqs), NT, smem, st, p);
}

}  // namespace

cudaError_t launch_linear_token(const LinArgs& p, bool bf16, cudaStream_t st) {
  if (bf16) return p.D == 64 ? launch<__nv_bfloat16, 64>(p, st) : launch<__nv_bfloat16, 128>(p, st);
  return p.D == 64 ? launch<float, 64>(p, st) : launch<float, 128>(p, st);
}

}  // namespace pathattn
