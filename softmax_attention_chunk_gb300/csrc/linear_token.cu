// Linear attention of single and draft tokens: the recurrence itself, S <- g S + k v^T, o = scale S^T q, token by token, with
// the state of a slot and key head in one block's registers (float32, read and written once per call).
// Bound: the state's bytes, 8 D^2 per slot and key head (4 D^2 where it is not written back).
#include "dev_common.cuh"
#include "linear.h"
#include "tc_common.cuh"

namespace pathattn {
namespace {

using namespace tc;

constexpr int NT = 256, W = NT / 32;
constexpr int OB = 8;  // rows of o (token, query head) whose sums the warps join at once

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

// A block holds V columns of a state.
template <typename T, int D, int V>
__global__ void __launch_bounds__(NT) linear_token_kernel(const LinArgs p) {
  chain();
  if (p.max_new > kLinTokenMax && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.err = 0;  // (of the kernels that follow)
  constexpr int CG = V / 4;      // lanes of a row, four columns each
  constexpr int RG = NT / CG;    // row groups
  constexpr int RP = D / RG;     // rows of a thread, one behind the other
  extern __shared__ uint8_t smem_raw[];
  T* tok = reinterpret_cast<T*>(smem_raw);  // per token: k, v, q of the group
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = tid % CG * 4, r0 = tid / CG * RP;
  const int h = blockIdx.x / (D / V), v0 = blockIdx.x % (D / V) * V, b = blockIdx.y, G = p.G;
  const LinSpan sp = lin_span(p.q_start, b, p.total, p.max_new);
  if (sp.code && blockIdx.x == 0 && tid == 0) paged_error(p.status, sp.code);
  const int n = sp.n;
  if (n == 0 || n > kLinTokenMax) return;
  float* own = p.state + (((size_t)b * p.heads + h) * D + r0) * D + v0 + c;
  ulonglong2 s[RP];  // pairs of floats
#pragma unroll
  for (int i = 0; i < RP; ++i) s[i] = *reinterpret_cast<const ulonglong2*>(own + i * D);
  const LinOp& op = p.op[0];
  const int per = (2 + G) * D;
  float* red = reinterpret_cast<float*>(tok + min(p.max_new, kLinTokenMax) * per);  // [2][OB][W][V]: the warps' sums
  for (int e = tid * 4; e < n * per; e += NT * 4) {
    const int t = e / per, x = e % per / D, col = e % D;
    const long long at = sp.q0 + t;
    const T* src = x == 0 ? (const T*)op.y + at * op.yt + h * op.yh
                 : x == 1 ? (const T*)op.z + at * op.yt + h * op.yh
                          : (const T*)op.x + at * op.xt + (long long)(h * G + x - 2) * op.xh;
    if (sizeof(T) == 4) *reinterpret_cast<float4*>(tok + e) = *reinterpret_cast<const float4*>(src + col);
    else *reinterpret_cast<uint2*>(tok + e) = *reinterpret_cast<const uint2*>(src + col);
  }
  const float g1 = exp2f(lin_log2(p.log_decay[h]));
  const uint64_t keep = f2(g1, g1);
  __syncthreads();
  T* o = (T*)op.o + (long long)sp.q0 * op.xt + (long long)h * G * op.xh + v0;
  const T* at = tok;
  int g = 0, t0 = 0, g0 = 0, buf = 0;  // head; token and head of the first row not joined yet
  const int rows = n * G;
  for (int i = 0; i < rows; ++i) {
    if (g == 0) {
      float v[4];
      load4s<T>(at + D + v0 + c, v);
      const uint64_t v0 = f2(v[0], v[1]), v1 = f2(v[2], v[3]);
#pragma unroll
      for (int j = 0; j < RP; j += 4) {
        float k[4];
        load4s<T>(at + r0 + j, k);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint64_t kk = f2(k[x], k[x]);
          s[j + x].x = f2_fma(s[j + x].x, keep, f2_mul(kk, v0));
          s[j + x].y = f2_fma(s[j + x].y, keep, f2_mul(kk, v1));
        }
      }
    }
    uint64_t o0 = 0, o1 = 0;
#pragma unroll
    for (int j = 0; j < RP; j += 4) {
      float q[4];
      load4s<T>(at + (2 + g) * D + r0 + j, q);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint64_t qq = f2(q[x], q[x]);
        o0 = f2_fma(s[j + x].x, qq, o0);
        o1 = f2_fma(s[j + x].y, qq, o1);
      }
    }
    float a[4];
    f2_split(o0, a[0], a[1]);
    f2_split(o1, a[2], a[3]);
    if (CG < 32)  // two row groups to a warp
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] += __shfl_xor_sync(0xffffffffu, a[j], 16);
    if (CG == 32 || lane < CG)
      *reinterpret_cast<float4*>(red + ((buf * OB + i % OB) * W + warp) * V + c) = make_float4(a[0], a[1], a[2], a[3]);
    if (++g == G) g = 0, at += per;
    const int done = i % OB + 1;
    if (done == OB || i + 1 == rows) {
      __syncthreads();  // (the other half of red was read before the block came here)
      for (int e = tid; e < done * V; e += NT) {
        const int row = g0 + e / V, col = e % V;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += red[((buf * OB + e / V) * W + w) * V + col];
        o[(t0 + row / G) * op.xt + (long long)(row % G) * op.xh + col] = from_f<T>(sum * p.scale);
      }
      buf ^= 1;
      t0 += (g0 + done) / G;
      g0 = (g0 + done) % G;
    }
  }
  if (p.update)
#pragma unroll
    for (int i = 0; i < RP; ++i) *reinterpret_cast<ulonglong2*>(own + i * D) = s[i];
}

template <typename T, int D, int V> cudaError_t launch(const LinArgs& p, cudaStream_t st) {
  const int most = p.max_new < kLinTokenMax ? p.max_new : kLinTokenMax, rows = most * p.G;
  const size_t smem = sizeof(T) * most * (2 + p.G) * D + sizeof(float) * W * V * (rows > OB ? 2 * OB : rows);
  if (smem > 48 << 10) {
    cudaError_t e = cudaFuncSetAttribute(linear_token_kernel<T, D, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_chained(linear_token_kernel<T, D, V>, dim3(p.heads * (D / V), p.seqs), NT, smem, st, p);
}
// Single tokens are bound by the states' bytes, whole rows to a block; with several tokens a block works between its loads, and
// half a state's columns make room for twice the blocks (48 slots x 8 heads of dim 128 with 2 .. 9 tokens: YY us in place of 16.7).
template <typename T> cudaError_t launch(const LinArgs& p, cudaStream_t st) {
  if (p.D == 64) return launch<T, 64, 64>(p, st);
  return p.max_new > 1 ? launch<T, 128, 64>(p, st) : launch<T, 128, 128>(p, st);
}

}  // namespace

cudaError_t launch_linear_token(const LinArgs& p, bool bf16, cudaStream_t st) {
  return bf16 ? launch<__nv_bfloat16>(p, st) : launch<float>(p, st);
}

}  // namespace pathattn
