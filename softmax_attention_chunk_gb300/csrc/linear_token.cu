// Linear attention of single and draft tokens: the recurrence itself, S <- g S + k v^T, o = scale S^T q, token by token, with
// the state of a slot and key head in one block's registers (float32, read and written once per call).
// Bound: the state's bytes, 8 D^2 per slot and key head (4 D^2 where it is not written back).
#include "dev_common.cuh"
#include "linear.h"

namespace pathattn {
namespace {

constexpr int NT = 256;
constexpr int GB = 4;  // query heads whose sums are joined at once

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

template <typename T, int D>
__global__ void __launch_bounds__(NT) linear_token_kernel(const LinArgs p) {
  chain();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.err = 0;
  constexpr int CG = D / 4;      // lanes of a row, four columns each
  constexpr int RG = NT / CG;    // row groups
  constexpr int RP = D / RG;     // rows of a thread, one behind the other
  constexpr int W = NT / 32;
  extern __shared__ uint8_t smem_raw[];
  float (*red)[GB][W][D] = reinterpret_cast<float (*)[GB][W][D]>(smem_raw);  // [2]: the warps' sums
  T* tok = reinterpret_cast<T*>(smem_raw + sizeof(float) * 2 * GB * W * D);  // per token: k, v, q of the group
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = tid % CG * 4, r0 = tid / CG * RP;
  const int h = blockIdx.x, b = blockIdx.y, G = p.G;
  const LinSpan sp = lin_span(p.q_start, b, p.total, p.max_new);
  if (sp.code && h == 0 && tid == 0) paged_error(p.status, sp.code);
  const int n = sp.n;
  if (n == 0 || n > kLinTokenMax) return;
  float* own = p.state + (((size_t)b * p.heads + h) * D + r0) * D + c;
  float4 s[RP];
#pragma unroll
  for (int i = 0; i < RP; ++i) s[i] = *reinterpret_cast<const float4*>(own + i * D);
  const LinOp& op = p.op[0];
  const int per = (2 + G) * D;
  for (int e = tid * 4; e < n * per; e += NT * 4) {
    const int t = e / per, x = e % per / D, col = e % D;
    const long long at = sp.q0 + t;
    const T* src = x == 0 ? (const T*)op.y + at * op.yt + h * op.yh
                 : x == 1 ? (const T*)op.z + at * op.yt + h * op.yh
                          : (const T*)op.x + at * op.xt + (long long)(h * G + x - 2) * op.xh;
    if (sizeof(T) == 4) *reinterpret_cast<float4*>(tok + e) = *reinterpret_cast<const float4*>(src + col);
    else *reinterpret_cast<uint2*>(tok + e) = *reinterpret_cast<const uint2*>(src + col);
  }
  const float keep = exp2f(lin_log2(p.log_decay[h]));
  __syncthreads();
  int buf = 0;
  for (int t = 0; t < n; ++t) {
    const T* at = tok + t * per;
    float v[4];
    load4s<T>(at + D + c, v);
#pragma unroll
    for (int i = 0; i < RP; i += 4) {
      float k[4];
      load4s<T>(at + r0 + i, k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4& a = s[i + j];
        a.x = a.x * keep + k[j] * v[0], a.y = a.y * keep + k[j] * v[1];
        a.z = a.z * keep + k[j] * v[2], a.w = a.w * keep + k[j] * v[3];
      }
    }
    for (int g0 = 0; g0 < G; g0 += GB, buf ^= 1) {
#pragma unroll
      for (int g = 0; g < GB; ++g) {
        if (g0 + g >= G) break;
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < RP; i += 4) {
          float q[4];
          load4s<T>(at + (2 + g0 + g) * D + r0 + i, q);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4& a = s[i + j];
            o[0] += a.x * q[j], o[1] += a.y * q[j], o[2] += a.z * q[j], o[3] += a.w * q[j];
          }
        }
        if (CG < 32)  // two row groups to a warp
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] += __shfl_xor_sync(0xffffffffu, o[j], 16);
        if (CG == 32 || lane < CG) *reinterpret_cast<float4*>(&red[buf][g][warp][c]) = make_float4(o[0], o[1], o[2], o[3]);
      }
      __syncthreads();  // (the other half of red was read before the block came here)
      for (int e = tid; e < min(GB, G - g0) * D; e += NT) {
        const int g = e / D, col = e % D;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += red[buf][g][w][col];
        ((T*)op.o)[(long long)(sp.q0 + t) * op.xt + (long long)(h * G + g0 + g) * op.xh + col] = from_f<T>(sum * p.scale);
      }
    }
  }
  if (p.update)
#pragma unroll
    for (int i = 0; i < RP; ++i) *reinterpret_cast<float4*>(own + i * D) = s[i];
}

template <typename T, int D> cudaError_t launch(const LinArgs& p, cudaStream_t st) {
  const int most = p.max_new < kLinTokenMax ? p.max_new : kLinTokenMax;
  const size_t smem = sizeof(float) * 2 * GB * (NT / 32) * D + sizeof(T) * most * (2 + p.G) * D;
  cudaError_t e = cudaFuncSetAttribute(linear_token_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_chained(linear_token_kernel<T, D>, dim3(p.heads, p.seqs), NT, smem, st, p);
}

}  // namespace

cudaError_t launch_linear_token(const LinArgs& p, bool bf16, cudaStream_t st) {
  if (bf16) return p.D == 64 ? launch<__nv_bfloat16, 64>(p, st) : launch<__nv_bfloat16, 128>(p, st);
  return p.D == 64 ? launch<float, 64>(p, st) : launch<float, 128>(p, st);
}

}  // namespace pathattn
