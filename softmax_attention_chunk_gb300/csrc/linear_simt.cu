// Linear attention in float32 on CUDA cores: the walk of linear.h in chunks of 32 tokens, one block per key head, segment and 64 columns
// of the state.  Inside a chunk the products x_i . y_j are masked and weighted with g^(i-j); what lies before goes through the
// state at the chunk's start.
#include "linear.h"

namespace pathattn {
namespace {

constexpr int NT = 256, C = 32, V = 64;

template <int D> struct Smem {
  float x[C][D + 4], y[C][D + 4], z[C][V + 4], s[D][V + 4], p[C][C + 1], pw[C + 1];
};

// Rows pos .. pos + m - 1 (walk order) of W columns into shared memory, zeros behind them.
template <int W, int LD>
__device__ __forceinline__ void load_rows(float (&dst)[C][LD], const float* src, long long stride, int pos, int m, int n, bool reverse) {
  for (int e = threadIdx.x; e < C * W / 4; e += NT) {
    const int r = e / (W / 4), c = e % (W / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < m) v = *reinterpret_cast<const float4*>(src + (reverse ? n - 1 - (pos + r) : pos + r) * stride + c);
    *reinterpret_cast<float4*>(&dst[r][c]) = v;
  }
}

template <int D, bool STATES>
__global__ void __launch_bounds__(NT) linear_simt_kernel(const LinArgs p) {
  chain();
  extern __shared__ uint8_t smem_raw[];
  Smem<D>& s = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, r = tid / 16, c4 = tid % 16 * 4;  // owns o rows r, r + 16 and state rows r + 16 k, columns c4 ..
  constexpr int NV = D / V;
  const int h = blockIdx.y / NV, v0 = blockIdx.y % NV * V, item = blockIdx.x;
  const LinOp& op = p.op[blockIdx.z];
  const LinItem it = lin_item(p, item);
  if (it.seg < 0) return;
  const bool rev = op.reverse;
  const float l2 = lin_log2(p.log_decay[h]);
  if (tid <= C) s.pw[tid] = exp2f(l2 * tid);
  float* part = p.parts + (((size_t)blockIdx.z * p.items + item) * p.heads + h) * D * D + v0;
  float* own = p.state ? p.state + ((size_t)it.seq * p.heads + h) * D * D + v0 : nullptr;
  const bool split = p.max_new > p.seg;  // the segments' starting states are in parts
  const float* from = STATES ? nullptr : split ? part : own;
  for (int e = tid; e < D * V; e += NT) s.s[e / V][e % V] = from ? from[(size_t)(e / V) * D + e % V] : 0.f;
  const float* x = (const float*)op.x + it.seq * op.xb + it.q0 * op.xt + (long long)h * op.gx * op.xh;
  float* o = (float*)op.o + it.seq * op.xb + it.q0 * op.xt + (long long)h * op.gx * op.xh + v0;
  const float* y = (const float*)op.y + it.seq * op.yb + it.q0 * op.yt + (long long)h * op.gy * op.yh;
  const float* z = (const float*)op.z + it.seq * op.yb + it.q0 * op.yt + (long long)h * op.gy * op.yh + v0;
  const int end = min(it.n, (it.seg + 1) * p.seg);
  for (int pos = it.seg * p.seg; pos < end; pos += C) {
    const int m = min(C, end - pos);
    float acc[2][4] = {};
    auto inter = [&]() {
#pragma unroll 4
      for (int e = 0; e < D; ++e) {
        const float4 b = *reinterpret_cast<const float4*>(&s.s[e][c4]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = s.x[r + 16 * i][e];
          acc[i][0] += a * b.x, acc[i][1] += a * b.y, acc[i][2] += a * b.z, acc[i][3] += a * b.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] *= s.pw[r + 16 * i + 1];
    };
    auto intra = [&]() {
      float d[2][2] = {};
      const int j0 = tid % 16;
#pragma unroll 4
      for (int e = 0; e < D; e += 4) {
        const float4 x0 = *reinterpret_cast<const float4*>(&s.x[r][e]), x1 = *reinterpret_cast<const float4*>(&s.x[r + 16][e]);
        const float4 y0 = *reinterpret_cast<const float4*>(&s.y[j0][e]), y1 = *reinterpret_cast<const float4*>(&s.y[j0 + 16][e]);
        d[0][0] += x0.x * y0.x + x0.y * y0.y + x0.z * y0.z + x0.w * y0.w;
        d[0][1] += x0.x * y1.x + x0.y * y1.y + x0.z * y1.z + x0.w * y1.w;
        d[1][0] += x1.x * y0.x + x1.y * y0.y + x1.z * y0.z + x1.w * y0.w;
        d[1][1] += x1.x * y1.x + x1.y * y1.y + x1.z * y1.z + x1.w * y1.w;
      }
      __syncthreads();  // the previous products' p has been read
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int gap = r + 16 * i - (j0 + 16 * j);
          s.p[r + 16 * i][j0 + 16 * j] = gap >= 0 ? d[i][j] * s.pw[gap] : 0.f;
        }
      __syncthreads();
#pragma unroll 4
      for (int j = 0; j < C; ++j) {
        const float4 b = *reinterpret_cast<const float4*>(&s.z[j][c4]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = s.p[r + 16 * i][j];
          acc[i][0] += a * b.x, acc[i][1] += a * b.y, acc[i][2] += a * b.z, acc[i][3] += a * b.w;
        }
      }
    };
    auto store = [&](int g) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (r + 16 * i >= m) continue;
        float* to = o + (long long)g * op.xh + (rev ? it.n - 1 - (pos + r + 16 * i) : pos + r + 16 * i) * op.xt + c4;
        *reinterpret_cast<float4*>(to) = make_float4(acc[i][0] * p.scale, acc[i][1] * p.scale, acc[i][2] * p.scale, acc[i][3] * p.scale);
      }
    };
    if (!STATES && op.gy > 1) {  // one x, its products with all heads of y
      __syncthreads();
      load_rows<D>(s.x, x, op.xt, pos, m, it.n, rev);
      __syncthreads();
      inter();
    }
    for (int g = 0; g < op.gy; ++g) {
      __syncthreads();  // y, z of the round before have been read
      load_rows<D>(s.y, y + (long long)g * op.yh, op.yt, pos, m, it.n, rev);
      load_rows<V>(s.z, z + (long long)g * op.yh, op.yt, pos, m, it.n, rev);
      __syncthreads();
      if (!STATES) {
        if (op.gy > 1) {
          intra();
        } else {
          for (int k = 0; k < op.gx; ++k) {
            __syncthreads();
            load_rows<D>(s.x, x + (long long)k * op.xh, op.xt, pos, m, it.n, rev);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i)
              for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
            inter();
            intra();
            store(k);
          }
        }
        __syncthreads();  // the state has been read
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        float a[4];
        const float keep = g == 0 ? s.pw[m] : 1.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = s.s[r + 16 * k][c4 + j] * keep;
        for (int j = 0; j < m; ++j) {
          const float w = s.y[j][r + 16 * k] * s.pw[m - 1 - j];
          const float4 b = *reinterpret_cast<const float4*>(&s.z[j][c4]);
          a[0] += w * b.x, a[1] += w * b.y, a[2] += w * b.z, a[3] += w * b.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s.s[r + 16 * k][c4 + j] = a[j];
      }
    }
    if (!STATES && op.gy > 1) store(0);
  }
  __syncthreads();
  float* to = STATES ? part : !split && p.update ? own : nullptr;
  if (to)
    for (int e = tid; e < D * V; e += NT) to[(size_t)(e / V) * D + e % V] = s.s[e / V][e % V];
}

template <int D, bool STATES> cudaError_t launch(const LinArgs& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(linear_simt_kernel<D, STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  return launch_chained(linear_simt_kernel<D, STATES>, dim3(p.items, p.heads * (D / V), p.ops), NT, sizeof(Smem<D>), st, p);
}

}  // namespace

cudaError_t launch_linear_simt(const LinArgs& p, bool states, cudaStream_t st) {
  if (p.D == 64) return states ? launch<64, true>(p, st) : launch<64, false>(p, st);
  return states ? launch<128, true>(p, st) : launch<128, false>(p, st);
}

}  // namespace pathattn
