// Linear attention in float32 on CUDA cores: the walk of linear.h in chunks of 64 tokens, one block per key head, segment and
// 64 columns of the state.  Inside a chunk the products x_i . y_j are masked and weighted with g^(i-j); what lies before goes
// through the state at the chunk's start.
// Bound: FP32 multiply-adds and the shared-memory reads that feed them; a thread holds 4 x 4 of every product, so a 16-byte
// read feeds 8 of them.
#include "linear.h"
#include "tc_common.cuh"

namespace pathattn {
namespace {

using namespace tc;

constexpr int NT = 256, C = kLinChunkF32, V = 64;

template <int D> struct Smem {
  float x[C][D + 4], y[C][D + 4], z[C][V + 4], s[D][V + 4], p[C][C + 4], pw[C + 1];
};

// Rows pos .. pos + m - 1 (walk order) of W columns into shared memory, zeros behind them.
template <int W, int LD>
__device__ __forceinline__ void load_rows(float (&dst)[C][LD], const float* src, long long stride, int pos, int m, int n, bool reverse) {
#pragma unroll
  for (int i = 0; i < C * W / 4 / NT; ++i) {
    const int e = threadIdx.x + i * NT, r = e / (W / 4), c = e % (W / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < m) v = *reinterpret_cast<const float4*>(src + (reverse ? n - 1 - (pos + r) : pos + r) * stride + c);
    *reinterpret_cast<float4*>(&dst[r][c]) = v;
  }
}
__device__ __forceinline__ void get4(const float* a, float (&v)[4]) {
  const float4 x = *reinterpret_cast<const float4*>(a);
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
// acc[4][4] += rows r0 .. r0 + 3 of a (K columns) times rows 0 .. K - 1 of b, columns c0 .. c0 + 3.
template <int K, int LA, int LB>
__device__ __forceinline__ void product(float (&acc)[4][4], const float (&a)[C][LA], const float (*b)[LB], int r0, int c0) {
#pragma unroll 4
  for (int e = 0; e < K; e += 4) {
    float x[4][4], y[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) get4(&a[r0 + i][e], x[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) get4(&b[e + i][c0], y[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += x[i][k] * y[k][j];
  }
}

template <int D, bool STATES>
__global__ void __launch_bounds__(NT) linear_simt_kernel(const LinArgs p) {
  chain();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D>& s = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, r0 = tid / 16 * 4, j0 = tid % 16, c0 = j0 * 4;  // owns o rows r0 .. r0 + 3, columns c0 .. c0 + 3
  constexpr int NV = D / V;
  const int h = blockIdx.y / NV, v0 = blockIdx.y % NV * V, item = blockIdx.x;
  const LinOp& op = p.op[STATES ? p.maker[blockIdx.z] : blockIdx.z];
  const LinItem it = lin_item(p, item);
  if (it.seg < 0) return;
  const bool rev = op.reverse;
  const float l2 = lin_log2(p.log_decay[h]);
  if (tid <= C) s.pw[tid] = exp2f(l2 * tid);
  const float2 whole = lin_decay(p.log_decay[h], C);
  float* part = p.parts + (((size_t)op.slot * p.items + item) * p.heads + h) * D * D;
  float* own = p.state ? p.state + ((size_t)it.seq * p.heads + h) * D * D : nullptr;
  const bool split = p.max_new > p.seg;  // the segments' starting states are in parts
  const float* from = STATES ? nullptr : split ? part : own;
  if (from && op.turned)
    for (int e = tid; e < D * V; e += NT) s.s[e % D][e / D] = from[(size_t)(v0 + e / D) * D + e % D];
  else
    for (int e = tid * 4; e < D * V; e += NT * 4)
      *reinterpret_cast<float4*>(&s.s[e / V][e % V]) =
          from ? *reinterpret_cast<const float4*>(from + (size_t)(e / V) * D + v0 + e % V) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float* x = (const float*)op.x + it.seq * op.xb + it.q0 * op.xt + (long long)h * op.gx * op.xh;
  float* o = (float*)op.o + it.seq * op.xb + it.q0 * op.xt + (long long)h * op.gx * op.xh + v0;
  const float* y = (const float*)op.y + it.seq * op.yb + it.q0 * op.yt + (long long)h * op.gy * op.yh;
  const float* z = (const float*)op.z + it.seq * op.yb + it.q0 * op.yt + (long long)h * op.gy * op.yh + v0;
  const int end = min(it.n, (it.seg + 1) * p.seg);
  for (int pos = it.seg * p.seg; pos < end; pos += C) {
    const int m = min(C, end - pos);
    float acc[4][4] = {};
    auto inter = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
      product<D>(acc, s.x, s.s, r0, c0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] *= s.pw[r0 + i + 1];
    };
    auto intra = [&]() {
      uint64_t d[4][4] = {};  // rows r0 .. r0 + 3, columns j0 + 16 j: sums over even and odd places
#pragma unroll 4
      for (int e = 0; e < D; e += 4) {
        ulonglong2 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(&s.x[r0 + i][e]);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const ulonglong2*>(&s.y[j0 + 16 * j][e]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) d[i][j] = f2_fma(a[i].y, b[j].y, f2_fma(a[i].x, b[j].x, d[i][j]));
      }
      __syncthreads();  // the previous products' p has been read
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int gap = r0 + i - (j0 + 16 * j);
          float even, odd;
          f2_split(d[i][j], even, odd);
          s.p[r0 + i][j0 + 16 * j] = gap >= 0 ? (even + odd) * s.pw[gap] : 0.f;
        }
      __syncthreads();
      product<C>(acc, s.p, s.z, r0, c0);
    };
    auto store = [&](int g) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r0 + i >= m) continue;
        float* to = o + (long long)g * op.xh + (rev ? it.n - 1 - (pos + r0 + i) : pos + r0 + i) * op.xt + c0;
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
      if (!STATES && op.gy == 1) load_rows<D>(s.x, x, op.xt, pos, m, it.n, rev);
      __syncthreads();
      if (!STATES) {
        if (op.gy > 1) {
          intra();
        } else {
          for (int k = 0; k < op.gx; ++k) {
            if (k > 0) {
              __syncthreads();
              load_rows<D>(s.x, x + (long long)k * op.xh, op.xt, pos, m, it.n, rev);
              __syncthreads();
            }
            inter();
            intra();
            store(k);
          }
        }
        __syncthreads();  // the state and z have been read
      }
      for (int e = tid * 4; e < m * V; e += NT * 4) {  // z weighted with its distance to the chunk's end
        float4& v = *reinterpret_cast<float4*>(&s.z[e / V][e % V]);
        const float w = s.pw[m - 1 - e / V];
        v = make_float4(v.x * w, v.y * w, v.z * w, v.w * w);
      }
      __syncthreads();
      const float2 keep = g > 0 ? make_float2(1.f, 0.f) : m == C ? whole : lin_decay(p.log_decay[h], m);
      float a[D / 64][4][4];  // state rows r0 + 64 k ..
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          get4(&s.s[64 * k + r0 + i][c0], a[k][i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) a[k][i][j] = __fmaf_rn(a[k][i][j], keep.x, a[k][i][j] * keep.y);
        }
#pragma unroll 4
      for (int t = 0; t < C; ++t) {  // (rows behind m are zeros)
        float b[4];
        get4(&s.z[t][c0], b);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          float w[4];
          get4(&s.y[t][64 * k + r0], w);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[k][i][j] += w[i] * b[j];
        }
      }
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(&s.s[64 * k + r0 + i][c0]) = make_float4(a[k][i][0], a[k][i][1], a[k][i][2], a[k][i][3]);
    }
    if (!STATES && op.gy > 1) store(0);
  }
  __syncthreads();
  float* to = STATES ? part : !split && p.update ? own : nullptr;
  if (to)
    for (int e = tid * 4; e < D * V; e += NT * 4)
      *reinterpret_cast<float4*>(to + (size_t)(e / V) * D + v0 + e % V) = *reinterpret_cast<const float4*>(&s.s[e / V][e % V]);
}

template <int D, bool STATES> cudaError_t launch(const LinArgs& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(linear_simt_kernel<D, STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  return launch_chained(linear_simt_kernel<D, STATES>, dim3(p.items, p.heads * (D / V), STATES ? p.slots : p.ops), NT, sizeof(Smem<D>), st, p);
}

}  // namespace

cudaError_t launch_linear_simt(const LinArgs& p, bool states, cudaStream_t st) {
  if (p.D == 64) return states ? launch<64, true>(p, st) : launch<64, false>(p, st);
  return states ? launch<128, true>(p, st) : launch<128, false>(p, st);
}

}  // namespace pathattn
