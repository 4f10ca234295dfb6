// Linear attention: states of single segments joined to states at the segments' starts, copies between slots, and the choice
// of segments.
#include "linear.h"

namespace pathattn {
namespace {

constexpr int NT = 256;

// parts[item] (what a segment adds to a state) becomes the state at the segment's start, for one key head of one sequence and
// four elements per thread; the state after the last segment goes back to the sequence's own.
__global__ void __launch_bounds__(NT) linear_scan_kernel(const LinArgs p) {
  chain();
  const int lane = threadIdx.x & 31, b = blockIdx.y, h = blockIdx.z % p.heads, slot = blockIdx.z / p.heads;
  int first = 0, n = p.L;
  if (!p.packed) {
    first = b * (p.items / p.seqs);
  } else {
    for (int base = 0; base <= b; base += 32) {  // items of the slots before this one
      LinSpan s{0, 0, 0};
      if (base + lane <= b) s = lin_span(p.q_start, base + lane, p.total, p.max_new);
      if (s.n < p.min_new) s.n = 0;
      first += (int)__reduce_add_sync(0xffffffffu, base + lane < b ? (s.n + p.seg - 1) / p.seg : 0);
      n = __shfl_sync(0xffffffffu, s.n, b & 31);
    }
  }
  const int count = min((n + p.seg - 1) / p.seg, p.items - first);
  if (n == 0 || count <= 0) return;
  const float l2 = lin_log2(p.log_decay[h]);
  const float whole = exp2f(l2 * p.seg), tail = exp2f(l2 * (n - (count - 1) * p.seg));
  const size_t dd = (size_t)p.D * p.D, step = (size_t)p.heads * dd, e = ((size_t)blockIdx.x * NT + threadIdx.x) * 4;
  float* part = p.parts + (((size_t)slot * p.items + first) * p.heads + h) * dd + e;
  float* own = p.state ? p.state + ((size_t)b * p.heads + h) * dd + e : nullptr;
  float4 s = own ? *reinterpret_cast<const float4*>(own) : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int AHEAD = 8;  // loads in flight
  for (int i0 = 0; i0 < count; i0 += AHEAD) {
    float4 add[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i0 + i < count) add[i] = *reinterpret_cast<const float4*>(part + (i0 + i) * step);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i0 + i < count) {
        *reinterpret_cast<float4*>(part + (i0 + i) * step) = s;
        const float w = i0 + i + 1 < count ? whole : tail;
        s.x = s.x * w + add[i].x, s.y = s.y * w + add[i].y, s.z = s.z * w + add[i].z, s.w = s.w * w + add[i].w;
      }
  }
  if (own && p.update) *reinterpret_cast<float4*>(own) = s;
}

// children[i] takes the state of parents[i] (null: zeros).  An entry that names no slot, or a child that is listed twice or is
// a parent too (blocks would race), is left out.
__global__ void __launch_bounds__(NT) linear_copy_kernel(float* state, int* status, int slots, size_t elems, const int* parents,
                                                         const int* children, int count) {
  chain();
  const int i = blockIdx.y;
  const int to = children[i], from = parents ? parents[i] : 0;
  bool bad = (unsigned)to >= (unsigned)slots || (unsigned)from >= (unsigned)slots;
  for (int j = threadIdx.x; j < count; j += NT) {
    const int c = children[j];
    bad |= (j != i && c == to) || (parents && (c == from || parents[j] == to));
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) paged_error(status, PATH_PAGED_BAD_SLOT);
    return;
  }
  const size_t n = elems / 4;
  float4* d = reinterpret_cast<float4*>(state + (size_t)to * elems);
  const float4* s = reinterpret_cast<const float4*>(state + (size_t)from * elems);
  for (size_t e = (size_t)blockIdx.x * NT + threadIdx.x; e < n; e += (size_t)gridDim.x * NT)
    d[e] = parents ? s[e] : make_float4(0.f, 0.f, 0.f, 0.f);
}

}  // namespace

cudaError_t launch_linear_scan(const LinArgs& p, cudaStream_t st) {
  return launch_chained(linear_scan_kernel, dim3(p.D * p.D / (4 * NT), p.seqs, p.heads * p.slots), NT, 0, st, p);
}

cudaError_t launch_linear_copy(float* state, int* status, int slots, size_t elems, const int* parents, const int* children,
                               int count, cudaStream_t st) {
  const unsigned x = (unsigned)((elems / 4 + 8 * NT - 1) / (8 * NT));
  return launch_chained(linear_copy_kernel, dim3(x < 64 ? x : 64, count), NT, 0, st, state, status, slots, elems, parents, children, count);
}

// Tokens per segment, a multiple of the chunk: as many segments as let the blocks' waves end evenly, where a call with
// several pays for their states first (`again` of the walk itself, and the launches and the joining, in chunks).
static int choose_seg(int seqs, int len, int units, int chunk, int blocks, double again, double launches) {
  const int chunks = (len + chunk - 1) / chunk;
  int best = chunks;
  double least = 0;
  for (int c = chunks; c >= 1; --c) {  // chunks of a segment
    const int n = (chunks + c - 1) / c;
    if (n > 1 && (chunks + n - 1) / n != c) continue;  // (fewer chunks make as many segments)
    const double waves = (double)(((long long)seqs * n * units + blocks - 1) / blocks);
    const double cost = waves * c * (n > 1 ? 1 + again : 1.0) + (n > 1 ? launches + 0.05 * n : 0.0);
    if (c == chunks || cost < least) {
      least = cost;
      best = c;
    }
  }
  return best * chunk;
}

void lin_plan(LinArgs& p, bool bf16) {
  const int len = p.packed ? p.max_new : p.L;
  const int seqs = p.packed ? (p.total + p.max_new - 1) / p.max_new : p.seqs;
  const int units = p.heads * p.ops, blocks = (p.D == 64 ? 2 : 1) * 152;
  // A state takes about half as long as a walk; of several query heads, each is a walk of its own (the launches then are less
  // beside a chunk) but dq's and the forward's states are made once.
  const double again = bf16 ? 0.5 * (p.ops == 1 ? 1.0 / p.G : (1.0 + p.G) / (3.0 * p.G)) : 0.35;
  p.seg = bf16 ? choose_seg(seqs, len, units, kLinChunk, blocks, again, 2.5 / p.G)
               : choose_seg(seqs, len, units * (p.D / 64), kLinChunkF32, blocks, again, 1.5);
  if (!p.packed) {
    p.max_new = p.L;
    p.items = p.seqs * ((p.L + p.seg - 1) / p.seg);
  } else {  // every slot of several tokens may end in a partly filled segment
    const int multi = p.total / p.min_new;
    p.items = p.total / p.seg + (multi < p.seqs ? multi : p.seqs);
  }
}

size_t lin_ws_bytes(const LinArgs& p) {
  return 256 + (p.max_new > p.seg ? (size_t)p.slots * p.items * p.heads * p.D * p.D * 4 : 0);
}

cudaError_t launch_linear(LinArgs p, bool bf16, char* ws, cudaStream_t st) {
  p.parts = (float*)(ws + 256);
  cudaError_t e = cudaSuccess;
  if (bf16 && !p.packed) e = cudaMemsetAsync(p.err, 0, sizeof(int), st);  // (packed: the token kernel has)
  auto pass = [&](bool states) { return bf16 ? launch_linear_tc(p, states, st) : launch_linear_simt(p, states, st); };
  if (e == cudaSuccess && p.max_new > p.seg) {
    e = pass(true);
    if (e == cudaSuccess) e = launch_linear_scan(p, st);
  }
  return e == cudaSuccess ? pass(false) : e;
}

}  // namespace pathattn
