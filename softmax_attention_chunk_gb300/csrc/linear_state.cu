// Linear attention: states of single segments joined to states at the segments' starts, copies between slots, and the choice
// of segments.
#include "linear.h"

namespace pathattn {
namespace {

constexpr int NT = 256;

// parts[item] (what a segment adds to a state) becomes the state at the segment's start, for one key head of one sequence and
// four elements per thread; the state after the last segment goes back to the sequence's own.  AHEAD: loads on their way, the one
// thing it waits for (32 heads x 16384 at d 64, nine segments: 94.6 us the call with eight, 92.9 with sixteen; prompts of up to
// six segments: 30.8 and 31.9).
template <int AHEAD>
__global__ void __launch_bounds__(NT) linear_scan_kernel(const LinArgs p) {
  chain();
  const int lane = threadIdx.x & 31, b = blockIdx.y, h = blockIdx.z % p.heads, slot = blockIdx.z / p.heads;
  int first = 0, n = p.L;
  if (!p.packed) {
    first = b * (p.items / p.seqs);
  } else {
    if (lin_span(p.q_start, b, p.total, p.max_new).n < p.min_new) return;
    LinOrder order;
    for (int base = 0; base <= b; base += 32) {  // items of the slots before this one
      LinSpan s = lin_spans(p, base, order);
      if (s.n < p.min_new) s.n = 0;
      first += (int)__reduce_add_sync(0xffffffffu, base + lane < b ? (s.n + p.seg - 1) / p.seg : 0);
      n = __shfl_sync(0xffffffffu, s.n, b & 31);  // (the last time: this slot's)
    }
  }
  const int count = (n + p.seg - 1) / p.seg;
  if (n == 0 || first + count > p.items) return;  // (the tokens are no two slots', so there are items for all)
  const float2 whole = lin_decay(p.log_decay[h], p.seg), tail = lin_decay(p.log_decay[h], n - (count - 1) * p.seg);
  const size_t dd = (size_t)p.D * p.D, step = (size_t)p.heads * dd, e = ((size_t)blockIdx.x * NT + threadIdx.x) * 4;
  float* part = p.parts + (((size_t)slot * p.items + first) * p.heads + h) * dd + e;
  float* own = p.state ? p.state + ((size_t)b * p.heads + h) * dd + e : nullptr;
  float4 s = own ? *reinterpret_cast<const float4*>(own) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < count; i0 += AHEAD) {
    float4 add[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i0 + i < count) add[i] = *reinterpret_cast<const float4*>(part + (i0 + i) * step);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i0 + i < count) {
        *reinterpret_cast<float4*>(part + (i0 + i) * step) = s;
        const float2 w = i0 + i + 1 < count ? whole : tail;
        s.x = s.x * w.x + (s.x * w.y + add[i].x), s.y = s.y * w.x + (s.y * w.y + add[i].y);
        s.z = s.z * w.x + (s.z * w.y + add[i].z), s.w = s.w * w.x + (s.w * w.y + add[i].w);
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
  const bool many = p.max_new > 8 * (long long)p.seg;  // segments
  return launch_chained(many ? linear_scan_kernel<16> : linear_scan_kernel<8>, dim3(p.D * p.D / (4 * NT), p.seqs, p.heads * p.slots), NT, 0, st, p);
}

cudaError_t launch_linear_copy(float* state, int* status, int slots, size_t elems, const int* parents, const int* children,
                               int count, cudaStream_t st) {
  const unsigned x = (unsigned)((elems / 4 + 8 * NT - 1) / (8 * NT));
  return launch_chained(linear_copy_kernel, dim3(x < 64 ? x : 64, count), NT, 0, st, state, status, slots, elems, parents, children, count);
}

// Microseconds of a step (a chunk of one query head) of a walk and of a state, with a block to an SM and with all the blocks an
// SM holds, as measured (bf16: the walks of several query heads overlap more than chunks of one do).
struct Steps {
  double walk, walk_full, state, state_full;
};
static Steps step_times(const LinArgs& p, bool bf16) {
  if (!bf16) return p.D == 64 ? Steps{10.4, 17.0, 3.2, 5.0} : Steps{15.5, 15.5, 4.6, 4.6};
  if (p.D == 64) return p.G == 1 ? Steps{2.4, 2.85, 1.0, 2.0} : Steps{1.65, 2.3, 1.0, 2.0};
  return p.G == 1 ? Steps{3.1, 3.1, 1.45, 1.45} : Steps{2.3, 2.3, 1.45, 1.45};
}
// Tokens per segment, a multiple of the chunk.  One segment to a sequence needs nothing but the walk; several run side by
// side, and cost the states at their starts: the states' own pass, two more launches and 16 D^2 bytes of traffic each (1 x 8 x
// 4096 d 64, forward: 78 us in one segment, 25 in sixteen; 8 x 32 x 4096: 103 in one, 174 in two).
static int choose_seg(const LinArgs& p, bool bf16, int seqs, int len, int chunk) {
  const Steps t = step_times(p, bf16);
  const int per_head = bf16 ? 1 : p.D / 64, full = 152 * (p.D == 64 ? 2 : 1);
  const int chunks = (len + chunk - 1) / chunk;
  int best = chunks;
  double least = 0;
  for (int s = 1; s <= chunks && s <= full; ++s) {  // segments
    const int c = (chunks + s - 1) / s, n = (chunks + c - 1) / c;  // chunks of one; as many of those as there then are
    if (n != s) continue;
    auto waves = [&](double blocks, double one, double all) { return blocks <= 152 ? one : all * (double)(long long)((blocks + full - 1) / full); };
    const double heads = (double)seqs * p.heads * n;
    double cost = c * p.G * waves(heads * p.ops * per_head, t.walk, t.walk_full);
    if (n > 1) {
      // (of a backward pass's two states one has all query heads to add up)
      const double most = p.slots == 1 ? 1 : p.G, mean = p.slots == 1 ? 1 : (1 + p.G) / 2.0;
      const double states = c * mean * waves(heads * p.slots * per_head, t.state, t.state_full);
      cost += (states > c * most * t.state ? states : c * most * t.state) + 7 + p.D / 64 * 0.45 * n + heads * p.slots * p.D * p.D * 16 / 5e6;
    }
    if (n == 1 || cost < least) {
      least = cost;
      best = c;
    }
  }
  return best * chunk;
}

void lin_plan(LinArgs& p, bool bf16) {
  const int len = p.packed ? p.max_new : p.L;
  const int seqs = p.packed ? (p.total + p.max_new - 1) / p.max_new : p.seqs;
  p.seg = choose_seg(p, bf16, seqs, len, bf16 ? kLinChunk : kLinChunkF32);
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
