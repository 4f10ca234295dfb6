// Linear attention with a decay per head: declarations shared by its translation units (not part of the ABI).
//
// All of it is one operation ("walk"), for a key head with decay g and its state S (D x D, float32):
//   S <- g S + y_i z_i^T,   o_i = scale S^T x_i      for the tokens i of a sequence in walk order,
//   o_i = scale sum_{j <= i} g^(i-j) (x_i . y_j) z_j + scale g^(i+1) S_0^T x_i.
// The forward is (x, y, z) = (q, k, v), and because the weight of a pair of tokens depends on their distance alone, each
// gradient is the same walk over other operands: dq = (do, v, k), and from the last token to the first
// dk = (v, do, q), dv = (k, q, do).  With several query heads to a key head, either x has them (o too: they read one state)
// or y and z do (their products add up in one state).
#pragma once

#include "../../include/path_attn.h"
#include "internal.h"
#include "paged.h"

namespace pathattn {

constexpr int kLinTokenMax = 16;  // slots with up to so many new tokens go through the recurrent kernel
constexpr int kLinChunk = 128;    // tokens of a chunk; segments are multiples of it
constexpr int kLinChunkF32 = 64;  // in float32

struct LinOp {
  const void *x, *y, *z;
  void* o;
  int gx, gy;                      // query heads of a key head in x and o, in y and z (one of them is 1)
  int reverse;                     // from the last token to the first
  long long xt, xh, xb;            // strides of x and o in elements: token, head, sequence
  long long yt, yh, yb;            // of y and z
  int slot, turned;                // its states in parts, and whether they lie there transposed
};

// What the kernels of a call need, by value.
struct LinArgs {
  LinOp op[3];
  int ops;
  int slots, maker[3];             // states in parts: dk's are dv's transposed; the operation that makes each slot's
  int D, heads, G;                 // G: query heads per key head
  int seqs, L;                     // dense: sequences of L tokens
  const int* q_start;              // packed: slot b's tokens are q_start[b] .. q_start[b + 1] - 1; null: one each
  int packed, total, max_new, min_new;  // packed: slots with fewer than min_new tokens are the recurrent kernel's
  int seg, items;                  // tokens of a segment; (sequence, segment) pairs that the grid covers
  float scale;
  const float* log_decay;          // [heads]
  float* state;                    // [seqs][heads][D][D] or null (zero): the state before, and after where update is set
  int update;
  float* parts;                    // [slots][items][heads][D][D]: states of single segments, then those at their starts
  int* err;                        // tensor-core kernels: first wait that gave up,
  int* status;                     // and where a cache keeps it (or null)
  unsigned stall_ns;               // test hook: nonzero makes every block give up a wait (debug_stall_ns)
};

// log2 of the decay: log_decay is kept in [-10000, 0] (exp of the lower end is 0 for any distance but 0), NaN stays.
PATH_HD float lin_log2(float ld) {
  const float c = ld > 0.f ? 0.f : ld < -10000.f ? -10000.f : ld;
  return c * kLog2e;
}

#ifdef __CUDACC__
// g^n as the sum of two floats (x: rounded, y: what that leaves).  A state is multiplied by it over and over: one float, off by
// up to 2^-24 near 1 and the same way every time, would let it forget at another rate (single tokens at log_decay -1e-5: 7e-4 of the
// state after 20000; with the rest under 1.1e-5, the sums' own rounding).  For x > -1/8, expm1(x) by five terms of its series (the sixth
// is 2^-24 of it at most), 1 + that as a float and a rest exactly; states that lose more at a time remember eight times at most.
__device__ __forceinline__ float2 lin_decay(float ld, int n) {
  const float x = (ld > 0.f ? 0.f : ld < -10000.f ? -10000.f : ld) * n;
  if (!(x > -0.125f)) return make_float2(exp2f(x * kLog2e), 0.f);  // (NaN too)
  const float e = x * (1.f + x * (0.5f + x * (1.f / 6 + x * (1.f / 24 + x * (1.f / 120))))), hi = 1.f + e;
  return make_float2(hi, (1.f - hi) + e);
}
#endif

// New tokens of slot b of a packed call; code for a bad row of q_start.  A row by itself: a good one that begins before an earlier good
// one's tokens end (which takes a row between them that falls) is as bad, and every kernel leaves its slot out.  So no token is two
// slots', and the slots' segments are no more than the tokens allow.
struct LinSpan {
  int q0, n, code;
};
PATH_HD LinSpan lin_span(const int* q_start, int b, int total, int max_new) {
  LinSpan s{b, 1, 0};
  if (!q_start) return s;
  s.q0 = q_start[b];
  const long long n = (long long)q_start[b + 1] - s.q0;
  if (s.q0 < 0 || n < 0 || (long long)s.q0 + n > total || n > max_new) {
    s.q0 = s.n = 0;
    s.code = PATH_PAGED_BAD_START;
    return s;
  }
  s.n = (int)n;
  return s;
}

#ifdef __CUDACC__
// The spans of slots base .. base + 31, one to a lane, by a whole warp that takes the slots in order.
struct LinOrder {
  int end = 0;        // of the tokens so far
  bool fell = false;  // a bad row was among the slots
};
__device__ __forceinline__ LinSpan lin_spans(const LinArgs& p, int base, LinOrder& o) {
  const int lane = threadIdx.x & 31;
  LinSpan s{0, 0, 0};
  if (base + lane < p.seqs) s = lin_span(p.q_start, base + lane, p.total, p.max_new);
  int upto = s.n ? s.q0 + s.n : 0;
  o.fell |= __any_sync(0xffffffffu, s.code != 0) != 0;
  if (o.fell) {  // (else the ends rise)
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto = max(upto, a);
    }
    const int before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (s.q0 < max(o.end, lane ? before : 0)) s.n = 0;
  }
  o.end = max(o.end, __reduce_max_sync(0xffffffffu, upto));
  return s;
}
struct LinItem {
  int seq, q0, n, seg;  // seg < 0: none
};
// Item `item` of a call, by a whole warp: the segments of all sequences in order.
__device__ __forceinline__ LinItem lin_item(const LinArgs& p, int item) {
  if (!p.packed) {
    const int per = p.items / p.seqs;
    return {item / per, 0, p.L, item % per};
  }
  const int lane = threadIdx.x & 31;
  int before = 0;
  LinOrder order;
  for (int base = 0; base < p.seqs; base += 32) {
    LinSpan s = lin_spans(p, base, order);
    if (s.n < p.min_new) s.n = 0;
    int upto = (s.n + p.seg - 1) / p.seg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += a;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > item);
    if (past) {
      const int at = __ffs(past) - 1;
      const int prev = at ? __shfl_sync(0xffffffffu, upto, at - 1) : 0;
      return {base + at, __shfl_sync(0xffffffffu, s.q0, at), __shfl_sync(0xffffffffu, s.n, at), item - before - prev};
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return {0, 0, 0, -1};
}
#endif

// ---- launchers ----
// Fills seg and items, chosen on the host from sizes alone.
void lin_plan(LinArgs& p, bool bf16);
size_t lin_ws_bytes(const LinArgs& p);
cudaError_t launch_linear(LinArgs p, bool bf16, char* ws, cudaStream_t st);

cudaError_t launch_linear_simt(const LinArgs& p, bool states, cudaStream_t st);  // float32
cudaError_t launch_linear_tc(const LinArgs& p, bool states, cudaStream_t st);    // bf16
cudaError_t launch_linear_scan(const LinArgs& p, cudaStream_t st);
// Slots with up to kLinTokenMax new tokens; reports bad rows of q_start and clears err.
cudaError_t launch_linear_token(const LinArgs& p, bool bf16, cudaStream_t st);
cudaError_t launch_linear_copy(float* state, int* status, int slots, size_t elems, const int* parents, const int* children,
                               int count, cudaStream_t st);

}  // namespace pathattn
