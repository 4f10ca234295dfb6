// Paged serving on the tensor cores: what the planning, preparing and merging kernels share with the attention.
#pragma once

#include "paged.h"

namespace pathattn {

constexpr int kTcKeys = 128;         // cached rows per step
constexpr int kTcPair = 256;         // query rows of a block: two 128-row tiles
constexpr int kTcBlocks = 152;       // one persistent block per SM
constexpr int kTcBlockTokens = 256;  // new tokens that share one version of the earlier new keys
constexpr int kTcPassTokens = 4096;  // new tokens of a slot per pass: bounds the versions (their rows grow with its square)
constexpr int kRewriteRows = 128;    // cached rows per rewrite tile

// Plan, operands and parts of a pass (device pointers into the workspace).  Row i G + g of a (slot, key head)
// is head g of new token i; 256 rows are a pair, G pairs hold the tokens of a block.
struct TcPlan {
  int pairs, blocks;        // query pairs of a head and blocks that the arrays hold
  int *cstart, *bstart;     // [slots + 1]: first chunk, first block of each slot
  int *pstart, *rstart;     // first query pair, first rewrite tile
  int *mstart;              // slots of the round before this one: the number of its M
  int group;                // slots that a round may have
  long long* vstart;        // first version row
  long long* ustart;        // first (head, pair, key tile) unit: a pair's cached tiles, then those of earlier blocks
  float *m, *l, *acc;       // parts [..][256](, [D]): thread block c's share of item i is part i + c; the items of
                            // query pair x of the list of all (slot, head, pair): 2 x cached, 2 x + 1 own
  const float* cn;          // sums of log f since the start of the pass [heads][blocks * 256]
  const void *z, *zs;       // queries at the start of the pass and of their block [rounded, rest][heads][pairs][256][D]; the
                            // rest at head dim 128 only of pairs with up to 128 rows
  const void* ver;          // version rows
  const void* mm;           // M: [high, rest][slots of the round][heads][D][D]
  long long ver_rows;
  int* err;                 // first wait that gave up
};

// Key tiles that the first `pairs` pairs of a slot meet in earlier blocks: a pair of block m meets 2 m.
PATH_HD long long new_units(long long pairs, int G) {
  const long long m = pairs / G, rest = pairs % G;
  return G * m * (m - 1) + 2 * rest * m;
}

#ifdef __CUDACC__
// The new tokens of a slot (of the whole call: s) in this pass; slots with fewer than min_new have none.
__device__ __forceinline__ SlotSpan pass_part(const PagedArgs& p, SlotSpan s) {
  if (s.n < p.min_new) s.n = 0;
  const int n = s.n - p.skip;
  s.q0 += p.skip;
  s.t0 += p.skip;
  s.n = n < 0 ? 0 : n < kTcPassTokens ? n : kTcPassTokens;
  return s;
}
__device__ __forceinline__ SlotSpan pass_span(const PagedArgs& p, int b) { return pass_part(p, slot_span(p, b)); }
__device__ __forceinline__ long long units_per_block(const TcPlan& pl, int slots) {
  return (pl.ustart[slots] + kTcBlocks - 1) / kTcBlocks;
}
#endif

cudaError_t launch_rewrite_tc(const PagedArgs& p, const TcPlan& pl, cudaStream_t st);
cudaError_t launch_attend_tc(const PagedArgs& p, const TcPlan& pl, cudaStream_t st);

}  // namespace pathattn
