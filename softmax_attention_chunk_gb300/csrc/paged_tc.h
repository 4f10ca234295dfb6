// Paged serving on the tensor cores: what the planning, preparing and merging kernels share with the attention.
#pragma once

#include "paged.h"

namespace pathattn {

constexpr int kTcKeys = 128;     // cached rows per step
constexpr int kTcPair = 256;     // query rows of a block: two 128-row tiles
constexpr int kTcBlocks = 152;   // one persistent block per SM

// Plan and parts of the tensor-core attention (device pointers into the workspace).
struct TcPlan {
  int pairs;                // query pairs that a head's z holds room for (at least those of any legal call)
  int* pstart;              // [slots + 1]: first query pair of each slot
  long long* ustart;        // [slots + 1]: first (head, pair, key tile) unit of each slot
  float *m, *l, *acc;       // parts [heads * pairs + kTcBlocks][256](, [D]): block c's share of item i is part i + c
  int* err;                 // first wait that gave up
};

cudaError_t launch_attend_tc(const PagedArgs& p, const TcPlan& pl, const void* z, cudaStream_t st);

}  // namespace pathattn
