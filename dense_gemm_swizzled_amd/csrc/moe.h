// moe.h -- launch parameters of the expert-routing kernels (moe.hip).
#pragma once

#include <stdint.h>

#include "../../include/swizzled_gemm.h"

namespace sg {

struct RouteParams {
  int64_t T;
  int E, top_k;
  const void* logits;       // [T][ldl]
  int64_t ldl;
  const float* bias;        // [E] or NULL (forward)
  int score, n_groups, top_groups, group_score;
  int renorm;
  float scale;
  bool by_score;            // order by score + bias (64 bits), not by logit
  bool vec, vec_d;          // four logits / gradients at a multiple of four: one access
  float* weights;           // [T][top_k] (forward)
  int32_t* ids;             // [T][top_k]; read by the backward pass
  const float* dweights;    // [T][top_k] (backward)
  void* dlogits;            // [T][lddl] of the logits' type (backward)
  int64_t lddl;
};

struct BalanceParams {
  int64_t T;
  int E, top_k;
  const void* logits;       // [T][ldl]
  int64_t ldl;
  int score;
  bool vec, vec_d;          // as above
  int64_t chunk;            // tokens of one workgroup (forward)
  const int32_t* ids;       // [T][top_k] (forward)
  float* loss;              // [1] (forward)
  int32_t* counts;          // [E]; read by the backward pass
  int32_t* tokens;          // [1]; read by the backward pass
  void* part;               // workspace: pairs, see balance.hip
  int parts;                // workgroups
  const float* dloss;       // [1] (backward)
  void* dlogits;            // [T][lddl] of the logits' type (backward)
  int64_t lddl;
};

struct PlanParams {
  int64_t P;                // pairs
  int E, top_k;
  int64_t chunk;            // pairs of one workgroup
  const int32_t* ids;       // [P]
  int32_t* offsets;         // [E + 1]
  int32_t* rows;            // [P]
  int32_t* slots;           // [P]
  int32_t* counts;          // workspace: [workgroups][E], or null for one launch
  uint32_t div_mul;         // of a division by top_k
  int div_shift;
};

}  // namespace sg
