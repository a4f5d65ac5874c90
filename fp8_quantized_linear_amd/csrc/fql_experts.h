// Internal declarations of the mixture of experts: the routing and the chosen
// experts' products.
#pragma once

#include "fql_internal.h"
#include "fql_serving.h"

namespace fql {

// ---- routing ------------------------------------------------------------------
constexpr int kRouteMaxExperts = 1024, kRouteMaxChosen = 64, kRouteMaxGroups = 64;
struct RouteArgs {
  const void* logits;  // [T][ld] bf16 or float32
  int64_t T, ld;
  int E, k;
  const float* bias;  // [E] or null
  int softmax;        // else sigmoid
  int groups, top_groups;
  int renormalize;
  float scale;
  float* weights;    // [T][k]
  int32_t* experts;  // [T][k]
  int lanes_shift;   // log2 of the lanes that score one group (set by launch_route)
};
hipError_t launch_route(bool f32, RouteArgs a, hipStream_t st);

}  // namespace fql
