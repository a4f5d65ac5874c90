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
  int lanes_shift;       // log2 of the lanes that score one group (set by launch_route, as the next)
  uint32_t group_magic;  // e * group_magic >> 20 is e divided by the experts of a group
};
hipError_t launch_route(bool f32, RouteArgs a, hipStream_t st);

// ---- the chosen experts' feed forward --------------------------------------------
// y_t = residual_t + sum_j w_tj (act(x_q Wu_e^T + bu_e))_q Wd_e^T + bd_e, e = experts_tj.
//
// The pairs (token, place) with an expert in [0, E) are sorted by expert; row r of
// the products is the r-th of them. Activations lie in rows of whole 128-deep
// chunks (ExpertRows), so that a product's row tile can take any rows:
//   codes [row][KC * 128 B] (MXFP4: KC * 64 B), columns past K zero
//   scales: MX [row][KC] dwords (byte j = the chunk's 32-block j), block FP8
//   [row][KC] floats (KC rounded up to 4 in both), INT8 [row] floats
// x lies so by token (the first product gathers its rows), the inner activation by
// sorted row.
struct ExpertRows {
  int64_t ld_codes, ld_scales;  // bytes of a row
};
inline ExpertRows expert_rows(int fmt, int64_t K) {
  const int64_t KC = round_up(K, 128) / 128;
  return ExpertRows{KC * (fmt == SC_MXFP4 ? 64 : 128), fmt == SC_FP8 ? 0 : fmt == SC_INT8 ? 4 : round_up(KC, 4) * 4};
}

constexpr int kMaxExperts = 1024;

struct ProductPlan {
  bool large;                // experts_tile_kernel or experts_block_kernel (32 x 32 tiles), else
                             // experts_product_kernel (16 x 16)
  int wm, wn, mtw, ntw, st;  // waves, tiles a wave, ring depth
  int rows, cols;            // of a workgroup's tile
  int64_t max_tiles;         // upper bound of a pass's row tiles
};

// What one call (or one pass of it: tokens are taken `tokens` at a time, so that
// offsets stay within 32 bits and the workspace within bounds) runs.
struct ExpertsPlan {
  int fmt;
  bool token;  // a few tokens: every pair for itself (experts_token.h), without sorting
  ProductPlan up, down;
  bool h_quantized;  // the first product quantizes the inner activation itself
  int64_t tokens;    // tokens a pass
  int64_t pairs;     // of a pass
  // workspace, in order (every size a multiple of 256)
  int64_t counter_bytes, meta_bytes, xcode_bytes, xscale_bytes, h_bytes, hcode_bytes, hscale_bytes, d_bytes, total_bytes;
};
// N: output columns of the first product (before the activation), I: its activation's, Ho: of the second.
ExpertsPlan plan_experts(int fmt, int64_t T, int64_t k, int64_t E, int64_t H, int64_t N, int64_t I, int64_t Ho);
// Workspace bytes of a call of T tokens or of any number below.
int64_t experts_workspace(int fmt, int64_t T, int64_t k, int64_t E, int64_t H, int64_t N, int64_t I, int64_t Ho);
std::string describe_experts(const ExpertsPlan& p);

struct ExpertWeights {
  const uint8_t* packed;  // E packed weights of [N][K]
  int64_t stride;         // bytes from one to the next
  int64_t N, K;
  float inv_scale;        // per-tensor FP8: fl32(1 / input_scale) of the product's activation
  const float* alpha;     // [E] output scales or null (1)
  const uint16_t* bias;   // bf16 [E][N] or null
};
struct ExpertsArgs {
  const uint16_t* x;  // bf16 [T][ldx]
  int64_t T, ldx;
  bool aligned;
  ExpertWeights up, down;
  int act;
  int64_t I;
  const float* weights;    // [T][k]
  const int32_t* experts;  // [T][k]
  int k, E;
  const uint16_t* residual;  // bf16 [T][ldr] or null; may be y
  int64_t ldr;
  uint16_t* y;
  int64_t ldy;
};
hipError_t launch_experts(const ExpertsPlan& p, const ExpertsArgs& a, uint8_t* workspace, hipStream_t st);

}  // namespace fql
