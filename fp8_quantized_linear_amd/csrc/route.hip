// Routing to experts (gfx950): scores of a router's logits and the choice of k
// experts a token.
//
//   s = softmax over the available experts, or 1 / (1 + e^-z)
//   c = s + bias, without a bias the logit z (which orders as s does)
//   group score = the sum of a group's two largest c (s without a bias)
//   chosen: the k largest c among the experts of the best groups, ties to the
//   lowest index;  w = s [/ sum of the chosen s] * factor
//
// An expert is available where its logit is neither NaN nor -inf (and can be
// chosen where its bias is neither, either); +inf counts as the largest finite
// float32. Places that no expert fills get expert -1 and weight 0.
//
// Scores are float64: whether two experts change places hangs on the last bits of
// c, and float32's would differ from one evaluation to the next. Without a bias
// the order is that of the logits themselves and exact.
//
// One wave a token, expert 64 i + lane in register i. The k largest come out one
// by one: c as an ordered 64-bit key, the largest upper half by six DPP steps, and
// only where several lanes share it the lower half and the index. What bounds it: a
// chain of short steps for few tokens, vector issue for many.
#include "fql_device.h"
#include "fql_experts.h"

namespace fql {

namespace {

constexpr int kWaves = 4;  // tokens a workgroup

// Wave-wide maximum of an unsigned number (all lanes active; DPP: shifts within 16
// lanes, then rows to the next ones; the last lane has it).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);  // row_bcast 15 into rows 1, 3
  v = dpp_max<0x143, 0xC>(v);  // row_bcast 31 into rows 2, 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Order-preserving integers: larger number, larger key, and every number's key
// above 0, which stands for "not to be chosen". -0 is made +0 first.
__device__ __forceinline__ uint32_t order32(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int R, typename X>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const RouteArgs a) {
  extern __shared__ double by_group[];  // [waves][E] what groups are scored by, then [64] their scores
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / 64) + wave;
  const bool mine = t < a.T;  // a wave past the last token goes along to the barriers
  const int E = a.E;
  float z[R];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 64 * i + lane;
    z[i] = -__builtin_inff();
    if (mine && e < E) {
      const X v = static_cast<const X*>(a.logits)[t * a.ld + e];
      float f;
      if constexpr (sizeof(X) == 2) f = bf16_bits_to_f32(v);
      else f = v;
      z[i] = f == f ? __builtin_fminf(f, 3.4028234663852886e38f) : z[i];
    }
    top = __builtin_fmaxf(top, z[i]);
  }
#define FQL_FREE(i) (z[i] > -__builtin_inff())
  double s[R];
  if (a.softmax) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      s[i] = FQL_FREE(i) ? exp((double)z[i] - (double)top) : 0.0;
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = FQL_FREE(i) ? s[i] / sum : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = FQL_FREE(i) ? 1.0 / (1.0 + exp(-(double)z[i])) : 0.0;
  }
  uint64_t key[R];
  const bool grouped = a.groups > a.top_groups;
  double* const own = by_group + wave * (E + 64);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 64 * i + lane;
    bool free = FQL_FREE(i);
    double c = s[i];
    key[i] = (uint64_t)order32(z[i]) << 32;
    if (a.bias != nullptr) {
      const float b = e < E ? a.bias[e] : 0.0f;
      free = free && b > -__builtin_inff();  // false for NaN
      c += (double)b;
      key[i] = order64(c);
    }
    if (!free) key[i] = 0;
    if (grouped && e < E) own[e] = free ? c : -__builtin_inf();
  }
#undef FQL_FREE
  if (grouped) {
    __syncthreads();
    // lanes of one group: a power of two, so that they join by butterflies
    const int G = a.groups, n = E / G, shift = a.lanes_shift, L = 1 << shift;
    const int g = lane >> shift;
    double b1 = -__builtin_inf(), b2 = -__builtin_inf();
    if (g < G)
      for (int j = lane & (L - 1); j < n; j += L) {
        const double v = own[g * n + j];
        const double lo = v < b1 ? v : b1;
        b1 = v > b1 ? v : b1;
        b2 = lo > b2 ? lo : b2;
      }
    for (int o = 1; o < L; o <<= 1) {
      const double o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
      const double lo = o1 < b1 ? o1 : b1, hi2 = o2 > b2 ? o2 : b2;
      b1 = o1 > b1 ? o1 : b1;
      b2 = lo > hi2 ? lo : hi2;
    }
    // a lone expert counts alone; a group without one is below all
    const double score = b2 > -__builtin_inf() ? b1 + b2 : b1;
    double* const scores = own + E;
    __syncthreads();
    if (g < G && (lane & (L - 1)) == 0) scores[g] = score;
    __syncthreads();
    // lane g: how many groups are before group g
    bool keep = false;
    if (lane < G) {
      const double mine_score = scores[lane];
      int before = 0;
      for (int o = 0; o < G; ++o) {
        const double v = scores[o];
        before += v > mine_score || (v == mine_score && o < lane) ? 1 : 0;
      }
      keep = before < a.top_groups && mine_score > -__builtin_inf();
    }
    const uint64_t kept = __ballot(keep);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int e = 64 * i + lane;
      if (e < E && !((kept >> (e / n)) & 1)) key[i] = 0;
    }
  }
  // lane j keeps the j-th choice
  double ws = 0.0;
  int we = -1;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < R; ++i) {  // equal keys: the lower i is the lower index
      bi = key[i] > best ? i : bi;
      best = key[i] > best ? key[i] : best;
    }
    const uint32_t hi = (uint32_t)(best >> 32);
    const uint32_t m = wave_max(hi);
    if (m == 0u) break;  // none left (every key to be chosen has an upper half above 0)
    uint64_t who = __ballot(hi == m);
    if (who & (who - 1)) {
      const uint32_t lo = hi == m ? (uint32_t)best : 0u;
      const uint32_t ml = wave_max(lo);
      who = __ballot(hi == m && (uint32_t)best == ml);
      if (who & (who - 1)) {
        const uint32_t inv = hi == m && (uint32_t)best == ml ? 0xFFFFFFFFu - (uint32_t)(64 * bi + lane) : 0u;
        who = __ballot(inv == wave_max(inv));
      }
    }
    const int from = __builtin_ctzll(who);
    const int i0 = __builtin_amdgcn_readlane(bi, from);
    double score = 0.0;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i == i0) {
        score = s[i];
        if (lane == from) key[i] = 0;
      }
    const uint64_t bits = (uint64_t)__double_as_longlong(score);
    const uint32_t s0 = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)bits, from);
    const uint32_t s1 = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(bits >> 32), from);
    if (lane == j) {
      ws = __longlong_as_double((long long)(((uint64_t)s1 << 32) | s0));
      we = 64 * i0 + from;
    }
  }
  if (a.renormalize) {
    const double sum = wave_sum(ws);
    ws = sum > 0.0 ? ws / sum : 0.0;
  }
  if (mine && lane < a.k) {
    a.weights[t * a.k + lane] = (float)(ws * (double)a.scale);
    a.experts[t * a.k + lane] = we;
  }
}

template <int R>
hipError_t launch_r(bool f32, const RouteArgs& a, hipStream_t st) {
  const int waves = a.T < kWaves ? 1 : kWaves;
  const unsigned grid = (unsigned)((a.T + waves - 1) / waves);
  const size_t lds = a.groups > a.top_groups ? (size_t)waves * (a.E + 64) * sizeof(double) : 0;
  if (f32) route_kernel<R, float><<<grid, 64 * waves, lds, st>>>(a);
  else route_kernel<R, uint16_t><<<grid, 64 * waves, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(bool f32, RouteArgs a, hipStream_t st) {
  a.lanes_shift = 0;
  while ((2 << a.lanes_shift) * a.groups <= 64) ++a.lanes_shift;
  if (a.E <= 64) return launch_r<1>(f32, a, st);
  if (a.E <= 128) return launch_r<2>(f32, a, st);
  if (a.E <= 256) return launch_r<4>(f32, a, st);
  if (a.E <= 512) return launch_r<8>(f32, a, st);
  return launch_r<16>(f32, a, st);
}

}  // namespace fql
