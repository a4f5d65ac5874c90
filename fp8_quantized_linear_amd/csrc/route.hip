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
// One wave a token, expert 64 i + lane in register i. Each lane sorts its own R keys
// once (c as an ordered 64-bit number); then the k largest come out one by one, each
// lane offering its first: the largest upper half by six DPP steps, and only where
// several lanes share it the lower half and the index. What bounds it: a chain of short
// steps for few tokens (one of 64 experts 2.9 us, 333 of 128 5.0, traced), vector issue for
// many: 8192 tokens of 256 float32 experts in 8 groups 14.4 us a call (traced 16.0), where their
// 9 MB take 1.8: 849 vector instructions a token, 140 to 180 of them float64.
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

// e^x in float64 for |x| up to 800 (inf and 0 beyond the range of the type): x = n ln 2 + r
// with ln 2 in two parts, the first of 40 bits so that n times it is exact (Cody and Waite's
// reduction), and Taylor's series of e^r to r^13 / 13!, whose rest is below 5e-18 for
// |r| <= ln 2 / 2.
__device__ __forceinline__ double exp64(double x) {
  x = __builtin_fmin(__builtin_fmax(x, -800.0), 800.0);
  const double n = __builtin_rint(x * 0x1.71547652b82fep+0);
  double r = __builtin_fma(-n, 0x1.62e42fefa2000p-1, x);
  r = __builtin_fma(-n, 0x1.9ef35793c7673p-41, r);
  constexpr double inverse_factorial[14] = {1.0,          1.0,           1.0 / 2,        1.0 / 6,         1.0 / 24,
                                            1.0 / 120,    1.0 / 720,     1.0 / 5040,     1.0 / 40320,     1.0 / 362880,
                                            1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600, 1.0 / 6227020800.0};
  double p = inverse_factorial[13];
#pragma unroll
  for (int i = 12; i >= 0; --i) p = __builtin_fma(p, r, inverse_factorial[i]);
  return __builtin_ldexp(p, (int)n);
}

// Orders a wave's own LDS writes before its reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int R, typename X>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const RouteArgs a) {
  // a wave's own: [E + 64] what groups are scored by, group after group with places
  // between them, then [E] all experts' s
  extern __shared__ double numbers[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / 64) + wave;
  if (t >= a.T) return;
  const int E = a.E;
  double* const own = numbers + wave * (E + 64);
  // all loads at once, all scores side by side: a lane past E takes the last expert and drops it
  X raw[R];
  float b[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 64 * i + lane < E ? 64 * i + lane : E - 1;
    raw[i] = static_cast<const X*>(a.logits)[t * a.ld + e];
    b[i] = 0.0f;
    if (a.bias != nullptr) b[i] = a.bias[e];
  }
  float z[R];
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float f;
    if constexpr (sizeof(X) == 2) f = bf16_bits_to_f32(raw[i]);
    else f = raw[i];
    // NaN fails the comparison as -inf does
    z[i] = f > -__builtin_inff() && 64 * i + lane < E ? __builtin_fminf(f, 3.4028234663852886e38f) : -__builtin_inff();
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
      const double v = exp64(FQL_FREE(i) ? (double)z[i] - (double)top : 0.0);
      s[i] = FQL_FREE(i) ? v : 0.0;
      sum += s[i];
    }
    sum = wave_sum(sum);
    const double one = sum > 0.0 ? sum : 1.0;
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = s[i] / one;
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const double v = 1.0 / (1.0 + exp64(FQL_FREE(i) ? -(double)z[i] : 0.0));
      s[i] = FQL_FREE(i) ? v : 0.0;
    }
  }
  uint64_t key[R];
  const bool grouped = a.groups > a.top_groups;
  // e / n, exactly: e < 1024 and e n < 2^20
  auto group_of = [&](int e) { return (int)(((uint32_t)e * a.group_magic) >> 20); };
  const int shift = a.lanes_shift, L = 1 << shift;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 64 * i + lane;
    bool free = FQL_FREE(i);
    double c = s[i];
    key[i] = (uint64_t)order32(z[i]) << 32;
    if (a.bias != nullptr) {
      free = free && b[i] > -__builtin_inff();  // false for NaN
      c += (double)b[i];
      key[i] = order64(c);
    }
    key[i] = free ? key[i] : 0;
    if (grouped && e < E) own[e + (group_of(e) << shift)] = free ? c : -__builtin_inf();
  }
#undef FQL_FREE
  if (grouped) {
    wave_sync();
    // lanes of one group: a power of two, so that they join by butterflies
    const int G = a.groups, n = E / G;
    const int g = lane >> shift;
    double b1 = -__builtin_inf(), b2 = -__builtin_inf();
    if (g < G)
      for (int j = lane & (L - 1); j < n; j += L) {
        const double v = own[g * (n + L) + j];
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
    const uint64_t score = (uint64_t)__double_as_longlong(b2 > -__builtin_inf() ? b1 + b2 : b1);
    const double mine = __longlong_as_double((long long)score);
    // how many groups are before the lane's
    int before = 0;
    for (int o = 0; o < G; ++o) {
      const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)score, o << shift);
      const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(score >> 32), o << shift);
      const double v = __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
      before += v > mine || (v == mine && o < g) ? 1 : 0;
    }
    // a kept group has its bit at its first lane
    const uint64_t kept = __ballot(g < G && before < a.top_groups && mine > -__builtin_inf());
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int e = 64 * i + lane;
      if (e < E && !((kept >> (group_of(e) << shift)) & 1)) key[i] = 0;
    }
    wave_sync();
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (64 * i + lane < E) own[64 * i + lane] = s[i];
  wave_sync();
  // largest first; equal ones stay in the order of their indexes
  int at[R];
#pragma unroll
  for (int i = 0; i < R; ++i) at[i] = 64 * i + lane;
#pragma unroll
  for (int n = R - 1; n > 0; --n)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool swap = key[i + 1] > key[i];
      const uint64_t k0 = key[i], k1 = key[i + 1];
      const int i0 = at[i], i1 = at[i + 1];
      key[i] = swap ? k1 : k0;
      key[i + 1] = swap ? k0 : k1;
      at[i] = swap ? i1 : i0;
      at[i + 1] = swap ? i0 : i1;
    }
  // lane j keeps the j-th choice
  int we = -1;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t hi = (uint32_t)(key[0] >> 32);
    const uint32_t m = wave_max(hi);
    if (m == 0u) break;  // none left (every key to be chosen has an upper half above 0)
    uint64_t who = __ballot(hi == m);
    if (who & (who - 1)) {
      const uint32_t lo = hi == m ? (uint32_t)key[0] : 0u;
      const uint32_t ml = wave_max(lo);
      who = __ballot(hi == m && (uint32_t)key[0] == ml);
      if (who & (who - 1)) {
        const uint32_t inv = hi == m && (uint32_t)key[0] == ml ? 0xFFFFFFFFu - (uint32_t)at[0] : 0u;
        who = __ballot(inv == wave_max(inv));
      }
    }
    const int from = __builtin_ctzll(who);
    const int e = __builtin_amdgcn_readlane(at[0], from);
    we = lane == j ? e : we;
    if (lane == from) {
#pragma unroll
      for (int i = 0; i + 1 < R; ++i) {
        key[i] = key[i + 1];
        at[i] = at[i + 1];
      }
      key[R - 1] = 0;
    }
  }
  double ws = we >= 0 ? own[we] : 0.0;
  if (a.renormalize) {
    const double sum = wave_sum(ws);
    ws = sum > 0.0 ? ws / sum : 0.0;
  }
  if (lane < a.k) {
    a.weights[t * a.k + lane] = (float)(ws * (double)a.scale);
    a.experts[t * a.k + lane] = we;
  }
}

template <int R>
hipError_t launch_r(bool f32, const RouteArgs& a, hipStream_t st) {
  const int waves = a.T < kWaves ? 1 : kWaves;
  const unsigned grid = (unsigned)((a.T + waves - 1) / waves);
  const size_t lds = (size_t)waves * (a.E + 64) * sizeof(double);
  if (f32) route_kernel<R, float><<<grid, 64 * waves, lds, st>>>(a);
  else route_kernel<R, uint16_t><<<grid, 64 * waves, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(bool f32, RouteArgs a, hipStream_t st) {
  a.lanes_shift = 0;
  while ((2 << a.lanes_shift) * a.groups <= 64) ++a.lanes_shift;
  const uint32_t n = (uint32_t)(a.E / a.groups);
  a.group_magic = ((1u << 20) + n - 1) / n;
  if (a.E <= 64) return launch_r<1>(f32, a, st);
  if (a.E <= 128) return launch_r<2>(f32, a, st);
  if (a.E <= 256) return launch_r<4>(f32, a, st);
  if (a.E <= 512) return launch_r<8>(f32, a, st);
  return launch_r<16>(f32, a, st);
}

}  // namespace fql
