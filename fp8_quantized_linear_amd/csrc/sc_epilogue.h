// Fused epilogue of the scaled-MFMA linear kernels: bias, activation
// (gated or not) and residual on the float32 accumulators, one rounding to
// bf16 at the end. act(z), z = alpha * acc + bias:
//   relu       max(z, 0)
//   gelu       z/2 (1 + erf(z / sqrt 2))
//   gelu_tanh  z/2 (1 + tanh(u)) = z sigma(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
//   silu       z sigma(z), sigma(z) = 1 / (1 + e^-z)
//   swiglu     silu(gate) * up; the tile's columns alternate 16 gate columns
//              and their 16 up columns, so a lane's accumulators of column
//              tiles 2j and 2j + 1 are one output's pair and nothing has to
//              move between lanes.
// What it costs: 4096 x 4096 x 14336 MXFP8, the product alone 229 us (2.10 PFLOP/s),
// with bias 230, SiLU 242, tanh-GELU 254, GELU 264, a residual 265 (it reads as much
// again as the output writes), SwiGLU 224 (half the output).
#pragma once

#include "fql_gemm.h"
#include "fql_serving.h"

namespace fql {

// z * sigma(t) in float32, the reciprocal and the exponential to about 1 ulp
// (the result is rounded to bf16). e^-t may overflow to infinity: the product
// is then -0, the limit. z = -inf would give -inf * 0; its limit 0 is given
// instead.
__device__ __forceinline__ float z_sigmoid(float z, float t) {
  const float r = z * __builtin_amdgcn_rcpf(1.0f + __expf(-t));
  return z == -__builtin_inff() ? 0.0f : r;
}

// |z| / 2 erfc(|z| / sqrt 2) in float32, relative error below 2e-6 up to |z| = 4
// and below 1e-5 down to float32's subnormals (|z| = 12.9): z^2 / 2 and its
// product with log2 e are rounded, and the exponential multiplies that error by
// z^2 / 2. The result is rounded to bf16 (4e-3). With x = |z| / sqrt 2 and t = 1 / (1 + 0.4 x): erfc(x) = e^(-x^2) t P(t), P the
// polynomial of degree 8 fitted to e^(x^2) erfc(x) / t for the least largest
// relative error over x >= 0 (3.9e-7; reweighted least squares). A relative
// bound keeps the far negative tail, which 1 + erf would cancel away;
// and this is about 15 instructions an element where the library's erff cost
// the 4096 x 14336 MXFP8 layer 40 us more.
__device__ __forceinline__ float half_erfc_tail(float a) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28284271f, a, 1.0f));
  float p = 0.05025898292660713f;
  p = __builtin_fmaf(p, t, -0.18288609385490417f);
  p = __builtin_fmaf(p, t, 0.16905444860458374f);
  p = __builtin_fmaf(p, t, -0.0055745309218764305f);
  p = __builtin_fmaf(p, t, 0.1414116770029068f);
  p = __builtin_fmaf(p, t, 0.16854849457740784f);
  p = __builtin_fmaf(p, t, 0.2078416347503662f);
  p = __builtin_fmaf(p, t, 0.22566966712474823f);
  p = __builtin_fmaf(p, t, 0.22567586600780487f);
  return 0.5f * a * t * p * __expf(-0.5f * a * a);
}

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if (ACT == kActRelu) return z > 0.0f ? z : (z == z ? 0.0f : z);  // NaN stays
  if (ACT == kActGelu) {
    const float h = half_erfc_tail(__builtin_fminf(__builtin_fabsf(z), 64.0f));  // 0 beyond
    return z > 0.0f ? z - h : (z == z ? -h : z);
  }
  if (ACT == kActGeluTanh) return z_sigmoid(z, 1.5957691216057308f * (z + 0.044715f * z * z * z));
  if (ACT == kActSilu) return z_sigmoid(z, z);
  return z;
}
__device__ __forceinline__ float apply_act(float z, int act) {
  switch (act) {
    case kActRelu: return act_of<kActRelu>(z);
    case kActGelu: return act_of<kActGelu>(z);
    case kActGeluTanh: return act_of<kActGeluTanh>(z);
    case kActSilu: return act_of<kActSilu>(z);
    default: return z;
  }
}

// The epilogue's per-call state. n counts the accumulators' columns, no the
// output's (half of them when gated).
struct EpiOut {
  int M, N;
  float alpha;
  const uint16_t* bias;
  ScEpilogue e;
  uint16_t* y;
  int64_t ldy;
  __device__ __forceinline__ bool gated() const { return e.act == kActSwiglu; }
  __device__ __forceinline__ float bias_at(int n) const {
    return bias != nullptr && n < N ? bf16_bits_to_f32(bias[n]) : 0.0f;
  }
  // four rows' values of one output column from the accumulators of column n
  // (gated: of gate column n and up column n + 16)
  __device__ __forceinline__ float4v plain(const float4v& s, int n) const {
    const float b = bias_at(n);
    float4v v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = apply_act(alpha * s[i] + b, e.act);
    return v;
  }
  __device__ __forceinline__ float4v gate(const float4v& g, const float4v& u, int n) const {
    const float bg = bias_at(n), bu = bias_at(n + 16);
    float4v v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float z = alpha * g[i] + bg;
      v[i] = z_sigmoid(z, z) * (alpha * u[i] + bu);
    }
    return v;
  }
  // rows m .. m + 3 of output column n, straight to memory
  __device__ __forceinline__ void put(const float4v& v, int m, int n, int n_end) const {
    if (n >= n_end) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (m + i >= M) continue;
      const float r = e.residual != nullptr ? bf16_bits_to_f32(e.residual[(int64_t)(m + i) * e.ldr + n]) : 0.0f;
      y[(int64_t)(m + i) * ldy + n] = (uint16_t)f32_to_bf16_bits(v[i] + r);
    }
  }
  // fragments of column tiles 2j, 2j + 1 at accumulator columns n, n + 16
  __device__ __forceinline__ void emit_pair(const float4v& a, const float4v& b, int m, int n) const {
    if (gated()) {
      // N is a multiple of 32, so a gate column below N has its up column below N
      put(gate(a, b, n), m, (n >> 5) * 16 + (n & 15), n < N ? N / 2 : 0);
    } else {
      put(plain(a, n), m, n, N);
      put(plain(b, n + 16), m, n + 16, N);
    }
  }
};

// finish_frags with the epilogue: the same split-K slab, arrival counter and
// order of the sum. Fragments come in pairs (2p, 2p + 1) of neighbouring
// column tiles of the same rows.
template <int FR, typename RowOf, typename ColOf, int NW>
__device__ __forceinline__ void finish_frags_fused(float4v (&frag)[FR], RowOf row_of, ColOf col_of, int m0, int n0,
                                                   int split, int splits, const EpiOut& o,
                                                   float4v* __restrict__ slab, uint32_t* counter,
                                                   uint32_t* s_flag) {
  static_assert(FR % 2 == 0, "fragment pairs");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (splits == 1) {
#pragma unroll
    for (int f = 0; f < FR; f += 2) o.emit_pair(frag[f], frag[f + 1], m0 + row_of(f, 0), n0 + col_of(f));
    return;
  }
  float4v* mine = slab + wave * FR * 64;
  const int64_t zstride = (int64_t)NW * FR * 64;
#pragma unroll
  for (int f = 0; f < FR; ++f) store_partial(mine + split * zstride + f * 64, lane, frag[f]);
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");  // partial stores have completed
  __syncthreads();
  if (tid == 0) {
    const uint32_t arrived =
        __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_flag = arrived == (uint32_t)(splits - 1) ? 1u : 0u;
  }
  __syncthreads();
  if (*s_flag == 0u) return;
  constexpr int FG = FR < 8 ? FR : 8;
  constexpr int ZB = 16 / FG < 8 ? 16 / FG : 8;
#pragma unroll
  for (int f0 = 0; f0 < FR; f0 += FG) {
    float4v sum[FG];
#pragma unroll
    for (int f = 0; f < FG; ++f) sum[f] = float4v{0.f, 0.f, 0.f, 0.f};
    for (int z0 = 0; z0 < splits; z0 += ZB) {
      float4v v[ZB][FG];
#pragma unroll
      for (int j = 0; j < ZB; ++j) {
        const int z = z0 + j < splits ? z0 + j : splits - 1;
#pragma unroll
        for (int f = 0; f < FG; ++f) v[j][f] = load_partial(mine + z * zstride + (f0 + f) * 64, lane);
      }
#pragma unroll
      for (int j = 0; j < ZB; ++j)
        if (z0 + j < splits)
#pragma unroll
          for (int f = 0; f < FG; ++f) sum[f] += v[j][f];
    }
#pragma unroll
    for (int f = 0; f < FG; f += 2) o.emit_pair(sum[f], sum[f + 1], m0 + row_of(f0 + f, 0), n0 + col_of(f0 + f));
  }
  if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The residual of an R x C output tile as 16-byte row pieces, piece q0 + tid of
// every round of 64 NW: loaded before the products begin, so that its way from
// memory passes under them (a workgroup that fills the LDS has no neighbour to
// hide it under). The residual may be y itself: the tile is read and written
// by this workgroup only.
template <int R, int C, int NW, int RP>
__device__ __forceinline__ void load_residual(const EpiOut& o, int m0, int no, int Nout, uint4v (&piece)[RP]) {
  static_assert(R * C / 8 <= 64 * NW * RP && R * C / 8 % (64 * NW) == 0, "whole pieces per thread");
  const bool vec = (o.e.ldr & 7) == 0 && (reinterpret_cast<uintptr_t>(o.e.residual) & 15) == 0;
#pragma unroll
  for (int i = 0; i < R * C / 8 / (64 * NW); ++i) {
    const int q = i * 64 * NW + threadIdx.x;
    const int m = m0 + q / (C / 8), n = no + (q % (C / 8)) * 8;
    piece[i] = uint4v{0u, 0u, 0u, 0u};
    if (m >= o.M) continue;
    const uint16_t* src = o.e.residual + (int64_t)m * o.e.ldr + n;
    if (vec && n + 8 <= Nout) {
      piece[i] = *reinterpret_cast<const uint4v*>(src);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < Nout) piece[i][j / 2] |= (uint32_t)src[j] << (16 * (j % 2));
    }
  }
}

// write_tile16_staged with the epilogue: the residual's pieces go into the
// staging buffer (in accumulator order they would be 2-byte gathers), each
// lane adds its element to the float32 value and puts the bf16 result in the
// same place, and the tile leaves by row pieces. GATED: half the columns.
template <int MT, int NT, int WM, int WN, bool GATED, int ACT, int RP>
__device__ __forceinline__ void write_tile16_act(const float4v (&acc)[MT][NT], int m0, int n0, int wm, int wn,
                                                 const EpiOut& o, const uint4v (&piece)[RP], uint16_t* lds) {
  constexpr int NW = WM * WN, R = WM * MT * 16, C = WN * NT * 16 / (GATED ? 2 : 1), P = StagedPitch<C>::P;
  const int lane = threadIdx.x & 63;
  const int no = GATED ? n0 / 2 : n0, Nout = GATED ? o.N / 2 : o.N;
  const bool res = o.e.residual != nullptr;
  if (res) {
#pragma unroll
    for (int i = 0; i < R * C / 8 / (64 * NW); ++i) {
      const int q = i * 64 * NW + threadIdx.x;
      *reinterpret_cast<uint4v*>(&lds[q / (C / 8) * P + (q % (C / 8)) * 8]) = piece[i];
    }
    __syncthreads();
  }
#pragma unroll
  for (int nt = 0; nt < NT; nt += GATED ? 2 : 1) {
    const int n = n0 + (wn * NT + nt) * 16 + (lane & 15);
    uint16_t* const p = &lds[(wm * MT * 16 + 4 * (lane >> 4)) * P + (wn * NT + nt) * 16 / (GATED ? 2 : 1) + (lane & 15)];
    // a column's residuals are read before its results are written: element by
    // element every read would wait for the write before it
    float4v r[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) r[mt][i] = res ? bf16_bits_to_f32(p[(mt * 16 + i) * P]) : 0.0f;
    const float b = o.bias_at(n);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float4v v;
      if (GATED) {
        v = o.gate(acc[mt][nt], acc[mt][GATED ? nt + 1 : nt], n);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = act_of<ACT>(o.alpha * acc[mt][nt][i] + b);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) p[(mt * 16 + i) * P] = (uint16_t)f32_to_bf16_bits(v[i] + r[mt][i]);
    }
  }
  __syncthreads();
  store_staged_tile<R, C, NW>(lds, o.M, Nout, m0, no, o.y, o.ldy);
}

template <int MT, int NT, int WM, int WN, int RP>
__device__ __forceinline__ void write_tile16_staged_fused(const float4v (&acc)[MT][NT], int m0, int n0, int wm, int wn,
                                                          const EpiOut& o, const uint4v (&piece)[RP], uint16_t* lds) {
#define FQL_ACT(GATED, ACT) write_tile16_act<MT, NT, WM, WN, GATED, ACT>(acc, m0, n0, wm, wn, o, piece, lds)
  switch (o.e.act) {  // once a tile, not once an element
    case kActRelu: return FQL_ACT(false, kActRelu);
    case kActGelu: return FQL_ACT(false, kActGelu);
    case kActGeluTanh: return FQL_ACT(false, kActGeluTanh);
    case kActSilu: return FQL_ACT(false, kActSilu);
    case kActSwiglu: return FQL_ACT(true, kActSwiglu);
    default: return FQL_ACT(false, kActNone);
  }
#undef FQL_ACT
}

}  // namespace fql
