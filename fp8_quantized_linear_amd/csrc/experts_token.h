// The experts' feed forward of a few tokens (gfx950), two launches: every pair (token,
// place) for itself, straight from the router's choice. Nothing is sorted, and nothing
// goes through LDS but sums and a wave's own codes: a wave reads its weight tiles into
// registers in the packed order, which is the matrix instruction's; all 16 rows of the
// instruction are the pair's one row. Bound by the weights and the chain of a launch, the
// loads and the join: one token of 8 in 64 experts (2048, 1024 inner, block FP8, 50 MB of
// weights) takes 15.5 us a call where the sorted way takes 27.9; traced up 7.9 and down 6.8,
// 3.4 TB/s together (FP8 7.7 and 6.7, MXFP8 8.1 and 7.2, MXFP4 5.8 and 6.4, INT8, whose waves
// read the whole row for its scale, 9.1 and 7.4).
#pragma once

#include "experts_tile.h"

namespace fql {
namespace {

// Four chunks of an activation row as a wave holds them: lane l the values 8 l .. 8 l + 7.
template <typename X>
struct RawRow {
  uint4v q[sizeof(X) / 2];
};

// No branch: behind K (a multiple of 8) the row's start is read, and dropped later.
template <typename X>
__device__ __forceinline__ RawRow<X> load_row(const X* __restrict__ row, int64_t K, int64_t c) {
  const int64_t k = c * 128 + (threadIdx.x & 63) * 8;
  RawRow<X> raw;
  __builtin_memcpy(&raw, row + (k < K ? k : 0), sizeof(raw));  // x may have any alignment
  return raw;
}

// Their codes in the wave's own place in LDS, in the order of k. E: E8M0 byte of the
// lane's 32-block (MX) or scale of its chunk (block FP8). r: the row's factor (FP8, INT8).
template <int F, typename X>
__device__ __forceinline__ uint32_t quant_row(const RawRow<X>& raw, int64_t K, int64_t c, float r, uint8_t* codes) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63;
  const bool live = c * 128 + lane * 8 < K;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (sizeof(X) == 4) {
      v[j] = __uint_as_float(live ? raw.q[j / 4][j % 4] : 0u);
    } else {
      const uint32_t u = raw.q[0][j / 2];
      v[j] = __uint_as_float(live ? (j % 2 ? u & 0xFFFF0000u : u << 16) : 0u);
    }
  }
  uint32_t out = 0u;
  float f = r;
  if constexpr (F == SC_MXFP4 || F == SC_MXFP8 || F == SC_FP8_BLOCK) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = __builtin_fmaxf(a, __builtin_fabsf(v[j]));
    a = __builtin_fmaxf(a, __shfl_xor(a, 1));
    a = __builtin_fmaxf(a, __shfl_xor(a, 2));
    if constexpr (F == SC_FP8_BLOCK) {
      a = __builtin_fmaxf(a, __shfl_xor(a, 4));
      a = __builtin_fmaxf(a, __shfl_xor(a, 8));
      const float s = a / 448.0f;
      f = safe_reciprocal(s);
      out = __float_as_uint(s);
    } else {
      const int e = mx_exponent(a, F == SC_MXFP4 ? 2 : 8);
      f = pow2_neg(e);
      out = (uint32_t)(e + 127);
    }
  }
  if constexpr (F == SC_MXFP4) {
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0] * f, v[1] * f, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * f, v[3] * f, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * f, v[5] * f, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * f, v[7] * f, 1.0f, 3);
    reinterpret_cast<uint32_t*>(codes)[lane] = w;
  } else {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (F == SC_INT8) w[j] = int8x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], f);
      else w[j] = fp8x4(v[4 * j] * f, v[4 * j + 1] * f, v[4 * j + 2] * f, v[4 * j + 3] * f);
    }
    reinterpret_cast<uint64_t*>(codes)[lane] = (uint64_t)w[1] << 32 | w[0];
  }
  return out;
}

// INT8: the scale of a row (every lane of the wave calls it and gets it).
template <typename X>
__device__ __forceinline__ float row_scale(const X* __restrict__ row, int64_t K) {
  uint32_t top = 0u;
  for (int64_t k = (threadIdx.x & 63) * 16; k < K; k += 1024) {
    X v[16];
    __builtin_memcpy(v, row + k, sizeof(v));
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if constexpr (sizeof(X) == 4) top = amax_bits(v[j], top);
      else top = amax_bits(bf16_bits_to_f32(v[j]), top);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t u = (uint32_t)__shfl_xor((int)top, o);
    top = u > top ? u : top;
  }
  return int8_scale(top);
}

// One row times NT column tiles of an expert over chunks [c0, c1): sums of the lane's
// column (lane % 16) of each tile, every row of the instruction being the one. Four
// chunks are in flight together, the row's before the weights': it is quantized, by all
// lanes once, while the weights come (each lane loading and quantizing its operand
// for itself took 6 us more for the token above). No branch but the loop, so
// that nothing is loaded late. codes: 512 bytes of LDS of the wave's own.
template <int F, int NT, typename X>
__device__ __forceinline__ void row_product(const X* __restrict__ row, int64_t K, float r, const uint8_t* __restrict__ wcodes,
                                            const uint8_t* __restrict__ wscales, int tile0, const ProductArgs& g, int64_t c0,
                                            int64_t c1, uint8_t* codes, float4v (&acc)[NT]) {
  typedef Traits<F> T;
  constexpr int H = T::H, U = 4;
  const int lane = threadIdx.x & 63, kg = lane >> 4;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt] = float4v{0.f, 0.f, 0.f, 0.f};
  int tile[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) tile[nt] = tile0 + nt < g.ntiles_w ? tile0 + nt : 0;  // past N: not stored
  for (int64_t cb = c0; cb < c1; cb += U) {
    const RawRow<X> raw = load_row(row, K, cb);
    uint4v b[U][NT][H];
    uint32_t ws[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = cb + u < c1 ? cb + u : c1 - 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < H; ++h)
          b[u][nt][h] = *reinterpret_cast<const uint4v*>(wcodes + ((int64_t)tile[nt] * g.KC + c) * (1024 * H) + h * 1024 + lane * 16);
        ws[u][nt] = 0u;
        if constexpr (T::MX)
          ws[u][nt] = *reinterpret_cast<const uint32_t*>(wscales + ((int64_t)(tile[nt] / 4) * g.KC + c) * 256 + lane * 4);
        else if constexpr (T::BLOCK)
          ws[u][nt] = *reinterpret_cast<const uint32_t*>(wscales + ((int64_t)(tile[nt] / 8) * g.KC + c) * 4);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_wave_barrier();  // a wave's LDS operations keep their order
    const uint32_t scale = quant_row<F>(raw, K, cb, r, codes);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = cb + u < c1;
      uint4v a0, a1 = uint4v{0u, 0u, 0u, 0u};
      if constexpr (H == 1) {
        a0 = *reinterpret_cast<const uint4v*>(codes + u * 64 + kg * 16);
      } else {
        a0 = *reinterpret_cast<const uint4v*>(codes + u * 128 + kg * 16);
        a1 = *reinterpret_cast<const uint4v*>(codes + u * 128 + 64 + kg * 16);
      }
      const int8v a = int8v{(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
      int sa = 127;
      float gs = 0.0f;
      if constexpr (T::MX) sa = __shfl((int)scale, u * 16 + kg * 4);
      if constexpr (T::BLOCK) gs = __uint_as_float(__builtin_amdgcn_readlane(scale, u * 16));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4v q0 = b[u][nt][0], q1 = b[u][nt][H - 1];
        float4v sum;
        if constexpr (T::INT) {
          int4v s = __builtin_bit_cast(int4v, acc[nt]);
          s = __builtin_amdgcn_mfma_i32_16x16x64_i8(int4v{a[0], a[1], a[2], a[3]}, __builtin_bit_cast(int4v, q0), s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_i32_16x16x64_i8(int4v{a[4], a[5], a[6], a[7]}, __builtin_bit_cast(int4v, q1), s, 0, 0, 0);
          sum = __builtin_bit_cast(float4v, s);
        } else {
          int8v w = int8v{(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, 0, 0, 0, 0};
          if (H == 2) w = int8v{(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, (int)q1.x, (int)q1.y, (int)q1.z, (int)q1.w};
          if constexpr (T::BLOCK) {
            const float4v z = float4v{0.f, 0.f, 0.f, 0.f};
            const float4v part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, w, z, 0, 0, 0, 127, 0, 127);
            sum = acc[nt] + part * (gs * __uint_as_float(ws[u][nt]));
          } else {
            const int sb = T::MX ? (int)((ws[u][nt] >> (8 * (tile[nt] % 4))) & 0xFFu) : 127;
            sum = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, w, acc[nt], T::FMT, T::FMT, 0, sa, 0, sb);
          }
        }
        acc[nt].x = live ? sum.x : acc[nt].x;  // all four rows a lane holds are the one row
      }
    }
  }
}

// The lane's column's sum as float32 (INT8: times the scales).
template <int F>
__device__ __forceinline__ float finished(float s, float row, const uint8_t* wscales, int n) {
  if constexpr (F == SC_INT8) return int8_value((int)__float_as_uint(s), row, reinterpret_cast<const float*>(wscales)[n]);
  else return s;
}

// Up: workgroup (32 columns, pair), its four waves a quarter of K each. h [pair][ld] float32.
template <int F>
__global__ __launch_bounds__(256, 2) void experts_token_up_kernel(const uint16_t* __restrict__ x, int64_t ldx, float inv_scale, int64_t K, const int32_t* __restrict__ experts,
                                                               int E, const ProductArgs g, float* __restrict__ h) {
  __shared__ float red[4][2][16];
  __shared__ __align__(16) uint8_t codes[4][512];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = blockIdx.y, e = experts[pair];
  if (e < 0 || e >= E) return;
  const uint16_t* const row = x + (int64_t)(pair / g.k) * ldx;
  const uint8_t* const wcodes = g.packed + e * g.stride;
  const uint8_t* const wscales = wcodes + g.code_bytes;
  const int tile0 = blockIdx.x * 2;
  const int64_t per = (g.KC + 3) / 4, c0 = wave * per < g.KC ? wave * per : g.KC, c1 = c0 + per < g.KC ? c0 + per : g.KC;
  float s = 0.0f, r = inv_scale;
  if constexpr (F == SC_INT8) {
    s = row_scale(row, K);
    r = safe_reciprocal(s);
  }
  float4v acc[2];
  row_product<F, 2>(row, K, r, wcodes, wscales, tile0, g, c0, c1, codes[wave], acc);
  if (lane < 16) {
    red[wave][0][lane] = acc[0][0];
    red[wave][1][lane] = acc[1][0];
  }
  __syncthreads();
  if (threadIdx.x >= 16) return;
  const float alpha = g.alpha != nullptr ? g.alpha[e] : 1.0f;
  float z[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    float sum = red[0][t][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      if constexpr (F == SC_INT8) sum = __uint_as_float(__float_as_uint(sum) + __float_as_uint(red[w][t][lane]));
      else sum += red[w][t][lane];
    }
    const int n = (tile0 + t) * 16 + lane;
    z[t] = 0.0f;
    if (n < g.N)
      z[t] = alpha * finished<F>(sum, s, wscales, n) +
             (g.bias != nullptr ? bf16_bits_to_f32(g.bias[(int64_t)e * g.N + n]) : 0.0f);
  }
  float* const out = h + (int64_t)pair * g.ld_out;
  if (g.act == kActSwiglu) {
    if (tile0 * 16 < g.N) out[blockIdx.x * 16 + lane] = z_sigmoid(z[0], z[0]) * z[1];
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if ((tile0 + t) * 16 + lane < g.N) out[(tile0 + t) * 16 + lane] = apply_act(z[t], g.act);
  }
}

// Down: workgroup (16 columns, token), 16 waves that share the token's k rows times
// `parts` ranges of K; the sum of the places in their order. y_t = bf16(residual_t +
// sum_j w_tj d_j), d in float32.
constexpr int kTokenItems = 64;  // k <= 64 places, or fewer than 17 in parts
template <int F>
__global__ __launch_bounds__(1024) void experts_token_down_kernel(const float* __restrict__ h, int64_t ldh, float inv_scale,
                                                                 int64_t K, const int32_t* __restrict__ experts,
                                                                 const float* __restrict__ weights, int E, int parts,
                                                                 const ProductArgs g, const uint16_t* residual, int64_t ldr,
                                                                 uint16_t* y, int64_t ldy) {
  __shared__ float red[kTokenItems][16];
  __shared__ __align__(16) uint8_t codes[16][512];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.y;
  const int tile0 = blockIdx.x;
  for (int item = wave; item < g.k * parts; item += 16) {
    const int j = item / parts, part = item - j * parts;
    const int64_t pair = t * g.k + j;
    const int e = __builtin_amdgcn_readfirstlane(experts[pair]);
    float v = 0.0f;
    if (e >= 0 && e < E) {
      const float* const row = h + pair * ldh;
      const uint8_t* const wcodes = g.packed + e * g.stride;
      const uint8_t* const wscales = wcodes + g.code_bytes;
      const int64_t per = (g.KC + parts - 1) / parts, c0 = part * per < g.KC ? part * per : g.KC;
      const int64_t c1 = c0 + per < g.KC ? c0 + per : g.KC;
      float s = 0.0f, r = inv_scale;
      if constexpr (F == SC_INT8) {
        s = row_scale(row, K);
        r = safe_reciprocal(s);
      }
      float4v acc[1];
      row_product<F, 1>(row, K, r, wcodes, wscales, tile0, g, c0, c1, codes[wave], acc);
      const int n = tile0 * 16 + (lane & 15);
      v = (g.alpha != nullptr ? g.alpha[e] : 1.0f) * finished<F>(acc[0][0], s, wscales, n);
      if (part == 0 && g.bias != nullptr && n < g.N) v += bf16_bits_to_f32(g.bias[(int64_t)e * g.N + n]);
    }
    if (lane < 16) red[item][lane] = v;
  }
  __syncthreads();
  const int n = tile0 * 16 + lane;
  if (threadIdx.x >= 16 || n >= g.N) return;
  float sum = residual != nullptr ? bf16_bits_to_f32(residual[t * ldr + n]) : 0.0f;
  for (int j = 0; j < g.k; ++j) {
    const int e = experts[t * g.k + j];
    if (e < 0 || e >= E) continue;
    float d = 0.0f;
    for (int p = 0; p < parts; ++p) d += red[j * parts + p][lane];
    sum = __builtin_fmaf(weights[t * g.k + j], d, sum);
  }
  y[t * ldy + n] = (uint16_t)f32_to_bf16_bits(sum);
}

}  // namespace
}  // namespace fql
