// Residual addition + root-mean-square norm + 8-bit quantizer, one pass
// (gfx950): the input of an 8-bit linear layer straight from the residual
// stream.
//
//   h = x + residual                       (float32; written back as bf16)
//   y = h * (1 / sqrt(mean(h^2) + eps)) * w
//   codes, scales = the linear layers' quantizer on y (per-tensor FP8, block
//   FP8 or MXFP8; quant_block8 below)
//
// Roundings: h is rounded to bf16 only where it is stored; the norm and the
// quantizer take the unrounded float32 sum. The sum of squares and the row's
// factor 1 / sqrt(..) are float64 (block FP8: float32 while they stay well inside
// its range), y is float32. Where the codes of FP8 and MXFP8 could differ for a
// y off by its rounding, they are made again from float64 (exact_codes): an MXFP8
// code carries one rounding, its own, an FP8 code that of fl32(1 / scale) besides.
// The codes of block FP8 are those of the float32 y over the float32 scale.
//
// A y that is not a number (a NaN or infinity in its row, 0 / 0 in an all-zero
// row under eps = 0) has a NaN code, and does not count for its block's scale.
#include <type_traits>

#include "fql_device.h"
#include "fql_serving.h"
#include "sc_quant.h"

namespace fql {

namespace {

// Eight consecutive values of a row.
struct Vec8 {
  float v[8];
};
__device__ __forceinline__ uint4v load_raw8(const uint16_t* p, bool aligned) {
  if (aligned) return *reinterpret_cast<const uint4v*>(p);
  uint4v u;
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
  return u;
}
__device__ __forceinline__ Vec8 widen(const uint4v& u) {
  Vec8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.v[2 * j] = __uint_as_float(u[j] << 16);
    r.v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
  return r;
}
__device__ __forceinline__ Vec8 load8(const uint16_t* p, bool aligned) { return widen(load_raw8(p, aligned)); }
__device__ __forceinline__ void store8(uint16_t* p, const Vec8& r, bool aligned) {
  if (aligned) {
    uint4v u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = f32_to_bf16_bits(r.v[2 * j]) | (f32_to_bf16_bits(r.v[2 * j + 1]) << 16);
    *reinterpret_cast<uint4v*>(p) = u;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = (uint16_t)f32_to_bf16_bits(r.v[j]);
  }
}

// Four float32 -> four E4M3 bytes; NaN stays NaN. minimum and maximum hand it
// on and cost what fp8x4's fmin and fmax do, which make it -448.
__device__ __forceinline__ float clamp_nan(float v) {
  return __builtin_elementwise_maximum(__builtin_elementwise_minimum(v, 448.0f), -448.0f);
}
__device__ __forceinline__ uint32_t fp8x4_nan(float a, float b, float c, float d) {
  short2v o = {0, 0};
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, clamp_nan(a), clamp_nan(b), 1.0f, false);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, clamp_nan(c), clamp_nan(d), 1.0f, true);
  return __builtin_bit_cast(uint32_t, o);
}

// 2^e-scaled or plain quotient d -> float32, rounded to odd: the E4M3 rounding
// of the result is that of d itself (float32 has more than two bits more).
__device__ __forceinline__ float round_to_odd(double d) {
  const float t = (float)d;
  uint32_t b = __float_as_uint(t);
  const double back = (double)t;
  if (back == d || d != d) return t;
  if (__builtin_fabs(back) > __builtin_fabs(d)) b -= 1u;
  return __uint_as_float(b | 1u);
}

// Codes of eight values h * rinv * w * f from float64, where those of the
// float32 product (off by at most 4 roundings, 2^-22) are not sure: one vector
// in some ten thousand.
__device__ __forceinline__ void exact_codes(const Vec8& h, const Vec8& wt, double rinv, const Vec8& y, float f,
                                            uint32_t w[2]) {
#pragma clang fp contract(off)
  const float lo = f * (1.0f - 0x1p-21f), hi = f * (1.0f + 0x1p-21f);
  uint32_t differ = 0u;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    differ |= fp8x4_nan(y.v[4 * j] * lo, y.v[4 * j + 1] * lo, y.v[4 * j + 2] * lo, y.v[4 * j + 3] * lo) ^
              fp8x4_nan(y.v[4 * j] * hi, y.v[4 * j + 1] * hi, y.v[4 * j + 2] * hi, y.v[4 * j + 3] * hi);
  if (differ == 0u) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u = h.v[4 * j + i];
      __asm__("" : "+v"(u));  // converted here: kept from the sum of squares, its float64 would spill
      c[i] = round_to_odd((double)u * rinv * (double)wt.v[4 * j + i] * (double)f);
    }
    w[j] = fp8x4_nan(c[0], c[1], c[2], c[3]);
  }
}

// Codes of eight consecutive values (two words) and the scale of their block.
// A block of 32 (MXFP8) or 128 (block FP8) values is held by 4 or 16
// neighbouring lanes, all of which must call this.
template <int F>
__device__ __forceinline__ void quant_block8(const Vec8& y, float inv_scale, uint32_t w[2], uint32_t& sbyte,
                                             float& gscale, float& f) {
#pragma clang fp contract(off)
  f = inv_scale;
  if (F != SC_FP8) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = __builtin_fmaxf(a, __builtin_fabsf(y.v[j]));
    a = __builtin_fmaxf(a, __shfl_xor(a, 1));
    a = __builtin_fmaxf(a, __shfl_xor(a, 2));
    if (F == SC_FP8_BLOCK) {
      a = __builtin_fmaxf(a, __shfl_xor(a, 4));
      a = __builtin_fmaxf(a, __shfl_xor(a, 8));
      gscale = a / 448.0f;
      f = safe_reciprocal(gscale);
    } else {
      const int e = mx_exponent(a, 8);
      sbyte = (uint32_t)(e + 127);
      f = pow2_neg(e);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    w[j] = fp8x4_nan(y.v[4 * j] * f, y.v[4 * j + 1] * f, y.v[4 * j + 2] * f, y.v[4 * j + 3] * f);
}

// Row-independent addressing of one workgroup's row.
struct NormFlags {
  bool x, r, w, h;  // 16-byte aligned rows
};

// Where the eight codes of columns 8v .. 8v+7 of row m go, with their scale.
template <int F, bool OP>
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t m, int64_t v, const uint32_t w[2],
                                            uint32_t sbyte, float gscale) {
  const int64_t k = 8 * v;
  uint64_t word = (uint64_t)w[0] | ((uint64_t)w[1] << 32);
  if (!OP) {
    *reinterpret_cast<uint64_t*>(a.codes + m * a.K + k) = word;
    if (F == SC_MXFP8 && (v & 3) == 0) static_cast<uint8_t*>(a.scales)[m * (a.K / 32) + k / 32] = (uint8_t)sbyte;
    if (F == SC_FP8_BLOCK && (v & 15) == 0) static_cast<float*>(a.scales)[m * (a.K / 128) + k / 128] = gscale;
  } else {
    // 16-element piece h16 of chunk c: half h16 / 4, lane (h16 % 4) * 16 + m % 16
    const int64_t KC = (a.K + 127) / 128, c = k / 128, tile = m / 16, quad = m / 64;
    const int r = (int)(m % 16), h16 = (int)(k % 128) / 16;
    uint8_t* dst = a.codes + (tile * KC + c) * 2048 + (h16 / 4) * 1024 + ((h16 % 4) * 16 + r) * 16 + k % 16;
    *reinterpret_cast<uint64_t*>(dst) = word;
    if (F == SC_MXFP8 && (v & 3) == 0)
      static_cast<uint8_t*>(a.scales)[((quad * KC + c) * 64 + (h16 / 2) * 16 + r) * 4 + (int)(m / 16) % 4] =
          (uint8_t)sbyte;
    if (F == SC_FP8_BLOCK && (v & 15) == 0) static_cast<float*>(a.scales)[(quad * KC + c) * 64 + m % 64] = gscale;
  }
}

// h = x + residual of one vector, stored back where there is a residual.
__device__ __forceinline__ Vec8 load_h(const NormArgs& a, const NormFlags& f, int64_t m, int64_t v, bool store) {
  Vec8 h = load8(a.x + m * a.ldx + 8 * v, f.x);
  if (a.residual != nullptr) {
    const Vec8 r = load8(a.residual + m * a.ldr + 8 * v, f.r);
#pragma unroll
    for (int j = 0; j < 8; ++j) h.v[j] += r.v[j];
    if (store && a.h != nullptr) store8(a.h + m * a.ldh + 8 * v, h, f.h);
  }
  return h;
}

// h and the weight are zeros past the row.
template <int F, bool OP>
__device__ __forceinline__ void finish_vec(const NormArgs& a, int64_t m, int64_t v, int64_t nv, int64_t nvp,
                                           const Vec8& h, const Vec8& w, double rinv) {
#pragma clang fp contract(off)
  Vec8 y;
  const float r = (float)rinv;
#pragma unroll
  for (int j = 0; j < 8; ++j) y.v[j] = v < nv ? h.v[j] * r * w.v[j] : 0.0f;
  uint32_t q[2], sb = 0;
  float gs = 0.0f, factor;
  quant_block8<F>(y, a.inv_scale, q, sb, gs, factor);
  if (F != SC_FP8_BLOCK) exact_codes(h, w, rinv, y, factor, q);
  if (OP && v >= nv) sb = 0;  // padding up to the chunk: zero codes, zero scale bytes
  if (v < (OP ? nvp : nv)) store_codes<F, OP>(a, m, v, q, sb, gs);
}

// One row per workgroup (WAVE: per wave, four rows a workgroup), its values in
// registers: vector v = t + T * i of thread t (T threads a row, I vectors a
// thread). STREAM: rows too long for that read x and the residual twice.
//
// Bound by memory where there are many rows: 8192 x 5120 block FP8 with a
// residual moves 294 MB in 54 to 58 us, 5.1 TB/s, what a large copy reaches (with
// the exact codes MXFP8 takes 60.5 us, FP8 61 to 67; into the operand, whose 16-byte
// pieces L2 joins, block FP8 63.5, FP8 65, MXFP8 70). Few rows are one dependent
// chain (load, reduce, barrier, encode): one row of 4096 takes 3.8 us, 333 x 5120
// MXFP8 7.9 us (two vectors a thread, so that one row's chain is short and its
// loads are all in flight at once).
template <int F, bool OP, int I, bool WAVE, bool STREAM>
__global__ __launch_bounds__(1024) void rms_norm_quant_kernel(const NormArgs a, const NormFlags f) {
  __shared__ double red[16];
  __shared__ float red32[16];
  int64_t m;
  int t, T;
  if (WAVE) {
    m = (int64_t)blockIdx.x * (blockDim.x / 64) + threadIdx.x / 64;
    t = threadIdx.x & 63;
    T = 64;
    if (m >= a.M) return;
  } else {
    m = blockIdx.x;
    // The operand interleaves 16 rows in every 256-byte run, so a row's stores
    // are 16-byte pieces. The workgroups of one 16-row tile are placed on one
    // XCD (workgroups go to the eight XCDs in turn), whose L2 then joins the
    // pieces into whole lines.
    if (OP) m = ((m / 128) * 8 + m % 8) * 16 + (m / 8) % 16;
    t = threadIdx.x;
    T = blockDim.x;
    if (m >= a.M) return;
  }
  const int64_t nv = a.K / 8, nvp = OP ? (a.K + 127) / 128 * 16 : nv;
  // the weight's loads run beside the sum of squares where registers allow it
  // (an access less in the chain: 8 x 4096 FP8 5.8 -> 5.4 us, 8192 x 5120 block
  // FP8 59.4 -> 58.3)
  constexpr bool EARLY = !STREAM && I <= 4;
  auto load_w = [&](int64_t v) { return v < nv ? load_raw8(a.weight + 8 * v, f.w) : uint4v{0u, 0u, 0u, 0u}; };
  uint4v w[EARLY ? I : 1];
  Vec8 h[I];
  if (!STREAM) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t v = t + (int64_t)T * i;
      if (EARLY) w[i] = load_w(v);
      if (v < nv) h[i] = load_h(a, f, m, v, true);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i].v[j] = 0.0f;
    }
  }
  // the row's sum of squares in the type of `ss`
  auto squares = [&](auto ss, auto* red) {
    typedef decltype(ss) Sum;
    if (!STREAM) {
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += (Sum)h[i].v[j] * (Sum)h[i].v[j];
    } else {
      for (int64_t v = t; v < nv; v += T) {
        const Vec8 u = load_h(a, f, m, v, false);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += (Sum)u.v[j] * (Sum)u.v[j];
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
    if (!WAVE) {
      if ((t & 63) == 0) red[t >> 6] = ss;
      __syncthreads();
      ss = (Sum)0;
      for (int i = 0; i < T / 64; ++i) ss += red[i];
    }
    return ss;
  };
  float shift = 1.0f;
  auto factor64 = [&]() {
    double r = 1.0 / __builtin_sqrt(squares(0.0, red) / (double)a.K + (double)a.eps);
    // rows of magnitude 1e38 (under eps = 0 also 1e-39), whose factor is no normal
    // float32: a power of two goes from it into the row, which changes no y
    if (!(r >= 0x1p-126 && r <= 0x1p127)) {
      shift = r > 1.0 ? 0x1p64f : 0x1p-64f;
      r /= (double)shift;
      if (!STREAM)
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i].v[j] *= shift;
    }
    return r;
  };
  // Block FP8, whose codes are those of a float32 y, sums in float32 and again in
  // float64 where the squares leave float32's range (float64 at once takes 8192 x
  // 5120 from 56 to 57.5 us).
  std::conditional_t<F == SC_FP8_BLOCK, float, double> rinv;
  if constexpr (F == SC_FP8_BLOCK) {
    const float ss = squares(0.0f, red32);
    rinv = 1.0f / __builtin_sqrtf(ss / (float)a.K + a.eps);
    if (!(ss >= 0x1p-100f && ss <= 0x1p126f)) rinv = (float)factor64();
  } else {
    rinv = factor64();
  }
  if (!STREAM) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      // whole groups of T vectors, so that every lane of a block takes part
      const int64_t v = t + (int64_t)T * i;
      if ((int64_t)T * i < nvp) finish_vec<F, OP>(a, m, v, nv, nvp, h[i], widen(EARLY ? w[i] : load_w(v)), rinv);
    }
  } else {
    for (int64_t v0 = 0; v0 < nvp; v0 += T) {
      const int64_t v = v0 + t;
      Vec8 u;
#pragma unroll
      for (int j = 0; j < 8; ++j) u.v[j] = 0.0f;
      if (v < nv) u = load_h(a, f, m, v, true);
#pragma unroll
      for (int j = 0; j < 8; ++j) u.v[j] *= shift;
      finish_vec<F, OP>(a, m, v, nv, nvp, u, widen(load_w(v)), rinv);
    }
  }
}

bool row_aligned(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

template <int F, bool OP>
hipError_t launch_t(const NormArgs& a, hipStream_t st) {
  const NormFlags f = {row_aligned(a.x, a.ldx), row_aligned(a.residual, a.ldr), row_aligned(a.weight, 0),
                       row_aligned(a.h, a.ldh)};
  const int64_t nv = OP ? (a.K + 127) / 128 * 16 : a.K / 8;
#define FQL_LAUNCH(I, W, S, grid, threads) \
  rms_norm_quant_kernel<F, OP, I, W, S><<<(unsigned)(grid), (unsigned)(threads), 0, st>>>(a, f)
  if (nv <= 128 && a.M > 1) {
    FQL_LAUNCH(2, true, false, (a.M + 3) / 4, 256);
    return hipGetLastError();
  }
  const int64_t rows = OP ? round_up(a.M, 128) : a.M;
  const int64_t per = nv <= 1024 ? 2 : nv <= 2048 ? 4 : 8;  // vectors a thread
  const int64_t threads = round_up((nv + per - 1) / per, 64);
  if (nv > 8192) FQL_LAUNCH(1, false, true, rows, 1024);
  else if (per == 2) FQL_LAUNCH(2, false, false, rows, threads);
  else if (per == 4) FQL_LAUNCH(4, false, false, rows, threads);
  else FQL_LAUNCH(8, false, false, rows, threads);
#undef FQL_LAUNCH
  return hipGetLastError();
}

// The formats' activation quantizer straight into an operand: one wave a
// 16-row tile and 128-deep chunk, lane 16 kg + r the 32-block kg of row r. The
// operand interleaves 16 rows in runs of 256 bytes, so in this order every
// store instruction fills whole runs; with a row's blocks in neighbouring
// lanes (the standalone quantizer's order) they are 16-byte pieces 256 bytes
// apart. The block arithmetic is quant_block32's. Rows past M are not written.
// 4096 x 4096 MXFP8: 10 us, 4.9 TB/s (15.9 us in the quantizer's order). It has
// the name of the plain linear call's operand quantizer: launch plans name it.
template <int F>
__global__ __launch_bounds__(256) void sc_quant_operand_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                            int64_t ldx, bool aligned, float inv_scale, int64_t KC,
                                                            int64_t waves, uint8_t* __restrict__ codes,
                                                            void* __restrict__ scales) {
  constexpr int H = F == SC_MXFP4 ? 1 : 2;
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w >= waves) return;
  const int lane = threadIdx.x & 63, r = lane & 15, kg = lane >> 4;
  const int64_t tile = w / KC, c = w - tile * KC, m = tile * 16 + r, b = 4 * c + kg;
  const bool valid = m < M && b * 32 < K;
  float v[32];
  if (valid) load32(x + m * ldx + b * 32, aligned, v);
  else
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
  uint32_t q[8], sb = 0;
  float gs = 0.0f;
  if (F == SC_FP8_BLOCK) {
    float a = amax32(v);
    a = __builtin_fmaxf(a, __shfl_xor(a, 16));
    a = __builtin_fmaxf(a, __shfl_xor(a, 32));
    gs = a / 448.0f;
    encode_fp8x32(v, safe_reciprocal(gs), q);
  } else {
    quant_block32<F>(v, valid, inv_scale, q, sb, gs);
  }
  if (m >= M) return;
  if (!valid) {  // past K: zero codes, zero scale bytes
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = 0u;
    sb = 0;
  }
  uint8_t* const base = codes + w * (H * 1024);
  if (F == SC_MXFP4) {
    *reinterpret_cast<uint4v*>(base + lane * 16) = uint4v{q[0], q[1], q[2], q[3]};
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h16 = 2 * kg + j;
      *reinterpret_cast<uint4v*>(base + (h16 / 4) * 1024 + ((h16 % 4) * 16 + r) * 16) =
          uint4v{q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]};
    }
  }
  const int64_t quad = m / 64;
  if (F == SC_MXFP4 || F == SC_MXFP8)
    static_cast<uint8_t*>(scales)[((quad * KC + c) * 64 + lane) * 4 + (int)(tile % 4)] = (uint8_t)sb;
  if (F == SC_FP8_BLOCK && kg == 0) static_cast<float*>(scales)[(quad * KC + c) * 64 + m % 64] = gs;
}

}  // namespace

hipError_t launch_quant_operand(int fmt, const uint16_t* x, int64_t M, int64_t K, int64_t ldx, bool aligned,
                                float inv_scale, uint8_t* codes, void* scales, hipStream_t st) {
  if (fmt == SC_INT8) return launch_int8_quant(false, true, x, M, K, ldx, codes, static_cast<float*>(scales), st);
  const int64_t KC = (K + 127) / 128, waves = (M + 15) / 16 * KC;
  const unsigned grid = (unsigned)((waves + 3) / 4);
#define FQL_Q(F)                                                                                                   \
  if (fmt == F) {                                                                                                  \
    sc_quant_operand_kernel<F><<<grid, 256, 0, st>>>(x, M, K, ldx, aligned, inv_scale, KC, waves, codes, scales);  \
    return hipGetLastError();                                                                                      \
  }
  FQL_Q(SC_MXFP4) FQL_Q(SC_MXFP8) FQL_Q(SC_FP8) FQL_Q(SC_FP8_BLOCK)
#undef FQL_Q
  return hipErrorInvalidValue;
}

hipError_t launch_rms_norm_quant(int fmt, bool operand, const NormArgs& a, hipStream_t st) {
  if (fmt == SC_INT8) return operand ? launch_rms_norm_int8(a, st) : hipErrorInvalidValue;
#define FQL_F(F) \
  if (fmt == F) return operand ? launch_t<F, true>(a, st) : launch_t<F, false>(a, st);
  FQL_F(SC_FP8) FQL_F(SC_FP8_BLOCK) FQL_F(SC_MXFP8)
#undef FQL_F
  return hipErrorInvalidValue;
}

}  // namespace fql
