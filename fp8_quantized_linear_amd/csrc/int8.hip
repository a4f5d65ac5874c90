// INT8 rows (gfx950): one float32 scale a token (or a weight's channel),
//
//   s = fl32(max|v| / 127),  code = rint(fl32(v * fl32(1 / s))), ties to even
//
// of a bf16 or float32 matrix, or of the residual addition and root-mean-square
// norm in front of a linear layer:
//
//   h = x + residual                       (float32; written back as bf16)
//   y = h * (1 / sqrt(mean(h^2) + eps)) * w
//
// The scale needs the whole row before its first code, so a row stays in one
// workgroup's registers between the two. The sum of squares, the row's factor and
// the product y are float64, y is rounded to float32 once and quantized from that.
// A row with a value that is not a number or not finite has scale NaN: integers
// cannot hold it, and the outputs of the row's product become NaN.
//
// Bound by memory, and for rows into an operand by its 16-byte pieces: 4096 x 4096 into the
// operand 12.3 us (50 MB, 4.1 TB/s; the FP8 quantizers, which take 16 rows a wave in the
// operand's order, 9.5), into plain codes 10.5 traced; the norm with a residual into the
// operand 8192 x 5120 89 us (294 MB, 3.3 TB/s; block FP8's 64, the bytes alone 59), 4096 x 4096
// 30 (block FP8's 27, the bytes 24).
#include "fql_device.h"
#include "fql_serving.h"
#include "sc_quant.h"

namespace fql {

namespace {

struct Int8Args {
  const void* x;  // [M][ldx] bf16 or float32
  int64_t M, K, ldx;
  uint8_t* codes;  // [M][K], or the operand's
  float* scales;   // [M]
  const uint16_t* residual;  // norm: bf16 [M][ldr] or null
  int64_t ldr;
  const uint16_t* weight;  // norm: bf16 [K]
  double eps;
  uint16_t* h;  // norm: bf16 [M][ldh] or null
  int64_t ldh;
  bool ax, ar, aw, ah;  // 16-byte aligned rows
};

struct Row8 {
  float v[8];
};
__device__ __forceinline__ Row8 row8(const uint16_t* p, bool aligned) {
  Row8 r;
  if (aligned) {
    const uint4v u = *reinterpret_cast<const uint4v*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.v[2 * j] = __uint_as_float(u[j] << 16);
      r.v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = bf16_bits_to_f32(p[j]);
  }
  return r;
}
__device__ __forceinline__ Row8 row8(const float* p, bool aligned) {
  Row8 r;
  if (aligned) {
    const float4v a = *reinterpret_cast<const float4v*>(p), b = *reinterpret_cast<const float4v*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.v[j] = a[j];
      r.v[4 + j] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = p[j];
  }
  return r;
}

// One row a workgroup: vector v = t + T i of thread t (T threads, I vectors of
// eight a thread). STREAM: rows too long for the registers are read again for
// each of the two (norm: three) passes.
template <typename X, bool NORM, bool OP, int I, bool STREAM>
__global__ __launch_bounds__(1024) void int8_row_kernel(const Int8Args a) {
  __shared__ double sums[16];
  __shared__ uint32_t tops[16];
  const int t = threadIdx.x, T = blockDim.x, waves = T / 64;
  int64_t m = blockIdx.x + ((int64_t)blockIdx.y << 20);
  // an operand's rows are 16-byte pieces, 16 rows in a run of 256 bytes: a tile's
  // workgroups are placed on one XCD (they go to the eight in turn), whose L2 joins
  // the pieces
  if (OP) m = ((m / 128) * 8 + m % 8) * 16 + (m / 8) % 16;
  if (m >= a.M) return;
  const int64_t nv = a.K / 8, nvp = OP ? (a.K + 127) / 128 * 16 : nv;
  const X* const row = static_cast<const X*>(a.x) + m * a.ldx;
  Row8 zero;
#pragma unroll
  for (int j = 0; j < 8; ++j) zero.v[j] = 0.0f;
  auto load = [&](int64_t v, bool store) {
    Row8 h = row8(row + 8 * v, a.ax);
    if (NORM && a.residual != nullptr) {
      const Row8 r = row8(a.residual + m * a.ldr + 8 * v, a.ar);
#pragma unroll
      for (int j = 0; j < 8; ++j) h.v[j] += r.v[j];
      if (store && a.h != nullptr) {
        uint16_t* const p = a.h + m * a.ldh + 8 * v;
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = f32_to_bf16_bits(h.v[j]);
        if (a.ah) {
          *reinterpret_cast<uint4v*>(p) =
              uint4v{b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16};
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = (uint16_t)b[j];
        }
      }
    }
    return h;
  };
  Row8 h[STREAM ? 1 : I];
  if (!STREAM) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t v = t + (int64_t)T * i;
      h[i] = v < nv ? load(v, true) : zero;
    }
  }
  double rinv = 1.0;
  if (NORM) {
    double ss = 0.0;
    if (!STREAM) {
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += (double)h[i].v[j] * (double)h[i].v[j];
    } else {
      for (int64_t v = t; v < nv; v += T) {
        const Row8 u = load(v, false);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += (double)u.v[j] * (double)u.v[j];
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) ss += __shfl_xor(ss, o);
    if ((t & 63) == 0) sums[t >> 6] = ss;
    __syncthreads();
    ss = 0.0;
    for (int i = 0; i < waves; ++i) ss += sums[i];
    rinv = 1.0 / __builtin_sqrt(ss / (double)a.K + a.eps);
  }
  auto value = [&](const Row8& u, int64_t v) {
    if (!NORM) return u;
    const Row8 w = row8(a.weight + 8 * v, a.aw);
    Row8 y;
#pragma unroll
    for (int j = 0; j < 8; ++j) y.v[j] = (float)((double)u.v[j] * rinv * (double)w.v[j]);
    return y;
  };
  uint32_t top = 0u;
  if (!STREAM) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t v = t + (int64_t)T * i;
      if (v < nv) h[i] = value(h[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = amax_bits(h[i].v[j], top);
    }
  } else {
    for (int64_t v = t; v < nv; v += T) {
      const Row8 y = value(load(v, false), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = amax_bits(y.v[j], top);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t b = (uint32_t)__shfl_xor((int)top, o);
    top = b > top ? b : top;
  }
  if ((t & 63) == 0) tops[t >> 6] = top;
  __syncthreads();
  top = 0u;
  for (int i = 0; i < waves; ++i) top = tops[i] > top ? tops[i] : top;
  const float s = int8_scale(top), r = safe_reciprocal(s);
  if (t == 0) a.scales[m] = s;
  auto put = [&](int64_t v, const Row8& y) {
    if (v >= nvp) return;
    const int64_t k = 8 * v;
    const uint64_t word = (uint64_t)int8x4(y.v[0], y.v[1], y.v[2], y.v[3], r) |
                          ((uint64_t)int8x4(y.v[4], y.v[5], y.v[6], y.v[7], r) << 32);
    if (!OP) {
      *reinterpret_cast<uint64_t*>(a.codes + m * a.K + k) = word;
    } else {
      // 16-element piece h16 of chunk c: half h16 / 4, lane (h16 % 4) * 16 + m % 16
      const int64_t KC = (a.K + 127) / 128, c = k / 128;
      const int h16 = (int)(k % 128) / 16;
      *reinterpret_cast<uint64_t*>(a.codes + ((m / 16) * KC + c) * 2048 + (h16 / 4) * 1024 +
                                   ((h16 % 4) * 16 + (int)(m % 16)) * 16 + k % 16) = word;
    }
  };
  if (!STREAM) {
#pragma unroll
    for (int i = 0; i < I; ++i) put(t + (int64_t)T * i, h[i]);
  } else {
    // the residual stream goes out last: it may be x or the residual itself
    for (int64_t v = t; v < nvp; v += T) put(v, v < nv ? value(load(v, true), v) : zero);
  }
}

bool row_aligned(const void* p, int64_t ld, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * bytes % 16 == 0;
}

template <typename X, bool NORM, bool OP>
hipError_t launch_rows(const Int8Args& a, hipStream_t st) {
  const int64_t nv = OP ? (a.K + 127) / 128 * 16 : a.K / 8;
  // a dimension of a grid holds less than 2^32 threads
  const int64_t whole = OP ? round_up(a.M, 128) : a.M;
  const dim3 rows((unsigned)std::min<int64_t>(whole, 1 << 20), (unsigned)((whole + (1 << 20) - 1) >> 20));
  // vectors a thread: two while that fills no more than a workgroup, so that a row's
  // chain is short
  const int64_t per = nv <= 1024 ? 2 : nv <= 2048 ? 4 : 8;
  const unsigned threads = (unsigned)round_up((nv + per - 1) / per, 64);
  if (nv > 8192) int8_row_kernel<X, NORM, OP, 1, true><<<rows, 1024, 0, st>>>(a);
  else if (per == 2) int8_row_kernel<X, NORM, OP, 2, false><<<rows, threads, 0, st>>>(a);
  else if (per == 4) int8_row_kernel<X, NORM, OP, 4, false><<<rows, threads, 0, st>>>(a);
  else int8_row_kernel<X, NORM, OP, 8, false><<<rows, threads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quant(bool f32_input, bool operand, const void* x, int64_t rows, int64_t K, int64_t ld,
                             uint8_t* codes, float* scales, hipStream_t st) {
  Int8Args a{};
  a.x = x;
  a.M = rows;
  a.K = K;
  a.ldx = ld;
  a.codes = codes;
  a.scales = scales;
  a.ax = row_aligned(x, ld, f32_input ? 4 : 2);
  if (f32_input) return operand ? hipErrorInvalidValue : launch_rows<float, false, false>(a, st);
  return operand ? launch_rows<uint16_t, false, true>(a, st) : launch_rows<uint16_t, false, false>(a, st);
}

hipError_t launch_rms_norm_int8(const NormArgs& n, hipStream_t st) {
  Int8Args a{};
  a.x = n.x;
  a.M = n.M;
  a.K = n.K;
  a.ldx = n.ldx;
  a.codes = n.codes;
  a.scales = static_cast<float*>(n.scales);
  a.residual = n.residual;
  a.ldr = n.ldr;
  a.weight = n.weight;
  a.eps = (double)n.eps;
  a.h = n.h;
  a.ldh = n.ldh;
  a.ax = row_aligned(n.x, n.ldx, 2);
  a.ar = row_aligned(n.residual, n.ldr, 2);
  a.aw = row_aligned(n.weight, 0, 2);
  a.ah = row_aligned(n.h, n.ldh, 2);
  return launch_rows<uint16_t, true, true>(a, st);
}

}  // namespace fql
