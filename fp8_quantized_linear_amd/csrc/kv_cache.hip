// New keys and values into the paged 8-bit cache (gfx950).
//
// For each block and head that gets tokens: a = max |v| over its new tokens
// (finite values), e = the smallest integer with a <= 448 * 2^e (a = 0: -127),
// the scale's exponent E = e where the block starts with these tokens, else
// max(E_old, e), and codes = E4M3_RNE_satfinite(v * 2^-E). Where E grew, the
// codes that the block already holds are multiplied by 2^(E_old - E) and
// rounded again. Scaling by a power of two is exact, so nothing else is
// rounded. Infinities saturate, NaN stays NaN; neither counts for a.
//
// One workgroup per (block, head, keys or values): the scale is a reduction
// over exactly what it writes, and nothing is exchanged between workgroups.
// Values are stored 16 tokens to a channel (see fql_serving.h); a group of 16
// that is only partly new is read, completed and written as a whole, which
// for a single token is one coalesced 16 * D byte run instead of D byte
// stores in as many places.
#include "fql_device.h"
#include "fql_serving.h"
#include "sc_quant.h"

namespace fql {

namespace {

// The exponent of a non-negative finite a: smallest e with a <= 448 * 2^e, in
// [-127, 127]. 448 = 1.75 * 2^8.
__device__ __forceinline__ int cover_exponent(float a) {
  const uint32_t b = __float_as_uint(a);
  if (b == 0u) return -127;
  if (b < 0x00800000u) return -127;  // float32 subnormals: below 448 * 2^-127
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// v * 2^-e, exact unless it leaves float32's range (codes saturate or vanish
// there anyway); e in [-127, 127], and 2^127 * 2^0 takes two factors.
__device__ __forceinline__ float scale_down(float v, int e) { return ldexpf(v, -e); }

// Four float32 -> four E4M3 bytes; NaN stays NaN (0x7F).
__device__ __forceinline__ float clamp_keep_nan(float v) { return v == v ? e4m3_clamp(v) : v; }
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  short2v o = {0, 0};
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, clamp_keep_nan(a), clamp_keep_nan(b), 1.0f, false);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, clamp_keep_nan(c), clamp_keep_nan(d), 1.0f, true);
  return __builtin_bit_cast(uint32_t, o);
}

// Four codes times 2^shift (shift <= 0), rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, int shift) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
  const bf2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
  return e4m3x4(ldexpf((float)lo[0], shift), ldexpf((float)lo[1], shift), ldexpf((float)hi[0], shift),
                ldexpf((float)hi[1], shift));
}

__device__ __forceinline__ void load8_bf16(const uint16_t* p, bool aligned, float v[8]) {
  if (aligned) {
    const uint4v u = *reinterpret_cast<const uint4v*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = bf16_bits_to_f32(p[j]);
  }
}

__global__ __launch_bounds__(256) void kv_append_kernel(const PagedCache c, const PagedBatch pb,
                                                        const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, int64_t k_ldt,
                                                        int64_t k_ldh, int64_t v_ldt, int64_t v_ldh,
                                                        bool aligned) {
  __shared__ float red[4];
  const bool values = blockIdx.x & 1;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, T = blockDim.x;
  const int bs = c.block_size, D = c.D;
  const SeqSpan s = seq_span(pb, b, bs);
  const int start = s.pos0 > 0 ? s.pos0 : 0;  // new tokens before position 0 are dropped
  const int blk = start / bs + (int)(blockIdx.x >> 1);
  const int end = s.pos0 + s.n < s.len ? s.pos0 + s.n : s.len;  // past the last new token
  if (blk >= pb.table_cols || (int64_t)blk * bs >= end) return;
  const int64_t page = pb.table[(int64_t)b * pb.ld_table + blk];
  if (page < 0 || page >= c.num_blocks) return;
  const int lo = start > blk * bs ? start - blk * bs : 0;  // offsets lo .. hi - 1 are new
  const int hi = end - blk * bs < bs ? end - blk * bs : bs;
  if (lo >= hi) return;
  const int64_t ldt = values ? v_ldt : k_ldt;
  const uint16_t* src = (values ? v + h * v_ldh : k + h * k_ldh) +
                        (s.row0 + (int64_t)blk * bs + lo - s.pos0) * ldt;  // offset lo's row
  const int dv = D / 8, nvec = (hi - lo) * dv;
  float a = 0.0f;
  for (int i = tid; i < nvec; i += T) {
    float f[8];
    load8_bf16(src + (int64_t)(i / dv) * ldt + (i % dv) * 8, aligned, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = __builtin_fabsf(f[j]);
      a = u < __builtin_inff() && u > a ? u : a;
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) a = __builtin_fmaxf(a, __shfl_xor(a, o));
  uint8_t* const scale = (values ? c.v_scale : c.k_scale) + page * c.heads + h;
  const int old = (int)*scale - 127;
  if ((tid & 63) == 0) red[tid >> 6] = a;
  __syncthreads();
  a = red[0];
  for (int w = 1; w < T / 64; ++w) a = __builtin_fmaxf(a, red[w]);
  int e = cover_exponent(a);
  if (lo > 0 && old > e) e = old;
  const bool grew = lo > 0 && e != old;
  if (tid == 0) *scale = (uint8_t)(e + 127);
  const int64_t head_bytes = (int64_t)bs * D;
  if (!values) {
    uint8_t* const dst = c.k + (page * c.heads + h) * head_bytes;
    if (grew)
      for (int i = tid; i < lo * D / 16; i += T) {
        uint4v* p = reinterpret_cast<uint4v*>(dst) + i;
        uint4v w = *p;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = rescale4(w[j], old - e);
        *p = w;
      }
    for (int i = tid; i < nvec; i += T) {
      const int t = i / dv, d = (i % dv) * 8;
      float f[8];
      load8_bf16(src + (int64_t)t * ldt + d, aligned, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = scale_down(f[j], e);
      *reinterpret_cast<uint64_t*>(dst + (int64_t)(lo + t) * D + d) =
          (uint64_t)e4m3x4(f[0], f[1], f[2], f[3]) | ((uint64_t)e4m3x4(f[4], f[5], f[6], f[7]) << 32);
    }
    return;
  }
  uint8_t* const dst = c.v + (page * c.heads + h) * head_bytes;
  const int g0 = grew ? 0 : lo / 16, g1 = (hi + 15) / 16;
  for (int i = tid; i < (g1 - g0) * D; i += T) {
    const int g = g0 + i / D, d = i % D, t0 = g * 16;
    uint4v* p = reinterpret_cast<uint4v*>(dst) + g * D + d;
    uint4v w = uint4v{0u, 0u, 0u, 0u};
    if (t0 < lo || t0 + 16 > hi) {
      w = *p;
      if (grew && t0 < lo)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t r = rescale4(w[j], old - e);
          // bytes below lo are the block's own; those above are overwritten or unused
          const int own = lo - t0 - 4 * j;
          const uint32_t mask = own >= 4 ? 0xFFFFFFFFu : own <= 0 ? 0u : (1u << (8 * own)) - 1u;
          w[j] = (r & mask) | (w[j] & ~mask);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4];
      uint32_t mask = 0u;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + 4 * j + u;
        const bool in = t >= lo && t < hi;
        f[u] = in ? scale_down(bf16_bits_to_f32(src[(int64_t)(t - lo) * ldt + d]), e) : 0.0f;
        mask |= in ? 0xFFu << (8 * u) : 0u;
      }
      w[j] = (e4m3x4(f[0], f[1], f[2], f[3]) & mask) | (w[j] & ~mask);
    }
    *p = w;
  }
}

}  // namespace

hipError_t launch_kv_append(const PagedCache& c, const PagedBatch& pb, const uint16_t* k, const uint16_t* v,
                            int64_t k_ld_token, int64_t k_ld_head, int64_t v_ld_token, int64_t v_ld_head,
                            bool aligned, hipStream_t st) {
  // blocks one sequence's new tokens can touch
  const int64_t per = (pb.max_new - 1 + c.block_size - 1) / c.block_size + 1;
  const int64_t span = per < pb.table_cols ? per : pb.table_cols;
  // a call of single tokens has D / 8 vectors of keys a workgroup: one wave
  const unsigned threads = (int64_t)pb.max_new * c.D / 8 <= 64 ? 64 : 256;
  const dim3 grid((unsigned)(2 * span), (unsigned)c.heads, (unsigned)pb.B);
  kv_append_kernel<<<grid, threads, 0, st>>>(c, pb, k, v, k_ld_token, k_ld_head, v_ld_token, v_ld_head, aligned);
  return hipGetLastError();
}

}  // namespace fql
