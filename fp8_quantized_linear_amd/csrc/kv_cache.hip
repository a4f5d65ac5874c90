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

// What one workgroup writes: offsets lo .. hi - 1 of a block and head, from
// rows at src (offset lo's row).
struct Span {
  int64_t page;
  int lo, hi;
  const uint16_t* src;
  int64_t ld;
};
// False: nothing to write (all threads agree).
__device__ __forceinline__ bool span_of(const PagedCache& c, const PagedBatch& pb, int j, int h, int b, bool values,
                                        const uint16_t* k, const uint16_t* v, int64_t k_ldt, int64_t k_ldh,
                                        int64_t v_ldt, int64_t v_ldh, Span* o) {
  const int bs = c.block_size;
  const SeqSpan s = seq_span(pb, b, bs);
  const int start = s.pos0 > 0 ? s.pos0 : 0;  // new tokens before position 0 are dropped
  const int blk = start / bs + j;
  const int end = s.pos0 + s.n < s.len ? s.pos0 + s.n : s.len;  // past the last new token
  if (blk >= pb.table_cols || (int64_t)blk * bs >= end) return false;
  o->page = pb.table[(int64_t)b * pb.ld_table + blk];
  if (o->page < 0 || o->page >= c.num_blocks) return false;
  o->lo = start > blk * bs ? start - blk * bs : 0;
  o->hi = end - blk * bs < bs ? end - blk * bs : bs;
  o->ld = values ? v_ldt : k_ldt;
  o->src = (values ? v + h * v_ldh : k + h * k_ldh) + (s.row0 + (int64_t)blk * bs + o->lo - s.pos0) * o->ld;
  return o->lo < o->hi;
}

// The block's new exponent from this thread's maximum, and the old one; the
// scale is stored. All threads must call it.
struct Exponents {
  int now, old;
  bool grew;  // codes below lo have to be rounded again
};
__device__ __forceinline__ Exponents settle_scale(uint8_t* scale, float a, int lo, float* red) {
  const int tid = threadIdx.x, T = blockDim.x;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) a = __builtin_fmaxf(a, __shfl_xor(a, o));
  Exponents e;
  e.old = (int)*scale - 127;
  if ((tid & 63) == 0) red[tid >> 6] = a;
  __syncthreads();
  a = red[0];
  for (int w = 1; w < T / 64; ++w) a = __builtin_fmaxf(a, red[w]);
  e.now = cover_exponent(a);
  if (lo > 0 && e.old > e.now) e.now = e.old;
  e.grew = lo > 0 && e.now != e.old;
  if (tid == 0) *scale = (uint8_t)(e.now + 127);
  return e;
}

// Codes of offsets below lo in four bytes of offsets t0 .. t0 + 3, rounded
// again for a grown scale; other bytes as they are.
__device__ __forceinline__ uint32_t regrow4(uint32_t w, int t0, int lo, int shift) {
  const int own = lo - t0;
  if (own <= 0) return w;
  const uint32_t mask = own >= 4 ? 0xFFFFFFFFu : (1u << (8 * own)) - 1u;
  return (rescale4(w, shift) & mask) | (w & ~mask);
}
__device__ __forceinline__ void regrow_keys(uint8_t* dst, int lo, int D, int shift) {
  for (int i = threadIdx.x; i < lo * D / 16; i += blockDim.x) {
    uint4v* p = reinterpret_cast<uint4v*>(dst) + i;
    uint4v w = *p;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = rescale4(w[j], shift);
    *p = w;
  }
}
__device__ __forceinline__ float finite_max(float a, float v) {
  const float u = __builtin_fabsf(v);
  return u < __builtin_inff() && u > a ? u : a;
}
__device__ __forceinline__ uint64_t codes8(const float f[8], int e) {
  return (uint64_t)e4m3x4(scale_down(f[0], e), scale_down(f[1], e), scale_down(f[2], e), scale_down(f[3], e)) |
         ((uint64_t)e4m3x4(scale_down(f[4], e), scale_down(f[5], e), scale_down(f[6], e), scale_down(f[7], e)) << 32);
}

// Few new tokens a sequence (decode): nothing is kept between the maximum and
// the codes, and one or a few waves do a block.
// Its time is its chain of dependent accesses (lengths, table, tokens, scale,
// group): 64 sequences x 8 heads x 128 channels, one token each, 5.5 us for 0.4 MB.
__global__ __launch_bounds__(256) void kv_append_kernel(const PagedCache c, const PagedBatch pb,
                                                        const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, int64_t k_ldt,
                                                        int64_t k_ldh, int64_t v_ldt, int64_t v_ldh,
                                                        bool aligned) {
  __shared__ float red[4];
  const bool values = blockIdx.x & 1;
  const int h = blockIdx.y, tid = threadIdx.x, T = blockDim.x, D = c.D;
  Span s;
  if (!span_of(c, pb, blockIdx.x >> 1, h, blockIdx.z, values, k, v, k_ldt, k_ldh, v_ldt, v_ldh, &s)) return;
  const int dv = D / 8, nvec = (s.hi - s.lo) * dv;
  float a = 0.0f;
  for (int i = tid; i < nvec; i += T) {
    float f[8];
    load8_bf16(s.src + (int64_t)(i / dv) * s.ld + (i % dv) * 8, aligned, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = finite_max(a, f[j]);
  }
  const int64_t at = s.page * c.heads + h;
  const Exponents e = settle_scale((values ? c.v_scale : c.k_scale) + at, a, s.lo, red);
  uint8_t* const dst = (values ? c.v : c.k) + at * c.block_size * D;
  if (!values) {
    if (e.grew) regrow_keys(dst, s.lo, D, e.old - e.now);
    for (int i = tid; i < nvec; i += T) {
      const int t = i / dv, d = (i % dv) * 8;
      float f[8];
      load8_bf16(s.src + (int64_t)t * s.ld + d, aligned, f);
      *reinterpret_cast<uint64_t*>(dst + (int64_t)(s.lo + t) * D + d) = codes8(f, e.now);
    }
    return;
  }
  const int g0 = e.grew ? 0 : s.lo / 16, g1 = (s.hi + 15) / 16;
  for (int i = tid; i < (g1 - g0) * D; i += T) {
    const int g = g0 + i / D, d = i % D, t0 = g * 16;
    uint4v* p = reinterpret_cast<uint4v*>(dst) + g * D + d;
    uint4v w = uint4v{0u, 0u, 0u, 0u};
    if (t0 < s.lo || t0 + 16 > s.hi) {
      w = *p;
      if (e.grew)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = regrow4(w[j], t0 + 4 * j, s.lo, e.old - e.now);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4];
      uint32_t mask = 0u;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + 4 * j + u;
        const bool in = t >= s.lo && t < s.hi;
        f[u] = in ? scale_down(bf16_bits_to_f32(s.src[(int64_t)(t - s.lo) * s.ld + d]), e.now) : 0.0f;
        mask |= in ? 0xFFu << (8 * u) : 0u;
      }
      w[j] = (e4m3x4(f[0], f[1], f[2], f[3]) & mask) | (w[j] & ~mask);
    }
    *p = w;
  }
}

// Exchanges within a quad of lanes: lane ^ 2, lane ^ 1.
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v) { return __builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true); }
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v) { return __builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true); }

// Many new tokens: a block and head is read once into registers (16 R
// registers a thread, R = block_size * D / 8192 rounded up), 16 bytes a lane.
// Values: lane q of a quad loads channels 8 d8 .. 8 d8 + 7 of tokens
// 4 q .. 4 q + 3 of a group of 16, packs each channel's four codes into a
// word, and a transposition within the quad leaves it channels 8 d8 + 2 q and
// + 1 with all 16 tokens: 32 contiguous bytes of the cache.
// Five prompts of up to 2500 tokens (8 heads, 128 channels, 52 MB): 16.5 us, 3.1
// TB/s, 28 us when a workgroup read its block twice and wrote values byte by
// byte. A workgroup's chain (lengths, table, tokens, maximum, scale) is exposed
// in part: there are 6.5 of them a CU at that size.
template <int R>
__global__ __launch_bounds__(256) void kv_append_block_kernel(const PagedCache c, const PagedBatch pb,
                                                              const uint16_t* __restrict__ k,
                                                              const uint16_t* __restrict__ v, int64_t k_ldt,
                                                              int64_t k_ldh, int64_t v_ldt, int64_t v_ldh,
                                                              bool aligned) {
  __shared__ float red[4];
  const bool values = blockIdx.x & 1;
  const int h = blockIdx.y, tid = threadIdx.x, D = c.D;
  Span s;
  if (!span_of(c, pb, blockIdx.x >> 1, h, blockIdx.z, values, k, v, k_ldt, k_ldh, v_ldt, v_ldh, &s)) return;
  const int dv = D / 8;
  const int64_t at = s.page * c.heads + h;
  uint8_t* const dst = (values ? c.v : c.k) + at * c.block_size * D;
  uint4v u[R][4];
  // the offset and channel vector of load (r, i) of this thread
  auto place = [&](int r, int i, int* t, int* d) {
    if (values) {
      const int unit = (tid >> 2) + 64 * r;
      *t = unit / dv * 16 + 4 * (tid & 3) + i;
      *d = unit % dv;
    } else {
      const int vec = tid + 256 * (4 * r + i);
      *t = s.lo + vec / dv;
      *d = vec % dv;
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int t, d;
      place(r, i, &t, &d);
      u[r][i] = uint4v{0u, 0u, 0u, 0u};
      if (t >= s.lo && t < s.hi) {
        const uint16_t* p = s.src + (int64_t)(t - s.lo) * s.ld + 8 * d;
        if (aligned) u[r][i] = *reinterpret_cast<const uint4v*>(p);
        else
#pragma unroll
          for (int j = 0; j < 4; ++j) u[r][i][j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
      }
    }
  float a = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a = finite_max(finite_max(a, __uint_as_float(u[r][i][j] << 16)), __uint_as_float(u[r][i][j] & 0xFFFF0000u));
  const Exponents e = settle_scale((values ? c.v_scale : c.k_scale) + at, a, s.lo, red);
  if (!values && e.grew) regrow_keys(dst, s.lo, D, e.old - e.now);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint64_t q8[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(u[r][i][j] << 16);
        f[2 * j + 1] = __uint_as_float(u[r][i][j] & 0xFFFF0000u);
      }
      q8[i] = codes8(f, e.now);
    }
    if (!values) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int t, d;
        place(r, i, &t, &d);
        if (t < s.hi) *reinterpret_cast<uint64_t*>(dst + (int64_t)t * D + 8 * d) = q8[i];
      }
      continue;
    }
    // w[j]: channel j's codes of this lane's four tokens
    uint32_t w[8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (uint32_t)(q8[i] >> (32 * half));
      // 4 x 4 bytes transposed: x[i] byte j -> w[4 half + j] byte i
      const uint32_t a0 = __builtin_amdgcn_perm(x[1], x[0], 0x05010400u), a1 = __builtin_amdgcn_perm(x[1], x[0], 0x07030602u);
      const uint32_t b0 = __builtin_amdgcn_perm(x[3], x[2], 0x05010400u), b1 = __builtin_amdgcn_perm(x[3], x[2], 0x07030602u);
      w[4 * half + 0] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
      w[4 * half + 1] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
      w[4 * half + 2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
      w[4 * half + 3] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
    }
    // lane q ends with channels 2 q, 2 q + 1 of all four lanes
    const int q = tid & 3;
    const bool hi = q & 2, odd = q & 1;
    uint4v out[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint32_t p0 = w[n], p1 = w[2 + n], p2 = w[4 + n], p3 = w[6 + n];  // channel pairs 0 .. 3
      // pairs of this lane's half from itself (a) and from lane ^ 2 (b)
      const uint32_t a0 = hi ? p2 : p0, a1 = hi ? p3 : p1;
      const uint32_t b0 = quad_xor2(hi ? p0 : p2), b1 = quad_xor2(hi ? p1 : p3);
      const uint32_t mine = odd ? a1 : a0, across = odd ? b1 : b0;              // lanes q, q ^ 2
      const uint32_t mine1 = quad_xor1(odd ? a0 : a1), across1 = quad_xor1(odd ? b0 : b1);  // q ^ 1, q ^ 3
      const uint32_t n0 = odd ? mine1 : mine, n1 = odd ? mine : mine1;          // this half's lanes in order
      const uint32_t f0 = odd ? across1 : across, f1 = odd ? across : across1;  // the other half's
      out[n] = hi ? uint4v{f0, f1, n0, n1} : uint4v{n0, n1, f0, f1};
    }
    const int unit = (tid >> 2) + 64 * r, g = unit / dv, t0 = 16 * g;
    if (t0 >= s.hi || (t0 + 16 <= s.lo && !e.grew)) continue;
    uint4v* p = reinterpret_cast<uint4v*>(dst) + g * D + 8 * (unit % dv) + 2 * q;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      if (t0 < s.lo || t0 + 16 > s.hi) {  // bytes outside lo .. hi - 1 stay the block's own
        uint4v held = p[n];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (e.grew) held[j] = regrow4(held[j], t0 + 4 * j, s.lo, e.old - e.now);
          uint32_t mask = 0u;
#pragma unroll
          for (int b = 0; b < 4; ++b) mask |= t0 + 4 * j + b >= s.lo && t0 + 4 * j + b < s.hi ? 0xFFu << (8 * b) : 0u;
          out[n][j] = (out[n][j] & mask) | (held[j] & ~mask);
        }
      }
      p[n] = out[n];
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const PagedCache& c, const PagedBatch& pb, const uint16_t* k, const uint16_t* v,
                            int64_t k_ld_token, int64_t k_ld_head, int64_t v_ld_token, int64_t v_ld_head,
                            bool aligned, hipStream_t st) {
  // blocks one sequence's new tokens can touch
  const int64_t per = (pb.max_new - 1 + c.block_size - 1) / c.block_size + 1;
  const int64_t span = per < pb.table_cols ? per : pb.table_cols;
  const dim3 grid((unsigned)(2 * span), (unsigned)c.heads, (unsigned)pb.B);
  // blocks that may be filled to a quarter or more are worth a workgroup that
  // holds them whole; below, one wave does a token's D / 8 vectors
  if (pb.max_new >= 16 && pb.max_new >= c.block_size / 4) {
#define FQL_R(R)                                                                                           \
  if (c.block_size * c.D <= 8192 * R) {                                                                    \
    kv_append_block_kernel<R><<<grid, 256, 0, st>>>(c, pb, k, v, k_ld_token, k_ld_head, v_ld_token, v_ld_head, \
                                                    aligned);                                              \
    return hipGetLastError();                                                                              \
  }
    FQL_R(1) FQL_R(2) FQL_R(4) FQL_R(8)
#undef FQL_R
  }
  const unsigned threads = (int64_t)pb.max_new * c.D / 8 <= 64 ? 64 : 256;
  kv_append_kernel<<<grid, threads, 0, st>>>(c, pb, k, v, k_ld_token, k_ld_head, v_ld_token, v_ld_head, aligned);
  return hipGetLastError();
}

}  // namespace fql
