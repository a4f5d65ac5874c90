// Softmax attention over the paged 8-bit cache (gfx950).
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale q_r . k_j - m_r)
//
// over the keys j that row r sees. Rows are (new token, query head) pairs of
// one kv head: its G query heads share every byte of cache that is read.
// q is bf16; the E4M3 codes widen exactly to bf16 for the matrix cores, the
// scales (powers of two) go into the scores and the weights p in float32.
// Scores, running maximum, running sum and output accumulators are float32;
// p (times its block's value scale, exact) is rounded to bf16 for the second
// product, the sum takes it unrounded.
//
// Both products use one trick to keep p in registers. The first computes
// S^T = K Q^T, so a lane holds scores of one query row (its column) and of
// several keys, and the second O^T = V^T P^T contracts over keys with the same
// lane holding the same rows. Which key sits in which matrix row is free, and
// it is chosen so that a lane's scores belong to 16 consecutive tokens: those
// are one 16-byte piece of a channel in the value cache, and they lie in one
// block, so each lane has one scale of each kind per tile.
#include <algorithm>
#include <cstdio>

#include "fql_device.h"
#include "fql_serving.h"

namespace fql {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Eight E4M3 bytes (two words, lowest first) -> bf16, exact.
__device__ __forceinline__ bf16x8 widen8(uint32_t a, uint32_t b) {
  const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf16x2 q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf16x2 s = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
}
__device__ __forceinline__ bf16x8 round8(const float* p) {
  return bf16x8{(__bf16)p[0], (__bf16)p[1], (__bf16)p[2], (__bf16)p[3],
                (__bf16)p[4], (__bf16)p[5], (__bf16)p[6], (__bf16)p[7]};
}
// 2^(byte - 127), also for byte 0 (a float32 subnormal)
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ bf16x8 load_q8(const uint16_t* p, bool aligned) {
  if (aligned) return *reinterpret_cast<const bf16x8*>(p);
  uint4v u;
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
  return __builtin_bit_cast(bf16x8, u);
}

// The keys row `r` of a sequence's rows sees: [lo, hi).
struct Visible {
  int lo, hi;
};
__device__ __forceinline__ Visible visible_of(const SeqSpan& s, int token, int causal, int window) {
  const int p = s.pos0 + token;
  Visible v;
  v.hi = causal ? (p + 1 < s.len ? p + 1 : s.len) : s.len;
  v.lo = window > 0 && p - window + 1 > 0 ? p - window + 1 : 0;
  return v;
}

__device__ __forceinline__ int clamp16(int v) { return v < 0 ? 0 : (v > 16 ? 16 : v); }

// A lane's 16-token pieces of VT channels: tokens skip .. have - 1 stay, the
// others become zero.
template <int VT>
__device__ __forceinline__ void mask_values(uint4v (&vw)[VT], int have, int skip) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = have - 4 * j, f = skip - 4 * j;
    const uint32_t upto = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
    const uint32_t below = f >= 4 ? 0xFFFFFFFFu : f <= 0 ? 0u : (1u << (8 * f)) - 1u;
#pragma unroll
    for (int i = 0; i < VT; ++i) vw[i][j] &= upto & ~below;
  }
}
// 0x80 in every byte that is E4M3's NaN (all seven magnitude bits set)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
template <int VT>
__device__ __forceinline__ bool has_nan(const uint4v (&vw)[VT]) {
  uint32_t any = 0u;
#pragma unroll
  for (int i = 0; i < VT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) any |= nan_bytes(vw[i][j]);
  return any != 0u;
}
// Replaces NaN values by zeros and makes NaN of every output whose row sees
// one in its channel: a product of 0/1 matrices counts them.
template <int NC, int VT>
__device__ __forceinline__ void nan_rows(uint4v (&vw)[VT], const uint32_t (&seen)[NC], float4v (&o)[NC][VT]) {
  bf16x8 p[NC][2];
#pragma unroll
  for (int t = 0; t < NC; ++t)
#pragma unroll
    for (int j = 0; j < 16; ++j) p[t][j / 8][j % 8] = (seen[t] >> j) & 1u ? (__bf16)1.0f : (__bf16)0.0f;
#pragma unroll
  for (int i = 0; i < VT; ++i) {
    uint32_t one[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t n = nan_bytes(vw[i][j]) >> 7;  // 1 in each such byte
      vw[i][j] &= ~(n * 0xFFu);
      one[j] = n * 0x38u;  // E4M3's code of 1
    }
    const bf16x8 v0 = widen8(one[0], one[1]), v1 = widen8(one[2], one[3]);
#pragma unroll
    for (int t = 0; t < NC; ++t) {
      float4v n = float4v{0.f, 0.f, 0.f, 0.f};
      n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, p[t][0], n, 0, 0, 0);
      n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, p[t][1], n, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) o[t][i][r] = n[r] > 0.0f ? __builtin_nanf("") : o[t][i][r];
    }
  }
}

// Float32 partial results cross XCDs (each with its own L2) like the GEMMs'
// split-K slabs: agent-scope relaxed stores and loads.
__device__ __forceinline__ void put_f4(float* p, const float4v& v) {
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  __hip_atomic_store(q, __builtin_bit_cast(uint64_t, float2v{v[0], v[1]}), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(q + 1, __builtin_bit_cast(uint64_t, float2v{v[2], v[3]}), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float4v get_f4(const float* p) {
  uint64_t* q = const_cast<uint64_t*>(reinterpret_cast<const uint64_t*>(p));
  const float2v a = __builtin_bit_cast(float2v, __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  const float2v b = __builtin_bit_cast(float2v, __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  return float4v{a[0], a[1], b[0], b[1]};
}
__device__ __forceinline__ void put_f2(float* p, float a, float b) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, float2v{a, b}), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2v get_f2(const float* p) {
  uint64_t* q = const_cast<uint64_t*>(reinterpret_cast<const uint64_t*>(p));
  return __builtin_bit_cast(float2v, __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// Four consecutive channels of one output row (sum / l; a row that sees no key
// gives zeros), and the row's log-sum-exp once.
__device__ __forceinline__ void write_out4(const AttnArgs& a, const SeqSpan& s, int kv_head, int G, int row, int d,
                                           const float4v& o, float m, float l) {
  const int64_t t = s.row0 + row / G;
  const int head = kv_head * G + row % G;
  uint16_t* dst = a.out + t * a.o_ld_token + head * a.o_ld_head + d;
  const float r = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = l == 0.0f ? 0u : f32_to_bf16_bits(o[i] * r);
  if ((reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
    *reinterpret_cast<uint64_t*>(dst) = (uint64_t)(b[0] | (b[1] << 16)) | ((uint64_t)(b[2] | (b[3] << 16)) << 32);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = (uint16_t)b[i];
  }
  if (a.lse != nullptr && d == 0) a.lse[t * a.Hq + head] = l == 0.0f ? neg_inf() : kLn2 * m + __logf(l);
}

// Partial results of one range of keys: float32 [rows][D] sums, then [rows]
// (maximum, sum) pairs.
template <int D>
__device__ __forceinline__ int64_t partial_floats(int rows) {
  return (int64_t)rows * (D + 2);
}

// The last workgroup of a row tile to arrive adds the ranges' results in
// order: every thread (thread tid of 256) takes items of four channels.
template <int D>
__device__ __forceinline__ void join_ranges(const AttnArgs& a, const SeqSpan& s, int kv_head, int G, int row0,
                                            int rows_in_tile, int tile_rows, int ns, const float* slab) {
  const int64_t stride = partial_floats<D>(tile_rows);
  for (int item = threadIdx.x; item < rows_in_tile * (D / 4); item += 256) {
    const int row = item / (D / 4), d = (item % (D / 4)) * 4;
    const float* ml = slab + (int64_t)tile_rows * D + row * 2;
    const float* po = slab + (int64_t)row * D + d;
    float M = neg_inf(), L = 0.0f;
    float4v o = float4v{0.f, 0.f, 0.f, 0.f};
    // eight ranges a round, all loads issued before any is used
    for (int z0 = 0; z0 < ns; z0 += 8) {
      float2v p[8];
      float4v v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int z = z0 + j < ns ? z0 + j : ns - 1;
        p[j] = get_f2(ml + z * stride);
        v[j] = get_f4(po + z * stride);
      }
      float top = M;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, p[j][0]);
      const float safe = top == neg_inf() ? 0.0f : top;
      const float back = exp2_fast(M - safe);
      M = top;
      L *= back;
      o *= back;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (z0 + j < ns) {
          const float w = exp2_fast(p[j][0] - safe);
          L += w * p[j][1];
          o += w * v[j];
        }
    }
    write_out4(a, s, kv_head, G, row0 + row, d, o, M, L);
  }
}

// Whether this workgroup is the last of `ns` to arrive (its partial results
// are written); the counter is put back to zero by the last.
__device__ __forceinline__ bool last_to_arrive(uint32_t* counter, int ns, uint32_t* s_flag) {
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");  // partial stores have completed
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t n = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_flag = n == (uint32_t)(ns - 1) ? 1u : 0u;
    if (n == (uint32_t)(ns - 1)) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *s_flag != 0u;
}

// ---------------------------------------------------------------------------
// few rows: every wave its own keys
// ---------------------------------------------------------------------------
//
// NC tiles of 16 rows; the four waves of a workgroup take 64-token tiles in
// turn and keep their own running maximum, sum and output, joined through LDS
// at the end. The call is a stream over the cache: codes go straight from
// memory into registers (16-byte loads; keys: a lane's 16 bytes of 4
// neighbouring lanes make 64 bytes of a row, values: 256-byte runs), the next
// tile's keys are loaded while this tile's weights and values are worked on
// and the other way round, so about one tile of keys or values per wave is
// always in flight and no barrier is in the loop.
//
// v_mfma_f32_16x16x32_bf16: A lane l holds row l % 16, k = 8 (l / 16) + j;
// B column l % 16, the same k; the result column l % 16, rows 4 (l / 16) + i.
//   S^T tile a (0..3) of 64 tokens: row r is token 16 (r / 4) + 4 a + r % 4,
//     so lane group g = l / 16 ends up with tokens 16 g + 4 a + i.
//   The contraction over D in step s: k = 8 g + j is channel
//     64 (s / 2) + 16 g + 8 (s % 2) + j (keys and queries alike).
//   O^T step s (0, 1): k = 8 g + j is token 16 g + 8 s + j, byte 8 s + j of the
//     lane's 16-byte piece of channel l % 16.
template <int D, int NC>
__global__ __launch_bounds__(256) void attn_kv8_stream_kernel(const AttnArgs a, const PagedCache c,
                                                              const PagedBatch pb, int bs_shift, int row_tiles,
                                                              int splits, int chunk, float* partial,
                                                              uint32_t* counters) {
  constexpr int KI = D / 64, VT = D / 16, SK = D / 32;
  __shared__ float4v so[4][NC * VT][64];
  __shared__ float2v sml[4][NC][16];
  __shared__ uint32_t s_flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int bh = blockIdx.x, H = c.heads, h = bh % H, b = bh / H;
  const int rt = blockIdx.y % row_tiles, z = blockIdx.y / row_tiles;
  const int G = a.Hq / H, bs = c.block_size;
  const SeqSpan s = seq_span(pb, b, bs);
  const int rows = s.n * G, row0 = rt * 16 * NC;
  if (row0 >= rows) return;
  const int last_row = row0 + 16 * NC < rows ? row0 + 16 * NC - 1 : rows - 1;
  const int kmin = visible_of(s, row0 / G, a.causal, a.window).lo & ~63;
  const int kmax = visible_of(s, last_row / G, a.causal, a.window).hi;
  int ns = kmax > kmin ? (kmax - kmin + chunk - 1) / chunk : 1;
  ns = ns < splits ? ns : splits;
  if (z >= ns) return;
  const int k0 = kmin + z * chunk;
  const int k1 = z == ns - 1 || k0 + chunk > kmax ? kmax : k0 + chunk;

  // this lane's columns (query rows)
  bf16x8 q[NC][SK];
  int vlo[NC], vhi[NC];
#pragma unroll
  for (int t = 0; t < NC; ++t) {
    const int row = row0 + 16 * t + col;
    const bool ok = row < rows;
    const int token = ok ? row / G : 0;
    const Visible v = visible_of(s, token, a.causal, a.window);
    vlo[t] = v.lo;
    vhi[t] = ok ? v.hi : 0;
    const uint16_t* qp = a.q + (s.row0 + token) * a.q_ld_token + (int64_t)(h * G + (ok ? row % G : 0)) * a.q_ld_head;
#pragma unroll
    for (int i = 0; i < SK; ++i) {
      q[t][i] = load_q8(qp + 64 * (i / 2) + 16 * g + 8 * (i % 2), a.aligned);
      if (!ok)
#pragma unroll
        for (int j = 0; j < 8; ++j) q[t][i][j] = (__bf16)0.0f;
    }
  }
  // keys below all_lo or from all_hi on are hidden from some row, keys below
  // any_lo from every row (as those from kmax on)
  const int all_lo = visible_of(s, last_row / G, a.causal, a.window).lo;
  const int all_hi = visible_of(s, row0 / G, a.causal, a.window).hi;
  const int any_lo = visible_of(s, row0 / G, a.causal, a.window).lo;

  const float sl2 = a.scale * kLog2e;
  float m[NC], l[NC];
  float4v o[NC][VT];
#pragma unroll
  for (int t = 0; t < NC; ++t) {
    m[t] = neg_inf();
    l[t] = 0.0f;
#pragma unroll
    for (int i = 0; i < VT; ++i) o[t][i] = float4v{0.f, 0.f, 0.f, 0.f};
  }

  const int64_t page_bytes = (int64_t)H * bs * D;
  const uint8_t* kbase = c.k + (int64_t)h * bs * D + (col & 3) * D + 16 * g;
  const uint8_t* vbase = c.v + (int64_t)h * bs * D + col * 16;
  const int32_t* table = pb.table + (int64_t)b * pb.ld_table;
  // the block of token t: -1 past the keys of this workgroup or outside the cache
  auto block_of = [&](int t) -> int64_t {
    if (t >= kmax) return -1;  // kmax <= len <= the table's capacity
    const int64_t p = table[t >> bs_shift];
    return p >= 0 && p < c.num_blocks ? p : -1;
  };
  uint4v kw[4][KI], vw[VT];
  uint32_t ksb = 0, vsb = 0;
  // loads of a tile; a block that is not there is read from block 0 and masked
  auto load_k = [&](int t0, int64_t blk) {
    const int t = t0 + 16 * (col >> 2);
    const uint8_t* p = kbase + (blk < 0 ? 0 : blk) * page_bytes + (int64_t)(t & (bs - 1)) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < KI; ++j) kw[i][j] = *reinterpret_cast<const uint4v*>(p + i * 4 * D + j * 64);
  };
  auto load_v = [&](int t0, int64_t blk) {
    const int t = t0 + 16 * g;
    const int64_t bk = blk < 0 ? 0 : blk;
    const uint8_t* p = vbase + bk * page_bytes + (int64_t)(t & (bs - 1)) * D;
#pragma unroll
    for (int i = 0; i < VT; ++i) vw[i] = *reinterpret_cast<const uint4v*>(p + i * 256);
  };
  auto load_scales = [&](int64_t blk) {
    const int64_t at = (blk < 0 ? 0 : blk) * H + h;
    ksb = c.k_scale[at];
    vsb = blk < 0 ? 0u : c.v_scale[at];  // its weights are zero, and stay so under a finite scale
  };

  int t0 = k0 + 64 * wave;
  int64_t blk = -1, blk_k = -1;
  if (t0 < k1) {
    blk = block_of(t0 + 16 * g);
    blk_k = block_of(t0 + 16 * (col >> 2));
    load_k(t0, blk_k);
    load_scales(blk);
    load_v(t0, blk);
  }
  for (; t0 < k1; t0 += 256) {
    const int64_t blk_next = block_of(t0 + 256 + 16 * g), blk_k_next = block_of(t0 + 256 + 16 * (col >> 2));
    const bool more = t0 + 256 < k1;
    float x[NC][16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4v acc[NC];
#pragma unroll
      for (int t = 0; t < NC; ++t) acc[t] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < SK; ++j) {
        const uint4v w = kw[i][j / 2];
        const bf16x8 kf = j % 2 == 0 ? widen8(w[0], w[1]) : widen8(w[2], w[3]);
#pragma unroll
        for (int t = 0; t < NC; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[t][j], acc[t], 0, 0, 0);
      }
#pragma unroll
      for (int t = 0; t < NC; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[t][4 * i + r] = acc[t][r];
    }
    const float ks = e8m0(ksb) * sl2, vs = e8m0(vsb);
    if (more) load_k(t0 + 256, blk_k_next);
    const int tg = t0 + 16 * g;  // this lane's 16 tokens start here
    // Masked in edge tiles only: keys hidden from some row, past this range
    // (the ranges meet at multiples of 64, so only past kmax) or of a block
    // that is not there.
    const bool edge = t0 < all_lo || t0 + 64 > all_hi || t0 + 64 > k1 || __any(blk < 0);
    if (edge) {
      const int have = blk < 0 ? 0 : clamp16(k1 - tg), skip = clamp16(any_lo - tg);
      uint32_t seen[NC];  // bit i: this lane's row sees its token i
#pragma unroll
      for (int t = 0; t < NC; ++t) {
        const int lo = clamp16(vlo[t] - tg), hi = clamp16(vhi[t] - tg);
        const int top = hi < have ? hi : have;
        seen[t] = ((1u << top) - 1u) & ~((1u << lo) - 1u);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[t][i] = (seen[t] >> i) & 1u ? x[t][i] * ks : neg_inf();
      }
      // Values of tokens that no row sees may hold anything, and 0 * NaN is
      // not 0: they are zeroed.
      mask_values<VT>(vw, have, skip);
      // NaN values of tokens that some rows see and others do not: taken out
      // of the product, and put back into the rows that see them.
      if ((all_lo > any_lo || all_hi < kmax) && __any(has_nan<VT>(vw))) nan_rows<NC, VT>(vw, seen, o);
    } else {
#pragma unroll
      for (int t = 0; t < NC; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[t][i] *= ks;
    }
    bf16x8 p[NC][2];
#pragma unroll
    for (int t = 0; t < NC; ++t) {
      float top = x[t][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, x[t][i]);
      top = __builtin_fmaxf(top, __shfl_xor(top, 16));
      top = __builtin_fmaxf(top, __shfl_xor(top, 32));
      top = __builtin_fmaxf(top, m[t]);
      const float safe = top == neg_inf() ? 0.0f : top;
      if (__any(top > m[t])) {
        const float back = exp2_fast(m[t] - safe);
        l[t] *= back;
#pragma unroll
        for (int i = 0; i < VT; ++i) o[t][i] *= back;
        m[t] = top;
      }
      float w[16];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = exp2_fast(x[t][i] - safe);
        sum += w[i];
        w[i] *= vs;
      }
      l[t] += sum;
      p[t][0] = round8(w);
      p[t][1] = round8(w + 8);
    }
#pragma unroll
    for (int i = 0; i < VT; ++i) {
      const bf16x8 v0 = widen8(vw[i][0], vw[i][1]), v1 = widen8(vw[i][2], vw[i][3]);
#pragma unroll
      for (int t = 0; t < NC; ++t) {
        o[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, p[t][0], o[t][i], 0, 0, 0);
        o[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, p[t][1], o[t][i], 0, 0, 0);
      }
    }
    blk = blk_next;
    if (more) {
      load_scales(blk);
      load_v(t0 + 256, blk);
    }
  }

  // join the four waves
#pragma unroll
  for (int t = 0; t < NC; ++t) {
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (g == 0) sml[wave][t][col] = float2v{m[t], l[t]};
#pragma unroll
    for (int i = 0; i < VT; ++i) so[wave][t * VT + i][lane] = o[t][i];
  }
  __syncthreads();
  const int tile = (bh * row_tiles + rt);
  float* slab = partial + (int64_t)tile * splits * partial_floats<D>(16 * NC);
  float* mine = slab + z * partial_floats<D>(16 * NC);
  for (int f = wave; f < NC * VT; f += 4) {
    const int t = f / VT, i = f % VT;
    float M = neg_inf();
#pragma unroll
    for (int w = 0; w < 4; ++w) M = __builtin_fmaxf(M, sml[w][t][col][0]);
    const float safe = M == neg_inf() ? 0.0f : M;
    float L = 0.0f;
    float4v sum = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2v ml = sml[w][t][col];
      const float f2 = exp2_fast(ml[0] - safe);
      L += f2 * ml[1];
      sum += f2 * so[w][f][lane];
    }
    const int row = 16 * t + col, d = 16 * i + 4 * g;
    if (row0 + row >= rows) continue;
    if (ns == 1) {
      write_out4(a, s, h, G, row0 + row, d, sum, M, L);
    } else {
      put_f4(mine + (int64_t)row * D + d, sum);
      if (d == 0) put_f2(mine + (int64_t)16 * NC * D + row * 2, M, L);
    }
  }
  if (ns == 1) return;
  if (last_to_arrive(counters + tile, ns, &s_flag))
    join_ranges<D>(a, s, h, G, row0, last_row - row0 + 1, 16 * NC, ns, slab);
}

}  // namespace

// ---------------------------------------------------------------------------
// plan, launcher
// ---------------------------------------------------------------------------

AttnPlan plan_attention(int B, int Hq, int Hkv, int D, int64_t max_new, int64_t max_len, int window) {
  AttnPlan p{};
  const int64_t rows = std::max<int64_t>(1, max_new) * (Hq / Hkv);
  p.kind = 0;
  p.cols = rows <= 16 ? 1 : 2;
  p.row_tiles = (int)((rows + 16 * p.cols - 1) / (16 * p.cols));
  const int64_t tiles = (int64_t)B * Hkv * p.row_tiles;
  // keys one row tile goes through; with a window it starts at a multiple of
  // 64 below its first visible key
  int64_t span = max_len < 1 ? 1 : max_len;
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + max_new - 1 + 63);
  // ranges: about 2048 workgroups, at least 256 keys each
  int64_t splits = std::max<int64_t>(1, std::min<int64_t>((2048 + tiles - 1) / tiles, (span + 255) / 256));
  // one arrival counter a tile, below the words a linear call keeps its device scalars in
  if (tiles > kWorkspaceScalarOffset / 4) splits = 1;
  int64_t chunk = round_up((span + splits - 1) / splits, 64);
  splits = (span + chunk - 1) / chunk;
  p.splits = (int)splits;
  p.chunk = (int)chunk;
  p.counter_bytes = kWorkspaceCounterBytes;
  p.partial_bytes = splits > 1 ? round_up(tiles * splits * (16 * p.cols) * (D + 2) * 4, 256) : 0;
  p.total_bytes = p.counter_bytes + p.partial_bytes;
  return p;
}

std::string describe_attention(const AttnPlan& p, int D) {
  char b[160];
  std::snprintf(b, sizeof(b), "attn_kv8_stream_kernel<D=%d,NC=%d> row_tiles=%d splits=%d chunk=%d", D, p.cols,
                p.row_tiles, p.splits, p.chunk);
  return std::string(b);
}

hipError_t launch_attention(const AttnPlan& p, const AttnArgs& a, const PagedCache& c, const PagedBatch& pb,
                            uint8_t* workspace, hipStream_t st) {
  int shift = 4;
  while ((1 << shift) < c.block_size) ++shift;
  uint32_t* counters = reinterpret_cast<uint32_t*>(workspace);
  float* partial = reinterpret_cast<float*>(workspace + p.counter_bytes);
  const dim3 grid((unsigned)(pb.B * c.heads), (unsigned)(p.row_tiles * p.splits), 1);
#define FQL_A(DD, NC)                                                                                    \
  if (c.D == DD && p.cols == NC) {                                                                       \
    attn_kv8_stream_kernel<DD, NC><<<grid, 256, 0, st>>>(a, c, pb, shift, p.row_tiles, p.splits, p.chunk, \
                                                         partial, counters);                             \
    return hipGetLastError();                                                                            \
  }
  FQL_A(64, 1) FQL_A(64, 2) FQL_A(128, 1) FQL_A(128, 2) FQL_A(256, 1) FQL_A(256, 2)
#undef FQL_A
  return hipErrorInvalidValue;
}

}  // namespace fql
