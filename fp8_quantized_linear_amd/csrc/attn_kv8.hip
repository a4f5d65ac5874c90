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
// product, which is how the matrix cores take it at full rate; the sum takes it
// unrounded. Against 64 bits the outputs are then off by 0.0019 to 0.0023 of their
// norm, where float32 weights give 0.0016 to 0.0017, most of it the output's own
// rounding.
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

// The new token of a row and its head within the group: rows of one kv head
// are (token, head) with the head running fastest.
struct Row {
  int token, head;
};
__device__ __forceinline__ Row row_of(const AttnArgs& a, int row) {
  const int t = (int)(((uint64_t)(uint32_t)row * a.group_mul) >> a.group_shift);
  return Row{t, row - t * a.group};
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
// Zeros in the place of NaN values; whether there were any.
template <int VT>
__device__ __forceinline__ bool drop_nan(uint4v (&vw)[VT]) {
  uint32_t any = 0u;
#pragma unroll
  for (int i = 0; i < VT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t n = nan_bytes(vw[i][j]);
      any |= n;
      vw[i][j] &= ~((n >> 7) * 0xFFu);
    }
  return any != 0u;
}

// Partial results of one range of keys, float32: for `rows` rows the sums, as
// [channel pair of four: 0, 1 / 2, 3][D / 4][rows] pairs, then [rows] pairs
// (maximum, sum of weights). Rows are neighbours in both kernels' lanes, so
// every store and load of 8 bytes a lane covers whole lines. They cross XCDs
// (each with its own L2) like the GEMMs' split-K slabs: agent-scope relaxed
// stores and loads.
template <int D>
struct Partial {
  uint64_t* p;
  int rows;
  static __device__ __forceinline__ int64_t floats(int rows) { return (int64_t)rows * (D + 2); }
  __device__ __forceinline__ Partial(float* slab, int z, int rows)
      : p(reinterpret_cast<uint64_t*>(slab + z * floats(rows))), rows(rows) {}
  static __device__ __forceinline__ void put(uint64_t* q, float a, float b) {
    __hip_atomic_store(q, __builtin_bit_cast(uint64_t, float2v{a, b}), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  static __device__ __forceinline__ float2v get(uint64_t* q) {
    return __builtin_bit_cast(float2v, __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  }
  __device__ __forceinline__ void put4(int row, int d4, const float4v& v) const {
    put(p + d4 * rows + row, v[0], v[1]);
    put(p + (D / 4 + d4) * rows + row, v[2], v[3]);
  }
  __device__ __forceinline__ float4v get4(int row, int d4) const {
    const float2v a = get(p + d4 * rows + row), b = get(p + (D / 4 + d4) * rows + row);
    return float4v{a[0], a[1], b[0], b[1]};
  }
  __device__ __forceinline__ void put_ml(int row, float m, float l) const { put(p + (D / 2) * rows + row, m, l); }
  __device__ __forceinline__ float2v get_ml(int row) const { return get(p + (D / 2) * rows + row); }
  __device__ __forceinline__ void put_nan(int row, int d) const {
    float* f = reinterpret_cast<float*>(p + ((d % 4 / 2) * (D / 4) + d / 4) * rows + row) + d % 2;
    __hip_atomic_store(f, __builtin_nanf(""), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
};

// Four consecutive channels of one output row (sum / l; a row that sees no key
// gives zeros), and the row's log-sum-exp once.
struct OutRow {
  uint16_t* p;
  float* lse;
};
__device__ __forceinline__ OutRow out_row(const AttnArgs& a, const SeqSpan& s, int kv_head, int row) {
  const Row r = row_of(a, row);
  const int64_t t = s.row0 + r.token;
  const int head = kv_head * a.group + r.head;
  return OutRow{a.out + t * a.o_ld_token + head * a.o_ld_head, a.lse == nullptr ? nullptr : a.lse + t * a.Hq + head};
}
__device__ __forceinline__ void put_out4(const OutRow& q, int d, const float4v& o, float l, float r) {
  uint16_t* dst = q.p + d;
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = l == 0.0f ? 0u : f32_to_bf16_bits(o[i] * r);
  if ((reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
    *reinterpret_cast<uint64_t*>(dst) = (uint64_t)(b[0] | (b[1] << 16)) | ((uint64_t)(b[2] | (b[3] << 16)) << 32);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = (uint16_t)b[i];
  }
}
__device__ __forceinline__ void put_lse(const OutRow& q, float m, float l) {
  if (q.lse != nullptr) *q.lse = l == 0.0f ? neg_inf() : kLn2 * m + __logf(l);
}
__device__ __forceinline__ void write_out4(const AttnArgs& a, const SeqSpan& s, int kv_head, int row, int d,
                                           const float4v& o, float m, float l) {
  const OutRow q = out_row(a, s, kv_head, row);
  put_out4(q, d, o, l, l == 0.0f ? 0.0f : 1.0f / l);
  if (d == 0) put_lse(q, m, l);
}

// A running softmax-weighted sum of four channels of one row.
struct Joined {
  float m, l;
  float4v o;
  __device__ __forceinline__ void add(float m2, float l2, const float4v& o2) {
    const float top = __builtin_fmaxf(m, m2);
    const float safe = top == neg_inf() ? 0.0f : top;
    const float a = exp2_fast(m - safe), b = exp2_fast(m2 - safe);
    l = l * a + l2 * b;
    o = o * a + o2 * b;
    m = top;
  }
};

// The last workgroup of a row tile to arrive joins the ranges' results. An
// item is four channels of one row. NT threads; where there are fewer items
// than threads, PT threads share an item (ranges p, p + PT, ...) and join
// through LDS (`lds`: NT * 24 bytes), else a thread takes items in turn. Loads
// are issued in rounds of 8 to 16 before any is used; every sum has a fixed
// order.
template <int D, int NT>
__device__ __forceinline__ void join_ranges(const AttnArgs& a, const SeqSpan& s, int kv_head, int row0, int rows,
                                            int ns, float* slab, float* lds) {
  const int items = rows * (D / 4), tid = threadIdx.x;
  if (items >= NT || ns <= 8) {
    constexpr int U = 2, Z = 4;  // items, ranges a round
    for (int i0 = tid; i0 < items; i0 += NT * U) {
      Joined acc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) acc[u] = Joined{neg_inf(), 0.0f, float4v{0.f, 0.f, 0.f, 0.f}};
      for (int z0 = 0; z0 < ns; z0 += Z) {
        float2v ml[U][Z];
        float4v o[U][Z];
#pragma unroll
        for (int z = 0; z < Z; ++z)
          if (z0 + z < ns) {
            const Partial<D> p(slab, z0 + z, rows);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int i = i0 + NT * u < items ? i0 + NT * u : i0;
              ml[u][z] = p.get_ml(i % rows);
              o[u][z] = p.get4(i % rows, i / rows);
            }
          }
#pragma unroll
        for (int z = 0; z < Z; ++z)
          if (z0 + z < ns)
#pragma unroll
            for (int u = 0; u < U; ++u) acc[u].add(ml[u][z][0], ml[u][z][1], o[u][z]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + NT * u;
        if (i < items) write_out4(a, s, kv_head, row0 + i % rows, i / rows * 4, acc[u].o, acc[u].m, acc[u].l);
      }
    }
    return;
  }
  const int PT = NT / items, part = tid / items, i = tid % items;
  Joined acc = {neg_inf(), 0.0f, float4v{0.f, 0.f, 0.f, 0.f}};
  if (part < PT) {
    constexpr int Z = 8;
    for (int z0 = part; z0 < ns; z0 += PT * Z) {
      float2v ml[Z];
      float4v o[Z];
#pragma unroll
      for (int z = 0; z < Z; ++z) {
        const int zz = z0 + PT * z < ns ? z0 + PT * z : z0;
        const Partial<D> p(slab, zz, rows);
        ml[z] = p.get_ml(i % rows);
        o[z] = p.get4(i % rows, i / rows);
      }
#pragma unroll
      for (int z = 0; z < Z; ++z)
        if (z0 + PT * z < ns) acc.add(ml[z][0], ml[z][1], o[z]);
    }
    float* q = lds + tid * 6;
    q[0] = acc.m; q[1] = acc.l; q[2] = acc.o[0]; q[3] = acc.o[1]; q[4] = acc.o[2]; q[5] = acc.o[3];
  }
  __syncthreads();
  if (part != 0) return;
  for (int t = 1; t < PT; ++t) {
    const float* q = lds + (t * items + i) * 6;
    acc.add(q[0], q[1], float4v{q[2], q[3], q[4], q[5]});
  }
  write_out4(a, s, kv_head, row0 + i % rows, i / rows * 4, acc.o, acc.m, acc.l);
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

// A NaN value of a token that some rows of a row tile see and others do not
// would reach all of them through the matrix product (0 * NaN). The kernels
// leave NaN values of such tiles of 64 tokens out of the product and, where
// one was there (s_nan), make NaN of the outputs that see it here, after they
// were written: straight (part null) or in the partial results.
template <int D>
__device__ void put_nan_rows(const AttnArgs& a, const PagedCache& c, const PagedBatch& pb, const SeqSpan& s, int b,
                             int h, int bs_shift, int row0, int nrows, int k0, int k1, const Visible& first,
                             const Visible& last, const Partial<D>* part) {
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's outputs are written
  __syncthreads();
  for (int t0 = k0; t0 < k1; t0 += 64) {
    if (t0 + 64 <= first.hi && t0 >= last.lo) continue;  // every row sees these
    for (int t = t0; t < t0 + 64 && t < k1; ++t) {
      const int64_t blk = pb.table[(int64_t)b * pb.ld_table + (t >> bs_shift)];
      if (blk < 0 || blk >= c.num_blocks) continue;
      const int off = t & (c.block_size - 1);
      const uint8_t* v = c.v + ((blk * c.heads + h) * (c.block_size / 16) + off / 16) * (D * 16) + off % 16;
      for (int d = threadIdx.x; d < D; d += blockDim.x) {
        if ((v[d * 16] & 0x7F) != 0x7F) continue;
        for (int r = 0; r < nrows; ++r) {
          const Visible w = visible_keys(s, row_of(a, row0 + r).token, a.causal, a.window);
          if (t < w.lo || t >= w.hi) continue;
          if (part != nullptr) part->put_nan(r, d);
          else out_row(a, s, h, row0 + r).p[d] = 0x7FC0;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// few rows: every wave its own keys
// ---------------------------------------------------------------------------
//
// NC tiles of 16 rows; the W waves of a workgroup (eight where their registers
// allow it: the more, the fewer ranges have to be joined across workgroups)
// take 64-token tiles in turn and keep their own running maximum, sum and
// output, joined through LDS at the end. The call is a stream over the cache:
// codes go straight from memory into registers (16-byte loads; keys: a lane's
// 16 bytes of 4 neighbouring lanes make 64 bytes of a row, values: 256-byte
// runs), the next tile's keys are loaded while this tile's weights and values
// are worked on and the other way round, so about one tile of keys or values
// per wave is always in flight and no barrier is in the loop.
//
// Bound by memory: 64 sequences of up to 16384 tokens, 64 query and 8 kv heads
// of 128 channels: 1.34 GB in 246 to 259 us, 5.2 to 5.4 TB/s (a large copy: 5.0, a
// bare read: 6.6). Part of the distance is the end, where the longest sequences
// run alone: 64 equal ones of 16384 reach 5.6 (head_dim 64 5.2, 256 5.8). One
// sequence of 1000 tokens is a chain of dependent accesses (lengths, table,
// keys, values, partial results, arrival, join): 8.9 us for 2 MB.
//
// v_mfma_f32_16x16x32_bf16: A lane l holds row l % 16, k = 8 (l / 16) + j;
// B column l % 16, the same k; the result column l % 16, rows 4 (l / 16) + i.
//   S^T tile a (0..3) of 64 tokens: row r is token 16 (r / 4) + 4 a + r % 4,
//     so lane group g = l / 16 ends up with tokens 16 g + 4 a + i.
//   The contraction over D in step s: k = 8 g + j is channel
//     64 (s / 2) + 16 g + 8 (s % 2) + j (keys and queries alike).
//   O^T step s (0, 1): k = 8 g + j is token 16 g + 8 s + j, byte 8 s + j of the
//     lane's 16-byte piece of channel l % 16.
constexpr int stream_waves(int D, int NC) { return D * NC <= 128 || D == 128 ? 8 : 4; }

template <int D, int NC>
__global__ __launch_bounds__(64 * stream_waves(D, NC)) void attn_kv8_stream_kernel(const AttnArgs a, const PagedCache c,
                                                              const PagedBatch pb, int bs_shift, int row_tiles,
                                                              int splits, int chunk, float* partial,
                                                              uint32_t* counters) {
  constexpr int KI = D / 64, VT = D / 16, SK = D / 32, W = stream_waves(D, NC), STEP = 64 * W;
  __shared__ float4v so[W][NC * VT][64];
  __shared__ float2v sml[W][NC][16];
  __shared__ uint32_t s_flag, s_nan;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int h = blockIdx.x, b = blockIdx.y, H = c.heads, bs = c.block_size;
  const int z = splits == 1 ? 0 : (int)blockIdx.z / row_tiles;
  const int rt = (int)blockIdx.z - z * row_tiles;
  const SeqSpan s = seq_span(pb, b, bs);
  const int rows = s.n * a.group, row0 = rt * 16 * NC;
  if (row0 >= rows) return;
  const int last_row = row0 + 16 * NC < rows ? row0 + 16 * NC - 1 : rows - 1;
  // every row sees [last.lo, first.hi), some row each of [first.lo, last.hi)
  const Visible first = visible_keys(s, row_of(a, row0).token, a.causal, a.window);
  const Visible last = visible_keys(s, row_of(a, last_row).token, a.causal, a.window);
  const int kmin = first.lo & ~63, kmax = last.hi;
  int ns = 1;
  if (splits > 1) {
    ns = kmax > kmin ? (kmax - kmin + chunk - 1) / chunk : 1;
    ns = ns < splits ? ns : splits;
  }
  if (z >= ns) return;
  const int k0 = kmin + z * chunk;
  const int k1 = z == ns - 1 || k0 + chunk > kmax ? kmax : k0 + chunk;

  if (tid == 0) s_nan = 0u;
  __syncthreads();

  // this lane's columns (query rows)
  bf16x8 q[NC][SK];
  int vlo[NC], vhi[NC];
#pragma unroll
  for (int t = 0; t < NC; ++t) {
    const int row = row0 + 16 * t + col;
    const bool ok = row < rows;
    const Row rw = row_of(a, ok ? row : 0);
    const Visible v = visible_keys(s, rw.token, a.causal, a.window);
    vlo[t] = v.lo;
    vhi[t] = ok ? v.hi : 0;
    const uint16_t* qp = a.q + (s.row0 + rw.token) * a.q_ld_token + (int64_t)(h * a.group + rw.head) * a.q_ld_head;
#pragma unroll
    for (int i = 0; i < SK; ++i) {
      q[t][i] = load_q8(qp + 64 * (i / 2) + 16 * g + 8 * (i % 2), a.aligned);
      if (!ok)
#pragma unroll
        for (int j = 0; j < 8; ++j) q[t][i][j] = (__bf16)0.0f;
    }
  }
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

  const uint64_t page_bytes = (uint64_t)H * bs * D;
  const uint8_t* kbase = c.k + (int64_t)h * bs * D + (col & 3) * D + 16 * g;
  const uint8_t* vbase = c.v + (int64_t)h * bs * D + col * 16;
  const int32_t* table = pb.table + (int64_t)b * pb.ld_table;
  // Blocks are looked up two tiles ahead, before that tile's loads are issued:
  // loads return in order, so a table entry asked for any later would make the
  // next keys wait for all loads before it. Past the last key the last entry
  // is taken; kmax <= len <= the table's capacity.
  struct Entries {
    int k, v;  // of this lane's keys (tokens 16 (col / 4) ..) and of its values and scales (16 g ..)
  };
  auto look_up = [&](int t0) -> Entries {
    const int tk = t0 + 16 * (col >> 2), tv = t0 + 16 * g;
    return Entries{table[(tk < kmax ? tk : kmax - 1) >> bs_shift], table[(tv < kmax ? tv : kmax - 1) >> bs_shift]};
  };
  uint4v kw[4][KI], vw[VT];
  uint32_t ksb = 0, vsb = 0;
  bool there = false;  // whether the block of this lane's tokens is in the cache
  // loads of a tile; a block that is not there is read from block 0 and masked
  auto load_k = [&](int t0, const Entries& e) {
    const int t = t0 + 16 * (col >> 2);
    const uint32_t blk = (uint32_t)e.k < (uint32_t)c.num_blocks ? (uint32_t)e.k : 0u;
    const uint8_t* p = kbase + blk * page_bytes + (uint32_t)((t & (bs - 1)) * D);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < KI; ++j) kw[i][j] = *reinterpret_cast<const uint4v*>(p + i * 4 * D + j * 64);
  };
  auto load_v = [&](int t0, const Entries& e) {
    const int t = t0 + 16 * g;
    there = (uint32_t)e.v < (uint32_t)c.num_blocks;
    const uint32_t blk = there ? (uint32_t)e.v : 0u, at = blk * (uint32_t)H + (uint32_t)h;
    ksb = c.k_scale[at];
    vsb = c.v_scale[at];
    const uint8_t* p = vbase + blk * page_bytes + (uint32_t)((t & (bs - 1)) * D);
#pragma unroll
    for (int i = 0; i < VT; ++i) vw[i] = *reinterpret_cast<const uint4v*>(p + i * 256);
  };

  int t0 = k0 + 64 * wave;
  Entries next = {0, 0}, after = {0, 0};
  if (t0 < k1) {
    next = look_up(t0);
    after = look_up(t0 + STEP);
    load_k(t0, next);
    load_v(t0, next);
  }
  for (; t0 < k1; t0 += STEP) {
    const bool more = t0 + STEP < k1;
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
    const bool in = there;
    const float ks = e8m0(ksb) * sl2;
    float vs = e8m0(vsb);
    next = after;
    if (more) {
      after = look_up(t0 + 2 * STEP);
      load_k(t0 + STEP, next);
    }
    const int tg = t0 + 16 * g;  // this lane's 16 tokens start here
    // Masked in edge tiles only: keys hidden from some row, past this range
    // (the ranges meet at multiples of 64, so only past kmax) or of a block
    // that is not there.
    const bool edge = t0 < last.lo || t0 + 64 > first.hi || t0 + 64 > k1 || __any(!in);
    if (edge) {
      const int have = in ? clamp16(k1 - tg) : 0, skip = clamp16(first.lo - tg);
#pragma unroll
      for (int t = 0; t < NC; ++t) {
        const int lo = clamp16(vlo[t] - tg), hi = clamp16(vhi[t] - tg);
        const int top = hi < have ? hi : have;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[t][i] = i >= lo && i < top ? x[t][i] * ks : neg_inf();
      }
      // Values of tokens that no row sees may hold anything, and 0 * NaN is
      // not 0: they are zeroed.
      mask_values<VT>(vw, have, skip);
      if (skip >= have) vs = 0.0f;  // and so may their block's scale (0 * 2^128)
      // NaN where rows differ in what they see: see put_nan_rows
      if ((t0 < last.lo || t0 + 64 > first.hi) && drop_nan<VT>(vw)) s_nan = 1u;
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
    if (more) load_v(t0 + STEP, next);
  }

  // join the waves
#pragma unroll
  for (int t = 0; t < NC; ++t) {
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (g == 0) sml[wave][t][col] = float2v{m[t], l[t]};
#pragma unroll
    for (int i = 0; i < VT; ++i) so[wave][t * VT + i][lane] = o[t][i];
  }
  __syncthreads();
  const int tile = (b * H + h) * row_tiles + rt;
  const int nrows = last_row - row0 + 1;
  float* slab = partial + (int64_t)tile * splits * Partial<D>::floats(16 * NC);
  const Partial<D> mine(slab, z, nrows);
  for (int f = wave; f < NC * VT; f += W) {
    const int t = f / VT, i = f % VT;
    float M = neg_inf();
#pragma unroll
    for (int w = 0; w < W; ++w) M = __builtin_fmaxf(M, sml[w][t][col][0]);
    const float safe = M == neg_inf() ? 0.0f : M;
    float L = 0.0f;
    float4v sum = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2v ml = sml[w][t][col];
      const float f2 = exp2_fast(ml[0] - safe);
      L += f2 * ml[1];
      sum += f2 * so[w][f][lane];
    }
    const int row = 16 * t + col, d = 16 * i + 4 * g;
    if (row0 + row >= rows) continue;
    if (ns == 1) {
      write_out4(a, s, h, row0 + row, d, sum, M, L);
    } else {
      mine.put4(row, d / 4, sum);
      if (d == 0) mine.put_ml(row, M, L);
    }
  }
  if (s_nan != 0u)
    put_nan_rows<D>(a, c, pb, s, b, h, bs_shift, row0, nrows, k0, k1, first, last,
                    ns == 1 ? nullptr : &mine);
  if (ns == 1) return;
  if (last_to_arrive(counters + tile, ns, &s_flag))
    join_ranges<D, 64 * W>(a, s, h, row0, nrows, ns, slab, reinterpret_cast<float*>(&so[0][0][0]));
}

// ---------------------------------------------------------------------------
// many rows: keys and values shared through LDS
// ---------------------------------------------------------------------------
//
// 32 rows a wave, NW waves a workgroup. Tiles of 64 tokens are widened to
// bf16 once per workgroup, on their way into LDS (two buffers; the next tile's
// codes are loaded at the start of a tile's work and written to the other
// buffer at its end, one barrier a tile).
//
// v_mfma_f32_32x32x16_bf16: A lane l holds row l % 32, k = 8 (l / 32) + j; B
// column l % 32, the same k; result register r: column l % 32, row
// 8 (r / 4) + 4 (l / 32) + r % 4.
//   S^T: row rho of 32 tokens is token 16 ((rho / 4) % 2) + 4 (rho / 8) + rho % 4,
//     so register r of lane half hf is token 16 hf + r.
//   O^T step s (0, 1): k = 8 hf + j is token 16 hf + 8 s + j.
// LDS: keys [64 rows in S^T order][D], values [D][64 tokens], in 16-byte
// chunks; a row's chunks are exchanged by an XOR with its number so that the
// 16 rows a quarter-wave reads at one chunk lie in 16 different bank groups.
//
// The running maximum moves only when a tile exceeds it by more than 2^8 (the
// weights then stay below 2^8, which costs no precision): the accumulators
// are rescaled a few times a row instead of at every tile. Tiles with a value
// scale outside 2^+-100 move it at once.
//
// Bound by the issue of vector instructions beside the matrix ones: a wave's 32
// products of a tile take 1024 cycles, its 32 exponentials 512 and the rest of
// the softmax, widening and addressing 500 to 740. 8192 causal tokens, 32 query
// and 8 kv heads of 128 channels: 570 to 640 us by the card and its clock, 860
// to 965 TFLOP/s (a large bf16 matrix product: 1140); four prompts of up to 2048
// tokens 99 us, 725 TFLOP/s, the starts and ends of their short workgroups being
// the rest; head_dim 64 630 to 700 TFLOP/s (per product the softmax weighs twice),
// 256 700 (one workgroup a CU).
// Tried at this size and slower: scales folded into the widening (640 us), the
// softmax interleaved with the products by hand, waves with raised priority.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void attn_kv8_tile_kernel(
    const AttnArgs a, const PagedCache c, const PagedBatch pb, int bs_shift, int row_tiles, int splits, int chunk,
    float* partial, uint32_t* counters) {
  constexpr int T = 64 * NW, ROWS = 32 * NW;
  constexpr int KP = 4 * D / T;                  // 16-byte pieces of keys (and of values) a thread stages
  constexpr int KC = D / 8;                      // 16-byte chunks of a key row in LDS
  constexpr int SK = D / 16, VT = D / 32;
  static_assert(KP >= 1 && 4 * D % T == 0 && T % D == 0 && D % 64 == 0, "a wave's pieces in one group");
  __shared__ uint4v sk[2][64 * KC];
  __shared__ uint4v sv[2][D * 8];
  __shared__ float4v ss[2][4];  // per group of 16 tokens: score factor (-1: no block), see stage_scales
  __shared__ uint32_t s_flag, s_nan;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hf = lane >> 5;
  // Workgroups go in turn to the XCDs and, within one, to its four shader
  // engines, so with blockIdx.y taken as it is the long sequences of a batch of
  // 2, 4 or 8 would all run on the same engines: the assignment moves on by one
  // every second blockIdx.z (prompts of 2048, 1098, 1685, 736 tokens, 32 heads:
  // 154 -> 104 us).
  const int h = blockIdx.x, H = c.heads, bs = c.block_size;
  const int b = gridDim.y == 1 ? 0 : (int)((blockIdx.y + blockIdx.z / 2) % gridDim.y);
  const int z = splits == 1 ? 0 : (int)blockIdx.z / row_tiles;
  // The last row tiles see the most keys under a causal mask: they start first.
  // Where all workgroups run at once, two a CU, the second half starts with the
  // fewest, so that long ones get short neighbours (a prompt of 2048 tokens, 32
  // heads: 66 -> 59 us).
  const int ri = (int)blockIdx.z - z * row_tiles, upper = (row_tiles + 1) / 2;
  const bool at_once = D != 256 && gridDim.x * gridDim.y * gridDim.z <= 512;
  const int rt = at_once && ri >= upper ? ri - upper : row_tiles - 1 - ri;
  const SeqSpan s = seq_span(pb, b, bs);
  const int rows = s.n * a.group, row0 = rt * ROWS;
  if (row0 >= rows) return;
  const int last_row = row0 + ROWS < rows ? row0 + ROWS - 1 : rows - 1;
  const Visible first = visible_keys(s, row_of(a, row0).token, a.causal, a.window);
  const Visible last = visible_keys(s, row_of(a, last_row).token, a.causal, a.window);
  const int kmin = first.lo & ~63, kmax = last.hi;
  int ns = 1;
  if (splits > 1) {
    ns = kmax > kmin ? (kmax - kmin + chunk - 1) / chunk : 1;
    ns = ns < splits ? ns : splits;
  }
  if (z >= ns) return;
  const int k0 = kmin + z * chunk;
  const int k1 = z == ns - 1 || k0 + chunk > kmax ? kmax : k0 + chunk;
  if (tid == 0) s_nan = 0u;
  __syncthreads();

  // this lane's query row, and the keys that all (some) rows of the wave see
  const int wrow = row0 + 32 * wave, row = wrow + col;
  const bool ok = row < rows;
  const Row rw = row_of(a, ok ? row : 0);
  const Visible mine = visible_keys(s, rw.token, a.causal, a.window);
  const int vlo = mine.lo, vhi = ok ? mine.hi : 0;
  const Visible wave_last = visible_keys(s, row_of(a, wrow + 31 < rows ? wrow + 31 : rows - 1).token, a.causal, a.window);
  const int wave_all_lo = wave_last.lo;
  const int wave_all_hi = visible_keys(s, row_of(a, wrow < rows ? wrow : rows - 1).token, a.causal, a.window).hi;
  const int wave_any_hi = wrow < rows ? wave_last.hi : 0;
  bf16x8 q[SK];
  {
    const uint16_t* qp = a.q + (s.row0 + rw.token) * a.q_ld_token + (int64_t)(h * a.group + rw.head) * a.q_ld_head + 8 * hf;
#pragma unroll
    for (int i = 0; i < SK; ++i) {
      q[i] = load_q8(qp + 16 * i, a.aligned);
      if (!ok)
#pragma unroll
        for (int j = 0; j < 8; ++j) q[i][j] = (__bf16)0.0f;
    }
  }

  const float sl2 = a.scale * kLog2e;
  float m = neg_inf(), l = 0.0f;
  float16v o[VT];
#pragma unroll
  for (int i = 0; i < VT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;

  // Staging. A tile's four groups of 16 tokens are 16 D contiguous bytes each,
  // of keys as of values, in one block: a thread takes the 16-byte piece pd of
  // one group in every pass, so a wave's group, its block and its scales are
  // scalars. Blocks are looked up one tile ahead of the loads.
  const int pd = tid % D, g0 = __builtin_amdgcn_readfirstlane(tid / D);
  constexpr int GS = T / D;  // groups a pass
  const int32_t* table = pb.table + (int64_t)b * pb.ld_table;
  const uint32_t head_bytes = (uint32_t)(bs * D);
  uint4v kw[KP], vw[KP];
  int blk[KP], entry[KP];  // blocks of the tile loaded last, table entries of the one after it
  uint32_t ksb[KP], vsb[KP];
  // Past the last key the last entry is looked up, and its block (or block 0
  // where it is none) is read and masked.
  auto look_up = [&](int t0) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int t = t0 + 16 * (g0 + GS * i);
      entry[i] = table[(t < kmax ? t : kmax - 1) >> bs_shift];
    }
  };
  auto load_tile = [&](int t0) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int e = __builtin_amdgcn_readfirstlane(entry[i]);
      const bool in = (uint32_t)e < (uint32_t)c.num_blocks;
      blk[i] = in && t0 + 16 * (g0 + GS * i) < kmax ? e : -1;
      const uint32_t at = (uint32_t)(in ? e : 0) * (uint32_t)H + (uint32_t)h;  // num_blocks * heads < 2^31
      const int off = (t0 + 16 * (g0 + GS * i)) & (bs - 1);
      const uint64_t base = (uint64_t)at * head_bytes + (uint32_t)(off * D);
      kw[i] = *reinterpret_cast<const uint4v*>(c.k + base + 16 * pd);
      vw[i] = *reinterpret_cast<const uint4v*>(c.v + base + 16 * pd);
      ksb[i] = c.k_scale[at];
      vsb[i] = c.v_scale[at];
    }
  };
  // Edges of the values loaded: tokens that no row sees may hold anything, they
  // become zeros; NaN where rows differ in what they see: see put_nan_rows.
  auto trim_values = [&](int t0) {
    bool absent = false;
#pragma unroll
    for (int i = 0; i < KP; ++i) absent |= blk[i] < 0;
    const bool differ = t0 + 64 > first.hi || t0 < last.lo;  // put_nan_rows' condition
    if (differ || absent) {
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        uint4v u[1] = {vw[i]};
        const int t = t0 + 16 * (g0 + GS * i);
        mask_values<1>(u, blk[i] < 0 ? 0 : clamp16(kmax - t), clamp16(first.lo - t));
        if (differ && drop_nan<1>(u)) s_nan = 1u;
        vw[i] = u[0];
      }
    }
  };
  auto widen_tile = [&](int buf) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int g = g0 + GS * i;
      const int tok = pd / (D / 16), kc = pd % (D / 16);
      const int lrow = 32 * (g >> 1) + 8 * (tok >> 2) + 4 * (g & 1) + (tok & 3);
      const int key = D == 64 ? (lrow >> 1) & 7 : lrow & 15, vkey = (pd >> 1) & 7;
      uint4v* kd = &sk[buf][lrow * KC];
      kd[(2 * kc) ^ key] = __builtin_bit_cast(uint4v, widen8(kw[i][0], kw[i][1]));
      kd[(2 * kc + 1) ^ key] = __builtin_bit_cast(uint4v, widen8(kw[i][2], kw[i][3]));
      uint4v* vd = &sv[buf][pd * 8];
      vd[(2 * g) ^ vkey] = __builtin_bit_cast(uint4v, widen8(vw[i][0], vw[i][1]));
      vd[(2 * g + 1) ^ vkey] = __builtin_bit_cast(uint4v, widen8(vw[i][2], vw[i][3]));
    }
  };
  auto stage_scales = [&](int buf) {
    if (pd == 0) {
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        // the weights take the value scale 2^ev in their exponent; what lies
        // outside +-100 (no exponent's bits are lost there) is a factor of its own
        const int ev = blk[i] < 0 ? 0 : (int)vsb[i] - 127;
        const int e = ev < -100 ? -100 : (ev > 100 ? 100 : ev);
        ss[buf][g0 + GS * i] =
            float4v{blk[i] < 0 ? -1.0f : e8m0(ksb[i]) * sl2, (float)e, __uint_as_float((uint32_t)(127 - e) << 23),
                    __uint_as_float((uint32_t)(127 + ev - e) << 23)};
      }
    }
  };

  if (k0 < k1) {
    look_up(k0);
    load_tile(k0);
    look_up(k0 + 64);
    trim_values(k0);
    widen_tile(0);
    stage_scales(0);
  }
  int buf = 0;
  for (int t0 = k0; t0 < k1; t0 += 64, buf ^= 1) {
    __syncthreads();
    load_tile(t0 + 64);  // after the last tile: masked, and never read
    look_up(t0 + 128);
    if (t0 >= wave_any_hi) {  // no row of this wave sees the tile
      trim_values(t0 + 64);
      widen_tile(buf ^ 1);
      stage_scales(buf ^ 1);
      continue;
    }
    float16v x[2];
#pragma unroll
    for (int r = 0; r < 16; ++r) x[0][r] = x[1][r] = 0.0f;
    const int key = D == 64 ? (col >> 1) & 7 : col & 15;  // of rows col and 32 + col alike
    // Fragments are read in batches ahead of the products: left to itself the
    // compiler reads each just before its use, and every pair of products then
    // waits out an LDS access.
    constexpr int KB = 8, VB = 4;
#pragma unroll
    for (int f0 = 0; f0 < 2 * SK; f0 += KB) {
      uint4v kf[KB];
#pragma unroll
      for (int f = 0; f < KB; ++f) kf[f] = sk[buf][(32 * (f % 2) + col) * KC + ((2 * ((f0 + f) / 2) + hf) ^ key)];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = 0; f < KB; ++f)
        x[f % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[f]), q[(f0 + f) / 2], x[f % 2], 0, 0, 0);
    }
    // the first values arrive during the softmax
    uint4v vf[2][VB];
    auto read_v = [&](int f0, uint4v (&dst)[VB]) {
#pragma unroll
      for (int f = 0; f < VB; ++f) {
        const int j = (f0 + f) / VT, d = 32 * ((f0 + f) % VT) + col;
        dst[f] = sv[buf][d * 8 + ((4 * (j / 2) + 2 * hf + j % 2) ^ ((d >> 1) & 7))];
      }
    };
    read_v(0, vf[0]);
    const float4v sc[2] = {ss[buf][hf], ss[buf][2 + hf]};
    float kk[2] = {sc[0][0], sc[1][0]};
    if (t0 < wave_all_lo || t0 + 64 > wave_all_hi || t0 + 64 > k1 || __any(__builtin_fminf(kk[0], kk[1]) < 0.0f)) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int tg = t0 + 32 * half + 16 * hf;
        const int have = kk[half] < 0.0f ? 0 : clamp16(k1 - tg);
        const int lo = clamp16(vlo - tg), hi = clamp16(vhi - tg);
        const int upto = hi < have ? hi : have;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[half][r] = r >= lo && r < upto ? x[half][r] * kk[half] : neg_inf();
        kk[half] = 1.0f;
      }
    }
    float top = neg_inf();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float t = x[half][0];
#pragma unroll
      for (int r = 1; r < 16; ++r) t = __builtin_fmaxf(t, x[half][r]);
      top = __builtin_fmaxf(top, t * kk[half]);  // kk >= 0
    }
    {
      const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
      top = __builtin_fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1]));
    }
    // weights of up to 2^8 times a value scale above 2^100 could leave float32
    const bool factor = __any(sc[0][3] != 1.0f || sc[1][3] != 1.0f);
    if (__any(top > (factor ? m : m + 8.0f))) {
      top = __builtin_fmaxf(top, m);
      const float back = exp2_fast(m - (top == neg_inf() ? 0.0f : top));
      l *= back;
#pragma unroll
      for (int i = 0; i < VT; ++i) o[i] *= back;
      m = top;
    }
    const float safe = m == neg_inf() ? 0.0f : m;
    trim_values(t0 + 64);
    bf16x8 p[2][2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float shift = sc[half][1] - safe;
      float w[16], sum = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        w[r] = exp2_fast(__builtin_fmaf(x[half][r], kk[half], shift));
        sum += w[r];
      }
      l += sum * sc[half][2];
      p[half][0] = round8(w);
      p[half][1] = round8(w + 8);
    }
    if (factor)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) p[j / 2][j % 2][e] = (__bf16)((float)p[j / 2][j % 2][e] * sc[j / 2][3]);  // exact
#pragma unroll
    for (int f0 = 0; f0 < 4 * VT; f0 += VB) {
      if (f0 + VB < 4 * VT) read_v(f0 + VB, vf[(f0 / VB + 1) % 2]);
#pragma unroll
      for (int f = 0; f < VB; ++f) {
        const int j = (f0 + f) / VT, i = (f0 + f) % VT;
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf[(f0 / VB) % 2][f]), p[j / 2][j % 2], o[i], 0, 0, 0);
      }
    }
    // the other buffer was last read before this tile's barrier
    widen_tile(buf ^ 1);
    stage_scales(buf ^ 1);
  }
  __syncthreads();  // the buffers are free, s_nan is whole

  {
    const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
  }
  const int tile = (b * H + h) * row_tiles + rt;
  const int nrows = last_row - row0 + 1;
  float* slab = partial + (int64_t)tile * splits * Partial<D>::floats(ROWS);
  const Partial<D> part(slab, z, nrows);
  if (ok) {
    const int lr = 32 * wave + col;
    const OutRow dst = out_row(a, s, h, row);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < VT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4v v = float4v{o[i][4 * r], o[i][4 * r + 1], o[i][4 * r + 2], o[i][4 * r + 3]};
        const int d = 32 * i + 8 * r + 4 * hf;
        if (ns == 1) put_out4(dst, d, v, l, inv);
        else part.put4(lr, d / 4, v);
      }
    if (hf == 0) {
      if (ns == 1) put_lse(dst, m, l);
      else part.put_ml(lr, m, l);
    }
  }
  if (s_nan != 0u)
    put_nan_rows<D>(a, c, pb, s, b, h, bs_shift, row0, nrows, k0, k1, first, last,
                    ns == 1 ? nullptr : &part);
  if (ns == 1) return;
  if (last_to_arrive(counters + tile, ns, &s_flag))
    join_ranges<D, T>(a, s, h, row0, nrows, ns, slab, reinterpret_cast<float*>(&sk[0][0]));
}

}  // namespace

// ---------------------------------------------------------------------------
// plan, launcher
// ---------------------------------------------------------------------------

static int rows_of(const AttnPlan& p) { return p.kind == 0 ? 16 * p.cols : 32 * p.cols; }

AttnPlan plan_attention(int B, int Hq, int Hkv, int D, int64_t max_new, int64_t max_len, int window) {
  AttnPlan p{};
  const int64_t rows = std::max<int64_t>(1, max_new) * (Hq / Hkv);
  p.kind = rows <= 32 ? 0 : 1;
  p.cols = p.kind == 1 ? 4 : rows <= 16 || D == 256 ? 1 : 2;
  p.row_tiles = (int)((rows + rows_of(p) - 1) / rows_of(p));
  const int64_t tiles = (int64_t)B * Hkv * p.row_tiles;
  // keys one row tile goes through; with a window it starts at a multiple of
  // 64 below its first visible key
  int64_t span = max_len < 1 ? 1 : max_len;
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + max_new - 1 + 63);
  // Ranges of keys. Every workgroup pays its start (about as long as one step
  // of 64 tokens a wave) and a call with several ranges their joining, so the
  // ranges are as few as fill the card: the count with the least rounds *
  // (steps + 1) + joining, a round being the workgroups that run at once. A
  // last step that not all waves take counts by its share, down to a half
  // (MI355X sweeps, 8 kv heads: 131072 tokens 57 us with 32 ranges, 77 with 16,
  // 63 with 64; 2000 tokens 9.7 us with 8, 10.1 with 4, 12.4 with 2; 1000 tokens
  // 9.0 with 4, 9.6 with 2, 9.3 with 8; eight sequences of up to 4096 tokens
  // 18.5 us with 4, 22 with 2, 23 with 8).
  int64_t splits = 1;
  if (p.kind == 0) {
    const int step = 64 * stream_waves(D, p.cols);
    const int64_t slots = D == 64 && p.cols == 1 ? 512 : 256;
    double best = 0.0;
    for (int64_t s = 1; s <= 64; ++s) {
      const int64_t keys = (span + s - 1) / s;
      const double steps = keys <= step / 2 ? 0.5 : (double)keys / step;
      const double cost = (double)((tiles * s + slots - 1) / slots) * (steps + 1.0) +
                          (s > 1 ? 0.75 + (double)s * (double)std::min<int64_t>(rows, rows_of(p)) / 512.0 : 0.0);
      if (s == 1 || cost < best) {
        best = cost;
        splits = s;
      }
      if (keys <= step / 2) break;  // more ranges only cost more
    }
  } else {
    // many rows: four rounds of workgroups (sequences differ in length), of at
    // least 2048 keys, which was measured where the tiles fill the card: with few
    // tiles shorter ranges would use more of it (8 tokens, 64 heads, on 4096 keys
    // 58 us in two ranges; 4 tokens, in the other kernel, 19). 512 and 274 new
    // tokens on 32768 and 17579, 64 heads: 1.03 ms whole, 1.00 in two ranges, 0.85 in four, 0.82 in eight; 512 each on
    // 32768: 1.14 in two and four, 1.17 in eight, 1.26 in ranges of 2048.
    splits = std::max<int64_t>(1, std::min<int64_t>((2048 + tiles - 1) / tiles, span / 2048));
  }
  // one arrival counter a tile, below the words a linear call keeps its device scalars in
  if (tiles > kWorkspaceScalarOffset / 4) splits = 1;
  int64_t chunk = round_up((span + splits - 1) / splits, 64);
  splits = (span + chunk - 1) / chunk;
  p.splits = (int)splits;
  p.chunk = (int)chunk;
  p.counter_bytes = kWorkspaceCounterBytes;
  p.partial_bytes = splits > 1 ? round_up(tiles * splits * rows_of(p) * (D + 2) * 4, 256) : 0;
  p.total_bytes = p.counter_bytes + p.partial_bytes;
  return p;
}

std::string describe_attention(const AttnPlan& p, int D) {
  char b[160];
  std::snprintf(b, sizeof(b), "%s<D=%d,%s=%d> row_tiles=%d splits=%d chunk=%d",
                p.kind == 0 ? "attn_kv8_stream_kernel" : "attn_kv8_tile_kernel", D, p.kind == 0 ? "NC" : "NW", p.cols,
                p.row_tiles, p.splits, p.chunk);
  return std::string(b);
}

hipError_t launch_attention(const AttnPlan& p, AttnArgs a, const PagedCache& c, const PagedBatch& pb,
                            uint8_t* workspace, hipStream_t st) {
  // n / group for n < 2^31: with 2^s >= group * 2^31 > 2^(s - 1) and mul =
  // floor(2^s / group) + 1 < 2^32, mul * group exceeds 2^s by at most group
  a.group = a.Hq / c.heads;
  a.group_shift = 31;
  while (((uint64_t)1 << (a.group_shift - 31)) < (uint64_t)a.group) ++a.group_shift;
  a.group_mul = (uint32_t)((((uint64_t)1 << a.group_shift) / (uint64_t)a.group) + 1);
  int shift = 4;
  while ((1 << shift) < c.block_size) ++shift;
  uint32_t* counters = reinterpret_cast<uint32_t*>(workspace);
  float* partial = reinterpret_cast<float*>(workspace + p.counter_bytes);
  const dim3 grid((unsigned)c.heads, (unsigned)pb.B, (unsigned)(p.row_tiles * p.splits));
#define FQL_A(KIND, KERNEL, DD, N, THREADS)                                                               \
  if (p.kind == KIND && c.D == DD && p.cols == N) {                                                       \
    KERNEL<DD, N><<<grid, THREADS, 0, st>>>(a, c, pb, shift, p.row_tiles, p.splits, p.chunk, partial,     \
                                            counters);                                                    \
    return hipGetLastError();                                                                             \
  }
  FQL_A(0, attn_kv8_stream_kernel, 64, 1, (64 * stream_waves(64, 1)))
  FQL_A(0, attn_kv8_stream_kernel, 64, 2, (64 * stream_waves(64, 2)))
  FQL_A(0, attn_kv8_stream_kernel, 128, 1, (64 * stream_waves(128, 1)))
  FQL_A(0, attn_kv8_stream_kernel, 128, 2, (64 * stream_waves(128, 2)))
  FQL_A(0, attn_kv8_stream_kernel, 256, 1, (64 * stream_waves(256, 1)))
  FQL_A(1, attn_kv8_tile_kernel, 64, 4, 256)
  FQL_A(1, attn_kv8_tile_kernel, 128, 4, 256)
  FQL_A(1, attn_kv8_tile_kernel, 256, 4, 256)
#undef FQL_A
  return hipErrorInvalidValue;
}

}  // namespace fql
