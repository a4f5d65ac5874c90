// The chosen experts' feed forward (gfx950): y_t = residual_t + sum_j w_tj
// down_e(act(up_e(x_t))), e = experts_tj, in the formats of the scaled-MFMA linear
// layers and INT8.
//
//   prepare   pairs (token, place) counted and placed by expert; x quantized, by token
//   product   up: rows gathered by the sorted order, activation, quantized or float32
//   quantize  the inner activation, from float32 (where the first product did not)
//   product   down: rows in sorted order, fp16 with a factor for 32 columns (few rows: float32)
//   combine   y_t = residual_t + the k rows of token t times their weights, float32
//
// A product's workgroup computes one tile of one expert: rows of its range of the
// sorted order, columns of its weight. An expert's row tiles that share columns are
// neighbours in the order of the workgroups, and every XCD takes a contiguous part
// of that order, so that a weight comes from HBM once and its row tiles share it in
// L2. The grid is the upper bound of tiles, known on the host; workgroups past the
// true number end at once.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdio>

#include "fql_device.h"
#include "fql_experts.h"
#include "experts_tile.h"
#include "experts_token.h"
#include "fql_gemm.h"
#include "sc_epilogue.h"
#include "sc_quant.h"

namespace fql {

namespace {

constexpr int64_t meta_bytes(int64_t pairs, int64_t up_tiles, int64_t down_tiles) {
  return 128 + 2 * (int64_t)kMaxExperts * (int64_t)sizeof(ExpertRange) + 4 * (up_tiles + down_tiles + 2 * pairs);
}
void meta_at(uint8_t* p, int64_t pairs, int64_t up_tiles, int64_t down_tiles, Meta (&m)[2]) {
  const int64_t tiles[2] = {up_tiles, down_tiles};
  ExpertRange* const ranges = reinterpret_cast<ExpertRange*>(p + 128);
  int* at = reinterpret_cast<int*>(ranges + 2 * kMaxExperts);
  for (int i = 0; i < 2; ++i) {
    m[i].total_tiles = reinterpret_cast<int*>(p + 64 * i);
    m[i].ranges = ranges + i * kMaxExperts;
    m[i].tile_expert = at;
    at += tiles[i];
  }
  m[0].row_pair = m[1].row_pair = at;
  m[0].pair_row = m[1].pair_row = at + pairs;
}

// ---------------------------------------------------------------------------
// sorting and quantizing
// ---------------------------------------------------------------------------

constexpr int kPrepThreads = 512;

// Counts the pairs of every expert, lays out their rows and tiles, places them.
// The order of an expert's rows is that of the atomics: no result depends on it
// (a product's row depends on its own activation row only).
// Each of `groups` workgroups places a part of the pairs, and counts all of them and
// those of the parts before its own: without a wait for another workgroup. (Placing
// is a scattered store a pair; one workgroup took 59 us for 32768 pairs.)
__device__ __forceinline__ void sort_pairs(const int32_t* __restrict__ experts, int64_t pairs, int E, int up_rows,
                                           int down_rows, int groups, const Meta& up, const Meta& down) {
  __shared__ int count[kMaxExperts], row_at[kMaxExperts];
  const int64_t per = (pairs + groups - 1) / groups;
  const int64_t mine0 = blockIdx.x * per, mine1 = mine0 + per < pairs ? mine0 + per : pairs;
  __shared__ int part_rows[kPrepThreads / 64], part_tiles[2][kPrepThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < E; e += kPrepThreads) count[e] = row_at[e] = 0;
  __syncthreads();
  // many pairs a thread at a time: their loads are in flight together
  constexpr int N = 16;
  auto load = [&](int64_t i0, int64_t i1, int (&e)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = i0 + tid + (int64_t)j * kPrepThreads;
      e[j] = i < i1 ? experts[i] : -1;
    }
  };
  for (int64_t i0 = 0; i0 < pairs; i0 += N * kPrepThreads) {
    int e[N];
    load(i0, pairs, e);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (e[j] >= 0 && e[j] < E) {
        atomicAdd(&count[e[j]], 1);
        if (i0 + tid + (int64_t)j * kPrepThreads < mine0) atomicAdd(&row_at[e[j]], 1);
      }
  }
  __syncthreads();
  // exclusive sums of rows and tiles over the experts, two experts a thread
  static_assert(kMaxExperts <= 2 * kPrepThreads, "experts a thread");
  int c[2], t[2][2];  // rows of an expert, its tiles in each product
  int rows = 0, tiles[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * tid + j;
    c[j] = e < E ? count[e] : 0;
    t[0][j] = (c[j] + up_rows - 1) / up_rows;
    t[1][j] = (c[j] + down_rows - 1) / down_rows;
    rows += c[j];
    tiles[0] += t[0][j];
    tiles[1] += t[1][j];
  }
  int rs = rows, ts[2] = {tiles[0], tiles[1]};
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int r1 = __shfl_up(rs, o), a1 = __shfl_up(ts[0], o), b1 = __shfl_up(ts[1], o);
    if (lane >= o) {
      rs += r1;
      ts[0] += a1;
      ts[1] += b1;
    }
  }
  if (lane == 63) {
    part_rows[wave] = rs;
    part_tiles[0][wave] = ts[0];
    part_tiles[1][wave] = ts[1];
  }
  __syncthreads();
  int row0 = rs - rows, tile0[2] = {ts[0] - tiles[0], ts[1] - tiles[1]}, all[2] = {0, 0};
  for (int w = 0; w < kPrepThreads / 64; ++w) {
    if (w < wave) {
      row0 += part_rows[w];
      tile0[0] += part_tiles[0][w];
      tile0[1] += part_tiles[1][w];
    }
    all[0] += part_tiles[0][w];
    all[1] += part_tiles[1][w];
  }
  if (tid == 0 && blockIdx.x == 0) {
    up.total_tiles[0] = all[0];
    down.total_tiles[0] = all[1];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * tid + j;
    if (e < E) {
      row_at[e] += row0;
      if (blockIdx.x == 0) {
        up.ranges[e] = ExpertRange{tile0[0], t[0][j], row0, c[j]};
        down.ranges[e] = ExpertRange{tile0[1], t[1][j], row0, c[j]};
        for (int i = 0; i < t[0][j]; ++i) up.tile_expert[tile0[0] + i] = e;
        for (int i = 0; i < t[1][j]; ++i) down.tile_expert[tile0[1] + i] = e;
      }
      row0 += c[j];
      tile0[0] += t[0][j];
      tile0[1] += t[1][j];
    }
  }
  __syncthreads();
  for (int64_t i0 = mine0; i0 < mine1; i0 += N * kPrepThreads) {
    int e[N], r[N];
    load(i0, mine1, e);
#pragma unroll
    for (int j = 0; j < N; ++j) r[j] = e[j] >= 0 && e[j] < E ? atomicAdd(&row_at[e[j]], 1) : -1;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t i = i0 + tid + (int64_t)j * kPrepThreads;
      if (r[j] >= 0) up.row_pair[r[j]] = (int)i;
      if (i < mine1) up.pair_row[i] = r[j];
    }
  }
}

struct QuantArgs {
  const void* x;  // bf16 or float32 [rows][ld]
  int64_t rows, K, ld;
  bool aligned;
  float inv_scale;
  ExpertRows out;
  uint8_t* codes;
  uint8_t* scales;
};

// Rows into the products' layout: a thread takes 32-blocks, the four of a chunk in
// neighbouring lanes; INT8, whose scale needs the whole row first, takes a row a
// workgroup. `unit` counts workgroups.
template <int F, typename X>
__device__ __forceinline__ void quant_rows(const QuantArgs& a, int64_t unit) {
  const int64_t nblk = a.out.ld_codes / (F == SC_MXFP4 ? 16 : 32);
  auto store = [&](int64_t m, int64_t b, const uint32_t* w) {
    uint8_t* const dst = a.codes + m * a.out.ld_codes;
    if (F == SC_MXFP4) {
      *reinterpret_cast<uint4v*>(dst + b * 16) = uint4v{w[0], w[1], w[2], w[3]};
    } else {
      *reinterpret_cast<uint4v*>(dst + b * 32) = uint4v{w[0], w[1], w[2], w[3]};
      *reinterpret_cast<uint4v*>(dst + b * 32 + 16) = uint4v{w[4], w[5], w[6], w[7]};
    }
  };
  auto load = [&](int64_t m, int64_t b, float v[32]) {
    if (b * 32 < a.K) load32(static_cast<const X*>(a.x) + m * a.ld + b * 32, a.aligned, v);
    else
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.0f;
  };
  if constexpr (F == SC_INT8) {
    __shared__ uint32_t tops[kPrepThreads / 64];
    const int64_t m = unit;
    uint32_t top = 0u;
    for (int64_t b = threadIdx.x; b < nblk; b += kPrepThreads) {
      float v[32];
      load(m, b, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) top = amax_bits(v[j], top);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const uint32_t u = (uint32_t)__shfl_xor((int)top, o);
      top = u > top ? u : top;
    }
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPrepThreads / 64; ++i) top = tops[i] > top ? tops[i] : top;
    const float s = int8_scale(top), r = safe_reciprocal(s);
    if (threadIdx.x == 0) *reinterpret_cast<float*>(a.scales + m * a.out.ld_scales) = s;
    for (int64_t b = threadIdx.x; b < nblk; b += kPrepThreads) {
      float v[32];
      load(m, b, v);
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = int8x4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], r);
      store(m, b, w);
    }
  } else {
    const int64_t i = unit * kPrepThreads + threadIdx.x;
    const bool inside = i < a.rows * nblk;
    const int64_t m = inside ? i / nblk : 0, b = inside ? i - m * nblk : 0;
    const bool valid = inside && b * 32 < a.K;
    float v[32];
    if (inside) load(m, b, v);
    else
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.0f;
    uint32_t w[8], sb = 0;
    float gs = 0.0f;
    quant_block32<F>(v, valid, a.inv_scale, w, sb, gs);
    if (!inside) return;
    if (!valid) {  // columns past K
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0u;
      sb = 0u;
    }
    store(m, b, w);
    if (F == SC_MXFP4 || F == SC_MXFP8) a.scales[m * a.out.ld_scales + b] = (uint8_t)sb;
    if (F == SC_FP8_BLOCK && (b & 3) == 0) *reinterpret_cast<float*>(a.scales + m * a.out.ld_scales + b) = gs;
  }
}

int64_t quant_units(int fmt, const QuantArgs& a) {
  if (fmt == SC_INT8) return a.rows;
  const int64_t nblk = a.out.ld_codes / (fmt == SC_MXFP4 ? 16 : 32);
  return (a.rows * nblk + kPrepThreads - 1) / kPrepThreads;
}

// The first workgroups sort while the others quantize.
template <int F>
__global__ __launch_bounds__(kPrepThreads) void experts_prepare_kernel(const int32_t* __restrict__ experts,
                                                                       int64_t pairs, int E, int up_rows, int down_rows,
                                                                       int groups, Meta up, Meta down, QuantArgs q) {
  if ((int)blockIdx.x < groups) sort_pairs(experts, pairs, E, up_rows, down_rows, groups, up, down);
  else quant_rows<F, uint16_t>(q, (int64_t)blockIdx.x - groups);
}

template <int F>
__global__ __launch_bounds__(kPrepThreads) void experts_quant_kernel(QuantArgs q) {
  quant_rows<F, float>(q, blockIdx.x);
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------

// LDS of one 128-deep chunk. Activation tiles: 16 rows of 128 (MXFP4: 64) bytes as
// they lie in memory, their 16-byte pieces exchanged (piece p of row r in place p ^
// swizzle(r)) so that the 16 lanes that read one piece of all rows spread over the
// banks. Weight tiles: the packed order, lane by lane.
template <int F, int WM, int WN, int MTW, int NTW>
struct Stage {
  static constexpr int H = Traits<F>::H;
  static constexpr int TA = WM * MTW, TB = WN * NTW;
  static constexpr int QA = (TA + 3) / 4, QB = TB / 4;
  static constexpr int NBS = (TB * 16 + 127) / 128;
  static constexpr int SA = Traits<F>::MX || Traits<F>::BLOCK ? QA : 0;
  static constexpr int SB = Traits<F>::MX ? QB : (Traits<F>::BLOCK ? NBS : 0);
  uint4v a[TA][H][64];
  uint4v b[TB][H][64];
  uint32_t as[SA > 0 ? SA : 1][64];
  uint32_t bs[SB > 0 ? SB : 1][64];
};

template <int F>
__device__ __forceinline__ int swizzle(int r) {
  return F == SC_MXFP4 ? (r >> 2) & 3 : (r >> 1) & 7;
}

template <int F, int WM, int WN, int MTW, int NTW, int ST, bool UP>
__global__ __launch_bounds__(64 * WM * WN) void experts_product_kernel(const ProductArgs g, const Meta meta) {
  typedef Traits<F> T;
  typedef Stage<F, WM, WN, MTW, NTW> Stg;
  constexpr int NW = WM * WN, H = T::H, TA = Stg::TA, TB = Stg::TB, R = TA * 16;
  constexpr int NA = TA * H, NB = TB * H, SA = Stg::SA, SB = Stg::SB;
  constexpr int ITEMS = NA + NB + SA + SB;
  constexpr int L = (ITEMS + NW - 1) / NW;
  constexpr int P = MTW * NTW;
  constexpr int CHUNK = 1024 * H;
  constexpr int PIECES = F == SC_MXFP4 ? 4 : 8;  // 16-byte pieces of a row's chunk
  static_assert(ST >= 3 && L * (ST - 2) <= 63, "ring");
  static_assert(TB % 4 == 0 && NTW % 2 == 0, "weight tiles come in quads, columns in pairs");
  static_assert(!T::BLOCK || (NTW * 16 <= 128 && 128 % (NTW * 16) == 0), "a wave's columns in one block");
  __shared__ Stg stage[ST];

  TileAt tile;
  if (!find_tile(g, meta, R, tile)) return;
  const int expert = tile.expert, row0 = tile.row0, rows = tile.rows;
  const int b_tile0 = tile.ngroup * TB;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint8_t* const wcodes = g.packed + expert * g.stride;
  const uint8_t* const wscales = wcodes + g.code_bytes;
  auto source = [&](int r) { return source_row<UP>(g, meta, tile, r); };

  // this wave's share of a stage (item e = wave + NW j): source, chunk stride, place,
  // and the lane's offset
  const uint8_t* it_src[L];
  uint32_t it_stride[L], it_lds[L], it_voff[L];
  bool it_wide[L];
#pragma unroll
  for (int j = 0; j < L; ++j) {
    int e = wave + NW * j;
    e = e < ITEMS ? e : ITEMS - 1;
    it_wide[j] = e < NA + NB;
    if (e < NA) {
      const int t = e / H, h = e % H;
      const int r = h * 8 + lane / PIECES;  // row of the tile (MXFP4: h = 0, 16 rows)
      const int p = (lane % PIECES) ^ swizzle<F>(r);
      it_src[j] = g.codes;
      it_voff[j] = source(t * 16 + r) * (uint32_t)g.rows.ld_codes + (uint32_t)p * 16u;
      it_stride[j] = PIECES * 16;
      it_lds[j] = (uint32_t)offsetof(Stg, a) + (t * H + h) * 1024;
    } else if (e < NA + NB) {
      const int t = (e - NA) / H, h = (e - NA) % H;
      const int64_t gt = b_tile0 + t < g.ntiles_w ? b_tile0 + t : 0;  // past N: tile 0, never stored
      it_src[j] = wcodes + gt * g.KC * CHUNK + h * 1024;
      it_voff[j] = (uint32_t)lane * 16u;
      it_stride[j] = CHUNK;
      it_lds[j] = (uint32_t)offsetof(Stg, b) + (t * H + h) * 1024;
    } else if (e < NA + NB + SA) {
      const int q = e - NA - NB;
      it_src[j] = g.scales;
      it_voff[j] = source(q * 64 + lane < R ? q * 64 + lane : R - 1) * (uint32_t)g.rows.ld_scales;
      it_stride[j] = 4;
      it_lds[j] = (uint32_t)offsetof(Stg, as) + q * 256;
    } else {
      const int q = e - NA - NB - SA;
      it_lds[j] = (uint32_t)offsetof(Stg, bs) + q * 256;
      if (T::MX) {
        const int64_t gq = b_tile0 / 4 + q < g.quads_w ? b_tile0 / 4 + q : 0;
        it_src[j] = wscales + gq * g.KC * 256;
        it_voff[j] = (uint32_t)lane * 4u;
        it_stride[j] = 256;
      } else {  // block FP8: the column block's scale in all 64 places
        int64_t nb = (b_tile0 * 16) / 128 + q;
        nb = nb < (int64_t)g.ntiles_w * 16 / 128 ? nb : 0;
        it_src[j] = wscales + nb * g.KC * 4;
        it_voff[j] = 0u;
        it_stride[j] = 4;
      }
    }
  }
  auto issue_item = [&](Stg& sg, uint32_t c, int j) {
    const uint32_t lds = lds_offset(&sg) + it_lds[j];
    const uint8_t* const src = it_src[j] + (uint64_t)c * it_stride[j];
    if (NW * j + NW <= NA + NB) lds_load16(src, it_voff[j], lds);
    else if (NW * j >= NA + NB) lds_load4(src, it_voff[j], lds);
    else if (it_wide[j]) lds_load16(src, it_voff[j], lds);
    else lds_load4(src, it_voff[j], lds);
  };

  float4v acc[MTW][NTW];
#pragma unroll
  for (int mt = 0; mt < MTW; ++mt)
#pragma unroll
    for (int nt = 0; nt < NTW; ++nt) acc[mt][nt] = float4v{0.f, 0.f, 0.f, 0.f};

  const int fr = lane & 15, kg = lane >> 4;
  uint32_t a_off[H];  // the lane's piece of half h within a tile, in 16-byte units
#pragma unroll
  for (int h = 0; h < H; ++h) a_off[h] = fr * PIECES + ((4 * h + kg) ^ swizzle<F>(fr));

  auto compute = [&](const Stg& sg, Stg& refill, uint32_t rc) {
    int8v b[NTW];
    int sb[NTW];
#pragma unroll
    for (int nt = 0; nt < NTW; ++nt) {
      const int t = wn * NTW + nt;
      const uint4v q0 = sg.b[t][0][lane];
      if (H == 1) {
        b[nt] = int8v{(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, 0, 0, 0, 0};
      } else {
        const uint4v q1 = sg.b[t][H - 1][lane];
        b[nt] = int8v{(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, (int)q1.x, (int)q1.y, (int)q1.z, (int)q1.w};
      }
      sb[nt] = T::MX ? (int)((sg.bs[t / 4][lane] >> (8 * (t % 4))) & 0xFFu) : 127;
    }
    float swv = 0.0f;
    if (T::BLOCK) swv = __uint_as_float(sg.bs[(wn * NTW * 16) / 128][0]);
    int p = 0;
#pragma unroll
    for (int mt = 0; mt < MTW; ++mt) {
      const int t = wm * MTW + mt;
      const uint4v* const at = &sg.a[t][0][0];
      const uint4v q0 = at[a_off[0]];
      int8v a;
      if (H == 1) {
        a = int8v{(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, 0, 0, 0, 0};
      } else {
        const uint4v q1 = at[a_off[H - 1]];
        a = int8v{(int)q0.x, (int)q0.y, (int)q0.z, (int)q0.w, (int)q1.x, (int)q1.y, (int)q1.z, (int)q1.w};
      }
      int sa = 127;
      if (T::MX) sa = (int)((sg.as[t / 4][(t % 4) * 16 + fr] >> (8 * kg)) & 0xFFu);
      float4v s4 = float4v{0.f, 0.f, 0.f, 0.f};
      if (T::BLOCK) {
        const float* rs = reinterpret_cast<const float*>(&sg.as[t / 4][0]) + 16 * (t % 4) + 4 * kg;
        s4 = float4v{rs[0] * swv, rs[1] * swv, rs[2] * swv, rs[3] * swv};
      }
#pragma unroll
      for (int nt = 0; nt < NTW; ++nt) {
#pragma unroll
        for (int j = 0; j < L; ++j)
          if ((j * P) / L == p) issue_item(refill, rc, j);
        if constexpr (T::BLOCK) {
          const float4v z = float4v{0.f, 0.f, 0.f, 0.f};
          const float4v part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[nt], z, 0, 0, 0, 127, 0, 127);
          acc[mt][nt] += part * s4;
        } else if constexpr (T::INT) {
          int4v s = __builtin_bit_cast(int4v, acc[mt][nt]);
          s = __builtin_amdgcn_mfma_i32_16x16x64_i8(int4v{a[0], a[1], a[2], a[3]},
                                                    int4v{b[nt][0], b[nt][1], b[nt][2], b[nt][3]}, s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_i32_16x16x64_i8(int4v{a[4], a[5], a[6], a[7]},
                                                    int4v{b[nt][4], b[nt][5], b[nt][6], b[nt][7]}, s, 0, 0, 0);
          acc[mt][nt] = __builtin_bit_cast(float4v, s);
        } else {
          acc[mt][nt] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[nt], acc[mt][nt], T::FMT, T::FMT, 0, sa,
                                                                         0, sb[nt]);
        }
        ++p;
      }
    }
  };

  // Ring: chunk i lives in stage i % ST. Before computing chunk i a wave waits for
  // its own loads of chunk i, passes the barrier (everyone's have landed and
  // everyone has finished chunk i - 1), then refills stage (i - 1) % ST with chunk i
  // + ST - 1 while computing (past the end: the last chunk again).
  const int nch = (int)g.KC;
#pragma unroll
  for (int p0 = 0; p0 < ST - 1; ++p0)
#pragma unroll
    for (int j = 0; j < L; ++j) issue_item(stage[p0], p0 < nch ? p0 : nch - 1, j);
  for (int i0 = 0; i0 < nch; i0 += ST) {
#pragma unroll
    for (int j = 0; j < ST; ++j) {
      if (i0 + j < nch) {
        wait_vmcnt<L * (ST - 2)>();
        stage_barrier();
        const int rc = i0 + j + ST - 1;
        compute(stage[j], stage[(j + ST - 1) % ST], rc < nch ? rc : nch - 1);
      }
    }
  }
  wait_vmcnt<0>();  // no LDS load may still be in flight when the workgroup ends

  const float alpha = g.alpha != nullptr ? g.alpha[expert] : 1.0f;
  const uint16_t* const bias = g.bias != nullptr ? g.bias + (int64_t)expert * g.N : nullptr;
  const int n0 = b_tile0 * 16;
  if constexpr (T::INT) {
#pragma unroll
    for (int mt = 0; mt < MTW; ++mt) {
      float4v row;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        row[i] = *reinterpret_cast<const float*>(
            g.scales + (int64_t)source((wm * MTW + mt) * 16 + 4 * kg + i) * g.rows.ld_scales);
#pragma unroll
      for (int nt = 0; nt < NTW; ++nt) {
        const int n = n0 + (wn * NTW + nt) * 16 + fr;
        const float col = n < g.ntiles_w * 16 ? reinterpret_cast<const float*>(wscales)[n] : 0.0f;
        const int4v s = __builtin_bit_cast(int4v, acc[mt][nt]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][nt][i] = int8_value(s[i], row[i], col);
      }
    }
  }
  if constexpr (UP) {
    const EpiOut o = {rows, g.N, alpha, bias, ScEpilogue{g.act, nullptr, 0}, nullptr, 0};
    float* const h = static_cast<float*>(g.out) + (int64_t)row0 * g.ld_out;
    auto put = [&](const float4v& v, int m, int n, int n_end) {
      if (n >= n_end) return;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (m + i < rows) h[(int64_t)(m + i) * g.ld_out + n] = v[i];
    };
#pragma unroll
    for (int mt = 0; mt < MTW; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTW; nt += 2) {
        const int m = (wm * MTW + mt) * 16 + 4 * kg, n = n0 + (wn * NTW + nt) * 16 + fr;
        if (o.gated()) {
          put(o.gate(acc[mt][nt], acc[mt][nt + 1], n), m, (n >> 5) * 16 + (n & 15), n < g.N ? g.N / 2 : 0);
        } else {
          put(o.plain(acc[mt][nt], n), m, n, g.N);
          put(o.plain(acc[mt][nt + 1], n + 16), m, n + 16, g.N);
        }
      }
  } else {
    // few rows: float32
    const EpiOut o = {rows, g.N, alpha, bias, ScEpilogue{kActNone, nullptr, 0}, nullptr, 0};
    float* const d = static_cast<float*>(g.out) + (int64_t)row0 * g.ld_out;
#pragma unroll
    for (int mt = 0; mt < MTW; ++mt)
#pragma unroll
      for (int nt = 0; nt < NTW; ++nt) {
        const int m = (wm * MTW + mt) * 16 + 4 * kg, n = n0 + (wn * NTW + nt) * 16 + fr;
        const float4v v = o.plain(acc[mt][nt], n);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (m + i < rows && n < g.N) d[(int64_t)(m + i) * g.ld_out + n] = v[i];
      }
  }
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------

// y_t = bf16(residual_t + sum_j w_tj d_row(t, j)), eight columns a thread, the sum in
// float32 in the order of the places. HALF: d's rows are fp16 with a factor for every 32
// columns (finish_tile), else float32; ldd columns either way, a multiple of 32. The rows
// of U places are loaded together.
template <bool HALF, int U>
__global__ __launch_bounds__(256) void experts_combine_kernel(const uint8_t* __restrict__ d,
                                                              const float* __restrict__ scales, int64_t ldd, int64_t T,
                                                              int64_t N, const float* __restrict__ weights,
                                                              const int* __restrict__ pair_row, int k,
                                                              const uint16_t* residual, int64_t ldr, uint16_t* y,
                                                              int64_t ldy, bool vec) {
  const int64_t nv = (N + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * nv) return;
  const int64_t t = i / nv, n = (i - t * nv) * 8;
  const bool whole = n + 8 <= N && vec;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  if (residual != nullptr) {
    const uint16_t* const r = residual + t * ldr + n;
    if (whole) {
      const uint4v u = *reinterpret_cast<const uint4v*>(r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[2 * j] = __uint_as_float(u[j] << 16);
        sum[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = n + j < N ? bf16_bits_to_f32(r[j]) : 0.0f;
    }
  }
  for (int p0 = 0; p0 < k; p0 += U) {
    int row[U];
    float w[U], f[U];
    uint4v q[U][HALF ? 1 : 2];
#pragma unroll
    for (int j = 0; j < U; ++j) {  // past the last place: it again, dropped below
      const int64_t at = t * k + (p0 + j < k ? p0 + j : k - 1);
      row[j] = pair_row[at];
      w[j] = weights[at];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t r = row[j] < 0 ? 0 : row[j];  // (row 0 for a place without an expert: dropped)
      f[j] = 1.0f;
      if constexpr (HALF) f[j] = scales[r * (ldd / 32) + n / 32];
#pragma unroll
      for (int i = 0; i < (HALF ? 1 : 2); ++i)  // columns past N: whatever is there, not stored
        q[j][i] = *reinterpret_cast<const uint4v*>(d + (r * ldd + n) * (HALF ? 2 : 4) + 16 * i);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (p0 + j >= k || row[j] < 0) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (HALF) {
          const half2v h = __builtin_bit_cast(half2v, (uint32_t)q[j][0][i]);
          v[2 * i] = (float)h.x * f[j];
          v[2 * i + 1] = (float)h.y * f[j];
        } else {
          v[i] = __uint_as_float(q[j][0][i]);
          v[4 + i] = __uint_as_float(q[j][1][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[j], v[i], sum[i]);
    }
  }
  uint16_t* const out = y + t * ldy + n;
  if (whole) {
    uint4v u;
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = f32_to_bf16_bits(sum[2 * j]) | (f32_to_bf16_bits(sum[2 * j + 1]) << 16);
    *reinterpret_cast<uint4v*>(out) = u;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (n + j < N) out[j] = (uint16_t)f32_to_bf16_bits(sum[j]);
  }
}

// ---------------------------------------------------------------------------
// configurations, plan, launcher
// ---------------------------------------------------------------------------

// (WM, WN, MTW, NTW, ST) of experts_product_kernel: row tiles of 16, 128 columns.
#define FQL_EXPERT_CONFIGS(X) X(1, 4, 1, 2, 4)
// (WM, MT, ST, EARLY) of experts_block_kernel: 64, 128 and 256 rows, 256 columns.
#define FQL_BLOCK_CONFIGS(X) X(1, 2, 3, 4) X(1, 4, 3, 8) X(2, 4, 2, 4)
// (WM, WN, MT, NT, ST) of experts_tile_kernel: 64, 128 and 256 rows, 256 columns.
#define FQL_TILE_CONFIGS(X) X(1, 4, 2, 2, 3) X(1, 4, 4, 2, 4) X(2, 2, 4, 4, 4)

template <int F, bool UP>
hipError_t launch_product(const ProductPlan& p, const ProductArgs& g, const Meta& m, hipStream_t st) {
  const unsigned grid = (unsigned)(p.max_tiles * g.ngroups);
#define FQL_X(A, B, C, D, S)                                                                       \
  if (!p.large && p.wm == A && p.wn == B && p.mtw == C && p.ntw == D && p.st == S) {                \
    experts_product_kernel<F, A, B, C, D, S, UP><<<grid, 64 * A * B, 0, st>>>(g, m);                \
    return hipGetLastError();                                                                       \
  }
  FQL_EXPERT_CONFIGS(FQL_X)
#undef FQL_X
  if constexpr (F == SC_FP8_BLOCK) {
#define FQL_X(A, C, S, E)                                                                                \
  if (p.large && p.wm == A && p.wn == 4 && p.ntw == 2 && p.mtw == C && p.st == S) {                      \
    experts_block_kernel<A, C, S, E, UP><<<grid, 256 * A, TileConfig<F, A, 4, C, 2, S>::LDS, st>>>(g, m); \
    return hipGetLastError();                                                                            \
  }
    FQL_BLOCK_CONFIGS(FQL_X)
#undef FQL_X
  } else {
#define FQL_X(A, B, C, D, S)                                                                       \
  if (p.large && p.wm == A && p.wn == B && p.mtw == C && p.ntw == D && p.st == S) {                 \
    experts_tile_kernel<F, A, B, C, D, S, UP><<<grid, 256, 0, st>>>(g, m);                          \
    return hipGetLastError();                                                                       \
  }
    FQL_TILE_CONFIGS(FQL_X)
#undef FQL_X
  }
  return hipErrorInvalidValue;
}

ProductArgs product_args(int fmt, const ProductPlan& p, const ExpertWeights& w, const uint8_t* codes,
                         const uint8_t* scales) {
  const ScDims d = sc_dims(fmt, w.N, w.K, true);
  ProductArgs g{};
  g.codes = codes;
  g.scales = scales;
  g.rows = expert_rows(fmt, w.K);
  g.packed = w.packed;
  g.stride = w.stride;
  g.code_bytes = d.code_bytes;
  g.N = (int)w.N;
  g.ntiles_w = (int)(d.rows_p / 16);
  g.ngroups = p.cols > 0 ? (int)((w.N + p.cols - 1) / p.cols) : 0;
  g.quads_w = d.quads;
  g.KC = d.KC;
  g.alpha = w.alpha;
  g.bias = w.bias;
  return g;
}

template <int F>
hipError_t launch_token(const ExpertsPlan& p, const ExpertsArgs& a, uint8_t* workspace, hipStream_t st) {
  float* const h = reinterpret_cast<float*>(workspace + p.counter_bytes);
  const ProductPlan none{};
  ProductArgs g = product_args(F, none, a.up, nullptr, nullptr);
  g.act = a.act;
  g.k = a.k;
  g.ld_out = round_up(a.I, 4);
  experts_token_up_kernel<F><<<dim3((unsigned)((a.up.N + 31) / 32), (unsigned)(a.T * a.k)), 256, 0, st>>>(
      a.x, a.ldx, a.up.inv_scale, a.up.K, a.experts, a.E, g, h);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  g = product_args(F, none, a.down, nullptr, nullptr);
  g.k = a.k;
  // waves without a row of their own share the others' K
  const int parts = (int)std::min<int64_t>(std::max(1, 16 / a.k), g.KC);
  experts_token_down_kernel<F><<<dim3((unsigned)((a.down.N + 15) / 16), (unsigned)a.T), 1024, 0, st>>>(
      h, round_up(a.I, 4), a.down.inv_scale, a.I, a.experts, a.weights, a.E, parts, g, a.residual, a.ldr, a.y, a.ldy);
  return hipGetLastError();
}

template <int F>
hipError_t launch_t(const ExpertsPlan& p, const ExpertsArgs& a, uint8_t* workspace, hipStream_t st) {
  if (p.token) return launch_token<F>(p, a, workspace, st);
  uint8_t* at = workspace + p.counter_bytes;
  auto take = [&](int64_t bytes) {
    uint8_t* const r = at;
    at += bytes;
    return r;
  };
  uint8_t* const meta = take(p.meta_bytes);
  uint8_t* const xc = take(p.xcode_bytes);
  uint8_t* const xs = take(p.xscale_bytes);
  uint8_t* const h = take(p.h_bytes);
  uint8_t* const hc = take(p.hcode_bytes);
  uint8_t* const hs = take(p.hscale_bytes);
  uint8_t* const d = take(p.d_bytes);
  float* const ds = reinterpret_cast<float*>(d + p.pairs * 2 * round_up(a.down.N, 32));  // of fp16 rows
  Meta m[2];
  meta_at(meta, p.pairs, p.up.max_tiles, p.down.max_tiles, m);
  for (int64_t t0 = 0; t0 < a.T; t0 += p.tokens) {
    const int64_t T = std::min(p.tokens, a.T - t0), pairs = T * a.k;
    QuantArgs q{a.x + t0 * a.ldx, T, a.up.K, a.ldx, a.aligned, a.up.inv_scale, expert_rows(F, a.up.K), xc, xs};
    const int groups = (int)std::min<int64_t>(32, (pairs + 2047) / 2048);
    experts_prepare_kernel<F><<<(unsigned)(groups + quant_units(F, q)), kPrepThreads, 0, st>>>(
        a.experts + t0 * a.k, pairs, a.E, p.up.rows, p.down.rows, groups, m[0], m[1], q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ProductArgs g = product_args(F, p.up, a.up, xc, xs);
    g.act = a.act;
    g.k = a.k;
    g.hrows = expert_rows(F, a.I);
    g.hscales = hs;
    g.inv_scale = a.down.inv_scale;
    g.out = p.h_quantized ? hc : h;
    g.ld_out = round_up(a.I, 4);
    e = launch_product<F, true>(p.up, g, m[0], st);
    if (e != hipSuccess) return e;
    if (!p.h_quantized) {
      q = QuantArgs{h, pairs, a.I, round_up(a.I, 4), true, a.down.inv_scale, expert_rows(F, a.I), hc, hs};
      experts_quant_kernel<F><<<(unsigned)quant_units(F, q), kPrepThreads, 0, st>>>(q);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    g = product_args(F, p.down, a.down, hc, hs);
    g.out = d;
    g.out_scales = ds;
    g.ld_out = round_up(a.down.N, 32);
    g.k = a.k;
    e = launch_product<F, false>(p.down, g, m[1], st);
    if (e != hipSuccess) return e;
    uint16_t* const y = a.y + t0 * a.ldy;
    const uint16_t* const r = a.residual != nullptr ? a.residual + t0 * a.ldr : nullptr;
    auto whole = [](const void* ptr, int64_t ld) { return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && ld % 8 == 0; };
    const bool vec = whole(a.y, a.ldy) && (r == nullptr || whole(a.residual, a.ldr));
    const int64_t items = T * ((a.down.N + 7) / 8);
    const auto combine = p.down.large ? (a.k > 2 ? experts_combine_kernel<true, 4> : experts_combine_kernel<true, 2>)
                                      : (a.k > 2 ? experts_combine_kernel<false, 4> : experts_combine_kernel<false, 2>);
    combine<<<(unsigned)((items + 255) / 256), 256, 0, st>>>(d, ds, round_up(a.down.N, 32), T, a.down.N, a.weights + t0 * a.k,
                                                             m[0].pair_row, a.k, r, a.ldr, y, a.ldy, vec);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// From how many rows an expert on a product takes the large tiles (why: plan_product).
static int64_t large_rows(int fmt) { return fmt == SC_INT8 ? 20 : 8; }
constexpr int64_t kTokenMax = 6;  // tokens of a call whose pairs stay for themselves, at most (plan_experts)

// The tile of one product, N columns of a K-deep product, `pairs` rows over E experts:
// 16 x 128 while an expert has few rows, else the tile of least time: rounds of the card's
// workgroups times (chunks * tc + f) us, with six tenths of a tile an expert for its last
// rows. tc is measured, full tiles on the whole card; past four rounds workgroups start
// as others end. f is fitted to 50 products (each tile forced, 24 to 4096 tokens, 4 to 128
// experts): the tile it picks costs a call 0.9% over the best of the three on average.
// (4 experts of FP8, 495 tokens, 5376, 288 inner: 64-row tiles 43.6 us, 128-row 53.2; 60 of
// MXFP4, 152 tokens, 672, 448 inner, down: 28.4 and 30.0, 256 rows 33.9.)
// Whole calls on 16-row tiles and on the larger ones, us, at 4, 8 and 16 rows an expert:
//   MXFP8      64 experts, 4096, 1024 inner   158, 151   166, 154   182, 157
//              32, 2048, 2048                  89, 85     92, 85    102, 87
//   block FP8  32, 4096, 2048                 152, 149   158, 151   170, 153
//              64, 2048, 1024                  88, 88     92, 90    101, 91
//   MXFP4      128, 4096, 1280                201, 195   210, 198   244, 206
//              32, 2048, 2048                  50, 48     50, 48     56, 48
//   FP8        8, 4096, 14336                 245, 256   250, 257   290, 260
//              32, 2048, 1408                  60, 60     61, 60     69, 61
// and INT8, which quantizes h in a launch of its own either way, at 8, 16, 20 and 24 rows:
//              32, 2048, 1408                  61, 65     72, 68     74, 69     75, 70
//              8, 4096, 7168                  138, 147   157, 150   163, 152   170, 155
//              64, 2048, 1024                  96, 98    102, 101   112, 103   118, 105
// So the limit of 8 costs few large FP8 experts 3% at 8 rows and the others up to 5% below it;
// INT8's of 20 costs 1 to 5% between 13 and 19 rows.
static ProductPlan plan_product(int fmt, int64_t pairs, int64_t E, int64_t N, int64_t K) {
  struct Tile {
    int wm, wn, mtw, ntw, st, resident;
    double tc[3], f;  // MXFP4, block FP8, the others
  };
  static constexpr Tile tiles[] = {{1, 4, 2, 2, 3, 2, {1.00, 1.00, 1.40}, 5.0},
                                   {1, 4, 4, 2, 4, 1, {0.85, 1.45, 1.35}, 7.5},
                                   {2, 2, 4, 4, 4, 1, {1.04, 1.92, 1.60}, 11.0}};
  const bool block = fmt == SC_FP8_BLOCK;
  const int64_t KC = round_up(K, 128) / 128;
  ProductPlan p{};
  if (pairs / E >= large_rows(fmt)) {
    double best = 0.0;
    for (const Tile& t : tiles) {
      const int64_t R = 32 * t.wm * t.mtw;
      const double rows = (double)pairs / (double)R + 0.6 * (double)E;
      const int resident = block ? 1 : t.resident;
      const double full = rows * (double)((N + 255) / 256) / (256.0 * resident);
      const double rounds = full < 4.0 ? std::ceil(full) : full + 0.3;
      const double cost = rounds * ((double)KC * t.tc[fmt == SC_MXFP4 ? 0 : block ? 1 : 2] + t.f);
      if (p.large && cost >= best) continue;
      best = cost;
      p = ProductPlan{true, t.wm, t.wn, t.mtw, t.ntw, t.st, (int)R, 256, 0};
      if (block) {  // experts_block_kernel's forms of them
        p.wn = 4;
        p.ntw = 2;
        p.st = t.wm == 2 ? 2 : 3;
      }
    }
  } else {
    p = ProductPlan{false, 1, 4, 1, 2, 4, 16, 128, 0};
  }
  p.max_tiles = std::min(pairs, pairs / p.rows + std::min(E, pairs));
  return p;
}

ExpertsPlan plan_experts(int fmt, int64_t T, int64_t k, int64_t E, int64_t H, int64_t N, int64_t I, int64_t Ho) {
  ExpertsPlan p{};
  p.fmt = fmt;
  const ExpertRows xr = expert_rows(fmt, H), hr = expert_rows(fmt, I);
  // a pass's activations lie within 32-bit offsets and 1 GiB of workspace
  const int64_t per_pair = hr.ld_codes + hr.ld_scales + 4 * round_up(I, 4) + 4 * round_up(Ho, 32);
  const int64_t per_token = xr.ld_codes + xr.ld_scales + k * per_pair;
  p.tokens = std::max<int64_t>(1, std::min<int64_t>(T, ((int64_t)1 << 30) / per_token));
  p.pairs = p.tokens * k;
  p.up = plan_product(fmt, p.pairs, E, N, H);
  p.down = plan_product(fmt, p.pairs, E, Ho, I);
  // A few tokens, every pair for itself: two launches for four or five, but an expert that
  // several tokens choose is read for each. A call each way, us (each pair, sorted):
  //   64 experts, 8 a token, 2048, 1024 inner   1 token   4 tokens   6 tokens   8 tokens
  //     block FP8                               16, 28    35, 48     48, 57     61, 64
  //     MXFP8                                   16, 28    37, 47     52, 60     64, 64
  //     INT8                                    17, 28    38, 49     52, 60     67, 68
  //     MXFP4                                   14, 24    23, 34     30, 40     38, 42
  //   64, 6 a token, 4096, 1024 (MXFP8)         20, 33    56, 68     80, 83    103, 100
  //   128, 8 a token, 4096, 1280 (MXFP4)        20, 31    56, 61     78, 76    102, 97
  //   32, 4 a token, 2048, 1408 (INT8)          16, 25    29, 37     40, 44     48, 49
  //   8, 2 a token, 4096, 14336 (FP8)           63, 94     (2 tokens) 119, 132  (3) 167, 150
  // 4 pairs < 3 experts keeps the last line's 3 tokens out, and the 6 tokens of the first lines
  // too, where each pair for itself would be 9 to 25% faster.
  p.token = T == 1 || (T <= kTokenMax && p.tokens == T && 4 * p.pairs < 3 * E);
  p.h_quantized = !p.token && p.up.large && fmt != SC_INT8;
  p.counter_bytes = 64 * 1024;
  // (the tiles of the smallest form, so that more tokens never take fewer bytes)
  const int64_t tiles = std::min(p.pairs, p.pairs / (p.up.large ? 64 : 16) + std::min(E, p.pairs));
  p.meta_bytes = round_up(meta_bytes(p.pairs, tiles, tiles), 256);
  p.xcode_bytes = round_up(p.tokens * xr.ld_codes, 256);
  p.xscale_bytes = round_up(p.tokens * xr.ld_scales, 256);
  p.h_bytes = p.h_quantized ? 0 : round_up(p.pairs * 4 * round_up(I, 4), 256);
  p.hcode_bytes = round_up(p.pairs * hr.ld_codes, 256);
  p.hscale_bytes = round_up(p.pairs * hr.ld_scales, 256);
  p.d_bytes = round_up(p.pairs * round_up(Ho, 32) * (p.down.large ? 2 : 4) + (p.down.large ? p.pairs * round_up(Ho, 32) / 8 : 0), 256);
  if (p.token) p.meta_bytes = p.xcode_bytes = p.xscale_bytes = p.hcode_bytes = p.hscale_bytes = p.d_bytes = 0;
  p.total_bytes = p.counter_bytes + p.meta_bytes + p.xcode_bytes + p.xscale_bytes + p.h_bytes + p.hcode_bytes +
                  p.hscale_bytes + p.d_bytes;
  return p;
}

// Larger tiles keep h as codes and d in 16 bits, so the call of the most tokens need not be
// the one of the most bytes: the largest calls of each of the three ways are looked at.
int64_t experts_workspace(int fmt, int64_t T, int64_t k, int64_t E, int64_t H, int64_t N, int64_t I, int64_t Ho) {
  auto bytes = [&](int64_t t) { return plan_experts(fmt, t, k, E, H, N, I, Ho).total_bytes; };
  int64_t most = bytes(T);
  for (int64_t t = 1; t <= std::min(T, kTokenMax); ++t) most = std::max(most, bytes(t));
  const int64_t small = (large_rows(fmt) * E - 1) / k;  // the most tokens on 16-row tiles
  if (small >= 1) most = std::max(most, bytes(std::min(T, small)));
  return most;
}

std::string describe_experts(const ExpertsPlan& p) {
  auto name = [&](const ProductPlan& q) {
    char b[100];
    std::snprintf(b, sizeof(b), "%s<WM=%d,WN=%d,MT=%d,NT=%d,ST=%d> tiles=%dx%d",
                  !q.large ? "experts_product_kernel" : p.fmt == SC_FP8_BLOCK ? "experts_block_kernel" : "experts_tile_kernel",
                  q.wm, q.wn, q.mtw, q.ntw, q.st, q.rows, q.cols);
    return std::string(b);
  };
  if (p.token) return "experts_token_up_kernel + experts_token_down_kernel tokens=" + std::to_string(p.tokens);
  return "up " + name(p.up) + " down " + name(p.down) + " tokens=" + std::to_string(p.tokens);
}

hipError_t launch_experts(const ExpertsPlan& p, const ExpertsArgs& a, uint8_t* workspace, hipStream_t st) {
#define FQL_F(F) \
  if (p.fmt == F) return launch_t<F>(p, a, workspace, st);
  FQL_F(SC_MXFP4) FQL_F(SC_MXFP8) FQL_F(SC_FP8) FQL_F(SC_FP8_BLOCK) FQL_F(SC_INT8)
#undef FQL_F
  return hipErrorInvalidValue;
}

}  // namespace fql
