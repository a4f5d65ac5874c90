// The experts' product on large tiles (gfx950): four waves, one a SIMD, each with
// MT x NT accumulator tiles of 32 x 32.
//
// What bounds a product of 8-bit operands is the way into the registers: a CU takes
// about 28 B a cycle into LDS from L2, LDS gives 128 B a cycle, and a SIMD's matrix
// core works 64 cycles on 4 KB of operands. So bytes a flop have to fall: a 256 x 256
// tile loads 64 KB for 128-deep products of 1024 cycles a SIMD and half, and waves of
// 128 x 128 read each loaded byte twice. The accumulators fill 256 registers, which
// leaves one wave a SIMD; what would wait for a neighbour is arranged within the wave:
// operands of stage i + 1 are read from LDS into a second register set while the
// matrix core works on stage i, and stages i + 2 .. i + ST are on their way from L2.
//
// A stage is 64 deep (MXFP4 128: 1 KB of a 16-row tile in every format), for block
// FP8 128, whose products of one 128-deep chunk go into a fresh accumulator and are
// added with the chunk's scales. In LDS:
//   activation tiles  16 rows of 64 bytes as they lie in memory, their four 16-byte
//                     pieces exchanged (piece p of row r in place p ^ (r / 4 % 4)), so
//                     that the 16 lanes that read one piece of all rows hit all banks
//   weight tiles      the packed order
//   scales            of four chunks at a time, two buffers in turn: a row's four
//                     dwords (one 16-byte load a row: a dword of every row is 64
//                     cache lines a load), a weight quad's four runs of 64 dwords
#pragma once

#include <cstddef>

#include "fql_device.h"
#include "fql_experts.h"
#include "fql_gemm.h"
#include "sc_epilogue.h"
#include "sc_quant.h"

namespace fql {
namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));

// One expert's part of a pass for one of the products: its first row tile, their
// number, its first row and the number of its rows.
struct ExpertRange {
  int tile0, tiles, row0, rows;
};

// Metadata of a pass in the workspace, as one of the products sees it.
struct Meta {
  int* total_tiles;     // [0]
  ExpertRange* ranges;  // [E]
  int* tile_expert;     // [max_tiles]
  int* row_pair;        // [pairs] pair t * k + j of a sorted row
  int* pair_row;        // [pairs] its inverse; -1: the pair has no expert
};

template <int F>
struct Traits {
  static constexpr int H = F == SC_MXFP4 ? 1 : 2;
  static constexpr int FMT = F == SC_MXFP4 ? 4 : 0;
  static constexpr bool MX = F == SC_MXFP4 || F == SC_MXFP8;
  static constexpr bool BLOCK = F == SC_FP8_BLOCK;
  static constexpr bool INT = F == SC_INT8;
};

struct ProductArgs {
  const uint8_t* codes;  // activation rows
  const uint8_t* scales;
  ExpertRows rows;
  const uint8_t* packed;  // weights
  int64_t stride, code_bytes;
  int N, ntiles_w, ngroups;
  int64_t quads_w, KC;
  const float* alpha;    // [E] or null
  const uint16_t* bias;  // [E][N] or null
  int act;               // up
  void* out;             // up: float32 [row][ld_out], or codes (hq); down: float32 or fp16 [row][ld_out]
  float* out_scales;     // down, fp16: [row][ld_out / 32]
  int64_t ld_out;
  int k;
  // up: the inner activation quantized in the epilogue (all but INT8)
  ExpertRows hrows;
  uint8_t* hscales;
  float inv_scale;
};

// A tile of a product: expert, rows and column group. An expert's row tiles of one
// column group are neighbours in the order of tiles, and every XCD has a contiguous part
// of that order (workgroups go to the eight XCDs in turn).
struct TileAt {
  int expert, row0, rows, ngroup;
};
// This workgroup's tile; false past the last one.
__device__ __forceinline__ bool find_tile(const ProductArgs& g, const Meta& meta, int R, TileAt& t) {
  const int total = meta.total_tiles[0] * g.ngroups;
  const int bid = blockIdx.x;
  if (bid >= total) return false;
  const int xcd = bid & 7, q8 = total >> 3, r8 = total & 7;
  const int logical = xcd * q8 + (xcd < r8 ? xcd : r8) + (bid >> 3);
  t.expert = meta.tile_expert[logical / g.ngroups];
  const ExpertRange er = meta.ranges[t.expert];
  const int within = logical - er.tile0 * g.ngroups;
  const int row_tile = within % er.tiles;
  t.ngroup = within / er.tiles;
  t.row0 = er.row0 + row_tile * R;
  t.rows = er.rows - row_tile * R < R ? er.rows - row_tile * R : R;  // at least 1
  return true;
}
// The activation row of tile row r; rows past the tile's take its last one.
template <bool UP>
__device__ __forceinline__ uint32_t source_row(const ProductArgs& g, const Meta& meta, const TileAt& t, int r) {
  const int s = t.row0 + (r < t.rows ? r : t.rows - 1);
  return (uint32_t)(UP ? meta.row_pair[s] / g.k : s);
}

// Four codes of values v * f: 32 bits (MXFP4: the lower 16).
template <int F>
__device__ __forceinline__ uint32_t encode4(const float v[4], float f) {
#pragma clang fp contract(off)
  if (F == SC_MXFP4) {
    const uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0] * f, v[1] * f, 1.0f, 0);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * f, v[3] * f, 1.0f, 1);
  }
  return fp8x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}
// Exchanges the upper 32 lanes of x with the lower 32 of y.
__device__ __forceinline__ void swap_halves(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  x = r[0];
  y = r[1];
}

template <int F, int WM, int WN, int MT, int NT, int ST>
struct TileConfig {
  static constexpr int SUB = Traits<F>::BLOCK ? 2 : 1;             // 1 KB pieces of a 16-row tile a stage
  static constexpr int PER_CHUNK = Traits<F>::H / SUB;             // stages of a 128-deep chunk
  static constexpr int TA = WM * MT * 2, TB = WN * NT * 2;         // 16-row tiles
  static constexpr int R = TA * 16, C = TB * 16;
  static constexpr int STAGE = (TA + TB) * SUB * 1024;
  static constexpr bool SCALED = Traits<F>::MX || Traits<F>::BLOCK;
  static constexpr int ASC = SCALED ? R * 16 : 0;                  // row scales of four chunks
  static constexpr int BSC = Traits<F>::MX ? C * 16 : Traits<F>::BLOCK ? (C / 128) * 256 : 0;
  static constexpr int RING = ST * STAGE;
  static constexpr int OUT = MT * 32 * (C + 4) * 4;                // float32 rows of one wave row (epilogue)
  static constexpr int LDS = RING + 2 * (ASC + BSC) > OUT ? RING + 2 * (ASC + BSC) : OUT;
  static constexpr int NW = WM * WN;                               // waves
  static constexpr int L = (TA + TB) * SUB / NW;                   // loads a wave and stage
  static_assert(TA % NW == 0 && TB % NW == 0 && NW % 4 == 0, "tiles a wave loads");
  static_assert(L * (ST - 1) <= 63, "vmcnt range");
  static_assert(LDS <= 160 * 1024, "LDS");
};

// A workgroup's loads from memory into the ring. Of a stage, wave w of NW takes the
// activation tiles w, w + NW, .. and the weight tiles likewise, each in SUB pieces.
template <int F, typename Cfg, bool UP>
struct TileLoads {
  typedef Traits<F> T;
  static constexpr int SUB = Cfg::SUB, TA = Cfg::TA, TB = Cfg::TB, L = Cfg::L, NW = Cfg::NW;
  static constexpr int QA = Cfg::R / 64, QB = Cfg::C / 64;
  const uint8_t *codes, *scales, *wscales, *b_src[TB / NW];
  uint32_t a_voff[TA / NW], as_voff, lds0;
  int KC, ntiles_w, b_tile0, wave, lane;
  int64_t quads_w;
  __device__ __forceinline__ TileLoads(const ProductArgs& g, const Meta& meta, const TileAt& tile, uint32_t lds0,
                                       int wave, int lane)
      : codes(g.codes), scales(g.scales), lds0(lds0), KC((int)g.KC), ntiles_w(g.ntiles_w), b_tile0(tile.ngroup * TB),
        wave(wave), lane(lane), quads_w(g.quads_w) {
    const uint8_t* const wcodes = g.packed + tile.expert * g.stride;
    wscales = wcodes + g.code_bytes;
#pragma unroll
    for (int j = 0; j < TA / NW; ++j) {
      const int r = lane >> 2, p = (lane & 3) ^ ((r >> 2) & 3);
      a_voff[j] = source_row<UP>(g, meta, tile, (wave + NW * j) * 16 + r) * (uint32_t)g.rows.ld_codes + (uint32_t)p * 16u;
    }
#pragma unroll
    for (int j = 0; j < TB / NW; ++j) {
      const int t = b_tile0 + wave + NW * j;
      b_src[j] = wcodes + (int64_t)(t < g.ntiles_w ? t : 0) * g.KC * (1024 * T::H);  // past N: tile 0, never stored
    }
    as_voff = 0u;
    if (Cfg::SCALED)
      as_voff = source_row<UP>(g, meta, tile, (wave < QA ? wave : QA - 1) * 64 + lane) * (uint32_t)g.rows.ld_scales;
  }
  // the lane's offset into the weight tiles of a stage
  __device__ __forceinline__ uint32_t b_voff(int stage) const {
    return (uint32_t)lane * 16u + (uint32_t)stage * (SUB * 1024u);
  }
  // load j of the wave's L of a stage, into a slot of the ring
  __device__ __forceinline__ void stage(int slot, int st, uint32_t bv, int j) const {
    if (j < TA / NW * SUB) {
      const int t = j / SUB, s = j % SUB;
      lds_load16(codes + (int64_t)(st * SUB + s) * 64, a_voff[t],
                 lds0 + slot * Cfg::STAGE + ((wave + NW * t) * SUB + s) * 1024);
    } else {
      const int t = (j - TA / NW * SUB) / SUB, s = (j - TA / NW * SUB) % SUB;
      lds_load16(b_src[t], bv + s * 1024u, lds0 + slot * Cfg::STAGE + ((TA + wave + NW * t) * SUB + s) * 1024);
    }
  }
  // scales of four chunks from chunk c0 on, into buffer q
  __device__ __forceinline__ void four_scales(int c0, int q) const {
    if constexpr (Cfg::SCALED) {
      const int quad = wave < QA ? wave : QA - 1;  // (waves past the last quad load it again)
      const uint32_t at = lds0 + Cfg::RING + q * (Cfg::ASC + Cfg::BSC);
      lds_load16(scales + (int64_t)c0 * 4, as_voff, at + quad * 1024);
      const int last = KC - 1;
      if constexpr (T::MX) {
        static_assert(QB <= 4, "a quad a wave");
        const int bq = wave < QB ? wave : QB - 1;
        const int64_t gq = b_tile0 / 4 + bq < quads_w ? b_tile0 / 4 + bq : 0;
        const int c = c0 + (lane >> 4) < last ? c0 + (lane >> 4) : last;  // past the last chunk: it again
        lds_load16(wscales + gq * KC * 256, (uint32_t)c * 256u + (uint32_t)(lane & 15) * 16u, at + Cfg::ASC + bq * 1024);
      } else {
        const int bb = wave % (Cfg::C / 128);
        int nb = b_tile0 / 8 + bb;
        nb = nb < ntiles_w / 8 ? nb : 0;
        const int c = c0 + (lane & 3) < last ? c0 + (lane & 3) : last;
        lds_load4(wscales + (int64_t)nb * KC * 4, (uint32_t)c * 4u, at + Cfg::ASC + bb * 256);
      }
    }
  }
};

// What becomes of a workgroup's accumulators: the way out of both kernels below. lds:
// free of other use, OUT bytes where the activation is not gated.
template <int F, int WM, int WN, int MT, int NT, bool UP>
__device__ __forceinline__ void finish_tile(const ProductArgs& g, const Meta& meta, const TileAt& tile,
                                            float16v (&acc)[MT][NT], const uint8_t* wscales, int n0, uint8_t* lds) {
  typedef Traits<F> T;
  constexpr int R = WM * MT * 32, C = WN * NT * 32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, kb = lane >> 5;
  // epilogue. Register r of a tile: row lane % 32, column 8 (r / 4) + 4 (lane / 32) + r % 4
  const float alpha = g.alpha != nullptr ? g.alpha[tile.expert] : 1.0f;
  const uint16_t* const bias = g.bias != nullptr ? g.bias + (int64_t)tile.expert * g.N : nullptr;
  float rsc[MT];  // INT8: the scale of the lane's row
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    rsc[mt] = 1.0f;
    if constexpr (T::INT) {
      const uint32_t row = source_row<UP>(g, meta, tile, (mt * WM + wm) * 32 + (lane & 31));
      rsc[mt] = *reinterpret_cast<const float*>(g.scales + (int64_t)row * g.rows.ld_scales);
    }
  }
  // alpha * product + bias of the wave's tiles: put(row of the wave row, column of the
  // tile, four neighbouring columns' values)
  auto finish = [&](auto put) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = (wn * NT + nt) * 32 + 8 * i + 4 * kb, n = n0 + c;
        float b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = bias != nullptr && n + e < g.N ? bf16_bits_to_f32(bias[n + e]) : 0.0f;
        float4v col = {1.f, 1.f, 1.f, 1.f};
        if constexpr (T::INT) {
          if (n < g.ntiles_w * 16) col = *reinterpret_cast<const float4v*>(wscales + (int64_t)n * 4);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float4v v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float s = acc[mt][nt][4 * i + e];
            if constexpr (T::INT) s = int8_value((int)__float_as_uint(s), rsc[mt], col[e]);
            v[e] = alpha * s + b[e];
          }
          put(mt * 32 + (lane & 31), c, v);
        }
      }
  };
  // the rows of one wave row at a time through LDS: row tiles pass, pass + WM, ..
  constexpr int PR = MT * 32;
  if (UP && g.act == kActSwiglu) {
    // Gated: 16 gate columns, then their 16 ups, so that registers r and r + 8 of a lane
    // are a pair. The outputs stay in registers: outputs 8 i + 4 kb .. + 3 (i = 0, 1) of a
    // tile's 16 take the place of its first eight
    const int Nout = g.N / 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = n0 + (wn * NT + nt) * 32 + 8 * i + 4 * kb;
        float bg[4], bu[4];
        float4v cg = {1.f, 1.f, 1.f, 1.f}, cu = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          bg[e] = bias != nullptr && n + e < g.N ? bf16_bits_to_f32(bias[n + e]) : 0.0f;
          bu[e] = bias != nullptr && n + e + 16 < g.N ? bf16_bits_to_f32(bias[n + e + 16]) : 0.0f;
        }
        if constexpr (T::INT) {  // (N is a multiple of 32: a gate's up is there)
          if (n < g.N) {
            cg = *reinterpret_cast<const float4v*>(wscales + (int64_t)n * 4);
            cu = *reinterpret_cast<const float4v*>(wscales + (int64_t)(n + 16) * 4);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a = acc[mt][nt][4 * i + e], u = acc[mt][nt][4 * i + e + 8];
            if constexpr (T::INT) {
              a = int8_value((int)__float_as_uint(a), rsc[mt], cg[e]);
              u = int8_value((int)__float_as_uint(u), rsc[mt], cu[e]);
            }
            const float z = alpha * a + bg[e];
            acc[mt][nt][4 * i + e] = z_sigmoid(z, z) * (alpha * u + bu[e]);
          }
      }
    const int no = n0 / 2 + wn * NT * 16;  // the wave's first output
    if constexpr (T::INT) {
      // float32 rows: their scale needs all columns
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int m = (mt * WM + wm) * 32 + (lane & 31);
        float* const out = static_cast<float*>(g.out) + (int64_t)(tile.row0 + m) * g.ld_out + no + 4 * kb;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (m < tile.rows && no + nt * 16 + 8 * i < Nout)
              *reinterpret_cast<float4v*>(out + nt * 16 + 8 * i) =
                  float4v{acc[mt][nt][4 * i], acc[mt][nt][4 * i + 1], acc[mt][nt][4 * i + 2], acc[mt][nt][4 * i + 3]};
      }
    } else {
      // A block of 32 outputs: two tiles, 16 outputs a lane and the others in lane ^ 32.
      const int64_t padded = g.hrows.ld_codes / (F == SC_MXFP4 ? 16 : 32);  // blocks of a row
      constexpr int NP = NT / 2;
      float top[MT][NP];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          float a = 0.0f;
#pragma unroll
          for (int j = 0; j < 16; ++j) a = __builtin_fmaxf(a, __builtin_fabsf(acc[mt][2 * p + j / 8][j % 8]));
          uint32_t x = __float_as_uint(a), y = x;
          swap_halves(x, y);
          top[mt][p] = __builtin_fmaxf(__uint_as_float(x), __uint_as_float(y));
        }
      if constexpr (T::BLOCK) {
        // the four blocks of a 128-group lie in as many waves (or half of them): joined through LDS
        static_assert((WN * NP) % 4 == 0, "a group's blocks in one workgroup");
        float* const tops = reinterpret_cast<float*>(lds);  // [block][row]
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int p = 0; p < NP; ++p)
            if (kb == 0) tops[(wn * NP + p) * R + (mt * WM + wm) * 32 + lane] = top[mt][p];
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const float* const t = tops + (wn * NP + p) / 4 * 4 * R + (mt * WM + wm) * 32 + (lane & 31);
            top[mt][p] = __builtin_fmaxf(__builtin_fmaxf(t[0], t[R]), __builtin_fmaxf(t[2 * R], t[3 * R]));
          }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int m = (mt * WM + wm) * 32 + (lane & 31);
        uint8_t* const dst = static_cast<uint8_t*>(g.out) + (int64_t)(tile.row0 + m) * g.hrows.ld_codes;
        uint8_t* const sc = g.hscales + (int64_t)(tile.row0 + m) * g.hrows.ld_scales;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int64_t at = no / 32 + p;  // block of the row
          const bool valid = at * 32 < Nout;  // past the columns, up to the chunk: zeros
          float f = g.inv_scale, group = 0.0f;
          uint32_t sbyte = 0u;
          if constexpr (T::MX) {
            const int e = mx_exponent(top[mt][p], F == SC_MXFP4 ? 2 : 8);
            f = pow2_neg(e);
            sbyte = (uint32_t)(e + 127);
          } else if constexpr (T::BLOCK) {
            group = top[mt][p] / 448.0f;
            f = safe_reciprocal(group);
          }
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float v[4] = {acc[mt][2 * p + j / 2][(j % 2) * 4], acc[mt][2 * p + j / 2][(j % 2) * 4 + 1],
                                acc[mt][2 * p + j / 2][(j % 2) * 4 + 2], acc[mt][2 * p + j / 2][(j % 2) * 4 + 3]};
            w[j] = valid ? encode4<F>(v, f) : 0u;
          }
          // w[j] holds outputs 8 j + 4 kb .. + 3; the lower lanes get the block's first half
          if constexpr (F == SC_MXFP4) {
            uint32_t x = (w[0] & 0xFFFFu) | (w[1] << 16), y = (w[2] & 0xFFFFu) | (w[3] << 16);
            swap_halves(x, y);
            const uint64_t codes = (uint64_t)((x & 0xFFFFu) | (y << 16)) | ((uint64_t)((x >> 16) | (y & 0xFFFF0000u)) << 32);
            if (m < tile.rows && at < padded) *reinterpret_cast<uint64_t*>(dst + at * 16 + 8 * kb) = codes;
          } else {
            swap_halves(w[0], w[2]);
            swap_halves(w[1], w[3]);
            if (m < tile.rows && at < padded)
              *reinterpret_cast<uint4v*>(dst + at * 32 + 16 * kb) = uint4v{w[0], w[2], w[1], w[3]};
          }
          if (m < tile.rows && at < padded && kb == 0) {
            if (T::MX) sc[at] = valid ? (uint8_t)sbyte : 0;
            if (T::BLOCK && (at & 3) == 0) *reinterpret_cast<float*>(sc + at) = group;
          }
        }
      }
    }
  } else if constexpr (UP) {
    // (the LDS way of the activations that are not gated)
    constexpr int pitch = C + 4;  // floats of a row
    constexpr int Co = C;
    const int no = n0, Nout = g.N;
    float* const z = reinterpret_cast<float*>(lds);
    // columns 8 j .. 8 j + 7 of row m, activated
    auto outputs8 = [&](int m, int j, float v[8]) {
      const float* const p = z + m * pitch + 8 * j;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4v a = *reinterpret_cast<const float4v*>(p + e);
#pragma unroll
        for (int x = 0; x < 4; ++x) v[e + x] = apply_act(a[x], g.act);
      }
    };
    for (int pass = 0; pass < WM; ++pass) {
      if (pass * 32 >= tile.rows) break;
      if (wm == pass) finish([&](int m, int c, const float4v& v) { *reinterpret_cast<float4v*>(z + m * pitch + c) = v; });
      __syncthreads();
      auto row_of = [&](int m) { return ((m / 32) * WM + pass) * 32 + m % 32; };  // row of the tile
      if constexpr (T::INT) {
        // float32 rows: their scale needs all columns
        float* const out = static_cast<float*>(g.out) + (int64_t)tile.row0 * g.ld_out + no;
        for (int i = tid; i < PR * (Co / 8); i += 64 * WM * WN) {
          const int m = i / (Co / 8), c = i % (Co / 8) * 8;
          if (row_of(m) < tile.rows && no + c < Nout) {  // Nout is a multiple of 32
            float v[8];
            outputs8(m, c / 8, v);
            float* const dst = out + (int64_t)row_of(m) * g.ld_out + c;
            *reinterpret_cast<float4v*>(dst) = float4v{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<float4v*>(dst + 4) = float4v{v[4], v[5], v[6], v[7]};
          }
        }
      } else {
        const int nb = Co / 32;  // a multiple of 4: a 128-group's blocks in neighbouring lanes
        const int64_t padded = g.hrows.ld_codes / (F == SC_MXFP4 ? 16 : 32);  // blocks of a row
        static_assert(PR * Co / 32 % (64 * WM * WN) == 0, "whole rounds of threads");
        for (int i = tid; i < PR * nb; i += 64 * WM * WN) {
          const int m = i / nb, b = i % nb;
          const int64_t at = no / 32 + b;  // block of the row
          const bool valid = no + b * 32 < Nout;
          float v[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) outputs8(m, 4 * b + j, v + 8 * j);
          uint32_t w[8], sbyte = 0;
          float gs = 0.0f;
          quant_block32<F>(v, valid, g.inv_scale, w, sbyte, gs);
          if (row_of(m) >= tile.rows || at >= padded) continue;
          if (!valid) {  // past the columns, up to the chunk: zeros
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0u;
            sbyte = 0u;
          }
          const int64_t row = tile.row0 + row_of(m);
          uint8_t* const dst = static_cast<uint8_t*>(g.out) + row * g.hrows.ld_codes;
          uint8_t* const sc = g.hscales + row * g.hrows.ld_scales;
          if (F == SC_MXFP4) {
            *reinterpret_cast<uint4v*>(dst + at * 16) = uint4v{w[0], w[1], w[2], w[3]};
          } else {
            *reinterpret_cast<uint4v*>(dst + at * 32) = uint4v{w[0], w[1], w[2], w[3]};
            *reinterpret_cast<uint4v*>(dst + at * 32 + 16) = uint4v{w[4], w[5], w[6], w[7]};
          }
          if (T::MX) sc[at] = (uint8_t)sbyte;
          if (T::BLOCK && (at & 3) == 0) *reinterpret_cast<float*>(sc + at) = gs;
        }
      }
      __syncthreads();
    }
  } else {
    // Rows for the weighted sum, 16 bits a column: fp16, and for 32 neighbouring columns of
    // a row a power of two that the values are divided by, so that the largest of them
    // comes to 2^14 .. 2^15. Each is off by at most 2^-11 of itself (2^-39 of the largest
    // where it is below 2^-28 of that): bf16 rows, of the same size, would be off by 2^-8,
    // as much as y's own rounding again, and float32 rows would be another 268 MB each way
    // at 4096 tokens of 8 experts and 4096 columns. Straight from the registers: with
    // the halves of a wave exchanged a lane has eight neighbouring columns. Columns past N
    // are zeros.
    uint16_t* const d = static_cast<uint16_t*>(g.out) + (int64_t)tile.row0 * g.ld_out;
    float* const scales = g.out_scales + (int64_t)tile.row0 * (g.ld_out / 32);
    const bool inside = n0 + C <= g.N;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int nb = n0 + (wn * NT + nt) * 32;
      float b[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) b[e] = 0.0f;
      if (bias != nullptr) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int n = nb + 8 * (e / 4) + 4 * kb + e % 4;
          b[e] = n < g.N ? bf16_bits_to_f32(bias[n]) : 0.0f;
        }
      }
      float4v col[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = nb + 8 * i + 4 * kb;
        col[i] = float4v{1.f, 1.f, 1.f, 1.f};
        if constexpr (T::INT) {
          if (n < g.ntiles_w * 16) col[i] = *reinterpret_cast<const float4v*>(wscales + (int64_t)n * 4);
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float v[16];
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float s = acc[mt][nt][e];
          if constexpr (T::INT) s = int8_value((int)__float_as_uint(s), rsc[mt], col[e / 4][e % 4]);
          v[e] = alpha * s + b[e];
        }
        if (!inside) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = nb + 8 * (e / 4) + 4 * kb + e % 4 < g.N ? v[e] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) top = __builtin_fmaxf(top, __builtin_fabsf(v[e]));  // NaN is passed over
        if (__any(top == __builtin_inff())) {  // the largest finite one
          top = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = __builtin_fabsf(v[e]);
            top = x < __builtin_inff() && x > top ? x : top;
          }
        }
        uint32_t t0 = __float_as_uint(top), t1 = t0;
        swap_halves(t0, t1);
        int ex = (int)((t0 > t1 ? t0 : t1) >> 23) - 127;
        ex = ex < -112 ? -112 : ex;
        const float f = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        uint32_t w[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const half2v h = __builtin_convertvector((float2v{v[2 * x] * f, v[2 * x + 1] * f}), half2v);
          w[x] = __builtin_bit_cast(uint32_t, h);
        }
        const int m = (mt * WM + wm) * 32 + (lane & 31);
        const bool live = m < tile.rows && nb < (int)g.ld_out;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          swap_halves(w[4 * j], w[4 * j + 2]);
          swap_halves(w[4 * j + 1], w[4 * j + 3]);
        }
        if (live) {  // a row's two lanes write the one factor
          uint16_t* const at = d + (int64_t)m * g.ld_out + nb + 8 * kb;
          *reinterpret_cast<uint4v*>(at) = uint4v{w[0], w[1], w[2], w[3]};
          *reinterpret_cast<uint4v*>(at + 16) = uint4v{w[4], w[5], w[6], w[7]};
          scales[(int64_t)m * (g.ld_out / 32) + nb / 32] = __uint_as_float((uint32_t)(127 + ex - 14) << 23);
        }
      }
    }
  }
}

template <int F, int WM, int WN, int MT, int NT, int ST, bool UP>
__global__ __launch_bounds__(256, MT * NT >= 8 ? 1 : 2) void experts_tile_kernel(
    const ProductArgs g, const Meta meta) {
  typedef Traits<F> T;
  typedef TileConfig<F, WM, WN, MT, NT, ST> Cfg;
  constexpr int SUB = Cfg::SUB, PER = Cfg::PER_CHUNK, TA = Cfg::TA, TB = Cfg::TB, R = Cfg::R, L = Cfg::L;
  static_assert(!T::BLOCK && SUB == 1, "block FP8 has a kernel of its own");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Cfg::LDS];
  TileAt tile;
  if (!find_tile(g, meta, R, tile)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = lds_offset(lds);
  const int stages = (int)g.KC * PER;

  const TileLoads<F, Cfg, UP> loads(g, meta, tile, lds0, wave, lane);
  float16v acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[mt][nt][i] = 0.0f;

  // operand registers of two stages in turn. Lane l holds row l % 32 of a 32-row tile
  // and, of its 64 bytes, the two pieces l / 32 and 2 + l / 32: of an 8-bit operand the
  // first four registers are k = 16 (l / 32) .. and the last four 32 + 16 (l / 32) ..,
  // so that a 32-block lies in both lane halves (its scale comes from lanes 32 j + row,
  // j the block); MXFP4's two pieces are two 64-deep steps
  const int kb = lane >> 5, r16 = lane & 15, half = (lane >> 4) & 1;
  const int p0 = kb, p1 = kb + 2;
  const int sw = (r16 >> 2) & 3;
  const uint32_t a_at0 = (uint32_t)(half * SUB * 1024 + r16 * 64 + (p0 ^ sw) * 16);
  const uint32_t a_at1 = (uint32_t)(half * SUB * 1024 + r16 * 64 + (p1 ^ sw) * 16);
  const uint32_t b_at0 = (uint32_t)(half * SUB * 1024 + p0 * 256 + r16 * 16);
  const uint32_t b_at1 = (uint32_t)(half * SUB * 1024 + p1 * 256 + r16 * 16);
  uint4v fa[2][MT][SUB][2], fb[2][NT][SUB][2];
  int sa[2][MT], sb[2][(NT + 1) / 2];  // MX: E8M0 words
  auto read_a = [&](int slot, int q, int mt) {
    const uint8_t* const base = lds + slot * Cfg::STAGE + (mt * WM + wm) * 2 * SUB * 1024;
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      fa[q][mt][s][0] = *reinterpret_cast<const uint4v*>(base + s * 1024 + a_at0);
      fa[q][mt][s][1] = *reinterpret_cast<const uint4v*>(base + s * 1024 + a_at1);
    }
  };
  auto read_b = [&](int slot, int q, int nt) {
    const uint8_t* const base = lds + slot * Cfg::STAGE + (TA + (wn * NT + nt) * 2) * SUB * 1024;
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      fb[q][nt][s][0] = *reinterpret_cast<const uint4v*>(base + s * 1024 + b_at0);
      fb[q][nt][s][1] = *reinterpret_cast<const uint4v*>(base + s * 1024 + b_at1);
    }
  };
  // scales of a stage: chunk c (its place among four), in the first half (h = 0) or second of it
  auto read_scales = [&](int c, int h, int q) {
    if constexpr (Cfg::SCALED) {
      const uint8_t* const at = lds + Cfg::RING + ((c >> 2) & 1) * (Cfg::ASC + Cfg::BSC);
      const int cc = c & 3;
      if constexpr (T::MX) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          sa[q][mt] = (int)(*reinterpret_cast<const uint32_t*>(at + ((mt * WM + wm) * 32 + (lane & 31)) * 16 + cc * 4) >>
                            (8 * kb));
#pragma unroll
        for (int np = 0; np < (NT + 1) / 2; ++np)
          // h: the lane's block of the stage's first step; MXFP4's second is two further
          sb[q][np] = (int)(*reinterpret_cast<const uint32_t*>(at + Cfg::ASC + ((wn * NT) / 2 + np) * 1024 + cc * 256 +
                                                               (16 * (2 * h + kb) + r16) * 4) >> (8 * half));
      }
    }
  };
  int sb2[2][(NT + 1) / 2];  // MXFP4: the words of the second step
  auto read_scales2 = [&](int c, int q) {
    if constexpr (F == SC_MXFP4) {
      const uint8_t* const at = lds + Cfg::RING + ((c >> 2) & 1) * (Cfg::ASC + Cfg::BSC);
#pragma unroll
      for (int np = 0; np < (NT + 1) / 2; ++np)
        sb2[q][np] = (int)(*reinterpret_cast<const uint32_t*>(at + Cfg::ASC + ((wn * NT) / 2 + np) * 1024 + (c & 3) * 256 +
                                                              (16 * (2 + kb) + r16) * 4) >> (8 * half));
    }
  };
  auto wide = [](const uint4v& x, const uint4v& y) {
    return int8v{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };
  auto narrow = [](const uint4v& x) { return int8v{(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0}; };
  auto ints = [](const uint4v& x) { return __builtin_bit_cast(int4v, x); };

  // one accumulator tile's products of a stage; h: which half of its chunk (64-deep
  // stages). The weight is the instruction's first operand: a lane then holds one
  // activation row (lane % 32), so that a row's scale is one register, and 16 weight
  // columns, of which four at a time are neighbours
  auto mfma = [&](int q, int mt, int nt, int h) {
#define FQL_SCALED(A, B, ACC, FMT, BB, SB, BA, SA) \
  __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(B, A, ACC, FMT, FMT, BB, SB, BA, SA)
    if constexpr (T::INT) {
      int16v c = __builtin_bit_cast(int16v, acc[mt][nt]);
      c = __builtin_amdgcn_mfma_i32_32x32x32_i8(ints(fb[q][nt][0][0]), ints(fa[q][mt][0][0]), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_i32_32x32x32_i8(ints(fb[q][nt][0][1]), ints(fa[q][mt][0][1]), c, 0, 0, 0);
      acc[mt][nt] = __builtin_bit_cast(float16v, c);
    } else if constexpr (F == SC_MXFP4) {
      // the scale bytes: block kb of the step in byte 0 (second step: byte 2) of the row's
      // word, tile nt % 2 of the quad in byte 0 or 2 of the column's
      const int8v a0 = narrow(fa[q][mt][0][0]), a1 = narrow(fa[q][mt][0][1]);
      const int8v b0 = narrow(fb[q][nt][0][0]), b1 = narrow(fb[q][nt][0][1]);
      if (nt % 2 == 0) {
        acc[mt][nt] = FQL_SCALED(a0, b0, acc[mt][nt], 4, 0, sb[q][nt / 2], 0, sa[q][mt]);
        acc[mt][nt] = FQL_SCALED(a1, b1, acc[mt][nt], 4, 0, sb2[q][nt / 2], 2, sa[q][mt]);
      } else {
        acc[mt][nt] = FQL_SCALED(a0, b0, acc[mt][nt], 4, 2, sb[q][nt / 2], 0, sa[q][mt]);
        acc[mt][nt] = FQL_SCALED(a1, b1, acc[mt][nt], 4, 2, sb2[q][nt / 2], 2, sa[q][mt]);
      }
    } else if constexpr (F == SC_MXFP8) {
      const int8v a = wide(fa[q][mt][0][0], fa[q][mt][0][1]), b = wide(fb[q][nt][0][0], fb[q][nt][0][1]);
      if (h == 0) {
        if (nt % 2 == 0) acc[mt][nt] = FQL_SCALED(a, b, acc[mt][nt], 0, 0, sb[q][nt / 2], 0, sa[q][mt]);
        else acc[mt][nt] = FQL_SCALED(a, b, acc[mt][nt], 0, 2, sb[q][nt / 2], 0, sa[q][mt]);
      } else {
        if (nt % 2 == 0) acc[mt][nt] = FQL_SCALED(a, b, acc[mt][nt], 0, 0, sb[q][nt / 2], 2, sa[q][mt]);
        else acc[mt][nt] = FQL_SCALED(a, b, acc[mt][nt], 0, 2, sb[q][nt / 2], 2, sa[q][mt]);
      }
    } else {
      acc[mt][nt] = FQL_SCALED(wide(fa[q][mt][0][0], fa[q][mt][0][1]), wide(fb[q][nt][0][0], fb[q][nt][0][1]),
                               acc[mt][nt], 0, 0, 127, 0, 127);
    }
#undef FQL_SCALED
  };

  // Ring: stage i lives in slot i % ST. Slots are filled up front and stage 0's
  // operands read. Iteration i waits for the wave's own loads of stage i + 1, passes
  // the barrier (everyone's have landed, and everyone has read stage i's operands out
  // of its slot), multiplies from registers while it reads stage i + 1's operands and
  // refills slot i % ST with stage i + ST. Stages past the end are the last one again,
  // so that every iteration issues the same loads. Scales of the next four chunks are
  // loaded at the first stage of each four; they are more loads than the wait counts,
  // which only makes it wait for more.
  loads.four_scales(0, 0);
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    const int c = s < stages ? s : stages - 1;
    const uint32_t bv = loads.b_voff(c);
#pragma unroll
    for (int j = 0; j < L; ++j) loads.stage(s, c, bv, j);
  }
  wait_vmcnt<L * (ST - 1)>();
  stage_barrier();
  read_scales(0, 0, 0);
  read_scales2(0, 0);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) read_b(0, 0, nt);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) read_a(0, 0, mt);

  constexpr int FOUR = 4 * PER;  // stages of four chunks
  // row tiles of this wave that hold rows: they go to the wave rows in turn, so that an
  // expert's last rows cost what they are (in steps of 32 WM)
  const int row_tiles = (tile.rows + 31) / 32;
  const int used = (row_tiles - wm + WM - 1) / WM;
  // A row's 64 bytes of a stage are half a cache line. Where the ring is even, the activation
  // loads of stages 2 c and 2 c + 1 go out together, both halves of a tile's lines one after
  // the other, when both slots are free: a stage apart the second half came from L2 again.
  constexpr bool PAIRS = ST % 2 == 0;
  constexpr int LA = TA / Cfg::NW, LB = L - LA;
  auto iteration = [&](int i, int slot, int q, int h, bool odd, bool first_of_four) {
    // loads that may be on their way when stage i + 1 has to be there: those issued after its own
    if constexpr (!PAIRS) wait_vmcnt<L * (ST - 2)>();
    else if (odd) wait_vmcnt<LB + (ST - 2) / 2 * LB + (ST - 4) / 2 * (2 * LA + LB)>();
    else wait_vmcnt<(ST - 2) * L>();
    stage_barrier();
    const int next_slot = (slot + 1) % ST;
    if (first_of_four) loads.four_scales((i / PER + 4 < (int)g.KC ? i / PER + 4 : 0), ((i / FOUR) + 1) & 1);
    int rc = i + ST, rb = rc - 1;
    rc = rc < stages ? rc : stages - 1;
    rb = rb < stages ? rb : stages - 1;
    const uint32_t bv = loads.b_voff(rc);
    auto load = [&](int j) {  // j-th load of the iteration
      if (!PAIRS) loads.stage(slot, rc, bv, j);
      else if (!odd) loads.stage(slot, rc, bv, LA + j);
      else if (j < 2 * LA) loads.stage(j % 2 ? slot : (slot + ST - 1) % ST, j % 2 ? rc : rb, bv, j / 2);
      else loads.stage(slot, rc, bv, j - LA);
    };
    const int n = !PAIRS ? L : odd ? 2 * LA + LB : LB;
    const int ni = i + 1;
    read_scales(ni / PER, PER == 2 ? (h ^ 1) : 0, q ^ 1);
    read_scales2(ni / PER, q ^ 1);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int j = 0; j < 2 * LA + LB; ++j)
        if (j < n && (j * MT) / n == mt) load(j);
      if (mt < used) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mfma(q, mt, nt, h);
        read_a(next_slot, q ^ 1, mt);
      }
      if (mt < NT) read_b(next_slot, q ^ 1, mt);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(NT <= MT, "weight tiles read beside the rows");
  // unrolled so that slots, register sets and halves are static
  constexpr int U = ST % 2 == 0 ? ST : 2 * ST;
  for (int i0 = 0; i0 < stages; i0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < stages) iteration(i0 + u, u % ST, u % 2, PER == 2 ? u % 2 : 0, u % 2 != 0, (i0 + u) % FOUR == 0);
  }
  wait_vmcnt<0>();  // no LDS load may still be in flight when the ring is used again
  __syncthreads();

  finish_tile<F, WM, WN, MT, NT, UP>(g, meta, tile, acc, loads.wscales, tile.ngroup * TB * 16, lds);
}

// Block FP8: 32 MT WM rows x 256 columns, 32 MT x 64 a wave. Every 128-deep chunk's products go
// into a fresh accumulator, which vector instructions add: from vector registers, since
// from accumulation registers each addition would cost a move besides. That leaves 256
// registers: 128 for the sums, 32 for the products of two tiles in turn (a tile's are
// added while the next one's are made), 32 for the chunk's weight tiles and 32 for two
// row tiles in turn. So operands are read one row tile ahead, and the weight tiles of
// the next chunk behind the last products that need the old ones.
// EARLY: a refill's loads go out in its first EARLY of P steps (a ring of two chunks
// leaves them little more than one chunk's time).
template <int WM, int MT, int ST, int EARLY, bool UP>
__global__ __launch_bounds__(256 * WM, 2) void experts_block_kernel(const ProductArgs g, const Meta meta) {
  constexpr int F = SC_FP8_BLOCK, WN = 4, NT = 2;
  typedef TileConfig<F, WM, WN, MT, NT, ST> Cfg;
  constexpr int TA = Cfg::TA, TB = Cfg::TB, R = Cfg::R, L = Cfg::L, P = MT * NT;
  static_assert(EARLY >= NT && EARLY <= P, "refill steps");
  static_assert(MT % 2 == 0, "row tiles in two register sets");
  extern __shared__ __attribute__((aligned(1024))) uint8_t block_lds[];  // Cfg::LDS bytes
  uint8_t* const lds = block_lds;
  TileAt tile;
  if (!find_tile(g, meta, R, tile)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const TileLoads<F, Cfg, UP> loads(g, meta, tile, lds_offset(lds), wave, lane);
  const int chunks = (int)g.KC;

  float16v acc[MT][NT], part[2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[mt][nt][i] = 0.0f;

  const int kb = lane >> 5, r16 = lane & 15, half = (lane >> 4) & 1;
  const int sw = (r16 >> 2) & 3;
  const uint32_t a_at0 = (uint32_t)(half * 2048 + r16 * 64 + (kb ^ sw) * 16);
  const uint32_t a_at1 = (uint32_t)(half * 2048 + r16 * 64 + ((kb + 2) ^ sw) * 16);
  const uint32_t b_at = (uint32_t)(half * 2048 + kb * 256 + r16 * 16);
  uint4v fa[2][2][2], fb[NT][2][2];  // [set or tile][piece of the chunk][16 bytes]
  float rs[MT];                      // the lane's row scales times the column block's
  auto read_a = [&](int slot, int mt) {
    const uint8_t* const base = lds + slot * Cfg::STAGE + (mt * WM + wm) * 4096;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      fa[mt & 1][s][0] = *reinterpret_cast<const uint4v*>(base + s * 1024 + a_at0);
      fa[mt & 1][s][1] = *reinterpret_cast<const uint4v*>(base + s * 1024 + a_at1);
    }
  };
  auto read_b = [&](int slot, int nt) {
    const uint8_t* const base = lds + slot * Cfg::STAGE + (TA + (wn * NT + nt) * 2) * 2048;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      fb[nt][s][0] = *reinterpret_cast<const uint4v*>(base + s * 1024 + b_at);
      fb[nt][s][1] = *reinterpret_cast<const uint4v*>(base + s * 1024 + b_at + 512);
    }
  };
  auto read_rs = [&](int c, int mt) {
    const uint8_t* const at = lds + Cfg::RING + ((c >> 2) & 1) * (Cfg::ASC + Cfg::BSC) + (c & 3) * 4;
    rs[mt] = *reinterpret_cast<const float*>(at + ((mt * WM + wm) * 32 + (lane & 31)) * 16) *
             *reinterpret_cast<const float*>(at + Cfg::ASC + (wn * NT * 32 / 128) * 256);
  };
  auto wide = [](const uint4v& x, const uint4v& y) {
    return int8v{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };
  auto add_part = [&](int t) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t / NT][t % NT][i] = __builtin_fmaf(part[t & 1][i], rs[t / NT], acc[t / NT][t % NT][i]);
    __asm__ volatile("" : "+v"(acc[t / NT][t % NT]));  // here, not where the sum is used next
  };
  // A chunk's refill (of the slot that it leaves, with the chunk ST further on) begins in
  // its last row tile, behind the barrier after which nobody reads the slot, and goes on
  // through the next chunk: load j at step (j EARLY) / L of the steps counted from there.
  auto refill = [&](int slot, int c, int step) {
    const int rc = c < chunks ? c : chunks - 1;  // past the end: the last chunk again
    const uint32_t bv = loads.b_voff(rc);
#pragma unroll
    for (int j = 0; j < L; ++j)
      if ((j * EARLY) / L == step) loads.stage(slot, rc, bv, j);
  };
  const int used = ((tile.rows + 31) / 32 - wm + WM - 1) / WM;  // row tiles of this wave that hold rows
  loads.four_scales(0, 0);
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) {
    const int c = s < chunks ? s : chunks - 1;
    const uint32_t bv = loads.b_voff(c);
#pragma unroll
    for (int j = 0; j < L; ++j) loads.stage(s, c, bv, j);
  }
  wait_vmcnt<L * (ST - 2)>();
  stage_barrier();
#pragma unroll
  for (int u = 0; u < NT; ++u) refill(ST - 1, ST - 1, u);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) read_b(0, nt);
  read_a(0, 0);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) read_rs(0, mt);
#pragma unroll
  for (int i = 0; i < 16; ++i) part[1][i] = 0.0f;  // (P is even: "the tile before" of the first one)

  auto chunk = [&](int i, int slot) {
    const int next = (slot + 1) % ST, before = (slot + ST - 1) % ST;
    if ((i & 3) == 0) loads.four_scales(i + 4 < chunks ? i + 4 : 0, ((i >> 2) + 1) & 1);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt == MT - 1) {
        wait_vmcnt<L * (ST - 2)>();  // this wave's loads of the next chunk
        stage_barrier();             // everyone's, and everyone is done with this chunk's slot
        read_a(next, 0);
      } else {
        read_a(slot, mt + 1);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int t = mt * NT + nt;
        if (mt < used) {
#pragma unroll
          for (int x = 0; x < 16; ++x) part[t & 1][x] = 0.0f;
#pragma unroll
          for (int s = 0; s < 2; ++s)
            part[t & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(fb[nt][s][0], fb[nt][s][1]),
                                                                          wide(fa[mt & 1][s][0], fa[mt & 1][s][1]),
                                                                          part[t & 1], 0, 0, 0, 127, 0, 127);
        }
        if (mt == MT - 1) refill(slot, i + ST, nt);
        else refill(before, i - 1 + ST, NT + t);
        // both products are on their way before the additions wait for the last ones
        __asm__ volatile("" : "+v"(part[t & 1]));
        __builtin_amdgcn_sched_barrier(0);
        if ((t + P - 1) % P / NT < used) add_part((t + P - 1) % P);
        if (t == 0) read_rs(i, MT - 1);
        if (mt == MT - 1) {
          read_b(next, nt);
          if (nt == NT - 1) {
#pragma unroll
            for (int r = 0; r < MT - 1; ++r) read_rs(i + 1, r);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  for (int i0 = 0; i0 < chunks; i0 += ST) {
#pragma unroll
    for (int u = 0; u < ST; ++u)
      if (i0 + u < chunks) chunk(i0 + u, u);
  }
  if (MT - 1 < used) add_part(P - 1);
  wait_vmcnt<0>();  // no LDS load may still be in flight when the ring is used again
  __syncthreads();
  finish_tile<F, WM, WN, MT, NT, UP>(g, meta, tile, acc, loads.wscales, tile.ngroup * TB * 16, lds);
}

}  // namespace
}  // namespace fql
