// Internal declarations of the 8-bit serving operators: the norm with an
// 8-bit output, the linear layer's fused epilogue, the paged 8-bit cache and
// the attention over it.
#pragma once

#include "fql_internal.h"

namespace fql {

// ---- 8-bit activation operands ---------------------------------------------
// The activation operand of the scaled-MFMA GEMMs (the layout of ScDims) on
// its own: [codes | scales] of M rows padded to kOperandRows, the largest row
// tile of any launch plan, so that one operand serves every plan. Rows past M
// are never written and may hold anything: an output row depends on its own
// activation row only, and rows past M are not stored. Columns past K (up to
// the chunk of 128) are written as zeros.
constexpr int64_t kOperandRows = 256;
inline ScDims operand_dims(int fmt, int64_t M, int64_t K) {
  return sc_dims(fmt, round_up(M, kOperandRows), K, false);
}

// bf16 x quantized into an operand's codes and scales (either layout's row
// padding; rows past M are not written).
hipError_t launch_quant_operand(int fmt, const uint16_t* x, int64_t M, int64_t K, int64_t ldx, bool aligned,
                                float inv_scale, uint8_t* codes, void* scales, hipStream_t st);

// ---- residual add + root-mean-square norm + 8-bit quantizer ------------------
struct NormArgs {
  const uint16_t* x;         // bf16 [M][ldx]
  int64_t M, K, ldx;
  const uint16_t* residual;  // bf16 [M][ldr] or null
  int64_t ldr;
  const uint16_t* weight;    // bf16 [K]
  float eps;
  float inv_scale;           // per-tensor FP8: fl32(1 / scale)
  uint8_t* codes;            // canonical [M][K], or the operand's codes
  void* scales;              // canonical (MXFP8 [M][K/32] bytes, block FP8 [M][K/128] floats), or the operand's
  uint16_t* h;               // bf16 [M][ldh]: x + residual (null without a residual)
  int64_t ldh;
};
hipError_t launch_rms_norm_quant(int fmt, bool operand, const NormArgs& a, hipStream_t st);
// INT8, as an operand (scales: float32, one a row)
hipError_t launch_rms_norm_int8(const NormArgs& a, hipStream_t st);

// ---- linear layer with a fused epilogue --------------------------------------
// y = bf16(act(alpha * acc + bias) + residual). kActSwiglu: the N columns come
// in groups of 16 gate columns followed by their 16 up columns, and the N / 2
// outputs are silu(gate) * up.
enum ScAct { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActSwiglu = 5 };
struct ScEpilogue {
  int act;
  const uint16_t* residual;  // bf16 [M][ldr] or null; may be y itself
  int64_t ldr;
};
ScPlan plan_sc_fused(int fmt, int64_t M, int64_t N, int64_t K);
ScPlan cached_plan_sc_fused(int fmt, int64_t M, int64_t N, int64_t K);
// launch_sc_linear with the epilogue above, on a plan of plan_sc_fused. x is used when x_operand is null;
// x_operand is an operand of operand_dims(p.fmt, M, K).
hipError_t launch_sc_linear_fused(const ScPlan& p, const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                  bool aligned, float inv_scale, const uint8_t* x_operand,
                                  const uint8_t* packed, int64_t N, float alpha, const float* alpha_dev,
                                  const uint16_t* bias, const ScEpilogue& epi, uint16_t* y, int64_t ldy,
                                  uint8_t* workspace, hipStream_t st);

// ---- paged 8-bit cache -------------------------------------------------------
// Keys   E4M3 [blocks][heads][block_size][D]
// Values E4M3 [blocks][heads][block_size / 16][D][16]: within 16 tokens the
//        tokens of one channel are neighbours, which is the order the second
//        matrix product of the attention reads them in.
// Scales E8M0 [blocks][heads] for each of the two (value = code * 2^(byte - 127)).
// Scales are powers of two: E4M3 keeps its relative precision under any scale,
// so a finer scale would buy less than a bit of range, and a grown scale then
// re-rounds the codes already stored only where they fall below E4M3's normal
// range.
struct PagedCache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int64_t num_blocks;
  int heads, block_size, D;
};
// Where the tokens of a batch lie. All arrays are in device memory and are
// not trusted: kernels clamp the row ranges to [0, T], the lengths to the
// table's capacity, and skip blocks whose number is outside the cache.
struct PagedBatch {
  const int32_t* table;  // [B][ld_table]
  int64_t ld_table;
  int table_cols;
  const int32_t* lens;  // [B] tokens of each sequence, the new ones included
  const int32_t* cu;    // [B + 1] first row of each sequence's new tokens
  int B;
  int64_t T;    // rows of the new-token tensors
  int max_new;  // upper bound of cu[b + 1] - cu[b]
};

#ifdef __HIPCC__
// One sequence's rows and positions from untrusted device metadata.
struct SeqSpan {
  int64_t row0;  // first row of its new tokens
  int n;         // new tokens
  int len;       // tokens with the new ones (at most the table's capacity)
  int pos0;      // position of its first new token (negative when lens[b] < n)
};
__host__ __device__ __forceinline__ SeqSpan seq_span(const PagedBatch& pb, int b, int block_size) {
  SeqSpan s;
  int64_t c0 = pb.cu[b], c1 = pb.cu[b + 1];
  c0 = c0 < 0 ? 0 : (c0 > pb.T ? pb.T : c0);
  c1 = c1 < c0 ? c0 : (c1 > pb.T ? pb.T : c1);
  const int64_t n = c1 - c0;
  s.row0 = c0;
  s.n = (int)(n < pb.max_new ? n : pb.max_new);
  const int64_t cap = (int64_t)pb.table_cols * block_size;
  const int64_t len = pb.lens[b];
  s.pos0 = (int)((len < 0 ? 0 : len) - n);
  s.len = (int)(len < 0 ? 0 : (len < cap ? len : cap));
  return s;
}

// The keys that the rows of a sequence's new token see: [lo, hi), empty where
// hi <= lo (hi may be negative).
struct Visible {
  int lo, hi;
};
__host__ __device__ __forceinline__ Visible visible_keys(const SeqSpan& s, int token, int causal, int window) {
  const int p = s.pos0 + token;
  Visible v;
  v.hi = causal ? (p + 1 < s.len ? p + 1 : s.len) : s.len;
  v.lo = window > 0 && p >= window ? p - window + 1 : 0;
  return v;
}
#endif

hipError_t launch_kv_append(const PagedCache& c, const PagedBatch& pb, const uint16_t* k, const uint16_t* v,
                            int64_t k_ld_token, int64_t k_ld_head, int64_t v_ld_token, int64_t v_ld_head,
                            bool aligned, hipStream_t st);

// ---- attention over the paged cache ------------------------------------------
struct AttnPlan {
  int kind;        // 0: 16 * cols query rows per workgroup, every wave its own keys;
                   // 1: 32 query rows per wave, cols waves, keys shared through LDS
  int cols;
  int row_tiles;   // row tiles of one (sequence, kv head)
  int splits;      // ranges of keys (1: written directly)
  int chunk;       // keys of one range (a multiple of 64)
  int64_t counter_bytes, partial_bytes, total_bytes;
};
// max_len: upper bound of lens.
AttnPlan plan_attention(int B, int Hq, int Hkv, int D, int64_t max_new, int64_t max_len, int window);
std::string describe_attention(const AttnPlan& p, int D);

struct AttnArgs {
  const uint16_t* q;  // bf16, element (t, h, d) at t * q_ld_token + h * q_ld_head + d
  int64_t q_ld_token, q_ld_head;
  uint16_t* out;      // bf16, likewise
  int64_t o_ld_token, o_ld_head;
  float* lse;         // float32 [T][Hq] or null: log of the softmax's denominator (natural)
  int Hq;
  int group;             // query heads of one kv head, Hq / heads
  uint32_t group_mul;    // n / group = (n * group_mul) >> group_shift for 0 <= n < 2^31
  int group_shift;       // (both set by launch_attention)
  float scale;        // of the scores
  int causal;
  int window;         // keys at positions <= p - window are hidden from position p; 0: none
  bool aligned;       // q rows 16-byte aligned
};
hipError_t launch_attention(const AttnPlan& p, AttnArgs a, const PagedCache& c, const PagedBatch& pb,
                            uint8_t* workspace, hipStream_t st);

}  // namespace fql
