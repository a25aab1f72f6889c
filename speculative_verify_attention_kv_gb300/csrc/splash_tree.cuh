// Row blocks, masks and workspace layout of attention over a tree of drafts.
#pragma once

#include "splash_common.cuh"

namespace splash {

// Nodes of a tree at most (8 words of a mask).
constexpr int kMaxTreeNodes = 256;

// The T * G query rows of a sequence and KV head (row t * G + g) are cut into as
// few row blocks of at most kMaxRows as hold them, all of about the same height,
// since a tile costs nearly the same whatever the rows (see tile_cost).
struct RowBlocks {
  int count;         // blocks
  int rows;          // rows of a block (the last may have fewer)
};
__host__ __device__ inline RowBlocks row_blocks(int T, int group) {
  const int all = T * group;
  const int n = (all + kMaxRows - 1) / kMaxRows;
  return RowBlocks{n, n > 0 ? (all + n - 1) / n : 0};
}

// Byte offsets of the workspace regions (256-aligned). A CTA's range of tiles
// shares at most its first and its last unit with other CTAs, so the partial rows
// need no plan: CTA c has two places of kMaxRows rows, 2c for a segment that
// begins inside a unit and 2c + 1 for one that begins a unit.
struct TreeLayout {
  size_t q_off;        // int32 [B+1]   first token row of each sequence
  size_t seq_T;        // int32 [B]     validated node count (0 if skipped)
  size_t seq_ctx;      // int32 [B]
  size_t stp;          // int32 [B+1]   exclusive prefix of tiles per sequence
  size_t wcost;        // int64 [B+1]   exclusive prefix of sequence costs
  size_t cta_start;    // int32 [kMaxCtas+1] first tile of each CTA
  size_t lse_part;     // fp32  [rows_bound]
  size_t o_part;       // fp32  [rows_bound, D]
  size_t total;
};

__host__ __device__ inline TreeLayout make_tree_layout(int B, int D, long long rows_bound) {
  TreeLayout L;
  size_t o = align256(sizeof(PlanHeader));
  L.q_off = o;      o = align256(o + sizeof(int) * (size_t)(B + 1));
  L.seq_T = o;      o = align256(o + sizeof(int) * (size_t)B);
  L.seq_ctx = o;    o = align256(o + sizeof(int) * (size_t)B);
  L.stp = o;        o = align256(o + sizeof(int) * (size_t)(B + 1));
  L.wcost = o;      o = align256(o + sizeof(long long) * (size_t)(B + 1));
  L.cta_start = o;  o = align256(o + sizeof(int) * (size_t)(kMaxCtas + 1));
  L.lse_part = o;   o = align256(o + sizeof(float) * (size_t)rows_bound);
  L.o_part = o;     o = align256(o + sizeof(float) * (size_t)rows_bound * D);
  L.total = o;
  return L;
}
__host__ __device__ inline long long tree_rows_bound(int ncta) { return 2LL * kMaxRows * ncta; }

struct TreeAttnParams : AttnParams {
  const int32_t* tree_masks;      // [num_q_tokens, mask_stride]
  int mask_stride;
};

// Which of the 16 keys from node n0 on (nodes below 0 are context keys) a row
// sees: bit i for node n0 + i. `mask`: the row's words; T nodes in the tree.
__device__ inline uint32_t tree_bits16(const int32_t* __restrict__ mask, int n0, int T) {
  if (n0 <= -16) return 0xffffu;
  const int lo = n0 > 0 ? n0 : 0;
  if (lo >= T) return n0 < 0 ? (1u << -n0) - 1 : 0u;       // T = 0 does not occur
  const int w = lo >> 5;
  const uint32_t w0 = (uint32_t)__ldg(mask + w);
  const uint32_t w1 = (w + 1) * 32 < T ? (uint32_t)__ldg(mask + w + 1) : 0u;
  uint32_t bits = __funnelshift_r(w0, w1, lo & 31);
  if (T - lo < 32) bits &= (1u << (T - lo)) - 1;
  if (n0 < 0) bits = (bits << -n0) | ((1u << -n0) - 1);
  return bits & 0xffffu;
}

}  // namespace splash
