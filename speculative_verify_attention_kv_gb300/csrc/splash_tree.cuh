// Row blocks, masks and workspace layout of attention over a tree of drafts.
#pragma once

#include <climits>

#include "splash_common.cuh"

namespace splash {

// Nodes of a tree at most (8 words of a mask).
constexpr int kMaxTreeNodes = 256;

// The T * G query rows of a sequence and KV head (row t * G + g) are cut into as
// few row blocks of at most kMaxRows as hold them, all of about the same height,
// since a tile costs nearly the same whatever the rows (see kTreeTileCost).
struct RowBlocks {
  int count;         // blocks
  int rows;          // rows of a block (the last may have fewer)
};
__host__ __device__ inline RowBlocks row_blocks(int T, int group) {
  const int all = T * group;
  const int n = (all + kMaxRows - 1) / kMaxRows;
  return RowBlocks{n, n > 0 ? (all + n - 1) / n : 0};
}

// Tiles of the stream (64 keys each) and its cut over the CTAs. Units are (sequence,
// KV head, row block), the blocks of a head next to each other; the rows of a sequence
// lie at the sum of the caller's lengths before it, a rejected sequence's too.
constexpr int kTreeTile = 64;
// What a query row adds to a tile and a segment to its tiles, a tile being 4096. Fits of
// the CTAs' times on ragged batches say, us a tile / row and tile / segment: heads of 256
// 0.93 / 0.0017 / 8.2, of 128 0.63 / 0.0030 / 5.6, of 64 0.57 / 0.0021 / 3.4. Calls, mean
// us of six ragged batches each at (row, segments in tiles) (6, 6), (6, 9), (14, 6), (14,
// 9), (19, 9): heads of 256 71.7, 70.7, 73.0, 70.8, 71.9; of 128 55.5, 54.7, 56.5, 54.1,
// 54.9; of 64 47.6, 48.9, 47.6, 48.6, 48.9. 32 sequences of 256..16384 keys, heads of
// 256: 172 us at (6, 6), 156 at (6, 9), 170 at (6, 20). (With the kernel as it is now
// tiles are 5% shorter and six batches of heads of 256 take 69.9, 67.3 and 67.6 us at
// (14, 6), (6, 9) and (14, 9): the same order.)
constexpr int kTreeTileCost = 4096;
__host__ __device__ constexpr int tree_row_cost(int D) { return D > 128 ? 6 : 14; }
__host__ __device__ constexpr int tree_segment_cost(int D) { return (D > 64 ? 9 : 6) * 4096; }
struct TreeSeq {
  bool ok;               // lengths in range; else T = ctx = 0
  int T, ctx;
  int laid;              // rows that the sequence takes up
  int tiles;             // of a unit
  RowBlocks rb;
  __device__ TreeSeq(int block_len, int context_len, int group, int max_block_len, int max_pages) {
    laid = block_len > 0 ? block_len : 0;
    ok = block_len >= 0 && context_len >= 0 && block_len <= max_block_len &&
                    (long long)context_len + block_len <= (long long)max_pages * kPageSize;
    T = ok ? block_len : 0;
    ctx = ok ? context_len : 0;
    rb = row_blocks(T, group);
    tiles = T > 0 ? (ctx + T + kTreeTile - 1) / kTreeTile : 0;
  }
  __device__ long long units(int hkv) const { return (long long)hkv * rb.count; }
  __device__ long long unit_cost(int row_cost, int segment_cost) const {
    return (long long)tiles * (kTreeTileCost + row_cost * rb.rows) + segment_cost;
  }
};

// Where a CTA's range begins: a tile of sequence b, whose rows begin at q_off.
struct TreeStart {
  int b, local, q_off, count;      // local: from the sequence's first tile; count: tiles
};
// A unit that CTAs cta .. cta + parts - 1 share: rows r0 .. of the sequence and head.
struct TreeSplit {
  int cta, parts, q_off, r0, rows, h, pad_[2];
};
static_assert(sizeof(TreeStart) == 16 && sizeof(TreeSplit) == 32, "plan records");
struct TreeHeader {
  int num_splits;
  int ncta;                        // CTAs that own tiles
};

// Byte offsets of the workspace regions (256-aligned). A CTA's range of tiles
// shares at most its first and its last unit with other CTAs, so the partial rows
// need no plan: CTA c has two places of kMaxRows rows, 2c for a segment that
// begins inside a unit and 2c + 1 for one that begins a unit.
struct TreeLayout {
  size_t starts;       // TreeStart [kMaxCtas]
  size_t splits;       // TreeSplit [kMaxCtas]
  size_t stp;          // int32 [B+1]   first tile of each sequence  (large batches only)
  size_t cost;         // int64 [B+1]   cost before each sequence    (large batches only)
  size_t q_off;        // int32 [B]     first row of each sequence   (large batches only)
  size_t lse_part;     // fp32  [rows_bound]
  size_t o_part;       // fp32  [rows_bound, D]
  size_t total;
};

// Batches that the attention kernel plans by itself, every CTA alike, with a thread
// per sequence. It costs about what a launch before it would (5500 clocks, 3 us, at 16
// sequences), but the pipeline's set-up and the tensor maps' fetch run beside it: a call
// of one sequence 16.5 us, with the planner as a launch 18.5 (17.7 since weights carry a
// factor for the V scales).
constexpr int kTreeSelfPlan = 512;

__host__ __device__ inline TreeLayout make_tree_layout(int B, int D, long long rows_bound) {
  TreeLayout L;
  const size_t n = B > kTreeSelfPlan ? (size_t)B + 1 : 0;
  size_t o = align256(sizeof(TreeHeader));
  L.starts = o;     o = align256(o + sizeof(TreeStart) * (size_t)kMaxCtas);
  L.splits = o;     o = align256(o + sizeof(TreeSplit) * (size_t)kMaxCtas);
  L.stp = o;        o = align256(o + sizeof(int) * n);
  L.cost = o;       o = align256(o + sizeof(long long) * n);
  L.q_off = o;      o = align256(o + sizeof(int) * n);
  L.lse_part = o;   o = align256(o + sizeof(float) * (size_t)rows_bound);
  L.o_part = o;     o = align256(o + sizeof(float) * (size_t)rows_bound * D);
  L.total = o;
  return L;
}
__host__ __device__ inline long long tree_rows_bound(int ncta) { return 2LL * kMaxRows * ncta; }

struct TreeAttnParams : AttnParams {
  const int32_t* context_lens;
  const int32_t* block_lens;
  int max_block_len;
  int num_q_tokens;
  const int32_t* tree_masks;      // [num_q_tokens, mask_stride]
  int mask_stride;
  int row_cost, segment_cost;
};

// ------------------------------------------------------------------------- plan
struct PlanSums {
  long long rows, tiles, cost;
  __device__ PlanSums operator+(const PlanSums& o) const {
    return PlanSums{rows + o.rows, tiles + o.tiles, cost + o.cost};
  }
};
__device__ inline PlanSums shfl_up(const PlanSums& v, int o) {
  return PlanSums{__shfl_up_sync(0xffffffffu, v.rows, o), __shfl_up_sync(0xffffffffu, v.tiles, o),
                  __shfl_up_sync(0xffffffffu, v.cost, o)};
}
// What the passes over a batch share: prefix sums in shared memory or the workspace.
struct PlanArrays {
  long long* cost;     // [B]
  int* stp;            // [B] first tile
  int* q_off;          // [B] first row
  int* start;          // [kMaxCtas + 1] first tile of each CTA (shared memory)
  PlanSums* warp_sums; // [32]
  int* warp_max;       // [32]
  int* carry;          // [1]
};

// Plans a batch with all threads of a CTA: fills the arrays and returns the CTAs that
// own tiles (0: nothing to do, or lengths that sum past the caller's rows). `speaks`:
// this CTA reports bad lengths.
__device__ inline int plan_tree(const TreeAttnParams& p, const PlanArrays& a, int ncta,
                                bool speaks) {
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int nw = threads >> 5, B = p.num_seqs, hkv = p.num_kv_heads;
  PlanSums run{0, 0, 0};
  for (int base = 0; base < B; base += threads) {
    const int b = base + tid;
    PlanSums mine{0, 0, 0};
    if (b < B) {
      const TreeSeq s(p.block_lens[b], p.context_lens[b], p.group, p.max_block_len,
                      p.max_pages_per_seq);
      if (speaks && !s.ok) report(p.device_status, SPLASH_DEVICE_BAD_LENGTH);
      const long long units = s.T > 0 ? s.units(hkv) : 0;
      mine = PlanSums{s.laid, units * s.tiles, units > 0 ? units * s.unit_cost(p.row_cost, p.segment_cost) : 0};
    }
    PlanSums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const PlanSums y = shfl_up(incl, o);
      if (lane >= o) incl = incl + y;
    }
    if (lane == 31) a.warp_sums[warp] = incl;
    __syncthreads();
    PlanSums before = run;
    for (int w = 0; w < nw; ++w) {
      if (w == warp) before = run;
      run = run + a.warp_sums[w];
    }
    if (b < B) {
      a.cost[b] = before.cost + incl.cost - mine.cost;
      a.stp[b] = (int)min(before.tiles + incl.tiles - mine.tiles, (long long)INT_MAX);
      a.q_off[b] = (int)min(before.rows + incl.rows - mine.rows, (long long)p.num_q_tokens);
    }
    __syncthreads();
  }
  const bool ok = run.rows <= p.num_q_tokens && run.tiles < INT_MAX;
  if (!ok && speaks && tid == 0) report(p.device_status, SPLASH_DEVICE_BAD_LENGTH);
  const int total = ok ? (int)run.tiles : 0;
  // at most one CTA per tile: every CTA owns tiles, and the CTAs of a unit are
  // consecutive
  const int n = min(min(ncta, total), kMaxCtas);
  if (tid == 0) *a.carry = INT_MIN;
  // CTA k starts where the cumulative cost reaches k / n of the total: the
  // sequence, then the unit, then the tile (a unit's first segment cost maps to
  // its first tile); then the starts are made strictly increasing, the last
  // ones pulled back so that every CTA has a tile
  for (int base = 0; n > 0 && base <= n; base += threads) {
    const int k = base + tid;
    int start = 0;
    if (k >= n) {
      start = total;
    } else if (k > 0) {
      const long long target = run.cost / n * k + run.cost % n * k / n;
      const int b = upper_index(a.cost, B - 1, target);
      const TreeSeq s(p.block_lens[b], p.context_lens[b], p.group, p.max_block_len,
                      p.max_pages_per_seq);
      const long long uc = s.unit_cost(p.row_cost, p.segment_cost), off = target - a.cost[b];
      const int u = (int)min(off / uc, s.units(hkv) - 1);
      const long long rem = off - u * uc - p.segment_cost;
      const long long w = kTreeTileCost + p.row_cost * s.rb.rows;
      const int t = rem < 0 ? 0 : (int)min(rem / w, (long long)s.tiles - 1);
      start = a.stp[b] + u * s.tiles + t;
    }
    int y = k <= n ? start - k : INT_MIN;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y = max(y, z);
    }
    if (lane == 31) a.warp_max[warp] = y;
    __syncthreads();
    y = max(y, *a.carry);
    for (int w = 0; w < warp; ++w) y = max(y, a.warp_max[w]);
    if (k <= n) a.start[k] = min(y + k, total - (n - k));
    __syncthreads();
    if (tid == threads - 1) *a.carry = y;
  }
  __syncthreads();
  return n;
}

// The start of CTA k of a plan.
__device__ inline TreeStart start_of(const PlanArrays& a, int B, int k) {
  const int t = a.start[k], b = upper_index(a.stp, B - 1, t);
  return TreeStart{b, t - a.stp[b], a.q_off[b], a.start[k + 1] - t};
}

// The start of this CTA of the attention kernel, false when it has no tiles. Small batches
// are planned here, with `room` (kTreePlanRoom bytes, free again afterwards) for the
// arrays; CTA 0 notes what the combine needs.
constexpr int kTreePlanRoom = kTreeSelfPlan * 16 + (kMaxCtas + 1) * 4 + 32 * 24 + 32 * 4 + 16;
__device__ inline void note_splits(const TreeAttnParams&, const PlanArrays&, int, TreeHeader*,
                                   TreeSplit*);
__device__ inline bool tree_start(const TreeAttnParams& p, unsigned char* room, TreeStart& start) {
  const TreeLayout L = make_tree_layout(p.num_seqs, p.head_dim, tree_rows_bound(gridDim.x));
  TreeHeader* hd = reinterpret_cast<TreeHeader*>(p.ws);
  const int c = blockIdx.x;
  if (p.num_seqs > kTreeSelfPlan) {
    if (c >= hd->ncta) return false;
    start = reinterpret_cast<const TreeStart*>(p.ws + L.starts)[c];
    return true;
  }
  PlanArrays a;
  a.cost = reinterpret_cast<long long*>(room);
  a.warp_sums = reinterpret_cast<PlanSums*>(a.cost + kTreeSelfPlan);
  a.stp = reinterpret_cast<int*>(a.warp_sums + 32);
  a.q_off = a.stp + kTreeSelfPlan;
  a.start = a.q_off + kTreeSelfPlan;
  a.warp_max = a.start + kMaxCtas + 1;
  a.carry = a.warp_max + 32;
  const int n = plan_tree(p, a, gridDim.x, c == 0);
  if (c < n) start = start_of(a, p.num_seqs, c);
  if (c == 0) note_splits(p, a, n, hd, reinterpret_cast<TreeSplit*>(p.ws + L.splits));
  __syncthreads();
  return c < n;
}

// The units that CTAs share, each once: CTA k finds the one that it continues, and notes
// it if CTA k - 1 began it. (All threads of one CTA; the order does not matter.)
__device__ inline void note_splits(const TreeAttnParams& p, const PlanArrays& a, int n,
                                   TreeHeader* hd, TreeSplit* splits) {
  __syncthreads();
  if (threadIdx.x == 0) *a.carry = 0;
  __syncthreads();
  for (int k = 1 + threadIdx.x; k < n; k += blockDim.x) {
    const TreeStart st = start_of(a, p.num_seqs, k);
    const TreeSeq s(p.block_lens[st.b], p.context_lens[st.b], p.group, p.max_block_len,
                    p.max_pages_per_seq);
    const int u = st.local / s.tiles, first = a.start[k] - (st.local - u * s.tiles);
    if (first == a.start[k] || a.start[k - 1] > first) continue;
    const int last = upper_index(a.start, n - 1, first + s.tiles - 1);
    const int h = u / s.rb.count, r0 = (u - h * s.rb.count) * s.rb.rows;
    splits[atomicAdd(a.carry, 1)] =
        TreeSplit{k - 1, last - k + 2, st.q_off, r0, min(s.rb.rows, s.T * p.group - r0), h, {0, 0}};
  }
  __syncthreads();
  if (threadIdx.x == 0) *hd = TreeHeader{*a.carry, n};
}

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
