// Attention over a tree of drafts: split plan, log-sum-exp combine and C entry. The
// attention itself is verify_tc.cu's kernel with tree masks.
//
// Work unit = (sequence b, KV head h, row block k): up to kMaxRows of the T_b * G
// query rows against keys 0 .. ctx_b + T_b - 1. As in the plan of a chain, the
// 64-key tiles of all units form one stream, cut over the persistent CTAs into
// ranges of about equal estimated cost. A unit inside one CTA's range is finished
// there; otherwise every CTA that shares it leaves a partial (o_i normalised by its
// own sum, lse_i) in one of its two places (splash_tree.cuh), and the combine
// merges them:
//   lse = ln sum_i exp(lse_i),  O = sum_i exp(lse_i - lse) o_i
// A row that sees nothing (an empty mask and no context) has lse = -inf and O = 0,
// whole or in parts.
#include <climits>

#include "splash_common.cuh"
#include "splash_host.cuh"
#include "splash_tree.cuh"

namespace splash {

cudaError_t launch_verify_tree(const TreeAttnParams&, int, cudaStream_t);
bool tc_supported(int head_dim);

namespace {

constexpr int kTile = 64;
// Threads of the plan's one CTA: few warps make its block-wide barriers cheaper.
constexpr int kPlanSmall = 128;
constexpr int kPlanLarge = 1024;
// Sequences whose prefix sums the plan keeps in shared memory (28 KB).
constexpr int kPlanSmemSeqs = 1024;

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
// Exclusive scan over the CTA (any multiple of 32 threads); *total receives the sum.
__device__ inline PlanSums exclusive_scan(const PlanSums& v, PlanSums* s_warp, PlanSums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const PlanSums zero{0, 0, 0};
  PlanSums incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const PlanSums y = shfl_up(incl, o);
    if (lane >= o) incl = incl + y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  PlanSums before = zero, all = zero;
  for (int w = 0; w < nw; ++w) {
    if (w == warp) before = all;
    all = all + s_warp[w];
  }
  *total = all;
  __syncthreads();
  return PlanSums{before.rows + incl.rows - v.rows, before.tiles + incl.tiles - v.tiles,
                  before.cost + incl.cost - v.cost};
}
// Inclusive max-scan over the CTA.
__device__ inline int inclusive_max(int v, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = max(incl, y);
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl = max(incl, s_warp[w]);
  __syncthreads();
  return incl;
}

struct PlanParams {
  const int32_t* context_lens;
  const int32_t* block_lens;
  int num_seqs, num_kv_heads, group, max_pages, max_block_len, ncta, num_q_tokens;
  unsigned char* ws;
  int* status;
};

__host__ __device__ inline long long unit_cost(int tiles, int rows) {
  return (long long)tiles * (tile_cost(kClassTensor) + row_cost(kClassTensor) * rows) +
         segment_cost(kClassTensor);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) tree_plan_kernel(PlanParams p) {
  __shared__ PlanSums s_warp[kThreads / 32];
  __shared__ int s_max[kThreads / 32];
  __shared__ int s_carry;
  __shared__ int s_T[kPlanSmemSeqs], s_ctx[kPlanSmemSeqs], s_stp[kPlanSmemSeqs + 1];
  __shared__ long long s_cost[kPlanSmemSeqs + 1];
  allow_dependent_launch();        // the attention kernel may get its SMs now
  const int B = p.num_seqs, tid = threadIdx.x;
  const long long rows_bound = tree_rows_bound(p.ncta);
  const TreeLayout L = make_tree_layout(B, 0, rows_bound);
  int* q_off = reinterpret_cast<int*>(p.ws + L.q_off);
  int* cta_start = reinterpret_cast<int*>(p.ws + L.cta_start);
  // per-sequence arrays that the later passes read: the workspace's, kept in
  // shared memory as well for the usual batches
  int* g_T = reinterpret_cast<int*>(p.ws + L.seq_T);
  int* g_ctx = reinterpret_cast<int*>(p.ws + L.seq_ctx);
  int* g_stp = reinterpret_cast<int*>(p.ws + L.stp);
  long long* g_cost = reinterpret_cast<long long*>(p.ws + L.wcost);
  const bool small = B <= kPlanSmemSeqs;

  PlanSums run{0, 0, 0};
  for (int base = 0; base < B; base += kThreads) {
    const int b = base + tid;
    PlanSums mine{0, 0, 0};
    int T = 0, ctx = 0;
    if (b < B) {
      T = p.block_lens[b];
      ctx = p.context_lens[b];
      // rows lie at the sums of the caller's lengths, a rejected sequence's too
      mine.rows = T > 0 ? T : 0;
      if (T < 0 || ctx < 0 || T > p.max_block_len ||
          (long long)ctx + T > (long long)p.max_pages * kPageSize) {
        report(p.status, SPLASH_DEVICE_BAD_LENGTH);
        T = ctx = 0;
      }
      if (T > 0) {
        const RowBlocks rb = row_blocks(T, p.group);
        const int tiles = (ctx + T + kTile - 1) / kTile;
        const long long units = (long long)p.num_kv_heads * rb.count;
        mine.tiles = units * tiles;
        mine.cost = units * unit_cost(tiles, rb.rows);
      }
    }
    PlanSums tot;
    const PlanSums ex = exclusive_scan(mine, s_warp, &tot);
    if (b < B) {
      // past the caller's rows only where the plan is dropped below
      q_off[b] = (int)min(run.rows + ex.rows, (long long)p.num_q_tokens);
      const int stp = (int)min(run.tiles + ex.tiles, (long long)INT_MAX);
      g_T[b] = T;
      g_ctx[b] = ctx;
      g_stp[b] = stp;
      if (small) {
        s_T[b] = T;
        s_ctx[b] = ctx;
        s_stp[b] = stp;
        s_cost[b] = run.cost + ex.cost;
      } else {
        g_cost[b] = run.cost + ex.cost;
      }
    }
    run = run + tot;
  }
  __syncthreads();
  // rows past the caller's, or more tiles than the stream can count: do nothing
  const bool ok = run.rows <= p.num_q_tokens && run.tiles < INT_MAX;
  const int total = ok ? (int)run.tiles : 0;
  // at most one CTA per tile: every CTA owns tiles, and the CTAs of a unit are
  // consecutive
  const int n = min(min(p.ncta, total), kMaxCtas);
  if (tid == 0) {
    q_off[B] = (int)min(run.rows, (long long)p.num_q_tokens);
    g_stp[B] = total;
    if (!ok) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
    PlanHeader* hd = reinterpret_cast<PlanHeader*>(p.ws);
    hd->ncta[kClassTensor] = n;
    hd->total_tiles[kClassTensor] = total;
    hd->rows_bound = (int)rows_bound;
    s_carry = INT_MIN;
  }
  if (!ok)                         // no row is combined either
    for (int b = tid; b < B; b += kThreads) g_T[b] = 0;
  __syncthreads();
  const int* rT = small ? s_T : g_T;
  const int* rctx = small ? s_ctx : g_ctx;
  const int* rstp = small ? s_stp : g_stp;
  const long long* rcost = small ? s_cost : g_cost;

  // CTA k starts where the cumulative cost reaches k / n of the total: the
  // sequence, then the unit, then the tile (a unit's first segment_cost maps to
  // its first tile); then the starts are made strictly increasing, the last
  // ones pulled back so that every CTA has a tile
  for (int base = 0; n > 0 && base <= n; base += kThreads) {
    const int k = base + tid;
    int start = 0;
    if (k >= n) {
      start = total;
    } else if (k > 0) {
      const long long target = run.cost / n * k + run.cost % n * k / n;
      const int b = upper_index(rcost, B - 1, target);
      const RowBlocks rb = row_blocks(rT[b], p.group);
      const int tiles = (rctx[b] + rT[b] + kTile - 1) / kTile;
      const int units = p.num_kv_heads * rb.count;
      const long long uc = unit_cost(tiles, rb.rows), off = target - rcost[b];
      const int u = (int)min(off / uc, (long long)units - 1);
      const long long rem = off - u * uc - segment_cost(kClassTensor);
      const long long w = tile_cost(kClassTensor) + row_cost(kClassTensor) * rb.rows;
      const int t = rem < 0 ? 0 : (int)min(rem / w, (long long)tiles - 1);
      start = rstp[b] + u * tiles + t;
    }
    const int y = max(inclusive_max(k <= n ? start - k : INT_MIN, s_max), s_carry);
    if (k <= n) cta_start[k] = min(y + k, total - (n - k));
    __syncthreads();
    if (tid == kThreads - 1) s_carry = y;
    __syncthreads();
  }
}

// WPR warps per output row of a unit that CTAs share; warp `sub` of a row adds the
// partials j = sub, sub + WPR, .. and the sums meet in shared memory.
template <int D, int WPR>
__global__ void __launch_bounds__(256, 2)
tree_combine_kernel(int num_q_tokens, int num_q_heads, int num_seqs, int group,
                    const unsigned char* __restrict__ ws, __nv_bfloat16* __restrict__ out,
                    float* __restrict__ lse_out) {
  constexpr int kPer = D / 32;                    // output columns per lane
  constexpr int kRowsPerBlock = 8 / WPR;
  constexpr int kUnroll = WPR >= 4 ? 8 : 4;       // partial rows in flight per warp
  using Vec = float2;
  __shared__ float s_acc[WPR > 1 ? 8 : 1][WPR > 1 ? D : 1];
  grid_dependency_wait();          // the attention kernel's partials are complete
  const PlanHeader* hd = reinterpret_cast<const PlanHeader*>(ws);
  const TreeLayout L = make_tree_layout(num_seqs, D, hd->rows_bound);
  const int* q_off = reinterpret_cast<const int*>(ws + L.q_off);
  const int* seq_T = reinterpret_cast<const int*>(ws + L.seq_T);
  const int* seq_ctx = reinterpret_cast<const int*>(ws + L.seq_ctx);
  const int* stp = reinterpret_cast<const int*>(ws + L.stp);
  const int* cst = reinterpret_cast<const int*>(ws + L.cta_start);
  const float* o_part = reinterpret_cast<const float*>(ws + L.o_part);
  const float* lse_part = reinterpret_cast<const float*>(ws + L.lse_part);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const long long row = (long long)blockIdx.x * kRowsPerBlock + warp / WPR;
  const int ncta = hd->ncta[kClassTensor];
  bool active = row < (long long)num_q_tokens * num_q_heads && ncta > 0;
  int n = 0, cf = 0, r = 0;
  if (active) {
    const int i = (int)(row / num_q_heads), hq = (int)(row % num_q_heads);
    const int b = upper_index(q_off, num_seqs - 1, i);
    const int t = i - q_off[b], T = seq_T[b];
    active = t < T;
    if (active) {
      const RowBlocks rb = row_blocks(T, group);
      const int h = hq / group, j = t * group + hq % group, k = j / rb.rows;
      r = j - k * rb.rows;
      const int tiles = (seq_ctx[b] + T + kTile - 1) / kTile;
      const int first = stp[b] + (h * rb.count + k) * tiles;
      cf = upper_index(cst, ncta - 1, first);
      n = upper_index(cst, ncta - 1, first + tiles - 1) - cf + 1;
      active = n > 1;
    }
  }
  // partial j: the unit's first segment in its CTA's second place, the others in
  // their CTAs' first
  const auto place = [&](int j) {
    return (long long)(2 * (cf + j) + (j == 0 ? 1 : 0)) * kMaxRows + r;
  };
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  float m = -INFINITY, sum = 0.f;
  if (active) {
    for (int j = lane; j < n; j += 32) {
      const float lj = lse_part[place(j)];
      if (lj > m) {
        sum = sum * __expf(m - lj) + 1.f;        // m = -inf: the sum is 0 and stays finite
        m = lj;
      } else if (lj != -INFINITY) {
        sum += __expf(lj - m);
      }
    }
    const float mw = warp_max(m);
    sum = warp_sum(m == -INFINITY ? 0.f : sum * __expf(m - mw));
    m = mw;
    for (int j0 = sub; j0 < n; j0 += kUnroll * WPR) {
      float w[kUnroll];
      Vec v[kUnroll][kPer / 2];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int j = j0 + k * WPR;
        w[k] = 0.f;
        if (j < n) {
          const long long pr = place(j);
          const float lj = lse_part[pr];
          w[k] = lj == -INFINITY ? 0.f : __expf(lj - m);
          const Vec* src = reinterpret_cast<const Vec*>(o_part + pr * D) + lane;
#pragma unroll
          for (int e = 0; e < kPer / 2; ++e) v[k][e] = src[32 * e];
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (w[k] == 0.f) continue;
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) {
          acc[2 * e] = fmaf(w[k], v[k][e].x, acc[2 * e]);
          acc[2 * e + 1] = fmaf(w[k], v[k][e].y, acc[2 * e + 1]);
        }
      }
    }
  }
  if (WPR > 1) {
    if (active) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) s_acc[warp][32 * e + lane] = acc[e];
    }
    __syncthreads();
    if (active && sub == 0) {
#pragma unroll
      for (int o = 1; o < WPR; ++o)
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] += s_acc[warp + o][32 * e + lane];
    }
  }
  if (!active || sub != 0) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;           // a row that sees nothing: 0
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(out + row * D) + lane;
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e)
    dst[32 * e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0) lse_out[row] = sum > 0.f ? m + logf(sum) : -INFINITY;
}

cudaError_t launch_combine(int num_q_tokens, int num_q_heads, int num_seqs, int group, int D,
                           int sms, const unsigned char* ws, __nv_bfloat16* out, float* lse,
                           cudaStream_t s) {
  const long long rows = (long long)num_q_tokens * num_q_heads;
  // warps per row: about 16 an SM when there are few rows, as in the chain's combine
  const long long want = 16LL * sms;
  const int wpr = rows * 4 <= want ? 8 : rows * 2 <= want ? 4 : rows <= want ? 2 : 1;
  const dim3 grid((unsigned)((rows + 8 / wpr - 1) / (8 / wpr)));
#define SPLASH_TREE_COMBINE(DD, WW)                                                          \
  return launch_dependent(tree_combine_kernel<DD, WW>, grid, dim3(256), 0, s, num_q_tokens, \
                          num_q_heads, num_seqs, group, ws, out, lse)
#define SPLASH_TREE_COMBINE_D(DD)               \
  switch (wpr) {                                \
    case 1: SPLASH_TREE_COMBINE(DD, 1);         \
    case 2: SPLASH_TREE_COMBINE(DD, 2);         \
    case 4: SPLASH_TREE_COMBINE(DD, 4);         \
    default: SPLASH_TREE_COMBINE(DD, 8);        \
  }
  switch (D) {
    case 64: SPLASH_TREE_COMBINE_D(64)
    case 128: SPLASH_TREE_COMBINE_D(128)
    default: SPLASH_TREE_COMBINE_D(256)
  }
#undef SPLASH_TREE_COMBINE_D
#undef SPLASH_TREE_COMBINE
}

int check_shape(int num_seqs, int num_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                int max_block_len, int ctas) {
  if (num_seqs < 0 || num_q_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      max_block_len < 0 || ctas < 0 || ctas > kMaxCtas || num_q_heads % num_kv_heads != 0 ||
      (long long)num_q_tokens * num_q_heads > INT_MAX)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || max_block_len > kMaxTreeNodes ||
      num_q_heads > (1 << 20))
    return SPLASH_ERR_UNSUPPORTED;
  return SPLASH_OK;
}

// CTAs of the attention kernel: one an SM.
int default_ctas(int sms) { return sms < kMaxCtas ? sms : kMaxCtas; }

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" {

size_t splash_verify_attention_tree_workspace_size(int num_seqs, int num_q_tokens,
                                                   int num_q_heads, int num_kv_heads,
                                                   int head_dim, int max_block_len, int ctas) {
  if (check_shape(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim, max_block_len,
                  ctas) != SPLASH_OK)
    return 0;
  const int sms = device_sm_count();
  if (sms <= 0) return 0;
  return make_tree_layout(num_seqs, head_dim,
                          tree_rows_bound(ctas > 0 ? ctas : default_ctas(sms))).total;
}

int splash_verify_attention_tree(
    const uint16_t* q, int num_q_tokens, const int8_t* k_pages, const int8_t* v_pages,
    const float* k_scales, const float* v_scales, const int32_t* page_table,
    int max_pages_per_seq, const int32_t* context_lens, const int32_t* block_lens,
    const int32_t* tree_masks, int mask_stride, int num_seqs, int num_q_heads, int num_kv_heads,
    int head_dim, int page_size, int num_pages, int max_block_len, float sm_scale, uint16_t* out,
    float* lse, void* workspace, size_t workspace_bytes, int* device_status,
    struct CUstream_st* stream, int ctas) {
  const int st = check_shape(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_dim,
                             max_block_len, ctas);
  if (st != SPLASH_OK) return st;
  if (max_pages_per_seq <= 0 || max_pages_per_seq > INT_MAX / kPageSize || num_pages < 0 ||
      mask_stride < (max_block_len + 31) / 32)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (page_size != kPageSize || !tc_supported(head_dim == 64 ? 128 : head_dim))
    return SPLASH_ERR_UNSUPPORTED;
  if (num_q_tokens == 0 || num_seqs == 0 || max_block_len == 0) return SPLASH_OK;
  if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !page_table || !context_lens ||
      !block_lens || !tree_masks || !out || !lse || !workspace ||
      v_pages != k_pages + (size_t)page_size * head_dim || !aligned16(k_pages) ||
      !aligned16(k_scales) || !aligned16(v_scales) || !aligned16(q) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (!(sm_scale > 0.f) || sm_scale == INFINITY) return SPLASH_ERR_INVALID_ARGUMENT;
  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  const int ncta = ctas > 0 ? ctas : default_ctas(sms);
  if (workspace_bytes < make_tree_layout(num_seqs, head_dim, tree_rows_bound(ncta)).total)
    return SPLASH_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const int G = num_q_heads / num_kv_heads;
  const PlanParams pl{context_lens, block_lens, num_seqs, num_kv_heads, G, max_pages_per_seq,
                      max_block_len, ncta, num_q_tokens, ws, device_status};
  if (num_seqs <= kPlanSmall) tree_plan_kernel<kPlanSmall><<<1, kPlanSmall, 0, s>>>(pl);
  else tree_plan_kernel<kPlanLarge><<<1, kPlanLarge, 0, s>>>(pl);
  if (counted(cudaGetLastError()) != cudaSuccess) return SPLASH_ERR_CUDA;

  TreeAttnParams p;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.page_table = page_table;
  p.max_pages_per_seq = max_pages_per_seq;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = G;
  p.head_dim = head_dim;
  p.num_pages = num_pages;
  p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  p.window = 0;
  p.wait_ns = wait_limit_ns();
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ws = ws;
  p.device_status = device_status;
  p.tree_masks = tree_masks;
  p.mask_stride = mask_stride;
  if (counted(launch_verify_tree(p, ncta, s)) != cudaSuccess) return SPLASH_ERR_CUDA;
  return counted(launch_combine(num_q_tokens, num_q_heads, num_seqs, G, head_dim, sms, ws, p.out,
                                lse, s)) == cudaSuccess
             ? SPLASH_OK
             : SPLASH_ERR_CUDA;
}

}  // extern "C"
