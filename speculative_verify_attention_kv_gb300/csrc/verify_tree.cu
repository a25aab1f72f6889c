// Attention over a tree of drafts: plan of large batches, log-sum-exp combine and C
// entry. The attention itself is verify_tc.cu's kernel with tree masks.
//
// Work unit = (sequence b, KV head h, row block k): up to kMaxRows of the T_b * G
// query rows against keys 0 .. ctx_b + T_b - 1. As in the plan of a chain, the
// 64-key tiles of all units form one stream, cut over the persistent CTAs into
// ranges of about equal estimated cost. A unit inside one CTA's range is finished
// there; otherwise every CTA that shares it leaves a partial (o_i normalised by its
// own sum, lse_i) in one of its two places (splash_tree.cuh), and the combine
// merges them:
//   lse = ln sum_i exp(lse_i),  O = sum_i exp(lse_i - lse) o_i
// (__expf of differences x <= 0 is off by (2 + 1.2 |x|) 2^-23 of a weight e^x: 2^-21 at most
// of the sum, below the partials' own errors)
// A row that sees nothing (an empty mask and no context) has lse = -inf and O = 0,
// whole or in parts. The combine goes by the list of shared units, of which there are
// fewer than CTAs: looking up every output row's unit in the plan instead made it 25
// us of a 218 us call (32 ragged sequences, 1,000 nodes, 24 heads of 256), this way it
// is 12 of 154. What is left of it is the launch and three loads one after the other
// (list, lse, rows) before the sums.
#include <climits>

#include "splash_common.cuh"
#include "splash_host.cuh"
#include "splash_tree.cuh"

namespace splash {

cudaError_t launch_verify_tree(const TreeAttnParams&, int, bool, cudaStream_t);
bool tc_supported(int head_dim);

namespace {

constexpr int kPlanThreads = 1024;

// The plan of a batch that is too large for the attention kernel's own.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(TreeAttnParams p, int ncta) {
  __shared__ PlanSums s_sums[32];
  __shared__ int s_max[32], s_start[kMaxCtas + 1], s_carry;
  allow_dependent_launch();        // the attention kernel may get its SMs now
  const TreeLayout L = make_tree_layout(p.num_seqs, p.head_dim, tree_rows_bound(ncta));
  const PlanArrays a{reinterpret_cast<long long*>(p.ws + L.cost),
                     reinterpret_cast<int*>(p.ws + L.stp), reinterpret_cast<int*>(p.ws + L.q_off),
                     s_start, s_sums, s_max, &s_carry};
  const int n = plan_tree(p, a, ncta, true);
  TreeStart* starts = reinterpret_cast<TreeStart*>(p.ws + L.starts);
  for (int k = threadIdx.x; k < n; k += kPlanThreads) starts[k] = start_of(a, p.num_seqs, k);
  note_splits(p, a, n, reinterpret_cast<TreeHeader*>(p.ws),
              reinterpret_cast<TreeSplit*>(p.ws + L.splits));
}

// A block per kRowsPerBlock rows of a shared unit, WPR warps a row; warp `sub` of a row
// adds the partials j = sub, sub + WPR, .. and the sums meet in shared memory.
template <int D, int WPR>
__global__ void __launch_bounds__(256, 2)
tree_combine_kernel(int num_q_heads, int num_seqs, int group, int ncta, int chunks,
                    const unsigned char* __restrict__ ws, __nv_bfloat16* __restrict__ out,
                    float* __restrict__ lse_out) {
  constexpr int kPer = D / 32;                    // output columns per lane
  constexpr int kRowsPerBlock = 8 / WPR;
  constexpr int kUnroll = WPR >= 4 ? 8 : 4;       // partial rows in flight per warp
  using Vec = float2;
  __shared__ float s_acc[WPR > 1 ? 8 : 1][WPR > 1 ? D : 1];
  grid_dependency_wait();          // the attention kernel's partials are complete
  const TreeLayout L = make_tree_layout(num_seqs, D, tree_rows_bound(ncta));
  const float* o_part = reinterpret_cast<const float*>(ws + L.o_part);
  const float* lse_part = reinterpret_cast<const float*>(ws + L.lse_part);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % WPR;
  const int unit = blockIdx.x / chunks;
  const int r = (blockIdx.x - unit * chunks) * kRowsPerBlock + warp / WPR;
  if (unit >= reinterpret_cast<const TreeHeader*>(ws)->num_splits) return;
  const TreeSplit sp = reinterpret_cast<const TreeSplit*>(ws + L.splits)[unit];
  const bool active = r < sp.rows;
  const int n = sp.parts;
  // partial j: the unit's first segment in its CTA's second place, the others in
  // their CTAs' first
  const auto place = [&](int j) {
    return (long long)(2 * (sp.cta + j) + (j == 0 ? 1 : 0)) * kMaxRows + r;
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
  const int j = sp.r0 + r, t = j / group;
  const long long row = (long long)(sp.q_off + t) * num_q_heads + sp.h * group + (j - t * group);
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(out + row * D) + lane;
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e)
    dst[32 * e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0) lse_out[row] = sum > 0.f ? m + logf(sum) : -INFINITY;
}

// The units that CTAs may share (fewer than CTAs, and than units) have at most
// kMaxRows rows each.
cudaError_t launch_combine(int num_q_heads, int num_seqs, int num_kv_heads, int max_block_len,
                           int D, int ncta, int sms, const unsigned char* ws, __nv_bfloat16* out,
                           float* lse, cudaStream_t s) {
  const int group = num_q_heads / num_kv_heads;
  const RowBlocks rb = row_blocks(max_block_len, group);
  const long long units = (long long)num_seqs * num_kv_heads * rb.count;
  const int shared = (int)(units < ncta - 1 ? units : ncta - 1);
  const int rows_max = rb.count > 1 ? kMaxRows : rb.rows;
  // warps per row: about 16 an SM when there are few rows, as in the chain's combine
  const long long rows = (long long)shared * rows_max, want = 16LL * sms;
  const int wpr = rows * 4 <= want ? 8 : rows * 2 <= want ? 4 : rows <= want ? 2 : 1;
  const int chunks = (rows_max + 8 / wpr - 1) / (8 / wpr);
  const dim3 grid((unsigned)(shared * chunks));
#define SPLASH_TREE_COMBINE(DD, WW)                                                          \
  return launch_dependent(tree_combine_kernel<DD, WW>, grid, dim3(256), 0, s, num_q_heads,  \
                          num_seqs, group, ncta, chunks, ws, out, lse)
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
  p.context_lens = context_lens;
  p.block_lens = block_lens;
  p.max_block_len = max_block_len;
  p.num_q_tokens = num_q_tokens;
  p.row_cost = tree_row_cost(head_dim);
  p.segment_cost = tree_segment_cost(head_dim);
  const bool planned = num_seqs > kTreeSelfPlan;
  if (planned) {
    tree_plan_kernel<<<1, kPlanThreads, 0, s>>>(p, ncta);
    if (counted(cudaGetLastError()) != cudaSuccess) return SPLASH_ERR_CUDA;
  }
  if (counted(launch_verify_tree(p, ncta, planned, s)) != cudaSuccess) return SPLASH_ERR_CUDA;
  if (ncta == 1) return SPLASH_OK;               // nothing is shared
  return counted(launch_combine(num_q_heads, num_seqs, num_kv_heads, max_block_len, head_dim,
                                ncta, sms, ws, p.out, lse, s)) == cudaSuccess
             ? SPLASH_OK
             : SPLASH_ERR_CUDA;
}

}  // extern "C"
