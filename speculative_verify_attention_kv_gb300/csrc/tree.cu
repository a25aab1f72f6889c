// Trees of drafts, apart from the attention: ancestor masks, depths and positions
// from the nodes' parents, and the path through the tree that the target accepts.
//
// A tree of T nodes is an array of parents: node 0 holds the token that the target
// produced at the step before, parent[t] < t is the node that node t continues, -1
// has none. Both kernels are chains of dependent steps on a few hundred bytes a
// tree: latency, not bytes, and so a tree stays in one CTA or one warp. In a replayed
// graph (an empty kernel takes 2 us of it) 16 trees of 16 nodes take 4.1 us for the masks
// and 4.4 for the path, 500 trees of up to 120 nodes 6.2 and 6.2; their bytes would be
// read and written in 0.001 to 0.12 us.
#include "splash_common.cuh"
#include "splash_host.cuh"
#include "splash_tree.cuh"

namespace splash {
namespace {

// Rows of a sequence from its offsets: false (and reported) where they are unusable.
__device__ inline bool tree_rows(const int32_t* __restrict__ q_offsets, int b, int num_tokens,
                                 int max_block_len, int* status, int& first, int& T) {
  first = q_offsets[b];
  const int end = q_offsets[b + 1];
  const bool ok = first >= 0 && end >= first && end <= num_tokens && end - first <= max_block_len;
  T = ok ? end - first : 0;
  if (!ok && (threadIdx.x & 31) == 0) report(status, SPLASH_DEVICE_BAD_LENGTH);
  return ok;
}

struct MasksParams {
  const int32_t* parents;
  const int32_t* q_offsets;
  const int32_t* context_lens;     // NULL: no positions
  int num_seqs, num_tokens, max_block_len;
  int32_t* masks;
  int mask_stride;
  int32_t* depths;                 // NULL: not written
  int32_t* positions;
  int* status;
};

// A CTA per tree, a thread per node. With up(t) the first ancestor that node t's
// mask does not cover yet, mask(t) |= mask(up(t)) doubles what a mask covers, so a
// tree of depth d is done after log2(d + 1) rounds (a walk up the parents would take
// d dependent reads). kWords: words of a mask.
template <int kWords>
__global__ void __launch_bounds__(kMaxTreeNodes) tree_masks_kernel(MasksParams p) {
  __shared__ uint32_t s_mask[kWords][kMaxTreeNodes];
  __shared__ int s_up[kMaxTreeNodes], s_covers[kMaxTreeNodes];
  const int b = blockIdx.x, t = threadIdx.x;
  int first, T;
  tree_rows(p.q_offsets, b, p.num_tokens, p.max_block_len, p.status, first, T);
  const bool live = t < T;
  int up = live ? p.parents[first + t] : -1;
  if (up < -1 || up >= t) {                    // its own root then
    if (live) report(p.status, SPLASH_DEVICE_BAD_TREE);
    up = -1;
  }
  int covers = 1;                              // nodes in the mask
  uint32_t m[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) m[w] = w == t >> 5 ? 1u << (t & 31) : 0u;
  while (true) {
    if (!__syncthreads_or(up >= 0)) break;     // and the round before has been read
#pragma unroll
    for (int w = 0; w < kWords; ++w) s_mask[w][t] = m[w];
    s_up[t] = up;
    s_covers[t] = covers;
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) m[w] |= s_mask[w][up];
      covers += s_covers[up];
      up = s_up[up];
    }
  }
  if (!live) return;
  const int row = first + t;
  int32_t* dst = p.masks + (size_t)row * p.mask_stride;
#pragma unroll
  for (int w = 0; w < kWords; ++w)
    if (w * 32 < p.max_block_len) dst[w] = (int32_t)m[w];
  if (p.depths) p.depths[row] = covers - 1;
  if (p.positions) p.positions[row] = p.context_lens[b] + covers - 1;
}

struct AcceptParams {
  const int32_t* block_tokens;
  const int32_t* parents;
  const int32_t* target_tokens;
  const int32_t* q_offsets;
  const int32_t* context_lens;
  int32_t* context_lens_out;
  int32_t* accepted;
  int32_t* next_tokens;
  int32_t* path_rows;
  int32_t* path_tokens;            // NULL: not written
  int num_seqs, num_tokens, max_block_len;
  int* status;
};

constexpr int kAcceptWarps = 4;

// A warp per tree: its nodes' parents and tokens in registers (node 32 i + lane), the
// targets and tokens by node in shared memory. A step finds the first child of the
// current node that holds the target's choice by a ballot per 32 nodes, from the
// current node's 32 on, since children follow their parents. kPer: nodes a lane.
template <int kPer>
__global__ void __launch_bounds__(32 * kAcceptWarps) accept_tree_kernel(AcceptParams p) {
  __shared__ int s_target[kAcceptWarps][32 * kPer], s_token[kAcceptWarps][32 * kPer];
  __shared__ int s_path[kAcceptWarps][32 * kPer];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x * kAcceptWarps + warp;
  if (b >= p.num_seqs) return;
  int first, T;
  tree_rows(p.q_offsets, b, p.num_tokens, p.max_block_len, p.status, first, T);
  const int ctx = p.context_lens[b];
  int parent[kPer], token[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int t = 32 * i + lane;
    parent[i] = token[i] = -1;
    if (t < T) {
      parent[i] = p.parents[first + t];
      token[i] = p.block_tokens[first + t];
      s_target[warp][t] = p.target_tokens[first + t];
      s_token[warp][t] = token[i];
      if (parent[i] < -1 || parent[i] >= t) {          // never accepted
        report(p.status, SPLASH_DEVICE_BAD_TREE);
        parent[i] = -1;
      }
      if (token[i] < 0) parent[i] = -1;                // nor a node without a token
    }
  }
  __syncwarp();
  int count = 0, last = -1;
  if (T > 0) {
    int cur = 0;
    while (cur >= 0) {
      if (lane == 0) s_path[warp][count] = cur;
      ++count;
      last = s_target[warp][cur];
      int next = -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (next >= 0 || 32 * i + 31 <= cur) continue;  // the same in every lane
        const unsigned hit = __ballot_sync(0xffffffffu, parent[i] == cur && token[i] == last);
        if (hit) next = 32 * i + __ffs(hit) - 1;
      }
      cur = next;
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int t = 32 * i + lane;
    if (t >= T) continue;
    const int node = t < count ? s_path[warp][t] : -1;
    p.path_rows[first + t] = node >= 0 ? first + node : -1;
    if (p.path_tokens) p.path_tokens[first + t] = node >= 0 ? s_token[warp][node] : -1;
  }
  if (lane == 0) {
    p.accepted[b] = T > 0 ? count - 1 : 0;
    p.next_tokens[b] = last;
    p.context_lens_out[b] = ctx + count;
  }
}

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" {

int splash_tree_masks(const int32_t* parents, int num_tokens, const int32_t* q_offsets,
                      const int32_t* context_lens, int num_seqs, int max_block_len,
                      int32_t* masks, int mask_stride, int32_t* depths, int32_t* positions,
                      int* device_status, struct CUstream_st* stream) {
  if (num_tokens < 0 || num_seqs < 0 || max_block_len < 0 ||
      mask_stride < (max_block_len + 31) / 32)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (max_block_len > kMaxTreeNodes) return SPLASH_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_seqs == 0 || max_block_len == 0) return SPLASH_OK;
  if (!parents || !q_offsets || !masks || (positions && !context_lens))
    return SPLASH_ERR_INVALID_ARGUMENT;
  const MasksParams p{parents, q_offsets, context_lens, num_seqs, num_tokens, max_block_len,
                      masks, mask_stride, depths, positions, device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int words = (max_block_len + 31) / 32, threads = 32 * words;
  if (words == 1) tree_masks_kernel<1><<<num_seqs, threads, 0, s>>>(p);
  else if (words == 2) tree_masks_kernel<2><<<num_seqs, threads, 0, s>>>(p);
  else if (words <= 4) tree_masks_kernel<4><<<num_seqs, threads, 0, s>>>(p);
  else tree_masks_kernel<8><<<num_seqs, threads, 0, s>>>(p);
  return counted(cudaGetLastError()) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}

int splash_accept_tree(const int32_t* block_tokens, const int32_t* parents,
                       const int32_t* target_tokens, int num_tokens, const int32_t* q_offsets,
                       const int32_t* context_lens, int32_t* context_lens_out, int32_t* accepted,
                       int32_t* next_tokens, int32_t* path_rows, int32_t* path_tokens,
                       int num_seqs, int max_block_len, int* device_status,
                       struct CUstream_st* stream) {
  if (num_tokens < 0 || num_seqs < 0 || max_block_len < 0) return SPLASH_ERR_INVALID_ARGUMENT;
  if (max_block_len > kMaxTreeNodes) return SPLASH_ERR_UNSUPPORTED;
  if (num_seqs == 0) return SPLASH_OK;
  if (!q_offsets || !context_lens || !context_lens_out || !accepted || !next_tokens ||
      (num_tokens > 0 && (!block_tokens || !parents || !target_tokens || !path_rows)))
    return SPLASH_ERR_INVALID_ARGUMENT;
  const AcceptParams p{block_tokens, parents, target_tokens, q_offsets, context_lens,
                       context_lens_out, accepted, next_tokens, path_rows, path_tokens, num_seqs,
                       num_tokens, max_block_len, device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = (num_seqs + kAcceptWarps - 1) / kAcceptWarps, threads = 32 * kAcceptWarps;
  if (max_block_len <= 32) accept_tree_kernel<1><<<grid, threads, 0, s>>>(p);
  else if (max_block_len <= 64) accept_tree_kernel<2><<<grid, threads, 0, s>>>(p);
  else if (max_block_len <= 128) accept_tree_kernel<4><<<grid, threads, 0, s>>>(p);
  else accept_tree_kernel<8><<<grid, threads, 0, s>>>(p);
  return counted(cudaGetLastError()) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}

}  // extern "C"
