// Accepted rows of a tree moved together in the cache: for i <= accepted[b], the
// slot of the block's row i receives the codes and scales of the slot of row
// path_rows[i], for every KV head and layer.
//
// Pure copy, 2 (2 D + 8) bytes a moved row, head and layer, in pieces of D and 4
// bytes that lie pages apart: latency of scattered sectors, so what counts is how
// many are in flight. A warp takes the rows of one (sequence, layer, head); a
// row's K and V codes are 2 D / 16 pieces of 16 bytes, so the warp moves 1, 2 or
// 4 rows at a time and has kBatch such loads in flight before it stores. 64 trees, 4
// heads of 256 in 48 layers: 23 us for 75 MB read and written, of which finding the
// slots takes 6, the reads 8 and the writes 8 (one after the other measured); the floor
// is 11. A thread a piece took 26 to 30, a CTA for all rows of a head 30 to 58, other
// batches and warps an SM 22.6 to 25.
//
// In place: path_rows[i] >= i (a node follows its ancestors), so no row at or
// before i is a source of a later one, and it is enough that a warp reads a batch
// of rows before it writes them, batches in order.
#include "splash_common.cuh"
#include "splash_host.cuh"
#include "splash_tree.cuh"

namespace splash {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 8;              // 16-byte loads of a lane in flight

struct CompactParams {
  int8_t* codes;
  float* k_scales;
  float* v_scales;
  const int32_t* slots;
  const int32_t* path_rows;
  const int32_t* q_offsets;
  const int32_t* accepted;
  int num_tokens, num_seqs, hkv, num_layers, num_pages;
  long long code_layer, scale_layer;   // elements between layers
  int* status;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 8) kv_compact_kernel(CompactParams p) {
  constexpr int kPieces = 2 * D / 16;            // of a row, K and V
  constexpr int kRows = 32 / kPieces;            // rows of one load of the warp
  const int lane = threadIdx.x & 31;
  const long long unit = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  if (unit >= (long long)p.num_seqs * p.num_layers * p.hkv) return;
  const int h = (int)(unit % p.hkv), bl = (int)(unit / p.hkv);
  const int l = bl % p.num_layers, b = bl / p.num_layers;
  const int first = p.q_offsets[b], end = p.q_offsets[b + 1];
  const bool usable = first >= 0 && first <= end && end <= p.num_tokens;
  int8_t* codes = p.codes + l * p.code_layer;
  float* ks = p.k_scales + l * p.scale_layer;
  float* vs = p.v_scales + l * p.scale_layer;
  const int sub = lane / kPieces, piece = lane % kPieces;
  // pieces of the K row, then of the V row, kPageSize rows further on
  const int off = (piece / (D / 16)) * kPageSize * D + (piece % (D / 16)) * 16;

  // a lane per row: where it comes from and goes to (read beside the count, not after it)
  int from = -1, dst = -1;
  if (usable && 1 + lane < end - first) {
    from = p.path_rows[first + 1 + lane];
    dst = p.slots[first + 1 + lane];
  }
  const int accepted = p.accepted[b];
  if (!usable || (accepted > 0 && accepted >= end - first)) {
    if (lane == 0) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
    return;
  }
  if (accepted <= 0) return;                     // the root is where it belongs
  const int count = accepted + 1;
  for (int base = 1; base < count; base += 32) {
    const int i = base + lane;
    if (base > 1 && i < count) {
      from = p.path_rows[first + i];
      dst = p.slots[first + i];
    }
    int src = -1;
    if (i < count) {
      if (from < first + i || from >= end) {
        report(p.status, SPLASH_DEVICE_BAD_TREE);
      } else if (from != first + i) {
        src = p.slots[from];
        if (src >= p.num_pages * kPageSize || dst >= p.num_pages * kPageSize) {
          report(p.status, SPLASH_DEVICE_BAD_PAGE);
          src = -1;
        }
        if (dst < 0) src = -1;
      }
    }
    const bool moved = src >= 0;
    float kscale = 0.f, vscale = 0.f;
    const size_t dscale = moved ? ((size_t)(dst / kPageSize) * p.hkv + h) * kPageSize + dst % kPageSize : 0;
    if (moved) {
      const size_t sscale = ((size_t)(src / kPageSize) * p.hkv + h) * kPageSize + src % kPageSize;
      kscale = ks[sscale];
      vscale = vs[sscale];
    }
    unsigned todo = __ballot_sync(0xffffffffu, moved);
    while (todo) {
      uint4 v[kBatch];
      int to[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        // the next kRows rows that move; this lane's is the sub-th of them
        int row = -1;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int at = __ffs(todo) - 1;
          if (r == sub) row = at;
          todo &= todo - 1;                      // 0 stays 0
        }
        const int s = __shfl_sync(0xffffffffu, src, row & 31);
        const int d = __shfl_sync(0xffffffffu, dst, row & 31);
        to[u] = row >= 0 ? d : -1;
        if (row >= 0)
          v[u] = *reinterpret_cast<const uint4*>(
              codes + code_offset(s / kPageSize, h, p.hkv, s % kPageSize, D) + off);
      }
      __syncwarp();                              // the batch is read: now it may be written
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (to[u] >= 0)
          *reinterpret_cast<uint4*>(
              codes + code_offset(to[u] / kPageSize, h, p.hkv, to[u] % kPageSize, D) + off) = v[u];
      __syncwarp();
    }
    if (moved) {
      ks[dscale] = kscale;
      vs[dscale] = vscale;
    }
    __syncwarp();
  }
}

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" int splash_kv_compact(int8_t* k_pages, int8_t* v_pages, float* k_scales,
                                 float* v_scales, long long code_layer_stride,
                                 long long scale_layer_stride, int num_layers,
                                 const int32_t* slots, const int32_t* path_rows, int num_tokens,
                                 const int32_t* q_offsets, const int32_t* accepted, int num_seqs,
                                 int num_kv_heads, int head_dim, int page_size, int num_pages,
                                 int* device_status, struct CUstream_st* stream) {
  if (num_tokens < 0 || num_seqs < 0 || num_kv_heads <= 0 || num_kv_heads > (1 << 20) ||
      num_layers < 0 || num_pages < 0 || num_pages > INT32_MAX / kPageSize)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (page_size != kPageSize || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return SPLASH_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_seqs == 0 || num_layers == 0) return SPLASH_OK;
  const long long pool = (long long)num_pages * num_kv_heads * 2 * kPageSize * head_dim;
  if (!k_pages || !v_pages || !k_scales || !v_scales || !slots || !path_rows || !q_offsets ||
      !accepted || v_pages != k_pages + (size_t)page_size * head_dim || !aligned16(k_pages) ||
      (num_layers > 1 && (code_layer_stride < pool || code_layer_stride % 16 != 0 ||
                          scale_layer_stride < pool / (2 * head_dim))))
    return SPLASH_ERR_INVALID_ARGUMENT;
  const long long units = (long long)num_seqs * num_layers * num_kv_heads;
  const long long grid = (units * 32 + kThreads - 1) / kThreads;
  if ((long long)num_seqs * num_layers > INT32_MAX || grid > INT32_MAX)
    return SPLASH_ERR_INVALID_ARGUMENT;
  const CompactParams p{k_pages, k_scales, v_scales, slots, path_rows, q_offsets, accepted,
                        num_tokens, num_seqs, num_kv_heads, num_layers, num_pages,
                        code_layer_stride, scale_layer_stride, device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (head_dim) {
    case 64: kv_compact_kernel<64><<<(int)grid, kThreads, 0, s>>>(p); break;
    case 128: kv_compact_kernel<128><<<(int)grid, kThreads, 0, s>>>(p); break;
    default: kv_compact_kernel<256><<<(int)grid, kThreads, 0, s>>>(p); break;
  }
  return counted(cudaGetLastError()) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}
