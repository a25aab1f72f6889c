// Cached rows back by slot: row i of k_out / v_out is the fp32 product code * scale
// of the K and V rows at slots[i], for every KV head, rounded to the output's type.
//
// Pure copy with a widening, bound by HBM: 2 (D + 4) bytes read and 2 D e
// written a (row, head). A lane takes one 16-byte piece of an output row (8 bf16
// or 4 fp32), so that the writes, two thirds of the bytes or more, are full
// sectors in order. What hides the latency is residency: every thread of the GPU
// with kUnroll pieces of K and V in flight. 131072 rows of 4 heads of 256, bf16
// (810 MB): 2 pieces and 8 CTAs to an SM 130 us, 92% of the measured copy rate (32
// registers a thread, of which the bf16 forms spill 36 bytes); 4 pieces at the 4 CTAs
// that their registers leave 145 us, 8 pieces 212 us.
#include "splash_common.cuh"
#include "splash_host.cuh"

namespace splash {

namespace {

constexpr int kGatherThreads = 256;
constexpr int kCtasPerSm = 8;        // resident: 32 registers a thread
constexpr int kUnroll = 2;

struct GatherParams {
  const int8_t* k_pages;
  const int8_t* v_pages;
  const float* k_scales;
  const float* v_scales;
  const int32_t* slots;
  int hkv;
  int num_pages;
  long long pieces;           // rows * hkv * (16-byte pieces of a head row)
  void* k_out;
  void* v_out;
  int* status;
};

__device__ inline uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

__device__ inline float code_at(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

__device__ inline uint4 widen(uint2 c, float s, __nv_bfloat16) {
  return make_uint4(bf16_pair(code_at(c.x, 0) * s, code_at(c.x, 1) * s),
                    bf16_pair(code_at(c.x, 2) * s, code_at(c.x, 3) * s),
                    bf16_pair(code_at(c.y, 0) * s, code_at(c.y, 1) * s),
                    bf16_pair(code_at(c.y, 2) * s, code_at(c.y, 3) * s));
}
__device__ inline uint4 widen(uint32_t c, float s, float) {
  return make_uint4(__float_as_uint(code_at(c, 0) * s), __float_as_uint(code_at(c, 1) * s),
                    __float_as_uint(code_at(c, 2) * s), __float_as_uint(code_at(c, 3) * s));
}

template <typename TOut>
struct CodeVec;
template <>
struct CodeVec<__nv_bfloat16> { using type = uint2; };
template <>
struct CodeVec<float> { using type = uint32_t; };

template <int D, typename TOut>
__global__ void __launch_bounds__(kGatherThreads, kCtasPerSm) kv_gather_kernel(GatherParams p) {
  using Codes = typename CodeVec<TOut>::type;
  constexpr int kPer = 16 / sizeof(TOut);        // values of a piece
  constexpr int kPieces = D / kPer;              // pieces of a head row
  const long long step = (long long)gridDim.x * kGatherThreads;
  for (long long i0 = (long long)blockIdx.x * kGatherThreads + threadIdx.x; i0 < p.pieces;
       i0 += kUnroll * step) {
    Codes kc[kUnroll], vc[kUnroll];
    float ks[kUnroll], vs[kUnroll];
    bool live[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long i = i0 + u * step;
      live[u] = false;
      if (i >= p.pieces) continue;
      const long long pair = i / kPieces;
      const int col = (int)(i % kPieces) * kPer;
      const int row = (int)(pair / p.hkv), h = (int)(pair % p.hkv);
      const int slot = p.slots[row];
      const int page = slot / kPageSize, at = slot % kPageSize;
      if (slot < 0) continue;                    // a padded row is left as it is
      if (page >= p.num_pages) {
        report(p.status, SPLASH_DEVICE_BAD_PAGE);
        continue;
      }
      live[u] = true;
      const size_t code = code_offset(page, h, p.hkv, at, D) + col;
      const size_t sc = ((size_t)page * p.hkv + h) * kPageSize + at;
      kc[u] = *reinterpret_cast<const Codes*>(p.k_pages + code);
      vc[u] = *reinterpret_cast<const Codes*>(p.v_pages + code);
      ks[u] = p.k_scales[sc];
      vs[u] = p.v_scales[sc];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!live[u]) continue;
      const long long i = i0 + u * step;
      reinterpret_cast<uint4*>(p.k_out)[i] = widen(kc[u], ks[u], TOut{});
      reinterpret_cast<uint4*>(p.v_out)[i] = widen(vc[u], vs[u], TOut{});
    }
  }
}

template <int D>
cudaError_t launch_gather(const GatherParams& p, int dtype, int grid, cudaStream_t s) {
  if (dtype == SPLASH_F32) kv_gather_kernel<D, float><<<grid, kGatherThreads, 0, s>>>(p);
  else kv_gather_kernel<D, __nv_bfloat16><<<grid, kGatherThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" int splash_kv_gather(const int8_t* k_pages, const int8_t* v_pages,
                                const float* k_scales, const float* v_scales, const int32_t* slots,
                                int num_rows, int num_kv_heads, int head_dim, int page_size,
                                int num_pages, void* k_out, void* v_out, int dtype,
                                int* device_status, struct CUstream_st* stream) {
  if (num_rows < 0 || num_kv_heads <= 0 || num_kv_heads > (1 << 20) || num_pages < 0)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (page_size != kPageSize || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (dtype != SPLASH_F32 && dtype != SPLASH_BF16))
    return SPLASH_ERR_UNSUPPORTED;
  if (num_rows == 0) return SPLASH_OK;
  if (!k_pages || !v_pages || !k_scales || !v_scales || !slots || !k_out || !v_out ||
      v_pages != k_pages + (size_t)page_size * head_dim || !aligned16(k_pages) ||
      !aligned16(k_out) || !aligned16(v_out))
    return SPLASH_ERR_INVALID_ARGUMENT;
  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  const int per = dtype == SPLASH_F32 ? 4 : 8;
  GatherParams p{k_pages, v_pages, k_scales, v_scales, slots, num_kv_heads, num_pages,
                 (long long)num_rows * num_kv_heads * (head_dim / per), k_out, v_out,
                 device_status};
  const long long want = (p.pieces + kGatherThreads - 1) / kGatherThreads;
  const long long most = (long long)kCtasPerSm * sms;
  const int grid = (int)(want < most ? want : most);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (head_dim) {
    case 64: e = launch_gather<64>(p, dtype, grid, s); break;
    case 128: e = launch_gather<128>(p, dtype, grid, s); break;
    default: e = launch_gather<256>(p, dtype, grid, s); break;
  }
  return counted(e) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}
