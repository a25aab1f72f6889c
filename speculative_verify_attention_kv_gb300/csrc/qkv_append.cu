// Per-head norm and rotation of q and k and the quantised append of k and v,
// in one pass over the projections of the new tokens.
//
// For a row x of D values (one token, one head):
//   q, k : y = x * w / sqrt(mean(x^2) + eps)        (w given; else y = x)
//   q, k : the first R = rotary_dim values of y are turned in pairs (u, v),
//          (y_i, y_{i+R/2}) or, interleaved, (y_2i, y_2i+1), by the angle
//          pos[axis_i] * inv_freq_i:  u' = (u cos - v sin) m, v' = (v cos + u sin) m
//   q    : rounded once to bf16
//   k, v : s = fl32(max|y| / 127), codes clamp(rne(fl32(y / s)), +-127) into the
//          page of the token's slot (splash_quant.cuh)
// Everything before the one rounding is fp32.
//
// The angle is taken modulo one turn in 64-bit fixed point: inv_freq_i / 2 pi is
// held as F_i / 2^64 turns (its 24-bit significand times a 96-bit 1 / 2 pi,
// shifted), and position * F_i wraps by itself. The error is below position *
// 2^-63 turns, so far positions keep the accuracy of near ones, at the cost of
// an integer product (fp64, the other way to it, runs at 2 FMA a clock and SM
// here). sincospif then needs no range reduction.
//
// A warp takes one token and a run of its heads, 8 values a lane (so a head of
// D values takes D/8 lanes, and a warp 256/D heads at once). A lane's column is
// the same for every head, so the token's 8 cosines and sines, the norm weights
// and the frequencies stay in registers, and there is neither shared memory nor
// a barrier. Loads of kBatch head rows are in flight while the angles are
// computed. Few tokens are split over more warps by heads (rows_per_item).
#include <cmath>

#include "splash_common.cuh"
#include "splash_host.cuh"
#include "splash_quant.cuh"

namespace splash {

namespace {

constexpr int kQkvWarps = 4;
constexpr int kQkvThreads = 32 * kQkvWarps;
constexpr int kEpl = 8;          // values a lane holds of a head row
constexpr int kBatch = 4;        // head rows in flight per lane

struct QkvParams {
  const void* q;
  const void* k;
  const void* v;
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head;   // strides in values
  int n;
  int hq, hkv;
  const float* q_weight;
  const float* k_weight;
  float eps;
  const float* inv_freq;
  const int32_t* freq_axis;
  int half;                      // rotary_dim / 2
  const int32_t* positions;      // [axes, n]
  int axes;
  float rope_scale;
  const int32_t* slots;
  __nv_bfloat16* q_out;
  int8_t* k_pages;
  int8_t* v_pages;
  float* k_scales;
  float* v_scales;
  int num_pages;
  int groups_per_item;           // warp-wide row groups an item handles
  int items_per_token;
  int* status;
};

// Raw 8 values of a row: 16 bytes of bf16, 32 of fp32.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&x)[kEpl]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ void get(float (&x)[kEpl]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

// f / (2 pi) turns as a 64-bit fraction of a turn (whole turns drop out).
__device__ inline unsigned long long turns64(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = (bits >> 23) & 255;
  const unsigned long long m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int shift = 32 - ((ex ? ex : 1) - 150);      // P / 2^shift, below
  // P = m * floor(2^96 / (2 pi)), 120 bits
  const unsigned long long lo = m * 0x7f09d5f4ull, mid = m * 0x9391054aull, top = m * 0x28be60dbull;
  const unsigned long long t1 = (lo >> 32) + (mid & 0xffffffffull);
  const unsigned long long plo = (t1 << 32) | (lo & 0xffffffffull);
  const unsigned long long phi = (t1 >> 32) + (mid >> 32) + top;
  unsigned long long r;
  if (shift >= 128) r = 0;
  else if (shift >= 64) r = phi >> (shift - 64);
  else if (shift > 0) r = (phi << (64 - shift)) | (plo >> shift);
  else r = shift > -64 ? plo << -shift : 0;
  return bits >> 31 ? 0ull - r : r;
}

template <int D, typename TIn>
__global__ void __launch_bounds__(kQkvThreads) qkv_append_kernel(QkvParams p) {
  constexpr int kLanes = D / kEpl;               // lanes of a head row
  constexpr int kRows = 32 / kLanes;             // head rows of a warp-wide group
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kQkvWarps + (threadIdx.x >> 5);
  const int tok = (int)(item / p.items_per_token);
  if (tok >= p.n) return;
  const int part = (int)(item % p.items_per_token);
  const int slot = p.slots[tok];
  if (slot < 0) return;                          // a padded row: nothing is written
  const int page = slot / kPageSize;
  if (page >= p.num_pages) {
    if (lane == 0) report(p.status, SPLASH_DEVICE_BAD_PAGE);
    return;
  }
  const int col = (lane % kLanes) * kEpl;
  const int rows = p.hq + 2 * p.hkv;
  const int g0 = part * p.groups_per_item;
  const int g1 = min(g0 + p.groups_per_item, (rows + kRows - 1) / kRows);

  auto load = [&](Raw<TIn>& raw, int r) {
    if (r >= rows) {
      raw.zero();
    } else if (r < p.hq) {
      raw.load(static_cast<const TIn*>(p.q) + tok * p.q_tok + r * p.q_head + col);
    } else if (r < p.hq + p.hkv) {
      raw.load(static_cast<const TIn*>(p.k) + tok * p.k_tok + (r - p.hq) * p.k_head + col);
    } else {
      raw.load(static_cast<const TIn*>(p.v) + tok * p.v_tok + (r - p.hq - p.hkv) * p.v_head + col);
    }
  };

  Raw<TIn> raw[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u)
    if (g0 + u < g1) load(raw[u], (g0 + u) * kRows + lane / kLanes);

  // This lane's columns of the rotation: x' = x * cs + partner * sn.
  const bool paired = p.half < 0;
  const int half = paired ? -p.half : p.half;
  const bool turns = col < 2 * half;
  float cs[kEpl], sn[kEpl];
  if (turns) {
    const int f0 = paired ? col / 2 : (col < half ? col : col - half);
    const int nf = paired ? kEpl / 2 : kEpl;
    const int pos0 = p.positions[tok];
#pragma unroll
    for (int i = 0; i < kEpl; ++i) {
      if (i < nf) {
        int pos = pos0;
        if (p.freq_axis) {
          const int a = max(0, min(p.freq_axis[f0 + i], p.axes - 1));
          pos = p.positions[(size_t)a * p.n + tok];
        }
        const unsigned long long ph = (unsigned long long)(long long)pos * turns64(p.inv_freq[f0 + i]);
        // signed 32-bit fraction of a turn -> half turns in [-1, 1)
        const float x = (float)(int)(ph >> 32) * 4.656612873077393e-10f;
        float s, c;
        sincospif(x, &s, &c);
        cs[i] = c * p.rope_scale;
        sn[i] = s * p.rope_scale;
      }
    }
    if (paired) {
#pragma unroll
      for (int i = kEpl / 2 - 1; i >= 0; --i) {
        cs[2 * i + 1] = cs[2 * i] = cs[i];
        sn[2 * i + 1] = sn[i];
        sn[2 * i] = -sn[2 * i + 1];
      }
    } else if (col < half) {
#pragma unroll
      for (int i = 0; i < kEpl; ++i) sn[i] = -sn[i];
    }
  }
  const int from = paired || !turns ? lane : (col < half ? lane + half / kEpl : lane - half / kEpl);
  float qw[kEpl], kw[kEpl];
  if (p.q_weight) {
#pragma unroll
    for (int i = 0; i < kEpl; ++i) qw[i] = p.q_weight[col + i];
  }
  if (p.k_weight) {
#pragma unroll
    for (int i = 0; i < kEpl; ++i) kw[i] = p.k_weight[col + i];
  }

  for (int g = g0; g < g1; g += kBatch) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (g + u >= g1) break;
      const int r = (g + u) * kRows + lane / kLanes;
      const bool is_q = r < p.hq, is_k = !is_q && r < p.hq + p.hkv, live = r < rows;
      float x[kEpl];
      raw[u].get(x);
      if (g + u + kBatch < g1) load(raw[u], r + kBatch * kRows);
      if (p.q_weight || p.k_weight) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kEpl; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rn = rsqrtf(ss * (1.f / D) + p.eps);
        if (is_q && p.q_weight) {
#pragma unroll
          for (int i = 0; i < kEpl; ++i) x[i] = x[i] * rn * qw[i];
        } else if (is_k && p.k_weight) {
#pragma unroll
          for (int i = 0; i < kEpl; ++i) x[i] = x[i] * rn * kw[i];
        }
      }
      if (half > 0) {
        float y[kEpl];
        if (paired) {
#pragma unroll
          for (int i = 0; i < kEpl; ++i) y[i] = x[i ^ 1];
        } else {
#pragma unroll
          for (int i = 0; i < kEpl; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
        }
        if (turns && (is_q || is_k)) {
#pragma unroll
          for (int i = 0; i < kEpl; ++i) x[i] = fmaf(y[i], sn[i], x[i] * cs[i]);
        }
      }
      if (__any_sync(0xffffffffu, live && !is_q)) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < kEpl; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (live && !is_q) {
          const int h = is_k ? r - p.hq : r - p.hq - p.hkv;
          const int at = slot % kPageSize;
          int8_t* codes = (is_k ? p.k_pages : p.v_pages) + code_offset(page, h, p.hkv, at, D) + col;
          float* scale = (is_k ? p.k_scales : p.v_scales) + ((size_t)page * p.hkv + h) * kPageSize + at;
          store_codes<kEpl>(x, a, codes, scale, col == 0);
        }
      }
      if (is_q) {
        uint4 w;
        __nv_bfloat162 t;
        t = __floats2bfloat162_rn(x[0], x[1]); w.x = *reinterpret_cast<uint32_t*>(&t);
        t = __floats2bfloat162_rn(x[2], x[3]); w.y = *reinterpret_cast<uint32_t*>(&t);
        t = __floats2bfloat162_rn(x[4], x[5]); w.z = *reinterpret_cast<uint32_t*>(&t);
        t = __floats2bfloat162_rn(x[6], x[7]); w.w = *reinterpret_cast<uint32_t*>(&t);
        *reinterpret_cast<uint4*>(p.q_out + ((size_t)tok * p.hq + r) * D + col) = w;
      }
    }
  }
}

template <int D>
cudaError_t launch_qkv(const QkvParams& p, int dtype, unsigned grid, cudaStream_t s) {
  if (dtype == SPLASH_F32) qkv_append_kernel<D, float><<<grid, kQkvThreads, 0, s>>>(p);
  else qkv_append_kernel<D, __nv_bfloat16><<<grid, kQkvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" int splash_qkv_append(
    const void* q, const void* k, const void* v, int dtype, int num_tokens, long long q_stride,
    long long q_head_stride, long long k_stride, long long k_head_stride, long long v_stride,
    long long v_head_stride, int num_q_heads, int num_kv_heads, int head_dim, const float* q_weight,
    const float* k_weight, float eps, const float* inv_freq, const int32_t* freq_axis,
    int rotary_dim, int interleaved, float rope_scale, const int32_t* positions, int num_axes,
    const int32_t* slots, uint16_t* q_out, int8_t* k_pages, int8_t* v_pages, float* k_scales,
    float* v_scales, int page_size, int num_pages, int* device_status,
    struct CUstream_st* stream) {
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_pages < 0 ||
      num_q_heads > (1 << 20) || num_kv_heads > (1 << 20) || rotary_dim < 0 ||
      !(eps >= 0.f) || eps == INFINITY)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (page_size != kPageSize || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (dtype != SPLASH_F32 && dtype != SPLASH_BF16) || rotary_dim > head_dim || rotary_dim % 16)
    return SPLASH_ERR_UNSUPPORTED;
  if (rotary_dim > 0 && (num_axes < 1 || !(fabsf(rope_scale) < INFINITY)))
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return SPLASH_OK;
  if (!q || !k || !v || !slots || !q_out || !k_pages || !v_pages || !k_scales || !v_scales ||
      (rotary_dim > 0 && (!inv_freq || !positions)))
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (v_pages != k_pages + (size_t)page_size * head_dim) return SPLASH_ERR_INVALID_ARGUMENT;
  // rows are read and written 16 bytes at a time
  const int per16 = dtype == SPLASH_F32 ? 4 : 8;
  const long long strides = q_stride | q_head_stride | k_stride | k_head_stride | v_stride | v_head_stride;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_pages) ||
      strides < 0 || strides % per16)
    return SPLASH_ERR_INVALID_ARGUMENT;

  QkvParams p{};
  p.q = q; p.k = k; p.v = v;
  p.q_tok = q_stride; p.q_head = q_head_stride;
  p.k_tok = k_stride; p.k_head = k_head_stride;
  p.v_tok = v_stride; p.v_head = v_head_stride;
  p.n = num_tokens;
  p.hq = num_q_heads; p.hkv = num_kv_heads;
  p.q_weight = q_weight; p.k_weight = k_weight; p.eps = eps;
  p.inv_freq = inv_freq; p.freq_axis = freq_axis;
  p.half = interleaved ? -(rotary_dim / 2) : rotary_dim / 2;
  p.positions = positions; p.axes = num_axes; p.rope_scale = rope_scale;
  p.slots = slots;
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  p.k_pages = k_pages; p.v_pages = v_pages; p.k_scales = k_scales; p.v_scales = v_scales;
  p.num_pages = num_pages;
  p.status = device_status;

  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  const int rows_per_group = 32 * kEpl / head_dim;
  const int groups = (num_q_heads + 2 * num_kv_heads + rows_per_group - 1) / rows_per_group;
  // A token's heads stay with one warp while there are warps enough to fill the
  // GPU; fewer tokens are split by heads.
  const long long warps = 32LL * sms;
  int per_item = (int)((groups * (long long)num_tokens + warps - 1) / warps);
  per_item = per_item < 1 ? 1 : (per_item > groups ? groups : per_item);
  p.groups_per_item = per_item;
  p.items_per_token = (groups + per_item - 1) / per_item;
  const long long items = (long long)p.items_per_token * num_tokens;
  const long long ctas = (items + kQkvWarps - 1) / kQkvWarps;
  if (ctas > 0x7fffffffLL) return SPLASH_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (head_dim) {
    case 64: e = launch_qkv<64>(p, dtype, (unsigned)ctas, s); break;
    case 128: e = launch_qkv<128>(p, dtype, (unsigned)ctas, s); break;
    default: e = launch_qkv<256>(p, dtype, (unsigned)ctas, s); break;
  }
  return counted(e) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}
