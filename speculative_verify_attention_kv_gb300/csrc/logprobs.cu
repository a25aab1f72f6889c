// Log probabilities of given tokens, entropy and the k likeliest tokens, from rows of
// logits in one pass over them.
//
//   m = max z,  S = sum e^(z - m),  W = sum (z - m) e^(z - m)
//   log p(v) = z_v - m - ln S       H = ln S - W / S
//
// Reading the logits is the floor (HBM); the exponentials are close behind it (one
// MUFU operation a value, 16 a clock and SM: 131072 values 4.3 us on one SM, against
// 5.9 us to read them as bf16 at its share of the copy rate), so everything else of a
// value is kept to a few packed instructions: the maximum is taken on the values as
// stored, the sums run on pairs, and the reference m is moved only when a block of 512
// values exceeds it by more than 2^8 (in e^: by 8 ln 2), for the whole warp at once.
// All sums are fp32, a few thousand terms to a lane before they are merged.
//
// The k largest come out of the maxima of segments of 512 values or more, which the
// pass has anyway: ordered by (maximum, lowest segment first), the k first segments
// hold the k largest values by (value, lowest index first), since a value of another
// segment has k values before it. Only those segments are read again, and of them
// only what reaches the k-th segment's maximum is ordered. (A vocabulary of fewer
// segments is read again whole, and the maxima of the threads' shares stand in for
// the segments'.)
//
// Kernel 1: a warp per run of 512-value blocks of a row -> (m, S, W) and the segments'
// maxima in the workspace. Kernel 2: a CTA per row joins them.
#include <climits>

#include "splash_common.cuh"
#include "splash_host.cuh"

namespace splash {
namespace {

constexpr int kBlock = 512;              // values that a warp takes at a time
constexpr int kMaxSegments = 512;        // of a row (and one more where it begins off 16 bytes)
constexpr int kMaxTop = 32;
constexpr int kPassThreads = 256;
constexpr int kJoinThreads = 128;
constexpr int kCandidates = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kMaxFinite = 3.402823466e38f;
constexpr float kMoveLog2 = 8.0f;

struct Params {
  const void* logits;
  long long stride;                      // elements
  int num_rows, vocab;
  const int32_t* rows;                   // NULL: row i
  int num_out;
  const int32_t* tokens;                 // by row of the logits; NULL: no log probabilities
  float* logprobs;
  float* entropy;                        // NULL: not written
  int top;
  int32_t* top_ids;
  float* top_logprobs;
  int blocks;                            // of a row at most
  int seg_blocks;                        // blocks of a segment
  int segments;                          // of a row at most
  int run_blocks, runs;                  // blocks of a run, runs of a row
  float* seg_max;                        // [num_out, segments]
  float4* part;                          // [num_out, runs]: m, S, W (to base 2), -
  int* status;
};

__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ inline float warp_fmax(float v) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
  return y;
}
// x as a whole number of the same order; -0 as 0, NaN as -inf.
__device__ inline uint32_t ordered(float x) {
  if (!(x >= -INFINITY)) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// The types' 16-byte vectors: clamped to at least kLow (NaN and -inf too), as pairs of
// fp32. A block whose maximum is above kFast holds nothing near kLow that counts: the
// clamped values' exponentials are 0.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kPer = 4;
  static constexpr float kFast = -9e37f;
  static __device__ uint4 empty() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  static __device__ void put(uint4& v, int i, float x) { (&v.x)[i] = __float_as_uint(x); }
  static __device__ float largest(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ float2 pair(const uint4& v, int i) {
    const uint32_t a = i == 0 ? v.x : v.z, b = i == 0 ? v.y : v.w;
    return make_float2(fmaxf(__uint_as_float(a), -1e38f), fmaxf(__uint_as_float(b), -1e38f));
  }
  static __device__ float raw(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kPer = 8;
  static constexpr float kFast = -9e37f;
  static __device__ uint4 empty() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  static __device__ __nv_bfloat162 as(uint32_t w) {
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  static __device__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  }
  static __device__ float largest(const uint4& v) {
    const __nv_bfloat162 m = __hmax2(__hmax2(as(v.x), as(v.y)), __hmax2(as(v.z), as(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ float2 pair(const uint4& v, int i) {
    const __nv_bfloat162 low = __floats2bfloat162_rn(-1e38f, -1e38f);
    const __nv_bfloat162 c = __hmax2(as(word(v, i)), low);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&c);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ float raw(const uint4& v, int i) {
    const uint32_t w = word(v, i >> 1);
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Vec<__half> {
  static constexpr int kPer = 8;
  static constexpr float kFast = -60000.f;
  static __device__ uint4 empty() {
    return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
  }
  static __device__ __half2 as(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
  static __device__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  }
  static __device__ float largest(const uint4& v) {
    const __half2 m = __hmax2(__hmax2(as(v.x), as(v.y)), __hmax2(as(v.z), as(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ float2 pair(const uint4& v, int i) {
    return __half22float2(__hmax2(as(word(v, i)), __floats2half2_rn(-65504.f, -65504.f)));
  }
  static __device__ float raw(const uint4& v, int i) {
    const float2 f = __half22float2(as(word(v, i >> 1)));
    return i & 1 ? f.y : f.x;
  }
};

// A row of logits from the 16-byte boundary at or below its first value: value v is at
// place shift + v.
template <typename T>
struct Row {
  const T* base;                         // the boundary
  int shift, end;                        // places [shift, end) are the row's
  __device__ Row(const void* logits, long long stride, int row, int vocab) {
    const T* p = reinterpret_cast<const T*>(logits) + (long long)row * stride;
    shift = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    base = p - shift;
    end = shift + vocab;
  }
  // 16 bytes from place p0 on (a multiple of a vector); -inf outside the row
  __device__ uint4 load(int p0) const {
    constexpr int kPer = Vec<T>::kPer;
    if (p0 >= shift && p0 + kPer <= end)
      return __ldg(reinterpret_cast<const uint4*>(base + p0));
    uint4 v = Vec<T>::empty();
    if (p0 < end) {
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (p0 + i < shift || p0 + i >= end) continue;
        if constexpr (sizeof(T) == 4) {
          w[i] = __ldg(reinterpret_cast<const uint32_t*>(base + p0 + i));
        } else {
          const uint32_t x = __ldg(reinterpret_cast<const uint16_t*>(base + p0 + i));
          w[i >> 1] = i & 1 ? (w[i >> 1] & 0xffffu) | x << 16 : (w[i >> 1] & 0xffff0000u) | x;
        }
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
  }
};

__device__ inline int out_row(const Params& p, int i) {
  const int r = p.rows ? p.rows[i] : i;
  if (r >= p.num_rows) {
    if ((threadIdx.x & 31) == 0) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
    return -1;
  }
  return r;
}

// Moves (S, W) from reference m to m2.
__device__ inline void move_reference(float m, float m2, float& S, float& W) {
  if (m == -INFINITY) {                  // nothing summed yet
    S = W = 0.f;
    return;
  }
  const float d = fmaxf((m - m2) * kLog2e, -2000.f), f = ex2(d);
  W = f * (W + d * S);
  S *= f;
}

template <typename T>
__global__ void __launch_bounds__(kPassThreads) logprobs_pass_kernel(Params p) {
  constexpr int kPer = Vec<T>::kPer, kLoads = kBlock / 32 / kPer;
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const long long unit = ((long long)blockIdx.x * kPassThreads + threadIdx.x) >> 5;
  const int i = (int)(unit / p.runs), run = (int)(unit % p.runs);
  if (i >= p.num_out) return;
  const int r = out_row(p, i);
  if (r < 0) return;
  const Row<T> row(p.logits, p.stride, r, p.vocab);
  const int b0 = run * p.run_blocks;
  const int b1 = min(b0 + p.run_blocks, (row.end + kBlock - 1) / kBlock);
  float m = -INFINITY, seg = -INFINITY;
  float2 S = make_float2(0.f, 0.f), W = make_float2(0.f, 0.f);
  float* seg_out = p.seg_max + (long long)i * p.segments + b0 / p.seg_blocks;
  int left = p.seg_blocks;
  uint4 v[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) v[u] = row.load(b0 * kBlock + (32 * u + lane) * kPer);
  for (int b = b0; b < b1; ++b) {
    uint4 x[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      x[u] = v[u];
      if (b + 1 < b1) v[u] = row.load((b + 1) * kBlock + (32 * u + lane) * kPer);
    }
    float top = Vec<T>::largest(x[0]);
#pragma unroll
    for (int u = 1; u < kLoads; ++u) top = fmaxf(top, Vec<T>::largest(x[u]));
    top = warp_fmax(fmaxf(top, -INFINITY));        // NaN is nothing
    seg = fmaxf(seg, top);
    if (--left == 0 || b + 1 == b1) {
      if (lane == 0) *seg_out = seg;
      ++seg_out;
      left = p.seg_blocks;
      seg = -INFINITY;
    }
    if (top > Vec<T>::kFast && fmaxf(top, m) < 1e37f) {
      if (!((top - m) * kLog2e <= kMoveLog2)) {
        float s = S.x + S.y, w = W.x + W.y;
        move_reference(m, top, s, w);
        S = make_float2(s, 0.f);
        W = make_float2(w, 0.f);
        m = top;
      }
      const float2 scale = make_float2(kLog2e, kLog2e), shift = make_float2(-m * kLog2e, -m * kLog2e);
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
          const float2 t = __ffma2_rn(Vec<T>::pair(x[u], k), scale, shift);
          const float2 e = make_float2(ex2(t.x), ex2(t.y));
          S = __fadd2_rn(S, e);
          W = __ffma2_rn(e, t, W);
        }
    } else if (top > -INFINITY) {
      // values at the ends of the types' range, infinity as the largest finite one
      const float lim = fminf(top, kMaxFinite);
      if (lim > m) {
        float s = S.x + S.y, w = W.x + W.y;
        move_reference(m, lim, s, w);
        S = make_float2(s, 0.f);
        W = make_float2(w, 0.f);
        m = lim;
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const float z = Vec<T>::raw(x[u], k);
          if (!(z > -INFINITY)) continue;          // NaN neither
          const float t = fmaxf((fminf(z, kMaxFinite) - m) * kLog2e, -2000.f), e = ex2(t);
          S.x += e;
          W.x += e * t;
        }
    }
  }
  const float s = warp_sum(S.x + S.y), w = warp_sum(W.x + W.y);
  if (lane == 0) p.part[(long long)i * p.runs + run] = make_float4(m, s, w, 0.f);
}

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) logprobs_join_kernel(Params p) {
  constexpr int kPer = Vec<T>::kPer;
  constexpr int kSegsPerLane = (kMaxSegments + 32) / 32;
  __shared__ int s_segs[kMaxTop];
  __shared__ float s_least;
  __shared__ int s_count;
  __shared__ float s_m, s_lns;
  __shared__ uint32_t s_own[kJoinThreads];
  __shared__ unsigned long long s_key[kCandidates];
  __shared__ unsigned long long s_best[kJoinThreads / 32];
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  const int r = out_row(p, i);
  if (r < 0) return;
  const Row<T> row(p.logits, p.stride, r, p.vocab);
  if (warp == 0) {
    const int runs = ((row.end + kBlock - 1) / kBlock + p.run_blocks - 1) / p.run_blocks;
    float m = -INFINITY, S = 0.f, W = 0.f;
    for (int j = lane; j < runs; j += 32) {
      float4 q = p.part[(long long)i * p.runs + j];
      if (q.x > m) {
        move_reference(m, q.x, S, W);
        m = q.x;
      } else {
        move_reference(q.x, m, q.y, q.z);
      }
      S += q.y;
      W += q.z;
    }
    const float all = warp_max(m);
    move_reference(m, all, S, W);
    S = warp_sum(S);
    W = warp_sum(W);
    if (lane == 0) {
      const float lns = logf(S);                   // S is 0 or at least about 2^-8
      s_m = all;
      s_lns = lns;
      if (p.entropy) p.entropy[i] = S > 0.f ? fmaxf(lns - kLn2 * (W / S), 0.f) : 0.f;
      if (p.tokens) {
        const int tok = p.tokens[r];
        float z = -INFINITY;
        if (tok >= 0 && tok < p.vocab) z = (float)row.base[row.shift + tok];
        p.logprobs[i] = z > -INFINITY ? (fminf(z, kMaxFinite) - all) - lns : -INFINITY;
      }
    }
  } else if (warp == 1 && p.top > 0) {
    // the segments of the `top` largest maxima, the lowest first among equal ones
    const int n = ((row.end + kBlock - 1) / kBlock + p.seg_blocks - 1) / p.seg_blocks;
    uint32_t key[kSegsPerLane];
#pragma unroll
    for (int u = 0; u < kSegsPerLane; ++u) {
      const int j = 32 * u + lane;
      key[u] = j < n ? ordered(p.seg_max[(long long)i * p.segments + j]) : 0u;
    }
    uint32_t last = 0;
    int found = 0;
    for (; found < p.top; ++found) {
      uint32_t mine = 0;
#pragma unroll
      for (int u = 0; u < kSegsPerLane; ++u) mine = max(mine, key[u]);
      const uint32_t best = __reduce_max_sync(0xffffffffu, mine);
      if (best == 0) break;                        // no segment is left
      int at = INT_MAX;
#pragma unroll
      for (int u = kSegsPerLane - 1; u >= 0; --u)
        if (key[u] == best) at = 32 * u + lane;
      const int j = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
      for (int u = 0; u < kSegsPerLane; ++u)
        if (32 * u + lane == j) key[u] = 0u;
      if (lane == 0) s_segs[found] = j;
      last = best;
    }
    if (lane == 0) {
      s_count = 0;
      s_least = unordered(last);
      for (int u = found; u < p.top; ++u) s_segs[u] = -1;
    }
  }
  if (p.top == 0) return;
  __syncthreads();
  const int seg_vecs = p.seg_blocks * (kBlock / kPer);
  const int vecs = p.top * seg_vecs;
  const auto place_of = [&](int v) {
    const int s = s_segs[v / seg_vecs];
    return s < 0 ? INT_MAX : s * (p.seg_blocks * kBlock) + v % seg_vecs * kPer;
  };
  const auto key_of = [&](float z, int place) {
    return (unsigned long long)ordered(z) << 32 | (uint32_t)~(place - row.shift);
  };
  if (s_segs[p.top - 1] < 0) {
    // fewer segments than that: the threads' own values take their place
    float mine = -INFINITY;
    for (int v = tid; v < vecs; v += kJoinThreads) {
      const int p0 = place_of(v);
      if (p0 < row.end) mine = fmaxf(mine, Vec<T>::largest(row.load(p0)));
    }
    s_own[tid] = ordered(mine);
    __syncthreads();
    int rank = 0;
    for (int j = 0; j < kJoinThreads; ++j)
      rank += s_own[j] > s_own[tid] || (s_own[j] == s_own[tid] && j < tid);
    if (rank == p.top - 1) s_least = mine;
    __syncthreads();
  }
  // what reaches the last of those maxima
  const float least = s_least;
  for (int v = tid; v < vecs; v += kJoinThreads) {
    const int p0 = place_of(v);
    if (p0 >= row.end) continue;
    const uint4 x = row.load(p0);
    if (!(Vec<T>::largest(x) >= least)) continue;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const float z = Vec<T>::raw(x, k);
      if (z >= least && z > -INFINITY) {
        const int c = atomicAdd(&s_count, 1);
        if (c < kCandidates) s_key[c] = key_of(z, p0 + k);
      }
    }
  }
  __syncthreads();
  const int count = s_count;
  const auto put = [&](int rank, unsigned long long key) {
    const float z = fminf(unordered((uint32_t)(key >> 32)), kMaxFinite);
    p.top_ids[(long long)i * p.top + rank] = (int32_t)~(uint32_t)key;
    p.top_logprobs[(long long)i * p.top + rank] = (z - s_m) - s_lns;
  };
  if (count <= kCandidates) {
    for (int c = tid; c < count; c += kJoinThreads) {
      const unsigned long long key = s_key[c];
      int rank = 0;
      for (int j = 0; j < count; ++j) rank += s_key[j] > key;
      if (rank < p.top) put(rank, key);
    }
    for (int c = count + tid; c < p.top; c += kJoinThreads) {
      p.top_ids[(long long)i * p.top + c] = -1;
      p.top_logprobs[(long long)i * p.top + c] = -INFINITY;
    }
    return;
  }
  // more equal values than the list holds: one maximum after another
  unsigned long long below = ~0ull;
  for (int rank = 0; rank < p.top; ++rank) {
    unsigned long long best = 0;
    for (int v = tid; v < vecs; v += kJoinThreads) {
      const int p0 = place_of(v);
      if (p0 >= row.end) continue;
      const uint4 x = row.load(p0);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const float z = Vec<T>::raw(x, k);
        const unsigned long long key = key_of(z, p0 + k);
        if (z >= least && z > -INFINITY && key < below && key > best) best = key;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long y = __shfl_xor_sync(0xffffffffu, best, o);
      best = y > best ? y : best;
    }
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
    for (int w = 0; w < kJoinThreads / 32; ++w) best = s_best[w] > best ? s_best[w] : best;
    __syncthreads();
    if (tid == 0) put(rank, best);
    below = best;
  }
}

struct Shape {
  int blocks, seg_blocks, segments;
};
Shape shape_of(int vocab) {
  Shape s;
  s.blocks = (vocab + 7 + kBlock - 1) / kBlock;      // a row may begin off 16 bytes
  s.seg_blocks = (s.blocks + kMaxSegments - 1) / kMaxSegments;
  s.segments = (s.blocks + s.seg_blocks - 1) / s.seg_blocks;
  return s;
}
size_t seg_bytes(const Shape& s, int num_out) {
  return ((size_t)num_out * s.segments * sizeof(float) + 15) & ~size_t(15);
}

template <typename T>
int launch(const Params& p, cudaStream_t s) {
  const long long warps = (long long)p.num_out * p.runs;
  const long long grid = (warps * 32 + kPassThreads - 1) / kPassThreads;
  if (grid > INT_MAX) return SPLASH_ERR_INVALID_ARGUMENT;
  logprobs_pass_kernel<T><<<(int)grid, kPassThreads, 0, s>>>(p);
  if (counted(cudaGetLastError()) != cudaSuccess) return SPLASH_ERR_CUDA;
  return counted(launch_dependent(logprobs_join_kernel<T>, dim3(p.num_out), dim3(kJoinThreads), 0,
                                  s, p)) == cudaSuccess
             ? SPLASH_OK
             : SPLASH_ERR_CUDA;
}

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" {

size_t splash_token_logprobs_workspace_size(int num_out, int vocab) {
  if (num_out <= 0 || vocab <= 0 || vocab > (1 << 30)) return 0;
  const Shape s = shape_of(vocab);
  return seg_bytes(s, num_out) + (size_t)num_out * s.blocks * sizeof(float4);
}

int splash_token_logprobs(const void* logits, int dtype, long long logits_stride, int num_rows,
                          int vocab, const int32_t* rows, int num_out, const int32_t* tokens,
                          float* logprobs, float* entropy, int top, int32_t* top_ids,
                          float* top_logprobs, void* workspace, size_t workspace_bytes,
                          int* device_status, struct CUstream_st* stream) {
  if (num_rows < 0 || num_out < 0 || vocab <= 0 || vocab > (1 << 30) || top < 0 ||
      (!rows && num_out > num_rows))
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (dtype < SPLASH_F32 || dtype > SPLASH_F16 || top > kMaxTop) return SPLASH_ERR_UNSUPPORTED;
  if (num_out == 0 || num_rows == 0) return SPLASH_OK;
  const size_t size = dtype == SPLASH_F32 ? 4 : 2;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % size != 0 || logits_stride < vocab ||
      !workspace || !aligned16(workspace) || (tokens && !logprobs) || (!tokens && logprobs) ||
      (top > 0 && (!top_ids || !top_logprobs)))
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < splash_token_logprobs_workspace_size(num_out, vocab))
    return SPLASH_ERR_WORKSPACE_TOO_SMALL;
  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  const Shape sh = shape_of(vocab);
  // runs: about a run for every resident warp, of whole segments; long ones where the
  // rows alone fill the GPU, since a run ends with a reduction over the warp
  const long long all = (long long)num_out * sh.blocks;
  long long per = (all + 32LL * sms - 1) / (32LL * sms);
  per = per < 1 ? 1 : per > 32 ? 32 : per;
  per = (per + sh.seg_blocks - 1) / sh.seg_blocks * sh.seg_blocks;
  Params p;
  p.logits = logits;
  p.stride = logits_stride;
  p.num_rows = num_rows;
  p.vocab = vocab;
  p.rows = rows;
  p.num_out = num_out;
  p.tokens = tokens;
  p.logprobs = logprobs;
  p.entropy = entropy;
  p.top = top;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.blocks = sh.blocks;
  p.seg_blocks = sh.seg_blocks;
  p.segments = sh.segments;
  p.run_blocks = (int)per;
  p.runs = (sh.blocks + p.run_blocks - 1) / p.run_blocks;
  p.seg_max = static_cast<float*>(workspace);
  p.part = reinterpret_cast<float4*>(static_cast<char*>(workspace) + seg_bytes(sh, num_out));
  p.status = device_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case SPLASH_F32: return launch<float>(p, s);
    case SPLASH_BF16: return launch<__nv_bfloat16>(p, s);
    default: return launch<__half>(p, s);
  }
}

}  // extern "C"
