// Log probabilities of given tokens, entropy and the k likeliest tokens, from rows of
// logits in one pass over them.
//
//   m = max z,  S = sum e^(z - m),  W = sum (z - m) e^(z - m)
//   log p(v) = z_v - m - ln S       H = ln S - W / S
//
// Reading the logits is the floor (HBM): 1500 rows of 131072 bf16 values 58 us, of which
// the pass takes 64 and a call 74; 112 rows of 100003 fp32 values 6.6, 9.4 and 20. A value
// costs the pass 9.0 instructions, which fill 73% of the issue slots: so the maximum is
// taken on the values as stored, the sums run on pairs, and the reference m is moved only
// where a block's maximum exceeds it by more than 2^8 (in e^: by 8 ln 2), for the whole
// warp at once. A block is 1024 values, or 512 of fp32: four 16-byte loads a lane.
// All sums are fp32, a few thousand terms to a lane before they are merged.
//
// The k largest come out of the maxima of segments of 256 values or more, which the
// pass has anyway: ordered by (maximum, lowest segment first), the k first segments
// hold the k largest values by (value, lowest index first), since a value of another
// segment has k values before it. Only those segments are read again, and of them
// only what reaches the k-th segment's maximum is ordered. (A vocabulary of no more than
// k segments is read again whole, and the maxima of the threads' shares stand in for
// the segments'.)
//
// Kernel 1: a warp per run of up to 8 blocks of a row -> (m, S, W) and the segments'
// maxima in the workspace. Kernel 2: a CTA per row joins them. One kernel with a CTA per
// row took 102 us for the 1500 rows, and one row would have had one SM.
#include <climits>

#include "splash_common.cuh"
#include "splash_host.cuh"

namespace splash {
namespace {

constexpr int kLoads = 4;                // 16-byte loads of a lane in a block
constexpr int kRunBlocks = 8;            // of a run at most
constexpr int kUnit = 256;               // values of the smallest segment
constexpr int kSegsPerThread = 6;        // of the join: it holds a row's segments in registers
constexpr int kMaxTop = 32;
constexpr int kPassThreads = 256;
constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kSelect = kThreads - 32;   // threads that hold segments
constexpr int kMaxSegments = kSelect * kSegsPerThread;
constexpr int kHot = 256, kCandidates = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kMaxFinite = 3.402823466e38f;
constexpr float kMoveLog2 = 8.0f;
constexpr float kNear = 65536.f;         // references that one fused product a value is right for
constexpr float kNothing = -200.f;       // 2^ this and less is 0 in fp32

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
  int seg_units;                         // of a segment, a power of two
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
// x as a whole number of the same order; -0 as 0, NaN as -inf, infinity as the largest finite.
__device__ inline uint32_t ordered(float x) {
  x = x >= -INFINITY ? fminf(x, kMaxFinite) : -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// The types' 16-byte vectors as pairs of fp32, as they are or raised to a low finite
// value (NaN and -inf too). In a block whose maximum is above kFast the exponentials of
// raised values are 0. kBlock: values that a warp takes at a time.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kPer = 4, kBlock = 32 * kLoads * kPer;
  static constexpr float kFast = -9e37f;
  static __device__ uint4 empty() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  static __device__ float largest1(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                 fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ float2 pair(const uint4& v, int i) {
    const uint32_t a = i == 0 ? v.x : v.z, b = i == 0 ? v.y : v.w;
    return make_float2(__uint_as_float(a), __uint_as_float(b));
  }
  static __device__ float2 raised(const uint4& v, int i) {
    const float2 f = pair(v, i);
    return make_float2(fmaxf(f.x, -1e38f), fmaxf(f.y, -1e38f));
  }
  static __device__ float raw(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kPer = 8, kBlock = 32 * kLoads * kPer;
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
  static __device__ __nv_bfloat162 largest2(const uint4& v) {
    return __hmax2(__hmax2(as(v.x), as(v.y)), __hmax2(as(v.z), as(v.w)));
  }
  static __device__ float largest1(const uint4& v) {
    const __nv_bfloat162 m = largest2(v);
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ float2 floats(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ float2 pair(const uint4& v, int i) { return floats(word(v, i)); }
  static __device__ float2 raised(const uint4& v, int i) {
    const __nv_bfloat162 c = __hmax2(as(word(v, i)), __floats2bfloat162_rn(-1e38f, -1e38f));
    return floats(*reinterpret_cast<const uint32_t*>(&c));
  }
  static __device__ float raw(const uint4& v, int i) {
    const uint32_t w = word(v, i >> 1);
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Vec<__half> {
  static constexpr int kPer = 8, kBlock = 32 * kLoads * kPer;
  static constexpr float kFast = -60000.f;
  static __device__ uint4 empty() {
    return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
  }
  static __device__ __half2 as(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
  static __device__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  }
  static __device__ __half2 largest2(const uint4& v) {
    return __hmax2(__hmax2(as(v.x), as(v.y)), __hmax2(as(v.z), as(v.w)));
  }
  static __device__ float largest1(const uint4& v) {
    const __half2 m = largest2(v);
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ float2 pair(const uint4& v, int i) { return __half22float2(as(word(v, i))); }
  static __device__ float2 raised(const uint4& v, int i) {
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

// (S, W) with every exponent d larger.
__device__ inline void shift_exponents(float d, float& S, float& W) {
  const float f = ex2(d);
  W = f * (W + d * S);
  S *= f;
}

// Moves (S, W) from reference m to m2.
__device__ inline void move_reference(float m, float m2, float& S, float& W) {
  if (m == -INFINITY) {                  // nothing summed yet
    S = W = 0.f;
    return;
  }
  shift_exponents(fmaxf((m - m2) * kLog2e, -2000.f), S, W);
}

// What a warp has summed: S and W as pairs that are added up at the end. With a
// reference near 0 an exponent is one fused product, z log2 e + shift, where shift is
// -m log2 e rounded: every exponent is too large by `rest`, what the rounding cut off,
// and the sums' are made good once, when the reference moves or the run ends. (Left in, it
// is 6e-4 of log p at a logit of 30000, and at 1e10 no weight is anywhere near its value.)
// Beyond kNear rest would grow: there the maximum is taken off first, at an instruction
// more a pair, and rest is 0.
struct Sums {
  float m = -INFINITY;                   // the same in every lane
  float shift = 0.f, rest = 0.f;
  float2 S = make_float2(0.f, 0.f), W = make_float2(0.f, 0.f);
  __device__ bool near() const { return fabsf(m) <= kNear; }
  // The sums about their reference itself.
  __device__ float2 plain() const {
    float s = S.x + S.y, w = W.x + W.y;
    shift_exponents(-rest, s, w);
    return make_float2(s, w);
  }
  __device__ void refer_to(float m2) {
    float2 a = plain();
    move_reference(m, m2, a.x, a.y);
    m = m2;
    shift = -__fmul_rn(m, kLog2e);
    rest = near() ? __fmaf_rn(m, kLog2e, shift) : 0.f;
    shift_exponents(rest, a.x, a.y);
    S = make_float2(a.x, 0.f);
    W = make_float2(a.y, 0.f);
  }
};

// A block value by value: the ends of a row, and values at the ends of the types'
// range (infinity counts as the largest finite value). Returns the units' maxima.
template <typename T>
__device__ inline void block_by_value(const Row<T>& row, int b, Sums& a,
                                      float (&unit)[Vec<T>::kBlock / kUnit]) {
#pragma unroll
  for (int g = 0; g < Vec<T>::kBlock / kUnit; ++g) {
    const int p0 = b * Vec<T>::kBlock + g * kUnit + (threadIdx.x & 31);
    float z[kUnit / 32], top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kUnit / 32; ++u) {
      const int at = p0 + 32 * u;
      z[u] = at >= row.shift && at < row.end ? (float)row.base[at] : -INFINITY;
      top = fmaxf(top, z[u]);            // NaN is nothing
    }
    top = warp_fmax(top);
    unit[g] = top;
    if (top == -INFINITY) continue;
    if (fminf(top, kMaxFinite) > a.m) a.refer_to(fminf(top, kMaxFinite));
#pragma unroll
    for (int u = 0; u < kUnit / 32; ++u) {
      if (!(z[u] > -INFINITY)) continue;           // NaN neither
      const float t = fmaxf((fminf(z[u], kMaxFinite) - a.m) * kLog2e, -2000.f) + a.rest, e = ex2(t);
      a.S.x += e;
      a.W.x += e * t;
    }
  }
}

// One warp over the blocks [b0, b1) of a row: its (m, S, W) in every lane, and the
// maxima of the segments that it covers, the first of them to seg_out[0].
template <typename T>
__device__ inline float3 run_over(const Row<T>& row, int b0, int b1, int seg_units,
                                  float* seg_out) {
  constexpr int kPer = Vec<T>::kPer, kBlock = Vec<T>::kBlock;
  constexpr int kUnits = kBlock / kUnit, kLoadsPerUnit = kLoads / kUnits;
  const int lane = threadIdx.x & 31;
  // the blocks that lie inside the row
  const int in0 = min(max(b0, row.shift > 0 ? 1 : 0), b1), in1 = max(min(b1, row.end / kBlock), in0);
  Sums a;
  float seg = -INFINITY;
  int left = seg_units / kUnits;         // blocks of the segment to come, where it has several
  bool careful = false;                  // the same in every lane
  const auto note = [&](const float (&unit)[kUnits], float top, bool last) {
    if (seg_units >= kUnits) {
      seg = fmaxf(seg, top);
      if (--left <= 0 || last) {
        if (lane == 0) *seg_out = seg;
        ++seg_out;
        left = seg_units / kUnits;
        seg = -INFINITY;
      }
    } else {                             // a lane per segment
      float mine = top;
#pragma unroll
      for (int g = 0; g < kUnits; ++g)
        if (lane * seg_units == g) mine = seg_units == 1 ? unit[g] : fmaxf(unit[g], unit[g ^ 1]);
      if (lane * seg_units < kUnits) seg_out[lane] = mine;
      seg_out += kUnits / seg_units;
    }
  };
  const auto edge = [&](int b) {
    float unit[kUnits];
    block_by_value(row, b, a, unit);
    float top = unit[0];
#pragma unroll
    for (int g = 1; g < kUnits; ++g) top = fmaxf(top, unit[g]);
    note(unit, top, b + 1 == b1);
  };
  uint4 v[kLoads], x[kLoads];
  const uint4* from = reinterpret_cast<const uint4*>(row.base) + (long long)in0 * (kBlock / kPer) + lane;
  const auto fetch = [&] {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) v[u] = __ldg(from + 32 * u);
    from += kBlock / kPer;
  };
  if (in0 < in1) fetch();
#pragma unroll 1
  for (int b = b0; b < in0; ++b) edge(b);
#pragma unroll 1
  for (int b = in0; b < in1; ++b) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) x[u] = v[u];
    if (b + 1 < in1) fetch();
    float unit[kUnits];
#pragma unroll
    for (int g = 0; g < kUnits; ++g) {
      float t = Vec<T>::largest1(x[g * kLoadsPerUnit]);
#pragma unroll
      for (int u = 1; u < kLoadsPerUnit; ++u)
        t = fmaxf(t, Vec<T>::largest1(x[g * kLoadsPerUnit + u]));
      unit[g] = warp_fmax(fmaxf(t, -INFINITY));    // NaN is nothing
    }
    float top = unit[0];
#pragma unroll
    for (int g = 1; g < kUnits; ++g) top = fmaxf(top, unit[g]);
    note(unit, top, b + 1 == b1);
    const float above = (top - a.m) * kLog2e;
    if (above < kNothing) continue;      // weights of 0, as a mask's values have
    if (!(top > Vec<T>::kFast && fmaxf(top, a.m) < 1e37f)) {
      if (top > -INFINITY) block_by_value(row, b, a, unit);
      continue;
    }
    if (!(above <= kMoveLog2)) a.refer_to(top);
    const float2 scale = make_float2(kLog2e, kLog2e);
    if (!careful && a.near()) {
      const float2 shift = make_float2(a.shift, a.shift);
      const float2 S0 = a.S, W0 = a.W;
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) {
          const float2 t = __ffma2_rn(Vec<T>::pair(x[u], k), scale, shift);
          const float2 e = make_float2(ex2(t.x), ex2(t.y));
          a.S = __fadd2_rn(a.S, e);
          a.W = __ffma2_rn(e, t, a.W);
        }
      // a value of -inf (or near it, or NaN) has made W NaN: this block again, and
      // the rest of the run, with such values raised (S stays finite: t <= 8)
      careful = __any_sync(0xffffffffu, !(a.W.x + a.W.y == a.W.x + a.W.y));
      if (!careful) continue;
      a.S = S0;
      a.W = W0;
    }
    const float2 minus = make_float2(-a.m, -a.m), rest = make_float2(a.rest, a.rest);
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
#pragma unroll
      for (int k = 0; k < kPer / 2; ++k) {
        const float2 t = __ffma2_rn(__fadd2_rn(Vec<T>::raised(x[u], k), minus), scale, rest);
        const float2 e = make_float2(ex2(t.x), ex2(t.y));
        a.S = __fadd2_rn(a.S, e);
        a.W = __ffma2_rn(e, t, a.W);
      }
  }
#pragma unroll 1
  for (int b = in1; b < b1; ++b) edge(b);
  const float2 q = a.plain();
  return make_float3(a.m, warp_sum(q.x), warp_sum(q.y));
}

// Adds a run to (m, S, W).
__device__ inline void add_run(float& m, float& S, float& W, float m2, float S2, float W2) {
  if (m2 > m) {
    move_reference(m, m2, S, W);
    m = m2;
  } else {
    move_reference(m2, m, S2, W2);
  }
  S += S2;
  W += W2;
}

// ln p of a value, which rounding does not take above 0.
__device__ inline float log_p(float z, float m, float lns) {
  return fminf((fminf(z, kMaxFinite) - m) - lns, 0.f);
}

struct JoinSmem {
  uint32_t bound[kSelect / 32];
  int maxima, hot, count;
  int segs[kMaxTop];
  float least, m, lns;
  unsigned long long max_key[kMaxSegments];        // maximum and segment
  int hot_place[kHot];
  unsigned long long key[kCandidates], best[kWarps];
};

// How many of v[0 .. n) are larger.
__device__ inline int rank_of(const unsigned long long* v, int n, unsigned long long mine) {
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < n; ++j) rank += v[j] > mine;
  return rank;
}

// A barrier of the warps that hold segments.
__device__ inline void select_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSelect) : "memory"); }

// A warp's entries u < N of its lanes for which `take` holds, put at consecutive places
// from *count on. (By ballots and one atomic: with an atomic an entry the two steps that
// do this made up 3000 of the join's 12500 cycles.)
template <int N, typename Take, typename Put>
__device__ inline void append(int* count, const Take& take, const Put& put) {
  const unsigned below = (1u << (threadIdx.x & 31)) - 1;
  unsigned who[N];
  int total = 0, at = 0;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    who[u] = __ballot_sync(0xffffffffu, take(u));
    total += __popc(who[u]);
  }
  if (total == 0) return;
  if ((threadIdx.x & 31) == 0) at = atomicAdd(count, total);
  at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    if (who[u] >> (threadIdx.x & 31) & 1) put(u, at + __popc(who[u] & below));
    at += __popc(who[u]);
  }
}

// A CTA per row: a chain of short steps, each with a warp to a scheduler or less, so that
// it costs what the steps have in instructions (4 to 5 cycles each) and round trips: 3.7 us
// for one row, 5.5 to 6 for rows of fp32 at odd addresses. The runs' sums (warp 3) are formed
// beside the selection of the segments: one after the other one row took 0.9 us more. With
// 16-bit logits ten CTAs an SM, 1500 rows 76.2 -> 73.9 us; fp32 needs the registers for
// its loads (33 rows 13.4 us at eight, 14.4 at ten).
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 8 : 10) logprobs_join_kernel(Params p) {
  constexpr int kPer = Vec<T>::kPer;
  __shared__ JoinSmem s;
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  const int r = out_row(p, i);
  if (r < 0) return;
  const Row<T> row(p.logits, p.stride, r, p.vocab);
  const int n = (row.end + p.seg_units * kUnit - 1) / (p.seg_units * kUnit);   // segments
  if (warp == kWarps - 1) {
    // the row's runs
    const int blocks = (row.end + Vec<T>::kBlock - 1) / Vec<T>::kBlock;
    const int runs = (blocks + p.run_blocks - 1) / p.run_blocks;
    float m = -INFINITY, S = 0.f, W = 0.f, z = -INFINITY;
    if (lane == 0 && p.tokens) {
      const int tok = p.tokens[r];
      if (tok >= 0 && tok < p.vocab) z = (float)row.base[row.shift + tok];
    }
    for (int j = lane; j < runs; j += 32) {
      const float4 q = p.part[(long long)i * p.runs + j];
      add_run(m, S, W, q.x, q.y, q.z);
    }
    const float all = warp_max(m);
    move_reference(m, all, S, W);
    S = warp_sum(S);
    W = warp_sum(W);
    if (lane == 0) {
      const float lns = logf(S);                   // S is 0 or at least about 2^-8
      s.m = all;
      s.lns = lns;
      if (p.entropy) p.entropy[i] = S > 0.f ? fmaxf(lns - kLn2 * (W / S), 0.f) : 0.f;
      if (p.tokens)
        p.logprobs[i] = z > -INFINITY ? log_p(z, all, lns) : -INFINITY;
    }
  }
  if (p.top == 0) return;
  // The segments of the `top` largest maxima, the lowest first among equal ones. First a
  // bound that so many reach: of each warp, what a share of its lanes reach.
  // (The runs' warp meets the others after that only.)
  if (warp < kWarps - 1) {
    uint32_t key[kSegsPerThread] = {}, mine = 0;
#pragma unroll
    for (int u = 0; u < kSegsPerThread; ++u) {
      const int j = kSelect * u + tid;
      if (j < n) key[u] = ordered(p.seg_max[(long long)i * p.segments + j]);
    }
    if (tid < kMaxTop) s.segs[tid] = -1;
    if (tid == 0) {
      s.maxima = s.hot = s.count = 0;
      s.least = -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < kSegsPerThread; ++u) mine = max(mine, key[u]);
    uint32_t reached = 0;
#pragma unroll 1
    for (int u = 0; u < p.top; u += kWarps - 1) {
      reached = __reduce_max_sync(0xffffffffu, mine);
      if (mine == reached) mine = 0;
    }
    if (lane == 0) s.bound[warp] = reached;
    select_sync();
    const uint32_t bound = max(min(min(s.bound[0], s.bound[1]), s.bound[2]), 1u);
    static_assert(kWarps == 4, "bounds of three warps");
    // (a place without a segment is 0)
    append<kSegsPerThread>(&s.maxima, [&](int u) { return key[u] >= bound; }, [&](int u, int c) {
      s.max_key[c] = (unsigned long long)key[u] << 32 | (uint32_t)~(kSelect * u + tid);
    });
    select_sync();
    for (int c = tid; c < s.maxima; c += kSelect) {
      const unsigned long long k = s.max_key[c];
      const int rank = rank_of(s.max_key, s.maxima, k);
      if (rank < p.top) s.segs[rank] = (int)~(uint32_t)k;
      if (rank == p.top - 1 && n > p.top) s.least = unordered((uint32_t)(k >> 32));
    }
  }
  __syncthreads();
  const int seg_vecs = p.seg_units * (kUnit / kPer);
  const int vecs = p.top * seg_vecs;
  const auto place_of = [&](int v) {
    const int g = s.segs[v / seg_vecs];
    return g < 0 ? INT_MAX : g * (p.seg_units * kUnit) + v % seg_vecs * kPer;
  };
  const auto key_of = [&](float z, int place) {
    return (unsigned long long)ordered(z) << 32 | (uint32_t)~(place - row.shift);
  };
  if (n <= p.top) {
    // no more segments than that: the threads' own values take their place
    float mine = -INFINITY;
    for (int v = tid; v < vecs; v += kThreads) {
      const int p0 = place_of(v);
      if (p0 < row.end) mine = fmaxf(mine, Vec<T>::largest1(row.load(p0)));
    }
    s.key[tid] = (unsigned long long)ordered(mine) << 32 | (uint32_t)~tid;
    __syncthreads();
    if (rank_of(s.key, kThreads, s.key[tid]) == p.top - 1) s.least = fminf(mine, kMaxFinite);
    __syncthreads();
  }
  // vectors with a value that reaches the last of those maxima: a warp per segment,
  // kBatch vectors of a lane on their way: those of five segments of 256 values, which is a
  // warp's share (top / 4) up to top = 20; above, and with longer segments, another round
  const float least = s.least;
  constexpr int kBatch = 5 * kUnit / (32 * kPer);
  const int per_seg = seg_vecs / 32, steps = (p.top + kWarps - 1 - warp) / kWarps * per_seg;
  for (int s0 = 0; s0 < steps; s0 += kBatch) {
    uint4 x[kBatch];
    int at[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int st = s0 + u, q = per_seg == 1 ? st : per_seg == 2 ? st >> 1 : st / per_seg;
      const int g = st < steps ? s.segs[warp + kWarps * q] : -1;
      at[u] = g * (p.seg_units * kUnit) + (32 * (st - q * per_seg) + lane) * kPer;
      const bool whole = g >= 0 && at[u] >= row.shift && at[u] + kPer <= row.end;
      x[u] = Vec<T>::empty();
      if (whole) x[u] = __ldg(reinterpret_cast<const uint4*>(row.base + at[u]));
    }
    append<kBatch>(
        &s.hot, [&](int u) { return Vec<T>::largest1(x[u]) >= fmaxf(least, -kMaxFinite); },
        [&](int u, int c) {
          if (c < kHot) s.hot_place[c] = at[u];
        });
  }
  __syncthreads();
  // their values, and those of the row's ends (which may lie in other segments)
  const auto offer = [&](int place) {
    const float z = (float)row.base[place];
    if (!(z >= least && z > -INFINITY)) return;
    const int c = atomicAdd(&s.count, 1);
    if (c < kCandidates) s.key[c] = key_of(z, place);
  };
  const int hot = s.hot;
  for (int e = tid; e < min(hot, kHot) * kPer; e += kThreads)
    offer(s.hot_place[e / kPer] + e % kPer);
  if (tid < kPer) {
    if (row.shift > 0 && tid >= row.shift && tid < row.end) offer(tid);
    const int place = row.end / kPer * kPer + tid;         // of the last vector, if cut
    if (place < row.end && (place >= kPer || row.shift == 0)) offer(place);
  }
  __syncthreads();
  const int count = s.count;
  const auto put = [&](int rank, unsigned long long k) {
    p.top_ids[(long long)i * p.top + rank] = (int32_t)~(uint32_t)k;
    p.top_logprobs[(long long)i * p.top + rank] =
        log_p(unordered((uint32_t)(k >> 32)), s.m, s.lns);
  };
  if (hot <= kHot && count <= kCandidates) {
    for (int c = tid; c < count; c += kThreads) {
      const unsigned long long k = s.key[c];
      const int rank = rank_of(s.key, count, k);
      if (rank < p.top) put(rank, k);
    }
    for (int c = count + tid; c < p.top; c += kThreads) {
      p.top_ids[(long long)i * p.top + c] = -1;
      p.top_logprobs[(long long)i * p.top + c] = -INFINITY;
    }
    return;
  }
  // more equal values than the list holds: one maximum after another
  unsigned long long below = ~0ull;
  for (int rank = 0; rank < p.top; ++rank) {
    unsigned long long best = 0;
    for (int v = tid; v < vecs; v += kThreads) {
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
    if (lane == 0) s.best[warp] = best;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) best = s.best[w] > best ? s.best[w] : best;
    __syncthreads();
    if (tid == 0) put(rank, best);
    below = best;
  }
}

// A warp per run.
template <typename T>
__global__ void __launch_bounds__(kPassThreads, 4) logprobs_pass_kernel(Params p) {
  allow_dependent_launch();
  const unsigned unit = blockIdx.x * (kPassThreads / 32) + (threadIdx.x >> 5);
  const int i = unit / (unsigned)p.runs, run = unit - i * p.runs;
  if (i >= p.num_out) return;
  const int r = out_row(p, i);
  if (r < 0) return;
  const Row<T> row(p.logits, p.stride, r, p.vocab);
  const int blocks = (row.end + Vec<T>::kBlock - 1) / Vec<T>::kBlock;
  const int b0 = run * p.run_blocks, b1 = min(b0 + p.run_blocks, blocks);
  const long long seg0 = (long long)i * p.segments + b0 * (Vec<T>::kBlock / kUnit) / p.seg_units;
  const float3 q = run_over<T>(row, b0, b1, p.seg_units, p.seg_max + seg0);
  if ((threadIdx.x & 31) == 0)
    p.part[(long long)i * p.runs + run] = make_float4(q.x, q.y, q.z, 0.f);
}

// Segments of a row (which may begin off 16 bytes): units, doubled until a warp's
// registers hold their maxima. With room for those that only a last block's rest has.
struct Shape {
  int units, seg_units, segments;
};
Shape shape_of(int vocab) {
  Shape s;
  s.units = (vocab + 7 + kUnit - 1) / kUnit;
  s.seg_units = 1;
  while ((s.units + s.seg_units - 1) / s.seg_units > kMaxSegments) s.seg_units *= 2;
  s.segments = (s.units + s.seg_units - 1) / s.seg_units + 3;
  return s;
}
size_t seg_bytes(const Shape& s, int num_out) {
  return ((size_t)num_out * s.segments * sizeof(float) + 15) & ~size_t(15);
}
int up(long long a, long long b) { return (int)((a + b - 1) / b * b); }

template <typename T>
int launch(Params& p, void* workspace, int sms, cudaStream_t s) {
  const Shape sh = shape_of(p.vocab);
  constexpr int kUnits = Vec<T>::kBlock / kUnit;
  p.seg_units = sh.seg_units;
  p.segments = sh.segments;
  // runs of whole segments, about one for each of 32 warps an SM, and no longer than
  // that leaves the last of them short
  const int blocks = (sh.units + kUnits - 1) / kUnits;
  const long long per = ((long long)p.num_out * blocks + 32LL * sms - 1) / (32LL * sms);
  p.run_blocks = up(per < kRunBlocks ? per : kRunBlocks,
                    sh.seg_units > kUnits ? sh.seg_units / kUnits : 1);
  p.runs = (blocks + p.run_blocks - 1) / p.run_blocks;
  p.seg_max = static_cast<float*>(workspace);
  p.part = reinterpret_cast<float4*>(static_cast<char*>(workspace) + seg_bytes(sh, p.num_out));
  constexpr int kWarpsPerCta = kPassThreads / 32;
  const long long grid = ((long long)p.num_out * p.runs + kWarpsPerCta - 1) / kWarpsPerCta;
  if (grid * kWarpsPerCta > INT_MAX) return SPLASH_ERR_INVALID_ARGUMENT;
  logprobs_pass_kernel<T><<<(int)grid, kPassThreads, 0, s>>>(p);
  if (counted(cudaGetLastError()) != cudaSuccess) return SPLASH_ERR_CUDA;
  return counted(launch_dependent(logprobs_join_kernel<T>, dim3(p.num_out), dim3(kThreads), 0, s,
                                  p)) == cudaSuccess
             ? SPLASH_OK
             : SPLASH_ERR_CUDA;
}

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" {

size_t splash_token_logprobs_workspace_size(int num_out, int vocab) {
  if (num_out <= 0 || vocab <= 0 || vocab > (1 << 30)) return 0;
  // a run has at least a block, 512 values of the widest type
  const Shape s = shape_of(vocab);
  return seg_bytes(s, num_out) + (size_t)num_out * ((s.units + 1) / 2) * sizeof(float4);
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
  p.status = device_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case SPLASH_F32: return launch<float>(p, workspace, sms, s);
    case SPLASH_BF16: return launch<__nv_bfloat16>(p, workspace, sms, s);
    default: return launch<__half>(p, workspace, sms, s);
  }
}

}  // extern "C"
