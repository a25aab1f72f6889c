// The target's choice for every verify row from its logits, under penalties for
// repeated tokens, biases and grammar masks; and the token history behind the
// penalties.
//
// State. state[b][v] (int16): bit 15 says that v is in sequence b's prompt, bits
// 0..14 count v in its committed output (held at 32767).
// Row t of sequence b, whose block is x_0 .. x_{T-1}: the block's own tokens up
// to the row are output too, although not committed yet, so
//   c  = count(b, v) + #{s <= t : x_s = v},   seen = c > 0 or in the prompt
//   z1 = seen ? (z > 0 ? z / r : z * r) : z   r = repetition_b
//   z2 = z1 - f * c                           f = frequency_b
//   z3 = z2 - (c > 0 ? p : 0)                 p = presence_b
//   z4 = z3 + bias_v                          (an id listed twice: its last entry)
//   z5 = allowed by the row's mask ? z4 : -inf
// each step rounded to fp32. The choice is the lowest index of the largest z5
// above -inf (NaN is never chosen), -1 where there is none.
//
// What bounds it is reading the logits once. Of a vocabulary only few tokens are
// touched by a penalty or a bias, so the work is split in two. A CTA takes a
// window of the vocabulary for up to kChunk rows of one sequence. It first marks
// the touched ("special") tokens of the window in a bitmap from the state, the
// block and the biases, all read once for the rows. The dense pass then streams
// the rows, the next ones' loads in flight, and takes only a maximum, of the logits as they are stored:
// excluded tokens (special ones, and those that the mask closes) become -inf by
// one logic operation a register, 16-bit types stay packed in pairs. One warp
// maximum a row tells which warp's stretch holds the window's best; its place is
// looked up once at the end. The special tokens (a few dozen a window) are done
// exactly, one a lane for a few rows at a time. Choices are 64-bit keys (ordered
// value, complement of the index) merged by maximum, which no order changes. A
// second kernel takes each row's maximum over the windows.
//
// Rows of an odd vocabulary start at any alignment. Each row's vector grid is
// shifted to its own 16-byte boundary and its window with it, so the loads stay
// full vectors; the bitmap and mask bits of a vector come from a funnel shift.
#include <climits>
#include <cmath>
#include <cstring>

#include "splash_common.cuh"
#include "splash_host.cuh"

namespace splash {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlock = 128;       // verify rows of a sequence
// Rows of a CTA: enough to share a window's set-up, few enough that sequences of
// long and short blocks end together and that few sequences fill the GPU.
constexpr int kChunk = 8;
constexpr int kWarps = kThreads / 32;
constexpr int kRowBatch = 4;         // rows a special token is done for at once
constexpr uint32_t kAll = 0xffffffffu;

struct TargetParams {
  const void* logits;
  long long stride;                  // values
  int num_rows;
  int vocab;
  const int32_t* q_off;
  int num_seqs;
  int max_block;
  const int32_t* tokens;
  const int16_t* state;
  long long state_stride;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_off;
  const int32_t* bias_ids;
  const float* bias_values;
  int num_bias;
  const int32_t* mask;
  long long mask_stride;             // words
  const int32_t* mask_rows;
  int num_masks;
  float* out;                        // may be the logits (fp32, same stride)
  long long out_stride;
  int32_t* targets;
  unsigned long long* part;          // [num_rows, windows]
  int windows;
  int chunks;                        // of kChunk rows, to max_block
  int* status;
};

template <typename T>
__device__ inline float widen(T v);
template <>
__device__ inline float widen<float>(float v) { return v; }
template <>
__device__ inline float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ inline float widen<__half>(__half v) { return __half2float(v); }

// 16 bytes of logits as they are stored, and the few operations the dense pass
// needs on them. `keep` has a bit per value; a value whose bit is 0 becomes -inf.
// A bit is spread over its value's bytes by a product that brings bit j to the
// top of byte j, and a byte permute that repeats the sign of a byte.
__device__ inline uint32_t spread4(uint32_t bits) { return (bits & 15u) * 0x10204080u; }
template <uint32_t kSel>
__device__ inline uint32_t signs(uint32_t w) {         // a selector nibble 8 + b: sign of byte b
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(kSel));
  return r;
}
__device__ inline uint32_t keep_or(uint32_t w, uint32_t m, uint32_t other) {
  return (w & m) | (other & ~m);
}

template <typename T>
struct Packed;
template <>
struct Packed<float> {
  static constexpr uint32_t kNone = 0xff800000u;      // -inf
  __device__ static void drop(uint4& w, uint32_t keep) {
    const uint32_t s = spread4(keep);
    w.x = keep_or(w.x, signs<0x8888>(s), kNone);
    w.y = keep_or(w.y, signs<0x9999>(s), kNone);
    w.z = keep_or(w.z, signs<0xaaaa>(s), kNone);
    w.w = keep_or(w.w, signs<0xbbbb>(s), kNone);
  }
  __device__ static uint32_t none() { return kNone; }
  __device__ static uint32_t max(uint32_t m, const uint4& w) {       // a NaN loses
    const float a = fmaxf(fmaxf(__uint_as_float(m), __uint_as_float(w.x)), __uint_as_float(w.y));
    return __float_as_uint(fmaxf(fmaxf(a, __uint_as_float(w.z)), __uint_as_float(w.w)));
  }
  __device__ static float value(uint32_t m) { return __uint_as_float(m); }
  __device__ static void unpack(const uint4& w, float (&z)[4]) {
    z[0] = __uint_as_float(w.x); z[1] = __uint_as_float(w.y);
    z[2] = __uint_as_float(w.z); z[3] = __uint_as_float(w.w);
  }
};
// Pairs of 16-bit values
template <typename T, typename T2, uint32_t kPairNone>
struct Packed16 {
  static constexpr uint32_t kNone = kPairNone;
  __device__ static void drop(uint4& w, uint32_t keep) {
    const uint32_t s = spread4(keep), t = spread4(keep >> 4);
    w.x = keep_or(w.x, signs<0x9988>(s), kNone);
    w.y = keep_or(w.y, signs<0xbbaa>(s), kNone);
    w.z = keep_or(w.z, signs<0x9988>(t), kNone);
    w.w = keep_or(w.w, signs<0xbbaa>(t), kNone);
  }
  __device__ static uint32_t none() { return kNone; }
  __device__ static T2 pair(uint32_t w) { return *reinterpret_cast<const T2*>(&w); }
  __device__ static uint32_t max(uint32_t m, const uint4& w) {       // a NaN loses
    const T2 a = __hmax2(__hmax2(pair(m), pair(w.x)), pair(w.y));
    const T2 b = __hmax2(__hmax2(a, pair(w.z)), pair(w.w));
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  __device__ static float value(uint32_t m) {
    const T2 p = pair(m);
    return fmaxf(widen(p.x), widen(p.y));
  }
  __device__ static void unpack(const uint4& w, float (&z)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = widen(pair(a[i]).x);
      z[2 * i + 1] = widen(pair(a[i]).y);
    }
  }
};
template <>
struct Packed<__nv_bfloat16> : Packed16<__nv_bfloat16, __nv_bfloat162, 0xff80ff80u> {};
template <>
struct Packed<__half> : Packed16<__half, __half2, 0xfc00fc00u> {};

// Unsigned order of the keys is the order of the floats; +0 and -0 are one
// value. Not for NaN.
__device__ inline uint32_t ordered(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ inline unsigned long long choice_key(float z, int v) {
  return ((unsigned long long)ordered(z) << 32) | (uint32_t)~v;
}

// The rows of sequence b, or none (T = 0) where its offsets are not usable.
__device__ inline int rows_of(const TargetParams& p, int b, int* first, bool tell) {
  const int lo = p.q_off[b], hi = p.q_off[b + 1];
  *first = lo;
  if (lo < 0 || hi < lo || hi > p.num_rows || hi - lo > p.max_block) {
    if (tell) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
    return 0;
  }
  return hi - lo;
}

// 32 bits of a bitmap from bit `o` on.
__device__ inline uint32_t bits_at(const uint32_t* map, int o) {
  return __funnelshift_r(map[o >> 5], map[(o >> 5) + 1], o & 31);
}

// The row's mask, or kNoMask / kShut (an index past the masks there are: closed
// rather than open).
constexpr int kNoMask = -1, kShut = -2;
__device__ inline int mask_of(const TargetParams& p, int row) {
  if (!p.mask) return kNoMask;
  const int m = p.mask_rows ? p.mask_rows[row] : row;
  if (m < 0) return kNoMask;
  if (m < p.num_masks) return m;
  report(p.status, SPLASH_DEVICE_BAD_LENGTH);
  return kShut;
}
__device__ inline const uint32_t* mask_words(const TargetParams& p, int m) {
  return reinterpret_cast<const uint32_t*>(p.mask) + (size_t)m * p.mask_stride;
}

template <typename T, int NV>
struct Window {
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kTokens = kThreads * kVec * NV;
  // The bitmap begins 32 tokens before the window: a shifted row's window
  // begins up to kVec - 1 tokens early.
  static constexpr int kBits = kTokens + 32;
  static constexpr int kWords = kBits / 32;
};

// One row's vectors of a thread: the logits and, where a mask applies, its bits.
template <typename T, int NV>
struct RowVecs {
  static constexpr int kVec = 16 / sizeof(T);
  uint4 raw[NV];
  uint32_t bits[NV];

  // v0: the thread's first token; vector n starts 32 * kVec * n after it.
  __device__ void load(const T* z_row, const uint32_t* mask, int v0, int V) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int v = v0 + n * 32 * kVec;
      bits[n] = kAll;
      if (v >= 0 && v + kVec <= V) {
        raw[n] = *reinterpret_cast<const uint4*>(z_row + v);
        if (mask) {
          bits[n] = mask[v >> 5] >> (v & 31);
          if ((v & 31) > 32 - kVec) bits[n] |= mask[(v >> 5) + 1] << (32 - (v & 31));
        }
      } else {                       // across an end of the row, or past it
        T part[kVec];
        uint32_t on = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const bool in = v + i >= 0 && v + i < V;
          part[i] = in ? z_row[v + i] : T{};
          if (in && (!mask || (mask[(v + i) >> 5] >> ((v + i) & 31)) & 1)) on |= 1u << i;
        }
        memcpy(&raw[n], part, 16);
        bits[n] = on;
      }
    }
  }
};

template <typename T, int NV, bool kOut>
__global__ void __launch_bounds__(kThreads) choose_kernel(TargetParams p) {
  using W = Window<T, NV>;
  using P = Packed<T>;
  constexpr int kVec = W::kVec;
  constexpr int kRows = 4 / NV;      // rows whose loads are in flight together
  __shared__ uint32_t s_special[W::kWords + 1], s_block[W::kWords + 1];
  __shared__ uint16_t s_list[W::kBits];
  __shared__ int s_count;
  __shared__ int s_tok[kMaxBlock], s_mask[kChunk];
  // best dense value (key of the warp that holds it), best special token
  __shared__ unsigned long long s_dense[kChunk], s_best[kChunk];
  extern __shared__ int s_bias[];    // [kBits] last bias entry + 1 of a token; with biases only

  allow_dependent_launch();
  const int win = blockIdx.x % p.windows, unit = blockIdx.x / p.windows;
  const int b = unit / p.chunks, skip = unit % p.chunks * kChunk;    // rows before this chunk
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int block_first;
  const int T_seq = rows_of(p, b, &block_first, win == 0 && skip == 0 && tid == 0);
  if (T_seq <= skip) return;
  const int T_b = min(T_seq - skip, kChunk), first = block_first + skip;
  const int V = p.vocab;
  const int lo = win * W::kTokens, base = lo - 32;          // first token of bitmap bit 0
  const int wlo = max(0, lo - (kVec - 1)), whi = min(V, lo + W::kTokens);
  const T* logits = static_cast<const T*>(p.logits);
  // First token of this thread's vectors in a row: a warp has 32 * NV vectors in
  // a stretch, so that warps follow the order of the tokens.
  auto shift_of = [&](const T* z_row) {
    return (int)((reinterpret_cast<uintptr_t>(z_row) & 15) / sizeof(T));
  };
  auto first_of = [&](int w, int shift) { return lo + (w * NV * 32 + lane) * kVec - shift; };
  RowVecs<T, NV> x[kRows];
  // Rows t0 .. of the chunk; mask(t) tells a row's mask.
  auto load_rows = [&](int t0, auto mask) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (t0 + u >= T_b) break;
      const T* z_row = logits + (first + t0 + u) * p.stride;
      const int m = mask(t0 + u);
      x[u].load(z_row, m >= 0 ? mask_words(p, m) : nullptr, first_of(warp, shift_of(z_row)), V);
    }
  };
  load_rows(0, [&](int t) { return mask_of(p, first + t); });

  // --- what is special in this window --------------------------------------
  const float rep = p.repetition ? p.repetition[b] : 1.f;
  const float r = rep > 0.f && rep < INFINITY ? rep : 1.f;
  const float pres = p.presence ? p.presence[b] : 0.f;
  const float freq = p.frequency ? p.frequency[b] : 0.f;
  const bool penal = p.state && (r != 1.f || pres != 0.f || freq != 0.f);
  int bias0 = 0, bias1 = 0;
  if (p.bias_off) {
    bias0 = p.bias_off[b];
    bias1 = p.bias_off[b + 1];
    if (bias0 < 0 || bias1 < bias0 || bias1 > p.num_bias) {
      if (win == 0 && skip == 0 && tid == 0) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
      bias0 = bias1 = 0;
    }
  }
  const bool biased = bias1 > bias0, special = penal || biased;
  for (int i = tid; i <= W::kWords; i += kThreads) s_special[i] = s_block[i] = 0;
  if (biased)
    for (int i = tid; i < W::kBits; i += kThreads) s_bias[i] = 0;
  for (int t = tid; t < skip + T_b; t += kThreads) s_tok[t] = penal ? p.tokens[block_first + t] : -1;
  if (tid < T_b) {
    s_dense[tid] = s_best[tid] = 0;
    s_mask[tid] = mask_of(p, first + tid);
  }
  if (tid == 0) s_count = 0;
  __syncthreads();
  if (special) {
    if (penal) {
      const int16_t* st = p.state + (size_t)b * p.state_stride;
      for (int v = (wlo & ~7) + tid * 8; v < whi; v += kThreads * 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(st + v);
        if (!(w.x | w.y | w.z | w.w)) continue;
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
        uint32_t hit = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          hit |= ((a[i] & 0xffffu) ? 1u << (2 * i) : 0u) | ((a[i] >> 16) ? 2u << (2 * i) : 0u);
        if (v + 8 > V) hit &= (1u << (V - v)) - 1;           // the row's padding
        const int o = v - base;
        atomicOr(&s_special[o >> 5], hit << (o & 31));      // v is a multiple of 8
      }
      for (int t = tid; t < skip + T_b; t += kThreads) {
        const int v = s_tok[t];
        if (v >= wlo && v < whi) {
          const int o = v - base;
          atomicOr(&s_special[o >> 5], 1u << (o & 31));
          atomicOr(&s_block[o >> 5], 1u << (o & 31));
        }
      }
    }
    for (int e = bias0 + tid; e < bias1; e += kThreads) {
      const int v = p.bias_ids[e];
      if (v >= wlo && v < whi) {
        const int o = v - base;
        atomicOr(&s_special[o >> 5], 1u << (o & 31));
        atomicMax(&s_bias[o], e - bias0 + 1);
      }
    }
    __syncthreads();
    for (int w = tid; w < W::kWords; w += kThreads) {
      uint32_t m = s_special[w];
      if (!m) continue;
      int at = atomicAdd(&s_count, __popc(m));
      for (; m; m &= m - 1) s_list[at++] = (uint16_t)(w * 32 + __ffs(m) - 1);
    }
    __syncthreads();
  }

  auto mask_at = [&](int t) {
    const int m = s_mask[t];
    return m >= 0 ? mask_words(p, m) : nullptr;
  };
  // The allowed values of vector n that are not special; the others -inf.
  auto keep_bits = [&](const RowVecs<T, NV>& x, int n, int v0, bool shut) -> uint32_t {
    if (shut) return 0;
    return special ? x.bits[n] & ~bits_at(s_special, v0 + n * 32 * kVec - base) : x.bits[n];
  };

  // --- dense pass: the largest value of every token that is not special -----
  for (int t0 = 0; t0 < T_b; t0 += kRows) {
    RowVecs<T, NV> now[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) now[u] = x[u];
    load_rows(t0 + kRows, [&](int t) { return s_mask[t]; });
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int t = t0 + u;
      if (t >= T_b) break;
      const int v0 = first_of(warp, shift_of(logits + (first + t) * p.stride));
      const bool shut = s_mask[t] == kShut;
      uint32_t m = P::none();
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const uint32_t keep = keep_bits(now[u], n, v0, shut);
        if constexpr (kOut) {
          // special tokens keep their logit: in place, the next pass reads it
          const int v = v0 + n * 32 * kVec;
          const uint32_t open = shut ? 0 : now[u].bits[n];
          const uint32_t sp = special ? bits_at(s_special, v - base) : 0;
          float* o = p.out + (first + t) * p.out_stride + v;
          float y[kVec];
          P::unpack(now[u].raw[n], y);
#pragma unroll
          for (int i = 0; i < kVec; ++i) y[i] = ((open | sp) >> i) & 1 ? y[i] : -INFINITY;
          if (v >= 0 && v + kVec <= V && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < kVec; i += 4)
              *reinterpret_cast<float4*>(o + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
              if (v + i >= 0 && v + i < V) o[i] = y[i];
          }
        }
        P::drop(now[u].raw[n], keep);
        m = P::max(m, now[u].raw[n]);
      }
      const uint32_t top = __reduce_max_sync(kAll, ordered(P::value(m)));
      if (lane == 0 && top > ordered(-INFINITY))
        atomicMax(&s_dense[t], ((unsigned long long)top << 32) | (uint32_t)~warp);
    }
  }
  __syncthreads();

  // --- where the dense best is: its first place in that warp's stretch ------
  for (int t = warp; t < T_b; t += kWarps) {
    const unsigned long long d = s_dense[t];
    if (d == 0) continue;
    const T* z_row = logits + (first + t) * p.stride;
    const int v0 = first_of((int)~(uint32_t)d, shift_of(z_row));
    RowVecs<T, NV> y;
    y.load(z_row, mask_at(t), v0, V);
    uint32_t at = UINT_MAX;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      P::drop(y.raw[n], keep_bits(y, n, v0, false));
      float z[kVec];
      P::unpack(y.raw[n], z);
#pragma unroll
      for (int i = kVec - 1; i >= 0; --i)
        if (ordered(z[i]) == (uint32_t)(d >> 32)) at = min(at, (uint32_t)(v0 + n * 32 * kVec + i));
    }
    at = __reduce_min_sync(kAll, at);
    if (lane == 0) atomicMax(&s_best[t], (d & 0xffffffff00000000ull) | (uint32_t)~at);
  }

  // --- the special tokens: a lane takes one for kRowBatch rows --------------
  const int listed = s_count, groups = (T_b + kRowBatch - 1) / kRowBatch;
  const int chunks = (listed + 31) / 32;
  for (int i = warp; i < chunks * groups; i += kWarps) {
    const int e = (i / groups) * 32 + lane;
    if (e >= listed) continue;
    const int o = s_list[e], v = base + o;
    const int t0 = i % groups * kRowBatch, t1 = min(t0 + kRowBatch, T_b);
    float z[kRowBatch];
    uint32_t word[kRowBatch];
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      if (t0 + u >= t1) continue;
      z[u] = widen(logits[(first + t0 + u) * p.stride + v]);
      const uint32_t* mask = mask_at(t0 + u);
      word[u] = mask ? mask[v >> 5] : (s_mask[t0 + u] == kShut ? 0 : kAll);
    }
    int count = 0;
    bool in_prompt = false;
    if (penal) {
      const int st = p.state[(size_t)b * p.state_stride + v];
      in_prompt = st < 0;
      count = st & 0x7fff;
    }
    const bool in_block = (s_block[o >> 5] >> (o & 31)) & 1;
    if (in_block)
      for (int s = 0; s < skip + t0; ++s) count += s_tok[s] == v;
    const int entry = biased ? s_bias[o] : 0;
    const float bias = entry ? p.bias_values[bias0 + entry - 1] : 0.f;
#pragma unroll
    for (int u = 0; u < kRowBatch; ++u) {
      const int t = t0 + u;
      if (t >= t1) break;
      if (in_block) count += s_tok[skip + t] == v;
      const int row = first + t;
      // the row's own window is shifted with it
      const int from = lo - shift_of(logits + row * p.stride);
      if (v < from || v >= from + W::kTokens) continue;
      float y = z[u];
      if (penal) {
        if (count > 0 || in_prompt) y = y > 0.f ? __fdiv_rn(y, r) : __fmul_rn(y, r);
        y = __fsub_rn(y, __fmul_rn(freq, (float)count));
        if (count > 0) y = __fsub_rn(y, pres);
      }
      if (entry) y = __fadd_rn(y, bias);
      if (!((word[u] >> (v & 31)) & 1)) y = -INFINITY;
      if constexpr (kOut) p.out[row * p.out_stride + v] = y;
      if (y > -INFINITY) {           // not for NaN
        const unsigned long long k = choice_key(y, v);
        if (k > s_best[t]) atomicMax(&s_best[t], k);
      }
    }
  }
  __syncthreads();
  if (tid < T_b) p.part[(size_t)(first + tid) * p.windows + win] = s_best[tid];
}

// One CTA a sequence, one warp a row: the largest key over the windows.
constexpr int kMergeThreads = 128;
__global__ void __launch_bounds__(kMergeThreads) choose_merge_kernel(TargetParams p) {
  grid_dependency_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  int first;
  const int T_b = rows_of(p, b, &first, false);
  for (int t = threadIdx.x >> 5; t < T_b; t += kMergeThreads / 32) {
    const unsigned long long* part = p.part + (size_t)(first + t) * p.windows;
    unsigned long long best = 0;
    for (int w = lane; w < p.windows; w += 32) best = part[w] > best ? part[w] : best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long y = __shfl_xor_sync(kAll, best, o);
      best = y > best ? y : best;
    }
    if (lane == 0) p.targets[first + t] = best ? (int32_t)~(uint32_t)best : -1;
  }
}

// Tokens of a window: one, two or four vectors a thread.
int window_tokens(int dtype, int nv) { return kThreads * (dtype == SPLASH_F32 ? 4 : 8) * nv; }

long long windows_for(int vocab, int dtype, int nv) {
  // a shifted row's grid begins up to a vector early
  const int w = window_tokens(dtype, nv), vec = dtype == SPLASH_F32 ? 4 : 8;
  return ((long long)vocab + vec - 1 + w - 1) / w;
}

template <typename T, int NV, bool kOut>
cudaError_t launch_choose(const TargetParams& p, cudaStream_t s) {
  const int smem = p.bias_off ? (int)sizeof(int) * Window<T, NV>::kBits : 0;
  if (smem > 0) {
    const cudaError_t e = ensure_dynamic_smem<choose_kernel<T, NV, kOut>>(smem);
    if (e != cudaSuccess) return e;
  }
  choose_kernel<T, NV, kOut>
      <<<(unsigned)((long long)p.num_seqs * p.chunks * p.windows), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_choose_nv(const TargetParams& p, int nv, cudaStream_t s) {
  if (p.out)
    return nv == 1   ? launch_choose<T, 1, true>(p, s)
           : nv == 2 ? launch_choose<T, 2, true>(p, s)
                     : launch_choose<T, 4, true>(p, s);
  return nv == 1   ? launch_choose<T, 1, false>(p, s)
         : nv == 2 ? launch_choose<T, 2, false>(p, s)
                   : launch_choose<T, 4, false>(p, s);
}

// ---------------------------------------------------------------------------
// Token history
// ---------------------------------------------------------------------------
struct HistoryParams {
  const int32_t* tokens;
  int num_tokens;
  const int32_t* q_off;
  int num_seqs;
  const int32_t* accepted;
  int16_t* state;
  long long stride;
  int vocab;
  int prompt;
  int* status;
};

// Tokens of sequence b that count: [*lo, return).
__device__ inline int counted_end(const HistoryParams& p, int b, int* lo, bool tell) {
  const int first = p.q_off[b];
  int end = p.q_off[b + 1];
  *lo = first;
  if (first < 0 || end < first || end > p.num_tokens) {
    if (tell) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
    *lo = 0;
    return 0;
  }
  if (p.accepted && end > first) {
    const int a = p.accepted[b];
    end = a < 0 ? first : (int)min((long long)end, (long long)first + a + 1);
  }
  return end;
}

// Adds the tokens to the rows in place, one token a thread. Equal tokens of a
// warp are counted once with their number; the 16-bit counter is moved by a
// compare-and-swap of its word, because it must stop at 32767. Sums of ones:
// the order changes nothing.
__global__ void __launch_bounds__(kThreads) history_add_kernel(HistoryParams p) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  int b = -1, tok = -1, lo;
  if (blockIdx.x == 0 && p.status)
    for (int c = threadIdx.x; c < p.num_seqs; c += kThreads) counted_end(p, c, &lo, true);
  if (i < p.num_tokens && p.num_seqs > 0 && i >= p.q_off[0] && i < p.q_off[p.num_seqs]) {
    b = upper_index(p.q_off, p.num_seqs, i);
    const int end = b < p.num_seqs ? counted_end(p, b, &lo, false) : 0;
    if (b < p.num_seqs && i >= lo && i < end) tok = p.tokens[i];
    if (tok < 0 || tok >= p.vocab) tok = -1;
  }
  const unsigned long long at = tok < 0 ? ~0ull : (unsigned long long)b * p.stride + tok;
  const uint32_t same = __match_any_sync(kAll, at);
  if (tok < 0 || lane != __ffs(same) - 1) return;
  // rows are 128 bytes apart at least, and the base is 16-byte aligned
  unsigned int* word = reinterpret_cast<unsigned int*>(p.state) + (at >> 1);
  const int sh = (int)(at & 1) * 16;
  if (p.prompt) {
    atomicOr(word, 0x8000u << sh);
    return;
  }
  const unsigned n = __popc(same);
  unsigned old = *reinterpret_cast<volatile unsigned int*>(word);
  for (;;) {
    const unsigned half = (old >> sh) & 0xffffu, c = half & 0x7fffu;
    const unsigned c2 = min(c + n, 32767u);
    if (c2 == c) return;
    const unsigned next = (old & ~(0xffffu << sh)) | (((half & 0x8000u) | c2) << sh);
    const unsigned seen = atomicCAS(word, old, next);
    if (seen == old) return;
    old = seen;
  }
}

// Rebuilds the rows: a CTA takes a window of `span` entries of one row, counts
// the sequence's tokens in it in shared memory and writes the window whole.
__global__ void __launch_bounds__(1024) history_reset_kernel(HistoryParams p, int span, int windows) {
  extern __shared__ int s_n[];
  const int b = blockIdx.x / windows, lo_v = blockIdx.x % windows * span;
  const int hi_v = (int)min((long long)lo_v + span, p.stride);
  for (int i = threadIdx.x; i < span; i += blockDim.x) s_n[i] = 0;
  __syncthreads();
  int lo;
  const int end = counted_end(p, b, &lo, threadIdx.x == 0 && lo_v == 0);
  const int top = min(hi_v, p.vocab);
  for (int i = lo + threadIdx.x; i < end; i += blockDim.x) {
    const int v = p.tokens[i];
    if (v >= lo_v && v < top) atomicAdd(&s_n[v - lo_v], 1);
  }
  __syncthreads();
  uint32_t* row = reinterpret_cast<uint32_t*>(p.state + (size_t)b * p.stride);
  // span and the stride are multiples of 64
  for (int i = lo_v / 2 + threadIdx.x; i < hi_v / 2; i += blockDim.x) {
    const int n0 = s_n[2 * i - lo_v], n1 = s_n[2 * i + 1 - lo_v];
    const uint32_t h0 = p.prompt ? (n0 ? 0x8000u : 0u) : (uint32_t)min(n0, 32767);
    const uint32_t h1 = p.prompt ? (n1 ? 0x8000u : 0u) : (uint32_t)min(n1, 32767);
    row[i] = h0 | (h1 << 16);
  }
}

constexpr int kSpanMost = 24576;     // entries: 96 KB of counters, two CTAs to an SM

}  // namespace
}  // namespace splash

using namespace splash;

extern "C" {

int splash_token_state_stride(int vocab) {
  return vocab <= 0 || vocab > INT_MAX - 63 ? 0 : (vocab + 63) / 64 * 64;
}

size_t splash_choose_targets_workspace_size(int num_rows, int vocab) {
  if (num_rows < 0 || vocab <= 0) return 0;
  // the smallest windows any call makes
  return sizeof(unsigned long long) * (size_t)num_rows * (size_t)windows_for(vocab, SPLASH_F32, 1);
}

int splash_choose_targets(const void* logits, int dtype, long long logits_stride, int num_rows,
                          int vocab, const int32_t* q_offsets, int num_seqs, int max_block_len,
                          const int32_t* block_tokens, const int16_t* state,
                          long long state_stride, const float* repetition, const float* presence,
                          const float* frequency, const int32_t* bias_offsets,
                          const int32_t* bias_ids, const float* bias_values, int num_bias,
                          const int32_t* mask, long long mask_stride, int num_masks,
                          const int32_t* mask_rows, float* out, long long out_stride,
                          int32_t* target_tokens, void* workspace, size_t workspace_bytes,
                          int* device_status, struct CUstream_st* stream) {
  if (num_rows < 0 || num_seqs < 0 || vocab <= 0 || vocab > (1 << 30) || max_block_len < 0 ||
      num_bias < 0 || num_masks < 0)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if ((dtype != SPLASH_F32 && dtype != SPLASH_BF16 && dtype != SPLASH_F16) ||
      max_block_len > kMaxBlock)
    return SPLASH_ERR_UNSUPPORTED;
  if (num_rows == 0 || num_seqs == 0 || max_block_len == 0) return SPLASH_OK;
  if (!logits || !q_offsets || !target_tokens || !workspace || logits_stride < vocab)
    return SPLASH_ERR_INVALID_ARGUMENT;
  const size_t es = dtype == SPLASH_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return SPLASH_ERR_INVALID_ARGUMENT;
  const bool penal = repetition || presence || frequency;
  if (penal && (!state || !block_tokens)) return SPLASH_ERR_INVALID_ARGUMENT;
  if (penal && (state_stride < vocab || state_stride % 64 || !aligned16(state)))
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (bias_offsets && num_bias > 0 && (!bias_ids || !bias_values)) return SPLASH_ERR_INVALID_ARGUMENT;
  if (mask && mask_stride < ((long long)vocab + 31) / 32) return SPLASH_ERR_INVALID_ARGUMENT;
  if (mask && !mask_rows && num_masks < num_rows) return SPLASH_ERR_INVALID_ARGUMENT;
  if (!mask && mask_rows) return SPLASH_ERR_INVALID_ARGUMENT;
  if (out && out_stride < vocab) return SPLASH_ERR_INVALID_ARGUMENT;
  if (out && static_cast<const void*>(out) == logits &&
      (dtype != SPLASH_F32 || out_stride != logits_stride))
    return SPLASH_ERR_INVALID_ARGUMENT;
  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;

  // Up to four vectors a thread and row as long as that still fills the GPU: a
  // window's set-up and merging are shared by more tokens. What the rows of a
  // sequence make in chunks counts only as far as there are rows.
  const int chunks = (max_block_len + kChunk - 1) / kChunk;
  const long long full = num_seqs + (long long)num_rows / kChunk;
  const long long units = num_seqs * (long long)chunks < full ? num_seqs * (long long)chunks : full;
  int nv = 4;
  while (nv > 1 && units * windows_for(vocab, dtype, nv) < 4LL * sms) nv /= 2;
  const long long windows = windows_for(vocab, dtype, nv);
  if (windows * num_seqs * chunks > INT_MAX) return SPLASH_ERR_UNSUPPORTED;
  if (workspace_bytes < sizeof(unsigned long long) * (size_t)num_rows * (size_t)windows)
    return SPLASH_ERR_WORKSPACE_TOO_SMALL;
  TargetParams p{logits, logits_stride, num_rows, vocab, q_offsets, num_seqs, max_block_len,
                 block_tokens, penal ? state : nullptr, state_stride, repetition, presence,
                 frequency, num_bias > 0 ? bias_offsets : nullptr, bias_ids, bias_values, num_bias,
                 mask, mask_stride, mask_rows, num_masks, out, out_stride, target_tokens,
                 static_cast<unsigned long long*>(workspace), (int)windows, chunks, device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == SPLASH_F32    ? launch_choose_nv<float>(p, nv, s)
                  : dtype == SPLASH_BF16 ? launch_choose_nv<__nv_bfloat16>(p, nv, s)
                                         : launch_choose_nv<__half>(p, nv, s);
  if (counted(e) != cudaSuccess) return SPLASH_ERR_CUDA;
  e = launch_dependent(choose_merge_kernel, dim3(num_seqs), dim3(kMergeThreads), 0, s, p);
  return counted(e) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}

int splash_token_state_add(const int32_t* tokens, int num_tokens, const int32_t* q_offsets,
                           int num_seqs, const int32_t* accepted, int16_t* state,
                           long long state_stride, int vocab, int prompt, int reset,
                           int* device_status, struct CUstream_st* stream) {
  if (num_tokens < 0 || num_seqs < 0 || vocab <= 0 || vocab > (1 << 30) || state_stride < vocab ||
      state_stride % 64 || state_stride > INT_MAX)
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (num_seqs == 0 || (num_tokens == 0 && !reset)) return SPLASH_OK;
  if ((num_tokens > 0 && !tokens) || !q_offsets || !state || !aligned16(state))
    return SPLASH_ERR_INVALID_ARGUMENT;
  HistoryParams p{tokens, num_tokens, q_offsets, num_seqs, accepted, state, state_stride, vocab,
                  prompt, device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!reset) {
    history_add_kernel<<<(num_tokens + kThreads - 1) / kThreads, kThreads, 0, s>>>(p);
    return counted(cudaGetLastError()) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
  }
  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  // Every window reads the sequence's tokens again: as few windows as fill the
  // GPU, in steps of 64 entries.
  long long windows = (sms + num_seqs - 1) / num_seqs;
  long long span = (state_stride / windows + 63) / 64 * 64;
  span = span < 2048 ? 2048 : (span > kSpanMost ? kSpanMost : span);
  windows = (state_stride + span - 1) / span;
  if (windows * num_seqs > INT_MAX) return SPLASH_ERR_UNSUPPORTED;
  const int bytes = (int)(span * sizeof(int));
  cudaError_t e = ensure_dynamic_smem<history_reset_kernel>(kSpanMost * (int)sizeof(int));
  if (e != cudaSuccess) return SPLASH_ERR_CUDA;
  history_reset_kernel<<<(unsigned)(windows * num_seqs), 1024, bytes, s>>>(p, (int)span, (int)windows);
  return counted(cudaGetLastError()) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}

}  // extern "C"
