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
// shifted), and position * F_i wraps by itself, with an error below position *
// 2^-63 turns; its upper 32 bits, rounded to fp32, are the angle. So far positions
// keep the accuracy of near ones, at the cost of an integer product (fp64, the
// other way to it, runs at 2 FMA a clock and SM here). sincospif then needs no
// range reduction.
//
// A warp takes one token and a run of its heads, 8 values a lane (so a head of
// D values takes D/8 lanes, and a warp 256/D heads at once). The 8 values are two
// pieces of 4 columns, chosen so that both halves of a rotated pair sit in one
// lane: columns 4l.. and R/2 + 4l.. (interleaved: 8 columns in a row). So the
// rotation needs no exchange between lanes, a lane has 4 angles for the token,
// the same for every head, and the cosines, sines, norm weights and frequencies
// stay in registers, without exchange through shared memory.
//
// By its bytes it is bound by HBM, but with 8192 values to a 16 KB token the
// instructions come close, so they are what the layout saves. Products run on
// pairs of fp32 (f32x2); the weight is folded into the token's cosines and sines.
// A batch of kB head rows is worked on together: their kB sums of squares are
// reduced in one exchange pattern (6 shuffles and one root for 4 rows instead of
// 20 and 4). A batch is all of one kind (q, k or v). Few tokens are split over more
// warps by batches.
//
// The loads run ahead: each warp has a ring of kStages batches in shared memory,
// filled by cp.async across the ends of tokens, two batches (4 KB) in flight under
// the one worked on. A lane reads only what it copied, so the ring needs no barrier.
//
// Measured, 32768 tokens of 24 + 2 x 4 heads of 256, bf16, normed and rotated (973
// MB): 156 us, 6.2 TB/s, 92% of the measured copy rate; fp32 226 us. Heads of 128 98 us
// and of 64 68 us for the same tokens, 8 + 2 x 1 heads of 128 67 us and of 64 50 us.
// 455 tokens: 7.4 us, a chain of loads and angles. Lanes without a head on the
// quantiser's fast path and a division for the values next to a border alone: with
// all 8 values of such a lane divided 158, 226, 102, 70, 81, 64 and 8.2 us.
// Earlier, at 158 us: one batch ahead in registers instead of the ring 174 us (a first
// version with a lane to 8 columns in a row, shuffled partners and divided codes: 317
// us). 2, 4 and 6 stages 173, 160 and 160 us; with fp32 inputs 3 stages 228 us, 4 245
// us. Batches of 2 rows at 16, 20 or 24 warps to an SM: 174, 180, 181 us; 20 warps with
// batches of 4 spill: 193 us.
#include <cmath>
#include <type_traits>

#include "splash_async.cuh"
#include "splash_common.cuh"
#include "splash_host.cuh"
#include "splash_quant.cuh"

namespace splash {

namespace {

constexpr int kQkvWarps = 4;
constexpr int kQkvThreads = 32 * kQkvWarps;
constexpr int kEpl = 8;          // values a lane holds of a head row
constexpr int kWarpsPerSm = 16;  // resident: what the registers leave room for
// Warp-wide rows of a batch: 64 bytes a lane. A row of heads of 64 values is 4
// heads already; batches of 2 leave fewer rows without a head: 24 + 2 x 4 heads 66 us
// instead of 73, 32 + 2 x 8 heads 85 instead of 86 (32768 tokens).
template <typename T>
constexpr int batch_rows(int head_dim) {
  return head_dim == 64 ? 2 : 8 / (int)sizeof(T);
}
constexpr int kStages = 3;         // batches of a warp's ring

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
  int batches_per_item;          // batches of head rows an item handles
  int items_per_token;
  int* status;
};

// A lane's 8 values of a row, two pieces of 4 at p and q (kPaired: 8 from p on),
// on their way through shared memory. A lane reads only what it copied itself.
// at: of the warp's row there.
template <typename T, bool kPaired>
struct Piece;
template <bool kPaired>
struct Piece<__nv_bfloat16, kPaired> {
  static constexpr int kBytes = 512;             // of a warp's row
  __device__ static void copy(uint32_t at, int lane, const __nv_bfloat16* p,
                              const __nv_bfloat16* q, bool live) {
    if constexpr (kPaired) {
      copy_async<16>(at + lane * 16, p, live ? 16 : 0);
    } else {
      copy_async<8>(at + lane * 16, p, live ? 8 : 0);
      copy_async<8>(at + lane * 16 + 8, q, live ? 8 : 0);
    }
  }
  __device__ static void get(const unsigned char* at, int lane, float (&x)[kEpl]) {
    const uint4 v = *reinterpret_cast<const uint4*>(at + lane * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <bool kPaired>
struct Piece<float, kPaired> {
  static constexpr int kBytes = 1024;
  __device__ static void copy(uint32_t at, int lane, const float* p, const float* q, bool live) {
    copy_async<16>(at + lane * 16, p, live ? 16 : 0);
    copy_async<16>(at + 512 + lane * 16, q, live ? 16 : 0);
  }
  __device__ static void get(const unsigned char* at, int lane, float (&x)[kEpl]) {
    const float4 a = *reinterpret_cast<const float4*>(at + lane * 16);
    const float4 b = *reinterpret_cast<const float4*>(at + 512 + lane * 16);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

__device__ inline uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&t);
}

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

// Sums v[i] over the kLanes lanes of a head row, for kB rows at once, and takes
// f(sum) of each: every step halves the values that a lane carries, the last ones
// carry one; f is computed once, and each row's result handed back to all lanes.
template <int kB, int kLanes, typename F>
__device__ inline void reduce_rows(float (&v)[kB], int lane, F f) {
  constexpr uint32_t kAll = 0xffffffffu;
  static_assert(kB == 2 || kB == 4, "rows of a batch");
  constexpr int h1 = kLanes / 2, h2 = kLanes / 4;
  const bool up = lane & h1;
  float a = (up ? v[1] : v[0]) + __shfl_xor_sync(kAll, up ? v[0] : v[1], h1);
  if constexpr (kB == 4) {
    const float b = (up ? v[3] : v[2]) + __shfl_xor_sync(kAll, up ? v[2] : v[3], h1);
    const bool up2 = lane & h2;
    a = (up2 ? b : a) + __shfl_xor_sync(kAll, up2 ? a : b, h2);
  }
#pragma unroll
  for (int o = kB == 4 ? kLanes / 8 : h2; o > 0; o >>= 1) a += __shfl_xor_sync(kAll, a, o);
  a = f(a);
  const int row0 = lane & ~(kLanes - 1);         // first lane of this lane's head row
#pragma unroll
  for (int i = 0; i < kB; ++i)
    v[i] = __shfl_sync(kAll, a, row0 + (i & 1 ? h1 : 0) + (i & 2 ? h2 : 0));
}

// kPaired: interleaved pairs. kFull: the whole head is rotated (known when compiled,
// it spares every row the choice between turning and not: 193 -> 174 us for a
// 32768-token prompt). Values are held as x[0..1] = u, x[2..3] = v of the
// lane's pairs (in column order where the lane's columns are not rotated and
// kPaired is false: then u is the first piece, v the second).
template <int D, typename TIn, bool kPaired, bool kFull>
__global__ void __launch_bounds__(kQkvThreads, kWarpsPerSm / kQkvWarps)
qkv_append_kernel(QkvParams p) {
  constexpr int kLanes = D / kEpl;               // lanes of a head row
  constexpr int kRows = 32 / kLanes;             // head rows of a warp-wide load
  constexpr int kB = batch_rows<TIn>(D);
  constexpr int kHeads = kB * kRows;             // heads of a batch
  const int lane = threadIdx.x & 31, l = lane % kLanes, hl = lane / kLanes;
  const int nq = (p.hq + kHeads - 1) / kHeads, nk = (p.hkv + kHeads - 1) / kHeads;
  const int half = kFull ? D / 2 : p.half;
  const bool turns = kFull || l < half / 4;      // at most D/8 lanes
  const int ca = kPaired ? 8 * l : (turns ? 4 * l : 8 * l);
  const int cb = kPaired ? ca + 4 : (turns ? half + 4 * l : ca + 4);

  // What a lane keeps for all tokens: its frequencies in turns, and its columns
  // of the norm weights in the order of x.
  unsigned long long turn[4];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn[i] = turns64(p.inv_freq[4 * l + i]);
  }
  auto weights = [&](const float* w, F2 (&out)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(w + ca), b = *reinterpret_cast<const float4*>(w + cb);
    if constexpr (kPaired) {
      out[0] = f2(a.x, a.z); out[1] = f2(b.x, b.z);
      out[2] = f2(a.y, a.w); out[3] = f2(b.y, b.w);
    } else {
      out[0] = f2(a.x, a.y); out[1] = f2(a.z, a.w);
      out[2] = f2(b.x, b.y); out[3] = f2(b.z, b.w);
    }
  };

  using Row = Piece<TIn, kPaired>;
  __shared__ __align__(16) unsigned char s_ring[kQkvWarps][kStages][kB * Row::kBytes];
  unsigned char (*ring)[kB * Row::kBytes] = s_ring[threadIdx.x >> 5];
  // Batch `bi` of token `tok` to a stage of the ring; rows past the last head are
  // zero.
  auto copy = [&](int stage, int tok, int bi) {
    const TIn* base;
    long long head;
    int h0, heads;
    if (bi < nq) {
      h0 = bi * kHeads; heads = p.hq; head = p.q_head;
      base = static_cast<const TIn*>(p.q) + tok * p.q_tok;
    } else if (bi < nq + nk) {
      h0 = (bi - nq) * kHeads; heads = p.hkv; head = p.k_head;
      base = static_cast<const TIn*>(p.k) + tok * p.k_tok;
    } else {
      h0 = (bi - nq - nk) * kHeads; heads = p.hkv; head = p.v_head;
      base = static_cast<const TIn*>(p.v) + tok * p.v_tok;
    }
    const TIn* row = base + (h0 + hl) * head;
    const uint32_t at = shared_address(ring[stage]);
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const bool live = h0 + u * kRows + hl < heads;
      const TIn* from = live ? row : base;
      Row::copy(at + u * Row::kBytes, lane, from + ca, from + cb, live);
      row += kRows * head;
    }
  };

  const unsigned per_token = p.items_per_token, items = p.n * per_token;
  const unsigned step = gridDim.x * kQkvWarps;
  auto token_of = [&](unsigned item) { return (int)(per_token == 1 ? item : item / per_token); };
  auto batch_of = [&](unsigned item) {
    return per_token == 1 ? 0 : (int)(item % per_token) * p.batches_per_item;
  };
  const int batches = nq + 2 * nk;
  unsigned item = blockIdx.x * kQkvWarps + (threadIdx.x >> 5);
  // The next batch to copy, kStages - 1 ahead of the one worked on
  unsigned next = item;
  int next_tok = 0, next_b = 0, next_end = 0, stage_in = 0, stage = 0;
  auto next_item = [&] {
    if (next >= items) return;
    next_tok = token_of(next);
    next_b = batch_of(next);
    next_end = min(next_b + p.batches_per_item, batches);
  };
  auto copy_next = [&] {
    if (next < items) {
      copy(stage_in, next_tok, next_b);
      if (++next_b == next_end) {
        next += step;
        next_item();
      }
    }
    copies_end();
    stage_in = stage_in == kStages - 1 ? 0 : stage_in + 1;
  };
  next_item();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) copy_next();

  for (; item < items; item += step) {
    const int tok = token_of(item), b0 = batch_of(item);
    const int b1 = min(b0 + p.batches_per_item, batches);
    const int slot = p.slots[tok];
    const int page = slot / kPageSize, at = slot % kPageSize;
    if (slot < 0 || page >= p.num_pages) {       // a padded row: nothing is written
      if (slot >= 0 && lane == 0) report(p.status, SPLASH_DEVICE_BAD_PAGE);
      // its batches that are on their way are dropped, no more of them read
      int copied = b1 - b0;
      if (next == item) {
        copied = next_b - b0;
        next += step;
        next_item();
      }
      for (; copied > 0; --copied) {
        copies_wait<kStages - 2>();
        copy_next();
        stage = stage == kStages - 1 ? 0 : stage + 1;
      }
      continue;
    }

    // u' = u c - v s, v' = v c + u s for the lane's four pairs
    F2 cs[2], sn[2];
    if (turns) {
      float c[4], s[4];
      const int pos0 = p.positions[tok];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int pos = pos0;
        if (p.freq_axis) {
          const int a = max(0, min(p.freq_axis[4 * l + i], p.axes - 1));
          pos = p.positions[(size_t)a * p.n + tok];
        }
        const unsigned long long ph = (unsigned long long)(long long)pos * turn[i];
        // signed 32-bit fraction of a turn -> half turns in [-1, 1)
        sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, &s[i], &c[i]);
        c[i] *= p.rope_scale;
        s[i] *= p.rope_scale;
      }
      cs[0] = f2(c[0], c[1]); cs[1] = f2(c[2], c[3]);
      sn[0] = f2(s[0], s[1]); sn[1] = f2(s[2], s[3]);
    }
    // With weights w = (a, b): u' = u (a c) - v (b s), v' = v (b c) + u (a s); where
    // nothing turns, u' = u a, v' = v b in co[0..1] and co[2..3].
    F2 co[8];                                    // a c, b c, -b s, a s, two pairs each
    auto coefficients = [&](const float* weight) {
      const F2 neg = f2(-1.f, -1.f);
      F2 w[4];
      if (weight) weights(weight, w);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (turns) {
          co[i] = weight ? mul2(w[i], cs[i]) : cs[i];
          co[2 + i] = weight ? mul2(w[2 + i], cs[i]) : cs[i];
          co[4 + i] = mul2(weight ? mul2(w[2 + i], sn[i]) : sn[i], neg);
          co[6 + i] = weight ? mul2(w[i], sn[i]) : sn[i];
        } else if (weight) {
          co[i] = w[i];
          co[2 + i] = w[2 + i];
        }
      }
    };

    // One batch; `kv` (a compile-time truth value): k or v. turned: norm and rotate.
    auto process = [&](auto kv, int bi, int h0, bool turned, const float* weight, auto* out_row,
                       float* scale) {
      constexpr bool kKv = decltype(kv)::value;
      F2 x[kB][4];
      copies_wait<kStages - 2>();
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        float y[kEpl];
        Row::get(ring[stage] + u * Row::kBytes, lane, y);
        if constexpr (kPaired) {
          x[u][0] = f2(y[0], y[2]); x[u][1] = f2(y[4], y[6]);
          x[u][2] = f2(y[1], y[3]); x[u][3] = f2(y[5], y[7]);
        } else {
          x[u][0] = f2(y[0], y[1]); x[u][1] = f2(y[2], y[3]);
          x[u][2] = f2(y[4], y[5]); x[u][3] = f2(y[6], y[7]);
        }
      }
      copy_next();                               // to the stage read before this one
      stage = stage == kStages - 1 ? 0 : stage + 1;
      if (turned) {
        float ss[kB];
        if (weight) {
#pragma unroll
          for (int u = 0; u < kB; ++u) {
            F2 sq = mul2(x[u][0], x[u][0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) sq = fma2(x[u][i], x[u][i], sq);
            float s1;
            split(sq, ss[u], s1);
            ss[u] += s1;
          }
          reduce_rows<kB, kLanes>(ss, lane, [&](float t) { return rsqrtf(t * (1.f / D) + p.eps); });
        }
#pragma unroll
        for (int u = 0; u < kB; ++u) {
          if (turns) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const F2 a = x[u][i], b = x[u][2 + i];
              x[u][i] = fma2(b, co[4 + i], mul2(a, co[i]));
              x[u][2 + i] = fma2(a, co[6 + i], mul2(b, co[2 + i]));
            }
          } else if (weight) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = mul2(x[u][i], co[i]);
          }
          if (weight) {
            const F2 rn = f2(ss[u], ss[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = mul2(x[u][i], rn);
          }
        }
      }
      const int heads = kKv ? p.hkv : p.hq;
      auto* out_b = out_row + (cb - ca);
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        if (h0 + u * kRows >= heads) break;
        const bool live = h0 + u * kRows + hl < heads;
        float y[kEpl];                           // back to column order
        if constexpr (kPaired) {
          split(x[u][0], y[0], y[2]); split(x[u][1], y[4], y[6]);
          split(x[u][2], y[1], y[3]); split(x[u][3], y[5], y[7]);
        } else {
          split(x[u][0], y[0], y[1]); split(x[u][1], y[2], y[3]);
          split(x[u][2], y[4], y[5]); split(x[u][3], y[6], y[7]);
        }
        if constexpr (!kKv) {
          constexpr int kNext = kRows * D;       // values between the heads of a lane
          const uint32_t w0 = bf16_pair(y[0], y[1]), w1 = bf16_pair(y[2], y[3]);
          const uint32_t w2 = bf16_pair(y[4], y[5]), w3 = bf16_pair(y[6], y[7]);
          if (live) {
            if constexpr (kPaired) {
              *reinterpret_cast<uint4*>(out_row + u * kNext) = make_uint4(w0, w1, w2, w3);
            } else {
              *reinterpret_cast<uint2*>(out_row + u * kNext) = make_uint2(w0, w1);
              *reinterpret_cast<uint2*>(out_b + u * kNext) = make_uint2(w2, w3);
            }
          }
        } else {
          constexpr int kNext = kRows * 2 * kPageSize * D;
          float a = 0.f;
#pragma unroll
          for (int i = 0; i < kEpl; ++i) a = fmaxf(a, fabsf(y[i]));
          if constexpr (kLanes == 32) {          // the order of fp32 >= 0 is that of its bits
            a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
          } else {
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
          }
          const float s = __fdiv_rn(a, 127.0f);
          uint32_t packed[2];
          quantise<kEpl>(y, s, packed);
          if (live) {
            if constexpr (kPaired) {
              *reinterpret_cast<uint2*>(out_row + u * kNext) = make_uint2(packed[0], packed[1]);
            } else {
              *reinterpret_cast<uint32_t*>(out_row + u * kNext) = packed[0];
              *reinterpret_cast<uint32_t*>(out_b + u * kNext) = packed[1];
            }
            if (l == 0) scale[u * kRows * kPageSize] = s;
          }
        }
      }
    };

    int bi = b0;
    if (bi < min(b1, nq)) {
      coefficients(p.q_weight);
      for (; bi < min(b1, nq); ++bi)
        process(std::false_type{}, bi, bi * kHeads, true, p.q_weight,
                p.q_out + ((size_t)tok * p.hq + bi * kHeads + hl) * D + ca, nullptr);
    }
    if (bi < min(b1, nq + nk)) coefficients(p.k_weight);
    for (; bi < b1; ++bi) {
      const bool is_k = bi < nq + nk;
      const int h0 = (is_k ? bi - nq : bi - nq - nk) * kHeads, h = h0 + hl;
      process(std::true_type{}, bi, h0, is_k, p.k_weight,
              (is_k ? p.k_pages : p.v_pages) + code_offset(page, h, p.hkv, at, D) + ca,
              (is_k ? p.k_scales : p.v_scales) + ((size_t)page * p.hkv + h) * kPageSize + at);
    }
  }
}

template <int D, bool kPaired, bool kFull>
cudaError_t launch_qkv(const QkvParams& p, int dtype, unsigned grid, cudaStream_t s) {
  if (dtype == SPLASH_F32)
    qkv_append_kernel<D, float, kPaired, kFull><<<grid, kQkvThreads, 0, s>>>(p);
  else
    qkv_append_kernel<D, __nv_bfloat16, kPaired, kFull><<<grid, kQkvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_qkv(const QkvParams& p, int dtype, bool paired, unsigned grid, cudaStream_t s) {
  if (p.half == D / 2)
    return paired ? launch_qkv<D, true, true>(p, dtype, grid, s)
                  : launch_qkv<D, false, true>(p, dtype, grid, s);
  return paired ? launch_qkv<D, true, false>(p, dtype, grid, s)
                : launch_qkv<D, false, false>(p, dtype, grid, s);
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
      !aligned16(q_weight) || !aligned16(k_weight) || strides < 0 || strides % per16)
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
  p.half = rotary_dim / 2;
  p.positions = positions; p.axes = num_axes; p.rope_scale = rope_scale;
  p.slots = slots;
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  p.k_pages = k_pages; p.v_pages = v_pages; p.k_scales = k_scales; p.v_scales = v_scales;
  p.num_pages = num_pages;
  p.status = device_status;

  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  const int heads = (dtype == SPLASH_F32 ? batch_rows<float>(head_dim)
                                         : batch_rows<__nv_bfloat16>(head_dim)) *
                    (32 * kEpl / head_dim);
  const int batches = (num_q_heads + heads - 1) / heads + 2 * ((num_kv_heads + heads - 1) / heads);
  // A token's heads stay with one warp while there are tokens enough to fill the
  // GPU; fewer are split by batches. More items than warps fit at once are taken
  // in turns, so that the frequencies are set up once a warp.
  const long long warps = (long long)kWarpsPerSm * sms;
  int per_item = (int)((batches * (long long)num_tokens + warps - 1) / warps);
  per_item = per_item < 1 ? 1 : (per_item > batches ? batches : per_item);
  p.batches_per_item = per_item;
  p.items_per_token = (batches + per_item - 1) / per_item;
  const long long items = (long long)p.items_per_token * num_tokens;
  const long long want = (items + kQkvWarps - 1) / kQkvWarps, most = warps / kQkvWarps;
  const unsigned grid = (unsigned)(want < most ? want : most);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (head_dim) {
    case 64: e = launch_qkv<64>(p, dtype, interleaved != 0, grid, s); break;
    case 128: e = launch_qkv<128>(p, dtype, interleaved != 0, grid, s); break;
    default: e = launch_qkv<256>(p, dtype, interleaved != 0, grid, s); break;
  }
  return counted(e) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}
