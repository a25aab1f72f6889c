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
// By its bytes the logits, read once, bound it. In fact neither memory nor the issue
// slots are full (2 of 4 instructions a clock): a step's rows are few, everything before
// the logits (offsets, state, biases, masks) is a chain of loads, and the largest
// stall after that is the wait for the instruction before. So a warp works for
// itself, without block barriers: it takes a run of segments of the vocabulary
// (1024 tokens) for up to 8 rows of a sequence. Of a segment only few tokens
// are touched by a penalty or a bias ("special"). It marks them in a bitmap, lists
// them and fetches what they need, a token a lane. Then, a row of a block after the
// other, with the next one's logits and mask on their way to shared memory:
//   - it computes the special tokens exactly and puts them back in the copy (-inf
//     and a key beside it where the logits have 16 bits);
//   - it takes the maximum of the row as it is stored: what the mask closes becomes
//     -inf by one logic operation a register, and 16-bit types stay packed in pairs;
//   - the place of the maximum is looked up only where it beats the run's best.
// Choices are 64-bit keys (ordered value, complement of the index) merged by
// maximum, which no order changes; a second kernel takes each row's maximum over
// its runs.
//
// Measured, 16 x 16 rows of 131072 bf16 logits with 2.6% of special tokens and
// half of the rows masked (73 MB): 27 us (2.7 TB/s); without penalties, biases and
// masks 16.6 us (4.0 TB/s). 426 rows of 100003 fp32 with masks and output (359 MB): 73
// us (4.9 TB/s), as bf16 without output 41 us. 16 warps to an SM instead of 20: 27, 16,
// 76 and 45 us; 24: 28, 17, 81 and 49 us. Earlier forms: special tokens kept out of the
// dense pass by their bitmap 27, 18, 79 and 41 us; that with 4 rows to a warp 32, 20,
// 78 and 45 us; those 4 in registers, one ahead, and their special tokens together
// from global memory 34, 18, 81 and 50 us. A CTA to a window of 4096 or 8192 tokens
// with block barriers 33 and 82 us; dense and special CTAs side by side 33 and 147.
//
// Rows of an odd vocabulary start at any alignment. Each row's vector grid is
// shifted to its own 16-byte boundary and its segments with it, so the loads stay
// full vectors; the bitmap and mask bits of a vector come from a funnel shift.
#include <climits>
#include <cmath>
#include <cstring>

#include "splash_async.cuh"
#include "splash_common.cuh"
#include "splash_host.cuh"

namespace splash {

namespace {

constexpr int kThreads = 256;        // of the history kernels
constexpr int kMaxBlock = 128;       // verify rows of a sequence
// Most rows of a warp: enough to share a segment's set-up, few enough that sequences
// of long and short blocks end together (16: 26 us instead of 27 for 16 x 16 rows, 91
// instead of 78 for the ragged fp32 batch).
constexpr int kChunkMost = 8;
constexpr int kWarpsPerCta = 4;
constexpr int kWarpsResident = 20;   // to an SM: 96 registers a thread, 44 KB to a CTA
// Warps beyond which segments are taken in turn, for each SM
constexpr long long kWarpsPerSm = 64;
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
  unsigned long long* part;          // [num_rows, runs]
  int segments;                      // of a row
  int span;                          // segments of a run
  int runs;
  int chunk;                         // rows of a warp
  int chunks;                        // to max_block
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

// Eight logits as they are stored, and the few operations the dense pass needs on
// them. `keep` has a bit per value; a value whose bit is 0 becomes -inf. A bit is
// spread over its value's bytes by a product that brings bit j to the top of byte
// j, and a byte permute that repeats the sign of a byte.
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
struct Octet;
template <>
struct Octet<float> {
  uint4 a, b;
  static constexpr uint32_t kNone = 0xff800000u;      // -inf
  __device__ static void drop4(uint4& w, uint32_t keep) {
    const uint32_t s = spread4(keep);
    w.x = keep_or(w.x, signs<0x8888>(s), kNone);
    w.y = keep_or(w.y, signs<0x9999>(s), kNone);
    w.z = keep_or(w.z, signs<0xaaaa>(s), kNone);
    w.w = keep_or(w.w, signs<0xbbbb>(s), kNone);
  }
  __device__ void drop(uint32_t keep) {
    drop4(a, keep);
    drop4(b, keep >> 4);
  }
  __device__ uint32_t max(uint32_t m) const {          // a NaN loses
    float x = __uint_as_float(m);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x = fmaxf(x, __uint_as_float(w[i]));
    return __float_as_uint(x);
  }
  __device__ static float value(uint32_t m) { return __uint_as_float(m); }
  __device__ void unpack(float (&z)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __uint_as_float(w[i]);
  }
};
// Pairs of 16-bit values
template <typename T, typename T2, uint32_t kPairNone>
struct Octet16 {
  uint4 a;
  static constexpr uint32_t kNone = kPairNone;
  __device__ void drop(uint32_t keep) {
    const uint32_t s = spread4(keep), t = spread4(keep >> 4);
    a.x = keep_or(a.x, signs<0x9988>(s), kNone);
    a.y = keep_or(a.y, signs<0xbbaa>(s), kNone);
    a.z = keep_or(a.z, signs<0x9988>(t), kNone);
    a.w = keep_or(a.w, signs<0xbbaa>(t), kNone);
  }
  __device__ static T2 pair(uint32_t w) { return *reinterpret_cast<const T2*>(&w); }
  __device__ uint32_t max(uint32_t m) const {          // a NaN loses
    const T2 x = __hmax2(__hmax2(pair(m), pair(a.x)), pair(a.y));
    const T2 y = __hmax2(__hmax2(x, pair(a.z)), pair(a.w));
    return *reinterpret_cast<const uint32_t*>(&y);
  }
  __device__ static float value(uint32_t m) {
    const T2 p = pair(m);
    return fmaxf(widen(p.x), widen(p.y));
  }
  __device__ void unpack(float (&z)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = widen(pair(w[i]).x);
      z[2 * i + 1] = widen(pair(w[i]).y);
    }
  }
};
template <>
struct Octet<__nv_bfloat16> : Octet16<__nv_bfloat16, __nv_bfloat162, 0xff80ff80u> {};
template <>
struct Octet<__half> : Octet16<__half, __half2, 0xfc00fc00u> {};

// Unsigned order of the keys is the order of the floats; +0 and -0 are one
// value. Not for NaN.
__device__ inline uint32_t ordered(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
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

// Parameters of sequence b
struct SeqParams {
  int first, T;                      // its rows
  float r, pres, freq;
  bool penal;
  int bias0, bias1;
  const int16_t* state;

  __device__ SeqParams(const TargetParams& p, int b, bool tell) {
    const float rep = p.repetition ? p.repetition[b] : 1.f;
    pres = p.presence ? p.presence[b] : 0.f;
    freq = p.frequency ? p.frequency[b] : 0.f;
    bias0 = p.bias_off ? p.bias_off[b] : 0;
    bias1 = p.bias_off ? p.bias_off[b + 1] : 0;
    T = rows_of(p, b, &first, tell);
    r = rep > 0.f && rep < INFINITY ? rep : 1.f;
    penal = p.state && (r != 1.f || pres != 0.f || freq != 0.f);
    state = p.state + (size_t)b * p.state_stride;
    if (bias0 < 0 || bias1 < bias0 || bias1 > p.num_bias) {
      if (tell) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
      bias0 = bias1 = 0;
    }
  }
  __device__ bool special() const { return penal || bias1 > bias0; }
};

// A bit for each of 8 state entries that is not zero
__device__ inline uint32_t touched(const uint4& w) {
  // bit 15 of a half that is not zero: the carry out of its lower 15 bits, or the
  // bit itself; then the eight bits side by side
  auto halves = [](uint32_t a) { return (((a & 0x7fff7fffu) + 0x7fff7fffu) | a) & 0x80008000u; };
  const uint32_t m = (halves(w.x) >> 15) | (halves(w.y) >> 13) | (halves(w.z) >> 11) | (halves(w.w) >> 9);
  return (m | (m >> 15)) & 0xffu;
}

template <typename T>
struct Segment {
  static constexpr int kTokens = 1024;
  static constexpr int kOctets = 8 / sizeof(T);  // a lane's of a block: 64 bytes
  static constexpr int kBlock = 32 * 8 * kOctets;        // tokens of a block: 2 KB of a row
  static constexpr int kBlocks = kTokens / kBlock;
  static constexpr int kEarly = 16 / sizeof(T) - 1;
  // The bitmap begins 32 tokens before the segment: a shifted row's segment
  // begins up to kEarly tokens early.
  static constexpr int kBits = kTokens + 32;
  static constexpr int kWords = kBits / 32;
};

// A block of a row on its way through shared memory: the logits from token g0 on and
// the words of the row's mask from word g0 / 32 on. What lies outside the row is
// undefined there.
constexpr int kStages = 2;           // one row ahead
template <typename T>
struct Stage {
  static constexpr int kWords = Segment<T>::kBlock / 32 + 1;
  alignas(16) Octet<T> raw[32 * Segment<T>::kOctets];
  uint32_t mask[kWords + 1];                     // the last one is read, not used

  // Starts the copies of the warp; the row is z_row[0, V). Its 16-byte pieces are
  // the row's own: one at most crosses each end.
  template <bool kAligned>
  __device__ void copy(const T* z_row, const uint32_t* mask_row, int g0, int V, int lane) {
    constexpr int E = 16 / sizeof(T), kPieces = Segment<T>::kBlock / E / 32;
    const T* src = z_row + (g0 + lane * E);
    const uint32_t dst = shared_address(raw) + lane * 16;
    if ((kAligned || g0 >= 0) && g0 + Segment<T>::kBlock <= V) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) copy_async<16>(dst + i * 512, src + i * 32 * E, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int v = g0 + (i * 32 + lane) * E;
        if (v >= 0 && v < V)
          copy_async<16>(dst + i * 512, src + i * 32 * E, min(V - v, E) * (int)sizeof(T));
      }
      if (!kAligned && g0 < 0 && lane < E && g0 + lane >= 0 && g0 + lane < V)
        reinterpret_cast<T*>(raw)[lane] = z_row[g0 + lane];
    }
    if (mask_row) {
      const int words = (V + 31) >> 5, w0 = g0 >> 5;
#pragma unroll
      for (int i = 0; i < kWords; i += 32) {
        const int w = w0 + i + lane;
        if (i + lane < kWords && w >= 0 && w < words)
          copy_async<4>(shared_address(mask + i + lane), mask_row + w, 4);
      }
    }
  }
  template <bool kAligned>
  __device__ bool at_end(int g0, int V) const {
    return (!kAligned && g0 < 0) || g0 + Segment<T>::kBlock > V;
  }
  // The bits of the 8 tokens from v on that are in the row and open in its mask
  // (upper bits: others').
  template <bool kAligned>
  __device__ uint32_t open(int v, int g0, int V, bool masked) const {
    uint32_t on = kAll;
    if (masked) {
      const int i = (v >> 5) - (g0 >> 5);
      on = kAligned ? mask[i] >> (v & 31) : __funnelshift_r(mask[i], mask[i + 1], v & 31);
    }
    if (at_end<kAligned>(g0, V)) {
      const int from = v < 0 ? -v : 0, to = V - v < 8 ? V - v : 8;
      on &= to > 0 && from < 8 ? ((1u << to) - 1) & ~((1u << from) - 1) : 0;
    }
    return on;
  }
};

// Shared memory of a warp. Where there are biases, int [kBits] for each warp
// follows all of them: a token's last bias entry + 1.
template <typename T>
struct WarpSmem {
  uint32_t map[Segment<T>::kWords + 1];    // special tokens
  uint32_t block[Segment<T>::kWords + 1];  // those of the block among them
  const uint32_t* words[kChunkMost];       // of the rows' masks, nullptr for none
  uint16_t list[Segment<T>::kBits];
  Stage<T> ring[kStages];
};

template <typename T, bool kOut, bool kAligned>
__global__ void __launch_bounds__(32 * kWarpsPerCta, kWarpsResident / kWarpsPerCta)
choose_kernel(TargetParams p) {
  using S = Segment<T>;
  constexpr int N = S::kOctets;
  constexpr int kGroups = S::kTokens / 8 / 32;   // state groups of 8 entries a lane
  constexpr int kIds = 10;
  extern __shared__ __align__(16) unsigned char smem[];
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  WarpSmem<T>& sm = reinterpret_cast<WarpSmem<T>*>(smem)[warp];
  int* s_bias = reinterpret_cast<int*>(smem + kWarpsPerCta * sizeof(WarpSmem<T>)) + warp * S::kBits;

  const unsigned work = blockIdx.x * kWarpsPerCta + warp;
  const int run = work % p.runs;
  const unsigned unit = work / p.runs;
  const int chunk = unit % p.chunks, b = unit / p.chunks;
  if (b >= p.num_seqs) return;
  const int skip = chunk * p.chunk;              // rows before this chunk
  const bool lead = chunk == 0 && run == 0 && lane == 0;
  const SeqParams q(p, b, lead);
  const int T_b = min(q.T - skip, p.chunk), first = q.first + skip;
  if (T_b <= 0) return;
  const int V = p.vocab;
  const bool biased = q.bias1 > q.bias0, special = q.special();
  const T* z_first = static_cast<const T*>(p.logits) + first * p.stride;
  const int seg0 = run * p.span, seg1 = min(seg0 + p.span, p.segments);

  unsigned long long best = 0;                   // lane t: the best choice of row t so far
  const int my_mask = lane < T_b ? mask_of(p, first + lane) : kNoMask;
  if (lane < T_b) sm.words[lane] = my_mask >= 0 ? mask_words(p, my_mask) : nullptr;
  __syncwarp();
  auto words_of = [&](int t) { return p.mask ? sm.words[t] : nullptr; };
  const unsigned shut = __ballot_sync(kAll, my_mask == kShut);
  auto shift_of = [&](int t) {
    return kAligned ? 0
                    : (int)((reinterpret_cast<uintptr_t>(z_first + t * p.stride) & 15) / sizeof(T));
  };
  // First token of row t of a block (kBlocks to a segment)
  auto first_of = [&](int block, int t) { return block * S::kBlock - shift_of(t); };
  // The next row of a block to copy, kStages - 1 ahead of the one worked on
  int next_block = seg0 * S::kBlocks, next_t = 0, stage_in = 0, stage = 0;
  auto copy_next = [&] {
    if (next_block < seg1 * S::kBlocks) {
      sm.ring[stage_in].template copy<kAligned>(z_first + next_t * p.stride, words_of(next_t),
                                                first_of(next_block, next_t), V, lane);
      if (++next_t == T_b) {
        next_t = 0;
        ++next_block;
      }
    }
    copies_end();
    stage_in = stage_in == kStages - 1 ? 0 : stage_in + 1;
  };
  uint4 st[kGroups];
  auto load_state = [&](int seg) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int v = seg * S::kTokens + (i * 32 + lane) * 8;
      st[i] = v < V ? *reinterpret_cast<const uint4*>(q.state + v) : make_uint4(0, 0, 0, 0);
    }
  };
  if (q.penal) load_state(seg0);
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) copy_next();
  if (biased)
    for (int i = lane; i < S::kBits; i += 32) s_bias[i] = 0;

  for (int seg = seg0; seg < seg1; ++seg) {
    const int lo = seg * S::kTokens, base = lo - 32;        // first token of bitmap bit 0
    const int wlo = max(0, lo - S::kEarly), whi = min(V, lo + S::kTokens);
    int listed = 0, below = 0;                   // below: before the second block's tokens
    auto special_bits = [&](int n, int v0) -> uint32_t {
      const uint32_t* w = sm.map + ((v0 - base) >> 5) + n * 8;
      return kAligned ? w[0] >> (v0 & 31) : __funnelshift_r(w[0], w[1], v0 & 31);
    };
    if (special) {
      // --- mark and list the special tokens -----------------------------------
      for (int i = lane; i <= S::kWords; i += 32) sm.block[i] = 0;
      if (lane == 0) {
        // the 8 tokens before the segment, of which a shifted row may have some
        sm.map[0] = !kAligned && q.penal && lo > 0
                        ? touched(*reinterpret_cast<const uint4*>(q.state + lo - 8)) << 24 : 0;
        sm.map[S::kWords] = 0;
      }
      uint8_t* bytes = reinterpret_cast<uint8_t*>(sm.map + 1);
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int g = i * 32 + lane, v = lo + 8 * g;
        uint32_t hit = q.penal ? touched(st[i]) : 0;
        if (lo + S::kTokens > V && v + 8 > V)          // the row's padding
          hit &= v < V ? (1u << (V - v)) - 1 : 0;
        bytes[g] = (uint8_t)hit;
      }
      __syncwarp();
      if (q.penal)
        for (int t = lane; t < skip + T_b; t += 32) {
          const int v = p.tokens[q.first + t];
          if (v >= wlo && v < whi) {
            atomicOr(&sm.map[(v - base) >> 5], 1u << ((v - base) & 31));
            atomicOr(&sm.block[(v - base) >> 5], 1u << ((v - base) & 31));
          }
        }
      for (int e0 = q.bias0 + lane; e0 < q.bias1; e0 += 32 * kIds) {
        int id[kIds];                            // the loads of all before the first use
#pragma unroll
        for (int i = 0; i < kIds; ++i) id[i] = e0 + 32 * i < q.bias1 ? p.bias_ids[e0 + 32 * i] : -1;
#pragma unroll
        for (int i = 0; i < kIds; ++i)
          if (id[i] >= wlo && id[i] < whi) {
            atomicOr(&sm.map[(id[i] - base) >> 5], 1u << ((id[i] - base) & 31));
            atomicMax(&s_bias[id[i] - base], e0 + 32 * i - q.bias0 + 1);
          }
      }
      __syncwarp();
      // a word a lane; the one before the segment goes to lane 0 as well
      static_assert(S::kWords <= 33, "words of a bitmap");
      uint32_t m = lane + 1 < S::kWords ? sm.map[lane + 1] : 0;
      const uint32_t before = !kAligned && lane == 0 ? sm.map[0] : 0;
      const int mine = __popc(m) + __popc(before);
      int at = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kAll, at, o);
        if (lane >= o) at += n;
      }
      listed = __shfl_sync(kAll, at, 31);
      at -= mine;
      below = __shfl_sync(kAll, at, 16);         // lane 16: tokens from lo + 512 on
      for (uint32_t w = before; w; w &= w - 1) sm.list[at++] = (uint16_t)(__ffs(w) - 1);
      for (; m; m &= m - 1) sm.list[at++] = (uint16_t)(lane * 32 + 31 + __ffs(m));
      __syncwarp();
    }

    // --- a lane's special tokens: list[e] and what its rows need --------------
    struct Entry {
      int v;                                     // the token; none: before every row
      int count;                                 // before the chunk's rows
      float bias;
      uint32_t flags;                            // bit t: row t's token is v
    };
    constexpr uint32_t kPrompt = 1u << kChunkMost, kBias = 2u << kChunkMost;
    auto entry_at = [&](int e) {
      Entry a{INT_MIN / 4, 0, 0.f, 0};
      const int o = e < listed ? sm.list[e] : 0, v = base + o;
      if (e >= listed || v >= V) return a;
      a.v = v;
      if (q.penal) {
        const int held = q.state[v];
        a.count = held & 0x7fff;
        if (held < 0) a.flags |= kPrompt;
        if ((sm.block[o >> 5] >> (o & 31)) & 1) {
          for (int s = 0; s < skip; ++s) a.count += p.tokens[q.first + s] == v;
          for (int t = 0; t < T_b; ++t) a.flags |= (uint32_t)(p.tokens[first + t] == v) << t;
        }
      }
      const int entry = biased ? s_bias[o] : 0;
      if (entry) {
        a.flags |= kBias;
        a.bias = p.bias_values[q.bias0 + entry - 1];
      }
      return a;
    };
    Entry first_entry, second_entry;
    if (listed > 0) first_entry = entry_at(lane);
    if (listed > 32) second_entry = entry_at(32 + lane);

    // --- a row of a block -----------------------------------------------------
    auto take_row = [&](Stage<T>& in, int block, int t) {
      constexpr bool kExact = sizeof(T) == 4;    // a processed logit has the logits' type
      const int g0 = first_of(block, t), v0 = g0 + lane * 8;
      const bool closed = (shut >> t) & 1, masked = words_of(t) != nullptr;
      const bool whole = !closed && !masked && !in.template at_end<kAligned>(g0, V);
      float* out = kOut ? p.out + (first + t) * p.out_stride : nullptr;
      T* values = reinterpret_cast<T*>(in.raw);
      // The special tokens, a lane's in ascending order. Their processed logits take
      // the logits' place; where those have fewer bits, -inf does, and the largest
      // of a lane's is kept beside it.
      // In the output of such a type a place is written after the dense pass; the
      // ones past 64 stay in that case and are done then.
      constexpr bool kLate = kOut && !kExact;
      uint32_t key = 0;
      int at = 0;
      auto special_token = [&](const Entry& a) {
        const int i = a.v - g0;
        if (i < 0 || i >= S::kBlock) return 0.f; // of another block
        float w = widen(values[i]);
        if (q.penal) {
          const int count = a.count + __popc(a.flags & ((2u << t) - 1));
          const bool seen = count > 0 || (a.flags & kPrompt);
          const float p1 = __fdiv_rn(w, q.r), p2 = __fmul_rn(w, q.r);
          w = seen ? (w > 0.f ? p1 : p2) : w;
          w = __fsub_rn(w, __fmul_rn(q.freq, (float)count));
          w = count > 0 ? __fsub_rn(w, q.pres) : w;
        }
        w = a.flags & kBias ? __fadd_rn(w, a.bias) : w;
        if constexpr (kExact) {
          values[i] = w;
        } else {
          if (!whole && (closed || !(in.template open<kAligned>(a.v, g0, V, masked) & 1))) w = -INFINITY;
          reinterpret_cast<uint16_t*>(values)[i] = (uint16_t)Octet<T>::kNone;
          const uint32_t k = w > -INFINITY ? ordered(w) : 0;     // a NaN is no candidate
          if (k > key) {
            key = k;
            at = a.v;
          }
        }
        return w;
      };
      float first_w = 0.f, second_w = 0.f;
      if (listed > 0) {
        first_w = special_token(first_entry);
        if (listed > 32) second_w = special_token(second_entry);
        if constexpr (!kLate) {
          // those of this block; a shifted row's second one begins a little earlier
          static_assert(S::kBlocks == 1 || S::kBlock == 512, "lane 16");
          const bool second = block % S::kBlocks != 0;
          const int e1 = S::kBlocks == 1 || second ? listed : below;
          for (int e0 = second ? max((below - S::kEarly) & ~31, 64) : 64; e0 < e1; e0 += 32)
            special_token(entry_at(e0 + lane));
        }
        __syncwarp();
      }
      const bool late = kLate && listed > 64;
      // the largest of the open ones
      uint32_t m = Octet<T>::kNone;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int v = v0 + n * 256;
        Octet<T> raw = in.raw[n * 32 + lane];
        if (!whole) raw.drop(closed ? 0 : in.template open<kAligned>(v, g0, V, masked));
        if constexpr (kOut) {
          float z[8];
          raw.unpack(z);
          if (v >= 0 && v <= V - 8 && (reinterpret_cast<uintptr_t>(out + v) & 15) == 0) {
            *reinterpret_cast<float4*>(out + v) = make_float4(z[0], z[1], z[2], z[3]);
            *reinterpret_cast<float4*>(out + v + 4) = make_float4(z[4], z[5], z[6], z[7]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (v + i >= 0 && v + i < V) out[v + i] = z[i];
          }
        }
        if (late) raw.drop(~special_bits(n, v0));
        m = raw.max(m);
      }
      const uint32_t dense = ordered(Octet<T>::value(m));
      if constexpr (kLate) {
        if (listed > 0) __syncwarp();            // the dense pass has written
        auto write = [&](int v, float w) {
          if (v >= g0 && v < g0 + S::kBlock) out[v] = w;
        };
        if (listed > 0) write(first_entry.v, first_w);
        if (listed > 32) write(second_entry.v, second_w);
        for (int e0 = 64; e0 < listed; e0 += 32) {
          const Entry a = entry_at(e0 + lane);
          write(a.v, special_token(a));
        }
        if (late) __syncwarp();                  // no special token has a value now
      }
      const uint32_t top = __reduce_max_sync(kAll, max(dense, key));
      // an equal value of an earlier block has the lower index
      const uint32_t held = __shfl_sync(kAll, (uint32_t)(best >> 32), t);
      if (top <= ordered(-INFINITY) || top <= held) return;
      // its place: the warp looks through the values of every lane that has it
      uint32_t place = UINT_MAX;
      if (!kExact && listed > 0) place = __reduce_min_sync(kAll, key == top ? (uint32_t)at : UINT_MAX);
      for (uint32_t has = __ballot_sync(kAll, dense == top); has; has &= has - 1) {
        const int i = (lane / 8 * 32 + __ffs(has) - 1) * 8 + lane % 8;
        bool found = lane < N * 8 && ordered(widen(values[lane < N * 8 ? i : 0])) == top;
        if (!whole) found = found && (in.template open<kAligned>(g0 + i, g0, V, masked) & 1);
        const uint32_t where = __ballot_sync(kAll, found);
        place = min(place, (uint32_t)__shfl_sync(kAll, g0 + i, __ffs(where) - 1));
      }
      if (lane == t) best = ((unsigned long long)top << 32) | (uint32_t)~place;
    };
    const int block1 = (seg + 1) * S::kBlocks;
    for (int block = seg * S::kBlocks; block < block1; ++block) {
      for (int t = 0; t < T_b; ++t) {
        copies_wait<kStages - 2>();
        __syncwarp();                            // every lane's copies, and the last row read
        copy_next();
        if (t + 1 == T_b && block + 1 == block1 && q.penal && seg + 1 < seg1) load_state(seg + 1);
        take_row(sm.ring[stage], block, t);
        stage = stage == kStages - 1 ? 0 : stage + 1;
      }
    }
    __syncwarp();
    if (biased)                                  // clean for the next segment
      for (int e = lane; e < listed; e += 32) s_bias[sm.list[e]] = 0;
    __syncwarp();
  }
  if (lane < T_b) p.part[(size_t)(first + lane) * p.runs + run] = best;
}

// One CTA a sequence, one warp a row: the largest key over the row's runs.
constexpr int kMergeThreads = 128;
__global__ void __launch_bounds__(kMergeThreads) choose_merge_kernel(TargetParams p) {
  grid_dependency_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  int first;
  const int T_b = rows_of(p, b, &first, false);
  for (int t = threadIdx.x >> 5; t < T_b; t += kMergeThreads / 32) {
    const unsigned long long* part = p.part + (size_t)(first + t) * p.runs;
    unsigned long long best = 0;
    for (int w = lane; w < p.runs; w += 32) best = part[w] > best ? part[w] : best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long y = __shfl_xor_sync(kAll, best, o);
      best = y > best ? y : best;
    }
    if (lane == 0) p.targets[first + t] = best ? (int32_t)~(uint32_t)best : -1;
  }
}

long long segments_for(int vocab, int dtype, bool aligned) {
  // a shifted row's grid begins early
  const int early = aligned ? 0 : dtype == SPLASH_F32 ? Segment<float>::kEarly : Segment<__half>::kEarly;
  constexpr int kTokens = Segment<float>::kTokens;
  return ((long long)vocab + early + kTokens - 1) / kTokens;
}

template <typename T, bool kOut, bool kAligned>
cudaError_t launch_choose(const TargetParams& p, cudaStream_t s) {
  const int smem = kWarpsPerCta * (int)(sizeof(WarpSmem<T>) +
                                        (p.bias_off ? Segment<T>::kBits * sizeof(int) : 0));
  const long long warps = (long long)p.num_seqs * p.chunks * p.runs;
  choose_kernel<T, kOut, kAligned>
      <<<(unsigned)((warps + kWarpsPerCta - 1) / kWarpsPerCta), 32 * kWarpsPerCta, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_choose(const TargetParams& p, bool aligned, cudaStream_t s) {
  static_assert(kWarpsPerCta * (sizeof(WarpSmem<T>) + Segment<T>::kBits * sizeof(int)) <= 48 * 1024,
                "shared memory");
  if (p.out) return aligned ? launch_choose<T, true, true>(p, s) : launch_choose<T, true, false>(p, s);
  return aligned ? launch_choose<T, false, true>(p, s) : launch_choose<T, false, false>(p, s);
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

// Counts the warp's tokens into row b of each lane (tok < 0: none). Equal tokens are
// counted once with their number; the 16-bit counter is moved by a compare-and-swap
// of its word, because it must stop at 32767. Sums of ones: the order changes nothing.
__device__ inline void count_tokens(const HistoryParams& p, int b, int tok) {
  const unsigned long long at = tok < 0 ? ~0ull : (unsigned long long)b * p.stride + tok;
  const uint32_t same = __match_any_sync(kAll, at);
  if (tok < 0 || (int)(threadIdx.x & 31) != __ffs(same) - 1) return;
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

// Adds the tokens to the rows in place, one token a thread, its sequence found by a
// search. That takes offsets in order; where some are not (their sequences are not
// usable, the others are), every sequence is asked whether it has the row.
constexpr int kSmemOffsets = 2048;
__global__ void __launch_bounds__(kThreads) history_add_kernel(HistoryParams p) {
  __shared__ int32_t s_off[kSmemOffsets + 1];
  const int i = blockIdx.x * kThreads + threadIdx.x;
  const int tok = i < p.num_tokens ? p.tokens[i] : -1;
  const int B = p.num_seqs;
  const bool in_smem = B <= kSmemOffsets;
  int lo, in_order = 1;
  if (in_smem && threadIdx.x == 0) s_off[0] = p.q_off[0];
#pragma unroll 4
  for (int c = threadIdx.x; c < B; c += kThreads) {
    const int first = p.q_off[c], next = p.q_off[c + 1];
    in_order &= first <= next;
    if (in_smem) s_off[c + 1] = next;
  }
  if (blockIdx.x == 0 && p.status)
    for (int c = threadIdx.x; c < B; c += kThreads) counted_end(p, c, &lo, true);
  in_order = __syncthreads_and(in_order);
  auto take = [&](int b) {           // b < 0: of no sequence; the whole warp calls it
    bool in = false;
    if (b >= 0 && tok >= 0 && tok < p.vocab) {
      const int end = counted_end(p, b, &lo, false);
      in = i >= lo && i < end;
    }
    count_tokens(p, b, in ? tok : -1);
  };
  if (in_order) {
    const int32_t* off = in_smem ? s_off : p.q_off;
    const int b = i >= off[0] && i < off[B] ? upper_index(off, B, i) : -1;
    take(b);
  } else {
#pragma unroll 1
    for (int b = 0; b < B; ++b) take(b);
  }
}

// Rebuilds the rows: a CTA takes a window of `span` entries of one row, counts
// the sequence's tokens in it in shared memory and writes the window whole, 16
// bytes at a time. Bound by the latency of one CTA's few steps: 16 sequences of 512
// to 32768 tokens, 131072 entries (5 MB) 5.2 us; with 160 windows instead of 144, so
// that 8 SMs take two in turn, 7.7 us. 32 registers (4 bytes spilled) let two CTAs share
// an SM: 256 sequences 32 us instead of 45.
__global__ void __launch_bounds__(1024, 2) history_reset_kernel(HistoryParams p, int span, int windows) {
  extern __shared__ __align__(16) int s_n[];
  const int b = blockIdx.x / windows, lo_v = blockIdx.x % windows * span;
  const int hi_v = (int)min((long long)lo_v + span, p.stride);
  int lo;
  const int end = counted_end(p, b, &lo, threadIdx.x == 0 && lo_v == 0);
  // span and the stride are multiples of 64
  for (int i = threadIdx.x; i < span / 4; i += blockDim.x)
    reinterpret_cast<int4*>(s_n)[i] = make_int4(0, 0, 0, 0);
  __syncthreads();
  const unsigned width = max(min(hi_v, p.vocab) - lo_v, 0);
  auto count = [&](int v) {
    if ((unsigned)v - (unsigned)lo_v < width) atomicAdd(&s_n[v - lo_v], 1);
  };
  // up to 3 tokens to the first 16-byte boundary, up to 3 behind the last one
  const int n = end - lo;
  const int32_t* tokens = p.tokens + lo;
  const int head = min((int)((0 - reinterpret_cast<uintptr_t>(tokens) / 4) & 3), n);
  const int quads = (n - head) / 4, tail = head + quads * 4;
  if ((int)threadIdx.x < head) count(tokens[threadIdx.x]);
  if ((int)threadIdx.x < n - tail) count(tokens[tail + threadIdx.x]);
  const int4* body = reinterpret_cast<const int4*>(tokens + head);
  constexpr int kAhead = 2;          // 16-byte loads in flight
  for (int i = threadIdx.x; i < quads; i += kAhead * 1024) {
    int4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      v[u] = i + u * 1024 < quads ? body[i + u * 1024] : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      count(v[u].x);
      count(v[u].y);
      count(v[u].z);
      count(v[u].w);
    }
  }
  __syncthreads();
  uint4* row = reinterpret_cast<uint4*>(p.state + (size_t)b * p.stride);
  auto pair = [&](int n0, int n1) {
    return p.prompt ? (n0 ? 0x8000u : 0u) | (n1 ? 0x80000000u : 0u)
                    : (uint32_t)min(n0, 32767) | (uint32_t)min(n1, 32767) << 16;
  };
  for (int i = threadIdx.x; i < (hi_v - lo_v) / 8; i += blockDim.x) {
    const int4 x = reinterpret_cast<const int4*>(s_n)[2 * i], y = reinterpret_cast<const int4*>(s_n)[2 * i + 1];
    row[lo_v / 8 + i] = make_uint4(pair(x.x, x.y), pair(x.z, x.w), pair(y.x, y.y), pair(y.z, y.w));
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
  // Runs are of 1024 tokens at least; shifted rows may have one more.
  return sizeof(unsigned long long) * (size_t)num_rows * (size_t)(vocab / 1024 + 2);
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

  const bool aligned = aligned16(logits) && logits_stride * es % 16 == 0;
  const long long segments = segments_for(vocab, dtype, aligned);
  // Fewer rows to a warp where 8 would leave more than a third of the GPU's warps
  // (20 to an SM) without work: 16 x 16 rows of 32000 logits 21 us at 8, 16 at 4, 18
  // at 2.
  // Chunks count only as far as there are rows.
  int chunk = kChunkMost;
  long long units = 0;
  for (;; chunk /= 2) {
    const long long by_block = num_seqs * (long long)((max_block_len + chunk - 1) / chunk);
    const long long by_rows = num_seqs + (long long)num_rows / chunk;
    units = by_block < by_rows ? by_block : by_rows;
    if (chunk == 1 || units * segments >= 12LL * sms) break;
  }
  const int chunks = (max_block_len + chunk - 1) / chunk;
  // A warp for each segment while that does not fill the GPU, then longer runs: a
  // run's first loads and last merge are shared by more tokens.
  long long span = units * segments / (kWarpsPerSm * sms);
  span = span < 1 ? 1 : span;
  const long long runs = (segments + span - 1) / span;
  if (runs * num_seqs > INT_MAX / (chunks + 1)) return SPLASH_ERR_UNSUPPORTED;
  if (workspace_bytes < sizeof(unsigned long long) * (size_t)num_rows * (size_t)runs)
    return SPLASH_ERR_WORKSPACE_TOO_SMALL;
  TargetParams p{logits, logits_stride, num_rows, vocab, q_offsets, num_seqs, max_block_len,
                 block_tokens, penal ? state : nullptr, state_stride, repetition, presence,
                 frequency, num_bias > 0 ? bias_offsets : nullptr, bias_ids, bias_values, num_bias,
                 mask, mask_stride, mask_rows, num_masks, out, out_stride, target_tokens,
                 static_cast<unsigned long long*>(workspace), (int)segments, (int)span, (int)runs,
                 chunk, chunks, device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == SPLASH_F32    ? launch_choose<float>(p, aligned, s)
                  : dtype == SPLASH_BF16 ? launch_choose<__nv_bfloat16>(p, aligned, s)
                                         : launch_choose<__half>(p, aligned, s);
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
  // Every window reads the sequence's tokens again: as many windows as SMs, in steps
  // of 64 entries.
  long long windows = num_seqs < sms ? sms / num_seqs : 1;
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
