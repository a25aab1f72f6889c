// Page tables and slot maps from the request lengths, and the way back of
// released pages. Integers only.
//
// Build. Sequence b holds held_b pages and is about to write positions
// ctx_b .. ctx_b + T_b - 1. It needs need_b = max(0, ceil((ctx_b + T_b)/16) -
// held_b) more pages (0 where T_b = 0). With incl_b = need_0 + .. + need_b, it
// gets them iff incl_b <= free pages: its i-th new page is
// free_pages[free - 1 - (incl_b - need_b + i)], the top of the stack first. The
// sequences that get pages are therefore a prefix of those that need some, and
// every place follows from one prefix sum: no atomics, the same result each
// time. Where the caller takes the served block lengths (T_b, or 0 for a sequence
// without slots), a second sum over them packs the rows. Release is the same sum
// over the pages that sequences give back.
//
// A first kernel of one CTA does the prefix sums (128 threads for up to 128
// sequences, 1024 above: fewer warps make its barriers cheaper, 128 sequences of 8
// rows 4.7 us, 129 of one row 9.7). The entries and the slot map are then one
// independent write each. Small calls write them in the same CTA; larger ones in a
// second kernel over the whole GPU, which starts under the first (programmatic
// dependent launch). What bounds both is latency, a chain of five or six dependent
// loads: a step of 64 sequences (449 slots) takes 5.4 us in one CTA; the admission of
// 1.96 million tokens (17 MB, 2.5 us at the measured copy rate) 2.1 us for the sums and
// 9 us for the fill; the release of 60,800 pages 2.0 and 2.9 us. Either is near or
// below the 10 us of host time that the call takes.
#include <climits>

#include "splash_common.cuh"
#include "splash_host.cuh"

namespace splash {

namespace {

constexpr int kScanSmall = 128, kScanLarge = 1024;
constexpr int kFillThreads = 256;
constexpr int kTokensPerThread = 4;
constexpr int kSmemSeqs = 2048;      // offsets kept in shared memory for the searches

struct TablesParams {
  const int32_t* ctx;
  const int32_t* T;
  int num_seqs;
  int num_tokens;
  int num_pages;
  int32_t* table;
  int max_pages;
  const int32_t* counts;       // may be counts_out
  int32_t* counts_out;
  const int32_t* free_pages;
  int free_cap;
  const int32_t* free_count;   // may be free_count_out
  int32_t* free_count_out;
  int32_t* q_off;              // [B + 1]
  int32_t* new_off;            // [B + 1]
  int32_t* positions;
  int32_t* slots;
  int32_t* served;             // [B], may be T, or nullptr: rows are packed by T
  int vec;                     // positions and slots are 16-byte aligned
  int* status;
};

struct ReleaseParams {
  const int32_t* keep;
  int num_seqs;
  const int32_t* table;
  int max_pages;
  const int32_t* counts;
  int32_t* counts_out;
  int32_t* free_pages;
  int free_cap;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* rel_off;            // [B + 1]
  int* status;
};

struct Sums {
  long long a, b;
};

// Inclusive scan of two sums over the CTA; *total gets the CTA's sums.
template <int N>
__device__ inline Sums block_inclusive(Sums v, Sums* s_warp, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v.a, o);
    const long long b = __shfl_up_sync(0xffffffffu, v.b, o);
    if (lane >= o) {
      v.a += a;
      v.b += b;
    }
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  Sums before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < N / 32; ++w) {
    const Sums x = s_warp[w];
    if (w < warp) {
      before.a += x.a;
      before.b += x.b;
    }
    all.a += x.a;
    all.b += x.b;
  }
  __syncthreads();
  *total = all;
  return Sums{before.a + v.a, before.b + v.b};
}

// Largest value over the CTA (values >= 0).
template <int N>
__device__ inline long long block_max(long long v, long long* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const long long y = __shfl_xor_sync(0xffffffffu, v, o);
    v = v > y ? v : y;
  }
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  long long r = 0;
#pragma unroll
  for (int w = 0; w < N / 32; ++w) r = s_warp[w] > r ? s_warp[w] : r;
  __syncthreads();
  return r;
}

__device__ inline long long pages_of(long long tokens) {
  return (tokens + kPageSize - 1) / kPageSize;
}

__device__ inline bool lengths_bad(int ctx, int T, int max_pages) {
  return T < 0 || ctx < 0 || (long long)ctx + T > (long long)max_pages * kPageSize;
}

// Such a sequence keeps its count as it is: cut to the table's width it would look
// like a valid one, whose entries are stale.
__device__ inline bool count_bad(int pages, int max_pages) { return pages < 0 || pages > max_pages; }

// Table entries and slots; thread `tid` of `threads` over the whole grid.
// q_off and new_off: the scan's sums [B + 1], in shared or global memory.
__device__ inline void fill_tables(const TablesParams& p, const int32_t* q_off,
                                   const int32_t* new_off, long long tid, long long threads) {
  const int B = p.num_seqs;
  const int taken = new_off[B], total = q_off[B];
  const int top = *p.free_count_out + taken;         // pages on the stack before the call
  // new table entries
  for (long long i = tid; i < taken; i += threads) {
    const int b = upper_index(new_off, B, (int)i);
    const int first = new_off[b], n = new_off[b + 1] - first;
    const int j = p.counts_out[b] - n + (int)(i - first);
    const int page = p.free_pages[top - 1 - (int)i];
    if (page < 0 || page >= p.num_pages) report(p.status, SPLASH_DEVICE_BAD_PAGE);
    p.table[(size_t)b * p.max_pages + j] = page;
  }
  // positions and slots, kTokensPerThread consecutive tokens a thread
  for (long long base = tid * kTokensPerThread; base < p.num_tokens;
       base += threads * kTokensPerThread) {
    int pos4[kTokensPerThread], slot4[kTokensPerThread];
    int b = 0, next = -1, first = 0, ctx = 0, held = 0, nfirst = 0;
    bool ok = false;
#pragma unroll
    for (int u = 0; u < kTokensPerThread; ++u) {
      pos4[u] = 0;
      slot4[u] = -1;
      const long long i = base + u;
      if (i >= p.num_tokens || i >= total) continue;
      if (i >= next) {           // the sequence that owns row i
        b = upper_index(q_off, B, (int)i);
        first = q_off[b];
        next = q_off[b + 1];
        ctx = p.ctx[b];
        const int T = p.T[b], have = p.counts_out[b];
        nfirst = new_off[b];
        held = have - (new_off[b + 1] - nfirst);
        ok = !lengths_bad(ctx, T, p.max_pages) && !count_bad(have, p.max_pages) &&
             (long long)first + T <= p.num_tokens && pages_of((long long)ctx + T) <= have;
      }
      if (!ok) continue;
      const int pos = ctx + (int)(i - first), j = pos / kPageSize;
      const int page = j < held ? p.table[(size_t)b * p.max_pages + j]
                                : p.free_pages[top - 1 - (nfirst + j - held)];
      if (page < 0 || page >= p.num_pages) {
        report(p.status, SPLASH_DEVICE_BAD_PAGE);
        continue;
      }
      pos4[u] = pos;
      slot4[u] = page * kPageSize + pos % kPageSize;
    }
    if (p.vec && base + kTokensPerThread <= p.num_tokens) {
      *reinterpret_cast<int4*>(p.positions + base) = make_int4(pos4[0], pos4[1], pos4[2], pos4[3]);
      *reinterpret_cast<int4*>(p.slots + base) = make_int4(slot4[0], slot4[1], slot4[2], slot4[3]);
    } else {
#pragma unroll
      for (int u = 0; u < kTokensPerThread; ++u) {
        if (base + u >= p.num_tokens) break;
        p.positions[base + u] = pos4[u];
        p.slots[base + u] = slot4[u];
      }
    }
  }
}

template <int N>
__global__ void __launch_bounds__(N) tables_scan_kernel(TablesParams p, int fill) {
  __shared__ Sums s_sums[N / 32];
  __shared__ long long s_max[N / 32];
  __shared__ int32_t s_off[kSmemSeqs + 1], s_new[kSmemSeqs + 1];
  allow_dependent_launch();
  const int tid = threadIdx.x, B = p.num_seqs;
  const int free_now = max(0, min(*p.free_count, p.free_cap));
  const bool in_smem = B <= kSmemSeqs;
  long long rows = 0, needed = 0, taken = 0;     // running sums before this chunk
  long long packed = 0;                          // rows of the served sequences
  for (int base = 0; base < B; base += N) {
    const int b = base + tid;
    int ctx = 0, T = 0, have = 0;
    bool bad = false;
    if (b < B) {
      ctx = p.ctx[b];
      T = p.T[b];
      have = p.counts[b];
      bad = lengths_bad(ctx, T, p.max_pages) || count_bad(have, p.max_pages);
      if (bad) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
      T = max(T, 0);
    }
    const long long want = bad || T == 0 ? 0 : pages_of((long long)ctx + T) - have;
    const long long need = want > 0 ? want : 0;
    Sums total, total_served;
    const Sums incl = block_inclusive<N>(Sums{T, need}, s_sums, &total);
    const long long row1 = rows + incl.a, need1 = needed + incl.b;
    const bool fits = row1 <= p.num_tokens;
    const bool given = fits && need1 <= free_now;
    if (b < B && !fits && T > 0) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
    if (b < B && fits && !given && need > 0) report(p.status, SPLASH_DEVICE_OUT_OF_PAGES);
    const long long here = block_max<N>(given ? need1 : 0, s_max);
    taken = here > taken ? here : taken;
    long long row0 = row1 - T;
    if (p.served) {                              // rows of the others have no place
      const int T_b = !bad && fits && (given || need == 0) ? T : 0;
      row0 = packed + block_inclusive<N>(Sums{T_b, 0}, s_sums, &total_served).a - T_b;
      packed += total_served.a;
      if (b < B) p.served[b] = T_b;
    }
    if (b < B) {
      const long long need0 = need1 - need;
      const int off = (int)(row0 < INT_MAX ? row0 : INT_MAX);
      p.q_off[b] = off;
      const int noff = (int)(need0 < taken ? need0 : taken);
      p.new_off[b] = noff;
      if (in_smem) {
        s_off[b] = off;
        s_new[b] = noff;
      }
      p.counts_out[b] = have + (given ? (int)need : 0);
    }
    rows += total.a;
    needed += total.b;
  }
  if (tid == 0) {
    const long long all = p.served ? packed : rows;
    const int off = (int)(all < INT_MAX ? all : INT_MAX);
    p.q_off[B] = off;
    p.new_off[B] = (int)taken;
    if (in_smem) {
      s_off[B] = off;
      s_new[B] = (int)taken;
    }
    *p.free_count_out = free_now - (int)taken;
  }
  if (!fill) return;
  __syncthreads();
  fill_tables(p, in_smem ? s_off : p.q_off, in_smem ? s_new : p.new_off, tid, N);
}

__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(TablesParams p) {
  __shared__ int32_t s_off[kSmemSeqs + 1], s_new[kSmemSeqs + 1];
  grid_dependency_wait();
  const bool in_smem = p.num_seqs <= kSmemSeqs;
  if (in_smem) {
    for (int i = threadIdx.x; i <= p.num_seqs; i += kFillThreads) {
      s_off[i] = p.q_off[i];
      s_new[i] = p.new_off[i];
    }
    __syncthreads();
  }
  fill_tables(p, in_smem ? s_off : p.q_off, in_smem ? s_new : p.new_off,
              (long long)blockIdx.x * kFillThreads + threadIdx.x,
              (long long)gridDim.x * kFillThreads);
}

// Released entries to the free list; thread `tid` of `threads` over the grid.
// rel_off: the scan's sums [B + 1], in shared or global memory.
__device__ inline void fill_released(const ReleaseParams& p, const int32_t* rel_off, long long tid,
                                     long long threads) {
  const int B = p.num_seqs;
  const int n = rel_off[B];
  const int before = *p.free_count_out - n;
  for (long long i = tid; i < n; i += threads) {
    const int b = upper_index(rel_off, B, (int)i);
    const int j = p.counts_out[b] + (int)(i - rel_off[b]);
    p.free_pages[before + i] = p.table[(size_t)b * p.max_pages + j];
  }
}

template <int N>
__global__ void __launch_bounds__(N) release_scan_kernel(ReleaseParams p, int fill) {
  __shared__ Sums s_sums[N / 32];
  __shared__ long long s_max[N / 32];
  __shared__ int32_t s_rel[kSmemSeqs + 1];
  allow_dependent_launch();
  const int tid = threadIdx.x, B = p.num_seqs;
  const int free_now = max(0, min(*p.free_count, p.free_cap));
  const bool in_smem = B <= kSmemSeqs;
  long long released = 0, moved = 0;
  for (int base = 0; base < B; base += N) {
    const int b = base + tid;
    int have = 0, left = 0;
    if (b < B) {
      have = p.counts[b];
      if (count_bad(have, p.max_pages)) {
        report(p.status, SPLASH_DEVICE_BAD_LENGTH);
        left = have;                                  // nothing given back
      } else {
        const int keep = p.keep[b];
        left = keep < 0 ? have : (int)min((long long)have, pages_of(keep));
      }
    }
    const long long n = have - left;
    Sums total;
    const long long n1 = released + block_inclusive<N>(Sums{n, 0}, s_sums, &total).a;
    const bool fits = free_now + n1 <= p.free_cap;
    if (b < B && !fits && n > 0) report(p.status, SPLASH_DEVICE_BAD_LENGTH);
    const long long here = block_max<N>(fits ? n1 : 0, s_max);
    moved = here > moved ? here : moved;
    if (b < B) {
      const long long n0 = n1 - n;
      const int off = (int)(n0 < moved ? n0 : moved);
      p.rel_off[b] = off;
      if (in_smem) s_rel[b] = off;
      p.counts_out[b] = fits ? left : have;
    }
    released += total.a;
  }
  if (tid == 0) {
    p.rel_off[B] = (int)moved;
    if (in_smem) s_rel[B] = (int)moved;
    *p.free_count_out = free_now + (int)moved;
  }
  if (!fill) return;
  __syncthreads();
  fill_released(p, in_smem ? s_rel : p.rel_off, tid, N);
}

__global__ void __launch_bounds__(kFillThreads) release_fill_kernel(ReleaseParams p) {
  __shared__ int32_t s_rel[kSmemSeqs + 1];
  grid_dependency_wait();
  const bool in_smem = p.num_seqs <= kSmemSeqs;
  if (in_smem) {
    for (int i = threadIdx.x; i <= p.num_seqs; i += kFillThreads) s_rel[i] = p.rel_off[i];
    __syncthreads();
  }
  fill_released(p, in_smem ? s_rel : p.rel_off, (long long)blockIdx.x * kFillThreads + threadIdx.x,
                (long long)gridDim.x * kFillThreads);
}

// Up to this many slots (build) or table entries (release) the scan's CTA writes them
// itself, more are a second kernel's. us, one CTA / two kernels:
//   128 threads  build 448 rows 4.7 / 5.8, 1024 rows 4.3 to 5.4 / 4.7 to 5.1, 1536 rows 6.6 to
//                7.0 / 4.9 to 5.4, 4096 rows 8.4 to 9.0 / 4.9 to 5.2; release of a quarter of 1024
//                entries 2.8 to 3.3 / 3.6 to 3.8, of 4096 5.5 / 3.7, of 16384 7.5 / 3.9
//   1024 threads build 512 rows 10.3 / 11.6, 2048 rows 8.3 to 9.6 / 9.3 to 10.8, 4096 rows 9.0 to
//                9.7 / 9.6 to 10.1, 8192 rows 11.2 / 9.8; release of a quarter of 4096 entries
//                5.8 / 6.9, of 16384 8.0 to 8.7 / 6.5 to 7.2
constexpr long long kFusedSmall = 1024, kFusedLarge = 4096;

bool one_cta(int num_seqs, long long items) {
  return items <= (num_seqs <= kScanSmall ? kFusedSmall : kFusedLarge);
}

bool lengths_args_ok(int num_seqs, int num_pages, int max_pages, int free_cap) {
  // a slot is page * 16 + offset in 32 bits; table places times 16 too
  return num_seqs >= 0 && num_pages >= 0 && num_pages <= INT_MAX / kPageSize && max_pages > 0 &&
         max_pages <= INT_MAX / kPageSize && free_cap >= 0;
}

}  // namespace
}  // namespace splash

using namespace splash;

static int build_tables(const int32_t* context_lens, const int32_t* block_lens, int num_seqs,
                        int num_tokens, int page_size, int num_pages, int32_t* page_table,
                        int max_pages_per_seq, const int32_t* page_counts,
                        int32_t* page_counts_out, const int32_t* free_pages, int free_capacity,
                        const int32_t* free_count, int32_t* free_count_out, int32_t* q_offsets,
                        int32_t* new_offsets, int32_t* positions, int32_t* slots,
                        int32_t* served_lens, int* device_status, struct CUstream_st* stream) {
  if (num_tokens < 0 || !lengths_args_ok(num_seqs, num_pages, max_pages_per_seq, free_capacity))
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (page_size != kPageSize) return SPLASH_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !q_offsets || !new_offsets ||
      (free_capacity > 0 && !free_pages) || (num_tokens > 0 && (!positions || !slots)) ||
      (num_seqs > 0 &&
       (!context_lens || !block_lens || !page_table || !page_counts || !page_counts_out)))
    return SPLASH_ERR_INVALID_ARGUMENT;
  TablesParams p{context_lens, block_lens, num_seqs, num_tokens, num_pages, page_table,
                 max_pages_per_seq, page_counts, page_counts_out, free_pages, free_capacity,
                 free_count, free_count_out, q_offsets, new_offsets, positions, slots, served_lens,
                 aligned16(positions) && aligned16(slots), device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int fused = one_cta(num_seqs, num_tokens);
  if (num_seqs <= kScanSmall)
    tables_scan_kernel<kScanSmall><<<1, kScanSmall, 0, s>>>(p, fused);
  else
    tables_scan_kernel<kScanLarge><<<1, kScanLarge, 0, s>>>(p, fused);
  if (counted(cudaGetLastError()) != cudaSuccess) return SPLASH_ERR_CUDA;
  if (fused) return SPLASH_OK;
  const long long per_cta = kFillThreads * kTokensPerThread;
  const long long want = (num_tokens + per_cta - 1) / per_cta;
  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  const int grid = (int)(want < 8LL * sms ? want : 8LL * sms);
  return counted(launch_dependent(tables_fill_kernel, dim3(grid), dim3(kFillThreads), 0, s, p)) ==
                 cudaSuccess
             ? SPLASH_OK
             : SPLASH_ERR_CUDA;
}

extern "C" {

int splash_build_tables(const int32_t* context_lens, const int32_t* block_lens, int num_seqs,
                        int num_tokens, int page_size, int num_pages, int32_t* page_table,
                        int max_pages_per_seq, const int32_t* page_counts,
                        int32_t* page_counts_out, const int32_t* free_pages, int free_capacity,
                        const int32_t* free_count, int32_t* free_count_out, int32_t* q_offsets,
                        int32_t* new_offsets, int32_t* positions, int32_t* slots,
                        int* device_status, struct CUstream_st* stream) {
  return build_tables(context_lens, block_lens, num_seqs, num_tokens, page_size, num_pages,
                      page_table, max_pages_per_seq, page_counts, page_counts_out, free_pages,
                      free_capacity, free_count, free_count_out, q_offsets, new_offsets, positions,
                      slots, nullptr, device_status, stream);
}

int splash_build_tables_served(const int32_t* context_lens, const int32_t* block_lens,
                               int num_seqs, int num_tokens, int page_size, int num_pages,
                               int32_t* page_table, int max_pages_per_seq,
                               const int32_t* page_counts, int32_t* page_counts_out,
                               const int32_t* free_pages, int free_capacity,
                               const int32_t* free_count, int32_t* free_count_out,
                               int32_t* q_offsets, int32_t* new_offsets, int32_t* positions,
                               int32_t* slots, int32_t* served_lens, int* device_status,
                               struct CUstream_st* stream) {
  if (num_seqs > 0 && !served_lens) return SPLASH_ERR_INVALID_ARGUMENT;
  return build_tables(context_lens, block_lens, num_seqs, num_tokens, page_size, num_pages,
                      page_table, max_pages_per_seq, page_counts, page_counts_out, free_pages,
                      free_capacity, free_count, free_count_out, q_offsets, new_offsets, positions,
                      slots, served_lens, device_status, stream);
}

int splash_release_pages(const int32_t* keep_lens, int num_seqs, const int32_t* page_table,
                         int max_pages_per_seq, int page_size, const int32_t* page_counts,
                         int32_t* page_counts_out, int32_t* free_pages, int free_capacity,
                         const int32_t* free_count, int32_t* free_count_out,
                         int32_t* released_offsets, int* device_status,
                         struct CUstream_st* stream) {
  if (!lengths_args_ok(num_seqs, 0, max_pages_per_seq, free_capacity))
    return SPLASH_ERR_INVALID_ARGUMENT;
  if (page_size != kPageSize) return SPLASH_ERR_UNSUPPORTED;
  if (!free_count || !free_count_out || !released_offsets || (free_capacity > 0 && !free_pages) ||
      (num_seqs > 0 && (!keep_lens || !page_table || !page_counts || !page_counts_out)))
    return SPLASH_ERR_INVALID_ARGUMENT;
  ReleaseParams p{keep_lens, num_seqs, page_table, max_pages_per_seq, page_counts,
                  page_counts_out, free_pages, free_capacity, free_count, free_count_out,
                  released_offsets, device_status};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long most = (long long)num_seqs * max_pages_per_seq;
  const int fused = one_cta(num_seqs, most);
  if (num_seqs <= kScanSmall)
    release_scan_kernel<kScanSmall><<<1, kScanSmall, 0, s>>>(p, fused);
  else
    release_scan_kernel<kScanLarge><<<1, kScanLarge, 0, s>>>(p, fused);
  if (counted(cudaGetLastError()) != cudaSuccess) return SPLASH_ERR_CUDA;
  if (fused) return SPLASH_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return SPLASH_ERR_CUDA;
  const long long want = (most + kFillThreads - 1) / kFillThreads;
  const int grid = (int)(want < 8LL * sms ? want : 8LL * sms);
  return counted(launch_dependent(release_fill_kernel, dim3(grid), dim3(kFillThreads), 0, s, p)) ==
                 cudaSuccess
             ? SPLASH_OK
             : SPLASH_ERR_CUDA;
}

}  // extern "C"
