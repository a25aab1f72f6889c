/*
 * splash_kv.h — C ABI of the int8 paged-KV verify-attention library (GB300, sm_103a).
 *
 * The operation. In-batch speculative decoding as the Splash engine describes it
 * ("Splash: 범용 엔진 대신 모델마다 커널과 초안 모델을 새로 만드는 Apple Silicon 추론
 * 엔진", discuss.pytorch.kr; section "옵션이 아니라 기본 경로인 DFlash 2 추측
 * 디코딩"): every sequence submits a block of T draft tokens that the target
 * model verifies in one forward pass, each sequence with its own T. Attention
 * state lives in a paged KV cache indexed by prefix, so sequences that share a
 * prefix share its pages (section "배치 스케줄링과 시작 시점에 확정되는 메모리
 * 예산"). The decode kernel reads the 8-bit KV cache directly and reuses each
 * KV tile across the query heads of a GQA group and across the verify tokens
 * (section "형상에 맞춰 자동으로 생성하는 Metal 커널"). The bnskd.com article
 * ("Splash：把推理引擎「围着模型造」…", section "技术内核") states the same.
 * The pages fix no quantisation scheme, layout, mask or precision; the ones
 * below are this library's readings.
 *
 * Conventions for every entry point
 *   - Pointers named *_pages, *_scales, q, out, lse, page_table, *_lens,
 *     k_new, v_new, workspace and device_status are DEVICE pointers owned by
 *     the caller. The library never allocates, frees or synchronises; all work
 *     is enqueued on `stream` (NULL = legacy default stream) and is async.
 *   - Return value: SPLASH_OK or a negative SPLASH_ERR_* code. Argument errors
 *     are detected on the host BEFORE anything is launched. A CUDA launch error
 *     returns SPLASH_ERR_CUDA (the CUDA error is left for cudaGetLastError).
 *   - Errors only visible on the device (a page id out of range or -1 where a
 *     page is needed, a length out of range) never trap: the kernel skips the
 *     affected work and, when device_status is non-NULL, stores the first such
 *     SPLASH_DEVICE_* code there (atomic compare-and-swap from 0). The caller
 *     zeroes *device_status before the call and reads it after the stream syncs.
 *
 * Shapes and layouts (row-major, innermost last)
 *   Hq = num_q_heads, Hkv = num_kv_heads, G = Hq / Hkv (query head hq uses KV
 *   head hq / G), D = head_dim in {64, 128, 256}, P = page_size = 16.
 *   codes            : int8  one pool [num_pages, Hkv, 2, P, D]; index 0 of the
 *                      third axis holds K codes, 1 holds V codes, so the K and V
 *                      codes of a (page, KV head) are one contiguous 2*P*D-byte
 *                      block. k_pages points at the pool, v_pages must equal
 *                      k_pages + P*D (anything else is SPLASH_ERR_INVALID_ARGUMENT).
 *                      v_pages is therefore fixed by k_pages: it carries no
 *                      information of its own, and separate K and V pools (the
 *                      layout of a two-pool cache) cannot be passed. The
 *                      interleaving lets one bulk copy move a (page, KV head)'s
 *                      K and V codes together; a copy's issue cost is mostly
 *                      per copy, and the same attention ran 6.8% faster than
 *                      with two pools of 4 KB copies at D = 256.
 *                      Slot s of (page, h): k_pages[((page*Hkv + h)*2*P + s)*D + d],
 *                      and the same offset from v_pages.
 *   k_scales, v_scales: fp32 [num_pages, Hkv, P]      one scale per (token, KV head)
 *   page_table       : int32 [num_seqs, max_pages_per_seq]; logical position j of
 *                      sequence b lives in page page_table[b][j / P], slot j % P.
 *                      Entries past a sequence's needed pages are ignored (-1 is
 *                      the customary sentinel). Pages may be shared between
 *                      sequences (shared prefix); they are read-only to attention.
 *   context_lens     : int32 [num_seqs] tokens cached before the block (ctx_b >= 0)
 *   block_lens       : int32 [num_seqs] verify-block length T_b >= 0 (0 = idle)
 *   Tokens of all blocks are packed by sequence: sequence b owns rows
 *   sum(block_lens[0..b-1]) .. + T_b - 1 of q / k_new / v_new / out / lse.
 */
#ifndef SPLASH_KV_H
#define SPLASH_KV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t */

enum {
  SPLASH_OK = 0,
  SPLASH_ERR_INVALID_ARGUMENT = -1,   /* null pointer, negative size, Hq % Hkv != 0 ... */
  SPLASH_ERR_UNSUPPORTED = -2,        /* D not in {64,128,256}, P != 16, T*G too large */
  SPLASH_ERR_WORKSPACE_TOO_SMALL = -3,
  SPLASH_ERR_CUDA = -4                /* a kernel launch failed */
};

enum {
  SPLASH_DEVICE_BAD_PAGE = 1,         /* page id < 0 or >= num_pages where a page is needed */
  SPLASH_DEVICE_BAD_LENGTH = 2,       /* ctx or T negative, T > max_block_len, or
                                         ctx + T > max_pages_per_seq * P, or
                                         sum(block_lens) > num_q_tokens */
  SPLASH_DEVICE_TIMEOUT = 3,          /* an internal wait of the tensor-core kernel gave
                                         up (after 1 s by default, see
                                         splash_set_wait_limit_ns); outputs of that
                                         call undefined */
  SPLASH_DEVICE_INTERNAL = 4,         /* the tensor-core kernel found its shared memory
                                         misaligned and did nothing */
  SPLASH_DEVICE_OUT_OF_PAGES = 5      /* the free list cannot serve every sequence
                                         (splash_build_tables) */
};

/* Element types of the entry points that take a dtype argument. */
enum { SPLASH_F32 = 0, SPLASH_BF16 = 1, SPLASH_F16 = 2 };

/* Human-readable name of a SPLASH_* status (static string, never NULL). */
const char* splash_status_string(int status);

/* Library ABI version (increments on any signature or layout change; 2 = the
 * interleaved K/V code pool). */
int splash_abi_version(void);

/* 1 if the tensor-core attention kernel is built for this head_dim, else 0
 * (units then run on the CUDA-core kernel). */
int splash_tensor_path_supported(int head_dim);

/* Number of kernels the library has enqueued since it was loaded (all entry
 * points, all threads; a host-side count of successful launches). Lets a
 * caller count the device work one call or one benchmark step issues. */
unsigned long long splash_launch_count(void);

/* Limit, in nanoseconds, of every internal pipeline wait of the tensor-core
 * attention kernel for the launches that follow (process-wide; 0 restores the
 * default of 1 s). When a wait runs out, the kernel stops the call's work,
 * lets the copies and MMAs it already issued complete, frees its tensor
 * memory, returns, and stores SPLASH_DEVICE_TIMEOUT in device_status; the
 * outputs of that call are undefined and later calls are unaffected. Meant
 * for tests of that path and for diagnosing a stalled GPU. Returns the
 * previous limit. */
unsigned long long splash_set_wait_limit_ns(unsigned long long ns);

/*
 * splash_kv_append — quantise a block of new K/V rows to int8 and write them
 * into the pages.
 *
 * For every sequence b and t < T_b, row r = sum(block_lens[0..b-1]) + t of
 * k_new / v_new (fp32 [num_new_tokens, Hkv, D]) is written at logical position
 * context_lens[b] + t, separately per KV head:
 *   a = max_d |x_d|;  s = fl32(a / 127);  c_d = clamp(rne(fl32(x_d / s)), -127, 127)
 *   (s == 0 gives all-zero codes), with correctly rounded fp32 division and
 *   round-half-to-even. Codes go to k_pages / v_pages, s to k_scales / v_scales.
 * num_new_tokens must equal sum(block_lens) (not checked on the host, which
 * cannot read device memory; rows past the sum are ignored). The target slots
 * must not be shared with another sequence (copy-on-write is the caller's).
 * Populating a cache uses the same call with context_lens = start positions.
 */
int splash_kv_append(const float* k_new, const float* v_new, int num_new_tokens,
                     int8_t* k_pages, int8_t* v_pages, float* k_scales, float* v_scales,
                     const int32_t* page_table, int max_pages_per_seq,
                     const int32_t* context_lens, const int32_t* block_lens, int num_seqs,
                     int num_kv_heads, int head_dim, int page_size, int num_pages,
                     int* device_status, struct CUstream_st* stream);

/*
 * splash_kv_append_bf16 — splash_kv_append for bf16 K/V rows (bit patterns,
 * [num_new_tokens, Hkv, D]), the dtype a projection usually produces. Each
 * value converts exactly to fp32, then the same quantiser applies; codes and
 * scales equal those of splash_kv_append on the fp32 copies of the same rows.
 */
int splash_kv_append_bf16(const uint16_t* k_new, const uint16_t* v_new, int num_new_tokens,
                          int8_t* k_pages, int8_t* v_pages, float* k_scales, float* v_scales,
                          const int32_t* page_table, int max_pages_per_seq,
                          const int32_t* context_lens, const int32_t* block_lens, int num_seqs,
                          int num_kv_heads, int head_dim, int page_size, int num_pages,
                          int* device_status, struct CUstream_st* stream);

/*
 * splash_accept_commit — the step after verification: each sequence advances
 * by the tokens it accepted (Splash article, section "옵션이 아니라 기본 경로인
 * DFlash 2 추측 디코딩": every request carries its own draft state and moves on
 * by its accepted tokens).
 *
 * block_tokens, target_tokens: int32 [num_tokens], packed by sequence like q.
 * Sequence b's block is x_0 .. x_{T_b-1} (x_0 = the token the target emitted at
 * the previous step, x_1.. = the draft's proposals); target_tokens holds the
 * target's next-token choice y_i after each x_i. Draft x_{i+1} is accepted
 * while x_{i+1} == y_i for all earlier i. With a accepted drafts:
 *   accepted[b] = a;  context_lens[b] += a + 1 (x_0 .. x_a are committed: their
 *   K/V were written by the block append);  next_tokens[b] = y_a.
 * Sequences with T_b = 0 get accepted = 0, next_tokens = -1 and keep their
 * length. Slots beyond the new length are overwritten by the next append.
 * context_lens is updated in place on the device; one small launch, no sync.
 */
int splash_accept_commit(const int32_t* block_tokens, const int32_t* target_tokens,
                         int num_tokens, const int32_t* block_lens, int32_t* context_lens,
                         int32_t* accepted, int32_t* next_tokens, int num_seqs,
                         int* device_status, struct CUstream_st* stream);

/*
 * splash_verify_attention_workspace_size — bytes of device workspace that
 * splash_verify_attention needs for these bounds on the current device
 * (depends on its SM count). Returns 0 for invalid arguments.
 */
size_t splash_verify_attention_workspace_size(int num_seqs, int num_q_tokens, int num_q_heads,
                                              int num_kv_heads, int head_dim, int max_block_len);

/*
 * splash_verify_attention — block-causal attention of every verify token over
 * its sequence's int8 paged cache (the block itself already appended).
 *
 * The target model checks a sequence's whole draft block in one forward pass
 * (Splash article on discuss.pytorch.kr, section "옵션이 아니라 기본 경로인
 * DFlash 2 추측 디코딩"); the kernel reads the 8-bit cache directly and serves
 * the G query heads of a KV head and the T verify tokens from each KV tile it
 * loads (section "형상에 맞춰 자동으로 생성하는 Metal 커널"). The mask that lets
 * verify token t see the block's tokens 0..t is this library's reading: the
 * pages do not state one.
 *
 * Verify token t of sequence b, query head hq (KV head h = hq / G) attends to
 * logical keys j = 0 .. context_lens[b] + t inclusive, dequantised as
 * code * scale:
 *   score_j = sm_scale * sum_d q[d] * k_hat_j[d]
 *   out     = sum_j softmax(score)_j * v_hat_j              -> bf16 (RNE)
 *   lse     = ln sum_j exp(score_j)   (sm_scale included)   -> fp32
 * q, out: bf16 bit patterns [num_q_tokens, Hq, D]; lse: fp32 [num_q_tokens, Hq].
 * num_q_tokens = sum(block_lens). max_block_len bounds every T_b (T_b * G must
 * be <= 128). sm_scale must be finite and > 0. The KV range of every
 * sequence is split across CTAs; partials
 * are merged by log-sum-exp in `workspace` (>= the size query's bytes, 256-byte
 * aligned). Deterministic: a fixed input, device and argument list gives
 * bitwise identical outputs, independent of the physical page numbering.
 */
int splash_verify_attention(const uint16_t* q, int num_q_tokens,
                            const int8_t* k_pages, const int8_t* v_pages,
                            const float* k_scales, const float* v_scales,
                            const int32_t* page_table, int max_pages_per_seq,
                            const int32_t* context_lens, const int32_t* block_lens, int num_seqs,
                            int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                            int num_pages, int max_block_len, float sm_scale,
                            uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                            int* device_status, struct CUstream_st* stream);

/*
 * splash_verify_attention_tuned — splash_verify_attention with the kernel
 * choice and the split granularity fixed by the caller (tests, benchmarks).
 *   path: 0 automatic; 1 CUDA-core kernel for every sequence; 2 tensor-core
 *         kernel for every sequence; 3 the transposed tensor-core kernel
 *         (S^T = K Q'^T: keys on the MMA's M side, no row padding) for every
 *         sequence, only at head_dim 256 with T * G <= 96
 *         (SPLASH_ERR_UNSUPPORTED otherwise). Path 3 exists for comparison:
 *         it is slower than path 2 on every workload measured.
 *   ctas_per_class: 0 automatic (fills the GPU); 0 < n <= 1023 uses n
 *         persistent CTAs per kernel (1 = every sequence's KV range handled
 *         unsplit); larger n is SPLASH_ERR_INVALID_ARGUMENT. The planner
 *         splits each kernel's stream of key tiles over its CTAs by estimated
 *         cost (a tile of a unit with more query rows costs more; every unit
 *         start adds one pipeline fill), from the lengths alone.
 * Same result contract as splash_verify_attention (within rounding across
 * different choices; bitwise for a fixed choice).
 */
int splash_verify_attention_tuned(const uint16_t* q, int num_q_tokens,
                                  const int8_t* k_pages, const int8_t* v_pages,
                                  const float* k_scales, const float* v_scales,
                                  const int32_t* page_table, int max_pages_per_seq,
                                  const int32_t* context_lens, const int32_t* block_lens,
                                  int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                  int page_size, int num_pages, int max_block_len, float sm_scale,
                                  uint16_t* out, float* lse, void* workspace,
                                  size_t workspace_bytes, int* device_status,
                                  struct CUstream_st* stream, int path, int ctas_per_class);

/*
 * splash_verify_attention_swa — splash_verify_attention_tuned with a sliding
 * window: verify token t of sequence b sees only the `window` most recent keys
 * up to its own position, context_lens[b] + t - window < j <= context_lens[b]
 * + t (the draft model's windowed attention, "옵션이 아니라 기본 경로인 DFlash 2
 * 추측 디코딩" section of the Splash article on discuss.pytorch.kr). window = 0
 * is the full mask of splash_verify_attention; window < 0 is an argument error.
 * Page-table entries of pages that lie wholly below key
 * context_lens[b] - window + 1 are never read (they may be -1). Same output,
 * workspace, determinism and error contract as splash_verify_attention.
 */
int splash_verify_attention_swa(const uint16_t* q, int num_q_tokens,
                                const int8_t* k_pages, const int8_t* v_pages,
                                const float* k_scales, const float* v_scales,
                                const int32_t* page_table, int max_pages_per_seq,
                                const int32_t* context_lens, const int32_t* block_lens,
                                int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                int page_size, int num_pages, int max_block_len, float sm_scale,
                                int window, uint16_t* out, float* lse, void* workspace,
                                size_t workspace_bytes, int* device_status,
                                struct CUstream_st* stream, int path, int ctas_per_class);

/*
 * splash_verify_attention_profiled — splash_verify_attention_tuned that also
 * records two caller-created CUDA events on `stream`: `attn_begin` just before
 * the attention kernel launch(es) and `attn_end` just after, so that the
 * attention kernels can be timed apart from the split planner and the
 * log-sum-exp combine. Either event may be NULL. Same work, same results.
 */
struct CUevent_st; /* cudaEvent_t */
int splash_verify_attention_profiled(const uint16_t* q, int num_q_tokens,
                                     const int8_t* k_pages, const int8_t* v_pages,
                                     const float* k_scales, const float* v_scales,
                                     const int32_t* page_table, int max_pages_per_seq,
                                     const int32_t* context_lens, const int32_t* block_lens,
                                     int num_seqs, int num_q_heads, int num_kv_heads,
                                     int head_dim, int page_size, int num_pages,
                                     int max_block_len, float sm_scale, uint16_t* out, float* lse,
                                     void* workspace, size_t workspace_bytes, int* device_status,
                                     struct CUstream_st* stream, int path, int ctas_per_class,
                                     struct CUevent_st* attn_begin, struct CUevent_st* attn_end);

/*
 * splash_verify_attention_shared — splash_verify_attention for a batch whose
 * sequences share prefix pages, reading each shared prefix tile once for the
 * stacked query rows of all sequences that share it.
 *
 * The Splash article on discuss.pytorch.kr indexes the paged KV cache by
 * prefix, so requests with a common prefix point at the same pages (section
 * "배치 스케줄링과 시작 시점에 확정되는 메모리 예산"), and it measures
 * concurrent agent requests that share a long prefix (section "동시 요청에서 더
 * 벌어지는 격차"). This entry point extends the reuse of one KV tile across the
 * query rows of a sequence to the rows of every sequence sharing the tile.
 *
 *   shared_lens: int32 [num_seqs] (device, non-NULL). shared_lens[b] > 0 states
 *     that logical keys 0 .. shared_lens[b] - 1 of sequence b sit in the same
 *     pages as those of sequence b - 1 (equal page-table entries); 0 states
 *     nothing; shared_lens[0] is ignored. The caller guarantees the claim.
 *     The library only clamps it to both sequences' context_lens: a claim
 *     whose pages differ gives sequence b the keys of sequence b - 1's pages.
 *
 * A run of consecutive sequences b0 .. b1, each linked to the one before it
 * by at least 64 keys, is a prefix group. Its common prefix is the smallest
 * link, cut to every member's context and down to a multiple of 64 keys. The
 * members' query rows (sum of T_b * G), stacked in sequence order, are cut
 * into blocks of 128 rows. Each block reads the common prefix through the
 * pages of b0's page-table row. Each member reads only its own keys after
 * the prefix. The log-sum-exp combine then merges the two partial results of
 * every row. A group is stacked only when it needs fewer blocks than it has
 * members (e.g. four sequences of T * G = 96 rows: 3 blocks instead of 4
 * passes over the prefix; four of 6 rows: 1 block).
 *
 * Output, result and error contract as splash_verify_attention. The result
 * equals splash_verify_attention's within rounding, since the same scores are
 * summed in a different split. Groups apply only on the tensor-core kernel
 * (path 0 or 2, head_dim 128 or 256), and on batches of at most 1024
 * sequences. Elsewhere the call computes the same result without stacking.
 * The workspace must hold splash_verify_attention_shared_workspace_size bytes
 * (more than splash_verify_attention's: every grouped row leaves two partial
 * rows). shared_lens == NULL is SPLASH_ERR_INVALID_ARGUMENT.
 */
size_t splash_verify_attention_shared_workspace_size(int num_seqs, int num_q_tokens,
                                                     int num_q_heads, int num_kv_heads,
                                                     int head_dim, int max_block_len);
int splash_verify_attention_shared(const uint16_t* q, int num_q_tokens,
                                   const int8_t* k_pages, const int8_t* v_pages,
                                   const float* k_scales, const float* v_scales,
                                   const int32_t* page_table, int max_pages_per_seq,
                                   const int32_t* context_lens, const int32_t* block_lens,
                                   const int32_t* shared_lens, int num_seqs, int num_q_heads,
                                   int num_kv_heads, int head_dim, int page_size, int num_pages,
                                   int max_block_len, float sm_scale, uint16_t* out, float* lse,
                                   void* workspace, size_t workspace_bytes, int* device_status,
                                   struct CUstream_st* stream);
/*
 * splash_verify_attention_shared_profiled — splash_verify_attention_shared
 * with path and ctas_per_class as in splash_verify_attention_tuned, and the
 * two events of splash_verify_attention_profiled (either may be NULL).
 */
int splash_verify_attention_shared_profiled(
    const uint16_t* q, int num_q_tokens, const int8_t* k_pages, const int8_t* v_pages,
    const float* k_scales, const float* v_scales, const int32_t* page_table,
    int max_pages_per_seq, const int32_t* context_lens, const int32_t* block_lens,
    const int32_t* shared_lens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int page_size, int num_pages, int max_block_len, float sm_scale, uint16_t* out, float* lse,
    void* workspace, size_t workspace_bytes, int* device_status, struct CUstream_st* stream,
    int path, int ctas_per_class, struct CUevent_st* attn_begin, struct CUevent_st* attn_end);

/*
 * splash_verify_attention_fixed_scratch — splash_verify_attention without a
 * caller-provided workspace, for callers that cannot allocate device memory:
 * for example code that runs under a memory manager owning every device
 * allocation, a plugin whose host forbids allocation calls, or a serving
 * loop that cannot afford the implicit device synchronisation of cudaMalloc.
 * (The source pages describe nothing like it; it is a packaging of the same
 * operation.)
 *
 * The workspace is instead a fixed 64 MiB array (see
 * splash_verify_attention_fixed_scratch_bytes) that is part of this library's
 * device image: every GPU that loads the library holds it until the process
 * exits. Nothing is allocated or freed by the call; no allocating library
 * routine is used. The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress), so make that first call before any stream
 * capture. All calls on a device share the one array, which keeps the last
 * call's contents; the planner rewrites everything a call reads, so nothing
 * needs clearing between calls. Calls that can overlap on the same GPU (issued
 * on different streams, or from different host threads) race on the array and
 * must be serialised by the caller.
 *
 * Same arguments, results and errors as splash_verify_attention minus the
 * workspace, with one CTA per SM for each attention kernel. Returns
 * SPLASH_ERR_WORKSPACE_TOO_SMALL when the shape needs more scratch than the
 * fixed array holds (for D = 256 that is beyond about T*G = 105 rows per
 * sequence on a 152-SM GB300).
 */
size_t splash_verify_attention_fixed_scratch_bytes(void);
int splash_verify_attention_fixed_scratch(const uint16_t* q, int num_q_tokens,
                                          const int8_t* k_pages, const int8_t* v_pages,
                                          const float* k_scales, const float* v_scales,
                                          const int32_t* page_table, int max_pages_per_seq,
                                          const int32_t* context_lens, const int32_t* block_lens,
                                          int num_seqs, int num_q_heads, int num_kv_heads,
                                          int head_dim, int page_size, int num_pages,
                                          int max_block_len, float sm_scale, uint16_t* out,
                                          float* lse, int* device_status,
                                          struct CUstream_st* stream);

/* ------------------------------------------------------------------------
 * The rest of a verify step. Page tables and slot maps, the projections'
 * norm, rotation and append, and the target's choices, so that a step's
 * lengths, pages and tokens stay on the device:
 *   splash_build_tables_served -> splash_qkv_append -> splash_verify_attention
 *   -> (the model's output head) -> splash_choose_targets
 *   -> splash_accept_commit -> splash_token_state_add
 * These are this library's own: the Splash pages describe none of them. All
 * are enqueued on `stream`, allocate nothing and can be captured in a graph.
 * ------------------------------------------------------------------------ */

/*
 * splash_build_tables — give every sequence the pages that its block needs and
 * map the block's tokens to cache slots.
 *
 * Sequence b holds its first page_counts[b] page-table entries. With T_b > 0 it
 * needs ceil((context_lens[b] + T_b) / P) of them. The missing ones come off
 * the top of the stack free_pages[0 .. *free_count - 1] in sequence order: with
 * need_b missing pages and incl_b = need_0 + .. + need_b, sequence b is served
 * iff incl_b <= *free_count, all of its pages or none; its i-th new page is
 * free_pages[*free_count - 1 - (incl_b - need_b) - i]. Not served: its tokens
 * get no slots, SPLASH_DEVICE_OUT_OF_PAGES is reported. Page-table entries
 * below page_counts[b] and past the new ones are not written.
 *   page_counts_out [num_seqs], free_count_out [1]: the counts after the call;
 *     each may be its input (in place).
 *   q_offsets [num_seqs + 1]: exclusive prefix of max(block_lens, 0).
 *   new_offsets [num_seqs + 1]: exclusive prefix of the pages handed out;
 *     sequence b's new entries are the last new_offsets[b+1] - new_offsets[b]
 *     of its page_counts_out[b].
 *   positions, slots [num_tokens]: position context_lens[b] + t and slot
 *     page * P + position % P of row q_offsets[b] + t. Rows without a slot (of
 *     a sequence that is not served or whose lengths are out of range, and the
 *     rows past the last sequence of a padded batch) get slot -1, position 0.
 * A length or page count out of range or a sequence whose rows pass num_tokens
 * reports SPLASH_DEVICE_BAD_LENGTH, gets no pages and no slots and keeps its page
 * count; the others keep their rows. A page id outside [0, num_pages) reports
 * SPLASH_DEVICE_BAD_PAGE and maps no slot. *free_count is cut to
 * [0, free_capacity]. num_pages * P must fit 32 bits. Page numbers only: no pool
 * is touched.
 *
 * A sequence without slots must not be attended and committed: its block is not
 * in the cache. splash_build_tables leaves it to the caller to take such
 * sequences out of block_lens (after a read of device_status).
 * splash_build_tables_served does it on the device: the same decisions, and
 *   served_lens [num_seqs] (may be block_lens): T_b of a sequence whose block has
 *     its pages, 0 of the others. q_offsets is the exclusive prefix of served_lens,
 *     and positions and slots are packed by it (a sequence without slots has no
 *     rows).
 * With served_lens for block_lens in the calls that follow, and tokens packed by
 * q_offsets, every other sequence is idle in the step: not attended, its context
 * length and token history as they were, accepted = 0, next_tokens = -1. It may
 * submit the same block again. (A bad page id is reported and leaves its sequence
 * served.)
 */
int splash_build_tables(const int32_t* context_lens, const int32_t* block_lens, int num_seqs,
                        int num_tokens, int page_size, int num_pages, int32_t* page_table,
                        int max_pages_per_seq, const int32_t* page_counts,
                        int32_t* page_counts_out, const int32_t* free_pages, int free_capacity,
                        const int32_t* free_count, int32_t* free_count_out, int32_t* q_offsets,
                        int32_t* new_offsets, int32_t* positions, int32_t* slots,
                        int* device_status, struct CUstream_st* stream);
int splash_build_tables_served(const int32_t* context_lens, const int32_t* block_lens,
                               int num_seqs, int num_tokens, int page_size, int num_pages,
                               int32_t* page_table, int max_pages_per_seq,
                               const int32_t* page_counts, int32_t* page_counts_out,
                               const int32_t* free_pages, int free_capacity,
                               const int32_t* free_count, int32_t* free_count_out,
                               int32_t* q_offsets, int32_t* new_offsets, int32_t* positions,
                               int32_t* slots, int32_t* served_lens, int* device_status,
                               struct CUstream_st* stream);

/*
 * splash_release_pages — put the pages past ceil(keep_lens[b] / P) of every
 * sequence back on the free list (keep_lens[b] = 0: a finished sequence; its
 * committed length: the pages of rejected drafts; negative: nothing).
 *
 * The entries go behind free_pages[*free_count - 1] in sequence and position
 * order. page_counts_out and free_count_out may be their inputs.
 * released_offsets [num_seqs + 1]: exclusive prefix of the pages given back. A
 * sequence whose pages do not fit free_capacity keeps them, and so does every
 * later one that gives some back (SPLASH_DEVICE_BAD_LENGTH); one whose page
 * count is out of range gives back nothing and keeps its count (the same code).
 * The page table is only read: entries past page_counts_out[b] are stale. A page
 * that sequences share is given back once per sequence that holds it, so shared
 * prefixes stay inside keep_lens of all but one.
 */
int splash_release_pages(const int32_t* keep_lens, int num_seqs, const int32_t* page_table,
                         int max_pages_per_seq, int page_size, const int32_t* page_counts,
                         int32_t* page_counts_out, int32_t* free_pages, int free_capacity,
                         const int32_t* free_count, int32_t* free_count_out,
                         int32_t* released_offsets, int* device_status,
                         struct CUstream_st* stream);

/*
 * splash_qkv_append — norm and rotate the q and k heads of new tokens, write q
 * for splash_verify_attention and quantise k and v into the cache, in one pass.
 *
 * q, k, v: `dtype` (SPLASH_F32 or SPLASH_BF16) [num_tokens, heads, D] with the
 * given token and head strides in elements (a packed projection is three views
 * of one buffer). Row, weight and pool pointers must be 16-byte aligned and
 * strides whole multiples of 16 bytes. Per row x of D values, everything in fp32:
 *   q, k: x_d * w_d / sqrt(mean(x^2) + eps), with q_weight / k_weight fp32 [D];
 *         NULL leaves that one un-normed
 *   q, k: with R = rotary_dim (a multiple of 16, 0 for none) the first R values
 *         are turned in pairs (u, v) = (x_i, x_{i+R/2}), or (x_2i, x_2i+1) when
 *         `interleaved`, i < R/2, by angle a = position * inv_freq[i]:
 *         u' = (u cos a - v sin a) * rope_scale, v' = (v cos a + u sin a) * rope_scale.
 *         inv_freq: fp32 [R/2]. positions: int32 [num_axes, num_tokens];
 *         frequency i uses axis freq_axis[i] (int32 [R/2], cut to the axes
 *         there are; NULL: axis 0). At any 32-bit position an angle is cut to a
 *         multiple of 2^-32 of a turn and rounded once to fp32.
 *   q:    rounded to bf16 into q_out [num_tokens, Hq, D] (contiguous; may be q
 *         itself when q is contiguous bf16)
 *   k, v: splash_kv_append's quantiser, into slot slots[row] (page * P +
 *         offset, as splash_build_tables writes them)
 * A row with a negative slot is skipped: nothing of it is written, q_out
 * included. A slot past the pool reports SPLASH_DEVICE_BAD_PAGE and is skipped.
 * Slots must differ. sum(x^2) must stay finite in fp32 where a norm is taken.
 */
int splash_qkv_append(const void* q, const void* k, const void* v, int dtype, int num_tokens,
                      long long q_stride, long long q_head_stride, long long k_stride,
                      long long k_head_stride, long long v_stride, long long v_head_stride,
                      int num_q_heads, int num_kv_heads, int head_dim, const float* q_weight,
                      const float* k_weight, float eps, const float* inv_freq,
                      const int32_t* freq_axis, int rotary_dim, int interleaved, float rope_scale,
                      const int32_t* positions, int num_axes, const int32_t* slots,
                      uint16_t* q_out, int8_t* k_pages, int8_t* v_pages, float* k_scales,
                      float* v_scales, int page_size, int num_pages, int* device_status,
                      struct CUstream_st* stream);

/*
 * splash_kv_gather — cached rows by slot, dequantised: row i of k_out / v_out
 * (dtype SPLASH_F32 or SPLASH_BF16, contiguous [num_rows, Hkv, D]) is
 * the fp32 product code * scale of slots[i], rounded to dtype. With the slots of
 * splash_build_tables this hands cached context to a dense attention. Rows with
 * a negative slot are left as they were, a slot past the pool too
 * (SPLASH_DEVICE_BAD_PAGE). A slot may appear more than once.
 */
int splash_kv_gather(const int8_t* k_pages, const int8_t* v_pages, const float* k_scales,
                     const float* v_scales, const int32_t* slots, int num_rows, int num_kv_heads,
                     int head_dim, int page_size, int num_pages, void* k_out, void* v_out,
                     int dtype, int* device_status, struct CUstream_st* stream);

/*
 * Token history of the penalties: int16 [num_seqs, stride] with stride =
 * splash_token_state_stride(vocab) (the vocabulary rounded up to 64; 0 for a
 * vocabulary out of range). Bit 15 of entry v: v occurs in the sequence's
 * prompt. Bits 0..14: how often it occurs in its committed output, held at
 * 32767.
 *
 * splash_token_state_add — count tokens into it: rows q_offsets[b] ..
 * q_offsets[b+1] - 1 of `tokens` belong to sequence b; with `accepted` non-NULL
 * only the first accepted[b] + 1 of them (what splash_accept_commit commits,
 * called before or after it). prompt != 0 sets bit 15 instead of counting.
 * reset != 0 clears every sequence's row first, whole (a call over the rows of
 * newly admitted sequences). Tokens outside [0, vocab) are passed over. A
 * sequence with unusable offsets reports SPLASH_DEVICE_BAD_LENGTH and has no
 * tokens; the others are counted.
 * `state` is 16-byte aligned, state_stride a multiple of 64.
 */
int splash_token_state_stride(int vocab);
int splash_token_state_add(const int32_t* tokens, int num_tokens, const int32_t* q_offsets,
                           int num_seqs, const int32_t* accepted, int16_t* state,
                           long long state_stride, int vocab, int prompt, int reset,
                           int* device_status, struct CUstream_st* stream);

/*
 * splash_choose_targets — the target's choice after every verify token, from
 * its logits under repetition, presence and frequency penalties, biases and
 * grammar masks; what splash_accept_commit takes as target_tokens.
 *
 * logits: `dtype` (F32, BF16 or F16) [num_rows, >= vocab], row stride
 * logits_stride elements. Rows q_offsets[b] .. q_offsets[b+1] - 1 are sequence
 * b's verify rows (at most max_block_len <= 128 of them). For row t and token v,
 * each step rounded to fp32, a NULL array leaving its step out:
 *   c    = output count of v in `state` + occurrences of v among the block's
 *          own tokens x_0 .. x_t (block_tokens), which are not committed yet
 *   seen = c > 0, or v is in the prompt
 *   z1 = seen ? (z > 0 ? z / repetition[b] : z * repetition[b]) : z
 *   z2 = z1 - frequency[b] * c
 *   z3 = c > 0 ? z2 - presence[b] : z2
 *   z4 = z3 + bias of v: entries bias_offsets[b] .. bias_offsets[b+1] - 1 of
 *        bias_ids / bias_values (num_bias in all); of entries with the same id
 *        the last counts; ids outside the vocabulary are passed over
 *   z5 = z4 where bit v % 32 of word v / 32 of the row's mask is 1, else -inf.
 *        mask: int32 [num_masks, mask_stride words]. Row i uses mask
 *        mask_rows[i] (-1: no mask), or mask i when mask_rows is NULL. An index
 *        past num_masks allows nothing (SPLASH_DEVICE_BAD_LENGTH).
 * repetition values must be > 0 and finite (others count as 1), frequency and
 * presence finite.
 * target_tokens[i]: the lowest v with the largest z5 above -inf; -1 where there
 * is none (splash_accept_commit then hands it on as next token). NaN is never
 * chosen.
 * out (NULL: not written): fp32 z5 [num_rows, vocab], row stride out_stride; may
 * be the logits themselves (F32, same stride).
 * Rows of no sequence, and of sequences with unusable offsets
 * (SPLASH_DEVICE_BAD_LENGTH), are left as they were. A row that two sequences
 * claim (offsets out of order) gets unspecified results. The workspace (256-byte
 * aligned) is scratch for the duration of the call.
 */
size_t splash_choose_targets_workspace_size(int num_rows, int vocab);
int splash_choose_targets(const void* logits, int dtype, long long logits_stride, int num_rows,
                          int vocab, const int32_t* q_offsets, int num_seqs, int max_block_len,
                          const int32_t* block_tokens, const int16_t* state,
                          long long state_stride, const float* repetition, const float* presence,
                          const float* frequency, const int32_t* bias_offsets,
                          const int32_t* bias_ids, const float* bias_values, int num_bias,
                          const int32_t* mask, long long mask_stride, int num_masks,
                          const int32_t* mask_rows, float* out, long long out_stride,
                          int32_t* target_tokens, void* workspace, size_t workspace_bytes,
                          int* device_status, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLASH_KV_H */
