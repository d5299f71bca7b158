/*
 * spec_kv.h -- C ABI of the paged KV cache beside the verification of
 * spec_verify.h (same library, libspecverify.so; gfx950).
 *
 * A speculative-decoding step appends k + 1 tokens per sequence to a paged
 * cache, attends from them over everything cached, verifies the drafts and
 * rolls the rejected ones back.  spec_verify.h does the last two; the calls
 * here do the first two:
 *
 *   kv_blocktable_extend   takes the blocks the new tokens need from a pool,
 *                          writes their ids into the block tables and gives
 *                          each token its slot (the counterpart of
 *                          kv_blocktable_truncate, whose freed blocks it takes
 *                          back into the pool);
 *   kv_cache_append        writes the tokens' keys and values to their slots;
 *   kv_paged_attention     softmax attention of the new tokens over the pages:
 *                          one token, a drafted window, a chunk of a prompt or
 *                          a whole prompt per sequence, in one batch.
 *
 * Conventions (ownership, asynchrony, status codes, spec_verify_last_error,
 * thread safety) are spec_verify.h's; status codes and the F32 and BF16
 * element types are its SV_* constants.  The calls launch on hip_stream; where
 * that stream is the null stream or a per-thread default stream, the current
 * device must be the one that holds the data.  Every call can be captured into
 * a HIP graph (kernels only: no memset, allocation or synchronisation).
 *
 * Cache layout.  k_cache and v_cache are [num_blocks, kv_heads, block_size,
 * head_dim], each block contiguous, consecutive blocks block_stride elements
 * apart (so that both may be views of one [num_blocks, 2, ...] allocation).
 * Slot s is row s % block_size of block s / block_size.  Token t of a sequence
 * lives at position t, in logical block t / block_size of its block table row.
 */
#ifndef SPEC_KV_H
#define SPEC_KV_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_KV_ABI_VERSION 1

#define SV_DTYPE_F16 2        /* float16, caches and attention only              */
#define SV_MAX_HEAD_DIM 256   /* head_dim of kv_paged_attention                  */
#define SV_MAX_ATTEND_BATCH 65536   /* sequences of kv_paged_attention; its work split
                                       costs every workgroup a pass over the batch
                                       (a tenth of the time at some 2000 sequences) */

int32_t spec_kv_abi_version(void);

/* Grows block tables by num_new tokens per sequence and maps the tokens to
 * slots (batch at most 2^24).  Sequence b holds L = seq_lens[b] tokens and gets
 * n = num_new[b] more, for which it needs ceil((L + n) / bs) - ceil(L / bs) blocks.
 *
 * The pool is a stack: free_blocks[0 .. *free_count), popped from its end.
 * First the blocks freed[b, 0 .. num_freed[b]) of every sequence in order
 * (freed_blocks / num_freed as kv_blocktable_truncate leaves them; a num_freed
 * of -1 adds none) are pushed.  Ids that free_capacity has no room for are
 * dropped, in no list from then on: free_count + the ids given back - the blocks
 * taken (num_taken) - free_left is how many; a stack with room for every block of
 * the cache drops none.  Then the sequences take theirs in order, ascending in
 * logical blocks.  When the pool runs short, the first sequence that it cannot
 * serve and every later one that needs a block get none.
 *
 *   block_table  [B, max_blocks] device int32, in/out: only new entries written
 *   seq_lens     [B]  device int32, read
 *   num_new      [B]  device int32, read: n >= 0
 *   free_blocks  [free_capacity] device int32, in/out: the stack
 *   free_count   [1]  device int32, read: ids in the stack before the call
 *   freed_blocks [B, max_freed] device int32 or NULL: ids to push
 *   num_freed    [B]  device int32 (required with freed_blocks)
 *   max_tokens   rows of the packed token arrays (the largest sum of num_new
 *                this call takes, 2^30 at most; a batch padded for a captured
 *                graph has more rows than tokens)
 *   new_lens     [B]  out: L + n, or L where the sequence was not served
 *   num_taken    [B]  out: blocks taken; -1: n < 0, L < 0, L + n beyond the
 *                table or beyond INT32_MAX, or tokens beyond max_tokens; -2:
 *                pool short.  Such a sequence's table and length stay as they
 *                were
 *   free_left    [1]  out: ids in the stack after the call
 *   cu_tokens    [B+1] out: sequence b's tokens are rows cu_tokens[b] ..
 *                cu_tokens[b+1]-1 (prefix sums of max(n, 0), served or not,
 *                limited to max_tokens)
 *   slot_map     [max_tokens] out int64: each token's slot; -1 for tokens of a
 *                sequence that was not served and for rows behind the last token
 *   positions    [max_tokens] out int32 or NULL: each token's position; -1 where
 *                slot_map is -1
 * new_lens may be seq_lens and free_left may be free_count (updated in place);
 * no other arrays may overlap.  Ids are not checked: the pool's are the
 * caller's.  Results do not depend on timing. */
int32_t kv_blocktable_extend(int32_t batch, int32_t max_blocks, int32_t block_size,
                             int32_t* block_table, const int32_t* seq_lens,
                             const int32_t* num_new, int32_t* free_blocks,
                             int32_t free_capacity, const int32_t* free_count,
                             const int32_t* freed_blocks, int32_t max_freed,
                             const int32_t* num_freed, int32_t max_tokens, int32_t* new_lens,
                             int32_t* num_taken, int32_t* free_left, int32_t* cu_tokens,
                             int64_t* slot_map, int32_t* positions, void* hip_stream);

typedef struct {
  int32_t tokens;         /* T >= 0 rows                                         */
  int32_t kv_heads;       /* >= 1                                                */
  int32_t head_dim;       /* >= 1                                                */
  int32_t block_size;     /* >= 1                                                */
  int32_t num_blocks;     /* >= 0; num_blocks * block_size < 2^31                */
  int32_t dtype;          /* SV_DTYPE_F32, _BF16 or _F16: rows and caches alike   */
  int64_t k_stride;       /* elements between token rows of k and of v; 0 =>     */
  int64_t v_stride;       /*   kv_heads * head_dim (heads contiguous in a row)    */
  int64_t block_stride;   /* elements between blocks of a cache; 0 =>            */
                          /*   kv_heads * block_size * head_dim                   */
} spec_kv_append_desc;

/* cache[slot / bs, h, slot % bs, :] = row[t, h, :] for both caches.  Rows whose
 * slot is negative or past the cache are skipped.  The slots of one call must
 * differ (kv_blocktable_extend's do): two rows sent to one slot leave a mixture
 * of both there.
 *   k, v        [T, kv_heads, head_dim] device, read-only, rows k_stride /
 *               v_stride elements apart (parts of a fused projection's rows)
 *   slot_map    [T] device int64
 * Rows and caches that lie on 16-byte boundaries are copied 16 bytes at a
 * time, others by the element (correct, at half the rate). */
int32_t kv_cache_append(const spec_kv_append_desc* desc, const void* k, const void* v,
                        const int64_t* slot_map, void* k_cache, void* v_cache,
                        void* hip_stream);

typedef struct {
  int32_t batch;          /* B in [0, SV_MAX_ATTEND_BATCH]                       */
  int32_t tokens;         /* T >= 0 query rows; T * heads < 2^31                 */
  int32_t heads;          /* query heads, a multiple of kv_heads                 */
  int32_t kv_heads;       /* >= 1; head h reads key head h / (heads / kv_heads)   */
  int32_t head_dim;       /* a multiple of 8 in [8, SV_MAX_HEAD_DIM]             */
  int32_t block_size;     /* >= 1                                                */
  int32_t num_blocks;     /* >= 0; num_blocks * block_size < 2^31                */
  int32_t max_blocks;     /* >= 0 columns of the block table                     */
  int32_t dtype;          /* SV_DTYPE_F32, _BF16 or _F16: q, caches and out alike */
  int32_t sliding_window; /* W > 0: a token sees itself and the W - 1 before it; 0: all */
  int32_t max_new;        /* the most new tokens of any sequence, 0 if unknown (the batch's
                             mean then): picks the tile shape, one for the call, and the
                             workspace's size, never the result's validity        */
  int32_t reserved;       /* must be 0                                           */
  int64_t q_stride;       /* elements between q's token rows; 0 => heads * head_dim */
  int64_t block_stride;   /* elements between blocks of a cache; 0 =>
                             kv_heads * block_size * head_dim                     */
  float scale;            /* of the scores, > 0, scale * log2(e) finite (often
                             head_dim^-0.5)                                       */
  float reserved_f;       /* must be 0                                           */
} spec_kv_attention_desc;

/* Workspace bytes of kv_paged_attention (partial results where a sequence's
 * keys are split over workgroups); 0 if the descriptor is invalid.  Depends on
 * the descriptor alone.  Pure host code. */
size_t kv_paged_attention_workspace_bytes(const spec_kv_attention_desc* desc);

/* Causal softmax attention of each sequence's last tokens over its pages.
 * Sequence b has n = cu_tokens[b+1] - cu_tokens[b] query rows, its last n of
 * seq_lens[b] tokens (their keys and values are in the cache already).  Row j
 * stands at position p = seq_lens[b] - n + j and sees the cached positions
 * max(0, p - W + 1) .. p (0 .. p without a window):
 *     out = sum_t softmax_t(scale * q . k_t) v_t,  lse = log sum_t exp(scale * q . k_t).
 * A row that sees no position (p < 0, or no page), or only scores of -inf, gets
 * out = 0 and lse = -inf.  Values at positions a row does not see never reach
 * it, whatever they hold (infinities and NaN included).
 *   q           [T, heads, head_dim] device, read-only, rows q_stride apart
 *   k_cache, v_cache  device, read-only (layout above)
 *   block_table [B, max_blocks] device int32; a block id outside [0, num_blocks)
 *               holds no positions (they are seen by no row), and neither do
 *               positions beyond the table
 *   seq_lens    [B] device int32 (with the new tokens)
 *   cu_tokens   [B+1] device int32, ascending within [0, T] (values outside are
 *               limited to it; where ranges overlap, which rows are written is
 *               undefined); rows before the first and behind the last sequence
 *               are left as they were
 *   out         [T, heads, head_dim] device
 *   lse         [T, heads] device float32 or NULL
 *   workspace   256-byte aligned, >= kv_paged_attention_workspace_bytes(desc);
 *               may be NULL if that is 0
 * q and the caches need 16-byte aligned pointers and strides (out: pointer).
 * Scores, softmax sums and the output are accumulated in float32; bf16 and f16
 * round the softmax weights to that type for the matrix cores (half a step of
 * the type relative to a weight; in f16 also up to 2^-32 of the largest weight
 * where that is more), not their sum.  The same call on the same data gives the
 * same bits. */
int32_t kv_paged_attention(const spec_kv_attention_desc* desc, const void* q,
                           const void* k_cache, const void* v_cache,
                           const int32_t* block_table, const int32_t* seq_lens,
                           const int32_t* cu_tokens, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV_H */
