/*
 * pkv.h — C ABI of libpkv: attention over a paged KV cache on GB300 (sm_103a).
 *
 * The method: a sequence's K/V rows live in fixed-size physical blocks of one pool
 * tensor, found through a per-sequence block table (logical block -> physical block),
 * as in "Lecture 33 — KV Cache management: PagedAttention, Continuous Batching,
 * Chunked Prefill", §2.2; attention kernels read the blocks in place (§2.3); shared
 * blocks are split by copy-on-write (§2.4); a prefill chunk attends its cached
 * history causally (§4.2).  The host block manager follows "PagedAttention: manage
 * the KV cache like virtual memory", §3.2–§3.3.
 *
 * Conventions for every device call below
 *   - Pointers marked (device) are device pointers owned by the caller; the library
 *     never allocates, frees or retains them.  All tensors are dense, row-major, with
 *     the layouts given per argument, and 16-byte aligned.
 *   - Work is enqueued asynchronously on `stream` (NULL = legacy default stream).
 *     Argument checks run on the host before anything is enqueued; a failed check
 *     returns PKV_ERR_INVALID_ARG / PKV_ERR_UNSUPPORTED and enqueues nothing.
 *     A launch failure returns PKV_ERR_CUDA.
 *   - Data-dependent faults the host cannot see (a block id outside the pool, a slot
 *     outside the pool, a context_len beyond the block table, a copy pair that chains)
 *     never fault the GPU: the kernel skips the access and sets a bit in the library's
 *     device error word, read with pkv_get_device_error().
 *   - No call aborts, traps, prints or spins without bound.
 *
 * KV cache layout (both K and V): [num_blocks][num_kv_heads][block_size][head_dim]
 * of kv_dtype.  Slot s addresses token row s % block_size of physical block
 * s / block_size (Lecture 33 §2.2: base + block * block_stride + offset * token_stride).
 *
 * 4-bit KV cache (kv_dtype PKV_FP4_E2M1): [num_blocks][num_kv_heads][block_size / 16][tile], a
 * tile being 16 rows in 9 * head_dim bytes.  First the codes, [16][head_dim / 2] bytes: element
 * 2j of a row is the low nibble of its byte j, element 2j + 1 the high one.  Then the scales,
 * [16][head_dim / 16] bytes: one e4m3 scale for every 16 elements of a row.  An element's value
 * is code * scale of its 16 * k_scale[kv_head] (v_scale for V); code * scale is exact in fp16.
 * head_dim and block_size are multiples of 16.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* pkv_stream_t;

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,   /* a host-visible argument is out of range / misaligned */
  PKV_ERR_UNSUPPORTED = 2,   /* valid, but the library has no kernel for it (e.g. head_dim 96) */
  PKV_ERR_WORKSPACE = 3,     /* workspace missing or smaller than pkv_decode_workspace_bytes() */
  PKV_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed */
  PKV_ERR_NO_BLOCKS = 5,     /* block manager: the free-block queue cannot cover the request */
  PKV_ERR_DEVICE_CHECK = 6   /* pkv_get_device_error() found a device-side check bit set */
} pkv_status;

typedef enum {
  PKV_F16 = 0,
  PKV_BF16 = 1,
  PKV_FP8_E4M3 = 2,          /* e4m3 "fn": bias 7, max 448, no inf; value = code * scale[kv_head] */
  PKV_FP4_E2M1 = 3           /* caches only: e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives), one e4m3
                                scale per 16 elements, and scale[kv_head]; layout above */
} pkv_dtype;

/* Device error word bits (pkv_get_device_error). */
enum {
  PKV_DEVERR_BLOCK_ID = 1u << 0,      /* a block table entry was outside [0, num_blocks) */
  PKV_DEVERR_CONTEXT_LEN = 1u << 1,   /* context_len < 0, > max_blocks_per_seq * block_size or > max_context_len */
  PKV_DEVERR_SLOT = 1u << 2,          /* a slot was >= num_blocks * block_size */
  PKV_DEVERR_COPY_PAIR = 1u << 3,     /* a copy pair was out of range or its dst is also a src */
  PKV_DEVERR_TIMEOUT = 1u << 4,       /* a bounded wait on an async copy / MMA gave up */
  PKV_DEVERR_CHUNK = 1u << 5          /* cu_q_lens, cu_k_lens, cu_lens or q_start_pos were inconsistent */
};

/* The paged pool (Lecture 33 §2.2, "physical KV block pool"): K and V are two such tensors. */
typedef struct {
  int num_blocks;            /* physical blocks in the pool */
  int num_kv_heads;
  int block_size;            /* tokens per block: 16, or 32 (the attention kernels read it as two 16-row tiles) */
  int head_dim;              /* 64 or 128 */
  pkv_dtype kv_dtype;
  const float* k_scale;      /* (device) [num_kv_heads] fp32, e4m3 caches; 4-bit caches: may be NULL (1); else NULL */
  const float* v_scale;      /* (device) [num_kv_heads] fp32, e4m3 caches; 4-bit caches: may be NULL (1); else NULL */
} pkv_cache_desc;

PKV_API const char* pkv_status_string(pkv_status s);
PKV_API int pkv_version(void);       /* (major << 16) | minor */

/*
 * kv_write ("reshape_and_cache").  "PagedAttention: manage the KV cache like virtual
 * memory" §3.3: each new token fills its sequence's current last block; Lecture 33
 * §4.2: a prefill chunk's K/V is written into the cache too.
 *   k_new, v_new   (device) [num_tokens][num_kv_heads][head_dim] of in_dtype
 *   slot_mapping   (device) int64 [num_tokens]; slot < 0 = padding token, skipped
 *   k_cache/v_cache (device) pool tensors described by `cache`
 * For every token t with slot s >= 0 and every kv head h:
 *   k_cache[s / B][h][s % B][:] = k_new[t][h][:]   (same for V)
 * in_dtype == kv_dtype copies bytes.  in_dtype f16/bf16 into an e4m3 cache quantises
 * x / scale[h] (fp32 divide) to e4m3, round-to-nearest-even, saturating at ±448.
 * f16/bf16 into a 4-bit cache quantises each 16 elements of a row together: with u = x / scale[h]
 * (fp32 divide; u = x without scales), s = max|u| / 6 (fp32 divide) rounded to e4m3 (to nearest
 * even, at least 2^-9, at most 448) and code = u / s rounded to e2m1 (to nearest even, saturating
 * at +-6).  A NaN among the 16 makes s NaN and so all 16 values.  Rows that are 4-bit already are
 * not taken (PKV_ERR_UNSUPPORTED).
 * Slots that repeat within one call: one of the writers wins (unspecified which); in a 4-bit cache
 * such a row may mix the writers' codes and scales.
 * Launch order (kv_write and copy_blocks alike): launched as a programmatic dependent of
 * the previous kernel on `stream`; the kernel touches no memory before that kernel has
 * completed, so stream order holds as for a plain launch.
 */
PKV_API pkv_status pkv_kv_write(const void* k_new, const void* v_new, pkv_dtype in_dtype, int num_tokens,
                        const int64_t* slot_mapping, void* k_cache, void* v_cache,
                        const pkv_cache_desc* cache, pkv_stream_t stream);

/*
 * kv_read: a sequence's cached rows out of their blocks, in order and dequantised; the way back of
 * kv_write.  A quantised history becomes plain rows, for instance for the attention of a chunk
 * that follows it (pkv_prompt_attention).
 *   k_out, v_out   (device) [total_tokens][num_kv_heads][head_dim] of out_dtype (f16 or bf16; for a
 *                  16-bit cache its own type)
 *   cu_lens        (device) int32 [num_seqs + 1], cu_lens[0] = 0, ascending, the last at most
 *                  total_tokens
 *   block_tables   (device) int32 [num_seqs][max_blocks_per_seq]
 * Output row cu_lens[i] + j becomes position j of sequence i, for K and for V:
 *   out[cu_lens[i] + j][h][:] = cache[T_i[j / B]][h][j % B][:]
 * 16-bit rows are copied.  Otherwise the code (4-bit: code * scale, exact) times k_scale / v_scale of the
 * head is rounded to fp32 and then to out_dtype.
 * Rows from cu_lens[num_seqs] on are left as they were.  A block id outside the pool leaves its rows
 * as they were and is flagged PKV_DEVERR_BLOCK_ID; so are rows of a sequence longer than its table
 * and, as far as the inconsistency reaches, rows under cu_lens that are not ascending from 0 or pass
 * total_tokens (PKV_DEVERR_CHUNK).
 * Launched like kv_write (programmatic dependent, waits before touching memory).
 */
PKV_API pkv_status pkv_kv_read(void* k_out, void* v_out, pkv_dtype out_dtype, int total_tokens,
                               const int32_t* cu_lens, int num_seqs, const int32_t* block_tables,
                               int max_blocks_per_seq, const void* k_cache, const void* v_cache,
                               const pkv_cache_desc* cache, pkv_stream_t stream);

/*
 * copy_blocks: the copy step of copy-on-write (Lecture 33 §2.4: the writer gets a new
 * block holding a copy of the shared block).
 *   block_pairs (device) int32 [num_pairs][2] = (src, dst)
 * For each pair, the whole block dst of K and of V (all kv heads, all rows) becomes a
 * copy of block src.  No dst may also appear as a src or twice as a dst (the result
 * would depend on order): such pairs, and ids outside the pool, are skipped and flagged
 * PKV_DEVERR_COPY_PAIR.
 */
PKV_API pkv_status pkv_copy_blocks(void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                           const int32_t* block_pairs, int num_pairs, pkv_stream_t stream);

/*
 * swap_blocks: preemption by swapping ("Lecture 33 — KV Cache management" §5.2: the
 * victim's blocks are copied to host RAM, its device blocks are released, and later the
 * blocks are copied back so the sequence can resume).  Block copies between two pools of
 * the same block layout: num_kv_heads, block_size, head_dim and kv_dtype come from `layout`
 * (its num_blocks is not used).  Either pool may be pinned host memory (cudaHostAlloc /
 * cudaHostRegister), passed by its device-visible address (with unified addressing, the
 * host pointer itself).
 *   dst_k/dst_v, src_k/src_v  [num_blocks][num_kv_heads][block_size][head_dim] each
 *   dst_num_blocks, src_num_blocks  pool sizes in blocks (ids are checked against them)
 *   block_pairs (device) int32 [num_pairs][2] = (src block, dst block)
 * For each pair, block dst of dst_k (and dst_v) becomes a copy of block src of src_k
 * (src_v).  Pairs with an id outside its pool, or whose dst another pair also names, are
 * skipped and flagged PKV_DEVERR_COPY_PAIR.  pkv_bm_swap_out / pkv_bm_swap_in produce the
 * pairs.  Launched like kv_write (programmatic dependent, waits before touching memory).
 */
PKV_API pkv_status pkv_swap_blocks(void* dst_k, void* dst_v, int dst_num_blocks, const void* src_k,
                                   const void* src_v, int src_num_blocks, const pkv_cache_desc* layout,
                                   const int32_t* block_pairs, int num_pairs, pkv_stream_t stream);

/*
 * Workspace bytes pkv_paged_decode needs on the current device: two partial-result
 * slots per worker warp (running max, sum of exponentials and unnormalised output per
 * query head).  It depends on the device's SM count and the group size, not on the number
 * of sequences or the context lengths.  The workspace needs no initialisation; each call
 * rewrites what it reads.  Calls that share a workspace must not overlap.
 */
PKV_API size_t pkv_decode_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                  int block_size, int max_context_len, int partition_size);

/*
 * paged_decode: one query token per running sequence (Lecture 33 §2.3).  For sequence
 * i, query head h and kv head g = h / (num_heads / num_kv_heads), with L = context_lens[i]:
 *   s_j = scale * q[i][h] . K_i[j]  for j < L, where K_i[j] = k_cache[T_i[j / B]][g][j % B]
 *   out[i][h] = sum_j softmax(s)_j V_i[j]                         (zeros when L == 0)
 * with T_i = block_tables[i].  Split-KV: the (sequence, kv head, block) tiles are cut into
 * one contiguous range per worker warp — at any block (partition_size = 0, "balanced")
 * or only at multiples of partition_size tokens.  A worker runs an online softmax over
 * its range (consecutive partitions merge in registers); pieces of one sequence held by
 * different workers are merged by log-sum-exp in a second kernel on the same stream,
 * launched as a programmatic dependent of the first.  fp32 accumulation; the softmax's exponentials
 * are rounded to the type of their products with V (the cache's; fp16 over e4m3 and 4 bits).
 *   out            (device) [num_seqs][num_heads][head_dim] of q_dtype
 *   q              (device) [num_seqs][num_heads][head_dim] of q_dtype (f16 or bf16)
 *   block_tables   (device) int32 [num_seqs][max_blocks_per_seq]
 *   context_lens   (device) int32 [num_seqs]; tokens to attend, including any token
 *                  written this step
 *   max_context_len host upper bound of context_lens; larger lengths are clamped to it
 *                  (and to max_blocks_per_seq * block_size) and flagged PKV_DEVERR_CONTEXT_LEN
 *   partition_size  0 = balanced split; else split granularity in tokens (multiple of 16)
 *   workspace       (device) >= pkv_decode_workspace_bytes(...) bytes
 * out, q, block_tables and context_lens may instead be pinned host memory (cudaHostAlloc /
 * cudaHostRegister, reachable through unified addressing): the kernels then read and write
 * them in place over the host link, so a serving loop needs no separate copies.  The caches
 * and the workspace must be device memory.
 * Supported: kv f16/bf16 with the same q dtype, or e4m3 (head_dim 128) or 4-bit kv with f16/bf16 q
 * (e4m3: q is taken as fp16, so bf16 |q| must stay below 65504 and loses bits below 2^-14; 4-bit: bf16
 * q of any size, each row times a power of two of its own); head_dim 64/128; block_size 16 or 32;
 * num_heads / num_kv_heads in 1..8; num_kv_heads * num_seqs * ceil(L_max / 16) < 2^31, where
 * L_max = min(max_context_len, max_blocks_per_seq * block_size); up to about 13,000 sequences, whose
 * prefix sums share an SM's shared memory with the tiles (4-bit kv 13,180, 16-bit kv of head_dim 128
 * 13,700, else 16,400) (else PKV_ERR_UNSUPPORTED).
 * Launch order: the decode kernel is launched as a programmatic dependent of the previous
 * kernel on `stream`.  If that kernel allows early dependent launch (pkv_kv_write, pkv_kv_read
 * and pkv_qk_rotary do), the decode kernel may already read context_lens and block_tables while it still runs; q, the
 * caches, out and the workspace are touched only after it has completed.  So the kernel
 * right before a decode call must not write context_lens or block_tables unless it leaves
 * dependent launch at its default (wait for completion).
 */
PKV_API pkv_status pkv_paged_decode(void* out, const void* q, pkv_dtype q_dtype, int num_seqs, int num_heads,
                            const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* context_lens, int max_context_len, float scale,
                            int partition_size, void* workspace, size_t workspace_bytes,
                            pkv_stream_t stream);

/*
 * paged_decode_append: pkv_kv_write of one new token per sequence fused into
 * pkv_paged_decode (PagedAttention §3.3: each new token fills its sequence's last block).
 * For every sequence i with L = context_lens[i] >= 1, the new rows k_new[i] and v_new[i] are
 * stored at position L - 1, i.e. slot block_tables[i][(L - 1) / B] * B + (L - 1) % B, quantised
 * for an e4m3 or 4-bit cache exactly as pkv_kv_write does, and the decode then attends positions
 * 0 .. L - 1, the new one included.  Caches and out are bit-identical to pkv_kv_write (with those
 * slots) followed by pkv_paged_decode.
 *   k_new, v_new  (device, or pinned host memory as for q) [num_seqs][num_kv_heads][head_dim]
 *                 of q_dtype, 16-byte aligned
 *   k_cache, v_cache  (device) written at those positions only
 * Sequences with L == 0 write nothing.  A length above the clamp bound (see pkv_paged_decode)
 * writes nothing and is flagged PKV_DEVERR_CONTEXT_LEN; a block id outside the pool writes
 * nothing and is flagged PKV_DEVERR_BLOCK_ID.  The written block must not be shared with
 * another sequence of the call (copy-on-write has run), as for pkv_kv_write.  Other
 * arguments, limits, launch order and results as pkv_paged_decode.
 */
PKV_API pkv_status pkv_paged_decode_append(void* out, const void* q, pkv_dtype q_dtype, int num_seqs,
                                   int num_heads, const void* k_new, const void* v_new, void* k_cache,
                                   void* v_cache, const pkv_cache_desc* cache, const int32_t* block_tables,
                                   int max_blocks_per_seq, const int32_t* context_lens,
                                   int max_context_len, float scale, int partition_size, void* workspace,
                                   size_t workspace_bytes, pkv_stream_t stream);

/*
 * paged_decode for callers that cannot allocate device memory.  The pages have no
 * counterpart to this entry point; it exists for callers that must not allocate at decode
 * time: a plain C host without a device allocator of its own for scratch space, or a
 * serving loop that may not call cudaMalloc on its hot path because cudaMalloc can
 * synchronise the whole device.  Same arguments and results as pkv_paged_decode, minus the
 * workspace: the library keeps one fixed scratch array of pkv_noalloc_scratch_bytes()
 * (24 MiB) on every device that loads it, resident until the process exits.  Arguments are
 * checked exactly as pkv_paged_decode checks them, in the same order, so an invalid call
 * returns the same status from both entry points.  The scratch a call needs (per
 * pkv_decode_workspace_bytes) depends on the SM count, the group size and head_dim only;
 * 24 MiB holds every supported call on a device of up to 252 SMs.  A valid call that needs
 * more than the array holds returns PKV_ERR_WORKSPACE and enqueues nothing.  No call allocates, frees or clears device memory: each call
 * rewrites the parts of the array it later reads, so leftovers of earlier calls do no
 * harm.  The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call before any
 * stream capture.  Every call on a device shares the one array, so calls whose kernels
 * may overlap on the GPU (different streams with no ordering between them) race and
 * corrupt each other's results: keep them on one stream or order them with events.
 */
PKV_API size_t pkv_noalloc_scratch_bytes(void);
PKV_API pkv_status pkv_paged_decode_noalloc(void* out, const void* q, pkv_dtype q_dtype, int num_seqs,
                                            int num_heads, const void* k_cache, const void* v_cache,
                                            const pkv_cache_desc* cache, const int32_t* block_tables,
                                            int max_blocks_per_seq, const int32_t* context_lens,
                                            int max_context_len, float scale, int partition_size,
                                            pkv_stream_t stream);

/*
 * SM budget of the decode calls (pkv_paged_decode, _append, _noalloc).  The decode runs one
 * persistent CTA per SM.  A budget n in 1 .. (SM count - 1) launches n CTAs instead, splitting
 * the same work over fewer worker warps and leaving the other SMs to a kernel that runs
 * beside it on another stream.  The use case is a chunk's tensor-bound prefill beside the
 * step's HBM-bound decodes (Lecture 33 §4.2 batches the two in one step).  Under a budget the
 * merge kernel launches when the decode grid has finished, not while it runs, so that its
 * waiting CTAs do not hold those SMs.
 *   num_sms  0 (the default) or >= the SM count: every SM.  Negative: PKV_ERR_INVALID_ARG,
 *            the budget is unchanged.
 * Results stay within the decode tolerances for any budget.  The split over workers
 * changes, so fp32 sums are rounded in another order, and outputs are not bit-identical
 * across budgets.  The setting is process-wide and applies to decode calls made after it,
 * on every device and thread.  A captured graph keeps the grid of the call it captured.
 * pkv_decode_workspace_bytes does not depend on the budget: it always sizes for every SM.
 */
PKV_API pkv_status pkv_set_decode_sm_budget(int num_sms);
PKV_API int pkv_get_decode_sm_budget(void);

/*
 * paged_prefill_chunk: causal attention of prefill chunks over their paged history
 * (Lecture 33 §4.2: a chunk attends the earlier chunks' cached KV, masked causally).
 * Chunk c holds query rows cu_q_lens[c] .. cu_q_lens[c+1]-1; row r of the chunk is at
 * absolute position p = q_start_pos[c] + r of sequence c and attends that sequence's
 * keys 0..p (its cached history and itself).  The chunk's own K/V must already be in the
 * cache (pkv_kv_write first).
 *   out, q        (device) [total_q][num_heads][head_dim] of q_dtype (bf16 or f16; same as kv)
 *   cu_q_lens     (device) int32 [num_chunks + 1], cu_q_lens[0] = 0, cu_q_lens[num_chunks] = total_q
 *   q_start_pos   (device) int32 [num_chunks]
 *   block_tables  (device) int32 [num_chunks][max_blocks_per_seq]
 *   max_q_len     host upper bound of the chunks' lengths (sizes the grid); a longer chunk
 *                 sets PKV_DEVERR_CHUNK and its rows past max_q_len stay unwritten.  0 says that
 *                 every chunk is empty: nothing is enqueued, and the lengths are not looked at
 * Supported: f16/bf16 cache with the same q dtype, head_dim 128, block_size 16 or 32,
 * num_heads a multiple of num_kv_heads (any group size).  Tensor cores (tcgen05, TMEM
 * accumulators), K/V tiles fetched by TMA straight from the physical blocks; with two or
 * more query heads per kv head they are multicast to the two CTAs of a cluster that read
 * the same keys.  q, k_cache and v_cache must be device memory of
 * the current GPU (checked with cudaPointerGetAttributes before anything is enqueued):
 * host, managed or another GPU's memory returns PKV_ERR_INVALID_ARG.
 * Launch order: launched as a programmatic dependent of the previous kernel on `stream`.
 * Only the kernel's own shared-memory and tensor-memory set-up runs before that kernel has
 * completed; no argument is read and no memory touched earlier, so stream order holds as
 * for a plain launch.
 */
PKV_API pkv_status pkv_paged_prefill_chunk(void* out, const void* q, pkv_dtype q_dtype,
                                   const int32_t* cu_q_lens, const int32_t* q_start_pos,
                                   int num_chunks, int total_q, int max_q_len, int num_heads,
                                   const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                                   const int32_t* block_tables, int max_blocks_per_seq, float scale,
                                   pkv_stream_t stream);

/*
 * prompt_attention: causal attention of packed prompts over keys and values that need not be in a
 * cache (the fresh rows of a prompt, or a history from pkv_kv_read with the chunk's own rows behind
 * it).  Sequence i holds query rows cu_q_lens[i] .. cu_q_lens[i+1]-1 and key rows cu_k_lens[i] ..
 * cu_k_lens[i+1]-1, Lq and Lk of them; its query rows are the last Lq positions.  Row r attends the
 * sequence's keys 0 .. r + Lk - Lq:
 *   out[r][h] = sum_j softmax_j(scale * q[r][h] . k[j][g]) v[j][g],  g = h / (num_heads / num_kv_heads)
 * A row without keys (r + Lk - Lq < 0, or Lk == 0) gives zeros.
 *   out, q         (device) [total_q] rows of [num_heads][head_dim] of dtype (f16 or bf16)
 *   k, v           (device) [total_k] rows of [num_kv_heads][head_dim] of dtype
 *   *_stride       elements from one row to the next (at least heads * head_dim, a multiple of 8), so
 *                  that q, k and v may be parts of one packed projection
 *   cu_q_lens, cu_k_lens (device) int32 [num_seqs + 1], from 0, ascending, the last at most total_q
 *                  (total_k); output rows from cu_q_lens[num_seqs] on are left as they were
 *   max_q_len      host upper bound of Lq (sizes the grid); a longer sequence sets PKV_DEVERR_CHUNK and
 *                  its rows past max_q_len stay unwritten.  0 says that every sequence is empty: the call
 *                  returns PKV_OK at once, enqueues nothing, and the lengths are not looked at
 * out must not overlap q, k or v.  Only what a row attends reaches it: infinities and NaN in other
 * rows' keys and values, and behind the sequences, do not.  cu_q_lens or cu_k_lens that are not
 * ascending from 0 or pass the totals set PKV_DEVERR_CHUNK and leave that sequence's rows unwritten.
 * Supported: head_dim 64 or 128, scale > 0, num_heads a multiple of num_kv_heads, num_seqs and
 * num_heads up to 65535.  P is rounded to dtype before its product with V, as the tensor cores take
 * it; sums and outputs are fp32 until the last rounding.  q, k and v must be device memory of the
 * current GPU (as for pkv_paged_prefill_chunk).  Launch order as pkv_paged_prefill_chunk.
 */
PKV_API pkv_status pkv_prompt_attention(void* out, const void* q, const void* k, const void* v, pkv_dtype dtype,
                                        const int32_t* cu_q_lens, const int32_t* cu_k_lens, int num_seqs,
                                        int total_q, int total_k, int max_q_len, int num_heads, int num_kv_heads,
                                        int head_dim, int64_t out_stride, int64_t q_stride, int64_t k_stride,
                                        int64_t v_stride, float scale, pkv_stream_t stream);

/*
 * Workspace bytes pkv_paged_chunk_attention needs on the current device.  It depends on the SM count and the
 * shapes given, not on the lengths.  The workspace needs no initialisation; calls that share one must not overlap.
 */
PKV_API size_t pkv_chunk_workspace_bytes(int total_q, int num_heads, int num_kv_heads, int head_dim);

/*
 * paged_chunk_attention: causal attention of each sequence's new rows over its paged cache, of any type:
 * drafted tokens to verify, a prompt's next chunk, or one token.  The keys are split over the GPU, so that few
 * rows over long histories use all of it.  Chunk c holds query rows cu_q_lens[c] .. cu_q_lens[c+1]-1; row r of the
 * chunk is at position p = q_start_pos[c] + r and attends keys 0 .. p, whose K/V must be in the cache
 * (pkv_kv_write first).  With g = h / (num_heads / num_kv_heads):
 *   s_j = scale * q[r][h] . K[j][g],   out[r][h] = sum_j softmax(s)_j V[j][g],   lse[r][h] = log sum_j exp(s_j)
 *   out, q         (device) [total_q][num_heads][head_dim] of q_dtype (f16 or bf16; for a 16-bit cache its type)
 *   lse            (device) fp32 [total_q][num_heads], or NULL
 *   cu_q_lens      (device) int32 [num_chunks + 1], from 0, ascending, the last at most total_q; output rows from
 *                  cu_q_lens[num_chunks] on are left as they were
 *   q_start_pos    (device) int32 [num_chunks]
 *   block_tables   (device) int32 [num_chunks][max_blocks_per_seq]
 *   workspace      (device) >= pkv_chunk_workspace_bytes(...) bytes
 * out must not overlap q.  Only what a row attends reaches it: infinities and NaN in other keys and values, in
 * stale rows of a block, and behind the chunks, do not.  A chunk whose lengths are inconsistent (cu_q_lens not
 * ascending from 0 or past total_q, q_start_pos < 0, or positions past its table) sets PKV_DEVERR_CHUNK and its
 * rows stay unwritten.  A block id outside the pool sets PKV_DEVERR_BLOCK_ID; its keys and values count as zeros.
 * Supported: f16, bf16, e4m3 and 4-bit caches, head_dim 64 or 128, block_size 16 or 32, any number of query heads
 * per kv head, scale > 0 and up to 2^127, num_chunks up to 65535, total_q * num_heads below 2^31 - 512,
 * max_blocks_per_seq * block_size up to 2^31 - 128, and
 * (total_q * (num_heads / num_kv_heads) / 64 + 3 num_chunks) * (max_blocks_per_seq * block_size / 128 + 2)
 * below 2^31.  Sums, maxima and outputs are fp32 until the last rounding; the softmax's exponentials are rounded to
 * the type of their product with V (q_dtype; fp16 over e4m3 and 4 bits): as fp16 by up to 2^-11 of each or 2^-32 of the
 * row's largest, whichever is more.  Over e4m3 and 4 bits, bf16 q is taken as fp16 after a power of two for each row
 * (elements lose at most 2^-39 of the row's largest).  All of it must be memory of the current GPU.  Launch order as
 * pkv_kv_write (waits before touching memory).
 */
PKV_API pkv_status pkv_paged_chunk_attention(void* out, float* lse, const void* q, pkv_dtype q_dtype,
                                             const int32_t* cu_q_lens, const int32_t* q_start_pos, int num_chunks,
                                             int total_q, int num_heads, const void* k_cache, const void* v_cache,
                                             const pkv_cache_desc* cache, const int32_t* block_tables,
                                             int max_blocks_per_seq, float scale, void* workspace,
                                             size_t workspace_bytes, pkv_stream_t stream);

/*
 * Eviction by attention weight: a sequence's cache is cut to the tokens that its queries look at.
 * pkv_attention_weights adds up the attention that each cached token gets, pkv_evict_select picks the tokens each
 * kv head keeps, pkv_bm_evict gives the sequence its new table, and pkv_evict_compact moves the kept rows to
 * its front.  Every head keeps the same number of tokens, not the same tokens.  Keys keep the positions that they
 * were rotated by; later tokens go on with their own.
 *
 * Weights are fp32 [num_rows][num_kv_heads][max_len]; sequence i has row rows[i] (row i if rows is NULL).  A
 * negative row says that the sequence has none (nothing is read or written for it); one from num_rows on sets
 * PKV_DEVERR_SLOT and counts as none.  Rows that repeat within one call: one of the writers wins.
 *
 * attention_weights: for the rows of chunk c (as in pkv_paged_chunk_attention) and key j < q_start_pos[c] + Lq
 *   w[j] = sum over rows r with q_start_pos[c] + r >= j and over the query heads h of the kv head of
 *          exp(scale * q[r][h] . K[j] - lse[r][h])
 *   out[row][kv head][j] = decay * weights[row][kv head][j] + w[j]   for j < q_start_pos[c] and weights given
 *                        = w[j]                                      otherwise (the chunk's own tokens are new)
 * Positions from q_start_pos[c] + Lq on, and the rows of chunks without query rows, are left as they were.  A token gets
 * its first weight when its own row is in the chunk: one that was attended by a decode call alone has none, and the row
 * still holds there what it held before, which later calls would take for its weight.
 *   out            (device) the weights' layout; may be `weights` itself, other overlaps not
 *   weights        (device) or NULL: none so far
 *   q, cu_q_lens, q_start_pos, block_tables, k_cache   as for pkv_paged_chunk_attention
 *   lse            (device) fp32 [total_q][num_heads], from pkv_paged_chunk_attention over the same keys
 *   decay          finite, >= 0
 * Errors as for pkv_paged_chunk_attention; a chunk longer than max_len sets PKV_DEVERR_CONTEXT_LEN and is left
 * out.  fp32 sums in an order that is the same for the same call on the same number of SMs; among other chunks, or on another
 * GPU, the last bits may differ.  Supported as there, scale included.
 */
PKV_API pkv_status pkv_attention_weights(float* out, const float* weights, float decay, int num_rows, int max_len,
                                         const int32_t* rows, const void* q, pkv_dtype q_dtype, const float* lse,
                                         const int32_t* cu_q_lens, const int32_t* q_start_pos, int num_chunks,
                                         int total_q, int num_heads, const void* k_cache, const pkv_cache_desc* cache,
                                         const int32_t* block_tables, int max_blocks_per_seq, float scale,
                                         pkv_stream_t stream);

/*
 * evict_select: kept[i][h][0 .. n-1] = the positions that kv head h of sequence i keeps, ascending; the rest of
 * its max_keep entries become -1.  With L = context_lens[i], n = min(keep_lens[i], L):
 *   the newest min(recent, n) positions, then the first min(first, what is left of n), then those of the largest
 *   weights; of equal weights (-0 equals 0; NaN is less than all) the lower position.
 * The positions that are chosen by weight have to have one (see above).  The work goes by max_len, not by the lengths: 64
 * sequences of 2,048 positions and 4 heads take 7.8 us in rows of 2,048 and 53 us in rows of 131,072.
 *   kept           (device) int32 [num_seqs][num_kv_heads][max_keep]
 *   context_lens, keep_lens (device) int32 [num_seqs]; a context_len outside 0 .. max_len or a keep_len outside
 *                  0 .. max_keep sets PKV_DEVERR_CONTEXT_LEN and gives -1 throughout, as does a sequence without a row
 * Supported: max_len and max_keep up to 2^30.
 */
PKV_API pkv_status pkv_evict_select(int32_t* kept, int max_keep, const float* weights, int num_rows, int max_len,
                                    const int32_t* rows, const int32_t* context_lens, const int32_t* keep_lens,
                                    int num_seqs, int num_kv_heads, int first, int recent, pkv_stream_t stream);

/*
 * evict_compact: for every sequence i, kv head h and j < keep_lens[i] with p = kept[i][h][j] >= 0, position j of
 * dst_tables[i] gets K, V and weight of position p of src_tables[i], in the cache's own type:
 *   cache[dst_tables[i][j / B]][h][j % B] = cache[src_tables[i][p / B]][h][p % B]
 *   weights[dst_rows[i]][h][j] = weights[rows[i]][h][p]
 * as if all were read before any is written.  dst_tables may be src_tables (in place); in general dst_tables[i][b]
 * is src_tables[i][b] or a block that no table of the call reads, as pkv_bm_evict gives them, and no two sequences write the same block.
 * kept has to ascend (pkv_evict_select): an entry that does not, or is past its table, sets PKV_DEVERR_CHUNK and is
 * left out.  keep_lens outside 0 .. max_keep set PKV_DEVERR_CONTEXT_LEN and leave the sequence alone, positions
 * past max_len the weight; block ids outside the pool set PKV_DEVERR_BLOCK_ID and leave the row out.
 *   src_tables     (device) int32 [num_seqs][src_max_blocks]; dst_tables [num_seqs][dst_max_blocks]
 *   weights        (device) or NULL: only K and V move
 *   dst_rows       (device) or NULL: rows.  Distinct rows; dst_rows[i] is rows[i] or a row that the call does not read
 * Any cache type, head_dim a multiple of 16 up to 256, max_keep up to 2^30; k_cache is not v_cache.
 * Launch order as pkv_kv_write, for all four calls.
 */
PKV_API pkv_status pkv_evict_compact(void* k_cache, void* v_cache, const pkv_cache_desc* cache, const int32_t* kept,
                                     int max_keep, const int32_t* keep_lens, const int32_t* src_tables,
                                     int src_max_blocks, const int32_t* dst_tables, int dst_max_blocks, float* weights,
                                     int num_rows, int max_len, const int32_t* rows, const int32_t* dst_rows,
                                     int num_seqs, pkv_stream_t stream);

/* Rotary positions.  Pair i of a head (0 <= i < rotary_dim / 2) turns by position * f_i. */
typedef enum {
  PKV_ROPE_HALF = 0,         /* pair i is elements i and i + rotary_dim / 2 */
  PKV_ROPE_INTERLEAVED = 1   /* pair i is elements 2i and 2i + 1 */
} pkv_rope_layout;

typedef enum {               /* how f_i = base^(-2i / rotary_dim) is scaled for contexts past original_context */
  PKV_ROPE_NONE = 0,
  PKV_ROPE_LINEAR = 1,       /* f_i / factor: positions are interpolated */
  PKV_ROPE_NTK = 2,          /* base * factor^(rotary_dim / (rotary_dim - 2)) in the place of base */
  PKV_ROPE_PARTS = 3         /* with r = original_context * f_i / (2 pi), the turns over the original context:
                                f_i where r >= beta, f_i / factor where r <= alpha, between them the blend
                                w f_i + (1 - w) f_i / factor, w = (r - alpha) / (beta - alpha) */
} pkv_rope_scaling;

/*
 * Frequencies for pkv_qk_rotary: table[i] (host memory, rotary_dim / 2 entries; copy it to the device
 * once) = f_i / (2 pi) turns per position in units of 2^-64 turns.  A position times an entry, modulo
 * 2^64, is the angle modulo one turn, so far positions lose nothing.  base > 1; factor >= 1 (not
 * read for PKV_ROPE_NONE); original_context > 0 and alpha < beta for PKV_ROPE_PARTS;
 * rotary_dim >= 4 for PKV_ROPE_NTK.
 */
PKV_API pkv_status pkv_rope_table(uint64_t* table, int rotary_dim, double base, pkv_rope_scaling scaling,
                                  double factor, double original_context, double alpha, double beta);

/*
 * qk_rotary: what a step does to its queries and keys between the projection and kv_write /
 * attention: an RMS norm of each head (optional) and its rotation by the token's position, in one
 * pass.  For each row x of head_dim elements, in fp32:
 *   y = x * rsqrt(mean(x^2) + eps) * weight     (y = x when the weight is NULL)
 *   (a, b) of pair i become magnitude * (a cos t - b sin t), magnitude * (b cos t + a sin t),
 *   t = position * f_i; elements from rotary_dim on stay y; one rounding to dtype.
 *   q_out, q       (device) [num_tokens] rows of [num_heads][head_dim] of dtype (f16 or bf16)
 *   k_out, k       (device) [num_tokens] rows of [num_kv_heads][head_dim] of dtype
 *   *_stride       elements from one token's row to the next, a multiple of 8 and at least
 *                  heads * head_dim; q_out == q and k_out == k with equal strides work in place, other
 *                  overlaps do not
 *   positions      (device) int32 [num_tokens]; a negative position marks a padding token, whose rows
 *                  in q_out and k_out are left as they were
 *   table          (device) uint64 [rotary_dim / 2], from pkv_rope_table
 *   q_weight, k_weight (device) [head_dim] of dtype, or NULL: no norm
 *   magnitude      factor on the rotated elements (1 if the context is not scaled)
 * num_heads or num_kv_heads may be 0 (its pointers are then not read).  Supported: head_dim a
 * multiple of 16 up to 256, rotary_dim a multiple of 16 up to head_dim.
 * Launched like kv_write (programmatic dependent, waits before touching memory).
 */
PKV_API pkv_status pkv_qk_rotary(void* q_out, const void* q, void* k_out, const void* k, pkv_dtype dtype,
                                 int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                 int64_t q_out_stride, int64_t q_stride, int64_t k_out_stride, int64_t k_stride,
                                 const int32_t* positions, const uint64_t* table, int rotary_dim,
                                 pkv_rope_layout layout, float magnitude, const void* q_weight,
                                 const void* k_weight, float eps, pkv_stream_t stream);

/*
 * Waits for `stream`, then reads and clears the library's device error word on the
 * current device.  *code receives the PKV_DEVERR_* bits (0 = clean).  Returns
 * PKV_ERR_DEVICE_CHECK when any bit was set, PKV_OK otherwise.
 */
PKV_API pkv_status pkv_get_device_error(int* code, pkv_stream_t stream);

/*
 * Measurement aid, not part of the method: reads the num_tiles K/V tiles whose first pool
 * rows are tile_rows[i] (16 rows of one (block, kv head), in K and in V) with the memory
 * pipeline pkv_paged_decode uses (persistent grid, 12 warps per SM, two stages of one K and
 * one V tile per warp, bulk asynchronous copies) and computes nothing but a checksum, XORed
 * into *checksum.  Timed on the tiles of a decode call, it is the memory ceiling of that
 * call.  Rows outside the pool are skipped and flagged PKV_DEVERR_BLOCK_ID.
 *   tile_rows (device) int32 [num_tiles]; checksum (device) one uint32
 */
PKV_API pkv_status pkv_stream_tiles(const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                                    const int32_t* tile_rows, int num_tiles, unsigned* checksum,
                                    pkv_stream_t stream);

/*
 * Diagnostic of the failure path every kernel shares: one warp waits on an mbarrier that
 * nothing arrives on, with the same bounded wait the kernels use, for limit_ns (0 < limit_ns
 * <= 1 s), then sets PKV_DEVERR_TIMEOUT and returns.  Nothing faults or hangs; the context
 * stays usable.  Read the bit with pkv_get_device_error.
 */
PKV_API pkv_status pkv_check_bounded_wait(uint64_t limit_ns, pkv_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * Host block manager ("PagedAttention: manage the KV cache like virtual memory" §3.2–§3.3;
 * Lecture 33 §2.2, §2.4).  A FIFO free-block queue (allocate pops the head, free pushes
 * the tail), a ref_cnt per block, and one block table per sequence.  It produces the
 * block tables, context lengths, slot mappings and copy-on-write pairs the device calls
 * consume.  Host memory only; not thread-safe (one manager per scheduler thread).
 * Every call that fails leaves the manager unchanged.
 * ------------------------------------------------------------------------------------- */
typedef struct pkv_block_manager pkv_block_manager;

/* A pool of num_blocks blocks of block_size tokens; the free queue starts as 0..num_blocks-1. */
PKV_API pkv_status pkv_bm_create(int num_blocks, int block_size, pkv_block_manager** out);
PKV_API void pkv_bm_destroy(pkv_block_manager* bm);

/* Claim the listed blocks for a new sequence holding n_tokens tokens (n_blocks must equal
 * ceil(n_tokens / block_size)); each block's ref_cnt rises by one and a free block leaves
 * the free queue.  Used to set up states such as shared prefixes. */
PKV_API pkv_status pkv_bm_import_seq(pkv_block_manager* bm, int64_t seq, const int32_t* blocks,
                             int n_blocks, int n_tokens);

/* Admit a sequence with an n_tokens prompt: pop ceil(n_tokens / block_size) blocks. */
PKV_API pkv_status pkv_bm_allocate(pkv_block_manager* bm, int64_t seq, int n_tokens);

/* Reserve the slot of the sequence's next token.  If the token starts a new block, one
 * block is popped.  If it lands in a block whose ref_cnt > 1, copy-on-write: a new block
 * is popped, (*cow_src, *cow_dst) = (old, new), the table points at the new block and the
 * old block's ref_cnt drops by one; otherwise both are set to -1. */
PKV_API pkv_status pkv_bm_append_slot(pkv_block_manager* bm, int64_t seq, int64_t* slot,
                              int32_t* cow_src, int32_t* cow_dst);

/* One decode step for a batch: append_slot for seqs[0..n) in order, then export.
 *   slot_mapping  int64 [n]; cow_pairs int32 [n][2] (first *n_cow rows used)
 *   tables        int32 [n][max_blocks] padded with -1; lens int32 [n] (after the step)
 * Fails with PKV_ERR_NO_BLOCKS, changing nothing, if the free queue cannot cover it. */
PKV_API pkv_status pkv_bm_step_decode(pkv_block_manager* bm, const int64_t* seqs, int n, int max_blocks,
                              int64_t* slot_mapping, int32_t* cow_pairs, int* n_cow,
                              int32_t* tables, int32_t* lens);

/* Reserve n consecutive slots (a prefill chunk); slots int64 [n], cow_pairs int32 [n][2]. */
PKV_API pkv_status pkv_bm_append_slots(pkv_block_manager* bm, int64_t seq, int n, int64_t* slots,
                               int32_t* cow_pairs, int* n_cow);

/* child's table becomes a copy of parent's; every block's ref_cnt rises by one. */
PKV_API pkv_status pkv_bm_fork(pkv_block_manager* bm, int64_t parent, int64_t child);

/* Drop the sequence: each block's ref_cnt falls by one; blocks reaching 0 go to the
 * tail of the free queue, in table order. */
PKV_API pkv_status pkv_bm_free(pkv_block_manager* bm, int64_t seq);

/* Eviction: sequence seqs[i] goes down to its first new_lens[i] positions, which pkv_evict_compact fills with the
 * tokens that it keeps.  src_tables and src_lens are what it had, dst_tables what it has now: the same blocks, but
 * a new one in the place of each that another holder shares, whose contents stay.  Blocks past the new length are
 * released, in table order, after every new block was popped; a block that is written loses its prefix-cache hash.
 * A sequence whose length does not change keeps its table.  Launch the compaction before anything that uses the
 * released blocks.
 *   src_tables int32 [n][src_max_blocks], dst_tables int32 [n][dst_max_blocks], padded with -1; src_lens int32 [n]
 * PKV_ERR_NO_BLOCKS, changing nothing, if the shared blocks outnumber the free ones. */
PKV_API pkv_status pkv_bm_evict(pkv_block_manager* bm, const int64_t* seqs, int n, const int32_t* new_lens,
                                int src_max_blocks, int32_t* src_tables, int32_t* src_lens, int dst_max_blocks,
                                int32_t* dst_tables);

/* tables int32 [n][max_blocks] (padded with -1), lens int32 [n]. */
PKV_API pkv_status pkv_bm_export(const pkv_block_manager* bm, const int64_t* seqs, int n, int max_blocks,
                         int32_t* tables, int32_t* lens);

/* Prefix caching ("PagedAttention: manage the KV cache like virtual memory" §3.4–§3.5;
 * Lecture 33 §6.2–§6.3).  A full block is named by h_i = FNV-1a-64(h_{i-1} as 8 bytes
 * little-endian, then its block_size token ids as 4 bytes little-endian each), with h_{-1} =
 * the FNV offset basis 0xcbf29ce484222325, so equal hashes mean equal prefixes.  Admission of
 * a prompt matches its full blocks in order against the cached hashes and stops at the first
 * miss; each hit is "touched" (ref_cnt + 1, and a block nobody held is unlinked from the
 * middle of the free queue in O(1)).  The remaining blocks are popped from the free queue's
 * head, and the new full blocks are registered under their hashes.  *n_cached_tokens = hits x
 * block_size: those tokens' K/V are already in the pool and need no prefill; the others'
 * K/V become valid once the caller's prefill for this sequence has run.  Freed blocks keep
 * their hash (cached and free) until popped for new contents, which drops the hash.  Blocks
 * that fill up during decode are not registered (the manager does not see token ids there).
 * PKV_ERR_NO_BLOCKS, changing nothing, if the misses need more blocks than are free once the
 * hit blocks leave the queue. */
PKV_API pkv_status pkv_bm_allocate_cached(pkv_block_manager* bm, int64_t seq, const int32_t* tokens, int n_tokens,
                                          int* n_cached_tokens);
/* 1 and *hash = the block's registered hash; 0 if it has none; -1 on bad arguments. */
PKV_API int pkv_bm_block_hash(const pkv_block_manager* bm, int block, uint64_t* hash);
PKV_API int pkv_bm_num_cached(const pkv_block_manager* bm);   /* registered hashes */

/* Preemption by swapping ("Lecture 33 — KV Cache management" §5.2).  The host pool is a
 * second set of num_host_blocks blocks (ids 0..num_host_blocks-1 of a caller-owned pinned
 * buffer with the device pool's block layout) with its own FIFO free queue.  Resizing is
 * allowed only while no sequence is swapped out; the queue restarts as 0..n-1. */
PKV_API pkv_status pkv_bm_set_host_pool(pkv_block_manager* bm, int num_host_blocks);

/* Swap a resident sequence out: for each table entry in order a host block is popped and
 * pairs[i] = (device block, host block); then the device blocks are released in table order
 * (ref_cnt - 1, free at 0), as by pkv_bm_free.  A block shared with another sequence stays on
 * the device for it; this sequence takes its own host copy.  Until swapped in, the sequence
 * can only be freed or swapped in (other calls on it return PKV_ERR_INVALID_ARG).
 *   pairs int32 [max_pairs][2]; *n_pairs = number of table entries.
 * PKV_ERR_NO_BLOCKS, changing nothing, if the host queue holds fewer blocks than the table. */
PKV_API pkv_status pkv_bm_swap_out(pkv_block_manager* bm, int64_t seq, int32_t* pairs, int max_pairs,
                                   int* n_pairs);

/* Swap a sequence back in: for each host block in table order a device block is popped and
 * pairs[i] = (host block, device block); the host blocks return to the host queue's tail in
 * table order.  PKV_ERR_NO_BLOCKS, changing nothing, if too few device blocks are free. */
PKV_API pkv_status pkv_bm_swap_in(pkv_block_manager* bm, int64_t seq, int32_t* pairs, int max_pairs,
                                  int* n_pairs);
PKV_API int pkv_bm_num_free_host(const pkv_block_manager* bm);
PKV_API int pkv_bm_is_swapped(const pkv_block_manager* bm, int64_t seq);   /* 1, 0, or -1 if unknown */

PKV_API int pkv_bm_ref_cnt(const pkv_block_manager* bm, int block);      /* -1 if out of range */
PKV_API int pkv_bm_num_free(const pkv_block_manager* bm);
/* The free queue from head to tail into out[0..max_n); returns the queue length. */
PKV_API int pkv_bm_free_queue(const pkv_block_manager* bm, int32_t* out, int max_n);

#ifdef __cplusplus
}
#endif
#endif /* PKV_H_ */
