/*
 * pa.h -- C ABI of the B200 (sm_100a) paged-KV-cache attention library.
 *
 * The KV cache of one attention layer lives in a pool of fixed-size physical
 * blocks; a per-sequence block table maps logical block j to a physical block.
 * Sources (page title, section):
 *   "vLLM 深度拆解：当大模型推理学会「分页注意力」" (chenxutan.com), 1.1 and 2.1:
 *       K and V of every past token are kept and attended to; they are split
 *       into fixed 16-token blocks placed anywhere in the pool; a block table
 *       maps logical to physical blocks.  2.3: decode is memory-bandwidth bound,
 *       prefill compute bound.  3.1: every step writes the new token's K/V back.
 *       3.3: shared prefix blocks, copy on write.  5.1: chunked prefill.
 *   devpress.csdn.net/amd vLLM v0.6.x teardown, section 核心代码拆解: tensor
 *       layouts (below), the physical block looked up through the table, the
 *       score scaled by `scale`, softmax and a V-weighted sum.  Section
 *       关键设计二: copy-on-write copies a whole shared block into a new one.
 *
 * Layouts (all row-major, all device pointers 16-byte aligned):
 *   key_cache, value_cache  [num_blocks, num_kv_heads, block_size, head_dim]
 *   query, out (decode)     [num_seqs, num_q_heads, head_dim]
 *   query, out (prefill)    [num_seqs, max_chunk, num_q_heads, head_dim]
 *   block_tables            int32 [num_seqs, max_blocks_per_seq]
 *   context_lens            int32 [num_seqs]
 *   slot_mapping            int64 [num_tokens]; slot = block * block_size + offset
 * Query head h reads kv head h / (num_q_heads / num_kv_heads).
 * Supported: dtype PA_F32 or PA_BF16 (cache, query, key/value and out share it),
 * head_dim 64 or 128, block_size 16, num_q_heads / num_kv_heads in {1,2,4,8}.
 * FP8 KV cache (chenxutan 5.3: FP8 KV is close to lossless and halves the bytes;
 * the devpress teardown's architecture figure puts FP8/INT8 quantisation in the
 * kernel layer): dtype PA_FP8_E4M3 stores the pools as one-byte e4m3 codes (OCP
 * 8-bit floating point: bias 7, largest finite 448, S.1111.111 NaN) with one
 * float scale per pool, code = e4m3(fp32(x) / scale) rounded to nearest even and
 * saturated to +-448, value = e4m3 * scale.  key/value inputs, query and out are
 * then bf16.  pa_cache_write, pa_copy_blocks, pa_decode and pa_append_decode take
 * it with head_dim 128; pa_prefill_chunk returns PA_ERR_UNSUPPORTED.
 * 8-bit KV cache with a scale per (block, kv head): pa_cache_write_scaled,
 * pa_copy_blocks_scaled and pa_decode_scaled take pools of PA_FP8_E4M3 or PA_INT8
 * codes beside float scale arrays; the other calls refuse PA_INT8.
 *
 * Conventions:
 *   - Ownership: the caller owns every buffer, the decode workspace included.
 *     The library allocates no device memory; its module holds two static device
 *     arrays (the scratch of pa_decode_static_scratch, 32 MiB, and the job
 *     counters of pa_prefill_chunk, 8 KB), set up when the library is loaded.
 *   - Asynchrony: each call validates its arguments on the host and enqueues its
 *     kernels on `stream` (a cudaStream_t; NULL = legacy default stream).
 *     PA_OK means "validated and launched", not "finished".
 *   - Host validation errors (PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED) launch
 *     nothing.  A CUDA launch failure returns PA_ERR_CUDA.
 *   - Device-side index faults (a table entry outside the pool, a slot outside
 *     the pool, a context longer than its table, a copy pair outside the pool)
 *     never trap: the kernel ORs a PA_DEVERR_* bit into *err_flag (when
 *     err_flag is not NULL), skips the offending element and carries on.  The
 *     affected outputs are then unspecified.  Read the flag with pa_wait().
 *   - Every wait inside a kernel is bounded; a wait that runs out sets
 *     PA_DEVERR_TIMEOUT and the kernel returns early.
 *   - CUDA graphs: a captured call replays the values its host side chose at
 *     capture time.  Cache writes, block copies, unsplit decodes, split decodes of
 *     fp32 or fp8 pools or head_dim 64, and prefills with more than 8 jobs per
 *     SM (jobs = num_seqs * num_kv_heads * ceil(max_chunk * g / 256)) replay
 *     correctly, and so do pa_step_plan, pa_step_release, pa_prefill_packed and the
 *     calls for pools with block scales.  Issue directly, not from a graph: a split decode (pa_decode,
 *     pa_append_decode, pa_decode_static_scratch) of bf16 pools with head_dim 128,
 *     whose shared-prefix detection tags its flags with a per-call value (a replay
 *     would read the previous replay's table comparison), and a pa_prefill_chunk
 *     with at most 8 jobs per SM, whose work counter is tagged per call (a replay
 *     would find its count spent and skip jobs).
 *   - Programmatic dependent launch: the kernels of a call are chained with it,
 *     and the last kernel of a split decode signals early that a dependent may
 *     launch.  A kernel the caller launches right after a call, with
 *     cudaLaunchAttributeProgrammaticStreamSerialization, must call
 *     cudaGridDependencySynchronize() before it reads the call's outputs (stream
 *     order is unchanged for every other kernel and for copies).  The first
 *     kernel of a split bf16 decode is itself launched that way: until the
 *     kernel before it has finished it only reads block_tables and context_lens,
 *     so the kernel just before the call must not write those two after it has
 *     called cudaTriggerProgrammaticLaunchCompletion() (kernels that never call
 *     it count as finished before the call starts).
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

/* Exported entry points (the library is built with hidden default visibility). */
#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned pointer, ... */
    PA_ERR_UNSUPPORTED = 2,   /* valid but not built: dtype, head_dim, group size, ... */
    PA_ERR_OOM = 3,           /* block pool exhausted (host block manager) */
    PA_ERR_DEVICE_INDEX = 4,  /* a kernel flagged an out-of-range index (pa_wait) */
    PA_ERR_CUDA = 5,          /* a CUDA runtime call failed */
    PA_ERR_TIMEOUT = 6,       /* pa_wait gave up, or a kernel's bounded wait ran out */
    PA_ERR_NOT_FOUND = 7      /* unknown sequence id (host block manager) */
} pa_status;

typedef enum pa_dtype { PA_F32 = 0, PA_BF16 = 1, PA_FP8_E4M3 = 2, PA_INT8 = 3 } pa_dtype;

/* Bits a kernel ORs into *err_flag. */
#define PA_DEVERR_BLOCK_ID 1     /* block table entry outside [0, num_blocks) */
#define PA_DEVERR_SLOT 2         /* slot_mapping entry >= num_blocks * block_size */
#define PA_DEVERR_CONTEXT_LEN 4  /* context_len < 0, > max_context_len or > table capacity */
#define PA_DEVERR_PAIR 8         /* copy pair id outside [0, num_blocks) */
#define PA_DEVERR_TIMEOUT 16     /* a bounded in-kernel wait ran out */
#define PA_DEVERR_CHUNK 32       /* chunk_len < 0, > max_chunk or > context_len */
#define PA_DEVERR_PLAN 64        /* a step does not fit: lengths, tables, slots or free blocks */

/* The KV pool one call works on. */
typedef struct pa_cache_desc {
    int32_t num_blocks;
    int32_t num_kv_heads;
    int32_t block_size;   /* must be 16 */
    int32_t head_dim;     /* 64 or 128 */
    int32_t dtype;        /* pa_dtype */
    float k_scale;        /* PA_FP8_E4M3: dequantisation scale of the key pool (finite, > 0) */
    float v_scale;        /* PA_FP8_E4M3: the same for the value pool; both ignored otherwise */
} pa_cache_desc;

/* Version of this ABI (bumped on any signature or layout change). */
PA_API int32_t pa_abi_version(void);

/* Human-readable name of a status code (static storage). */
PA_API const char *pa_status_string(pa_status status);

/*
 * KV append through a slot mapping (reshape-and-cache).
 * For every token i < num_tokens with slot = slot_mapping[i] >= 0 and every kv
 * head h:  key_cache[slot / block_size][h][slot % block_size][:] = key[i][h][:]
 * and the same for value.  key/value: [num_tokens, num_kv_heads, head_dim].
 * slot < 0 is padding (skipped).  slot >= num_blocks * block_size sets
 * PA_DEVERR_SLOT and that token is skipped.  Two tokens with the same slot:
 * unspecified which one lands.  num_tokens == 0 launches nothing.
 * PA_FP8_E4M3 pools: key/value are bf16 and each element is stored as
 * e4m3(fp32(x) / k_scale) (v_scale for value), nearest even, saturated.
 * Source: chenxutan 3.1 (write the new token's K/V back into the cache) and 3.3
 * (append_slot: the token goes into the current block).
 */
PA_API pa_status pa_cache_write(const void *key, const void *value, const int64_t *slot_mapping,
                         int32_t num_tokens, void *key_cache, void *value_cache,
                         const pa_cache_desc *cache, int32_t *err_flag, void *stream);

/*
 * Copy-on-Write block copy.  For each pair p < num_pairs, (src, dst) =
 * (src_dst_pairs[2p], src_dst_pairs[2p+1]): block dst of key_cache and of
 * value_cache becomes a copy of block src (every kv head, slot and dim).
 * Pairs must be independent (no dst repeated, no dst that is also a src); the
 * host block manager only emits such pairs.  An id outside [0, num_blocks) sets
 * PA_DEVERR_PAIR and that pair is skipped.  num_pairs == 0 launches nothing.
 * Source: devpress teardown, 关键设计二 (allocate a new block, copy the shared
 * one into it, drop a reference to the old one).
 */
PA_API pa_status pa_copy_blocks(void *key_cache, void *value_cache, const int32_t *src_dst_pairs,
                         int32_t num_pairs, const pa_cache_desc *cache, int32_t *err_flag,
                         void *stream);

/*
 * Checked mode for copy pairs (host function, host pointer): PA_OK when every id of
 * the num_pairs (src, dst) pairs in src_dst_pairs[2 * num_pairs] lies in
 * [0, num_blocks), src != dst, no dst repeats and no block is both a source and a
 * destination -- the conditions under which pa_copy_blocks's result does not depend
 * on the order its pairs run in; PA_ERR_INVALID_ARG otherwise (also for negative
 * counts or a null pointer with num_pairs > 0); PA_ERR_OOM when the host scratch
 * of num_blocks bytes cannot be allocated.  Reads the pairs only; launches nothing.
 * The host block manager only emits valid pairs.
 */
PA_API pa_status pa_check_copy_pairs(const int32_t *src_dst_pairs, int32_t num_pairs, int32_t num_blocks);

/*
 * Bytes of workspace pa_decode needs for a split (partitioned) context:
 * partials of num_seqs * num_q_heads * ceil(max_context_len / partition_size)
 * partitions (head_dim fp32 accumulators plus a running max and sum each), then
 * the shared-prefix group area (a shared-token count, a 16-byte group record and
 * a table-comparison result per sequence, 32 bytes of counts and 512 bytes of
 * flags).  Returns 0 when partition_size <= 0
 * (no split, no workspace).
 */
PA_API size_t pa_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t head_dim,
                                int32_t max_context_len, int32_t partition_size);

/*
 * Number of kernels one pa_decode call with these arguments launches on its
 * stream (for launch accounting): 1 unsplit; 2 split (the
 * partition kernel and the combine); with a split, dtype PA_BF16, head_dim 128 and
 * num_seqs <= 4096 the shared-prefix detection kernel and the tcgen05 group tiles
 * run first (4), and for g = num_q_heads / num_kv_heads <= 4 also the 16-row
 * group kernel for small sibling groups (5).  0 when num_seqs <= 0 or the head
 * counts are not positive.  Pure host function.
 */
PA_API int32_t pa_decode_launches(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t dtype, int32_t partition_size);

/*
 * Decode attention over the paged cache, one query token per sequence:
 *   out[s][h][:] = sum_{t < L_s} softmax_t(scale * <query[s][h], K_s[t]>) V_s[t]
 * with L_s = context_lens[s], K_s[t] = key_cache[block_tables[s][t / 16]][h / g]
 * [t % 16][:] (V alike) and g = num_q_heads / num_kv_heads.  L_s == 0 gives 0.
 * Softmax is computed online in fp32 (running max and sum), products and sums in
 * fp32; bf16 outputs are rounded to nearest even from fp32.
 * partition_size == 0: each (sequence, kv head) is one work unit.
 * partition_size > 0 (a multiple of 16): the context is split into partitions of
 * that many tokens (split-K); each partition keeps its running max m_p, sum
 * l_p and unnormalised accumulator o_p in `workspace`, and a second kernel
 * combines them: out = sum_p e^{m_p - M} o_p / sum_p e^{m_p - M} l_p with
 * M = max_p m_p.  Sequences with a single partition are finished by the first
 * kernel.  With a split, bf16 caches, head_dim 128 and num_seqs <= 4096, adjacent
 * sequences whose block tables begin with the same block ids (forked siblings, a
 * common prompt; at least partition_size tokens of full blocks shared with the
 * previous sequence) read those shared full blocks once per group, with all the
 * group's queries against each K/V tile: for g = num_q_heads / num_kv_heads <= 4,
 * groups of 2 to 16 / g members on 16-row tensor-core tiles; groups of at least 4
 * members (at most 128 / g) on the tcgen05 tile kernel.  The result is the same
 * sum, and the shared blocks cross the memory bus once instead of once per
 * sibling (devpress teardown, 关键设计二: siblings point at the same physical
 * blocks).  workspace_bytes must be >= pa_decode_workspace_size(...) for the same
 * num_seqs, num_q_heads, head_dim, max_context_len and partition_size.
 * max_context_len bounds every context_lens[s] (larger sets PA_DEVERR_CONTEXT_LEN
 * and that sequence's outputs are unspecified).  num_seqs <= 16384.
 * Source: chenxutan 2.3 (one query token per step, bandwidth bound); devpress
 * teardown 核心代码拆解 (table lookup per logical block, scaled scores, softmax,
 * weighted V sum).
 */
PA_API pa_status pa_decode(const void *query, const void *key_cache, const void *value_cache,
                    const int32_t *block_tables, int32_t max_blocks_per_seq,
                    const int32_t *context_lens, int32_t max_context_len, int32_t num_seqs,
                    int32_t num_q_heads, float scale, int32_t partition_size, void *workspace,
                    size_t workspace_bytes, void *out, const pa_cache_desc *cache,
                    int32_t *err_flag, void *stream);

/*
 * One decode step in one call: pa_cache_write(key, value, slot_mapping,
 * num_tokens, ...) followed by pa_decode(...) on the same stream, with the same
 * results (the same kernels run).  The write and the decode's shared-prefix
 * detection run side by side and the decode kernels start without a launch gap
 * (programmatic dependent launch); everything that reads the cache still waits
 * for the write.  Copy-on-write pairs must be applied (pa_copy_blocks) before.
 * Both sets of arguments are validated before anything is launched; argument
 * meaning and errors are those of the two calls.  num_tokens == 0 skips the write.
 * Source: chenxutan 3.1 (each step writes the new token's K/V back into the
 * cache, then attends over it).
 */
PA_API pa_status pa_append_decode(const void *key, const void *value, const int64_t *slot_mapping,
                                  int32_t num_tokens, const void *query, void *key_cache,
                                  void *value_cache, const int32_t *block_tables,
                                  int32_t max_blocks_per_seq, const int32_t *context_lens,
                                  int32_t max_context_len, int32_t num_seqs, int32_t num_q_heads,
                                  float scale, int32_t partition_size, void *workspace,
                                  size_t workspace_bytes, void *out, const pa_cache_desc *cache,
                                  int32_t *err_flag, void *stream);

/*
 * pa_decode with its split-K scratch taken from a fixed array inside the library
 * instead of a caller-provided workspace.  The pages have no counterpart: this
 * exists for callers that cannot allocate device memory -- code running inside an
 * allocator's callbacks, in a process whose device memory is owned and capped by
 * another framework, or in a plugin handed only the step's tensors.  Arguments and
 * results are those of pa_decode without workspace/workspace_bytes.
 * Limit: pa_decode_workspace_size(num_seqs, num_q_heads, head_dim,
 * max_context_len, partition_size) must be <= PA_DECODE_STATIC_SCRATCH_BYTES
 * (32 MiB), else PA_ERR_UNSUPPORTED and nothing is launched.  Every GPU that loads
 * the library holds that array until the process exits.
 * The first call on a device looks up the array's device address (with that
 * device current); make it before any stream capture.  No allocation happens.
 * The address is kept for the life of the process: after cudaDeviceReset (or
 * anything else that destroys the device's primary context) the process must be
 * restarted before this entry point is called again on that device.
 * All calls share the one array and it keeps the last call's contents; nothing in
 * it needs to start at zero.  Calls whose kernels overlap on the GPU (different
 * streams, no ordering between them) race on the array and give wrong results:
 * order them on one stream or with events.
 */
#define PA_DECODE_STATIC_SCRATCH_BYTES (32u << 20)
PA_API pa_status pa_decode_static_scratch(const void *query, const void *key_cache,
                                          const void *value_cache, const int32_t *block_tables,
                                          int32_t max_blocks_per_seq, const int32_t *context_lens,
                                          int32_t max_context_len, int32_t num_seqs,
                                          int32_t num_q_heads, float scale, int32_t partition_size,
                                          void *out, const pa_cache_desc *cache, int32_t *err_flag,
                                          void *stream);

/*
 * Causal chunked prefill against the paged cache.  Sequence s has
 * C_s = chunk_lens[s] new query rows, the last C_s positions of its context of
 * L_s = context_lens[s] tokens (their K/V already written with pa_cache_write).
 * Row i < C_s sits at position p = L_s - C_s + i and
 *   out[s][i][h][:] = sum_{t <= p} softmax_t(scale * <query[s][i][h], K_s[t]>) V_s[t].
 * query/out: [num_seqs, max_chunk, num_q_heads, head_dim]; rows i >= C_s of out
 * are not written.  Requires dtype PA_BF16 and head_dim 128 (tcgen05 tensor-core
 * tiles, bf16 operands, fp32 accumulation in tensor memory).
 * A speculative-decoding verify step is the same operation: each sequence appends
 * its k_s draft tokens (pa_cache_write), then the k_s new positions attend
 * causally with chunk_lens[s] = k_s (chenxutan 5.4, speculative decoding: the
 * target model checks several proposed tokens in one pass).
 * Work distribution (no effect on results): a job is (sequence, kv head, 256
 * packed rows).  With at most 8 jobs per SM they are handed out from a work
 * counter, one of a static pool of 1,024; each call tags its counter with a
 * per-process ticket, so calls need no ordering between them and nothing is
 * reset.  A call whose kernel still runs after 1,024 later pa_prefill_chunk
 * calls of the process have started (impossible on one stream) sets
 * PA_DEVERR_TIMEOUT and its outputs are unspecified.  With more jobs per SM the
 * order is a fixed round robin.
 * Source: chenxutan 2.3 (prefill computes a whole prompt and is compute bound)
 * and 4.3/5.1 (long prompts are cut into chunks that run between decodes).
 */
PA_API pa_status pa_prefill_chunk(const void *query, const void *key_cache, const void *value_cache,
                           const int32_t *block_tables, int32_t max_blocks_per_seq,
                           const int32_t *context_lens, const int32_t *chunk_lens,
                           int32_t num_seqs, int32_t max_chunk, int32_t num_q_heads, float scale,
                           void *out, const pa_cache_desc *cache, int32_t *err_flag,
                           void *stream);

/*
 * One step's block tables, slot mapping and sequence starts, built on the GPU from
 * the requests' lengths: pa_bm_append_step for callers that keep tables, lengths and
 * free blocks on the device (no copy to or from the host, replayable from a graph).
 * Sequence s holds context_lens[s] tokens in the first ceil(context_lens[s] / 16)
 * entries of its table and appends counts[s] >= 0.  The blocks it lacks are popped
 * from free_blocks[0 .. *num_free), last entry first, sequence by sequence:
 *   block_tables[s][ceil(len / 16) ..] get the popped ids (other entries are kept),
 *   slot_mapping[i], for the i-th appended token of the step (sequence by sequence),
 *     = block * 16 + offset of its position; entries behind the last token become -1
 *     (padding, as the cache writes take it), up to slot_capacity,
 *   seq_starts[0 .. num_seqs] = where each sequence's tokens start (the exclusive sums
 *     of counts, then their total) -- also what pa_prefill_packed takes,
 *   new_context_lens[s] = len + count, *new_num_free = *num_free - blocks popped.
 * new_context_lens may be context_lens and new_num_free may be num_free (the step in
 * place); otherwise outputs and inputs must not overlap.  Sequences that share blocks
 * (forks) need the host manager's copy on write before they append.
 * All or nothing: a negative count or length, a table row, slot_mapping or the free
 * stack too short, or *num_free outside [0, free_capacity] sets PA_DEVERR_PLAN, and
 * then tables, lengths and stack height stay as they were (copied to the new ones),
 * every slot is -1 and every start 0.  Ids on the stack are not checked here (the
 * calls that use them do); a negative id gives slot -1 and PA_DEVERR_BLOCK_ID.
 * num_seqs <= 16384, slot_capacity <= 2^30.
 * Source: devpress teardown, 关键设计一 (append_slot takes a block from the free list
 * when the current one is full); chenxutan 3.3.
 */
PA_API pa_status pa_step_plan(const int32_t *counts, const int32_t *context_lens, int32_t num_seqs,
                              int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *free_blocks,
                              int32_t free_capacity, const int32_t *num_free, int64_t *slot_mapping,
                              int32_t slot_capacity, int32_t *seq_starts, int32_t *new_context_lens,
                              int32_t *new_num_free, int32_t *err_flag, void *stream);

/*
 * The return of finished sequences' blocks to pa_step_plan's stack: for every s with
 * finished[s] != 0, in order, its blocks are pushed in logical order (as
 * pa_bm_free_seq does for blocks nobody shares), their table entries become -1 and
 * new_context_lens[s] = 0; the other sequences keep theirs.  In place as above; all
 * or nothing (PA_DEVERR_PLAN) when a length does not fit its table or the stack its
 * capacity.  A block must be in one table only: blocks shared by a fork belong to
 * the host manager.  Ids are pushed as they stand; a negative one within a length sets
 * PA_DEVERR_BLOCK_ID too.
 */
PA_API pa_status pa_step_release(const int32_t *finished, const int32_t *context_lens, int32_t num_seqs,
                                 int32_t *block_tables, int32_t max_blocks_per_seq, int32_t *free_blocks,
                                 int32_t free_capacity, const int32_t *num_free, int32_t *new_context_lens,
                                 int32_t *new_num_free, int32_t *err_flag, void *stream);

/*
 * 8-bit cache with a scale per (block, kv head).  The pools hold one-byte codes in
 * the layout of the other pools, dtype PA_FP8_E4M3 or PA_INT8 (two's complement, -127
 * .. 127); key_scales and value_scales are float [num_blocks, num_kv_heads], and a
 * value is code * scale.  Nothing has to be calibrated: the scale follows the data.
 * (k_scale and v_scale of the descriptor are not used.)  head_dim 64 or 128; key,
 * value, query and out are bf16.
 *
 * The append: for the tokens of this call that go to block b, kv head h, let A be the
 * largest |x| over their finite elements, Q = 448 (e4m3) or 127 (int8), and
 *   need  = the smallest power of two with A <= need * Q, at least 2^-64;
 *   sigma = max(stored scale, need), or need when slot 0 of the block is among the
 *           call's (the block starts anew) or the stored scale is no finite positive number.
 * The tokens' codes are round(x / sigma), nearest even (infinities saturate; NaN is
 * the e4m3 NaN, or 0 in int8).  Where sigma is larger than the stored scale, the codes
 * of the block's other slots in front of the last one written become round(code *
 * stored / sigma).  Slots behind it, and all other blocks, are left as they are.
 * sigma is stored.  Powers of two make both roundings exact up to that one rounding.
 * key and value: [num_tokens, num_kv_heads, head_dim], a token's heads and dims
 * contiguous, tokens key_stride / value_stride elements apart (at least num_kv_heads *
 * head_dim, a multiple of 8), so that they can be views of one fused projection.
 * Slots as in pa_cache_write.  The tokens of one block must stand next to each other
 * in slot_mapping, as pa_bm_append_step and pa_step_plan put them (in any order, with
 * no padding in between); a block whose tokens stand in two places gets an unspecified
 * scale and codes.  Two tokens with the same slot: unspecified which one lands.
 * Scales need no initial value.
 * Source: chenxutan 5.3 (8-bit KV); devpress architecture figure (FP8/INT8).
 */
PA_API pa_status pa_cache_write_scaled(const void *key, const void *value, int64_t key_stride,
                                       int64_t value_stride, const int64_t *slot_mapping, int32_t num_tokens,
                                       void *key_cache, void *value_cache, float *key_scales,
                                       float *value_scales, const pa_cache_desc *cache, int32_t *err_flag,
                                       void *stream);

/* pa_copy_blocks for such pools: codes and scales of every pair's block. */
PA_API pa_status pa_copy_blocks_scaled(void *key_cache, void *value_cache, float *key_scales,
                                       float *value_scales, const int32_t *src_dst_pairs, int32_t num_pairs,
                                       const pa_cache_desc *cache, int32_t *err_flag, void *stream);

/* Bytes of workspace pa_decode_scaled needs: it depends on the heads only, not on the
 * number or length of the contexts.  0 for head counts that do not divide. */
PA_API size_t pa_decode_scaled_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);

/*
 * pa_decode over such pools: one query token per sequence,
 *   out[s][h][:] = sum_t softmax_t(scale * <query[s][h], K_s[t]>) V_s[t],
 * K_s[t] = key code * key_scales[block][kv head] (V alike).  Arguments and errors as in
 * pa_decode; L_s == 0 gives 0.  The scales of blocks in use are not negative and at most
 * 2^122 (the append leaves 2^-64 to 2^122).  The context is always split evenly over the
 * GPU; where it is cut depends on the other sequences' lengths, so in another batch a result may
 * differ by rounding (the order of the fp32 sums, and the 16-bit weights below).  Two kernels (one
 * where max_context_len < 512).  The workspace's contents need not be set and mean nothing
 * afterwards; calls that overlap on the GPU need workspaces of their own.  Replays correctly
 * from a graph, following context_lens.  num_seqs <= 16384 and
 * num_seqs * (max_context_len / 16 + 2) < 2^31.  Scores, sums and the accumulator are fp32;
 * probabilities times value scales are rounded to f16 for the product with V (2^-11 of each, or 2^-32
 * of the row's largest where that is more); the query is exact (elements below 2^-24 of
 * their head's largest: to 2^-32 of it).
 */
PA_API pa_status pa_decode_scaled(const void *query, const void *key_cache, const void *value_cache,
                                  const float *key_scales, const float *value_scales,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *context_lens, int32_t max_context_len, int32_t num_seqs,
                                  int32_t num_q_heads, float scale, void *workspace, size_t workspace_bytes,
                                  void *out, const pa_cache_desc *cache, int32_t *err_flag, void *stream);

/* Bytes of workspace pa_prefill_packed needs (its job list). */
PA_API size_t pa_prefill_packed_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                               int32_t num_kv_heads);

/*
 * Causal attention over whole prompts packed without padding, before (or without) any
 * cache: sequence s owns rows seq_starts[s] .. seq_starts[s + 1] - 1 (int32
 * [num_seqs + 1], ascending, as pa_step_plan writes it) of query, key, value and out, and
 *   out[i][h] = sum_{j <= i, j in s} softmax_j(scale * <query[i][h], key[j][h / g]>) value[j][h / g].
 * query, out: bf16 [num_tokens, num_q_heads, head_dim]; key, value: bf16 [num_tokens,
 * num_kv_heads, head_dim]; a token's heads and dims are contiguous, the tokens of query,
 * key and value *_stride elements apart (at least a token's size, a multiple of 8: views of
 * one fused projection are taken as they are); out is contiguous and must not overlap the
 * inputs.  head_dim 64 or 128, num_q_heads / num_kv_heads in {1, 2, 4, 8}.  Rows outside
 * every sequence are neither read as keys nor written.  Values and scores of keys
 * behind a row never reach it, infinities and NaN included (rows whose tile holds such a
 * value behind them are computed again, slowly: 16,384 tokens, 32/8 heads, the last value NaN: 37 ms
 * instead of 1.7).
 * A sequence whose starts do not ascend, leave [0, num_tokens] or span more than
 * max_seq_len tokens sets PA_DEVERR_CHUNK and is skipped.  num_seqs <= 16384.
 * tcgen05 tensor-core tiles, bf16 operands, fp32 accumulation, softmax statistics and
 * sums; probabilities are rounded to bf16 for the product with V.  Two kernels (the
 * first lists the jobs from the lengths, in `workspace`, whose contents need not be set;
 * calls that overlap on the GPU need workspaces of their own), or one for a few short
 * sequences (min(max_seq_len, num_tokens) * num_q_heads / num_kv_heads <= 256).  Replays correctly from a
 * graph, following seq_starts.
 * Source: chenxutan 2.3 (prefill computes the whole prompt, compute bound).
 */
PA_API pa_status pa_prefill_packed(const void *query, const void *key, const void *value, int64_t query_stride,
                                   int64_t key_stride, int64_t value_stride, const int32_t *seq_starts,
                                   int32_t num_seqs, int32_t num_tokens, int32_t max_seq_len,
                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                                   void *workspace, size_t workspace_bytes, void *out, int32_t *err_flag,
                                   void *stream);

/*
 * Wait for `stream` to finish (polling, at most timeout_ms milliseconds) and read
 * the device error flag.  *flag_out (if not NULL) receives the flag value.
 * Returns PA_OK, PA_ERR_DEVICE_INDEX (flag has an index bit), PA_ERR_TIMEOUT
 * (stream still busy, or the flag has PA_DEVERR_TIMEOUT) or PA_ERR_CUDA.
 * err_flag may be NULL (then only the wait is done).  Not for use during
 * stream capture.
 */
PA_API pa_status pa_wait(void *stream, const int32_t *err_flag, int32_t timeout_ms, int32_t *flag_out);

/*
 * Bound, in nanoseconds, of every wait inside the kernels launched from now on by
 * this process (mbarrier hand-overs between the warps of a CTA); 0 restores the
 * default of one second.  Returns the previous bound.  A wait that runs out sets
 * PA_DEVERR_TIMEOUT in *err_flag, and the kernel stops its work, waits (with the
 * default bound) for the copies and tensor-core operations it has in flight,
 * releases its tensor memory and returns; the outputs of that call are then
 * unspecified and later calls are unaffected.  It exists to exercise that path:
 * a bound of a few nanoseconds makes ordinary waits run out.  Not a per-call or
 * per-thread setting: it applies to launches from every host thread.
 * Source: none on the pages (failure handling of this library).
 */
PA_API uint64_t pa_set_wait_timeout_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
