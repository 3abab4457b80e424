// Internal launch interface of the serving-step operators: the step plan, the 8-bit
// cache with a scale per (block, kv head), and attention over packed prompts.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "pa.h"

namespace pa {

// ---- step plan ------------------------------------------------------------------
constexpr int32_t kMaxPlanSeqs = 16384;  // lengths and two prefix sums live in shared memory

struct StepPlan {
    const int32_t *counts;   // tokens to append (release: nonzero = finished)
    const int32_t *lens;
    int32_t num_seqs;
    int32_t *tables;
    int32_t max_blocks;
    const int32_t *free_blocks;
    int32_t *free_out;       // release: the same stack, written
    int32_t free_capacity;
    const int32_t *num_free;
    int64_t *slots;
    int32_t slot_capacity;
    int32_t *starts;
    int32_t *new_lens;       // may be lens
    int32_t *new_num_free;   // may be num_free
    int32_t *err;
};

cudaError_t launch_step_plan(const StepPlan &p, bool release, cudaStream_t stream);

// ---- 8-bit cache with a scale per (block, kv head) --------------------------------
struct ScaledPool {
    void *kc, *vc;           // codes [num_blocks][Hkv][16][head_dim]
    float *ks, *vs;          // scales [num_blocks][Hkv]
    int32_t num_blocks, num_kv_heads, head_dim;
    bool int8;               // codes are int8, else e4m3
};

struct ScaledWrite {
    const void *key, *value;  // bf16 rows [T][Hkv][head_dim], tokens key_stride / value_stride elements apart
    int64_t key_stride, value_stride;
    const int64_t *slots;
    int32_t num_tokens;
    ScaledPool pool;
    int32_t *err;
};

cudaError_t launch_cache_write_scaled(const ScaledWrite &w, cudaStream_t stream);
cudaError_t launch_copy_blocks_scaled(const ScaledPool &pool, const int32_t *pairs, int32_t num_pairs, int32_t *err,
                                      cudaStream_t stream);

struct ScaledDecode {
    const void *query;       // [S][Hq][head_dim] bf16
    ScaledPool pool;
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *lens;
    int32_t max_context;
    int32_t num_seqs, num_q_heads;
    float scale;
    void *workspace;
    void *out;
    int32_t *err;
};

size_t scaled_decode_workspace(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
cudaError_t launch_decode_scaled(const ScaledDecode &a, cudaStream_t stream);

// ---- attention over packed prompts ---------------------------------------------------
struct PackedPrefill {
    const void *query, *key, *value;              // bf16 [T][heads][head_dim], tokens strided (elements)
    int64_t q_stride, k_stride, v_stride;
    const int32_t *starts;
    int32_t num_tokens, num_seqs, max_seq_len, num_q_heads, num_kv_heads, head_dim;
    float scale;
    void *workspace;
    void *out;                                    // [T][Hq][head_dim]
    int32_t *err;
};

size_t packed_workspace(int32_t num_tokens, int32_t num_seqs, int32_t g);
cudaError_t launch_prefill_packed(const PackedPrefill &a, cudaStream_t stream);

}  // namespace pa
