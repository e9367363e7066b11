// pagedkv_weights.cuh -- what the two forms of the prompt-weights kernels
// (mma.sync in pagedkv_weights.cu, tcgen05 in pagedkv_weights_tc.cu) share.
// Internal only.
#pragma once

#include "pagedkv_common.cuh"

namespace pagedkv {

struct PromptArgs {
  float* weights;            // [B, Hkv, stride]
  const void* q;             // bf16 [T, Hq, D]
  const void* k_cache;
  const float* k_scale;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start;
  float* stats;              // [T, Hq, splits, 2] (m, l)
  unsigned int* flags;
  int64_t stride;
  int batch, num_tokens, max_query_len, num_q_heads, num_kv_heads, num_blocks, max_blocks;
  int max_seq_len, part_tokens, splits, accumulate;
  float scale_log2;
  int tile_tokens;           // tcgen05 kernels: query tokens per 128-row tile
};

// Row and key range of sequence b; false (and a flag once per head) when its
// length or offsets are bad.  n == 0: no queries.
__device__ __forceinline__ bool prompt_rows(const PromptArgs& a, int b, int bs, int* q0, int* n, int* L) {
  *q0 = a.query_start[b];
  *n = a.query_start[b + 1] - *q0;
  *L = a.seq_lens[b];
  return *q0 >= 0 && *n >= 0 && *q0 <= a.num_tokens - *n && *n <= a.max_query_len && *L > 0 &&
         *n <= *L && *L <= a.max_seq_len && (int64_t)*L <= (int64_t)a.max_blocks * bs &&
         (int64_t)*L <= a.stride;
}


// Row statistics and column sums on the tensor cores with TMEM accumulators;
// `tiles` row tiles of a.tile_tokens tokens at most per sequence (positive
// scale).
kv_status launch_prompt_tc(const PromptArgs& a, int head_dim, int block_size, kv_dtype dtype,
                           int tiles, cudaStream_t stream);

// At most this many rows (query tokens x grouped heads) per KV head: one pass
// over K with the scores kept in TMEM, on a cluster of `ctas` CTAs per
// (sequence, KV head) (bf16 pools).  few_rows_ctas is 0 when sequences of
// max_seq_len tokens do not fit the largest cluster.
constexpr int kFewRows = 32;
int few_rows_ctas(int batch, int num_kv_heads, int max_seq_len, int num_sms);
kv_status launch_prompt_few(const PromptArgs& a, int head_dim, int block_size, int ctas,
                            cudaStream_t stream);

}  // namespace pagedkv
