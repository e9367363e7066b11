// pagedkv_weights.cuh -- what the two forms of the prompt-weights kernels
// (mma.sync in pagedkv_weights.cu, tcgen05 in pagedkv_weights_tc.cu) share.
// Internal only.
#pragma once

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_requant.cuh"
#include "pagedkv_tc.cuh"

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

namespace dev {

// 8-bit pools: the codes of the 128 keys from `from` (zeros from L on), loaded by
// a set of 128 threads (warps 4k .. 4k + 3) and widened into a swizzled bf16
// image [D / 64][128 rows][128 bytes]; a piece is 16 codes of a key.
template <int D, int BS, int kKind>
struct Codes {
  static constexpr int kKeys = 128;                      // = threads of the set
  static constexpr int kRowPieces = D / 16;
  static constexpr int kParts = 2;                       // held one at a time
  static constexpr int kPieces = kKeys * kRowPieces / kKeys / kParts;
  uint4 x[kPieces];

  __device__ __forceinline__ static int piece(int part, int u) {
    return (part * kPieces + u) * kKeys + (int)(threadIdx.x % kKeys);
  }

  // False when a key's block is outside the pool.
  __device__ __forceinline__ bool load(const PromptArgs& a, const int32_t* bt, int hk, int from, int L, int part) {
    bool ok = true;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = piece(part, u), key = from + i / kRowPieces;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (key >= L) continue;
      const int p = bt[key / BS];
      if (p < 0 || p >= a.num_blocks) {
        ok = false;
        continue;
      }
      x[u] = static_cast<const uint4*>(a.k_cache)[(((int64_t)p * BS + key % BS) * a.num_kv_heads + hk) * kRowPieces +
                                                  i % kRowPieces];
    }
    return ok;
  }

  __device__ __forceinline__ void store(unsigned char* img, int part) const {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = piece(part, u), r = i / kRowPieces;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[4];
        code_values<kKind == KV_DTYPE_FP8_E4M3>(w[k], v);
        o[2 * k] = pack2<false>(v[0], v[1]);
        o[2 * k + 1] = pack2<false>(v[2], v[3]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = 2 * (i % kRowPieces) + k;          // 8-element chunk of the row
        *reinterpret_cast<uint4*>(img + (c / 8) * (kKeys * 128) + sw128(r, c % 8)) =
            make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
  }

  // The other part, after the one that is held; then the image is complete.
  __device__ __forceinline__ bool finish(const PromptArgs& a, const int32_t* bt, int hk, int from, int L,
                                         unsigned char* img) {
    store(img, 0);
    const bool ok = load(a, bt, hk, from, L, 1);
    store(img, 1);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return ok;
  }
};

}  // namespace dev

// Row statistics and column sums on the tensor cores with TMEM accumulators;
// `tiles` row tiles of a.tile_tokens tokens at most per sequence (positive
// scale).
kv_status launch_prompt_tc(const PromptArgs& a, int head_dim, int block_size, kv_dtype dtype,
                           int tiles, cudaStream_t stream);

// At most this many rows (query tokens x grouped heads) per KV head: one pass
// over K with the scores kept in TMEM, on a cluster of `ctas` CTAs per
// (sequence, KV head).  few_rows_ctas is 0 when sequences of
// max_seq_len tokens do not fit the largest cluster.
constexpr int kFewRows = 32;
int few_rows_ctas(int batch, int num_kv_heads, int max_seq_len, int num_sms);
kv_status launch_prompt_few(const PromptArgs& a, int head_dim, int block_size, kv_dtype dtype, int ctas,
                            cudaStream_t stream);

}  // namespace pagedkv
