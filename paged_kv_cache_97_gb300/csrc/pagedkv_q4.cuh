// pagedkv_q4.cuh -- the 4-bit pool's records, shared by the kernels that write
// and read them.  Internal only.
//
// One record per (physical block, KV head): the codes of K, the codes of V,
// then the (scale, min) bf16 pairs of K and of V, one pair per 64 values of a
// row; a code c in 0..15 stands for min + scale * c.  Everything an attention
// CTA needs of a block is one contiguous, 16-byte aligned piece of
// BS * D * 9 / 8 bytes (2304 for 16 tokens of 128), which one bulk copy moves.
//
// Element e of a row is nibble e % 8 of 32-bit word (e % 64 / 8) * (D / 64) +
// e / 64 of its codes: the words of equal place in every 64-group are
// neighbours, so that a lane reads its share of all groups with one load.
#pragma once

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"

namespace pagedkv {

template <int D, int BS>
struct Geo4 {
  static constexpr int kGroups = D / 64;
  static constexpr int kRowBytes = D / 2;                 // codes of a row
  static constexpr int kParBytes = kGroups * 4;           // (scale, min) pairs of a row
  static constexpr int kCodes = BS * kRowBytes;           // one tensor's codes
  static constexpr int kParams = BS * kParBytes;
  static constexpr int kParAt = 2 * kCodes;               // K's pairs; V's follow
  static constexpr int kRecord = 2 * (kCodes + kParams);
};

// Byte of a record where row `row` of tensor x (0 K, 1 V) has its codes / pairs.
__device__ __forceinline__ int q4_codes_at(int x, int row, int bs, int d) {
  return (x * bs + row) * (d / 2);
}
__device__ __forceinline__ int q4_pairs_at(int x, int row, int bs, int d) {
  return bs * d + (x * bs + row) * (d / 16);
}

// `bytes` consecutive bytes into shared memory, counted on a barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------------------
// Long queries (pagedkv_q4_tc.cu): sequences whose query tokens x grouped heads
// fill a 128-row tile at least, as many of them as there are slots for.
//
// Both ways measured (GB300, 8 KV heads of 128, us; rows of a sequence: as few
// queries / through images), by sequences and their lengths:
//                         128 rows    256 rows    512 rows
//   64 of 512..4096        464 / 258   878 / 280  1690 / 378
//   16 of 512..4096        159 /  96   253 / 107   459 / 137
//    4 of 1024..4096        53 /  68    85 /  77   141 /  79
//    1 of 8192              52 / 111    68 / 129   104 / 131
//    1 of 32768            110 / 364   183 / 425   333 / 427
// Images pay from the first whole tile on where there are sequences enough to give
// every SM a pair of tiles; the few sequences that do not have a chunk's keys worked
// off by one CTA per pair, and would be the faster as few queries up to 512 rows.
// The rule looks at the rows alone: how many sequences are long is known on the
// device only, and a caller who knows better gives the smaller workspace.
// ---------------------------------------------------------------------------

constexpr int kLongRows = 128;

struct Q4LongArgs {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const unsigned char* kv;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start;
  unsigned int* flags;
  int* slot_of;                // [batch]: a sequence's slot, or -1 (written by the plan)
  // set by launch_q4_long
  unsigned char* images;       // [slots, Hkv, chunks, 2, 128 rows] fp16 operand images of K and V
  int2* exps;                  // [slots, Hkv, chunks]: their powers of two
  int* list;                   // [slots]: the listed sequences
  int* bad;                    // [slots]: a block outside the pool
  int* counters;               // [2]: sequences listed, units taken
  int slots, chunks;
  int max_blocks, batch, num_tokens, max_query_len, num_kv_heads, group, head_dim, num_blocks, block_size, max_seq_len;
  float scale_log2;
};

// Bytes of a slot, and of the plan with `batch` slot_of entries before it.
size_t q4_slot_bytes(int num_kv_heads, int head_dim, int max_seq_len);
size_t q4_plan_bytes(int batch, int slots);
// Plan, images and attention of the long sequences; `memory` (128-byte aligned)
// holds slots * q4_slot_bytes and the lists.
kv_status launch_q4_long(Q4LongArgs a, void* memory, int sms, cudaStream_t s);

}  // namespace pagedkv
