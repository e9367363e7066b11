// pagedkv_append_scaled.cu -- append into an 8-bit pool whose per-(block, KV
// head) scales follow the data (“让 Agent 跑得快：LLM 推理服务”, §四 FP8 量化;
// “The engineering behind LLM inference” notes, §3.2): reshape_and_cache codes
// a row under the scale it is given, this append makes the scale.
//
// Sequence b's n_b new tokens are its last ones.  One warp per (sequence,
// touched block, KV head, K or V): it holds the block's new rows of that head
// in registers, finds their largest magnitude, and sets the block's scale to
//   max(old scale, amax / 127 or 448),   without the old one when row 0 of the
// block is among the new rows (the token opens the block).  When the scale
// grows, the rows already in the block are coded again under the new one.
// Warps never share a block, so there are no atomics and no second pass.
//
// The arithmetic of the codes and the loads' latency bound it together (issue
// slots 59 %, DRAM 51 % in use): eight prompts of 1..8K tokens (8 heads of 128)
// take 52 us on E4M3, 4470 GB/s or 66 % of the copy rate (84 us with a division
// per element), and 67 us on int8; 128 single tokens 10.6 us, the call itself.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_requant.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kAppendWarps = 4;

struct AppendArgs {
  const uint4* rows[2];      // new K, V: bf16 [num_tokens, Hkv, D]
  void* cache[2];
  float* scale[2];
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start;  // [batch + 1], or null: one token per sequence
  unsigned int* flags;
  int64_t units;             // batch * touched * Hkv * 2
  int touched;               // blocks a sequence's new tokens may touch, at most
  int max_blocks, num_tokens, max_query_len, num_blocks, num_kv_heads;
};

template <int D, int BS, bool kFp8>
__global__ void __launch_bounds__(kAppendWarps * 32) append_scaled_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 16;                     // lanes per row, 16 elements each
  constexpr int kRows = 32 / kLanes;                 // rows per step
  constexpr int kSteps = BS / kRows;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  // K and V of one (block, head) are neighbours, then the heads of a block
  const int kv = (int)(unit & 1), Hkv = a.num_kv_heads;
  const int h = (int)((unit >> 1) % Hkv);
  const int64_t bj = (unit >> 1) / Hkv;
  const int j = (int)(bj % a.touched), b = (int)(bj / a.touched);
  int q0 = b, n = 1;
  if (a.query_start) {
    q0 = a.query_start[b];
    n = a.query_start[b + 1] - q0;
  }
  const int L = a.seq_lens[b];
  if (n == 0) return;
  if (q0 < 0 || n < 0 || q0 > a.num_tokens - n || n > L || n > a.max_query_len) {
    if (j == 0 && lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    return;
  }
  const int first = L - n;                           // position of the first new token
  const int lb = first / BS + j;
  if ((int64_t)lb * BS >= L) return;
  if (lb >= a.max_blocks) {
    if (lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    return;
  }
  const int p = a.block_tables[(int64_t)b * a.max_blocks + lb];
  if (p < 0 || p >= a.num_blocks) {
    if (lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
    return;
  }
  const int r0 = max(first - lb * BS, 0), r1 = min(L - lb * BS, BS);  // the new rows
  const uint4* src = kv ? a.rows[1] : a.rows[0];
  float* scale = (kv ? a.scale[1] : a.scale[0]) + (int64_t)p * Hkv + h;
  const int sub = lane / kLanes, piece = lane % kLanes;
  uint4 x[kSteps][2];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int r = u * kRows + sub;
    if (r >= r0 && r < r1) {
      const int64_t token = (int64_t)q0 + (lb * BS + r - first);
      const uint4* at = src + (token * Hkv + h) * (D / 8) + 2 * piece;
      x[u][0] = at[0];
      x[u][1] = at[1];
    }
  }
  const float old = r0 > 0 ? *scale : 0.0f;
  // The magnitudes of finite bf16 values order as their bits do, and every
  // non-finite one is above them.
  uint32_t most = 0u;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int r = u * kRows + sub;
    if (r >= r0 && r < r1) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        most = max_u16x2(max_u16x2(max_u16x2(most, x[u][k].x & 0x7fff7fffu), x[u][k].y & 0x7fff7fffu),
                         max_u16x2(x[u][k].z & 0x7fff7fffu, x[u][k].w & 0x7fff7fffu));
    }
  }
  const uint32_t bits = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
  float amax = __uint_as_float(bits << 16);
  const bool finite = bits < 0x7f80u;
  if (!finite) {
    amax = 0.0f;
    for (int u = 0; u < kSteps; ++u) {
      const int r = u * kRows + sub;
      if (r < r0 || r >= r1) continue;
      const int64_t token = (int64_t)q0 + (lb * BS + r - first);
      const __nv_bfloat16* at = reinterpret_cast<const __nv_bfloat16*>(src) + (token * Hkv + h) * D + 16 * piece;
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, finite_abs(__bfloat162float(at[i])));
    }
    amax = warp_max(amax);
  }
  const float made = block_scale<kFp8>(amax);
  const float s = fmaxf(old, made);                  // (a NaN old scale gives way)
  uint4* pool = static_cast<uint4*>(kv ? a.cache[1] : a.cache[0]);
  const int64_t base = ((int64_t)p * BS * Hkv + h) * kLanes + piece;  // row r: + r * Hkv * kLanes
  if (s > old && r0 > 0) {
    const Interval again = quotients(old, s);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int r = u * kRows + sub;
      if (r < r0) {
        uint4* at = pool + base + (int64_t)r * Hkv * kLanes;
        *at = recode16<kFp8>(*at, again, old, s);
      }
    }
  }
  Interval q = quotients(s);
  q.on &= finite;                                    // (an infinity saturates, NaN has its code)
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int r = u * kRows + sub;
    if (r >= r0 && r < r1) {
      pool[base + (int64_t)r * Hkv * kLanes] = code16<kFp8>(x[u][0], x[u][1], q, s);
    }
  }
  if (lane == 0) *scale = s;
}

template <int D, int BS>
kv_status launch_append(const AppendArgs& a, kv_dtype dtype, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.units + kAppendWarps - 1) / kAppendWarps);
  if (dtype == KV_DTYPE_INT8) append_scaled_kernel<D, BS, false><<<grid, kAppendWarps * 32, 0, s>>>(a);
  else append_scaled_kernel<D, BS, true><<<grid, kAppendWarps * 32, 0, s>>>(a);
  return cuda_check(cudaGetLastError(), "append_scaled_kernel launch");
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" kv_status pagedkv_append_scaled(const void* new_k, const void* new_v, void* k_cache,
                                           void* v_cache, float* k_scale, float* v_scale,
                                           const int32_t* block_tables, int max_blocks_per_seq,
                                           const int32_t* seq_lens, const int32_t* query_start,
                                           int batch, int num_tokens, int max_query_len,
                                           int num_blocks, int block_size, int num_kv_heads,
                                           int head_dim, kv_dtype dtype, void* stream) {
  if (batch < 0 || num_tokens < 0 || max_query_len <= 0 || num_blocks <= 0 || num_kv_heads <= 0 ||
      max_blocks_per_seq <= 0)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_append_scaled: bad sizes");
  if (dtype != KV_DTYPE_INT8 && dtype != KV_DTYPE_FP8_E4M3)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_append_scaled: the pools must be int8 or E4M3");
  if (head_dim != 64 && head_dim != 128)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_append_scaled: head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_append_scaled: block_size must be 16 or 32");
  if (!query_start && (num_tokens != batch))
    return fail(KV_ERR_INVALID_ARG,
                "pagedkv_append_scaled: without query_start there is one token per sequence");
  if (batch == 0 || num_tokens == 0) return KV_OK;
  if (!new_k || !new_v || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !seq_lens)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_append_scaled: NULL pointer");
  if (!aligned16(new_k) || !aligned16(new_v) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(KV_ERR_INVALID_ARG,
                "pagedkv_append_scaled: the new rows and the pools must be 16-byte aligned");
  AppendArgs a = {};
  const int longest = query_start ? (max_query_len < num_tokens ? max_query_len : num_tokens) : 1;
  a.touched = (longest + block_size - 2) / block_size + 1;
  a.units = (int64_t)batch * a.touched * num_kv_heads * 2;
  if ((a.units + kAppendWarps - 1) / kAppendWarps > 0x7fffffffLL)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_append_scaled: too many tokens");
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  a.rows[0] = static_cast<const uint4*>(new_k);
  a.rows[1] = static_cast<const uint4*>(new_v);
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.flags = di.flags;
  a.max_blocks = max_blocks_per_seq;
  a.num_tokens = num_tokens;
  a.max_query_len = query_start ? max_query_len : 1;
  a.num_blocks = num_blocks;
  a.num_kv_heads = num_kv_heads;
  cudaStream_t s = (cudaStream_t)stream;
  if (head_dim == 128)
    return block_size == 32 ? launch_append<128, 32>(a, dtype, s) : launch_append<128, 16>(a, dtype, s);
  return block_size == 32 ? launch_append<64, 32>(a, dtype, s) : launch_append<64, 16>(a, dtype, s);
}
