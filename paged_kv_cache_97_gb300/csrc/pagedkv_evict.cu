// pagedkv_evict.cu -- eviction from the paged cache by accumulated attention
// weight: which tokens each (sequence, KV head) keeps (pagedkv_select_tokens)
// and the packing of the kept rows into the sequence's first blocks
// (pagedkv_evict_tokens).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cooperative_groups.h>

#include <mutex>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_requant.cuh"

namespace cg = cooperative_groups;

namespace pagedkv {
namespace {

using namespace dev;

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------
//
// One cluster of C CTAs per (sequence, KV head).  With L tokens, the last
// `recent` are kept; of the C = L - recent candidates, the k = budget - recent
// of largest weight, ties to the lowest position:
//   1. a radix select over the weights as 32-bit ordered integers, three
//      digits (11, 11, 10 bits) from the top, finds the k-th largest value T
//      and how many candidates equal to T are kept (r);
//   2. a counting pass and a writing pass place every candidate above T and
//      the first r equal to T in ascending order of position.
// Each CTA holds a contiguous slice of the candidates in shared memory (what
// does not fit is read again from global memory), so the weights are read
// once; histograms and counts of the other CTAs are read through distributed
// shared memory.

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kPasses = 3;

struct SelectArgs {
  const float* weights;      // [B, Hkv, stride]
  const int32_t* seq_lens;   // [B]
  int32_t* keep_idx;         // [B, Hkv, budget]
  int32_t* keep_len;         // [B]
  unsigned int* flags;
  int64_t stride;
  int num_kv_heads, budget, recent, max_len;
  int cap;                   // candidates of a slice kept in shared memory
};

// Ordered integer of a weight: larger weight, larger key; -0 equals +0, NaN
// counts as -inf.
__device__ __forceinline__ uint32_t order_key(float w) {
  uint32_t u = __float_as_uint(w);
  if (w != w) u = 0xff800000u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of v over the CTA's threads; `total` gets the sum.
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int s = lane < kSelWarps ? warp_sums[lane] : 0;
  int before = lane < warp ? s : 0;
  before = __reduce_add_sync(0xffffffffu, before);
  *total = __reduce_add_sync(0xffffffffu, s);
  __syncthreads();                                   // warp_sums may be written again
  return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  extern __shared__ uint32_t sel_smem[];
  uint32_t* hist = sel_smem;                         // [kPasses][kBins]
  uint32_t* keys = sel_smem + kPasses * kBins;       // [cap]
  __shared__ int warp_sums[kSelWarps], sh_bin, sh_need;
  __shared__ int sh_counts[2];                       // this CTA's (above, equal) counts
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C;                    // (sequence, KV head)
  const int b = row / a.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = a.keep_idx + (int64_t)row * a.budget;
  const int L = a.seq_lens[b];
  const bool bad = L <= 0 || L > a.max_len;          // (cluster-uniform)
  if (bad || L <= a.budget) {
    for (int i = rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads)
      out[i] = !bad && i < L ? i : -1;
    if (row % a.num_kv_heads == 0 && rank == 0 && tid == 0) {
      a.keep_len[b] = bad ? 0 : L;
      if (bad) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    }
    return;
  }
  if (row % a.num_kv_heads == 0 && rank == 0 && tid == 0) a.keep_len[b] = a.budget;
  const int cand = L - a.recent, k = a.budget - a.recent;
  for (int i = rank * kSelThreads + tid; i < a.recent; i += C * kSelThreads) out[k + i] = cand + i;
  if (k == 0) return;

  const int per = (cand + C - 1) / C;
  const int lo = min(rank * per, cand), n = min(cand - lo, per);   // this CTA's slice
  const float* w = a.weights + (int64_t)row * a.stride + lo;
  auto key_at = [&](int i) { return i < a.cap ? keys[i] : order_key(w[i]); };

  for (int i = tid; i < kPasses * kBins; i += kSelThreads) hist[i] = 0u;
  __syncthreads();
  uint32_t prefix = 0u, mask = 0u;
  int need = k;
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const int bins = pass == 2 ? 1024 : 2048;
    uint32_t* h = hist + pass * kBins;
    if (pass == 0) {
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t key = order_key(w[i]);
        if (i < a.cap) keys[i] = key;
        atomicAdd(&h[key >> 21], 1u);
      }
    } else {
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t key = key_at(i);
        if ((key & mask) == prefix) atomicAdd(&h[(key >> shift) & (bins - 1)], 1u);
      }
    }
    cluster.sync();
    // bins from the top: this thread's two, summed over the cluster
    uint32_t c0 = 0u, c1 = 0u;
    const int top = bins - 1 - 2 * tid;
    if (top > 0)
      for (int r = 0; r < C; ++r) {
        const uint32_t* o = cluster.map_shared_rank(h, r);
        c0 += o[top];
        c1 += o[top - 1];
      }
    int total;
    const int before = block_exclusive((int)(c0 + c1), warp_sums, &total);
    if (before < need && need <= before + (int)(c0 + c1)) {
      const bool first = need <= before + (int)c0;
      sh_bin = first ? top : top - 1;
      sh_need = need - before - (first ? 0 : (int)c0);
    }
    __syncthreads();
    need = sh_need;
    prefix |= (uint32_t)sh_bin << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    __syncthreads();                                 // sh_bin, sh_need may be written again
  }
  // T = prefix; all candidates above it and the first `need` equal to it.
  // Each warp takes a contiguous part of the slice.
  const int seg = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int s0 = min(warp * seg, n), s1 = min(s0 + seg, n);
  int above = 0, equal = 0;
  for (int i = s0 + lane; i < s1; i += 32) {
    const uint32_t key = key_at(i);
    above += key > prefix;
    equal += key == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  int total_above, total_equal;
  int above_before = block_exclusive(lane == 0 ? above : 0, warp_sums, &total_above);
  int equal_before = block_exclusive(lane == 0 ? equal : 0, warp_sums, &total_equal);
  above_before = __shfl_sync(0xffffffffu, above_before, 0);
  equal_before = __shfl_sync(0xffffffffu, equal_before, 0);
  if (tid == 0) {
    sh_counts[0] = total_above;
    sh_counts[1] = total_equal;
  }
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    const int* o = cluster.map_shared_rank(sh_counts, r);
    above_before += o[0];
    equal_before += o[1];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < s1 ? key_at(i) : 0u;
    const bool gt = i < s1 && key > prefix, eq = i < s1 && key == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    const int g = above_before + __popc(bg & below), e = equal_before + __popc(be & below);
    if (gt || (eq && e < need)) out[g + min(e, need)] = lo + i;
    above_before += __popc(bg);
    equal_before += __popc(be);
  }
  cluster.sync();                                    // peers may still read this CTA's counts
}

// ---------------------------------------------------------------------------
// Packing
// ---------------------------------------------------------------------------
//
// Row j of the packed sequence is token keep_idx[j] >= j of the old one (the
// list ascends), so a CTA that packs destination blocks in ascending order
// may work in place: the rows it stores lie before every row it still has to
// load, and the loads of one round are all done before its stores.  One CTA
// per (KV head, sequence, K or V); one warp per destination block and round,
// holding the whole block of one head in registers.  For 8-bit pools the warp
// also finds the block's new scale from the rows it holds.

constexpr int kEvictWarps = 8;

struct EvictArgs {
  void* cache[2];            // K, V
  float* scale[2];
  float* weights;            // [B, Hkv, weights_stride] or null
  const int32_t* block_tables;
  const int32_t* dst_tables;
  const int32_t* seq_lens;
  const int32_t* keep_idx;   // [B, Hkv, budget]
  const int32_t* keep_len;   // [B]
  unsigned int* flags;
  int64_t weights_stride;
  int max_blocks, dst_max_blocks, num_kv_heads, num_blocks, budget;
};

template <int D, int BS, int kKind>
__global__ void __launch_bounds__(kEvictWarps * 32) evict_kernel(const EvictArgs a) {
  constexpr bool kQ8 = kKind != KV_DTYPE_BF16, kFp8 = kKind == KV_DTYPE_FP8_E4M3;
  constexpr int kRow = D * (kQ8 ? 1 : 2) / 16;       // 16-byte pieces per row
  constexpr int kPer = BS * kRow / 32;               // pieces per lane
  const int h = blockIdx.x, b = blockIdx.y, kv = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads;
  const int L = a.seq_lens[b], m = a.keep_len[b];
  if (m < 0 || m > L || m > a.budget || (int64_t)L > (int64_t)a.max_blocks * BS ||
      (m + BS - 1) / BS > a.dst_max_blocks || (a.weights && L > a.weights_stride)) {
    if (threadIdx.x == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    return;
  }
  const int32_t* idx = a.keep_idx + ((int64_t)b * Hkv + h) * a.budget;
  bool bad = false;
  for (int j = threadIdx.x; j < m; j += blockDim.x) {
    const int t = idx[j];
    bad |= t >= L || t <= (j > 0 ? idx[j - 1] : -1);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_INDEX);
    return;
  }
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks;
  const int32_t* dt = a.dst_tables + (int64_t)b * a.dst_max_blocks;
  uint4* cache = static_cast<uint4*>(a.cache[kv]);
  float* scale = a.scale[kv];
  float* wrow = kv == 0 && a.weights ? a.weights + ((int64_t)b * Hkv + h) * a.weights_stride : nullptr;
  const int nblk = (m + BS - 1) / BS;
  for (int j0 = 0; j0 < nblk; j0 += kEvictWarps) {
    const int j = j0 + warp;                         // this warp's destination block
    bool move = j < nblk;
    const int rows = move ? min(BS, m - j * BS) : 0;
    int64_t slot = 0;                                // lane r: row r's source slot
    int dst = 0;
    float s = 0.0f, wt = 0.0f;
    if (move) {
      dst = dt[j];
      const int from = bt[j];
      const int t = lane < rows ? idx[j * BS + lane] : 0;
      const int sb = lane < rows ? bt[t / BS] : 0;
      const bool off = dst < 0 || dst >= a.num_blocks || sb < 0 || sb >= a.num_blocks;
      const bool still = from == dst && (lane >= rows || t == j * BS + lane);
      if (__any_sync(0xffffffffu, off)) {
        if (lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
        move = false;
      } else if (__all_sync(0xffffffffu, still)) {
        move = false;
      } else {
        slot = (int64_t)sb * BS + t % BS;
        if (kQ8 && lane < rows) s = scale[(int64_t)sb * Hkv + h];
        if (wrow && lane < rows) wt = wrow[t];
      }
    }
    uint4 x[kPer];
    if (move) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int piece = u * 32 + lane, r = piece / kRow;
        const int64_t sl = __shfl_sync(0xffffffffu, slot, r);
        if (r < rows) x[u] = cache[(sl * Hkv + h) * kRow + piece % kRow];
      }
    }
    float ns = 0.0f;
    if constexpr (kQ8) {
      if (move) {
        float amax = 0.0f;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          const int r = (u * 32 + lane) / kRow;
          const float sr = __shfl_sync(0xffffffffu, s, r);
          if (r < rows) amax = fmaxf(amax, codes_amax<kFp8>(x[u], sr));
        }
        ns = block_scale<kFp8>(warp_max(amax));
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          const int r = (u * 32 + lane) / kRow;
          const float sr = __shfl_sync(0xffffffffu, s, r);
          if (r < rows) x[u] = recode16<kFp8>(x[u], sr, ns);
        }
      }
    }
    __syncthreads();                                 // the round's loads are done
    if (move) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int piece = u * 32 + lane, r = piece / kRow;
        if (r < rows) cache[(((int64_t)dst * BS + r) * Hkv + h) * kRow + piece % kRow] = x[u];
      }
      if (kQ8 && lane == 0) scale[(int64_t)dst * Hkv + h] = ns;
      if (wrow && lane < rows) wrow[j * BS + lane] = wt;
    }
  }
}

template <int D, int BS>
kv_status launch_evict(const EvictArgs& a, kv_dtype dtype, int batch, cudaStream_t s) {
  const dim3 grid((unsigned)a.num_kv_heads, (unsigned)batch, 2);
  const int threads = kEvictWarps * 32;
  if (dtype == KV_DTYPE_INT8) evict_kernel<D, BS, KV_DTYPE_INT8><<<grid, threads, 0, s>>>(a);
  else if (dtype == KV_DTYPE_FP8_E4M3) evict_kernel<D, BS, KV_DTYPE_FP8_E4M3><<<grid, threads, 0, s>>>(a);
  else evict_kernel<D, BS, KV_DTYPE_BF16><<<grid, threads, 0, s>>>(a);
  return cuda_check(cudaGetLastError(), "evict_kernel launch");
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" {

kv_status pagedkv_select_tokens(int32_t* keep_idx, int32_t* keep_len, const float* weights,
                                int weights_stride, const int32_t* seq_lens, int batch,
                                int num_kv_heads, int max_seq_len, int budget, int recent,
                                void* stream) {
  if (batch < 0 || num_kv_heads <= 0 || max_seq_len <= 0 || weights_stride <= 0)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_select_tokens: bad sizes");
  if (budget <= 0 || recent < 0 || recent > budget)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_select_tokens: needs budget >= 1 and 0 <= recent <= budget");
  if (max_seq_len > weights_stride)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_select_tokens: max_seq_len %d exceeds the weights' rows of %d",
                max_seq_len, weights_stride);
  if (batch == 0) return KV_OK;
  if (!keep_idx || !keep_len || !weights || !seq_lens)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_select_tokens: NULL pointer");
  const int64_t rows = (int64_t)batch * num_kv_heads;
  // CTAs per row: slices of about 4096 candidates, at most 8 CTAs
  int C = 1;
  while (C < 8 && (int64_t)C * 4096 < max_seq_len) C *= 2;
  if (rows * C > 0x7fffffffLL)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_select_tokens: too many rows");
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  SelectArgs a = {};
  a.weights = weights;
  a.seq_lens = seq_lens;
  a.keep_idx = keep_idx;
  a.keep_len = keep_len;
  a.flags = di.flags;
  a.stride = weights_stride;
  a.num_kv_heads = num_kv_heads;
  a.budget = budget;
  a.recent = recent;
  a.max_len = max_seq_len;
  constexpr int kMostKeys = 40 * 1024;
  const int per = (max_seq_len + C - 1) / C;
  a.cap = per < kMostKeys ? per : kMostKeys;
  const size_t smem = (size_t)(kPasses * kBins + a.cap) * sizeof(uint32_t);
  {
    static std::mutex mu;
    static bool attr_set[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[di.device]) {
      st = cuda_check(cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)((kPasses * kBins + kMostKeys) * sizeof(uint32_t))),
                      "cudaFuncSetAttribute(select_kernel)");
      if (st != KV_OK) return st;
      attr_set[di.device] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, select_kernel, a), "select_kernel launch");
}

kv_status pagedkv_evict_tokens(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                               const int32_t* block_tables, int max_blocks_per_seq,
                               const int32_t* dst_block_tables, int dst_max_blocks,
                               const int32_t* seq_lens, const int32_t* keep_idx,
                               const int32_t* keep_len, int budget, float* weights,
                               int weights_stride, int batch, int num_blocks, int block_size,
                               int num_kv_heads, int head_dim, kv_dtype dtype, void* stream) {
  if (batch < 0 || num_blocks <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
      dst_max_blocks <= 0 || budget <= 0 || !valid_dtype(dtype) || (weights && weights_stride <= 0))
    return fail(KV_ERR_INVALID_ARG, "pagedkv_evict_tokens: bad sizes");
  if (head_dim != 64 && head_dim != 128)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_evict_tokens: head_dim must be 64 or 128");
  if (block_size != 16 && block_size != 32)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_evict_tokens: block_size must be 16 or 32");
  if (batch > 65535) return fail(KV_ERR_INVALID_ARG, "pagedkv_evict_tokens: at most 65535 sequences");
  if (batch == 0) return KV_OK;
  if (!k_cache || !v_cache || !block_tables || !dst_block_tables || !seq_lens || !keep_idx || !keep_len)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_evict_tokens: NULL pointer");
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return fail(KV_ERR_INVALID_ARG, "pagedkv_evict_tokens: the pools must be 16-byte aligned");
  const bool q8 = dtype != KV_DTYPE_BF16;
  if (q8 != (k_scale != nullptr) || q8 != (v_scale != nullptr))
    return fail(KV_ERR_INVALID_ARG,
                "pagedkv_evict_tokens: 8-bit pools need k_scale and v_scale; bf16 pools take NULL");
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  EvictArgs a = {};
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.weights = weights;
  a.block_tables = block_tables;
  a.dst_tables = dst_block_tables;
  a.seq_lens = seq_lens;
  a.keep_idx = keep_idx;
  a.keep_len = keep_len;
  a.flags = di.flags;
  a.weights_stride = weights_stride;
  a.max_blocks = max_blocks_per_seq;
  a.dst_max_blocks = dst_max_blocks;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  a.budget = budget;
  cudaStream_t s = (cudaStream_t)stream;
  if (head_dim == 128)
    return block_size == 32 ? launch_evict<128, 32>(a, dtype, batch, s) : launch_evict<128, 16>(a, dtype, batch, s);
  return block_size == 32 ? launch_evict<64, 32>(a, dtype, batch, s) : launch_evict<64, 16>(a, dtype, batch, s);
}

}  // extern "C"
