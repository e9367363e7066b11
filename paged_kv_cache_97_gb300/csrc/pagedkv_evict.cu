// pagedkv_evict.cu -- eviction from the paged cache by accumulated attention
// weight: which tokens each (sequence, KV head) keeps (pagedkv_select_tokens)
// and the packing of the kept rows into the sequence's first blocks
// (pagedkv_evict_tokens).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cooperative_groups.h>

#include <mutex>
#include <type_traits>

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
// `recent` are kept; of the L - recent candidates, the k = budget - recent of
// largest weight, ties to the lowest position.  A radix select over the
// weights as 32-bit ordered integers, digits of 11, 11 and 10 bits from the
// top, finds the k-th largest key T and how many candidates equal to T are
// kept.  Each CTA holds a contiguous slice of the candidates in shared memory
// (what does not fit is read again from global memory) and two bits per
// candidate, in chunks of 32: "kept" (its leading digits are above T's) and
// "open" (equal so far).  The first two digits go over all keys, after which
// few are open, and the rest is done by one thread per chunk on its open bits
// alone.  Histograms and counts of the other CTAs are read through distributed
// shared memory; the chunks' counts give every kept position its place, in
// ascending order.
//
// What bounds it is the chain of barriers and shared-memory steps (a digit:
// histogram, two cluster barriers, a scan), not bytes: 64 x 8 rows of 512..4096
// tokens take 12.3 us, 8 x 8 rows of 131072 tokens 37 us, in two waves of
// clusters (4 x 8 rows: 24.6).  Longer rows on 256-thread CTAs four to an SM,
// with most keys read again from L2, came to 34 us there but to 33 instead of
// 17.8 for one row, and were not taken.

constexpr int kBins = 2048;
constexpr int kPasses = 3;
template <int n>
using Bins = std::integral_constant<int, n>;
constexpr int kMostCtas = 8;                         // of a cluster
constexpr int kBatch = 4;                            // loads in flight per thread

struct SelectArgs {
  const float* weights;      // [B, Hkv, stride]
  const int32_t* seq_lens;   // [B]
  int32_t* keep_idx;         // [B, Hkv, budget]
  int32_t* keep_len;         // [B]
  unsigned int* flags;
  int64_t stride;
  int num_kv_heads, budget, recent, max_len;
  int cap;                   // candidates of a slice kept in shared memory
  int chunk_cap;             // 32-candidate chunks of the longest slice
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
template <int kThreads>
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int* total) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int s = lane < kWarps ? warp_sums[lane] : 0;
  int before = lane < warp ? s : 0;
  before = __reduce_add_sync(0xffffffffu, before);
  *total = __reduce_add_sync(0xffffffffu, s);
  __syncthreads();                                   // warp_sums may be written again
  return before + x - v;
}

// Four CTAs of 256 threads per SM (64 registers): the barriers and histogram
// adds of one wait while others run.  64 x 8 rows: of 4096 tokens 18.7 -> 14.6
// us against two CTAs per SM, of 8192 43 -> 35.6, of 32768 172 -> 140; 64 x 8
// rows of mixed 512..4096 tokens, which two per SM balance better, 12.3 ->
// 13.5.  The 512-thread form (longer rows, fewer of them) gains nothing from a
// third CTA (8 x 8 rows of 131072 tokens: 37.8 us with two, 40.0 with three).
template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 2) select_kernel(const SelectArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t sel_smem[];
  uint32_t* hist = sel_smem;                         // [kPasses][kBins]
  __shared__ int warp_sums[kWarps], sh_bin, sh_need;
  __shared__ int sh_counts[2];                       // this CTA's (above, equal) counts
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C;                    // (sequence, KV head)
  const int b = row / a.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = a.keep_idx + (int64_t)row * a.budget;
  for (int i = tid; i < kPasses * kBins / 4; i += kThreads)
    reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  const int L = a.seq_lens[b];
  const bool bad = L <= 0 || L > a.max_len;          // (cluster-uniform)
  if (bad || L <= a.budget) {
    for (int i = rank * kThreads + tid; i < a.budget; i += C * kThreads)
      out[i] = !bad && i < L ? i : -1;
    if (row % a.num_kv_heads == 0 && rank == 0 && tid == 0) {
      a.keep_len[b] = bad ? 0 : L;
      if (bad) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    }
    return;
  }
  if (row % a.num_kv_heads == 0 && rank == 0 && tid == 0) a.keep_len[b] = a.budget;
  const int cand = L - a.recent, k = a.budget - a.recent;
  for (int i = rank * kThreads + tid; i < a.recent; i += C * kThreads) out[k + i] = cand + i;
  if (k == 0) return;

  const int per = (cand + C - 1) / C;
  const int lo = min(rank * per, cand), n = min(cand - lo, per);   // this CTA's slice
  const float* w = a.weights + (int64_t)row * a.stride + lo;
  const int chunks = (n + 31) / 32;
  uint32_t* shared_sums = hist + kPasses * kBins;    // [kBins]
  uint32_t* open = shared_sums + kBins;              // [chunks of a slice], then as many kept
  uint32_t* kept = open + a.chunk_cap;
  uint32_t* keys = kept + a.chunk_cap;               // [cap]
  auto key_at = [&](int i) { return i < a.cap ? keys[i] : order_key(w[i]); };
  __syncthreads();                                   // the histograms are zero

  // first digit of every key; a batch of loads is under way at a time
  for (int i0 = tid; i0 < n; i0 += kThreads * kBatch) {
    float x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (i0 + u * kThreads < n) x[u] = w[i0 + u * kThreads];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kThreads;
      if (i < n) {
        const uint32_t key = order_key(x[u]);
        if (i < a.cap) keys[i] = key;
        atomicAdd(&hist[key >> 21], 1u);
      }
    }
  }
  uint32_t prefix = 0u;
  int need = k;
  // The digit of T among `h`'s bins from the top, summed over the cluster:
  // each CTA adds up its share of the bins and hands the sums to all (every
  // CTA reading every peer's whole histogram took eight times the traffic).
  auto digit = [&](const uint32_t* h, auto bins) {
    constexpr int kBinsOf = decltype(bins)::value;
    const uint32_t* sums = h;
    if (C > 1) {
      cluster.sync();
      const int share = kBinsOf / C;
      for (int i = rank * share + tid; i < (rank + 1) * share; i += kThreads) {
        uint32_t v = 0u;
#pragma unroll
        for (int r = 0; r < kMostCtas; ++r)
          if (r < C) v += cluster.map_shared_rank(h, r)[i];
#pragma unroll
        for (int r = 0; r < kMostCtas; ++r)
          if (r < C) cluster.map_shared_rank(shared_sums, r)[i] = v;
      }
      cluster.sync();
      sums = shared_sums;
    } else {
      __syncthreads();
    }
    constexpr int run = kBinsOf / kThreads;          // bins per thread, loaded as vectors
    const int top = kBinsOf - 1 - run * tid;
    int c[run], sum = 0;                             // from the top down
    if constexpr (run >= 4) {
#pragma unroll
      for (int i = 0; i < run; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(sums + top - i - 3);
        c[i] = (int)v.w, c[i + 1] = (int)v.z, c[i + 2] = (int)v.y, c[i + 3] = (int)v.x;
      }
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(sums + top - 1);
      c[0] = (int)v.y, c[1] = (int)v.x;
    }
#pragma unroll
    for (int i = 0; i < run; ++i) sum += c[i];
    int total;
    int before = block_exclusive<kThreads>(sum, warp_sums, &total);
    if (before < need && need <= before + sum) {
      int at = top;
#pragma unroll
      for (int i = 0; i < run; ++i) {
        if (before + c[i] >= need) break;
        before += c[i];
        --at;
      }
      sh_bin = at;
      sh_need = need - before;
    }
    __syncthreads();
    need = sh_need;
    return (uint32_t)sh_bin;                         // (written again after further barriers only)
  };
  prefix = digit(hist, Bins<kBins>()) << 21;

  // second digit of the open keys; the chunks' bits
  uint32_t* h2 = hist + kBins;
  for (int c0 = warp; c0 < chunks; c0 += kWarps * kBatch) {
    uint32_t key[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = (c0 + u * kWarps) * 32 + lane;
      key[u] = i < n ? key_at(i) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int c = c0 + u * kWarps;
      if (c >= chunks) break;
      const bool in = c * 32 + lane < n;
      const bool eq = in && (key[u] >> 21) == (prefix >> 21);
      const uint32_t bo = __ballot_sync(0xffffffffu, eq);
      const uint32_t bk = __ballot_sync(0xffffffffu, in && (key[u] >> 21) > (prefix >> 21));
      if (eq) atomicAdd(&h2[(key[u] >> 10) & 2047u], 1u);
      if (lane == 0) {
        open[c] = bo;
        kept[c] = bk;
      }
    }
  }
  prefix |= digit(h2, Bins<kBins>()) << 10;

  // From here on a thread owns a run of chunks.  An open key whose bits above
  // `shift` are above T's is kept, one below is dropped.
  const int mine = (chunks + kThreads - 1) / kThreads;
  const int c_lo = min(tid * mine, chunks), c_hi = min(c_lo + mine, chunks);
  auto settle = [&](int shift, auto still) {
    for (int c = c_lo; c < c_hi; ++c) {
      uint32_t o = open[c], k_bits = kept[c];
      for (uint32_t left = o; left; left &= left - 1) {
        const int bit = __ffs((int)left) - 1;
        const uint32_t key = key_at(c * 32 + bit);
        if ((key >> shift) == (prefix >> shift)) {
          still(key);
        } else {
          o &= ~(1u << bit);
          if ((key >> shift) > (prefix >> shift)) k_bits |= 1u << bit;
        }
      }
      open[c] = o;
      kept[c] = k_bits;
    }
  };
  uint32_t* h3 = hist + 2 * kBins;
  settle(10, [&](uint32_t key) { atomicAdd(&h3[key & 1023u], 1u); });
  prefix |= digit(h3, Bins<1024>());                         // = T; `need` of the keys equal to it are kept
  settle(0, [](uint32_t) {});

  int above = 0, equal = 0;
  for (int c = c_lo; c < c_hi; ++c) {
    above += __popc(kept[c]);
    equal += __popc(open[c]);
  }
  int total_above, total_equal;
  int above_before = block_exclusive<kThreads>(above, warp_sums, &total_above);
  int equal_before = block_exclusive<kThreads>(equal, warp_sums, &total_equal);
  if (C > 1) {
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
  }
  for (int c = c_lo; c < c_hi; ++c) {
    const uint32_t eq = open[c];
    for (uint32_t left = eq | kept[c]; left; left &= left - 1) {
      const int bit = __ffs((int)left) - 1;
      if (eq >> bit & 1u) {
        if (equal_before < need) out[above_before + equal_before] = lo + c * 32 + bit;
        ++equal_before;
      } else {
        out[above_before + min(equal_before, need)] = lo + c * 32 + bit;
        ++above_before;
      }
    }
  }
  if (C > 1) cluster.sync();                         // peers may still read this CTA's counts
}

// Shared memory of a CTA at most, and the longest rows whose chunk bits fit it.
constexpr int kMostSmem = 200 * 1024;
constexpr int kMostTokens = 1 << 21;

template <int kThreads>
kv_status launch_select(const SelectArgs& a, int64_t rows, int C, int dev, cudaStream_t s) {
  static std::mutex mu;
  static bool attr_set[64] = {};
  kv_status st;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      st = cuda_check(cudaFuncSetAttribute(select_kernel<kThreads>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMostSmem),
                      "cudaFuncSetAttribute(select_kernel)");
      if (st != KV_OK) return st;
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)((kPasses + 1) * kBins + 2 * a.chunk_cap + a.cap) * sizeof(uint32_t);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, select_kernel<kThreads>, a), "select_kernel launch");
}

// ---------------------------------------------------------------------------
// Packing
// ---------------------------------------------------------------------------
//
// Row j of the packed sequence is token keep_idx[j] >= j of the old one (the
// list ascends), so a CTA that packs destination blocks in ascending order
// may work in place: the rows it stores lie before every row it still has to
// load, and the loads of one round are all done before its stores.  One CTA
// (or, in small batches, a cluster) per (KV head, sequence) and one of K, V and
// the weights; one warp per destination block and round, holding the whole
// block of one head in registers.  For 8-bit pools the warp also finds the
// block's new scale from the rows it holds.  Where no destination block is its own source, nothing is
// stored where anything is read and the warps run on without the barrier.
//
// bf16 is bound by HBM, 8-bit pools by the arithmetic of the codes (about nine
// issue slots per E4M3 code and eleven per int8 code, logic and permutes
// counting double).  128 sequences of 1..8K tokens packed to 2K: E4M3 276 us to
// fresh blocks, 284 in place (56 % of the copy rate), int8 372 and 302; four
// CTAs per SM with the registers held to 64 against three: 276 and 305.  64
// sequences of 512..4096 packed to 1K, bf16 in place: 85 us (90 %).  Tried and
// dropped: the rows a round ahead by asynchronous copies (321 -> 349 us), the
// lists and tables of several rounds staged in shared memory (352 -> 465).

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

// One destination block's codes: rows [0, rows) of 16-byte pieces from the
// byte offsets `from` (lane r: row r's) of `pool` to `to` + r * row_bytes,
// coded again under the block's own scale, which is returned.  scale_r: lane
// r's old scale.  `stored` is called between the loads and the stores.
// kFull: rows == BS.
template <int D, int BS, bool kFp8, bool kFull, class Barrier>
__device__ __forceinline__ float recode_block(unsigned char* pool, int64_t from, int64_t to, int64_t row_bytes,
                                              float scale_r, int rows, Barrier loaded) {
  constexpr int kRow = D / 16;                       // 16-byte pieces per row
  constexpr int kPer = BS * kRow / 32;               // pieces per lane
  constexpr int kStep = 32 / kRow;                   // rows per step
  const int lane = threadIdx.x & 31, sub = lane / kRow;
  const unsigned char* src = pool + (lane % kRow) * 16;
  uint4 x[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t off = __shfl_sync(0xffffffffu, from, u * kStep + sub);
    if (kFull || u * kStep + sub < rows) x[u] = *reinterpret_cast<const uint4*>(src + off);
    else x[u] = make_uint4(0u, 0u, 0u, 0u);
  }
  // |c * s| in fp32 grows with |c|, so a piece's largest code decides unless
  // its product is not finite
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const float s = __shfl_sync(0xffffffffu, scale_r, u * kStep + sub);
    amax = fmaxf(amax, fabsf(__fmul_rn(largest_code<kFp8>(x[u]), s)));  // (passes over NaN)
  }
  if (__any_sync(0xffffffffu, amax > kLargestFinite)) {
    amax = 0.0f;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      amax = fmaxf(amax, codes_amax_each<kFp8>(x[u], __shfl_sync(0xffffffffu, scale_r, u * kStep + sub)));
  }
  const float ns = block_scale<kFp8>(warp_max(amax));
  // lane r: the interval of row r's quotients
  const Interval q = quotients(scale_r, ns);
  const bool on = __all_sync(0xffffffffu, q.on || lane >= rows);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const float lo = __shfl_sync(0xffffffffu, q.lo, u * kStep + sub);
    const float hi = __shfl_sync(0xffffffffu, q.hi, u * kStep + sub);
    // (opaque here, or the values converted above would be kept for all pieces
    // and spill)
    asm volatile("" : "+r"(x[u].x), "+r"(x[u].y), "+r"(x[u].z), "+r"(x[u].w));
    uint4 o, off;
    const bool some = recode16_between<kFp8>(x[u], lo, hi, o, off);
    if (__any_sync(0xffffffffu, some) || !on)
      o = divide_words<kFp8>(x[u], o, off, __shfl_sync(0xffffffffu, scale_r, u * kStep + sub), ns, !on);
    x[u] = o;
  }
  loaded();
  unsigned char* dst = pool + to + sub * row_bytes + (lane % kRow) * 16;
#pragma unroll
  for (int u = 0; u < kPer; ++u)
    if (kFull || u * kStep + sub < rows) *reinterpret_cast<uint4*>(dst + u * kStep * row_bytes) = x[u];
  return ns;
}

template <int D, int BS, int kKind>
__global__ void __launch_bounds__(kEvictWarps * 32, kKind != KV_DTYPE_BF16 ? 4 : 2)
    evict_kernel(const EvictArgs a) {
  constexpr bool kQ8 = kKind != KV_DTYPE_BF16, kFp8 = kKind == KV_DTYPE_FP8_E4M3;
  constexpr int kRow = D * (kQ8 ? 1 : 2) / 16;       // 16-byte pieces per row
  constexpr int kPer = BS * kRow / 32;               // pieces per lane
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int h = blockIdx.x / C, b = blockIdx.y, kv = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hkv = a.num_kv_heads;
  const int L = a.seq_lens[b], m = a.keep_len[b];
  if (m < 0 || m > L || m > a.budget || (int64_t)L > (int64_t)a.max_blocks * BS ||
      (m + BS - 1) / BS > a.dst_max_blocks || (a.weights && L > a.weights_stride)) {
    if (threadIdx.x == 0 && rank == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    return;
  }
  const int32_t* idx = a.keep_idx + ((int64_t)b * Hkv + h) * a.budget;
  bool bad = false;
  for (int j = threadIdx.x; j < m; j += blockDim.x) {
    const int t = idx[j];
    bad |= t >= L || t <= (j > 0 ? idx[j - 1] : -1);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && rank == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_INDEX);
    return;
  }
  if (kv == 2) {
    // the weights, always in place: entry keep_idx[j] to entry j
    if (rank != 0) return;
    constexpr int kBatchRows = 8;
    float* w = a.weights + ((int64_t)b * Hkv + h) * a.weights_stride;
    for (int j0 = 0; j0 < m; j0 += kBatchRows * kEvictWarps * 32) {
      float x[kBatchRows];
#pragma unroll
      for (int u = 0; u < kBatchRows; ++u) {
        const int j = j0 + u * kEvictWarps * 32 + (int)threadIdx.x;
        if (j < m) x[u] = w[idx[j]];
      }
      __syncthreads();                               // the round's loads are done
#pragma unroll
      for (int u = 0; u < kBatchRows; ++u) {
        const int j = j0 + u * kEvictWarps * 32 + (int)threadIdx.x;
        if (j < m) w[j] = x[u];
      }
    }
    return;
  }
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks;
  const int32_t* dt = a.dst_tables + (int64_t)b * a.dst_max_blocks;
  const int nblk = (m + BS - 1) / BS;
  // no block stays: nothing is stored where something is still to be read
  bool stays = false;
  for (int j = threadIdx.x; j < nblk; j += blockDim.x) stays |= dt[j] == bt[j];
  const bool in_place = __syncthreads_or(stays);
  unsigned char* pool = static_cast<unsigned char*>(kv ? a.cache[1] : a.cache[0]);
  float* scale = kv ? a.scale[1] : a.scale[0];
  const int64_t row_bytes = (int64_t)Hkv * kRow * 16;  // between rows of a block
  auto loaded = [&]() {                              // the round's loads are done
    if (in_place) {
      if (C > 1) cluster.sync();
      else __syncthreads();
    }
  };
  for (int j0 = 0; j0 < nblk; j0 += C * kEvictWarps) {
    const int j = j0 + rank * kEvictWarps + warp;    // this warp's destination block
    bool move = j < nblk;
    const int rows = move ? min(BS, m - j * BS) : 0;
    int64_t from = 0, to = 0;                        // byte offsets; lane r: row r's source
    int dst = 0;
    float s = 0.0f;
    if (move) {
      dst = dt[j];
      const int own = bt[j];
      const int t = lane < rows ? idx[j * BS + lane] : 0;
      const int sb = lane < rows ? bt[t / BS] : 0;
      const bool off = dst < 0 || dst >= a.num_blocks || sb < 0 || sb >= a.num_blocks;
      const bool still = own == dst && (lane >= rows || t == j * BS + lane);
      if (__any_sync(0xffffffffu, off)) {
        if (lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
        move = false;
      } else if (__all_sync(0xffffffffu, still)) {
        move = false;
      } else {
        from = (((int64_t)sb * BS + t % BS) * Hkv + h) * (kRow * 16);
        to = ((int64_t)dst * BS * Hkv + h) * (kRow * 16);
        if (kQ8 && lane < rows) s = scale[(int64_t)sb * Hkv + h];
      }
    }
    if constexpr (kQ8) {
      if (!move) {
        loaded();
      } else {
        const float ns = rows == BS
            ? recode_block<D, BS, kFp8, true>(pool, from, to, row_bytes, s, rows, loaded)
            : recode_block<D, BS, kFp8, false>(pool, from, to, row_bytes, s, rows, loaded);
        if (lane == 0) scale[(int64_t)dst * Hkv + h] = ns;
      }
    } else {
      uint4 x[kPer];
      constexpr int kStep = kRow < 32 ? 32 / kRow : 1;
      const int sub = lane / kRow;
      if (move) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          const int64_t at = __shfl_sync(0xffffffffu, from, u * kStep + sub);
          if (u * kStep + sub < rows) x[u] = *reinterpret_cast<const uint4*>(pool + at + (lane % kRow) * 16);
        }
      }
      loaded();
      if (move) {
        unsigned char* out = pool + to + sub * row_bytes + (lane % kRow) * 16;
#pragma unroll
        for (int u = 0; u < kPer; ++u)
          if (u * kStep + sub < rows) *reinterpret_cast<uint4*>(out + u * kStep * row_bytes) = x[u];
      }
    }
  }
}

template <int D, int BS, int kKind>
kv_status launch_evict_t(const EvictArgs& a, int batch, int C, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_kv_heads * C), (unsigned)batch, a.weights ? 3 : 2);
  cfg.blockDim = dim3(kEvictWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cuda_check(cudaLaunchKernelEx(&cfg, evict_kernel<D, BS, kKind>, a), "evict_kernel launch");
}

template <int D, int BS>
kv_status launch_evict(const EvictArgs& a, kv_dtype dtype, int batch, int num_sms, cudaStream_t s) {
  // CTAs of a (KV head, sequence, K or V): one, or a cluster while those alone
  // leave SMs idle and there are further rounds to share
  int C = 1;
  while (C < kMostCtas && (int64_t)a.num_kv_heads * batch * 4 * C <= num_sms &&
         (int64_t)C * kEvictWarps * BS < a.budget)
    C *= 2;
  if (dtype == KV_DTYPE_INT8) return launch_evict_t<D, BS, KV_DTYPE_INT8>(a, batch, C, s);
  if (dtype == KV_DTYPE_FP8_E4M3) return launch_evict_t<D, BS, KV_DTYPE_FP8_E4M3>(a, batch, C, s);
  return launch_evict_t<D, BS, KV_DTYPE_BF16>(a, batch, C, s);
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
  if (max_seq_len > kMostTokens)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_select_tokens: max_seq_len is at most %d", kMostTokens);
  if (batch == 0) return KV_OK;
  if (!keep_idx || !keep_len || !weights || !seq_lens)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_select_tokens: NULL pointer");
  const int64_t rows = (int64_t)batch * num_kv_heads;
  // CTAs per row: slices of about 4096 candidates, at most 8 CTAs
  int C = 1;
  while (C < kMostCtas && (int64_t)C * 4096 < max_seq_len) C *= 2;
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
  const int per = (max_seq_len + C - 1) / C;
  a.chunk_cap = (per + 31) / 32;
  const int room = kMostSmem / (int)sizeof(uint32_t) - (kPasses + 1) * kBins - 2 * a.chunk_cap;
  a.cap = per < room ? per : room;
  cudaStream_t s = (cudaStream_t)stream;
  return per <= 4096 ? launch_select<256>(a, rows, C, di.device, s)
                     : launch_select<512>(a, rows, C, di.device, s);
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
  if (num_kv_heads > 65535) return fail(KV_ERR_INVALID_ARG, "pagedkv_evict_tokens: at most 65535 KV heads");
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
    return block_size == 32 ? launch_evict<128, 32>(a, dtype, batch, di.num_sms, s)
                            : launch_evict<128, 16>(a, dtype, batch, di.num_sms, s);
  return block_size == 32 ? launch_evict<64, 32>(a, dtype, batch, di.num_sms, s)
                          : launch_evict<64, 16>(a, dtype, batch, di.num_sms, s);
}

}  // extern "C"
