// pagedkv_weights_few.cu -- the attention weights of a few query tokens per
// sequence (speculative verification) in one pass over K: pagedkv_attention_
// weights for at most 32 rows (query tokens times grouped heads) per KV head.
//
// With so few rows the keys' bytes bound it, and a second pass over K Q^T
// would read them again.  Here the scores of a whole sequence stay in TMEM
// until the rows' denominators are known: a cluster of C CTAs shares the keys
// of one (sequence, KV head), each CTA streams its part of K through three TMA
// stages, and
//   S[128 keys x 32 rows] = K . Q^T          (tcgen05, one MMA group a chunk)
// of its up to 8 chunks lie side by side in 256 TMEM columns (128 KB), so two
// CTAs fit an SM.  Three sweeps over them, a thread per key (TMEM lane) and a
// warp per 32 keys:
//   1. each row's maximum over the CTA's keys, as the chunks arrive,
//   2. each row's sum of 2^(s - max),  after which the cluster exchanges
//      (max, sum) through distributed shared memory and every CTA has
//      m' = m + log2 l,
//   3. each key's sum of 2^(s - m') over the rows: its weight.
// A thread joins its keys' values row by row; the reduction over keys then
// takes one transposing butterfly per sweep and warp (31 shuffles leave row
// j's result in lane j).
//
// 64 sequences of 512..4096 tokens, five queries each, 32/8 heads: 102 us, of
// which the bytes of K would take 47 at the copy rate (two passes of the
// mma.sync kernels: 189).  K is read at the copy rate while the first sweep
// runs; the other two sweeps and the exchange read no memory, and only the
// second CTA of an SM hides them.
//
// 8-bit pools: the key warps load the codes themselves, a chunk ahead, and widen
// them to bf16 (exact) into the stage; a key's K scale multiplies its scores.
// The same batch: int8 140 us, E4M3 136 (196 and 189 in two passes), bound by
// the widening beside the sweeps.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_tc.cuh"
#include "pagedkv_weights.cuh"

namespace cg = cooperative_groups;

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kTile = 128;                             // keys per chunk
constexpr int kRows = kFewRows;                        // rows: the MMA's N
constexpr int kChunks = 8;                             // chunks per CTA, at most
constexpr int kTmemCols = kChunks * kRows;
constexpr int kStages = 3;
constexpr int kSets = 2;                               // sets of four key warps
constexpr int kKeyWarps = 4 * kSets, kMmaWarp = kKeyWarps, kLoadWarp = kKeyWarps + 1;
constexpr int kThreads = (kKeyWarps + 2) * 32;
constexpr int kMostCtas = 8;                           // of a cluster

template <int D>
struct FGeo {
  static constexpr int kBands = D / 64;
  static constexpr int kImage = kTile * D * 2;         // a chunk of K
  static constexpr int kQImage = kRows * D * 2;
  static constexpr int kUsed = kStages * kImage + kQImage + 1024;
  // at least 100 KB, so that no more than two CTAs (512 TMEM columns) share an SM
  static constexpr int kSmemBytes = kUsed > 100 * 1024 ? kUsed : 100 * 1024;
};

struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};

// Lane j gets op over the warp's lanes of their v[j].
template <class Op>
__device__ __forceinline__ float transpose_reduce(float (&v)[32], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const bool up = lane & off;
      const float send = up ? v[i] : v[i + off], keep = up ? v[i + off] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  return v[0];
}

template <int D, int BS, int kKind>
__global__ void __launch_bounds__(kThreads, 2)
    few_rows_kernel(const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap q_map, const PromptArgs a) {
  using F = FGeo<D>;
  constexpr bool kQ8 = kKind != KV_DTYPE_BF16;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t q_full, full[kStages], empty[kStages], s_full[kChunks], drain_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int sh_bad, sh_fail;
  __shared__ float part[kKeyWarps][kRows];             // the warps' maxima, then sums
  __shared__ float cta_max[kRows], cta_sum[kRows];     // read by the cluster
  __shared__ __align__(16) float neg_m[kRows];         // -m'
  __shared__ float key_scale[kQ8 ? kChunks : 1][kTile];  // 8-bit: a key's score scale, its thread's own
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x / C, b = blockIdx.y;
  const int G = a.num_q_heads / a.num_kv_heads;
  int q0, n, L;
  if (!prompt_rows(a, b, BS, &q0, &n, &L)) {           // (cluster-uniform)
    if (blockIdx.x == 0 && tid == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    return;
  }
  if (n == 0) return;
  const int R = n * G;
  const int all = (L + kTile - 1) / kTile, per = (all + C - 1) / C;
  const int c_lo = min(rank * per, all), nch = min(per, all - c_lo);  // <= kChunks by the host's C
  const int k0 = c_lo * kTile;
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks;

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  auto stage_img = [&](int s) { return base + (uint32_t)(s * F::kImage); };
  const uint32_t q_img = base + kStages * F::kImage;
  if (tid == 0) {
    sh_bad = 0;
    sh_fail = 0;
    mbar_init(smem_addr(&q_full), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&full[s]), kQ8 ? 4 : 1);
      mbar_init(smem_addr(&empty[s]), 1);
    }
    for (int c = 0; c < kChunks; ++c) mbar_init(smem_addr(&s_full[c]), 1);
    mbar_init(smem_addr(&drain_bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(&tmem_base)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;

  if (warp == kLoadWarp) {
    // ======================= loads (TMA) ====================================
    if (lane == 0 && nch > 0) {
      // whole tokens: tile_tokens of them times the G heads (rows of later
      // tokens are masked)
      mbar_expect_tx(smem_addr(&q_full), (uint32_t)(a.tile_tokens * G * D * 2));
#pragma unroll
      for (int x = 0; x < F::kBands; ++x)
        tma_load_3d(q_img + x * (kRows * 128), &q_map, smem_addr(&q_full), x * 64, hk * G, q0);
    }
    __syncwarp();
    int issued = 0;
    bool ok = true;
    for (int c = 0; c < (kQ8 ? 0 : nch); ++c) {
      const int s = c % kStages, from = k0 + c * kTile;
      const int nb = min(kTile / BS, (L - from + BS - 1) / BS);
      int p = lane < nb ? bt[from / BS + lane] : 0;
      if (p < 0 || p >= a.num_blocks) {
        sh_bad = 1;
        p = 0;
      }
      if (c >= kStages && !warp_wait(smem_addr(&empty[s]), ((c / kStages) - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_expect_tx(smem_addr(&full[s]), (uint32_t)(nb * BS * D * 2));
      __syncwarp();
      if (lane < nb) {
#pragma unroll
        for (int x = 0; x < F::kBands; ++x)
          tma_load_4d(stage_img(s) + x * (kTile * 128) + lane * (BS * 128), &k_map, smem_addr(&full[s]),
                      x * 64, hk, 0, p);
      }
      __syncwarp();
      issued = c + 1;
    }
    // every load has landed before the CTA ends (bounded; normally it has)
    if (nch > 0 && !warp_wait(smem_addr(&q_full), 0)) ok = false;
    for (int s = 0; s < kStages && s < issued; ++s) {
      const int last = s + kStages * ((issued - 1 - s) / kStages);
      if (!warp_wait(smem_addr(&full[s]), (last / kStages) & 1)) ok = false;
    }
    if (!ok && lane == 0) sh_fail = 1;
  } else if (warp == kMmaWarp) {
    // ======================= tensor-core issue (one lane) ===================
    if (lane == 0 && nch > 0) {
      const uint32_t idesc = mma_idesc<false>(kTile, kRows, 0);
      bool ok = mbar_wait(smem_addr(&q_full), 0);
      for (int c = 0; c < nch && ok; ++c) {
        const int s = c % kStages;
        ok = mbar_wait(smem_addr(&full[s]), (c / kStages) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss(tm + c * kRows, smem_desc(stage_img(s) + (ks / 4) * (kTile * 128) + (ks % 4) * 32, 16, 1024),
                 smem_desc(q_img + (ks / 4) * (kRows * 128) + (ks % 4) * 32, 16, 1024), idesc, ks > 0);
        mma_commit(smem_addr(&s_full[c]));
        mma_commit(smem_addr(&empty[s]));
      }
      if (!ok) sh_fail = 1;
      // the tensor core is done with shared memory and TMEM before they go
      mma_commit(smem_addr(&drain_bar));
      mbar_wait(smem_addr(&drain_bar), 0);
    }
    __syncwarp();
  }

  // ======================= the sweeps (warps 0-7; barriers are the CTA's) ====
  // warps 0-3 take the even chunks, 4-7 the odd ones
  const int row = tid & (kTile - 1), first = warp >> 2;
  const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
  const float sl2 = a.scale_log2;
  // scaled scores of this thread's key of chunk c: -inf for the rows that do
  // not see it (rows at position L - n + r / G < key); rows of padding, j >= R,
  // hold anything and are left out of every sum over rows
  auto scores = [&](int c, float (&v)[32]) {
    uint32_t x[32];
    __syncwarp();
    tmem_read32(lanes + c * kRows, x);
    const int key = k0 + c * kTile + row;
    const int from = max(0, key - (L - n)) * G;
    const float f = kQ8 ? key_scale[c][row] : sl2;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(x[j]) * f;
    if (k0 + c * kTile + kTile > L - n + 1) {          // (CTA-uniform)
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < from) v[j] = -INFINITY;
    }
  };
  if (warp < kKeyWarps) {
    bool ok = true;
    float m[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) m[j] = -INFINITY;
    // 8-bit pools: chunk c's codes into its stage, once part 0 of them is held
    // and the MMA of the chunk before it there is done
    [[maybe_unused]] Codes<D, BS, kQ8 ? kKind : KV_DTYPE_INT8> codes;
    if constexpr (kQ8) {
      if (first < nch && !codes.load(a, bt, hk, k0 + first * kTile, L, 0)) sh_bad = 1;
    }
    for (int c = first; c < nch; c += kSets) {
      if constexpr (kQ8) {
        const int from = k0 + c * kTile, key = from + row;
        float f = 0.0f;
        if (key < L) {
          const int p = bt[key / BS];
          if (p >= 0 && p < a.num_blocks) f = sl2 * a.k_scale[(int64_t)p * a.num_kv_heads + hk];
        }
        key_scale[c][row] = f;
        if (c >= kStages && !warp_wait(smem_addr(&s_full[c - kStages]), 0)) {
          ok = false;
          break;
        }
        if (!codes.finish(a, bt, hk, from, L, smem_raw + (stage_img(c % kStages) - smem_addr(smem_raw)))) sh_bad = 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&full[c % kStages]));
        if (c + kSets < nch && !codes.load(a, bt, hk, from + kSets * kTile, L, 0)) sh_bad = 1;
      }
      if (!warp_wait(smem_addr(&s_full[c]), 0)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float v[32];
      scores(c, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) m[j] = fmaxf(m[j], v[j]);
    }
    if (!ok && lane == 0) sh_fail = 1;
    part[warp][lane] = transpose_reduce(m, Max());
  }
  __syncthreads();
  const bool ok_cta = sh_fail == 0;
  if (warp == 0) {
    float m = part[0][lane];
#pragma unroll
    for (int w = 1; w < kKeyWarps; ++w) m = fmaxf(m, part[w][lane]);
    cta_max[lane] = m;
    neg_m[lane] = m == -INFINITY ? 0.0f : -m;
  }
  __syncthreads();
  if (warp < kKeyWarps) {
    float l[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) l[j] = 0.0f;
    for (int c = first; c < (ok_cta ? nch : 0); c += kSets) {
      float v[32];
      scores(c, v);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        if (j >= R) break;
        const float4 o = *reinterpret_cast<const float4*>(neg_m + j);
        l[j] += ex2(v[j] + o.x);
        l[j + 1] += ex2(v[j + 1] + o.y);
        l[j + 2] += ex2(v[j + 2] + o.z);
        l[j + 3] += ex2(v[j + 3] + o.w);
      }
    }
    part[warp][lane] = transpose_reduce(l, Add());
  }
  __syncthreads();
  if (warp == 0) {
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < kKeyWarps; ++w) l += part[w][lane];
    // a CTA without a result (a bad block, a wait that gave up): l < 0
    cta_sum[lane] = !ok_cta || sh_bad ? -1.0f : l;
  }
  cluster.sync();
  bool lost = false;
  if (warp == 0) {
    float M = -INFINITY, l = 0.0f, m[kMostCtas], x[kMostCtas];
#pragma unroll
    for (int r = 0; r < kMostCtas; ++r)
      if (r < C) {
        m[r] = cluster.map_shared_rank(cta_max, r)[lane];
        x[r] = cluster.map_shared_rank(cta_sum, r)[lane];
      }
#pragma unroll
    for (int r = 0; r < kMostCtas; ++r)
      if (r < C) {
        lost |= x[r] < 0.0f && lane < R;
        M = fmaxf(M, m[r]);
      }
#pragma unroll
    for (int r = 0; r < kMostCtas; ++r)
      if (r < C && (m[r] > -INFINITY || x[r] != x[r])) l = fmaf(x[r], ex2(m[r] - M), l);
    neg_m[lane] = -(M + log2f(l));
  }
  lost = __syncthreads_or(lost);
  if (warp < kKeyWarps && !lost) {
    float* w = a.weights + ((int64_t)b * a.num_kv_heads + hk) * a.stride;
    for (int c = first; c < nch; c += kSets) {
      const int key = k0 + c * kTile + row;
      const bool add = a.accumulate && key < L - n;
      const float old = add ? w[key] : 0.0f;
      float v[32], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      scores(c, v);
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        if (j >= R) break;
        const float4 o = *reinterpret_cast<const float4*>(neg_m + j);
        const float e1 = ex2(v[j + 1] + o.y), e2 = ex2(v[j + 2] + o.z), e3 = ex2(v[j + 3] + o.w);
        sum[0] += ex2(v[j] + o.x);
        sum[1] += j + 1 < R ? e1 : 0.0f;
        sum[2] += j + 2 < R ? e2 : 0.0f;
        sum[3] += j + 3 < R ? e3 : 0.0f;
      }
      if (key < L) w[key] = old + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmemCols) : "memory");
  if (tid == 0 && sh_bad) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
  if (tid == 0 && sh_fail) atomicOr(a.flags, PAGEDKV_FLAG_WAIT_TIMEOUT);
  cluster.sync();                                      // peers may still read this CTA's statistics
}

template <int D, int BS, int kKind>
kv_status launch_few_t(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, int C, cudaStream_t s) {
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  kv_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != KV_OK) return st;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
      st = cuda_check(cudaFuncSetAttribute(few_rows_kernel<D, BS, kKind>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           FGeo<D>::kSmemBytes),
                      "cudaFuncSetAttribute(few_rows_kernel)");
      if (st != KV_OK) return st;
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_kv_heads * C), (unsigned)a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = FGeo<D>::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, few_rows_kernel<D, BS, kKind>, km, qm, a), "few_rows_kernel launch");
}

template <int D, int BS>
kv_status launch_few(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, kv_dtype dtype, int C,
                     cudaStream_t s) {
  if (dtype == KV_DTYPE_INT8) return launch_few_t<D, BS, KV_DTYPE_INT8>(a, km, qm, C, s);
  if (dtype == KV_DTYPE_FP8_E4M3) return launch_few_t<D, BS, KV_DTYPE_FP8_E4M3>(a, km, qm, C, s);
  return launch_few_t<D, BS, KV_DTYPE_BF16>(a, km, qm, C, s);
}

}  // namespace

int few_rows_ctas(int batch, int num_kv_heads, int max_seq_len, int num_sms) {
  const int chunks = (max_seq_len - 1) / kTile + 1;
  int C = 1;
  while (C < kMostCtas && C * kChunks < chunks) C *= 2;
  if (C * kChunks < chunks) return 0;
  // more CTAs while two per SM are not reached and each has keys
  while (C < kMostCtas && C < chunks && (int64_t)batch * num_kv_heads * C * 2 <= 2 * num_sms) C *= 2;
  return C;
}

kv_status launch_prompt_few(const PromptArgs& a, int head_dim, int block_size, kv_dtype dtype, int ctas,
                            cudaStream_t s) {
  DecodeArgs d = {};
  d.k_cache = a.k_cache;
  d.v_cache = a.k_cache;                               // (the V map is not used)
  d.num_kv_heads = a.num_kv_heads;
  d.num_blocks = a.num_blocks;
  d.head_dim = head_dim;
  d.block_size = block_size;
  d.dtype = dtype;
  alignas(64) CUtensorMap km, vm, qm;
  kv_status st = make_kv_maps(d, &km, &vm);
  if (st == KV_OK)
    st = make_query_map(&qm, a.q, a.num_tokens, a.num_q_heads, head_dim, a.num_q_heads / a.num_kv_heads,
                        a.tile_tokens);
  if (st != KV_OK) return st;
  if (head_dim == 128)
    return block_size == 32 ? launch_few<128, 32>(a, km, qm, dtype, ctas, s) : launch_few<128, 16>(a, km, qm, dtype, ctas, s);
  return block_size == 32 ? launch_few<64, 32>(a, km, qm, dtype, ctas, s) : launch_few<64, 16>(a, km, qm, dtype, ctas, s);
}

}  // namespace pagedkv
