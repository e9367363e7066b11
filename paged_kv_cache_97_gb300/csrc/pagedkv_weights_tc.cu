// pagedkv_weights_tc.cu -- the attention weights of long multi-token queries
// (prompts, prefill chunks) on the fifth-generation tensor cores: both passes
// of pagedkv_attention_weights over Q K^T (pagedkv_weights.cu) with the scores
// in TMEM.
//
// The two passes are one kernel with the operands exchanged.  A CTA keeps one
// tile of 128 rows of one operand in shared memory and streams tiles of 128
// rows of the other through two stages:
//   row statistics   fixed: 128 query rows,  streamed: the keys they see;
//                    a thread owns a query row and keeps its (m, l)
//   column sums      fixed: 128 keys,        streamed: the row tiles that see
//                    them; a thread owns a key and adds 2^(s - m') over the
//                    rows, m' = m + log2 l of each row from shared memory
// so that neither a maximum nor a sum crosses threads.  Warps 0-3 hold one
// fixed row per thread (a TMEM lane), warp 4 issues the MMAs (S[128 x 128] =
// fixed . streamed^T into one of two TMEM buffers), warp 5 the TMA loads, and
// in the column sums warps 6-9 join each row tile's statistics.  A query tile
// is whole tokens, tile_tokens = 128 / G of them times the G heads, as one TMA
// box; rows past the sequence's queries are masked.
//
// The exponentials bound it: 128 x 128 of them take 1024 cycles of an SM's
// special-function unit, the MMAs of a tile 256.  Two CTAs per SM (256 TMEM
// columns and about 100 KB of shared memory each) so that one's start and end
// overlap the other's work.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_tc.cuh"
#include "pagedkv_weights.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kTile = 128;                             // rows of either operand
constexpr int kStages = 2;                             // = TMEM buffers
constexpr int kMmaWarp = 4, kLoadWarp = 5, kStatWarp = 6;
constexpr int kTmemCols = kStages * kTile;
constexpr float kMoveLog2 = 8.0f;                      // move a row's reference past 2^8

template <int D>
struct PGeo {
  static constexpr int kBands = D / 64;
  static constexpr int kImage = kTile * D * 2;         // bytes of 128 rows
  static constexpr int kUsed = (1 + kStages) * kImage + 1024;
  // at least 100 KB, so that no more than two CTAs (512 TMEM columns) share an SM
  static constexpr int kSmemBytes = kUsed > 100 * 1024 ? kUsed : 100 * 1024;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Running statistics of a query row: 2^(s sl2 - ref) summed to l.  The
// reference moves only when a score passes it by 2^8, so l <= 2^8 keys.
struct RowStats {
  float ref, l;
};

// 32 scores of the row (of keys up to `lim` of the 32 when kMask).
template <bool kMask>
__device__ __forceinline__ void add_scores(RowStats& st, uint32_t (&raw)[32], float sl2, int lim) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (kMask && j > lim) raw[j] = 0xff800000u;        // -inf
    mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(raw[j]));
  }
  const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
  if (m > st.ref + kMoveLog2) {
    st.l *= ex2(st.ref - m);
    st.ref = m;
  }
  const float off = st.ref == -INFINITY ? 0.0f : st.ref;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 32; ++j) s[j & 3] += ex2(fmaf(__uint_as_float(raw[j]), sl2, -off));
  st.l += (s[0] + s[1]) + (s[2] + s[3]);
}

// sum over 32 rows of 2^(s sl2 - m') (rows at or past `key` when kMask).
template <bool kMask>
__device__ __forceinline__ float column_part(const uint32_t (&raw)[32], float sl2, const float* m,
                                             const int* pos, int key) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 r = *reinterpret_cast<const float4*>(m + j);
    const float e0 = ex2(fmaf(__uint_as_float(raw[j]), sl2, -r.x));
    const float e1 = ex2(fmaf(__uint_as_float(raw[j + 1]), sl2, -r.y));
    const float e2 = ex2(fmaf(__uint_as_float(raw[j + 2]), sl2, -r.z));
    const float e3 = ex2(fmaf(__uint_as_float(raw[j + 3]), sl2, -r.w));
    if constexpr (kMask) {
      const int4 p = *reinterpret_cast<const int4*>(pos + j);
      s[0] += p.x >= key ? e0 : 0.0f;
      s[1] += p.y >= key ? e1 : 0.0f;
      s[2] += p.z >= key ? e2 : 0.0f;
      s[3] += p.w >= key ? e3 : 0.0f;
    } else {
      s[0] += e0;
      s[1] += e1;
      s[2] += e2;
      s[3] += e3;
    }
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int D, int BS, bool kStats>
__global__ void __launch_bounds__(kStats ? 192 : 320, 2)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap q_map, const PromptArgs a) {
  using P = PGeo<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t fixed_full, full[kStages], empty[kStages], s_full[kStages], buf_free[kStages],
      stat_full[kStages], drain_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int sh_bad, sh_fail;
  __shared__ __align__(16) float row_m[kStages][kTile];
  __shared__ __align__(16) int row_pos[kStages][kTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x, b = blockIdx.y;
  const int G = a.num_q_heads / a.num_kv_heads, TT = a.tile_tokens;
  int q0, n, L;
  const bool ok_seq = prompt_rows(a, b, BS, &q0, &n, &L);
  if (!ok_seq) {
    if (kStats && blockIdx.z == 0 && tid == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    return;
  }
  // The unit.  Row statistics: row tile (the last ones, with most keys, first)
  // and key split; column sums: key tile.
  const int split = kStats ? (int)(blockIdx.z % a.splits) : 0;
  const int unit = kStats ? (int)((gridDim.z - 1 - blockIdx.z) / a.splits) : (int)blockIdx.z;
  const int i0 = unit * TT;                            // first query token of the fixed tile
  const int tn = min(TT, n - i0);                      // its tokens
  const int k0 = kStats ? split * a.part_tokens : unit * kTile;  // first key
  if (kStats ? tn <= 0 : (n == 0 || k0 >= L)) return;
  const int first_pos = L - n + i0;
  const int kend = kStats ? min(first_pos + tn, k0 + a.part_tokens) : min(L, k0 + kTile);
  const int rt0 = kStats ? 0 : max(0, k0 - (L - n)) / TT;        // first row tile that sees a key
  const int nch = kStats ? max(0, (kend - k0 + kTile - 1) / kTile) : (n - 1) / TT + 1 - rt0;
  // global row of row r of the tile that starts at token i
  auto row_at = [&](int i, int r) { return (int64_t)(q0 + i + r / G) * a.num_q_heads + hk * G + r % G; };
  const int my_rows = kStats ? tn * G : 0;
  if (kStats && nch == 0) {                            // no key of this split
    if (tid < my_rows) {
      float* o = a.stats + (row_at(i0, tid) * a.splits + split) * 2;
      o[0] = -INFINITY;
      o[1] = 0.0f;
    }
    return;
  }

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  auto stage_img = [&](int s) { return base + (uint32_t)((1 + s) * P::kImage); };
  if (tid == 0) {
    sh_bad = 0;
    sh_fail = 0;
    mbar_init(smem_addr(&fixed_full), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), 1);
      mbar_init(smem_addr(&s_full[s]), 1);
      mbar_init(smem_addr(&buf_free[s]), 4);
      mbar_init(smem_addr(&stat_full[s]), 4);
    }
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
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks;

  RowStats st = {-INFINITY, 0.0f};
  float acc = 0.0f;

  if (warp == kLoadWarp) {
    // ======================= loads (TMA) ====================================
    // Keys [from, from + 128) (up to L) into an image, one block per lane.
    auto load_k = [&](uint32_t img, uint64_t* bar, int from) {
      const int nb = min(kTile / BS, (L - from + BS - 1) / BS);
      int p = lane < nb ? bt[from / BS + lane] : 0;
      if (p < 0 || p >= a.num_blocks) {
        sh_bad = 1;
        p = 0;
      }
      if (lane == 0) mbar_expect_tx(smem_addr(bar), (uint32_t)(nb * BS * D * 2));
      __syncwarp();
      if (lane < nb) {
#pragma unroll
        for (int x = 0; x < P::kBands; ++x)
          tma_load_4d(img + x * (kTile * 128) + lane * (BS * 128), &k_map, smem_addr(bar), x * 64, hk, 0, p);
      }
      __syncwarp();
    };
    // The row tile that starts at query token i (whole boxes; rows past the
    // tensor are zeros).
    auto load_q = [&](uint32_t img, uint64_t* bar, int i) {
      if (lane == 0) {
        mbar_expect_tx(smem_addr(bar), (uint32_t)(TT * G * D * 2));
#pragma unroll
        for (int x = 0; x < P::kBands; ++x)
          tma_load_3d(img + x * (kTile * 128), &q_map, smem_addr(bar), x * 64, hk * G, q0 + i);
      }
      __syncwarp();
    };
    if (kStats) load_q(base, &fixed_full, i0);
    else load_k(base, &fixed_full, k0);
    int issued = 0;
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
      const int s = c % kStages;
      if (c >= kStages && !warp_wait(smem_addr(&empty[s]), ((c / kStages) - 1) & 1)) {
        ok = false;
        break;
      }
      if (kStats) load_k(stage_img(s), &full[s], k0 + c * kTile);
      else load_q(stage_img(s), &full[s], (rt0 + c) * TT);
      issued = c + 1;
    }
    // every load has landed before the CTA ends (bounded; normally it has)
    if (!warp_wait(smem_addr(&fixed_full), 0)) ok = false;
    for (int s = 0; s < kStages && s < issued; ++s) {
      const int last = s + kStages * ((issued - 1 - s) / kStages);
      if (!warp_wait(smem_addr(&full[s]), (last / kStages) & 1)) ok = false;
    }
    if (!ok && lane == 0) sh_fail = 1;
  } else if (warp == kMmaWarp) {
    // ======================= tensor-core issue (one lane) ===================
    if (lane == 0) {
      const uint32_t idesc = mma_idesc<false>(kTile, kTile, 0);
      bool ok = mbar_wait(smem_addr(&fixed_full), 0);
      for (int c = 0; c < nch && ok; ++c) {
        const int s = c % kStages, ph = (c / kStages) & 1;
        ok = mbar_wait(smem_addr(&full[s]), ph) &&
             (c < kStages || mbar_wait(smem_addr(&buf_free[s]), ph ^ 1));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks / 4) * (kTile * 128) + (ks % 4) * 32;
          mma_ss(tm + s * kTile, smem_desc(base + off, 16, 1024), smem_desc(stage_img(s) + off, 16, 1024),
                 idesc, ks > 0);
        }
        mma_commit(smem_addr(&s_full[s]));
        mma_commit(smem_addr(&empty[s]));
      }
      if (!ok) sh_fail = 1;
      // the tensor core is done with shared memory and TMEM before they go
      mma_commit(smem_addr(&drain_bar));
      mbar_wait(smem_addr(&drain_bar), 0);
    }
    __syncwarp();
  } else if (!kStats && warp >= kStatWarp) {
    // ======================= column sums: the row tiles' statistics =========
    const int r = tid - kStatWarp * 32;
    bool bad = false, ok = true;
    for (int c = 0; c < nch; ++c) {
      const int s = c % kStages, i = (rt0 + c) * TT;
      float m = 0.0f;
      int pos = -1;
      if (r < min(TT, n - i) * G) {
        pos = L - n + i + r / G;
        const float* ml = a.stats + row_at(i, r) * a.splits * 2;
        const int ns = pos / a.part_tokens + 1;        // splits with keys of this row
        float M = -INFINITY, den = 0.0f;
        for (int k = 0; k < ns; ++k) M = fmaxf(M, ml[2 * k]);
        for (int k = 0; k < ns; ++k) {
          bad |= ml[2 * k + 1] < 0.0f;
          den = fmaf(exp2f(ml[2 * k] - M), ml[2 * k + 1], den);
        }
        m = M + log2f(den);
      }
      if (c >= kStages && !warp_wait(smem_addr(&buf_free[s]), ((c / kStages) - 1) & 1)) {
        ok = false;
        break;
      }
      row_m[s][r] = m;
      row_pos[s][r] = pos;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&stat_full[s]));
    }
    if (bad) sh_bad = 1;
    if (!ok) sh_fail = 1;
  } else {
    // ======================= one fixed row per thread (warps 0-3) ===========
    bool ok = true;
    const int key = k0 + tid;                          // column sums
    const int pos = kStats && tid < my_rows ? first_pos + tid / G : -1;
    // a warp whose rows are all padding only keeps the barriers' phases
    const bool live = kStats ? warp * 32 < my_rows : k0 + warp * 32 < kend;
    const float sl2 = a.scale_log2;
    const uint32_t lanes = tm + ((uint32_t)(warp * 32) << 16);
    for (int c = 0; c < nch; ++c) {
      const int s = c % kStages, ph = (c / kStages) & 1;
      if (!warp_wait(smem_addr(&s_full[s]), ph) ||
          (!kStats && !warp_wait(smem_addr(&stat_full[s]), ph))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (live) {
        uint32_t x[2][32];
        const uint32_t at = lanes + s * kTile;
        const int c0 = k0 + c * kTile;                 // row statistics: the chunk's first key
        const int i = (rt0 + c) * TT;                  // column sums: the tile's first token
        const int cols = kStats ? kTile : min(TT, n - i) * G;
        const bool whole = kStats ? c0 + kTile - 1 <= first_pos
                                  : cols == kTile && L - n + i >= k0 + kTile - 1;
        tmem_ld32(at, x[0]);
        tmem_wait_ld32(x[0]);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          __syncwarp();                                // (the TMEM loads are the whole warp's)
          if (h < 3 && 32 * (h + 1) < cols) tmem_ld32(at + 32 * (h + 1), x[(h + 1) & 1]);
          if constexpr (kStats) {
            if (whole) add_scores<false>(st, x[h & 1], sl2, 0);
            else add_scores<true>(st, x[h & 1], sl2, pos - c0 - 32 * h);
          } else {
            if (whole) acc += column_part<false>(x[h & 1], sl2, row_m[s] + 32 * h, row_pos[s] + 32 * h, key);
            else if (32 * h < cols) acc += column_part<true>(x[h & 1], sl2, row_m[s] + 32 * h, row_pos[s] + 32 * h, key);
          }
          __syncwarp();
          if (h < 3 && 32 * (h + 1) < cols) tmem_wait_ld32(x[(h + 1) & 1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&buf_free[s]));
    }
    if (!ok && lane == 0) sh_fail = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmemCols) : "memory");
  const bool failed = sh_fail != 0;
  if (tid == 0 && failed) atomicOr(a.flags, PAGEDKV_FLAG_WAIT_TIMEOUT);
  if constexpr (kStats) {
    if (tid == 0 && sh_bad) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
    if (tid < my_rows) {
      float* o = a.stats + (row_at(i0, tid) * a.splits + split) * 2;
      o[0] = st.ref;
      o[1] = failed || sh_bad ? -1.0f : st.l;          // l < 0: the weights stay as they are
    }
  } else if (!failed && !sh_bad && tid < kend - k0) {
    float* w = a.weights + ((int64_t)b * a.num_kv_heads + hk) * a.stride + k0 + tid;
    *w = a.accumulate && k0 + tid < L - n ? *w + acc : acc;
  }
}

template <int D, int BS, bool kStats>
kv_status launch_tc_t(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, unsigned z,
                      cudaStream_t s) {
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  kv_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != KV_OK) return st;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
      st = cuda_check(cudaFuncSetAttribute(prompt_tc_kernel<D, BS, kStats>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, PGeo<D>::kSmemBytes),
                      "cudaFuncSetAttribute(prompt_tc_kernel)");
      if (st != KV_OK) return st;
      attr_set[dev] = true;
    }
  }
  const dim3 grid((unsigned)a.num_kv_heads, (unsigned)a.batch, z);
  prompt_tc_kernel<D, BS, kStats><<<grid, kStats ? 192 : 320, PGeo<D>::kSmemBytes, s>>>(km, qm, a);
  return cuda_check(cudaGetLastError(), "prompt_tc_kernel launch");
}

template <int D, int BS>
kv_status launch_tc(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, int tiles, cudaStream_t s) {
  const kv_status st = launch_tc_t<D, BS, true>(a, km, qm, (unsigned)(tiles * a.splits), s);
  if (st != KV_OK) return st;
  return launch_tc_t<D, BS, false>(a, km, qm, (unsigned)((a.max_seq_len - 1) / kTile + 1), s);
}

}  // namespace

kv_status launch_prompt_tc(const PromptArgs& a, int head_dim, int block_size, int tiles, cudaStream_t s) {
  DecodeArgs d = {};
  d.k_cache = a.k_cache;
  d.v_cache = a.k_cache;                               // (the V map is not used)
  d.num_kv_heads = a.num_kv_heads;
  d.num_blocks = a.num_blocks;
  d.head_dim = head_dim;
  d.block_size = block_size;
  d.dtype = KV_DTYPE_BF16;
  alignas(64) CUtensorMap km, vm, qm;
  kv_status st = make_kv_maps(d, &km, &vm);
  if (st == KV_OK)
    st = make_query_map(&qm, a.q, a.num_tokens, a.num_q_heads, head_dim, a.num_q_heads / a.num_kv_heads,
                        a.tile_tokens);
  if (st != KV_OK) return st;
  if (head_dim == 128)
    return block_size == 32 ? launch_tc<128, 32>(a, km, qm, tiles, s) : launch_tc<128, 16>(a, km, qm, tiles, s);
  return block_size == 32 ? launch_tc<64, 32>(a, km, qm, tiles, s) : launch_tc<64, 16>(a, km, qm, tiles, s);
}

}  // namespace pagedkv
