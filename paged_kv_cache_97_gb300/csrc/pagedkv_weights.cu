// pagedkv_weights.cu -- the attention weight each cached token receives,
// summed over the query heads of its KV head and over steps:
//   p[h, t] = softmax_t(scale q_h . K_t),   w[t] = sum over rows of p[row, t].
// An eviction rule ranks tokens by it (pagedkv_evict.cu).  The weights live
// with the batch's sequences, fp32 [batch, Hkv, weights_stride], like the
// block tables, not with the pool's blocks: sequences that share blocks keep
// weights of their own, and no two CTAs ever add to the same entry.
//
// A weight needs its row's softmax denominator, which is known only after the
// last key.  One-token decode (paged_attention_decode_weights) keeps the
// scores that the attention computes anyway and turns them into weights once
// the partials are there (step_weights_kernel).  Several query tokens per
// sequence (pagedkv_attention_weights) take two passes over Q K^T: row
// statistics, then column sums; no value of V is needed.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_requant.cuh"
#include "pagedkv_tc.cuh"
#include "pagedkv_weights.cuh"

namespace pagedkv {
namespace {

using namespace dev;

// ---------------------------------------------------------------------------
// One-token decode
// ---------------------------------------------------------------------------

constexpr int kStepThreads = 256;
constexpr int kStepTokens = 4 * kStepThreads;          // tokens per CTA

struct StepArgs {
  float* weights;            // [B, Hkv, stride]
  const float* scores;       // [B, Hq, score_stride], base 2
  const float* ml;           // [B, Hq, slots, 2]
  const int32_t* seq_lens;
  int64_t stride, score_stride;
  int num_q_heads, num_kv_heads, part_tokens, slots, max_len;
};

// One CTA per (1024 tokens, KV head, sequence): (m, 1 / l) of the KV head's
// rows from their partials, then sum_g 2^(s_g - m_g) / l_g per token.  The
// token of this step (position L - 1) has no earlier weight: it is stored,
// the others are added to.  Bound by bytes: the scores are read once (from L2
// as far as they stayed there), the weights read and written.  128 sequences of
// 1..8K tokens, 64/8 heads, int8: 36 us behind an attention of 228 + 8 (211
// without the scores), 278 together; reading K a second time for the scores
// instead of keeping them would take 90 for its bytes alone.
__global__ void __launch_bounds__(kStepThreads) step_weights_kernel(const StepArgs a) {
  __shared__ float row_m[kMaxGroup], row_inv[kMaxGroup];
  __shared__ int row_bad;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int GQ = a.num_q_heads / a.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) row_bad = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = a.seq_lens[b];
  const int t0 = blockIdx.x * kStepTokens;
  if (L <= 0 || L > a.max_len || t0 >= L) return;      // a bad length was flagged by the attention
  __syncthreads();
  const int64_t row0 = (int64_t)b * a.num_q_heads + (int64_t)hk * GQ;
  if (warp < GQ) {
    const float* ml = a.ml + (row0 + warp) * a.slots * 2;
    const int np = (L + a.part_tokens - 1) / a.part_tokens;
    float M = -INFINITY, den = 0.0f;
    bool bad = false;
    for (int i = lane; i < np; i += 32) {
      M = fmaxf(M, ml[2 * i]);
      bad |= ml[2 * i + 1] < 0.0f;
    }
    M = warp_max(M);
    for (int i = lane; i < np; i += 32) den = fmaf(exp2f(ml[2 * i] - M), ml[2 * i + 1], den);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
    if (__any_sync(0xffffffffu, bad) && lane == 0) row_bad = 1;
    if (lane == 0) {
      row_m[warp] = M;
      row_inv[warp] = 1.0f / den;
    }
  }
  __syncthreads();
  if (row_bad) return;                                 // a bad block: the weights stay
  // four consecutive tokens per thread: every row's scores in one 16-byte load
  // each, all under way before the first is used
  float* w = a.weights + ((int64_t)b * a.num_kv_heads + hk) * a.stride;
  const float* sc = a.scores + row0 * a.score_stride;
  const int t = t0 + 4 * threadIdx.x;
  if (t >= L) return;
  float4 s[kMaxGroup];
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g)
    if (g < GQ) s[g] = __ldcs(reinterpret_cast<const float4*>(sc + g * a.score_stride + t));
  float old[4], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 4; ++k) old[k] = t + k < L - 1 ? w[t + k] : 0.0f;
  // (the rows' sum first: added one by one to an entry that has grown, weights
  // below half its last place would all be lost)
#pragma unroll
  for (int g = 0; g < kMaxGroup; ++g) {
    if (g >= GQ) break;
    const float m = row_m[g], inv = row_inv[g];
    sum[0] = fmaf(ex2(s[g].x - m), inv, sum[0]);
    sum[1] = fmaf(ex2(s[g].y - m), inv, sum[1]);
    sum[2] = fmaf(ex2(s[g].z - m), inv, sum[2]);
    sum[3] = fmaf(ex2(s[g].w - m), inv, sum[3]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (t + k < L) w[t + k] = old[k] + sum[k];
}

// ---------------------------------------------------------------------------
// Several query tokens per sequence
// ---------------------------------------------------------------------------
//
// The rows of a (sequence, KV head) are its (query token, grouped head)
// pairs, r = i * G + g, at position L - n + i.  Scores are computed as
//   S^T[16 keys x 8 rows] = K . Q^T            (mma.sync m16n8k16, fp32)
// with the key tile's A fragments in registers, straight from the pool (each
// key belongs to one warp), and a 64-row tile of Q in shared memory.  The k
// order of both operands is permuted so that a lane's fragments of two k-steps
// are one 16-byte piece of a row: lane t of a quad takes pieces t + 4c, and
// piece p holds elements 8p .. 8p + 7.  8-bit codes become bf16, exactly
// (|c| <= 127 and E4M3's 4 significant bits fit bf16's 8).
//
// These kernels serve what the tcgen05 ones do not: up to 64 rows on 8-bit pools
// and 15 on bf16 pools where the one-pass kernel does not hold them, scales that
// are not positive, groups of more than 128 heads.  The two reads of K and the
// issue of the loads' and exponentials' instructions share the bound: 64
// sequences of 512..4096 tokens x five queries, 32/8 heads, 189 us on a bf16
// pool and 196 on int8 (one pass with the scores in TMEM: 103 and 140), 64/8
// heads on int8 232.

constexpr int kRowTile = 64;                           // rows of Q per tile
constexpr int kNTiles = kRowTile / 8;
constexpr int kWarps = 4;
constexpr int kWarpKeys = 32;                          // keys per warp and step
constexpr int kCtaKeys = kWarps * kWarpKeys;

template <int D>
constexpr int kQStride = D * 2 + 64;                   // bytes; 16-byte pieces of 2 rows fill 32 banks

// Rows [r0, r0 + rows) of (sequence, KV head) into shared memory, zeros after.
template <int D>
__device__ __forceinline__ void load_q_tile(const PromptArgs& a, unsigned char* qs, int q0, int hk, int G,
                                            int r0, int rows) {
  constexpr int kPieces = D / 8;
  for (int i = threadIdx.x; i < kRowTile * kPieces; i += kWarps * 32) {
    const int r = i / kPieces, p = i % kPieces;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const int64_t row = (int64_t)(q0 + (r0 + r) / G) * a.num_q_heads + hk * G + (r0 + r) % G;
      x = static_cast<const uint4*>(a.q)[row * kPieces + p];
    }
    *reinterpret_cast<uint4*>(qs + r * kQStride<D> + p * 16) = x;
  }
}

// A fragments of the 32 keys from k0 (keys k0 + g + 8 i, i = 0..3, of lane
// 4g + t), zeros from `kend` on, and the keys' score factors.  Returns false
// when a key's block is outside the pool.
template <int D, int BS, int kKind>
__device__ __forceinline__ bool load_keys(const PromptArgs& a, const int32_t* bt, int hk, int k0, int kend,
                                          uint32_t (&ka)[4][D / 8], float (&kf)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = k0 + g + 8 * i;
    kf[i] = a.scale_log2;
    int p = key < kend ? bt[key / BS] : 0;
    const bool in = p >= 0 && p < a.num_blocks;
    ok &= in;
    const bool use = key < kend && in;
    const int64_t row = (((int64_t)(in ? p : 0) * BS + key % BS) * a.num_kv_heads + hk);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t* o = &ka[i][4 * c];
      if constexpr (kKind == KV_DTYPE_BF16) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (use) x = static_cast<const uint4*>(a.k_cache)[row * (D / 8) + t + 4 * c];
        o[0] = x.x;
        o[1] = x.y;
        o[2] = x.z;
        o[3] = x.w;
      } else {
        uint2 x = make_uint2(0u, 0u);
        if (use) x = static_cast<const uint2*>(a.k_cache)[row * (D / 8) + t + 4 * c];
        float v[4];
        code_values<kKind == KV_DTYPE_FP8_E4M3>(x.x, v);
        o[0] = pack2<false>(v[0], v[1]);
        o[1] = pack2<false>(v[2], v[3]);
        code_values<kKind == KV_DTYPE_FP8_E4M3>(x.y, v);
        o[2] = pack2<false>(v[0], v[1]);
        o[3] = pack2<false>(v[2], v[3]);
      }
    }
    if (kKind != KV_DTYPE_BF16 && use) kf[i] *= a.k_scale[(int64_t)p * a.num_kv_heads + hk];
  }
  return __all_sync(0xffffffffu, ok);
}

// S^T of the warp's 32 keys and the 8 rows of Q tile `nt`: s[i][e] = key
// g + 8 i, row 8 nt + 2t + e (unscaled).
template <int D>
__device__ __forceinline__ void score_tile(const unsigned char* qs, int nt, const uint32_t (&ka)[4][D / 8],
                                           float (&s)[4][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  const unsigned char* row = qs + (nt * 8 + g) * kQStride<D> + t * 16;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + c * 64);
    const uint32_t b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t fa[4] = {ka[2 * m][4 * c + 2 * h], ka[2 * m + 1][4 * c + 2 * h],
                                ka[2 * m][4 * c + 2 * h + 1], ka[2 * m + 1][4 * c + 2 * h + 1]};
        mma16816<false>(acc[m], fa, b[2 * h], b[2 * h + 1]);
      }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    s[2 * m][0] = acc[m][0];
    s[2 * m][1] = acc[m][1];
    s[2 * m + 1][0] = acc[m][2];
    s[2 * m + 1][1] = acc[m][3];
  }
}

// (m, l) of every row over the keys of one split: one CTA per (KV head,
// sequence, row tile x split); its warps take 32 keys in turn, each lane
// keeping (m, l) of its keys alone until the end.
template <int D, int BS, int kKind>
__global__ void __launch_bounds__(kWarps * 32) row_stats_kernel(const PromptArgs a) {
  extern __shared__ __align__(16) unsigned char qs[];
  __shared__ int pos[kRowTile];
  __shared__ float red[kWarps][kRowTile][2];
  __shared__ int cta_bad;
  const int hk = blockIdx.x, b = blockIdx.y;
  const int split = blockIdx.z % a.splits, tile = blockIdx.z / a.splits;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  int q0, n, L;
  if (!prompt_rows(a, b, BS, &q0, &n, &L)) {
    if (blockIdx.z == 0 && threadIdx.x == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    return;
  }
  const int64_t R = (int64_t)n * G;
  if ((int64_t)tile * kRowTile >= R) return;
  const int r0 = tile * kRowTile, rows = (int)(R - r0 < kRowTile ? R - r0 : kRowTile);
  const int first_pos = L - n + r0 / G, last_pos = L - n + (r0 + rows - 1) / G;
  const int kbeg = split * a.part_tokens;
  const int kend = min(last_pos + 1, kbeg + a.part_tokens);
  if (threadIdx.x == 0) cta_bad = 0;
  if (threadIdx.x < kRowTile)
    pos[threadIdx.x] = threadIdx.x < rows ? L - n + (r0 + (int)threadIdx.x) / G : -1;
  if (kbeg < kend) load_q_tile<D>(a, qs, q0, hk, G, r0, rows);
  __syncthreads();
  float m[kNTiles][2], l[kNTiles][2];
#pragma unroll
  for (int i = 0; i < kNTiles; ++i) m[i][0] = m[i][1] = -INFINITY, l[i][0] = l[i][1] = 0.0f;
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks;
  for (int k0 = kbeg + warp * kWarpKeys; k0 < kend; k0 += kCtaKeys) {
    uint32_t ka[4][D / 8];
    float kf[4];
    if (!load_keys<D, BS, kKind>(a, bt, hk, k0, kend, ka, kf)) cta_bad = 1;
    const bool whole = k0 + kWarpKeys <= kend && k0 + kWarpKeys - 1 <= first_pos;
#pragma unroll
    for (int nt = 0; nt < kNTiles; ++nt) {
      if (nt * 8 >= rows) break;
      float s[4][2];
      score_tile<D>(qs, nt, ka, s);
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int p = pos[nt * 8 + 2 * t + e];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = s[i][e] * kf[i];
          s[i][e] = whole || (k0 + g + 8 * i <= p && k0 + g + 8 * i < kend) ? v : -INFINITY;
          mx[e] = fmaxf(mx[e], s[i][e]);
        }
      }
      if (__any_sync(0xffffffffu, mx[0] > m[nt][0] || mx[1] > m[nt][1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[nt][e], mx[e]);
          l[nt][e] *= mn == -INFINITY ? 1.0f : ex2(m[nt][e] - mn);
          m[nt][e] = mn;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mz = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
#pragma unroll
        for (int i = 0; i < 4; ++i) l[nt][e] += ex2(s[i][e] - mz);
      }
    }
  }
  // join the lanes of a row (g), then the warps
#pragma unroll
  for (int nt = 0; nt < kNTiles; ++nt) {
    if (nt * 8 >= rows) break;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float M = m[nt][e];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      float x = M == -INFINITY ? 0.0f : l[nt][e] * ex2(m[nt][e] - M);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (g == 0) {
        red[warp][nt * 8 + 2 * t + e][0] = M;
        red[warp][nt * 8 + 2 * t + e][1] = x;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float M = -INFINITY, x = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[w][r][0]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (red[w][r][1] > 0.0f || red[w][r][1] != red[w][r][1])
        x = fmaf(ex2(red[w][r][0] - M), red[w][r][1], x);
    const int64_t row = (int64_t)(q0 + (r0 + r) / G) * a.num_q_heads + hk * G + (r0 + r) % G;
    float* o = a.stats + (row * a.splits + split) * 2;
    o[0] = M;
    o[1] = cta_bad ? -1.0f : x;                        // l < 0: the weights stay as they are
  }
  if (cta_bad && threadIdx.x == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
}

// Column sums: one CTA per (KV head, sequence, 128 keys), over every row that
// sees one of its keys.
template <int D, int BS, int kKind>
__global__ void __launch_bounds__(kWarps * 32) column_sums_kernel(const PromptArgs a) {
  extern __shared__ __align__(16) unsigned char qs[];
  __shared__ int pos[kRowTile];
  __shared__ float row_m[kRowTile], row_inv[kRowTile];
  const int hk = blockIdx.x, b = blockIdx.y;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  int q0, n, L;
  if (!prompt_rows(a, b, BS, &q0, &n, &L) || n == 0) return;
  const int c0 = blockIdx.z * kCtaKeys;                // the CTA's first key
  if (c0 >= L) return;
  const int k0 = c0 + warp * kWarpKeys;
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks;
  uint32_t ka[4][D / 8];
  float kf[4];
  load_keys<D, BS, kKind>(a, bt, hk, k0, L, ka, kf);    // (bad blocks: flagged with the row statistics)
  const int64_t R = (int64_t)n * G;
  const int seen = c0 - (L - n);                        // query token at the first key
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  for (int64_t rt = (seen > 0 ? (int64_t)seen * G : 0) / kRowTile * kRowTile; rt < R; rt += kRowTile) {
    const int r0 = (int)rt, rows = (int)(R - rt < kRowTile ? R - rt : kRowTile);
    __syncthreads();                                   // the last tile's reads are done
    load_q_tile<D>(a, qs, q0, hk, G, r0, rows);
    if (threadIdx.x < kRowTile) {
      const int r = threadIdx.x;
      float M = 0.0f, inv = 0.0f;
      int p = -1;
      if (r < rows) {
        p = L - n + (r0 + r) / G;
        const int64_t row = (int64_t)(q0 + (r0 + r) / G) * a.num_q_heads + hk * G + (r0 + r) % G;
        const float* st = a.stats + row * a.splits * 2;
        const int ns = p / a.part_tokens + 1;           // splits with keys of this row
        M = -INFINITY;
        float den = 0.0f;
        for (int i = 0; i < ns; ++i) M = fmaxf(M, st[2 * i]);
        for (int i = 0; i < ns; ++i) {
          bad |= st[2 * i + 1] < 0.0f;
          den = fmaf(exp2f(st[2 * i] - M), st[2 * i + 1], den);
        }
        inv = 1.0f / den;
      }
      pos[r] = p;
      row_m[r] = M;
      row_inv[r] = inv;
    }
    __syncthreads();
    const bool whole = rows == kRowTile && pos[0] >= k0 + kWarpKeys - 1;
#pragma unroll 2
    for (int nt = 0; nt < kNTiles; ++nt) {
      if (nt * 8 >= rows) break;
      float s[4][2];
      score_tile<D>(qs, nt, ka, s);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * t + e;
        const int p = pos[r];
        const float M = row_m[r], inv = row_inv[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = ex2(fmaf(s[i][e], kf[i], -M));
          sum[i] = fmaf(whole || k0 + g + 8 * i <= p ? w : 0.0f, inv, sum[i]);
        }
      }
    }
  }
  if (__syncthreads_or(bad)) return;                   // a bad block: the weights stay
  float* w = a.weights + ((int64_t)b * a.num_kv_heads + hk) * a.stride;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    const int key = k0 + g + 8 * i;
    if (t == 0 && key < L) w[key] = a.accumulate && key < L - n ? w[key] + sum[i] : sum[i];
  }
}

template <int D, int BS, int kKind>
kv_status launch_prompt_t(const PromptArgs& a, int tiles, cudaStream_t s) {
  const size_t smem = (size_t)kRowTile * kQStride<D>;
  const dim3 g1((unsigned)a.num_kv_heads, (unsigned)a.batch, (unsigned)(tiles * a.splits));
  row_stats_kernel<D, BS, kKind><<<g1, kWarps * 32, smem, s>>>(a);
  kv_status st = cuda_check(cudaGetLastError(), "row_stats_kernel launch");
  if (st != KV_OK) return st;
  const dim3 g2((unsigned)a.num_kv_heads, (unsigned)a.batch, (unsigned)((a.max_seq_len - 1) / kCtaKeys + 1));
  column_sums_kernel<D, BS, kKind><<<g2, kWarps * 32, smem, s>>>(a);
  return cuda_check(cudaGetLastError(), "column_sums_kernel launch");
}

template <int D, int BS>
kv_status launch_prompt_mma(const PromptArgs& a, kv_dtype dtype, int tiles, cudaStream_t s) {
  if (dtype == KV_DTYPE_INT8) return launch_prompt_t<D, BS, KV_DTYPE_INT8>(a, tiles, s);
  if (dtype == KV_DTYPE_FP8_E4M3) return launch_prompt_t<D, BS, KV_DTYPE_FP8_E4M3>(a, tiles, s);
  return launch_prompt_t<D, BS, KV_DTYPE_BF16>(a, tiles, s);
}

// Floats of a row of kept scores.
int64_t score_row(int max_seq_len) { return ((int64_t)max_seq_len + 7) & ~(int64_t)7; }

size_t step_need(int batch, int num_q_heads, int head_dim, int max_seq_len, int slots) {
  const size_t rows = (size_t)batch * num_q_heads;
  return (ml_region_floats(rows, slots) + (slots > 1 ? rows * slots * head_dim : 0) +
          rows * (size_t)score_row(max_seq_len)) * sizeof(float);
}

size_t prompt_need(int num_tokens, int num_q_heads, int splits) {
  return (size_t)num_tokens * num_q_heads * splits * 2 * sizeof(float);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" {

size_t pagedkv_weights_workspace_bytes(int batch, int num_q_heads, int head_dim, int max_seq_len,
                                       int block_size) {
  (void)block_size;
  if (batch <= 0 || num_q_heads <= 0 || head_dim <= 0 || max_seq_len <= 0) return 0;
  return step_need(batch, num_q_heads, head_dim, max_seq_len, (max_seq_len - 1) / kMinPartTokens + 1);
}

kv_status paged_attention_decode_weights(void* out, float* weights, int weights_stride, const void* q,
                                         const void* k_cache, const void* v_cache,
                                         const float* k_scale, const float* v_scale,
                                         const int32_t* block_tables, int max_blocks_per_seq,
                                         const int32_t* seq_lens, int batch, int num_q_heads,
                                         int num_kv_heads, int head_dim, int num_blocks,
                                         int block_size, int max_seq_len, float scale,
                                         kv_dtype dtype, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  const char* who = "paged_attention_decode_weights";
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
      max_blocks_per_seq <= 0 || num_blocks <= 0 || max_seq_len <= 0 || weights_stride <= 0 ||
      !valid_dtype(dtype))
    return fail(KV_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (num_q_heads / num_kv_heads > kMaxGroup)
    return fail(KV_ERR_INVALID_ARG, "%s: at most 8 query heads per KV head (got %d)", who,
                num_q_heads / num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return fail(KV_ERR_INVALID_ARG, "%s: head_dim must be 64 or 128", who);
  if (block_size != 16 && block_size != 32)
    return fail(KV_ERR_INVALID_ARG, "%s: block_size must be 16 or 32", who);
  if (weights_stride < max_seq_len)
    return fail(KV_ERR_INVALID_ARG, "%s: max_seq_len %d exceeds the weights' rows of %d", who,
                max_seq_len, weights_stride);
  if (batch > 65535 || num_kv_heads > 65535)
    return fail(KV_ERR_INVALID_ARG, "%s: at most 65535 sequences and KV heads", who);
  if (batch == 0) return KV_OK;
  if (!out || !weights || !q || !k_cache || !v_cache || !block_tables || !seq_lens)
    return fail(KV_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(KV_ERR_INVALID_ARG, "%s: out, q and the pools must be 16-byte aligned", who);
  const bool q8 = dtype != KV_DTYPE_BF16;
  if (q8 != (k_scale != nullptr) || q8 != (v_scale != nullptr))
    return fail(KV_ERR_INVALID_ARG, "%s: 8-bit pools need k_scale and v_scale; bf16 pools take NULL", who);
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  DecodeArgs a = {};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.flags = di.flags;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.batch = batch;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.max_seq_len = max_seq_len;
  a.part_tokens = choose_part_tokens(batch, num_kv_heads, max_seq_len, di.num_sms, true);
  a.max_parts = (max_seq_len - 1) / a.part_tokens + 1;
  a.reverse_parts = a.max_parts <= 8;
  a.slots = a.max_parts;
  a.scale_log2 = scale * kLog2e;
  a.dtype = dtype;
  const size_t need = step_need(batch, num_q_heads, head_dim, max_seq_len, a.slots);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(KV_ERR_INVALID_ARG,
                "%s: workspace must be 16-byte aligned and hold %zu bytes "
                "(pagedkv_weights_workspace_bytes gives a safe size)", who, need);
  const size_t rows = (size_t)batch * num_q_heads;
  a.ws_ml = static_cast<float*>(workspace);
  a.ws_acc = a.ws_ml + ml_region_floats(rows, a.slots);
  a.ws_scores = a.ws_acc + (a.slots > 1 ? rows * a.slots * head_dim : 0);  // (16-byte aligned rows)
  a.score_stride = score_row(max_seq_len);
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = launch_decode(a, s)) != KV_OK || (st = launch_merge(a, s)) != KV_OK) return st;
  StepArgs w = {};
  w.weights = weights;
  w.scores = a.ws_scores;
  w.ml = a.ws_ml;
  w.seq_lens = seq_lens;
  w.stride = weights_stride;
  w.score_stride = a.score_stride;
  w.num_q_heads = num_q_heads;
  w.num_kv_heads = num_kv_heads;
  w.part_tokens = a.part_tokens;
  w.slots = a.slots;
  const int64_t table = (int64_t)max_blocks_per_seq * block_size;
  w.max_len = (int)(table < max_seq_len ? table : max_seq_len);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((max_seq_len - 1) / kStepTokens + 1), (unsigned)num_kv_heads, (unsigned)batch);
  cfg.blockDim = dim3(kStepThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, step_weights_kernel, w), "step_weights_kernel launch");
}

size_t pagedkv_attention_weights_workspace_bytes(int num_tokens, int num_q_heads, int max_seq_len) {
  if (num_tokens <= 0 || num_q_heads <= 0 || max_seq_len <= 0) return 0;
  return prompt_need(num_tokens, num_q_heads, (max_seq_len - 1) / kMinPartTokens + 1);
}

kv_status pagedkv_attention_weights(float* weights, int weights_stride, const void* q,
                                    const void* k_cache, const float* k_scale,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* seq_lens, const int32_t* query_start, int batch,
                                    int num_tokens, int max_query_len, int num_q_heads,
                                    int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                    int max_seq_len, float scale, int accumulate, kv_dtype dtype,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "pagedkv_attention_weights";
  if (batch < 0 || num_tokens < 0 || max_query_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads || max_blocks_per_seq <= 0 || num_blocks <= 0 || max_seq_len <= 0 ||
      weights_stride <= 0 || !valid_dtype(dtype))
    return fail(KV_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != 64 && head_dim != 128)
    return fail(KV_ERR_INVALID_ARG, "%s: head_dim must be 64 or 128", who);
  if (block_size != 16 && block_size != 32)
    return fail(KV_ERR_INVALID_ARG, "%s: block_size must be 16 or 32", who);
  if (weights_stride < max_seq_len)
    return fail(KV_ERR_INVALID_ARG, "%s: max_seq_len %d exceeds the weights' rows of %d", who,
                max_seq_len, weights_stride);
  if (batch > 65535) return fail(KV_ERR_INVALID_ARG, "%s: at most 65535 sequences", who);
  if (batch == 0 || num_tokens == 0) return KV_OK;
  if (!weights || !q || !k_cache || !block_tables || !seq_lens || !query_start)
    return fail(KV_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned16(q) || !aligned16(k_cache))
    return fail(KV_ERR_INVALID_ARG, "%s: q and the pool must be 16-byte aligned", who);
  if ((dtype != KV_DTYPE_BF16) != (k_scale != nullptr))
    return fail(KV_ERR_INVALID_ARG, "%s: 8-bit pools need k_scale; bf16 pools take NULL", who);
  const int64_t G = num_q_heads / num_kv_heads;
  const int longest = max_query_len < num_tokens ? max_query_len : num_tokens;
  // Many rows per KV head: the tcgen05 kernels, whose row tile is 128 rows of
  // whole tokens; else the mma.sync kernels above.  (Their score scale is
  // positive.)  On bf16 pools they win from some 16 rows on (8 KV heads: 64 x
  // 512..4096 tokens x 48 rows 246 -> 176 us, four of 16K x 16 rows 132 -> 103, one
  // of 131072 x 20 rows 587 -> 209; 16 x 16K x 4 rows, two heads of 64: 43 -> 69).
  // On 8-bit pools a unit's keys are widened for one tile of rows, which pays for
  // more than 64 rows or in long sequences (one of 32K x 64 rows 248 -> 115, eight
  // of 32K x 48 rows 619 -> 527; 64 x 512..4096 x 48 rows 252 -> 365, four of 16K x
  // 16 rows 122 -> 160).
  const int64_t most_rows = longest * G;
  const bool tc = scale > 0.0f && G <= 128 &&
                  (most_rows > kRowTile || (dtype == KV_DTYPE_BF16 && most_rows >= 16) ||
                   (most_rows > 32 && max_seq_len >= 8192));
  const int64_t tile_tokens = tc ? 128 / G : 0;
  const int64_t tiles = tc ? (longest + tile_tokens - 1) / tile_tokens
                           : (longest * G + kRowTile - 1) / kRowTile;
  if (longest * G > 0x7fffff00LL || tiles > 65535 || tiles * batch > 0x7fffffffLL ||
      (max_seq_len - 1) / kCtaKeys + 1 > 65535)
    return fail(KV_ERR_INVALID_ARG, "%s: too many query tokens or too long sequences", who);
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  PromptArgs a = {};
  a.weights = weights;
  a.q = q;
  a.k_cache = k_cache;
  a.k_scale = k_scale;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.flags = di.flags;
  a.stride = weights_stride;
  a.batch = batch;
  a.num_tokens = num_tokens;
  a.max_query_len = max_query_len;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.part_tokens = choose_part_tokens((int)(tiles * batch), num_kv_heads, max_seq_len, di.num_sms, false, 1 << 17);
  a.splits = (max_seq_len - 1) / a.part_tokens + 1;
  a.accumulate = accumulate != 0;
  a.scale_log2 = scale * kLog2e;
  if (tiles * a.splits > 65535)
    return fail(KV_ERR_INVALID_ARG, "%s: too many query tokens or too long sequences", who);
  const size_t need = prompt_need(num_tokens, num_q_heads, a.splits);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(KV_ERR_INVALID_ARG,
                "%s: workspace must be 16-byte aligned and hold %zu bytes "
                "(pagedkv_attention_weights_workspace_bytes gives a safe size)", who, need);
  a.stats = static_cast<float*>(workspace);
  a.tile_tokens = (int)tile_tokens;
  cudaStream_t s = (cudaStream_t)stream;
  // Few rows whose scores fit a cluster's TMEM: one pass over K (64 sequences of
  // 512..4096 tokens, five queries each, 32/8 heads: two passes of the mma.sync
  // kernels 189 us, one pass 103; int8 196 and 140).
  const int ctas = longest * G <= kFewRows ? few_rows_ctas(batch, num_kv_heads, max_seq_len, di.num_sms) : 0;
  if (ctas > 0) {
    a.tile_tokens = (int)(kFewRows / G);
    return launch_prompt_few(a, head_dim, block_size, dtype, ctas, s);
  }
  if (tc) return launch_prompt_tc(a, head_dim, block_size, dtype, (int)tiles, s);
  if (head_dim == 128)
    return block_size == 32 ? launch_prompt_mma<128, 32>(a, dtype, (int)tiles, s)
                            : launch_prompt_mma<128, 16>(a, dtype, (int)tiles, s);
  return block_size == 32 ? launch_prompt_mma<64, 32>(a, dtype, (int)tiles, s)
                          : launch_prompt_mma<64, 16>(a, dtype, (int)tiles, s);
}

}  // extern "C"
