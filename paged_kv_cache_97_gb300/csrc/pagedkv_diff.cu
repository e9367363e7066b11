// pagedkv_diff.cu -- differential attention for one query token per sequence
// over the paged pool.
//
// A differential head h of KV head j has two query rows, 2h and 2h + 1, two
// keys per token, pool heads 2j and 2j + 1 of the K pool, and one value of
// 2 d elements per token, pool heads 2j and 2j + 1 of the V pool side by side:
//   a_i = softmax(scale q_i . K_i) V,   y = a_1 - lambda_h a_2,
//   out = y / sqrt(mean(y^2) + eps) * norm_weight      (norm_weight may be null)
//
// One CTA serves one (token partition, KV head and up to four of its heads,
// sequence), so every K and V byte is read once for up to four heads.  Both
// maps run in one pass: the 8 columns of the MMA tiles are (head, map) pairs,
// column 2i + m = map m of the CTA's head i, and lane 4g + t of a warp holds
// columns 2t and 2t + 1: both maps of head t.  Per 16-token tile
//   S^T[16 x 8] = K_1 . Q^T and K_2 . Q^T, of which the even columns of the
//   first and the odd ones of the second are the scores,
//   O^T[2 d x 8] += (V_1 | V_2)^T . P^T.
// P enters the second product in 16 bits.  a_1 - lambda a_2 may cancel, and the
// row is normalised after it, so an error of P counts times |a| / |y|.  On bf16
// pools P is therefore the sum of two bf16 numbers (2^-16 of it is lost, not
// bf16's 2^-8) and has two MMAs per V fragment: 109.7 -> 110.6 us on the batch
// below, 192.9 -> 194.2 with 8 heads over 8.  On 8-bit pools it is one fp16
// number (2^-11): a second one would cost 5 % there (82.6 -> 87.6 us on int8), for
// values that 8 bits hold to 2^-8 or worse.
//
// The pipeline (a producer warp issuing TMA loads of whole blocks, consumer
// warps with their own online softmax, partials joined by log-sum-exp) and the
// treatment of 8-bit codes are those of the decode kernel.
//
// Bound by the bytes of K and V: 64 sequences of 512..4096 tokens, 16 heads
// over 4 KV heads of 2 x 128 (bf16), 110.6 us, 5530 GB/s or 81 % of the copy
// rate; paged_attention_decode takes 105 for the same bytes.  Half of the scores'
// MMA columns are computed and not used (each K tile meets both maps'
// queries), which the tensor cores have to spare.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kDiffConsumers = 3;
constexpr int kThreads = (kDiffConsumers + 1) * 32;
constexpr int kHeads = 4;                              // differential heads per CTA
constexpr int kMaxBlocks = kMaxPartTokens / 16;        // blocks per partition
constexpr int kSpec = (kMaxBlocks + kThreads - 1) / kThreads;

template <int D, int BS, bool kQ8>
struct DiffGeo : Geo<D, BS, kQ8> {
  using G = Geo<D, BS, kQ8>;
  static constexpr int kPairBytes = 4 * G::kTensorBytes;              // K1, K2, V1, V2 of a block
  static constexpr int kStageBytes = kDiffConsumers * kPairBytes;
  static constexpr int kStages0 = kStageBudget / kStageBytes;
  static constexpr int kStages = kStages0 < 2 ? 2 : (kStages0 > kMaxStages ? kMaxStages : kStages0);
  static constexpr int kReduceBytes = kDiffConsumers * 8 * (2 + 2 * D) * 4;
  static constexpr int kSmemBytes =
      (kStages * kStageBytes > kReduceBytes ? kStages * kStageBytes : kReduceBytes) + 1024;
};

struct DiffArgs {
  DecodeArgs d;              // num_kv_heads = pool heads; q rows = 2 * num_heads
  const float* lam;          // [num_heads]
  const float* norm_weight;  // [2 * D] or null
  float eps;
  int num_heads;             // differential heads
  int kv_heads;              // differential KV heads
  int head_groups;           // CTAs per KV head: ceil(group / kHeads)
};

// One output row from y[k] = element lane + 32 k, written by one warp.
template <int D>
__device__ __forceinline__ void write_row(const DiffArgs& a, __nv_bfloat16* row, float (&y)[D / 16],
                                          int lane) {
  if (a.norm_weight) {
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) ss = fmaf(y[k], y[k], ss);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(ss * (1.0f / (2 * D)) + a.eps);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) y[k] *= r * a.norm_weight[lane + 32 * k];
  }
#pragma unroll
  for (int k = 0; k < D / 16; ++k) row[lane + 32 * k] = __float2bfloat16_rn(y[k]);
}

template <int D, int BS, bool kQ8, bool kFp8>
__global__ void __launch_bounds__(kThreads)
    diff_decode_kernel(const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const DiffArgs da) {
  using G = DiffGeo<D, BS, kQ8>;
  const DecodeArgs& a = da.d;
  constexpr int S = G::kStages;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full_bar[kMaxStages], empty_bar[kMaxStages];
  __shared__ int32_t blk_id[kMaxBlocks];
  // K scales of the two maps, V scales of the two value halves, each relative
  // to the CTA's largest of that half: the halves are different output elements
  // of pool heads with scales of their own, so under one maximum the half with
  // the smaller scales would have its probabilities in fp16's subnormals
  __shared__ float blk_ks[kQ8 ? 2 * kMaxBlocks : 1], blk_vr[kQ8 ? 2 * kMaxBlocks : 1];
  __shared__ int cta_bad, cta_timeout;
  __shared__ float v_max_scale[2];

  const int j = blockIdx.x / da.head_groups, hg = blockIdx.x % da.head_groups;
  const int part = a.reverse_parts ? (int)(gridDim.z - 1 - blockIdx.z) : (int)blockIdx.z;
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int GH = da.num_heads / da.kv_heads;           // heads per KV head
  const int nh = min(kHeads, GH - hg * kHeads);        // heads of this CTA
  const int h0 = j * GH + hg * kHeads;                 // its first head
  const int P = a.num_kv_heads;                        // pool heads
  const int ncols = 2 * nh;
  const int64_t row0 = ((int64_t)b * da.num_heads + h0) * 2;   // q row of column 0
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)b * da.num_heads + h0) * 2 * D;

  // block-table entries and q fragments before the length arrives
  const int t0 = part * a.part_tokens;
  const int first_blk = t0 / BS;
  const int spec_blk = min(a.part_tokens / BS, a.max_blocks_per_seq - first_blk);
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks_per_seq + first_blk;
  int32_t spec_id[kSpec];
#pragma unroll
  for (int r = 0; r < kSpec; ++r) {
    const int i = threadIdx.x + r * kThreads;
    spec_id[r] = i < spec_blk ? bt[i] : -1;
  }
  uint32_t qraw[G::kKSteps][2];
  if (warp < kDiffConsumers) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (row0 + (g < ncols ? g : 0)) * D;
#pragma unroll
    for (int ks = 0; ks < G::kKSteps; ++ks)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // (8-bit: the order in which a lane reads its chunks of a K row)
        constexpr int NC = D / 64;
        const int d0 = kQ8 ? 16 * (t * NC + ks / 4) + 4 * (ks % 4) + 2 * r : 16 * ks + 2 * t + 8 * r;
        qraw[ks][r] = g < ncols ? *reinterpret_cast<const uint32_t*>(q + d0) : 0u;
      }
  }

  const int L = a.seq_lens[b];
  if (L <= 0 || L > a.max_seq_len || (int64_t)L > (int64_t)a.max_blocks_per_seq * BS) {
    if (part == 0) {
      if (threadIdx.x == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
      for (int i = threadIdx.x; i < nh * 2 * D; i += kThreads) out[i] = __float2bfloat16_rn(0.0f);
    }
    return;
  }
  if (t0 >= L) return;
  const int t1 = min(t0 + a.part_tokens, L);
  const bool direct = L <= a.part_tokens;              // the row's only partial
  const int nblk = (t1 - 1) / BS - first_blk + 1;

  const uint32_t stages = (smem_addr(smem_raw) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    cta_bad = 0;
    cta_timeout = 0;
    v_max_scale[0] = v_max_scale[1] = 0.0f;
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_addr(&full_bar[s]), 1);
      mbar_init(smem_addr(&empty_bar[s]), kDiffConsumers);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSpec; ++r) {
    const int i = threadIdx.x + r * kThreads;
    if (i >= nblk) continue;
    const int32_t p = spec_id[r];
    const bool ok = p >= 0 && p < a.num_blocks;
    blk_id[i] = ok ? p : 0;
    if (!ok) cta_bad = 1;
    if constexpr (kQ8) {
      if (ok) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          blk_ks[2 * i + m] = a.k_scale[(int64_t)p * P + 2 * j + m];
          const float vs = a.v_scale[(int64_t)p * P + 2 * j + m];
          blk_vr[2 * i + m] = vs;
          atomicMax(reinterpret_cast<int*>(&v_max_scale[m]), __float_as_int(fabsf(vs)));
        }
      }
    }
  }
  __syncthreads();
  if constexpr (kQ8) {
    // p enters the second product times (V scale / the half's largest), in
    // fp16 range; the output is multiplied back by the largest
    for (int i = threadIdx.x; i < 2 * nblk; i += kThreads) {
      const float vmax = v_max_scale[i & 1];
      blk_vr[i] = blk_vr[i] / (vmax > 0.0f ? vmax : 1.0f);
    }
    __syncthreads();
  }
  const bool bad = cta_bad != 0;
  const int n_iter = (nblk + kDiffConsumers - 1) / kDiffConsumers;

  // softmax state of columns 2t, 2t + 1 and O^T of the two value halves
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
  float o[2][G::kMTiles][4];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < G::kMTiles; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.0f;

  if (!bad && warp == kDiffConsumers) {
    // ======================= producer =======================================
    int issued = 0;
    bool ok = true;
    for (int it = 0; it < n_iter; ++it) {
      const int s = it % S;
      if (it >= S && !mbar_wait(smem_addr(&empty_bar[s]), ((it / S) - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const int j0 = it * kDiffConsumers;
        const int cnt = min(kDiffConsumers, nblk - j0);
        const uint32_t fb = smem_addr(&full_bar[s]);
        mbar_expect_tx(fb, (uint32_t)(cnt * G::kPairBytes));
        for (int c = 0; c < cnt; ++c) {
          const int p = blk_id[j0 + c];
          const uint32_t dst = stages + (uint32_t)((s * kDiffConsumers + c) * G::kPairBytes);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int x = 0; x < G::kBoxes; ++x) {
              const uint32_t off = m * G::kTensorBytes + x * G::kBoxBytes;
              tma_load_4d(dst + off, &k_map, fb, x * G::kBoxElems, 2 * j + m, 0, p);
              tma_load_4d(dst + 2 * G::kTensorBytes + off, &v_map, fb, x * G::kBoxElems, 2 * j + m, 0, p);
            }
        }
      }
      __syncwarp();
      issued = it + 1;
    }
    for (int s = 0; s < S && s < issued; ++s) {        // every fill lands before the CTA moves on
      const int last = s + S * ((issued - 1 - s) / S);
      if (!mbar_wait(smem_addr(&full_bar[s]), (last / S) & 1)) ok = false;
    }
    if (!ok && lane == 0) cta_timeout = 1;
  } else if (!bad) {
    // ======================= consumers =====================================
    const int w = warp;
    constexpr bool kF16 = kQ8;
    uint32_t qf[G::kKSteps][2];
    float qscale = 1.0f;
    {
      float amax = 0.0f;
      if constexpr (kQ8) {
        // fp16 holds |q| < 65504: a power of two taken out where needed
#pragma unroll
        for (int ks = 0; ks < G::kKSteps; ++ks)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qraw[ks][r] << 16)),
                                     fabsf(__uint_as_float(qraw[ks][r] & 0xffff0000u))));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        int e = 0;
        if (amax >= 16384.0f) {
          frexpf(amax, &e);
          e -= 14;
        }
        qscale = ldexpf(1.0f, -e);
      }
#pragma unroll
      for (int ks = 0; ks < G::kKSteps; ++ks)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          qf[ks][r] = kQ8 ? pack2<true>(__uint_as_float(qraw[ks][r] << 16) * qscale,
                                        __uint_as_float(qraw[ks][r] & 0xffff0000u) * qscale)
                          : qraw[ks][r];
    }
    const float score_scale = a.scale_log2 / qscale;
    // P^T transpose sources: token 2t (and 2t+8) of column g sits in lane
    // (2t)*4 + g/2, token 2t+1 (2t+9) in the lane 4 higher
    const int src_a = (2 * t) * 4 + (g >> 1), src_b = src_a + 4;
    const uint32_t half_sel = (g & 1) ? 0x7632u : 0x5410u;

    bool ok = true;
    for (int it = 0; it < n_iter; ++it) {
      const int s = it % S;
      if (!mbar_wait(smem_addr(&full_bar[s]), (it / S) & 1)) {
        ok = false;
        break;
      }
      const int jb = it * kDiffConsumers + w;
      if (jb < nblk) {
        const uint32_t kb = stages + (uint32_t)((s * kDiffConsumers + w) * G::kPairBytes);
        const uint32_t vb = kb + 2 * G::kTensorBytes;
        const int valid = min(BS, L - (first_blk + jb) * BS);
        const float kf0 = kQ8 ? score_scale * blk_ks[2 * jb] : score_scale;
        const float kf1 = kQ8 ? score_scale * blk_ks[2 * jb + 1] : score_scale;

        // ---- scores: even columns from map 1, odd ones from map 2 -----------
        float sc[G::kTiles][4];
#pragma unroll
        for (int tile = 0; tile < G::kTiles; ++tile) {
          float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t km = kb + m * G::kTensorBytes;
            if constexpr (!kQ8) {
              const int row = tile * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
              for (int ks = 0; ks < G::kKSteps; ++ks) {
                uint32_t fa[4];
                ldsm_x4(fa, km + chunk_off<Geo<D, BS, kQ8>>(row, 2 * ks + (lane >> 4)));
                mma16816<false>(c[m], fa, qf[ks][0], qf[ks][1]);
              }
            } else {
              constexpr int NC = D / 64;
              uint32_t kw[2][NC][4];
#pragma unroll
              for (int rr = 0; rr < 2; ++rr)
#pragma unroll
                for (int ci = 0; ci < NC; ++ci) {
                  const uint4 v = lds128(km + chunk_off<Geo<D, BS, kQ8>>(tile * 16 + g + 8 * rr, t * NC + ci));
                  kw[rr][ci][0] = v.x ^ kCodeBias<kFp8>;
                  kw[rr][ci][1] = v.y ^ kCodeBias<kFp8>;
                  kw[rr][ci][2] = v.z ^ kCodeBias<kFp8>;
                  kw[rr][ci][3] = v.w ^ kCodeBias<kFp8>;
                }
#pragma unroll
              for (int ks = 0; ks < G::kKSteps; ++ks) {
                const uint32_t w0 = kw[0][ks / 4][ks % 4], w1 = kw[1][ks / 4][ks % 4];
                const uint32_t fa[4] = {codes_to_f16x2<kFp8>(w0, 0x4140u), codes_to_f16x2<kFp8>(w1, 0x4140u),
                                        codes_to_f16x2<kFp8>(w0, 0x4342u), codes_to_f16x2<kFp8>(w1, 0x4342u)};
                mma16816<true>(c[m], fa, qf[ks][0], qf[ks][1]);
              }
            }
          }
          const int tok_lo = tile * 16 + g, tok_hi = tok_lo + 8;
          sc[tile][0] = tok_lo < valid ? c[0][0] * kf0 : -INFINITY;
          sc[tile][1] = tok_lo < valid ? c[1][1] * kf1 : -INFINITY;
          sc[tile][2] = tok_hi < valid ? c[0][2] * kf0 : -INFINITY;
          sc[tile][3] = tok_hi < valid ? c[1][3] * kf1 : -INFINITY;
        }

        // ---- online softmax of columns 2t and 2t + 1 ------------------------
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int tile = 0; tile < G::kTiles; ++tile) {
          mx0 = fmaxf(mx0, fmaxf(sc[tile][0], sc[tile][2]));
          mx1 = fmaxf(mx1, fmaxf(sc[tile][1], sc[tile][3]));
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
        }
        const float mn0 = fmaxf(m_run[0], mx0), mn1 = fmaxf(m_run[1], mx1);
        const float al0 = exp2f(m_run[0] - mn0), al1 = exp2f(m_run[1] - mn1);
        m_run[0] = mn0;
        m_run[1] = mn1;
        l_run[0] *= al0;
        l_run[1] *= al1;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < G::kMTiles; ++i) {
            o[x][i][0] *= al0;
            o[x][i][1] *= al1;
            o[x][i][2] *= al0;
            o[x][i][3] *= al1;
          }

#pragma unroll
        for (int tile = 0; tile < G::kTiles; ++tile) {
          if (tile * 16 >= valid) break;
          const float p0 = exp2f(sc[tile][0] - mn0), p1 = exp2f(sc[tile][1] - mn1);
          const float p2 = exp2f(sc[tile][2] - mn0), p3 = exp2f(sc[tile][3] - mn1);
          l_run[0] += p0 + p2;
          l_run[1] += p1 + p3;
          // V rows past `valid` are zeroed (p is 0 there, the pool may hold
          // NaN patterns); int8 codes are always finite
          uint32_t mlo = 0xffffffffu, mhi = 0xffffffffu;
          if ((!kQ8 || kFp8) && valid < BS) {
            const int k0 = tile * 16 + 2 * t;
            mlo = (k0 < valid ? 0x0000ffffu : 0u) | (k0 + 1 < valid ? 0xffff0000u : 0u);
            mhi = (k0 + 8 < valid ? 0x0000ffffu : 0u) | (k0 + 9 < valid ? 0xffff0000u : 0u);
          }
          // P^T as the B operand: tokens 2t, 2t + 1 of column g, and those 8 up
          auto turned = [&](uint32_t r) {
            const uint32_t a = __shfl_sync(0xffffffffu, r, src_a), b = __shfl_sync(0xffffffffu, r, src_b);
            return prmt(a, b, half_sel);
          };
          uint32_t ph[2] = {0u, 0u};
          [[maybe_unused]] uint32_t pl[2] = {0u, 0u};     // bf16: what the rounding to ph left
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // (8-bit: one per value half, with its scale)
            if (x == 0 || kQ8) {
              const float vr = kQ8 ? blk_vr[2 * jb + x] : 1.0f;
              const float q0 = p0 * vr, q1 = p1 * vr, q2 = p2 * vr, q3 = p3 * vr;
              const uint32_t r0 = pack2<kF16>(q0, q1), r1 = pack2<kF16>(q2, q3);
              ph[0] = turned(r0);
              ph[1] = turned(r1);
              if constexpr (!kQ8) {
                auto left = [](uint32_t r, float lo, float hi) {
                  return pack2<false>(lo - __uint_as_float(r << 16), hi - __uint_as_float(r & 0xffff0000u));
                };
                pl[0] = turned(left(r0, q0, q1));
                pl[1] = turned(left(r1, q2, q3));
              }
            }
            const uint32_t vx = vb + x * G::kTensorBytes;
            if constexpr (!kQ8) {
              const int row = tile * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
              for (int i = 0; i < G::kMTiles; ++i) {
                uint32_t fa[4];
                ldsm_x4_t(fa, vx + chunk_off<Geo<D, BS, kQ8>>(row, 2 * i + ((lane >> 3) & 1)));
                fa[0] &= mlo;
                fa[1] &= mlo;
                fa[2] &= mhi;
                fa[3] &= mhi;
                mma16816<false>(o[x][i], fa, ph[0], ph[1]);
                mma16816<false>(o[x][i], fa, pl[0], pl[1]);
              }
            } else {
              constexpr int NB = D / 8;                 // bytes per lane per token
              constexpr int NW = NB / 4;
              uint32_t vw[4][NW];
#pragma unroll
              for (int rr = 0; rr < 4; ++rr) {
                const int row = tile * 16 + 2 * t + (rr & 1) + 8 * (rr >> 1);
                if constexpr (NB == 16) {
                  const uint4 v = lds128(vx + chunk_off<Geo<D, BS, kQ8>>(row, g));
                  vw[rr][0] = v.x ^ kCodeBias<kFp8>;
                  vw[rr][1] = v.y ^ kCodeBias<kFp8>;
                  vw[rr][2] = v.z ^ kCodeBias<kFp8>;
                  vw[rr][3] = v.w ^ kCodeBias<kFp8>;
                } else {
                  const uint2 v = lds64(vx + chunk_off<Geo<D, BS, kQ8>>(row, g / 2) + (g & 1) * 8);
                  vw[rr][0] = v.x ^ kCodeBias<kFp8>;
                  vw[rr][1] = v.y ^ kCodeBias<kFp8>;
                }
              }
#pragma unroll
              for (int i = 0; i < G::kMTiles; ++i) {
                const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;  // bytes 2,3 or 0,1
                const uint32_t ulo = prmt(vw[0][i / 2], vw[1][i / 2], sel);  // tokens 2t, 2t+1
                const uint32_t uhi = prmt(vw[2][i / 2], vw[3][i / 2], sel);  // tokens 2t+8, 2t+9
                uint32_t fa[4] = {codes_to_f16x2<kFp8>(ulo, 0x4140u), codes_to_f16x2<kFp8>(ulo, 0x4342u),
                                  codes_to_f16x2<kFp8>(uhi, 0x4140u), codes_to_f16x2<kFp8>(uhi, 0x4342u)};
                if constexpr (kFp8) {
                  fa[0] &= mlo;
                  fa[1] &= mlo;
                  fa[2] &= mhi;
                  fa[3] &= mhi;
                }
                mma16816<true>(o[x][i], fa, ph[0], ph[1]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&empty_bar[s]));
    }
    if (!ok) cta_timeout = 1;
  }

  // ---- combine the consumer warps -------------------------------------------
  __syncthreads();  // all fills landed and all stage reads done
  const bool failed = bad || cta_timeout != 0;
  float* red = reinterpret_cast<float*>(smem_raw + (stages - smem_addr(smem_raw)));
  float* red_m = red;                                   // [consumers][8]
  float* red_l = red + kDiffConsumers * 8;
  float* red_acc = red + 2 * kDiffConsumers * 8;        // [consumers][8][2 D]
  if (!failed && warp < kDiffConsumers) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l_run[0] += __shfl_xor_sync(0xffffffffu, l_run[0], off);
      l_run[1] += __shfl_xor_sync(0xffffffffu, l_run[1], off);
    }
    if (g == 0) {
      red_m[warp * 8 + 2 * t] = m_run[0];
      red_m[warp * 8 + 2 * t + 1] = m_run[1];
      red_l[warp * 8 + 2 * t] = l_run[0];
      red_l[warp * 8 + 2 * t + 1] = l_run[1];
    }
    float* acc = red_acc + warp * 8 * 2 * D;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < G::kMTiles; ++i) {
        const int d_lo = x * D + (kQ8 ? g * (D / 8) + 2 * i : 16 * i + g);
        const int d_hi = d_lo + (kQ8 ? 1 : 8);
        acc[(2 * t) * 2 * D + d_lo] = o[x][i][0];
        acc[(2 * t + 1) * 2 * D + d_lo] = o[x][i][1];
        acc[(2 * t) * 2 * D + d_hi] = o[x][i][2];
        acc[(2 * t + 1) * 2 * D + d_hi] = o[x][i][3];
      }
  }
  __syncthreads();

  if (failed && threadIdx.x == 0)
    atomicOr(a.flags, bad ? PAGEDKV_FLAG_BAD_BLOCK : PAGEDKV_FLAG_WAIT_TIMEOUT);
  float out_scale[2] = {1.0f, 1.0f};
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (kQ8 && v_max_scale[x] > 0.0f) out_scale[x] = v_max_scale[x];
  // column c's joined element e, max and denominator over the warps
  auto joined = [&](int c, int e, float* M, float* den) {
    *M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDiffConsumers; ++w) *M = fmaxf(*M, red_m[w * 8 + c]);
    float num = 0.0f;
    *den = 0.0f;
#pragma unroll
    for (int w = 0; w < kDiffConsumers; ++w) {
      const float f = exp2f(red_m[w * 8 + c] - *M);     // 0 for a warp that saw no token
      num = fmaf(f, red_acc[(w * 8 + c) * 2 * D + e], num);
      *den = fmaf(f, red_l[w * 8 + c], *den);
    }
    return num * (e < D ? out_scale[0] : out_scale[1]);
  };
  if (direct) {
    for (int i = warp; i < nh; i += kThreads / 32) {
      float y[D / 16];
      const float lam = da.lam[h0 + i];
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        float M, den1, den2;
        if (failed) {
          y[k] = 0.0f;
          continue;
        }
        const float a1 = joined(2 * i, lane + 32 * k, &M, &den1);
        const float a2 = joined(2 * i + 1, lane + 32 * k, &M, &den2);
        y[k] = a1 / den1 - lam * (a2 / den2);
      }
      if (failed) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) out[i * 2 * D + lane + 32 * k] = __float2bfloat16_rn(0.0f);
      } else {
        write_row<D>(da, out + i * 2 * D, y, lane);
      }
    }
  } else {
    for (int i = threadIdx.x; i < ncols * 2 * D; i += kThreads) {
      const int c = i / (2 * D), e = i % (2 * D);
      const int64_t r = (row0 + c) * a.slots + part;
      float M = 0.0f, den = -1.0f, num = 0.0f;          // l < 0 marks the row bad for the merge
      if (!failed) num = joined(c, e, &M, &den);
      a.ws_acc[r * 2 * D + e] = num;
      if (e == 0) {
        a.ws_ml[2 * r] = M;
        a.ws_ml[2 * r + 1] = den;
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the partials of both maps of one head (one CTA per (sequence, head)):
// even warps take the first map's partials in turn, odd ones the second's, and
// warp 0 writes the row.
template <int D>
__global__ void __launch_bounds__(512) diff_merge_kernel(const DiffArgs da) {
  extern __shared__ float merge_red[];                  // [warps][2 D + 1]
  const DecodeArgs& a = da.d;
  const int b = blockIdx.x / da.num_heads, h = blockIdx.x % da.num_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = a.seq_lens[b];
  if (L <= a.part_tokens || L > a.max_seq_len ||
      (int64_t)L > (int64_t)a.max_blocks_per_seq * a.block_size)
    return;                                             // written whole, or zeroed
  const int np = (L + a.part_tokens - 1) / a.part_tokens;
  constexpr int E = D / 64;                             // float4 pieces per lane
  const int64_t row = ((int64_t)b * da.num_heads + h) * 2 + (warp & 1);
  const float* ml = a.ws_ml + row * a.slots * 2;
  const float4* acc = reinterpret_cast<const float4*>(a.ws_acc + row * a.slots * 2 * D) + lane;
  bool bad = false;
  float M = -INFINITY;
  for (int i = lane; i < np; i += 32) {
    M = fmaxf(M, ml[2 * i]);
    bad |= ml[2 * i + 1] < 0.0f;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float4 num[E];
  float den = 0.0f;
#pragma unroll
  for (int k = 0; k < E; ++k) num[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp >> 1; i < np; i += warps >> 1) {
    const float w = exp2f(ml[2 * i] - M);
    den = fmaf(w, ml[2 * i + 1], den);
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float4 x = acc[(int64_t)i * (D / 2) + 32 * k];
      num[k].x = fmaf(w, x.x, num[k].x);
      num[k].y = fmaf(w, x.y, num[k].y);
      num[k].z = fmaf(w, x.z, num[k].z);
      num[k].w = fmaf(w, x.w, num[k].w);
    }
  }
  float* r = merge_red + warp * (2 * D + 4);
#pragma unroll
  for (int k = 0; k < E; ++k) reinterpret_cast<float4*>(r)[lane + 32 * k] = num[k];
  if (lane == 0) r[2 * D] = den;
  if (__syncthreads_or(bad)) {
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x)
      static_cast<__nv_bfloat16*>(a.out)[((int64_t)b * da.num_heads + h) * 2 * D + i] = __float2bfloat16_rn(0.0f);
    return;
  }
  if (warp != 0) return;
  float y[D / 16], a2[D / 16], d1 = 0.0f, d2 = 0.0f;
#pragma unroll
  for (int k = 0; k < D / 16; ++k) y[k] = a2[k] = 0.0f;
  for (int w = 0; w < warps; w += 2) {
    const float* r1 = merge_red + w * (2 * D + 4);
    const float* r2 = r1 + 2 * D + 4;
    d1 += r1[2 * D];
    d2 += r2[2 * D];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      y[k] += r1[lane + 32 * k];
      a2[k] += r2[lane + 32 * k];
    }
  }
  const float lam = da.lam[h];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) y[k] = y[k] / d1 - lam * (a2[k] / d2);
  write_row<D>(da, static_cast<__nv_bfloat16*>(a.out) + ((int64_t)b * da.num_heads + h) * 2 * D, y, lane);
}

template <int D, int BS, bool kQ8, bool kFp8>
kv_status launch_diff_t(const DiffArgs& da, int dev, cudaStream_t s) {
  using G = DiffGeo<D, BS, kQ8>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  kv_status st;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      st = cuda_check(cudaFuncSetAttribute(diff_decode_kernel<D, BS, kQ8, kFp8>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmemBytes),
                      "cudaFuncSetAttribute(diff_decode_kernel)");
      if (st != KV_OK) return st;
      attr_set[dev] = true;
    }
  }
  alignas(64) CUtensorMap km, vm;
  if ((st = make_kv_maps(da.d, &km, &vm)) != KV_OK) return st;
  const dim3 grid((unsigned)(da.kv_heads * da.head_groups), (unsigned)da.d.batch, (unsigned)da.d.max_parts);
  diff_decode_kernel<D, BS, kQ8, kFp8><<<grid, kThreads, G::kSmemBytes, s>>>(km, vm, da);
  if ((st = cuda_check(cudaGetLastError(), "diff_decode_kernel launch")) != KV_OK) return st;
  if (da.d.max_parts == 1) return KV_OK;
  // about 4 partials per warp, an even number of warps
  int warps = 2 * ((da.d.max_parts + 3) / 4);
  warps = warps > 16 ? 16 : warps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(da.d.batch * da.num_heads));
  cfg.blockDim = dim3((unsigned)(32 * warps));
  cfg.dynamicSmemBytes = (size_t)warps * (2 * D + 4) * sizeof(float);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, diff_merge_kernel<D>, da), "diff_merge_kernel launch");
}

template <int D, int BS>
kv_status launch_diff(const DiffArgs& a, int dev, cudaStream_t s) {
  if (a.d.dtype == KV_DTYPE_FP8_E4M3) return launch_diff_t<D, BS, true, true>(a, dev, s);
  return a.d.dtype == KV_DTYPE_INT8 ? launch_diff_t<D, BS, true, false>(a, dev, s)
                                    : launch_diff_t<D, BS, false, false>(a, dev, s);
}

size_t diff_need(int batch, int num_heads, int head_dim, int parts) {
  return decode_workspace_need(batch, 2 * num_heads, 2 * head_dim, parts);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" {

size_t pagedkv_diff_workspace_bytes(int batch, int num_heads, int head_dim, int max_seq_len,
                                    int block_size) {
  (void)block_size;
  if (batch <= 0 || num_heads <= 0 || head_dim <= 0 || max_seq_len <= 0) return 0;
  return diff_need(batch, num_heads, head_dim, (max_seq_len - 1) / kMinPartTokens + 1);
}

kv_status paged_diff_attention_decode(void* out, const void* q, const void* k_cache,
                                      const void* v_cache, const float* k_scale,
                                      const float* v_scale, const int32_t* block_tables,
                                      int max_blocks_per_seq, const int32_t* seq_lens, int batch,
                                      int num_heads, int num_kv_heads, int head_dim, int num_blocks,
                                      int block_size, int max_seq_len, float scale,
                                      const float* lambda, const float* norm_weight, float eps,
                                      kv_dtype dtype, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  const char* who = "paged_diff_attention_decode";
  if (batch < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads ||
      max_blocks_per_seq <= 0 || num_blocks <= 0 || max_seq_len <= 0 || !valid_dtype(dtype))
    return fail(KV_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (head_dim != 64 && head_dim != 128)
    return fail(KV_ERR_INVALID_ARG, "%s: head_dim must be 64 or 128", who);
  if (block_size != 16 && block_size != 32)
    return fail(KV_ERR_INVALID_ARG, "%s: block_size must be 16 or 32", who);
  if (norm_weight && !(eps >= 0.0f))
    return fail(KV_ERR_INVALID_ARG, "%s: eps must not be negative", who);
  if (batch > 65535 || num_heads > 65535)
    return fail(KV_ERR_INVALID_ARG, "%s: at most 65535 sequences and heads", who);
  if (batch == 0) return KV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !lambda)
    return fail(KV_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(KV_ERR_INVALID_ARG, "%s: out, q and the pools must be 16-byte aligned", who);
  const bool q8 = dtype != KV_DTYPE_BF16;
  if (q8 != (k_scale != nullptr) || q8 != (v_scale != nullptr))
    return fail(KV_ERR_INVALID_ARG, "%s: 8-bit pools need k_scale and v_scale; bf16 pools take NULL", who);
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  DiffArgs da = {};
  da.lam = lambda;
  da.norm_weight = norm_weight;
  da.eps = eps;
  da.num_heads = num_heads;
  da.kv_heads = num_kv_heads;
  da.head_groups = (num_heads / num_kv_heads + kHeads - 1) / kHeads;
  DecodeArgs& a = da.d;
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
  a.num_q_heads = 2 * num_heads;
  a.num_kv_heads = 2 * num_kv_heads;
  a.head_dim = head_dim;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.max_seq_len = max_seq_len;
  a.part_tokens = choose_part_tokens(batch, num_kv_heads * da.head_groups, max_seq_len, di.num_sms, true);
  a.max_parts = (max_seq_len - 1) / a.part_tokens + 1;
  if (a.max_parts > 65535) return fail(KV_ERR_INVALID_ARG, "%s: too many partitions", who);
  a.reverse_parts = a.max_parts <= 8;
  a.slots = a.max_parts;
  a.scale_log2 = scale * kLog2e;
  a.dtype = dtype;
  const size_t need = diff_need(batch, num_heads, head_dim, a.max_parts);
  if (need > 0) {
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
      return fail(KV_ERR_INVALID_ARG,
                  "%s: workspace must be 16-byte aligned and hold %zu bytes "
                  "(pagedkv_diff_workspace_bytes gives a safe size)", who, need);
    a.ws_ml = static_cast<float*>(workspace);
    a.ws_acc = a.ws_ml + ml_region_floats((size_t)batch * 2 * num_heads, a.slots);
  }
  cudaStream_t s = (cudaStream_t)stream;
  if (head_dim == 128)
    return block_size == 32 ? launch_diff<128, 32>(da, di.device, s) : launch_diff<128, 16>(da, di.device, s);
  return block_size == 32 ? launch_diff<64, 32>(da, di.device, s) : launch_diff<64, 16>(da, di.device, s);
}

}  // extern "C"
