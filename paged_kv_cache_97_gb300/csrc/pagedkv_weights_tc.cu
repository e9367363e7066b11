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
// fixed row per thread (a TMEM lane) and take the even chunks, warps 4-7 the
// odd ones (so a set, a stage and a TMEM buffer go together), warp 8 issues
// the MMAs (S[128 x 128] = fixed . streamed^T into one of two TMEM buffers),
// warp 9 the TMA loads and, in the column sums, each row tile's m'.  A query tile is whole tokens, tile_tokens = 128 / G of them times the G
// heads, as one TMA box; rows past the sequence's queries are masked.
//
// What bounds it is the exponentials, 16 per clock and SM: a 128 x 128 tile has
// 16384 of them, 1024 cycles against 256 of MMA, and one prompt of 16K tokens
// (32/8 heads, bf16) takes about 1030 per tile and pass: 1857 us.  Beside each
// stand one packed half of a multiply-add and of an add (f32x2) and no
// maximum: a row's reference is its first scores' and moves only when a sum
// grows past 2^60.  4 prompts of 1..4K tokens take 267 us, where the
// exponentials alone would take about 229; the rest is the CTAs' start and end
// and the masked halves of diagonal tiles.  Measured and not taken: the fixed
// operand in TMEM and the streamed tiles shared by two CTAs through TMA
// multicast (1857 -> 1870..1880 us, 267 -> 286..288): the feeding of the MMA is
// not what it waits for.
//
// 8-bit pools: the row warps load the codes themselves, widen them to bf16
// (exact: 8 significant bits hold every int8 and E4M3 code) and write them into
// the swizzled image, the streamed keys two chunks ahead, right after the
// scores of the chunk that used the stage before; a block's K scale multiplies
// its scores (one prompt of 8K tokens, E4M3: 791 us).  Two CTAs per SM (256
// TMEM columns and about 100 KB of shared memory each), so that one's start
// and end overlap the other's work.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_requant.cuh"
#include "pagedkv_tc.cuh"
#include "pagedkv_weights.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kTile = 128;                             // rows of either operand
constexpr int kStages = 2;                             // = TMEM buffers
constexpr int kRowWarps = 8;                           // two sets of four, by the chunk's parity
constexpr int kSetWarps = kRowWarps / 2, kSetThreads = kSetWarps * 32;
constexpr int kMmaWarp = kRowWarps, kLoadWarp = kRowWarps + 1;
constexpr int kThreads = (kRowWarps + 2) * 32;
constexpr int kRowSlots = 8;                           // chunks whose rows' m' may be in use
constexpr int kTmemCols = kStages * kTile;
constexpr float kMoveSum = 0x1p60f;                    // a sum of 32 that moves a row's reference

template <int D>
struct PGeo {
  static constexpr int kBands = D / 64;
  static constexpr int kImage = kTile * D * 2;         // bytes of 128 rows
  static constexpr int kUsed = (1 + kStages) * kImage + 1024;
  // at least 100 KB, so that no more than two CTAs (512 TMEM columns) share an SM
  static constexpr int kSmemBytes = kUsed > 100 * 1024 ? kUsed : 100 * 1024;
};

__device__ __forceinline__ uint64_t pack_f32x2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t both(float x) { return pack_f32x2(__float_as_uint(x), __float_as_uint(x)); }

// 2^x of both halves.
__device__ __forceinline__ uint64_t ex2_f32x2(uint64_t v) {
  float lo, hi;
  unpack_f32x2(v, lo, hi);
  return pack_f32x2(__float_as_uint(ex2(lo)), __float_as_uint(ex2(hi)));
}

// Sum of the halves of two pairs.
__device__ __forceinline__ float sum_f32x2(uint64_t a, uint64_t b) {
  float lo, hi;
  unpack_f32x2(add_f32x2(a, b), lo, hi);
  return lo + hi;
}

// raw *= f (the first 16 by f0, the others by f1).
__device__ __forceinline__ void scale_scores(uint32_t* raw, float f0, float f1) {
  const uint64_t f[2] = {both(f0), both(f1)};
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    float lo, hi;
    uint64_t v = pack_f32x2(raw[j], raw[j + 1]);
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(f[j >> 4]));
    unpack_f32x2(v, lo, hi);
    raw[j] = __float_as_uint(lo);
    raw[j + 1] = __float_as_uint(hi);
  }
}

// sum over 32 scores of 2^(s sl2 + off).
__device__ __forceinline__ float exp_sum(const uint32_t* raw, float sl2, float off) {
  const uint64_t f = both(sl2), o = both(off);
  uint64_t s[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int j = 0; j < 32; j += 2)
    s[(j >> 1) & 3] = add_f32x2(s[(j >> 1) & 3], ex2_f32x2(fma_f32x2(pack_f32x2(raw[j], raw[j + 1]), f, o)));
  return sum_f32x2(add_f32x2(s[0], s[1]), add_f32x2(s[2], s[3]));
}

// Running statistics of a query row: l = sum of 2^(s sl2 - ref).  Any
// reference serves as long as nothing overflows (fp32 sums keep their relative
// precision), so it is the largest of the row's first scores and moves only
// when 32 scores sum to more than 2^60 against it.
struct RowStats {
  float ref, l;
};

__device__ __forceinline__ float largest(const uint32_t* raw) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(raw[j]));
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// 32 scores of the row (of keys up to `lim` of the 32 unless `whole`).
__device__ __forceinline__ void add_scores(RowStats& st, uint32_t* raw, float sl2, bool whole, int lim) {
  if (!whole) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j > lim) raw[j] = 0xff800000u;               // -inf
  }
  if (st.ref == -INFINITY) st.ref = largest(raw) * sl2;
  float part = exp_sum(raw, sl2, st.ref == -INFINITY ? 0.0f : -st.ref);
  if (part > kMoveSum) {
    const float m = largest(raw) * sl2;
    st.l *= ex2(st.ref - m);
    st.ref = m;
    part = exp_sum(raw, sl2, -m);
  }
  st.l += part;
}

// sum over 32 rows of 2^(s sl2 - m'), neg_m = -m' (rows in [from, to) of the
// 32 when kMask).
template <bool kMask>
__device__ __forceinline__ float column_part(const uint32_t* raw, float sl2, const float* neg_m,
                                             int from, int to) {
  const uint64_t f = both(sl2);
  uint64_t s[2] = {0ull, 0ull};
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const uint4 m = *reinterpret_cast<const uint4*>(neg_m + j);
    uint64_t e0 = ex2_f32x2(fma_f32x2(pack_f32x2(raw[j], raw[j + 1]), f, pack_f32x2(m.x, m.y)));
    uint64_t e1 = ex2_f32x2(fma_f32x2(pack_f32x2(raw[j + 2], raw[j + 3]), f, pack_f32x2(m.z, m.w)));
    if constexpr (kMask) {
      float a, b, c, d;
      unpack_f32x2(e0, a, b);
      unpack_f32x2(e1, c, d);
      a = j >= from && j < to ? a : 0.0f;
      b = j + 1 >= from && j + 1 < to ? b : 0.0f;
      c = j + 2 >= from && j + 2 < to ? c : 0.0f;
      d = j + 3 >= from && j + 3 < to ? d : 0.0f;
      e0 = pack_f32x2(__float_as_uint(a), __float_as_uint(b));
      e1 = pack_f32x2(__float_as_uint(c), __float_as_uint(d));
    }
    s[0] = add_f32x2(s[0], e0);
    s[1] = add_f32x2(s[1], e1);
  }
  return sum_f32x2(s[0], s[1]);
}

// m + log2 l of a row.
__device__ __forceinline__ float row_log_sum(float m, float l) {
  return m == -INFINITY ? __uint_as_float(0x7fc00000u) : m + log2f(l);
}

// 8-bit pools: the codes of the 128 keys from `from` (zeros from L on), loaded
// by one set of row warps and widened into a swizzled bf16 image; a piece is 16
// codes of a key.
template <int D, int BS, int kKind>
struct Codes {
  static constexpr int kRowPieces = D / 16;
  static constexpr int kParts = 2;                       // held one at a time
  static constexpr int kPieces = kTile * kRowPieces / kSetThreads / kParts;
  uint4 x[kPieces];

  __device__ __forceinline__ static int piece(int part, int u) {
    return (part * kPieces + u) * kSetThreads + (int)(threadIdx.x % kSetThreads);
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
        *reinterpret_cast<uint4*>(img + (c / 8) * (kTile * 128) + sw128(r, c % 8)) =
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

template <int D, int BS, int kKind, bool kStats>
__global__ void __launch_bounds__(kThreads, 2)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap q_map, const PromptArgs a) {
  using P = PGeo<D>;
  constexpr bool kQ8 = kKind != KV_DTYPE_BF16;
  constexpr bool kWidenStream = kQ8 && kStats, kWidenFixed = kQ8 && !kStats;
  constexpr int kRead = kWidenStream ? 32 : 64;        // scores of a row in registers at a time
  constexpr int kScaleSlots = 4;                       // chunks whose scales may be in use
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t fixed_full, full[kStages], empty[kStages], s_full[kStages], buf_free[kStages],
      stat_full[kRowSlots], drain_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int sh_bad, sh_fail;
  __shared__ __align__(16) float row_m[kStats ? 1 : kRowSlots][kTile];  // -m' of the row tiles' rows
  __shared__ float half_part[kTile], half_ref[kTile];  // the odd chunks' results
  __shared__ float blk_ks[kWidenStream ? kScaleSlots : 1][kTile / BS];  // K scales of the chunks' blocks
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x, b = blockIdx.y;
  const int G = a.num_q_heads / a.num_kv_heads, TT = a.tile_tokens;
  int q0, n, L;
  const bool ok_seq = prompt_rows(a, b, BS, &q0, &n, &L);
  if (!ok_seq) {
    if (kStats && blockIdx.z == 0 && tid == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    if (!kStats) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // The unit.  Row statistics: row tile (the last ones, with most keys, first)
  // and key split; column sums: key tile.
  const int split = kStats ? (int)(blockIdx.z % a.splits) : 0;
  const int unit = kStats ? (int)((gridDim.z - 1 - blockIdx.z) / a.splits) : (int)blockIdx.z;
  const int i0 = unit * TT;                            // first query token of the fixed tile
  const int tn = min(TT, n - i0);                      // its tokens
  const int k0 = kStats ? split * a.part_tokens : unit * kTile;  // first key
  if (kStats ? tn <= 0 : (n == 0 || k0 >= L)) {
    if (!kStats) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int first_pos = L - n + i0;
  const int kend = kStats ? min(first_pos + tn, k0 + a.part_tokens) : min(L, k0 + kTile);
  const int rt0 = kStats ? 0 : max(0, k0 - (L - n)) / TT;        // first row tile that sees a key
  const int nch = kStats ? max(0, (kend - k0 + kTile - 1) / kTile) : (n - 1) / TT + 1 - rt0;
  // statistics of row 0 of the tile that starts at token i: [Hkv][T][G], so
  // that a tile's rows lie together
  auto stats_at = [&](int i) {
    return a.stats + ((int64_t)hk * a.num_tokens + q0 + i) * G * a.splits * 2;
  };
  const int my_rows = kStats ? tn * G : 0;
  if (kStats && nch == 0) {                            // no key of this split
    if (tid < my_rows) {
      float* o = stats_at(i0) + ((int64_t)tid * a.splits + split) * 2;
      o[0] = -INFINITY;
      o[1] = 0.0f;
    }
    return;
  }

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - smem_addr(smem_raw));
  auto stage_img = [&](int s) { return base + (uint32_t)((1 + s) * P::kImage); };
  if (tid == 0) {
    sh_bad = 0;
    sh_fail = 0;
    mbar_init(smem_addr(&fixed_full), kWidenFixed ? kSetWarps : 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&full[s]), kWidenStream ? kSetWarps : 1);
      mbar_init(smem_addr(&empty[s]), 1);
      mbar_init(smem_addr(&s_full[s]), 1);
      mbar_init(smem_addr(&buf_free[s]), kSetWarps);
    }
    for (int s = 0; s < kRowSlots; ++s) mbar_init(smem_addr(&stat_full[s]), 1);
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
  if (kStats) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tm = tmem_base;
  const int32_t* bt = a.block_tables + (int64_t)b * a.max_blocks;

  RowStats st = {-INFINITY, 0.0f};
  float acc = 0.0f;

  if (warp == kLoadWarp) {
    // ======================= loads (TMA) ====================================
    // Keys [from, from + 128) (up to L) into an image, one block per lane: its
    // table entry, read ahead of the wait for the image, then the load.
    auto entry = [&](int from) {
      return lane < min(kTile / BS, (L - from + BS - 1) / BS) ? bt[from / BS + lane] : 0;
    };
    auto load_k = [&](uint32_t img, uint64_t* bar, int from, int p) {
      const int nb = min(kTile / BS, (L - from + BS - 1) / BS);
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
    else if (!kQ8) load_k(base, &fixed_full, k0, entry(k0));
    // column sums: m' of the rows of chunk c's row tile
    [[maybe_unused]] float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto fetch = [&](int c) {
      const int i = (rt0 + c) * TT, rows = min(TT, n - i) * G;
      const float* st_row = stats_at(i);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = u * 32 + lane;
        m[u] = r < rows ? st_row[(int64_t)r * a.splits * 2] : 0.0f;
      }
    };
    int issued = 0;
    bool ok = true, bad = false;
    [[maybe_unused]] int next = kStats && !kWidenStream ? entry(k0) : 0;
    for (int c = 0; c < (kWidenStream ? 0 : nch); ++c) {
      const int s = c % kStages;
      if (c >= kStages && !warp_wait(smem_addr(&empty[s]), ((c / kStages) - 1) & 1)) {
        ok = false;
        break;
      }
      if (kStats) {
        load_k(stage_img(s), &full[s], k0 + c * kTile, next);
        next = entry(k0 + (c + 1) * kTile);
      }
      if (!kStats) load_q(stage_img(s), &full[s], (rt0 + c) * TT);
      issued = c + 1;
      if constexpr (!kStats) {
        if (c == 0) {
          // The kernel may start beside the last CTAs of the one before it (a
          // programmatic dependent); from here on that one has ended.
          asm volatile("griddepcontrol.wait;" ::: "memory");
          fetch(0);
        }
        // (the MMA of chunk c - 2 is done, so chunk c - 4's scores were read, and
        // before them chunk c - 6 was finished: its slot and barrier phase are free)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          bad |= m[u] == -INFINITY;                    // a row without statistics
          row_m[c % kRowSlots][u * 32 + lane] = -m[u];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&stat_full[c % kRowSlots]));
        if (c + 1 < nch) fetch(c + 1);
      }
    }
    if (bad) sh_bad = 1;
    // every load has landed before the CTA ends (bounded; normally it has)
    if (!kWidenFixed && !warp_wait(smem_addr(&fixed_full), 0)) ok = false;
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
  } else {
    // ======================= one fixed row per thread =======================
    bool ok = true;
    const int row = tid & (kTile - 1), set = warp / kSetWarps;
    const int key = k0 + row;                          // column sums
    const int pos = kStats && row < my_rows ? first_pos + row / G : -1;
    // a warp whose rows are all padding only keeps the barriers' phases
    const int row_lo = (warp % kSetWarps) * 32;
    const bool live = kStats ? row_lo < my_rows : k0 + row_lo < kend;
    float sl2 = a.scale_log2;
    const uint32_t scores = tm + ((uint32_t)row_lo << 16) + set * kTile;
    [[maybe_unused]] Codes<D, BS, kQ8 ? kKind : KV_DTYPE_INT8> codes;
    // K scales of the blocks of a chunk that this set widens
    auto put_scales = [&](int c) {
      const int j = row, from = k0 + c * kTile + j * BS;
      if (j < kTile / BS) {
        const int p = from < L ? bt[from / BS] : -1;
        blk_ks[c & (kScaleSlots - 1)][j] =
            p >= 0 && p < a.num_blocks ? a.k_scale[(int64_t)p * a.num_kv_heads + hk] : 0.0f;
      }
    };
    if constexpr (kWidenFixed) {
      if (set == 0) {
        bool all = codes.load(a, bt, hk, k0, L, 0);
        all &= codes.finish(a, bt, hk, k0, L, gbase);
        if (!all) sh_bad = 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&fixed_full));
      }
      if (key < kend) {
        const int p = bt[key / BS];
        if (p >= 0 && p < a.num_blocks) sl2 *= a.k_scale[(int64_t)p * a.num_kv_heads + hk];
      }
    }
    // chunk c of this set into its stage, once part 0 of its codes is held
    auto put_chunk = [&](int c) {
      put_scales(c);
      if (!codes.finish(a, bt, hk, k0 + c * kTile, L, gbase + (1 + set) * P::kImage)) sh_bad = 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&full[set]));
    };
    if constexpr (kWidenStream) {
      if (set < nch) {
        if (!codes.load(a, bt, hk, k0 + set * kTile, L, 0)) sh_bad = 1;
        put_chunk(set);
      }
    }
    for (int c = set; c < nch; c += kStages) {
      if constexpr (kWidenStream) {
        if (c + kStages < nch && !codes.load(a, bt, hk, k0 + (c + kStages) * kTile, L, 0)) sh_bad = 1;
      }
      const int ph = (c / kStages) & 1;
      if (!warp_wait(smem_addr(&s_full[set]), ph) ||
          (!kStats && !warp_wait(smem_addr(&stat_full[c % kRowSlots]), (c / kRowSlots) & 1)) ||
          (kWidenStream && !warp_wait(smem_addr(&full[set]), ph))) {  // (the other warps' scales)
        ok = false;
        break;
      }
      tc_fence_after();
      const int c0 = k0 + c * kTile;                   // row statistics: the chunk's first key
      const int i = (rt0 + c) * TT;                    // column sums: the tile's first token
      const int cols = kStats ? kTile : min(TT, n - i) * G;
      auto free_buf = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&buf_free[set]));
      };
      if (live) {
        const bool whole = kStats ? c0 + kTile - 1 <= first_pos
                                  : cols == kTile && L - n + i >= k0 + kTile - 1;
        const int from = max(0, key - (L - n + i)) * G;  // column sums: the rows [from, cols) see the key
#pragma unroll
        for (int at = 0; at < kTile; at += kRead) {
          if (at >= cols) break;
          uint32_t x[kRead];
          __syncwarp();                                // (the TMEM loads are the whole warp's)
          if constexpr (kRead == 64) tmem_read64(scores + at, x);
          else tmem_read32(scores + at, x);
          if (at + kRead >= cols) free_buf();          // the buffer's last scores are in registers
#pragma unroll
          for (int h = 0; h < kRead; h += 32) {
            if constexpr (kStats) {
              if constexpr (kWidenStream) {
                const float* ks = blk_ks[c & (kScaleSlots - 1)];
                scale_scores(x + h, ks[(at + h) / BS], ks[(at + h + 16) / BS]);
              }
              add_scores(st, x + h, sl2, whole, pos - c0 - at - h);
            } else {
              const float* m = row_m[c % kRowSlots] + at + h;
              acc += whole ? column_part<false>(x + h, sl2, m, 0, 32)
                           : column_part<true>(x + h, sl2, m, from - at - h, cols - at - h);
            }
          }
        }
      }
      if (!live) free_buf();
      if constexpr (kWidenStream) {
        // the scores of chunk c are complete, so its stage is free
        if (c + kStages < nch) put_chunk(c + kStages);
      }
    }
    if (!ok && lane == 0) sh_fail = 1;
    if (set == 1) {
      half_part[row] = kStats ? st.l : acc;
      half_ref[row] = st.ref;
    }
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
      const float r1 = half_ref[tid], M = fmaxf(st.ref, r1);
      float l = 0.0f;
      if (st.ref > -INFINITY || st.l != st.l) l = st.l * ex2(st.ref - M);
      if (r1 > -INFINITY || half_part[tid] != half_part[tid]) l = fmaf(half_part[tid], ex2(r1 - M), l);
      const bool lost = failed || sh_bad;
      float* o = stats_at(i0) + ((int64_t)tid * a.splits + split) * 2;
      // one split: m' at once (-inf: no statistics, the weights stay as they
      // are; a row whose every score is -inf has NaN weights)
      o[0] = a.splits > 1 ? M : (lost ? -INFINITY : row_log_sum(M, l));
      o[1] = lost ? -1.0f : l;
    }
  } else if (!failed && !sh_bad && tid < kend - k0) {
    acc += half_part[tid];
    float* w = a.weights + ((int64_t)b * a.num_kv_heads + hk) * a.stride + k0 + tid;
    *w = a.accumulate && k0 + tid < L - n ? *w + acc : acc;
  }
}

// Row statistics of several key splits: m' of a row into its first entry.
__global__ void __launch_bounds__(256) join_stats_kernel(float* stats, int64_t rows, int splits) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= rows) return;
  float* ml = stats + r * splits * 2;
  float M = -INFINITY, l = 0.0f;
  bool lost = false;
  for (int i = 0; i < splits; ++i) M = fmaxf(M, ml[2 * i]);
  for (int i = 0; i < splits; ++i) {
    const float m = ml[2 * i], x = ml[2 * i + 1];
    lost |= x < 0.0f;
    if (m > -INFINITY || x != x) l = fmaf(x, ex2(m - M), l);
  }
  ml[0] = lost ? -INFINITY : row_log_sum(M, l);
}

template <int D, int BS, int kKind, bool kStats>
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
      st = cuda_check(cudaFuncSetAttribute(prompt_tc_kernel<D, BS, kKind, kStats>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, PGeo<D>::kSmemBytes),
                      "cudaFuncSetAttribute(prompt_tc_kernel)");
      if (st != KV_OK) return st;
      attr_set[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.num_kv_heads, (unsigned)a.batch, z);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = PGeo<D>::kSmemBytes;
  cfg.stream = s;
  // the column sums start in the tail of the kernel before them
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kStats ? 0 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, prompt_tc_kernel<D, BS, kKind, kStats>, km, qm, a),
                    "prompt_tc_kernel launch");
}

template <int D, int BS, int kKind>
kv_status launch_tc_kind(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, int tiles, cudaStream_t s) {
  kv_status st = launch_tc_t<D, BS, kKind, true>(a, km, qm, (unsigned)(tiles * a.splits), s);
  if (st != KV_OK) return st;
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.num_tokens * a.num_q_heads;
    if ((rows + 255) / 256 > 0x7fffffffLL)
      return fail(KV_ERR_INVALID_ARG, "pagedkv_attention_weights: too many query tokens");
    join_stats_kernel<<<(unsigned)((rows + 255) / 256), 256, 0, s>>>(a.stats, rows, a.splits);
    if ((st = cuda_check(cudaGetLastError(), "join_stats_kernel launch")) != KV_OK) return st;
  }
  return launch_tc_t<D, BS, kKind, false>(a, km, qm, (unsigned)((a.max_seq_len - 1) / kTile + 1), s);
}

template <int D, int BS>
kv_status launch_tc(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, kv_dtype dtype, int tiles,
                    cudaStream_t s) {
  if (dtype == KV_DTYPE_INT8) return launch_tc_kind<D, BS, KV_DTYPE_INT8>(a, km, qm, tiles, s);
  if (dtype == KV_DTYPE_FP8_E4M3) return launch_tc_kind<D, BS, KV_DTYPE_FP8_E4M3>(a, km, qm, tiles, s);
  return launch_tc_kind<D, BS, KV_DTYPE_BF16>(a, km, qm, tiles, s);
}

}  // namespace

kv_status launch_prompt_tc(const PromptArgs& a, int head_dim, int block_size, kv_dtype dtype, int tiles,
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
    return block_size == 32 ? launch_tc<128, 32>(a, km, qm, dtype, tiles, s)
                            : launch_tc<128, 16>(a, km, qm, dtype, tiles, s);
  return block_size == 32 ? launch_tc<64, 32>(a, km, qm, dtype, tiles, s)
                            : launch_tc<64, 16>(a, km, qm, dtype, tiles, s);
}

}  // namespace pagedkv
