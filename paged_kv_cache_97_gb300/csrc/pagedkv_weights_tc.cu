// pagedkv_weights_tc.cu -- the attention weights of long multi-token queries
// (prompts, prefill chunks) on the fifth-generation tensor cores: both passes
// of pagedkv_attention_weights over Q K^T (pagedkv_weights.cu) with the scores
// in TMEM.
//
// The two passes are one kernel with the operands exchanged.  A unit of work
// keeps one tile of 128 rows of one operand in shared memory and streams tiles
// of 128 rows of the other (chunks) through two stages:
//   row statistics   fixed: 128 query rows,  streamed: the keys they see;
//                    a thread owns a query row and keeps its (m, l)
//   column sums      fixed: 128 keys,        streamed: the row tiles that see
//                    them; a thread owns a key and adds 2^(s - m') over the
//                    rows, m' = m + log2 l of each row from shared memory
// so that neither a maximum nor a sum crosses threads but for the joining of
// the sets.  Warps 0-3 hold one fixed row per thread (a TMEM lane) and take the
// even chunks, warps 4-7 the odd ones (so a set, a stage and a TMEM buffer go
// together), warp 8 issues the MMAs (S[128 x 128] = fixed . streamed^T into one
// of two TMEM buffers), warp 9 the TMA loads and, in the column sums, each row
// tile's m'.  A query tile is whole tokens, tile_tokens = 128 / G of them times
// the G heads, as one TMA box; rows past the sequence's queries are masked.
// Two CTAs per SM (256 TMEM columns and about 110 KB of shared memory each).
//
// A CTA goes on with units of the grid that have not been launched (cluster
// launch control): it starts up once, its next unit's loads run beside the last
// chunks of this one, and the balance stays the hardware's.  A CTA per unit
// instead: 4 prompts of 1..4K tokens 251 us against 231, 64 sequences x 32
// queries, whose column sums have one chunk a unit, 283 against 187; units
// dealt out in advance: 273..294 and 165; claimed at a unit's start and not
// near its end: 290.
//
// No unit of the SM is busy more than about 55 % of a long prompt (one of 16K
// tokens, 32/8 heads, bf16: 1678 us, 900 cycles per 128 x 128 tile): its
// 16384 exponentials take 512 cycles at 32 per clock, its MMAs 512, its
// instructions about as many issue slots.  The rest is the chain of a chunk: its
// load into one of two stages, its MMA and the hand-over, which two CTAs per SM
// hide in part (with the row warps idle the row statistics of 8K tokens take 198
// of 227 us).  So each score costs one
// packed half of a multiply-add and of an add (f32x2), and no maximum: a row's
// reference is its first scores' and moves only when a sum grows past 2^60; the
// scores are read 64 columns at a time and their buffer is free before they are
// used.  Measured and not taken: the fixed operand in TMEM, streamed tiles
// shared by two CTAs through TMA multicast (neither changed a long prompt, 286
// to 288 us for the short ones), one CTA per SM with four stages, four sets and
// two MMA and load warps (270), an eighth to a half of the exponentials as
// polynomials on the FMA pipe (3 to 42 % slower).
//
// 8-bit pools: the row warps load the codes themselves, widen them to bf16
// (exact: 8 significant bits hold every int8 and E4M3 code) and write them into
// the swizzled image, the streamed keys two chunks ahead, right after the
// scores of the chunk that used the stage before; a block's K scale multiplies
// its scores (one prompt of 8K tokens: E4M3 787 us, int8 827, bf16 477).
//
// Before the first pass every row is marked as without statistics, so that what
// a unit leaves out when a wait gives up is left out of the weights too (2 us:
// 4 prompts 230 -> 232).
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
constexpr int kSets = 2;                               // sets of four row warps
static_assert(kSets == 2, "the sets' results are joined symmetrically");
constexpr int kStages = kSets;                         // = TMEM buffers; chunk g of a CTA: number g % 2 of each
constexpr int kRowWarps = 4 * kSets, kSetThreads = 128;
constexpr int kMmaWarp = kRowWarps, kLoadWarp = kRowWarps + 1;
constexpr int kThreads = (kRowWarps + 2) * 32;
constexpr int kNotes = 8;                              // chunks whose notes (rows' m', bad blocks) may be in use
constexpr int kClaimChunks = 3;                        // chunks left to load when the next unit is claimed
constexpr int kClaims = 4;                             // claims whose answers may be in use
constexpr int kUnits = 8;                              // units whose verdicts may be in use
constexpr int kParts = 4;                              // units whose sets' results may be in use
constexpr int kTmemCols = kStages * kTile;
constexpr float kMoveSum = 0x1p60f;                    // a sum of 32 that moves a row's reference

template <int D>
struct PGeo {
  static constexpr int kBands = D / 64;
  static constexpr int kImage = kTile * D * 2;         // bytes of 128 rows
  static constexpr int kUsed = (1 + kStages) * kImage + 1024;
  // at least 80 KB, so that no more than two CTAs (512 TMEM columns) share an SM
  static constexpr int kSmemBytes = kUsed > 80 * 1024 ? kUsed : 80 * 1024;
};

// One unit of a CTA's work: a fixed tile and the chunks streamed past it.
struct Unit {
  int hk, b, q0, n, L;
  int split;                 // row statistics: the key split
  int i0, tn;                // row statistics: first query token of the fixed tile, its tokens
  int k0, kend;              // keys: of the split, or of the fixed tile
  int first_pos;             // row statistics: position of token i0
  int rt0;                   // column sums: first row tile that sees a key
  int nch;                   // chunks
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

// Statistics of a row that has none (yet): the weights of its sequence stay as
// they are.
constexpr float kNoMax = -INFINITY, kNoSum = -1.0f;

// Marks every row as without statistics before the row statistics: a unit whose
// CTA gives up (a bounded wait) stores none, and what the workspace held from
// before, finite numbers of an earlier call as a rule, must not pass for its.
__global__ void __launch_bounds__(256) mark_stats_kernel(float2* stats, int64_t n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;
  if (i + 1 < n) *reinterpret_cast<float4*>(stats + i) = make_float4(kNoMax, kNoSum, kNoMax, kNoSum);
  else if (i < n) stats[i] = make_float2(kNoMax, kNoSum);
}

// m + log2 l of a row.
__device__ __forceinline__ float row_log_sum(float m, float l) {
  return m == -INFINITY ? __uint_as_float(0x7fc00000u) : m + log2f(l);
}

template <int D, int BS, int kKind, bool kStats>
__global__ void __launch_bounds__(kThreads, 2)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap q_map, const PromptArgs a, int tiles) {
  using P = PGeo<D>;
  constexpr bool kQ8 = kKind != KV_DTYPE_BF16;
  constexpr bool kWidenStream = kQ8 && kStats, kWidenFixed = kQ8 && !kStats;
  constexpr int kRead = kWidenStream ? 32 : 64;        // scores of a row in registers at a time
  constexpr int kScaleSlots = 2 * kSets;               // chunks whose scales may be in use
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t fixed_full, fixed_free, full[kStages], s_full[kStages], buf_free[kStages],
      noted[kNotes], checked[kUnits], claim_full[kClaims], claim_free[kClaims], part_full[kParts], part_free[kParts], drain_bar, near_end;
  __shared__ __align__(16) uint4 claim[kClaims];
  __shared__ uint32_t tmem_base;
  __shared__ int sh_fail;
  __shared__ __align__(16) float row_m[kStats ? 1 : kNotes][kTile];  // -m' of the row tiles' rows
  __shared__ int unit_bad[kUnits];                     // a block or a row of the unit is bad
  __shared__ float part_sum[kParts][kSets][kTile], part_ref[kStats ? kParts : 1][kSets][kTile];
  __shared__ int part_bad[kParts][kRowWarps];
  __shared__ float blk_ks[kWidenStream ? kScaleSlots : 1][kTile / BS];  // K scales of the chunks' blocks
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.num_q_heads / a.num_kv_heads, TT = a.tile_tokens;
  bool ok = true;

  // Unit u is (KV head, sequence, tile), tiles slowest, those with most chunks
  // first: the last row tiles of the row statistics, the first key tiles of the
  // column sums.  There is a CTA for each in the grid; one that runs takes over
  // CTAs that have not been launched yet (cluster launch control), so that it
  // starts up once and loads the next unit beside the last chunks of this one.
  const unsigned per_tile = (unsigned)(a.num_kv_heads * a.batch);
  // The CTA's unit number k (> 0), claimed by the loading warp; false: no more.
  auto claimed = [&](int k, unsigned& u) {
    uint32_t yes, x;
    asm volatile("{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
                 : "=r"(yes), "=r"(x) : "r"(smem_addr(&claim[(k - 1) % kClaims])) : "memory");
    u = x;
    return yes != 0;
  };
  auto next_unit = [&](int k, unsigned& u) {           // (a whole warp)
    if (!warp_wait(smem_addr(&claim_full[(k - 1) % kClaims]), ((k - 1) / kClaims) & 1)) {
      ok = false;
      return false;
    }
    const bool yes = claimed(k, u);
    __syncwarp();
    if (warp < kRowWarps && lane == 0) mbar_arrive(smem_addr(&claim_free[(k - 1) % kClaims]));
    return yes;
  };
  // False: nothing to stream past the tile (un.nch == 0).  A bad sequence is
  // flagged by the loading warp.
  auto locate = [&](unsigned u, Unit& un) {
    un.nch = un.tn = 0;
    if (u >= gridDim.x) return false;
    const int z = (int)(u / per_tile), r = (int)(u % per_tile);
    un.hk = r % a.num_kv_heads;
    un.b = r / a.num_kv_heads;
    if (!prompt_rows(a, un.b, BS, &un.q0, &un.n, &un.L)) {
      if (kStats && z == 0 && warp == kLoadWarp && lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
      return false;
    }
    const int tile = kStats ? (tiles - 1 - z) / a.splits : z;
    un.split = kStats ? (tiles - 1 - z) % a.splits : 0;
    un.k0 = kStats ? un.split * a.part_tokens : tile * kTile;
    if (kStats) {
      if ((int64_t)tile * TT >= un.n) return false;
      un.i0 = tile * TT;
      un.tn = min(TT, un.n - un.i0);
      un.first_pos = un.L - un.n + un.i0;
      un.kend = min(un.first_pos + un.tn, un.k0 + a.part_tokens);
      un.rt0 = 0;
      un.nch = max(0, (un.kend - un.k0 + kTile - 1) / kTile);
    } else {
      if (un.n == 0 || un.k0 >= un.L) return false;
      un.i0 = un.first_pos = 0;
      un.kend = min(un.L, un.k0 + kTile);
      un.rt0 = max(0, un.k0 - (un.L - un.n)) / TT;
      un.nch = (un.n - 1) / TT + 1 - un.rt0;
    }
    return un.nch > 0;
  };
  // statistics of row 0 of the tile that starts at token i of the unit's
  // sequence: [Hkv][T][G], so that a tile's rows lie together
  auto stats_at = [&](const Unit& un, int i) {
    return a.stats + ((int64_t)un.hk * a.num_tokens + un.q0 + i) * G * a.splits * 2;
  };

  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - smem_addr(smem_raw));
  auto stage_img = [&](int s) { return base + (uint32_t)((1 + s) * P::kImage); };
  if (tid == 0) {
    sh_fail = 0;
    mbar_init(smem_addr(&fixed_full), kWidenFixed ? kSetThreads / 32 : 1);
    mbar_init(smem_addr(&fixed_free), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&full[s]), kWidenStream ? kSetThreads / 32 : 1);
      mbar_init(smem_addr(&s_full[s]), 1);
      mbar_init(smem_addr(&buf_free[s]), kSetThreads / 32);
    }
    for (int s = 0; s < kNotes; ++s) mbar_init(smem_addr(&noted[s]), 1);
    for (int s = 0; s < kUnits; ++s) mbar_init(smem_addr(&checked[s]), 1);
    for (int s = 0; s < kClaims; ++s) {
      mbar_init(smem_addr(&claim_full[s]), 1);
      mbar_init(smem_addr(&claim_free[s]), kRowWarps + 1);
    }
    for (int s = 0; s < kParts; ++s) {
      mbar_init(smem_addr(&part_full[s]), kRowWarps);
      mbar_init(smem_addr(&part_free[s]), kSetThreads / 32);
    }
    mbar_init(smem_addr(&drain_bar), 1);
    mbar_init(smem_addr(&near_end), 1);
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

  // Every role walks the same units and counts the same chunks: g of them
  // before the unit, us units with chunks before it.
  Unit un = {};
  int g = 0, us = 0;
  unsigned u = blockIdx.x;
  if (warp == kLoadWarp) {
    // ======================= loads (TMA) and notes ==========================
    const int32_t* bt = nullptr;
    // Keys [from, from + 128) (up to L) into an image, one block per lane: its
    // table entry, read ahead of the wait for the image, then the load.
    auto entry = [&](int from) {
      return lane < min(kTile / BS, (un.L - from + BS - 1) / BS) ? bt[from / BS + lane] : 0;
    };
    // False when a key's block is outside the pool.
    auto load_k = [&](uint32_t img, uint64_t* bar, int from, int p) {
      const int nb = min(kTile / BS, (un.L - from + BS - 1) / BS);
      const bool in = p >= 0 && p < a.num_blocks;
      if (lane == 0) mbar_expect_tx(smem_addr(bar), (uint32_t)(nb * BS * D * 2));
      __syncwarp();
      if (lane < nb) {
#pragma unroll
        for (int x = 0; x < P::kBands; ++x)
          tma_load_4d(img + x * (kTile * 128) + lane * (BS * 128), &k_map, smem_addr(bar), x * 64, un.hk, 0,
                      in ? p : 0);
      }
      return __all_sync(0xffffffffu, in);
    };
    // The row tile that starts at query token i (whole boxes; rows past the
    // tensor are zeros).
    auto load_q = [&](uint32_t img, uint64_t* bar, int i) {
      if (lane == 0) {
        mbar_expect_tx(smem_addr(bar), (uint32_t)(TT * G * D * 2));
#pragma unroll
        for (int x = 0; x < P::kBands; ++x)
          tma_load_3d(img + x * (kTile * 128), &q_map, smem_addr(bar), x * 64, un.hk * G, un.q0 + i);
      }
      __syncwarp();
    };
    bool first = true;
    int fixed_issued = 0, issued = 0, last_claim = 0;
    bool have = true;
    for (int nth = 0; have; have = ok && next_unit(++nth, u)) {
      // claim unit nth + 1
      auto claim_next = [&] {
        const int slot = nth % kClaims, turn = nth / kClaims;
        if (turn > 0 && !warp_wait(smem_addr(&claim_free[slot]), (turn - 1) & 1)) return false;
        if (lane == 0) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_expect_tx(smem_addr(&claim_full[slot]), 16);
          asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                       ::"r"(smem_addr(&claim[slot])), "r"(smem_addr(&claim_full[slot])) : "memory");
        }
        __syncwarp();
        last_claim = nth + 1;
        return true;
      };
      if (!locate(u, un)) {
        ok = claim_next();
        continue;
      }
      // Late, when few chunks remain: a unit claimed early would be out of reach
      // of CTAs that finish sooner.
      const int claim_at = max(0, un.nch - kClaimChunks);
      bt = a.block_tables + (int64_t)un.b * a.max_blocks;
      bool good = true;
      int next = kStats && !kWidenStream ? entry(un.k0) : 0;
      const int p = kStats || kWidenFixed ? 0 : entry(un.k0);
      // the fixed tile, once the last unit's MMAs are done (behind the unit's
      // first chunk, whose stage is free before)
      auto load_fixed = [&] {
        if (kWidenFixed) return true;
        if (us >= 1 && !warp_wait(smem_addr(&fixed_free), (us - 1) & 1)) return false;
        if (kStats) load_q(base, &fixed_full, un.i0);
        else good = load_k(base, &fixed_full, un.k0, p);
        fixed_issued = us + 1;
        return true;
      };
      if (kWidenStream && (!load_fixed() || !warp_wait(smem_addr(&near_end), us & 1) || !claim_next())) {
        ok = false;
        break;
      }
      // column sums: m' of the rows of chunk c's row tile
      [[maybe_unused]] float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      auto fetch = [&](int c) {
        const int i = (un.rt0 + c) * TT, rows = min(TT, un.n - i) * G;
        const float* st_row = stats_at(un, i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k * 32 + lane;
          m[k] = r < rows ? st_row[(int64_t)r * a.splits * 2] : 0.0f;
        }
      };
      for (int c = 0; c < (kWidenStream ? 0 : un.nch); ++c) {
        const int gc = g + c, s = gc % kStages, note = gc % kNotes;
        if (gc >= kStages && !warp_wait(smem_addr(&s_full[s]), ((gc / kStages) - 1) & 1)) {
          ok = false;
          break;
        }
        if (kStats) {
          good &= load_k(stage_img(s), &full[s], un.k0 + c * kTile, next);
          next = entry(un.k0 + (c + 1) * kTile);
        } else {
          load_q(stage_img(s), &full[s], (un.rt0 + c) * TT);
        }
        issued = gc + 1;
        if ((c == 0 && !load_fixed()) || (c == claim_at && !claim_next())) {
          ok = false;
          break;
        }
        // (the MMA of chunk gc - 2 is done, so chunk gc - 4's scores were read,
        // and before them chunk gc - 6 was finished: its note's slot and the
        // slot's barrier phase are free)
        if constexpr (!kStats) {
          if (first) {
            // The kernel may start beside the last CTAs of the one before it (a
            // programmatic dependent); from here on that one has ended.
            asm volatile("griddepcontrol.wait;" ::: "memory");
            first = false;
          }
          if (c == 0) fetch(0);
          bool lost = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            lost |= m[k] == -INFINITY;                 // a row without statistics
            row_m[note][k * 32 + lane] = -m[k];
          }
          good &= !__any_sync(0xffffffffu, lost);
        }
        if constexpr (!kStats) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&noted[note]));
          if (c + 1 < un.nch) fetch(c + 1);
        }
      }
      // (the chunk 6 before the last one is finished, so a unit that ended there
      // was joined: eight slots do)
      if (lane == 0) {
        unit_bad[us % kUnits] = !good;
        mbar_arrive(smem_addr(&checked[us % kUnits]));
      }
      __syncwarp();
      g += un.nch;
      ++us;
    }
    // (row statistics: the marks are there before the column sums start, whether
    // this CTA stored anything behind them or not)
    if (kStats || first) asm volatile("griddepcontrol.wait;" ::: "memory");
    // every load and claim has landed before the CTA ends (bounded; normally it has)
    if (last_claim > 0 && !warp_wait(smem_addr(&claim_full[(last_claim - 1) % kClaims]), ((last_claim - 1) / kClaims) & 1)) ok = false;
    if (fixed_issued > 0 && !warp_wait(smem_addr(&fixed_full), (fixed_issued - 1) & 1)) ok = false;
    for (int s = 0; s < kStages && s < issued; ++s) {
      const int last = s + kStages * ((issued - 1 - s) / kStages);
      if (!warp_wait(smem_addr(&full[s]), (last / kStages) & 1)) ok = false;
    }
    if (!ok && lane == 0) sh_fail = 1;
  } else if (warp == kMmaWarp) {
    // ======================= tensor-core issue (one lane) ===================
    if (lane == 0) {
      const uint32_t idesc = mma_idesc<false>(kTile, kTile, 0);
      bool have = true;
      for (int nth = 0; have;) {
        if (locate(u, un)) {
          ok = mbar_wait(smem_addr(&fixed_full), us & 1);
          for (int c = 0; c < un.nch && ok; ++c) {
            const int gc = g + c, s = gc % kStages, ph = (gc / kStages) & 1;
            ok = mbar_wait(smem_addr(&full[s]), ph) &&
                 (gc < kStages || mbar_wait(smem_addr(&buf_free[s]), ph ^ 1));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = (ks / 4) * (kTile * 128) + (ks % 4) * 32;
              mma_ss(tm + s * kTile, smem_desc(base + off, 16, 1024), smem_desc(stage_img(s) + off, 16, 1024),
                     idesc, ks > 0);
            }
            mma_commit(smem_addr(&s_full[s]));
          }
          if (ok) mma_commit(smem_addr(&fixed_free));
          g += un.nch;
          ++us;
        }
        ++nth;
        ok = ok && mbar_wait(smem_addr(&claim_full[(nth - 1) % kClaims]), ((nth - 1) / kClaims) & 1);
        have = ok && claimed(nth, u);
        if (ok) mbar_arrive(smem_addr(&claim_free[(nth - 1) % kClaims]));
      }
      if (!ok) sh_fail = 1;
      // the tensor core is done with shared memory and TMEM before they go
      mma_commit(smem_addr(&drain_bar));
      mbar_wait(smem_addr(&drain_bar), 0);
    }
    __syncwarp();
  } else {
    // ======================= one fixed row per thread =======================
    const int row = tid % kSetThreads, set = warp / 4, row_lo = (warp % 4) * 32;
    const uint32_t scores = tm + ((uint32_t)row_lo << 16) + set * kTile;
    [[maybe_unused]] Codes<D, BS, kQ8 ? kKind : KV_DTYPE_INT8> codes;
    bool have = true;
    for (int nth = 0; have; have = ok && next_unit(++nth, u)) {
      const bool any = locate(u, un);
      const int my_rows = un.tn * G;                   // row statistics: rows of the tile
      if (!any) {
        if (kStats && set == 0 && row < my_rows) {     // no key of this split
          asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows are marked
          float* o = stats_at(un, un.i0) + ((int64_t)row * a.splits + un.split) * 2;
          o[0] = -INFINITY;
          o[1] = 0.0f;
        }
        continue;
      }
      const int32_t* bt = a.block_tables + (int64_t)un.b * a.max_blocks;
      RowStats st = {-INFINITY, 0.0f};
      float acc = 0.0f;
      bool bad = false;
      const int key = un.k0 + row;                     // column sums
      const int pos = kStats && row < my_rows ? un.first_pos + row / G : -1;
      // a warp whose rows are all padding only keeps the barriers' phases
      const bool live = kStats ? row_lo < my_rows : un.k0 + row_lo < un.kend;
      float sl2 = a.scale_log2;
      if constexpr (kWidenFixed) {
        if (set == us % kSets) {
          bad = !codes.load(a, bt, un.hk, un.k0, un.L, 0);
          if (us >= 1 && !warp_wait(smem_addr(&fixed_free), (us - 1) & 1)) {
            ok = false;
            break;
          }
          bad |= !codes.finish(a, bt, un.hk, un.k0, un.L, gbase);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&fixed_full));
        }
        if (key < un.kend) {
          const int p = bt[key / BS];
          if (p >= 0 && p < a.num_blocks) sl2 *= a.k_scale[(int64_t)p * a.num_kv_heads + un.hk];
        }
      }
      // chunk c of this set into its stage (the set has waited for the MMA of
      // the chunk before), once part 0 of its codes is held, and the K scales
      // of its blocks
      auto put_chunk = [&](int c) {
        const int from = un.k0 + c * kTile + row * BS;
        if (row < kTile / BS) {
          const int p = from < un.L ? bt[from / BS] : -1;
          blk_ks[(g + c) % kScaleSlots][row] =
              p >= 0 && p < a.num_blocks ? a.k_scale[(int64_t)p * a.num_kv_heads + un.hk] : 0.0f;
        }
        bad |= !codes.finish(a, bt, un.hk, un.k0 + c * kTile, un.L, gbase + (1 + set) * P::kImage);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&full[set]));
      };
      const int c_first = (set - g) & (kSets - 1);     // the set's first chunk of the unit
      if constexpr (kWidenStream) {
        if (c_first < un.nch) {
          bad |= !codes.load(a, bt, un.hk, un.k0 + c_first * kTile, un.L, 0);
          put_chunk(c_first);
        }
      }
      for (int c = c_first; c < un.nch; c += kSets) {
        const bool more = kWidenStream && c + kSets < un.nch;
        if constexpr (kWidenStream) {
          if (more) bad |= !codes.load(a, bt, un.hk, un.k0 + (c + kSets) * kTile, un.L, 0);
        }
        const int gc = g + c, ph = (gc / kStages) & 1, note = gc % kNotes;
        if (!warp_wait(smem_addr(&s_full[set]), ph) ||
            (kWidenStream && !warp_wait(smem_addr(&full[set]), ph)) ||  // (the other warps' scales)
            (!kStats && !warp_wait(smem_addr(&noted[note]), (gc / kNotes) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int c0 = un.k0 + c * kTile;              // row statistics: the chunk's first key
        const int i = (un.rt0 + c) * TT;               // column sums: the tile's first token
        const int cols = kStats ? kTile : min(TT, un.n - i) * G;
        auto free_buf = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&buf_free[set]));
        };
        if (live) {
          const bool whole = kStats ? c0 + kTile - 1 <= un.first_pos
                                    : cols == kTile && un.L - un.n + i >= un.k0 + kTile - 1;
          const int from = max(0, key - (un.L - un.n + i)) * G;  // column sums: rows [from, cols) see the key
#pragma unroll
          for (int at = 0; at < kTile; at += kRead) {
            if (at >= cols) break;
            uint32_t x[kRead];
            __syncwarp();                              // (the TMEM loads are the whole warp's)
            if constexpr (kRead == 64) tmem_read64(scores + at, x);
            else tmem_read32(scores + at, x);
            if (at + kRead >= cols) free_buf();        // the buffer's last scores are in registers
#pragma unroll
            for (int h = 0; h < kRead; h += 32) {
              if constexpr (kStats) {
                if constexpr (kWidenStream) {
                  const float* ks = blk_ks[gc % kScaleSlots];
                  scale_scores(x + h, ks[(at + h) / BS], ks[(at + h + 16) / BS]);
                }
                add_scores(st, x + h, sl2, whole, pos - c0 - at - h);
              } else {
                const float* m = row_m[note] + at + h;
                acc += whole ? column_part<false>(x + h, sl2, m, 0, 32)
                             : column_part<true>(x + h, sl2, m, from - at - h, cols - at - h);
              }
            }
          }
        } else {
          free_buf();
        }
        if constexpr (kWidenStream) {
          if (more) put_chunk(c + kSets);
          // (the loading warp claims the next unit)
          if (c == max(0, un.nch - kClaimChunks) && warp % 4 == 0 && lane == 0) mbar_arrive(smem_addr(&near_end));
        }
      }
      if (!ok) break;
      // The sets' results of the unit; the set of its last chunk joins them.
      const int slot = us % kParts, turn = us / kParts;
      if (turn > 0 && !warp_wait(smem_addr(&part_free[slot]), (turn - 1) & 1)) {
        ok = false;
        break;
      }
      part_sum[slot][set][row] = kStats ? st.l : acc;
      if constexpr (kStats) part_ref[slot][set][row] = st.ref;
      const bool warp_bad = __any_sync(0xffffffffu, bad);
      if (lane == 0) part_bad[slot][warp] = warp_bad;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&part_full[slot]));
      if (set == (g + un.nch - 1) % kSets) {
        if (!warp_wait(smem_addr(&part_full[slot]), turn & 1) ||
            !warp_wait(smem_addr(&checked[us % kUnits]), (us / kUnits) & 1)) {
          ok = false;
          break;
        }
        const bool lost = unit_bad[us % kUnits] != 0 ||
                          __any_sync(0xffffffffu, lane < kRowWarps && part_bad[slot][lane % kRowWarps] != 0);
        if constexpr (kStats) {
          if (lost && row == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
          if (row < my_rows) {
            asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows are marked
            // (which set had the even chunks depends on the CTA's earlier units:
            // the join is the same with the two exchanged)
            const float r0 = part_ref[slot][0][row], r1 = part_ref[slot][1][row];
            const float p0 = part_sum[slot][0][row], p1 = part_sum[slot][1][row];
            const float M = fmaxf(r0, r1);
            const float l = __fadd_rn(r0 > -INFINITY || p0 != p0 ? __fmul_rn(p0, ex2(r0 - M)) : 0.0f,
                                      r1 > -INFINITY || p1 != p1 ? __fmul_rn(p1, ex2(r1 - M)) : 0.0f);
            float* o = stats_at(un, un.i0) + ((int64_t)row * a.splits + un.split) * 2;
            // one split: m' at once (-inf: no statistics, the weights stay as
            // they are; a row whose every score is -inf has NaN weights)
            o[0] = a.splits > 1 ? M : (lost ? kNoMax : row_log_sum(M, l));
            o[1] = lost ? kNoSum : l;
          }
        } else if (!lost && key < un.kend) {
          const float sum = part_sum[slot][0][row] + part_sum[slot][1][row];
          float* w = a.weights + ((int64_t)un.b * a.num_kv_heads + un.hk) * a.stride + key;
          *w = a.accumulate && key < un.L - un.n ? *w + sum : sum;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&part_free[slot]));
      }
      g += un.nch;
      ++us;
    }
    if (!ok && lane == 0) sh_fail = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmemCols) : "memory");
  if (tid == 0 && sh_fail) atomicOr(a.flags, PAGEDKV_FLAG_WAIT_TIMEOUT);
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
  ml[0] = lost ? kNoMax : row_log_sum(M, l);
}

template <int D, int BS, int kKind, bool kStats>
kv_status launch_tc_t(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, int tiles,
                      cudaStream_t s) {
  static std::mutex mu;
  static bool attr_set[64] = {};
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  const int dev = di.device;
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
  const int64_t units = (int64_t)a.num_kv_heads * a.batch * tiles;
  if (units > 0x7fff0000LL) return fail(KV_ERR_INVALID_ARG, "pagedkv_attention_weights: too many row or key tiles");
  cfg.gridDim = dim3((unsigned)units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = PGeo<D>::kSmemBytes;
  cfg.stream = s;
  // both start beside the end of the kernel before them
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, prompt_tc_kernel<D, BS, kKind, kStats>, km, qm, a, tiles),
                    "prompt_tc_kernel launch");
}

template <int D, int BS, int kKind>
kv_status launch_tc_kind(const PromptArgs& a, const CUtensorMap& km, const CUtensorMap& qm, int tiles, cudaStream_t s) {
  const int64_t rows = (int64_t)a.num_tokens * a.num_q_heads;
  const int64_t marks = (rows * a.splits + 511) / 512;
  if ((rows + 255) / 256 > 0x7fffffffLL || marks > 0x7fffffffLL)
    return fail(KV_ERR_INVALID_ARG, "pagedkv_attention_weights: too many query tokens");
  mark_stats_kernel<<<(unsigned)marks, 256, 0, s>>>(reinterpret_cast<float2*>(a.stats), rows * a.splits);
  kv_status st = cuda_check(cudaGetLastError(), "mark_stats_kernel launch");
  if (st == KV_OK) st = launch_tc_t<D, BS, kKind, true>(a, km, qm, tiles * a.splits, s);
  if (st != KV_OK) return st;
  if (a.splits > 1) {
    join_stats_kernel<<<(unsigned)((rows + 255) / 256), 256, 0, s>>>(a.stats, rows, a.splits);
    if ((st = cuda_check(cudaGetLastError(), "join_stats_kernel launch")) != KV_OK) return st;
  }
  return launch_tc_t<D, BS, kKind, false>(a, km, qm, (a.max_seq_len - 1) / kTile + 1, s);
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
