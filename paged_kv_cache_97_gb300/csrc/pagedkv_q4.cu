// pagedkv_q4.cu -- attention over the 4-bit pool, for one query token per
// sequence or several causal ones.
//
//   out[j, h] = softmax_t(scale * q[j, h] . K_t) . V_t,
//   K_t[e] = kmin + kscale * c, V_t[e] = vmin + vscale * c  per 64 values.
//
// The codes go to the tensor cores as they are.  c masked out of a word,
// (w & 0x000F000F) or (w & 0x00F000F0), is an fp16 pair c * 2^-24 or c * 2^-20
// (subnormals, exact), so a word of eight codes is four registers after five
// instructions; scale and min enter outside of the product:
//   q . K_t = sum over the row's groups of kscale * (q . c) + kmin * sum(q),
//   sum_t p_t V_t = (sum_t (p_t vscale_t) c_t) + (sum_t p_t vmin_t).
// q is fp16, scaled by a power of two (and by 1/16 where its code is a high
// nibble); kscale and kmin multiply in fp32; p * vscale is rounded once, to
// fp16; p * vmin is summed in fp32.  A column's reference is the largest of
// score + exponent of max(vscale, |vmin| / 16) so far, less five, not of the
// score alone: p * vscale then has fp16's whole range below 2^11 whatever the
// scales are, and p * vmin stays below 2^15.  It moves only when p times that maximum
// passes 2^11 (or a weight 2^32).
//
// Tile products (mma.sync m16n8k16, fp32 sums) with tokens, then dims, on M and
// the columns (query token x grouped head) on N: the unpacked codes are used for
// all kNT * 8 columns of the CTA, eight for one query token per sequence, up to
// 32 for several.  S's layout becomes P's operand by one 8x8 transposition
// (movmatrix) per 8 tokens and group.
//
// A warp runs on its own: it copies the records of every fourth 32 tokens of
// the CTA's range into its own ring of stages (one bulk copy per block) and works on them
// in turn; the four warps meet where a sequence ends.  The CTAs of a KV head cut
// the whole batch's blocks into equal ranges (each finds its own from the
// lengths), so the last wave is as full as the first whatever the lengths are; a
// sequence cut by a range leaves partials, at most two per CTA, which the merge
// kernel joins.
//
// Measured (GB300, 32 / 8 heads of 128, one query token): 8 sequences of up to
// 131072 tokens 142 us, 4.9 TB/s of the pool (floor 104 at 6.8); 128 of up to
// 8192, 64 query heads, 134 us (98); 64 of up to 4096 48 us (25).  With a pool that
// L2 holds, the first still takes 138 us, and memory alone 115: what bounds it is the
// arithmetic of the codes (ALU pipe 55 % busy, legacy tensor pipe 23 %, issue
// slots 53 %), with the memory close behind.  Three CTAs on an SM for eight
// columns: two took 151 us for 137 with the pool in L2, four (and fewer registers) 146.  Five query tokens (20
// columns, two CTAs on an SM): 64 of up to 4096 90 us, eight warps that wait on
// their own chains (issue 43 %, each warp issues every fourth cycle).
// Not better: q as two e4m3 numbers in an 8-bit product (175 us for 143: the fp8
// form of mma.sync takes five times the f16 form's cycles), codes shifted by
// high multiplies instead of shifts (150).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>
#include <type_traits>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_q4.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kWarps = 4;
constexpr int kThreads4 = kWarps * 32;
// Ranges are not cut below this many tokens: a warp then has two blocks of 16,
// and the partials of a range cost less than its blocks.
constexpr int kMinRangeTokens = 128;
// Lengths up to this many tokens take one CTA per sequence, with no merge behind it.
constexpr int kWholeTokens = 512;
constexpr int kAloneParts = 8;        // partials that one warp joins by itself
constexpr float kNoRef = -1e30f;      // the reference of a column without a key

struct Q4Args {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const unsigned char* kv;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start;  // [batch + 1], or null: one query token per sequence
  float* ws_acc;               // [Hkv, ctas, 2, columns, D]
  float* ws_ml;                // [Hkv, ctas, 2, columns, 2]: (reference, sum)
  int4* ws_meta;               // [Hkv, ctas]: {CTAs that follow, first token row, tokens, -}
  unsigned int* flags;
  const int* slot_of;          // [batch]: >= 0 where the long queries' kernel has the sequence; or null
  int max_blocks, batch, num_tokens, max_query_len, num_q_heads, num_kv_heads;
  int num_blocks, max_seq_len;
  int group;                   // query heads per KV head
  int tile_tokens;             // query tokens per column tile
  int ctas;                    // ranges per KV head (or, whole: column tiles at most)
  int whole;                   // one CTA per column tile of a sequence
  float scale_log2;
};

// What the kernel needs of a sequence; nct == 0: nothing to do (or not valid).
struct Seq {
  int q0, n, L, nblk, nct;
  bool bad;
};

template <int BS, bool kMulti>
__device__ __forceinline__ Seq seq_of(const Q4Args& a, int b) {
  Seq s;
  s.L = __ldg(a.seq_lens + b);
  s.q0 = b;
  s.n = 1;
  bool rows = true;
  if constexpr (kMulti) {
    s.q0 = __ldg(a.query_start + b);
    const int q1 = __ldg(a.query_start + b + 1);
    rows = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.num_tokens;
    s.n = rows ? q1 - s.q0 : 0;                    // rows that may be written
  }
  const bool len = s.L > 0 && s.L <= a.max_seq_len && (s.L - 1) / BS < a.max_blocks &&
                   s.n <= s.L && s.n <= a.max_query_len;
  s.bad = !rows || (!len && (!kMulti || s.n > 0));
  bool use = !s.bad && s.n > 0;
  if constexpr (kMulti)
    if (a.slot_of != nullptr && use) use = __ldg(a.slot_of + b) < 0;
  s.nblk = use ? (s.L + BS - 1) / BS : 0;
  s.nct = use ? (kMulti ? (s.n + a.tile_tokens - 1) / a.tile_tokens : 1) : 0;
  return s;
}

// A walk over the pieces of [0, len) block positions of one CTA: unit (b, ct)
// (a sequence's column tile) begins at position `us` (negative where the CTA's
// range begins inside it).
template <int BS, bool kMulti>
struct Walk {
  Seq s;
  int b, ct, us, len;
  int j0, j1;                                      // blocks of this piece: [j0, j1)

  __device__ __forceinline__ int visible(const Q4Args& a) const {
    if constexpr (!kMulti) return s.nblk;
    const int last = min(s.n, (ct + 1) * a.tile_tokens);
    return (s.L - s.n + last + BS - 1) / BS;       // blocks its last query sees
  }
  __device__ __forceinline__ bool done() const { return us >= len; }
  __device__ __forceinline__ void piece(const Q4Args& a) {
    j0 = max(0, -us);
    j1 = min(visible(a), len - us);
  }
  __device__ __forceinline__ void start(const Q4Args& a, int b_, int ct_, int us_, int len_) {
    b = b_;
    ct = ct_;
    us = us_;
    len = len_;
    s = seq_of<BS, kMulti>(a, b);
    piece(a);
  }
  __device__ __forceinline__ void next(const Q4Args& a) {
    us += s.nblk;
    if (us >= len) return;
    if (++ct >= s.nct) {
      ct = 0;
      // (us < len: a further valid sequence exists)
      do {
        s = seq_of<BS, kMulti>(a, ++b);
      } while (s.nct == 0 && b + 1 < a.batch);
    }
    piece(a);
  }
};

// 8x8 16-bit matrix over the warp (row = lane / 4, columns 2 (lane % 4), +1), transposed.
__device__ __forceinline__ uint32_t transposed8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x * 2^d: a reference may move by more octaves than one factor holds, where V's
// scales lie far apart, and a sum of weights that is then small still counts.
__device__ __forceinline__ float times_ex2(float x, float d) {
  const float h = ex2(0.5f * d);
  return x * h * h;
}

// mma16816<true> on an accumulator of zeros.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// kGroups consecutive words.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t addr) {
  if constexpr (N == 4) {
    const uint4 v = lds128(addr);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = lds64(addr);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = lds32(addr);
  }
}

// The exponent of a row's largest V scale or |min| / 16, from its (scale, min) pairs.
template <int N>
__device__ __forceinline__ float value_exponent(const uint32_t (&pairs)[N]) {
  uint32_t x = pairs[0] & 0x7fff7fffu;
  if constexpr (N == 2) x = __vmaxu2(x, pairs[1] & 0x7fff7fffu);
  const int s = (int)(x >> 7 & 0xffu), m = (int)(x >> 23);
  return (float)(max(max(s, m - 4), 27) - 127);
}

__device__ __forceinline__ float pair_scale(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float pair_min(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;   // codes * 2^-24, * 2^-20

// CTAs of q4_kernel on an SM with `nt` column tiles.
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }

// A stage holds a step's blocks: 32 tokens, two MMA tiles.
template <int D, int BS, int NT>
struct Cfg4 {
  using G = Geo4<D, BS>;
  static constexpr int kCols = 8 * NT;
  static constexpr int kCtasPerSm = ctas_per_sm(NT);
  static constexpr int kBlocks = 32 / BS;                 // blocks of a step
  static constexpr int kStage = kBlocks * G::kRecord;
  static constexpr int kTiles = NT <= 2 ? 2 : 1;          // tiles worked on together
  static constexpr bool kQShared = NT > 2;               // q's fragments stay in shared memory
  static constexpr int kQBytes = (D / 16) * NT * 32 * 8;
  // what the warps hand over at the end of a sequence: O, then (reference, sum)
  static constexpr int kRow = NT == 4 ? D : D + 4;        // floats of a column
  static constexpr int kDumpBytes = kWarps * kCols * (kRow + 2) * 4;
  static constexpr int kBudget = (225 / kCtasPerSm - 1) * 1024 - kDumpBytes - kQBytes - 1024;
  static constexpr int kStages0 = kBudget / (kWarps * kStage);
  static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
  static constexpr int kSmem = kWarps * kStages * kStage + kDumpBytes + kQBytes;
  static_assert(kStages >= 2, "a ring has two stages at least");
};

template <int D, int BS, int NT, bool kMulti>
__global__ void __launch_bounds__(kThreads4, Cfg4<D, BS, NT>::kCtasPerSm) q4_kernel(const Q4Args a) {
  using C = Cfg4<D, BS, NT>;
  using G = Geo4<D, BS>;
  constexpr int S = C::kStages, NG = G::kGroups;
  constexpr int kKSteps = D / 16, kMTiles = D / 16;
  extern __shared__ __align__(128) unsigned char smem4[];
  __shared__ uint64_t bars[kWarps][8];
  __shared__ long long scan[kWarps];
  __shared__ int start_b, start_ct, start_us, range_len;
  __shared__ int range_per;
  __shared__ unsigned int q_top;                    // bits of the largest finite |q| of a piece
  __shared__ float q_sum[C::kCols][NG];

  const int hk = blockIdx.x, c = a.whole ? (int)(gridDim.y - 1 - blockIdx.y) : (int)blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int GQ = a.group, Hq = a.num_q_heads;

  // (launched as a programmatic dependent: what is before may still run until here)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane < S) mbar_init(smem_addr(&bars[warp][lane]), 1);     // (a warp uses its own only)
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();

  // ---- this CTA's range of the head's block positions ----------------------
  const bool one = !kMulti && a.whole;              // one CTA per sequence
  int b0 = c, ct0 = 0, us0 = 0, len0 = 0, fid = 0;
  if (one) {
    // the first blocks' ids and the queries are asked for beside the length
    const int j = warp * C::kBlocks + lane;
    if (lane < C::kBlocks && j < a.max_blocks) fid = __ldg(a.block_tables + (int64_t)c * a.max_blocks + j);
    const __nv_bfloat16* row = a.q + ((int64_t)c * Hq + (int64_t)hk * GQ) * D;
    if ((int)threadIdx.x * 64 < GQ * D) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + threadIdx.x * 64));
    const Seq s = seq_of<BS, kMulti>(a, c);
    if (s.bad) {
      if (threadIdx.x == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
      uint4* o = reinterpret_cast<uint4*>(a.out + ((int64_t)c * Hq + (int64_t)hk * GQ) * D);
      for (int e = threadIdx.x; e < GQ * D / 8; e += kThreads4) o[e] = make_uint4(0, 0, 0, 0);
      return;
    }
    len0 = s.nblk;
  } else {
    // Every thread sums a run of sequences; the sums' prefix says where the
    // range begins.  Positions are blocks (whole: column tiles).
    if (threadIdx.x == 0) start_b = -1;
    const int run = (a.batch + kThreads4 - 1) / kThreads4;
    const int r0 = threadIdx.x * run, r1 = min(a.batch, r0 + run);
    long long sum = 0;
    for (int b = r0; b < r1; ++b) {
      const Seq s = seq_of<BS, kMulti>(a, b);
      sum += a.whole ? s.nct : (long long)s.nct * s.nblk;
      if (s.bad && b % a.ctas == c) {
        if (hk == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
        for (int i = 0; i < s.n; ++i) {
          uint4* o = reinterpret_cast<uint4*>(a.out + ((int64_t)(s.q0 + i) * Hq + (int64_t)hk * GQ) * D);
          for (int e = 0; e < GQ * D / 8; ++e) o[e] = make_uint4(0, 0, 0, 0);
        }
      }
    }
    long long at = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, at, off);
      if (lane >= off) at += x;
    }
    if (lane == 31) scan[warp] = at;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += scan[w];
      total += scan[w];
    }
    at -= sum;                                      // sequences before this thread's
    constexpr int kMinRange = kMinRangeTokens / BS;
    const long long even = total < 0x7fffffff - a.ctas ? ((int)total + a.ctas - 1) / a.ctas
                                                       : (total + a.ctas - 1) / a.ctas;
    const long long per = a.whole ? 1 : (even > kMinRange ? even : kMinRange);
    const long long u0 = (long long)c * per;
    if (u0 >= at && u0 < at + sum) {
      for (int b = r0; b < r1; ++b) {
        const Seq s = seq_of<BS, kMulti>(a, b);
        const long long w = a.whole ? s.nct : (long long)s.nct * s.nblk;
        if (u0 < at + w) {
          const long long in = u0 - at;
          start_b = b;
          if (a.whole) {
            start_ct = (int)in;
            start_us = 0;
            range_len = s.nblk;
          } else {
            start_ct = kMulti ? (int)(in / s.nblk) : 0;
            start_us = -(int)(in - (long long)start_ct * s.nblk);
            range_len = (int)(u0 + per < total ? per : total - u0);
            range_per = (int)per;
          }
          break;
        }
        at += w;
      }
    }
    __syncthreads();
    if (start_b < 0) {                              // nothing for this CTA
      if (!a.whole && threadIdx.x == 0) a.ws_meta[(int64_t)hk * a.ctas + c] = make_int4(0, 0, 0, 0);
      return;
    }
    b0 = start_b;
    ct0 = start_ct;
    us0 = start_us;
    len0 = range_len;
  }
  const int64_t cell = (int64_t)hk * a.ctas + c;
  const uint32_t ring = smem_addr(smem4) + warp * S * C::kStage;
  float* dump = reinterpret_cast<float*>(smem4 + kWarps * S * C::kStage);   // [warp][column][kRow]
  float* dump_ml = dump + kWarps * C::kCols * C::kRow;                      // [warp][column][2]
  const uint32_t qsm = smem_addr(smem4) + kWarps * S * C::kStage + C::kDumpBytes;

  // ---- the warp's ring: every fourth step of each piece ---------------------
  constexpr int PB = C::kBlocks;
  Walk<BS, kMulti> f, w;
  f.start(a, b0, ct0, us0, len0);
  w = f;
  int fj = f.j0 + warp * PB;                        // next blocks to copy; lane i < PB has the i-th's id
  int fs = 0, cs = 0, ahead = 0;                    // stages: next to fill, to use; filled
  uint32_t phase = 0, bad_stages = 0;
  bool dead = false;
  auto settle = [&](bool known) {                   // to the next step the warp will copy
    while (!f.done() && fj >= f.j1) {
      f.next(a);
      fj = f.j0 + warp * PB;
    }
    if (!known && !f.done() && lane < min(PB, f.j1 - fj))
      fid = __ldg(a.block_tables + (int64_t)f.b * a.max_blocks + fj + lane);
  };
  settle(one);
  auto fetch = [&]() {
    if (f.done() || dead) return;
    const int have = min(PB, f.j1 - fj);
    const bool ok = __all_sync(0xffffffffu, lane >= have || (unsigned)fid < (unsigned)a.num_blocks);
    bad_stages = (bad_stages & ~(1u << fs)) | (ok ? 0u : 1u << fs);
    if (lane < have) {
      const uint32_t bar = smem_addr(&bars[warp][fs]);
      if (lane == 0) {
        if (!ok) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
        mbar_expect_tx(bar, have * G::kRecord);
      }
      bulk_load(ring + fs * C::kStage + lane * G::kRecord,
                a.kv + ((int64_t)(ok ? fid : 0) * a.num_kv_heads + hk) * G::kRecord, G::kRecord, bar);
    }
    fs = fs + 1 == S ? 0 : fs + 1;
    ++ahead;
    fj += kWarps * PB;
    settle(false);
  };
#pragma unroll 1
  for (int s = 0; s < S; ++s) fetch();

  // rows of a 16-token tile: MMA row r holds token tau(r) (and 8 + tau), so
  // that both products read shared memory with few conflicts
  const int tau = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;
  const int va = t, vb = 4 + (t ^ 1);               // tau(2t), tau(2t + 1)

  bool merged = false;                              // this CTA's meta entry is written
  for (; !w.done(); w.next(a)) {
    if (w.j0 >= w.j1) continue;                     // no query of the tile sees these blocks
    // ---- queries: columns 8 nt + c are (token ct * tile + col / G, head col % G)
    const int tok0 = w.ct * a.tile_tokens;
    const int ntok = kMulti ? min(a.tile_tokens, w.s.n - tok0) : 1;
    const int nta = (ntok * GQ + 7) / 8;            // column tiles in use
    float kfac;
    {
      // A thread takes words (8 elements) word, of columns first, first + step, ..
      constexpr int kWords = D / 8, kStep = kThreads4 / kWords, kEach = (C::kCols + kStep - 1) / kStep;
      const int word = threadIdx.x % kWords, col0 = threadIdx.x / kWords;
      uint4 x[kEach];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int col = col0 + i * kStep, tok = col / GQ;
        x[i] = make_uint4(0, 0, 0, 0);
        if (tok < ntok && col < a.tile_tokens * GQ)
          x[i] = __ldg(reinterpret_cast<const uint4*>(
                           a.q + ((int64_t)(w.s.q0 + tok0 + tok) * Hq + (int64_t)hk * GQ + col % GQ) * D) + word);
        // the largest finite magnitude, both halves of a word at once
        const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t lo = xw[k] & 0x7fffu, hi = xw[k] >> 16 & 0x7fffu;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (threadIdx.x == 0) q_top = 0;
      __syncthreads();                              // the last piece's fragments and sums are no longer read
      if (lane == 0) atomicMax(&q_top, top);
      __syncthreads();
      top = q_top;
      // largest * 2^e in [2^14, 2^15): q / 16 is exact in fp16 from 2^-27 of it on (the
      // last of bf16's 8 bits is then 2^-24 at least)
      int e = top > 0 ? 141 - (int)(top >> 7) : 0;
      e = min(e, 126);                              // (-113 at least)
      // (a negative scale turns q's sign, a zero one takes q as 0: kfac is positive,
      // so that a masked score of -infinity stays one)
      float up = __uint_as_float((uint32_t)(127 + e) << 23);
      // (finite too: no score of 0 becomes NaN)
      kfac = fabsf(a.scale_log2) * 16777216.0f * __uint_as_float((uint32_t)(127 - e) << 23);
      kfac = fminf(fmaxf(kfac, 1e-37f), 3e38f);
      if (a.scale_log2 <= 0.0f) up = a.scale_log2 < 0.0f ? -up : 0.0f;
      const float down = up * 0.0625f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int col = col0 + i * kStep;
        if (C::kCols % kStep != 0 && col >= C::kCols) break;        // (whole groups of 8 lanes)
        const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        float v[8], sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] = __uint_as_float(xw[k] << 16);
          v[2 * k + 1] = __uint_as_float(xw[k] & 0xffff0000u);
          sum += v[2 * k] * up + v[2 * k + 1] * up;      // (unscaled it may pass fp32)
        }
        // B fragment of k-step ks: lane (g = column % 8, t) holds elements 2 hh, 2 hh
        // + 4 and (times 1/16, its codes are high nibbles) 2 hh + 1, 2 hh + 5 of word
        // 2 t + ci of the group
        const int gr = word / 8, tt = word % 8 / 2, ci = word % 2;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int ks = (gr * 2 + ci) * 2 + hh;
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(
                           qsm + ((ks * NT + col / 8) * 32 + col % 8 * 4 + tt) * 8),
                       "r"(pack2<true>(v[2 * hh] * up, v[2 * hh + 4] * up)),
                       "r"(pack2<true>(v[2 * hh + 1] * down, v[2 * hh + 5] * down))
                       : "memory");
        }
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) sum += __shfl_xor_sync(__activemask(), sum, off);
        if (word % 8 == 0) q_sum[col][gr] = sum * 5.9604644775390625e-8f;   // * 2^-24
      }
      __syncthreads();
    }
    uint32_t qf[C::kQShared ? 1 : kKSteps][C::kQShared ? 1 : NT][2];
    if constexpr (!C::kQShared) {
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 b = lds64(qsm + ((ks * NT + nt) * 32 + lane) * 8);
          qf[ks][nt][0] = b.x;
          qf[ks][nt][1] = b.y;
        }
    }
    // sums of q over a group, in units of the products with codes
    float qs[NT][NG][2];
    int cpos[kMulti ? NT : 1][2];                   // last token a column sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = 8 * nt + 2 * t + k;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) qs[nt][gr][k] = q_sum[col][gr];
        if constexpr (kMulti) cpos[nt][k] = w.s.L - w.s.n + tok0 + min(col / GQ, ntok - 1);
      }
    }
    const int all_see = kMulti ? w.s.L - w.s.n + tok0 + 1 : w.s.L;   // tokens every column sees

    float o[NT][kMTiles][4];
    float ref[NT][2], l[NT][2], pm[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < kMTiles; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
      ref[nt][0] = ref[nt][1] = kNoRef;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) pm[nt][gr][0] = pm[nt][gr][1] = 0.0f;
    }
    bool bad = dead;

    // kA of the kNT column tiles in use: a sequence with few queries in a call
    // with long ones pays for one
    auto steps = [&](auto tiles_in_use) {
      constexpr int A = decltype(tiles_in_use)::value;
      constexpr int T = C::kTiles;
      for (int j = w.j0 + warp * PB; j < w.j1; j += kWarps * PB) {
        if (ahead == 0) break;                      // (after a wait that gave up)
        const uint32_t bar = smem_addr(&bars[warp][cs]);
        // (the lanes agree on the outcome: what follows is the whole warp's)
        if (__any_sync(0xffffffffu, !mbar_wait(bar, (phase >> cs) & 1u))) {
          if (lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_WAIT_TIMEOUT);
          dead = true;
        }
        bad |= dead || ((bad_stages >> cs) & 1u);
        const uint32_t stage = ring + cs * C::kStage;
        phase ^= 1u << cs;
        cs = cs + 1 == S ? 0 : cs + 1;
        --ahead;
        const int first = j * BS;                   // the step's first token
        const int have = min((j + PB <= w.j1 ? PB : 1) * BS, w.s.L - first);
        const bool inner = first + 32 <= all_see && have == 32;   // every row written and seen by every column
        if (!bad) {
#pragma unroll 1
          for (int base = 0; base < 32; base += 16 * T) {
            if (base >= have) break;
            // this lane's rows of tile x: its block's record, rows lo and lo + 8 of it
            uint32_t rec[T];
            int row0[T];
#pragma unroll
            for (int x = 0; x < T; ++x) {
              const int at = base + 16 * x;
              rec[x] = stage + (BS == 16 ? at / 16 * G::kRecord : 0);
              row0[x] = BS == 16 ? 0 : at;
            }
            // ---- scores ------------------------------------------------------
            float sc[T][A][4];
            {
              uint32_t kw[T][2][2 * NG], kp[T][2][NG];
#pragma unroll
              for (int x = 0; x < T; ++x) {
                const int lo = row0[x] + tau;
                lds_words(kw[x][0], rec[x] + lo * G::kRowBytes + t * (D / 8));
                lds_words(kw[x][1], rec[x] + (lo + 8) * G::kRowBytes + t * (D / 8));
                lds_words(kp[x][0], rec[x] + G::kParAt + lo * G::kParBytes);
                lds_words(kp[x][1], rec[x] + G::kParAt + (lo + 8) * G::kParBytes);
              }
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) {
                float acc[T][A][4];
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {    // word ci = ks / 2 of the lane's two, half ks % 2
                  uint2 b[A];
#pragma unroll
                  for (int nt = 0; nt < A; ++nt) {
                    if constexpr (C::kQShared) b[nt] = lds64(qsm + (((gr * 4 + ks) * NT + nt) * 32 + lane) * 8);
                    else b[nt] = make_uint2(qf[gr * 4 + ks][nt][0], qf[gr * 4 + ks][nt][1]);
                  }
#pragma unroll
                  for (int x = 0; x < T; ++x) {
                    const uint32_t u = kw[x][0][ks / 2 * NG + gr] >> (ks % 2 * 8);
                    const uint32_t v = kw[x][1][ks / 2 * NG + gr] >> (ks % 2 * 8);
                    const uint32_t fa[4] = {u & kLow, v & kLow, u & kHigh, v & kHigh};
#pragma unroll
                    for (int nt = 0; nt < A; ++nt) {
                      if (ks == 0) mma16816_first(acc[x][nt], fa, b[nt].x, b[nt].y);
                      else mma16816<true>(acc[x][nt], fa, b[nt].x, b[nt].y);
                    }
                  }
                }
#pragma unroll
                for (int x = 0; x < T; ++x) {
                  const uint32_t k0 = kp[x][0][gr], k1 = kp[x][1][gr];
                  const float s0 = pair_scale(k0), s1 = pair_scale(k1);
                  const float m0 = pair_min(k0), m1 = pair_min(k1);
#pragma unroll
                  for (int nt = 0; nt < A; ++nt) {
                    const float* qq = qs[nt][gr];
                    float* y = sc[x][nt];
                    y[0] = fmaf(s0, acc[x][nt][0], gr ? fmaf(m0, qq[0], y[0]) : m0 * qq[0]);
                    y[1] = fmaf(s0, acc[x][nt][1], gr ? fmaf(m0, qq[1], y[1]) : m0 * qq[1]);
                    y[2] = fmaf(s1, acc[x][nt][2], gr ? fmaf(m1, qq[0], y[2]) : m1 * qq[0]);
                    y[3] = fmaf(s1, acc[x][nt][3], gr ? fmaf(m1, qq[1], y[3]) : m1 * qq[1]);
                  }
                }
              }
            }
            // ---- V's scales and minima of the same tokens ----------------------
            uint32_t vp[T][2][NG];
#pragma unroll
            for (int x = 0; x < T; ++x) {
              const uint32_t at = rec[x] + G::kParAt + G::kParams + (row0[x] + tau) * G::kParBytes;
              lds_words(vp[x][0], at);
              lds_words(vp[x][1], at + 8 * G::kParBytes);
            }
            if (!inner) {
#pragma unroll
              for (int x = 0; x < T; ++x) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const int tok = base + 16 * x + tau + 8 * r;
                  const bool out = tok >= have;
#pragma unroll
                  for (int gr = 0; gr < NG; ++gr)
                    if (out) vp[x][r][gr] = 0;          // a row never written may hold NaN
#pragma unroll
                  for (int nt = 0; nt < A; ++nt) {
                    if (out || (kMulti && first + tok > cpos[nt][0])) sc[x][nt][2 * r] = -INFINITY;
                    if (out || (kMulti && first + tok > cpos[nt][1])) sc[x][nt][2 * r + 1] = -INFINITY;
                  }
                }
              }
            }
            // ---- weights against the columns' references -------------------------
            // p, and p * max(vscale, |vmin| / 16), with p * vscale as it enters the
            // product (rows of equal values have the least scale, and p * vmin has to
            // stay within fp32 too); where one of them passes its bound (in the first
            // tile, and rarely after it) the references move to the largest score +
            // exponent of that maximum, less five (exponents are -100 at least), and p
            // is taken again.
            // (The products are made again where they are packed: held meanwhile for 32
            // columns they would not fit the registers.)
            float p[T][A][4];
            auto weigh = [&]() {
              float top = 0.0f, top_s = 0.0f;
#pragma unroll
              for (int x = 0; x < T; ++x) {
                float row[2] = {0.0f, 0.0f};       // a token's largest p; times its largest scale or |min| / 16
#pragma unroll
                for (int nt = 0; nt < A; ++nt) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) p[x][nt][k] = ex2(fmaf(sc[x][nt][k], kfac, -ref[nt][k & 1]));
                  row[0] = fmaxf(fmaxf(row[0], p[x][nt][0]), p[x][nt][1]);
                  row[1] = fmaxf(fmaxf(row[1], p[x][nt][2]), p[x][nt][3]);
                }
                top = fmaxf(fmaxf(top, row[0]), row[1]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  // (a pair's word as a number is its min, off by less than 2^-7 of it)
                  float most = fabsf(__uint_as_float(vp[x][r][0]));
#pragma unroll
                  for (int gr = 1; gr < NG; ++gr) most = fmaxf(most, fabsf(__uint_as_float(vp[x][r][gr])));
                  most *= 0.0625f;
#pragma unroll
                  for (int gr = 0; gr < NG; ++gr) most = fmaxf(most, pair_scale(vp[x][r][gr]));
                  top_s = fmaxf(top_s, row[r] * most);
                }
              }
              return top > 4294967296.0f || top_s > 2048.0f;
            };
            if (__any_sync(0xffffffffu, weigh())) {
#pragma unroll
              for (int nt = 0; nt < A; ++nt) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float mx = -INFINITY;
#pragma unroll
                  for (int x = 0; x < T; ++x)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                      mx = fmaxf(mx, fmaf(sc[x][nt][k + 2 * r], kfac, value_exponent(vp[x][r])));
#pragma unroll
                  for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                  const float to = fmaxf(ref[nt][k], mx - 5.0f);
                  const float al = ex2(ref[nt][k] - to);
                  l[nt][k] = times_ex2(l[nt][k], ref[nt][k] - to);
                  ref[nt][k] = to;
#pragma unroll
                  for (int gr = 0; gr < NG; ++gr) pm[nt][gr][k] *= al;
#pragma unroll
                  for (int i = 0; i < kMTiles; ++i) {
                    o[nt][i][k] *= al;
                    o[nt][i][k + 2] *= al;
                  }
                }
              }
              weigh();
            }
#pragma unroll
            for (int x = 0; x < T; ++x) {
              // ---- V's codes: lane g has word g of every group --------------------
              uint32_t vw[4][NG];
              const uint32_t vrow = rec[x] + G::kCodes + row0[x] * G::kRowBytes + g * (NG * 4);
              lds_words(vw[0], vrow + va * G::kRowBytes);
              lds_words(vw[1], vrow + vb * G::kRowBytes);
              lds_words(vw[2], vrow + (va + 8) * G::kRowBytes);
              lds_words(vw[3], vrow + (vb + 8) * G::kRowBytes);
              uint32_t pb[A][NG][2];
#pragma unroll
              for (int nt = 0; nt < A; ++nt) {
                const float* y = p[x][nt];
                l[nt][0] += y[0] + y[2];
                l[nt][1] += y[1] + y[3];
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                  const float m0 = pair_min(vp[x][0][gr]), m1 = pair_min(vp[x][1][gr]);
                  const float s0 = pair_scale(vp[x][0][gr]), s1 = pair_scale(vp[x][1][gr]);
                  pb[nt][gr][0] = transposed8(pack2<true>(y[0] * s0, y[1] * s0));
                  pb[nt][gr][1] = transposed8(pack2<true>(y[2] * s1, y[3] * s1));
                  pm[nt][gr][0] = fmaf(y[0], m0, fmaf(y[2], m1, pm[nt][gr][0]));
                  pm[nt][gr][1] = fmaf(y[1], m0, fmaf(y[3], m1, pm[nt][gr][1]));
                }
              }
              // ---- O^T += V^T . P^T ---------------------------------------------------
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  // tokens 2t, 2t + 1 and 2t + 8, 2t + 9; nibbles 2k and 2k + 1
                  uint32_t u = prmt(vw[0][gr], vw[1][gr], k >= 2 ? 0x7632u : 0x5410u);
                  uint32_t v = prmt(vw[2][gr], vw[3][gr], k >= 2 ? 0x7632u : 0x5410u);
                  if (k % 2) u >>= 8, v >>= 8;
                  const uint32_t fa[4] = {u & kLow, u & kHigh, v & kLow, v & kHigh};
#pragma unroll
                  for (int nt = 0; nt < A; ++nt) mma16816<true>(o[nt][gr * 4 + k], fa, pb[nt][gr][0], pb[nt][gr][1]);
                }
              }
            }
          }
        }
        __syncwarp();
        fetch();
      }
    };
    if constexpr (NT > 1) {
      if (nta == 1) steps(std::integral_constant<int, 1>{});
      else steps(std::integral_constant<int, NT>{});
    } else {
      steps(std::integral_constant<int, 1>{});
    }

    // ---- the four warps' (reference, sum, O), joined ---------------------------
    // O[nt][gr * 4 + k]: elements gr * 64 + 8 g + 2 k (c0, c1: * 2^24) and + 1 (c2, c3: * 2^20)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], off);
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) pm[nt][gr][k] += __shfl_xor_sync(0xffffffffu, pm[nt][gr][k], off);
        }
        if (bad) l[nt][k] = -1.0f;
#pragma unroll
        for (int i = 0; i < kMTiles; ++i) {
          o[nt][i][k] = fmaf(o[nt][i][k], 16777216.0f, pm[nt][i / 4][k]);
          o[nt][i][k + 2] = fmaf(o[nt][i][k + 2], 1048576.0f, pm[nt][i / 4][k]);
        }
      }
    }
    // columns in use; the warps' shares are added by all threads, four elements each
    const int used = ntok * GQ;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = 8 * nt + 2 * t + k;
        if (col >= used) continue;
        float* to = dump + (warp * C::kCols + col) * C::kRow;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const int i = gr * 4;
          float4* y = reinterpret_cast<float4*>(to + gr * 64 + 8 * g);
          y[0] = make_float4(o[nt][i][k], o[nt][i][k + 2], o[nt][i + 1][k], o[nt][i + 1][k + 2]);
          y[1] = make_float4(o[nt][i + 2][k], o[nt][i + 2][k + 2], o[nt][i + 3][k], o[nt][i + 3][k + 2]);
        }
        if (g == 0) {
          dump_ml[(warp * C::kCols + col) * 2] = ref[nt][k];
          dump_ml[(warp * C::kCols + col) * 2 + 1] = l[nt][k];
        }
      }
    }
    __syncthreads();
    const bool starts = w.j0 == 0;
    // CTAs that hold the rest of the unit's visible blocks
    const int follow = !starts || a.whole ? 0 : (w.us + w.visible(a) - 1) / range_per;
    const bool direct = starts && follow == 0;
    if (!direct && starts) {
      merged = true;
      if (threadIdx.x == 0) a.ws_meta[cell] = make_int4(follow, w.s.q0 + tok0, ntok, 0);
    }
    const int64_t part = cell * 2 + (starts ? 1 : 0);
#pragma unroll 1
    for (int i = threadIdx.x; i < used * (D / 4); i += kThreads4) {
      const int col = i / (D / 4), e = i % (D / 4) * 4;
      float R = kNoRef, den = 0.0f;
      bool any_bad = false;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) R = fmaxf(R, dump_ml[(v * C::kCols + col) * 2]);
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float2 ml = *reinterpret_cast<const float2*>(dump_ml + (v * C::kCols + col) * 2);
        const float4 y = *reinterpret_cast<const float4*>(dump + (v * C::kCols + col) * C::kRow + e);
        const float f = ex2(ml.x - R);
        any_bad |= ml.y < 0.0f;
        den += times_ex2(ml.y, ml.x - R);
        sum.x = fmaf(f, y.x, sum.x);
        sum.y = fmaf(f, y.y, sum.y);
        sum.z = fmaf(f, y.z, sum.z);
        sum.w = fmaf(f, y.w, sum.w);
      }
      if (direct) {
        const float r = 1.0f / den;
        uint2 y = make_uint2(0u, 0u);
        if (!any_bad) y = make_uint2(pack2<false>(sum.x * r, sum.y * r), pack2<false>(sum.z * r, sum.w * r));
        *reinterpret_cast<uint2*>(
            a.out + ((int64_t)(w.s.q0 + tok0 + col / GQ) * Hq + (int64_t)hk * GQ + col % GQ) * D + e) = y;
      } else {
        *reinterpret_cast<float4*>(a.ws_acc + (part * C::kCols + col) * D + e) = sum;
        if (e == 0)
          *reinterpret_cast<float2*>(a.ws_ml + (part * C::kCols + col) * 2) = make_float2(R, any_bad ? -1.0f : den);
      }
    }
  }
  if (!a.whole && threadIdx.x == 0 && !merged) a.ws_meta[cell] = make_int4(0, 0, 0, 0);
  // copies still in flight (after a wait that gave up) land before the CTA ends
  for (; ahead > 0; --ahead) {
    mbar_wait(smem_addr(&bars[warp][cs]), (phase >> cs) & 1u);
    cs = cs + 1 == S ? 0 : cs + 1;
  }
}

// Joins the partials of the unit that CTA c of a KV head began and later CTAs
// ended: out = sum_i 2^(r_i - R) acc_i / sum_i 2^(r_i - R) l_i.  One CTA per
// (range, KV head, column or four of them); its warps take a column each where the
// partials are few, else a column's partials in turn.
template <int D>
__global__ void __launch_bounds__(128) q4_merge_kernel(const Q4Args a, int cols) {
  constexpr int E = D / 32;
  __shared__ float part[4][32][E + 1];
  const int c = blockIdx.x, hk = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t cell = (int64_t)hk * a.ctas + c;
  const int4 meta = a.ws_meta[cell];
  if (meta.x == 0) return;
  const int count = meta.x + 1;                     // partial 0: this CTA's second, k: CTA c + k's first
  const bool alone = count <= kAloneParts;          // few partials: a warp has a column to itself
  const int first = alone ? 0 : warp, step = alone ? 1 : 4;
  for (int col = blockIdx.z + (alone ? warp * gridDim.z : 0); col < meta.z * a.group;
       col += alone ? 4 * gridDim.z : gridDim.z) {
    const int64_t p0 = (cell * 2 + 1) * cols + col;
    auto at = [&](int k) { return k == 0 ? p0 : (cell + k) * 2 * cols + col; };
    float R = kNoRef;
    bool bad = false;
    for (int k = lane; k < count; k += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(a.ws_ml + at(k) * 2);
      R = fmaxf(R, ml.x);
      bad |= ml.y < 0.0f;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, off));
    bad = __any_sync(0xffffffffu, bad);
    float num[E], den = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) num[e] = 0.0f;
#pragma unroll 4
    for (int k = first; k < count; k += step) {
      const float2 ml = *reinterpret_cast<const float2*>(a.ws_ml + at(k) * 2);
      const float f = ex2(ml.x - R);
      den += times_ex2(ml.y, ml.x - R);
      const float* acc = a.ws_acc + at(k) * D + lane * E;
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(acc);
        num[0] = fmaf(f, x.x, num[0]);
        num[1] = fmaf(f, x.y, num[1]);
        num[2] = fmaf(f, x.z, num[2]);
        num[3] = fmaf(f, x.w, num[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(acc);
        num[0] = fmaf(f, x.x, num[0]);
        num[1] = fmaf(f, x.y, num[1]);
      }
    }
    if (!alone) {
      __syncthreads();                              // (the last column's shares are read)
#pragma unroll
      for (int e = 0; e < E; ++e) part[warp][lane][e] = num[e];
      part[warp][lane][E] = den;
      __syncthreads();
      if (warp != 0) continue;
      for (int k = 1; k < 4; ++k) {
#pragma unroll
        for (int e = 0; e < E; ++e) num[e] += part[k][lane][e];
        den += part[k][lane][E];
      }
    }
    const float r = bad ? 0.0f : 1.0f / den;
    uint32_t x[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) x[e] = bad ? 0u : pack2<false>(num[2 * e] * r, num[2 * e + 1] * r);
    __nv_bfloat16* out =
        a.out + ((int64_t)(meta.y + col / a.group) * a.num_q_heads + (int64_t)hk * a.group + col % a.group) * D + lane * E;
    if constexpr (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(x[0], x[1]);
    else *reinterpret_cast<uint32_t*>(out) = x[0];
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

template <int D, int BS, int NT, bool kMulti>
kv_status launch_q4(const Q4Args& a, cudaStream_t s) {
  using C = Cfg4<D, BS, NT>;
  static std::mutex mu;
  static bool set[64] = {};
  int dev = 0;
  kv_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != KV_OK) return st;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && !set[dev]) {
      st = cuda_check(cudaFuncSetAttribute(q4_kernel<D, BS, NT, kMulti>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem),
                      "cudaFuncSetAttribute(q4_kernel)");
      if (st != KV_OK) return st;
      set[dev] = true;
    }
  }
  // Both launches are programmatic dependents of what is before them (each waits
  // for it on the device before its first access), so that their launches overlap it.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.num_kv_heads, (unsigned)a.ctas);
  cfg.blockDim = dim3(kThreads4);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  st = cuda_check(cudaLaunchKernelEx(&cfg, q4_kernel<D, BS, NT, kMulti>, a), "q4_kernel launch");
  if (st != KV_OK || a.whole) return st;
  const int used = (kMulti ? min(a.max_query_len, a.tile_tokens) : 1) * a.group;
  // Four columns per CTA where a sequence has few ranges on average (a warp joins
  // each) or columns are many; one where the partials are many and the cells few.
  const bool several = used > 8 || a.ctas <= kAloneParts / 2 * a.batch;
  cfg.gridDim = dim3((unsigned)a.ctas, (unsigned)a.num_kv_heads, (unsigned)(several ? (used + 3) / 4 : used));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_merge_kernel<D>, a, C::kCols), "q4_merge_kernel launch");
}

template <int D, int BS>
kv_status launch_q4_nt(const Q4Args& a, int nt, cudaStream_t s) {
  if (a.query_start == nullptr) return launch_q4<D, BS, 1, false>(a, s);
  if (nt == 1) return launch_q4<D, BS, 1, true>(a, s);
  if (nt == 2) return launch_q4<D, BS, 2, true>(a, s);
  if (nt == 3) return launch_q4<D, BS, 3, true>(a, s);
  return launch_q4<D, BS, 4, true>(a, s);
}

// Column tiles of 8 that hold a sequence's queries, four at most.
int column_tiles(int max_query_len, int group) {
  const long long cols = (long long)max_query_len * group;
  return cols >= 32 ? 4 : (int)((cols + 7) / 8);
}

// CTAs per KV head of a split call: one wave of them over all heads.
int split_ctas(int sms, int nt, int num_kv_heads) {
  const int all = sms * ctas_per_sm(nt);
  return all / num_kv_heads > 0 ? all / num_kv_heads : 1;
}

size_t q4_workspace(int ctas, int num_kv_heads, int nt, int head_dim) {
  const size_t cells = (size_t)ctas * num_kv_heads;
  return cells * (16 + 2 * 8 * (size_t)nt * (head_dim + 2) * sizeof(float));
}

// Sequences that may have long queries.
int long_slots(int batch, int num_tokens, int max_query_len, int group) {
  const int least = (kLongRows + group - 1) / group;
  if (max_query_len < least) return 0;
  const int most = num_tokens / least < batch ? num_tokens / least : batch;
  return most < 65535 ? most : 65535;
}

constexpr int kMostSms = 160;                       // what the size query sizes for

kv_status q4_common(void* out, const void* q, const void* kv_cache, const int32_t* block_tables,
                    int max_blocks, const int32_t* seq_lens, const int32_t* query_start, int batch,
                    int num_tokens, int max_query_len, int num_q_heads, int num_kv_heads, int head_dim,
                    int num_blocks, int block_size, int max_seq_len, float scale, void* workspace,
                    size_t workspace_bytes, void* stream, bool multi, const char* who) {
  if (batch < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
      max_blocks <= 0 || num_blocks <= 0 || max_seq_len <= 0 || max_query_len <= 0)
    return fail(KV_ERR_INVALID_ARG, "%s: bad sizes", who);
  const int G = num_q_heads / num_kv_heads;
  if (G > kMaxGroup) return fail(KV_ERR_INVALID_ARG, "%s: at most 8 query heads per KV head (got %d)", who, G);
  if (num_kv_heads > 65535) return fail(KV_ERR_INVALID_ARG, "%s: at most 65535 KV heads (got %d)", who, num_kv_heads);
  if (head_dim != 64 && head_dim != 128) return fail(KV_ERR_INVALID_ARG, "%s: head_dim must be 64 or 128", who);
  if (block_size != 16 && block_size != 32) return fail(KV_ERR_INVALID_ARG, "%s: block_size must be 16 or 32", who);
  if (batch == 0 || num_tokens == 0) return KV_OK;
  if (!out || !q || !kv_cache || !block_tables || !seq_lens || (multi && !query_start))
    return fail(KV_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned16(out) || !aligned16(q) || !aligned16(kv_cache))
    return fail(KV_ERR_INVALID_ARG, "%s: out, q and the pool must be 16-byte aligned", who);
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  Q4Args a = {};
  a.out = static_cast<__nv_bfloat16*>(out);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.kv = static_cast<const unsigned char*>(kv_cache);
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = multi ? query_start : nullptr;
  a.flags = di.flags;
  a.max_blocks = max_blocks;
  a.batch = batch;
  a.num_tokens = num_tokens;
  a.max_query_len = multi ? max_query_len : 1;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_seq_len = max_seq_len;
  a.group = G;
  a.scale_log2 = scale * kLog2e;
  const int nt = multi ? column_tiles(max_query_len, G) : 1;
  a.tile_tokens = multi ? 8 * nt / G : 1;
  // Column tiles of the whole batch, at most.  Short sequences, and calls with
  // long queries whose tiles alone fill the GPU twice, take a CTA for each tile.
  const int sms = di.num_sms < kMostSms ? di.num_sms : kMostSms;
  const bool long_queries = multi && max_query_len > a.tile_tokens;
  const int64_t tiles = long_queries ? (int64_t)num_tokens / a.tile_tokens + batch : batch;
  const int split = split_ctas(sms, nt, num_kv_heads);
  a.whole = (max_seq_len <= kWholeTokens || (long_queries && tiles >= 2 * (int64_t)split)) && tiles <= 65535;
  // Long queries, as many sequences as the workspace has room for beside the partials
  const size_t few = (q4_workspace(split, num_kv_heads, nt, head_dim) + 127) & ~(size_t)127;
  const int slots = multi ? long_slots(batch, num_tokens, max_query_len, G) : 0;
  const size_t slot = q4_slot_bytes(num_kv_heads, head_dim, max_seq_len), plan = q4_plan_bytes(batch, slots);
  int fit = 0;
  if (slots > 0 && workspace && aligned16(workspace) && workspace_bytes > few + 128 + plan) {
    const size_t room = (workspace_bytes - few - 128 - plan) / slot;
    fit = room < (size_t)slots ? (int)room : slots;
  }
  if (fit == slots && fit > 0) a.whole = 0;         // what is left has few rows
  a.ctas = a.whole ? (int)tiles : split;
  if (!a.whole) {
    // (a CTA counts the blocks of its range in 32 bits)
    if (tiles * ((max_seq_len + (int64_t)block_size - 1) / block_size) / split >= (int64_t)1 << 30)
      return fail(KV_ERR_INVALID_ARG, "%s: more than 2^30 blocks of %d tokens per range", who, block_size);
    const size_t need = q4_workspace(a.ctas, num_kv_heads, nt, head_dim);
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
      return fail(KV_ERR_INVALID_ARG,
                  "%s: workspace must be 16-byte aligned and hold %zu bytes "
                  "(pagedkv_q4_workspace_bytes gives a safe size)", who, need);
    const size_t cells = (size_t)a.ctas * num_kv_heads;
    a.ws_meta = static_cast<int4*>(workspace);
    a.ws_acc = reinterpret_cast<float*>(a.ws_meta + cells);
    a.ws_ml = a.ws_acc + cells * 2 * 8 * nt * head_dim;
  }
  cudaStream_t s = (cudaStream_t)stream;
  if (fit > 0) {
    unsigned char* w = static_cast<unsigned char*>(workspace) + few;
    w += (0 - reinterpret_cast<uintptr_t>(w)) & 127;
    Q4LongArgs g = {};
    g.out = a.out;
    g.q = a.q;
    g.kv = a.kv;
    g.block_tables = block_tables;
    g.seq_lens = seq_lens;
    g.query_start = query_start;
    g.flags = di.flags;
    g.slots = fit;
    g.max_blocks = max_blocks;
    g.batch = batch;
    g.num_tokens = num_tokens;
    g.max_query_len = max_query_len;
    g.num_kv_heads = num_kv_heads;
    g.group = G;
    g.head_dim = head_dim;
    g.num_blocks = num_blocks;
    g.block_size = block_size;
    g.max_seq_len = max_seq_len;
    g.scale_log2 = a.scale_log2;
    // slot_of at the end of what the slots and lists take
    g.slot_of = reinterpret_cast<int*>(w + fit * slot) + 2 * fit + 2;
    a.slot_of = g.slot_of;
    if ((st = launch_q4_long(g, w, di.num_sms, s)) != KV_OK) return st;
  }
  if (head_dim == 128)
    return block_size == 32 ? launch_q4_nt<128, 32>(a, nt, s) : launch_q4_nt<128, 16>(a, nt, s);
  return block_size == 32 ? launch_q4_nt<64, 32>(a, nt, s) : launch_q4_nt<64, 16>(a, nt, s);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" {

size_t pagedkv_q4_record_bytes(int block_size, int head_dim) {
  if ((block_size != 16 && block_size != 32) || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)block_size * head_dim * 9 / 8;
}

size_t pagedkv_q4_long_workspace_bytes(int batch, int num_tokens, int max_query_len, int max_seq_len, int num_q_heads,
                                       int num_kv_heads, int head_dim) {
  const size_t few = pagedkv_q4_workspace_bytes(max_query_len, num_q_heads, num_kv_heads, head_dim);
  if (few == 0 || batch <= 0 || num_tokens <= 0 || max_seq_len <= 0) return few;
  const int slots = long_slots(batch, num_tokens, max_query_len, num_q_heads / num_kv_heads);
  if (slots == 0) return few;
  return few + 512 + slots * q4_slot_bytes(num_kv_heads, head_dim, max_seq_len) + q4_plan_bytes(batch, slots);
}

size_t pagedkv_q4_workspace_bytes(int max_query_len, int num_q_heads, int num_kv_heads, int head_dim) {
  if (max_query_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || head_dim <= 0)
    return 0;
  const int nt = column_tiles(max_query_len, num_q_heads / num_kv_heads);
  return q4_workspace(split_ctas(kMostSms, nt, num_kv_heads), num_kv_heads, nt, head_dim);
}

kv_status paged_attention_decode_q4(void* out, const void* q, const void* kv_cache, const int32_t* block_tables,
                                    int max_blocks_per_seq, const int32_t* seq_lens, int batch, int num_q_heads,
                                    int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                    int max_seq_len, float scale, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  return q4_common(out, q, kv_cache, block_tables, max_blocks_per_seq, seq_lens, nullptr, batch, batch, 1,
                   num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, max_seq_len, scale, workspace,
                   workspace_bytes, stream, false, "paged_attention_decode_q4");
}

kv_status paged_attention_multi_q4(void* out, const void* q, const void* kv_cache, const int32_t* block_tables,
                                   int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* query_start,
                                   int batch, int num_tokens, int max_query_len, int num_q_heads,
                                   int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                   int max_seq_len, float scale, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return q4_common(out, q, kv_cache, block_tables, max_blocks_per_seq, seq_lens, query_start, batch, num_tokens,
                   max_query_len, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, max_seq_len, scale,
                   workspace, workspace_bytes, stream, true, "paged_attention_multi_q4");
}

}  // extern "C"
