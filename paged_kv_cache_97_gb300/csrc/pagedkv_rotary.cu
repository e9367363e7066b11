// pagedkv_rotary.cu -- a step's queries and keys rotated by their positions and
// its keys and values stored, in one pass; the 4-bit pool's rows read back.
//
// For frequency j of a head's rotated part (R elements), with (c, s) the cosine
// and sine that the table has for j at the position of j's axis, the pair
// (x1, x2) = elements (j, j + R/2), or (2j, 2j + 1), becomes
//   (x1 c - x2 s, x2 c + x1 s)
// in fp32, every product and sum rounded once, then rounded to bf16.  A key is
// stored from that bf16 row by the pool's own rule, so the codes are those that
// a rotation followed by an append would give.
//
// A CTA works on one token (or a slice of its rows): its sequence, position, block
// and table row are found once and serve all rows (heads of q, k and v).  D / 16
// lanes hold a row, each two runs of 8 elements that are each other's pairs, 16
// bytes a load; a lane loads its up to four rows before it works on the first.
// Few tokens take one row per lane group (more CTAs, shorter chains).
//
// HBM bound: a prompt token of 32 + 8 + 8 heads of 128 moves 24 KB, against the
// 512 bytes of its table row, which L2 holds.  Measured (GB300), eight prompts of 1 to
// 8 K tokens: bf16 147 us, 93 % of the copy rate; E4M3 161 us (78 %); 4-bit with
// three position axes 187 us (64 %), the codes' arithmetic beside the loads, and
// reading them back 38 us (29 at the copy rate).  Eight CTAs per SM (64 registers)
// hide the chain sequence -> length -> block -> store: six took 170 us for bf16.  The
// table row is read once per CTA into shared memory; each thread's own loads of it for
// two axes spilled (387 us for 304 at that time).  128 single tokens 6 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_q4.cuh"
#include "pagedkv_requant.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kRotaryThreads = 128;
constexpr int kRotaryWarps = kRotaryThreads / 32;
constexpr int kMaxAxes = 4;
constexpr int kKindQ4 = 3;                          // beside the kv_dtype values

struct RotaryArgs {
  __nv_bfloat16* q_out;        // [T, Hq, D] at q_out_stride, or null: keys and values alone
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_out_stride, q_stride, k_stride, v_stride;   // elements from token to token
  void *k_cache, *v_cache;     // (4-bit: k_cache is the pool)
  const float *k_scale, *v_scale;
  const float* cos_sin;        // [max_position, R]: cosines, then sines; or null: no rotation
  const int32_t* positions;    // [axes, T], or null: the cache position
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start;  // [batch + 1], or null: one token per sequence
  unsigned int* flags;
  int max_position, rotary_dim, interleaved, axes;
  int section_end[kMaxAxes];   // frequencies below it belong to this axis or an earlier one
  int max_blocks, batch, num_tokens, max_query_len, num_q_heads, num_kv_heads, num_blocks;
  int slices;                  // CTAs per token
};

// The sequence of token t: the last b with query_start[b] <= t (32 samples a
// round), or -1.  Uniform over the warp.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ query_start, int batch, int t, int lane) {
  int lo = 0, hi = batch;                           // b in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int j = lo + lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, j < hi && __ldg(query_start + j) <= t);
    if (m == 0) return -1;
    const int last = 31 - __clz(m);
    lo += last * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// Eight fp32 as bf16 (rounded to nearest).
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
  return make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]), pack2<false>(v[4], v[5]),
                    pack2<false>(v[6], v[7]));
}

// Largest magnitude of 16 bf16 values, as bits (NaN above infinity above the finite).
__device__ __forceinline__ uint32_t magnitude_bits(const uint4& a, const uint4& b) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t m = max_u16x2(max_u16x2(a.x & kAbs, a.y & kAbs), max_u16x2(a.z & kAbs, a.w & kAbs));
  m = max_u16x2(m, max_u16x2(max_u16x2(b.x & kAbs, b.y & kAbs), max_u16x2(b.z & kAbs, b.w & kAbs)));
  return max(m & 0xffffu, m >> 16);
}

// The codes of 16 bf16 values under scale s, which the data did not set: the
// quotients may pass the largest code.  As code16 for values up to 2^40 (E4M3:
// the two corrections and a saturating conversion; int8: both ends of the
// interval held in -127 .. 127), by division above.
template <bool kFp8>
__device__ __forceinline__ uint4 codes16(const uint4& a, const uint4& b, const Interval& q, float s) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4], off = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
    bf16_values(w[2 * i], w[2 * i + 1], v);
    if constexpr (kFp8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float y = v[k] * q.r;
        y = fmaf(fmaf(y, q.s, -v[k]), -q.r, y);
        v[k] = fmaf(fmaf(y, q.s, -v[k]), -q.r, y);
      }
      o[i] = code4_times<true>(v, 1.0f);
    } else {
      float u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[k] = fminf(fmaxf(v[k] * q.lo, -127.0f), 127.0f);
        v[k] = fminf(fmaxf(v[k] * q.hi, -127.0f), 127.0f);
      }
      o[i] = code4_times<false>(u, 1.0f);
      off |= o[i] ^ code4_times<false>(v, 1.0f);
    }
  }
  if (q.on && off == 0u && magnitude_bits(a, b) <= 0x5380u) return make_uint4(o[0], o[1], o[2], o[3]);   // 2^40
  return code16_divided<kFp8>(a, b, s);
}

// Two fp32 numbers in one register pair.  A packed sum of packed products becomes
// a multiply-add in spite of its .rn, so what has to be rounded twice takes its
// products packed and its sums one by one.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// The bf16 pair of a word as fp32.
__device__ __forceinline__ F2 widen2(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
// The pairs (p, q) turned: p c - q s and q c + p s, as words of bf16.
__device__ __forceinline__ void turn2(F2 p, F2 q, F2 c, F2 s, uint32_t& pw, uint32_t& qw) {
  float a0, a1, b0, b1;
  split(mul2(p, c), a0, a1);
  split(mul2(q, s), b0, b1);
  pw = pack2<false>(__fsub_rn(a0, b0), __fsub_rn(a1, b1));
  split(mul2(q, c), a0, a1);
  split(mul2(p, s), b0, b1);
  qw = pack2<false>(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A row's two runs of 8 (elements 8 ca .. and 8 cb ..) as 4-bit codes under one
// (scale, min) per 64 elements, over the D / 16 lanes that hold the row:
//   min = the least value, scale = (largest - least) / 15 up to the next bf16
//   number (2^-126 at least), code = round((x - min) * (1 / scale)).
// NaN counts as 0, magnitudes above 2^126 as 2^126.  Every lane of the warp
// calls; lanes without `store` write nothing.
template <int D>
__device__ __forceinline__ void store_q4(bool store, unsigned char* rec, int x, int row, int bs, uint4 ra, uint4 rb,
                                         int ca, int cb, int sub) {
  constexpr int kGroups = D / 64, kLanes = D / 16;
  if (__any_sync(0xffffffffu, magnitude_bits(ra, rb) > 0x7e80u)) {       // NaN or above 2^126 (rare)
    uint32_t* w[2] = {&ra.x, &rb.x};
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo = w[p][i] & 0xffffu, hi = w[p][i] >> 16;
        lo = (lo & 0x7fffu) > 0x7f80u ? 0u : (lo & 0x7fffu) > 0x7e80u ? (lo & 0x8000u) | 0x7e80u : lo;
        hi = (hi & 0x7fffu) > 0x7f80u ? 0u : (hi & 0x7fffu) > 0x7e80u ? (hi & 0x8000u) | 0x7e80u : hi;
        w[p][i] = lo | hi << 16;
      }
  }
  // (min, min of the negated) of a run as a bf16 pair: one instruction and one
  // shuffle take both ends of two values
  auto ends = [](const uint4& r) {
    constexpr uint32_t kSign = 0x80008000u;
    const uint32_t lo = min_bf16x2(min_bf16x2(r.x, r.y), min_bf16x2(r.z, r.w));
    const uint32_t hi = min_bf16x2(min_bf16x2(r.x ^ kSign, r.y ^ kSign), min_bf16x2(r.z ^ kSign, r.w ^ kSign));
    return min_bf16x2(prmt(lo, hi, 0x5410u), prmt(lo, hi, 0x7632u));
  };
  const uint32_t ea = ends(ra), eb = ends(rb);
  float low[kGroups], inv[kGroups];
  uint32_t pair[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    constexpr uint32_t kNone = 0x7f807f80u;         // infinities
    uint32_t e = min_bf16x2(ca / 8 == g ? ea : kNone, cb / 8 == g ? eb : kNone);
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) e = min_bf16x2(e, __shfl_xor_sync(0xffffffffu, e, off));
    low[g] = __fadd_rn(__uint_as_float(e << 16), 0.0f);                  // -0 is 0
    const float high = -__uint_as_float(e & 0xffff0000u);
    const float step = __fmul_rn(__fsub_rn(high, low[g]), 0.06666667014360428f);   // fp32 1 / 15
    const uint32_t up = (__float_as_uint(step) + 0xffffu) & 0xffff0000u;
    const float s = fmaxf(__uint_as_float(up), 1.1754943508222875e-38f);
    inv[g] = __frcp_rn(s);
    pair[g] = (__float_as_uint(s) >> 16) | (__float_as_uint(low[g]) & 0xffff0000u);   // both bf16 already
  }
  const uint4 r[2] = {ra, rb};
  const int at[2] = {ca, cb};
  uint32_t word[2] = {0u, 0u};
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int g = at[p] / 8;
    const float lo = kGroups > 1 && g ? low[kGroups - 1] : low[0], f = kGroups > 1 && g ? inv[kGroups - 1] : inv[0];
    const uint32_t w[4] = {r[p].x, r[p].y, r[p].z, r[p].w};
    // y = (x - min) / scale is in [0, 15] but for a last place: added to 2^23 its
    // nearest integer (ties to even) stands in the low bits, and the words of eight,
    // times 16^i, add up to the codes and a constant
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 y = mul2(add2(widen2(w[i]), f2(-lo, -lo)), f2(f, f));
      float c0, c1;
      split(y, c0, c1);
      word[p] += (__float_as_uint(__fadd_rn(c0, 8388608.0f)) << (8 * i)) +
                 (__float_as_uint(__fadd_rn(c1, 8388608.0f)) << (8 * i + 4));
    }
    // 0x4B000000 * (1 + 16 + .. + 16^7) mod 2^32
    word[p] -= 0x4B000000u * 0x11111111u;
  }
  if (store) {
    unsigned char* to = rec + q4_codes_at(x, row, bs, D);
    if (kGroups == 2 && ca + 8 == cb) {             // the same word of both groups: neighbours
      *reinterpret_cast<uint2*>(to + ca * 8) = make_uint2(word[0], word[1]);
    } else {
      *reinterpret_cast<uint32_t*>(to + ((ca & 7) * kGroups + ca / 8) * 4) = word[0];
      *reinterpret_cast<uint32_t*>(to + ((cb & 7) * kGroups + cb / 8) * 4) = word[1];
    }
  }
  if (store && sub < kGroups)
    *reinterpret_cast<uint32_t*>(rec + q4_pairs_at(x, row, bs, D) + sub * 4) =
        kGroups > 1 && sub ? pair[kGroups - 1] : pair[0];
}

template <int D, int kKind, int kRows>
__global__ void __launch_bounds__(kRotaryThreads, kRows <= 3 ? 8 : 6) append_rotary_kernel(const RotaryArgs a, int bs) {
  constexpr int kLanes = D / 16, kStep = kRotaryThreads / kLanes;        // rows taken side by side
  __shared__ __align__(16) float table[128];        // the token's cosines, then its sines
  const int lane = threadIdx.x & 31;
  const int64_t tok = blockIdx.x / a.slices;
  const int t = (int)tok, slice = blockIdx.x % a.slices;
  const int sub = lane % kLanes, row0 = slice * kStep * kRows + threadIdx.x / kLanes;
  const int Hq = a.q_out ? a.num_q_heads : 0, Hkv = a.num_kv_heads;
  const int rows = Hq + 2 * Hkv;
  const int R = a.cos_sin ? a.rotary_dim : 0, half = R / 2;

  // this lane's two runs: each other's pairs where rotated, else neighbours
  const bool turn = sub < R / 16;
  int ca, cb;                                       // in runs of 8 elements
  if (!turn) {
    ca = R / 8 + 2 * (sub - R / 16);
    cb = ca + 1;
  } else if (a.interleaved) {
    ca = 2 * sub;
    cb = ca + 1;
  } else {
    ca = sub;
    cb = sub + half / 8;
  }

  // rows are loaded before the sequence is known: the loads need the token alone
  uint4 xa[kRows], xb[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i * kStep;
    xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    if (r >= rows) continue;
    const __nv_bfloat16* p = r < Hq          ? a.q + tok * a.q_stride + (int64_t)r * D
                             : r < Hq + Hkv ? a.k + tok * a.k_stride + (int64_t)(r - Hq) * D
                                            : a.v + tok * a.v_stride + (int64_t)(r - Hq - Hkv) * D;
    xa[i] = reinterpret_cast<const uint4*>(p)[ca];
    xb[i] = reinterpret_cast<const uint4*>(p)[cb];
  }

  // ---- the token's sequence, position and block (uniform over the CTA) -----------
  int b = t, n = 1, q0 = t;
  if (a.query_start) {
    b = sequence_of(a.query_start, a.batch, t, lane);
    if (b < 0) return;                              // a row of no sequence: left as it is
    q0 = __ldg(a.query_start + b);
    n = __ldg(a.query_start + b + 1) - q0;
    if (t < q0 || t - q0 >= n) return;
  }
  const int L = __ldg(a.seq_lens + b);
  bool use = true, kv_ok = true;
  const bool teller = slice == 0 && threadIdx.x == 0;
  if (L <= 0 || q0 < 0 || q0 > a.num_tokens - n || n > L || n > a.max_query_len || (L - 1) / bs >= a.max_blocks) {
    if (teller) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
    use = false;
  }
  const int pos = L - n + (t - q0);
  int blk = 0;
  if (use) {
    blk = __ldg(a.block_tables + (int64_t)b * a.max_blocks + pos / bs);
    if (blk < 0 || blk >= a.num_blocks) {
      if (teller) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
      kv_ok = false;
    }
  }
  const int in = pos % bs;

  // ---- the token's table row, each frequency from its own axis's position ---------
  if (R > 0) {
    bool lost = false;
    if (use && (int)threadIdx.x < R) {
      const int j = threadIdx.x < half ? threadIdx.x : threadIdx.x - half;
      int x = 0;                                    // the first axis whose section ends behind j
#pragma unroll
      for (int k = 0; k < kMaxAxes - 1; ++k) x += k < a.axes - 1 && j >= a.section_end[k];
      const int at = a.positions ? __ldg(a.positions + (int64_t)x * a.num_tokens + t) : pos;
      lost = at < 0 || at >= a.max_position;
      if (!lost) table[threadIdx.x] = __ldg(a.cos_sin + (int64_t)at * R + threadIdx.x);
    }
    if (__syncthreads_or(lost)) {
      if (teller) atomicOr(a.flags, PAGEDKV_FLAG_BAD_INDEX);
      use = false;
    }
  }
  float co[8], si[8];
  if (turn) {
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const float4 y = *reinterpret_cast<const float4*>(table + 8 * sub + k);
      const float4 z = *reinterpret_cast<const float4*>(table + half + 8 * sub + k);
      co[k] = y.x, co[k + 1] = y.y, co[k + 2] = y.z, co[k + 3] = y.w;
      si[k] = z.x, si[k + 1] = z.y, si[k + 2] = z.z, si[k + 3] = z.w;
    }
  }

  // ---- rows ---------------------------------------------------------------------
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i * kStep;
    const bool real = r < rows;
    const bool is_q = r < Hq, is_v = r >= Hq + Hkv;
    if (real && !is_v && use && turn) {
      uint32_t u[4] = {xa[i].x, xa[i].y, xa[i].z, xa[i].w}, w[4] = {xb[i].x, xb[i].y, xb[i].z, xb[i].w};
      if (a.interleaved) {
        // pairs are neighbours: frequency k < 4 in the first run, the others in the second
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const F2 c = f2(co[k], co[k + 4]), s = f2(si[k], si[k + 4]);
          const F2 p = f2(__uint_as_float(u[k] << 16), __uint_as_float(w[k] << 16));
          const F2 q = f2(__uint_as_float(u[k] & 0xffff0000u), __uint_as_float(w[k] & 0xffff0000u));
          uint32_t pw, qw;                          // (first run's, second run's)
          turn2(p, q, c, s, pw, qw);
          u[k] = prmt(pw, qw, 0x5410u);
          w[k] = prmt(pw, qw, 0x7632u);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          turn2(widen2(u[k]), widen2(w[k]), f2(co[2 * k], co[2 * k + 1]), f2(si[2 * k], si[2 * k + 1]),
                u[k], w[k]);
      }
      xa[i] = make_uint4(u[0], u[1], u[2], u[3]);
      xb[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (real && is_q) {
      uint4* o = reinterpret_cast<uint4*>(a.q_out + tok * a.q_out_stride + (int64_t)r * D);
      o[ca] = use ? xa[i] : make_uint4(0, 0, 0, 0);
      o[cb] = use ? xb[i] : make_uint4(0, 0, 0, 0);
    }
    const bool store = real && !is_q && use && kv_ok;
    const int h = is_v ? r - Hq - Hkv : r - Hq;
    if constexpr (kKind == kKindQ4) {
      // (the reduction runs over a row's lanes: every lane of the warp takes part)
      if (__any_sync(0xffffffffu, store)) {
        unsigned char* rec = static_cast<unsigned char*>(a.k_cache) +
                             ((int64_t)(store ? blk : 0) * Hkv + (store ? h : 0)) * (bs * D * 9 / 8);
        store_q4<D>(store, rec, is_v, in, bs, xa[i], xb[i], ca, cb, sub);
      }
    } else if (store) {
      const int64_t dst = (((int64_t)blk * bs + in) * Hkv + h) * D;
      void* cache = is_v ? a.v_cache : a.k_cache;
      if constexpr (kKind == KV_DTYPE_BF16) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + dst);
        o[ca] = xa[i];
        o[cb] = xb[i];
      } else {
        constexpr bool kFp8 = kKind == KV_DTYPE_FP8_E4M3;
        const float s = __ldg((is_v ? a.v_scale : a.k_scale) + (int64_t)blk * Hkv + h);
        uint2* o = reinterpret_cast<uint2*>(static_cast<unsigned char*>(cache) + dst);
        const uint4 y = codes16<kFp8>(xa[i], xb[i], quotients(s), s);
        o[ca] = make_uint2(y.x, y.y);
        o[cb] = make_uint2(y.z, y.w);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The 4-bit pool's rows as values: min + scale * code in fp32, rounded to bf16.
// One warp per token; a lane takes eight elements (one code word, its group's
// pair, 16 bytes out) at a time.
// ---------------------------------------------------------------------------

struct ReadArgs {
  uint4 *k_out, *v_out;        // bf16 [T, Hkv, D]
  const unsigned char* kv;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start;
  unsigned int* flags;
  int max_blocks, batch, num_tokens, max_query_len, num_kv_heads, num_blocks;
};

template <int D>
__global__ void __launch_bounds__(kRotaryWarps * 32) read_q4_kernel(const ReadArgs a, int bs) {
  constexpr int kGroups = D / 64, kWords = D / 8;
  const int lane = threadIdx.x & 31;
  const int64_t tok = (int64_t)blockIdx.x * kRotaryWarps + (threadIdx.x >> 5);
  if (tok >= a.num_tokens) return;
  const int t = (int)tok;
  int b = t, n = 1, q0 = t;
  if (a.query_start) {
    b = sequence_of(a.query_start, a.batch, t, lane);
    if (b < 0) return;
    q0 = __ldg(a.query_start + b);
    n = __ldg(a.query_start + b + 1) - q0;
    if (t < q0 || t - q0 >= n) return;
  }
  const int L = __ldg(a.seq_lens + b);
  const int pos = L - n + (t - q0);
  int blk = -1;
  if (L <= 0 || q0 < 0 || q0 > a.num_tokens - n || n > L || n > a.max_query_len || (L - 1) / bs >= a.max_blocks) {
    if (lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
  } else {
    blk = __ldg(a.block_tables + (int64_t)b * a.max_blocks + pos / bs);
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
      blk = -1;
    }
  }
  // lane: word `e` of heads h0, h0 + 32 / kWords, .. ; elements 8 e .. 8 e + 7
  constexpr int kSide = 32 / kWords;
  const int H = a.num_kv_heads, in = pos % bs, rec_bytes = bs * D * 9 / 8;
  const int e = lane % kWords, h0 = lane / kWords;
  const unsigned char* block = a.kv + (int64_t)(blk >= 0 ? blk : 0) * H * rec_bytes;
  uint4* out[2] = {a.k_out + tok * H * kWords, a.v_out + tok * H * kWords};
  int word_at[2], pair_at[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    word_at[x] = q4_codes_at(x, in, bs, D) + ((e & 7) * kGroups + e / 8) * 4;
    pair_at[x] = q4_pairs_at(x, in, bs, D) + (e / 8) * 4;
  }
  constexpr int kBatch = 4;                         // heads whose K and V words are asked for together
  for (int h1 = h0; h1 < H; h1 += kBatch * kSide) {
    uint32_t w[kBatch][2], p[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h1 + i * kSide;
      const unsigned char* rec = block + (int64_t)h * rec_bytes;
      const bool live = blk >= 0 && h < H;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        w[i][x] = live ? __ldg(reinterpret_cast<const uint32_t*>(rec + word_at[x])) : 0u;
        p[i][x] = live ? __ldg(reinterpret_cast<const uint32_t*>(rec + pair_at[x])) : 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h1 + i * kSide;
      if (h >= H) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float s = __uint_as_float(p[i][x] << 16), m = __uint_as_float(p[i][x] & 0xffff0000u);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)                 // c: the low bits of 2^23 + c; s * c is exact
          v[k] = fmaf(s, __uint_as_float(0x4B000000u | (w[i][x] >> (4 * k) & 15u)) - 8388608.0f, m);
        out[x][h * kWords + e] = narrow8(v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

template <int D, int kKind, int kRows>
kv_status launch_rotary(RotaryArgs& a, int bs, cudaStream_t s) {
  const int rows = (a.q_out ? a.num_q_heads : 0) + 2 * a.num_kv_heads;
  constexpr int kStep = kRotaryThreads / (D / 16) * kRows;
  a.slices = (rows + kStep - 1) / kStep;
  const int64_t grid = (int64_t)a.num_tokens * a.slices;
  if (grid > 0x7fffffffLL) return fail(KV_ERR_INVALID_ARG, "pagedkv_append_rotary: too many tokens");
  append_rotary_kernel<D, kKind, kRows><<<(unsigned)grid, kRotaryThreads, 0, s>>>(a, bs);
  return cuda_check(cudaGetLastError(), "append_rotary_kernel launch");
}

template <int D, int kKind>
kv_status launch_rotary_rows(RotaryArgs& a, int bs, int sms, cudaStream_t s) {
  // up to four rows a lane group once that leaves two CTAs per SM
  constexpr int kStep = kRotaryThreads / (D / 16);
  const int rows = (a.q_out ? a.num_q_heads : 0) + 2 * a.num_kv_heads;
  const int64_t most = (int64_t)a.num_tokens * ((rows + 4 * kStep - 1) / (4 * kStep));
  if (most < 2LL * sms) return launch_rotary<D, kKind, 1>(a, bs, s);
  // the fewest rows a group that take a token in as few CTAs
  const int per = (rows + kStep - 1) / kStep;
  if (per <= 2) return launch_rotary<D, kKind, 2>(a, bs, s);
  return per == 3 ? launch_rotary<D, kKind, 3>(a, bs, s) : launch_rotary<D, kKind, 4>(a, bs, s);
}

template <int D>
kv_status launch_rotary_kind(RotaryArgs& a, int kind, int bs, int sms, cudaStream_t s) {
  if (kind == kKindQ4) return launch_rotary_rows<D, kKindQ4>(a, bs, sms, s);
  if (kind == KV_DTYPE_INT8) return launch_rotary_rows<D, KV_DTYPE_INT8>(a, bs, sms, s);
  if (kind == KV_DTYPE_FP8_E4M3) return launch_rotary_rows<D, KV_DTYPE_FP8_E4M3>(a, bs, sms, s);
  return launch_rotary_rows<D, KV_DTYPE_BF16>(a, bs, sms, s);
}

bool good_stride(int64_t stride, int heads, int head_dim) {
  return stride % 8 == 0 && stride >= (int64_t)heads * head_dim;
}

kv_status rotary_common(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, void* k_cache, void* v_cache,
                        const float* k_scale, const float* v_scale, const float* cos_sin, int max_position,
                        int rotary_dim, int interleaved, const int32_t* positions, int num_axes,
                        const int32_t* axis_sections, const int32_t* block_tables, int max_blocks,
                        const int32_t* seq_lens, const int32_t* query_start, int batch, int num_tokens,
                        int max_query_len, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                        int block_size, int kind, void* stream, const char* who) {
  if (batch < 0 || num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks <= 0 ||
      max_query_len <= 0)
    return fail(KV_ERR_INVALID_ARG, "%s: bad sizes", who);
  if ((q && num_q_heads > (1 << 24)) || num_kv_heads > (1 << 24))
    return fail(KV_ERR_INVALID_ARG, "%s: at most 2^24 heads", who);
  if (head_dim != 64 && head_dim != 128) return fail(KV_ERR_INVALID_ARG, "%s: head_dim must be 64 or 128", who);
  if (block_size != 16 && block_size != 32) return fail(KV_ERR_INVALID_ARG, "%s: block_size must be 16 or 32", who);
  if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && num_q_heads == 0))
    return fail(KV_ERR_INVALID_ARG, "%s: q, q_out and num_q_heads belong together", who);
  RotaryArgs a = {};
  if (cos_sin) {
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 || max_position <= 0)
      return fail(KV_ERR_INVALID_ARG, "%s: rotary_dim must be a multiple of 16 up to head_dim, max_position positive", who);
    if (num_axes < 1 || num_axes > kMaxAxes || (num_axes > 1 && (!positions || !axis_sections)))
      return fail(KV_ERR_INVALID_ARG, "%s: 1 to %d axes, several with positions and sections", who, kMaxAxes);
    int64_t end = 0;
    for (int x = 0; x < num_axes; ++x) {
      const int64_t size = axis_sections ? axis_sections[x] : rotary_dim / 2;
      if (size < 0) return fail(KV_ERR_INVALID_ARG, "%s: a negative section", who);
      end += size;
      a.section_end[x] = (int)(end < rotary_dim ? end : rotary_dim);
    }
    if (end != rotary_dim / 2)
      return fail(KV_ERR_INVALID_ARG, "%s: the sections must add up to rotary_dim / 2", who);
  }
  if (batch == 0 || num_tokens == 0) return KV_OK;
  if (!k || !v || !k_cache || (kind != kKindQ4 && !v_cache) || !block_tables || !seq_lens)
    return fail(KV_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!query_start && num_tokens != batch)
    return fail(KV_ERR_INVALID_ARG, "%s: without query_start there is one token per sequence", who);
  if (!aligned16(q_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(cos_sin))
    return fail(KV_ERR_INVALID_ARG, "%s: rows, table and pools must be 16-byte aligned", who);
  if ((q && (!good_stride(q_stride, num_q_heads, head_dim) || !good_stride(q_out_stride, num_q_heads, head_dim))) ||
      !good_stride(k_stride, num_kv_heads, head_dim) || !good_stride(v_stride, num_kv_heads, head_dim))
    return fail(KV_ERR_INVALID_ARG, "%s: token strides must be multiples of 8 elements that hold a token's heads", who);
  if (q && q == q_out && q_stride != q_out_stride)
    return fail(KV_ERR_INVALID_ARG, "%s: rotating in place needs equal strides", who);
  const bool scaled = kind == KV_DTYPE_INT8 || kind == KV_DTYPE_FP8_E4M3;
  if (scaled != (k_scale != nullptr) || scaled != (v_scale != nullptr))
    return fail(KV_ERR_INVALID_ARG, "%s: 8-bit pools need k_scale and v_scale, others take NULL", who);
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_out_stride = q_out_stride;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.flags = di.flags;
  a.max_position = max_position;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved != 0;
  a.axes = num_axes;
  a.max_blocks = max_blocks;
  a.batch = batch;
  a.num_tokens = num_tokens;
  a.max_query_len = max_query_len;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  cudaStream_t s = (cudaStream_t)stream;
  return head_dim == 128 ? launch_rotary_kind<128>(a, kind, block_size, di.num_sms, s)
                         : launch_rotary_kind<64>(a, kind, block_size, di.num_sms, s);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" {

kv_status pagedkv_append_rotary(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride, void* k_cache, void* v_cache,
                                const float* k_scale, const float* v_scale, const float* cos_sin, int max_position,
                                int rotary_dim, int interleaved, const int32_t* positions, int num_axes,
                                const int32_t* axis_sections, const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* seq_lens, const int32_t* query_start, int batch, int num_tokens,
                                int max_query_len, int num_q_heads, int num_kv_heads, int head_dim, int num_blocks,
                                int block_size, kv_dtype dtype, void* stream) {
  if (!valid_dtype(dtype)) return fail(KV_ERR_INVALID_ARG, "pagedkv_append_rotary: bad dtype");
  return rotary_common(q_out, q_out_stride, q, q_stride, k, k_stride, v, v_stride, k_cache, v_cache, k_scale, v_scale,
                       cos_sin, max_position, rotary_dim, interleaved, positions, num_axes, axis_sections,
                       block_tables, max_blocks_per_seq, seq_lens, query_start, batch, num_tokens, max_query_len,
                       num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, (int)dtype, stream,
                       "pagedkv_append_rotary");
}

kv_status pagedkv_append_rotary_q4(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* v, int64_t v_stride, void* kv_cache,
                                   const float* cos_sin, int max_position, int rotary_dim, int interleaved,
                                   const int32_t* positions, int num_axes, const int32_t* axis_sections,
                                   const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                   const int32_t* query_start, int batch, int num_tokens, int max_query_len,
                                   int num_q_heads, int num_kv_heads, int head_dim, int num_blocks, int block_size,
                                   void* stream) {
  return rotary_common(q_out, q_out_stride, q, q_stride, k, k_stride, v, v_stride, kv_cache, nullptr, nullptr, nullptr,
                       cos_sin, max_position, rotary_dim, interleaved, positions, num_axes, axis_sections,
                       block_tables, max_blocks_per_seq, seq_lens, query_start, batch, num_tokens, max_query_len,
                       num_q_heads, num_kv_heads, head_dim, num_blocks, block_size, kKindQ4, stream,
                       "pagedkv_append_rotary_q4");
}

kv_status pagedkv_read_q4(void* k_out, void* v_out, const void* kv_cache, const int32_t* block_tables,
                          int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* query_start, int batch,
                          int num_tokens, int max_query_len, int num_kv_heads, int head_dim, int num_blocks,
                          int block_size, void* stream) {
  const char* who = "pagedkv_read_q4";
  if (batch < 0 || num_tokens < 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 ||
      max_query_len <= 0 || (head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32) ||
      num_kv_heads > (1 << 24))
    return fail(KV_ERR_INVALID_ARG, "%s: bad sizes (head_dim 64 or 128, block_size 16 or 32)", who);
  if (batch == 0 || num_tokens == 0) return KV_OK;
  if (!k_out || !v_out || !kv_cache || !block_tables || !seq_lens)
    return fail(KV_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(kv_cache))
    return fail(KV_ERR_INVALID_ARG, "%s: the outputs and the pool must be 16-byte aligned", who);
  if (!query_start && num_tokens != batch)
    return fail(KV_ERR_INVALID_ARG, "%s: without query_start there is one token per sequence", who);
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  ReadArgs a = {};
  a.k_out = static_cast<uint4*>(k_out);
  a.v_out = static_cast<uint4*>(v_out);
  a.kv = static_cast<const unsigned char*>(kv_cache);
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start = query_start;
  a.flags = di.flags;
  a.max_blocks = max_blocks_per_seq;
  a.batch = batch;
  a.num_tokens = num_tokens;
  a.max_query_len = max_query_len;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  const unsigned grid = (unsigned)(((int64_t)num_tokens + kRotaryWarps - 1) / kRotaryWarps);
  cudaStream_t s = (cudaStream_t)stream;
  if (head_dim == 128) read_q4_kernel<128><<<grid, kRotaryWarps * 32, 0, s>>>(a, block_size);
  else read_q4_kernel<64><<<grid, kRotaryWarps * 32, 0, s>>>(a, block_size);
  return cuda_check(cudaGetLastError(), "read_q4_kernel launch");
}

}  // extern "C"
