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
// A warp works on one token: its position, its slot and (R <= D) its part of the
// table's row are found once and serve all the rows (heads of q, k and v) it
// takes.  D / 16 lanes hold a row, each two runs of 8 elements that are each
// other's pairs, 16 bytes a load; a lane loads kRows rows before it works on
// the first.  Few tokens take one row per lane group (more warps, shorter
// chains), many take four.
//
// HBM bound: a prompt token of 32 + 8 + 8 heads of 128 moves 24 KB, against the
// 512 bytes of its table row, which L2 holds.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_q4.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kRotaryWarps = 4;
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
  int slices;                  // warps per token
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

// Eight bf16 of a row as fp32, and back (rounded to nearest).
__device__ __forceinline__ void widen8(const uint4& x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
  return make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]), pack2<false>(v[4], v[5]),
                    pack2<false>(v[6], v[7]));
}

template <bool kFp8>
__device__ __forceinline__ uint2 codes8(const uint4& x, float s) {
  float v[8];
  widen8(x, v);
  uint32_t o[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i / 4] |= (uint32_t)code8<kFp8>(v[i], s) << (8 * (i % 4));
  return make_uint2(o[0], o[1]);
}

// A row's two runs of 8 (elements 8 ca .. and 8 cb ..) as 4-bit codes under one
// (scale, min) per 64 elements, over the D / 16 lanes that hold the row:
//   min = the least value, scale = (largest - least) / 15 up to the next bf16
//   number (2^-126 at least), code = round((x - min) * (1 / scale)).
// NaN counts as 0, magnitudes above 2^126 as 2^126.  Every lane of the warp
// calls; lanes without `store` write nothing.
template <int D>
__device__ __forceinline__ void store_q4(bool store, unsigned char* rec, int x, int row, int bs, const uint4& ra,
                                         const uint4& rb, int ca, int cb, int sub) {
  constexpr int kGroups = D / 64, kLanes = D / 16;
  constexpr float kMost = 8.507059173023462e37f;   // 2^126
  float v[2][8];
  widen8(ra, v[0]);
  widen8(rb, v[1]);
  const int at[2] = {ca, cb};
  float lo[kGroups], hi[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    lo[g] = INFINITY;
    hi[g] = -INFINITY;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float l = INFINITY, h = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y = v[p][i];
      y = y != y ? 0.0f : fminf(fmaxf(y, -kMost), kMost);
      y = __fadd_rn(y, 0.0f);                       // -0 is 0
      v[p][i] = y;
      l = fminf(l, y);
      h = fmaxf(h, y);
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      if (at[p] / 8 == g) {
        lo[g] = fminf(lo[g], l);
        hi[g] = fmaxf(hi[g], h);
      }
  }
  float inv[kGroups];
  uint32_t pair[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) {
      lo[g] = fminf(lo[g], __shfl_xor_sync(0xffffffffu, lo[g], off));
      hi[g] = fmaxf(hi[g], __shfl_xor_sync(0xffffffffu, hi[g], off));
    }
    const float step = __fmul_rn(__fsub_rn(hi[g], lo[g]), 0.06666667014360428f);   // fp32 1 / 15
    const uint32_t up = (__float_as_uint(step) + 0xffffu) & 0xffff0000u;
    const float s = fmaxf(__uint_as_float(up), 1.1754943508222875e-38f);
    inv[g] = __fdiv_rn(1.0f, s);
    pair[g] = (__float_as_uint(s) >> 16) | (__float_as_uint(lo[g]) & 0xffff0000u);   // both bf16 already
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int g = at[p] / 8;
    const float low = kGroups > 1 && g ? lo[kGroups - 1] : lo[0], f = kGroups > 1 && g ? inv[kGroups - 1] : inv[0];
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = __float2int_rn(__fmul_rn(__fsub_rn(v[p][i], low), f));
      word |= (uint32_t)min(max(c, 0), 15) << (4 * i);
    }
    if (store) *reinterpret_cast<uint32_t*>(rec + q4_codes_at(x, row, bs, D) + ((at[p] & 7) * kGroups + g) * 4) = word;
  }
  if (store && sub < kGroups)
    *reinterpret_cast<uint32_t*>(rec + q4_pairs_at(x, row, bs, D) + sub * 4) = sub ? pair[kGroups - 1] : pair[0];
}

template <int D, int kKind, int kRows>
__global__ void __launch_bounds__(kRotaryWarps * 32) append_rotary_kernel(const RotaryArgs a, int bs) {
  constexpr int kLanes = D / 16, kPerWarp = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kRotaryWarps + (threadIdx.x >> 5);
  const int64_t tok = unit / a.slices;
  if (tok >= a.num_tokens) return;                  // (warp-uniform, as all below)
  const int t = (int)tok, slice = (int)(unit % a.slices);
  const int sub = lane % kLanes, row0 = (slice * kPerWarp + lane / kLanes) * kRows;
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
    const int r = row0 + i;
    xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    if (r >= rows) continue;
    const __nv_bfloat16* p = r < Hq          ? a.q + tok * a.q_stride + (int64_t)r * D
                             : r < Hq + Hkv ? a.k + tok * a.k_stride + (int64_t)(r - Hq) * D
                                            : a.v + tok * a.v_stride + (int64_t)(r - Hq - Hkv) * D;
    xa[i] = reinterpret_cast<const uint4*>(p)[ca];
    xb[i] = reinterpret_cast<const uint4*>(p)[cb];
  }

  // ---- the token's sequence, position and block --------------------------------
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
  const bool teller = slice == 0 && lane == 0;
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

  // ---- this lane's eight frequencies ----------------------------------------
  float co[8], si[8];
  if (R > 0 && use) {
    int where[kMaxAxes];
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) {
      where[x] = 0;
      if (x < a.axes) {
        where[x] = a.positions ? __ldg(a.positions + (int64_t)x * a.num_tokens + t) : pos;
        if (where[x] < 0 || where[x] >= a.max_position) {
          if (teller) atomicOr(a.flags, PAGEDKV_FLAG_BAD_INDEX);
          use = false;
        }
      }
    }
    if (use && turn) {
      const int j0 = 8 * sub;
      // the axis of frequency j: the first whose section ends behind it
      auto axis_of = [&](int j) {
        int x = 0;
#pragma unroll
        for (int k = 0; k < kMaxAxes - 1; ++k) x += k < a.axes - 1 && j >= a.section_end[k];
        return x;
      };
      auto at = [&](int x) {
        int w = where[0];
#pragma unroll
        for (int k = 1; k < kMaxAxes; ++k) w = x == k ? where[k] : w;
        return a.cos_sin + (int64_t)w * R;
      };
      const int xf = axis_of(j0), xl = axis_of(j0 + 7);
      if (xf == xl) {
        const float* p = at(xf) + j0;
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(p)), c1 = __ldg(reinterpret_cast<const float4*>(p) + 1);
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(p + half));
        const float4 s1 = __ldg(reinterpret_cast<const float4*>(p + half) + 1);
        co[0] = c0.x, co[1] = c0.y, co[2] = c0.z, co[3] = c0.w, co[4] = c1.x, co[5] = c1.y, co[6] = c1.z, co[7] = c1.w;
        si[0] = s0.x, si[1] = s0.y, si[2] = s0.z, si[3] = s0.w, si[4] = s1.x, si[5] = s1.y, si[6] = s1.z, si[7] = s1.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float* p = at(axis_of(j0 + i)) + j0 + i;
          co[i] = __ldg(p);
          si[i] = __ldg(p + half);
        }
      }
    }
  }

  // ---- rows ---------------------------------------------------------------------
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = row0 + i;
    const bool real = r < rows;
    const bool is_q = r < Hq, is_v = r >= Hq + Hkv;
    if (real && !is_v && use && turn) {
      float u[8], w[8];
      widen8(xa[i], u);
      widen8(xb[i], w);
      if (a.interleaved) {
        // pairs are neighbours: frequency k < 4 in the first run, the others in the second
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = u[2 * k], q = u[2 * k + 1];
          u[2 * k] = __fsub_rn(__fmul_rn(p, co[k]), __fmul_rn(q, si[k]));
          u[2 * k + 1] = __fadd_rn(__fmul_rn(q, co[k]), __fmul_rn(p, si[k]));
          const float y = w[2 * k], z = w[2 * k + 1];
          w[2 * k] = __fsub_rn(__fmul_rn(y, co[k + 4]), __fmul_rn(z, si[k + 4]));
          w[2 * k + 1] = __fadd_rn(__fmul_rn(z, co[k + 4]), __fmul_rn(y, si[k + 4]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float p = u[k], q = w[k];
          u[k] = __fsub_rn(__fmul_rn(p, co[k]), __fmul_rn(q, si[k]));
          w[k] = __fadd_rn(__fmul_rn(q, co[k]), __fmul_rn(p, si[k]));
        }
      }
      xa[i] = narrow8(u);
      xb[i] = narrow8(w);
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
        o[ca] = codes8<kFp8>(xa[i], s);
        o[cb] = codes8<kFp8>(xb[i], s);
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
  const int H = a.num_kv_heads, in = pos % bs;
  const int64_t base = (int64_t)blk * H;
#pragma unroll 4
  for (int i = lane; i < 2 * H * kWords; i += 32) {
    const int x = i >= H * kWords;                  // 0: K, 1: V
    const int hw = i - x * H * kWords, h = hw / kWords, e = hw % kWords;   // elements 8 e .. 8 e + 7
    uint4 o = make_uint4(0, 0, 0, 0);
    if (blk >= 0) {
      const unsigned char* rec = a.kv + (base + h) * (bs * D * 9 / 8);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + q4_codes_at(x, in, bs, D) +
                                                            ((e & 7) * kGroups + e / 8) * 4);
      const uint32_t p = *reinterpret_cast<const uint32_t*>(rec + q4_pairs_at(x, in, bs, D) + (e / 8) * 4);
      const float s = __uint_as_float(p << 16), m = __uint_as_float(p & 0xffff0000u);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(s, (float)((w >> (4 * k)) & 15u), m);   // s * c is exact
      o = narrow8(v);
    }
    (x ? a.v_out : a.k_out)[tok * H * kWords + hw] = o;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

template <int D, int kKind, int kRows>
kv_status launch_rotary(RotaryArgs& a, int bs, cudaStream_t s) {
  const int rows = (a.q_out ? a.num_q_heads : 0) + 2 * a.num_kv_heads;
  constexpr int kStep = 32 / (D / 16) * kRows;
  a.slices = (rows + kStep - 1) / kStep;
  const int64_t grid = ((int64_t)a.num_tokens * a.slices + kRotaryWarps - 1) / kRotaryWarps;
  if (grid > 0x7fffffffLL) return fail(KV_ERR_INVALID_ARG, "pagedkv_append_rotary: too many tokens");
  append_rotary_kernel<D, kKind, kRows><<<(unsigned)grid, kRotaryWarps * 32, 0, s>>>(a, bs);
  return cuda_check(cudaGetLastError(), "append_rotary_kernel launch");
}

template <int D, int kKind>
kv_status launch_rotary_rows(RotaryArgs& a, int bs, int sms, cudaStream_t s) {
  // four rows a lane group once that leaves eight warps per SM
  const int rows = (a.q_out ? a.num_q_heads : 0) + 2 * a.num_kv_heads;
  const int64_t warps = (int64_t)a.num_tokens * rows / (4 * 32 / (D / 16));
  return warps >= 8LL * sms ? launch_rotary<D, kKind, 4>(a, bs, s) : launch_rotary<D, kKind, 1>(a, bs, s);
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
