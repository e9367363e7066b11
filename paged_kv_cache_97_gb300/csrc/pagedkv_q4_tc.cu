// pagedkv_q4_tc.cu -- attention of long queries (prompts, chunks of them) over
// the 4-bit pool on tcgen05 with TMEM accumulators.
//
// 256 rows (query token x grouped head) of a sequence share every key, so the
// codes are widened once per call instead of once per row tile: a first kernel
// writes, for every sequence with long queries and KV head, the rows of each 128
// keys as two fp16 operand images (K and V, 128-byte-swizzled bands of 64
// elements, exactly as the tensor core reads them), each under one power of two
// that puts its largest magnitude in [2^12, 2^13).  A value is then within 2^-11
// of itself, or 2^-37 of the largest of its 128 rows.  The attention kernel loads
// an image with one bulk copy; K's power multiplies the scores, V's goes into the
// softmax's reference: with s a score in base 2 and E the chunk's power,
//   p = 2^(s + E - m),  O += p V / 2^E,  l += p / 2^E,  out = O / l,
// m at most the row's largest s + E less five, so that p as an fp16 number is
// within 2^-11 of itself, or 2^-30 of the row's largest.
//
// Images cost 4 d bytes per token and KV head written once and read by every 256
// rows.
//
// What bounds it: the two row tiles of a CTA take turns on the tensor pipe, and a
// tile's chunk is a chain: its scores and P . V (1024 cycles of MMA), the softmax of a
// row per thread (1600) and the hand-overs (350), in all 2650 cycles for two tiles'
// 2048 of MMA, so the pipe is busy 3 / 4 of the time inside a unit.  Around it a
// unit ends with 3000 cycles for its rows and 3000 for the next one's queries.
// Measured (GB300, 32 / 8 heads of 128): one prompt of 8192 tokens 405 us, 1358
// TFLOP/s; four of 1.5 to 3.5 K 208 us, 1034 TFLOP/s (plan 3, images 14, attention
// 180, and 5 for the kernels of short queries that find nothing); 512 tokens over 8192
// 133 us (64 units for 152 SMs).
// What made it fast, the prompt of 8192 (the four): MMAs issued by a whole warp, one
// elected lane (operands in uniform registers; a divergent lane needs 100 cycles
// per step of K 16 for the pipe's 64) 549 -> 487 us (316 -> 290); roles that walk the
// units at their own pace 471 (278); P . V that begins with the first half of P
// 446 (270); units by length, launches that overlap 454 (260); one form of the
// softmax, rolled, masks beforehand: code that runs once a unit is fetched from far
// away, 416 (221); queries turned four rows side by side 412 (215); the images
// written 64 bytes at a time 406 (209).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"
#include "pagedkv_q4.cuh"
#include "pagedkv_tc.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kRows = 128;                // query rows per tile (the MMA's M)
constexpr int kTiles = 2;                 // row tiles per CTA, computed in ping-pong
constexpr int kChunk = 128;               // keys per chunk
constexpr int kKStages = 2, kVStages = 3; // V is released later than K
constexpr int kSoftmaxWarps = 4 * kTiles; // one row per thread
constexpr int kMmaWarp = kSoftmaxWarps, kKWarp = kMmaWarp + 1, kVWarp = kMmaWarp + 2;
constexpr int kUnitWarp = kMmaWarp + 3;
constexpr int kThreadsTc = (kUnitWarp + 1) * 32;
constexpr int kTmemCols = 512;            // the whole TMEM: one CTA per SM
constexpr float kSlack = 8.0f;            // octaves a row may pass its reference by
constexpr float kHead = 5.0f;             // octaves above 1 a reference leaves p
constexpr float kFar = 100.0f;            // octaves below its reference where a weight is summed by itself

template <int D>
struct Img {
  static constexpr int kBytes = kChunk * D * 2;          // K (or V) of a chunk; Q of a tile
  static constexpr int kUsed = (kTiles + kKStages + kVStages) * kBytes + 1024;
  // at least 120 KB, so that two CTAs never share an SM (each takes the whole TMEM)
  static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  __host__ __device__ static constexpr uint32_t ocol(int g) { return (uint32_t)(g * D); }
  __host__ __device__ static constexpr uint32_t scol(int g) { return (uint32_t)(2 * D + 128 * g); }
};

// ---------------------------------------------------------------------------
// Plan: the sequences with long queries, as many as have images
// ---------------------------------------------------------------------------

__device__ __forceinline__ bool long_sequence(const Q4LongArgs& a, int b) {
  const int q0 = a.query_start[b], q1 = a.query_start[b + 1], n = q1 - q0, L = a.seq_lens[b];
  return q0 >= 0 && n > 0 && q1 <= a.num_tokens && L > 0 && L <= a.max_seq_len &&
         (L - 1) / a.block_size < a.max_blocks && n <= L && n <= a.max_query_len &&
         (int64_t)n * a.group >= kLongRows;
}

__global__ void __launch_bounds__(256) q4_plan_kernel(const Q4LongArgs a) {
  __shared__ int sums[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (each launch is a programmatic dependent of the one before and waits for it here)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int run = (a.batch + 255) / 256;
  const int b0 = threadIdx.x * run, b1 = min(a.batch, b0 + run);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += long_sequence(a, b);
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int rank = incl - mine, total = 0;
  for (int w = 0; w < 8; ++w) {
    if (w < warp) rank += sums[w];
    total += sums[w];
  }
  for (int b = b0; b < b1; ++b) {
    int slot = -1;
    if (long_sequence(a, b)) {
      if (rank < a.slots) {
        slot = rank;
        a.list[rank] = b;
        a.bad[rank] = 0;
      }
      ++rank;
    }
    a.slot_of[b] = slot;
  }
  if (threadIdx.x == 0) {
    a.counters[0] = min(total, a.slots);
    a.counters[1] = 0;                              // units taken
  }
}

// ---------------------------------------------------------------------------
// Images
// ---------------------------------------------------------------------------

template <int D, int BS>
__global__ void __launch_bounds__(256) q4_widen_kernel(const Q4LongArgs a) {
  using G = Geo4<D, BS>;
  constexpr int NG = G::kGroups;
  __shared__ unsigned int top[2];
  __shared__ int32_t blk[kChunk / 16];
  __shared__ int any_bad;
  const int c = blockIdx.x, hk = blockIdx.y, slot = blockIdx.z;
  if (threadIdx.x < 2) top[threadIdx.x] = 0;
  if (threadIdx.x == 0) any_bad = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (slot >= a.counters[0]) return;
  const int b = a.list[slot], L = a.seq_lens[b];
  const int t0 = c * kChunk, rows = min(kChunk, L - t0);
  if (rows <= 0) return;
  __syncthreads();
  if (threadIdx.x < kChunk / BS && (int)threadIdx.x * BS < rows) {
    const int id = a.block_tables[(int64_t)b * a.max_blocks + t0 / BS + threadIdx.x];
    const bool ok = id >= 0 && id < a.num_blocks;
    if (!ok) any_bad = 1;
    blk[threadIdx.x] = ok ? id : 0;
  }
  __syncthreads();
  if (any_bad) {
    if (threadIdx.x == 0) {
      a.bad[slot] = 1;
      atomicOr(a.flags, PAGEDKV_FLAG_BAD_BLOCK);
    }
    return;
  }
  // Four lanes have a row (words t and t + 4 of every group each, so that they write
  // 64 bytes of the image together), a thread four rows, all asked for at once.
  constexpr int kTurns = kChunk / 32;
  const int x = threadIdx.x >> 7;                   // 0: K, 1: V
  const int w4 = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t w[kTurns][2 * NG], pair[kTurns][NG];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int r = i * 32 + w4 * 8 + g;
#pragma unroll
    for (int k = 0; k < 2 * NG; ++k) w[i][k] = 0;
#pragma unroll
    for (int k = 0; k < NG; ++k) pair[i][k] = 0;
    if (r < rows) {
      const unsigned char* rec = a.kv + ((int64_t)blk[r / BS] * a.num_kv_heads + hk) * G::kRecord;
      const unsigned char* from = rec + q4_codes_at(x, r % BS, BS, D) + t * (4 * NG);
#pragma unroll
      for (int ci = 0; ci < 2; ++ci) {
        if constexpr (NG == 2) {
          const uint2 y = __ldg(reinterpret_cast<const uint2*>(from + ci * 32));
          w[i][2 * ci] = y.x, w[i][2 * ci + 1] = y.y;
        } else {
          w[i][ci] = __ldg(reinterpret_cast<const uint32_t*>(from + ci * 16));
        }
      }
#pragma unroll
      for (int k = 0; k < NG; ++k)
        pair[i][k] = __ldg(reinterpret_cast<const uint32_t*>(rec + q4_pairs_at(x, r % BS, BS, D)) + k);
    }
  }
  // the largest magnitude of the rows: a group's values lie between min and min + 15 scale
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const float s = __uint_as_float(pair[i][k] << 16), lo = __uint_as_float(pair[i][k] & 0xffff0000u);
      m = fmaxf(m, fmaxf(fabsf(lo), fabsf(fmaf(15.0f, s, lo))));
    }
  }
  const unsigned int u = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
  if (lane == 0) atomicMax(&top[x], u);
  __syncthreads();
  // value * 2^-e is at most [2^12, 2^13) (|value| < 2^128); -80 keeps the sums of
  // p / 2^E within fp32
  const int e = min(max((int)(top[x] >> 23) - 127 - 12, -80), 115);
  const int64_t cell = ((int64_t)slot * a.num_kv_heads + hk) * a.chunks + c;
  if ((threadIdx.x & 127) == 0) reinterpret_cast<int*>(a.exps + cell)[x] = e;
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
  unsigned char* img = a.images + (cell * 2 + x) * Img<D>::kBytes;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int r = i * 32 + w4 * 8 + g;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const float s = __uint_as_float(pair[i][gr] << 16) * f, lo = __uint_as_float(pair[i][gr] & 0xffff0000u) * f;
#pragma unroll
      for (int ci = 0; ci < 2; ++ci) {
        const uint32_t y = w[i][ci * NG + gr];
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // c as fp32: the low bits of 2^23 + c
          const float c0 = __uint_as_float(0x4B000000u | (y >> (8 * k) & 15u)) - 8388608.0f;
          const float c1 = __uint_as_float(0x4B000000u | (y >> (8 * k + 4) & 15u)) - 8388608.0f;
          o[k] = pack2<true>(fmaf(s, c0, lo), fmaf(s, c1, lo));
        }
        *reinterpret_cast<uint4*>(img + gr * (kChunk * 128) + sw128(r, t + 4 * ci)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------

// Two fp32 numbers as one operand of the packed multiply-add and add.
__device__ __forceinline__ uint64_t pack_f32x2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
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

// Largest of 64 scores.
__device__ __forceinline__ float half_max(const uint32_t (&raw)[64]) {
  float mr[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 64; j += 2)
    mr[j / 2 & 3] = fmaxf(fmaxf(mr[j / 2 & 3], __uint_as_float(raw[j])), __uint_as_float(raw[j + 1]));
  return fmaxf(fmaxf(mr[0], mr[1]), fmaxf(mr[2], mr[3]));
}

// p = 2^(raw * k + add) as fp16 pairs; their fp32 sum.
__device__ __forceinline__ float half_exp(const uint32_t (&raw)[64], uint32_t (&pw)[32], float k, float add) {
  const uint64_t kk = pack_f32x2(k, k), aa = pack_f32x2(add, add);
  uint64_t ls[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float p0, p1;
    unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1])), kk, aa), p0, p1);
    p0 = ex2(p0);
    p1 = ex2(p1);
    ls[j & 1] = add_f32x2(ls[j & 1], pack_f32x2(p0, p1));
    pw[j] = pack2<true>(p0, p1);
  }
  float l0, l1, l2, l3;
  unpack_f32x2(ls[0], l0, l1);
  unpack_f32x2(ls[1], l2, l3);
  return (l0 + l1) + (l2 + l3);
}

__device__ __forceinline__ void bulk_image(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  mbar_expect_tx(bar, bytes);
  bulk_load(dst, src, bytes, bar);
}

// A unit of work: 256 rows of a sequence and KV head.
struct Unit {
  int chunks;                  // of keys; 0: a bad sequence, its rows are zeroed; -1: no more units
  int keys;                    // that the last row sees
  int row0, rows;              // first row; rows of the sequence
  int q0, before;              // first query token's row of q; keys before the first query's own
  int head, cell;              // KV head; slot * heads + head

  __device__ __forceinline__ bool live(int tile) const { return row0 + tile * kRows < rows; }
};

// Roles: warps 0-7 softmax (four per row tile), then one each for the MMAs, K's
// and V's images, and the units.  Every role walks the same units at its own pace:
// K and V of the next unit are loaded, and its first scores made, beside the end
// of the last.  Waits are bounded; a role whose wait gives up sets sh_fail and
// leaves, the others' waits then give up as well, and the units in hand stay
// unwritten (flagged).
template <int D>
__global__ void __launch_bounds__(kThreadsTc, 1) q4_tc_kernel(const Q4LongArgs a) {
  using I = Img<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  __shared__ uint64_t q_full[kTiles], s_full[kTiles], p_half[kTiles], p_full[kTiles], o_half[kTiles], o_done[kTiles];
  __shared__ uint64_t o_free[kTiles];
  __shared__ uint64_t unit_full, unit_empty, drain_bar;
  __shared__ uint32_t tmem_base;
  __shared__ Unit sh_unit;
  __shared__ int sh_fail;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int Hkv = a.num_kv_heads, GQ = a.group, Hq = Hkv * GQ;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - smem_addr(smem_raw));
  auto q_img = [&](int g) { return base + (uint32_t)(g * I::kBytes); };
  auto k_img = [&](int s) { return base + (uint32_t)((kTiles + s) * I::kBytes); };
  auto v_img = [&](int s) { return base + (uint32_t)((kTiles + kKStages + s) * I::kBytes); };

  if (tid == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(smem_addr(&k_full[s]), 1);
      mbar_init(smem_addr(&k_empty[s]), 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(smem_addr(&v_full[s]), 1);
      mbar_init(smem_addr(&v_empty[s]), 1);
    }
    for (int g = 0; g < kTiles; ++g) {
      mbar_init(smem_addr(&q_full[g]), kRows);
      mbar_init(smem_addr(&s_full[g]), 1);
      mbar_init(smem_addr(&p_half[g]), kRows);
      mbar_init(smem_addr(&p_full[g]), kRows);
      mbar_init(smem_addr(&o_half[g]), 1);
      mbar_init(smem_addr(&o_done[g]), 1);
      mbar_init(smem_addr(&o_free[g]), kRows);
    }
    mbar_init(smem_addr(&unit_full), 1);
    mbar_init(smem_addr(&unit_empty), kUnitWarp);   // the other roles' warps
    mbar_init(smem_addr(&drain_bar), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    sh_fail = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(&tmem_base)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
  // (a programmatic dependent: plan and images may still be in the making until here)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int count = a.counters[0];

  bool ok = true;
  int taken = 0;                                    // units read
  // The next unit (whole warp); chunks == -1 also after a wait that gave up.
  auto next_unit = [&]() {
    Unit u;
    u.chunks = -1;
    ok = warp_wait(smem_addr(&unit_full), taken & 1);
    if (ok) {
      u = sh_unit;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&unit_empty));
      ++taken;
    }
    return u;
  };

  if (warp == kUnitWarp) {
    // Units are taken as CTAs become free, one ahead of the roles, those with the
    // most chunks first: what a CTA holds when the last is taken is short.  Which one
    // the i-th is follows from how many have k chunks at least, for any k.
    // pairs of row tiles of a slot whose last row sees k chunks at least
    auto pairs_from = [&](int slot, int k) {
      const int b = a.list[slot], n = a.query_start[b + 1] - a.query_start[b], rows = n * GQ;
      const int64_t row = ((int64_t)(k - 1) * kChunk - (a.seq_lens[b] - n)) * GQ;   // the first that does
      const int all = (rows + kTiles * kRows - 1) / (kTiles * kRows);
      if (row >= rows) return 0;
      return all - (row > 0 ? (int)(row / (kTiles * kRows)) : 0);
    };
    auto units_from = [&](int k) {
      int mine = 0;
      for (int i = lane; i < count; i += 32) mine += pairs_from(i, k);
      return __reduce_add_sync(0xffffffffu, mine);
    };
    const int pairs = units_from(1);
    const long long units = (long long)pairs * Hkv;
    int most = 1;
    for (int i = lane; i < count; i += 32) most = max(most, (a.seq_lens[a.list[i]] + kChunk - 1) / kChunk);
    most = __reduce_max_sync(0xffffffffu, most);
    for (;; ++taken) {
      int u = 0;
      if (lane == 0) u = atomicAdd(&a.counters[1], 1);
      u = __shfl_sync(0xffffffffu, u, 0);
      Unit x = {};
      x.chunks = -1;
      if (u < units) {
        const int at = u / Hkv;
        // the largest k with more than `at` pairs: not above the last unit's, and near it
        int lo = most, hi = most;
        for (int step = 1; lo > 1 && units_from(lo) <= at; step *= 2) {
          hi = lo - 1;
          lo = max(1, hi - step);
        }
        while (lo < hi) {
          const int k = (lo + hi + 1) / 2;
          if (units_from(k) > at) lo = k;
          else hi = k - 1;
        }
        most = lo;                                  // (the next unit has no more)
        const int more = units_from(lo + 1);
        // the (at - more)-th pair of exactly `lo` chunks, by slot
        int slot = 0, pr = 0, left = at - more;
        bool found = false;
        for (int s0 = 0; s0 < count && !found; s0 += 32) {
          const int i = s0 + lane, from = i < count ? pairs_from(i, lo) : 0, mine = from - (i < count ? pairs_from(i, lo + 1) : 0);
          int incl = mine;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
          }
          const unsigned here = __ballot_sync(0xffffffffu, left < incl);
          if (here != 0) {
            const int src = __ffs(here) - 1;
            slot = s0 + src;
            // a slot's pairs of `lo` chunks are consecutive, the first has `from` pairs from it on
            const int all = i < count ? pairs_from(i, 1) : 0;
            pr = __shfl_sync(0xffffffffu, all - from + (left - (incl - mine)), src);
            found = true;
          } else {
            left -= __shfl_sync(0xffffffffu, incl, 31);
          }
        }
        const int b = a.list[slot], n = a.query_start[b + 1] - a.query_start[b];
        x.head = u % Hkv;
        x.cell = slot * Hkv + x.head;
        x.q0 = a.query_start[b];
        x.before = a.seq_lens[b] - n;
        x.rows = n * GQ;
        x.row0 = pr * (kTiles * kRows);
        const int last = min(x.row0 + kTiles * kRows, x.rows) - 1;
        x.keys = x.before + last / GQ + 1;          // keys the last row sees
        x.chunks = a.bad[slot] != 0 ? 0 : (x.keys + kChunk - 1) / kChunk;
      }
      if (taken > 0 && !warp_wait(smem_addr(&unit_empty), (taken - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        sh_unit = x;
        mbar_arrive(smem_addr(&unit_full));
      }
      __syncwarp();
      if (x.chunks < 0) break;
      // its queries into L2
      const int last = min(x.row0 + kTiles * kRows, x.rows) - 1;
      for (int t = x.row0 / GQ + lane; t <= last / GQ; t += 32) {
        const __nv_bfloat16* row = a.q + ((int64_t)(x.q0 + t) * Hq + (int64_t)x.head * GQ) * D;
        for (int e = 0; e < GQ * D; e += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + e));
      }
    }
  } else if (warp == kMmaWarp) {
    // Per chunk c: P . V_0(c), S_0(c+1), P . V_1(c), [V stage free], S_1(c+1), [K
    // stage free]: one tile's softmax runs beside the other tile's products.
    // (S_g(c+1) overwrites the columns that P . V_g(c) reads; the MMAs of one
    // issuing thread run in order.)  Where a unit ends, both tiles' P . V come
    // before the next unit's scores, which wait for its queries.
    const uint32_t id_s = mma_idesc<true>(kRows, kChunk, 0), id_o = mma_idesc<true>(kRows, D, 1);
    int kc = 0, vc = 0;                             // chunks of K and V used
    int nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;         // units and chunks of each tile
    auto issue_s = [&](int g) {
      const uint64_t qd = smem_desc(q_img(g), 16, 1024), kd = smem_desc(k_img(kc % kKStages), 16, 1024);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int at = ((ks / 4) * (kRows * 128) + (ks % 4) * 32) / 16;
        warp_mma_ss(tm + I::scol(g), qd + at, kd + at, id_s, ks > 0);
      }
      warp_mma_commit(smem_addr(&s_full[g]));
    };
    // P . V of a chunk, 64 keys as soon as P of them is written, then the others.
    auto issue_pv = [&](int g, bool first, int nsub, int np) {
      const uint64_t vd = smem_desc(v_img(vc % kVStages), kChunk * 128, 1024);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!warp_wait(smem_addr(half ? &p_full[g] : &p_half[g]), np & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = half * 4; kk < half * 4 + 4; ++kk)
          if (kk < nsub)
            warp_mma_ts(tm + I::ocol(g), tm + I::scol(g) + kk * 8, vd + kk * (16 * 128 / 16), id_o,
                        (!first || kk > 0) ? 1u : 0u);
        warp_mma_commit(smem_addr(half ? &o_done[g] : &o_half[g]));
      }
      return true;
    };
    auto wait_k = [&]() { return warp_wait(smem_addr(&k_full[kc % kKStages]), (kc / kKStages) & 1); };
    // the first scores of a unit
    auto begin = [&](const Unit& u) {
      if (!wait_k() || !warp_wait(smem_addr(&q_full[0]), nq0 & 1)) return false;
      ++nq0;
      tc_fence_after();
      issue_s(0);
      if (u.live(1)) {
        if (!warp_wait(smem_addr(&q_full[1]), nq1 & 1)) return false;
        ++nq1;
        tc_fence_after();
        issue_s(1);
      }
      warp_mma_commit(smem_addr(&k_empty[kc % kKStages]));
      ++kc;
      return true;
    };
    auto next_of = [&]() {
      Unit u = next_unit();
      while (u.chunks == 0) u = next_unit();
      return u;
    };
    Unit u = next_of();
    if (u.chunks > 0) ok = begin(u);
    while (ok && u.chunks > 0) {
      const bool live1 = u.live(1);
      for (int c = 0; c < u.chunks; ++c) {
        const int nsub = (min(u.keys - c * kChunk, kChunk) + 15) / 16;
        const bool more = c + 1 < u.chunks;
        ok = warp_wait(smem_addr(&v_full[vc % kVStages]), (vc / kVStages) & 1) && (!more || wait_k());
        // (the last unit's O is read)
        if (ok && c == 0 && nq0 > 1) ok = warp_wait(smem_addr(&o_free[0]), nq0 & 1);
        if (!ok || !issue_pv(0, c == 0, nsub, np0++)) { ok = false; break; }
        if (more) issue_s(0);
        if (live1) {
          if (c == 0 && nq1 > 1) ok = warp_wait(smem_addr(&o_free[1]), nq1 & 1);
          if (!ok || !issue_pv(1, c == 0, nsub, np1++)) { ok = false; break; }
        }
        warp_mma_commit(smem_addr(&v_empty[vc % kVStages]));
        ++vc;
        if (more) {
          if (live1) issue_s(1);
          warp_mma_commit(smem_addr(&k_empty[kc % kKStages]));
          ++kc;
        }
      }
      if (!ok) break;
      u = next_of();
      if (ok && u.chunks > 0) ok = begin(u);
    }
    // all tensor-core work of this CTA completes before TMEM is freed
    tc_fence_after();
    warp_mma_commit(smem_addr(&drain_bar));
    if (!warp_wait(smem_addr(&drain_bar), 0)) ok = false;
  } else if (warp == kKWarp || warp == kVWarp) {
    // one lane copies: chunk i into stage i % stages once the MMAs are done with it
    const bool is_k = warp == kKWarp;
    const int nst = is_k ? kKStages : kVStages;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    int i = 0;
    for (Unit u = next_unit(); ok && u.chunks >= 0; u = next_unit()) {
      const unsigned char* src = a.images + ((int64_t)u.cell * a.chunks * 2 + (is_k ? 0 : 1)) * I::kBytes;
      for (int c = 0; c < u.chunks; ++c, ++i) {
        const int st = i % nst;
        if (i >= nst && !warp_wait(smem_addr(&empty[st]), (i / nst - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0)
          bulk_image(is_k ? k_img(st) : v_img(st), src + (int64_t)c * 2 * I::kBytes, I::kBytes, smem_addr(&full[st]));
      }
      if (!ok) break;
    }
    // every copy has landed before the CTA ends (normally already so)
    for (int st = 0; st < nst && st < i; ++st) warp_wait(smem_addr(&full[st]), ((i - 1 - st) / nst) & 1);
  } else {
    const int tile = warp >> 2, wrow = (warp & 3) * 32, ri = wrow + lane;   // this thread's row of the tile
    const uint32_t lane_base = (uint32_t)wrow << 16;
    const uint32_t s_tmem = tm + lane_base + I::scol(tile), o_tmem = tm + lane_base + I::ocol(tile);
    constexpr int kLanes = D / 8, kEach = 32 / kLanes, kTurns = 32 / kEach;   // lanes of a row, rows of a turn
    const int part = lane % kLanes, sub = lane / kLanes;
    const uint32_t q_band = q_img(tile) + (part / 8) * (kRows * 128);
    // Asks for the warp's 32 rows of q, into their places of the tile's swizzled bands.
    auto fetch_q = [&](const Unit& u) {
      int r = u.row0 + tile * kRows + wrow + sub;
      const int tok = r / GQ, dtok = kEach / GQ, dh = kEach - dtok * GQ;
      int h = r - tok * GQ;
      const __nv_bfloat16* from = a.q + ((int64_t)(u.q0 + tok) * Hq + (int64_t)u.head * GQ + h) * D + part * 8;
      const int step = (dtok * Hq + dh) * D, wrap = (Hq - GQ) * D;
#pragma unroll 4
      for (int i = 0; i < kTurns; ++i) {
        const bool in = r < u.rows;                 // (rows behind the last are zeros)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         q_band + sw128(wrow + i * kEach + sub, part % 8)),
                     "l"(in ? from : a.q), "r"(in ? 16 : 0)
                     : "memory");
        r += kEach;
        h += dh;
        from += step;
        if (h >= GQ) {
          h -= GQ;
          from += wrap;
        }
      }
    };
    // Turns them to fp16 in place (each lane what it asked for), each row under a power
    // of two (largest in [2^13, 2^14)); returns what this thread's own row multiplies
    // the scores by.  A negative scale turns q's sign, a zero one takes it as 0.
    auto turn_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      float own = 0.0f;
      // (four turns side by side: one alone is a chain of shuffles)
#pragma unroll 1
      for (int i0 = 0; i0 < kTurns; i0 += 4) {
        uint4 x[4];
        uint32_t top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lds128(q_band + sw128(wrow + (i0 + i) * kEach + sub, part % 8));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t m = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                      __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
          top[i] = max(m & 0xffffu, m >> 16);       // (255: an infinity or NaN, and so is the row)
        }
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = __shfl_xor_sync(0xffffffffu, top[i], off);
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = max(top[i], y[i]);
        }
        float up[4], theirs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = min(top[i] > 0 ? 140 - (int)(top[i] >> 7) : 0, 110);   // (-115 at least)
          up[i] = __uint_as_float((uint32_t)(127 + e) << 23);
          theirs[i] = __uint_as_float((uint32_t)(127 - e) << 23);
          if (a.scale_log2 <= 0.0f) up[i] = a.scale_log2 < 0.0f ? -up[i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) theirs[i] = __shfl_sync(0xffffffffu, theirs[i], lane % kEach * kLanes);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (lane / kEach == i0 + i) own = theirs[i];
          const uint32_t w4[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t o4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o4[k] = pack2<true>(__uint_as_float(w4[k] << 16) * up[i], __uint_as_float(w4[k] & 0xffff0000u) * up[i]);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           q_band + sw128(wrow + (i0 + i) * kEach + sub, part % 8)),
                       "r"(o4[0]), "r"(o4[1]), "r"(o4[2]), "r"(o4[3])
                       : "memory");
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the images -> tensor core
      mbar_arrive(smem_addr(&q_full[tile]));
      return fmaxf(fabsf(a.scale_log2) * own, 1e-37f);
    };
    Unit u = next_unit();
    float sl2 = 0.0f;
    if (u.chunks > 0 && u.live(tile)) {
      fetch_q(u);
      sl2 = turn_q();
    }
    int j = 0;                                      // chunks of this tile
    while (ok && u.chunks >= 0) {
      const int r = u.row0 + tile * kRows + ri;
      const bool valid = r < u.rows, mine = u.chunks > 0 && u.live(tile);
      const int lim = valid ? u.before + r / GQ : -1;
      // One row per thread.  A chunk row's 128 scores in two halves, each read from
      // TMEM once: its largest is tested against the reference, then P is written
      // over the columns the half has read.  When a half passes the reference by
      // more than kSlack octaves the reference moves by whole octaves, so that the
      // rescaling of O (once the P . V before is done) is exact.
      float m_ref = -INFINITY, l = 0.0f;
      Unit nu = {};
      if (mine) {
        const bool warp_live = __any_sync(0xffffffffu, valid);
        const int2* exps = a.exps + (int64_t)u.cell * a.chunks;
        int2 ex = __ldg(exps);
        for (int c = 0; c < u.chunks; ++c, ++j) {
          const int2 now = ex;
          if (c + 1 < u.chunks) ex = __ldg(exps + c + 1);
          if (!warp_wait(smem_addr(&s_full[tile]), j & 1)) { ok = false; break; }
          tc_fence_after();
          if (c + 1 == u.chunks) {                  // every score of this unit is made: the next one's queries
            nu = next_unit();
            if (!ok) break;
            if (nu.chunks > 0 && nu.live(tile)) fetch_q(nu);
          }
          if (!warp_live) {                         // padding rows: keep the barriers' phases
            tc_fence_before();
            mbar_arrive(smem_addr(&p_half[tile]));
            mbar_arrive(smem_addr(&p_full[tile]));
            continue;
          }
          // (positive in any case: a masked score of -infinity stays one)
          const float kf = fmaxf(sl2 * __uint_as_float((uint32_t)(127 + now.x) << 23), 1e-37f), ev = (float)now.y;
          const int cstart = c * kChunk;
          const bool masked = __any_sync(0xffffffffu, cstart + kChunk - 1 > lim);
          float lsum = 0.0f;
          // (rolled, and masks applied beforehand: code that runs once a unit comes from
          // far away, 2500 cycles for a masked form of its own)
#pragma unroll 1
          for (int ps = 0; ps < 2; ++ps) {
            uint32_t raw[64];
            tmem_read64(s_tmem + 64 * ps, raw);
            const int first = cstart + 64 * ps;
            if (masked) {
#pragma unroll
              for (int x = 0; x < 64; ++x)
                if (x > lim - first) raw[x] = 0xff800000u;
            }
            const float mx_raw = half_max(raw);
            const float mx = mx_raw == -INFINITY ? -INFINITY : fmaf(mx_raw, kf, ev - kHead);
            const bool need = m_ref == -INFINITY ? mx > -INFINITY : mx > m_ref + kSlack;
            // V's magnitudes may lie further apart than fp32's exponents: p of rows of
            // small values is then nothing while its weight 2^(s - m) still counts.
            const bool far = mx > -INFINITY && mx < m_ref - kFar;
            if (__any_sync(0xffffffffu, far)) {
              const float by = m_ref == -INFINITY ? 0.0f : m_ref;
              float sum = 0.0f;
#pragma unroll 1
              for (int c0 = 0; c0 < 64; c0 += 16) {
                uint32_t sv[16];
                tmem_ld16(s_tmem + 64 * ps + c0, sv);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  sum += first + c0 + j <= lim ? ex2(fmaf(__uint_as_float(sv[j]), kf, -by)) : 0.0f;
              }
              if (far) l += sum;
            }
            if (__any_sync(0xffffffffu, need)) {
              const float k = (need && m_ref != -INFINITY) ? ceilf(mx - m_ref) : 0.0f;
              const float m_new = !need ? m_ref : (m_ref == -INFINITY ? mx : m_ref + k);
              const float alpha = need ? (m_ref == -INFINITY ? 0.0f : ldexpf(1.0f, -(int)k)) : 1.0f;
              // O so far: of the chunks before, or (second half) of the first half too
              if (c > 0 || ps > 0) {
                if (!(ps > 0 ? warp_wait(smem_addr(&o_half[tile]), j & 1)
                             : warp_wait(smem_addr(&o_done[tile]), (j - 1) & 1))) {
                  ok = false;
                  break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                  uint32_t ov[16];
                  tmem_ld16(o_tmem + c0, ov);
                  tmem_wait_ld();
#pragma unroll
                  for (int j = 0; j < 16; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
                  tmem_st16(o_tmem + c0, ov);
                }
                tmem_wait_st();
              }
              lsum *= alpha;
              if (need) l = m_ref == -INFINITY ? 0.0f : ldexpf(l, -(int)k);
              m_ref = m_new;
            }
            const float add = m_ref == -INFINITY ? 0.0f : ev - m_ref;
            uint32_t pw[32];
            const float part = half_exp(raw, pw, kf, add);
            if (!far) lsum += part;
            tmem_st32(s_tmem + 32 * ps, pw);
            if (ps == 0) {
              tmem_wait_st();
              tc_fence_before();
              mbar_arrive(smem_addr(&p_half[tile]));
            }
          }
          if (!ok) break;
          tmem_wait_st();
          l = fmaf(lsum, __uint_as_float((uint32_t)(127 - now.y) << 23), l);
          tc_fence_before();
          mbar_arrive(smem_addr(&p_full[tile]));
        }
        if (!ok) break;
      }
      if (!mine) {
        nu = next_unit();
        if (nu.chunks > 0 && nu.live(tile)) fetch_q(nu);
      }
      if (nu.chunks > 0 && nu.live(tile)) sl2 = turn_q();
      if (mine && !warp_wait(smem_addr(&o_done[tile]), (j - 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (u.live(tile)) {
        // 32 columns of a row are four 16-byte pieces; four lanes exchange theirs, so
        // that each store writes 64 bytes of eight rows instead of 16 bytes of 32.
        const float inv = mine && valid ? 1.0f / l : 0.0f;
        const int first = r - (lane & 3);
        int64_t at[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int tok = (first + x) / GQ;
          at[x] = first + x < u.rows
                      ? ((int64_t)(u.q0 + tok) * Hq + (int64_t)u.head * GQ + (first + x - tok * GQ)) * D + (lane & 3) * 8
                      : -1;
        }
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t ov[32], w[4][4];
          if (mine) {
            tmem_read32(o_tmem + c0, ov);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) ov[x] = 0u;
          }
#pragma unroll
          for (int x = 0; x < 16; ++x)
            w[x / 4][x % 4] = pack2<false>(__uint_as_float(ov[2 * x]) * inv, __uint_as_float(ov[2 * x + 1]) * inv);
#pragma unroll
          for (int bit = 1; bit <= 2; bit <<= 1) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (x & bit) continue;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & bit ? w[x][y] : w[x | bit][y], bit);
                if (lane & bit) w[x][y] = got;
                else w[x | bit][y] = got;
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (at[x] >= 0)
              *reinterpret_cast<uint4*>(a.out + at[x] + c0) = make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
        }
      }
      tc_fence_before();
      if (mine) mbar_arrive(smem_addr(&o_free[tile]));
      u = nu;
    }
  }
  if (!ok) sh_fail = 1;
  asm volatile("cp.async.wait_all;" ::: "memory");   // (after a wait that gave up)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sh_fail && tid == 0) atomicOr(a.flags, PAGEDKV_FLAG_WAIT_TIMEOUT);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(kTmemCols) : "memory");
}

// A launch as programmatic dependent of the one before it.
kv_status launch_after(void (*kernel)(Q4LongArgs), dim3 grid, int threads, int smem, cudaStream_t s,
                       const Q4LongArgs& a, const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, kernel, a), what);
}

template <int D>
kv_status launch_tc(const Q4LongArgs& a, int ctas, cudaStream_t s) {
  static std::mutex mu;
  static bool set[64] = {};
  int dev = 0;
  kv_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != KV_OK) return st;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && !set[dev]) {
      st = cuda_check(cudaFuncSetAttribute(q4_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Img<D>::kSmem),
                      "cudaFuncSetAttribute(q4_tc_kernel)");
      if (st != KV_OK) return st;
      set[dev] = true;
    }
  }
  return launch_after(q4_tc_kernel<D>, dim3((unsigned)ctas), kThreadsTc, Img<D>::kSmem, s, a, "q4_tc_kernel launch");
}

}  // namespace

size_t q4_slot_bytes(int num_kv_heads, int head_dim, int max_seq_len) {
  const size_t chunks = ((size_t)max_seq_len + kChunk - 1) / kChunk;
  return (size_t)num_kv_heads * chunks * (2 * kChunk * (size_t)head_dim * 2 + sizeof(int2));
}

size_t q4_plan_bytes(int batch, int slots) {
  return (((size_t)batch + 2 * (size_t)slots + 2) * 4 + 127) & ~(size_t)127;
}

kv_status launch_q4_long(Q4LongArgs a, void* memory, int sms, cudaStream_t s) {
  // [images][exponents][slot of each sequence][list][bad][counters]; images 128-byte aligned
  a.chunks = (a.max_seq_len + kChunk - 1) / kChunk;
  const size_t cells = (size_t)a.slots * a.num_kv_heads * a.chunks;
  a.images = static_cast<unsigned char*>(memory);
  a.exps = reinterpret_cast<int2*>(a.images + cells * 2 * kChunk * a.head_dim * 2);
  a.list = reinterpret_cast<int*>(a.exps + cells);
  a.bad = a.list + a.slots;
  a.counters = a.bad + a.slots;
  kv_status st = launch_after(q4_plan_kernel, dim3(1), 256, 0, s, a, "q4_plan_kernel launch");
  if (st != KV_OK) return st;
  const bool wide = a.head_dim == 128, big = a.block_size == 32;
  void (*widen)(Q4LongArgs) = wide ? (big ? q4_widen_kernel<128, 32> : q4_widen_kernel<128, 16>)
                                   : (big ? q4_widen_kernel<64, 32> : q4_widen_kernel<64, 16>);
  const dim3 grid((unsigned)a.chunks, (unsigned)a.num_kv_heads, (unsigned)a.slots);
  if ((st = launch_after(widen, grid, 256, 0, s, a, "q4_widen_kernel launch")) != KV_OK) return st;
  const long long units = ((long long)a.num_tokens * a.group / (kTiles * kRows) + a.slots) * a.num_kv_heads;
  const int ctas = (int)(units < sms ? units : sms);
  return wide ? launch_tc<128>(a, ctas, s) : launch_tc<64>(a, ctas, s);
}

}  // namespace pagedkv
