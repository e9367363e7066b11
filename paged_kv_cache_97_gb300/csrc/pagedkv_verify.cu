// pagedkv_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers (“让 Agent 跑得快：LLM 推理服务”, §六 投机
// 解码: the target scores the drafts in one parallel pass and keeps a prefix).
//
// Draft x at position i is kept while u_i q_i(x) < p_i(x).  At the first refusal
// the token is drawn from max(p_i - q_i, 0), after all drafts from p_i: the
// lowest z whose inclusive sum of weights exceeds u * (the sum of all).  So that
// every split of the row gives the same token, the weights are added as whole
// numbers of 2^-44 (64 bits): w + 1 in fp32 has round(w 2^23) in its last bits,
// and what that leaves off, added to 1.5 * 2^-21, the next 21; two integer adds
// per weight and no conversion.
//
// A cluster of up to 8 CTAs takes a sequence: every CTA finds the row from the
// drafts by itself, each sums its part of the row, the parts' sums go to all
// CTAs through distributed shared memory (once a barrier begun at the start has shown
// that all of them run), and the one warp whose part holds the
// drawn place finds it by the sums of its rounds and steps (a round that is not its
// last is read again, from L2; so is every one past the 64 whose sums are kept).  Bound by the one row (two with q) that
// has to be read per sequence, and in small batches by the chain of loads:
// offsets, drafts, their probabilities, the row, the part again.  Measured (GB300,
// 128256 tokens): 64 sequences of 5 drafts, fp32 p and q, 21 us (9.7 at the copy
// rate), 256 of bf16 32 us (19), 8 of fp32 10 us; one of 4 drafts over 32000, 8.5 us; drafts
// without probabilities, 64 of 5 16.5 us (4.8), 256 of bf16 31 us (9.7).  Other
// counts of threads and sizes of clusters took up to 28.7 us where these took 24.4.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pagedkv_common.cuh"
#include "pagedkv_device.cuh"

namespace pagedkv {
namespace {

using namespace dev;

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kRounds = 64;                         // rounds of a warp whose sums are kept

struct VerifyArgs {
  int32_t* out_tokens;         // [T]
  int32_t* accepted;           // [batch]
  int32_t* new_lens;           // [batch], or null
  const int32_t* seq_lens;
  const int32_t* tokens;       // [T]
  const void* target;          // [T, V]
  const void* draft;           // [T - batch, V], or null: q is 1 at the draft
  const float* uniform;        // [T]
  const int32_t* query_start;  // [batch + 1]
  unsigned int* flags;
  int batch, num_tokens, max_query_len, vocab, cluster;
};

template <typename T>
__device__ __forceinline__ float prob(const T* p) {
  if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const float*>(p));
  else return static_cast<float>(*p);
}

// N consecutive probabilities (kVec: one aligned 16-byte load, all or none of
// them there; else one).  `have` false: zeros.
template <typename T, int N, bool kVec>
__device__ __forceinline__ void probs(const T* p, bool have, float (&v)[N]) {
  if constexpr (kVec) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (have) x = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const unsigned short h = (unsigned short)(w[i / 2] >> (16 * (i & 1)));
        T t;
        memcpy(&t, &h, 2);
        v[i] = static_cast<float>(t);
      }
    }
  } else {
    static_assert(N == 1, "one element a load");
    v[0] = have ? prob(p) : 0.0f;
  }
}

// What the token is drawn by: p; max(p - q, 0); or p without the draft's own.
enum { kPlain = 0, kLess = 1, kWithout = 2 };

struct Row {
  int how, without;
};

// Weights of U runs of N elements, a run every `step`, from element i on (0 from
// `end` on), in [0, 1]; NaN counts as 0.  All loads are issued before the first is
// used.
template <typename T, int N, int U, bool kVec>
__device__ __forceinline__ void weights_of(const T* p, const T* q, const Row& r, int i, int step, int end,
                                           float (&w)[U][N]) {
  if (r.how == kLess) {
    float x[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool have = i + u * step < end;
      probs<T, N, kVec>(p + i + u * step, have, w[u]);
      probs<T, N, kVec>(q + i + u * step, have, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) w[u][k] = __fsub_rn(w[u][k], x[u][k]);
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) probs<T, N, kVec>(p + i + u * step, i + u * step < end, w[u]);
    if (r.how == kWithout) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (i + u * step + k == r.without) w[u][k] = 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < N; ++k) w[u][k] = fminf(fmaxf(w[u][k], 0.0f), 1.0f);
}

constexpr uint32_t kHiZero = 0x3f800000u;           // 1
constexpr uint32_t kLoZero = 0x35400000u;           // 1.5 * 2^-21

// Adds w's 2^-23 units and its further 2^-44 units (each with its zero's bits).
__device__ __forceinline__ void add_units(float w, uint32_t& hi, uint32_t& lo) {
  const float a = __fadd_rn(w, 1.0f);
  const float e = __fsub_rn(w, __fsub_rn(a, 1.0f));
  hi += __float_as_uint(a);
  lo += __float_as_uint(__fadd_rn(e, __uint_as_float(kLoZero)));
}
// The sum of n <= 511 weights in 2^-44 units.
__device__ __forceinline__ long long units(uint32_t hi, uint32_t lo, int n) {
  return ((long long)(hi - (uint32_t)n * kHiZero) << 21) + (int32_t)(lo - (uint32_t)n * kLoZero);
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kVerifyThreads, 1024 / kVerifyThreads) verify_kernel(const VerifyArgs a) {
  constexpr int N = kVec ? 16 / (int)sizeof(T) : 1;
  constexpr int U = kVec ? 32 / N : 8;              // runs taken together
  __shared__ int first_refused, refused_token;
  __shared__ long long warp_sum[kVerifyWarps], cta_sum[2][kMaxCluster], round_sum[kVerifyWarps][kRounds];
  const int b = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q0 = __ldg(a.query_start + b), n = __ldg(a.query_start + b + 1) - q0;
  const int64_t d0 = (int64_t)q0 - b;               // the sequence's first row of draft
  const bool lens = a.seq_lens != nullptr;
  const int L = lens ? __ldg(a.seq_lens + b) : 0;
  // (uniform over the cluster)
  const bool rows = q0 >= 0 && n >= 0 && q0 <= a.num_tokens - n;
  if (!rows || n > a.max_query_len || (lens && n > L) ||
      (a.draft != nullptr && (n == 0 || d0 < 0 || d0 + n - 1 > a.num_tokens - a.batch))) {
    if (rank == 0) {
      if (threadIdx.x == 0) {
        atomicOr(a.flags, PAGEDKV_FLAG_BAD_SEQ_LEN);
        a.accepted[b] = 0;
        if (lens) a.new_lens[b] = L;
      }
      if (rows)
        for (int i = threadIdx.x; i < n; i += kVerifyThreads) a.out_tokens[q0 + i] = -1;
    }
    return;
  }
  if (n == 0) {
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[b] = 0;
      if (lens) a.new_lens[b] = L;
    }
    return;
  }
  // This CTA runs: its peers may store into it.  (Relaxed: they find nothing of it.
  // What left above left with its whole cluster.)
  if (a.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int V = a.vocab;
  const T* target = static_cast<const T*>(a.target);
  const T* draft = static_cast<const T*>(a.draft);

  // ---- drafts kept -----------------------------------------------------------
  if (threadIdx.x == 0) {
    first_refused = n - 1;
    refused_token = -1;
  }
  float u = __ldg(a.uniform + q0 + n - 1);
  __syncthreads();
  int last = -1, last_x = -1;                       // this thread's latest refusal
  for (int i = threadIdx.x; i < n - 1; i += kVerifyThreads) {
    const int x = __ldg(a.tokens + q0 + i + 1);
    bool keep = false;
    if (x < 0 || x >= V) {
      if (rank == 0) atomicOr(a.flags, PAGEDKV_FLAG_BAD_INDEX);
    } else {
      const float p = prob(target + (int64_t)(q0 + i) * V + x);
      const float q = draft ? prob(draft + (d0 + i) * V + x) : 1.0f;
      // (products of two fp32 numbers are exact in fp64)
      keep = (double)__ldg(a.uniform + q0 + i) * (double)q < (double)p;
    }
    if (!keep) {
      atomicMin(&first_refused, i);
      last = i;
      last_x = x;
      break;                                        // (a thread's later drafts come after this one)
    }
  }
  __syncthreads();
  const int kept = first_refused;
  if (last == kept) refused_token = last_x;
  __syncthreads();
  Row r = {kPlain, -1};
  if (kept < n - 1) {
    r.without = refused_token;
    const bool in = r.without >= 0 && r.without < V;
    r.how = !in ? kPlain : draft ? kLess : kWithout;   // a draft outside the vocabulary: from p
  }
  const T* p = target + (int64_t)(q0 + kept) * V;
  const T* q = r.how == kLess ? draft + (d0 + kept) * V : p;
  u = u >= 0.0f ? fminf(u, 0.99999994f) : 0.0f;

  if (rank == 0) {
    for (int i = threadIdx.x; i < n; i += kVerifyThreads)
      if (i != kept) a.out_tokens[q0 + i] = i < kept ? __ldg(a.tokens + q0 + i + 1) : -1;
    if (threadIdx.x == 0) a.accepted[b] = kept;
  }

  // ---- this warp's part of the row: [w0, w1) ----------------------------------
  constexpr int kStep = 32 * N;
  const int all_warps = a.cluster * kVerifyWarps;
  const int per = ((V + all_warps - 1) / all_warps + kStep - 1) / kStep * kStep;
  const int64_t at = (int64_t)(rank * kVerifyWarps + warp) * per;
  const int w0 = (int)(at < V ? at : V), w1 = (int)(at + per < V ? at + per : V);
  for (int pass = 0;; ++pass) {
    long long sum = 0;
    float w[U][N];                                  // the weights taken last
#pragma unroll 1
    for (int i0 = w0, round = 0; i0 < w1; i0 += U * kStep, ++round) {
      weights_of<T, N, U, kVec>(p, q, r, i0 + lane * N, kStep, w1, w);
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) add_units(w[k][e], hi, lo);
      long long part = units(hi, lo, U * N);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
      if (lane == 0 && round < kRounds) round_sum[warp][round] = part;
      sum += part;
    }
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    long long mine = 0, before = 0;
#pragma unroll
    for (int k = 0; k < kVerifyWarps; ++k) {
      if (k < warp) before += warp_sum[k];
      mine += warp_sum[k];
    }
    long long total = mine;
    if (a.cluster > 1) {
      // (a peer's shared memory is there only once the peer has begun)
      if (pass == 0) cluster_wait();
      if (threadIdx.x < a.cluster) {
        uint32_t to;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(to)
                     : "r"(smem_addr(&cta_sum[pass][rank])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(mine) : "memory");
      }
      cluster_arrive();
      cluster_wait();
      total = 0;
      for (int k = 0; k < a.cluster; ++k) {
        if (k < rank) before += cta_sum[pass][k];
        total += cta_sum[pass][k];
      }
    }
    // (after the barrier: new_lens may be seq_lens, which every CTA has read by now)
    if (rank == 0 && threadIdx.x == 0 && lens) a.new_lens[b] = L - n + 1 + kept;
    if (total == 0 && r.how != kPlain) {            // nothing is left of p: drawn from p itself
      r.how = kPlain;
      __syncthreads();
      continue;
    }
    const double goal = (double)u * (double)total;
    if (total == 0) {
      if (rank == 0 && threadIdx.x == 0) a.out_tokens[q0 + kept] = V - 1;
      return;
    }
    // ---- the place is this warp's if its sums pass the goal first --------------
    if (!((double)before <= goal && (double)(before + sum) > goal)) return;
    // Its round by the rounds' sums, its step by the steps' (redux of the 2^-23 units
    // and of the further ones, which stay within 32 bits), its place by a scan.
#pragma unroll 1
    for (int i0 = w0, round = 0; i0 < w1; i0 += U * kStep, ++round) {
      if (round < kRounds) {
        const long long part = round_sum[warp][round];
        if (!((double)(before + part) > goal)) {
          before += part;
          continue;
        }
      }
      // (the last round's weights are still held, but for rounds without a sum of their
      // own that were looked through since)
      if (round >= kRounds || i0 + U * kStep < w1)
        weights_of<T, N, U, kVec>(p, q, r, i0 + lane * N, kStep, w1, w);
      uint32_t hi[U];
      int32_t lo[U];
      long long step[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        uint32_t h = 0, l = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) add_units(w[k][e], h, l);
        hi[k] = h - (uint32_t)N * kHiZero;
        lo[k] = (int32_t)(l - (uint32_t)N * kLoZero);
        step[k] = ((long long)__reduce_add_sync(0xffffffffu, hi[k]) << 21) + __reduce_add_sync(0xffffffffu, lo[k]);
      }
      // the step, its units and weights picked by selects
      int at_step = -1;
      uint32_t h0 = 0;
      int32_t l0 = 0;
      float v[N];
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = 0.0f;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool here = at_step < 0 && (double)(before + step[k]) > goal;
        if (at_step < 0 && !here) before += step[k];
        at_step = here ? k : at_step;
        h0 = here ? hi[k] : h0;
        l0 = here ? lo[k] : l0;
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = here ? w[k][e] : v[e];
      }
      if (at_step < 0) continue;
      const long long own = ((long long)h0 << 21) + l0;
      long long incl = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, (double)(before + incl) > goal);
      if (lane == __ffs(past) - 1) {
        long long sofar = before + incl - own;
        int z = i0 + at_step * kStep + lane * N;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          uint32_t h1 = 0, l1 = 0;
          add_units(v[e], h1, l1);
          sofar += units(h1, l1, 1);
          if ((double)sofar <= goal) ++z;
        }
        a.out_tokens[q0 + kept] = z;
      }
      return;
    }
    return;
  }
}

template <typename T>
kv_status launch_verify(const VerifyArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.batch * a.cluster));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool vec = (int64_t)a.vocab * sizeof(T) % 16 == 0 && aligned16(a.target) && aligned16(a.draft);
  return cuda_check(vec ? cudaLaunchKernelEx(&cfg, verify_kernel<T, true>, a)
                        : cudaLaunchKernelEx(&cfg, verify_kernel<T, false>, a),
                    "verify_kernel launch");
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" kv_status pagedkv_verify_drafts(int32_t* out_tokens, int32_t* num_accepted, const int32_t* tokens,
                                           const void* target_probs, const void* draft_probs, const float* uniform,
                                           const int32_t* query_start, const int32_t* seq_lens, int32_t* new_lens,
                                           int batch, int num_tokens, int max_query_len, int vocab,
                                           pagedkv_prob_dtype dtype, void* stream) {
  const char* who = "pagedkv_verify_drafts";
  if (batch < 0 || num_tokens < 0 || max_query_len <= 0 || vocab <= 0 || vocab >= (1 << 19) ||
      (dtype != PAGEDKV_PROB_F32 && dtype != PAGEDKV_PROB_BF16 && dtype != PAGEDKV_PROB_F16))
    return fail(KV_ERR_INVALID_ARG, "%s: bad sizes or dtype (vocab 1 to 2^19 - 1)", who);
  if (batch > (1 << 24)) return fail(KV_ERR_INVALID_ARG, "%s: too many sequences", who);
  if (batch == 0) return KV_OK;
  if (!num_accepted || !query_start ||
      (num_tokens > 0 && (!out_tokens || !tokens || !target_probs || !uniform)))
    return fail(KV_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if ((seq_lens == nullptr) != (new_lens == nullptr))
    return fail(KV_ERR_INVALID_ARG, "%s: give both seq_lens and new_lens, or neither", who);
  if (draft_probs && num_tokens < batch)
    return fail(KV_ERR_INVALID_ARG, "%s: with draft_probs every sequence has a token at least", who);
  const uintptr_t unit = dtype == PAGEDKV_PROB_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(target_probs) & unit) || (reinterpret_cast<uintptr_t>(draft_probs) & unit))
    return fail(KV_ERR_INVALID_ARG, "%s: the probabilities must be aligned to their type", who);
  if (out_tokens == tokens && num_tokens > 0)
    return fail(KV_ERR_INVALID_ARG, "%s: out_tokens must not be tokens", who);
  DeviceInfo di;
  kv_status st = device_info(&di);
  if (st != KV_OK) return st;
  VerifyArgs a = {out_tokens, num_accepted, new_lens, seq_lens, tokens, target_probs, draft_probs, uniform,
                  query_start, di.flags, batch, num_tokens, max_query_len, vocab, 1};
  // as many CTAs a sequence as the GPU holds at once (four of 256 threads per SM
  // are enough to keep the loads coming), while a warp has 256 weights
  while (a.cluster < kMaxCluster && 2LL * a.cluster * batch <= 4LL * di.num_sms &&
         vocab >= a.cluster * kVerifyWarps * 256)
    a.cluster *= 2;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == PAGEDKV_PROB_F32) return launch_verify<float>(a, s);
  if (dtype == PAGEDKV_PROB_BF16) return launch_verify<__nv_bfloat16>(a, s);
  return launch_verify<__half>(a, s);
}
