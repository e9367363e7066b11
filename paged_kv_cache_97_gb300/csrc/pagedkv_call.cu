// pagedkv_call.cu -- calls with their arguments as one array.
#include <cstring>
#include <tuple>
#include <utility>

#include "pagedkv_common.cuh"

using namespace pagedkv;

namespace {

template <typename T>
T argument(int64_t x) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<uintptr_t>(x));
  } else if constexpr (std::is_same_v<T, float>) {
    const uint32_t bits = static_cast<uint32_t>(x);
    float f;
    memcpy(&f, &bits, sizeof f);
    return f;
  } else {
    return static_cast<T>(x);
  }
}

template <typename... A, size_t... I>
kv_status spread(kv_status (*f)(A...), const int64_t* a, std::index_sequence<I...>) {
  return f(argument<A>(a[I])...);
}

template <typename... A>
kv_status call(kv_status (*f)(A...), const int64_t* a, int n) {
  if (a == nullptr || n != (int)sizeof...(A))
    return fail(KV_ERR_INVALID_ARG, "pagedkv_call: %d arguments where %d are needed", n, (int)sizeof...(A));
  return spread(f, a, std::index_sequence_for<A...>{});
}

}  // namespace

extern "C" kv_status pagedkv_call(int which, const int64_t* args, int num_args) {
  switch (which) {
    case PAGEDKV_CALL_APPEND_ROTARY: return call(pagedkv_append_rotary, args, num_args);
    case PAGEDKV_CALL_APPEND_ROTARY_Q4: return call(pagedkv_append_rotary_q4, args, num_args);
    case PAGEDKV_CALL_READ_Q4: return call(pagedkv_read_q4, args, num_args);
    case PAGEDKV_CALL_ATTENTION_DECODE_Q4: return call(paged_attention_decode_q4, args, num_args);
    case PAGEDKV_CALL_ATTENTION_MULTI_Q4: return call(paged_attention_multi_q4, args, num_args);
    case PAGEDKV_CALL_VERIFY_DRAFTS: return call(pagedkv_verify_drafts, args, num_args);
    default: return fail(KV_ERR_INVALID_ARG, "pagedkv_call: no call %d", which);
  }
}
