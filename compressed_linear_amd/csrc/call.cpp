// call.cpp -- entries of cl_serving.h with their arguments in an array.
#include <cstring>
#include <type_traits>
#include <utility>

#include "cl_serving.h"
#include "internal.h"

namespace {

template <typename T>
T argument(int64_t word) {
  if constexpr (std::is_pointer_v<T>) {
    return reinterpret_cast<T>(static_cast<uintptr_t>(word));
  } else if constexpr (std::is_floating_point_v<T>) {
    double d;
    std::memcpy(&d, &word, sizeof d);
    return static_cast<T>(d);
  } else {
    return static_cast<T>(word);
  }
}

// An integer that its parameter cannot hold is refused.
template <typename T>
bool fits(int64_t word) {
  if constexpr (std::is_integral_v<T>) return static_cast<int64_t>(static_cast<T>(word)) == word;
  return true;
}

template <typename... A, size_t... I>
cl_status spread(cl_status (*f)(A...), const int64_t* args, std::index_sequence<I...>) {
  if (!(fits<A>(args[I]) && ...)) return cl::fail(CL_EINVAL, "call: an argument is out of its type's range");
  return f(argument<A>(args[I])...);
}

template <typename... A>
cl_status spread(cl_status (*f)(A...), const int64_t* args) {
  return spread(f, args, std::index_sequence_for<A...>());
}

}  // namespace

extern "C" cl_status cl_call(int32_t entry, const int64_t* args) {
  if (!args) return cl::fail(CL_EINVAL, "call: args is NULL");
  switch (entry) {
    case CL_CALL_ROPE: return spread(cl_rope, args);
    case CL_CALL_KV_APPEND: return spread(cl_kv_append, args);
    case CL_CALL_KV_READ: return spread(cl_kv_read, args);
    case CL_CALL_TREE_ATTENTION: return spread(cl_tree_attention, args);
    case CL_CALL_TOKEN_LOGPROBS: return spread(cl_token_logprobs, args);
    default: return cl::fail(CL_EINVAL, "call: unknown entry %d", entry);
  }
}
