// Operators called with one pointer to their arguments.
//
// A call through a foreign-function interface costs by the argument (Python's
// ctypes 0.1 us each, and these operators have 9 to 33); packed into 8-byte
// slots first, 32 cost 1 us in all.
#include <limits.h>

#include <type_traits>
#include <utility>

#include "../../include/vt_paged_attn.h"

namespace vt {
namespace {

template <typename T>
bool fits(const vt_arg& a) {
  if constexpr (std::is_same_v<T, int> || std::is_enum_v<T>) return a.i >= INT_MIN && a.i <= INT_MAX;
  return true;
}

template <typename T>
T value(const vt_arg& a) {
  if constexpr (std::is_pointer_v<T>)
    return reinterpret_cast<T>(a.i);
  else if constexpr (std::is_floating_point_v<T>)
    return static_cast<T>(a.f);
  else
    return static_cast<T>(a.i);
}

template <typename... A, size_t... I>
vt_status call(vt_status (*f)(A...), const vt_arg* a, std::index_sequence<I...>) {
  return (fits<A>(a[I]) && ...) ? f(value<A>(a[I])...) : VT_ERR_INVALID_ARG;
}
template <typename... A>
vt_status call(vt_status (*f)(A...), const vt_arg* a, long long count) {
  return count == sizeof...(A) ? call(f, a, std::index_sequence_for<A...>()) : VT_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace vt

extern "C" vt_status vt_call(const vt_arg* args) {
  if (!args) return VT_ERR_INVALID_ARG;
  const vt_arg* const a = args + 2;
  const long long n = args[1].i;
  switch (args[0].i) {
    case VT_OP_STEP_TABLES: return vt::call(vt_paged_step_tables, a, n);
    case VT_OP_TREE_MASKS: return vt::call(vt_tree_masks, a, n);
    case VT_OP_NORM_ROPE: return vt::call(vt_norm_rope, a, n);
    case VT_OP_NORM_APPEND: return vt::call(vt_paged_kv_norm_append, a, n);
    case VT_OP_NORM_APPEND_FP8: return vt::call(vt_paged_kv_norm_append_fp8, a, n);
    case VT_OP_PREFILL_TREE: return vt::call(vt_paged_attn_prefill_tree, a, n);
    case VT_OP_PREFILL_TREE_FP8: return vt::call(vt_paged_attn_prefill_tree_fp8, a, n);
    case VT_OP_KEEP_PATH: return vt::call(vt_paged_kv_keep_path, a, n);
  }
  return VT_ERR_INVALID_ARG;
}
