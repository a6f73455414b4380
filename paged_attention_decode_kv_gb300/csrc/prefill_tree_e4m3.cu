// Tensor-core attention of trees of drafted tokens over FP8 (E4M3) caches: the
// prefill's kernel with a mask for each row.  The two-tile variants spill 56
// (head_dim 64) and 52 bytes a thread.
#include "prefill_tc.cuh"

namespace vt {

const PrefillVariant* tree_e4m3_variant(int head_dim) {
  static const PrefillVariant table[] = {
      TcVariant<TcConfig<true, 64, 2, 64, 64, 4, 128, 3, 3, true>>::info(),
      TcVariant<TcConfig<true, 128, 2, 128, 128, 3, 128, 3, 2, true>>::info(),
      TcVariant<TcConfig<true, 256, 1, 256, 256, 2, 64, 2, 2, true>>::info(),
  };
  return head_dim == 64 ? &table[0] : head_dim == 128 ? &table[1] : head_dim == 256 ? &table[2] : nullptr;
}

}  // namespace vt
