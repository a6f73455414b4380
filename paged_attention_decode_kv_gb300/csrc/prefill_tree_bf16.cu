// Tensor-core attention of trees of drafted tokens over bf16 caches: the
// prefill's kernel with a mask for each row.
#include "prefill_tc.cuh"

namespace vt {

const PrefillVariant* tree_bf16_variant(int head_dim) {
  static const PrefillVariant table[] = {
      TcVariant<TcConfig<false, 64, 2, 64, 64, 5, 128, 4, 1, true>>::info(),
      TcVariant<TcConfig<false, 128, 2, 128, 128, 3, 128, 2, 1, true>>::info(),
      TcVariant<TcConfig<false, 256, 1, 256, 128, 3, 64, 2, 1, true>>::info(),
      TcVariant<TcConfig<false, 512, 1, 256, 128, 2, 32, 2, 1, true>>::info(),
  };
  return head_dim == 64 ? &table[0] : head_dim == 128 ? &table[1] : head_dim == 256 ? &table[2]
         : head_dim == 512 ? &table[3] : nullptr;
}

}  // namespace vt
