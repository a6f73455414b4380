// Tensor-core prefill variants for FP8 (E4M3) caches.  Codes enter the MMAs as
// they are (kind::f8f6f4, twice the bf16 rate); Q and P, which carry more
// bits, are each the sum of two E4M3 terms, so a block costs the tensor cores
// what a bf16 block does and no code is ever widened.
#include "prefill_tc.cuh"

namespace vt {

const PrefillVariant* prefill_e4m3_variant(int head_dim) {
  static const PrefillVariant table[] = {
      TcVariant<TcConfig<true, 64, 2, 64, 64, 6, 128, 6>>::info(),
      TcVariant<TcConfig<true, 128, 2, 128, 128, 5, 128, 5>>::info(),
      TcVariant<TcConfig<true, 256, 1, 256, 128, 5, 64, 4>>::info(),
  };
  return head_dim == 64 ? &table[0] : head_dim == 128 ? &table[1] : head_dim == 256 ? &table[2] : nullptr;
}

}  // namespace vt
