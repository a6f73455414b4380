// Tensor-core prefill variants for FP8 (E4M3) caches.  K's codes enter the MMAs
// of Q K^T as they are (kind::f8f6f4, twice the bf16 rate) and Q, which carries
// more bits, is the sum of two E4M3 terms, so they cost the tensor cores what
// bf16 ones do.  V's codes are widened to f16 in shared memory for P V.
// The two-tile variants have 640 threads of 96 registers each at launch and spill
// 52 bytes a thread.
#include "prefill_tc.cuh"

namespace vt {

const PrefillVariant* prefill_e4m3_variant(int head_dim) {
  static const PrefillVariant table[] = {
      TcVariant<TcConfig<true, 64, 2, 64, 64, 4, 128, 3, 3>>::info(),
      TcVariant<TcConfig<true, 128, 2, 128, 128, 3, 128, 3, 2>>::info(),
      TcVariant<TcConfig<true, 256, 1, 256, 256, 2, 64, 2, 2>>::info(),
  };
  return head_dim == 64 ? &table[0] : head_dim == 128 ? &table[1] : head_dim == 256 ? &table[2] : nullptr;
}

}  // namespace vt
