// Launch descriptors of the ragged prefill's kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "prefill_plan.cuh"

namespace vt {

struct PrefillVariant {
  int threads;
  int rows;         // query rows (tokens x heads of one kv head) of an item
  int tile_rows;    // rows of one tile: a tile holds tile_rows / group tokens
  int cols;         // V columns of an item
  int tensor_cores;
  int stages;
  int item_weight;  // an item's fixed cost in tokens (PrefillArgs)
  size_t smem_bytes;
  const void* func;
  cudaError_t (*launch)(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefillArgs& a,
                        int grid, cudaStream_t stream);
};

// nullptr: not taken.
const PrefillVariant* prefill_simt_variant(int head_dim);  // fp32
const PrefillVariant* prefill_bf16_variant(int head_dim);
const PrefillVariant* prefill_e4m3_variant(int head_dim);

// Joins the pieces of split items (see prefill_plan.cuh).  dtype_out: 0 bf16, 1 fp32.
cudaError_t launch_prefill_combine(const PrefillArgs& a, int grid, int rows, int tile_rows, int cols, int head_dim,
                                   int dtype_out, cudaStream_t stream);

}  // namespace vt
