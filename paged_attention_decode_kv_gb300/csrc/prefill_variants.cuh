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
  int one_weight;   // of a block of a one-tile item of a tree
  size_t smem_bytes;
  const void* func;
  cudaError_t (*launch)(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefillArgs& a,
                        int grid, cudaStream_t stream);
};

// nullptr: not taken.
const PrefillVariant* prefill_simt_variant(int head_dim);  // fp32
const PrefillVariant* prefill_bf16_variant(int head_dim);
const PrefillVariant* prefill_e4m3_variant(int head_dim);
// Trees of drafted tokens.
const PrefillVariant* tree_simt_variant(int head_dim);  // fp32
const PrefillVariant* tree_bf16_variant(int head_dim);
const PrefillVariant* tree_e4m3_variant(int head_dim);

// Joins the pieces of split items (see prefill_plan.cuh).  dtype_out: 0 bf16, 1 fp32.
cudaError_t launch_prefill_combine(const PrefillArgs& a, int grid, int rows, int tile_rows, int cols, int head_dim,
                                   int dtype_out, cudaStream_t stream);

// The same for trees on tensor cores (bf16 results), whose partials lie four columns of a tile's 128 rows after another.
cudaError_t launch_tree_combine(const PrefillArgs& a, int ctas, int rows, int cols, int head_dim, int num_sms,
                                cudaStream_t stream);

}  // namespace vt
