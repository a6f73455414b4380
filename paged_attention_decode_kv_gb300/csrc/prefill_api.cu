// C entry points of the ragged prefill: checks, scratch, tensor maps, launch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <new>

#include "../../include/vt_paged_attn.h"
#include "decode_kernel.cuh"
#include "host_state.cuh"
#include "prefill_variants.cuh"

namespace vt {
namespace {

using namespace vt::host;

// A CTA's least share is one 128-key block: calls too small for the GPU are over
// soonest when every block and item has a CTA of its own (8 new tokens, 16 q /
// 4 kv heads of 128: 10 us; with 4 blocks 19 us).  But each piece of an item
// costs the combine 0.3 us, so where items have more than 8 blocks on average
// it is two blocks (1 token over 4000: 18 us; with one block 23 us, with four
// 19).  On CUDA cores a block takes longer than that, and one is always best.
constexpr long long kLongItem = 8 * kPfBlock;

struct PrefillCall {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* q_starts;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size;
  float scale;
  int window;
  cudaStream_t stream;
  int max_blocks, num_blocks;
  vt_dtype dtype;
  // trees of drafted tokens
  bool tree;
  const int32_t* masks;
  int mask_words;
};

const PrefillVariant* find_prefill(int head_dim, vt_dtype dtype, bool tree) {
  if (tree) {
    if (dtype == VT_F32) return tree_simt_variant(head_dim);
    if (dtype == VT_BF16) return tree_bf16_variant(head_dim);
    return tree_e4m3_variant(head_dim);
  }
  if (dtype == VT_F32) return prefill_simt_variant(head_dim);
  if (dtype == VT_BF16) return prefill_bf16_variant(head_dim);
  return prefill_e4m3_variant(head_dim);
}

vt_status encode(CUtensorMap* m, CUtensorMapDataType type, bool wide_rows, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
  auto fn = encode_fn();
  if (!fn) {
    g_last_cuda_error = "cuTensorMapEncodeTiled entry point unavailable";
    return VT_ERR_CUDA;
  }
  const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
  const CUresult r = fn(m, type, rank, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        wide_rows ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    g_last_cuda_error = "cuTensorMapEncodeTiled failed (code " + std::to_string(static_cast<int>(r)) + ")";
    return VT_ERR_CUDA;
  }
  return VT_OK;
}

// Queries as (64 columns, head of the group, token, column block, kv head):
// one box is the rows of a tile, token by token, for one column block.
vt_status query_map(CUtensorMap* m, const PrefillCall& c, int group) {
  const cuuint64_t D = c.head_dim, row = static_cast<cuuint64_t>(c.num_q_heads) * D * 2;
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(group), static_cast<cuuint64_t>(c.num_tokens), D / 64,
                              static_cast<cuuint64_t>(c.num_kv_heads)};
  const cuuint64_t strides[4] = {D * 2, row, 128, static_cast<cuuint64_t>(group) * D * 2};
  const cuuint32_t box[5] = {64u, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group), 1u, 1u};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, true, c.q, 5, dims, strides, box);
}

// A pool as (columns of a block, token, column block, kv head), blocks of 64
// bf16 columns or 128 codes (64 at head_dim 64): one box is one column block of
// a page, so that a stage's four pages lie one after another.
vt_status pool_map(CUtensorMap* m, const void* pool, const PrefillCall& c) {
  const bool fp8 = c.dtype == VT_E4M3;
  const cuuint64_t es = fp8 ? 1 : 2, D = c.head_dim, cols = fp8 && D >= 128 ? 128 : 64;
  const cuuint64_t row = static_cast<cuuint64_t>(c.num_kv_heads) * D * es;
  const cuuint64_t dims[4] = {cols, static_cast<cuuint64_t>(c.num_blocks) * kPfPage, D / cols,
                              static_cast<cuuint64_t>(c.num_kv_heads)};
  const cuuint64_t strides[3] = {row, cols * es, D * es};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(kPfPage), 1u, 1u};
  return encode(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cols * es == 128, pool, 4,
                dims, strides, box);
}

vt_status validate(const PrefillCall& c) {
  if (c.num_seqs < 0 || c.num_tokens < 0) return VT_ERR_INVALID_ARG;
  if (!c.out || !c.q || !c.k_cache || !c.v_cache || !c.q_starts || !c.block_tables || !c.context_lens)
    return VT_ERR_INVALID_ARG;
  if (c.tree && (!c.masks || !aligned(c.masks, 4) || c.mask_words <= 0)) return VT_ERR_INVALID_ARG;
  if (c.out == c.q) return VT_ERR_INVALID_ARG;  // rows are read again after others' results are written
  if (c.dtype != VT_BF16 && c.dtype != VT_F32 && c.dtype != VT_E4M3) return VT_ERR_INVALID_ARG;
  if (c.dtype == VT_E4M3 && (!c.k_scale || !c.v_scale || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)))
    return VT_ERR_INVALID_ARG;
  if (c.num_q_heads <= 0 || c.num_kv_heads <= 0 || c.num_q_heads % c.num_kv_heads != 0) return VT_ERR_INVALID_ARG;
  if (c.max_blocks <= 0 || c.num_blocks <= 0 || c.block_size <= 0 || c.head_dim <= 0) return VT_ERR_INVALID_ARG;
  if (!std::isfinite(c.scale)) return VT_ERR_INVALID_ARG;
  if (!aligned(c.out, 16) || !aligned(c.q, 16) || !aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) ||
      !aligned(c.q_starts, 4) || !aligned(c.block_tables, 4) || !aligned(c.context_lens, 4))
    return VT_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256 && c.head_dim != 512) return VT_ERR_UNSUPPORTED;
  if (c.block_size != kPfPage) return VT_ERR_UNSUPPORTED;
  if (c.num_tokens > kMaxTokens || c.num_seqs > kMaxTokens) return VT_ERR_UNSUPPORTED;
  if (static_cast<long long>(c.num_blocks) * kPfPage > 0x7fffffffLL ||
      static_cast<long long>(c.max_blocks) * kPfPage > 0x7fffffffLL)
    return VT_ERR_UNSUPPORTED;
  if (c.tree && c.mask_words > kMaxMaskWords) return VT_ERR_UNSUPPORTED;
  const PrefillVariant* v = find_prefill(c.head_dim, c.dtype, c.tree);
  if (!v || c.num_q_heads / c.num_kv_heads > v->tile_rows) return VT_ERR_UNSUPPORTED;
  return VT_OK;
}

size_t splits_bytes(int grid) { return align_up(sizeof(PrefillSplit) * static_cast<size_t>(grid), 256); }
size_t ml_bytes(const PrefillVariant& v, int grid) { return sizeof(float2) * 2 * static_cast<size_t>(grid) * v.rows; }
size_t part_bytes(const PrefillVariant& v, int grid) {
  return sizeof(float) * 2 * static_cast<size_t>(grid) * v.rows * v.cols;
}
size_t scratch_bytes(const PrefillVariant& v, int grid) {
  return splits_bytes(grid) + ml_bytes(v, grid) + part_bytes(v, grid);
}

// Caller holds g_mutex.
vt_status prepare(DeviceState& ds, const PrefillVariant& v, int* per_sm) {
  for (auto& p : ds.occupancy)
    if (p.first == v.func) {
      *per_sm = p.second;
      return VT_OK;
    }
  cudaError_t e = cudaFuncSetAttribute(v.func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(v.smem_bytes));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, v.func, v.threads, v.smem_bytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
  if (n < 1) {
    g_last_cuda_error = "prefill kernel variant cannot be resident on this device";
    return VT_ERR_UNSUPPORTED;
  }
  if (v.tensor_cores) n = 1;  // each CTA takes all of an SM's tensor memory
  ds.occupancy.emplace_back(v.func, n);
  *per_sm = n;
  return VT_OK;
}

// The call's scratch: [status 256 B | splits | ml | part], or in the caller's
// area [status | counters of decodes ... | splits | ml | part], at its end: the
// counters, which larger decodes extend and which keep their contents between
// calls, stay off what a captured prefill names there (captured_tail).
// Caller holds g_mutex.
vt_status scratch(DeviceState& ds, size_t need, cudaStream_t stream, char** status, char** base, int* source) {
  auto capturing = [&](bool* yes) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing(stream, &cap);
    *yes = cap != cudaStreamCaptureStatusNone;
    return e == cudaSuccess ? VT_OK : cuda_fail(e, "cudaStreamIsCapturing");
  };
  bool in_capture = false;
  if (ds.user.base) {
    const size_t at = kStatusBytes + align_up(ds.user.counters_cap, 256);
    if (at + need > ds.user.bytes) {
      g_last_cuda_error = "vt_paged_attn_prefill: this call needs " + std::to_string(at + need) +
                          " bytes of workspace; the caller's workspace holds " + std::to_string(ds.user.bytes);
      return VT_ERR_SCRATCH_LIMIT;
    }
    const vt_status st = capturing(&in_capture);
    if (st != VT_OK) return st;
    const size_t from = (ds.user.bytes - need) / 256 * 256;
    if (in_capture) ds.user.captured_tail = std::max(ds.user.captured_tail, ds.user.bytes - from);
    *status = ds.user.base;
    *base = ds.user.base + from;
    *source = 1;
    return VT_OK;
  }
  if (ds.prefill.bytes < kStatusBytes + need) {
    const vt_status st = capturing(&in_capture);
    if (st != VT_OK) return st;
    if (in_capture) {
      g_last_cuda_error = "vt_paged_attn_prefill: the first call with this head_dim allocates scratch; make it "
                          "outside stream capture";
      return VT_ERR_SCRATCH_LIMIT;
    }
    void* p = nullptr;
    const size_t bytes = kStatusBytes + need;
    cudaError_t e = cudaMalloc(&p, bytes);
    if (e != cudaSuccess) {
      cudaGetLastError();
      g_last_cuda_error = std::string("cudaMalloc: ") + cudaGetErrorString(e);
      return VT_ERR_OOM;
    }
    e = cudaMemsetAsync(p, 0, kStatusBytes, stream);
    if (e != cudaSuccess) {
      cudaFree(p);
      return cuda_fail(e, "cudaMemsetAsync");
    }
    if (ds.prefill.base) ds.prefill_retired.push_back(ds.prefill.base);
    ds.prefill = Scratch{static_cast<char*>(p), bytes, 0};
  }
  *status = ds.prefill.base;
  *base = ds.prefill.base + kStatusBytes;
  *source = 0;
  return VT_OK;
}

vt_status prefill(const PrefillCall& c) {
  if (c.num_seqs == 0 || c.num_tokens == 0) return VT_OK;
  vt_status st = validate(c);
  if (st != VT_OK) return st;
  const PrefillVariant& v = *find_prefill(c.head_dim, c.dtype, c.tree);
  int dev = 0, per_sm = 0, source = 0, grid = 0, sms = 0;
  char* status = nullptr;
  char* base = nullptr;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceState& ds = device_state(dev);
    st = prepare_device(dev, ds);
    if (st != VT_OK) return st;
    st = prepare(ds, v, &per_sm);
    if (st != VT_OK) return st;
    sms = ds.num_sms;
    grid = g_override_grid > 0 ? g_override_grid : sms * per_sm;
    st = scratch(ds, scratch_bytes(v, grid), c.stream, &status, &base, &source);
    if (st != VT_OK) return st;
  }

  PrefillArgs a{};
  a.out = c.out;
  a.q = c.q;
  a.k_cache = c.k_cache;
  a.v_cache = c.v_cache;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.q_starts = c.q_starts;
  a.block_tables = c.block_tables;
  a.context_lens = c.context_lens;
  a.num_seqs = c.num_seqs;
  a.num_tokens = c.num_tokens;
  a.num_q_heads = c.num_q_heads;
  a.num_kv_heads = c.num_kv_heads;
  a.group = c.num_q_heads / c.num_kv_heads;
  a.max_blocks = c.max_blocks;
  a.num_blocks = c.num_blocks;
  // (a window no context can fill is none, and no sum with it overflows)
  a.window = c.window > 0 && c.window < c.max_blocks * kPfPage ? c.window : 0;
  a.masks = c.masks;
  a.mask_words = c.mask_words;
  // (a hidden score is -inf, which a scale of 0 would turn into NaN: 1e-37 leaves any finite score at 0)
  a.scale_log2 = c.scale == 0.f ? 1e-37f : std::fabs(c.scale) * 1.4426950408889634f;
  a.neg_scale = c.scale < 0.f;
  a.tile_tokens = v.rows / v.tile_rows * (v.tile_rows / a.group);
  // Division by T = tile_tokens: with s = ceil(log2 T), 2^(31 + s) < mul T <= 2^(31 + s) + 2^s.
  unsigned log2_up = 0;
  while ((1u << log2_up) < static_cast<unsigned>(a.tile_tokens)) ++log2_up;
  a.tile_shift = 31 + log2_up;
  a.tile_mul = static_cast<unsigned>((1ull << a.tile_shift) / static_cast<unsigned>(a.tile_tokens) + 1);
  a.group_mul = (65535 + a.group) / a.group;  // (128 rows x an excess below 128 stay below 2^16)
  a.v_parts = c.head_dim / v.cols;
  a.item_weight = v.item_weight;
  a.one_tile = v.tensor_cores && v.rows > v.tile_rows ? v.tile_rows / a.group : 0;
  a.one_weight = v.one_weight;
  a.one_mul = ~0ull / static_cast<unsigned>(v.one_weight) + 1;
  const bool set = g_override_min_units > 0;
  a.min_weight = kPfBlock * (set ? std::min(g_override_min_units, 1 << 20) : 1);
  const long long items = (static_cast<long long>(c.num_tokens) / a.tile_tokens + c.num_seqs) * c.num_kv_heads * a.v_parts;
  a.long_total = set || !v.tensor_cores ? std::numeric_limits<long long>::max() : items * (v.item_weight + kLongItem);
  a.status = reinterpret_cast<unsigned*>(status);
  a.splits = reinterpret_cast<PrefillSplit*>(base);
  a.ml = reinterpret_cast<float2*>(base + splits_bytes(grid));
  a.part = reinterpret_cast<float*>(base + splits_bytes(grid) + ml_bytes(v, grid));
  a.wait_limit = static_cast<unsigned>(
      g_test_wait_limit > 0 ? std::min(g_test_wait_limit, kWaitLimitCycles) : kWaitLimitCycles);
  a.withhold_cta = g_test_withhold_tile >= 0 ? g_test_withhold_cta : -1;
  a.withhold_block = g_test_withhold_tile;

  CUtensorMap tq{}, tk{}, tv{};
  if (v.tensor_cores) {
    st = query_map(&tq, c, a.group);
    if (st == VT_OK) st = pool_map(&tk, c.k_cache, c);
    if (st == VT_OK) st = pool_map(&tv, c.v_cache, c);
    if (st != VT_OK) return st;
  }
  e = v.launch(tq, tk, tv, a, grid, c.stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
  if (c.tree && v.tensor_cores)
    e = launch_tree_combine(a, grid, v.rows, v.cols, c.head_dim, sms, c.stream);
  else
    e = launch_prefill_combine(a, grid, v.rows, v.tile_rows, v.cols, c.head_dim, c.dtype == VT_F32 ? 1 : 0, c.stream);
  if (e != cudaSuccess) return cuda_fail(e, "prefill combine launch");

  vt_plan& r = g_last_plan;
  r = vt_plan{};
  r.grid_ctas = grid;
  r.ctas_per_sm = per_sm;
  r.num_sms = sms;
  r.consumer_warps = v.threads / 32;
  r.tensor_cores = v.tensor_cores;
  r.stages = v.stages;
  r.group_tile = v.rows;
  r.subgroups = 1;
  r.min_units_per_cta = a.min_weight / kPfBlock;
  r.head_dim = c.head_dim;
  r.dtype = c.dtype;
  r.smem_bytes = v.smem_bytes;
  r.workspace_bytes = kStatusBytes + scratch_bytes(v, grid);
  r.scratch_source = source;
  g_have_plan = true;
  return VT_OK;
}

}  // namespace
}  // namespace vt

extern "C" {

vt_status vt_paged_attn_prefill(void* out, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* q_starts, const int32_t* block_tables, const int32_t* context_lens,
                                int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                int block_size, float scale, int window, vt_stream_t stream, int max_blocks_per_seq,
                                int num_blocks, vt_dtype dtype) {
  if (dtype == VT_E4M3) return VT_ERR_INVALID_ARG;
  try {
    return vt::prefill(vt::PrefillCall{out, q, k_cache, v_cache, nullptr, nullptr, q_starts, block_tables,
                                       context_lens, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                       block_size, scale, window, reinterpret_cast<cudaStream_t>(stream),
                                       max_blocks_per_seq, num_blocks, dtype, false, nullptr, 0});
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

vt_status vt_paged_attn_prefill_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                    const float* k_scale, const float* v_scale, const int32_t* q_starts,
                                    const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                                    int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                    float scale, int window, vt_stream_t stream, int max_blocks_per_seq,
                                    int num_blocks) {
  try {
    return vt::prefill(vt::PrefillCall{out, q, k_cache, v_cache, k_scale, v_scale, q_starts, block_tables,
                                       context_lens, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                       block_size, scale, window, reinterpret_cast<cudaStream_t>(stream),
                                       max_blocks_per_seq, num_blocks, VT_E4M3, false, nullptr, 0});
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

vt_status vt_paged_attn_prefill_tree(void* out, const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* masks, const int32_t* q_starts, const int32_t* block_tables,
                                     const int32_t* context_lens, int num_seqs, int num_tokens, int mask_words,
                                     int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale,
                                     int window, vt_stream_t stream, int max_blocks_per_seq, int num_blocks,
                                     vt_dtype dtype) {
  if (dtype == VT_E4M3) return VT_ERR_INVALID_ARG;
  try {
    return vt::prefill(vt::PrefillCall{out, q, k_cache, v_cache, nullptr, nullptr, q_starts, block_tables,
                                       context_lens, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                       block_size, scale, window, reinterpret_cast<cudaStream_t>(stream),
                                       max_blocks_per_seq, num_blocks, dtype, true, masks, mask_words});
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

vt_status vt_paged_attn_prefill_tree_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                         const float* k_scale, const float* v_scale, const int32_t* masks,
                                         const int32_t* q_starts, const int32_t* block_tables,
                                         const int32_t* context_lens, int num_seqs, int num_tokens, int mask_words,
                                         int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                         float scale, int window, vt_stream_t stream, int max_blocks_per_seq,
                                         int num_blocks) {
  try {
    return vt::prefill(vt::PrefillCall{out, q, k_cache, v_cache, k_scale, v_scale, q_starts, block_tables,
                                       context_lens, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                       block_size, scale, window, reinterpret_cast<cudaStream_t>(stream),
                                       max_blocks_per_seq, num_blocks, VT_E4M3, true, masks, mask_words});
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

size_t vt_paged_attn_prefill_workspace_bytes(int head_dim, vt_dtype dtype) {
  using namespace vt;
  if (!find_prefill(head_dim, dtype, false)) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  try {
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceState& ds = device_state(dev);
    if (prepare_device(dev, ds) != VT_OK) return 0;
    size_t need = 0;
    for (const bool tree : {false, true}) {  // (each has an occupancy of its own)
      const PrefillVariant* v = find_prefill(head_dim, dtype, tree);
      int per_sm = 0;
      if (!v) continue;
      if (prepare(ds, *v, &per_sm) != VT_OK) return 0;
      const int grid = g_override_grid > 0 ? g_override_grid : ds.num_sms * per_sm;
      need = std::max(need, kStatusBytes + scratch_bytes(*v, grid));
    }
    return need;
  } catch (const std::bad_alloc&) {
    return 0;
  }
}

}  // extern "C"
