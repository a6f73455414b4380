// Trees of drafted tokens: their masks and positions, and the accepted
// branch's keys and values moved to consecutive slots.
//
// Masks.  A drafted token sees itself and what its parent sees.  With u_0(j)
// the parent of j and m_0(j) = {j}, m_{i+1}(j) = m_i(j) | m_i(u_i(j)) and
// u_{i+1} = u_i u_i double the ancestors known in a step: a block takes a
// sequence, a thread a row, and the steps end when no row has an ancestor
// left (log2 of the deepest branch; following parents one by one costs a
// branch's length in dependent loads).  A row's position is the context's end
// plus its ancestors.  What bounds it: those steps' latency, and of many blocks
// the launch: 64 trees of 24 to 64 tokens 3.3 us from a graph, 256 of 200 to 256
// (2.3 MB) 5.9, with words stored row by row 6.8.
//
// Accepted branches.  Bit i_r, the r-th in ascending order, of the accepted
// row's mask names the token whose rows go to place r behind the context.
// i_r >= r, and i_r' > r for r' > r, so rows moved in ascending order never
// overwrite one that is still to be read: a thread takes 16 bytes of a row
// (of keys or values, of a layer) and walks the branch, a few loads in flight.
// What bounds it: the launch, and latency: lengths, the mask with the block
// table, the rows: 8 branches in one layer 2.8 us from a graph, 64 in 16 layers
// (24.5 MB read and written) 7.5 on caches out of L2, 5.2 on the same ones again.
#include <cuda_runtime.h>
#include <stdint.h>

#include <new>

#include "../../include/vt_paged_attn.h"
#include "host_state.cuh"

namespace vt {
namespace {

constexpr int kPage = 32;
constexpr int kMaxWords = host::kMaxMaskWords;

struct Rows {
  int row0, n, L;
};

// Sequence b's rows and context; n = 0 where its starts are no rows.
__device__ __forceinline__ Rows rows_of(const int* q_starts, const int* context_lens, int b, int num_tokens) {
  const int s = q_starts[b], e = q_starts[b + 1];
  return Rows{s, s >= 0 && e > s && e <= num_tokens ? e - s : 0, context_lens[b]};
}

// ------------------------------------------------------------------- masks
struct MasksArgs {
  int* masks;
  int* positions;
  const int* parents;
  const int* q_starts;
  const int* context_lens;
  int num_tokens, words;
};

constexpr int kChunk = 8;  // words of a row that a thread holds

__global__ void tree_masks_kernel(const MasksArgs a) {
  extern __shared__ unsigned bits[];  // [words][threads + 1] (a row's words in different banks)
  const int j = threadIdx.x, threads = blockDim.x + 1;
  int* const up = reinterpret_cast<int*>(bits + a.words * threads);  // [threads]
  const Rows r = rows_of(a.q_starts, a.context_lens, blockIdx.x, a.num_tokens);
  if (r.n == 0 || r.n > 32 * a.words || r.L < r.n) return;
  const bool live = j < r.n;
  int parent = live ? a.parents[r.row0 + j] : -1;
  if (parent < 0 || parent >= j) parent = -1;
  up[j] = parent;
  for (int w = 0; w < a.words; ++w) bits[w * threads + j] = j >> 5 == w ? 1u << (j & 31) : 0u;
  while (__syncthreads_or(parent >= 0)) {
    const int next = parent >= 0 ? up[parent] : -1;
    for (int w0 = 0; w0 < a.words; w0 += kChunk) {
      unsigned x[kChunk];
#pragma unroll
      for (int w = 0; w < kChunk; ++w)
        x[w] = parent >= 0 && w0 + w < a.words ? bits[(w0 + w) * threads + parent] : 0u;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kChunk; ++w)
        if (x[w]) bits[(w0 + w) * threads + j] |= x[w];
      __syncthreads();
    }
    up[j] = parent = next;
  }
  int* const to = a.masks + static_cast<long long>(r.row0) * a.words;
  for (int i = j; i < r.n * a.words; i += blockDim.x) {
    const int row = i / a.words, w = i - row * a.words;
    to[i] = static_cast<int>(bits[w * threads + row]);
  }
  if (live && a.positions) {
    int seen = 0;
    for (int w = 0; w < a.words; ++w) seen += __popc(bits[w * threads + j]);
    a.positions[r.row0 + j] = r.L - r.n + seen - 1;
  }
}

// ------------------------------------------------------------------- accepted branches
struct KeepArgs {
  char* k_cache;
  char* v_cache;
  int* kept_lens;
  const int* accepted;
  const int* masks;
  const int* q_starts;
  const int* block_tables;
  const int* context_lens;
  int num_tokens, words, layers;
  int pieces;                // 16-byte pieces of a slot's row
  long long k_layer, v_layer;  // bytes from layer to layer
  int max_blocks, num_blocks;
  int blocks;                // of a sequence
};

constexpr int kKeepThreads = 256;
constexpr int kFlight = 4;   // rows whose loads are in flight

__global__ void __launch_bounds__(kKeepThreads) keep_path_kernel(const KeepArgs a) {
  __shared__ int from[32 * kMaxWords];  // slots to read, and to write, of the branch's tokens that move
  __shared__ int to[32 * kMaxWords];
  __shared__ int moved;
  const int b = blockIdx.x / a.blocks, part = blockIdx.x - b * a.blocks;
  const int tid = threadIdx.x, lane = tid & 31;
  const Rows r = rows_of(a.q_starts, a.context_lens, b, a.num_tokens);
  const bool whole = r.n > 0 && r.n <= 32 * a.words && r.L >= r.n &&
                     r.L <= static_cast<long long>(a.max_blocks) * kPage;
  const int base = r.L - r.n, took = a.accepted[b];
  const bool any = whole && took >= 0 && took < r.n;
  if (tid < 32) {  // the branch, by one warp: a lane a word
    // the block table from the first new token's page on, 33 pages at most, while the mask is on its way
    const int* const table = a.block_tables + static_cast<long long>(b) * a.max_blocks;
    const int page0 = base / kPage, pages = (r.L - 1) / kPage - page0 + 1;
    int page = -1, page32 = -1;
    if (any) {
      if (lane < pages) page = table[page0 + lane];
      if (pages > 32) page32 = table[page0 + 32];
    }
    auto page_of = [&](int token) {
      const int i = token / kPage - page0, p = __shfl_sync(0xffffffffu, page, i & 31);
      return i < 32 ? p : page32;
    };
    unsigned x = 0;
    if (any && lane < a.words) {
      x = static_cast<unsigned>(a.masks[static_cast<long long>(r.row0 + took) * a.words + lane]);
      const int left = r.n - 32 * lane;  // tokens there are from this word on
      if (left < 32) x = left <= 0 ? 0u : x & ((1u << left) - 1u);
    }
    const int count = __popc(x);
    int rank = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, rank, d);
      if (lane >= d) rank += o;
    }
    const int all = __shfl_sync(0xffffffffu, rank, 31);
    rank -= count;
    if (part == 0 && lane == 0) a.kept_lens[b] = whole ? base + all : r.L;
    for (; x; x &= x - 1u, ++rank) from[rank] = 32 * lane + __ffs(x) - 1;
    __syncwarp();
    // slots; tokens that are in their place already, and those of pages out of range, stay out
    int at = 0;
    for (int r0 = 0; r0 < all; r0 += 32) {
      const int i = r0 + lane, f = i < all ? from[i] : 0;
      const int ts = base + f, tt = base + (i < all ? i : 0);
      const int ps = page_of(ts), pt = page_of(tt);
      int source = -1, target = -1;
      if (i < all && f != i && ps >= 0 && ps < a.num_blocks && pt >= 0 && pt < a.num_blocks) {
        source = ps * kPage + ts % kPage;
        target = pt * kPage + tt % kPage;
      }
      const unsigned moves = __ballot_sync(0xffffffffu, source >= 0);
      if (source >= 0) {
        const int place = at + __popc(moves & ((1u << lane) - 1u));
        from[place] = source;  // (place <= i: what is still to be looked up stays)
        to[place] = target;
      }
      at += __popc(moves);
      __syncwarp();
    }
    if (lane == 0) moved = at;
  }
  __syncthreads();
  const int unit = part * kKeepThreads + tid;  // piece, keys or values, layer
  const int layer = unit / (2 * a.pieces), rest = unit - layer * 2 * a.pieces;
  if (layer >= a.layers) return;
  const bool of_v = rest >= a.pieces;
  const int piece = of_v ? rest - a.pieces : rest;
  char* const pool = (of_v ? a.v_cache + layer * a.v_layer : a.k_cache + layer * a.k_layer) + 16ll * piece;
  const long long row = 16ll * a.pieces;
  for (int i = 0; i < moved; i += kFlight) {
    uint4 x[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (i + u < moved) x[u] = *reinterpret_cast<const uint4*>(pool + from[i + u] * row);
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (i + u < moved) *reinterpret_cast<uint4*>(pool + to[i + u] * row) = x[u];
  }
}

using namespace vt::host;

size_t masks_smem(int words) { return sizeof(int) * (32 * static_cast<size_t>(words) + 1) * (words + 1); }

vt_status tree_masks(const MasksArgs& a, int num_seqs, cudaStream_t stream) {
  if (num_seqs < 0 || a.num_tokens < 0) return VT_ERR_INVALID_ARG;
  if (num_seqs == 0 || a.num_tokens == 0) return VT_OK;
  if (!a.masks || !a.parents || !a.q_starts || !a.context_lens || a.words <= 0) return VT_ERR_INVALID_ARG;
  if (!aligned(a.masks, 4) || !aligned(a.positions, 4) || !aligned(a.parents, 4) || !aligned(a.q_starts, 4) ||
      !aligned(a.context_lens, 4))
    return VT_ERR_INVALID_ARG;
  // (other blocks, and other threads of a block, still read what would be written)
  for (const int* out : {a.masks, a.positions})
    if (out && (out == a.parents || out == a.q_starts || out == a.context_lens)) return VT_ERR_INVALID_ARG;
  if (a.masks == a.positions) return VT_ERR_INVALID_ARG;
  if (a.words > kMaxWords || num_seqs > kMaxTokens || a.num_tokens > kMaxTokens) return VT_ERR_UNSUPPORTED;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int threads = 32 * a.words;
  const size_t smem = masks_smem(a.words);
  if (smem > 48 * 1024) {
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceState& ds = device_state(dev);
    const vt_status st = prepare_device(dev, ds);
    if (st != VT_OK) return st;
    const void* const func = reinterpret_cast<const void*>(&tree_masks_kernel);
    bool known = false;
    for (auto& p : ds.occupancy) known |= p.first == func;
    if (!known) {
      e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(masks_smem(kMaxWords)));
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
      ds.occupancy.emplace_back(func, 1);
    }
  }
  tree_masks_kernel<<<num_seqs, threads, smem, stream>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? VT_OK : cuda_fail(e, "tree masks launch");
}

int element_bytes(vt_dtype dtype) { return dtype == VT_F32 ? 4 : dtype == VT_BF16 ? 2 : 1; }

vt_status keep_path(KeepArgs a, int num_seqs, int num_kv_heads, int head_dim, int block_size, long long k_stride,
                    long long v_stride, cudaStream_t stream, vt_dtype dtype) {
  if (num_seqs < 0 || a.num_tokens < 0 || a.layers < 0) return VT_ERR_INVALID_ARG;
  if (num_seqs == 0) return VT_OK;
  if (!a.kept_lens || !a.accepted || !a.q_starts || !a.context_lens || !a.block_tables) return VT_ERR_INVALID_ARG;
  if (a.num_tokens > 0 && !a.masks) return VT_ERR_INVALID_ARG;
  if (dtype != VT_BF16 && dtype != VT_F32 && dtype != VT_E4M3) return VT_ERR_INVALID_ARG;
  if (a.words <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || a.max_blocks <= 0 || a.num_blocks <= 0)
    return VT_ERR_INVALID_ARG;
  if (a.layers > 0 && (!a.k_cache || !a.v_cache)) return VT_ERR_INVALID_ARG;
  // (other blocks of the sequence still read what would be written)
  for (const int* in : {a.context_lens, a.accepted, a.q_starts, a.block_tables, a.masks})
    if (a.kept_lens == in) return VT_ERR_INVALID_ARG;
  if (!aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.kept_lens, 4) || !aligned(a.accepted, 4) ||
      !aligned(a.masks, 4) || !aligned(a.q_starts, 4) || !aligned(a.block_tables, 4) || !aligned(a.context_lens, 4))
    return VT_ERR_INVALID_ARG;
  if (block_size != kPage || a.words > kMaxWords || a.num_tokens > kMaxTokens || num_seqs > kMaxTokens)
    return VT_ERR_UNSUPPORTED;
  if (static_cast<long long>(a.num_blocks) * kPage > 0x7fffffffLL ||
      static_cast<long long>(a.max_blocks) * kPage > 0x7fffffffLL)
    return VT_ERR_UNSUPPORTED;
  const int es = element_bytes(dtype);
  const long long row = static_cast<long long>(num_kv_heads) * head_dim * es;
  if (row % 16 != 0 || row > (1ll << 30)) return VT_ERR_UNSUPPORTED;
  const long long pool = static_cast<long long>(a.num_blocks) * kPage * num_kv_heads * head_dim;
  if (a.layers > 1) {
    if (k_stride < pool || v_stride < pool || k_stride * es % 16 != 0 || v_stride * es % 16 != 0)
      return VT_ERR_INVALID_ARG;
    a.k_layer = k_stride * es;
    a.v_layer = v_stride * es;
  }
  a.pieces = static_cast<int>(row / 16);
  const long long units = 2ll * a.pieces * a.layers;
  const long long blocks = (units + kKeepThreads - 1) / kKeepThreads;
  if (units > 0x7fffffffLL - kKeepThreads || blocks * num_seqs > 0x7fffffffLL) return VT_ERR_UNSUPPORTED;
  a.blocks = blocks > 0 ? static_cast<int>(blocks) : 1;
  keep_path_kernel<<<static_cast<unsigned>(a.blocks) * num_seqs, kKeepThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VT_OK : cuda_fail(e, "keep path launch");
}

}  // namespace
}  // namespace vt

extern "C" {

vt_status vt_tree_masks(int32_t* masks, int32_t* positions, const int32_t* parents, const int32_t* q_starts,
                        const int32_t* context_lens, int num_seqs, int num_tokens, int mask_words,
                        vt_stream_t stream) {
  try {
    return vt::tree_masks(vt::MasksArgs{masks, positions, parents, q_starts, context_lens, num_tokens, mask_words},
                          num_seqs, reinterpret_cast<cudaStream_t>(stream));
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

vt_status vt_paged_kv_keep_path(void* k_cache, void* v_cache, int32_t* kept_lens, const int32_t* accepted,
                                const int32_t* masks, const int32_t* q_starts, const int32_t* block_tables,
                                const int32_t* context_lens, int num_seqs, int num_tokens, int mask_words,
                                int num_layers, int num_kv_heads, int head_dim, int block_size,
                                long long k_layer_stride, long long v_layer_stride, vt_stream_t stream,
                                int max_blocks_per_seq, int num_blocks, vt_dtype dtype) {
  try {
    return vt::keep_path(vt::KeepArgs{static_cast<char*>(k_cache), static_cast<char*>(v_cache), kept_lens, accepted,
                                      masks, q_starts, block_tables, context_lens, num_tokens, mask_words, num_layers,
                                      0, 0, 0, max_blocks_per_seq, num_blocks, 1},
                         num_seqs, num_kv_heads, head_dim, block_size, k_layer_stride, v_layer_stride,
                         reinterpret_cast<cudaStream_t>(stream), dtype);
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

}  // extern "C"
