// Joins the pieces of split items of drafted trees (bf16 results): with
// (m_k, l_k, o_k) of an item's pieces, in piece order,
//   m = max m_k,   out = sum 2^(m_k - m) o_k / sum 2^(m_k - m) l_k,
// in one pass with a running m.
//
// What bounds it: a launch and two dependent latencies (the splits, the pieces)
// where there are few items, the partials' bytes in L2 where there are many.  So
// the rows of all split items are dealt out evenly over the grid, eight rows by
// 32 columns a warp, and a warp has eight pieces' loads in flight; a partial
// lies as the prefill's threads hold it, four columns of a tile's 128 rows after
// another, which both sides read and write in whole lines.  (With the causal
// prefill's combine, a block for each CTA and 32 rows of it, one tree of 26 tokens
// over a context of 3800, 16 q / 4 kv heads of 64, took 15.8 us a call, now 13.7,
// and 16 trees at head_dim 256 with a window of 1024 24.4, now 19.2.  Four lanes a
// row with every fourth piece each, for more than eight pieces, took 0.4 off the
// first and added 0.3 to the second.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "decode_kernel.cuh"  // ex2, pack_bf16
#include "prefill_variants.cuh"

namespace vt {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8, kCols = 32;  // of a warp's unit
constexpr int kFlight = 8;            // pieces

template <int COLS>
__global__ void __launch_bounds__(kThreads) tree_combine_kernel(const PrefillArgs a, int ctas, int rows, int head_dim) {
  __shared__ PrefillSplit split[kThreads];
  __shared__ int start[kThreads + 1];  // units of the splits before
  __shared__ int of_warp[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kColUnits = COLS / kCols;
  grid_dependency_wait();
  for (int c0 = 0; c0 < ctas; c0 += kThreads) {
    PrefillSplit sp{};
    if (c0 + tid < ctas) sp = a.splits[c0 + tid];
    const int units = sp.pieces > 0 ? (sp.ntok * a.group + kRows - 1) / kRows * kColUnits : 0;
    int sum = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    if (c0 > 0) __syncthreads();  // the last window is done with
    if (lane == 31) of_warp[warp] = sum;
    __syncthreads();
    for (int i = 0; i < warp; ++i) sum += of_warp[i];
    split[tid] = sp;
    start[tid + 1] = sum;
    if (tid == 0) start[0] = 0;
    __syncthreads();
    const int total = start[kThreads];
#pragma unroll 1
    for (int u = blockIdx.x * (kThreads / 32) + warp; u < total; u += gridDim.x * (kThreads / 32)) {
      int lo = 0, hi = kThreads;  // start[lo] <= u < start[hi]
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= u)
          lo = mid;
        else
          hi = mid;
      }
      const PrefillSplit& it = split[lo];
      const int unit = u - start[lo];
      const int v = unit / kColUnits * kRows + (lane & 7);  // row of the item: token, head
      const int col = unit % kColUnits * kCols + (lane >> 3) * 8;
      const int tok = v / a.group, g = v - tok * a.group;
      const bool valid = tok < it.ntok;
      const int tile_toks = 128 / a.group, tile = tok / tile_toks;
      const int row = (tok - tile * tile_toks) * a.group + g;  // of the tile
      const int c = c0 + lo, pieces = it.pieces;
      float m = -CUDART_INF_F, l = 0.f;
      float o[8] = {};
      bool bad = false;
#pragma unroll 1
      for (int p0 = 0; p0 < pieces && valid; p0 += kFlight) {
        float2 ml[kFlight];
        float4 x[kFlight][2];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          ml[i] = make_float2(-CUDART_INF_F, 0.f);
          if (p0 + i < pieces) {
            const long long rec = p0 + i == 0 ? 2ll * c : 2ll * (c + p0 + i) + 1;
            ml[i] = a.ml[rec * rows + tile * 128 + row];
            const float4* src = reinterpret_cast<const float4*>(a.part + (rec * rows + tile * 128) * COLS) + col / 4 * 128 + row;
            x[i][0] = src[0];
            x[i][1] = src[128];
          }
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          bad |= isnan(ml[i].x);
          top = fmaxf(top, ml[i].x);
        }
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        const float keep = ex2(m - ref);
        m = top;
        l *= keep;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= keep;
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const float f = ex2(ml[i].x - ref);
          l += f * ml[i].y;
          if (ml[i].x == -CUDART_INF_F) continue;  // nothing attended there, nothing written (a weight of 0 still
                                                   // makes NaN of a value that is not finite)
          o[0] += f * x[i][0].x, o[1] += f * x[i][0].y, o[2] += f * x[i][0].z, o[3] += f * x[i][0].w;
          o[4] += f * x[i][1].x, o[5] += f * x[i][1].y, o[6] += f * x[i][1].z, o[7] += f * x[i][1].w;
        }
      }
      if (valid) {
        // (a row that sees no key is 0)
        const float inv = bad ? CUDART_NAN_F : m == -CUDART_INF_F ? 0.f : 1.f / l;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                             (static_cast<long long>(it.row0 + tok) * a.num_q_heads + it.head * a.group + g) * head_dim +
                             it.part * COLS + col;
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                                                    pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
      }
    }
  }
}

}  // namespace

cudaError_t launch_tree_combine(const PrefillArgs& a, int ctas, int rows, int cols, int head_dim, int num_sms,
                                cudaStream_t stream) {
  // a programmatic dependent, as the prefill's combine is
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_sms);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cols == 64    ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<64>, a, ctas, rows, head_dim)
         : cols == 128 ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<128>, a, ctas, rows, head_dim)
                       : cudaLaunchKernelEx(&cfg, tree_combine_kernel<256>, a, ctas, rows, head_dim);
}

}  // namespace vt
