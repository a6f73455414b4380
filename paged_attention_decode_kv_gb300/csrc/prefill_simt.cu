// Ragged prefill on CUDA cores (fp32 storage), and the combine of split items.
//
// Per item: S = Q K^T, online softmax, O += P V with everything in fp32, 64
// query rows against one 32-token page at a time.  Bound by the FMA pipes
// (4 D flop a row and key): each of 256 threads holds 4 rows x 2 keys of S
// and 4 rows x D / 16 columns of O in registers, so a 16-byte shared load
// feeds at least 5 FMAs a lane; rows of Q and P are read as broadcasts and K
// rows are padded by 16 bytes, so loads have no bank conflicts.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "decode_kernel.cuh"  // e4m3x4_to_f16, ex2, packs
#include "prefill_variants.cuh"

namespace vt {
namespace {

constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 64;

template <int D>
struct SimtSmem {
  float q[kSimtRows][D + 4];
  float k[kPfPage][D + 4];
  float v[kPfPage][D];
  float p[kSimtRows][kPfPage + 4];
  int bad;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ void store_part(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

template <int D>
__global__ void __launch_bounds__(kSimtThreads) prefill_simt_kernel(const PrefillArgs a) {
  extern __shared__ char raw[];
  SimtSmem<D>& s = *reinterpret_cast<SimtSmem<D>*>(raw);
  const int tid = threadIdx.x;
  const int ty = tid >> 4, tx = tid & 15;  // rows 4 ty..+3; keys tx, tx + 16; columns 4 tx + 64 c
  constexpr int NC = D / 64;
  if (tid == 0) a.splits[blockIdx.x].pieces = 0;
  PfWalk w;
  pf_begin(a, tid & 31, w);  // each warp for itself
  PfItem it;
  const float sign = a.neg_scale ? -1.f : 1.f;
  while (w.next(a, it)) {
    __syncthreads();  // the previous item's tiles are done with
    if (tid == 0) s.bad = it.bad;
    const int rows = it.ntok * a.group;
    for (int i = tid; i < kSimtRows * (D / 4); i += kSimtThreads) {
      const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int t = r / a.group, g = r - t * a.group;
        x = load4(static_cast<const float*>(a.q) +
                  (static_cast<long long>(it.row0 + t) * a.num_q_heads + it.head * a.group + g) * D + c);
        x.x *= sign, x.y *= sign, x.z *= sign, x.w *= sign;
      }
      *reinterpret_cast<float4*>(&s.q[r][c]) = x;
    }
    float m[4], l[4];
    float4 o[4][NC];
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
      pos[i] = it.pos0 + min((ty * 4 + i) / a.group, it.ntok - 1);
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int first = it.lo + it.kb0 * kPfBlock;
    const int last = min(it.hi, it.lo + it.kb1 * kPfBlock);
    for (int t0 = first; t0 < last; t0 += kPfPage) {
      int page = a.block_tables[static_cast<long long>(it.b) * a.max_blocks + t0 / kPfPage];
      if (page < 0 || page >= a.num_blocks) {
        if (tid == 0) s.bad = 1;
        page = 0;
      }
      __syncthreads();
      // slots outside [lo_exact, last) hold nothing a row may use: zeros
      for (int i = tid; i < kPfPage * (D / 4); i += kSimtThreads) {
        const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
        const int t = t0 + r;
        float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
        if (t >= it.lo_exact && t < last) {
          const long long at = ((static_cast<long long>(page) * kPfPage + r) * a.num_kv_heads + it.head) * D + c;
          kx = load4(static_cast<const float*>(a.k_cache) + at);
          vx = load4(static_cast<const float*>(a.v_cache) + at);
        }
        *reinterpret_cast<float4*>(&s.k[r][c]) = kx;
        *reinterpret_cast<float4*>(&s.v[r][c]) = vx;
      }
      __syncthreads();
      float x[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k0 = load4(&s.k[tx][d]), k1 = load4(&s.k[tx + 16][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 q = load4(&s.q[ty * 4 + i][d]);
          x[i][0] += q.x * k0.x;
          x[i][0] += q.y * k0.y;
          x[i][0] += q.z * k0.z;
          x[i][0] += q.w * k0.w;
          x[i][1] += q.x * k1.x;
          x[i][1] += q.y * k1.y;
          x[i][1] += q.z * k1.z;
          x[i][1] += q.w * k1.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = -CUDART_INF_F;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = t0 + tx + 16 * e;
          const bool seen = t <= pos[i] && t < last && (a.window == 0 || t > pos[i] - a.window);
          x[i][e] = seen ? x[i][e] * a.scale_log2 : -CUDART_INF_F;
          top = fmaxf(top, x[i][e]);
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(m[i], top);
        const float mb = mn == -CUDART_INF_F ? 0.f : mn;
        const float keep = exp2f(m[i] - mb);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = exp2f(x[i][e] - mb);
          sum += p;
          s.p[ty * 4 + i][tx + 16 * e] = p;
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[i] = l[i] * keep + sum;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          o[i][c].x *= keep;
          o[i][c].y *= keep;
          o[i][c].z *= keep;
          o[i][c].w *= keep;
        }
      }
      __syncwarp();  // a row group's weights are written and read by one warp
      // Where some row sees only part of the page, weights of 0 take no part:
      // 0 times a value that is not finite would be NaN.
      const bool partial = t0 + kPfPage > it.pos0 + 1 || (a.window > 0 && t0 < it.hi - a.window);
      if (partial) {
#pragma unroll 1
        for (int t = 0; t < kPfPage; ++t) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = load4(&s.v[t][4 * tx + 64 * c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float pe = s.p[ty * 4 + i][t];
              if (pe != 0.f) {
                o[i][c].x += pe * v.x;
                o[i][c].y += pe * v.y;
                o[i][c].z += pe * v.z;
                o[i][c].w += pe * v.w;
              }
            }
          }
        }
        continue;
      }
#pragma unroll 2
      for (int t = 0; t < kPfPage; t += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = load4(&s.p[ty * 4 + i][t]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = load4(&s.v[t + e][4 * tx + 64 * c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float pe = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
              o[i][c].x += pe * v.x;
              o[i][c].y += pe * v.y;
              o[i][c].z += pe * v.z;
              o[i][c].w += pe * v.w;
            }
          }
        }
      }
    }
    __syncthreads();
    const bool bad = s.bad != 0;
    const bool split = it.kb0 > 0 || it.pieces > 0;
    const long long slot = 2ll * blockIdx.x + (it.kb0 > 0 ? 1 : 0);
    if (it.pieces > 0 && tid == 0)
      a.splits[blockIdx.x] = PrefillSplit{it.pieces, it.row0, it.ntok, it.head, it.part};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= rows) continue;
      if (split) {
        float* dst = a.part + (slot * kSimtRows + r) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c) store_part(dst + 4 * tx + 64 * c, o[i][c]);
        if (tx == 0) a.ml[slot * kSimtRows + r] = make_float2(bad ? CUDART_NAN_F : m[i], l[i]);
      } else {
        const int t = r / a.group, g = r - t * a.group;
        float* dst = static_cast<float*>(a.out) +
                     (static_cast<long long>(it.row0 + t) * a.num_q_heads + it.head * a.group + g) * D;
        const float inv = bad ? CUDART_NAN_F : 1.f / l[i];
#pragma unroll
        for (int c = 0; c < NC; ++c)
          store_part(dst + 4 * tx + 64 * c,
                     make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv));
      }
    }
  }
}

template <int D>
struct SimtVariant {
  static cudaError_t launch(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const PrefillArgs& a, int grid,
                            cudaStream_t stream) {
    prefill_simt_kernel<D><<<grid, kSimtThreads, sizeof(SimtSmem<D>), stream>>>(a);
    return cudaGetLastError();
  }
  static PrefillVariant info() {
    return PrefillVariant{kSimtThreads, kSimtRows, kSimtRows, D, 0, 1, sizeof(SimtSmem<D>),
                          reinterpret_cast<const void*>(&prefill_simt_kernel<D>), &launch};
  }
};

// ---------------------------------------------------------------------------
// Combine: with (m_k, l_k, o_k) of an item's pieces, in piece order (so the
// result does not depend on which CTA finished first),
//   m = max m_k,   out = sum 2^(m_k - m) o_k / sum 2^(m_k - m) l_k.
// A warp takes a row; blocks of CTAs without a split item leave at once.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;
constexpr int kCombineRows = 32;  // rows of a block

template <typename T>
__global__ void __launch_bounds__(kCombineThreads)
    prefill_combine_kernel(const PrefillArgs a, int rows, int tile_rows, int cols, int head_dim) {
  grid_dependency_wait();
  const int c = blockIdx.x;
  const PrefillSplit sp = a.splits[c];
  if (sp.pieces == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_toks = tile_rows / a.group;
  for (int k = warp; k < kCombineRows; k += kCombineThreads / 32) {
    const int r = blockIdx.y * kCombineRows + k;
    const int tile = r / tile_rows, rr = r - tile * tile_rows;
    const int g = rr % a.group;
    const int tok = tile * tile_toks + rr / a.group;
    if (r >= rows || rr >= tile_toks * a.group || tok >= sp.ntok) continue;
    float m = -CUDART_INF_F;
    bool bad = false;
    for (int p = 0; p < sp.pieces; ++p) {
      const long long slot = p == 0 ? 2ll * c : 2ll * (c + p) + 1;
      const float mk = a.ml[slot * rows + r].x;
      bad |= isnan(mk);
      m = fmaxf(m, mk);
    }
    const float mb = m == -CUDART_INF_F ? 0.f : m;
    float l = 0.f;
    const int n4 = cols / 4;  // float4s of a row, 16 to 64
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int p = 0; p < sp.pieces; ++p) {
      const long long slot = p == 0 ? 2ll * c : 2ll * (c + p) + 1;
      const float2 ml = a.ml[slot * rows + r];
      const float f = exp2f(ml.x - mb);
      if (f == 0.f) continue;  // nothing attended there
      l += f * ml.y;
      const float* src = a.part + (slot * rows + r) * cols;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (lane + 32 * e < n4) {
          const float4 x = load4(src + 4 * (lane + 32 * e));
          o[e].x += f * x.x;
          o[e].y += f * x.y;
          o[e].z += f * x.z;
          o[e].w += f * x.w;
        }
      }
    }
    const float inv = bad ? CUDART_NAN_F : 1.f / l;
    T* dst = static_cast<T*>(a.out) +
             (static_cast<long long>(sp.row0 + tok) * a.num_q_heads + sp.head * a.group + g) * head_dim +
             sp.part * cols;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (lane + 32 * e >= n4) continue;
      const int col = 4 * (lane + 32 * e);
      if constexpr (sizeof(T) == 4)
        store_part(reinterpret_cast<float*>(dst) + col,
                   make_float4(o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv));
      else
        *reinterpret_cast<uint2*>(dst + col) =
            make_uint2(pack_bf16(o[e].x * inv, o[e].y * inv), pack_bf16(o[e].z * inv, o[e].w * inv));
    }
  }
}

}  // namespace

const PrefillVariant* prefill_simt_variant(int head_dim) {
  static const PrefillVariant table[] = {SimtVariant<64>::info(), SimtVariant<128>::info(),
                                         SimtVariant<256>::info()};
  return head_dim == 64 ? &table[0] : head_dim == 128 ? &table[1] : head_dim == 256 ? &table[2] : nullptr;
}

cudaError_t launch_prefill_combine(const PrefillArgs& a, int grid, int rows, int tile_rows, int cols, int head_dim,
                                   int dtype_out, cudaStream_t stream) {
  // a programmatic dependent: its blocks are resident by the time the pieces are written
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (rows + kCombineRows - 1) / kCombineRows);
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (dtype_out == 0)
    return cudaLaunchKernelEx(&cfg, prefill_combine_kernel<__nv_bfloat16>, a, rows, tile_rows, cols, head_dim);
  return cudaLaunchKernelEx(&cfg, prefill_combine_kernel<float>, a, rows, tile_rows, cols, head_dim);
}

}  // namespace vt
