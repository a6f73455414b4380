// Ragged prefill on CUDA cores (fp32 storage), and the combine of split items.
//
// Per item: S = Q K^T, online softmax, O += P V with everything in fp32, 64
// query rows against 64 keys (two pages) at a time.  Bound by shared memory: a
// 16-byte load takes the SM four cycles whatever its lanes share, so what
// counts is how many FMAs a loaded value feeds.  Each of 128 threads holds 8
// rows x 4 keys of S and 8 rows x D / 16 columns of O: 12 loads for 64 f32x2
// FMAs of Q K^T and 24 for 128 of P V at head_dim 128.  (4 x 2 and 4 rows, with
// 256 threads, took 227 us where this takes 204: 1263 tokens over contexts of
// up to 972, 16 q / 8 kv heads of 128.)  P lies over K's tile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "decode_kernel.cuh"  // e4m3x4_to_f16, ex2, packs
#include "packed.cuh"
#include "prefill_variants.cuh"

namespace vt {
namespace {

constexpr int kSimtThreads = 128;
constexpr int kSimtRows = 64;
constexpr int kSimtKeys = 64;

template <int D>
struct SimtSmem {
  float q[kSimtRows][D + 4];
  union {
    float k[kSimtKeys][D + 4];
    float p[kSimtRows][kSimtKeys + 4];
  };
  float v[kSimtKeys][D];
  int bad;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ void store_part(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

// 16 bytes from global to shared memory, asynchronously; zeros if !valid.
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kSimtThreads) prefill_simt_kernel(const PrefillArgs a) {
  extern __shared__ char raw[];
  SimtSmem<D>& s = *reinterpret_cast<SimtSmem<D>*>(raw);
  const int tid = threadIdx.x;
  const int ty = tid >> 4, tx = tid & 15;  // rows 8 ty..+7; keys tx + 16 e; columns 4 tx + 64 c
  constexpr int NC = D / 64, NR = 8, NK = 4;
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
    float m[NR], l[NR];
    float2 o[NR][NC][2];  // columns 4 tx + 64 c, +1 and +2, +3
    int pos[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
      pos[i] = it.pos0 + min((ty * NR + i) / a.group, it.ntok - 1);
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c][0] = o[i][c][1] = make_float2(0.f, 0.f);
    }
    const int first = it.lo + it.kb0 * kPfBlock;
    const int last = min(it.hi, it.lo + it.kb1 * kPfBlock);
    // K or V of 64 keys: slots outside [lo_exact, last) hold nothing a row may
    // use and are zeros
    auto fetch = [&](const void* cache, int t0, float* to, int stride) {
      const int* row = a.block_tables + static_cast<long long>(it.b) * a.max_blocks;
      int page[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = t0 / kPfPage + i;
        page[i] = t0 + i * kPfPage < last ? row[at] : 0;
        if (page[i] < 0 || page[i] >= a.num_blocks) {
          if (tid == 0) s.bad = 1;
          page[i] = 0;
        }
      }
      for (int i = tid; i < kSimtKeys * (D / 4); i += kSimtThreads) {
        const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
        const bool valid = t0 + r >= it.lo_exact && t0 + r < last;
        const long long at =
            ((static_cast<long long>(page[r / kPfPage]) * kPfPage + r % kPfPage) * a.num_kv_heads + it.head) * D + c;
        copy_async(to + r * stride + c, static_cast<const float*>(cache) + at, valid);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int t0 = first; t0 < last; t0 += kSimtKeys) {
      fetch(a.k_cache, t0, &s.k[0][0], D + 4);
      fetch(a.v_cache, t0, &s.v[0][0], D);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      float2 y[NR][NK];  // sums over even and odd columns
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < NK; ++e) y[i][e] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int d = 0; d < D; d += 4) {
        float4 k[NK];
#pragma unroll
        for (int e = 0; e < NK; ++e) k[e] = load4(&s.k[tx + 16 * e][d]);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float4 q = load4(&s.q[ty * NR + i][d]);
#pragma unroll
          for (int e = 0; e < NK; ++e) {
            y[i][e] = fma2(make_float2(q.x, q.y), make_float2(k[e].x, k[e].y), y[i][e]);
            y[i][e] = fma2(make_float2(q.z, q.w), make_float2(k[e].z, k[e].w), y[i][e]);
          }
        }
      }
      __syncthreads();  // P goes over K
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float x[NK], top = -CUDART_INF_F;
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          const int t = t0 + tx + 16 * e;
          const bool seen = t <= pos[i] && t < last && (a.window == 0 || t > pos[i] - a.window);
          x[e] = seen ? (y[i][e].x + y[i][e].y) * a.scale_log2 : -CUDART_INF_F;
          top = fmaxf(top, x[e]);
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(m[i], top);
        const float mb = mn == -CUDART_INF_F ? 0.f : mn;
        const float keep = exp2f(m[i] - mb);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          const float p = exp2f(x[e] - mb);
          sum += p;
          s.p[ty * NR + i][tx + 16 * e] = p;
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[i] = l[i] * keep + sum;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int x2 = 0; x2 < 2; ++x2) {
            o[i][c][x2].x *= keep;
            o[i][c][x2].y *= keep;
          }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      // Where some row sees only part of the keys, weights of 0 take no part:
      // 0 times a value that is not finite would be NaN.
      const bool partial = t0 + kSimtKeys > it.pos0 + 1 || (a.window > 0 && t0 < it.hi - a.window);
      const int keys = min(kSimtKeys, last - t0);
      if (partial) {
#pragma unroll 1
        for (int t = 0; t < keys; ++t) {
          float pe[NR];
#pragma unroll
          for (int i = 0; i < NR; ++i) pe[i] = s.p[ty * NR + i][t];
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float4 v = load4(&s.v[t][4 * tx + 64 * c]);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
              if (pe[i] != 0.f) {
                o[i][c][0] = fma2(make_float2(pe[i], pe[i]), make_float2(v.x, v.y), o[i][c][0]);
                o[i][c][1] = fma2(make_float2(pe[i], pe[i]), make_float2(v.z, v.w), o[i][c][1]);
              }
            }
          }
        }
      } else {
#pragma unroll 1
        for (int t = 0; t < kSimtKeys; t += 4) {
          float4 p[NR];
#pragma unroll
          for (int i = 0; i < NR; ++i) p[i] = load4(&s.p[ty * NR + i][t]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float4 v = load4(&s.v[t + e][4 * tx + 64 * c]);
#pragma unroll
              for (int i = 0; i < NR; ++i) {
                const float pe = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                o[i][c][0] = fma2(make_float2(pe, pe), make_float2(v.x, v.y), o[i][c][0]);
                o[i][c][1] = fma2(make_float2(pe, pe), make_float2(v.z, v.w), o[i][c][1]);
              }
            }
          }
        }
      }
      __syncthreads();  // before the tiles are filled again
    }
    __syncthreads();
    const bool bad = s.bad != 0;
    const bool split = it.kb0 > 0 || it.pieces > 0;
    const long long slot = 2ll * blockIdx.x + (it.kb0 > 0 ? 1 : 0);
    if (it.pieces > 0 && tid == 0)
      a.splits[blockIdx.x] = PrefillSplit{it.pieces, it.row0, it.ntok, it.head, it.part};
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = ty * NR + i;
      if (r >= rows) continue;
      float* dst;
      float mul = 1.f;
      if (split) {
        dst = a.part + (slot * kSimtRows + r) * D;
        if (tx == 0) a.ml[slot * kSimtRows + r] = make_float2(bad ? CUDART_NAN_F : m[i], l[i]);
      } else {
        const int t = r / a.group, g = r - t * a.group;
        dst = static_cast<float*>(a.out) +
              (static_cast<long long>(it.row0 + t) * a.num_q_heads + it.head * a.group + g) * D;
        mul = bad ? CUDART_NAN_F : 1.f / l[i];
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
        store_part(dst + 4 * tx + 64 * c, make_float4(o[i][c][0].x * mul, o[i][c][0].y * mul, o[i][c][1].x * mul,
                                                      o[i][c][1].y * mul));
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
// Eight lanes take a row, so a warp has the loads of four rows in flight (one
// row at a time, a warp's rows cost a memory latency each: 16 us a call).
// Blocks of CTAs without a split item leave at once.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;
constexpr int kCombineRows = 32;  // rows of a block

template <typename T, int COLS>
__global__ void __launch_bounds__(kCombineThreads)
    prefill_combine_kernel(const PrefillArgs a, int rows, int tile_rows, int head_dim) {
  grid_dependency_wait();
  const int c = blockIdx.x;
  const PrefillSplit sp = a.splits[c];
  if (sp.pieces == 0) return;
  const int lane = threadIdx.x & 7;
  const int r = blockIdx.y * kCombineRows + (threadIdx.x >> 3);
  const int tile_toks = tile_rows / a.group;
  const int tile = r / tile_rows, rr = r - tile * tile_rows;
  const int g = rr % a.group;
  const int tok = tile * tile_toks + rr / a.group;
  if (r >= rows || rr >= tile_toks * a.group || tok >= sp.ntok) return;
  auto record = [&](int p) { return (p == 0 ? 2ll * c : 2ll * (c + p) + 1) * rows + r; };
  float m = -CUDART_INF_F;
  bool bad = false;
  for (int p = 0; p < sp.pieces; ++p) {
    const float mk = a.ml[record(p)].x;
    bad |= isnan(mk);
    m = fmaxf(m, mk);
  }
  const float mb = m == -CUDART_INF_F ? 0.f : m;
  float l = 0.f;
  constexpr int N = COLS / 32;  // float4s of a lane: columns 4 lane + 32 e
  float4 o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p = 0; p < sp.pieces; ++p) {
    const float2 ml = a.ml[record(p)];
    const float f = exp2f(ml.x - mb);
    if (f == 0.f) continue;  // nothing attended there
    l += f * ml.y;
    const float* src = a.part + record(p) * COLS + 4 * lane;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float4 x = load4(src + 32 * e);
      o[e].x += f * x.x;
      o[e].y += f * x.y;
      o[e].z += f * x.z;
      o[e].w += f * x.w;
    }
  }
  const float inv = bad ? CUDART_NAN_F : 1.f / l;
  T* dst = static_cast<T*>(a.out) +
           (static_cast<long long>(sp.row0 + tok) * a.num_q_heads + sp.head * a.group + g) * head_dim +
           sp.part * COLS + 4 * lane;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if constexpr (sizeof(T) == 4)
      store_part(reinterpret_cast<float*>(dst) + 32 * e,
                 make_float4(o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv));
    else
      *reinterpret_cast<uint2*>(dst + 32 * e) =
          make_uint2(pack_bf16(o[e].x * inv, o[e].y * inv), pack_bf16(o[e].z * inv, o[e].w * inv));
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
    return cols == 64    ? cudaLaunchKernelEx(&cfg, prefill_combine_kernel<__nv_bfloat16, 64>, a, rows, tile_rows, head_dim)
           : cols == 128 ? cudaLaunchKernelEx(&cfg, prefill_combine_kernel<__nv_bfloat16, 128>, a, rows, tile_rows, head_dim)
                         : cudaLaunchKernelEx(&cfg, prefill_combine_kernel<__nv_bfloat16, 256>, a, rows, tile_rows, head_dim);
  return cols == 64    ? cudaLaunchKernelEx(&cfg, prefill_combine_kernel<float, 64>, a, rows, tile_rows, head_dim)
         : cols == 128 ? cudaLaunchKernelEx(&cfg, prefill_combine_kernel<float, 128>, a, rows, tile_rows, head_dim)
                       : cudaLaunchKernelEx(&cfg, prefill_combine_kernel<float, 256>, a, rows, tile_rows, head_dim);
}

}  // namespace vt
