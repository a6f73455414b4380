// Ragged prefill on CUDA cores (fp32 storage), and the combine of split items.
//
// Per item: S = Q K^T, online softmax, O += P V with everything in fp32, 64
// query rows against 64 keys (two pages) at a time.  A 16-byte load from shared
// memory takes the SM four cycles whatever its lanes share, so what counts is
// how many FMAs a loaded value feeds.  Each of 128 threads holds 8 rows x 4 keys
// of S and 8 rows x D / 16 columns of O: 12 loads for 64 f32x2 FMAs of Q K^T and
// 16 for 128 of P V at head_dim 128.  (4 x 2 and 4 rows, with 256 threads, took
// 227 us where 8 x 4 took 204: 1263 tokens over contexts of up to 972, 16 q / 8
// kv heads of 128.)  At that tile the bound is dependent latency, not the loads:
// two warps a scheduler, the FMA pipe 57 % busy, the load pipe 22 %, and `wait`
// the first stall; at head_dim 128 its 255 registers spill 76 bytes.  Q, K and V
// come by asynchronous copies; at head_dim 128 P lies over K's tile.  Values are
// looked at only in tiles that some row sees in part, and only if one is not
// finite do weights of 0 branch around it: 182 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "decode_kernel.cuh"  // ex2, smem_addr
#include "packed.cuh"
#include "prefill_variants.cuh"

namespace vt {
namespace {

constexpr int kSimtRows = 64;
constexpr int kSimtKeys = 64;

// 8 rows x 4 keys and 8 rows x D / 16 columns a thread; at head_dim 256 there is
// room for one CTA an SM and not for that in a thread's registers: 4 rows, and
// twice the threads.
template <int D>
constexpr int kSimtThreads = D == 256 ? 256 : 128;

// Where it fits beside them (at head_dim 128 two CTAs an SM would no longer),
// P has a place of its own, and the next K is fetched behind the softmax and P V.
template <int D>
constexpr bool kOwnP = D != 128;

template <int D>
struct SimtSmem {
  float q[kSimtRows][D + 4];
  float k[kSimtKeys][D + 4];  // and P, where that has no place of its own
  float v[kSimtKeys][D];
  float p[kOwnP<D> ? kSimtRows : 1][kSimtKeys + 4];
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
__global__ void __launch_bounds__(kSimtThreads<D>) prefill_simt_kernel(const PrefillArgs a) {
  extern __shared__ char raw[];
  SimtSmem<D>& s = *reinterpret_cast<SimtSmem<D>*>(raw);
  const int tid = threadIdx.x;
  const int ty = tid >> 4, tx = tid & 15;  // rows NR ty ...; keys tx + 16 e; columns 4 tx + 64 c
  constexpr int NC = D / 64, NR = 1024 / kSimtThreads<D>, NK = 4;
  if (tid == 0) a.splits[blockIdx.x].pieces = 0;
  PfWalk w;
  pf_begin(a, tid & 31, w);  // each warp for itself
  PfItem it;
  const float scale = a.neg_scale ? -a.scale_log2 : a.scale_log2;
  float(*const ps)[kSimtKeys + 4] = reinterpret_cast<float(*)[kSimtKeys + 4]>(kOwnP<D> ? &s.p[0][0] : &s.k[0][0]);
  constexpr int kLanes = D / 4, kLines = kSimtThreads<D> / kLanes;  // lanes of a row, rows at a time
  const int line = tid / kLanes, col = tid % kLanes * 4;
  while (w.next(a, it)) {
    __syncthreads();  // the previous item's tiles are done with
    if (tid == 0) s.bad = it.bad;
    const int rows = it.ntok * a.group;
    float m[NR], l[NR];
    float2 o[NR][NC][2];  // columns 4 tx + 64 c, +1 and +2, +3
    int pos[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
      pos[i] = it.pos0 + min(pf_token_of(a, ty * NR + i), it.ntok - 1);
#pragma unroll
      for (int c = 0; c < NC; ++c) o[i][c][0] = o[i][c][1] = make_float2(0.f, 0.f);
    }
    const int first = it.lo + it.kb0 * kPfBlock;
    const int last = min(it.hi, it.lo + it.kb1 * kPfBlock);
    // K or V of 64 keys: slots outside [lo_exact, last) hold nothing a row may
    // use and are zeros
    auto fetch = [&](bool of_v, int t0) {
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int t = t0 + i * kPfPage;
        int page = t < last ? a.block_tables[static_cast<long long>(it.b) * a.max_blocks + t / kPfPage] : 0;
        if (page < 0 || page >= a.num_blocks) {
          if (tid == 0) s.bad = 1;
          page = 0;
        }
        const long long step = static_cast<long long>(a.num_kv_heads) * D;
        const float* from = static_cast<const float*>(of_v ? a.v_cache : a.k_cache) +
                            (static_cast<long long>(page) * kPfPage + line) * step + it.head * D + col;
        float* to = of_v ? &s.v[i * kPfPage + line][col] : &s.k[i * kPfPage + line][col];
        const int stride = kLines * (of_v ? D : D + 4);
#pragma unroll 2
        for (int r = t + line; r < t + kPfPage; r += kLines) {
          copy_async(to, from, r >= it.lo_exact && r < last);
          from += kLines * step;
          to += stride;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (first < last) {
#pragma unroll 2
      for (int r = line; r < kSimtRows; r += kLines) {
        const int t = pf_token_of(a, r), g = r - t * a.group;
        const long long at = (static_cast<long long>(it.row0 + (r < rows ? t : 0)) * a.num_q_heads + it.head * a.group + g) * D;
        copy_async(&s.q[r][col], static_cast<const float*>(a.q) + at + col, r < rows);
      }
#pragma unroll 1
      for (int i = 0; i < 2; ++i) fetch(i, first);  // (Q comes with K)
    }
    for (int t0 = first; t0 < last; t0 += kSimtKeys) {
      const int next = t0 + kSimtKeys;
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
      __syncthreads();  // K is done with
      if (kOwnP<D> && next < last) fetch(false, next);
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float x[NK], top = -CUDART_INF_F;
        const int at = t0 + tx, upto = min(pos[i], last - 1) - at;
        const int from = a.window > 0 ? pos[i] - a.window + 1 - at : 0;
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          const bool seen = 16 * e <= upto && 16 * e >= from;
          x[e] = seen ? (y[i][e].x + y[i][e].y) * scale : -CUDART_INF_F;
          top = fmaxf(top, x[e]);
        }
#pragma unroll
        for (int d = 8; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(m[i], top);
        const float mb = mn == -CUDART_INF_F ? 0.f : mn;
        const float keep = ex2(m[i] - mb);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < NK; ++e) {
          const float p = ex2(x[e] - mb);
          sum += p;
          ps[ty * NR + i][tx + 16 * e] = p;
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
      if (kOwnP<D> && next < last)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      // Where some row sees only part of the keys, and a value is not finite,
      // weights of 0 take no part: 0 times such a value would be NaN.
      const int keys = min(kSimtKeys, last - t0);
      bool apart = false;
      if (t0 + kSimtKeys > it.pos0 + 1 || (a.window > 0 && t0 < it.hi - a.window)) {
        unsigned seen = 0;
#pragma unroll 1
        for (int i = tid; i < keys * (D / 4); i += kSimtThreads<D>) {
          const uint4 x = reinterpret_cast<const uint4*>(&s.v[0][0])[i];
          seen |= ((x.x & 0x7f800000u) + 0x00800000u) | ((x.y & 0x7f800000u) + 0x00800000u) |
                  ((x.z & 0x7f800000u) + 0x00800000u) | ((x.w & 0x7f800000u) + 0x00800000u);
        }
        apart = __syncthreads_or(static_cast<int>(seen >> 31));
      }
      if (apart) {
#pragma unroll 1
        for (int t = 0; t < keys; ++t) {
          float pe[NR];
#pragma unroll
          for (int i = 0; i < NR; ++i) pe[i] = ps[ty * NR + i][t];
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
        for (int t = 0; t < keys; t += 4) {
          float4 p[NR];
#pragma unroll
          for (int i = 0; i < NR; ++i) p[i] = load4(&ps[ty * NR + i][t]);
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
      if (next < last) {
#pragma unroll 1
        for (int i = kOwnP<D> ? 1 : 0; i < 2; ++i) fetch(i, next);
      }
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
        const int t = pf_token_of(a, r), g = r - t * a.group;
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
    prefill_simt_kernel<D><<<grid, kSimtThreads<D>, sizeof(SimtSmem<D>), stream>>>(a);
    return cudaGetLastError();
  }
  static PrefillVariant info() {
    return PrefillVariant{kSimtThreads<D>, kSimtRows, kSimtRows, D, 0, 1, 128, sizeof(SimtSmem<D>),
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
  const int g = rr - pf_token_of(a, rr) * a.group;
  const int tok = tile * tile_toks + pf_token_of(a, rr);
  if (r >= rows || rr >= tile_toks * a.group || tok >= sp.ntok) return;
  auto record = [&](int p) { return (p == 0 ? 2ll * c : 2ll * (c + p) + 1) * rows + r; };
  float m = -CUDART_INF_F;
  bool bad = false;
#pragma unroll 4
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
  constexpr int U = COLS >= 256 ? 1 : 256 / COLS;  // pieces whose loads are in flight together
#pragma unroll 1
  for (int p0 = 0; p0 < sp.pieces; p0 += U) {
    float f[U];
    float4 x[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f[u] = 0.f;
      if (p0 + u < sp.pieces) {
        const float2 ml = a.ml[record(p0 + u)];
        f[u] = ex2(ml.x - mb);
        l += f[u] * ml.y;
        const float* src = a.part + record(p0 + u) * COLS + 4 * lane;
#pragma unroll
        for (int e = 0; e < N; ++e) x[u][e] = load4(src + 32 * e);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (f[u] == 0.f) continue;  // nothing attended there, nothing written
#pragma unroll
      for (int e = 0; e < N; ++e) {
        o[e].x += f[u] * x[u][e].x;
        o[e].y += f[u] * x[u][e].y;
        o[e].z += f[u] * x[u][e].z;
        o[e].w += f[u] * x[u][e].w;
      }
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
  // a programmatic dependent: the launch itself is prepared while the prefill runs (its blocks start when the last
  // CTA has ended, since none releases them before)
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
