// Rotary positions and the append of new keys and values to the paged cache.
//
// Mathematics.  A pair (a, b) of a head's row at position p becomes
// A (a cos w - b sin w), A (b cos w + a sin w) with w = p f_j.  Positions are
// integers, so only the fraction of a turn that f_j stands for matters: with
// u_j = frac(f_j / 2 pi) held as a 64-bit fixed-point fraction, p u_j modulo
// 2^64 is the reduced angle exactly as the hardware's integer product wraps,
// for either sign of p and at any distance.  Its top 32 bits become a float
// in [-1/2, 1/2) turns, and sincospi() takes it from there.  (In fp32 an
// angle of 10^5 radians would be off by 4e-3.)
//
// What bounds it: every element is read and written once, so HBM for long
// batches and the launch for short ones.  A warp takes tokens one by one (or a
// part of one's heads at either end of its share).  A lane has a fixed place in
// a head's row, 16 elements with 16-byte accesses, and walks over the token's
// heads four rounds at a time; the first rounds' loads are issued before the
// token is looked up (a warp-wide search of the row starts, then the block
// table).  Each angle is formed once for all heads: the lanes share out a
// token's pairs and hand (cos, sin) round by shuffles, so there is no table in
// shared memory and no block-wide wait, and a warp's next token reuses its
// frequencies.
// Measured (bf16, head_dim 128): 16803 tokens of 32 + 8 + 8 heads appended in
// 74 to 77 us, 5.5 TB/s of reads and writes; 5173 tokens of 64 + 8 + 8 into
// E4M3 pages 43 us; a block-wide kernel with a table in shared memory took 86
// and 54.  That one remains for rows the lanes do not divide (rot_dim or
// head_dim not a multiple of 16, head_dim 80 or 1024, say).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <new>
#include <type_traits>

#include "../../include/vt_paged_attn.h"
#include "host_state.cuh"

namespace vt {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kPage = 32;
constexpr int kMaxTokensPerBlock = 4;

struct RopeArgs {
  // queries (or vt_rope's rows): x -> out
  const void* q;
  void* q_out;
  long long q_stride, q_out_stride;
  int q_heads;
  // append only
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  long long k_stride, v_stride;
  int kv_heads;
  const float* k_scale;  // E4M3 caches
  const float* v_scale;
  const int* q_starts;
  const int* block_tables;
  const int* context_lens;
  int num_seqs, max_blocks, num_blocks;
  // both
  const int* positions;
  const double* inv_freq;
  int num_tokens, head_dim, rot_dim;
  int tokens_per_block;
  float amplitude;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Four E4M3 codes of x[0..3]: nearest, ties to even, held at +-448; NaN kept.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Eight contiguous elements at p (16-byte aligned for bf16, 32 for fp32's pair of vectors).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8], float) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8], float) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
// x / scale as a product (2^-23 of it off at most; a code keeps 2^-4) where the
// reciprocal is an ordinary number.
__device__ __forceinline__ void store8(uint8_t* p, const float (&x)[8], float scale) {
  const float inv = 1.f / scale;
  float y[8];
  if (fabsf(inv) < 1e38f && inv != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] / scale;
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x, float) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(float* p, float x, float) { *p = x; }
__device__ __forceinline__ void store1(uint8_t* p, float x, float scale) {
  const float y = x / scale;
  *p = static_cast<uint8_t>(e4m3x4(y, y, y, y));
}

// The sequence that owns packed row t: the last b with starts[b] <= t, found
// by one warp, 32 probes at a time.  Any starts are safe (b stays in range).
__device__ __forceinline__ int find_sequence(const int* starts, int num_seqs, int t, int lane) {
  int lo = 0, hi = num_seqs;  // starts[lo] <= t; the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && starts[at] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    // probes are taken as sorted; a decreasing array only gives some b in range
    const int nlo = lo + n * step;
    hi = min(hi, nlo + step);
    lo = min(nlo, hi - 1);
  }
  return lo;
}

// The fraction of a turn a position is worth, as a 64-bit fixed-point number.
__device__ __forceinline__ unsigned long long turn_fraction(double inv_freq) {
  const double turns = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}
// (cos, sin) of position p's angle, times the amplitude.
__device__ __forceinline__ float2 cos_sin(unsigned long long fraction, int p, float amplitude) {
  const unsigned long long w = fraction * static_cast<unsigned long long>(static_cast<long long>(p));
  // the top 32 bits, rounded, as a signed fraction of a turn; sincospi takes half turns
  const int top = static_cast<int>(static_cast<unsigned>((w + 0x80000000ull) >> 32));
  float s, c;
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);  // 2^-31
  return make_float2(c * amplitude, s * amplitude);
}

// What a block knows of each of its tokens.
struct Token {
  int position;
  int live;         // 0: padding, 1: rotate and write, 2: NaN query row, nothing cached
  long long slot;   // cache row (page * 32 + slot); -1: not written
};

// What is known of packed row t if sequence b owns it.  Starts that are no
// array of rows (below 0, past num_tokens) own none: whatever they hold,
// 0 <= p < L, and no difference leaves 32 bits.
__device__ __forceinline__ Token token_of(const RopeArgs& a, int t, int b) {
  const int s = a.q_starts[b], e = a.q_starts[b + 1], L = a.context_lens[b];
  Token k{0, 0, -1};
  if (s >= 0 && t >= s && t < e && e <= a.num_tokens) {
    const int n = e - s;
    if (L < n || L > static_cast<long long>(a.max_blocks) * kPage) {
      k.live = 2;
    } else {
      const int p = L - n + (t - s);
      k.live = 1;
      k.position = a.positions ? a.positions[t] : p;
      const int page = a.block_tables[static_cast<long long>(b) * a.max_blocks + p / kPage];
      if (page >= 0 && page < a.num_blocks) k.slot = static_cast<long long>(page) * kPage + p % kPage;
    }
  }
  return k;
}

// Any head_dim and rot_dim: a block takes a few tokens, fills a (cos, sin) table
// of tokens x pairs in shared memory, then walks units of the tokens' heads.
// APPEND: keys and values go to the cache as KV elements; otherwise only
// q -> q_out.  VEC: 16 | rot_dim and 16 | head_dim, so a unit is two 8-element
// vectors; else a unit is two single elements.
template <typename T, typename KV, bool APPEND, bool VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  extern __shared__ float2 table[];  // [tokens_per_block][rot_dim / 2]
  __shared__ Token tok[kMaxTokensPerBlock];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * a.tokens_per_block;
  const int nt = min(a.tokens_per_block, a.num_tokens - t0);
  const int half = a.rot_dim / 2;
  const int D = a.head_dim;
  constexpr int E = VEC ? 16 : 2;  // elements of a unit
  const int units = D / E;         // units of a head
  const int rot_units = a.rot_dim / E;
  const int heads = a.q_heads + (APPEND ? 2 * a.kv_heads : 0);
  const int total = nt * heads * units;
  const int stride = kRopeThreads * gridDim.y;

  struct Unit {
    int t, head, off0, off1, pair;  // elements [off0, +E/2) and [off1, +E/2) of the head's row; first pair, -1: copy
    const T* src;
  };
  auto locate = [&](int i) {
    Unit u;
    const int per_token = heads * units;
    u.t = i / per_token;
    int r = i - u.t * per_token;
    u.head = r / units;
    r -= u.head * units;
    if (r < rot_units) {
      u.pair = r * (E / 2);
      u.off0 = INTER ? r * E : r * (E / 2);
      u.off1 = INTER ? u.off0 + E / 2 : half + u.off0;
    } else {
      u.pair = -1;
      u.off0 = r * E;
      u.off1 = u.off0 + E / 2;
    }
    const long long row = t0 + u.t;
    if (!APPEND || u.head < a.q_heads)
      u.src = static_cast<const T*>(a.q) + row * a.q_stride + static_cast<long long>(u.head) * D;
    else if (u.head < a.q_heads + a.kv_heads)
      u.src = static_cast<const T*>(a.k) + row * a.k_stride + static_cast<long long>(u.head - a.q_heads) * D;
    else
      u.src = static_cast<const T*>(a.v) + row * a.v_stride +
              static_cast<long long>(u.head - a.q_heads - a.kv_heads) * D;
    return u;
  };
  constexpr int H = E / 2;
  float x0[H], x1[H];
  auto fetch = [&](const Unit& u) {
    if constexpr (VEC) {
      load8(u.src + u.off0, x0);
      load8(u.src + u.off1, x1);
    } else {
      x0[0] = load1(u.src + u.off0);
      x1[0] = load1(u.src + u.off1);
    }
  };

  int i = blockIdx.y * kRopeThreads + tid;
  Unit u{};
  if (i < total) {
    u = locate(i);
    fetch(u);
  }

  if constexpr (APPEND) {
    const int warp = tid >> 5, lane = tid & 31;
    if (warp < nt) {
      const int t = t0 + warp;
      const int b = find_sequence(a.q_starts, a.num_seqs, t, lane);
      if (lane == 0) tok[warp] = token_of(a, t, b);
    }
    __syncthreads();
  }
  for (int r = tid; r < nt * half; r += kRopeThreads) {
    const int t = r / half, j = r - t * half;
    table[r] = cos_sin(turn_fraction(a.inv_freq[j]), APPEND ? tok[t].position : a.positions[t0 + t], a.amplitude);
  }
  __syncthreads();

  while (i < total) {
    const int live = APPEND ? tok[u.t].live : 1;
    float y0[H], y1[H];
    const bool is_v = APPEND && u.head >= a.q_heads + a.kv_heads;
    if (u.pair >= 0 && !is_v) {
      const float2* cs = table + u.t * half + u.pair;
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 w = cs[e];
        if constexpr (INTER && VEC) {
          // pairs are (2e, 2e + 1) of the 16 contiguous elements x0, x1
          float& lo = e < H / 2 ? x0[2 * e] : x1[2 * e - H];
          float& hi = e < H / 2 ? x0[2 * e + 1] : x1[2 * e + 1 - H];
          float& ylo = e < H / 2 ? y0[2 * e] : y1[2 * e - H];
          float& yhi = e < H / 2 ? y0[2 * e + 1] : y1[2 * e + 1 - H];
          ylo = lo * w.x - hi * w.y;
          yhi = hi * w.x + lo * w.y;
        } else {
          y0[e] = x0[e] * w.x - x1[e] * w.y;
          y1[e] = x1[e] * w.x + x0[e] * w.y;
        }
      }
    } else {
      // a copy; v's units are contiguous whatever the layout, so its offsets
      // are a permutation of the row all the same
#pragma unroll
      for (int e = 0; e < H; ++e) {
        y0[e] = x0[e];
        y1[e] = x1[e];
      }
    }
    const Unit d = u;
    i += stride;
    if (i < total) {
      u = locate(i);
      fetch(u);
    }
    if (!APPEND || d.head < a.q_heads) {
      if (live == 2) {
#pragma unroll
        for (int e = 0; e < H; ++e) y0[e] = y1[e] = __int_as_float(0x7fffffff);
      }
      if (live) {
        T* dst = static_cast<T*>(a.q_out) + static_cast<long long>(t0 + d.t) * a.q_out_stride +
                 static_cast<long long>(d.head) * D;
        if constexpr (VEC) {
          store8(dst + d.off0, y0, 1.f);
          store8(dst + d.off1, y1, 1.f);
        } else {
          store1(dst + d.off0, y0[0], 1.f);
          store1(dst + d.off1, y1[0], 1.f);
        }
      }
    } else if constexpr (APPEND) {
      const long long slot = tok[d.t].slot;
      if (slot >= 0) {
        const int h = d.head - a.q_heads - (is_v ? a.kv_heads : 0);
        KV* dst = static_cast<KV*>(is_v ? a.v_cache : a.k_cache) + (slot * a.kv_heads + h) * D;
        const float scale = sizeof(KV) == 1 ? (is_v ? a.v_scale : a.k_scale)[h] : 1.f;
        if constexpr (VEC) {
          store8(dst + d.off0, y0, scale);
          store8(dst + d.off1, y1, scale);
        } else {
          store1(dst + d.off0, y0[0], scale);
          store1(dst + d.off1, y1[0], scale);
        }
      }
    }
  }
}

// The same, the sequence found by a whole warp.  `b` is where the last one was
// found (rows are looked up in order), or -1.
__device__ __forceinline__ Token look_up(const RopeArgs& a, int t, int lane, int& b) {
  if (b < 0 || t >= a.q_starts[b + 1]) b = find_sequence(a.q_starts, a.num_seqs, t, lane);
  return token_of(a, t, b);
}

// U lanes to a head's row of 16 U elements (U = 4 to 32, a power of two), 16 |
// rot_dim.  The work is units of `unit` rounds of R heads, nb of them a token;
// a warp takes consecutive ones, `per` or (the first `extra` warps) per + 1.
template <typename T, typename KV, bool APPEND, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_warp_kernel(const RopeArgs a, int nb, int unit, int warps, long long per, int extra) {
  constexpr int R = 32 / U;                // heads of a round
  constexpr int NP = U >= 4 ? U / 4 : 1;   // pairs a lane forms: pairs NP lane ..
  constexpr int P = sizeof(T) == 2 ? 4 : 2;  // rounds in flight
  constexpr int D = 16 * U;
  const int lane = threadIdx.x & 31;
  const int warp = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (warp >= warps) return;
  long long todo = per + (warp < extra ? 1 : 0);
  const long long from = warp * per + min(warp, extra);
  int t = static_cast<int>(from / nb);
  int part = static_cast<int>(from - static_cast<long long>(t) * nb);  // the token's first unit to do
  const int heads = a.q_heads + (APPEND ? 2 * a.kv_heads : 0);
  const int u = lane & (U - 1), r = lane / U;
  const int half = a.rot_dim >> 1;
  const bool turns = u < (a.rot_dim >> 4);  // else this lane's elements are copied
  const int off0 = turns && !INTER ? 8 * u : 16 * u, off1 = turns && !INTER ? half + off0 : off0 + 8;

  unsigned long long frac[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) frac[i] = NP * lane + i < half ? turn_fraction(a.inv_freq[NP * lane + i]) : 0ull;

  struct Raw {
    float4 v[sizeof(T)];  // 16 elements
  } raw[P];
  auto source = [&](int t, int head) {
    const T* p;
    if (!APPEND || head < a.q_heads)
      p = static_cast<const T*>(a.q) + t * a.q_stride + static_cast<long long>(head) * D;
    else if (head < a.q_heads + a.kv_heads)
      p = static_cast<const T*>(a.k) + t * a.k_stride + static_cast<long long>(head - a.q_heads) * D;
    else
      p = static_cast<const T*>(a.v) + t * a.v_stride + static_cast<long long>(head - a.q_heads - a.kv_heads) * D;
    return p;
  };
  int last = 0;  // heads of the token at hand up to here
  auto fetch = [&](int t, int h0) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int head = h0 + i * R + r;
      if (head < last) {
        const T* p = source(t, head);
        constexpr int N = sizeof(T) / 2;  // 16-byte vectors of 8 elements
#pragma unroll
        for (int k = 0; k < N; ++k) {
          raw[i].v[k] = reinterpret_cast<const float4*>(p + off0)[k];
          raw[i].v[N + k] = reinterpret_cast<const float4*>(p + off1)[k];
        }
      }
    }
  };
  int b = -1;
#pragma unroll 1
  for (int parts; todo > 0; todo -= parts, ++t, part = 0) {
    parts = todo < nb - part ? static_cast<int>(todo) : nb - part;
    const int first = part * unit * R;
    last = min((part + parts) * unit * R, heads);
    fetch(t, first);
    Token k{0, 1, -1};
    if constexpr (APPEND)
      k = look_up(a, t, lane, b);
    else
      k.position = a.positions[t];
    if (k.live == 0) continue;  // the warp's
    float2 mine[NP], cs[8];
#pragma unroll
    for (int i = 0; i < NP; ++i) mine[i] = cos_sin(frac[i], k.position, a.amplitude);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int from = (8 * u + e) / NP;
      cs[e].x = __shfl_sync(0xffffffffu, mine[e % NP].x, from);
      cs[e].y = __shfl_sync(0xffffffffu, mine[e % NP].y, from);
    }
#pragma unroll 1
    for (int h0 = first; h0 < last; h0 += P * R) {
      if (h0 != first) fetch(t, h0);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int head = h0 + i * R + r;
        if (head >= last) continue;
        float x0[8], x1[8], y0[8], y1[8];
        load8(reinterpret_cast<const T*>(&raw[i].v[0]), x0);
        load8(reinterpret_cast<const T*>(&raw[i].v[sizeof(T) / 2]), x1);
        const bool is_v = APPEND && head >= a.q_heads + a.kv_heads;
        if (turns && !is_v) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (INTER) {  // pairs (2e, 2e + 1) of the 16 elements
              const float(&x)[8] = e < 4 ? x0 : x1;
              float(&y)[8] = e < 4 ? y0 : y1;
              y[2 * (e % 4)] = x[2 * (e % 4)] * cs[e].x - x[2 * (e % 4) + 1] * cs[e].y;
              y[2 * (e % 4) + 1] = x[2 * (e % 4) + 1] * cs[e].x + x[2 * (e % 4)] * cs[e].y;
            } else {
              y0[e] = x0[e] * cs[e].x - x1[e] * cs[e].y;
              y1[e] = x1[e] * cs[e].x + x0[e] * cs[e].y;
            }
          }
        } else {
          // a copy (v's elements are taken in k's order, and stored so)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y0[e] = x0[e];
            y1[e] = x1[e];
          }
        }
        if (!APPEND || head < a.q_heads) {
          if (k.live == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y0[e] = y1[e] = __int_as_float(0x7fffffff);
          }
          T* dst = static_cast<T*>(a.q_out) + t * a.q_out_stride + static_cast<long long>(head) * D;
          store8(dst + off0, y0, 1.f);
          store8(dst + off1, y1, 1.f);
        } else if constexpr (APPEND) {
          if (k.slot >= 0) {
            const int h = head - a.q_heads - (is_v ? a.kv_heads : 0);
            KV* dst = static_cast<KV*>(is_v ? a.v_cache : a.k_cache) + (k.slot * a.kv_heads + h) * D;
            const float scale = sizeof(KV) == 1 ? (is_v ? a.v_scale : a.k_scale)[h] : 1.f;
            store8(dst + off0, y0, scale);
            store8(dst + off1, y1, scale);
          }
        }
      }
    }
  }
}

// The warp kernel where a head's row is 4, 8, 16 or 32 lanes of 16 elements
// and the rotated part whole units; false: not taken.
template <typename T, typename KV, bool APPEND>
bool launch_rope_warps(const RopeArgs& a, int interleaved, int num_sms, cudaStream_t stream) {
  const int U = a.head_dim / 16;
  if (a.rot_dim % 16 != 0 || a.head_dim % 16 != 0 || (U != 4 && U != 8 && U != 16 && U != 32)) return false;
  const int heads = a.q_heads + (APPEND ? 2 * a.kv_heads : 0), R = 32 / U;
  // One wave of 16 warps an SM, all with the same share of the heads' rounds
  // (with whole tokens a warp a quarter of them idled, and 5173 tokens into
  // E4M3 pages took 46 us, 43 so), in units of as many rounds as a warp has in flight,
  // and single rounds where there are few.
  constexpr int kFlight = sizeof(T) == 2 ? 4 : 2;
  const long long want = 16ll * num_sms;
  const long long rounds = (heads + R - 1) / R;
  const int unit = a.num_tokens * rounds >= 2 * kFlight * want ? kFlight : 1;
  const long long nb = (rounds + unit - 1) / unit, total = a.num_tokens * nb;
  const long long warps = total < want ? total : want;
  const unsigned blocks = static_cast<unsigned>((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
  auto go = [&](auto inter, auto units) {
    rope_warp_kernel<T, KV, APPEND, decltype(inter)::value, decltype(units)::value>
        <<<blocks, kRopeThreads, 0, stream>>>(a, static_cast<int>(nb), unit, static_cast<int>(warps), total / warps,
                                              static_cast<int>(total % warps));
  };
  auto with = [&](auto inter) {
    if (U == 4) go(inter, std::integral_constant<int, 4>());
    if (U == 8) go(inter, std::integral_constant<int, 8>());
    if (U == 16) go(inter, std::integral_constant<int, 16>());
    if (U == 32) go(inter, std::integral_constant<int, 32>());
  };
  if (interleaved)
    with(std::true_type());
  else
    with(std::false_type());
  return true;
}

template <typename T, typename KV, bool APPEND>
cudaError_t launch_rope(RopeArgs a, int interleaved, int num_sms, cudaStream_t stream) {
  if (launch_rope_warps<T, KV, APPEND>(a, interleaved, num_sms, stream)) return cudaGetLastError();
  const bool vec = a.rot_dim % 16 == 0 && a.head_dim % 16 == 0;
  // Four tokens a block once that still fills the device several times over;
  // one token a block, its units over several blocks, for short batches.
  a.tokens_per_block = a.num_tokens >= 4 * 4 * num_sms ? kMaxTokensPerBlock : 1;
  const int heads = a.q_heads + (APPEND ? 2 * a.kv_heads : 0);
  const long long units = static_cast<long long>(heads) * (a.head_dim / (vec ? 16 : 2));
  dim3 grid((a.num_tokens + a.tokens_per_block - 1) / a.tokens_per_block, 1);
  if (a.tokens_per_block == 1) {
    const long long want = (units + kRopeThreads - 1) / kRopeThreads;
    grid.y = static_cast<unsigned>(want < 64 ? want : 64);
  }
  const size_t smem = static_cast<size_t>(a.tokens_per_block) * (a.rot_dim / 2) * sizeof(float2);
  if (vec && interleaved)
    rope_kernel<T, KV, APPEND, true, true><<<grid, kRopeThreads, smem, stream>>>(a);
  else if (vec)
    rope_kernel<T, KV, APPEND, true, false><<<grid, kRopeThreads, smem, stream>>>(a);
  else if (interleaved)
    rope_kernel<T, KV, APPEND, false, true><<<grid, kRopeThreads, smem, stream>>>(a);
  else
    rope_kernel<T, KV, APPEND, false, false><<<grid, kRopeThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

using namespace vt::host;

vt_status current_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceState& ds = device_state(dev);
  const vt_status st = prepare_device(dev, ds);
  *sms = ds.num_sms;
  return st;
}

bool stride_ok(long long stride, int heads, int head_dim, int elem) {
  return stride >= static_cast<long long>(heads) * head_dim && stride % (16 / elem) == 0;
}

// interleaved, amplitude, rot_dim and its table; rot_dim 0 only where allowed
bool rotation_ok(const double* inv_freq, int rot_dim, int head_dim, int interleaved, float amplitude, bool may_be_none) {
  if (interleaved != 0 && interleaved != 1) return false;
  if (!std::isfinite(amplitude)) return false;
  if (rot_dim == 0) return may_be_none && !inv_freq;
  return inv_freq && aligned(inv_freq, 8) && rot_dim > 0 && rot_dim % 2 == 0 && rot_dim <= head_dim;
}

// No exception leaves a C entry point (the host state allocates).
template <typename F>
vt_status guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

vt_status append(const RopeArgs& a, int block_size, int interleaved, cudaStream_t stream, vt_dtype dtype) {
  if (a.num_seqs < 0 || a.num_tokens < 0) return VT_ERR_INVALID_ARG;
  if (a.num_seqs == 0 || a.num_tokens == 0) return VT_OK;
  if (dtype != VT_BF16 && dtype != VT_F32 && dtype != VT_E4M3) return VT_ERR_INVALID_ARG;
  if (!a.k_cache || !a.v_cache || !a.k || !a.v || !a.q_starts || !a.block_tables || !a.context_lens)
    return VT_ERR_INVALID_ARG;
  if ((a.q == nullptr) != (a.q_out == nullptr)) return VT_ERR_INVALID_ARG;
  if (a.q && a.q == a.q_out && a.q_stride != a.q_out_stride) return VT_ERR_INVALID_ARG;
  if (dtype == VT_E4M3 && (!a.k_scale || !a.v_scale || !aligned(a.k_scale, 4) || !aligned(a.v_scale, 4)))
    return VT_ERR_INVALID_ARG;
  if (a.kv_heads <= 0 || (a.q && a.q_heads <= 0) || a.max_blocks <= 0 || a.num_blocks <= 0 || block_size <= 0 ||
      a.head_dim <= 0)
    return VT_ERR_INVALID_ARG;
  if (!aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) ||
      !aligned(a.q, 16) || !aligned(a.q_out, 16) || !aligned(a.q_starts, 4) || !aligned(a.block_tables, 4) ||
      !aligned(a.context_lens, 4) || !aligned(a.positions, 4))
    return VT_ERR_INVALID_ARG;
  if (!rotation_ok(a.inv_freq, a.rot_dim, a.head_dim, interleaved, a.amplitude, true)) return VT_ERR_INVALID_ARG;
  if (a.num_tokens > kMaxTokens || a.num_seqs > kMaxTokens) return VT_ERR_UNSUPPORTED;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256 && a.head_dim != 512) return VT_ERR_UNSUPPORTED;
  if (a.head_dim == 512 && dtype != VT_BF16) return VT_ERR_UNSUPPORTED;
  if (block_size != kPage) return VT_ERR_UNSUPPORTED;
  const int es = dtype == VT_F32 ? 4 : 2;
  if (!stride_ok(a.k_stride, a.kv_heads, a.head_dim, es) || !stride_ok(a.v_stride, a.kv_heads, a.head_dim, es) ||
      (a.q && !stride_ok(a.q_stride, a.q_heads, a.head_dim, es)))
    return VT_ERR_INVALID_ARG;
  if (static_cast<long long>(a.num_blocks) * kPage > 0x7fffffffLL ||
      static_cast<long long>(a.max_blocks) * kPage > 0x7fffffffLL)
    return VT_ERR_UNSUPPORTED;
  if ((static_cast<long long>(a.q_heads) + 2ll * a.kv_heads) * a.head_dim * kMaxTokensPerBlock > 0x3fffffffLL)
    return VT_ERR_UNSUPPORTED;
  int sms = 0;
  const vt_status st = current_sms(&sms);
  if (st != VT_OK) return st;
  cudaError_t e;
  if (dtype == VT_BF16)
    e = launch_rope<__nv_bfloat16, __nv_bfloat16, true>(a, interleaved, sms, stream);
  else if (dtype == VT_F32)
    e = launch_rope<float, float, true>(a, interleaved, sms, stream);
  else
    e = launch_rope<__nv_bfloat16, uint8_t, true>(a, interleaved, sms, stream);
  return e == cudaSuccess ? VT_OK : cuda_fail(e, "append launch");
}

RopeArgs append_args(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v, const void* q,
                     const float* k_scale, const float* v_scale, const int32_t* q_starts,
                     const int32_t* block_tables, const int32_t* context_lens, const int32_t* positions,
                     const double* inv_freq, int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                     int head_dim, int rot_dim, float amplitude, long long q_stride, long long k_stride,
                     long long v_stride, int max_blocks_per_seq, int num_blocks) {
  RopeArgs a{};
  a.q = q;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.q_out_stride = static_cast<long long>(num_q_heads) * head_dim;
  a.q_heads = q ? num_q_heads : 0;
  a.k = k;
  a.v = v;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.kv_heads = num_kv_heads;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.q_starts = q_starts;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.num_seqs = num_seqs;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.num_tokens = num_tokens;
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.amplitude = amplitude;
  return a;
}

}  // namespace
}  // namespace vt

extern "C" {

vt_status vt_rope_frequencies(double* inv_freq, float* amplitude, int rot_dim, double base,
                              const vt_rope_stretch* stretch) {
  if (!inv_freq || !amplitude || rot_dim <= 0 || rot_dim % 2 != 0 || !std::isfinite(base) || !(base > 1.0))
    return VT_ERR_INVALID_ARG;
  vt_rope_stretch s{};
  if (stretch) s = *stretch;
  if (s.kind < VT_ROPE_PLAIN || s.kind > VT_ROPE_BANDED) return VT_ERR_INVALID_ARG;
  if (s.kind != VT_ROPE_PLAIN && (!std::isfinite(s.factor) || !(s.factor > 0.0))) return VT_ERR_INVALID_ARG;
  if (s.kind == VT_ROPE_NTK && rot_dim < 4) return VT_ERR_INVALID_ARG;
  if ((s.kind == VT_ROPE_YARN || s.kind == VT_ROPE_BANDED) &&
      (!std::isfinite(s.original_context) || !(s.original_context > 0.0) || !std::isfinite(s.beta_fast) ||
       !(s.beta_slow > 0.0) || !(s.beta_fast > s.beta_slow)))
    return VT_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925;
  const double b = s.kind == VT_ROPE_NTK ? base * std::pow(s.factor, rot_dim / (rot_dim - 2.0)) : base;
  // YaRN's ramp runs over the pair index, between the (fractional) pairs that make beta_fast and beta_slow turns
  double first = 0.0, last = 0.0;
  if (s.kind == VT_ROPE_YARN) {
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(s.original_context / (turns * kTwoPi)) / (2.0 * std::log(base));
    };
    first = std::fmax(std::floor(pair_of(s.beta_fast)), 0.0);
    last = std::fmin(std::ceil(pair_of(s.beta_slow)), rot_dim - 1.0);
    if (!(last > first)) last = first + 0.001;
  }
  for (int j = 0; j < rot_dim / 2; ++j) {
    const double f = std::pow(b, -2.0 * j / rot_dim);
    double keep = 1.0;  // share of the pair that keeps its frequency
    if (s.kind == VT_ROPE_YARN) {
      keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (j - first) / (last - first)));
    } else if (s.kind == VT_ROPE_BANDED) {
      const double turns = s.original_context * f / kTwoPi;
      keep = std::fmin(1.0, std::fmax(0.0, (turns - s.beta_slow) / (s.beta_fast - s.beta_slow)));
    } else if (s.kind == VT_ROPE_LINEAR) {
      keep = 0.0;
    }
    const bool stretched = s.kind == VT_ROPE_LINEAR || s.kind == VT_ROPE_YARN || s.kind == VT_ROPE_BANDED;
    inv_freq[j] = stretched ? keep * f + (1.0 - keep) * f / s.factor : f;
  }
  *amplitude = s.kind == VT_ROPE_YARN && s.factor > 1.0 ? static_cast<float>(0.1 * std::log(s.factor) + 1.0) : 1.0f;
  return VT_OK;
}

vt_status vt_rope(void* out, const void* x, const int32_t* positions, const double* inv_freq, int num_tokens,
                  int num_heads, int head_dim, int rot_dim, int interleaved, float amplitude, long long x_stride,
                  long long out_stride, vt_stream_t stream, vt_dtype dtype) {
  using namespace vt;
  if (num_tokens < 0) return VT_ERR_INVALID_ARG;
  if (num_tokens == 0) return VT_OK;
  if (!out || !x || !positions || (dtype != VT_BF16 && dtype != VT_F32) || num_heads <= 0 || head_dim <= 0)
    return VT_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(x, 16) || !aligned(positions, 4)) return VT_ERR_INVALID_ARG;
  if (!rotation_ok(inv_freq, rot_dim, head_dim, interleaved, amplitude, false)) return VT_ERR_INVALID_ARG;
  const int es = dtype == VT_F32 ? 4 : 2;
  if (!stride_ok(x_stride, num_heads, head_dim, es) || !stride_ok(out_stride, num_heads, head_dim, es))
    return VT_ERR_INVALID_ARG;
  if (out == x && x_stride != out_stride) return VT_ERR_INVALID_ARG;
  if (num_tokens > kMaxTokens || head_dim % 8 != 0 || head_dim > 1024) return VT_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_heads) * head_dim * kMaxTokensPerBlock > 0x3fffffffLL) return VT_ERR_UNSUPPORTED;
  RopeArgs a{};
  a.q = x;
  a.q_out = out;
  a.q_stride = x_stride;
  a.q_out_stride = out_stride;
  a.q_heads = num_heads;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.num_tokens = num_tokens;
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.amplitude = amplitude;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return guarded([&] {
    int sms = 0;
    const vt_status st = current_sms(&sms);
    if (st != VT_OK) return st;
    const cudaError_t e = dtype == VT_BF16 ? launch_rope<__nv_bfloat16, __nv_bfloat16, false>(a, interleaved, sms, s)
                                           : launch_rope<float, float, false>(a, interleaved, sms, s);
    return e == cudaSuccess ? VT_OK : cuda_fail(e, "rope launch");
  });
}

vt_status vt_paged_kv_append(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v, const void* q,
                             const int32_t* q_starts, const int32_t* block_tables, const int32_t* context_lens,
                             const int32_t* positions, const double* inv_freq, int num_seqs, int num_tokens,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size, int rot_dim,
                             int interleaved, float amplitude, long long q_stride, long long k_stride,
                             long long v_stride, vt_stream_t stream, int max_blocks_per_seq, int num_blocks,
                             vt_dtype dtype) {
  if (dtype == VT_E4M3) return VT_ERR_INVALID_ARG;
  return vt::guarded([&] {
    return vt::append(vt::append_args(k_cache, v_cache, q_out, k, v, q, nullptr, nullptr, q_starts, block_tables,
                                      context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads,
                                      num_kv_heads, head_dim, rot_dim, amplitude, q_stride, k_stride, v_stride,
                                      max_blocks_per_seq, num_blocks),
                      block_size, interleaved, reinterpret_cast<cudaStream_t>(stream), dtype);
  });
}

vt_status vt_paged_kv_append_fp8(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v,
                                 const void* q, const float* k_scale, const float* v_scale, const int32_t* q_starts,
                                 const int32_t* block_tables, const int32_t* context_lens, const int32_t* positions,
                                 const double* inv_freq, int num_seqs, int num_tokens, int num_q_heads,
                                 int num_kv_heads, int head_dim, int block_size, int rot_dim, int interleaved,
                                 float amplitude, long long q_stride, long long k_stride, long long v_stride,
                                 vt_stream_t stream, int max_blocks_per_seq, int num_blocks) {
  return vt::guarded([&] {
    return vt::append(vt::append_args(k_cache, v_cache, q_out, k, v, q, k_scale, v_scale, q_starts, block_tables,
                                      context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads,
                                      num_kv_heads, head_dim, rot_dim, amplitude, q_stride, k_stride, v_stride,
                                      max_blocks_per_seq, num_blocks),
                      block_size, interleaved, reinterpret_cast<cudaStream_t>(stream), VT_E4M3);
  });
}

}  // extern "C"
