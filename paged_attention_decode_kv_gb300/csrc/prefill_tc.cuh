// Ragged prefill over the paged cache on the 5th-generation tensor cores.
//
// Per item (prefill_plan.cuh): NT tiles of 128 query rows (tokens x the query
// heads of one kv head), against 128 keys (four pages) at a time:
//   S = Q K^T   tcgen05.mma, Q and K in shared memory, S in tensor memory;
//   P = 2^(scale S - m), rows masked and summed in registers, one row to a
//       thread, rounded to bf16 (f16 against codes, whose V is f16: at most
//       2^-8 or 2^-11 of a weight) and written over S in tensor memory;
//   O += P V    tcgen05.mma, P from tensor memory, V as it lies in its pages
//       (token-major, i.e. the N-major right operand), O in tensor memory.
// A row's reference maximum m moves only when a score passes it by more than
// 2^8 (weights then stay below 2^8, sums below 2^8 n, and the quotient is
// the same), so O is rescaled a few times an item and not once a block.
//
// One bf16 term a weight is a choice of speed: results are off by 0.0020 to
// 0.0023 of their rms, where the rounding of a result alone makes 0.0017.  With
// two terms, as the decode has them, that is what is left, but P V is twice the
// products: an 8192-token prompt (below) takes 485 us where one term takes 350,
// GQA-8 chunks 215 where 160, a few new tokens over long contexts 213 where 198.
// f16 weights against codes add nothing that shows.
//
// Roles: one warp loads (walks the CTA's share, passes its items on through a
// queue, and fetches Q tiles and K and V pages by TMA into two rings of
// stages), two issue MMAs, one prepares V (below; for codes four warps, which
// widen them too); a warpgroup of softmax threads a tile; one warpgroup writes
// results.  With two tiles (head_dim 64 and 128) each has an issuer of its
// own, and one tile's products run while the other's softmax does.  With one
// tile (head_dim 256 and 512, whose O takes half of tensor memory) S is
// double-buffered, one warp issues Q K^T, a block ahead, and the other P V.
//
// What bounds it: a tile's softmax (1300 cycles a block of 128 keys, 512 of them
// exponentials) and its products (16 MMAs of 64 cycles) follow one another, and
// two tiles take 2900 to 3000 cycles where the products alone take 2048: 8192
// tokens, 32 q / 8 kv heads, head_dim 128 in 350 us a call of calls in a row,
// 1570 TFLOP/s, 0.84 of the measured 1863 (a call at a time, with its scratch and
// inputs out of L2, 365 to 376).  Short items keep the tensor pipe 15 % busy
// (48 prompts of 1 to 401, head_dim 64): waits are two fifths of their stalls, Q
// and O having one buffer a tile; instruction fetch, which bound them while the
// code was 100 KB, is a tenth, so what is inlined often or runs once an item is
// kept short.
//
// V preparation: in blocks that some row of the item may see only in part,
// slots outside the item's keys are zeroed (0 * NaN is NaN, whatever P is),
// and values that are not finite in the keys only some rows see are zeroed
// too and given back to the rows that do attend to them at the end.
#pragma once

#include <math_constants.h>

#include "decode_kernel.cuh"
#include "packed.cuh"
#include "prefill_variants.cuh"
#include "tcgen05.cuh"

namespace vt {

template <bool FP8, int D, int NT, int DV, int KCW, int NSK, int VK, int NSV, int NSW = 1>
struct TcConfig {
  static constexpr bool kFp8 = FP8;                    // E4M3 codes in the cache, else bf16
  static constexpr int kD = D, kNT = NT, kDV = DV;
  static constexpr int kElem = FP8 ? 1 : 2;            // bytes of a cached element
  // One TMA box and one swizzled block are kCols columns wide: 128-byte rows,
  // or 64-byte ones for the 64 codes of an FP8 head_dim 64.
  static constexpr int kCols = FP8 ? (D < 128 ? D : 128) : 64;
  static constexpr int kRow = kCols * kElem;
  static constexpr uint32_t kSwizzle = kRow == 128 ? 2 : 4;
  // A K stage: 128 keys x KCW columns.  A V stage: VK keys x all DV columns,
  // so that an MMA of P V is as wide as O (one MMA, not several narrow ones).
  static constexpr int kStagesK = NSK, kStagesV = NSV, kVK = VK;
  static constexpr int kKBlocks = KCW / kCols, kVBlocks = DV / kCols;  // swizzled blocks of a stage
  static constexpr int kKChunks = D / KCW;             // K stages of a block of keys
  static constexpr int kKBlockBytes = kPfBlock * kRow, kVBlockBytes = VK * kRow;
  static constexpr int kKBytes = kKBlocks * kKBlockBytes, kVBytes = kVBlocks * kVBlockBytes;
  static constexpr int kQBytes = 128 * D * 2;          // FP8: two E4M3 terms of each element, high terms first
  // What P V reads: V's stages (bf16), or for codes stages of their f16 values
  // in the same layout (64-column blocks of 128-byte rows).
  static constexpr int kStagesP = FP8 ? NSW : NSV;
  static constexpr int kPBlockBytes = VK * 128, kPBytes = DV / 64 * kPBlockBytes;
  static constexpr int kThreads = NT * 128 + 256 + (FP8 ? 128 : 0);  // softmax, epilogue, control; widening
  static constexpr int kTmemO = 256;                   // S of tile (or buffer) i at 128 i
  static constexpr int kNumS = 2;                      // tiles, or buffers of one tile
  static constexpr int kItems = 4;                     // queue of items
  static_assert(VK == 128 || VK == 64 || VK == 32, "whole pages, whole halves of a block");
  static_assert(4 * kKBlocks <= 32 && VK / kPfPage * kVBlocks <= 32, "a lane for each box of a stage");
};

// Widened stages of V, for codes.
template <typename C, bool FP8>
struct TcWide {};
template <typename C>
struct TcWide<C, true> {
  alignas(1024) unsigned char w[C::kStagesP][C::kPBytes];
};

template <typename C>
struct TcSmem {
  alignas(1024) unsigned char q[C::kNT][C::kQBytes];
  alignas(1024) unsigned char k[C::kStagesK][C::kKBytes];
  alignas(1024) unsigned char v[C::kStagesV][C::kVBytes];
  TcWide<C, C::kFp8> wide;
  alignas(8) unsigned long long k_full[C::kStagesK], k_empty[C::kStagesK];
  unsigned long long v_full[C::kStagesV], v_empty[C::kStagesV], v_ready[C::kStagesV];
  unsigned long long w_full[C::kStagesP], w_empty[C::kStagesP];  // FP8
  unsigned long long q_full[C::kNT], q_empty[C::kNT];
  unsigned long long s_full[C::kNumS], s_free[C::kNumS];  // s_free: one tile only
  unsigned long long p_ready[2][C::kNumS];                // weights of the block's first and second 64 keys
  unsigned long long l_full[C::kNT], l_free[C::kNT];
  unsigned long long o_full[C::kNT], o_free[C::kNT];
  unsigned long long item_full[C::kItems], item_empty[C::kItems];
  unsigned long long turn[2], drain[2];
  PfItem items[C::kItems];
  alignas(16) int4 spans[C::kItems][C::kNT];  // of the items' tiles
  float2 ml[C::kNT][128];               // rows' (reference maximum, sum) for the epilogue
  uint32_t tmem;
  volatile int stage_bad[C::kStagesV];  // a page id of this stage was out of range
  volatile int stage_fix[C::kStagesV];  // V preparation took out a value that is not finite
  volatile int flags[C::kNT];           // of the item whose O is full
  alignas(4) volatile unsigned char w_flags[C::kStagesP][4];  // FP8: of the four widening warps
  // A wait that gave up: status bit | thread << 8 (0: none), its barrier, its parity.
  alignas(16) volatile uint32_t abort_at[4];
};

// An item's start and end cost as much as 1.5 blocks of keys; with codes the
// softmax threads write Q's terms first, and it is three.  What the shares
// assume is what balances them: a 4096-token prompt (32 q / 8 kv heads of 128)
// takes 140 us over codes with 384, 169 with 128, 145 with 768; an 8192-token
// one over bf16 383 us with 192, 389 with 128, 387 with 256.
template <bool FP8>
constexpr int kItemWeight = FP8 ? 384 : 192;

// Weights are 2^(score - m) with m at most kLazy below the largest score.
constexpr float kLazy = 8.f;

enum : int { kItemBad = 1, kItemFix = 2 };

// Key blocks [jb, je) of this piece that tile t of the item takes part in.
struct TileSpan {
  int jb, je;
  int tok0, ntok;  // the tile's tokens
};
__device__ __forceinline__ TileSpan tile_span(const PrefillArgs& a, const PfItem& it, int t, int tile_toks) {
  TileSpan s;
  s.tok0 = t * tile_toks;
  s.ntok = max(0, min(tile_toks, it.ntok - s.tok0));
  const int first = it.pos0 + s.tok0;
  const int lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
  s.jb = max(it.kb0, (lo - it.lo) / kPfBlock);
  s.je = s.ntok > 0 ? min(it.kb1, (first + s.ntok - it.lo + kPfBlock - 1) / kPfBlock) : 0;
  s.je = max(s.jb, s.je);
  return s;
}

// Whether block j holds keys that not every row of the item sees.
__device__ __forceinline__ bool needs_prep(const PrefillArgs& a, const PfItem& it, int j) {
  const int k0 = it.lo + j * kPfBlock;
  return k0 + kPfBlock > it.pos0 + 1 || (a.window > 0 && k0 < it.hi - a.window);
}

// V stages of block j.
template <typename C>
__device__ __forceinline__ int v_stages(const PfItem& it, int j) {
  return (min(kPfBlock, it.hi - (it.lo + j * kPfBlock)) + C::kVK - 1) / C::kVK;
}

// Position in a ring of stages.
template <int N>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == N) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Adds the values that preparation took out to a row's sums, in tensor memory
// from column 0 of `o` on: they are not finite, so neither is the result.  They
// lie among the keys that only some rows see, as many at either end as the item
// has tokens and whatever the context is (a walk over a whole context of 30000
// keys took longer than a bounded wait of 8 million cycles).  A warp looks at 32
// of them at a time.  (All threads of a warp together; rare, so compact.)
template <bool FP8>
__device__ __forceinline__ void add_taken_values(const PrefillArgs& a, const PfItem& it, int head_dim, int pos, int cols,
                                              uint32_t o) {
  const int lane = threadIdx.x & 31;
  const int first = max(it.lo_exact, it.lo + it.kb0 * kPfBlock);
  const int last = min(it.hi, it.lo + it.kb1 * kPfBlock);
  // before `early` some rows' windows have not begun, from `late` on are some rows' later tokens
  const int early = a.window > 0 ? min(last, max(first, it.hi - a.window)) : first;
  const int late = min(last, max(early, it.pos0 + 1));
#pragma unroll 1
  for (int c = 0; c < cols; ++c) {
    float add = 0.f;
#pragma unroll 1
    for (int t0 = first; t0 < last; t0 += 32) {
      if (t0 >= early && t0 < late) t0 = late;
      const int t = t0 + lane;
      float x = 0.f;
      if (t < last && (t < early || t >= late)) {
        const int page = a.block_tables[static_cast<long long>(it.b) * a.max_blocks + t / kPfPage];
        if (page >= 0 && page < a.num_blocks) {
          const long long at = ((static_cast<long long>(page) * kPfPage + t % kPfPage) * a.num_kv_heads + it.head) *
                                   head_dim + it.part * cols + c;
          if constexpr (FP8)
            x = (static_cast<const uint8_t*>(a.v_cache)[at] & 0x7f) == 0x7f ? CUDART_NAN_F : 0.f;
          else
            x = __bfloat162float(static_cast<const __nv_bfloat16*>(a.v_cache)[at]);
        }
      }
      unsigned taken = __ballot_sync(0xffffffffu, !isfinite(x));
#pragma unroll 1
      for (; taken; taken &= taken - 1) {
        const int i = __ffs(taken) - 1, key = t0 + i;
        const float y = __shfl_sync(0xffffffffu, x, i);
        if (key <= pos && (a.window == 0 || key > pos - a.window)) add += y;
      }
    }
    uint32_t sum;
    tmem_ld1(o + c, sum);
    tmem_wait_ld();
    tmem_st1(o + c, __float_as_uint(__uint_as_float(sum) + add));
    tmem_wait_st();
  }
}

// A word whose elements that are not finite (exponents of all ones; the E4M3
// codes 0x7f and 0xff) carry into the bits of kCarry, and all ones in their place.
template <bool FP8>
constexpr uint32_t kCarry = FP8 ? 0x80808080u : 0x80008000u;
template <bool FP8>
__device__ __forceinline__ uint32_t carries(uint32_t w) {
  return FP8 ? (w & 0x7f7f7f7fu) + 0x01010101u : (w & 0x7f807f80u) + 0x00800080u;
}
template <bool FP8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  const uint32_t m = carries<FP8>(w) & kCarry<FP8>;
  return FP8 ? (m >> 7) * 0xffu : (m >> 15) * 0xffffu;
}

// Two floats as E4M3 terms, hi + lo: lo is the rest that hi leaves, itself
// rounded, so together they keep 8 significant bits (and 2^-10 absolutely).
// The rest is taken in f16, whose 11 bits hold it exactly.
__device__ __forceinline__ void e4m3x2_terms(float x, float y, uint32_t& hi, uint32_t& lo) {
  uint32_t h, back, rest;
  uint16_t a, b;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(h));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(a));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h), "r"(back));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(rest));
  hi = a;
  lo = b;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// In each group of four lanes: lane k's x[r] becomes what lane r held in x[k].
__device__ __forceinline__ void transpose4(uint4 (&x)[4], int lane) {
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      const bool up = lane & d;
      uint4 give = up ? x[i] : x[i | d];
      give.x = __shfl_xor_sync(0xffffffffu, give.x, d);
      give.y = __shfl_xor_sync(0xffffffffu, give.y, d);
      give.z = __shfl_xor_sync(0xffffffffu, give.z, d);
      give.w = __shfl_xor_sync(0xffffffffu, give.w, d);
      if (up)
        x[i] = give;
      else
        x[i | d] = give;
    }
  }
}

// Probes an mbarrier phase until it is met (1), or another wait has given up or
// this one takes more than `limit` clock cycles and says so in `abort_at` (0).
__device__ __forceinline__ uint32_t wait_or_abort(unsigned long long* bar, uint32_t parity, volatile uint32_t* abort_at,
                                                  uint32_t limit, uint32_t code) {
  uint32_t met;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 t0, t;\n\tmov.u32 t0, %%clock;\n\t"
      "PROBE_%=:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra MET_%=;\n\t"
      "ld.volatile.shared.u32 t, [%3];\n\tsetp.ne.u32 q, t, 0;\n\t@q bra MET_%=;\n\t"
      "mov.u32 t, %%clock;\n\tsub.u32 t, t, t0;\n\tsetp.le.u32 q, t, %4;\n\t@q bra PROBE_%=;\n\t"
      "mov.u32 t, %%tid.x;\n\tshl.b32 t, t, 8;\n\tor.b32 t, t, %5;\n\t"
      "st.volatile.shared.v4.u32 [%3], {t, %1, %2, %5};\n\t"
      "MET_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(met)
      : "r"(smem_addr(bar)), "r"(parity), "r"(smem_addr(const_cast<uint32_t*>(abort_at))), "r"(limit), "r"(code)
      : "memory");
  return met;
}

// Everything a role needs besides its own state.
template <typename C>
struct TcRole {
  const PrefillArgs& a;
  TcSmem<C>& s;
  int lane;
  bool live = true;  // false once a bounded wait has given up; uniform over a warp

  // Bounded wait on an mbarrier phase.  A wait that passes the limit (clock
  // cycles) raises the CTA's abort flag, with what to report at the end, and
  // every other wait then gives up too.  (Few instructions: it is inlined
  // often, and the roles' loops together have to stay in the instruction
  // caches.)
  __device__ __forceinline__ bool wait(unsigned long long* bar, uint32_t parity, unsigned code) {
    // (most waits end in the first probe, which sleeps a while: with the clock
    // read before it an 8192-token prompt took 366 us where this takes 352)
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u)), 1)) return live;
    const uint32_t met = wait_or_abort(bar, parity & 1u, s.abort_at, a.wait_limit, code);
    if (__builtin_expect(!__all_sync(0xffffffffu, met), 0)) live = false;
    return live;
  }
  // For copies and MMAs in flight, whatever the abort flag says.
  __device__ __forceinline__ void drain(unsigned long long* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity & 1u))
      if (clock64() - t0 > kDrainLimitCycles) {
        s.abort_at[0] = kStatusDrain | (threadIdx.x << 8);
        break;
      }
    __syncwarp();
  }
  // Item n of the CTA's share; false at the end.
  __device__ __forceinline__ bool item(uint32_t n, PfItem& it) {
    if (!wait(&s.item_full[n % C::kItems], n / C::kItems, kStatusSync)) return false;
    it = s.items[n % C::kItems];
    return it.b >= 0;
  }
  // The blocks and tokens of its tile t.
  __device__ __forceinline__ TileSpan span(uint32_t n, int t) {
    const int4 x = s.spans[n % C::kItems][t];
    return TileSpan{x.x, x.y, x.z, x.w};
  }
  __device__ __forceinline__ void item_done(uint32_t n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.item_empty[n % C::kItems]);
  }
};

// --------------------------------------------------------------------- loader
template <typename C>
__device__ __forceinline__ void tc_loader(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                          const PrefillArgs& a, TcSmem<C>& s, PfWalk& w, int lane) {
  TcRole<C> role{a, s, lane};
  Ring<C::kStagesK> rk;
  Ring<C::kStagesV> rv;
  uint32_t nq = 0, used = 0, items = 0;  // nq: parity of a tile's Q loads in bit 16 t
  long long nk = 0, nv = 0;
  int blocks = 0;
  const int tile_toks = a.tile_tokens / C::kNT;
  int ids = 0, ids_at = -1;  // 32 table entries, one a lane, from page index ids_at
  PfItem it{};
  // This lane's box of a stage whose first page is the item's page p0: page
  // p0 + box % pages, column block box / pages.
  auto read_ids = [&](int p0) {
    if (ids_at < 0 || p0 < ids_at || p0 + 4 > ids_at + 32) {
      ids_at = max(0, p0 - 4);  // K runs a block ahead of V
      const int at = ids_at + lane;
      ids = at < a.max_blocks ? a.block_tables[static_cast<long long>(it.b) * a.max_blocks + at] : 0;
    }
  };
  auto page_of = [&](int p0, int i) {
    read_ids(p0);
    return __shfl_sync(0xffffffffu, ids, p0 - ids_at + i);
  };
  auto load_k = [&](int j) {
    const int k0 = it.lo + j * kPfBlock;
    const int pages = min(kPfBlock, it.hi - k0 + kPfPage - 1) / kPfPage;  // those that hold keys of the item
    int page = page_of(k0 / kPfPage, lane & 3);
    const bool use = (lane & 3) < pages && lane < 4 * C::kKBlocks;
    if (page < 0 || page >= a.num_blocks) page = 0;  // (load_v reports it)
#pragma unroll 1
    for (int c = 0; c < C::kKChunks; ++c) {
      if (!role.wait(&s.k_empty[rk.stage], rk.phase ^ 1u, kStatusEmpty)) return;
      if (lane == 0) mbar_arrive_expect_tx(&s.k_full[rk.stage], pages * C::kKBlocks * kPfPage * C::kRow);
      __syncwarp();
      if (use)
        tma_load_4d(s.k[rk.stage] + (lane >> 2) * C::kKBlockBytes + (lane & 3) * kPfPage * C::kRow, &tk, 0,
                    page * kPfPage, c * C::kKBlocks + (lane >> 2), it.head, &s.k_full[rk.stage]);
      ++nk;
      rk.next();
    }
  };
  auto load_v = [&](int j) {
    constexpr int kPages = C::kVK / kPfPage;  // of a stage
    const int stages = v_stages<C>(it, j);
#pragma unroll 1
    for (int i = 0; i < stages; ++i) {
      const int k0 = it.lo + j * kPfBlock + i * C::kVK;
      const int pages = min(C::kVK, it.hi - k0 + kPfPage - 1) / kPfPage;
      int page = page_of((it.lo + j * kPfBlock) / kPfPage, i * kPages + lane % kPages);
      const bool use = lane % kPages < pages && lane < kPages * C::kVBlocks;
      const bool bad = use && (page < 0 || page >= a.num_blocks);
      const bool any_bad = __any_sync(0xffffffffu, bad);
      if (bad) page = 0;
      if (!role.wait(&s.v_empty[rv.stage], rv.phase ^ 1u, kStatusEmpty)) return;
      if (lane == 0) {
        s.stage_bad[rv.stage] = any_bad;
        mbar_arrive_expect_tx(&s.v_full[rv.stage], pages * C::kVBlocks * kPfPage * C::kRow);
      }
      __syncwarp();
      if (use)
        tma_load_4d(s.v[rv.stage] + (lane / kPages) * C::kVBlockBytes + (lane % kPages) * kPfPage * C::kRow, &tv, 0,
                    page * kPfPage, it.part * C::kVBlocks + lane / kPages, it.head, &s.v_full[rv.stage]);
      ++nv;
      rv.next();
    }
  };
  while (role.live) {
    const bool more = w.next(a, it);
    if (!role.wait(&s.item_empty[items % C::kItems], (items / C::kItems) ^ 1u, kStatusEmpty)) break;
    if (!more) it.b = -1;
    if (lane < C::kNT) {
      const TileSpan sp = tile_span(a, it, lane, tile_toks);
      s.spans[items % C::kItems][lane] = make_int4(sp.jb, sp.je, sp.tok0, sp.ntok);
      if (lane == 0) s.items[items % C::kItems] = it;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.item_full[items % C::kItems]);
    if (!more) break;
    ids_at = -1;
    if (it.kb1 > it.kb0) read_ids((it.lo + it.kb0 * kPfBlock) / kPfPage);  // on their way while Q is asked for
#pragma unroll 1
    for (int t = 0; t < C::kNT && !C::kFp8; ++t) {
      const TileSpan sp = role.span(items, t);
      if (sp.je <= sp.jb) continue;
      if (!role.wait(&s.q_empty[t], (nq >> (16 * t)) ^ 1u, kStatusEmpty)) break;
      nq ^= 1u << (16 * t);
      used |= 1u << t;
      if (lane == 0) mbar_arrive_expect_tx(&s.q_full[t], tile_toks * a.group * C::kD * 2);
      __syncwarp();
      if (lane < C::kD / 64)
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(s.q[t] + lane * 128 * 128)),
            "l"(reinterpret_cast<uint64_t>(&tq)), "r"(0), "r"(0), "r"(it.row0 + sp.tok0), "r"(lane), "r"(it.head),
            "r"(smem_addr(&s.q_full[t]))
            : "memory");
    }
#pragma unroll 1
    for (int j = it.kb0 - 1; j < it.kb1 && role.live; ++j) {  // K of block j + 1, then V of block j
      if (j + 1 < it.kb1) {
        if (static_cast<int>(blockIdx.x) == a.withhold_cta && blocks >= a.withhold_block) {
          role.live = false;  // test hook: an issuer's wait for this block runs out
          break;
        }
        ++blocks;
        load_k(j + 1);
      }
      if (role.live && j >= it.kb0) load_v(j);
    }
    ++items;
  }
  if (!role.live) {
    // let this CTA's copies land before it exits
#pragma unroll 1
    for (long long k = 1; k <= (nk < C::kStagesK ? nk : C::kStagesK); ++k)
      role.drain(&s.k_full[(nk - k) % C::kStagesK], static_cast<uint32_t>((nk - k) / C::kStagesK));
#pragma unroll 1
    for (long long k = 1; k <= (nv < C::kStagesV ? nv : C::kStagesV); ++k)
      role.drain(&s.v_full[(nv - k) % C::kStagesV], static_cast<uint32_t>((nv - k) / C::kStagesV));
    for (int t = 0; t < C::kNT; ++t)
      if (used >> t & 1u) role.drain(&s.q_full[t], (nq >> (16 * t)) ^ 1u);
  }
}

// --------------------------------------------------------------------- MMA issue
// With two tiles, issuer `who` owns tile `who`: Q K^T of block j + 1 follows
// P V of block j on the same thread, which orders them (P lies over S).  With
// one tile, issuer 0 runs Q K^T a block ahead into the other S buffer and
// issuer 1 runs P V; s_free hands the buffers back.
template <typename C>
__device__ __forceinline__ void tc_issuer(const PrefillArgs& a, TcSmem<C>& s, uint32_t tmem, int who, int lane) {
  constexpr int NT = C::kNT, KS = 16, ROW = C::kRow;  // KS: keys of an MMA of P V
  constexpr bool FP8 = C::kFp8;
  constexpr uint32_t kHi = umma_desc_hi(8 * ROW, C::kSwizzle), kHiP = umma_desc_hi(1024, 2);
  TcRole<C> role{a, s, lane};
  Ring<C::kStagesK> rk;
  Ring<C::kStagesP> rv;
  uint32_t vphase = 0;  // of v_ready, one bit a stage
  uint32_t items = 0, nq = 0, no = 0, np[2] = {}, turns = 0;
  uint32_t nblk = 0;    // one tile: blocks so far, whose parity is the buffer
  const int t = NT == 2 ? who : 0;
  const bool do_qk = NT == 2 || who == 0, do_pv = NT == 2 || who == 1;
  const int tile_toks = a.tile_tokens / C::kNT;
  PfItem it{};

  // S(buf) = Q K^T for block j's keys: the MMAs of chunk c and what follows them.  One lane.
  auto qk_issue = [&](int j, int buf, int c, const TileSpan& sp) {
    const bool active = j >= sp.jb && j < sp.je;
    if (active) {
      const int keys = min(kPfBlock, it.hi - (it.lo + j * kPfBlock));
      const uint32_t idesc = (FP8 ? umma_idesc_e4m3(0)
                                  : umma_idesc_f16(true, 0, false) | (a.neg_scale ? kUmmaNegateA : 0u)) |
                             (static_cast<uint32_t>((keys + 15) / 16 * 2) << 17);
      const uint32_t qa = umma_desc_lo(smem_addr(s.q[t]) + c * C::kKBytes, 16);
      const uint32_t kb = umma_desc_lo(smem_addr(s.k[rk.stage]), 16);
      const uint32_t d = tmem + buf * 128, more = c > 0;
      // (rolled loops: an MMA takes 64 cycles, and unrolled code of a warp that
      // runs once a block is fetched anew each time)
      uint32_t acc = more;
#pragma unroll 1
      for (int b = 0; b < (FP8 ? 2 : 1) * C::kKBlocks; ++b) {
        const int blk = FP8 ? b % C::kKBlocks : b;  // FP8: the high terms of Q, then the low ones
        uint32_t qx = qa + ((blk * C::kKBlockBytes + (FP8 ? b / C::kKBlocks * 128 * C::kD : 0)) >> 4);
        uint32_t kx = kb + ((blk * C::kKBlockBytes) >> 4);
#pragma unroll 1
        for (int k = 0; k < ROW / 32; ++k, qx += 2, kx += 2, acc = 1u) umma_ss<FP8>(d, qx, kHi, kx, kHi, idesc, acc);
      }
    }
    umma_commit(&s.k_empty[rk.stage]);
    if (active && c == C::kKChunks - 1) {
      umma_commit(&s.s_full[buf]);
      if (j == sp.je - 1) umma_commit(&s.q_empty[t]);
    }
  };
  auto qk = [&](int j, int buf, const TileSpan& sp) {
#pragma unroll 1
    for (int c = 0; c < C::kKChunks; ++c) {
      if (!role.wait(&s.k_full[rk.stage], rk.phase, kStatusFull)) return;
      tc_fence_after();
      if (elect_one()) qk_issue(j, buf, c, sp);
      __syncwarp();
      rk.next();
    }
  };
  // The tile's O is whole once its products so far are done.
  auto finish = [&](int flags) {
    if (elect_one()) {
      s.flags[t] = flags;
      umma_commit(&s.o_full[t]);
      mbar_arrive(&s.o_full[t]);
    }
    __syncwarp();
    ++no;
  };
  // Waits for the V stage at hand (and its preparation, where block j needs it).
  auto v_here = [&](bool prepared, int& flags) {
    if constexpr (FP8) {
      if (!role.wait(&s.w_full[rv.stage], rv.phase, kStatusFull)) return false;
      const uint32_t f = *reinterpret_cast<volatile uint32_t*>(const_cast<unsigned char*>(s.w_flags[rv.stage]));
      if (f) flags |= (f | f >> 8 | f >> 16 | f >> 24) & 0xffu;
    } else {
      if (!role.wait(&s.v_full[rv.stage], rv.phase, kStatusFull)) return false;
      if (prepared) {
        if (!role.wait(&s.v_ready[rv.stage], vphase >> rv.stage, kStatusSync)) return false;
        vphase ^= 1u << rv.stage;
        if (s.stage_fix[rv.stage]) flags |= kItemFix;
      }
      if (s.stage_bad[rv.stage]) flags |= kItemBad;
    }
    return true;
  };
  auto v_addr = [&] {
    if constexpr (FP8)
      return smem_addr(s.wide.w[rv.stage]);
    else
      return smem_addr(s.v[rv.stage]);
  };
  auto v_free = [&] {
    if constexpr (FP8)
      return &s.w_empty[rv.stage];
    else
      return &s.v_empty[rv.stage];
  };
  // k-steps of block j that the tile's rows need
  auto steps_of = [&](int j, const TileSpan& sp) {
    return (min(it.pos0 + sp.tok0 + sp.ntok - (it.lo + j * kPfBlock), kPfBlock) + KS - 1) / KS;
  };
  constexpr int kHalf = kPfBlock / 2 / KS;  // k-steps of half a block
  const uint32_t idesc_pv = umma_idesc_f16(!FP8, C::kDV, true);
  const uint32_t d_pv = tmem + C::kTmemO + t * C::kDV;
  // k-steps [first, last) of P V; vb: the V stage at step `first`.  One lane.
  auto pv_steps = [&](int buf, int first, int last, uint32_t vb, uint32_t acc) {
    uint32_t from = tmem + buf * 128 + first * 8;
#pragma unroll 1
    for (int k = first; k < last; ++k, from += 8, vb += (KS * 128) >> 4, acc = 1u)
      umma_ts(d_pv, from, vb, kHiP, idesc_pv, acc);
  };
  // One tile: O (+)= P(buf) V for block j's keys, V in stages of VK keys.
  auto pv = [&](int j, int buf, const TileSpan& sp, int& flags) {
    const bool prepared = needs_prep(a, it, j);
    const int stages = v_stages<C>(it, j), steps = steps_of(j, sp);
    constexpr int kSteps = C::kVK < 64 ? C::kVK / KS : kHalf;  // of a stage
    constexpr int kPer = kHalf / kSteps;                       // stages of half a block
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      if (!role.wait(&s.p_ready[h][buf], np[buf], kStatusSync)) return;
      if (h == 0 && j == sp.jb && !role.wait(&s.o_free[t], no ^ 1u, kStatusSync)) return;
#pragma unroll 1
      for (int i = 0; i < kPer; ++i) {
        if (h * kPer + i >= stages) continue;
        if (!v_here(prepared, flags)) return;
        tc_fence_after();
        const int first = (h * kPer + i) * kSteps;
        if (elect_one()) {
          pv_steps(buf, first, min(steps, first + kSteps), umma_desc_lo(v_addr(), C::kPBlockBytes),
                   first > 0 || j > sp.jb);
          umma_commit(v_free());
        }
        __syncwarp();
        rv.next();
      }
    }
    ++np[buf];
    if (elect_one()) umma_commit(&s.s_free[buf]);
    __syncwarp();
    if (j == sp.je - 1) finish(flags);
  };

  for (; role.item(items, it); ++items) {
    if (it.kb1 > it.kb0) {
      const TileSpan sp = role.span(items, t);
      int flags = 0;
      if (do_qk && sp.je > sp.jb) {
        if (!role.wait(&s.q_full[t], nq, kStatusFull)) break;
        ++nq;
      }
      if constexpr (NT == 2) {
        static_assert(NT == 1 || (C::kVK == kPfBlock && C::kKChunks == 1), "one stage a block");
        // The tiles take turns: all of one's P V and next Q K^T, then the
        // other's.  Left to themselves the two issuers' MMAs interleave, both
        // tiles wait for twice the products and then both wait for the
        // softmax, in step.  The turn passes when all is issued: passed a few
        // MMAs earlier, the two tiles' products mix again (8192-token prompt
        // 2 % slower).
        const bool both = it.ntok > tile_toks;
        for (int j = it.kb0 - 1; j < it.kb1 && role.live; ++j) {  // P V of block j, then Q K^T of block j + 1
          // What can be waited for ahead of the weights is: after them this
          // thread only issues.
          const bool mine = j >= it.kb0, active = j >= sp.jb && j < sp.je, next = j + 1 < it.kb1;
          if (mine && !v_here(needs_prep(a, it, j), flags)) break;
          if (next && !role.wait(&s.k_full[rk.stage], rk.phase, kStatusFull)) break;
          if (active && j == sp.jb && !role.wait(&s.o_free[t], no ^ 1u, kStatusSync)) break;
          const int steps = active ? steps_of(j, sp) : 0;
          const uint32_t vb = umma_desc_lo(v_addr(), C::kPBlockBytes);
          int from = 0;
          if (active && !both) {  // nothing else to run meanwhile: the first half's products at once
            if (!role.wait(&s.p_ready[0][t], np[0], kStatusSync)) break;
            tc_fence_after();
            from = kHalf;
            if (elect_one()) pv_steps(t, 0, min(steps, kHalf), vb, j > sp.jb);
            __syncwarp();
          }
          // (the turn before the weights, which are there last: a wait costs
          // 250 cycles even if it is over when it begins)
          if (both && !role.wait(&s.turn[t], turns++ ^ (t ^ 1u), kStatusSync)) break;
          if (active && !role.wait(&s.p_ready[1][t], np[0]++, kStatusSync)) break;
          tc_fence_after();
          if (elect_one()) {
            if (active) pv_steps(t, from, steps, vb + ((from * KS * 128) >> 4), from > 0 || j > sp.jb);
            if (mine) umma_commit(v_free());
            if (next) qk_issue(j + 1, t, 0, sp);
            if (both) mbar_arrive(&s.turn[t ^ 1]);
          }
          __syncwarp();
          if (mine) rv.next();
          if (next) rk.next();
          if (active && j == sp.je - 1) finish(flags);
        }
      } else {
        for (int j = it.kb0; j < it.kb1 && role.live; ++j, ++nblk) {
          const int buf = nblk & 1u;
          if (do_qk) {
            if (!role.wait(&s.s_free[buf], (nblk >> 1) ^ 1u, kStatusSync)) break;
            qk(j, buf, sp);
          }
          if (do_pv) pv(j, buf, sp, flags);
        }
      }
    }
    if (!role.live) break;
    role.item_done(items);
  }
  // every MMA has to be done before tensor memory is given back
  __syncwarp();
  if (elect_one()) umma_commit(&s.drain[who]);
  __syncwarp();
  role.drain(&s.drain[who], 0);
}

// --------------------------------------------------------------------- V preparation
template <typename C>
__device__ __forceinline__ void tc_prepare(const PrefillArgs& a, TcSmem<C>& s, int lane) {
  constexpr int KS = 16;
  TcRole<C> role{a, s, lane};
  Ring<C::kStagesV> rv;
  PfItem it{};
  uint32_t items = 0;
  for (; role.item(items, it); ++items) {
#pragma unroll 1
    for (int j = it.kb0; j < it.kb1 && role.live; ++j) {
      const bool prepare = needs_prep(a, it, j);
      const int stages = v_stages<C>(it, j);
#pragma unroll 1
      for (int i = 0; i < stages; ++i, rv.next()) {
        // (stages are passed over in order too: a wait tells phases apart by parity only)
        if (!role.wait(&s.v_full[rv.stage], rv.phase, kStatusFull)) break;
        if (prepare) {
          const int k0 = it.lo + j * kPfBlock + i * C::kVK;
          constexpr int kPieces = C::kRow / 16;  // 16-byte pieces of a slot's row
          constexpr int kLines = 32 / kPieces;   // slots a warp takes at a time
          const int end = min(C::kVK, (it.hi - k0 + KS - 1) / KS * KS);  // slots the products read
          const int lo = min(end, max(0, it.lo_exact - k0)), hi = min(end, max(lo, it.hi - k0));  // item's keys
          const int early = a.window == 0 ? 0 : min(hi, max(lo, it.hi - a.window - k0));  // before it some rows' windows
          const int late = min(hi, max(early, it.pos0 + 1 - k0));                         // from it on later tokens
          // [0, lo) and [hi, end) zeroed; [lo, early) and [late, hi) looked at
          unsigned char* piece = s.v[rv.stage] + lane * 16;
          const int line = lane / kPieces;
          auto zero = [&](int first, int last) {
#pragma unroll 1
            for (int slot = first; slot + line < last; slot += kLines)
#pragma unroll
              for (int cb = 0; cb < C::kVBlocks; ++cb)
                *reinterpret_cast<uint4*>(piece + cb * C::kVBlockBytes + slot * C::kRow) = make_uint4(0, 0, 0, 0);
          };
          bool fix = false;
          auto look = [&](int first, int last) {
            uint32_t seen = 0;
#pragma unroll 1
            for (int slot = first; slot < last; slot += 4 * kLines) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int at = min(slot + u * kLines, last - 1 - line);  // (a piece may be looked at twice)
                if (at < 0) continue;
#pragma unroll
                for (int cb = 0; cb < C::kVBlocks; ++cb) {
                  const uint4 x = *reinterpret_cast<const uint4*>(piece + cb * C::kVBlockBytes + at * C::kRow);
                  seen |= carries<false>(x.x) | carries<false>(x.y) | carries<false>(x.z) | carries<false>(x.w);
                }
              }
            }
            if (!__any_sync(0xffffffffu, seen & kCarry<false>)) return;
#pragma unroll 1
            for (int slot = first; slot + line < last; slot += kLines)
#pragma unroll 1
              for (int cb = 0; cb < C::kVBlocks; ++cb) {
                uint4* at = reinterpret_cast<uint4*>(piece + cb * C::kVBlockBytes + slot * C::kRow);
                uint4 x = *at;
                x.x &= ~not_finite<false>(x.x), x.y &= ~not_finite<false>(x.y);
                x.z &= ~not_finite<false>(x.z), x.w &= ~not_finite<false>(x.w);
                *at = x;
              }
            fix = true;
          };
#pragma unroll 1
          for (int side = 0; side < 2; ++side) {
            zero(side ? hi : 0, side ? end : lo);
            look(side ? late : lo, side ? hi : early);
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            s.stage_fix[rv.stage] = fix;
            mbar_arrive(&s.v_ready[rv.stage]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.v_empty[rv.stage]);
      }
    }
    if (!role.live) break;
    role.item_done(items);
  }
}

// --------------------------------------------------------------------- widening
// FP8: four warps turn V's codes into f16, exactly, in the layout bf16 pages
// have; a code is widened once for the item's 256 rows.  (As E4M3 MMA operands
// codes would need P as two E4M3 terms: 12 more cycles of conversions for two
// weights in the softmax: four chunks of 500 to 2000 tokens took 436 us where
// f16 weights took 381.)  Preparation is part of it.
template <typename C>
__device__ __forceinline__ void tc_widen(const PrefillArgs& a, TcSmem<C>& s, int tid) {
  constexpr int KS = 16;
  const int lane = tid & 31, warp = tid >> 5;
  TcRole<C> role{a, s, lane};
  Ring<C::kStagesV> rv;
  Ring<C::kStagesP> rw;
  PfItem it{};
  uint32_t items = 0;
  for (; role.item(items, it); ++items) {
#pragma unroll 1
    for (int j = it.kb0; j < it.kb1 && role.live; ++j) {
      const bool prepare = needs_prep(a, it, j);
      const int stages = v_stages<C>(it, j);
#pragma unroll 1
      for (int i = 0; i < stages; ++i, rv.next(), rw.next()) {
        if (!role.wait(&s.w_empty[rw.stage], rw.phase ^ 1u, kStatusEmpty)) break;
        if (!role.wait(&s.v_full[rv.stage], rv.phase, kStatusFull)) break;
        const int k0 = it.lo + j * kPfBlock + i * C::kVK;
        const int end = min(C::kVK, (it.hi - k0 + KS - 1) / KS * KS);  // slots the products read
        const unsigned char* src = s.v[rv.stage];
        unsigned char* dst = s.wide.w[rw.stage];
        bool fix = false;
        constexpr int kRowPieces = C::kDV / 16;  // 16 codes each
        constexpr int kPieces = C::kRow / 16;    // of a swizzled block's row
#pragma unroll 2
        for (int p = tid; p < end * kRowPieces; p += 128) {
          const int slot = p / kRowPieces, piece = p % kRowPieces;
          const int cb = piece / kPieces, ch = piece % kPieces;
          const int swz = C::kRow == 128 ? ch ^ (slot & 7) : ch ^ ((slot >> 1) & 3);
          uint4 x = *reinterpret_cast<const uint4*>(src + cb * C::kVBlockBytes + slot * C::kRow + swz * 16);
          if (prepare) {
            const int t = k0 + slot;
            if (t < it.lo_exact || t >= it.hi) {
              x = make_uint4(0, 0, 0, 0);
            } else if (t > it.pos0 || (a.window > 0 && t < it.hi - a.window)) {
              const uint32_t m = (carries<true>(x.x) | carries<true>(x.y) | carries<true>(x.z) | carries<true>(x.w)) &
                                 kCarry<true>;
              if (m) {
                fix = true;
                x.x &= ~not_finite<true>(x.x), x.y &= ~not_finite<true>(x.y);
                x.z &= ~not_finite<true>(x.z), x.w &= ~not_finite<true>(x.w);
              }
            }
          }
          uint4 y[2];
          e4m3x4_to_f16(x.x, y[0].x, y[0].y);
          e4m3x4_to_f16(x.y, y[0].z, y[0].w);
          e4m3x4_to_f16(x.z, y[1].x, y[1].y);
          e4m3x4_to_f16(x.w, y[1].z, y[1].w);
          // two 16-byte pieces of a 128-byte row of 64 columns; the lanes of
          // every other block store them the other way round (no bank conflicts)
          unsigned char* row = dst + (piece >> 2) * C::kPBlockBytes + slot * 128;
          const int at = (piece & 3) * 2, odd = (piece >> 2) & 1;
          *reinterpret_cast<uint4*>(row + (((at + odd) ^ (slot & 7)) << 4)) = odd ? y[1] : y[0];
          *reinterpret_cast<uint4*>(row + (((at + (odd ^ 1)) ^ (slot & 7)) << 4)) = odd ? y[0] : y[1];
        }
        fix = __any_sync(0xffffffffu, fix);
        const bool bad = s.stage_bad[rv.stage] != 0;
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          s.w_flags[rw.stage][warp] = static_cast<unsigned char>((bad ? kItemBad : 0) | (fix ? kItemFix : 0));
          mbar_arrive(&s.w_full[rw.stage]);
          mbar_arrive(&s.v_empty[rv.stage]);
        }
      }
    }
    if (!role.live) break;
    role.item_done(items);
  }
}

// --------------------------------------------------------------------- softmax: one row a thread
template <typename C>
__device__ __forceinline__ void tc_softmax(const PrefillArgs& a, TcSmem<C>& s, uint32_t tmem, int tid) {
  constexpr int D = C::kD, NT = C::kNT, DV = C::kDV, ROW = C::kRow;
  constexpr bool FP8 = C::kFp8;
  const int warp = tid >> 5, lane = tid & 31;
  const int tile_toks = a.tile_tokens / C::kNT;
  const int t = NT == 2 ? warp >> 2 : 0;
  const int row = tid & 127;
  const int tok = pf_token_of(a, row);
  const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, lane in bits 16..
  const uint32_t tO = tmem + lane_base + C::kTmemO + t * DV;
  TcRole<C> role{a, s, lane};
  PfItem it{};
  uint32_t items = 0;
  uint32_t blocks = 0;  // of this tile; one tile: the parity is the buffer
  for (; role.item(items, it); ++items) {
    const TileSpan sp = role.span(items, t);
    const int pos = it.pos0 + sp.tok0 + min(tok, max(sp.ntok, 1) - 1);
    float m = -CUDART_INF_F, l = 0.f;
    float scale = a.scale_log2;  // from a score in tensor memory to the log2 domain
    if constexpr (FP8) {
      // Q as two E4M3 terms in the layout TMA gives K.  (The previous item's last
      // scores are here, so its Q is done with.)  A warp takes its 32 rows a few
      // at a time, 16 elements a lane, the next loads under way while it
      // converts (a row a thread, read twice, took that prompt 203 us where
      // this takes 169).
      if (sp.je > sp.jb) {
        const float ks = a.k_scale[it.head] * (a.neg_scale ? -1.f : 1.f);
        constexpr int kLanes = D / 16, kRows = 32 / kLanes, kSteps = kLanes;  // lanes of a row, rows of a step
        constexpr int kAhead = 2;                                             // steps of a batch of loads
        const int piece = lane % kLanes;
        const int blk = piece / (ROW / 16), ch = piece % (ROW / 16);
        uint4 in[kAhead][2], next[kAhead][2];
        auto load = [&](int step) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int r = (row & ~31) + (step + u) * kRows + lane / kLanes;
            const int rt = pf_token_of(a, r);
            next[u][0] = next[u][1] = make_uint4(0, 0, 0, 0);
            if (step < kSteps && rt < min(tile_toks, sp.ntok)) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  static_cast<const __nv_bfloat16*>(a.q) +
                  (static_cast<long long>(it.row0 + sp.tok0 + rt) * a.num_q_heads + it.head * a.group + r -
                   rt * a.group) * D);
              next[u][0] = src[2 * piece];
              next[u][1] = src[2 * piece + 1];
            }
          }
        };
        uint32_t own = 0;  // largest magnitude of this thread's row, as bf16 bits
        load(0);
#pragma unroll 1
        for (int step = 0; step < kSteps; step += kAhead) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u) in[u][0] = next[u][0], in[u][1] = next[u][1];
          load(step + kAhead);
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const uint32_t x[8] = {in[u][0].x, in[u][0].y, in[u][0].z, in[u][0].w,
                                   in[u][1].x, in[u][1].y, in[u][1].z, in[u][1].w};
            uint32_t most = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) most = __vmaxu2(most, x[k] & 0x7fff7fffu);
            most = max(most & 0xffffu, most >> 16);
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
            const uint32_t given = __shfl_sync(0xffffffffu, most, lane % kRows * kLanes);
            if (lane / kRows == step + u) own = given;
            // the largest magnitude goes to [2^7, 2^8); rows below 2^-100 count as zero
            const int e = min(max(static_cast<int>(most >> 7) - 127, -100), 127);
            const float up = pow2f(7 - max(e, -119));
            const float mul = ks < 0.f ? -up : up;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h0, h1, l0, l1;
              e4m3x2_terms(bf16_lo_f(x[2 * k]) * mul, bf16_hi_f(x[2 * k]) * mul, h0, l0);
              e4m3x2_terms(bf16_lo_f(x[2 * k + 1]) * mul, bf16_hi_f(x[2 * k + 1]) * mul, h1, l1);
              hi[k] = h0 | (h1 << 16);
              lo[k] = l0 | (l1 << 16);
            }
            const int r = (row & ~31) + (step + u) * kRows + lane / kLanes;
            const int swz = ROW == 128 ? (ch ^ (r & 7)) : (ch ^ ((r >> 1) & 3));
            unsigned char* dst = s.q[t] + blk * C::kKBlockBytes + r * ROW + swz * 16;
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + 128 * D) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        const int e = min(max(static_cast<int>(own >> 7) - 127, -100), 127);
        scale = a.scale_log2 * fabsf(ks) * pow2f(max(e, -119) - 7);
        if (scale == 0.f) scale = 1e-37f;
        if (own >= 0x7f80u) scale = CUDART_NAN_F;  // a query that is not finite, which codes cannot hold
        fence_proxy_async_shared();
        mbar_arrive(&s.q_full[t]);
      }
    }
    for (int j = sp.jb; j < sp.je; ++j, ++blocks) {
      const int buf = NT == 2 ? t : static_cast<int>(blocks & 1u);
      const uint32_t tS = tmem + lane_base + buf * 128;
      if (!role.wait(&s.s_full[buf], NT == 2 ? blocks : blocks >> 1, kStatusSync)) break;
      tc_fence_after();
      const int k0 = it.lo + j * kPfBlock;
      // rows see keys (pos - window, pos]; block columns [from, upto]
      if (k0 + kPfBlock > it.pos0 + sp.tok0 + 1 ||
          (a.window > 0 && k0 < it.pos0 + sp.tok0 + sp.ntok - a.window)) {
        const int upto = pos - k0, from = a.window > 0 ? pos - a.window + 1 - k0 : 0;
#pragma unroll 1
        for (int q = 0; q < kPfBlock; q += 32) {
          if (__all_sync(0xffffffffu, upto - q >= 31 && from - q <= 0)) continue;  // all seen
          const int last = upto - q, first = from - q;
          const uint32_t seen = (last < 0 ? 0u : last >= 31 ? ~0u : (2u << last) - 1u) &
                                (first <= 0 ? ~0u : first > 31 ? 0u : ~0u << first);
          float x[32];
          tmem_ld32(tS + q, reinterpret_cast<uint32_t*>(x));
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(seen & (1u << c))) x[c] = -CUDART_INF_F;
          tmem_st32(tS + q, reinterpret_cast<const uint32_t*>(x));
        }
        tmem_wait_st();
      }
      // The second half of the scores is read twice, for the maximum and for the
      // weights: a row of 128 has no room beside them, and the loop over halves
      // keeps the code of a block short enough for the instruction caches.
      float most = -CUDART_INF_F;
      float x[64];  // the first half's stay
      {
        float z[64];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(tS + 32 * c, reinterpret_cast<uint32_t*>(x) + 32 * c);
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(tS + 64 + 32 * c, reinterpret_cast<uint32_t*>(z) + 32 * c);
        tmem_wait_ld();
        float top[4] = {x[0], x[1], x[2], x[3]};  // independent chains
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = max3(top[e], x[c + 2 * e], x[c + 2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = max3(top[e], x[60 + e], z[e]);
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = max3(top[e], z[c + 2 * e], z[c + 2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], z[60 + e]);
        most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
      }
      if (__any_sync(0xffffffffu, most > m + kLazy)) {
        const float mn = fmaxf(m, most);
        const float keep = m == -CUDART_INF_F ? 0.f : ex2(m - mn);
        if (j > sp.jb) {
          // The accumulator is still: two tiles, S came after this tile's
          // earlier products on the same thread; one, they are waited for.
          if constexpr (NT == 1) {
            if (!role.wait(&s.s_free[buf ^ 1], (blocks - 1) >> 1, kStatusSync)) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < DV; c += 32) {
            float o[32];
            tmem_ld32(tO + c, reinterpret_cast<uint32_t*>(o));
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= keep;
            tmem_st32(tO + c, reinterpret_cast<const uint32_t*>(o));
          }
        }
        l *= keep;
        m = mn;
      }
      const float mb = m == -CUDART_INF_F ? 0.f : -m;
      const float2 scale2 = make_float2(scale, scale), mb2 = make_float2(mb, mb);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        // weights of keys 64 h .. 64 h + 63; the issuer may start on the first half at once
        if (h == 1) {
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld32(tS + 64 + 32 * c, reinterpret_cast<uint32_t*>(x) + 32 * c);
          tmem_wait_ld();
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float2 w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c = 32 * q + 4 * e + 2 * i;
              w[i] = fma2(make_float2(x[c], x[c + 1]), scale2, mb2);
              w[i].x = ex2(w[i].x);
              w[i].y = ex2(w[i].y);
              sum[i] = add2(sum[i], w[i]);
            }
            if constexpr (FP8) {
              p[2 * e] = pack_f16(w[0].x, w[0].y);
              p[2 * e + 1] = pack_f16(w[1].x, w[1].y);
            } else {
              p[2 * e] = pack_bf16(w[0].x, w[0].y);
              p[2 * e + 1] = pack_bf16(w[1].x, w[1].y);
            }
          }
          tmem_st16(tS + 32 * h + 16 * q, p);  // (P lies over scores that have been read)
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_ready[h][buf]);
      }
      const float2 both = add2(sum[0], sum[1]);
      l += both.x + both.y;
    }
    if (!role.live) break;

    if (!role.wait(&s.l_free[t], items ^ 1u, kStatusSync)) break;
    s.ml[t][row] = make_float2(m, l);
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.l_full[t]);
    role.item_done(items);
  }
}

// --------------------------------------------------------------------- epilogue
// A warpgroup of its own divides O by the rows' sums and stores it (or, of a
// split item, the sums as they are), tile by tile, while the softmax threads
// are at the next item.
template <typename C>
__device__ __forceinline__ void tc_epilogue(const PrefillArgs& a, TcSmem<C>& s, uint32_t tmem, int row) {
  constexpr int D = C::kD, NT = C::kNT, DV = C::kDV;
  constexpr bool FP8 = C::kFp8;
  const int lane = row & 31;
  const int tile_toks = a.tile_tokens / C::kNT;
  const int tok = pf_token_of(a, row), g = row - tok * a.group;
  const uint32_t lane_base = static_cast<uint32_t>(row >> 5) << 21;
  TcRole<C> role{a, s, lane};
  PfItem it{};
  uint32_t items = 0, no = 0;  // no: parity of a tile's accumulators in bit t
  for (; role.item(items, it); ++items) {
#pragma unroll 1
    for (int t = 0; t < NT; ++t) {
      const uint32_t tO = tmem + lane_base + C::kTmemO + t * DV;
      const TileSpan sp = role.span(items, t);
      const bool valid = tok < tile_toks && tok < sp.ntok;
      const int pos = it.pos0 + sp.tok0 + min(tok, max(sp.ntok, 1) - 1);
      if (!role.wait(&s.l_full[t], items, kStatusSync)) break;
      const float m = s.ml[t][row].x, l = s.ml[t][row].y;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.l_free[t]);
      const bool any = sp.je > sp.jb;  // O holds sums of this tile
      int flags = 0;
      if (any) {
        if (!role.wait(&s.o_full[t], no >> t, kStatusSync)) break;
        no ^= 1u << t;
        tc_fence_after();
        flags = s.flags[t];
        if (flags & kItemFix) add_taken_values<FP8>(a, it, D, pos, DV, tO);
      }
      const bool split = it.kb0 > 0 || it.pieces > 0;
      if (it.pieces > 0 && t == 0 && row == 0)
        a.splits[blockIdx.x] = PrefillSplit{it.pieces, it.row0, it.ntok, it.head, it.part};
      const long long rec = (2ll * blockIdx.x + (it.kb0 > 0 ? 1 : 0)) * (NT * 128) + t * 128 + row;
      const bool bad = it.bad || (flags & kItemBad);
      const float vs = FP8 ? a.v_scale[it.head] : 1.f;
      const float mul = split ? vs : bad ? CUDART_NAN_F : vs / l;
      if (split && valid) a.ml[rec] = make_float2(bad ? CUDART_NAN_F : m, l);
      // Rows go out four lanes to a row: a lane's 16-byte pieces of its own row
      // are exchanged within groups of four, so that a store touches eight rows
      // of 64 bytes and not 32 of 16 (which took 7000 cycles an item).
      const bool put = valid && !(split && l == 0.f);  // (the combine reads no sums of a row without weight)
      char* const to = split ? reinterpret_cast<char*>(a.part) : static_cast<char*>(a.out);
      const long long mine = split ? rec * DV * 4
                                   : ((static_cast<long long>(it.row0 + sp.tok0 + tok) * a.num_q_heads +
                                       it.head * a.group + g) * D + it.part * DV) * 2;
      long long at[4];  // byte offsets of the group's rows; -1: not written
#pragma unroll
      for (int r = 0; r < 4; ++r) at[r] = __shfl_sync(0xffffffffu, put ? mine : -1ll, (lane & ~3) + r);
      // 64 bytes of a row at a time: 32 bf16 or 16 fp32 columns, from 32 columns read
#pragma unroll 1
      for (int c = 0; c < DV; c += split ? 16 : 32) {
        float o[32];
        uint4 x[4];
        if (any) {
          tmem_ld32(tO + (c & ~31), reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= mul;
        if (split) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = c & 16 ? o[16 + 4 * e + i] : o[4 * e + i];
            x[e] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                              pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
        }
        transpose4(x, lane);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (at[r] >= 0) *reinterpret_cast<uint4*>(to + at[r] + c * (split ? 4 : 2) + 16 * (lane & 3)) = x[r];
        __syncwarp();  // the next load of tensor memory is the whole warp's
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_free[t]);
      }
    }
    if (!role.live) break;
    role.item_done(items);
  }
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ PrefillArgs a) {
  constexpr int NT = C::kNT;
  extern __shared__ __align__(1024) unsigned char raw[];  // whole swizzle atoms
  TcSmem<C>& s = *reinterpret_cast<TcSmem<C>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kEpilogue = NT * 4, kLoader = kEpilogue + 4, kWiden = kLoader + 4, kIssuer = kLoader + 1, kPrep = kLoader + 3;

  if (tid == 0) {
    a.splits[blockIdx.x].pieces = 0;
    s.abort_at[0] = 0;
    for (int i = 0; i < C::kStagesK; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], NT);      // the issuers of Q K^T
    }
    for (int i = 0; i < C::kStagesV; ++i) {
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_empty[i], C::kFp8 ? 4 : NT + 1);  // widening; or the issuers of P V, and preparation
      mbar_init(&s.v_ready[i], 1);
    }
    if constexpr (C::kFp8)
      for (int i = 0; i < C::kStagesP; ++i) {
        mbar_init(&s.w_full[i], 4);
        mbar_init(&s.w_empty[i], NT);
      }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&s.q_full[i], C::kFp8 ? 128 : 1);
      mbar_init(&s.q_empty[i], 1);
      mbar_init(&s.o_full[i], 2);        // the commit, and the issuer's flags
      mbar_init(&s.o_free[i], 4);        // warps of a warpgroup
      mbar_init(&s.l_full[i], 4);
      mbar_init(&s.l_free[i], 4);
    }
    for (int i = 0; i < C::kNumS; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_free[i], 1);
      mbar_init(&s.p_ready[0][i], 4);
      mbar_init(&s.p_ready[1][i], 4);
      mbar_init(&s.turn[i], 1);
      mbar_init(&s.drain[i], 1);
    }
    for (int i = 0; i < C::kItems; ++i) {
      mbar_init(&s.item_full[i], 1);
      mbar_init(&s.item_empty[i], (C::kFp8 ? 10 : 7) + 4 * NT);  // every warp but the loader
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssuer) tmem_alloc(&s.tmem, 512);
  if (warp == kLoader && lane == 0) {
    prefetch_tensormap(&tq);
    prefetch_tensormap(&tk);
    prefetch_tensormap(&tv);
  }
  tc_fence_before();
  PfWalk w;
  if (warp == kLoader) pf_begin(a, lane, w);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  // A softmax thread holds a row of 128 scores; with two tiles registers move
  // to it from the other warpgroups (512 x 128 = 128 x (96 + 96) + 256 x 160;
  // with widening 640 x 96 >= 128 x 3 x 72 + 256 x 128).
  constexpr bool kMove = NT == 2;
  constexpr int kFew = C::kFp8 ? 72 : 96, kMany = C::kFp8 ? 128 : 160;
  if (warp >= kWiden) {
    if constexpr (kMove) regs_dec<kFew>();
    if constexpr (C::kFp8) tc_widen<C>(a, s, tid - kWiden * 32);
  } else if (warp >= kLoader) {
    if constexpr (kMove) regs_dec<kFew>();
    if (warp == kLoader) {
      tc_loader<C>(tq, tk, tv, a, s, w, lane);
    } else if (warp == kPrep) {
      if constexpr (!C::kFp8) tc_prepare<C>(a, s, lane);
    } else {
      tc_issuer<C>(a, s, tmem, warp - kIssuer, lane);
    }
  } else if (warp >= kEpilogue) {
    if constexpr (kMove) regs_dec<kFew>();
    tc_epilogue<C>(a, s, tmem, tid - kEpilogue * 32);
  } else {
    if constexpr (kMove) regs_inc<kMany>();
    tc_softmax<C>(a, s, tmem, tid);
  }
  // every role is done with tensor memory
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && s.abort_at[0]) {
    atomicOr(a.status, s.abort_at[0] & 0xffu);
    if (atomicCAS(a.status + 1, 0u, 1u + blockIdx.x) == 0u) {  // first in the grid: where
      a.status[2] = s.abort_at[0];
      a.status[3] = s.abort_at[1];
      a.status[4] = s.abort_at[2];
    }
  }
}

template <typename C>
struct TcVariant {
  static constexpr size_t smem = sizeof(TcSmem<C>);
  static_assert(smem <= 232448, "does not fit in shared memory");
  static cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefillArgs& a,
                            int grid, cudaStream_t stream) {
    prefill_tc_kernel<C><<<grid, C::kThreads, smem, stream>>>(tq, tk, tv, a);
    return cudaGetLastError();
  }
  static PrefillVariant info() {
    return PrefillVariant{C::kThreads, C::kNT * 128, 128, C::kDV, 1, C::kStagesK + C::kStagesV, kItemWeight<C::kFp8>, smem,
                          reinterpret_cast<const void*>(&prefill_tc_kernel<C>), &launch};
  }
};

}  // namespace vt
