// Ragged prefill over the paged cache on the 5th-generation tensor cores.
//
// Per item (prefill_plan.cuh): NT tiles of 128 query rows (tokens x the query
// heads of one kv head), against 128 keys (four pages) at a time:
//   S = Q K^T   tcgen05.mma, Q and K in shared memory, S in tensor memory;
//   P = 2^(scale S - m), rows masked and summed in registers, one row to a
//       thread, rounded to bf16 and written over S in tensor memory;
//   O += P V    tcgen05.mma, P from tensor memory, V as it lies in its pages
//       (token-major, i.e. the N-major right operand), O in tensor memory.
// A row's reference maximum m moves only when a score passes it by more than
// 2^8 (weights then stay below 2^8, sums below 2^8 n, and the quotient is
// the same), so O is rescaled a few times an item and not once a block.
//
// Roles, one warp each: loader (Q tiles, and K and V pages through the block
// table, TMA into a ring of stages), MMA issuer, V preparation (below); and
// one warpgroup of softmax threads a tile.  With two tiles (head_dim 64 and
// 128) the issuer alternates them, P V and the next Q K^T of one tile running
// while the other's softmax does; with one (head_dim 256 and 512, whose O
// takes half of tensor memory) S is double-buffered and the next block's
// Q K^T runs during the softmax.
//
// V preparation: in blocks that some row of the item may see only in part,
// slots outside the item's keys are zeroed (0 * NaN is NaN, whatever P is),
// and values that are not finite in the keys only some rows see are zeroed
// too and given back to the rows that do attend to them at the end.
#pragma once

#include <math_constants.h>

#include "decode_kernel.cuh"
#include "prefill_variants.cuh"
#include "tcgen05.cuh"

namespace vt {

template <bool FP8, int D, int NT, int DV, int CW, int NS>
struct TcConfig {
  static constexpr bool kFp8 = FP8;                    // E4M3 codes in the cache, else bf16
  static constexpr int kD = D, kNT = NT, kDV = DV;
  static constexpr int kElem = FP8 ? 1 : 2;            // bytes of a cached element
  // One TMA box and one swizzled block are kCols columns wide: 128-byte rows,
  // or 64-byte ones for the 64 codes of an FP8 head_dim 64.
  static constexpr int kCols = FP8 ? (D < 128 ? D : 128) : 64;
  static constexpr int kRow = kCols * kElem;
  static constexpr uint32_t kSwizzle = kRow == 128 ? 2 : 4;
  static constexpr int kKStep = 32 / kElem;            // k extent of an MMA
  static constexpr int kCW = CW;                       // columns of a stage
  static constexpr int kStages = NS;
  static constexpr int kKChunks = D / CW, kVChunks = DV / CW;
  static constexpr int kBlocks = CW / kCols;           // swizzled blocks of a stage
  static constexpr int kBlockBytes = kPfBlock * kRow;
  static constexpr int kStageBytes = kBlocks * kBlockBytes;
  static constexpr int kQBytes = 128 * D * 2;          // FP8: two E4M3 terms of each element, high terms first
  static constexpr int kThreads = NT * 128 + 128;
  static constexpr int kTmemO = 256;                   // S of tile (or buffer) i at 128 i
  static constexpr int kNumS = 2;                      // tiles, or buffers of one tile
};

template <typename C>
struct TcSmem {
  alignas(1024) unsigned char q[C::kNT][C::kQBytes];
  alignas(1024) unsigned char ring[C::kStages][C::kStageBytes];
  alignas(8) unsigned long long full[C::kStages];
  unsigned long long empty[C::kStages];
  unsigned long long vready[C::kStages];
  unsigned long long q_full[C::kNT], q_empty[C::kNT];
  unsigned long long s_full[C::kNumS], p_ready[C::kNumS];
  unsigned long long o_full[C::kNT], o_free[C::kNT];
  unsigned long long prep_go;
  unsigned long long pv_done, drain;
  long long scan[C::kThreads / 32 + 4];
  uint32_t tmem;
  volatile int stage_bad[C::kStages];  // a page id of this stage was out of range
  volatile int stage_fix[C::kStages];  // V preparation took out a value that is not finite
  volatile int flags[C::kNT];          // of the item whose O is full: 1 bad, 2 fix
  volatile int abort_flag;
};

// Weights are 2^(score - m + kWeightExp) with m at most kLazy below the largest
// score: at most 2^8 in bf16, 2^8.5 as E4M3 terms (largest 448), whose
// absolute step of 2^-10 is then 2^-17 of a row's largest weight.
template <bool FP8>
constexpr float lazy_bound() { return FP8 ? 1.5f : 8.f; }
template <bool FP8>
constexpr float weight_exp() { return FP8 ? 7.f : 0.f; }

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

// Position in the ring of stages.
template <int NS>
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == NS) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Adds the values that preparation took out to the output columns [c0, c0 + 32)
// of a row at `pos`: they are not finite, so neither is the result.
template <bool FP8>
__device__ __forceinline__ void add_taken_values(const PrefillArgs& a, const PfItem& it, int head_dim, int pos, int c0,
                                                 float (&o)[32]) {
  const int first = max(it.lo_exact, it.lo + it.kb0 * kPfBlock);
  const int last = min(it.hi, it.lo + it.kb1 * kPfBlock);
#pragma unroll 1
  for (int t = first; t < last; ++t) {
    const bool all = t <= it.pos0 && (a.window == 0 || t >= it.hi - a.window);
    if (all) continue;  // seen by every row: was left in place
    if (t > pos || (a.window > 0 && t <= pos - a.window)) continue;
    const int page = a.block_tables[static_cast<long long>(it.b) * a.max_blocks + t / kPfPage];
    if (page < 0 || page >= a.num_blocks) continue;
    const long long at = ((static_cast<long long>(page) * kPfPage + t % kPfPage) * a.num_kv_heads + it.head) *
                             head_dim + c0;
    if constexpr (FP8) {
      const uint8_t* v = static_cast<const uint8_t*>(a.v_cache) + at;
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if ((v[c] & 0x7f) == 0x7f) o[c] = CUDART_NAN_F;
    } else {
      const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_cache) + at;
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(v + c);
        if ((w & 0x7f80u) == 0x7f80u) o[c] += bf16_lo_f(w);
        if ((w & 0x7f800000u) == 0x7f800000u) o[c + 1] += bf16_hi_f(w);
      }
    }
  }
}

// All ones in the place of a word's elements that are not finite.
template <bool FP8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  uint32_t m = 0;
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      if (((w >> i) & 0x7fu) == 0x7fu) m |= 0xffu << i;
    return m;
  }
  if ((w & 0x7f80u) == 0x7f80u) m |= 0xffffu;
  if ((w & 0x7f800000u) == 0x7f800000u) m |= 0xffff0000u;
  return m;
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

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ PrefillArgs a) {
  constexpr int D = C::kD, NT = C::kNT, DV = C::kDV, CW = C::kCW, NS = C::kStages;
  constexpr int NKC = C::kKChunks, NVC = C::kVChunks;
  constexpr bool FP8 = C::kFp8;
  constexpr int ROW = C::kRow, KS = C::kKStep;
  constexpr float kLazy = lazy_bound<FP8>(), kWeightExp = weight_exp<FP8>();
  extern __shared__ unsigned char raw[];
  TcSmem<C>& s = *reinterpret_cast<TcSmem<C>*>(
      raw + ((1024 - (static_cast<uint32_t>(__cvta_generic_to_shared(raw)) & 1023)) & 1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kLoader = NT * 4, kIssuer = kLoader + 1, kPrep = kLoader + 2;
  const int tile_toks = 128 / a.group;

  if (tid == 0) {
    a.splits[blockIdx.x].pieces = 0;
    s.abort_flag = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
      mbar_init(&s.vready[i], 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&s.q_full[i], FP8 ? 128 : 1);
      mbar_init(&s.q_empty[i], 1);
      mbar_init(&s.o_full[i], 2);  // the commit, and the issuer's flags
      mbar_init(&s.o_free[i], 128);
    }
    for (int i = 0; i < C::kNumS; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_ready[i], 128);
    }
    mbar_init(&s.prep_go, 1);
    mbar_init(&s.pv_done, 1);
    mbar_init(&s.drain, 1);
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
  pf_begin(a, s.scan, w);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  PfItem it{};
  // A softmax thread holds a row of 128 scores: with two softmax warpgroups
  // the 168 registers a thread is launched with are moved to them (128 x 88 +
  // 256 x 208 = 384 x 168).
  if (warp >= kLoader) {
    if constexpr (NT == 2) regs_dec<88>();
    if (warp == kLoader) {
      // ---------------------------------------------------------------- loader
      Ring<NS> r;
      uint32_t nq[NT] = {};
      long long issued = 0;
      int blocks = 0;
      bool live = true;
      int ids = 0, ids_at = -1;  // 32 table entries, one a lane, from page index ids_at
      auto load = [&](const CUtensorMap* map, int chunk0, int j, int item_b, int head, int chunks) {
        const int k0 = it.lo + j * kPfBlock;
        const int pages = min(kPfBlock, it.hi - k0 + kPfPage - 1) / kPfPage;  // those that hold keys of the item
        const int p0 = k0 / kPfPage;
        if (ids_at < 0 || p0 < ids_at || p0 + 4 > ids_at + 32) {
          ids_at = p0;
          const int at = p0 + lane;
          ids = at < a.max_blocks ? a.block_tables[static_cast<long long>(item_b) * a.max_blocks + at] : 0;
        }
        int page = __shfl_sync(0xffffffffu, ids, p0 - ids_at + (lane & 3));
        const bool use = (lane & 3) < pages && lane < 4 * C::kBlocks;
        const bool bad = use && (page < 0 || page >= a.num_blocks);
        const bool any_bad = __any_sync(0xffffffffu, bad);
        if (bad) page = 0;
        for (int c = 0; c < chunks && live; ++c) {
          live = wait_phase(&s.empty[r.stage], r.phase ^ 1u, &s.abort_flag, a.status, kStatusEmpty, a.wait_limit);
          live = __all_sync(0xffffffffu, live);
          if (!live) break;
          if (lane == 0) {
            s.stage_bad[r.stage] = any_bad;
            mbar_arrive_expect_tx(&s.full[r.stage], pages * C::kBlocks * kPfPage * ROW);
          }
          __syncwarp();
          if (use)
            tma_load_4d(s.ring[r.stage] + (lane >> 2) * C::kBlockBytes + (lane & 3) * kPfPage * ROW, map, 0,
                        page * kPfPage, chunk0 + c * C::kBlocks + (lane >> 2), head, &s.full[r.stage]);
          ++issued;
          r.next();
        }
      };
      while (live && w.next(a, it)) {
        if (it.kb1 <= it.kb0) continue;
        ids_at = -1;
        for (int t = 0; t < NT && live && !FP8; ++t) {
          const TileSpan sp = tile_span(a, it, t, tile_toks);
          if (sp.je <= sp.jb) continue;
          live = wait_phase(&s.q_empty[t], (nq[t] & 1u) ^ 1u, &s.abort_flag, a.status, kStatusEmpty, a.wait_limit);
          live = __all_sync(0xffffffffu, live);
          if (!live) break;
          ++nq[t];
          if (lane == 0) {
            mbar_arrive_expect_tx(&s.q_full[t], tile_toks * a.group * D * 2);
            for (int c = 0; c < D / 64; ++c)
              asm volatile(
                  "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
                  " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(s.q[t] + c * 128 * 128)),
                  "l"(reinterpret_cast<uint64_t>(&tq)), "r"(0), "r"(0), "r"(it.row0 + sp.tok0), "r"(c), "r"(it.head),
                  "r"(smem_addr(&s.q_full[t]))
                  : "memory");
          }
        }
        const int vc0 = it.part * (DV / C::kCols);
        for (int j = it.kb0; j < it.kb1 && live; ++j) {
          if (static_cast<int>(blockIdx.x) == a.withhold_cta && blocks >= a.withhold_block) {
            live = false;  // test hook: the issuer's wait for this block runs out
            break;
          }
          ++blocks;
          if constexpr (NT == 2) {
            load(&tk, 0, j, it.b, it.head, NKC);
            if (live) load(&tv, vc0, j, it.b, it.head, NVC);
          } else {
            if (j == it.kb0) load(&tk, 0, j, it.b, it.head, NKC);
            if (live && j + 1 < it.kb1) load(&tk, 0, j + 1, it.b, it.head, NKC);
            if (live) load(&tv, vc0, j, it.b, it.head, NVC);
          }
        }
      }
      if (!live) {
        // let this CTA's copies land before it exits
        volatile int never = 0;
        for (long long k = 1; k <= (issued < NS ? issued : NS); ++k) {
          const long long n = issued - k;
          if (!wait_phase(&s.full[n % NS], static_cast<uint32_t>((n / NS) & 1), &never, a.status, kStatusDrain,
                          kDrainLimitCycles))
            break;
        }
        for (int t = 0; t < NT; ++t)
          if (nq[t])
            wait_phase(&s.q_full[t], (nq[t] - 1) & 1u, &never, a.status, kStatusDrain, kDrainLimitCycles);
      }
    } else if (warp == kIssuer) {
      // ---------------------------------------------------------------- MMA issuer
      Ring<NS> r;
      uint32_t nq[NT] = {}, np[C::kNumS] = {}, no[NT] = {};
      uint32_t vphase = 0;  // one bit a stage
      bool live = true;
      const uint32_t idesc_qk = FP8 ? umma_idesc_e4m3(kPfBlock, false)
                                    : umma_idesc_f16(true, kPfBlock, false) | (a.neg_scale ? kUmmaNegateA : 0u);
      const uint32_t idesc_pv = FP8 ? umma_idesc_e4m3(CW, true) : umma_idesc_f16(true, CW, true);
      auto wait = [&](unsigned long long* bar, uint32_t parity, unsigned code) {
        if (live) live = wait_phase(bar, parity, &s.abort_flag, a.status, code, a.wait_limit);
        return live;
      };
      // S(buf) (+)= Q_t chunk c x K chunk in the stage
      auto qk = [&](int t, int buf, int c, int stage) {
        if (lane != 0) return;
        const uint32_t qa = smem_addr(s.q[t]), kb = smem_addr(s.ring[stage]);
        constexpr int kSteps = ROW / 32;  // MMAs of a block's columns
#pragma unroll
        for (int term = 0; term < (FP8 ? 2 : 1); ++term)
#pragma unroll
          for (int k = 0; k < C::kBlocks * kSteps; ++k) {
            const uint32_t at = (k / kSteps) * C::kBlockBytes + (k % kSteps) * 32;
            umma_ss<FP8>(tmem + buf * 128,
                         umma_desc(qa + term * (128 * D) + c * C::kStageBytes + at, 16, 8 * ROW, C::kSwizzle),
                         umma_desc(kb + at, 16, 8 * ROW, C::kSwizzle), idesc_qk, c > 0 || term > 0 || k > 0);
          }
      };
      // O_t chunk c (+)= P(buf) x V chunk in the stage, over ksteps of KS keys
      auto pv = [&](int t, int buf, int c, int stage, int ksteps, bool acc) {
        if (lane != 0) return;
        const uint32_t vb = smem_addr(s.ring[stage]);
        const uint32_t d = tmem + C::kTmemO + t * DV + c * CW, p = tmem + buf * 128;
        for (int k = 0; k < ksteps; ++k) {
          const uint64_t v = umma_desc(vb + k * KS * ROW, C::kBlockBytes, 8 * ROW, C::kSwizzle);
          umma_ts<FP8>(d, p + k * 8, v, idesc_pv, acc || k > 0);
          if constexpr (FP8) umma_ts<FP8>(d, p + 32 + k * 8, v, idesc_pv, true);  // P's low terms
        }
      };
      while (live && w.next(a, it)) {
        if (it.kb1 <= it.kb0) continue;
        TileSpan sp[NT];
        int flags = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          sp[t] = tile_span(a, it, t, tile_toks);
          if (sp[t].je > sp[t].jb) {
            if (!wait(&s.q_full[t], nq[t] & 1u, kStatusFull)) break;
            ++nq[t];
          }
        }
        auto finish = [&](int t) {  // after the tile's last P V
          if (lane == 0) {
            s.flags[t] = flags;
            umma_commit(&s.o_full[t]);
            mbar_arrive(&s.o_full[t]);
          }
          ++no[t];
        };
        auto prep_wait = [&](int stage, int j) {
          if (!needs_prep(a, it, j)) return;
          wait(&s.vready[stage], (vphase >> stage) & 1u, kStatusSync);
          vphase ^= 1u << stage;
          if (live && s.stage_fix[stage]) flags |= kItemFix;
        };
        // Preparation of block j may start: it must not look at a stage's barrier
        // while an earlier use of the stage is outstanding (a wait tells phases
        // apart by parity only).
        auto prep_go = [&](int j) {
          if (!needs_prep(a, it, j)) return;
          if (lane == 0) mbar_arrive(&s.prep_go);
        };
        auto keys_to = [&](int t, int j) {  // k-steps of block j that tile t's rows need
          const int n = it.pos0 + sp[t].tok0 + sp[t].ntok - (it.lo + j * kPfBlock);
          return (min(n, kPfBlock) + KS - 1) / KS;
        };
        if constexpr (NT == 2) {
          Ring<NS> k = r;  // K of block j + 1
          auto first_qk = [&](int t, int j) {
            if (j < sp[t].jb || j >= sp[t].je) return;
            qk(t, t, 0, k.stage);
            if (lane == 0) {
              umma_commit(&s.s_full[t]);
              if (j == sp[t].je - 1) umma_commit(&s.q_empty[t]);
            }
          };
          if (!wait(&s.full[k.stage], k.phase, kStatusFull)) break;
          tc_fence_after();
          if (s.stage_bad[k.stage]) flags |= kItemBad;
          prep_go(it.kb0);
          for (int t = 0; t < NT; ++t) first_qk(t, it.kb0);
          if (lane == 0) umma_commit(&s.empty[k.stage]);
          k.next();
          for (int j = it.kb0; j < it.kb1 && live; ++j) {
            const Ring<NS> v = k;  // the ring holds K0 V0 K1 V1 ...
            k.next();
            bool have_v = false, have_k = false;
            for (int t = 0; t < NT && live; ++t) {
              if (j >= sp[t].jb && j < sp[t].je) {
                if (!wait(&s.p_ready[t], np[t] & 1u, kStatusSync)) break;
                ++np[t];
                if (j == sp[t].jb && !wait(&s.o_free[t], (no[t] & 1u) ^ 1u, kStatusSync)) break;
                if (!have_v) {
                  if (!wait(&s.full[v.stage], v.phase, kStatusFull)) break;
                  prep_wait(v.stage, j);
                  if (!live) break;
                  have_v = true;
                }
                tc_fence_after();
                pv(t, t, 0, v.stage, keys_to(t, j), j > sp[t].jb);
                if (j == sp[t].je - 1) finish(t);
              }
              if (j + 1 < it.kb1 && j + 1 >= sp[t].jb && j + 1 < sp[t].je) {
                if (!have_k) {
                  if (!wait(&s.full[k.stage], k.phase, kStatusFull)) break;
                  if (s.stage_bad[k.stage]) flags |= kItemBad;
                  prep_go(j + 1);
                  have_k = true;
                }
                tc_fence_after();
                first_qk(t, j + 1);
              }
            }
            if (!live) break;
            if (lane == 0) umma_commit(&s.empty[v.stage]);
            if (j + 1 < it.kb1) {
              if (lane == 0) umma_commit(&s.empty[k.stage]);
              k.next();
            }
          }
          r = k;
        } else {
          auto all_qk = [&](int j) {
            const int buf = (np[0] + np[1] + (j > it.kb0 ? 1 : 0)) & 1;  // blocks alternate buffers
            for (int c = 0; c < NKC && live; ++c) {
              if (!wait(&s.full[r.stage], r.phase, kStatusFull)) break;
              tc_fence_after();
              if (s.stage_bad[r.stage]) flags |= kItemBad;
              qk(0, buf, c, r.stage);
              if (lane == 0) umma_commit(&s.empty[r.stage]);
              r.next();
            }
            if (live && lane == 0) {
              umma_commit(&s.s_full[buf]);
              if (j == it.kb1 - 1) umma_commit(&s.q_empty[0]);
            }
          };
          all_qk(it.kb0);
          for (int j = it.kb0; j < it.kb1 && live; ++j) {
            if (j + 1 < it.kb1) all_qk(j + 1);
            if (live) prep_go(j);  // the ring holds K0 K1 V0 K2 V1 ...: whatever used V's stages before is done
            const int buf = (np[0] + np[1]) & 1;
            if (!live || !wait(&s.p_ready[buf], np[buf] & 1u, kStatusSync)) break;
            ++np[buf];
            if (j == it.kb0 && !wait(&s.o_free[0], (no[0] & 1u) ^ 1u, kStatusSync)) break;
            for (int c = 0; c < NVC; ++c) {
              if (!wait(&s.full[r.stage], r.phase, kStatusFull)) break;
              prep_wait(r.stage, j);
              if (!live) break;
              tc_fence_after();
              pv(0, buf, c, r.stage, keys_to(0, j), j > it.kb0);
              if (lane == 0) umma_commit(&s.empty[r.stage]);
              r.next();
            }
            if (!live) break;
            if (j == it.kb1 - 1) finish(0);
            if (lane == 0) umma_commit(&s.pv_done);
          }
        }
      }
      __syncwarp();
      // every MMA has to be done before tensor memory is given back
      if (lane == 0) umma_commit(&s.drain);
      volatile int never = 0;
      wait_phase(&s.drain, 0, &never, a.status, kStatusDrain, kDrainLimitCycles);
    } else if (warp == kPrep) {
      // ---------------------------------------------------------------- V preparation
      Ring<NS> r;
      bool live = true;
      uint32_t ngo = 0;
      while (live && w.next(a, it)) {
        if (it.kb1 <= it.kb0) continue;
        auto skip = [&](int n) {
          for (int i = 0; i < n; ++i) r.next();
        };
        if constexpr (NT == 1) skip(NKC);
        for (int j = it.kb0; j < it.kb1 && live; ++j) {
          if (NT == 2 || j + 1 < it.kb1) skip(NKC);
          if (!needs_prep(a, it, j)) {
            skip(NVC);
            continue;
          }
          live = wait_phase(&s.prep_go, ngo & 1u, &s.abort_flag, a.status, kStatusSync, a.wait_limit);
          live = __all_sync(0xffffffffu, live);
          if (!live) break;
          ++ngo;
          const int k0 = it.lo + j * kPfBlock;
          const int end = min(kPfBlock, (it.hi - k0 + KS - 1) / KS * KS);  // slots the products read
          for (int c = 0; c < NVC && live; ++c) {
            live = wait_phase(&s.full[r.stage], r.phase, &s.abort_flag, a.status, kStatusFull, a.wait_limit);
            live = __all_sync(0xffffffffu, live);
            if (!live) break;
            bool fix = false;
            constexpr int kPieces = ROW / 16;
            for (int i = lane; i < end * kPieces; i += 32) {  // a 16-byte piece of a slot's row
              const int slot = i / kPieces, t = k0 + slot;
              const bool none = t < it.lo_exact || t >= it.hi;
              const bool all = t <= it.pos0 && (a.window == 0 || t >= it.hi - a.window);
              if (all && !none) continue;
              for (int cb = 0; cb < C::kBlocks; ++cb) {
                uint4* p = reinterpret_cast<uint4*>(s.ring[r.stage] + cb * C::kBlockBytes + i * 16);
                if (none) {
                  *p = make_uint4(0, 0, 0, 0);
                } else {
                  uint4 x = *p;
                  const uint32_t m0 = not_finite<FP8>(x.x), m1 = not_finite<FP8>(x.y), m2 = not_finite<FP8>(x.z),
                                 m3 = not_finite<FP8>(x.w);
                  if (m0 | m1 | m2 | m3) {
                    fix = true;
                    x.x &= ~m0, x.y &= ~m1, x.z &= ~m2, x.w &= ~m3;
                    *p = x;
                  }
                }
              }
            }
            fix = __any_sync(0xffffffffu, fix);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              s.stage_fix[r.stage] = fix;
              mbar_arrive(&s.vready[r.stage]);
            }
            r.next();
          }
        }
      }
    }
  } else {
    if constexpr (NT == 2) regs_inc<208>();
    // ---------------------------------------------------------------- softmax: one row a thread
    const int t = NT == 2 ? warp >> 2 : 0;
    const int row = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, lane in bits 16..
    uint32_t ns[C::kNumS] = {}, no = 0;
    uint32_t blocks = 0;  // of NT == 1: buffers alternate
    bool live = true;
    while (live && w.next(a, it)) {
      const TileSpan sp = tile_span(a, it, t, tile_toks);
      const int tok = row / a.group, g = row - tok * a.group;
      const bool valid = tok < tile_toks && tok < sp.ntok;
      const int pos = it.pos0 + sp.tok0 + min(tok, max(sp.ntok, 1) - 1);
      float m = -CUDART_INF_F, l = 0.f;
      float scale = a.scale_log2;  // from a score in tensor memory to the log2 domain
      if constexpr (FP8) {
        // This row of Q as two E4M3 terms in the layout TMA gives K.  (The
        // previous item's last scores are here, so its Q is done with.)
        if (sp.je > sp.jb) {
          const float ks = a.k_scale[it.head] * (a.neg_scale ? -1.f : 1.f);
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(a.q) +
              (static_cast<long long>(it.row0 + sp.tok0 + tok) * a.num_q_heads + it.head * a.group + g) * D);
          uint32_t most = 0;  // largest magnitude, as bf16 bits
          if (valid) {
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {
              const uint4 x = src[i];
              most = __vmaxu2(most, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                             __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
            }
          }
          most = max(most & 0xffffu, most >> 16);
          // the largest magnitude goes to [2^7, 2^8); rows below 2^-100 count as zero
          const int e = min(max(static_cast<int>(most >> 7) - 127, -100), 127);
          const float up = pow2f(7 - max(e, -119));
          scale = a.scale_log2 * fabsf(ks) * pow2f(max(e, -119) - 7);
          if (scale == 0.f) scale = 1e-37f;
          const float mul = ks < 0.f ? -up : up;
#pragma unroll 2
          for (int i = 0; i < D / 16; ++i) {
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            if (valid) {
              x0 = src[2 * i];
              x1 = src[2 * i + 1];
            }
            const uint32_t in[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h0, h1, l0, l1;
              e4m3x2_terms(bf16_lo_f(in[2 * k]) * mul, bf16_hi_f(in[2 * k]) * mul, h0, l0);
              e4m3x2_terms(bf16_lo_f(in[2 * k + 1]) * mul, bf16_hi_f(in[2 * k + 1]) * mul, h1, l1);
              hi[k] = h0 | (h1 << 16);
              lo[k] = l0 | (l1 << 16);
            }
            const int blk = i / (ROW / 16), ch = i % (ROW / 16);
            const int swz = ROW == 128 ? (ch ^ (row & 7)) : (ch ^ ((row >> 1) & 3));
            unsigned char* dst = s.q[t] + blk * C::kBlockBytes + row * ROW + swz * 16;
            *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + 128 * D) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          fence_proxy_async_shared();
          mbar_arrive(&s.q_full[t]);
        }
      }
      for (int j = sp.jb; j < sp.je; ++j) {
        const int buf = NT == 2 ? t : static_cast<int>(blocks & 1u);
        const uint32_t tS = tmem + lane_base + buf * 128;
        live = wait_phase(&s.s_full[buf], ns[buf] & 1u, &s.abort_flag, a.status, kStatusSync, a.wait_limit);
        live = __all_sync(0xffffffffu, live);
        if (!live) break;
        ++ns[buf];
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, reinterpret_cast<uint32_t*>(x) + 32 * c);
        tmem_wait_ld();
        const int k0 = it.lo + j * kPfBlock;
        // rows see keys (pos - window, pos]; block columns [from, upto]
        const bool masked = k0 + kPfBlock > it.pos0 + sp.tok0 + 1 ||
                            (a.window > 0 && k0 < it.pos0 + sp.tok0 + sp.ntok - a.window);
        if (masked) {
          const int upto = pos - k0, from = a.window > 0 ? pos - a.window + 1 - k0 : 0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > upto || c < from) x[c] = -CUDART_INF_F;
        }
        float top0 = x[0], top1 = x[1];
#pragma unroll
        for (int c = 2; c < 128; c += 2) {
          top0 = fmaxf(top0, x[c]);
          top1 = fmaxf(top1, x[c + 1]);
        }
        const float top = fmaxf(top0, top1) * scale;
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          const float mn = fmaxf(m, top);
          const float keep = m == -CUDART_INF_F ? 0.f : ex2(m - mn);
          if (j > sp.jb) {
            // the accumulator is still: this tile's earlier products are done
            if constexpr (NT == 1) {
              live = wait_phase(&s.pv_done, (blocks & 1u) ^ 1u, &s.abort_flag, a.status, kStatusSync, a.wait_limit);
              live = __all_sync(0xffffffffu, live);
              if (!live) break;
              tc_fence_after();
            }
            const uint32_t tO = tmem + lane_base + C::kTmemO + t * DV;
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
        const float mb = (m == -CUDART_INF_F ? 0.f : m) - kWeightExp;
        float sum0 = 0.f, sum1 = 0.f;
        if constexpr (FP8) {
          uint32_t hi[32], lo[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = ex2(fmaf(x[4 * e], scale, -mb)), p1 = ex2(fmaf(x[4 * e + 1], scale, -mb));
            const float p2 = ex2(fmaf(x[4 * e + 2], scale, -mb)), p3 = ex2(fmaf(x[4 * e + 3], scale, -mb));
            sum0 += p0 + p2;
            sum1 += p1 + p3;
            uint32_t h0, h1, l0, l1;
            e4m3x2_terms(p0, p1, h0, l0);
            e4m3x2_terms(p2, p3, h1, l1);
            hi[e] = h0 | (h1 << 16);
            lo[e] = l0 | (l1 << 16);
          }
          tmem_st32(tS, hi);
          tmem_st32(tS + 32, lo);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float p0 = ex2(fmaf(x[64 * h + 2 * e], scale, -mb));
              const float p1 = ex2(fmaf(x[64 * h + 2 * e + 1], scale, -mb));
              sum0 += p0;
              sum1 += p1;
              p[e] = pack_bf16(p0, p1);
            }
            tmem_st32(tS + 32 * h, p);
          }
        }
        l += sum0 + sum1;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&s.p_ready[buf]);
        ++blocks;
      }
      if (!live) break;

      const bool any = sp.je > sp.jb;  // O holds sums of this tile
      int flags = 0;
      if (any) {
        live = wait_phase(&s.o_full[t], no & 1u, &s.abort_flag, a.status, kStatusSync, a.wait_limit);
        live = __all_sync(0xffffffffu, live);
        if (!live) break;
        ++no;
        tc_fence_after();
        flags = s.flags[t];
      }
      const bool split = it.kb0 > 0 || it.pieces > 0;
      if (it.pieces > 0 && tid == 0)
        a.splits[blockIdx.x] = PrefillSplit{it.pieces, it.row0, it.ntok, it.head, it.part};
      const long long rec = (2ll * blockIdx.x + (it.kb0 > 0 ? 1 : 0)) * (NT * 128) + t * 128 + row;
      const bool bad = it.bad || (flags & kItemBad);
      const float vs = FP8 ? a.v_scale[it.head] : 1.f;
      const float inv = bad ? CUDART_NAN_F : vs / l;
      const uint32_t tO = tmem + lane_base + C::kTmemO + t * DV;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                           (static_cast<long long>(it.row0 + sp.tok0 + tok) * a.num_q_heads + it.head * a.group + g) *
                               D + it.part * DV;
      if (split && valid) a.ml[rec] = make_float2(bad ? CUDART_NAN_F : m, l);
#pragma unroll 1
      for (int c = 0; c < DV; c += 32) {
        float o[32];
        if (any) {
          tmem_ld32(tO + c, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
          if (flags & kItemFix) {
            add_taken_values<FP8>(a, it, D, pos, it.part * DV + c, o);
            __syncwarp();
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (valid && split && l != 0.f) {  // (the combine reads no sums of a row without weight)
          float4* p = reinterpret_cast<float4*>(a.part + rec * DV + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = make_float4(o[4 * e] * vs, o[4 * e + 1] * vs, o[4 * e + 2] * vs, o[4 * e + 3] * vs);
        } else if (valid && !split) {
          uint4* p = reinterpret_cast<uint4*>(dst + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = make_uint4(pack_bf16(o[8 * e] * inv, o[8 * e + 1] * inv),
                              pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                              pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                              pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        }
        __syncwarp();  // the next load of tensor memory is the whole warp's
      }
      if (any) {
        tc_fence_before();
        mbar_arrive(&s.o_free[t]);
      }
    }
  }
  // every role is done with tensor memory
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename C>
struct TcVariant {
  static constexpr size_t smem = sizeof(TcSmem<C>) + 1024;
  static_assert(smem <= 232448, "does not fit in shared memory");
  static cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefillArgs& a,
                            int grid, cudaStream_t stream) {
    prefill_tc_kernel<C><<<grid, C::kThreads, smem, stream>>>(tq, tk, tv, a);
    return cudaGetLastError();
  }
  static PrefillVariant info() {
    return PrefillVariant{C::kThreads, C::kNT * 128, 128, C::kDV, 1, C::kStages, smem,
                          reinterpret_cast<const void*>(&prefill_tc_kernel<C>), &launch};
  }
};

}  // namespace vt
