// Work partition of the ragged prefill, computed on the device by every CTA.
//
// An item is (sequence, kv head (times a part of V's columns), q tile): the
// rows of tile_tokens consecutive new tokens for the query heads of one kv
// head, over the keys any of them attends to.  Items are ordered sequence,
// head, tile; item weights are lengths in tokens,
//   W = hi - lo + item_weight,
// the attended span plus a fixed part for the query load and the epilogue.
// The total weight is cut into even shares, one for each CTA, wherever the
// cuts fall: a share's items inside it are done whole, an item that a cut
// falls into is done in pieces of whole 128-key blocks by consecutive CTAs,
// whose partial sums prefill_combine_kernel joins.  Even shares need no host
// knowledge of lengths and no queue, and they balance causal tiles (whose
// cost grows with their position) as well as long contexts with few rows.
//
// A tree of drafted tokens (TREE) is the same with spans of its own: a row sees
// all tokens before the sequence's first new one, and of the new ones those
// its mask names, so every tile's span ends with the context.
//
// Weights of a sequence's first K tiles have a closed form (sums of
// arithmetic progressions, clipped where a window has not yet started), so a
// CTA finds its first item by a scan over sequences and a binary search over
// tiles, in exact integers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vt {

constexpr int kPfPage = 32;         // tokens per KV page
constexpr int kPfBlock = 128;       // keys per step

struct PrefillArgs {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int* q_starts;
  const int* block_tables;
  const int* context_lens;
  int num_seqs, num_tokens, num_q_heads, num_kv_heads, group;
  int max_blocks, num_blocks;
  int window;        // 0: none
  const int* masks;  // trees: [num_tokens][mask_words], bit i of a row: it sees new token i of its sequence
  int mask_words;
  float scale_log2;  // |scale| * log2(e); the sign is applied where the product is formed
  int neg_scale;
  int tile_tokens;   // new tokens of an item
  unsigned tile_mul, tile_shift;  // x / tile_tokens = x * tile_mul >> tile_shift for 0 <= x < 2^31
  int group_mul;     // r / group = r * group_mul >> 16 for 0 <= r <= 128
  int v_parts;       // items that share a (kv head, tile), each with a part of V's columns
  int item_weight;   // an item's fixed cost in tokens
  // Trees: new tokens up to which an item is one tile's.  A block of such an item weighs one_weight, where one of
  // two tiles weighs kPfBlock; x / one_weight is the high word of x * one_mul.
  int one_tile, one_weight;
  unsigned long long one_mul;
  int min_weight;    // least share of a CTA, whole kPfBlocks (every cut of an item then takes a block)
  long long long_total;  // total weight above which it doubles
  // Partials: record s (2 for each CTA: 2c an item's head piece, 2c + 1 a later piece) holds `rows` rows of
  // `cols` unnormalised fp32 sums; ml the rows' (running maximum, sum) in the log2 domain.
  float* part;
  float2* ml;
  struct PrefillSplit* splits;  // [grid] the item whose head piece CTA c has, if it is split
  unsigned* status;
  unsigned wait_limit;   // clock cycles
  int withhold_cta, withhold_block;  // test hook: this CTA stops loading before its withhold_block-th key block
};

// Written by the CTA that has an item's head piece, read by the combine.
struct PrefillSplit {
  int pieces;  // 0: none
  int row0, ntok, head, part;
};

// A sequence as the partition sees it.
struct PfSeq {
  int row0, n;       // first packed row, new tokens
  int p0;            // position of the first new token
  int bad;           // context outside [n, capacity]: its rows are NaN
  int tiles;
};

// x / tile_tokens, 0 <= x < 2^31 (a division's code is long).
__device__ __forceinline__ int pf_tiles_in(const PrefillArgs& a, int x) {
  return static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(x)) * a.tile_mul >> a.tile_shift);
}

// Token of a tile's row r.
__device__ __forceinline__ int pf_token_of(const PrefillArgs& a, int r) { return r * a.group_mul >> 16; }

template <bool TREE>
__device__ __forceinline__ PfSeq pf_seq(const PrefillArgs& a, int b) {
  PfSeq s;
  const int r0 = a.q_starts[b], r1 = a.q_starts[b + 1];
  const int L = a.context_lens[b];
  s.row0 = r0;
  s.n = (r0 >= 0 && r1 > r0 && r1 <= a.num_tokens) ? r1 - r0 : 0;
  s.bad = L < s.n || static_cast<long long>(L) > static_cast<long long>(a.max_blocks) * kPfPage;
  if (TREE && s.n > 32ll * a.mask_words) s.bad = 1;
  s.p0 = s.bad ? 0 : L - s.n;
  s.tiles = s.n > 0 ? pf_tiles_in(a, s.n - 1) + 1 : 0;
  return s;
}

__device__ __forceinline__ long long pf_mul(int a, int b) { return static_cast<long long>(a) * b; }

// Weight of the first K of the sequence's tiles (one head).  (Products of two
// 32-bit numbers and one 32-bit division: 64-bit ones are long code.)
template <bool TREE>
__device__ __forceinline__ long long pf_weight(const PrefillArgs& a, const PfSeq& s, int K) {
  const int T = a.tile_tokens;
  if (K <= 0) return 0;
  if (s.bad) return pf_mul(K, a.item_weight);
  if (TREE) {
    const int span = s.p0 + s.n - (a.window > 0 ? max(0, s.p0 - a.window) : 0);
    long long w = pf_mul(K, span) + pf_mul(K, a.item_weight);
    if (K == s.tiles && s.n - (K - 1) * T <= a.one_tile) w -= span - (pf_mul(span, a.one_weight) >> 7);
    return w;
  }
  long long w = ((pf_mul(K, K) + K) >> 1) * T + pf_mul(K, s.p0) + pf_mul(K, a.item_weight);
  if (K == s.tiles) w -= pf_mul(T, K) - s.n;
  if (a.window > 0) {
    const int A = s.p0 - a.window + 1;            // window start of the first token
    // first tile whose start is not clipped
    const int f = A >= 0 ? 0 : pf_tiles_in(a, -A - 1) + 1;
    if (K > f) w -= pf_mul(K - f, A) + ((pf_mul(K, K - 1) - pf_mul(f, f - 1)) >> 1) * T;
  }
  return w;
}

// One item, or a CTA's piece of it.
struct PfItem {
  int b, vh, tile;
  int row0;          // packed row of the tile's first token
  int ntok;          // tokens of the tile
  int pos0;          // position of its first token; of a tree, of the last token that every row sees
  int head, part;    // kv head, part of V's columns
  int lo;            // first attended key, rounded down to a page
  int lo_exact;      // first attended key
  int hi;            // one past the last attended key
  int L;             // context length
  int nkv;           // 128-key blocks of the item
  int kb0, kb1;      // this piece's blocks
  int pieces;        // head piece of a split item: pieces in all; else 0
  int bad;
};

// Walks a CTA's share.  Uniform over the threads that use it together, whole warps.
template <bool TREE = false>
struct PfWalk {
  long long x, end;       // weights: next item's part starts at x
  long long item_x;       // weight where the current item starts
  long long total, quot;  // total weight, and of one share (the last takes the remainder)
  int ctas;               // CTAs with a share
  int cta;                // this CTA
  PfSeq s;
  int b, vh, tile, heads;

  // Where CTA c's share starts.
  __device__ __forceinline__ long long share(unsigned c) const { return c >= static_cast<unsigned>(ctas) ? total : quot * c; }

  // kb(r): block boundary nearest to weight r of an item.
  __device__ __forceinline__ static int cut(const PrefillArgs& a, long long r, long long W, int nkv, int ntok) {
    if (r >= W) return nkv;
    long long k = (r - a.item_weight + kPfBlock / 2) >> 7;
    if (TREE && ntok <= a.one_tile) {
      const long long x = r - a.item_weight + (a.one_weight >> 1);
      k = x < 0 ? 0 : static_cast<long long>(__umul64hi(static_cast<unsigned long long>(x), a.one_mul));
    }
    return k < 0 ? 0 : (k > nkv ? nkv : static_cast<int>(k));
  }

  // The next sequence with rows.  In a padded batch many may have none, and
  // one after the other would cost a memory latency each: 32 at a time.
  __device__ __forceinline__ void next_sequence(const PrefillArgs& a) {
    if (++b < a.num_seqs) s = pf_seq<TREE>(a, b);
#pragma unroll 1
    while (b < a.num_seqs && s.tiles == 0) {
      const int at = b + 1 + static_cast<int>(threadIdx.x & 31);
      const unsigned with_rows = __ballot_sync(0xffffffffu, at < a.num_seqs && pf_seq<TREE>(a, at).tiles > 0);
      b += with_rows ? __ffs(with_rows) : 32;
      if (with_rows) s = pf_seq<TREE>(a, b);
    }
    if (b >= a.num_seqs) x = end;
  }

  // False when the share is done.  Items without this CTA's blocks are skipped.
  __device__ __forceinline__ bool next(const PrefillArgs& a, PfItem& it) {
    while (x < end) {
      long long W = 0;  // of the item: the difference of two sums (a loop: one copy of the code)
#pragma unroll 1
      for (int i = 0; i < 2; ++i) W = pf_weight<TREE>(a, s, tile + i) - W;
      it.b = b;
      it.vh = vh;
      it.tile = tile;
      it.head = vh >> (a.v_parts - 1);  // v_parts is 1 or 2
      it.part = vh & (a.v_parts - 1);
      it.row0 = s.row0 + tile * a.tile_tokens;
      it.ntok = min(a.tile_tokens, s.n - tile * a.tile_tokens);
      it.pos0 = TREE ? s.p0 - 1 : s.p0 + tile * a.tile_tokens;
      it.L = s.p0 + s.n;
      it.hi = TREE ? it.L : it.pos0 + it.ntok;
      it.lo_exact = a.window > 0 ? max(0, it.pos0 - a.window + 1) : 0;
      it.lo = it.lo_exact & ~(kPfPage - 1);
      it.nkv = s.bad ? 0 : (it.hi - it.lo + kPfBlock - 1) >> 7;
      it.bad = s.bad;
      it.pieces = 0;
      const long long ra = x - item_x, rb = end - item_x;
      const bool whole_end = rb >= W;
      it.kb0 = ra <= 0 ? 0 : cut(a, ra, W, it.nkv, it.ntok);
      it.kb1 = whole_end ? it.nkv : cut(a, rb, W, it.nkv, it.ntok);
      if (it.kb0 == 0 && it.kb1 < it.nkv && it.kb1 > 0) {
        // the head piece of a split item: count the cuts inside it
        it.pieces = 1;
#pragma unroll 1
        for (unsigned c = cta + 1;; ++c) {
          const long long e = share(c) - item_x;
          if ((e >= W ? it.nkv : cut(a, e, W, it.nkv, it.ntok)) >= it.nkv) break;
          ++it.pieces;
        }
      }
      const bool mine = it.nkv == 0 ? ra <= 0 : it.kb1 > it.kb0;
      if (whole_end) {
        x = item_x = item_x + W;
        if (++tile == s.tiles && x < end) {  // (else the share is over, whatever follows)
          tile = 0;
          if (++vh == heads) {
            vh = 0;
            next_sequence(a);
          }
        }
      } else {
        x = end;
      }
      if (mine) return true;
    }
    return false;
  }
};

// CTAs that get a share of a total weight: shares of min_weight (twice that
// above long_total) at least, in blocks.  (A 32-bit division: 2^32 blocks and
// more count as 2^32 - 1, which is more than there are CTAs.)
__host__ __device__ __forceinline__ unsigned pf_share_count(long long total, int min_weight, long long long_total,
                                                            unsigned grid) {
  const unsigned blocks = total >> 39 ? 0xffffffffu : static_cast<unsigned>(total >> 7);
  const unsigned most = blocks / static_cast<unsigned>(min_weight >> (total > long_total ? 6 : 7));
  return most < 1 ? 1u : most < grid ? most : grid;
}

// What one of `ctas` shares weighs; the last also takes the remainder.  (A 32-bit
// division of the total's leading 32 bits: of 152 shares the last is at most
// 152 * 152 / 2^31 of a share larger.)
__host__ __device__ __forceinline__ long long pf_share_weight(long long total, unsigned ctas) {
  int shift = 0;
  while (total >> shift >> 32) ++shift;
  return static_cast<long long>(static_cast<unsigned>(total >> shift) / ctas) << shift;
}

// The share of this CTA in a total weight; false if it has none.
template <bool TREE>
__device__ __forceinline__ bool pf_share(const PrefillArgs& a, long long total, PfWalk<TREE>& w) {
  w.heads = a.num_kv_heads * a.v_parts;
  w.ctas = static_cast<int>(pf_share_count(total, a.min_weight, a.long_total, gridDim.x));
  w.cta = blockIdx.x;
  w.x = w.end = 0;
  if (total == 0 || w.cta >= w.ctas) return false;
  w.total = total;
  w.quot = pf_share_weight(total, w.ctas);
  w.x = w.share(blockIdx.x);
  w.end = w.share(blockIdx.x + 1);
  return w.x < w.end;
}

// The item that holds weight w.x, in sequence b whose items start at weight
// `start`.  By one whole warp: 32 tiles are weighed at a time.
template <bool TREE>
__device__ __forceinline__ void pf_locate(const PrefillArgs& a, int b, long long start, int lane, PfWalk<TREE>& w) {
  w.b = b;
  w.s = pf_seq<TREE>(a, b);
  int lo = 0, hi = w.s.tiles, step = w.s.tiles;  // first the head (weight of all tiles), then the tile: W(0) = 0
  long long at_lo = 0;
  w.vh = -1;
#pragma unroll 1
  do {
    const int K = min(lo + (lane + 1) * step, hi);
    const long long m = pf_weight<TREE>(a, w.s, K);
    if (w.vh < 0) {
      for (w.vh = 0; w.x - start >= m; start += m) ++w.vh;
    } else {
      const unsigned below = __ballot_sync(0xffffffffu, K < hi && m <= w.x - start);
      const int n = __popc(below);  // candidates up to there weigh no more
      if (n > 0) at_lo = __shfl_sync(0xffffffffu, m, n - 1);
      hi = min(hi, lo + (n + 1) * step);
      lo += n * step;
    }
    step = (hi - lo + 31) / 32;
  } while (hi - lo > 1);
  w.tile = lo;
  w.item_x = start + at_lo;
}

__device__ __forceinline__ long long pf_warp_scan(long long x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  return x;
}

// The CTA's share, by one whole warp: each lane sums the weights of a run of
// consecutive sequences, a scan over lanes gives the total and the run that
// holds the share's start, and the warp looks through that run.
template <bool TREE>
__device__ __forceinline__ void pf_begin(const PrefillArgs& a, int lane, PfWalk<TREE>& w) {
  const int heads = a.num_kv_heads * a.v_parts;
  const int run = static_cast<int>((static_cast<unsigned>(a.num_seqs) + 31u) >> 5);
  int from = lane * run, to = min(from + run, a.num_seqs);
  long long before = 0;
  // first runs of `run` sequences, then the one run, in runs of its own
#pragma unroll 1
  for (int depth = 0;; ++depth) {
    long long mine = 0;
#pragma unroll 1
    for (int b = from; b < to; ++b) {
      const PfSeq s = pf_seq<TREE>(a, b);
      mine += heads * pf_weight<TREE>(a, s, s.tiles);
    }
    const long long inc = before + pf_warp_scan(mine, lane);
    if (depth == 0 && !pf_share(a, __shfl_sync(0xffffffffu, inc, 31), w)) return;
    const int hit = __ffs(__ballot_sync(0xffffffffu, w.x < inc)) - 1;
    before = __shfl_sync(0xffffffffu, inc - mine, hit);
    const int first = __shfl_sync(0xffffffffu, from, hit), last = __shfl_sync(0xffffffffu, to, hit);
    if (last - first <= 1) {
      pf_locate(a, first, before, lane, w);
      return;
    }
    const int step = (last - first + 31) >> 5;
    from = min(first + lane * step, last);
    to = min(from + step, last);
  }
}

// ---- trees
// The mask of packed row `row`.
__device__ __forceinline__ const int* tree_mask(const PrefillArgs& a, int row) {
  return a.masks + static_cast<long long>(row) * a.mask_words;
}

// Word i of a mask of a sequence with n new tokens.
__device__ __forceinline__ unsigned tree_word(const int* mask, int i, int n) {
  const int left = n - 32 * i;
  if (left <= 0) return 0u;
  const unsigned w = static_cast<unsigned>(mask[i]);
  return left < 32 ? w & ((1u << left) - 1u) : w;
}

// What a row of a tree sees.  The first words of its mask are read when the row
// is taken up, long before they are needed (a load takes 2400 cycles while all
// SMs read keys and values).
struct TreeRow {
  const int* mask = nullptr;
  int n = 0;        // new tokens of its sequence
  int base = 0;     // position of the first
  int from = 0;     // the first key its window takes in
  unsigned w0 = 0, w1 = 0;

  __device__ __forceinline__ unsigned word(int i) const { return i == 0 ? w0 : i == 1 ? w1 : tree_word(mask, i, n); }

  // Packed row `row` of a sequence with n new tokens from position `base` on.
  __device__ __forceinline__ void take(const PrefillArgs& a, int row, int n_, int base_) {
    mask = tree_mask(a, row);
    n = n_;
    base = base_;
    w0 = tree_word(mask, 0, n);
    w1 = tree_word(mask, 1, n);
    from = 0;
    if (a.window > 0) from = window_start(a.window);
  }
  // Of the tokens the row may see (those before `base`, then the new ones its
  // mask names) it sees the last `window`.
  __device__ __forceinline__ int window_start(int window) const {
    int count = 0;
#pragma unroll 1
    for (int i = 0; 32 * i < n; ++i) count += __popc(word(i));
    int skip = count - window;  // new tokens before the window
    if (skip < 0) return max(0, base + skip);
#pragma unroll 1
    for (int i = 0;; ++i) {
      unsigned w = word(i);
      const int c = __popc(w);
      if (skip < c) {
        for (; skip > 0; --skip) w &= w - 1u;
        return base + 32 * i + __ffs(w) - 1;
      }
      skip -= c;
    }
  }
  // Which of the keys k .. k + 31 it sees: bit by bit.
  __device__ __forceinline__ unsigned seen(int k) const {
    const int ahead = k - base, i = ahead >> 5;  // (rounded down)
    const unsigned lo = i < 0 ? ~0u : word(i);
    const unsigned hi = i + 1 < 0 ? ~0u : word(i + 1);
    const int before = from - k;
    return __funnelshift_r(lo, hi, ahead & 31) & (before <= 0 ? ~0u : before > 31 ? 0u : ~0u << before);
  }
};

}  // namespace vt
