// Work partition of the ragged prefill, computed on the device by every CTA.
//
// An item is (sequence, kv head (times a part of V's columns), q tile): the
// rows of tile_tokens consecutive new tokens for the query heads of one kv
// head, over the keys any of them attends to.  Items are ordered sequence,
// head, tile; item weights are lengths in tokens,
//   W = hi - lo + kItemWeight,
// the attended span plus a fixed part for the query load and the epilogue.
// The total weight is cut into even shares, one for each CTA, wherever the
// cuts fall: a share's items inside it are done whole, an item that a cut
// falls into is done in pieces of whole 128-key blocks by consecutive CTAs,
// whose partial sums prefill_combine_kernel joins.  Even shares need no host
// knowledge of lengths and no queue, and they balance causal tiles (whose
// cost grows with their position) as well as long contexts with few rows.
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
constexpr int kPfItemWeight = 128;  // an item's fixed cost in tokens

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
  float scale_log2;  // |scale| * log2(e); the sign is applied where the product is formed
  int neg_scale;
  int tile_tokens;   // new tokens of an item
  int v_parts;       // items that share a (kv head, tile), each with a part of V's columns
  int min_weight;    // least share of a CTA, at least 2 * kPfBlock
  // Partials: record s (2 for each CTA: 2c an item's head piece, 2c + 1 a later piece) holds `rows` rows of
  // `cols` unnormalised fp32 sums; ml the rows' (running maximum, sum) in the log2 domain.
  float* part;
  float2* ml;
  struct PrefillSplit* splits;  // [grid] the item whose head piece CTA c has, if it is split
  unsigned* status;
  long long wait_limit;
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

__device__ __forceinline__ PfSeq pf_seq(const PrefillArgs& a, int b) {
  PfSeq s;
  const int r0 = a.q_starts[b], r1 = a.q_starts[b + 1];
  const int L = a.context_lens[b];
  s.row0 = r0;
  s.n = (r0 >= 0 && r1 > r0 && r1 <= a.num_tokens) ? r1 - r0 : 0;
  s.bad = L < s.n || static_cast<long long>(L) > static_cast<long long>(a.max_blocks) * kPfPage;
  s.p0 = s.bad ? 0 : L - s.n;
  s.tiles = (s.n + a.tile_tokens - 1) / a.tile_tokens;
  return s;
}

// Weight of the first K of the sequence's tiles (one head).
__device__ __forceinline__ long long pf_weight(const PrefillArgs& a, const PfSeq& s, int K) {
  const long long T = a.tile_tokens, k = K;
  if (K <= 0) return 0;
  if (s.bad) return k * kPfItemWeight;
  long long w = T * k * (k + 1) / 2 + k * (static_cast<long long>(s.p0) + kPfItemWeight);
  if (K == s.tiles) w -= T * k - s.n;
  if (a.window > 0) {
    const long long A = static_cast<long long>(s.p0) - a.window + 1;  // window start of the first token
    const long long f = A >= 0 ? 0 : (-A + T - 1) / T;                // first tile whose start is clipped
    if (k > f) w -= (k - f) * A + T * ((k * (k - 1) - f * (f - 1)) / 2);
  }
  return w;
}

// One item, or a CTA's piece of it.
struct PfItem {
  int b, vh, tile;
  int row0;          // packed row of the tile's first token
  int ntok;          // tokens of the tile
  int pos0;          // position of its first token
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

// Walks a CTA's share.  Uniform over the threads that use it together.
struct PfWalk {
  long long x, end;       // weights: next item's part starts at x
  long long item_x;       // weight where the current item starts
  long long total;
  int ctas;               // CTAs with a share
  int cta;                // this CTA
  PfSeq s;
  int b, vh, tile, heads;

  // kb(r): block boundary nearest to weight r of an item.
  __device__ __forceinline__ static int cut(long long r, long long W, int nkv) {
    if (r >= W) return nkv;
    const long long k = (r - kPfItemWeight + kPfBlock / 2) >> 7;
    return k < 0 ? 0 : (k > nkv ? nkv : static_cast<int>(k));
  }

  // False when the share is done.  Items without this CTA's blocks are skipped.
  __device__ __forceinline__ bool next(const PrefillArgs& a, PfItem& it) {
    while (x < end) {
      const long long W = pf_weight(a, s, tile + 1) - pf_weight(a, s, tile);
      it.b = b;
      it.vh = vh;
      it.tile = tile;
      it.head = vh / a.v_parts;
      it.part = vh - it.head * a.v_parts;
      it.row0 = s.row0 + tile * a.tile_tokens;
      it.ntok = min(a.tile_tokens, s.n - tile * a.tile_tokens);
      it.pos0 = s.p0 + tile * a.tile_tokens;
      it.L = s.p0 + s.n;
      it.hi = it.pos0 + it.ntok;
      it.lo_exact = a.window > 0 ? max(0, it.pos0 - a.window + 1) : 0;
      it.lo = it.lo_exact / kPfPage * kPfPage;
      it.nkv = s.bad ? 0 : (it.hi - it.lo + kPfBlock - 1) / kPfBlock;
      it.bad = s.bad;
      it.pieces = 0;
      const long long ra = x - item_x, rb = end - item_x;
      const bool whole_end = rb >= W;
      it.kb0 = ra <= 0 ? 0 : cut(ra, W, it.nkv);
      it.kb1 = whole_end ? it.nkv : cut(rb, W, it.nkv);
      if (it.kb0 == 0 && it.kb1 < it.nkv && it.kb1 > 0) {
        // the head piece of a split item: count the cuts inside it
        it.pieces = 1;
        long long c = cta;
        for (;;) {
          ++c;
          const long long e = total * c / ctas;
          const int k = e - item_x >= W ? it.nkv : cut(e - item_x, W, it.nkv);
          if (k >= it.nkv) break;
          ++it.pieces;
        }
      }
      const bool mine = it.nkv == 0 ? ra <= 0 : it.kb1 > it.kb0;
      if (whole_end) {
        x = item_x = item_x + W;
        if (++tile == s.tiles) {
          tile = 0;
          if (++vh == heads) {
            vh = 0;
            do {
              if (++b >= a.num_seqs) {
                x = end;
                break;
              }
              s = pf_seq(a, b);
            } while (s.tiles == 0);
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

// The CTA's share: every thread calls it once, with all threads of the CTA;
// `scan` holds blockDim.x / 32 + 4 values of shared memory.
__device__ inline void pf_begin(const PrefillArgs& a, long long* scan, PfWalk& w) {
  const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nth >> 5;
  const int heads = a.num_kv_heads * a.v_parts;
  // total weight, in chunks of blockDim.x sequences
  long long sum = 0;
  for (int b = tid; b < a.num_seqs; b += nth) {
    const PfSeq s = pf_seq(a, b);
    sum += heads * pf_weight(a, s, s.tiles);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) scan[warp] = sum;
  __syncthreads();
  long long total = 0;
  for (int k = 0; k < warps; ++k) total += scan[k];
  __syncthreads();
  w.total = total;
  w.heads = heads;
  const long long most = total / a.min_weight;
  w.ctas = static_cast<int>(most < 1 ? 1 : (most < gridDim.x ? most : gridDim.x));
  w.cta = blockIdx.x;
  const long long c = blockIdx.x;
  w.x = w.cta < w.ctas ? total * c / w.ctas : 0;
  w.end = w.cta < w.ctas ? total * (c + 1) / w.ctas : 0;
  if (total == 0 || w.x >= w.end) {  // nothing to do
    w.x = w.end = 0;
    return;
  }
  // the sequence that holds weight x: inclusive scan over chunks
  long long before = 0;
  if (tid == 0) scan[warps] = -1;
  for (int b0 = 0; b0 < a.num_seqs; b0 += nth) {
    const int b = b0 + tid;
    long long mine = 0;
    if (b < a.num_seqs) {
      const PfSeq s = pf_seq(a, b);
      mine = heads * pf_weight(a, s, s.tiles);
    }
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    long long base = before, chunk = 0;
    for (int k = 0; k < warps; ++k) {
      if (k < warp) base += scan[k];
      chunk += scan[k];
    }
    const long long lo = base + inc - mine;
    if (mine > 0 && w.x >= lo && w.x < base + inc) {
      scan[warps] = b;
      scan[warps + 1] = lo;
    }
    before += chunk;
    __syncthreads();
    if (scan[warps] >= 0) break;
  }
  w.b = static_cast<int>(scan[warps]);
  long long start = scan[warps + 1];
  w.s = pf_seq(a, w.b);
  const long long per_head = pf_weight(a, w.s, w.s.tiles);
  w.vh = static_cast<int>((w.x - start) / per_head);
  start += w.vh * per_head;
  int lo = 0, hi = w.s.tiles;  // pf_weight(lo) <= x - start < pf_weight(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pf_weight(a, w.s, mid) <= w.x - start) lo = mid; else hi = mid;
  }
  w.tile = lo;
  w.item_x = start + pf_weight(a, w.s, lo);
}

}  // namespace vt
