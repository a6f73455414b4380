// The bookkeeping of a serving step on the GPU: pages given back and taken,
// block tables, row starts, positions and slots, from request lengths.
//
// Mathematics.  With pg(x) = ceil(x / 32), a sequence that keeps k of its L
// tokens and gets n new ones gives back pg(L) - pg(k) pages and takes
// pg(k + n) - pg(k).  Three prefix sums over the sequences (pages given back,
// pages taken, rows) say where each one's pages lie on the stack of free pages
// and where its rows begin; everything else is a lookup.
//
// What bounds it: a chain of latencies (lengths, sums, the barrier between
// pages put on the stack and pages taken from it, a search for each row's
// sequence), not its few bytes.  So it is one launch of one cluster: every CTA
// forms all sums for itself, in shared memory, and the cluster's barrier is all
// that is waited for.  Measured, calls in a row from a graph: 256 sequences with
// one new token each 5.0 us, 33 thousand prompt tokens beside 40 sequences that
// end 7.7 (four CTAs 10.6, CTAs of 256 threads 11.7, one row a thread at a time
// 9.3; the launch alone takes 2.5).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <new>

#include "../../include/vt_paged_attn.h"
#include "host_state.cuh"

namespace vt {
namespace {

constexpr int kPage = 32;
constexpr int kThreads = 512;
constexpr int kCtas = 8;           // of the cluster
constexpr int kMaxSeqs = 16384;    // 12 bytes of shared memory each
constexpr int kRowsAhead = 4;      // rows whose searches and loads a thread has under way

struct TablesArgs {
  int* block_tables;
  int* context_lens;
  int* free_pages;
  int* counters;  // pages on the stack, sequences refused
  int* q_starts;
  int* positions;
  int* slots;
  const int* keep_lens;
  const int* new_lens;
  int num_seqs, num_tokens, max_blocks, num_blocks;
};

__device__ __forceinline__ int pages_of(int tokens) {  // tokens >= 0
  return static_cast<int>((static_cast<unsigned>(tokens) + kPage - 1) / kPage);
}

// What a sequence asks for.
struct Ask {
  int keep;            // tokens kept
  int have, kept;      // pages before, and of the tokens kept
  int need, rows;      // pages and rows of its growth (0 if it does not grow, or on its own cannot)
  bool valid, refused; // refused: lengths that are none, or a table's row that is too short
};

__device__ __forceinline__ Ask ask_of(const TablesArgs& a, int b) {
  Ask q{0, 0, 0, 0, 0, true, false};
  if (b >= a.num_seqs) return q;
  const long long room = static_cast<long long>(a.max_blocks) * kPage;
  const int L = a.context_lens[b], n = a.new_lens[b];
  q.keep = a.keep_lens ? a.keep_lens[b] : L;
  if (L < 0 || L > room || q.keep < 0 || q.keep > L || n < 0) {
    q.valid = false;
    q.refused = true;
    q.keep = L;
    return q;
  }
  q.have = pages_of(L);
  q.kept = pages_of(q.keep);
  if (q.keep + static_cast<long long>(n) > room) {
    q.refused = true;
  } else {
    q.rows = n;
    q.need = pages_of(q.keep + n) - q.kept;
  }
  return q;
}

struct Sums {
  long long given, need, rows;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.given + b.given, a.need + b.need, a.rows + b.rows};
}
__device__ __forceinline__ Sums shift_up(const Sums& a, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, a.given, d), __shfl_up_sync(0xffffffffu, a.need, d),
              __shfl_up_sync(0xffffffffu, a.rows, d)};
}

// Inclusive sums over the block's threads; `total` the last one's.
__device__ __forceinline__ Sums block_scan(Sums x, Sums (&of_warp)[kThreads / 32], Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shift_up(x, d);
    if (lane >= d) x = x + o;
  }
  __syncthreads();  // the array's last use is over
  if (lane == 31) of_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Sums y = lane < kThreads / 32 ? of_warp[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shift_up(y, d);
      if (lane >= d) y = y + o;
    }
    if (lane < kThreads / 32) of_warp[lane] = y;
  }
  __syncthreads();
  total = of_warp[kThreads / 32 - 1];
  return warp > 0 ? x + of_warp[warp - 1] : x;
}

__global__ void __launch_bounds__(kThreads) step_tables_kernel(const TablesArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ int raw[];
  int* const row_start = raw;                     // [num_seqs + 1] rows of the sequences before
  int* const page_start = row_start + a.num_seqs + 1;  // [num_seqs] pages they take
  int* const keep = page_start + a.num_seqs;      // [num_seqs]
  __shared__ Sums of_warp[kThreads / 32];
  __shared__ int given_start[kThreads];
  __shared__ int first_out;  // first growing sequence that does not fit
  __shared__ int refused;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int B = a.num_seqs, cap = a.num_blocks;
  if (tid == 0) {
    first_out = B;
    refused = 0;
  }
  const int on_stack = max(0, min(a.counters[0], cap));

  // pages given back in all: they lie on top of the stack (with one sequence a
  // thread the sums below say it at once)
  long long given = 0;
  for (int b0 = 0; b0 < B && B > kThreads; b0 += kThreads) {
    const Ask q = ask_of(a, b0 + tid);
    Sums sum;
    block_scan(Sums{q.have - q.kept, 0, 0}, of_warp, sum);
    given += sum.given;
  }
  long long top = on_stack + given;  // of the stack with them
  int avail = on_stack;              // pages to take

  Sums before{0, 0, 0};
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    const Ask q = ask_of(a, b);
    Sums sum;
    const Sums mine{q.have - q.kept, q.need, q.rows};
    const Sums end = before + block_scan(mine, of_warp, sum);
    before = before + sum;
    if (B <= kThreads) top = on_stack + sum.given;
    avail = static_cast<int>(top < cap ? top : cap);  // (more than the pool has: such pages are not kept)
    const long long big = 0x7fffffff;
    if (b < B) {
      row_start[b] = static_cast<int>(min(big, end.rows - q.rows));
      page_start[b] = static_cast<int>(min(big, end.need - q.need));
      keep[b] = q.keep;
      if (q.rows > 0 && (end.need > avail || end.rows > a.num_tokens)) atomicMin(&first_out, b);
      if (q.refused) atomicAdd(&refused, 1);
    }
    given_start[tid] = static_cast<int>(min(big, end.given - mine.given));
    __syncthreads();
    // given back, the first on top; a warp a sequence
    for (int i = warp * ctas + rank; i < kThreads && b0 + i < B; i += kThreads / 32 * ctas) {
      const Ask o = ask_of(a, b0 + i);
      for (int p = o.kept + lane; p < o.have; p += 32) {
        const long long at = top - 1 - (static_cast<long long>(given_start[i]) + (p - o.kept));
        if (at >= 0 && at < cap) a.free_pages[at] = a.block_tables[static_cast<long long>(b0 + i) * a.max_blocks + p];
      }
    }
  }
  if (tid == 0) row_start[B] = static_cast<int>(min(0x7fffffffll, before.rows));
  __syncthreads();
  const int out = first_out;  // sequences from here on do not grow
  if (rank == 0) {
    int late = 0;
    for (int b = out + tid; b < B; b += kThreads) late += ask_of(a, b).rows > 0;
    if (late) atomicAdd(&refused, late);
  }
  // every CTA has read the lengths and the stack's size, and all pages given back are on it
  cluster.sync();

  const int rows = row_start[out];
  const int threads = kThreads * ctas, thread = rank * kThreads + tid;
  for (int b = thread; b <= B; b += threads) {
    a.q_starts[b] = row_start[min(b, out)];
    if (b < B) a.context_lens[b] = keep[b] + (b < out ? row_start[b + 1] - row_start[b] : 0);
  }
  int first_step = 1;  // of a search: the power of two below out
  while (2 * first_step < out) first_step *= 2;
#pragma unroll 1
  for (int i0 = thread; i0 < rows; i0 += kRowsAhead * threads) {
    int lo[kRowsAhead] = {}, page[kRowsAhead], pos[kRowsAhead];
#pragma unroll 1
    for (int d = first_step; d > 0; d >>= 1)  // the last sequence whose rows begin at or before i
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        if (lo[u] + d < out && row_start[lo[u] + d] <= i0 + u * threads) lo[u] += d;
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int i = i0 + u * threads;
      if (i >= rows) continue;
      const int k = keep[lo[u]], kept = pages_of(k);
      pos[u] = k + (i - row_start[lo[u]]);
      const int p = pos[u] / kPage;
      page[u] = p >= kept ? __ldcg(a.free_pages + (avail - 1 - (page_start[lo[u]] + (p - kept))))
                          : a.block_tables[static_cast<long long>(lo[u]) * a.max_blocks + p];
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int i = i0 + u * threads;
      if (i >= rows) continue;
      // (a position on a page's first slot is behind the tokens kept: a page that was taken)
      if (pos[u] % kPage == 0) a.block_tables[static_cast<long long>(lo[u]) * a.max_blocks + pos[u] / kPage] = page[u];
      if (a.positions) a.positions[i] = pos[u];
      if (a.slots) a.slots[i] = page[u] >= 0 && page[u] < cap ? page[u] * kPage + pos[u] % kPage : -1;
    }
  }
  if (thread == 0) {
    const int taken = out < B ? page_start[out] : static_cast<int>(before.need);
    a.counters[0] = avail - taken;
    a.counters[1] = refused;
  }
}

using namespace vt::host;

size_t tables_smem(int num_seqs) { return sizeof(int) * (3 * static_cast<size_t>(num_seqs) + 1); }

vt_status step_tables(const TablesArgs& a, int block_size, cudaStream_t stream) {
  if (a.num_seqs < 0 || a.num_tokens < 0 || a.max_blocks <= 0 || a.num_blocks <= 0 || block_size <= 0)
    return VT_ERR_INVALID_ARG;
  if (!a.free_pages || !a.counters || !a.q_starts) return VT_ERR_INVALID_ARG;
  if (a.num_seqs > 0 && (!a.block_tables || !a.context_lens || !a.new_lens)) return VT_ERR_INVALID_ARG;
  if (!aligned(a.block_tables, 4) || !aligned(a.context_lens, 4) || !aligned(a.free_pages, 4) ||
      !aligned(a.counters, 4) || !aligned(a.q_starts, 4) || !aligned(a.positions, 4) || !aligned(a.slots, 4) ||
      !aligned(a.keep_lens, 4) || !aligned(a.new_lens, 4))
    return VT_ERR_INVALID_ARG;
  if (block_size != kPage || a.num_seqs > kMaxSeqs || a.num_tokens > kMaxTokens) return VT_ERR_UNSUPPORTED;
  if (static_cast<long long>(a.num_blocks) * kPage > 0x7fffffffLL ||
      static_cast<long long>(a.max_blocks) * kPage > 0x7fffffffLL)
    return VT_ERR_UNSUPPORTED;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceState& ds = device_state(dev);
    const vt_status st = prepare_device(dev, ds);
    if (st != VT_OK) return st;
    const void* const func = reinterpret_cast<const void*>(&step_tables_kernel);
    bool known = false;
    for (auto& p : ds.occupancy) known |= p.first == func;
    if (!known) {
      e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(tables_smem(kMaxSeqs)));
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
      ds.occupancy.emplace_back(func, 1);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = tables_smem(a.num_seqs);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, step_tables_kernel, a);
  return e == cudaSuccess ? VT_OK : cuda_fail(e, "step tables launch");
}

}  // namespace
}  // namespace vt

extern "C" {

vt_status vt_paged_step_tables(int32_t* block_tables, int32_t* context_lens, int32_t* free_pages, int32_t* counters,
                               int32_t* q_starts, int32_t* positions, int32_t* slots, const int32_t* keep_lens,
                               const int32_t* new_lens, int num_seqs, int num_tokens, int block_size,
                               vt_stream_t stream, int max_blocks_per_seq, int num_blocks) {
  try {
    return vt::step_tables(vt::TablesArgs{block_tables, context_lens, free_pages, counters, q_starts, positions,
                                          slots, keep_lens, new_lens, num_seqs, num_tokens, max_blocks_per_seq,
                                          num_blocks},
                           block_size, reinterpret_cast<cudaStream_t>(stream));
  } catch (const std::bad_alloc&) {
    return VT_ERR_OOM;
  }
}

}  // extern "C"
