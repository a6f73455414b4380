// Host-side state and helpers shared by the library's entry points; defined
// in vt_paged_attn_api.cu.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "../../include/vt_paged_attn.h"

namespace vt {
namespace host {

constexpr size_t kStatusBytes = 256;
// Packed rows, and sequences, of a ragged batch: numbers a little past the last
// one (of a search's probes, of a tile's end) stay in 32 bits.
constexpr int kMaxTokens = 0x7fffffff - (1 << 20);

constexpr int kMaxMaskWords = 32;  // of a drafted token's mask: 1024 of them a sequence

struct Scratch {
  char* base = nullptr;
  size_t bytes = 0;
  size_t counters_cap = 0;  // bytes after the status words that hold zeroed counters
  size_t captured_tail = 0;  // caller-owned: bytes at the end that captured prefills name, where no counter may go
};

struct DeviceState {
  bool init = false;
  int num_sms = 0;
  Scratch lib;               // library-owned (cudaMallocAsync, grows)
  Scratch user;              // caller-owned (vt_paged_attn_set_workspace)
  char* noalloc = nullptr;   // device address of the static array, once looked up
  // Prefill scratch, library-owned.  A buffer that became too small is kept
  // until vt_paged_attn_release: captured graphs may still name it.
  Scratch prefill;
  std::vector<char*> prefill_retired;
  std::vector<std::pair<const void*, int>> occupancy;
};

// Per host thread: text of the last CUDA error, and the test overrides.
extern thread_local std::string g_last_cuda_error;
extern thread_local long long g_test_wait_limit;  // <= 0: the kernels' default
extern thread_local int g_test_withhold_cta;
extern thread_local int g_test_withhold_tile;
extern thread_local int g_override_grid;
extern thread_local int g_override_min_units;

extern thread_local vt_plan g_last_plan;  // what the thread's last decode or prefill launched
extern thread_local bool g_have_plan;

extern std::mutex g_mutex;  // guards every DeviceState

DeviceState& device_state(int dev);                     // caller holds g_mutex
vt_status prepare_device(int dev, DeviceState& ds);     // caller holds g_mutex
vt_status cuda_fail(cudaError_t e, const char* where);  // records the text, returns VT_ERR_CUDA
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();          // nullptr if the driver lacks it

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace host
}  // namespace vt
