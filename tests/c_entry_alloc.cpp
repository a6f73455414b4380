// The serving operators' C entry points when host memory runs out: operator
// new fails on demand, and each call has to come back with a status.  Meant for
// a machine without a GPU, where the calls allocate the text of the CUDA error
// and launch nothing.
#include <cstdio>
#include <cstdlib>
#include <exception>
#include <new>

#include "vt_paged_attn.h"

static bool g_fail = false;

void* operator new(std::size_t n) {
  if (g_fail) throw std::bad_alloc();
  void* p = std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

static char* at(long n) { return reinterpret_cast<char*>(n); }

template <typename F>
static int call(const char* name, F f) {
  int status = -1;
  try {
    g_fail = true;
    status = f();
    g_fail = false;
  } catch (...) {
    g_fail = false;
    std::printf("%s: an exception left the call\n", name);
    return 1;
  }
  std::printf("%s: %s\n", name, vt_status_string(static_cast<vt_status>(status)));
  return status == VT_ERR_OOM ? 0 : 1;
}

int main() {
  std::set_terminate([] {
    std::puts("terminated");
    std::abort();
  });
  const int32_t* i32 = reinterpret_cast<const int32_t*>(at(0x3000));
  const double* freq = reinterpret_cast<const double*>(at(0x4000));
  const float* f32 = reinterpret_cast<const float*>(at(0x5000));
  int bad = 0;
  bad += call("vt_rope", [&] {
    return vt_rope(at(0x1000), at(0x2000), i32, freq, 2, 4, 128, 128, 0, 1.f, 512, 512, nullptr, VT_BF16);
  });
  bad += call("vt_paged_kv_append", [&] {
    return vt_paged_kv_append(at(0x1000), at(0x2000), nullptr, at(0x6000), at(0x7000), nullptr, i32, i32, i32, nullptr,
                              freq, 2, 5, 0, 2, 128, 32, 128, 0, 1.f, 0, 256, 256, nullptr, 4, 16, VT_BF16);
  });
  bad += call("vt_paged_kv_append_fp8", [&] {
    return vt_paged_kv_append_fp8(at(0x1000), at(0x2000), nullptr, at(0x6000), at(0x7000), nullptr, f32, f32, i32, i32,
                                  i32, nullptr, freq, 2, 5, 0, 2, 128, 32, 128, 0, 1.f, 0, 256, 256, nullptr, 4, 16);
  });
  bad += call("vt_paged_attn_prefill", [&] {
    return vt_paged_attn_prefill(at(0x1000), at(0x2000), at(0x6000), at(0x7000), i32, i32, i32, 2, 5, 8, 2, 128, 32,
                                 0.1f, 0, nullptr, 4, 16, VT_BF16);
  });
  bad += call("vt_paged_attn_prefill_fp8", [&] {
    return vt_paged_attn_prefill_fp8(at(0x1000), at(0x2000), at(0x6000), at(0x7000), f32, f32, i32, i32, i32, 2, 5, 8,
                                     2, 128, 32, 0.1f, 0, nullptr, 4, 16);
  });
  if (!bad) std::puts("c entries: ok");
  return bad;
}
