// Error reporting and version entry points of the C ABI.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "pkv_internal.h"

namespace pkv {

static thread_local std::string g_last_error;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

void clear_error() { g_last_error.clear(); }

namespace {

// One check word per translation unit that launches kernels.
int (*const kWords[])(void**) = {device_error_word_attention,  device_error_word_cache_ops,
                                 device_error_word_prefill,    device_error_word_rope,
                                 device_error_word_cache_int4, device_error_word_attention_int4,
                                 device_error_word_prompt,     device_error_word_tree_attention,
                                 device_error_word_drafts};
constexpr int kUnits = sizeof(kWords) / sizeof(kWords[0]);

// Page-locked memory for one call's words, so that they come in copies one behind the other with one wait
// (an idle stream is checked in 19 us; one blocking copy per word took 66).  Kept for later calls: as many as have
// ever run at once.
std::mutex g_pinned_mutex;
int* g_pinned_free = nullptr;                                 // a list through the buffers themselves

struct PinnedInts {
  union Buffer {
    int ints[kUnits];
    int* next;
  };
  int* at = nullptr;
  PinnedInts() {
    {
      std::lock_guard<std::mutex> g(g_pinned_mutex);
      if (g_pinned_free) {
        at = g_pinned_free;
        g_pinned_free = reinterpret_cast<Buffer*>(at)->next;
      }
    }
    void* p = nullptr;
    if (!at && cudaHostAlloc(&p, sizeof(Buffer), cudaHostAllocPortable) == cudaSuccess) at = static_cast<int*>(p);
  }
  ~PinnedInts() {
    if (!at) return;
    std::lock_guard<std::mutex> g(g_pinned_mutex);
    reinterpret_cast<Buffer*>(at)->next = g_pinned_free;
    g_pinned_free = at;
  }
  PinnedInts(const PinnedInts&) = delete;
  PinnedInts& operator=(const PinnedInts&) = delete;
};

}  // namespace

}  // namespace pkv

extern "C" {

const char* pkv_last_error(void) { return pkv::g_last_error.c_str(); }

int pkv_version(void) { return 100; }

int pkv_device_error(void* stream, int reset, int* code) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess)
    return pkv::fail(PKV_ERR_CUDA, "pkv_device_error: cudaStreamSynchronize: %s", cudaGetErrorString(e));
  pkv::PinnedInts words;
  if (!words.at) return pkv::fail(PKV_ERR_CUDA, "pkv_device_error: no page-locked host memory");
  void* place[pkv::kUnits];
  for (int i = 0; i < pkv::kUnits && e == cudaSuccess; ++i) {
    e = static_cast<cudaError_t>(pkv::kWords[i](&place[i]));
    if (e == cudaSuccess) e = cudaMemcpyAsync(words.at + i, place[i], sizeof(int), cudaMemcpyDeviceToHost, st);
  }
  cudaError_t done = cudaStreamSynchronize(st);               // also where a copy could not be issued: the others end
  if (e == cudaSuccess) e = done;
  int first = 0;
  for (int i = 0; i < pkv::kUnits && e == cudaSuccess; ++i) {
    if (words.at[i] == 0) continue;
    if (!first) first = words.at[i];
    if (reset) e = cudaMemsetAsync(place[i], 0, sizeof(int), st);
  }
  if (e == cudaSuccess && first && reset) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "reading the check words: %s", cudaGetErrorString(e));
  if (code) *code = first;
  if (first) return pkv::fail(PKV_ERR_DEVICE_CHECK, "a kernel recorded device check code %d", first);
  return PKV_OK;
}

}  // extern "C"
