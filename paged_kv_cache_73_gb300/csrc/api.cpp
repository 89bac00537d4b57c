// Error reporting and version entry points of the C ABI.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
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

}  // namespace pkv

extern "C" {

const char* pkv_last_error(void) { return pkv::g_last_error.c_str(); }

int pkv_version(void) { return 100; }

int pkv_device_error(void* stream, int reset, int* code) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess)
    return pkv::fail(PKV_ERR_CUDA, "pkv_device_error: cudaStreamSynchronize: %s", cudaGetErrorString(e));
  // one check word per translation unit that launches kernels
  int (*const readers[])(int, int*) = {pkv::read_device_error_attention, pkv::read_device_error_cache_ops,
                                       pkv::read_device_error_prefill, pkv::read_device_error_rope,
                                       pkv::read_device_error_cache_int4, pkv::read_device_error_attention_int4,
                                       pkv::read_device_error_prompt};
  int first = 0;
  for (auto read : readers) {
    int word = 0;
    const int st = read(reset, &word);
    if (st != PKV_OK) return st;
    if (!first) first = word;
  }
  if (code) *code = first;
  if (first) return pkv::fail(PKV_ERR_DEVICE_CHECK, "a kernel recorded device check code %d", first);
  return PKV_OK;
}

}  // extern "C"
