// The status word of the stand-alone operators: one per device, for every call that brings none of its own, so that a
// wait that runs out inside a kernel is never lost.  A device variable: it needs no allocation, which a captured call
// could not make, and lives as long as the graphs that hold its address.
#include <atomic>

#include "api_internal.h"
#include "moe_b200.h"

namespace {

__device__ int operator_status;

int cuda_failed(cudaError_t e) {
  cudaGetLastError();  // reported here; not left behind for another caller's check
  return moe::api_fail(MOE_ERR_CUDA, "operator_status: %s", cudaGetErrorString(e));
}

}  // namespace

cudaError_t moe::operator_status_word(int** word) {
  static std::atomic<int*> known[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  *word = known[dev].load(std::memory_order_acquire);
  if (*word != nullptr) return cudaSuccess;
  void* p = nullptr;
  if ((e = cudaGetSymbolAddress(&p, operator_status)) != cudaSuccess) return e;
  *word = static_cast<int*>(p);
  known[dev].store(*word, std::memory_order_release);
  return cudaSuccess;
}

extern "C" {

int moe_operator_status_word(int32_t** word) {
  if (!word) return moe::api_fail(MOE_ERR_INVALID, "operator_status_word: NULL pointer");
  const int rc = moe::api_device_check(nullptr);
  if (rc != MOE_OK) return rc;
  const cudaError_t e = moe::operator_status_word(word);
  return e == cudaSuccess ? MOE_OK : cuda_failed(e);
}

int moe_operator_status(int32_t clear, int32_t* status, void* stream) {
  if (!status) return moe::api_fail(MOE_ERR_INVALID, "operator_status: NULL pointer");
  int32_t* word = nullptr;
  const int rc = moe_operator_status_word(&word);
  if (rc != MOE_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(status, word, sizeof(int32_t), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess && clear) e = cudaMemsetAsync(word, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? MOE_OK : cuda_failed(e);
}

}  // extern "C"
