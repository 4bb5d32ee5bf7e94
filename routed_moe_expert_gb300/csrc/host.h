// What the C-ABI sources share on the host: the handle, error reporting and pointer checks.
#pragma once

#include "../../include/moe_lora.h"
#include "kernels.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct moe_lora_handle {
  int device = 0;
  int num_sms = 0;
  cudaStream_t side = nullptr;
  cudaEvent_t ev_fork = nullptr, ev_ready = nullptr;
  EncodeTiledFn encode = nullptr;
  int coop_ctas[mlk::kMaxExperts + 1];   // cache of route_max_coop_ctas by E (0 = unknown)
  uint64_t launches = 0;                  // kernels launched through this handle
  int2* linear_flags = nullptr;            // flags of the projection kernels, zero between calls; behind them those
                                          // of the attention kernels
  bool linear_ready = false;              // the projection kernels have their shared memory limits
  bool attention_ready = false;           // the attention kernels have theirs
  int linear_pairs_by_two = 0;            // LinearMachine's, after that
};

namespace mlk {

// Records `err` as the calling thread's last CUDA error and returns MOE_LORA_ERR_CUDA.
moe_lora_status cuda_fail(cudaError_t err, const char* what);

// Makes the handle's device current for a call, and the caller's again after it.
class OnDevice {
 public:
  explicit OnDevice(const moe_lora_handle* h) {
    err_ = cudaGetDevice(&before_);
    if (err_ != cudaSuccess || before_ == h->device) return;
    err_ = cudaSetDevice(h->device);
    set_ = err_ == cudaSuccess;
  }
  ~OnDevice() {
    if (set_) cudaSetDevice(before_);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;
  cudaError_t error() const { return err_; }

 private:
  int before_ = 0;
  bool set_ = false;
  cudaError_t err_ = cudaSuccess;
};

// Tokens, rows and columns that the operators around the layer take: indices of whole tiles stay in 32 bits.
constexpr int kMaxExtent = 0x7fffffff - 255;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

}  // namespace mlk

#define ML_CUDA(call, what)                                  \
  do {                                                       \
    cudaError_t _e = (call);                                 \
    if (_e != cudaSuccess) return mlk::cuda_fail(_e, what);  \
  } while (0)

// From here to the end of the call on the handle's device.
#define ML_ON_DEVICE(h)              \
  const mlk::OnDevice on_device(h);  \
  ML_CUDA(on_device.error(), "cudaSetDevice")

// A launch of one of this library's kernels, counted on the handle (moe_lora_launch_count).
#define ML_LAUNCH(h, call, what)                    \
  do {                                              \
    ML_CUDA(call, what);                            \
    ++(h)->launches;                                \
  } while (0)
