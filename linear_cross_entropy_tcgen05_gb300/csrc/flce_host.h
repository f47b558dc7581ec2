// flce_host.h -- host-side checks that the entry points outside flce_api.cu share with it
// (defined there). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/flce.h"

namespace flce {

// The current device, refused unless it is compute capability 10.3; binds its context.
flce_status api_device(int* sms, int* dev);
// FLCE_ERR_INVALID_ARG (with a detail naming the buffer) unless p is null or memory of device dev.
flce_status api_check_memory(int dev, const char* name, const void* p);
// Records what failed as the calling thread's error detail.
void api_note_error(const char* what, const char* why);
// FLCE_OK, or FLCE_ERR_CUDA with the detail recorded and the sticky error cleared.
flce_status api_cuda(const char* what, cudaError_t e);

inline bool api_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t api_align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace flce
