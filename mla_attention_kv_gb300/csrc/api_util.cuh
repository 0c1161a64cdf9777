// api_util.cuh -- host helpers shared by the C-ABI files of the attention and
// the e4m3 operators.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/mla_prolog.h"
#include "internal.h"

namespace {

using mla::set_error_text;

// Reports an error and takes it from the runtime, so that the next launch that
// asks does not find it.
mla_status fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  char text[256];
  snprintf(text, sizeof(text), "%s: %s (%d)", what, cudaGetErrorString(e), (int)e);
  set_error_text(text);
  return MLA_ERR_CUDA;
}

// Most rows, columns or blocks: from here on the kernels' sums of a count and a
// step could leave 32 bits.
constexpr int kMostCount = 0x7fff0000;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Reads and clears the status word in one step (the second word keeps what was
// read): calls that overlap on another stream may set bits meanwhile.
__global__ void take_status_kernel(unsigned* status) { status[1] = atomicExch(status, 0u); }

// Synchronise the stream, read and clear the status word.
cudaError_t take_status(unsigned* status, unsigned* value, cudaStream_t stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  take_status_kernel<<<1, 1, 0, stream>>>(status);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpyAsync(value, status + 1, sizeof(unsigned), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

// Makes the handle's device current for the length of a call.
struct DeviceGuard {
  int before = -1;
  cudaError_t err;
  explicit DeviceGuard(int device) {
    err = cudaGetDevice(&before);
    if (err == cudaSuccess && before != device)
      err = cudaSetDevice(device);
    else
      before = -1;
  }
  ~DeviceGuard() {
    if (before >= 0) cudaSetDevice(before);
  }
};

}  // namespace
