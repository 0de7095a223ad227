// Helpers of the extern "C" layers: error returns that never let an exception cross the ABI, and
// the checks several entry points share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <exception>
#include <new>
#include <stdexcept>
#include <string>
#include <utility>

#include "internal.h"

namespace mesh {

template <typename F>
int guarded_call(F&& f) {
  try {
    set_last_error(MESH_ATTN_OK, std::string());
    return f();
  } catch (const std::bad_alloc&) {
    return MESH_ATTN_ERR_NO_MEMORY;  // no message: building one could throw again
  } catch (const std::invalid_argument& e) {
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, e.what());
  } catch (const std::exception& e) {
    return set_last_error(MESH_ATTN_ERR_INTERNAL, e.what());
  } catch (...) {
    return set_last_error(MESH_ATTN_ERR_INTERNAL, "unknown exception");
  }
}

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// SMs of the current device, asked once per device (a constant of it).
inline cudaError_t current_sms(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev >= 0 && dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return e;
}

// Whether `what` still has to be done on the current device: a kernel's shared-memory limit is set once
// per device and kernel.  `mark` records that it was.
struct OncePerDevice {
  std::atomic<uint64_t> bits{0};
  static int device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 ? dev : -1;
  }
  bool pending(int dev) const { return dev < 0 || !(bits.load(std::memory_order_acquire) >> dev & 1); }
  void mark(int dev) {
    if (dev >= 0) bits.fetch_or((uint64_t)1 << dev, std::memory_order_release);
  }
};

// Launch of a kernel that begins with wait_for_kernel_before: its launch and set-up overlap the end of the
// kernel before it, 1 to 2 us where kernels are short.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, std::forward<A>(args)...);
}

// A launcher's result (a cudaError_t value and its message) as a status.
inline int launch_status(int ce, const std::string& err) {
  if (ce == (int)cudaSuccess) return MESH_ATTN_OK;
  return set_last_error(MESH_ATTN_ERR_CUDA, err.empty() ? cudaGetErrorString((cudaError_t)ce) : err);
}

}  // namespace mesh
