// Helpers of the extern "C" layers: error returns that never let an exception cross the ABI, and
// the checks several entry points share.
#pragma once

#include <cuda_runtime.h>

#include <exception>
#include <new>
#include <stdexcept>
#include <string>

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

// A launcher's result (a cudaError_t value and its message) as a status.
inline int launch_status(int ce, const std::string& err) {
  if (ce == (int)cudaSuccess) return MESH_ATTN_OK;
  return set_last_error(MESH_ATTN_ERR_CUDA, err.empty() ? cudaGetErrorString((cudaError_t)ce) : err);
}

}  // namespace mesh
