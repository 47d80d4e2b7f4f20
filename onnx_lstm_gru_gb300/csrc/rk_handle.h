// rk_handle.h -- the handle behind the C ABI and the host helpers that the
// translation units of its entry points share.  Not part of the ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "rk.h"
#include "rk_internal.h"

struct rk_handle {
  uint32_t flags = 0;
  std::string last_error;
  uint64_t launches = 0;
  long long timeout_ns = 2000000000LL;  // 2 s
  bool dev_ready = false;
  int device = -1;
  int sms = 152;
  int smem_optin = 232448;
  int* status = nullptr;
  // status word of the fixed array rk_encode_noalloc last used (device
  // address; null until that entry point has run on this handle)
  int* noalloc_status = nullptr;
  float* xw = nullptr;
  size_t xw_cap = 0;
  float* state = nullptr;
  size_t state_cap = 0;
  // scratch of the state space operators (scan chunks, gradients' partial sums)
  float* work = nullptr;
  size_t work_cap = 0;
  unsigned char* host_arena = nullptr;  // device buffers for rk_encode_host
  size_t host_arena_cap = 0;
  bool profiling = false;
  cudaEvent_t ev[4] = {nullptr, nullptr, nullptr, nullptr};  // proj start/end, step start/end
  bool ev_proj = false, ev_step = false;
  // rk_encode_host: a second stream copies X and the (pageable) operands only
  // the step kernel reads while the first copies W and runs the projection
  cudaStream_t copy_stream = nullptr;
  // fork from the caller's stream; join before the step; X copied (join before the projection)
  cudaEvent_t copy_ev[3] = {nullptr, nullptr, nullptr};
  bool can_map_host = false;  // the device can address page-locked host memory
  // Plans of the last problems encoded (the planner's occupancy queries cost
  // more host time than a small layer takes on the GPU)
  struct PlanEntry {
    bool valid = false;
    rk_problem key;
    uint32_t flags = 0;
    int device = -1;
    rk::StepParams sp;
    rk::StepPlan pl;
  };
  PlanEntry plans[4];
  int plan_next = 0;
};

namespace rk {

// Records the message of a failed call on the handle and returns its code.
inline rk_status fail(rk_handle* h, rk_status code, const char* fmt, ...) {
  if (h != nullptr) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    try {
      h->last_error = buf;
    } catch (...) {  // no memory for the message: the code alone reports the failure
    }
  }
  return code;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }
inline bool add_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_add_overflow(a, b, out); }
inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Takes the device of the handle's first encode: its SM count and limits,
// and the status word.
inline rk_status ensure_device(rk_handle* h) {
  if (h->dev_ready) return RK_OK;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, h->device);
  int map = 0;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&map, cudaDevAttrCanMapHostMemory, h->device);
  h->can_map_host = map != 0;
  if (e == cudaSuccess) e = cudaMalloc(&h->status, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, sizeof(int));
  if (e != cudaSuccess) return fail(h, RK_ERR_CUDA, "recurrent: device setup failed: %s", cudaGetErrorName(e));
  h->dev_ready = true;
  return RK_OK;
}

}  // namespace rk
