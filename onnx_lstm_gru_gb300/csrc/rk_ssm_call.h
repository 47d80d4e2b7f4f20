// rk_ssm_call.h -- one call of a state space operator as its host side sees
// it: the checks of its operands in 64-bit arithmetic and its scratch.  Not
// part of the ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "rk.h"
#include "rk_handle.h"
#include "rk_ssm.h"

namespace rk {

constexpr int64_t kMaxRows = 0x7fffffffLL;   // batch * seq, rows
constexpr int64_t kMaxSteps = 1LL << 30;     // seq, batch
constexpr int64_t kMaxInner = 1LL << 24;     // elements of a row

// One operator call: its name, handle and element size, and the checks of its
// operands.  A failed check records its message; the first one stands.
struct Call {
  rk_handle* h;
  const char* op;
  int eb;
  rk_status st = RK_OK;

  bool ok() const { return st == RK_OK; }
  template <typename... A>
  void bad(rk_status code, const char* fmt, A... a) {
    if (ok()) st = fail(h, code, fmt, op, a...);
  }
  // A size in [lo, hi].
  void size(const char* name, int64_t v, int64_t lo, int64_t hi) {
    if (!ok()) return;
    if (v < lo) bad(RK_ERR_SHAPE, "%s: %s: %lld out of range", name, (long long)v);
    else if (v > hi) bad(RK_ERR_UNSUPPORTED, "%s: %s: %lld exceeds %lld", name, (long long)v, (long long)hi);
  }
  void dtype(int32_t d) {
    if (ok() && d != RK_F32 && d != RK_F16 && d != RK_BF16) bad(RK_ERR_SHAPE, "%s: dtype: unknown value %d", d);
    eb = d == RK_F32 ? 4 : 2;
  }
  void layout(int32_t l) {
    if (ok() && l != 0 && l != 1) bad(RK_ERR_SHAPE, "%s: layout: must be 0 or 1, got %d", l);
  }
  // `count` elements from ptr + offset lie in the buffer; the address.
  template <typename P>
  P* range(const char* name, void* ptr, int64_t offset, int64_t length, int64_t count, int elem, bool required) {
    if (!ok()) return nullptr;
    if (ptr == nullptr) {
      if (required && count > 0) bad(RK_ERR_SHAPE, "%s: %s: required tensor is null", name);
      return nullptr;
    }
    int64_t end;
    if (offset < 0) {
      bad(RK_ERR_SHAPE, "%s: %s: negative offset %lld", name, (long long)offset);
    } else if (length < 0) {
      bad(RK_ERR_SHAPE, "%s: %s: negative length %lld", name, (long long)length);
    } else if (!add_ok(offset, count, &end)) {
      bad(RK_ERR_SHAPE, "%s: %s: offset %lld + extent %lld overflows", name, (long long)offset, (long long)count);
    } else if (end > length) {
      bad(RK_ERR_SHAPE, "%s: %s: offset %lld + extent %lld exceeds buffer length %lld", name, (long long)offset,
          (long long)count, (long long)length);
    } else if (reinterpret_cast<uintptr_t>(ptr) % elem != 0) {
      bad(RK_ERR_SHAPE, "%s: %s: address is not a multiple of its %d-byte elements", name, elem);
    }
    return ok() ? reinterpret_cast<P*>(static_cast<char*>(ptr) + offset * elem) : nullptr;
  }
  template <typename P>
  P* tensor(const char* name, const rk_tensor& t, int64_t count, int elem, bool required = false) {
    return range<P>(name, t.ptr, t.offset, t.length, count, elem, required);
  }
  // [outer][inner] rows of `elems` elements.  On return ss is the distance
  // along the outer index, ns along the inner one.
  RowsArg rows(const char* name, const rk_rows& t, int64_t outer, int64_t inner, int64_t elems, int group,
               bool required) {
    RowsArg a{};
    if (!ok()) return a;
    const int piece = 16 / eb;
    if (t.ptr == nullptr || outer == 0 || inner == 0) {
      a.p = range<void>(name, t.ptr, t.offset, t.length, 0, eb, required && outer > 0 && inner > 0);
      if (t.ptr == nullptr && required && outer > 0 && inner > 0) bad(RK_ERR_SHAPE, "%s: %s: required tensor is null", name);
      a.vec = group % piece == 0;  // no rows stand in the way of pieces, but their elements still have to divide
      return a;
    }
    const int64_t pitch = t.pitch == 0 ? elems : t.pitch;
    if (pitch < elems) {
      bad(RK_ERR_SHAPE, "%s: %s: pitch %lld is less than a row's %lld elements", name, (long long)t.pitch,
          (long long)elems);
      return a;
    }
    // the elements that one outer index spans, and one inner index
    int64_t by_inner, by_outer, step = t.outer_pitch, count;
    bool fits = mul_ok(inner - 1, pitch, &by_inner) && add_ok(by_inner, elems, &by_inner);
    if (fits && step == 0) fits = mul_ok(inner, pitch, &step);
    if (fits && outer > 1 && step < elems) {
      bad(RK_ERR_SHAPE, "%s: %s: outer_pitch %lld is less than a row's %lld elements", name, (long long)step,
          (long long)elems);
      return a;
    }
    if (outer == 1) step = 0;
    fits = fits && mul_ok(outer - 1, step, &by_outer) && add_ok(by_outer, elems, &by_outer) &&
           add_ok(by_outer, by_inner - elems, &count);
    if (!fits) {
      bad(RK_ERR_SHAPE, "%s: %s: pitch %lld, outer_pitch %lld: the extent overflows", name, (long long)t.pitch,
          (long long)t.outer_pitch);
      return a;
    }
    if (outer > 1 && inner > 1 && step < by_inner && pitch < by_outer) {
      bad(RK_ERR_SHAPE, "%s: %s: pitch %lld, outer_pitch %lld: rows overlap", name, (long long)pitch, (long long)step);
      return a;
    }
    a.p = range<void>(name, t.ptr, t.offset, t.length, count, eb, required);
    a.ss = step;
    a.ns = inner == 1 ? 0 : pitch;
    // 16-byte pieces: `group` consecutive elements, the ones that tiles are
    // cut from, hold whole pieces
    a.vec = reinterpret_cast<uintptr_t>(a.p) % 16 == 0 && a.ss % piece == 0 && a.ns % piece == 0 && group % piece == 0;
    return a;
  }
  // The same by (step, batch row) of a problem's layout.
  template <typename P>
  RowsArg steps(const char* name, const rk_rows& t, const P* p, int64_t elems, int group, bool required) {
    RowsArg a = rows(name, t, p->layout == 0 ? p->seq : p->batch, p->layout == 0 ? p->batch : p->seq, elems, group,
                     required);
    if (p->layout == 1) std::swap(a.ss, a.ns);
    return a;
  }
  // Likewise for pieces of m elements.
  static bool pieces(const RowsArg& a, int m, int eb, int group) {
    return a.p == nullptr || (reinterpret_cast<uintptr_t>(a.p) % (m * eb) == 0 && a.ss % m == 0 && a.ns % m == 0 &&
                              group % m == 0);
  }
  void cuda(const char* what, cudaError_t e) {
    if (!ok() || e == cudaSuccess) return;
    cudaGetLastError();
    bad(e == cudaErrorInvalidConfiguration ? RK_ERR_UNSUPPORTED : RK_ERR_CUDA, "%s: %s: %s (%s)", what,
        cudaGetErrorName(e), cudaGetErrorString(e));
  }
  // `need` floats of scratch: the caller's, or the handle's own.
  float* scratch(const rk_workspace* w, int64_t need, cudaStream_t stream) {
    if (!ok() || need == 0) return nullptr;
    if (w != nullptr && w->ptr != nullptr) {
      if (w->offset < 0 || w->offset > w->length || w->length - w->offset < need) {
        bad(RK_ERR_SHAPE, "%s: scratch: offset %lld + %lld floats exceeds length %lld", (long long)w->offset,
            (long long)need, (long long)w->length);
        return nullptr;
      }
      float* p = w->ptr + w->offset;
      if (reinterpret_cast<uintptr_t>(p) % 16 != 0) bad(RK_ERR_SHAPE, "%s: scratch: base + offset must be 16-byte aligned");
      return ok() ? p : nullptr;
    }
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cuda("capture query", cudaStreamIsCapturing(stream, &cap));
    if (ok() && cap != cudaStreamCaptureStatusNone)
      // a graph would keep the address of memory that a later call may free
      bad(RK_ERR_UNSUPPORTED, "%s: scratch: place it (%lld floats) to capture this call", (long long)need);
    if (!ok()) return nullptr;
    if (h->work_cap < (size_t)need) {
      if (h->work) {
        cuda("scratch", cudaDeviceSynchronize());
        if (!ok()) return nullptr;
        cudaFree(h->work);
        h->work = nullptr;
        h->work_cap = 0;
      }
      if (cudaMalloc(&h->work, (size_t)need * sizeof(float)) != cudaSuccess) {
        cudaGetLastError();
        h->work = nullptr;
        bad(RK_ERR_OOM, "%s: scratch: cannot allocate %lld floats", (long long)need);
        return nullptr;
      }
      h->work_cap = (size_t)need;
    }
    return h->work;
  }
  void zero(void* p, int64_t bytes, cudaStream_t s) {
    if (ok() && p != nullptr && bytes > 0) cuda("memset", cudaMemsetAsync(p, 0, (size_t)bytes, s));
  }
  // dst = src, or zeros without src.
  void copy(void* dst, const void* src, int64_t bytes, cudaStream_t s) {
    if (!ok() || dst == nullptr || dst == src || bytes == 0) return;
    if (src == nullptr) zero(dst, bytes, s);
    else cuda("copy", cudaMemcpyAsync(dst, src, (size_t)bytes, cudaMemcpyDeviceToDevice, s));
  }
};

inline bool aligned16(const void* p) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 == 0; }

inline Call begin(rk_handle* h, const char* op, const void* problem, const void* ops, bool need_ops) {
  Call c{h, op, 4};
  if (h != nullptr) h->last_error.clear();
  if (problem == nullptr) c.bad(RK_ERR_ARG, "%s: problem is null");
  else if (need_ops && ops == nullptr) c.bad(RK_ERR_ARG, "%s: operands: null");
  return c;
}

}  // namespace rk
