// rk_ssm_api.cpp -- host side of the state space operators of include/rk.h:
// argument checks in 64-bit arithmetic, scratch, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <utility>

#include "rk.h"
#include "rk_handle.h"
#include "rk_ssm.h"

namespace {

using rk::add_ok;
using rk::fail;
using rk::mul_ok;
using rk::RowsArg;

constexpr int64_t kMaxRows = 0x7fffffffLL;   // batch * seq, rows
constexpr int64_t kMaxSteps = 1LL << 30;     // seq, batch
constexpr int64_t kMaxInner = 1LL << 24;     // elements of a row
constexpr int64_t kMaxState = 128;
constexpr int64_t kMaxWidth = 8;

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

bool aligned16(const void* p) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 == 0; }

Call begin(rk_handle* h, const char* op, const void* problem, const void* ops, bool need_ops) {
  Call c{h, op, 4};
  if (h != nullptr) h->last_error.clear();
  if (problem == nullptr) c.bad(RK_ERR_ARG, "%s: problem is null");
  else if (need_ops && ops == nullptr) c.bad(RK_ERR_ARG, "%s: operands: null");
  return c;
}

void check(Call& c, const rk_norm_problem* p) {
  c.dtype(p->dtype);
  if (c.ok() && !(p->epsilon >= 0.0f)) c.bad(RK_ERR_SHAPE, "%s: epsilon: must be >= 0, got %g", (double)p->epsilon);
  c.size("rows", p->rows, 0, kMaxRows);
  c.size("cols", p->cols, 1, kMaxInner);
}

void check_steps(Call& c, int64_t seq, int64_t batch, int64_t channels) {
  c.size("seq", seq, 0, kMaxSteps);
  c.size("batch", batch, 0, kMaxSteps);
  c.size("channels", channels, 1, kMaxInner);
  int64_t m;
  if (c.ok() && (!mul_ok(seq, batch, &m) || m > kMaxRows)) c.bad(RK_ERR_UNSUPPORTED, "%s: seq*batch exceeds 2^31 - 1");
}

void check(Call& c, const rk_conv_problem* p) {
  c.dtype(p->dtype);
  c.layout(p->layout);
  check_steps(c, p->seq, p->batch, p->channels);
  c.size("width", p->width, 1, kMaxWidth);
  if (c.ok() && p->activation != 0 && p->activation != 1)
    c.bad(RK_ERR_SHAPE, "%s: activation: unknown value %d", p->activation);
}

void check(Call& c, const rk_scan_problem* p) {
  c.dtype(p->dtype);
  c.layout(p->layout);
  check_steps(c, p->seq, p->batch, p->channels);
  c.size("state", p->state, 1, kMaxState);
  c.size("groups", p->groups, 1, kMaxInner);
  if (c.ok() && p->channels % p->groups != 0)
    c.bad(RK_ERR_SHAPE, "%s: groups: %d does not divide %lld channels", p->groups, (long long)p->channels);
  if (c.ok() && p->groups * p->state > kMaxInner)
    c.bad(RK_ERR_UNSUPPORTED, "%s: groups*state: %lld exceeds %lld", (long long)(p->groups * p->state),
          (long long)kMaxInner);
  if (c.ok() && p->softplus != 0 && p->softplus != 1)
    c.bad(RK_ERR_SHAPE, "%s: softplus: must be 0 or 1, got %d", p->softplus);
}

// The normalisation's rows, `ss` apart.
RowsArg norm_rows(Call& c, const char* name, const rk_rows& t, const rk_norm_problem* p, bool required) {
  rk_rows one = t;
  one.outer_pitch = 0;
  RowsArg a = c.rows(name, one, 1, p->rows, p->cols, (int)p->cols, required);
  std::swap(a.ss, a.ns);
  return a;
}

int64_t norm_scratch(const rk_norm_problem* p) {
  return (int64_t)rk::norm_grad_blocks(p->rows, (int)p->cols) * 2 * p->cols;
}
int64_t conv_scratch(const rk_conv_problem* p) {
  return (int64_t)rk::conv_grad_slices(p->seq, p->batch, p->channels) * (p->width + 1) * p->channels;
}
// What a call takes with row lengths or without them.
template <typename PLAN>
int64_t scan_scratch(PLAN plan, const rk_scan_problem* p) {
  auto total = [&](bool ragged) {
    return (int64_t)plan(p->seq, p->batch, p->channels, (int)p->state, (int)p->groups, ragged).total();
  };
  return std::max(total(false), total(true));
}

// The operands that the scan and its gradient share.
template <typename O>
rk::ScanParams scan_params(Call& c, const rk_scan_problem* p, const O* o) {
  rk::ScanParams sp{};
  const int per = (int)(p->channels / p->groups), K = (int)p->state;
  const int64_t states = p->batch * p->channels;  // <= 2^54
  sp.dtype = p->dtype, sp.softplus = p->softplus;
  sp.S = (int)p->seq, sp.N = (int)p->batch, sp.C = (int)p->channels, sp.K = K, sp.G = (int)p->groups;
  sp.X = c.steps("X", o->X, p, p->channels, per, true);
  sp.Delta = c.steps("Delta", o->Delta, p, p->channels, per, true);
  sp.Bm = c.steps("B", o->B, p, (int64_t)p->groups * K, K, true);
  sp.Cm = c.steps("C", o->C, p, (int64_t)p->groups * K, K, true);
  sp.Z = c.steps("Z", o->Z, p, p->channels, per, false);
  sp.A = c.tensor<float>("A", o->A, p->channels * K, 4, true);
  sp.D = c.tensor<float>("D", o->D, p->channels, 4);
  sp.bias = c.tensor<float>("delta_bias", o->delta_bias, p->channels, 4);
  sp.lens = c.tensor<int>("sequence_lens", o->sequence_lens, p->batch, 4);
  sp.h0 = c.tensor<float>("initial_state", o->initial_state, states * K, 4);
  sp.k_vec = K % 4 == 0 && aligned16(sp.A) && aligned16(sp.h0);
  sp.bc_vec = Call::pieces(sp.Bm, 4, c.eb, K) && Call::pieces(sp.Cm, 4, c.eb, K);
  return sp;
}

}  // namespace

extern "C" {

int64_t rk_norm_grad_scratch_length(const rk_norm_problem* p) {
  Call c = begin(nullptr, "LayerNormalizationGrad", p, nullptr, false);
  if (c.ok()) check(c, p);
  return c.ok() ? norm_scratch(p) : -1;
}

int64_t rk_conv_grad_scratch_length(const rk_conv_problem* p) {
  Call c = begin(nullptr, "CausalConvGrad", p, nullptr, false);
  if (c.ok()) check(c, p);
  return c.ok() ? conv_scratch(p) : -1;
}

int64_t rk_scan_scratch_length(const rk_scan_problem* p) {
  Call c = begin(nullptr, "SelectiveScan", p, nullptr, false);
  if (c.ok()) check(c, p);
  return c.ok() ? scan_scratch(rk::scan_plan, p) : -1;
}

int64_t rk_scan_grad_scratch_length(const rk_scan_problem* p) {
  Call c = begin(nullptr, "SelectiveScanGrad", p, nullptr, false);
  if (c.ok()) check(c, p);
  return c.ok() ? scan_scratch(rk::scan_grad_plan, p) : -1;
}

rk_status rk_norm_encode(rk_handle* h, const rk_norm_problem* p, const rk_norm_operands* o, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "LayerNormalization", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  rk::NormParams np{};
  const int cols = (int)p->cols;
  np.dtype = p->dtype, np.epsilon = p->epsilon, np.rows = p->rows, np.cols = cols;
  np.X = norm_rows(c, "X", o->X, p, true);
  np.Y = norm_rows(c, "Y", o->Y, p, false);
  np.scale = c.tensor<void>("Scale", o->Scale, cols, c.eb);
  np.bias = c.tensor<void>("B", o->B, cols, c.eb);
  np.mean = c.tensor<float>("Mean", o->Mean, p->rows, 4);
  np.inv = c.tensor<float>("InvStdDev", o->InvStdDev, p->rows, 4);
  if (!c.ok() || p->rows == 0) return c.st;
  np.vec = np.X.vec && np.Y.vec && aligned16(np.scale) && aligned16(np.bias);
  c.cuda("launch", rk::launch_norm(np, static_cast<cudaStream_t>(stream)));
  if (c.ok()) h->launches += 1;
  return c.st;
}

rk_status rk_norm_grad_encode(rk_handle* h, const rk_norm_problem* p, const rk_norm_grad_operands* o,
                              const rk_workspace* scratch, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "LayerNormalizationGrad", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rk::NormParams np{};
  const int cols = (int)p->cols;
  np.dtype = p->dtype, np.epsilon = p->epsilon, np.rows = p->rows, np.cols = cols;
  np.X = norm_rows(c, "X", o->X, p, true);
  np.dY = norm_rows(c, "dY", o->dY, p, true);
  np.dX = norm_rows(c, "dX", o->dX, p, false);
  np.scale = c.tensor<void>("Scale", o->Scale, cols, c.eb);
  np.mean_in = c.tensor<float>("Mean", o->Mean, p->rows, 4, true);
  np.inv_in = c.tensor<float>("InvStdDev", o->InvStdDev, p->rows, 4, true);
  np.dscale = c.tensor<float>("dScale", o->dScale, cols, 4);
  np.dbias = c.tensor<float>("dB", o->dB, cols, 4);
  if (!c.ok()) return c.st;
  if (p->rows == 0) {
    c.zero(np.dscale, cols * 4LL, s);
    c.zero(np.dbias, cols * 4LL, s);
    return c.st;
  }
  if (np.dscale || np.dbias) np.partial = c.scratch(scratch, norm_scratch(p), s);
  if (!c.ok()) return c.st;
  np.blocks = rk::norm_grad_blocks(p->rows, cols);
  np.vec = np.X.vec && np.dY.vec && np.dX.vec && aligned16(np.scale);
  int launches = 0;
  c.cuda("launch", rk::launch_norm_grad(np, s, &launches));
  h->launches += launches;
  return c.st;
}

rk_status rk_conv_encode(rk_handle* h, const rk_conv_problem* p, const rk_conv_operands* o, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "CausalConv", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  rk::ConvParams cp{};
  const int64_t state = p->batch * p->channels * (p->width - 1);
  const int C = (int)p->channels;
  cp.dtype = p->dtype, cp.width = p->width, cp.silu = p->activation;
  cp.S = (int)p->seq, cp.N = (int)p->batch, cp.C = C;
  cp.X = c.steps("X", o->X, p, C, C, true);
  cp.Y = c.steps("Y", o->Y, p, C, C, false);
  cp.W = c.tensor<void>("W", o->W, (int64_t)C * p->width, c.eb, true);
  cp.B = c.tensor<void>("B", o->B, C, c.eb);
  cp.lens = c.tensor<int>("sequence_lens", o->sequence_lens, p->batch, 4);
  cp.init = c.tensor<void>("initial_state", o->initial_state, state, c.eb);
  cp.final_state = c.tensor<void>("final_state", o->final_state, state, c.eb);
  if (!c.ok() || p->batch == 0) return c.st;
  if (p->seq == 0) {
    c.copy(cp.final_state, cp.init, state * c.eb, static_cast<cudaStream_t>(stream));
    return c.st;
  }
  cp.vec = cp.X.vec && cp.Y.vec && aligned16(cp.W) && aligned16(cp.B) && aligned16(cp.init) && aligned16(cp.final_state);
  c.cuda("launch", rk::launch_conv(cp, static_cast<cudaStream_t>(stream)));
  if (c.ok()) h->launches += 1;
  return c.st;
}

rk_status rk_conv_grad_encode(rk_handle* h, const rk_conv_problem* p, const rk_conv_grad_operands* o,
                              const rk_workspace* scratch, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "CausalConvGrad", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rk::ConvParams cp{};
  const int64_t rows = p->seq * p->batch, state = p->batch * p->channels * (p->width - 1);
  const int C = (int)p->channels;
  cp.dtype = p->dtype, cp.width = p->width, cp.silu = p->activation;
  cp.S = (int)p->seq, cp.N = (int)p->batch, cp.C = C;
  cp.X = c.steps("X", o->X, p, C, C, true);
  cp.dY = c.steps("dY", o->dY, p, C, C, true);
  cp.dX = c.steps("dX", o->dX, p, C, C, false);
  cp.W = c.tensor<void>("W", o->W, (int64_t)C * p->width, c.eb, true);
  cp.B = c.tensor<void>("B", o->B, C, c.eb);
  cp.lens = c.tensor<int>("sequence_lens", o->sequence_lens, p->batch, 4);
  cp.init = c.tensor<void>("initial_state", o->initial_state, state, c.eb);
  cp.dfinal = c.tensor<void>("d_final_state", o->d_final_state, state, c.eb);
  cp.dW = c.tensor<float>("dW", o->dW, (int64_t)C * p->width, 4);
  cp.dB = c.tensor<float>("dB", o->dB, C, 4);
  cp.dinit = c.tensor<void>("d_initial_state", o->d_initial_state, state, c.eb);
  if (!c.ok()) return c.st;
  if (rows == 0) {
    c.zero(cp.dW, (int64_t)C * p->width * 4, s);
    c.zero(cp.dB, C * 4LL, s);
    c.copy(cp.dinit, cp.dfinal, state * c.eb, s);
    return c.st;
  }
  if (cp.dW || cp.dB) cp.partial = c.scratch(scratch, conv_scratch(p), s);
  if (!c.ok()) return c.st;
  cp.chunk = rk::conv_grad_chunk(p->seq, p->batch, p->channels);
  cp.slices = rk::conv_grad_slices(p->seq, p->batch, p->channels);
  cp.vec = cp.X.vec && cp.dY.vec && cp.dX.vec && aligned16(cp.W) && aligned16(cp.B) && aligned16(cp.init) && aligned16(cp.dfinal) &&
           aligned16(cp.dinit);
  int launches = 0;
  c.cuda("launch", rk::launch_conv_grad(cp, s, &launches));
  h->launches += launches;
  return c.st;
}

rk_status rk_scan_encode(rk_handle* h, const rk_scan_problem* p, const rk_scan_operands* o,
                         const rk_workspace* scratch, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "SelectiveScan", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = p->seq * p->batch, states = p->batch * p->channels * p->state;
  rk::ScanParams sp = scan_params(c, p, o);
  sp.Y = c.steps("Y", o->Y, p, p->channels, (int)(p->channels / p->groups), false);
  sp.hT = c.tensor<float>("final_state", o->final_state, states, 4);
  sp.k_vec = sp.k_vec && aligned16(sp.hT);
  if (!c.ok()) return c.st;
  if (rows == 0) {
    c.copy(sp.hT, sp.h0, states * 4, s);
    return c.st;
  }
  const rk::ScanPlan pl = rk::scan_plan(p->seq, p->batch, p->channels, sp.K, sp.G, sp.lens != nullptr);
  float* w = c.scratch(scratch, scan_scratch(rk::scan_plan, p), s);
  if (!c.ok()) return c.st;
  sp.chunks = pl.chunks, sp.chunk = pl.chunk;
  sp.carry = w;
  sp.sumdt = w + pl.carry;
  int launches = 0;
  c.cuda("launch", rk::launch_scan(sp, s, &launches));
  h->launches += launches;
  return c.st;
}

rk_status rk_scan_grad_encode(rk_handle* h, const rk_scan_problem* p, const rk_scan_grad_operands* o,
                              const rk_workspace* scratch, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "SelectiveScanGrad", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = p->seq * p->batch, states = p->batch * p->channels * p->state, ck = p->channels * p->state;
  rk::ScanParams sp = scan_params(c, p, o);
  const int per = (int)(p->channels / p->groups);
  sp.dY = c.steps("dY", o->dY, p, p->channels, per, true);
  sp.dX = c.steps("dX", o->dX, p, p->channels, per, false);
  sp.dDelta = c.steps("dDelta", o->dDelta, p, p->channels, per, false);
  sp.dB = c.steps("dB", o->dB, p, (int64_t)p->groups * sp.K, sp.K, false);
  sp.dC = c.steps("dC", o->dC, p, (int64_t)p->groups * sp.K, sp.K, false);
  sp.dZ = c.steps("dZ", o->dZ, p, p->channels, per, false);
  if (c.ok() && sp.dZ.p && !sp.Z.p) c.bad(RK_ERR_SHAPE, "%s: dZ: exists only with Z");
  sp.dhT = c.tensor<float>("d_final_state", o->d_final_state, states, 4);
  sp.dA = c.tensor<float>("dA", o->dA, ck, 4);
  sp.dD = c.tensor<float>("dD", o->dD, p->channels, 4);
  sp.dbias = c.tensor<float>("d_delta_bias", o->d_delta_bias, p->channels, 4);
  sp.dh0 = c.tensor<float>("d_initial_state", o->d_initial_state, states, 4);
  sp.k_vec = sp.k_vec && aligned16(sp.dhT) && aligned16(sp.dh0);
  sp.vec = sp.X.vec && sp.Delta.vec && sp.Z.vec && sp.dY.vec && sp.dX.vec && sp.dDelta.vec && sp.dZ.vec;
  if (!c.ok()) return c.st;
  if (rows == 0) {
    c.zero(sp.dA, ck * 4, s);
    c.zero(sp.dD, p->channels * 4, s);
    c.zero(sp.dbias, p->channels * 4, s);
    c.copy(sp.dh0, sp.dhT, states * 4, s);
    return c.st;
  }
  const rk::ScanPlan pl = rk::scan_grad_plan(p->seq, p->batch, p->channels, sp.K, sp.G, sp.lens != nullptr);
  float* w = c.scratch(scratch, scan_scratch(rk::scan_grad_plan, p), s);
  if (!c.ok()) return c.st;
  sp.chunks = pl.chunks, sp.chunk = pl.chunk, sp.slices = pl.slices, sp.slice_tiles = pl.slice_tiles;
  sp.carry = w, w += pl.carry;
  sp.sumdt = w, w += pl.sumdt;
  sp.gcarry = w, w += pl.gcarry;
  sp.ckpt = w, w += pl.ckpt;
  sp.cum = w, w += pl.cum;
  sp.bc_part = (sp.dB.p || sp.dC.p) ? w : nullptr, w += pl.bc_part;
  sp.w_part = (sp.dA || sp.dD || sp.dbias) ? w : nullptr;
  int launches = 0;
  c.cuda("launch", rk::launch_scan_grad(sp, s, &launches));
  h->launches += launches;
  return c.st;
}

}  // extern "C"
