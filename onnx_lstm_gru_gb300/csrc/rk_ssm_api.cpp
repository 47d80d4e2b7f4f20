// rk_ssm_api.cpp -- host side of the state space operators of include/rk.h:
// argument checks in 64-bit arithmetic, scratch, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <utility>

#include "rk_ssm_call.h"

namespace {

using rk::aligned16;
using rk::begin;
using rk::Call;
using rk::kMaxInner;
using rk::kMaxRows;
using rk::kMaxSteps;
using rk::mul_ok;
using rk::RowsArg;

constexpr int64_t kMaxState = 128;
constexpr int64_t kMaxWidth = 8;

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
