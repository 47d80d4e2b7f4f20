// rk_attn_api.cpp -- host side of the linear attention operators of
// include/rk.h: argument checks in 64-bit arithmetic, scratch, the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <utility>

#include "rk_attn.h"
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

constexpr int64_t kMaxQk = 256, kMaxHead = 128, kMaxHeads = 1LL << 24;

void check_rows(Call& c, int64_t seq, int64_t batch) {
  c.size("seq", seq, 0, kMaxSteps);
  c.size("batch", batch, 0, kMaxSteps);
  int64_t m;
  if (c.ok() && (!mul_ok(seq, batch, &m) || m > kMaxRows)) c.bad(RK_ERR_UNSUPPORTED, "%s: seq*batch exceeds 2^31 - 1");
}

void check_row(Call& c, const char* name, int64_t heads, int64_t size) {
  int64_t m;
  if (c.ok() && (!mul_ok(heads, size, &m) || m > kMaxInner))
    c.bad(RK_ERR_UNSUPPORTED, "%s: %s: %lld of %lld elements exceed a row of %lld", name, (long long)heads,
          (long long)size, (long long)kMaxInner);
}

void check(Call& c, const rk_qk_problem* p) {
  c.dtype(p->dtype);
  c.layout(p->layout);
  check_rows(c, p->seq, p->batch);
  c.size("heads", p->heads, 1, kMaxInner);
  c.size("key_heads", p->key_heads, 1, kMaxInner);
  c.size("size", p->size, 1, kMaxQk);
  check_row(c, "heads", p->heads, p->size);
  check_row(c, "key_heads", p->key_heads, p->size);
  if (c.ok() && (p->norm < 0 || p->norm > 2)) c.bad(RK_ERR_SHAPE, "%s: norm: unknown value %d", p->norm);
  if (c.ok() && p->interleaved != 0 && p->interleaved != 1)
    c.bad(RK_ERR_SHAPE, "%s: interleaved: must be 0 or 1, got %d", p->interleaved);
  if (c.ok() && (p->rotary < 0 || p->rotary % 2 != 0 || p->rotary > p->size))
    c.bad(RK_ERR_SHAPE, "%s: rotary: %d is not an even number of at most %lld elements", p->rotary, (long long)p->size);
  if (c.ok() && !(p->epsilon >= 0.0f)) c.bad(RK_ERR_SHAPE, "%s: epsilon: must be >= 0, got %g", (double)p->epsilon);
}

int shared(int64_t heads, int32_t given) { return given == 0 ? 1 : (int)(heads / given); }

void check(Call& c, const rk_attn_problem* p) {
  c.dtype(p->dtype);
  c.layout(p->layout);
  check_rows(c, p->seq, p->batch);
  c.size("heads", p->heads, 1, kMaxHeads);
  c.size("key_size", p->key_size, 1, kMaxHead);
  c.size("value_size", p->value_size, 1, kMaxHead);
  const std::pair<const char*, int32_t> some[] = {
      {"query_heads", p->query_heads}, {"key_heads", p->key_heads}, {"value_heads", p->value_heads}};
  for (const auto& s : some) {
    if (c.ok() && (s.second < 0 || (s.second > 0 && p->heads % s.second != 0)))
      c.bad(RK_ERR_SHAPE, "%s: %s: %d does not divide %lld heads", s.first, s.second, (long long)p->heads);
  }
  check_row(c, "heads", p->heads, std::max(p->key_size, p->value_size));
  int64_t m;
  if (c.ok() && (!mul_ok(p->batch, p->heads, &m) || m > kMaxHeads))
    c.bad(RK_ERR_UNSUPPORTED, "%s: batch*heads exceeds 2^24");
  if (c.ok() && !(p->scale - p->scale == 0.0f)) c.bad(RK_ERR_SHAPE, "%s: scale: must be finite, got %g", (double)p->scale);
}

// The operands that the queries' and keys' operator and its gradient share.
template <typename O>
rk::QkParams qk_params(Call& c, const rk_qk_problem* p, const O* o) {
  rk::QkParams q{};
  q.dtype = p->dtype, q.norm = p->norm, q.interleaved = p->interleaved, q.rotary = p->rotary, q.size = (int)p->size;
  q.epsilon = p->epsilon, q.S = (int)p->seq, q.N = (int)p->batch, q.layout = p->layout;
  q.side[0].heads = (int)p->heads, q.side[1].heads = (int)p->key_heads;
  q.side[0].X = c.steps("Q", o->Q, p, p->heads * p->size, 1, true);
  q.side[1].X = c.steps("K", o->K, p, p->key_heads * p->size, 1, true);
  q.side[0].scale = c.tensor<void>("QScale", o->QScale, p->size, c.eb);
  q.side[1].scale = c.tensor<void>("KScale", o->KScale, p->size, c.eb);
  q.freq = c.tensor<float>("Frequencies", o->Frequencies, p->rotary / 2, 4, true);
  q.positions = c.tensor<int>("positions", o->positions, p->seq * p->batch, 4);
  q.lens = c.tensor<int>("sequence_lens", o->sequence_lens, p->batch, 4);
  return q;
}

// The largest pieces that the sizes and every operand allow.
void qk_pieces(rk::QkParams& q, int eb) {
  q.piece = rk::qk_piece(eb, q.size, q.rotary, q.interleaved);
  for (; q.piece > 1; q.piece /= 2) {
    bool fits = true;
    for (const rk::QkSide& s : q.side) {
      for (const RowsArg* a : {&s.X, &s.Y, &s.dY, &s.dX}) fits = fits && Call::pieces(*a, q.piece, eb, q.size);
      fits = fits && reinterpret_cast<uintptr_t>(s.scale) % (q.piece * eb) == 0;
    }
    if (fits) return;
  }
}

// The float32 rows of the decays, or their gradient's.
RowsArg decay_rows(Call& c, const char* name, const rk_rows& t, const rk_attn_problem* p) {
  const int eb = c.eb;
  c.eb = 4;
  const RowsArg a = c.steps(name, t, p, p->heads, 1, false);
  c.eb = eb;
  return a;
}

// What a gradient needs: its passes' products for the decays, and float32
// outputs where heads share.
struct GradPlan {
  int64_t to, of, cross, partial, q32, k32, v32, between, marks, chunks;  // marks: of one pass
  int64_t total() const { return to + of + cross + partial + q32 + k32 + v32 + between + 2 * marks + chunks; }
};
rk::AttnPlan plan_of(const rk_attn_problem* p, int passes, bool bias = false) {
  return rk::attn_plan(p->seq, p->batch, p->heads, (int)p->key_size, (int)p->value_size, passes, bias);
}
int64_t plan_scratch(const rk_attn_problem* p, int passes) {
  if (p->seq * p->batch == 0 || (passes == 1 && p->seq <= rk::kAttnSteps)) return 0;
  return rk::attn_plan_scratch(plan_of(p, passes), p->batch, p->heads, (int)p->key_size, (int)p->value_size, passes);
}
// Its regions, from w on: states, and four floats for each.
void place(rk::AttnPlan& plan, float* w, int64_t floats) {
  const int64_t state = plan.deep * 128;
  plan.states = w;
  plan.left = w + floats / (state + 4) * state;
}
int64_t four(int64_t x) { return (x + 3) / 4 * 4; }
struct GradWants {
  bool q, k, v, decay, bias, first;
  bool has_bias;  // among the operands: dDecay is the same then whether the bias' gradient is wanted or not
  bool any() const { return q || k || v || decay || bias || first; }
};
constexpr GradWants kEverything = {true, true, true, true, true, true, true};
GradPlan grad_plan(const rk_attn_problem* p, const GradWants& want) {
  const int64_t heads = p->batch * p->heads, rows = heads * p->seq;
  GradPlan g{};
  if (rows == 0 || !want.any()) return g;
  // the pieces are those of the whole gradient whatever is wanted: equal bits
  const rk::AttnPlan plan = plan_of(p, 3, want.bias || want.has_bias);
  if (want.decay || want.bias) {
    g.to = g.of = four(rows);
    g.cross = four(2 * heads);
    if (want.bias) g.partial = four(2 * heads * rk::attn_decay_tiles(p->seq, plan.every));
    const int together = rk::attn_together((int)p->key_size, (int)p->value_size);
    g.between = four(heads * plan.marks);
    g.marks = p->batch * ((p->heads + together - 1) / together) * plan.marks * plan.deep * 128;
  }
  if (want.q && shared(p->heads, p->query_heads) > 1) g.q32 = four(rows * p->key_size);
  if (want.k && shared(p->heads, p->key_heads) > 1) g.k32 = four(rows * p->key_size);
  if (want.v && shared(p->heads, p->value_heads) > 1) g.v32 = four(rows * p->value_size);
  g.chunks = plan_scratch(p, 3);
  return g;
}

// Failed waits by device; devices past the last share its place.
std::mutex failures_lock;
uint64_t failures[rk_handle::kDevices];

int device_place() {
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess) cudaGetLastError();
  return std::min(std::max(d, 0), rk_handle::kDevices - 1);
}

}  // namespace

namespace rk {

void use_attn_waits(rk_handle* h) {
  auto& w = h->attn_waits[device_place()];
  if (w.used) return;
  std::lock_guard<std::mutex> lock(failures_lock);
  w.used = h->attn_used = true;
  w.seen = failures[&w - h->attn_waits];
}

cudaError_t poll_attn(rk_handle* h, cudaStream_t s, int* failed) {
  const int d = device_place();
  auto& w = h->attn_waits[d];
  *failed = 0;
  if (!w.used) return cudaSuccess;
  std::lock_guard<std::mutex> lock(failures_lock);
  int now = 0;
  const cudaError_t e = take_attn_status(s, &now);
  if (e != cudaSuccess) return e;
  failures[d] += now != 0;
  *failed = w.seen != failures[d];
  w.seen = failures[d];
  return e;
}

}  // namespace rk

extern "C" {

int64_t rk_qk_grad_scratch_length(const rk_qk_problem* p) {
  Call c = begin(nullptr, "QueryKeyGrad", p, nullptr, false);
  if (c.ok()) check(c, p);
  return c.ok() ? (int64_t)rk::qk_grad_blocks(p->seq * p->batch) * 2 * p->size : -1;
}

int64_t rk_attn_scratch_length(const rk_attn_problem* p) {
  Call c = begin(nullptr, "LinearAttention", p, nullptr, false);
  if (c.ok()) check(c, p);
  return c.ok() ? plan_scratch(p, 1) : -1;
}

int64_t rk_attn_grad_scratch_length(const rk_attn_problem* p) {
  Call c = begin(nullptr, "LinearAttentionGrad", p, nullptr, false);
  if (c.ok()) check(c, p);
  return c.ok() ? grad_plan(p, kEverything).total() : -1;
}

int64_t rk_attn_grad_scratch_needed(const rk_attn_problem* p, const rk_attn_grad_operands* o) {
  Call c = begin(nullptr, "LinearAttentionGrad", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return -1;
  const GradWants want = {o->dQ.ptr != nullptr,           o->dK.ptr != nullptr,
                          o->dV.ptr != nullptr,           o->dDecay.ptr != nullptr,
                          o->d_decay_bias.ptr != nullptr, o->d_initial_state.ptr != nullptr,
                          o->decay_bias.ptr != nullptr};
  return grad_plan(p, want).total();
}

rk_status rk_qk_encode(rk_handle* h, const rk_qk_problem* p, const rk_qk_operands* o, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "QueryKey", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  rk::QkParams q = qk_params(c, p, o);
  q.side[0].Y = c.steps("YQ", o->YQ, p, p->heads * p->size, 1, false);
  q.side[1].Y = c.steps("YK", o->YK, p, p->key_heads * p->size, 1, false);
  if (!c.ok() || p->seq * p->batch == 0 || (q.side[0].Y.p == nullptr && q.side[1].Y.p == nullptr)) return c.st;
  qk_pieces(q, c.eb);
  c.cuda("launch", rk::launch_qk(q, static_cast<cudaStream_t>(stream)));
  if (c.ok()) h->launches += 1;
  return c.st;
}

rk_status rk_qk_grad_encode(rk_handle* h, const rk_qk_problem* p, const rk_qk_grad_operands* o,
                            const rk_workspace* scratch, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "QueryKeyGrad", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rk::QkParams q = qk_params(c, p, o);
  q.side[0].dY = c.steps("dYQ", o->dYQ, p, p->heads * p->size, 1, true);
  q.side[1].dY = c.steps("dYK", o->dYK, p, p->key_heads * p->size, 1, true);
  q.side[0].dX = c.steps("dQ", o->dQ, p, p->heads * p->size, 1, false);
  q.side[1].dX = c.steps("dK", o->dK, p, p->key_heads * p->size, 1, false);
  q.side[0].dscale = c.tensor<float>("dQScale", o->dQScale, p->size, 4);
  q.side[1].dscale = c.tensor<float>("dKScale", o->dKScale, p->size, 4);
  bool wanted = false;
  for (const rk::QkSide& side : q.side) wanted = wanted || side.dX.p || side.dscale;
  if (!c.ok() || !wanted) return c.st;
  if (p->seq * p->batch == 0) {
    for (const rk::QkSide& side : q.side) c.zero(side.dscale, p->size * 4, s);
    return c.st;
  }
  q.blocks = rk::qk_grad_blocks(p->seq * p->batch);
  if (q.side[0].dscale || q.side[1].dscale) q.partial = c.scratch(scratch, (int64_t)q.blocks * 2 * p->size, s);
  if (!c.ok()) return c.st;
  qk_pieces(q, c.eb);
  int launches = 0;
  c.cuda("launch", rk::launch_qk_grad(q, s, &launches));
  h->launches += launches;
  return c.st;
}

rk_status rk_attn_encode(rk_handle* h, const rk_attn_problem* p, const rk_attn_operands* o,
                         const rk_workspace* scratch, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "LinearAttention", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t states = p->batch * p->heads * p->key_size * p->value_size;
  const int dk = (int)p->key_size, dv = (int)p->value_size;
  rk::AttnParams ap{};
  ap.dtype = p->dtype, ap.S = (int)p->seq, ap.N = (int)p->batch, ap.H = (int)p->heads, ap.passes = 1;
  rk::AttnPass& a = ap.pass[0];
  a.q_of = shared(p->heads, p->query_heads), a.k_of = shared(p->heads, p->key_heads);
  a.v_of = shared(p->heads, p->value_heads), a.o_of = 1;
  a.K = dk, a.V = dv, a.su = 1.0f, a.so = p->scale;
  a.q = c.steps("Q", o->Q, p, p->heads / a.q_of * dk, dk, true);
  a.k = c.steps("K", o->K, p, p->heads / a.k_of * dk, dk, true);
  a.v = c.steps("V", o->V, p, p->heads / a.v_of * dv, dv, true);
  ap.decay = decay_rows(c, "Decay", o->Decay, p);
  a.o = c.steps("Y", o->Y, p, p->heads * dv, dv, false);
  ap.bias = c.tensor<float>("decay_bias", o->decay_bias, p->heads, 4);
  ap.lens = c.tensor<int>("sequence_lens", o->sequence_lens, p->batch, 4);
  a.first = c.tensor<float>("initial_state", o->initial_state, states, 4);
  a.last = c.tensor<float>("final_state", o->final_state, states, 4);
  if (!c.ok() || (a.o.p == nullptr && a.last == nullptr)) return c.st;
  if (p->seq * p->batch == 0) {
    c.copy(a.last, a.first, states * 4, s);
    return c.st;
  }
  int launches = 0;
  if (p->seq <= rk::kAttnSteps) {
    c.cuda("launch", rk::launch_attn_steps(ap, s, &launches));
  } else {
    ap.plan = plan_of(p, 1);
    const int64_t need = plan_scratch(p, 1);
    place(ap.plan, c.scratch(scratch, need, s), need);
    ap.plan.vec = a.q.vec && a.k.vec && a.v.vec;
    if (c.ok()) rk::use_attn_waits(h);
    if (c.ok()) c.cuda("launch", rk::launch_attn_chunks(ap, s, &launches));
  }
  h->launches += launches;
  return c.st;
}

rk_status rk_attn_grad_encode(rk_handle* h, const rk_attn_problem* p, const rk_attn_grad_operands* o,
                              const rk_workspace* scratch, void* stream) {
  if (h == nullptr) return RK_ERR_ARG;
  Call c = begin(h, "LinearAttentionGrad", p, o, true);
  if (c.ok()) check(c, p);
  if (!c.ok()) return c.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t heads = p->batch * p->heads, states = heads * p->key_size * p->value_size;
  const int dk = (int)p->key_size, dv = (int)p->value_size, H = (int)p->heads;
  const int q_of = shared(H, p->query_heads), k_of = shared(H, p->key_heads), v_of = shared(H, p->value_heads);
  rk::AttnParams ap{};
  ap.dtype = p->dtype, ap.S = (int)p->seq, ap.N = (int)p->batch, ap.H = H, ap.gradient = 1;
  const RowsArg Q = c.steps("Q", o->Q, p, (int64_t)(H / q_of) * dk, dk, true);
  const RowsArg K = c.steps("K", o->K, p, (int64_t)(H / k_of) * dk, dk, true);
  const RowsArg V = c.steps("V", o->V, p, (int64_t)(H / v_of) * dv, dv, true);
  ap.decay = decay_rows(c, "Decay", o->Decay, p);
  const RowsArg dY = c.steps("dY", o->dY, p, (int64_t)H * dv, dv, true);
  const RowsArg dQ = c.steps("dQ", o->dQ, p, (int64_t)(H / q_of) * dk, dk, false);
  const RowsArg dK = c.steps("dK", o->dK, p, (int64_t)(H / k_of) * dk, dk, false);
  const RowsArg dV = c.steps("dV", o->dV, p, (int64_t)(H / v_of) * dv, dv, false);
  const RowsArg dDecay = decay_rows(c, "dDecay", o->dDecay, p);
  ap.bias = c.tensor<float>("decay_bias", o->decay_bias, H, 4);
  ap.lens = c.tensor<int>("sequence_lens", o->sequence_lens, p->batch, 4);
  const float* first = c.tensor<float>("initial_state", o->initial_state, states, 4);
  const float* dlast = c.tensor<float>("d_final_state", o->d_final_state, states, 4);
  float* dbias = c.tensor<float>("d_decay_bias", o->d_decay_bias, H, 4);
  float* dfirst = c.tensor<float>("d_initial_state", o->d_initial_state, states, 4);
  const GradWants want = {dQ.p != nullptr,  dK.p != nullptr,   dV.p != nullptr,   dDecay.p != nullptr,
                          dbias != nullptr, dfirst != nullptr, ap.bias != nullptr};
  if (!c.ok() || !want.any()) return c.st;
  if (p->seq * p->batch == 0) {
    c.zero(dbias, H * 4LL, s);
    c.copy(dfirst, dlast, states * 4, s);
    return c.st;
  }
  const GradPlan g = grad_plan(p, want);
  float* w = c.scratch(scratch, g.total(), s);
  if (!c.ok()) return c.st;
  const bool decays = dDecay.p || dbias;
  float *to = w, *of = to + g.to, *cross = of + g.of, *partial = cross + g.cross;
  float *q32 = partial + g.partial, *k32 = q32 + g.q32, *v32 = k32 + g.k32;
  float *between = v32 + g.v32, *marks = between + g.between;

  // dQ: the rows that wrote the state, read by dY
  auto next = [&]() -> rk::AttnPass& { return ap.pass[ap.passes++]; };
  if (dQ.p || decays) {
    rk::AttnPass& a = next();
    a.q = dY, a.k = V, a.v = K, a.o = dQ;
    a.q_of = 1, a.k_of = v_of, a.v_of = k_of, a.o_of = q_of;
    a.K = dv, a.V = dk, a.su = 1.0f, a.so = p->scale, a.v_major = 1;
    a.first = first;
    if (decays) a.dot = to, a.dot_with = Q;
    if (decays && g.marks) a.marks = marks;
    if (decays && dlast) a.with = dlast, a.cross = cross + heads;
    if (q_of > 1 && dQ.p) a.o32 = q32;
  }
  // dV: dY, written by the queries and read by the keys, backward
  if (dV.p || dfirst) {
    rk::AttnPass& a = next();
    a.q = K, a.k = Q, a.v = dY, a.o = dV;
    a.q_of = k_of, a.k_of = q_of, a.v_of = 1, a.o_of = v_of;
    a.K = dk, a.V = dv, a.su = p->scale, a.so = 1.0f, a.backward = 1;
    a.first = dlast, a.last = dfirst;
    if (v_of > 1 && dV.p) a.o32 = v32;
  }
  // dK: the queries, written by dY and read by the values, backward
  if (dK.p || decays) {
    rk::AttnPass& a = next();
    a.q = V, a.k = dY, a.v = Q, a.o = dK;
    a.q_of = v_of, a.k_of = 1, a.v_of = q_of, a.o_of = k_of;
    a.K = dv, a.V = dk, a.su = p->scale, a.so = 1.0f, a.backward = 1, a.v_major = 1;
    a.first = dlast;
    if (decays) a.dot = of, a.dot_with = K;
    if (decays && g.marks) a.marks = marks + g.marks;
    if (decays && first) a.with = first, a.cross = cross;
    if (k_of > 1 && dK.p) a.o32 = k32;
  }
  int launches = 0;
  if (ap.passes) {
    ap.plan = plan_of(p, 3, want.bias || want.has_bias);
    place(ap.plan, marks + 2 * g.marks, g.chunks);
    ap.plan.vec = Q.vec && K.vec && V.vec && dY.vec;
    rk::use_attn_waits(h);
    c.cuda("launch", rk::launch_attn_chunks(ap, s, &launches));
  }
  if (c.ok() && decays) {
    rk::AttnDecayParams d{};
    d.S = ap.S, d.N = ap.N, d.H = H, d.lens = ap.lens;
    d.decay = ap.decay, d.bias = ap.bias, d.dDecay = dDecay;
    d.to = to, d.of = of, d.dbias = dbias;
    d.first = first ? cross : nullptr, d.last = dlast ? cross + heads : nullptr;
    d.states = marks, d.between = between, d.deep = ap.plan.deep;
    d.every = ap.plan.every, d.marks = ap.plan.marks;
    d.together = rk::attn_together(dk, dv);
    d.partial = dbias ? reinterpret_cast<double*>(partial) : nullptr;
    c.cuda("launch", rk::launch_attn_decay(d, s, &launches));
  }
  rk::AttnShareParams sp{p->dtype, ap.S, ap.N, H};
  auto share = [&](const RowsArg& out, const float* o32, int V_, int n) {
    if (n > 1 && out.p) sp.out[sp.count++] = {V_, n, o32, out};
  };
  share(dQ, q32, dk, q_of);
  share(dK, k32, dk, k_of);
  share(dV, v32, dv, v_of);
  if (c.ok() && sp.count) c.cuda("launch", rk::launch_attn_share(sp, s, &launches));
  h->launches += launches;
  return c.st;
}

}  // extern "C"
