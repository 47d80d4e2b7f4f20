// rk_scan_grad.cu -- the gradient of the selective scan.
//
// With e the state's gradient on its way back, step s from the last to the
// first does, per channel and state,
//   g = e + C dy;  dC += dy h;  dB += (dt u) g;  du += dt B g;
//   x = g a h_before;  ddt += A x + u B g;  dA += dt x;  e = a g.
// It needs the states in reverse order.  They are computed again rather than
// kept: a launch forward (scan_grad_states_kernel) leaves the state, and the
// sum of dt since the chunk's start, at every eighth step (counted from the
// last one back, first_subtile) in global memory, and
// the way back (scan_grad_kernel) runs one such subtile at a time, forward and
// then back.  Of the bytes per element that the gradient reads and writes there
// are 4 / 8 per state for that, twice.
//
// A thread holds four states of two neighbouring channels, TPC threads a pair
// of channels: what a step loads from shared memory serves two channels, and
// dB and dC, sums over the channels of a group, are half added up before they
// leave the registers.  Four steps' states are in registers at once: the
// subtile's later half is run first, from the checkpoint through the earlier
// half, which is then computed again.  All eight in registers leave no room to
// overlap steps (the compiler spills); eight in shared memory measured
// slower, and so did 16 states of one channel per thread, two blocks per SM
// (546 us against 357 for the case below: 31 exchanges instead of 7 for dB and
// dC of a step, 8 warps per SM instead of 16).
// The sums over states (for du and ddt) and over a warp's channels (for dB and
// dC) halve the values with each exchange of halves between lanes, so eight
// values over eight lanes take seven shuffles.  Over a block's warps dB and dC
// are added in shared memory, over the blocks in a second launch that adds
// their slices in order.  dA, dD and d_delta_bias are sums over steps and
// sequences, kept per block and added the same way.
//
// Chunks of one sequence that run side by side are joined as in the forward
// scan; e is linear in what arrives at a chunk's end with the same factor
// exp(A sum dt), so one launch prepares both directions.
//
// Bound by instructions: 39 per step, channel and state on the way back, half
// of them the formulas above (2.5 decays, each an exponential, among them) and
// half exchanges, shared memory and what belongs to a channel's step.
// 512 steps x 8 sequences x 2048 channels x 16 states, bf16 with a gate: 353 us
// in all, of which forward 87 us, chunks' carry 14, back 243 (2.2 instructions
// per clock and SM, 16 warps), rows 10, weights 4; the bytes alone would take
// 18 us, the exponentials of two passes 29.
#include <algorithm>
#include <type_traits>

#include "rk.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kT = 8;  // steps of a subtile
constexpr int kHalf = 4;   // of them whose states are in registers at once

constexpr int tpc_of(int states) {
  return states <= 8 ? 2 : states <= 16 ? 4 : states <= 32 ? 8 : states <= 64 ? 16 : 32;
}

// A block's shared memory.  Rows are steps of the subtile; channel 2 j + e of
// the tile has place e * P + j.
template <typename T, int TPC>
struct GradSmem {
  static constexpr int P = kThreads / TPC, CH = 2 * P, NSP = 4 * TPC;
  static constexpr int kPieces = kT * CH * (int)sizeof(T) / 16;  // 16-byte pieces of a row tensor's subtile
  static constexpr int kQuads = kT * NSP / 4;                    // of B's or C's
  using Quad = std::conditional_t<sizeof(T) == 4, float4, uint2>;
  float4 dtu[kT][CH];   // dt, dt, dt u, dt u: packed operands
  float2 dy[kT][CH];    // dy, dy: past the gate
  float u[kT][CH];
  float slope[kT][CH];  // of softplus
  float gate[kT][CH];   // dY times the gate's slope
  float y[kT][CH];      // sum of C h
  float gb[kT][CH];     // sum of g B
  float th[kT][CH];     // sum of x A, in base-2 rates
  float B[kT][NSP], C[kT][NSP];
  float part[kT][kWarps][2 * NSP];  // the warps' sums of dB and dC
  float acc[kThreads][4];
  uint4 raw[4][kPieces];  // the next subtile's Delta, X, dY and Z as stored, rows of CH elements
  uint4 out[3][kPieces];  // this one's dX, dDelta and dZ
  Quad quads[2][kQuads];  // the next one's B and C
  float bias[CH], skip[CH];
};

// Two neighbouring elements of a row.
template <typename T>
struct Duo {
  T v[2];
  __device__ __forceinline__ void load(const RowsArg& a, int n, int s, int c, bool second) {
    const T* p = static_cast<const T*>(a.p) + n * a.ns + s * a.ss + c;
    v[0] = p[0];
    v[1] = second ? p[1] : v[0];
  }
  __device__ __forceinline__ float operator[](int i) const { return Elem<T>::to_f(v[i]); }
  static __device__ __forceinline__ void store(const RowsArg& a, int n, int s, int c, bool second, float x, float y) {
    T* p = static_cast<T*>(a.p) + n * a.ns + s * a.ss + c;
    p[0] = Elem<T>::from_f(x);
    if (second) p[1] = Elem<T>::from_f(y);
  }
};

// One channel tile of one group of one chunk of one sequence.  fetch() starts
// the copies of a subtile's elements to shared memory, as stored, while the
// subtile before is computed; put() turns them into what the steps need:
// kItems pairs of channels per thread, of one step each and always the same
// pair.  Operands that do not take 16-byte pieces are read by put() itself.
// STATES: dt and dt u.  DY: dy too.  ALL: everything the way back needs.
enum Stage { STATES, DY, ALL };

// The subtiles of a chunk whose steps are t0 .. live - 1 end where they end;
// the first one starts up to seven steps before t0.  Its steps before t0 have
// dt = 0, and the way back comes to them when it has done with all others:
// what a rate that is no number makes of them reaches no step.
__device__ __forceinline__ int first_subtile(int t0, int live) { return live - (live - t0 + kT - 1) / kT * kT; }
// Which one of its sequence the subtile that starts at t is (t0 is a multiple of kT).
__device__ __forceinline__ int subtile_index(int t, int t0) { return t0 / kT + (t - t0 + kT - 1) / kT; }

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T, int TPC>
struct Tile {
  using Sm = GradSmem<T, TPC>;
  static constexpr int P = Sm::P, CH = Sm::CH, NSP = Sm::NSP, V = kPiece<T>;
  static constexpr int kItems = kT * P > kThreads ? kT * P / kThreads : 1;
  const ScanParams& p;
  Sm& sm;
  int n, g, c0, width, begin;

  __device__ __forceinline__ int pair_of() const { return threadIdx.x % P; }
  __device__ __forceinline__ int row_of(int i) const { return threadIdx.x / P + i * (kThreads / P); }
  __device__ __forceinline__ bool has(int i, int t) const {
    return row_of(i) < kT && t + row_of(i) >= begin && 2 * pair_of() < width;
  }

  __device__ __forceinline__ void fetch_rows(const RowsArg& src, int slot, int t) {
    const T* base = static_cast<const T*>(src.p) + n * src.ns + t * src.ss + c0;
#pragma unroll
    for (int i = threadIdx.x; i < Sm::kPieces; i += kThreads) {
      const int r = i / (CH / V), x = i % (CH / V) * V;
      if (t + r >= begin && x < width) copy_async<16>(&sm.raw[slot][i], base + r * src.ss + x);
    }
  }
  __device__ __forceinline__ void fetch_quads(const RowsArg& src, int slot, int t) {
    const T* base = static_cast<const T*>(src.p) + n * src.ns + t * src.ss + (long long)g * p.K;
#pragma unroll
    for (int i = threadIdx.x; i < Sm::kQuads; i += kThreads) {
      const int r = i / (NSP / 4), k = i % (NSP / 4) * 4;
      if (t + r >= begin && k < p.K) copy_async<sizeof(typename Sm::Quad)>(&sm.quads[slot][i], base + r * src.ss + k);
    }
  }
  template <Stage S>
  __device__ __forceinline__ void fetch(int t) {
    if (p.vec) {
      fetch_rows(p.Delta, 0, t);
      fetch_rows(p.X, 1, t);
      if constexpr (S != STATES) {
        fetch_rows(p.dY, 2, t);
        if (p.Z.p) fetch_rows(p.Z, 3, t);
      }
    }
    if (p.bc_vec) {
      fetch_quads(p.Bm, 0, t);
      if constexpr (S != STATES) fetch_quads(p.Cm, 1, t);
    }
  }

  __device__ __forceinline__ void put_quads(const RowsArg& src, int slot, float* to, int t) {
#pragma unroll
    for (int i = threadIdx.x; i < Sm::kQuads; i += kThreads) {
      const int r = i / (NSP / 4), k = i % (NSP / 4) * 4;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (t + r >= begin && k < p.K) {
        if (p.bc_vec) {
          Piece<T, 4>::load(reinterpret_cast<const T*>(&sm.quads[slot][i]), v);
        } else {
          const T* from = static_cast<const T*>(src.p) + n * src.ns + (t + r) * src.ss + (long long)g * p.K + k;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k + e < p.K) v[e] = Elem<T>::to_f(from[e]);
        }
      }
      *reinterpret_cast<float4*>(to + 4 * i) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  // The pair of item i of one of the four row tensors.
  __device__ __forceinline__ Duo<T> pair_at(const RowsArg& src, int slot, int i, int t, bool second) const {
    Duo<T> d;
    if (p.vec) {
      using W = std::conditional_t<sizeof(T) == 4, uint2, uint32_t>;
      const W w = reinterpret_cast<const W*>(sm.raw[slot])[row_of(i) * P + pair_of()];
      __builtin_memcpy(d.v, &w, sizeof(w));
    } else {
      d.load(src, n, t + row_of(i), c0 + 2 * pair_of(), second);
    }
    return d;
  }

  template <Stage S>
  __device__ __forceinline__ void put(int t) {
    const bool second = 2 * pair_of() + 1 < width;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int r = row_of(i);
      if (r >= kT) continue;
      Duo<T> d{}, x{}, gy2{}, z2{};
      const bool on = has(i, t);
      if (on) {
        d = pair_at(p.Delta, 0, i, t, second);
        x = pair_at(p.X, 1, i, t, second);
        if constexpr (S != STATES) {
          gy2 = pair_at(p.dY, 2, i, t, second);
          if (p.Z.p) z2 = pair_at(p.Z, 3, i, t, second);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = e * P + pair_of();
        float dt = 0.0f, u = 0.0f, gy = 0.0f, slope = 0.0f, gate = 0.0f;
        if (on && (e == 0 || second)) {
          u = x[e];
          dt = d[e] + sm.bias[at];
          slope = 1.0f;
          if (p.softplus) {
            if constexpr (S == ALL) dt = softplus_slope(dt, slope);
            else dt = softplus_f(dt);
          }
          if constexpr (S != STATES) {
            gy = gy2[e];
            if (p.Z.p) {
              const float zz = z2[e], sg = sigmoid_of<T>(zz);
              if constexpr (S == ALL) gate = gy * sg * (1.0f + zz * (1.0f - sg));
              gy *= zz * sg;
            }
          }
        }
        sm.dtu[r][at] = make_float4(dt, dt, dt * u, dt * u);
        if constexpr (S != STATES) sm.dy[r][at] = make_float2(gy, gy);
        if constexpr (S == ALL) {
          sm.u[r][at] = u;
          sm.slope[r][at] = slope;
          sm.gate[r][at] = gate;
        }
      }
    }
    put_quads(p.Bm, 0, sm.B[0], t);
    if constexpr (S != STATES) put_quads(p.Cm, 1, sm.C[0], t);
  }

  // A pair of a row gradient: into shared memory where the rows take pieces
  // (stored by flush), else to its place.
  __device__ __forceinline__ void emit(const RowsArg& to, int slot, int i, int t, bool second, float a, float b) {
    if (!to.p) return;
    if (p.vec) {
      if constexpr (sizeof(T) == 4) reinterpret_cast<float2*>(sm.out[slot])[row_of(i) * P + pair_of()] = make_float2(a, b);
      else reinterpret_cast<uint32_t*>(sm.out[slot])[row_of(i) * P + pair_of()] = Elem<T>::pair_from_f(a, b);
    } else {
      Duo<T>::store(to, n, t + row_of(i), c0 + 2 * pair_of(), second, a, b);
    }
  }
  __device__ __forceinline__ void flush(const RowsArg& to, int slot, int t) {
    if (!to.p || !p.vec) return;
    T* base = static_cast<T*>(to.p) + n * to.ns + t * to.ss + c0;
#pragma unroll
    for (int i = threadIdx.x; i < Sm::kPieces; i += kThreads) {
      const int r = i / (CH / V), x = i % (CH / V) * V;
      if (t + r >= begin && x < width) *reinterpret_cast<uint4*>(base + r * to.ss + x) = sm.out[slot][i];
    }
  }

  __device__ __forceinline__ void constants() {
    for (int i = threadIdx.x; i < CH; i += kThreads) {
      const int ch = 2 * (i % P) + i / P;
      sm.bias[i] = (p.bias && ch < width) ? p.bias[c0 + ch] : 0.0f;
      sm.skip[i] = (p.D && ch < width) ? p.D[c0 + ch] : 0.0f;
    }
  }
};

// Four states of two channels, as packed halves: [channel][half].
struct States {
  F2 v[2][2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i / 2][i % 2] = f2(0.0f, 0.0f);
  }
  template <int TPC>
  __device__ __forceinline__ void load(const float* rows, int c, int width_left, const ScanParams& p, int part) {
    zero();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (e >= width_left) continue;
      float x[4];
      load_states<4, TPC>(rows + (long long)(c + e) * p.K, p.K, part, p.k_vec, x);
      v[e][0] = f2(x[0], x[1]), v[e][1] = f2(x[2], x[3]);
    }
  }
  template <int TPC>
  __device__ __forceinline__ void store(float* rows, int c, int width_left, const ScanParams& p, int part) const {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (e >= width_left) continue;
      const float2 a = f2_get(v[e][0]), b = f2_get(v[e][1]);
      const float x[4] = {a.x, a.y, b.x, b.y};
      store_states<4, TPC>(rows + (long long)(c + e) * p.K, p.K, part, p.k_vec, x);
    }
  }
  __device__ __forceinline__ bool finite() const {
    bool all = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = f2_get(v[i / 2][i % 2]);
      all = all && isfinite(a.x) && isfinite(a.y);
    }
    return all;
  }
  __device__ __forceinline__ void to_rates() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = f2_get(v[i / 2][i % 2]);
      v[i / 2][i % 2] = f2(rate2(a.x), rate2(a.y));
    }
  }
};

// Values left of COUNT after log2(LANES) exchanges.
template <int COUNT, int LANES>
constexpr int kLeft = COUNT > LANES ? COUNT / LANES : 1;

__device__ __forceinline__ float halves(F2 a) {
  const float2 v = f2_get(a);
  return v.x + v.y;
}

// 2^(2 half A2) start + own, the factor in two halves: no infinity meets a start
// of 0, and a small one grows as far as float32 goes.
__device__ __forceinline__ F2 join2(F2 half, F2 A2, F2 start, F2 own) {
  float2 x = f2_get(fma2(half, A2, f2(3e-8f, 3e-8f)));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(127.0f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(127.0f));
  const F2 root = exp2_fast2(f2(x.x, x.y));
  return fma2(root, mul2(root, start), own);
}

// h = a h + (dt u) B of one step.
template <typename Sm>
__device__ __forceinline__ void update(const Sm& sm, int r, int j, int part, const States& A2, States& h) {
  const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sm.B[r][part * 4]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&sm.dtu[r][e * Sm::P + j]);
    const F2 dt{w.x}, du{w.y};
    h.v[e][0] = fma2(decay2(dt, A2.v[e][0]), h.v[e][0], mul2(du, F2{B.x}));
    h.v[e][1] = fma2(decay2(dt, A2.v[e][1]), h.v[e][1], mul2(du, F2{B.y}));
  }
}

// The way forward, every chunk from a zero state: the state and the sum of dt
// at the start of each subtile (the true state is that plus the chunk's start
// decayed by the sum) and at the chunk's end.  ADJOINT, for chunks that run
// side by side: what leaves the chunk's start of the state's gradient when
// nothing arrives at its end, the sum over its steps of (product of a from
// the chunk's start) C dy.  The product is carried along; where it overflowed,
// for states that grow, the block sums once more from its exponent.
template <typename T, int TPC, bool ADJOINT>
__global__ void __launch_bounds__(kThreads, 4) scan_grad_states_kernel(ScanParams p) {
  using Sm = GradSmem<T, TPC>;
  constexpr Stage S = ADJOINT ? DY : STATES;
  extern __shared__ __align__(16) unsigned char smem[];
  Sm& sm = *reinterpret_cast<Sm*>(smem);
  next_may_start();
  const int per = p.C / p.G, tiles = (per + Sm::CH - 1) / Sm::CH;
  const int tile = blockIdx.x % tiles;
  int q = blockIdx.x / tiles;
  const int g = q % p.G;
  q /= p.G;
  const int chunk = q % p.chunks, n = q / p.chunks;
  const int t0 = chunk * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const int live = min(t1, row_length(p.lens, n, p.S));
  Tile<T, TPC> b{p, sm, n, g, g * per + tile * Sm::CH, min(Sm::CH, per - tile * Sm::CH), t0};
  const int j = threadIdx.x / TPC, part = threadIdx.x % TPC;
  const int left = b.width - 2 * j, c = b.c0 + (left > 0 ? 2 * j : 0);
  const int subs = (p.S + kT - 1) / kT;
  const int first = first_subtile(t0, live);
  if (t0 < live) b.template fetch<S>(first);
  b.constants();
  States A2, h, pr, e;
  A2.template load<TPC>(p.A, c, left, p, part);
  A2.to_rates();
  h.zero(), e.zero();
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) pr.v[i / 2][i % 2] = f2(1.0f, 1.0f);
  for (int t = first; t < live; t += kT) {
    copies_done();
    __syncthreads();
    b.template put<S>(t);
    __syncthreads();
    if (t + kT < live) b.template fetch<S>(t + kT);
    const long long at = (long long)n * subs + subtile_index(t, t0);
    h.template store<TPC>(p.ckpt + at * p.C * p.K, c, left, p, part);
    if (part == 0) {
      if (left > 0) p.cum[at * p.C + c] = sum[0];
      if (left > 1) p.cum[at * p.C + c + 1] = sum[1];
    }
#pragma unroll 2
    for (int r = 0; r < kT; ++r) {
      const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sm.B[r][part * 4]);
      ulonglong2 C;
      if constexpr (ADJOINT) C = *reinterpret_cast<const ulonglong2*>(&sm.C[r][part * 4]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&sm.dtu[r][k * Sm::P + j]);
        const F2 dt{w.x}, du{w.y};
        F2 dy;
        if constexpr (ADJOINT) dy.v = *reinterpret_cast<const unsigned long long*>(&sm.dy[r][k * Sm::P + j]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const F2 a = decay2(dt, A2.v[k][i]);
          h.v[k][i] = fma2(a, h.v[k][i], mul2(du, F2{i ? B.y : B.x}));
          if constexpr (ADJOINT) {
            pr.v[k][i] = mul2(pr.v[k][i], a);
            e.v[k][i] = fma2(pr.v[k][i], mul2(F2{i ? C.y : C.x}, dy), e.v[k][i]);
          }
        }
        sum[k] += f2_get(dt).x;
      }
    }
  }
  if constexpr (ADJOINT) {
    // Products past float32's range (states that grow): the sum again, from the
    // products' exponents
    if (__syncthreads_or(!pr.finite())) {
      pr.zero(), e.zero();
      if (t0 < live) b.template fetch<S>(first);
      for (int t = first; t < live; t += kT) {
        copies_done();
        __syncthreads();
        b.template put<S>(t);
        __syncthreads();
        if (t + kT < live) b.template fetch<S>(t + kT);
#pragma unroll 1
        for (int r = 0; r < kT; ++r) {
          const ulonglong2 C = *reinterpret_cast<const ulonglong2*>(&sm.C[r][part * 4]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const F2 dt{reinterpret_cast<const ulonglong2*>(&sm.dtu[r][k * Sm::P + j])->x};
            const F2 dy{*reinterpret_cast<const unsigned long long*>(&sm.dy[r][k * Sm::P + j])};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              pr.v[k][i] = fma2(dt, A2.v[k][i], pr.v[k][i]);
              const float2 x = f2_get(pr.v[k][i]), v = f2_get(mul2(F2{i ? C.y : C.x}, dy));
              e.v[k][i] = add2(e.v[k][i], f2(scale2(x.x, v.x), scale2(x.y, v.y)));
            }
          }
        }
      }
    }
    const long long row = ((long long)n * p.chunks + chunk) * p.C;
    h.template store<TPC>(p.carry + row * p.K, c, left, p, part);
    e.template store<TPC>(p.gcarry + row * p.K, c, left, p, part);
    if (part == 0) {
      if (left > 0) p.sumdt[row + c] = sum[0];
      if (left > 1) p.sumdt[row + c + 1] = sum[1];
    }
  }
}

// The chunks in order, forward for the states and backward for their gradient.
__global__ void __launch_bounds__(64) scan_grad_carry_kernel(ScanParams p) {
  const unsigned all = (unsigned)p.C * (unsigned)p.K;  // at most 2^31
  const unsigned at = blockIdx.x * 64u + threadIdx.x;
  const bool back = blockIdx.z != 0, on = at < all;
  next_may_start();
  const float A2 = on ? rate2(p.A[at]) : 0.0f;
  previous_done();
  if (!on) return;
  const long long ck = all;
  const unsigned c = at / (unsigned)p.K;
  for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
    const long long i = n * ck + at;
    float* carry = (back ? p.gcarry : p.carry) + (long long)n * p.chunks * ck + at;
    const float* sumdt = p.sumdt + (long long)n * p.chunks * p.C + c;
    const float* from = back ? p.dhT : p.h0;
    float run = from ? from[i] : 0.0f;
    run = may_grow(p, A2) ? join_batches<4, true>(carry, ck, sumdt, p.C, p.chunks, back, A2, run)
                          : join_batches<16, false>(carry, ck, sumdt, p.C, p.chunks, back, A2, run);
    if (back && p.dh0) p.dh0[i] = run;
  }
}

// A channel tile's chunk, from its end to its start.
template <typename T, int TPC>
__device__ __forceinline__ void grad_tile(const ScanParams& p, GradSmem<T, TPC>& sm, int n, int g, int chunk, int slice,
                                          int tile, bool first) {
  using Sm = GradSmem<T, TPC>;
  constexpr int P = Sm::P, CH = Sm::CH, NSP = Sm::NSP;
  const int per = p.C / p.G;
  const int t0 = chunk * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const int live = min(t1, row_length(p.lens, n, p.S));
  const int j = threadIdx.x / TPC, part = threadIdx.x % TPC;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int subs = (p.S + kT - 1) / kT;
  const long long chunk_row = ((long long)n * p.chunks + chunk) * p.C;
  Tile<T, TPC> b{p, sm, n, g, g * per + tile * CH, min(CH, per - tile * CH), t0};
  const int left = b.width - 2 * j, c = b.c0 + (left > 0 ? 2 * j : 0);
  __syncthreads();
  if (live > t0) b.template fetch<ALL>(live - kT);
  b.constants();
  States A2, e, dA;
  A2.template load<TPC>(p.A, c, left, p, part);
  A2.to_rates();
  e.zero(), dA.zero();
  previous_done();
  if (p.chunks > 1) e.template load<TPC>(p.gcarry + chunk_row * p.K, c, left, p, part);
  else if (p.dhT) e.template load<TPC>(p.dhT + (long long)n * p.C * p.K, c, left, p, part);
  const float* start = p.chunks > 1 ? p.carry + chunk_row * p.K : p.h0 ? p.h0 + (long long)n * p.C * p.K : nullptr;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // dD and d_delta_bias of this thread's pair
  for (int t = live - kT; t > t0 - kT; t -= kT) {
    // the state at the subtile's start: the chunk's own, and what is left of its start's
    States h;
    {
      const long long at = (long long)n * subs + subtile_index(t, t0);
      h.template load<TPC>(p.ckpt + at * p.C * p.K, c, left, p, part);
      if (start) {
        States h0;
        h0.template load<TPC>(start, c, left, p, part);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float cum = k < left ? p.cum[at * p.C + c + k] : 0.0f;
          const F2 half = f2(0.5f * cum, 0.5f * cum);
#pragma unroll
          for (int i = 0; i < 2; ++i) h.v[k][i] = join2(half, A2.v[k][i], h0.v[k][i], h.v[k][i]);
        }
      }
    }
    copies_done();
    __syncthreads();
    b.template put<ALL>(t);
    __syncthreads();
    if (t > t0) b.template fetch<ALL>(t - kT);
    // Half of the subtile's steps at a time, the later ones first: as many
    // states as leave the registers room to overlap steps.  Before the chunk
    // dt, dt u and dy are 0: the state and its gradient stand still
    States dAt;  // of this subtile: long sums of short ones keep more bits
    dAt.zero();
#pragma unroll 1
    for (int base = kT - kHalf; base >= 0; base -= kHalf) {
      States hs[kHalf + 1];  // hs[r]: the state before step base + r
      hs[0] = h;
#pragma unroll 1
      for (int r = 0; r < base; ++r) update(sm, r, j, part, A2, hs[0]);
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        const int r = base + i;
        hs[i + 1] = hs[i];
        update(sm, r, j, part, A2, hs[i + 1]);
        if (p.dZ.p) {
          const ulonglong2 C = *reinterpret_cast<const ulonglong2*>(&sm.C[r][part * 4]);
          float y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            y[k] = halves(fma2(F2{C.y}, hs[i + 1].v[k][1], mul2(F2{C.x}, hs[i + 1].v[k][0])));
          int at = 0;
          lanes_sum<2, TPC / 2, 1>(y, lane, at);
          constexpr int L = kLeft<2, TPC>;
#pragma unroll
          for (int m = 0; m < L; ++m) sm.y[r][(at + m) * P + j] = y[m];
        }
      }
#pragma unroll
      for (int q = kHalf - 1; q >= 0; --q) {
        const int r = base + q;
        const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(&sm.B[r][part * 4]);
        const ulonglong2 C = *reinterpret_cast<const ulonglong2*>(&sm.C[r][part * 4]);
        F2 vb[2], vc[2];
        float s[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&sm.dtu[r][k * P + j]);
          const F2 dt{w.x}, du{w.y}, dy{*reinterpret_cast<const unsigned long long*>(&sm.dy[r][k * P + j])};
          F2 gb, th;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const F2 bi{i ? B.y : B.x}, ci{i ? C.y : C.x}, a2 = A2.v[k][i];
            const F2 a = decay2(dt, a2), gg = fma2(ci, dy, e.v[k][i]);
            vc[i] = k ? fma2(hs[q + 1].v[k][i], dy, vc[i]) : mul2(hs[q + 1].v[k][i], dy);
            vb[i] = k ? fma2(gg, du, vb[i]) : mul2(gg, du);
            gb = i ? fma2(gg, bi, gb) : mul2(gg, bi);
            e.v[k][i] = mul2(gg, a);
            const F2 x = mul2(e.v[k][i], hs[q].v[k][i]);
            th = i ? fma2(x, a2, th) : mul2(x, a2);
            dAt.v[k][i] = fma2(x, dt, dAt.v[k][i]);
          }
          s[k] = halves(gb), s[2 + k] = halves(th);
        }
        int at = 0;
        lanes_sum<4, TPC / 2, 1>(s, lane, at);
        constexpr int L = kLeft<4, TPC>;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          const int v = at + i;
          (v < 2 ? sm.gb : sm.th)[r][(v & 1) * P + j] = s[i];
        }
        const float2 b0 = f2_get(vb[0]), b1 = f2_get(vb[1]), c0 = f2_get(vc[0]), c1 = f2_get(vc[1]);
        float v[8] = {b0.x, b0.y, b1.x, b1.y, c0.x, c0.y, c1.x, c1.y};
        at = 0;
        lanes_sum<8, 16, TPC>(v, lane, at);
        constexpr int M = kLeft<8, 32 / TPC>;
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const int w = at + i;
          sm.part[r][warp][w / 4 * NSP + part * 4 + w % 4] = v[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) dA.v[i / 2][i % 2] = add2(dA.v[i / 2][i % 2], dAt.v[i / 2][i % 2]);
    __syncthreads();
    // the subtile's row gradients
    const int pj = b.pair_of();
    const bool second = 2 * pj + 1 < b.width;
#pragma unroll
    for (int i = 0; i < Tile<T, TPC>::kItems; ++i) {
      if (!b.has(i, t)) continue;
      const int r = b.row_of(i);
      float du[2], dd[2], dz[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = k * P + pj;
        const float gb = sm.gb[r][at], u = sm.u[r][at], dy = sm.dy[r][at].x;
        du[k] = fmaf(gb, sm.dtu[r][at].x, sm.skip[at] * dy);
        dd[k] = fmaf(gb, u, sm.th[r][at] * kLn2) * sm.slope[r][at];
        dz[k] = sm.gate[r][at] * fmaf(sm.skip[at], u, sm.y[r][at]);
        acc[k] = fmaf(dy, u, acc[k]);
        acc[2 + k] += dd[k];
      }
      b.emit(p.dX, 0, i, t, second, du[0], du[1]);
      b.emit(p.dDelta, 1, i, t, second, dd[0], dd[1]);
      b.emit(p.dZ, 2, i, t, second, dz[0], dz[1]);
    }
    if (p.bc_part) {
      float* to = p.bc_part + ((((long long)slice * p.N + n) * p.S + t) * p.G + g) * 2 * p.K;
#pragma unroll
      for (int i = threadIdx.x; i < kT * 2 * NSP; i += kThreads) {
        const int r = i / (2 * NSP), w = i % (2 * NSP), k = w % NSP;
        if (k >= p.K || t + r < t0) continue;
        float v = sm.part[r][0][w];
#pragma unroll
        for (int m = 1; m < kWarps; ++m) v += sm.part[r][m][w];
        float* at = to + r * p.G * 2 * p.K + w / NSP * p.K + k;
        *at = first ? v : *at + v;
      }
    }
    if (p.vec) {
      __syncthreads();
      b.flush(p.dX, 0, t);
      b.flush(p.dDelta, 1, t);
      b.flush(p.dZ, 2, t);
    }
  }

  // what is left: zeros past the length, the state's gradient, the sums over the chunk's steps
  const int from = max(t0, live);
  for (int i = threadIdx.x; i < (t1 - from) * P; i += kThreads) {
    const int s = from + i / P, k = 2 * (i % P);
    if (k >= b.width) continue;
    for (const RowsArg* a : {&p.dX, &p.dDelta, &p.dZ})
      if (a->p) Duo<T>::store(*a, n, s, b.c0 + k, k + 1 < b.width, 0.0f, 0.0f);
  }
  if (p.chunks == 1 && p.dh0) e.template store<TPC>(p.dh0 + (long long)n * p.C * p.K, c, left, p, part);
  if (p.w_part) {
    float* w = p.w_part + chunk_row * (p.K + 2);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k >= left) continue;
      const float2 lo = f2_get(dA.v[k][0]), hi = f2_get(dA.v[k][1]);
      const float x[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (part * 4 + i < p.K) w[(long long)(c + k) * p.K + part * 4 + i] = x[i];
    }
    w += (long long)p.C * p.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) sm.acc[threadIdx.x][i] = acc[i];
    __syncthreads();
    for (int ch = threadIdx.x; ch < b.width; ch += kThreads) {
      float d = 0.0f, v = 0.0f;
#pragma unroll 4
      for (int q = ch / 2; q < kThreads; q += P) d += sm.acc[q][ch & 1], v += sm.acc[q][2 + (ch & 1)];
      w[b.c0 + ch] = d;
      w[p.C + b.c0 + ch] = v;
    }
  }
}

template <typename T, int TPC>
__global__ void __launch_bounds__(kThreads, 4) scan_grad_kernel(ScanParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  using Sm = GradSmem<T, TPC>;
  Sm& sm = *reinterpret_cast<Sm*>(smem);
  next_may_start();
  const int tiles = (p.C / p.G + Sm::CH - 1) / Sm::CH;
  const int slice = blockIdx.x % p.slices;
  int q = blockIdx.x / p.slices;
  const int g = q % p.G;
  q /= p.G;
  const int chunk = q % p.chunks, n = q / p.chunks;
  const int from = slice * p.slice_tiles, to = min(from + p.slice_tiles, tiles);
  for (int tile = from; tile < to; ++tile) grad_tile<T, TPC>(p, sm, n, g, chunk, slice, tile, tile == from);
}

// dB and dC from the slices, in order; zeros past the length.  V values per
// thread, all of one row of dB or dC.
template <typename T, int V>
__global__ void __launch_bounds__(128) scan_grad_rows_kernel(ScanParams p) {
  const int row = p.G * 2 * p.K;
  const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) * V;
  next_may_start();
  previous_done();
  const long long all = (long long)p.N * p.S * row;
  if (i >= all) return;
  const int j = (int)(i % row);
  const long long ns = i / row;
  const int s = (int)(ns % p.S), n = (int)(ns / p.S);
  const int g = j / (2 * p.K), which = j / p.K % 2, k = j % p.K;
  float v[V];
  fill(v, 0.0f);
  if (s < row_length(p.lens, n, p.S)) {
#pragma unroll 16
    for (int q = 0; q < p.slices; ++q) {
      float w[V];
      Piece<float, V>::load(p.bc_part + q * all + i, w);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] += w[e];
    }
  }
  const RowsArg& to = which ? p.dC : p.dB;
  if (!to.p) return;
  T* out = static_cast<T*>(to.p) + n * to.ns + s * to.ss + (long long)g * p.K + k;
#pragma unroll
  for (int e = 0; e < V; ++e) out[e] = Elem<T>::from_f(v[e]);
}

// dA, dD and d_delta_bias from the sequences' and chunks' sums, in a fixed order.
__global__ void __launch_bounds__(256) scan_grad_weights_kernel(ScanParams p) {
  __shared__ float buf[8][33];
  const long long cols = (long long)p.C * (p.K + 2);
  const long long col = (long long)blockIdx.x * 32 + threadIdx.x % 32;
  const int part = threadIdx.x / 32;
  const long long rows = (long long)p.N * p.chunks;
  float s = 0.0f;
  previous_done();
  if (col < cols) {
#pragma unroll 4
    for (long long b = part; b < rows; b += 8) s += p.w_part[b * cols + col];
  }
  buf[part][threadIdx.x % 32] = s;
  __syncthreads();
  if (part == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += buf[i][threadIdx.x];
    const long long ck = (long long)p.C * p.K;
    if (col < ck) {
      if (p.dA) p.dA[col] = s;
    } else if (col < ck + p.C) {
      if (p.dD) p.dD[col - ck] = s;
    } else if (p.dbias) {
      p.dbias[col - ck - p.C] = s;
    }
  }
}

template <typename T, int TPC, bool ADJOINT>
cudaError_t run_states(const ScanParams& p, long long blocks, cudaStream_t s) {
  constexpr int smem = (int)sizeof(GradSmem<T, TPC>);
  const cudaError_t e = cudaFuncSetAttribute(scan_grad_states_kernel<T, TPC, ADJOINT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) scan_grad_states_kernel<T, TPC, ADJOINT><<<(unsigned)blocks, kThreads, smem, s>>>(p);
  return e;
}

template <typename T, int TPC>
cudaError_t run_grad(const ScanParams& p, cudaStream_t s, int* launches) {
  using Sm = GradSmem<T, TPC>;
  const long long tiles = (p.C / p.G + Sm::CH - 1) / Sm::CH;
  const long long rest = (long long)p.N * p.chunks * p.G;
  if (rest * tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(scan_grad_kernel<T, TPC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Sm));
  if (e != cudaSuccess) return e;
  e = p.chunks > 1 ? run_states<T, TPC, true>(p, rest * tiles, s) : run_states<T, TPC, false>(p, rest * tiles, s);
  if (e != cudaSuccess) return e;
  if (p.chunks > 1) {
    const long long states = (long long)p.C * p.K;
    e = launch_chained(scan_grad_carry_kernel, dim3((unsigned)((states + 63) / 64), std::min(p.N, 65535), 2), 64, 0,
                       s, p);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  e = launch_chained(scan_grad_kernel<T, TPC>, (unsigned)(rest * p.slices), kThreads, sizeof(Sm), s, p);
  *launches += 2;
  if (e == cudaSuccess && p.bc_part) {
    const long long all = (long long)p.N * p.S * p.G * 2 * p.K;
    const int v = p.K % 4 == 0 ? 4 : 1;
    e = launch_chained(v == 4 ? scan_grad_rows_kernel<T, 4> : scan_grad_rows_kernel<T, 1>,
                       (unsigned)((all / v + 127) / 128), 128, 0, s, p);
    *launches += 1;
  }
  if (e == cudaSuccess && p.w_part) {
    e = launch_chained(scan_grad_weights_kernel, (unsigned)(((long long)p.C * (p.K + 2) + 31) / 32), 256, 0, s, p);
    *launches += 1;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t grad_typed(const ScanParams& p, cudaStream_t s, int* launches) {
  switch (tpc_of(p.K)) {
    case 2: return run_grad<T, 2>(p, s, launches);
    case 4: return run_grad<T, 4>(p, s, launches);
    case 8: return run_grad<T, 8>(p, s, launches);
    case 16: return run_grad<T, 16>(p, s, launches);
    default: return run_grad<T, 32>(p, s, launches);
  }
}

long long up4(long long n) { return (n + 3) / 4 * 4; }

// Most floats that the slices' sums of dB and dC may take: beyond it a block
// runs several channel tiles one after the other and adds to its own slice.
constexpr long long kSliceFloats = 64LL << 20;

}  // namespace

ScanPlan scan_grad_plan(long long seq, long long batch, long long channels, int state, int groups, bool ragged) {
  ScanPlan pl{};
  pl.chunks = 1;
  pl.chunk = (int)std::max<long long>(seq, 1);
  pl.slices = pl.slice_tiles = 1;
  if (seq == 0 || batch == 0) return pl;
  const long long per = channels / groups, ch = 2 * kThreads / tpc_of(state);
  const long long tiles = (per + ch - 1) / ch;
  const long long blocks = batch * groups * tiles;
  // Chunks where the sequences alone fill up to two thirds of the card's places
  // (four blocks per SM, which the registers leave room for; with at most 8
  // states shared memory leaves it for two in float32 and three in 16 bits, and
  // the rule was not measured there): 1024 steps x 2048 channels x 16 states bf16, 8
  // sequences 831 us without and 625 with, 12 sequences 1084 and 899, 14
  // sequences 1081 and 1134.  Twice as many blocks as places fill the card more
  // evenly (8 sequences 625 against 677 us) while a chunk keeps 64 steps (a
  // single sequence's chunks of 32 would cost 101 us against 94); up to the
  // places chunks go down to a subtile (201 steps x 3 x 519 x 24: 38 us, with 16
  // steps at least 44, with 32 53).  From 24 steps on (2048 channels: 24 steps
  // 24.6 us against 28.9 without chunks, 16 steps the same).  Where rows have
  // lengths, half of the steps are taken to be past them, and twice the blocks
  // wanted (lengths uniform in 1..1024: 8 sequences 373 us without that and 319
  // with, 16 sequences 863 and 665, 24 sequences 1209 and 1217).
  const long long places = kPlanSms * 4 * (ragged ? 2 : 1);
  if (seq >= 24 && blocks * 3 <= places * 2) {
    const long long chunks = std::max(std::min(seq / 64, places * 2 / blocks), std::min(seq / kT, places / blocks));
    if (chunks > 1) {
      pl.chunk = (int)((((seq + chunks - 1) / chunks) + kT - 1) / kT * kT);
      pl.chunks = (int)((seq + pl.chunk - 1) / pl.chunk);
    }
  }
  const long long row = batch * seq * groups * 2 * state;
  pl.slice_tiles = (int)std::min<long long>(tiles, std::max<long long>((tiles * row + kSliceFloats - 1) / kSliceFloats, 1));
  pl.slices = (int)((tiles + pl.slice_tiles - 1) / pl.slice_tiles);
  if (pl.chunks > 1) {
    pl.carry = pl.gcarry = up4(batch * pl.chunks * channels * state);
    pl.sumdt = up4(batch * pl.chunks * channels);
  }
  pl.ckpt = up4(batch * ((seq + kT - 1) / kT) * channels * state);
  pl.cum = up4(batch * ((seq + kT - 1) / kT) * channels);
  pl.bc_part = up4(pl.slices * row);
  pl.w_part = up4(batch * pl.chunks * channels * (state + 2));
  return pl;
}

cudaError_t launch_scan_grad(const ScanParams& p, cudaStream_t s, int* launches) {
  switch (p.dtype) {
    case RK_F32: return grad_typed<float>(p, s, launches);
    case RK_F16: return grad_typed<__half>(p, s, launches);
    default: return grad_typed<__nv_bfloat16>(p, s, launches);
  }
}

}  // namespace rk
