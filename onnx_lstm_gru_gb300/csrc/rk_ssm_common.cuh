// rk_ssm_common.cuh -- what the state space operators' kernels share: loads
// and stores of 16-byte pieces of any element type, and the scalar functions
// in float32.
#pragma once
#include <type_traits>

#include "rk_elem.cuh"
#include "rk_ssm.h"

namespace rk {

// V consecutive elements as floats; one 16- or 8-byte access where V > 1.
template <typename T, int V>
struct Piece {
  static_assert(V == 1 || V * sizeof(T) == 16 || V * sizeof(T) == 8, "one access");
  static __device__ __forceinline__ void load(const T* p, float (&o)[V]) {
    if constexpr (V == 1) {
      o[0] = Elem<T>::to_f(*p);
    } else if constexpr (sizeof(T) == 4) {
      if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        o[0] = v.x, o[1] = v.y;
      }
    } else {
      uint32_t u[V / 2];
      if constexpr (V == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        u[0] = v.x, u[1] = v.y;
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 f = Elem<T>::pair_to_f(u[i]);
        o[2 * i] = f.x, o[2 * i + 1] = f.y;
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&o)[V]) {
    if constexpr (V == 1) {
      *p = Elem<T>::from_f(o[0]);
    } else if constexpr (sizeof(T) == 4) {
      if constexpr (V == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
        *reinterpret_cast<float2*>(p) = make_float2(o[0], o[1]);
      }
    } else {
      uint32_t u[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) u[i] = Elem<T>::pair_from_f(o[2 * i], o[2 * i + 1]);
      if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
      }
    }
  }
};

// V consecutive elements as stored, to be widened later.
template <typename T, int V>
struct Packed {
  using Raw = std::conditional_t<V * sizeof(T) == 16, uint4,
                                 std::conditional_t<V * sizeof(T) == 8, uint2,
                                                    std::conditional_t<V * sizeof(T) == 4, uint32_t, uint16_t>>>;
  Raw raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
  // read once: leaves the caches first
  __device__ __forceinline__ void load_streaming(const T* p) { raw = __ldcs(reinterpret_cast<const Raw*>(p)); }
  __device__ __forceinline__ void widen(float (&o)[V]) const {
    T t[V];
    __builtin_memcpy(t, &raw, sizeof(raw));
    if constexpr (sizeof(T) == 2 && V > 1) {
      uint32_t u[V / 2];
      __builtin_memcpy(u, &raw, sizeof(raw));
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 f = Elem<T>::pair_to_f(u[i]);
        o[2 * i] = f.x, o[2 * i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = Elem<T>::to_f(t[i]);
    }
  }
  __device__ __forceinline__ void narrow(const float (&o)[V]) {
    if constexpr (sizeof(T) == 2 && V > 1) {
      uint32_t u[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) u[i] = Elem<T>::pair_from_f(o[2 * i], o[2 * i + 1]);
      __builtin_memcpy(&raw, u, sizeof(raw));
    } else {
      T t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] = Elem<T>::from_f(o[i]);
      __builtin_memcpy(&raw, t, sizeof(raw));
    }
  }
  __device__ __forceinline__ void store_streaming(T* p) const { __stcs(reinterpret_cast<Raw*>(p), raw); }
};

// Elements of a 16-byte piece.
template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);

template <int V>
__device__ __forceinline__ void fill(float (&o)[V], float v) {
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = v;
}

// 2^x by the special function unit (relative error about 2^-22).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / x by the special function unit (relative error about 2^-23; 0 for an infinite x).
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLn2 = 0.6931471805599453f;

// sigmoid(x) for tensors of T.  2^t of the rounded product t = -x log2(e) alone
// is off by a relative error that grows with -x (7e-7 at -20, 4e-6 at -80), far
// below what a 16-bit element keeps.  float32 ones get the rest too: e^-x is
// 2^t e^r with r = -x - t ln(2), which the fused multiply-add leaves exact but
// for ln(2)'s own rounding, t 2e-9, and e^r = 1 + r, |r| being under 1e-5.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float x) {
  const float t = -kLog2e * x;
  float e = exp2_fast(t);
  // at least a half: beyond the exponential's range r is anything, and e is 0 or infinite
  if constexpr (sizeof(T) == 4) e *= fmaxf(1.0f + fmaf(-t, kLn2, -x), 0.5f);
  return rcp_fast(1.0f + e);
}

// log(1 + e^x) = max(x, 0) + log(1 + e) with e = e^-|x| <= 1, and
// log(1 + e) = 2 artanh(s), s = e / (2 + e) <= 1/3; artanh(s) / s is a
// polynomial in s^2, interpolated at the Chebyshev nodes of [0, 1/9] (relative
// error 4e-9).  Nothing of a small result (steps of a thousandth are common)
// is lost to 1 + e.
__device__ __forceinline__ float softplus_from(float x, float& e) {
  const float n = -(fabsf(x) < 100.0f ? fabsf(x) : 100.0f), t = n * kLog2e;
  // what the product rounded away, its own factor's rounding too, put back
  // behind the exponential: a fused multiply-add gives the first exactly
  // (Dekker's two-product), the second is what kLog2e is short of log2(e)
  constexpr float kLow = (float)(1.4426950408889634 - (double)kLog2e);
  const float lo = fmaf(n, kLog2e, -t) + n * kLow;
  const float e0 = exp2_fast(t);
  e = fmaf(e0, lo * kLn2, e0);
  const float s = e * rcp_fast(2.0f + e), q = s * s;
  float r = fmaf(q, 0.14078889f, 0.13982579f);
  r = fmaf(r, q, 0.20012298f);
  r = fmaf(r, q, 0.33333161f);
  r = fmaf(r, q, 1.0f);
  const float y = fmaf(2.0f * s, r, fmaxf(x, 0.0f));
  return x == x ? y : x;  // the comparisons above drop a NaN
}

__device__ __forceinline__ float softplus_f(float x) {
  float e;
  return softplus_from(x, e);
}
// And its slope, sigmoid(x).
__device__ __forceinline__ float softplus_slope(float x, float& slope) {
  float e;
  const float y = softplus_from(x, e), r = rcp_fast(1.0f + e);
  slope = x >= 0.0f ? r : e * r;
  return x == x ? y : (slope = x);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Two float32 in one register pair: the packed forms take one issue slot for
// two results.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 exp2_fast2(F2 x) {
  const float2 t = f2_get(x);
  return f2(exp2_fast(t.x), exp2_fast(t.y));
}

// The decays 2^(dt A2).  The unit's results near 1 are 2.5e-8 too small on
// average (measured), which a state that remembers a thousand steps adds up;
// 3e-8 more in the exponent takes that out (left: under 6e-9) and still gives
// exactly 1 for dt = 0.
__device__ __forceinline__ F2 decay2(F2 dt, F2 A2) { return exp2_fast2(fma2(dt, A2, f2(3e-8f, 3e-8f))); }
__device__ __forceinline__ float decay(float dt, float A2) { return exp2_fast(fmaf(dt, A2, 3e-8f)); }

// A decay rate in base-2 exponents per unit of dt, not infinite, so that a
// step of dt = 0 keeps the state.  A rate that is no number stays none, and
// with it the state: these forms of min and max hand a NaN on.
__device__ __forceinline__ float rate2(float a) {
  float r = a * kLog2e;
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(-3.0e38f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(3.0e38f));
  return r;
}

// Where decays may grow a state (a rate above 0, or steps that no softplus keeps
// from being negative) 2^x can pass float32's range.  2^x v is then taken in two
// parts, so that it is 0 for v = 0 and finite wherever it can be.
__device__ __forceinline__ bool may_grow(const ScanParams& p, float A2) { return A2 > 0.0f || !p.softplus; }
__device__ __forceinline__ float scale2(float x, float v) {
  const float over = fminf(fmaxf(x - 127.0f, 0.0f), 127.0f);
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(127.0f));
  return exp2_fast(x) * (exp2_fast(over) * v);
}

// The chunks of a sequence in order, for one state of one channel: from what
// enters the first one, run, each chunk's own end (carry) is replaced by what
// enters it; returns what leaves the last one.  The chunk whose steps sum to d
// leaves 2^(A2 d) run and its own end; all of run where no step is within the
// row's length, whatever the rate.  BACK: from the last chunk to the first.
// A batch is read before any of it is overwritten: its loads are in flight
// together.  States that may grow go through a loop of their own, with fewer.
template <int BATCH, bool GROWS>
__device__ __forceinline__ float join_batches(float* carry, long long ck, const float* sumdt, int C, int chunks,
                                              bool back, float A2, float run) {
#pragma unroll 1
  for (int q0 = 0; q0 < chunks; q0 += BATCH) {
    float s[BATCH], d[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int q = back ? chunks - 1 - q0 - j : q0 + j;
      if (q0 + j < chunks) s[j] = carry[q * ck], d[j] = sumdt[(long long)q * C];
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      if (q0 + j < chunks) {
        carry[(back ? chunks - 1 - q0 - j : q0 + j) * ck] = run;
        if constexpr (GROWS) run = s[j] + scale2(d[j] == 0.0f ? 0.0f : A2 * d[j], run);
        else run = fmaf(d[j] == 0.0f ? 1.0f : exp2_fast(A2 * d[j]), run, s[j]);
      }
    }
  }
  return run;
}

// Adds COUNT values over the lanes whose bits from FIRST down to LAST
// differ.  Each exchange leaves a lane half of its values until one is left;
// on return v[0 .. left) are the sums of values at + 0 .. left - 1.
template <int COUNT, int FIRST, int LAST>
__device__ __forceinline__ void lanes_sum(float* v, int lane, int& at) {
  if constexpr (FIRST >= LAST && FIRST > 0) {
    if constexpr (COUNT > 1) {
      constexpr int H = COUNT / 2;
      const bool hi = lane & FIRST;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = hi ? v[i] : v[i + H], keep = hi ? v[i + H] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, FIRST);
      }
      if (hi) at += H;
      lanes_sum<H, FIRST / 2, LAST>(v, lane, at);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], FIRST);
      lanes_sum<1, FIRST / 2, LAST>(v, lane, at);
    }
  }
}
// The launches of one call are chained: the next kernel's blocks may take
// their places as soon as every block of this one runs (next_may_start), and
// wait there until this one has ended and its writes are visible
// (previous_done; at once where nothing was chained).
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename P>
cudaError_t launch_chained(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const P& p) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid, config.blockDim = block, config.dynamicSmemBytes = smem, config.stream = stream;
  config.attrs = &attr, config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, p);
}

// A row's length, clamped to the steps there are.
__device__ __forceinline__ int row_length(const int* lens, int n, int S) {
  return lens ? min(max(lens[n], 0), S) : S;
}

// State that thread `part` of TPC holds in its register i: pieces of four,
// dealt out in turn, so that the threads of a channel read one row of
// shared memory together.
template <int TPC>
__device__ __forceinline__ int state_of(int i, int part) {
  return (i / 4 * TPC + part) * 4 + i % 4;
}

// The K states of a thread from a row of global memory; vec: rows take
// 16-byte pieces.
template <int K, int TPC>
__device__ __forceinline__ void load_states(const float* row, int states, int part, bool vec, float (&h)[K]) {
#pragma unroll
  for (int i = 0; i < K; i += 4) {
    const int k = state_of<TPC>(i, part);
    if (vec) {
      if (k < states) {
        const float4 v = *reinterpret_cast<const float4*>(row + k);
        h[i] = v.x, h[i + 1] = v.y, h[i + 2] = v.z, h[i + 3] = v.w;
      } else {
        h[i] = h[i + 1] = h[i + 2] = h[i + 3] = 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) h[i + j] = k + j < states ? row[k + j] : 0.0f;
    }
  }
}

template <int K, int TPC>
__device__ __forceinline__ void store_states(float* row, int states, int part, bool vec, const float (&h)[K]) {
#pragma unroll
  for (int i = 0; i < K; i += 4) {
    const int k = state_of<TPC>(i, part);
    if (vec) {
      if (k < states) *reinterpret_cast<float4*>(row + k) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k + j < states) row[k + j] = h[i + j];
    }
  }
}

}  // namespace rk
