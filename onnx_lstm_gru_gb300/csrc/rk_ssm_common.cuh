// rk_ssm_common.cuh -- what the state space operators' kernels share: loads
// and stores of 16-byte pieces of any element type, and the scalar functions
// in float32.
#pragma once
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

__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + exp2_fast(-kLog2e * x)); }

// log(1 + e^x); x itself where e^-x is lost beside it.
__device__ __forceinline__ float softplus_f(float x) { return x > 20.0f ? x : log1pf(__expf(x)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

// The K states of a thread from a [K]-row of global memory.
template <int K, int TPC>
__device__ __forceinline__ void load_states(const float* row, int states, int part, float (&h)[K]) {
#pragma unroll
  for (int i = 0; i < K; i += 4) {
    const int k = state_of<TPC>(i, part);
    if (states % 4 == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
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
__device__ __forceinline__ void store_states(float* row, int states, int part, const float (&h)[K]) {
#pragma unroll
  for (int i = 0; i < K; i += 4) {
    const int k = state_of<TPC>(i, part);
    if (states % 4 == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
      if (k < states) *reinterpret_cast<float4*>(row + k) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k + j < states) row[k + j] = h[i + j];
    }
  }
}

}  // namespace rk
