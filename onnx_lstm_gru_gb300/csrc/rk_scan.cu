// rk_scan.cu -- selective scan: prompts (many steps) and single tokens.
//
// Per step, channel and state: one exponential, a = exp(dt A), and the update
// h = a h + (dt u) B, y += C h.  A thread keeps K states of one channel in
// registers and runs along the steps; TPC neighbouring threads share a channel
// of more states and add their parts of y by shuffles.  Every step's dt, u, B
// and C are staged in shared memory by the whole block, in 16-byte loads, so
// softplus is taken once per element and not once per thread.
//
// One sequence of a few thousand channels does not fill the card, so the
// sequence is cut into chunks that run side by side.  The state that leaves a
// chunk is linear in the one that enters it, h_out = exp(A sum dt) h_in + S:
// one launch computes every chunk's S and sum dt from a zero start, a second
// runs through the chunks in order, and a third starts each chunk from its
// state and computes the outputs.
#include <algorithm>

#include "rk.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

constexpr int kThreads = 128;
constexpr int kSub = 16;  // steps staged at once

template <typename T, int V, int NSP>
__device__ __forceinline__ void stage_group(const RowsArg& src, int n, int g, int states, int t, int live,
                                            float (*dst)[NSP]) {
  constexpr int kPieces = NSP / V;
  for (int i = threadIdx.x; i < kSub * kPieces; i += kThreads) {
    const int r = i / kPieces, k = i % kPieces * V;
    float v[V];
    if (t + r < live && k < states) {
      Piece<T, V>::load(static_cast<const T*>(src.p) + n * src.ns + (t + r) * src.ss + (long long)g * states + k, v);
    } else {
      fill(v, 0.0f);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) dst[r][k + j] = v[j];
  }
}

// K states per thread, TPC threads per channel.  OUT: the outputs, each chunk
// from its own start; else every chunk's final state from zero and its sum of dt.
template <typename T, int K, int TPC, bool OUT>
__global__ void __launch_bounds__(kThreads) scan_kernel(ScanParams p) {
  constexpr int CH = kThreads / TPC, NSP = K * TPC;
  __shared__ float2 sd[kSub][CH];  // dt, u
  __shared__ __align__(16) float sB[kSub][NSP];
  __shared__ __align__(16) float sC[OUT ? kSub : 1][NSP];
  __shared__ float sY[OUT ? kSub : 1][CH];
  __shared__ float sbias[CH], sskip[CH];
  const int per = p.C / p.G, tiles = (per + CH - 1) / CH;
  const int tile = blockIdx.x % tiles;
  int q = blockIdx.x / tiles;
  const int g = q % p.G;
  q /= p.G;
  const int chunk = q % p.chunks, n = q / p.chunks;
  const int c0 = g * per + tile * CH, width = min(CH, per - tile * CH);
  const int t0 = chunk * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const int live = min(t1, row_length(p.lens, n, p.S));
  const int lc = threadIdx.x / TPC, part = threadIdx.x % TPC;
  const bool mine = lc < width;
  const int c = c0 + (mine ? lc : 0);
  const long long row = ((long long)n * p.chunks + chunk) * p.C + c;

  for (int i = threadIdx.x; i < CH; i += kThreads) {
    sbias[i] = (p.bias && i < width) ? p.bias[c0 + i] : 0.0f;
    sskip[i] = (p.D && i < width) ? p.D[c0 + i] : 0.0f;
  }
  float A2[K], h[K];
  load_states<K, TPC>(p.A + (long long)c * p.K, p.K, part, A2);
#pragma unroll
  for (int i = 0; i < K; ++i) A2[i] *= kLog2e;
  fill(h, 0.0f);
  if (OUT) {
    if (p.chunks > 1) load_states<K, TPC>(p.carry + row * p.K, p.K, part, h);
    else if (p.h0) load_states<K, TPC>(p.h0 + ((long long)n * p.C + c) * p.K, p.K, part, h);
  }
  float sum = 0.0f;
  __syncthreads();

  auto stage = [&](auto piece, int t) {
    constexpr int V = decltype(piece)::value;
    constexpr int kPieces = CH / V > 0 ? CH / V : 1;
    for (int i = threadIdx.x; i < kSub * kPieces; i += kThreads) {
      const int r = i / kPieces, x = i % kPieces * V;
      float d[V], u[V];
      const bool on = t + r < live && x < width;
      if (on) {
        Piece<T, V>::load(static_cast<const T*>(p.Delta.p) + n * p.Delta.ns + (t + r) * p.Delta.ss + c0 + x, d);
        Piece<T, V>::load(static_cast<const T*>(p.X.p) + n * p.X.ns + (t + r) * p.X.ss + c0 + x, u);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float dt = 0.0f, uu = 0.0f;
        if (on) {
          dt = d[j] + sbias[x + j];
          if (p.softplus) dt = softplus_f(dt);
          uu = u[j];
        }
        sd[r][x + j] = make_float2(dt, uu);
      }
    }
  };
  auto emit = [&](auto piece, int t) {
    constexpr int V = decltype(piece)::value;
    constexpr int kPieces = CH / V > 0 ? CH / V : 1;
    for (int i = threadIdx.x; i < kSub * kPieces; i += kThreads) {
      const int r = i / kPieces, x = i % kPieces * V;
      if (t + r >= live || x >= width) continue;
      float y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = fmaf(sskip[x + j], sd[r][x + j].y, sY[r][x + j]);
      if (p.Z.p) {
        float z[V];
        Piece<T, V>::load(static_cast<const T*>(p.Z.p) + n * p.Z.ns + (t + r) * p.Z.ss + c0 + x, z);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] *= z[j] * sigmoid_fast(z[j]);
      }
      Piece<T, V>::store(static_cast<T*>(p.Y.p) + n * p.Y.ns + (t + r) * p.Y.ss + c0 + x, y);
    }
  };
  using Wide = std::integral_constant<int, (CH >= kPiece<T> ? kPiece<T> : 1)>;
  using One = std::integral_constant<int, 1>;

  for (int t = t0; t < live; t += kSub) {
    if (p.vec) stage(Wide{}, t);
    else stage(One{}, t);
    if (p.bc_vec) {
      stage_group<T, 4, NSP>(p.Bm, n, g, p.K, t, live, sB);
      if constexpr (OUT) stage_group<T, 4, NSP>(p.Cm, n, g, p.K, t, live, sC);
    } else {
      stage_group<T, 1, NSP>(p.Bm, n, g, p.K, t, live, sB);
      if constexpr (OUT) stage_group<T, 1, NSP>(p.Cm, n, g, p.K, t, live, sC);
    }
    __syncthreads();
    const int steps = min(kSub, live - t);
#pragma unroll 4
    for (int r = 0; r < steps; ++r) {
      const float2 v = sd[r][lc];
      const float dtu = v.x * v.y;
      float y = 0.0f;
#pragma unroll
      for (int i = 0; i < K; i += 4) {
        const int k = state_of<TPC>(i, part);
        const float4 b = *reinterpret_cast<const float4*>(&sB[r][k]);
        h[i] = fmaf(exp2_fast(v.x * A2[i]), h[i], dtu * b.x);
        h[i + 1] = fmaf(exp2_fast(v.x * A2[i + 1]), h[i + 1], dtu * b.y);
        h[i + 2] = fmaf(exp2_fast(v.x * A2[i + 2]), h[i + 2], dtu * b.z);
        h[i + 3] = fmaf(exp2_fast(v.x * A2[i + 3]), h[i + 3], dtu * b.w);
        if constexpr (OUT) {
          const float4 e = *reinterpret_cast<const float4*>(&sC[r][k]);
          y = fmaf(e.x, h[i], y);
          y = fmaf(e.y, h[i + 1], y);
          y = fmaf(e.z, h[i + 2], y);
          y = fmaf(e.w, h[i + 3], y);
        }
      }
      if constexpr (OUT) {
#pragma unroll
        for (int o = TPC / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (part == 0) sY[r][lc] = y;
      } else {
        sum += v.x;
      }
    }
    __syncthreads();
    if constexpr (OUT) {
      if (p.Y.p) {
        if (p.vec) emit(Wide{}, t);
        else emit(One{}, t);
      }
      __syncthreads();
    }
  }
  if constexpr (OUT) {
    if (p.Y.p) {
      const int from = max(t0, live);
      for (int i = threadIdx.x; i < CH; i += kThreads) {
        if (i >= width) continue;
        T* y = static_cast<T*>(p.Y.p) + n * p.Y.ns + c0 + i;
        for (int t = from; t < t1; ++t) y[t * p.Y.ss] = Elem<T>::from_f(0.0f);
      }
    }
    if (p.chunks == 1 && p.hT && mine) store_states<K, TPC>(p.hT + ((long long)n * p.C + c) * p.K, p.K, part, h);
  } else if (mine) {
    store_states<K, TPC>(p.carry + row * p.K, p.K, part, h);
    if (part == 0) p.sumdt[row] = sum;
  }
}

// Runs through the chunks of each (sequence, channel, state): the state each
// starts from takes the place of its own final state.
__global__ void __launch_bounds__(256) scan_carry_kernel(ScanParams p) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long ck = (long long)p.C * p.K;
  if (i >= p.N * ck) return;
  const int n = (int)(i / ck);
  const long long at = i % ck;
  const int c = (int)(at / p.K);
  const float A2 = p.A[at] * kLog2e;
  float run = p.h0 ? p.h0[i] : 0.0f;
  float* carry = p.carry + (long long)n * p.chunks * ck + at;
  const float* sumdt = p.sumdt + (long long)n * p.chunks * p.C + c;
#pragma unroll 4
  for (int q = 0; q < p.chunks; ++q) {
    const float s = carry[q * ck], d = sumdt[(long long)q * p.C];
    const float a = d == 0.0f ? 1.0f : exp2_fast(A2 * d);  // a chunk past the length keeps the state, whatever A
    carry[q * ck] = run;
    run = fmaf(a, run, s);
  }
  if (p.hT) p.hT[i] = run;
}

// A few steps: four states per thread, TPC threads per channel, the state
// read and written once in 16-byte pieces and everything else straight from
// global memory.  Bound by the state's bytes.
template <typename T, int TPC>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanParams p) {
  const long long item = ((long long)blockIdx.x * kThreads + threadIdx.x) / TPC;
  const int part = threadIdx.x % TPC;
  const bool mine = item < (long long)p.N * p.C;
  const int n = mine ? (int)(item / p.C) : 0, c = mine ? (int)(item % p.C) : 0;
  const int g = c / (p.C / p.G);
  float A2[4], h[4];
  load_states<4, TPC>(p.A + (long long)c * p.K, p.K, part, A2);
  fill(h, 0.0f);
  if (p.h0) load_states<4, TPC>(p.h0 + ((long long)n * p.C + c) * p.K, p.K, part, h);
  const int len = row_length(p.lens, n, p.S);
  const float bias = p.bias ? p.bias[c] : 0.0f, skip = p.D ? p.D[c] : 0.0f;
  for (int t = 0; t < p.S; ++t) {
    float y = 0.0f;
    if (t < len) {  // the threads of a channel share its sequence
      const float u = Elem<T>::to_f(static_cast<const T*>(p.X.p)[n * p.X.ns + t * p.X.ss + c]);
      float dt = Elem<T>::to_f(static_cast<const T*>(p.Delta.p)[n * p.Delta.ns + t * p.Delta.ss + c]) + bias;
      if (p.softplus) dt = softplus_f(dt);
      const T* B = static_cast<const T*>(p.Bm.p) + n * p.Bm.ns + t * p.Bm.ss + (long long)g * p.K;
      const T* C = static_cast<const T*>(p.Cm.p) + n * p.Cm.ns + t * p.Cm.ss + (long long)g * p.K;
      float b[4], e[4];
      if (p.bc_vec) {
        fill(b, 0.0f), fill(e, 0.0f);
        if (part * 4 < p.K) {
          Piece<T, 4>::load(B + part * 4, b);
          Piece<T, 4>::load(C + part * 4, e);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool on = part * 4 + j < p.K;
          b[j] = on ? Elem<T>::to_f(B[part * 4 + j]) : 0.0f;
          e[j] = on ? Elem<T>::to_f(C[part * 4 + j]) : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = fmaf(exp2_fast(dt * A2[j] * kLog2e), h[j], dt * u * b[j]);
        y = fmaf(e[j], h[j], y);
      }
      if (part == 0) y = fmaf(skip, u, y);
    }
#pragma unroll
    for (int o = TPC / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (mine && part == 0 && p.Y.p) {
      if (t < len && p.Z.p) {
        const float z = Elem<T>::to_f(static_cast<const T*>(p.Z.p)[n * p.Z.ns + t * p.Z.ss + c]);
        y *= z * sigmoid_fast(z);
      }
      static_cast<T*>(p.Y.p)[n * p.Y.ns + t * p.Y.ss + c] = Elem<T>::from_f(y);
    }
  }
  if (mine && p.hT) store_states<4, TPC>(p.hT + ((long long)n * p.C + c) * p.K, p.K, part, h);
}

template <typename T, int K, int TPC>
cudaError_t run_scan(const ScanParams& p, cudaStream_t s, int* launches) {
  constexpr int CH = kThreads / TPC;
  const long long tiles = (p.C / p.G + CH - 1) / CH;
  const long long blocks = (long long)p.N * p.chunks * p.G * tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (p.chunks > 1) {
    scan_kernel<T, K, TPC, false><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    const long long states = (long long)p.N * p.C * p.K;
    scan_carry_kernel<<<(unsigned)((states + 255) / 256), 256, 0, s>>>(p);
    *launches += 2;
  }
  if (p.Y.p || p.chunks == 1) {
    scan_kernel<T, K, TPC, true><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    *launches += 1;
  }
  return cudaGetLastError();
}

template <typename T, int TPC>
cudaError_t run_step(const ScanParams& p, cudaStream_t s, int* launches) {
  const long long threads = (long long)p.N * p.C * TPC;
  scan_step_kernel<T, TPC><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, s>>>(p);
  *launches += 1;
  return cudaGetLastError();
}

constexpr int kStepSeq = 4;  // sequences of at most this many steps take the step kernel

template <typename T>
cudaError_t scan_typed(const ScanParams& p, cudaStream_t s, int* launches) {
  if (p.S <= kStepSeq) {
    if (p.K <= 4) return run_step<T, 1>(p, s, launches);
    if (p.K <= 8) return run_step<T, 2>(p, s, launches);
    if (p.K <= 16) return run_step<T, 4>(p, s, launches);
    if (p.K <= 32) return run_step<T, 8>(p, s, launches);
    if (p.K <= 64) return run_step<T, 16>(p, s, launches);
    return run_step<T, 32>(p, s, launches);
  }
  if (p.K <= 4) return run_scan<T, 4, 1>(p, s, launches);
  if (p.K <= 8) return run_scan<T, 8, 1>(p, s, launches);
  if (p.K <= 16) return run_scan<T, 16, 1>(p, s, launches);
  if (p.K <= 32) return run_scan<T, 16, 2>(p, s, launches);
  if (p.K <= 64) return run_scan<T, 16, 4>(p, s, launches);
  return run_scan<T, 16, 8>(p, s, launches);
}

}  // namespace

ScanPlan scan_plan(long long seq, long long batch, long long channels, int state, int groups) {
  ScanPlan pl{};
  pl.chunks = 1;
  pl.chunk = (int)std::max<long long>(seq, 1);
  if (seq <= kStepSeq || batch == 0) return pl;
  const int tpc = state <= 16 ? 1 : state <= 32 ? 2 : state <= 64 ? 4 : 8;
  const long long per = channels / groups, ch = kThreads / tpc;
  const long long blocks = batch * groups * ((per + ch - 1) / ch);
  // blocks that fill the card: five of 128 threads per SM
  const long long want = kPlanSms * 5;
  if (blocks < want / 2) {
    const long long most = std::max<long long>(seq / 64, 1);
    const long long chunks = std::min(most, std::max<long long>(want / blocks, 1));
    if (chunks > 1) {
      pl.chunk = (int)((((seq + chunks - 1) / chunks) + kSub - 1) / kSub * kSub);
      pl.chunks = (int)((seq + pl.chunk - 1) / pl.chunk);
    }
  }
  if (pl.chunks > 1) {
    pl.carry = (batch * pl.chunks * channels * state + 3) / 4 * 4;
    pl.sumdt = (batch * pl.chunks * channels + 3) / 4 * 4;
  }
  return pl;
}

cudaError_t launch_scan(const ScanParams& p, cudaStream_t s, int* launches) {
  switch (p.dtype) {
    case RK_F32: return scan_typed<float>(p, s, launches);
    case RK_F16: return scan_typed<__half>(p, s, launches);
    default: return scan_typed<__nv_bfloat16>(p, s, launches);
  }
}

}  // namespace rk
