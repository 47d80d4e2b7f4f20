// rk_scan_grad.cu -- the gradient of the selective scan.
//
// With e the state's gradient on its way back, step s from the last to the
// first does, per channel and state,
//   g = e + C dy;  dC += dy h;  dB += (dt u) g;  du += dt B g;
//   x = g a h_before;  ddt += A x + u B g;  dA += dt x;  e = a g.
// It needs the states in reverse order.  They are computed again rather than
// kept: a pass forward leaves the state at the start of every subtile in
// global memory, and the way back runs one subtile at a time, forward with
// its states in shared memory and then back.  Of the few bytes per element
// that the gradient reads and writes none is per state.
//
// Four states per thread, TPC threads per channel.  dB and dC are sums over
// the channels of a group: over a warp's channels by shuffles, over a block's
// warps in shared memory, over the blocks in a second launch that adds their
// slices in order.  dA, dD and d_delta_bias are sums over steps and
// sequences, kept per block and added the same way.
//
// Chunks of one sequence that run side by side are joined as in the forward
// scan; e is linear in what arrives at a chunk's end with the same factor
// exp(A sum dt), so one launch prepares both directions.
#include <algorithm>

#include "rk.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Steps of a subtile, by threads per channel: what the shared memory of two
// blocks per SM holds.
constexpr int sub_steps(int tpc) { return (tpc == 2 || tpc == 4) ? 16 : 8; }
constexpr int tpc_of(int states) {
  return states <= 4 ? 1 : states <= 8 ? 2 : states <= 16 ? 4 : states <= 32 ? 8 : states <= 64 ? 16 : 32;
}

template <int TPC>
struct GradShape {
  static constexpr int CH = kThreads / TPC, NSP = 4 * TPC, T = sub_steps(TPC);
  // floats of shared memory: dt, u, dy, two sums and y per (step, channel);
  // B, C; the states; the warps' sums of dB and dC; per-channel constants
  static constexpr int kRows = T * CH;
  static constexpr size_t smem =
      sizeof(float) * (6 * kRows + 2 * T * NSP + T * kThreads * 4 + T * kWarps * 2 * NSP + 2 * CH);
};

// A row piece (step t + r, channels x..) of a block's tile, or zeros.
template <typename T, int V>
__device__ __forceinline__ void tile_load(const RowsArg& a, int n, int s, int c, float (&o)[V]) {
  Piece<T, V>::load(static_cast<const T*>(a.p) + n * a.ns + s * a.ss + c, o);
}
template <typename T, int V>
__device__ __forceinline__ void tile_store(const RowsArg& a, int n, int s, int c, const float (&o)[V]) {
  Piece<T, V>::store(static_cast<T*>(a.p) + n * a.ns + s * a.ss + c, o);
}

template <typename T, int V, int NSP, int TT>
__device__ __forceinline__ void stage_group(const RowsArg& src, int n, int g, int states, int t, int live,
                                            float* dst) {
  constexpr int kPieces = NSP / V;
  for (int i = threadIdx.x; i < TT * kPieces; i += kThreads) {
    const int r = i / kPieces, k = i % kPieces * V;
    float v[V];
    if (t + r < live && k < states) {
      Piece<T, V>::load(static_cast<const T*>(src.p) + n * src.ns + (t + r) * src.ss + (long long)g * states + k, v);
    } else {
      fill(v, 0.0f);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) dst[r * NSP + k + j] = v[j];
  }
}

// What every kernel here works on: one channel tile of one group of one
// chunk of one sequence.
template <typename T, int TPC>
struct Tile {
  using Sh = GradShape<TPC>;
  static constexpr int CH = Sh::CH, NSP = Sh::NSP, TT = Sh::T;
  const ScanParams& p;
  int n, g, c0, width, t0, t1, live;
  float *dt, *u, *dy, *sB, *sC, *bias, *skip;

  template <int V>
  __device__ __forceinline__ void stage_v(int t, bool grads) {
    constexpr int kPieces = CH / V > 0 ? CH / V : 1;
    for (int i = threadIdx.x; i < TT * kPieces; i += kThreads) {
      const int r = i / kPieces, x = i % kPieces * V;
      float d[V], uu[V], gy[V];
      if (t + r < live && x < width) {
        tile_load<T, V>(p.Delta, n, t + r, c0 + x, d);
        tile_load<T, V>(p.X, n, t + r, c0 + x, uu);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          d[j] += bias[x + j];
          if (p.softplus) d[j] = softplus_f(d[j]);
        }
        if (grads) {
          tile_load<T, V>(p.dY, n, t + r, c0 + x, gy);
          if (p.Z.p) {
            float z[V];
            tile_load<T, V>(p.Z, n, t + r, c0 + x, z);
#pragma unroll
            for (int j = 0; j < V; ++j) gy[j] *= z[j] * sigmoid_fast(z[j]);
          }
        }
      } else {
        fill(d, 0.0f), fill(uu, 0.0f), fill(gy, 0.0f);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dt[r * CH + x + j] = d[j];
        u[r * CH + x + j] = uu[j];
        if (grads) dy[r * CH + x + j] = gy[j];
      }
    }
  }
  __device__ __forceinline__ void stage(int t, bool grads) {
    constexpr int V = kPiece<T>;
    if (CH >= V && p.vec) stage_v<(CH >= V ? V : 1)>(t, grads);
    else stage_v<1>(t, grads);
    if (p.bc_vec) {
      stage_group<T, 4, NSP, TT>(p.Bm, n, g, p.K, t, live, sB);
      if (grads) stage_group<T, 4, NSP, TT>(p.Cm, n, g, p.K, t, live, sC);
    } else {
      stage_group<T, 1, NSP, TT>(p.Bm, n, g, p.K, t, live, sB);
      if (grads) stage_group<T, 1, NSP, TT>(p.Cm, n, g, p.K, t, live, sC);
    }
  }
  __device__ __forceinline__ void constants() {
    for (int i = threadIdx.x; i < CH; i += kThreads) {
      bias[i] = (p.bias && i < width) ? p.bias[c0 + i] : 0.0f;
      skip[i] = (p.D && i < width) ? p.D[c0 + i] : 0.0f;
    }
  }
};

// Every chunk's final state from zero, its sum of dt, and what leaves its
// start of the state's gradient when nothing arrives at its end:
// sum over its steps of (product of a from the chunk's start) C dy.
template <typename T, int TPC>
__global__ void __launch_bounds__(kThreads) scan_grad_chunks_kernel(ScanParams p) {
  using Sh = GradShape<TPC>;
  constexpr int CH = Sh::CH, NSP = Sh::NSP, TT = Sh::T;
  __shared__ __align__(16) float sB[TT * NSP], sC[TT * NSP];
  __shared__ float sdt[TT * CH], su[TT * CH], sdy[TT * CH], sbias[CH], sskip[CH];
  const int per = p.C / p.G, tiles = (per + CH - 1) / CH;
  const int tile = blockIdx.x % tiles;
  int q = blockIdx.x / tiles;
  const int g = q % p.G;
  q /= p.G;
  const int chunk = q % p.chunks, n = q / p.chunks;
  const int t0 = chunk * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const int live = min(t1, row_length(p.lens, n, p.S));
  Tile<T, TPC> b{p, n, g, g * per + tile * CH, min(CH, per - tile * CH), t0, t1, live,
                 sdt, su, sdy, sB, sC, sbias, sskip};
  const int lc = threadIdx.x / TPC, part = threadIdx.x % TPC;
  const bool mine = lc < b.width;
  const int c = b.c0 + (mine ? lc : 0);
  b.constants();
  float A2[4], h[4], pr[4], e[4];
  load_states<4, TPC>(p.A + (long long)c * p.K, p.K, part, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= kLog2e, h[i] = 0.0f, pr[i] = 1.0f, e[i] = 0.0f;
  float sum = 0.0f;
  __syncthreads();
  for (int t = t0; t < live; t += TT) {
    b.stage(t, true);
    __syncthreads();
    const int steps = min(TT, live - t);
    for (int r = 0; r < steps; ++r) {
      const float dt = sdt[r * CH + lc], dtu = dt * su[r * CH + lc], dy = sdy[r * CH + lc];
      const float4 B = *reinterpret_cast<const float4*>(&sB[r * NSP + part * 4]);
      const float4 C = *reinterpret_cast<const float4*>(&sC[r * NSP + part * 4]);
      const float bb[4] = {B.x, B.y, B.z, B.w}, cc[4] = {C.x, C.y, C.z, C.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = exp2_fast(dt * A2[i]);
        h[i] = fmaf(a, h[i], dtu * bb[i]);
        pr[i] *= a;
        e[i] = fmaf(pr[i], cc[i] * dy, e[i]);
      }
      sum += dt;
    }
    __syncthreads();
  }
  if (mine) {
    const long long row = ((long long)n * p.chunks + chunk) * p.C + c;
    store_states<4, TPC>(p.carry + row * p.K, p.K, part, h);
    store_states<4, TPC>(p.gcarry + row * p.K, p.K, part, e);
    if (part == 0) p.sumdt[row] = sum;
  }
}

// The chunks in order, forward for the states and backward for their gradient.
__global__ void __launch_bounds__(256) scan_grad_carry_kernel(ScanParams p) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long ck = (long long)p.C * p.K;
  if (i >= p.N * ck) return;
  const int n = (int)(i / ck);
  const long long at = i % ck;
  const float A2 = p.A[at] * kLog2e;
  const long long base = (long long)n * p.chunks * ck + at;
  const float* sumdt = p.sumdt + (long long)n * p.chunks * p.C + at / p.K;
  if (blockIdx.y == 0) {
    float run = p.h0 ? p.h0[i] : 0.0f;
#pragma unroll 4
    for (int q = 0; q < p.chunks; ++q) {
      const float s = p.carry[base + q * ck], d = sumdt[(long long)q * p.C];
      p.carry[base + q * ck] = run;
      run = fmaf(d == 0.0f ? 1.0f : exp2_fast(A2 * d), run, s);
    }
  } else {
    float run = p.dhT ? p.dhT[i] : 0.0f;
#pragma unroll 4
    for (int q = p.chunks - 1; q >= 0; --q) {
      const float s = p.gcarry[base + q * ck], d = sumdt[(long long)q * p.C];
      p.gcarry[base + q * ck] = run;
      run = fmaf(d == 0.0f ? 1.0f : exp2_fast(A2 * d), run, s);
    }
    if (p.dh0) p.dh0[i] = run;
  }
}

template <typename T, int TPC>
__global__ void __launch_bounds__(kThreads) scan_grad_kernel(ScanParams p) {
  using Sh = GradShape<TPC>;
  constexpr int CH = Sh::CH, NSP = Sh::NSP, TT = Sh::T, kRows = Sh::kRows;
  extern __shared__ __align__(16) float smem[];
  float4* sh = reinterpret_cast<float4*>(smem);            // [TT][kThreads]
  float* sB = smem + TT * kThreads * 4;                    // [TT][NSP]
  float* sC = sB + TT * NSP;
  float* spart = sC + TT * NSP;                            // [TT][kWarps][2][NSP]
  float* sdt = spart + TT * kWarps * 2 * NSP;              // [TT][CH], and the next five
  float* su = sdt + kRows;
  float* sdy = su + kRows;
  float* sgb = sdy + kRows;  // sum of g B, then ddelta
  float* sth = sgb + kRows;  // sum of A x, then dy u
  float* sy = sth + kRows;   // sum of C h
  float* sbias = sy + kRows;
  float* sskip = sbias + CH;
  const int per = p.C / p.G, tiles = (per + CH - 1) / CH;
  const int slice = blockIdx.x % p.slices;
  int q = blockIdx.x / p.slices;
  const int g = q % p.G;
  q /= p.G;
  const int chunk = q % p.chunks, n = q / p.chunks;
  const int t0 = chunk * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const int live = min(t1, row_length(p.lens, n, p.S));
  const int lc = threadIdx.x / TPC, part = threadIdx.x % TPC;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int subs = (p.S + TT - 1) / TT;
  const long long chunk_row = (long long)n * p.chunks + chunk;

  for (int tile = slice * p.slice_tiles; tile < min((slice + 1) * p.slice_tiles, tiles); ++tile) {
    const bool first = tile == slice * p.slice_tiles;
    Tile<T, TPC> b{p, n, g, g * per + tile * CH, min(CH, per - tile * CH), t0, t1, live,
                   sdt, su, sdy, sB, sC, sbias, sskip};
    const bool mine = lc < b.width;
    const int c = b.c0 + (mine ? lc : 0);
    __syncthreads();
    b.constants();
    float A2[4], h[4];
    fill(A2, 0.0f), fill(h, 0.0f);  // what a thread without a channel keeps: it adds 0 to its warp's sums
    if (mine) load_states<4, TPC>(p.A + (long long)c * p.K, p.K, part, A2);
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] *= kLog2e;
    if (!mine) {
    } else if (p.chunks > 1) load_states<4, TPC>(p.carry + (chunk_row * p.C + c) * p.K, p.K, part, h);
    else if (p.h0) load_states<4, TPC>(p.h0 + ((long long)n * p.C + c) * p.K, p.K, part, h);
    auto ckpt = [&](int t) { return p.ckpt + (((long long)n * subs + t / TT) * p.C + c) * p.K; };
    __syncthreads();

    // forward: the state at the start of each subtile
    int last = t0;
    for (int t = t0; t < live; t += TT) {
      last = t;
      if (mine) store_states<4, TPC>(ckpt(t), p.K, part, h);
      if (t + TT >= live) break;
      b.stage(t, false);
      __syncthreads();
#pragma unroll 4
      for (int r = 0; r < TT; ++r) {
        const float dt = sdt[r * CH + lc], dtu = dt * su[r * CH + lc];
        const float4 B = *reinterpret_cast<const float4*>(&sB[r * NSP + part * 4]);
        const float bb[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = fmaf(exp2_fast(dt * A2[i]), h[i], dtu * bb[i]);
      }
      __syncthreads();
    }

    // backward, one subtile at a time
    float e[4], dA[4], dD = 0.0f, dbias = 0.0f;
    fill(e, 0.0f), fill(dA, 0.0f);
    if (!mine) {
    } else if (p.chunks > 1) load_states<4, TPC>(p.gcarry + (chunk_row * p.C + c) * p.K, p.K, part, e);
    else if (p.dhT) load_states<4, TPC>(p.dhT + ((long long)n * p.C + c) * p.K, p.K, part, e);
    for (int t = last; t >= t0 && live > t0; t -= TT) {
      const int steps = min(TT, live - t);
      b.stage(t, true);
      float start[4];
      fill(start, 0.0f);
      if (mine) load_states<4, TPC>(ckpt(t), p.K, part, start);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = start[i];
#pragma unroll 4
      for (int r = 0; r < steps; ++r) {
        const float dt = sdt[r * CH + lc], dtu = dt * su[r * CH + lc];
        const float4 B = *reinterpret_cast<const float4*>(&sB[r * NSP + part * 4]);
        const float bb[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = fmaf(exp2_fast(dt * A2[i]), h[i], dtu * bb[i]);
        sh[r * kThreads + threadIdx.x] = make_float4(h[0], h[1], h[2], h[3]);
        if (p.Z.p) {
          const float4 C = *reinterpret_cast<const float4*>(&sC[r * NSP + part * 4]);
          float y = h[0] * C.x + h[1] * C.y + h[2] * C.z + h[3] * C.w;
#pragma unroll
          for (int o = TPC / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
          if (part == 0) sy[r * CH + lc] = y;
        }
      }
#pragma unroll 2
      for (int r = steps - 1; r >= 0; --r) {
        const float dt = sdt[r * CH + lc], dtu = dt * su[r * CH + lc], dy = sdy[r * CH + lc];
        const float4 B = *reinterpret_cast<const float4*>(&sB[r * NSP + part * 4]);
        const float4 C = *reinterpret_cast<const float4*>(&sC[r * NSP + part * 4]);
        const float bb[4] = {B.x, B.y, B.z, B.w}, cc[4] = {C.x, C.y, C.z, C.w};
        float before[4];
        if (r > 0) {
          const float4 v = sh[(r - 1) * kThreads + threadIdx.x];
          before[0] = v.x, before[1] = v.y, before[2] = v.z, before[3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) before[i] = start[i];
        }
        float gb = 0.0f, th = 0.0f, vb[4], vc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = exp2_fast(dt * A2[i]);
          const float gg = fmaf(cc[i], dy, e[i]);
          vc[i] = h[i] * dy;
          vb[i] = gg * dtu;
          gb = fmaf(gg, bb[i], gb);
          e[i] = gg * a;
          const float x = e[i] * before[i];
          th = fmaf(x, A2[i], th);
          dA[i] = fmaf(x, dt, dA[i]);
          h[i] = before[i];
        }
#pragma unroll
        for (int o = TPC / 2; o > 0; o >>= 1) {
          gb += __shfl_xor_sync(0xffffffffu, gb, o);
          th += __shfl_xor_sync(0xffffffffu, th, o);
        }
        if (part == 0) sgb[r * CH + lc] = gb, sth[r * CH + lc] = th * (1.0f / kLog2e);
#pragma unroll
        for (int o = 16; o >= TPC; o >>= 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            vb[i] += __shfl_xor_sync(0xffffffffu, vb[i], o);
            vc[i] += __shfl_xor_sync(0xffffffffu, vc[i], o);
          }
        }
        if (lane < TPC) {
          float* to = spart + (r * kWarps + warp) * 2 * NSP + part * 4;
          *reinterpret_cast<float4*>(to) = make_float4(vb[0], vb[1], vb[2], vb[3]);
          *reinterpret_cast<float4*>(to + NSP) = make_float4(vc[0], vc[1], vc[2], vc[3]);
        }
      }
      __syncthreads();
      // the subtile's row gradients
      auto emit = [&](auto piece) {
        constexpr int V = decltype(piece)::value;
        constexpr int kPieces = CH / V > 0 ? CH / V : 1;
        for (int i = threadIdx.x; i < steps * kPieces; i += kThreads) {
          const int r = i / kPieces, x = i % kPieces * V;
          if (x >= b.width) continue;
          const int s = t + r;
          float du[V], dd[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int at = r * CH + x + j;
            const float gb = sgb[at], uu = su[at];
            du[j] = fmaf(gb, sdt[at], sskip[x + j] * sdy[at]);
            dd[j] = fmaf(gb, uu, sth[at]);
            sth[at] = sdy[at] * uu;
          }
          if (p.softplus) {
            float raw[V];
            tile_load<T, V>(p.Delta, n, s, b.c0 + x, raw);
#pragma unroll
            for (int j = 0; j < V; ++j) dd[j] *= sigmoid_fast(raw[j] + sbias[x + j]);
          }
#pragma unroll
          for (int j = 0; j < V; ++j) sgb[r * CH + x + j] = dd[j];
          if (p.dX.p) tile_store<T, V>(p.dX, n, s, b.c0 + x, du);
          if (p.dDelta.p) tile_store<T, V>(p.dDelta, n, s, b.c0 + x, dd);
          if (p.dZ.p) {
            float z[V], gy[V];
            tile_load<T, V>(p.Z, n, s, b.c0 + x, z);
            tile_load<T, V>(p.dY, n, s, b.c0 + x, gy);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const int at = r * CH + x + j;
              const float sg = sigmoid_fast(z[j]);
              const float y = fmaf(sskip[x + j], su[at], sy[at]);
              gy[j] *= y * sg * (1.0f + z[j] * (1.0f - sg));
            }
            tile_store<T, V>(p.dZ, n, s, b.c0 + x, gy);
          }
        }
      };
      constexpr int V = kPiece<T>;
      if (CH >= V && p.vec) emit(std::integral_constant<int, (CH >= V ? V : 1)>{});
      else emit(std::integral_constant<int, 1>{});
      if (p.bc_part) {
        for (int i = threadIdx.x; i < steps * 2 * NSP; i += kThreads) {
          const int r = i / (2 * NSP), j = i % (2 * NSP);
          const int k = j % NSP;
          if (k >= p.K) continue;
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += spart[(r * kWarps + w) * 2 * NSP + j];
          float* to = p.bc_part + ((((long long)slice * p.N + n) * p.S + t + r) * p.G + g) * 2 * p.K + (j / NSP) * p.K + k;
          *to = first ? v : *to + v;
        }
      }
      __syncthreads();
      if (threadIdx.x < CH && threadIdx.x < b.width) {
        for (int r = 0; r < steps; ++r) {
          dbias += sgb[r * CH + threadIdx.x];
          dD += sth[r * CH + threadIdx.x];
        }
      }
      __syncthreads();
    }

    // what is left: zeros past the length, the state's gradient, the sums over the chunk's steps
    const int from = max(t0, live);
    for (int i = threadIdx.x; i < CH; i += kThreads) {
      if (i >= b.width) continue;
      for (int t = from; t < t1; ++t) {
        const float zero[1] = {0.0f};
        if (p.dX.p) tile_store<T, 1>(p.dX, n, t, b.c0 + i, zero);
        if (p.dDelta.p) tile_store<T, 1>(p.dDelta, n, t, b.c0 + i, zero);
        if (p.dZ.p) tile_store<T, 1>(p.dZ, n, t, b.c0 + i, zero);
      }
    }
    if (mine && p.chunks == 1 && p.dh0)
      store_states<4, TPC>(p.dh0 + ((long long)n * p.C + c) * p.K, p.K, part, e);
    if (p.w_part) {
      float* w = p.w_part + chunk_row * p.C * (p.K + 2);
      if (mine) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (part * 4 + i < p.K) w[(long long)c * p.K + part * 4 + i] = dA[i];
      }
      w += (long long)p.C * p.K;
      if (threadIdx.x < CH && threadIdx.x < b.width) {
        w[b.c0 + threadIdx.x] = dD;
        w[p.C + b.c0 + threadIdx.x] = dbias;
      }
    }
  }
}

// dB and dC from the slices, in order; zeros past the length.
template <typename T>
__global__ void __launch_bounds__(256) scan_grad_rows_kernel(ScanParams p) {
  const int row = p.G * 2 * p.K;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long all = (long long)p.N * p.S * row;
  if (i >= all) return;
  const int j = (int)(i % row);
  const long long ns = i / row;
  const int s = (int)(ns % p.S), n = (int)(ns / p.S);
  const int g = j / (2 * p.K), which = j / p.K % 2, k = j % p.K;
  float v = 0.0f;
  if (s < row_length(p.lens, n, p.S)) {
#pragma unroll 8
    for (int q = 0; q < p.slices; ++q) v += p.bc_part[q * all + i];
  }
  const RowsArg& to = which ? p.dC : p.dB;
  if (to.p) static_cast<T*>(to.p)[n * to.ns + s * to.ss + (long long)g * p.K + k] = Elem<T>::from_f(v);
}

// dA, dD and d_delta_bias from the sequences' and chunks' sums, in a fixed order.
__global__ void __launch_bounds__(256) scan_grad_weights_kernel(ScanParams p) {
  __shared__ float buf[8][33];
  const long long cols = (long long)p.C * (p.K + 2);
  const long long col = (long long)blockIdx.x * 32 + threadIdx.x % 32;
  const int part = threadIdx.x / 32;
  const long long rows = (long long)p.N * p.chunks;
  float s = 0.0f;
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

template <typename T, int TPC>
cudaError_t run_grad(const ScanParams& p, cudaStream_t s, int* launches) {
  using Sh = GradShape<TPC>;
  const long long tiles = (p.C / p.G + Sh::CH - 1) / Sh::CH;
  const long long rest = (long long)p.N * p.chunks * p.G;
  if (rest * tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(scan_grad_kernel<T, TPC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Sh::smem);
  if (e != cudaSuccess) return e;
  if (p.chunks > 1) {
    scan_grad_chunks_kernel<T, TPC><<<(unsigned)(rest * tiles), kThreads, 0, s>>>(p);
    const long long states = (long long)p.N * p.C * p.K;
    scan_grad_carry_kernel<<<dim3((unsigned)((states + 255) / 256), 2), 256, 0, s>>>(p);
    *launches += 2;
  }
  scan_grad_kernel<T, TPC><<<(unsigned)(rest * p.slices), kThreads, Sh::smem, s>>>(p);
  *launches += 1;
  if (p.bc_part) {
    const long long all = (long long)p.N * p.S * p.G * 2 * p.K;
    scan_grad_rows_kernel<T><<<(unsigned)((all + 255) / 256), 256, 0, s>>>(p);
    *launches += 1;
  }
  if (p.w_part) {
    scan_grad_weights_kernel<<<(unsigned)(((long long)p.C * (p.K + 2) + 31) / 32), 256, 0, s>>>(p);
    *launches += 1;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t grad_typed(const ScanParams& p, cudaStream_t s, int* launches) {
  switch (tpc_of(p.K)) {
    case 1: return run_grad<T, 1>(p, s, launches);
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

ScanPlan scan_grad_plan(long long seq, long long batch, long long channels, int state, int groups) {
  ScanPlan pl{};
  pl.chunks = 1;
  pl.chunk = (int)std::max<long long>(seq, 1);
  pl.slices = pl.slice_tiles = 1;
  if (seq == 0 || batch == 0) return pl;
  const int tpc = tpc_of(state), sub = sub_steps(tpc);
  const long long per = channels / groups, ch = kThreads / tpc;
  const long long tiles = (per + ch - 1) / ch;
  const long long blocks = batch * groups * tiles;
  const long long want = kPlanSms * 2;
  if (blocks < want / 2) {
    const long long most = std::max<long long>(seq / 64, 1);
    const long long chunks = std::min(most, std::max<long long>(want / blocks, 1));
    if (chunks > 1) {
      pl.chunk = (int)((((seq + chunks - 1) / chunks) + 15) / 16 * 16);
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
  pl.ckpt = up4(batch * ((seq + sub - 1) / sub) * channels * state);
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
