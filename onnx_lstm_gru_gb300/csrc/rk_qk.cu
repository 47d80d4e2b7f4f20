// rk_qk.cu -- queries and keys normalised and rotated by head, and the gradient.
//
//   n = x inv w;  a' = a c - b s, b' = b c + a s for each pair (a, b) of n
//   backward: g = the turn back of dy;  dw = sum of g x inv;
//   dx = inv (g w) - x inv^3 sum(g w x) / m,  m = size (root mean square) or 1
// Both are bound by HBM: a row is read once and everything is computed in
// registers.  A warp takes a row's heads in turns, so that a row's cosines and
// sines, which all heads share, are computed once; a lane holds both elements
// of its pairs, and a head's sum is a few exchanges of lanes.
#include <algorithm>

#include "rk.h"
#include "rk_attn.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

constexpr int kQkThreads = 256, kQkWarps = kQkThreads / 32;

// Where unit u's two pieces of V elements start in a head (-1: there is none),
// and its pairs' first number (rotary / 2 and more: pairs that stay).
// Interleaved pairs are the neighbours of the two pieces, which lie side by
// side; else pieces of a pair lie half of `rotary` apart, and what is not
// rotated is dealt out the same way.
struct Unit {
  int a, b, pair;
};
template <int V>
__device__ __forceinline__ Unit unit_of(int u, int size, int rotary, bool interleaved) {
  const int half = rotary / 2;
  if (interleaved) {
    const int a = 2 * u * V;
    return {a < size ? a : -1, a + V < size ? a + V : -1, u * V};
  }
  if (u * V < half) return {u * V, u * V + half, u * V};
  const int w = u - half / V, rest = (size - rotary) / V, up = (rest + 1) / 2;
  if (w >= up) return {-1, -1, half};
  return {rotary + w * V, w + up < rest ? rotary + (w + up) * V : -1, half};
}

// Positions times frequency in turns, by 64-bit integers that wrap at a turn:
// the frequency as a fraction of 2^64 of a turn (its error is 2^-53 of it,
// which position 2^31 makes 2^-22), and the product exact.
__device__ __forceinline__ unsigned long long turn_of(float f) {
  const double t = (double)f * 0.15915494309189533576888;
  const double r = t - floor(t);
  return __double2ull_rz(r * 18446744073709551616.0);
}
__device__ __forceinline__ void turn(unsigned long long step, int position, float& c, float& s) {
  const long long phase = (long long)(step * (unsigned long long)(long long)position);
  sincospif((float)phase * 1.0842021724855044e-19f, &s, &c);  // 2^-63: in half turns
}

// LPH lanes hold a head's units, U each; pieces of V elements.
template <typename T, int V, int LPH, int U>
struct Lane {
  int a[U], b[U], pair[U];
  unsigned long long step[U][V];
  __device__ __forceinline__ void init(const QkParams& p, int sub) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit x = unit_of<V>(sub + u * LPH, p.size, p.rotary, p.interleaved);
      a[u] = x.a, b[u] = x.b, pair[u] = x.pair;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = pair[u] + i;
        step[u][i] = a[u] >= 0 && j < p.rotary / 2 ? turn_of(p.freq[j]) : 0;
      }
    }
  }
  // An infinite or NaN frequency has no turn: its pairs are NaN.
  __device__ __forceinline__ void angles(const QkParams& p, int position, float (&c)[U][V], float (&s)[U][V]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = pair[u] + i;
        c[u][i] = 1.0f, s[u][i] = 0.0f;
        if (a[u] >= 0 && j < p.rotary / 2) {
          turn(step[u][i], position, c[u][i], s[u][i]);
          const float f = p.freq[j];
          if (!(fabsf(f) <= 3.402823466e38f)) c[u][i] = s[u][i] = __int_as_float(0x7fffffff);
        }
      }
  }
  __device__ __forceinline__ bool turns(const QkParams& p, int u, int i) const { return pair[u] + i < p.rotary / 2; }
};

// A unit's elements as pairs x[0] (a) and x[1] (b).
template <typename T, int V>
__device__ __forceinline__ void load_unit(const T* row, int a, int b, bool interleaved, float (&x)[2][V]) {
  float e[2][V];
  fill(e[0], 0.0f);
  fill(e[1], 0.0f);
  if (a >= 0) Piece<T, V>::load(row + a, e[0]);
  if (b >= 0) Piece<T, V>::load(row + b, e[1]);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[0][i] = interleaved ? e[2 * i / V][2 * i % V] : e[0][i];
    x[1][i] = interleaved ? e[(2 * i + 1) / V][(2 * i + 1) % V] : e[1][i];
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_unit(T* row, int a, int b, bool interleaved, const float (&x)[2][V]) {
  float e[2][V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    e[0][i] = interleaved ? x[i % 2][i / 2] : x[0][i];
    e[1][i] = interleaved ? x[(V + i) % 2][(V + i) / 2] : x[1][i];
  }
  if (a >= 0) Piece<T, V>::store(row + a, e[0]);
  if (b >= 0) Piece<T, V>::store(row + b, e[1]);
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row r of the layout as step and batch row, and whether it holds work.
__device__ __forceinline__ bool row_of(const QkParams& p, long long r, int& s, int& n) {
  const int inner = p.layout == 0 ? p.N : p.S;
  const int o = (int)(r / inner), i = (int)(r - (long long)o * inner);
  s = p.layout == 0 ? o : i;
  n = p.layout == 0 ? i : o;
  return s < row_length(p.lens, n, p.S);
}

__device__ __forceinline__ float inverse(const QkParams& p, float square) {
  if (p.norm == 0) return 1.0f;
  return 1.0f / sqrtf((p.norm == 1 ? square / (float)p.size : square) + p.epsilon);
}

template <typename T, int V, int LPH, int U>
__global__ void __launch_bounds__(kQkThreads) qk_kernel(QkParams p) {
  constexpr int kHeads = 32 / LPH;  // heads that a warp takes at a time
  const int lane = threadIdx.x % 32, sub = lane % LPH;
  Lane<T, V, LPH, U> l;
  l.init(p, sub);
  const long long rows = (long long)p.S * p.N * p.share;
  const bool il = p.interleaved;
  for (long long w = (long long)blockIdx.x * kQkWarps + threadIdx.x / 32; w < rows; w += (long long)gridDim.x * kQkWarps) {
    const long long r = w / p.share;
    const int part = (int)(w - r * p.share);
    int s, n;
    const bool live = row_of(p, r, s, n);
    float c[U][V], sn[U][V];
    if (live) l.angles(p, p.positions ? p.positions[r] : s, c, sn);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const QkSide& q = p.side[side];
      if (q.Y.p == nullptr) continue;
      const T* X = static_cast<const T*>(q.X.p) + s * q.X.ss + n * q.X.ns;
      T* Y = static_cast<T*>(q.Y.p) + s * q.Y.ss + n * q.Y.ns;
      const T* W = static_cast<const T*>(q.scale);
#pragma unroll 2
      for (int h0 = part * kHeads; h0 < q.heads; h0 += kHeads * p.share) {
        const int h = h0 + lane / LPH;
        const bool on = h < q.heads;
        float x[U][2][V];
        float square = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          load_unit<T, V>(X + (long long)h * p.size, on && live ? l.a[u] : -1, on && live ? l.b[u] : -1, il, x[u]);
#pragma unroll
          for (int i = 0; i < V; ++i) square = fmaf(x[u][0][i], x[u][0][i], fmaf(x[u][1][i], x[u][1][i], square));
        }
        const float inv = inverse(p, p.norm ? head_sum<LPH>(square) : 0.0f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (live) {
            float sc[2][V];
            if (W) load_unit<T, V>(W, l.a[u], l.b[u], il, sc);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              float a = x[u][0][i] * inv, b = x[u][1][i] * inv;
              if (W) a *= sc[0][i], b *= sc[1][i];
              const bool t = l.turns(p, u, i);
              x[u][0][i] = t ? a * c[u][i] - b * sn[u][i] : a;
              x[u][1][i] = t ? b * c[u][i] + a * sn[u][i] : b;
            }
          }
          store_unit<T, V>(Y + (long long)h * p.size, on ? l.a[u] : -1, on ? l.b[u] : -1, il, x[u]);
        }
      }
    }
  }
}

template <typename T, int V, int LPH, int U>
__global__ void __launch_bounds__(kQkThreads) qk_grad_kernel(QkParams p) {
  constexpr int kHeads = 32 / LPH;
  const int lane = threadIdx.x % 32, sub = lane % LPH;
  Lane<T, V, LPH, U> l;
  l.init(p, sub);
  const long long rows = (long long)p.S * p.N;
  const bool il = p.interleaved;
  float dw[2][U][2][V];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < 2; ++j) fill(dw[0][u][j], 0.0f), fill(dw[1][u][j], 0.0f);
  const float m = p.norm == 1 ? 1.0f / (float)p.size : 1.0f;
  for (long long r = (long long)blockIdx.x * kQkWarps + threadIdx.x / 32; r < rows; r += (long long)gridDim.x * kQkWarps) {
    int s, n;
    const bool live = row_of(p, r, s, n);
    float c[U][V], sn[U][V];
    if (live) l.angles(p, p.positions ? p.positions[r] : s, c, sn);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkSide& q = p.side[side];
      if (q.dX.p == nullptr && q.dscale == nullptr) continue;
      const T* X = static_cast<const T*>(q.X.p) + s * q.X.ss + n * q.X.ns;
      const T* dY = static_cast<const T*>(q.dY.p) + s * q.dY.ss + n * q.dY.ns;
      T* dX = static_cast<T*>(q.dX.p) + s * q.dX.ss + n * q.dX.ns;
      const T* W = static_cast<const T*>(q.scale);
#pragma unroll 1
      for (int h0 = 0; h0 < q.heads; h0 += kHeads) {
        const int h = h0 + lane / LPH;
        const bool on = h < q.heads, work = on && live;
        float x[U][2][V], g[U][2][V];
        float square = 0.0f, dot = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          load_unit<T, V>(X + (long long)h * p.size, work ? l.a[u] : -1, work ? l.b[u] : -1, il, x[u]);
          load_unit<T, V>(dY + (long long)h * p.size, work ? l.a[u] : -1, work ? l.b[u] : -1, il, g[u]);
#pragma unroll
          for (int i = 0; i < V; ++i) square = fmaf(x[u][0][i], x[u][0][i], fmaf(x[u][1][i], x[u][1][i], square));
        }
        const float inv = inverse(p, p.norm ? head_sum<LPH>(square) : 0.0f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (live) {
            float sc[2][V];
            if (W) load_unit<T, V>(W, l.a[u], l.b[u], il, sc);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float a = g[u][0][i], b = g[u][1][i];
              const bool t = l.turns(p, u, i);
              const float ga = t ? a * c[u][i] + b * sn[u][i] : a, gb = t ? b * c[u][i] - a * sn[u][i] : b;
              if (work) {
                dw[side][u][0][i] = fmaf(ga, x[u][0][i] * inv, dw[side][u][0][i]);
                dw[side][u][1][i] = fmaf(gb, x[u][1][i] * inv, dw[side][u][1][i]);
              }
              g[u][0][i] = W ? ga * sc[0][i] : ga;
              g[u][1][i] = W ? gb * sc[1][i] : gb;
              dot = fmaf(g[u][0][i], x[u][0][i], fmaf(g[u][1][i], x[u][1][i], dot));
            }
          }
        }
        // inv (dot / m) inv inv x, from the left: inv^3 alone may pass float32's range
        const float f = p.norm ? inv * (head_sum<LPH>(dot) * m) * inv : 0.0f;
        if (q.dX.p) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (live) {
#pragma unroll
              for (int i = 0; i < V; ++i) {
                g[u][0][i] = inv * (p.norm ? g[u][0][i] - f * x[u][0][i] : g[u][0][i]);
                g[u][1][i] = inv * (p.norm ? g[u][1][i] - f * x[u][1][i] : g[u][1][i]);
              }
            }
            store_unit<T, V>(dX + (long long)h * p.size, on ? l.a[u] : -1, on ? l.b[u] : -1, il, g[u]);
          }
        }
      }
    }
  }
  if (p.partial == nullptr) return;
  // the block's sums: over the head groups of a warp, then over the warps
  __shared__ float sums[kQkWarps][256];
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = side ? dw[1][u][j][i] : dw[0][u][j][i];
#pragma unroll
          for (int o = 16; o >= LPH; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          const int at = il ? (2 * i + j < V ? l.a[u] + 2 * i + j : l.b[u] + 2 * i + j - V) : (j ? l.b[u] : l.a[u]) + i;
          const bool is = il ? (2 * i + j < V ? l.a[u] : l.b[u]) >= 0 : (j ? l.b[u] : l.a[u]) >= 0;
          if (lane < LPH && is) sums[threadIdx.x / 32][at] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < p.size; i += kQkThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kQkWarps; ++w) v += sums[w][i];
      p.partial[((long long)blockIdx.x * 2 + side) * p.size + i] = v;
    }
    __syncthreads();
  }
}

// Sums over the blocks, one warp for each element of the two scales.
__global__ void __launch_bounds__(256) qk_scale_kernel(QkParams p) {
  const int i = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (i >= 2 * p.size) return;
  float* out = i < p.size ? p.side[0].dscale : p.side[1].dscale;
  if (out == nullptr) return;
  float v = 0.0f;
  for (int b = lane; b < p.blocks; b += 32) v += p.partial[(long long)b * 2 * p.size + i];
  v = warp_sum(v);
  if (lane == 0) out[i < p.size ? i : i - p.size] = v;
}

// Units of V elements' pieces that cover a head.
int units(const QkParams& p, int V) {
  if (p.interleaved) return (p.size + 2 * V - 1) / (2 * V);
  return p.rotary / 2 / V + ((p.size - p.rotary) / V + 1) / 2;
}

template <typename T, int V, int LPH, int U, bool GRAD>
cudaError_t launch_form(const QkParams& p, cudaStream_t s) {
  if constexpr (GRAD) {
    qk_grad_kernel<T, V, LPH, U><<<p.blocks, kQkThreads, 0, s>>>(p);
  } else {
    const long long warps = (long long)p.S * p.N * p.share;
    const long long blocks = (warps + kQkWarps - 1) / kQkWarps;
    qk_kernel<T, V, LPH, U><<<(unsigned)std::min<long long>(blocks, kPlanSms * 8), kQkThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int V, bool GRAD>
cudaError_t launch_lanes(QkParams p, cudaStream_t s) {
  const int n = units(p, V);
  int lanes = 1;
  while (lanes < n && lanes < 32) lanes *= 2;
  if constexpr (V == 1) lanes = std::max(lanes, 8);
  const int turns = (std::max(p.side[0].heads, p.side[1].heads) * lanes + 31) / 32;
  const long long rows = (long long)p.S * p.N;
  // few rows: as many warps as there are turns of heads share one
  p.share = GRAD ? 1 : (int)std::max<long long>(1, std::min<long long>(turns, kPlanSms * 16 / std::max<long long>(rows, 1)));
  if constexpr (V == 1) {
    switch (lanes) {
      case 8: return launch_form<T, V, 8, 1, GRAD>(p, s);
      case 16: return launch_form<T, V, 16, 1, GRAD>(p, s);
      default: return n <= 32 ? launch_form<T, V, 32, 1, GRAD>(p, s) : launch_form<T, V, 32, 4, GRAD>(p, s);
    }
  } else {
    switch (lanes) {
      case 1: return launch_form<T, V, 1, 1, GRAD>(p, s);
      case 2: return launch_form<T, V, 2, 1, GRAD>(p, s);
      case 4: return launch_form<T, V, 4, 1, GRAD>(p, s);
      case 8: return launch_form<T, V, 8, 1, GRAD>(p, s);
      case 16: return launch_form<T, V, 16, 1, GRAD>(p, s);
      default: return launch_form<T, V, 32, 1, GRAD>(p, s);
    }
  }
}

template <bool GRAD>
cudaError_t launch_any(const QkParams& p, cudaStream_t s) {
  if (p.dtype == RK_F32)
    return p.piece == 4 ? launch_lanes<float, 4, GRAD>(p, s) : launch_lanes<float, 1, GRAD>(p, s);
  if (p.dtype == RK_F16) {
    if (p.piece == 8) return launch_lanes<__half, 8, GRAD>(p, s);
    return p.piece == 4 ? launch_lanes<__half, 4, GRAD>(p, s) : launch_lanes<__half, 1, GRAD>(p, s);
  }
  if (p.piece == 8) return launch_lanes<__nv_bfloat16, 8, GRAD>(p, s);
  return p.piece == 4 ? launch_lanes<__nv_bfloat16, 4, GRAD>(p, s) : launch_lanes<__nv_bfloat16, 1, GRAD>(p, s);
}

}  // namespace

int qk_piece(int eb, int size, int rotary, int interleaved) {
  for (int v = 16 / eb; v >= 4; v /= 2)
    if (interleaved ? size % (2 * v) == 0 : rotary / 2 % v == 0 && (size - rotary) % v == 0) return v;
  return 1;
}

int qk_grad_blocks(long long rows) {
  return (int)std::max<long long>(1, std::min<long long>((rows + kQkWarps - 1) / kQkWarps, kPlanSms * 3));
}

cudaError_t launch_qk(const QkParams& p, cudaStream_t s) { return launch_any<false>(p, s); }

cudaError_t launch_qk_grad(const QkParams& p, cudaStream_t s, int* launches) {
  cudaError_t e = launch_any<true>(p, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.partial == nullptr) return e;
  qk_scale_kernel<<<(2 * p.size + 7) / 8, 256, 0, s>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace rk
