// rk_norm.cu -- layer normalisation and its gradient.
//
// Both are bound by HBM: a row is read once, kept in registers, and everything
// it needs is computed from there.  The sums are taken in two passes over the
// registers (the mean, then the squares around it), which loses nothing to
// cancellation; all of them are float32 in a fixed order.
#include <algorithm>

#include "rk.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

// Sums of N values over the TPR threads of a row: shuffles inside a warp,
// shared memory across the warps of a wider row (buf: [2][N][TPR / 32], its
// halves used in turn so that one barrier per sum is enough).
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* buf, int& flip) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float* b = buf + flip * N * W;
    flip ^= 1;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) b[i * W + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += b[i * W + w];
      v[i] = s;
    }
  }
}

// TPR threads per row, NV pieces of V elements per thread: cols <= TPR * V * NV.
// Blocks of one-warp rows hold four of them; a wider row has its block alone.
template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 128) norm_kernel(NormParams p) {
  constexpr int kRows = TPR > 32 ? 1 : 128 / TPR;
  __shared__ float buf[2 * (TPR / 32)];
  int flip = 0;
  const int lane = threadIdx.x % TPR;
  const float rn = 1.0f / (float)p.cols;
  const T* scale = static_cast<const T*>(p.scale);
  const T* bias = static_cast<const T*>(p.bias);
  for (long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR; row < p.rows;
       row += (long long)gridDim.x * kRows) {
    const T* x = static_cast<const T*>(p.X.p) + row * p.X.ss;
    float v[NV][V];
    float sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * V;
      if (c < p.cols) {
        Piece<T, V>::load(x + c, v[j]);
      } else {
        fill(v[j], 0.0f);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) sum[0] += v[j][i];
    row_sum<TPR>(sum, buf, flip);
    const float mean = sum[0] * rn;
    float sq[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * V;
      if (c < p.cols) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[j][i] -= mean;
          sq[0] += v[j][i] * v[j][i];
        }
      }
    }
    row_sum<TPR>(sq, buf, flip);
    const float inv = rsqrtf(sq[0] * rn + p.epsilon);
    if (lane == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.inv) p.inv[row] = inv;
    }
    if (p.Y.p) {
      T* y = static_cast<T*>(p.Y.p) + row * p.Y.ss;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + lane) * V;
        if (c < p.cols) {
          float w[V], b[V];
          if (scale) Piece<T, V>::load(scale + c, w);
          else fill(w, 1.0f);
          if (bias) Piece<T, V>::load(bias + c, b);
          else fill(b, 0.0f);
#pragma unroll
          for (int i = 0; i < V; ++i) w[i] = fmaf(v[j][i] * inv, w[i], b[i]);
          Piece<T, V>::store(y + c, w);
        }
      }
    }
  }
}

// Rows too wide for a block's registers: read three times (from L2 after the
// first).
constexpr int kWide = 1024;
template <typename T>
__global__ void __launch_bounds__(kWide) norm_wide_kernel(NormParams p) {
  __shared__ float buf[2 * (kWide / 32)];
  int flip = 0;
  const float rn = 1.0f / (float)p.cols;
  const T* scale = static_cast<const T*>(p.scale);
  const T* bias = static_cast<const T*>(p.bias);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.X.p) + row * p.X.ss;
    float sum[1] = {0.0f};
    for (int c = threadIdx.x; c < p.cols; c += kWide) sum[0] += Elem<T>::to_f(x[c]);
    row_sum<kWide>(sum, buf, flip);
    const float mean = sum[0] * rn;
    float sq[1] = {0.0f};
    for (int c = threadIdx.x; c < p.cols; c += kWide) {
      const float d = Elem<T>::to_f(x[c]) - mean;
      sq[0] += d * d;
    }
    row_sum<kWide>(sq, buf, flip);
    const float inv = rsqrtf(sq[0] * rn + p.epsilon);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.inv) p.inv[row] = inv;
    }
    if (p.Y.p) {
      T* y = static_cast<T*>(p.Y.p) + row * p.Y.ss;
      for (int c = threadIdx.x; c < p.cols; c += kWide) {
        const float w = scale ? Elem<T>::to_f(scale[c]) : 1.0f, b = bias ? Elem<T>::to_f(bias[c]) : 0.0f;
        y[c] = Elem<T>::from_f(fmaf((Elem<T>::to_f(x[c]) - mean) * inv, w, b));
      }
    }
  }
}

// The gradient: each thread keeps the sums of its own columns over the rows
// its block runs; the block adds its rows' threads up at the end and writes
// one partial row of dScale and dB.
template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 128) norm_grad_kernel(NormParams p) {
  constexpr int kRows = TPR > 32 ? 1 : 128 / TPR;
  constexpr int kBuf = 4 * (TPR / 32);
  __shared__ float buf[kRows > 1 ? (kRows * TPR * V * 2 > kBuf ? kRows * TPR * V * 2 : kBuf) : kBuf];
  int flip = 0;
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const float rn = 1.0f / (float)p.cols;
  const T* scale = static_cast<const T*>(p.scale);
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) fill(dw[j], 0.0f), fill(db[j], 0.0f);
  for (long long row = (long long)blockIdx.x * kRows + grp; row < p.rows; row += (long long)gridDim.x * kRows) {
    const T* x = static_cast<const T*>(p.X.p) + row * p.X.ss;
    const T* dy = static_cast<const T*>(p.dY.p) + row * p.dY.ss;
    const float mean = p.mean_in[row], inv = p.inv_in[row];
    float xh[NV][V], g[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * V;
      if (c < p.cols) {
        Piece<T, V>::load(x + c, xh[j]);
        Piece<T, V>::load(dy + c, g[j]);
      } else {
        fill(xh[j], mean), fill(g[j], 0.0f);
      }
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * V;
      float w[V];
      if (scale && c < p.cols) Piece<T, V>::load(scale + c, w);
      else fill(w, 1.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xh[j][i] = (xh[j][i] - mean) * inv;
        dw[j][i] = fmaf(g[j][i], xh[j][i], dw[j][i]);
        db[j][i] += g[j][i];
        g[j][i] *= w[i];
        sum[0] += g[j][i];
        sum[1] = fmaf(g[j][i], xh[j][i], sum[1]);
      }
    }
    if (p.dX.p) {
      row_sum<TPR>(sum, buf, flip);
      const float a = sum[0] * rn, b = sum[1] * rn;
      T* dx = static_cast<T*>(p.dX.p) + row * p.dX.ss;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + lane) * V;
        if (c < p.cols) {
#pragma unroll
          for (int i = 0; i < V; ++i) g[j][i] = inv * (g[j][i] - a - xh[j][i] * b);
          Piece<T, V>::store(dx + c, g[j]);
        }
      }
    }
  }
  if (p.partial == nullptr) return;
  float* out = p.partial + (long long)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + lane) * V;
    if constexpr (kRows > 1) {
      __syncthreads();
      float* mine = buf + (grp * TPR + lane) * V * 2;
#pragma unroll
      for (int i = 0; i < V; ++i) mine[2 * i] = dw[j][i], mine[2 * i + 1] = db[j][i];
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float a = 0.0f, b = 0.0f;
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            a += buf[((r * TPR + lane) * V + i) * 2];
            b += buf[((r * TPR + lane) * V + i) * 2 + 1];
          }
          dw[j][i] = a, db[j][i] = b;
        }
      }
    }
    if (grp == 0 && c < p.cols) {
#pragma unroll
      for (int i = 0; i < V; ++i) out[c + i] = dw[j][i], out[p.cols + c + i] = db[j][i];
    }
  }
}

// The gradient of rows too wide for a block's registers: dX row by row, the
// weights' gradients column by column.
template <typename T>
__global__ void __launch_bounds__(kWide) norm_grad_wide_kernel(NormParams p) {
  __shared__ float buf[4 * (kWide / 32)];
  int flip = 0;
  const float rn = 1.0f / (float)p.cols;
  const T* scale = static_cast<const T*>(p.scale);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.X.p) + row * p.X.ss;
    const T* dy = static_cast<const T*>(p.dY.p) + row * p.dY.ss;
    T* dx = static_cast<T*>(p.dX.p) + row * p.dX.ss;
    const float mean = p.mean_in[row], inv = p.inv_in[row];
    float sum[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < p.cols; c += kWide) {
      const float g = Elem<T>::to_f(dy[c]) * (scale ? Elem<T>::to_f(scale[c]) : 1.0f);
      sum[0] += g;
      sum[1] = fmaf(g, (Elem<T>::to_f(x[c]) - mean) * inv, sum[1]);
    }
    row_sum<kWide>(sum, buf, flip);
    const float a = sum[0] * rn, b = sum[1] * rn;
    for (int c = threadIdx.x; c < p.cols; c += kWide) {
      const float g = Elem<T>::to_f(dy[c]) * (scale ? Elem<T>::to_f(scale[c]) : 1.0f);
      dx[c] = Elem<T>::from_f(inv * (g - a - (Elem<T>::to_f(x[c]) - mean) * inv * b));
    }
  }
}
template <typename T>
__global__ void __launch_bounds__(256) norm_grad_wide_weights_kernel(NormParams p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float g = Elem<T>::to_f(static_cast<const T*>(p.dY.p)[row * p.dY.ss + c]);
    const float x = Elem<T>::to_f(static_cast<const T*>(p.X.p)[row * p.X.ss + c]);
    dw = fmaf(g, (x - p.mean_in[row]) * p.inv_in[row], dw);
    db += g;
  }
  float* out = p.partial + (long long)blockIdx.y * 2 * p.cols;
  out[c] = dw, out[p.cols + c] = db;
}

// dScale and dB from the partial rows: 32 columns per block, eight threads
// per column over the rows, added in a fixed order.
__global__ void __launch_bounds__(256) norm_grad_reduce_kernel(NormParams p) {
  __shared__ float buf[8][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, part = threadIdx.x / 32;
  // columns of dScale, then of dB: a partial row is both, one after the other
  float s = 0.0f;
  if (col < 2 * p.cols) {
#pragma unroll 4
    for (int b = part; b < p.blocks; b += 8) s += p.partial[(long long)b * 2 * p.cols + col];
  }
  buf[part][threadIdx.x % 32] = s;
  __syncthreads();
  if (part == 0 && col < 2 * p.cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += buf[i][threadIdx.x];
    float* out = col < p.cols ? p.dscale : p.dbias;
    if (out) out[col < p.cols ? col : col - p.cols] = s;
  }
}

template <typename T, int V, int NV, int TPR>
cudaError_t run_norm(const NormParams& p, cudaStream_t s) {
  constexpr int kRows = TPR > 32 ? 1 : 128 / TPR;
  const long long blocks = (p.rows + kRows - 1) / kRows;
  norm_kernel<T, V, NV, TPR><<<(unsigned)std::min<long long>(blocks, 1 << 20), TPR > 32 ? TPR : 128, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int V, int NV, int TPR>
cudaError_t run_norm_grad(const NormParams& p, cudaStream_t s) {
  norm_grad_kernel<T, V, NV, TPR><<<p.blocks, TPR > 32 ? TPR : 128, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_typed(const NormParams& p, cudaStream_t s) {
  constexpr int V = kPiece<T>;
  const int c = p.cols;
  if (p.vec) {
    if (c <= 32 * V) return run_norm<T, V, 1, 32>(p, s);
    if (c <= 64 * V) return run_norm<T, V, 2, 32>(p, s);
    if (c <= 128 * V) return run_norm<T, V, 4, 32>(p, s);
    if (c <= 256 * V) return run_norm<T, V, 2, 128>(p, s);
    if (c <= 512 * V) return run_norm<T, V, 4, 128>(p, s);
    if (c <= 1024 * V) return run_norm<T, V, 4, 256>(p, s);
    if (c <= 4096 * V) return run_norm<T, V, 4, 1024>(p, s);
  } else {
    if (c <= 128) return run_norm<T, 1, 4, 32>(p, s);
    if (c <= 512) return run_norm<T, 1, 16, 32>(p, s);
    if (c <= 2048) return run_norm<T, 1, 16, 128>(p, s);
    if (c <= 4096) return run_norm<T, 1, 16, 256>(p, s);
    if (c <= 16384) return run_norm<T, 1, 16, 1024>(p, s);
  }
  norm_wide_kernel<T><<<(unsigned)std::min<long long>(p.rows, 1 << 20), kWide, 0, s>>>(p);
  return cudaGetLastError();
}

// Widest row the gradient's register form takes: 512 threads x 16 elements of
// any type and alignment.
constexpr int kGradCols = 512 * 16;

template <typename T>
cudaError_t norm_grad_typed(const NormParams& p, cudaStream_t s) {
  constexpr int V = kPiece<T>;
  const int c = p.cols;
  if (c > kGradCols) {
    if (p.dX.p && p.rows > 0)
      norm_grad_wide_kernel<T><<<(unsigned)std::min<long long>(p.rows, 1 << 20), kWide, 0, s>>>(p);
    if (p.partial)
      norm_grad_wide_weights_kernel<T><<<dim3((c + 255) / 256, p.blocks), 256, 0, s>>>(p);
    return cudaGetLastError();
  }
  if (p.vec) {
    constexpr int E = 16 / V;  // pieces of 16 elements
    if (c <= 32 * V) return run_norm_grad<T, V, 1, 32>(p, s);
    if (c <= 512) return run_norm_grad<T, V, E, 32>(p, s);
    if (c <= 1024) return run_norm_grad<T, V, 2 * E, 32>(p, s);
    if (c <= 2048) return run_norm_grad<T, V, E, 128>(p, s);
    if (c <= 4096) return run_norm_grad<T, V, E, 256>(p, s);
    return run_norm_grad<T, V, E, 512>(p, s);
  }
  if (c <= 128) return run_norm_grad<T, 1, 4, 32>(p, s);
  if (c <= 512) return run_norm_grad<T, 1, 16, 32>(p, s);
  if (c <= 1024) return run_norm_grad<T, 1, 8, 128>(p, s);
  if (c <= 4096) return run_norm_grad<T, 1, 16, 256>(p, s);
  return run_norm_grad<T, 1, 16, 512>(p, s);
}

}  // namespace

int norm_grad_blocks(int dtype, long long rows, int cols) {
  // enough blocks to fill the card, few enough that their partial rows stay small
  if (cols > kGradCols) return (int)std::min<long long>(std::max<long long>(rows, 1), 32);
  const long long groups = cols <= 1024 ? (rows + 3) / 4 : rows;
  return (int)std::min<long long>(std::max<long long>(groups, 1), kPlanSms * (cols <= 4096 ? 4 : 2));
}

cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  switch (p.dtype) {
    case RK_F32: return norm_typed<float>(p, s);
    case RK_F16: return norm_typed<__half>(p, s);
    default: return norm_typed<__nv_bfloat16>(p, s);
  }
}

cudaError_t launch_norm_grad(const NormParams& p, cudaStream_t s, int* launches) {
  cudaError_t e;
  switch (p.dtype) {
    case RK_F32: e = norm_grad_typed<float>(p, s); break;
    case RK_F16: e = norm_grad_typed<__half>(p, s); break;
    default: e = norm_grad_typed<__nv_bfloat16>(p, s);
  }
  *launches = 1;
  if (e != cudaSuccess || p.partial == nullptr) return e;
  norm_grad_reduce_kernel<<<(unsigned)((2LL * p.cols + 31) / 32), 256, 0, s>>>(p);
  *launches = 2;
  return cudaGetLastError();
}

}  // namespace rk
