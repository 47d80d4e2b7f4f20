// rk_norm.cu -- layer normalisation and its gradient.
//
// Both are bound by HBM: a row is read once, kept in registers, and everything
// it needs is computed from there.  The sums are taken in two passes over the
// registers (the mean, then the squares around it), which loses nothing to
// cancellation; all of them are float32 in a fixed order.
//   y = (x - mean) inv w + b, inv = 1 / sqrt(var + epsilon)
//   g = dy w, xh = (x - mean) inv; dx = inv (g - avg(g) - xh avg(g xh))
//   dw = sum over rows of dy xh; db = sum over rows of dy
// A block runs rows one after the other with the next ones' loads in flight.
// 32768 x 1024 bf16: forward 24.6 us (5.5 TB/s over its 134 MB), gradient 43.6
// us (4.6 TB/s over 202 MB, about 4 us of it the second launch).  The gradient
// is held back by the loads that 12 warps per SM keep in flight, which is what
// its registers leave (four rows' elements as read, and the column sums), and by
// 23 instructions per element; one or two rows at a time, packed arithmetic and
// loads that stay in L2 measured slower.
#include <algorithm>

#include "rk.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

// Sums of N values (a power of two up to 8) over the TPR threads of a row
// group, in a fixed order; every thread gets them.  Inside a warp the values
// are halved with each exchange of lanes until a lane has one; across the
// warps of a wider group they go through shared memory (two halves used in
// turn, so that one barrier per call is enough).
template <int TPR, int N>
struct RowSum {
  static constexpr int W = TPR / 32;
  __align__(16) float buf[2][W][N];
  template <int M>
  __device__ __forceinline__ void operator()(float (&v)[M], int& flip) {
    static_assert(M == N, "as many values as the buffer holds");
    const int lane = threadIdx.x % 32;
    int at = 0;
    lanes_sum<N, 16, 1>(v, lane, at);
    if constexpr (W == 1) {
      const float mine = v[0];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, mine, i * (32 / N));
    } else {
      if (lane % (32 / N) == 0) buf[flip][threadIdx.x / 32][lane / (32 / N)] = v[0];
      __syncthreads();
      if constexpr (W <= 8) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          v[i] = buf[flip][0][i];
#pragma unroll
          for (int w = 1; w < W; ++w) v[i] += buf[flip][w][i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < W ? buf[flip][lane][i] : 0.0f);
      }
      flip ^= 1;
    }
  }
};

// Threads of a block: a group of one warp shares it with three more.
template <int TPR>
constexpr int kBlock = TPR > 32 ? TPR : 128;

// Threads per SM that the registers of a form leave room for, and the blocks
// that makes: the grids are one wave of them, each block running many rows.
constexpr int kNormThreads = 640, kGradThreads = 384;
template <int TPR, int THREADS>
constexpr int kResident = THREADS / kBlock<TPR> > 0 ? THREADS / kBlock<TPR> : 1;

// TPR threads run R rows at a time, E elements of each per thread in pieces of
// V (cols <= TPR * E).  The next rows are on their way while these are
// computed.
template <typename T, int V, int E, int TPR, int R>
__global__ void __launch_bounds__(kBlock<TPR>, R > 1 ? kResident<TPR, kNormThreads> : 1) norm_kernel(NormParams p) {
  constexpr int kGroups = kBlock<TPR> / TPR, NV = E / V;
  __shared__ RowSum<TPR, R> sums;
  int flip = 0;
  const int lane = threadIdx.x % TPR;
  const float rn = 1.0f / (float)p.cols;
  const T* scale = static_cast<const T*>(p.scale);
  const T* bias = static_cast<const T*>(p.bias);
  const long long stride = (long long)gridDim.x * kGroups * R;
  const long long row = ((long long)blockIdx.x * kGroups + threadIdx.x / TPR) * R;
  const T* x = static_cast<const T*>(p.X.p) + row * p.X.ss + lane * V;
  T* y = static_cast<T*>(p.Y.p) + row * p.Y.ss + lane * V;
  float* mean_to = p.mean ? p.mean + row : nullptr;
  float* inv_to = p.inv ? p.inv + row : nullptr;
  bool on[NV];  // pieces of this thread that are columns
  Packed<T, V> next[R][NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    on[j] = (j * TPR + lane) * V < p.cols;
#pragma unroll
    for (int r = 0; r < R; ++r) next[r][j].raw = {};  // and stay 0 where they are not
  }
  auto fetch = [&](long long rows) {
    const T* at = x;
#pragma unroll
    for (int r = 0; r < R; ++r, at += p.X.ss) {
      if (r >= rows) break;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j]) next[r][j].load_streaming(at + j * TPR * V);
    }
    x += stride * p.X.ss;
  };
  long long left = p.rows - row;  // from this thread's next row on
  fetch(left);
  for (; left > 0; left -= stride) {
    // past the last row: an earlier one again, not stored
    const int rows = (int)min(left, (long long)R);
    float v[R][NV][V], mean[R], inv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        next[r][j].widen(v[r][j]);
#pragma unroll
        for (int i = 0; i < V; ++i) mean[r] += v[r][j][i];
      }
    }
    fetch(left - stride);
    sums(mean, flip);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] *= rn;
      inv[r] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[r][j][i] -= mean[r];
          inv[r] = fmaf(v[r][j][i], v[r][j][i], inv[r]);
        }
      }
    }
    sums(inv, flip);
#pragma unroll
    for (int r = 0; r < R; ++r) inv[r] = rsqrtf(inv[r] * rn + p.epsilon);
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        if (mean_to) mean_to[r] = mean[r];
        if (inv_to) inv_to[r] = inv[r];
      }
    }
    if (mean_to) mean_to += stride;
    if (inv_to) inv_to += stride;
    if (!p.Y.p) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
      const int c = (j * TPR + lane) * V;
      float w[V], b[V];
      if (scale) Piece<T, V>::load(scale + c, w);
      else fill(w, 1.0f);
      if (bias) Piece<T, V>::load(bias + c, b);
      else fill(b, 0.0f);
      T* at = y + j * TPR * V;
#pragma unroll
      for (int r = 0; r < R; ++r, at += p.Y.ss) {
        if (r >= rows) break;
#pragma unroll
        for (int i = 0; i < V; ++i) v[r][j][i] = fmaf(v[r][j][i] * inv[r], w[i], b[i]);
        Packed<T, V> out;
        out.narrow(v[r][j]);
        out.store_streaming(at);
      }
    }
    y += stride * p.Y.ss;
  }
}

// The sum of one value over a block.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, RowSum<THREADS, 1>& sums, int& flip) {
  float a[1] = {v};
  sums(a, flip);
  return a[0];
}

// Rows too wide for a block's registers: read three times (from L2 after the
// first).  2048 x 16384 bf16: 53.8 us, against 41.4 for the register form, which
// ends there.
constexpr int kWide = 1024;
template <typename T>
__global__ void __launch_bounds__(kWide) norm_wide_kernel(NormParams p) {
  __shared__ RowSum<kWide, 1> sums;
  int flip = 0;
  const float rn = 1.0f / (float)p.cols;
  const T* scale = static_cast<const T*>(p.scale);
  const T* bias = static_cast<const T*>(p.bias);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.X.p) + row * p.X.ss;
    float sum = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += kWide) sum += Elem<T>::to_f(x[c]);
    const float mean = block_sum(sum, sums, flip) * rn;
    float sq = 0.0f;
    for (int c = threadIdx.x; c < p.cols; c += kWide) {
      const float d = Elem<T>::to_f(x[c]) - mean;
      sq += d * d;
    }
    const float inv = rsqrtf(block_sum(sq, sums, flip) * rn + p.epsilon);
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

// The gradient: R rows at a time as above; each thread keeps the sums of its
// own columns over the rows its block runs, and the block writes one partial
// row of dScale and dB.
template <typename T, int V, int E, int TPR, int R>
__global__ void __launch_bounds__(kBlock<TPR>, kResident<TPR, kGradThreads>) norm_grad_kernel(NormParams p) {
  constexpr int kGroups = kBlock<TPR> / TPR, NV = E / V;
  __shared__ RowSum<TPR, 2 * R> sums;
  __shared__ float cols[kGroups > 1 ? kBlock<TPR> * V * 2 : 1];
  int flip = 0;
  next_may_start();
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const float rn = 1.0f / (float)p.cols;
  const T* scale = static_cast<const T*>(p.scale);
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) fill(dw[j], 0.0f), fill(db[j], 0.0f);
  const long long stride = (long long)gridDim.x * kGroups * R;
  const long long row = ((long long)blockIdx.x * kGroups + grp) * R;
  const T* x = static_cast<const T*>(p.X.p) + row * p.X.ss + lane * V;
  const T* dy = static_cast<const T*>(p.dY.p) + row * p.dY.ss + lane * V;
  T* dx = static_cast<T*>(p.dX.p) + row * p.dX.ss + lane * V;
  const float *mean = p.mean_in + row, *scale_of = p.inv_in + row;
  bool on[NV];  // pieces of this thread that are columns
#pragma unroll
  for (int j = 0; j < NV; ++j) on[j] = (j * TPR + lane) * V < p.cols;
  Packed<T, V> nx[R][NV], ny[R][NV];
  float nmean[R], ninv[R];
  auto fetch = [&](long long rows) {
    const T *ax = x, *ay = dy;
#pragma unroll
    for (int r = 0; r < R; ++r, ax += p.X.ss, ay += p.dY.ss) {
      if (r >= rows) break;
      nmean[r] = mean[r], ninv[r] = scale_of[r];
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j]) nx[r][j].load_streaming(ax + j * TPR * V), ny[r][j].load_streaming(ay + j * TPR * V);
    }
    x += stride * p.X.ss, dy += stride * p.dY.ss, mean += stride, scale_of += stride;
  };
  long long left = p.rows - row;  // from this thread's next row on
  fetch(left);
  for (; left > 0; left -= stride) {
    const int rows = (int)min(left, (long long)R);
    float xh[R][NV][V], g[R][NV][V], inv[R], sum[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) inv[r] = ninv[r], sum[r] = sum[R + r] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
      float w[V];
      if (scale) Piece<T, V>::load(scale + (j * TPR + lane) * V, w);
      else fill(w, 1.0f);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        nx[r][j].widen(xh[r][j]);
        ny[r][j].widen(g[r][j]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float& a = xh[r][j][i];
          float& y = g[r][j][i];
          a = (a - nmean[r]) * inv[r];
          dw[j][i] = fmaf(y, a, dw[j][i]);
          db[j][i] += y;
          y *= w[i];
          sum[r] += y;
          sum[R + r] = fmaf(y, a, sum[R + r]);
        }
      }
    }
    fetch(left - stride);
    if (!p.dX.p) continue;
    sums(sum, flip);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!on[j]) continue;
      T* at = dx + j * TPR * V;
#pragma unroll
      for (int r = 0; r < R; ++r, at += p.dX.ss) {
        if (r >= rows) break;
        const float a = sum[r] * rn, b = sum[R + r] * rn;
#pragma unroll
        for (int i = 0; i < V; ++i) g[r][j][i] = inv[r] * (g[r][j][i] - a - xh[r][j][i] * b);
        Packed<T, V> out;
        out.narrow(g[r][j]);
        out.store_streaming(at);
      }
    }
    dx += stride * p.dX.ss;
  }
  if (p.partial == nullptr) return;
  float* out = p.partial + (long long)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + lane) * V;
    if constexpr (kGroups > 1) {
      __syncthreads();
      float* mine = cols + (grp * TPR + lane) * V * 2;
#pragma unroll
      for (int i = 0; i < V; ++i) mine[2 * i] = dw[j][i], mine[2 * i + 1] = db[j][i];
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float a = 0.0f, b = 0.0f;
#pragma unroll
          for (int r = 0; r < kGroups; ++r) {
            a += cols[((r * TPR + lane) * V + i) * 2];
            b += cols[((r * TPR + lane) * V + i) * 2 + 1];
          }
          dw[j][i] = a, db[j][i] = b;
        }
      }
    }
    if (grp == 0 && c < p.cols) {
      // rows of the partial sums start anywhere: single floats
#pragma unroll
      for (int i = 0; i < V; ++i) out[c + i] = dw[j][i], out[p.cols + c + i] = db[j][i];
    }
  }
}

// The gradient of rows too wide for a block's registers: dX row by row, the
// weights' gradients column by column.
template <typename T>
__global__ void __launch_bounds__(kWide) norm_grad_wide_kernel(NormParams p) {
  __shared__ RowSum<kWide, 2> sums;
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
    sums(sum, flip);
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
  next_may_start();
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

// dScale and dB from the partial rows: 8 columns per block, 32 threads per
// column over the rows, added in a fixed order.  All loads of a thread are in
// flight at once: bound by one round trip to L2.
constexpr int kParts = 32, kReduceCols = 8;
__global__ void __launch_bounds__(kReduceCols * kParts) norm_grad_reduce_kernel(NormParams p) {
  __shared__ float buf[kParts][kReduceCols + 1];
  const int lane = threadIdx.x % kReduceCols, part = threadIdx.x / kReduceCols;
  // columns of dScale, then of dB: a partial row is both, one after the other
  const int all = 2 * p.cols, col = blockIdx.x * kReduceCols + lane;
  constexpr int kBatch = 16;
  float s = 0.0f;
  previous_done();
  if (col < all) {
    const float* at = p.partial + (long long)part * all + col;
    for (int b = part; b < p.blocks; b += kParts * kBatch) {
      float v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i, at += (long long)kParts * all) v[i] = b + i * kParts < p.blocks ? *at : 0.0f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) s += v[i];
    }
  }
  buf[part][lane] = s;
  __syncthreads();
  // a warp adds a column's parts up
  const int warp = threadIdx.x / 32, out_col = blockIdx.x * kReduceCols + warp;
  s = warp_sum(buf[threadIdx.x % 32][warp]);
  if (threadIdx.x % 32 == 0 && out_col < all) {
    float* out = out_col < p.cols ? p.dscale : p.dbias;
    if (out) out[out_col < p.cols ? out_col : out_col - p.cols] = s;
  }
}

template <typename T, int V, int E, int TPR>
cudaError_t run_norm(const NormParams& p, cudaStream_t s) {
  constexpr int kGroups = kBlock<TPR> / TPR, kRows = E > 8 || TPR > 512 ? 1 : TPR > 256 ? 2 : 4;
  const long long full = kPlanSms * kResident<TPR, kNormThreads>;
  // Rows one by one where that is what it takes to give every SM some: x 1024
  // bf16, 256 rows 3.4 us against 4.1 with four at a time, 1024 rows 4.0 and
  // 4.3, 1536 rows (just past the rule) 5.2 and 4.3, 8192 rows 10.3 and 8.3.
  if (kRows == 1 || p.rows < full * kGroups * kRows / 2) {
    const long long blocks = (p.rows + kGroups - 1) / kGroups;
    norm_kernel<T, V, E, TPR, 1><<<(unsigned)std::min(blocks, kPlanSms * 16LL), kBlock<TPR>, 0, s>>>(p);
  } else {
    const long long blocks = (p.rows + kGroups * kRows - 1) / (kGroups * kRows);
    norm_kernel<T, V, E, TPR, kRows><<<(unsigned)std::min(blocks, full), kBlock<TPR>, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_typed(const NormParams& p, cudaStream_t s) {
  constexpr int V = kPiece<T>;
  const int c = p.cols;
  if (p.vec) {
    if (c <= 256) return run_norm<T, V, 8, 32>(p, s);
    if (c <= 512) return run_norm<T, V, 8, 64>(p, s);
    if (c <= 1024) return run_norm<T, V, 8, 128>(p, s);
    if (c <= 2048) return run_norm<T, V, 8, 256>(p, s);
    if (c <= 4096) return run_norm<T, V, 8, 512>(p, s);
    if (c <= 8192) return run_norm<T, V, 8, 1024>(p, s);
    if (c <= 16384) return run_norm<T, V, 16, 1024>(p, s);
  } else {
    if (c <= 256) return run_norm<T, 1, 8, 32>(p, s);
    if (c <= 1024) return run_norm<T, 1, 8, 128>(p, s);
    if (c <= 4096) return run_norm<T, 1, 8, 512>(p, s);
    if (c <= 16384) return run_norm<T, 1, 16, 1024>(p, s);
  }
  norm_wide_kernel<T><<<(unsigned)std::min<long long>(p.rows, 1 << 20), kWide, 0, s>>>(p);
  return cudaGetLastError();
}

// The gradient's form for a width: threads per row group and rows at a time.
// Eight elements per thread and row up to 8192 columns, then the wide form
// (2048 x 8192 bf16: 39.5 us in registers, 64.1 in the wide form; sixteen
// elements per thread do not fit next to the column sums).
constexpr int kGradCols = 8192;
int grad_threads(int cols, bool vec) {
  if (vec)
    for (int t = 32; t < 512; t *= 2)
      if (cols <= 8 * t) return t;
  return cols <= 256 ? 32 : cols <= 1024 ? 128 : cols <= 4096 ? 512 : 1024;
}
template <typename T, int V, int TPR, int R>
cudaError_t run_norm_grad(NormParams& p, cudaStream_t s) {
  // as few blocks as take the same number of turns: each writes a partial row
  constexpr long long kTurn = kBlock<TPR> / TPR * R, kFull = kPlanSms * kResident<TPR, kGradThreads>;
  const long long turns = std::max((p.rows + kTurn - 1) / kTurn, 1LL), most = std::min<long long>(p.blocks, kFull);
  const long long each = (turns + most - 1) / most;
  p.blocks = (int)((turns + each - 1) / each);
  norm_grad_kernel<T, V, 8, TPR, R><<<p.blocks, kBlock<TPR>, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int TPR>
cudaError_t norm_grad_rows(NormParams& p, cudaStream_t s) {
  // rows at a time: what the registers hold twice, as read and as floats
  constexpr int R = TPR == 1024 ? 1 : sizeof(T) == 2 && TPR < 512 ? 4 : 2;
  if (p.vec) return run_norm_grad<T, kPiece<T>, TPR, R>(p, s);
  if constexpr (TPR != 64 && TPR != 256) {
    // Element by element one row leaves more warps the room to wait in, until
    // there are many rows (x 777 float32: 2048 rows 10.4 us against 12.4 with
    // two at a time, 8192 rows 18.8 both, 32768 rows 68.2 and 57.8).
    if constexpr (R > 1) {
      if (p.rows > 16LL * kPlanSms * kResident<TPR, kGradThreads> * (kBlock<TPR> / TPR))
        return run_norm_grad<T, 1, TPR, 2>(p, s);
    }
    return run_norm_grad<T, 1, TPR, 1>(p, s);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t norm_grad_typed(NormParams& p, cudaStream_t s) {
  const int c = p.cols;
  if (c > kGradCols) {
    if (p.dX.p)
      norm_grad_wide_kernel<T><<<(unsigned)std::min<long long>(p.rows, 1 << 20), kWide, 0, s>>>(p);
    if (p.partial)
      norm_grad_wide_weights_kernel<T><<<dim3((c + 255) / 256, p.blocks), 256, 0, s>>>(p);
    return cudaGetLastError();
  }
  switch (grad_threads(c, p.vec)) {
    case 32: return norm_grad_rows<T, 32>(p, s);
    case 64: return norm_grad_rows<T, 64>(p, s);
    case 128: return norm_grad_rows<T, 128>(p, s);
    case 256: return norm_grad_rows<T, 256>(p, s);
    case 512: return norm_grad_rows<T, 512>(p, s);
    default: return norm_grad_rows<T, 1024>(p, s);
  }
}

}  // namespace

int norm_grad_blocks(long long rows, int cols) {
  rows = std::max<long long>(rows, 1);
  if (cols > kGradCols) return (int)std::min<long long>(rows, 32);
  auto most = [&](bool vec) {
    const int tpr = grad_threads(cols, vec), block = tpr > 32 ? tpr : 128, groups = block / tpr;
    return (int)std::min<long long>((rows + groups - 1) / groups, kPlanSms * std::max(kGradThreads / block, 1));
  };
  return std::max(most(false), most(true));
}

cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  switch (p.dtype) {
    case RK_F32: return norm_typed<float>(p, s);
    case RK_F16: return norm_typed<__half>(p, s);
    default: return norm_typed<__nv_bfloat16>(p, s);
  }
}

cudaError_t launch_norm_grad(const NormParams& all, cudaStream_t s, int* launches) {
  NormParams p = all;
  cudaError_t e;
  switch (p.dtype) {
    case RK_F32: e = norm_grad_typed<float>(p, s); break;
    case RK_F16: e = norm_grad_typed<__half>(p, s); break;
    default: e = norm_grad_typed<__nv_bfloat16>(p, s);
  }
  // wide rows: a launch for dX, one for the weights' partial sums
  *launches = p.cols > kGradCols ? (p.dX.p != nullptr) + (p.partial != nullptr) : 1;
  if (e != cudaSuccess || p.partial == nullptr) return e;
  *launches += 1;
  return launch_chained(norm_grad_reduce_kernel, (unsigned)((2LL * p.cols + kReduceCols - 1) / kReduceCols),
                        kReduceCols * kParts, 0, s, p);
}

}  // namespace rk
