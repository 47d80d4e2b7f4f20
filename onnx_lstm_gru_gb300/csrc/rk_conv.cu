// rk_conv.cu -- short causal convolution of each channel, its SiLU and its
// gradient.
//
// Bound by HBM: each input element is used by `width` outputs, so a thread
// runs along the steps of one 16-byte piece of channels with the last
// width - 1 inputs in registers, and neighbouring threads hold neighbouring
// pieces.  The sequence is cut into chunks that run side by side; a chunk
// reads the width - 1 inputs before it once more (from L2).
//   p[s] = b + sum_j w[j] x[s - (width - 1) + j], y = p sigmoid(p) or p
// 512 steps x 8 x 2048 Half, width 4, half of the steps past their length: 8.3
// us, the floor of its bytes being 3.8: two waves of blocks, mostly starting and
// draining them.  4096 x 4 x 2048 bf16 without lengths: 31.1 us (4.3 TB/s) over
// seven waves; a block loads all it needs, computes and ends, so nothing of its
// own is on the way while it computes, and three of its eleven rows are read
// again.
#include <algorithm>

#include "rk.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

// Steps of a forward chunk: all of its inputs are on their way at once (512 x 8 x
// 2048 bf16: 10.4 us, with 16 steps 12.4; 4096 x 4 x 2048 31.3 and 37.3).  At
// least width - 1, so that only the first chunk's thread reads the initial
// state, which the same thread may then overwrite with the final state.
constexpr int kFwdChunk = 8;

template <typename T, int V>
__device__ __forceinline__ const T* row_at(const RowsArg& a, int s, int n) {
  return static_cast<const T*>(a.p) + s * a.ss + n * a.ns;
}

// The input of step s of a sequence: a row of X, of the initial state before
// step 0, or 0.
template <typename T, int V, int W>
__device__ __forceinline__ void load_input(const ConvParams& p, int s, int n, int c, float (&o)[V]) {
  if (s >= 0) {
    Piece<T, V>::load(row_at<T, V>(p.X, s, n) + c, o);
  } else if (p.init != nullptr) {
    Piece<T, V>::load(static_cast<const T*>(p.init) + ((long long)n * (W - 1) + s + W - 1) * p.C + c, o);
  } else {
    fill(o, 0.0f);
  }
}

// The taps of V channels, which lie together: w[j][i] is tap j of channel i.
template <typename T, int V, int W>
__device__ __forceinline__ void load_taps(const ConvParams& p, int c, float (&w)[W][V], float (&b)[V]) {
  const T* at = static_cast<const T*>(p.W) + (long long)c * W;
  float t[W][V];
#pragma unroll
  for (int j = 0; j < W; ++j) Piece<T, V>::load(at + j * V, t[j]);
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) w[j][i] = t[(i * W + j) / V][(i * W + j) % V];
  if (p.B) Piece<T, V>::load(static_cast<const T*>(p.B) + c, b);
  else fill(b, 0.0f);
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(128) conv_kernel(ConvParams p) {
  const int pieces = p.C / V;
  const int chunks = (p.S + kFwdChunk - 1) / kFwdChunk;
  const long long item = (long long)blockIdx.x * 128 + threadIdx.x;
  if (item >= (long long)pieces * chunks * p.N) return;
  const unsigned q = (unsigned)(item / pieces);  // fits: chunks and N are at most 2^31 together
  const int c = (int)(item - (long long)q * pieces) * V;
  const int k = (int)(q % chunks), n = (int)(q / chunks);
  const int len = row_length(p.lens, n, p.S);
  const int s0 = k * kFwdChunk, s1 = min(s0 + kFwdChunk, p.S), live = min(s1, len);
  if (p.Y.p) {
    T* y = static_cast<T*>(p.Y.p) + n * p.Y.ns + s0 * p.Y.ss + c;
    if (s0 < live) {
      Packed<T, V> raw[kFwdChunk + W - 1];  // the inputs of steps s0 - (W - 1) ..
      const T* in = static_cast<const T*>(p.X.p) + n * p.X.ns + (s0 - (W - 1)) * p.X.ss + c;
      const T* init = static_cast<const T*>(p.init) + ((long long)n * (W - 1) + s0) * p.C + c;
#pragma unroll
      for (int j = 0; j < kFwdChunk + W - 1; ++j, in += p.X.ss, init += p.C) {
        const int s = s0 - (W - 1) + j;
        raw[j].raw = {};
        if (s >= 0) {
          if (s < live) raw[j].load(in);
        } else if (j < W - 1 && p.init) {
          raw[j].load(init);
        }
      }
      float w[W][V], b[V], x[W][V];  // x[j]: the input of step s - (W - 1) + j
      load_taps<T, V, W>(p, c, w, b);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) raw[j].widen(x[j + 1]);
#pragma unroll
      for (int r = 0; r < kFwdChunk; ++r, y += p.Y.ss) {
        if (s0 + r >= live) break;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) x[j][i] = x[j + 1][i];
        raw[r + W - 1].widen(x[W - 1]);
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          o[i] = b[i];
#pragma unroll
          for (int j = 0; j < W; ++j) o[i] = fmaf(w[j][i], x[j][i], o[i]);
          if (p.silu) o[i] *= sigmoid_of<T>(o[i]);
        }
        Piece<T, V>::store(y, o);
      }
    }
    float zero[V];
    fill(zero, 0.0f);
    T* past = static_cast<T*>(p.Y.p) + n * p.Y.ns + c;
    for (int s = max(s0, live); s < s1; ++s) Piece<T, V>::store(past + s * p.Y.ss, zero);
  }
  if (k == 0 && p.final_state) {
    // rows in increasing order: row j of the new state is row j + len of the
    // old one, read before it is overwritten
    T* f = static_cast<T*>(p.final_state) + (long long)n * (W - 1) * p.C + c;
    float x[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_input<T, V, W>(p, len - (W - 1) + j, n, c, x[j]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) Piece<T, V>::store(f + (long long)j * p.C, x[j]);
  }
}

// The gradient.  Per step s of the chunk the pre-activation is computed again
// from the inputs, dp[s] = dy[s] act'(p[s]) joins the last width of them, and
// dx[s - (W - 1)] = sum_j W[j] dp[s - j] is complete.  The W - 1 steps after
// the chunk are run for their dp alone.  Steps go in groups of four, the next
// group's elements on their way.  A block is 32 pieces of channels by
// kGradRows chunks; its weights' gradients are added up in shared memory and
// written as one slice.  512 x 8 x 2048 bf16, width 4: 24.3 us with the second
// launch's 3.8 (50 MB: 2.1 TB/s); bound by its instructions, 39 per element,
// most of them for the pre-activation, SiLU's slope, dx and dw, and by the
// registers (two groups' elements, inputs, gradients, taps), which leave few
// warps.
constexpr int kGradRows = 4;
constexpr int kGroup = 4;  // steps loaded ahead

template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * kGradRows) conv_grad_kernel(ConvParams p) {
  __shared__ float sums[kGradRows][32 * V];
  next_may_start();
  const int lane = threadIdx.x % 32, part = threadIdx.x / 32;
  const int tiles = (p.C / V + 31) / 32;
  const int tile = blockIdx.x % tiles, slice = blockIdx.x / tiles;
  const int c = (tile * 32 + lane) * V;
  const int chunks = (p.S + p.chunk - 1) / p.chunk;
  const long long q = (long long)slice * kGradRows + part;  // which chunk of which sequence
  const long long n64 = q / chunks;
  const int n = (int)min(n64, (long long)p.N), k = (int)(q % chunks);
  float dw[W + 1][V];
#pragma unroll
  for (int j = 0; j <= W; ++j) fill(dw[j], 0.0f);
  if (c < p.C && n < p.N) {
    const int len = row_length(p.lens, n, p.S);
    const int s0 = k * p.chunk, s1 = min(s0 + p.chunk, p.S);
    const int end = min(s1 + W - 1, len), own = min(s1, len);  // steps from here on are none, or another chunk's
    float w[W][V], b[V];
    load_taps<T, V, W>(p, c, w, b);
    float probe = 0.0f;  // NaN where a weight is infinite or none
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) probe = fmaf(w[j][i], 0.0f, probe);
    const bool special = probe != 0.0f;
    // the inputs and the pre-activations' gradients of a group's steps and the
    // W - 1 before it
    float x[W - 1 + kGroup][V], dp[W - 1 + kGroup][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      fill(dp[kGroup + j], 0.0f);
      if (s0 < len) load_input<T, V, W>(p, s0 - (W - 1) + j, n, c, x[kGroup + j]);
      else fill(x[kGroup + j], 0.0f);
    }
    T* dx = p.dX.p ? static_cast<T*>(p.dX.p) + n * p.dX.ns + (s0 - (W - 1)) * p.dX.ss + c : nullptr;
    const T* df = p.dfinal ? static_cast<const T*>(p.dfinal) + (long long)n * (W - 1) * p.C + c : nullptr;
    T* di = (p.dinit && k == 0) ? static_cast<T*>(p.dinit) + (long long)n * (W - 1) * p.C + c : nullptr;
    // the next group's inputs and gradients, on their way while one is computed
    Packed<T, V> nx[kGroup], ny[kGroup];
    const T* in = row_at<T, V>(p.X, s0, n) + c;
    const T* gr = row_at<T, V>(p.dY, s0, n) + c;
    auto fetch = [&](int s) {
#pragma unroll
      for (int q = 0; q < kGroup; ++q, in += p.X.ss, gr += p.dY.ss)
        if (s + q < end) nx[q].load(in), ny[q].load(gr);
    };
    // one group; inside: all of its steps are the chunk's own and within the
    // length, and the inputs it completes are the chunk's
    auto group = [&](int first, auto inside) {
      constexpr bool kInside = decltype(inside)::value;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) x[j][i] = x[kGroup + j][i], dp[j][i] = dp[kGroup + j][i];
#pragma unroll
      for (int q = 0; q < kGroup; ++q) {
        if (kInside || first + q < end) nx[q].widen(x[W - 1 + q]), ny[q].widen(dp[W - 1 + q]);
        else fill(x[W - 1 + q], 0.0f), fill(dp[W - 1 + q], 0.0f);
      }
      fetch(first + kGroup);
#pragma unroll
      for (int q = 0; q < kGroup; ++q) {
        float(&d)[V] = dp[W - 1 + q];
        // past the length d stays 0, whatever the last inputs and the weights
        // would make of a step there
        const bool on = kInside || first + q < end;
        if (p.silu && on) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float pre = b[i];
#pragma unroll
            for (int j = 0; j < W; ++j) pre = fmaf(w[j][i], x[q + j][i], pre);
            const float sg = sigmoid_of<T>(pre);
            d[i] *= sg * fmaf(pre, 1.0f - sg, 1.0f);
          }
        }
        // the steps after the chunk are another's: their gradients count for
        // this one's inputs alone
        if (kInside || first + q < own) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][i] = fmaf(d[i], x[q + j][i], dw[j][i]);
            dw[W][i] += d[i];
          }
        }
        const int t = first + q - (W - 1);  // the input whose gradient is complete
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          o[i] = w[0][i] * dp[W - 1 + q][i];
#pragma unroll
          for (int j = 1; j < W; ++j) o[i] = fmaf(w[j][i], dp[W - 1 + q - j][i], o[i]);
        }
        if (!kInside && special) {  // their products with steps that there are not are not 0: left out
          fill(o, 0.0f);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            if (first + q - j < s0 || first + q - j >= end) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = fmaf(w[j][i], dp[W - 1 + q - j][i], o[i]);
          }
        }
        if (kInside) {
          if (dx) Piece<T, V>::store(dx, o);
        } else if (t < s1) {
          const int f = t - len + (W - 1);  // the row of the final state that this input is
          if (df && f >= 0 && f < W - 1) {
            float g[V];
            Piece<T, V>::load(df + (long long)f * p.C, g);
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] += g[i];
          }
          // before the chunk: another chunk's input, or a row of the initial state
          if (t >= s0 && dx) Piece<T, V>::store(dx, o);
          else if (t < 0 && di) Piece<T, V>::store(di + (long long)(t + W - 1) * p.C, o);
        }
        if (dx) dx += p.dX.ss;
      }
    };
    fetch(s0);
    for (int first = s0; first < s1 + W - 1; first += kGroup) {
      if (first - (W - 1) >= s0 && first + kGroup <= own) group(first, std::true_type{});
      else group(first, std::false_type{});
    }
  }
  if (p.partial == nullptr) return;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) sums[part][lane * V + i] = dw[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 32 * kGradRows) {
      const int ch = tile * 32 * V + i;
      float a = 0.0f;
#pragma unroll
      for (int r = 0; r < kGradRows; ++r) a += sums[r][i];
      if (ch < p.C) p.partial[((long long)slice * (W + 1) + j) * p.C + ch] = a;
    }
  }
}

// dW and dB from the slices, added in a fixed order.
__global__ void __launch_bounds__(256) conv_grad_reduce_kernel(ConvParams p) {
  __shared__ float buf[8][33];
  const int taps = p.width + 1;
  const int col = blockIdx.x * 32 + threadIdx.x % 32, part = threadIdx.x / 32;  // tap-major
  const int cols = taps * p.C;
  float s = 0.0f;
  previous_done();
  if (col < cols) {
#pragma unroll 4
    for (int b = part; b < p.slices; b += 8) s += p.partial[(long long)b * cols + col];
  }
  buf[part][threadIdx.x % 32] = s;
  __syncthreads();
  if (part == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += buf[i][threadIdx.x];
    const int j = col / p.C, c = col % p.C;
    if (j < p.width) {
      if (p.dW) p.dW[(long long)c * p.width + j] = s;
    } else if (p.dB) {
      p.dB[c] = s;
    }
  }
}

template <typename T, int V, int W>
cudaError_t run_conv(const ConvParams& p, cudaStream_t s) {
  const long long items = (long long)(p.C / V) * ((p.S + kFwdChunk - 1) / kFwdChunk) * p.N;
  conv_kernel<T, V, W><<<(unsigned)((items + 127) / 128), 128, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t run_conv_grad(const ConvParams& p, cudaStream_t s) {
  conv_grad_kernel<T, V, W><<<(unsigned)((p.C / V + 31) / 32 * p.slices), 32 * kGradRows, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, bool GRAD>
cudaError_t by_width(const ConvParams& p, cudaStream_t s) {
#define RK_CONV_WIDTH(w)                                       \
  case w:                                                      \
    if constexpr (GRAD) return run_conv_grad<T, V, w>(p, s);   \
    else return run_conv<T, V, w>(p, s);
  switch (p.width) {
    RK_CONV_WIDTH(1)
    RK_CONV_WIDTH(2)
    RK_CONV_WIDTH(3)
    RK_CONV_WIDTH(4)
    RK_CONV_WIDTH(5)
    RK_CONV_WIDTH(6)
    RK_CONV_WIDTH(7)
    RK_CONV_WIDTH(8)
  }
#undef RK_CONV_WIDTH
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t conv_typed(const ConvParams& p, cudaStream_t s, bool grad) {
  // the gradient keeps twice the registers of the forward pass per channel:
  // pieces of 8 bytes (512 x 8 x 2048 bf16: 23.0 us, with 16 bytes 33.2)
  constexpr int VG = sizeof(T) == 4 ? 2 : 4;
  if (grad) return p.vec ? by_width<T, VG, true>(p, s) : by_width<T, 1, true>(p, s);
  return p.vec ? by_width<T, kPiece<T>, false>(p, s) : by_width<T, 1, false>(p, s);
}

cudaError_t conv_any(const ConvParams& p, cudaStream_t s, bool grad) {
  switch (p.dtype) {
    case RK_F32: return conv_typed<float>(p, s, grad);
    case RK_F16: return conv_typed<__half>(p, s, grad);
    default: return conv_typed<__nv_bfloat16>(p, s, grad);
  }
}

}  // namespace

// Steps of a gradient's chunk: up to 64, beyond which the steps after a chunk
// that are run twice no longer show; fewer where that leaves SMs without their
// six warps (512x8x2048 bf16: 30.7 us with chunks of 16, 27.9 with 32, 24.6
// with 64).
int conv_grad_chunk(long long seq, long long batch, long long channels) {
  const long long warps = kPlanSms * 6, tiles = (channels + 127) / 128;
  const long long steps = seq * batch * tiles / warps / kGroup * kGroup;
  return (int)std::min(std::max(steps, 8LL), 64LL);
}

int conv_grad_slices(long long seq, long long batch, long long channels) {
  const long long chunk = conv_grad_chunk(seq, batch, channels);
  return (int)(((seq + chunk - 1) / chunk * batch + kGradRows - 1) / kGradRows);
}

cudaError_t launch_conv(const ConvParams& p, cudaStream_t s) { return conv_any(p, s, false); }

cudaError_t launch_conv_grad(const ConvParams& p, cudaStream_t s, int* launches) {
  *launches = 0;
  cudaError_t e = cudaSuccess;
  if (p.slices > 0) {
    e = conv_any(p, s, true);
    *launches += 1;
  }
  if (e != cudaSuccess || p.partial == nullptr) return e;
  const long long cols = (long long)(p.width + 1) * p.C;
  *launches += 1;
  return launch_chained(conv_grad_reduce_kernel, (unsigned)((cols + 31) / 32), 256, 0, s, p);
}

}  // namespace rk
