// rk_ssm.h -- what the host side of the state space operators passes to their
// kernels: operands with element offsets applied, strides in elements, and
// the launch plan's numbers.  Not part of the ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace rk {

// SMs that the launch plans divide work over.  A constant of the chip, so
// that a problem's plan, and with it the scratch length and the order of
// every sum, follows from the problem alone.
constexpr int kPlanSms = 152;

// A row tensor: element (s, n, i) is at p[s * ss + n * ns + i].  vec: rows
// start on 16-byte boundaries and hold whole 16-byte pieces.
struct RowsArg {
  void* p;
  long long ss, ns;
  int vec;
};

// ---- layer normalisation ------------------------------------------------------

struct NormParams {
  int dtype;
  float epsilon;
  long long rows;
  int cols;
  RowsArg X, Y, dY, dX;  // ss: the row pitch; ns unused
  int vec;               // every row operand and the weights take 16-byte pieces
  const void* scale;
  const void* bias;
  float* mean;
  float* inv;
  const float* mean_in;
  const float* inv_in;
  float* dscale;
  float* dbias;
  float* partial;  // [blocks][2][cols]
  int blocks;      // most blocks of the gradient kernel
};
// Most blocks that the gradient kernel runs, one partial row of the weights' gradients each.
int norm_grad_blocks(long long rows, int cols);
cudaError_t launch_norm(const NormParams& p, cudaStream_t s);
cudaError_t launch_norm_grad(const NormParams& p, cudaStream_t s, int* launches);

// ---- causal convolution ----------------------------------------------------------

struct ConvParams {
  int dtype, width, silu;
  int S, N, C;
  RowsArg X, Y, dY, dX;
  int vec;  // every row operand, the states and the weights take 16-byte pieces
  const void* W;
  const void* B;
  const int* lens;
  const void* init;
  void* final_state;
  const void* dfinal;
  float* dW;
  float* dB;
  void* dinit;
  float* partial;  // [slices][width + 1][C]
  int slices;
  int chunk;       // steps a thread runs
};
int conv_grad_chunk(long long seq, long long batch, long long channels);
int conv_grad_slices(long long seq, long long batch, long long channels);
cudaError_t launch_conv(const ConvParams& p, cudaStream_t s);
cudaError_t launch_conv_grad(const ConvParams& p, cudaStream_t s, int* launches);

// ---- selective scan ------------------------------------------------------------------

struct ScanParams {
  int dtype, softplus;
  int S, N, C, K, G;   // K states, G groups
  RowsArg X, Delta, Bm, Cm, Z, Y;
  RowsArg dY, dX, dDelta, dB, dC, dZ;
  int vec;             // every operand with rows of C elements takes 16-byte pieces (the gradient's)
  int k_vec;           // rows of K states take 16-byte pieces
  int bc_vec;          // operands with rows of G * K take pieces of four within a group
  const float* A;
  const float* D;
  const float* bias;
  const int* lens;
  const float* h0;
  float* hT;
  const float* dhT;
  float* dA;
  float* dD;
  float* dbias;
  float* dh0;
  // plan
  int chunks;          // pieces of the sequence that run side by side
  int chunk;           // steps of each
  float* carry;        // [N][chunks][C][K]: a chunk's own final state, then the state it starts from
  float* sumdt;        // [N][chunks][C]
  // gradient
  float* gcarry;       // [N][chunks][C][K]: the same for the state's gradient, from the chunk's end
  float* ckpt;         // [N][subtiles][C][K]: states at the starts of the subtiles, from the chunk's zero start
  float* cum;          // [N][subtiles][C]: the chunk's sum of dt up to there
  float* bc_part;      // [slices][N * S][G][2][K]: sums over a slice's channels
  float* w_part;       // [N * chunks][C][K + 2]: dA, dD, d_delta_bias
  int slices;          // per group
  int slice_tiles;     // channel tiles that one block runs one after the other
};

struct ScanPlan {
  int chunks, chunk;
  // floats of each scratch region (multiples of 4), in the order they are placed
  long long carry, sumdt, gcarry, ckpt, cum, bc_part, w_part;
  int slices, slice_tiles;
  long long total() const { return carry + sumdt + gcarry + ckpt + cum + bc_part + w_part; }
};
// ragged: rows have lengths of their own.
ScanPlan scan_plan(long long seq, long long batch, long long channels, int state, int groups, bool ragged);
ScanPlan scan_grad_plan(long long seq, long long batch, long long channels, int state, int groups, bool ragged);
cudaError_t launch_scan(const ScanParams& p, cudaStream_t s, int* launches);
cudaError_t launch_scan_grad(const ScanParams& p, cudaStream_t s, int* launches);

}  // namespace rk
