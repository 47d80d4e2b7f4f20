// rk_attn.h -- what the host side of the linear attention operators passes to
// their kernels: operands with element offsets applied, strides in elements,
// and the launch plans.  Not part of the ABI.
#pragma once

#include "rk_ssm.h"

struct rk_handle;

namespace rk {

// ---- queries and keys --------------------------------------------------------------

struct QkSide {          // the queries, or the keys
  RowsArg X, Y, dY, dX;  // a row of `heads` heads
  const void* scale;
  float* dscale;
  int heads;
};
struct QkParams {
  int dtype, norm, interleaved, rotary, size;
  int piece;             // elements of one access: 16 bytes' at most
  float epsilon;
  int S, N;
  int layout;
  QkSide side[2];
  const float* freq;
  const int* positions;  // by row of the layout
  const int* lens;
  float* partial;        // [blocks][2][size]
  int blocks;            // the gradient's
  int share;             // warps that share a row's heads
  int lanes;             // lanes that hold a head
};
// Elements of one access that every row, scale and pair allows.
int qk_piece(int eb, int size, int rotary, int interleaved);
int qk_grad_blocks(long long rows);
cudaError_t launch_qk(const QkParams& p, cudaStream_t s);
cudaError_t launch_qk_grad(const QkParams& p, cudaStream_t s, int* launches);

// ---- attention -----------------------------------------------------------------------

// One linear attention of rows q, k, v to o over the steps, forward or
// backward in time:
//   forward:   H = e^g H + su k v^T,  o = so H^T q
//   backward:  H = H + su k v^T,      o = so H^T q,  then H = e^g H
// The layer is one forward pass; its gradient is three: dQ is the pass of (dY,
// V, K), forward, and dV and dK are those of (K, Q, dY) and (V, dY, Q),
// backward.  H is [K, V], or its transpose as the operand has it.
struct AttnPass {
  RowsArg q, k, v, o;
  int q_of, k_of, v_of, o_of;  // heads that share one of the rows' heads
  int K, V;                    // elements of q and k; of v and o
  float su, so;
  int backward;
  int v_major;                 // a state's element (k, v) lies at [v][k]
  const float* first;          // [N][H][..], or null
  float* last;
  const float* with;           // a state like `last`: its product with what `last` is goes to cross
  float* cross;                // [N][H]
  RowsArg dot_with;            // rows like o's: their products with the unrounded o
  float* dot;                  // [N][H][S], or null
  float* o32;                  // [N * S][H][V] in o's place: heads that share are added up from there
  float* marks;                // [streams of the pass][marks][deep][128], or null: the states at the marks
};
// How a call's sequences are cut: pieces that run side by side where there are
// too few states to fill the card, and what each adds to the state.
struct AttnPlan {
  int segments, per;  // pieces of a sequence, and the chunks of 64 steps in each
  int deep;           // elements that a kernel's states have along q and k: 64 or 128
  int vec;            // rows take 16-byte pieces
  int every, marks;   // chunks from one mark to the next, and the marks of a sequence
  float* states;      // [streams][segments][deep][128]
  float* left;        // [streams][segments][2][2]: logarithms (base 2) of what a piece leaves of its first state
};
// Chunks between two of the states at which the decays' gradient is taken from
// the state and its gradient themselves: every chunk where there is a bias, whose
// gradient adds up what is lost between two, and these states of both directions
// are at most so many bytes, a quarter of L2 (512 x 2 x 16 heads of 128, 29 MB: 66 us
// for 54; 201 x 3 x 12, 14 MB: 56 for 47; 590 x 4 alone: 41 for 40).  More of them cost
// large calls a third of their time (512 x 8 x 16 heads of 128, every second chunk
// 165 us for 140), and there many heads and rows make up for it.
constexpr int kMarkChunks = 8, kNearMarkChunks = 1;
constexpr long long kNearMarkBytes = 32LL << 20;
struct AttnParams {
  int dtype;
  int S, N, H;
  RowsArg decay;
  const float* bias;
  const int* lens;
  int gradient;  // its passes, rather than the one forward pass
  int passes;
  AttnPass pass[3];
  AttnPlan plan;
};
// The longest sequences that run step by step.  16 heads with their states, 8
// steps and 12 against one chunk of 13, us: heads of 128, 1 batch row 12.4 and
// 14.8 against 12.5, 64 batch rows 52 and 68 against 82, float32 against 18.6 and
// 119; heads of 64, two to a block, 8.3 and 10.3 against 10.5, 25 and 32 against 36,
// float32 against 14.5 and 51.
constexpr int kAttnSteps = 12;
// Heads that share a block.
int attn_together(int key_size, int value_size);
// The plan of `passes` passes, its pointers left out; and the floats of its scratch.
AttnPlan attn_plan(long long seq, long long batch, long long heads, int key_size, int value_size, int passes,
                   bool bias = false);
long long attn_plan_scratch(const AttnPlan& plan, long long batch, long long heads, int key_size, int value_size,
                            int passes);
// Step by step: one forward pass.
cudaError_t launch_attn_steps(const AttnParams& p, cudaStream_t s, int* launches);
// In chunks.
cudaError_t launch_attn_chunks(const AttnParams& p, cudaStream_t s, int* launches);
cudaError_t launch_attn_chunks_f32(const AttnParams& p, cudaStream_t s, int* launches);
cudaError_t launch_attn_chunks_f16(const AttnParams& p, cudaStream_t s, int* launches);
cudaError_t launch_attn_chunks_bf16(const AttnParams& p, cudaStream_t s, int* launches);
// Whether a wait of theirs has failed on the current device; cleared.
cudaError_t take_attn_status(cudaStream_t s, int* to);
cudaError_t take_attn_status_f32(cudaStream_t s, int* to);
cudaError_t take_attn_status_f16(cudaStream_t s, int* to);
cudaError_t take_attn_status_bf16(cudaStream_t s, int* to);
// The same on behalf of one handle: the failures on the current device are
// counted by process, and every handle that has run there learns of each.
void use_attn_waits(rk_handle* h);
cudaError_t poll_attn(rk_handle* h, cudaStream_t s, int* failed);
// A wait that runs out after so many tries, for each element type's unit.
cudaError_t launch_attn_selftest(int tries, cudaStream_t s, int* launches);
cudaError_t launch_attn_selftest_f32(int tries, cudaStream_t s);
cudaError_t launch_attn_selftest_f16(int tries, cudaStream_t s);
cudaError_t launch_attn_selftest_bf16(int tries, cudaStream_t s);
constexpr int kAttnTryNs = 2000;  // one try waits for so long at most

// dDecay and d_decay_bias from the products of q and dQ (to) and k and dK (of).
struct AttnDecayParams {
  int S, N, H;
  RowsArg decay, dDecay;
  const float* bias;
  const int* lens;
  const float* to;
  const float* of;
  const float* first;  // [N][H], or null: the state's product with its gradient before the first step
  const float* last;   // and behind the last
  const float* states; // at the marks, the two passes' one after the other, and [N][H][marks] their products
  float* between;
  int every, marks, deep, together;  // heads that share a block
  double* partial;     // [N][H][tiles]
  float* dbias;        // [H], or null
  int tiles;           // set by the launch
};
int attn_decay_tiles(long long seq, int every);
cudaError_t launch_attn_decay(AttnDecayParams p, cudaStream_t s, int* launches);

// o = sums over the heads that share of o32, for up to three outputs.
struct AttnShareParams {
  int dtype, S, N, H, count;
  struct {
    int V, of;
    const float* o32;
    RowsArg o;
  } out[3];
};
cudaError_t launch_attn_share(const AttnShareParams& p, cudaStream_t s, int* launches);

}  // namespace rk
