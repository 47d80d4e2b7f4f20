// rk_scan.cu -- selective scan: prompts (many steps) and single tokens.
//
// Per step, channel and state: one exponential, a = exp(dt A), and the update
// h = a h + (dt u) B, y += C h.  A thread keeps K states of one channel in
// registers and runs along the steps; TPC neighbouring threads share a channel
// of more states and add their parts of y by shuffles.  B and C are the same
// for all channels of a group: the block stages them in shared memory as
// float32.  A channel's own elements go from global memory to its thread.
//
// One sequence of a few thousand channels does not fill the card, so the
// sequence is cut into chunks that run side by side.  The state that leaves a
// chunk is linear in the one that enters it, h_out = exp(A sum dt) h_in + S:
// one launch computes every chunk's S and sum dt from a zero start, a second
// runs through the chunks in order, and a third starts each chunk from its
// state and computes the outputs.
//
// Bound by instructions and the latency between them, not by bytes: one
// exponential (the unit takes 32 lanes per clock and SM) and three (states) or
// four (outputs) multiply-adds per step, channel and state.  Two states to a
// packed register halve the issue slots of the multiply-adds.  4096 steps x 1
// sequence x 2048 channels x 16 states, bf16 with a gate: 92 us, of which
// states 38, carry 6, outputs 52; the exponentials of both passes would take
// 28 us alone, the bytes 10.  One thread per channel of 16 states keeps the
// sum for y in registers; two channels per thread, one-warp blocks with
// asynchronous copies, groups of two steps and six blocks per SM all measured
// 50 to 56 us for the outputs.
#include <algorithm>
#include <type_traits>

#include "rk.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

constexpr int kThreads = 128;  // most threads of a block
constexpr int kBlocks = 5;     // of them per SM: what 96 registers per thread leave room for
constexpr int kGroup = 4;      // steps whose elements are loaded ahead, while the group before is computed

// Steps of B and C staged at once.
template <int PADDED>
constexpr int kSubSteps = PADDED <= 32 ? 16 : 8;

// Threads per channel, for 16 states per thread.
constexpr int tpc_of(int states) { return states <= 16 ? 1 : states <= 32 ? 2 : states <= 64 ? 4 : 8; }

// Threads of a block: the most whose channel tiles waste little of a group.
int block_threads(int per, int states) {
  const int tpc = tpc_of(states);
  auto padded = [&](int nt) {
    const long long ch = nt / tpc;
    return (per + ch - 1) / ch * ch;
  };
  for (int nt = kThreads; nt > 32; nt /= 2)
    if (padded(nt) * 15 <= padded(32) * 16) return nt;
  return 32;
}

// B and C of a subtile in shared memory, as float32: B's steps, then C's.
template <typename T, int NSP, int TT, bool WITH_C>
struct GroupTile {
  static constexpr int kRow = NSP / 4;  // float4s of a step's row
  static constexpr int kQuads = TT * kRow;
  static constexpr int kAll = WITH_C ? 2 * kQuads : kQuads;
  float4 v[kAll];

  __device__ __forceinline__ void put(const ScanParams& p, int n, int g, int t, int live) {
    for (int i = threadIdx.x; i < kAll; i += blockDim.x) {
      const bool is_c = WITH_C && i >= kQuads;
      const RowsArg& src = is_c ? p.Cm : p.Bm;
      const int j = is_c ? i - kQuads : i;
      const int s = t + j / kRow, k = j % kRow * 4;
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (s < live && k < p.K) {
        const T* from = static_cast<const T*>(src.p) + n * src.ns + s * src.ss + (long long)g * p.K + k;
        if (p.bc_vec) {
          Piece<T, 4>::load(from, x);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k + e < p.K) x[e] = Elem<T>::to_f(from[e]);
        }
      }
      v[i] = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
};

// K states of one channel per thread, TPC threads per channel, two states to
// a packed register.  OUT: the outputs, each chunk from its own start; else
// every chunk's final state from zero and its sum of dt.  A group's elements
// are loaded while the group before is computed; two buffers of B and C need
// one barrier per subtile.
template <typename T, int K, int TPC, bool OUT>
__global__ void __launch_bounds__(kThreads, kBlocks) scan_kernel(ScanParams p) {
  constexpr int NSP = K * TPC, TT = kSubSteps<NSP>, P = K / 2;
  using Tile = GroupTile<T, NSP, TT, OUT>;
  __shared__ Tile bc[2];
  if (!OUT) next_may_start();
  const int CH = blockDim.x / TPC;
  const int per = p.C / p.G, tiles = (per + CH - 1) / CH;
  const int tile = blockIdx.x % tiles;
  int q = blockIdx.x / tiles;
  const int g = q % p.G;
  q /= p.G;
  const int chunk = q % p.chunks, n = q / p.chunks;
  const int t0 = chunk * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const int live = min(t1, row_length(p.lens, n, p.S));
  const int lc = tile * CH + threadIdx.x / TPC, part = threadIdx.x % TPC;
  const bool mine = lc < per;
  const int c = g * per + (mine ? lc : 0);
  const long long row = ((long long)n * p.chunks + chunk) * p.C + c;

  const T* delta = static_cast<const T*>(p.Delta.p) + n * p.Delta.ns + t0 * p.Delta.ss + c;
  const T* x = static_cast<const T*>(p.X.p) + n * p.X.ns + t0 * p.X.ss + c;
  const T* z = OUT && p.Z.p ? static_cast<const T*>(p.Z.p) + n * p.Z.ns + t0 * p.Z.ss + c : nullptr;
  T* y = OUT && p.Y.p ? static_cast<T*>(p.Y.p) + n * p.Y.ns + t0 * p.Y.ss + c : nullptr;
  const bool stores = y != nullptr && mine && part == 0;
  // elements of the next group; the pointers stand at its first step
  T nd[kGroup], nu[kGroup], nz[kGroup];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (t + i < live) {
        nd[i] = *delta, nu[i] = *x;
        delta += p.Delta.ss, x += p.X.ss;
        if (OUT && z) {
          nz[i] = *z;
          z += p.Z.ss;
        }
      }
    }
  };
  if (t0 < live) {
    fetch(t0);
    bc[0].put(p, n, g, t0, live);
  }
  const float bias = p.bias ? p.bias[c] : 0.0f;
  const float skip = OUT && p.D ? p.D[c] : 0.0f;
  F2 A2[P], h[P];
  float sum = 0.0f;
  {
    float a[K], v[K];
    load_states<K, TPC>(p.A + (long long)c * p.K, p.K, part, p.k_vec, a);
    fill(v, 0.0f);
    if (OUT) {
      if (p.chunks > 1) previous_done();
      if (p.chunks > 1) load_states<K, TPC>(p.carry + row * p.K, p.K, part, p.k_vec, v);
      else if (p.h0) load_states<K, TPC>(p.h0 + ((long long)n * p.C + c) * p.K, p.K, part, p.k_vec, v);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      A2[i] = f2(rate2(a[2 * i]), rate2(a[2 * i + 1]));
      h[i] = f2(v[2 * i], v[2 * i + 1]);
    }
  }
  __syncthreads();

  int b = 0;
  for (int t = t0; t < live; t += TT, b ^= 1) {
    if (t + TT < live) bc[b ^ 1].put(p, n, g, t + TT, live);
#pragma unroll 1
    for (int r = 0; r < TT && t + r < live; r += kGroup) {
      T d[kGroup], u[kGroup], zz[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) d[i] = nd[i], u[i] = nu[i], zz[i] = nz[i];
      fetch(t + r + kGroup);
      const ulonglong2* B = reinterpret_cast<const ulonglong2*>(&bc[b].v[r * Tile::kRow + part]);
      const int steps = live - t - r;  // of the group; the rest stands still
#pragma unroll
      for (int i = 0; i < kGroup; ++i, B += Tile::kRow) {
        const bool on = i < steps;
        float dt = Elem<T>::to_f(d[i]) + bias, uu = Elem<T>::to_f(u[i]);
        if (p.softplus) dt = softplus_f(dt);
        if (!on) dt = 0.0f, uu = 0.0f;
        // float32's longer gate is computed before the states, where it does not
        // wait (4096 x 1 x 2048 x 16: 94.2 us, behind them 96.3), 16-bit tensors'
        // behind them (bf16 93.3 us, before them 94.3)
        float gate = 1.0f;
        auto gated = [&] {
          const float zf = Elem<T>::to_f(zz[i]);
          return zf * sigmoid_of<T>(zf);
        };
        if (OUT && sizeof(T) == 4 && z) gate = gated();
        const float du = dt * uu;
        const F2 dt2 = f2(dt, dt), du2 = f2(du, du);
        F2 y0 = f2(0.0f, 0.0f), y1 = y0;
#pragma unroll
        for (int k = 0; k < K / 4; ++k) {
          const ulonglong2 v = B[k * TPC];
          h[2 * k] = fma2(decay2(dt2, A2[2 * k]), h[2 * k], mul2(du2, F2{v.x}));
          h[2 * k + 1] = fma2(decay2(dt2, A2[2 * k + 1]), h[2 * k + 1], mul2(du2, F2{v.y}));
          if constexpr (OUT) {
            const ulonglong2 e = B[Tile::kQuads + k * TPC];
            y0 = k == 0 ? mul2(F2{e.x}, h[0]) : fma2(F2{e.x}, h[2 * k], y0);
            y1 = k == 0 ? mul2(F2{e.y}, h[1]) : fma2(F2{e.y}, h[2 * k + 1], y1);
          }
        }
        if constexpr (OUT) {
          const float2 s2 = f2_get(add2(y0, y1));
          float o = s2.x + s2.y;
#pragma unroll
          for (int m = TPC / 2; m > 0; m >>= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
          o = fmaf(skip, uu, o);
          if (sizeof(T) == 4) o *= gate;
          else if (z) o *= gated();
          if (on && stores) *y = Elem<T>::from_f(o);
          y += p.Y.ss;
        } else {
          sum += dt;
        }
      }
    }
    __syncthreads();
  }
  if (!mine) return;
  if constexpr (OUT) {
    if (stores) {
      const int from = max(t0, live);
      y = static_cast<T*>(p.Y.p) + n * p.Y.ns + from * p.Y.ss + c;
      for (int t = from; t < t1; ++t, y += p.Y.ss) *y = Elem<T>::from_f(0.0f);
    }
  }
  float v[K];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float2 w = f2_get(h[i]);
    v[2 * i] = w.x, v[2 * i + 1] = w.y;
  }
  if constexpr (OUT) {
    if (p.chunks == 1 && p.hT) store_states<K, TPC>(p.hT + ((long long)n * p.C + c) * p.K, p.K, part, p.k_vec, v);
  } else {
    store_states<K, TPC>(p.carry + row * p.K, p.K, part, p.k_vec, v);
    if (part == 0) p.sumdt[row] = sum;
  }
}

// The chunks' states in order: what each starts from takes the place of its own
// final state.
__global__ void __launch_bounds__(64) scan_carry_kernel(ScanParams p) {
  const unsigned ck = (unsigned)p.C * (unsigned)p.K;  // at most 2^31
  const unsigned at = blockIdx.x * 64u + threadIdx.x;
  next_may_start();
  const bool on = at < ck;
  const float A2 = on ? rate2(p.A[at]) : 0.0f;
  previous_done();
  if (!on) return;
  const unsigned c = at / (unsigned)p.K;
  for (int n = blockIdx.y; n < p.N; n += gridDim.y) {
    const long long i = (long long)n * ck + at;
    float* carry = p.carry + (long long)n * p.chunks * ck + at;
    const float* sumdt = p.sumdt + (long long)n * p.chunks * p.C + c;
    float run = p.h0 ? p.h0[i] : 0.0f;
    run = may_grow(p, A2) ? join_batches<4, true>(carry, ck, sumdt, p.C, p.chunks, false, A2, run)
                          : join_batches<24, false>(carry, ck, sumdt, p.C, p.chunks, false, A2, run);
    if (p.hT) p.hT[i] = run;
  }
}

// Single tokens: four states per thread, TPC threads per channel, the state
// read and written once in 16-byte pieces and everything else straight from
// global memory.  Bound by the state's bytes; next to that by instructions, so
// the threads of a channel share out what belongs to the channel: each
// prepares its part of kTokens sequences, and stores its outputs.  VEC: states,
// B and C take pieces of four; then all loads are issued before the first is
// used.  64 sequences x 2048 channels x 16 states: 4.4 us on the device, 4.1
// TB/s over 18 MB; back to back calls from the L2 6.3 us against the prompt
// kernel's 10.4, 256 sequences 14.5 against 26.8.  From two steps on the
// prompt kernel is ahead (four steps of 64 sequences: 8.9 us against 14.4).
constexpr int kTokenThreads = 128, kTokens = 4;
template <typename T, int TPC, bool VEC>
__global__ void __launch_bounds__(kTokenThreads) scan_token_kernel(ScanParams p) {
  constexpr int kOwn = (kTokens + TPC - 1) / TPC;  // sequences per thread
  const int part = threadIdx.x % TPC;
  const int c0 = blockIdx.x * (kTokenThreads / TPC) + threadIdx.x / TPC;
  const bool mine = c0 < p.C;
  const int c = mine ? c0 : 0, g = c / (p.C / p.G);
  const bool holds = part * 4 < p.K;  // this thread has states
  const int k = holds ? part * 4 : 0;
  const long long row = (long long)p.C * p.K;  // a sequence's states
  for (long long n0 = (long long)blockIdx.y * kTokens; n0 < p.N; n0 += (long long)gridDim.y * kTokens) {
    const int left = (int)min((long long)kTokens, p.N - n0);
    T u[kOwn], d[kOwn], z[kOwn];
    int len[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      // past the last sequence: the last one again, not stored
      const long long n = n0 + min(j * TPC + part, left - 1);
      len[j] = p.lens ? p.lens[n] : 1;
      u[j] = static_cast<const T*>(p.X.p)[n * p.X.ns + c];
      d[j] = static_cast<const T*>(p.Delta.p)[n * p.Delta.ns + c];
      z[j] = p.Z.p ? static_cast<const T*>(p.Z.p)[n * p.Z.ns + c] : u[j];
    }
    const float* rates = p.A + (long long)c * p.K + k;
    const float* from = p.h0 ? p.h0 + n0 * row + (long long)c * p.K + k : nullptr;
    const T* B = static_cast<const T*>(p.Bm.p) + n0 * p.Bm.ns + (long long)g * p.K + k;
    const T* C = static_cast<const T*>(p.Cm.p) + n0 * p.Cm.ns + (long long)g * p.K + k;
    float A2[4], h[kTokens][4], b[kTokens][4], e[kTokens][4];
    if constexpr (VEC) {
      Packed<T, 4> rb[kTokens], rc[kTokens];
      Packed<float, 4> rh[kTokens], ra;
      ra.load(rates);
#pragma unroll
      for (int i = 0; i < kTokens; ++i) {
        const int at = min(i, left - 1);
        rb[i].load(B + at * p.Bm.ns);
        rc[i].load(C + at * p.Cm.ns);
        rh[i].raw = {};
        if (from) rh[i].load(from + at * row);
      }
      ra.widen(A2);
#pragma unroll
      for (int i = 0; i < kTokens; ++i) rb[i].widen(b[i]), rc[i].widen(e[i]), rh[i].widen(h[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool on = k + j < p.K;
        A2[j] = on ? rates[j] : 0.0f;
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
          const int at = min(i, left - 1);
          b[i][j] = on ? Elem<T>::to_f(B[at * p.Bm.ns + j]) : 0.0f;
          e[i][j] = on ? Elem<T>::to_f(C[at * p.Cm.ns + j]) : 0.0f;
          h[i][j] = on && from ? from[at * row + j] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] = rate2(A2[j]);
    // this thread's sequences: dt, dt u, D u, and the gate
    const float bias = p.bias ? p.bias[c] : 0.0f, skip = p.D ? p.D[c] : 0.0f;
    float dt[kOwn], du[kOwn], sk[kOwn], gate[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const float uu = Elem<T>::to_f(u[j]), zz = Elem<T>::to_f(z[j]);
      dt[j] = Elem<T>::to_f(d[j]) + bias;
      if (p.softplus) dt[j] = softplus_f(dt[j]);
      gate[j] = p.Z.p ? zz * sigmoid_of<T>(zz) : 1.0f;
      du[j] = dt[j] * uu;
      sk[j] = skip * uu;
    }
    float* to = p.hT ? p.hT + n0 * row + (long long)c * p.K + k : nullptr;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const float dti = __shfl_sync(0xffffffffu, dt[i / TPC], i % TPC, TPC);
      const float dui = __shfl_sync(0xffffffffu, du[i / TPC], i % TPC, TPC);
      // a sequence without this step keeps its state, whatever its row holds
      const bool live = __shfl_sync(0xffffffffu, len[i / TPC], i % TPC, TPC) > 0;
      float y = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float next = fmaf(decay(dti, A2[j]), h[i][j], dui * b[i][j]);
        if (live) h[i][j] = next;
        y = fmaf(e[i][j], h[i][j], y);
      }
      if (!holds) y = 0.0f;
#pragma unroll
      for (int o = TPC / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      if (!mine || i >= left) continue;
      if (part == i % TPC && p.Y.p)
        static_cast<T*>(p.Y.p)[(n0 + i) * p.Y.ns + c] =
            Elem<T>::from_f(live ? (y + sk[i / TPC]) * gate[i / TPC] : 0.0f);
      if (!to || !holds) continue;
      if constexpr (VEC) {
        *reinterpret_cast<float4*>(to + i * row) = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k + j < p.K) to[i * row + j] = h[i][j];
      }
    }
  }
}

template <typename T, int K, int TPC>
cudaError_t run_scan(const ScanParams& p, cudaStream_t s, int* launches) {
  const int nt = block_threads(p.C / p.G, p.K), CH = nt / TPC;
  const long long tiles = (p.C / p.G + CH - 1) / CH;
  const long long blocks = (long long)p.N * p.chunks * p.G * tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  if (p.chunks > 1) {
    scan_kernel<T, K, TPC, false><<<(unsigned)blocks, nt, 0, s>>>(p);
    const long long states = (long long)p.C * p.K;
    e = launch_chained(scan_carry_kernel, dim3((unsigned)((states + 63) / 64), std::min(p.N, 65535)), 64, 0, s, p);
    *launches += 2;
    if (e == cudaSuccess && p.Y.p) {
      e = launch_chained(scan_kernel<T, K, TPC, true>, (unsigned)blocks, nt, 0, s, p);
      *launches += 1;
    }
  } else {
    scan_kernel<T, K, TPC, true><<<(unsigned)blocks, nt, 0, s>>>(p);
    *launches += 1;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int TPC>
cudaError_t run_token(const ScanParams& p, cudaStream_t s, int* launches) {
  const int per = kTokenThreads / TPC, tiles = (p.C + per - 1) / per;
  const int rows = std::min((p.N + kTokens - 1) / kTokens, 65535);
  const dim3 grid(tiles, rows);
  if (p.k_vec && p.bc_vec) scan_token_kernel<T, TPC, true><<<grid, kTokenThreads, 0, s>>>(p);
  else scan_token_kernel<T, TPC, false><<<grid, kTokenThreads, 0, s>>>(p);
  *launches += 1;
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_typed(const ScanParams& p, cudaStream_t s, int* launches) {
  if (p.S == 1) {  // the figures are at the token kernel
    if (p.K <= 4) return run_token<T, 1>(p, s, launches);
    if (p.K <= 8) return run_token<T, 2>(p, s, launches);
    if (p.K <= 16) return run_token<T, 4>(p, s, launches);
    if (p.K <= 32) return run_token<T, 8>(p, s, launches);
    if (p.K <= 64) return run_token<T, 16>(p, s, launches);
    return run_token<T, 32>(p, s, launches);
  }
  if (p.K <= 4) return run_scan<T, 4, 1>(p, s, launches);
  if (p.K <= 8) return run_scan<T, 8, 1>(p, s, launches);
  if (p.K <= 16) return run_scan<T, 16, 1>(p, s, launches);
  if (p.K <= 32) return run_scan<T, 16, 2>(p, s, launches);
  if (p.K <= 64) return run_scan<T, 16, 4>(p, s, launches);
  return run_scan<T, 16, 8>(p, s, launches);
}

}  // namespace

ScanPlan scan_plan(long long seq, long long batch, long long channels, int state, int groups, bool ragged) {
  ScanPlan pl{};
  pl.chunks = 1;
  pl.chunk = (int)std::max<long long>(seq, 1);
  if (seq <= 1 || batch == 0) return pl;
  const int nt = block_threads((int)(channels / groups), state);
  const long long per = channels / groups, ch = nt / tpc_of(state);
  const long long warps = batch * groups * ((per + ch - 1) / ch) * (nt / 32);
  // Warps that the card holds: registers for 20 per SM.  Below a third of them
  // chunks pay for their second pass over the exponentials: 1024 steps x 2048
  // channels x 16 states bf16, 1 sequence (64 warps) 247 us without and 37
  // with, 8 sequences 270 and 201, 12 sequences 305 and 306, 16 sequences 308
  // and 447.  Where rows have lengths, chunks past them end at once: twice as
  // many keep the card full where half of the steps are (lengths uniform in
  // 1..1024: 2 sequences 47 us with as many, 37 with twice, 8 sequences 162 and
  // 105), and they pay up to 0.4 of the warps (16 sequences 285 us without and
  // 210 with, 24 sequences 317 and 407).  A chunk of 8 steps is as short as pays
  // (128 steps of one sequence: 12.7 us, with 16 at least 14.6, with 32 22.7),
  // and the two launches more from 40 steps on (40 steps 12.3 us against 14.4,
  // 24 steps 12.1 against 10.4).
  const long long places = kPlanSms * kBlocks * (kThreads / 32);
  const long long want = ragged ? places * 2 : places;
  if (seq >= 40 && (ragged ? warps * 5 < places * 2 : warps * 3 < places)) {
    const long long chunks = std::min(want / warps, seq / 8);
    if (chunks > 1) {
      pl.chunk = (int)((((seq + chunks - 1) / chunks) + kGroup - 1) / kGroup * kGroup);
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
