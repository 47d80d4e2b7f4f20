// rk_attn_tc.cuh -- attention through a decaying state in chunks of 64 steps,
// on the tensor cores.
//
// With G_i the sum of the decays' logarithms from a chunk's start up to step
// i, a pass forward in time is, for the steps m of a chunk,
//   o_m = so (su sum_{n <= m} 2^(G_m - G_n) (q_m k_n) v_n + 2^(G_m) H^T q_m),
//   H   = 2^(G_end) H + su sum_n 2^(G_end - G_n) k_n v_n^T,
// and backward in time the same with n >= m and the signs of G's differences
// turned: the step itself is read after it is written, its decay lies between
// it and the step before.  Four matrix products:
//   S  = Q K^T            [m][n]     then P = S 2^(..) where n is allowed
//   Oi = H^T Q^T          [v][m]     (the state's transpose in tensor memory)
//   O  = V^T P^T          [v][m]
//   U  = V^T (ck K)       [v][k]     then H^T = 2^(G_end) H^T + su U
// Values run along the 128 lanes of tensor memory, so that the state, which a
// lane's thread keeps in float32 registers, needs no transposition between U,
// where it is added to, and Oi, where it is the product's A operand.
//
// The tensor cores multiply bfloat16.  A factor of more bits is a sum of two
// or three bfloat16 terms (each the rounding of what the ones before left),
// and a product the sum of the terms' products down to 2^-24 of it, smallest
// first; bfloat16 operands are one term, Half two, float32 three, and what is
// computed here (P, ck K, H) three.  Differences of G are exact to 2^-24: sums
// are 64-bit whole numbers of 2^-32, kept as whole part and fraction.
//
// A block runs one state (two, stacked along the lanes, where heads have at
// most 64 elements: of the products' 128 x 128 blocks the diagonal ones are
// used) over a piece of the sequence.
//
// Infinities and NaN must not reach other steps through the products' zeros:
// a chunk in which an operand, a product of P or the state is not finite is
// run step by step instead.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "rk_attn.h"
#include "rk_proj_tc.cuh"
#include "rk_ssm_common.cuh"

namespace rk {
namespace atc {

using namespace ptc;

constexpr int kChunk = 64, kThreads = 256, kTerms = 3;
constexpr uint32_t kSub = kChunk * 128;      // bytes of 64 rows of 64 elements
constexpr uint32_t kTile = 2 * kSub;         // an operand's term: 64 rows of 128 elements, or of two heads of 64
constexpr long long kWaitNs = 2000000000LL;  // a wait that takes this long has failed

template <typename T>
constexpr int kSplit = sizeof(T) == 4 ? 3 : 2;
template <>
constexpr int kSplit<__nv_bfloat16> = 1;

// Shared memory: operand tiles (bfloat16: two stages), ck K, P (float32: where
// K was), and small arrays.
template <typename T, int HPC>
struct Layout {
  static constexpr int kIn = kSplit<T>;
  static constexpr int kStages = kIn == 1 ? 2 : 1;
  static constexpr uint32_t kQ = 0, kK = kIn * kTile, kV = 2 * kIn * kTile, kStage = 3 * kIn * kTile;
  static constexpr uint32_t kScaled = kStages * kStage;
  static constexpr bool kOver = kIn == 3;
  static constexpr uint32_t kP = kOver ? kK : kScaled + kTerms * kTile;
  static constexpr uint32_t kPTerm = HPC * kSub;
  static constexpr uint32_t kEnd = kScaled + kTerms * kTile + (kOver ? 0 : kTerms * kPTerm);
  static_assert(kTerms * kPTerm <= kIn * kTile || !kOver, "P fits over K");
  static constexpr size_t kBytes = kEnd + 1024;  // alignment
};

// Decays of a chunk, by head of the block.
struct Decays {
  float hi[kChunk], lo[kChunk];  // signed G: whole part and fraction
  float cq[kChunk], ck[kChunk];  // 2^.. of the state's part of a step's output, and of its part of the state
  float d[kChunk];               // a step's own decay
  double log2;                   // of the chunk's whole decay
  float total;                   // the decay
};

struct Small {
  Decays decays[2][2];
  float dots[8][32];
  float part[2][128];
  uint64_t bars[4];
  uint32_t tmem;
  int wrong[2];
  volatile int gave_up;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return Elem<__nv_bfloat16>::pair_from_f(lo, hi); }
__device__ __forceinline__ float low_of(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_of(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Two factors as N terms each; the first terms' product with 0 goes to
// `finite`, which they leave 0 unless one of them is infinite or NaN.
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&t)[N], float& finite) {
  t[0] = pack2(a, b);
  finite = fmaf(low_of(t[0]), 0.0f, fmaf(high_of(t[0]), 0.0f, finite));
#pragma unroll
  for (int i = 1; i < N; ++i) {
    a -= low_of(t[i - 1]), b -= high_of(t[i - 1]);
    t[i] = pack2(a, b);
  }
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of the same tile read along its rows: 64 elements of the outer
// matrix dimension are a row's 128 bytes, the next 64 lie a sub-tile on, eight
// steps of the inner one are 1024 bytes.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return smem_desc_sw128(addr) & ~((uint64_t)0x3FFF << 16) | ((uint64_t)(kSub >> 4) << 16);
}

constexpr uint32_t kRowsA = 1u << 15, kRowsB = 1u << 16;  // operand read along its rows
__host__ __device__ constexpr uint32_t idesc_of(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (8u << 24);  // bfloat16, M = 128
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Set where a wait has failed (one per element type's unit).
static __device__ int gave_up_status;

// What a block works on.
template <int HPC>
struct Place {
  int n, h0, segment, order, stream;
  const AttnPass* pass;
  __device__ __forceinline__ Place(const AttnParams& p, int segments) {
    long long id = blockIdx.x;
    segment = (int)(id % segments);
    id /= segments;
    stream = (int)id;
    const int groups = (p.H + HPC - 1) / HPC;
    h0 = (int)(id % groups) * HPC;
    id /= groups;
    n = (int)(id % p.N);
    pass = &p.pass[id / p.N];
  }
};

// 2^(whole + fraction) without rounding the sum.
__device__ __forceinline__ float pow2_of(long long g) {
  const int whole = (int)(g >> 32);
  const float part = exp2_fast((float)((uint32_t)g >> 8) * 5.9604644775390625e-8f);
  if (whole < -126) return 0.0f;
  return whole > 127 ? __int_as_float(0x7f800000) : part * __int_as_float((whole + 127) << 23);
}

// One warp: the decays of the chunk that starts at t0, L the row's length.
__device__ __forceinline__ void chunk_decays(const AttnParams& p, bool backward, int n, int h, int t0, int L,
                                             Decays& out, int* wrong) {
  const int lane = threadIdx.x % 32;
  const float* g = static_cast<const float*>(p.decay.p) + n * p.decay.ns + h;
  const float bias = p.bias ? p.bias[h] : 0.0f;
  long long fix[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = t0 + 2 * lane + j;
    float x = 0.0f;
    if (t < L) x = (p.decay.p ? g[t * p.decay.ss] : 0.0f) + bias;
    out.d[2 * lane + j] = expf(x);
    if (!(x < 80.0f)) *wrong = 1;  // NaN, or growth that no float32 holds for long
    // what is below leaves nothing in float32; a chunk's sum stays within 2^25
    fix[j] = __double2ll_rn((double)fminf(fmaxf(x, -1.0e5f), 80.0f) * (1.4426950408889634074 * 4294967296.0));
  }
  long long sum = fix[0] + fix[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  const long long total = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long G = j ? sum : sum - fix[1], s = backward ? -G : G;
    const int i = 2 * lane + j;
    out.hi[i] = (float)(int)(s >> 32);
    out.lo[i] = (float)((uint32_t)s >> 8) * 5.9604644775390625e-8f;
    if (G >> 32 > 120 || (total - G) >> 32 > 120) *wrong = 1;
    const float up = pow2_of(G), down = pow2_of(total - G);
    out.cq[i] = backward ? down : up;
    out.ck[i] = backward ? up : down;
  }
  if (lane == 0) out.total = pow2_of(total), out.log2 = (double)total * 2.3283064365386962890625e-10;
}

// Row operands of a block, as pointers to its first head's elements.
template <typename T>
__device__ __forceinline__ const T* head_rows(const RowsArg& a, int n, int h, int of, int size) {
  return static_cast<const T*>(a.p) + n * a.ns + (long long)(h / of) * size;
}

// Fetches 64 rows of an operand into its tile: sub-tile b is the elements
// from 64 b on, or head b.  Steps from L on, elements from `size` on and heads
// that there are not are zeros.
template <typename T, int HPC, int KB>
__device__ __forceinline__ void load_tile(unsigned char* tile, const RowsArg& a, int n, int h0, int heads, int of, int size,
                                          int t0, int L, int vec) {
  constexpr int kIn = kSplit<T>;
  constexpr int kPieces = HPC == 2 ? 2 : KB;
#pragma unroll
  for (int b = 0; b < kPieces; ++b) {
    const int h = HPC == 2 ? h0 + b : h0, first = HPC == 2 ? 0 : 64 * b;
    const T* rows = head_rows<T>(a, n, min(h, heads - 1), of, size) + first;
#pragma unroll
    for (int r0 = 0; r0 < kChunk; r0 += kThreads / 8) {
      const int r = r0 + threadIdx.x / 8, c = threadIdx.x % 8, t = t0 + r;
      const bool on = t < L && h < heads;
      const T* src = rows + (long long)t * a.ss + 8 * c;
      unsigned char* dst = tile + b * kSub + r * 128 + ((c ^ (r & 7)) << 4);
      if constexpr (kIn == 1) {
        if (vec) {
          const bool fetch = on && first + 8 * c < size;
          cp16(su32(dst), fetch ? src : static_cast<const T*>(a.p), fetch);
          continue;
        }
      }
      float x[8];
      if (vec) {
        if (on && first + 8 * c < size) {
          if constexpr (sizeof(T) == 4) {
            float y[4];
            Piece<T, 4>::load(src, y);
            x[0] = y[0], x[1] = y[1], x[2] = y[2], x[3] = y[3];
            if (first + 8 * c + 4 < size) Piece<T, 4>::load(src + 4, y);
            else fill(y, 0.0f);
            x[4] = y[0], x[5] = y[1], x[6] = y[2], x[7] = y[3];
          } else {
            Piece<T, 8>::load(src, x);
          }
        } else {
          fill(x, 0.0f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = on && first + 8 * c + i < size ? Elem<T>::to_f(src[i]) : 0.0f;
      }
      uint32_t w[kIn][4];
      float unused = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t s[kIn];
        split<kIn>(x[2 * i], x[2 * i + 1], s, unused);
#pragma unroll
        for (int j = 0; j < kIn; ++j) w[j][i] = s[j];
      }
#pragma unroll
      for (int j = 0; j < kIn; ++j) *reinterpret_cast<uint4*>(dst + j * kTile) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
    }
  }
}

// ck K as three terms, and whether all of K and V is finite.
template <typename T, int HPC, int KB>
__device__ __forceinline__ void scale_tile(const unsigned char* k, unsigned char* out, const Decays* d, float& finite) {
  constexpr int kIn = kSplit<T>;
  constexpr int kPieces = HPC == 2 ? 2 : KB;
#pragma unroll
  for (int b = 0; b < kPieces; ++b) {
#pragma unroll
    for (int r0 = 0; r0 < kChunk; r0 += kThreads / 8) {
      const int r = r0 + threadIdx.x / 8, c = threadIdx.x % 8;
      const uint32_t at = b * kSub + r * 128 + ((c ^ (r & 7)) << 4);
      const float f = d[HPC == 2 ? b : 0].ck[r];
      float x[8];
      fill(x, 0.0f);
#pragma unroll
      for (int j = kIn - 1; j >= 0; --j) {
        const uint4 u = *reinterpret_cast<const uint4*>(k + j * kTile + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] += low_of(w[i]), x[2 * i + 1] += high_of(w[i]);
      }
      uint32_t w[kTerms][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t s[kTerms];
        split<kTerms>(x[2 * i] * f, x[2 * i + 1] * f, s, finite);
#pragma unroll
        for (int j = 0; j < kTerms; ++j) w[j][i] = s[j];
      }
#pragma unroll
      for (int j = 0; j < kTerms; ++j)
        *reinterpret_cast<uint4*>(out + j * kTile + at) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
    }
  }
}

// Whether a tile's first term is finite: its exponents are not all ones.
template <int PIECES>
__device__ __forceinline__ bool tile_finite(const unsigned char* tile) {
  uint32_t bad = 0;
#pragma unroll
  for (int b = 0; b < PIECES; ++b) {
#pragma unroll
    for (int i = 0; i < (int)kSub / 16 / kThreads; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(tile + b * kSub + (i * kThreads + threadIdx.x) * 16);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) bad |= ((w[j] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    }
  }
  return bad == 0;
}

// One thread: all products of NA terms of A and NB of B down to 2^-24,
// smallest first, STEPS products of 16 each.
template <int NA, int NB, int STEPS, typename F>
__device__ __forceinline__ void products(F mma) {
  uint32_t more = 0;
#pragma unroll
  for (int sum = (NA + NB - 2 < kTerms - 1 ? NA + NB - 2 : kTerms - 1); sum >= 0; --sum) {
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int b = sum - a;
      if (b < 0 || b >= NB) continue;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        mma(a, b, s, more);
        more = 1;
      }
    }
  }
}

// OUT: the outputs too; else only what the segment adds to the state.
template <typename T, int HPC, int KB, bool OUT>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const __grid_constant__ AttnParams p) {
  using Lay = Layout<T, HPC>;
  constexpr int kIn = kSplit<T>;
  constexpr int NH = HPC == 2 ? 32 : 32 * KB;       // state elements of a thread
  constexpr int KW = HPC == 2 ? 32 : 32 * KB;       // tensor memory columns of one of the state's terms
  constexpr uint32_t kS = 0, kOi = 64 * HPC, kU = 128 * HPC, kH = kU + 128;
  static_assert(kH + kTerms * KW <= 512, "tensor memory");
  constexpr int kHeadSteps = HPC == 2 ? 4 : 4 * KB;  // steps of 16 over a head's elements
  extern __shared__ unsigned char raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  __shared__ Small sh;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, quarter = warp & 3, half = warp >> 2;
  const int r = quarter * 32 + lane;
  const Place<HPC> at(p, OUT ? p.plan.segments : p.plan.segments - 1);
  const AttnPass& a = *at.pass;
  const bool back = a.backward;
  // the segments' order is the pass's; the one that the last state leaves adds to none
  const int segments = p.plan.segments, order = at.segment, segment = back ? segments - 1 - order : order;
  const int head = HPC == 2 ? r >> 6 : 0, h = at.h0 + head, v = HPC == 2 ? r & 63 : r;
  const bool mine = v < a.V && h < p.H;
  const int k0 = half * NH, ucol = HPC == 2 ? head * 64 + half * 32 : half * NH;  // state elements, U's columns
  const int S = p.S, L = row_length(p.lens, at.n, S);
  const int chunks = (S + kChunk - 1) / kChunk, live = (L + kChunk - 1) / kChunk;
  const int c_begin = segment * p.plan.per, c_end = min(c_begin + p.plan.per, chunks);
  const int c_live = min(c_end, live), count = max(c_live - c_begin, 0);
  auto chunk_at = [&](int i) { return back ? c_live - 1 - i : c_begin + i; };

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) bar_init(su32(&sh.bars[i]), 1);
    sh.gave_up = 0;
    sh.wrong[0] = sh.wrong[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sh.tmem)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem, lanes = tmem + ((uint32_t)(quarter * 32) << 16);

  // the state, transposed: lane v, elements k0 ..
  const long long state = ((long long)at.n * p.H + h) * a.K * a.V;
  auto state_at = [&](int i) {
    return state + (a.v_major ? (long long)v * a.K + k0 + i : (long long)(k0 + i) * a.V + v);
  };
  const long long kept = (long long)KB * 64 * 128;  // a state in scratch: [k][lane]
  const int heads_k = HPC == 2 ? 64 : 64 * KB;
  float H[NH];
  if (OUT && segments > 1) {
    const float* from = p.plan.states + ((long long)at.stream * segments + order) * kept;
#pragma unroll
    for (int i = 0; i < NH; ++i) H[i] = k0 + i < heads_k ? from[(k0 + i) * 128 + r] : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < NH; ++i) H[i] = OUT && a.first && mine && k0 + i < a.K ? a.first[state_at(i)] : 0.0f;
  }

  float bad_state = 0.0f;  // 0 while the state is finite
  auto publish = [&]() {   // the state's terms to tensor memory
#pragma unroll
    for (int j = 0; j < NH; j += 32) {
      uint32_t w[kTerms][16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t s[kTerms];
        split<kTerms>(H[j + 2 * i], H[j + 2 * i + 1], s, bad_state);
#pragma unroll
        for (int x = 0; x < kTerms; ++x) w[x][i] = s[x];
      }
#pragma unroll
      for (int x = 0; x < kTerms; ++x) tmem_st16(lanes + kH + x * KW + (k0 + j) / 2, w[x]);
    }
    tmem_st_done();
  };
  auto fetch = [&](int c, int stage) {
    unsigned char* tiles = sm + stage * Lay::kStage;
    const int t0 = c * kChunk;
    if (OUT) load_tile<T, HPC, KB>(tiles + Lay::kQ, a.q, at.n, at.h0, p.H, a.q_of, a.K, t0, L, p.plan.vec);
    load_tile<T, HPC, KB>(tiles + Lay::kK, a.k, at.n, at.h0, p.H, a.k_of, a.K, t0, L, p.plan.vec);
    load_tile<T, HPC, 2>(tiles + Lay::kV, a.v, at.n, at.h0, p.H, a.v_of, a.V, t0, L, p.plan.vec);
    cp_commit();
  };
  auto decays_of = [&](int i) {
    if (warp < HPC && at.h0 + warp < p.H)
      chunk_decays(p, back, at.n, at.h0 + warp, chunk_at(i) * kChunk, L, sh.decays[i & 1][warp], &sh.wrong[i & 1]);
    else if (warp < HPC)
      chunk_decays(p, back, at.n, at.h0, S, 0, sh.decays[i & 1][warp], &sh.wrong[i & 1]);
  };
  auto wait = [&](int bar, uint32_t phase) {
    if (!sh.gave_up && !bar_wait(su32(&sh.bars[bar]), phase, kWaitNs)) {
      sh.gave_up = 1;
      atomicOr(&gave_up_status, 1);
    }
    tc_fence_after();
  };
  auto dots_out = [&](int c) {  // the products of a chunk's outputs, added up over the lanes' warps
    if (OUT && a.dot && tid < 64 * HPC) {
      const int hd = tid / 64, i = tid % 64, t = c * kChunk + i;
      if (t < L && at.h0 + hd < p.H) {
        const float* x = &sh.dots[(i / 32) * 4][i % 32];
        const float y = HPC == 2 ? x[(2 * hd) * 32] + x[(2 * hd + 1) * 32] : (x[0] + x[32]) + (x[64] + x[96]);
        a.dot[((long long)at.n * p.H + at.h0 + hd) * S + t] = y;
      }
    }
  };
  // outputs of lane v at step t
  T* out = static_cast<T*>(a.o.p) + at.n * a.o.ns + (long long)(h / a.o_of) * a.V + v;
  const T* dot_row = static_cast<const T*>(a.dot_with.p) + at.n * a.dot_with.ns + (long long)(h / a.o_of) * a.V + v;
  auto put = [&](int t, float y) {
    if (!mine || t >= S) return;
    if (a.o32) a.o32[(((long long)at.n * S + t) * p.H + h) * a.V + v] = y;
    else if (a.o.p) out[t * a.o.ss] = Elem<T>::from_f(y);
  };

  if (count > 0) {
    fetch(chunk_at(0), 0);
    decays_of(0);
  }
  if (OUT) publish();
  uint32_t phase = 0;
  double left = 0.0;  // logarithm of the segment's decay
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int c = chunk_at(i), t0 = c * kChunk;
    const int stage = Lay::kStages == 2 ? i & 1 : 0;
    unsigned char* tiles = sm + stage * Lay::kStage;
    const Decays* dec = sh.decays[i & 1];
    cp_wait();
    to_async();
    tc_fence_before();
    const bool failed = __syncthreads_or(sh.gave_up);
    tc_fence_after();
    if (failed) break;
    const uint32_t tq = su32(tiles + Lay::kQ), tk = su32(tiles + Lay::kK), tv = su32(tiles + Lay::kV);
    const uint32_t ts = su32(sm + Lay::kScaled), tp = (Lay::kOver ? tk : su32(sm + Lay::kP));
    if (OUT && tid == 0) {
      constexpr uint32_t id = idesc_of(64 * HPC);
      products<kIn, kIn, kHeadSteps>([&](int x, int y, int s, uint32_t more) {
        const uint32_t o = (s / 4) * kSub + (s % 4) * 32;
        tc_mma(tmem + kS, smem_desc_sw128(tq + x * kTile + o), smem_desc_sw128(tk + y * kTile + o), id, more);
      });
      tc_commit(su32(&sh.bars[0]));
      products<kTerms, kIn, kHeadSteps>([&](int x, int y, int s, uint32_t more) {
        tc_mma_ts(tmem + kOi, tmem + kH + x * KW + s * 8, smem_desc_sw128(tq + y * kTile + (s / 4) * kSub + (s % 4) * 32), id,
                  more);
      });
      tc_commit(su32(&sh.bars[1]));
    }
    if (i > 0) dots_out(chunk_at(i - 1));
    if (Lay::kStages == 2 && i + 1 < count) fetch(chunk_at(i + 1), stage ^ 1);
    float finite = 0.0f;
    scale_tile<T, HPC, KB>(tiles + Lay::kK, sm + Lay::kScaled, dec, finite);
    bool bad = !tile_finite<2>(tiles + Lay::kV);
    if (i + 1 < count) decays_of(i + 1);
    if (OUT) {
      if constexpr (Lay::kOver) __syncthreads();  // K is read before P takes its place
      wait(0, phase);
      if (HPC == 2 || quarter < 2) {
        // row m of S, 32 of its columns
        const int m = r & 63;
        const Decays& d = dec[head];
        float s[32];
        tmem_ld32(lanes + kS + (HPC == 2 ? head * 64 : 0) + half * 32, reinterpret_cast<uint32_t(&)[32]>(s));
        const float hi = d.hi[m], lo = d.lo[m];
        uint32_t w[kTerms][16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int nn = half * 32 + j + e;
            finite = fmaf(s[j + e], 0.0f, finite);
            const float f = exp2_fast((hi - d.hi[nn]) + (lo - d.lo[nn]));
            x[e] = (back ? nn >= m : nn <= m) ? s[j + e] * f : 0.0f;
          }
          uint32_t t[kTerms];
          split<kTerms>(x[0], x[1], t, finite);
#pragma unroll
          for (int e = 0; e < kTerms; ++e) w[e][j / 2] = t[e];
        }
        unsigned char* row = (Lay::kOver ? tiles + Lay::kK : sm + Lay::kP) + (HPC == 2 ? r : m) * 128;
#pragma unroll
        for (int e = 0; e < kTerms; ++e)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(row + e * Lay::kPTerm + (((half * 4 + x) ^ (m & 7)) << 4)) =
                make_uint4(w[e][4 * x], w[e][4 * x + 1], w[e][4 * x + 2], w[e][4 * x + 3]);
      }
    }
    bad = bad || !(finite == 0.0f) || (mine && !(bad_state == 0.0f)) || sh.wrong[i & 1];
    to_async();
    tc_fence_before();
    const bool by_step = __syncthreads_or(bad);
    tc_fence_after();
    if (tid == 0) sh.wrong[i & 1] = 0;
    left += dec[head].log2;
    if (!by_step) {
      if (tid == 0) {
        constexpr uint32_t idu = idesc_of(HPC == 2 ? 128 : 64 * KB) | kRowsA | kRowsB;
        products<kIn, kTerms, 4>([&](int x, int y, int s, uint32_t more) {
          tc_mma(tmem + kU, desc_mn(tv + x * kTile + s * 2048), desc_mn(ts + y * kTile + s * 2048), idu, more);
        });
        tc_commit(su32(&sh.bars[2]));
        if (OUT) {
          constexpr uint32_t ido = idesc_of(64 * HPC) | kRowsA;
          products<kIn, kTerms, 4>([&](int x, int y, int s, uint32_t more) {
            tc_mma(tmem + kS, desc_mn(tv + x * kTile + s * 2048), smem_desc_sw128(tp + y * Lay::kPTerm + s * 32), ido, more);
          });
          tc_commit(su32(&sh.bars[3]));
        }
      }
      float far[32];
      if (OUT) {
        wait(1, phase);
        tmem_ld32(lanes + kOi + (HPC == 2 ? head * 64 : 0) + half * 32, reinterpret_cast<uint32_t(&)[32]>(far));
      }
      wait(2, phase);
      const float e = dec[head].total;
#pragma unroll
      for (int j = 0; j < NH; j += 32) {
        float u[32];
        tmem_ld32(lanes + kU + ucol + j, reinterpret_cast<uint32_t(&)[32]>(u));
#pragma unroll
        for (int x = 0; x < 32; ++x) H[j + x] = fmaf(e, H[j + x], a.su * u[x]);
      }
      if (OUT) {
        publish();
        wait(3, phase);
        float o[32];
        tmem_ld32(lanes + kS + (HPC == 2 ? head * 64 : 0) + half * 32, reinterpret_cast<uint32_t(&)[32]>(o));
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          o[x] = a.so * fmaf(dec[head].cq[half * 32 + x], far[x], a.su * o[x]);
          put(t0 + half * 32 + x, o[x]);
        }
        if (a.dot) {
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const int t = t0 + half * 32 + x;
            o[x] = mine && t < L ? o[x] * Elem<T>::to_f(dot_row[t * a.dot_with.ss]) : 0.0f;
          }
          int to = 0;
          lanes_sum<32, 16, 1>(o, lane, to);
          sh.dots[warp][to] = o[0];
        }
      } else {
#pragma unroll
        for (int x = 0; x < NH; ++x) bad_state = fmaf(H[x], 0.0f, bad_state);
      }
      if (Lay::kStages == 1 && i + 1 < count) fetch(chunk_at(i + 1), 0);
    } else {
      // step by step, from the operands themselves
      if (OUT) wait(1, phase);
      const int rows = min(kChunk, L - t0);
      const int hc = min(h, p.H - 1);
      const T* q = head_rows<T>(a.q, at.n, hc, a.q_of, a.K);
      const T* k = head_rows<T>(a.k, at.n, hc, a.k_of, a.K);
      const T* x = head_rows<T>(a.v, at.n, hc, a.v_of, a.V);
#pragma unroll 1
      for (int j = 0; j < rows; ++j) {
        const int m = back ? rows - 1 - j : j;
        const long long t = t0 + m;
        const float d = dec[head].d[m], val = mine ? a.su * Elem<T>::to_f(x[t * a.v.ss + v]) : 0.0f;
        float y = 0.0f;
#pragma unroll
        for (int b = 0; b < NH; ++b) {
          if (mine && k0 + b < a.K) {
            H[b] = fmaf(Elem<T>::to_f(k[t * a.k.ss + k0 + b]), val, back ? H[b] : d * H[b]);
            if (OUT) y = fmaf(Elem<T>::to_f(q[t * a.q.ss + k0 + b]), H[b], y);
            if (back) H[b] *= d;
          }
        }
        if (OUT) {
          sh.part[half][r] = y;
          __syncthreads();
          if (half == 0) {
            y = a.so * (sh.part[0][r] + sh.part[1][r]);
            put((int)t, y);
            if (a.dot) {
              const float w = warp_sum(mine ? y * Elem<T>::to_f(dot_row[t * a.dot_with.ss]) : 0.0f);
              if (lane == 0) sh.dots[(m / 32) * 4 + quarter][m % 32] = w;
            }
          }
          __syncthreads();
        }
      }
      if (OUT)
        for (int m = rows + half; m < kChunk; m += 2) put(t0 + m, 0.0f);
      bad_state = 0.0f;
      if (OUT) {
        publish();
      } else {
#pragma unroll
        for (int b = 0; b < NH; ++b) bad_state = fmaf(H[b], 0.0f, bad_state);
      }
      // the barriers that this chunk did not use complete all the same
      if (tid == 0) {
        tc_commit(su32(&sh.bars[2]));
        if (OUT) tc_commit(su32(&sh.bars[3]));
      }
      wait(2, phase);
      if (OUT) wait(3, phase);
      __syncthreads();
      if (Lay::kStages == 1 && i + 1 < count) fetch(chunk_at(i + 1), 0);
    }
    phase ^= 1;
  }
  cp_wait();
  if (count > 0) {
    __syncthreads();
    if (!sh.gave_up) dots_out(chunk_at(count - 1));
  }
  if (OUT) {
    // the rows behind the last live chunk
    for (int t = max(c_live, c_begin) * kChunk + half; t < min(c_end * kChunk, S); t += 2) put(t, 0.0f);
    if (order == segments - 1) {
      float with = 0.0f;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        if (mine && k0 + i < a.K) {
          if (a.last) a.last[state_at(i)] = H[i];
          if (a.with) with = fmaf(a.with[state_at(i)], H[i], with);
        }
      }
      if (a.cross) {
        __syncthreads();
        with = warp_sum(with);
        if (lane == 0) sh.part[0][warp] = with;
        __syncthreads();
        if (tid < HPC && at.h0 + tid < p.H) {
          const float* x = sh.part[0];
          const float y = HPC == 2 ? (x[2 * tid] + x[2 * tid + 1]) + (x[2 * tid + 4] + x[2 * tid + 5])
                                   : ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
          a.cross[(long long)at.n * p.H + at.h0 + tid] = y;
        }
      }
    }
  } else {
    float* to = p.plan.states + ((long long)at.stream * segments + order) * kept;
#pragma unroll
    for (int i = 0; i < NH; ++i)
      if (k0 + i < heads_k) to[(k0 + i) * 128 + r] = mine && k0 + i < a.K ? H[i] : 0.0f;
    if (half == 0 && lane == 0 && (HPC == 2 ? quarter % 2 == 0 : quarter == 0))
      p.plan.left[((long long)at.stream * segments + order) * 2 + head] = left;
  }
  // nothing is in flight any more, unless a wait has failed: then what was issued gets as long again
  if (sh.gave_up && tid == 0) {
    tc_commit(su32(&sh.bars[3]));
    const unsigned long long begin = gtime();
    while ((long long)(gtime() - begin) < kWaitNs / 4) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// The states that a stream's segments start from, from what each adds: in the
// pass's order, element by element.
template <int HPC, int KB>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kept = KB * 64 * 128;
  const int element = blockIdx.y * 256 + threadIdx.x;
  const int k = element / 128, r = element % 128;
  if (HPC == 2 && k >= 64) return;
  long long id = blockIdx.x;
  const int groups = (p.H + HPC - 1) / HPC;
  const int h = (int)(id % groups) * HPC + (HPC == 2 ? r >> 6 : 0), v = HPC == 2 ? r & 63 : r;
  const int n = (int)(id / groups % p.N);
  const AttnPass& a = p.pass[id / groups / p.N];
  const bool mine = h < p.H && v < a.V && k < a.K;
  float run = 0.0f;
  if (mine && a.first)
    run = a.first[((long long)n * p.H + h) * a.K * a.V + (a.v_major ? (long long)v * a.K + k : (long long)k * a.V + v)];
  float* s = p.plan.states + id * p.plan.segments * kept + element;
  const double* f = p.plan.left + id * p.plan.segments * 2 + (HPC == 2 ? r >> 6 : 0);
  for (int i = 0; i < p.plan.segments; ++i) {
    const bool more = i + 1 < p.plan.segments;
    const float add = more ? s[(long long)i * kept] : 0.0f;
    s[(long long)i * kept] = run;
    if (!more) break;
    // 2^x run in two parts: where decays grow a state the power alone may pass float32's range
    const double x = fmin(fmax(f[2 * i], -300.0), 250.0);
    const int whole = (int)floor(x);
    const int w1 = max(min(whole, 127), -126), w2 = max(min(whole - w1, 127), -126);
    run = run * exp2f((float)(x - whole)) * __int_as_float((w1 + 127) << 23) * __int_as_float((w2 + 127) << 23) + add;
  }
}

template <typename T, int HPC, int KB>
cudaError_t launch_chunks_of(const AttnParams& p, cudaStream_t s, int* launches) {
  constexpr size_t smem = Layout<T, HPC>::kBytes;
  const long long streams = (long long)p.passes * p.N * ((p.H + HPC - 1) / HPC);
  cudaError_t e = cudaFuncSetAttribute(attn_chunk_kernel<T, HPC, KB, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (p.plan.segments > 1) {
    e = cudaFuncSetAttribute(attn_chunk_kernel<T, HPC, KB, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attn_chunk_kernel<T, HPC, KB, false><<<(unsigned)(streams * (p.plan.segments - 1)), kThreads, smem, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
    attn_join_kernel<HPC, KB><<<dim3((unsigned)streams, KB * 64 * 128 / 256), 256, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
  }
  attn_chunk_kernel<T, HPC, KB, true><<<(unsigned)(streams * p.plan.segments), kThreads, smem, s>>>(p);
  if ((e = cudaGetLastError()) == cudaSuccess) ++*launches;
  return e;
}

template <typename T>
cudaError_t launch_chunks(const AttnParams& p, cudaStream_t s, int* launches) {
  // every pass has the same two sizes, in one order or the other
  if (p.pass[0].K <= 64 && p.pass[0].V <= 64) return launch_chunks_of<T, 2, 1>(p, s, launches);
  return p.plan.deep == 64 ? launch_chunks_of<T, 1, 1>(p, s, launches) : launch_chunks_of<T, 1, 2>(p, s, launches);
}

// Reads and clears the status word, in stream order; the caller synchronises.
inline cudaError_t take_status(cudaStream_t s, int* to) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(to, gave_up_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || *to == 0) return e;
  const int zero = 0;
  e = cudaMemcpyToSymbolAsync(gave_up_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace atc
}  // namespace rk
