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

constexpr int kChunk = 64, kThreads = 512, kTerms = 3;
constexpr uint32_t kSub = kChunk * 128;      // bytes of 64 rows of 64 elements
constexpr uint32_t kTile = 2 * kSub;         // an operand's term: 64 rows of 128 elements, or of two heads of 64
constexpr int kCols = kChunk / 4;            // of a chunk's columns of S and O, those of a thread
constexpr long long kWaitNs = 2000000000LL;  // a wait that takes this long has failed

template <typename T>
constexpr int kSplit = sizeof(T) == 4 ? 3 : 2;
template <>
constexpr int kSplit<__nv_bfloat16> = 1;

// Shared memory: operand tiles (bfloat16: two stages), ck K, P in NT terms
// (float32: where K was), and small arrays.
template <typename T, int HPC, int NT>
struct Layout {
  static constexpr int kIn = kSplit<T>;
  static constexpr int kStages = kIn == 1 ? 2 : 1;
  static constexpr uint32_t kQ = 0, kK = kIn * kTile, kV = 2 * kIn * kTile, kStage = 3 * kIn * kTile;
  static constexpr uint32_t kScaled = kStages * kStage;
  static constexpr bool kOver = kIn == 3;
  static constexpr uint32_t kP = kOver ? kK : kScaled + kTerms * kTile;
  static constexpr uint32_t kPTerm = HPC * kSub;
  static constexpr uint32_t kEnd = kScaled + kTerms * kTile + (kOver ? 0 : NT * kPTerm);
  static_assert(NT * kPTerm <= kIn * kTile || !kOver, "P fits over K");
  static constexpr size_t kBytes = kEnd + 1024;  // alignment
};

// Decays of a chunk, by head of the block.
struct Decays {
  float hi[kChunk], lo[kChunk];    // signed G: whole part and fraction
  float nhi[kChunk], nlo[kChunk];  // their negatives
  float cq[kChunk], ck[kChunk];    // so 2^.. of the state's part of a step's output, su 2^.. of a step's part of the state
  float d[kChunk];                 // a step's own decay
  double log2;                     // of the chunk's whole decay
  float total;                     // the decay
};

struct Small {
  __align__(16) Decays decays[2][2];
  float dots[16][kCols];
  float part[4][128];
  uint64_t bars[4];
  uint32_t tmem;
  int wrong[2];
  volatile int gave_up;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return Elem<__nv_bfloat16>::pair_from_f(lo, hi); }
__device__ __forceinline__ F2 pair_of(uint32_t u) { return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }

// Two factors as N terms each; the first terms' product with 0 goes to
// `finite`, which they leave 0 unless one of them is infinite or NaN.
template <int N>
__device__ __forceinline__ void split(F2 x, uint32_t (&t)[N], F2& finite) {
  float2 v = f2_get(x);
  t[0] = pack2(v.x, v.y);
  F2 h = pair_of(t[0]);
  finite = fma2(h, f2(0.0f, 0.0f), finite);
#pragma unroll
  for (int i = 1; i < N; ++i) {
    x = fma2(h, f2(-1.0f, -1.0f), x);
    v = f2_get(x);
    t[i] = pack2(v.x, v.y);
    if (i + 1 < N) h = pair_of(t[i]);
  }
}
__device__ __forceinline__ bool is_finite(F2 finite) {
  const float2 v = f2_get(finite);
  return v.x == 0.0f && v.y == 0.0f;
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t* r) {
  static_assert(N == 8 || N == 16, "columns");
  if constexpr (N == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  }
}
__device__ __forceinline__ void tmem_st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 16 columns; complete after tmem_ld_done, which the values pass through.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&x)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}

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
  return (smem_desc_sw128(addr) & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(kSub >> 4) << 16);
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
__device__ __forceinline__ void chunk_decays(const AttnParams& p, const AttnPass& a, int n, int h, int t0, int L,
                                             Decays& out, int* wrong) {
  const bool backward = a.backward;
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
    const float hi = (float)(int)(s >> 32), lo = (float)((uint32_t)s >> 8) * 5.9604644775390625e-8f;
    out.hi[i] = hi, out.lo[i] = lo;
    out.nhi[i] = -hi, out.nlo[i] = -lo;
    if (G >> 32 > 120 || (total - G) >> 32 > 120) *wrong = 1;
    const float up = pow2_of(G), down = pow2_of(total - G);
    out.cq[i] = a.so * (backward ? down : up);
    out.ck[i] = a.su * (backward ? up : down);
  }
  if (lane == 0) out.total = pow2_of(total), out.log2 = (double)total * 2.3283064365386962890625e-10;
}

// Row operands of a block, as pointers to its first head's elements.
template <typename T>
__device__ __forceinline__ const T* head_rows(const RowsArg& a, int n, int h, int of, int size) {
  return static_cast<const T*>(a.p) + n * a.ns + (long long)(h / of) * size;
}

// A thread's part of an operand's tiles: one piece of 8 elements of a row of
// each of the two sub-tiles, which are the elements from 0 and 64 on, or two
// heads.
template <typename T, int HPC>
struct Rows {
  const T* src;       // the thread's first step's piece of sub-tile 0
  long long next, ss; // to sub-tile 1; to the next step
  int size, heads;    // elements of a head; heads that there are from the block's first on
  __device__ __forceinline__ Rows(const RowsArg& a, int n, int h0, int H, int of, int size_)
      : ss(a.ss), size(size_), heads(H - h0) {
    src = head_rows<T>(a, n, h0, of, size) + (threadIdx.x / 8) * a.ss + 8 * (threadIdx.x % 8);
    next = HPC == 1 ? 64 : (long long)(min(h0 + 1, H - 1) / of - h0 / of) * size;
  }
  // Fetches the 64 rows from t0 on into the tile at `tile`.  Steps from L on,
  // elements from `size` on and heads that there are not are zeros.
  template <int SUBS>
  __device__ __forceinline__ void load(unsigned char* tile, int t0, int L, int vec) const {
    constexpr int kIn = kSplit<T>;
    const int r = threadIdx.x / 8, c = threadIdx.x % 8;
    const T* at = src + t0 * ss;
    unsigned char* to = tile + r * 128 + ((c ^ (r & 7)) << 4);
#pragma unroll
    for (int b = 0; b < SUBS; ++b) {
      const int first = (HPC == 2 ? 0 : 64 * b) + 8 * c;
      const bool on = t0 + r < L && (HPC == 1 || b < heads);
      unsigned char* dst = to + b * kSub;
      const T* from = at + b * next;
      if constexpr (kIn == 1) {
        if (vec) {
          const bool fetch = on && first < size;
          cp16(su32(dst), fetch ? from : src, fetch);
          continue;
        }
      }
      float x[8];
      fill(x, 0.0f);
      if (vec) {
        if (on && first < size) {
          if constexpr (sizeof(T) == 4) {
            float y[4];
            Piece<T, 4>::load(from, y);
            x[0] = y[0], x[1] = y[1], x[2] = y[2], x[3] = y[3];
            if (first + 4 < size) {
              Piece<T, 4>::load(from + 4, y);
              x[4] = y[0], x[5] = y[1], x[6] = y[2], x[7] = y[3];
            }
          } else {
            Piece<T, 8>::load(from, x);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (on && first + i < size) x[i] = Elem<T>::to_f(from[i]);
      }
      uint32_t w[kIn][4];
      F2 unused = f2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t s[kIn];
        split<kIn>(f2(x[2 * i], x[2 * i + 1]), s, unused);
#pragma unroll
        for (int j = 0; j < kIn; ++j) w[j][i] = s[j];
      }
#pragma unroll
      for (int j = 0; j < kIn; ++j) *reinterpret_cast<uint4*>(dst + j * kTile) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
    }
  }
  // Has the rows from t0 on brought into L2.
  __device__ __forceinline__ void prefetch(int t0, int L) const {
    if (t0 + (int)(threadIdx.x / 8) >= L) return;
    const T* at = src + t0 * ss;
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if ((HPC == 1 ? 64 * b + 8 * (int)(threadIdx.x % 8) < size : b < heads && 8 * (int)(threadIdx.x % 8) < size))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + b * next));
  }
};

// ck K as three terms, of the tile's SUBS sub-tiles, by THREADS threads.
template <typename T, int HPC, int SUBS, int THREADS>
__device__ __forceinline__ void scale_tile(const unsigned char* k, unsigned char* out, const Decays* d, int thread, F2& finite) {
  constexpr int kIn = kSplit<T>;
#pragma unroll
  for (int i0 = 0; i0 < SUBS * 512; i0 += THREADS) {
    const int i = i0 + thread, r = i / 8 % kChunk, b = i / 512;
    const uint32_t at = b * kSub + i % 512 * 16;  // its swizzled place: any order of a row's pieces does
    const float f = d[HPC == 2 ? b : 0].ck[r];
    uint32_t w[kTerms][4];
    uint32_t t[kIn][4];
#pragma unroll
    for (int j = 0; j < kIn; ++j) {
      const uint4 u = *reinterpret_cast<const uint4*>(k + j * kTile + at);
      t[j][0] = u.x, t[j][1] = u.y, t[j][2] = u.z, t[j][3] = u.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      F2 x = pair_of(t[kIn - 1][e]);
#pragma unroll
      for (int j = kIn - 2; j >= 0; --j) x = add2(x, pair_of(t[j][e]));
      uint32_t s[kTerms];
      split<kTerms>(mul2(x, f2(f, f)), s, finite);
#pragma unroll
      for (int j = 0; j < kTerms; ++j) w[j][e] = s[j];
    }
#pragma unroll
    for (int j = 0; j < kTerms; ++j)
      *reinterpret_cast<uint4*>(out + j * kTile + at) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
  }
}

// Whether a tile's first term is finite, by THREADS threads: the largest of
// its magnitudes as whole numbers, 16 bits each.
template <int THREADS>
__device__ __forceinline__ bool tile_finite(const unsigned char* tile, int thread) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < (int)kTile / 16 / THREADS; ++i) {
    const uint4 u = *reinterpret_cast<const uint4*>(tile + (i * THREADS + thread) * 16);
    top = __vmaxu2(top, u.x & 0x7fff7fffu), top = __vmaxu2(top, u.y & 0x7fff7fffu);
    top = __vmaxu2(top, u.z & 0x7fff7fffu), top = __vmaxu2(top, u.w & 0x7fff7fffu);
  }
  return (top & 0xffffu) < 0x7f80u && (top >> 16) < 0x7f80u;
}

// One thread: the products of NA terms of A and NB of B down to 2^-8 NT,
// smallest first, STEPS products of 16 each.
template <int NA, int NB, int NT, int STEPS, typename F>
__device__ __forceinline__ void products(F mma) {
  uint32_t more = 0;
#pragma unroll
  for (int sum = (NA + NB - 2 < NT - 1 ? NA + NB - 2 : NT - 1); sum >= 0; --sum) {
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

// OUT: the outputs too, with P and the state in NT terms; else only what the
// segment adds to the state.
template <typename T, int HPC, int KB, int NT, bool OUT>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const __grid_constant__ AttnParams p) {
  using Lay = Layout<T, HPC, NT>;
  constexpr int kIn = kSplit<T>;
  constexpr int NH = HPC == 2 ? 16 : 16 * KB;  // state elements of a thread
  constexpr int KW = HPC == 2 ? 32 : 32 * KB;  // tensor memory columns of one of the state's terms
  constexpr uint32_t kS = 0, kOi = 64 * HPC, kU = 128 * HPC, kH = kU + 128;
  static_assert(kH + NT * KW <= 512, "tensor memory");
  constexpr int kHeadSteps = HPC == 2 ? 4 : 4 * KB;  // steps of 16 over a head's elements
  extern __shared__ unsigned char raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  __shared__ Small sh;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, quarter = warp & 3, part = warp >> 2;
  const int r = quarter * 32 + lane;
  const int segments = p.plan.segments;
  const Place<HPC> at(p, OUT ? segments : segments - 1);
  const AttnPass& a = *at.pass;
  const bool back = a.backward;
  // the segments' order is the pass's; the last one's state is the pass's own
  const int order = at.segment, segment = back ? segments - 1 - order : order;
  const int head = HPC == 2 ? r >> 6 : 0, h = at.h0 + head, v = HPC == 2 ? r & 63 : r;
  const bool mine = v < a.V && h < p.H;
  const int k0 = part * NH, ucol = HPC == 2 ? head * 64 + part * 16 : part * NH;  // state elements, U's columns
  const int ocol = (HPC == 2 ? head * 64 : 0) + part * kCols;                     // columns of S and O
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
  constexpr long long kept = (long long)KB * 64 * 128;  // a state in scratch: [k][lane]
  F2 H[NH / 2];
  {
    float first[NH];
    if (OUT && segments > 1) {
      const float* from = p.plan.states + ((long long)at.stream * segments + order) * kept;
#pragma unroll
      for (int i = 0; i < NH; ++i) first[i] = from[(k0 + i) * 128 + r];
    } else {
#pragma unroll
      for (int i = 0; i < NH; ++i) first[i] = OUT && a.first && mine && k0 + i < a.K ? a.first[state_at(i)] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NH / 2; ++i) H[i] = f2(first[2 * i], first[2 * i + 1]);
  }

  const F2 zero = f2(0.0f, 0.0f);
  F2 state_finite = zero;
  auto publish = [&]() {  // the state's terms to tensor memory
    uint32_t w[NT][NH / 2];
#pragma unroll
    for (int i = 0; i < NH / 2; ++i) {
      uint32_t s[NT];
      split<NT>(H[i], s, state_finite);
#pragma unroll
      for (int x = 0; x < NT; ++x) w[x][i] = s[x];
    }
#pragma unroll
    for (int x = 0; x < NT; ++x) tmem_st<NH / 2>(lanes + kH + x * KW + k0 / 2, w[x]);
    tmem_st_done();
  };
  const Rows<T, HPC> rq(a.q, at.n, at.h0, p.H, a.q_of, a.K), rk(a.k, at.n, at.h0, p.H, a.k_of, a.K),
      rv(a.v, at.n, at.h0, p.H, a.v_of, a.V);
  constexpr int kSubs = HPC == 2 ? 2 : KB;
  auto fetch = [&](int c, int stage) {
    unsigned char* tiles = sm + stage * Lay::kStage;
    if (OUT) rq.template load<kSubs>(tiles + Lay::kQ, c * kChunk, L, p.plan.vec);
    rk.template load<kSubs>(tiles + Lay::kK, c * kChunk, L, p.plan.vec);
    rv.template load<2>(tiles + Lay::kV, c * kChunk, L, p.plan.vec);
    cp_commit();
  };
  auto decays_of = [&](int i) {  // by the last warps: warp 0 issues the products
    const int x = warp - (16 - HPC);
    if (x >= 0)
      chunk_decays(p, a, at.n, min(at.h0 + x, p.H - 1), chunk_at(i) * kChunk, at.h0 + x < p.H ? L : 0, sh.decays[i & 1][x],
                   &sh.wrong[i & 1]);
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
        const float* x = &sh.dots[i / kCols * 4][i % kCols];
        const float y = HPC == 2 ? x[2 * hd * kCols] + x[(2 * hd + 1) * kCols]
                                 : (x[0] + x[kCols]) + (x[2 * kCols] + x[3 * kCols]);
        a.dot[((long long)at.n * p.H + at.h0 + hd) * S + t] = y;
      }
    }
  };
  // outputs of lane v
  T* out = static_cast<T*>(a.o.p) + at.n * a.o.ns + (long long)(h / a.o_of) * a.V + v;
  float* out32 = a.o32 + ((long long)at.n * S * p.H + h) * a.V + v;
  const long long ss32 = (long long)p.H * a.V;
  const T* dot_row = static_cast<const T*>(a.dot_with.p) + at.n * a.dot_with.ns + (long long)(h / a.o_of) * a.V + v;
  auto put = [&](int t, float y) {
    if (!mine || t >= S) return;
    if (a.o32) out32[t * ss32] = y;
    else if (a.o.p) out[t * a.o.ss] = Elem<T>::from_f(y);
  };

  if (count > 0) {
    fetch(chunk_at(0), 0);
    decays_of(0);
  }
  if (OUT) publish();
  uint32_t phase = 0;
  double left = 0.0;  // logarithm of the segment's decay
  const float near = a.so * a.su;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int c = chunk_at(i), t0 = c * kChunk;
    const int stage = Lay::kStages == 2 ? i & 1 : 0;
    unsigned char* tiles = sm + stage * Lay::kStage;
    const Decays* dec = sh.decays[i & 1];
    cp_wait();
    to_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tq = su32(tiles + Lay::kQ), tk = su32(tiles + Lay::kK), tv = su32(tiles + Lay::kV);
    const uint32_t ts = su32(sm + Lay::kScaled), tp = Lay::kOver ? tk : su32(sm + Lay::kP);
    if (OUT && tid == 0) {
      constexpr uint32_t id = idesc_of(64 * HPC);
      const uint64_t dq = smem_desc_sw128(tq), dk = smem_desc_sw128(tk);
      products<kIn, kIn, NT, kHeadSteps>([&](int x, int y, int s, uint32_t more) {
        const uint32_t o = ((s / 4) * kSub + (s % 4) * 32) >> 4;
        tc_mma(tmem + kS, dq + (x * kTile >> 4) + o, dk + (y * kTile >> 4) + o, id, more);
      });
      tc_commit(su32(&sh.bars[0]));
      products<NT, kIn, NT, kHeadSteps>([&](int x, int y, int s, uint32_t more) {
        tc_mma_ts(tmem + kOi, tmem + kH + x * KW + s * 8, dq + ((y * kTile + (s / 4) * kSub + (s % 4) * 32) >> 4), id, more);
      });
      tc_commit(su32(&sh.bars[1]));
    }
    if (Lay::kStages == 2 && i + 1 < count) fetch(chunk_at(i + 1), stage ^ 1);
    if (Lay::kStages == 1 && i + 1 < count) {
      const int t1 = chunk_at(i + 1) * kChunk;
      if (OUT) rq.prefetch(t1, L);
      rk.prefetch(t1, L);
      rv.prefetch(t1, L);
    }
    if (i > 0) dots_out(chunk_at(i - 1));
    F2 finite = zero;
    bool bad = false;
    // a warp's quarter of the lanes is also its quarter of the SM: with one
    // head S has rows for two of them, and the other two scale K
    if constexpr (OUT && HPC == 1 && !Lay::kOver) {
      const int thread = (part * 2 + (quarter & 1)) * 32 + lane;
      if (quarter >= 2) scale_tile<T, HPC, kSubs, kThreads / 2>(tiles + Lay::kK, sm + Lay::kScaled, dec, thread, finite);
      else bad = !tile_finite<kThreads / 2>(tiles + Lay::kV, thread);
    } else {
      scale_tile<T, HPC, kSubs, kThreads>(tiles + Lay::kK, sm + Lay::kScaled, dec, tid, finite);
      bad = !tile_finite<kThreads>(tiles + Lay::kV, tid);
    }
    if (i + 1 < count) decays_of(i + 1);
    if constexpr (OUT) {
      if constexpr (Lay::kOver) __syncthreads();  // K is read before P takes its place
      wait(0, phase);
      if (HPC == 2 || quarter < 2) {
        // row m of S, 16 of its columns
        const int m = r & 63, n0 = part * kCols;
        const Decays& d = dec[head];
        float s[kCols];
        tmem_ld16(lanes + kS + ocol, s);
        const F2 hi = f2(d.hi[m], d.hi[m]), lo = f2(d.lo[m], d.lo[m]);
        uint32_t w[NT][kCols / 2];
#pragma unroll
        for (int j = 0; j < kCols; j += 2) {
          const float2 nh = *reinterpret_cast<const float2*>(&d.nhi[n0 + j]), nl = *reinterpret_cast<const float2*>(&d.nlo[n0 + j]);
          const F2 f = exp2_fast2(add2(add2(hi, f2(nh.x, nh.y)), add2(lo, f2(nl.x, nl.y))));
          float2 x = f2_get(mul2(f2(s[j], s[j + 1]), f));
          const int n = n0 + j;
          x.x = (back ? n >= m : n <= m) ? x.x : 0.0f;
          x.y = (back ? n + 1 >= m : n + 1 <= m) ? x.y : 0.0f;
          uint32_t t[NT];
          split<NT>(f2(x.x, x.y), t, finite);
#pragma unroll
          for (int e = 0; e < NT; ++e) w[e][j / 2] = t[e];
        }
        unsigned char* row = (Lay::kOver ? tiles + Lay::kK : sm + Lay::kP) + (HPC == 2 ? r : m) * 128;
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
          for (int x = 0; x < kCols / 8; ++x)
            *reinterpret_cast<uint4*>(row + e * Lay::kPTerm + (((part * (kCols / 8) + x) ^ (m & 7)) << 4)) =
                make_uint4(w[e][4 * x], w[e][4 * x + 1], w[e][4 * x + 2], w[e][4 * x + 3]);
      }
    }
    bad = bad || !is_finite(finite) || (mine && !is_finite(state_finite)) || sh.wrong[i & 1] || sh.gave_up;
    to_async();
    tc_fence_before();
    const bool by_step = __syncthreads_or(bad);
    tc_fence_after();
    if (tid == 0) sh.wrong[i & 1] = 0;
    left += dec[head].log2;
    if (!by_step) {
      if (tid == 0) {
        const uint64_t dv = desc_mn(tv), ds = desc_mn(ts), dp = smem_desc_sw128(tp);
        constexpr uint32_t idu = idesc_of(HPC == 2 ? 128 : 64 * KB) | kRowsA | kRowsB;
        products<kIn, kTerms, kTerms, 4>([&](int x, int y, int s, uint32_t more) {
          tc_mma(tmem + kU, dv + ((x * kTile + s * 2048) >> 4), ds + ((y * kTile + s * 2048) >> 4), idu, more);
        });
        tc_commit(su32(&sh.bars[2]));
        if (OUT) {
          constexpr uint32_t ido = idesc_of(64 * HPC) | kRowsA;
          products<kIn, NT, NT, 4>([&](int x, int y, int s, uint32_t more) {
            tc_mma(tmem + kS, dv + ((x * kTile + s * 2048) >> 4), dp + ((y * Lay::kPTerm + s * 32) >> 4), ido, more);
          });
          tc_commit(su32(&sh.bars[3]));
        }
      }
      float far[kCols];
      if constexpr (OUT) {
        wait(1, phase);
        tmem_ld16(lanes + kOi + ocol, far);
      }
      wait(2, phase);
      const float e = dec[head].total;
#pragma unroll
      for (int j = 0; j < NH; j += 16) {
        float u[16];
        tmem_ld16(lanes + kU + ucol + j, u);
#pragma unroll
        for (int x = 0; x < 8; ++x) H[j / 2 + x] = fma2(f2(e, e), H[j / 2 + x], f2(u[2 * x], u[2 * x + 1]));
      }
      if constexpr (OUT) {
        publish();
        wait(3, phase);
        float o[kCols];
        tmem_ld16(lanes + kS + ocol, o);
        const float* cq = &dec[head].cq[part * kCols];
#pragma unroll
        for (int x = 0; x < kCols; x += 2) {
          const float2 f = *reinterpret_cast<const float2*>(cq + x);
          const float2 y = f2_get(fma2(f2(f.x, f.y), f2(far[x], far[x + 1]), mul2(f2(near, near), f2(o[x], o[x + 1]))));
          o[x] = y.x, o[x + 1] = y.y;
        }
        const int t1 = t0 + part * kCols, rows = min(kCols, S - t1);
        if (mine) {
          if (a.o32) {
            float* to = out32 + t1 * ss32;
#pragma unroll
            for (int x = 0; x < kCols; ++x, to += ss32)
              if (x < rows) *to = o[x];
          } else if (a.o.p) {
            T* to = out + t1 * a.o.ss;
#pragma unroll
            for (int x = 0; x < kCols; ++x, to += a.o.ss)
              if (x < rows) *to = Elem<T>::from_f(o[x]);
          }
        }
        if (a.dot) {
          const T* with = dot_row + t1 * a.dot_with.ss;
#pragma unroll
          for (int x = 0; x < kCols; ++x, with += a.dot_with.ss) o[x] = mine && t1 + x < L ? o[x] * Elem<T>::to_f(*with) : 0.0f;
          int to = 0;
          lanes_sum<kCols, 16, 1>(o, lane, to);
          sh.dots[warp][to] = o[0];
        }
      } else {
#pragma unroll
        for (int x = 0; x < NH / 2; ++x) state_finite = fma2(H[x], zero, state_finite);
      }
    } else {
      if (__syncthreads_or(sh.gave_up)) break;
      // step by step, from the operands themselves
      if (OUT) wait(1, phase);
      const int rows = min(kChunk, L - t0);
      const int hc = min(h, p.H - 1);
      const T* q = head_rows<T>(a.q, at.n, hc, a.q_of, a.K);
      const T* k = head_rows<T>(a.k, at.n, hc, a.k_of, a.K);
      const T* x = head_rows<T>(a.v, at.n, hc, a.v_of, a.V);
      float g[NH];
#pragma unroll
      for (int b = 0; b < NH / 2; ++b) {
        const float2 y = f2_get(H[b]);
        g[2 * b] = y.x, g[2 * b + 1] = y.y;
      }
#pragma unroll 1
      for (int j = 0; j < rows; ++j) {
        const int m = back ? rows - 1 - j : j;
        const long long t = t0 + m;
        const float d = dec[head].d[m], val = mine ? a.su * Elem<T>::to_f(x[t * a.v.ss + v]) : 0.0f;
        float y = 0.0f;
#pragma unroll
        for (int b = 0; b < NH; ++b) {
          if (mine && k0 + b < a.K) {
            g[b] = fmaf(Elem<T>::to_f(k[t * a.k.ss + k0 + b]), val, back ? g[b] : d * g[b]);
            if (OUT) y = fmaf(Elem<T>::to_f(q[t * a.q.ss + k0 + b]), g[b], y);
            if (back) g[b] *= d;
          }
        }
        if (OUT) {
          sh.part[part][r] = y;
          __syncthreads();
          if (part == 0) {
            y = a.so * ((sh.part[0][r] + sh.part[1][r]) + (sh.part[2][r] + sh.part[3][r]));
            put((int)t, y);
            if (a.dot) {
              const float w = warp_sum(mine ? y * Elem<T>::to_f(dot_row[t * a.dot_with.ss]) : 0.0f);
              if (lane == 0) sh.dots[m / kCols * 4 + quarter][m % kCols] = w;
            }
          }
          __syncthreads();
        }
      }
      if (OUT)
        for (int m = rows + part; m < kChunk; m += 4) put(t0 + m, 0.0f);
#pragma unroll
      for (int b = 0; b < NH / 2; ++b) H[b] = f2(g[2 * b], g[2 * b + 1]);
      state_finite = zero;
      if (OUT) {
        publish();
      } else {
#pragma unroll
        for (int b = 0; b < NH / 2; ++b) state_finite = fma2(H[b], zero, state_finite);
      }
      // the barriers that this chunk did not use complete all the same
      if (tid == 0) {
        tc_commit(su32(&sh.bars[2]));
        if (OUT) tc_commit(su32(&sh.bars[3]));
      }
      wait(2, phase);
      if (OUT) wait(3, phase);
      __syncthreads();
    }
    if (Lay::kStages == 1 && i + 1 < count) fetch(chunk_at(i + 1), 0);
    phase ^= 1;
  }
  cp_wait();
  __syncthreads();
  if (count > 0 && !sh.gave_up) dots_out(chunk_at(count - 1));
  if (OUT) {
    // the rows behind the last live chunk
    for (int t = max(c_live, c_begin) * kChunk + part; t < min(c_end * kChunk, S); t += 4) put(t, 0.0f);
    if (order == segments - 1) {
      float with = 0.0f;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const float2 y = f2_get(H[i / 2]);
        if (mine && k0 + i < a.K) {
          if (a.last) a.last[state_at(i)] = i % 2 ? y.y : y.x;
          if (a.with) with = fmaf(a.with[state_at(i)], i % 2 ? y.y : y.x, with);
        }
      }
      if (a.cross) {
        with = warp_sum(with);
        if (lane == 0) sh.part[0][warp] = with;
        __syncthreads();
        if (tid < HPC && at.h0 + tid < p.H) {
          const float* x = sh.part[0];
          float y = 0.0f;
          for (int w = 0; w < 16; ++w)
            if (HPC == 1 || (w & 3) >> 1 == tid) y += x[w];
          a.cross[(long long)at.n * p.H + at.h0 + tid] = y;
        }
      }
    }
  } else {
    float* to = p.plan.states + ((long long)at.stream * segments + order) * kept;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const float2 y = f2_get(H[i / 2]);
      to[(k0 + i) * 128 + r] = mine && k0 + i < a.K ? (i % 2 ? y.y : y.x) : 0.0f;
    }
    if (part == 0 && lane == 0 && (HPC == 2 ? quarter % 2 == 0 : quarter == 0))
      p.plan.left[((long long)at.stream * segments + order) * 2 + head] = left;
  }
  // nothing is in flight any more, unless a wait has failed: then what was issued gets some time
  if (sh.gave_up && tid == 0) {
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

template <typename T, int HPC, int KB, int NT>
cudaError_t launch_chunks_of(const AttnParams& p, cudaStream_t s, int* launches) {
  constexpr size_t smem = Layout<T, HPC, NT>::kBytes;
  const long long streams = (long long)p.passes * p.N * ((p.H + HPC - 1) / HPC);
  auto whole = attn_chunk_kernel<T, HPC, KB, NT, true>;
  cudaError_t e = cudaFuncSetAttribute(whole, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (p.plan.segments > 1) {
    auto sums = attn_chunk_kernel<T, HPC, KB, kTerms, false>;
    constexpr size_t sums_smem = Layout<T, HPC, kTerms>::kBytes;
    e = cudaFuncSetAttribute(sums, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sums_smem);
    if (e != cudaSuccess) return e;
    sums<<<(unsigned)(streams * (p.plan.segments - 1)), kThreads, sums_smem, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
    attn_join_kernel<HPC, KB><<<dim3((unsigned)streams, KB * 64 * 128 / 256), 256, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
  }
  whole<<<(unsigned)(streams * p.plan.segments), kThreads, smem, s>>>(p);
  if ((e = cudaGetLastError()) == cudaSuccess) ++*launches;
  return e;
}

template <typename T, int NT>
cudaError_t launch_chunks_in(const AttnParams& p, cudaStream_t s, int* launches) {
  // every pass has the same two sizes, in one order or the other
  if (p.pass[0].K <= 64 && p.pass[0].V <= 64) return launch_chunks_of<T, 2, 1, NT>(p, s, launches);
  return p.plan.deep == 64 ? launch_chunks_of<T, 1, 1, NT>(p, s, launches) : launch_chunks_of<T, 1, 2, NT>(p, s, launches);
}

// P and the state as three terms where float32 comes of them: for float32
// rows, and in gradients, whose products for the decays are added up over the
// sequence.  A 16-bit output keeps less than the 2^-17 of two.
template <typename T>
cudaError_t launch_chunks(const AttnParams& p, cudaStream_t s, int* launches) {
  if constexpr (kSplit<T> < kTerms)
    if (!p.gradient) return launch_chunks_in<T, 2>(p, s, launches);
  return launch_chunks_in<T, kTerms>(p, s, launches);
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
