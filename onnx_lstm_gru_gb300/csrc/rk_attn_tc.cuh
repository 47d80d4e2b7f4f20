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
// Values run along the 128 lanes of tensor memory, where the state lives too:
// it needs no transposition between U, where it is added to, and Oi, where it
// is the product's A operand.  It is kept in float32, or as three bfloat16 terms
// that add up to it.
//
// The tensor cores multiply bfloat16.  A factor of more bits is a sum of two
// or three bfloat16 terms (each the rounding of what the ones before left),
// and a product the sum of the terms' products down to 2^-24 of it, smallest
// first; bfloat16 operands are one term, Half two, float32 three, and what is
// computed here (P, ck K, H) three, or P and H two where only a 16-bit output
// comes of them (launch_chunks).  Differences of G are exact to 2^-24: sums
// are 64-bit whole numbers of 2^-32, kept as whole part and fraction.
//
// Where a chunk's decays (and the scale) stay between 2^-80 and 2^20, P_mn 2^-G_m is
// S_mn 2^-G_n: then no power is taken for each pair, and O is added to Oi before
// 2^G_m scales both.  (Backward the same from the chunk's end.)  Chunks that decay
// or grow further take the powers pair by pair and keep the two apart.
//
// A block runs one state (two, stacked along the lanes, where heads have at
// most 64 elements: of the products' 128 x 128 blocks the diagonal ones are
// used) over a piece of the sequence, in groups of warps that meet at
// mbarriers:
//   eight read S and write P;
//   eight hand out the outputs;
//   eight keep the state, add U to it and scale K for the next chunk;
//   one issues the products, one copies tiles in and out (TMA, for bfloat16
//   rows of whole 16-byte pieces; else the three groups do), and one for each
//   head takes the decays of later chunks.
// The products of one chunk run while the next one's operands are made ready:
// O_i follows P_i; S_(i+1) and U_(i+1) follow ck K; Oi_(i+1), or with three terms
// what is small of it, follows the outputs of i.
//
// Infinities and NaN must not reach other steps through the products' zeros, and
// sums that are scaled down once they are complete must not pass float32's range
// before.  So a chunk is run step by step instead where a product of P, a scaled
// key or an element of the state is 2^100 or more (looked at while they are split
// into terms; from 2^94 on at the earliest), or an element of the queries or values
// 2^20 or more: below that O + Oi is at most 64 + 128 products of 2^120, and U 64.
//
// What bounds it are the warps' own instructions and their waits for each
// other, not the products or HBM: 512 x 64 x 16 heads of 64, bf16, 114 us (2.5
// TB/s, 2.2 warp instructions a clock and multiprocessor, the tensor pipe 29 %
// busy); the gradient of 512 x 8 x 16 heads of 128 141 us (2.1, 20 %); 777 x 8 x 10
// heads of 72 x 103 in float32, 80 blocks, 110 to 126 us as the lengths are (1.8,
// 25 %).  Step by step the three take 2316, 2319 and 646 us.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include <cudaTypedefs.h>

#include "rk_attn.h"
#include "rk_proj_tc.cuh"
#include "rk_ssm_common.cuh"

namespace rk {
namespace atc {

using namespace ptc;

constexpr int kChunk = 64, kGroup = 256, kThreads = 3 * kGroup + 128, kTerms = 3;
constexpr int kGroupWarps = kGroup / 32;
constexpr uint32_t kSub = kChunk * 128;      // bytes of 64 rows of 64 elements
constexpr uint32_t kTile = 2 * kSub;         // an operand's term: 64 rows of 128 elements, or of two heads of 64
constexpr int kCols = kChunk / 2;            // of a chunk's columns of S and O, those of a thread
// A wait that has failed: so many tries, each of which may take up to kTryNs
// (together two seconds at most, and some tens of milliseconds at least).
constexpr int kWaitTries = 1000000;
constexpr uint32_t kTryNs = kAttnTryNs;

template <typename T>
constexpr int kSplit = sizeof(T) == 4 ? 3 : 2;
template <>
constexpr int kSplit<__nv_bfloat16> = 1;

// Shared memory: operand tiles (bfloat16: two stages), ck K (two where only
// sums of states are wanted), P in NT terms (float32: where K was).
template <typename T, int HPC, int NT, bool OUT>
struct Layout {
  static constexpr int kIn = kSplit<T>;
  static constexpr int kStages = kIn == 1 ? 2 : 1;
  static constexpr uint32_t kK = 0, kV = kIn * kTile, kQ = 2 * kIn * kTile, kStage = (OUT ? 3 : 2) * kIn * kTile;
  static constexpr uint32_t kScaled = kStages * kStage;
  static constexpr int kScaledCount = OUT ? 1 : 2;
  static constexpr uint32_t kAfter = kScaled + kScaledCount * kTerms * kTile;
  static constexpr bool kOver = kIn == 3;
  static constexpr uint32_t kP = kOver ? kK : kAfter;
  static constexpr uint32_t kPTerm = HPC * kSub;
  static constexpr uint32_t kOut = kAfter + (kOver || !OUT ? 0 : NT * kPTerm);  // outputs, where they are copied out
  static constexpr uint32_t kAfterOut = kOut + (OUT && kIn == 1 ? kTile : 0);
  // what outputs are multiplied with for the decays: where K was, if there is no room
  static constexpr bool kWithApart = kIn == 1 && OUT && NT == kTerms && HPC == 1;
  static constexpr uint32_t kEnd = kAfterOut + (kWithApart ? kTile : 0);
  static_assert(NT * kPTerm <= kIn * kTile || !kOver, "P fits over K");
  static constexpr size_t kBytes = kEnd + 1024;  // alignment
};

// Decays of a chunk, by head of the block.
struct Decays {
  float hi[kChunk], lo[kChunk];  // signed G: whole part and fraction
  float cq[kChunk], ck[kChunk];  // so 2^.. of the state's part of a step's output, su 2^.. of a step's part of the state
  float bn[kChunk];              // su over 2^.. of cq: what takes S to P where the chunk's decays are mild
  long long log2;                // the whole chunk's G
  float total;                   // the decay
  int mild;
};

// A barrier that could be two phases ahead of one who waits for it has a
// second one for odd chunks.
enum Bar {
  kTiles, kDone = kTiles + 2, kPairs = kDone + 2, kSteps = kPairs + 2,  // of warps
  kGotS, kGotU, kGotOi = kGotU + 2, kGotO, kFull = kGotO + 2, kWith = kFull + 2, kStored, kDecay, kBars = kDecay + 3
};

// Chunks' flags take turns.  Two heads' decay warps may each set one, and the
// first head's clears the flag of chunk i + kClear while it is at chunk i.  Nobody
// sets that flag before: the second head's warp comes to a chunk once the one
// three before it is done, for which both heads' decays have been taken, and the
// others wait for the chunk's own decays.  Nobody still reads it for chunk i +
// kClear - kFlags, eleven back: chunk i - 3 is done, with which all but the copying
// warp have read its flag, and that one fetched its tiles after it had read the
// flag of chunk i - 6.
constexpr int kFlags = 16, kClear = 5;
struct Small {
  __align__(16) Decays decays[3][2];
  float dots[2][kGroupWarps][kCols];  // of a chunk and the one before
  float part[2][128];
  uint64_t bars[kBars];
  uint32_t tmem;
  int bad[kFlags];  // chunks to be run step by step
  volatile int gave_up;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return Elem<__nv_bfloat16>::pair_from_f(lo, hi); }
__device__ __forceinline__ F2 pair_of(uint32_t u) { return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }

// Two factors as N terms each; the first terms are added to `sum` 2^29 times,
// which stays finite only while all of them are below 2^100 (one of 2^100 alone is
// 2^129, and what has been added up is not below -2^128).
constexpr float kFar = 536870912.0f;
template <int N>
__device__ __forceinline__ void split(F2 x, uint32_t (&t)[N], F2& sum) {
  float2 v = f2_get(x);
  t[0] = pack2(v.x, v.y);
  F2 h = pair_of(t[0]);
  sum = fma2(h, f2(kFar, kFar), sum);
#pragma unroll
  for (int i = 1; i < N; ++i) {
    x = fma2(h, f2(-1.0f, -1.0f), x);
    v = f2_get(x);
    t[i] = pack2(v.x, v.y);
    if (i + 1 < N) h = pair_of(t[i]);
  }
}
__device__ __forceinline__ bool in_range(F2 sum) {
  const float2 v = f2_get(sum);
  return v.x - v.x == 0.0f && v.y - v.y == 0.0f;
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
// 8 or 16 columns; what is read may be used after tmem_ld_done.
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&x)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
        "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
      : "r"(addr)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld_done(float (&x)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));  // not before
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

__device__ __forceinline__ void to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Whether the barrier's phase has ended; the warp is taken off the scheduler
// for some time while it has not.
__device__ __forceinline__ bool bar_try_long(uint32_t b, uint32_t par) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b), "r"(par), "r"(kTryNs)
      : "memory");
  return ok != 0;
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}
__device__ __forceinline__ void copy_in(uint32_t dst, const CUtensorMap* map, int x, int h, int t, int n, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(t), "r"(n), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void copy_out(const CUtensorMap* map, int x, int h, int t, int n, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(h), "r"(t), "r"(n), "r"(src)
               : "memory");
}

// Set where a wait has failed (one per element type's unit; what reads it is static, too).
static __device__ int gave_up_status;

// What a launch gets: the call, and where tiles are copied by TMA the rows of
// each pass as tensors (elements, heads, steps, batch rows) in boxes of 64
// elements of 64 steps.
struct ChunkArgs {
  CUtensorMap q[3], k[3], v[3], o[3], with[3];
  AttnParams p;
};

// What a block works on.
template <int HPC>
struct Place {
  int n, h0, segment, stream, pass;
  __device__ __forceinline__ Place(const AttnParams& p, int segments) {
    long long id = blockIdx.x;
    segment = (int)(id % segments);
    id /= segments;
    stream = (int)id;
    const int groups = (p.H + HPC - 1) / HPC;
    h0 = (int)(id % groups) * HPC;
    id /= groups;
    n = (int)(id % p.N);
    pass = (int)(id / p.N);
  }
};

// 2^(whole + fraction) without rounding the sum.
__device__ __forceinline__ float pow2_of(long long g) {
  const int whole = (int)(g >> 32);
  const float part = exp2_fast((float)(uint32_t)g * 2.3283064365386963e-10f);
  if (whole < -126) return 0.0f;
  return whole > 127 ? __int_as_float(0x7f800000) : part * __int_as_float((whole + 127) << 23);
}

// 2^300 in units of 2^-32 of its logarithm: every float32 but 0 times that is infinite, and through it 0.
constexpr long long kAll = 300LL << 32;
// The logarithm x of a decay to base 2 in units of 2^-32, to the nearest: a
// memory of thousands of steps adds up as many of the same rounding.  What is
// below -1e5 leaves nothing in float32, what is above 1e5 more than there is, and a
// chunk's sum of either stays within 2^24.
__device__ __forceinline__ long long fixed_log2(float x) {
  x = fminf(fmaxf(x, -1.0e5f), 1.0e5f);
  constexpr float kLow = (float)(1.4426950408889634074 - (double)kLog2e);
  const float t = x * kLog2e, rest = fmaf(x, kLog2e, -t) + x * kLow;
  return __float2ll_rn(t * 4294967296.0f) + (long long)__float2int_rn(rest * 4294967296.0f);
}

// One warp: the decays of a chunk of which the lane has x0 and x1, the
// logarithms of two steps; whether it has to be run step by step.
__device__ __forceinline__ bool chunk_decays(const AttnPass& a, float x0, float x1, Decays& out) {
  const bool backward = a.backward;
  const int lane = threadIdx.x % 32;
  long long fix[2];
  // NaN, or growth that no float32 holds for long
  bool bad = !(x0 < 80.0f) || !(x1 < 80.0f);
  fix[0] = fixed_log2(x0), fix[1] = fixed_log2(x1);
  long long sum = fix[0] + fix[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  const long long total = __shfl_sync(0xffffffffu, sum, 31);
  // the scale's power goes with the decays': together they stay in float32's range
  const int limit = 80 - abs((int)(__float_as_uint(a.so * a.su) >> 23 & 255) - 127);
  bool mild = true;
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const long long G = j ? sum : sum - fix[1], s = backward ? -G : G;
    const int i = 2 * lane + j;
    out.hi[i] = (float)(int)(s >> 32);
    out.lo[i] = (float)((uint32_t)s >> 8) * 5.9604644775390625e-8f;
    const long long from = backward ? total - G : G;
    bad = bad || G >> 32 > 120 || (total - G) >> 32 > 120;
    mild = mild && from >> 32 >= -limit && from >> 32 < min(limit, 20);
    const float up = pow2_of(G), down = pow2_of(total - G);
    out.cq[i] = a.so * (backward ? down : up);
    out.ck[i] = a.su * (backward ? up : down);
    out.bn[i] = a.su * pow2_of(-from);
  }
  mild = __all_sync(0xffffffffu, mild);
  if (lane == 0) out.total = pow2_of(total), out.log2 = total, out.mild = mild;
  return __any_sync(0xffffffffu, bad);
}

// Row operands of a block, as pointers to its first head's elements.
template <typename T>
__device__ __forceinline__ const T* head_rows(const RowsArg& a, int n, int h, int of, int size) {
  return static_cast<const T*>(a.p) + n * a.ns + (long long)(h / of) * size;
}

// A group's threads' parts of a tile: pieces of 8 elements of rows, 512 in each
// of the two sub-tiles, which are the elements from 0 and 64 on, or two heads.
__device__ __forceinline__ uint32_t piece_at(int i) {  // i: 0 .. 511
  const int r = i / 8, c = i % 8;
  return r * 128 + ((c ^ (r & 7)) << 4);
}
template <typename T, int HPC>
struct Rows {
  const T* src;        // the thread's first piece of sub-tile 0 of the next chunk; 32 rows on lies its second
  long long ss, step;  // from row to row; to the chunk after it
  int next;            // to sub-tile 1
  int on;              // bit b: sub-tile b has the thread's elements
  int size;
  // t0: the first chunk's start; step: to the next one's
  __device__ __forceinline__ Rows(const RowsArg& a, int n, int h0, int H, int of, int size_, int t0, int step_)
      : ss(a.ss), step(step_ * a.ss), size(size_) {
    const int thread = threadIdx.x % kGroup, c = 8 * (thread % 8);
    src = head_rows<T>(a, n, h0, of, size) + (t0 + thread / 8) * a.ss + c;
    next = HPC == 1 ? 64 : (min(h0 + 1, H - 1) / of - h0 / of) * size;
    on = (c < size ? 1 : 0) | ((HPC == 1 ? 64 + c < size : c < size && h0 + 1 < H) ? 2 : 0);
  }
  // Reads the next chunk's 64 rows, of which `rows` are steps, into the tile.
  // Other steps, elements from `size` on and heads that there are not are zeros.
  template <int SUBS>
  __device__ __forceinline__ void load(unsigned char* tile, int rows, int vec) {
    constexpr int kIn = kSplit<T>;
    const int thread = threadIdx.x % kGroup;
#pragma unroll 1
    for (int b = 0; b < SUBS; ++b) {
      const int first = (HPC == 2 ? 0 : 64 * b) + 8 * (thread % 8);
      float x[2][8];  // both are on their way together
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const bool fetch = thread / 8 + 32 * half < rows && (on >> b & 1);
        const T* from = src + b * next + half * 32 * ss;
        fill(x[half], 0.0f);
        if (vec) {
          if (fetch) {
            if constexpr (sizeof(T) == 4) {
              float y[4];
              Piece<T, 4>::load(from, y);
              x[half][0] = y[0], x[half][1] = y[1], x[half][2] = y[2], x[half][3] = y[3];
              if (first + 4 < size) {
                Piece<T, 4>::load(from + 4, y);
                x[half][4] = y[0], x[half][5] = y[1], x[half][6] = y[2], x[half][7] = y[3];
              }
            } else {
              Piece<T, 8>::load(from, x[half]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (fetch && first + i < size) x[half][i] = Elem<T>::to_f(from[i]);
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        unsigned char* dst = tile + b * kSub + piece_at(thread + half * kGroup);
        uint32_t w[kIn][4];
        F2 unused = f2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t s[kIn];
          split<kIn>(f2(x[half][2 * i], x[half][2 * i + 1]), s, unused);
#pragma unroll
          for (int j = 0; j < kIn; ++j) w[j][i] = s[j];
        }
#pragma unroll
        for (int j = 0; j < kIn; ++j) *reinterpret_cast<uint4*>(dst + j * kTile) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
      }
    }
    src += step;
  }
  // Has the next chunk's rows brought into L2.
  __device__ __forceinline__ void prefetch(int rows) const {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int half = 0; half < 2; ++half)
        if ((int)(threadIdx.x % kGroup) / 8 + 32 * half < rows && (on >> b & 1))
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src + b * next + half * 32 * ss));
  }
};

// ck K as three terms, by a group.
template <typename T, int HPC, int SUBS>
__device__ __forceinline__ void scale_tile(const unsigned char* k, unsigned char* out, const Decays* d, F2& range) {
  constexpr int kIn = kSplit<T>;
  const int thread = threadIdx.x % kGroup;
#pragma unroll 2
  for (int i = 0; i < 2 * SUBS; ++i) {
    const int b = i / 2, piece = thread + i % 2 * kGroup;
    const uint32_t at = b * kSub + piece_at(piece);
    const float f = d[HPC == 2 ? b : 0].ck[piece / 8];
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
      split<kTerms>(mul2(x, f2(f, f)), s, range);
#pragma unroll
      for (int j = 0; j < kTerms; ++j) w[j][e] = s[j];
    }
#pragma unroll
    for (int j = 0; j < kTerms; ++j)
      *reinterpret_cast<uint4*>(out + j * kTile + at) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
  }
}

// Whether a tile's first term is below 2^20, by THREADS threads: the largest of
// the magnitudes as whole numbers, 16 bits each.
constexpr uint32_t kMost = (127 + 20) << 7;
template <int THREADS, int BYTES>
__device__ __forceinline__ bool tile_in_range(const unsigned char* tile, int thread) {
  uint32_t top = 0;
#pragma unroll 4
  for (int i = 0; i < BYTES / 16 / THREADS; ++i) {
    const uint4 u = *reinterpret_cast<const uint4*>(tile + (i * THREADS + thread) * 16);
    top = __vmaxu2(top, u.x & 0x7fff7fffu), top = __vmaxu2(top, u.y & 0x7fff7fffu);
    top = __vmaxu2(top, u.z & 0x7fff7fffu), top = __vmaxu2(top, u.w & 0x7fff7fffu);
  }
  return (top & 0xffffu) < kMost && (top >> 16) < kMost;
}

// One thread: the products of NA terms of A and NB of B down to 2^-8 NT,
// smallest first, STEPS products of 16 each.  LAST 1: all but the first terms'
// own, which FIRST 0 are.
template <int NA, int NB, int NT, int STEPS, int LAST = 0, int FIRST = NT - 1, typename F>
__device__ __forceinline__ void products(F mma, uint32_t more = 0) {
#pragma unroll
  for (int sum = (NA + NB - 2 < FIRST ? NA + NB - 2 : FIRST); sum >= LAST; --sum) {
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int b = sum - a;
      if (b < 0 || b >= NB) continue;
#pragma unroll 1
      for (int s = 0; s < STEPS; ++s) {
        mma(a, b, s, more);
        more = 1;
      }
    }
  }
}

// Waits for a barrier's phase of parity par.  Once a wait has failed all of
// them return at once: the loops run out, and what they compute is undefined.
// There are waits everywhere, and the code around them has to stay in the
// instruction cache: a count of tries is less of it than a clock.
__device__ __forceinline__ void wait_bar(Small& sh, int bar, uint32_t par, int limit = kWaitTries) {
  const uint32_t b = su32(&sh.bars[bar]);
#pragma unroll 1
  for (int tries = limit; !bar_try_long(b, par); --tries)
    if (tries == 0 || sh.gave_up) {
      sh.gave_up = gave_up_status = 1;
      break;
    }
  tc_fence_after();
}
// The warp's writes and reads so far are done: to shared memory for the
// products, and of tensor memory.
__device__ __forceinline__ void arrive_bar(Small& sh, int bar) {
  to_async();
  tc_fence_before();
  __syncwarp();
  if (threadIdx.x % 32 == 0) bar_arrive(su32(&sh.bars[bar]));
}

// The chunk that starts at t0 step by step, by the group that keeps the state;
// g: the thread's elements of it.  Returns the phases that the steps' barrier has had.
// Not inlined: it is there for infinities and NaN.
template <typename T, int HPC, int NH, bool OUT>
__device__ __noinline__ int run_steps(const AttnParams& p, int pass, int n, int h0, int t0, int L, float (*dots)[kCols],
                                      Small& sh, int meetings, float* g) {
  const AttnPass& a = p.pass[pass];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, quarter = warp & 3, part = warp >> 2 & 1, r = quarter * 32 + lane;
  const int head = HPC == 2 ? r >> 6 : 0, h = h0 + head, v = HPC == 2 ? r & 63 : r, k0 = part * NH;
  const bool mine = v < a.V && h < p.H, back = a.backward;
  const int rows = min(kChunk, L - t0), hc = min(h, p.H - 1);
  const T* q = head_rows<T>(a.q, n, hc, a.q_of, a.K);
  const T* k = head_rows<T>(a.k, n, hc, a.k_of, a.K);
  const T* x = head_rows<T>(a.v, n, hc, a.v_of, a.V);
  const float* decay = static_cast<const float*>(p.decay.p) + n * p.decay.ns + hc;
  T* out = static_cast<T*>(a.o.p) + n * a.o.ns + (long long)(hc / a.o_of) * a.V + v;
  const T* with = static_cast<const T*>(a.dot_with.p) + n * a.dot_with.ns + (long long)(hc / a.o_of) * a.V + v;
  auto put = [&](long long t, float y) {
    if (!mine || t >= p.S) return;
    if (a.o32) a.o32[(((long long)n * p.S + t) * p.H + h) * a.V + v] = y;
    else if (a.o.p) out[t * a.o.ss] = Elem<T>::from_f(y);
  };
#pragma unroll 1
  for (int j = 0; j < rows; ++j) {
    const int m = back ? rows - 1 - j : j;
    const long long t = t0 + m;
    const float d = expf((p.decay.p ? decay[t * p.decay.ss] : 0.0f) + (p.bias ? p.bias[hc] : 0.0f)), val = mine ? a.su * Elem<T>::to_f(x[t * a.v.ss + v]) : 0.0f;
    float y = 0.0f;
#pragma unroll 4
    for (int b = 0; b < NH; ++b) {
      if (mine && k0 + b < a.K) {
        g[b] = fmaf(Elem<T>::to_f(k[t * a.k.ss + k0 + b]), val, back ? g[b] : d * g[b]);
        if (OUT) y = fmaf(Elem<T>::to_f(q[t * a.q.ss + k0 + b]), g[b], y);
        if (back) g[b] *= d;
      }
    }
    if (OUT) {
      sh.part[part][r] = y;
      arrive_bar(sh, kSteps);
      wait_bar(sh, kSteps, meetings++ & 1);
      if (part == 0) {
        y = a.so * (sh.part[0][r] + sh.part[1][r]);
        put(t, y);
        if (a.dot) {
          const float z = warp_sum(mine ? y * Elem<T>::to_f(with[t * a.dot_with.ss]) : 0.0f);
          if (lane == 0) dots[m / kCols * 4 + quarter][m % kCols] = z;
        }
      }
      arrive_bar(sh, kSteps);
      wait_bar(sh, kSteps, meetings++ & 1);
    }
  }
  if (OUT)
    for (int m = rows + part; m < kChunk; m += 2) put(t0 + m, 0.0f);
  return meetings;
}

// OUT: the outputs too, with P and the state in NT terms; else only what the
// segment adds to the state.  TMA: tiles are copied by it.
template <typename T, int HPC, int KB, int NT, bool OUT, bool TMA>
__global__ void __launch_bounds__(kThreads, 1) attn_chunk_kernel(const __grid_constant__ ChunkArgs args) {
  static_assert(!TMA || kSplit<T> == 1, "what is split into terms goes through registers");
  const AttnParams& p = args.p;
  using Lay = Layout<T, HPC, NT, OUT>;
  constexpr int kIn = kSplit<T>;
  constexpr int NH = HPC == 2 ? 32 : 32 * KB;  // state elements of a thread
  constexpr int KW = HPC == 2 ? 32 : 32 * KB;  // tensor memory columns of one of the state's terms
  constexpr uint32_t kS = 0, kOi = 64 * HPC, kU = 128 * HPC, kH = kU + 128;
  // the state itself: the sum of its terms where there are three, which hold all of float32's bits; else beside
  // them, or where S would be
  constexpr bool kSum = OUT && NT == 3;
  constexpr uint32_t kF = OUT ? kH + NT * KW : 256;
  static_assert(kF + (kSum ? 0 : 2 * KW) <= 512, "tensor memory");
  constexpr int kHeadSteps = HPC == 2 ? 4 : 4 * KB;  // steps of 16 over a head's elements
  constexpr int kSubs = HPC == 2 ? 2 : KB;
  extern __shared__ unsigned char raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  __shared__ Small sh;
  // of one value for a warp, which is what addresses and descriptors of copies and products are made of
  const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  const int quarter = warp & 3, part = warp >> 2 & 1;
  const int segments = p.plan.segments;
  const Place<HPC> at(p, OUT ? segments : segments - 1);
  const AttnPass& a = p.pass[at.pass];  // by index: it stays in constant memory
  const bool back = a.backward;
  // the segments' order is the pass's; the last one's state is the pass's own
  const int order = at.segment, segment = back ? segments - 1 - order : order;
  const int S = p.S, L = row_length(p.lens, at.n, S);
  const int chunks = (S + kChunk - 1) / kChunk, live = (L + kChunk - 1) / kChunk;
  const int c_begin = segment * p.plan.per, c_end = min(c_begin + p.plan.per, chunks);
  const int c_live = min(c_end, live), count = max(c_live - c_begin, 0);
  auto chunk_at = [&](int i) { return back ? c_live - 1 - i : c_begin + i; };

  if (tid == 0) {
    // who arrives; without outputs the first group scales and the third adds
    for (int i = 0; i < kBars; ++i) {
      int n = i >= kDecay ? HPC : 1;
      if (i < kDone) n = OUT && !TMA ? 3 * kGroupWarps : kGroupWarps;
      else if (i < kPairs) n = OUT ? 2 * kGroupWarps : kGroupWarps;
      else if (i <= kSteps) n = kGroupWarps;
      bar_init(su32(&sh.bars[i]), n);
    }
    sh.gave_up = 0;
    for (int i = 0; i < kFlags; ++i) sh.bad[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // The states that are read at either end are on their way from HBM: a gradient of 6 x 8 x 4 heads of 128 with
  // states 19 us, 35 without this and with single elements of those that lie along the lanes' way.
  if (OUT && (a.first || a.with)) {
    const long long from = ((long long)at.n * p.H + at.h0) * a.K * a.V;
    const int many = min(HPC, p.H - at.h0) * a.K * a.V;
    for (int i = tid * 32; i < many; i += kThreads * 32) {
      if (a.first && segments == 1) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.first + from + i));
      if (a.with && order == segments - 1) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.with + from + i));
    }
  }
  if (TMA && warp == 3 * kGroupWarps + 1 && lane < 5) {
    const CUtensorMap* maps[] = {args.k, args.v, args.q, args.o, args.with};
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(maps[lane] + at.pass)) : "memory");
  }
  if (warp == 3 * kGroupWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sh.tmem)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  next_may_start();
  if (OUT) previous_done();  // the states that segments start from
  // Where U of chunk i is: without outputs there is room for two, and the next is on its way while one is added.
  auto u_at = [](int i) { return OUT ? kU : 128u * (i & 1); };
  struct Phase {
    int bar, n;
  };
  auto ready = [](int i) { return Phase{kTiles + (i & 1), i >> 1}; };
  auto done = [](int i) { return Phase{kDone + (i & 1), i >> 1}; };
  auto paired = [](int i) { return Phase{kPairs + (i & 1), i >> 1}; };
  auto got_u = [](int i) { return Phase{kGotU + (i & 1), i >> 1}; };
  auto got_o = [](int i) { return Phase{kGotO + (i & 1), i >> 1}; };
  auto full = [](int i) { return Phase{kFull + (i & 1), i >> 1}; };
  auto decayed = [](int i) { return Phase{kDecay + i % 3, i / 3}; };
  auto wait = [&](int bar, int n) { wait_bar(sh, bar, n & 1); };
  auto wait_for = [&](Phase x) { wait(x.bar, x.n); };
  auto arrive = [&](int bar) { arrive_bar(sh, bar); };
  auto stage_of = [&](int i) { return (Lay::kStages == 2 ? i & 1 : 0) * Lay::kStage; };
  auto scaled_of = [&](int i) { return Lay::kScaled + (OUT ? 0 : i & 1) * kTerms * kTile; };
  // A chunk's tiles are there with the copies, but for the one whose last rows have to be cleared.
  auto early = [&](int i) { return TMA && L - chunk_at(i) * kChunk >= kChunk; };
  auto mild_of = [&](int i) { return sh.decays[i % 3][0].mild && (HPC == 1 || sh.decays[i % 3][1].mild); };

  // the groups' lanes: a value of a head
  const int r = quarter * 32 + lane;
  const int head = HPC == 2 ? r >> 6 : 0, h = at.h0 + head, v = HPC == 2 ? r & 63 : r;
  const bool mine = v < a.V && h < p.H;
  const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  const int step = back ? -kChunk : kChunk, t_first = chunk_at(0) * kChunk, vec = p.plan.vec;
  const F2 zero = f2(0.0f, 0.0f);
  // The group that has K scales it, and clears rows behind the row's end.
  auto prepare = [&](int i) {
    unsigned char* tiles = sm + stage_of(i);
    if constexpr (TMA) {
      wait_for(full(i));
      const int rows = L - chunk_at(i) * kChunk;
      if (rows < kChunk) {
        const uint4 none = make_uint4(0, 0, 0, 0);
        for (int x = 0; x < 4; ++x) {
          const int piece = tid % kGroup + x % 2 * kGroup, b = x / 2;
          if (piece / 8 < rows) continue;
          unsigned char* to = tiles + b * kSub + piece_at(piece);
          *reinterpret_cast<uint4*>(to + Lay::kV) = none;
          if (b < kSubs) *reinterpret_cast<uint4*>(to + Lay::kK) = none;
          if (OUT && b < kSubs) *reinterpret_cast<uint4*>(to + Lay::kQ) = none;
        }
      }
    }
    wait_for(decayed(i));
    F2 range = zero;
    scale_tile<T, HPC, kSubs>(tiles + Lay::kK, sm + scaled_of(i), sh.decays[i % 3], range);
    if (!in_range(range)) sh.bad[i % kFlags] = 1;
  };

  if (warp < kGroupWarps) {
    // ---------------- pairs
    if constexpr (!OUT) {
      // without outputs: K of the next chunk, while the third group adds
      Rows<T, HPC> rv(a.v, at.n, at.h0, p.H, a.v_of, a.V, t_first, step);
      Rows<T, HPC> rk(a.k, at.n, at.h0, p.H, a.k_of, a.K, t_first, step);
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        if (!TMA && i >= Lay::kStages) wait_for(got_u(i - Lay::kStages));  // whose tiles these take
        else if (i >= 2) wait_for(got_u(i - 2));                          // whose ck K this takes
        if (!TMA) {
          rk.template load<kSubs>(sm + stage_of(i) + Lay::kK, L - chunk_at(i) * kChunk, vec);
          rv.template load<2>(sm + stage_of(i) + Lay::kV, L - chunk_at(i) * kChunk, vec);
          if (i + 1 < count) {
            const int rows = L - chunk_at(i + 1) * kChunk;
            rk.prefetch(rows), rv.prefetch(rows);
          }
        }
        prepare(i);
        if (!tile_in_range<kGroup, kTile>(sm + stage_of(i) + Lay::kV, tid)) sh.bad[i % kFlags] = 1;
        arrive(ready(i).bar);
      }
    } else {
      const int ocol = (HPC == 2 ? head * 64 : 0) + part * kCols;  // columns of S and O
      // The loops below go by 8 columns and are not unrolled: what runs between
      // two of a chunk's barriers has to stay in the instruction cache.
      // P of row m of S, 32 of its columns
      auto pairs = [&](int i) {
        const int m = r & 63;
        const Decays& d = sh.decays[i % 3][head];
        const bool mild = mild_of(i);
        const float hi = d.hi[m], lo = d.lo[m];
        F2 range = zero;
        unsigned char* row = (Lay::kOver ? sm + Lay::kK : sm + Lay::kP) + (HPC == 2 ? r : m) * 128;
        float next[8];
        tmem_ld(lanes + kS + ocol, next);
#pragma unroll 1
        for (int c = 0; c < kCols; c += 8) {
          const int n0 = part * kCols + c;
          float s[8];
          tmem_ld_done(next);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = next[j];
          if (c + 8 < kCols) tmem_ld(lanes + kS + ocol + c + 8, next);
          F2 x[4];
          if (mild) {
            const float4 f = *reinterpret_cast<const float4*>(&d.bn[n0]), g = *reinterpret_cast<const float4*>(&d.bn[n0 + 4]);
            x[0] = mul2(f2(s[0], s[1]), f2(f.x, f.y)), x[1] = mul2(f2(s[2], s[3]), f2(f.z, f.w));
            x[2] = mul2(f2(s[4], s[5]), f2(g.x, g.y)), x[3] = mul2(f2(s[6], s[7]), f2(g.z, g.w));
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] *= a.su * exp2_fast((hi - d.hi[n0 + j]) + (lo - d.lo[n0 + j]));
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = f2(s[2 * j], s[2 * j + 1]);
          }
          uint32_t w[NT][4];
          const int last = back ? n0 + 7 - m : m - n0;  // of the columns, counted from the first or backward
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float2 y = f2_get(x[j / 2]);
            y.x = (back ? 7 - j : j) <= last ? y.x : 0.0f;
            y.y = (back ? 6 - j : j + 1) <= last ? y.y : 0.0f;
            uint32_t t[NT];
            split<NT>(f2(y.x, y.y), t, range);
#pragma unroll
            for (int e = 0; e < NT; ++e) w[e][j / 2] = t[e];
          }
          unsigned char* to = row + (((n0 / 8) ^ (m & 7)) << 4);
#pragma unroll
          for (int e = 0; e < NT; ++e) *reinterpret_cast<uint4*>(to + e * Lay::kPTerm) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
        }
        if (!in_range(range)) sh.bad[i % kFlags] = 1;
      };
      Rows<T, HPC> rq(a.q, at.n, at.h0, p.H, a.q_of, a.K, t_first, step);
      auto fetch = [&](int i) {
        rq.template load<kSubs>(sm + stage_of(i) + Lay::kQ, L - chunk_at(i) * kChunk, vec);
        arrive(ready(i).bar);
      };
      if (!TMA)
        for (int i = 0; i < min(count, Lay::kStages); ++i) fetch(i);
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        if (!TMA && i + Lay::kStages < count) rq.prefetch(L - chunk_at(i + Lay::kStages) * kChunk);
        wait_for(decayed(i));
        // while S is on its way, and the product that P was written for: Q and V are looked over, with one head by the
        // two quarters of the lanes that S has no rows for
        if (HPC == 2 || quarter >= 2) {
          constexpr int kLook = HPC == 2 ? kGroup : kGroup / 2;
          const int thread = HPC == 2 ? tid : (part * 2 + (quarter & 1)) * 32 + lane;
          if (early(i)) wait_for(full(i));
          else wait_for(ready(i));
          bool fine = tile_in_range<kLook, kTile>(sm + stage_of(i) + Lay::kV, thread);
          // Half goes up to 2^16, and what is infinite makes P so
          if constexpr (!std::is_same_v<T, __half>)
            fine = tile_in_range<kLook, kSubs * kSub>(sm + stage_of(i) + Lay::kQ, thread) && fine;
          if (!fine) sh.bad[i % kFlags] = 1;
        }
        wait(kGotS, i);
        if (i > 0) wait_for(got_o(i - 1));  // which P was multiplied for
        if (HPC == 2 || quarter < 2) pairs(i);
        arrive(paired(i).bar);
        if (!TMA && i + Lay::kStages < count) {
          wait(kGotOi, i);
          fetch(i + Lay::kStages);
        }
      }
    }
  } else if (warp < 2 * kGroupWarps) {
    // ---------------- outputs
    if constexpr (OUT) {
      const int ocol = (HPC == 2 ? head * 64 : 0) + part * kCols;  // columns of S and O
      const int thread = tid - kGroup;
      // outputs of lane v
      T* out = static_cast<T*>(a.o.p) + at.n * a.o.ns + (long long)(h / a.o_of) * a.V + v;
      float* out32 = a.o32 + ((long long)at.n * S * p.H + h) * a.V + v;
      const long long ss32 = (long long)p.H * a.V;
      const T* dot_row = static_cast<const T*>(a.dot_with.p) + at.n * a.dot_with.ns + (long long)(h / a.o_of) * a.V + v;
      // The products of chunk i's outputs, added up over the lanes' warps.
      auto dots_out = [&](int i) {
        if (thread < 64 * HPC) {
          const int hd = thread / 64, m = thread % 64, t = chunk_at(i) * kChunk + m;
          if (t < L && at.h0 + hd < p.H) {
            const float* x = &sh.dots[i & 1][m / kCols * 4][m % kCols];
            const float y = HPC == 2 ? x[2 * hd * kCols] + x[(2 * hd + 1) * kCols]
                                     : (x[0] + x[kCols]) + (x[2 * kCols] + x[3 * kCols]);
            a.dot[((long long)at.n * p.H + at.h0 + hd) * S + t] = y;
          }
        }
      };
      auto outputs = [&](int i) {
        const Decays* dec = sh.decays[i % 3];
        const bool mild = mild_of(i), dot = a.dot, wide = a.o32, any = a.o.p;
        const int t0 = chunk_at(i) * kChunk + part * kCols;
        float next[8];
        tmem_ld(lanes + kOi + ocol, next);
#pragma unroll 1
        for (int c = 0; c < kCols; c += 8) {
          float o[8], near[8];
          tmem_ld_done(next);
#pragma unroll
          for (int x = 0; x < 8; ++x) o[x] = next[x];
          if (c + 8 < kCols) tmem_ld(lanes + kOi + ocol + c + 8, next);
          if (!mild) tmem_ld(lanes + kS + ocol + c, near);
          const float* cq = &dec[head].cq[part * kCols + c];
#pragma unroll
          for (int x = 0; x < 8; x += 4) {
            const float4 f = *reinterpret_cast<const float4*>(cq + x);
            const float2 y = f2_get(mul2(f2(f.x, f.y), f2(o[x], o[x + 1]))), z = f2_get(mul2(f2(f.z, f.w), f2(o[x + 2], o[x + 3])));
            o[x] = y.x, o[x + 1] = y.y, o[x + 2] = z.x, o[x + 3] = z.y;
          }
          if (!mild) {
            tmem_ld_done(near);
            asm volatile("" ::: "memory");
#pragma unroll
            for (int x = 0; x < 8; ++x) o[x] = fmaf(a.so, near[x], o[x]);
          }
          const int t1 = t0 + c, rows = mine ? S - t1 : 0;
          // a lane's element of 8 rows of the tile, where tiles are copied; it is unused where o32 is written
          const int at_tile = (r >> 6) * (int)kSub / (int)sizeof(T) + (part * kCols + c) * 64 + (r & 63);
          if (TMA && !wide) {
            T* to = reinterpret_cast<T*>(sm + Lay::kOut) + at_tile;
#pragma unroll
            for (int x = 0; x < 8; ++x) to[x * 64] = Elem<T>::from_f(o[x]);
          } else if (wide) {
            float* to = out32 + t1 * ss32;
#pragma unroll
            for (int x = 0; x < 8; ++x, to += ss32)
              if (x < rows) *to = o[x];
          } else if (!TMA && any) {
            T* to = out + t1 * a.o.ss;
#pragma unroll
            for (int x = 0; x < 8; ++x, to += a.o.ss)
              if (x < rows) *to = Elem<T>::from_f(o[x]);
          }
          if (dot) {
            const int live_rows = mine ? L - t1 : 0;
            if constexpr (TMA) {
              const T* from = reinterpret_cast<const T*>(sm + (Lay::kWithApart ? Lay::kAfterOut : stage_of(i) + Lay::kK)) + at_tile;
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float w = Elem<T>::to_f(from[x * 64]);
                o[x] = x < live_rows ? o[x] * w : 0.0f;
              }
            } else {
              const T* with = dot_row + t1 * a.dot_with.ss;
#pragma unroll
              for (int x = 0; x < 8; ++x, with += a.dot_with.ss) o[x] = x < live_rows ? o[x] * Elem<T>::to_f(*with) : 0.0f;
            }
            int to = 0;
            lanes_sum<8, 16, 1>(o, lane, to);
            sh.dots[i & 1][warp - kGroupWarps][c + to] = o[0];
          }
        }
      };
      Rows<T, HPC> rv(a.v, at.n, at.h0, p.H, a.v_of, a.V, t_first, step);
      auto fetch = [&](int i) {
        rv.template load<2>(sm + stage_of(i) + Lay::kV, L - chunk_at(i) * kChunk, vec);
        arrive(ready(i).bar);
      };
      if (!TMA)
        for (int i = 0; i < min(count, Lay::kStages); ++i) fetch(i);
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        if (!TMA && i + Lay::kStages < count) rv.prefetch(L - chunk_at(i + Lay::kStages) * kChunk);
        wait_for(decayed(i));
        wait_for(paired(i));  // all of the chunk's flags are set
        if (a.dot && i > 0) {
          wait_for(done(i - 1));
          dots_out(i - 1);
        }
        wait_for(got_o(i));
        if (!TMA && i + Lay::kStages < count) fetch(i + Lay::kStages);
        // the chunk before is on its way out of the tile, this one's factors are there; also where neither is used,
        // as a barrier's phases have to be waited for one by one
        if (TMA && i > 0) wait(kStored, i - 1);
        if (TMA && a.dot) wait(kWith, i);
        if (!sh.bad[i % kFlags]) outputs(i);
        arrive(done(i).bar);
      }
      if (a.dot && count > 0) {
        wait_for(done(count - 1));
        if (!sh.gave_up) dots_out(count - 1);
      }
      // the rows behind the last live chunk
      for (int t = max(c_live, c_begin) * kChunk + part; t < min(c_end * kChunk, S); t += 2) {
        if (!mine) break;
        if (a.o32) out32[t * ss32] = 0.0f;
        else if (a.o.p) out[t * a.o.ss] = Elem<T>::from_f(0.0f);
      }
    }
  } else if (warp < 3 * kGroupWarps) {
    // ---------------- the state
    const int k0 = part * NH, ucol = HPC == 2 ? head * 64 + part * 32 : part * NH;  // state elements, U's columns
    // the state, transposed: lane v, elements k0 ..
    const long long state = ((long long)at.n * p.H + h) * a.K * a.V + (a.v_major ? (long long)v * a.K + k0 : (long long)k0 * a.V + v);
    const int apart = a.v_major ? 1 : a.V;            // of two of a thread's elements
    const int elements = mine ? min(NH, a.K - k0) : 0;  // that there are
    constexpr long long kept = (long long)KB * 64 * 128;  // a state in scratch: [k][lane]
    Rows<T, HPC> rk(a.k, at.n, at.h0, p.H, a.k_of, a.K, t_first, step);
    auto fetch = [&](int i) { rk.template load<kSubs>(sm + stage_of(i) + Lay::kK, L - chunk_at(i) * kChunk, vec); };
    // The state lives in tensor memory.  Elements j .. j + 15 of it, from there:
    auto read_state = [&](int j, F2 (&H)[8]) {
      if constexpr (kSum) {
        float t[NT][8];
#pragma unroll
        for (int x = 0; x < NT; ++x) tmem_ld(lanes + kH + x * KW + (k0 + j) / 2, t[x]);
#pragma unroll
        for (int x = 0; x < NT; ++x) tmem_ld_done(t[x]);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          H[x] = pair_of(__float_as_uint(t[NT - 1][x]));
#pragma unroll
          for (int y = NT - 2; y >= 0; --y) H[x] = add2(H[x], pair_of(__float_as_uint(t[y][x])));
        }
      } else {
        float t[16];
        tmem_ld(lanes + kF + k0 + j, t);
        tmem_ld_done(t);
#pragma unroll
        for (int x = 0; x < 8; ++x) H[x] = f2(t[2 * x], t[2 * x + 1]);
      }
    };
    // Elements j .. j + 15 to there, for chunk i.
    auto write_state = [&](int j, const F2 (&H)[8], F2& range) {
      if constexpr (OUT) {
        uint32_t w[NT][8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          uint32_t s[NT];
          split<NT>(H[x], s, range);
#pragma unroll
          for (int y = 0; y < NT; ++y) w[y][x] = s[y];
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) tmem_st<8>(lanes + kH + x * KW + (k0 + j) / 2, w[x]);
      }
      if constexpr (!kSum) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float2 y = f2_get(H[x]);
          w[2 * x] = __float_as_uint(y.x), w[2 * x + 1] = __float_as_uint(y.y);
        }
        tmem_st<16>(lanes + kF + k0 + j, w);
      }
    };
    auto wrote = [&](F2 range, int i) {
      tmem_st_done();
      if (OUT && mine && !in_range(range)) sh.bad[i % kFlags] = 1;
    };
    // Elements j .. j + 15 of the `there` that there are of a state, `far` apart; side by side in pieces of four.
    auto read16 = [&](const float* from, int j, int far, int there, float (&y)[16]) {
      if (far == 1 && a.K % 4 == 0 && reinterpret_cast<uintptr_t>(from) % 16 == 0) {
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (j + x < there) f = *reinterpret_cast<const float4*>(from + j + x);
          y[x] = f.x, y[x + 1] = f.y, y[x + 2] = f.z, y[x + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int x = 0; x < 16; ++x) y[x] = j + x < there ? from[(j + x) * far] : 0.0f;
      }
    };
    // The state before the first chunk.
    auto begin_state = [&]() {
      const bool pieces = OUT && segments > 1;
      const float* from = pieces ? p.plan.states + ((long long)at.stream * segments + order) * kept + k0 * 128 + r : a.first + state;
      const int far = pieces ? 128 : apart, there = pieces ? NH : OUT && a.first ? elements : 0;
      F2 range = zero;
#pragma unroll 1
      for (int j = 0; j < NH; j += 16) {
        float y[16];
        read16(from, j, far, there, y);
        F2 H[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) H[x] = f2(y[2 * x], y[2 * x + 1]);
        write_state(j, H, range);
      }
      wrote(range, 0);
    };
    // H = e H + U for chunk i, and its terms for the next.
    auto advance = [&](int i) {
      const float e = sh.decays[i % 3][head].total;
      F2 range = zero;
#pragma unroll 1
      for (int j = 0; j < NH; j += 16) {
        float u[16];
        tmem_ld(lanes + u_at(i) + ucol + j, u);
        F2 H[8];
        read_state(j, H);
        tmem_ld_done(u);
#pragma unroll
        for (int x = 0; x < 8; ++x) H[x] = fma2(f2(e, e), H[x], f2(u[2 * x], u[2 * x + 1]));
        write_state(j, H, range);
      }
      wrote(range, i + 1);
    };
    // An element of the state on its own, infinities too: where it is not finite its first term alone has it.
    auto one_state = [&](int j, float (&y)[16]) {
      F2 H[8];
      read_state(j, H);
      float first[8];
      if constexpr (kSum) {
        tmem_ld(lanes + kH + (k0 + j) / 2, first);
        tmem_ld_done(first);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        float2 z = f2_get(H[x]);
        if constexpr (kSum) {
          const float2 t = f2_get(pair_of(__float_as_uint(first[x])));
          if (!(t.x - t.x == 0.0f)) z.x = t.x;
          if (!(t.y - t.y == 0.0f)) z.y = t.y;
        }
        y[2 * x] = z.x, y[2 * x + 1] = z.y;
      }
    };
    // The state at the start of chunk c, where the decays' gradient wants it.
    auto mark = [&](int c) {
      const int every = p.plan.every;
      if (NT != kTerms || !a.marks || c == 0 || (every > 1 && c % every != 0)) return;  // gradients have all terms
      float* to = a.marks + ((long long)(at.stream - at.pass * p.N * ((p.H + HPC - 1) / HPC)) * p.plan.marks + c / every - 1) * kept;
#pragma unroll 1
      for (int j = 0; j < NH; j += 16) {
        float y[16];
        one_state(j, y);
#pragma unroll
        for (int x = 0; x < 16; ++x) to[(k0 + j + x) * 128 + r] = j + x < elements ? y[x] : 0.0f;
      }
    };
    int meetings = 0;
    // Chunk i step by step, from the operands themselves.
    auto by_step = [&](int i) {
      float g[NH];
#pragma unroll 1
      for (int j = 0; j < NH; j += 16) {
        float y[16];
        one_state(j, y);
#pragma unroll
        for (int x = 0; x < 16; ++x) g[j + x] = y[x];
      }
      meetings = run_steps<T, HPC, NH, OUT>(args.p, at.pass, at.n, at.h0, chunk_at(i) * kChunk, L, sh.dots[i & 1], sh, meetings, g);
      F2 range = zero;
#pragma unroll 1
      for (int j = 0; j < NH; j += 16) {
        F2 H[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) H[x] = f2(g[j + 2 * x], g[j + 2 * x + 1]);
        write_state(j, H, range);
      }
      wrote(range, i + 1);
    };
    if constexpr (OUT) {
      if (!TMA && count > 0) fetch(0);
      begin_state();
      if (count > 0) {
        prepare(0);
        arrive(ready(0).bar);
        if (!back) mark(c_begin);
        if (!TMA && Lay::kStages == 2 && count > 1) fetch(1);
      }
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        const bool more = i + 1 < count;
        if (Lay::kStages == 1 && more) rk.prefetch(L - chunk_at(i + 1) * kChunk);
        wait_for(got_u(i));
        // ck K of the next chunk takes the place of this one's, and K where there is room
        if (more && Lay::kStages == 2) prepare(i + 1);
        wait_for(paired(i));  // all of the chunk's flags are set
        wait(kGotOi, i);
        if (more) wait_for(decayed(i + 1));
        if (__builtin_expect(!sh.bad[i % kFlags], 1)) advance(i);
        else by_step(i);
        arrive(done(i).bar);
        if (more) {
          if (Lay::kStages == 1) {  // K's place is free once P, which may be there, has been multiplied
            if (Lay::kOver) wait_for(got_o(i));
            fetch(i + 1);
            prepare(i + 1);
          }
          arrive(ready(i + 1).bar);
          if (!TMA && Lay::kStages == 2 && i + 2 < count) fetch(i + 2);
        }
        if (back || more) mark(back ? chunk_at(i) : chunk_at(i + 1));
      }
      if (order == segments - 1 && (a.last || a.with)) {
        float with = 0.0f;
#pragma unroll 1
        for (int j = 0; j < NH; j += 16) {
          float y[16];
          one_state(j, y);
          if (a.last) {  // of passes that have the state's rows along their values only
#pragma unroll
            for (int x = 0; x < 16; ++x)
              if (j + x < elements) a.last[state + (j + x) * apart] = y[x];
          }
          if (a.with) {
            float z[16];
            read16(a.with + state, j, apart, elements, z);
#pragma unroll
            for (int x = 0; x < 16; ++x)
              if (j + x < elements) with = fmaf(z[x], y[x], with);
          }
        }
        with = warp_sum(with);
        if (lane == 0) sh.part[0][warp % kGroupWarps] = with;
      }
    } else {
      long long left = 0;  // logarithm of the segment's decay
      begin_state();
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        wait_for(got_u(i));
        if (__builtin_expect(!sh.bad[i % kFlags], 1)) advance(i);
        else by_step(i);
        // what has left nothing leaves nothing, what has passed float32's range stays beyond it
        if (left > -kAll && left < kAll) left += sh.decays[i % 3][head].log2;
        arrive(done(i).bar);
      }
      float* to = p.plan.states + ((long long)at.stream * segments + order) * kept;
#pragma unroll 1
      for (int j = 0; j < NH; j += 16) {
        float y[16];
        one_state(j, y);
#pragma unroll
        for (int x = 0; x < 16; ++x) to[(k0 + j + x) * 128 + r] = j + x < elements ? y[x] : 0.0f;
      }
      if (part == 0 && lane == 0 && (HPC == 2 ? quarter % 2 == 0 : quarter == 0)) {
        // as whole part and fraction
        const long long x = min(max(left, -kAll), kAll);
        float* to2 = p.plan.left + (((long long)at.stream * segments + order) * 2 + head) * 2;
        to2[0] = (float)(int)(x >> 32), to2[1] = (float)((uint32_t)x >> 8) * 5.9604644775390625e-8f;
      }
    }
  } else {
    if (warp == 3 * kGroupWarps) {
      // ---------------- products
      const bool leader = elect();
      auto pairs_of = [&](int i) {  // S
        const uint32_t tiles = su32(sm) + stage_of(i);
        const uint64_t dq = smem_desc_sw128(tiles + Lay::kQ), dk = smem_desc_sw128(tiles + Lay::kK);
        if (leader) {
          products<kIn, kIn, NT, kHeadSteps>([&](int x, int y, int s, uint32_t more) {
            const uint32_t o = ((s / 4) * kSub + (s % 4) * 32) >> 4;
            tc_mma(tmem + kS, dq + (x * kTile >> 4) + o, dk + (y * kTile >> 4) + o, idesc_of(64 * HPC), more);
          });
          tc_commit(su32(&sh.bars[kGotS]));
        }
        __syncwarp();
      };
      if (OUT && count > 0 && early(0)) {
        wait_for(full(0));
        pairs_of(0);
      }
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        const uint32_t tiles = su32(sm) + stage_of(i);
        const uint64_t dv = desc_mn(tiles + Lay::kV), ds = desc_mn(su32(sm) + scaled_of(i));
        wait_for(ready(i));
        if (!OUT && i >= 2) wait_for(done(i - 2));  // whose U is where this one's goes
        if (OUT && !early(i)) {
          if (i > 0) wait_for(done(i - 1));  // whose outputs may be where S goes
          pairs_of(i);
        }
        if (leader) {
          const uint32_t du = tmem + u_at(i);
          products<kIn, kTerms, kTerms, 4>([&](int x, int y, int s, uint32_t more) {
            tc_mma(du, dv + ((x * kTile + s * 2048) >> 4), ds + ((y * kTile + s * 2048) >> 4),
                   idesc_of(HPC == 2 ? 128 : 64 * KB) | kRowsA | kRowsB, more);
          });
          tc_commit(su32(&sh.bars[got_u(i).bar]));
        }
        __syncwarp();
        if (!OUT) continue;
        if (i > 0) wait_for(done(i - 1));
        const uint64_t dq = smem_desc_sw128(tiles + Lay::kQ);
        auto oi = [&](int x, int y, int s, uint32_t more) {
          tc_mma_ts(tmem + kOi, tmem + kH + x * KW + s * 8, dq + ((y * kTile + (s / 4) * kSub + (s % 4) * 32) >> 4),
                    idesc_of(64 * HPC), more);
        };
        // The tensor cores' sums are cut off, not rounded: each product that is added to a sum takes something of it,
        // always towards zero.  Where float32 comes of it the small products of both Oi and O come first, then the
        // large ones: without decays float32 outputs are off by 2e-7 of their size so, by 6e-7 with all of O behind
        // Oi, for a fiftieth of a gradient's time.
        if (leader) {
          if constexpr (kSum) {
            products<NT, kIn, NT, kHeadSteps, 1>(oi);
          } else {
            products<NT, kIn, NT, kHeadSteps>(oi);
            tc_commit(su32(&sh.bars[kGotOi]));
          }
        }
        __syncwarp();
        const bool apart = !mild_of(i);  // its outputs go where S is
        wait_for(paired(i));
        const uint64_t dp = smem_desc_sw128(Lay::kOver ? tiles + Lay::kK : su32(sm) + Lay::kP);
        const uint32_t to = tmem + (apart ? kS : kOi);
        if (leader) {
          const bool good = !sh.bad[i % kFlags];
          auto o = [&](int x, int y, int s, uint32_t more) {
            tc_mma(to, dv + ((x * kTile + s * 2048) >> 4), dp + ((y * Lay::kPTerm + s * 32) >> 4), idesc_of(64 * HPC) | kRowsA,
                   apart ? more : 1u);
          };
          if constexpr (kSum) {
            if (good) {
              products<kIn, NT, NT, 4, 1>(o);
              products<NT, kIn, NT, kHeadSteps, 0, 0>(oi, 1);
            }
            tc_commit(su32(&sh.bars[kGotOi]));
            if (good) products<kIn, NT, NT, 4, 0, 0>(o, 1);
          } else if (good) {
            products<kIn, NT, NT, 4>(o);
          }
          tc_commit(su32(&sh.bars[got_o(i).bar]));
        }
        __syncwarp();
        if (i + 1 < count && early(i + 1)) {
          if (apart) wait_for(done(i));
          wait_for(full(i + 1));
          pairs_of(i + 1);
        }
      }
      if (count > 0) {  // all of them complete before tensor memory is given back
        wait_for(got_u(count - 1));
        if (OUT) wait_for(got_o(count - 1));
      }
    } else if (warp == 3 * kGroupWarps + 1) {
      // ---------------- copies
      if constexpr (TMA) {
        const int z = at.pass;
        const bool leader = elect();
        // sub-tile b of an operand whose heads `of` heads share
        auto head_of = [&](int b, int of) { return HPC == 2 ? (at.h0 + b) / of : at.h0 / of; };
        auto load = [&](int i) {
          const uint32_t tiles = su32(sm) + stage_of(i), bar = su32(&sh.bars[full(i).bar]);
          const int t = chunk_at(i) * kChunk;
          if (leader) {
            bar_expect(bar, (2 + kSubs * (OUT ? 2 : 1)) * kSub);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int x = HPC == 2 ? 0 : 64 * b;
              if (b < kSubs) copy_in(tiles + Lay::kK + b * kSub, &args.k[z], x, head_of(b, a.k_of), t, at.n, bar);
              if (OUT && b < kSubs) copy_in(tiles + Lay::kQ + b * kSub, &args.q[z], x, head_of(b, a.q_of), t, at.n, bar);
              copy_in(tiles + Lay::kV + b * kSub, &args.v[z], x, head_of(b, a.v_of), t, at.n, bar);
            }
          }
          __syncwarp();
        };
        for (int i = 0; i < min(count, 2); ++i) load(i);
        const bool out = OUT && a.o.p && !a.o32;
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
          const int t = chunk_at(i) * kChunk;
          if (OUT && a.dot && !sh.gave_up) {
            if (Lay::kWithApart) {
              if (i > 0) wait_for(done(i - 1));
            } else {  // takes the place of K, which S and ck K have been made from
              wait_for(paired(i));
              wait_for(ready(i));
            }
            if (leader) {
              const uint32_t bar = su32(&sh.bars[kWith]), to = su32(sm) + (Lay::kWithApart ? Lay::kAfterOut : stage_of(i) + Lay::kK);
              bar_expect(bar, 2 * kSub);
#pragma unroll
              for (int b = 0; b < 2; ++b)
                copy_in(to + b * kSub, &args.with[z], HPC == 2 ? 0 : 64 * b, head_of(b, a.o_of), t, at.n, bar);
            }
            __syncwarp();
          }
          // the stage is free with the last product of the chunk, or once the outputs have been multiplied
          const bool early = OUT && (Lay::kWithApart || !a.dot);
          if (early) {
            wait_for(got_o(i));
            if (i + 2 < count && !sh.gave_up) load(i + 2);
          }
          wait_for(done(i));
          if (OUT && a.dot) wait(kWith, i);  // also where nobody has read it
          const bool good = !sh.bad[i % kFlags] && !sh.gave_up;
          if (!early && i + 2 < count && !sh.gave_up) load(i + 2);
          if (OUT && leader) {
            if (out && good) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
                if (HPC == 1 ? 64 * b < a.V : at.h0 + b < p.H)
                  copy_out(&args.o[z], HPC == 2 ? 0 : 64 * b, head_of(b, a.o_of), t, at.n, su32(sm) + Lay::kOut + b * kSub);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            bar_arrive(su32(&sh.bars[kStored]));
          }
          __syncwarp();
        }
        if (leader) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
      }
    } else {
      // ---------------- decays: a warp for each head
      const int x = warp - (3 * kGroupWarps + 2), hx = min(at.h0 + x, p.H - 1), end = at.h0 + x < p.H ? L : 0;
      if (x < HPC) {
        const float* g = static_cast<const float*>(p.decay.p) + at.n * p.decay.ns + hx;
        const float bias = p.bias ? p.bias[hx] : 0.0f;
        auto read = [&](int i, int j) {
          const int t = chunk_at(i) * kChunk + 2 * lane + j;
          return t < end ? (p.decay.p ? g[t * p.decay.ss] : 0.0f) + bias : 0.0f;
        };
        float x0 = 0.0f, x1 = 0.0f;
        if (count > 0) x0 = read(0, 0), x1 = read(0, 1);
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
          if (i >= 3) wait_for(done(i - 3));  // whose place these take
          const float y0 = x0, y1 = x1;
          if (i + 1 < count) x0 = read(i + 1, 0), x1 = read(i + 1, 1);
          const bool bad = chunk_decays(a, y0, y1, sh.decays[i % 3][x]);
          if (lane == 0) {
            if (x == 0) sh.bad[(i + kClear) % kFlags] = 0;
            if (bad) sh.bad[i % kFlags] = 1;
          }
          __syncwarp();
          if (lane == 0) bar_arrive(su32(&sh.bars[decayed(i).bar]));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (OUT && a.cross && order == segments - 1 && tid < HPC && at.h0 + tid < p.H) {
    const float* x = sh.part[0];
    float y = 0.0f;
    for (int w = 0; w < kGroupWarps; ++w)
      if (HPC == 1 || (w & 3) >> 1 == tid) y += x[w];
    a.cross[(long long)at.n * p.H + at.h0 + tid] = y;
  }
  // nothing is in flight any more, unless a wait has failed: then what was issued gets some time
  if (sh.gave_up && warp == 3 * kGroupWarps) {
    const unsigned long long begin = gtime();
    while (gtime() - begin < 500000000ull) {
    }
  }
  if (warp == 3 * kGroupWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// The states that a stream's segments start from, from what each adds: in the
// pass's order, four elements of a thread at a time (5.7 us for 16 states of 128 x
// 128 in eight segments, 13 us element by element; both are round trips).
constexpr int kJoin = 4 * 256;  // elements of a block
template <int HPC, int KB>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kept = KB * 64 * 128;
  next_may_start();
  previous_done();
  const int element = blockIdx.y * kJoin + threadIdx.x * 4;
  const int k = element / 128, r = element % 128, head = HPC == 2 ? r >> 6 : 0;
  long long id = blockIdx.x;
  const int groups = (p.H + HPC - 1) / HPC;
  const int h = (int)(id % groups) * HPC + head, v = HPC == 2 ? r & 63 : r;
  const int n = (int)(id / groups % p.N);
  const AttnPass& a = p.pass[id / groups / p.N];
  float run[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (h < p.H && k < a.K && a.first) {
    const float* from = a.first + ((long long)n * p.H + h) * a.K * a.V;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (v + e < a.V) run[e] = from[a.v_major ? (long long)(v + e) * a.K + k : (long long)k * a.V + v + e];
  }
  float4* s = reinterpret_cast<float4*>(p.plan.states + id * p.plan.segments * kept + element);
  const float* f = p.plan.left + (id * p.plan.segments * 2 + head) * 2;
  constexpr int kBatch = 8;  // read before any of it is written: on their way together
#pragma unroll 1
  for (int i0 = 0; i0 < p.plan.segments; i0 += kBatch) {
    float4 add[kBatch];
    float2 left[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j;
      if (i + 1 < p.plan.segments)
        add[j] = s[(long long)i * (kept / 4)], left[j] = *reinterpret_cast<const float2*>(f + 4 * i);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j;
      if (i >= p.plan.segments) break;
      s[(long long)i * (kept / 4)] = make_float4(run[0], run[1], run[2], run[3]);
      if (i + 1 >= p.plan.segments) break;
      // 2^left run, which may be a float32 where the power alone is none
      const int whole = (int)left[j].x;
      const float part = exp2_fast(left[j].y), x[4] = {add[j].x, add[j].y, add[j].z, add[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) run[e] = fmaf(ldexpf(run[e], whole), part, x[e]);
    }
  }
}

// operand: swizzled for the products; else plain, for the workers' lanes.
// Rows as a tensor of (elements, heads, steps, batch rows); heads: those that rows have.
inline bool make_map(CUtensorMap* map, const RowsArg& a, int size, int heads, int S, int N, bool operand = true) {
  static const auto encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (encode == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)size, (cuuint64_t)heads, (cuuint64_t)S, (cuuint64_t)N};
  // a distance that nothing is away has to be one all the same
  const cuuint64_t strides[3] = {(cuuint64_t)size * 2, (cuuint64_t)(S > 1 ? a.ss * 2 : 16), (cuuint64_t)(N > 1 ? a.ns * 2 : 16)};
  const cuuint32_t box[4] = {64, 1, kChunk, 1}, each[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.p, dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                operand ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The maps of all passes, where every operand takes them.
inline bool make_maps(ChunkArgs& args) {
  const AttnParams& p = args.p;
  for (int i = 0; i < p.passes; ++i) {
    const AttnPass& a = p.pass[i];
    if (!a.q.vec || !a.k.vec || !a.v.vec || (a.o.p && !a.o32 && !a.o.vec) || (a.dot && !a.dot_with.vec)) return false;
  }
  for (int i = 0; i < p.passes; ++i) {
    const AttnPass& a = p.pass[i];
    if (!make_map(&args.q[i], a.q, a.K, p.H / a.q_of, p.S, p.N) || !make_map(&args.k[i], a.k, a.K, p.H / a.k_of, p.S, p.N) ||
        !make_map(&args.v[i], a.v, a.V, p.H / a.v_of, p.S, p.N) ||
        (a.o.p && !a.o32 && !make_map(&args.o[i], a.o, a.V, p.H / a.o_of, p.S, p.N, false)) ||
        (a.dot && !make_map(&args.with[i], a.dot_with, a.V, p.H / a.o_of, p.S, p.N, false)))
      return false;
  }
  return true;
}

template <typename T, int HPC, int KB, int NT, bool TMA>
cudaError_t launch_chunks_of(const ChunkArgs& args, cudaStream_t s, int* launches) {
  const AttnParams& p = args.p;
  constexpr size_t smem = Layout<T, HPC, NT, true>::kBytes;
  const long long streams = (long long)p.passes * p.N * ((p.H + HPC - 1) / HPC);
  auto whole = attn_chunk_kernel<T, HPC, KB, NT, true, TMA>;
  cudaError_t e = cudaFuncSetAttribute(whole, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (p.plan.segments > 1) {
    auto sums = attn_chunk_kernel<T, HPC, KB, kTerms, false, TMA>;
    constexpr size_t sums_smem = Layout<T, HPC, kTerms, false>::kBytes;
    e = cudaFuncSetAttribute(sums, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sums_smem);
    if (e != cudaSuccess) return e;
    sums<<<(unsigned)(streams * (p.plan.segments - 1)), kThreads, sums_smem, s>>>(args);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ++*launches;
    e = launch_chained(attn_join_kernel<HPC, KB>, dim3((unsigned)streams, KB * 64 * 128 / kJoin), 256, 0, s, p);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  if (p.plan.segments > 1) {
    e = launch_chained(whole, (unsigned)(streams * p.plan.segments), kThreads, smem, s, args);
  } else {
    whole<<<(unsigned)streams, kThreads, smem, s>>>(args);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <typename T, int NT, bool TMA>
cudaError_t launch_chunks_in(const ChunkArgs& args, cudaStream_t s, int* launches) {
  // every pass has the same two sizes, in one order or the other
  const AttnParams& p = args.p;
  if (p.pass[0].K <= 64 && p.pass[0].V <= 64) return launch_chunks_of<T, 2, 1, NT, TMA>(args, s, launches);
  // 16-bit rows have all terms in gradients alone, whose states are as deep as the larger size
  if constexpr (NT != kTerms || kSplit<T> == kTerms)
    if (p.plan.deep == 64) return launch_chunks_of<T, 1, 1, NT, TMA>(args, s, launches);
  return launch_chunks_of<T, 1, 2, NT, TMA>(args, s, launches);
}

// P and the state as three terms where float32 comes of them: for float32
// rows, and in gradients, whose products for the decays are added up over the
// sequence.  Where 16-bit outputs alone do, two: off by 2^-17 of what they are,
// while the rows that they come of are rounded to 2^-9 or 2^-12 of theirs.  An
// output that is far smaller than its terms keeps 2^-17 of those.  Three cost a
// seventh: 512 x 64 x 16 heads of 64, bf16, 132 us for 114, 4096 x 1 x 16 of 128 68
// for 59 (three of the state alone 123 and 65); the outputs are then 3e-5 to 4e-5
// (7e-5 to 9e-5) of their size from float32 arithmetic's, rounded, in the mean
// square, and 9e-5 to 1e-4 with two.  From the definition all are 1.7e-3 (Half
// 2.1e-4), which is their own rounding.
template <typename T>
cudaError_t launch_chunks(const AttnParams& p, cudaStream_t s, int* launches) {
  ChunkArgs args{};
  args.p = p;
  if constexpr (kSplit<T> == 1) {
    if (make_maps(args))
      return p.gradient ? launch_chunks_in<T, kTerms, true>(args, s, launches) : launch_chunks_in<T, 2, true>(args, s, launches);
  }
  if constexpr (kSplit<T> < kTerms)
    if (!p.gradient) return launch_chunks_in<T, 2, false>(args, s, launches);
  return launch_chunks_in<T, kTerms, false>(args, s, launches);
}

// A wait for a phase that nothing ends: it gives up after so many tries and sets
// the status word.
static __global__ void selftest_kernel(int tries) {
  __shared__ Small sh;
  if (threadIdx.x == 0) {
    bar_init(su32(&sh.bars[0]), 1);
    sh.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  wait_bar(sh, 0, 0, tries);
}
static cudaError_t launch_selftest(int tries, cudaStream_t s) {
  selftest_kernel<<<1, 32, 0, s>>>(tries);
  return cudaGetLastError();
}

// Reads and clears the status word, in stream order; the caller synchronises.
static cudaError_t take_status(cudaStream_t s, int* to) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(to, gave_up_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || *to == 0) return e;
  const int zero = 0;
  e = cudaMemcpyToSymbolAsync(gave_up_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace atc
}  // namespace rk
