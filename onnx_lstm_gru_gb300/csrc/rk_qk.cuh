// rk_qk.cuh -- queries and keys normalised and rotated by head, and the gradient.
//
//   n = x inv w;  a' = a c - b s, b' = b c + a s for each pair (a, b) of n
//   backward: g = the turn back of dy;  dw = sum of g x inv;
//   dx = inv (g w) - x inv^3 sum(g w x) / m,  m = size (root mean square) or 1
// A row is read once and everything is computed in registers.  A warp takes a
// row's heads in turns, so that a row's cosines and sines, which all heads
// share, are computed once; a lane holds both elements of its pairs, and a
// head's sum is a few exchanges of lanes.
// What bounds them is HBM and, next to it, instructions: 32768 rows of 16 + 16
// heads of 64, bf16, 53.3 us or 5.0 TB/s (74 % of a copy) at 2.4 warp instructions a
// clock and multiprocessor, 284 for a warp's 512 elements; the gradient of 8 + 8
// heads of 128 94 us, 4.3 TB/s (63 %), at 2.4, its 16 warps bound by registers.
#pragma once
#include <algorithm>

#include "rk.h"
#include "rk_attn.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace qk {
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
template <int V, bool IL>
__device__ __forceinline__ Unit unit_of(int u, int size, int rotary) {
  const int half = rotary / 2;
  if (IL) {
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
// Every pair's turn, taken once by a block as float64 is slow here, and the
// scales.
struct Turns {
  unsigned long long step[128];
  bool none[128];  // the frequency is infinite or NaN
  __align__(16) float scale[2][256];  // 1 where there is none
  // Whether there is a pair without a turn.
  template <typename T>
  __device__ __forceinline__ bool fill(const QkParams& p) {
    bool any = false;
    for (int i = threadIdx.x; i < p.rotary / 2; i += kQkThreads) {
      step[i] = turn_of(p.freq[i]);
      none[i] = !(fabsf(p.freq[i]) <= 3.402823466e38f);
      any |= none[i];
    }
    for (int i = threadIdx.x; i < 2 * p.size; i += kQkThreads) {
      const int side = i >= p.size, e = side ? i - p.size : i;
      const T* w = static_cast<const T*>(p.side[side].scale);
      scale[side][e] = w ? Elem<T>::to_f(w[e]) : 1.0f;
    }
    return __syncthreads_or(any);
  }
};

// Cosines and sines of the turns of two pairs.  float32 elements get CUDA's
// function, 16-bit ones polynomials of the distance x to the nearest quarter turn,
// |x| <= 1/2 quarters, in packed arithmetic: sin(pi x / 2) / x and (cos(pi x / 2) -
// 1) / x^2 as cubics in x^2, interpolated at the Chebyshev nodes of [0, 1/4].  They
// are off by 1e-7 at most, x's own rounding included.  (The special function unit
// is off by 4e-7, which elements turned to near zero show in Half and bfloat16.)
template <typename T>
__device__ __forceinline__ void turns_of(const long long (&phase)[2], F2& c, F2& s) {
  float cs[2], sn[2];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 2; ++e) sincospif((float)phase[e] * 1.0842021724855044e-19f, &sn[e], &cs[e]);  // 2^-63: in half turns
  } else {
    int quarter[2];
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t top = (uint32_t)((unsigned long long)phase[e] >> 32);  // turns in units of 2^-32
      quarter[e] = (int)((top + (1u << 29)) >> 30);
      x[e] = (float)(int)(top - ((uint32_t)quarter[e] << 30)) * 9.31322574615478515625e-10f;  // 2^-30
    }
    const F2 v = f2(x[0], x[1]), z = mul2(v, v);
    F2 p = f2(-0.004602149f, -0.004602149f), q = f2(0.0009067399f, 0.0009067399f);
    p = fma2(p, z, f2(0.07968022f, 0.07968022f)), q = fma2(q, z, f2(-0.020861529f, -0.020861529f));
    p = fma2(p, z, f2(-0.6459635f, -0.6459635f)), q = fma2(q, z, f2(0.2536694f, 0.2536694f));
    p = fma2(p, z, f2(1.5707964f, 1.5707964f)), q = fma2(q, z, f2(-1.2337005f, -1.2337005f));
    const float2 sine = f2_get(mul2(p, v)), cosine = f2_get(fma2(q, z, f2(1.0f, 1.0f)));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float a = e ? sine.y : sine.x, b = e ? cosine.y : cosine.x;
      const uint32_t odd = quarter[e] & 1, half = (uint32_t)quarter[e] >> 1 & 1;
      sn[e] = __uint_as_float(__float_as_uint(odd ? b : a) ^ half << 31);
      cs[e] = __uint_as_float(__float_as_uint(odd ? a : b) ^ (odd ^ half) << 31);
    }
  }
  c = f2(cs[0], cs[1]), s = f2(sn[0], sn[1]);
}

// A lane's units of a head: `lanes` lanes hold them, U each, in pieces of V
// elements.  Values are kept as packed pairs along V: a[j] the first elements
// of two of the rotated pairs, b[j] the second ones.
template <typename T, int V, int U, bool IL>
struct Lane {
  static constexpr int J = (V + 1) / 2;
  using Raw = Packed<T, V>;
  int a[U], b[U], pair[U];
  int na[U], nb[U];  // bytes of the two pieces that there are
  const Turns* table;
  F2 c[U][J], s[U][J], minus[U][J];  // of the position they were last taken for; -s
  int position;
  bool known, all, none;  // all pairs turn; some have none
  __device__ __forceinline__ Lane(const QkParams& p, const Turns* turns, bool none) : table(turns), known(false), all(p.rotary == p.size), none(none) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit x = unit_of<V, IL>(threadIdx.x % p.lanes + u * p.lanes, p.size, p.rotary);
      a[u] = x.a > 0 ? x.a : 0, b[u] = x.b > 0 ? x.b : 0, pair[u] = x.pair;
      na[u] = x.a >= 0 ? (int)sizeof(Raw) : 0, nb[u] = x.b >= 0 ? (int)sizeof(Raw) : 0;
    }
  }
  __device__ __forceinline__ bool turns(const QkParams& p, int u, int i) const { return pair[u] + i < p.rotary / 2; }
  // Rows at the same position, which whole batches are at, share their angles.
  // An infinite or NaN frequency has no turn: its pairs are NaN.
  __device__ __forceinline__ void angles(const QkParams& p, int at) {
    if (known && at == position) return;
    known = true, position = at;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        long long phase[2] = {0, 0};  // of a pair that stays
        bool nan[2] = {false, false};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * j + e;
          if (i < V && na[u] && turns(p, u, i)) {
            phase[e] = (long long)(table->step[pair[u] + i] * (unsigned long long)(long long)at);
            nan[e] = none && table->none[pair[u] + i];
          }
        }
        turns_of<T>(phase, c[u][j], s[u][j]);
        if (none) {
          const float2 x = f2_get(c[u][j]), y = f2_get(s[u][j]);
          const float bad = __int_as_float(0x7fffffff);
          c[u][j] = f2(nan[0] ? bad : x.x, nan[1] ? bad : x.y), s[u][j] = f2(nan[0] ? bad : y.x, nan[1] ? bad : y.y);
        }
        minus[u][j] = mul2(s[u][j], f2(-1.0f, -1.0f));
      }
  }
  // A unit's two pieces of a head's row on their way.
  template <typename S>
  __device__ __forceinline__ void start(const T* row, int u, bool on, const S& to, int i) const {
    to.start(i, row + a[u], on ? na[u] : 0);
    to.start(i + 1, row + b[u], on ? nb[u] : 0);
  }
  __device__ __forceinline__ static void pairs(const float (&e)[2 * V], F2 (&va)[J], F2 (&vb)[J]) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = 2 * j, k = V > 1 ? i + 1 : i;
      va[j] = f2(IL ? e[2 * i] : e[i], V > 1 ? (IL ? e[2 * k] : e[k]) : 0.0f);
      vb[j] = f2(IL ? e[2 * i + 1] : e[V + i], V > 1 ? (IL ? e[2 * k + 1] : e[V + k]) : 0.0f);
    }
  }
  template <typename S>
  __device__ __forceinline__ static void take(const S& from, int i, F2 (&va)[J], F2 (&vb)[J]) {
    float lo[V], hi[V], e[2 * V];
    Raw x[2];
    x[0].raw = from.piece(i), x[1].raw = from.piece(i + 1);
    x[0].widen(lo), x[1].widen(hi);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = lo[i], e[V + i] = hi[i];
    pairs(e, va, vb);
  }
  __device__ __forceinline__ void scales(int side, int u, F2 (&va)[J], F2 (&vb)[J]) const {
    float e[2 * V];
    const float* x = table->scale[side];
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(x + a[u] + i), g = *reinterpret_cast<const float4*>(x + b[u] + i);
        e[i] = f.x, e[i + 1] = f.y, e[i + 2] = f.z, e[i + 3] = f.w;
        e[V + i] = g.x, e[V + i + 1] = g.y, e[V + i + 2] = g.z, e[V + i + 3] = g.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = x[a[u] + i], e[V + i] = x[b[u] + i];
    }
    pairs(e, va, vb);
  }
  __device__ __forceinline__ void write(T* row, int u, bool on, const F2 (&va)[J], const F2 (&vb)[J]) const {
    float e[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 x = f2_get(va[i / 2]), y = f2_get(vb[i / 2]);
      const float fa = i % 2 ? x.y : x.x, fb = i % 2 ? y.y : y.x;
      e[0][i] = fa, e[1][i] = fb;
    }
    if constexpr (IL) {
      float z[2][V];
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) z[i / V][i % V] = e[i % 2][i / 2];
#pragma unroll
      for (int i = 0; i < V; ++i) e[0][i] = z[0][i], e[1][i] = z[1][i];
    }
    Raw x[2];
    x[0].narrow(e[0]), x[1].narrow(e[1]);
    if (on && na[u]) x[0].store(row + a[u]);
    if (on && nb[u]) x[1].store(row + b[u]);
  }
  __device__ __forceinline__ void forth(int u, int j, F2 x, F2 y, F2& tx, F2& ty) const {
    tx = fma2(x, c[u][j], mul2(y, minus[u][j])), ty = fma2(y, c[u][j], mul2(x, s[u][j]));
  }
  __device__ __forceinline__ void back(int u, int j, F2 x, F2 y, F2& tx, F2& ty) const {
    tx = fma2(x, c[u][j], mul2(y, s[u][j])), ty = fma2(y, c[u][j], mul2(mul2(x, s[u][j]), f2(-1.0f, -1.0f)));  // registers are short there
  }
  // Pairs that stay are left as they are, infinities too.
  __device__ __forceinline__ void pick(const QkParams& p, int u, int j, F2 ta, F2 tb, F2& va, F2& vb) const {
    const float2 x0 = f2_get(va), y0 = f2_get(vb), x1 = f2_get(ta), y1 = f2_get(tb);
    const bool t0 = turns(p, u, 2 * j), t1 = turns(p, u, 2 * j + 1);
    va = f2(t0 ? x1.x : x0.x, t1 ? x1.y : x0.y), vb = f2(t0 ? y1.x : y0.x, t1 ? y1.y : y0.y);
  }
};
__device__ __forceinline__ float sum_of(F2 x) {
  const float2 v = f2_get(x);
  return v.x + v.y;
}

__device__ __forceinline__ float head_sum(const QkParams& p, float v) {
#pragma unroll 1
  for (int o = p.lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row number i in the order that they are taken in, as step and batch row, and
// whether it holds work.  Without positions the rows of a step, which are at
// the same one, follow each other in either layout.
__device__ __forceinline__ bool row_of(const QkParams& p, long long i, int& s, int& n) {
  const bool by_step = p.layout == 0 || p.positions == nullptr;
  const int inner = by_step ? p.N : p.S;
  const int o = (int)(i / inner), k = (int)(i - (long long)o * inner);
  s = by_step ? o : k;
  n = by_step ? k : o;
  return s < row_length(p.lens, n, p.S);
}
__device__ __forceinline__ int position_of(const QkParams& p, int s, int n) {
  return p.positions ? p.positions[p.layout == 0 ? (long long)s * p.N + n : (long long)n * p.S + s] : s;
}

// The reciprocal square root is off by 2^-22 at most, which no 16-bit element
// keeps; `mean` is 1 / size or 1.
template <typename T>
__device__ __forceinline__ float inverse(const QkParams& p, float square, float mean) {
  if constexpr (sizeof(T) == 2) return p.norm == 0 ? 1.0f : rsqrtf(fmaf(square, mean, p.epsilon));
  if (p.norm == 0) return 1.0f;
  return 1.0f / sqrtf((p.norm == 1 ? square / (float)p.size : square) + p.epsilon);
}

// A warp's way through its rows, and through a row's heads in turns of heads:
// queries first, where both sides are taken.  Rows are counted in the order of
// row_of; `share` warps take a row's turns between them.
template <typename T, bool GRAD>
struct Way {
  long long item, last;
  int s, n, side, part, h0;
  bool live;
  const T* X;  // of the row
  const T* dY;
  T* out;
  __device__ __forceinline__ bool more() const { return item < last; }
  __device__ __forceinline__ void place(const QkParams& p, int heads) {
    const QkSide& q = p.side[side];
    X = static_cast<const T*>(q.X.p) + s * q.X.ss + n * q.X.ns;
    if constexpr (GRAD) dY = static_cast<const T*>(q.dY.p) + s * q.dY.ss + n * q.dY.ns;
    const RowsArg& o = GRAD ? q.dX : q.Y;
    out = static_cast<T*>(o.p) + s * o.ss + n * o.ns;
    h0 = part * heads;
  }
  __device__ __forceinline__ void row(const QkParams& p) {
    const long long r = p.share == 1 ? item : item / p.share;
    part = (int)(item - r * p.share);
    live = row_of(p, r, s, n);
  }
  __device__ __forceinline__ Way(const QkParams& p, int first_side, int heads, long long items, long long warps, int warp) {
    const long long per = (items + warps - 1) / warps;
    item = per * warp, last = item + per < items ? item + per : items;
    side = first_side;
    if (more()) {
      row(p);
      place(p, heads);
    }
  }
  // One turn on: the next heads of the row, the other side, or the next row.
  __device__ __forceinline__ void step(const QkParams& p, int heads) {
    h0 += heads * p.share;
    if (h0 < p.side[side].heads) return;
    if (!GRAD && side == 0 && p.side[1].Y.p) {
      side = 1;
    } else {
      if (!GRAD && p.side[0].Y.p) side = 0;
      ++item;
      if (!more()) return;
      // the next row in most cases by counting
      const bool by_step = p.layout == 0 || p.positions == nullptr;
      if (p.share == 1 && (by_step ? n + 1 < p.N : s + 1 < p.S)) {
        by_step ? ++n : ++s;
        live = s < row_length(p.lens, n, p.S);
      } else {
        row(p);
      }
    }
    place(p, heads);
  }
};

// Turns on their way: kAhead of them, N pieces each, every thread in its own
// places, so that only its own copies have to be waited for.  Registers for as
// many would leave no room for two blocks on a multiprocessor.
constexpr int kAhead = 3, kSlots = kAhead + 1;
struct __align__(16) Turn {
  void* out;
  int at;  // bits 0, 1, 2: a turn, of a live row, of a head that there is; 3: of the keys
  int position;
};
template <typename Raw, int N>
struct Slot {
  static constexpr int kBytes = kSlots * kQkThreads * (int)(sizeof(Turn) + N * sizeof(Raw));
  char* smem;
  int slot;
  __device__ __forceinline__ explicit Slot(char* s) : smem(s), slot(0) {}
  __device__ __forceinline__ void next() { slot = (slot + 1) % kSlots; }
  __device__ __forceinline__ Turn& turn() const { return reinterpret_cast<Turn*>(smem)[slot * kQkThreads + threadIdx.x]; }
  __device__ __forceinline__ Raw& piece(int i) const {
    return reinterpret_cast<Raw*>(smem + kSlots * kQkThreads * sizeof(Turn))[(slot * N + i) * kQkThreads + threadIdx.x];
  }
  // A piece, or zeros; copies are of 4 bytes at least.
  __device__ __forceinline__ void start(int i, const void* from, int bytes) const {
    constexpr int kSize = sizeof(Raw);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(&piece(i));
    if constexpr (kSize == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    else if constexpr (kSize >= 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(kSize), "r"(bytes)
                   : "memory");
    else piece(i) = bytes ? *static_cast<const Raw*>(from) : Raw{};
  }
  __device__ __forceinline__ static void sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest of kSlots that were sent is there.
  __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory"); }
};

template <typename T, int V, int U, bool IL>
__global__ void __launch_bounds__(kQkThreads, U > 2 ? 1 : 2) qk_kernel(QkParams p) {
  using L = Lane<T, V, U, IL>;
  constexpr int J = L::J;
  const int lane = threadIdx.x % 32, heads = 32 / p.lanes, mine = lane / p.lanes, own = mine * p.size;
  const float mean = p.norm == 1 ? 1.0f / (float)p.size : 1.0f;
  __shared__ Turns turns;
  const bool none = turns.fill<T>(p);
  L l(p, &turns, none);
  const long long items = (long long)p.S * p.N * p.share, warps = (long long)gridDim.x * kQkWarps;
  Way<T, false> way(p, p.side[0].Y.p ? 0 : 1, heads, items, warps, (int)(blockIdx.x * kQkWarps + threadIdx.x / 32));

  extern __shared__ __align__(16) char smem[];
  using S = Slot<typename L::Raw::Raw, 2 * U>;
  S into(smem), from(smem);
  auto fetch = [&] {
    Turn t = {nullptr, 0, 0};
    if (way.more()) {
      const bool is = way.h0 + mine < p.side[way.side].heads;
      const int at = is ? way.h0 * p.size + own : 0;
      t.out = way.out + at;
      t.at = 1 | (way.live ? 2 : 0) | (is ? 4 : 0) | (way.side ? 8 : 0);
      t.position = way.live ? position_of(p, way.s, way.n) : 0;
#pragma unroll
      for (int u = 0; u < U; ++u) l.start(way.X + at, u, is && way.live, into, 2 * u);
      way.step(p, heads);
    }
    S::sent();
    into.turn() = t;
    into.next();
  };
  auto compute = [&](const Turn& t) {
    const bool live = t.at & 2;
    if (live) l.angles(p, t.position);
    F2 a[U][J], b[U][J], square = f2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      L::take(from, 2 * u, a[u], b[u]);
#pragma unroll
      for (int j = 0; j < J; ++j) square = fma2(a[u][j], a[u][j], fma2(b[u][j], b[u][j], square));
    }
    const float inv = inverse<T>(p, p.norm ? head_sum(p, sum_of(square)) : 0.0f, mean);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (live) {
        F2 wa[J], wb[J];
        l.scales(t.at >> 3, u, wa, wb);
#pragma unroll
        for (int j = 0; j < J; ++j)
          a[u][j] = mul2(mul2(a[u][j], f2(inv, inv)), wa[j]), b[u][j] = mul2(mul2(b[u][j], f2(inv, inv)), wb[j]);
        if (l.all) {
#pragma unroll
          for (int j = 0; j < J; ++j) l.forth(u, j, a[u][j], b[u][j], a[u][j], b[u][j]);
        } else {
#pragma unroll
          for (int j = 0; j < J; ++j) {
            F2 ta, tb;
            l.forth(u, j, a[u][j], b[u][j], ta, tb);
            l.pick(p, u, j, ta, tb, a[u][j], b[u][j]);
          }
        }
      }
      l.write(static_cast<T*>(t.out), u, t.at & 4, a[u], b[u]);
    }
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) fetch();
#pragma unroll 1
  for (;;) {
    fetch();
    const Turn t = from.turn();
    if (!t.at) break;
    S::wait();
    compute(t);
    from.next();
  }
}

template <typename T, int V, int U, bool IL>
__global__ void __launch_bounds__(kQkThreads, U > 2 ? 1 : 2) qk_grad_kernel(QkParams p) {
  next_may_start();
  using L = Lane<T, V, U, IL>;
  constexpr int J = L::J;
  const int lane = threadIdx.x % 32, heads = 32 / p.lanes, mine = lane / p.lanes, own = mine * p.size;
  const float mean = p.norm == 1 ? 1.0f / (float)p.size : 1.0f;
  __shared__ Turns turns;
  const bool none = turns.fill<T>(p);
  L l(p, &turns, none);
  const long long rows = (long long)p.S * p.N, warps = (long long)gridDim.x * kQkWarps;
  extern __shared__ __align__(16) char smem[];
  using S = Slot<typename L::Raw::Raw, 4 * U>;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const QkSide& q = p.side[side];
    S into(smem), from(smem);
    F2 dwa[U][J], dwb[U][J];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < J; ++j) dwa[u][j] = dwb[u][j] = f2(0.0f, 0.0f);
    }
    Way<T, true> way(p, side, heads, q.dX.p || q.dscale ? rows : 0, warps, (int)(blockIdx.x * kQkWarps + threadIdx.x / 32));
    auto fetch = [&] {
      Turn t = {nullptr, 0, 0};
      if (way.more()) {
        const bool is = way.h0 + mine < q.heads;
        const int at = is ? way.h0 * p.size + own : 0;
        t.out = way.out + at;
        t.at = 1 | (way.live ? 2 : 0) | (is ? 4 : 0);
        t.position = way.live ? position_of(p, way.s, way.n) : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          l.start(way.X + at, u, is && way.live, into, 4 * u);
          l.start(way.dY + at, u, is && way.live, into, 4 * u + 2);
        }
        way.step(p, heads);
      }
      S::sent();
      into.turn() = t;
      into.next();
    };
    auto compute = [&](const Turn& t) {
      const bool live = t.at & 2, is = t.at & 4;
      if (live) l.angles(p, t.position);
      F2 a[U][J], b[U][J], ga[U][J], gb[U][J], square = f2(0.0f, 0.0f), dot = f2(0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        L::take(from, 4 * u, a[u], b[u]);
        L::take(from, 4 * u + 2, ga[u], gb[u]);
#pragma unroll
        for (int j = 0; j < J; ++j) square = fma2(a[u][j], a[u][j], fma2(b[u][j], b[u][j], square));
      }
      const float inv = inverse<T>(p, p.norm ? head_sum(p, sum_of(square)) : 0.0f, mean);
      if (live) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          F2 wa[J], wb[J];
          l.scales(side, u, wa, wb);
          if (l.all) {
#pragma unroll
            for (int j = 0; j < J; ++j) l.back(u, j, ga[u][j], gb[u][j], ga[u][j], gb[u][j]);
          } else {
#pragma unroll
            for (int j = 0; j < J; ++j) {
              F2 ta, tb;
              l.back(u, j, ga[u][j], gb[u][j], ta, tb);
              l.pick(p, u, j, ta, tb, ga[u][j], gb[u][j]);
            }
          }
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const F2 va = ga[u][j], vb = gb[u][j];
            a[u][j] = mul2(a[u][j], f2(inv, inv)), b[u][j] = mul2(b[u][j], f2(inv, inv));  // x inv from here on
            if (is) dwa[u][j] = fma2(va, a[u][j], dwa[u][j]), dwb[u][j] = fma2(vb, b[u][j], dwb[u][j]);
            ga[u][j] = mul2(va, wa[j]), gb[u][j] = mul2(vb, wb[j]);
            dot = fma2(ga[u][j], a[u][j], fma2(gb[u][j], b[u][j], dot));
          }
        }
      }
      // inv (g - (x inv) sum(g x inv) / m): x inv is of the head's own size, and inv^3 alone may pass float32's range
      const float f = p.norm ? -head_sum(p, sum_of(dot)) * mean : 0.0f;
      if (q.dX.p) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (live) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
              if (p.norm) ga[u][j] = fma2(f2(f, f), a[u][j], ga[u][j]), gb[u][j] = fma2(f2(f, f), b[u][j], gb[u][j]);
              ga[u][j] = mul2(ga[u][j], f2(inv, inv)), gb[u][j] = mul2(gb[u][j], f2(inv, inv));
            }
          }
          l.write(static_cast<T*>(t.out), u, is, ga[u], gb[u]);
        }
      }
    };
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) fetch();
#pragma unroll 1
    for (;;) {
      fetch();
      const Turn t = from.turn();
      if (!t.at) break;
      S::wait();
      compute(t);
      from.next();
    }
    if (p.partial == nullptr) continue;
    // the block's sums: over the head groups of a warp, then over the warps
    __shared__ float sums[kQkWarps][256];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 y = f2_get(j ? dwb[u][i / 2] : dwa[u][i / 2]);
          float v = i % 2 ? y.y : y.x;
#pragma unroll
          for (int o = 16; o >= p.lanes; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          const int e = IL ? 2 * i + j : i;  // place in the two pieces, or in its own
          const bool second = IL ? e >= V : j;
          const int from = second ? l.b[u] : l.a[u];
          if (lane < p.lanes && (second ? l.nb[u] : l.na[u])) sums[threadIdx.x / 32][from + (IL && e >= V ? e - V : e)] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < p.size; i += kQkThreads) {
      float v = 0.0f;
#pragma unroll
      for (int x = 0; x < kQkWarps; ++x) v += sums[x][i];
      p.partial[((long long)blockIdx.x * 2 + side) * p.size + i] = v;
    }
    __syncthreads();
  }
}

// Units of V elements' pieces that cover a head.
int units(const QkParams& p, int V) {
  if (p.interleaved) return (p.size + 2 * V - 1) / (2 * V);
  return p.rotary / 2 / V + ((p.size - p.rotary) / V + 1) / 2;
}

template <typename T, int V, int U, bool IL, bool GRAD>
cudaError_t launch_form(const QkParams& p, cudaStream_t s) {
  constexpr int smem = Slot<typename Packed<T, V>::Raw, (GRAD ? 4 : 2) * U>::kBytes;
  void (*kernel)(QkParams);
  if constexpr (GRAD) kernel = qk_grad_kernel<T, V, U, IL>;
  else kernel = qk_kernel<T, V, U, IL>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)p.S * p.N * p.share, blocks = (warps + kQkWarps - 1) / kQkWarps;
  const unsigned grid = GRAD ? (unsigned)p.blocks : (unsigned)std::min<long long>(blocks, kPlanSms * 2);
  kernel<<<grid, kQkThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, bool IL, bool GRAD>
cudaError_t launch_lanes(QkParams p, cudaStream_t s) {
  const int n = units(p, V);
  int lanes = 1;
  while (lanes < n && lanes < 32) lanes *= 2;
  p.lanes = lanes;
  const int turns = (std::max(p.side[0].heads, p.side[1].heads) * lanes + 31) / 32;
  const long long rows = (long long)p.S * p.N;
  // few rows: as many warps as there are turns of heads share one
  p.share = GRAD ? 1 : (int)std::max<long long>(1, std::min<long long>(turns, kPlanSms * 16 / std::max<long long>(rows, 1)));
  // 256 elements are 128 / V units
  if constexpr (V == 1)
    if (n > 64) return launch_form<T, V, 4, IL, GRAD>(p, s);
  if constexpr (V <= 2)
    if (n > 32) return launch_form<T, V, 2, IL, GRAD>(p, s);
  return launch_form<T, V, 1, IL, GRAD>(p, s);
}

template <typename T, int V, bool GRAD>
cudaError_t launch_order(const QkParams& p, cudaStream_t s) {
  return p.interleaved ? launch_lanes<T, V, true, GRAD>(p, s) : launch_lanes<T, V, false, GRAD>(p, s);
}

template <typename T, bool GRAD>
cudaError_t launch_type(const QkParams& p, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (p.piece == 8) return launch_order<T, 8, GRAD>(p, s);
  if (p.piece == 4) return launch_order<T, 4, GRAD>(p, s);
  return p.piece == 2 ? launch_order<T, 2, GRAD>(p, s) : launch_order<T, 1, GRAD>(p, s);
}

template <bool GRAD>
cudaError_t launch_any(const QkParams& p, cudaStream_t s) {
  if (p.dtype == RK_F32) return launch_type<float, GRAD>(p, s);
  return p.dtype == RK_F16 ? launch_type<__half, GRAD>(p, s) : launch_type<__nv_bfloat16, GRAD>(p, s);
}

}  // namespace
}  // namespace qk
}  // namespace rk
