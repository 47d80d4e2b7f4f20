// rk_qk.cu -- queries and keys normalised and rotated by head, and the gradient.
//
//   n = x inv w;  a' = a c - b s, b' = b c + a s for each pair (a, b) of n
//   backward: g = the turn back of dy;  dw = sum of g x inv;
//   dx = inv (g w) - x inv^3 sum(g w x) / m,  m = size (root mean square) or 1
// Both are bound by HBM: a row is read once and everything is computed in
// registers.  A warp takes a row's heads in turns, so that a row's cosines and
// sines, which all heads share, are computed once; a lane holds both elements
// of its pairs, and a head's sum is a few exchanges of lanes.
#include <algorithm>

#include "rk.h"
#include "rk_attn.h"
#include "rk_ssm_common.cuh"

namespace rk {
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
template <int V>
__device__ __forceinline__ Unit unit_of(int u, int size, int rotary, bool interleaved) {
  const int half = rotary / 2;
  if (interleaved) {
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
// Every pair's turn, taken once by a block: float64 is slow here.
struct Turns {
  unsigned long long step[128];
  bool none[128];  // the frequency is infinite or NaN
  __device__ __forceinline__ void fill(const QkParams& p) {
    for (int i = threadIdx.x; i < p.rotary / 2; i += kQkThreads) {
      step[i] = turn_of(p.freq[i]);
      none[i] = !(fabsf(p.freq[i]) <= 3.402823466e38f);
    }
    __syncthreads();
  }
};

// Cosine and sine of a turn.  The special function unit's are off by 2^-20 at
// most within half a turn, which no 16-bit element keeps.
template <typename T>
__device__ __forceinline__ void turn(unsigned long long step, int position, float& c, float& s) {
  const long long phase = (long long)(step * (unsigned long long)(long long)position);
  if constexpr (sizeof(T) == 4) {
    sincospif((float)phase * 1.0842021724855044e-19f, &s, &c);  // 2^-63: in half turns
  } else {
    const float angle = (float)(int)(phase >> 32) * (float)(3.14159265358979323846 / 2147483648.0);
    s = __sinf(angle), c = __cosf(angle);
  }
}

// A lane's units of a head: LPH lanes hold them, U each, in pieces of V
// elements.  Values are kept as packed pairs along V: a[j] the first elements
// of two of the rotated pairs, b[j] the second ones.
template <typename T, int V, int LPH, int U>
struct Lane {
  static constexpr int J = (V + 1) / 2;
  using Raw = Packed<T, V>;
  int a[U], b[U], pair[U];
  const Turns* table;
  F2 c[U][J], s[U][J];  // of the position they were last taken for
  int position;
  bool known;
  __device__ __forceinline__ Lane(const QkParams& p, int sub, const Turns* turns) : table(turns), known(false) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit x = unit_of<V>(sub + u * LPH, p.size, p.rotary, p.interleaved);
      a[u] = x.a, b[u] = x.b, pair[u] = x.pair;
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
        float cs[2] = {1.0f, 1.0f}, sn[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * j + e;
          if (i < V && a[u] >= 0 && turns(p, u, i)) {
            turn<T>(table->step[pair[u] + i], at, cs[e], sn[e]);
            if (table->none[pair[u] + i]) cs[e] = sn[e] = __int_as_float(0x7fffffff);
          }
        }
        c[u][j] = f2(cs[0], cs[1]), s[u][j] = f2(sn[0], sn[1]);
      }
  }
  // A unit's two pieces of a head's row as read.
  __device__ __forceinline__ void read(const T* row, int u, bool on, Raw (&x)[2]) const {
    if (on && a[u] >= 0) x[0].load(row + a[u]);
    else x[0].raw = {};
    if (on && b[u] >= 0) x[1].load(row + b[u]);
    else x[1].raw = {};
  }
  __device__ __forceinline__ static void widen(bool interleaved, const Raw (&x)[2], F2 (&va)[J], F2 (&vb)[J]) {
    float e[2 * V];
    {
      float lo[V], hi[V];
      x[0].widen(lo), x[1].widen(hi);
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = lo[i], e[V + i] = hi[i];
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int i = 2 * j, k = V > 1 ? i + 1 : i;
      const float y = V > 1 ? 1.0f : 0.0f;
      va[j] = f2(interleaved ? e[2 * i] : e[i], V > 1 ? (interleaved ? e[2 * k] : e[k]) : y);
      vb[j] = f2(interleaved ? e[2 * i + 1] : e[V + i], V > 1 ? (interleaved ? e[2 * k + 1] : e[V + k]) : y);
    }
  }
  __device__ __forceinline__ void write(T* row, int u, bool on, bool interleaved, const F2 (&va)[J], const F2 (&vb)[J]) const {
    float e[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 x = f2_get(va[i / 2]), y = f2_get(vb[i / 2]);
      const float fa = i % 2 ? x.y : x.x, fb = i % 2 ? y.y : y.x;
      e[0][i] = fa, e[1][i] = fb;
    }
    if (interleaved) {
      float z[2][V];
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) z[i / V][i % V] = e[i % 2][i / 2];
#pragma unroll
      for (int i = 0; i < V; ++i) e[0][i] = z[0][i], e[1][i] = z[1][i];
    }
    if (on && a[u] >= 0) Piece<T, V>::store(row + a[u], e[0]);
    if (on && b[u] >= 0) Piece<T, V>::store(row + b[u], e[1]);
  }
};
__device__ __forceinline__ F2 negated(F2 x) { return mul2(x, f2(-1.0f, -1.0f)); }
__device__ __forceinline__ float sum_of(F2 x) {
  const float2 v = f2_get(x);
  return v.x + v.y;
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

__device__ __forceinline__ float inverse(const QkParams& p, float square) {
  if (p.norm == 0) return 1.0f;
  return 1.0f / sqrtf((p.norm == 1 ? square / (float)p.size : square) + p.epsilon);
}

// A warp's way through its rows, and through a row's heads in turns of kHeads:
// queries first, where both sides are taken.  Rows are counted in the order of
// row_of; `share` warps take a row's turns between them.
struct Way {
  long long item, last;
  int s, n, side, part, h0;
  bool live;
  __device__ __forceinline__ bool more() const { return item < last; }
  __device__ __forceinline__ void row(const QkParams& p) {
    const long long r = p.share == 1 ? item : item / p.share;
    part = (int)(item - r * p.share);
    live = row_of(p, r, s, n);
  }
  __device__ __forceinline__ Way(const QkParams& p, int first_side, int heads, long long items, long long warps, int warp) {
    const long long per = (items + warps - 1) / warps;
    item = per * warp, last = item + per < items ? item + per : items;
    side = first_side;
    s = n = part = h0 = 0;
    live = false;
    if (more()) {
      row(p);
      h0 = part * heads;
    }
  }
  // One turn on: the next heads of the row, the other side, or the next row.
  template <bool BOTH>
  __device__ __forceinline__ void step(const QkParams& p, int heads) {
    h0 += heads * p.share;
    if (h0 < p.side[side].heads) return;
    if (BOTH && side == 0 && p.side[1].Y.p) {
      side = 1, h0 = part * heads;
      return;
    }
    if (BOTH && p.side[0].Y.p) side = 0;
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
    h0 = part * heads;
  }
};

// Turns' elements are on their way two turns ahead.
template <typename T, int V, int LPH, int U>
__global__ void __launch_bounds__(kQkThreads, U > 1 ? 1 : V > 1 ? 2 : 3) qk_kernel(QkParams p) {
  constexpr int kHeads = 32 / LPH;
  using L = Lane<T, V, LPH, U>;
  constexpr int J = L::J;
  const int lane = threadIdx.x % 32, sub = lane % LPH;
  __shared__ Turns turns;
  turns.fill(p);
  L l(p, sub, &turns);
  const bool il = p.interleaved;
  typename L::Raw w[2][U][2];
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int u = 0; u < U; ++u) l.read(static_cast<const T*>(p.side[side].scale), u, p.side[side].scale != nullptr, w[side][u]);
  const long long items = (long long)p.S * p.N * p.share, warps = (long long)gridDim.x * kQkWarps;
  Way way(p, p.side[0].Y.p ? 0 : 1, kHeads, items, warps, (int)(blockIdx.x * kQkWarps + threadIdx.x / 32));

  struct Turn {
    T* Y;
    int at;  // bits 0, 1, 2: a turn, of a live row, of a head that there is; 3: of the keys
    int position;
    typename L::Raw x[U][2];
  };
  auto fetch = [&](Turn& t) {
    t.at = 0;
    if (!way.more()) return;
    const QkSide& q = p.side[way.side];
    const int h = way.h0 + lane / LPH;
    const T* X = static_cast<const T*>(q.X.p) + way.s * q.X.ss + way.n * q.X.ns + h * p.size;
    t.Y = static_cast<T*>(q.Y.p) + way.s * q.Y.ss + way.n * q.Y.ns + h * p.size;
    t.at = 1 | (way.live ? 2 : 0) | (h < q.heads ? 4 : 0) | (way.side ? 8 : 0);
    t.position = way.live ? position_of(p, way.s, way.n) : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) l.read(X, u, (t.at & 6) == 6, t.x[u]);
    way.step<true>(p, kHeads);
  };
  auto compute = [&](Turn& t) {
    const bool live = t.at & 2, keys = t.at & 8, scaled = p.side[keys].scale;
    if (live) l.angles(p, t.position);
    F2 a[U][J], b[U][J], square = f2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      L::widen(il, t.x[u], a[u], b[u]);
      if constexpr (V == 1) a[u][0] = mul2(a[u][0], f2(1.0f, 0.0f)), b[u][0] = mul2(b[u][0], f2(1.0f, 0.0f));
#pragma unroll
      for (int j = 0; j < J; ++j) square = fma2(a[u][j], a[u][j], fma2(b[u][j], b[u][j], square));
    }
    const float inv = inverse(p, p.norm ? head_sum<LPH>(sum_of(square)) : 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (live) {
        F2 wa[J], wb[J];
        typename L::Raw ws[2] = {keys ? w[1][u][0] : w[0][u][0], keys ? w[1][u][1] : w[0][u][1]};
        L::widen(il, ws, wa, wb);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          F2 va = mul2(a[u][j], f2(inv, inv)), vb = mul2(b[u][j], f2(inv, inv));
          if (scaled) va = mul2(va, wa[j]), vb = mul2(vb, wb[j]);
          F2 ta = fma2(va, l.c[u][j], negated(mul2(vb, l.s[u][j]))), tb = fma2(vb, l.c[u][j], mul2(va, l.s[u][j]));
          // pairs that stay are left as they are, infinities too
          const float2 x0 = f2_get(va), y0 = f2_get(vb), x1 = f2_get(ta), y1 = f2_get(tb);
          const bool t0 = l.turns(p, u, 2 * j), t1 = l.turns(p, u, 2 * j + 1);
          a[u][j] = f2(t0 ? x1.x : x0.x, t1 ? x1.y : x0.y), b[u][j] = f2(t0 ? y1.x : y0.x, t1 ? y1.y : y0.y);
        }
      }
      l.write(t.Y, u, t.at & 4, il, a[u], b[u]);
    }
  };
  Turn t0, t1, t2;
  fetch(t0);
  fetch(t1);
#pragma unroll 1
  while (t0.at) {
    fetch(t2);
    compute(t0);
    t0 = t1, t1 = t2;
  }
}

template <typename T, int V, int LPH, int U>
__global__ void __launch_bounds__(kQkThreads, U == 1 ? 2 : 1) qk_grad_kernel(QkParams p) {
  constexpr int kHeads = 32 / LPH;
  using L = Lane<T, V, LPH, U>;
  constexpr int J = L::J;
  const int lane = threadIdx.x % 32, sub = lane % LPH;
  __shared__ Turns turns;
  turns.fill(p);
  L l(p, sub, &turns);
  const long long rows = (long long)p.S * p.N, warps = (long long)gridDim.x * kQkWarps;
  const bool il = p.interleaved;
  const float m = p.norm == 1 ? 1.0f / (float)p.size : 1.0f;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const QkSide& q = p.side[side];
    typename L::Raw w[U][2];
    F2 dwa[U][J], dwb[U][J];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      l.read(static_cast<const T*>(q.scale), u, q.scale != nullptr, w[u]);
#pragma unroll
      for (int j = 0; j < J; ++j) dwa[u][j] = dwb[u][j] = f2(0.0f, 0.0f);
    }
    struct Turn {
      T* dX;
      int at;  // bits 0, 1, 2: a turn, of a live row, of a head that there is
      int position;
      typename L::Raw x[U][2], g[U][2];
    };
    Way way(p, side, kHeads, q.dX.p || q.dscale ? rows : 0, warps, (int)(blockIdx.x * kQkWarps + threadIdx.x / 32));
    auto fetch = [&](Turn& t) {
      t.at = 0;
      if (!way.more()) return;
      const int h = way.h0 + lane / LPH;
      const T* X = static_cast<const T*>(q.X.p) + way.s * q.X.ss + way.n * q.X.ns + h * p.size;
      const T* dY = static_cast<const T*>(q.dY.p) + way.s * q.dY.ss + way.n * q.dY.ns + h * p.size;
      t.dX = static_cast<T*>(q.dX.p) + way.s * q.dX.ss + way.n * q.dX.ns + h * p.size;
      t.at = 1 | (way.live ? 2 : 0) | (h < q.heads ? 4 : 0);
      t.position = way.live ? position_of(p, way.s, way.n) : 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        l.read(X, u, (t.at & 6) == 6, t.x[u]);
        l.read(dY, u, (t.at & 6) == 6, t.g[u]);
      }
      way.step<false>(p, kHeads);
    };
    auto compute = [&](Turn& t) {
      const bool live = t.at & 2, is = t.at & 4;
      if (live) l.angles(p, t.position);
      F2 a[U][J], b[U][J], ga[U][J], gb[U][J], square = f2(0.0f, 0.0f), dot = f2(0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        L::widen(il, t.x[u], a[u], b[u]);
        L::widen(il, t.g[u], ga[u], gb[u]);
        if constexpr (V == 1) {
          a[u][0] = mul2(a[u][0], f2(1.0f, 0.0f)), b[u][0] = mul2(b[u][0], f2(1.0f, 0.0f));
          ga[u][0] = mul2(ga[u][0], f2(1.0f, 0.0f)), gb[u][0] = mul2(gb[u][0], f2(1.0f, 0.0f));
        }
#pragma unroll
        for (int j = 0; j < J; ++j) square = fma2(a[u][j], a[u][j], fma2(b[u][j], b[u][j], square));
      }
      const float inv = inverse(p, p.norm ? head_sum<LPH>(sum_of(square)) : 0.0f);
      if (live) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          F2 wa[J], wb[J];
          L::widen(il, w[u], wa, wb);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const F2 ta = fma2(ga[u][j], l.c[u][j], mul2(gb[u][j], l.s[u][j]));
            const F2 tb = fma2(gb[u][j], l.c[u][j], negated(mul2(ga[u][j], l.s[u][j])));
            const float2 x0 = f2_get(ga[u][j]), y0 = f2_get(gb[u][j]), x2 = f2_get(ta), y2 = f2_get(tb);
            const bool t0 = l.turns(p, u, 2 * j), t1 = l.turns(p, u, 2 * j + 1);
            F2 va = f2(t0 ? x2.x : x0.x, t1 ? x2.y : x0.y), vb = f2(t0 ? y2.x : y0.x, t1 ? y2.y : y0.y);
            a[u][j] = mul2(a[u][j], f2(inv, inv)), b[u][j] = mul2(b[u][j], f2(inv, inv));  // x inv from here on
            if (is) dwa[u][j] = fma2(va, a[u][j], dwa[u][j]), dwb[u][j] = fma2(vb, b[u][j], dwb[u][j]);
            if (q.scale) va = mul2(va, wa[j]), vb = mul2(vb, wb[j]);
            ga[u][j] = va, gb[u][j] = vb;
            dot = fma2(va, a[u][j], fma2(vb, b[u][j], dot));
          }
        }
      }
      // inv (g - (x inv) sum(g x inv) / m): x inv is of the head's own size, and inv^3 alone may pass float32's range
      const float f = p.norm ? -head_sum<LPH>(sum_of(dot)) * m : 0.0f;
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
          l.write(t.dX, u, is, il, ga[u], gb[u]);
        }
      }
    };
    Turn t0, t1;
    fetch(t0);
#pragma unroll 1
    while (t0.at) {
      fetch(t1);
      compute(t0);
      t0 = t1;
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
          for (int o = 16; o >= LPH; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          const int e = il ? 2 * i + j : i;  // place in the two pieces, or in its own
          const int from = il ? (e < V ? l.a[u] : l.b[u]) : (j ? l.b[u] : l.a[u]);
          if (lane < LPH && from >= 0) sums[threadIdx.x / 32][from + (il && e >= V ? e - V : e)] = v;
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

// Sums over the blocks, one warp for each element of the two scales.
__global__ void __launch_bounds__(256) qk_scale_kernel(QkParams p) {
  const int i = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (i >= 2 * p.size) return;
  float* out = i < p.size ? p.side[0].dscale : p.side[1].dscale;
  if (out == nullptr) return;
  float v = 0.0f;
  for (int b = lane; b < p.blocks; b += 32) v += p.partial[(long long)b * 2 * p.size + i];
  v = warp_sum(v);
  if (lane == 0) out[i < p.size ? i : i - p.size] = v;
}

// Units of V elements' pieces that cover a head.
int units(const QkParams& p, int V) {
  if (p.interleaved) return (p.size + 2 * V - 1) / (2 * V);
  return p.rotary / 2 / V + ((p.size - p.rotary) / V + 1) / 2;
}

template <typename T, int V, int LPH, int U, bool GRAD>
cudaError_t launch_form(const QkParams& p, cudaStream_t s) {
  if constexpr (GRAD) {
    qk_grad_kernel<T, V, LPH, U><<<p.blocks, kQkThreads, 0, s>>>(p);
  } else {
    const long long warps = (long long)p.S * p.N * p.share;
    const long long blocks = (warps + kQkWarps - 1) / kQkWarps;
    qk_kernel<T, V, LPH, U><<<(unsigned)std::min<long long>(blocks, kPlanSms * (V > 1 ? 2 : 3)), kQkThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int V, bool GRAD>
cudaError_t launch_lanes(QkParams p, cudaStream_t s) {
  const int n = units(p, V);
  int lanes = 1;
  while (lanes < n && lanes < 32) lanes *= 2;
  if constexpr (V == 1) lanes = std::max(lanes, 8);
  const int turns = (std::max(p.side[0].heads, p.side[1].heads) * lanes + 31) / 32;
  const long long rows = (long long)p.S * p.N;
  // few rows: as many warps as there are turns of heads share one
  p.share = GRAD ? 1 : (int)std::max<long long>(1, std::min<long long>(turns, kPlanSms * 16 / std::max<long long>(rows, 1)));
  if constexpr (V == 1) {
    switch (lanes) {
      case 8: return launch_form<T, V, 8, 1, GRAD>(p, s);
      case 16: return launch_form<T, V, 16, 1, GRAD>(p, s);
      default: return n <= 32 ? launch_form<T, V, 32, 1, GRAD>(p, s) : launch_form<T, V, 32, 4, GRAD>(p, s);
    }
  } else {
    switch (lanes) {
      case 1: return launch_form<T, V, 1, 1, GRAD>(p, s);
      case 2: return launch_form<T, V, 2, 1, GRAD>(p, s);
      case 4: return launch_form<T, V, 4, 1, GRAD>(p, s);
      case 8: return launch_form<T, V, 8, 1, GRAD>(p, s);
      case 16: return launch_form<T, V, 16, 1, GRAD>(p, s);
      default: return launch_form<T, V, 32, 1, GRAD>(p, s);
    }
  }
}

template <bool GRAD>
cudaError_t launch_any(const QkParams& p, cudaStream_t s) {
  if (p.dtype == RK_F32)
    return p.piece == 4 ? launch_lanes<float, 4, GRAD>(p, s) : launch_lanes<float, 1, GRAD>(p, s);
  if (p.dtype == RK_F16) {
    if (p.piece == 8) return launch_lanes<__half, 8, GRAD>(p, s);
    return p.piece == 4 ? launch_lanes<__half, 4, GRAD>(p, s) : launch_lanes<__half, 1, GRAD>(p, s);
  }
  if (p.piece == 8) return launch_lanes<__nv_bfloat16, 8, GRAD>(p, s);
  return p.piece == 4 ? launch_lanes<__nv_bfloat16, 4, GRAD>(p, s) : launch_lanes<__nv_bfloat16, 1, GRAD>(p, s);
}

}  // namespace

int qk_piece(int eb, int size, int rotary, int interleaved) {
  for (int v = 16 / eb; v >= 4; v /= 2)
    if (interleaved ? size % (2 * v) == 0 : rotary / 2 % v == 0 && (size - rotary) % v == 0) return v;
  return 1;
}

int qk_grad_blocks(long long rows) {
  return (int)std::max<long long>(1, std::min<long long>((rows + kQkWarps - 1) / kQkWarps, kPlanSms * 2));
}

cudaError_t launch_qk(const QkParams& p, cudaStream_t s) { return launch_any<false>(p, s); }

cudaError_t launch_qk_grad(const QkParams& p, cudaStream_t s, int* launches) {
  cudaError_t e = launch_any<true>(p, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.partial == nullptr) return e;
  qk_scale_kernel<<<(2 * p.size + 7) / 8, 256, 0, s>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace rk
