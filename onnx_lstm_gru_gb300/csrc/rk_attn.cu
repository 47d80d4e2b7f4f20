// rk_attn.cu -- attention through a state that decays by head, step by step;
// the decays' gradient and the sums over heads that share.
//
//   H = e^g H + su k v^T,  o = so H^T q          (a pass of rk_attn.h)
#include <algorithm>

#include "rk.h"
#include "rk_attn.h"
#include "rk_ssm_common.cuh"

namespace rk {
namespace {

constexpr int kStepThreads = 256, kMaxHead = 128;

// The recurrence as it stands, forward: a block holds one state, a thread VEC
// columns of some of its rows in registers.  LANES threads hold a row, the
// block's 256 / LANES groups take rows in turn.  Some steps' queries, keys and
// values are fetched together; the outputs are added up over the groups at the
// end.  A single token's time is that of its state, read and written
// once, in pieces of 16 bytes where its rows are whole pieces, past the caches:
// 64 tokens of 16 heads, states of 128 x 128, 28.6 us or 4.7 TB/s (31.7 through
// the caches; 31.3 with three blocks on a multiprocessor instead of two, 33.0
// with half the columns in a block).
template <typename T, int VEC, int LANES>
__global__ void __launch_bounds__(kStepThreads, 2) attn_step_kernel(AttnParams p) {
  constexpr int kGroups = kStepThreads / LANES, kRows = kMaxHead / kGroups, kWide = VEC * LANES;
  constexpr int kStepRows = VEC == 1 ? 16 : 4;
  constexpr int kTogether = 32 / LANES > 0 ? 32 / LANES : 1;  // groups of one warp, added up by exchanges
  constexpr int kParts = kGroups / kTogether;
  __shared__ float sq[kStepRows][kMaxHead], sk[kStepRows][kMaxHead], sd[kStepRows];
  __shared__ __align__(16) float sv[kStepRows][kWide];
  __shared__ __align__(16) float part[kStepRows][kParts][kWide];
  const AttnPass& a = p.pass[0];
  const int blocks = (a.V + kWide - 1) / kWide;
  long long id = blockIdx.x / blocks;
  const int v0 = (int)(blockIdx.x - id * blocks) * kWide;
  const int h = (int)(id % p.H), n = (int)(id / p.H);
  const int group = threadIdx.x / LANES, v = v0 + threadIdx.x % LANES * VEC;
  const bool mine = v < a.V;  // VEC divides V
  const long long state = ((long long)n * p.H + h) * a.K * a.V + v;
  float s[kRows][VEC];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int k = group + i * kGroups;
    fill(s[i], 0.0f);
    if (a.first && mine && k < a.K) {
      Packed<float, VEC> x;
      x.load_streaming(a.first + state + (long long)k * a.V);
      x.widen(s[i]);
    }
  }
  const int L = row_length(p.lens, n, p.S);
  const float bias = p.bias ? p.bias[h] : 0.0f;
  const T* q = static_cast<const T*>(a.q.p) + n * a.q.ns + (long long)(h / a.q_of) * a.K;
  const T* k = static_cast<const T*>(a.k.p) + n * a.k.ns + (long long)(h / a.k_of) * a.K;
  const T* x = static_cast<const T*>(a.v.p) + n * a.v.ns + (long long)(h / a.v_of) * a.V;
  const float* g = static_cast<const float*>(p.decay.p) + n * p.decay.ns + h;
  T* o = static_cast<T*>(a.o.p) + n * a.o.ns + (long long)h * a.V;
#pragma unroll 1
  for (int base = 0; base < L; base += kStepRows) {
    const int rows = min(kStepRows, L - base);
    for (int i = threadIdx.x; i < rows * kMaxHead; i += kStepThreads) {
      const int j = i / kMaxHead, c = i % kMaxHead;
      const long long t = base + j;
      if (c < a.K) sq[j][c] = Elem<T>::to_f(q[t * a.q.ss + c]), sk[j][c] = Elem<T>::to_f(k[t * a.k.ss + c]);
    }
    for (int i = threadIdx.x; i < rows * kWide; i += kStepThreads) {
      const int j = i / kWide, c = v0 + i % kWide;
      sv[j][i % kWide] = c < a.V ? a.su * Elem<T>::to_f(x[(base + j) * a.v.ss + c]) : 0.0f;
    }
    if (threadIdx.x < rows) sd[threadIdx.x] = expf((p.decay.p ? g[(base + threadIdx.x) * p.decay.ss] : 0.0f) + bias);
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < rows; ++j) {
      const float d = sd[j];
      float c[VEC], y[VEC];
      Piece<float, VEC>::load(&sv[j][v - v0], c);
      fill(y, 0.0f);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = group + i * kGroups;
        if (r < a.K) {
          const float kk = sk[j][r], qq = sq[j][r];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            s[i][e] = fmaf(kk, c[e], d * s[i][e]);
            y[e] = fmaf(qq, s[i][e], y[e]);
          }
        }
      }
#pragma unroll
      for (int m = LANES; m < 32; m *= 2)
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] += __shfl_xor_sync(0xffffffffu, y[e], m);
      if (group % kTogether == 0) Piece<float, VEC>::store(&part[j][group / kTogether][v - v0], y);
    }
    __syncthreads();
    if (a.o.p) {
      for (int i = threadIdx.x; i < rows * kWide; i += kStepThreads) {
        const int j = i / kWide, c = i % kWide;
        float y = 0.0f;
#pragma unroll
        for (int e = 0; e < kParts; ++e) y += part[j][e][c];
        if (v0 + c < a.V) o[(base + j) * a.o.ss + v0 + c] = Elem<T>::from_f(a.so * y);
      }
    }
    // no wait: the next rows are read after the first barrier, `part` is written after it
  }
  if (a.o.p)
    for (int t = L + group; t < p.S; t += kGroups)
      if (mine)
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[t * a.o.ss + v + e] = Elem<T>::from_f(0.0f);
  if (a.last && mine) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = group + i * kGroups;
      if (r < a.K) {
        Packed<float, VEC> x;
        x.narrow(s[i]);
        x.store_streaming(a.last + state + (long long)r * a.V);
      }
    }
  }
}

template <typename T>
cudaError_t launch_steps(const AttnParams& p, cudaStream_t s) {
  const AttnPass& a = p.pass[0];
  auto run = [&](auto kernel, int wide) {
    kernel<<<(unsigned)((long long)p.N * p.H * ((a.V + wide - 1) / wide)), kStepThreads, 0, s>>>(p);
    return cudaGetLastError();
  };
  const bool pieces = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.first) % 16 == 0 && reinterpret_cast<uintptr_t>(a.last) % 16 == 0;
  // the same case element by element, a block for 32 columns: 34.8 us, 31.3 in
  // pieces (both through the caches)
  if (!pieces) return run(attn_step_kernel<T, 1, 32>, 32);
  return a.V <= 64 ? run(attn_step_kernel<T, 4, 16>, 64) : run(attn_step_kernel<T, 4, 32>, 128);
}

// A step's decay lies between the steps before it, which wrote the state, and
// those from it on, which read it: its gradient is E = <H, dH>, the product of
// the state before the step with its gradient.  With A_t = q dq and B_t = k dk
// of a step, E grows by B_t - A_t from one step to the next.  The sums run from
// one mark to the next, eight chunks on or one, where E is taken from the states
// themselves, as it is at both ends of the sequence: what the float32 products are
// off by (1e-7 of them) adds up on the way, and a bias' gradient adds that up once
// more.  What they leave at a mark is taken back evenly on the way to it.  Of 500
// cases drawn around those measured dDecay is off by 2.5e-7 of its size in the
// middle and 9e-7 at most, a bias' gradient by 1.4e-7 and 7e-6, where short
// memories leave little of its sum (with marks every eight chunks alone 2.2e-7 and
// 2.4e-5; plain form in float32: 1.8e-7 and 4e-7, 1.6e-7 and 3.1e-6).  A block takes the steps
// between two marks; the sums are pairs of float32 that keep what each addition
// rounds away (Knuth's two-sum), as the card has few float64 units and the kernel
// is a chain of sums, bound by their latency (128 heads of 512 steps 11.8 us with
// float64, 6.7 so).  EVERY: chunks from mark to mark.
constexpr int kDecayThreads = 256, kDecayWarps = kDecayThreads / 32, kDecayEach = 2;
__host__ __device__ constexpr int decay_threads(int every) { return every * 64 / kDecayEach; }
static_assert(decay_threads(kMarkChunks) == kDecayThreads, "a block's steps are those between two marks");
struct Exact {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void add(Exact x) {
    add(x.hi);
    lo += x.lo;
    const float s = hi + lo;  // keeps lo far below hi
    lo -= s - hi;
    hi = s;
  }
  __device__ __forceinline__ float value() const { return hi + lo; }
  __device__ __forceinline__ Exact operator-() const { return {-hi, -lo}; }
};
constexpr Exact kNothing = {0.0f, 0.0f};
// The sum over groups of `lanes` lanes, in each of them the same.
__device__ __forceinline__ Exact pair_sum(Exact x, int lanes) {
#pragma unroll
  for (int o = 1; o < lanes; o <<= 1) {
    const Exact y = {__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
    const bool second = threadIdx.x & o;  // one order for both
    Exact z = second ? y : x;
    z.add(second ? x : y);
    x = z;
  }
  return x;
}
// The running sum over groups of `lanes` lanes.
__device__ __forceinline__ Exact pair_scan(Exact x, int lanes) {
#pragma unroll
  for (int o = 1; o < lanes; o <<= 1) {
    Exact y = {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
    if ((int)(threadIdx.x & (lanes - 1)) >= o) {
      y.add(x);
      x = y;
    }
  }
  return x;
}
// The products of the states at a mark, heads of a block apart.
__global__ void __launch_bounds__(kDecayThreads) attn_mark_kernel(AttnDecayParams p) {
  __shared__ float sums[kDecayWarps];
  previous_done();
  next_may_start();
  const long long all = (long long)gridDim.x * p.deep * 128;
  const float4* x = reinterpret_cast<const float4*>(p.states + (long long)blockIdx.x * p.deep * 128);
  const float4* y = reinterpret_cast<const float4*>(p.states + all + (long long)blockIdx.x * p.deep * 128);
  float e = 0.0f;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < p.deep * 32; i0 += 8 * kDecayThreads) {  // 64 rows at a time
    float4 f[8], g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = x[i0 + i * kDecayThreads], g[i] = y[i0 + i * kDecayThreads];
#pragma unroll
    for (int i = 0; i < 8; ++i) e = fmaf(f[i].x, g[i].x, fmaf(f[i].y, g[i].y, fmaf(f[i].z, g[i].z, fmaf(f[i].w, g[i].w, e))));
  }
  // 32 lanes hold a row of 128: the second head's are the upper ones
  const int together = p.together;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
  const float other = __shfl_xor_sync(0xffffffffu, e, 16);
  if (together == 1) e += other;
  __shared__ float upper[kDecayWarps];
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = e, upper[threadIdx.x / 32] = other;
  __syncthreads();
  const long long group = blockIdx.x / p.marks;
  const int m = (int)(blockIdx.x - group * p.marks), groups = (p.H + together - 1) / together;
  const int n = (int)(group / groups), h = (int)(group - (long long)n * groups) * together + threadIdx.x;
  if (threadIdx.x < together && h < p.H) {
    float z = 0.0f;
    for (int w = 0; w < kDecayWarps; ++w) z += threadIdx.x == 0 ? sums[w] : upper[w];
    p.between[((long long)n * p.H + h) * p.marks + m] = z;
  }
}

template <int EVERY>
__global__ void __launch_bounds__(decay_threads(EVERY)) attn_decay_kernel(AttnDecayParams p) {
  constexpr int kDecayThreads = decay_threads(EVERY), kDecayWarps = kDecayThreads / 32, kDecayTile = EVERY * 64;
  __shared__ Exact sums[2][kDecayWarps];
  previous_done();
  next_may_start();
  const long long head = blockIdx.x / p.tiles;
  const int tile = (int)(blockIdx.x - head * p.tiles), h = (int)(head % p.H), n = (int)(head / p.H);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int L = row_length(p.lens, n, p.S), begin = tile * kDecayTile, end = min(begin + kDecayTile, L), steps = end - begin;
  float* out = static_cast<float*>(p.dDecay.p) + n * p.dDecay.ns + h;
  const float* g = static_cast<const float*>(p.decay.p) + n * p.decay.ns + h;
  const float* to = p.to + head * p.S;
  const float* of = p.of + head * p.S;
  const float bias = p.bias ? p.bias[h] : 0.0f;
  Exact total = kNothing;
  if (steps > 0) {
    const float* between = p.between + head * p.marks;
    const float first = tile > 0 ? between[tile - 1] : p.first ? p.first[head] : 0.0f;
    const float last = end < L ? between[tile] : p.last ? p.last[head] : 0.0f;
    // the thread's own steps, and what comes before each
    const int t0 = begin + threadIdx.x * kDecayEach;
    float d[kDecayEach];
    Exact own[kDecayEach], x = kNothing;
#pragma unroll
    for (int i = 0; i < kDecayEach; ++i) d[i] = t0 + i < end && p.decay.p ? g[(t0 + i) * p.decay.ss] : 0.0f;
#pragma unroll
    for (int i = 0; i < kDecayEach; ++i) {
      own[i] = x;
      if (t0 + i < end) x.add(of[t0 + i]), x.add(-to[t0 + i]);
    }
    const Exact scan = pair_scan(x, 32);
    if (lane == 31) sums[0][warp] = scan;
    __syncthreads();
    const Exact warps = pair_scan(sums[0][lane % kDecayWarps], kDecayWarps);
    auto of_warp = [&](int w) { return Exact{__shfl_sync(0xffffffffu, warps.hi, w), __shfl_sync(0xffffffffu, warps.lo, w)}; };
    Exact left = -of_warp(kDecayWarps - 1), base = of_warp(max(warp - 1, 0));
    if (warp == 0) base = kNothing;
    Exact lanes = {__shfl_up_sync(0xffffffffu, scan.hi, 1), __shfl_up_sync(0xffffffffu, scan.lo, 1)};
    if (lane == 0) lanes = kNothing;
    left.add(last), left.add(-first);
    const float back = left.value() / (float)steps;
    base.add(lanes), base.add(first);
#pragma unroll
    for (int i = 0; i < kDecayEach; ++i) {
      const int t = t0 + i;
      if (t < end) {
        Exact y = base;
        y.add(own[i]), y.add(back * (float)(t - begin));
        // a decay of 0 has no gradient: the factor itself is in it
        const float z = d[i] + bias < -104.0f ? 0.0f : y.value();
        if (p.dDecay.p) out[t * p.dDecay.ss] = z;
        total.add(z);
      }
    }
  }
  if (p.dDecay.p)
    for (int t = begin + threadIdx.x; t < min(begin + kDecayTile, p.S); t += kDecayThreads)
      if (t >= L) out[t * p.dDecay.ss] = 0.0f;
  if (p.partial) {
    total = pair_sum(total, 32);
    if (lane == 0) sums[1][warp] = total;
    __syncthreads();
    total = pair_sum(sums[1][lane % kDecayWarps], kDecayWarps);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = (double)total.hi + (double)total.lo;
  }
}

__global__ void __launch_bounds__(256) attn_decay_bias_kernel(AttnDecayParams p) {
  previous_done();
  next_may_start();
  const int tiles = p.tiles;
  const int h = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (h >= p.H) return;
  double x = 0.0;
  for (long long i = lane; i < (long long)p.N * tiles; i += 32)
    x += p.partial[(i / tiles * p.H + h) * tiles + i % tiles];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0) p.dbias[h] = (float)x;
}

template <typename T>
__global__ void __launch_bounds__(256) attn_share_kernel(AttnShareParams p) {
  previous_done();
  next_may_start();
  const auto& out = p.out[blockIdx.y];
  const int width = p.H / out.of * out.V;
  const long long count = (long long)p.N * p.S * width;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < count; i += (long long)gridDim.x * 256) {
    const long long r = i / width;
    const int c = (int)(i - r * width), head = c / out.V, v = c - head * out.V;
    const int n = (int)(r / p.S), s = (int)(r - (long long)n * p.S);
    const float* x = out.o32 + (r * p.H + (long long)head * out.of) * out.V + v;
    float y = 0.0f;
    for (int j = 0; j < out.of; ++j) y += x[(long long)j * out.V];
    static_cast<T*>(out.o.p)[s * out.o.ss + n * out.o.ns + c] = Elem<T>::from_f(y);
  }
}

}  // namespace

cudaError_t launch_attn_steps(const AttnParams& p, cudaStream_t s, int* launches) {
  const cudaError_t e = p.dtype == RK_F32   ? launch_steps<float>(p, s)
                        : p.dtype == RK_F16 ? launch_steps<__half>(p, s)
                                            : launch_steps<__nv_bfloat16>(p, s);
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_attn_chunks(const AttnParams& p, cudaStream_t s, int* launches) {
  switch (p.dtype) {
    case RK_F32: return launch_attn_chunks_f32(p, s, launches);
    case RK_F16: return launch_attn_chunks_f16(p, s, launches);
    default: return launch_attn_chunks_bf16(p, s, launches);
  }
}

cudaError_t take_attn_status(cudaStream_t s, int* to) {
  int one = 0;
  *to = 0;
  for (auto take : {take_attn_status_f32, take_attn_status_f16, take_attn_status_bf16}) {
    const cudaError_t e = take(s, &one);
    if (e != cudaSuccess) return e;
    *to |= one;
  }
  return cudaSuccess;
}

cudaError_t launch_attn_selftest(int tries, cudaStream_t s, int* launches) {
  for (auto launch : {launch_attn_selftest_f32, launch_attn_selftest_f16, launch_attn_selftest_bf16}) {
    const cudaError_t e = launch(tries, s);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

int attn_together(int key_size, int value_size) { return key_size <= 64 && value_size <= 64 ? 2 : 1; }

namespace {
// States that run side by side.
long long streams_of(long long batch, long long heads, int key_size, int value_size, int passes) {
  const int together = attn_together(key_size, value_size);
  return passes * batch * ((heads + together - 1) / together);
}
}  // namespace

AttnPlan attn_plan(long long seq, long long batch, long long heads, int key_size, int value_size, int passes,
                   bool bias) {
  AttnPlan plan{};
  const long long streams = streams_of(batch, heads, key_size, value_size, passes);
  const long long chunks = (seq + 63) / 64;
  // pieces of two chunks at least, and as many as fit the card together: 4096 x
  // 1 x 16 heads of 128 in eight, 59 us; in sixteen 71, in four 90, whole 189.  More
  // than fit together cost their sums of states and bring nothing (8 x 777 x 10
  // heads, float32, whole 128 us, in two 180; gradient 8 x 512 x 16 135 and 209).
  long long segments = streams > 0 ? std::min(kPlanSms / streams, chunks / 2) : 1;
  segments = std::max<long long>(segments, 1);
  plan.per = (int)((chunks + segments - 1) / segments);
  plan.segments = plan.per > 0 ? (int)((chunks + plan.per - 1) / plan.per) : 1;
  // a gradient's passes contract over keys or values
  plan.deep = std::max(key_size, passes > 1 ? value_size : 0) > 64 ? 128 : 64;
  const long long marks = std::max<long long>(chunks - 1, 0);
  const bool near = bias && 2 * (streams / passes) * marks * plan.deep * 128 * 4 <= kNearMarkBytes;
  plan.every = near ? kNearMarkChunks : kMarkChunks;
  plan.marks = (int)(marks / plan.every);
  return plan;
}

long long attn_plan_scratch(const AttnPlan& plan, long long batch, long long heads, int key_size, int value_size,
                            int passes) {
  if (plan.segments <= 1) return 0;
  const long long streams = streams_of(batch, heads, key_size, value_size, passes);
  return streams * plan.segments * (plan.deep * 128LL + 4);
}

int attn_decay_tiles(long long seq, int every) { return (int)((seq + every * 64 - 1) / (every * 64)); }

cudaError_t launch_attn_decay(AttnDecayParams p, cudaStream_t s, int* launches) {
  p.tiles = attn_decay_tiles(p.S, p.every);
  const long long blocks = (long long)p.N * p.H * p.tiles;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  if (p.marks > 0) {
    const long long at = (long long)p.N * ((p.H + p.together - 1) / p.together) * p.marks;
    if (at > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    e = launch_chained(attn_mark_kernel, (unsigned)at, kDecayThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  e = launch_chained(p.every == kMarkChunks ? attn_decay_kernel<kMarkChunks> : attn_decay_kernel<kNearMarkChunks>,
                     (unsigned)blocks, decay_threads(p.every), 0, s, p);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.dbias == nullptr) return e;
  e = launch_chained(attn_decay_bias_kernel, (unsigned)((p.H + 7) / 8), 256, 0, s, p);
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_attn_share(const AttnShareParams& p, cudaStream_t s, int* launches) {
  long long most = 0;
  for (int i = 0; i < p.count; ++i) most = std::max(most, (long long)p.N * p.S * (p.H / p.out[i].of) * p.out[i].V);
  const dim3 grid((unsigned)std::min<long long>((most + 255) / 256, kPlanSms * 32), p.count);
  const cudaError_t e = launch_chained(p.dtype == RK_F32   ? attn_share_kernel<float>
                                       : p.dtype == RK_F16 ? attn_share_kernel<__half>
                                                           : attn_share_kernel<__nv_bfloat16>,
                                       grid, 256, 0, s, p);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace rk
