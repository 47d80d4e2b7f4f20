// rk_qk_grad.cu -- the gradient of queries and keys normalised and rotated.
#include "rk_qk.cuh"

namespace rk {
namespace {

// Sums over the blocks, one warp for each element of the two scales.
__global__ void __launch_bounds__(256) qk_scale_kernel(QkParams p) {
  previous_done();
  const int i = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (i >= 2 * p.size) return;
  float* out = i < p.size ? p.side[0].dscale : p.side[1].dscale;
  if (out == nullptr) return;
  float v = 0.0f;
  for (int b = lane; b < p.blocks; b += 32) v += p.partial[(long long)b * 2 * p.size + i];
  v = warp_sum(v);
  if (lane == 0) out[i < p.size ? i : i - p.size] = v;
}

}  // namespace

int qk_grad_blocks(long long rows) {
  return (int)std::max<long long>(1, std::min<long long>((rows + qk::kQkWarps - 1) / qk::kQkWarps, kPlanSms * 2));
}

cudaError_t launch_qk_grad(const QkParams& p, cudaStream_t s, int* launches) {
  cudaError_t e = qk::launch_any<true>(p, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (p.partial == nullptr) return e;
  e = launch_chained(qk_scale_kernel, (unsigned)((2 * p.size + 7) / 8), 256, 0, s, p);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace rk
