// rk_attn_tc_bf16.cu -- the chunked attention kernels for bfloat16 rows.
#include "rk_attn_tc.cuh"

namespace rk {

cudaError_t launch_attn_chunks_bf16(const AttnParams& p, cudaStream_t s, int* launches) {
  return atc::launch_chunks<__nv_bfloat16>(p, s, launches);
}
cudaError_t take_attn_status_bf16(cudaStream_t s, int* to) { return atc::take_status(s, to); }
cudaError_t launch_attn_selftest_bf16(int tries, cudaStream_t s) { return atc::launch_selftest(tries, s); }

}  // namespace rk
