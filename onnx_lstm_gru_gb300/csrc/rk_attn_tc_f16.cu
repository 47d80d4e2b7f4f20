// rk_attn_tc_f16.cu -- the chunked attention kernels for Half rows.
#include "rk_attn_tc.cuh"

namespace rk {

cudaError_t launch_attn_chunks_f16(const AttnParams& p, cudaStream_t s, int* launches) {
  return atc::launch_chunks<__half>(p, s, launches);
}
cudaError_t take_attn_status_f16(cudaStream_t s, int* to) { return atc::take_status(s, to); }
cudaError_t launch_attn_selftest_f16(int tries, cudaStream_t s) { return atc::launch_selftest(tries, s); }

}  // namespace rk
