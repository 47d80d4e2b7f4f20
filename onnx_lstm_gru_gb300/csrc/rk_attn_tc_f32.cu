// rk_attn_tc_f32.cu -- the chunked attention kernels for float32 rows.
#include "rk_attn_tc.cuh"

namespace rk {

cudaError_t launch_attn_chunks_f32(const AttnParams& p, cudaStream_t s, int* launches) {
  return atc::launch_chunks<float>(p, s, launches);
}
cudaError_t take_attn_status_f32(cudaStream_t s, int* to) { return atc::take_status(s, to); }
cudaError_t launch_attn_selftest_f32(int tries, cudaStream_t s) { return atc::launch_selftest(tries, s); }

}  // namespace rk
