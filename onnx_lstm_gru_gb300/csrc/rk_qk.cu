// rk_qk.cu -- queries and keys normalised and rotated: forward, and the choice of pieces.
#include "rk_qk.cuh"

namespace rk {

// Interleaved pairs lie in neighbouring pieces; the others' halves and what is
// not rotated have to end with a piece.
int qk_piece(int eb, int size, int rotary, int interleaved) {
  for (int v = 16 / eb; v >= 2; v /= 2)
    if (interleaved ? size % v == 0 : rotary / 2 % v == 0 && (size - rotary) % v == 0) return v;
  return 1;
}

cudaError_t launch_qk(const QkParams& p, cudaStream_t s) { return qk::launch_any<false>(p, s); }

}  // namespace rk
