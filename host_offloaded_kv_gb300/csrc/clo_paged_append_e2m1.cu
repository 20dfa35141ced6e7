// Paged append to 4-bit pages.
#include "clo_paged_append.cuh"

namespace clo {

void launch_append_e2m1(const AppendParams& a, int head_dim, int64_t blocks, int per, cudaStream_t st) { launch_append_bits<4>(a, head_dim, blocks, per, st); }

}  // namespace clo
