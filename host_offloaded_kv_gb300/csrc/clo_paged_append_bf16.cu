// Paged append to bf16 pages.
#include "clo_paged_append.cuh"

namespace clo {

void launch_append_bf16(const AppendParams& a, int head_dim, int64_t blocks, int per, cudaStream_t st) { launch_append_bits<16>(a, head_dim, blocks, per, st); }

}  // namespace clo
