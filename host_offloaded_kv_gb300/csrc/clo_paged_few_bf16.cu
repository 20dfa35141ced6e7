// Decode attention over bf16 pages.
#include "clo_paged_few.cuh"

namespace clo {

cudaError_t launch_attend_few_bf16(const AttendParams& a, int head_dim, cudaStream_t st) { return few<16>(a, head_dim, nullptr, st); }

int64_t attend_few_bf16_bytes(const AttendParams& a, int head_dim) {
  int64_t bytes = 0;
  few<16>(a, head_dim, &bytes, nullptr);
  return bytes;
}

}  // namespace clo
