// Decode attention over 4-bit pages.
#include "clo_paged_few.cuh"

namespace clo {

cudaError_t launch_attend_few_e2m1(const AttendParams& a, int head_dim, cudaStream_t st) { return few<4>(a, head_dim, nullptr, st); }

int64_t attend_few_e2m1_bytes(const AttendParams& a, int head_dim) {
  int64_t bytes = 0;
  few<4>(a, head_dim, &bytes, nullptr);
  return bytes;
}

}  // namespace clo
