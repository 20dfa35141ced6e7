// Decode attention over 8-bit pages.
#include "clo_paged_few.cuh"

namespace clo {

cudaError_t launch_attend_few_e4m3(const AttendParams& a, int head_dim, cudaStream_t st) { return few<8>(a, head_dim, nullptr, st); }

int64_t attend_few_e4m3_bytes(const AttendParams& a, int head_dim) {
  int64_t bytes = 0;
  few<8>(a, head_dim, &bytes, nullptr);
  return bytes;
}

}  // namespace clo
