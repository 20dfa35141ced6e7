// Decode attention over bf16 pages.
#include "clo_paged_few.cuh"

namespace clo {

cudaError_t launch_attend_few_bf16(const AttendParams& a, int head_dim, int rows, cudaStream_t st) {
  if (head_dim == 128) {
    if (rows <= 8) return launch_few_rows<128, 16, 1>(a, st);
    return rows <= 16 ? launch_few_rows<128, 16, 2>(a, st) : launch_few_rows<128, 16, 4>(a, st);
  }
  if (rows <= 8) return launch_few_rows<64, 16, 1>(a, st);
  return rows <= 16 ? launch_few_rows<64, 16, 2>(a, st) : launch_few_rows<64, 16, 4>(a, st);
}

}  // namespace clo
