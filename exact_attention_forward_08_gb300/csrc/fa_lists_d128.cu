// attention over lists of pages, d_qk = 128
#include "fa_paged_launch.cuh"

namespace fa {

int lists_launch_d128(const PagedParams& p, int d_v, int grid, cudaStream_t stream) {
  if (d_v == 64) return paged_launch_lists<128, 64>(p, grid, stream);
  return paged_launch_lists<128, 128>(p, grid, stream);
}

}  // namespace fa
