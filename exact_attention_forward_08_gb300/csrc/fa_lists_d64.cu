// attention over lists of pages, d_qk = 64
#include "fa_paged_launch.cuh"

namespace fa {

int lists_launch_d64(const PagedParams& p, int grid, cudaStream_t stream) {
  return paged_launch_lists<64, 64>(p, grid, stream);
}

}  // namespace fa
