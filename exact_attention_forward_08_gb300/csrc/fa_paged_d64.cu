// paged attention kernels, d_qk = 64
#include "fa_paged_launch.cuh"

namespace fa {

int paged_launch_d64(const PagedParams& p, const PagedParts* parts, const fa_kv_cache& c, PagedSplit split, int grid,
                     cudaStream_t stream) {
  if (c.d_v == 64) return paged_launch_pages<64, 64>(p, parts, c, split, grid, stream);
  return FA_ERR_UNSUPPORTED;
}

}  // namespace fa
