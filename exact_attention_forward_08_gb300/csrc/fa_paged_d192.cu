// paged attention kernels, d_qk = 192
#include "fa_paged_launch.cuh"

namespace fa {

int paged_launch_d192(const PagedParams& p, const fa_kv_cache& c, int d_v, int rows, int grid, cudaStream_t stream) {
  if (d_v == 64) return paged_launch_pages<192, 64>(p, c, rows, grid, stream);
  if (d_v == 128) return paged_launch_pages<192, 128>(p, c, rows, grid, stream);
  return FA_ERR_UNSUPPORTED;
}

}  // namespace fa
