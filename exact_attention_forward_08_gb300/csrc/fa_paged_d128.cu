// paged attention kernels, d_qk = 128
#include "fa_paged_launch.cuh"

namespace fa {

int paged_launch_d128(const PagedParams& p, const PagedParts* parts, const fa_kv_cache& c, PagedSplit split, int grid,
                      cudaStream_t stream) {
  if (c.d_v == 64) return paged_launch_pages<128, 64>(p, parts, c, split, grid, stream);
  if (c.d_v == 128) return paged_launch_pages<128, 128>(p, parts, c, split, grid, stream);
  return FA_ERR_UNSUPPORTED;
}

}  // namespace fa
