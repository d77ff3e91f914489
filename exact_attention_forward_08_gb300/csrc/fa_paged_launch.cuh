// Launch of one instantiation of the paged attention kernel and its merge.
#pragma once
#include <mutex>

#include "fa_paged.h"
#include "fa_paged_attn.cuh"

namespace fa {

template <int DQK, int DV, int NT, int TW, bool G16>
int paged_launch(const PagedParams& p, int grid, cudaStream_t stream) {
  using Shape = PagedShape<DQK, DV, NT, TW>;
  static std::mutex mutex;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(paged_attn_kernel<DQK, DV, NT, TW, G16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Shape::kBytes) != cudaSuccess)
        return FA_ERR_CUDA;
      ready[dev] = true;
    }
  }
  paged_attn_kernel<DQK, DV, NT, TW, G16><<<grid, Shape::kThreads, Shape::kBytes, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  // the merge's blocks may be placed while the attention kernel still runs; they wait for its end
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * Shape::kTeams, Shape::kRows / 8, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_merge_kernel<DV, Shape::kRows>, p) != cudaSuccess) return FA_ERR_CUDA;
  return FA_OK;
}

// rows of a team: the smallest build that holds a sequence's rows, at most 64.
template <int DQK, int DV, bool G16>
int paged_launch_rows(const PagedParams& p, int rows, int grid, cudaStream_t stream) {
  if (rows <= 8) return paged_launch<DQK, DV, 1, 1, G16>(p, grid, stream);
  if (rows <= 16) return paged_launch<DQK, DV, 2, 1, G16>(p, grid, stream);
  if (rows <= 32) return paged_launch<DQK, DV, 2, 2, G16>(p, grid, stream);
  return paged_launch<DQK, DV, 2, 4, G16>(p, grid, stream);
}

template <int DQK, int DV>
int paged_launch_pages(const PagedParams& p, int rows, int grid, cudaStream_t stream) {
  return p.page_shift == 4 ? paged_launch_rows<DQK, DV, true>(p, rows, grid, stream)
                           : paged_launch_rows<DQK, DV, false>(p, rows, grid, stream);
}

}  // namespace fa
