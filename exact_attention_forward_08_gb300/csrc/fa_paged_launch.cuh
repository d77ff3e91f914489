// Launch of one instantiation of the paged attention kernel and its merge.
#pragma once
#include <mutex>

#include "fa_host.h"
#include "fa_paged.h"
#include "fa_paged_attn.cuh"
#include "fa_paged_tc.cuh"

namespace fa {

// Lets `kernel` use `smem` bytes of dynamic shared memory, once a device.
inline int paged_allow_smem(const void* kernel, int smem, bool (&ready)[64]) {
  static std::mutex mutex;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mutex);
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return FA_ERR_CUDA;
    ready[dev] = true;
  }
  return FA_OK;
}

// The merge's blocks may be placed while the attention kernel still runs; they wait for its end.
template <int DV, int ROWS>
int paged_merge_launch(const PagedParams& p, int rows, int pieces, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pieces, (rows + 7) / 8, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<DV, ROWS>, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int DQK, int DV, int NT, bool G16>
int paged_launch(const PagedParams& p, int grid, cudaStream_t stream) {
  using Shape = PagedShape<DQK, DV, NT>;
  static bool ready[64] = {};
  auto* kernel = paged_attn_kernel<DQK, DV, NT, G16>;
  const int rc = paged_allow_smem(reinterpret_cast<const void*>(kernel), Shape::kBytes, ready);
  if (rc != FA_OK) return rc;
  kernel<<<grid, Shape::kThreads, Shape::kBytes, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  return paged_merge_launch<DV, Shape::kRows>(p, Shape::kRows, grid * Shape::kTeams, stream);
}

// Codes viewed as (d, token, head, page); a box is a page of one head, `columns` wide.
inline int paged_encode(CUtensorMap* m, const void* base, const int64_t* s, const fa_kv_cache& c, int d, int columns) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(c.page_size),
                            static_cast<uint64_t>(c.heads_kv), static_cast<uint64_t>(c.num_pages)};
  // the stride of a dimension of extent 1 is never used, but has to be one
  const uint64_t token = s[2], head = c.heads_kv > 1 ? s[1] : token, page = c.num_pages > 1 ? s[0] : token;
  const uint64_t strides[3] = {token, head, page};
  const uint32_t box[4] = {static_cast<uint32_t>(columns), static_cast<uint32_t>(c.page_size), 1, 1};
  return host_encode_bytes(m, base, 4, dims, strides, box, columns);
}

template <int DQK, int DV>
int paged_tc_launch(const PagedParams& shared, const fa_kv_cache& c, int rows, int grid, cudaStream_t stream) {
  using Shape = TcShape<DQK, DV>;
  static bool ready[64] = {};
  auto* kernel = paged_tc_kernel<DQK, DV>;
  int rc = paged_allow_smem(reinterpret_cast<const void*>(kernel), Shape::kBytes, ready);
  if (rc != FA_OK) return rc;
  TcParams p;
  static_cast<PagedParams&>(p) = shared;
  p.copy_shift = rows <= 32 ? 2 : rows <= 64 ? 1 : 0;
  rc = paged_encode(&p.tm_k, c.k, c.k_stride, c, DQK, DQK == 128 ? 128 : 64);
  if (rc == FA_OK) rc = paged_encode(&p.tm_v, c.v, c.v_stride, c, DV, DV);
  if (rc != FA_OK) return rc;
  kernel<<<grid, Shape::kThreads, Shape::kBytes, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  return paged_merge_launch<DV, Shape::kRows>(p, rows, grid, stream);
}

// rows: the most that a sequence has
template <int DQK, int DV, bool G16>
int paged_launch_rows(const PagedParams& p, const fa_kv_cache& c, int rows, int grid, cudaStream_t stream) {
  if (rows <= 8) return paged_launch<DQK, DV, 1, G16>(p, grid, stream);
  if (rows <= 16) return paged_launch<DQK, DV, 2, G16>(p, grid, stream);
  return paged_tc_launch<DQK, DV>(p, c, rows, grid, stream);
}

template <int DQK, int DV>
int paged_launch_pages(const PagedParams& p, const fa_kv_cache& c, int rows, int grid, cudaStream_t stream) {
  return p.page_shift == 4 ? paged_launch_rows<DQK, DV, true>(p, c, rows, grid, stream)
                           : paged_launch_rows<DQK, DV, false>(p, c, rows, grid, stream);
}

}  // namespace fa
