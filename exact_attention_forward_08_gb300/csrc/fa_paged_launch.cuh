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

// `early`: the blocks may be placed while the kernel before this one on the stream still runs.
template <typename P>
int paged_start(void (*kernel)(P), const P& p, int grid, int threads, int smem, bool early, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = early ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int DQK, int DV, int NT, bool G16>
int paged_few_launch(const PagedParams& p, int grid, cudaStream_t stream) {
  using Shape = PagedShape<DQK, DV, NT>;
  static bool ready[64] = {};
  auto* kernel = paged_attn_kernel<DQK, DV, NT, G16>;
  const int rc = paged_allow_smem(reinterpret_cast<const void*>(kernel), Shape::kBytes, ready);
  if (rc != FA_OK) return rc;
  return paged_start(kernel, p, grid, Shape::kThreads, Shape::kBytes, false, stream);
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
int paged_many_launch(const PagedParams& shared, const fa_kv_cache& c, int rows, int grid, cudaStream_t stream) {
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
  return paged_start(kernel, p, grid, Shape::kThreads, Shape::kBytes, shared.after != 0, stream);
}

// The kernel for few rows, the one for many, and the merge of what both cut: each may begin before the one in front
// of it has ended, and ends after it.
template <int DQK, int DV>
int paged_launch_pages(const PagedParams& shared, const PagedParts* parts, const fa_kv_cache& c, PagedSplit split,
                       int grid, cudaStream_t stream) {
  PagedMerge m = {};
  PagedParams p = shared;
  if (split.few > 0) {
    p.part = parts[0];
    p.row_least = 1;
    p.row_limit = split.few;
    int rc;
    if (p.page_shift == 4)
      rc = split.few <= 8 ? paged_few_launch<DQK, DV, 1, true>(p, grid, stream)
                          : paged_few_launch<DQK, DV, 2, true>(p, grid, stream);
    else
      rc = split.few <= 8 ? paged_few_launch<DQK, DV, 1, false>(p, grid, stream)
                          : paged_few_launch<DQK, DV, 2, false>(p, grid, stream);
    if (rc != FA_OK) return rc;
    m.set[0].part = parts[0];
    m.set[0].rows = paged_few_rows(split.few);
    m.set[0].pieces = PagedShape<DQK, DV, 1>::kTeams;
    m.set[0].shares = m.set[0].rows / 4;
    m.set[0].blocks = grid * m.set[0].shares;
  }
  if (split.many > 0) {
    p.part = parts[1];
    p.row_least = split.few + 1;
    p.row_limit = split.many;
    p.after = split.few > 0;
    const int rc = paged_many_launch<DQK, DV>(p, c, split.many, grid, stream);
    if (rc != FA_OK) return rc;
    m.set[1].part = parts[1];
    m.set[1].rows = TcShape<DQK, DV>::kRows;
    m.set[1].pieces = 1;
    m.set[1].shares = (split.many + 7) / 8;
    m.set[1].blocks = grid * m.set[1].shares;
  }
  m.o = p.o;
  m.lse = p.lse;
  m.total_q = p.total_q;
  m.heads_q = p.heads_q;
  m.ratio = p.ratio;
  m.cu = p.cu;
  m.batch = p.batch;
  m.max_n = p.max_n;
  const int blocks = m.set[0].blocks + m.set[1].blocks;
  if (p.unpacked) return paged_start(paged_merge_kernel<DV, 4, true>, m, blocks, 256, 0, true, stream);
  if (split.many > 0) return paged_start(paged_merge_kernel<DV, 4, false>, m, blocks, 256, 0, true, stream);
  return paged_start(paged_merge_kernel<DV, 8, false>, m, blocks, 256, 0, true, stream);
}

}  // namespace fa
