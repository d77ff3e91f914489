// Host interface between fa_paged_api.cu and the kernels of the paged 8-bit cache.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {

struct PagedParams;

constexpr int kPagedMaxTeams = 8;     // most teams of a block
constexpr int kPagedMaxBlocks = 160;  // most blocks of the attention kernel (one an SM)
// Sequences with at most this many rows (new tokens x query heads a key head)
// are read straight from the pages; longer ones are unpacked first.
constexpr int kPagedRowLimit = 128;

// fa_paged_append.cu
int append_launch(const fa_kv_cache& c, const void* q, const void* k, const void* v, int64_t q_stride,
                  int64_t k_stride, int64_t v_stride, void* q_out, const int* cu, int batch, int64_t total,
                  int heads_q, const float* cos_sin, int max_pos, int rot, int interleaved, unsigned int* status, int sms,
                  cudaStream_t stream);

// fa_paged_d{64,128,192}.cu: the attention kernel and the merge for rows of a
// team 8, 16, 32 or 64; `smem_ready` remembers the shared-memory attribute
int paged_launch_d64(const PagedParams& p, const fa_kv_cache& c, int d_v, int rows, int grid, cudaStream_t stream);
int paged_launch_d128(const PagedParams& p, const fa_kv_cache& c, int d_v, int rows, int grid, cudaStream_t stream);
int paged_launch_d192(const PagedParams& p, const fa_kv_cache& c, int d_v, int rows, int grid, cudaStream_t stream);

// fa_paged_unpack.cu: the codes of the long sequences as bf16 rows, packed, and their offsets
struct UnpackParams {
  const uint8_t* src[2];
  int64_t page_stride[2], head_stride[2], token_stride[2];
  const uint8_t* scale[2];
  uint16_t* dst[2];  // K, V: [total_k, heads_kv, d]
  int* cu_k;         // [batch + 1]
  const int* cu_q;
  const int* seqlens;
  const int* table;
  int64_t table_stride, total_q, total_k;
  unsigned int* status;
  int batch, heads_kv, ratio, num_pages, max_pages, page_shift, max_n, row_limit;
};
int unpack_launch(const UnpackParams& p, int d_qk, int d_v, int sms, cudaStream_t stream);

}  // namespace fa
