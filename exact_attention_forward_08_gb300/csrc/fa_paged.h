// Host interface between fa_paged_api.cu and the kernels of the paged 8-bit cache.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {

struct PagedParams;
struct PagedJoin;

constexpr int kPagedMaxTeams = 8;     // most teams of a block
constexpr int kPagedMaxBlocks = 160;  // most blocks of an attention kernel (one an SM)
// Sequences with at most this many rows (new tokens x query heads a key head)
// are read straight from the pages; longer ones are unpacked first.  16 x 32 new
// tokens of 32/8 heads of 128 over 4000 keys: 87 us from the pages, 146 unpacked
// (over 500 keys 35 and 41; 16 heads of 64, 128 tokens: 142 and 173).
constexpr int kPagedRowLimit = 128;

// The most rows of the sequences that each of the two kernels on pages takes
// (0: not launched): paged_attn_kernel for few rows, paged_tc_kernel for more.
// With 32 sequences of 32767 keys and 2 heads of 128, 16 rows take 120 us in the
// first and 153 in the second (8 rows of 8 heads: 95 and 151; 16 heads of 64:
// 123 and 367), 24 rows and more only the second can.  A ragged batch that may
// hold both kinds gets both kernels, at about 5 us; where all sequences have
// max_n tokens, or one token is more than 8 rows already, one is enough.
struct PagedSplit {
  int few, many;
};
inline PagedSplit paged_split(int64_t rows, int ratio, int batch, int max_n, int64_t total_q) {
  if (rows <= 16) return {static_cast<int>(rows), 0};
  const int many = static_cast<int>(rows < kPagedRowLimit ? rows : kPagedRowLimit);
  return {ratio > 8 || static_cast<int64_t>(batch) * max_n == total_q ? 0 : 8, many};
}
// rows that the parts of cut units are laid out for
constexpr int paged_few_rows(int few) { return few <= 8 ? 8 : 16; }

// Where a kernel leaves the parts of its cut units.
struct PagedParts {
  float* o;          // [2 * pieces][rows][d_v]
  float2* ml;        // [2 * pieces][rows] {reference, sum}
  PagedJoin* joins;  // [pieces]
};

// fa_paged_append.cu
int append_launch(const fa_kv_cache& c, const void* q, const void* k, const void* v, int64_t q_stride,
                  int64_t k_stride, int64_t v_stride, void* q_out, const int* cu, int batch, int64_t total,
                  int heads_q, const float* cos_sin, int max_pos, int rot, int interleaved, unsigned int* status, int sms,
                  cudaStream_t stream);

// fa_paged_d{64,128,192}.cu: the attention kernels and the merge; parts[0] is for the few rows, parts[1] for the many
int paged_launch_d64(const PagedParams& p, const PagedParts* parts, const fa_kv_cache& c, PagedSplit split, int grid,
                     cudaStream_t stream);
int paged_launch_d128(const PagedParams& p, const PagedParts* parts, const fa_kv_cache& c, PagedSplit split, int grid,
                      cudaStream_t stream);
int paged_launch_d192(const PagedParams& p, const PagedParts* parts, const fa_kv_cache& c, PagedSplit split, int grid,
                      cudaStream_t stream);

// fa_lists_d{64,128,192}.cu: attention over lists of pages and the merge
int lists_launch_d64(const PagedParams& p, int grid, cudaStream_t stream);
int lists_launch_d128(const PagedParams& p, int d_v, int grid, cudaStream_t stream);
int lists_launch_d192(const PagedParams& p, int d_v, int grid, cudaStream_t stream);

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
