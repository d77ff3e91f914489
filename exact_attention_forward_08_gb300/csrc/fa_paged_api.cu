// C ABI of the paged 8-bit key/value cache: argument checks, tensor maps,
// workspace layout and launches.  See include/fa.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged.h"
#include "fa_paged_attn.cuh"
#include "fa_paged_check.h"

using namespace fa;

namespace {

constexpr int64_t kMaxListTokens = int64_t(1) << 20;  // each block of the attention over lists looks at all lengths

// Rows of the unpacked keys.  At least one: without any the variable-length
// forward takes all queries for rows without a key, those of no sequence too.
int64_t unpacked_keys(int64_t total_k) { return total_k > 0 ? total_k : 1; }

// The workspace: for each of the two kernels the parts, references and sums, and
// joins of its cut units, then (for calls with long sequences) offsets, unpacked
// keys and values, and the variable-length forward's own workspace.
struct Workspace {
  size_t part_o[2], part_ml[2], joins[2], cu_k, k, v, varlen, varlen_bytes, bytes;
};

Workspace workspace_of(int batch, int heads_q, int heads_kv, int64_t total_q, int max_n, int64_t total_k, int d_qk,
                       int d_v) {
  Workspace w;
  std::memset(&w, 0, sizeof(w));
  const int ratio = heads_q / heads_kv;
  const int64_t rows = static_cast<int64_t>(max_n) * ratio;
  const fa::PagedSplit split = fa::paged_split(rows, ratio, batch, max_n, -1);  // enough for any total_q
  size_t at = 0;
  for (int i = 0; i < 2; ++i) {
    if ((i == 0 ? split.few : split.many) == 0) continue;
    const size_t pieces = static_cast<size_t>(fa::kPagedMaxBlocks) * (i == 0 ? fa::kPagedMaxTeams : 1);
    const size_t part_rows = i == 0 ? fa::paged_few_rows(split.few) : fa::kPagedRowLimit;
    w.part_o[i] = at;
    at += up256(2 * pieces * part_rows * d_v * sizeof(float));
    w.part_ml[i] = at;
    at += up256(2 * pieces * part_rows * sizeof(float2));
    w.joins[i] = at;
    at += up256(pieces * sizeof(fa::PagedJoin));
  }
  if (rows > fa::kPagedRowLimit) {
    w.cu_k = at;
    at += up256((static_cast<size_t>(batch) + 1) * sizeof(int));
    const size_t keys = static_cast<size_t>(unpacked_keys(total_k));
    w.k = at;
    at += up256(keys * heads_kv * d_qk * 2);
    w.v = at;
    at += up256(keys * heads_kv * d_v * 2);
    w.varlen = at;
    w.varlen_bytes = fa_varlen_workspace_size(batch, heads_q, total_q);
    at += up256(w.varlen_bytes);
  }
  w.bytes = at;
  return w;
}

// What the kernels on pages take of the cache and the call alike.
void fill_params(fa::PagedParams& p, const fa_kv_cache& c, const void* q, void* o, float* lse, int64_t total_q,
                 int heads_q, float scale, unsigned int* status) {
  std::memset(&p, 0, sizeof(p));
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.k_page = c.k_stride[0];
  p.k_head = c.k_stride[1];
  p.k_token = static_cast<uint32_t>(c.k_stride[2]);
  p.v_page = c.v_stride[0];
  p.v_head = c.v_stride[1];
  p.v_token = static_cast<uint32_t>(c.v_stride[2]);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.status = status;
  p.total_q = total_q;
  p.heads_q = heads_q;
  p.num_pages = c.num_pages;
  p.page_shift = page_shift(c.page_size);
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
}

// Groups of a key head's query heads whose rows fit a tile of 16, all of one size, so that
// a row's head is a quotient.  Each group reads the pages, so ratios without a divisor near 16
// pay: 64 tokens over 32 pages of 64, one key head of 64: 16 heads 16.0 us, 32 20.0, 48 24.9,
// 64 29.8, but 17 and 34 56 (17 groups), 37 109 (37), 71 205 (71).
int list_groups(int ratio) {
  int groups = (ratio + 15) / 16;
  while (ratio % groups != 0) ++groups;
  return groups;
}

// The workspace of attention over lists: parts, references and sums, joins.
struct ListsWorkspace {
  size_t part_o, part_ml, joins, bytes;
};
ListsWorkspace lists_workspace(int rows, int d_v) {
  ListsWorkspace w;
  const size_t pieces = static_cast<size_t>(fa::kPagedMaxBlocks) * fa::kPagedMaxTeams;
  const size_t part_rows = fa::paged_few_rows(rows);
  w.part_o = 0;
  w.part_ml = w.part_o + up256(2 * pieces * part_rows * d_v * sizeof(float));
  w.joins = w.part_ml + up256(2 * pieces * part_rows * sizeof(float2));
  w.bytes = w.joins + up256(pieces * sizeof(fa::PagedJoin));
  return w;
}

}  // namespace

extern "C" {

int fa_kv_append(const fa_kv_cache* cache, const void* q, const void* k, const void* v, int64_t q_stride,
                 int64_t k_stride, int64_t v_stride, void* q_out, const int* cu_seqlens, int batch, int64_t total,
                 int heads_q, const float* cos_sin, int max_positions, int rot_dim, int interleaved,
                 fa_stream_t stream) {
  int rc = check_cache(cache);
  if (rc != FA_OK) return rc;
  if (batch < 0 || batch > kMaxBatch || total < 0 || total >= (int64_t(1) << 31)) return FA_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > cache->d_qk || rot_dim % 16 != 0) return FA_ERR_INVALID_ARG;
  if (rot_dim > 0 && max_positions < 1) return FA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (q != nullptr && (heads_q < 1 || heads_q % cache->heads_kv != 0)) return FA_ERR_INVALID_ARG;
  if (batch == 0 || total == 0) return FA_OK;
  rc = check_cache_pointers(cache);
  if (rc != FA_OK) return rc;
  if (k == nullptr || v == nullptr || cu_seqlens == nullptr || (rot_dim > 0 && cos_sin == nullptr))
    return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(cos_sin, 16) ||
      !aligned(cu_seqlens, 4))
    return FA_ERR_INVALID_ARG;
  // rows of heads side by side, 16-byte steps from token to token
  const int64_t most = int64_t(1) << 40;
  if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < static_cast<int64_t>(cache->heads_kv) * cache->d_qk ||
      v_stride < static_cast<int64_t>(cache->heads_kv) * cache->d_v || k_stride >= most || v_stride >= most)
    return FA_ERR_INVALID_ARG;
  if (q != nullptr && (q_stride % 8 != 0 || q_stride < static_cast<int64_t>(heads_q) * cache->d_qk || q_stride >= most))
    return FA_ERR_INVALID_ARG;
  // in place only where both rows are the same
  if (q != nullptr && q == q_out && q_stride != static_cast<int64_t>(heads_q) * cache->d_qk) return FA_ERR_INVALID_ARG;

  fa::HostDevice host;
  rc = fa::host_device(&host);
  if (rc != FA_OK) return rc;
  if (!cache_on_device(cache, host.dev) || !fa::host_is_device_ptr(k, host.dev) ||
      !fa::host_is_device_ptr(v, host.dev) || !fa::host_is_device_ptr(cu_seqlens, host.dev) ||
      (q != nullptr && (!fa::host_is_device_ptr(q, host.dev) || !fa::host_is_device_ptr(q_out, host.dev))) ||
      (rot_dim > 0 && !fa::host_is_device_ptr(cos_sin, host.dev)))
    return FA_ERR_INVALID_ARG;
  return fa::append_launch(*cache, q, k, v, q_stride, k_stride, v_stride, q_out, cu_seqlens, batch, total, heads_q,
                           cos_sin, max_positions, rot_dim, interleaved, host.status, host.sms,
                           reinterpret_cast<cudaStream_t>(stream));
}

size_t fa_fwd_paged_workspace_size(int batch, int heads_q, int heads_kv, int64_t total_q, int max_seqlen_q,
                                   int64_t total_k, int d_qk, int d_v) {
  if (batch < 0 || heads_q < 1 || heads_kv < 1 || heads_q % heads_kv != 0 || total_q < 0 || max_seqlen_q < 0 ||
      total_k < 0 || !dims_supported(d_qk, d_v))
    return 0;
  return workspace_of(batch, heads_q, heads_kv, total_q, max_seqlen_q, total_k, d_qk, d_v).bytes;
}

int fa_fwd_paged(const void* q, const fa_kv_cache* cache, void* o, float* lse, const int* cu_seqlens_q, int batch,
                 int64_t total_q, int max_seqlen_q, int64_t total_k, int heads_q, int causal, float scale,
                 void* workspace, size_t workspace_bytes, fa_stream_t stream_) {
  int rc = check_cache(cache);
  if (rc != FA_OK) return rc;
  const fa_kv_cache& c = *cache;
  if (batch < 0 || batch > kMaxBatch || total_q < 0 || total_k < 0 || max_seqlen_q < 0) return FA_ERR_INVALID_ARG;
  if (heads_q < 1 || heads_q % c.heads_kv != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID_ARG;
  if (total_q >= (int64_t(1) << 31)) return FA_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0) return FA_OK;
  if (max_seqlen_q < 1) return FA_ERR_INVALID_ARG;
  const int ratio = heads_q / c.heads_kv;
  const int64_t rows = static_cast<int64_t>(max_seqlen_q) * ratio;
  const bool unpack = rows > fa::kPagedRowLimit;
  // the variable-length forward counts rows in 32 bits
  if (unpack && total_q + total_k + 512 >= (int64_t(1) << 31)) return FA_ERR_INVALID_ARG;
  rc = check_cache_pointers(cache);
  if (rc != FA_OK) return rc;
  if (q == nullptr || o == nullptr || cu_seqlens_q == nullptr || workspace == nullptr) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(workspace, 16) || !aligned(cu_seqlens_q, 4))
    return FA_ERR_INVALID_ARG;
  const Workspace w = workspace_of(batch, heads_q, c.heads_kv, total_q, max_seqlen_q, total_k, c.d_qk, c.d_v);
  if (workspace_bytes < w.bytes) return FA_ERR_INVALID_ARG;
  if (scale == 0.f) scale = 1.0f / std::sqrt(static_cast<float>(c.d_qk));

  fa::HostDevice host;
  rc = fa::host_device(&host);
  if (rc != FA_OK) return rc;
  if (!cache_on_device(cache, host.dev) || !fa::host_is_device_ptr(q, host.dev) ||
      !fa::host_is_device_ptr(o, host.dev) || !fa::host_is_device_ptr(cu_seqlens_q, host.dev) ||
      !fa::host_is_device_ptr(workspace, host.dev) || (lse != nullptr && !fa::host_is_device_ptr(lse, host.dev)))
    return FA_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  if (unpack) {
    fa::UnpackParams u;
    std::memset(&u, 0, sizeof(u));
    for (int i = 0; i < 2; ++i) {
      const int64_t* s = i == 0 ? c.k_stride : c.v_stride;
      u.src[i] = static_cast<const uint8_t*>(i == 0 ? c.k : c.v);
      u.scale[i] = i == 0 ? c.k_scale : c.v_scale;
      u.page_stride[i] = s[0];
      u.head_stride[i] = s[1];
      u.token_stride[i] = s[2];
    }
    u.dst[0] = reinterpret_cast<uint16_t*>(ws + w.k);
    u.dst[1] = reinterpret_cast<uint16_t*>(ws + w.v);
    u.cu_k = reinterpret_cast<int*>(ws + w.cu_k);
    u.cu_q = cu_seqlens_q;
    u.seqlens = c.seqlens_k;
    u.table = c.block_table;
    u.table_stride = c.table_stride;
    u.total_q = total_q;
    u.total_k = total_k;
    u.status = host.status;
    u.batch = batch;
    u.heads_kv = c.heads_kv;
    u.ratio = ratio;
    u.num_pages = c.num_pages;
    u.max_pages = c.max_pages;
    u.page_shift = page_shift(c.page_size);
    u.max_n = max_seqlen_q;
    u.row_limit = fa::kPagedRowLimit;
    rc = fa::unpack_launch(u, c.d_qk, c.d_v, host.sms, stream);
    if (rc != FA_OK) return rc;
    // rows of the short sequences get no keys here and are written below
    rc = fa_fwd_varlen(q, u.dst[0], u.dst[1], o, lse, cu_seqlens_q, u.cu_k, batch, total_q, unpacked_keys(total_k),
                       heads_q, c.heads_kv, c.d_qk, c.d_v, causal, scale, ws + w.varlen, w.varlen_bytes, stream_);
    if (rc != FA_OK) return rc;
  }

  fa::PagedParams p;
  fill_params(p, c, q, o, lse, total_q, heads_q, scale, host.status);
  p.table = c.block_table;
  p.table_stride = c.table_stride;
  p.seqlens = c.seqlens_k;
  p.cu = cu_seqlens_q;
  p.batch = batch;
  p.heads_kv = c.heads_kv;
  p.ratio = ratio;
  p.max_pages = c.max_pages;
  p.causal = causal ? 1 : 0;
  p.timeout_ns = 1000000000ull;
  p.max_n = max_seqlen_q;
  p.unpacked = unpack ? 1 : 0;
  const int grid = host.sms < fa::kPagedMaxBlocks ? host.sms : fa::kPagedMaxBlocks;
  fa::PagedParts parts[2];
  for (int i = 0; i < 2; ++i) {
    parts[i].o = reinterpret_cast<float*>(ws + w.part_o[i]);
    parts[i].ml = reinterpret_cast<float2*>(ws + w.part_ml[i]);
    parts[i].joins = reinterpret_cast<fa::PagedJoin*>(ws + w.joins[i]);
  }
  const fa::PagedSplit split = fa::paged_split(rows, ratio, batch, max_seqlen_q, total_q);
  if (c.d_qk == 64) return fa::paged_launch_d64(p, parts, c, split, grid, stream);
  if (c.d_qk == 128) return fa::paged_launch_d128(p, parts, c, split, grid, stream);
  return fa::paged_launch_d192(p, parts, c, split, grid, stream);
}

size_t fa_fwd_lists_workspace_size(int heads_q, int heads_kv, int d_v) {
  if (heads_q < 1 || heads_kv < 1 || heads_q % heads_kv != 0 || (d_v != 64 && d_v != 128)) return 0;
  const int ratio = heads_q / heads_kv;
  return lists_workspace(ratio / list_groups(ratio), d_v).bytes;
}

int fa_fwd_lists(const void* q, const fa_kv_cache* cache, const int* lists, const int* list_lens, int width, void* o,
                 float* lse, int64_t total_q, int heads_q, float scale, void* workspace, size_t workspace_bytes,
                 fa_stream_t stream_) {
  if (cache == nullptr) return FA_ERR_INVALID_ARG;
  fa_kv_cache c = *cache;
  c.block_table = lists;
  c.seqlens_k = list_lens;
  c.table_stride = c.max_pages = width;
  int rc = check_cache(&c);
  if (rc != FA_OK) return rc;
  if (total_q < 0 || total_q > kMaxListTokens || heads_q < 1 || heads_q % c.heads_kv != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID_ARG;
  if (total_q == 0) return FA_OK;
  rc = check_cache_pointers(&c);
  if (rc != FA_OK) return rc;
  if (q == nullptr || o == nullptr || workspace == nullptr) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(workspace, 16)) return FA_ERR_INVALID_ARG;
  const int ratio = heads_q / c.heads_kv, groups = list_groups(ratio);
  const ListsWorkspace w = lists_workspace(ratio / groups, c.d_v);
  if (workspace_bytes < w.bytes) return FA_ERR_INVALID_ARG;
  if (scale == 0.f) scale = 1.0f / std::sqrt(static_cast<float>(c.d_qk));
  fa::HostDevice host;
  rc = fa::host_device(&host);
  if (rc != FA_OK) return rc;
  if (!cache_on_device(&c, host.dev) || !fa::host_is_device_ptr(q, host.dev) || !fa::host_is_device_ptr(o, host.dev) ||
      !fa::host_is_device_ptr(workspace, host.dev) || (lse != nullptr && !fa::host_is_device_ptr(lse, host.dev)))
    return FA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  fa::PagedParams p;
  fill_params(p, c, q, o, lse, total_q, heads_q, scale, host.status);
  p.lists = lists;
  p.seqlens = list_lens;
  p.lists_heads = c.heads_kv;
  p.groups = groups;
  p.batch = static_cast<int>(total_q);
  p.heads_kv = c.heads_kv * groups;
  p.ratio = ratio / groups;
  p.max_pages = width;
  p.max_n = 1;
  p.part.o = reinterpret_cast<float*>(ws + w.part_o);
  p.part.ml = reinterpret_cast<float2*>(ws + w.part_ml);
  p.part.joins = reinterpret_cast<fa::PagedJoin*>(ws + w.joins);
  const int grid = host.sms < fa::kPagedMaxBlocks ? host.sms : fa::kPagedMaxBlocks;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (c.d_qk == 64) return fa::lists_launch_d64(p, grid, stream);
  if (c.d_qk == 128) return fa::lists_launch_d128(p, c.d_v, grid, stream);
  return fa::lists_launch_d192(p, c.d_v, grid, stream);
}

}  // extern "C"
