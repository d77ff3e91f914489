// fa_kv_fork and fa_kv_compact: which rows of a block table use which pages of
// the 8-bit cache, decided on the device.
//
// Both are integer work on a few thousand numbers with several steps that each
// need all of the step before, and after that copies of whole or part pages.
// The steps run in one cluster of 8 blocks, whose barrier takes less time than a
// launch; the copies in a second kernel over the whole GPU, which is placed while
// the first still runs.
//
// Every result is determined by the inputs alone: sums by atomics are of
// integers, a parent's first heir is found as a minimum, pages are numbered by
// scans in order of rows and of pages.
//
// Bound by latency, but for large copies.  GPU time: 64 beams over one another's
// rows of 624 to 2554 tokens, 854 pages, 19 partly filled ones copied, 12.5 us; 256
// requests in 14613 pages, a tenth of which changes, 13.1 us; 64 rows of 2000 tokens
// 10.5 us, 12.3 if a holder beside the table has each row's last page, and 39.1 and
// 40.8 with rows of 131000 tokens, whose tables the eight blocks write; compaction of 1042 pages
// among 1147 of 16 tokens 8.3 us, of 1910 among 3821 of 64 tokens, 257 MB read and
// written, 50.0 us: 8 for the steps, 38 for the copies, 6.8 TB/s.  In a pool of a
// million pages 68 and 52 us.
#include <cuda_runtime.h>

#include <climits>
#include <cstring>
#include <initializer_list>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged.cuh"
#include "fa_paged_check.h"

namespace fa {
namespace {

constexpr int kCluster = 8;     // blocks that decide
constexpr int kThreads = 1024;  // of each
constexpr int kAll = kCluster * kThreads;

struct PagesHead {
  int copies;  // pages to copy
  int skip;    // where their list begins
  int count[kCluster];
};

struct PagesParams {
  const int* table;
  int64_t table_stride;
  const int* seqlens;
  const int* refs;
  const int* parents;
  const int* grow;
  int* table_out;
  int64_t out_stride;
  int* seqlens_out;
  int* refs_out;
  int* page_map;
  int* used;
  unsigned int* status;
  PagesHead* head;
  int* valid;               // [batch] 0: a row whose length or pages are out of range; 2: its last page is not full and
                            // has other uses; 1: any other
  int* owner;               // [num_pages] of such pages, the first of the new rows that would keep it
  int *src, *dst, *tokens;  // copies
  int batch, rows, num_pages, max_pages, page_shift;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive scan over the block's threads; `total` is the sum.  All threads call.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sum, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  long long w = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0);
}

// The pages that a warp of block `rank` counts, 32 at a time: equal runs in order.
struct PageRun {
  int64_t begin, end;
};
__device__ __forceinline__ PageRun page_run(const PagesParams& p, int rank) {
  const int64_t per = (p.num_pages + kAll - 1) / kAll * 32;
  const int64_t begin = (static_cast<int64_t>(rank) * (kThreads / 32) + (threadIdx.x >> 5)) * per;
  const int64_t end = begin + per;
  return {begin < p.num_pages ? begin : p.num_pages, end < p.num_pages ? end : p.num_pages};
}

// How many pages of the warp's run, and of all runs, `counts` holds for; `before` are those of the runs before.
template <class F>
__device__ __forceinline__ int cluster_count(const PagesParams& p, int rank, const PageRun& run, F counts,
                                             long long* warp_sum, long long& before) {
  const int lane = threadIdx.x & 31;
  int mine = 0;
#pragma unroll 4
  for (int64_t i = run.begin + lane; i < run.end; i += 32) mine += counts(i);
  mine = __reduce_add_sync(0xffffffffu, mine);
  long long total;
  before = block_scan(lane == 0 ? mine : 0, warp_sum, total) - (lane == 0 ? mine : 0);
  before = __shfl_sync(0xffffffffu, before, 0);
  if (threadIdx.x == 0) p.head->count[rank] = static_cast<int>(total);
  cluster_sync();
  int all = 0;
#pragma unroll
  for (int i = 0; i < kCluster; ++i) {
    const int n = __ldcg(&p.head->count[i]);
    if (i < rank) before += n;
    all += n;
  }
  return all;
}

__device__ __forceinline__ bool length_fits(const PagesParams& p, int len) {
  return len >= 0 && len <= static_cast<int64_t>(p.max_pages) << p.page_shift;
}

// A row of the new table as far as it does not depend on other rows.
struct ForkRow {
  int src, len, grow;  // parent (-1: none), its tokens; new tokens (0 if not known)
  bool bad;
  bool shared;         // the parent's last page is not full and has other uses (false if not known)
  __device__ __forceinline__ uint64_t pack() const {  // without the new tokens
    return static_cast<uint64_t>(src + 1) | static_cast<uint64_t>(len) << 16 | static_cast<uint64_t>(bad) << 63;
  }
  static __device__ __forceinline__ ForkRow unpack(uint64_t x) {
    return {static_cast<int>(x & 0xffff) - 1, static_cast<int>(x >> 16 & 0x7fffffff), 0, (x >> 63) != 0, false};
  }
};
__device__ __forceinline__ ForkRow fork_row(const PagesParams& p, int r) {
  ForkRow w = {p.parents[r], 0, p.grow != nullptr ? p.grow[r] : 0, false, false};
  w.bad = w.src < -1 || w.src >= p.batch || w.grow < 0;
  if (!w.bad && w.src >= 0) {
    const int valid = __ldcg(p.valid + w.src), len = p.seqlens[w.src];
    w.bad = valid == 0;
    w.shared = valid == 2;
    w.len = w.bad ? 0 : len;
  }
  w.bad = w.bad || static_cast<int64_t>(w.len) + w.grow > static_cast<int64_t>(p.max_pages) << p.page_shift;
  return w.bad ? ForkRow{-1, 0, 0, true, false} : w;
}

constexpr int kSharedHeir = 1 << 30;  // among a row's heirs: its last page is not full and has other uses

// Three barriers of the cluster, two more where a last page that is not full has uses beside its row.  What all rows need of one another (heirs, first
// heirs, the pages needed before each row) every block works out for itself in
// shared memory, which takes less time than an exchange; pages are shared out.  Rows
// are kept there once they are known (CACHED), as far as they fit: 12.3 us for 64
// beams, 14.1 if they are worked out again in each step.
template <bool CACHED>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    kv_fork_kernel(const __grid_constant__ PagesParams p) {
  extern __shared__ int fork_smem[];
  int* const heirs = fork_smem;          // [batch]
  int* const first = heirs + p.batch;    // [batch] the heir that keeps a last page that is not full, -1: none does
  int* const start = first + p.batch;    // [rows + 1] pages that the rows before need
  uint64_t* const known = reinterpret_cast<uint64_t*>(fork_smem + ((2 * p.batch + p.rows + 2) & ~1));  // [rows]
  auto row_of = [&](int r) { return CACHED ? ForkRow::unpack(known[r]) : fork_row(p, r); };
  __shared__ long long warp_sum[32];
  const int rank = blockIdx.x, tid = rank * kThreads + threadIdx.x;
  const int lane = threadIdx.x & 31, warp = tid >> 5;
  const int part_mask = (1 << p.page_shift) - 1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- counts start from the old ones; a warp looks at an old row's pages ----
  if (tid == 0) p.head->copies = p.head->skip = 0;
  for (int b = warp; b < p.batch; b += kAll / 32) {
    const int* row = p.table + b * p.table_stride;
    const int head = lane < p.max_pages ? row[lane] : 0;  // before the length is known
    const int len = p.seqlens[b];
    const bool fits = length_fits(p, len);
    const int pages = fits ? (len + part_mask) >> p.page_shift : 0;
    bool page_bad = lane < pages && (head < 0 || head >= p.num_pages);
    for (int j = lane + 32; j < pages; j += 32) page_bad |= row[j] < 0 || row[j] >= p.num_pages;
    page_bad = __any_sync(0xffffffffu, page_bad);
    if (lane == 0 && (!fits || page_bad)) paged_error(p.status, fits ? kSitePagedPage : kSitePagedSeq, b);
    int valid = fits && !page_bad ? 1 : 0;
    if (valid != 0 && (len & part_mask) != 0) {
      const int last = pages - 1;
      const int page = last < 32 ? __shfl_sync(0xffffffffu, head, last) : row[last];
      if (p.refs[page] > 1) {
        valid = 2;
        if (lane == 0) p.owner[page] = INT_MAX;
      }
    }
    if (lane == 0) p.valid[b] = valid;
  }
  for (int i = tid; i < p.num_pages; i += kAll) p.refs_out[i] = p.refs[i];
  for (int b = threadIdx.x; b < p.batch; b += kThreads) heirs[b] = 0, first[b] = INT_MAX;
  cluster_sync();

  // ---- heirs ----
  bool shares = false;
  for (int r = threadIdx.x; r < p.rows; r += kThreads) {
    const ForkRow w = fork_row(p, r);
    if constexpr (CACHED) known[r] = w.pack();
    if (rank == 0) {
      p.seqlens_out[r] = w.len + w.grow;
      if (w.bad) paged_error(p.status, kSitePagedSeq, r);
    }
    if (w.src >= 0) {
      atomicAdd(heirs + w.src, 1);
      atomicMin(first + w.src, r);
      if (w.shared) atomicOr(heirs + w.src, kSharedHeir), shares = true;
    }
  }
  shares = __syncthreads_or(shares) != 0;  // the same in all blocks

  // ---- what the old rows' heirs make of their pages' counts ----
  for (int b = warp; b < p.batch; b += kAll / 32) {
    const int n = heirs[b] & ~kSharedHeir;
    if (heirs[b] == 1) continue;
    const int valid = __ldcg(p.valid + b);
    if (valid == 0) continue;
    const int len = p.seqlens[b], full = len >> p.page_shift;
    const int* row = p.table + b * p.table_stride;
    for (int j = lane; n != 1 && j < full; j += 32) atomicAdd(p.refs_out + row[j], n - 1);
    if ((len & part_mask) != 0 && lane == 0) {
      if (n == 0 || valid == 2) atomicAdd(p.refs_out + row[full], -1);
      if (n > 0 && valid == 2) atomicMin(p.owner + row[full], first[b]);
    }
  }
  if (shares) {
    // ---- a last page that is not full and had other uses: kept by the first heir of all its rows, if no use is left ----
    cluster_sync();
    auto last_page = [&](int b) { return p.table[b * p.table_stride + (p.seqlens[b] >> p.page_shift)]; };
    for (int b = threadIdx.x; b < p.batch; b += kThreads)
      if ((heirs[b] & kSharedHeir) != 0) {
        const int page = last_page(b);
        if (__ldcg(p.refs_out + page) > 0 || __ldcg(p.owner + page) != first[b]) first[b] = -1;
      }
    cluster_sync();  // all blocks have read the counts
    if (rank == 0)
      for (int b = threadIdx.x; b < p.batch; b += kThreads)
        if ((heirs[b] & kSharedHeir) != 0 && first[b] >= 0) atomicAdd(p.refs_out + last_page(b), 1);
  }

  // ---- the pages that rows need ----
  auto copies = [&](const ForkRow& w, int r) { return w.src >= 0 && (w.len & part_mask) != 0 && first[w.src] != r; };
  auto kept_pages = [&](const ForkRow& w, int r) {  // that come from the parent
    return (w.len >> p.page_shift) + ((w.len & part_mask) != 0 && !copies(w, r) ? 1 : 0);
  };
  long long needed = 0;
  for (int base = 0; base < p.rows; base += kThreads) {
    const int r = base + threadIdx.x;
    int need = 0;
    if (r < p.rows) {
      const ForkRow w = row_of(r);
      const int64_t len = w.bad ? 0 : static_cast<int64_t>(w.len) + (p.grow != nullptr ? p.grow[r] : 0);
      need = static_cast<int>((len + part_mask) >> p.page_shift) - kept_pages(w, r);
    }
    long long total;
    const long long upto = needed + block_scan(need, warp_sum, total);
    if (r < p.rows) start[r + 1] = static_cast<int>(upto < INT_MAX ? upto : INT_MAX);
    needed += total;
  }
  if (threadIdx.x == 0) start[0] = 0;

  cluster_sync();

  // ---- the lowest free pages go to the rows in order ----
  const PageRun run = page_run(p, rank);
  auto is_free = [&](int64_t i) { return __ldcg(p.refs_out + i) <= 0; };
  long long at;
  const int free_pages = cluster_count(p, rank, run, is_free, warp_sum, at);
  for (int64_t i0 = run.begin; i0 < run.end && at < needed; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool mine = i < run.end && is_free(i);
    const uint32_t mask = __ballot_sync(0xffffffffu, mine);
    const long long rank_of = at + __popc(mask & ((1u << lane) - 1));
    at += __popc(mask);
    if (!mine || rank_of >= needed) continue;
    const int page = static_cast<int>(i), place = static_cast<int>(rank_of);
    int lo = 0, hi = p.rows - 1;  // the last row that starts at `place` or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= place) lo = mid;
      else hi = mid - 1;
    }
    if (start[lo + 1] > free_pages) continue;  // too few for the row
    const ForkRow w = row_of(lo);
    const bool copy = copies(w, lo);
    const int kept = kept_pages(w, lo), j = kept + place - start[lo];
    if (j >= p.max_pages) continue;  // only where inputs change while they are read
    p.table_out[lo * p.out_stride + j] = page;
    p.refs_out[page] = 1;
    if (copy && j == kept) {
      const int c = atomicAdd(&p.head->copies, 1);  // in any order: they are independent
      p.src[c] = p.table[w.src * p.table_stride + kept];
      p.dst[c] = page;
      p.tokens[c] = w.len & part_mask;
    }
  }
  const bool some_fail = needed > free_pages;
  if (some_fail) cluster_sync();  // counts are lowered below, above they have been read

  // ---- a warp writes the rest of a row ----
  for (int r = warp; r < p.rows; r += kAll / 32) {
    const ForkRow w = row_of(r);
    const int kept = kept_pages(w, r), total = kept + (start[r + 1] - start[r]);
    // needs that sum to more than fits are held at the most that does
    const bool needs = start[r + 1] > start[r] ||
                       (start[r + 1] == INT_MAX && static_cast<int64_t>(w.len) + (p.grow != nullptr ? p.grow[r] : 0) >
                                                       static_cast<int64_t>(kept) << p.page_shift);
    const bool fails = needs && start[r + 1] > free_pages;
    const int* row = p.table + (w.src >= 0 ? w.src : 0) * p.table_stride;
    int* out = p.table_out + r * p.out_stride;
    if (fails && lane == 0) {
      p.seqlens_out[r] = 0;
      if (start[r] <= free_pages) paged_error(p.status, kSitePagedFull, r);
    }
    for (int j = lane; j < p.max_pages; j += 32) {
      if (j < kept && !fails) out[j] = row[j];
      else if (j >= total || fails) out[j] = -1;
      // a row without enough pages gives back what it shares, and a page that is partly filled if it keeps one
      if (j < kept && fails && (j < w.len >> p.page_shift || first[w.src] == r)) atomicAdd(p.refs_out + row[j], -1);
    }
  }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    kv_compact_kernel(const __grid_constant__ PagesParams p) {
  __shared__ long long warp_sum[32];
  const int rank = blockIdx.x, tid = rank * kThreads + threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- pages in use: how many, and before each page ----
  const PageRun run = page_run(p, rank);
  const int lane = threadIdx.x & 31;
  long long at;
  const int used = cluster_count(p, rank, run, [&](int64_t i) { return p.refs[i] > 0; }, warp_sum, at);
  if (tid == 0) {
    p.used[0] = used;
    if (used == p.num_pages) p.head->skip = used;
  }
  // ---- pages behind go to the holes before, both in order; the k-th page in use stands at src[k] if it is behind ----
  for (int64_t i0 = run.begin; i0 < run.end; i0 += 32) {
    const int64_t i = i0 + lane;
    const int n = i < run.end ? p.refs[i] : 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, n > 0);
    const int before = static_cast<int>(at) + __popc(mask & ((1u << lane) - 1));  // pages in use before this one
    at += __popc(mask);
    if (i >= run.end) continue;
    if (i == used) p.head->skip = before;  // pages in use that stay
    if (i < used) {
      if (n > 0) p.refs_out[i] = n;
      else p.dst[i - before] = static_cast<int>(i);
    } else if (n > 0) {
      p.src[before] = static_cast<int>(i);
    } else {
      p.refs_out[i] = 0;
    }
    p.page_map[i] = n > 0 ? static_cast<int>(i) : -1;
  }
  cluster_sync();
  const int skip = __ldcg(&p.head->skip), moves = used - skip;
  for (int i = tid; i < moves; i += kAll) {
    const int from = __ldcg(p.src + skip + i), to = __ldcg(p.dst + i);
    const int n = p.refs[from];
    p.refs_out[to] = n;
    p.refs_out[from] = 0;
    p.page_map[from] = to;
  }
  if (tid == 0) p.head->copies = moves;
}

// The table follows the pages: a warp rewrites a row.
__device__ __forceinline__ void compact_row(const PagesParams& p, int b) {
  const int lane = threadIdx.x & 31;
  const int len = p.seqlens[b];
  const bool fits = length_fits(p, len);
  const int pages = fits ? static_cast<int>((static_cast<int64_t>(len) + (1 << p.page_shift) - 1) >> p.page_shift) : 0;
  const int* row = p.table + b * p.table_stride;
  int* out = p.table_out + b * p.out_stride;
  if (!fits && lane == 0) paged_error(p.status, kSitePagedSeq, b);
  for (int j = lane; j < p.max_pages; j += 32) {
    int page = -1;
    if (j < pages) {
      page = row[j];
      page = page >= 0 && page < p.num_pages ? p.page_map[page] : -1;
      if (page < 0) paged_error(p.status, kSitePagedPage, b);
    }
    out[j] = page;
  }
}

struct CopyParams {
  uint8_t* base[2];
  int64_t page_stride[2], head_stride[2];
  uint32_t token_stride[2];
  uint8_t* scale[2];
  uint8_t* bounds;
  const PagesHead* head;
  const int *src, *dst, *tokens;  // tokens: of each copy, unless all of a page
  int heads, page;
  PagesParams table;  // whose rows follow (WHOLE)
};

constexpr int kCopyWarps = 8;   // of a block
// of an SM; us with 2 / 3 / 4: compaction of 1910 pages 48.6 / 49.7 / 49.8, of 1042 small ones 8.7 / 8.7 / 7.9
constexpr int kCopyBlocks = 4;
constexpr int kCopyAhead = 8;   // 16-byte loads of a lane under way

// The first `tokens` tokens of one head's D codes by a warp, in columns of 128 or 64 bytes.
template <int D>
__device__ __forceinline__ void copy_codes(const uint8_t* src, uint8_t* dst, uint32_t ts, int tokens) {
  constexpr int kChunks = D == 128 ? 8 : 4, kRows = 32 / kChunks;
  const int lane = threadIdx.x & 31;
  const uint32_t step = kRows * ts;
#pragma unroll 1
  for (int column = 0; column < D; column += kChunks * 16) {
    uint32_t at = (lane / kChunks) * ts + column + (lane % kChunks) * 16;
    int row = lane / kChunks;
#pragma unroll 1
    for (; row + (kCopyAhead - 1) * kRows < tokens; row += kRows * kCopyAhead) {
      uint4 v[kCopyAhead];
#pragma unroll
      for (int k = 0; k < kCopyAhead; ++k) v[k] = *reinterpret_cast<const uint4*>(src + (at + k * step));
#pragma unroll
      for (int k = 0; k < kCopyAhead; ++k) *reinterpret_cast<uint4*>(dst + (at + k * step)) = v[k];
      at += kCopyAhead * step;
    }
#pragma unroll 1
    for (; row < tokens; row += kRows * 4) {  // the rest, four at a time
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = make_uint4(0, 0, 0, 0);
        if (row + k * kRows < tokens) v[k] = *reinterpret_cast<const uint4*>(src + (at + k * step));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row + k * kRows < tokens) *reinterpret_cast<uint4*>(dst + (at + k * step)) = v[k];
      at += 4 * step;
    }
  }
}

// A warp copies one head's keys or values of a page, with their scale (and the bounds of the keys): all of a page
// (WHOLE, compaction, whose table is rewritten here beside the copies) or its first tokens.
template <int DQK, int DV, bool WHOLE>
__global__ void __launch_bounds__(32 * kCopyWarps, kCopyBlocks) kv_copy_kernel(const __grid_constant__ CopyParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t units = static_cast<int64_t>(p.head->copies) * p.heads * 2;
  const int* src_pages = p.src + p.head->skip;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyWarps;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5); u < units; u += step) {
    const int x = static_cast<int>(u & 1);
    const int64_t copy = (u >> 1) / p.heads;
    const int head = static_cast<int>((u >> 1) - copy * p.heads);
    const int from = src_pages[copy], to = p.dst[copy];
    const int tokens = WHOLE ? p.page : p.tokens[copy];
    const uint8_t* src = p.base[x] + from * p.page_stride[x] + head * p.head_stride[x];
    uint8_t* dst = p.base[x] + to * p.page_stride[x] + head * p.head_stride[x];
    const int64_t from_head = static_cast<int64_t>(from) * p.heads + head, to_head = static_cast<int64_t>(to) * p.heads + head;
    if (lane == 0) p.scale[x][to_head] = p.scale[x][from_head];
    if (x == 0 && p.bounds != nullptr && lane < DQK / 8)
      reinterpret_cast<uint4*>(p.bounds)[to_head * (DQK / 8) + lane] =
          reinterpret_cast<const uint4*>(p.bounds)[from_head * (DQK / 8) + lane];
    if (x == 0) copy_codes<DQK>(src, dst, p.token_stride[0], tokens);
    else copy_codes<DV>(src, dst, p.token_stride[1], tokens);
  }
  if constexpr (WHOLE)
    for (int b = blockIdx.x * kCopyWarps + (threadIdx.x >> 5); b < p.table.batch; b += static_cast<int>(step))
      compact_row(p.table, b);
}

struct PagesWorkspace {
  size_t head, valid, owner, src, dst, tokens, bytes;
};
PagesWorkspace pages_workspace(int batch, int rows, int num_pages) {
  PagesWorkspace w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up256(n * sizeof(int));
    return here;
  };
  const size_t copies = static_cast<size_t>(rows > num_pages ? rows : num_pages);
  w.head = take(sizeof(PagesHead) / sizeof(int));
  w.valid = take(batch);
  w.owner = take(rows > 0 ? num_pages : 0);
  w.src = take(copies);
  w.dst = take(copies);
  w.tokens = take(rows);
  w.bytes = at;
  return w;
}

void pages_fill(PagesParams& p, uint8_t* ws, int batch, int rows, const fa_kv_cache& c) {
  const PagesWorkspace w = pages_workspace(batch, rows, c.num_pages);
  p.head = reinterpret_cast<PagesHead*>(ws + w.head);
  p.valid = reinterpret_cast<int*>(ws + w.valid);
  p.owner = reinterpret_cast<int*>(ws + w.owner);
  p.src = reinterpret_cast<int*>(ws + w.src);
  p.dst = reinterpret_cast<int*>(ws + w.dst);
  p.tokens = reinterpret_cast<int*>(ws + w.tokens);
  p.table = c.block_table;
  p.table_stride = c.table_stride;
  p.seqlens = c.seqlens_k;
  p.batch = batch;
  p.rows = rows;
  p.num_pages = c.num_pages;
  p.max_pages = c.max_pages;
  p.page_shift = page_shift(c.page_size);
}

// Shared memory of the fork's blocks: enough without known rows for the largest tables.
constexpr size_t kForkSmem = 200 * 1024;
static_assert(sizeof(int) * (3 * kMaxBatch + 2) <= kForkSmem, "the largest tables");

template <bool CACHED>
int fork_start(const PagesParams& p, size_t smem, cudaStream_t stream) {
  static bool ready[64] = {};
  const int rc = allow_smem(reinterpret_cast<const void*>(kv_fork_kernel<CACHED>), kForkSmem, ready);
  if (rc != FA_OK) return rc;
  kv_fork_kernel<CACHED><<<kCluster, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int DQK, int DV>
int copy_start(const CopyParams& p, bool whole, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCopyBlocks * sms, 1, 1);
  cfg.blockDim = dim3(32 * kCopyWarps, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, whole ? kv_copy_kernel<DQK, DV, true> : kv_copy_kernel<DQK, DV, false>, p) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int copy_launch(const PagesParams& m, const fa_kv_cache& c, uint8_t* bounds, bool whole, int sms, cudaStream_t stream) {
  CopyParams p;
  std::memset(&p, 0, sizeof(p));
  for (int x = 0; x < 2; ++x) {
    const int64_t* s = x == 0 ? c.k_stride : c.v_stride;
    p.base[x] = static_cast<uint8_t*>(x == 0 ? c.k : c.v);
    p.page_stride[x] = s[0];
    p.head_stride[x] = s[1];
    p.token_stride[x] = static_cast<uint32_t>(s[2]);
    p.scale[x] = x == 0 ? c.k_scale : c.v_scale;
  }
  p.bounds = bounds;
  p.head = m.head;
  p.src = m.src;
  p.dst = m.dst;
  p.tokens = m.tokens;
  p.heads = c.heads_kv;
  p.page = c.page_size;
  p.table = m;
  if (c.d_qk == 64) return copy_start<64, 64>(p, whole, sms, stream);
  if (c.d_qk == 128) return c.d_v == 64 ? copy_start<128, 64>(p, whole, sms, stream) : copy_start<128, 128>(p, whole, sms, stream);
  return c.d_v == 64 ? copy_start<192, 64>(p, whole, sms, stream) : copy_start<192, 128>(p, whole, sms, stream);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_kv_pages_workspace_size(int batch, int rows, int num_pages) {
  if (batch < 0 || rows < 0 || num_pages < 1) return 0;
  return pages_workspace(batch, rows, num_pages).bytes;
}

int fa_kv_fork(const fa_kv_cache* cache, void* k_bounds, const int* page_refs, int batch, const int* parents,
               const int* new_tokens, int rows, int* table_out, int64_t table_out_stride, int* seqlens_out,
               int* refs_out, void* workspace, size_t workspace_bytes, fa_stream_t stream_) {
  int rc = check_cache(cache);
  if (rc != FA_OK) return rc;
  const fa_kv_cache& c = *cache;
  if (batch < 1 || batch > kMaxBatch || rows < 1 || rows > kMaxBatch || table_out_stride < c.max_pages)
    return FA_ERR_INVALID_ARG;
  rc = check_cache_pointers(cache);
  if (rc != FA_OK) return rc;
  if (page_refs == nullptr || parents == nullptr || table_out == nullptr || seqlens_out == nullptr ||
      refs_out == nullptr || workspace == nullptr)
    return FA_ERR_INVALID_ARG;
  // the old rows are read while the new ones are written
  for (const int* in : {c.block_table, c.seqlens_k, parents, new_tokens})
    if (table_out == in || seqlens_out == in || refs_out == in) return FA_ERR_INVALID_ARG;
  if (table_out == seqlens_out || table_out == refs_out || seqlens_out == refs_out || table_out == page_refs ||
      seqlens_out == page_refs)
    return FA_ERR_INVALID_ARG;
  if (!aligned(k_bounds, 16) || !aligned(workspace, 16) || !aligned(page_refs, 4) || !aligned(parents, 4) ||
      !aligned(new_tokens, 4) || !aligned(table_out, 4) || !aligned(seqlens_out, 4) || !aligned(refs_out, 4))
    return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa_kv_pages_workspace_size(batch, rows, c.num_pages)) return FA_ERR_INVALID_ARG;
  HostDevice host;
  rc = host_device(&host);
  if (rc != FA_OK) return rc;
  if (!cache_on_device(cache, host.dev) || !host_is_device_ptr(page_refs, host.dev) ||
      !host_is_device_ptr(parents, host.dev) || (new_tokens != nullptr && !host_is_device_ptr(new_tokens, host.dev)) ||
      (k_bounds != nullptr && !host_is_device_ptr(k_bounds, host.dev)) || !host_is_device_ptr(table_out, host.dev) ||
      !host_is_device_ptr(seqlens_out, host.dev) || !host_is_device_ptr(refs_out, host.dev) ||
      !host_is_device_ptr(workspace, host.dev))
    return FA_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  PagesParams p;
  std::memset(&p, 0, sizeof(p));
  pages_fill(p, static_cast<uint8_t*>(workspace), batch, rows, c);
  p.refs = page_refs;
  p.parents = parents;
  p.grow = new_tokens;
  p.table_out = table_out;
  p.out_stride = table_out_stride;
  p.seqlens_out = seqlens_out;
  p.refs_out = refs_out;
  p.status = host.status;
  const size_t least = sizeof(int) * ((2 * static_cast<size_t>(batch) + rows + 2) & ~size_t(1));
  const size_t cached = least + sizeof(uint64_t) * rows;
  rc = cached <= kForkSmem ? fork_start<true>(p, cached, stream) : fork_start<false>(p, least, stream);
  if (rc != FA_OK) return rc;
  return copy_launch(p, c, static_cast<uint8_t*>(k_bounds), false, host.sms, stream);
}

int fa_kv_compact(const fa_kv_cache* cache, void* k_bounds, const int* page_refs, int batch, int* table_out,
                  int64_t table_out_stride, int* refs_out, int* page_map, int* used, void* workspace,
                  size_t workspace_bytes, fa_stream_t stream_) {
  int rc = check_cache(cache);
  if (rc != FA_OK) return rc;
  fa_kv_cache c = *cache;
  if (batch < 0 || batch > kMaxBatch || table_out_stride < c.max_pages) return FA_ERR_INVALID_ARG;
  if (batch == 0) {  // pages that only their counts know: no table is looked at
    c.block_table = c.seqlens_k = page_refs;
    table_out = refs_out;
  }
  rc = check_cache_pointers(&c);
  if (rc != FA_OK) return rc;
  if (page_refs == nullptr || table_out == nullptr || refs_out == nullptr || page_map == nullptr || used == nullptr ||
      workspace == nullptr)
    return FA_ERR_INVALID_ARG;
  // of the inputs, table_out may be the table and refs_out the counts
  for (const int* out : {static_cast<const int*>(page_map), static_cast<const int*>(used)})
    if (out == refs_out || out == page_refs || out == table_out || (batch > 0 && (out == c.block_table || out == c.seqlens_k)))
      return FA_ERR_INVALID_ARG;
  if (page_map == used || (batch > 0 && (table_out == refs_out || table_out == page_refs || table_out == c.seqlens_k ||
                                         refs_out == c.block_table || refs_out == c.seqlens_k)))
    return FA_ERR_INVALID_ARG;
  if (table_out == c.block_table && table_out_stride != c.table_stride && batch > 1) return FA_ERR_INVALID_ARG;
  if (!aligned(k_bounds, 16) || !aligned(workspace, 16) || !aligned(page_refs, 4) || !aligned(table_out, 4) ||
      !aligned(refs_out, 4) || !aligned(page_map, 4) || !aligned(used, 4))
    return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa_kv_pages_workspace_size(batch, 0, c.num_pages)) return FA_ERR_INVALID_ARG;
  HostDevice host;
  rc = host_device(&host);
  if (rc != FA_OK) return rc;
  if (!cache_on_device(&c, host.dev) || !host_is_device_ptr(page_refs, host.dev) ||
      (k_bounds != nullptr && !host_is_device_ptr(k_bounds, host.dev)) || !host_is_device_ptr(table_out, host.dev) ||
      !host_is_device_ptr(refs_out, host.dev) || !host_is_device_ptr(page_map, host.dev) ||
      !host_is_device_ptr(used, host.dev) || !host_is_device_ptr(workspace, host.dev))
    return FA_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  PagesParams p;
  std::memset(&p, 0, sizeof(p));
  pages_fill(p, static_cast<uint8_t*>(workspace), batch, 0, c);
  p.refs = page_refs;
  p.table_out = table_out;
  p.out_stride = table_out_stride;
  p.refs_out = refs_out;
  p.page_map = page_map;
  p.used = used;
  p.status = host.status;
  kv_compact_kernel<<<kCluster, kThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  return copy_launch(p, c, static_cast<uint8_t*>(k_bounds), true, host.sms, stream);
}

}  // extern "C"
