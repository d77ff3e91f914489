// fa_fwd_paged for few rows a sequence (tokens, drafts): attention of the new
// tokens over 8-bit pages.
//
// With codes c and scales s per page, S = (scale s_K) q . c_K and
// O = sum_pages s_V (P c_V): a scale is one factor per 16 tokens, never a
// multiplication per code.  The products run on the tensor cores transposed,
// so that the few query rows are the small dimension (n8) and the tokens (for
// S) or value columns (for O) the large one (m16):
//     S^T[16 tokens x 8 rows] += K[16 x 16] Q^T[16 x 8]
//     O^T[16 columns x 8 rows] += V^T[16 x 16 tokens] P^T[16 x 8]
// Codes become f16 exactly.  A query row is multiplied by a power of two that
// puts its largest value at the top of f16's range, so that its bf16 values are
// exact down to 2^-31 of the largest and off by at most 2^-39 of it below (what
// counts against keys that are 0 where the query is large; with the largest at 1
// rounding began at 2^-18).  P is rounded to f16 scaled by 2^7: 11 bits where
// bf16 would keep 8, for weights down to 2^-21 of the row's reference; below that
// a weight is off by at most 2^-32, whatever the scales of its values.
// Scores, maxima, sums and O stay in fp32.
//
// Work: a tile is 32 or 64 tokens of one key/value head; the tiles of all
// sequences and heads form one line that is cut into equal pieces, one for
// each warp ("team").  A warp streams its piece through its own ring of slots,
// K and V tiles by turns, filled by asynchronous 16-byte copies kSlots - 1 slots
// ahead, independently of the others.  A (sequence, head) that lies in one piece
// is written out at once, one that is cut leaves unnormalised parts that
// paged_merge_kernel joins.
//
// Bound by DRAM: B8 x 32767 keys, 32/8 heads of 128: 94 us with the merge, 5.7
// TB/s of codes (the copies alone: 84 us); 16 heads of 192/128: 60 us, 5.5 TB/s;
// 16 heads of 64 in pages of 16, copies of 1 KB: 123 us, 4.4 TB/s (copies alone
// 102).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fa_paged.cuh"
#include "fa_paged.h"
#include "fa_paged_range.h"
#include "ptx.cuh"

namespace fa {

struct PagedParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const uint8_t* k;  // codes
  const uint8_t* v;
  int64_t k_page, k_head, v_page, v_head;  // bytes between pages and heads
  uint32_t k_token, v_token;               // and tokens
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const int* table;
  int64_t table_stride;
  const int* seqlens;
  const int* cu;
  unsigned int* status;
  PagedParts part;
  int64_t total_q;
  int batch, heads_q, heads_kv, ratio, num_pages, max_pages, page_shift, causal;
  unsigned long long timeout_ns;  // of a wait (paged_tc_kernel)
  int copy_shift;  // 2^this copies of the rows in the 128 lanes (paged_tc_kernel), each with its share of the tokens
  int max_n;      // longest sequence of new tokens allowed
  int row_least, row_limit;  // sequences with fewer or more rows (new tokens x ratio) are not this kernel's
  int unpacked;              // the call has sequences of more than kPagedRowLimit rows, computed before
  int after;                 // launched while the kernel before it may still run: ends after that (paged_tc_kernel)
  float scale_log2;
};

// A cut (sequence, head) that starts in a piece and ends in piece `last`.
struct PagedJoin {
  int last;  // -1: none
  int cu0, head, rows;
};

constexpr int kMinTokens = 64;        // a piece is not cut smaller
constexpr float kPShift = 7.f;        // P is scaled by 2^7: f16 then holds weights down to 2^-31
constexpr float kRefLag = 8.f;        // the reference follows the maximum when it lags by more (log2 units)

// NT groups of 8 rows.  64 tokens a tile halve what a
// tile costs beside its products (B8 x 32768, 32/8 heads of 128: 93 us against
// 97 with 32; 16 heads of 64 in pages of 16: 123 against 150); more rows or
// wider keys leave registers for 32.  Two warps a scheduler: with three, 168
// registers a thread spill (116 us for the first of these).  With two, 255 spill 12
// to 24 bytes at (128, 128) and 8 rows, 100 to 116 at (128, 128) and (192, 128) and 16
// rows, nothing elsewhere.
template <int DQK, int DV, int NT>
struct PagedShape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = NT == 1 && DQK <= 128 ? 64 : 32;  // tokens
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kTeams = kWarps;  // each warp streams a piece of its own
  static constexpr int kSlotBytes = kTile * (DQK > DV ? DQK : DV);
  static constexpr int kSlots = 206 * 1024 / kSlotBytes / kTeams;  // of a team's ring
  static constexpr int kBytes = kTeams * kSlots * kSlotBytes + 128;
  static_assert(kSlots >= 3, "a tile in use and one under way");
};

// Bounded wait for an mbarrier phase; false after the time limit or an abort.
// The clock is read only now and then: that takes longer than most waits here.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, const WaitCtx& w) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0u) {
      if (*w.abort_flag) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > w.timeout_ns) {
        raise_abort(w, kStatusTimeout, kSitePagedWait);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same from a sum of 0
__device__ __forceinline__ void mma_f16_zero(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Where a tile's 16-byte chunk `chunk` of token `row` lies in its slot, so that
// the reads below meet no bank twice.  K is read as chunks of eight tokens
// (two a quarter warp), V as chunks of the even or the odd of eight tokens.
template <int D>
__device__ __forceinline__ uint32_t k_place(int row, int chunk) {
  if constexpr (D == 128) return row * 128 + ((chunk ^ (row & 7)) << 4);
  return row * D + (chunk << 4);  // rows of 64 and 192 bytes: neighbours fall on different halves of the banks
}
template <int D>
__device__ __forceinline__ uint32_t v_place(int row, int chunk) {
  if constexpr (D == 128) return row * 128 + ((chunk ^ (row & 7)) << 4);
  const int at = (row & ~7) | ((row >> 1) & 3) | ((row & 1) << 2);  // even tokens first
  return at * 64 + ((chunk ^ (at & 2)) << 4);
}
// K chunk number `step` of lane column c: all chunks of a row once, and query columns by the same rule
template <int DQK>
__device__ __forceinline__ int k_chunk(int c, int step) {
  return DQK == 128 ? 2 * c + step : 4 * step + c;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of this thread's groups of copies are under way
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One sequence as the kernel sees it.
struct PagedSeq {
  int cu0, n, len;
  int rows, tiles;  // new tokens x ratio (0: not this kernel's), tiles
  bool bad;
};

template <int TILE>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  PagedSeq s;
  s.cu0 = p.cu[b];
  s.len = p.seqlens[b];
  s.bad = !paged_attend_range(s.cu0, p.cu[b + 1], s.len, p.total_q, p.max_n,
                              static_cast<int64_t>(p.max_pages) << p.page_shift, s.n);
  const int64_t rows = s.bad ? 0 : static_cast<int64_t>(s.n) * p.ratio;
  s.rows = rows > p.row_limit || rows < p.row_least ? 0 : static_cast<int>(rows);
  s.tiles = s.len > 0 ? (s.len - 1) / TILE + 1 : 1;  // without a key: one tile that is masked
  return s;
}

// A place on the line of tiles.
struct PagedCursor {
  PagedSeq s;
  int b, head, tile;
  long long at;  // on the line, where units have a start that costs something
};

// To the next tile (the caller knows that there is one).
template <int TILE, int START = 0>
__device__ __forceinline__ void paged_next(const PagedParams& p, PagedCursor& c) {
  if constexpr (START > 0) ++c.at;
  if (++c.tile < c.s.tiles) return;
  if constexpr (START > 0) c.at += START;
  c.tile = 0;
  if (++c.head < p.heads_kv) return;
  c.head = 0;
  do {
    if (c.b + 1 >= p.batch) return;
    c.s = paged_seq<TILE>(p, ++c.b);
  } while (c.s.rows == 0);
}

// The line of tiles of all sequences and heads, and its equal pieces.  A unit,
// a (sequence, head), takes as many places as it has tiles and START more in
// front of them, for what its start and its end cost.
struct PagedLine {
  long long total, per, used;  // places, places of a piece, pieces that hold some
  int teams_used;              // of a block
  __device__ __forceinline__ long long piece(int team) const {
    return static_cast<long long>(blockIdx.x) * teams_used + team;
  }
  __device__ __forceinline__ int count(int team) const {  // places of a team of this block
    const long long left = total - piece(team) * per;
    return team >= teams_used || left <= 0 ? 0 : static_cast<int>(left < per ? left : per);
  }
};

// By all threads of the block: cuts the line, finds the places where this
// block's pieces begin, and says that no piece leaves anything to join yet.
// With START > 0 (one team) also counts the piece's tiles.  Ends with a barrier.
template <int TILE, int THREADS, int TEAMS, int START>
__device__ __forceinline__ void paged_line(const PagedParams& p, long long* scan, long long* warp_sum,
                                           PagedCursor* begin_at, int* tiles, PagedLine& line) {
  static_assert(START == 0 || TEAMS == 1, "tiles are counted for one team");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (START > 0 && tid == 0) *tiles = 0;
  PagedSeq mine;
  long long v;                                   // places of this thread's sequence
  auto scan_block = [&](int base) -> long long {  // inclusive scan of THREADS sequences' places into scan[]
    const int b = base + tid;
    v = 0;
    if (b < p.batch) {
      mine = paged_seq<TILE>(p, b);
      if (mine.bad && blockIdx.x == 0) paged_error(p.status, kSitePagedSeq, b);
      v = mine.rows > 0 ? (static_cast<long long>(mine.tiles) + START) * p.heads_kv : 0;
    }
    long long sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    scan[tid] = before + sum;
    __syncthreads();
    return scan[THREADS - 1];
  };
  line.total = 0;
  for (int base = 0; base < p.batch; base += THREADS) line.total += scan_block(base);
  const long long pieces = static_cast<long long>(gridDim.x) * TEAMS;
  line.per = (line.total + pieces - 1) / pieces;
  if (line.per < kMinTokens / TILE) line.per = kMinTokens / TILE;
  if (line.per < 1) line.per = 1;
  line.used = (line.total + line.per - 1) / line.per;
  line.teams_used = static_cast<int>((line.used + gridDim.x - 1) / gridDim.x);

  long long offset = 0;
  for (int base = 0; base < p.batch; base += THREADS) {
    if (p.batch > THREADS) scan_block(base);
    const long long sum = scan[THREADS - 1];
    if constexpr (START > 0) {  // each thread for its own sequence
      const long long before = offset + scan[tid] - v, x0 = line.piece(0) * line.per;
      const long long x1 = x0 + line.per < line.total ? x0 + line.per : line.total;
      const long long lo = (x0 > before ? x0 : before) - before, hi = (x1 < before + v ? x1 : before + v) - before;
      if (lo < hi) {
        const long long unit = mine.tiles + START;
        const long long head0 = lo / unit, in0 = lo - head0 * unit - START;
        const long long head1 = hi / unit, in1 = hi - head1 * unit - START;
        atomicAdd(tiles, static_cast<int>((head1 - head0) * mine.tiles + (in1 > 0 ? in1 : 0) - (in0 > 0 ? in0 : 0)));
        if (lo + before == x0) {
          PagedCursor c;
          c.s = mine;
          c.b = base + tid;
          c.head = static_cast<int>(head0);
          c.tile = static_cast<int>(in0 > 0 ? in0 : 0);
          c.at = x0 + (in0 < 0 ? -in0 : 0);
          *begin_at = c;
        }
      }
    } else if (tid < TEAMS && line.count(tid) > 0) {
      const long long x = line.piece(tid) * line.per - offset;
      if (x >= 0 && x < sum) {  // the first sequence whose inclusive sum exceeds x
        int lo = 0, hi = THREADS - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (scan[mid] > x) hi = mid;
          else lo = mid + 1;
        }
        PagedCursor c;
        c.b = base + lo;
        c.s = paged_seq<TILE>(p, c.b);
        const long long in = x - (lo > 0 ? scan[lo - 1] : 0);
        c.head = static_cast<int>(in / c.s.tiles);
        c.tile = static_cast<int>(in - static_cast<long long>(c.head) * c.s.tiles);
        begin_at[tid] = c;
      }
    }
    offset += sum;
    if (p.batch > THREADS) __syncthreads();
  }
  // pieces beyond the used ones are cleared in plain order
  if (tid < TEAMS) {
    if (line.count(tid) > 0) p.part.joins[line.piece(tid)].last = -1;
    const long long plain = static_cast<long long>(blockIdx.x) * TEAMS + tid;
    if (plain >= line.used) p.part.joins[plain].last = -1;
  }
  __syncthreads();
}

// G16: pages of 16 tokens, each with its own scale; else a scale holds for 32 tokens at least.
template <int DQK, int DV, int NT, bool G16>
__global__ void __launch_bounds__(PagedShape<DQK, DV, NT>::kThreads, 1)
    paged_attn_kernel(const __grid_constant__ PagedParams p) {
  using Shape = PagedShape<DQK, DV, NT>;
  constexpr int kTile = Shape::kTile;
  constexpr int kSteps = DQK / 64;       // 64-column groups of K
  constexpr int kVWords = DV / 32;       // 32-bit words of V codes a lane reads per token
  constexpr int kVTiles = DV / 16;       // m16 tiles of O^T
  constexpr int kMT = kTile / 16;        // m16 tiles of S^T
  constexpr int kTeams = Shape::kTeams, kSlots = Shape::kSlots, kRows = Shape::kRows, kThreads = Shape::kThreads;
  constexpr int kWarps = Shape::kWarps;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) float slot_scale[kTeams * kSlots][4];  // of 16 tokens each
  __shared__ PagedCursor begin_at[kTeams];
  __shared__ long long scan[kThreads];
  __shared__ long long warp_sum[kWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t smem0 = (smem_u32(smem_raw) + 127u) & ~127u;

  // let the merge kernel's blocks take their places early: they wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  PagedLine line;
  paged_line<kTile, kThreads, kTeams, 0>(p, scan, warp_sum, begin_at, nullptr, line);

  const int team = warp;
  const int g = lane >> 2, c = lane & 3;
  const int count = line.count(team);
  if (count == 0) return;
  const long long piece = line.piece(team), begin = piece * line.per;
  PagedCursor cur = begin_at[team];
  const uint32_t ring = smem0 + team * kSlots * Shape::kSlotBytes;

  // ---- the warp fills its ring: tile after tile, K and V by turns ----
  constexpr int kRun = G16 ? 16 : 32;  // tokens that surely lie in one page
  PagedCursor ahead = cur;  // the tile that is filled in next
  int filled = 0;           // slots filled so far
  int fill_slot = 0;
  // lane l holds page page0 + l of the cursor's sequence: its index, the scales of the cursor's head, and (as
  // loaded) those of the next head
  int page0 = 0, entry = 0, ks_next = 127, vs_next = 127;
  float ks = 1.f, vs = 1.f;
  bool fresh = true;  // the pages' scales are still to be taken over
  auto load_scales = [&](int head) {
    ks_next = vs_next = 127;
    if (((page0 + lane) << p.page_shift) < ahead.s.len) {
      const int64_t at = static_cast<int64_t>(entry) * p.heads_kv + head;
      ks_next = p.k_scale[at];
      vs_next = p.v_scale[at];
    }
  };
  auto take_scales = [&]() {
    ks = vs_next == 255 ? scale_of(255) : scale_of(ks_next);  // NaN in either: NaN scores
    vs = vs_next == 255 ? 1.f : scale_of(vs_next);
    if (ahead.head + 1 < p.heads_kv) load_scales(ahead.head + 1);
  };
  auto load_pages = [&](int first) {
    page0 = first;
    entry = 0;
    if (((first + lane) << p.page_shift) < ahead.s.len) {
      entry = p.table[ahead.b * p.table_stride + first + lane];
      if (entry < 0 || entry >= p.num_pages) {
        paged_error(p.status, kSitePagedPage, ahead.b);
        entry = 0;
      }
    }
    load_scales(ahead.head);
    fresh = true;
  };
  // scale k of a slot belongs to 16 tokens: their page's lane, counted from the tile's first
  const int scale_lane = G16 ? lane : lane >> (p.page_shift - 4);
  // The tokens of a tile, 16 bytes a lane; pages behind the last are left out.  Lane l's chunks in a run
  // of tokens are l, l + 32, ..: with rows of 4 or 8 chunks they are one column, with 12 the rows repeat by 8.
  auto lane_offset = [&](int d, uint32_t token_stride, int i) -> uint32_t {
    const int at = i * 32 + lane, chunks = d / 16;
    return static_cast<uint32_t>(at / chunks) * token_stride + (at % chunks) * 16;
  };
  constexpr int kOffsets = DQK == 192 ? 3 : 1;
  uint32_t k_off[kOffsets];
#pragma unroll
  for (int i = 0; i < kOffsets; ++i) k_off[i] = lane_offset(DQK, p.k_token, i);
  const uint32_t v_off = lane_offset(DV, p.v_token, 0);
  const uint8_t *k_at, *v_at;  // of the cursor's head
  auto set_head = [&]() {
    k_at = p.k + ahead.head * p.k_head;
    v_at = p.v + ahead.head * p.v_head;
  };
  auto copy = [&](auto is_k, uint32_t dst, int token) {
    constexpr bool kK = decltype(is_k)::value;
    constexpr int D = kK ? DQK : DV, kChunks = D / 16;
    static_assert(kRun * kChunks % 32 == 0, "whole warps of chunks");
    const uint32_t ts = kK ? p.k_token : p.v_token;
#pragma unroll
    for (int row0 = 0; row0 < kTile; row0 += kRun) {
      const int t = token + row0;
      const int e = __shfl_sync(0xffffffffu, entry, (t >> p.page_shift) - page0);
      if (t < ahead.s.len) {
        const uint8_t* src = (kK ? k_at : v_at) + e * (kK ? p.k_page : p.v_page) +
                             static_cast<uint64_t>(static_cast<uint32_t>(t & ((1 << p.page_shift) - 1)) * ts);
        if constexpr (D != 192) src += kK ? k_off[0] : v_off;
#pragma unroll
        for (int i = 0; i < kRun * kChunks / 32; ++i) {
          const int at = i * 32 + lane, row = at / kChunks, chunk = at % kChunks;
          const uint8_t* from = D == 192 ? src + k_off[i % kOffsets] + (i / 3) * 8 * ts : src + i * (32 / kChunks) * ts;
          cp_async16(dst + (kK ? k_place<D>(row0 + row, chunk) : v_place<D>(row0 + row, chunk)), from);
        }
      }
    }
  };
  auto fill = [&]() {  // the next slot, which has been read
    if (filled < 2 * count) {
      const bool is_k = (filled & 1) == 0;
      const int token = ahead.tile * kTile;
      const uint32_t dst = ring + fill_slot * Shape::kSlotBytes;
      if (is_k) copy(std::true_type{}, dst, token);
      else copy(std::false_type{}, dst, token);
      if (fresh) {
        take_scales();
        fresh = false;
      }
      const float scale = __shfl_sync(0xffffffffu, is_k ? ks : vs, (token >> p.page_shift) - page0 + scale_lane);
      if (lane < kTile / 16) slot_scale[team * kSlots + fill_slot][lane] = scale;
      ++filled;
      if (++fill_slot == kSlots) fill_slot = 0;
      if (!is_k && filled < 2 * count) {  // on to the next tile
        const int b = ahead.b, head = ahead.head;
        paged_next<kTile>(p, ahead);
        if (ahead.head != head) set_head();
        const int next = (ahead.tile * kTile) >> p.page_shift;
        if (ahead.b == b && ahead.head == head + 1 && page0 == 0) take_scales();  // the same pages, the next head
        else if (ahead.b != b || ahead.head != head || next + kTile / 16 > page0 + 32) load_pages(next);
      }
    }
    cp_async_commit();  // a group for each slot, empty ones at the end
  };
  set_head();
  load_pages((ahead.tile * kTile) >> p.page_shift);
  for (int e = 0; e < kSlots - 1; ++e) fill();
  int slot = -1;
  // The next slot's tokens are there for all lanes, which have read the slot before: that one is refilled.
  auto advance = [&]() {
    cp_async_wait<kSlots - 2>();
    __syncwarp();
    if (++slot == kSlots) slot = 0;
    fill();
  };

  uint32_t qf[NT][kSteps * 4][2];
  float qfac[NT][2], ref[NT][2], sum[NT][2];
  int limit[NT][2];
  float o[NT][kVTiles][4];
  int min_limit = 0;
  bool started_here = false;

  for (int i = 0; i < count; ++i) {
    if (i == 0 || cur.tile == 0) {
      // ---- a new (sequence, head): the query rows as B fragments ----
      started_here = cur.tile == 0;
      min_limit = cur.s.len;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        uint4 raw[kSteps * 2];
        if (r < cur.s.rows) {
          const int pos = r / p.ratio, hr = r - pos * p.ratio;
          const __nv_bfloat16* src =
              p.q + (static_cast<int64_t>(cur.s.cu0 + pos) * p.heads_q + cur.head * p.ratio + hr) * DQK;
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              raw[s * 2 + h] = __ldg(reinterpret_cast<const uint4*>(src + 16 * k_chunk<DQK>(c, s) + 8 * h));
        } else {
#pragma unroll
          for (int s = 0; s < kSteps * 2; ++s) raw[s] = make_uint4(0, 0, 0, 0);
        }
        // the row's largest exponent: its values times a power of two fit f16
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < kSteps * 2; ++s) {
          const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a = w[k] & 0x7f80u, b = (w[k] >> 16) & 0x7f80u;
            top = top > a ? top : a;
            top = top > b ? top : b;
          }
        }
        uint32_t y = __shfl_xor_sync(0xffffffffu, top, 1);
        top = top > y ? top : y;
        y = __shfl_xor_sync(0xffffffffu, top, 2);
        top = top > y ? top : y;
        const QueryScale qs = query_scale(static_cast<int>(top >> 7));
        const float down = qs.down;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t f[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = raw[s * 2 + h];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)  // word k holds columns 8 h + 2 k, + 1: step (8 h + 2 k) / 4, half k & 1
              f[4 * h + k] = pack_f16x2(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            qf[nt][s * 4 + k][0] = f[2 * k], qf[nt][s * 4 + k][1] = f[2 * k + 1];
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // this lane's columns of S^T are rows 2 c and 2 c + 1
          qfac[nt][k] = p.scale_log2 * __shfl_sync(0xffffffffu, qs.up, (2 * c + k) * 4);
          ref[nt][k] = -INFINITY;
          sum[nt][k] = 0.f;
          const int rr = nt * 8 + 2 * c + k;
          int lim = cur.s.len;
          if (p.causal && rr < cur.s.rows) {
            lim = cur.s.len - cur.s.n + rr / p.ratio + 1;
            lim = lim < 0 ? 0 : lim > cur.s.len ? cur.s.len : lim;
          }
          limit[nt][k] = lim;
          min_limit = min_limit < lim ? min_limit : lim;
        }
#pragma unroll
        for (int v = 0; v < kVTiles; ++v)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][v][k] = 0.f;
      }
      min_limit = min(min_limit, __shfl_xor_sync(0xffffffffu, min_limit, 1));
      min_limit = min(min_limit, __shfl_xor_sync(0xffffffffu, min_limit, 2));
    }

    const int token0 = cur.tile * kTile;
    const bool masked = token0 + kTile > min_limit;

    // ---- S^T: kMT x 16 tokens ----
    advance();
    float s[kMT][NT][4];
    {
      const uint32_t tk = ring + slot * Shape::kSlotBytes;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        uint32_t wa[kMT][4], wb[kMT][4];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          const uint4 ra = lds128(tk + k_place<DQK>(16 * mt + g, k_chunk<DQK>(c, st)));
          const uint4 rb = lds128(tk + k_place<DQK>(16 * mt + 8 + g, k_chunk<DQK>(c, st)));
          wa[mt][0] = ra.x, wa[mt][1] = ra.y, wa[mt][2] = ra.z, wa[mt][3] = ra.w;
          wb[mt][0] = rb.x, wb[mt][1] = rb.y, wb[mt][2] = rb.z, wb[mt][3] = rb.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            const uint32_t a0 = e4m3x2_f16x2(wa[mt][k]), a1 = e4m3x2_f16x2(wb[mt][k]);
            const uint32_t a2 = e4m3x2_hi_f16x2(wa[mt][k]), a3 = e4m3x2_hi_f16x2(wb[mt][k]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (st == 0 && k == 0) mma_f16_zero(s[mt][nt], a0, a1, a2, a3, qf[nt][st * 4 + k][0], qf[nt][st * 4 + k][1]);
              else mma_f16(s[mt][nt], a0, a1, a2, a3, qf[nt][st * 4 + k][0], qf[nt][st * 4 + k][1]);
            }
          }
        }
      }
      // scores in log2 units
      const float4 m = *reinterpret_cast<const float4*>(slot_scale[team * kSlots + slot]);
      const float ms[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[mt][nt][k] *= qfac[nt][k & 1] * ms[G16 ? mt : mt & ~1];
    }
    advance();
    const uint32_t tv = ring + slot * Shape::kSlotBytes;
    uint32_t keep[kTile / 32];
    if (masked) {
      // A hidden token has weight 0, but 0 times a value that is no number is none: tokens behind the
      // sequence's end count as 0, and a token whose values hold a NaN code counts as 0 with a NaN score,
      // which only the rows that see it take in.
#pragma unroll
      for (int h = 0; h < kTile / 32; ++h) {
        const int row = 32 * h + lane;
        const bool inside = token0 + row < cur.s.len;
        uint32_t nan = 0;
        if (inside) {
#pragma unroll
          for (int k = 0; k < DV / 16; ++k) {
            const uint4 v = lds128(tv + v_place<DV>(row, k));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) nan |= ((w[x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
          }
        }
        const uint32_t poison = __ballot_sync(0xffffffffu, nan != 0);
        keep[h] = __ballot_sync(0xffffffffu, inside) & ~poison;
#pragma unroll
        for (int mt = 2 * h; mt < 2 * h + 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = 16 * (mt & 1) + g + (k >> 1) * 8;
              const float x = (poison >> at) & 1 ? __uint_as_float(0x7fc00000u) : s[mt][nt][k];
              s[mt][nt][k] = token0 + 32 * h + at < limit[nt][k & 1] ? x : -INFINITY;
            }
      }
    }

    // ---- online softmax: the reference moves only when it lags the maximum by more than 2^8 ----
    uint32_t pf[kMT][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float alpha[2];
      bool moved = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = fmaxf(s[0][nt][k], s[0][nt][k + 2]);
#pragma unroll
        for (int mt = 1; mt < kMT; ++mt) mx = fmax3(mx, s[mt][nt][k], s[mt][nt][k + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        alpha[k] = 1.f;
        if (mx > ref[nt][k] + kRefLag) {  // also from -inf
          alpha[k] = ex2_approx(ref[nt][k] - mx);
          ref[nt][k] = mx;
          moved = true;
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int v = 0; v < kVTiles; ++v) {
          o[nt][v][0] *= alpha[0], o[nt][v][1] *= alpha[1];
          o[nt][v][2] *= alpha[0], o[nt][v][3] *= alpha[1];
        }
        sum[nt][0] *= alpha[0], sum[nt][1] *= alpha[1];
      }
      const float r0 = ref[nt][0] == -INFINITY ? 0.f : kPShift - ref[nt][0];
      const float r1 = ref[nt][1] == -INFINITY ? 0.f : kPShift - ref[nt][1];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = ex2_approx(s[mt][nt][k] + ((k & 1) ? r1 : r0));
        sum[nt][0] += e[0] + e[2];
        sum[nt][1] += e[1] + e[3];
        // accumulator layout (token g, rows 2 c ..) to operand layout (tokens 2 c .., row g)
        pf[mt][nt][0] = transpose_8x8(pack_f16x2(e[0], e[1]));
        pf[mt][nt][1] = transpose_8x8(pack_f16x2(e[2], e[3]));
      }
    }

    // ---- O^T += V^T P^T, the page's scale applied to each 16 or 32 tokens' product ----
    const float4 m = *reinterpret_cast<const float4*>(slot_scale[team * kSlots + slot]);
    const float ms[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
    for (int h = 0; h < kTile / 32; ++h) {
      // codes of this lane: tokens 16 t + {2 c, 2 c + 1, 2 c + 8, 2 c + 9} of the half, columns DV / 8 * g ..
      uint32_t vw[2][4][kVWords];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int row = 32 * h + 16 * mt + 2 * c + (t & 1) + (t >> 1) * 8;
          if constexpr (DV == 128) {
            const uint4 v = lds128(tv + v_place<DV>(row, g));
            vw[mt][t][0] = v.x, vw[mt][t][1] = v.y, vw[mt][t][2] = v.z, vw[mt][t][3] = v.w;
          } else {
            const uint2 v = lds64(tv + v_place<DV>(row, g >> 1) + (g & 1) * 8);
            vw[mt][t][0] = v.x, vw[mt][t][1] = v.y;
          }
        }
      if (masked) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int row = 16 * mt + 2 * c + (t & 1) + (t >> 1) * 8;
#pragma unroll
            for (int k = 0; k < kVWords; ++k) vw[mt][t][k] = (keep[h] >> row) & 1 ? vw[mt][t][k] : 0u;
          }
      }
#pragma unroll
      for (int w = 0; w < kVWords; ++w) {
        uint32_t pair[2][2][2];  // [16 tokens][columns 4 w + 0, 1 or 2, 3][tokens (0, 1) or (2, 3)]
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            pair[mt][0][t] = __byte_perm(vw[mt][2 * t][w], vw[mt][2 * t + 1][w], 0x5140);
            pair[mt][1][t] = __byte_perm(vw[mt][2 * t][w], vw[mt][2 * t + 1][w], 0x7362);
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t a[2][4];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              a[mt][2 * t] = e4m3x2_f16x2(pair[mt][x][t]);
              a[mt][2 * t + 1] = e4m3x2_hi_f16x2(pair[mt][x][t]);
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float* const out = o[nt][2 * w + x];
            float acc[4];
            mma_f16_zero(acc, a[0][0], a[0][1], a[0][2], a[0][3], pf[2 * h][nt][0], pf[2 * h][nt][1]);
            if constexpr (G16) {
              float acc1[4];
              mma_f16_zero(acc1, a[1][0], a[1][1], a[1][2], a[1][3], pf[2 * h + 1][nt][0], pf[2 * h + 1][nt][1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) out[k] = fmaf(acc1[k], ms[2 * h + 1], fmaf(acc[k], ms[2 * h], out[k]));
            } else {
              mma_f16(acc, a[1][0], a[1][1], a[1][2], a[1][3], pf[2 * h + 1][nt][0], pf[2 * h + 1][nt][1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) out[k] = fmaf(acc[k], ms[2 * h], out[k]);
            }
          }
        }
      }
    }
    // ---- the end of the unit or of the piece: write out ----
    const bool unit_end = cur.tile + 1 == cur.s.tiles;
    if (unit_end || i + 1 == count) {
      const bool whole = started_here && unit_end;
      const int64_t part = 2 * piece + (started_here ? 1 : 0);
      if (!whole && started_here && lane == 0) {
        // the rest of the unit lies in the pieces that follow
        PagedJoin j;
        j.last = static_cast<int>((begin + i + (cur.s.tiles - 1 - cur.tile)) / line.per);
        j.cu0 = cur.s.cu0;
        j.head = cur.head;
        j.rows = cur.s.rows;
        p.part.joins[piece] = j;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // A value that is no number makes its whole row so, here as where its tile is masked: this lane's columns
          // of O tell, the sum takes it to all others.
          uint32_t top = 0;  // of O's bits without their signs
#pragma unroll
          for (int v = 0; v < kVTiles; ++v)
            top = max(top, max(__float_as_uint(o[nt][v][k]) & 0x7fffffffu, __float_as_uint(o[nt][v][k + 2]) & 0x7fffffffu));
          float l = top > 0x7f800000u ? __uint_as_float(0x7fc00000u) : sum[nt][k];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const int r = nt * 8 + 2 * c + k;
          const float rf = l != 0.f && ref[nt][k] == -INFINITY ? kPShift : ref[nt][k];
          if (r < cur.s.rows) {
            if (whole) {
              const int pos = r / p.ratio, hq = cur.head * p.ratio + (r - pos * p.ratio);
              const int64_t token = cur.s.cu0 + pos;
              const float inv = l == 0.f ? 0.f : 1.f / l;
              uint32_t out[kVTiles];
#pragma unroll
              for (int v = 0; v < kVTiles; ++v) out[v] = pack_bf16x2(o[nt][v][k] * inv, o[nt][v][k + 2] * inv);
              uint4* dst = reinterpret_cast<uint4*>(p.o + (token * p.heads_q + hq) * DV + g * (DV / 8));
#pragma unroll
              for (int v = 0; v < kVTiles / 4; ++v)
                dst[v] = make_uint4(out[4 * v], out[4 * v + 1], out[4 * v + 2], out[4 * v + 3]);
              if (p.lse != nullptr && g == 0)
                p.lse[hq * p.total_q + token] =
                    l == 0.f ? -INFINITY : (rf - kPShift + log2f(l)) * 0.6931471805599453f;
            } else {
              float4* dst = reinterpret_cast<float4*>(p.part.o + (part * kRows + r) * DV + g * (DV / 8));
#pragma unroll
              for (int v = 0; v < kVTiles / 2; ++v)
                dst[v] = make_float4(o[nt][2 * v][k], o[nt][2 * v][k + 2], o[nt][2 * v + 1][k], o[nt][2 * v + 1][k + 2]);
              if (g == 0) p.part.ml[part * kRows + r] = make_float2(rf, l);
            }
          }
        }
    }
    if (i + 1 < count) paged_next<kTile>(p, cur);
  }
}

// Joins the parts of the cut units: with references m_i and sums l_i of the
// parts and M = max m_i,
//     O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// A block takes the rows of a few pieces' units, a warp a row; parts are taken in
// their order, so the result does not depend on timing.  Bound by latency (4 us
// beside the launch): loads of a row's first FIRST parts do not wait for its
// weights, and there are few blocks, for most pieces leave nothing to join.  Eight
// parts where only few rows are joined (127 registers, 80 at d_v = 64), four (64)
// where blocks are many: single tokens over 1026 keys 10.7 and 11.7 us, 128 rows of
// 32 x 8000 keys 50.5 and 48.1.
struct PagedMerge {
  struct Set {
    PagedParts part;
    int blocks, pieces, shares, rows;  // blocks; pieces of a block, blocks that share them; rows of the parts' layout
  } set[2];
  __nv_bfloat16* o;
  float* lse;
  const int* cu;
  int64_t total_q;
  int heads_q, ratio, batch, max_n;
};

// The variable-length forward gives -inf for the log-sum-exp of a row that met a
// NaN.  A row without a key has that too, but O = 0: where O is NaN, and the row
// is one of an unpacked sequence, the log-sum-exp becomes NaN as in the other
// kernels.  Thread i of the grid looks at 4 i .. 4 i + 3, which it asks for before
// parts are joined: 6.9 us with it for 2 x 2048 x 32 rows, 5.8 without.
__device__ __forceinline__ float4 paged_lse4(const PagedMerge& p, int64_t i) {
  const int64_t rows = p.total_q * p.heads_q, at = 4 * i;
  if (at + 4 <= rows) return *reinterpret_cast<const float4*>(p.lse + at);
  return make_float4(at < rows ? p.lse[at] : 0.f, at + 1 < rows ? p.lse[at + 1] : 0.f, at + 2 < rows ? p.lse[at + 2] : 0.f,
                     0.f);
}
template <int DV>
__device__ __forceinline__ void paged_nan_lse(const PagedMerge& p, int64_t at) {
  const int hq = static_cast<int>(at / p.total_q);
  const int64_t token = at - hq * p.total_q;
  if (!isnan(__bfloat162float(p.o[(token * p.heads_q + hq) * DV]))) return;
  int lo = 0, hi = p.batch - 1;  // the last sequence that begins at the token or before
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu[mid] <= token) lo = mid;
    else hi = mid - 1;
  }
  const int c0 = p.cu[lo], c1 = p.cu[lo + 1], n = paged_difference(c1, c0);
  if (paged_offsets_ok(c0, c1, p.total_q) && n <= p.max_n && token >= c0 && token < c1 &&
      static_cast<int64_t>(n) * p.ratio > kPagedRowLimit)
    p.lse[at] = __uint_as_float(0x7fc00000u);
}

template <int DV, int FIRST>
__device__ __forceinline__ void paged_merge_row(const PagedMerge& p, const PagedParts& part, int rows, int piece,
                                                const PagedJoin& j, int local) {
  constexpr int kPer = DV / 32;
  using Vec = std::conditional_t<kPer == 4, float4, float2>;
  const int lane = threadIdx.x & 31;
  const int parts = j.last - piece + 1;
  auto row = [&](int i) { return (2 * static_cast<int64_t>(piece + i) + (i == 0 ? 1 : 0)) * rows + local; };
  auto values = [&](int i) { return *reinterpret_cast<const Vec*>(part.o + row(i) * DV + lane * kPer); };
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < parts) ml = part.ml[row(lane)];
  Vec first[FIRST];
#pragma unroll
  for (int i = 0; i < FIRST; ++i)
    if (i < parts) first[i] = values(i);
  float top = ml.x;
  for (int i = lane + 32; i < parts; i += 32) top = fmaxf(top, part.ml[row(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.f : top;
  float acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  auto add = [&](float w, const Vec& x) {
    acc[0] = fmaf(w, x.x, acc[0]), acc[1] = fmaf(w, x.y, acc[1]);
    if constexpr (kPer == 4) acc[2] = fmaf(w, x.z, acc[2]), acc[3] = fmaf(w, x.w, acc[3]);
  };
  float l = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < parts) {
      if (i0 > 0) ml = part.ml[row(i0 + lane)];
      w = ex2_approx(ml.x - base);
      l += w * ml.y;
    }
    const int n = parts - i0 < 32 ? parts - i0 : 32;
    if (i0 == 0) {
#pragma unroll
      for (int i = 0; i < FIRST; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        if (i < parts) add(wi, first[i]);
      }
    }
#pragma unroll 8
    for (int i = i0 == 0 ? FIRST : 0; i < n; ++i) add(__shfl_sync(0xffffffffu, w, i), values(i0 + i));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const int pos = local / p.ratio, hq = j.head * p.ratio + (local - pos * p.ratio);
  const int64_t token = j.cu0 + pos;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (token * p.heads_q + hq) * DV + lane * kPer);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) dst[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[hq * p.total_q + token] = l == 0.f ? -INFINITY : (base - kPShift + log2f(l)) * 0.6931471805599453f;
}

// LONG: the call has unpacked sequences.
template <int DV, int FIRST, bool LONG>
__global__ void __launch_bounds__(256, LONG ? 4 : 0) paged_merge_kernel(const __grid_constant__ PagedMerge p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  float4 lse4 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (LONG && p.lse != nullptr) lse4 = paged_lse4(p, at);
  const bool second = static_cast<int>(blockIdx.x) >= p.set[0].blocks;
  const PagedMerge::Set& set = p.set[second ? 1 : 0];
  const int block = blockIdx.x - (second ? p.set[0].blocks : 0);
  const int piece0 = block / set.shares * set.pieces, share = block % set.shares;
  const int lane = threadIdx.x & 31;
  PagedJoin mine = {-1, 0, 0, 0};  // lane l: of the piece piece0 + l
  if (lane < set.pieces) mine = set.part.joins[piece0 + lane];
  const int rows = mine.last < 0 ? 0 : mine.rows;
  int upto = rows;  // rows of the lanes up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const int total = __shfl_sync(0xffffffffu, upto, 31);
  for (int item = 8 * share + (threadIdx.x >> 5); item < total; item += 8 * set.shares) {
    const int from = __popc(__ballot_sync(0xffffffffu, upto <= item));
    PagedJoin j;
    j.last = __shfl_sync(0xffffffffu, mine.last, from);
    j.cu0 = __shfl_sync(0xffffffffu, mine.cu0, from);
    j.head = __shfl_sync(0xffffffffu, mine.head, from);
    j.rows = __shfl_sync(0xffffffffu, rows, from);
    const int local = item - (__shfl_sync(0xffffffffu, upto, from) - j.rows);
    paged_merge_row<DV, FIRST>(p, set.part, set.rows, piece0 + from, j, local);
  }
  if constexpr (LONG) {
    if (p.lse == nullptr) return;
#pragma unroll 1
    for (;;) {
      if (lse4.x == -INFINITY) paged_nan_lse<DV>(p, 4 * at);
      if (lse4.y == -INFINITY) paged_nan_lse<DV>(p, 4 * at + 1);
      if (lse4.z == -INFINITY) paged_nan_lse<DV>(p, 4 * at + 2);
      if (lse4.w == -INFINITY) paged_nan_lse<DV>(p, 4 * at + 3);
      at += static_cast<int64_t>(gridDim.x) * blockDim.x;
      if (4 * at >= p.total_q * p.heads_q) return;
      lse4 = paged_lse4(p, at);
    }
  }
}

}  // namespace fa
