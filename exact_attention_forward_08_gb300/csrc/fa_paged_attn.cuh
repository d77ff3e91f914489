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
// Codes become f16 exactly; a query row is divided by a power of two first so
// that f16 holds its bf16 values (below 2^-24 of the row's largest they round);
// P is rounded to f16 scaled by 2^7, 11 bits where bf16 would keep 8.
// Scores, maxima, sums and O stay in fp32.
//
// Work: a tile is 32 tokens of one key/value head; the tiles of all sequences,
// heads and row groups form one line that is cut into equal pieces, one for
// each team of warps (a team is 1 to 4 warps with 8 or 16 rows each that read
// the same tiles).  A team streams its piece through its own ring of stages
// (TMA, one mbarrier a stage), independently of the others.  A (sequence, head)
// that lies in one piece is written out at once, one that is cut leaves
// unnormalised parts that paged_merge_kernel joins.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_paged.cuh"
#include "ptx.cuh"

namespace fa {

struct PagedParams {
  CUtensorMap tm_k, tm_v;  // (d, token, head, page) of codes
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const int* table;
  int64_t table_stride;
  const int* seqlens;
  const int* cu;
  unsigned int* status;
  float* part_o;   // [2 * pieces][rows][DV]
  float2* part_ml;  // [2 * pieces][rows] {reference, sum}
  struct PagedJoin* joins;  // [pieces]
  int64_t total_q;
  unsigned long long timeout_ns;
  int batch, heads_q, heads_kv, ratio, num_pages, max_pages, page_shift, causal;
  int max_n;      // longest sequence of new tokens allowed
  int row_limit;  // sequences with more rows (new tokens x ratio) are not this kernel's
  float scale_log2;
};

// A cut (sequence, head, row group) that starts in a piece and ends in piece `last`.
struct PagedJoin {
  int last;  // -1: none
  int cu0, head, row0, rows, pad;
};

constexpr int kPagedWarps = 8;
constexpr int kPagedThreads = kPagedWarps * 32;
constexpr int kTileTokens = 32;
constexpr int kMinTiles = 2;          // a piece is not cut smaller
constexpr float kPShift = 7.f;        // P is scaled by 2^7: f16 then holds weights down to 2^-31
constexpr float kRefLag = 8.f;        // the reference follows the maximum when it lags by more (log2 units)

template <int DQK, int DV, int NT, int TW>
struct PagedShape {
  static constexpr int kRows = 8 * NT * TW;  // rows of a team
  static constexpr int kTeams = kPagedWarps / TW;
  static constexpr int kTileK = kTileTokens * DQK, kTileV = kTileTokens * DV;
  static constexpr int kTileBytes = kTileK + kTileV;
  static constexpr int kSmemTiles = (200 * 1024) / kTileBytes / kPagedWarps * kPagedWarps;
  static constexpr int kStages = kSmemTiles / kTeams;
  static constexpr int kLag = TW > 1 ? 1 : 0;  // tiles between reading a stage and refilling it
  static constexpr int kBytes = kSmemTiles * kTileBytes + 1024;
};

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// shared-memory offset of 16-byte chunk `chunk` of row `row`: the layouts that
// TMA writes with 128-byte rows (128-byte swizzle) and 64-byte rows (64-byte)
__device__ __forceinline__ uint32_t sw128(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }
__device__ __forceinline__ uint32_t sw64(int row, int chunk) { return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4); }

// K chunk (16 codes) number `step` (0 .. DQK/64 - 1) of lane column c: 128-byte rows hold chunk 2 c + step,
// 64-byte sub-tiles chunk c of sub-tile `step`.  The same rule gives the query columns below.
template <int DQK>
__device__ __forceinline__ uint32_t k_offset(int row, int c, int step) {
  if constexpr (DQK == 128) return sw128(row, 2 * c + step);
  return step * (kTileTokens * 64) + sw64(row, c);
}
template <int DQK>
__device__ __forceinline__ int k_column(int c, int step) {
  return DQK == 128 ? 16 * (2 * c + step) : 64 * step + 16 * c;
}

// One sequence as the kernel sees it.
struct PagedSeq {
  int cu0, n, len;
  int rows, groups, tiles;  // new tokens x ratio, row groups, tiles of 32 tokens
  bool bad;
};

template <int ROWS>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  PagedSeq s;
  s.cu0 = p.cu[b];
  const int c1 = p.cu[b + 1];
  s.len = p.seqlens[b];
  s.n = c1 - s.cu0;
  s.bad = s.cu0 < 0 || c1 < s.cu0 || c1 > p.total_q || s.n > p.max_n || s.len < 0 ||
          s.len > (static_cast<int64_t>(p.max_pages) << p.page_shift);
  const int64_t rows = s.bad ? 0 : static_cast<int64_t>(s.n) * p.ratio;
  s.rows = rows > p.row_limit ? 0 : static_cast<int>(rows);
  s.groups = (s.rows + ROWS - 1) / ROWS;
  s.tiles = s.len > 0 ? (s.len + kTileTokens - 1) / kTileTokens : 1;  // without a key: one tile that is masked
  return s;
}

// A place on the line of tiles.
struct PagedCursor {
  PagedSeq s;
  int b, head, group, tile;
};

template <int ROWS>
__device__ __forceinline__ void paged_next_unit(const PagedParams& p, PagedCursor& c) {
  c.tile = 0;
  if (++c.group < c.s.groups) return;
  c.group = 0;
  if (++c.head < p.heads_kv) return;
  c.head = 0;
  do {
    if (c.b + 1 >= p.batch) return;
    c.s = paged_seq<ROWS>(p, ++c.b);
  } while (c.s.groups == 0);
}

template <int DQK, int DV, int NT, int TW>
__global__ void __launch_bounds__(kPagedThreads, 1) paged_attn_kernel(const __grid_constant__ PagedParams p) {
  using Shape = PagedShape<DQK, DV, NT, TW>;
  constexpr int kSteps = DQK / 64;       // 64-column groups of K
  constexpr int kVWords = DV / 32;       // 32-bit words of V codes a lane reads per token
  constexpr int kVTiles = DV / 16;       // m16 tiles of O^T
  constexpr int kTeams = Shape::kTeams, kStages = Shape::kStages, kRows = Shape::kRows;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kTeams * kStages];
  __shared__ float4 meta[kTeams * kStages];  // {K scale of tokens 0-15, 16-31, V scale of the same}
  __shared__ long long scan[kPagedThreads];
  __shared__ long long warp_sum[kPagedWarps];
  __shared__ int abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int team = warp / TW, sub = warp % TW;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + team * kStages * Shape::kTileBytes;
  const uint32_t full0 = smem_u32(&bars[team * 2 * kStages]), empty0 = full0 + 8 * kStages;
  WaitCtx wc{&abort_flag, p.status, p.timeout_ns};

  // let the merge kernel's blocks take their places early: they wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < kTeams; ++i)
      for (int s = 0; s < kStages; ++s) {
        mbar_init(smem_u32(&bars[i * 2 * kStages + s]), 1);
        mbar_init(smem_u32(&bars[i * 2 * kStages + kStages + s]), TW);
      }
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }

  // ---- the line of tiles: its length, and where this team's piece begins ----
  auto scan_block = [&](int base) -> long long {  // inclusive scan of 256 sequences' tiles into scan[]
    const int b = base + tid;
    long long v = 0;
    if (b < p.batch) {
      const PagedSeq s = paged_seq<kRows>(p, b);
      if (s.bad && blockIdx.x == 0) paged_error(p.status, kSitePagedSeq, b);
      v = static_cast<long long>(s.groups) * s.tiles * p.heads_kv;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    scan[tid] = before + v;
    __syncthreads();
    return scan[kPagedThreads - 1];
  };
  long long total = 0;
  for (int base = 0; base < p.batch; base += kPagedThreads) total += scan_block(base);
  const long long pieces = static_cast<long long>(gridDim.x) * kTeams;
  long long per = (total + pieces - 1) / pieces;
  if (per < kMinTiles) per = kMinTiles;
  const long long used = (total + per - 1) / per;  // pieces that hold tiles
  const int teams_used = static_cast<int>((used + gridDim.x - 1) / gridDim.x);  // of a block
  const long long piece = static_cast<long long>(blockIdx.x) * teams_used + team;
  const bool active = team < teams_used && piece < used;
  const long long begin = piece * per;
  const int count = !active ? 0 : static_cast<int>(total - begin < per ? total - begin : per);

  PagedCursor cur;
  cur.b = -1;
  long long offset = 0;
  for (int base = 0; base < p.batch; base += kPagedThreads) {
    if (p.batch > kPagedThreads) scan_block(base);
    const long long sum = scan[kPagedThreads - 1];
    if (active && begin >= offset && begin < offset + sum) {
      const long long x = begin - offset;  // the first sequence whose inclusive sum exceeds x
      int lo = 0, hi = kPagedThreads - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (scan[mid] > x) hi = mid;
        else lo = mid + 1;
      }
      cur.b = base + lo;
      cur.s = paged_seq<kRows>(p, cur.b);
      const long long in = x - (lo > 0 ? scan[lo - 1] : 0);
      const int unit = static_cast<int>(in / cur.s.tiles);
      cur.tile = static_cast<int>(in - static_cast<long long>(unit) * cur.s.tiles);
      cur.head = unit / cur.s.groups;
      cur.group = unit - cur.head * cur.s.groups;
    }
    offset += sum;
    if (p.batch > kPagedThreads) __syncthreads();
  }
  __syncthreads();  // barriers are initialised

  // every piece that could hold something says first that it leaves nothing to join
  if (sub == 0 && lane == 0) {
    // the pieces of this launch are numbered 0 .. gridDim.x * kTeams - 1; those that no team of the
    // assignment above owns are cleared by the team with the same place in plain order
    const int64_t own = active ? piece : -1;
    const int64_t plain = static_cast<int64_t>(blockIdx.x) * kTeams + team;
    if (own >= 0) p.joins[own].last = -1;
    if (plain >= used) p.joins[plain].last = -1;
  }
  if (!active || count == 0) return;

  // ---- producer: the warp walks the line `kStages` tiles ahead ----
  PagedCursor pc = cur;
  int page_base = -1, page_entry = 0, page_b = -1, page_head = -1;
  float page_ks = 0.f, page_vs = 0.f;
  int issued = 0;
  const int page_tokens = 1 << p.page_shift;
  const int box_rows = page_tokens < kTileTokens ? page_tokens : kTileTokens;

  auto issue = [&]() {  // the next tile into its stage (warp-uniform; the team's first warp only)
    const int stage = issued % kStages;
    const uint32_t full = full0 + 8 * stage;
    const uint32_t at = ring + stage * Shape::kTileBytes;
    const int token = pc.tile * kTileTokens;
    const int pages = (pc.s.len + page_tokens - 1) >> p.page_shift;
    const int first = token >> p.page_shift;
    if (pc.b != page_b || pc.head != page_head || first < page_base || first >= page_base + 31) {
      // 32 entries of the block table and their scales, one a lane
      page_b = pc.b;
      page_head = pc.head;
      page_base = first;
      const int idx = first + lane;
      page_entry = 0;
      page_ks = page_vs = 1.f;
      if (idx < pages) {
        page_entry = p.table[pc.b * p.table_stride + idx];
        if (page_entry < 0 || page_entry >= p.num_pages) {
          paged_error(p.status, kSitePagedPage, pc.b);
          page_entry = 0;
        }
        const int64_t at_scale = static_cast<int64_t>(page_entry) * p.heads_kv + pc.head;
        const int ek = p.k_scale[at_scale], ev = p.v_scale[at_scale];
        page_ks = ev == 255 ? scale_of(255) : scale_of(ek);  // no number in either: rows that see it are NaN
        page_vs = ev == 255 ? 1.f : scale_of(ev);
      }
    }
    const int i0 = first - page_base;
    const int e0 = __shfl_sync(0xffffffffu, page_entry, i0), e1 = __shfl_sync(0xffffffffu, page_entry, i0 + 1);
    const float k0 = __shfl_sync(0xffffffffu, page_ks, i0), k1 = __shfl_sync(0xffffffffu, page_ks, i0 + 1);
    const float v0 = __shfl_sync(0xffffffffu, page_vs, i0), v1 = __shfl_sync(0xffffffffu, page_vs, i0 + 1);
    if (lane == 0) {
      const bool split = page_tokens < kTileTokens;  // two pages of 16 tokens
      meta[team * kStages + stage] = split ? make_float4(k0, k1, v0, v1) : make_float4(k0, k0, v0, v0);
      const int boxes = pc.s.len == 0 ? 0 : (split && first + 1 < pages) ? 2 : 1;
      if (boxes == 0) {
        mbar_arrive(full);
      } else {
        mbar_arrive_expect_tx(full, boxes * box_rows * (DQK + DV));
        for (int i = 0; i < boxes; ++i) {
          const int e = i == 0 ? e0 : e1;
          const int row = split ? 0 : token & (page_tokens - 1);
          if constexpr (DQK == 128) {
            tma_load_4d(at + i * 16 * 128, &p.tm_k, full, 0, row, pc.head, e);
          } else {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
              tma_load_4d(at + s * kTileTokens * 64 + i * 16 * 64, &p.tm_k, full, 64 * s, row, pc.head, e);
          }
          tma_load_4d(at + Shape::kTileK + i * 16 * DV, &p.tm_v, full, 0, row, pc.head, e);
        }
      }
    }
    __syncwarp();
    ++issued;
    if (++pc.tile == pc.s.tiles && issued < count) paged_next_unit<kRows>(p, pc);
  };

  // after a failed wait: the copies in flight land before the block's memory is given up
  auto drain = [&](int from) {
    if (sub != 0) return;
    const uint64_t t0 = globaltimer_ns();
    for (int i = from; i < issued; ++i)
      while (!mbar_try_wait(full0 + 8 * (i % kStages), (i / kStages) & 1))
        if (globaltimer_ns() - t0 > 1000000000ull) return;
  };

  if (sub == 0)
    for (int i = 0; i < kStages && i < count; ++i) issue();

  // ---- consumer ----
  uint32_t qf[NT][kSteps * 4][2];
  float qfac[NT][2], ref[NT][2], sum[NT][2];
  int limit[NT][2];
  float o[NT][kVTiles][4];
  int min_limit = 0;
  bool started_here = false;

  for (int i = 0; i < count; ++i) {
    if (i == 0 || cur.tile == 0) {
      // ---- a new (sequence, head, row group): the query rows as B fragments ----
      started_here = cur.tile == 0;
      const int row0 = cur.group * kRows + sub * 8 * NT;
      min_limit = cur.s.len;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + g;
        uint4 raw[kSteps * 2];
        if (r < cur.s.rows) {
          const int pos = r / p.ratio, hr = r - pos * p.ratio;
          const __nv_bfloat16* src =
              p.q + (static_cast<int64_t>(cur.s.cu0 + pos) * p.heads_q + cur.head * p.ratio + hr) * DQK;
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              raw[s * 2 + h] = __ldg(reinterpret_cast<const uint4*>(src + k_column<DQK>(c, s) + 8 * h));
        } else {
#pragma unroll
          for (int s = 0; s < kSteps * 2; ++s) raw[s] = make_uint4(0, 0, 0, 0);
        }
        // the row's largest exponent: its values divided by that power of two fit f16
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < kSteps * 2; ++s) {
          const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a = w[j] & 0x7f80u, b = (w[j] >> 16) & 0x7f80u;
            top = top > a ? top : a;
            top = top > b ? top : b;
          }
        }
        uint32_t y = __shfl_xor_sync(0xffffffffu, top, 1);
        top = top > y ? top : y;
        y = __shfl_xor_sync(0xffffffffu, top, 2);
        top = top > y ? top : y;
        int ex = static_cast<int>(top >> 7);  // biased
        ex = ex == 0 || ex == 255 ? 127 : ex;  // a row of zeros, or one that holds no numbers
        const float down = scale_of(254 - ex);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = raw[s * 2 + h];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)  // word j holds columns 8 h + 2 j, + 1: step (8 h + 2 j) / 4, half j & 1
              qf[nt][s * 4 + h * 2 + (j >> 1)][j & 1] =
                  pack_f16x2(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xffff0000u) * down);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // this lane's columns of S^T are rows 2 c and 2 c + 1
          const int e = __shfl_sync(0xffffffffu, ex, (2 * c + k) * 4);
          qfac[nt][k] = p.scale_log2 * scale_of(e);
          ref[nt][k] = -INFINITY;
          sum[nt][k] = 0.f;
          const int rr = row0 + nt * 8 + 2 * c + k;
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

    const int stage = i % kStages;
    if (!mbar_wait(full0 + 8 * stage, (i / kStages) & 1, wc, kSitePagedWait)) {
      drain(i);
      return;
    }
    const uint32_t tk = ring + stage * Shape::kTileBytes, tv = tk + Shape::kTileK;
    const float4 m = meta[team * kStages + stage];
    const int token0 = cur.tile * kTileTokens;
    const bool masked = token0 + kTileTokens > min_limit;

    // S^T of 2 x 16 tokens
    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[mt][nt][k] = 0.f;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const uint4 ra = lds128(tk + k_offset<DQK>(16 * mt + g, c, st));
        const uint4 rb = lds128(tk + k_offset<DQK>(16 * mt + 8 + g, c, st));
        const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = e4m3x2_f16x2(wa[j]), a1 = e4m3x2_f16x2(wb[j]);
          const uint32_t a2 = e4m3x2_hi_f16x2(wa[j]), a3 = e4m3x2_hi_f16x2(wb[j]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(s[mt][nt], a0, a1, a2, a3, qf[nt][st * 4 + j][0], qf[nt][st * 4 + j][1]);
        }
      }
    }

    // V codes of this lane: tokens 16 mt + {2 c, 2 c + 1, 2 c + 8, 2 c + 9}, columns DV / 8 * g ..
    uint32_t vw[2][4][kVWords];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 16 * mt + 2 * c + (t & 1) + (t >> 1) * 8;
        if constexpr (DV == 128) {
          const uint4 v = lds128(tv + sw128(row, g));
          vw[mt][t][0] = v.x, vw[mt][t][1] = v.y, vw[mt][t][2] = v.z, vw[mt][t][3] = v.w;
        } else {
          const uint2 v = lds64(tv + sw64(row, g >> 1) + (g & 1) * 8);
          vw[mt][t][0] = v.x, vw[mt][t][1] = v.y;
        }
      }

    // scores in log2 units
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[mt][nt][k] *= qfac[nt][k & 1] * (mt == 0 ? m.x : m.y);

    if (masked) {
      // A hidden token has weight 0, but 0 times a value that is no number is none: tokens behind the
      // sequence's end count as 0, and a token whose values hold a NaN code counts as 0 with a NaN score,
      // which only the rows that see it take in.
      const int mine = token0 + lane;
      uint32_t nan = 0;
      if (mine < cur.s.len) {
#pragma unroll
        for (int j = 0; j < DV / 16; ++j) {
          const uint4 v = lds128(tv + (DV == 128 ? sw128(lane, j) : sw64(lane, j)));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) nan |= ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        }
      }
      const uint32_t poison = __ballot_sync(0xffffffffu, nan != 0);
      const uint32_t inside = __ballot_sync(0xffffffffu, mine < cur.s.len);
      const uint32_t keep = inside & ~poison;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int row = 16 * mt + 2 * c + (t & 1) + (t >> 1) * 8;
#pragma unroll
          for (int j = 0; j < kVWords; ++j) vw[mt][t][j] = (keep >> row) & 1 ? vw[mt][t][j] : 0u;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 16 * mt + g + (k >> 1) * 8;
            float x = (poison >> row) & 1 ? __uint_as_float(0x7fc00000u) : s[mt][nt][k];
            s[mt][nt][k] = token0 + row < limit[nt][k & 1] ? x : -INFINITY;
          }
      }
    }

    // online softmax: the reference moves only when it lags the maximum by more than 2^8
    uint32_t pf[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float alpha[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = fmaxf(fmaxf(s[0][nt][k], s[0][nt][k + 2]), fmaxf(s[1][nt][k], s[1][nt][k + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        alpha[k] = 1.f;
        if (mx > ref[nt][k] + kRefLag) {  // also from -inf
          alpha[k] = ex2_approx(ref[nt][k] - mx);
          ref[nt][k] = mx;
        }
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int v = 0; v < kVTiles; ++v) {
          o[nt][v][0] *= alpha[0], o[nt][v][1] *= alpha[1];
          o[nt][v][2] *= alpha[0], o[nt][v][3] *= alpha[1];
        }
        sum[nt][0] *= alpha[0], sum[nt][1] *= alpha[1];
      }
      const float r0 = ref[nt][0] == -INFINITY ? 0.f : ref[nt][0], r1 = ref[nt][1] == -INFINITY ? 0.f : ref[nt][1];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = ex2_approx(s[mt][nt][k] - ((k & 1) ? r1 : r0) + kPShift);
        sum[nt][0] += e[0] + e[2];
        sum[nt][1] += e[1] + e[3];
        // accumulator layout (token g, rows 2 c ..) to operand layout (tokens 2 c .., row g)
        pf[mt][nt][0] = transpose_8x8(pack_f16x2(e[0], e[1]));
        pf[mt][nt][1] = transpose_8x8(pack_f16x2(e[2], e[3]));
      }
    }

    // O^T += V^T P^T, the page's scale applied to each 16 or 32 tokens' product
    const bool two_scales = m.z != m.w;
#pragma unroll
    for (int w = 0; w < kVWords; ++w) {
      uint32_t lo[2][2], hi[2][2];  // tokens (0, 1) and (2, 3) of columns 4 w, 4 w + 1 and 4 w + 2, 4 w + 3
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          lo[mt][t] = __byte_perm(vw[mt][2 * t][w], vw[mt][2 * t + 1][w], 0x5140);
          hi[mt][t] = __byte_perm(vw[mt][2 * t][w], vw[mt][2 * t + 1][w], 0x7362);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t a[2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t pair = x == 0 ? lo[mt][t] : hi[mt][t];
            a[mt][2 * t] = e4m3x2_f16x2(pair);
            a[mt][2 * t + 1] = e4m3x2_hi_f16x2(pair);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(acc, a[0][0], a[0][1], a[0][2], a[0][3], pf[0][nt][0], pf[0][nt][1]);
          if (two_scales) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[nt][2 * w + x][k] = fmaf(acc[k], m.z, o[nt][2 * w + x][k]);
              acc[k] = 0.f;
            }
          }
          mma_f16(acc, a[1][0], a[1][1], a[1][2], a[1][3], pf[1][nt][0], pf[1][nt][1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][2 * w + x][k] = fmaf(acc[k], m.w, o[nt][2 * w + x][k]);
        }
      }
    }

    // the stage is read: refill
    __syncwarp();
    if constexpr (TW == 1) {
      if (issued < count) issue();
    } else {
      if (lane == 0) mbar_arrive(empty0 + 8 * stage);
      if (sub == 0 && issued < count && i >= Shape::kLag) {
        const int k = issued / kStages;  // times the stage was used before
        if (k > 0 && !mbar_wait(empty0 + 8 * (issued % kStages), (k - 1) & 1, wc, kSitePagedWait)) {
          drain(i + 1);
          return;
        }
        issue();
      }
    }

    // ---- the end of the unit or of the piece: write out ----
    const bool unit_end = cur.tile + 1 == cur.s.tiles;
    if (unit_end || i + 1 == count) {
      const bool whole = started_here && unit_end;
      const int64_t slot = 2 * piece + (started_here ? 1 : 0);
      if (!whole && started_here && sub == 0 && lane == 0) {
        // the rest of the unit lies in the pieces that follow
        PagedJoin j;
        j.last = static_cast<int>((begin + i + (cur.s.tiles - 1 - cur.tile)) / per);
        j.cu0 = cur.s.cu0;
        j.head = cur.head;
        j.row0 = cur.group * kRows;
        j.rows = cur.s.rows;
        j.pad = 0;
        p.joins[piece] = j;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float l = sum[nt][k];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const int local = sub * 8 * NT + nt * 8 + 2 * c + k;
          const int r = cur.group * kRows + local;
          const float rf = l != 0.f && ref[nt][k] == -INFINITY ? 0.f : ref[nt][k];
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
              float4* dst = reinterpret_cast<float4*>(p.part_o + (slot * kRows + local) * DV + g * (DV / 8));
#pragma unroll
              for (int v = 0; v < kVTiles / 2; ++v)
                dst[v] = make_float4(o[nt][2 * v][k], o[nt][2 * v][k + 2], o[nt][2 * v + 1][k], o[nt][2 * v + 1][k + 2]);
              if (g == 0) p.part_ml[slot * kRows + local] = make_float2(rf, l);
            }
          }
        }
    }
    if (++cur.tile == cur.s.tiles && i + 1 < count) paged_next_unit<kRows>(p, cur);
  }
}

// Joins the parts of the cut units: with references m_i and sums l_i of the
// parts and M = max m_i,
//     O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
// One block for each piece and 8 rows, a warp a row; parts are taken in their
// order, so the result does not depend on timing.
template <int DV, int ROWS>
__global__ void __launch_bounds__(256) paged_merge_kernel(const __grid_constant__ PagedParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kPer = DV / 32;
  const int piece = blockIdx.x;
  const PagedJoin j = p.joins[piece];
  if (j.last < 0) return;
  const int lane = threadIdx.x & 31;
  const int local = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int r = j.row0 + local;
  if (r >= j.rows) return;
  const int parts = j.last - piece + 1;
  auto slot = [&](int i) { return 2 * static_cast<int64_t>(piece + i) + (i == 0 ? 1 : 0); };
  float top = -INFINITY;
  for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_ml[slot(i) * ROWS + local].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.f : top;
  float acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  float l = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float w = 0.f;
    if (i0 + lane < parts) {
      const float2 ml = p.part_ml[slot(i0 + lane) * ROWS + local];
      w = ex2_approx(ml.x - base);
      l += w * ml.y;
    }
    const int n = parts - i0 < 32 ? parts - i0 : 32;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* src = p.part_o + (slot(i0 + i) * ROWS + local) * DV + lane * kPer;
      if constexpr (kPer == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(wi, x.x, acc[0]), acc[1] = fmaf(wi, x.y, acc[1]);
        acc[2] = fmaf(wi, x.z, acc[2]), acc[3] = fmaf(wi, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(wi, x.x, acc[0]), acc[1] = fmaf(wi, x.y, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const int pos = r / p.ratio, hq = j.head * p.ratio + (r - pos * p.ratio);
  const int64_t token = j.cu0 + pos;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + (token * p.heads_q + hq) * DV + lane * kPer);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) dst[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[hq * p.total_q + token] = l == 0.f ? -INFINITY : (base - kPShift + log2f(l)) * 0.6931471805599453f;
}

}  // namespace fa
