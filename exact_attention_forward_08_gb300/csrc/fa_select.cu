// fa_kv_bounds and fa_kv_select: which pages of the 8-bit cache a new token
// attends to.
//
// With hi_j and lo_j the largest and smallest key of page j in each channel, no
// key of the page scores more than sum_d max(q_d hi_jd, q_d lo_jd) against q.  Of
// the query heads that share a key head the sum of these bounds counts:
//     score_j = sum_h sum_d max(q_hd hi_jd, q_hd lo_jd) = q+ . hi_j + q- . lo_j,
//     q+ = sum_h max(q_h, 0),  q- = sum_h min(q_h, 0)
// one product of length 2 d whatever the number of query heads.
//
// Which pages have the largest scores has to be decided exactly, equal scores by
// the lowest index, and not by how fp32 rounds.  So scores are computed in fp32
// and kept with 20 bits of their fraction; their error is below a bound eps known
// from the inputs, and with T the k-th largest of them every page above T + 2 eps
// is in and every page below T - 2 eps is out.  The others, mostly none, get
// scores in fp64, where sums of products of 8-bit and 4-bit fractions are exact
// for all but extreme ranges.
//
// Three kernels: bounds of the pages with new tokens, scores of all pages, the
// choice for each token and key head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstring>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged.cuh"
#include "fa_paged_check.h"
#include "fa_paged_range.h"

namespace fa {
namespace {

// ---------------------------------------------------------------------------
// bounds
// ---------------------------------------------------------------------------

struct BoundsParams {
  const uint8_t* k;
  int64_t page_stride, head_stride;
  uint32_t token_stride;
  uint8_t* bounds;
  const int* table;
  int64_t table_stride;
  const int* seqlens;
  const int* cu;
  unsigned int* status;
  int64_t total, slots;
  int batch, heads, num_pages, max_pages, page_shift;
};

constexpr int kBoundsWarps = 8;

__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// four f16 that are e4m3 values (or NaN) as codes
__device__ __forceinline__ uint32_t f16x4_codes(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "r"(a), "r"(b));
  return r;
}

// A warp takes one head of one page: lanes hold 16 columns of every kRows-th token.
template <int D>
__global__ void __launch_bounds__(32 * kBoundsWarps) kv_bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int kChunks = D == 128 ? 8 : 4, kRows = 32 / kChunks, kAhead = 4;
  const int lane = threadIdx.x & 31;
  const int64_t most = static_cast<int64_t>(p.max_pages) << p.page_shift;
  int start, n;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < p.batch; i += gridDim.x * blockDim.x)
    if (!paged_append_range(p.cu[i], p.cu[i + 1], p.seqlens[i], p.total, most, start, n)) paged_error(p.status, kSitePagedSeq, i);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kBoundsWarps + (threadIdx.x >> 5);
  const int64_t slot = unit / p.heads;
  const int head = static_cast<int>(unit - slot * p.heads);
  if (slot >= p.slots) return;
  // sequence b has the places (cu[b] >> page_shift) + 2 b .., at least as many as its new tokens touch pages
  const int b = warp_search(p.batch, slot, [&](int i) { return static_cast<int64_t>(p.cu[i] >> p.page_shift) + 2 * i; });
  const int c0 = p.cu[b], len = p.seqlens[b];
  if (!paged_append_range(c0, p.cu[b + 1], len, p.total, most, start, n)) return;
  const int64_t place = slot - (static_cast<int64_t>(c0 >> p.page_shift) + 2 * b);
  const int64_t j64 = (start >> p.page_shift) + place;
  if (n == 0 || place < 0 || (j64 << p.page_shift) >= len) return;
  const int j = static_cast<int>(j64);
  const int page = p.table[b * p.table_stride + j];
  if (page < 0 || page >= p.num_pages) {
    if (head == 0 && lane == 0) paged_error(p.status, kSitePagedPage, b);
    return;
  }
  const int left = len - (j << p.page_shift);
  const int tokens = left < 1 << p.page_shift ? left : 1 << p.page_shift;
  const uint8_t* src = p.k + page * p.page_stride + head * p.head_stride;
  uint8_t* dst = p.bounds + (static_cast<int64_t>(page) * p.heads + head) * 2 * D;
#pragma unroll 1
  for (int column = (lane % kChunks) * 16; column < D; column += kChunks * 16) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[i] = 0xfc00fc00u, lo[i] = 0x7c007c00u;  // -inf, inf
    // rows behind the last are read as the last again
    for (int row0 = lane / kChunks; row0 < tokens; row0 += kRows * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int row = row0 + a * kRows < tokens ? row0 + a * kRows : tokens - 1;
        v[a] = *reinterpret_cast<const uint4*>(src + static_cast<uint64_t>(static_cast<uint32_t>(row) * p.token_stride) + column);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const uint32_t w[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f0 = e4m3x2_f16x2(w[i]), f1 = e4m3x2_hi_f16x2(w[i]);
          hi[2 * i] = max_nan(hi[2 * i], f0), hi[2 * i + 1] = max_nan(hi[2 * i + 1], f1);
          lo[2 * i] = min_nan(lo[2 * i], f0), lo[2 * i + 1] = min_nan(lo[2 * i + 1], f1);
        }
      }
    }
#pragma unroll
    for (int o = kChunks; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hi[i] = max_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      }
    if (lane < kChunks) {
      *reinterpret_cast<uint4*>(dst + column) = make_uint4(f16x4_codes(hi[0], hi[1]), f16x4_codes(hi[2], hi[3]),
                                                           f16x4_codes(hi[4], hi[5]), f16x4_codes(hi[6], hi[7]));
      *reinterpret_cast<uint4*>(dst + D + column) = make_uint4(f16x4_codes(lo[0], lo[1]), f16x4_codes(lo[2], lo[3]),
                                                               f16x4_codes(lo[4], lo[5]), f16x4_codes(lo[6], lo[7]));
    }
  }
}

template <int D>
cudaError_t bounds_launch(const BoundsParams& p, cudaStream_t stream) {
  const int64_t blocks = (p.slots * p.heads + kBoundsWarps - 1) / kBoundsWarps;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  kv_bounds_kernel<D><<<static_cast<int>(blocks), 32 * kBoundsWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------

struct SelectParams {
  const __nv_bfloat16* q;
  const uint8_t* bounds;
  const uint8_t* k_scale;
  const int* table;
  int64_t table_stride;
  const int* seqlens;
  const int* cu;
  unsigned int* status;
  uint32_t* keys;    // [total][heads][width] scores as ordered integers
  uint64_t* exact;   // the same in 64 bits, where they were needed
  uint8_t* top_e;    // [batch][heads][groups] largest scale of 8 pages
  int* lists;        // [total][heads][top]
  int* list_lens;    // [total]
  int64_t total;
  int batch, heads, ratio, num_pages, max_pages, page_shift, max_n, causal, top, first, last;
  int width, groups;  // pages and groups of 8 pages that rows are laid out for
};

constexpr int kScoreWarps = 8, kScoreThreads = 32 * kScoreWarps;
constexpr int kWarpPages = 8, kTilePages = kWarpPages * kScoreWarps;

struct SelectSeq {
  int c0, n, len, pages;  // pages 0: no scores
};
__device__ __forceinline__ SelectSeq select_seq(const SelectParams& p, int b, bool& bad) {
  SelectSeq s;
  s.c0 = p.cu[b];
  s.len = p.seqlens[b];
  bad = !paged_attend_range(s.c0, p.cu[b + 1], s.len, p.total, p.max_n, static_cast<int64_t>(p.max_pages) << p.page_shift, s.n);
  const int round = (1 << p.page_shift) - 1;
  s.pages = bad || s.n == 0 ? 0 : (s.len + round) >> p.page_shift;
  return s;
}

// A score's place in the order: the upper half of its double's bits, made ordered.  NaN counts as +inf.
__device__ __forceinline__ uint32_t score_key(double x) {
  const uint32_t h = x != x ? 0x7ff00000u : static_cast<uint32_t>(__double2hiint(x));
  return h & 0x80000000u ? ~h : h | 0x80000000u;
}
__device__ __forceinline__ double key_score(uint32_t k) {
  return __hiloint2double(static_cast<int>(k & 0x80000000u ? k ^ 0x80000000u : ~k), 0);
}
// the same of all 64 bits; both zeros are one
__device__ __forceinline__ uint64_t score_key64(double x) {
  const uint64_t h = x != x ? 0x7ff0000000000000ull : static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return h >> 63 ? ~h : h | (1ull << 63);
}

// 2^(e - 127) of an e8m0 byte; 255 is NaN
__device__ __forceinline__ double scale_double(int e) {
  return e == 255 ? __longlong_as_double(0x7ff8000000000000ll) : __longlong_as_double(static_cast<long long>(e - 127 + 1023) << 52);
}

// The power of two that brings queries whose largest biased exponent is `top` to at most 1; and its inverse.
__device__ __forceinline__ float query_down(int top) {
  return top >= 253 ? 0x1p-126f : top < 1 ? 0x1p126f : __uint_as_float(static_cast<uint32_t>(253 - top) << 23);
}
__device__ __forceinline__ double query_up(int top) {
  return top >= 253 ? 0x1p126 : top < 1 ? 0x1p-126 : __longlong_as_double(static_cast<long long>(top - 126 + 1023) << 52);
}

// D / 16 codes of a page that belong to a lane
template <int D>
struct LaneCodes {
  uint32_t w[D / 64];
};
template <int D>
__device__ __forceinline__ LaneCodes<D> load_lane_codes(const uint8_t* row, int lane) {
  LaneCodes<D> c;
  if constexpr (D == 64) {
    c.w[0] = __ldg(reinterpret_cast<const uint32_t*>(row) + lane);
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(row) + lane);
    c.w[0] = v.x, c.w[1] = v.y;
    if constexpr (D == 192) c.w[2] = __ldg(reinterpret_cast<const uint32_t*>(row + 256) + lane);
  }
  return c;
}
// the place in a page's 2 D bounds of code i of a lane
template <int D>
__device__ __forceinline__ int lane_column(int lane, int i) {
  if constexpr (D == 64) return 4 * lane + i;
  return i < 8 ? 8 * lane + i : 256 + 4 * lane + (i - 8);
}

// TOK tokens at a time.  Blocks take equal runs of the line of tiles of 64 pages
// of all sequences and heads; a warp has 8 pages, whose codes it loads together
// and multiplies lane by lane, D / 16 codes each, the sums of 8 pages crossing the
// warp in 9 exchanges.
template <int D, int TOK>
__global__ void __launch_bounds__(kScoreThreads, TOK == 1 ? 4 : 2) select_score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kCodes = D / 16;
  __shared__ float qs[TOK][2 * D];
  __shared__ int q_top[TOK];
  __shared__ long long scan[kScoreThreads], warp_sum[kScoreWarps];
  __shared__ int begin_b, begin_head, begin_tile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the run of this block ----
  auto scan_block = [&](int base) -> long long {
    long long v = 0;
    if (base + tid < p.batch) {
      bool bad;
      const SelectSeq s = select_seq(p, base + tid, bad);
      if (bad && blockIdx.x == 0) paged_error(p.status, kSitePagedSeq, base + tid);
      v = static_cast<long long>((s.pages + kTilePages - 1) / kTilePages) * p.heads;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += warp_sum[w];
    scan[tid] = v;
    __syncthreads();
    return scan[kScoreThreads - 1];
  };
  long long total = 0;
  for (int base = 0; base < p.batch; base += kScoreThreads) total += scan_block(base);
  const long long per = (total + gridDim.x - 1) / gridDim.x, x0 = per * blockIdx.x;
  const long long x1 = x0 + per < total ? x0 + per : total;
  if (x0 >= x1) return;
  long long offset = 0;
  for (int base = 0; base < p.batch; base += kScoreThreads) {
    if (p.batch > kScoreThreads) scan_block(base);
    const long long before = offset + (tid > 0 ? scan[tid - 1] : 0), upto = offset + scan[tid];
    if (before <= x0 && x0 < upto) {
      bool bad;
      const SelectSeq s = select_seq(p, base + tid, bad);
      const int tiles = (s.pages + kTilePages - 1) / kTilePages;
      begin_b = base + tid;
      begin_head = static_cast<int>((x0 - before) / tiles);
      begin_tile = static_cast<int>((x0 - before) % tiles);
    }
    offset += scan[kScoreThreads - 1];
  }
  __syncthreads();

  int b = begin_b, head = begin_head, tile = begin_tile;
  bool bad;
  SelectSeq s = select_seq(p, b, bad);
  int loaded_b = -1, loaded_head = -1, loaded_token = -1;
  for (long long x = x0; x < x1; ++x) {
    const int j0 = tile * kTilePages + warp * kWarpPages;
    const int count = s.pages - j0 < kWarpPages ? s.pages - j0 : kWarpPages;  // pages of this warp
    int entry = -1, e = 0;
    if (lane < count) {
      entry = p.table[b * p.table_stride + j0 + lane];
      if (entry < 0 || entry >= p.num_pages) {
        paged_error(p.status, kSitePagedPage, b);
        entry = -1;
      } else {
        e = p.k_scale[static_cast<int64_t>(entry) * p.heads + head];
      }
    }
    LaneCodes<D> codes[kWarpPages];
#pragma unroll
    for (int k = 0; k < kWarpPages; ++k) {
      const int page = __shfl_sync(0xffffffffu, entry, k);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) codes[k].w[i] = 0;
      if (page >= 0) codes[k] = load_lane_codes<D>(p.bounds + (static_cast<int64_t>(page) * p.heads + head) * 2 * D, lane);
    }
    if (count > 0) {
      const int top = __reduce_max_sync(0xffffffffu, e == 255 ? 0 : e);
      if (lane == 0)
        p.top_e[(static_cast<int64_t>(b) * p.heads + head) * p.groups + j0 / kWarpPages] = static_cast<uint8_t>(top);
    }

    for (int t0 = 0; t0 < s.n; t0 += TOK) {
      if (b != loaded_b || head != loaded_head || t0 != loaded_token) {
        // ---- q+ and q- of TOK tokens ----
        __syncthreads();
        for (int w = warp; w < TOK; w += kScoreWarps) {
          const bool there = t0 + w < s.n;
          const __nv_bfloat16* row = p.q + ((static_cast<int64_t>(s.c0) + t0 + w) * p.heads + head) * p.ratio * D;
          uint32_t top = 0;
          if (there)
            for (int i = lane; i < p.ratio * D / 8; i += 32) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(row) + i);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) top = max(top, max(u[k] & 0x7f80u, (u[k] >> 16) & 0x7f80u));
            }
          top = __reduce_max_sync(0xffffffffu, top) >> 7;
          if (lane == 0) q_top[w] = static_cast<int>(top);
          const float down = query_down(static_cast<int>(top));
          for (int i = lane; i < D / 2; i += 32) {
            float pos0 = 0.f, pos1 = 0.f, neg0 = 0.f, neg1 = 0.f;
            if (there)
              for (int h = 0; h < p.ratio; ++h) {
                const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(row + h * D) + i);
                const float a = __uint_as_float(u << 16) * down, c = __uint_as_float(u & 0xffff0000u) * down;
                // a NaN goes into both
                pos0 += a < 0.f ? 0.f : a, neg0 += a > 0.f ? 0.f : a;
                pos1 += c < 0.f ? 0.f : c, neg1 += c > 0.f ? 0.f : c;
              }
            *reinterpret_cast<float2*>(&qs[w][2 * i]) = make_float2(pos0, pos1);
            *reinterpret_cast<float2*>(&qs[w][D + 2 * i]) = make_float2(neg0, neg1);
          }
        }
        loaded_b = b, loaded_head = head, loaded_token = t0;
        __syncthreads();
      }
      if (count <= 0) continue;
      float q[TOK][kCodes], acc[TOK][kWarpPages];
#pragma unroll
      for (int t = 0; t < TOK; ++t)
#pragma unroll
        for (int i = 0; i < kCodes; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(&qs[t][lane_column<D>(lane, i)]);
          q[t][i] = v.x, q[t][i + 1] = v.y, q[t][i + 2] = v.z, q[t][i + 3] = v.w;
        }
#pragma unroll
      for (int k = 0; k < kWarpPages; ++k) {
        float x[kCodes];
#pragma unroll
        for (int i = 0; i < kCodes / 4; ++i) {
          const float2 f0 = f16x2_float2(e4m3x2_f16x2(codes[k].w[i])), f1 = f16x2_float2(e4m3x2_hi_f16x2(codes[k].w[i]));
          x[4 * i] = f0.x, x[4 * i + 1] = f0.y, x[4 * i + 2] = f1.x, x[4 * i + 3] = f1.y;
        }
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
          float a = x[0] * q[t][0];
#pragma unroll
          for (int i = 1; i < kCodes; ++i) a = fmaf(x[i], q[t][i], a);
          acc[t][k] = a;
        }
      }
      // lane l ends with the sum of page (l >> 4 & 1) * 4 + (l >> 3 & 1) * 2 + (l >> 2 & 1)
      const int mine = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
      const int e_mine = __shfl_sync(0xffffffffu, e, mine), entry_mine = __shfl_sync(0xffffffffu, entry, mine);
#pragma unroll
      for (int t = 0; t < TOK; ++t) {
        float(&a)[kWarpPages] = acc[t];
#pragma unroll
        for (int half = 4; half >= 1; half >>= 1) {
          const bool upper = (lane & (4 * half)) != 0;
#pragma unroll
          for (int k = 0; k < half; ++k) {
            const float give = upper ? a[k] : a[k + half];
            const float keep = upper ? a[k + half] : a[k];
            a[k] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * half);
          }
        }
        float sum = a[0];
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        if ((lane & 3) == 0 && mine < count && t0 + t < s.n) {
          const uint32_t key = entry_mine < 0 ? 0u : score_key(static_cast<double>(sum) * scale_double(e_mine) * query_up(q_top[t]));
          p.keys[((static_cast<int64_t>(s.c0) + t0 + t) * p.heads + head) * p.width + j0 + mine] = key;
        }
      }
    }
    // ---- the next tile ----
    if (x + 1 < x1 && ++tile * kTilePages >= s.pages) {
      tile = 0;
      if (++head == p.heads) {
        head = 0;
        do s = select_seq(p, ++b, bad);
        while (s.pages == 0 && b + 1 < p.batch);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the choice
// ---------------------------------------------------------------------------

constexpr int kChooseWarps = 8, kChooseThreads = 32 * kChooseWarps;
constexpr int kStagePages = 4096;  // keys of a row that are kept in shared memory

// Sum over the block; two buffers by turns, one barrier a call.
__device__ __forceinline__ int block_sum(int v, int (*buffer)[kChooseWarps], int& turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) buffer[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kChooseWarps; ++w) sum += buffer[turn][w];
  turn ^= 1;
  return sum;
}

// A block takes one token and key head.
template <int D>
__global__ void __launch_bounds__(kChooseThreads) select_choose_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t stage[kStagePages];
  __shared__ double qd[2 * D];
  __shared__ int sums[2][kChooseWarps];
  __shared__ uint32_t least[kChooseWarps], most[kChooseWarps];
  __shared__ uint64_t least64[kChooseWarps], most64[kChooseWarps];
  __shared__ float q_sum[kChooseWarps];
  __shared__ int warp_count[kChooseWarps], warp_ties[kChooseWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int turn = 0;
  const int64_t unit = blockIdx.x;
  const int64_t t = unit / p.heads;
  const int head = static_cast<int>(unit - t * p.heads);

  const int b = warp_search(p.batch, t, [&](int i) { return p.cu[i]; });
  bool bad;
  const SelectSeq s = select_seq(p, b, bad);
  if (bad || t < s.c0 || t >= s.c0 + s.n) {  // of no sequence: left as it is
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  int seen = s.len;
  if (p.causal) {
    seen = s.len - s.n + static_cast<int>(t - s.c0) + 1;
    seen = seen < 0 ? 0 : seen;
  }
  const int pages = (seen + (1 << p.page_shift) - 1) >> p.page_shift;
  const int count = pages < p.top ? pages : p.top;
  int* out = p.lists + unit * p.top;
  if (head == 0 && tid == 0) p.list_lens[t] = seen - ((pages - count) << p.page_shift);
  const int* row = p.table + b * p.table_stride;
  auto listed = [&](int j) {
    const int page = row[j];
    return page >= 0 && page < p.num_pages ? page : -1;
  };
  for (int i = count + tid; i < p.top; i += kChooseThreads) out[i] = -1;
  if (pages <= p.top) {
    for (int i = tid; i < pages; i += kChooseThreads) out[i] = listed(i);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // pages first .. end - 1 compete for k places, which are fewer
  const int end = pages - p.last, k = p.top - p.first - p.last;

  // ---- q+ and q- in 64 bits, and the bound of a score's error ----
  {
    const __nv_bfloat16* q = p.q + unit * p.ratio * D;
    float part = 0.f;
    for (int i = tid; i < D; i += kChooseThreads) {
      double pos = 0.0, neg = 0.0;
      for (int h = 0; h < p.ratio; ++h) {
        const float a = __bfloat162float(q[h * D + i]);
        pos += a < 0.f ? 0.0 : static_cast<double>(a), neg += a > 0.f ? 0.0 : static_cast<double>(a);
      }
      qd[i] = pos, qd[D + i] = neg;
      part += __double2float_ru(pos) - __double2float_rd(neg);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0) q_sum[warp] = part;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are there
  const uint32_t* keys = p.keys + unit * p.width;
  uint32_t low = 0xffffffffu, high = 0;
  const bool staged = pages <= kStagePages;
  for (int j = p.first + tid; j < end; j += kChooseThreads) {
    const uint32_t x = __ldcg(keys + j);
    if (staged) stage[j] = x;
    low = min(low, x), high = max(high, x);
  }
  int top_e = 0;
  const uint8_t* es = p.top_e + (static_cast<int64_t>(b) * p.heads + head) * p.groups;
  for (int i = tid; i < (pages + kWarpPages - 1) / kWarpPages; i += kChooseThreads) top_e = max(top_e, static_cast<int>(__ldcg(es + i)));
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  top_e = __reduce_max_sync(0xffffffffu, top_e);
  if (lane == 0) least[warp] = low, most[warp] = high, warp_count[warp] = top_e;
  __syncthreads();
  double size = 0.0;
#pragma unroll
  for (int w = 0; w < kChooseWarps; ++w) {
    low = min(low, least[w]), high = max(high, most[w]);
    top_e = max(top_e, warp_count[w]);
    size += q_sum[w];
  }
  auto key = [&](int j) { return staged ? stage[j] : __ldcg(keys + j); };
  // No score is larger than `size`.  Of it, the sums of q+ and q- are off by `ratio` roundings of 2^-24, the products
  // and their sum by 12 + 5, and the key drops what is below 2^-20; a few more for the rounding of `size` itself.
  size *= 448.0 * scale_double(top_e);
  const double margin = 2.0 * size * ((p.ratio + 24) * 0x1p-24 + 0x1p-20);

  // ---- the least key of the k largest: [lo, hi) keeps count(>= lo) >= k > count(>= hi) ----
  uint32_t lo = low, hi = high;  // hi: one below it, so that it fits
  bool split = false;
  int at_least = end - p.first;
  while (k > 0 && !split && lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2 + 1;
    int n = 0;
    for (int j = p.first + tid; j < end; j += kChooseThreads) n += key(j) >= mid;
    n = block_sum(n, sums, turn);
    if (n >= k) lo = mid, at_least = n, split = n == k;
    else hi = mid - 1;
  }
  uint32_t cut = lo;  // in from here on, if nothing is near
  if (k == 0) cut = 0xffffffffu, at_least = 0;
  bool close = k > 0 && at_least != k;
  double t_value = key_score(cut);
  if (k > 0 && at_least == k) {
    uint32_t in = 0xffffffffu, below = 0;
    for (int j = p.first + tid; j < end; j += kChooseThreads) {
      const uint32_t x = key(j);
      if (x >= cut) in = min(in, x);
      else below = max(below, x);
    }
    in = __reduce_min_sync(0xffffffffu, in);
    below = __reduce_max_sync(0xffffffffu, below);
    __syncthreads();
    if (lane == 0) least[warp] = in, most[warp] = below;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kChooseWarps; ++w) in = min(in, least[w]), below = max(below, most[w]);
    t_value = key_score(in);
    close = !(key_score(below) < t_value - margin);
  }

  // ---- pages too near to tell get scores in 64 bits ----
  const double sure_in = t_value + margin, sure_out = t_value - margin;
  auto near = [&](int j) {
    const double x = key_score(key(j));
    return !(x > sure_in) && !(x < sure_out);
  };
  uint64_t* exact = p.exact + unit * p.width;
  uint64_t cut64 = 0;
  int ties = 0;  // of the pages at cut64, so many are in
  if (close) {
    int in = 0;
    uint64_t low64 = ~0ull, high64 = 0;
    for (int j0 = p.first + warp * 32; j0 < end; j0 += kChooseThreads) {
      const int j = j0 + lane;
      const bool is_near = j < end && near(j);
      in += j < end && !is_near && key_score(key(j)) > sure_in;
      uint32_t todo = __ballot_sync(0xffffffffu, is_near);
      while (todo != 0) {
        const int at = j0 + __ffs(todo) - 1;
        todo &= todo - 1;
        const int page = listed(at);
        double sum = 0.0;
        if (page >= 0) {
          const int64_t ph = static_cast<int64_t>(page) * p.heads + head;
          const uint8_t* codes = p.bounds + ph * 2 * D;
          for (int i = lane; i < D / 2; i += 32) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
            const float2 f0 = f16x2_float2(e4m3x2_f16x2(w)), f1 = f16x2_float2(e4m3x2_hi_f16x2(w));
            sum += qd[4 * i] * f0.x + qd[4 * i + 1] * f0.y + qd[4 * i + 2] * f1.x + qd[4 * i + 3] * f1.y;
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          sum *= scale_double(p.k_scale[ph]);
        } else {
          sum = -__longlong_as_double(0x7ff0000000000000ll);
        }
        const uint64_t x = score_key64(sum);
        low64 = x < low64 ? x : low64, high64 = x > high64 ? x : high64;
        if (lane == 0) exact[at] = x;
      }
    }
    in = block_sum(in, sums, turn);  // its barrier: the stores above are there for the block
    if (lane == 0) least64[warp] = low64, most64[warp] = high64;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kChooseWarps; ++w) {
      low64 = least64[w] < low64 ? least64[w] : low64;
      high64 = most64[w] > high64 ? most64[w] : high64;
    }
    const int need = k - in;  // 1 at least, and no more than are near
    auto count64 = [&](uint64_t from) {
      int n = 0;
      for (int j = p.first + tid; j < end; j += kChooseThreads) n += near(j) && exact[j] >= from;
      return block_sum(n, sums, turn);
    };
    int n = count64(low64);
    bool found = n == need;
    uint64_t lo64 = low64, hi64 = high64;
    while (!found && lo64 < hi64) {
      const uint64_t mid = lo64 + (hi64 - lo64) / 2 + 1;
      const int m = count64(mid);
      if (m >= need) lo64 = mid, n = m, found = m == need;
      else hi64 = mid - 1;
    }
    cut64 = lo64;
    ties = INT_MAX;
    if (n != need) ties = need - count64(lo64 + 1);  // lo64 is a score of several pages
  }

  // ---- the chosen pages in order: a warp counts, then writes, a run of pages ----
  auto state = [&](int j) {  // 2: in, 1: a tie, 0: out
    if (j < p.first || j >= end) return 2;
    if (!close) return key(j) >= cut ? 2 : 0;
    if (!near(j)) return key_score(key(j)) > sure_in ? 2 : 0;
    const uint64_t x = exact[j];
    return x > cut64 ? 2 : x == cut64 ? (ties == INT_MAX ? 2 : 1) : 0;
  };
  const int per = ((pages + kChooseThreads - 1) / kChooseThreads) * 32;  // pages of a warp
  const int j_begin = warp * per, j_end = j_begin + per < pages ? j_begin + per : pages;
  int sure = 0, tied = 0;
  for (int j0 = j_begin; j0 < j_end; j0 += 32) {
    const int x = j0 + lane < j_end ? state(j0 + lane) : 0;
    sure += __popc(__ballot_sync(0xffffffffu, x == 2));
    tied += __popc(__ballot_sync(0xffffffffu, x == 1));
  }
  __syncthreads();
  if (lane == 0) warp_count[warp] = sure, warp_ties[warp] = tied;
  __syncthreads();
  int at = 0, ties_before = 0;
  for (int w = 0; w < warp; ++w) {
    const int left = ties - ties_before;
    at += warp_count[w] + (warp_ties[w] < left ? warp_ties[w] : left > 0 ? left : 0);
    ties_before += warp_ties[w];
  }
  for (int j0 = j_begin; j0 < j_end; j0 += 32) {
    const int x = j0 + lane < j_end ? state(j0 + lane) : 0;
    const uint32_t tie_mask = __ballot_sync(0xffffffffu, x == 1);
    const uint32_t below = (1u << lane) - 1;
    const bool in = x == 2 || (x == 1 && ties_before + __popc(tie_mask & below) < ties);
    const uint32_t mask = __ballot_sync(0xffffffffu, in);
    const int place = at + __popc(mask & below);
    if (in && place < p.top) out[place] = listed(j0 + lane);
    at += __popc(mask);
    ties_before += __popc(tie_mask);
  }
}

struct SelectWorkspace {
  size_t keys, exact, top_e, bytes;
};
SelectWorkspace select_workspace(int batch, int64_t total, int heads, int max_pages) {
  SelectWorkspace w;
  const size_t cells = static_cast<size_t>(total) * heads * max_pages;
  w.keys = 0;
  w.exact = up256(cells * sizeof(uint32_t));
  w.top_e = w.exact + up256(cells * sizeof(uint64_t));
  w.bytes = w.top_e + up256(static_cast<size_t>(batch) * heads * ((max_pages + kWarpPages - 1) / kWarpPages));
  return w;
}

template <int D>
int select_launch(const SelectParams& p, int sms, cudaStream_t stream) {
  const int64_t tiles = static_cast<int64_t>(p.batch) * p.heads * ((p.max_pages + kTilePages - 1) / kTilePages);
  const int64_t most = static_cast<int64_t>(sms) * (p.max_n == 1 ? 4 : 2);
  const int grid = static_cast<int>(tiles < most ? tiles : most);
  if (p.max_n == 1) select_score_kernel<D, 1><<<grid, kScoreThreads, 0, stream>>>(p);
  else select_score_kernel<D, 4><<<grid, kScoreThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(p.total * p.heads), 1, 1);
  cfg.blockDim = dim3(kChooseThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_choose_kernel<D>, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

bool page_size_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_kv_bounds(const fa_kv_cache* cache, void* k_bounds, const int* cu_seqlens, int batch, int64_t total,
                 fa_stream_t stream_) {
  if (cache == nullptr) return FA_ERR_INVALID_ARG;
  fa_kv_cache c = *cache;  // of the keys only: the values' fields are not looked at
  c.d_v = 64;
  for (int i = 0; i < 3; ++i) c.v_stride[i] = c.k_stride[i];
  int rc = check_cache(&c);
  if (rc != FA_OK) return rc;
  if (batch < 0 || batch > kMaxBatch || total < 0 || total >= (int64_t(1) << 31)) return FA_ERR_INVALID_ARG;
  if (batch == 0 || total == 0) return FA_OK;
  if (c.k == nullptr || c.block_table == nullptr || c.seqlens_k == nullptr || k_bounds == nullptr || cu_seqlens == nullptr)
    return FA_ERR_INVALID_ARG;
  if (!aligned(c.k, 16) || !aligned(k_bounds, 16) || !aligned(c.block_table, 4) || !aligned(c.seqlens_k, 4) ||
      !aligned(cu_seqlens, 4))
    return FA_ERR_INVALID_ARG;
  HostDevice host;
  rc = host_device(&host);
  if (rc != FA_OK) return rc;
  if (!host_is_device_ptr(c.k, host.dev) || !host_is_device_ptr(c.block_table, host.dev) ||
      !host_is_device_ptr(c.seqlens_k, host.dev) || !host_is_device_ptr(k_bounds, host.dev) ||
      !host_is_device_ptr(cu_seqlens, host.dev))
    return FA_ERR_INVALID_ARG;
  BoundsParams p;
  std::memset(&p, 0, sizeof(p));
  p.k = static_cast<const uint8_t*>(c.k);
  p.page_stride = c.k_stride[0];
  p.head_stride = c.k_stride[1];
  p.token_stride = static_cast<uint32_t>(c.k_stride[2]);
  p.bounds = static_cast<uint8_t*>(k_bounds);
  p.table = c.block_table;
  p.table_stride = c.table_stride;
  p.seqlens = c.seqlens_k;
  p.cu = cu_seqlens;
  p.status = host.status;
  p.total = total;
  p.batch = batch;
  p.heads = c.heads_kv;
  p.num_pages = c.num_pages;
  p.max_pages = c.max_pages;
  p.page_shift = page_shift(c.page_size);
  p.slots = (total >> p.page_shift) + 2 * static_cast<int64_t>(batch);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const cudaError_t e = c.d_qk == 64    ? bounds_launch<64>(p, stream)
                        : c.d_qk == 128 ? bounds_launch<128>(p, stream)
                                        : bounds_launch<192>(p, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_kv_select_workspace_size(int batch, int64_t total_q, int heads_kv, int max_pages) {
  if (batch < 0 || total_q < 0 || heads_kv < 1 || max_pages < 1) return 0;
  return select_workspace(batch, total_q, heads_kv, max_pages).bytes;
}

int fa_kv_select(const void* q, const void* k_bounds, const uint8_t* k_scale, const int* block_table,
                 int64_t table_stride, const int* seqlens_k, const int* cu_seqlens_q, int batch, int64_t total_q,
                 int max_seqlen_q, int heads_q, int heads_kv, int d_qk, int num_pages, int page_size, int max_pages,
                 int causal, int top, int keep_first, int keep_last, int* lists, int* list_lens, void* workspace,
                 size_t workspace_bytes, fa_stream_t stream_) {
  if (d_qk != 64 && d_qk != 128 && d_qk != 192) return FA_ERR_UNSUPPORTED;
  if (!page_size_ok(page_size)) return FA_ERR_UNSUPPORTED;
  if (batch < 0 || batch > kMaxBatch || total_q < 0 || total_q >= (int64_t(1) << 31) || max_seqlen_q < 0)
    return FA_ERR_INVALID_ARG;
  if (heads_kv < 1 || heads_q < 1 || heads_q % heads_kv != 0 || heads_q > 65536) return FA_ERR_INVALID_ARG;
  if (num_pages < 1 || max_pages < 1 || table_stride < max_pages ||
      static_cast<int64_t>(max_pages) * page_size > (int64_t(1) << 30))
    return FA_ERR_INVALID_ARG;
  if (keep_first < 0 || keep_last < 1 || top < 1 || static_cast<int64_t>(keep_first) + keep_last > top || top > 1 << 24)
    return FA_ERR_INVALID_ARG;
  if (batch == 0 || total_q == 0) return FA_OK;
  if (max_seqlen_q < 1 || total_q * heads_kv >= (int64_t(1) << 31)) return FA_ERR_INVALID_ARG;
  if (q == nullptr || k_bounds == nullptr || k_scale == nullptr || block_table == nullptr || seqlens_k == nullptr ||
      cu_seqlens_q == nullptr || lists == nullptr || list_lens == nullptr || workspace == nullptr)
    return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_bounds, 16) || !aligned(workspace, 16) || !aligned(block_table, 4) ||
      !aligned(seqlens_k, 4) || !aligned(cu_seqlens_q, 4) || !aligned(lists, 4) || !aligned(list_lens, 4))
    return FA_ERR_INVALID_ARG;
  const SelectWorkspace w = select_workspace(batch, total_q, heads_kv, max_pages);
  if (workspace_bytes < w.bytes) return FA_ERR_INVALID_ARG;
  HostDevice host;
  const int rc = host_device(&host);
  if (rc != FA_OK) return rc;
  for (const void* x : {q, k_bounds, static_cast<const void*>(k_scale), static_cast<const void*>(block_table),
                        static_cast<const void*>(seqlens_k), static_cast<const void*>(cu_seqlens_q),
                        static_cast<const void*>(lists), static_cast<const void*>(list_lens),
                        static_cast<const void*>(workspace)})
    if (!host_is_device_ptr(x, host.dev)) return FA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SelectParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.bounds = static_cast<const uint8_t*>(k_bounds);
  p.k_scale = k_scale;
  p.table = block_table;
  p.table_stride = table_stride;
  p.seqlens = seqlens_k;
  p.cu = cu_seqlens_q;
  p.status = host.status;
  p.keys = reinterpret_cast<uint32_t*>(ws + w.keys);
  p.exact = reinterpret_cast<uint64_t*>(ws + w.exact);
  p.top_e = ws + w.top_e;
  p.lists = lists;
  p.list_lens = list_lens;
  p.total = total_q;
  p.batch = batch;
  p.heads = heads_kv;
  p.ratio = heads_q / heads_kv;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.page_shift = page_shift(page_size);
  p.max_n = max_seqlen_q;
  p.causal = causal ? 1 : 0;
  p.top = top;
  p.first = keep_first;
  p.last = keep_last;
  p.width = max_pages;
  p.groups = (max_pages + kWarpPages - 1) / kWarpPages;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (d_qk == 64) return select_launch<64>(p, host.sms, stream);
  if (d_qk == 128) return select_launch<128>(p, host.sms, stream);
  return select_launch<192>(p, host.sms, stream);
}

}  // extern "C"
