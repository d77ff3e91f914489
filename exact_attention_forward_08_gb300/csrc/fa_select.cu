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
// the lowest index, and not by how fp32 rounds.  So scores are computed on the
// tensor cores with sums in fp32 and kept with 20 bits of their fraction; their
// error is below a bound eps known from the inputs, and with T the k-th largest of
// them every page above T + 2 eps is in and every page below T - 2 eps is out.  The
// others, none or two or three as a rule, get scores in fp64, where sums of products
// of 8-bit and 4-bit fractions are exact for all but extreme ranges.
//
// Three kernels: bounds of the pages with new tokens, scores of all pages, the
// choice for each token and key head.  The work is a few MB and a few dozen steps
// that each wait for the one before, so latency bounds all three.  GPU time of all
// three, 32/8 heads of 128, pages of 64: one token after 131000, 15.7 us; 24
// sequences of 100 to 131000 tokens with 3 drafted ones each, 31.4 us (45 MB of
// bounds, 7 us at the copy rate).  The second with scores in FMAs: 64.6 us; with
// comparisons of scores in fp64, whose unit is slow here: 93; with score and choice
// in one kernel of clusters, which the longest sequence then holds up: 106.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstddef>
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
  const int64_t threads = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.batch; i += threads)
    if (!paged_append_range(p.cu[i], p.cu[i + 1], p.seqlens[i], p.total, most, start, n))
      paged_error(p.status, kSitePagedSeq, static_cast<int>(i));
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
int bounds_launch(const BoundsParams& p, cudaStream_t stream) {
  const int64_t blocks = (p.slots * p.heads + kBoundsWarps - 1) / kBoundsWarps;
  if (blocks > INT_MAX) return FA_ERR_INVALID_ARG;
  kv_bounds_kernel<D><<<static_cast<int>(blocks), 32 * kBoundsWarps, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// selection
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
  int* top_e;        // [batch][heads][tiles] largest scale of a tile's pages
  int* lists;        // [total][heads][top]
  int* list_lens;    // [total]
  int64_t total;
  int batch, heads, ratio, num_pages, max_pages, page_shift, max_n, causal, top, first, last;
  int tiles;     // of a sequence and head
  double error;  // of a score, in terms of the largest that it could be
};

constexpr int kSelectWarps = 8, kSelectThreads = 32 * kSelectWarps;
constexpr int kScoreBlocks = 5;    // of an SM (4: the same time)
constexpr int kChunk = 8;          // tokens whose queries a block holds
constexpr int kWarpPages = 16;     // pages of a warp
constexpr int kTilePages = kSelectWarps * kWarpPages;

struct SelectSeq {
  int c0, n, len;
};
__device__ __forceinline__ SelectSeq select_seq(const SelectParams& p, int b, bool& bad) {
  SelectSeq s;
  s.c0 = p.cu[b];
  s.len = p.seqlens[b];
  bad = !paged_attend_range(s.c0, p.cu[b + 1], s.len, p.total, p.max_n, static_cast<int64_t>(p.max_pages) << p.page_shift, s.n);
  return s;
}
// tokens that new token i of a sequence sees
__device__ __forceinline__ int select_seen(const SelectParams& p, const SelectSeq& s, int i) {
  const int seen = p.causal ? s.len - s.n + i + 1 : s.len;
  return seen < 0 ? 0 : seen;
}

// A score's place in the order: the upper half of the bits of x 2^shift as a double, made ordered.  NaN counts as
// +inf; what is subnormal in fp32 is far below the error of a score and counts as 0.
__device__ __forceinline__ uint32_t score_key(float x, int shift) {
  const uint32_t u = __float_as_uint(x), e = (u >> 23) & 0xffu;
  if (e == 0) return 0x80000000u;  // of either sign
  const uint32_t h = e == 255 ? 0x7ff00000u : ((e + static_cast<uint32_t>(1023 - 127 + shift)) << 20) | ((u & 0x7fffffu) >> 3);
  const bool negative = u >> 31 && !(e == 255 && (u & 0x7fffffu) != 0);
  return negative ? ~(h | 0x80000000u) : h | 0x80000000u;
}
__device__ __forceinline__ double key_score(uint32_t k) {
  return __hiloint2double(static_cast<int>(k & 0x80000000u ? k ^ 0x80000000u : ~k), 0);
}
// all 64 bits of a double made ordered; NaN counts as +inf, both zeros are one
__device__ __forceinline__ uint64_t order64(double x) {
  const uint64_t h = x != x ? 0x7ff0000000000000ull : static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return h >> 63 ? ~h : h | (1ull << 63);
}
// order64 of the score that a key stands for
__device__ __forceinline__ uint64_t key_order64(uint32_t k) {
  return static_cast<uint64_t>(k) << 32 | (k & 0x80000000u ? 0u : 0xffffffffu);
}

// 2^(e - 127) of an e8m0 byte; 255 is NaN
__device__ __forceinline__ double scale_double(int e) {
  return e == 255 ? __longlong_as_double(0x7ff8000000000000ll) : __longlong_as_double(static_cast<long long>(e - 127 + 1023) << 52);
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of this thread's groups of copies are under way
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sum over the block; two buffers by turns, one barrier a call.
template <int WARPS>
__device__ __forceinline__ int block_sum(int v, int (*buffer)[WARPS], int& turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) buffer[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) sum += buffer[turn][w];
  turn ^= 1;
  return sum;
}

constexpr int kTokens = 4;    // tokens of one product: a column for the upper and one for the lower part of each
constexpr int kQueryTop = 14; // q+ and q- are brought below 2^14

template <int D>
struct ScoreShared {
  static constexpr int kRow = 2 * D * 2 + 16;  // bytes of a column: neighbours fall on other banks
  alignas(16) uint8_t q[kChunk][2][kRow];      // f16 upper and lower parts of q+ and q- of each token
  alignas(16) uint8_t codes[kSelectWarps][kWarpPages][2 * D];
  int q_shift[kChunk];  // the power of two that they were divided by
  int top_e;
};

// Where 16-byte chunk `chunk` of a page's bounds lies: two rows read together meet no bank twice.
template <int D>
__device__ __forceinline__ int code_place(int row, int chunk) {
  return row * 2 * D + ((chunk ^ ((row & 1) << 2)) << 4);
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// A block takes 128 pages of a sequence and one key head, 16 a warp, whose bounds it
// asks for at once (4 KB a warp at d = 128) and keeps for all new tokens; it holds q+
// and q- of 8 tokens at a time.  The codes are exact as f16; q+ and q- are the sums
// of two f16, off by 2^-22 of themselves (2^-39 of the row's largest if that is
// more).  So a warp's 16 pages are one operand of m16n8k16 products and 4 tokens,
// an upper and a lower part each, the other, and a lane ends with both parts of a
// token's score of two pages.  The order of columns is free: a lane takes those of
// one 16-byte chunk for four products, which go to four sums.
template <int D>
__global__ void __launch_bounds__(kSelectThreads, kScoreBlocks) kv_score_kernel(const __grid_constant__ SelectParams p) {
  static_assert(D % 64 == 0, "whole steps of four products");
  using Shared = ScoreShared<D>;
  static_assert(offsetof(Shared, codes) % 16 == 0 && Shared::kRow % 16 == 0, "16-byte copies");
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t bh = blockIdx.x / p.tiles;
  const int tile = blockIdx.x - static_cast<int>(bh) * p.tiles;
  const int b = static_cast<int>(bh / p.heads), head = static_cast<int>(bh - static_cast<int64_t>(b) * p.heads);
  const int j0 = tile * kTilePages + warp * kWarpPages;
  const int* row = p.table + b * p.table_stride;
  int entry = lane < kWarpPages && j0 + lane < p.max_pages ? row[j0 + lane] : -1;  // before the length is known
  bool bad;
  const SelectSeq s = select_seq(p, b, bad);
  if (bad && tile == 0 && head == 0 && tid == 0) paged_error(p.status, kSitePagedSeq, b);
  if (bad || static_cast<int64_t>(blockIdx.y) * kChunk >= s.n) return;
  const int round = (1 << p.page_shift) - 1;
  const int pages = (select_seen(p, s, s.n - 1) + round) >> p.page_shift;  // that the last token sees
  if (pages <= p.top || tile * kTilePages >= pages) return;

  // ---- the pages ----
  if (entry < 0 || entry >= p.num_pages || j0 + lane >= pages) {
    if (lane < kWarpPages && j0 + lane < pages) paged_error(p.status, kSitePagedPage, b);
    entry = -1;
  }
  constexpr int kChunks = 2 * D / 16;
  uint8_t* const codes = &sh.codes[warp][0][0];
#pragma unroll
  for (int k = 0; k < kWarpPages * kChunks / 32; ++k) {
    const int i = 32 * k + lane, at = i / kChunks, chunk = i % kChunks;
    const int page = __shfl_sync(0xffffffffu, entry, at);
    if (page >= 0)
      copy_async16(codes + code_place<D>(at, chunk),
                   p.bounds + (static_cast<int64_t>(page) * p.heads + head) * 2 * D + chunk * 16);
  }
  copy_commit();
  const int e = entry >= 0 ? p.k_scale[static_cast<int64_t>(entry) * p.heads + head] : 0;
  if (tid == 0) sh.top_e = 0;
  const int g = lane >> 2, c = lane & 3;
  // this lane's pages of the result
  const int e_g[2] = {__shfl_sync(0xffffffffu, e, g), __shfl_sync(0xffffffffu, e, g + 8)};
  const int entry_g[2] = {__shfl_sync(0xffffffffu, entry, g), __shfl_sync(0xffffffffu, entry, g + 8)};

  bool first = true;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * kChunk; t0 < s.n; t0 += static_cast<int64_t>(gridDim.y) * kChunk) {
    const int tokens = s.n - t0 < kChunk ? static_cast<int>(s.n - t0) : kChunk;
    const int64_t first_token = s.c0 + t0;
    if (!first) __syncthreads();
    if (warp < tokens) {  // ---- q+ and q- ----
      const __nv_bfloat16* q = p.q + ((first_token + warp) * p.heads + head) * p.ratio * D;
      constexpr int kPairs = D / 64;  // pairs of columns of a lane
      float pos[kPairs][2] = {}, neg[kPairs][2] = {};
#pragma unroll 4
      for (int h = 0; h < p.ratio; ++h)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(q + h * D) + 32 * i + lane);
          const float v[2] = {__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)};
#pragma unroll
          for (int x = 0; x < 2; ++x) pos[i][x] += v[x] < 0.f ? 0.f : v[x], neg[i][x] += v[x] > 0.f ? 0.f : v[x];  // a NaN goes into both
        }
      uint32_t top = 0;  // of their bits without signs
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) top = max(top, max(__float_as_uint(pos[i][x]), __float_as_uint(neg[i][x]) & 0x7fffffffu));
      top = __reduce_max_sync(0xffffffffu, top) >> 23;
      // 2^shift brings the largest, below 2^(top - 126), to 2^14; between 2^-126 and 2^127
      int shift = kQueryTop + 126 - static_cast<int>(top);
      shift = shift > 126 ? 126 : shift;
      const float scale = __uint_as_float(static_cast<uint32_t>(shift + 127) << 23);
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
#pragma unroll
        for (int sign = 0; sign < 2; ++sign) {
          const float u = (sign ? neg[i][0] : pos[i][0]) * scale, v = (sign ? neg[i][1] : pos[i][1]) * scale;
          const __half2 upper = __floats2half2_rn(u, v);
          const float2 back = __half22float2(upper);
          const __half2 lower = __floats2half2_rn(u - back.x, v - back.y);
          const int column = sign * D + 2 * (32 * i + lane);
          *reinterpret_cast<__half2*>(&sh.q[warp][0][2 * column]) = upper;
          *reinterpret_cast<__half2*>(&sh.q[warp][1][2 * column]) = lower;
        }
      if (lane == 0) sh.q_shift[warp] = shift;
    }
    if (first) copy_wait<0>();
    first = false;
    __syncthreads();
    if (j0 >= pages) continue;
#pragma unroll 1
    for (int x0 = 0; x0 < tokens; x0 += kTokens) {
      // column g of the second operand: part g & 1 of token x0 + g / 2 (of any content behind the last)
      const uint8_t* q = &sh.q[x0 + (g >> 1)][g & 1][0];
      float acc[4] = {};
#pragma unroll 1
      for (int st = 0; st < D / 32; ++st) {
        const int chunk = 4 * st + c;
        const uint4 lo = *reinterpret_cast<const uint4*>(codes + code_place<D>(g, chunk));
        const uint4 hi = *reinterpret_cast<const uint4*>(codes + code_place<D>(g + 8, chunk));
        const uint4 q0 = *reinterpret_cast<const uint4*>(q + 32 * chunk), q1 = *reinterpret_cast<const uint4*>(q + 32 * chunk + 16);
        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
        const uint32_t wq[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        float part[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_16x8x16(part[k], e4m3x2_f16x2(wl[k]), e4m3x2_f16x2(wh[k]), e4m3x2_hi_f16x2(wl[k]), e4m3x2_hi_f16x2(wh[k]),
                      wq[2 * k], wq[2 * k + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
      }
      const int x = x0 + c;  // this lane's token
      if (x >= tokens) continue;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int j = j0 + g + 8 * half;
        if (j >= pages) break;
        const float sum = e_g[half] == 255 ? __uint_as_float(0x7fc00000u) : acc[2 * half] + acc[2 * half + 1];
        p.keys[((first_token + x) * p.heads + head) * p.max_pages + j] =
            entry_g[half] < 0 ? 0u : score_key(sum, e_g[half] - 127 - sh.q_shift[x]);
      }
    }
  }
  const int top_e = __reduce_max_sync(0xffffffffu, e == 255 ? 0 : e);
  if (lane == 0) atomicMax(&sh.top_e, top_e);
  __syncthreads();
  if (tid == 0) p.top_e[bh * p.tiles + tile] = sh.top_e;  // the same from all blocks of the tile
}

// ---- the choice ----

// Blocks for tables of up to PAGES pages: their keys are kept in shared memory, WARPS warps look at them, histograms
// have 2^BITS bins; the table's entries are kept too (ENTRIES), which saves a wait (16.3 and 15.6 us for one token after
// 131000), or not, where room for more blocks counts (141 and 151 for 2048 tokens over 160 pages).
template <int PAGES, int WARPS, int BITS, bool ENTRIES>
struct ChooseShape {
  static constexpr bool kEntries = ENTRIES;
  static constexpr int kPages = PAGES, kWarps = WARPS, kThreads = 32 * WARPS, kBinBits = BITS, kBins = 1 << BITS;
};
using ChooseSmall = ChooseShape<1024, 4, 9, false>;
using ChooseLarge = ChooseShape<4096, 8, 11, true>;

// Pages near the cut that are compared with one another; more are searched by halving.  All searched: 39.1 us instead of
// 31.5 for 24 sequences with drafts.
constexpr int kFewPages = 64;

template <class S>
struct ChooseShared {
  uint32_t stage[S::kPages];  // keys
  int entries[S::kEntries ? S::kPages : 1];  // of the table's row
  int bins[S::kBins], bin, rank, in_bin, listed, near;
  int few[kFewPages];           // pages near the cut, and their scores in 64 bits
  uint64_t few_score[kFewPages];
  double q[2 * 192];            // q+ and q- in 64 bits
  int sums[2][S::kWarps];
  uint32_t least[S::kWarps], most[S::kWarps], near_low, near_high;
  bool tied;
  uint64_t least64[S::kWarps], most64[S::kWarps];
  int count[S::kWarps], ties[S::kWarps], top_e[S::kWarps];
  float q_size[S::kWarps];
};

// A block takes one token and key head: keys from the score kernel, T from a histogram of 2048 bins (512 in the small
// blocks), pages near T, the list.  Ten barriers and as many waits for loads: 9 us for 2048 pages, 15 us where four
// blocks share an SM.  What does not depend on the scores is done while they are computed.  Of more pages than are
// staged every pass reads the keys from global memory, and pages near T, two as well as many, are searched by halving:
// the call for one token over 8188 pages takes 50.8 us, over 4094 18.1; for 24 sequences of 3 tokens 173 and 62.
template <int D, class S>
__global__ void __launch_bounds__(S::kThreads) kv_choose_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kThreads = S::kThreads, kWarps = S::kWarps, kBins = S::kBins, kBinBits = S::kBinBits;
  __shared__ ChooseShared<S> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t unit = blockIdx.x, t = unit / p.heads;
  const int head = static_cast<int>(unit - t * p.heads);
  const int b = warp_search(p.batch, t, [&](int i) { return p.cu[i]; });
  bool bad;
  const SelectSeq s = select_seq(p, b, bad);
  const bool mine = !bad && t >= s.c0 && t < s.c0 + s.n;
  const int seen = mine ? select_seen(p, s, static_cast<int>(t - s.c0)) : 0;
  const int pages = (seen + (1 << p.page_shift) - 1) >> p.page_shift;
  const int* row = p.table + (mine ? b : 0) * p.table_stride;
  const bool staged = pages <= S::kPages;
  auto listed = [&](int j) {
    const int page = S::kEntries && pages > p.top && staged ? sh.entries[j] : row[j];
    return page >= 0 && page < p.num_pages ? page : -1;
  };
  int* out = p.lists + unit * p.top;
  if (mine && head == 0 && tid == 0) p.list_lens[t] = pages > p.top ? seen - ((pages - p.top) << p.page_shift) : seen;
  if (pages <= p.top) {  // all of them; a token of no sequence is left as it is
    for (int i = tid; mine && i < p.top; i += kThreads) {
      const int page = i < pages ? listed(i) : -1;
      if (i < pages && page < 0) paged_error(p.status, kSitePagedPage, b);
      out[i] = page;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // pages first .. end - 1 compete for k places, which are fewer
  const int end = pages - p.last, k = p.top - p.first - p.last;
  const uint32_t* keys = p.keys + unit * p.max_pages;
  uint64_t* exact = p.exact + unit * p.max_pages;
  int turn = 0;
  // while scores are computed: the table's entries; q+ and q- in 64 bits, for pages whose scores are near; the sum of
  // their sizes
  if constexpr (S::kEntries)
    for (int j = tid; staged && j < pages; j += kThreads) sh.entries[j] = row[j];
  float q_size = 0.f;
  {
    const __nv_bfloat16* q = p.q + unit * p.ratio * D;
    for (int i = tid; i < D; i += kThreads) {
      double pos = 0.0, neg = 0.0;
#pragma unroll 4
      for (int h = 0; h < p.ratio; ++h) {
        const float v = __bfloat162float(q[h * D + i]);  // a NaN goes into both
        if (!(v < 0.f)) pos += static_cast<double>(v);
        if (!(v > 0.f)) neg += static_cast<double>(v);
        q_size += fabsf(v);
      }
      sh.q[i] = pos, sh.q[D + i] = neg;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) q_size += __shfl_xor_sync(0xffffffffu, q_size, o);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are there
  int top_e = 0;
  {
    const int* es = p.top_e + (static_cast<int64_t>(b) * p.heads + head) * p.tiles;
    for (int i = tid; i * kTilePages < pages; i += kThreads) top_e = max(top_e, __ldcg(es + i));
    top_e = __reduce_max_sync(0xffffffffu, top_e);
    if (lane == 0) sh.top_e[warp] = top_e, sh.q_size[warp] = q_size;
  }
  uint32_t low = 0xffffffffu, high = 0;
  for (int j = p.first + tid; k > 0 && j < end; j += kThreads) {
    const uint32_t v = __ldcg(keys + j);
    if (staged) sh.stage[j] = v;
    low = min(low, v), high = max(high, v);
  }
  auto key = [&](int j) { return staged ? sh.stage[j] : __ldcg(keys + j); };

  // ---- T, the k-th largest key: a histogram of the keys from low to high, again of the bin that holds it if that
  // holds many ----
  uint32_t near_low = 0xffffffffu, near_high = 0xffffffffu;
  bool close = false, tied = false;  // tied: the keys near T are equal scores
  int above_near = 0;                // pages
  if (k > 0) {
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) sh.least[warp] = low, sh.most[warp] = high;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) low = min(low, sh.least[w]), high = max(high, sh.most[w]);
    int rank = k;
    while (low < high) {
      const int bits = 32 - __clz(high - low), shift = bits > kBinBits ? bits - kBinBits : 0;
      for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = 0;
      __syncthreads();
      for (int j = p.first + tid; j < end; j += kThreads) {
        const uint32_t v = key(j);
        if (v >= low && v <= high) atomicAdd(&sh.bins[(v - low) >> shift], 1);
      }
      __syncthreads();
      // a thread's bins, the last thread's are the lowest; those above come from the scan
      constexpr int kMine = kBins / kThreads;
      int count[kMine], mine_count = 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i) mine_count += count[i] = sh.bins[kBins - 1 - (tid * kMine + i)];
      int upto = mine_count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) sh.count[warp] = upto;
      __syncthreads();
      for (int w = 0; w < warp; ++w) upto += sh.count[w];
      int above = upto - mine_count;
      if (above < rank && rank <= upto) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          if (above < rank && rank <= above + count[i]) {
            sh.bin = kBins - 1 - (tid * kMine + i);
            sh.rank = rank - above;
            sh.in_bin = count[i];
          }
          above += count[i];
        }
      }
      __syncthreads();
      rank = sh.rank;
      const uint32_t from = low + (static_cast<uint32_t>(sh.bin) << shift), to = from + ((1u << shift) - 1);
      high = to < from || to > high ? high : to;
      low = from;
      const int in_bin = sh.in_bin;
      if (in_bin <= 32 && low < high) {  // few: a warp finds the one that has `rank` - 1 above it
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        for (int j = p.first + tid; j < end; j += kThreads) {
          const uint32_t v = key(j);
          if (v >= low && v <= high) sh.few[atomicAdd(&sh.listed, 1)] = static_cast<int>(v);
        }
        __syncthreads();
        const uint32_t v = lane < in_bin ? static_cast<uint32_t>(sh.few[lane]) : 0u;  // every warp for itself
        int above = 0, with = 0;
        for (int i = 0; i < in_bin; ++i) {
          const uint32_t other = __shfl_sync(0xffffffffu, v, i);
          above += other > v;
          with += other >= v;
        }
        const uint32_t found = __ballot_sync(0xffffffffu, lane < in_bin && above < rank && rank <= with);
        low = high = __shfl_sync(0xffffffffu, v, __ffs(found) - 1);
      }
    }
    if (tid == 0) {
      float q_all = 0.f;
      for (int w = 0; w < kWarps; ++w) q_all += sh.q_size[w], top_e = max(top_e, sh.top_e[w]);
      // No score is larger than `size`; computed ones are off by `error` of it at most.  Queries below 2^-90 are not
      // scaled all the way: all pages are near then, but for queries of 0, whose scores are what they are.
      const double size = 448.0 * q_all * scale_double(top_e), margin = 2.0 * size * p.error;
      const double middle = key_score(low), above = middle + margin, under = middle - margin;
      uint32_t last_near = 0xffffffffu, first_near = 0;
      if (above == above && under == under && q_all > 0x1p-90f) {
        const uint64_t a = order64(above), u = order64(under);
        last_near = static_cast<uint32_t>(a >> 32);  // the largest key that is not above
        if (key_order64(last_near) > a) --last_near;
        first_near = static_cast<uint32_t>(u >> 32);  // the smallest that is not below
        if (key_order64(first_near) < u) ++first_near;
      }
      sh.tied = q_all == 0.f;
      sh.near = 0;
      sh.near_low = sh.tied ? low : first_near, sh.near_high = sh.tied ? low : last_near;
    }
    __syncthreads();
    near_low = sh.near_low, near_high = sh.near_high;
    tied = sh.tied;
    for (int j = p.first + tid; j < end; j += kThreads) {
      const uint32_t v = key(j);
      above_near += v > near_high;
      if (v >= near_low && v <= near_high) {
        const int place = atomicAdd(&sh.near, 1);
        if (place < kFewPages) sh.few[place] = j;
      }
    }
    above_near = block_sum<kWarps>(above_near, sh.sums, turn);
    close = above_near + sh.near != k;
  }
  const int need = k - above_near;  // of the pages near, 1 at least

  // ---- pages too near to tell get scores in 64 bits ----
  uint64_t cut64 = 0;
  int ties = 0;  // of the pages at cut64, so many are in
  if (close && tied) {
    ties = need;
  } else if (close) {
    auto score = [&](int j) {  // by a warp
      const int page = listed(j);
      if (page < 0) return order64(-__longlong_as_double(0x7ff0000000000000ll));
      const int64_t ph = static_cast<int64_t>(page) * p.heads + head;
      const uint8_t* codes = p.bounds + ph * 2 * D;
      const int e = p.k_scale[ph];
      double sum = 0.0;
#pragma unroll
      for (int i = lane; i < D / 2; i += 32) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
        const float2 f0 = f16x2_float2(e4m3x2_f16x2(w)), f1 = f16x2_float2(e4m3x2_hi_f16x2(w));
        sum += (sh.q[4 * i] * f0.x + sh.q[4 * i + 1] * f0.y) + (sh.q[4 * i + 2] * f1.x + sh.q[4 * i + 3] * f1.y);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      return order64(sum * scale_double(e));
    };
    const int few = sh.near;
    if (few <= kFewPages && staged) {
      // ---- few: each is compared with the others, and its key becomes the largest or the least ----
      for (int i = warp; i < few; i += kWarps) {
        const uint64_t o = score(sh.few[i]);
        if (lane == 0) sh.few_score[i] = o;
      }
      __syncthreads();
      if (tid < few) {
        const uint64_t o = sh.few_score[tid];
        const int j = sh.few[tid];
        int before = 0;
        for (int i = 0; i < few; ++i) before += sh.few_score[i] > o || (sh.few_score[i] == o && sh.few[i] < j);
        sh.stage[j] = before < need ? 0xffffffffu : 0u;
      }
      close = false;
      near_low = max(near_low, 1u);
      __syncthreads();
    } else {
      uint64_t low64 = ~0ull, high64 = 0;
      for (int j0 = p.first + warp * 32; j0 < end; j0 += kThreads) {
        const int j = j0 + lane;
        const uint32_t v = j < end ? key(j) : 0u;
        uint32_t todo = __ballot_sync(0xffffffffu, j < end && v >= near_low && v <= near_high);
        while (todo != 0) {
          const int at = j0 + __ffs(todo) - 1;
          todo &= todo - 1;
          const uint64_t o = score(at);
          low64 = o < low64 ? o : low64, high64 = o > high64 ? o : high64;
          if (lane == 0) exact[at] = o;
        }
      }
      if (lane == 0) sh.least64[warp] = low64, sh.most64[warp] = high64;
      __syncthreads();  // the stores above are there for the block
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        low64 = sh.least64[w] < low64 ? sh.least64[w] : low64;
        high64 = sh.most64[w] > high64 ? sh.most64[w] : high64;
      }
      auto count64 = [&](uint64_t from) {
        int n = 0;
        for (int j = p.first + tid; j < end; j += kThreads) {
          const uint32_t v = key(j);
          n += v >= near_low && v <= near_high && exact[j] >= from;
        }
        return block_sum<kWarps>(n, sh.sums, turn);
      };
      int n = count64(low64);
      uint64_t lo64 = low64, hi64 = high64;
      while (n != need && lo64 < hi64) {
        const uint64_t mid = lo64 + (hi64 - lo64) / 2 + 1;
        const int m = count64(mid);
        if (m >= need) lo64 = mid, n = m;
        else hi64 = mid - 1;
      }
      cut64 = lo64;
      ties = INT_MAX;
      if (n != need) ties = need - count64(lo64 + 1);  // lo64 is a score of several pages
    }
  }

  // ---- the chosen pages in order: a warp counts, then writes, a run of pages ----
  auto state = [&](int j) {  // 2: in, 1: a tie, 0: out
    if (j < p.first || j >= end) return 2;
    if (k == 0) return 0;  // all places are taken: no keys were staged
    const uint32_t v = key(j);
    if (!close) return v >= near_low ? 2 : 0;
    if (v > near_high) return 2;
    if (v < near_low) return 0;
    if (tied) return 1;
    const uint64_t o = exact[j];
    return o > cut64 ? 2 : o == cut64 ? (ties == INT_MAX ? 2 : 1) : 0;
  };
  const int per = ((pages + kThreads - 1) / kThreads) * 32;  // pages of a warp
  const int j_begin = warp * per, j_end = j_begin + per < pages ? j_begin + per : pages;
  int sure = 0, ties_here = 0;
  for (int j0 = j_begin; j0 < j_end; j0 += 32) {
    const int v = j0 + lane < j_end ? state(j0 + lane) : 0;
    sure += __popc(__ballot_sync(0xffffffffu, v == 2));
    ties_here += __popc(__ballot_sync(0xffffffffu, v == 1));
  }
  if (lane == 0) sh.count[warp] = sure, sh.ties[warp] = ties_here;
  __syncthreads();
  int at = 0, ties_before = 0;
  for (int w = 0; w < warp; ++w) {
    const int left = ties - ties_before;
    at += sh.count[w] + (sh.ties[w] < left ? sh.ties[w] : left > 0 ? left : 0);
    ties_before += sh.ties[w];
  }
  for (int j0 = j_begin; j0 < j_end; j0 += 32) {
    const int v = j0 + lane < j_end ? state(j0 + lane) : 0;
    const uint32_t tie_mask = __ballot_sync(0xffffffffu, v == 1);
    const uint32_t below = (1u << lane) - 1;
    const bool in = v == 2 || (v == 1 && ties_before + __popc(tie_mask & below) < ties);
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
  w.bytes = w.top_e + up256(static_cast<size_t>(batch) * heads * ((max_pages + kTilePages - 1) / kTilePages) * sizeof(int));
  return w;
}

// Roundings of a score: 2^-24 for each addition to q+ and q-; 2^-22 and less than 2^-28 for their two parts; 2^-23 for
// each of 16 additions of a product (single precision, rounded in any way), 2^-24 for each of the d / 32 + 3 after it;
// 2^-20 for what the key drops; 1 / 256 more of it all for the products of these factors and the bound's own rounding.
// Scores of normal, of positive and of widely spread queries and codes were off by 12 % of it at most, nearly all the key's.
double score_error(int ratio, int d) {
  return (ratio * 0x1p-24 + 0x1p-22 + 0x1p-28 + 16 * 0x1p-23 + (d / 32 + 3) * 0x1p-24 + 0x1p-20) * (1.0 + 0x1p-8);
}

template <int D, class S>
int choose_launch(const SelectParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(p.total * p.heads), 1, 1);
  cfg.blockDim = dim3(S::kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_choose_kernel<D, S>, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
int select_launch(const SelectParams& p, int sms, cudaStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(p.batch) * p.heads * p.tiles;
  if (blocks > INT_MAX) return FA_ERR_INVALID_ARG;
  static bool ready[64] = {};
  const int rc = allow_smem(reinterpret_cast<const void*>(kv_score_kernel<D>), sizeof(ScoreShared<D>), ready);
  if (rc != FA_OK) return rc;
  // tokens over blocks as well, where pages alone make few
  const int64_t chunks = (static_cast<int64_t>(p.max_n) + kChunk - 1) / kChunk, room = 8 * static_cast<int64_t>(sms) / blocks;
  const int64_t splits = chunks < room ? chunks : room < 1 ? 1 : room;
  kv_score_kernel<D><<<dim3(static_cast<unsigned int>(blocks), static_cast<unsigned int>(splits)), kSelectThreads,
                       sizeof(ScoreShared<D>), stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  // Small blocks where more choices are to be made than large ones fit the GPU at once (5 an SM).  us of the call, small
  // and large: 2048 tokens of 8 key heads over 160 pages 141 and 216, 512 tokens 61 and 81; 24 x 3 tokens over 1024 pages
  // 25.3 and 24.3, one token 13.3 and 11.3.
  const bool many = p.total * p.heads > 5 * static_cast<int64_t>(sms);
  return many && p.max_pages <= ChooseSmall::kPages ? choose_launch<D, ChooseSmall>(p, stream)
                                                    : choose_launch<D, ChooseLarge>(p, stream);
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
  if (c.d_qk == 64) return bounds_launch<64>(p, stream);
  if (c.d_qk == 128) return bounds_launch<128>(p, stream);
  return bounds_launch<192>(p, stream);
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
  p.top_e = reinterpret_cast<int*>(ws + w.top_e);
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
  p.tiles = (max_pages + kTilePages - 1) / kTilePages;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  p.error = score_error(p.ratio, d_qk);
  if (d_qk == 64) return select_launch<64>(p, host.sms, stream);
  if (d_qk == 128) return select_launch<128>(p, host.sms, stream);
  return select_launch<192>(p, host.sms, stream);
}

}  // extern "C"
