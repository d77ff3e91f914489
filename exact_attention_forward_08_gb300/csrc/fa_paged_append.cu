// fa_kv_append: new keys and values into a paged 8-bit cache, rotated by their
// positions on the way, and the new queries rotated in the same launch.
//
// For a page and head with older codes c_j under scale s and new values x_i:
//     s' = max(s, min { 2^e : max_i |x_i| <= 448 * 2^e }),   e >= -63
//     c_i = rn_e4m3(x_i / s'),   c_j' = rn_e4m3(c_j * (s / s'))
// e4m3 is a floating format, so with a power of two for the scale a code keeps
// its relative precision whatever the scale, dividing by it is exact, and
// moving older codes to a larger scale changes only those that fall below the
// smallest normal code.  Rotation, maximum and division are in fp32 from the
// bf16 inputs; the one rounding is that to the code.
//
// A team of 1 to 8 warps takes a unit, one head's K or V in one page.  It reads
// the new tokens in blocks of 8 rows: once for the maximum, and again, out of
// the caches, to round and store them (a warp with one block keeps it).  More
// warps a unit where there are few units.  Nothing waits on anything but the
// team's one maximum, so loads of many units are under way at a time.
//
// Bound by the latency of loads: 80 registers let 24 warps on an SM.  8191 tokens
// of 32/8 heads of 128: 39 us, 4.8 TB/s of what has to move (28 us at the copy
// rate); 24 prompts of 1 to 900 tokens, 16/16 heads of 192/128: 56 us (38.5);
// one token of one or of 128 sequences: 3.5 and 5.3 us.  Queries take three heads a
// lane at once and ask for the first before their token's sequence is known: 42.0
// and 57.9 us with two, afterwards.  Registers for 16 warps: 45.6 and 64.5, for 32:
// 40.5 and 58.4.  With those for 24 a thread spills 8 bytes at d_qk = 128 and 40 at
// 192 (136 read back), nothing at 64.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged.cuh"
#include "fa_paged_range.h"
#include "ptx.cuh"

namespace fa {
namespace {

struct AppendParams {
  const __nv_bfloat16* src[2];  // K, V: [total, heads_kv, d], token stride src_stride elements
  int64_t src_stride[2];
  uint8_t* dst[2];
  int64_t page_stride[2], head_stride[2], token_stride[2];  // bytes
  uint8_t* scale[2];
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  int64_t q_stride;
  const float* cos_sin;
  const int* cu;
  const int* seqlens;
  const int* table;
  int64_t table_stride;
  unsigned int* status;
  int64_t total, slots, kv_blocks, q_blocks;
  int batch, heads_q, heads_kv, num_pages, max_pages, page_shift, max_pos, rot, interleaved;
  int q_heads;  // heads of a token that one warp turns
  int team;     // warps of a unit
};

constexpr int kBlockRows = 8;  // rows a warp holds at a time
constexpr int kWarps = 8;      // of a block
// Warps an SM that units are spread over: a unit gets two, four or eight where
// there are fewer units than that.  us with 32 / 64 / 128:
//   8191 tokens, 32/8 heads of 128, pages of 64        39.5 / 38.9 / 38.9
//   24 prompts of 1..900, 16/16 of 192/128, pages of 32  55.8 / 55.8 / 61.5
//   16 prompts of 450..900, 16/16 of 192/128, of 64      68.6 / 65.6 / 69.2
//   64 prompts of 50..100, 32/8 of 128, of 64            22.6 / 25.9 / 31.9
//   4 prompts of 256..512, 16/4 of 64, and one of 2000, 32/8 of 128: within 0.4 %
constexpr int kTeamWarps = 64;

// The sequence's range of new positions [start, start + n) if it can be
// appended: offsets ordered and inside the batch, positions inside the block
// table and the rotation table.
__device__ __forceinline__ bool append_range(const AppendParams& p, int b, int& c0, int& start, int& n) {
  c0 = p.cu[b];
  int64_t most = static_cast<int64_t>(p.max_pages) << p.page_shift;
  if (p.rot > 0 && p.max_pos < most) most = p.max_pos;
  return paged_append_range(c0, p.cu[b + 1], p.seqlens[b], p.total, most, start, n);
}

// Item i of a row holds 16 values: two groups of 8, at columns c0 and c1.  The
// first rot / 16 items hold what is rotated, a group of the first half of those
// columns and its partner of the second; the others pair the rest the same
// way, so that neighbouring lanes always touch neighbouring groups.
template <int D>
__device__ __forceinline__ void item_columns(int i, int rot, int& c0, int& c1) {
  if (i * 16 < rot) {
    c0 = 8 * i;
    c1 = c0 + (rot >> 1);
  } else {
    c0 = 8 * i + (rot >> 1);
    c1 = c0 + ((D - rot) >> 1);
  }
}

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The cosines (first 8) and sines of item i's pairs; `cs` points at the position's row.
__device__ __forceinline__ void load_cos_sin(float* c, const float* cs, int i, int rot, int interleaved) {
  const float* first = cs + (interleaved ? 4 * i : 8 * i);
  const float* second = first + (interleaved ? rot >> 2 : 4);
  *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(first));
  *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(second));
  *reinterpret_cast<float4*>(c + 8) = __ldg(reinterpret_cast<const float4*>(first + (rot >> 1)));
  *reinterpret_cast<float4*>(c + 12) = __ldg(reinterpret_cast<const float4*>(second + (rot >> 1)));
}

// Rotate the item's 16 values.  Products and sums are rounded one by one, so
// that the result does not depend on which of them a compiler fuses.
template <bool kPairs>
__device__ __forceinline__ void turn16_as(float* x, const float* cs) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float &a = x[kPairs ? 2 * j : j], &b = x[kPairs ? 2 * j + 1 : j + 8];
    const float c = cs[j], s = cs[j + 8];
    const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = ra;
  }
}
__device__ __forceinline__ void turn16(float* x, const float* cs, int interleaved) {
  if (interleaved) turn16_as<true>(x, cs);
  else turn16_as<false>(x, cs);
}

// The largest |x|; NaN does not count, an infinity does
__device__ __forceinline__ float item_max(const float* x, float m) {
#pragma unroll
  for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(x[j]));
  return m;
}
// the same of 16 packed bf16
__device__ __forceinline__ float packed_max(const uint4& u, const uint4& v, float m) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  __nv_bfloat162 t = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) t = __hmax2(t, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));
  return fmaxf(m, fmaxf(__low2float(t), __high2float(t)));
}
__device__ __forceinline__ float item_finite_max(const float* x, float m) {
#pragma unroll
  for (int j = 0; j < 16; ++j) m = fabsf(x[j]) < INFINITY ? fmaxf(m, fabsf(x[j])) : m;
  return m;
}
// An infinity would be stored as the largest code: NaN in its place
__device__ __forceinline__ void item_no_infinity(float* x) {
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = fabsf(x[j]) < INFINITY ? x[j] : __uint_as_float(0x7fc00000u);
}

// of values that are not negative: their bits are ordered as they are
__device__ __forceinline__ float warp_maximum(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// 16 values as codes, two groups of 8
__device__ __forceinline__ void store_item(uint8_t* c0, uint8_t* c1, const float* x, float inv) {
  uint32_t w[4];
  const uint64_t f = f2_pack(inv, inv);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float y[4];
    f2_unpack(f2_mul(f2_pack(x[4 * j], x[4 * j + 1]), f), y[0], y[1]);
    f2_unpack(f2_mul(f2_pack(x[4 * j + 2], x[4 * j + 3]), f), y[2], y[3]);
    w[j] = e4m3x4(y[0], y[1], y[2], y[3]);
  }
  *reinterpret_cast<uint2*>(c0) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(c1) = make_uint2(w[2], w[3]);
}

// The exponent of the smallest scale that holds amax: 448 = 1.75 * 2^8
__device__ __forceinline__ int needed_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return e < kMinScale ? kMinScale : e;
}
__device__ __forceinline__ float inverse_scale(int e) {
  return e < 254 ? __uint_as_float(static_cast<uint32_t>(254 - e) << 23) : 0.f;
}

// Older codes of a page move to a scale that is 2^shift as large.
template <int D>
__device__ __forceinline__ void shrink_codes(uint8_t* dst, int64_t ts, int rows, int shift, int tid, int threads) {
  constexpr int kRowItems = D / 16;
  const float f = shift < 127 ? __uint_as_float(static_cast<uint32_t>(127 - shift) << 23) : 0.f;
  for (int it = tid; it < rows * kRowItems; it += threads) {
    uint4* at = reinterpret_cast<uint4*>(dst + (it / kRowItems) * ts + (it % kRowItems) * 16);
    uint4 v = *at;
    uint32_t* w = &v.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u0 = f16x2_float2(e4m3x2_f16x2(w[j])), u1 = f16x2_float2(e4m3x2_hi_f16x2(w[j]));
      w[j] = e4m3x4(u0.x * f, u0.y * f, u1.x * f, u1.y * f);
    }
    *at = v;
  }
}

// The page that a block or warp appends to, and its new tokens there.
struct AppendPage {
  int page, old_rows, rows, pos, token;  // index, tokens there before, new ones, the first one's position and row
};
__device__ __forceinline__ bool append_page_of(const AppendParams& p, int b, int c0, int start, int n, int page_index,
                                               bool report, AppendPage& a) {
  a.page = p.table[b * p.table_stride + page_index];
  if (a.page < 0 || a.page >= p.num_pages) {
    if (report) paged_error(p.status, kSitePagedPage, b);
    return false;
  }
  const int page0 = page_index << p.page_shift, page_end = page0 + (1 << p.page_shift);
  a.pos = start > page0 ? start : page0;
  a.old_rows = a.pos - page0;
  a.rows = (start + n < page_end ? start + n : page_end) - a.pos;
  a.token = c0 + a.pos - start;
  return true;
}

// The sequence and page of a page slot; -1 if the slot is not used.  Sequence
// b owns the slots from floor(cu[b] / page) + 2 b on: no fewer than the pages
// its new tokens can touch.
__device__ __forceinline__ int append_slot(const AppendParams& p, int64_t slot, int& c0, int& start, int& n,
                                           int& page_index) {
  const int b = warp_search(p.batch, slot, [&](int i) { return static_cast<int64_t>(p.cu[i] >> p.page_shift) + 2 * i; });
  if (!append_range(p, b, c0, start, n) || n == 0) return -1;
  const int64_t j = slot - ((c0 >> p.page_shift) + 2 * b);
  const int first = start >> p.page_shift, last = (start + n - 1) >> p.page_shift;
  if (j < 0 || first + j > last) return -1;
  page_index = first + static_cast<int>(j);
  return b;
}

// One head's K or V of one page by the team's warps `sub` of `team`.  The items
// of a block are dealt out lane after lane, those that are rotated first, so
// that whole warps rotate or do not; a lane's rows and columns are the same in
// every block.
template <int D, bool ROTATE>
__device__ __forceinline__ void append_unit(const AppendParams& p, int kv, int head, const AppendPage& a, int sub,
                                            int team, int barrier, float* team_max) {
  constexpr int kItems = kBlockRows * D / 16 / 32;
  const int lane = threadIdx.x & 31;
  const int rot = ROTATE ? p.rot : 0;
  const int64_t ss = p.src_stride[kv], ts = p.token_stride[kv];
  const __nv_bfloat16* src = p.src[kv] + a.token * ss + head * D;
  uint8_t* dst = p.dst[kv] + a.page * p.page_stride[kv] + head * p.head_stride[kv];
  uint8_t* scale = p.scale[kv] + static_cast<int64_t>(a.page) * p.heads_kv + head;
  const int e_old = a.old_rows > 0 ? *scale : 0;

  int row_of[kItems], item[kItems], ca[kItems], cb[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int at = k * 32 + lane;
    if constexpr (ROTATE) {
      const int turned = rot >> 4, rest = D / 16 - turned;  // items of a row
      const int other = at - kBlockRows * turned;
      row_of[k] = other < 0 ? at / turned : other / rest;
      item[k] = other < 0 ? at - row_of[k] * turned : turned + other - row_of[k] * rest;
    } else {
      row_of[k] = at / (D / 16);
      item[k] = at % (D / 16);
    }
    item_columns<D>(item[k], rot, ca[k], cb[k]);
  }
  auto load = [&](int block, uint4 (*raw)[2]) {
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int row = block * kBlockRows + row_of[k];
      if (row < a.rows) {
        const __nv_bfloat16* r = src + row * ss;
        raw[k][0] = __ldg(reinterpret_cast<const uint4*>(r + ca[k]));
        raw[k][1] = __ldg(reinterpret_cast<const uint4*>(r + cb[k]));
      }
    }
  };
  // an item's values as they are stored
  auto values = [&](const uint4* raw, int row, int i, float* x) {
    unpack8(raw[0], x);
    unpack8(raw[1], x + 8);
    if (ROTATE && i * 16 < rot) {
      float cs[16];
      load_cos_sin(cs, p.cos_sin + static_cast<int64_t>(a.pos + row) * rot, i, rot, p.interleaved);
      turn16(x, cs, p.interleaved);
    }
  };
  auto team_maximum = [&](float m) {
    m = warp_maximum(m);
    if (team > 1) {
      if (lane == 0) team_max[sub] = m;
      asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * team) : "memory");
      m = warp_maximum(lane < team ? team_max[lane] : 0.f);
      asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * team) : "memory");  // read before it is written again
    }
    return m;
  };

  const int blocks = (a.rows + kBlockRows - 1) / kBlockRows;
  uint4 raw[kItems][2];
  float amax = 0.f;
  for (int block = sub; block < blocks; block += team) {
    load(block, raw);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int row = block * kBlockRows + row_of[k];
      if (row < a.rows) {
        if (ROTATE && item[k] * 16 < rot) {
          float x[16];
          values(raw[k], row, item[k], x);
          amax = item_max(x, amax);
        } else {
          amax = packed_max(raw[k][0], raw[k][1], amax);
        }
      }
    }
  }
  amax = team_maximum(amax);
  const bool infinite = amax == INFINITY;
  if (infinite) {  // infinities do not count either
    amax = 0.f;
    for (int block = sub; block < blocks; block += team) {
      load(block, raw);
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int row = block * kBlockRows + row_of[k];
        if (row < a.rows) {
          float x[16];
          values(raw[k], row, item[k], x);
          amax = item_finite_max(x, amax);
        }
      }
    }
    amax = team_maximum(amax);
  }
  int e = needed_exponent(amax);
  e = e < e_old ? e_old : e;
  if (sub == 0 && lane == 0) *scale = static_cast<uint8_t>(e);
  const float inv = inverse_scale(e);
  for (int block = sub; block < blocks; block += team) {
    if (blocks > team) load(block, raw);  // else the one block is still here
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int row = block * kBlockRows + row_of[k];
      if (row < a.rows) {
        float x[16];
        values(raw[k], row, item[k], x);
        if (infinite) item_no_infinity(x);
        uint8_t* r = dst + (a.old_rows + row) * ts;
        store_item(r + ca[k], r + cb[k], x, inv);
      }
    }
  }
  if (a.old_rows > 0 && e > e_old) shrink_codes<D>(dst, ts, a.old_rows, e - e_old, sub * 32 + lane, team * 32);
}

// The queries of one token, or q_heads of them: a lane keeps its columns'
// cosines and sines for all heads that it turns.
template <int D>
__device__ __forceinline__ void append_query(const AppendParams& p, int64_t unit, int parts) {
  constexpr int kRowItems = D / 16, kRows = 32 / kRowItems, kBatch = 3;  // heads a warp, and heads a lane, at once
  const int lane = threadIdx.x & 31;
  const int64_t t = unit / parts;
  if (t >= p.total) return;
  const int part = static_cast<int>(unit - t * parts);
  const bool has_item = lane < kRows * kRowItems;  // 12 columns: 24 lanes
  const int i = lane % kRowItems;
  int ca, cb;
  item_columns<D>(i, p.rot, ca, cb);
  const __nv_bfloat16* src = p.q + t * p.q_stride;
  __nv_bfloat16* dst = p.q_out + t * (static_cast<int64_t>(p.heads_q) * D);
  const int end = p.heads_q < (part + 1) * p.q_heads ? p.heads_q : (part + 1) * p.q_heads;
  uint4 raw[kBatch][2];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * kRows;
      if (h < end && has_item) {
        raw[k][0] = *reinterpret_cast<const uint4*>(src + h * D + ca);
        raw[k][1] = *reinterpret_cast<const uint4*>(src + h * D + cb);
      }
    }
  };
  const int h_first = part * p.q_heads + lane / kRowItems;
  load(h_first);  // on the way while the token's sequence is looked up
  const int b = warp_search(p.batch, t, [&](int i) { return static_cast<int64_t>(p.cu[i]); });
  int c0, start, n;
  if (!append_range(p, b, c0, start, n) || t < c0 || t >= c0 + n || !has_item) return;
  float cs[16];
  const bool turned = i * 16 < p.rot;
  if (turned) load_cos_sin(cs, p.cos_sin + (start + (t - c0)) * p.rot, i, p.rot, p.interleaved);
  for (int h0 = h_first; h0 < end; h0 += kBatch * kRows) {
    if (h0 != h_first) load(h0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * kRows;
      if (h < end) {
        float x[16];
        unpack8(raw[k][0], x);
        unpack8(raw[k][1], x + 8);
        if (turned) turn16(x, cs, p.interleaved);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(dst + h * D + ca) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(dst + h * D + cb) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
}

template <int DQK, int DV>
__global__ void __launch_bounds__(32 * kWarps, 3) kv_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float team_max[kWarps];
  const int64_t blk = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  if (blk < p.kv_blocks) {
    // the units of a page slot are its heads, K and V by turns
    const int team = p.team, sub = warp % team, first = warp - sub;
    const int64_t unit = blk * (kWarps / team) + warp / team, slot = unit / (2 * p.heads_kv);
    if (slot >= p.slots) return;
    const int rest = static_cast<int>(unit - slot * (2 * p.heads_kv)), head = rest >> 1;
    int c0, start, n, page_index;
    const int b = append_slot(p, slot, c0, start, n, page_index);
    AppendPage a;
    if (b < 0 || !append_page_of(p, b, c0, start, n, page_index, (threadIdx.x & 31) == 0, a)) return;
    if ((rest & 1) != 0) append_unit<DV, false>(p, 1, head, a, sub, team, 1 + first, team_max + first);
    else if (p.rot > 0) append_unit<DQK, true>(p, 0, head, a, sub, team, 1 + first, team_max + first);
    else append_unit<DQK, false>(p, 0, head, a, sub, team, 1 + first, team_max + first);
    return;
  }
  if (blk < p.kv_blocks + p.q_blocks) {
    append_query<DQK>(p, (blk - p.kv_blocks) * kWarps + warp, (p.heads_q + p.q_heads - 1) / p.q_heads);
    return;
  }
  // the last block looks every sequence over
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    int c0, start, n;
    if (!append_range(p, b, c0, start, n)) paged_error(p.status, kSitePagedSeq, b);
  }
}

template <int DQK, int DV>
cudaError_t launch_append(const AppendParams& p, int64_t blocks, cudaStream_t stream) {
  kv_append_kernel<DQK, DV><<<static_cast<unsigned int>(blocks), 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int append_launch(const fa_kv_cache& c, const void* q, const void* k, const void* v, int64_t q_stride,
                  int64_t k_stride, int64_t v_stride, void* q_out, const int* cu, int batch, int64_t total,
                  int heads_q, const float* cos_sin, int max_pos, int rot, int interleaved, unsigned int* status, int sms,
                  cudaStream_t stream) {
  AppendParams p;
  p.src[0] = static_cast<const __nv_bfloat16*>(k);
  p.src[1] = static_cast<const __nv_bfloat16*>(v);
  p.src_stride[0] = k_stride;
  p.src_stride[1] = v_stride;
  p.dst[0] = static_cast<uint8_t*>(c.k);
  p.dst[1] = static_cast<uint8_t*>(c.v);
  for (int i = 0; i < 2; ++i) {
    const int64_t* s = i == 0 ? c.k_stride : c.v_stride;
    p.page_stride[i] = s[0];
    p.head_stride[i] = s[1];
    p.token_stride[i] = s[2];
  }
  p.scale[0] = c.k_scale;
  p.scale[1] = c.v_scale;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_stride = q_stride;
  p.cos_sin = cos_sin;
  p.cu = cu;
  p.seqlens = c.seqlens_k;
  p.table = c.block_table;
  p.table_stride = c.table_stride;
  p.status = status;
  p.total = total;
  p.batch = batch;
  p.heads_q = heads_q;
  p.heads_kv = c.heads_kv;
  p.num_pages = c.num_pages;
  p.max_pages = c.max_pages;
  p.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  p.max_pos = max_pos;
  p.rot = rot;
  p.interleaved = interleaved;
  p.slots = (total >> p.page_shift) + 2 * static_cast<int64_t>(batch);
  // the warps of a unit: more where units are few, as many as a page has blocks of rows
  const int64_t units = p.slots * 2 * c.heads_kv;
  p.team = 1;
  if (total > kBlockRows / 2 * static_cast<int64_t>(batch))
    while (p.team < kWarps && p.team < c.page_size / kBlockRows && units * p.team < kTeamWarps * static_cast<int64_t>(sms))
      p.team *= 2;
  p.kv_blocks = (units * p.team + kWarps - 1) / kWarps;
  p.q_blocks = 0;
  p.q_heads = 1;
  if (q != nullptr) {
    // a warp turns all heads of a token where there are tokens enough to fill the GPU
    p.q_heads = total >= 2048 ? heads_q : (heads_q < 8 ? heads_q : 8);
    p.q_blocks = (total * ((heads_q + p.q_heads - 1) / p.q_heads) + kWarps - 1) / kWarps;
  }
  const int64_t blocks = p.kv_blocks + p.q_blocks + 1;
  if (blocks > INT_MAX) return FA_ERR_INVALID_ARG;
  cudaError_t rc = cudaErrorInvalidValue;
  if (c.d_qk == 64 && c.d_v == 64) rc = launch_append<64, 64>(p, blocks, stream);
  if (c.d_qk == 128 && c.d_v == 64) rc = launch_append<128, 64>(p, blocks, stream);
  if (c.d_qk == 128 && c.d_v == 128) rc = launch_append<128, 128>(p, blocks, stream);
  if (c.d_qk == 192 && c.d_v == 64) rc = launch_append<192, 64>(p, blocks, stream);
  if (c.d_qk == 192 && c.d_v == 128) rc = launch_append<192, 128>(p, blocks, stream);
  return rc == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
