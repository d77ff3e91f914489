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
// One block per (page that gets tokens, head, K or V): the values stay in
// registers between the maximum and the rounding, so each input is read once.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged.cuh"

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
  int64_t total, kv_blocks, q_blocks;
  int batch, heads_q, heads_kv, num_pages, max_pages, page_shift, max_pos, rot, interleaved;
};

constexpr int kItems = 4;         // items of 16 values a thread holds
constexpr int kQItemsPerWarp = 64;  // items of a token's queries one warp rotates

// The sequence's range of new positions [start, start + n) if it can be
// appended: offsets ordered and inside the batch, positions inside the block
// table and the rotation table.
__device__ __forceinline__ bool append_range(const AppendParams& p, int b, int& c0, int& start, int& n) {
  c0 = p.cu[b];
  const int c1 = p.cu[b + 1], len = p.seqlens[b];
  n = c1 - c0;
  start = len - n;
  return c0 >= 0 && c1 >= c0 && c1 <= p.total && start >= 0 &&
         len <= (static_cast<int64_t>(p.max_pages) << p.page_shift) && (p.rot == 0 || len <= p.max_pos);
}

// Item i of a row holds 16 values: two groups of 8 at columns c0 and c1.  The
// first rot / 16 items hold what is rotated; in the half-split order a group
// and its partner group rot / 2 further, in pairs order 16 in a row.
__device__ __forceinline__ void item_columns(int i, int rot, int interleaved, int& c0, int& c1) {
  if (i * 16 < rot && !interleaved) {
    c0 = 8 * i;
    c1 = 8 * i + (rot >> 1);
  } else {
    c0 = 16 * i;
    c1 = c0 + 8;
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

// Rotate the item's 16 values; cs points at the position's cos of pair 0.
// Products and sums are rounded one by one, so that the result does not
// depend on which of them a compiler fuses.
__device__ __forceinline__ void rotate16(float* x, const float* cs, int i, int rot, int interleaved) {
  float c[8], s[8];
  const float4* pc = reinterpret_cast<const float4*>(cs + 8 * i);
  const float4* ps = reinterpret_cast<const float4*>(cs + (rot >> 1) + 8 * i);
  *reinterpret_cast<float4*>(c) = __ldg(pc);
  *reinterpret_cast<float4*>(c + 4) = __ldg(pc + 1);
  *reinterpret_cast<float4*>(s) = __ldg(ps);
  *reinterpret_cast<float4*>(s + 4) = __ldg(ps + 1);
  auto turn = [](float& a, float& b, float cj, float sj) {
    const float ra = __fsub_rn(__fmul_rn(a, cj), __fmul_rn(b, sj));
    b = __fadd_rn(__fmul_rn(b, cj), __fmul_rn(a, sj));
    a = ra;
  };
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn(x[2 * j], x[2 * j + 1], c[j], s[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn(x[j], x[j + 8], c[j], s[j]);
  }
}

template <int D>
__device__ __forceinline__ void append_page(const AppendParams& p, int kv, int head, int b, int c0, int start, int n,
                                            int page_index, int rot) {
  constexpr int kRowItems = D / 16;
  __shared__ float warp_max[32];
  const int tid = threadIdx.x, threads = blockDim.x, page_size = 1 << p.page_shift;
  const int page = p.table[b * p.table_stride + page_index];
  if (page < 0 || page >= p.num_pages) {
    if (tid == 0) paged_error(p.status, kSitePagedPage, b);
    return;
  }
  const int page0 = page_index << p.page_shift;
  const int lo = start > page0 ? start : page0;
  const int hi = start + n < page0 + page_size ? start + n : page0 + page_size;
  const int old_rows = lo - page0, rows = hi - lo;
  uint8_t* dst = p.dst[kv] + page * p.page_stride[kv] + head * p.head_stride[kv];
  const int64_t ts = p.token_stride[kv];
  const __nv_bfloat16* src = p.src[kv] + static_cast<int64_t>(c0 + lo - start) * p.src_stride[kv] + head * D;
  uint8_t* scale = p.scale[kv] + static_cast<int64_t>(page) * p.heads_kv + head;
  const int e_old = old_rows > 0 ? *scale : 0;

  float x[kItems][16];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int it = tid + k * threads;
    const int row = it / kRowItems, i = it % kRowItems;
    if (row < rows) {
      int ca, cb;
      item_columns(i, rot, p.interleaved, ca, cb);
      const __nv_bfloat16* r = src + row * p.src_stride[kv];
      unpack8(__ldg(reinterpret_cast<const uint4*>(r + ca)), x[k]);
      unpack8(__ldg(reinterpret_cast<const uint4*>(r + cb)), x[k] + 8);
      if (i * 16 < rot)
        rotate16(x[k], p.cos_sin + static_cast<int64_t>(lo + row) * rot, i, rot, p.interleaved);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float a = fabsf(x[k][j]);
        amax = a < INFINITY ? fmaxf(amax, a) : amax;  // what is no number does not count
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < (threads >> 5); ++w) amax = fmaxf(amax, warp_max[w]);

  // 448 = 1.75 * 2^8: the exponent by which amax / 2^e stays at or below it
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  e = e < kMinScale ? kMinScale : e;
  e = e < e_old ? e_old : e;
  if (tid == 0) *scale = static_cast<uint8_t>(e);
  const float inv = e < 254 ? __uint_as_float(static_cast<uint32_t>(254 - e) << 23) : 0.f;

#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int it = tid + k * threads;
    const int row = it / kRowItems, i = it % kRowItems;
    if (row < rows) {
      int ca, cb;
      item_columns(i, rot, p.interleaved, ca, cb);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y[4];
#pragma unroll
        for (int l = 0; l < 4; ++l)  // an infinity would saturate: inf * 0 makes it NaN
          y[l] = __fmaf_rn(x[k][4 * j + l], 0.f, __fmul_rn(x[k][4 * j + l], inv));
        w[j] = e4m3x4(y[0], y[1], y[2], y[3]);
      }
      uint8_t* r = dst + (old_rows + row) * ts;
      if (cb == ca + 8) {
        *reinterpret_cast<uint4*>(r + ca) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<uint2*>(r + ca) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(r + cb) = make_uint2(w[2], w[3]);
      }
    }
  }

  if (old_rows > 0 && e > e_old) {  // the scale grew: older codes move to it
    const int shift = e - e_old;
    const float f = shift < 127 ? __uint_as_float(static_cast<uint32_t>(127 - shift) << 23) : 0.f;
    for (int it = tid; it < old_rows * kRowItems; it += threads) {
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
}

template <int DQK, int DV>
__global__ void __launch_bounds__(384) kv_append_kernel(const AppendParams p) {
  const int64_t blk = blockIdx.x;
  const int lane = threadIdx.x & 31;
  if (blk < p.kv_blocks) {
    // blocks of one page run over heads, K and V next to each other
    const int per_page = 2 * p.heads_kv;
    const int64_t slot = blk / per_page;
    const int rest = static_cast<int>(blk - slot * per_page);
    const int kv = rest & 1, head = rest >> 1;
    // sequence b owns the page slots from floor(cu[b] / page) + 2 b on: no
    // fewer than the pages its new tokens can touch
    const int b = warp_search(p.batch, slot, [&](int i) { return static_cast<int64_t>(p.cu[i] >> p.page_shift) + 2 * i; });
    int c0, start, n;
    if (!append_range(p, b, c0, start, n) || n == 0) return;
    const int64_t j = slot - ((c0 >> p.page_shift) + 2 * b);
    const int first = start >> p.page_shift, last = (start + n - 1) >> p.page_shift;
    if (j < 0 || first + j > last) return;
    const int page_index = first + static_cast<int>(j);
    if (kv == 0)
      append_page<DQK>(p, 0, head, b, c0, start, n, page_index, p.rot);
    else
      append_page<DV>(p, 1, head, b, c0, start, n, page_index, 0);
    return;
  }
  if (blk < p.kv_blocks + p.q_blocks) {
    constexpr int kRowItems = DQK / 16;
    const int items = p.heads_q * kRowItems;
    const int parts = (items + kQItemsPerWarp - 1) / kQItemsPerWarp;
    const int64_t unit = (blk - p.kv_blocks) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t t = unit / parts;
    if (t >= p.total) return;
    const int part = static_cast<int>(unit - t * parts);
    const int b = warp_search(p.batch, t, [&](int i) { return static_cast<int64_t>(p.cu[i]); });
    int c0, start, n;
    if (!append_range(p, b, c0, start, n) || t < c0 || t >= c0 + n) return;
    const float* cs = p.cos_sin + (start + (t - c0)) * p.rot;
    const __nv_bfloat16* src = p.q + t * p.q_stride;
    __nv_bfloat16* dst = p.q_out + t * (static_cast<int64_t>(p.heads_q) * DQK);
    float x[kQItemsPerWarp / 32][16];
#pragma unroll
    for (int k = 0; k < kQItemsPerWarp / 32; ++k) {
      const int it = part * kQItemsPerWarp + k * 32 + lane;
      if (it < items) {
        const int h = it / kRowItems, i = it % kRowItems;
        int ca, cb;
        item_columns(i, p.rot, p.interleaved, ca, cb);
        unpack8(*reinterpret_cast<const uint4*>(src + h * DQK + ca), x[k]);
        unpack8(*reinterpret_cast<const uint4*>(src + h * DQK + cb), x[k] + 8);
        if (i * 16 < p.rot) rotate16(x[k], cs, i, p.rot, p.interleaved);
      }
    }
    __syncwarp();  // q_out may be q: a row's values are all read before any is written
#pragma unroll
    for (int k = 0; k < kQItemsPerWarp / 32; ++k) {
      const int it = part * kQItemsPerWarp + k * 32 + lane;
      if (it < items) {
        const int h = it / kRowItems, i = it % kRowItems;
        int ca, cb;
        item_columns(i, p.rot, p.interleaved, ca, cb);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(x[k][2 * j], x[k][2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(dst + h * DQK + ca) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(dst + h * DQK + cb) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    return;
  }
  // the last block looks every sequence over
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    int c0, start, n;
    if (!append_range(p, b, c0, start, n)) paged_error(p.status, kSitePagedSeq, b);
  }
}

template <int DQK, int DV>
cudaError_t launch_append(const AppendParams& p, int64_t blocks, int threads, cudaStream_t stream) {
  kv_append_kernel<DQK, DV><<<static_cast<unsigned int>(blocks), threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int append_launch(const fa_kv_cache& c, const void* q, const void* k, const void* v, int64_t q_stride,
                  int64_t k_stride, int64_t v_stride, void* q_out, const int* cu, int batch, int64_t total,
                  int heads_q, const float* cos_sin, int max_pos, int rot, int interleaved, unsigned int* status,
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
  // a thread holds kItems items of 16 values
  int threads = c.page_size * c.d_qk / (16 * kItems);
  threads = (threads + 31) / 32 * 32;
  p.kv_blocks = ((total >> p.page_shift) + 2 * static_cast<int64_t>(batch)) * 2 * c.heads_kv;
  p.q_blocks = 0;
  if (q != nullptr) {
    const int64_t parts = (static_cast<int64_t>(heads_q) * (c.d_qk / 16) + kQItemsPerWarp - 1) / kQItemsPerWarp;
    p.q_blocks = (total * parts + threads / 32 - 1) / (threads / 32);
  }
  const int64_t blocks = p.kv_blocks + p.q_blocks + 1;
  if (blocks > INT_MAX) return FA_ERR_INVALID_ARG;
  cudaError_t rc = cudaErrorInvalidValue;
  if (c.d_qk == 64 && c.d_v == 64) rc = launch_append<64, 64>(p, blocks, threads, stream);
  if (c.d_qk == 128 && c.d_v == 64) rc = launch_append<128, 64>(p, blocks, threads, stream);
  if (c.d_qk == 128 && c.d_v == 128) rc = launch_append<128, 128>(p, blocks, threads, stream);
  if (c.d_qk == 192 && c.d_v == 64) rc = launch_append<192, 64>(p, blocks, threads, stream);
  if (c.d_qk == 192 && c.d_v == 128) rc = launch_append<192, 128>(p, blocks, threads, stream);
  return rc == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
