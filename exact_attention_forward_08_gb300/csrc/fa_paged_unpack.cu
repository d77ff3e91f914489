// fa_fwd_paged for long sequences of new tokens (prompts): their pages are
// unpacked to bf16 rows, which the variable-length forward then reads.  A code
// times a power of two is a bf16 number, so nothing is rounded here.  With n
// new tokens the attention reads each key n x ratio times; unpacking moves it
// once, 1 byte in and 2 out: bound by bandwidth, 23 us for 16384 tokens of 8
// heads of 128 and 128 (101 MB, 4.4 TB/s) where the forward of 2 x 2048 new tokens
// takes 381.
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_paged.cuh"
#include "fa_paged.h"
#include "fa_paged_range.h"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;

// One block: the key offsets of the sequences that take this path.  Others get no
// keys, also those whose length or number of new tokens is out of range: the rest is
// computed.  -1 throughout, so that nothing is, where the offsets of the new tokens
// are broken or the keys do not fit.
__global__ void __launch_bounds__(kPlanThreads) unpack_plan_kernel(const UnpackParams p) {
  __shared__ long long warp_sum[32];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) bad = 0;
  __syncthreads();
  long long before = 0;
  for (int base = 0; base < p.batch; base += kPlanThreads) {
    const int b = base + tid;
    long long v = 0;
    if (b < p.batch) {
      const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], len = p.seqlens[b];
      int n;
      if (!paged_attend_range(c0, c1, len, p.total_q, p.max_n,
                              static_cast<int64_t>(p.max_pages) << p.page_shift, n)) {
        paged_error(p.status, kSitePagedSeq, b);
        if (!paged_offsets_ok(c0, c1, p.total_q)) bad = 1;  // the variable-length forward reads the same offsets
      } else if (static_cast<long long>(n) * p.ratio > p.row_limit) {
        v = len;
      }
    }
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long mine = before;
    for (int w = 0; w < warp; ++w) mine += warp_sum[w];
    long long all = before;
    for (int w = 0; w < kPlanThreads / 32; ++w) all += warp_sum[w];
    // beyond total_k the values are replaced below
    if (b < p.batch) p.cu_k[b + 1] = mine + incl > p.total_k ? -1 : static_cast<int>(mine + incl);
    before = all;
    __syncthreads();
  }
  if (tid == 0) {
    p.cu_k[0] = 0;
    if (before > p.total_k) {
      paged_error(p.status, kSitePagedTotal, 0);
      bad = 1;
    }
  }
  __syncthreads();
  if (bad)
    for (int i = tid; i <= p.batch; i += kPlanThreads) p.cu_k[i] = -1;
}

// two codes times the scale as two bf16
__device__ __forceinline__ uint32_t bf16x2_of(uint32_t f16x2, float scale) {
  const float2 x = f16x2_float2(f16x2);
  const __nv_bfloat162 v = __floats2bfloat162_rn(x.x * scale, x.y * scale);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// 16 codes to 16 bf16
__device__ __forceinline__ void store16(uint16_t* dst, const uint4& v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    out[2 * j] = bf16x2_of(e4m3x2_f16x2(w[j]), scale);
    out[2 * j + 1] = bf16x2_of(e4m3x2_hi_f16x2(w[j]), scale);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(out[0], out[1], out[2], out[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// A warp for 16 tokens (inside one page) of a head.  The attention multiplies
// the values of hidden tokens by weights of 0, so no value may be NaN: a token
// with a NaN code among its values gets the value 0 where the code is, and NaN
// keys, which reach only the rows that see it.  128 rows behind the last are 0.
template <int DQK, int DV>
__global__ void __launch_bounds__(256) unpack_kernel(const UnpackParams p) {
  constexpr int kKChunks = DQK / 16, kVChunks = DV / 16;
  const int lane = threadIdx.x & 31;
  const int64_t total = p.cu_k[p.batch];
  if (total < 0) return;
  const int64_t slots = (total >> 4) + p.batch;
  const int64_t units = (slots + 8) * p.heads_kv;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t slot = u / p.heads_kv;
    const int head = static_cast<int>(u - slot * p.heads_kv);
    if (slot >= slots) {
      for (int t = 0; t < 16; ++t) {
        const int64_t row = total + (slot - slots) * 16 + t;
        if (row >= p.total_k) break;
        uint4* k = reinterpret_cast<uint4*>(p.dst[0] + (row * p.heads_kv + head) * DQK);
        uint4* v = reinterpret_cast<uint4*>(p.dst[1] + (row * p.heads_kv + head) * DV);
        if (lane < DQK / 8) k[lane] = make_uint4(0, 0, 0, 0);
        if (lane < DV / 8) v[lane] = make_uint4(0, 0, 0, 0);
      }
      continue;
    }
    // sequence b owns the slots from floor(cu_k[b] / 16) + b on: no fewer than its blocks of 16 tokens
    const int b = warp_search(p.batch, slot, [&](int i) { return static_cast<int64_t>(p.cu_k[i] >> 4) + i; });
    const int k0 = p.cu_k[b], len = p.cu_k[b + 1] - k0;
    const int token0 = static_cast<int>(slot - ((k0 >> 4) + b)) * 16;
    if (token0 >= len) continue;
    const int tokens = len - token0 < 16 ? len - token0 : 16;
    int page = p.table[b * p.table_stride + (token0 >> p.page_shift)];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) paged_error(p.status, kSitePagedPage, b);
      page = 0;
    }
    const int64_t row0 = k0 + static_cast<int64_t>(token0);
    const int in_page = token0 & ((1 << p.page_shift) - 1);
    const int64_t si = static_cast<int64_t>(page) * p.heads_kv + head;
    const int ek = p.scale[0][si], ev = p.scale[1][si];
    const uint8_t* ks = p.src[0] + page * p.page_stride[0] + head * p.head_stride[0] + in_page * p.token_stride[0];
    const uint8_t* vs = p.src[1] + page * p.page_stride[1] + head * p.head_stride[1] + in_page * p.token_stride[1];
    uint4 kc[kKChunks / 2], vc[kVChunks / 2];  // 16 rows x chunks over 32 lanes
#pragma unroll
    for (int i = 0; i < kVChunks / 2; ++i) {
      const int at = i * 32 + lane, t = at / kVChunks, ch = at % kVChunks;
      vc[i] = t < tokens ? *reinterpret_cast<const uint4*>(vs + t * p.token_stride[1] + ch * 16) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kKChunks / 2; ++i) {
      const int at = i * 32 + lane, t = at / kKChunks, ch = at % kKChunks;
      kc[i] = t < tokens ? *reinterpret_cast<const uint4*>(ks + t * p.token_stride[0] + ch * 16) : make_uint4(0, 0, 0, 0);
    }
    uint32_t poison = 0;  // tokens with a NaN among their values
    const float vscale = ev == 255 ? 1.f : scale_of(ev);
#pragma unroll
    for (int i = 0; i < kVChunks / 2; ++i) {
      uint32_t* w = &vc[i].x;
      uint32_t any = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t nan = nan_codes(w[j]);
        any |= nan;
        w[j] &= ~((nan >> 7) * 0xffu);
      }
      const uint32_t votes = __ballot_sync(0xffffffffu, any != 0 || ev == 255);
#pragma unroll
      for (int k = 0; k < 32 / kVChunks; ++k)
        if ((votes >> (k * kVChunks)) & ((1u << kVChunks) - 1u)) poison |= 1u << (i * (32 / kVChunks) + k);
      const int at = i * 32 + lane, t = at / kVChunks, ch = at % kVChunks;
      if (t < tokens) store16(p.dst[1] + ((row0 + t) * p.heads_kv + head) * DV + ch * 16, vc[i], vscale);
    }
    const float kscale = scale_of(ek), nan = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < kKChunks / 2; ++i) {
      const int at = i * 32 + lane, t = at / kKChunks, ch = at % kKChunks;
      if (t < tokens)
        store16(p.dst[0] + ((row0 + t) * p.heads_kv + head) * DQK + ch * 16, kc[i], (poison >> t) & 1 ? nan : kscale);
    }
  }
}

template <int DQK, int DV>
void launch_unpack(const UnpackParams& p, int sms, cudaStream_t stream) {
  const int64_t blocks = (((p.total_k >> 4) + p.batch + 8) * p.heads_kv + 7) / 8;
  const int64_t most = static_cast<int64_t>(sms) * 32;
  unpack_kernel<DQK, DV><<<static_cast<unsigned int>(blocks < most ? blocks : most), 256, 0, stream>>>(p);
}

}  // namespace

int unpack_launch(const UnpackParams& p, int d_qk, int d_v, int sms, cudaStream_t stream) {
  unpack_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (d_qk == 64 && d_v == 64) launch_unpack<64, 64>(p, sms, stream);
  else if (d_qk == 128 && d_v == 64) launch_unpack<128, 64>(p, sms, stream);
  else if (d_qk == 128 && d_v == 128) launch_unpack<128, 128>(p, sms, stream);
  else if (d_qk == 192 && d_v == 64) launch_unpack<192, 64>(p, sms, stream);
  else if (d_qk == 192 && d_v == 128) launch_unpack<192, 128>(p, sms, stream);
  else return FA_ERR_UNSUPPORTED;
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
