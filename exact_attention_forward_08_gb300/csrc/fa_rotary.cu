// Rotary positions: the table of cosines and sines (fa_rotary_table) and the
// rotation of queries and keys, or of their gradients, by it (fa_rotary).
//
// Table.  With the frequency f_i of pair i (radians a position), the angle of
// position p is p f_i.  In turns it is p F_i with F_i = f_i / (2 pi), of which
// only the part behind the point counts: F_i as a 64-bit fraction times p, taken
// modulo 2^64, is that part, exact but for p times F_i's own rounding, a few 2^-53 of
// it.  The nearest quarter turn is split off as an integer, so the sine and cosine are
// taken of an angle x of at most an eighth of a turn that has all its 24 bits: by
// Taylor's series, to x^9 and x^10, whose next terms are below 2^-28 and 2^-32 of
// the values there.  Bound by the stores and the arithmetic alike: 131072 positions of
// 128, 67 MB, 10.9 us (10.0 at the copy rate; 14.7 before two pairs went through packed
// arithmetic together, 19 with sincospif).
//
// Rotation.  A pair (a, b) becomes (a cos - b sin, b cos + a sin) in fp32, each
// product and sum rounded by itself, then rounded to bf16; the gradient turns
// back (sin with its sign changed), which is the transposed map, scaled alike.  Bound
// by DRAM: 20128 tokens of 16/16 heads of 192, 503 MB, 85 us, 5.9 TB/s (75 at the copy
// rate); one token of 32/8 heads of 128: 2.5 to 2.7 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged.cuh"
#include "fa_paged_check.h"
#include "fa_paged_range.h"
#include "fa_rotary.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kMaxRot = 192;

struct TableParams {
  uint64_t turn[kMaxRot / 2];  // turns a position, as a fraction of 2^64
  float* out;
  float magnitude;
  int positions, rot;
};

constexpr int kTableThreads = 256;

__global__ void __launch_bounds__(kTableThreads) rotary_table_kernel(const __grid_constant__ TableParams p) {
  const int half = p.rot >> 1, groups = half >> 2;  // of 4 pairs
  const int rows = kTableThreads / groups;          // positions of a block's step
  const int g = threadIdx.x % groups, r = threadIdx.x / groups;
  if (r >= rows) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  int64_t pos = static_cast<int64_t>(blockIdx.x) * rows + r;
  uint64_t turns[4], more[4];  // at this position, and for a step
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    turns[k] = static_cast<uint64_t>(pos) * p.turn[4 * g + k];
    more[k] = static_cast<uint64_t>(step) * p.turn[4 * g + k];
  }
  for (; pos < p.positions; pos += step) {
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {  // two pairs at a time, in packed arithmetic
      float x[2];
      uint32_t shifted[2];  // the angle plus an eighth of a turn: the quarter in its upper two bits
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        shifted[i] = static_cast<uint32_t>(turns[k + i] >> 32) + 0x20000000u;
        const int rest = static_cast<int>((shifted[i] & 0x3fffffffu) - 0x20000000u);  // of 2^32 a turn
        x[i] = fmaf(static_cast<float>(rest), 0x1p-32f * 6.28318530717958647692f,
                    static_cast<float>(static_cast<uint32_t>(turns[k + i])) * (0x1p-64f * 6.28318530717958647692f));
        turns[k + i] += more[k + i];
      }
      auto both = [](float v) { return f2_pack(v, v); };
      const uint64_t xx = f2_pack(x[0], x[1]), x2 = f2_mul(xx, xx);
      uint64_t sine = f2_fma(x2, both(1.f / 362880.f), both(-1.f / 5040.f));
      sine = f2_fma(sine, x2, both(1.f / 120.f));
      sine = f2_fma(sine, x2, both(-1.f / 6.f));
      sine = f2_fma(f2_mul(sine, x2), xx, xx);
      uint64_t cosine = f2_fma(x2, both(-1.f / 3628800.f), both(1.f / 40320.f));
      cosine = f2_fma(cosine, x2, both(-1.f / 720.f));
      cosine = f2_fma(cosine, x2, both(1.f / 24.f));
      cosine = f2_fma(cosine, x2, both(-0.5f));
      cosine = f2_fma(cosine, x2, both(1.f));
      float sx[2], cx[2];
      f2_unpack(f2_mul(sine, both(p.magnitude)), sx[0], sx[1]);
      f2_unpack(f2_mul(cosine, both(p.magnitude)), cx[0], cx[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool odd = (shifted[i] & 0x40000000u) != 0;
        const uint32_t a = __float_as_uint(odd ? sx[i] : cx[i]), b = __float_as_uint(odd ? cx[i] : sx[i]);
        c[k + i] = __uint_as_float(a ^ ((shifted[i] + 0x40000000u) & 0x80000000u));
        s[k + i] = __uint_as_float(b ^ (shifted[i] & 0x80000000u));
      }
    }
    float* row = p.out + pos * p.rot + 4 * g;
    *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(row + half) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

struct RotaryParams {
  const __nv_bfloat16* src[2];  // queries, keys: rows of heads side by side
  __nv_bfloat16* dst[2];
  int64_t src_stride[2], dst_stride[2];  // elements from token to token
  int heads[2];
  int groups[2], splits;  // groups of heads, warps of a token
  const float* cos_sin;
  const int* positions;  // or
  const int* cu;         // or neither: a token's index modulo seqlen
  unsigned int* status;
  int64_t total, seqlen;
  int batch, max_pos, rot, interleaved;
  uint32_t flip;  // sign bit to change in the sines
};

// A warp holds kHeads heads at a time, 16 values a lane (at d = 192 eight lanes have none).
template <int D>
struct RotaryShape {
  static constexpr int kItems = D / 16;
  static constexpr int kHeads = 32 / kItems;
  // groups of heads whose loads are under way together; us with 2 / 3 / 4 / 6: one token of 32/8 heads of 128 2.7 / 2.8 /
  // 3.1 / 3.4, 8000 tokens 28.1 / 31.6 / 30.5 / 34.4; the 20128 of 16/16 heads of 192 86.3 / 89.3 / 84.6 / 101
  static constexpr int kAhead = D == 192 ? 4 : 2;
  static constexpr int kWarps = 8;
};

// The position of token t, or -1 where it has none (nothing is written then).
__device__ __forceinline__ int rotary_position(const RotaryParams& p, int64_t t) {
  int pos = -1;
  if (p.positions != nullptr) {
    pos = p.positions[t];
  } else if (p.cu != nullptr) {
    const int b = warp_search(p.batch, t, [&](int i) { return p.cu[i]; });
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    if (!paged_offsets_ok(c0, c1, p.total) || t < c0 || t >= c1) return -1;
    pos = static_cast<int>(t) - c0;
  } else {
    pos = static_cast<int>(t % p.seqlen);
  }
  if (pos < 0 || pos >= p.max_pos) {
    paged_error(p.status, kSiteRotaryPosition, static_cast<int>(t));
    return -1;
  }
  return pos;
}

template <int D>
__global__ void __launch_bounds__(32 * RotaryShape<D>::kWarps) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using Shape = RotaryShape<D>;
  const int lane = threadIdx.x & 31;
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (p.cu != nullptr)
    for (int64_t b = thread; b < p.batch; b += static_cast<int64_t>(gridDim.x) * blockDim.x)
      if (!paged_offsets_ok(p.cu[b], p.cu[b + 1], p.total)) paged_error(p.status, kSitePagedSeq, static_cast<int>(b));
  const int64_t warp = thread >> 5, t = warp / p.splits;
  const int split = static_cast<int>(warp - t * p.splits);
  if (t >= p.total) return;
  const int all = p.groups[0] + p.groups[1];
  const int begin = static_cast<int>(static_cast<int64_t>(all) * split / p.splits);
  const int end = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / p.splits);

  const int item = lane % Shape::kItems, off = lane / Shape::kItems;
  const bool turned = item * 16 < p.rot, active = off < Shape::kHeads;
  int first, second;
  item_columns<D>(item, p.rot, first, second);
  uint4 raw[Shape::kAhead][2];
  // the row of this lane's head in group `group`, or NULL
  auto row_of = [&](int group, auto* const (&base)[2], const int64_t (&stride)[2]) {
    const int x = group >= p.groups[0];
    const int head = (x ? group - p.groups[0] : group) * Shape::kHeads + off;
    return active && group < end && head < p.heads[x] ? base[x] + t * stride[x] + head * D : nullptr;
  };
  auto load = [&](int group0) {
#pragma unroll
    for (int i = 0; i < Shape::kAhead; ++i) {
      const __nv_bfloat16* at = row_of(group0 + i, p.src, p.src_stride);
      if (at != nullptr) {
        raw[i][0] = *reinterpret_cast<const uint4*>(at + first);
        raw[i][1] = *reinterpret_cast<const uint4*>(at + second);
      }
    }
  };
  load(begin);  // before the position is known

  const int pos = rotary_position(p, t);
  if (pos < 0) return;
  float cs[16];
  if (turned) {
    load_cos_sin(cs, p.cos_sin + static_cast<int64_t>(pos) * p.rot, item, p.rot, p.interleaved);
#pragma unroll
    for (int j = 8; j < 16; ++j) cs[j] = __uint_as_float(__float_as_uint(cs[j]) ^ p.flip);
  }

  for (int group0 = begin; group0 < end; group0 += Shape::kAhead) {
    if (group0 != begin) load(group0);
#pragma unroll
    for (int i = 0; i < Shape::kAhead; ++i) {
      __nv_bfloat16* at = row_of(group0 + i, p.dst, p.dst_stride);
      if (at == nullptr) continue;
      uint4 (&v)[2] = raw[i];
      if (turned) {
        float y[16];
        unpack8(v[0], y);
        unpack8(v[1], y + 8);
        turn16(y, cs, p.interleaved);
        v[0] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                          pack_bf16x2(y[6], y[7]));
        v[1] = make_uint4(pack_bf16x2(y[8], y[9]), pack_bf16x2(y[10], y[11]), pack_bf16x2(y[12], y[13]),
                          pack_bf16x2(y[14], y[15]));
      }
      *reinterpret_cast<uint4*>(at + first) = v[0];
      *reinterpret_cast<uint4*>(at + second) = v[1];
    }
  }
}

// Warps an SM that a call's tokens are spread over before a warp takes all heads of one.  us with 8 / 32 / 128, 32/8
// heads of 128, four groups ahead: 1000 tokens 5.95 / 4.81 / 4.76, 3000 tokens 9.43 / 9.45 / 10.22, 8000 tokens 30.5 /
// 30.5 / 32.0; up to 256 tokens the same.
constexpr int kRotaryWarps = 32;

template <int D>
cudaError_t rotary_launch(RotaryParams& p, int sms, cudaStream_t stream) {
  using Shape = RotaryShape<D>;
  for (int x = 0; x < 2; ++x) p.groups[x] = (p.heads[x] + Shape::kHeads - 1) / Shape::kHeads;
  const int all = p.groups[0] + p.groups[1], most = (all + Shape::kAhead - 1) / Shape::kAhead;
  int64_t splits = kRotaryWarps * static_cast<int64_t>(sms) / p.total;
  splits = splits < 1 ? 1 : splits > most ? most : splits;
  p.splits = static_cast<int>(splits);
  const int64_t blocks = (p.total * splits + Shape::kWarps - 1) / Shape::kWarps;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  rotary_kernel<D><<<static_cast<int>(blocks), 32 * Shape::kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_rotary_table(float* cos_sin, int positions, int rot_dim, double base, const fa_rotary_scaling* scaling,
                    fa_stream_t stream) {
  fa_rotary_scaling s = {FA_ROTARY_PLAIN, 1.0, 0.0, 1.0, 2.0, 1.0};
  if (scaling != nullptr) s = *scaling;
  if (positions < 0 || rot_dim < 16 || rot_dim > kMaxRot || rot_dim % 16 != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base < 1.0) return FA_ERR_INVALID_ARG;
  if (s.kind < FA_ROTARY_PLAIN || s.kind > FA_ROTARY_BY_PARTS) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(s.magnitude) || s.magnitude < 0x1p-64 || s.magnitude > 0x1p64) return FA_ERR_INVALID_ARG;
  if (s.kind != FA_ROTARY_PLAIN && (!std::isfinite(s.factor) || s.factor < 1.0)) return FA_ERR_INVALID_ARG;
  if (s.kind == FA_ROTARY_BY_PARTS && (!std::isfinite(s.original) || s.original <= 0.0 || !std::isfinite(s.low) ||
                                       !std::isfinite(s.high) || s.low < 0.0 || s.high <= s.low))
    return FA_ERR_INVALID_ARG;
  if (s.kind == FA_ROTARY_BASE) base *= std::pow(s.factor, rot_dim / (rot_dim - 2.0));
  if (!std::isfinite(base)) return FA_ERR_INVALID_ARG;
  if (positions == 0) return FA_OK;
  if (cos_sin == nullptr || !aligned(cos_sin, 16)) return FA_ERR_INVALID_ARG;

  TableParams p;
  std::memset(&p, 0, sizeof(p));
  const double two_pi = 6.283185307179586476925;
  const int half = rot_dim / 2;
  for (int i = 0; i < half; ++i) {
    double f = std::pow(base, -static_cast<double>(i) / half);
    if (s.kind == FA_ROTARY_LINEAR) f /= s.factor;
    if (s.kind == FA_ROTARY_BY_PARTS) {
      double keep = (s.original * f / two_pi - s.low) / (s.high - s.low);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = f * keep + f / s.factor * (1.0 - keep);
    }
    p.turn[i] = static_cast<uint64_t>(std::nearbyint(f / two_pi * 0x1p64));  // f <= 1: below 2^62
  }
  p.out = cos_sin;
  p.magnitude = static_cast<float>(s.magnitude);
  p.positions = positions;
  p.rot = rot_dim;

  HostDevice host;
  const int rc = host_device(&host);
  if (rc != FA_OK) return rc;
  if (!host_is_device_ptr(cos_sin, host.dev)) return FA_ERR_INVALID_ARG;
  const int rows = kTableThreads / (half / 4);
  const int64_t blocks = (static_cast<int64_t>(positions) + rows - 1) / rows, most = 8 * static_cast<int64_t>(host.sms);
  rotary_table_kernel<<<static_cast<int>(blocks < most ? blocks : most), kTableThreads, 0,
                        reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_rotary(const void* q, const void* k, void* q_out, void* k_out, int64_t q_stride, int64_t k_stride,
              int64_t q_out_stride, int64_t k_out_stride, const int* positions, const int* cu_seqlens, int batch,
              int64_t seqlen, int64_t total, int heads_q, int heads_k, int d, const float* cos_sin, int max_positions,
              int rot_dim, int interleaved, int backward, fa_stream_t stream_) {
  if (d != 64 && d != 128 && d != 192) return FA_ERR_UNSUPPORTED;
  if (total < 0 || total >= (int64_t(1) << 31) || heads_q < 0 || heads_k < 0) return FA_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0 || max_positions < 1) return FA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (backward != 0 && backward != 1)) return FA_ERR_INVALID_ARG;
  if (positions != nullptr && cu_seqlens != nullptr) return FA_ERR_INVALID_ARG;
  if (cu_seqlens != nullptr && (batch < 0 || batch > kMaxBatch)) return FA_ERR_INVALID_ARG;
  if (positions == nullptr && cu_seqlens == nullptr && seqlen < 1 && total > 0) return FA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (q == nullptr) heads_q = 0;
  if (k == nullptr) heads_k = 0;
  // the batch kept at 65536 heads a token: offsets inside a token fit 32 bits
  if (heads_q > 65536 || heads_k > 65536) return FA_ERR_INVALID_ARG;
  if (total == 0 || heads_q + heads_k == 0 || (cu_seqlens != nullptr && batch == 0)) return FA_OK;
  if (cos_sin == nullptr || !aligned(cos_sin, 16) || !aligned(positions, 4) || !aligned(cu_seqlens, 4))
    return FA_ERR_INVALID_ARG;
  const int64_t most = int64_t(1) << 40;
  const void* src[2] = {q, k};
  void* dst[2] = {q_out, k_out};
  const int64_t in[2] = {q_stride, k_stride}, out[2] = {q_out_stride, k_out_stride};
  const int heads[2] = {heads_q, heads_k};
  for (int x = 0; x < 2; ++x) {
    if (heads[x] == 0) continue;
    const int64_t row = static_cast<int64_t>(heads[x]) * d;
    if (!aligned(src[x], 16) || !aligned(dst[x], 16)) return FA_ERR_INVALID_ARG;
    for (int64_t s : {in[x], out[x]})
      if (s % 8 != 0 || s < row || s >= most) return FA_ERR_INVALID_ARG;
    if (src[x] == dst[x] && in[x] != out[x] && total > 1) return FA_ERR_INVALID_ARG;  // in place: the same rows
  }

  if (heads_q > 0 && heads_k > 0 && (q_out == k_out || q_out == k || k_out == q)) return FA_ERR_INVALID_ARG;

  HostDevice host;
  const int rc = host_device(&host);
  if (rc != FA_OK) return rc;
  for (int x = 0; x < 2; ++x)
    if (heads[x] > 0 && (!host_is_device_ptr(src[x], host.dev) || !host_is_device_ptr(dst[x], host.dev)))
      return FA_ERR_INVALID_ARG;
  if (!host_is_device_ptr(cos_sin, host.dev) || (positions != nullptr && !host_is_device_ptr(positions, host.dev)) ||
      (cu_seqlens != nullptr && !host_is_device_ptr(cu_seqlens, host.dev)))
    return FA_ERR_INVALID_ARG;

  RotaryParams p;
  std::memset(&p, 0, sizeof(p));
  for (int x = 0; x < 2; ++x) {
    p.src[x] = static_cast<const __nv_bfloat16*>(src[x]);
    p.dst[x] = static_cast<__nv_bfloat16*>(dst[x]);
    p.src_stride[x] = in[x];
    p.dst_stride[x] = out[x];
    p.heads[x] = heads[x];
  }
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.cu = cu_seqlens;
  p.status = host.status;
  p.total = total;
  p.seqlen = seqlen;
  p.batch = batch;
  p.max_pos = max_positions;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.flip = backward ? 0x80000000u : 0u;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const cudaError_t e = d == 64    ? rotary_launch<64>(p, host.sms, stream)
                        : d == 128 ? rotary_launch<128>(p, host.sms, stream)
                                   : rotary_launch<192>(p, host.sms, stream);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
