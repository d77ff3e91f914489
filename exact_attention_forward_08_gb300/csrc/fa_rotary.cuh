// Rotation of rows by their positions, shared by fa_kv_append and fa_rotary: the
// columns that a lane holds, its cosines and sines, and the turn itself.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace fa {

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

}  // namespace fa
