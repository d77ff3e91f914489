// Device helpers of the paged 8-bit key/value cache (fa_kv_append,
// fa_fwd_paged): e4m3 and e8m0 conversions and the search that maps a block of
// work to its sequence.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fa {

// sites of the status word (fa_device_status_detail)
constexpr unsigned int kSitePagedSeq = 511;   // a sequence's offsets, length or position out of range (index: sequence)
constexpr unsigned int kSitePagedPage = 512;  // a block-table entry out of range (index: sequence)
constexpr unsigned int kSitePagedWait = 520;  // a bounded wait of paged_tc_kernel expired
constexpr unsigned int kSitePagedTotal = 513; // the lengths sum to more than total_k (index: 0)
constexpr unsigned int kSiteRotaryPosition = 514;  // a position outside the rotation table (index: token)
constexpr unsigned int kSitePagedFull = 515;  // too few free pages (index: the first row without)

// the smallest scale that the append writes: 2^-63
constexpr int kMinScale = 64;

__device__ __forceinline__ void paged_error(unsigned int* status, unsigned int site, int index) {
  if (atomicCAS(&status[0], 0u, 1u /* FA_ERR_INVALID_ARG */) == 0u) {
    status[1] = site;
    status[2] = static_cast<unsigned int>(index);
  }
}

// two e4m3 codes (low byte first) to two f16, exact; 0x7f and 0xff are NaN
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
// the same for the upper two bytes
__device__ __forceinline__ uint32_t e4m3x2_hi_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}

// four floats to e4m3 codes, rounded to nearest even, beyond 448 saturated, NaN to 0x7f; a in the low byte
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// the scale 2^(e - 127) that an e8m0 byte stands for; 255 is NaN
__device__ __forceinline__ float scale_of(int e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : static_cast<uint32_t>(e) << 23);
}

// A query row whose largest biased bf16 exponent is `top`, as f16: values times
// 2^x, x = 14 - (exponent), which puts the largest into [2^14, 2^15).  Its bf16
// values are then exact down to 2^-31 of 2^exponent (2^-17, 8 bits above f16's
// smallest step of 2^-24); below that they are off by at most 2^-39 of it.  Rows
// whose largest is below 2^-94 are all multiplied by 2^109, which makes the
// smallest bf16 number f16's smallest.  Infinities stay what they are (255: the
// finite values beside them must not become infinite).
struct QueryScale {
  float down, up;  // the factor, and its inverse
};
__device__ __forceinline__ QueryScale query_scale(int top) {
  const int e = top < 32 ? 32 : top > 254 ? 254 : top;
  return {scale_of(268 - e), scale_of(e - 14)};
}

__device__ __forceinline__ float2 f16x2_float2(uint32_t v) {
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}

// The largest i in [0, n) with key(i) <= x for a non-decreasing key (0 if
// there is none), found by the 32 lanes of a warp together: n shrinks 32-fold
// with each round of loads.  Any values of key give an i in range.
template <class F>
__device__ __forceinline__ int warp_search(int n, int64_t x, F key) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int off = lane * step;
    const bool le = off < n && key(lo + off) <= x;
    const int count = __popc(__ballot_sync(0xffffffffu, le));
    const int sel = count > 0 ? (count - 1) * step : 0;
    lo += sel;
    n = n - sel < step ? n - sel : step;
  }
  return lo;
}

}  // namespace fa
