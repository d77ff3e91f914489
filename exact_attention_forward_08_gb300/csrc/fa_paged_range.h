// Which sequences of a call on the paged cache are in range.  The offsets and
// lengths come from device memory and may hold anything: a difference counts only
// where the comparisons beside it say that it fits.  Plain integer arithmetic,
// compiled for the host too, where a test runs it.
#pragma once
#include <cstdint>

#ifndef FA_HD
#ifdef __CUDACC__
#define FA_HD __host__ __device__ __forceinline__
#else
#define FA_HD inline
#endif
#endif

namespace fa {

// a - b, wrapped where it does not fit
FA_HD int paged_difference(int a, int b) {
  return static_cast<int>(static_cast<uint32_t>(a) - static_cast<uint32_t>(b));
}

// All conditions are evaluated, without a branch: the loads that bring the
// arguments then do not wait for one another.

// Do c0 .. c1 - 1 lie among `total` rows?  Then their number, c1 - c0, fits.
FA_HD bool paged_offsets_ok(int c0, int c1, int64_t total) { return (c0 >= 0) & (c1 >= c0) & (c1 <= total); }

// The n new tokens of a sequence of len tokens, and the position `start` of the
// first; false unless the offsets are in range and n <= len <= most.
FA_HD bool paged_append_range(int c0, int c1, int len, int64_t total, int64_t most, int& start, int& n) {
  n = paged_difference(c1, c0);
  start = paged_difference(len, n);
  return paged_offsets_ok(c0, c1, total) & (len >= n) & (len <= most);
}

// The n new tokens of a sequence whose len tokens are in the cache already (len
// may be below n: rows without a key); false unless the offsets are in range,
// n <= max_new and 0 <= len <= most.
FA_HD bool paged_attend_range(int c0, int c1, int len, int64_t total, int max_new, int64_t most, int& n) {
  n = paged_difference(c1, c0);
  return paged_offsets_ok(c0, c1, total) & (n <= max_new) & (len >= 0) & (len <= most);
}

}  // namespace fa
