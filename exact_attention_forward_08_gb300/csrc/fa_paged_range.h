// Which sequences of a call on the paged cache are in range.  The offsets and
// lengths come from device memory and may hold anything, so nothing here is
// subtracted or shifted before it is known to fit.  Plain integer arithmetic,
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

// New tokens of the rows c0 .. c1 - 1 of `total`; -1 if there are no such rows.
FA_HD int paged_new_tokens(int c0, int c1, int64_t total) {
  return c0 >= 0 && c1 >= c0 && c1 <= total ? c1 - c0 : -1;
}

// The n new tokens of a sequence of len tokens, and the position `start` of the
// first; false unless 0 <= n <= len <= most.
FA_HD bool paged_append_range(int c0, int c1, int len, int64_t total, int64_t most, int& start, int& n) {
  n = paged_new_tokens(c0, c1, total);
  start = 0;
  if (n < 0 || len < n || len > most) return false;
  start = len - n;
  return true;
}

// The n new tokens of a sequence whose len tokens are in the cache already (len
// may be below n: rows without a key); false unless 0 <= n <= max_new and 0 <= len <= most.
FA_HD bool paged_attend_range(int c0, int c1, int len, int64_t total, int max_new, int64_t most, int& n) {
  n = paged_new_tokens(c0, c1, total);
  return n >= 0 && n <= max_new && len >= 0 && len <= most;
}

}  // namespace fa
