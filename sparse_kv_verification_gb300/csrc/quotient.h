// Integer quotients from a reciprocal in fp32, exact within stated limits.
// Plain C++, so that a test on the host holds the arithmetic.
#pragma once

#ifdef __CUDACC__
#define DUSTIN_HD __host__ __device__ __forceinline__
#else
#define DUSTIN_HD inline
#endif

namespace dustin {

DUSTIN_HD float reciprocal(int d) {
#ifdef __CUDA_ARCH__
  return __frcp_rn((float)d);
#else
  return 1.f / (float)d;
#endif
}

// floor(x / d) for x >= 0, d > 0, from inv, 1 / d rounded to fp32.  x, 1 / d and
// their product are rounded by 2^-24 each (relative), so a quotient below 2^22
// is estimated to within one.
DUSTIN_HD int quotient(int x, int d, float inv) {
  const int q = (int)((float)x * inv), r = x - q * d;
  return q + (r >= d) - (r < 0);
}
DUSTIN_HD int quotient(int x, int d) { return quotient(x, d, reciprocal(d)); }
DUSTIN_HD int quotient_up(int x, int d, float inv) { return quotient(x + d - 1, d, inv); }
DUSTIN_HD int quotient_up(int x, int d) { return quotient(x + d - 1, d); }

// The same for quotients of any size, x < 2^30: the estimate is off by at most 3 x
// 2^-24 of the quotient and one, so the rest that it leaves is divided once more.
DUSTIN_HD int quotient_wide(int x, int d, float inv) {
  const int q = (int)((float)x * inv);
  int r = x - q * d;
  const int more = (int)((float)r * inv);   // rounded to zero
  r -= more * d;
  return q + more + (r >= d) - (r < 0);
}
DUSTIN_HD int quotient_wide(int x, int d) { return quotient_wide(x, d, reciprocal(d)); }

}  // namespace dustin
