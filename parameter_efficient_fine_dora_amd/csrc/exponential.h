// exp(x) and exp(x) - 1 in float64 for every x: infinite where float64's are, 0 and -1 far below, NaN for
// NaN.  (Includes nothing of HIP, so that the host can look at it too.)
#pragma once
#include <cmath>

namespace dora {

// exp(x) = 2^n (1 + q) with x = n log 2 + r, |r| <= 0.35, and q the Taylor sum to r^10 / 10!: what is
// left out is under 0.35^11 / 11! = 2.4e-13 of the result, a thousandth of a float32 rounding and
// less.  (Memory should bound the kernels that use it: the library's exponentials, exact to the last bit of
// float64, took 5 us more of 1M tokens' sums, 17 against 12.)
struct Exponential {
  double q, n;
  __device__ __forceinline__ explicit Exponential(double x) {
    x = x > 1100.0 ? 1100.0 : x < -1100.0 ? -1100.0 : x;   // beyond, both are 0 or infinite; NaN stays
    n = __builtin_rint(x * 1.4426950408889634);
    const double r = fma(n, -0.6931471805599453, x);
    double p = 1.0 / 3628800.0;
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    q = fma(p * r, r, r);
  }
  // 2^n alone is infinite from n = 1024 on, where 2^n (1 + q) may not be and 2^n q is not its part.
  __device__ __forceinline__ double value() const { return ldexp(1.0 + q, (int)n); }
  __device__ __forceinline__ double less_one() const {
    if (n > 64.0) return value();   // (the 1 is below its last bit)
    const double two = ldexp(1.0, (int)n);
    return fma(q, two, two - 1.0);
  }
};

}  // namespace dora
