// exp(x) and exp(x) - 1 in float64 for every x: infinite where float64's are, 0 and -1 far below, NaN for
// NaN.  (Includes nothing of HIP, so that the host can look at it too.)
#pragma once
#include <cmath>

namespace dora {

// exp(x) = 2^n (1 + q) with x = n log 2 + r, |r| <= 0.35, and q the Taylor sum to r^13 / 13!: what is
// left out is under 0.35^14 / 14! = 5e-18, less than float64's own rounding, 2^-53.  log 2 is taken off in
// two parts (Cody and Waite's reduction), the first the float32 next to it, whose products with n are
// exact.  Of 2 10^6 numbers exp is at most 0.7 2^-52 of itself off, exp - 1 1.2 2^-52.
// (Sums of a hundred thousand random terms stay far below a float32 rounding with fewer terms too; a
// ratio next to its bound, whose slope is all or nothing, and a divergence, the small rest of a
// difference, have no such room.)
struct Exponential {
  double q, n;
  __device__ __forceinline__ explicit Exponential(double x) {
    x = x > 1100.0 ? 1100.0 : x < -1100.0 ? -1100.0 : x;   // beyond, both are 0 or infinite; NaN stays
    constexpr double kLog2 = 0.6931471805599453094, kHigh = 0.693147182464599609375;
    constexpr double kLow = -1.904654299957767878e-9;   // log 2 - kHigh
    static_assert(kHigh + kLow == kLog2, "log 2 in two parts");
    n = __builtin_rint(x * 1.4426950408889634);
    const double r = fma(n, -kLow, fma(n, -kHigh, x));
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
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
