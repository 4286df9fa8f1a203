// An fp64 exponential for the kernels that compare scores and draw tokens (cbk_moe.hip, cbk_sample.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cbk {
namespace {

// e^x for |x| < 700 to some 1e-14 of its value, 0 below -690: 2^n times the exponential series at the rest,
// |r| <= ln 2 / 2, whose first left-out term is r^12 / 12! < 7e-15.  n is rounded by adding 1.5 * 2^52, whose sum then
// holds it in its low bits, and goes into the result's exponent as an integer: conversions and ldexp take as long as four
// multiplications each.
__device__ __forceinline__ double exponential(double x) {
    constexpr double round = 6755399441055744.0;
    const double t = fma(x, 1.4426950408889634074, round), n = t - round;
    double r = fma(n, -0.69314718055994528623, x);
    r = fma(n, -2.3190468138462995584e-17, r);  // ln 2 less its rounding
    double s = 1.0 / 39916800.0;
    s = fma(s, r, 1.0 / 3628800.0);
    s = fma(s, r, 1.0 / 362880.0);
    s = fma(s, r, 1.0 / 40320.0);
    s = fma(s, r, 1.0 / 5040.0);
    s = fma(s, r, 1.0 / 720.0);
    s = fma(s, r, 1.0 / 120.0);
    s = fma(s, r, 1.0 / 24.0);
    s = fma(s, r, 1.0 / 6.0);
    s = fma(s, r, 0.5);
    s = fma(s, r, 1.0);
    s = fma(s, r, 1.0);
    const uint64_t bits = __builtin_bit_cast(uint64_t, s) + (static_cast<uint64_t>(static_cast<uint32_t>(__builtin_bit_cast(uint64_t, t))) << 52);
    return x < -690.0 ? 0.0 : __builtin_bit_cast(double, bits);
}

}  // namespace
}  // namespace cbk
