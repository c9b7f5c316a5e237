// Sums of exponentials in powers of two against an integer reference, for the kernels over logits that take a
// temperature.
#pragma once

#include "group.hpp"

namespace lx {

constexpr float kMasked = -1.0e30f;  // a logit below it has no mass
constexpr double kInf64 = __builtin_inf();

// The scale of the exponents, log2(e) / T.
inline double scale_of(float temperature) { return kLog2e64 / (double)temperature; }

__device__ __forceinline__ double log2_64(double s) { return log_64(s) * kLog2e64; }

// s 2^n = sum 2^(c x).  c x - n is one fused multiply-add with no rounding of the reference.
struct Sum2 {
  float n, s;
};

// The smallest reference: a masked logit's c x lies below it, so its power of two is 0 against any.
__device__ __forceinline__ float floor_of(float c) { return kMasked * c; }
__device__ __forceinline__ float ref_for(float m, float c) { return fmaxf(__builtin_rintf(m * c), floor_of(c)); }

__device__ __forceinline__ void sum8(const float (&x)[8], float c, float n, float& s0, float& s1) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    s0 += exp2_hw(__builtin_fmaf(x[e], c, -n));
    s1 += exp2_hw(__builtin_fmaf(x[e + 1], c, -n));
  }
}

__device__ __forceinline__ Sum2 wave_sum2(Sum2 a) {
  const float n = wave_max(a.n);
  return Sum2{n, wave_sum32(a.s * exp2_hw(a.n - n))};
}
__device__ __forceinline__ void add_sum2(Sum2& a, const Sum2& b) {
  const float n = fmaxf(a.n, b.n);
  a.s = a.s * exp2_hw(a.n - n) + b.s * exp2_hw(b.n - n);
  a.n = n;
}
// log2 of the sum, -inf without any
__device__ __forceinline__ double log2_of(const Sum2& a) {
  return a.s > 0.0f ? (double)a.n + log2_64((double)a.s) : -kInf64;
}

// The same with the sum in fp64, for what joins the threads' sums: kd is the difference of two logarithms that often
// agree to 10^-2, and a thread's own rounding averages out over a row where that of its last few additions does not
// (fp32, 70 x 438, K 46, T 4: kd off by 5.6e-6 of its value, in fp64 by 6e-8; no time lost).
struct Sum2d {
  float n;
  double s;
};
__device__ __forceinline__ Sum2d wave_sum2d(const Sum2& a) {
  const float n = wave_max(a.n);
  return Sum2d{n, wave_sum64((double)(a.s * exp2_hw(a.n - n)))};
}
__device__ __forceinline__ Sum2d wave_sum2d(const Sum2d& a) {
  const float n = wave_max(a.n);
  return Sum2d{n, wave_sum64(a.s * (double)exp2_hw(a.n - n))};
}
__device__ __forceinline__ void add_sum2d(Sum2d& a, const Sum2d& b) {
  const float n = fmaxf(a.n, b.n);
  a.s = a.s * (double)exp2_hw(a.n - n) + b.s * (double)exp2_hw(b.n - n);
  a.n = n;
}
__device__ __forceinline__ double log2_of(const Sum2d& a) {
  return a.s > 0.0 ? (double)a.n + log2_64(a.s) : -kInf64;
}

// Adds a group's powers of two to s 2^n.  n is a group's maximum before it: a group that goes 2^100 beyond it is taken
// again against its own (as the first one is: n starts below every logit).
__device__ __forceinline__ void add_group(const float (&x)[8], float c, Sum2& a) {
  float p0 = 0.0f, p1 = 0.0f;
  sum8(x, c, a.n, p0, p1);
  if (p0 + p1 >= kRefSumLimit) {
    const float n = fmaxf(a.n, ref_for(max8(x), c));
    a = Sum2{n, a.s * exp2_hw(a.n - n)};
    p0 = p1 = 0.0f;
    sum8(x, c, n, p0, p1);
  }
  a.s += p0 + p1;
}

// One logit.
__device__ __forceinline__ void add_one(Sum2& a, float x, float c) {
  const float n = ref_for(x, c);
  add_sum2(a, Sum2{n, exp2_hw(__builtin_fmaf(x, c, -n))});
}

// The logits of the columns whose bit is set count as masked.
__device__ __forceinline__ void leave_out_bits(uint32_t byte, float (&x)[8]) {
  if (byte) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (byte >> e) & 1u ? ninf() : x[e];
  }
}

}  // namespace lx
