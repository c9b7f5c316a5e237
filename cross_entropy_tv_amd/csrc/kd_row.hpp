// A row's teacher and the loss from its sums (the kernels over logits and the lm_head path share it).
//
// A token's teacher is K of its logits u_j with their ids and the log-sum-exp R of the others (or
// nothing of the others).  With T the temperature, in units of base-2 exponents (c = log2(e) / T):
//
//   lq  = log2( sum_j 2^(c u_j) + 2^(R log2 e) ),  q_j = 2^(c u_j - lq),  q_r = 2^(R log2 e - lq)
//   lr  = log2 of the student's sum outside the teacher's ids,  lz = log2 of its whole sum
//   kd  = ln 2 ( sum_j q_j ((c u_j - lq) - (c z_j - lz)) + q_r ((R log2 e - lq) - (lr - lz)) )
//
// The student's sum outside the ids is added up without the ids' logits, never as a difference, so
// that p_r = 2^(lr - lz) is good to fp32 relatively however small it is.  The K terms of a row are
// formed in fp64: kd is the difference of two logarithms of size 10 that often agree to 10^-2.
//
// A logit below -1e30 is masked.  An entry is left out where its id is negative or its logit masked;
// an id of V or more makes the row's kd and gradient NaN.  An id given twice is two entries of one
// token: its p counts once, its q is the sum.
#pragma once

#include "distill.hpp"
#include "group.hpp"
#include "sum2.hpp"

namespace lx {

__device__ __forceinline__ double wave_max64(double v) {
  return wave_all(v, [](double a, double b) { return __builtin_fmax(a, b); });
}

// What the K entries of a row say, held by one wave: lane l has entries l + 64 k.
struct Teacher {
  double lq, lr, q_rest;  // lr: R log2 e, -inf without one
  bool any;               // something has mass
};

constexpr int kLaneTop = kKdMaxTop / 64;

// a[k]: c u of the lane's entries, -inf for those left out; q[k] their masses.
__device__ __forceinline__ Teacher teacher_of(const int* id, const float* u, int K, int lane, double c, float rest,
                                              double (&a)[kLaneTop], double (&q)[kLaneTop]) {
  Teacher t;
  t.lr = rest < kMasked ? -kInf64 : (double)rest * kLog2e64;
  double m = t.lr;
#pragma unroll
  for (int k = 0; k < kLaneTop; ++k) {
    const int j = lane + 64 * k;
    a[k] = j < K && id[j] >= 0 ? (double)u[j] * c : -kInf64;
    m = __builtin_fmax(m, a[k]);
  }
  m = wave_max64(m);
  t.any = m > -kInf64;
  const double ref = t.any ? m : 0.0;
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kLaneTop; ++k) {
    q[k] = exp2_64(a[k] - ref);
    s += q[k];
  }
  t.q_rest = exp2_64(t.lr - ref);
  s = wave_sum64(s) + t.q_rest;
  const double inv = t.any ? 1.0 / s : 0.0;
  t.lq = t.any ? ref + log2_64(s) : 0.0;
#pragma unroll
  for (int k = 0; k < kLaneTop; ++k) q[k] *= inv;
  t.q_rest *= inv;
  return t;
}

// Whether entry j names a token that an entry before it names.
__device__ __forceinline__ bool named_before(const int* id, int j) {
  bool seen = false;
  for (int i = 0; i < j; ++i) seen |= id[i] == id[j];
  return seen;
}

struct RowOut {
  float kd, lse_t, lse_rest, off, norm;
};

// kd and the row's state from its log-sums (base 2; lr -inf: nothing outside the ids) and
// terms = sum_j q_j (c u_j - c z_j).
__device__ __forceinline__ RowOut row_out(const Teacher& t, double terms, double lz, double lr) {
  RowOut o;
  terms += (lz - t.lq) * (1.0 - t.q_rest);
  if (t.q_rest > 0.0) terms += t.q_rest * ((t.lr - t.lq) - (lr - lz));
  o.kd = t.any ? (float)(terms * kLn2) : 0.0f;
  o.lse_t = (float)(lz * kLn2);
  o.lse_rest = lr > -kInf64 ? (float)(lr * kLn2) : 0.0f;
  o.off = t.any ? (float)(exp2_64(lr - lz) - t.q_rest) : 0.0f;
  o.norm = (float)(t.lq * kLn2);
  return o;
}

// The mask of a row's ids over the columns [lo, hi) in LDS: bit v - lo of `bits`.
__device__ __forceinline__ void mark(uint32_t* bits, int64_t v, int64_t lo, int64_t hi) {
  if (v >= lo && v < hi) atomicOr(bits + ((v - lo) >> 5), 1u << ((v - lo) & 31));
}

}  // namespace lx
