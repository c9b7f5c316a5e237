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
    q[k] = 0.0;
    if (64 * k < K) q[k] = exp2_64(a[k] - ref);  // (uniform: the lanes' k-th entries may all be missing)
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

// ------------------------------------------------------------------ the teacher's entries in LDS

struct Entries {
  int id[kKdMaxTop];    // -1: left out
  float u[kKdMaxTop];
  float z[kKdMaxTop];   // the student's logit there, -inf where masked
};

// Entry j of row r as thread j < K takes it; id -1 where it is left out, bad where its id is past the
// vocabulary.
__device__ __forceinline__ int entry_id(const KdLoss& l, int64_t r, int j, float& u, bool& bad) {
  const int v = l.ids[r * l.K + j];
  u = l.top[r * l.K + j];
  bad = v >= l.V;
  return bad || v < 0 || u < kMasked ? -1 : v;
}

// ------------------------------------------------------------------ a row's results

struct RowResult {
  float ce, kd, lse, lse_t, lse_rest, off, norm;  // all 0: an ignored row
  uint32_t bad;                                   // bit 0: ce is NaN, bit 1: kd is NaN
};

// One thread writes them.  kd and state may be absent (cross entropy alone).
__device__ __forceinline__ void store_row(const KdLoss& l, int64_t r, const RowResult& o) {
  l.lse[r] = o.lse;
  if (o.bad & 1u) store_nan(l.ce + r);
  else l.ce[r] = o.ce;
  if (!l.kd) return;
  if (o.bad & 2u) store_nan(l.kd + r);
  else l.kd[r] = o.kd;
  *reinterpret_cast<float4*>(l.state + kKdState * r) = make_float4(o.lse_t, o.lse_rest, o.off, o.norm);
}

// The row's results from its log-sums in base 2 (lz: the whole row at the temperature, -inf: no unmasked logit; lr:
// outside the ids), l1 = log sum exp(z), terms = sum_j q_j (c u_j - c z_j).
__device__ __forceinline__ RowResult row_result(const KdLoss& l, const Teacher& te, bool bad, int64_t t, float zt,
                                                double terms, double lz, double lr, double l1) {
  RowResult o{};
  if (!(lz > -kInf64)) {
    o.lse = o.lse_t = ninf();
    return o;
  }
  terms += (lz - te.lq) * (1.0 - te.q_rest);
  if (te.q_rest > 0.0) terms += te.q_rest * ((te.lr - te.lq) - (lr - lz));
  o.kd = te.any ? (float)(terms * kLn2) : 0.0f;
  o.lse = (float)l1;
  o.ce = zt < kMasked ? -ninf() : (float)(l1 - (double)zt);
  o.lse_t = (float)(lz * kLn2);
  o.lse_rest = lr > -kInf64 ? (float)(lr * kLn2) : 0.0f;
  o.off = te.any ? (float)(exp2_64(lr - lz) - te.q_rest) : 0.0f;
  o.norm = (float)(te.lq * kLn2);
  o.bad = (t >= 0 && t < l.V ? 0u : 1u) | (bad ? 2u : 0u);
  return o;
}

// One wave: the row's results from its sums (a: outside the ids at the temperature; TEMP, a1: all columns at
// temperature 1) and entries, valid in every lane; q: the masses of the lane's entries.  t, zt: the target and its
// logit.
template <bool TEMP>
__device__ __forceinline__ RowResult finish_row(const KdLoss& l, int64_t r, const Entries& en, bool bad, int64_t t,
                                                float zt, double c, const Sum2d& a, const Sum2d& a1,
                                                double (&q)[kLaneTop]) {
  const int lane = tid_x() & 63, K = (int)l.K;
  double ua[kLaneTop];
  const Teacher te = teacher_of(en.id, en.u, K, lane, c, l.rest ? l.rest[r] : ninf(), ua, q);
  const double lr = log2_of(a);
  double t2[kLaneTop], m = lr;
#pragma unroll
  for (int k = 0; k < kLaneTop; ++k) {
    const int j = lane + 64 * k;
    const bool here = j < K && en.id[j] >= 0;
    t2[k] = here && !(en.z[j] < kMasked) ? (double)en.z[j] * c : -kInf64;
    m = __builtin_fmax(m, t2[k]);
  }
  m = wave_max64(m);
  if (!(m > -kInf64)) return row_result(l, te, bad, t, zt, 0.0, m, lr, 0.0);
  double s = 0.0, terms = 0.0;
#pragma unroll
  for (int k = 0; k < kLaneTop; ++k) {
    const int j = lane + 64 * k;
    if (j < K && en.id[j] >= 0) {
      if (!named_before(en.id, j)) s += exp2_64(t2[k] - m);
      if (q[k] > 0.0) terms += q[k] * (ua[k] - t2[k]);
    }
  }
  s = wave_sum64(s) + exp2_64(lr - m);
  const double lz = m + log2_64(s);
  return row_result(l, te, bad, t, zt, wave_sum64(terms), lz, lr, TEMP ? log2_of(a1) * kLn2 : lz * kLn2);
}

// ------------------------------------------------------------------ a row's gradient

// What the gradient of a row needs, in fp32 (uniform).
struct RowGrad {
  float kce, kkd;     // k g_ce, k g_kd / T, with the row's factors
  float n1;           // lse log2 e
  float nz, nr;       // log-sums (base 2) at T: the row's, and that of its outside
  float out;          // outside: factor of 2^(c z - nr); at T = 1 with ce's part
};

// k g_ce and k g_kd / T with the row's factors.
struct RowFactors {
  float kce, kkd;
};
__device__ __forceinline__ RowFactors row_factors(const KdGrad& g, const KdLoss& l, int64_t r) {
  const float k = g.g_scale ? *g.g_scale : 1.0f;
  return RowFactors{k * g.g_ce * (g.ce_rows ? g.ce_rows[r] : 1.0f),
                    k * g.g_kd * (g.kd_rows ? g.kd_rows[r] : 1.0f) / l.temperature};
}

template <bool TEMP>
__device__ __forceinline__ RowGrad row_grad(const KdGrad& g, const KdLoss& l, int64_t r, float lse, float lse_t,
                                            float lse_rest, float off) {
  const RowFactors f = row_factors(g, l, r);
  RowGrad o;
  o.kce = f.kce;
  o.kkd = f.kkd;
  o.n1 = lse * kLog2e;
  o.nz = lse_t * kLog2e;
  o.nr = lse_rest * kLog2e;
  o.out = o.kkd * off;
  // (without anything outside, lse_rest is 0 and every such logit masked: the factor only has to be finite)
  if (!TEMP) o.out += o.kce * fminf(exp2_hw(o.nr - o.nz), 1.0f);
  return o;
}

// The gradient at a column outside the ids.
template <bool TEMP>
__device__ __forceinline__ float grad_outside(const RowGrad& g, float x, float c) {
  const float e = g.out * exp2_hw(__builtin_fmaf(x, c, -g.nr));
  return TEMP ? __builtin_fmaf(g.kce, exp2_hw(__builtin_fmaf(x, kLog2e, -g.n1)), e) : e;
}

// At a column of the ids with the teacher's mass q.
__device__ __forceinline__ float grad_named(const RowGrad& g, float x, float c, float q) {
  return g.kce * exp2_hw(__builtin_fmaf(x, kLog2e, -g.n1)) + g.kkd * (exp2_hw(__builtin_fmaf(x, c, -g.nz)) - q);
}

// The mask of a row's ids over the columns [lo, hi) in LDS: bit v - lo of `bits`.  Whether it was set before.
__device__ __forceinline__ bool mark(uint32_t* bits, int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v >= hi) return false;
  const uint32_t bit = 1u << ((v - lo) & 31);
  return (atomicOr(bits + ((v - lo) >> 5), bit) & bit) != 0u;
}

template <typename T>
__device__ __forceinline__ void store8_any(T* p, const float (&o)[8]) {
  unsigned w[sizeof(T) * 2];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (__is_same(T, _Float16)) w[e] = pack_f16x2_rne(o[2 * e], o[2 * e + 1]);
      else w[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
    }
  }
  loose16_t* to = reinterpret_cast<loose16_t*>(p);
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) / 2; ++k)
    __builtin_nontemporal_store((u32x4_t){w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]}, to + k);
}
// For every column of the lanes' groups that an entry names, one after the other: f(lane, e, j), with column base + e of
// that lane's group the one that entry j names (the first of them).  byte: the mask of the lane's group.  All lanes of
// the wave call it, and f, together: an entry is found by all comparing theirs, and not by a walk over K of them.
template <typename F>
__device__ __forceinline__ void for_named(uint32_t byte, int base, const int* id, int K, F f) {
  const int lane = tid_x() & 63;
  uint64_t some = __ballot(byte != 0u);
  while (some) {
    const int at = __builtin_ctzll(some);
    some &= some - 1;
    uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)byte, at);
    const int v = __builtin_amdgcn_readlane(base, at);
    while (b) {
      const int e = __builtin_ctz(b);
      b &= b - 1;
      for (int k = 0; k < K; k += 64) {
        const uint64_t match = __ballot(k + lane < K && id[k + lane] == v + e);
        if (match) {
          f(at, e, k + __builtin_ctzll(match));
          break;
        }
      }
    }
  }
}

}  // namespace lx
