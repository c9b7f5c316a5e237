// Rows in groups of 8 logits, fp64 exponentials and logarithms of a row's few sums, reductions over
// a wave and the exchange of values between workgroups, for the kernels over logits whose rows may
// start on any element.
#pragma once

#include "common.hpp"

namespace lx {

constexpr double kLog2e64 = 1.4426950408889634074;
constexpr double kLn2 = 0.69314718055994530942;


typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
// 16 bytes at any element (gfx950 loads and stores them at any address).
typedef u32x4_t __attribute__((aligned(2))) loose16_t;

// ------------------------------------------------------------------ rows

// 8 consecutive logits as they lie in memory.  Rows may start on any element
// (odd vocabularies, views), so the loads carry the element's alignment only;
// gfx950 runs 16-byte loads at any address.
template <typename T>
struct Group;
template <>
struct Group<uint16_t> {
  u32x4_t w;
  __device__ __forceinline__ void load(const uint16_t* p) { __builtin_memcpy(&w, p, 16); }
  // read once: non-temporal
  __device__ __forceinline__ void load_once(const uint16_t* p) {
    w = __builtin_nontemporal_load(reinterpret_cast<const loose16_t*>(p));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const unsigned w0 = w.x, w1 = w.y, w2 = w.z, w3 = w.w;
    x[0] = __uint_as_float(w0 << 16); x[1] = __uint_as_float(w0 & 0xffff0000u);
    x[2] = __uint_as_float(w1 << 16); x[3] = __uint_as_float(w1 & 0xffff0000u);
    x[4] = __uint_as_float(w2 << 16); x[5] = __uint_as_float(w2 & 0xffff0000u);
    x[6] = __uint_as_float(w3 << 16); x[7] = __uint_as_float(w3 & 0xffff0000u);
  }
};
template <>
struct Group<_Float16> {
  u32x4_t w;
  __device__ __forceinline__ void load(const _Float16* p) { __builtin_memcpy(&w, p, 16); }
  __device__ __forceinline__ void load_once(const _Float16* p) {
    w = __builtin_nontemporal_load(reinterpret_cast<const loose16_t*>(p));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const unsigned w0 = w.x, w1 = w.y, w2 = w.z, w3 = w.w;
    unpack_f16x2(w0, x[0], x[1]); unpack_f16x2(w1, x[2], x[3]);
    unpack_f16x2(w2, x[4], x[5]); unpack_f16x2(w3, x[6], x[7]);
  }
};
template <>
struct Group<float> {
  u32x4_t w, v;
  __device__ __forceinline__ void load(const float* p) {
    __builtin_memcpy(&w, p, 16);
    __builtin_memcpy(&v, p + 4, 16);
  }
  __device__ __forceinline__ void load_once(const float* p) {
    w = __builtin_nontemporal_load(reinterpret_cast<const loose16_t*>(p));
    v = __builtin_nontemporal_load(reinterpret_cast<const loose16_t*>(p + 4));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const unsigned a[8] = {w.x, w.y, w.z, w.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(a[k]);
  }
};

__device__ __forceinline__ float ninf() { return -__builtin_inff(); }

// The 8 logits of elements v .. v + 7 of a row, -inf (mass 0) from `end` on.
template <typename T>
__device__ __forceinline__ void load_edge(const T* row, int64_t v, int64_t end, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = v + k < end ? load1(row + v + k) : ninf();
}

// Hides a held group from common-subexpression elimination, so that its packed registers live
// from one use to the next and not the (two to four times as many) widened floats.
__device__ __forceinline__ void launder(u32x4_t& w) {
  unsigned a = w.x, b = w.y, c = w.z, d = w.w;
  asm volatile("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
  w = (u32x4_t){a, b, c, d};
}
template <typename T>
__device__ __forceinline__ void launder(Group<T>& g) {
  launder(g.w);
  if constexpr (sizeof(T) == 4) launder(g.v);
}

// ------------------------------------------------------------------ arithmetic

// 2^t for t <= 0 in fp64 to a few 1e-15: t = n + f with |f| <= 1/2, and the Taylor
// series of e^(f ln 2) to the 12th power (|f ln 2| <= 0.347: the rest is below 2e-16).
__device__ __forceinline__ double exp2_64(double t) {
  t = t > -1100.0 ? t : -1100.0;  // 2^-1100 is 0 in fp64, and -inf would make n - n below NaN
  const double n = __builtin_rint(t);
  const double g = (t - n) * kLn2;
  double s = 1.0 / 479001600.0;
  s = __builtin_fma(s, g, 1.0 / 39916800.0);
  s = __builtin_fma(s, g, 1.0 / 3628800.0);
  s = __builtin_fma(s, g, 1.0 / 362880.0);
  s = __builtin_fma(s, g, 1.0 / 40320.0);
  s = __builtin_fma(s, g, 1.0 / 5040.0);
  s = __builtin_fma(s, g, 1.0 / 720.0);
  s = __builtin_fma(s, g, 1.0 / 120.0);
  s = __builtin_fma(s, g, 1.0 / 24.0);
  s = __builtin_fma(s, g, 1.0 / 6.0);
  s = __builtin_fma(s, g, 0.5);
  s = __builtin_fma(s, g, 1.0);
  s = __builtin_fma(s, g, 1.0);
  return __builtin_ldexp(s, (int)n);
}

// log s for 0 < s < inf: s = 2^k m with m in [1/sqrt 2, sqrt 2), and log m = 2 atanh(y),
// y = (m - 1) / (m + 1), |y| <= 0.1716, by its series to y^19 (the rest is below 1e-17).
__device__ __forceinline__ double log_64(double s) {
  const uint64_t b = __builtin_bit_cast(uint64_t, s);
  int k = (int)(b >> 52) - 1023;
  double m = __builtin_bit_cast(double, (b & 0xfffffffffffffull) | 0x3ff0000000000000ull);
  if (m > 1.4142135623730951) {
    m *= 0.5;
    k += 1;
  }
  const double y = (m - 1.0) / (m + 1.0), y2 = y * y;
  double t = 1.0 / 19.0;
#pragma unroll
  for (int d = 17; d >= 1; d -= 2) t = __builtin_fma(t, y2, 1.0 / (double)d);
  return __builtin_fma((double)k, kLn2, 2.0 * y * t);
}

// ------------------------------------------------------------------ reductions over a wave

// Over the 64 lanes on the vector ALU: quad permutations and rotations inside each row of 16
// lanes, then the gfx950 swaps of rows and of halves.  (These reductions sit one behind the
// other on every call's critical path; through LDS permutes they took several times as long.)
template <int CTRL>
__device__ __forceinline__ unsigned dpp(unsigned v) {
  return (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
template <typename T, typename F>
__device__ __forceinline__ T wave_all(T v, F f) {
  constexpr int kWords = sizeof(T) / 4;
  struct Words {
    unsigned w[kWords];
  };
  auto step = [&](auto move) {
    Words a = __builtin_bit_cast(Words, v), o;
#pragma unroll
    for (int k = 0; k < kWords; ++k) o.w[k] = move(a.w[k]);
    v = f(v, __builtin_bit_cast(T, o));
  };
  step([](unsigned u) { return dpp<0xB1>(u); });   // quad_perm [1, 0, 3, 2]
  step([](unsigned u) { return dpp<0x4E>(u); });   // quad_perm [2, 3, 0, 1]
  step([](unsigned u) { return dpp<0x124>(u); });  // row_ror 4
  step([](unsigned u) { return dpp<0x128>(u); });  // row_ror 8
  // (a swap of a value with itself leaves one row's value in the first result and the other's in the
  // second, for the lanes of both; the elements go through scalars, which this compiler needs)
  auto both = [&](auto swap) {
    Words a = __builtin_bit_cast(Words, v), x, y;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const auto pr = swap(a.w[k]);
      const unsigned lo = pr[0], hi = pr[1];
      x.w[k] = lo;
      y.w[k] = hi;
    }
    v = f(__builtin_bit_cast(T, x), __builtin_bit_cast(T, y));
  };
  both([](unsigned u) { return __builtin_amdgcn_permlane16_swap(u, u, false, false); });
  both([](unsigned u) { return __builtin_amdgcn_permlane32_swap(u, u, false, false); });
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_all(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum32(float v) {
  return wave_all(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ double wave_sum64(double v) {
  return wave_all(v, [](double a, double b) { return a + b; });
}
__device__ __forceinline__ unsigned wave_min_u(unsigned v) {
  return wave_all(v, [](unsigned a, unsigned b) { return a < b ? a : b; });
}

// ------------------------------------------------------------------ exchange between workgroups

// What one workgroup hands to another inside a launch goes through device-coherent
// atomics, which pass the caches of the chip's dies by.  A workgroup publishes,
// waits until its stores have been acknowledged, and counts itself; the one that
// counts last reads.  Nobody waits for anybody.
__device__ __forceinline__ void publish(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t fetch(const uint64_t* p) {
  return __hip_atomic_load(const_cast<uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint64_t* p, double v) { publish(p, __builtin_bit_cast(uint64_t, v)); }
__device__ __forceinline__ double fetch64(const uint64_t* p) { return __builtin_bit_cast(double, fetch(p)); }
__device__ __forceinline__ uint64_t pack(float lo, unsigned hi) {
  return (uint64_t)__float_as_uint(lo) | ((uint64_t)hi << 32);
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((unsigned)v); }
__device__ __forceinline__ unsigned hi_of(uint64_t v) { return (unsigned)(v >> 32); }

// Called by thread 0 after its publish(): whether this workgroup is the last of `of`.
__device__ __forceinline__ bool count_last(int* counter, int of) {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);  // the published values have reached memory
  asm volatile("" ::: "memory");
  const bool last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == of - 1;
  asm volatile("" ::: "memory");
  return last;
}

}  // namespace lx
