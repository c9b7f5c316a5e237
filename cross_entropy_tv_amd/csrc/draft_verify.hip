// Verification of drafted tokens against the target's probabilities.
//
// Sequence i has n_i drafted tokens x_0 .. x_{n_i - 1}, a row of target logits
// for each of them and one more for the token behind the last, and a row of
// draft logits for each.  With p = softmax(z / T), q = softmax(u / T) of a
// position and its random number r in [0, 1):
//
//   x is accepted when r q(x) < p(x)                  (probability min(1, p / q));
//   the first rejection at position a ends the sequence, and its token is drawn
//   from max(p - q, 0) / sum max(p - q, 0)             (1 / sum = 1 / tvd);
//   with every draft accepted (a = n_i) the token is drawn from p.
//
// The emitted tokens are then distributed as the target's own (the total
// variation distance that the loss trains down is the rejection probability).
// A token is drawn by inversion: the smallest v whose running sum of masses
// exceeds w * total, w in [0, 1) given.  Without draft logits q is 1 at the
// drafted token: accepted when r < p(x), and x is left out of the draw.  T = 0
// takes the first largest logit throughout.
//
// What bounds it: reading the logits, once for every position that is reached.
// Three steps:
//
//   1. verify_accept_kernel, one workgroup per (position, sequence, chunk of the
//      row), position by position: partial sums of exponentials of target and draft in
//      fp32; the last workgroup of a position merges them and decides.  Workgroups
//      of positions behind a rejection already decided read nothing: they look,
//      and never wait (the results do not depend on what they see).
//   2. verify_sums_kernel, one workgroup per (sequence, chunk) of the one row that
//      the token is drawn from: fp64 sums of the masses.  Where they need no draft
//      the last workgroup draws.
//   3. verify_draw_kernel (draft logits): the fp64 sums of max(p - q, 0), and
//      the draw by the last workgroup.
//
// A few sequences, whose rows all fit on the chip at once, are bound by latency instead: two steps,
// verify_rows_kernel with fp64 sums of every position and of the row behind the drafts, and the draw.
//
// Precision.  An answer here is a whole number that a comparison decides, so the
// values compared are held tighter than the rounding of the logits would ask
// for.  The acceptance compares r q(x) with p(x) from fp32 sums (of 64 elements a
// lane at most, 48 additions one behind the other: good to 2^-18, a few 2^-21 as a
// rule; chunks are joined in fp64) and, where the two lie within 2^-15 of each
// other, again from fp64 sums over both rows.  The draw's running sums are fp64 throughout: with 150 000
// tokens the borders between them lie too close for fp32 sums to tell which side
// w * total falls on.
#include "common.hpp"
#include "verify.hpp"

namespace lx {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWaves = kVThreads / 64;
constexpr int kVUnit = kVThreads * 8;  // elements that one load of every thread covers
constexpr int kVMaxChunks = 1024;      // chunks of a row at most (the draw keeps their sums in LDS)
constexpr float kBorder = 0x1p-15f;
// max(p - q, 0) sums to the total variation distance.  Below 2^-40 it is the rounding of equal rows
// (a rejection there has a probability of less than that).
constexpr double kNothing = 0x1p-40;
constexpr double kLog2e64 = 1.4426950408889634074;
constexpr double kLn2 = 0.69314718055994530942;

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

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

// H groups of a thread: elements b + k kVUnit + 8 tid .. + 7 of a row of V, k < H, -inf behind its
// end.  In two parts, so that several rows' loads can be in flight; no load is conditional.
template <typename T, int H>
__device__ __forceinline__ void hold(const T* row, int64_t b, int64_t V, Group<T> (&g)[H]) {
  if (V < 8) return;
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const int64_t v = b + k * kVUnit + tid_x() * 8;
    g[k].load(row + (v < V - 8 ? v : V - 8));
  }
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
template <typename T>
__device__ __forceinline__ void held(const T* row, int64_t v, int64_t V, const Group<T>& g, float (&x)[8]) {
  if (v + 8 <= V) g.get(x);
  else load_edge(row, v, V, x);
}

// Element `at` (-1: none) of v .. v + 7 has no mass.
__device__ __forceinline__ void leave_out(int64_t v, int64_t at, float (&x)[8]) {
  if (at >= v && at < v + 8) {
    const int out = (int)(at - v);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k == out ? ninf() : x[k];
  }
}

// Elements [lo, hi) of a row of V, lo a multiple of kVUnit: f(v, x) for every group of 8 of this
// thread, with H groups loaded at once.
template <int H, typename T, typename F>
__device__ __forceinline__ void for_groups(const T* row, int64_t lo, int64_t hi, int64_t V, F f) {
  for (int64_t b = lo; b < hi; b += kVUnit * H) {
    Group<T> g[H];
    hold<T, H>(row, b, V, g);
    float x[8];
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const int64_t v = b + k * kVUnit + tid_x() * 8;
      if (v < hi) {
        held(row, v, V, g[k], x);
        f(v, x);
      }
    }
  }
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

// The same for the passes over whole rows, with 2^(j / 64) from a table in LDS: t = k / 64 + f with |f| <=
// 1/128 leaves 5 powers (|f ln 2| <= 0.0054: the rest is below 4e-17), two thirds of the instructions.  k
// comes from adding 1.5 2^46, whose last place is 1/64.
constexpr int kExpTable = 64;
__device__ __forceinline__ void exp_table(double (&tab)[kExpTable]) {
  if (tid_x() < kExpTable) tab[tid_x()] = exp2_64(((double)(int)tid_x() - kExpTable) / kExpTable) * 2.0;
}
__device__ __forceinline__ double exp2_64(double t, const double (&tab)[kExpTable]) {
  constexpr double l = kLn2, round = 0x1.8p46;
  t = __builtin_fmax(t, -1100.0);
  const double u = t + round, f = t - (u - round);
  const int k = (int)(unsigned)__builtin_bit_cast(uint64_t, u);
  double s = l * l * l * l * l / 120.0;
  s = __builtin_fma(s, f, l * l * l * l / 24.0);
  s = __builtin_fma(s, f, l * l * l / 6.0);
  s = __builtin_fma(s, f, l * l / 2.0);
  s = __builtin_fma(s, f, l);
  const double e = tab[k & (kExpTable - 1)];
  return __builtin_ldexp(__builtin_fma(e, s * f, e), k >> 6);
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

// The scale of a sequence's exponents: e^((z - m) / T) = 2^((z - m) scale).
struct Temp {
  bool greedy;
  float c;
  double c64, inv;
};
__device__ __forceinline__ Temp temp_of(const float* temperature, int i) {
  const float t = temperature ? temperature[i] : 1.0f;
  Temp r;
  r.greedy = !(t > 0.0f);
  // (infinitely hot: all finite logits alike; -inf times the scale must stay -inf)
  const double d = r.greedy ? 1.0 : (double)fminf(t, 1.0e37f);
  r.inv = 1.0 / d;
  r.c64 = kLog2e64 / d;
  // (finite also for the smallest temperatures: 0 * c must stay 0 at the largest logit)
  r.c = r.c64 < 3.0e38 ? (float)r.c64 : 3.0e38f;
  return r;
}

// A reference for exponents: the maximum, or 0 for a row without any mass (-inf - 0 = -inf: all masses 0).
__device__ __forceinline__ float ref_of(float m) { return m == ninf() ? 0.0f : m; }

struct Sum64 {
  float m;
  double s;
};
struct Best {
  float v;
  unsigned at;
};
constexpr unsigned kNone = 0xffffffffu;

__device__ __forceinline__ void add8(Best& a, int64_t v, const float (&x)[8]) {
  const float m = max8(x);
  if (m > a.v) {
    a.v = m;
#pragma unroll
    for (int k = 7; k >= 0; --k) {
      if (x[k] == m) a.at = (unsigned)(v + k);
    }
  }
}

// ------------------------------------------------------------------ reductions over a workgroup

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

// Inclusive prefix sums over the wave: row shifts inside the rows of 16 lanes, then the
// last lane of a row to the next row, and of the first half to the second.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_shift64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWS, 0xF, true);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWS, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double wave_scan64(double v) {
  v += dpp_shift64<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8 (0 comes in)
  v += dpp_shift64<0x112, 0xF>(v);
  v += dpp_shift64<0x114, 0xF>(v);
  v += dpp_shift64<0x118, 0xF>(v);
  v += dpp_shift64<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
  v += dpp_shift64<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
  return v;
}

// A sum of exponentials against its maximum, as what there is beside one element at the
// maximum: the sum is 1 + rest.  A token of probability near 1 has log p = -log(1 + rest), which
// rest gives to its own relative precision and a rounded sum would not.
struct Sum32 {
  float m, rest;  // m = -inf: nothing with mass
};

// A lane's running sum: s = sum of 2^((x - m) c).
struct LaneSum {
  float m, s;
};
__device__ __forceinline__ void add8(LaneSum& a, const float (&x)[8], float c) {
  const float mn = fmaxf(a.m, max8(x));
  const float ref = ref_of(mn);
  float s0 = a.s * exp2_hw((a.m - ref) * c), s1 = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    s0 += exp2_hw((x[k] - ref) * c);
    s1 += exp2_hw((x[k + 1] - ref) * c);
  }
  a.m = mn;
  a.s = s0 + s1;
}

// The wave's sum over elements [lo, hi) of a row of V, of which lane l of the workgroup's wave took
// elements lo + k kVUnit + 8 tid .. + 7.  What a lane's sum lost below the 1 of its largest element
// matters in one lane only, the (first) one that holds the wave's maximum: its elements are summed
// once more, an element a lane, without it.
template <typename T>
__device__ __forceinline__ Sum32 wave_rest(const T* row, int64_t lo, int64_t hi, int64_t V, const LaneSum& a, float c) {
  const int lane = tid_x() & 63;
  const float m = wave_max(a.m), ref = ref_of(m);
  // (NaNs are assumed absent from the arithmetic here: what is compared may not decide where is read, so a lane is
  // named in any case)
  const int top = __builtin_ctzll(__ballot(a.m == m) | 1ull << 63);
  float r = lane == top ? 0.0f : a.s * exp2_hw((a.m - ref) * c);
  int at = 0;
  for (int64_t b = lo + (lane >> 3) * kVUnit; b < hi; b += 8 * kVUnit) {
    const int64_t v = b + (((tid_x() & ~63) + top) * 8 + (lane & 7));
    const float x = v < V ? load1(row + v) : ninf();
    at += x == m ? 1 : 0;
    r += x == m ? 0.0f : exp2_hw((x - ref) * c);
  }
  return Sum32{m, wave_sum32(r) + (wave_sum32((float)at) - 1.0f)};
}

__device__ __forceinline__ Sum64 wave_merge(Sum64 a, double c) {
  const float m = wave_max(a.m);
  return Sum64{m, wave_sum64(a.s * exp2_64(((double)a.m - (double)ref_of(m)) * c))};
}
// the first of the largest
__device__ __forceinline__ Best wave_merge(Best a) {
  const float m = wave_max(a.v);
  return Best{m, wave_min_u(a.v == m ? a.at : kNone)};
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

// ------------------------------------------------------------------ workspace

constexpr int kP1 = 2;  // 64-bit words of a chunk's partials in step 1: (m, rest) of target and of draft
constexpr int kP2 = 3;  // in step 2 (and of verify_rows): (m_t, m_d), s_t, s_d
constexpr int kSt = 3;  // merged sums for the draw: (m_t, m_d), s_t, s_d

struct Ws {
  int* first;      // [S] the first rejected position, or INT_MAX
  bool direct;     // verify_rows: positions P = L + 1 and part2, state [P][S]; else P = L
  int* count1;     // [P][S] arrivals of step 1, `apart1` ints apart
  int* count2;     // [S], `apart` ints apart
  int* count3;     // [S], likewise
  int apart, apart1;
  int* best;       // [P][S] greedy: the target's token
  float* logp;     // [P][S] log p of the drafted token
  uint64_t *part1, *part2, *part3, *state;
  int K1, K2;
  int64_t chunk1, chunk2;
  int64_t n_zero;  // ints from count1 on that start at 0
  size_t bytes;
};

// Chunks of a row: `least` (a power of two) units of kVUnit elements each, or 2, 4 .. times as many, as few as keep
// `rows` rows within `wanted` workgroups, and at most `most` (with `fit` but for rows of more than kVMaxChunks such
// chunks).
void chunking(int64_t rows, int64_t V, int64_t wanted, int64_t least, int64_t most, bool fit, int64_t& chunk, int& K) {
  const int64_t units = (V + kVUnit - 1) / kVUnit;
  int64_t per = least;
  while (per < most && rows * ((units + per - 1) / per) > wanted) per *= 2;
  while (fit && (units + per - 1) / per > kVMaxChunks) per *= 2;
  chunk = per * kVUnit;
  K = (int)((units + per - 1) / per);
}

// Whether verify_rows takes the first two steps' place: while the fp64 masses of all rows (about 1.6e12 a
// second at best) cost less than the second step's launch and way through memory.  Sequences of 4 drafts,
// V = 151936, two launches against three: 16 and 21 us for 1, 24 and 31 for 4, 31 and 34 for 8, 45 and 44
// for 16; without draft logits 17 and 19 for 4, 22 and 21 for 8, 34 and 26 for 16.  Without drafts (one row:
// 14 and 12) the second step is the only one.
bool direct_rows(int64_t S, int64_t L, int64_t V) { return L > 0 && S * (L + 1) * V <= (1 << 23); }

Ws verify_ws(void* base, int64_t S, int64_t L, int64_t V) {
  Ws w{};
  w.direct = direct_rows(S, L, V);
  const int64_t P = w.direct ? L + 1 : L;
  // step 1: at most 16384 elements (a longer chunk delays the decision that spares later positions, and its fp32
  // sums would be less good than kBorder asks for), and whole rounds of what verify_accept holds (up to 4 units:
  // with fewer, S L rows would be 1024 chunks or less of 2 units or less, and S (L + 1) V below 2^23: direct);
  // steps 2 and 3: what a thread holds at once
  chunking(S * P, V, 1024, w.direct ? 1 : 4, 8, w.direct, w.chunk1, w.K1);
  chunking(S, V, 1280, 1, 4, true, w.chunk2, w.K2);
  size_t off = 0;
  char* p = static_cast<char*>(base);
  auto take = [&](size_t bytes) {
    char* q = p ? p + off : nullptr;
    off += (bytes + 255) & ~(size_t)255;
    return q;
  };
  w.first = reinterpret_cast<int*>(take((size_t)S * 4));
  // (a line each for a few sequences, whose workgroups all count at once: 19.6 against 17.2 us for
  // the sums of 32 x 151936)
  w.apart = S <= 1024 ? 32 : 1;
  w.apart1 = S * P <= 1024 ? 32 : 1;
  w.n_zero = S * P * w.apart1 + 2 * S * w.apart;
  w.count1 = reinterpret_cast<int*>(take((size_t)w.n_zero * 4));
  w.count2 = w.count1 ? w.count1 + S * P * w.apart1 : nullptr;
  w.count3 = w.count1 ? w.count2 + S * w.apart : nullptr;
  w.best = reinterpret_cast<int*>(take((size_t)S * P * 4));
  w.logp = reinterpret_cast<float*>(take((size_t)S * P * 4));
  w.part1 = reinterpret_cast<uint64_t*>(w.direct ? nullptr : take((size_t)S * P * w.K1 * kP1 * 8));
  w.part2 = reinterpret_cast<uint64_t*>(take((size_t)(w.direct ? S * P * w.K1 : S * w.K2) * kP2 * 8));
  w.part3 = reinterpret_cast<uint64_t*>(take((size_t)S * w.K2 * 8));
  w.state = reinterpret_cast<uint64_t*>(take((size_t)(w.direct ? S * P : S) * kSt * 8));
  w.bytes = off;
  return w;
}

struct Args {
  VerifyArgs a;
  Ws w;
  bool look;  // step 1: whether to look for rejections in front (not when all workgroups run at once)
};

__global__ __launch_bounds__(kVThreads) void verify_init_kernel(int* __restrict__ first, int S, int* __restrict__ zero,
                                                                int64_t n_zero) {
  const int64_t i = (int64_t)bid_x() * kVThreads + tid_x();
  if (i < S) first[i] = 0x7fffffff;
  if (i < n_zero) zero[i] = 0;
}

// A sequence's place in the arrays; ok: its rows lie inside them.
struct Seq {
  int64_t first;  // its first draft
  int n;
  bool ok;
};
__device__ __forceinline__ Seq seq_of(const VerifyArgs& a, int i) {
  const int64_t s = a.start[i], e = a.start[i + 1];
  Seq q;
  q.ok = s >= 0 && e >= s && e <= a.N && e - s <= a.L;
  q.first = q.ok ? s : 0;
  q.n = q.ok ? (int)(e - s) : 0;
  return q;
}

// ------------------------------------------------------------------ step 1: accept

// The fp64 sum of a whole row against its maximum, by the workgroup (valid in every thread).
template <typename T>
__device__ double row_sum64(const T* row, int64_t V, float m, double c, double* red) {
  const double ref = (double)ref_of(m);
  double s = 0.0;
  for_groups<2>(row, 0, V, V, [&](int64_t, const float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) s += exp2_64(((double)x[k] - ref) * c);
  });
  s = wave_sum64(s);
  __syncthreads();
  if ((tid_x() & 63) == 0) red[tid_x() >> 6] = s;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kVWaves; ++w) t += red[w];
  return t;
}

// H: groups of 8 that a thread holds (a chunk is one or more rounds of them).
// Bound by reading the logits where there are many: 180 us for 1.04 GB of fp32 at 96 sequences of up to 7 drafts,
// V = 262144 (5.8 TB/s); by the way through memory where there are few: 19 us for 32 x 151936.
template <typename T, int H>
__global__ __launch_bounds__(kVThreads) void verify_accept_kernel(Args g) {
  const VerifyArgs& a = g.a;
  const Ws& w = g.w;
  __shared__ uint64_t red[2][kVWaves];
  __shared__ double red64[kVWaves];
  __shared__ float sh_m[2];
  __shared__ double sh_s[2];
  __shared__ int sh_flag;
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6;
  const int K = w.K1;
  const int c = (int)(large_bid() % (unsigned)K);
  const unsigned slot = large_bid() / (unsigned)K;  // position-major: all first positions, then all second ones, ...
  const int i = (int)(slot % (unsigned)a.S), j = (int)(slot / (unsigned)a.S);
  const Seq q = seq_of(a, i);
  if (j >= q.n) return;
  // a rejection before this position: nothing here is asked for (one load per
  // workgroup, so that all its threads go the same way)
  if (g.look && j > 0) {
    if (tid == 0) sh_flag = __hip_atomic_load(w.first + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < j;
    __syncthreads();
    if (sh_flag) return;
  }
  const Temp t = temp_of(a.temperature, i);
  const T* zr = static_cast<const T*>(a.target) + (q.first + i + j) * a.ldt;
  const bool has_d = a.draft != nullptr && !t.greedy;
  const T* ur = has_d ? static_cast<const T*>(a.draft) + (q.first + j) * a.ldd : nullptr;
  const int64_t lo = c * w.chunk1, hi = lo + w.chunk1 < a.V ? lo + w.chunk1 : a.V;
  // what the decision needs is requested ahead of it: the token with the row, its logits behind the row's loads
  const int64_t x = a.tokens[q.first + j];
  const bool x_ok = x >= 0 && x < a.V;
  const float r32 = a.u_accept[q.first + j];
  float zx = ninf(), ux = ninf();

  if (t.greedy) {
    Best b{ninf(), kNone};
    for_groups<H>(zr, lo, hi, a.V, [&](int64_t v, const float (&e)[8]) { add8(b, v, e); });
    b = wave_merge(b);
    if (lane == 0) red[0][wave] = pack(b.v, b.at);
  } else {
    LaneSum lt{ninf(), 0.0f}, ld{ninf(), 0.0f};
    for (int64_t b = lo; b < hi; b += kVUnit * H) {
      Group<T> gz[H], gu[H];
      hold<T, H>(zr, b, a.V, gz);
      if (has_d) hold<T, H>(ur, b, a.V, gu);
      float e[8];
#pragma unroll
      for (int k = 0; k < H; ++k) {
        held(zr, b + k * kVUnit + tid * 8, a.V, gz[k], e);
        add8(lt, e, t.c);
      }
      if (has_d) {
#pragma unroll
        for (int k = 0; k < H; ++k) {
          held(ur, b + k * kVUnit + tid * 8, a.V, gu[k], e);
          add8(ld, e, t.c);
        }
      }
    }
    if (x_ok) zx = load1(zr + x);
    if (x_ok && has_d) ux = load1(ur + x);
    const Sum32 st = wave_rest(zr, lo, hi, a.V, lt, t.c);
    Sum32 sd{ninf(), 0.0f};
    if (has_d) sd = wave_rest(ur, lo, hi, a.V, ld, t.c);
    if (lane == 0) {
      red[0][wave] = pack(st.m, __float_as_uint(st.rest));
      red[1][wave] = pack(sd.m, __float_as_uint(sd.rest));
    }
  }
  __syncthreads();
  uint64_t* part = w.part1 + ((int64_t)slot * K + c) * kP1;
  if (tid == 0) {
    if (t.greedy) {
      Best b{ninf(), kNone};
#pragma unroll
      for (int k = 0; k < kVWaves; ++k) {  // waves hold ascending runs only inside a pass: compare places too
        const float v = lo_of(red[0][k]);
        const unsigned at = hi_of(red[0][k]);
        if (v > b.v || (v == b.v && at < b.at)) b = Best{v, at};
      }
      publish(part, pack(b.v, b.at));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float m = ninf();
#pragma unroll
        for (int k = 0; k < kVWaves; ++k) m = fmaxf(m, lo_of(red[h][k]));
        // the rest of one wave at the maximum, and the whole sums of the others
        float rest = 0.0f;
        bool first = true;
#pragma unroll
        for (int k = 0; k < kVWaves; ++k) {
          const float mk = lo_of(red[h][k]), rk = __uint_as_float(hi_of(red[h][k]));
          const bool at = first && mk == m;
          rest += at ? rk : (1.0f + rk) * exp2_hw((mk - ref_of(m)) * t.c);
          first = first && !at;
        }
        if (h == 0 || has_d) publish(part + h, pack(m, __float_as_uint(rest)));
      }
    }
    sh_flag = count_last(w.count1 + (int64_t)slot * w.apart1, K);
  }
  __syncthreads();
  if (!sh_flag) return;

  // the position's last workgroup: merge the chunks and decide
  const uint64_t* parts = w.part1 + (int64_t)slot * K * kP1;
  if (t.greedy) {
    if (wave == 0) {
      Best b{ninf(), kNone};
      for (int k = lane; k < K; k += 64) {
        const uint64_t v = fetch(parts + k * kP1);
        if (lo_of(v) > b.v || (lo_of(v) == b.v && hi_of(v) < b.at)) b = Best{lo_of(v), hi_of(v)};
      }
      b = wave_merge(b);
      if (lane == 0) {
        // a row with no mass has no largest logit: nothing is accepted, no token drawn
        const int at = b.v == ninf() ? -1 : (int)b.at;
        w.best[slot] = at;
        w.logp[slot] = 0.0f;
        if (!x_ok || x != at) __hip_atomic_fetch_min(w.first + i, j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    return;
  }
  if (wave == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !has_d) break;
      Sum64 s{ninf(), 0.0};
      for (int k = lane; k < K; k += 64) {
        const uint64_t v = fetch(parts + k * kP1 + h);
        const float mn = fmaxf(s.m, lo_of(v)), ref = ref_of(mn);
        s.s = s.s * exp2_64(((double)s.m - ref) * t.c64) +
              (1.0 + (double)__uint_as_float(hi_of(v))) * exp2_64(((double)lo_of(v) - ref) * t.c64);
        s.m = mn;
      }
      s = wave_merge(s, t.c64);
      if (lane == 0) {
        sh_m[h] = s.m;
        sh_s[h] = s.s;
      }
    }
  }
  __syncthreads();
  const double r = (double)r32;
  const double ez = exp2_64(((double)zx - (double)ref_of(sh_m[0])) * t.c64);
  const double eu = has_d ? exp2_64(((double)ux - (double)ref_of(sh_m[1])) * t.c64) : 1.0;
  double St = sh_s[0], Sd = has_d ? sh_s[1] : 1.0;
  // r q < p with p = ez / St and q = eu / Sd (q = 1 without draft logits), multiplied out;
  // a row without mass has p = 0 or q = 0
  double left = r * eu * St, right = ez * Sd;
  bool pz = ez > 0.0 && St > 0.0, qz = eu > 0.0 && Sd > 0.0;
  if (pz && qz && __builtin_fabs(left - right) <= (double)kBorder * right) {
    St = row_sum64(zr, a.V, sh_m[0], t.c64, red64);
    if (has_d) Sd = row_sum64(ur, a.V, sh_m[1], t.c64, red64);
    left = r * eu * St;
    right = ez * Sd;
  }
  if (tid == 0) {
    const bool accept = pz && (!qz || left < right);
    w.logp[slot] = pz ? (float)(((double)zx - (double)sh_m[0]) * t.inv - log_64(St)) : ninf();
    if (!accept) __hip_atomic_fetch_min(w.first + i, j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// ------------------------------------------------------------------ steps 1 and 2 in one

// A thread's fp64 sum over its H groups of a round, against its own maximum (no thread waits for
// another's loads).  out_at: an element left out, or -1.
template <int H, typename T>
__device__ __forceinline__ void add_round(const T* row, int64_t b, int64_t V, Group<T> (&g)[H], double c, int64_t out_at,
                                          const double (&tab)[kExpTable], Sum64& a) {
  float top = a.m, x[8];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    held(row, b + h * kVUnit + tid_x() * 8, V, g[h], x);
    top = fmaxf(top, max8(x));
  }
  const double ref = (double)ref_of(top);
  double s = a.s * exp2_64(((double)a.m - ref) * c, tab);
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int64_t v = b + h * kVUnit + tid_x() * 8;
    launder(g[h]);
    held(row, v, V, g[h], x);
    leave_out(v, out_at, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) s += exp2_64(((double)x[k] - ref) * c, tab);
    asm volatile("" : "+v"(s));  // (now: what a sum waits for is not kept for several groups)
    __builtin_amdgcn_sched_barrier(0);  // (a group at a time: registers)
  }
  a.m = top;
  a.s = s;
}

// Steps 1 and 2 of few rows: fp64 sums of every position's rows and of the row behind the last draft.  Bound by
// latency: 9.4 us for 5 rows of 151936 in chunks of 2048 (two launches in its place 20 us).
template <typename T, int H>
__global__ __launch_bounds__(kVThreads) void verify_rows_kernel(Args g) {
  const VerifyArgs& a = g.a;
  const Ws& w = g.w;
  __shared__ uint64_t red[kVWaves];
  __shared__ Sum64 red64[2][kVWaves];
  __shared__ double tab[kExpTable];
  __shared__ int sh_flag;
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6;
  const int K = w.K1;
  const int c = (int)(bid_x() % (unsigned)K);
  const unsigned slot = bid_x() / (unsigned)K;
  const int i = (int)(slot % (unsigned)a.S), j = (int)(slot / (unsigned)a.S);
  const Seq q = seq_of(a, i);
  if (j > q.n || !q.ok) return;
  const Temp t = temp_of(a.temperature, i);
  const bool drafted = j < q.n;  // else the row behind the last draft, which only the draw asks for
  const T* zr = static_cast<const T*>(a.target) + (q.first + i + j) * a.ldt;
  const bool has_d = drafted && a.draft != nullptr && !t.greedy;
  const T* ur = has_d ? static_cast<const T*>(a.draft) + (q.first + j) * a.ldd : nullptr;
  const int64_t lo = c * w.chunk1, hi = lo + w.chunk1 < a.V ? lo + w.chunk1 : a.V;
  // what the decision needs is requested ahead of it: the token with the row, its logits behind the row's loads
  const int64_t x = drafted ? a.tokens[q.first + j] : -1;
  const bool x_ok = x >= 0 && x < a.V;
  const double r = drafted ? (double)a.u_accept[q.first + j] : 0.0;
  float zx = ninf(), ux = ninf();
  uint64_t* part = w.part2 + ((int64_t)slot * K + c) * kP2;

  if (t.greedy) {
    Best b{ninf(), kNone};
    for_groups<H>(zr, lo, hi, a.V, [&](int64_t v, const float (&e)[8]) { add8(b, v, e); });
    b = wave_merge(b);
    if (lane == 0) red[wave] = pack(b.v, b.at);
    __syncthreads();
    if (tid == 0) {
      b = Best{ninf(), kNone};
#pragma unroll
      for (int k = 0; k < kVWaves; ++k) {  // waves hold ascending runs only inside a pass: compare places too
        const float v = lo_of(red[k]);
        const unsigned at = hi_of(red[k]);
        if (v > b.v || (v == b.v && at < b.at)) b = Best{v, at};
      }
      publish(part, pack(b.v, b.at));
    }
  } else {
    // (a draft without a distribution is on its own in the sums: it is left out of the draw)
    const int64_t out_at = drafted && !a.draft ? x : -1;
    exp_table(tab);
    __syncthreads();
    Sum64 st{ninf(), 0.0}, sd{ninf(), 0.0};
    for (int64_t b = lo; b < hi; b += kVUnit * H) {
      Group<T> gz[H], gu[H];
      hold<T, H>(zr, b, a.V, gz);
      if (has_d) hold<T, H>(ur, b, a.V, gu);
      add_round<H>(zr, b, a.V, gz, t.c64, out_at, tab, st);
      if (has_d) add_round<H>(ur, b, a.V, gu, t.c64, -1, tab, sd);
    }
    if (x_ok) zx = load1(zr + x);
    if (x_ok && has_d) ux = load1(ur + x);
    st = wave_merge(st, t.c64);
    if (has_d) sd = wave_merge(sd, t.c64);
    if (lane == 0) {
      red64[0][wave] = st;
      red64[1][wave] = sd;
    }
    __syncthreads();
    if (tid == 0) {
      float m[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h && !has_d) break;
        m[h] = red64[h][0].m;
#pragma unroll
        for (int k = 1; k < kVWaves; ++k) m[h] = fmaxf(m[h], red64[h][k].m);
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < kVWaves; ++k)
          sum += red64[h][k].s * exp2_64(((double)red64[h][k].m - (double)ref_of(m[h])) * t.c64, tab);
        publish(part + 1 + h, sum);
      }
      publish(part, pack(m[0], has_d ? __float_as_uint(m[1]) : 0u));
    }
  }
  if (tid == 0) sh_flag = count_last(w.count1 + (int64_t)slot * w.apart1, K);
  __syncthreads();
  if (!sh_flag) return;

  // the position's last workgroup: merge the chunks and decide
  const uint64_t* parts = w.part2 + (int64_t)slot * K * kP2;
  if (t.greedy) {
    if (wave == 0) {
      Best b{ninf(), kNone};
      for (int k = lane; k < K; k += 64) {
        const uint64_t v = fetch(parts + k * kP2);
        if (lo_of(v) > b.v || (lo_of(v) == b.v && hi_of(v) < b.at)) b = Best{lo_of(v), hi_of(v)};
      }
      b = wave_merge(b);
      if (lane == 0) {
        // a row with no mass has no largest logit: nothing is accepted, no token drawn
        const int at = b.v == ninf() ? -1 : (int)b.at;
        w.best[slot] = at;
        w.logp[slot] = 0.0f;
        if (drafted && (!x_ok || x != at))
          __hip_atomic_fetch_min(w.first + i, j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    return;
  }
  if (wave < (has_d ? 2 : 1)) {  // the first wave the target's, the second the draft's
    Sum64 s{ninf(), 0.0};
    for (int k = lane; k < K; k += 64) {
      const uint64_t v = fetch(parts + k * kP2);
      const double e = fetch64(parts + k * kP2 + 1 + wave);
      const float m = wave ? __uint_as_float(hi_of(v)) : lo_of(v), mn = fmaxf(s.m, m);
      const double ref = (double)ref_of(mn);
      s.s = s.s * exp2_64(((double)s.m - ref) * t.c64, tab) + e * exp2_64(((double)m - ref) * t.c64, tab);
      s.m = mn;
    }
    s = wave_merge(s, t.c64);
    if (lane == 0) red64[wave][0] = s;
  }
  __syncthreads();
  if (tid > 0) return;
  const float mt = red64[0][0].m, md = has_d ? red64[1][0].m : ninf();
  const double ez = exp2_64(((double)zx - (double)ref_of(mt)) * t.c64, tab);
  // (the token left out of the target's sum is part of p)
  double St = red64[0][0].s, Sd = 1.0, eu = 1.0;
  if (drafted && !a.draft) St += ez;
  if (has_d) {
    Sd = red64[1][0].s;
    eu = exp2_64(((double)ux - (double)ref_of(md)) * t.c64, tab);
  }
  uint64_t* state = w.state + (int64_t)slot * kSt;
  state[0] = pack(mt, __float_as_uint(md));
  state[1] = __builtin_bit_cast(uint64_t, St);
  state[2] = __builtin_bit_cast(uint64_t, Sd);
  if (!drafted) return;
  // r q < p with p = ez / St and q = eu / Sd (q = 1 without draft logits), multiplied out;
  // a row without mass has p = 0 or q = 0
  const bool pz = ez > 0.0 && St > 0.0, qz = eu > 0.0 && Sd > 0.0;
  const bool accept = pz && (!qz || r * eu * St < ez * Sd);
  w.logp[slot] = pz ? (float)(((double)zx - (double)mt) * t.inv - log_64(St)) : ninf();
  if (!accept) __hip_atomic_fetch_min(w.first + i, j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ------------------------------------------------------------------ steps 2 and 3: the token behind the accepted ones

// The masses that the token is drawn from: max(p - q, 0) (RES), or p relative to mt.
template <typename T, bool RES>
struct Masses {
  const T *zr, *ur;  // ur: the draft's row (RES)
  int64_t V, skip;   // skip: a token left out, or -1 (not RES)
  double c, mt, md;  // references
  double it, id;     // residual: 1 / S_t, 1 / S_d
  const double (&tab)[kExpTable];

  __device__ __forceinline__ void of(int64_t v, const float (&x)[8], const float (&y)[8], double (&e)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double p = exp2_64(((double)x[k] - mt) * c, tab);
      if (RES) {
        const double d = p * it - exp2_64(((double)y[k] - md) * c, tab) * id;
        e[k] = d > 0.0 ? d : 0.0;
      } else {
        e[k] = p;
      }
    }
  }
  // of a held group (its target logits in x)
  __device__ __forceinline__ void of(int64_t v, const Group<T>& z, const Group<T>& u, float (&x)[8], double (&e)[8]) const {
    float y[8];
    held(zr, v, V, z, x);
    if (RES) held(ur, v, V, u, y);
    if (!RES) leave_out(v, skip, x);
    of(v, x, y, e);
  }
};

constexpr int kMaxHold = 4;
struct PickShared {
  double sums[kVMaxChunks];
  double wave[kMaxHold][kVWaves];
  double before;  // the sum in front of the chosen chunk
  int chunk;
  int found[kVWaves];  // token + 1 of a wave's first element above the goal, 0: none
  int last[kVWaves];   // token + 1 of its last element with mass
  float z[kVWaves];    // target logit of the former
};

// The token at w of the total, by the workgroup: the chunk whose running sum first
// exceeds w * total (sums[0..K) filled by the caller, scaled like the masses), then
// the element.  The running sums are in vocabulary order.  Should rounding leave no
// element above the goal, the last one with mass is the token; -1: no mass at all.
// z: its target logit.  (The finds are gathered by ballots: LDS atomics of 64 lanes on one
// word are taken lane by lane.)
template <int H, typename T, bool RES>
__device__ __forceinline__ int64_t pick(const Masses<T, RES>& m, PickShared& sh, int K, int64_t chunk, double w, float& z) {
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6;
  if (wave == 0) {
    // each lane a run of consecutive chunks
    const int per = (K + 63) / 64, k0 = lane * per, k1 = k0 + per < K ? k0 + per : K;
    double own = 0.0;
    for (int k = k0; k < k1; ++k) own += sh.sums[k];
    const double upto = wave_scan64(own);
    const double total = __shfl(upto, 63, 64);
    const double goal = w * total;
    double run = upto - own;
    int at = 0x7fffffff, last = -1;
    double before = 0.0;
    for (int k = k0; k < k1; ++k) {
      if (sh.sums[k] > 0.0) {
        if (at == 0x7fffffff && run + sh.sums[k] > goal) {
          at = k;
          before = run;
        }
        last = k;
      }
      run += sh.sums[k];
    }
    // the lowest lane's find; else the last chunk with mass
    const unsigned long long hit = __ballot(at != 0x7fffffff), some = __ballot(last >= 0);
    const int hl = hit ? __builtin_ctzll(hit) : 0, ll = some ? 63 - __builtin_clzll(some) : 0;
    const int at_h = __shfl(at, hl, 64), last_l = __shfl(last, ll, 64);
    const double before_h = __shfl(before, hl, 64);
    if (lane == 0) {
      sh.chunk = hit ? at_h : some ? last_l : -1;
      // (no running sum above the goal: a goal no sum of the chunk exceeds, so that its last element is taken)
      sh.before = hit ? goal - before_h : __builtin_inf();
    }
  }
  __syncthreads();
  z = 0.0f;
  if (sh.chunk < 0) return -1;
  const double goal = sh.before;
  const int64_t lo = sh.chunk * chunk, hi = lo + chunk < m.V ? lo + chunk : m.V;
  double base = 0.0;
  for (int64_t b = lo; b < hi; b += kVUnit * H) {
    // the sums of H groups, then the elements of the one that crosses the goal
    Group<T> gz[H], gu[H];
    hold<T, H>(m.zr, b, m.V, gz);
    if (RES) hold<T, H>(m.ur, b, m.V, gu);
    float x[8];
    double e[8], own[H], incl[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int64_t v = b + h * kVUnit + tid * 8;
      m.of(v, gz[h], gu[h], x, e);  // (0 behind the row's end, which is the only place a chunk ends short)
      own[h] = 0.0;
#pragma unroll
      for (int k = 0; k < 8; ++k) own[h] += e[k];
      asm volatile("" : "+v"(own[h]));
      incl[h] = wave_scan64(own[h]);
      if (lane == 63) sh.wave[h][wave] = incl[h];
      launder(gz[h]);
      if (RES) launder(gu[h]);
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
#pragma unroll 1
    for (int h = 0; h < H; ++h) {
      Group<T> z1 = gz[0], u1 = gu[0];
      double sum = own[0], upto = incl[0];
#pragma unroll
      for (int k = 1; k < H; ++k) {
        if (k == h) {
          z1 = gz[k];
          u1 = gu[k];
          sum = own[k];
          upto = incl[k];
        }
      }
      double run = base + upto - sum, all = base;
#pragma unroll
      for (int k = 0; k < kVWaves; ++k) {
        if (k < wave) run += sh.wave[h][k];
        all += sh.wave[h][k];
      }
      if (all > goal) {
        // the first element whose running sum exceeds the goal: the lowest token among the finds
        const int64_t v = b + h * kVUnit + tid * 8;
        int at = 0;
        float zx = 0.0f;
        if (run + sum > goal) {
          m.of(v, z1, u1, x, e);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            run += e[k];
            if (!at && e[k] > 0.0 && run > goal) {
              at = (int)(v + k) + 1;
              zx = x[k];
            }
          }
          at = at <= m.V ? at : 0;  // (with NaN masses)
        }
        const unsigned long long hit = __ballot(at != 0);
        if (lane == (hit ? __builtin_ctzll(hit) : 0)) {
          sh.found[wave] = at;
          sh.z[wave] = zx;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kVWaves; ++k) {
          if (sh.found[k]) {
            z = sh.z[k];
            return sh.found[k] - 1;
          }
        }
        __syncthreads();  // (sh.found may be written again)
      }
      base = all;
    }
    __syncthreads();  // (sh.wave is written again)
  }
  // the last element with mass (lanes and waves hold ascending runs inside a pass only, so the largest)
  int last = 0;
  for (int64_t b = lo; b < hi; b += kVUnit) {
    const int64_t v = b + tid * 8;
    Group<T> z1[1], u1[1];
    hold<T, 1>(m.zr, b, m.V, z1);
    if (RES) hold<T, 1>(m.ur, b, m.V, u1);
    float x[8];
    double e[8];
    m.of(v, z1[0], u1[0], x, e);
#pragma unroll
    for (int k = 0; k < 8; ++k) last = e[k] > 0.0 ? (int)(v + k) + 1 : last;
  }
  last = last <= m.V ? last : 0;  // (with NaN masses)
  last = wave_all(last, [](int p, int q) { return p > q ? p : q; });
  if (lane == 0) sh.last[wave] = last;
  __syncthreads();
  last = sh.last[0];
#pragma unroll
  for (int k = 1; k < kVWaves; ++k) last = sh.last[k] > last ? sh.last[k] : last;
  z = last > 0 ? load1(m.zr + last - 1) : 0.0f;
  return last - 1;
}

// The outputs of sequence i: the accepted tokens, the drawn one, -1 behind it.
__device__ __forceinline__ void write_out(const VerifyArgs& a, const Ws& w, int i, const Seq& q, int acc, int64_t tok,
                                          float lp) {
  for (int64_t k = tid_x(); k <= a.L; k += kVThreads) {
    const int64_t o = i * (a.L + 1) + k;
    a.out[o] = k < acc ? a.tokens[q.first + k] : k == acc ? tok : -1;
    if (a.logprobs) a.logprobs[o] = k < acc ? w.logp[k * a.S + i] : k == acc && tok >= 0 ? lp : 0.0f;
  }
  if (tid_x() == 0) a.n_accepted[i] = q.ok ? acc : -1;
}

// log p of a token from its logit and the row's sum.
__device__ __forceinline__ float logp_of(int64_t tok, float z, float m, double s, const Temp& t) {
  return tok < 0 ? 0.0f : (float)(((double)z - (double)m) * t.inv - log_64(s));
}

// max over the workgroup of two values (red: scratch, free afterwards behind the caller's next barrier)
__device__ __forceinline__ void block_max2(float& a, float& b, float (&red)[2][kVWaves]) {
  a = wave_max(a);
  b = wave_max(b);
  if ((tid_x() & 63) == 0) {
    red[0][tid_x() >> 6] = a;
    red[1][tid_x() >> 6] = b;
  }
  __syncthreads();
  a = red[0][0];
  b = red[1][0];
#pragma unroll
  for (int k = 1; k < kVWaves; ++k) {
    a = fmaxf(a, red[0][k]);
    b = fmaxf(b, red[1][k]);
  }
}

// H: groups of 8 that a thread holds (a chunk is one or more rounds of them).
// Bound by the exponentials (1.6e12 a second at best: 95 cycles of a SIMD for 64) and by the way of the chunk's sums
// through memory: 17 us for 32 x 151936, 31 us for 256 x 50001, 64 us for 96 x 262144 fp32.
template <typename T, int H>
__global__ __launch_bounds__(kVThreads) void verify_sums_kernel(Args g) {
  const VerifyArgs& a = g.a;
  const Ws& w = g.w;
  __shared__ uint64_t red[kVWaves];
  __shared__ double red64[2][kVWaves];
  __shared__ float red_m[2][kVWaves];
  __shared__ double tab[kExpTable];
  __shared__ PickShared sh;
  __shared__ int sh_flag;
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6;
  const int K = w.K2;
  const int c = (int)(large_bid() % (unsigned)K), at_i = (int)(large_bid() / (unsigned)K);
  const int i = min(at_i, (int)a.S - 1);
  const Seq q = seq_of(a, i);
  const Temp t = temp_of(a.temperature, i);
  const int acc = min(w.first[i], q.n);
  const float u = a.u_sample[i];
  if (at_i >= a.S) return;  // (behind the loads, none of which waits for it)
  if (!q.ok || (t.greedy && acc < q.n)) {
    if (c == 0) write_out(a, w, i, q, acc, q.ok ? w.best[(int64_t)acc * a.S + i] : -1, 0.0f);
    return;
  }
  const T* zr = static_cast<const T*>(a.target) + (q.first + i + acc) * a.ldt;
  const bool residual = a.draft != nullptr && acc < q.n;  // (not greedy: returned above)
  const T* ur = residual ? static_cast<const T*>(a.draft) + (q.first + acc) * a.ldd : nullptr;
  // a rejected draft without a distribution is left out of the draw
  const int64_t skip = !residual && acc < q.n ? a.tokens[q.first + acc] : -1;
  const int64_t lo = c * w.chunk2, hi = lo + w.chunk2 < a.V ? lo + w.chunk2 : a.V;
  uint64_t* part = w.part2 + ((int64_t)i * K + c) * kP2;
  if (t.greedy) {
    Best b{ninf(), kNone};
    for_groups<H>(zr, lo, hi, a.V, [&](int64_t v, const float (&x)[8]) { add8(b, v, x); });
    b = wave_merge(b);
    if (lane == 0) red[wave] = pack(b.v, b.at);
    __syncthreads();
    if (tid == 0) {
      b = Best{ninf(), kNone};
#pragma unroll
      for (int k = 0; k < kVWaves; ++k)
        if (lo_of(red[k]) > b.v || (lo_of(red[k]) == b.v && hi_of(red[k]) < b.at)) b = Best{lo_of(red[k]), hi_of(red[k])};
      publish(part, pack(b.v, b.at));
      sh_flag = count_last(w.count2 + i * w.apart, K);
    }
    __syncthreads();
    if (!sh_flag) return;
    if (wave == 0) {
      b = Best{ninf(), kNone};
      for (int k = lane; k < K; k += 64) {
        const uint64_t v = fetch(w.part2 + ((int64_t)i * K + k) * kP2);
        if (lo_of(v) > b.v || (lo_of(v) == b.v && hi_of(v) < b.at)) b = Best{lo_of(v), hi_of(v)};
      }
      b = wave_merge(b);
      if (lane == 0) sh.chunk = b.v == ninf() ? -1 : (int)b.at;  // (not sh_flag: other waves may still be reading it)
    }
    __syncthreads();
    write_out(a, w, i, q, acc, sh.chunk, 0.0f);
    return;
  }

  // fp64 sums of the chunk, each thread's against its own maximum (no thread waits for another's
  // loads); the token left out on its own
  Sum64 pt{ninf(), 0.0}, pd{ninf(), 0.0};
  exp_table(tab);
  __syncthreads();
  if (tid == 0 && skip >= lo && skip < hi) {
    pd.m = load1(zr + skip);
    pd.s = pd.m > ninf() ? 1.0 : 0.0;
  }
  for (int64_t b = lo; b < hi; b += kVUnit * H) {
    Group<T> gz[H], gu[H];
    hold<T, H>(zr, b, a.V, gz);
    if (residual) hold<T, H>(ur, b, a.V, gu);
    add_round<H>(zr, b, a.V, gz, t.c64, skip, tab, pt);
    if (residual) add_round<H>(ur, b, a.V, gu, t.c64, -1, tab, pd);
  }
  const Sum64 wt = wave_merge(pt, t.c64), wd = wave_merge(pd, t.c64);
  if (lane == 0) {
    red_m[0][wave] = wt.m;
    red_m[1][wave] = wd.m;
    red64[0][wave] = wt.s;
    red64[1][wave] = wd.s;
  }
  __syncthreads();
  if (tid == 0) {
    float mt = ninf(), md = ninf();
    double st = 0.0, sd = 0.0;
#pragma unroll
    for (int k = 0; k < kVWaves; ++k) {
      mt = fmaxf(mt, red_m[0][k]);
      md = fmaxf(md, red_m[1][k]);
    }
#pragma unroll
    for (int k = 0; k < kVWaves; ++k) {
      st += red64[0][k] * exp2_64(((double)red_m[0][k] - (double)ref_of(mt)) * t.c64, tab);
      sd += red64[1][k] * exp2_64(((double)red_m[1][k] - (double)ref_of(md)) * t.c64, tab);
    }
    publish(part, pack(mt, __float_as_uint(md)));
    publish(part + 1, st);
    publish(part + 2, sd);
    sh_flag = count_last(w.count2 + i * w.apart, K);
  }
  __syncthreads();
  if (!sh_flag) return;

  // the sequence's last workgroup: the row's sums.  A thread takes every kVThreads-th chunk.
  const uint64_t* parts = w.part2 + (int64_t)i * K * kP2;
  float m0 = ninf(), m1 = ninf();
  uint64_t pm[kVMaxChunks / kVThreads];
  double p0[kVMaxChunks / kVThreads], p1[kVMaxChunks / kVThreads];
#pragma unroll
  for (int n = 0; n < kVMaxChunks / kVThreads; ++n) {
    const int k = tid + n * kVThreads;
    if (k < K) {
      pm[n] = fetch(parts + k * kP2);
      p0[n] = fetch64(parts + k * kP2 + 1);
      p1[n] = fetch64(parts + k * kP2 + 2);
      m0 = fmaxf(m0, lo_of(pm[n]));
      m1 = fmaxf(m1, __uint_as_float(hi_of(pm[n])));
    }
  }
  block_max2(m0, m1, red_m);
  double s0 = 0.0, s1 = 0.0;
#pragma unroll
  for (int n = 0; n < kVMaxChunks / kVThreads; ++n) {
    const int k = tid + n * kVThreads;
    if (k < K) {
      const double e = p0[n] * exp2_64(((double)lo_of(pm[n]) - (double)ref_of(m0)) * t.c64);
      sh.sums[k] = e;
      s0 += e;
      s1 += p1[n] * exp2_64(((double)__uint_as_float(hi_of(pm[n])) - (double)ref_of(m1)) * t.c64);
    }
  }
  s0 = wave_sum64(s0);
  s1 = wave_sum64(s1);
  if (lane == 0) {
    red64[0][wave] = s0;
    red64[1][wave] = s1;
  }
  __syncthreads();
  s0 = red64[0][0];
  s1 = red64[1][0];
#pragma unroll
  for (int k = 1; k < kVWaves; ++k) {
    s0 += red64[0][k];
    s1 += red64[1][k];
  }
  if (residual) {
    if (tid == 0) {
      uint64_t* st_out = w.state + (int64_t)i * kSt;
      st_out[0] = pack(m0, __float_as_uint(m1));
      st_out[1] = __builtin_bit_cast(uint64_t, s0);
      st_out[2] = __builtin_bit_cast(uint64_t, s1);
    }
    return;
  }
  // p's sum is the token left out and the rest together; with no mass in the rest, that token is
  // drawn after all (p is 1 there)
  const float mn = skip >= 0 ? fmaxf(m0, m1) : m0;
  const double full = skip >= 0 ? s0 * exp2_64(((double)m0 - (double)ref_of(mn)) * t.c64) +
                                      s1 * exp2_64(((double)m1 - (double)ref_of(mn)) * t.c64)
                                : s0;
  const bool only = skip >= 0 && !(s0 > 0.0);
  if (only && tid == 0 && skip < a.V) sh.sums[skip / w.chunk2] = s1;
  const Masses<T, false> ms{zr, nullptr, a.V, only ? -1 : skip, t.c64, (double)ref_of(only ? mn : m0), 0.0, 0.0, 0.0,
                     tab};
  __syncthreads();  // (sh.sums)
  float z;
  const int64_t tok = pick<H>(ms, sh, K, w.chunk2, (double)u, z);
  write_out(a, w, i, q, acc, tok, logp_of(tok, z, mn, full, t));
}

// H: groups of 8 that a thread holds (a chunk is one or more rounds of them).
// Bound like verify_sums_kernel, on two rows, with the draw by one workgroup behind it (about 5 us of each call):
// 5.6 us for one sequence, 14.5 for 32 x 151936, 49 for 96 x 262144 fp32.
template <typename T, int H>
__global__ __launch_bounds__(kVThreads) void verify_draw_kernel(Args g, int K) {
  const VerifyArgs& a = g.a;
  const Ws& w = g.w;
  __shared__ double red64[kVWaves];
  __shared__ double tab[kExpTable];
  __shared__ PickShared sh;
  __shared__ int sh_flag;
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6;
  const int c = (int)(large_bid() % (unsigned)K), at_i = (int)(large_bid() / (unsigned)K);
  const int i = min(at_i, (int)a.S - 1);
  const Seq q = seq_of(a, i);
  const int acc = min(w.first[i], q.n);
  const bool residual = a.draft != nullptr && acc < q.n;
  const Temp t = temp_of(a.temperature, i);
  const int64_t slot = (int64_t)acc * a.S + i;
  if (at_i >= a.S) return;  // (behind the loads, none of which waits for it)
  if (!q.ok || t.greedy || !residual) {
    if (c > 0 || !w.direct) return;  // (drawn in step 2)
    if (!q.ok || t.greedy) {
      write_out(a, w, i, q, acc, q.ok ? w.best[slot] : -1, 0.0f);
      return;
    }
  }
  // sums of the rows that the token is drawn from, and of p's chunks
  const int64_t at = w.direct ? slot : i, p_chunk = w.direct ? w.chunk1 : w.chunk2;
  const int p_chunks = w.direct ? w.K1 : w.K2;
  const float u = a.u_sample[i];
  const uint64_t* state = w.state + at * kSt;
  const float mt = lo_of(state[0]), md = __uint_as_float(hi_of(state[0]));
  const double St = __builtin_bit_cast(double, state[1]), Sd = __builtin_bit_cast(double, state[2]);
  const T* zr = static_cast<const T*>(a.target) + (q.first + i + acc) * a.ldt;
  const T* ur = residual ? static_cast<const T*>(a.draft) + (q.first + acc) * a.ldd : nullptr;
  // a rejected draft without a distribution is left out of the draw
  const int64_t skip = !residual && acc < q.n ? a.tokens[q.first + acc] : -1;
  const double rt = (double)ref_of(mt), rd = (double)ref_of(md);
  exp_table(tab);
  __syncthreads();
  float z;
  if (residual) {
    const int64_t lo = c * w.chunk2, hi = lo + w.chunk2 < a.V ? lo + w.chunk2 : a.V;
    const Masses<T, true> ms{zr, ur, a.V, -1, t.c64, rt, rd, St > 0.0 ? 1.0 / St : 0.0, Sd > 0.0 ? 1.0 / Sd : 0.0, tab};
    double s = 0.0;
    for (int64_t b = lo; b < hi; b += kVUnit * H) {
      Group<T> gz[H], gu[H];
      hold<T, H>(zr, b, a.V, gz);
      hold<T, H>(ur, b, a.V, gu);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int64_t v = b + h * kVUnit + tid * 8;
        float x[8], y[8];
        double e[8];
        held(zr, v, a.V, gz[h], x);
        held(ur, v, a.V, gu[h], y);
        ms.of(v, x, y, e);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += e[k];
        asm volatile("" : "+v"(s));
        __builtin_amdgcn_sched_barrier(0);  // (a group at a time: registers)
      }
    }
    s = wave_sum64(s);
    if (lane == 0) red64[wave] = s;
    __syncthreads();
    if (tid == 0) {
      double r = 0.0;
#pragma unroll
      for (int k = 0; k < kVWaves; ++k) r += red64[k];
      publish(w.part3 + (int64_t)i * K + c, r);
      sh_flag = count_last(w.count3 + i * w.apart, K);
    }
    __syncthreads();
    if (!sh_flag) return;
    double any = 0.0;
    for (int k = tid; k < K; k += kVThreads) {
      sh.sums[k] = fetch64(w.part3 + (int64_t)i * K + k);
      any += sh.sums[k];
    }
    __syncthreads();  // (red64 is written again)
    any = wave_sum64(any);
    if (lane == 0) red64[wave] = any;
    __syncthreads();
    any = 0.0;
#pragma unroll
    for (int k = 0; k < kVWaves; ++k) any += red64[k];
    if (any > kNothing) {
      const int64_t tok = pick<H>(ms, sh, K, w.chunk2, (double)u, z);
      write_out(a, w, i, q, acc, tok, logp_of(tok, z, mt, St, t));
      return;
    }
    // nothing in p beyond q (a draft that neither row could have produced): drawn from p
  }
  for (int k = tid; k < p_chunks; k += kVThreads) {
    const uint64_t* part = w.part2 + (at * p_chunks + k) * kP2;
    sh.sums[k] = __builtin_bit_cast(double, part[1]) * exp2_64(((double)lo_of(part[0]) - rt) * t.c64, tab);
  }
  __syncthreads();
  const Masses<T, false> ms{zr, nullptr, a.V, skip, t.c64, rt, rd, 0.0, 0.0, tab};
  int64_t tok = pick<H>(ms, sh, p_chunks, p_chunk, (double)u, z);
  if (tok < 0 && skip >= 0 && skip < a.V && load1(zr + skip) > ninf()) {
    // no mass but the token left out: drawn after all (p is 1 there)
    tok = skip;
    z = load1(zr + skip);
  }
  write_out(a, w, i, q, acc, tok, logp_of(tok, z, mt, St, t));
}

template <typename T>
hipError_t launch_verify_t(const VerifyArgs& a, hipStream_t st) {
  (void)hipGetLastError();
  Args g{a, verify_ws(a.workspace, a.S, a.L, a.V), false};
  const Ws& w = g.w;
  // (2048 workgroups run at once: none of them could spare another anything)
  g.look = a.S * a.L * w.K1 > 2048;
  const int64_t n = w.n_zero > a.S ? w.n_zero : a.S;
  hipLaunchKernelGGL(verify_init_kernel, dim3((unsigned)((n + kVThreads - 1) / kVThreads)), dim3(kVThreads), 0, st,
                     w.first, (int)a.S, w.count1, w.n_zero);
  if (hipError_t e = hipGetLastError()) return e;
  // (verify_rows: at most 2^23 workgroups, as direct_rows says)
  const int64_t n_rows = a.S * (w.direct ? a.L + 1 : a.L) * w.K1;
  const dim3 block(kVThreads), draws = large_grid(a.S * w.K2);
  const int64_t held = w.chunk2 / kVUnit;
  if (w.direct) {
    if (w.chunk1 == kVUnit) hipLaunchKernelGGL((verify_rows_kernel<T, 1>), dim3((unsigned)n_rows), block, 0, st, g);
    else hipLaunchKernelGGL((verify_rows_kernel<T, 2>), dim3((unsigned)n_rows), block, 0, st, g);
  } else {
    if (a.L > 0) {
      // groups held at once, two rows of them: 2 of 2-byte logits (4: 23.7 against 21.4 us at 256 x
      // 50001, the registers halve the workgroups at once), 4 of fp32 (2: 191 against 183 us at 96 x 262144)
      constexpr int kHold = sizeof(T) == 4 ? 4 : 2;
      hipLaunchKernelGGL((verify_accept_kernel<T, kHold>), large_grid(n_rows), block, 0, st, g);
      if (hipError_t e = hipGetLastError()) return e;
    }
    // (fp32: a chunk of 4 in two rounds of 2; 4 held took 75 us where 2 take 58, 96 x 262144)
    if (held == 1) hipLaunchKernelGGL((verify_sums_kernel<T, 1>), draws, block, 0, st, g);
    else if (held == 2 || sizeof(T) == 4) hipLaunchKernelGGL((verify_sums_kernel<T, 2>), draws, block, 0, st, g);
    else hipLaunchKernelGGL((verify_sums_kernel<T, sizeof(T) == 4 ? 2 : 4>), draws, block, 0, st, g);
    if (a.L == 0 || !a.draft) return hipGetLastError();
  }
  if (hipError_t e = hipGetLastError()) return e;
  // (without draft logits every draw is from p, by one workgroup)
  const int K = a.draft ? w.K2 : 1;
  const dim3 all = large_grid(a.S * K);
  if (held == 1) hipLaunchKernelGGL((verify_draw_kernel<T, 1>), all, block, 0, st, g, K);
  else hipLaunchKernelGGL((verify_draw_kernel<T, 2>), all, block, 0, st, g, K);
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int64_t S, int64_t L, int64_t V) { return verify_ws(nullptr, S, L, V).bytes; }

hipError_t launch_verify(const VerifyArgs& a, Dt dt, hipStream_t st) {
  switch (dt) {
    case Dt::BF16: return launch_verify_t<uint16_t>(a, st);
    case Dt::F16: return launch_verify_t<_Float16>(a, st);
    default: return launch_verify_t<float>(a, st);
  }
}

}  // namespace lx
