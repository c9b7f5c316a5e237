// The 256 x 256 tiles of the lm_head path: their launch shape, and reductions of accumulators over columns.
#pragma once

#include "common.hpp"
#include "mm.hpp"

namespace lx {

// LDS of the main loop: 2 stages of a 64-k slice, 64 KB each.
constexpr int kLds = 2 * 65536;
// The 256 x 256 kernels (the gradient products and pass 1) run 8 waves, two per
// SIMD, each 128 x 64 of the tile (4 x 2 accumulators, 128 registers): while one
// wave of a SIMD waits for its slice data the other issues its MFMAs (6-7%
// faster than 4 waves of 128 x 128 on the same main loop); each MFMA is then
// followed by up to three of the slice's memory instructions.
constexpr int kWideThreads = 512;
constexpr int kWideMem = 3;

// Reductions over the 32 lanes of each half-wave (the 32 columns of one
// accumulator row), on the vector ALU: two quad permutations and two rotations
// inside each row of 16 lanes (DPP), then the gfx950 swap of rows 0 <-> 1 and
// 2 <-> 3.  Every lane ends with the reduction of its half; the sum's
// association order is fixed, so the half's first lane always sees the same
// value for the same data.
template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float swap16(float v, float* other) {
  const unsigned u = __float_as_uint(v);
  const auto pr = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  // the elements go through scalars: this compiler's __builtin_bit_cast of an
  // element of the returned pair reads element 0 whatever the index
  const unsigned lo = pr[0], hi = pr[1];
  *other = __uint_as_float(hi);
  return __uint_as_float(lo);
}
__device__ __forceinline__ float half_max(float v) {
  v = fmaxf(v, dpp_mov<0xB1>(v));   // quad_perm [1, 0, 3, 2]
  v = fmaxf(v, dpp_mov<0x4E>(v));   // quad_perm [2, 3, 0, 1]
  v = fmaxf(v, dpp_mov<0x124>(v));  // row_ror 4
  v = fmaxf(v, dpp_mov<0x128>(v));  // row_ror 8
  float hi;
  const float lo = swap16(v, &hi);
  return fmaxf(lo, hi);
}
__device__ __forceinline__ float half_sum(float v) {
  v += dpp_mov<0xB1>(v);
  v += dpp_mov<0x4E>(v);
  v += dpp_mov<0x124>(v);
  v += dpp_mov<0x128>(v);
  float hi;
  const float lo = swap16(v, &hi);
  return lo + hi;
}

// Row sums of a 32 x 32 accumulator block (one column per lane of each
// half-wave, v[r] the lane's value in row r of its half, r = 0..15), all rows at
// once: at the level of lane bit b every lane keeps half of its rows (those
// its bit b selects), sends the other half to its partner (the lane differing
// only in bit b) and adds what it receives.  Bit 4: the row-pair swap, two rows
// an instruction; bit 3: row_ror 8; bits 0 and 1: quad permutations; then one
// row per lane is left, and bit 2 (a swizzle) completes its sum.  Lane L of a
// half ends with the total of row xsum_row(L) = b1 + 2 b0 + 4 b3 + 8 b4 (lanes
// L and L ^ 4 the same row).  The association order is fixed.
__device__ __forceinline__ int xsum_row(int lane) {
  return ((lane >> 1) & 1) | ((lane & 1) << 1) | (((lane >> 3) & 1) << 2) | (((lane >> 4) & 1) << 3);
}
template <int CTRL>
__device__ __forceinline__ float xsum_level(float lo, float hi, bool bit) {
  const float keep = bit ? hi : lo, send = bit ? lo : hi;
  return keep + dpp_mov<CTRL>(send);
}
__device__ __forceinline__ float xsum16(const float (&v)[16], int lane) {
  float w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // rows 0 and 2 of v[k] stay, rows 1 and 3 receive v[k + 8] of rows 0 and 2,
    // and the reverse in the second result: a lane of row 0 gets v[k] of both
    // partners, a lane of row 1 v[k + 8] of both
    const auto pr = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 8]), false, false);
    const unsigned a = pr[0], b = pr[1];  // copied out: see swap16
    w[k] = __uint_as_float(a) + __uint_as_float(b);
  }
  const bool b3 = (lane >> 3) & 1, b0 = lane & 1, b1 = (lane >> 1) & 1;
  float u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) u[k] = xsum_level<0x128>(w[k], w[k + 4], b3);  // row_ror 8
  float t[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) t[k] = xsum_level<0xB1>(u[k], u[k + 2], b0);    // quad_perm [1, 0, 3, 2]
  const float x = xsum_level<0x4E>(t[0], t[1], b1);                           // quad_perm [2, 3, 0, 1]
  // lane ^ 4 within each 32 lanes: and-mask 31, or-mask 0, xor-mask 4
  return x + __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, x), 0x101F));
}

}  // namespace lx
