// Low-rank adapters of many requests at once beside a shared projection, and
// their gradients.
//
// Rows start[i] .. start[i + 1] - 1 of x (T, H) are request i, which uses adapter
// a = adapter[i]: a scale s_a and the first rank[a] of the r ranks of A_a (r, H) and
// B_a (N, r), all bf16.  Forward, with base the shared projection's output:
//
//   u = s_a x A_a^T  (T, r)         y = base + u B_a^T  (T, N)
//
// and backward from dy (T, N):
//
//   v = s_a dy B_a (T, r)    dx = base + v A_a    dA_a = v^T x    dB_a = dy^T u
//
// the last two summed over all rows that use the adapter.  The products over H and
// over N are long and thin: what bounds each is reading x and dy, and reading base
// and writing y.  So each is one pass over those, with the r-sized side kept on chip:
//
//   down   P = X M^T over a long axis (u from x and A; v from dy and B^T)
//   up     Y = base + P M^T (y from u and B; dx from v and A^T)
//   grad   W^T X over the rows (dA from v and x; dB from u and dy)
//
// Precision.  u and v are sums of bf16 products in fp32 and stay fp32: where they
// enter a matrix-core product they are cut into three bf16 terms (hi + mid + lo, 24
// bits together), so the products are exact and the results as good as fp32
// arithmetic (two terms would leave 2^-17).  The extra MFMAs are on the r-sized side.
//
// MFMA layout used throughout (v_mfma_f32_16x16x32_bf16): lane l supplies row (or
// column) l % 16 and k = 8 (l / 16) .. + 7 of the operands; result register i of lane
// l is row 4 (l / 16) + i, column l % 16.
#include "common.hpp"
#include "lora.hpp"

namespace lx {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kLThreads = 256;
constexpr int kTileRows = 32;    // rows of a tile of the matrix-core kernels
constexpr int kDownK = 128;      // k that a wave of the down kernel takes at once
constexpr int kMaxSplits = 16;

__device__ __forceinline__ f32x4_t mfma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}
__device__ __forceinline__ u32x4_t load16(const uint16_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }

// ------------------------------------------------------------------ requests

// The last request that starts at or before `row`, by the whole wave (64 probes a step); -1: none.
__device__ __forceinline__ int find_request(const int64_t* start, int R, int64_t row) {
  const int lane = tid_x() & 63;
  int lo = 0, n = R;
  while (true) {
    const int step = (n + 63) / 64;
    const int at = lane * step;
    const unsigned long long b = __ballot(at < n && start[lo + at] <= row);
    if (!b) return -1;  // (only in the first step: later ones begin at a start found to be <= row)
    const int j = 63 - __builtin_clzll(b);
    lo += j * step;
    if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
    n = min(step, n - j * step);
  }
}

// Rows of request i within [r0, r1), and its adapter: id in [0, n), kNoAdapter or kBadAdapter.
constexpr int kNoAdapter = -1, kBadAdapter = -2;
struct Part {
  int64_t lo, hi;
  int adapter;
};
__device__ __forceinline__ Part part_of(const LoraSet& s, int i, int64_t r0, int64_t r1) {
  Part p;
  const int64_t a = s.start[i], b = s.start[i + 1];
  p.lo = a > r0 ? a : r0;
  p.hi = b < r1 ? b : r1;
  const int64_t id = s.adapter[i];
  p.adapter = id < 0 ? kNoAdapter : id >= s.n ? kBadAdapter : (int)id;
  return p;
}
__device__ __forceinline__ int rank_of(const LoraSet& s, int a) {
  if (!s.rank) return (int)s.r;
  const int64_t k = s.rank[a];
  return k < 0 ? 0 : k > s.r ? (int)s.r : (int)k;
}

// Elements k0 .. k0 + 7 with those at `end` and behind replaced by 0 (what lies there is not looked at).
__device__ __forceinline__ u32x4_t keep_below(u32x4_t w, int k0, int end) {
  unsigned v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = end - k0 - 2 * i;
    v[i] = left >= 2 ? v[i] : left == 1 ? v[i] & 0xffffu : 0u;
  }
  return (u32x4_t){v[0], v[1], v[2], v[3]};
}
// ... and those in front of `begin`.
__device__ __forceinline__ u32x4_t keep_from(u32x4_t w, int k0, int begin) {
  unsigned v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int skip = begin - k0 - 2 * i;
    v[i] = skip <= 0 ? v[i] : skip == 1 ? v[i] & 0xffff0000u : 0u;
  }
  return (u32x4_t){v[0], v[1], v[2], v[3]};
}

// Term s (0: hi, 1: mid, 2: lo) of fp32 values cut into three bf16 terms.  A value that
// is not finite is all in hi.
__device__ __forceinline__ float term(float v, int s) {
  const float hi = __uint_as_float(pack_bf16x2(v, 0.0f) << 16);
  if (s == 0) return hi;
  if ((__float_as_uint(hi) & 0x7f800000u) == 0x7f800000u) return 0.0f;
  const float rest = v - hi;
  const float mid = __uint_as_float(pack_bf16x2(rest, 0.0f) << 16);
  return s == 1 ? mid : rest - mid;
}
__device__ __forceinline__ u32x4_t terms8(const float (&v)[8], int s) {
  return (u32x4_t){pack_bf16x2(term(v[0], s), term(v[1], s)), pack_bf16x2(term(v[2], s), term(v[3], s)),
                   pack_bf16x2(term(v[4], s), term(v[5], s)), pack_bf16x2(term(v[6], s), term(v[7], s))};
}

// s_a times the sum of the down kernel's split partials, ranks k0 .. k0 + 7 of row t (0 from `rank` on).
__device__ __forceinline__ void load_low(const float* P, int splits, int64_t plane, int64_t t, int r, int k0, int rank,
                                         float scale, float (&v)[8]) {
  f32x4_t a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(P + s * plane + t * r + k0);
    a += p[0];
    b += p[1];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = k0 + k < rank ? scale * a[k] : 0.0f;
    v[4 + k] = k0 + 4 + k < rank ? scale * b[k] : 0.0f;
  }
}

// ------------------------------------------------------------------ down: P = X M^T

struct DownArgs {
  LoraSet s;
  const uint16_t* X;  // (T, K)
  int64_t ldx;
  const uint16_t* M;  // (n, r, K)
  int64_t K;
  float* P;  // [splits][T][r]
  int splits;
  int64_t kslice;  // k of a split, a multiple of kDownK
};

// Long requests: a workgroup per (tile of 32 rows, split of K); its four waves take the
// 128-k chunks of the split in turn and add up in LDS.  In a chunk a lane holds 32
// consecutive k (64 bytes) of its row, so that four MFMAs use whole lines: their k's are
// permuted alike in both operands.  RB: blocks of 16 ranks.
template <int RB>
__global__ __launch_bounds__(kLThreads) void lora_down_tile_kernel(DownArgs g) {
  __shared__ float red[3][2 * RB * 4][64];
  const LoraSet& s = g.s;
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6;
  const int split = (int)(bid_x() % (unsigned)g.splits);
  const int64_t r0 = (int64_t)(bid_x() / (unsigned)g.splits) * kTileRows;
  const int64_t r1 = r0 + kTileRows < s.T ? r0 + kTileRows : s.T;
  const int64_t kb = split * g.kslice, ke = kb + g.kslice < g.K ? kb + g.kslice : g.K;
  const int c16 = lane & 15, q = lane >> 4;
  float* P = g.P + split * s.T * s.r;
  const uint16_t* xrow[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = r0 + 16 * h + c16;
    xrow[h] = g.X + (row < s.T ? row : s.T - 1) * g.ldx;
  }
  for (int i = max(find_request(s.start, (int)s.R, r0), 0); i < s.R && s.start[i] < r1; ++i) {
    const Part p = part_of(s, i, r0, r1);
    if (p.hi <= p.lo || p.adapter < 0) continue;
    const uint16_t* mrow[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int rho = 16 * b + c16;
      mrow[b] = g.M + ((int64_t)p.adapter * s.r + (rho < s.r ? rho : (int)s.r - 1)) * g.K;
    }
    f32x4_t acc[2][RB];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[h][b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = kb + wave * kDownK; k0 < ke; k0 += 4 * kDownK) {
      const int64_t k = k0 + 32 * q;
      const u32x4_t zero = {0u, 0u, 0u, 0u};
      u32x4_t xv[2][4], mv[RB][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = k + 8 * j < ke;
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[h][j] = in ? load16(xrow[h] + k + 8 * j) : zero;
#pragma unroll
        for (int b = 0; b < RB; ++b) mv[b][j] = in ? load16(mrow[b] + k + 8 * j) : zero;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[h][b] = mfma(xv[h][j], mv[b][j], acc[h][b]);
    }
    __syncthreads();  // (the previous request's sums have been read)
    if (wave > 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) red[wave - 1][(h * RB + b) * 4 + e][lane] = acc[h][b][e];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int f = (h * RB + b) * 4 + e;
            const float v = acc[h][b][e] + red[0][f][lane] + red[1][f][lane] + red[2][f][lane];
            const int64_t t = r0 + 16 * h + 4 * q + e;
            const int rho = 16 * b + c16;
            if (t >= p.lo && t < p.hi && rho < s.r) P[t * s.r + rho] = v;
          }
    }
  }
}

// Requests of a few rows: a wave per (row, 4 ranks, split of K).
constexpr int kRowRanks = 4;
__global__ __launch_bounds__(kLThreads) void lora_down_row_kernel(DownArgs g) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63, wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6);
  const int quads = (int)(s.r / kRowRanks);
  const int64_t unit = (int64_t)bid_x() * 4 + wave;
  const int64_t t = unit / (quads * g.splits);
  if (t >= s.T) return;
  const int in_row = (int)(unit - t * (quads * g.splits));
  const int split = in_row / quads, rho = in_row % quads * kRowRanks;
  const int i = find_request(s.start, (int)s.R, t);
  if (i < 0) return;
  const Part p = part_of(s, i, t, t + 1);
  if (p.hi <= p.lo || p.adapter < 0 || rho >= rank_of(s, p.adapter)) return;
  const int64_t kb = split * g.kslice, ke = kb + g.kslice < g.K ? kb + g.kslice : g.K;
  const uint16_t* x = g.X + t * g.ldx;
  const uint16_t* m = g.M + ((int64_t)p.adapter * s.r + rho) * g.K;
  float acc[kRowRanks] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int64_t k = kb + lane * 8; k < ke; k += 512) {
    float xv[8], mv[8];
    load8(x + k, xv);
#pragma unroll
    for (int j = 0; j < kRowRanks; ++j) {
      load8(m + j * g.K + k, mv);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[j] = __builtin_fmaf(xv[e], mv[e], acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kRowRanks; ++j) acc[j] = wave_sum(acc[j]);
  if (lane == 0)
    *reinterpret_cast<f32x4_t*>(g.P + ((int64_t)split * s.T + t) * s.r + rho) = (f32x4_t){acc[0], acc[1], acc[2], acc[3]};
}

// ------------------------------------------------------------------ up: Y = base + P M^T

struct UpArgs {
  LoraSet s;
  const float* P;  // [splits][T][r]
  int splits;
  const uint16_t* M;  // (n, C, r)
  int64_t C;
  bool m_clean;  // M is 0 beyond an adapter's rank (else what lies there is not used)
  const void* base;
  int64_t ldb;
  void* y;
  int64_t ldy;
  int steps;  // tile kernel: 64-column steps of a wave
};

// Four consecutive values of a row, read as fp32 or bf16, written likewise.
__device__ __forceinline__ f32x4_t load4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
__device__ __forceinline__ f32x4_t load4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return (f32x4_t){__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                   __uint_as_float(w.y & 0xffff0000u)};
}
__device__ __forceinline__ void store4(float* p, const f32x4_t& v) { *reinterpret_cast<f32x4_t*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, const f32x4_t& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void nan4(float* p) { *reinterpret_cast<uint4*>(p) = make_uint4(kQNaN32, kQNaN32, kQNaN32, kQNaN32); }
__device__ __forceinline__ void nan4(uint16_t* p) { *reinterpret_cast<uint2*>(p) = make_uint2(kQNaN16 * 0x10001u, kQNaN16 * 0x10001u); }

// Long requests: a wave per (tile of 32 rows, steps x 64 columns).  K is the ranks three
// times over (hi, mid, lo terms of P), in chunks of 8: chunk c is term c / (r / 8) of
// ranks 8 (c mod r / 8) .. + 7, so r = 16 takes two MFMAs and not three half-empty ones.
// The tile's P terms stay in registers; M's rows are read once per tile.  Column block b
// of a step holds columns 4 (l % 16) + b, so that a lane ends with four consecutive
// columns: whole 256-byte (fp32) or 128-byte (bf16) pieces of 4 rows per access.
// NM: MFMAs of a product, ceil(3 r / 32).
template <int NM, typename YT, typename BT, bool BASE>
__global__ __launch_bounds__(kLThreads) void lora_up_tile_kernel(UpArgs g) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63, wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6);
  const int r = (int)s.r, r8 = r / 8;
  const int64_t per = (int64_t)4 * 64 * g.steps;
  const unsigned nch = (unsigned)((g.C + per - 1) / per);
  const int64_t n0 = (int64_t)(bid_x() % nch) * per + wave * 64 * g.steps;
  const int64_t n1 = n0 + 64 * g.steps < g.C ? n0 + 64 * g.steps : g.C;
  const int64_t r0 = (int64_t)(bid_x() / nch) * kTileRows;
  const int64_t r1 = r0 + kTileRows < s.T ? r0 + kTileRows : s.T;
  const int c16 = lane & 15, q = lane >> 4;
  int ck[NM];  // first rank of this lane's chunk
#pragma unroll
  for (int m = 0; m < NM; ++m) ck[m] = (4 * m + q) % r8 * 8;
  YT* Y = static_cast<YT*>(g.y);
  const BT* base = static_cast<const BT*>(g.base);
  for (int i = max(find_request(s.start, (int)s.R, r0), 0); i < s.R && s.start[i] < r1; ++i) {
    const Part p = part_of(s, i, r0, r1);
    if (p.hi <= p.lo) continue;
    const bool some = p.adapter >= 0;
    const int rank = some ? rank_of(s, p.adapter) : 0;
    u32x4_t u[2][NM];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t t = r0 + 16 * h + c16;
      const bool in = some && t >= p.lo && t < p.hi;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        u[h][m] = (u32x4_t){0u, 0u, 0u, 0u};
        const int tm = (4 * m + q) / r8;
        if (in && tm < 3) {
          float v[8];
          load_low(g.P, g.splits, s.T * s.r, t, r, ck[m], rank, s.scale[p.adapter], v);
          u[h][m] = terms8(v, tm);
        }
      }
    }
    const uint16_t* M = g.M + (some ? (int64_t)p.adapter * g.C * r : 0);
    const bool mask = !g.m_clean && rank < r;
    for (int64_t n = n0; n < n1; n += 64) {
      const int64_t col = n + 4 * c16;
      f32x4_t acc[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[h][b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
      if (rank > 0) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint16_t* row = M + (col + b < g.C ? col + b : g.C - 1) * r;
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            u32x4_t w = load16(row + ck[m]);
            if (mask) w = keep_below(w, ck[m], rank);
#pragma unroll
            for (int h = 0; h < 2; ++h) acc[h][b] = mfma(u[h][m], w, acc[h][b]);
          }
        }
      }
      if (col < g.C) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int64_t t = r0 + 16 * h + 4 * q + e;
            if (t >= p.lo && t < p.hi) {
              if (p.adapter == kBadAdapter) {
                nan4(Y + t * g.ldy + col);
              } else {
                f32x4_t v = {acc[h][0][e], acc[h][1][e], acc[h][2][e], acc[h][3][e]};
                if (BASE) v += load4(base + t * g.ldb + col);
                store4(Y + t * g.ldy + col, v);
              }
            }
          }
      }
    }
  }
}

// Requests of a few rows: a workgroup per (row, 256 columns).  G lanes share a column
// (G the power of two from r / 8 on), each with 8 ranks; in step j of G the wave takes 64 / G columns
// and lane j of each group keeps the sum, so a wave ends with 64 consecutive columns.
template <int G, typename YT, typename BT, bool BASE>
__global__ __launch_bounds__(kLThreads) void lora_up_row_kernel(UpArgs g) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63, wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6);
  const unsigned nch = (unsigned)((g.C + 255) / 256);
  const int64_t t = bid_x() / nch;
  const int64_t n0 = (int64_t)(bid_x() % nch) * 256 + wave * 64;
  if (n0 >= g.C) return;
  const int i = find_request(s.start, (int)s.R, t);
  if (i < 0) return;
  const Part p = part_of(s, i, t, t + 1);
  if (p.hi <= p.lo) return;
  const int j0 = lane & (G - 1), cl = lane / G;
  const int64_t mine = n0 + j0 * (64 / G) + cl;  // this lane's column in the end
  YT* y = static_cast<YT*>(g.y) + t * g.ldy;
  if (p.adapter == kBadAdapter) {
    if (mine < g.C) store_bits1(y + mine, kQNaN32);
    return;
  }
  float out = 0.0f;
  if (BASE && mine < g.C) out = load1(static_cast<const BT*>(g.base) + t * g.ldb + mine);
  const int rank = p.adapter >= 0 ? rank_of(s, p.adapter) : 0;
  if (rank > 0) {
    const int r = (int)s.r, k0 = j0 * 8;
    const bool live = k0 < rank;
    float u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = 0.0f;
    if (live) load_low(g.P, g.splits, s.T * s.r, t, r, k0, rank, s.scale[p.adapter], u);
    const uint16_t* M = g.M + (int64_t)p.adapter * g.C * r + (live ? k0 : 0);
    const bool mask = !g.m_clean && live && k0 + 8 > rank;
    float sums[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int64_t n = n0 + j * (64 / G) + cl;
      u32x4_t w = load16(M + (n < g.C ? n : g.C - 1) * r);
      if (mask) w = keep_below(w, k0, rank);
      const unsigned wv[4] = {w.x, w.y, w.z, w.w};
      float a = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a = __builtin_fmaf(u[2 * e], __uint_as_float(wv[e] << 16), a);
        a = __builtin_fmaf(u[2 * e + 1], __uint_as_float(wv[e] & 0xffff0000u), a);
      }
      sums[j] = live ? a : 0.0f;
    }
    float add = 0.0f;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float a = sums[j];
#pragma unroll
      for (int off = G / 2; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);
      if (j == j0) add = a;
    }
    out += add;
  }
  if (mine < g.C) store1(y + mine, out);
}

// ------------------------------------------------------------------ transposed adapters, terms of u and v

// (n, R0, C0) bf16 -> (n, C0, R0), 8 x 8 blocks a thread, with 0 where the rank axis (rows of
// the input if RANK_ROWS, else its columns) is at the adapter's rank or beyond.
template <bool RANK_ROWS>
__device__ __forceinline__ void transpose_block(const LoraSet& s, const uint16_t* in, uint16_t* out, int64_t R0,
                                                int64_t C0, int64_t at) {
  const int64_t cb = C0 / 8, rb = R0 / 8;
  const int64_t a = at / (cb * rb), in_a = at - a * cb * rb;
  // neighbouring threads along the long axis
  const int64_t b8 = RANK_ROWS ? in_a / cb : in_a % rb, c8 = RANK_ROWS ? in_a % cb : in_a / rb;
  const int rank = rank_of(s, (int)a);
  const int64_t r0 = b8 * 8, c0 = c8 * 8;
  u32x4_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] = load16(in + (a * R0 + r0 + j) * C0 + c0);
    if (RANK_ROWS) {
      if (r0 + j >= rank) w[j] = (u32x4_t){0u, 0u, 0u, 0u};
    } else {
      w[j] = keep_below(w[j], (int)c0, rank);
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    unsigned o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned lo = w[2 * j][c / 2], hi = w[2 * j + 1][c / 2];
      o[j] = c & 1 ? (lo >> 16) | (hi & 0xffff0000u) : (lo & 0xffffu) | (hi << 16);
    }
    *reinterpret_cast<u32x4_t*>(out + (a * C0 + c0 + c) * R0 + r0) = (u32x4_t){o[0], o[1], o[2], o[3]};
  }
}

__global__ __launch_bounds__(kLThreads) void lora_transpose_kernel(LoraSet s, uint16_t* At, uint16_t* Bt) {
  const int64_t na = At ? s.n * (s.r / 8) * (s.H / 8) : 0, nb = Bt ? s.n * (s.r / 8) * (s.N / 8) : 0;
  const int64_t at = (int64_t)bid_x() * kLThreads + tid_x();
  if (at < na) transpose_block<true>(s, s.A, At, s.r, s.H, at);
  else if (at - na < nb) transpose_block<false>(s, s.B, Bt, s.N, s.r, at - na);
}

// The three terms of s_a P along the rows: W[term][rank][Tp], 0 for rows without an adapter,
// ranks beyond the adapter's and rows behind T.  A thread takes 8 rows of one rank.
struct TermArgs {
  LoraSet s;
  const float* P;
  int splits;
  uint16_t* W;
  int64_t Tp;
};
__global__ __launch_bounds__(kLThreads) void lora_terms_kernel(TermArgs g0, TermArgs g1) {
  const int64_t half = nblocks_x() / 2;
  const bool second = bid_x() >= half;
  const TermArgs& g = second ? g1 : g0;
  const LoraSet& s = g.s;
  const int r = (int)s.r;
  const int64_t unit = ((int64_t)bid_x() - (second ? half : 0)) * kLThreads + tid_x();
  const int64_t t0 = unit / r * 8;
  const int rho = (int)(unit % r);
  // (every lane of the wave takes part in the search: one request lookup per wave, then steps along it)
  const int64_t wave_t0 = (unit & ~(int64_t)63) / r * 8;
  int i = find_request(s.start, (int)s.R, wave_t0 < s.T ? wave_t0 : s.T - 1);
  if (t0 >= g.Tp || !g.W) return;
  if (i < 0) i = 0;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t t = t0 + k;
    v[k] = 0.0f;
    if (t >= s.T) continue;
    while (i + 1 < s.R && s.start[i + 1] <= t) ++i;
    const Part p = part_of(s, i, t, t + 1);
    if (p.hi <= p.lo || p.adapter < 0 || rho >= rank_of(s, p.adapter)) continue;
    float a = 0.0f;
    for (int sp = 0; sp < g.splits; ++sp) a += g.P[((int64_t)sp * s.T + t) * r + rho];
    v[k] = a * s.scale[p.adapter];
  }
#pragma unroll
  for (int tm = 0; tm < 3; ++tm)
    *reinterpret_cast<u32x4_t*>(g.W + ((int64_t)tm * r + rho) * g.Tp + t0) = terms8(v, tm);
}

// ------------------------------------------------------------------ grad: W^T X over the rows of an adapter

constexpr int kGradCols = 128;  // columns of X of a workgroup (32 a wave)
constexpr int kGradRows = 64;   // rows staged at once
constexpr int kGradStride = 288;  // bytes of a staged row: 256 and 32, so that the rows of a transposing read fall on different banks

struct GradArgs {
  LoraSet s;
  const uint16_t* X;  // (T, C)
  int64_t ldx, C;
  const uint16_t* W;  // [3][r][Tp] terms
  int64_t Tp;
  float* out;  // (n, r, C) or, transposed, (n, C, r); [splits] of them when splits > 1
  int splits;
  int64_t tslice;  // rows of a split
};

// The next kGradRows rows of adapter `a` within [t0, t1): requests in order.
struct RowWalk {
  int i;
  int64_t lo, hi, at;  // rows of the current request, and the first of the next stage
};
__device__ __forceinline__ bool next_request(const LoraSet& s, int a, int64_t t0, int64_t t1, RowWalk& w) {
  const int lane = tid_x() & 63;
  for (int i = w.i + 1; i < s.R; i += 64) {
    const int mine = i + lane;
    bool hit = false;
    if (mine < s.R) {
      const Part p = part_of(s, mine, t0, t1);
      hit = p.adapter == a && p.hi > p.lo;
    }
    const unsigned long long b = __ballot(hit);
    if (b) {
      w.i = __builtin_amdgcn_readfirstlane(i + __builtin_ctzll(b));
      const Part p = part_of(s, w.i, t0, t1);
      w.lo = p.lo;
      w.hi = p.hi;
      w.at = p.lo & ~(int64_t)7;
      return true;
    }
  }
  return false;
}

// A workgroup per (adapter, 128 columns, split of the rows).  64 rows of X at a time go
// through LDS, double buffered, and are read back transposed (ds_read_b64_tr_b16: 16 lanes
// supply a 4 x 16 block of rows k, and lane i receives its column i), which gives the MFMA
// its 8 consecutive rows; the W terms lie along the rows already.  RB: blocks of 16 ranks.
// TRANS: the result is (C, r), so the columns of X are the rows of the product.
template <int RB, bool TRANS>
__device__ __forceinline__ void grad_tile(const GradArgs& g, unsigned block, uint8_t* lds) {
  const LoraSet& s = g.s;
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6;
  const int c16 = lane & 15, q = lane >> 4;
  const unsigned cols = (unsigned)((g.C + kGradCols - 1) / kGradCols);
  const int64_t c0 = (int64_t)(block % cols) * kGradCols;
  const int split = (int)(block / cols % (unsigned)g.splits);
  const int a = (int)(block / cols / (unsigned)g.splits);
  const int64_t t0 = split * g.tslice, t1 = t0 + g.tslice < s.T ? t0 + g.tslice : s.T;
  f32x4_t acc[2][RB];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[h][b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // staging: thread tid moves 16 bytes of rows tid / 16 + 16 j
  const int srow = tid >> 4, scol = (tid & 15) * 8;
  const bool scol_in = c0 + scol < g.C;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  auto fetch = [&](const RowWalk& w, u32x4_t (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = w.at + srow + 16 * j;
      v[j] = scol_in && t >= w.lo && t < w.hi ? load16(g.X + t * g.ldx + c0 + scol) : zero;
    }
  };
  RowWalk w{-1, 0, 0, 0};
  bool more = next_request(s, a, t0, t1, w);
  u32x4_t held[4];
  if (more) fetch(w, held);
  int stage = 0;
  while (more) {
    uint8_t* T = lds + stage * (kGradRows * kGradStride);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<u32x4_t*>(T + (srow + 16 * j) * kGradStride + scol * 2) = held[j];
    const RowWalk now = w;
    w.at += kGradRows;
    if (w.at >= w.hi) more = next_request(s, a, t0, t1, w);
    if (more) fetch(w, held);
    __syncthreads();
    const bool edge = now.at < now.lo || now.at + kGradRows > now.hi;
#pragma unroll
    for (int ks = 0; ks < kGradRows; ks += 32) {
      if (now.at + ks >= now.hi) break;
      // this lane's 8 rows of W: now.at + ks + 8 q (the rows of W reach Tp, kGradRows beyond T)
      const int64_t t = now.at + ks + 8 * q;
      u32x4_t x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
        const uint8_t* p = T + (ks + 8 * q + (c16 >> 2)) * kGradStride + (wave * 32 + h * 16 + 4 * (c16 & 3)) * 2;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * kGradStride));
        const s16x4_t v8[2] = {lo, hi};
        x[h] = __builtin_bit_cast(u32x4_t, v8);
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int rho = 16 * b + c16;
        const uint16_t* wr = g.W + (int64_t)(rho < s.r ? rho : (int)s.r - 1) * g.Tp + t;
#pragma unroll
        for (int tm = 0; tm < 3; ++tm) {
          u32x4_t wv = load16(wr + (int64_t)tm * s.r * g.Tp);
          if (edge) {
            // rows of other requests may hold anything: neither side may keep them
            wv = keep_below(wv, (int)(t - now.at), (int)(now.hi - now.at < kGradRows ? now.hi - now.at : kGradRows));
            wv = keep_from(wv, (int)(t - now.at), (int)(now.lo - now.at > 0 ? now.lo - now.at : 0));
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) acc[h][b] = TRANS ? mfma(x[h], wv, acc[h][b]) : mfma(wv, x[h], acc[h][b]);
        }
      }
    }
    stage ^= 1;
    // (the stage written next was last read before the barrier above)
  }
  const int rank = rank_of(s, a);
  float* out = g.out + (int64_t)split * s.n * s.r * g.C + (int64_t)a * s.r * g.C;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int along = c16, down = 4 * q + e;
        const int64_t col = c0 + wave * 32 + h * 16 + (TRANS ? down : along);
        const int rho = 16 * b + (TRANS ? along : down);
        if (col < g.C && rho < s.r) {
          const float v = rho < rank ? acc[h][b][e] : 0.0f;
          out[TRANS ? col * s.r + rho : (int64_t)rho * g.C + col] = v;
        }
      }
}

template <int RB>
__global__ __launch_bounds__(kLThreads) void lora_grad_kernel(GradArgs ga, unsigned blocks_a, GradArgs gb) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kGradRows * kGradStride];
  if (bid_x() < blocks_a) grad_tile<RB, false>(ga, bid_x(), lds);
  else grad_tile<RB, true>(gb, bid_x() - blocks_a, lds);
}

// out = the sum of the splits' partials, in split order.
struct SplitSum {
  const float* P;
  float* out;
  int64_t plane;  // a multiple of 4
  int splits;
};
__global__ __launch_bounds__(kLThreads) void lora_split_sum_kernel(SplitSum a, SplitSum b) {
  const int64_t na = a.splits > 1 ? a.plane / 4 : 0, nb = b.splits > 1 ? b.plane / 4 : 0;
  for (int64_t i = (int64_t)bid_x() * kLThreads + tid_x(); i < na + nb; i += (int64_t)nblocks_x() * kLThreads) {
    const SplitSum& s = i < na ? a : b;
    const int64_t at = i < na ? i : i - na;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < s.splits; ++k) v += reinterpret_cast<const f32x4_t*>(s.P + k * s.plane)[at];
    reinterpret_cast<f32x4_t*>(s.out)[at] = v;
  }
}

// Gradients of adapters that no row uses.
__global__ __launch_bounds__(kLThreads) void lora_zero_kernel(float* a, int64_t na, float* b, int64_t nb) {
  for (int64_t i = (int64_t)bid_x() * kLThreads + tid_x(); i < na + nb; i += (int64_t)nblocks_x() * kLThreads) {
    if (i < na) a[i] = 0.0f;
    else b[i - na] = 0.0f;
  }
}

// ------------------------------------------------------------------ launches

// Mean rows of a request below which the kernels take single rows, and not tiles of 32.
constexpr int kShortRows = 8;
bool short_requests(int64_t T, int64_t R, int64_t widest) {
  return T < kShortRows * R && T * ((widest + 255) / 256) < (1 << 30);
}

// Splits of a down product's K: 512 workgroups at least where K allows ranges of 512.
void down_split(int64_t T, bool rows, int64_t K, int64_t r, int& splits, int64_t& kslice) {
  const int64_t units = rows ? (T * (r / kRowRanks) + 3) / 4 : (T + kTileRows - 1) / kTileRows;
  int64_t want = (512 + units - 1) / units, most = K / 512;
  if (want > most) want = most;
  if (want > kMaxSplits) want = kMaxSplits;
  if (want < 1) want = 1;
  const int64_t per = (K + want - 1) / want;
  kslice = (per + kDownK - 1) / kDownK * kDownK;
  splits = (int)((K + kslice - 1) / kslice);
}

hipError_t launch_down(const LoraSet& s, const uint16_t* X, int64_t ldx, const uint16_t* M, int64_t K, float* P,
                       bool rows, int& splits, hipStream_t st) {
  DownArgs g{s, X, ldx, M, K, P, 1, 0};
  down_split(s.T, rows, K, s.r, g.splits, g.kslice);
  splits = g.splits;
  if (rows) {
    const int64_t units = s.T * (s.r / kRowRanks) * g.splits;
    hipLaunchKernelGGL(lora_down_row_kernel, dim3((unsigned)((units + 3) / 4)), dim3(kLThreads), 0, st, g);
  } else {
    const dim3 grid((unsigned)((s.T + kTileRows - 1) / kTileRows * g.splits));
    if (s.r <= 16) hipLaunchKernelGGL(lora_down_tile_kernel<1>, grid, dim3(kLThreads), 0, st, g);
    else if (s.r <= 32) hipLaunchKernelGGL(lora_down_tile_kernel<2>, grid, dim3(kLThreads), 0, st, g);
    else if (s.r <= 64) hipLaunchKernelGGL(lora_down_tile_kernel<4>, grid, dim3(kLThreads), 0, st, g);
    else hipLaunchKernelGGL(lora_down_tile_kernel<8>, grid, dim3(kLThreads), 0, st, g);
  }
  return hipGetLastError();
}

template <typename YT, typename BT, bool BASE>
hipError_t launch_up_t(UpArgs g, bool rows, hipStream_t st) {
  const int64_t r = g.s.r;
  if (rows) {
    const dim3 grid((unsigned)(g.s.T * ((g.C + 255) / 256)));
    if (r <= 8) hipLaunchKernelGGL((lora_up_row_kernel<1, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else if (r <= 16) hipLaunchKernelGGL((lora_up_row_kernel<2, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else if (r <= 32) hipLaunchKernelGGL((lora_up_row_kernel<4, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else if (r <= 64) hipLaunchKernelGGL((lora_up_row_kernel<8, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else hipLaunchKernelGGL((lora_up_row_kernel<16, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    return hipGetLastError();
  }
  // a wave's columns: 4 steps of 64, fewer where that leaves less than 1024 workgroups
  const int64_t tiles = (g.s.T + kTileRows - 1) / kTileRows;
  g.steps = 4;
  while (g.steps > 1 && tiles * ((g.C + 256 * g.steps - 1) / (256 * g.steps)) < 1024) g.steps /= 2;
  const int64_t per = 256 * g.steps;
  const dim3 grid((unsigned)(tiles * ((g.C + per - 1) / per)));
  if (r <= 8) hipLaunchKernelGGL((lora_up_tile_kernel<1, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else if (r <= 16) hipLaunchKernelGGL((lora_up_tile_kernel<2, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else if (r <= 32) hipLaunchKernelGGL((lora_up_tile_kernel<3, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else if (r <= 64) hipLaunchKernelGGL((lora_up_tile_kernel<6, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else hipLaunchKernelGGL((lora_up_tile_kernel<12, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  return hipGetLastError();
}

template <typename YT>
hipError_t launch_up_y(const UpArgs& g, Dt base_dt, bool rows, hipStream_t st) {
  if (!g.base) return launch_up_t<YT, float, false>(g, rows, st);
  return base_dt == Dt::BF16 ? launch_up_t<YT, uint16_t, true>(g, rows, st) : launch_up_t<YT, float, true>(g, rows, st);
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

// Row splits of a grad product: 512 workgroups at least where the rows allow 512 each.
void grad_split(int64_t T, int64_t n, int64_t C, int& splits, int64_t& tslice) {
  const int64_t units = n * ((C + kGradCols - 1) / kGradCols);
  int64_t want = (512 + units - 1) / units, most = T / 512;
  if (want > most) want = most;
  if (want > kMaxSplits) want = kMaxSplits;
  if (want < 1) want = 1;
  const int64_t per = (T + want - 1) / want;
  tslice = (per + 63) / 64 * 64;
  splits = (int)((T + tslice - 1) / tslice);
}

struct BackwardWs {
  float *Pu, *Pv;
  uint16_t *At, *Bt, *Wu, *Wv;
  float *partA, *partB;
  int64_t Tp;
  bool rows;
  int splits_A, splits_B;
  int64_t tslice_A, tslice_B;
  size_t bytes;
};
BackwardWs backward_ws(void* base, int64_t T, int64_t R, int64_t n, int64_t H, int64_t N, int64_t r) {
  BackwardWs w{};
  size_t off = 0;
  char* p = static_cast<char*>(base);
  auto take = [&](size_t bytes) {
    char* q = p ? p + off : nullptr;
    off += align256(bytes);
    return q;
  };
  w.rows = short_requests(T, R, H > N ? H : N);
  int su, sv;
  int64_t ks;
  down_split(T, w.rows, H, r, su, ks);
  down_split(T, w.rows, N, r, sv, ks);
  w.Tp = (T + kGradRows + 7) / 8 * 8;
  grad_split(T, n, H, w.splits_A, w.tslice_A);
  grad_split(T, n, N, w.splits_B, w.tslice_B);
  w.Pu = reinterpret_cast<float*>(take((size_t)su * T * r * 4));
  w.Pv = reinterpret_cast<float*>(take((size_t)sv * T * r * 4));
  w.At = reinterpret_cast<uint16_t*>(take((size_t)n * H * r * 2));
  w.Bt = reinterpret_cast<uint16_t*>(take((size_t)n * N * r * 2));
  w.Wu = reinterpret_cast<uint16_t*>(take((size_t)3 * r * w.Tp * 2));
  w.Wv = reinterpret_cast<uint16_t*>(take((size_t)3 * r * w.Tp * 2));
  w.partA = w.splits_A > 1 ? reinterpret_cast<float*>(take((size_t)w.splits_A * n * r * H * 4)) : nullptr;
  w.partB = w.splits_B > 1 ? reinterpret_cast<float*>(take((size_t)w.splits_B * n * r * N * 4)) : nullptr;
  w.bytes = off;
  return w;
}

}  // namespace

size_t lora_forward_workspace_bytes(int64_t T, int64_t R, int64_t H, int64_t N, int64_t r) {
  int splits;
  int64_t ks;
  down_split(T, short_requests(T, R, N), H, r, splits, ks);
  return align256((size_t)splits * T * r * 4);
}

size_t lora_backward_workspace_bytes(int64_t T, int64_t R, int64_t n, int64_t H, int64_t N, int64_t r) {
  return backward_ws(nullptr, T, R, n, H, N, r).bytes;
}

hipError_t launch_lora_forward(const LoraForwardArgs& a, hipStream_t st) {
  (void)hipGetLastError();
  const bool rows = short_requests(a.s.T, a.s.R, a.s.N);
  float* P = static_cast<float*>(a.workspace);
  int splits;
  if (hipError_t e = launch_down(a.s, a.x, a.ldx, a.s.A, a.s.H, P, rows, splits, st)) return e;
  const UpArgs g{a.s, P, splits, a.s.B, a.s.N, false, a.base, a.ldb, a.y, a.ldy, 0};
  return a.y_dt == Dt::BF16 ? launch_up_y<uint16_t>(g, a.base_dt, rows, st) : launch_up_y<float>(g, a.base_dt, rows, st);
}

hipError_t launch_lora_backward(const LoraBackwardArgs& a, hipStream_t st) {
  (void)hipGetLastError();
  const LoraSet& s = a.s;
  if (s.T == 0 || s.R == 0) {
    const int64_t na = a.gA ? s.n * s.r * s.H : 0, nb = a.gB ? s.n * s.r * s.N : 0;
    if (na + nb == 0) return hipSuccess;
    const int64_t blocks = (na + nb + kLThreads - 1) / kLThreads;
    hipLaunchKernelGGL(lora_zero_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(kLThreads), 0, st, a.gA,
                       na, a.gB, nb);
    return hipGetLastError();
  }
  const BackwardWs w = backward_ws(a.workspace, s.T, s.R, s.n, s.H, s.N, s.r);
  const bool need_v = a.gx || a.gA;
  if (need_v) {
    const int64_t blocks = s.n * (s.r / 8) * ((a.gx ? s.H / 8 : 0) + s.N / 8);
    hipLaunchKernelGGL(lora_transpose_kernel, dim3((unsigned)((blocks + kLThreads - 1) / kLThreads)), dim3(kLThreads), 0,
                       st, s, a.gx ? w.At : nullptr, w.Bt);
    if (hipError_t e = hipGetLastError()) return e;
  }
  int su = 1, sv = 1;
  if (a.gB)
    if (hipError_t e = launch_down(s, a.x, a.ldx, s.A, s.H, w.Pu, w.rows, su, st)) return e;
  if (need_v)
    if (hipError_t e = launch_down(s, a.dy, a.lddy, w.Bt, s.N, w.Pv, w.rows, sv, st)) return e;
  if (a.gx) {
    const UpArgs g{s, w.Pv, sv, w.At, s.H, true, a.base, a.ldb, a.gx, a.ldgx, 0};
    if (hipError_t e = launch_up_y<float>(g, Dt::F32, w.rows, st)) return e;
  }
  if (!a.gA && !a.gB) return hipSuccess;
  const TermArgs tu{s, w.Pu, su, a.gB ? w.Wu : nullptr, w.Tp}, tv{s, w.Pv, sv, a.gA ? w.Wv : nullptr, w.Tp};
  const int64_t half = (w.Tp / 8 * s.r + kLThreads - 1) / kLThreads;
  hipLaunchKernelGGL(lora_terms_kernel, dim3((unsigned)(2 * half)), dim3(kLThreads), 0, st, tu, tv);
  if (hipError_t e = hipGetLastError()) return e;
  const GradArgs ga{s, a.x, a.ldx, s.H, w.Wv, w.Tp, w.splits_A > 1 ? w.partA : a.gA, w.splits_A, w.tslice_A};
  const GradArgs gb{s, a.dy, a.lddy, s.N, w.Wu, w.Tp, w.splits_B > 1 ? w.partB : a.gB, w.splits_B, w.tslice_B};
  const unsigned ba = a.gA ? (unsigned)(s.n * w.splits_A * ((s.H + kGradCols - 1) / kGradCols)) : 0u;
  const unsigned bb = a.gB ? (unsigned)(s.n * w.splits_B * ((s.N + kGradCols - 1) / kGradCols)) : 0u;
  if (s.r <= 16) hipLaunchKernelGGL(lora_grad_kernel<1>, dim3(ba + bb), dim3(kLThreads), 0, st, ga, ba, gb);
  else if (s.r <= 32) hipLaunchKernelGGL(lora_grad_kernel<2>, dim3(ba + bb), dim3(kLThreads), 0, st, ga, ba, gb);
  else if (s.r <= 64) hipLaunchKernelGGL(lora_grad_kernel<4>, dim3(ba + bb), dim3(kLThreads), 0, st, ga, ba, gb);
  else hipLaunchKernelGGL(lora_grad_kernel<8>, dim3(ba + bb), dim3(kLThreads), 0, st, ga, ba, gb);
  if (hipError_t e = hipGetLastError()) return e;
  const SplitSum sa{w.partA, a.gA, s.n * s.r * s.H, a.gA ? w.splits_A : 0};
  const SplitSum sb{w.partB, a.gB, s.n * s.r * s.N, a.gB ? w.splits_B : 0};
  if (sa.splits > 1 || sb.splits > 1) {
    const int64_t quads = (sa.splits > 1 ? sa.plane / 4 : 0) + (sb.splits > 1 ? sb.plane / 4 : 0);
    const int64_t blocks = (quads + kLThreads - 1) / kLThreads;
    hipLaunchKernelGGL(lora_split_sum_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(kLThreads), 0, st, sa,
                       sb);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace lx
