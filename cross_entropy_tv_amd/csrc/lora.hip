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
// Long requests go in tiles of 32 rows on the matrix cores; single rows (a token of each request) are
// vector products that read an adapter once for every row, from the L2s (single_rows decides).
//
// Precision.  u and v are sums of bf16 products in fp32 and stay fp32: where they
// enter a matrix-core product they are cut into three bf16 terms (24 bits together),
// so the products are exact and the results as good as fp32 arithmetic (two terms
// would leave 2^-17).  The extra MFMAs are on the r-sized side.  The cut leaves no
// term 0 (terms8), so a product with an infinity is the infinity that it should be.
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
constexpr int kDownK = 128;      // k of a slice of the down kernel
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

// Eight fp32 values, each cut into N bf16 terms that add up to it.  A term is the largest bf16 number strictly below
// (in magnitude) what the terms in front of it leave, the last one is the rest: 8 bits at a time, a value's 24 bits
// fit three terms, a fourth splits the third.  So the terms of a value other than 0 are all of its sign and none of
// them is 0 (from 2^-87 on; below, the last ones run out of exponents), which keeps its product with an infinity that
// infinity (rounded terms of either sign, or 0, would make it NaN), and none exceeds a finite value.  A value that is
// not finite is all of its terms.
__device__ __forceinline__ unsigned bf16_below(unsigned f32bits) {
  return f32bits & 0x7fffffffu ? (f32bits - 1u) & 0xffff0000u : f32bits;
}
template <int N>
__device__ __forceinline__ void terms8(const float (&v)[8], u32x4_t (&t)[N]) {
  unsigned w[N][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned a[2][N];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const unsigned x = __float_as_uint(v[2 * i + e]);
      const bool finite = (x & 0x7f800000u) != 0x7f800000u;
      const unsigned whole = (x & 0x7fffffffu) > 0x7f800000u ? x | 0x400000u : x;  // (a NaN in its upper half, too)
      unsigned rest = x;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const unsigned term = n < N - 1 ? bf16_below(rest) : rest;
        if (n < N - 1) rest = __float_as_uint(__uint_as_float(rest) - __uint_as_float(term));
        a[e][n] = finite ? term : whole;
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) w[n][i] = a[0][n] >> 16 | (a[1][n] & 0xffff0000u);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) t[n] = (u32x4_t){w[n][0], w[n][1], w[n][2], w[n][3]};
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

// ------------------------------------------------------------------ transposed adapters

// The backward's tiles take A and B the other way round: (n, R0, C0) bf16 -> (n, C0, R0), an 8 x 8
// block a thread, with 0 where the rank axis (rows of the input if RANK_ROWS, else its columns) is at
// the adapter's rank or beyond.
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

struct TransposeArgs {
  LoraSet s;
  uint16_t *At, *Bt;  // nullptr: not wanted
  unsigned blocks;    // workgroups that do this, in front of the others of the launch
};
__device__ __forceinline__ void transpose_blocks(const TransposeArgs& g, int64_t at) {
  const LoraSet& s = g.s;
  uint16_t *At = g.At, *Bt = g.Bt;
  const int64_t na = At ? s.n * (s.r / 8) * (s.H / 8) : 0, nb = Bt ? s.n * (s.r / 8) * (s.N / 8) : 0;
  if (at < na) transpose_block<true>(s, s.A, At, s.r, s.H, at);
  else if (at - na < nb) transpose_block<false>(s, s.B, Bt, s.N, s.r, at - na);
}

// ------------------------------------------------------------------ down: P = X M^T

// u or v as the other products take it, its bf16 terms cut into MFMA operands of 64
// lanes x 16 bytes (a wave's load of one is 1 KB of consecutive memory; operands loaded
// straight from row-major arrays touch 16 rows per 16 lanes and run at a quarter of that):
//   U: rows as operand rows, for the up product: [tile of 32 rows][half h][block l][j], where
//      lane (row, q) of operand (l, j) holds 8 ranks of one term (up_chunk);
//   W: rows along k, for the gradients: [tile of 32 rows][block of 16 ranks][term].
// Either may be nullptr.
struct Terms {
  uint16_t *U, *W;
};
// Operands of a tile for the up product with room for r ranks: LD blocks of ranks, TM MFMAs each.
// r = 8: the four k-groups of one MFMA are four terms; r = 16: two terms of 16 ranks an MFMA, four in two; else
// one term of 32 ranks, three MFMAs.
__host__ __device__ constexpr int up_ld(int r) { return r <= 32 ? 1 : r <= 64 ? 2 : 4; }
__host__ __device__ constexpr int up_tm(int r) { return r <= 8 ? 1 : r <= 16 ? 2 : 3; }
// blocks of 16 ranks that the down and gradient kernels take
__host__ __device__ constexpr int rank_blocks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }
// First rank (-1: none) of k-group q of block l.
__device__ __forceinline__ int up_chunk(int r, int l, int q) {
  if (r <= 8) return 0;
  if (r <= 16) return (q & 1) * 8;
  return 32 * l + 8 * q < r ? 32 * l + 8 * q : -1;
}

// vals: the fp32 values of rows t0 .. t0 + 31 (t0 a multiple of 32; rows behind T: 0), row stride vs.
template <int NT>
__device__ __forceinline__ void emit_terms(const Terms& o, const float* vals, int vs, int64_t t0, int r) {
  const int64_t tile = t0 / kTileRows;
  if (o.U) {
    const int ld = up_ld(r), tm = up_tm(r), kcs = r <= 8 ? 1 : r <= 16 ? 2 : 4 * ld;  // chunks of 8 ranks
    uint16_t* U = o.U + tile * 2 * ld * tm * 512;
    for (int i = tid_x(); i < kTileRows * kcs; i += NT) {
      const int row = i % kTileRows, kc = i / kTileRows, h = row >> 4, c16 = row & 15;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 8 * kc < r ? vals[row * vs + 8 * kc + k] : 0.0f;
      // operand and lane (k-group q) of term n of this chunk
      auto put = [&](int f, int q, const u32x4_t& w) {
        *reinterpret_cast<u32x4_t*>(U + f * 512 + (c16 + 16 * q) * 8) = w;
      };
      if (r <= 16) {
        u32x4_t t4[4];
        terms8(v, t4);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (r <= 8) put(h, n, t4[n]);
          else put(2 * h + (n >> 1), kc + 2 * (n & 1), t4[n]);
        }
      } else {
        u32x4_t t3[3];
        terms8(v, t3);
#pragma unroll
        for (int n = 0; n < 3; ++n) put((h * ld + kc / 4) * 3 + n, kc % 4, t3[n]);
      }
    }
  }
  if (o.W) {
    const int nb = rank_blocks(r);
    for (int i = tid_x(); i < nb * 64; i += NT) {
      const int lane = i & 63, b = i >> 6, rho = 16 * b + (lane & 15);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = rho < r ? vals[((lane >> 4) * 8 + k) * vs + rho] : 0.0f;
      u32x4_t t3[3];
      terms8(v, t3);
#pragma unroll
      for (int n = 0; n < 3; ++n)
        *reinterpret_cast<u32x4_t*>(o.W + ((tile * nb + b) * 3 + n) * 512 + lane * 8) = t3[n];
    }
  }
}

struct DownArgs {
  LoraSet s;
  const uint16_t* X;  // (T, K)
  int64_t ldx;
  const uint16_t* M;  // (n, r, K)
  int64_t K;
  float* P;  // [splits][T][r]
  int splits;
  int64_t kslice;  // k of a split, a multiple of kDownK
  Terms o;  // tile kernel with one split: where the result goes
};

// Long requests: a workgroup per (tile of 32 rows, split of K).  K goes in slices of 128 through
// LDS, 16-byte pieces of a row swapped by its number so that the 16 rows of an operand read fall
// on different banks.  x is on its way in registers four slices ahead and M two, and
// (up to 64 ranks) two groups of four waves take every other slice each: with one workgroup per
// compute unit, as 8192 rows make, that is what keeps enough loads in flight.  Bound by reading x and
// by the steps between barriers: 31 us at 8192 x 4096, r 64 (67 MB of x: 2.2 TB/s; about 10 us of it
// start and end, 1.3 us every two slices), 17 us at 4096 x 4096, r 16.  A group's four
// waves share out the row halves and the ranks (RB = 1: the slice's k).  With one split the
// workgroup finishes u itself (scale, rank, terms); with several it leaves its partial sums for
// lora_terms_kernel.  RB: blocks of 16 ranks.
template <int RB>
struct Down {
  static constexpr int kGroups = RB == 8 ? 1 : 2, kThreads = 256 * kGroups;
  static constexpr int kRows = kTileRows + 16 * RB;         // staged rows: x, then M
  static constexpr int kStage = kRows * kDownK * 2;          // bytes
  static constexpr int kLoads = kRows * (kDownK / 8) / 256;  // 16-byte pieces of a thread and slice
  static constexpr int kBlocks = RB == 1 ? 1 : RB / 2;       // blocks of ranks of a wave
  static constexpr int kVs = 16 * RB + 1;                    // row stride of the fp32 result
  // (the waves' sums lie in the stages' place, behind them the result)
  static constexpr int kLds = 2 * kGroups * kStage;
  static_assert(4 * kGroups * kBlocks * 4 * 64 * 4 <= kLds, "sums exceed the stages");
};

template <int RB>
__global__ __attribute__((amdgpu_flat_work_group_size(Down<RB>::kThreads, Down<RB>::kThreads), amdgpu_waves_per_eu(2)))
void lora_down_tile_kernel(DownArgs g, TransposeArgs tr) {
  using D = Down<RB>;
  if (bid_x() < tr.blocks) {
    transpose_blocks(tr, (int64_t)bid_x() * D::kThreads + tid_x());
    return;
  }
  const unsigned block = bid_x() - tr.blocks;
  __shared__ __attribute__((aligned(16))) uint8_t lds[D::kLds];
  __shared__ float vals[kTileRows * D::kVs];
  const LoraSet& s = g.s;
  const int tid = tid_x(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = wave >> 2, gw = wave & 3, gt = tid & 255;
  const int split = (int)(block % (unsigned)g.splits);
  const int64_t r0 = (int64_t)(block / (unsigned)g.splits) * kTileRows;
  const int64_t r1 = r0 + kTileRows < s.T ? r0 + kTileRows : s.T;
  const uint32_t kb = (uint32_t)(split * g.kslice), ke = (uint32_t)(kb + g.kslice < g.K ? kb + g.kslice : g.K);
  const int c16 = lane & 15, q = lane >> 4, r = (int)s.r;
  const bool whole = g.splits == 1;
  if (whole)
    for (int i = tid; i < kTileRows * D::kVs; i += D::kThreads) vals[i] = 0.0f;
  // this thread's pieces of a slice: rows gt / 16 + 16 p (first the 32 of x), piece gt % 16.  The
  // tile's rows and an adapter's M lie within 2^30 bytes: 32-bit offsets from uniform bases.
  const int prow = gt >> 4, piece = gt & 15;
  const uint16_t* X = g.X + r0 * g.ldx;
  uint32_t off[D::kLoads];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int64_t row = prow + 16 * p;
    off[p] = (uint32_t)((r0 + row < s.T ? row : s.T - 1 - r0) * g.ldx);
  }
#pragma unroll
  for (int p = 2; p < D::kLoads; ++p) {
    const int rho = prow + 16 * (p - 2);
    off[p] = (uint32_t)((rho < r ? rho : r - 1) * g.K);
  }
  uint8_t* const stage0 = lds + group * 2 * D::kStage;
  const int h = gw & 1, hb = gw >> 1;  // row half; half of the ranks (RB = 1: of the slice's k)
  // Slices of the split, and rounds of a group.  Tiles start at different rounds and go round: all
  // at the same slice they would ask the same few channels of the L2s for M at once (38 against 35 us
  // at 8192 x 4096, r 64).
  const uint32_t slices = (ke - kb + kDownK - 1) / kDownK;
  const uint32_t rounds = (slices + D::kGroups - 1) / D::kGroups;
  const uint32_t turn = (uint32_t)(r0 / kTileRows * 5 % rounds);
  for (int i = max(find_request(s.start, (int)s.R, r0), 0); i < s.R && s.start[i] < r1; ++i) {
    const Part p = part_of(s, i, r0, r1);
    if (p.hi <= p.lo || p.adapter < 0) continue;
    const uint16_t* M = g.M + (int64_t)p.adapter * r * g.K;
    const int rank = rank_of(s, p.adapter);
    const float scale = s.scale[p.adapter];
    f32x4_t acc[D::kBlocks];
#pragma unroll
    for (int b = 0; b < D::kBlocks; ++b) acc[b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    // x comes from memory and is asked for four slices ahead, M from the L2s two slices ahead
    u32x4_t xs[4][2], ms[2][D::kLoads - 2];
    // slice c of this group into registers; a piece behind the end comes from the last one in front
    // of it (no load is conditional) and is 0 in LDS
    auto slice_k = [&](uint32_t c) {  // (behind the last round: behind the end)
      const uint32_t n = c < rounds ? (c + turn < rounds ? c + turn : c + turn - rounds) : rounds;
      return kb + (n * D::kGroups + group) * kDownK + piece * 8;
    };
    auto load_x = [&](u32x4_t (&v)[2], uint32_t c) {
      const uint32_t at = min(slice_k(c), ke - 8);
#pragma unroll
      for (int n = 0; n < 2; ++n) v[n] = load16(X + (off[n] + at));
    };
    auto load_m = [&](u32x4_t (&v)[D::kLoads - 2], uint32_t c) {
      const uint32_t at = min(slice_k(c), ke - 8);
#pragma unroll
      for (int n = 0; n < D::kLoads - 2; ++n) v[n] = load16(M + (off[2 + n] + at));
    };
    auto put = [&](const u32x4_t (&vx)[2], const u32x4_t (&vm)[D::kLoads - 2], uint32_t c) {
      const bool in = slice_k(c) < ke;
      uint8_t* T = stage0 + (c & 1) * D::kStage;
#pragma unroll
      for (int n = 0; n < D::kLoads; ++n) {
        const u32x4_t z = {0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4_t*>(T + (prow + 16 * n) * (kDownK * 2) + ((piece ^ prow) << 4)) =
            in ? (n < 2 ? vx[n < 2 ? n : 0] : vm[n < 2 ? 0 : n - 2]) : z;
      }
    };
    auto multiply = [&](uint32_t c) {
      const uint8_t* T = stage0 + (c & 1) * D::kStage;
      constexpr int kSteps = kDownK / 32 / (RB == 1 ? 2 : 1);
#pragma unroll
      for (int n = 0; n < kSteps; ++n) {
        const int at = ((4 * (RB == 1 ? hb * kSteps + n : n) + q) ^ c16) << 4;
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(T + (16 * h + c16) * (kDownK * 2) + at);
#pragma unroll
        for (int b = 0; b < D::kBlocks; ++b) {
          const int row = kTileRows + 16 * (RB == 1 ? 0 : hb * D::kBlocks + b) + c16;
          acc[b] = mfma(x, *reinterpret_cast<const u32x4_t*>(T + row * (kDownK * 2) + at), acc[b]);
        }
      }
    };
    auto round = [&](int n, uint32_t c) {  // n = c % 4
      put(xs[n], ms[n & 1], c);
      load_m(ms[n & 1], c + 2);
      load_x(xs[n], c + 4);
      __syncthreads();
      multiply(c);
      // (a stage is written again only after the barrier behind its reads)
    };
    // (in the loop's order, so that its waits are the same from the first round on)
    load_x(xs[0], 0);
    load_x(xs[1], 1);
    load_m(ms[0], 0);
    load_x(xs[2], 2);
    load_m(ms[1], 1);
    load_x(xs[3], 3);
    __syncthreads();  // (the previous request's sums have been read)
    uint32_t c = 0;
    for (; c + 4 <= rounds; c += 4) {
#pragma unroll
      for (int n = 0; n < 4; ++n) round(n, c + n);
    }
#pragma unroll
    for (int n = 0; n < 3; ++n)
      if (c + n < rounds) round(n, c + n);
    __syncthreads();
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int b = 0; b < D::kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[((wave * D::kBlocks + b) * 4 + e) * 64 + lane] = acc[b][e];
    __syncthreads();
    for (int f = tid; f < kTileRows * 16 * RB; f += D::kThreads) {
      // place f: register e of lane l, block b, row half hh; summed over the waves that share it
      const int l = f & 63, e = (f >> 6) & 3, b = (f >> 8) % RB, hh = (f >> 8) / RB;
      float v = 0.0f;
#pragma unroll
      for (int n = 0; n < D::kGroups * (RB == 1 ? 2 : 1); ++n) {
        const int w = (RB == 1 ? n >> 1 : n) * 4 + 2 * (RB == 1 ? n & 1 : b / D::kBlocks) + hh;
        v += red[((w * D::kBlocks + b % D::kBlocks) * 4 + e) * 64 + l];
      }
      const int row = 16 * hh + 4 * (l >> 4) + e, rho = 16 * b + (l & 15);
      const int64_t t = r0 + row;
      if (t >= p.lo && t < p.hi && rho < r) {
        if (whole) vals[row * D::kVs + rho] = rho < rank ? scale * v : 0.0f;
        else g.P[((int64_t)split * s.T + t) * r + rho] = v;
      }
    }
  }
  if (whole) {
    __syncthreads();
    emit_terms<D::kThreads>(g.o, vals, D::kVs, r0, r);
  }
}

// Requests of a few rows.  u: a wave per (row, 4 ranks, split of K), along the rows of A.  Bound by latency:
// 4 us for 64 rows of 4096, r 16, and by the L2s (8 TB/s) for more.
constexpr int kRowRanks = 4;
__device__ __forceinline__ void down_row(const DownArgs& g, int64_t unit) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63;
  const int quads = (int)(s.r / kRowRanks);
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

// v: a wave per (row, 16 ranks, split of N), down the rows of B (M is (n, K, r) here): a lane takes
// every 64th row and holds the 16 sums of its rows.
constexpr int kRowWide = 16;
__device__ __forceinline__ void down_row_strided(const DownArgs& g, int64_t unit) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63, r = (int)s.r;
  const int wides = (r + kRowWide - 1) / kRowWide;
  const int64_t t = unit / (wides * g.splits);
  if (t >= s.T) return;
  const int in_row = (int)(unit - t * (wides * g.splits));
  const int split = in_row / wides, rho = in_row % wides * kRowWide;
  const int i = find_request(s.start, (int)s.R, t);
  if (i < 0) return;
  const Part p = part_of(s, i, t, t + 1);
  if (p.hi <= p.lo || p.adapter < 0 || rho >= rank_of(s, p.adapter)) return;
  const int64_t kb = split * g.kslice, ke = kb + g.kslice < g.K ? kb + g.kslice : g.K;
  const uint16_t* x = g.X + t * g.ldx;
  const int next = rho + 8 < r ? 8 : 0;  // (8 ranks: the second half is the first again and not stored)
  const uint16_t* m = g.M + (int64_t)p.adapter * g.K * r + rho;
  float acc[kRowWide];
#pragma unroll
  for (int j = 0; j < kRowWide; ++j) acc[j] = 0.0f;
#pragma unroll 4
  for (int64_t k = kb + lane; k < ke; k += 64) {
    const float xv = load1(x + k);
    float a[8], b[8];
    load8(m + k * r, a);
    load8(m + k * r + next, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[e] = __builtin_fmaf(xv, a[e], acc[e]);
      acc[8 + e] = __builtin_fmaf(xv, b[e], acc[8 + e]);
    }
  }
  float mine = 0.0f;  // lane j keeps sum j
#pragma unroll
  for (int j = 0; j < kRowWide; ++j) {
    const float v = wave_sum(acc[j]);
    mine = lane == j ? v : mine;
  }
  if (lane < kRowWide && rho + lane < r) g.P[((int64_t)split * s.T + t) * r + rho + lane] = mine;
}

// Both in one launch (blocks of four waves, blocks_u of them for u and blocks_v for v).
__global__ __launch_bounds__(kLThreads) void lora_down_row_kernel(DownArgs u, unsigned blocks_u, DownArgs v,
                                                                  unsigned blocks_v) {
  const int wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6);
  const unsigned block = large_bid();
  if (block < blocks_u) down_row(u, (int64_t)block * 4 + wave);
  else if (block - blocks_u < blocks_v) down_row_strided(v, (int64_t)(block - blocks_u) * 4 + wave);
}

// ------------------------------------------------------------------ up: Y = base + P M^T

struct UpArgs {
  LoraSet s;
  const float* P;  // single rows: [splits][T][r]
  int splits;
  const uint16_t* U;  // tiles: Terms::U
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

// Long requests: a wave per (tile of 32 rows, steps x 64 columns).  The tile's operands of P
// (Terms::U) stay in registers; a block of M is read once and multiplied by its terms one
// after the other.  Column block b of a step holds columns 4 (l % 16) + b, so that a lane ends
// with four consecutive columns: whole 256-byte (fp32) or 128-byte (bf16) pieces of 4 rows per
// access.  Bound by reading base and writing y: 62 to 69 us for 268 MB at 8192 x 4096 fp32, r 64 (4.1
// TB/s where a copy reaches 4.7).
template <int LD, int TM, typename YT, typename BT, bool BASE>
__global__ __attribute__((amdgpu_flat_work_group_size(kLThreads, kLThreads), amdgpu_waves_per_eu(2)))
void lora_up_tile_kernel(UpArgs g) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63, wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6);
  const int r = (int)s.r;
  const int64_t per = (int64_t)4 * 64 * g.steps;
  const unsigned nch = (unsigned)((g.C + per - 1) / per);
  const int64_t n0 = (int64_t)(bid_x() % nch) * per + wave * 64 * g.steps;
  const int64_t n1 = n0 + 64 * g.steps < g.C ? n0 + 64 * g.steps : g.C;
  const int64_t r0 = (int64_t)(bid_x() / nch) * kTileRows;
  const int64_t r1 = r0 + kTileRows < s.T ? r0 + kTileRows : s.T;
  const int c16 = lane & 15, q = lane >> 4;
  // this lane's 8 ranks of block l, and how they count against an adapter's rank; none (u is 0 there): the first 8
  // are loaded and made 0, so that no infinity among them meets the 0
  int ck[LD], first[LD];
#pragma unroll
  for (int l = 0; l < LD; ++l) {
    const int c = up_chunk(r, l, q);
    ck[l] = TM == 3 ? max(c, 0) : c;
    first[l] = TM == 3 && c < 0 ? r : c;
  }
  const bool some_none = TM == 3 && r < 32 * LD;
  // the tile's rows and an adapter's M lie within 2^30 bytes: 32-bit offsets from uniform bases
  YT* Y = static_cast<YT*>(g.y) + r0 * g.ldy;
  const BT* base = static_cast<const BT*>(g.base) + (BASE ? r0 * g.ldb : 0);
  const uint16_t* U = g.U + r0 / kTileRows * (2 * LD * TM * 512);
  const uint32_t ldy = (uint32_t)g.ldy, ldb = (uint32_t)g.ldb, C = (uint32_t)g.C;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  __shared__ u32x4_t shared[LD == 4 ? 2 * LD * TM * 64 : 1];  // beyond 64 ranks U does not fit the registers beside M
  for (int i = max(find_request(s.start, (int)s.R, r0), 0); i < s.R && s.start[i] < r1; ++i) {
    const Part p = part_of(s, i, r0, r1);
    if (p.hi <= p.lo) continue;
    const bool some = p.adapter >= 0;
    const int rank = some ? rank_of(s, p.adapter) : 0;
    const int lo = (int)(p.lo - r0), hi = (int)(p.hi - r0);
    u32x4_t u[2][LD == 4 ? 1 : LD][TM];
    if constexpr (LD == 4) {
      __syncthreads();  // (the previous request's products are done)
      for (int n = tid_x(); n < 2 * LD * TM * 64; n += kLThreads) {
        const int row = n / (LD * TM * 64) * 16 + (n & 15);
        const u32x4_t v = load16(U + n * 8);
        shared[n] = rank > 0 && row >= lo && row < hi ? v : zero;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * h + c16;
        const bool in = rank > 0 && row >= lo && row < hi;
#pragma unroll
        for (int l = 0; l < LD; ++l)
#pragma unroll
          for (int j = 0; j < TM; ++j) {
            const u32x4_t v = load16(U + (((h * LD + l) * TM + j) * 512 + lane * 8));
            u[h][l][j] = in ? v : zero;
          }
      }
    }
    auto operand = [&](int h, int l, int j) {
      if constexpr (LD == 4) return shared[((h * LD + l) * TM + j) * 64 + lane];
      else return u[h][l][j];
    };
    const uint16_t* M = g.M + (some ? (int64_t)p.adapter * g.C * r : 0);
    const bool mask = some_none || (!g.m_clean && rank < r);
    for (uint32_t n = (uint32_t)n0; n < (uint32_t)n1; n += 64) {
      const uint32_t col = n + 4 * c16;
      u32x4_t w[4][LD];
      if (rank > 0) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t row = (col + b < C ? col + b : C - 1) * (uint32_t)r;
#pragma unroll
          for (int l = 0; l < LD; ++l) w[b][l] = load16(M + (row + ck[l]));
        }
      }
      f32x4_t old[2][4];
      if (BASE) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 16 * h + 4 * q + e;
            // (a row or column of the request for those that are not written, so that no load is conditional)
            old[h][e] = load4(base + ((uint32_t)min(max(row, lo), hi - 1) * ldb + min(col, C - 4)));
          }
      }
      f32x4_t acc[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[h][b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
      if (rank > 0) {
        if (mask) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int l = 0; l < LD; ++l) w[b][l] = keep_below(w[b][l], first[l], rank);
        }
#pragma unroll
        for (int l = 0; l < LD; ++l)
#pragma unroll
          for (int j = 0; j < TM; ++j) {
            const u32x4_t u0 = operand(0, l, j), u1 = operand(1, l, j);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              acc[0][b] = mfma(u0, w[b][l], acc[0][b]);
              acc[1][b] = mfma(u1, w[b][l], acc[1][b]);
            }
          }
      }
      if (col < C) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 16 * h + 4 * q + e;
            if (row >= lo && row < hi) {
              if (p.adapter == kBadAdapter) {
                nan4(Y + (row * ldy + col));
              } else {
                f32x4_t v = {acc[h][0][e], acc[h][1][e], acc[h][2][e], acc[h][3][e]};
                if (BASE) v += old[h][e];
                store4(Y + (row * ldy + col), v);
              }
            }
          }
      }
    }
  }
}

// Requests of a few rows: a wave per (row, steps x 64 columns).  Up to 32 ranks (CH chunks of 8) a
// lane takes a whole column, 16 CH bytes of M; beyond, lanes share a column (lora_up_row_kernel).
// Bound by reading M from the L2s, once a row, beside base and y: 64 x 151936, fp32 to bf16, r 16,
// 29.5 us (369 MB, 311 of them M's).  Workgroups go column range by column range, and the rows of one range on one die (id mod
// 8), so that rows with the same adapter find its part of M in that die's L2.
struct RowPlace {
  int64_t t, n0, n1;
  Part p;
  bool ok;
};
__device__ __forceinline__ RowPlace row_place(const UpArgs& g, int columns) {
  const LoraSet& s = g.s;
  const int wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6);
  const unsigned die = large_bid() % 8u, on_die = large_bid() / 8u;
  RowPlace o{};
  o.t = on_die % (unsigned)s.T;
  const int64_t ch = (int64_t)(on_die / (unsigned)s.T) * 8 + die;
  o.n0 = (ch * 4 + wave) * columns * g.steps;
  if (o.n0 >= g.C) return o;
  o.n1 = o.n0 + columns * g.steps < g.C ? o.n0 + columns * g.steps : g.C;
  const int i = find_request(s.start, (int)s.R, o.t);
  if (i < 0) return o;
  o.p = part_of(s, i, o.t, o.t + 1);
  o.ok = o.p.hi > o.p.lo;
  return o;
}

template <int CH, typename YT, typename BT, bool BASE>
__global__ __launch_bounds__(kLThreads) void lora_up_lane_kernel(UpArgs g) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63, r = (int)s.r;
  const RowPlace o = row_place(g, 64);
  if (!o.ok) return;
  const int a = o.p.adapter, rank = a >= 0 ? rank_of(s, a) : 0;
  YT* y = static_cast<YT*>(g.y) + o.t * g.ldy;
  const BT* base = static_cast<const BT*>(g.base) + (BASE ? o.t * g.ldb : 0);
  // the row's u, the same in every lane
  float u[CH][8];
  int kc[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    kc[c] = 8 * c < r ? 8 * c : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) u[c][e] = 0.0f;
    if (8 * c < rank) load_low(g.P, g.splits, s.T * s.r, o.t, r, 8 * c, rank, s.scale[a], u[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      u[c][e] = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(u[c][e])));
  }
  const uint16_t* M = g.M + (a >= 0 ? (int64_t)a * g.C * r : 0);
  const bool mask = rank < r;
  for (int64_t n = o.n0; n < o.n1; n += 64) {
    const uint32_t col = (uint32_t)n + lane, at = min(col, (uint32_t)g.C - 1);
    float out = 0.0f;
    if (BASE) out = load1(base + at);
    if (rank > 0) {
      u32x4_t w[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) w[c] = load16(M + (at * (uint32_t)r + kc[c]));
      float sum[CH];  // (a sum of every chunk: shorter chains)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (mask) w[c] = keep_below(w[c], kc[c], rank);
        const unsigned wv[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
        sum[c] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[c] = __builtin_fmaf(u[c][2 * e], __uint_as_float(wv[e] << 16), sum[c]);
          sum[c] = __builtin_fmaf(u[c][2 * e + 1], __uint_as_float(wv[e] & 0xffff0000u), sum[c]);
        }
        if (c == 3 && r == 24) sum[c] = 0.0f;  // (the last chunk is the first again)
      }
#pragma unroll
      for (int c = 1; c < CH; ++c) sum[0] += sum[c];
      out += sum[0];
    }
    if (col < g.C) {
      if (a == kBadAdapter) store_bits1(y + col, kQNaN32);
      else store1(y + col, out);
    }
  }
}

// The same with u formed by every workgroup itself, its waves sharing out the ranks: a few rows are bound by
// the launches, and A's part is read from the L2s once for every 256 steps columns of a row.  4096 x 4096,
// r 16: 6.2 us for one row, 8 for 64 (in two launches 11 and 11).
struct RowArgs {
  const uint16_t *X, *A;
  int64_t ldx, K;
};
template <int CH, typename YT, typename BT, bool BASE>
__global__ __launch_bounds__(kLThreads) void lora_row_kernel(UpArgs g, RowArgs d) {
  __shared__ float sh[8 * CH];
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63, wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6), r = (int)s.r;
  const int64_t t = bid_x() % (unsigned)s.T;
  const int64_t wide = 64 * g.steps, n0 = ((int64_t)(bid_x() / (unsigned)s.T) * 4 + wave) * wide;
  const int64_t n1 = n0 + wide < g.C ? n0 + wide : g.C;
  const int i = find_request(s.start, (int)s.R, t);
  if (i < 0) return;
  const Part p = part_of(s, i, t, t + 1);
  if (p.hi <= p.lo) return;
  const int a = p.adapter, rank = a >= 0 ? rank_of(s, a) : 0;
  YT* y = static_cast<YT*>(g.y) + t * g.ldy;
  const BT* base = static_cast<const BT*>(g.base) + (BASE ? t * g.ldb : 0);
  const uint16_t* M = g.M + (a >= 0 ? (int64_t)a * g.C * r : 0);
  u32x4_t w[CH];
  float old = 0.0f;
  auto load = [&](int64_t n) {
    const uint32_t at = min((uint32_t)n + lane, (uint32_t)g.C - 1);
    if (BASE) old = load1(base + at);
#pragma unroll
    for (int c = 0; c < CH; ++c) w[c] = load16(M + (at * (uint32_t)r + (8 * c < r ? 8 * c : 0)));
  };
  load(n0);  // (ahead of u)
  if (rank > 0) {
    // ranks 2 CH wave .. of u
    const uint16_t *x = d.X + t * d.ldx, *m = d.A + (int64_t)a * r * d.K;
    float acc[2 * CH];
#pragma unroll
    for (int j = 0; j < 2 * CH; ++j) acc[j] = 0.0f;
#pragma unroll 2
    for (int64_t k = lane * 8; k < d.K; k += 512) {
      float xv[8], mv[8];
      load8(x + k, xv);
#pragma unroll
      for (int j = 0; j < 2 * CH; ++j) {
        const int rho = min(2 * CH * wave + j, r - 1);
        load8(m + rho * d.K + k, mv);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[j] = __builtin_fmaf(xv[e], mv[e], acc[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2 * CH; ++j) {
      const float v = wave_sum(acc[j]);
      const int rho = 2 * CH * wave + j;
      if (lane == 0) sh[rho] = rho < rank ? s.scale[a] * v : 0.0f;
    }
  }
  __syncthreads();
  float u[CH][8];
  if (rank > 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        u[c][e] = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sh[8 * c + e])));
  }
  const bool mask = rank < r;
  for (int64_t n = n0; n < n1; n += 64) {
    float out = old;
    if (rank > 0) {
      float sum[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (mask) w[c] = keep_below(w[c], 8 * c, rank);
        const unsigned wv[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
        sum[c] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[c] = __builtin_fmaf(u[c][2 * e], __uint_as_float(wv[e] << 16), sum[c]);
          sum[c] = __builtin_fmaf(u[c][2 * e + 1], __uint_as_float(wv[e] & 0xffff0000u), sum[c]);
        }
        if (8 * c >= r) sum[c] = 0.0f;  // (24 ranks: the last chunk is the first again)
      }
#pragma unroll
      for (int c = 1; c < CH; ++c) sum[0] += sum[c];
      out += sum[0];
    }
    const int64_t col = n + lane;
    if (col < g.C) {
      if (a == kBadAdapter) store_bits1(y + col, kQNaN32);
      else store1(y + col, out);
    }
    if (n + 64 < n1) load(n + 64);
  }
}

// More ranks: G lanes (8 or 16) share a column, each with 8 ranks; in step j of G the wave takes
// 64 / G columns and lane j of each group keeps the sum, so 64 consecutive columns come out at once.
template <int G, typename YT, typename BT, bool BASE>
__global__ __launch_bounds__(kLThreads) void lora_up_row_kernel(UpArgs g) {
  const LoraSet& s = g.s;
  const int lane = tid_x() & 63;
  const RowPlace o = row_place(g, 64);
  if (!o.ok) return;
  const Part& p = o.p;
  const int64_t t = o.t;
  const int j0 = lane & (G - 1), cl = lane / G;
  YT* y = static_cast<YT*>(g.y) + t * g.ldy;
  const int rank = p.adapter >= 0 ? rank_of(s, p.adapter) : 0;
  const int r = (int)s.r, k0 = j0 * 8;
  const bool live = k0 < rank;
  float u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = 0.0f;
  if (live) load_low(g.P, g.splits, s.T * s.r, t, r, k0, rank, s.scale[p.adapter], u);
  const uint16_t* M = g.M + (live ? (int64_t)p.adapter * g.C * r + k0 : 0);
  const bool mask = live && k0 + 8 > rank;
  for (int64_t n = o.n0; n < o.n1; n += 64) {
    const int64_t mine = n + j0 * (64 / G) + cl;  // this lane's column in the end
    float out = 0.0f;
    if (BASE && mine < g.C) out = load1(static_cast<const BT*>(g.base) + t * g.ldb + mine);
    if (rank > 0) {
      u32x4_t w[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int64_t c = n + j * (64 / G) + cl;
        w[j] = load16(M + (c < g.C ? c : g.C - 1) * r);
      }
      float add = 0.0f;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (mask) w[j] = keep_below(w[j], k0, rank);
        const unsigned wv[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        float a = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a = __builtin_fmaf(u[2 * e], __uint_as_float(wv[e] << 16), a);
          a = __builtin_fmaf(u[2 * e + 1], __uint_as_float(wv[e] & 0xffff0000u), a);
        }
        a = live ? a : 0.0f;
#pragma unroll
        for (int off = G / 2; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);
        if (j == j0) add = a;
      }
      out += add;
    }
    if (mine < g.C) {
      if (p.adapter == kBadAdapter) store_bits1(y + mine, kQNaN32);
      else store1(y + mine, out);
    }
  }
}

// dx of single rows: M is A as it lies, (n, r, C), so a lane takes 8 columns and adds up the ranks, 1 KB of
// A's row a wave and rank.  A workgroup per (row, 512 columns); its waves share out the ranks (a wave
// alone with 128 ranks waits for 16 rounds of loads: 20 us for 3 rows).
template <bool BASE>
__global__ __launch_bounds__(kLThreads) void lora_up_strided_kernel(UpArgs g, unsigned ranges) {
  constexpr int kCols = 512;
  __shared__ float part[4][kCols];
  const LoraSet& s = g.s;
  const int tid = tid_x(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = (int)s.r;
  // (ranges a multiple of 8, or below 8: the rows of one range on one die, for A's part in its L2)
  const int64_t t = large_bid() / ranges, c0 = (int64_t)(large_bid() % ranges) * kCols;
  if (c0 >= g.C || t >= s.T) return;
  const int i = find_request(s.start, (int)s.R, t);
  if (i < 0) return;
  const Part p = part_of(s, i, t, t + 1);
  if (p.hi <= p.lo) return;
  const int a = p.adapter, rank = a >= 0 ? rank_of(s, a) : 0;
  const int64_t col = c0 + lane * 8, at = col < g.C ? col : 0;
  // this wave's ranks, and (lane l) v of the l-th of them
  const int per = (rank + 3) / 4, k0 = min(wave * per, rank), n = min(k0 + per, rank) - k0;
  float v = 0.0f;
  if (lane < n) {
    for (int sp = 0; sp < g.splits; ++sp) v += g.P[((int64_t)sp * s.T + t) * r + k0 + lane];
    v *= s.scale[a];
  }
  float out[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = 0.0f;
  const uint16_t* M = g.M + (a >= 0 ? ((int64_t)a * r + k0) * g.C : 0) + at;
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float vr = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), k));
    float w[8];
    load8(M + (int64_t)k * g.C, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = __builtin_fmaf(vr, w[e], out[e]);
  }
  f32x4_t* mine = reinterpret_cast<f32x4_t*>(part[wave] + lane * 8);
  mine[0] = (f32x4_t){out[0], out[1], out[2], out[3]};
  mine[1] = (f32x4_t){out[4], out[5], out[6], out[7]};
  __syncthreads();
  // two columns a thread (C is even)
  const int64_t c = c0 + 2 * tid;
  if (c >= g.C) return;
  float* y = static_cast<float*>(g.y) + t * g.ldy + c;
  const float* base = static_cast<const float*>(g.base) + (BASE ? t * g.ldb + c : 0);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float sum = BASE ? base[e] : 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) sum += part[w][2 * tid + e];
    if (a == kBadAdapter) store_bits1(y + e, kQNaN32);
    else y[e] = sum;
  }
}

// ------------------------------------------------------------------ terms of u and v from partial sums

constexpr int kValStride = kLoraMaxRank + 1;
// The terms of s_a P from the down kernels' partial sums: a workgroup per 32 rows; 0 for rows
// without an adapter and ranks beyond the adapter's.
struct TermArgs {
  LoraSet s;
  const float* P;
  int splits;
  Terms o;
};
__global__ __launch_bounds__(kLThreads) void lora_terms_kernel(TermArgs g0, TermArgs g1, unsigned blocks0) {
  __shared__ float vals[kTileRows * kValStride];
  const bool second = bid_x() >= blocks0;
  const TermArgs& g = second ? g1 : g0;
  const LoraSet& s = g.s;
  const int r = (int)s.r, r4 = r / 4;
  const int64_t t0 = (int64_t)(bid_x() - (second ? blocks0 : 0)) * kTileRows;
  const int first = max(find_request(s.start, (int)s.R, t0), 0);
  for (int n = tid_x(); n < kTileRows * r4; n += kLThreads) {
    const int row = n / r4, k0 = (n - row * r4) * 4;
    const int64_t t = t0 + row;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    if (t < s.T) {
      int i = first;
      while (i + 1 < s.R && s.start[i + 1] <= t) ++i;
      const Part p = part_of(s, i, t, t + 1);
      if (p.hi > p.lo && p.adapter >= 0) {
        const int rank = rank_of(s, p.adapter);
        const float scale = s.scale[p.adapter];
        const float* P = g.P + t * r + k0;
        for (int sp = 0; sp < g.splits; ++sp) v += *reinterpret_cast<const f32x4_t*>(P + sp * s.T * r);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k0 + k < rank ? scale * v[k] : 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) vals[row * kValStride + k0 + k] = v[k];
  }
  __syncthreads();
  emit_terms<kLThreads>(g.o, vals, kValStride, t0, r);
}

// ------------------------------------------------------------------ grad: W^T X over the rows of an adapter

constexpr int kGradCols = 256;  // columns of X of a workgroup
constexpr int kGradRows = 64;   // rows staged at once

struct GradArgs {
  LoraSet s;
  const uint16_t* X;  // (T, C)
  int64_t ldx, C;
  const uint16_t* W;  // Terms::W
  float* out;  // (n, r, C) or, transposed, (n, C, r); [splits] of them when splits > 1
  int splits;
  int64_t tslice;  // rows of a split
  float* P;  // v in the same pass (TRANS): partial sums [blocks of columns][T][r], or nullptr
};

// Rows at .. at + 63 (at a multiple of 32), and those of them that use the adapter.
struct Stage {
  int at;
  unsigned long long rows;
};
// The stages of adapter a within [t0, t1), in order, 64 requests looked at together (each lane keeps one's rows), so
// that going on to the next takes no load.  A stage takes all requests that reach into it: a batch of requests of
// a row each is as quick as one request of all rows (256 requests of 3 adapters: 168 us with a stage each).
struct RowWalk {
  int base, lo, hi;          // requests base .. + 63; the rows of this lane's
  unsigned long long left;   // those of the adapter that are still to come
  int from, to;              // rows of the request at hand that no stage has taken; from = to: none

  __device__ __forceinline__ void look(const LoraSet& s, int a, int64_t t0, int64_t t1) {
    const int i = base + (tid_x() & 63);
    bool hit = false;
    lo = hi = 0;
    if (i < s.R) {
      const Part p = part_of(s, i, t0, t1);
      hit = p.adapter == a && p.hi > p.lo;
      lo = (int)p.lo;
      hi = (int)p.hi;
    }
    left = __ballot(hit);
  }
  __device__ __forceinline__ bool next_request(const LoraSet& s, int a, int64_t t0, int64_t t1) {
    while (!left) {
      base += 64;
      if (base >= s.R) return false;
      look(s, a, t0, t1);
    }
    const int i = __builtin_ctzll(left);
    left &= left - 1;
    from = __builtin_amdgcn_readlane(lo, i);
    to = __builtin_amdgcn_readlane(hi, i);
    return true;
  }
  // (st is left as it is when there is none)
  __device__ __forceinline__ bool next(const LoraSet& s, int a, int64_t t0, int64_t t1, Stage& st) {
    if (from >= to && !next_request(s, a, t0, t1)) return false;
    const int at = from & ~31, end = at + 64;
    unsigned long long rows = 0;
    while (true) {
      const int upto = min(to, end);
      rows |= (~0ull >> (64 - (upto - from))) << (from - at);
      if (to > end) {
        from = end;
        break;
      }
      from = to;
      if (!next_request(s, a, t0, t1)) break;
      if (from < at || from >= end) break;
    }
    st = Stage{at, rows};
    return true;
  }
};

// A workgroup per (adapter, 256 columns, split of the rows).  64 rows of X at a time go
// through LDS, double buffered, and are read back transposed (ds_read_b64_tr_b16: 16 lanes
// supply a 4 x 16 block of rows k, and lane i receives its column i), which gives the MFMA
// its 8 consecutive rows; the W terms lie along the rows already (a stage starts at a multiple of 32 rows).  The 16-byte pieces of a
// staged row are swapped by (row % 4, row / 8 % 2), so that the 8 rows that 32 lanes read
// together fall on different banks.
// RB: blocks of 16 ranks.  The waves share the ranks first (WR groups, RBW blocks each) and
// then the columns, so that a W term is read by as few waves as can be and serves 4 to 16
// blocks of columns.  TRANS: the result is (C, r), so the columns of X are the rows of the
// product.
// VP: X is dy, and the pass that adds up dB also multiplies each staged row by its columns' rows of
// B (in registers), so that dy is read once: v = dy B comes out as partial sums of 256 columns.  They
// take r / 64 of dy's bytes to write and to read, so up to 16 ranks.
// Bound by reading x and dy between barriers, two workgroups a compute unit (LDS): 41 us for both of 8192 x 4096,
// r 64 (134 MB: 3.3 TB/s), 19 us for 4096 x 4096 of 4 adapters, r 16; dy of 2048 x 151936 with v 159 us
// (622 MB: 3.9 TB/s).  W's terms asked for a stage ahead, and x two stages ahead, took longer (registers).
__device__ __forceinline__ int stage_at(int row, int piece) {
  return row * (kGradCols * 2) + ((piece ^ (2 * (row & 3) + 8 * ((row >> 3) & 1))) << 4);
}
template <int RB, bool TRANS, bool VP = false>
__device__ __forceinline__ void grad_tile(const GradArgs& g, unsigned block, uint8_t* lds) {
  constexpr int WR = RB < 4 ? RB : 4, RBW = RB / WR, CB = kGradCols / 16 * WR / 4;
  const LoraSet& s = g.s;
  const int tid = tid_x(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, q = lane >> 4, r = (int)s.r;
  const int wr = wave % WR, wc = wave / WR;  // ranks 16 RBW wr .., columns 16 CB wc ..
  const unsigned cols = (unsigned)((g.C + kGradCols - 1) / kGradCols);
  const int64_t c0 = (int64_t)(block % cols) * kGradCols;
  const int split = (int)(block / cols % (unsigned)g.splits);
  const int a = (int)(block / cols / (unsigned)g.splits);
  if (a >= s.n) return;
  const int64_t t0 = split * g.tslice, t1 = t0 + g.tslice < s.T ? t0 + g.tslice : s.T;
  f32x4_t acc[CB][RBW];
#pragma unroll
  for (int h = 0; h < CB; ++h)
#pragma unroll
    for (int b = 0; b < RBW; ++b) acc[h][b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  // staging: thread tid moves 16 bytes of rows tid / 32 + 8 j
  const int srow = tid >> 5, spiece = tid & 31;
  const int64_t scol = c0 + spiece * 8 < g.C ? spiece * 8 : 0;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  // (loaded without conditions, from rows between the stage's first and last, and cut where it is written: a
  // select here would have to wait for the load; columns behind the last are 0, as B's rows there are for v)
  const bool scol_in = c0 + spiece * 8 < g.C;
  const uint32_t ldx = (uint32_t)g.ldx;
  auto fetch = [&](const Stage& w, u32x4_t (&v)[8]) {
    const uint16_t* X = g.X + w.at * g.ldx + c0;
    const int lo = __builtin_ctzll(w.rows), hi = 63 - __builtin_clzll(w.rows);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = load16(X + ((uint32_t)min(max(srow + 8 * j, lo), hi) * ldx + (uint32_t)scol));
  };
  // B's rows c0 .. c0 + 255 as operands: column rho, 8 consecutive rows of k-step ks
  u32x4_t bv[VP ? kGradCols / 32 : 1];
  if (VP) {
    static_assert(!VP || RB == 1, "one block of ranks");
    const int rho = min(c16, r - 1);
#pragma unroll
    for (int ks = 0; ks < kGradCols / 32; ++ks) {
      unsigned e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t col = c0 + 32 * ks + 8 * q + k;
        const unsigned v = s.B[((int64_t)a * g.C + (col < g.C ? col : g.C - 1)) * r + rho];
        e[k] = col < g.C ? v : 0u;
      }
      bv[ks] = (u32x4_t){e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    }
  }
  RowWalk w{-64, 0, 0, 0ull, 0, 0};
  Stage coming{0, 0ull};
  bool more = w.next(s, a, t0, t1, coming);
  u32x4_t held[8];
  if (more) fetch(coming, held);
  int stage = 0;
  while (more) {
    uint8_t* T = lds + stage * (kGradRows * kGradCols * 2);
    const Stage now = coming;
    const unsigned long long mine = scol_in ? now.rows >> srow : 0ull;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      *reinterpret_cast<u32x4_t*>(T + stage_at(srow + 8 * j, spiece)) = mine >> (8 * j) & 1 ? held[j] : zero;
    }
    // the W operands of the two k-steps (rows now.at .. and now.at + 32 ..)
    u32x4_t wv[2][RBW][3];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int b = 0; b < RBW; ++b)
#pragma unroll
        for (int tm = 0; tm < 3; ++tm)
          wv[ks][b][tm] = load16(g.W + (((int64_t)(now.at / 32 + ks) * RB + wr * RBW + b) * 3 + tm) * 512 + lane * 8);
    // (behind the last stage its own rows once more, so that the loads are not conditional)
    more = w.next(s, a, t0, t1, coming);
    fetch(coming, held);
    __syncthreads();
    if (~now.rows) {
      // rows of other requests may hold anything: neither side may keep them
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const unsigned m = (unsigned)(now.rows >> (32 * ks)) >> (8 * q);
        unsigned keep[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) keep[e] = (m >> (2 * e) & 1 ? 0xffffu : 0u) | (m >> (2 * e) & 2 ? 0xffff0000u : 0u);
        const u32x4_t k4 = {keep[0], keep[1], keep[2], keep[3]};
#pragma unroll
        for (int b = 0; b < RBW; ++b)
#pragma unroll
          for (int tm = 0; tm < 3; ++tm) wv[ks][b][tm] &= k4;
      }
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int h = 0; h < CB; ++h) {
        typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
        const int row = 32 * ks + 8 * q + (c16 >> 2), col = 16 * (wc * CB + h) + 4 * (c16 & 3);
        const int in = (col & 7) * 2;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(T + stage_at(row, col >> 3) + in));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(T + stage_at(row + 4, col >> 3) + in));
        const s16x4_t v8[2] = {lo, hi};
        const u32x4_t x = __builtin_bit_cast(u32x4_t, v8);
#pragma unroll
        for (int b = 0; b < RBW; ++b)
#pragma unroll
          for (int tm = 0; tm < 3; ++tm)
            acc[h][b] = TRANS ? mfma(x, wv[ks][b][tm], acc[h][b]) : mfma(wv[ks][b][tm], x, acc[h][b]);
      }
    }
    if (VP) {
      // rows 16 wave .. + 15 of the stage
      f32x4_t vp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kGradCols / 32; ++ks)
        vp = mfma(*reinterpret_cast<const u32x4_t*>(T + stage_at(16 * wave + c16, 4 * ks + q)), bv[ks], vp);
      float* P = g.P + (int64_t)(block % cols) * s.T * r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * wave + 4 * q + e;
        if ((now.rows >> row & 1) && c16 < r) P[(int64_t)(now.at + row) * r + c16] = vp[e];
      }
    }
    stage ^= 1;  // (a stage is written again only behind the next barrier, which is behind its reads)
  }
  const int rank = rank_of(s, a);
  float* out = g.out + (int64_t)split * s.n * s.r * g.C + (int64_t)a * s.r * g.C;
#pragma unroll
  for (int h = 0; h < CB; ++h)
#pragma unroll
    for (int b = 0; b < RBW; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int along = c16, down = 4 * q + e;
        const int64_t col = c0 + 16 * (wc * CB + h) + (TRANS ? down : along);
        const int rho = 16 * (wr * RBW + b) + (TRANS ? along : down);
        if (col < g.C && rho < r) {
          const float v = rho < rank ? acc[h][b][e] : 0.0f;
          out[TRANS ? col * r + rho : (int64_t)rho * g.C + col] = v;
        }
      }
}

template <int RB>
__global__ __launch_bounds__(kLThreads) void lora_grad_kernel(GradArgs ga, unsigned blocks_a, GradArgs gb,
                                                              unsigned blocks_b) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kGradRows * kGradCols * 2];
  const unsigned block = large_bid();
  if (block < blocks_a) grad_tile<RB, false>(ga, block, lds);
  else if (block - blocks_a < blocks_b) grad_tile<RB, true>(gb, block - blocks_a, lds);
}

__global__ __launch_bounds__(kLThreads) void lora_grad_v_kernel(GradArgs g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kGradRows * kGradCols * 2];
  grad_tile<1, true, true>(g, large_bid(), lds);
}

// The partial sums of the column blocks, [n][plane], added up in order to [parts][plane]: part p takes
// per of them.
__global__ __launch_bounds__(kLThreads) void lora_reduce_kernel(const float* P, int n, int64_t plane, int per, float* out) {
  const int64_t quads = plane / 4, at = (int64_t)bid_x() * kLThreads + tid_x();
  const int64_t part = at / quads, i = at - part * quads;
  const int k0 = (int)part * per, k1 = min(k0 + per, n);
  if (k0 >= n) return;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int k = k0; k < k1; ++k) v += reinterpret_cast<const f32x4_t*>(P + k * plane)[i];
  reinterpret_cast<f32x4_t*>(out + part * plane)[i] = v;
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

// Whether the kernels of single rows are taken, and not those of tiles of 32 rows: by what each
// is estimated to cost, in us, from times measured over T = 16..2048, R = 1..256, r = 16, 64, H =
// 4096, N = 4096 and 151936.  Single rows read an adapter once for every row, from the L2s at about 8
// TB/s.  A tile takes the requests that share it (1 + 32 R / T on average) one after the other,
// each a pass over the down products' axes (a split's share of them) and over the tile's columns of y.
//   T 64, R 1 / 8 / 64: 9.4 / 9.4 / 9.3 us as rows (in two launches), 13.3 / 35.6 / 236 as tiles;
//   T 512, R 1, r 64: 37 as rows, 24 as tiles; T 1024, R 2 / 128: 35 / 38 as rows, 18 / 44 as tiles;
//   T 64, R 1 / 8, N 151936: 43 / 43 as rows, 27 / 61 as tiles.
// Beyond 64 ranks tiles take about twice as long (T 256, R 13, 2048 x 1024: 33 us with r 64, 75 with 128, where rows
// take 14 and 24).
bool single_rows(int64_t T, int64_t R, int64_t r, int64_t H, int64_t N, bool backward) {
  const double read = 2.0 * (double)T * (double)r * (double)(backward ? 2 * H + N : H + N);
  const double rows = 4.0 + read / 8.0e6;
  double shared = 1.0 + 32.0 * (double)R / (double)T;
  if (shared > 32.0) shared = 32.0;
  auto pass = [](int64_t K) { return 1.0 + 3.0 * (double)(K <= 8192 ? K : 8192) / 4096.0; };
  double tiles = 13.0 + shared * (pass(H) + (backward ? pass(N) : 0.0)) +
                 (shared - 1.0) * (double)T * (double)(backward ? H : N) * 8.0 / 10.0e6;
  if (r > 64) tiles *= 2.0;
  // (and single rows' workgroups are counted in 32 bits)
  return rows < tiles && T * (((H > N ? H : N) + 255) / 256) < (1 << 30);
}

// Splits of a down product's K.  Single rows (units: waves a row): enough for 512 workgroups where K
// allows ranges of 512.  Tiles: one, whose workgroups finish the product themselves, unless K is long
// (beyond 8192) and the tiles are few; then enough for 512 workgroups, of 4096 k at least.
void down_split(int64_t T, bool rows, int64_t K, int64_t units, int& splits, int64_t& kslice) {
  const int64_t groups = rows ? (T * units + 3) / 4 : (T + kTileRows - 1) / kTileRows;
  int64_t want = (512 + groups - 1) / groups, most = rows ? K / 512 : K <= 8192 ? 1 : K / 4096;
  if (want > most) want = most;
  if (want > kMaxSplits) want = kMaxSplits;
  if (want < 1) want = 1;
  const int64_t per = (K + want - 1) / want;
  kslice = (per + kDownK - 1) / kDownK * kDownK;
  splits = (int)((K + kslice - 1) / kslice);
}
int64_t quads_of(int64_t r) { return r / kRowRanks; }
int64_t wides_of(int64_t r) { return (r + kRowWide - 1) / kRowWide; }

// u and, when v.P is given, v of single rows.
hipError_t launch_down_rows(const DownArgs& u, bool want_u, const DownArgs& v, bool want_v, hipStream_t st) {
  const unsigned bu = want_u ? (unsigned)((u.s.T * quads_of(u.s.r) * u.splits + 3) / 4) : 0u;
  const unsigned bv = want_v ? (unsigned)((v.s.T * wides_of(v.s.r) * v.splits + 3) / 4) : 0u;
  if (bu + bv == 0) return hipSuccess;
  hipLaunchKernelGGL(lora_down_row_kernel, large_grid((int64_t)bu + bv), dim3(kLThreads), 0, st, u, bu, v, bv);
  return hipGetLastError();
}

template <int RB>
hipError_t launch_down_t(const DownArgs& g, TransposeArgs tr, bool product, hipStream_t st) {
  const int64_t blocks = tr.s.n * (tr.s.r / 8) * ((tr.At ? tr.s.H / 8 : 0) + (tr.Bt ? tr.s.N / 8 : 0));
  tr.blocks = (unsigned)((blocks + Down<RB>::kThreads - 1) / Down<RB>::kThreads);
  const unsigned tiles = product ? (unsigned)((g.s.T + kTileRows - 1) / kTileRows * g.splits) : 0u;
  if (tr.blocks + tiles == 0) return hipSuccess;
  hipLaunchKernelGGL(lora_down_tile_kernel<RB>, dim3(tr.blocks + tiles), dim3(Down<RB>::kThreads), 0, st, g, tr);
  return hipGetLastError();
}
// A product of tiles (if wanted), and the transposes of tr in the same launch.
hipError_t launch_down_tiles(const DownArgs& g, bool product, const TransposeArgs& tr, hipStream_t st) {
  const int64_t r = g.s.r;
  if (r <= 16) return launch_down_t<1>(g, tr, product, st);
  if (r <= 32) return launch_down_t<2>(g, tr, product, st);
  if (r <= 64) return launch_down_t<4>(g, tr, product, st);
  return launch_down_t<8>(g, tr, product, st);
}

hipError_t launch_terms(const TermArgs& a, const TermArgs& b, hipStream_t st) {
  const unsigned tiles = (unsigned)((a.s.T + kTileRows - 1) / kTileRows);
  const bool both = (a.o.U || a.o.W) && (b.o.U || b.o.W), one = a.o.U || a.o.W || b.o.U || b.o.W;
  if (!one) return hipSuccess;
  const TermArgs& f = a.o.U || a.o.W ? a : b;
  hipLaunchKernelGGL(lora_terms_kernel, dim3(both ? 2 * tiles : tiles), dim3(kLThreads), 0, st, f, b, tiles);
  return hipGetLastError();
}

// Single rows: `columns` a wave and step; more steps once there are 16384 waves.
dim3 up_rows_grid(UpArgs& g, int64_t columns) {
  const int64_t T = g.s.T;
  g.steps = (int)(T * ((g.C + columns - 1) / columns) / 16384);
  g.steps = g.steps < 1 ? 1 : g.steps > 16 ? 16 : g.steps;
  const int64_t ranges = (g.C + 4 * columns * g.steps - 1) / (4 * columns * g.steps);
  return large_grid((ranges + 7) / 8 * 8 * T);
}

hipError_t launch_up_strided(const UpArgs& g, hipStream_t st) {
  unsigned ranges = (unsigned)((g.C + 511) / 512);
  if (ranges > 8) ranges = (ranges + 7) / 8 * 8;
  const dim3 grid = large_grid(ranges * g.s.T);
  if (g.base) hipLaunchKernelGGL(lora_up_strided_kernel<true>, grid, dim3(kLThreads), 0, st, g, ranges);
  else hipLaunchKernelGGL(lora_up_strided_kernel<false>, grid, dim3(kLThreads), 0, st, g, ranges);
  return hipGetLastError();
}

// Single rows in one launch: steps of 256 columns of a workgroup for about 256 workgroups, and whether A's part,
// read by each of them from the L2s at about 8 TB/s, costs less than the second launch (about 4 us).
bool one_launch(int64_t T, int64_t r, int64_t H, int64_t N, int& steps) {
  const int64_t units = (N + 255) / 256;
  steps = (int)((T * units + 255) / 256);
  steps = steps > 16 ? 16 : steps;
  return r <= 32 && T * ((units + steps - 1) / steps) * r * H * 2 <= (1 << 25);
}

template <typename YT, typename BT, bool BASE>
hipError_t launch_up_t(UpArgs g, bool rows, hipStream_t st, const RowArgs& d) {
  const int64_t r = g.s.r, T = g.s.T;
  if (rows && d.X) {
    const dim3 grid((unsigned)(T * ((g.C + 256 * g.steps - 1) / (256 * g.steps))));
    if (r <= 8) hipLaunchKernelGGL((lora_row_kernel<1, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g, d);
    else if (r <= 16) hipLaunchKernelGGL((lora_row_kernel<2, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g, d);
    else hipLaunchKernelGGL((lora_row_kernel<4, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g, d);
    return hipGetLastError();
  }
  if (rows) {
    const dim3 grid = up_rows_grid(g, 64);
    if (r <= 8) hipLaunchKernelGGL((lora_up_lane_kernel<1, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else if (r <= 16) hipLaunchKernelGGL((lora_up_lane_kernel<2, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else if (r <= 32) hipLaunchKernelGGL((lora_up_lane_kernel<4, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else if (r <= 64) hipLaunchKernelGGL((lora_up_row_kernel<8, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    else hipLaunchKernelGGL((lora_up_row_kernel<16, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
    return hipGetLastError();
  }
  // a wave's columns: 4 steps of 64, fewer where that leaves less than 1024 workgroups
  const int64_t tiles = (T + kTileRows - 1) / kTileRows;
  g.steps = 4;
  while (g.steps > 1 && tiles * ((g.C + 256 * g.steps - 1) / (256 * g.steps)) < 1024) g.steps /= 2;
  const int64_t per = 256 * g.steps;
  const dim3 grid((unsigned)(tiles * ((g.C + per - 1) / per)));
  if (r <= 8) hipLaunchKernelGGL((lora_up_tile_kernel<1, 1, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else if (r <= 16) hipLaunchKernelGGL((lora_up_tile_kernel<1, 2, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else if (r <= 32) hipLaunchKernelGGL((lora_up_tile_kernel<1, 3, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else if (r <= 64) hipLaunchKernelGGL((lora_up_tile_kernel<2, 3, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  else hipLaunchKernelGGL((lora_up_tile_kernel<4, 3, YT, BT, BASE>), grid, dim3(kLThreads), 0, st, g);
  return hipGetLastError();
}

template <typename YT>
hipError_t launch_up_y(const UpArgs& g, Dt base_dt, bool rows, hipStream_t st, const RowArgs& d = RowArgs{}) {
  if (!g.base) return launch_up_t<YT, float, false>(g, rows, st, d);
  return base_dt == Dt::BF16 ? launch_up_t<YT, uint16_t, true>(g, rows, st, d)
                             : launch_up_t<YT, float, true>(g, rows, st, d);
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

size_t u_bytes(int64_t T, int64_t r) {
  return (size_t)((T + kTileRows - 1) / kTileRows) * 2 * up_ld((int)r) * up_tm((int)r) * 1024;
}

struct ForwardWs {
  float* P;     // partial sums: single rows, or several splits
  uint16_t* U;  // tiles: the terms of u
  bool rows;
  int splits;
  int64_t kslice;
  size_t bytes;
};
ForwardWs forward_ws(void* base, int64_t T, int64_t R, int64_t H, int64_t N, int64_t r) {
  ForwardWs w{};
  w.rows = single_rows(T, R, r, H, N, false);
  down_split(T, w.rows, H, quads_of(r), w.splits, w.kslice);
  const size_t p = w.rows || w.splits > 1 ? align256((size_t)w.splits * T * r * 4) : 0;
  const size_t u = w.rows ? 0 : align256(u_bytes(T, r));
  char* b = static_cast<char*>(base);
  w.P = reinterpret_cast<float*>(b);
  w.U = b ? reinterpret_cast<uint16_t*>(b + p) : nullptr;
  w.bytes = p + u;
  return w;
}

// Whether dB's pass over dy forms v as well: up to 16 ranks and from 2^28 bytes of dy on.  2048 x
// 151936: 300 us in two passes, 242 in one; but 4096 x 4096 69 and 79, 8192 x 4096 88 and 99 (its
// launches follow one another, and the pass holds fewer workgroups at once); r 32, 2048 x 151936: 336
// and 606 (registers).
bool one_pass_over_dy(int64_t T, int64_t N, int64_t r) { return r <= 16 && T * N * 2 >= (1 << 28); }
constexpr int kReduceParts = 16;

struct BackwardWs {
  float *Pu, *Pv;
  uint16_t *At, *Bt, *Wu, *Wv, *Uv;
  float *partA, *partB;
  float* Pf;  // v's partial sums of dB's pass
  bool rows;
  int splits_u, splits_v;
  int64_t kslice_u, kslice_v;
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
  w.rows = single_rows(T, R, r, H, N, true);
  down_split(T, w.rows, H, quads_of(r), w.splits_u, w.kslice_u);
  down_split(T, w.rows, N, wides_of(r), w.splits_v, w.kslice_v);
  grad_split(T, n, H, w.splits_A, w.tslice_A);
  grad_split(T, n, N, w.splits_B, w.tslice_B);
  const bool fused = !w.rows && one_pass_over_dy(T, N, r);
  const int parts = fused && kReduceParts > w.splits_v ? kReduceParts : w.splits_v;
  if (w.rows || w.splits_u > 1) w.Pu = reinterpret_cast<float*>(take((size_t)w.splits_u * T * r * 4));
  if (w.rows || fused || w.splits_v > 1) w.Pv = reinterpret_cast<float*>(take((size_t)parts * T * r * 4));
  if (!w.rows) {
    w.At = reinterpret_cast<uint16_t*>(take((size_t)n * H * r * 2));
    w.Uv = reinterpret_cast<uint16_t*>(take(u_bytes(T, r)));
    // B the other way round, or (one pass over dy) v's partial sums: never both
    const size_t bt = (size_t)n * N * r * 2, pf = fused ? (size_t)((N + kGradCols - 1) / kGradCols) * T * r * 4 : 0;
    char* q = take(bt > pf ? bt : pf);
    w.Bt = reinterpret_cast<uint16_t*>(q);
    w.Pf = fused ? reinterpret_cast<float*>(q) : nullptr;
  }
  // (a stage of the gradients may reach one tile beyond the last)
  const size_t wb = ((size_t)((T + kTileRows - 1) / kTileRows) + 1) * rank_blocks((int)r) * 3 * 1024;
  w.Wu = reinterpret_cast<uint16_t*>(take(wb));
  w.Wv = reinterpret_cast<uint16_t*>(take(wb));
  w.partA = w.splits_A > 1 ? reinterpret_cast<float*>(take((size_t)w.splits_A * n * r * H * 4)) : nullptr;
  w.partB = w.splits_B > 1 ? reinterpret_cast<float*>(take((size_t)w.splits_B * n * r * N * 4)) : nullptr;
  w.bytes = off;
  return w;
}

template <int RB>
hipError_t launch_grad_t(const GradArgs& ga, unsigned ba, const GradArgs& gb, unsigned bb, hipStream_t st) {
  if (ba + bb == 0) return hipSuccess;
  hipLaunchKernelGGL(lora_grad_kernel<RB>, large_grid((int64_t)ba + bb), dim3(kLThreads), 0, st, ga, ba, gb, bb);
  return hipGetLastError();
}
hipError_t launch_grad(const GradArgs& ga, unsigned ba, const GradArgs& gb, unsigned bb, hipStream_t st) {
  const int64_t r = ga.s.r;
  if (r <= 16) return launch_grad_t<1>(ga, ba, gb, bb, st);
  if (r <= 32) return launch_grad_t<2>(ga, ba, gb, bb, st);
  if (r <= 64) return launch_grad_t<4>(ga, ba, gb, bb, st);
  return launch_grad_t<8>(ga, ba, gb, bb, st);
}

}  // namespace

size_t lora_forward_workspace_bytes(int64_t T, int64_t R, int64_t H, int64_t N, int64_t r) {
  return forward_ws(nullptr, T, R, H, N, r).bytes;
}

size_t lora_backward_workspace_bytes(int64_t T, int64_t R, int64_t n, int64_t H, int64_t N, int64_t r) {
  return backward_ws(nullptr, T, R, n, H, N, r).bytes;
}

hipError_t launch_lora_forward(const LoraForwardArgs& a, hipStream_t st) {
  (void)hipGetLastError();
  const LoraSet& s = a.s;
  const ForwardWs w = forward_ws(a.workspace, s.T, s.R, s.H, s.N, s.r);
  const Terms o{w.U, nullptr};
  const DownArgs d{s, a.x, a.ldx, s.A, s.H, w.P, w.splits, w.kslice, o};
  RowArgs row{};
  int steps = 0;
  if (w.rows && one_launch(s.T, s.r, s.H, s.N, steps)) {
    row = RowArgs{a.x, s.A, a.ldx, s.H};
  } else if (w.rows) {
    if (hipError_t e = launch_down_rows(d, true, DownArgs{}, false, st)) return e;
  } else {
    const TransposeArgs none{s, nullptr, nullptr, 0};
    if (hipError_t e = launch_down_tiles(d, true, none, st)) return e;
    if (w.splits > 1) {
      const TermArgs t{s, w.P, w.splits, o}, no{};
      if (hipError_t e = launch_terms(t, no, st)) return e;
    }
  }
  const UpArgs g{s, w.P, w.splits, w.U, s.B, s.N, false, a.base, a.ldb, a.y, a.ldy, steps};
  return a.y_dt == Dt::BF16 ? launch_up_y<uint16_t>(g, a.base_dt, w.rows, st, row)
                            : launch_up_y<float>(g, a.base_dt, w.rows, st, row);
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
  const bool one_pass = w.Pf && a.gB && need_v;  // v in dB's pass over dy
  // u for dB (terms along the rows); v for dx (terms along the ranks, or partial sums for single rows) and dA
  const Terms ou{nullptr, a.gB ? w.Wu : nullptr};
  const Terms ov{a.gx ? w.Uv : nullptr, a.gA ? w.Wv : nullptr};
  const DownArgs du{s, a.x, a.ldx, s.A, s.H, w.Pu, w.splits_u, w.kslice_u, ou};
  int splits_v = w.splits_v;
  if (w.rows) {
    const DownArgs dv{s, a.dy, a.lddy, s.B, s.N, w.Pv, splits_v, w.kslice_v, Terms{}};
    if (hipError_t e = launch_down_rows(du, a.gB != nullptr, dv, need_v, st)) return e;
    const TermArgs tu{s, w.Pu, w.splits_u, ou}, tv{s, w.Pv, splits_v, Terms{nullptr, ov.W}};
    if (hipError_t e = launch_terms(tu, tv, st)) return e;
  } else {
    const TransposeArgs tr{s, a.gx ? w.At : nullptr, need_v && !one_pass ? w.Bt : nullptr, 0};
    if (hipError_t e = launch_down_tiles(du, a.gB != nullptr, tr, st)) return e;
    const bool tu = a.gB && w.splits_u > 1;
    if (need_v && !one_pass) {
      const DownArgs dv{s, a.dy, a.lddy, w.Bt, s.N, w.Pv, splits_v, w.kslice_v, ov};
      if (hipError_t e = launch_down_tiles(dv, true, TransposeArgs{s, nullptr, nullptr, 0}, st)) return e;
    }
    const TermArgs gu{s, w.Pu, w.splits_u, tu ? ou : Terms{}};
    const TermArgs gv{s, w.Pv, splits_v, need_v && !one_pass && splits_v > 1 ? ov : Terms{}};
    if (hipError_t e = launch_terms(gu, gv, st)) return e;
  }
  const int64_t cols_A = (s.H + kGradCols - 1) / kGradCols, cols_B = (s.N + kGradCols - 1) / kGradCols;
  const GradArgs ga{s, a.x, a.ldx, s.H, w.Wv, w.splits_A > 1 ? w.partA : a.gA, w.splits_A, w.tslice_A, nullptr};
  const GradArgs gb{s, a.dy, a.lddy, s.N, w.Wu, w.splits_B > 1 ? w.partB : a.gB, w.splits_B, w.tslice_B, w.Pf};
  const unsigned ba = a.gA ? (unsigned)(s.n * w.splits_A * cols_A) : 0u;
  const unsigned bb = a.gB ? (unsigned)(s.n * w.splits_B * cols_B) : 0u;
  if (one_pass) {
    hipLaunchKernelGGL(lora_grad_v_kernel, large_grid(bb), dim3(kLThreads), 0, st, gb);
    if (hipError_t e = hipGetLastError()) return e;
    const float* P = w.Pf;
    splits_v = (int)cols_B;
    if (splits_v > kReduceParts) {
      const int per = (splits_v + kReduceParts - 1) / kReduceParts;
      splits_v = (splits_v + per - 1) / per;
      const int64_t threads = splits_v * (s.T * s.r / 4);
      hipLaunchKernelGGL(lora_reduce_kernel, dim3((unsigned)((threads + kLThreads - 1) / kLThreads)), dim3(kLThreads), 0,
                         st, P, (int)cols_B, s.T * s.r, per, w.Pv);
      if (hipError_t e = hipGetLastError()) return e;
      P = w.Pv;
    }
    const TermArgs gv{s, P, splits_v, ov}, no{};
    if (hipError_t e = launch_terms(gv, no, st)) return e;
  }
  if (a.gx) {
    UpArgs g{s, w.Pv, splits_v, w.Uv, w.rows ? s.A : w.At, s.H, true, a.base, a.ldb, a.gx, a.ldgx, 0};
    if (hipError_t e = w.rows ? launch_up_strided(g, st) : launch_up_y<float>(g, Dt::F32, false, st)) return e;
  }
  if (hipError_t e = launch_grad(ga, ba, gb, one_pass ? 0u : bb, st)) return e;
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
