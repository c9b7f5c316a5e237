// The lm_head product, cross entropy and distillation from a teacher's top logits together, in pieces of the
// vocabulary: no logit is kept, and what is kept of the gradient of the logits is one piece.
//
//   z = x w^T                                   (bf16 operands, fp32 accumulation on the matrix cores)
//   ce, kd per row                              (kd_row.hpp)
//   G = k (g_ce d ce/dz + g_kd d kd/dz)         (bf16, a piece of the columns at a time)
//   grad_x += G w[piece],  grad_w[piece] = G^T x
//
// Two passes over 256 x 256 tiles of z (every tile is computed twice, in the same order of k, so both passes see
// the same bits): the first leaves for each row and tile the sum of exponentials outside the teacher's ids, and
// the logits at the ids and the target; a wave a row joins the sums.  The second, piece by piece, forms G from the
// joined sums in the product's epilogue.  Keeping the first pass's logits instead would take BT V values, which is
// what this path is there to avoid; a piece of the vocabulary makes grad_w's rows complete at once (no
// accumulation over pieces), and only grad_x, BT H values, is added up in fp32 from piece to piece.
//
// What bounds it: the matrix cores, four products of 2 BT V H.  At 8192 x 151936 x 4096, K 64: first pass 9.1 ms (1124
// TFLOP/s; a large library product reaches 1077 to 1216), second 8.4, grad_x 8.5, grad_w 8.1, all else 0.1.  An epilogue takes its ids from a scan of its 256
// rows' K ids (64 KB at K = 64, from L2, against 125 us of products a tile at H = 4096), which sets the mask of the
// tile in LDS and lists the entries that fall into it.
//
// G is rounded to bf16 (2^-8 relative at most per element, the operands' own precision): it is an operand of the
// matrix cores.
#include "distill.hpp"
#include "gemm.hpp"
#include "kd_row.hpp"
#include "mm_wide.hpp"

namespace lx {

namespace {

using mm::f32x16_t;

// ------------------------------------------------------------------ LDS beside the main loop

// The second pass stages its tile of G in the main loop's LDS, rows padded by 16 bytes (the half-waves'
// rows, 4 apart, fall on different banks).  In the first pass the same memory is a table of one float for each of the
// tile's rows and half of its columns, through which the logits at the ids pass from the lanes that hold them to the
// threads that know whose they are.
constexpr int kStagePitch = 264;  // halves
constexpr int kMainBytes = 256 * kStagePitch * 2;
static_assert(kMainBytes >= kLds && kMainBytes >= 256 * 128 * 4, "LDS of the main loop and of the table");
constexpr int kTileEntries = 2048;  // entries of a tile that are listed; with more, its rows' ids are scanned again

struct RowParam {  // a row of the second pass
  RowGrad g;
  int target;  // kNanRow, kZeroRow
};
constexpr int kNanRow = -2;
constexpr int kZeroRow = -3;  // ignored, or without any unmasked logit: 0 whatever its logits are

struct TileLds {
  uint32_t mask[256][8];        // bit c of row r: column n0 + c is one of the row's ids
  uint32_t list[kTileEntries];  // row << 16 | column << 8 | entry
  int listed;
  int target[256];              // the target's column in the tile, or -1; second pass: kNanRow, kZeroRow
  float4 p[256];                // second pass: what every column takes, {out, nr, n1, kce}
  float2 p_named[256];          // {kkd, nz}
};

struct TileArgs {
  const uint16_t *x, *w;
  int64_t H;
  int rows, V, first, width;  // columns [first, first + width) of the vocabulary
  const int32_t* ids;         // (rows, K): cleaned
  int K;
  float c;
  const int64_t* target;
  int64_t ignore_index;
  int tiles_m, tiles_n;
  // first pass
  float* parts;       // [rows][tiles_n][2 or 4]
  float* z_top;       // [rows][K]
  float* z_target;    // [rows]
  // second pass
  const RowParam* param;  // [rows]
  const float* q;         // [rows][K]: a token's mass at its one entry
  uint16_t* g;            // [rows][ldg]
  int64_t ldg;
};

// The tile's mask and list, by the whole workgroup; ends behind a barrier.
template <bool MASK>
__device__ __forceinline__ void scan_ids(TileLds& s, const TileArgs& a, int m0, int n0) {
  const int tid = tid_x();
  if (MASK)
    for (int i = tid; i < 256 * 8; i += kWideThreads) s.mask[i >> 3][i & 7] = 0u;
  if (tid == 0) s.listed = 0;
  __syncthreads();
  if (a.K) {
    const int total = min(256, a.rows - m0) * a.K;
    const int32_t* ids = a.ids + (int64_t)m0 * a.K;
    // eight requested at once: one by one they would cost a memory latency each
    for (int i0 = tid; i0 < total; i0 += 8 * kWideThreads) {
      int col[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) col[k] = ids[min(i0 + k * kWideThreads, total - 1)] - n0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * kWideThreads;
        if (i < total && (unsigned)col[k] < 256u) {
          const int r = i / a.K, j = i - r * a.K;
          if (MASK) atomicOr(&s.mask[r][col[k] >> 5], 1u << (col[k] & 31));
          const int at = atomicAdd(&s.listed, 1);
          if (at < kTileEntries) s.list[at] = (uint32_t)(r << 16 | col[k] << 8 | j);
        }
      }
    }
  }
  __syncthreads();
}

// f(row, column, entry) for every entry that names one of the tile's columns [128 h, 128 h + 128), by the whole
// workgroup.
template <typename F>
__device__ __forceinline__ void for_entries(const TileLds& s, const TileArgs& a, int m0, int n0, int h, F f) {
  const int tid = tid_x();
  if (s.listed <= kTileEntries) {
    for (int i = tid; i < s.listed; i += kWideThreads) {
      const uint32_t e = s.list[i];
      const int col = (int)(e >> 8 & 255u);
      if (col >> 7 == h) f((int)(e >> 16), col, (int)(e & 255u));
    }
  } else {
    const int total = min(256, a.rows - m0) * a.K;
    const int32_t* ids = a.ids + (int64_t)m0 * a.K;
    for (int i = tid; i < total; i += kWideThreads) {
      const int col = ids[i] - n0 - 128 * h;
      if ((unsigned)col < 128u) f(i / a.K, col + 128 * h, i % a.K);
    }
  }
}

// ------------------------------------------------------------------ passes over the tiles

template <bool GRAD, bool TEMP>
__global__ __attribute__((amdgpu_flat_work_group_size(kWideThreads, kWideThreads), amdgpu_waves_per_eu(2, 2)))
void kd_tile_kernel(TileArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kMainBytes];
  __shared__ TileLds s;
  static_assert(sizeof(TileLds) + kMainBytes <= 160 * 1024, "LDS");
  int tm, tn;
  if (!mm::tile_coords(a.tiles_m, a.tiles_n, tm, tn)) return;
  const int m0 = tm * mm::kBM, n0 = a.first + tn * 256, end = a.first + a.width;
  const int lane = tid_x() & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid_x() >> 6);
  const int wm = (wave & 1) * 128, wn = (wave >> 1) * 64;
  f32x16_t acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = (f32x16_t){};
  {
    mm::SliceLoader<true, 256, kWideThreads> la;
    mm::SliceLoader<true, 256, kWideThreads> lb;
    la.init(a.x, a.H, 2 * (int64_t)a.rows * a.H, a.rows, (int)a.H, m0, wave);
    lb.init(a.w, a.H, 2 * (int64_t)a.V * a.H, end, (int)a.H, n0, wave);
    mm::mainloop<true, true, 2, 256, kWideThreads, kWideMem>(acc, lds, la, lb, (int)a.H, wm, wn, wave);
  }
  const int tid = tid_x();
  if (tid < 256) {
    const int m = m0 + tid;
    int col = -1;
    if (m < a.rows) {
      if (GRAD) {
        const RowParam p = a.param[m];
        col = p.target < -1 ? p.target : p.target >= n0 && p.target < n0 + 256 ? p.target - n0 : -1;
        s.p[tid] = make_float4(p.g.out, p.g.nr, p.g.n1, p.g.kce);
        s.p_named[tid] = make_float2(p.g.kkd, p.g.nz);
      } else {
        const int64_t t = a.target[m];
        col = t != a.ignore_index && t >= n0 && t < n0 + 256 ? (int)(t - n0) : -1;
      }
    }
    s.target[tid] = col;
  }
  scan_ids<!GRAD>(s, a, m0, n0);
  if constexpr (!GRAD) {
    float* table = reinterpret_cast<float*>(lds);  // [256][128]
    const int half = wn >> 7;
    // the logits at the ids
    for (int h = 0; h < 2 && s.listed; ++h) {
      if (half == h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int lr = wm + 32 * i + mm::acc_row(r, lane);
            const uint2 mask = *reinterpret_cast<const uint2*>(&s.mask[lr][wn >> 5]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int lc = wn + 32 * j + (lane & 31);
              if (((j ? mask.y : mask.x) >> (lane & 31)) & 1u) table[lr * 128 + (lc & 127)] = acc[i][j][r];
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      __syncthreads();
      for_entries(s, a, m0, n0, h, [&](int row, int col, int k) {
        a.z_top[(int64_t)(m0 + row) * a.K + k] = table[row * 128 + (col & 127)];
      });
      __syncthreads();
    }
    // per row: the sum outside the ids (TEMP: and of all columns at temperature 1) over the wave's 64 columns
    Sum2* red = reinterpret_cast<Sum2*>(lds);          // [4][256]
    Sum2* red1 = reinterpret_cast<Sum2*>(lds) + 1024;  // [4][256]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sr[16], sr1[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int lr = wm + 32 * i + mm::acc_row(r, lane);
        const uint2 mask = *reinterpret_cast<const uint2*>(&s.mask[lr][wn >> 5]);
        const int tcol = s.target[lr];
        float v[2], y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int lc = wn + 32 * j + (lane & 31);
          if (lc == tcol) a.z_target[m0 + lr] = acc[i][j][r];
          y[j] = n0 + lc < end ? acc[i][j][r] : ninf();
          v[j] = ((j ? mask.y : mask.x) >> (lane & 31)) & 1u ? ninf() : y[j];
        }
        const float n = ref_for(half_max(fmaxf(v[0], v[1])), a.c);
        sr[r] = exp2_hw(__builtin_fmaf(v[0], a.c, -n)) + exp2_hw(__builtin_fmaf(v[1], a.c, -n));
        if ((lane & 31) == 0) red[(wn >> 6) * 256 + lr].n = n;
        if (TEMP) {
          const float n1 = ref_for(half_max(fmaxf(y[0], y[1])), kLog2e);
          sr1[r] = exp2_hw(__builtin_fmaf(y[0], kLog2e, -n1)) + exp2_hw(__builtin_fmaf(y[1], kLog2e, -n1));
          if ((lane & 31) == 0) red1[(wn >> 6) * 256 + lr].n = n1;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const int lr = wm + 32 * i + mm::acc_row(xsum_row(lane & 31), lane);
      red[(wn >> 6) * 256 + lr].s = xsum16(sr, lane);
      if (TEMP) red1[(wn >> 6) * 256 + lr].s = xsum16(sr1, lane);
    }
    __syncthreads();
    const int m = m0 + tid;
    if (tid < 256 && m < a.rows) {
      Sum2 f = red[tid], f1 = red1[tid];
      for (int w = 1; w < 4; ++w) {
        add_sum2(f, red[w * 256 + tid]);
        if (TEMP) add_sum2(f1, red1[w * 256 + tid]);
      }
      float* o = a.parts + ((int64_t)m * a.tiles_n + tn) * (TEMP ? 4 : 2);
      *reinterpret_cast<float2*>(o) = make_float2(f.n, f.s);
      if (TEMP) *reinterpret_cast<float2*>(o + 2) = make_float2(f1.n, f1.s);
    }
  } else {
    // every column as one outside the ids, staged in bf16
    uint16_t* stage = reinterpret_cast<uint16_t*>(lds);  // [256][kStagePitch]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int lr = wm + 32 * i + mm::acc_row(r, lane);
        const float4 p = s.p[lr];
        RowGrad g;
        g.out = p.x; g.nr = p.y;
        if (TEMP) { g.n1 = p.z; g.kce = p.w; }
        const uint32_t two = pack_bf16x2(grad_outside<TEMP>(g, acc[i][0][r], a.c), grad_outside<TEMP>(g, acc[i][1][r], a.c));
        stage[lr * kStagePitch + wn + (lane & 31)] = (uint16_t)two;
        stage[lr * kStagePitch + wn + 32 + (lane & 31)] = (uint16_t)(two >> 16);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
    // the target, then the ids (one of them may be the target), from their logits as the first pass left them
    auto row_of = [&](int row) {
      const float4 p = s.p[row];
      const float2 n = s.p_named[row];
      return RowGrad{p.w, n.x, p.z, n.y, p.y, p.x};
    };
    if (tid < 256) {
      const int col = s.target[tid];
      if (col >= 0) {
        const RowGrad g = row_of(tid);
        const float o = grad_outside<TEMP>(g, a.z_target[m0 + tid], a.c) - g.kce;
        stage[tid * kStagePitch + col] = (uint16_t)pack_bf16x2(o, 0.0f);
      }
    }
    __syncthreads();
    for (int h = 0; h < 2; ++h) {
      for_entries(s, a, m0, n0, h, [&](int row, int col, int k) {
        const int64_t at = (int64_t)(m0 + row) * a.K + k;
        const RowGrad g = row_of(row);
        float o = grad_named(g, a.z_top[at], a.c, a.q[at]);
        if (col == s.target[row]) o -= g.kce;
        stage[row * kStagePitch + col] = (uint16_t)pack_bf16x2(o, 0.0f);
      });
    }
    __syncthreads();
    // 256 rows of 512 bytes: 32 threads a row, 16 bytes each; 0 behind the vocabulary's end
    const int c = (tid & 31) * 8;
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
      const int row = (tid >> 5) + 16 * k, m = m0 + row;
      if (m >= a.rows) continue;
      uint4 v = *reinterpret_cast<const uint4*>(stage + row * kStagePitch + c);
      if (s.target[row] == kNanRow) v.x = v.y = v.z = v.w = (uint32_t)kQNaN16 * 0x10001u;
      if (s.target[row] == kZeroRow) v = make_uint4(0u, 0u, 0u, 0u);
      if (n0 + 256 > end) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n0 + c + e >= end) w[e >> 1] &= (e & 1) ? 0xffffu : 0xffff0000u;
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(a.g + (int64_t)m * a.ldg + tn * 256 + c) = v;
    }
  }
}

// ------------------------------------------------------------------ rows

// The ids with what is left out made -1.
__global__ __launch_bounds__(256) void kd_ids_kernel(KdLoss l, int64_t total, int32_t* ids) {
  for (int64_t i = (int64_t)bid_x() * 256 + tid_x(); i < total; i += (int64_t)nblocks_x() * 256) {
    const int v = l.ids[i];
    ids[i] = v < 0 || v >= l.V || l.top[i] < kMasked ? -1 : v;
  }
}

struct RowsArgs {
  KdLoss l;
  KdGrad g;
  double c;
  int tiles_n;
  const float *parts, *z_top, *z_target;
  float* q;         // [BT][K] or nullptr (no gradients)
  int32_t* ids;     // [BT][K]: cleaned; a token's entries behind its first leave it with gradients
  RowParam* param;  // [BT] or nullptr (no gradients)
};

// A wave a row: joins the tiles' sums, lane by lane and then the lanes; writes the row's results and what the second
// pass needs of it.
template <bool TEMP>
__global__ __launch_bounds__(64) void kd_rows_kernel(RowsArgs a) {
  __shared__ Entries en;
  const KdLoss& l = a.l;
  const int64_t r = large_bid();
  if (r >= l.BT) return;
  const int lane = tid_x(), K = (int)l.K;
  const int64_t t = l.target[r];
  const float none = 1.0e30f;  // 2^(c z - none) is 0
  RowParam p{RowGrad{0.0f, 0.0f, none, none, none, 0.0f}, kZeroRow};
  if (t == l.ignore_index) {
    if (lane == 0) {
      store_row(l, r, RowResult{});
      if (a.param) a.param[r] = p;
    }
    if (a.param)
      for (int j = lane; j < K; j += 64) a.ids[r * K + j] = -1;
    return;
  }
  bool bad_any = false;
  for (int j = lane; j < K; j += 64) {
    float u;
    bool bad;
    const int v = entry_id(l, r, j, u, bad);
    bad_any |= bad;
    en.id[j] = v;
    en.u[j] = u;
    en.z[j] = v >= 0 ? a.z_top[r * K + j] : ninf();
  }
  const float zt = t >= 0 && t < l.V ? a.z_target[r] : 0.0f;
  Sum2d s{floor_of((float)a.c), 0.0}, s1{floor_of(kLog2e), 0.0};
  const float* parts = a.parts + r * a.tiles_n * (TEMP ? 4 : 2);
  for (int k = lane; k < a.tiles_n; k += 64) {
    const float2 w = *reinterpret_cast<const float2*>(parts + k * (TEMP ? 4 : 2));
    add_sum2d(s, Sum2d{w.x, w.y});
    if (TEMP) {
      const float2 w1 = *reinterpret_cast<const float2*>(parts + k * 4 + 2);
      add_sum2d(s1, Sum2d{w1.x, w1.y});
    }
  }
  s = wave_sum2d(s);
  if (TEMP) s1 = wave_sum2d(s1);
  __syncthreads();
  double q[kLaneTop];
  const RowResult o = finish_row<TEMP>(l, r, en, __any(bad_any), t, zt, a.c, s, s1, q);
  if (lane == 0) store_row(l, r, o);
  if (!a.param) return;
#pragma unroll
  for (int k = 0; k < kLaneTop; ++k) {
    const int j = lane + 64 * k;
    if (j < K) {
      // a token's masses in the order of its entries, at the first of them
      float sum = 0.0f;
      if (en.id[j] >= 0 && !named_before(en.id, j)) {
        for (int i = j; i < K; ++i)
          if (en.id[i] == en.id[j]) sum += exp2_hw((float)((double)en.u[i] * a.c - (double)o.norm * kLog2e64));
      }
      a.q[r * K + j] = sum;
      if (en.id[j] >= 0 && named_before(en.id, j)) a.ids[r * K + j] = -1;
    }
  }
  if (lane == 0) {
    if (o.lse != ninf()) p.g = row_grad<TEMP>(a.g, l, r, o.lse, o.lse_t, o.lse_rest, o.off);
    p.target = o.bad || t < 0 || t >= l.V ? kNanRow : o.lse == ninf() ? kZeroRow : (int)t;
    a.param[r] = p;
  }
}

// grad_x from its fp32 sum.
__global__ __launch_bounds__(256) void kd_round_kernel(const float* __restrict__ from, uint16_t* __restrict__ to,
                                                       int64_t groups) {
  for (int64_t i = (int64_t)bid_x() * 256 + tid_x(); i < groups; i += (int64_t)nblocks_x() * 256) {
    float x[8];
    load8(from + 8 * i, x);
    store8(to + 8 * i, x);
  }
}

__global__ __launch_bounds__(256) void kd_zero_kernel(uint4* p, int64_t units) {
  for (int64_t i = (int64_t)bid_x() * 256 + tid_x(); i < units; i += (int64_t)nblocks_x() * 256)
    p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ workspace

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

struct Ws {
  float *parts, *z_top, *z_target, *q, *gx, *gx_parts;
  int32_t* ids;
  RowParam* param;
  uint16_t* g;
  int64_t ldg;
  int splits;
  size_t bytes;
};

// Splits of grad_x's product over a piece: few tiles would leave compute units idle through it (64 x 32000 x 4096 whole
// call 833 us without, 353 with; 300 x 2000 x 576 112 and 90; 512 x 151936 x 4096 5.0 and 2.6 ms).
int splits_of(int64_t BT, int64_t H, int64_t piece) {
  const int64_t tiles = ((BT + 255) / 256) * ((H + 255) / 256);
  int64_t s = (256 + tiles - 1) / tiles;
  if (s > 16) s = 16;
  if (s > piece / 512) s = piece / 512;
  return s < 1 ? 1 : (int)s;
}

Ws workspace(void* base, int64_t BT, int64_t V, int64_t H, int64_t K, int64_t piece, bool grads) {
  Ws w{};
  size_t off = 0;
  char* p = static_cast<char*>(base);
  auto take = [&](int64_t bytes) {
    char* q = p ? p + off : nullptr;
    off += align256((size_t)bytes);
    return q;
  };
  const int64_t tiles_n = (V + 255) / 256;
  w.parts = reinterpret_cast<float*>(take(BT * tiles_n * 16));
  w.z_target = reinterpret_cast<float*>(take(BT * 4));
  w.z_top = reinterpret_cast<float*>(take(BT * K * 4));
  w.ids = reinterpret_cast<int32_t*>(take(BT * K * 4));
  if (grads) {
    w.q = reinterpret_cast<float*>(take(BT * K * 4));
    w.param = reinterpret_cast<RowParam*>(take(BT * (int64_t)sizeof(RowParam)));
    w.ldg = ((piece < V ? piece : V) + 255) / 256 * 256;
    w.g = reinterpret_cast<uint16_t*>(take(BT * w.ldg * 2));
    w.gx = reinterpret_cast<float*>(take(BT * H * 4));
    w.splits = splits_of(BT, H, w.ldg);
    if (w.splits > 1) w.gx_parts = reinterpret_cast<float*>(take(w.splits * BT * H * 4));
  }
  w.bytes = off;
  return w;
}

template <bool TEMP>
hipError_t run(const KdLinearArgs& a, hipStream_t st) {
  const KdLoss& l = a.l;
  const bool grads = a.grad_x || a.grad_w;
  const int64_t piece = ((a.piece < l.V ? a.piece : l.V) + 255) / 256 * 256;
  const Ws w = workspace(a.workspace, l.BT, l.V, a.H, l.K, piece, grads);
  const double c64 = scale_of(l.temperature);
  hipError_t e;
  (void)hipGetLastError();
  if (l.K) {
    const int64_t total = l.BT * l.K, blocks = (total + 255) / 256;
    kd_ids_kernel<<<dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st>>>(l, total, w.ids);
    if ((e = hipGetLastError())) return e;
  }
  TileArgs t{};
  t.x = a.x; t.w = a.w; t.H = a.H; t.rows = (int)l.BT; t.V = (int)l.V; t.first = 0; t.width = (int)l.V;
  t.ids = w.ids; t.K = (int)l.K; t.c = (float)c64; t.target = l.target; t.ignore_index = l.ignore_index;
  t.tiles_m = (int)((l.BT + mm::kBM - 1) / mm::kBM);
  t.tiles_n = (int)((l.V + 255) / 256);
  t.parts = w.parts; t.z_top = w.z_top; t.z_target = w.z_target;
  kd_tile_kernel<false, TEMP><<<dim3(mm::grid_for(t.tiles_m, t.tiles_n)), dim3(kWideThreads), 0, st>>>(t);
  if ((e = hipGetLastError())) return e;
  RowsArgs r{};
  r.l = l; r.g = a.g; r.c = c64; r.tiles_n = t.tiles_n;
  r.parts = w.parts; r.z_top = w.z_top; r.z_target = w.z_target; r.q = w.q; r.ids = w.ids; r.param = w.param;
  kd_rows_kernel<TEMP><<<large_grid(l.BT), dim3(64), 0, st>>>(r);
  if ((e = hipGetLastError())) return e;
  if (!grads) return hipSuccess;
  t.param = w.param; t.q = w.q; t.g = w.g; t.ldg = w.ldg;
  const bool bf16 = a.grad_dt == Dt::BF16;
  float* gx = bf16 ? w.gx : static_cast<float*>(a.grad_x);
  for (int64_t first = 0; first < l.V; first += piece) {
    const int64_t width = l.V - first < piece ? l.V - first : piece, wide = (width + 7) / 8 * 8;
    t.first = (int)first; t.width = (int)width;
    t.tiles_n = (int)((width + 255) / 256);
    kd_tile_kernel<true, TEMP><<<dim3(mm::grid_for(t.tiles_m, t.tiles_n)), dim3(kWideThreads), 0, st>>>(t);
    if ((e = hipGetLastError())) return e;
    if (a.grad_x) {  // += G w[piece]: K = width, w read down its columns; G's columns behind the vocabulary are 0
      GemmArgs p{w.g, w.ldg, a.w + first * a.H, a.H, gx, a.H, l.BT, a.H, wide, true, false, first > 0};
      p.splits = w.splits; p.partials = w.gx_parts;
      p.b_end = 2 * width * a.H;
      if ((e = launch_gemm_bf16(p, st))) return e;
    }
    if (a.grad_w) {  // = G^T x: M = width, K = BT, both read down their columns
      char* to = static_cast<char*>(a.grad_w) + first * a.H * (bf16 ? 2 : 4);
      GemmArgs p{w.g, w.ldg, a.x, a.H, reinterpret_cast<float*>(to), a.H, width, a.H, l.BT, false, false, false};
      p.c_bf16 = bf16;
      p.a_end = 2 * l.BT * w.ldg;
      if ((e = launch_gemm_bf16(p, st))) return e;
    }
  }
  if (a.grad_x && bf16) {
    const int64_t groups = l.BT * a.H / 8, blocks = (groups + 255) / 256;
    kd_round_kernel<<<dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st>>>(
        gx, static_cast<uint16_t*>(a.grad_x), groups);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

size_t kd_linear_workspace_bytes(int64_t BT, int64_t V, int64_t H, int64_t K, int64_t piece, bool grads) {
  return BT <= 0 ? 0 : workspace(nullptr, BT, V, H, K, piece, grads).bytes;
}

hipError_t launch_kd_linear_zero(void* p, int64_t units, hipStream_t st) {
  const int64_t blocks = (units + 255) / 256;
  (void)hipGetLastError();
  kd_zero_kernel<<<dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st>>>(static_cast<uint4*>(p), units);
  return hipGetLastError();
}

hipError_t launch_kd_linear(const KdLinearArgs& a, hipStream_t st) {
  return a.l.temperature != 1.0f ? run<true>(a, st) : run<false>(a, st);
}

}  // namespace lx
