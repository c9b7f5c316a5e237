// Cross entropy and distillation from a teacher's top logits, over student logits: forward, backward
// and both in one pass.
//
// With p = softmax(z / T) and the teacher's q (kd_row.hpp), for the columns named by the teacher's ids
// and for all others
//
//   d kd / dz_v = (p_v - q_v) / T                               v among the ids
//               = e_v (p_r - q_r) / T,  e_v = exp(z_v / T - lse_rest)   v outside
//
// (e_v is p_v / p_r: formed from the outside's own log-sum it never divides by a p_r that has
// vanished), and ce's gradient p1_v - [v == t] is added, p1 = softmax(z).  At T = 1 p1_v = p_r e_v
// outside, so one exponential an element serves both.
//
// What bounds them: reading the logits once (forward), reading and writing them once (backward, one
// pass).  The ids are K of up to 10^5 columns; which groups of 8 hold one is a byte of a bit mask in LDS
// that each workgroup sets for its columns, read beside the group, so that a group without one (all but
// a few in a thousand) costs a compare.
//
// Sums of exponentials are taken against an integer exponent n per thread, sum 2^(c z - n): c z - n is
// one fused multiply-add with no rounding of the reference.
#include "common.hpp"
#include "distill.hpp"
#include "kd_row.hpp"
#include "sum2.hpp"

namespace lx {

namespace {

// ------------------------------------------------------------------ forward

// Rows of up to 2^18 columns are one workgroup's (its mask is 32 KB); 512 threads, H groups at once; three or
// four of them on a compute unit.  8192 x 151936 bf16: 366 us, 6.8 TB/s (T 2: 385); 64 x 262144 fp32,
// T 2: 17 us and 5 for the second launch.
constexpr int kFwdThreads = 512;
constexpr int kFwdHeld = 4;
constexpr int64_t kMaxChunk = 1 << 18;
constexpr int64_t kMinChunk = 8192;
constexpr int64_t kWantedChunks = 512;

// Chunks of a row.  A workgroup a row while there is one for every compute unit; fewer long rows are cut so that about
// 512 workgroups run, which a second launch joins (5 us).  Whole against cut: 1 x 151936 bf16 18.6 and 9.4 us, 40 of them
// 20.9 and 13.6, 127 21.5 and 17.4, 256 24.0 and 23.1; 64 x 262144 fp32 43 and 23, 256 51 and 58; 16 x 32000 bf16 9.3 and
// 9.9.
struct Split {
  int64_t chunks, columns;
};
Split split_of(int64_t BT, int64_t V) {
  int64_t s = (kWantedChunks + BT - 1) / BT;
  if (BT >= kWantedChunks / 2 || V < 4 * kMinChunk) s = 1;
  if (s > V / kMinChunk) s = V / kMinChunk;
  const int64_t fit = (V + kMaxChunk - 1) / kMaxChunk;
  if (s < fit) s = fit;
  if (s < 1) s = 1;
  constexpr int64_t unit = kFwdThreads * 8;
  const int64_t columns = ((V + s - 1) / s + unit - 1) / unit * unit;
  return Split{(V + columns - 1) / columns, columns};
}

// What a chunk leaves behind: the sums outside the ids, and of all its columns at temperature 1.
struct ChunkSums {
  Sum2d outside, whole;
};

// Outside-the-ids sums of the columns [lo, hi) of a row (and, TEMP, sums at temperature 1 of all of
// them), this thread's share.
template <typename T, bool TEMP, int NT, int H>
__device__ __forceinline__ void chunk_sums(const T* row, int64_t lo, int64_t hi, int64_t V, const uint8_t* mask,
                                           float c, Sum2& a, Sum2& a1) {
  a = Sum2{floor_of(c), 0.0f};
  a1 = Sum2{floor_of(kLog2e), 0.0f};
  const int count = (int)(hi - lo);
  row += lo;
  const int last = (int)(V - lo) - 8;  // the last whole group that may be read
  for (int b = tid_x() * 8; b < count; b += NT * 8 * H) {
    Group<T> g[H];
    if (last >= 0) {
#pragma unroll
      for (int k = 0; k < H; ++k) g[k].load_once(row + min(b + k * (NT * 8), last));
    }
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const int v = b + k * (NT * 8);
      if (v < count) {
        float x[8];
        if (v + 8 <= count) g[k].get(x);
        else load_edge(row, v, count, x);  // -inf behind the end
        if (TEMP) add_group(x, kLog2e, a1);
        leave_out_bits(mask[v >> 3], x);
        add_group(x, c, a);
      }
    }
  }
}

// One workgroup per (row, chunk).  A whole row (chunks == 1) is finished here; chunks leave their sums
// in parts [row][chunk].
template <typename T, bool TEMP>
__global__ __attribute__((amdgpu_flat_work_group_size(kFwdThreads, kFwdThreads), amdgpu_waves_per_eu(sizeof(T) == 4 ? 6 : 8)))
void kd_forward_kernel(KdLoss l, const T* __restrict__ z, int64_t ldz,
                                                                 double c64, int chunks, int64_t columns, ChunkSums* parts) {
  extern __shared__ uint32_t bits[];
  constexpr int W = kFwdThreads / 64;
  __shared__ Entries en;
  __shared__ Sum2d red[2][W];
  __shared__ int bad_any;
  const int64_t tile = large_bid();
  const int64_t r = tile / chunks;
  if (r >= l.BT) return;
  const int ch = (int)(tile - r * chunks), tid = tid_x();
  const int64_t t = l.target[r];
  if (t == l.ignore_index) {
    if (ch == 0 && tid == 0) store_row(l, r, RowResult{});
    return;
  }
  const int K = (int)l.K;
  const int64_t lo = ch * columns, hi = l.V < lo + columns ? l.V : lo + columns;
  const T* row = z + r * ldz;
  const float c = (float)c64;
  if (tid == 0) bad_any = 0;
  for (int w = tid; w < (int)(columns / 32); w += kFwdThreads) bits[w] = 0u;
  __syncthreads();
  float zj = ninf(), zt = 0.0f;
  if (tid < K) {
    float u;
    bool bad;
    const int v = entry_id(l, r, tid, u, bad);
    en.id[tid] = v;
    en.u[tid] = u;
    if (bad) bad_any = 1;
    if (v >= 0) {
      mark(bits, v, lo, hi);
      if (chunks == 1) zj = load1(row + v);
    }
  }
  if (chunks == 1 && tid == 0 && t >= 0 && t < l.V) zt = load1(row + t);
  __syncthreads();
  Sum2 a, a1;
  chunk_sums<T, TEMP, kFwdThreads, kFwdHeld>(row, lo, hi, l.V, reinterpret_cast<const uint8_t*>(bits), c, a, a1);
  Sum2d all = wave_sum2d(a), all1 = {};
  if (TEMP) all1 = wave_sum2d(a1);
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = all;
    red[1][tid >> 6] = all1;
  }
  if (tid < K) en.z[tid] = zj;
  __syncthreads();
  if (tid >= 64) return;
  all = red[0][0];
  all1 = red[1][0];
  for (int w = 1; w < W; ++w) {
    add_sum2d(all, red[0][w]);
    if (TEMP) add_sum2d(all1, red[1][w]);
  }
  if (chunks > 1) {
    if (tid == 0) parts[tile] = ChunkSums{all, all1};
    return;
  }
  double q[kLaneTop];
  const RowResult o = finish_row<TEMP>(l, r, en, bad_any != 0, t, zt, c64, all, all1, q);
  if (tid == 0) store_row(l, r, o);
}

// Rows cut into chunks: a wave a row joins its chunks' sums, lane by lane and then the lanes, in a fixed
// order.
template <typename T, bool TEMP>
__global__ __launch_bounds__(64) void kd_finish_kernel(KdLoss l, const T* __restrict__ z, int64_t ldz, double c64,
                                                       int chunks, const ChunkSums* __restrict__ parts) {
  __shared__ Entries en;
  const int64_t r = large_bid();
  if (r >= l.BT) return;
  const int64_t t = l.target[r];
  if (t == l.ignore_index) return;
  const int lane = tid_x(), K = (int)l.K;
  const T* row = z + r * ldz;
  bool bad_any = false;
  for (int j = lane; j < K; j += 64) {
    float u;
    bool bad;
    const int v = entry_id(l, r, j, u, bad);
    bad_any |= bad;
    en.id[j] = v;
    en.u[j] = u;
    en.z[j] = v >= 0 ? load1(row + v) : ninf();
  }
  const float zt = t >= 0 && t < l.V ? load1(row + t) : 0.0f;
  Sum2d a{floor_of((float)c64), 0.0}, a1{floor_of(kLog2e), 0.0};
  for (int k = lane; k < chunks; k += 64) {
    const ChunkSums p = parts[r * chunks + k];
    add_sum2d(a, p.outside);
    if (TEMP) add_sum2d(a1, p.whole);
  }
  a = wave_sum2d(a);
  if (TEMP) a1 = wave_sum2d(a1);
  __syncthreads();
  double q[kLaneTop];
  const RowResult o = finish_row<TEMP>(l, r, en, __any(bad_any), t, zt, c64, a, a1, q);
  if (lane == 0) store_row(l, r, o);
}

template <typename T, bool TEMP>
hipError_t launch_kd_forward_t(const KdArgs& a, double c64, hipStream_t st) {
  const Split s = split_of(a.l.BT, a.l.V);
  const T* z = static_cast<const T*>(a.z);
  ChunkSums* parts = static_cast<ChunkSums*>(a.workspace);
  (void)hipGetLastError();
  kd_forward_kernel<T, TEMP><<<large_grid(a.l.BT * s.chunks), dim3(kFwdThreads), (size_t)(s.columns / 8), st>>>(
      a.l, z, a.ldz, c64, (int)s.chunks, s.columns, parts);
  if (hipError_t e = hipGetLastError()) return e;
  if (s.chunks == 1) return hipSuccess;
  kd_finish_kernel<T, TEMP><<<large_grid(a.l.BT), dim3(64), 0, st>>>(a.l, z, a.ldz, c64, (int)s.chunks, parts);
  return hipGetLastError();
}

// ------------------------------------------------------------------ the gradient of a row's columns

// ------------------------------------------------------------------ backward

constexpr int kBwdThreads = 256;
constexpr int kBwdHeld = 2;
constexpr int kBwdColumns = kBwdThreads * 8 * kBwdHeld;

// One workgroup per (row, 4096 columns): short ones, of which eight a compute unit cover each other's chain of loads, mask
// and stores.  8192 x 151936 bf16 in 770 to 820 us (6.1 to 6.5 TB/s), 1024 x 151936 in 97.  The logits are requested first;
// the mask of the ids is made while they arrive.  Each thread reads a group before it writes it: the gradient may be the logits.
template <typename T, bool TEMP>
__global__ __launch_bounds__(kBwdThreads) void kd_backward_kernel(KdLoss l, KdGrad g, const T* z, int64_t ldz, T* grad,
                                                                  int64_t ldg, float c, int chunks) {
  __shared__ uint32_t bits[kBwdColumns / 32];
  __shared__ int id[kKdMaxTop];
  __shared__ float q[kKdMaxTop];
  __shared__ int bad_any, twice;
  const int64_t tile = large_bid();
  const int64_t r = tile / chunks;
  if (r >= l.BT) return;
  const int tid = tid_x(), K = (int)l.K;
  const int64_t lo = (tile - r * chunks) * kBwdColumns;
  const int64_t hi = l.V < lo + kBwdColumns ? l.V : lo + kBwdColumns;
  const T* row = z + r * ldz;
  T* out = grad + r * ldg;
  const int64_t t = l.target[r];
  const float lse = l.lse[r];
  const bool t_ok = t >= 0 && t < l.V;
  if (t == l.ignore_index || !t_ok || lse == ninf()) {
    const uint32_t fill = t == l.ignore_index || t_ok ? 0u : kQNaN32;
    for (int64_t v = lo + tid; v < hi; v += kBwdThreads) store_bits1(out + v, fill);
    return;
  }
  Group<T> gr[kBwdHeld];
  if (l.V >= 8) {
#pragma unroll
    for (int k = 0; k < kBwdHeld; ++k) {
      const int64_t v = lo + k * (kBwdThreads * 8) + tid * 8;
      gr[k].load_once(row + (v < l.V - 8 ? v : l.V - 8));
    }
  }
  const float4 state = *reinterpret_cast<const float4*>(l.state + kKdState * r);
  if (tid < kBwdColumns / 32) bits[tid] = 0u;
  if (tid == 0) bad_any = twice = 0;
  __syncthreads();
  if (tid < K) {
    float u;
    bool bad;
    const int v = entry_id(l, r, tid, u, bad);
    id[tid] = v;
    if (bad) bad_any = 1;
    if (mark(bits, v, lo, hi)) twice = 1;
    q[tid] = exp2_hw(__builtin_fmaf(u, c, -state.w * kLog2e));
  }
  const RowGrad rg = row_grad<TEMP>(g, l, r, lse, state.x, state.y, state.z);
  __syncthreads();
  const bool bad = bad_any != 0;
  if (twice) {  // a token's masses, in the order of its entries, at each of them
    float sum = 0.0f;
    if (tid < K)
      for (int i = 0; i < K; ++i) sum += id[i] == id[tid] ? q[i] : 0.0f;
    __syncthreads();
    if (tid < K) q[tid] = sum;
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < kBwdHeld; ++k) {
    const int at = k * (kBwdThreads * 8) + tid * 8;
    const int64_t v = lo + at;
    const uint32_t byte = v < hi ? reinterpret_cast<const uint8_t*>(bits)[at >> 3] : 0u;
    float x[8], o[8];
    if (v + 8 <= l.V) gr[k].get(x);
    else load_edge(row, v, l.V, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = grad_outside<TEMP>(rg, x[e], c);
    for_named(byte, (int)v, id, K, [&](int lane, int place, int j) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((tid & 63) == lane && e == place) o[e] = grad_named(rg, x[e], c, q[j]);
    });
    if (v >= hi) continue;
    const int64_t rel = t - v;
    if (rel >= 0 && rel < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = e == (int)rel ? o[e] - rg.kce : o[e];
    }
    if (bad) {
      for (int e = 0; e < 8 && v + e < l.V; ++e) store_bits1(out + v + e, kQNaN32);
    } else if (v + 8 <= l.V) {
      store8_any(out + v, o);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (v + e < l.V) store1(out + v + e, o[e]);
    }
  }
}

template <typename T, bool TEMP>
hipError_t launch_kd_backward_t(const KdArgs& a, double c64, hipStream_t st) {
  const int64_t chunks = (a.l.V + kBwdColumns - 1) / kBwdColumns;
  (void)hipGetLastError();
  kd_backward_kernel<T, TEMP><<<large_grid(a.l.BT * chunks), dim3(kBwdThreads), 0, st>>>(
      a.l, a.g, static_cast<const T*>(a.z), a.ldz, static_cast<T*>(a.grad), a.ldg, (float)c64, (int)chunks);
  return hipGetLastError();
}

}  // namespace

size_t kd_forward_workspace_bytes(int64_t BT, int64_t V) {
  if (BT <= 0 || V <= 0) return 0;
  const Split s = split_of(BT, V);
  return s.chunks == 1 ? 0 : ((size_t)(BT * s.chunks) * sizeof(ChunkSums) + 255) & ~(size_t)255;
}

#define LX_BY_TYPE(F, ...)                                                                     \
  const double c64 = scale_of(a.l.temperature);                                                \
  const bool temp = a.l.temperature != 1.0f;                                                   \
  switch (dt) {                                                                                \
    case Dt::BF16: return temp ? F<uint16_t, true>(a, c64, st) : F<uint16_t, false>(a, c64, st); \
    case Dt::F16: return temp ? F<_Float16, true>(a, c64, st) : F<_Float16, false>(a, c64, st);  \
    default: return temp ? F<float, true>(a, c64, st) : F<float, false>(a, c64, st);             \
  }

hipError_t launch_kd_forward(const KdArgs& a, Dt dt, hipStream_t st) { LX_BY_TYPE(launch_kd_forward_t) }
hipError_t launch_kd_backward(const KdArgs& a, Dt dt, hipStream_t st) { LX_BY_TYPE(launch_kd_backward_t) }

}  // namespace lx
