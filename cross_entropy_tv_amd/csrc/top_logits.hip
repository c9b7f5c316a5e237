// The K largest logits of every row, largest first and of equal ones the lowest id first, with the row's
// log-sum-exp and that of the logits outside the K.
//
// What bounds it: reading the logits once.  A workgroup passes over its columns in tiles of 32768 held in
// registers, with a threshold that at least K logits before it reach: only logits above it (a few K of a row,
// most of them in the first tile) enter a list in LDS, all others go into a sum of exponentials at once.  The
// list is settled at the end: a logit's rank is the number of larger ones in it.
//
//   threshold  the first tile's: the K-th largest of the threads' maxima, by a search over the upper 16 bits of
//              their ordered values (two bits a step: eight counts over the workgroup).  Later ones: the
//              same over the list.  Truncated to 16 bits it is still one that K logits reach; a later logit
//              has to exceed it (an equal one would have the higher id).
//   list       2048 keys (value, id).  Where a tile has more logits above the threshold than there is room (rows
//              of equal logits, rising rows), it is gone through again 1024 columns at a time, with the list
//              cut to the K largest whenever it fills.
//   the rest   a logit that has entered the list and leaves it joins the sum then, so that the
//              log-sum-exp of the rest is a sum of positive terms and no difference, good to fp32 relatively
//              however small the rest is.
//
// Few rows are cut into chunks, each chunk's K largest and sum left in the workspace, and a second kernel
// joins them.  Which logits enter a list depends on the data alone, and what is added up is added in the order of
// threads and ranks: the results do not depend on timing.
#include "common.hpp"
#include "distill.hpp"
#include "sum2.hpp"

namespace lx {

namespace {

constexpr int kTopThreads = 1024;
constexpr int kTopHeld = 4;  // groups of 8 a thread
constexpr int kTopTile = kTopThreads * 8 * kTopHeld;
constexpr int kTopList = 2048;
constexpr int kTopWaves = kTopThreads / 64;

// ------------------------------------------------------------------ keys

// Whole numbers in the order of the values (equal zeros made one).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
// larger value first, then lower id; 0: none
__device__ __forceinline__ uint64_t key_of(float x, uint32_t id) { return ((uint64_t)ordered(x) << 32) | (uint32_t)~id; }
__device__ __forceinline__ float key_value(uint64_t k) { return value_of((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_id(uint64_t k) { return (int)~(uint32_t)k; }

struct List {
  uint64_t keys[kTopList + 2];
  uint64_t sorted[kTopList];
  int n;
  int counts[8][3];
  Sum2 red[kTopWaves];
};

// The largest 16-bit prefix that at least K of the workgroup's values o (0: none) reach; 0 if there is none.
// Called by every thread, with counts zeroed and a barrier since; ends behind a barrier.
__device__ __forceinline__ uint32_t prefix_of(List& s, uint32_t o, int K) {
  const int lane = tid_x() & 63;
  const uint32_t mine = o >> 16;
  uint32_t p = 0;
  for (int step = 0; step < 8; ++step) {
    const int shift = 14 - 2 * step;
    int c[3];
#pragma unroll
    for (int d = 0; d < 3; ++d) c[d] = __popcll(__ballot(mine >= (p | ((uint32_t)(d + 1) << shift))));
    if (lane < 3) atomicAdd(&s.counts[step][lane], lane == 0 ? c[0] : lane == 1 ? c[1] : c[2]);
    __syncthreads();
    const int a = s.counts[step][0], b = s.counts[step][1], d = s.counts[step][2];
    p |= (uint32_t)(d >= K ? 3 : b >= K ? 2 : a >= K ? 1 : 0) << shift;
  }
  __syncthreads();
  return p;
}
__device__ __forceinline__ void zero_counts(List& s) {
  if (tid_x() < 24) s.counts[tid_x() / 3][tid_x() % 3] = 0;
}

// The smallest value that a logit has to reach where it has to exceed prefix p (0: any unmasked).
__device__ __forceinline__ float above(uint32_t p) {
  return p == 0u ? kMasked : fmaxf(kMasked, value_of((p << 16) + 1u));
}

// Sorts keys[0, n) into sorted[0, n), largest first.  Called by every thread behind a barrier; ends behind one.
__device__ __forceinline__ void rank_keys(List& s, int n) {
  const int tid = tid_x();
  if (tid < 2) s.keys[n + tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kTopThreads) {
    const uint64_t mine = s.keys[i];
    int r = 0;
    for (int j = 0; j < n; j += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(s.keys + j);
      r += (two.x > mine) + (two.y > mine);
    }
    s.sorted[r] = mine;
  }
  __syncthreads();
}

// Cuts the list to its K largest; those that leave join the sums.  Every thread, behind a barrier; ends behind one.
__device__ __forceinline__ int cut_list(List& s, int n, int K, float c, Sum2& a) {
  rank_keys(s, n);
  const int tid = tid_x(), keep = n < K ? n : K;
  for (int i = tid; i < n; i += kTopThreads) {
    if (i < K) s.keys[i] = s.sorted[i];
    else add_one(a, key_value(s.sorted[i]), c);
  }
  if (tid == 0) s.n = keep;
  __syncthreads();
  return keep;
}

// Sum over the workgroup in the order of the waves; valid in every thread of wave 0.
__device__ __forceinline__ Sum2 block_sum2(List& s, Sum2 a) {
  a = wave_sum2(a);
  if ((tid_x() & 63) == 0) s.red[tid_x() >> 6] = a;
  __syncthreads();
  Sum2 f = s.red[0];
  for (int w = 1; w < kTopWaves; ++w) add_sum2(f, s.red[w]);
  return f;
}

// The row's outputs from its sorted keys (n of them, at most K) and the sum of the rest.
__device__ __forceinline__ void write_row(const TopArgs& g, int64_t r, const uint64_t* sorted, int n, double c64,
                                          const Sum2& rest) {
  const int tid = tid_x(), K = (int)g.K;
  if (tid < K) {
    const uint64_t k = tid < n ? sorted[tid] : 0;
    g.top[r * K + tid] = k ? key_value(k) : ninf();
    g.ids[r * K + tid] = k ? key_id(k) : -1;
  }
  if (tid >= 64 || (!g.lse && !g.rest)) return;
  const double lr = log2_of(rest);
  const double first = n > 0 ? (double)key_value(sorted[0]) * c64 : -kInf64;
  const double ref = __builtin_fmax(first, lr);
  double s = 0.0;
  if (n > 0) {
    for (int j = tid; j < n; j += 64) s += exp2_64((double)key_value(sorted[j]) * c64 - ref);
  }
  s = wave_sum64(s);
  if (tid == 0) {
    const bool any = ref > -kInf64;
    if (g.lse) g.lse[r] = any ? (float)((ref + log2_64(s + exp2_64(lr - ref))) * kLn2) : ninf();
    if (g.rest) g.rest[r] = lr > -kInf64 ? (float)(lr * kLn2) : ninf();
  }
}

// ------------------------------------------------------------------ one pass

// One workgroup per (row, chunk of columns); with one chunk a row it writes the row's outputs, else
// the chunk's K largest keys (0 behind them) and its sum.
template <typename T>
__global__ __launch_bounds__(kTopThreads) void top_kernel(TopArgs g, double c64, int chunks, int64_t columns,
                                                          uint64_t* keys_out, Sum2* sums_out) {
  __shared__ List s;
  const int64_t tile = large_bid();
  const int64_t r = tile / chunks;
  if (r >= g.BT) return;
  const int tid = tid_x(), K = (int)g.K;
  const int64_t lo = (tile - r * chunks) * columns;
  const int64_t hi = g.V < lo + columns ? g.V : lo + columns;
  const T* row = static_cast<const T*>(g.z) + r * g.ldz;
  const float c = (float)c64;
  if (tid == 0) s.n = 0;
  Sum2 a{floor_of(c), 0.0f};
  float least = kMasked;  // a logit enters the list from here on
  int n = 0;
  for (int64_t b = lo; b < hi; b += kTopTile) {
    Group<T> h[kTopHeld];
    if (g.V >= 8) {
#pragma unroll
      for (int k = 0; k < kTopHeld; ++k) {
        const int64_t v = b + k * (kTopThreads * 8) + tid * 8;
        h[k].load(row + (v < g.V - 8 ? v : g.V - 8));
      }
    }
    auto get = [&](int k, float(&x)[8]) {
      const int64_t v = b + k * (kTopThreads * 8) + tid * 8;
      launder(h[k]);
      if (v + 8 <= hi) {
        h[k].get(x);
      } else {
        load_edge(row, v, hi, x);
      }
    };
    const int64_t end = hi < b + kTopTile ? hi : b + kTopTile;
    const bool last = end == hi;
    zero_counts(s);
    __syncthreads();
    if (b == lo && hi - lo > kTopList) {
      float m = ninf();
#pragma unroll
      for (int k = 0; k < kTopHeld; ++k) {
        float x[8];
        get(k, x);
        m = fmaxf(m, max8(x));
      }
      const uint32_t p = prefix_of(s, m < kMasked ? 0u : ordered(m), K);
      least = p == 0u ? kMasked : fmaxf(kMasked, value_of(p << 16));
      zero_counts(s);
    }
    // those below join the sums, those from `least` on the list
    const Sum2 before = a;
    float b0 = 0.0f, b1 = 0.0f;
#pragma unroll
    for (int k = 0; k < kTopHeld; ++k) {
      float x[8];
      get(k, x);
      const float m = max8(x);
      if (m >= least) {
        const uint32_t v = (uint32_t)(b + k * (kTopThreads * 8) + tid * 8);
        int count = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) count += x[e] >= least;
        int at = atomicAdd(&s.n, count);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (x[e] >= least) {
            if (at < kTopList) s.keys[at] = key_of(x[e], v + e);
            ++at;
            x[e] = ninf();
          }
        }
      }
      if (k == 0) {  // the thread's reference
        const float ref = fmaxf(a.n, ref_for(max8(x), c));
        a = Sum2{ref, a.s * exp2_hw(a.n - ref)};
      }
      sum8(x, c, a.n, b0, b1);
    }
    if (b0 + b1 >= kRefSumLimit) {  // again, against the true maximum
      float m = ninf();
#pragma unroll
      for (int k = 0; k < kTopHeld; ++k) {
        float x[8];
        get(k, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = x[e] >= least ? m : fmaxf(m, x[e]);
      }
      const float ref = fmaxf(a.n, ref_for(m, c));
      a = Sum2{ref, a.s * exp2_hw(a.n - ref)};
      b0 = b1 = 0.0f;
#pragma unroll
      for (int k = 0; k < kTopHeld; ++k) {
        float x[8];
        get(k, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] >= least ? ninf() : x[e];
        sum8(x, c, a.n, b0, b1);
      }
    }
    a.s += b0 + b1;
    __syncthreads();
    const int now = s.n;
    if (now > kTopList) {
      // too many at once: this tile again, 1024 columns at a time, against the K-th key of the list
      a = before;
      __syncthreads();
      n = cut_list(s, n, K, c, a);
      for (int64_t w = b; w < end; w += kTopThreads) {
        const uint64_t kth = n >= K ? s.keys[K - 1] : 0;
        const int64_t v = w + tid;
        const float x = v < end ? load1(row + v) : ninf();
        const uint64_t key = key_of(x, (uint32_t)v);
        if (x >= kMasked) {
          if (key > kth) s.keys[atomicAdd(&s.n, 1)] = key;
          else add_one(a, x, c);
        }
        __syncthreads();
        const int have = s.n;
        __syncthreads();
        n = cut_list(s, have, K, c, a);  // (in order: the last of K is the K-th)
      }
      if (n >= K) least = fmaxf(kMasked, value_of((uint32_t)(s.keys[K - 1] >> 32) + 1u));
      __syncthreads();
      continue;
    }
    n = now;
    if (!last) {
      if (n > kTopList / 2) {
        n = cut_list(s, n, K, c, a);
        if (n >= K) least = fmaxf(least, fmaxf(kMasked, value_of((uint32_t)(s.keys[K - 1] >> 32) + 1u)));
      } else if (n >= K) {
        const uint32_t p = prefix_of(s, tid < n ? (uint32_t)(s.keys[tid] >> 32) : 0u, K);
        least = fmaxf(least, above(p));
      }
    }
  }
  rank_keys(s, n);
  for (int i = tid; i < n; i += kTopThreads)
    if (i >= K) add_one(a, key_value(s.sorted[i]), c);
  const Sum2 rest = block_sum2(s, a);
  const int kept = n < K ? n : K;
  if (chunks == 1) {
    write_row(g, r, s.sorted, kept, c64, rest);
    return;
  }
  if (tid < K) keys_out[tile * K + tid] = tid < kept ? s.sorted[tid] : 0;
  if (tid == 0) sums_out[tile] = rest;
}

// ------------------------------------------------------------------ rows cut into chunks

// One workgroup a row: of the chunks' keys those that reach the largest of the chunks' K-th ones, ranked.
__global__ __launch_bounds__(kTopThreads) void top_join_kernel(TopArgs g, double c64, int chunks,
                                                               const uint64_t* __restrict__ keys,
                                                               const Sum2* __restrict__ sums) {
  __shared__ List s;
  __shared__ uint64_t kth[kTopWaves];
  const int64_t r = large_bid();
  if (r >= g.BT) return;
  const int tid = tid_x(), K = (int)g.K, total = chunks * K;
  const float c = (float)c64;
  const uint64_t* mine = keys + r * total;
  if (tid == 0) s.n = 0;
  uint64_t lower = 0;  // K keys reach it
  for (int i = tid; i < chunks; i += kTopThreads) {
    const uint64_t k = mine[i * K + K - 1];
    lower = k > lower ? k : lower;
  }
  lower = wave_all(lower, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
  if ((tid & 63) == 0) kth[tid >> 6] = lower;
  __syncthreads();
  lower = 0;
  for (int w = 0; w < kTopWaves; ++w) lower = kth[w] > lower ? kth[w] : lower;
  for (int i = tid; i < total; i += kTopThreads) {
    const uint64_t k = mine[i];
    if (k != 0 && k >= lower) s.keys[atomicAdd(&s.n, 1)] = k;
  }
  __syncthreads();
  const int n = s.n;
  rank_keys(s, n);
  const uint64_t last = n >= K ? s.sorted[K - 1] : 0;
  Sum2 a{floor_of(c), 0.0f};
  for (int i = tid; i < chunks; i += kTopThreads) add_sum2(a, sums[r * chunks + i]);
  for (int i = tid; i < total; i += kTopThreads) {
    const uint64_t k = mine[i];
    if (k != 0 && k < last) add_one(a, key_value(k), c);
  }
  const Sum2 rest = block_sum2(s, a);
  write_row(g, r, s.sorted, n < K ? n : K, c64, rest);
}

// Chunks of a row: about 256 workgroups, chunks of at least 2048 columns, and their keys within one list.
struct TopSplit {
  int64_t chunks, columns;
};
TopSplit top_split(int64_t BT, int64_t V, int64_t K) {
  int64_t s = (256 + BT - 1) / BT;
  if (BT >= 128) s = 1;
  if (s > kTopList / K) s = kTopList / K;
  if (s > V / 2048) s = V / 2048;
  if (s < 1) s = 1;
  const int64_t columns = ((V + s - 1) / s + 7) / 8 * 8;
  return TopSplit{(V + columns - 1) / columns, columns};
}

template <typename T>
hipError_t launch_top_t(const TopArgs& a, hipStream_t st) {
  const TopSplit s = top_split(a.BT, a.V, a.K);
  uint64_t* keys = static_cast<uint64_t*>(a.workspace);
  Sum2* sums = reinterpret_cast<Sum2*>(keys + a.BT * s.chunks * a.K);
  const double c64 = scale_of(a.temperature);
  (void)hipGetLastError();
  top_kernel<T><<<large_grid(a.BT * s.chunks), dim3(kTopThreads), 0, st>>>(a, c64, (int)s.chunks, s.columns, keys, sums);
  if (hipError_t e = hipGetLastError()) return e;
  if (s.chunks == 1) return hipSuccess;
  top_join_kernel<<<large_grid(a.BT), dim3(kTopThreads), 0, st>>>(a, c64, (int)s.chunks, keys, sums);
  return hipGetLastError();
}

}  // namespace

size_t top_workspace_bytes(int64_t BT, int64_t V, int64_t K) {
  if (BT <= 0) return 0;
  const TopSplit s = top_split(BT, V, K);
  if (s.chunks == 1) return 0;
  return ((size_t)(BT * s.chunks) * ((size_t)K * 8 + sizeof(Sum2)) + 255) & ~(size_t)255;
}

hipError_t launch_top(const TopArgs& a, Dt dt, hipStream_t st) {
  switch (dt) {
    case Dt::BF16: return launch_top_t<uint16_t>(a, st);
    case Dt::F16: return launch_top_t<_Float16>(a, st);
    default: return launch_top_t<float>(a, st);
  }
}

}  // namespace lx
