// The K largest logits of every row, largest first and of equal ones the lowest id first, with the row's
// log-sum-exp and that of the logits outside the K.
//
// What bounds it: reading the logits once.  A workgroup passes over its columns in tiles held in registers, with a
// threshold that at least K logits before it reach: only logits above it (a few K of a row, most of them in the first
// tile) enter a list in LDS, all others go into a sum of exponentials at once.  The list is settled at the end: a
// logit's rank is the number of larger ones in it.
//
//   threshold  the first tile's: the K-th largest of maxima over a few threads' logits each, by a search over the
//              upper 16 bits of their ordered values (one wave, a bit a step).  Later ones: the same over the list.
//              Truncated to 16 bits it is still one that K logits reach; a later logit has to
//              exceed it (an equal one would have the higher id).
//   the list   1024 keys (value, id), cut to those that reach the K-th behind each tile.  A thread marks its groups of
//              8 that reach the threshold and goes on; they are loaded again behind the tile, shared out among all
//              threads (a wave meets one at two groups of three, and would spend as much on them where it meets them as
//              on the sums).  Where a tile has more logits above the threshold than there is room it is gone
//              through again in smaller tiles, and where a part of one still has (rows of equal logits, rising
//              rows), 256 columns at a time, with the list cut to the K largest each time.
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

// A row's sums cost 47 vector instructions a group of 8 and wave, what ends a tile some hundred a wave: four waves a row
// pay that half as often as eight (8192 x 151936 bf16, K 64: 505-540 us against 640-680; the loss's forward over the same
// logits, without the selection, takes 366).
constexpr int kTopThreads = 256;
constexpr int kTopWaves = kTopThreads / 64;
constexpr int kTopList = 1024;
constexpr int kTopWaveList = 320;  // what a wave finds in a tile
constexpr int kTopHeld = 4;   // groups of 8 a thread holds,
constexpr int kTopPart = kTopThreads * 8 * kTopHeld;
constexpr int kTopMarked = 1024;  // marked groups of a tile
// Parts of a tile.  The first part's threshold serves the whole first tile and lets 34 logits of a part pass for K = 32, 74
// for 64, 137 for 128, 295 for 256 (of logits in any order; give or take K^(-1/2) of them): so many parts as the list and
// the waves' shares of it hold three deviations of.
__device__ __forceinline__ int tile_parts(int K) { return K <= 32 ? 16 : K <= 64 ? 10 : K <= 128 ? 5 : 2; }
// Rows cut into chunks: their keys, and the workgroup that joins them.
constexpr int kJoinThreads = 512;
constexpr int kJoinList = 2048;

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

template <int NT, int LIST>
struct List {
  alignas(16) uint64_t keys[LIST + 8];  // (zeros behind the last are ranked along)
  // in a tile: kTopWaveList of each wave
  alignas(16) uint64_t sorted[LIST > kTopWaves * kTopWaveList ? LIST : kTopWaves * kTopWaveList];
  int n;
  int found[NT / 64];
  uint32_t prefix;
  union {
    uint32_t maxima[4 * NT];
    uint16_t marked[kTopMarked];
  };
  Sum2 red[NT / 64];
};
typedef List<kTopThreads, kTopList> TopList;
typedef List<kJoinThreads, kJoinList> JoinList;

// Inclusive sum over the lanes.
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned dpp_shift(unsigned v) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}
__device__ __forceinline__ unsigned wave_scan(unsigned v) {
  v += dpp_shift<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8 (0 comes in)
  v += dpp_shift<0x112, 0xF>(v);
  v += dpp_shift<0x114, 0xF>(v);
  v += dpp_shift<0x118, 0xF>(v);
  v += dpp_shift<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
  v += dpp_shift<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
  return v;
}

// One wave: the largest 16-bit prefix that at least K of the lanes' R values each (ordered; 0: none) reach; 0 if there is
// none.
template <int R>
__device__ __forceinline__ uint32_t prefix_of(const uint32_t (&o)[R], int K) {
  uint32_t p = 0;
  for (int bit = 15; bit >= 0; --bit) {
    const uint32_t c = (p | 1u << bit) << 16;
    int n = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) n += __popcll(__ballot(o[k] >= c));
    if (n >= K) p |= 1u << bit;
  }
  return p;
}

// The smallest value that a logit has to reach to exceed prefix p (0: any unmasked).
__device__ __forceinline__ float above(uint32_t p) {
  return p == 0u ? kMasked : fmaxf(kMasked, value_of((p << 16) + 1u));
}

// Sorts keys[0, n) into sorted[0, n), largest first.  Called by every thread behind a barrier; ends behind one.
template <int NT, int LIST>
__device__ __forceinline__ void rank_keys(List<NT, LIST>& s, int n) {
  const int tid = tid_x();
  if (tid < 8) s.keys[n + tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const uint64_t mine = s.keys[i];
    int r = 0;
    for (int j = 0; j < n; j += 8) {  // (all read at once: every lane reads the same)
      ulonglong2 two[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) two[k] = reinterpret_cast<const ulonglong2*>(s.keys + j)[k];
#pragma unroll
      for (int k = 0; k < 4; ++k) r += (two[k].x > mine) + (two[k].y > mine);
    }
    s.sorted[r] = mine;
  }
  __syncthreads();
}

// Cuts the list to its K largest; those that leave join the sums.  Every thread, behind a barrier; ends behind one.
__device__ __forceinline__ int cut_list(TopList& s, int n, int K, float c, Sum2& a) {
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

// Wave 0: prefix_of the upper halves of the list's first 64 R keys.
template <int R>
__device__ __forceinline__ uint32_t list_prefix(const TopList& s, int n, int K) {
  const int lane = tid_x();
  uint32_t o[R];
#pragma unroll
  for (int k = 0; k < R; ++k) o[k] = lane + 64 * k < n ? (uint32_t)(s.keys[lane + 64 * k] >> 32) : 0u;
  return prefix_of(o, K);
}

// Cuts the list to the keys that reach its K-th largest value in 16 bits, in their order; those that leave join the
// sums.  That value's prefix goes to p (0: fewer than K).  Every thread, behind a barrier; ends behind one.
__device__ __forceinline__ int prune_list(TopList& s, int n, int K, float c, Sum2& a, uint32_t& p) {
  constexpr int kEach = kTopList / kTopThreads;
  const int tid = tid_x(), wave = tid >> 6, lane = tid & 63;
  if (tid < 64) {
    const uint32_t q = n <= 256 ? list_prefix<4>(s, n, K) : list_prefix<kTopList / 64>(s, n, K);
    if (tid == 0) s.prefix = q;
  }
  uint64_t mine[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) mine[k] = tid + k * kTopThreads < n ? s.keys[tid + k * kTopThreads] : 0;
  __syncthreads();
  p = s.prefix;
  int total = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (k * kTopThreads >= n) break;
    const bool stays = mine[k] != 0 && (uint32_t)(mine[k] >> 48) >= p;
    if (mine[k] != 0 && !stays) add_one(a, key_value(mine[k]), c);
    const uint64_t all = __ballot(stays);
    if (lane == 0) s.found[wave] = __popcll(all);
    __syncthreads();
    int at = total + __popcll(all & ((1ull << lane) - 1));
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w) {
      at += w < wave ? s.found[w] : 0;
      total += s.found[w];
    }
    if (stays) s.keys[at] = mine[k];
    __syncthreads();
  }
  return total;
}

// Sum over the workgroup in the order of the waves; valid in every thread of wave 0.
template <int NT, int LIST>
__device__ __forceinline__ Sum2 block_sum2(List<NT, LIST>& s, Sum2 a) {
  a = wave_sum2(a);
  if ((tid_x() & 63) == 0) s.red[tid_x() >> 6] = a;
  __syncthreads();
  Sum2 f = s.red[0];
  for (int w = 1; w < NT / 64; ++w) add_sum2(f, s.red[w]);
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
__global__ __attribute__((amdgpu_flat_work_group_size(kTopThreads, kTopThreads), amdgpu_waves_per_eu(6)))
void top_kernel(TopArgs g, double c64, int chunks, int64_t columns, uint64_t* keys_out, Sum2* sums_out) {
  constexpr int H = kTopHeld;
  __shared__ TopList s;
  const int64_t tile = large_bid();
  const int64_t r = tile / chunks;
  if (r >= g.BT) return;
  const int tid = tid_x(), lane = tid & 63, wave = tid >> 6, K = (int)g.K;
  const int64_t first = (tile - r * chunks) * columns;
  const T* row = static_cast<const T*>(g.z) + r * g.ldz + first;  // columns are counted from the chunk's first
  const int count = (int)(g.V < first + columns ? g.V - first : columns);
  const int whole = (int)(g.V - first) - 8;  // the last whole group that may be read (< 0: none)
  const float c = (float)c64;
  if (tid == 0) s.n = 0;
  Sum2 a{floor_of(c), 0.0f};
  float least = kMasked;  // a logit enters the list from here on
  int n = 0;
  uint32_t p = 0;
  // (a chunk's columns are a multiple of 8 but for the row's last, so that a group past its end is past it whole)
  auto only_mine = [&](int v, float(&x)[8]) {
    if (v + 8 > count) {
      const int d = v < count ? v - whole : 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = e < d ? ninf() : x[e];
    }
  };
  int parts = tile_parts(K);
  for (int b = 0; b < count;) {
    const int size = parts * kTopPart;
    const Sum2 before = a;
    // A thread's k-th group (of the tile's) is columns v .. v + 7, read from v or, at the row's end, from `whole`, where
    // its first places are other groups' columns.
    auto place = [&](int k) { return b + (k * kTopThreads + tid) * 8; };
    uint64_t marked = 0;
    if (whole >= 0) {
      for (int part = 0; part < parts && b + part * kTopPart < count; ++part) {
        Group<T> h[H];
#pragma unroll
        for (int k = 0; k < H; ++k) h[k].load_once(row + min(place(part * H + k), whole));
        auto get = [&](int k, float(&x)[8]) {
          launder(h[k]);
          h[k].get(x);
          only_mine(place(part * H + k), x);
        };
        if (b == 0 && part == 0 && count > kTopThreads) {
          // maxima over some more sets of logits than K, so that few logits more than K reach the K-th of them
          float all = ninf();
#pragma unroll
          for (int k = 0; k < H; ++k) {
            float x[8];
            get(k, x);
            const float m = max8(x);
            all = fmaxf(all, m);
            if (K > 64) s.maxima[k * kTopThreads + tid] = m < kMasked ? 0u : ordered(m);
          }
          if (K <= 64) s.maxima[tid] = all < kMasked ? 0u : ordered(all);
          __syncthreads();
          if (tid < 64) {
            uint32_t q;
            if (K <= 64) {
              uint32_t o[kTopWaves];
#pragma unroll
              for (int k = 0; k < kTopWaves; ++k) o[k] = s.maxima[tid + 64 * k];
              q = prefix_of(o, K);
            } else {
              uint32_t o[4 * kTopWaves];
#pragma unroll
              for (int k = 0; k < 4 * kTopWaves; ++k) o[k] = s.maxima[tid + 64 * k];
              q = prefix_of(o, K);
            }
            if (tid == 0) s.prefix = q;
          }
          __syncthreads();
          p = s.prefix;
          least = p == 0u ? kMasked : fmaxf(kMasked, value_of(p << 16));
        }
        // those below join the sums; groups with one from `least` on are marked
#pragma unroll
        for (int k = 0; k < H; ++k) {
          float x[8];
          get(k, x);
          if (max8(x) >= least) marked |= 1ull << (part * H + k);
          else add_group(x, c, a);
        }
      }
    }
    // the marked groups, in the order of threads and parts
    const int own = __popcll(marked), upto = (int)wave_scan((unsigned)own);
    if (lane == 63) s.found[wave] = upto;
    __syncthreads();
    int at = upto - own, groups = 0;
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w) {
      at += w < wave ? s.found[w] : 0;
      groups += s.found[w];
    }
    bool room = whole >= 0 && groups <= kTopMarked;
    if (room) {
      while (marked) {
        s.marked[at++] = (uint16_t)(__builtin_ctzll(marked) * kTopThreads + tid);
        marked &= marked - 1;
      }
    }
    __syncthreads();
    // their logits from `least` on, in the order of the groups
    int found = 0;  // (of the wave)
    if (room) {
      const int share = (groups + kTopWaves - 1) / kTopWaves, until = min(groups, (wave + 1) * share);
      for (int i = wave * share; i < until; i += 64) {
        float x[8];
        int from = 0;
        uint32_t high = 0;
        if (i + lane < until) {
          const int v = b + s.marked[i + lane] * 8;
          from = min(v, whole);
          Group<T> again;
          again.load(row + from);
          again.get(x);
          only_mine(v, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) high |= x[e] >= least ? 1u << e : 0u;
        }
        const int some = __popc(high);
        const int sum = (int)wave_scan((unsigned)some);
        int to = found + sum - some;
        found += __builtin_amdgcn_readlane(sum, 63);
        uint32_t left = high;
        while (left) {  // (mostly one)
          const int e = __builtin_ctz(left);
          left &= left - 1;
          float y = x[0];
#pragma unroll
          for (int k = 1; k < 8; ++k) y = k == e ? x[k] : y;
          if (to < kTopWaveList) s.sorted[wave * kTopWaveList + to] = key_of(y, (uint32_t)(first + from + e));
          ++to;
        }
        if (high) {
          leave_out_bits(high, x);
          add_group(x, c, a);
        }
      }
    }
    if (lane == 0) s.found[wave] = found;
    __syncthreads();
    int now = n;
    at = n;
#pragma unroll
    for (int w = 0; w < kTopWaves; ++w) {
      const int f = s.found[w];
      room = room && f <= kTopWaveList;
      at += w < wave ? f : 0;
      now += f;
    }
    if ((!room || now > kTopList) && parts > 1 && whole >= 0) {  // (by chance, or the logits rise): a part at a time
      a = before;
      parts = 1;
      __syncthreads();
      continue;
    }
    if (!room || now > kTopList) {
      // too many in a part (or a row of fewer than 8 columns): this tile again, 256 columns at a time, against the K-th
      // key of the list
      a = before;
      __syncthreads();
      n = cut_list(s, n, K, c, a);
      const int end = min(count, b + size);
      for (int w = b; w < end; w += kTopThreads) {
        const uint64_t kth = n >= K ? s.keys[K - 1] : 0;
        const int v = w + tid;
        const float x = v < end ? load1(row + v) : ninf();
        const uint64_t key = key_of(x, (uint32_t)(first + v));
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
      b += size;
      continue;
    }
    for (int i = lane; i < found; i += 64) s.keys[at + i] = s.sorted[wave * kTopWaveList + i];
    __syncthreads();
    n = now;
    if (n > K) {
      n = prune_list(s, n, K, c, a, p);
      least = fmaxf(least, above(p));
    }
    b += size;
    parts = tile_parts(K);
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

// One workgroup a row: of the chunks' keys those that reach a value that K of them do, ranked.
__global__ __launch_bounds__(kJoinThreads) void top_join_kernel(TopArgs g, double c64, int chunks,
                                                               const uint64_t* __restrict__ keys,
                                                               const Sum2* __restrict__ sums) {
  __shared__ JoinList s;
  const int64_t r = large_bid();
  if (r >= g.BT) return;
  const int tid = tid_x(), K = (int)g.K, total = chunks * K;
  const float c = (float)c64;
  const uint64_t* mine = keys + r * total;
  if (tid == 0) s.n = 0;
  // a value that K keys reach: the K-th of each chunk's first few, about twice K of them
  const int each = min(min(K, (2 * K + chunks - 1) / chunks), kJoinThreads / chunks);
  s.maxima[tid] = tid < chunks * each ? (uint32_t)(mine[(tid / each) * K + tid % each] >> 32) : 0u;
  __syncthreads();
  if (tid < 64) {
    uint32_t o[(kJoinThreads / 64)];
#pragma unroll
    for (int k = 0; k < (kJoinThreads / 64); ++k) o[k] = s.maxima[tid + 64 * k];
    const uint32_t p = prefix_of(o, K);
    if (tid == 0) s.prefix = p;
  }
  __syncthreads();
  const uint64_t lower = (uint64_t)s.prefix << 48;
  for (int i = tid; i < total; i += kJoinThreads) {
    const uint64_t k = mine[i];
    if (k != 0 && k >= lower) s.keys[atomicAdd(&s.n, 1)] = k;
  }
  __syncthreads();
  const int n = s.n;
  rank_keys(s, n);
  const uint64_t last = n >= K ? s.sorted[K - 1] : 0;
  Sum2 a{floor_of(c), 0.0f};
  for (int i = tid; i < chunks; i += kJoinThreads) add_sum2(a, sums[r * chunks + i]);
  for (int i = tid; i < total; i += kJoinThreads) {
    const uint64_t k = mine[i];
    if (k != 0 && k < last) add_one(a, key_value(k), c);
  }
  const Sum2 rest = block_sum2(s, a);
  write_row(g, r, s.sorted, n < K ? n : K, c64, rest);
}

// Chunks of a row: a workgroup for every compute unit, of at least 2048 columns, and of long rows (16384 columns a chunk
// and more) about as many as run at once; their keys within one list.  A second launch joins them (7 us).  Whole rows, one
// a compute unit, and this: 1 x 151936 bf16, K 64, 35 and 17 us, 128 of them 52 and 28, 256 52 and 37 (K 256: 109 and 60),
// 511 75 and 58; 300 x 128256 fp32 84 and 61, 600 of them 116 and 98; 256 x 262144 fp32 83 and 91.
constexpr int64_t kTopWanted = 1280;
struct TopSplit {
  int64_t chunks, columns;
};
TopSplit top_split(int64_t BT, int64_t V, int64_t K) {
  int64_t s = BT >= 128 ? 1 : (256 + BT - 1) / BT, more = kTopWanted / BT;
  if (s > V / 2048) s = V / 2048;
  if (more > V / 16384) more = V / 16384;
  if (s < more) s = more;
  if (s > kJoinList / K) s = kJoinList / K;
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
  top_join_kernel<<<large_grid(a.BT), dim3(kJoinThreads), 0, st>>>(a, c64, (int)s.chunks, keys, sums);
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
