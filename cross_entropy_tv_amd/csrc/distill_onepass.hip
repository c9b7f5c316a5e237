// Cross entropy and distillation from a teacher's top logits: the loss and the gradient of the logits in one pass.
//
// A row is cut into up to 12 members' chunks, each held in the registers of one workgroup between the row's sums and
// the gradient, so every logit is read once.  Tiles are taken by ticket: a workgroup waits only for members
// of its own row, whose tickets lie within 12 of its own, so with 12 workgroups running the exchange cannot
// deadlock; every wait is bounded, and one that gives up leaves NaN in the row.
//
//   1. the chunk is requested, and while it arrives the ids that fall into it are marked in LDS and wave 0 forms
//      the teacher's masses;
//   2. each thread's sum of 2^(c z - n) outside the ids and, at another temperature than 1, of 2^(z log2 e - n1) of
//      all columns, as the chunk arrives;
//   3. a member publishes its sums, those of its ids' logits, and its part of kd, and waits
//      for the row's;
//   4. the gradient of its chunk.
//
// Every member has read its chunk, its ids' logits and the target's before it publishes, and stores after all have
// published: the gradient may overwrite the logits.  What is published is one 64-bit word a slot, preset to a
// pattern that no result has, so that a slot is its own flag.
//
// The logits stay in the registers as they lie in memory, and their exponentials are formed twice: kept in fp32 they
// would take twice the registers, three workgroups a compute unit instead of four, which cost more (8192 x 151936 bf16:
// 965 against 860 us) than 1.2 G exponentials.
//
// What bounds it: reading and writing the logits once, by workgroups whose life is a chain (ids, chunk, sums, exchange,
// stores: 17 us) that four of them a compute unit cover: 860 us, 5.8 TB/s (the same pass of cross entropy alone takes
// 832).  Loads and stores are non-temporal (with plain loads 1400).  Code size matters as well: what happens at the ids
// once stood in every group's code.
#include "common.hpp"
#include "distill.hpp"
#include "kd_row.hpp"
#include "mm.hpp"
#include "sum2.hpp"

namespace lx {

namespace {

constexpr int kStepThreads = 256;
constexpr int kStepWaves = kStepThreads / 64;
constexpr int kStepGroups = 15;    // groups of 8 a thread holds (five members of 151936 columns)
constexpr int kStepShort = 2;      // of a short row,
constexpr int kStepMiddle = 6;     // and of a middling one
constexpr int kMaxMembers = 12;
constexpr int kSlots = 5;          // words a member publishes (a wave reads a row's)
constexpr uint64_t kEmpty = ~0ull;
constexpr unsigned kSpinLimit = 1u << 18;
constexpr int64_t kStepTiles = 256;  // workgroups that few rows are cut into

struct StepArgs {
  KdLoss l;
  KdGrad g;
  const void* z;
  void* grad;
  int64_t ldz, ldg;
  double c64;
  int members, gpm;  // workgroups a row, groups a member
  uint64_t* slots;   // [BT][members][kSlots]
  unsigned* ticket;
};

struct Plan {
  int members, gpm;
};
// A row takes as many members as hold it, and few rows more of them, so that about 256 workgroups run (1 x 151936 bf16:
// 12 members 11.8 us, 5 14.5; 40 rows: 12 members 19.8, 5 18.3).  A thread's groups in code: what is
// held is unrolled, so short and middling chunks have their own (8 x 1000 bf16 6.1 us against 7.0, 2048 x 3200 15 against
// 20, 2048 x 11000 24 against 27).
// members 0: rows too long.  The last member also has the V % 8 columns behind the row's whole groups.
Plan plan_of(int64_t BT, int64_t V) {
  const int64_t groups = V < 8 ? 1 : V / 8, most = (int64_t)kStepThreads * kStepGroups;
  const int64_t fit = (groups + most - 1) / most;
  int64_t fill = (kStepTiles + BT - 1) / BT;
  if (fill > groups / (2 * kStepThreads)) fill = groups / (2 * kStepThreads);
  int64_t k = fit > fill ? fit : fill;
  if (fit > kMaxMembers || BT > ((int64_t)1 << 26)) return Plan{0, 0};
  if (k > kMaxMembers) k = kMaxMembers;
  const int64_t gpm = (groups + k - 1) / k;
  return Plan{(int)((groups + gpm - 1) / gpm), (int)gpm};
}

// Lanes [0, n) of wave 0 wait for slots sl[0 .. n) and keep what they read in got.  Whether the wait gave up.
__device__ __forceinline__ bool wait_slots(const uint64_t* sl, int n, uint64_t* got) {
  const int lane = tid_x();
  const bool mine = lane < n;
  uint64_t v = kEmpty;
  bool gave_up = false;
  __builtin_amdgcn_s_setprio(2);
  for (unsigned spins = 0;; ++spins) {
    if (mine && v == kEmpty) v = fetch(sl + lane);
    if (__all(!mine || v != kEmpty)) break;
    if (spins > kSpinLimit) {
      gave_up = true;
      break;
    }
    __builtin_amdgcn_s_sleep(1);
  }
  __builtin_amdgcn_s_setprio(0);
  if (mine) got[lane] = v;
  return gave_up;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ float lo_of32(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of32(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ double double_of(uint64_t v) { return __builtin_bit_cast(double, v); }

struct StepLds {
  uint32_t bits[kStepThreads * kStepGroups / 4 + 1];  // of the chunk's columns, those behind its groups last
  // Groups that hold an id: their numbers in the order in which they were found, and by number what becomes of their
  // columns.
  uint16_t number[kStepThreads * kStepGroups + 1];
  float value[kKdMaxTop][8];
  int groups;
  int id[kKdMaxTop];    // in the chunk, else -1
  float u[kKdMaxTop], z[kKdMaxTop], q[kKdMaxTop];
  int all[kKdMaxTop];   // ids wherever they are, -1: left out
  Sum2d red[2][kStepWaves];
  uint64_t got[kMaxMembers * kSlots];
  unsigned tile;
  int bad, twice;       // an id past the vocabulary; one given twice
  // the row's sums as the gradient takes them, from wave 0
  float out, rest_n;    // outside the ids: factor of 2^(c z - rest_n)
  float ce1, n1;        // ce's part: factor of 2^(z log2 e - n1)
  float kd, n;          // at the ids: factor of 2^(c z - n) / kkd
  int state;            // 0, 1: no unmasked logit, 2: NaN
};

// G groups of 8 a thread (0: rows of fewer than 8 columns).
template <typename T, bool TEMP, int G>
__global__ __attribute__((amdgpu_flat_work_group_size(kStepThreads, kStepThreads), amdgpu_waves_per_eu(sizeof(T) == 4 && G > 6 ? 3 : 4)))
void kd_step_kernel(StepArgs a) {
  __shared__ StepLds s;
  const int tid = tid_x();
  const KdLoss& l = a.l;
  const int K = (int)l.K, members = a.members;
  __builtin_amdgcn_s_setprio(3);  // until the chunk is requested: ahead of the arithmetic of other workgroups
  unsigned tile = large_bid();
#pragma unroll
  for (int w = 0; w <= kStepThreads * G / 4; w += kStepThreads)
    if (w + tid <= kStepThreads * G / 4) s.bits[w + tid] = 0u;
  if (tid == 0) {
    s.bad = s.twice = s.groups = 0;
    if (members > 1) s.tile = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  // (uniform: what is read by row goes through scalar loads, which the wait for the chunk does not hold back)
  if (members > 1) tile = (unsigned)__builtin_amdgcn_readfirstlane((int)s.tile);
  const int64_t r = tile / (unsigned)members;
  if (r >= l.BT) return;
  const int member = (int)(tile - (unsigned)r * (unsigned)members);
  const int V = (int)l.V;
  // the chunk's whole groups and columns [first, end)
  const int first = member * a.gpm * 8;
  const int count = min(a.gpm, V / 8 - member * a.gpm);
  const int behind = member == members - 1 ? V - first - 8 * count : 0;  // columns behind its groups
  const int end = first + 8 * count + behind;
  const T* row = static_cast<const T*>(a.z) + r * a.ldz;
  T* out = static_cast<T*>(a.grad) + r * a.ldg;
  const int64_t t = l.target[r];
  if (t == l.ignore_index) {
    if (member == 0 && tid == 0) store_row(l, r, RowResult{});
    const float zero[8] = {};
    for (int g = tid; g < count; g += kStepThreads) store8_any(out + first + 8 * g, zero);
    if (tid < behind) store_bits1(out + first + 8 * count + tid, 0u);
    return;
  }

  // ---- the ids, then the chunk (loads return in order); no load is conditional, so that the compiler knows how
  // many are in flight behind the one that it waits for
  const int entry = min(tid, K - 1);
  const int raw_id = l.ids[r * K + entry];
  const float my_u = l.top[r * K + entry];
  // groups tid + k 256; past the chunk's end its last one again, which counts for nothing
  Group<T> h[G > 0 ? G : 1];
  const T* mine = row + first;
  if constexpr (G > 0) {
    const int last = 8 * (count - 1);
#pragma unroll
    for (int k = 0; k < G; ++k) h[k].load_once(mine + min(8 * (tid + k * kStepThreads), last));
  }
  __builtin_amdgcn_s_setprio(0);
  const bool t_here = t >= first && t < end;
  const bool my_bad = tid < K && raw_id >= V;
  const int my_id = tid >= K || my_bad || raw_id < 0 || my_u < kMasked ? -1 : raw_id;
  const bool here = my_id >= first && my_id < end;
  // (wanted after the sums)
  const T raw_z = row[here ? my_id : 0], raw_zt = row[t >= 0 && t < V ? (int)t : 0];
  const T raw_extra = row[tid < behind ? first + 8 * count + tid : 0];
  if (tid < K) {
    if (here) {
      const int at = my_id - first;
      const uint32_t old = atomicOr(&s.bits[at >> 5], 1u << (at & 31));
      if (old >> (at & 31) & 1u) s.twice = 1;
      if ((old >> (at & 24) & 0xffu) == 0u) s.number[at >> 3] = (uint16_t)atomicAdd(&s.groups, 1);
    }
    s.id[tid] = here ? my_id : -1;
    s.all[tid] = my_id;
    s.u[tid] = my_u;
    if (my_bad) s.bad = 1;
  }
  const RowFactors f = row_factors(a.g, l, r);
  mm::lds_barrier();  // (the chunk stays in flight)
  Teacher te{};
  double ua[kLaneTop], q[kLaneTop];
  if (tid < 64) te = teacher_of(s.all, s.u, K, tid, a.c64, l.rest ? l.rest[r] : ninf(), ua, q);

  // ---- sums
  const float c = (float)a.c64;
  const uint8_t* mask = reinterpret_cast<const uint8_t*>(s.bits);
  auto get = [&](int k, float(&x)[8]) {
    launder(h[k]);
    h[k].get(x);
  };
  auto is_mine = [&](int k) { return tid + k * kStepThreads < count; };
  const bool extra_named = tid < behind && (mask[count] >> tid & 1u);
  const float extra = tid < behind ? load1(&raw_extra) : ninf();  // the thread's column behind the groups
  Sum2 sum{floor_of(c), 0.0f}, sum1{floor_of(kLog2e), 0.0f};
  if (!extra_named) add_one(sum, extra, c);
  if (TEMP) add_one(sum1, extra, kLog2e);
#pragma unroll
  for (int k = 0; k < G; ++k) {
    if (is_mine(k)) {
      float x[8];
      get(k, x);
      if (TEMP) add_group(x, kLog2e, sum1);
      leave_out_bits(mask[tid + k * kStepThreads], x);
      add_group(x, c, sum);
    }
  }
  {
    const Sum2d w = wave_sum2d(sum);
    Sum2d w1{};
    if (TEMP) w1 = wave_sum2d(sum1);
    if ((tid & 63) == 0) {
      s.red[0][tid >> 6] = w;
      s.red[1][tid >> 6] = w1;
    }
  }
  const float my_z = here ? load1(&raw_z) : ninf();
  if (tid < K) s.z[tid] = my_z;
  __syncthreads();

  // ---- wave 0: the member's part, the exchange, the row
  Sum2d rest{}, whole{}, all{};
  double terms = 0.0;
  float zt = load1(&raw_zt);
  asm volatile("" : "+v"(zt)::"memory");  // read before anything is published: its owner may overwrite it then
  bool gave_up = false;
  if (tid < 64) {
    Sum2d top{floor_of(c), 0.0};
    const bool twice = s.twice != 0;
#pragma unroll
    for (int k = 0; k < kLaneTop; ++k) {
      const int j = tid + 64 * k;
      if (j < K) {
        s.q[j] = (float)q[k];  // (a token's whole mass, see below)
        if (s.id[j] >= 0) {
          const float z = s.z[j];
          if (q[k] > 0.0) terms += z < kMasked ? kInf64 : q[k] * (ua[k] - (double)z * a.c64);
          if (!(z < kMasked) && !(twice && named_before(s.id, j))) {
            const double t2 = (double)z * a.c64, n = __builtin_rint(t2);
            add_sum2d(top, Sum2d{(float)n, exp2_64(t2 - n)});
          }
        }
      }
    }
    if (twice) {  // the masses of a token's entries, in their order, at each of them
      float whole_q[kLaneTop] = {};
#pragma unroll
      for (int k = 0; k < kLaneTop; ++k) {
        const int j = tid + 64 * k;
        if (j < K)
          for (int i = 0; i < K; ++i) whole_q[k] += s.id[i] == s.id[j] ? s.q[i] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kLaneTop; ++k)
        if (tid + 64 * k < K) s.q[tid + 64 * k] = whole_q[k];
    }
    top = wave_sum2d(top);
    terms = wave_sum64(terms);
    rest = s.red[0][0];
    whole = s.red[1][0];
    for (int w = 1; w < kStepWaves; ++w) {
      add_sum2d(rest, s.red[0][w]);
      if (TEMP) add_sum2d(whole, s.red[1][w]);
    }
    if (members > 1) {
      uint64_t* slots = a.slots + r * (int64_t)(members * kSlots);
      const uint64_t w = tid == 0   ? pack2(rest.n, top.n)
                         : tid == 1 ? __builtin_bit_cast(uint64_t, rest.s)
                         : tid == 2 ? __builtin_bit_cast(uint64_t, top.s)
                         : tid == 3 ? __builtin_bit_cast(uint64_t, terms)
                                    : pack2(whole.n, (float)whole.s);
      if (tid < kSlots) publish(slots + member * kSlots + tid, w);
      gave_up = wait_slots(slots, members * kSlots, s.got);
      const bool theirs = tid < members;  // lane k has member k's
      const uint64_t* got = s.got + (theirs ? tid : 0) * kSlots;
      const Sum2d nothing{floor_of(c), 0.0};
      rest = wave_sum2d(theirs ? Sum2d{lo_of32(got[0]), double_of(got[1])} : nothing);
      top = wave_sum2d(theirs ? Sum2d{hi_of32(got[0]), double_of(got[2])} : nothing);
      if (TEMP) whole = wave_sum2d(theirs ? Sum2d{lo_of32(got[4]), (double)hi_of32(got[4])} : Sum2d{floor_of(kLog2e), 0.0});
      terms = wave_sum64(theirs ? double_of(got[3]) : 0.0);
    }
    all = top;
    add_sum2d(all, rest);
    if (!TEMP) whole = all;
    if (tid == 0) {
      const float rest_s = (float)rest.s, all_s = (float)all.s;
      const bool any = all_s > 0.0f;
      const float p_rest = any ? rest_s * exp2_hw(rest.n - all.n) / all_s : 0.0f;
      const float off = te.any ? p_rest - (float)te.q_rest : 0.0f;
      const float part = f.kkd * off + (TEMP ? 0.0f : f.kce * p_rest);
      s.out = rest_s > 0.0f ? part / rest_s : 0.0f;
      s.rest_n = rest.n;
      s.ce1 = any ? f.kce / (float)whole.s : 0.0f;
      s.n1 = whole.n;
      s.kd = any ? 1.0f / all_s : 0.0f;
      s.n = all.n;
      s.state = gave_up || t < 0 || t >= V ? 2 : !any ? 1 : s.bad ? 2 : 0;
    }
  }
  __syncthreads();
  if (tid < 64 && member == 0) {  // the row's results
    const double lr = log2_of(rest), lz = log2_of(all);
    RowResult o = row_result(l, te, s.bad != 0, t, zt, terms, lz, lr, TEMP ? log2_of(whole) * kLn2 : lz * kLn2);
    if (gave_up) o.bad = 3u;
    if (tid == 0) store_row(l, r, o);
  }

  // ---- the gradient
  const float g_out = s.out, rest_n = s.rest_n, ce1 = s.ce1, n1 = s.n1;
  if (tid < K && s.id[tid] >= 0) {  // at the ids
    const int at = s.id[tid] - first;
    const float v = ce1 * exp2_hw(__builtin_fmaf(my_z, kLog2e, -n1)) +
                    f.kkd * (s.kd * exp2_hw(__builtin_fmaf(my_z, c, -s.n)) - s.q[tid]);
    s.value[s.number[at >> 3]][at & 7] = v;
  }
  __syncthreads();
  const int state = s.state;
  if (state != 0) {  // (nothing or NaN)
    const uint32_t fill = state == 2 ? kQNaN32 : 0u;
    for (int v = first + tid; v < end; v += kStepThreads) store_bits1(out + v, fill);
    return;
  }
  const int t_at = t_here ? (int)t - first : -8;
  auto outside = [&](float x) {
    const float w = g_out * exp2_hw(__builtin_fmaf(x, c, -rest_n));
    return TEMP ? __builtin_fmaf(ce1, exp2_hw(__builtin_fmaf(x, kLog2e, -n1)), w) : w;
  };
  T* to = out + first;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    if (is_mine(k)) {
      const int at = tid + k * kStepThreads;
      const uint32_t byte = mask[at];
      float w[8];
      float x[8];
      get(k, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = outside(x[e]);
      if (byte) {
        const float4* v = reinterpret_cast<const float4*>(s.value[s.number[at]]);
        const float4 lo = v[0], hi = v[1];
        const float n[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = byte >> e & 1u ? n[e] : w[e];
      }
      if (at == t_at >> 3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e == (t_at & 7) ? w[e] - f.kce : w[e];
      }
      store8_any(to + 8 * at, w);
    }
  }
  if (tid < behind) {
    float w = extra_named ? s.value[s.number[count]][tid] : outside(extra);
    if (8 * count + tid == t_at) w -= f.kce;
    store1(to + 8 * count + tid, w);
  }
}

__global__ __launch_bounds__(256) void kd_step_init_kernel(uint64_t* slots, int64_t n, unsigned* ticket) {
  const int64_t i0 = (int64_t)bid_x() * 256 + tid_x();
  if (i0 == 0) *ticket = 0u;
  for (int64_t i = i0; i < n; i += (int64_t)nblocks_x() * 256) slots[i] = kEmpty;
}

template <typename T, bool TEMP>
hipError_t launch_t(const KdArgs& a, const Plan& p, hipStream_t st) {
  StepArgs s{};
  s.l = a.l; s.g = a.g; s.z = a.z; s.grad = a.grad; s.ldz = a.ldz; s.ldg = a.ldg;
  s.c64 = scale_of(a.l.temperature);
  s.members = p.members; s.gpm = p.gpm;
  (void)hipGetLastError();
  if (p.members > 1) {
    const int64_t n = a.l.BT * p.members * kSlots, blocks = (n + 255) / 256;
    s.slots = static_cast<uint64_t*>(a.workspace);
    s.ticket = reinterpret_cast<unsigned*>(s.slots + n);
    kd_step_init_kernel<<<dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st>>>(s.slots, n, s.ticket);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const dim3 grid = large_grid(a.l.BT * p.members);
  if (a.l.V < 8) kd_step_kernel<T, TEMP, 0><<<grid, dim3(kStepThreads), 0, st>>>(s);
  else if (p.gpm <= kStepShort * kStepThreads) kd_step_kernel<T, TEMP, kStepShort><<<grid, dim3(kStepThreads), 0, st>>>(s);
  else if (p.gpm <= kStepMiddle * kStepThreads) kd_step_kernel<T, TEMP, kStepMiddle><<<grid, dim3(kStepThreads), 0, st>>>(s);
  else kd_step_kernel<T, TEMP, kStepGroups><<<grid, dim3(kStepThreads), 0, st>>>(s);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_dt(const KdArgs& a, const Plan& p, hipStream_t st) {
  return a.l.temperature != 1.0f ? launch_t<T, true>(a, p, st) : launch_t<T, false>(a, p, st);
}

}  // namespace

size_t kd_step_workspace_bytes(int64_t BT, int64_t V) {
  if (BT <= 0 || V <= 0) return 0;
  const Plan p = plan_of(BT, V);
  if (p.members == 0) return kd_forward_workspace_bytes(BT, V);
  if (p.members == 1) return 0;
  return ((size_t)(BT * p.members) * kSlots * 8 + 4 + 255) & ~(size_t)255;
}

hipError_t launch_kd_step(const KdArgs& a, Dt dt, hipStream_t st) {
  const Plan p = plan_of(a.l.BT, a.l.V);
  if (p.members == 0) {  // rows too long to be held: the forward, then the backward
    if (hipError_t e = launch_kd_forward(a, dt, st)) return e;
    return launch_kd_backward(a, dt, st);
  }
  switch (dt) {
    case Dt::BF16: return launch_dt<uint16_t>(a, p, st);
    case Dt::F16: return launch_dt<_Float16>(a, p, st);
    default: return launch_dt<float>(a, p, st);
  }
}

}  // namespace lx
