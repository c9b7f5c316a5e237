// Host interface of cross entropy with distillation from a teacher's top logits (distill.hip,
// distill_linear.hip) and of the selection of top logits (top_logits.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"

namespace lx {

// Largest number of top logits a row.
constexpr int kKdMaxTop = 256;
constexpr int kKdState = 4;

// The loss's inputs beside the logits, and what the forward leaves behind.
struct KdLoss {
  const int64_t* target;  // [BT]
  int64_t ignore_index;
  const int32_t* ids;     // [BT][K]
  const float* top;       // [BT][K]
  const float* rest;      // [BT] or nullptr: the teacher is its top logits alone
  int64_t BT, V, K;
  float temperature;
  float *ce, *kd, *lse, *state;  // [BT], [BT], [BT], [BT][4]
};

// The gradient's factors.
struct KdGrad {
  float g_ce, g_kd;
  const float *ce_rows, *kd_rows;  // [BT] or nullptr (1)
  const float* g_scale;            // one float or nullptr (1)
};

struct KdArgs {
  KdLoss l;
  const void* z;  // (BT, V) logits
  int64_t ldz;
  void* grad;     // (BT, V) or nullptr (forward)
  int64_t ldg;
  KdGrad g;
  void* workspace;
};

size_t kd_forward_workspace_bytes(int64_t BT, int64_t V);
size_t kd_step_workspace_bytes(int64_t BT, int64_t V);
hipError_t launch_kd_forward(const KdArgs& a, Dt dt, hipStream_t stream);
hipError_t launch_kd_backward(const KdArgs& a, Dt dt, hipStream_t stream);
hipError_t launch_kd_step(const KdArgs& a, Dt dt, hipStream_t stream);

struct TopArgs {
  const void* z;  // (BT, V) logits
  int64_t ldz, BT, V, K;
  float temperature;
  float* top;           // [BT][K]
  int32_t* ids;         // [BT][K]
  float *lse, *rest;    // [BT] or nullptr
  void* workspace;
};

size_t top_workspace_bytes(int64_t BT, int64_t V, int64_t K);
hipError_t launch_top(const TopArgs& a, Dt dt, hipStream_t stream);

struct KdLinearArgs {
  KdLoss l;               // ids nullptr (K = 0): cross entropy alone
  const uint16_t *x, *w;  // bf16 (BT, H), (V, H)
  int64_t H;
  void *grad_x, *grad_w;  // (BT, H), (V, H), fp32 or bf16, or nullptr
  Dt grad_dt;
  KdGrad g;
  int64_t piece;          // columns of a piece of the vocabulary
  void* workspace;
};

size_t kd_linear_workspace_bytes(int64_t BT, int64_t V, int64_t H, int64_t K, int64_t piece, bool grads);
hipError_t launch_kd_linear(const KdLinearArgs& a, hipStream_t stream);
// 16-byte units of zeros
hipError_t launch_kd_linear_zero(void* p, int64_t units, hipStream_t stream);

}  // namespace lx
