// Host interface of the low-rank adapters (lora.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"

namespace lx {

// Largest rank the stacked adapters may have room for.
constexpr int kLoraMaxRank = 128;

// The adapters and the requests that use them.
struct LoraSet {
  const uint16_t *A, *B;    // bf16 (n, r, H), (n, N, r)
  const float* scale;       // [n]
  const int64_t* rank;      // [n] or nullptr (r)
  const int64_t* adapter;   // [R]
  const int64_t* start;     // [R + 1]
  int64_t T, R, n, H, N, r;
};

struct LoraForwardArgs {
  LoraSet s;
  const uint16_t* x;  // bf16 (T, H)
  int64_t ldx;
  const void* base;  // (T, N) or nullptr
  int64_t ldb;
  Dt base_dt;
  void* y;  // (T, N)
  int64_t ldy;
  Dt y_dt;
  void* workspace;
};

struct LoraBackwardArgs {
  LoraSet s;
  const uint16_t *dy, *x;  // bf16 (T, N), (T, H)
  int64_t lddy, ldx;
  const float* base;  // (T, H) or nullptr
  int64_t ldb;
  float* gx;  // (T, H) or nullptr
  int64_t ldgx;
  float *gA, *gB;  // (n, r, H), (n, N, r) or nullptr
  void* workspace;
};

size_t lora_forward_workspace_bytes(int64_t T, int64_t R, int64_t H, int64_t N, int64_t r);
size_t lora_backward_workspace_bytes(int64_t T, int64_t R, int64_t n, int64_t H, int64_t N, int64_t r);
hipError_t launch_lora_forward(const LoraForwardArgs& a, hipStream_t stream);
hipError_t launch_lora_backward(const LoraBackwardArgs& a, hipStream_t stream);

}  // namespace lx
