// Host interface of the verification of drafted tokens (draft_verify.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"

namespace lx {

struct VerifyArgs {
  const void* target;  // (N + S, V) logits, row stride ldt
  const void* draft;   // (N, V) logits, row stride ldd; nullptr: drafts without a distribution
  int64_t ldt, ldd;
  const int64_t* tokens;  // [N]
  const int64_t* start;   // [S + 1]
  int64_t S, N, L, V;     // L: the largest number of drafts of a sequence
  const float* temperature;  // [S] or nullptr (1)
  const float *u_accept, *u_sample;
  int64_t *n_accepted, *out;  // [S], [S][L + 1]
  float* logprobs;            // [S][L + 1] or nullptr
  void* workspace;
};

size_t verify_workspace_bytes(int64_t S, int64_t L, int64_t V);
hipError_t launch_verify(const VerifyArgs& a, Dt dt, hipStream_t stream);

}  // namespace lx
