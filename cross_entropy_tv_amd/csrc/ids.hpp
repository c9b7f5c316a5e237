// Work-item and grid indices for the kernels.
#pragma once

#include <hip/hip_runtime.h>

namespace lx {

// Work-item and grid indices read straight from the hardware and the dispatch
// packet.  The kernels are compiled with IEEE mode off, the device library's
// index functions with it on, and the compiler does not inline a function
// built for another floating-point mode: threadIdx / blockIdx / blockDim /
// gridDim would each become a real call, with the calling convention's
// register traffic around it.
__device__ __forceinline__ int tid_x() { return (int)__builtin_amdgcn_workitem_id_x(); }
__device__ __forceinline__ unsigned bid_x() { return __builtin_amdgcn_workgroup_id_x(); }
__device__ __forceinline__ unsigned bdim_x() { return __builtin_amdgcn_workgroup_size_x(); }
// The number of workgroups is the first implicit kernel argument (code object
// v5 layout), which sits with the explicit ones in the kernel-argument
// segment.  The dispatch packet also holds the grid size, but the packet lives
// in the queue's ring buffer: reading it at every workgroup's start measurably
// slowed kernels made of many short workgroups.
__device__ __forceinline__ unsigned nblocks_x() {
  return *(const unsigned*)__builtin_amdgcn_implicitarg_ptr();
}

// Large grids.  One dimension of a launch holds less than 2^32 threads (2^24 workgroups of 256), and the runtime does
// not refuse more but launches what is left modulo 2^32.  Grids that may be larger are cut into rows of 2^20
// workgroups (a multiple of 8: workgroup id mod 8 stays the die), and their kernels take their place from large_bid;
// the last row's workgroups behind the end find no work at their place.
constexpr int kGridRowBits = 20;
__device__ __forceinline__ unsigned large_bid() {
  return (__builtin_amdgcn_workgroup_id_y() << kGridRowBits) + __builtin_amdgcn_workgroup_id_x();
}
inline dim3 large_grid(int64_t workgroups) {
  constexpr int64_t row = (int64_t)1 << kGridRowBits;
  if (workgroups <= row) return dim3((unsigned)workgroups);
  return dim3((unsigned)row, (unsigned)((workgroups + row - 1) / row));
}

}  // namespace lx
