// rr_norm.h -- argument blocks and launchers of the norm over the ranks' rows
// (internal to librr.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rr.h"
#include "rr_kernels.h"

namespace rr {

constexpr uint32_t kNormDim = 16384;  // a row is kept in registers

// Floats of a workgroup's line of sums: both, and 256 bytes, without which lines of
// 4096 columns would all start at the same memory channel.
constexpr __host__ __device__ uint32_t norm_line(uint32_t dim) { return 2 * ((dim + 3) / 4 * 4) + 64; }

// Row i of all ranks' rows: row i mod rows of rank i / rows.
struct NormArgs {
  const void* in[RR_MAX_RANKS];
  void* out[RR_MAX_RANKS];
  const void* weight;  // NULL: ones
  const void* bias;    // NULL: zeros
  float* mean;         // NULL: not kept
  float* rstd;         // NULL: not kept
  uint32_t rows, total;
  uint32_t dim;
  float eps;
  float fit, back;  // a power of two that a lane's sum of squares is scaled with, and 1 / fit
  int32_t center;
};

struct NormGradArgs {
  const void* dy[RR_MAX_RANKS];
  const void* x[RR_MAX_RANKS];
  const void* res[RR_MAX_RANKS];
  void* dx[RR_MAX_RANKS];
  const void* weight;  // NULL: ones
  const float* mean;   // center
  const float* rstd;
  float* part;         // [grid][norm_line(dim)]: sums of dy xhat and, dim rounded up to 4 further, of dy;
                       // NULL: not needed
  uint32_t rows, total;
  uint32_t dim;
  int32_t center, has_dx, has_res;
};

struct NormJoinArgs {
  const float* part;
  void* dweight;  // NULL: not needed
  void* dbias;    // NULL: not needed
  uint32_t parts, dim;
};

// Workgroups of the gradient, each with sums of its own; 0 for no rows.
uint32_t norm_grad_grid(uint32_t total, uint32_t dim, Kind k);

hipError_t launch_norm(const NormArgs& a, Kind k, hipStream_t s);
hipError_t launch_norm_grad(const NormGradArgs& a, Kind k, hipStream_t s);
hipError_t launch_norm_join(const NormJoinArgs& a, Kind k, hipStream_t s);

}  // namespace rr
