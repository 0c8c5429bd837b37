// column_sum.hpp -- sums over the rows of a matrix of partial sums (epilogue_backward.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace igc {

// out[n] = round(sum_{k < chunks} part[k * N + n]) for n < N, in a fixed order; out of a storage type (igc_out_t).
hipError_t launch_column_sum(const float* part, int64_t N, int chunks, void* out, int kind, hipStream_t stream);

}  // namespace igc
