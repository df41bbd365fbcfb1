// rows.cuh -- host entry point of rows.cu.
#pragma once

#include "common.cuh"
#include "rows.h"

namespace kda {
namespace rows {

constexpr int kMaxMoves = KDA_STATE_MOVES_MAX;

cudaError_t run(void *dst, const void *src, size_t row_bytes, const Plan &p, int n, cudaStream_t st);

}  // namespace rows
}  // namespace kda
