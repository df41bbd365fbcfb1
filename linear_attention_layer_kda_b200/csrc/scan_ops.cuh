// scan_ops.cuh -- host entry points of the scan kernels (scan.cu, scan_grad.cu).
#pragma once

#include "scan.cuh"

namespace kda {
namespace scan {

// The chunked forward pass; `backward`: what the backward pass needs of it instead of the outputs.
template <int DK, int DV, typename T>
cudaError_t forward(const Args &a, bool backward, cudaStream_t st);
// The recurrence token by token (no workspace).
template <int DK, int DV, typename T>
cudaError_t tokens(const Args &a, cudaStream_t st);
// The gradient of the states, from the last chunk to the first.
template <int DK, int DV, typename T>
cudaError_t reverse(const Args &a, cudaStream_t st);
// Backward: recomputes the forward's states, then the gradients.
template <int DK, int DV, typename T>
cudaError_t backward(const Args &a, cudaStream_t st);

}  // namespace scan
}  // namespace kda
