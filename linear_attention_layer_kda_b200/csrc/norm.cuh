// norm.cuh -- host entry points of norm.cu.
#pragma once

#include "common.cuh"

namespace kda {
namespace norm {

struct Args {
    const void *x, *residual, *weight;  // residual may be null (zeros); weight bf16
    void *residual_out;
    void *y;       // bf16 or null
    uint8_t *y8;   // E4M3 codes or null
    float *scale;  // with y8: [rows, hidden / 128]
    float *rstd;   // or null
    long long rows;
    int hidden;
    float eps;
};

struct GradArgs {
    const void *dy, *residual, *weight, *dres;  // dres may be null
    const float *rstd;
    void *dres_out;
    float *parts, *dweight;  // parts: [grad_parts, hidden]
    long long rows;
    int hidden;
};

cudaError_t forward(const Args &a, bool x_bf16, bool res_bf16, cudaStream_t st);
int grad_parts(long long rows, int hidden, int sms);
cudaError_t backward(const GradArgs &a, bool res_bf16, int parts, cudaStream_t st);

}  // namespace norm
}  // namespace kda
