// Launch interface of the add + RMS norm + e4m3 quantisation kernel (norm_quant.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/idx.h"

namespace idx {

constexpr int kNormMaxCols = 32768;

struct NormArgs {
    const void* x;         // [rows, x_stride >= N]
    const void* residual;  // [rows, N] or null
    const void* weight;    // [N]
    void* residual_out;    // [rows, N] or null; may be `residual`
    uint8_t* out;          // [rows, N] e4m3
    float* scale;          // [rows] or [rows, N / group]
    long long x_stride;
    int rows, N, group;
    float eps;
    bool vec;              // every row starts on a 16-byte boundary and N % 8 == 0
};

cudaError_t launch_norm_quant(const NormArgs& a, idx_dtype dt, int sm_count, cudaStream_t s);

}  // namespace idx
