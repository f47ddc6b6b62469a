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
    int unit;              // columns per access: 8 when every row starts on a 16-byte boundary
                           // (its codes on an 8-byte one) and N % 8 == 0; 2 when every row starts
                           // on a pair of elements and N is even; else 1
};

cudaError_t launch_norm_quant(const NormArgs& a, idx_dtype dt, int sm_count, cudaStream_t s);

}  // namespace idx
