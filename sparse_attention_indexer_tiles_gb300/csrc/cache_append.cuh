// Launch interface of the append to an MXFP4 cache (cache_append.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/idx.h"

namespace idx {

struct AppendArgs {
    const void* k;          // [T, Hkv, D], tokens k_stride elements apart
    const void* v;
    uint8_t* k_codes;       // [pages, Hkv, page_size, D / 2]
    uint8_t* k_sf;          // [pages, Hkv, page_size, D / 32]
    uint8_t* v_codes;
    uint8_t* v_sf;
    const int* table;       // [B, table_stride]
    const int* lens;        // [B]
    const int* q_start;     // [B + 1], or null: T / B tokens each
    long long table_stride, k_stride, v_stride;
    int B, T, Hkv, D, pages, page_size, page_shift;
    int* d_status;
};

// wide: rows of k and v lie on 16-byte boundaries
cudaError_t launch_append(const AppendArgs& a, idx_dtype dt, bool wide, cudaStream_t s);

}  // namespace idx
