// Launch interface of the cache eviction kernels (evict.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/idx.h"

namespace idx {

struct EvictArgs {
    uint8_t* k;            // [pages, Hkv, page_size, row_bytes]
    uint8_t* v;
    const int* table;      // [B, table_stride]
    const int* lens;       // [B]
    const float* w;        // [B, Hkv, slots]
    const int* pos;        // [B, Hkv, slots]
    const int* next_pos;   // [B]
    int* lens_out;         // [B]
    float* w_out;          // [B, Hkv, slots]; may be w
    int* pos_out;          // [B, Hkv, slots]; may be pos
    int* moves;            // workspace [B * Hkv, 2, max_moves]: holes, then sources
    int* counts;           // workspace [B * Hkv]: moves of each
    long long slots, table_stride;
    int B, Hkv, page_size, page_shift, pages, row_bytes;
    int budget, recent, sink, max_len, max_moves;
    int* d_status;
};

// Moves a (request, head) can need: no more than the kept slots or the evicted ones.
inline int evict_max_moves(int budget, int max_len) {
    const int gone = max_len - budget;
    return gone <= 0 ? 0 : (gone < budget ? gone : budget);
}

// Adds the number of kernels launched to *launched.
cudaError_t launch_evict(const EvictArgs& a, int sm_count, cudaStream_t s, int* launched);

}  // namespace idx
