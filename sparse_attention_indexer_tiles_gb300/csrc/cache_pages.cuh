// Launch interface of the calls that say which row of a page table holds which page (cache_pages.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/idx.h"

namespace idx {

constexpr int kMaxCaches = 8;
constexpr int kMostPages = 0x7fffff00;

// The arrays whose pages move with the tables: [pages][bytes] each.
struct PageArrays {
    uint8_t* p[kMaxCaches];
    long long bytes[kMaxCaches];  // of a page, a multiple of 16
    int n;
};

struct PagesArgs {
    PageArrays caches;
    const int* refs;       // [pages]
    const int* table;      // [B, table_stride]
    const int* lens;       // [B]
    const int* arg;        // [B]: parents (fork), new lengths (resize)
    int* refs_out;         // each may be its input
    int* table_out;
    int* lens_out;
    int* live;             // [1] (compact)
    long long table_stride;
    int B, pages, page_size, page_shift;
    // workspace of the call at hand (see the kernels)
    int* ws;
    bool one_cta;          // rank with one CTA, whatever the sizes are
    int* d_status;
};

// ints of workspace
size_t fork_workspace_ints(int B, long long table_stride);
size_t resize_workspace_ints(int B, int pages, long long table_stride);
size_t compact_workspace_ints(int B, int pages);

// Add the number of kernels launched to *launched.  fork wants a workspace (ws not null) when
// table_out or lens_out is its input.
cudaError_t launch_fork(const PagesArgs& a, int sm_count, cudaStream_t s, int* launched);
cudaError_t launch_resize(const PagesArgs& a, int sm_count, cudaStream_t s, int* launched);
cudaError_t launch_compact(const PagesArgs& a, int sm_count, cudaStream_t s, int* launched);

}  // namespace idx
