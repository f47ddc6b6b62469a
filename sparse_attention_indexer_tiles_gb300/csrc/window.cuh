// Launch interface of the attention over an MXFP4 cache with a window and sinks (attention_window.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/idx.h"

namespace idx {

constexpr int kWindowMaxGroup = 128;  // query heads per key head
constexpr int kWindowStep = 32;       // keys that a warp takes at a time
constexpr int kWindowCluster = 8;     // the largest portable cluster

// One call.  Query row (token, head) = token * Hq + head; the tokens of request b are
// q_start[b] .. q_start[b + 1] - 1.  The rows of a request and key head are taken in tiles, the
// keys that a tile sees in splits; a split's mean of V and log2-sum-exp2 go to the workspace, or stay in a
// cluster's shared memory, unless there is one split.
struct WindowArgs {
    const void* q;           // [T, Hq, D], tokens q_stride elements apart
    const uint8_t* k_codes;  // [pages, Hkv, page_size, D / 2]
    const uint8_t* k_sf;     // [pages, Hkv, page_size, D / 32]
    const uint8_t* v_codes;
    const uint8_t* v_sf;
    const int* table;        // [B, table_stride]
    const int* lens;         // [B]
    const int* q_start;      // [B + 1], or null: T / B tokens each
    void* out;               // [T, Hq, D]
    float* lse;              // [T, Hq] or null
    float* part;             // [T * Hq, splits, D]
    float* part_lse;         // [T * Hq, splits], log2 units; -inf: no keys
    long long table_stride, q_stride;
    int B, T, Hq, Hkv, G, D, pages, page_size, page_shift;
    int max_q, max_len, window, sink;
    int row_tiles;           // per request and key head (dense: pairs of them)
    int splits, chunk;       // steps of kWindowStep keys per split (dense: key tiles)
    bool clustered;          // a tile's splits are one cluster, which joins them in shared memory
    float scale_log2;        // scale * log2(e)
    long long wait_limit;    // SM clocks that a wait of the dense path may take
    int withhold_step;       // test only: the dense path's key tile that is never loaded, or -1
    int* d_status;
};

struct WindowPlan {
    bool dense;              // on the tensor cores' dense path (attention_window_dense.cu)
    bool clustered;
    int tile_rows, row_tiles, splits, chunk;
    size_t part, part_lse, total;
};

// path: 0 the cheaper one, -1 tiles of few rows, 1 the dense path
WindowPlan window_plan(int B, int T, int max_q, int Hq, int Hkv, int D, int max_len, int window, int sink, int path,
                       int sm_count);

// The dense path: keys per tile, and the launch.
int window_dense_keys(int D);
cudaError_t launch_window_dense(const WindowArgs& a, idx_dtype dt, cudaStream_t s);

// Adds the number of kernels launched to *launched.
cudaError_t launch_window(const WindowArgs& a, const WindowPlan& p, idx_dtype dt, cudaStream_t s, int* launched);

}  // namespace idx
