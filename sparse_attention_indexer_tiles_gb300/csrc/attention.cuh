// Launch interface of the shared-prefix decode attention (attention.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/idx.h"

namespace idx {

constexpr int kAttnMaxTokens = 16;   // new tokens per request
constexpr int kAttnMaxGroup = 128;   // query heads per key head

// Keys per tile of the prefix kernel (see there).
__host__ __device__ constexpr int attn_prefix_keys(int D) { return D == 128 ? 80 : 128; }

// One attention call.  Rows: query row (b, t, head) = (b * Q + t) * Hq + head.  The
// keys of a row are cut into `splits` parts, the prefix's first; each part leaves its
// softmax-weighted mean of V and its log2-sum-exp2 in the workspace.
struct AttnArgs {
    const void* q;            // [B, Q, Hq, D]
    const void* k;            // [pages, Hkv, page_size, D]
    const void* v;
    const int* prefix_table;  // [ceil(prefix_len / page_size)]
    const int* table;         // [B, table_stride]
    const int* lens;          // [B]
    const float* w;           // [B, Hkv, slots] or null
    float* w_out;             // [B, Hkv, slots] or null; may be w
    void* out;                // [B, Q, Hq, D]
    float* lse;               // [B, Q, Hq] or null
    // workspace
    float* part;              // [rows, splits, D]
    float* part_lse;          // [rows, splits], log2 units; -inf: no keys
    float* logits;            // [B, Hkv, Q * G, logit_stride] log2 units, or null
    long long table_stride, slots, logit_stride;
    int B, Q, Hq, Hkv, G, D, pages, page_size, page_shift;
    int prefix_len, max_len;
    int prefix_splits, prefix_chunk;    // keys per prefix part (whole key tiles)
    int prefix_unit, prefix_tokens;     // keys per copy, query tokens per row tile (set by
                                        // launch_prefix_parts)
    int private_splits, private_chunk;  // keys per private part (a multiple of 64)
    bool private_dense;                 // private parts on the tensor cores' dense path (their
                                        // chunk: whole key tiles)
    float scale_log2;                   // scale * log2(e)
    long long wait_limit;               // SM clocks a wait of the prefix kernel may take
    int withhold_tile;                  // test only: the key tile that is never loaded, or -1
    int* d_status;
};

struct AttnPlan {
    int prefix_splits, prefix_chunk, private_splits, private_chunk;
    bool private_dense;
    size_t part, part_lse, logits, total;
    long long logit_stride;
};

AttnPlan attn_plan(int B, int Q, int Hq, int Hkv, int D, int prefix_len, int max_len, bool weights,
                   int sm_count);

// The prefix's parts, and the private ones of requests with many rows (attention_prefix.cu).
cudaError_t launch_prefix_parts(const AttnArgs& a, idx_dtype dt, cudaStream_t s);
cudaError_t launch_private_dense(const AttnArgs& a, idx_dtype dt, cudaStream_t s);

// Returns the number of kernels launched through *launched.
cudaError_t launch_attention(const AttnArgs& a, idx_dtype dt, int sm_count, cudaStream_t s,
                             int* launched);

}  // namespace idx
