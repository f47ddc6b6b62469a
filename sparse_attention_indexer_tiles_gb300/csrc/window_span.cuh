// What the kernels of the windowed attention share (attention_window*.cu): the tokens of a request in a call, and
// the copies of a cache's rows.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "window.cuh"

namespace idx {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

struct Span {
    int first, count;  // tokens
    int len;           // cached slots, the new tokens' among them
};
IDX_DEVI Span span_of(const WindowArgs& a, int b, bool report) {
    Span s;
    int end;
    if (a.q_start) {
        s.first = a.q_start[b];
        end = a.q_start[b + 1];
    } else {
        const int per = a.T / a.B;
        s.first = b * per;
        end = s.first + per;
    }
    s.len = a.lens[b];
    const bool wrong = s.first < 0 || end < s.first || end > a.T;
    if (report && (wrong || end - s.first > a.max_q || s.len < 0 || s.len > a.max_len))
        raise_status(a.d_status, IDX_DEV_RANGE);
    s.count = wrong ? 0 : min(end - s.first, a.max_q);
    if (wrong) s.first = 0;
    s.len = min(max(s.len, 0), a.max_len);
    return s;
}

IDX_DEVI void tma_rows(uint32_t dst, const void* tmap, uint64_t* bar, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(0), "r"(row)
        : "memory");
}
IDX_DEVI void bulk_rows(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Map of rows of codes (D / 2 bytes), `unit` rows per copy, their 16-byte chunks swizzled.
inline CUresult code_map(CUtensorMap* m, const uint8_t* base, int D, long long rows, int unit) {
    auto enc = tensor_map_encoder();
    if (!enc) return CUDA_ERROR_NOT_SUPPORTED;
    const cuuint64_t dims[2] = {(cuuint64_t)D / 2, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)D / 2};
    const cuuint32_t box[2] = {(cuuint32_t)D / 2, (cuuint32_t)unit}, one[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace idx
