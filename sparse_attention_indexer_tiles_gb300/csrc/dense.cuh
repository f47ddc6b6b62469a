// Device helpers of the attention kernels on the 5th-generation tensor cores (attention_prefix.cu,
// attention_window_dense.cu): two products per key tile, S = Q K^T and O += P V, with P in TMEM.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cudaTypedefs.h>

#include "serve.cuh"

namespace idx {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

constexpr float kRenew = 8.f;  // growth of a row's maximum (in log2 units) that renews it

IDX_DEVI float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// One lane of a converged warp.
IDX_DEVI bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

IDX_DEVI void tma_load_4d(uint32_t dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2,
                          int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
        "r"(c3)
        : "memory");
}
// mbar_wait on two barriers, their tests in flight together.
IDX_DEVI bool mbar_wait2(uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1,
                         volatile int* abort, long long limit) {
    bool ok0 = mbar_try_wait(bar0, parity0), ok1 = mbar_try_wait(bar1, parity1);
    if (ok0 && ok1) return true;
    const long long t0 = clock64();
    for (;;) {
        if (!ok0) ok0 = mbar_try_wait(bar0, parity0);
        if (!ok1) ok1 = mbar_try_wait(bar1, parity1);
        if (ok0 && ok1) return true;
        if (*abort || clock64() - t0 > limit) return false;
    }
}

// D[tmem] (+)= A[tmem] * B[smem], 16-bit inputs, fp32 accumulator.
IDX_DEVI void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                     uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32x32b shape, N columns (8 or 32): thread t writes lane t.
template <int N>
IDX_DEVI void tmem_st32x32b(uint32_t taddr, const uint32_t* r) {
    if constexpr (N == 8) {
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
            : "memory");
    } else {
        static_assert(N == 32, "8 or 32 columns");
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, "
            "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
            "%27, %28, %29, %30, %31, %32};" ::"r"(taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
            "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
            "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
            "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
            "r"(r[29]), "r"(r[30]), "r"(r[31])
            : "memory");
    }
}
IDX_DEVI void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptors of a K tile as a K-major operand and of a V tile as an MN-major one, both
// 128-byte swizzled: 8 keys are `group` bytes apart (stride offset); V's next 64 columns are
// 1024 bytes further (leading offset).
IDX_DEVI uint64_t kv_desc(uint32_t saddr, uint32_t group) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(1024 >> 4) << 16) |
           ((uint64_t)(group >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// FMT: the instruction descriptor's; LIFT: m stays this far below the row's maximum.  P is then up to
// 2^(LIFT + kRenew) = 2^15, inside fp16, whose numbers below 2^-14 have fewer bits than the others:
// weights down to 2^-21 of the largest have all of them.
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static constexpr uint32_t FMT = 1;
    static constexpr float LIFT = 0.f;
};
template <> struct Elem<__half> {
    static constexpr uint32_t FMT = 0;
    static constexpr float LIFT = 7.f;
};

// Map of 16-bit elements with a 128-byte inner box, swizzled at that width.
template <int N>
inline CUresult make_map(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[N],
                  const cuuint64_t (&strides)[N - 1], const cuuint32_t (&box)[N]) {
    auto enc = tensor_map_encoder();
    if (!enc) return CUDA_ERROR_NOT_SUPPORTED;
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, N, const_cast<void*>(base), dims, strides, box,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace idx
