// h = x + residual; y = h * rsqrt(mean(h^2) + eps) * weight; e4m3 codes of y with
// one fp32 scale per row or per group of columns:
//
//     scale = max(max|y| / 448, 2^-100),   code = e4m3(y / scale)
//
// (448 is the largest e4m3 value; the floor keeps the scale of a row of zeros
// positive, as the scorer's k_scale has to be).  h stays in fp32 between its sum
// and the code; it is rounded to the tensor's type only where it is stored.
//
// One pass: a row lives in the registers of its threads, 8 consecutive columns per
// vector.  rsqrt(mean) is a positive factor common to the row, so max|y| is that
// factor times max|h * weight|, and the sum of squares and the maximum are reduced
// together behind one barrier.  HBM-bound: each input is read once, each output
// written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cfloat>
#include <cmath>
#include <mutex>

#include "norm_quant.cuh"
#include "serve.cuh"

namespace idx {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

// The largest magnitude, NaN when one is.
IDX_DEVI float max_abs_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 8 consecutive columns as they lie in memory, taken as four pairs of fp32.
template <typename T> struct alignas(16) Raw8 {  // 16-bit types
    uint32_t u[4];
    IDX_DEVI void clear() { u[0] = u[1] = u[2] = u[3] = 0u; }
    IDX_DEVI float2 pair(int i) const;
    IDX_DEVI void set(int i, float2 v);
};
template <> IDX_DEVI float2 Raw8<__nv_bfloat16>::pair(int i) const {
    return make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
template <> IDX_DEVI void Raw8<__nv_bfloat16>::set(int i, float2 v) {
    u[i] = pack2<__nv_bfloat16>(v.x, v.y);
}
template <> IDX_DEVI float2 Raw8<__half>::pair(int i) const {
    return __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
}
template <> IDX_DEVI void Raw8<__half>::set(int i, float2 v) {
    u[i] = pack2<__half>(v.x, v.y);
}
template <> struct alignas(16) Raw8<float> {
    float f[8];
    IDX_DEVI void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
    }
    IDX_DEVI float2 pair(int i) const { return make_float2(f[2 * i], f[2 * i + 1]); }
    IDX_DEVI void set(int i, float2 v) {
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
};

// A thread's eight columns of a row, in accesses of U columns: eight consecutive ones (U = 8),
// or every `step`-th pair or single column from the c-th on, so that a warp's accesses are
// consecutive when rows are not on 16-byte boundaries.  `have` of its accesses are inside the
// row.
template <typename T, int U> struct Unit;  // U columns as they are loaded
template <> struct Unit<float, 2> { using type = float2; };
template <> struct Unit<__nv_bfloat16, 2> { using type = uint32_t; };
template <> struct Unit<__half, 2> { using type = uint32_t; };
template <typename T> struct Unit<T, 8> { using type = Raw8<T>; };
template <typename T> struct Unit<T, 1> { using type = T; };

template <int U, typename T>
IDX_DEVI void load8(Raw8<T>& r, const T* row, int c, int step, int have) {
    using V = typename Unit<T, U>::type;
#pragma unroll
    for (int i = 0; i < 8 / U; ++i)
        if (i < have)
            reinterpret_cast<V*>(&r)[i] = *reinterpret_cast<const V*>(row + (c + i * step) * U);
}
template <int U, typename T>
IDX_DEVI void store8(T* row, const Raw8<T>& r, int c, int step, int have) {
    using V = typename Unit<T, U>::type;
#pragma unroll
    for (int i = 0; i < 8 / U; ++i)
        if (i < have)
            *reinterpret_cast<V*>(row + (c + i * step) * U) = reinterpret_cast<const V*>(&r)[i];
}
template <int U>
IDX_DEVI void store_codes(uint8_t* row, const float2 (&v)[4], int c, int step, int have) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __nv_cvt_float2_to_fp8x2(v[i], __NV_SATFINITE, __NV_E4M3);
#pragma unroll
    for (int i = 0; i < 8 / U; ++i) {
        if (i >= have) break;
        uint8_t* at = row + (c + i * step) * U;
        if constexpr (U == 8)
            *reinterpret_cast<uint2*>(at) = make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
        else if constexpr (U == 2)
            *reinterpret_cast<uint16_t*>(at) = (uint16_t)p[i];
        else
            *at = (uint8_t)(p[i >> 1] >> (8 * (i & 1)));
    }
}

// TPR threads per row, VPT vectors of 8 columns per thread, blocks of max(TPR, 128)
// threads.  A block takes every gridDim.x-th group of rows and has the next one's x and
// residual on their way while it works on the current one.  Columns and rows past the end
// are zeros.  The arithmetic is on pairs of fp32: at 16-bit inputs the instructions per
// element, not HBM, bound the first version (44 per element, 62 us at 4096 x 8192).
// (16-bit rows of 128 threads: ten blocks per SM; at nine, which the compiler's own choice of
// registers allows, 3001 x 926 takes 5.5 us instead of 5.1.)
template <typename T, int TPR, int VPT, int U, bool RES>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, TPR == 128 && sizeof(T) == 2 ? 10 : 0)
norm_quant_kernel(NormArgs a) {
    constexpr int kThreads = TPR < 128 ? 128 : TPR;
    constexpr int kRows = kThreads / TPR;  // rows side by side in a block
    constexpr int kWarps = TPR / 32;       // warps of a row, where it has several
    // Launched while the kernel before it ends (1 x 4096: 4.1 -> 3.0 us a call, 65536 x 128: 8.2
    // -> 6.1); letting the next launch begin early as well cost the latter 0.5.
    pdl_wait();
    const int t = (int)threadIdx.x % TPR, lane = threadIdx.x & 31;
    const int units = (a.rows - 1) / kRows + 1;
    auto row_of = [&](int u) { return (long long)u * kRows + (int)threadIdx.x / TPR; };
    // vector v's first access, in units of U columns, and how many of its 8 / U are in the row
    auto unit_of = [&](int v) { return v * (8 / U) * TPR + t; };
    int have[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int left = a.N / U - unit_of(v);
        have[v] = left <= 0 ? 0 : min(8 / U, (left + TPR - 1) / TPR);
    }
    struct Row {
        Raw8<T> x[VPT], res[RES ? VPT : 1];
    };
    auto fetch = [&](Row& r, int u) {
        const long long row = row_of(u);
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* res = static_cast<const T*>(a.residual) + row * a.N;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            r.x[v].clear();
            if constexpr (RES) r.res[v].clear();
            if (row < a.rows) {
                load8<U>(r.x[v], x, unit_of(v), TPR, have[v]);
                if constexpr (RES) load8<U>(r.res[v], res, unit_of(v), TPR, have[v]);
            }
        }
    };
    Row next;
    fetch(next, blockIdx.x);
    Raw8<T> wgt[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        wgt[v].clear();
        load8<U>(wgt[v], static_cast<const T*>(a.weight), unit_of(v), TPR, have[v]);
    }
    const float per_col = 1.f / (float)a.N;
    const int lanes = a.group / 8;  // consecutive threads of a group: 4, 8 or 16
    for (int u = blockIdx.x, it = 0; u < units; u += gridDim.x, ++it) {
        const Row cur = next;
        if (u + (int)gridDim.x < units) fetch(next, u + gridDim.x);
        const long long row = row_of(u);
        const bool row_live = row < a.rows;
        float2 hw[VPT][4], sum2 = make_float2(0.f, 0.f);
        float gmost[VPT], most = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            Raw8<T> h_out;
            gmost[v] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 h = cur.x[v].pair(i);
                if constexpr (RES) h = add2(h, cur.res[v].pair(i));
                sum2 = fma2(h, h, sum2);
                hw[v][i] = mul2(h, wgt[v].pair(i));
                gmost[v] = max_abs_nan(gmost[v], hw[v][i].x, hw[v][i].y);
                h_out.set(i, h);
            }
            if (a.residual_out && row_live)
                store8<U>(static_cast<T*>(a.residual_out) + row * a.N, h_out, unit_of(v), TPR, have[v]);
            most = max_nan(most, gmost[v]);
        }
        float sum = sum2.x + sum2.y;
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o /= 2) {
            sum += __shfl_xor_sync(~0u, sum, o);
            most = max_nan(most, __shfl_xor_sync(~0u, most, o));
        }
        if constexpr (TPR > 32) {
            __shared__ float2 part[2][kWarps];  // two: a block's barrier per row group is enough
            if (lane == 0) part[it & 1][threadIdx.x / 32] = make_float2(sum, most);
            __syncthreads();
            constexpr int kSpan = kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : kWarps <= 16 ? 16 : 32;
            const bool there = lane % kSpan < kWarps;
            sum = there ? part[it & 1][lane % kSpan].x : 0.f;
            most = there ? part[it & 1][lane % kSpan].y : 0.f;
#pragma unroll
            for (int o = kSpan / 2; o > 0; o /= 2) {  // the same sum in every thread
                sum += __shfl_xor_sync(~0u, sum, o);
                most = max_nan(most, __shfl_xor_sync(~0u, most, o));
            }
        }
        // Where the squares leave fp32 (|h| from about 2^63 on; without eps, all |h| below 2^-63) there
        // is no rstd: NaN, so that the row cannot pass for one.  An infinite mean times 0 is NaN.
        const float mean = fmaf(sum, per_col, a.eps);
        float rstd = rsqrtf(fmaf(mean, 0.f, mean));
        if (mean < 0x1p-56f) {  // 448 / max|h weight| could be infinite below: h times 2^64
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
#pragma unroll
                for (int i = 0; i < 4; ++i) hw[v][i] = mul2(hw[v][i], make_float2(0x1p64f, 0x1p64f));
                gmost[v] *= 0x1p64f;
            }
            most *= 0x1p64f;
            rstd = mean >= FLT_MIN ? rstd * 0x1p-64f : NAN;
        }
        const float row_scale = max_nan(rstd * most * (1.f / kE4m3Max), kScaleFloor);
        if (a.group == 0 && row_live && t == 0) a.scale[row] = row_scale;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float scale = row_scale, top = most;
            if (U == 8 && a.group != 0) {
                float m = gmost[v];
                if (lanes > 8) m = max_nan(m, __shfl_xor_sync(~0u, m, 8));
                if (lanes > 4) m = max_nan(m, __shfl_xor_sync(~0u, m, 4));
                m = max_nan(m, __shfl_xor_sync(~0u, m, 2));
                m = max_nan(m, __shfl_xor_sync(~0u, m, 1));
                scale = max_nan(rstd * m * (1.f / kE4m3Max), kScaleFloor);
                top = m;
                if (row_live && have[v] > 0 && (t & (lanes - 1)) == 0)
                    a.scale[row * (a.N / a.group) + unit_of(v) * 8 / a.group] = scale;
            }
            // y / scale = h weight (rstd / scale), and rstd cancels unless the scale is its floor:
            // 448 / max|h weight| has one rounding where rstd / scale has four.  (Where |h weight| is
            // 3/4, 3/8, .. of the largest, the quotient is halfway between two codes, and these
            // roundings decide, as the one of the scale would in y / scale.)
            const float f = scale > kScaleFloor ? __fdiv_rn(kE4m3Max, top)
                                                : fmaf(top, 0.f, rstd) / kScaleFloor;  // NaN of either stays
#pragma unroll
            for (int i = 0; i < 4; ++i) hw[v][i] = mul2(hw[v][i], make_float2(f, f));
            if (row_live) store_codes<U>(a.out + row * a.N, hw[v], unit_of(v), TPR, have[v]);
        }
    }
}

template <typename T, int TPR, int VPT, int U, bool RES>
cudaError_t launch_blocks(const NormArgs& a, int sm_count, cudaStream_t s) {
    constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
    static std::once_flag once;
    static int resident = 1;  // blocks per SM
    std::call_once(once, [] {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                &resident, norm_quant_kernel<T, TPR, VPT, U, RES>, kThreads, 0) != cudaSuccess ||
            resident < 1)
            resident = 1;
    });
    // as many blocks as are resident, each with the same number of row groups
    const long long units = ((long long)a.rows + kRows - 1) / kRows;
    const long long room = (long long)resident * sm_count;
    const long long each = (units + room - 1) / room;
    const long long grid = (units + each - 1) / each;
    return launch_k(norm_quant_kernel<T, TPR, VPT, U, RES>, dim3((unsigned)grid), dim3(kThreads), 0,
                    s, true, a);
}

template <typename T, int TPR, int VPT>
cudaError_t launch_shape(const NormArgs& a, int sm_count, cudaStream_t s) {
    if (a.unit == 8)
        return a.residual ? launch_blocks<T, TPR, VPT, 8, true>(a, sm_count, s)
                          : launch_blocks<T, TPR, VPT, 8, false>(a, sm_count, s);
    if (a.unit == 2)
        return a.residual ? launch_blocks<T, TPR, VPT, 2, true>(a, sm_count, s)
                          : launch_blocks<T, TPR, VPT, 2, false>(a, sm_count, s);
    return a.residual ? launch_blocks<T, TPR, VPT, 1, true>(a, sm_count, s)
                      : launch_blocks<T, TPR, VPT, 1, false>(a, sm_count, s);
}

// Shapes: a narrow row is a half-warp's or a warp's (65536 x 256 bf16 by half-warps of two
// vectors a thread 11.1 us, by warps of one 13.4; 30000 x 512 by warps 11.0, by 128 threads
// 23.5).  A wide one's threads hold as many vectors as measured fastest (bf16 with residual:
// 8192 x 4096 with one 41.4 us, two 37.3, four 38.6; 777 x 5000 fp16 with one 7.5, two 5.3,
// three 5.7; 4096 x 8192 with one 44.4, two 43.4, four 37.9).  The last two rows and fp32 have the
// 16-bit rows' shapes and were not compared with others.  With residual, and of what HBM alone would
// take: 2048 x 16384 bf16 41 of 35 us, 8192 x 4096 fp32 69 of 64; where a thread's rows do not fit
// its registers much more: 2048 x 16384 fp32 93 of 64, 1000 x 32768 bf16 75 of 34, fp32 350 of 63.
template <typename T>
cudaError_t launch_type(const NormArgs& a, int sm_count, cudaStream_t s) {
    if (a.N <= 128) return launch_shape<T, 16, 1>(a, sm_count, s);
    if (a.N <= 256) return launch_shape<T, 16, 2>(a, sm_count, s);
    if (a.N <= 512) return launch_shape<T, 32, 2>(a, sm_count, s);
    if (a.N <= 1024) return launch_shape<T, 128, 1>(a, sm_count, s);
    if (a.N <= 2048) return launch_shape<T, 256, 1>(a, sm_count, s);
    if (a.N <= 4096) return launch_shape<T, 256, 2>(a, sm_count, s);
    if (a.N <= 6144) return launch_shape<T, 384, 2>(a, sm_count, s);
    if (a.N <= 8192) return launch_shape<T, 256, 4>(a, sm_count, s);
    if (a.N <= 16384) return launch_shape<T, 512, 4>(a, sm_count, s);
    return launch_shape<T, 1024, 4>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_norm_quant(const NormArgs& a, idx_dtype dt, int sm_count, cudaStream_t s) {
    if (dt == IDX_BF16) return launch_type<__nv_bfloat16>(a, sm_count, s);
    if (dt == IDX_FP16) return launch_type<__half>(a, sm_count, s);
    return launch_type<float>(a, sm_count, s);
}

}  // namespace idx
