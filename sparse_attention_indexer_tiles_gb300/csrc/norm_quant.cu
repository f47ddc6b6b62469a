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

#include "common.cuh"
#include "norm_quant.cuh"

namespace idx {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

template <typename T> struct Vec8;  // 8 consecutive elements
template <> struct Vec8<float> { float4 a, b; };
template <> struct Vec8<__nv_bfloat16> { uint4 a; };
template <> struct Vec8<__half> { uint4 a; };

IDX_DEVI float to_f(float v) { return v; }
IDX_DEVI float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
IDX_DEVI float to_f(__half v) { return __half2float(v); }
template <typename T> IDX_DEVI T from_f(float v);
template <> IDX_DEVI float from_f<float>(float v) { return v; }
template <> IDX_DEVI __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> IDX_DEVI __half from_f<__half>(float v) { return __float2half_rn(v); }

// n valid elements at p (fewer than 8 only on the element-wise path)
template <typename T, bool VEC>
IDX_DEVI void load8(const T* p, int n, float (&v)[8]) {
    if constexpr (VEC) {
        const Vec8<T> raw = *reinterpret_cast<const Vec8<T>*>(p);
        const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
    }
}

template <typename T, bool VEC>
IDX_DEVI void store8(T* p, int n, const float (&v)[8]) {
    if constexpr (VEC) {
        Vec8<T> raw;
        T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = from_f<T>(v[i]);
        *reinterpret_cast<Vec8<T>*>(p) = raw;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f<T>(v[i]);
    }
}

template <bool VEC>
IDX_DEVI void store_codes(uint8_t* p, int n, const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                     __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
}

// TPR threads per row, VPT vectors of 8 columns per thread; a block of
// max(TPR, 128) threads.
template <typename T, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_quant_kernel(NormArgs a) {
    constexpr int kThreads = TPR < 128 ? 128 : TPR;
    constexpr int kRows = kThreads / TPR;
    const int t = (int)threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * kRows + (int)threadIdx.x / TPR;
    const bool live = row < a.rows;
    float h[VPT][8], hw[VPT][8];
    float sum = 0.f, most = 0.f;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = static_cast<const T*>(a.residual) + row * a.N;
    T* res_out = static_cast<T*>(a.residual_out) + row * a.N;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (v * TPR + t) * 8;
        if (live && c < a.N) {
            load8<T, VEC>(x + c, a.N - c, h[v]);
            if (a.residual) {
                float r[8];
                load8<T, VEC>(res + c, a.N - c, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[v][i] += r[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] = 0.f;
        }
    }
    float gmost[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (v * TPR + t) * 8;
        gmost[v] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) hw[v][i] = 0.f;
        if (c < a.N) {
            load8<T, VEC>(static_cast<const T*>(a.weight) + c, a.N - c, hw[v]);
            if (live && a.residual_out) store8<T, VEC>(res_out + c, a.N - c, h[v]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = fmaf(h[v][i], h[v][i], sum);
            hw[v][i] *= h[v][i];
            gmost[v] = fmaxf(gmost[v], fabsf(hw[v][i]));
        }
        most = fmaxf(most, gmost[v]);
    }
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o /= 2) {
        sum += __shfl_xor_sync(~0u, sum, o);
        most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
    }
    if constexpr (TPR > 32) {
        __shared__ float s_sum[TPR / 32], s_most[TPR / 32];
        if ((threadIdx.x & 31) == 0) {
            s_sum[threadIdx.x / 32] = sum;
            s_most[threadIdx.x / 32] = most;
        }
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) {  // the same order in every thread
            sum += s_sum[i];
            most = fmaxf(most, s_most[i]);
        }
    }
    const float rstd = rsqrtf(sum / (float)a.N + a.eps);
    if (a.group == 0) {
        const float scale = fmaxf(rstd * most / kE4m3Max, kScaleFloor);
        if (live && t == 0) a.scale[row] = scale;
        const float f = rstd / scale;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) hw[v][i] *= f;
    } else {
        const int lanes = a.group / 8;  // consecutive threads of a group: 4, 8 or 16
        const int groups = a.N / a.group;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float m = gmost[v];
            for (int o = lanes / 2; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
            const float scale = fmaxf(rstd * m / kE4m3Max, kScaleFloor);
            const int c = (v * TPR + t) * 8;
            if (live && c < a.N && t % lanes == 0) a.scale[row * groups + c / a.group] = scale;
            const float f = rstd / scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) hw[v][i] *= f;
        }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = (v * TPR + t) * 8;
        if (live && c < a.N) store_codes<VEC>(a.out + row * a.N + c, a.N - c, hw[v]);
    }
}

template <typename T, int TPR, int VPT>
cudaError_t launch_shape(const NormArgs& a, cudaStream_t s) {
    constexpr int kThreads = TPR < 128 ? 128 : TPR;
    const int grid = (int)(((long long)a.rows * TPR + kThreads - 1) / kThreads);
    if (a.vec)
        norm_quant_kernel<T, TPR, VPT, true><<<grid, kThreads, 0, s>>>(a);
    else
        norm_quant_kernel<T, TPR, VPT, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const NormArgs& a, cudaStream_t s) {
    if (a.N <= 128) return launch_shape<T, 16, 1>(a, s);
    if (a.N <= 256) return launch_shape<T, 32, 1>(a, s);
    if (a.N <= 1024) return launch_shape<T, 128, 1>(a, s);
    if (a.N <= 2048) return launch_shape<T, 256, 1>(a, s);
    if (a.N <= 4096) return launch_shape<T, 512, 1>(a, s);
    if (a.N <= 8192) return launch_shape<T, 1024, 1>(a, s);
    if (a.N <= 16384) return launch_shape<T, 1024, 2>(a, s);
    return launch_shape<T, 1024, 4>(a, s);
}

}  // namespace

cudaError_t launch_norm_quant(const NormArgs& a, idx_dtype dt, int sm_count, cudaStream_t s) {
    (void)sm_count;
    if (dt == IDX_BF16) return launch_type<__nv_bfloat16>(a, s);
    if (dt == IDX_FP16) return launch_type<__half>(a, s);
    return launch_type<float>(a, s);
}

}  // namespace idx
