// New keys and values into a paged MXFP4 cache.
//
// A block of 32 elements of a row gets the scale 2^e, e = floor(log2 max|x|) - 2 (so that the
// largest lies in [4, 8) under it; e >= -127, and 0 for a block of zeros), and the e2m1 codes
// nearest to x / 2^e, ties to the even code, saturated at 6.  2^-e is a power of two and x has at
// most 11 significant bits, so x * 2^-e and with it every code is exact.
//
// HBM-bound: 16-bit rows in, 17/64 of them out.  A warp takes a token's row: a lane holds 8
// elements (one 16-byte load, one 4-byte store), four lanes a block; K and V together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "cache_append.cuh"
#include "serve.cuh"

namespace idx {

namespace {

constexpr int kAppendThreads = 128;

// Four lanes' 8 elements each, one block: this lane's codes, and the block's scale.
template <typename T> IDX_DEVI uint32_t quantise8(const uint4& raw, uint32_t& sf) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
    uint32_t top = 0;  // of the magnitudes' bits
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        top = max(top, max(__float_as_uint(x[2 * i]) & 0x7fffffffu, __float_as_uint(x[2 * i + 1]) & 0x7fffffffu));
    }
    top = max(top, __shfl_xor_sync(~0u, top, 1));
    top = max(top, __shfl_xor_sync(~0u, top, 2));
    const int ex = (int)(top >> 23);
    if (ex == 255) {  // not finite: the block is NaN
        sf = 255u;
        return 0u;
    }
    const int e = top == 0 ? 127 : max(ex - 2, 0);
    sf = (uint32_t)e;
    const float f = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^-(e - 127); e is at most 252
    uint32_t codes;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(codes)
        : "f"(x[0] * f), "f"(x[1] * f), "f"(x[2] * f), "f"(x[3] * f), "f"(x[4] * f), "f"(x[5] * f), "f"(x[6] * f),
          "f"(x[7] * f));
    return codes;
}

// The request of a token: how many of q_start[1 .. B] are at most it, by a warp, 32 of them at a time.
IDX_DEVI int request_of(const int* q_start, int B, int token, int lane) {
    int lo = 0, hi = B;  // in (lo, hi], counted from 1: all before are at most the token
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const bool below = at <= hi && q_start[at] <= token;
        const int n = __popc(__ballot_sync(~0u, below));
        lo += n * step;
        if (step == 1) break;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int token = (int)(((long long)blockIdx.x * kAppendThreads + threadIdx.x) >> 5);
    if (token >= a.T) return;
    const int per_head = a.D / 8, shift = a.D == 128 ? 4 : 3, units = a.Hkv * per_head;
    const T* k = static_cast<const T*>(a.k) + token * a.k_stride;
    const T* v = static_cast<const T*>(a.v) + token * a.v_stride;
    auto load = [&](const T* x, int u) {
        uint4 r;
        if constexpr (WIDE) {
            r = *reinterpret_cast<const uint4*>(x + u * 8);
        } else {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(x) + u * 8;
            r.x = e[0] | (uint32_t)e[1] << 16;
            r.y = e[2] | (uint32_t)e[3] << 16;
            r.z = e[4] | (uint32_t)e[5] << 16;
            r.w = e[6] | (uint32_t)e[7] << 16;
        }
        return r;
    };
    // units is a multiple of 8 (D >= 64): four lanes of a block are in it together
    constexpr int kDeep = WIDE ? 4 : 1;
    uint4 rk[kDeep], rv[kDeep];
    auto load_from = [&](int u0) {
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int u = u0 + i * 32 + lane;
            rk[i] = u < units ? load(k, u) : make_uint4(0u, 0u, 0u, 0u);
            rv[i] = u < units ? load(v, u) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    // where the token goes takes a chain of loads: the row's first elements are on their way meanwhile (35k
    // tokens 47 us with the chain first)
    int b = 0, end = a.T, first = 0;
    if (a.q_start && (token < a.q_start[0] || token >= a.q_start[a.B])) return;  // of no request
    load_from(0);
    if (a.q_start) {
        b = request_of(a.q_start, a.B, token, lane);
        if (b >= a.B) return;  // (q_start out of order)
        first = a.q_start[b];
        end = a.q_start[b + 1];
    } else {
        const int per = a.T / a.B;
        b = token / per;
        end = (b + 1) * per;
    }
    const long long at = (long long)a.lens[b] - end + token;  // position of the token
    // (a request that ends behind the call's tokens: where they belong is not known)
    if (token < first || end > a.T || at < 0 || at >= a.table_stride << a.page_shift) {
        if (lane == 0) raise_status(a.d_status, IDX_DEV_RANGE);
        return;
    }
    const int page = a.table[b * a.table_stride + (at >> a.page_shift)];
    if (page < 0) return;  // a page that is not kept
    if (page >= a.pages) {
        if (lane == 0) raise_status(a.d_status, IDX_DEV_RANGE);
        return;
    }
    const long long row0 = (long long)page * a.Hkv * a.page_size + (at & (a.page_size - 1));
    for (int u0 = 0; u0 < units; u0 += 32 * kDeep) {
        if (u0 > 0) load_from(u0);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int u = u0 + i * 32 + lane;
            uint32_t sk, sv;
            const uint32_t ck = quantise8<T>(rk[i], sk), cv = quantise8<T>(rv[i], sv);
            if (u < units) {
                const int h = u >> shift, d8 = u & (per_head - 1);
                const long long row = row0 + (long long)h * a.page_size;
                reinterpret_cast<uint32_t*>(a.k_codes)[row * per_head + d8] = ck;
                reinterpret_cast<uint32_t*>(a.v_codes)[row * per_head + d8] = cv;
                if ((d8 & 3) == 0) {
                    a.k_sf[row * (per_head / 4) + d8 / 4] = (uint8_t)sk;
                    a.v_sf[row * (per_head / 4) + d8 / 4] = (uint8_t)sv;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, idx_dtype dt, bool wide, cudaStream_t s) {
    const auto kern = dt == IDX_BF16 ? (wide ? append_kernel<__nv_bfloat16, true> : append_kernel<__nv_bfloat16, false>)
                                     : (wide ? append_kernel<__half, true> : append_kernel<__half, false>);
    const long long per = kAppendThreads / 32, blocks = ((long long)a.T + per - 1) / per;
    return launch_k(kern, dim3((unsigned)blocks), dim3(kAppendThreads), 0, s, true, a);
}

}  // namespace idx
