// The private parts of the decode attention: a request's rows of a key head against its own
// cached keys, on warp-level matrix instructions (at most 16 rows read a key: bound by HBM,
// not by the tensor cores).  Each part leaves m + log2(sum) and its normalised o.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.cuh"
#include "common.cuh"

namespace idx {

namespace {

constexpr int kPartWarps = 4;
constexpr int kStep = 16;    // keys a warp takes at a time; pages hold at least as many
constexpr int kStages = 2;   // steps in flight per warp

IDX_DEVI float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-byte asynchronous copy; bytes = 0 writes zeros and reads nothing
IDX_DEVI void cp_async16_zfill(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
IDX_DEVI void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> IDX_DEVI void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

IDX_DEVI void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
IDX_DEVI void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
    static IDX_DEVI void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static IDX_DEVI uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};
template <> struct Mma<__half> {
    static IDX_DEVI void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static IDX_DEVI uint32_t pack(float lo, float hi) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};

// Shared memory of a part: per warp a ring of kStages steps of K and V, rows of D
// elements whose 16-byte chunks are xor-ed with the row's low bits (ldmatrix reads
// eight rows at one chunk without bank conflicts).  The ring is reused for the join.
template <int D> constexpr int part_smem() { return kPartWarps * kStages * 2 * kStep * D * 2; }

// Parts of a call: requests x row blocks x key heads x splits, the splits next to each other.
__host__ __device__ inline long long private_parts(const AttnArgs& a) {
    return (long long)a.B * ((a.Q * a.G + 15) / 16) * a.Hkv * a.private_splits;
}

// One private part: 16 rows against a request's keys [lo, hi), by kPartWarps warps that
// `sync` brings together.  The warps take the 16-key steps in turn, each with its own softmax
// state; the states are joined at the end.
template <typename T, int D, typename Sync>
IDX_DEVI void private_part(const AttnArgs& a, int item, uint8_t* smem, int tid, const Sync& sync) {
    const int lane = tid & 31, warp = tid >> 5;
    const int split = item % a.private_splits;
    const int hk = item / a.private_splits % a.Hkv;
    const int row_blocks = (a.Q * a.G + 15) / 16;
    const int rb = item / a.private_splits / a.Hkv % row_blocks;
    const int b = item / a.private_splits / a.Hkv / row_blocks;
    const int rows = a.Q * a.G;
    const int total_splits = a.prefix_splits + a.private_splits;
    const int slot = a.prefix_splits + split;

    const int lo = split * a.private_chunk;
    const int* table = a.table + (long long)b * a.table_stride;
    // The length, the first pages and q are on their way together: the pages are looked up to
    // max_len, which the table covers.
    int n = a.lens[b];
    int pages_from = 0, page_of = 0;  // 32 steps of this warp at a time, one per lane
    const int far = min(a.max_len, lo + a.private_chunk);
    auto look_up = [&](int i) {
        pages_from = i;
        const int at = lo + ((i + lane) * kPartWarps + warp) * kStep;
        page_of = at < far ? table[at >> a.page_shift] : 0;
    };
    look_up(0);

    // row i of the block: query token t, head g of the group
    auto query_row = [&](int i) {
        const int r = rb * 16 + i, t = r / a.G;
        return ((long long)b * a.Q + t) * a.Hq + hk * a.G + (r - t * a.G);
    };
    const int r0 = rb * 16 + lane / 4, r1 = r0 + 8;  // this thread's two rows
    const bool live0 = r0 < rows, live1 = r1 < rows;
    uint32_t qf[D / 16][4];
    {
        const T* q = static_cast<const T*>(a.q);
        const T* p0 = q + (live0 ? query_row(lane / 4) : 0) * D + (lane % 4) * 2;
        const T* p1 = q + (live1 ? query_row(lane / 4 + 8) : 0) * D + (lane % 4) * 2;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            qf[k][0] = live0 ? *reinterpret_cast<const uint32_t*>(p0 + k * 16) : 0u;
            qf[k][1] = live1 ? *reinterpret_cast<const uint32_t*>(p1 + k * 16) : 0u;
            qf[k][2] = live0 ? *reinterpret_cast<const uint32_t*>(p0 + k * 16 + 8) : 0u;
            qf[k][3] = live1 ? *reinterpret_cast<const uint32_t*>(p1 + k * 16 + 8) : 0u;
        }
    }

    if ((n < 0 || n > a.max_len) && tid == 0) raise_status(a.d_status, IDX_DEV_RANGE);
    n = min(max(n, 0), a.max_len);
    const int hi = min(n, lo + a.private_chunk);
    if (lo >= hi) {  // no keys in this part
        for (int i = tid; i < 16 && rb * 16 + i < rows; i += kPartWarps * 32)
            a.part_lse[query_row(i) * total_splits + slot] = -INFINITY;
        return;
    }
    // keys a row sees: all but the tokens after its own
    const int see0 = live0 ? n - (a.Q - 1 - r0 / a.G) : 0;
    const int see1 = live1 ? n - (a.Q - 1 - r1 / a.G) : 0;

    constexpr int kRowBytes = D * 2, kChunks = D / 8, kTile = kStep * kRowBytes;
    const uint32_t ring = smem_u32(smem) + warp * kStages * 2 * kTile;
    const int steps = (hi - lo + kStep - 1) / kStep;
    const int mine = warp < steps ? (steps - 1 - warp) / kPartWarps + 1 : 0;
    bool bad = false;
    auto fetch = [&](int i) {
        if (i - pages_from >= 32) look_up(i);
        const int page = __shfl_sync(~0u, page_of, i - pages_from);
        const bool ok = page >= 0 && page < a.pages;
        bad |= !ok;
        const int key = lo + (i * kPartWarps + warp) * kStep;
        const long long row = ((long long)(ok ? page : 0) * a.Hkv + hk) * a.page_size +
                              (key & (a.page_size - 1));
        const uint8_t* kp = static_cast<const uint8_t*>(a.k) + row * kRowBytes;
        const uint8_t* vp = static_cast<const uint8_t*>(a.v) + row * kRowBytes;
        const uint32_t dst = ring + (i % kStages) * 2 * kTile;
#pragma unroll
        for (int j = 0; j < kStep * kChunks / 32; ++j) {
            const int c = j * 32 + lane, rr = c / kChunks, cc = c % kChunks;
            const uint32_t off = rr * kRowBytes + ((cc ^ (rr & 7)) * 16);
            const uint32_t bytes = ok && key + rr < hi ? 16u : 0u;  // zeros past the end
            cp_async16_zfill(dst + off, kp + rr * kRowBytes + cc * 16, bytes);
            cp_async16_zfill(dst + kTile + off, vp + rr * kRowBytes + cc * 16, bytes);
        }
    };

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float* logits = nullptr;
    if (a.logits)
        logits = a.logits + ((long long)b * a.Hkv + hk) * (a.Q * a.G) * a.logit_stride;

    for (int i = 0; i < kStages - 1; ++i) {
        if (i < mine) fetch(i);
        cp_async_commit();
    }
    for (int i = 0; i < mine; ++i) {
        if (i + kStages - 1 < mine) fetch(i + kStages - 1);
        cp_async_commit();
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint32_t kt = ring + (i % kStages) * 2 * kTile, vt = kt + kTile;
        const int key = lo + (i * kPartWarps + warp) * kStep;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            // matrices: keys 0-7 and 8-15, each at d 16k .. and 16k + 8 ..
            const int rr = (lane & 7) + ((lane >> 4) & 1) * 8, cc = 2 * k + ((lane >> 3) & 1);
            uint32_t f[4];
            ldsm4(kt + rr * kRowBytes + ((cc ^ (rr & 7)) * 16), f);
            Mma<T>::run(s[0], qf[k], f[0], f[1]);
            Mma<T>::run(s[1], qf[k], f[2], f[3]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = key + t * 8 + (lane % 4) * 2 + j;
                s[t][j] = c < hi && c < see0 ? s[t][j] * a.scale_log2 : -INFINITY;
                s[t][j + 2] = c < hi && c < see1 ? s[t][j + 2] * a.scale_log2 : -INFINITY;
            }
        if (logits) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int c = key + t * 8 + (lane % 4) * 2;
                if (live0)
                    *reinterpret_cast<float2*>(logits + r0 * a.logit_stride + c) =
                        make_float2(s[t][0], s[t][1]);
                if (live1)
                    *reinterpret_cast<float2*>(logits + r1 * a.logit_stride + c) =
                        make_float2(s[t][2], s[t][3]);
            }
        }
        float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, 2));
        if (__any_sync(~0u, x0 > m0 || x1 > m1)) {
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float f0 = n0 == -INFINITY ? 1.f : exp2_approx(m0 - n0);
            const float f1 = n1 == -INFINITY ? 1.f : exp2_approx(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                o[d][0] *= f0;
                o[d][1] *= f0;
                o[d][2] *= f1;
                o[d][3] *= f1;
            }
        }
        // rows that have seen no key yet keep m = -inf: their weights are 0
        const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t][0] = exp2_approx(s[t][0] - b0);
            s[t][1] = exp2_approx(s[t][1] - b0);
            s[t][2] = exp2_approx(s[t][2] - b1);
            s[t][3] = exp2_approx(s[t][3] - b1);
            l0 += s[t][0] + s[t][1];
            l1 += s[t][2] + s[t][3];
        }
        const uint32_t p[4] = {Mma<T>::pack(s[0][0], s[0][1]), Mma<T>::pack(s[0][2], s[0][3]),
                               Mma<T>::pack(s[1][0], s[1][1]), Mma<T>::pack(s[1][2], s[1][3])};
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            // matrices: keys 0-7 and 8-15 at d 16d .., then at 16d + 8 ..
            const int rr = lane & 15, cc = 2 * d + (lane >> 4);
            uint32_t f[4];
            ldsm4_t(vt + rr * kRowBytes + ((cc ^ (rr & 7)) * 16), f);
            Mma<T>::run(o[2 * d], p, f[0], f[1]);
            Mma<T>::run(o[2 * d + 1], p, f[2], f[3]);
        }
        __syncwarp();
    }
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
    l0 += __shfl_xor_sync(~0u, l0, 1);
    l1 += __shfl_xor_sync(~0u, l1, 1);
    l0 += __shfl_xor_sync(~0u, l0, 2);
    l1 += __shfl_xor_sync(~0u, l1, 2);

    // join the warps' states through shared memory
    cp_async_wait<0>();
    sync();
    float* so = reinterpret_cast<float*>(smem);           // [warps][16][D + 4]
    constexpr int kPitch = D + 4;
    float* sm = so + kPartWarps * 16 * kPitch;             // [warps][16] maxima, then sums
    float* sl = sm + kPartWarps * 16;
#pragma unroll
    for (int d = 0; d < D / 8; ++d) {
        float* p = so + (warp * 16 + lane / 4) * kPitch + d * 8 + (lane % 4) * 2;
        *reinterpret_cast<float2*>(p) = make_float2(o[d][0], o[d][1]);
        *reinterpret_cast<float2*>(p + 8 * kPitch) = make_float2(o[d][2], o[d][3]);
    }
    if (lane % 4 == 0) {
        sm[warp * 16 + lane / 4] = m0;
        sm[warp * 16 + lane / 4 + 8] = m1;
        sl[warp * 16 + lane / 4] = l0;
        sl[warp * 16 + lane / 4 + 8] = l1;
    }
    sync();
    for (int i = tid; i < 16 * (D / 4); i += kPartWarps * 32) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        if (rb * 16 + r >= rows) break;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kPartWarps; ++w) m = fmaxf(m, sm[w * 16 + r]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPartWarps; ++w) {
            const float f = exp2_approx(sm[w * 16 + r] - base);
            const float4 x = *reinterpret_cast<const float4*>(so + (w * 16 + r) * kPitch + d);
            l += f * sl[w * 16 + r];
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const long long at = query_row(r) * total_splits + slot;
        *reinterpret_cast<float4*>(a.part + at * D + d) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (d == 0) a.part_lse[at] = l > 0.f ? m + log2f(l) : -INFINITY;
    }
}

}  // namespace

}  // namespace idx
