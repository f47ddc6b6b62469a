// Decode attention of a batch over a shared prefix and private paged caches.
//
// For row r (one query token and head) over the prefix's keys and its request's own,
//     o = sum_j exp(z_j) v_j / sum_j exp(z_j),   z_j = scale * q . k_j,
//     lse = log sum_j exp(z_j).
// The keys of a row are cut into parts.  A part's rows are the rows that read the same
// keys: the query heads of a key head for a private part, those of the whole batch for
// a part of the prefix, so the prefix is read once however many requests share it.
// Each part leaves m + log2(sum) and its normalised o; the parts are joined by
//     o = sum_p 2^(l_p - L) o_p,   L = log2 sum_p 2^(l_p).
// All exponentials are base 2 on z * log2(e); sums, maxima and o are fp32, and the
// weights enter the second product in the tensors' own type (a relative rounding of
// half a step per weight, as V itself carries; in fp16 they are taken times a power of
// two, since its numbers below 2^-14 have fewer bits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attention.cuh"
#include "serve.cuh"

namespace idx {

namespace {

constexpr int kPartWarps = 4;
constexpr int kStep = 16;    // keys a warp takes at a time; pages hold at least as many
constexpr int kRing = 3;     // copies of 16 rows, of K and of V in turn, per warp

// 16-byte asynchronous copy; bytes = 0 writes zeros and reads nothing
IDX_DEVI void cp_async16_zfill(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}
// L2 policies: data that is not read again leaves first; the default.
IDX_DEVI uint64_t l2_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
IDX_DEVI uint64_t l2_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
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

// Transposes an 8x8 matrix of 16-bit elements held across the warp.
IDX_DEVI uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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
};
template <> struct Mma<__half> {
    static IDX_DEVI void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// Shared memory of a block: per warp a ring of kRing tiles of 16 keys, rows of D elements
// whose 16-byte chunks are xor-ed with the row's low bits (ldmatrix reads eight rows at one
// chunk without bank conflicts).  The ring is reused for the join.
template <int D> constexpr int part_smem() { return kPartWarps * kRing * kStep * D * 2; }

// One private part: 8 NT query rows against a request's keys [lo, hi).  The products are
// taken transposed, S^T = K Q^T and O^T += V^T P^T, so that the keys and D are the long axes
// of the matrix instructions and the rows, often 8 or fewer, the short one (with the rows on
// the long axis half of it was empty, at 163 registers and 12 warps per SM: the call of 64
// requests with 64-1024 keys behind a 32768-key prefix took 84 us instead of 80).
// The block's warps take the 16-key steps in turn, each with its own softmax state; the
// states are joined at the end.  blockIdx.x: row block, split and key head; blockIdx.y: the
// request.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kPartWarps * 32, NT == 1 ? 4 : 3) attn_part_kernel(AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    if (a.prefix_splits == 0) pdl_wait();  // the call's first launch
    pdl_trigger();
    // This grid reads nothing that the prefix's writes; one block's wait for it makes the
    // join's wait for this grid cover both.
    const bool last = blockIdx.x == 0 && blockIdx.y == 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kRows = 8 * NT;
    // fp16 weights are taken times 2^15, so that they have all their bits down to 2^-29 of the largest
    constexpr float kLift = std::is_same<T, __half>::value ? 15.f : 0.f;
    const int rows = a.Q * a.G;
    // row blocks next to each other: they read the same keys, from L2 but for the first
    const int row_blocks = (rows + kRows - 1) / kRows;
    const int rb = blockIdx.x % row_blocks, split = blockIdx.x / row_blocks % a.private_splits;
    const int hk = blockIdx.x / row_blocks / a.private_splits, b = blockIdx.y;
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
        const int r = rb * kRows + i, t = r / a.G;
        return ((long long)b * a.Q + t) * a.Hq + hk * a.G + (r - t * a.G);
    };
    // q as the products' second operand: row lane / 4 of each eight, pairs of columns
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int i = t * 8 + lane / 4;
        const bool live = rb * kRows + i < rows;
        const T* q = static_cast<const T*>(a.q) + (live ? query_row(i) : 0) * D + (lane % 4) * 2;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            qf[t][k][0] = live ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
            qf[t][k][1] = live ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
        }
    }

    if ((n < 0 || n > a.max_len) && tid == 0) raise_status(a.d_status, IDX_DEV_RANGE);
    n = min(max(n, 0), a.max_len);
    const int hi = min(n, lo + a.private_chunk);
    if (lo >= hi) {  // no keys in this part
        for (int i = tid; i < kRows && rb * kRows + i < rows; i += kPartWarps * 32)
            a.part_lse[query_row(i) * total_splits + slot] = -INFINITY;
        if (last) pdl_wait();
        return;
    }
    // This thread's columns of S^T and O^T: rows 2 (lane % 4) and the next of each eight.
    // A row sees all keys but those of the tokens after its own.
    int see[NT][2];
    bool live[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = rb * kRows + t * 8 + (lane % 4) * 2 + j;
            live[t][j] = r < rows;
            see[t][j] = min(hi, live[t][j] ? n - (a.Q - 1 - r / a.G) : 0);
        }

    constexpr int kRowBytes = D * 2, kChunks = D / 8, kTile = kStep * kRowBytes;
    const uint32_t ring = smem_u32(smem) + warp * kRing * kTile;
    const int steps = (hi - lo + kStep - 1) / kStep;
    const int mine = warp < steps ? (steps - 1 - warp) / kPartWarps + 1 : 0;
    bool bad = false;
    // K and V that one block reads pass through L2 without pushing out the logits and parts
    // that the join reads back
    const uint64_t policy = rows <= kRows ? l2_evict_first() : l2_evict_normal();
    // tile u: K of step u / 2, or V of it
    auto fetch = [&](int u) {
        const int i = u >> 1;
        if (i - pages_from >= 32) look_up(i);
        const int page = __shfl_sync(~0u, page_of, i - pages_from);
        const bool ok = page >= 0 && page < a.pages;
        bad |= !ok;
        const int key = lo + (i * kPartWarps + warp) * kStep;
        const long long row = ((long long)(ok ? page : 0) * a.Hkv + hk) * a.page_size +
                              (key & (a.page_size - 1));
        const uint8_t* src = static_cast<const uint8_t*>(u & 1 ? a.v : a.k) + row * kRowBytes;
        const uint32_t dst = ring + (u % kRing) * kTile;
#pragma unroll
        for (int j = 0; j < kStep * kChunks / 32; ++j) {
            const int c = j * 32 + lane, rr = c / kChunks, cc = c % kChunks;
            cp_async16_zfill(dst + rr * kRowBytes + ((cc ^ (rr & 7)) * 16),
                             src + rr * kRowBytes + cc * 16,
                             ok && key + rr < hi ? 16u : 0u, policy);  // zeros past the end
        }
    };

    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[t][j] = -INFINITY;
            l[t][j] = 0.f;
        }
    }
    float* logits = nullptr;
    if (a.logits)
        logits = a.logits + (((long long)b * a.Hkv + hk) * rows + rb * kRows) * a.logit_stride;

    for (int u = 0; u < 2; ++u) {
        if (u < 2 * mine) fetch(u);
        cp_async_commit();
    }
    for (int i = 0; i < mine; ++i) {
        if (i + 1 < mine) fetch(2 * i + 2);
        cp_async_commit();
        cp_async_wait<2>();
        __syncwarp();
        const uint32_t kt = ring + (2 * i % kRing) * kTile, vt = ring + ((2 * i + 1) % kRing) * kTile;
        const int key = lo + (i * kPartWarps + warp) * kStep + lane / 4;  // and key + 8
        float s[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            // matrices: keys 0-7 and 8-15 at d 16k .., then at 16k + 8 ..
            const int rr = lane & 15, cc = 2 * k + (lane >> 4);
            uint32_t f[4];
            ldsm4(kt + rr * kRowBytes + ((cc ^ (rr & 7)) * 16), f);
#pragma unroll
            for (int t = 0; t < NT; ++t) Mma<T>::run(s[t], f, qf[t][k][0], qf[t][k][1]);
        }
        __syncwarp();  // K has been read
        if (i + 1 < mine) fetch(2 * i + 3);
        cp_async_commit();
        uint32_t p[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            // s[0], s[1]: key, rows r and r + 1; s[2], s[3]: key + 8
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = key + (e >> 1) * 8;
                s[t][e] = at < see[t][e & 1] ? s[t][e] * a.scale_log2 : -INFINITY;
                if (logits && live[t][e & 1] && at < hi)
                    logits[(t * 8 + (lane % 4) * 2 + (e & 1)) * a.logit_stride + at] = s[t][e];
            }
            float x0 = fmaxf(s[t][0], s[t][2]), x1 = fmaxf(s[t][1], s[t][3]);
#pragma unroll
            for (int d = 4; d < 32; d *= 2) {
                x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, d));
                x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, d));
            }
            if (__any_sync(~0u, x0 > m[t][0] || x1 > m[t][1])) {
                const float n0 = fmaxf(m[t][0], x0), n1 = fmaxf(m[t][1], x1);
                const float f0 = n0 == -INFINITY ? 1.f : exp2_approx(m[t][0] - n0);
                const float f1 = n1 == -INFINITY ? 1.f : exp2_approx(m[t][1] - n1);
                m[t][0] = n0;
                m[t][1] = n1;
                l[t][0] *= f0;
                l[t][1] *= f1;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    o[t][d][0] *= f0;
                    o[t][d][1] *= f1;
                    o[t][d][2] *= f0;
                    o[t][d][3] *= f1;
                }
            }
            // rows that have seen no key yet keep m = -inf: their weights are 0
            const float b0 = m[t][0] == -INFINITY ? 0.f : m[t][0] - kLift;
            const float b1 = m[t][1] == -INFINITY ? 0.f : m[t][1] - kLift;
            s[t][0] = exp2_approx(s[t][0] - b0);
            s[t][1] = exp2_approx(s[t][1] - b1);
            s[t][2] = exp2_approx(s[t][2] - b0);
            s[t][3] = exp2_approx(s[t][3] - b1);
            l[t][0] += s[t][0] + s[t][2];
            l[t][1] += s[t][1] + s[t][3];
            // as the second operand of the second product: pairs of keys of a row
            p[t][0] = transpose8(pack2<T>(s[t][0], s[t][1]));
            p[t][1] = transpose8(pack2<T>(s[t][2], s[t][3]));
        }
        cp_async_wait<2>();
        __syncwarp();
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            // matrices: d 16d .. and 16d + 8 .. of keys 0-7, then of keys 8-15
            const int rr = (lane & 7) + (lane >> 4) * 8, cc = 2 * d + ((lane >> 3) & 1);
            uint32_t f[4];
            ldsm4_t(vt + rr * kRowBytes + ((cc ^ (rr & 7)) * 16), f);
#pragma unroll
            for (int t = 0; t < NT; ++t) Mma<T>::run(o[t][d], f, p[t][0], p[t][1]);
        }
        __syncwarp();  // V has been read
    }
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);

    // join the warps' states through shared memory
    cp_async_wait<0>();
    __syncthreads();
    float* so = reinterpret_cast<float*>(smem);             // [warps][rows][D + 4]
    constexpr int kPitch = D + 4;
    float* sm = so + kPartWarps * kRows * kPitch;           // [warps][rows] maxima, then sums
    float* sl = sm + kPartWarps * kRows;
    static_assert((kPartWarps * kRows * (kPitch + 2)) * 4 <= part_smem<D>(), "");
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l[t][j] += __shfl_xor_sync(~0u, l[t][j], d);
            const int r = warp * kRows + t * 8 + (lane % 4) * 2 + j;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                so[r * kPitch + d * 16 + lane / 4] = o[t][d][j];
                so[r * kPitch + d * 16 + lane / 4 + 8] = o[t][d][j + 2];
            }
            if (lane < 4) {
                sm[r] = m[t][j] - kLift;
                sl[r] = l[t][j];
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < kRows * (D / 4); i += kPartWarps * 32) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        if (rb * kRows + r >= rows) break;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kPartWarps; ++w) top = fmaxf(top, sm[w * kRows + r]);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPartWarps; ++w) {
            const float f = exp2_approx(sm[w * kRows + r] - base);
            const float4 x = *reinterpret_cast<const float4*>(so + (w * kRows + r) * kPitch + d);
            sum += f * sl[w * kRows + r];
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays one
        const long long at = query_row(r) * total_splits + slot;
        *reinterpret_cast<float4*>(a.part + at * D + d) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (d == 0) a.part_lse[at] = sum == 0.f ? -INFINITY : top + log2f(sum);
    }
    if (last) pdl_wait();
}

// log2-sum-exp2 of a row's parts: every lane of the warp gets it; NaN when a part's is, so that
// a NaN or infinite logit is not lost
IDX_DEVI float join_lse(const float* part_lse, int splits, int lane) {
    float m = -INFINITY;
    for (int i = lane; i < splits; i += 32) m = max_nan(m, part_lse[i]);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
    if (m == -INFINITY) return m;
    float l = 0.f;
    for (int i = lane; i < splits; i += 32) l += exp2_approx(part_lse[i] - m);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(~0u, l, o);
    return m + log2f(l);
}

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kSlotsPerThread = 4, kWeightSlots = kJoinThreads * kSlotsPerThread;

// A row that does not see its request's last keys weighs them with 0, and 0 times a V that is not
// finite is NaN.  This is the row's sum over its parts again (`lane`'s columns of it), those that
// reach past what it sees taken key by key up to there: called for such rows when their result is
// not finite, so rarely that its speed does not count.
template <typename T, int D>
__device__ __noinline__ void sum_visible(const AttnArgs& a, long long row, float lse, int lane,
                                         float* sum) {
    constexpr int W = D / 32;
    const int splits = a.prefix_splits + a.private_splits;
    const int head = (int)(row % a.Hq), hk = head / a.G;
    const int t = (int)(row / a.Hq % a.Q), b = (int)(row / a.Hq / a.Q);
    const int n = min(max(a.lens[b], 0), a.max_len), see = n - (a.Q - 1 - t);
    const int* table = a.table + (long long)b * a.table_stride;
    const T* q = static_cast<const T*>(a.q) + row * D + lane * W;
    for (int i = 0; i < W; ++i) sum[i] = 0.f;
    for (int p = 0; p < splits; ++p) {
        const float f = a.part_lse[row * splits + p];
        if (f == -INFINITY) continue;
        const int lo = (p - a.prefix_splits) * a.private_chunk;  // of a private part
        if (p < a.prefix_splits || min(n, lo + a.private_chunk) <= see) {
            const float w = exp2_approx(f - lse);
            for (int i = 0; i < W; ++i)
                sum[i] = fmaf(w, a.part[(row * splits + p) * D + lane * W + i], sum[i]);
            continue;
        }
        for (int j = lo; j < see; ++j) {
            const int page = table[j >> a.page_shift];
            if (page < 0 || page >= a.pages) continue;  // V reads as zeros
            const long long at = (((long long)page * a.Hkv + hk) * a.page_size +
                                  (j & (a.page_size - 1))) * D + lane * W;
            float z = 0.f;
            for (int i = 0; i < W; ++i)
                z = fmaf((float)q[i], (float)static_cast<const T*>(a.k)[at + i], z);
            for (int o = 16; o > 0; o /= 2) z += __shfl_xor_sync(~0u, z, o);
            const float w = exp2_approx(z * a.scale_log2 - lse);
            for (int i = 0; i < W; ++i)
                sum[i] = fmaf(w, (float)static_cast<const T*>(a.v)[at + i], sum[i]);
        }
    }
}

// The join of a query row's parts by WPR warps: lane l holds D / 32 columns, the warps
// take the parts in turn and add up through shared memory.
template <typename T, int D, int WPR, bool SEVERAL>
IDX_DEVI void join_row(const AttnArgs& a, long long row, int lane, int warp, float* sums) {
    constexpr int W = D / 32, kBatch = WPR == 1 ? 8 : 4;
    const int splits = a.prefix_splits + a.private_splits;
    const float* pl = a.part_lse + row * splits;
    const float lse = join_lse(pl, splits, lane);
    float acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.f;
    if (lse != -INFINITY) {
        const float* part = a.part + row * splits * D + lane * W;
        // kBatch parts at a time, all their loads before the first use; a part without
        // keys has written nothing and is not read
        for (int p = warp; p < splits; p += WPR * kBatch) {
            float f[kBatch], v[kBatch][W];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                f[k] = p + k * WPR < splits ? pl[p + k * WPR] : -INFINITY;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    v[k][i] = f[k] != -INFINITY ? part[(long long)(p + k * WPR) * D + i] : 0.f;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i) acc[i] = fmaf(exp2_approx(f[k] - lse), v[k][i], acc[i]);
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int i = 0; i < W; ++i) sums[warp * D + lane * W + i] = acc[i];
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int k = 1; k < WPR; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] += sums[k * D + lane * W + i];
    }
    if (SEVERAL && row / a.Hq % a.Q < a.Q - 1) {  // not the newest token: there are later keys
        bool odd = false;
#pragma unroll
        for (int i = 0; i < W; ++i) odd |= !isfinite(acc[i]);
        if (__any_sync(~0u, odd) && isfinite(lse)) {
            float sum[W];
            sum_visible<T, D>(a, row, lse, lane, sum);
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] = sum[i];
        }
    }
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row * D) + lane * (W / 2);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) out[i] = pack2<T>(acc[2 * i], acc[2 * i + 1]);
    if (a.lse && lane == 0) a.lse[row] = lse * 0.6931471805599453f;
}

// The weight that private slots received from their request's rows: block `u` takes
// kWeightSlots slots of a request and key head.
IDX_DEVI void add_weights(const AttnArgs& a, int u, float* row_lse) {
    const int per = (a.max_len + kWeightSlots - 1) / kWeightSlots;
    const int bh = u / per, b = bh / a.Hkv, hk = bh % a.Hkv;
    const int n = min(max(a.lens[b], 0), a.max_len);
    const int first = (u % per) * kWeightSlots;
    if (first >= n) return;
    const int rows = a.Q * a.G, splits = a.prefix_splits + a.private_splits;
    for (int r = threadIdx.x / 32; r < rows; r += kJoinWarps) {
        const long long row = ((long long)b * a.Q + r / a.G) * a.Hq + hk * a.G + r % a.G;
        const float l = join_lse(a.part_lse + row * splits, splits, threadIdx.x & 31);
        // a row that sees nothing has logits -inf only: any finite value gives weight 0
        if ((threadIdx.x & 31) == 0) row_lse[r] = l == -INFINITY ? 0.f : l;
    }
    __syncthreads();
    const float* z = a.logits + (long long)bh * rows * a.logit_stride;
    const float* w = a.w + (long long)bh * a.slots;
    float* w_out = a.w_out + (long long)bh * a.slots;
    float sum[kSlotsPerThread];
#pragma unroll
    for (int k = 0; k < kSlotsPerThread; ++k) {
        // the newest tokens' slots have gathered nothing yet, whatever the array holds
        const int j = first + k * kJoinThreads + (int)threadIdx.x;
        sum[k] = j < n - a.Q ? w[j] : 0.f;
    }
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
        const float l = row_lse[r];
#pragma unroll
        for (int k = 0; k < kSlotsPerThread; ++k) {
            const int j = first + k * kJoinThreads + (int)threadIdx.x;
            if (j < n) sum[k] += exp2_approx(z[r * a.logit_stride + j] - l);
        }
    }
#pragma unroll
    for (int k = 0; k < kSlotsPerThread; ++k) {
        const int j = first + k * kJoinThreads + (int)threadIdx.x;
        if (j < n) w_out[j] = sum[k];
    }
}

// Blocks [0, join_blocks) join the parts of query rows (WPR warps each), the others add up
// the weights of the private slots.  SEVERAL: calls of several tokens; with the call of sum_visible in
// it the kernel is slower (16 requests of one token 18.1 and 19.0 us), so the others go without.
template <typename T, int D, int WPR, bool SEVERAL>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a, int join_blocks) {
    __shared__ float scratch[kAttnMaxTokens * kAttnMaxGroup];
    pdl_wait();  // (no pdl_trigger: the next call's prefix grid came in its way, 74 -> 81 us)
    if ((int)blockIdx.x < join_blocks) {
        const int warp = threadIdx.x >> 5;
        const long long row = (long long)blockIdx.x * (kJoinWarps / WPR) + warp / WPR;
        if (row < (long long)a.B * a.Q * a.Hq)
            join_row<T, D, WPR, SEVERAL>(a, row, threadIdx.x & 31, warp % WPR, scratch);
    } else {
        add_weights(a, blockIdx.x - join_blocks, scratch);
    }
}

template <typename T, int D, int NT>
cudaError_t launch_private(const AttnArgs& a, cudaStream_t s) {
    static PerDevice ready;
    const cudaError_t e = allow_smem(ready, attn_part_kernel<T, D, NT>, part_smem<D>());
    if (e != cudaSuccess) return e;
    const dim3 grid((a.Q * a.G + 8 * NT - 1) / (8 * NT) * a.Hkv * a.private_splits, a.B);
    return launch_k(attn_part_kernel<T, D, NT>, grid, dim3(kPartWarps * 32), part_smem<D>(), s,
                    true, a);
}

template <typename T, int D>
cudaError_t launch_typed(const AttnArgs& a, idx_dtype dt, int sm_count, cudaStream_t s,
                         int* launched) {
    cudaError_t e = cudaSuccess;
    if (a.prefix_splits > 0) {
        if ((e = launch_prefix_parts(a, dt, s)) != cudaSuccess) return e;
        ++*launched;
    }
    if (a.private_splits > 0) {
        e = a.private_dense  ? launch_private_dense(a, dt, s)
            : a.Q * a.G <= 8 ? launch_private<T, D, 1>(a, s)
                             : launch_private<T, D, 2>(a, s);
        if (e != cudaSuccess) return e;
        ++*launched;
    }
    // A block per row while there are few rows with many parts: 576 rows of 25 parts 22.3 us for
    // the call by warps, 17.6 by blocks; 4096 rows of 11 parts 84 by warps, 88 by blocks.
    const long long rows = (long long)a.B * a.Q * a.Hq;
    const bool wide = a.prefix_splits + a.private_splits > 8 && rows <= 4ll * sm_count;
    const int per_block = wide ? 1 : kJoinWarps;
    const long long join_blocks = (rows + per_block - 1) / per_block;
    const long long weight_blocks =
        a.w_out ? (long long)a.B * a.Hkv * ((a.max_len + kWeightSlots - 1) / kWeightSlots) : 0;
    if (join_blocks + weight_blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const auto kern = a.Q > 1 ? (wide ? attn_join_kernel<T, D, kJoinWarps, true>
                                      : attn_join_kernel<T, D, 1, true>)
                              : (wide ? attn_join_kernel<T, D, kJoinWarps, false>
                                      : attn_join_kernel<T, D, 1, false>);
    e = launch_k(kern, dim3((unsigned)(join_blocks + weight_blocks)), dim3(kJoinThreads), 0, s,
                 true, a, (int)join_blocks);
    if (e == cudaSuccess) ++*launched;
    return e;
}

}  // namespace

// Row parts (a row's results of one part: D + 1 floats of workspace) that the plan may take of the
// prefix or of the private keys, when up to `splits` parts would be possible: all of them, but no more
// than kRowParts unless every row has one.  The plan chooses within this and the workspace is sized by
// it, so that the size grows with the rows and the lengths, as the choice itself does not.  65536 (34
// MB at D = 128) leaves all but one in a thousand of the plans of 1-64 requests as they would be.
constexpr size_t kRowParts = 65536;
static size_t most_row_parts(size_t rows, size_t splits) {
    return splits == 0 ? 0 : std::max(rows, std::min(rows * splits, kRowParts));
}

AttnPlan attn_plan(int B, int Q, int Hq, int Hkv, int D, int prefix_len, int max_len, bool weights,
                   int sm_count) {
    AttnPlan p;
    const int G = Hq / Hkv;
    p.prefix_splits = p.prefix_chunk = p.private_splits = p.private_chunk = 0;
    // the join reads D floats per row and part, about 5 MB per us
    const double join_us = (double)B * Q * Hq * D * 8 / 5e6;
    const size_t rows = (size_t)B * Q * Hq;
    size_t row_parts = 0;

    // Keys per private part: a block takes about 4 us and, among three on an SM, 34 ns per key
    // (D = 128: 512 bytes at a third of the SM's share of HBM), so whole waves of long parts are
    // cheap but a wave that is mostly empty is not.  (The kernel of up to 8 rows has four blocks on
    // an SM; the figures are from when it had three as well, and it is counted so.)  The lengths are on
    // the device: the mean of the times with all of them at max_len and at half of it is taken.
    //
    // More than 16 rows read a key several times over that way, at about its HBM time each; the
    // dense path of the prefix kernel reads it once, for about 8 us per CTA, one per SM.  The
    // cheaper is taken (16 requests of 4 tokens, 8 heads, 100-1000 keys: 24.7 and dense 18.4 us;
    // 16 of 7 tokens, 16 heads, 1024-8192 keys 150 and 52; 8 of 4 tokens, 16 heads, 100-500 keys
    // 14.3 and 18.0).  Beside logits, which the dense path writes a row per thread, it gains only
    // at D = 128 (16 of 7 tokens with weights, the one shape that was compared: D 128 224 and 164 us,
    // D 64 157 and 183).
    double private_us = 0;
    p.private_dense = false;
    if (max_len > 0) {
        constexpr int kMostSplits = 32;
        const int steps = (max_len + 63) / 64;  // 64: four warps' 16
        const size_t most = most_row_parts(rows, std::min(kMostSplits, steps));
        row_parts += most;
        double best = 0;
        auto consider = [&](bool dense, double items, int unit, int units, int s, double per_unit,
                            double base) {  // s parts of `units` units of keys
            const int t = (units + s - 1) / s, all = (units + t - 1) / t, half = (units / 2 + t) / t;
            if (all * rows > most) return;
            const double us =
                (std::ceil(items * all) + std::ceil(items * half)) / 2 * (t * per_unit + base);
            if (best == 0 || us + s * join_us < best) {
                best = us + s * join_us;
                private_us = us;
                p.private_chunk = t * unit;
                p.private_dense = dense;
            }
        };
        const int row_blocks = (Q * G + 15) / 16;
        for (int s = 1; s <= kMostSplits && s <= steps; s += s < 8 ? 1 : s / 4)
            consider(false, (double)row_blocks * Hkv * B / (3 * sm_count), 64, steps, s,
                     64 * (D * 34e-3 / 128), 4.0);
        if (row_blocks > 1 && !(weights && D == 64)) {
            const int keys = attn_prefix_keys(D), tiles = (max_len + keys - 1) / keys;
            const int row_tiles = (Q + 128 / G - 1) / (128 / G);
            for (int s = 1; s <= kMostSplits && s <= tiles; s += s < 8 ? 1 : s / 4)
                consider(true, (double)B * Hkv * ((row_tiles + 1) / 2) / sm_count, keys, tiles, s,
                         keys * D * 4 / 45e3, 8.0);
        }
        p.private_splits = (max_len + p.private_chunk - 1) / p.private_chunk;
    }

    // Key tiles per prefix part: a CTA, one per SM, takes about 1.4 us per 128 keys of a pair of
    // row tiles (0.75 us of a single one, whose keys two streams share) and 4 us besides.  SMs
    // without one take private parts meanwhile, so the time is the longer of a CTA's and the
    // mean over all SMs of both kinds' work: with private parts, fewer and longer prefix parts.
    // The estimate above is for the largest lengths and no overlap; about a third of it is what
    // the private parts take beside the prefix.  (With no share and with it: 64 requests of
    // 64-1024 keys behind 32768 81 and 74 us, 32 of 100-2048 behind 16384 62 and 52, 64 of
    // 512-4096 behind 4096 120 and 104, 16 of 64-1024 behind 4096 22.1 and 20.4; the whole
    // estimate makes the prefix parts too few: 104, 68, 105 and 24.)
    constexpr double kShare = 0.35;
    if (prefix_len > 0) {
        const int keys = attn_prefix_keys(D), tokens = 128 / G, tiles = (prefix_len + keys - 1) / keys;
        const long long row_tiles = ((long long)B * Q + tokens - 1) / tokens;
        const long long items = (row_tiles + 1) / 2 * Hkv;
        const double per_tile = (row_tiles > 1 ? 1.4 : 0.75) * keys / 128;
        const int most_splits = std::min(tiles, 4 * sm_count);  // (a grid dimension, too)
        const size_t most = most_row_parts(rows, most_splits);
        row_parts += most;
        double best = 0;
        const double per_sm = 1.0 / sm_count;
        auto consider = [&](int t) {  // t tiles per part
            t = t < 1 ? 1 : t > tiles ? tiles : t;
            const int s = (tiles + t - 1) / t;
            if (s > most_splits || s * rows > most) return;
            const double one = t * per_tile + 4.0, waves = (double)items * s * per_sm;
            const double dense = std::ceil(waves) * one, mean = waves * one + private_us * kShare;
            const double us = (dense > mean ? dense : mean) + s * join_us;
            if (best == 0 || us < best) {
                best = us;
                p.prefix_chunk = (int)t * keys;
            }
        };
        for (int t = 1; t <= 4; ++t) consider(t);
        consider((tiles + 1023) / 1024);
        for (int eighths = 2; eighths <= 48; eighths += eighths < 8 ? 1 : 8) {  // of a wave's CTAs
            const int n = (int)(eighths * sm_count / (8 * items));
            consider(n > 1 ? (tiles + n - 1) / n : tiles);
        }
        if (best == 0) consider(tiles);
        p.prefix_splits = (prefix_len + p.prefix_chunk - 1) / p.prefix_chunk;
    }
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    p.logit_stride = ((long long)max_len + 15) / 16 * 16;
    p.part = 0;
    p.part_lse = up(row_parts * D * sizeof(float));
    p.logits = p.part_lse + up(row_parts * sizeof(float));
    p.total = p.logits + (weights ? up(rows * p.logit_stride * sizeof(float)) : 0);
    return p;
}

cudaError_t launch_attention(const AttnArgs& a, idx_dtype dt, int sm_count, cudaStream_t s,
                             int* launched) {
    if (dt == IDX_BF16)
        return a.D == 128 ? launch_typed<__nv_bfloat16, 128>(a, dt, sm_count, s, launched)
                          : launch_typed<__nv_bfloat16, 64>(a, dt, sm_count, s, launched);
    return a.D == 128 ? launch_typed<__half, 128>(a, dt, sm_count, s, launched)
                      : launch_typed<__half, 64>(a, dt, sm_count, s, launched);
}

}  // namespace idx
