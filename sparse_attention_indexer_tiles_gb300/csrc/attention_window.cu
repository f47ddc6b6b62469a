// Attention over a paged MXFP4 cache, with a sliding window and first tokens that stay visible.
//
// Row (token at position p, head) sees the keys j <= p with j < sink or j > p - window (all of
// them when window is 0), z_j = scale * q . k_j:
//     o = sum_j exp(z_j) v_j / sum_j exp(z_j),   lse = log sum_j exp(z_j).
// k and v are e2m1 codes c times a power of two per 32 elements.  The operands of the matrix instructions are codes as
// fp16, which holds them exactly, times the powers of two relative to running ones: 2^EK for all of K, 2^E for
// each block of V's columns.  Sums come in units of 2^EK, o in units of 2^E.  Blocks whose power lies outside the 26
// powers below the running one, or above it, are rare: their step takes another path, a pass per 26 powers.
//
// bf16 queries are made fp16 by a power of two per row (the largest element just below 2^15): an
// element below 2^-32 of the row's largest loses bits, 2^-40 of that one at most.  The weights
// enter the second product as fp16 times 2^7; the running maximum is renewed when a row grows
// past it by 2^8.  Weights below 2^-21 of a row's largest have fewer bits than fp16, those below
// 2^-31 count as 0.  Maxima, sums and o are fp32, exponentials base 2 on z * log2(e).
//
// HBM-bound in theory (68 bytes per key row of 128); in practice the instructions that expand the codes come close. A
// block's warps each take 32 keys at a time through a ring of their own, filled by the lanes' 16-byte copies (bulk
// copies of a step's rows cost more instructions to issue; tensor copies of swizzled rows took 9 % longer still).  The products are taken transposed, S^T = K Q^T
// and O^T += V^T P^T: keys and D are the long axes of the matrix instructions, the rows (8 or 16) the short one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "serve.cuh"
#include "window_span.cuh"

namespace cg = cooperative_groups;

namespace idx {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 2;
constexpr float kLift = 7.f;    // weights are taken times 2^kLift
constexpr float kRenew = 8.f;   // growth of a row's maximum that renews it; 2^(kLift + kRenew) fits fp16
// Fields of an fp16 power of two 2^(field - 15) that codes take: 28 for a block at the running power, so that 6 * 2^13
// is the largest value; blocks below 2^-26 of it are taken in another pass over the step.
constexpr int kTopField = 28, kBand = 26;
constexpr int kMargin = 3;      // running powers are set this far above what asked for them

template <int D> struct Ring {
    static constexpr int ROW = D / 2;                        // bytes of codes
    static constexpr int CODES = kWindowStep * ROW;
    static constexpr int SF = kWindowStep * (D / 32);
    static constexpr int OFF_V = CODES, OFF_KSF = 2 * CODES, OFF_VSF = 2 * CODES + SF;
    static constexpr int STAGE = 2 * CODES + 2 * SF;
    static constexpr int RING = kWarps * kStages * STAGE;
    static_assert(STAGE % 128 == 0, "");
    static constexpr int JOIN = kWarps * 16 * (D + 6) * 4;   // of 16 rows
    static constexpr int OFF_ROWS = RING > JOIN ? RING : JOIN;  // per row: its logits' factor, its position
    static constexpr int OFF_RESULT = OFF_ROWS + 16 * 8;  // of a split in a cluster: rows of D, then their sums
    static constexpr int OFF_Q = (OFF_RESULT + 16 * (D + 1) * 4 + 15) / 16 * 16;  // tiles of 16 rows: the operand of q
    static constexpr int SMEM = OFF_Q + 16 * D * 2;
};

// Eight e2m1 codes as fp16, pairs in order.
IDX_DEVI void expand8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
IDX_DEVI uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The bits of a where mask is set, those of b elsewhere.
IDX_DEVI uint32_t pick(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }

IDX_DEVI void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8x8 matrix of 16-bit elements held across the warp.
IDX_DEVI uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <int N> IDX_DEVI void lds(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
        static_assert(N == 4, "one, two or four words");
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr));
    }
}
// 16-byte asynchronous copies, past L1, in groups.
IDX_DEVI void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
IDX_DEVI void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> IDX_DEVI void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
IDX_DEVI uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
IDX_DEVI void sts8(uint32_t addr, uint32_t v) { asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v)); }
// 2^n for any n that a scale can need, as two factors.
IDX_DEVI float times_pow2(float x, int n) {
    const int a = n / 2, b = n - a;
    return x * __int_as_float((a + 127) << 23) * __int_as_float((b + 127) << 23);
}

// A block: 8 NT rows of a request and key head against one split of the keys that they see.  Warps
// take the split's steps in turn, each with its own softmax state, joined at the end.
// blockIdx.x: split, row tile, key head; blockIdx.y: request.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 3)
window_kernel(const __grid_constant__ WindowArgs a) {
    using R = Ring<D>;
    constexpr int BLOCKS = D / 32;      // of K's and V's scales in a row
    constexpr int KW = D / 32, VW = D / 64;  // words of a K row and of a V row that a lane takes
    constexpr int TILES = D / 16;       // of O^T: 16 columns of D each
    constexpr int kRows = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t smem0 = smem_u32(smem);
    pdl_wait();
    pdl_trigger();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits % a.row_tiles;
    const int hk = blockIdx.x / a.splits / a.row_tiles, b = blockIdx.y;
    const Span sp = span_of(a, b, tid == 0 && blockIdx.x == 0);
    const int rows = sp.count * a.G, row0 = tile * kRows;
    if (row0 >= rows) return;
    // row i of the tile: token, head of the group
    auto query_row = [&](int i) {
        const int r = row0 + i, token = r / a.G;
        return (long long)(sp.first + token) * a.Hq + hk * a.G + (r - token * a.G);
    };
    const int pos0 = sp.len - sp.count;  // position of the request's first new token
    const int low = pos0 + row0 / a.G, high = pos0 + (min(row0 + kRows, rows) - 1) / a.G;
    const int hi = max(0, min(sp.len, high + 1));
    // the oldest key inside the first row's window, and how the steps lie: the sinks' and from the window's
    const int wlo = a.window > 0 ? max(0, low - a.window + 1) : 0;
    const int sink = min(a.sink, hi);
    int sink_steps = (sink + kWindowStep - 1) / kWindowStep, from = wlo / kWindowStep;
    if (from <= sink_steps) sink_steps = from = 0;  // no gap
    const int total = sink_steps + max(0, (hi + kWindowStep - 1) / kWindowStep - from);
    const int first = split * a.chunk, end = min(total, first + a.chunk);
    const int mine = first + warp < end ? (end - 1 - first - warp) / kWarps + 1 : 0;
    if (first >= end) {
        for (int i = tid; i < kRows && row0 + i < rows; i += kWarps * 32) {
            if (a.splits > 1 && !a.clustered) a.part_lse[query_row(i) * a.splits + split] = -INFINITY;
        }
        // (a cluster's barrier does not wait for blocks that have ended, and its first block stays)
        if (a.splits > 1 && !(a.clustered && split == 0)) return;
    }
    auto base_of = [&](int i) {  // first key of the warp's i-th step
        const int v = first + i * kWarps + warp;
        return kWindowStep * (v < sink_steps ? v : v - sink_steps + from);
    };

    const uint32_t ring = smem0 + warp * kStages * R::STAGE;
    // Pages of the warp's next steps, one 16-key half per lane: 16 steps at a time.  A half that no
    // row sees is not looked up (its page may be gone): its place is filled from the other half's page, and masked.
    const int* table = a.table + b * a.table_stride;
    bool bad = false;
    int pages_from = 0, page_of = 0;
    auto look_up = [&](int i) {
        pages_from = i;
        const int s = i + (lane >> 1);
        page_of = -1;
        if (s < mine) {
            const int key = base_of(s) + (lane & 1) * 16;
            if (key < hi && (key < sink || key + 16 > wlo)) {
                page_of = table[key >> a.page_shift];
                if (page_of < 0 || page_of >= a.pages) {
                    page_of = 0;
                    bad = true;
                }
            }
        }
        // (a row sees a key of every step; where a page holds a whole step, both halves name it or one does)
        const int other = __shfl_xor_sync(~0u, page_of, 1);
        if (page_of < 0) page_of = max(other, 0);
    };
    const bool whole = a.page_size >= kWindowStep;  // a step lies in one page
    // The copies of a step: codes of 16 keys are kHalf adjacent 16-byte chunks, dealt to the lanes; scales a chunk for
    // each of the first lanes, K's and then V's.
    constexpr int kHalf = R::ROW, kSfChunks = R::SF / 16;
    const uint8_t* const sf = lane < kSfChunks ? a.k_sf : a.v_sf;
    const int sf_chunk = lane & (kSfChunks - 1);
    auto fetch = [&](int i) {
        if (i - pages_from >= 16 || i == 0) look_up(i);
        const int base = base_of(i);
        const int p0 = __shfl_sync(~0u, page_of, 2 * (i - pages_from));
        const int p1 = __shfl_sync(~0u, page_of, 2 * (i - pages_from) + 1);
        const int in_page = base & (a.page_size - 1);
        const long long row0 = (long long)(p0 * a.Hkv + hk) * a.page_size + in_page;
        const long long row1 = whole ? row0 + 16 : (long long)(p1 * a.Hkv + hk) * a.page_size;
        const uint32_t dst = ring + i % kStages * R::STAGE + lane * 16;
        const uint8_t* const k0 = a.k_codes + row0 * R::ROW + lane * 16;
        const uint8_t* const k1 = a.k_codes + row1 * R::ROW + lane * 16;
        const uint8_t* const v0 = a.v_codes + row0 * R::ROW + lane * 16;
        const uint8_t* const v1 = a.v_codes + row1 * R::ROW + lane * 16;
#pragma unroll
        for (int j = 0; j < kHalf; j += 32) {
            copy16(dst + j * 16, k0 + j * 16);
            copy16(dst + (kHalf + j) * 16, k1 + j * 16);
            copy16(dst + R::OFF_V + j * 16, v0 + j * 16);
            copy16(dst + R::OFF_V + (kHalf + j) * 16, v1 + j * 16);
        }
        if (lane < 2 * kSfChunks) {
            constexpr int kPerHalf = kSfChunks / 2;
            const bool second = sf_chunk >= kPerHalf;
            copy16(ring + i % kStages * R::STAGE + R::OFF_KSF + lane * 16,
                   sf + (second ? row1 : row0) * BLOCKS + (second ? sf_chunk - kPerHalf : sf_chunk) * 16);
        }
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
        if (i < mine) fetch(i);
        copies_commit();
    }

    // q as the products' second operand: row g of each eight, a quarter of its columns per lane; the i-th step of 16
    // columns takes 4 i .. 4 i + 3 of each quarter (as the words of codes have them)
    // (of 16 rows they stay in shared memory: the registers would not hold them beside o)
    constexpr bool kKeepQ = NT == 1;
    uint32_t qf[NT][KW][4];
    const uint32_t q_at = smem0 + R::OFF_Q + lane * 16;
    float2* const row_info = reinterpret_cast<float2*>(smem + R::OFF_ROWS);  // read in steps that are not plain
    float zscale[NT][2];  // the logits' factors at 2^EK, of this thread's columns of S^T: rows 2 t and 2 t + 1
    const float scale = a.scale_log2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int i = n * 8 + g;
        const bool live = row0 + i < rows;
        const long long row = live ? query_row(i) : 0;
        const T* q = static_cast<const T*>(a.q) + row / a.Hq * a.q_stride + row % a.Hq * D + t * (D / 4);
        uint4 raw[KW];
#pragma unroll
        for (int k = 0; k < KW; ++k)
            raw[k] = live ? *reinterpret_cast<const uint4*>(q + k * 8) : make_uint4(0u, 0u, 0u, 0u);
        float factor = 1.f;
        const uint32_t flip = scale < 0.f ? 0x80008000u : 0u;  // the scale's sign goes to q
        if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                qf[n][k][0] = raw[k].x ^ flip;
                qf[n][k][1] = raw[k].y ^ flip;
                qf[n][k][2] = raw[k].z ^ flip;
                qf[n][k][3] = raw[k].w ^ flip;
            }
        } else {
            uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max(top, max(w[j] << 16 & 0x7fff0000u, w[j] & 0x7fff0000u));
            }
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            // 2^up brings it to [2^14, 2^15); rows of tiny numbers (below 2^-100) keep their distance
            const int ex = (int)(top >> 23);
            const int up = top == 0 ? 0 : min(127 + 14 - ex, 114);
            const float f = __int_as_float((up + 127) << 23);
            factor = __int_as_float((127 - up) << 23);
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    // a row that is not finite is NaN for every key that it sees
                    qf[n][k][j] = ex == 255 ? 0x7e007e00u
                                            : flip ^ pack2<__half>(__uint_as_float(w[j] << 16) * f,
                                                                   __uint_as_float(w[j] & 0xffff0000u) * f);
            }
        }
        if constexpr (!kKeepQ) {
            if (warp == 0) {
#pragma unroll
                for (int k = 0; k < KW; ++k)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q_at + (n * KW + k) * 512), "r"(qf[n][k][0]),
                                 "r"(qf[n][k][1]), "r"(qf[n][k][2]), "r"(qf[n][k][3])
                                 : "memory");
            }
        }
        if (warp == 0 && t == 0)
            row_info[i] = make_float2(factor * fabsf(scale), __int_as_float(live ? pos0 + (row0 + i) / a.G : -1));
    }
    __syncthreads();
    const int all_see = low + 1, all_from = a.window > 0 ? high - a.window + 1 : 0;  // of every row

    // This lane's key of row g of the products, kg, and its keys of V: t, t + 4, + 8 and + 12.  The first product's
    // transpose hands over the weights of the keys of rows 2 t and 2 t + 1.
    const int kg = g >> 1 | (g & 1) << 2;
    const int kblock = t / (4 / BLOCKS), vblock = g / (8 / BLOCKS);  // of this lane's columns

    float o[NT][TILES][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
    }
    int E = 0, EK = 0;  // units of o and of S are 2^E and 2^EK (biased as the scales) over 2^13
    auto scale_logits = [&] {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // within the normal numbers: a masked logit times it stays -inf, a logit of 0 stays 0
                const float z = times_pow2(row_info[n * 8 + 2 * t + j].x, EK - 140);
                zscale[n][j] = fminf(fmaxf(z, 0x1p-126f), 0x1p127f);
            }
    };
    for (int i = 0; i < mine; ++i) {
        copies_wait<kStages - 1>();
        __syncwarp();
        const uint32_t at = ring + i % kStages * R::STAGE;
        const int base = base_of(i);
        const bool plain = base + kWindowStep <= all_see && (base >= all_from || base + kWindowStep <= a.sink);
        // a key of the step that a row of the tile sees
        auto seen = [&](int in) {
            const int key = base + in;
            return plain || (key < hi && (key < sink || key >= wlo));
        };
        if (!plain) {
            // keys that no row sees get the scales of one that is seen: whatever theirs are, they don't count
            const bool mine = seen(lane);
            const uint32_t some = __ballot_sync(~0u, mine);
            const int from = __ffs(some) - 1;
            if (!mine && from >= 0)
#pragma unroll 1
                for (int k = 0; k < BLOCKS; ++k) {
                    sts8(at + R::OFF_KSF + lane * BLOCKS + k, lds8(at + R::OFF_KSF + from * BLOCKS + k));
                    sts8(at + R::OFF_VSF + lane * BLOCKS + k, lds8(at + R::OFF_VSF + from * BLOCKS + k));
                }
            __syncwarp();
        }
        if (i == 0) {
            // the first powers are a little above the first step's
            int k = 0, v = 0;
            for (int j = lane & 3; j < kWindowStep; j += 4) v = max(v, (int)lds8(at + R::OFF_VSF + j * BLOCKS + vblock));
            v = max(v, __shfl_xor_sync(~0u, v, 1));
            v = max(v, __shfl_xor_sync(~0u, v, 2));
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j) k = max(k, (int)lds8(at + R::OFF_KSF + lane * BLOCKS + j));
            k = __reduce_max_sync(~0u, k);
            E = v < 255 ? min(v + kMargin, 254) : 0;
            EK = k < 255 ? min(k + kMargin, 254) : 0;
            scale_logits();
        }

        // ---- scales: whether the running powers and their bands hold them
        uint32_t ks[2][2];  // [half][keys kg, kg + 8]
        uint32_t vs[2][2];  // [half][keys t, t + 4; then both + 8]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ks[h][k] = lds8(at + R::OFF_KSF + kblock + kg * BLOCKS + (h * 16 + 8 * k) * BLOCKS);
                const uint32_t v = at + R::OFF_VSF + vblock + t * BLOCKS + (h * 16 + 8 * k) * BLOCKS;
                vs[h][k] = lds8(v) | lds8(v + 4 * BLOCKS) << 16;
            }
        bool out = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) out |= ks[h][k] - (uint32_t)(EK - kBand) > (uint32_t)kBand;
        const uint32_t most = __vmaxu2(__vmaxu2(vs[0][0], vs[0][1]), __vmaxu2(vs[1][0], vs[1][1]));
        const uint32_t least = __vminu2(__vminu2(vs[0][0], vs[0][1]), __vminu2(vs[1][0], vs[1][1]));
        const uint32_t top = (uint32_t)E * 0x10001u, low_end = (uint32_t)max(E - kBand, 0) * 0x10001u;
        const bool slow = __any_sync(~0u, out || __vmaxu2(most, top) != top || __vminu2(least, low_end) != low_end);

        // ---- S^T of the two halves of 16 keys: K's codes times 2^(field - 15), both halves of `sc` the same
        float s[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[h][n][j] = 0.f;
        auto add_s = [&](const uint32_t (&sc)[2][2], auto direct, float unit) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[2][KW];
                lds<KW>(at + (h * 16 + kg) * R::ROW + t * (R::ROW / 4), w[0]);
                lds<KW>(at + (h * 16 + kg) * R::ROW + t * (R::ROW / 4) + 8 * R::ROW, w[1]);
                float c[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[n][j] = 0.f;
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    uint32_t x0[4], x1[4];
                    expand8(w[0][k], x0);
                    expand8(w[1][k], x1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x0[j] = hmul2(x0[j], sc[h][0]);
                        x1[j] = hmul2(x1[j], sc[h][1]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t q[4] = {qf[n][k][0], qf[n][k][1], qf[n][k][2], qf[n][k][3]};
                        if constexpr (!kKeepQ) lds<4>(q_at + (n * KW + k) * 512, q);
                        mma_f16(c[n], x0[0], x1[0], x0[1], x1[1], q[0], q[1]);
                        mma_f16(c[n], x0[2], x1[2], x0[3], x1[3], q[2], q[3]);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[h][n][j] = decltype(direct)::value ? c[n][j] : fmaf(c[n][j], unit, s[h][n][j]);
            }
        };
        if (!slow) {
            uint32_t sc[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) sc[h][k] = ks[h][k] * 0x04000400u + (uint32_t)(kTopField - EK) * 0x04000400u;
            add_s(sc, std::true_type{}, 1.f);
        } else {
            uint32_t pending = 0;  // bit 2 h + k: a key that a row sees and whose block is still to be added
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (seen((j >> 1) * 16 + kg + 8 * (j & 1))) pending |= 1u << j;
            do {
                int top = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (pending >> j & 1 && ks[j >> 1][j & 1] != 255u) top = max(top, (int)ks[j >> 1][j & 1]);
                top = __reduce_max_sync(~0u, top);
                if (top > EK) EK = min(top + kMargin, 254);  // (in the first pass: nothing has been added)
                const int Eb = top < EK - kBand / 2 ? top : EK;  // this pass's unit
                uint32_t sc[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int bit = 2 * h + k, x = (int)ks[h][k];
                        const bool in = pending >> bit & 1 && x >= Eb - kBand;
                        // a scale of 255: the key's logits are NaN
                        sc[h][k] = !in ? 0u : x == 255 ? 0x7e007e00u : (uint32_t)(x - Eb + kTopField) * 0x04000400u;
                        if (in) pending &= ~(1u << bit);
                    }
                add_s(sc, std::false_type{}, times_pow2(1.f, max(Eb - EK, -250)));
            } while (__any_sync(~0u, pending != 0));
            scale_logits();
        }

        // ---- softmax
        uint32_t p[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (slow || !plain) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int in = h * 16 + kg + (j >> 1) * 8, key = base + in;
                        // a V scale of 255 counts as a NaN logit of the rows that see it
                        uint32_t x = 0;
#pragma unroll
                        for (int k = 0; k < BLOCKS; ++k) x = max(x, lds8(at + R::OFF_VSF + in * BLOCKS + k));
                        if (x == 255u) s[h][n][j] = NAN;
                        const int pos = __float_as_int(row_info[n * 8 + 2 * t + (j & 1)].y);
                        if (key > pos || key >= sp.len || (a.window > 0 && key >= a.sink && key <= pos - a.window))
                            s[h][n][j] = -INFINITY;
                    }
            }
            float x0 = fmaxf(fmaxf(s[0][n][0], s[0][n][2]), fmaxf(s[1][n][0], s[1][n][2])) * zscale[n][0];
            float x1 = fmaxf(fmaxf(s[0][n][1], s[0][n][3]), fmaxf(s[1][n][1], s[1][n][3])) * zscale[n][1];
            if (__any_sync(~0u, x0 > m[n][0] + kRenew || x1 > m[n][1] + kRenew)) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) {
                    x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, d));
                    x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, d));
                }
                const float n0 = fmaxf(m[n][0], x0), n1 = fmaxf(m[n][1], x1);
                const float f0 = n0 == -INFINITY ? 1.f : exp2_approx(m[n][0] - n0);
                const float f1 = n1 == -INFINITY ? 1.f : exp2_approx(m[n][1] - n1);
                m[n][0] = n0;
                m[n][1] = n1;
                l[n][0] *= f0;
                l[n][1] *= f1;
#pragma unroll
                for (int d = 0; d < TILES; ++d) {
                    o[n][d][0] *= f0;
                    o[n][d][1] *= f1;
                    o[n][d][2] *= f0;
                    o[n][d][3] *= f1;
                }
            }
            // rows that have seen no key yet keep m = -inf: their weights are 0
            const float b0 = m[n][0] == -INFINITY ? 0.f : kLift - m[n][0];
            const float b1 = m[n][1] == -INFINITY ? 0.f : kLift - m[n][1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s[h][n][0] = exp2_approx(fmaf(s[h][n][0], zscale[n][0], b0));
                s[h][n][1] = exp2_approx(fmaf(s[h][n][1], zscale[n][1], b1));
                s[h][n][2] = exp2_approx(fmaf(s[h][n][2], zscale[n][0], b0));
                s[h][n][3] = exp2_approx(fmaf(s[h][n][3], zscale[n][1], b1));
                l[n][0] += s[h][n][0] + s[h][n][2];
                l[n][1] += s[h][n][1] + s[h][n][3];
                p[h][n][0] = transpose8(pack2<__half>(s[h][n][0], s[h][n][1]));
                p[h][n][1] = transpose8(pack2<__half>(s[h][n][2], s[h][n][3]));
            }
        }

        // ---- O^T += V^T P^T, V's codes times 2^(field - 15) of each pair of keys; in slow steps
        // the sums come in units of their own, `unit` of o's
        auto add_v = [&](const uint32_t (&sc)[2][2], auto direct, float unit) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[4][VW];  // keys t, t + 4, t + 8, t + 12
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    lds<VW>(at + R::OFF_V + t * R::ROW + g * (R::ROW / 8) + (h * 16 + 4 * k) * R::ROW, w[k]);
#pragma unroll
                for (int v = 0; v < VW; ++v) {
                    // nibbles of two keys side by side: even and odd columns
                    uint32_t x[2][2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t lo = w[2 * k][v], up = w[2 * k + 1][v];
                        expand8(pick(0x0f0f0f0fu, lo, up << 4), x[k][0]);
                        expand8(pick(0x0f0f0f0fu, lo >> 4, up), x[k][1]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            x[k][0][j] = hmul2(x[k][0][j], sc[h][k]);
                            x[k][1][j] = hmul2(x[k][1][j], sc[h][k]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float(&to)[4] = o[n][v * 4 + j];
                            if constexpr (decltype(direct)::value) {
                                mma_f16(to, x[0][0][j], x[0][1][j], x[1][0][j], x[1][1][j], p[h][n][0], p[h][n][1]);
                            } else {
                                float c[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(c, x[0][0][j], x[0][1][j], x[1][0][j], x[1][1][j], p[h][n][0], p[h][n][1]);
#pragma unroll
                                for (int y = 0; y < 4; ++y) to[y] = fmaf(c[y], unit, to[y]);
                            }
                        }
                }
            }
        };
        uint32_t sc[2][2];
        if (!slow) {
            const uint32_t c = (uint32_t)(kTopField - E) * 0x04000400u;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) sc[h][k] = vs[h][k] * 1024u + c;
            add_v(sc, std::true_type{}, 1.f);
        } else {
            uint32_t pending = 0;  // bit 4 h + 2 k + j: a key that a row sees and whose V is still to be added
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (seen((j >> 2) * 16 + (j >> 1 & 1) * 8 + (j & 1) * 4 + t)) pending |= 1u << j;
            do {
                // the largest scale still to be taken, of the block's four lanes
                int top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int x = (int)(vs[j >> 2][j >> 1 & 1] >> (16 * (j & 1)) & 0xffu);
                    if (x == 255) pending &= ~(1u << j);  // its rows are NaN already
                    if (pending >> j & 1) top = max(top, x);
                }
                top = max(top, __shfl_xor_sync(~0u, top, 1));
                top = max(top, __shfl_xor_sync(~0u, top, 2));
                if (top > E) {
                    const int to = min(top + kMargin, 254);
                    const float f = times_pow2(1.f, max(E - to, -250));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int d = 0; d < TILES; ++d)
#pragma unroll
                            for (int j = 0; j < 4; ++j) o[n][d][j] *= f;
                    E = to;
                }
                const int Eb = top < E - kBand / 2 ? top : E;  // this pass's unit
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t both = 0;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int bit = 4 * h + 2 * k + j, x = (int)(vs[h][k] >> (16 * j) & 0xffu);
                            const bool in = pending >> bit & 1 && x >= Eb - kBand;
                            if (in) both |= (uint32_t)(x - Eb + kTopField) << (10 + 16 * j);
                            if (in) pending &= ~(1u << bit);
                        }
                        sc[h][k] = both;
                    }
                add_v(sc, std::false_type{}, times_pow2(1.f, max(Eb - E, -250)));
            } while (__any_sync(~0u, pending != 0));
        }
        __syncwarp();  // the stage has been read
        if (i + kStages < mine) fetch(i + kStages);
        copies_commit();
    }
    copies_wait<0>();
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);

    // ---- join the warps' states through shared memory
    __syncthreads();
    constexpr int kPitch = D + 4;
    float* so = reinterpret_cast<float*>(smem);       // [warps][rows][kPitch]
    float* sm = so + kWarps * kRows * kPitch;         // [warps][rows] maxima, then sums
    float* sl = sm + kWarps * kRows;
    static_assert(kWarps * kRows * (kPitch + 2) * 4 <= R::JOIN, "");
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l[n][j] += __shfl_xor_sync(~0u, l[n][j], d);
            const int r = warp * kRows + n * 8 + 2 * t + j;
            // (means, not sums: the largest values of V times the weights' lift would leave fp32)
            const float inv = l[n][j] == 0.f ? 0.f : 1.f / l[n][j];
#pragma unroll
            for (int d = 0; d < TILES; ++d) {
                // codes * 2^(sf - E + 13) summed, times 2^(E - 127 - 13)
                so[r * kPitch + g * (2 * TILES) + 2 * d] = times_pow2(o[n][d][j] * inv, E - 140);
                so[r * kPitch + g * (2 * TILES) + 2 * d + 1] = times_pow2(o[n][d][j + 2] * inv, E - 140);
            }
            if (g == 0) {
                sm[r] = m[n][j] - kLift;
                sl[r] = l[n][j];
            }
        }
    __syncthreads();
    auto write = [&](int r, int d, const float4& acc, float lse) {
        const long long row = query_row(r);
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + d) =
            make_uint2(pack2<T>(acc.x, acc.y), pack2<T>(acc.z, acc.w));
        if (d == 0 && a.lse) a.lse[row] = lse * 0.6931471805599453f;
    };
    for (int x = tid; x < kRows * (D / 4); x += kWarps * 32) {
        const int r = x / (D / 4), d = x % (D / 4) * 4;
        if (row0 + r >= rows) break;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * kRows + r]);
        const float from_top = top == -INFINITY ? 0.f : top;
        float share[kWarps], sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += share[w] = exp2_approx(sm[w * kRows + r] - from_top) * sl[w * kRows + r];
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays one
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = share[w] * inv;
            const float4 v = *reinterpret_cast<const float4*>(so + (w * kRows + r) * kPitch + d);
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        }
        const float lse = sum == 0.f ? -INFINITY : top + log2f(sum);
        if (a.clustered) {
            float* result = reinterpret_cast<float*>(smem + R::OFF_RESULT);
            *reinterpret_cast<float4*>(result + r * D + d) = acc;
            if (d == 0) result[16 * D + r] = lse;
        } else if (a.splits > 1) {
            const long long to = query_row(r) * a.splits + split;
            *reinterpret_cast<float4*>(a.part + to * D + d) = acc;
            if (d == 0) a.part_lse[to] = lse;
        } else {
            write(r, d, acc, lse);
        }
    }
    if (!a.clustered) return;
    // The cluster's blocks with keys join a share of the tile's columns each.
    const cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int parts = max(1, min(a.splits, (total + a.chunk - 1) / a.chunk));
    for (int x = split * (kWarps * 32) + tid; x < kRows * (D / 4); x += parts * (kWarps * 32)) {
        const int r = x / (D / 4), d = x % (D / 4) * 4;
        if (row0 + r >= rows) break;
        const float* result = reinterpret_cast<const float*>(smem + R::OFF_RESULT);
        float lse[kWindowCluster], top = -INFINITY;
#pragma unroll
        for (int p = 0; p < kWindowCluster; ++p) {
            lse[p] = p < parts ? cluster.map_shared_rank(result, p)[16 * D + r] : -INFINITY;
            top = max_nan(top, lse[p]);
        }
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < kWindowCluster; ++p) sum += lse[p] = lse[p] == -INFINITY ? 0.f : exp2_approx(lse[p] - top);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // NaN stays one
#pragma unroll
        for (int p = 0; p < kWindowCluster; ++p) {
            if (p >= parts) break;
            const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(result, p) + r * D + d);
            const float f = lse[p] * inv;
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        }
        write(r, d, acc, sum == 0.f ? -INFINITY : top + log2f(sum));
    }
    cluster.sync();  // no block ends while another reads its results
}

// Joins a row's splits: a warp per row, lane l holds D / 32 columns.
constexpr int kJoinThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) window_join_kernel(const __grid_constant__ WindowArgs a) {
    constexpr int W = D / 32, kBatch = 8;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32;
    // tokens behind the last request's are not touched
    const long long from = a.q_start ? a.q_start[0] : 0, to = a.q_start ? a.q_start[a.B] : a.T;
    if (row >= min(to, (long long)a.T) * a.Hq || row < from * a.Hq) return;
    const float* pl = a.part_lse + row * a.splits;
    float m = -INFINITY;
    for (int i = lane; i < a.splits; i += 32) m = max_nan(m, pl[i]);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = max_nan(m, __shfl_xor_sync(~0u, m, d));
    float acc[W], lse = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.f;
    if (m != -INFINITY) {
        float l = 0.f;
        for (int i = lane; i < a.splits; i += 32) l += exp2_approx(pl[i] - m);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(~0u, l, d);
        lse = m + log2f(l);
        const float* part = a.part + row * a.splits * D + lane * W;
        // kBatch parts at a time, their loads before the first use; one without keys is not read
        for (int p = 0; p < a.splits; p += kBatch) {
            float f[kBatch], v[kBatch][W];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) f[k] = p + k < a.splits ? pl[p + k] : -INFINITY;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i) v[k][i] = f[k] != -INFINITY ? part[(long long)(p + k) * D + i] : 0.f;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i) acc[i] = fmaf(exp2_approx(f[k] - lse), v[k][i], acc[i]);
        }
    }
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row * D) + lane * (W / 2);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) out[i] = pack2<T>(acc[2 * i], acc[2 * i + 1]);
    if (a.lse && lane == 0) a.lse[row] = lse * 0.6931471805599453f;
}

template <typename T, int D, int NT> cudaError_t launch_rows(const WindowArgs& a, cudaStream_t s) {
    static PerDevice ready;
    const cudaError_t e = allow_smem(ready, window_kernel<T, D, NT>, Ring<D>::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.splits * a.row_tiles * a.Hkv), (unsigned)a.B);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = Ring<D>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.clustered ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, window_kernel<T, D, NT>, a);
}

template <typename T, int D>
cudaError_t launch_typed(const WindowArgs& a, const WindowPlan& p, cudaStream_t s, int* launched) {
    cudaError_t e = p.dense          ? launch_window_dense(a, std::is_same<T, __half>::value ? IDX_FP16 : IDX_BF16, s)
                    : p.tile_rows == 8 ? launch_rows<T, D, 1>(a, s) : launch_rows<T, D, 2>(a, s);
    if (e != cudaSuccess) return e;
    ++*launched;
    if (a.splits == 1 || a.clustered) return e;
    const long long rows = (long long)a.T * a.Hq, per = kJoinThreads / 32;
    e = launch_k(window_join_kernel<T, D>, dim3((unsigned)((rows + per - 1) / per)), dim3(kJoinThreads), 0, s, true, a);
    if (e == cudaSuccess) ++*launched;
    return e;
}

}  // namespace

// Row splits (a row's results of one split: D + 1 floats of workspace) that a plan may take: 34 MB at D =
// 128.  The plan chooses within this and the workspace is sized by it, so that the size grows with the
// rows and the lengths, as the choice itself does not.
constexpr size_t kRowSplits = 65536;
constexpr int kMostSplits = 64;

WindowPlan window_plan(int B, int T, int max_q, int Hq, int Hkv, int D, int max_len, int window, int sink, int path,
                       int sm_count) {
    WindowPlan p;
    const int G = Hq / Hkv;
    const size_t rows = (size_t)T * Hq;
    if (max_len == 0) path = -1;  // no key at all, perhaps no cache: nothing for the dense path to copy
    const long long most_rows = (long long)max_q * G;  // of a request and key head
    // keys that a tile of `tokens` tokens sees at most
    auto keys_of = [&](long long tokens) {
        return window == 0 ? (long long)max_len : std::min<long long>(max_len, (long long)window + sink + tokens);
    };
    // steps of `keys` keys that they lie in at most: those of the first tokens, and one more at either end of the window
    auto steps_of = [&](long long tokens, int keys) {
        const long long all = std::max<long long>(1, ((long long)max_len + keys - 1) / keys);
        return window == 0 ? all
                           : std::min(all, ((long long)sink + keys - 1) / keys + ((long long)window + tokens) / keys + 2);
    };
    // row tiles over the batch: of requests with max_q tokens, but no more than the call's tokens fill
    auto tiles_over = [&](long long per_request, double rows_per_tile) {
        return Hkv * std::min((double)B * per_request, (double)T * G / rows_per_tile + B);
    };
    const int dense_keys = window_dense_keys(D);
    const long long far = keys_of(max_q);
    const size_t most = far <= dense_keys
                            ? 0
                            : std::min<size_t>(rows * std::min<long long>(kMostSplits, (far + dense_keys - 1) / dense_keys),
                                               kRowSplits);
    const double join_us = (double)rows * D * 8 / 5e6;
    double best = 0;
    // `count` tiles whose keys are `units` units, in s splits; time(t, blocks): that of blocks of t units each
    // A cluster joins its splits sooner than a second launch does (16 requests behind a window of 4096 in 4 splits: 27
    // and 30 us), but must find room for all of its blocks at once: where blocks wait for others to end it costs
    // more (64 requests of 8192-16384 keys in 6 splits: 231 and 203 us).  `resident`: blocks that run at the same time.
    auto consider = [&](bool dense, int tile_rows, long long row_tiles, double count, long long units, int unit, int s,
                        double resident, auto time) {
        const long long t = (units + s - 1) / s, all = (units + t - 1) / t, half = (units / 2 + t) / t;
        if (all > 1 && all * rows > most) return;
        // lengths are on the device: the mean of the times with all of them at max_len and at half of it
        const bool clustered = !dense && all > 1 && all <= kWindowCluster && count * all <= resident;
        const double us = (time(t, count * all) + time(t, count * half)) / 2 +
                          (clustered ? 1.0 : all > 1 ? all * join_us + 3.5 : 0.0);
        if (best != 0 && us >= best) return;
        best = us;
        p.dense = dense;
        p.clustered = clustered;
        p.tile_rows = tile_rows;
        p.row_tiles = (int)row_tiles;
        p.splits = (int)all;
        p.chunk = (int)t * unit;
    };
    auto more = [](int s) { return s + (s < 8 ? 1 : s / 4); };
    if (path <= 0) {
        // Tiles of 8 or 16 rows: one of n blocks on an SM, four at most (three of 16 rows), takes 128 keys in 0.75 +
        // 0.3 n us, and 5 us to start and end (D = 128, 8 rows).
        const int tile_rows = most_rows <= 8 ? 8 : 16, slots = tile_rows == 8 ? 4 : 3;
        const double slower = (tile_rows == 8 ? 1.0 : 1.6) * (D == 128 ? 1.0 : 0.6);
        const long long tiles = (most_rows + tile_rows - 1) / tile_rows, tokens = (tile_rows + G - 1) / G + 1;
        const long long units = (steps_of(tokens, kWindowStep) + kWarps - 1) / kWarps;
        for (int s = 1; s <= kMostSplits && s <= units; s = more(s))
            consider(false, tile_rows, tiles, tiles_over(tiles, tile_rows), units, kWarps, s,
                     (double)slots * sm_count, [&](long long t, double blocks) {
                         const double on_sm = std::ceil(blocks / sm_count), full = std::floor(on_sm / slots);
                         const double rest = on_sm - full * slots;
                         auto wave = [&](double n) { return t * (0.75 + 0.3 * n) * slower + 5.0; };
                         return full * wave(slots) + (rest > 0 ? wave(rest) : 0.0);
                     });
    }
    if (path > 0 || (path == 0 && most_rows > 16)) {
        // Dense: a CTA per SM takes a key tile for 256 rows in about 1.7 us, for 128 (two streams in turn) in 1.1.
        const int tokens = 128 / G;
        const long long pairs = ((max_q + tokens - 1) / tokens + 1) / 2;
        const long long units = steps_of(2 * tokens, dense_keys);
        const double tile_us = max_q > tokens ? 1.7 : 1.1;
        for (int s = 1; s <= kMostSplits && s <= units; s = more(s))
            consider(true, 128, pairs, tiles_over(pairs, 2.0 * tokens * G), units, 1, s, 0.0,
                     [&](long long t, double blocks) { return std::ceil(blocks / sm_count) * (t * tile_us + 6.0); });
    }
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    p.part = 0;
    p.part_lse = up(most * D * sizeof(float));
    p.total = p.part_lse + up(most * sizeof(float));
    return p;
}

cudaError_t launch_window(const WindowArgs& a, const WindowPlan& p, idx_dtype dt, cudaStream_t s, int* launched) {
    if (dt == IDX_BF16)
        return a.D == 128 ? launch_typed<__nv_bfloat16, 128>(a, p, s, launched)
                          : launch_typed<__nv_bfloat16, 64>(a, p, s, launched);
    return a.D == 128 ? launch_typed<__half, 128>(a, p, s, launched) : launch_typed<__half, 64>(a, p, s, launched);
}

}  // namespace idx
