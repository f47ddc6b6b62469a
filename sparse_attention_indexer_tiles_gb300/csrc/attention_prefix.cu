// The shared prefix's parts of the decode attention on the 5th-generation tensor cores.
//
// The rows of a key head over the whole batch (B * Q * G of them) read the same prefix
// keys, so they are the rows of two dense products per key tile,
//     S = Q K^T  (128 rows x tile keys, over D),    O += P V  (128 rows x D, over keys),
// with P = 2^(S scale_log2 - m) between them.  A CTA runs two streams, each with its own
// S, P and O in TMEM and its own four softmax warps (one thread per row):
//   * two row tiles over the same keys (each K and V tile in shared memory serves both), or
//   * for a last, odd row tile, the same rows over the even and the odd key tiles, joined
//     through shared memory at the end.
// P is written to TMEM in the tensors' type and is the A operand of the second product; V is
// used as it lies in memory (its rows are the product's K axis, so the B operand is
// MN-major).  Warps 8 and 10 issue the streams' MMAs, warps 9 and 11 the TMA copies of K and
// of V through one ring.  A copy brings whole rows of a page into groups of 8 keys, each
// group's 64-column halves one after the other (1024 bytes each, 128-byte swizzled).
//
// Tile width: S and P have columns of their own, so the next S is computed while the
// softmax works on this one, and nothing waits for a product's end before the next is
// issued.  Beside two O of D columns, 512 columns leave 128 per stream at D = 128: 80 keys
// (80 + 40).  Tiles of 128 keys with P over S cost a wait for P V before every Q K^T.
//
// The private parts of requests with many rows per key head (several new tokens) are taken the
// same way, with a request's own rows, pages and length (PRIVATE): they also mask the tokens
// after a row's own and leave the logits that the weights are made from.
//
// The running maximum m is renewed only when a row's maximum has grown by more than 8 (a
// factor 256; P <= 256 then in bf16, 2^15 in fp16), so O is rarely rescaled; the sum l
// and O stay relative to the m in use, in fp32, and the result does not depend on it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.cuh"
#include "dense.cuh"

namespace idx {

namespace {

constexpr int kRows = 128;                 // rows per tile
constexpr int kHalfQ = kRows * 128;        // 64 columns of a row tile, 128-byte swizzled
constexpr int kSoftmaxWarps = 8;
constexpr int kPrefixThreads = (kSoftmaxWarps + 4) * 32;  // and two issuers, two producers

template <int D> struct PrefixCfg {
    static constexpr int KEYS = attn_prefix_keys(D);         // per tile
    static constexpr int HALVES = D / 64;
    static constexpr int QTILE = HALVES * kHalfQ;
    static constexpr int GROUP = HALVES * 1024;              // 8 keys of a K or V tile
    static constexpr int TILE = KEYS / 8 * GROUP;
    // Ring slots, K and V tiles in turn.  An even number, so that a slot only ever holds K or
    // only V and its one producer sees every phase of its barriers: with an odd number a
    // producer could wait on a slot whose last tile but one, of the other producer's, was
    // still wanted, and the parity of its wait would let it through.
    static constexpr int NS = 8;
    static_assert(NS % 2 == 0, "");
    static constexpr int OFF_KV = 2 * QTILE;
    static constexpr int OFF_BAR = OFF_KV + NS * TILE;
    static constexpr int NBAR = 1 + 2 * NS + 10;
    static constexpr int OFF_CTL = OFF_BAR + NBAR * 8;       // [0] TMEM base, [1] abort flag
    static constexpr int OFF_ML = OFF_CTL + 8;              // the odd stream's m and l
    static constexpr int SMEM = OFF_ML + kRows * 8 + 1024;
    // TMEM columns: S and P of a stream, then both O
    static constexpr int COL_P = KEYS, COL_STREAM = D == 128 ? 128 : KEYS + KEYS / 2;
    static constexpr int COL_O = 512 - 2 * D;
    static_assert(SMEM <= 227 * 1024, "");
    static_assert(KEYS + KEYS / 2 <= COL_STREAM && 2 * COL_STREAM <= COL_O, "");
    static_assert(kRows * D * 4 <= NS * TILE, "the odd stream's O is joined through the ring");
};

// Registers: the launch gives 384 x 168; the softmax warps (a row of S each thread) take
// 256 x 208, the others keep 128 x 80.
IDX_DEVI void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory"); }
IDX_DEVI void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" ::: "memory"); }
static_assert(256 * 208 + 128 * 80 <= 384 * 168, "");

// From the start of the first three axes.
IDX_DEVI void tma_load_5d(uint32_t dst, const void* tmap, uint64_t* bar, int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(0), "r"(c3), "r"(c4)
        : "memory");
}

template <typename T, int D, bool PRIVATE>
__global__ void __launch_bounds__(kPrefixThreads, 1)
attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnArgs a) {
    using C = PrefixCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* full = qfull + 1;
    uint64_t* empty = full + C::NS;
    uint64_t* sfull = empty + C::NS;  // per stream: S is there
    uint64_t* sfree = sfull + 2;      // S has been read
    uint64_t* pfull = sfree + 2;      // P is there
    uint64_t* pvdone = pfull + 2;     // O has the tile's P V, P has been read
    uint64_t* done = pvdone + 2;      // every MMA of the stream
    volatile uint32_t* tslot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_CTL);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_CTL + 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!PRIVATE || a.prefix_splits == 0) pdl_wait();  // the call's first launch
    pdl_trigger();  // the private parts may take the SMs that this grid leaves idle

    // this CTA: key head, pair of row tiles, part of the prefix
    const int tokens = a.prefix_tokens;  // query tokens per row tile (its rows: tokens * G <= 128)
    const int pair = blockIdx.x, split = blockIdx.y;
    const int hk = PRIVATE ? blockIdx.z % a.Hkv : blockIdx.z, b = PRIVATE ? blockIdx.z / a.Hkv : 0;
    const int all_tokens = PRIVATE ? a.Q : a.B * a.Q, token0 = b * a.Q;  // whose rows these are
    const bool solo = (2 * pair + 1) * tokens >= all_tokens;
    const int total_splits = a.prefix_splits + a.private_splits;
    const int slot = PRIVATE ? a.prefix_splits + split : split;
    const int* const table = PRIVATE ? a.table + b * a.table_stride : a.prefix_table;
    int len = a.prefix_len;
    if constexpr (PRIVATE) {
        len = a.lens[b];
        if ((len < 0 || len > a.max_len) && tid == 0) raise_status(a.d_status, IDX_DEV_RANGE);
        len = min(max(len, 0), a.max_len);
    }
    const int chunk = PRIVATE ? a.private_chunk : a.prefix_chunk;
    const int lo = split * chunk, hi = min(len, lo + chunk);
    // (one CTA's wait for the prefix's grid makes the join's wait for this one cover both)
    const bool last = PRIVATE && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
    if (PRIVATE && lo >= hi) {  // no keys in this part
        for (int i = tid; i < 2 * tokens * a.G; i += kPrefixThreads) {
            const int t = 2 * pair * tokens + i / a.G;
            if (t < all_tokens)
                a.part_lse[((long long)(token0 + t) * a.Hq + hk * a.G + i % a.G) * total_splits + slot] =
                    -INFINITY;
        }
        if (last) pdl_wait();
        return;
    }
    const int n = (hi - lo + C::KEYS - 1) / C::KEYS;  // key tiles, at least one

    const uint32_t kv = smem_u32(smem + C::OFF_KV);
    // K and V tiles in turn, `unit` keys of a page per copy; keys past the end and pages that
    // do not exist read as zeros past the last page.  A lane looks up a copy's page.
    bool bad = false;
    const int unit = a.prefix_unit, copies = C::KEYS / unit;
    auto page_of = [&](int x) {
        const int key = lo + (x >> 1) * C::KEYS + lane * unit;
        int page = a.pages;
        if (lane < copies && x < 2 * n && key < hi) {
            page = table[key >> a.page_shift];
            if (page < 0 || page >= a.pages) {
                page = a.pages;
                bad = true;
            }
        }
        return page;
    };
    auto fetch = [&](int x, int pages) {
        const int slot = x % C::NS;
        if (elect_one()) mbar_arrive_expect_tx(&full[slot], C::TILE);
        __syncwarp();
        for (int u = 0; u < copies; ++u) {
            const int page = __shfl_sync(~0u, pages, u);
            const int key = lo + (x >> 1) * C::KEYS + u * unit;
            if (elect_one())
                tma_load_5d(kv + slot * C::TILE + u * unit / 8 * C::GROUP, x & 1 ? &tm_v : &tm_k,
                            &full[slot], (key & (a.page_size - 1)) / 8,
                            page == a.pages ? a.pages * a.Hkv : page * a.Hkv + hk);
            __syncwarp();
        }
    };
    const int first = a.withhold_tile >= 0 ? min(2 * n, 2 * a.withhold_tile) : 2 * n;  // tiles that come
    int page = 0;  // of the producer's next tile, looked up ahead
    if (warp == 9 || warp == 11) page = page_of(warp == 11);
    if (warp == 9) {
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            *abort_flag = 0;
        }
        // a barrier per lane, in their order: q; full, empty (the streams that read a tile);
        // per stream S, S free, P (a warp each), P V, done
        for (int i = lane; i < C::NBAR; i += 32) {
            const int k = (i - 1 - 2 * C::NS) / 2;
            mbar_init(qfull + i, i <= C::NS ? 1 : i <= 2 * C::NS ? (solo ? 1 : 2)
                                                                 : k == 1 || k == 2 ? 4 : 1);
        }
        fence_barrier_init();
        __syncwarp();
        if (lane == 0) {
            // q does not wait for the rest of the block
            const int tiles = solo ? 1 : 2;
            mbar_arrive_expect_tx(qfull, tiles * C::HALVES * tokens * a.G * 128);
            for (int t = 0; t < tiles; ++t)
                for (int h = 0; h < C::HALVES; ++h)
                    tma_load_4d(smem_u32(smem) + t * C::QTILE + h * kHalfQ, &tm_q, qfull, h * 64, 0,
                                hk, token0 + (2 * pair + t) * tokens);
        }
        __syncwarp();
    }
    if (warp == 8) {
        tmem_alloc(const_cast<uint32_t*>(tslot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto give_up = [&] {
        *abort_flag = 1;
        raise_status(a.d_status, IDX_DEV_TIMEOUT);
    };

    if (warp >= 8) {
        regs_less();
        if (warp == 9 || warp == 11) {
            // ----------------------------------------- TMA producers: K tiles, V tiles
            int x = warp == 11;
            for (; x < first; x += 2) {
                const int next = page_of(x + 2);  // looked up a tile ahead
                bool ok = true;
                if (x >= C::NS)
                    ok = __all_sync(~0u, mbar_wait(&empty[x % C::NS], ((x / C::NS) & 1) ^ 1,
                                                   abort_flag, a.wait_limit));
                if (!ok) {
                    if (lane == 0) give_up();
                    break;
                }
                fetch(x, page);
                page = next;
            }
            if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
            // Nothing may be in flight when the CTA ends: the last copy into each of this
            // warp's slots has landed.
            for (int y = x - 2; y >= 0 && y >= x - C::NS; y -= 2)
                if (y < first) mbar_wait(&full[y % C::NS], (y / C::NS) & 1, nullptr, 1ll << 28);
            if (warp == 9) mbar_wait(qfull, 0, nullptr, 1ll << 28);
            __syncwarp();
        } else {
            // -------------------------------------------------- MMA issuers
            // One warp per stream: while the tensor core reads its operands an mbarrier
            // access takes about 140 clocks, and one warp that waited for both streams
            // was the bottleneck (4200 clocks per pair of tiles against 2048 of MMAs).
            // The whole warp runs the control flow, so that descriptors stay in uniform
            // registers, and one elected lane issues.
            const int s = warp == 10;
            const uint32_t id_s = instr_desc(Elem<T>::FMT, kRows, C::KEYS);
            const uint32_t id_o = instr_desc(Elem<T>::FMT, kRows, D) | (1u << 16);  // B is MN-major
            const uint32_t t_s = tmem + s * C::COL_STREAM, t_p = t_s + C::COL_P;
            const uint32_t t_o = tmem + C::COL_O + s * D;
            const int mine = solo ? (n + 1 - s) / 2 : n;
            auto tile_of = [&](int i) { return solo ? 2 * i + s : i; };
            // K or V tile x has landed, and a softmax barrier's i-th phase has completed
            auto both = [&](int x, uint64_t* bar, int i) {
                return __all_sync(~0u, mbar_wait2(&full[x % C::NS], (x / C::NS) & 1, bar, i & 1,
                                                  abort_flag, a.wait_limit));
            };
            const uint64_t q = smem_desc(smem_u32(smem) + (solo ? 0 : s) * C::QTILE, 128);
            // S of the i-th tile (K has landed, the last S has been read)
            auto qk = [&](int i) {
                const int x = 2 * tile_of(i);
                tc_fence_after();
                const uint64_t k = kv_desc(kv + (x % C::NS) * C::TILE, C::GROUP);
                if (elect_one()) {
#pragma unroll
                    for (int d = 0; d < D / 16; ++d)
                        mma_bf16(t_s, q + (((d / 4) * kHalfQ + (d % 4) * 32) >> 4),
                                 k + (((d / 4) * 1024 + (d % 4) * 32) >> 4), id_s, d > 0);
                    mma_commit(&sfull[s]);
                    mma_commit(&empty[x % C::NS]);
                }
                __syncwarp();
            };
            // O += P V (V has landed, P is there)
            auto pv = [&](int i) {
                const int x = 2 * tile_of(i) + 1;
                tc_fence_after();
                const uint64_t v = kv_desc(kv + (x % C::NS) * C::TILE, C::GROUP);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < C::KEYS / 16; ++k)
                        mma_ts(t_o, t_p + k * 8, v + k * (2 * C::GROUP >> 4), id_o, i > 0 || k > 0);
                    mma_commit(&pvdone[s]);
                    mma_commit(&empty[x % C::NS]);
                }
                __syncwarp();
            };
            bool ok = true;
            if (mine > 0) {
                ok = both(2 * tile_of(0), qfull, 0);
                if (ok) qk(0);
            }
            for (int i = 0; i < mine && ok; ++i) {
                if (i + 1 < mine) {  // S of the next tile under this one's softmax
                    if (!(ok = both(2 * tile_of(i + 1), &sfree[s], i))) break;
                    qk(i + 1);
                }
                if (!(ok = both(2 * tile_of(i) + 1, &pfull[s], i))) break;
                pv(i);
            }
            if (!ok && lane == 0) give_up();
            if (elect_one()) {
                mma_commit(&done[s]);  // nothing may be in flight when TMEM is freed
                mbar_wait(&done[s], 0, nullptr, 1ll << 28);
            }
            __syncwarp();
        }
    } else {
        regs_more();
        // --------------------------------------------- softmax, one thread per row
        const int s = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + s * C::COL_STREAM, to = tmem + lanes + C::COL_O + s * D;
        const int tile = 2 * pair + (solo ? 0 : s);
        const int bt = tile * tokens + row / a.G;  // token of the row, from token0 on
        const bool live = row < tokens * a.G && bt < all_tokens;
        // a private row does not see the tokens after its own
        const int see = PRIVATE ? min(hi, len - (a.Q - 1 - bt)) : hi;
        const int see_all = PRIVATE ? min(hi, len - (a.Q - 1)) : hi;  // what every row sees
        float* logits = nullptr;
        if (PRIVATE && a.logits && live)
            logits = a.logits + (((long long)b * a.Hkv + hk) * (a.Q * a.G) +
                                 tile * tokens * a.G + row) * a.logit_stride + lo;
        const int mine = solo ? (n + 1 - s) / 2 : n;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < mine; ++i) {
            const int t = solo ? 2 * i + s : i;
            ok = __all_sync(~0u, mbar_wait(&sfull[s], i & 1, abort_flag, a.wait_limit));
            if (!ok) break;
            tc_fence_after();
            float z[C::KEYS];
#pragma unroll
            for (int c = 0; c < C::KEYS / 32; ++c) tmem_ld32x32b<32>(ts + c * 32, z + c * 32);
            if constexpr (C::KEYS % 32 != 0)
                tmem_ld32x32b<C::KEYS % 32>(ts + C::KEYS / 32 * 32, z + C::KEYS / 32 * 32);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfree[s]);  // the next S may be computed
            const int valid = hi - lo - t * C::KEYS;  // keys of this tile
            float scale = a.scale_log2;
            // uniform; the maximum below wants scale >= 0
            if (see_all - lo - t * C::KEYS < C::KEYS || scale < 0.f || (PRIVATE && a.logits)) {
                const int mine_valid = see - lo - t * C::KEYS;
#pragma unroll
                for (int c = 0; c < C::KEYS; ++c) z[c] = c < mine_valid ? z[c] * scale : -INFINITY;
                scale = 1.f;
                if (PRIVATE && logits) {
#pragma unroll
                    for (int c = 0; c < C::KEYS; c += 4)
                        if (c < valid)
                            *reinterpret_cast<float4*>(logits + t * C::KEYS + c) =
                                make_float4(z[c], z[c + 1], z[c + 2], z[c + 3]);
                }
            }
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < C::KEYS; c += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = max3(x[j], z[c + 2 * j], z[c + 2 * j + 1]);
            const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * scale - Elem<T>::LIFT;
            // O is at rest and P has been read once the last P V has completed
            auto last_done = [&] {
                return i == 0 || __all_sync(~0u, mbar_wait(&pvdone[s], (i - 1) & 1, abort_flag,
                                                           a.wait_limit));
            };
            if (i == 0) {
                m = top == -INFINITY ? 0.f : top;
            } else if (__any_sync(~0u, live && top > m + kRenew)) {
                const float next = live ? fmaxf(m, top) : m;
                const float f = exp2_approx(m - next);
                m = next;
                l *= f;
                if (!(ok = last_done())) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    uint32_t r[32];
                    tmem_ld32x32b<32>(to + c * 32, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(o[j] * f);
                    tmem_st32x32b<32>(to + c * 32, r);
                }
            }
            if (valid < C::KEYS) {
                // V's rows past the end hold anything; their weights are 0, so they must be finite
                const int v = 2 * t + 1;
                ok = __all_sync(~0u, mbar_wait(&full[v % C::NS], (v / C::NS) & 1, abort_flag,
                                               a.wait_limit));
                if (!ok) break;
                uint8_t* vt = smem + C::OFF_KV + (v % C::NS) * C::TILE;
                for (int c = row; c < (C::KEYS - valid) * 8 * C::HALVES; c += 128) {
                    const int key = valid + c / (8 * C::HALVES), at = c % (8 * C::HALVES);
                    *reinterpret_cast<uint4*>(vt + key / 8 * C::GROUP + at / 8 * 1024 +
                                              key % 8 * 128 + at % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 scale2 = make_float2(scale, scale), less_m = make_float2(-m, -m);
            uint32_t p[C::KEYS / 2];
#pragma unroll
            for (int c = 0; c < C::KEYS / 2; ++c) {
                float2 e = fma2(make_float2(z[2 * c], z[2 * c + 1]), scale2, less_m);
                e.x = exp2_approx(e.x);
                e.y = exp2_approx(e.y);
                sum[c & 1] = add2(sum[c & 1], e);
                p[c] = pack2<T>(e.x, e.y);
            }
            const float2 both = add2(sum[0], sum[1]);
            l += both.x + both.y;
            if (!(ok = last_done())) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < C::KEYS / 64; ++c) tmem_st32x32b<32>(ts + C::COL_P + c * 32, p + c * 32);
            if constexpr (C::KEYS % 64 != 0)
                tmem_st32x32b<C::KEYS % 64 / 2>(ts + C::COL_P + C::KEYS / 64 * 32, p + C::KEYS / 64 * 32);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[s]);
        }
        if (mine > 0 && ok)
            ok = __all_sync(~0u, mbar_wait(&pvdone[s], (mine - 1) & 1, abort_flag, a.wait_limit));
        if (!ok && lane == 0) give_up();
        tc_fence_after();
        if (l == 0.f) m = -INFINITY;  // nothing seen: no part in a join
        float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
        float4* join = reinterpret_cast<float4*>(smem + C::OFF_KV);  // [D / 4][128]
        if (solo && s == 1) {
            // hand O over to stream 0, which waits until both streams' MMAs are done
            named_bar_sync(1, 256);
            if (mine > 0 && ok) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32x32b<32>(to + c * 32, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        join[(c * 8 + j) * 128 + row] =
                            make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
            }
            ml[row] = mine > 0 && ok ? m : -INFINITY;
            ml[128 + row] = mine > 0 && ok ? l : 0.f;
            named_bar_sync(1, 256);
        } else {
            float f0 = 1.f, f1 = 0.f;
            float top = m;
            if (solo) {
                named_bar_sync(1, 256);
                named_bar_sync(1, 256);
                top = fmaxf(m, ml[row]);
                const float base = top == -INFINITY ? 0.f : top;
                f0 = exp2_approx(m - base);
                f1 = exp2_approx(ml[row] - base);
                l = l * f0 + ml[128 + row] * f1;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays one
            f0 *= inv;
            f1 *= inv;
            // Rows leave through the stream's own Q tile (its products are done): a thread
            // holds a row, a warp writes whole rows.  16-byte chunks are xor-ed with the row.
            constexpr int kCols = C::QTILE / (128 * 4), kChunk = kCols / 4;
            uint8_t* stage = smem + s * C::QTILE;
            const int r0 = row & ~31;
            const long long part =
                ((long long)(token0 + bt) * a.Hq + hk * a.G + row % a.G) * total_splits + slot;
            float* const mine_at = live ? a.part + part * D : nullptr;
            for (int c0 = 0; c0 < D; c0 += kCols) {
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    float o[32];
                    tmem_ld32x32b<32>(to + c0 + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float4 v = make_float4(o[4 * j] * f0, o[4 * j + 1] * f0, o[4 * j + 2] * f0,
                                               o[4 * j + 3] * f0);
                        if (solo && f1 > 0.f) {
                            const float4 w = join[((c0 + c) / 4 + j) * 128 + row];
                            v.x += w.x * f1;
                            v.y += w.y * f1;
                            v.z += w.z * f1;
                            v.w += w.w * f1;
                        }
                        *reinterpret_cast<float4*>(stage + row * (kCols * 4) +
                                                   (((c / 4 + j) ^ (row & (kChunk - 1))) * 16)) = v;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                    const int r = (k * 32 + lane) / kChunk, c = lane % kChunk;
                    float* to_row = reinterpret_cast<float*>(
                        __shfl_sync(~0u, reinterpret_cast<unsigned long long>(mine_at), r));
                    const float4 v = *reinterpret_cast<const float4*>(
                        stage + (r0 + r) * (kCols * 4) + ((c ^ (r & (kChunk - 1))) * 16));
                    if (to_row) *reinterpret_cast<float4*>(to_row + c0 + c * 4) = v;
                }
                __syncwarp();
            }
            if (live) a.part_lse[part] = l == 0.f ? -INFINITY : top + log2f(l);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (last) pdl_wait();
}

template <typename T, int D, bool PRIVATE>
cudaError_t launch_t(const AttnArgs& args, cudaStream_t s) {
    using C = PrefixCfg<D>;
    AttnArgs a = args;
    // keys per copy: a whole page where it divides the tile, else 16 (no page is smaller)
    a.prefix_unit = C::KEYS % a.page_size == 0 ? a.page_size : 16;
    CUtensorMap tq, tk, tv;
    const int tokens = kRows / a.G;
    a.prefix_tokens = tokens;
    const uint64_t row = D * 2;
    // q: 64 columns, the heads of a group, groups, tokens
    const cuuint64_t qd[4] = {(uint64_t)D, (uint64_t)a.G, (uint64_t)a.Hkv, (uint64_t)a.B * a.Q};
    const cuuint64_t qs[3] = {row, row * a.G, row * a.Hq};
    const cuuint32_t qb[4] = {64, (uint32_t)a.G, 1, (uint32_t)tokens};
    // K, V: 64 columns, 8 keys, the halves of a row, groups of 8 keys, pages and heads
    const cuuint64_t kd[5] = {64, 8, (uint64_t)C::HALVES, (uint64_t)a.page_size / 8,
                              (uint64_t)a.pages * a.Hkv};
    const cuuint64_t ks[4] = {row, 128, row * 8, row * a.page_size};
    const cuuint32_t kb[5] = {64, 8, (uint32_t)C::HALVES, (uint32_t)a.prefix_unit / 8, 1};
    if (make_map<4>(&tq, a.q, qd, qs, qb) != CUDA_SUCCESS ||
        make_map<5>(&tk, a.k, kd, ks, kb) != CUDA_SUCCESS ||
        make_map<5>(&tv, a.v, kd, ks, kb) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static PerDevice ready;
    const cudaError_t e = allow_smem(ready, attn_prefix_kernel<T, D, PRIVATE>, C::SMEM);
    if (e != cudaSuccess) return e;
    const int ntiles = ((PRIVATE ? a.Q : a.B * a.Q) + tokens - 1) / tokens;
    return launch_k(attn_prefix_kernel<T, D, PRIVATE>,
                    dim3((ntiles + 1) / 2, PRIVATE ? a.private_splits : a.prefix_splits,
                         PRIVATE ? a.B * a.Hkv : a.Hkv),
                    dim3(kPrefixThreads), C::SMEM, s, true, tq, tk, tv, a);
}

template <bool PRIVATE>
cudaError_t launch_dense(const AttnArgs& a, idx_dtype dt, cudaStream_t s) {
    if (dt == IDX_BF16)
        return a.D == 128 ? launch_t<__nv_bfloat16, 128, PRIVATE>(a, s)
                          : launch_t<__nv_bfloat16, 64, PRIVATE>(a, s);
    return a.D == 128 ? launch_t<__half, 128, PRIVATE>(a, s)
                      : launch_t<__half, 64, PRIVATE>(a, s);
}

}  // namespace

cudaError_t launch_prefix_parts(const AttnArgs& a, idx_dtype dt, cudaStream_t s) {
    return launch_dense<false>(a, dt, s);
}

cudaError_t launch_private_dense(const AttnArgs& a, idx_dtype dt, cudaStream_t s) {
    return launch_dense<true>(a, dt, s);
}

}  // namespace idx
