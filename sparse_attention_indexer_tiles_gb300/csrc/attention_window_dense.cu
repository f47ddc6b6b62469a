// The windowed attention over an MXFP4 cache (attention_window.cu) for requests with many rows per key head,
// prompts above all, on the 5th-generation tensor cores.
//
// The rows of a request and key head (its new tokens times the heads of the group) read the same keys: per key
// tile S = Q K^T (128 rows x tile keys, over D) and O += P V, as the shared prefix's parts are taken
// (attention_prefix.cu: two streams of 128 rows with S, P and O in TMEM columns of their own, a softmax thread per
// row, an issuing warp per stream, K and V tiles in turn through one ring).  What differs is how tiles come: TMA
// brings codes and scales to a small ring of their own, and five warps write the values that they stand for, in q's
// type, where the matrix instructions read them (rows of 64 columns, 128-byte swizzled).  (Codes that these warps
// loaded into registers a tile ahead were late: 4096 tokens behind one another 381 us, 315 from the ring.)  The values
// are the codes times powers of two, so bf16 holds them exactly; fp16 does from 2^-23 on and rounds smaller ones
// to multiples of 2^-24.  A value that q's type cannot hold (scales above 2^125, in fp16 above 2^13) counts as a NaN
// scale.  K of a slot with a NaN scale becomes NaN and its V 0, so that exactly the rows that see it are NaN.
//
// The keys that rows of the two streams see are taken in units of 16 (a copy each), those of the first tokens before
// those of the window, and tiles are made of units in this order, so that the first tokens do not cost a tile of their
// own (ragged prompts behind a window of 1024: 931 us with a tile of their own, 846 without).  Bounded by the
// instructions of the softmax and the expansion.
#include "dense.cuh"
#include "window_span.cuh"

namespace idx {

namespace {

constexpr int kRows = 128;                 // rows per tile
constexpr int kHalfQ = kRows * 128;        // 64 columns of a row tile, 128-byte swizzled
constexpr int kThreads = 16 * 32;          // 8 softmax warps, 2 issuers, one for copies, 5 that expand codes
constexpr int kExpandWarp = 11, kExpandWarps = 5;  // the first of them, and how many

// Keys per tile: what TMEM holds at D = 128, what a softmax thread's registers hold at D = 64.
__host__ __device__ constexpr int dense_keys(int D) { return D == 128 ? 80 : 96; }

template <int D> struct DenseCfg {
    static constexpr int KEYS = dense_keys(D);               // per tile
    static constexpr int HALVES = D / 64;
    static constexpr int BLOCKS = D / 32;                    // of a row's scales
    static constexpr int QTILE = HALVES * kHalfQ;
    static constexpr int GROUP = HALVES * 1024;              // 8 keys of a K or V tile
    static constexpr int TILE = KEYS / 8 * GROUP;
    static constexpr int NS = 6;                             // ring slots, an even number: K or V only
    // codes and scales as they lie in the cache: a ring of tiles of their own
    static constexpr int ROW = D / 2;
    static constexpr int RS = 3;
    static constexpr int OFF_RV = KEYS * ROW, OFF_RKSF = 2 * KEYS * ROW, OFF_RVSF = OFF_RKSF + KEYS * BLOCKS;
    static constexpr int RAW = (OFF_RVSF + KEYS * BLOCKS + 1023) / 1024 * 1024;
    static constexpr int UNITS = KEYS / 16;                  // copies of 16 keys per tile
    static constexpr int UNIT = 16 * ROW, UNIT_SF = 16 * BLOCKS;
    static constexpr int SUBS = 4 / BLOCKS;                  // groups of 8 keys that a warp expands at once
    static constexpr int ITEMS = (KEYS / 8 / SUBS + kExpandWarps - 1) / kExpandWarps;  // of them, per warp
    static constexpr int OFF_RAW = 2 * QTILE;
    static constexpr int OFF_KV = OFF_RAW + RS * RAW;
    static constexpr int OFF_BAR = OFF_KV + NS * TILE;
    static constexpr int NBAR = 1 + 2 * NS + 10 + 2 * RS;
    static constexpr int OFF_CTL = OFF_BAR + NBAR * 8;       // [0] TMEM base, [1] abort flag
    static constexpr int OFF_ML = OFF_CTL + 8;              // the odd stream's m and l
    static constexpr int OFF_LARGE = OFF_ML + kRows * 8;     // the last tile of each 8 that holds large values of V
    static constexpr int SMEM = OFF_LARGE + 8 * 4 + 1024;
    // TMEM columns: S and P of a stream, then both O
    static constexpr int COL_P = KEYS, COL_STREAM = D == 128 ? 128 : KEYS + KEYS / 2;
    static constexpr int COL_O = 512 - 2 * D;
    static_assert(SMEM <= 227 * 1024 && KEYS / 8 % SUBS == 0 && NBAR <= 64, "");
    static_assert(4 * UNITS <= 32 && KEYS % 16 == 0 && KEYS * ROW % 512 == 0, "a lane per copy");
    static_assert(KEYS + KEYS / 2 <= COL_STREAM && 2 * COL_STREAM <= COL_O, "");
    static_assert(kRows * D * 4 <= NS * TILE, "the odd stream's O is joined through the ring");
};

// Registers: the launch gives 512 x 128.
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= 512 * 128, "");
template <int N> IDX_DEVI void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N) : "memory"); }
template <int N> IDX_DEVI void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N) : "memory"); }

// The largest scale whose values the type holds, and its NaN twice.  LARGE: the largest scale of V with which O stays
// inside fp32 whatever the keys are: weights of a tile are at most 2^kRenew before a row's maximum is renewed, and
// 2^30 keys 2^8 6 2^87 < 2^128.  In a tile with larger ones the maximum counts as kLargeLift more, which makes its
// weights, and through the renewal all the row's others, that much smaller: 2^30 2^(8 - 40) 6 2^125 < 2^126, and the sum
// of both kinds is below 2^128.  (For all tiles it would cost small values their bits: 2^-40 of those below 2^-60 leaves
// fp32's 24.)  fp16's values are far inside.
template <typename T> struct Held;
template <> struct Held<__nv_bfloat16> {
    static constexpr uint32_t MOST = 127 + 125, NANS = 0x7fff7fffu, LARGE = 127 + 87;
};
template <> struct Held<__half> {
    static constexpr uint32_t MOST = 127 + 13, NANS = 0x7fff7fffu, LARGE = MOST;
};
constexpr float kLargeLift = 40.f;

IDX_DEVI uint32_t mul2_f16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
IDX_DEVI uint32_t mul2_bf16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A pair of codes in fp16 times 2^(sf - 127), in T, rounded once.  Scales from LEAST to EASY take one product; for
// others, up to MOST, it is the product of two factors.
template <typename T> struct Expand;
template <> struct Expand<__half> {
    // from 2^-24 on the scale is an fp16 number; below, 2^-12 of a code is one, and the second product rounds
    static constexpr uint32_t LEAST = 127 - 24, EASY = Held<__half>::MOST;
    uint32_t scale;
    IDX_DEVI explicit Expand(uint32_t sf) : Expand((int)sf - 127, 0) {}
    IDX_DEVI static Expand first(uint32_t sf) { return Expand(sf < LEAST ? -12 : (int)min(sf, EASY) - 127, 0); }
    IDX_DEVI static Expand second(uint32_t sf) { return Expand(sf < LEAST ? max((int)sf - 127 + 12, -25) : 0, 0); }
    IDX_DEVI uint32_t operator()(uint32_t h) const { return mul2_f16(h, scale); }
    IDX_DEVI uint32_t times(uint32_t x) const { return mul2_f16(x, scale); }

private:
    // 2^n, n from -24 to 15; 0 for -25 (no value of a scale below 2^-36 reaches half a step of fp16)
    IDX_DEVI Expand(int n, int) {
        const uint32_t bits = n > -15 ? (uint32_t)(n + 15) << 10 : 1u << (n + 25) >> 1;
        scale = bits | bits << 16;
    }
};
template <> struct Expand<__nv_bfloat16> {
    // an fp16 code moved to bf16's fields stands for 2^-112 of itself
    static constexpr uint32_t LEAST = 0, EASY = 254 - 112;
    uint32_t scale;
    IDX_DEVI explicit Expand(uint32_t sf) { scale = (sf + 112u) * 0x00800080u; }
    IDX_DEVI static Expand first(uint32_t sf) { return Expand(min(sf, EASY)); }
    IDX_DEVI static Expand second(uint32_t sf) {
        return Expand(15u + max(min(sf, Held<__nv_bfloat16>::MOST), EASY) - EASY);
    }
    IDX_DEVI uint32_t operator()(uint32_t h) const {
        return mul2_bf16((h >> 3 & 0x0fff0fffu) | (h & 0x80008000u), scale);
    }
    IDX_DEVI uint32_t times(uint32_t x) const { return mul2_bf16(x, scale); }
};
template <typename T> IDX_DEVI uint4 expand8(uint32_t w, const Expand<T>& f) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
    return make_uint4(f(h[0]), f(h[1]), f(h[2]), f(h[3]));
}

// blockIdx.x: pair of row tiles (the last, with the most keys, first), split, key head, request.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
window_dense_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WindowArgs a) {
    using C = DenseCfg<D>;
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
    uint64_t* rfull = done + 2;       // codes and scales of a tile have landed
    uint64_t* rempty = rfull + C::RS;
    volatile uint32_t* tslot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_CTL);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_CTL + 4);
    volatile int* large = reinterpret_cast<volatile int*>(smem + C::OFF_LARGE);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();

    const int tokens = kRows / a.G;  // query tokens per row tile
    const int pairs = a.row_tiles, pair = pairs - 1 - (int)(blockIdx.x % pairs);
    int at = blockIdx.x / pairs;
    const int split = at % a.splits;
    at /= a.splits;
    const int hk = at % a.Hkv, b = at / a.Hkv;
    const Span sp = span_of(a, b, tid == 0 && blockIdx.x % (pairs * a.splits) == 0 && hk == 0);
    const int token0 = 2 * pair * tokens;  // of the request's
    if (token0 >= sp.count) return;
    const bool solo = token0 + tokens >= sp.count;
    const int pos0 = sp.len - sp.count, last_token = min(sp.count, token0 + 2 * tokens) - 1;
    // the keys that rows of the pair see: the first tokens' and those from the oldest row's window on
    const int hi = max(0, min(sp.len, pos0 + last_token + 1));
    const int wlo = a.window > 0 ? max(0, pos0 + token0 - a.window + 1) : 0;
    const int sink = min(a.sink, hi);
    // in the order of their units: below `sinks` as they are, from there on `skip` further on
    int sinks = (sink + 15) / 16 * 16, skip = wlo / 16 * 16 - sinks;
    if (skip <= 0) sinks = skip = 0;  // no gap
    const int total = (max(0, hi - skip) + C::KEYS - 1) / C::KEYS;
    const int first = split * a.chunk, n = min(total, first + a.chunk) - first;
    auto row_of = [&](int token, int head) { return (long long)(sp.first + token) * a.Hq + hk * a.G + head; };
    if (n <= 0) {  // no keys in this split
        const int rows = (last_token + 1 - token0) * a.G;
        if (a.splits > 1) {
            for (int i = tid; i < rows; i += kThreads)
                a.part_lse[row_of(token0 + i / a.G, i % a.G) * a.splits + split] = -INFINITY;
        } else {
            for (int i = tid; i < rows * (D / 8); i += kThreads) {
                const int r = i / (D / 8);
                const long long row = row_of(token0 + r / a.G, r % a.G);
                reinterpret_cast<uint4*>(a.out)[row * (D / 8) + i % (D / 8)] = make_uint4(0u, 0u, 0u, 0u);
                if (a.lse && i % (D / 8) == 0) a.lse[row] = -INFINITY;
            }
        }
        return;
    }
    if (warp == 9) {
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            *abort_flag = 0;
        }
        // a barrier per lane, in their order: q; full (the warps that write a tile), empty (the streams
        // that read it); per stream S, S free, P (a warp each), P V, done; codes landed, read (a warp each)
        for (int i = lane; i < C::NBAR; i += 32) {
            const int k = (i - 1 - 2 * C::NS) / 2;
            const bool read = i >= 1 + 2 * C::NS + 10 + C::RS;
            mbar_init(qfull + i, i == 0                 ? 1
                                 : i <= C::NS || read   ? kExpandWarps
                                 : i <= 2 * C::NS       ? (solo ? 1 : 2)
                                 : k == 1 || k == 2     ? 4
                                                        : 1);
        }
        fence_barrier_init();
        __syncwarp();
        if (lane == 0) {
            // q does not wait for the rest of the block
            const int tiles = solo ? 1 : 2;
            mbar_arrive_expect_tx(qfull, tiles * C::HALVES * tokens * a.G * 128);
            for (int t = 0; t < tiles; ++t)
                for (int h = 0; h < C::HALVES; ++h)
                    tma_load_4d(smem_u32(smem) + t * C::QTILE + h * kHalfQ, &tm_q, qfull, h * 64, 0, hk,
                                sp.first + token0 + t * tokens);
        }
        __syncwarp();
    }
    if (tid < 8) large[tid] = -1;
    if (warp == 8) {
        tmem_alloc(const_cast<uint32_t*>(tslot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const uint32_t kv = smem_u32(smem + C::OFF_KV);
    const int tiles = a.withhold_step >= 0 ? min(n, a.withhold_step) : n;  // that come
    auto give_up = [&] {
        *abort_flag = 1;
        raise_status(a.d_status, IDX_DEV_TIMEOUT);
    };

    if (warp >= 8) {
        regs_less<kOtherRegs>();
        if (warp >= kExpandWarp) {
            // -------------------------- codes to values: K's items of a tile dealt to the warps, then V's
            const int key_in = lane & 7, block = lane >> 3 & (C::BLOCKS - 1), sub = lane / (8 * C::BLOCKS);
            const int turn = warp - kExpandWarp;
            bool ok = true;
            // one array of tile t: codes at `codes`, scales at `scales`; a NaN scale makes K (seen: also V's, at
            // `others`) NaN and V 0.  K's pass tells the softmax of large values of V that a row of the pair sees
            // (before K is there, and so before S; a place of `large` is free again 8 tiles on, the ring holds 3).
            auto expand = [&](int t, uint32_t codes, uint32_t scales, uint32_t others, bool is_v, uint32_t to) {
                uint32_t w[C::ITEMS][4], own[C::ITEMS], other[C::ITEMS];
#pragma unroll
                for (int i = 0; i < C::ITEMS; ++i) {  // all loads before the first use
                    const int key = ((i * kExpandWarps + turn) * C::SUBS + sub) * 8 + key_in;
                    if ((i * kExpandWarps + turn) * C::SUBS >= C::KEYS / 8) break;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                                 : "r"(codes + key * C::ROW +
                                       16 * (D == 128 ? block ^ (key >> 1 & 3) : block ^ (key >> 2 & 1))));
                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(own[i]) : "r"(scales + key * C::BLOCKS + block));
                    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(other[i]) : "r"(others + key * C::BLOCKS + block));
                }
#pragma unroll
                for (int i = 0; i < C::ITEMS; ++i) {
                    const int group = (i * kExpandWarps + turn) * C::SUBS + sub;
                    if ((i * kExpandWarps + turn) * C::SUBS >= C::KEYS / 8) break;
                    const uint32_t row = to + group * C::GROUP + block / 2 * 1024 + key_in * 128;
                    const uint32_t most = max(own[i], other[i]);
                    auto put = [&](int c, uint4 v) {
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         row + ((((block & 1) * 4 + c) ^ key_in) * 16)),
                                     "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                                     : "memory");
                    };
                    if (!__any_sync(~0u, most > Expand<T>::EASY || own[i] < Expand<T>::LEAST)) {
                        const Expand<T> f(own[i]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) put(c, expand8<T>(w[i][c], f));
                    } else {
                        const Expand<T> f = Expand<T>::first(own[i]), more = Expand<T>::second(own[i]);
                        const uint32_t gone = is_v ? 0u : Held<T>::NANS;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint4 v = expand8<T>(w[i][c], f);
                            v = make_uint4(more.times(v.x), more.times(v.y), more.times(v.z), more.times(v.w));
                            put(c, most > Held<T>::MOST ? make_uint4(gone, gone, gone, gone) : v);
                        }
                        if (Held<T>::LARGE < Held<T>::MOST && !is_v) {
                            const int place = (first + t) * C::KEYS + group * 8 + key_in;
                            const int key = place + (place < sinks ? 0 : skip);
                            const bool seen = key < hi && (key < sink || key >= wlo);
                            if (seen && other[i] > Held<T>::LARGE && other[i] <= Held<T>::MOST) large[t & 7] = t;
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            };
            for (int t = 0; t < tiles; ++t) {
                const uint32_t raw = smem_u32(smem + C::OFF_RAW + t % C::RS * C::RAW);
                ok = mbar_wait(&rfull[t % C::RS], t / C::RS & 1, abort_flag, a.wait_limit);
#pragma unroll
                for (int is_v = 0; is_v < 2; ++is_v) {
                    const int x = 2 * t + is_v, slot = x % C::NS;
                    if (x >= C::NS) ok = mbar_wait(&empty[slot], ((x / C::NS) & 1) ^ 1, abort_flag, a.wait_limit) && ok;
                    if (!(ok = __all_sync(~0u, ok))) break;
                    expand(t, raw + is_v * C::OFF_RV, raw + (is_v ? C::OFF_RVSF : C::OFF_RKSF), raw + C::OFF_RVSF, is_v,
                           kv + slot * C::TILE);
                    if (lane == 0) mbar_arrive(&full[slot]);
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(&rempty[t % C::RS]);
            }
            if (!ok && lane == 0) give_up();
        } else if (warp == 8 || warp == 10) {
            // ------------------------------------------------------------ MMA issuers
            // The whole warp runs the control flow, so that descriptors stay in uniform registers, and one
            // elected lane issues.
            const int s = warp == 10;
            const uint32_t id_s = instr_desc(Elem<T>::FMT, kRows, C::KEYS);
            const uint32_t id_o = instr_desc(Elem<T>::FMT, kRows, D) | (1u << 16);  // B is MN-major
            const uint32_t t_s = tmem + s * C::COL_STREAM, t_p = t_s + C::COL_P;
            const uint32_t t_o = tmem + C::COL_O + s * D;
            const int mine = solo ? (n + 1 - s) / 2 : n;
            auto tile_of = [&](int i) { return solo ? 2 * i + s : i; };
            // K or V tile x has been written, and a softmax barrier's i-th phase has completed
            auto both = [&](int x, uint64_t* bar, int i) {
                return __all_sync(~0u, mbar_wait2(&full[x % C::NS], (x / C::NS) & 1, bar, i & 1, abort_flag,
                                                  a.wait_limit));
            };
            const uint64_t q = smem_desc(smem_u32(smem) + (solo ? 0 : s) * C::QTILE, 128);
            // S of the i-th tile (K has been written, the last S has been read)
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
            // O += P V (V has been written, P is there)
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
        } else if (warp == 9) {
            // ------------------------------- codes and scales as they lie: a copy of 16 keys per lane and array
            const int unit = lane >> 2, what = lane & 3;  // K, V, K's scales, V's
            const int* const table = a.table + b * a.table_stride;
            bool bad = false;
            // first row of this lane's copy of tile i in the cache; -1: no row of the pair sees its keys
            auto look_up = [&](int i) {
                int row = -1;
                if (unit < C::UNITS && i < tiles) {
                    const int place = (first + i) * C::KEYS + unit * 16, key = place + (place < sinks ? 0 : skip);
                    if (key < hi && (key < sink || key + 16 > wlo)) {
                        const int page = table[key >> a.page_shift];
                        if (page < 0 || page >= a.pages)
                            bad = true;
                        else
                            row = (page * a.Hkv + hk) * a.page_size + (key & (a.page_size - 1));
                    }
                }
                return row;
            };
            int row = look_up(0), t = 0;
            for (; t < tiles; ++t) {
                const int next = look_up(t + 1);
                uint64_t* const bar = &rfull[t % C::RS];
                bool ok = true;
                if (t >= C::RS)
                    ok = __all_sync(~0u, mbar_wait(&rempty[t % C::RS], (t / C::RS & 1) ^ 1, abort_flag, a.wait_limit));
                if (!ok) {
                    if (lane == 0) give_up();
                    break;
                }
                const uint32_t copies = __ballot_sync(~0u, row >= 0);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, __popc(copies & 0x33333333u) * C::UNIT + __popc(copies & 0xccccccccu) * C::UNIT_SF);
                __syncwarp();
                if (row >= 0) {
                    const uint32_t raw = smem_u32(smem + C::OFF_RAW + t % C::RS * C::RAW);
                    if (what < 2)
                        tma_rows(raw + what * C::OFF_RV + unit * C::UNIT, what ? &tm_v : &tm_k, bar, row);
                    else
                        bulk_rows(raw + (what == 3 ? C::OFF_RVSF : C::OFF_RKSF) + unit * C::UNIT_SF,
                                  (what == 3 ? a.v_sf : a.k_sf) + (long long)row * C::BLOCKS, C::UNIT_SF, bar);
                }
                __syncwarp();
                row = next;
            }
            if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
            // no copy may be in flight when the CTA ends
            mbar_wait(qfull, 0, nullptr, 1ll << 28);
            for (int y = max(0, t - C::RS); y < t; ++y) mbar_wait(&rfull[y % C::RS], y / C::RS & 1, nullptr, 1ll << 28);
            __syncwarp();
        }
    } else {
        regs_more<kSoftmaxRegs>();
        // ------------------------------------------------------- softmax, one thread per row
        const int s = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + s * C::COL_STREAM, to = tmem + lanes + C::COL_O + s * D;
        const int token1 = token0 + (solo ? 0 : s) * tokens, token = token1 + row / a.G;  // of the request's
        const bool live = row < tokens * a.G && token < sp.count;
        const int pos = pos0 + token;
        const int see = live ? min(pos + 1, hi) : 0, wl = a.window > 0 ? pos - a.window + 1 : 0;
        // what every row of the stream sees
        const int all_see = min(pos0 + token1 + 1, hi) - skip;
        const int all_from = a.window > 0 ? max(sinks, pos0 + min(sp.count, token1 + tokens) - a.window - skip) : 0;
        const int mine = solo ? (n + 1 - s) / 2 : n;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < mine; ++i) {
            const int base = (first + (solo ? 2 * i + s : i)) * C::KEYS;  // the tile's place in the order of units
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
            float scale = a.scale_log2;
            // uniform; the maximum below wants scale >= 0
            const bool all = base + C::KEYS <= all_see && base >= all_from;
            if (!all || scale < 0.f) {
                // the window's keys from `begin` on, `width` of them (none: 0), and the first tokens below `firsts`
                const int begin = max(wl - skip, sinks) - base, width = max(0, see - skip - base - begin);
                if (base < sink) {
                    const int firsts = min(sink, see) - base;  // (the first tokens keep their places)
#pragma unroll
                    for (int c = 0; c < C::KEYS; ++c)
                        z[c] = (unsigned)(c - begin) < (unsigned)width || c < firsts ? z[c] * scale : -INFINITY;
                } else {
#pragma unroll
                    for (int c = 0; c < C::KEYS; ++c) z[c] = (unsigned)(c - begin) < (unsigned)width ? z[c] * scale : -INFINITY;
                }
                scale = 1.f;
            }
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < C::KEYS; c += 8)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = max3(x[j], z[c + 2 * j], z[c + 2 * j + 1]);
            float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * scale - Elem<T>::LIFT;
            if constexpr (Held<T>::LARGE < Held<T>::MOST) {
                const int tile = solo ? 2 * i + s : i;
                if (large[tile & 7] == tile) top += kLargeLift;
            }
            // O is at rest and P has been read once the last P V has completed
            auto last_done = [&] {
                return i == 0 ||
                       __all_sync(~0u, mbar_wait(&pvdone[s], (i - 1) & 1, abort_flag, a.wait_limit));
            };
            if (i == 0) {
                m = top;
            } else if (__any_sync(~0u, live && top > m + kRenew)) {
                const float next = live ? fmaxf(m, top) : m;
                // (-inf: a row that has seen nothing yet, with O and l 0)
                const float f = next == -INFINITY ? 1.f : exp2_approx(m - next);
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
            const float less = m == -INFINITY ? 0.f : -m;
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 scale2 = make_float2(scale, scale), less_m = make_float2(less, less);
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
#pragma unroll
            for (int c = C::KEYS / 64 * 32; c < C::KEYS / 2; c += 8) tmem_st32x32b<8>(ts + C::COL_P + c, p + c);
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
                        join[(c * 8 + j) * 128 + row] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
            }
            ml[row] = mine > 0 && ok ? m : -INFINITY;
            ml[128 + row] = mine > 0 && ok ? l : 0.f;
            named_bar_sync(1, 256);
        } else {
            float f0 = 1.f, f1 = 0.f, top = m;
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
            const float lse = l == 0.f ? -INFINITY : top + log2f(l);
            // Rows leave through the stream's own Q tile (its products are done): a thread holds a row, a
            // warp writes whole rows.  16-byte chunks are xor-ed with the row.
            constexpr int kCols = C::QTILE / (128 * 4), kChunk = kCols / 4;
            uint8_t* stage = smem + s * C::QTILE;
            const int r0 = row & ~31;
            const long long mine_row = live ? row_of(token, row % a.G) : -1;
            for (int c0 = 0; c0 < D; c0 += kCols) {
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    float o[32];
                    tmem_ld32x32b<32>(to + c0 + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float4 v = make_float4(o[4 * j] * f0, o[4 * j + 1] * f0, o[4 * j + 2] * f0, o[4 * j + 3] * f0);
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
                    const long long to_row = __shfl_sync(~0u, mine_row, r);
                    const float4 v = *reinterpret_cast<const float4*>(stage + (r0 + r) * (kCols * 4) +
                                                                      ((c ^ (r & (kChunk - 1))) * 16));
                    if (to_row < 0) continue;
                    if (a.splits > 1)
                        *reinterpret_cast<float4*>(a.part + (to_row * a.splits + split) * D + c0 + c * 4) = v;
                    else
                        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + to_row * D + c0 + c * 4) =
                            make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
                }
                __syncwarp();
            }
            if (live) {
                if (a.splits > 1)
                    a.part_lse[mine_row * a.splits + split] = lse;
                else if (a.lse)
                    a.lse[mine_row] = lse * 0.6931471805599453f;
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D> cudaError_t launch_t(const WindowArgs& a, cudaStream_t s) {
    using C = DenseCfg<D>;
    CUtensorMap tq, tk, tv;
    const int tokens = kRows / a.G;
    // q: 64 columns, the heads of a group, groups, tokens
    const cuuint64_t qd[4] = {(uint64_t)D, (uint64_t)a.G, (uint64_t)a.Hkv, (uint64_t)a.T};
    const cuuint64_t qs[3] = {(uint64_t)D * 2, (uint64_t)D * 2 * a.G, (uint64_t)(a.T > 1 ? a.q_stride : (long long)a.Hq * D) * 2};
    const cuuint32_t qb[4] = {64, (uint32_t)a.G, 1, (uint32_t)tokens};
    const long long rows = (long long)a.pages * a.Hkv * a.page_size;
    if (make_map<4>(&tq, a.q, qd, qs, qb) != CUDA_SUCCESS || code_map(&tk, a.k_codes, D, rows, 16) != CUDA_SUCCESS ||
        code_map(&tv, a.v_codes, D, rows, 16) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static PerDevice ready;
    const cudaError_t e = allow_smem(ready, window_dense_kernel<T, D>, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_k(window_dense_kernel<T, D>, dim3((unsigned)(a.row_tiles * a.splits * a.Hkv * a.B)), dim3(kThreads),
                    C::SMEM, s, true, tq, tk, tv, a);
}

}  // namespace

int window_dense_keys(int D) { return dense_keys(D); }

cudaError_t launch_window_dense(const WindowArgs& a, idx_dtype dt, cudaStream_t s) {
    if (dt == IDX_BF16) return a.D == 128 ? launch_t<__nv_bfloat16, 128>(a, s) : launch_t<__nv_bfloat16, 64>(a, s);
    return a.D == 128 ? launch_t<__half, 128>(a, s) : launch_t<__half, 64>(a, s);
}

}  // namespace idx
