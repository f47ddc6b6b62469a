// Eviction from a paged K/V cache by accumulated attention weight.
//
// For each (request, head) with n cached slots the `budget` best stay: protected
// slots first (position < sink, or position >= next_pos - recent), then by weight,
// ties to the lower slot.  Attention does not depend on the order of the keys, so
// the kept slots below the budget stay where they are and only the holes among
// them are filled: the i-th hole takes the i-th kept slot from the budget on, both
// ascending.  That moves the fewest rows (one when a request is one token over its
// budget), and sources and destinations are disjoint, so the moves have no order.
//
// Selection: slots are ranked by a 32-bit key whose unsigned order is the weights'
// order (protected slots hold the largest key).  One pass reads weights and positions,
// leaves the keys in shared memory and finds their range; then a histogram over the range
// (1024 bins, for short rows 512) finds the bin that holds the rank, which is the next
// range.  The bits of a float grow with its logarithm, so heavy-tailed weights spread over
// the bins, and a bin is usually decided (all of it stays) after two.  Few long rows take a cluster
// of CTAs each, every CTA with a slice of the row and the histograms summed through
// distributed shared memory.  The moves are a second launch, so that they spread over the
// whole GPU whichever rows they belong to.  HBM-bound: 8 bytes per slot read, 8 per kept
// slot written, and the moved rows.
#include <cooperative_groups.h>

#include <cmath>

#include "evict.cuh"
#include "serve.cuh"

namespace cg = cooperative_groups;

namespace idx {

namespace {

constexpr int kBinsPerThread = 2;
constexpr int kMaxCluster = 8;           // the portable limit
constexpr int kSliceMax = 48 * 1024;     // keys a CTA keeps in shared memory
constexpr uint32_t kProtected = 0xffffffffu;

// Rank key of a slot.  A NaN weight of either sign counts as -inf (fmaxf gives the other operand), so
// unprotected keys end at that of infinity, below kProtected.
IDX_DEVI uint32_t slot_key(float w, int pos, int sink, int recent_from) {
    return (pos < sink || pos >= recent_from) ? kProtected : fkey(fmaxf(w, -INFINITY));
}

// Row of slot j in the caches; 0xffffffff when its page is not one.
IDX_DEVI uint32_t cache_row(const EvictArgs& a, int b, int h, int j) {
    const int page = a.table[b * a.table_stride + (j >> a.page_shift)];
    if (page < 0 || page >= a.pages) return 0xffffffffu;
    return ((uint32_t)page * a.Hkv + h) * a.page_size + (j & (a.page_size - 1));
}

// What a CTA tells its cluster.
template <int kThreads> struct alignas(16) Shared {
    static constexpr int kWarps = kThreads / 32, kBins = kThreads * kBinsPerThread;
    uint32_t hist[2][kBins];
    uint4 range;             // of this CTA's unprotected keys (x .. y), and its protected slots (z)
    int4 cnt;                // its slots: above the cut and equal to it, below / from the budget on
    // the CTA's own
    uint32_t warp_sum[kWarps];
    int warp_cnt[kWarps][4];
    int warp_eq[kWarps], warp_hole[kWarps], warp_src[kWarps];  // before a warp's range
    uint32_t bin, above, in_bin;
};

// Inclusive sum over the lanes of a warp.
IDX_DEVI int warp_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// One contiguous range of slots: what stays of it above the cut and equal to it, below the
// budget (c[0], c[2]) and from it on (c[1], c[3]); `nlow` of its slots are below the budget
// and `eq` slots before it equal the cut, of which the first `ties` stay.
struct Range {
    int holes, srcs;
};
IDX_DEVI Range fill(const int (&c)[4], int nlow, int eq, int ties) {
    return {nlow - c[0] - min(max(ties - eq, 0), c[2]),
            c[1] + min(max(ties - eq - c[2], 0), c[3])};
}

// One request and head per cluster.  STAGED: the slice's keys are in shared memory;
// otherwise (slices above kSliceMax) they are made again from the arrays in every pass.
template <bool CLUSTER, bool STAGED, int kThreads>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a, int C) {
    using S = Shared<kThreads>;
    constexpr int kWarps = S::kWarps, kBins = S::kBins;
    constexpr int kBinBits = kThreads == 256 ? 9 : 10;
    static_assert(kBins == 1 << kBinBits, "");
    __shared__ S sh;
    extern __shared__ uint32_t keys[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CLUSTER ? (int)cg::this_cluster().block_rank() : 0;
    const int bh = (int)blockIdx.x / C, h = bh % a.Hkv, b = bh / a.Hkv;
    auto sync_all = [&] {
        if constexpr (CLUSTER)
            cg::this_cluster().sync();
        else
            __syncthreads();
    };
    auto of = [&](int r) -> const S& {
        if constexpr (CLUSTER) return *cg::this_cluster().map_shared_rank(&sh, r);
        return sh;
    };
    pdl_wait();  // launched while the kernel before it ends: 512 rows of 2049 13.9 -> 11.2 us a call
    int n = a.lens[b];
    const bool bad = n < 0 || n > a.max_len;
    n = min(max(n, 0), a.max_len);
    const int keep = min(n, a.budget);
    if (rank == 0 && tid == 0) {
        if (h == 0) a.lens_out[b] = keep;
        if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
        if (n <= a.budget && a.max_moves > 0) a.counts[bh] = 0;
    }
    const long long base = (long long)bh * a.slots;
    const float* w = a.w + base;
    const int* pos = a.pos + base;
    float* w_out = a.w_out + base;
    int* pos_out = a.pos_out + base;
    const bool copy_w = a.w_out != a.w, copy_pos = a.pos_out != a.pos;
    // this CTA's slots: whole groups of 32
    const int groups = (n + 31) / 32, per_cta = (groups + C - 1) / C;
    const int first = min(rank * per_cta * 32, n), end = min(first + per_cta * 32, n);
    if (n <= a.budget) {  // the same for the whole cluster
        for (int j = first + tid; j < end; j += kThreads) {
            if (copy_w) w_out[j] = w[j];
            if (copy_pos) pos_out[j] = pos[j];
        }
        return;
    }
    const int recent_from = a.next_pos[b] - a.recent;
    auto key_of = [&](int j) {
        return STAGED ? keys[j - first] : slot_key(w[j], pos[j], a.sink, recent_from);
    };

    // Keys, their range and the protected slots; what lies below the budget is copied on the
    // way (the holes among it are written by the moves).
    if (tid == 0) sh.range = make_uint4(0xffffffffu, 0u, 0u, 0u);
    for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = sh.hist[1][i] = 0u;
    __syncthreads();
    uint32_t lo = 0xffffffffu, hi = 0u;
    int guarded = 0;
    constexpr int kLoads = 8;
    for (int j0 = first + tid; j0 < end; j0 += kLoads * kThreads) {
        float wv[kLoads];
        int pv[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int j = j0 + u * kThreads;
            wv[u] = j < end ? w[j] : 0.f;
            pv[u] = j < end ? pos[j] : 0;
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int j = j0 + u * kThreads;
            if (j >= end) break;
            const uint32_t k = slot_key(wv[u], pv[u], a.sink, recent_from);
            if constexpr (STAGED) keys[j - first] = k;
            if (k == kProtected) {
                ++guarded;
            } else {
                lo = min(lo, k);
                hi = max(hi, k);
            }
            if (j < keep) {
                if (copy_w) w_out[j] = wv[u];
                if (copy_pos) pos_out[j] = pv[u];
            }
        }
    }
    lo = __reduce_min_sync(~0u, lo);
    hi = __reduce_max_sync(~0u, hi);
    guarded = __reduce_add_sync(~0u, guarded);
    if (lane == 0) {
        atomicMin(&sh.range.x, lo);
        atomicMax(&sh.range.y, hi);
        atomicAdd(&sh.range.z, (uint32_t)guarded);
    }
    sync_all();
    {
        const uint4 r = of(lane < C ? lane : 0).range;
        lo = __reduce_min_sync(~0u, r.x);
        hi = __reduce_max_sync(~0u, r.y);
        guarded = (int)__reduce_add_sync(~0u, lane < C ? r.z : 0u);
    }

    // keys above `cut` stay, and the first `ties` slots that equal it
    uint32_t cut;
    int ties;
    if (guarded >= a.budget) {
        cut = kProtected;
        ties = a.budget;
    } else {
        uint32_t want = (uint32_t)(a.budget - guarded);  // >= 1; n > budget: the range holds more
        for (int pass = 0;; ++pass) {
            const uint32_t span = hi - lo;
            const int shift = span < kBins ? 0 : 32 - __clz(span) - kBinBits;  // span >> shift < kBins
            uint32_t* hist = sh.hist[pass & 1];
#pragma unroll 4
            for (int j = first + tid; j < end; j += kThreads) {
                const uint32_t d = key_of(j) - lo;
                if (d <= span) atomicAdd(&hist[d >> shift], 1u);
            }
            sync_all();
            // counts from the top: thread t has the two bins below kBins - 2 t
            const int low_bin = kBins - kBinsPerThread * (tid + 1);
            uint32_t c[kBinsPerThread] = {0u, 0u};
            {
                uint2 v[CLUSTER ? kMaxCluster : 1];
#pragma unroll
                for (int r = 0; r < (CLUSTER ? kMaxCluster : 1); ++r)
                    v[r] = r < C ? *reinterpret_cast<const uint2*>(&of(r).hist[pass & 1][low_bin])
                                 : make_uint2(0u, 0u);
#pragma unroll
                for (int r = 0; r < (CLUSTER ? kMaxCluster : 1); ++r) {
                    c[0] += v[r].y;
                    c[1] += v[r].x;
                }
            }
            const uint32_t sum = c[0] + c[1];
            // (the other buffer has been read by nobody since the last sync_all)
            *reinterpret_cast<uint2*>(&sh.hist[(pass & 1) ^ 1][low_bin]) = make_uint2(0u, 0u);
            const uint32_t run = (uint32_t)warp_scan((int)sum, lane);
            if (lane == 31) sh.warp_sum[warp] = run;
            __syncthreads();
            uint32_t above = run - sum;
            for (int i = 0; i < warp; ++i) above += sh.warp_sum[i];
            if (above < want && want <= above + sum) {
#pragma unroll
                for (int i = 0; i < kBinsPerThread; ++i) {
                    if (above < want && want <= above + c[i]) {
                        sh.bin = low_bin + kBinsPerThread - 1 - i;
                        sh.above = above;
                        sh.in_bin = c[i];
                    }
                    above += c[i];
                }
            }
            __syncthreads();
            lo += sh.bin << shift;
            hi = hi - lo < (1u << shift) ? hi : lo + ((1u << shift) - 1u);
            want -= sh.above;
            if (shift == 0) {
                cut = lo;
                ties = (int)want;
                break;
            }
            if (want == sh.in_bin && lo > 0u) {  // the whole bin stays
                cut = lo - 1u;
                ties = 0;
                break;
            }
        }
    }

    // each warp owns a contiguous range of 32-slot groups: what it keeps, below the budget
    // and from it on
    const int mine = (end - first + 31) / 32, per = (mine + kWarps - 1) / kWarps;
    const int g0 = min(warp * per, mine), g1 = min(g0 + per, mine);
    {
        int cnt[4] = {0, 0, 0, 0};
        const int begin = first + g0 * 32, stop = min(first + g1 * 32, end);
        auto count = [&](int from, int to, int& gt, int& eq) {
#pragma unroll 4
            for (int j = from + lane; j < to; j += 32) {
                const uint32_t k = key_of(j);
                gt += k > cut;
                eq += k == cut;
            }
        };
        count(begin, min(stop, keep), cnt[0], cnt[2]);
        count(max(begin, keep), stop, cnt[1], cnt[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = __reduce_add_sync(~0u, cnt[i]);
            if (lane == 0) sh.warp_cnt[warp][i] = v;
        }
    }
    __syncthreads();
    if (tid < 4) {
        int v = 0;
        for (int i = 0; i < kWarps; ++i) v += sh.warp_cnt[i][tid];
        reinterpret_cast<int*>(&sh.cnt)[tid] = v;
    }
    sync_all();
    if (warp == 0) {
        // a lane per CTA of the cluster, then a lane per warp of this one
        int c[4] = {0, 0, 0, 0};
        auto before = [&](int lo_slot, int hi_slot, int eq0, int& eq, Range& r) {
            const int both = c[2] + c[3];
            eq = eq0 + warp_scan(both, lane) - both;
            r = fill(c, max(0, min(hi_slot, keep) - lo_slot), eq, ties);
        };
        int eq;
        Range r;
        if (lane < C) {
            const int4 v = of(lane).cnt;
            c[0] = v.x;
            c[1] = v.y;
            c[2] = v.z;
            c[3] = v.w;
        }
        int lo_slot = min(lane * per_cta * 32, n);
        before(lo_slot, lane < C ? min(lo_slot + per_cta * 32, n) : lo_slot, 0, eq, r);
        const int holes = warp_scan(r.holes, lane), srcs = warp_scan(r.srcs, lane);
        if (rank == 0 && lane == 31) a.counts[bh] = holes;
        const int eq0 = __shfl_sync(~0u, eq, rank);
        const int hole0 = __shfl_sync(~0u, holes - r.holes, rank);
        const int src0 = __shfl_sync(~0u, srcs - r.srcs, rank);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = lane < kWarps ? sh.warp_cnt[lane % kWarps][i] : 0;
        lo_slot = first + min(lane * per, mine) * 32;
        before(lo_slot, lane < kWarps ? min(first + min((lane + 1) * per, mine) * 32, end) : lo_slot,
               eq0, eq, r);
        const int hole = hole0 + warp_scan(r.holes, lane) - r.holes;
        const int src = src0 + warp_scan(r.srcs, lane) - r.srcs;
        if (lane < kWarps) {
            sh.warp_eq[lane] = eq;
            sh.warp_hole[lane] = hole;
            sh.warp_src[lane] = src;
        }
    }
    sync_all();  // (also: no CTA ends while another reads its counts)
    int eq = sh.warp_eq[warp], hole = sh.warp_hole[warp], from = sh.warp_src[warp];
    int* dst = a.moves + (long long)bh * 2 * a.max_moves;
    int* src = dst + a.max_moves;
    const uint32_t lt = (1u << lane) - 1u;
    constexpr int kAhead = 4;  // groups whose keys are read and voted on together
    for (int g = g0; g < g1; g += kAhead) {
        uint32_t mgt[kAhead], meq[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int j = first + (g + u) * 32 + lane;
            const bool in = g + u < g1 && j < end;
            const uint32_t k = in ? key_of(j) : 0u;
            mgt[u] = __ballot_sync(~0u, in && k > cut);
            meq[u] = __ballot_sync(~0u, in && k == cut);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (g + u >= g1) break;
            const int j0 = first + (g + u) * 32;
            uint32_t stays = mgt[u];
            if (meq[u]) {
                const uint32_t tie = __ballot_sync(~0u, (meq[u] >> lane & 1u) &&
                                                            eq + __popc(meq[u] & lt) < ties);
                stays |= tie;
                eq += __popc(meq[u]);
            }
            // holes are the slots below `keep` that go, sources those from it on that stay
            // (`keep` is the budget here, so every slot below it exists)
            const int low = min(max(keep - j0, 0), 32);
            const uint32_t below = low < 32 ? (1u << low) - 1u : ~0u;
            const uint32_t holes = below & ~stays, srcs = stays & ~below;
            if (holes >> lane & 1u) dst[hole + __popc(holes & lt)] = j0 + lane;
            if (srcs >> lane & 1u) src[from + __popc(srcs & lt)] = j0 + lane;
            hole += __popc(holes);
            from += __popc(srcs);
        }
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMovesPerWarp = 16;

// The moves: a warp takes kMovesPerWarp of one request and head.  A lane looks up one
// move's rows, then the warp copies, K and V rows side by side, four units of 16 bytes
// per lane at a time.  Sources and destinations are disjoint.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a) {
    pdl_wait();  // (no pdl_trigger: the next call's selection on these SMs cost 1 to 6 us)
    const int lane = threadIdx.x & 31;
    const int per_row = (a.max_moves + kMovesPerWarp - 1) / kMovesPerWarp;
    const long long u = (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5);
    const long long bh = u / per_row;
    if (bh >= (long long)a.B * a.Hkv) return;
    const int m0 = (int)(u - bh * per_row) * kMovesPerWarp;
    const int have = min(kMovesPerWarp, a.counts[bh] - m0);
    if (have <= 0) return;
    const int h = (int)(bh % a.Hkv), b = (int)(bh / a.Hkv);
    uint32_t to = 0xffffffffu, fr = 0xffffffffu;
    if (lane < have) {
        const int* dst = a.moves + bh * 2 * a.max_moves + m0;
        const int d = dst[lane], s = dst[a.max_moves + lane];
        to = cache_row(a, b, h, d);
        fr = cache_row(a, b, h, s);
        a.w_out[bh * a.slots + d] = a.w[bh * a.slots + s];
        a.pos_out[bh * a.slots + d] = a.pos[bh * a.slots + s];
        if (to == 0xffffffffu || fr == 0xffffffffu) raise_status(a.d_status, IDX_DEV_RANGE);
    }
    const int row16 = a.row_bytes / 16, lanes = 2 * row16;  // 16 or 32 lanes per move
    const int sub = lane / lanes, unit = lane % lanes, step = 32 / lanes;
    uint4* cache = reinterpret_cast<uint4*>(unit < row16 ? a.k : a.v);
    const int at = unit < row16 ? unit : unit - row16;
    constexpr int kDeep = 4;
    for (int i = 0; i < have; i += kDeep * step) {
        uint4 v[kDeep];
        uint32_t r[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int x = i + k * step + sub;
            const uint32_t f = __shfl_sync(~0u, fr, x & 31);
            r[k] = __shfl_sync(~0u, to, x & 31);
            if (x >= have || f == 0xffffffffu) r[k] = 0xffffffffu;
            if (r[k] != 0xffffffffu) v[k] = cache[(unsigned long long)f * row16 + at];
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (r[k] != 0xffffffffu) cache[(unsigned long long)r[k] * row16 + at] = v[k];
    }
}

template <bool CLUSTER, bool STAGED, int kThreads>
cudaError_t launch_select(const EvictArgs& a, int C, size_t smem, cudaStream_t s) {
    const auto kern = evict_select_kernel<CLUSTER, STAGED, kThreads>;
    static PerDevice ready;
    const cudaError_t e = allow_smem(ready, kern, kSliceMax * sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, C);
}

template <int kThreads>
cudaError_t launch_threads(const EvictArgs& a, int C, int slice, cudaStream_t s) {
    const size_t smem = (size_t)slice * sizeof(uint32_t);
    return C > 1 ? launch_select<true, true, kThreads>(a, C, smem, s)
                 : launch_select<false, true, kThreads>(a, 1, smem, s);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, int sm_count, cudaStream_t s, int* launched) {
    // CTAs per row: more than one when the row's keys do not fit one CTA's shared memory, or
    // when the rows leave half of the SMs idle and every slice keeps over 4096 keys
    // (32 rows x 65536 to 2048, the whole call: 35.5 us with four CTAs each, 46.7 with the two
    // that the keys need, 42.5 with eight).
    const long long rows = (long long)a.B * a.Hkv;
    int C = 1;
    while (C < kMaxCluster && (a.max_len > C * kSliceMax ||
                               (rows * C * 2 <= sm_count && a.max_len > C * 4096)))
        C *= 2;
    const int slice = ((a.max_len + 31) / 32 + C - 1) / C * 32;
    // Threads: the scans cost the same whatever the slice, so short slices take few threads.
    cudaError_t e;
    if (slice > kSliceMax)
        e = launch_select<true, false, 512>(a, C, 0, s);
    else if (slice > 4096)
        e = launch_threads<512>(a, C, slice, s);
    else
        e = launch_threads<256>(a, C, slice, s);
    if (e != cudaSuccess) return e;
    ++*launched;
    if (a.max_moves == 0) return e;
    const long long warps = rows * ((a.max_moves + kMovesPerWarp - 1) / kMovesPerWarp);
    const long long blocks = (warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    e = launch_k(evict_move_kernel, dim3((unsigned)blocks), dim3(kMoveThreads), 0, s, true, a);
    if (e == cudaSuccess) ++*launched;
    return e;
}

}  // namespace idx
