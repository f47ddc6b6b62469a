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
// order (protected slots hold the largest key), and the key of rank `budget` is
// found digit by digit from histograms.  HBM-bound: 8 bytes per slot read, 8 per
// kept slot written, and the moved rows.
#include "common.cuh"
#include "evict.cuh"

namespace idx {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Rank key of a slot: 0xffffffff when protected; an unprotected weight stays below it.
IDX_DEVI uint32_t slot_key(float w, int pos, int sink, int recent_from) {
    const uint32_t k = fkey(w);
    return (pos < sink || pos >= recent_from) ? 0xffffffffu : (k == 0xffffffffu ? k - 1u : k);
}

// Row of slot j, in bytes from the cache's start; -1 when its page is not one.
IDX_DEVI long long row_offset(const EvictArgs& a, int b, int h, int j) {
    const int page = a.table[b * a.table_stride + (j >> a.page_shift)];
    if (page < 0 || page >= a.pages) return -1;
    return (((long long)page * a.Hkv + h) * a.page_size + (j & (a.page_size - 1))) * a.row_bytes;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(EvictArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_want;
    __shared__ int s_cnt[kWarps][4];
    __shared__ int s_hole[kWarps + 1], s_src[kWarps + 1], s_eq[kWarps + 1];
    const int h = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n = a.lens[b];
    bool bad = n < 0 || n > a.max_len;
    n = min(max(n, 0), a.max_len);
    const int keep = min(n, a.budget);
    if (h == 0 && tid == 0) {
        a.lens_out[b] = keep;
        if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
    }
    const long long base = (long long)blockIdx.x * a.slots;
    const float* w = a.w + base;
    const int* pos = a.pos + base;
    float* w_out = a.w_out + base;
    int* pos_out = a.pos_out + base;
    if (n <= a.budget) {
        if (a.w_out != a.w)
            for (int j = tid; j < n; j += kThreads) w_out[j] = w[j];
        if (a.pos_out != a.pos)
            for (int j = tid; j < n; j += kThreads) pos_out[j] = pos[j];
        return;
    }
    const int recent_from = a.next_pos[b] - a.recent;

    // the key of rank `budget` (largest first), 8 bits at a time
    uint32_t prefix = 0, want = (uint32_t)a.budget;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
        for (int j = tid; j < n; j += kThreads) {
            const uint32_t k = slot_key(w[j], pos[j], a.sink, recent_from);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds bins 255 - 8l .. 248 - 8l, so a scan over lanes counts from the top
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
            uint32_t run = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t v = __shfl_up_sync(~0u, run, o);
                if (lane >= o) run += v;
            }
            uint32_t above = run - sum;
            if (above < want && want <= run) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (above < want && want <= above + c[i]) {
                        s_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
                        s_want = want - above;
                    }
                    above += c[i];
                }
            }
        }
        __syncthreads();
        prefix = s_prefix;
        want = s_want;
    }
    const uint32_t cut = prefix;  // keys above stay, and the first `want` slots that equal it
    const int ties = (int)want;

    // each warp owns a contiguous range of whole 32-slot groups
    const int groups = (n + 31) / 32, per = (groups + kWarps - 1) / kWarps;
    const int g0 = min(warp * per, groups), g1 = min(g0 + per, groups);
    int gt[2] = {0, 0}, eq[2] = {0, 0};  // below / from the budget on
    for (int g = g0; g < g1; ++g) {
        const int j = g * 32 + lane;
        const uint32_t k = j < n ? slot_key(w[j], pos[j], a.sink, recent_from) : 0u;
        const bool is_gt = j < n && k > cut, is_eq = j < n && k == cut, low = j < keep;
        gt[0] += __popc(__ballot_sync(~0u, is_gt && low));
        gt[1] += __popc(__ballot_sync(~0u, is_gt && !low));
        eq[0] += __popc(__ballot_sync(~0u, is_eq && low));
        eq[1] += __popc(__ballot_sync(~0u, is_eq && !low));
    }
    if (lane == 0) {
        s_cnt[warp][0] = gt[0];
        s_cnt[warp][1] = gt[1];
        s_cnt[warp][2] = eq[0];
        s_cnt[warp][3] = eq[1];
    }
    __syncthreads();
    if (tid == 0) {
        int e = 0, holes = 0, srcs = 0;
        for (int i = 0; i < kWarps; ++i) {
            const int lo = min(i * per, groups) * 32, hi = min(min((i + 1) * per, groups) * 32, n);
            const int nlow = max(0, min(hi, keep) - lo);
            s_eq[i] = e;
            s_hole[i] = holes;
            s_src[i] = srcs;
            holes += nlow - s_cnt[i][0] - min(max(ties - e, 0), s_cnt[i][2]);
            srcs += s_cnt[i][1] + min(max(ties - e - s_cnt[i][2], 0), s_cnt[i][3]);
            e += s_cnt[i][2] + s_cnt[i][3];
        }
        s_hole[kWarps] = holes;
    }
    __syncthreads();
    int* dst = a.moves + (long long)blockIdx.x * 2 * a.max_moves;
    int* src = dst + a.max_moves;
    int e = s_eq[warp], hole = s_hole[warp], from = s_src[warp];
    const uint32_t lt = (1u << lane) - 1u;
    for (int g = g0; g < g1; ++g) {
        const int j = g * 32 + lane;
        const float wj = j < n ? w[j] : 0.f;
        const int pj = j < n ? pos[j] : 0;
        const uint32_t k = j < n ? slot_key(wj, pj, a.sink, recent_from) : 0u;
        const uint32_t meq = __ballot_sync(~0u, j < n && k == cut);
        const bool stays = j < n && (k > cut || (k == cut && e + __popc(meq & lt) < ties));
        e += __popc(meq);
        const uint32_t mh = __ballot_sync(~0u, j < keep && !stays);
        const uint32_t ms = __ballot_sync(~0u, j >= keep && stays);
        if (j < keep && !stays) dst[hole + __popc(mh & lt)] = j;
        if (j >= keep && stays) src[from + __popc(ms & lt)] = j;
        hole += __popc(mh);
        from += __popc(ms);
        if (j < keep && stays) {
            if (a.w_out != a.w) w_out[j] = wj;
            if (a.pos_out != a.pos) pos_out[j] = pj;
        }
    }
    __syncthreads();  // the lists, and every read of w and pos above, before the moves
    const int moves = s_hole[kWarps];
    const int chunks = a.row_bytes / 16;  // per row of K and of V
    for (int i = warp; i < moves; i += kWarps) {
        const int d = dst[i], s = src[i];
        const long long od = row_offset(a, b, h, d), os = row_offset(a, b, h, s);
        if (lane == 0) {
            w_out[d] = w[s];
            pos_out[d] = pos[s];
        }
        if (od < 0 || os < 0) {
            bad = true;
            continue;
        }
        for (int c = lane; c < 2 * chunks; c += 32) {
            uint8_t* cache = c < chunks ? a.k : a.v;
            const int at = (c < chunks ? c : c - chunks) * 16;
            *reinterpret_cast<uint4*>(cache + od + at) =
                *reinterpret_cast<const uint4*>(cache + os + at);
        }
    }
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, int sm_count, cudaStream_t s) {
    (void)sm_count;
    evict_kernel<<<a.B * a.Hkv, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace idx
