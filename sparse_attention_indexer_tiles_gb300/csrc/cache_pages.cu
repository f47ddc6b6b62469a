// Pages of a cache: rows of a page table that take over one another's pages (fork), give pages back and
// take free ones (resize), and a pool whose live pages move together (compact).
//
// refs[p] counts the table entries that hold page p; a page is free when it is 0 (or less).  Free pages
// are taken lowest first and rows are served in their order, so that the result of a call does not
// depend on how its threads run: what is added up atomically are whole numbers, and pages are ranked by
// counting them.  A fork only counts; the copy of a page that several rows hold and that one of them is
// about to write to is made by the resize that lets it grow.
//
// resize and compact are two launches: one cluster of CTAs ranks rows and pages (its barriers are far
// cheaper than launches, and the counts of a million pages are 4 MB), then the whole GPU copies pages
// and writes the tables.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "cache_pages.cuh"
#include "serve.cuh"

namespace cg = cooperative_groups;

namespace idx {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCluster = 16;                // the most that a launch may ask for (8 are portable)
constexpr int kUnit = kCopyThreads * 16 * 4;  // bytes of a page that a block copies at a time

IDX_DEVI int warp_sum(int v) { return __reduce_add_sync(~0u, v); }
// Inclusive sum over the lanes of a warp.
IDX_DEVI int warp_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// A row's length, 0 when it is outside [0, table_stride * page_size].
IDX_DEVI bool len_ok(const PagesArgs& a, int n) { return n >= 0 && n <= a.table_stride << a.page_shift; }
IDX_DEVI int pages_of(const PagesArgs& a, int n) { return (int)(((long long)n + a.page_size - 1) >> a.page_shift); }
IDX_DEVI bool page_ok(const PagesArgs& a, int p) { return p >= 0 && p < a.pages; }

// ---------------------------------------------------------------------- fork

// The workspace of a call in place: the rows' lengths, then their pages, as they were.
IDX_DEVI int* staged_lens(const PagesArgs& a) { return a.ws; }
IDX_DEVI int* staged_table(const PagesArgs& a) { return a.ws + (a.B + 3) / 4 * 4; }

// The counts, and in place what the rows hold before any is written.
__global__ void __launch_bounds__(256) fork_stage_kernel(const __grid_constant__ PagesArgs a) {
    pdl_wait();
    const long long step = (long long)gridDim.x * 256, at = (long long)blockIdx.x * 256 + threadIdx.x;
    if (a.refs_out != a.refs)
        for (long long i = at; i < a.pages; i += step) a.refs_out[i] = a.refs[i];
    if (a.ws) {
        const int lane = threadIdx.x & 31;
        for (long long i = at >> 5; i < a.B; i += step >> 5) {
            const int n = a.lens[i];
            if (lane == 0) staged_lens(a)[i] = n;
            const int used = len_ok(a, n) ? pages_of(a, n) : 0;
            for (int j = lane; j < used; j += 32)
                staged_table(a)[i * a.table_stride + j] = a.table[i * a.table_stride + j];
        }
    }
}

// A block per row, which takes over its parent's pages.  Counts: the row's own pages gain one for each row that it is
// the parent of and lose its own entry, so a row whose only child is one row (itself or another) changes no count.  Up to
// kScanRows rows a block finds its row's children among all parents; for more, a row counts off its own pages
// and counts on its parent's (two sums for an entry: 1024 rows of 256-2048 pages 14.5 us).
constexpr int kScanRows = 4096;

template <bool SCAN> __global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ PagesArgs a) {
    __shared__ int children_of;
    pdl_wait();
    const int i = blockIdx.x;
    const int* const lens = a.ws ? staged_lens(a) : a.lens;
    const int* const table = a.ws ? staged_table(a) : a.table;
    int parent = a.arg[i], n0 = lens[i];
    bool bad = !len_ok(a, n0);
    if (bad) n0 = 0;
    if (parent < -1 || parent >= a.B) {
        bad = true;
        parent = i;
    }
    int n1 = parent < 0 ? 0 : lens[parent];
    if (!len_ok(a, n1)) n1 = 0;
    int more = 0;  // of the row's own pages
    if constexpr (SCAN) {
        if (threadIdx.x == 0) children_of = 0;
        __syncthreads();
        int n = 0;
        for (int j = threadIdx.x; j < a.B; j += 256) {
            const int p = a.arg[j];
            n += p == i || (j == i && (p < -1 || p >= a.B));
        }
        n = __reduce_add_sync(~0u, n);
        if ((threadIdx.x & 31) == 0 && n) atomicAdd(&children_of, n);
        __syncthreads();
        more = children_of - 1;
    }
    const int own = pages_of(a, n0), use = pages_of(a, n1);
    const int* const mine = table + i * a.table_stride;
    const int* const from = table + max(parent, 0) * a.table_stride;
    int* const out = a.table_out + i * a.table_stride;
#pragma unroll 4
    for (int j = threadIdx.x; j < max(own, use); j += 256) {
        const int p1 = j < use ? from[j] : -1;
        const int p0 = j < own && (!SCAN || more != 0 || parent != i) ? mine[j] : -1;
        if constexpr (SCAN) {
            if (more != 0 && page_ok(a, p0)) atomicAdd(a.refs_out + p0, more);
        } else if (p0 != p1) {
            if (page_ok(a, p0)) atomicSub(a.refs_out + p0, 1);
            if (page_ok(a, p1)) atomicAdd(a.refs_out + p1, 1);
        }
        bad |= (j < own && !page_ok(a, parent == i ? p1 : p0)) || (j < use && !page_ok(a, p1));
        if (j < use) out[j] = p1;
    }
    if (threadIdx.x == 0) a.lens_out[i] = n1;
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
}

// Both steps in one launch for few rows of few pages: a CTA, and a warp per row.  A second launch costs the host 2 us,
// one CTA the GPU some: 4 rows of 32 pages take 3.0 us instead of 4.8 (2.0 and 2.4 in a graph), 32 rows of 64 among 4096
// pages 3.4 and 4.7 (3.4 and 2.9 in a graph), 32 rows of 512 10.5 and 4.7.
constexpr int kSmallRows = 32, kSmallWidth = 64, kSmallPages = 4096;

__global__ void __launch_bounds__(1024, 1) fork_small_kernel(const __grid_constant__ PagesArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31, i = threadIdx.x >> 5;
    if (a.refs_out != a.refs)
        for (int p = threadIdx.x; p < a.pages; p += 1024) a.refs_out[p] = a.refs[p];
    const bool mine = i < a.B;
    int parent = mine ? a.arg[i] : -1, n0 = mine ? a.lens[i] : 0;
    bool bad = !len_ok(a, n0) || parent < -1 || parent >= a.B;
    if (!len_ok(a, n0)) n0 = 0;
    if (parent < -1 || parent >= a.B) parent = i;
    // a row's children, of at most 32
    const int other = lane < a.B ? a.arg[lane] : -1;
    const int more = __popc(__ballot_sync(~0u, other == i || (lane == i && lane < a.B && parent == i))) - 1;
    int n1 = parent < 0 ? 0 : a.lens[parent];
    if (!len_ok(a, n1)) n1 = 0;
    const int own = mine ? pages_of(a, n0) : 0, use = mine ? pages_of(a, n1) : 0;
    const int* const from = a.table + max(parent, 0) * a.table_stride;
    int* const out = a.table_out + i * a.table_stride;
    // what this row will hold, before any row is written (a workspace: the call is in place)
    if (a.ws)
        for (int j = lane; j < use; j += 32) staged_table(a)[i * a.table_stride + j] = from[j];
    __syncthreads();
    const int* const mine_now = a.table + i * a.table_stride;
#pragma unroll 4
    for (int j = lane; j < own; j += 32) {
        const int p = mine_now[j];
        bad |= !page_ok(a, p);
        if (more != 0 && page_ok(a, p)) atomicAdd(a.refs_out + p, more);
    }
    __syncthreads();
    const int* const taken = a.ws ? staged_table(a) + i * a.table_stride : from;
#pragma unroll 4
    for (int j = lane; j < use; j += 32) {
        const int p = taken[j];
        bad |= !page_ok(a, p);
        out[j] = p;
    }
    if (mine && lane == 0) a.lens_out[i] = n1;
    if (bad && mine) raise_status(a.d_status, IDX_DEV_RANGE);
}

// --------------------------------------------------------- ranking by a cluster

// What a CTA has counted of its pages.
struct Counts {
    int before[kWarps];  // in the warps before one
    int total;
};

// The CTAs of a ranking: kCluster of them, or one.
template <bool CLUSTER> struct Team {
    static constexpr int CTAS = CLUSTER ? kCluster : 1;
    int rank;
    IDX_DEVI Team() : rank(0) {
        if constexpr (CLUSTER) rank = (int)cg::this_cluster().block_rank();
    }
    // Everything written before is visible after (to loads past L1): the cluster's barrier releases and
    // acquires.
    IDX_DEVI void sync() const {
        if constexpr (CLUSTER)
            cg::this_cluster().sync();
        else
            __syncthreads();
    }
    // A barrier in two halves: a CTA that has arrived reads no other's shared memory any more.
    IDX_DEVI void arrive() const {
        if constexpr (CLUSTER) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    }
    IDX_DEVI void wait() const {
        if constexpr (CLUSTER) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    template <typename S> IDX_DEVI const S& of(S& mine, int r) const {
        if constexpr (CLUSTER) return *cg::this_cluster().map_shared_rank(&mine, r);
        return mine;
    }
};

// Pages [first, end) of a warp: contiguous ranges in the order of CTAs and warps, whole groups of 32.
struct Range {
    int first, end;
};
template <bool CLUSTER> IDX_DEVI Range warp_pages(const Team<CLUSTER>& team, int pages, int warp) {
    const long long groups = ((long long)pages + 31) / 32, of = Team<CLUSTER>::CTAS * kWarps;
    const long long per = (groups + of - 1) / of * 32, first = (team.rank * kWarps + warp) * per;
    return {(int)min(first, (long long)pages), (int)min(first + per, (long long)pages)};
}

constexpr int kBatch = 8;  // groups of 32 pages whose loads are in flight together

// Counts the pages of the CTA for which f holds; published by the next team.sync().
template <typename F> IDX_DEVI void count_pages(Counts& sh, Range r, int warp, int lane, F f) {
    int c = 0;
#pragma unroll 8
    for (int p = r.first + lane; p < r.end; p += 32) c += f(p);
    c = warp_sum(c);
    if (lane == 0) sh.before[warp] = c;
    __syncthreads();
    if (warp == 0) {
        const int s = sh.before[lane], i = warp_scan(s, lane);
        sh.before[lane] = i - s;
        if (lane == 31) sh.total = i;
    }
}
// What the CTAs before this one counted, and all of them.
template <bool CLUSTER> IDX_DEVI void totals(const Team<CLUSTER>& team, Counts& sh, int& before, int& all) {
    before = all = 0;
#pragma unroll
    for (int r = 0; r < Team<CLUSTER>::CTAS; ++r) {
        const int n = team.of(sh, r).total;
        if (r < team.rank) before += n;
        all += n;
    }
}

// -------------------------------------------------------------------- resize

// Workspace: per row what it asks for, then its new length as served and the rank of its first page; the rows that copy
// a page (their number first); the pages that rows take, by rank.
struct Row {
    int old_len, new_len;
    int rank;
    int from;  // the page that it copies, or -1
};
IDX_DEVI int4* row_wants(const PagesArgs& a) { return reinterpret_cast<int4*>(a.ws); }  // old, new, from
IDX_DEVI int2* row_places(const PagesArgs& a) { return reinterpret_cast<int2*>(a.ws + 4ll * a.B); }
IDX_DEVI int* copy_rows(const PagesArgs& a) { return a.ws + 6ll * a.B; }
IDX_DEVI int* taken_pages(const PagesArgs& a) { return a.ws + 7ll * a.B + 1; }
IDX_DEVI Row served_row(const PagesArgs& a, long long i) {
    const int4 want = row_wants(a)[i];
    const int2 place = row_places(a)[i];
    return {want.x, place.x, place.y, place.x > want.x ? want.z : -1};
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1) resize_rank_kernel(const __grid_constant__ PagesArgs a) {
    __shared__ Counts sh;
    __shared__ int served, copies;  // pages that rows take, rows that copy
    const Team<CLUSTER> team;
    constexpr int kAll = Team<CLUSTER>::CTAS * kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, at = team.rank * kThreads + tid;
    if (tid == 0) served = copies = 0;
    pdl_wait();
    pdl_trigger();
    const Range r = warp_pages(team, a.pages, warp);
    if (a.refs_out != a.refs) {
#pragma unroll 8
        for (int p = r.first + lane; p < r.end; p += 32) a.refs_out[p] = a.refs[p];
        team.sync();
    }
    // rows that shrink give pages back
    bool bad = false;
    for (int i = at >> 5; i < a.B; i += kAll / 32) {
        const int n0 = a.lens[i], n1 = a.arg[i];
        if (!len_ok(a, n0) || !len_ok(a, n1) || n1 >= n0) continue;
        const int* const in = a.table + i * a.table_stride;
        const int end = pages_of(a, n0);
        for (int j0 = pages_of(a, n1) + lane; j0 < end; j0 += 32 * kBatch) {
            int p[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) p[k] = j0 + 32 * k < end ? in[j0 + 32 * k] : 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (j0 + 32 * k >= end) break;
                if (page_ok(a, p[k]))
                    atomicSub(a.refs_out + p[k], 1);
                else
                    bad = true;
            }
        }
    }
    team.sync();
    // what rows that grow copy, and which pages are free
    for (int i = at; i < a.B; i += kAll) {
        Row row = {a.lens[i], a.arg[i], 0, -1};
        if (!len_ok(a, row.old_len) || !len_ok(a, row.new_len)) {
            bad = true;
            row.new_len = row.old_len;  // left as it is
        } else if (row.new_len > row.old_len && (row.old_len & (a.page_size - 1))) {
            const int p = a.table[i * a.table_stride + (row.old_len >> a.page_shift)];
            if (!page_ok(a, p))
                bad = true;
            else if (__ldcg(a.refs_out + p) > 1)
                row.from = p;
        }
        row_wants(a)[i] = make_int4(row.old_len, row.new_len, row.from, 0);
    }
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
    count_pages(sh, r, warp, lane, [&](int p) { return __ldcg(a.refs_out + p) <= 0 ? 1 : 0; });
    team.sync();
    int before, all;
    totals(team, sh, before, all);
    team.arrive();
    {
        // rows in their order, until the free pages do not suffice for one: every CTA goes through them (a barrier
        // costs more), the first writes
        __shared__ long long part[kWarps];
        __shared__ int part_copies[kWarps];
        long long taken = 0;  // by the rows before these, served or not
        int copied = 0;
        for (int i0 = 0; i0 < a.B; i0 += kThreads) {
            const int i = i0 + tid;
            Row row = {0, 0, 0, -1};
            if (i < a.B) {
                const int4 x = __ldcg(row_wants(a) + i);
                row = {x.x, x.y, 0, x.z};
            }
            const bool copy = row.from >= 0;
            const int want =
                row.new_len > row.old_len ? pages_of(a, row.new_len) - pages_of(a, row.old_len) + copy : 0;
            long long upto = want;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const long long u = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += u;
            }
            const unsigned copying = __ballot_sync(~0u, copy);
            int nth = copied + __popc(copying & ((1u << lane) - 1));
            if (lane == 31) {
                part[warp] = upto;
                part_copies[warp] = __popc(copying);
            }
            __syncthreads();
            upto += taken;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) {
                    upto += part[w];
                    nth += part_copies[w];
                }
                taken += part[w];
                copied += part_copies[w];
            }
            // (what is served of the rows that want pages comes before all that is not)
            const bool ok = want == 0 || upto <= all;
            if (i < a.B) {
                if (!ok) {
                    row.new_len = row.old_len;
                    row.from = -1;
                } else if (want > 0) {
                    row.rank = (int)(upto - want);
                    if (copy) atomicMax(&copies, nth + 1);
                    atomicMax(&served, (int)upto);
                }
                if (team.rank == 0) {
                    if (!ok) raise_status(a.d_status, IDX_DEV_PAGES);
                    if (row.from >= 0) copy_rows(a)[nth + 1] = i;
                    row_places(a)[i] = make_int2(row.new_len, row.rank);
                    a.lens_out[i] = row.new_len;
                }
            }
            __syncthreads();
        }
        if (team.rank == 0 && tid == 0) copy_rows(a)[0] = copies;
    }
    // the free pages by rank, as many as rows take
    const int most = served;
    int rank = before + sh.before[warp];
    for (int p0 = r.first; p0 < r.end && rank < most; p0 += 32 * kBatch) {
        int n[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) n[i] = p0 + i * 32 + lane < r.end ? __ldcg(a.refs_out + p0 + i * 32 + lane) : 1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const unsigned m = __ballot_sync(~0u, n[i] <= 0);
            const int k = rank + __popc(m & ((1u << lane) - 1)), p = p0 + i * 32 + lane;
            if (n[i] <= 0 && k < most) {
                taken_pages(a)[k] = p;
                a.refs_out[p] = 1;
            }
            rank += __popc(m);
        }
    }
    team.wait();
}

// Copies pages pair(k) = (from, to) for k < n, a unit of one of them per block at a time.
template <typename F> IDX_DEVI void copy_pages(const PageArrays& c, int n, F pair) {
    long long units = 0;  // of one pair
    for (int x = 0; x < c.n; ++x) units += (c.bytes[x] + kUnit - 1) / kUnit;
    for (long long u = blockIdx.x; u < n * units; u += gridDim.x) {
        const int k = (int)(u / units);
        long long at = u - k * units;
        int x = 0;
        for (; x < c.n - 1; ++x) {
            const long long of = (c.bytes[x] + kUnit - 1) / kUnit;
            if (at < of) break;
            at -= of;
        }
        const int2 p = pair(k);
        const long long bytes = c.bytes[x], first = at * kUnit + threadIdx.x * 16;
        const uint8_t* from = c.p[x] + p.x * bytes;
        uint8_t* to = c.p[x] + p.y * bytes;
        uint4 v[kUnit / (kCopyThreads * 16)];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (first + j * (kCopyThreads * 16) < bytes)
                v[j] = *reinterpret_cast<const uint4*>(from + first + j * (kCopyThreads * 16));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (first + j * (kCopyThreads * 16) < bytes)
                *reinterpret_cast<uint4*>(to + first + j * (kCopyThreads * 16)) = v[j];
    }
}

__global__ void __launch_bounds__(kCopyThreads) resize_move_kernel(const __grid_constant__ PagesArgs a) {
    pdl_wait();
    const int* const taken = taken_pages(a);
    const int lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * (kCopyThreads / 32);
    bool bad = false;
    for (long long i = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) >> 5; i < a.B; i += step) {
        const Row row = served_row(a, i);
        if (!len_ok(a, row.old_len)) continue;
        const int* in = a.table + i * a.table_stride;
        int* out = a.table_out + i * a.table_stride;
        const int had = pages_of(a, row.old_len), has = pages_of(a, row.new_len);
        const bool copy = row.from >= 0;
        const int kept = min(had - copy, has);
        // (kept entries are checked here, given back and copied ones by the ranking)
        for (int j0 = lane; j0 < kept; j0 += 32 * kBatch) {
            int p[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) p[k] = j0 + 32 * k < kept ? in[j0 + 32 * k] : 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (j0 + 32 * k >= kept) break;
                bad |= !page_ok(a, p[k]);
                if (out != in) out[j0 + 32 * k] = p[k];
            }
        }
        for (int j = kept + lane; j < has; j += 32) out[j] = taken[row.rank + j - kept];
        if (copy && lane == 0) atomicSub(a.refs_out + row.from, 1);
    }
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
    const int* const list = copy_rows(a);
    copy_pages(a.caches, list[0], [&](int k) {
        const Row row = served_row(a, list[k + 1]);
        return make_int2(row.from, taken[row.rank]);
    });
}

// ------------------------------------------------------------------- compact

// Workspace: the number of moves and of live pages; the pages to fill, by rank; the pages that move, the last one
// first; where a page from the live count on goes.
IDX_DEVI int* holes_of(const PagesArgs& a) { return a.ws + 4; }
IDX_DEVI int* movers_of(const PagesArgs& a) { return a.ws + 4 + (a.pages / 2 + 1); }
IDX_DEVI int* moved_to(const PagesArgs& a) { return a.ws + 4 + 2ll * (a.pages / 2 + 1); }

// One count of the live pages ranks both kinds: page p with l live pages before it is the (p - l)-th free one, and as
// many live pages follow it as the live count says; the page at the live count knows how many move.
template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1) compact_rank_kernel(const __grid_constant__ PagesArgs a) {
    __shared__ Counts sh;
    const Team<CLUSTER> team;
    constexpr int kAll = Team<CLUSTER>::CTAS * kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, at = team.rank * kThreads + tid;
    pdl_wait();
    pdl_trigger();
    const Range r = warp_pages(team, a.pages, warp);
    count_pages(sh, r, warp, lane, [&](int p) { return a.refs[p] > 0; });
    team.sync();
    int before, live;
    totals(team, sh, before, live);
    int rank = before + sh.before[warp];  // live pages before the warp's
    for (int p0 = r.first; p0 < r.end; p0 += 32 * kBatch) {
        int n[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) n[i] = p0 + i * 32 + lane < r.end ? a.refs[p0 + i * 32 + lane] : 0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int p = p0 + i * 32 + lane;
            const unsigned m = __ballot_sync(~0u, n[i] > 0);
            const int l = rank + __popc(m & ((1u << lane) - 1));
            rank += __popc(m);
            if (p >= r.end) continue;
            if (p == live - 1) a.ws[0] = live - (l + (n[i] > 0));  // live pages from the live count on
            if (p < live) {
                if (n[i] <= 0)
                    holes_of(a)[p - l] = p;
                else if (a.refs_out != a.refs)
                    a.refs_out[p] = n[i];
            } else if (n[i] > 0) {
                movers_of(a)[live - 1 - l] = p;
            } else {
                moved_to(a)[p] = p;
                a.refs_out[p] = 0;
            }
        }
    }
    team.sync();
    const int moves = live > 0 ? __ldcg(a.ws) : 0;
    for (int k = at; k < moves; k += kAll) {
        const int to = __ldcg(holes_of(a) + k), from = __ldcg(movers_of(a) + moves - 1 - k);
        moved_to(a)[from] = to;
        const int n = a.refs[from];
        a.refs_out[to] = n;
        a.refs_out[from] = 0;
    }
    if (at == 0) {
        a.ws[1] = live;
        *a.live = live;
    }
}

__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const __grid_constant__ PagesArgs a) {
    pdl_wait();
    const int live = a.ws[1], moves = live > 0 ? a.ws[0] : 0;
    const int lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * (kCopyThreads / 32);
    bool bad = false;
    for (long long i = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) >> 5; i < a.B; i += step) {
        const int n = a.lens[i];
        if (!len_ok(a, n)) {
            bad = true;
            continue;
        }
        const int* in = a.table + i * a.table_stride;
        int* out = a.table_out + i * a.table_stride;
        for (int j = lane; j < pages_of(a, n); j += 32) {
            const int p = in[j];
            if (!page_ok(a, p)) bad = true;
            const int to = page_ok(a, p) && p >= live ? moved_to(a)[p] : p;
            if (out != in || to != p) out[j] = to;
        }
    }
    if (bad) raise_status(a.d_status, IDX_DEV_RANGE);
    copy_pages(a.caches, moves, [&](int k) { return make_int2(movers_of(a)[moves - 1 - k], holes_of(a)[k]); });
}

// A ranking kernel: a cluster when its pages or rows are many (see kClusterFrom), one CTA otherwise.
constexpr int kClusterFrom = 4096;

// The devices that place a cluster of kCluster CTAs of a kernel: more than the portable eight, so a part of a GPU may
// not.
class ClusterDevices {
    PerDevice asked_;
    std::atomic<uint64_t> without_{0};

public:
    cudaError_t place(void (*kernel)(PagesArgs), bool* yes) {
        int device = -1, clusters = 1;
        const cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        asked_.run(device, [&] {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kCluster);
            cfg.blockDim = dim3(kThreads);
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = kCluster;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
                cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                clusters = 0;
            }
            if (clusters < 1 && device < 64) without_.fetch_or(1ull << device);
            return 0;
        });
        *yes = clusters > 0 && !(device < 64 && without_.load() >> device & 1);
        return cudaSuccess;
    }
};

cudaError_t launch_rank(void (*one)(PagesArgs), void (*many)(PagesArgs), ClusterDevices& devices, const PagesArgs& a,
                        cudaStream_t s) {
    bool cluster = !a.one_cta && (a.pages >= kClusterFrom || a.B * 16ll >= kClusterFrom);
    if (cluster) {
        const cudaError_t e = devices.place(many, &cluster);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster ? kCluster : 1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, cluster ? many : one, a);
}

// Blocks of a moving kernel: what is to be copied is known on the device only; a few waves.
unsigned move_blocks(int sm_count) { return (unsigned)sm_count * 8; }

}  // namespace

size_t fork_workspace_ints(int B, long long table_stride) {
    return (size_t)(B + 3) / 4 * 4 + (size_t)B * (size_t)table_stride;
}
size_t resize_workspace_ints(int B, int pages, long long table_stride) {
    return 7 * (size_t)B + 1 + (size_t)std::min<long long>(pages, (long long)B * (table_stride + 1));
}
size_t compact_workspace_ints(int, int pages) { return 4 + 2 * (size_t)(pages / 2 + 1) + (size_t)pages; }

cudaError_t launch_fork(const PagesArgs& a, int sm_count, cudaStream_t s, int* launched) {
    cudaError_t e = cudaSuccess;
    if (a.B > 0 && a.B <= kSmallRows && a.table_stride <= kSmallWidth && a.pages <= kSmallPages) {
        e = launch_k(fork_small_kernel, dim3(1), dim3(1024), 0, s, true, a);
        if (e == cudaSuccess) ++*launched;
        return e;
    }
    if (a.ws || a.refs_out != a.refs) {
        const long long work = std::max<long long>(a.pages, a.ws ? a.B * 32ll : 0);
        const long long blocks = std::min<long long>((work + 255) / 256, sm_count * 8ll);
        e = launch_k(fork_stage_kernel, dim3((unsigned)std::max<long long>(blocks, 1)), dim3(256), 0, s, true, a);
        if (e != cudaSuccess) return e;
        ++*launched;
    }
    if (a.B == 0) return e;
    e = launch_k(a.B <= kScanRows ? fork_kernel<true> : fork_kernel<false>, dim3((unsigned)a.B), dim3(256), 0, s, true, a);
    if (e == cudaSuccess) ++*launched;
    return e;
}

cudaError_t launch_resize(const PagesArgs& a, int sm_count, cudaStream_t s, int* launched) {
    static ClusterDevices devices;
    cudaError_t e = launch_rank(resize_rank_kernel<false>, resize_rank_kernel<true>, devices, a, s);
    if (e != cudaSuccess) return e;
    ++*launched;
    e = launch_k(resize_move_kernel, dim3(move_blocks(sm_count)), dim3(kCopyThreads), 0, s, true, a);
    if (e == cudaSuccess) ++*launched;
    return e;
}

cudaError_t launch_compact(const PagesArgs& a, int sm_count, cudaStream_t s, int* launched) {
    static ClusterDevices devices;
    cudaError_t e = launch_rank(compact_rank_kernel<false>, compact_rank_kernel<true>, devices, a, s);
    if (e != cudaSuccess) return e;
    ++*launched;
    e = launch_k(compact_move_kernel, dim3(move_blocks(sm_count)), dim3(kCopyThreads), 0, s, true, a);
    if (e == cudaSuccess) ++*launched;
    return e;
}

}  // namespace idx
