// kv_pages.cu -- pages of a paged cache given out, shared, copied before they are written, and
// moved together.
//
// refs[p] counts the table entries in use (column c of a unit with n rows: c < ceil(n / page_size))
// that name page p; a page with no references is free.  That array is all the state there is: free
// pages are found by a scan of it, lowest first, so what a call does follows from the cache alone.
//
// A plan (pages for a step's tokens, or which pages move where) is scans of a few KB to a few MB
// and chains of dependent loads, bound by latency: one cluster of 8 blocks, whose counts meet in
// distributed shared memory, does it in one launch.  The pages themselves are then copied by all
// SMs, bound by HBM.
//
// Measured (us, cold caches): 8 hypotheses of 256 units and 59000 pages fork 6, plan 13, enter and
// copy up to 2048 pages of 32 KB 19; a compaction of 1.3 GB plans in 14.7 and moves at 6.3 TB/s, 93% of
// what a copy reaches.
#include <algorithm>

#include <cooperative_groups.h>

#include "kv_compact.cuh"
#include "kv_paged_attend.cuh"
#include "kv_pages.cuh"

namespace kvevict {
namespace {
namespace cg = cooperative_groups;

__device__ __forceinline__ int pages_of(const DevPaged &C, int rows) {
    return (int)(((long long)rows + C.ps - 1) >> C.ps_log2);
}
__device__ __forceinline__ bool page_ok(const DevPaged &C, int page) {
    return page >= 0 && page < C.num_pages;
}
__device__ __forceinline__ int32_t *table_of(const DevPaged &C, long long u) {
    return const_cast<int32_t *>(C.table) + u * C.max_pages;
}

// Sums of counts over the threads of kCtas blocks (a cluster), in rank and thread order: each thread
// gets what lies before its own, and the total.  The blocks leave together (leave_cluster).
template <int N>
struct ClusterScan {
    int before[N], total[N];
};
template <int kCtas, int N>
__device__ __forceinline__ ClusterScan<N> cluster_scan(const int (&mine)[N]) {
    __shared__ int s_warp[N][kPlanThreads / 32], s_block[N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ClusterScan<N> r;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int x = mine[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_warp[k][warp] = x;
        r.before[k] = x - mine[k];
    }
    __syncthreads();
    if (warp < N) {
        const int t = s_warp[warp][lane];
        int x = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        s_warp[warp][lane] = x - t;
        if (lane == 31) s_block[warp] = x;
    }
    if constexpr (kCtas == 1) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            r.before[k] += s_warp[k][warp];
            r.total[k] = s_block[k];
        }
    } else {
        cg::cluster_group cl = cg::this_cluster();
        const int rank = (int)cl.block_rank();
        cl.sync();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            int base = 0, all = 0;
#pragma unroll
            for (int b = 0; b < kCtas; ++b) {
                const int x = cl.map_shared_rank(s_block, b)[k];
                if (b < rank) base += x;
                all += x;
            }
            r.before[k] += base + s_warp[k][warp];
            r.total[k] = all;
        }
    }
    return r;
}
// No block leaves while another reads its sums.
template <int kCtas>
__device__ __forceinline__ void leave_cluster() {
    if constexpr (kCtas > 1) cg::this_cluster().sync();
}

// A warp's share of the pages: consecutive, a multiple of 32 (its first page may lie past the end).
template <int kCtas>
struct WarpPages {
    long long begin, end;
    __device__ __forceinline__ explicit WarpPages(long long pages) {
        constexpr int kWarps = kCtas * kPlanThreads / 32;
        const long long per = ((pages + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int w = (int)((blockIdx.x * kPlanThreads + threadIdx.x) >> 5);
        begin = min(pages, w * per);
        end = min(pages, begin + per);
    }
};

constexpr int kScanDepth = 8;         // loads of 32 pages in flight a warp

// Walks the warp's pages in order, 32 at a time: f(page, used, mask of the used among the 32, lanes
// that hold a page).
template <typename W, typename F>
__device__ __forceinline__ void scan_pages(const W &w, const int32_t *refs, F f) {
    const int lane = threadIdx.x & 31;
    for (long long p0 = w.begin; p0 < w.end; p0 += 32 * kScanDepth) {
        int x[kScanDepth];
#pragma unroll
        for (int i = 0; i < kScanDepth; ++i) {
            const long long p = p0 + 32 * i + lane;
            x[i] = p < w.end ? refs[p] : 0;
        }
#pragma unroll
        for (int i = 0; i < kScanDepth; ++i) {
            const long long p = p0 + 32 * i + lane;
            if (p0 + 32 * i >= w.end) break;
            const unsigned there = __ballot_sync(0xffffffffu, p < w.end);
            const unsigned used = __ballot_sync(0xffffffffu, x[i] > 0);
            f(p, x[i] > 0, used, there);
        }
    }
}

// ---------------------------------------------------------------------------
// Pages copied: K, V, weights and positions of every row.  A piece is 2 KB of a page's K and the
// same of its V, all in flight in a warp.
// ---------------------------------------------------------------------------
constexpr int kPieceVecs = 128;       // 16-byte vectors of K (and of V) in a piece

__device__ __forceinline__ void copy_piece(const DevPaged &C, int32_t *row_pos, int src, int dst,
                                           int piece) {
    const int lane = threadIdx.x & 31;
    const long long page_vecs = (long long)C.ps * C.d / 8;
    const uint4 *k = static_cast<const uint4 *>(C.k), *v = static_cast<const uint4 *>(C.v);
    uint4 *kd = static_cast<uint4 *>(C.k), *vd = static_cast<uint4 *>(C.v);
    const long long from = src * page_vecs + piece * kPieceVecs + lane;
    const long long to = dst * page_vecs + piece * kPieceVecs + lane;
    uint4 a[kPieceVecs / 32], b[kPieceVecs / 32];
#pragma unroll
    for (int i = 0; i < kPieceVecs / 32; ++i) {
        a[i] = ld_nc(k + from + 32 * i);
        b[i] = ld_nc(v + from + 32 * i);
    }
    if (piece == 0) {
        const long long r0 = (long long)src << C.ps_log2, r1 = (long long)dst << C.ps_log2;
        for (int j = lane; j < C.ps; j += 32) {
            if (C.mass) C.mass[r1 + j] = C.mass[r0 + j];
            if (row_pos) row_pos[r1 + j] = row_pos[r0 + j];
        }
    }
#pragma unroll
    for (int i = 0; i < kPieceVecs / 32; ++i) {
        st_cs(kd + to + 32 * i, a[i]);
        st_cs(vd + to + 32 * i, b[i]);
    }
}

// ---------------------------------------------------------------------------
// Pages for a step's tokens.  A unit of n rows that gets t more needs the pages of rows n .. n + t - 1
// that it has none for, and one more if its last page is part full and shared: that page is copied
// and the copy takes its place.  The k-th page needed, units in order, tail first, is the k-th
// free page.  Nothing changes unless all fit; what the step has queued behind the call then finds a
// mark in the status word and writes nothing either (without_rows).
//
// The plan leaves every unit what it needs and the free pages in order; the second kernel, a
// warp a unit and piece of its copied page, enters and copies them.  (All in the plan's cluster, the
// tables' entries were a chain of loads more in a kernel of 8 blocks: 14.3 us for 2048 units
// and 59000 pages, 11.5 now, without the copies.)
// ---------------------------------------------------------------------------
// Warp w of `warps`: the units' pages entered and copied, `run` pieces of a page by a warp.
__device__ __forceinline__ void enter_pages(const DevPaged &C, const DevChunk &T, int32_t *refs,
                                            int32_t *row_pos, const PagesWs &ws, int run,
                                            long long w, long long warps) {
    const int lane = threadIdx.x & 31, pieces = C.ps * C.d / 8 / kPieceVecs;     // at least one
    const int per = C.L * C.H, runs = (pieces + run - 1) / run;
    for (long long i = w; i < C.units * runs; i += warps) {
        const int u = (int)(i / runs), piece = (int)(i - (long long)u * runs) * run;
        const UnitNeed need = ws.need[u];
        if (need.from >= 0) {
            const int to = ws.list[need.at];
            for (int k = piece; k < min(pieces, piece + run); ++k)
                copy_piece(C, row_pos, need.from, to, k);
        }
        if (piece) continue;
        int32_t *tab = table_of(C, u) + need.col;
        for (int j = lane; j < need.pages; j += 32) {
            const int page = ws.list[need.at + j];
            tab[j] = page;
            refs[page] = 1;
        }
        if (lane == 0) {
            if (need.from >= 0) atomicSub(refs + need.from, 1);
            const int r = u / per;
            C.lens[u] += (int)(T.off[r + 1] - T.off[r]);
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads, 4)
reserve_enter_kernel(const DevPaged C, const DevChunk T, int32_t *refs, int32_t *row_pos,
                     const PagesWs ws, int run) {
    pdl_wait();
    pdl_trigger();
    if (ws.plan->count == 0) return;
    enter_pages(C, T, refs, row_pos, ws, run, (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5),
                (long long)gridDim.x * (kCopyThreads / 32));
}

// whole (one block): the block enters the pages too.
template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads, 1)
reserve_plan_kernel(const DevPaged C, const DevChunk T, int32_t *refs, int32_t *row_pos,
                    const PagesWs ws, bool whole) {
    constexpr int kAll = kCtas * kPlanThreads;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int units = (int)C.units, chunk = (units + kAll - 1) / kAll;   // units: at most 2^28
    const int gt = (int)(blockIdx.x * kPlanThreads + threadIdx.x);
    const int u0 = (int)min((long long)units, (long long)gt * chunk);
    const int u1 = min(units, u0 + chunk);
    const int per = C.L * C.H;
    // pages needed, free pages, units that cannot be, units longer than their table; the first is
    // at most num_pages + 2 units (the host has checked the tokens)
    int mine[4] = {0, 0, 0, 0};
    UnitNeed last{0, 0, -1, 0};
    for (int u = u0; u < u1; ++u) {
        const int r = u / per, t = (int)(T.off[r + 1] - T.off[r]);
        int n;
        UnitNeed need{0, 0, -1, 0};
        if (!unit_len(C, u, n)) {
            mine[2] += 1;
        } else if (t > C.cap - n) {
            mine[3] += 1;
        } else if (t > 0) {
            need.col = pages_of(C, n);
            need.pages = pages_of(C, n + t) - need.col;
            if (n & (C.ps - 1)) {
                const int page = C.table[(long long)u * C.max_pages + need.col - 1];
                if (!page_ok(C, page)) {
                    mine[2] += 1;
                } else if (refs[page] > 1) {
                    need.from = page;
                    need.col -= 1;
                    need.pages += 1;
                }
            }
        }
        need.at = mine[0];                       // after the thread's own before it
        mine[0] += need.pages;
        last = need;
        if (chunk > 1) ws.need[u] = need;
    }
    const WarpPages<kCtas> W(C.num_pages);
    int free_pages = 0;
    scan_pages(W, refs, [&](long long, bool, unsigned used, unsigned there) {
        free_pages += __popc(there & ~used);
    });
    if (lane == 0) mine[1] = free_pages;
    const auto s = cluster_scan<kCtas>(mine);
    const bool fits = s.total[2] == 0 && s.total[3] == 0 && s.total[0] <= s.total[1];
    if (gt == 0) {
        ws.plan->count = fits ? 1 : 0;
        if (fits) {
            atomicAnd(C.status, ~kStatusNoRows);
        } else {
            post_status(C.status, s.total[2] > 0 ? KV_ERR_INVALID_ARG : KV_ERR_BUDGET);
            atomicOr(C.status, kStatusNoRows);
        }
    }
    if (fits) {
        for (int u = u0; u < u1; ++u) {
            UnitNeed need = chunk > 1 ? ws.need[u] : last;
            need.at += s.before[0];
            ws.need[u] = need;
        }
        // the free pages that are given out, in order
        int rank = __shfl_sync(0xffffffffu, s.before[1], 0);
        scan_pages(W, refs, [&](long long p, bool is_used, unsigned used, unsigned there) {
            const unsigned open = there & ~used;
            const int k = rank + __popc(open & low_bits(lane));
            if (!is_used && (there >> lane & 1) && k < s.total[0]) ws.list[k] = (int)p;
            rank += __popc(open);
        });
        if (kCtas == 1 && whole) {
            __syncthreads();
            enter_pages(C, T, refs, row_pos, ws, 1, threadIdx.x >> 5, kPlanThreads / 32);
        }
    }
    leave_cluster<kCtas>();
}

// ---------------------------------------------------------------------------
// Compaction.  With `live` pages in use, the k-th page in use from page `live` on goes to the k-th
// free page before it.  The plan lists both, the pages to move from the last one on (their
// number is known to no block while they are listed), so the k-th listed goes to the hole listed
// k-th from the end.
// ---------------------------------------------------------------------------
// Warp w of `warps`: the tables follow their pages, then the pages move, a piece at a time.
__device__ __forceinline__ void move_pages(const DevPaged &C, int32_t *refs, int32_t *row_pos,
                                           const PagesWs &ws, int count, int live, long long w,
                                           long long warps) {
    const int lane = threadIdx.x & 31;
    for (long long u = w; u < C.units; u += warps) {
        int n;
        if (!unit_len(C, u, n)) {
            if (lane == 0) post_status(C.status, KV_ERR_INVALID_ARG);
            continue;
        }
        int32_t *tab = table_of(C, u);
        const int held = pages_of(C, n);
        for (int c = lane; c < held; c += 32) {
            const int page = tab[c];
            if (!page_ok(C, page)) post_status(C.status, KV_ERR_INVALID_ARG);
            else if (page >= live) {
                // a page without a reference, which a table names all the same, goes nowhere
                const int k = ws.list[page];
                if (k < 0) post_status(C.status, KV_ERR_INVALID_ARG);
                else tab[c] = ws.dst[count - 1 - k];
            }
        }
    }
    const int pieces = C.ps * C.d / 8 / kPieceVecs;          // at least one
    for (long long i = w; i < (long long)count * pieces; i += warps) {
        const int j = (int)(i / pieces), piece = (int)(i - (long long)j * pieces);
        const int from = ws.src[j], to = ws.dst[count - 1 - j];
        copy_piece(C, row_pos, from, to, piece);
        if (piece == 0 && lane == 0) {
            refs[to] = refs[from];
            refs[from] = 0;
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads, 4)
compact_move_kernel(const DevPaged C, int32_t *refs, int32_t *row_pos, const PagesWs ws) {
    pdl_wait();
    pdl_trigger();
    const int count = ws.plan->count;
    if (count)
        move_pages(C, refs, row_pos, ws, count, ws.plan->live,
                   (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5),
                   (long long)gridDim.x * (kCopyThreads / 32));
}

template <int kCtas>
__global__ void __launch_bounds__(kPlanThreads, 1)
compact_plan_kernel(const DevPaged C, int32_t *refs, int32_t *row_pos, int32_t *live_out,
                    const PagesWs ws, bool whole) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && threadIdx.x == 0) ws.plan->count = 0;
    const WarpPages<kCtas> W(C.num_pages);
    int in_use = 0;
    scan_pages(W, refs, [&](long long, bool, unsigned used, unsigned) { in_use += __popc(used); });
    const int mine[1] = {lane == 0 ? in_use : 0};
    const auto s = cluster_scan<kCtas>(mine);
    const int live = s.total[0];
    int at = __shfl_sync(0xffffffffu, s.before[0], 0);       // in use before the 32 looked at
    int holes = 0;                                           // this warp's free pages before `live`
    scan_pages(W, refs, [&](long long p, bool is_used, unsigned used, unsigned there) {
        const int used_before = at + __popc(used & low_bits(lane));
        if (there >> lane & 1) {
            if (p < live) {
                // as many pages lie before p as are free or in use
                if (!is_used) ws.dst[(int)p - used_before] = (int)p;
            } else {
                const int k = live - 1 - used_before;
                if (is_used) ws.src[k] = (int)p;
                ws.list[p] = is_used ? k : -1;
            }
        }
        holes += __popc(there & ~used & __ballot_sync(0xffffffffu, p < live));
        at += __popc(used);
    });
    // (the count's zero came before the cluster's first barrier)
    if (lane == 0 && holes) atomicAdd(&ws.plan->count, holes);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        ws.plan->live = live;
        if (live_out) *live_out = live;
    }
    if (kCtas == 1 && whole) {
        __syncthreads();
        const int count = ws.plan->count;
        if (count)
            move_pages(C, refs, row_pos, ws, count, live, threadIdx.x >> 5, kPlanThreads / 32);
    }
    leave_cluster<kCtas>();
}

// ---------------------------------------------------------------------------
// Requests go on from others' caches.  A block takes one (layer, head) of all requests, so that it
// alone reads and writes their entries and lengths: a strip of columns of every request into
// shared memory, then out to the requests that go on from another.  8 hypotheses of 256 units of 1638 rows
// 3.1 us replayed, 64 of them 9.8; 1000 requests of one (layer, head), one block's work, 58.
// ---------------------------------------------------------------------------
constexpr int kForkThreads = 256;
constexpr int kForkSmem = 192 * 1024;

__global__ void __launch_bounds__(kForkThreads)
fork_kernel(const DevPaged C, int32_t *refs, const int32_t *parents, int strip) {
    extern __shared__ __align__(16) int s_fork[];
    int *s_parent = s_fork, *s_len = s_parent + C.R, *s_page = s_len + C.R;   // [R][strip]
    __shared__ int s_most;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0) s_most = 0;
    __syncthreads();
    const int lh = blockIdx.x;
    auto unit = [&](int r) { return (long long)r * C.L * C.H + lh; };
    auto held = [&](int r) {
        const int n = s_len[r];
        return n >= 0 && n <= C.cap ? pages_of(C, n) : 0;
    };
    bool any = false;
    for (int r = threadIdx.x; r < C.R; r += kForkThreads) {
        int p = parents[r];
        if (p < -1 || p >= C.R) {
            post_status(C.status, KV_ERR_INVALID_ARG);
            p = r;
        }
        s_parent[r] = p;
        const int n = C.lens[unit(r)];
        s_len[r] = n;
        if (n < 0 || n > C.cap) post_status(C.status, KV_ERR_INVALID_ARG);
        else atomicMax(&s_most, pages_of(C, n));
        any |= p != r;
    }
    if (!__syncthreads_or(any)) return;
    const int cols = s_most;
    for (int c0 = 0; c0 < cols; c0 += strip) {
        for (int i = threadIdx.x; i < C.R * strip; i += kForkThreads) {
            const int r = i / strip, c = c0 + i - r * strip;
            s_page[i] = c < held(r) ? C.table[unit(r) * C.max_pages + c] : -1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < C.R * strip; i += kForkThreads) {
            const int r = i / strip, j = i - r * strip, c = c0 + j, p = s_parent[r];
            if (p == r) continue;
            const int old = s_page[i], page = p >= 0 && c < held(p) ? s_page[p * strip + j] : -1;
            if (p >= 0 && c < held(p)) {
                table_of(C, unit(r))[c] = page;
                if (page_ok(C, page)) atomicAdd(refs + page, 1);
                else post_status(C.status, KV_ERR_INVALID_ARG);
            }
            if (c < held(r)) {
                if (page_ok(C, old)) atomicSub(refs + old, 1);
                else post_status(C.status, KV_ERR_INVALID_ARG);
            }
        }
        __syncthreads();
    }
    for (int r = threadIdx.x; r < C.R; r += kForkThreads) {
        const int p = s_parent[r];
        if (p != r) C.lens[unit(r)] = p >= 0 ? s_len[p] : 0;
    }
}

// Table entries in use, counted: a warp a unit, 32 entries a step.  Bound by latency: 256 units of 1638 rows
// 3.1 us with the zeroing, 2048 of them 3.4; 16 units of 131072 rows, 64 steps each, 16.
__global__ void __launch_bounds__(256) count_refs_kernel(const DevPaged C, int32_t *refs) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * 8;
    for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < C.units; u += warps) {
        int n;
        if (!unit_len(C, u, n)) {
            if (lane == 0) post_status(C.status, KV_ERR_INVALID_ARG);
            continue;
        }
        const int held = pages_of(C, n);
        for (int c = lane; c < held; c += 32) {
            const int page = C.table[u * C.max_pages + c];
            if (page_ok(C, page)) atomicAdd(refs + page, 1);
            else post_status(C.status, KV_ERR_INVALID_ARG);
        }
    }
}

// Positions of every unit's rows: a warp a unit, 32 rows a step, each step a chain of list, table and
// (with a source) position before its store.  Bound by that latency, once after a load or an eviction: 256 units of
// 1638 rows by their lists 14.3 us, 2048 of them 14.8 (27 MB); 112 units of 6553 rows 51, of a source's rows 93;
// 16 of 131072 rows 990.  Long units would want several warps each.
__global__ void __launch_bounds__(256)
place_positions_kernel(const DevPaged D, int32_t *dst_pos, const DevPaged S, const int32_t *src_pos,
                       const int32_t *index, long long stride, const int64_t *offsets) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * 8;
    for (long long u = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); u < D.units; u += warps) {
        int n;
        bool bad = !unit_len(D, u, n);
        const int32_t *list = index ? index + (offsets ? offsets[u] : u * stride) : nullptr;
        const long long listed = !index ? n : offsets ? offsets[u + 1] - offsets[u] : stride;
        if (n > listed) {
            // more rows than the unit's list names
            bad = true;
            n = (int)max(0ll, listed);
        }
        for (int i = lane; i < n; i += 32) {
            int p = list ? list[i] : i;
            if (src_pos) {
                // a row of the source cache
                const long long row =
                    p >= 0 && p < S.cap ? page_row(S, S.table + u * S.max_pages, p) : -1;
                bad |= row < 0;
                p = row < 0 ? -1 : src_pos[row];
            }
            const long long to = page_row(D, D.table + u * D.max_pages, i);
            if (to >= 0) dst_pos[to] = p;
            bad |= to < 0;
        }
        if (bad) post_status(D.status, KV_ERR_INVALID_ARG);
    }
}

unsigned unit_grid(long long units) {
    const long long n = (units + 7) / 8;
    return (unsigned)(n < 1 ? 1 : n < 4096 ? n : 4096);
}

PagesWs layout(const DevPaged &C, bool reserve, void *base) {
    PagesWs ws{};
    char *b = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = b ? b + off : nullptr;
        off = (off + bytes + 255) / 256 * 256;
        return p;
    };
    const size_t pages = (size_t)C.num_pages;
    ws.plan = reinterpret_cast<PagePlan *>(take(sizeof(PagePlan)));
    ws.list = reinterpret_cast<int *>(take(pages * sizeof(int)));
    if (reserve) {
        ws.need = reinterpret_cast<UnitNeed *>(take((size_t)C.units * sizeof(UnitNeed)));
    } else {
        ws.src = reinterpret_cast<int *>(take(pages * sizeof(int)));
        ws.dst = reinterpret_cast<int *>(take(pages * sizeof(int)));
    }
    ws.total = off;
    return ws;
}

// A plan by one block, whose threads meet without a cluster's barrier, where it has few pages and
// units a thread.  One block / a cluster, us a call (reserve, compaction that moves nothing):
//   64 pages, 8 units    5.5 / 8.9   3.6 / 5.1     8192 pages, 2048 units   10.4 / 10.0   6.2 / 6.5
//   4096 pages, 64 units 6.9 / 9.0   5.3 / 6.6    16384 pages, 2048 units   12.6 / 10.7   9.8 / 7.4
//   8192 pages, 512 units 7.9 / 9.7  6.3 / 6.4    57344 pages, 2048 units   23.9 / 11.2  21.9 / 8.8
bool one_block(const DevPaged &C) {
    return C.num_pages <= 8 * kPlanThreads && C.units <= 2 * kPlanThreads;
}
unsigned copy_grid(long long warps) {
    constexpr int kWarps = kCopyThreads / 32;
    const long long grid = (warps + kWarps - 1) / kWarps;
    return (unsigned)std::min<long long>(std::max<long long>(grid, 1), kCopyCtas);
}
// The block of such a plan also does what follows, in place of a second launch, where that is a
// few rounds of its 32 warps.
constexpr int kWholePieces = 256;
int page_pieces(const DevPaged &C) { return C.ps * C.d / 8 / kPieceVecs; }

}  // namespace

PagesWs reserve_ws_layout(const DevPaged &C, void *base) { return layout(C, true, base); }
PagesWs compact_ws_layout(const DevPaged &C, void *base) { return layout(C, false, base); }

cudaError_t launch_reserve(const DevPaged &C, const DevChunk &T, int32_t *refs, int32_t *row_pos,
                           const PagesWs &ws, cudaStream_t s) {
    const long long pieces = C.units * page_pieces(C);
    if (one_block(C)) {
        const bool whole = pieces <= kWholePieces;
        const cudaError_t e = launch_dependent(reserve_plan_kernel<1>, dim3(1), kPlanThreads, 0, s, C, T,
                                               refs, row_pos, ws, whole);
        if (e != cudaSuccess || whole) return e;
    } else {
        const cudaError_t e =
            launch_cluster_dependent(reserve_plan_kernel<kPlanCtas>, kPlanCtas, dim3(kPlanCtas),
                                     kPlanThreads, 0, s, C, T, refs, row_pos, ws, false);
        if (e != cudaSuccess) return e;
    }
    // four pieces a warp where all warps have one: what a unit needs is then looked up once for them
    // (2048 units with pages of 16 pieces: 29 us with the fork and the plan, 32 a piece at a time)
    const int run = pieces > kCopyCtas * (kCopyThreads / 32) ? 4 : 1;
    return launch_dependent(reserve_enter_kernel, dim3(copy_grid((pieces + run - 1) / run)), kCopyThreads,
                            0, s, C, T, refs, row_pos, ws, run);
}

cudaError_t launch_compact_pages(const DevPaged &C, int32_t *refs, int32_t *row_pos, int32_t *live,
                                 const PagesWs &ws, cudaStream_t s) {
    const long long moved = (C.num_pages + 1) / 2 * page_pieces(C);      // pieces at most
    const long long work = std::max(moved, C.units);
    if (one_block(C)) {
        const bool whole = work <= kWholePieces;
        const cudaError_t e = launch_dependent(compact_plan_kernel<1>, dim3(1), kPlanThreads, 0, s, C,
                                               refs, row_pos, live, ws, whole);
        if (e != cudaSuccess || whole) return e;
    } else {
        const cudaError_t e =
            launch_cluster_dependent(compact_plan_kernel<kPlanCtas>, kPlanCtas, dim3(kPlanCtas),
                                     kPlanThreads, 0, s, C, refs, row_pos, live, ws, false);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(compact_move_kernel, dim3(copy_grid(work)), kCopyThreads, 0, s, C, refs,
                            row_pos, ws);
}

cudaError_t launch_fork(const DevPaged &C, int32_t *refs, const int32_t *parents, cudaStream_t s) {
    const size_t fixed = (size_t)C.R * 2 * sizeof(int);
    // columns a step: a warp's width at least where they fit, the table's at most
    long long strip = (long long)(kForkSmem - fixed) / ((long long)C.R * sizeof(int));
    strip = strip > kForkThreads ? kForkThreads : strip;
    strip = strip > C.max_pages ? C.max_pages : strip;
    const size_t smem = fixed + (size_t)C.R * strip * sizeof(int);
    // (a block has 48 KB unasked, of which its static word takes a part)
    const cudaError_t e = cudaFuncSetAttribute(
        fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kForkSmem);
    return e != cudaSuccess ? e
                            : launch_dependent(fork_kernel, dim3((unsigned)(C.L * C.H)), kForkThreads,
                                               smem, s, C, refs, parents, (int)strip);
}

cudaError_t launch_count_refs(const DevPaged &C, int32_t *refs, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(refs, 0, (size_t)C.num_pages * sizeof(int32_t), s);
    return e != cudaSuccess ? e
                            : launch_dependent(count_refs_kernel, dim3(unit_grid(C.units)), 256, 0, s, C,
                                               refs);
}

cudaError_t launch_place_positions(const DevPaged &D, int32_t *dst_pos, const DevPaged &S,
                                   const int32_t *src_pos, const int32_t *index, long long stride,
                                   const int64_t *offsets, cudaStream_t s) {
    return launch_dependent(place_positions_kernel, dim3(unit_grid(D.units)), 256, 0, s, D, dst_pos, S,
                            src_pos, index, stride, offsets);
}

}  // namespace kvevict
