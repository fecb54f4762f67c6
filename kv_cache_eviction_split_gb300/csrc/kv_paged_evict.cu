// kv_paged_evict.cu -- eviction by accumulated attention weight.
//
// select: per unit with n rows and budget b < n, theta = the k-th largest weight of the
// rows between the pinned ones (k = b - sinks - recent), by a radix select on the fp32
// bit patterns, and the kept rows in order: those above theta, and of those equal to it
// the first ones.  gather: kept row i of src becomes row i of dst.
//
// The weights are read once, as vectors of four rows of a page: a unit's rows are spread
// over the registers and shared memory of a block (tables to 4096 and to 16384 rows) or of a
// cluster of 8 (131072 rows; longer slices are re-read), and the three digit passes (11, 11
// and 10 bits) count from there; a cluster's counts are added bin range by bin range through
// distributed shared memory.  The passes are bound by latencies: of 85 us for 112 units of
// 131072 rows, 25 load, 13 + 2 x 18 are the passes, 12 order the rows; 4 of each pass's are
// the cluster's exchange.  Keys in registers (51 clusters
// at a time in place of 36) and vectors together took 5 us off.
// The gather is bound by HBM (6.05 TB/s at 112 units of 6553 rows, d = 128): it is a kernel
// of its own, which spreads the rows evenly over the SMs; a cluster that moved its own rows
// beside the other clusters' passes took 8 us longer in all.
#include <cooperative_groups.h>

#include "kv_compact.cuh"
#include "kv_paged_attend.cuh"

namespace kvevict {
namespace {
namespace cg = cooperative_groups;

constexpr int kBins = 2048;      // digits of 11, 11 and 10 bits

struct EvictArgs {
    const int32_t *budgets;
    int sinks, recent;
    int32_t *kept;
    long long kept_stride;
    int *status;
};

// Sums over the block's warps: `before` of the warps before this one, and the total.
template <int kT>
__device__ __forceinline__ void warp_prefix(unsigned x, unsigned *s_warp, unsigned &before,
                                            unsigned &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    const unsigned y = lane < kT / 32 ? s_warp[lane] : 0u;
    before = __reduce_add_sync(0xffffffffu, lane < warp ? y : 0u);
    total = __reduce_add_sync(0xffffffffu, y);
}

// Rows i0 .. i1 - 1 of unit u's kept list, by the kWarps warps of a block.  A warp moves 32
// consecutive rows: each lane looks up one row's two places (kept index, page tables), then
// the warp copies the rows in batches of kBatch with all their loads in flight, K and V of
// a row (or of two, d = 64) side by side over its lanes.
template <int D, int kWarps>
__device__ __forceinline__ void gather_rows(const DevPaged &S, const DevPaged &Q,
                                            const EvictArgs &A, long long u, int i0, int i1) {
    constexpr int kVecs = D / 8, kLanes = 2 * kVecs, kRows = 32 / kLanes, kBatch = 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / kLanes, which = (lane % kLanes) / kVecs, ch = lane % kVecs;
    const uint4 *src = static_cast<const uint4 *>(which ? S.v : S.k);
    uint4 *dst = static_cast<uint4 *>(which ? Q.v : Q.k);
#pragma unroll 1
    for (int w0 = i0 + warp * 32; w0 < i1; w0 += kWarps * 32) {
        long long from = -1, to = -1;
        if (w0 + lane < i1) {
            const int j = A.kept[u * A.kept_stride + w0 + lane];
            from = page_row(S, S.table + u * S.max_pages, j);
            to = page_row(Q, Q.table + u * Q.max_pages, w0 + lane);
            if (from < 0 || to < 0) {
                post_status(A.status, KV_ERR_INVALID_ARG);
                from = -1;
            } else if (Q.mass) {
                Q.mass[to] = S.mass[from];
            }
        }
#pragma unroll 1
        for (int r0 = 0; r0 < 32 && w0 + r0 < i1; r0 += kBatch * kRows) {
            uint4 buf[kBatch];
            bool ok[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const long long a = __shfl_sync(0xffffffffu, from, r0 + q * kRows + sub);
                ok[q] = a >= 0;
                if (ok[q]) buf[q] = ld_nc(src + a * kVecs + ch);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const long long z = __shfl_sync(0xffffffffu, to, r0 + q * kRows + sub);
                if (ok[q]) st_cs(dst + z * kVecs + ch, buf[q]);
            }
        }
    }
}

// One unit by a block of kT threads (kCluster = 1) or a cluster of such blocks.  Rows are
// dealt to blocks in equal consecutive slices, which a block walks in rounds of kT * kQuads
// quads of rows (one, where the slice fits: its keys are loaded once).  A quad never leaves
// its page and is loaded as one vector; quad q * kT + t of a round is thread t's, kRegs of
// its kQuads in registers and the others in shared memory, which no other thread reads.
template <int kT, int kQuads, int kRegs, int kCluster>
__global__ void __launch_bounds__(kT, kCluster > 1 ? 3 : 1)
evict_select_kernel(const DevPaged S, const DevPaged Q, const EvictArgs A) {
    constexpr int kRound = kT * kQuads * 4, kW = kT / 32;
    extern __shared__ __align__(16) uint4 s_key[];         // [kQuads - kRegs][kT]
    __shared__ unsigned hist[kBins], sums[kCluster > 1 ? kBins : 1];
    __shared__ int s_tab[kRound / 16 + 2];                 // the round's page table entries
    __shared__ unsigned s_cnt[kCluster > 1 ? kT : kQuads * kW];
    __shared__ unsigned s_warp[32], s_pick[2], s_counts[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kCluster > 1 ? (int)(blockIdx.x % kCluster) : 0;
    const long long u = blockIdx.x / kCluster;
    auto sync_all = [&]() {
        if constexpr (kCluster > 1) cg::this_cluster().sync();
        else __syncthreads();
    };
    int n;
    const bool len_ok = unit_len(S, u, n);
    const long long b = A.budgets[u];
    const long long keep = b < n ? b : n;
    // The gather's blocks may be set up when all of these run; those of a cluster's launch,
    // which fill the SMs several times over, leave room for it at their end (11 us sooner).
    if (kCluster == 1) pdl_trigger();
    if (!len_ok || b < (long long)A.sinks + A.recent || keep > A.kept_stride || keep > Q.cap) {
        if (rank == 0 && tid == 0) {
            post_status(A.status, len_ok ? KV_ERR_BUDGET : KV_ERR_INVALID_ARG);
            Q.lens[u] = -1;
        }
        return;                                   // the same in every block of the cluster
    }
    if (rank == 0 && tid == 0) Q.lens[u] = (int)keep;
    int32_t *out = A.kept + u * A.kept_stride;
    // rows kept whatever their weight: this block's share, in rank order
    const unsigned k = n <= b ? 0u : (unsigned)(b - A.sinks - A.recent);
    if (k == 0) {
        // all rows, or the pinned ones alone
        const int part = ((int)keep + kCluster - 1) / kCluster;
        const int i0 = min((int)keep, rank * part), i1 = min((int)keep, i0 + part);
        for (int i = i0 + tid; i < i1; i += kT) out[i] = n <= b || i < A.sinks ? i : n - (int)b + i;
        return;
    }
    if (rank == 0)
        for (int j = tid; j < A.sinks; j += kT) out[j] = j;
    if (rank == kCluster - 1)
        for (int j = tid; j < A.recent; j += kT) out[b - A.recent + j] = n - A.recent + j;

    // this block's slice [lo, hi) of the rows between the pinned ones; lo a quad's first row,
    // which may be pinned itself
    const int first = A.sinks, end = n - A.recent;
    const int slice = ((end - (first & ~3) + kCluster - 1) / kCluster + 31) / 32 * 32;
    const int lo = min(end, (first & ~3) + rank * slice), hi = min(end, lo + slice);
    const int32_t *tab = S.table + u * S.max_pages;
    const bool held = hi - lo <= kRound;
    uint4 rk[kRegs];
    // Keys of the round that starts at r0: its table entries, then two vectors a thread in
    // flight (kRegs at first).  Rows past the slice's end get key 0, the smallest: the passes
    // below may count them, as at least as many rows as are wanted lie above them.  A page
    // that does not exist is posted; its rows count as weight 0.
    auto load = [&](int r0) {
        const int m = min(kRound, hi - r0);
        if (m <= 0) return;
        if (!held) __syncthreads();               // the entries before are read
        const int e0 = r0 >> S.ps_log2, e1 = (r0 + m - 1) >> S.ps_log2;
        for (int e = e0 + tid; e <= e1; e += kT) {
            const int page = __ldg(tab + e);
            const bool ok = page >= 0 && page < S.num_pages;
            if (!ok) post_status(A.status, KV_ERR_INVALID_ARG);
            s_tab[e - e0] = ok ? page : -1;
        }
        __syncthreads();
        auto quad = [&](int q) {
            const int i = (q * kT + tid) * 4, j = r0 + i;
            const int page = i < m ? s_tab[(j >> S.ps_log2) - e0] : -1;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (page >= 0)
                x = __ldg(reinterpret_cast<const uint4 *>(
                    S.mass + ((long long)page << S.ps_log2) + (j & (S.ps - 1))));
            if (i + 1 >= m) x.y = 0u;
            if (i + 2 >= m) x.z = 0u;
            if (i + 3 >= m) x.w = 0u;
            return x;
        };
#pragma unroll
        for (int q = 0; q < kRegs; ++q) rk[q] = quad(q);
#pragma unroll 2
        for (int q = kRegs; q < kQuads; ++q) s_key[(q - kRegs) * kT + tid] = quad(q);
    };
    // f(q, keys of quad q) for the thread's quads of the round of m rows
    auto each_quad = [&](int m, auto f) {
#pragma unroll
        for (int q = 0; q < kQuads; ++q)
            if (q * kT * 4 < m) f(q, q < kRegs ? rk[q < kRegs ? q : 0] : s_key[(q - kRegs) * kT + tid]);
    };
    if (held) load(lo);
    unsigned prefix = 0, mask = 0, remaining = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const unsigned digit = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < kBins; i += kT) hist[i] = 0;
        __syncthreads();
        for (int r0 = lo; r0 < hi; r0 += kRound) {
            if (!held) load(r0);
            const bool pinned = r0 + tid * 4 < first;        // in the thread's first quad
            const int m = min(kRound, hi - r0);
            each_quad(m, [&](int q, const uint4 &key) {
                if ((q * kT + tid) * 4 >= m) return;
                auto add = [&](unsigned x) {
                    if ((x & mask) == prefix) atomicAdd(&hist[x >> shift & digit], 1u);
                };
                if (q > 0 || !pinned) {
                    add(key.x);
                    add(key.y);
                    add(key.z);
                    add(key.w);
                } else {
                    const int i = r0 + tid * 4 - first;      // -1 .. -3
                    if (i >= -1) add(key.y);
                    if (i >= -2) add(key.z);
                    add(key.w);
                }
            });
        }
        sync_all();
        const unsigned *count = hist;
        if constexpr (kCluster > 1) {
            // block r adds up bins [r * kBins / kCluster, ...) of all blocks and hands the
            // sums to all of them
            constexpr int kMine = kBins / kCluster;
            static_assert(kT % kMine == 0 || kMine % kT == 0, "whole bins a thread");
            constexpr int kSplit = kT / kMine, kRanks = kCluster / kSplit;
            static_assert(kSplit >= 1 && kCluster % kSplit == 0, "ranks split evenly");
            const int bin = rank * kMine + tid % kMine, r0 = tid / kMine * kRanks;
            unsigned x = 0;
#pragma unroll
            for (int r = 0; r < kRanks; ++r)
                x += *cg::this_cluster().map_shared_rank(&hist[bin], r0 + r);
            if (kSplit > 1) {
                // the other parts of a bin's sum are in threads kMine apart
                s_cnt[tid] = x;
                __syncthreads();
                x = 0;
#pragma unroll
                for (int i = 0; i < kSplit; ++i) x += s_cnt[tid % kMine + i * kMine];
            }
#pragma unroll
            for (int r = 0; r < kRanks; ++r)
                *cg::this_cluster().map_shared_rank(&sums[bin], r0 + r) = x;
            sync_all();
            count = sums;
        }
        // digits from the top: the bin where the running count reaches `remaining`
        constexpr int kPer = kBins / kT;          // bins a thread sums, highest first
        unsigned x[kPer], sum = 0;
        const int low = kBins - (tid + 1) * kPer;
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum += x[i] = count[low + kPer - 1 - i];
        unsigned incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        unsigned before, total;
        warp_prefix<kT>(__shfl_sync(0xffffffffu, incl, 31), s_warp, before, total);
        unsigned above = before + incl - sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (above < remaining && above + x[i] >= remaining) {
                s_pick[0] = low + kPer - 1 - i;
                s_pick[1] = above;
            }
            above += x[i];
        }
        __syncthreads();
        prefix |= s_pick[0] << shift;
        remaining -= s_pick[1];
        mask |= digit << shift;
    }
    const unsigned theta = prefix, need = remaining;   // `need` of the keys equal to theta

    // Rows of the round above theta and equal to it, as bits of the thread's quads, and
    // their numbers (16 bits each of a word) before them: in the warp's part of the quad's
    // row (excl), and before that part in the round (s_cnt).
    constexpr int kEntries = kQuads * kW;
    static_assert(kEntries <= kT && kQuads <= 8, "an entry a thread, a bit a row");
    unsigned gt = 0, is = 0, total = 0, excl[kQuads];
    auto classify = [&](int r0) {
        const int m = min(kRound, hi - r0), j0 = r0 + tid * 4;
        gt = is = 0;
        each_quad(m, [&](int q, const uint4 &key) {
            unsigned valid = 0xfu;
            const int i = (q * kT + tid) * 4;
            if (i + 4 > m) valid = i < m ? (1u << (m - i)) - 1u : 0u;
            if (q == 0 && j0 < first) valid &= 0xfu << (first - j0);
            const unsigned g = (key.x > theta) | (key.y > theta) << 1 | (key.z > theta) << 2 |
                               (key.w > theta) << 3;
            const unsigned e = (key.x == theta) | (key.y == theta) << 1 | (key.z == theta) << 2 |
                               (key.w == theta) << 3;
            gt |= (g & valid) << 4 * q;
            is |= (e & valid) << 4 * q;
        });
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            const unsigned x = (unsigned)(__popc(gt >> 4 * q & 0xfu) | __popc(is >> 4 * q & 0xfu) << 16);
            unsigned incl = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            excl[q] = incl - x;
            if (lane == 31) s_cnt[q * kW + warp] = incl;
        }
        __syncthreads();
        const unsigned x = tid < kEntries ? s_cnt[tid] : 0u;
        unsigned incl = x, before;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        warp_prefix<kT>(__shfl_sync(0xffffffffu, incl, 31), s_warp, before, total);
        if (tid < kEntries) s_cnt[tid] = before + incl - x;
        __syncthreads();
    };
    if (held) classify(lo);
    unsigned at = 0, eq = 0;                      // kept and equal rows before this block
    if constexpr (kCluster > 1) {
        unsigned c0 = total & 0xffffu, c1 = total >> 16;
        if (!held) {
            c0 = c1 = 0;
            for (int r0 = lo; r0 < hi; r0 += kRound) {
                load(r0);
                classify(r0);
                c0 += total & 0xffffu;
                c1 += total >> 16;
            }
        }
        if (tid == 0) {
            s_counts[0] = c0;
            s_counts[1] = c1;
        }
        sync_all();
        unsigned x0 = 0;
        if (lane < rank) {
            const unsigned *c = cg::this_cluster().map_shared_rank(s_counts, lane);
            x0 = c[0];
            eq = c[1];
        }
        x0 = __reduce_add_sync(0xffffffffu, x0);
        eq = __reduce_add_sync(0xffffffffu, eq);
        at = x0 + min(eq, need);
    }
    for (int r0 = lo; r0 < hi; r0 += kRound) {
        if (!held) {
            load(r0);
            classify(r0);
        }
        const unsigned left = need > eq ? need - eq : 0u;   // equal rows still wanted
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            unsigned todo = (gt | is) >> 4 * q & 0xfu;
            if (!todo) continue;
            const unsigned base = s_cnt[q * kW + warp] + excl[q];
            unsigned above = base & 0xffffu, same = base >> 16;   // before the row
            do {
                const int c = __ffs(todo) - 1;
                todo &= todo - 1;
                const bool eq_row = is >> (4 * q + c) & 1u;
                const unsigned dst = at + above + min(same, left);
                if ((!eq_row || same < left) && dst < k)
                    out[first + dst] = r0 + (q * kT + tid) * 4 + c;
                if (eq_row) ++same; else ++above;
            } while (todo);
        }
        at += (total & 0xffffu) + min(total >> 16, left);
        eq += total >> 16;
    }
    if constexpr (kCluster > 1) {
        pdl_trigger();
        sync_all();                               // no block leaves while its counts are read
    }
}

constexpr int kWarps = 8;
template <int D>
__global__ void __launch_bounds__(kWarps * 32, 3)
evict_gather_kernel(const DevPaged S, const DevPaged Q, const EvictArgs A, long long u0) {
    pdl_wait();
    pdl_trigger();
    const long long u = u0 + blockIdx.y;
    const int i0 = blockIdx.x * kWarps * 32;
    gather_rows<D, kWarps>(S, Q, A, u, i0, min(Q.lens[u], i0 + kWarps * 32));
}

template <int kT, int kQuads, int kRegs, int kCluster>
cudaError_t launch_select(const DevPaged &S, const DevPaged &Q, const EvictArgs &A,
                          cudaStream_t s) {
    constexpr int kSmem = kT * (kQuads - kRegs) * 16;
    static_assert(kT * kQuads * 4 <= 32768, "counts of a round are 16-bit");
    auto kernel = evict_select_kernel<kT, kQuads, kRegs, kCluster>;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(S.units * kCluster));
    cfg.blockDim = dim3(kT);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = kCluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, S, Q, A);
}

}  // namespace

cudaError_t launch_paged_evict(const DevPaged &S, const DevPaged &D, const int32_t *budgets,
                               int sinks, int recent, int32_t *kept, long long kept_stride,
                               int *status, cudaStream_t s) {
    const EvictArgs A{budgets, sinks, recent, kept, kept_stride, status};
    // the smallest shape that holds the longest possible unit in shared memory
    cudaError_t e = S.cap <= 4096    ? launch_select<256, 4, 4, 1>(S, D, A, s)
                    : S.cap <= 16384 ? launch_select<512, 8, 8, 1>(S, D, A, s)
                                     : launch_select<512, 8, 2, 8>(S, D, A, s);
    const long long most = kept_stride < D.cap ? kept_stride : D.cap;
    const unsigned gx = (unsigned)((most + kWarps * 32 - 1) / (kWarps * 32));
    // grid.y is limited to 65535 units a launch
    for (long long u0 = 0; e == cudaSuccess && u0 < S.units; u0 += 65535) {
        const dim3 grid(gx, (unsigned)(S.units - u0 < 65535 ? S.units - u0 : 65535));
        e = S.d == 64 ? launch_dependent(evict_gather_kernel<64>, grid, kWarps * 32, 0, s, S, D, A, u0)
                      : launch_dependent(evict_gather_kernel<128>, grid, kWarps * 32, 0, s, S, D, A,
                                         u0);
    }
    return e;
}

}  // namespace kvevict
