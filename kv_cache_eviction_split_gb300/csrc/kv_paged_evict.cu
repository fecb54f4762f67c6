// kv_paged_evict.cu -- eviction by accumulated attention weight.
//
// select: per unit with n rows and budget b < n, theta = the k-th largest weight of the
// rows between the pinned ones (k = b - sinks - recent), by a radix select on the fp32
// bit patterns, and the kept rows in order: those above theta, and of those equal to it
// the first ones.  gather: kept row i of src becomes row i of dst.
//
// The weights are read once: a unit's rows are spread over the shared memory of a block or
// of a cluster of 8 (up to 131072 rows; longer slices are re-read), and the three digit
// passes (11, 11 and 10 bits) count from there; a cluster's counts are added bin range by
// bin range through distributed shared memory.  The passes are bound by latencies
// (cluster barriers, remote reads), the gather by HBM: it is a kernel of its own, which
// spreads the rows evenly over the SMs.
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

// Shared-memory place of key i: a word of padding every 32, so that lanes may walk keys
// side by side or runs of kKeys each without bank conflicts.
__device__ __forceinline__ int key_at(int i) { return i + (i >> 5); }

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
// dealt to blocks in equal consecutive slices, which a block walks in rounds of kT * kKeys
// rows (one, where the slice fits: its keys are loaded once).
template <int kT, int kKeys, int kCluster>
__global__ void __launch_bounds__(kT, kCluster > 1 ? 2 : 1)
evict_select_kernel(const DevPaged S, const DevPaged Q, const EvictArgs A) {
    constexpr int kRound = kT * kKeys;
    extern __shared__ __align__(16) unsigned s_key[];      // [key_at(kRound)]
    __shared__ unsigned hist[kBins], sums[kCluster > 1 ? kBins : 1];
    __shared__ int s_tab[kRound / 16 + 2];                 // the round's page table entries
    __shared__ unsigned s_warp[32], s_pick[2], s_counts[2];
    const int tid = threadIdx.x, lane = tid & 31;
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
    pdl_trigger();
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

    // this block's slice [lo, hi) of the rows between the pinned ones
    const int first = A.sinks, rows = n - A.recent - first;
    const int slice = ((rows + kCluster - 1) / kCluster + 31) / 32 * 32;
    const int lo = first + min(rows, rank * slice), hi = first + min(rows, (rank + 1) * slice);
    const int32_t *tab = S.table + u * S.max_pages;
    const bool held = hi - lo <= kRound;
    // keys of the round that starts at r0: its table entries, then kBatch weights a thread
    // in flight.  A page that does not exist is posted; its rows count as weight 0.
    constexpr int kBatch = 16;
    auto load = [&](int r0) {
        const int m = min(kRound, hi - r0);
        if (m <= 0) return;
        if (!held) __syncthreads();               // the keys before are read
        const int e0 = r0 >> S.ps_log2, e1 = (r0 + m - 1) >> S.ps_log2;
        for (int e = e0 + tid; e <= e1; e += kT) {
            const int page = __ldg(tab + e);
            const bool ok = page >= 0 && page < S.num_pages;
            if (!ok) post_status(A.status, KV_ERR_INVALID_ARG);
            s_tab[e - e0] = ok ? page : -1;
        }
        __syncthreads();
#pragma unroll 1
        for (int q0 = 0; q0 < kKeys && q0 * kT < m; q0 += kBatch) {
            unsigned key[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int i = (q0 + q) * kT + tid, j = r0 + i;
                const int page = i < m ? s_tab[(j >> S.ps_log2) - e0] : -1;
                key[q] = page >= 0 ? __float_as_uint(__ldg(
                                         S.mass + ((long long)page << S.ps_log2) + (j & (S.ps - 1))))
                                   : 0u;
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) s_key[key_at((q0 + q) * kT + tid)] = key[q];
        }
        __syncthreads();
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
            const int m = min(kRound, hi - r0);
#pragma unroll 8
            for (int i = tid; i < m; i += kT) {
                const unsigned key = s_key[key_at(i)];
                if ((key & mask) == prefix) atomicAdd(&hist[key >> shift & digit], 1u);
            }
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
                unsigned *part = s_key + key_at(kRound);
                part[tid] = x;
                __syncthreads();
                x = 0;
#pragma unroll
                for (int i = 0; i < kSplit; ++i) x += part[tid % kMine + i * kMine];
            }
#pragma unroll
            for (int r = 0; r < kRanks; ++r)
                *cg::this_cluster().map_shared_rank(&sums[bin], r0 + r) = x;
            sync_all();
            count = sums;
        }
        // digits from the top: the bin where the running count reaches `remaining`
        constexpr int kPer = kBins / kT;          // bins a thread sums, highest first
        unsigned x[kPer], mine = 0;
        const int low = kBins - (tid + 1) * kPer;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine += x[i] = count[low + kPer - 1 - i];
        unsigned incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        unsigned before, total;
        warp_prefix<kT>(__shfl_sync(0xffffffffu, incl, 31), s_warp, before, total);
        unsigned above = before + incl - mine;
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

    // A thread takes kKeys consecutive rows of a round as bit masks, above theta and equal
    // to it; their numbers packed into one word for the prefix over the block.
    unsigned gt = 0, is = 0, before = 0, total = 0;
    auto classify = [&](int r0) {
        const int i0 = tid * kKeys, m = min(kRound, hi - r0) - i0;
        gt = is = 0;
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
            const unsigned key = s_key[key_at(i0 + q)];
            if (q < m && key > theta) gt |= 1u << q;
            if (q < m && key == theta) is |= 1u << q;
        }
        const unsigned mine = (unsigned)__popc(gt) | (unsigned)__popc(is) << 16;
        unsigned incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        warp_prefix<kT>(__shfl_sync(0xffffffffu, incl, 31), s_warp, before, total);
        before += incl - mine;
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
        // equal rows still wanted when this round begins, and when this thread's do
        const unsigned left = need > eq ? need - eq : 0u;
        const unsigned eq_before = before >> 16;
        unsigned dst = at + (before & 0xffffu) + min(eq_before, left);
        unsigned want = left > eq_before ? left - eq_before : 0u;
        unsigned todo = gt | is;
        while (todo) {
            const int q = __ffs(todo) - 1;
            todo &= todo - 1;
            if (is >> q & 1u) {
                if (want == 0) continue;
                --want;
            }
            if (dst < k) out[first + dst] = r0 + tid * kKeys + q;
            ++dst;
        }
        at += (total & 0xffffu) + min(total >> 16, left);
        eq += total >> 16;
    }
    if constexpr (kCluster > 1) sync_all();       // no block leaves while its counts are read
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

template <int kT, int kKeys, int kCluster>
cudaError_t launch_select(const DevPaged &S, const DevPaged &Q, const EvictArgs &A,
                          cudaStream_t s) {
    constexpr int kSmem = (kT * kKeys + kT * kKeys / 32 + kT) * 4;   // keys, a word a thread
    static_assert(kT * kKeys <= 32768, "counts of a round are 16-bit");
    auto kernel = evict_select_kernel<kT, kKeys, kCluster>;
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
    cudaError_t e = S.cap <= 4096    ? launch_select<256, 16, 1>(S, D, A, s)
                    : S.cap <= 16384 ? launch_select<512, 32, 1>(S, D, A, s)
                                     : launch_select<512, 32, 8>(S, D, A, s);
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
