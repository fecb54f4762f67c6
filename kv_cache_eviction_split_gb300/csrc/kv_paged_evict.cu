// kv_paged_evict.cu -- eviction by accumulated attention weight.
//
// select: per unit with n rows and budget b < n, theta = the k-th largest weight of the
// rows between the pinned ones (k = b - sinks - recent), by a radix select on the fp32
// bit patterns, and the kept rows in order: those above theta, and of those equal to it
// the first ones.  gather: kept row i of src becomes row i of dst.
//
// The weights are read once: a unit's rows are spread over the registers of a block or of
// a cluster of 8 (kKeys a thread, warps holding consecutive rows), and the three digit
// passes (11, 11 and 10 bits) count from there, the cluster's counts added through
// distributed shared memory.  The first version re-read the weights through the page
// table in every pass with one block a unit: 247 us for 112 units of 131072 rows, bound by
// the latency of its two dependent loads.
#include <cooperative_groups.h>

#include "kv_compact.cuh"
#include "kv_paged_attend.cuh"

namespace kvevict {
namespace {
namespace cg = cooperative_groups;

constexpr int kKeys = 16;        // rows a thread holds
constexpr int kBins = 2048;      // digits of 11, 11 and 10 bits

struct EvictArgs {
    const int32_t *budgets;
    int sinks, recent;
    int32_t *kept;
    long long kept_stride;
    int *status;
};

// Bit pattern of the weight of row j (0 for a page that does not exist, posted).
__device__ __forceinline__ unsigned mass_key(const DevPaged &S, const int32_t *tab, int j,
                                             int *status) {
    const long long row = page_row(S, tab, j);
    if (row < 0) {
        post_status(status, KV_ERR_INVALID_ARG);
        return 0u;
    }
    return __float_as_uint(__ldg(S.mass + row));
}

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

// One unit by a block of kT threads (kCluster = 1) or a cluster of such blocks.  Rows are
// dealt to blocks in equal consecutive slices; a slice longer than kT * kKeys rows is
// walked in rounds of that many, re-read in every pass.
template <int kT, int kCluster>
__global__ void __launch_bounds__(kT)
evict_select_kernel(const DevPaged S, const DevPaged D, const EvictArgs A) {
    __shared__ unsigned hist[kBins];
    __shared__ unsigned sums[kCluster > 1 ? kBins : 1];
    __shared__ unsigned s_warp[32], s_pick[2], s_counts[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kCluster > 1 ? (int)(blockIdx.x % kCluster) : 0;
    const long long u = blockIdx.x / kCluster;
    auto sync_all = [&]() {
        if constexpr (kCluster > 1) cg::this_cluster().sync();
        else __syncthreads();
    };
    pdl_wait();
    pdl_trigger();
    int n;
    const bool len_ok = unit_len(S, u, n);
    const long long b = A.budgets[u];
    const long long keep = b < n ? b : n;
    if (!len_ok || b < (long long)A.sinks + A.recent || keep > A.kept_stride || keep > D.cap) {
        if (rank == 0 && tid == 0) {
            post_status(A.status, len_ok ? KV_ERR_BUDGET : KV_ERR_INVALID_ARG);
            D.lens[u] = -1;
        }
        return;                                   // the same in every block of the cluster
    }
    if (rank == 0 && tid == 0) D.lens[u] = (int)keep;
    int32_t *out = A.kept + u * A.kept_stride;
    const int all = kT * kCluster, me = rank * kT + tid;
    if (n <= b) {
        for (int j = me; j < n; j += all) out[j] = j;
        return;
    }
    for (int j = me; j < A.sinks; j += all) out[j] = j;
    for (int j = me; j < A.recent; j += all) out[b - A.recent + j] = n - A.recent + j;
    const unsigned k = (unsigned)(b - A.sinks - A.recent);
    if (k == 0) return;

    // this block's slice [lo, hi) of the rows between the pinned ones
    const int first = A.sinks, rows = n - A.recent - first;
    const int slice = ((rows + kCluster - 1) / kCluster + 31) / 32 * 32;
    const int lo = first + min(rows, rank * slice), hi = first + min(rows, (rank + 1) * slice);
    const int32_t *tab = S.table + u * S.max_pages;
    constexpr int kRound = kT * kKeys;
    const bool held = hi - lo <= kRound;          // one round: the keys stay in registers
    unsigned key[kKeys];
    // row of key q of this thread in the round that starts at r0
    auto row_of = [&](int r0, int q) { return r0 + (warp * kKeys + q) * 32 + lane; };
    auto load = [&](int r0) {
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
            const int j = row_of(r0, q);
            key[q] = j < hi ? mass_key(S, tab, j, A.status) : 0u;
        }
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
#pragma unroll
            for (int q = 0; q < kKeys; ++q)
                if (row_of(r0, q) < hi && (key[q] & mask) == prefix)
                    atomicAdd(&hist[key[q] >> shift & digit], 1u);
        }
        sync_all();
        const unsigned *count = hist;
        if constexpr (kCluster > 1) {
            for (int i = tid; i < kBins; i += kT) {
                unsigned x = 0;
#pragma unroll
                for (int r = 0; r < kCluster; ++r)
                    x += *cg::this_cluster().map_shared_rank(&hist[i], r);
                sums[i] = x;
            }
            count = sums;
            sync_all();                           // every block has read before hist is cleared
        }
        // digits from the top: the bin where the running count reaches `remaining`
        constexpr int kPer = kBins / kT;          // bins a thread sums, highest first
        unsigned x[kPer], mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine += x[i] = count[kBins - 1 - (tid * kPer + i)];
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
                s_pick[0] = kBins - 1 - (tid * kPer + i);
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

    // keys above theta and equal to it in this slice, then in the slices before it
    unsigned above = 0, equal = 0;
    for (int r0 = lo; r0 < hi; r0 += kRound) {
        if (!held) load(r0);
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
            const bool in = row_of(r0, q) < hi;
            above += in && key[q] > theta;
            equal += in && key[q] == theta;
        }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    unsigned x0, x1, in_block[2];
    warp_prefix<kT>(above, s_warp, x0, in_block[0]);
    warp_prefix<kT>(equal, s_warp, x1, in_block[1]);
    unsigned at = 0, eq = 0;                      // kept and equal rows before this block
    if constexpr (kCluster > 1) {
        if (tid < 2) s_counts[tid] = in_block[tid];
        sync_all();
        unsigned gt = 0;
        for (int r = 0; r < rank; ++r) {
            const unsigned *c = cg::this_cluster().map_shared_rank(s_counts, r);
            gt += c[0];
            eq += c[1];
        }
        at = gt + min(eq, need);
        sync_all();                               // no block leaves while its counts are read
    }
    for (int r0 = lo; r0 < hi; r0 += kRound) {
        if (!held) load(r0);
        unsigned n_eq = 0;
#pragma unroll
        for (int q = 0; q < kKeys; ++q)
            n_eq += __popc(__ballot_sync(0xffffffffu, row_of(r0, q) < hi && key[q] == theta));
        unsigned eq_before, eq_total, before, total, bits = 0, kept_n = 0;
        warp_prefix<kT>(n_eq, s_warp, eq_before, eq_total);
        unsigned seen = eq + eq_before;
        const unsigned lower = (1u << lane) - 1u;
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
            const bool in = row_of(r0, q) < hi, is = in && key[q] == theta;
            const unsigned e = __ballot_sync(0xffffffffu, is);
            const bool take = in && (key[q] > theta || (is && seen + __popc(e & lower) < need));
            seen += __popc(e);
            bits |= (unsigned)take << q;
            kept_n += __popc(__ballot_sync(0xffffffffu, take));
        }
        warp_prefix<kT>(kept_n, s_warp, before, total);
        unsigned to = at + before;
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
            const bool take = bits >> q & 1u;
            const unsigned t = __ballot_sync(0xffffffffu, take);
            const unsigned i = to + __popc(t & lower);
            if (take && i < k) out[first + i] = row_of(r0, q);
            to += __popc(t);
        }
        at += total;
        eq += eq_total;
    }
}

// A warp moves 32 consecutive kept rows: each lane looks up one row's two places (kept
// index, page table), then the warp copies the rows in batches of kBatch with all their
// loads in flight, K and V of a row (or of two, d = 64) side by side over its lanes.
constexpr int kWarps = 8;
constexpr int kBatch = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
evict_gather_kernel(const DevPaged S, const DevPaged Q, const EvictArgs A, long long u0) {
    constexpr int kVecs = D / 8, kLanes = 2 * kVecs, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / kLanes, which = (lane % kLanes) / kVecs, ch = lane % kVecs;
    pdl_wait();
    pdl_trigger();
    const long long u = u0 + blockIdx.y;
    const int n = Q.lens[u];
    const int i0 = (blockIdx.x * kWarps + warp) * 32;
    if (i0 >= n) return;
    const uint4 *src = static_cast<const uint4 *>(which ? S.v : S.k);
    uint4 *dst = static_cast<uint4 *>(which ? Q.v : Q.k);
    long long from = -1, to = -1;
    if (i0 + lane < n) {
        const int j = A.kept[u * A.kept_stride + i0 + lane];
        from = page_row(S, S.table + u * S.max_pages, j);
        to = page_row(Q, Q.table + u * Q.max_pages, i0 + lane);
        if (from < 0 || to < 0) {
            post_status(A.status, KV_ERR_INVALID_ARG);
            from = -1;
        } else if (Q.mass) {
            Q.mass[to] = S.mass[from];
        }
    }
#pragma unroll 1
    for (int r0 = 0; r0 < 32 && i0 + r0 < n; r0 += kBatch * kRows) {
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

template <int kT, int kCluster>
cudaError_t launch_select(const DevPaged &S, const DevPaged &D, const EvictArgs &A,
                          cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(S.units * kCluster));
    cfg.blockDim = dim3(kT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = kCluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<kT, kCluster>, S, D, A);
}

}  // namespace

cudaError_t launch_paged_evict(const DevPaged &S, const DevPaged &D, const int32_t *budgets,
                               int sinks, int recent, int32_t *kept, long long kept_stride,
                               int *status, cudaStream_t s) {
    const EvictArgs A{budgets, sinks, recent, kept, kept_stride, status};
    // the smallest shape that holds the longest possible unit in registers
    cudaError_t e = S.cap <= 256 * kKeys     ? launch_select<256, 1>(S, D, A, s)
                    : S.cap <= 1024 * kKeys ? launch_select<1024, 1>(S, D, A, s)
                                            : launch_select<1024, 8>(S, D, A, s);
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
