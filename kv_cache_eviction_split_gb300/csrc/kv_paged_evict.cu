// kv_paged_evict.cu -- eviction by accumulated attention weight.
//
// select: per unit with n rows and budget b < n, theta = the k-th largest weight
// of the rows between the pinned ones (k = b - sinks - recent), by radix select
// on the fp32 bit patterns, and the kept rows in order: those above theta, and of
// those equal to it the first ones.  gather: kept row i of src becomes row i of dst.
#include "kv_compact.cuh"
#include "kv_paged.cuh"
#include "kv_select.cuh"

namespace kvevict {
namespace {

constexpr int kSelT = 1024;
constexpr int kSelPer = 8;     // rows a thread holds in the ordered pass

// Bit pattern of the weight of row j (0 for a page that does not exist, posted).
__device__ __forceinline__ unsigned mass_key(const DevPaged &S, const int32_t *tab, int j,
                                             int *status) {
    const long long row = page_row(S, tab, j);
    if (row < 0) {
        post_status(status, KV_ERR_INVALID_ARG);
        return 0u;
    }
    return __float_as_uint(S.mass[row]);
}

__global__ void __launch_bounds__(kSelT)
evict_select_kernel(const DevPaged S, const DevPaged D, const int32_t *__restrict__ budgets,
                    int sinks, int recent, int32_t *__restrict__ kept, long long kept_stride,
                    int *status) {
    __shared__ unsigned hist[256], warp_sums[32], scalars[2];
    const int tid = threadIdx.x;
    const long long u = blockIdx.x;
    int n;
    const bool len_ok = unit_len(S, u, n);
    const long long b = budgets[u];
    const long long keep = b < n ? b : n;
    if (!len_ok || b < (long long)sinks + recent || keep > kept_stride || keep > D.cap) {
        if (tid == 0) {
            post_status(status, len_ok ? KV_ERR_BUDGET : KV_ERR_INVALID_ARG);
            D.lens[u] = -1;
        }
        return;
    }
    if (tid == 0) D.lens[u] = (int)keep;
    int32_t *out = kept + u * kept_stride;
    if (n <= b) {
        for (int j = tid; j < n; j += kSelT) out[j] = j;
        return;
    }
    for (int j = tid; j < sinks; j += kSelT) out[j] = j;
    for (int j = tid; j < recent; j += kSelT) out[b - recent + j] = n - recent + j;
    const int lo = sinks, hi = n - recent;
    const unsigned k = (unsigned)(b - sinks - recent);
    if (k == 0) return;
    const int32_t *tab = S.table + u * S.max_pages;
    unsigned prefix = 0, mask = 0, remaining = k;
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int i = tid; i < 256; i += kSelT) hist[i] = 0;
        __syncthreads();
        for (int j = lo + tid; j < hi; j += kSelT) {
            const unsigned key = mass_key(S, tab, j, status);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
        }
        __syncthreads();
        const unsigned h = tid < 256 ? hist[255 - tid] : 0u;
        unsigned tot;
        const unsigned excl = sel_block_scan<kSelT>(h, warp_sums, &tot);
        if (tid < 256 && excl + h >= remaining && excl < remaining) {
            scalars[0] = 255u - tid;
            scalars[1] = excl;
        }
        __syncthreads();
        remaining -= scalars[1];
        prefix |= scalars[0] << shift;
        mask |= 255u << shift;
        __syncthreads();
    }
    const unsigned theta = prefix, need_eq = remaining;
    unsigned base = 0, eq_seen = 0;
    for (int c0 = lo; c0 < hi; c0 += kSelT * kSelPer) {
        unsigned key[kSelPer], n_eq = 0;
#pragma unroll
        for (int i = 0; i < kSelPer; ++i) {
            const int j = c0 + tid * kSelPer + i;
            key[i] = j < hi ? mass_key(S, tab, j, status) : 0u;
            n_eq += j < hi && key[i] == theta;
        }
        unsigned eq_total, keep_total, bits = 0;
        unsigned rank = eq_seen + sel_block_scan<kSelT>(n_eq, warp_sums, &eq_total);
#pragma unroll
        for (int i = 0; i < kSelPer; ++i) {
            const int j = c0 + tid * kSelPer + i;
            if (j >= hi) break;
            bool take = key[i] > theta;
            if (key[i] == theta) take = rank++ < need_eq;
            bits |= (unsigned)take << i;
        }
        unsigned at = base + sel_block_scan<kSelT>(__popc(bits), warp_sums, &keep_total);
#pragma unroll
        for (int i = 0; i < kSelPer; ++i)
            if (bits >> i & 1u) {
                if (at < k) out[sinks + at] = c0 + tid * kSelPer + i;
                ++at;
            }
        base += keep_total;
        eq_seen += eq_total;
    }
}

constexpr int kWarps = 8;
constexpr int kUnroll = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
evict_gather_kernel(const DevPaged S, const DevPaged Q, const int32_t *__restrict__ kept,
                    long long kept_stride, int *status) {
    constexpr int kVecs = D / 8, kLanes = 2 * kVecs, kRows = 32 / kLanes, kStep = kWarps * kRows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = (lane % kLanes) / kVecs, ch = lane % kVecs;
    const long long u = blockIdx.y;
    const int n = Q.lens[u];
    const int i0 = blockIdx.x * kStep * kUnroll + warp * kRows + lane / kLanes;
    if (i0 >= n) return;
    const int32_t *from = S.table + u * S.max_pages, *to = Q.table + u * Q.max_pages;
    const uint4 *src = static_cast<const uint4 *>(which ? S.v : S.k);
    uint4 *dst = static_cast<uint4 *>(which ? Q.v : Q.k);
    long long a[kUnroll], z[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
        const int i = i0 + q * kStep;
        a[q] = i < n ? page_row(S, from, kept[u * kept_stride + i]) : -1;
        z[q] = i < n ? page_row(Q, to, i) : -1;
        if (i < n && (a[q] < 0 || z[q] < 0)) {
            post_status(status, KV_ERR_INVALID_ARG);
            a[q] = -1;
        }
    }
    uint4 buf[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q)
        if (a[q] >= 0) buf[q] = ld_nc(src + a[q] * kVecs + ch);
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
        if (a[q] < 0) continue;
        st_cs(dst + z[q] * kVecs + ch, buf[q]);
        if (Q.mass && which == 0 && ch == 0) Q.mass[z[q]] = S.mass[a[q]];
    }
}

}  // namespace

cudaError_t launch_paged_evict(const DevPaged &S, const DevPaged &D, const int32_t *budgets,
                               int sinks, int recent, int32_t *kept, long long kept_stride,
                               int *status, cudaStream_t s) {
    evict_select_kernel<<<(unsigned)S.units, kSelT, 0, s>>>(S, D, budgets, sinks, recent, kept,
                                                            kept_stride, status);
    const int rows = kWarps * kUnroll * (S.d == 64 ? 2 : 1);
    const long long most = kept_stride < D.cap ? kept_stride : D.cap;
    for (long long u0 = 0; u0 < S.units; u0 += 65535) {
        // grid.y is limited to 65535 units a launch
        DevPaged s1 = S, d1 = D;
        s1.table += u0 * S.max_pages;
        s1.lens += u0;
        d1.table += u0 * D.max_pages;
        d1.lens += u0;
        const dim3 grid((unsigned)((most + rows - 1) / rows),
                        (unsigned)(S.units - u0 < 65535 ? S.units - u0 : 65535));
        if (S.d == 64)
            evict_gather_kernel<64><<<grid, kWarps * 32, 0, s>>>(s1, d1, kept + u0 * kept_stride,
                                                                 kept_stride, status);
        else
            evict_gather_kernel<128><<<grid, kWarps * 32, 0, s>>>(s1, d1, kept + u0 * kept_stride,
                                                                  kept_stride, status);
    }
    return cudaGetLastError();
}

}  // namespace kvevict
