// kv_paged.cuh -- the paged cache as the kernels see it (not part of the ABI).
//
// Cache row j of unit u is pool row page_table[u][j / ps] * ps + j % ps.  Page
// indices come from device memory, so every kernel checks them before use
// (page_row): an index outside [0, num_pages) is not followed.
#pragma once

#include "kv_internal.cuh"

namespace kvevict {

struct DevPaged {
    int R, L, H, Hq, G, d;
    int ps, ps_log2;           // rows per page, a power of two
    int max_pages, cap;        // table columns; cap = max_pages * ps rows
    int dtype;                 // kv_dtype
    long long num_pages, units;
    const int32_t *table;      // [units][max_pages]
    int32_t *lens;             // [units]
    void *k, *v;               // [num_pages][ps][d]
    float *mass;               // [num_pages][ps] or null
};

// The new tokens of a step.
struct DevChunk {
    const long long *off;      // device [R + 1]
    const long long *host_off; // host copy (host code only)
    long long tokens;          // off[R]
    int max_t;                 // most new tokens of one request
};

// Which cache rows a query sees, and the scale of its logits.
struct AttendMask {
    int window, sinks;         // window 0: every row up to the query's own
    float scale_log2;          // softmax_scale * log2(e)
};

// Rows that unit u holds; false (and 0) when the length is not one a table can hold.
__device__ __forceinline__ bool unit_len(const DevPaged &C, long long u, int &n) {
    n = C.lens[u];
    const bool ok = n >= 0 && n <= C.cap;
    n = ok ? n : 0;
    return ok;
}

// Pool row of cache row j of the unit whose table is `tab`; -1 if its page does not exist.
__device__ __forceinline__ long long page_row(const DevPaged &C, const int32_t *tab, int j) {
    const int page = tab[j >> C.ps_log2];
    if (page < 0 || page >= C.num_pages) return -1;
    return ((long long)page << C.ps_log2) + (j & (C.ps - 1));
}

// Request of token `tok`: the r with off[r] <= tok < off[r + 1].
__device__ __forceinline__ int request_of(const DevChunk &T, int R, long long tok) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (T.off[mid] <= tok) lo = mid; else hi = mid;
    }
    return lo;
}

// First row of the sliding window of a query at row t (0 without a window).
__host__ __device__ __forceinline__ int window_lo(const AttendMask &M, int t) {
    return M.window > 0 && t - M.window + 1 > 0 ? t - M.window + 1 : 0;
}

cudaError_t launch_paged_append(const DevPaged &C, const DevChunk &T, int layer, const void *k_new,
                                long long k_stride, const void *v_new, long long v_stride,
                                cudaStream_t s);
cudaError_t launch_paged_load(const DevPaged &C, const void *k_rows, const void *v_rows,
                              const float *mass_rows, const int64_t *offsets, long long total_rows,
                              cudaStream_t s);
cudaError_t launch_paged_evict(const DevPaged &S, const DevPaged &D, const int32_t *budgets,
                               int sinks, int recent, int32_t *kept, long long kept_stride,
                               int *status, cudaStream_t s);

// Workspace of the attention (all offsets 256-byte aligned).
struct AttendWs {
    int *status;
    float *lse2;               // [tokens][Hq] log2 of the softmax sums, for the mass pass
    size_t total;
};
AttendWs attend_ws_layout(const DevPaged &C, const DevChunk &T, bool add_mass, void *base);

struct AttendIo {
    const void *q;
    void *out;
    float *lse;                // or null
    long long q_stride, out_stride;
};
cudaError_t launch_paged_attention(const DevPaged &C, const DevChunk &T, int layer,
                                   const AttendMask &M, const AttendIo &io, bool add_mass,
                                   const AttendWs &ws, cudaStream_t s);

}  // namespace kvevict
