// kv_paged_many_scored.cu -- the many-rows kernel (kv_paged_many.cu) with scores capped, lowered by
// distance, or masked by rows of their own, and the rows that queries see from the positions that
// a caller gives.
#include "kv_paged_many.cuh"

namespace kvevict {
namespace {

constexpr int kBoundThreads = 128;

// How many of the unit's first n rows lie at positions below `key` (positions never fall from a
// row to the next).  A thread by itself, seven probes at a time, or a warp, 32.
template <bool kWarp>
__device__ __forceinline__ int rows_below(const DevPaged &C, const int32_t *pos,
                                          const int32_t *table, int n, long long key) {
    if (!pos) return (int)max(0ll, min((long long)n, key));
    auto less = [&](int j) {
        const long long row = page_row(C, table, j);
        return row >= 0 && pos[row] < key;
    };
    int a = 0, b = n;
    while (a < b) {
        int c = 0;
        if constexpr (kWarp) {
            const int step = (b - a + 31) / 32, j = a + ((int)(threadIdx.x & 31) + 1) * step - 1;
            c = __popc(__ballot_sync(0xffffffffu, j < b && less(j)));
            const int next = a + (c + 1) * step - 1;
            a += c * step;
            if (c < 32 && next < b) b = next;
            a = min(a, b);
        } else {
            const int step = (b - a + 7) / 8;
#pragma unroll
            for (int k = 1; k < 8; ++k) {
                const int j = a + k * step - 1;
                c += j < b && less(j);
            }
            const int next = a + (c + 1) * step - 1;
            a += c * step;
            if (c < 7 && next < b) b = next;
            a = min(a, b);
        }
    }
    return a;
}

// The rows that a unit's queries see, 128 query rows (row i * G + g) to a block, and what those of a
// block see together.
__global__ void __launch_bounds__(kBoundThreads)
row_bounds_kernel(const DevPaged C, const DevChunk T, int layer, const AttendMask M,
                  const ScoreBounds B, RowBounds *rows, BlockBounds *blocks, int unit_blocks) {
    __shared__ int s_found[2 * 8];
    __shared__ int s_min[4][kBoundThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long all = (long long)C.R * C.H * unit_blocks;
    for (long long at = blockIdx.x; at < all; at += gridDim.x) {
        const int v = (int)(at / unit_blocks), blk = (int)(at - (long long)v * unit_blocks);
        const UnitRows U = unit_rows(C, T, layer, v);
        const int most = U.count * C.G, row0 = blk * 128;
        if (row0 >= most) continue;
        const int i0 = row0 / C.G, n_tok = (min(most, row0 + 128) - 1) / C.G - i0 + 1;
        // few tokens: a warp a search
        const bool by_warp = n_tok <= 8;
        if (by_warp) {
            for (int k = warp; k < 2 * n_tok; k += kBoundThreads / 32) {
                const long long tok = U.tok0 + i0 + (k >> 1);
                const int32_t *bound = k & 1 ? B.last : B.first;
                if (!bound) continue;
                const int f = rows_below<true>(C, B.pos, U.table, U.n,
                                               (long long)bound[tok] + (k & 1));
                if (lane == 0) s_found[k] = f;
            }
            __syncthreads();
        }
        RowBounds r{kNoLo, -1};
        bool some = false;
        if (threadIdx.x < n_tok) {
            const int i = i0 + threadIdx.x, t = U.n - U.count + i;
            const long long tok = U.tok0 + i;
            if (t >= 0) {
                r.lo = window_lo(M, t);
                r.hi = t;
                if (B.first)
                    r.lo = max(r.lo, by_warp ? s_found[2 * threadIdx.x]
                                             : rows_below<false>(C, B.pos, U.table, U.n, B.first[tok]));
                if (B.last)
                    r.hi = (by_warp ? s_found[2 * threadIdx.x + 1]
                                    : rows_below<false>(C, B.pos, U.table, U.n,
                                                        (long long)B.last[tok] + 1)) - 1;
                if (r.hi < 0 || (r.lo > r.hi && M.sinks == 0)) r = RowBounds{kNoLo, -1};
                else if (r.lo > r.hi) r.lo = r.hi + 1;
            }
            some = r.hi >= 0;
            rows[tok * C.H + U.h] = r;
        }
        // of the threads with a token: least lo, greatest hi, greatest lo, least hi
        const bool on = threadIdx.x < n_tok;
        const int m[4] = {__reduce_min_sync(0xffffffffu, some ? r.lo : kNoLo),
                          __reduce_max_sync(0xffffffffu, some ? r.hi : -1),
                          __reduce_max_sync(0xffffffffu, on ? r.lo : 0),
                          __reduce_min_sync(0xffffffffu, on ? r.hi : 0x7fffffff)};
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < 4; ++k) s_min[k][warp] = m[k];
        __syncthreads();
        if (threadIdx.x == 0 && blocks) {
            BlockBounds b{kNoLo, -1, 0, 0x7fffffff};
#pragma unroll
            for (int w = 0; w < kBoundThreads / 32; ++w) {
                b.lo = min(b.lo, s_min[0][w]);
                b.hi = max(b.hi, s_min[1][w]);
                b.lo_all = max(b.lo_all, s_min[2][w]);
                b.hi_all = min(b.hi_all, s_min[3][w]);
            }
            blocks[at] = b;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_row_bounds(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                              const ScoreBounds &B, RowBounds *rows, BlockBounds *blocks,
                              int unit_blocks, cudaStream_t s) {
    const long long all = (long long)C.R * C.H * unit_blocks;
    const unsigned grid = (unsigned)(all < (1 << 20) ? all : 1 << 20);
    return launch_dependent(row_bounds_kernel, dim3(grid), kBoundThreads, 0, s, C, T, layer, M, B, rows,
                            blocks, unit_blocks);
}

cudaError_t launch_attend_many_scored(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s) {
    if (form.cap2 != 0.f) return launch_attend_many_capped(C, T, layer, M, form, io, ws, s);
    if (form.slopes) return launch_attend_many_sloped(C, T, layer, M, form, io, ws, s);
    return attend_many<kBounds>(C, T, layer, M, form, io, ws, s);
}

}  // namespace kvevict
