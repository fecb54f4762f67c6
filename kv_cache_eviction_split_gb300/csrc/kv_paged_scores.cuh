// kv_paged_scores.cuh -- attention scores that are changed before the softmax, and the rows that
// queries see by position, as the kernels see them (not part of the ABI).
//
// Of a product s = q.k and softmax scale c, in units of log2:
//   z = c s, or cap tanh(c s / cap);  z - slope_h |p_q - p_j|
// tanh(x) = 1 - 2 / (1 + e^2x): two approximate operations, off by a few 2^-23 of cap, which is
// what counts in an exponent.
#pragma once
#include "kv_paged_attend.cuh"

namespace kvevict {

constexpr float kLog2e = 1.4426950408889634f;

// Rows lo .. hi of a unit, those a query sees beside the sinks; hi < 0: none.
struct RowBounds {
    int lo, hi;
};
// Of 128 query rows of a unit: the least lo and greatest hi of rows that see any, then the
// greatest lo and least hi.
struct BlockBounds {
    int lo, hi, lo_all, hi_all;
};
constexpr int kNoLo = 0x3fffffff;          // lo of a query that sees nothing

struct ScoreForm {
    float cap2, cap_u;         // cap log2(e), 0: none; 2 c log2(e) / cap, the exponent of e^2x
    const float *slopes;       // [Hq], or null
    const int32_t *pos;        // positions of pool rows, or null: a row's number; null without slopes
    const RowBounds *rows;     // [tokens][H], or null: up to the query's own row, and the window
    const BlockBounds *blocks; // [R * H][unit_blocks], with rows
    int unit_blocks;
};

// z without the distance, in units of log2.
__device__ __forceinline__ float form_logit(const ScoreForm &F, float scale_log2, float s) {
    if (F.cap2 == 0.f) return s * scale_log2;
    const float e = sm100::ex2_approx(fminf(s * F.cap_u, 64.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return fmaf(-2.f * F.cap2, r, F.cap2);
}

// Rows that query i of a request's chunk sees of unit U.
__device__ __forceinline__ RowBounds row_bounds(const DevPaged &C, const AttendMask &M,
                                                const ScoreForm &F, const UnitRows &U, int i) {
    if (F.rows) return F.rows[(U.tok0 + i) * C.H + U.h];
    const int t = U.n - U.count + i;
    return RowBounds{window_lo(M, max(t, 0)), t};
}

// As tile_span, of the rows from lo (or below the sinks) to hi that any query sees.
__device__ __forceinline__ TileSpan bounds_span(const AttendMask &M, int lo, int hi, int log2) {
    TileSpan s{0, 0, 1};
    if (hi < 0) return s;
    const int sinks = min(M.sinks, lo);
    s.first = lo >> log2;
    s.ns = min((sinks + (1 << log2) - 1) >> log2, s.first);
    s.total = s.ns + (hi >> log2) + 1 - s.first;
    return s;
}

// Position of cache row t of unit U (0 where its page does not exist).
__device__ __forceinline__ int position_of(const DevPaged &C, const ScoreForm &F, const UnitRows &U,
                                           int t) {
    const long long row = t >= 0 && t < C.cap ? page_row(C, U.table, t) : -1;
    return row >= 0 ? F.pos[row] : 0;
}

// Copies `bytes` (a multiple of 16) of global memory into shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            sm100::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
        : "memory");
}

// What a caller gives: the bounds in positions, which become rows.
struct ScoreBounds {
    const int32_t *pos;            // positions of pool rows, or null
    const int32_t *first, *last;   // [tokens], or null
};
cudaError_t launch_row_bounds(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                              const ScoreBounds &B, RowBounds *rows, BlockBounds *blocks,
                              int unit_blocks, cudaStream_t s);

cudaError_t launch_attend_few_scored(const DevPaged &C, const DevChunk &T, int layer,
                                     const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                     bool add_mass, long long seen, long long items, int max_rows,
                                     int blocks, const AttendWs &ws, cudaStream_t s);
cudaError_t launch_attend_many_scored(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s);
// kv_paged_attention with changed scores (form.rows and form.blocks are filled in).
cudaError_t launch_paged_attention_scored(const DevPaged &C, const DevChunk &T, int layer,
                                          const AttendMask &M, const ScoreForm &form,
                                          const ScoreBounds &bounds, const AttendIo &io,
                                          bool add_mass, const AttendWs &ws, cudaStream_t s);

}  // namespace kvevict
