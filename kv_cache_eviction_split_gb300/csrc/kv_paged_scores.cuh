// kv_paged_scores.cuh -- attention scores that are changed before the softmax, and the rows that
// queries see by position, as the kernels see them (not part of the ABI).
//
// Of a product s = q.k and softmax scale c, in units of log2:
//   z = c s, or cap tanh(c s / cap);  z - slope_h |p_q - p_j|
// tanh(x) = 1 - 2 / (1 + e^2x): two approximate operations, off by a few 2^-23 of 1.  For |x| < 1/4,
// where that is more and more of tanh(x), its series, so that a capped logit is off by a few 2^-21 of
// itself however large the cap.  (The many-rows kernel takes small ones by polynomials, and goes
// without the series in the exact form, which it would slow by a fifth to a half.)
#pragma once
#include <algorithm>
#include <cfloat>
#include <cmath>

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
    float cap2;                // cap log2(e), 0: none
    float cap_u;               // 2 c log2(e) / cap: s to the exponent of e^2x, x = c s / cap
    float cap_x;               // c / cap: s to x
    float cap_z;               // c log2(e): s to what it is without a cap
    float slope_s;             // 1 / c: a slope in units of s
    int two_way;               // whether a query may see keys behind it
    const float *slopes;       // [Hq], or null
    const int32_t *pos;        // positions of pool rows, or null: a row's number; null without slopes
    const RowBounds *rows;     // [tokens][H], or null: up to the query's own row, and the window
    const BlockBounds *blocks; // [R * H][unit_blocks], with rows
    int unit_blocks;
    // cap2 tanh(x) = s (c0 + c1 s^2 + ...) with x = cap_x s, for two logits at a time, where |s| is at
    // most most4 (|x| <= 1/2) and most5 (|x| <= 3/4): fitted in x with the largest error of tanh
    // least, 1.6e-7 and 2.5e-7 in fp32 (the exact form's 1 has steps of 1.2e-7).  Below 0: never.
    float most4, most5;
    float2 co4[4], co5[5];

    void set_cap(float cap, float scale) {
        constexpr double k4[4] = {0.9999976754188538, -0.33320656418800354, 0.1314515471458435,
                                  -0.043372705578804016};
        constexpr double k5[5] = {0.9999972581863403, -0.33323076367378235, 0.13226093351840973,
                                  -0.04928047955036163, 0.012318850494921207};
        const double x = (double)scale / cap, most = (double)cap * kLog2e;
        cap2 = (float)most;
        // finite, so that a logit of 0 stays 0 with the smallest caps
        cap_u = (float)std::min(2.0 * x * kLog2e, (double)FLT_MAX);
        cap_x = (float)std::min(x, (double)FLT_MAX);
        cap_z = (float)((double)scale * kLog2e);
        // caps far above c: smaller x, where the terms that fp32 has not are of no account; and s^2
        // stays finite
        double power = x * most;
        auto has = [&](int i) { return power * std::pow(x, 2 * i) > 1e-35; };
        const double part = has(2) ? 1.0 / 8 : has(1) ? 1.0 / 64 : 1.0 / 4096;
        most4 = x <= 4096 ? (float)std::min((has(3) ? 0.5 : part) / x, 1e18) : -1.0f;
        most5 = x <= 4096 ? (float)std::min((has(4) ? 0.75 : has(3) ? 0.25 : part) / x, 1e18) : -1.0f;
        for (int i = 0; i < 5; ++i, power *= x * x) {
            if (i < 4) co4[i] = make_float2((float)(k4[i] * power), (float)(k4[i] * power));
            co5[i] = make_float2((float)(k5[i] * power), (float)(k5[i] * power));
        }
    }
};

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The smaller of two, NaN if one is: fminf would make a bound of a logit of NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Capped, in units of log2.  The series up to x^9: what it leaves out is 9e-9 of tanh(1/4).
__device__ __forceinline__ float cap_logit(const ScoreForm &F, float s) {
    const float e = sm100::ex2_approx(min_nan(s * F.cap_u, 64.f));
    const float z1 = fmaf(-2.f * F.cap2, rcp_approx(1.f + e), F.cap2);
    const float x = s * F.cap_x, x2 = x * x;
    float t = fmaf(x2, 62.f / 2835, -17.f / 315);
    t = fmaf(x2, t, 2.f / 15);
    t = fmaf(x2, t, -1.f / 3);
    const float z = s * F.cap_z;
    return fabsf(x) < 0.25f ? fmaf(z * x2, t, z) : z1;
}

// Two logits without the series, by one reciprocal of both denominators: three products on units
// that have time for them save one of five operations on the one that has none.  NaN in one makes both
// NaN: logits behind keys that the row does not see are set to something else before.
__device__ __forceinline__ float2 cap_pair(const ScoreForm &F, float2 s) {
    const float a = 1.f + sm100::ex2_approx(min_nan(s.x * F.cap_u, 60.f));
    const float b = 1.f + sm100::ex2_approx(min_nan(s.y * F.cap_u, 60.f));
    const float r = rcp_approx(a * b);
    return make_float2(fmaf(-2.f * F.cap2, r * b, F.cap2), fmaf(-2.f * F.cap2, r * a, F.cap2));
}

// The same of one logit of at most most5 by the polynomial: a shorter chain of operations.
__device__ __forceinline__ float cap_poly1(const ScoreForm &F, float s) {
    const float s2 = s * s;
    float t = F.co5[4].x;
#pragma unroll
    for (int i = 3; i >= 0; --i) t = fmaf(t, s2, F.co5[i].x);
    return t * s;
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
cudaError_t launch_attend_many_capped(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s);
cudaError_t launch_attend_many_sloped(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s);
// kv_paged_attention with changed scores (form.rows and form.blocks are filled in).
cudaError_t launch_paged_attention_scored(const DevPaged &C, const DevChunk &T, int layer,
                                          const AttendMask &M, const ScoreForm &form,
                                          const ScoreBounds &bounds, const AttendIo &io,
                                          bool add_mass, const AttendWs &ws, cudaStream_t s);

}  // namespace kvevict
