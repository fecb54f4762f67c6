// kv_paged_few.cuh -- the few-rows attention kernels; kv_paged_few.cu says what they do, and
// instantiates them for plain scores, kv_paged_few_scored.cu for changed ones (kMod).
#pragma once
#include <algorithm>

#include <cooperative_groups.h>

#include "kv_paged_attend.cuh"
#include "kv_paged_scores.cuh"

namespace kvevict {
namespace {
using namespace sm100;
namespace cg = cooperative_groups;

constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kHalfBytes = kFewTile * 128;     // [64 keys][64 columns], 128 B swizzle

template <int D, int NT>
struct Layout {
    static constexpr int kOp = (D / 64) * kHalfBytes;        // K or V of a tile
    static constexpr int kStages = D == 64 ? 6 : 3;
    static constexpr int kStage = 2 * kOp;
    static constexpr int kBuf = kStages * kStage;
    static constexpr int kBufBytes = (D / 16 * 4 + 4) * 32 * 4;   // one warp's O, m, l of 8 rows
    static constexpr int kBars = kBuf + 2 * kBufBytes;
    static constexpr int kTotal = kBars + 2 * kStages * 8 + 32;
    // kMod: the positions of a stage's keys
    static constexpr int kPos = (kTotal + 15) / 16 * 16;
    static constexpr int kPosStage = kFewTile * 4;
    static constexpr int kTotalMod = kPos + kStages * kPosStage;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Transpose of an 8x8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <typename E>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    if constexpr (E::kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void bar_consumers() {
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}
// Barrier of the consumers; true in all of them if `ok` is in all of them.
__device__ __forceinline__ bool bar_consumers_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(kConsumers * 32)
        : "memory");
    return r != 0;
}

struct FewArgs {
    int layer;
    AttendMask M;
    AttendIo io;
    CutItem *cut;
    int *unit_cut;
    float2 *part_ml;
    float *part_o;
    float *lse2;
    float *logits;             // null without add_mass
    int unit_tiles;            // tiles of the logits to a unit
    int logit_rows;            // rows of a tile of them
    int blocks;                // kCluster > 0: row blocks to a unit
    ScoreForm form;            // kMod
};

// At most NT * 8 query rows of a unit, and the tiles they see: the rows up to t_hi, from lo on or
// below sinks; all rows see those up to t_lo and (kMod) from lo_all on.
template <bool kMod>
struct FewItem {
    int row0, rows, t_lo, t_hi, lo, sinks, lo_all;
    TileSpan span;
    __device__ __forceinline__ FewItem(const DevPaged &C, const AttendMask &M, const ScoreForm &F,
                                       const UnitRows &U, int block, int most) {
        row0 = block * most;
        rows = min(most, U.count * C.G - row0);
        if constexpr (kMod) {
            const int i0 = row0 / C.G, i1 = (row0 + rows - 1) / C.G;
            RowBounds all = row_bounds(C, M, F, U, i0);
            lo = lo_all = all.lo;
            t_lo = t_hi = all.hi;
            for (int i = i0 + 1; i <= i1; ++i) {
                const RowBounds b = row_bounds(C, M, F, U, i);
                lo = min(lo, b.lo);
                lo_all = max(lo_all, b.lo);
                t_lo = min(t_lo, b.hi);
                t_hi = max(t_hi, b.hi);
            }
            sinks = min(M.sinks, lo);
            span = bounds_span(M, lo, t_hi, 6);
            return;
        }
        t_lo = U.n - U.count + row0 / C.G;
        t_hi = U.n - U.count + (row0 + rows - 1) / C.G;
        lo = window_lo(M, max(t_lo, 0));
        sinks = min(M.sinks, lo);
        span = tile_span(M, t_lo, t_hi, 6);
        lo_all = 0;
    }
};

// Whether the few-rows kernels take a unit's rows.
__device__ __forceinline__ bool few_rows(const DevPaged &C, const DevChunk &T, const UnitRows &U) {
    return U.count > 0 && !many_rows(C, T, U);
}

template <typename E, int D, int NT, int kCluster, bool kMod>
__global__ void __launch_bounds__(kThreads, 2)
few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
           const DevPaged C, const DevChunk T, const FewArgs A) {
    using Ly = Layout<D, NT>;
    constexpr int kSt = Ly::kStages, kRows = NT * 8, kCost = kCluster == 0 ? kFewCost : 0;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Ly::kBars), *empty = full + kSt;
    volatile int *s_abort = reinterpret_cast<volatile int *>(empty + kSt);
    CutItem *s_cut = reinterpret_cast<CutItem *>(empty + kSt + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *s_abort = (smem_u32(smem) & 1023u) ? 1 : 0;
        if (*s_abort) post_status(C.status, KV_ERR_UNSUPPORTED);
        *s_cut = CutItem{-1, 0, 0, 0};
        for (int s = 0; s < kSt; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumers);
        }
        fence_barrier_init();
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    pdl_wait();
    pdl_trigger();
    const int units = C.R * C.H;
    CtaRun run;
    int rank = 0, block = 0;
    if constexpr (kCluster == 0) {
        run = cut_run<kThreads>(
            units, reinterpret_cast<int *>(smem),
            [&](int v) { return unit_rows(C, T, A.layer, v); },
            [&](const UnitRows &U) { return (int)few_rows(C, T, U); },
            [&](const UnitRows &U, int) { 
                return kCost + FewItem<kMod>(C, A.M, A.form, U, 0, kRows).span.total;
            });
    } else {
        // one item a cluster: its tiles are the whole order, each CTA's run a part of them
        rank = (int)(blockIdx.x % kCluster);
        const int i = (int)(blockIdx.x / kCluster);
        run.unit = i / A.blocks;
        block = i % A.blocks;
        const UnitRows U = unit_rows(C, T, A.layer, run.unit);
        if (!few_rows(C, T, U) || block * kRows >= U.count * C.G) return;   // a whole cluster
        run.total = FewItem<kMod>(C, A.M, A.form, U, block, kRows).span.total;
        run.per = (run.total + kCluster - 1) / kCluster;
        run.begin = min(run.total, rank * run.per);
        run.end = min(run.total, run.begin + run.per);
        run.part_begin = 0;
        __syncthreads();
    }
    const bool go = *s_abort == 0;
    // the loop over items ends after the run's last tile, or after the cluster's one item
    auto more = [&](int at) { return kCluster > 0 ? at == 0 : at < run.end; };

    if (warp == kConsumers) {
        // ---------------------------------------------------------------- producer
        fence_proxy_async_global();    // rows that earlier kernels stored, before TMA reads them
        constexpr int kParts = 2 * (D / 64);                   // K and V halves of a box
        const int box = min(C.ps, kFewTile);
        const int subs = kFewTile / box, boxes = subs * kParts;
        const int kv = lane & 1, half = (lane >> 1) % (D / 64), sub = lane / kParts;
        const CUtensorMap *map = kv ? &tm_v : &tm_k;
        int cnt = 0;
        bool ok = go;
        for (int v = run.unit, at = run.part_begin; ok && more(at); ++v) {
            const UnitRows U = unit_rows(C, T, A.layer, v);
            if (!few_rows(C, T, U)) continue;
            const FewItem<kMod> it(C, A.M, A.form, U, block, kRows);
            if (!U.ok && lane == 0) post_status(C.status, KV_ERR_INVALID_ARG);
            const int x1 = min(it.span.total, run.end - at - kCost);
            int base = -1, pg = -1;
            for (int x = max(run.begin - at - kCost, 0); x < x1; ++x) {
                const int key0 = it.span.tile(x) * kFewTile;
                const int e0 = key0 >> C.ps_log2;
                if ((e0 & ~31) != base) {
                    base = e0 & ~31;
                    pg = base + lane < C.max_pages ? U.table[base + lane] : -1;
                }
                const int j = key0 + sub * box;
                const int page = __shfl_sync(0xffffffffu, pg, (j >> C.ps_log2) & 31);
                // a box with no row in use is not read: its page may not exist
                const bool use = lane < boxes && j <= it.t_hi && !(j >= it.sinks && j + box <= it.lo);
                const bool bad = use && (page < 0 || page >= C.num_pages);
                if (bad) post_status(C.status, KV_ERR_INVALID_ARG);
                // rows past the pools' end read as zero
                const long long y = bad ? C.num_pages * C.ps
                                        : ((long long)page << C.ps_log2) + (j & (C.ps - 1));
                const int n_use = __popc(__ballot_sync(0xffffffffu, use));
                // positions of the box's rows, where distances count
                const bool use_pos = kMod && A.form.pos && use && !bad && kv == 0 && half == 0;
                const int n_pos = kMod ? __popc(__ballot_sync(0xffffffffu, use_pos)) : 0;
                const int s = cnt % kSt;
                ok = mbar_wait(&empty[s], (uint32_t)((cnt / kSt) & 1) ^ 1u, s_abort, C.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    if (n_use)
                        mbar_arrive_expect_tx(&full[s], n_use * box * 128 + n_pos * box * 4);
                    else mbar_arrive(&full[s]);
                }
                __syncwarp();
                if (use_pos)
                    bulk_load(smem + Ly::kPos + s * Ly::kPosStage + sub * box * 4, A.form.pos + y,
                              box * 4, &full[s]);
                if (use)
                    tma_load_2d(smem + s * Ly::kStage + kv * Ly::kOp + half * kHalfBytes +
                                    sub * box * 128,
                                map, &full[s], half * 64, (int)y);
                ++cnt;
            }
            at += kCost + it.span.total;
        }
        if (!ok && lane == 0) {
            *s_abort = 1;
            post_status(C.status, KV_ERR_TIMEOUT);
        }
        // the last load into every stage lands before the CTA exits
        for (int s = 0; s < kSt; ++s) {
            const int uses = cnt / kSt + (cnt % kSt > s ? 1 : 0);
            if (uses > 0) mbar_drain(&full[s], (uint32_t)((uses - 1) & 1), kDrainNs);
        }
    } else {
        // ---------------------------------------------------------------- consumers
        const int quad = lane >> 2, pair = 2 * (lane & 3);
        const float cs = A.M.scale_log2;
        int cnt = 0;
        bool ok = go;
        for (int v = run.unit, at = run.part_begin; ok && more(at); ++v) {
            const UnitRows U = unit_rows(C, T, A.layer, v);
            if (!few_rows(C, T, U)) continue;
            const FewItem<kMod> it(C, A.M, A.form, U, block, kRows);
            const int rows = it.rows, t_lo = it.t_lo, t_hi = it.t_hi, total = it.span.total;
            const int x0 = max(run.begin - at - kCost, 0), x1 = min(total, run.end - at - kCost);
            if (kCluster == 0 && x0 >= x1) {
                at += kCost + total;
                continue;
            }
            // Q^T: columns are query rows (those past the last are zero)
            uint32_t qf[NT][D / 16][2];
            float m[NT][2], l[NT][2], o[NT][D / 16][4];
            int t_row[NT][2], lo_row[NT][2], p_row[NT][2];
            float slope[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = it.row0 + nt * 8 + quad;
                const uint32_t *qp = nullptr;
                if (nt * 8 + quad < rows)
                    qp = reinterpret_cast<const uint32_t *>(
                        static_cast<const typename E::T *>(A.io.q) +
                        (U.tok0 + row / C.G) * A.io.q_stride +
                        (long long)(U.h * C.G + row % C.G) * D + pair);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qf[nt][ks][0] = qp ? __ldg(qp + ks * 8) : 0u;
                    qf[nt][ks][1] = qp ? __ldg(qp + ks * 8 + 4) : 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[nt][ks][i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    m[nt][i] = -INFINITY;
                    l[nt][i] = 0.f;
                    const int r2 = nt * 8 + pair + i;
                    t_row[nt][i] = r2 < rows ? U.n - U.count + (it.row0 + r2) / C.G : -1;
                    if constexpr (kMod) {
                        const int row2 = it.row0 + r2, head = U.h * C.G + row2 % C.G;
                        slope[nt][i] = 0.f;
                        p_row[nt][i] = t_row[nt][i];
                        if (A.form.slopes && r2 < rows) {
                            slope[nt][i] = A.form.slopes[head] * kLog2e;
                            if (A.form.pos) p_row[nt][i] = position_of(C, A.form, U, t_row[nt][i]);
                        }
                        RowBounds b{0, -1};
                        if (r2 < rows) b = row_bounds(C, A.M, A.form, U, row2 / C.G);
                        lo_row[nt][i] = b.lo;
                        t_row[nt][i] = b.hi;
                    }
                }
            }
            for (int x = x0; x < x1; ++x) {
                const int key0 = it.span.tile(x) * kFewTile;
                const int s = cnt % kSt;
                ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (uint32_t)((cnt / kSt) & 1),
                                                       s_abort, C.wait_ns));
                if (!ok) break;
                uint8_t *kt = smem + s * Ly::kStage, *vt = kt + Ly::kOp;
                const int wk = warp * 16;                       // this warp's keys of the tile
                float sc[NT][4];
                {
                    // two chains of products per column tile
                    float s1[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[nt][i] = s1[nt][i] = 0.f;
                    const int kr = wk + (lane & 7) + ((lane >> 3) & 1) * 8;
                    const uint32_t kbase = smem_u32(kt) + kr * 128;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const int ch = ks * 2 + (lane >> 4);    // 16-byte chunk of the row
                        uint32_t a[4];
                        ldsm4(a, kbase + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (kr & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma<E>(ks & 1 ? s1[nt] : sc[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sc[nt][i] = (sc[nt][i] + s1[nt][i]) * (kMod ? 1.f : cs);
                }
                if constexpr (kMod) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sc[nt][i] = A.form.cap2 == 0.f ? sc[nt][i] * cs
                                                           : cap_logit(A.form, sc[nt][i]);
                    if (A.form.slopes) {
                        const int *ps = reinterpret_cast<const int *>(smem + Ly::kPos +
                                                                      s * Ly::kPosStage);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = wk + quad + (i >> 1) * 8;
                            const int pj = A.form.pos ? ps[j] : key0 + j;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                sc[nt][i] -= slope[nt][i & 1] *
                                             fabsf((float)(pj - p_row[nt][i & 1]));
                        }
                    }
                }
                const int last = key0 + kFewTile - 1;
                const bool all =
                    last <= t_lo && (kMod ? key0 >= it.lo_all || last < A.M.sinks
                                          : A.M.window == 0 || key0 > t_hi - A.M.window ||
                                                last < A.M.sinks);
                if (!all) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = key0 + wk + quad + (i >> 1) * 8;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int t = t_row[nt][i & 1];
                            const bool see =
                                j <= t && (kMod ? j >= lo_row[nt][i & 1] || j < A.M.sinks
                                                : A.M.window == 0 || j > t - A.M.window ||
                                                      j < A.M.sinks);
                            if (!see) sc[nt][i] = -INFINITY;
                        }
                    }
                    // V rows that no query sees may hold anything: 0 weight times NaN
#pragma unroll 1
                    for (int c = lane; c < 16 * (D / 8); c += 32) {
                        const int kr = wk + c / (D / 8), ch = c % (D / 8), j = key0 + kr;
                        if (j > t_hi || (j >= it.sinks && j < it.lo))
                            *reinterpret_cast<uint4 *>(vt + (ch >> 3) * kHalfBytes + kr * 128 +
                                                       (((ch & 7) ^ (kr & 7)) << 4)) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();   // before TMA fills the stage again
                    __syncwarp();
                }
                if (A.logits) {
                    const long long tile = (long long)v * A.unit_tiles + x;
                    float *lg = A.logits + tile * (A.logit_rows * kFewTile) + wk + quad;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (nt * 8 + pair + (i & 1) < min(rows, A.logit_rows))
                                lg[(nt * 8 + pair + (i & 1)) * kFewTile + (i >> 1) * 8] = sc[nt][i];
                }
                bool up = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        up |= fmaxf(sc[nt][i], sc[nt][i + 2]) > m[nt][i] + kLazyLog2;
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float mx = fmaxf(sc[nt][i], sc[nt][i + 2]);
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                            if (mx > m[nt][i] + kLazyLog2) {
                                const float f = shrink(m[nt][i], mx);
                                m[nt][i] = mx;
                                l[nt][i] *= f;
#pragma unroll
                                for (int ks = 0; ks < D / 16; ++ks) {
                                    o[nt][ks][i] *= f;
                                    o[nt][ks][i + 2] *= f;
                                }
                            }
                        }
                }
                // P^T: hi and lo parts of the 16 keys x 8 rows, as the products' B operand
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float n0 = m[nt][0] == -INFINITY ? 0.f : E::kShift - m[nt][0];
                    const float n1 = m[nt][1] == -INFINITY ? 0.f : E::kShift - m[nt][1];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float p0 = ex2_approx(sc[nt][2 * i] + n0);
                        const float p1 = ex2_approx(sc[nt][2 * i + 1] + n1);
                        l[nt][0] += p0;
                        l[nt][1] += p1;
                        const uint32_t hi = E::pack(p0, p1);
                        const float2 back = E::unpack(hi);
                        ph[nt][i] = transpose8(hi);
                        pl[nt][i] = transpose8(E::pack(p0 - back.x, p1 - back.y));
                    }
                }
                const int vr = wk + (lane & 7) + (lane >> 4) * 8;
                const uint32_t vbase = smem_u32(vt) + vr * 128;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    const int ch = mt * 2 + ((lane >> 3) & 1);
                    uint32_t a[4];
                    ldsm4t(a, vbase + (ch >> 3) * kHalfBytes + (((ch & 7) ^ (vr & 7)) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma<E>(o[nt][mt], a, ph[nt][0], ph[nt][1]);
                        mma<E>(o[nt][mt], a, pl[nt][0], pl[nt][1]);
                    }
                }
                // The lanes' reads of the stage come before TMA's next writes to it: the arrival
                // alone does not order the two proxies, and beside other kernels on the SM reads
                // of V did find the tile that came after.
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                ++cnt;
            }
            // ---- merge the four warps: 2 and 3 into 0 and 1, then 1 into 0.  A warp whose
            // wait expired meets the others here, and all leave together.
            ok = bar_consumers_all(ok);
            if (!ok) break;
            float *buf = reinterpret_cast<float *>(smem + Ly::kBuf);
            constexpr int kWords = Ly::kBufBytes / 4;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 4);
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 8);
                    l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 16);
                }
#pragma unroll
                for (int step = 2; step >= 1; step >>= 1) {
                    if (nt > 0 || step < 2) bar_consumers();     // the buffers are read
                    if (warp >= step && warp < 2 * step) {
                        float *b = buf + (warp - step) * kWords + lane;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            b[i * 32] = m[nt][i];
                            b[(2 + i) * 32] = l[nt][i];
                        }
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                            for (int i = 0; i < 4; ++i) b[(4 + ks * 4 + i) * 32] = o[nt][ks][i];
                    }
                    bar_consumers();
                    if (warp < step) {
                        const float *b = buf + warp * kWords + lane;
                        float f1[2], f2[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float m2 = b[i * 32], l2 = b[(2 + i) * 32];
                            const float mm = fmaxf(m[nt][i], m2);
                            f1[i] = shrink(m[nt][i], mm);
                            f2[i] = shrink(m2, mm);
                            m[nt][i] = mm;
                            l[nt][i] = l[nt][i] * f1[i] + l2 * f2[i];
                        }
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o[nt][ks][i] = o[nt][ks][i] * f1[i & 1] +
                                               b[(4 + ks * 4 + i) * 32] * f2[i & 1];
                    }
                }
            }
            if (kCluster > 1) bar_consumers();                   // the buffers are read
            if (warp == 0) {
                const bool whole = kCluster == 1 || (kCluster == 0 && x0 == 0 && x1 == total);
                const long long slot = part_slot(blockIdx.x, x0 == 0);
                if (kCluster == 0 && lane == 0 && x1 == total) {
                    if (x0 > 0) *s_cut = CutItem{v, (at + kCost) / run.per, 0, rows};
                    A.unit_cut[v] = x0 > 0 ? (int)blockIdx.x : -1;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r2 = nt * 8 + pair + i;
                        if (r2 >= rows) continue;
                        const float mm = m[nt][i] - E::kShift, ll = l[nt][i];
                        if (whole) {
                            const int row = it.row0 + r2;
                            const long long tok = U.tok0 + row / C.G;
                            const int head = U.h * C.G + row % C.G;
                            const float inv = ll == 0.f ? 0.f : 1.f / ll;
                            typename E::T *op = static_cast<typename E::T *>(A.io.out) +
                                                tok * A.io.out_stride + (long long)head * D + quad;
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks) {
                                op[ks * 16] = E::one(o[nt][ks][i] * inv);
                                op[ks * 16 + 8] = E::one(o[nt][ks][i + 2] * inv);
                            }
                            if (quad == 0) {
                                const float z = row_lse2(mm, ll);
                                if (A.io.lse) A.io.lse[tok * C.Hq + head] = z * kLn2;
                                if (A.lse2) A.lse2[packed_row(C, U, row)] = z;
                            }
                        } else {
                            // this CTA's part: in its shared memory, or the workspace
                            float *ml = kCluster > 1
                                            ? buf + 2 * r2
                                            : reinterpret_cast<float *>(A.part_ml +
                                                                        slot * kFewRows + r2);
                            float *op = kCluster > 1 ? buf + 2 * kRows + r2 * D + quad
                                                     : A.part_o + (slot * kFewRows + r2) * D + quad;
                            if (quad == 0) {
                                ml[0] = mm;
                                ml[1] = ll;
                            }
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks) {
                                op[ks * 16] = o[nt][ks][i];
                                op[ks * 16 + 8] = o[nt][ks][i + 2];
                            }
                        }
                    }
            }
            at += kCost + total;
        }
        if (!ok && lane == 0) {
            *s_abort = 1;
            post_status(C.status, KV_ERR_TIMEOUT);
        }
    }
    if constexpr (kCluster > 1) {
        // the cluster's parts of the item: CTA `rank` merges every kCluster-th row
        static_assert((2 + D) * kRows * 4 <= 2 * Ly::kBufBytes, "a part fits the merge buffers");
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        const UnitRows U = unit_rows(C, T, A.layer, run.unit);
        const FewItem<kMod> it(C, A.M, A.form, U, block, kRows);
        float *buf = reinterpret_cast<float *>(smem + Ly::kBuf);
        const float *part[kCluster];
#pragma unroll
        for (int r = 0; r < kCluster; ++r) part[r] = cl.map_shared_rank(buf, r);
        constexpr int kAtOnce = 128 / D;                     // rows of 128 threads
        for (int r2 = rank + kCluster * (threadIdx.x / D); threadIdx.x < 128 && r2 < it.rows;
             r2 += kCluster * kAtOnce) {
            const int e = threadIdx.x % D;
            float mr[kCluster], lr[kCluster], mm = -INFINITY, ll = 0.f, acc = 0.f;
#pragma unroll
            for (int r = 0; r < kCluster; ++r) {
                mr[r] = part[r][2 * r2];
                lr[r] = part[r][2 * r2 + 1];
            }
#pragma unroll
            for (int r = 0; r < kCluster; ++r) mm = fmaxf(mm, mr[r]);
#pragma unroll
            for (int r = 0; r < kCluster; ++r) {
                const float w = shrink(mr[r], mm);
                ll += lr[r] * w;
                acc += part[r][2 * kRows + r2 * D + e] * w;
            }
            const int row = it.row0 + r2;
            const long long tok = U.tok0 + row / C.G;
            const int head = U.h * C.G + row % C.G;
            static_cast<typename E::T *>(A.io.out)[tok * A.io.out_stride + (long long)head * D + e] =
                E::one(ll == 0.f ? 0.f : acc / ll);
            if (e == 0) {
                const float z = row_lse2(mm, ll);
                if (A.io.lse) A.io.lse[tok * C.Hq + head] = z * kLn2;
                if (A.lse2) A.lse2[packed_row(C, U, row)] = z;
            }
        }
        cl.sync();                                           // no CTA leaves while it is read
    } else if constexpr (kCluster == 0) {
        __syncthreads();
        if (threadIdx.x == 0) A.cut[blockIdx.x] = *s_cut;
    }
}

// ---------------------------------------------------------------------------
// What is left after the tiles: cut items merged, weights added.  Two kinds of block in
// one launch, neither waiting for the other: the first merge_rows * units blocks merge a row
// each; the rest add the weights, whose normaliser they merge for themselves (the partials'
// maxima and sums are a few KB; as a launch after the merge they cost 8 us more).
// ---------------------------------------------------------------------------
constexpr int kFinishThreads = 256;

// The cut item of unit v and the CTA that held its last tile; false if one CTA held it all
// (or, after an expired wait, if nothing valid was left).
__device__ __forceinline__ bool cut_of(const FewArgs &A, int v, CutItem &it, int &last) {
    last = A.unit_cut[v];
    if (last < 0 || last >= kFewCtas) return false;
    it = A.cut[last];
    return it.unit == v && it.cta0 >= 0 && it.cta0 <= last;
}

// One row of a cut item: the partials' weights 2^(m_p - m), then their outputs, every
// eighth to a warp, added up in order.
template <typename E, int D>
__device__ __forceinline__ void merge_row(const DevPaged &C, const DevChunk &T, const FewArgs &A,
                                          const CutItem &it, int last_cta, int row) {
    constexpr int kV = D / 32, kW = kFinishThreads / 32;
    __shared__ float sm_o[kW][D], sm_w[kFewCtas], sm_l[kW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = last_cta - it.cta0 + 1;
    auto slot_row = [&](int p) {
        return (long long)part_slot(it.cta0 + p, p == 0) * kFewRows + row;
    };
    float m = -INFINITY, l = 0.f;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, A.part_ml[slot_row(p)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int p = threadIdx.x; p < parts; p += kFinishThreads) {
        const float2 ml = A.part_ml[slot_row(p)];
        sm_w[p] = shrink(ml.x, m);
        l += ml.y * sm_w[p];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) sm_l[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) l += sm_l[w];
    float acc[kV] = {};
#pragma unroll 8
    for (int p = warp; p < parts; p += kW) {
        const float f = sm_w[p];
        const float *src = A.part_o + slot_row(p) * D + lane * kV;
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[i] += src[i] * f;
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) sm_o[warp][lane * kV + i] = acc[i];
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int k = 1; k < kW; ++k)
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[i] += sm_o[k][lane * kV + i];
    store_merged<E, D>(C, T, A.layer, A.io, A.lse2, it, row, m, l, acc);
}

// Weights of tiles [t0, t1): sums over the unit's query rows of 2^(logit - lse), in row
// order, 64 threads a tile, a thread a key.  Unit by unit: the block first finds the rows'
// lse, of a cut item from its partials, while its first tiles' logits and weights arrive.
template <int kRows, bool kMod>
__device__ __forceinline__ void add_weights(const DevPaged &C, const DevChunk &T, const FewArgs &A,
                                            bool cut, long long t0, long long t1) {
    constexpr int kK = kFinishThreads / kFewRows, kTiles = kFinishThreads / kFewTile;
    __shared__ float sm_m[kK][kFewRows], sm_l[kK][kFewRows], sm_z[kFewRows];
    const int key = threadIdx.x % kFewTile, group = threadIdx.x / kFewTile;
    const bool none = without_rows(C);
    for (long long t = t0; t < t1;) {
        const int v = (int)(t / A.unit_tiles);
        const long long base = (long long)v * A.unit_tiles, end = min(t1, base + A.unit_tiles);
        const UnitRows U = unit_rows(C, T, A.layer, v);
        const int x0 = (int)(t - base);
        t = end;
        if (!few_rows(C, T, U)) continue;
        const FewItem<kMod> it(C, A.M, A.form, U, 0, kFewRows);
        const int x1 = min((int)(end - base), it.span.total);
        const int rows = min(it.rows, A.logit_rows);
        if (x0 >= x1) continue;
        // what a thread needs of its key in a tile: the rows' logits (-inf past the last or
        // unseen) and the weight so far
        float lg[kRows], old = 0.f;
        int at = -1;                                 // pool rows are counted in 31 bits
        auto fetch = [&](int x) {
            const int j = it.span.tile(x) * kFewTile + key;
            const float *src = A.logits + (base + x) * (A.logit_rows * kFewTile) + key;
#pragma unroll
            for (int row = 0; row < kRows; ++row)
                lg[row] = row < rows ? src[row * kFewTile] : -INFINITY;
            at = j <= it.t_hi ? (int)page_row(C, U.table, j) : -1;
            old = at >= 0 ? C.mass[at] : 0.f;
        };
        int x = x0 + group;
        if (x < x1) fetch(x);
        CutItem item;
        int last;
        if (!cut || !cut_of(A, v, item, last)) {
            if (threadIdx.x < it.rows) sm_z[threadIdx.x] = A.lse2[packed_row(C, U, threadIdx.x)];
        } else {
            const int row = threadIdx.x % kFewRows, k = threadIdx.x / kFewRows;
            float m = -INFINITY, l = 0.f;
            if (row < it.rows) {
#pragma unroll 4
                for (int c = item.cta0 + k; c <= last; c += kK) {
                    const float2 ml =
                        A.part_ml[(long long)part_slot(c, c == item.cta0) * kFewRows + row];
                    const float mm = fmaxf(m, ml.x);
                    l = l * shrink(m, mm) + ml.y * shrink(ml.x, mm);
                    m = mm;
                }
            }
            sm_m[k][row] = m;
            sm_l[k][row] = l;
            __syncthreads();
            if (k == 0) {
                float mm = -INFINITY, ll = 0.f;
#pragma unroll
                for (int i = 0; i < kK; ++i) mm = fmaxf(mm, sm_m[i][row]);
#pragma unroll
                for (int i = 0; i < kK; ++i) ll += sm_l[i][row] * shrink(sm_m[i][row], mm);
                sm_z[row] = row_lse2(mm, ll);
            }
        }
        __syncthreads();
        while (x < x1) {
            float acc = 0.f;
            bool seen = false;
#pragma unroll
            for (int row = 0; row < kRows; ++row) {
                const bool see = lg[row] != -INFINITY;
                seen |= see;
                acc += see ? ex2_approx(lg[row] - sm_z[row]) : 0.f;
            }
            if (seen && at >= 0 && !none) C.mass[at] = old + acc;
            x += kTiles;
            if (x < x1) fetch(x);
        }
        __syncthreads();                             // sm_z is read
    }
}

// cut: whether the tiles came from the cut form (else every unit's lse2 is written).
template <typename E, int D, int NT, bool kMod>
__global__ void __launch_bounds__(kFinishThreads, NT == 1 ? 6 : 5)
few_finish_kernel(const DevPaged C, const DevChunk T, const FewArgs A, int merge_rows, bool cut) {
    pdl_wait();
    pdl_trigger();
    const int units = C.R * C.H, merges = cut ? units * merge_rows : 0;
    if ((int)blockIdx.x < merges) {
        const int v = blockIdx.x / merge_rows, row = blockIdx.x % merge_rows;
        const UnitRows U = unit_rows(C, T, A.layer, v);
        if (!few_rows(C, T, U) || row >= U.count * C.G) return;
        CutItem it;
        int last;
        if (cut_of(A, v, it, last)) merge_row<E, D>(C, T, A, it, last, row);
        return;
    }
    const long long tiles = (long long)units * A.unit_tiles;
    const int blocks = (int)gridDim.x - merges;
    const long long per = (tiles + blocks - 1) / blocks, t0 = ((int)blockIdx.x - merges) * per;
    add_weights<NT * 8, kMod>(C, T, A, cut, min(tiles, t0), min(tiles, t0 + per));
}

template <typename E, int D, int NT, int kCluster, bool kMod>
cudaError_t few(const DevPaged &C, const DevChunk &T, const FewArgs &A, cudaStream_t s) {
    using Ly = Layout<D, NT>;
    CUtensorMap mk, mv;
    const int box = C.ps < kFewTile ? C.ps : kFewTile;
    if (!make_tile_map(&mk, C.k, C.num_pages * C.ps, D, box) ||
        !make_tile_map(&mv, C.v, C.num_pages * C.ps, D, box))
        return cudaErrorInvalidValue;
    auto kernel = few_kernel<E, D, NT, kCluster, kMod>;
    constexpr int kSmem = kMod ? Ly::kTotalMod : Ly::kTotal;
    static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs on an SM");
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    const unsigned grid = kCluster == 0 ? kFewCtas : (unsigned)(C.R * C.H * A.blocks * kCluster);
    if (e == cudaSuccess)
        e = launch_cluster_dependent(kernel, kCluster, dim3(grid), kThreads, kSmem, s, mk, mv, C, T,
                                     A);
    if (e == cudaSuccess && (kCluster == 0 || A.logits)) {
        const int rows = NT * 8 < T.max_t * (long long)C.G ? NT * 8 : T.max_t * C.G;
        const long long merges = kCluster == 0 ? (long long)C.R * C.H * rows : 0;
        // eight tiles a block, or what one round of blocks (six an SM) needs (4 heads of 131072
        // rows, in us: 4 tiles 68.2, 8 66.5, 12 66.4, 16 67.5)
        const long long tiles = A.logits ? (long long)C.R * C.H * A.unit_tiles : 0;
        const long long adds = std::min<long long>((tiles + 7) / 8, 6 * 152);
        e = launch_dependent(few_finish_kernel<E, D, NT, kMod>, dim3((unsigned)(merges + adds)),
                             kFinishThreads, 0, s, C, T, A, rows, kCluster == 0);
    }
    return e;
}

template <typename E, int D, int NT, bool kMod>
cudaError_t few_form(const DevPaged &C, const DevChunk &T, const FewArgs &A, int cluster,
                     cudaStream_t s) {
    switch (cluster) {
        case 0: return few<E, D, NT, 0, kMod>(C, T, A, s);
        case 1: return few<E, D, NT, 1, kMod>(C, T, A, s);
        case 2: return few<E, D, NT, 2, kMod>(C, T, A, s);
        case 4: return few<E, D, NT, 4, kMod>(C, T, A, s);
        default: return few<E, D, NT, 8, kMod>(C, T, A, s);
    }
}

template <bool kMod>
cudaError_t attend_few(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                       const ScoreForm &form, const AttendIo &io, bool add_mass, long long seen,
                       long long items, int max_rows, int blocks, const AttendWs &ws,
                       cudaStream_t s) {
    const FewArgs A{layer,      M,         io,      ws.cut,
                    ws.unit_cut, ws.part_ml, ws.part_o, ws.lse2, add_mass ? ws.logits : nullptr,
                    (C.cap + kFewTile - 1) / kFewTile, max_rows, blocks,
                    form};
    // short: the largest cluster that leaves every CTA a tile and the GPU in one round
    int cluster = 0;
    if (seen <= kShortRows) {
        cluster = 8;
        while (cluster > 1 && (cluster * kFewTile > seen || items * cluster > kFewCtas))
            cluster /= 2;
    }
    const int nt = max_rows <= 8 ? 1 : 2;
    if (C.dtype == KV_FP16) {
        if (C.d == 64)
            return nt == 1 ? few_form<Fp16, 64, 1, kMod>(C, T, A, cluster, s)
                           : few_form<Fp16, 64, 2, kMod>(C, T, A, cluster, s);
        return nt == 1 ? few_form<Fp16, 128, 1, kMod>(C, T, A, cluster, s)
                       : few_form<Fp16, 128, 2, kMod>(C, T, A, cluster, s);
    }
    if (C.d == 64)
        return nt == 1 ? few_form<Bf16, 64, 1, kMod>(C, T, A, cluster, s)
                       : few_form<Bf16, 64, 2, kMod>(C, T, A, cluster, s);
    return nt == 1 ? few_form<Bf16, 128, 1, kMod>(C, T, A, cluster, s)
                   : few_form<Bf16, 128, 2, kMod>(C, T, A, cluster, s);
}

}  // namespace
}  // namespace kvevict
