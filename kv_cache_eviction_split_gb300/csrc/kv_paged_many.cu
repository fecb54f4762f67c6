// kv_paged_many.cu -- attention over the pages for more than 16 query rows a head (prompt
// chunks, whole prompts): bound by the tensor cores, 4 d flops per (query row, key).
//
// An item is 256 query rows of one unit (row i * G + g: token i, head g of the group, so
// that a group's heads share every K and V tile) and the 128-key tiles that any of them
// sees.  A CTA per SM works on two row tiles of 128 ("lanes"), each with S / P and O in
// tensor memory (4 x 128 columns):
//   S_L = Q_L K^T      128 x 128 x d, both operands in shared memory
//   P_L = 2^(S c - m)  a thread per row, all 128 logits in its registers: row max and sum
//                      need no exchange; P is rounded once to the pools' type and
//                      overwrites S
//   O_L += P_L V       P from tensor memory, V as it lies in the page
// The issuing thread runs, per lane, P V of one tile and S of the next; while the tensor
// cores work for one lane, the other lane's four warps take their softmax.  O is rescaled
// only when a row's maximum rises by more than 2^8.
//
// One rounding of P (at most 2^-8 relative in bf16, random signs) adds to an output about as much as
// its own rounding does; two parts, as in the few-rows kernel, would cost half as many
// products again in the kernel's bottleneck.
//
// Warps: 0 loads K and 2 loads V (page boxes by TMA, 3- and 2-tile rings, a lane per
// box), 1 issues the products, 3 describes the items ahead, 4-7 and 8-11 are the lanes' rows;
// they also bring their Q rows into shared memory and write the output.  Tiles no lane sees
// are skipped.
//
// Measured (32 query heads on 8, d = 128, bf16): 2048 tokens over 67584 rows 1.46 ms, 1.52
// PFLOP/s, where the card's sustained library rate is 1.72 (it holds the clock to ~1.7 GHz);
// a prompt of 8192 tokens, window 4096, 340 us, 1.21 PFLOP/s: 6.7 items a CTA, whose ends
// cost about four tiles each (the last products, the output's stores: 12 us in all, the
// first softmax) and the masked halves of the tiles at the window's and diagonal's edges.
#include "kv_paged_attend.cuh"

namespace kvevict {
namespace {
using namespace sm100;

constexpr int kThreads = 12 * 32;
constexpr int kKWarp = 0, kMmaWarp = 1, kVWarp = 2, kSchedWarp = 3, kRowWarp = 4;
// Registers a thread after the split, of 168 at launch (384 x 168 = 128 x 72 + 256 x 216):
// a row thread holds its 128 logits.
constexpr int kLoadRegs = 72, kRowRegs = 216;
constexpr int kBlockBytes = 128 * 128;       // [128 rows][64 columns], 128 B swizzle
constexpr uint32_t kOCol = 256;              // O of lane L at column kOCol + 128 L

constexpr int kItems = 3;                    // items described ahead
// P V of a tile begins when P of its first kPFirst keys is written, beside the exponentials
// of the others (8192 tokens, window 4096, in us: 32 keys 344, 64 339, 96 343, all 128 346).
constexpr int kPFirst = 64;

// Query rows of one lane in an item, and the tiles (counted as in the item's span) of
// which it sees a key: [0, ns) and [a, b).
struct Lane {
    int rows;                  // 0: none
    int t_lo, t_hi;            // cache rows of its first and last query
    int ns, a, b;
    __device__ __forceinline__ bool sees(int x) const { return x < ns || (x >= a && x < b); }
};
// An item and the part of it in this CTA's run, as the scheduler warp writes it.
struct Item {
    int cta;                   // this CTA, counted on through the phases
    int cta0;                  // and the one that holds the item's first tile
    int v, h, n, count;        // unit of the layer, its head, rows held, new tokens
    int row0, rows;            // query rows
    int x0, x1;                // this run's tiles of the item
    TileSpan span;
    int t_hi, lo, sinks;       // rows seen by any query: [0, sinks) and [lo, t_hi]
    int stop;                  // 1: the run has ended, nothing else is set
    Lane lane[2];
    long long tok0, prow0;     // first token; the unit's first packed row
    const int32_t *table;
};

template <int D>
struct Layout {
    static constexpr int kOp = (D / 64) * kBlockBytes;
    static constexpr int kKSt = 3, kVSt = 2;
    static constexpr int kQ = 0;                          // Q of lane 0, then lane 1
    static constexpr int kK = 2 * kOp;
    static constexpr int kV = kK + kKSt * kOp;
    static constexpr int kBars = kV + kVSt * kOp;
    static constexpr int kNumBars = 2 * kKSt + 2 * kVSt + 12 + 1 + 2 * kItems;
    static constexpr int kMisc = (kBars + kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kCut = kMisc + 32;               // [kMaxPhases] CutItem
    static constexpr int kRuns = kCut + kMaxPhases * (int)sizeof(CutItem);
    static constexpr int kFirst = kRuns + (kMaxPhases * (int)sizeof(CtaRun) + 15) / 16 * 16;
    static constexpr int kDesc = kFirst + 32;
    static constexpr int kTotal = kDesc + kItems * (int)sizeof(Item);
    static_assert(kTotal + 1024 <= 227 * 1024, "with cut_run's and TMEM's few static words");
};

struct ManyArgs {
    int layer;
    AttendMask M;
    AttendIo io;
    CutItem *cut;
    float2 *part_ml;
    float *part_o;
    float *lse2;               // null without add_mass, as is q_packed
    void *q_packed;
    int phases;
};

__device__ __forceinline__ void make_item(Item &it, const DevPaged &C, const AttendMask &M,
                                          const UnitRows &U, int pair) {
    const int all = U.count * C.G, t0 = U.n - U.count;
    it.h = U.h;
    it.n = U.n;
    it.count = U.count;
    it.tok0 = U.tok0;
    it.prow0 = packed_row(C, U, 0);
    it.table = U.table;
    it.row0 = pair * kManyRows;
    it.rows = min(kManyRows, all - it.row0);
    const int t_lo = t0 + it.row0 / C.G;
    it.t_hi = t0 + (it.row0 + it.rows - 1) / C.G;
    it.span = tile_span(M, t_lo, it.t_hi, 7);
    it.lo = window_lo(M, max(t_lo, 0));
    it.sinks = min(M.sinks, it.lo);
    const TileSpan &sp = it.span;
#pragma unroll
    for (int L = 0; L < 2; ++L) {
        Lane &a = it.lane[L];
        const int row0 = it.row0 + L * 128;
        a.rows = max(0, min(128, all - row0));
        a.t_lo = t0 + row0 / C.G;
        a.t_hi = a.rows ? t0 + (row0 + a.rows - 1) / C.G : -1;
        const bool some = a.t_hi >= 0;
        a.ns = some ? sp.ns : 0;
        // Sinks that reach into the tile where the item's window begins, or past it, are not
        // among the span's first `ns` tiles: the lane sees them before its own window.
        const int from = M.sinks > sp.first << 7 ? it.lo : window_lo(M, max(a.t_lo, 0));
        a.a = some ? sp.ns + (from >> 7) - sp.first : 0;
        a.b = some ? sp.ns + (a.t_hi >> 7) + 1 - sp.first : 0;
    }
}

// Items of a unit, and the tiles of one of them.
__device__ __forceinline__ int unit_items(const DevPaged &C, const DevChunk &T, const UnitRows &U) {
    return many_rows(C, T, U) ? (U.count * C.G + kManyRows - 1) / kManyRows : 0;
}
__device__ __forceinline__ int item_tiles(const DevPaged &C, const AttendMask &M, const UnitRows &U,
                                          int pair) {
    const int all = U.count * C.G, t0 = U.n - U.count, r0 = pair * kManyRows;
    return tile_span(M, t0 + r0 / C.G, t0 + (min(all, r0 + kManyRows) - 1) / C.G, 7).total;
}

__device__ __forceinline__ float max32(const float (&v)[32]) {
    float a[11];
#pragma unroll
    for (int i = 0; i < 10; ++i) a[i] = fmax3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
    a[10] = fmaxf(v[30], v[31]);
    const float b0 = fmax3(a[0], a[1], a[2]), b1 = fmax3(a[3], a[4], a[5]);
    const float b2 = fmax3(a[6], a[7], a[8]), b3 = fmaxf(a[9], a[10]);
    return fmaxf(fmax3(b0, b1, b2), b3);
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
many_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            const DevPaged C, const DevChunk T, const ManyArgs A) {
    using Ly = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int lane = threadIdx.x & 31;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Ly::kBars);
    uint64_t *k_full = bars, *k_empty = k_full + Ly::kKSt;
    uint64_t *v_full = k_empty + Ly::kKSt, *v_empty = v_full + Ly::kVSt;
    uint64_t *q_full = v_empty + Ly::kVSt;   // [lane]: Q rows are in shared memory (4 warps)
    uint64_t *s_full = q_full + 2;           // [lane]: S of the lane's tile is complete
    uint64_t *p_full = s_full + 2;           // [lane]: P of the first kPFirst keys written (4 warps)
    uint64_t *p_rest = p_full + 2;           // [lane]: all of P
    uint64_t *o_final = p_rest + 2;          // [lane]: the lane's last P V of the item is done
    uint64_t *o_empty = o_final + 2;         // [lane]: O read out (4 warps)
    uint64_t *mma_done = o_empty + 2;
    uint64_t *i_full = mma_done + 1, *i_empty = i_full + kItems;   // item descriptions
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + Ly::kMisc);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + Ly::kMisc + 4);
    CutItem *s_cut = reinterpret_cast<CutItem *>(smem + Ly::kCut);
    CtaRun *s_run = reinterpret_cast<CtaRun *>(smem + Ly::kRuns);
    int *s_first = reinterpret_cast<int *>(smem + Ly::kFirst);
    Item *s_item = reinterpret_cast<Item *>(smem + Ly::kDesc);

    if (threadIdx.x == 0) {
        *s_abort = (smem_u32(smem) & 1023u) ? 1 : 0;
        if (*s_abort) post_status(C.status, KV_ERR_UNSUPPORTED);
        for (int g = 0; g < kMaxPhases; ++g) s_cut[g] = CutItem{-1, 0, 0, 0};
        for (int s = 0; s < Ly::kKSt; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < Ly::kVSt; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int L = 0; L < 2; ++L) {
            mbar_init(&q_full[L], 4);
            mbar_init(&s_full[L], 1);
            mbar_init(&p_full[L], 4);
            mbar_init(&p_rest[L], 4);
            mbar_init(&o_final[L], 1);
            mbar_init(&o_empty[L], 4);
        }
        mbar_init(mma_done, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 3 + 8);    // two loaders, the issuer, eight row warps
        }
        fence_barrier_init();
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = tmem_acquire_all(s_tmem);
    // the phases' units, and this CTA's run in each
    cut_units<kThreads>(
        C.R * C.H, A.phases, kPhaseBytes / (D * 4), (long long)kManyCtas * kPhaseTiles, s_first,
        [&](int v) {
            const UnitRows U = unit_rows(C, T, A.layer, v);
            return many_rows(C, T, U) ? U.n : 0;
        },
        [&](int v) {
            const UnitRows U = unit_rows(C, T, A.layer, v);
            const int items = unit_items(C, T, U);
            return items ? (long long)items * item_tiles(C, A.M, U, items / 2) : 0ll;
        });
    for (int g = 0; g < A.phases; ++g) {
        const int u0 = s_first[g], units = s_first[g + 1] - u0;
        CtaRun run{};
        if (units > 0)
            run = cut_run<kThreads>(
                units, reinterpret_cast<int *>(smem),
                [&](int v) { return unit_rows(C, T, A.layer, u0 + v); },
                [&](const UnitRows &U) { return unit_items(C, T, U); },
                [&](const UnitRows &U, int i) { return kManyCost + item_tiles(C, A.M, U, i); });
        if (threadIdx.x == 0) s_run[g] = run;
        __syncthreads();
    }
    bool ok = *s_abort == 0;

    // Item i of the run for the roles (one lane or a whole warp waits); null at its end or
    // when a wait expired (ok false).
    auto item = [&](int i, bool &fine) -> const Item * {
        fine = fine && mbar_wait(&i_full[i % kItems], (uint32_t)((i / kItems) & 1), s_abort,
                                 C.wait_ns);
        if (!fine) return nullptr;
        const Item *it = &s_item[i % kItems];
        return it->stop ? nullptr : it;
    };
    if (warp >= kRowWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
        // ---------------------------------------------------------------- rows
        const int L = (warp - kRowWarp) >> 2;
        const int quarter = warp & 3;
        const int rr = quarter * 32 + lane;               // row of the lane = its TMEM lane
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_base = tmem + lane_addr + 128 * L;
        const uint32_t o_base = tmem + lane_addr + kOCol + 128 * L;
        const float cs = A.M.scale_log2;
        int kc = 0, sc = 0, ic = 0;
        // This thread's row of an item.
        struct Row {
            bool valid, any;           // a row of the lane; the lane sees a tile of the run
            int t, head, row;          // its query's cache row, query head, row of the unit
            long long tok, prow0;
        };
        auto row_of = [&](const Item *w) {
            Row r;
            const int ns = w->lane[L].ns, x0 = w->x0, x1 = w->x1;
            r.row = w->row0 + L * 128 + rr;
            r.valid = rr < w->lane[L].rows;
            const int token = r.row / C.G;
            r.tok = w->tok0 + token;
            r.head = w->h * C.G + r.row - token * C.G;
            r.t = r.valid ? w->n - w->count + token : -1;
            r.prow0 = w->prow0;
            r.any = x0 < min(ns, x1) || max(x0, w->lane[L].a) < min(x1, w->lane[L].b);
            return r;
        };
        auto load_q = [&](const Row &r, uint4 (&q)[D / 8]) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const typename E::T *>(A.io.q) + r.tok * A.io.q_stride +
                (long long)r.head * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) q[c] = r.valid ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        };
        // Q into shared memory for the products, once those of the item before are done
        auto store_q = [&](const Row &r, const Item *w, const uint4 (&q)[D / 8]) {
            uint8_t *qs = smem + Ly::kQ + L * Ly::kOp + rr * 128;
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4 *>(qs + (c >> 3) * kBlockBytes +
                                           (((c & 7) ^ (rr & 7)) << 4)) = q[c];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[L]);
            if (A.q_packed && r.valid && w->x0 <= (w->lane[L].ns ? 0 : w->lane[L].a)) {
                // the weights' pass takes the rows by TMA; one CTA of a cut item writes them
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<typename E::T *>(A.q_packed) +
                                                       (r.prow0 + r.row) * D);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) dst[c] = q[c];
            }
        };
        const Item *w = item(0, ok);
        ok = __all_sync(0xffffffffu, ok);
        Row cur{}, nxt{};
        if (ok && w) {
            cur = row_of(w);
            if (cur.any) {
                uint4 q[D / 8];
                load_q(cur, q);
                store_q(cur, w, q);
            }
        }
        for (int i = 0; ok && w; ++i) {
            const Lane me = w->lane[L], other = w->lane[1 - L];
            const TileSpan span = w->span;
            const int x0 = w->x0, x1 = w->x1, cta = w->cta, t = cur.t;
            float m = -INFINITY, l = 0.f;
            bool begun = false;
            for (int x = x0; x < x1; ++x) {
                const int key0 = span.tile(x) * kManyTile;
                if (!me.sees(x)) {
                    kc += other.sees(x);
                    continue;
                }
                const int last = key0 + kManyTile - 1;
                const bool full = last <= me.t_lo && (A.M.window == 0 ||
                                                      key0 > me.t_hi - A.M.window ||
                                                      last < A.M.sinks);
                if (!full && (L == 0 || !other.sees(x)) &&
                    (last > w->t_hi || (last >= w->sinks && key0 < w->lo))) {
                    // V rows that no query sees may hold anything: 0 weight times NaN.  The
                    // first lane of the tile clears them before its P goes to the products.
                    const int s = kc % Ly::kVSt;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&v_full[s], (uint32_t)((kc / Ly::kVSt) & 1), s_abort,
                                              C.wait_ns));
                    if (!ok) break;
                    const int j = key0 + rr;
                    if (j > w->t_hi || (j >= w->sinks && j < w->lo)) {
                        uint8_t *vr = smem + Ly::kV + s * Ly::kOp + rr * 128;
#pragma unroll 1
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4 *>(vr + (c >> 3) * kBlockBytes + (c & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                ++kc;
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[L], (uint32_t)(sc & 1), s_abort,
                                                       C.wait_ns));
                if (!ok) break;
                tc_fence_after();
                float s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s_base + 32 * c, s[c]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) reg_fence(s[c]);
                if (!full) {
                    const int lim = t - key0 + 1;
                    const int wlo = A.M.window > 0 ? lim - A.M.window : -1;
                    const int sk = A.M.sinks - key0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t see = low_bits(lim - 32 * c) &
                                             (~low_bits(wlo - 32 * c) | low_bits(sk - 32 * c));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(see >> i & 1u)) s[c][i] = -INFINITY;
                    }
                }
                const float mt =
                    fmaxf(fmaxf(max32(s[0]), max32(s[1])), fmaxf(max32(s[2]), max32(s[3]))) * cs;
                const bool up = mt > m + kLazyLog2;
                if (__any_sync(0xffffffffu, up)) {
                    const float f = up ? shrink(m, mt) : 1.f;
                    if (begun) {
                        // O_L holds the earlier tiles' P V, complete before this S was
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            float o[16];
                            tmem_ld16(o_base + 16 * c, o);
                            tmem_ld_wait();
                            reg_fence(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= f;
                            tmem_st16(o_base + 16 * c, o);
                        }
                    }
                    l *= f;
                    if (up) m = mt;
                }
                begun = true;
                // nothing seen so far: every p is 0
                const float nm = m == -INFINITY ? 0.f : E::kShift - m;
                const float2 cs2 = make_float2(cs, cs), nm2 = make_float2(nm, nm);
                float2 sum[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[c] = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pw[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 e = __ffma2_rn(make_float2(s[c][i], s[c][i + 1]), cs2, nm2);
                        const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                        sum[(i >> 1) & 3] = __fadd2_rn(sum[(i >> 1) & 3], p);
                        pw[i >> 1] = E::pack(p.x, p.y);
                    }
                    tmem_st16u(s_base + 16 * c, pw);
                    if (c == kPFirst / 32 - 1) {
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[L]);
                    }
                }
                const float2 a = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                l += a.x + a.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_rest[L]);
                ++sc;
            }
            if (!ok) break;
            // ---- the item's end: finished rows, or this run's part of them
            const bool whole = x0 == 0 && x1 == span.total;
            if (L == 0 && rr == 0 && x0 > 0 && x1 == span.total)
                s_cut[cta / kManyCtas] = CutItem{w->v, w->cta0, w->row0, w->rows};
            // the description is read
            __syncwarp();
            if (lane == 0) mbar_arrive(&i_empty[i % kItems]);
            // The next item's Q goes to shared memory beside this one's last P V (its last
            // S is complete), so that S of the next follows at once.
            w = item(i + 1, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            nxt.any = false;
            if (w) {
                nxt = row_of(w);
                if (nxt.any) {
                    uint4 q[D / 8];
                    load_q(nxt, q);
                    store_q(nxt, w, q);
                }
            }
            if (begun) {
                ok = __all_sync(0xffffffffu, mbar_wait(&o_final[L], (uint32_t)(ic & 1), s_abort,
                                                       C.wait_ns));
                if (!ok) break;
                tc_fence_after();
                ++ic;
            }
            const float mm = m - E::kShift;
            const long long prow =
                (long long)part_slot(cta, x0 == 0) * kManyRows + L * 128 + rr;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            typename E::T *op = static_cast<typename E::T *>(A.io.out) + cur.tok * A.io.out_stride +
                                (long long)cur.head * D;
            float *pp = A.part_o + prow * D;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
                if (begun) {
                    tmem_ld32(o_base + 32 * c, o);
                    tmem_ld_wait();
                    reg_fence(o);
                }
                if (!cur.valid) continue;
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4 *>(op + 32 * c + i) = make_uint4(
                            E::pack(o[i] * inv, o[i + 1] * inv),
                            E::pack(o[i + 2] * inv, o[i + 3] * inv),
                            E::pack(o[i + 4] * inv, o[i + 5] * inv),
                            E::pack(o[i + 6] * inv, o[i + 7] * inv));
                } else if (begun) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4 *>(pp + 32 * c + i) =
                            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
            if (begun) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty[L]);
            }
            if (cur.valid) {
                if (whole) {
                    const float z = row_lse2(mm, l);
                    if (A.io.lse) A.io.lse[cur.tok * C.Hq + cur.head] = z * kLn2;
                    if (A.lse2) A.lse2[cur.prow0 + cur.row] = z;
                } else A.part_ml[prow] = make_float2(begun ? mm : -INFINITY, l);
            }
            cur = nxt;
        }
        if (!ok && lane == 0) {
            *s_abort = 1;
            post_status(C.status, KV_ERR_TIMEOUT);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        if (warp == kSchedWarp) {
            // ---------------------------------------------------------------- scheduler
            if (lane == 0 && ok) {
                int i = 0;
                auto put = [&](const Item &next) {
                    ok = mbar_wait(&i_empty[i % kItems], (uint32_t)((i / kItems) & 1) ^ 1u, s_abort,
                                   C.wait_ns);
                    if (!ok) return;
                    s_item[i % kItems] = next;
                    mbar_arrive(&i_full[i % kItems]);
                    ++i;
                };
                Item next;
                next.stop = 0;
                for (int g = 0; ok && g < A.phases; ++g) {
                    const CtaRun run = s_run[g];
                    int at = run.part_begin, pair = run.part;
                    for (int v = s_first[g] + run.unit; ok && at < run.end; ++v, pair = 0) {
                        const UnitRows U = unit_rows(C, T, A.layer, v);
                        const int pairs = unit_items(C, T, U);
                        if (pairs && !U.ok) post_status(C.status, KV_ERR_INVALID_ARG);
                        for (; ok && pair < pairs && at < run.end; ++pair) {
                            make_item(next, C, A.M, U, pair);
                            next.v = v;
                            next.cta = g * kManyCtas + blockIdx.x;
                            at += kManyCost;
                            next.cta0 = g * kManyCtas + at / run.per;
                            next.x0 = max(run.begin - at, 0);
                            next.x1 = min(next.span.total, run.end - at);
                            at += next.span.total;
                            if (next.x0 < next.x1) put(next);
                        }
                    }
                }
                next.stop = 1;
                if (ok) put(next);
                if (!ok) {
                    *s_abort = 1;
                    post_status(C.status, KV_ERR_TIMEOUT);
                }
            }
        } else if (warp == kKWarp || warp == kVWarp) {
            // ---------------------------------------------------------------- producers
            fence_proxy_async_global();   // rows that earlier kernels stored, before TMA reads them
            const bool is_k = warp == kKWarp;
            const CUtensorMap *map = is_k ? &tm_k : &tm_v;
            uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
            const int stages = is_k ? Ly::kKSt : Ly::kVSt, ring = is_k ? Ly::kK : Ly::kV;
            const int subs = kManyTile / C.ps, boxes = subs * (D / 64);
            const int half = lane % (D / 64), sub = lane / (D / 64);
            int cnt = 0;
            for (int i = 0;; ++i) {
                const Item *w = item(i, ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok || !w) break;
                const int t_hi = w->t_hi, lo = w->lo, sinks = w->sinks;
                const int x1 = t_hi < 0 ? 0 : w->x1;              // nothing seen: nothing loaded
                const TileSpan span = w->span;
                const int32_t *table = w->table;
                int base = -1, pg = -1;
                for (int x = w->x0; x < x1; ++x) {
                    const int key0 = span.tile(x) * kManyTile, e0 = key0 >> C.ps_log2;
                    if ((e0 & ~31) != base) {
                        base = e0 & ~31;
                        pg = base + lane < C.max_pages ? table[base + lane] : -1;
                    }
                    const int j = key0 + sub * C.ps;
                    const int page = __shfl_sync(0xffffffffu, pg, (j >> C.ps_log2) & 31);
                    // a box with no row in use is not read: its page may not exist
                    const bool use = lane < boxes && j <= t_hi && !(j >= sinks && j + C.ps <= lo);
                    const bool bad = use && (page < 0 || page >= C.num_pages);
                    if (bad) post_status(C.status, KV_ERR_INVALID_ARG);
                    // rows past the pools' end read as zero
                    const long long y = bad ? C.num_pages * C.ps : (long long)page << C.ps_log2;
                    const int n_use = __popc(__ballot_sync(0xffffffffu, use));
                    const int s = cnt % stages;
                    ok = mbar_wait(&empty[s], (uint32_t)((cnt / stages) & 1) ^ 1u, s_abort, C.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        if (n_use) mbar_arrive_expect_tx(&full[s], n_use * C.ps * 128);
                        else mbar_arrive(&full[s]);
                    }
                    __syncwarp();
                    if (use)
                        tma_load_2d(smem + ring + s * Ly::kOp + half * kBlockBytes + sub * C.ps * 128,
                                    map, &full[s], half * 64, (int)y);
                    ++cnt;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&i_empty[i % kItems]);
            }
            if (!ok && lane == 0) {
                *s_abort = 1;
                post_status(C.status, KV_ERR_TIMEOUT);
            }
            for (int s = 0; s < stages; ++s) {
                const int uses = cnt / stages + (cnt % stages > s ? 1 : 0);
                if (uses > 0) mbar_drain(&full[s], (uint32_t)((uses - 1) & 1), kDrainNs);
            }
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- products
            // The whole warp walks the loop with uniform operands and one lane issues.
            {
                const uint32_t el = elect_one();
                constexpr uint32_t idesc_s = E::kHalf ? idesc_f16_f32(128, kManyTile)
                                                      : idesc_bf16_f32(128, kManyTile);
                constexpr uint32_t idesc_o = E::kHalf ? idesc_f16_f32_bmn(128, D)
                                                      : idesc_bf16_f32_bmn(128, D);
                auto uni = [](int x) { return __reduce_max_sync(0xffffffffu, x); };
                auto wait = [&](uint64_t *bar, int count) {
                    return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(count & 1), s_abort,
                                                             C.wait_ns)) != 0;
                };
                const uint32_t tm = (uint32_t)uni((int)tmem);
                int kc = 0;                      // tiles of the rings used so far
                int sc[2] = {0, 0};              // P V issued per lane
                int ic[2] = {0, 0};              // items in which the lane took part
                for (int i = 0;; ++i) {
                    const Item *w = item(i, ok);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok || uni(w == nullptr)) break;
                    auto lane_of = [&](int L) {
                        const Lane &a = w->lane[L];
                        return Lane{0, 0, 0, uni(a.ns), uni(a.a), uni(a.b)};
                    };
                    const Lane l0 = lane_of(0), l1 = lane_of(1);
                    const int x0 = uni(w->x0), x1 = uni(w->x1), w_seen = w->t_hi >= 0;
                    __syncwarp();
                    if (el) mbar_arrive(&i_empty[i % kItems]);
                    // Slot x: P V of the lanes' tiles of slot x - 1, then S of tile x.  Their
                    // K and V are waited for once, before the lanes' P, so that nothing
                    // lies between a lane's P and its sixteen products.  Every tile of a
                    // run is loaded and seen by a lane, unless the item sees nothing.
                    bool pend[2] = {false, false}, begun[2] = {false, false};
                    const int slots = uni(w_seen) ? x1 - x0 : 0;
                    for (int i = 0; ok && i < slots + 1; ++i) {
                        const int x = x0 + i;
                        const bool see[2] = {i < slots && l0.sees(x), i < slots && l1.sees(x)};
                        const int ks = (kc + i) % Ly::kKSt, vs = (kc + i + 1) % Ly::kVSt;
                        if (i < slots) ok = wait(&k_full[ks], (kc + i) / Ly::kKSt);
                        if (ok && i > 0) ok = wait(&v_full[vs], (kc + i - 1) / Ly::kVSt);
                        const bool two = pend[1];        // lane 1's P V is the tile's last
                        const uint64_t vb =
                            sdesc_mn_sw128(smem_u32(smem + Ly::kV) + vs * Ly::kOp, kBlockBytes);
                        const uint64_t ka = sdesc_k_sw128(smem_u32(smem + Ly::kK) + ks * Ly::kOp);
#pragma unroll
                        for (int L = 0; L < 2; ++L) {
                            const uint32_t s_col = tm + 128 * L, o_col = tm + kOCol + 128 * L;
                            if (ok && !begun[L] && see[L]) ok = wait(&q_full[L], ic[L]);
                            if (ok && pend[L]) {
                                // O_L (+)= P V of the lane's previous tile
                                const bool first = !begun[L];
                                if (first) ok = wait(&o_empty[L], ic[L] + 1);
                                ok = ok && wait(&p_full[L], sc[L]);
                                if (ok) {
                                    tc_fence_after();
                                    if (first)
                                        mma_ts_e<false>(o_col, s_col, vb, idesc_o, el);
                                    else
                                        mma_ts_e<true>(o_col, s_col, vb, idesc_o, el);
#pragma unroll
                                    for (int q = 1; q < kPFirst / 16; ++q)
                                        mma_ts_e<true>(o_col, s_col + q * 8,
                                                       sdesc_at(vb, q * 16 * 128), idesc_o, el);
                                    ok = wait(&p_rest[L], sc[L]);
                                }
                                if (ok) {
                                    tc_fence_after();
#pragma unroll
                                    for (int q = kPFirst / 16; q < kManyTile / 16; ++q)
                                        mma_ts_e<true>(o_col, s_col + q * 8,
                                                       sdesc_at(vb, q * 16 * 128), idesc_o, el);
                                    if (L == 1 || !two) mma_commit_e(&v_empty[vs], el);
                                    begun[L] = true;
                                    ++sc[L];
                                }
                                pend[L] = false;
                            }
                            if (ok && see[L]) {
                                // S_L = Q_L K^T
                                tc_fence_after();
                                const uint64_t qa =
                                    sdesc_k_sw128(smem_u32(smem + Ly::kQ + L * Ly::kOp));
#pragma unroll
                                for (int k = 0; k < D / 16; ++k) {
                                    const uint32_t o = (k >> 2) * kBlockBytes + (k & 3) * 32;
                                    if (k)
                                        mma_ss_e<true>(s_col, sdesc_at(qa, o), sdesc_at(ka, o),
                                                       idesc_s, el);
                                    else
                                        mma_ss_e<false>(s_col, qa, ka, idesc_s, el);
                                }
                                mma_commit_e(&s_full[L], el);
                                if (L == 1 || !see[1]) mma_commit_e(&k_empty[ks], el);
                                pend[L] = true;
                            }
                        }
                    }
                    kc += slots;
#pragma unroll
                    for (int L = 0; L < 2; ++L)
                        if (ok && begun[L]) {
                            mma_commit_e(&o_final[L], el);
                            ++ic[L];
                        }
                }
                if (!ok && el) {
                    *s_abort = 1;
                    post_status(C.status, KV_ERR_TIMEOUT);
                }
                // every product issued completes before tensor memory is freed
                mma_commit_e(mma_done, el);
                mbar_drain(mma_done, 0, kDrainNs);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem_release_all(tmem);
    if (threadIdx.x < A.phases) A.cut[threadIdx.x * kManyCtas + blockIdx.x] = s_cut[threadIdx.x];
}

template <typename E, int D>
cudaError_t many(const DevPaged &C, const DevChunk &T, const ManyArgs &A, const AttendWs &ws, cudaStream_t s) {
    using Ly = Layout<D>;
    CUtensorMap mk, mv;
    if (!make_tile_map(&mk, C.k, C.num_pages * C.ps, D, C.ps) ||
        !make_tile_map(&mv, C.v, C.num_pages * C.ps, D, C.ps))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(many_kernel<E, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::kTotal);
    if (e == cudaSuccess)
        e = launch_dependent(many_kernel<E, D>, dim3(kManyCtas), kThreads, Ly::kTotal, s, mk, mv, C,
                             T, A);
    if (e == cudaSuccess)
        e = launch_many_merge(C, T, A.layer, A.io, A.lse2, ws, A.phases, s);
    return e;
}

}  // namespace

cudaError_t launch_attend_many(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                               const AttendIo &io, const AttendWs &ws, cudaStream_t s) {
    const ManyArgs A{layer, M, io, ws.cut, ws.part_ml, ws.part_o, ws.lse2, ws.q_packed,
                     many_phases(C)};
    if (C.dtype == KV_FP16)
        return C.d == 64 ? many<Fp16, 64>(C, T, A, ws, s)
                         : many<Fp16, 128>(C, T, A, ws, s);
    return C.d == 64 ? many<Bf16, 64>(C, T, A, ws, s)
                     : many<Bf16, 128>(C, T, A, ws, s);
}

}  // namespace kvevict
