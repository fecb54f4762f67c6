// kv_paged_mass.cu -- accumulated attention weights of prompt chunks: for every cache row j,
// mass_j += sum over the query rows that see it of 2^(s c - lse2), after the attention pass
// has left each row's lse.
//
// Keys are the rows of the product: S^T = K Q^T with 128 keys x 128 query rows, so that a
// thread owns a key and adds its weights up in a register, in row order: no atomics, and
// no exchange between threads but one.  An item is 256 keys (two tiles) of one unit, against
// every tile of 128 query rows that sees any of them; K stays in shared memory for the item
// (the next one's loads meanwhile), packed Q tiles stream through a ring (32 KB per two
// products at d = 128).  Four groups of four warps take the two key tiles' products, of even
// and odd row tiles, each from a tensor-memory buffer of its own: four warps a scheduler hide
// each other's waits and loads.  At the item's end the odd rows' sums go to the even rows'
// threads.  The query rows that see key j are a run of packed rows,
// [ (j - t0) G, (j + window - t0) G ), so the mask is two bounds.
//
// Measured (2 requests, 301 .. 511 new tokens of 32 query heads over 8 x 13107 .. 32768 rows,
// d = 128, bf16): 163 us of the call's 442, where the products alone would take 90.  Both
// operands of a product come from shared memory, as much of its bandwidth as of the tensor
// cores' time, which the Q tiles' arrival and the rows' lse share.  Without the exponentials
// 25 us less, with half the products 20 us less, with half the Q traffic the same.  Eight
// key warps were as fast until the two tiles' products were issued after one wait (178 us);
// an issuing warp for each tile was slower (172 us).
#include <type_traits>

#include "kv_paged_attend.cuh"

namespace kvevict {
namespace {
using namespace sm100;

constexpr int kThreads = 20 * 32;
constexpr int kKWarp = 0, kMmaWarp = 1, kQWarp = 2, kSchedWarp = 3, kKeyWarp = 4;
// Registers a thread after the split, of 96 at launch (640 x 96 = 128 x 64 + 512 x 104).
constexpr int kLoadRegs = 64, kKeyRegs = 104;
constexpr int kBlockBytes = 128 * 128;       // [128 rows][64 columns], 128 B swizzle
constexpr int kGroup = 2;                    // key tiles per item
constexpr int kGroupCost = 2;                // an item's own cost in row tiles
constexpr int kItems = 3;                    // items described ahead
constexpr int kQSt = 3;                      // Q ring
constexpr int kLSt = 2;                      // ring of the rows' lse: even, a warp sees every other step

struct Item {
    int stop;
    int tile0, tiles;          // key tiles
    int rt0, rt1;              // tiles of 128 query rows
    int n, rows, t0;           // rows held, query rows, cache row of the first query
    long long prow0;           // first packed row
    const int32_t *table;
};

template <int D>
struct Layout {
    static constexpr int kOp = (D / 64) * kBlockBytes;
    static constexpr int kK = 0;                          // [2 items][kGroup]
    static constexpr int kQ = 2 * kGroup * kOp;
    static constexpr int kLse = kQ + kQSt * kOp;          // [kLSt][128] -lse2
    static constexpr int kAcc = kLse + kLSt * 128 * 4;    // [kGroup][128] sums of odd row tiles
    static constexpr int kTotal = kAcc + kGroup * 128 * 4;
    // the static words lie below the first 1024 bytes' end
    static_assert(kTotal + 1024 <= 227 * 1024, "fits with the static words");
};

struct MassArgs {
    int layer;
    AttendMask M;
    const float *lse2;
};

// Key groups of a unit, and of each the query row tiles [rt0, rt1) that see it.
struct Groups {
    int t0, rows, groups;
    __device__ __forceinline__ Groups(const DevPaged &C, const DevChunk &T, const UnitRows &U) {
        rows = U.count * C.G;
        t0 = U.n - U.count;
        groups = many_rows(C, T, U) ? (U.n + kGroup * kManyTile - 1) / (kGroup * kManyTile) : 0;
    }
    __device__ __forceinline__ void range(const DevPaged &C, const AttendMask &M, int n, int g,
                                          int &rt0, int &rt1) const {
        const int key0 = g * kGroup * kManyTile, last = min(n, key0 + kGroup * kManyTile) - 1;
        const int i0 = max(0, key0 - t0);
        int i1 = n - 1 - t0;                       // last query
        if (M.window > 0 && key0 >= M.sinks)
            i1 = (int)min((long long)i1, (long long)last - t0 + M.window - 1);
        rt0 = (int)((long long)i0 * C.G >> 7);
        rt1 = i1 < i0 ? rt0 : (int)(((long long)(i1 + 1) * C.G + 127) >> 7);
    }
};

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
            const DevPaged C, const DevChunk T, const MassArgs A) {
    using Ly = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);   // uniform
    const int lane = threadIdx.x & 31;
    __shared__ uint64_t k_full[2], k_empty[2];               // [item parity]
    __shared__ uint64_t q_full[kQSt], q_empty[kQSt], l_full[kLSt], l_empty[kLSt];
    __shared__ uint64_t s_full[2], s_free[2];                // [row tile parity]
    __shared__ uint64_t a_full[kGroup], a_empty[kGroup];     // the odd row tiles' sums
    __shared__ uint64_t mma_done[1], i_full[kItems], i_empty[kItems];
    __shared__ Item s_item[kItems];
    __shared__ uint32_t s_tmem[1];
    __shared__ int s_abort_word;
    volatile int *s_abort = &s_abort_word;
    float *s_lse = reinterpret_cast<float *>(smem + Ly::kLse);
    float *s_acc = reinterpret_cast<float *>(smem + Ly::kAcc);

    if (threadIdx.x == 0) {
        *s_abort = (smem_u32(smem) & 1023u) ? 1 : 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < kQSt; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < kLSt; ++i) {
            mbar_init(&l_full[i], 1);
            mbar_init(&l_empty[i], 8);       // the warps of the row tile's parity
        }
        for (int i = 0; i < kGroup; ++i) {
            mbar_init(&a_full[i], 4);
            mbar_init(&a_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 8);
        }
        mbar_init(mma_done, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 3 + 16);
        }
        fence_barrier_init();
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_q);
    }
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0 && *s_abort) post_status(C.status, KV_ERR_UNSUPPORTED);
    const uint32_t tmem = tmem_acquire_all(s_tmem);
    // runs of equal numbers of (key group, row tile) steps; a group belongs to the run
    // that its first step lies in
    const CtaRun run = cut_run<kThreads>(
        C.R * C.H, reinterpret_cast<int *>(smem),
        [&](int v) { return unit_rows(C, T, A.layer, v); },
        [&](const UnitRows &U) { return Groups(C, T, U).groups; },
        [&](const UnitRows &U, int i) {
            int r0, r1;
            Groups(C, T, U).range(C, A.M, U.n, i, r0, r1);
            return r1 > r0 ? r1 - r0 + kGroupCost : 0;
        });
    bool ok = *s_abort == 0;
    auto item = [&](int i, bool &fine) -> const Item * {
        fine = fine && mbar_wait(&i_full[i % kItems], (uint32_t)((i / kItems) & 1), s_abort,
                                 C.wait_ns);
        if (!fine) return nullptr;
        const Item *it = &s_item[i % kItems];
        return it->stop ? nullptr : it;
    };
    auto expired = [&]() {
        *s_abort = 1;
        post_status(C.status, KV_ERR_TIMEOUT);
    };

    if (warp >= kKeyWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kKeyRegs));
        // ---------------------------------------------------------------- keys
        const int b = (warp - kKeyWarp) >> 2;             // tensor-memory buffer
        const int k = b & 1, par = b >> 1;                // key tile of the item, row tiles' parity
        const int quarter = warp & 3;
        const int rr = quarter * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
        const float cs = A.M.scale_log2;
        const float2 cs2 = make_float2(cs, cs);
        int rc = 0, summed = 0;
        for (int i = 0;; ++i) {
            const Item *w = item(i, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !w) break;
            const int rt0 = w->rt0, rt1 = w->rt1, rows = w->rows, n = w->n, t0 = w->t0;
            const bool mine = k < w->tiles;
            const int key0 = (w->tile0 + k) * kManyTile, j = key0 + rr;
            const int32_t *table = w->table;
            __syncwarp();
            if (lane == 0) mbar_arrive(&i_empty[i % kItems]);
            // the packed rows that see key j: [r_lo, r_hi); those that see every key of the
            // tile: [a_lo, a_hi)
            const bool held = mine && j < n;
            const long long G = C.G;
            const bool sink = j < A.M.sinks || A.M.window == 0;
            const int r_lo = held ? (int)min((long long)rows, max(0ll, (j - t0) * G)) : rows;
            const int r_hi =
                sink ? rows
                     : (int)min((long long)rows, max(0ll, ((long long)j + A.M.window - t0) * G));
            const int last = key0 + kManyTile - 1;
            const int a_lo = last < n ? (int)min((long long)rows, max(0ll, (last - t0) * G)) : rows;
            const int a_hi =
                last < A.M.sinks || A.M.window == 0
                    ? rows
                    : (int)min((long long)rows, max(0ll, ((long long)key0 + A.M.window - t0) * G));
            // the key's weight so far is looked up beside the first steps: its page here, its
            // value after the first
            const int page = par == 0 && held && r_lo < r_hi ? table[j >> C.ps_log2] : -1;
            float *to = nullptr;
            float acc = 0.f, old = 0.f;
            auto find = [&]() {
                if (to == nullptr && page >= 0 && page < C.num_pages) {
                    to = C.mass + ((long long)page << C.ps_log2) + (j & (C.ps - 1));
                    old = *to;
                }
            };
            const int step0 = rc - rt0;
            rc += rt1 - rt0;
            for (int rt = rt0 + ((step0 + rt0 + par) & 1); rt < rt1; rt += 2) {
                const int step = step0 + rt, ls = step % kLSt;
                ok = mbar_wait(&l_full[ls], (uint32_t)((step / kLSt) & 1), s_abort, C.wait_ns);
                ok = ok && mbar_wait(&s_full[par], (uint32_t)((step >> 1) & 1), s_abort, C.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (mine) {
                    tc_fence_after();
                    const int row0 = rt * 128;
                    const bool all = row0 >= a_lo && row0 + 128 <= a_hi;
                    const uint32_t base = tmem + lane_addr + 128 * b;
                    const float4 *lse = reinterpret_cast<const float4 *>(s_lse + ls * 128);
                    float2 sum[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum[c] = make_float2(0.f, 0.f);
                    // every row of the tile sees the thread's key, or a run of its bits does
                    auto add = [&](auto masked) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float s[32];
                            tmem_ld32(base + 32 * c, s);
                            tmem_ld_wait();
                            reg_fence(s);
                            if (c == 3) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&s_free[par]);
                            }
                            uint32_t see = 0;
                            if (masked)
                                see = low_bits(r_hi - row0 - 32 * c) &
                                      ~low_bits(r_lo - row0 - 32 * c);
#pragma unroll
                            for (int x = 0; x < 32; x += 4) {
                                const float4 z = lse[c * 8 + x / 4];
                                const float2 e0 = __ffma2_rn(make_float2(s[x], s[x + 1]), cs2,
                                                             make_float2(z.x, z.y));
                                const float2 e1 = __ffma2_rn(make_float2(s[x + 2], s[x + 3]), cs2,
                                                             make_float2(z.z, z.w));
                                float2 p0 = make_float2(ex2_approx(e0.x), ex2_approx(e0.y));
                                float2 p1 = make_float2(ex2_approx(e1.x), ex2_approx(e1.y));
                                if (masked) {
                                    if (!(see >> x & 1u)) p0.x = 0.f;
                                    if (!(see >> (x + 1) & 1u)) p0.y = 0.f;
                                    if (!(see >> (x + 2) & 1u)) p1.x = 0.f;
                                    if (!(see >> (x + 3) & 1u)) p1.y = 0.f;
                                }
                                sum[(x >> 1) & 3] = __fadd2_rn(sum[(x >> 1) & 3], p0);
                                sum[((x >> 1) + 1) & 3] = __fadd2_rn(sum[((x >> 1) + 1) & 3], p1);
                            }
                        }
                    };
                    if (__all_sync(0xffffffffu, all)) add(std::false_type{});
                    else add(std::true_type{});
                    const float2 a = __fadd2_rn(__fadd2_rn(sum[0], sum[1]),
                                                __fadd2_rn(sum[2], sum[3]));
                    acc += a.x + a.y;
                } else if (lane == 0) {
                    mbar_arrive(&s_free[par]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&l_empty[ls]);
                find();
            }
            if (!ok) break;
            if (!mine) continue;
            // the odd row tiles' sums to the even ones' threads
            float *part = s_acc + k * 128 + rr;
            ok = __all_sync(0xffffffffu,
                            par ? mbar_wait(&a_empty[k], (uint32_t)(summed & 1) ^ 1u, s_abort, C.wait_ns)
                                : mbar_wait(&a_full[k], (uint32_t)(summed & 1), s_abort, C.wait_ns));
            if (!ok) break;
            ++summed;
            if (par) *part = acc;
            else acc += *part;
            __syncwarp();
            if (lane == 0) mbar_arrive(par ? &a_full[k] : &a_empty[k]);
            find();
            if (to) *to = old + acc;
        }
        if (!ok && lane == 0) expired();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        if (warp == kSchedWarp) {
            if (lane == 0 && ok) {
                int i = 0, at = run.part_begin, j = run.part;
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
                for (int v = run.unit; ok && at < run.end; ++v) {
                    const UnitRows U = unit_rows(C, T, A.layer, v);
                    const Groups g(C, T, U);
                    next.n = U.n;
                    next.rows = g.rows;
                    next.t0 = g.t0;
                    next.prow0 = packed_row(C, U, 0);
                    next.table = U.table;
                    for (; ok && j < g.groups && at < run.end; ++j) {
                        g.range(C, A.M, U.n, j, next.rt0, next.rt1);
                        const int steps = next.rt1 - next.rt0;
                        if (steps > 0 && at >= run.begin) {
                            next.tile0 = j * kGroup;
                            next.tiles = min(kGroup, ((U.n + kManyTile - 1) >> 7) - next.tile0);
                            put(next);
                        }
                        at += steps > 0 ? steps + kGroupCost : 0;
                    }
                    j = 0;
                }
                next.stop = 1;
                if (ok) put(next);
                if (!ok) expired();
            }
        } else if (warp == kKWarp) {
            fence_proxy_async_global();    // rows that earlier kernels stored, before TMA reads them
            const int subs = kManyTile / C.ps, boxes = subs * (D / 64);
            const int half = lane % (D / 64), sub = lane / (D / 64);
            int cnt = 0;
            for (int i = 0;; ++i) {
                const Item *w = item(i, ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok || !w) break;
                const int n = w->n, tiles = w->tiles, tile0 = w->tile0, s = i & 1;
                const int32_t *table = w->table;
                int y[kGroup], n_use = 0;
                bool use[kGroup];
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    // a page that does not exist was reported by the attention pass
                    const int j = (tile0 + k) * kManyTile + sub * C.ps;
                    use[k] = k < tiles && lane < boxes && j < n;
                    const int page = use[k] ? table[j >> C.ps_log2] : -1;
                    use[k] = use[k] && page >= 0 && page < C.num_pages;
                    y[k] = page << C.ps_log2;
                    n_use += __popc(__ballot_sync(0xffffffffu, use[k]));
                }
                ok = mbar_wait(&k_empty[s], (uint32_t)((i >> 1) & 1) ^ 1u, s_abort, C.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    if (n_use) mbar_arrive_expect_tx(&k_full[s], n_use * C.ps * 128);
                    else mbar_arrive(&k_full[s]);
                    mbar_arrive(&i_empty[i % kItems]);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kGroup; ++k)
                    if (use[k])
                        tma_load_2d(smem + Ly::kK + (s * kGroup + k) * Ly::kOp + half * kBlockBytes +
                                        sub * C.ps * 128,
                                    &tm_k, &k_full[s], half * 64, y[k]);
                ++cnt;
            }
            if (!ok && lane == 0) expired();
            for (int s = 0; s < 2; ++s) {
                const int uses = cnt / 2 + (cnt % 2 > s ? 1 : 0);
                if (uses > 0) mbar_drain(&k_full[s], (uint32_t)((uses - 1) & 1), kDrainNs);
            }
        } else if (warp == kQWarp) {
            fence_proxy_async_global();
            int cnt = 0;
            for (int i = 0;; ++i) {
                const Item *w = item(i, ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok || !w) break;
                const int rt0 = w->rt0, rt1 = w->rt1, rows = w->rows;
                const long long prow0 = w->prow0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&i_empty[i % kItems]);
                // the rows' lse are read a step ahead: their latency is about a step's products
                float z[4];
                auto fetch = [&](int rt) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = rt * 128 + lane * 4 + k;
                        z[k] = row < rows ? -A.lse2[prow0 + row] : 0.f;
                    }
                };
                fetch(rt0);
                for (int rt = rt0; rt < rt1; ++rt, ++cnt) {
                    const int s = cnt % kQSt;
                    const int ls = cnt % kLSt;
                    ok = mbar_wait(&q_empty[s], (uint32_t)((cnt / kQSt) & 1) ^ 1u, s_abort, C.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[s], Ly::kOp);
                        for (int kb = 0; kb < D / 64; ++kb)
                            tma_load_2d(smem + Ly::kQ + s * Ly::kOp + kb * kBlockBytes, &tm_q,
                                        &q_full[s], kb * 64, (int)(prow0 + rt * 128));
                    }
                    __syncwarp();
                    ok = mbar_wait(&l_empty[ls], (uint32_t)((cnt / kLSt) & 1) ^ 1u, s_abort, C.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) {
                        ++cnt;                       // its copy is drained below
                        break;
                    }
                    *reinterpret_cast<float4 *>(s_lse + ls * 128 + lane * 4) =
                        make_float4(z[0], z[1], z[2], z[3]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&l_full[ls]);
                    if (rt + 1 < rt1) fetch(rt + 1);
                }
            }
            if (!ok && lane == 0) expired();
            for (int s = 0; s < kQSt; ++s) {
                const int uses = cnt / kQSt + (cnt % kQSt > s ? 1 : 0);
                if (uses > 0) mbar_drain(&q_full[s], (uint32_t)((uses - 1) & 1), kDrainNs);
            }
        } else if (warp == kMmaWarp) {
            // the whole warp walks the loop with uniform operands and one lane issues
            {
                const uint32_t el = elect_one();
                auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
                auto wait = [&](uint64_t *bar, int count) {
                    return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)(count & 1), s_abort,
                                                             C.wait_ns)) != 0;
                };
                const uint32_t tm = (uint32_t)uni((int)tmem);
                constexpr uint32_t idesc = E::kHalf ? idesc_f16_f32(128, 128) : idesc_bf16_f32(128, 128);
                int rc = 0, s = 0, turn = 0;     // row tiles so far, Q slot, its round
                for (int i = 0;; ++i) {
                    const Item *w = item(i, ok);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok || uni(w == nullptr)) break;
                    const int steps = uni(w->rt1 - w->rt0), tiles = uni(w->tiles), ks = i & 1;
                    __syncwarp();
                    if (el) mbar_arrive(&i_empty[i % kItems]);
                    ok = wait(&k_full[ks], i >> 1);
                    const uint64_t ka = sdesc_k_sw128(smem_u32(smem + Ly::kK) + ks * kGroup * Ly::kOp);
                    for (int r = 0; ok && r < steps; ++r, ++rc) {
                        const int par = rc & 1;
                        ok = wait(&q_full[s], turn) && wait(&s_free[par], (rc >> 1) + 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t qb = sdesc_k_sw128(smem_u32(smem + Ly::kQ) + s * Ly::kOp);
#pragma unroll
                        for (int k = 0; k < kGroup; ++k) {
                            if (k >= tiles) continue;
                            const uint32_t col = tm + 256 * par + 128 * k;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t o = (kk >> 2) * kBlockBytes + (kk & 3) * 32;
                                if (kk)
                                    mma_ss_e<true>(col, sdesc_at(ka, k * Ly::kOp + o),
                                                   sdesc_at(qb, o), idesc, el);
                                else
                                    mma_ss_e<false>(col, sdesc_at(ka, k * Ly::kOp), qb, idesc, el);
                            }
                        }
                        mma_commit_e(&s_full[par], el);
                        mma_commit_e(&q_empty[s], el);
                        if (++s == kQSt) {
                            s = 0;
                            turn ^= 1;
                        }
                    }
                    if (ok) mma_commit_e(&k_empty[ks], el);
                }
                if (!ok && el) expired();
                mma_commit_e(mma_done, el);
                mbar_drain(mma_done, 0, kDrainNs);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem_release_all(tmem);
}

template <typename E, int D>
cudaError_t mass(const DevPaged &C, const DevChunk &T, const MassArgs &A, const AttendWs &ws,
                 cudaStream_t s) {
    using Ly = Layout<D>;
    CUtensorMap mk, mq;
    if (!make_tile_map(&mk, C.k, C.num_pages * C.ps, D, C.ps) ||
        !make_tile_map(&mq, ws.q_packed, T.tokens * C.Hq, D, 128))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(mass_kernel<E, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::kTotal);
    if (e == cudaSuccess)
        e = launch_dependent(mass_kernel<E, D>, dim3(kManyCtas), kThreads, Ly::kTotal, s, mk, mq, C,
                             T, A);
    return e;
}

}  // namespace

cudaError_t launch_many_mass(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                             const AttendWs &ws, cudaStream_t s) {
    const MassArgs A{layer, M, ws.lse2};
    if (C.dtype == KV_FP16)
        return C.d == 64 ? mass<Fp16, 64>(C, T, A, ws, s) : mass<Fp16, 128>(C, T, A, ws, s);
    return C.d == 64 ? mass<Bf16, 64>(C, T, A, ws, s) : mass<Bf16, 128>(C, T, A, ws, s);
}

}  // namespace kvevict
