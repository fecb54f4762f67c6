// kv_paged_few.cu -- attention over the pages for at most 16 query rows a head (decode
// steps, short runs of tokens): bound by reading K and V once.
//
// Per unit, with rows x = (token, head of the group):
//   S^T = K Q^T        m16n8k16 products, 16 keys x 8 rows, K through ldmatrix
//   p = 2^(s c - m)    running maximum m and sum l per row, in registers
//   O^T += V^T P^T     V through transposing ldmatrix; P^T by an 8x8 transpose of the
//                      S^T registers, as two 16-bit parts (p = hi + lo: 16 bits of p in
//                      bf16, 22 in fp16), so the weights cost no precision
// Keys go down the 16 rows of the product and query rows across its 8 columns: with 4 or
// 7 rows a head half of the columns carry work, where rows on the 16 side would leave
// three quarters of it idle.  Tensor-memory products (128 rows at least) would be padded
// 16 to 32 times over here and add their round trips to a kernel that has to be short.
//
// A CTA has 4 consumer warps, each taking 16 of a tile's 64 keys with statistics and
// output of its own (no exchange inside the loop), and a producer warp that fills a ring
// of tiles by TMA (3 x 32 KB at d = 128): its lanes hold 32 page-table entries and issue
// one box each.  Two CTAs an SM keep ~190 KB in flight.  The consumers merge through
// shared memory once per item.
#include "kv_paged_attend.cuh"

namespace kvevict {
namespace {
using namespace sm100;

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
    int *cta_status;
    CutItem *cut;
    float2 *part_ml;
    float *part_o;
    float *lse2;
    int *tiles;
    int2 *tile_at;
    float *logits;             // null without add_mass
};

template <typename E, int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
           const DevPaged C, const DevChunk T, const FewArgs A) {
    using Ly = Layout<D, NT>;
    constexpr int kSt = Ly::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Ly::kBars), *empty = full + kSt;
    int *s_status = reinterpret_cast<int *>(empty + kSt);
    volatile int *s_abort = s_status + 1;
    CutItem *s_cut = reinterpret_cast<CutItem *>(s_status + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *s_status = (smem_u32(smem) & 1023u) ? KV_ERR_UNSUPPORTED : 0;
        *s_abort = *s_status;
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
    const CtaRun run = cut_run<kThreads>(units, 1, [&](int v) {
        const UnitRows U = unit_rows(C, T, A.layer, v);
        if (U.count <= 0 || (long long)U.count * C.G > NT * 8) return 0;
        return tile_span(A.M, U.n - U.count, U.n - 1, 6).total;
    });
    const bool go = *s_abort == 0;

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
        int v = run.unit, at = run.unit_begin;
        while (ok && at < run.end) {
            const UnitRows U = unit_rows(C, T, A.layer, v);
            const bool mine = U.count > 0 && (long long)U.count * C.G <= NT * 8;
            const TileSpan span = tile_span(A.M, U.n - U.count, U.n - 1, 6);
            const int total = mine ? span.total : 0;
            if (total && !U.ok && lane == 0) atomicCAS(s_status, 0, KV_ERR_INVALID_ARG);
            const int lo = window_lo(A.M, max(U.n - U.count, 0)), sinks = min(A.M.sinks, lo);
            const int x1 = min(total, run.end - at);
            int base = -1, pg = -1;
            for (int x = max(run.begin - at, 0); ok && x < x1; ++x) {
                const int key0 = span.tile(x) * kFewTile;
                const int e0 = key0 >> C.ps_log2;
                if ((e0 & ~31) != base) {
                    base = e0 & ~31;
                    pg = base + lane < C.max_pages ? U.table[base + lane] : -1;
                }
                const int j = key0 + sub * box;
                const int page = __shfl_sync(0xffffffffu, pg, (j >> C.ps_log2) & 31);
                // a box with no row in use is not read: its page may not exist
                const bool use = lane < boxes && j < U.n && !(j >= sinks && j + box <= lo);
                const bool bad = use && (page < 0 || page >= C.num_pages);
                if (bad) atomicCAS(s_status, 0, KV_ERR_INVALID_ARG);
                // rows past the pools' end read as zero
                const long long y = bad ? C.num_pages * C.ps
                                        : ((long long)page << C.ps_log2) + (j & (C.ps - 1));
                const int n_use = __popc(__ballot_sync(0xffffffffu, use));
                const int s = cnt % kSt;
                ok = mbar_wait(&empty[s], (uint32_t)((cnt / kSt) & 1) ^ 1u, s_abort, C.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    if (n_use) mbar_arrive_expect_tx(&full[s], n_use * box * 128);
                    else mbar_arrive(&full[s]);
                }
                __syncwarp();
                if (use)
                    tma_load_2d(smem + s * Ly::kStage + kv * Ly::kOp + half * kHalfBytes +
                                    sub * box * 128,
                                map, &full[s], half * 64, (int)y);
                ++cnt;
            }
            at += total;
            ++v;
        }
        if (!ok && lane == 0) {
            *s_abort = 1;
            atomicCAS(s_status, 0, KV_ERR_TIMEOUT);
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
        int v = run.unit, at = run.unit_begin;
        while (ok && at < run.end) {
            const UnitRows U = unit_rows(C, T, A.layer, v);
            const int rows = U.count * C.G;
            const bool mine = U.count > 0 && (long long)U.count * C.G <= NT * 8;
            const int t_lo = U.n - U.count, t_hi = U.n - 1;
            const TileSpan span = tile_span(A.M, t_lo, t_hi, 6);
            const int total = mine ? span.total : 0;
            const int x0 = max(run.begin - at, 0), x1 = min(total, run.end - at);
            if (x0 >= x1) {
                at += total;
                ++v;
                continue;
            }
            const int lo = window_lo(A.M, max(t_lo, 0)), sinks = min(A.M.sinks, lo);
            // Q^T: columns are query rows (those past the last are zero)
            uint32_t qf[NT][D / 16][2];
            float m[NT][2], l[NT][2], o[NT][D / 16][4];
            int t_row[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = nt * 8 + quad;
                const uint32_t *qp = nullptr;
                if (row < rows)
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
                    const int row2 = nt * 8 + pair + i;
                    t_row[nt][i] = row2 < rows ? t_lo + row2 / C.G : -1;
                }
            }
            for (int x = x0; x < x1; ++x) {
                const int tile = span.tile(x), key0 = tile * kFewTile;
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
                        for (int i = 0; i < 4; ++i) sc[nt][i] = (sc[nt][i] + s1[nt][i]) * cs;
                }
                const int last = key0 + kFewTile - 1;
                const bool all = last <= t_lo && (A.M.window == 0 || key0 > t_hi - A.M.window ||
                                                  last < A.M.sinks);
                if (!all) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = key0 + wk + quad + (i >> 1) * 8;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int t = t_row[nt][i & 1];
                            const bool see = j <= t && (A.M.window == 0 || j > t - A.M.window ||
                                                        j < A.M.sinks);
                            if (!see) sc[nt][i] = -INFINITY;
                        }
                    }
                    // V rows that no query sees may hold anything: 0 weight times NaN
#pragma unroll 1
                    for (int c = lane; c < 16 * (D / 8); c += 32) {
                        const int kr = wk + c / (D / 8), ch = c % (D / 8), j = key0 + kr;
                        if (j > t_hi || (j >= sinks && j < lo))
                            *reinterpret_cast<uint4 *>(vt + (ch >> 3) * kHalfBytes + kr * 128 +
                                                       (((ch & 7) ^ (kr & 7)) << 4)) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();   // before TMA fills the stage again
                    __syncwarp();
                }
                if (A.logits) {
                    float *lg = A.logits + ((long long)(at + x) * kFewRows) * kFewTile;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (nt * 8 + pair + (i & 1) < rows)
                                lg[(nt * 8 + pair + (i & 1)) * kFewTile + wk + quad + (i >> 1) * 8] =
                                    sc[nt][i];
                    if (warp == 0 && lane == 0) A.tile_at[at + x] = make_int2(v, tile);
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
            if (warp == 0) {
                const bool whole = x0 == 0 && x1 == total;
                const long long slot = part_slot(blockIdx.x, x0 == 0);
                if (lane == 0 && x0 > 0 && x1 == total)
                    *s_cut = CutItem{v, at / run.per, 0, rows};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int row = nt * 8 + pair + i;
                        if (row >= rows) continue;
                        const float mm = m[nt][i] - E::kShift, ll = l[nt][i];
                        if (whole) {
                            const long long tok = U.tok0 + row / C.G;
                            const int head = U.h * C.G + row % C.G;
                            const float inv = ll > 0.f ? 1.f / ll : 0.f;
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
                            const long long at_row = slot * kFewRows + row;
                            if (quad == 0) A.part_ml[at_row] = make_float2(mm, ll);
                            float *op = A.part_o + at_row * D + quad;
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks) {
                                op[ks * 16] = o[nt][ks][i];
                                op[ks * 16 + 8] = o[nt][ks][i + 2];
                            }
                        }
                    }
            }
            at += total;
            ++v;
        }
        if (!ok && lane == 0) {
            *s_abort = 1;
            atomicCAS(s_status, 0, KV_ERR_TIMEOUT);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        A.cta_status[blockIdx.x] = *s_status;
        A.cut[blockIdx.x] = *s_cut;
        if (blockIdx.x == 0 && A.logits) *A.tiles = run.total;
    }
}

// mass of the rows of every tile: sum over the unit's query rows of 2^(logit - lse), in
// row order.  One 64-thread group per tile, a thread per key.
constexpr int kMassThreads = 256;
__global__ void __launch_bounds__(kMassThreads)
few_mass_kernel(const DevPaged C, const DevChunk T, const FewArgs A) {
    pdl_wait();
    pdl_trigger();
    const int tiles = *A.tiles;
    constexpr int kGroups = kMassThreads / kFewTile;
    const int key = threadIdx.x % kFewTile;
    for (int t = blockIdx.x * kGroups + threadIdx.x / kFewTile; t < tiles;
         t += gridDim.x * kGroups) {
        const int2 where = A.tile_at[t];
        const UnitRows U = unit_rows(C, T, A.layer, where.x);
        const int j = where.y * kFewTile + key, rows = U.count * C.G;
        if (j >= U.n) continue;
        const float *lg = A.logits + (long long)t * kFewRows * kFewTile + key;
        const float *lse2 = A.lse2 + packed_row(C, U, 0);
        float acc = 0.f;
        bool seen = false;
        for (int row = 0; row < rows; ++row) {
            const float x = lg[row * kFewTile];
            if (x == -INFINITY) continue;
            seen = true;
            acc += ex2_approx(x - lse2[row]);
        }
        if (!seen) continue;
        const long long at = page_row(C, U.table, j);
        if (at >= 0) C.mass[at] += acc;
    }
}

template <typename E, int D, int NT>
cudaError_t few(const DevPaged &C, const DevChunk &T, const FewArgs &A, bool first,
                const AttendWs &ws, cudaStream_t s) {
    using Ly = Layout<D, NT>;
    CUtensorMap mk, mv;
    const int box = C.ps < kFewTile ? C.ps : kFewTile;
    if (!make_tile_map(&mk, C.k, C.num_pages * C.ps, D, box) ||
        !make_tile_map(&mv, C.v, C.num_pages * C.ps, D, box))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(few_kernel<E, D, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::kTotal);
    if (e == cudaSuccess)
        e = launch_dependent(few_kernel<E, D, NT>, dim3(kFewCtas), kThreads, Ly::kTotal, s, mk, mv,
                             C, T, A);
    if (e == cudaSuccess)
        e = launch_attend_merge(C, T, A.layer, A.io, A.lse2, ws, kFewCtas, kFewRows, first, s);
    if (e == cudaSuccess && A.logits)
        e = launch_dependent(few_mass_kernel, dim3(kFewCtas), kMassThreads, 0, s, C, T, A);
    return e;
}

}  // namespace

cudaError_t launch_attend_few(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                              const AttendIo &io, bool add_mass, int max_rows, bool first,
                              const AttendWs &ws, cudaStream_t s) {
    const FewArgs A{layer,      M,       io,       ws.cta_status, ws.cut,
                    ws.part_ml, ws.part_o, ws.lse2, ws.tiles,      ws.tile_at,
                    add_mass ? ws.logits : nullptr};
    const int nt = max_rows <= 8 ? 1 : 2;
    if (C.dtype == KV_FP16) {
        if (C.d == 64)
            return nt == 1 ? few<Fp16, 64, 1>(C, T, A, first, ws, s)
                           : few<Fp16, 64, 2>(C, T, A, first, ws, s);
        return nt == 1 ? few<Fp16, 128, 1>(C, T, A, first, ws, s)
                       : few<Fp16, 128, 2>(C, T, A, first, ws, s);
    }
    if (C.d == 64)
        return nt == 1 ? few<Bf16, 64, 1>(C, T, A, first, ws, s)
                       : few<Bf16, 64, 2>(C, T, A, first, ws, s);
    return nt == 1 ? few<Bf16, 128, 1>(C, T, A, first, ws, s)
                   : few<Bf16, 128, 2>(C, T, A, first, ws, s);
}

}  // namespace kvevict
