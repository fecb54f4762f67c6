// kv_paged_attention.cu -- attention of new tokens over the pages: which kernel takes a
// request (few or many query rows a head), the merge of items that several CTAs held, and
// the workspace they share.
#include <algorithm>

#include "kv_paged_attend.cuh"
#include "kv_paged_scores.cuh"

namespace kvevict {
namespace {

// ---------------------------------------------------------------------------
// Merge of the many-rows kernel's cut items.  The CTA that held an item's last tile left
// its description; block (b, y) merges rows of CTA b's item of every phase.  Partials are
// added in order: the result does not depend on timing.  A partial that saw nothing
// (m = -inf) has no output written.  Its inputs are not __restrict__: the kernel before
// writes them while this one may already run, and loads through restricted pointers need not
// stay behind the wait for it.
// ---------------------------------------------------------------------------
// Up to 256 rows, few partials: kMergeRows rows a warp, their loads together; 14 us for 152 cut
// items of 256 rows, d = 128, 40 MB of partials (18 us with a block for every phase's slot, most of
// them empty).  Whole calls, us, with the first two partials behind the maxima and 4 rows / beside
// them and 4 / 2 / 1 / 8 rows: 2048 tokens over 34816 rows 702 / 699 / 695 / 694 / 707; 8192 tokens
// in 5 documents, capped, 212 / 210 / 209 / 209 / 215; 2 x 511 tokens with weights, 16 units, 430 / 427 /
// 436 / 442.
constexpr int kMergeRows = 4;
template <typename X, int D>
__global__ void __launch_bounds__(128)
merge_many_kernel(const DevPaged C, const DevChunk T, int layer, const AttendIo io, float *lse2,
                  const CutItem *cut, const float2 *part_ml, const float *part_o, int phases) {
    constexpr int kV = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int row0 = ((int)blockIdx.y * 4 + warp) * kMergeRows;
    for (int g = 0; g < phases; ++g) {
        const int last = g * kManyCtas + (int)blockIdx.x;
        const CutItem it = cut[last];
        if (it.unit < 0 || row0 >= it.rows) continue;
        const int parts = last - it.cta0 + 1;
        auto slot_row = [&](int p, int r) {
            return (long long)part_slot(it.cta0 + p, p == 0) * kManyRows +
                   min(row0 + r, it.rows - 1);
        };
        float m[kMergeRows], l[kMergeRows], acc[kMergeRows][kV];
#pragma unroll
        for (int r = 0; r < kMergeRows; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[r][i] = 0.f;
        }
        auto fetch = [&](int p, float2 (&ml)[kMergeRows], float (&x)[kMergeRows][kV]) {
#pragma unroll
            for (int r = 0; r < kMergeRows; ++r) {
                const long long at = slot_row(p, r);
                ml[r] = part_ml[at];
                if constexpr (kV == 4)
                    *reinterpret_cast<float4 *>(x[r]) =
                        *reinterpret_cast<const float4 *>(part_o + at * D + lane * kV);
                else
                    *reinterpret_cast<float2 *>(x[r]) =
                        *reinterpret_cast<const float2 *>(part_o + at * D + lane * kV);
            }
        };
        auto add = [&](const float2 (&ml)[kMergeRows], const float (&x)[kMergeRows][kV]) {
#pragma unroll
            for (int r = 0; r < kMergeRows; ++r) {
                const float f = shrink(ml[r].x, m[r]);
                l[r] += ml[r].y * f;
#pragma unroll
                for (int i = 0; i < kV; ++i) acc[r][i] += f == 0.f ? 0.f : x[r][i] * f;
            }
        };
        // a cut item has two parts at least: theirs come beside the maxima
        float2 ml0[kMergeRows], ml1[kMergeRows];
        float o0[kMergeRows][kV], o1[kMergeRows][kV];
        fetch(0, ml0, o0);
        fetch(1, ml1, o1);
#pragma unroll
        for (int r = 0; r < kMergeRows; ++r) m[r] = fmaxf(ml0[r].x, ml1[r].x);
        for (int p = 2; p < parts; ++p)
#pragma unroll
            for (int r = 0; r < kMergeRows; ++r) m[r] = fmaxf(m[r], part_ml[slot_row(p, r)].x);
        add(ml0, o0);
        add(ml1, o1);
        for (int p = 2; p < parts; ++p) {
            fetch(p, ml0, o0);
            add(ml0, o0);
        }
#pragma unroll
        for (int r = 0; r < kMergeRows; ++r)
            if (row0 + r < it.rows)
                store_merged<X, D>(C, T, layer, io, lse2, it, row0 + r, m[r], l[r], acc[r]);
    }
}

template <typename X, int D>
cudaError_t merge(const DevPaged &C, const DevChunk &T, int layer, const AttendIo &io, float *lse2,
                  const AttendWs &ws, int phases, cudaStream_t s) {
    return launch_dependent(merge_many_kernel<X, D>,
                            dim3(kManyCtas, kManyRows / (4 * kMergeRows)), 128, 0, s, C, T, layer,
                            io, lse2, ws.cut, ws.part_ml, ws.part_o, phases);
}

}  // namespace

cudaError_t launch_many_merge(const DevPaged &C, const DevChunk &T, int layer, const AttendIo &io,
                              float *lse2, const AttendWs &ws, int phases, cudaStream_t s) {
    if (C.dtype == KV_FP16)
        return C.d == 64 ? merge<Fp16, 64>(C, T, layer, io, lse2, ws, phases, s)
                         : merge<Fp16, 128>(C, T, layer, io, lse2, ws, phases, s);
    return C.d == 64 ? merge<Bf16, 64>(C, T, layer, io, lse2, ws, phases, s)
                     : merge<Bf16, 128>(C, T, layer, io, lse2, ws, phases, s);
}

namespace {
// Which kernels take the step's requests.
struct Classes {
    int few_max;               // most query rows a head of the few-rows kernels
    int few_requests, max_rows, blocks;   // rows and row blocks of the largest of them
    long long items;           // their items
    int many;                  // the others
};
// seen: most rows of a unit that the step's queries see.
Classes classify(const DevPaged &C, const DevChunk &T, long long seen, bool add_mass, bool scored) {
    auto with = [&](int few_max) {
        Classes k{};
        k.few_max = few_max;
        k.blocks = 1;
        for (int r = 0; r < C.R; ++r) {
            const long long rows = (T.host_off[r + 1] - T.host_off[r]) * C.G;
            if (rows > few_max) {
                ++k.many;
            } else if (rows > 0) {
                const int blocks = (int)(rows + kFewRows - 1) / kFewRows;
                ++k.few_requests;
                k.max_rows = std::max(k.max_rows, (int)rows);
                k.blocks = std::max(k.blocks, blocks);
                k.items += (long long)blocks * C.H;
            }
        }
        return k;
    };
    if (seen <= kShortRows && !add_mass) {
        const Classes k = with(scored ? kShortScoredRows : kShortFewRows);
        if (k.items <= kFewCtas && k.items * ((seen + kFewTile - 1) / kFewTile) <= kShortVisits)
            return k;
    }
    return with(kFewRows);
}
}  // namespace

namespace {
// Blocks of 128 query rows to a unit.
int unit_blocks(const DevPaged &C, const DevChunk &T) {
    return (int)(((long long)T.max_t * C.G + 127) / 128);
}
}  // namespace

AttendWs attend_ws_layout(const DevPaged &C, const DevChunk &T, bool add_mass, void *base,
                          bool bounds) {
    AttendWs ws{};
    char *b = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = b ? b + off : nullptr;
        off = (off + bytes + 255) / 256 * 256;
        return p;
    };
    // whatever the window: a call without one needs most
    const Classes k = classify(C, T, C.cap, add_mass, false);
    // the two kernels run one after the other: they share the partials (scored calls take the
    // many-rows kernel for no more steps than others, which they may turn out to be)
    const bool cut_few = k.few_requests && C.cap > kShortRows;
    const size_t slots = std::max<size_t>(cut_few ? 2 * kFewCtas * (size_t)kFewRows : 0,
                                          k.many ? 2 * (size_t)many_phases(C) * kManyCtas * kManyRows : 0);
    ws.cut = reinterpret_cast<CutItem *>(take(std::max(kFewCtas, kManyCtas * kMaxPhases) * sizeof(CutItem)));
    ws.unit_cut = reinterpret_cast<int *>(take((size_t)C.R * C.H * sizeof(int)));
    ws.part_ml = reinterpret_cast<float2 *>(take(slots * sizeof(float2)));
    ws.part_o = reinterpret_cast<float *>(take(slots * C.d * sizeof(float)));
    if (add_mass) {
        const size_t tiles = (size_t)C.R * C.H * ((C.cap + kFewTile - 1) / kFewTile);
        ws.lse2 = reinterpret_cast<float *>(take((size_t)T.tokens * C.Hq * sizeof(float)));
        ws.q_packed = take(k.many ? (size_t)T.tokens * C.Hq * C.d * 2 : 0);
        ws.logits = reinterpret_cast<float *>(
            take(k.few_requests ? tiles * k.max_rows * kFewTile * sizeof(float) : 0));
    }
    if (bounds) {
        ws.rows = reinterpret_cast<RowBounds *>(take((size_t)T.tokens * C.H * sizeof(RowBounds)));
        ws.blocks = reinterpret_cast<BlockBounds *>(
            take((size_t)C.R * C.H * unit_blocks(C, T) * sizeof(BlockBounds)));
    }
    ws.total = off;
    return ws;
}

namespace {
// Most rows of a unit that a step's queries see; a window's rows and the sinks' may begin and
// end inside a tile.
long long rows_seen(const DevPaged &C, const DevChunk &T, const AttendMask &M) {
    return M.window > 0 ? std::min<long long>(C.cap, (long long)M.window + M.sinks + T.max_t +
                                                         2 * kFewTile)
                        : C.cap;
}
}  // namespace

bool attend_tiles_fit(const DevPaged &C, const DevChunk &T, const AttendMask &M, bool add_mass) {
    const long long seen = rows_seen(C, T, M), few_tiles = seen / kFewTile + 2;
    const long long many_tiles = seen / kManyTile + 2;
    const long long groups = C.cap / (2 * kManyTile) + 1;      // of the weights' pass
    double few = 0, many = 0, weights = 0;
    for (int r = 0; r < C.R; ++r) {
        const long long rows = (T.host_off[r + 1] - T.host_off[r]) * C.G;
        if (rows == 0) continue;
        few += (double)C.H * (few_tiles + kFewCost);
        many += (double)C.H * (rows / kManyRows + 1) * (many_tiles + kManyCost);
        weights += (double)C.H * groups * (rows / 128 + 1 + kManyCost);
    }
    // the count is rounded up to a whole number of tiles for each CTA
    const double most = 2147483647.0 - std::max(kFewCtas, kManyCtas);
    return few <= most && many <= most && (!add_mass || weights <= most);
}

bool attend_few_only(const DevPaged &C, const DevChunk &T) {
    return (long long)T.max_t * C.G <= kFewRows;
}

namespace {
// form: null for plain scores.
cudaError_t attend(const DevPaged &C, const DevChunk &T0, int layer, const AttendMask &M,
                   const ScoreForm *form, const AttendIo &io, bool add_mass, const AttendWs &ws,
                   cudaStream_t s) {
    const long long seen = rows_seen(C, T0, M);
    const Classes k = classify(C, T0, seen, add_mass, form != nullptr);
    DevChunk T = T0;
    T.few_max = k.few_max;
    cudaError_t e = cudaSuccess;
    if (k.few_requests)
        e = form ? launch_attend_few_scored(C, T, layer, M, *form, io, add_mass, seen, k.items,
                                            k.max_rows, k.blocks, ws, s)
                 : launch_attend_few(C, T, layer, M, io, add_mass, seen, k.items, k.max_rows,
                                     k.blocks, ws, s);
    if (e == cudaSuccess && k.many) {
        e = form ? launch_attend_many_scored(C, T, layer, M, *form, io, ws, s)
                 : launch_attend_many(C, T, layer, M, io, ws, s);
        // (changed scores: kv_paged_attention_scored refuses add_mass for such steps)
        if (e == cudaSuccess && add_mass) e = launch_many_mass(C, T, layer, M, ws, s);
    }
    return e;
}
}  // namespace

cudaError_t launch_paged_attention(const DevPaged &C, const DevChunk &T, int layer,
                                   const AttendMask &M, const AttendIo &io, bool add_mass,
                                   const AttendWs &ws, cudaStream_t s) {
    return attend(C, T, layer, M, nullptr, io, add_mass, ws, s);
}

cudaError_t launch_paged_attention_scored(const DevPaged &C, const DevChunk &T, int layer,
                                          const AttendMask &M, const ScoreForm &form0,
                                          const ScoreBounds &bounds, const AttendIo &io,
                                          bool add_mass, const AttendWs &ws, cudaStream_t s) {
    ScoreForm form = form0;
    if (bounds.first || bounds.last) {
        form.rows = ws.rows;
        form.blocks = ws.blocks;
        form.unit_blocks = unit_blocks(C, T);
        const cudaError_t e = launch_row_bounds(C, T, layer, M, bounds, ws.rows, ws.blocks,
                                                form.unit_blocks, s);
        if (e != cudaSuccess) return e;
    }
    return attend(C, T, layer, M, &form, io, add_mass, ws, s);
}

}  // namespace kvevict
