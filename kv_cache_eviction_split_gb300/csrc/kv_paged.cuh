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
    int *status;               // the cache's status word
    unsigned long long wait_ns;   // limit of the pipeline waits (kv_set_wait_limit_ns)
};

// The new tokens of a step.
struct DevChunk {
    const long long *off;      // device [R + 1]
    const long long *host_off; // host copy (host code only)
    long long tokens;          // off[R]
    int max_t;                 // most new tokens of one request
    int few_max;               // query rows a head (T * G) that the few-rows kernels take
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

// ---------------------------------------------------------------------------
// Attention: how the work is cut
// ---------------------------------------------------------------------------
// A work item is the query rows of one unit that share a kernel's row tile (a row
// is a query of the group: row i * G + g is token i, head g of the group); its work
// is the key tiles that any of the rows sees.  All items' tiles, one after another,
// are cut into equal runs, one per CTA, whatever the lengths: a CTA's run can end
// inside an item.  An item that one CTA holds is finished there; of a cut item
// every CTA writes a partial (row max, row sum, unnormalised output), and the CTA
// that holds its last tile leaves a description for the merge.  Everything is
// computed from device memory (lens, token offsets), so a captured call follows
// the lengths of each replay.

constexpr int kFewRows = 16;       // most query rows of an item of the few-rows kernels
constexpr int kFewTile = 64;       // keys per tile there
constexpr int kFewCtas = 2 * 152;  // two CTAs on each SM
constexpr int kFewCost = 3;        // an item's own cost in tiles (its merge and output)
// Tables of at most kShortRows rows, and windows that see no more of longer ones, take the
// few-rows kernel's one-launch form.  One new token, 8 KV heads of 4 query heads, d = 128,
// GPU time in us one-launch / cut and merged:
//   1 request   1024 rows 5.6 / 10.6   4096 8.0 / 11.3   8192 11.7 / 12.6   16384 18.5 / 16.8
//   64 requests 1024 rows 44 / 52      4096 148 / 161    8192 288 / 308
// Longer tables are cut: lengths that differ (30% of 16384 .. 131072 rows, 8 requests) then
// cost nothing.
constexpr int kShortRows = 8192;
// There the kernel also takes up to kShortFewRows query rows a head, in blocks of kFewRows
// that each read the keys again, while a step has no more than kFewCtas such items and
// kShortVisits key tiles over all of them (without add_mass).  In us, this / the many-rows
// kernel:  1 request   64 rows on 1024 keys 9.9 / 23.0   256 on 4096 35 / 44   512 on 4096 57 / 37
//          16 requests 64 rows on 1024 keys 38 / 28 (512 items)
constexpr int kShortFewRows = 512;
constexpr int kShortVisits = 8192;
constexpr int kManyTile = 128;     // keys per tile of the tensor-memory kernel
constexpr int kManyRows = 256;     // query rows per item there: two tiles of 128
constexpr int kManyCtas = 152;
// An item's own cost in tiles; a prompt of 8192 tokens, window 4096, in us by cost: 2 360,
// 3 351, 4 350, 5 351.
constexpr int kManyCost = 4;
// The many-rows kernel takes the units in up to kMaxPhases groups, one after another, each
// cut into runs over all CTAs: a group's rows (kPhaseBytes, where that gives few enough
// groups) stay in L2 while all its items read them.
constexpr int kMaxPhases = 4;
// A phase is worth its merge (~10 us) from kPhaseTiles tiles a CTA on (~200 us).
constexpr long long kPhaseBytes = 64ll << 20;
constexpr int kPhaseTiles = 128;
inline int many_phases(const DevPaged &C) {
    const long long bytes = (long long)C.R * C.H * C.cap * C.d * 4;
    const long long n = (bytes + kPhaseBytes - 1) / kPhaseBytes;
    return (int)(n < 1 ? 1 : n < kMaxPhases ? n : kMaxPhases);
}

// Key tiles of 2^log2 rows that the queries at cache rows t_lo .. t_hi see: the
// sinks' tiles [0, ns), then the window's from `first` on; `total` together, at least
// one (with t_hi < 0 nothing is seen and the one tile is empty).
struct TileSpan {
    int first, ns, total;
    __device__ __forceinline__ int tile(int x) const { return x < ns ? x : first + x - ns; }
};

__host__ __device__ __forceinline__ TileSpan tile_span(const AttendMask &M, int t_lo, int t_hi,
                                                       int log2) {
    TileSpan s{0, 0, 1};
    if (t_hi < 0) return s;
    const int lo = window_lo(M, t_lo > 0 ? t_lo : 0);
    const int sinks = M.sinks < lo ? M.sinks : lo;
    s.first = lo >> log2;
    s.ns = (sinks + (1 << log2) - 1) >> log2;
    if (s.ns > s.first) s.ns = s.first;
    s.total = s.ns + (t_hi >> log2) + 1 - s.first;
    return s;
}

// A cut item: unit of the layer (r * H + h), first of the CTAs that hold it (the last
// is the one whose slot this is), first query row and number of rows.
struct CutItem {
    int unit, cta0, row0, rows;
};

// Partials: CTA b (counted on through the phases) writes slot 2 b for an item begun by an
// earlier CTA and 2 b + 1 for one it begins and a later CTA ends.
__device__ __forceinline__ int part_slot(int cta, bool begun_here) {
    return 2 * cta + (begun_here ? 1 : 0);
}

// Workspace of the attention (all offsets 256-byte aligned).
struct AttendWs {
    CutItem *cut;              // [ctas], a set for each phase; unit -1: no item ends here that
                               // an earlier CTA began
    int *unit_cut;             // [R * H] few rows: the CTA whose `cut` is the unit's, or -1
    float2 *part_ml;           // [2 ctas][rows of an item] (m in log2 units, l)
    float *part_o;             // [2 ctas][rows of an item][d]
    // add_mass: log2 of the softmax sums of the query rows, and the rows themselves, in
    // packed order (packed_row)
    float *lse2;               // [tokens * Hq]
    void *q_packed;            // [tokens * Hq][d], of the requests the many-rows kernel takes
    // few rows with add_mass: the logits (log2 units, -inf unseen) of every tile of every
    // unit of the layer, in its span's order; rows: the most of a unit that these kernels take
    float *logits;             // [R * H][ceil(cap / kFewTile)][rows][kFewTile]
    size_t total;
};
AttendWs attend_ws_layout(const DevPaged &C, const DevChunk &T, bool add_mass, void *base);

struct AttendIo {
    const void *q;
    void *out;
    float *lse;                // or null
    long long q_stride, out_stride;
};

// Whether every kernel's count of tiles (as above, for units as long as their tables) fits
// in 32 bits.
bool attend_tiles_fit(const DevPaged &C, const DevChunk &T, const AttendMask &M, bool add_mass);
cudaError_t launch_paged_attention(const DevPaged &C, const DevChunk &T, int layer,
                                   const AttendMask &M, const AttendIo &io, bool add_mass,
                                   const AttendWs &ws, cudaStream_t s);

}  // namespace kvevict
