// kv_pages.cuh -- who holds which page of a paged cache: the kernels' workspaces and launchers
// (not part of the ABI).
#pragma once

#include "kv_paged.cuh"

namespace kvevict {

// The plans run as one cluster of kPlanCtas blocks: their counts meet in distributed shared memory,
// so that a plan is one launch.
constexpr int kPlanCtas = 8, kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyCtas = 8 * 152;

struct PagePlan {
    int count;                 // compaction: pages moved; reservation: whether all fit
    int live;                  // compaction: pages in use
};
// What a unit gets: `pages` pages from list[at] on, entered from column `col` on; the first takes the
// place of page `from`, whose copy it is (-1: none is copied).
struct alignas(16) UnitNeed {
    int at, pages, from, col;
};

// Workspace of a reservation or compaction (offsets 256-byte aligned).
struct PagesWs {
    PagePlan *plan;
    int *list;                 // reservation: free pages; compaction: which to move a page is, or -1
    UnitNeed *need;            // reservation
    int *src, *dst;            // compaction: pages to move, holes
    size_t total;
};
PagesWs reserve_ws_layout(const DevPaged &C, void *base);
PagesWs compact_ws_layout(const DevPaged &C, void *base);

// Requests whose columns a block of the fork can stage.
constexpr int kForkRequests = 16384;

cudaError_t launch_count_refs(const DevPaged &C, int32_t *refs, cudaStream_t s);
cudaError_t launch_reserve(const DevPaged &C, const DevChunk &T, int32_t *refs, int32_t *row_pos,
                           const PagesWs &ws, cudaStream_t s);
cudaError_t launch_fork(const DevPaged &C, int32_t *refs, const int32_t *parents, cudaStream_t s);
cudaError_t launch_compact_pages(const DevPaged &C, int32_t *refs, int32_t *row_pos, int32_t *live,
                                 const PagesWs &ws, cudaStream_t s);
cudaError_t launch_place_positions(const DevPaged &D, int32_t *dst_pos, const DevPaged &S,
                                   const int32_t *src_pos, const int32_t *index, long long stride,
                                   const int64_t *offsets, cudaStream_t s);

}  // namespace kvevict
