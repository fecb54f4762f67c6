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
//
// Two forms.  Long tables (kCluster = 0): all items' tiles cut into 304 equal runs, cut items
// merged by a second kernel (few_finish_kernel, which also adds the weights).  Short tables
// and windows (kCluster = 1 .. 8): a cluster per item, each CTA a part of its tiles, merged
// through distributed shared memory: one launch, which is what a short call costs; there an
// item's row block may also be one of several of a unit, each reading K and V again.
// kv_paged.cuh has the rules and what both forms take.
//
// Measured (d = 128, bf16, one layer's call).  HBM-bound: 8 requests of 4915 .. 39321 rows
// in 8 heads each 115 us (6.3 TB/s); 4 heads of 131072 rows, weights added, 67.6 us of which
// the tiles 47 (5.7 TB/s) and the finish 12; 16 requests, window 4096 of longer tables,
// 48 us (5.6 TB/s).  Latency-bound: 8 heads of 1638 rows 6.4 us on the GPU.  As products of
// 128-row tiles in tensor memory the same work would be padded 32 times over.
#include "kv_paged_few.cuh"

namespace kvevict {

cudaError_t launch_attend_few(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                              const AttendIo &io, bool add_mass, long long seen, long long items,
                              int max_rows, int blocks, const AttendWs &ws, cudaStream_t s) {
    return attend_few<false>(C, T, layer, M, ScoreForm{}, io, add_mass, seen, items, max_rows, blocks,
                             ws, s);
}

}  // namespace kvevict
