// kv_paged_few_scored.cu -- the few-rows kernels (kv_paged_few.cu) with scores capped, lowered by
// distance, or masked by rows of their own: a thread's four logits a tile and query column are
// changed in registers, between the products, where the kernel waits for HBM anyway.  Positions come
// with their boxes of K, 4 bytes a row more.
//
// Measured (d = 128, bf16): 8 requests of 4915 .. 39321 rows in 8 heads each, positions with
// gaps and slopes, 118 us, 6.2 TB/s, 92% of what a copy reaches (plain scores 115); 8 requests of 39000
// rows, capped, 190 us; 8 heads of 1638 rows, capped, 7.3 us on the GPU (plain 6.4); 300 tokens on 401
// rows, both ways in a prefix, 14 us with the bounds' 5.
#include "kv_paged_few.cuh"

namespace kvevict {

cudaError_t launch_attend_few_scored(const DevPaged &C, const DevChunk &T, int layer,
                                     const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                     bool add_mass, long long seen, long long items, int max_rows,
                                     int blocks, const AttendWs &ws, cudaStream_t s) {
    return attend_few<true>(C, T, layer, M, form, io, add_mass, seen, items, max_rows, blocks, ws, s);
}

}  // namespace kvevict
