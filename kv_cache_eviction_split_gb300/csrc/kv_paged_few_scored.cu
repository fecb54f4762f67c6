// kv_paged_few_scored.cu -- the few-rows kernels (kv_paged_few.cu) with scores capped, lowered by
// distance, or masked by rows of their own: a thread's four logits a tile and query column are
// changed in registers, between the products, where the kernel waits for HBM anyway.
#include "kv_paged_few.cuh"

namespace kvevict {

cudaError_t launch_attend_few_scored(const DevPaged &C, const DevChunk &T, int layer,
                                     const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                     bool add_mass, long long seen, long long items, int max_rows,
                                     int blocks, const AttendWs &ws, cudaStream_t s) {
    return attend_few<true>(C, T, layer, M, form, io, add_mass, seen, items, max_rows, blocks, ws, s);
}

}  // namespace kvevict
