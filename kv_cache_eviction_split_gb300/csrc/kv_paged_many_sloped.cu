// kv_paged_many_sloped.cu -- the many-rows kernel (kv_paged_many.cu) of scores lowered by distance.
//
// Bound by the row warps, whose logits pass through tensor memory once more than plain ones do.  32 query
// heads on 8, d = 128, bf16: 2048 tokens over 34816 rows with positions 1013 us, 1.12 PFLOP/s (plain 699); a
// prompt of 8192 tokens 527 us, in 5 documents 194.
#include "kv_paged_many.cuh"

namespace kvevict {

cudaError_t launch_attend_many_sloped(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s) {
    return attend_many<kBounds | kSloped>(C, T, layer, M, form, io, ws, s);
}

}  // namespace kvevict
