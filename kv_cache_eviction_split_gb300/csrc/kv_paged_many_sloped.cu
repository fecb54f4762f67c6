// kv_paged_many_sloped.cu -- the many-rows kernel (kv_paged_many.cu) of scores lowered by distance.
#include "kv_paged_many.cuh"

namespace kvevict {

cudaError_t launch_attend_many_sloped(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s) {
    return attend_many<kBounds | kSloped>(C, T, layer, M, form, io, ws, s);
}

}  // namespace kvevict
