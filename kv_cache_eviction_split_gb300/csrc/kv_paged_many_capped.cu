// kv_paged_many_capped.cu -- the many-rows kernel (kv_paged_many.cu) of scores capped by a tanh.
#include "kv_paged_many.cuh"

namespace kvevict {

cudaError_t launch_attend_many_capped(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s) {
    return form.slopes ? attend_many<kBounds | kCapped | kSloped>(C, T, layer, M, form, io, ws, s)
                       : attend_many<kBounds | kCapped>(C, T, layer, M, form, io, ws, s);
}

}  // namespace kvevict
