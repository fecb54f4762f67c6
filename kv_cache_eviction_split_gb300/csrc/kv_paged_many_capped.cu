// kv_paged_many_capped.cu -- the many-rows kernel (kv_paged_many.cu) of scores capped by a tanh.
//
// Bound by the row warps: the cap's polynomial and the exponentials in turn (ScoreForm, cap_tier).  32 query
// heads on 8, d = 128, bf16: a prompt of 8192 tokens in 5 documents 212 us (masked alone 174), 2048 tokens
// over 34816 rows 1180 us, 0.96 PFLOP/s (plain 699); saturated, with the exact form, 285 and 1600; with
// slopes too 261 and 1510.
#include "kv_paged_many.cuh"

namespace kvevict {

cudaError_t launch_attend_many_capped(const DevPaged &C, const DevChunk &T, int layer,
                                      const AttendMask &M, const ScoreForm &form, const AttendIo &io,
                                      const AttendWs &ws, cudaStream_t s) {
    return form.slopes ? attend_many<kBounds | kCapped | kSloped>(C, T, layer, M, form, io, ws, s)
                       : attend_many<kBounds | kCapped>(C, T, layer, M, form, io, ws, s);
}

}  // namespace kvevict
