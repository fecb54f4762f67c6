// kv_paged_many.cu -- attention over the pages for more than 16 query rows a head (prompt
// chunks, whole prompts): bound by the tensor cores, 4 d flops per (query row, key).
//
// An item is 256 query rows of one unit (row i * G + g: token i, head g of the group, so
// that a group's heads share every K and V tile) and the 128-key tiles that any of them
// sees.  A CTA per SM works on two row tiles of 128 ("lanes"), each with S / P and O in
// tensor memory (4 x 128 columns):
//   S_L = Q_L K^T      128 x 128 x d, both operands in shared memory
//   P_L = 2^(S c - m)  a thread per row, all 128 logits in its registers: row max and sum
//                      need no exchange; P is rounded once to the pools' type and
//                      overwrites S
//   O_L += P_L V       P from tensor memory, V as it lies in the page
// The issuing thread runs, per lane, P V of one tile and S of the next; while the tensor
// cores work for one lane, the other lane's four warps take their softmax.  O is rescaled
// only when a row's maximum rises by more than 2^8.
//
// One rounding of P (at most 2^-8 relative in bf16, random signs) adds to an output about as much as
// its own rounding does; two parts, as in the few-rows kernel, would cost half as many
// products again in the kernel's bottleneck.
//
// Warps: 0 loads K and 2 loads V (page boxes by TMA, 3- and 2-tile rings, a lane per
// box), 1 issues the products, 3 describes the items ahead, 4-7 and 8-11 are the lanes' rows;
// they also bring their Q rows into shared memory and write the output.  Tiles no lane sees
// are skipped.
//
// Measured (32 query heads on 8, d = 128, bf16): 2048 tokens over 67584 rows 1.46 ms, 1.52
// PFLOP/s, where the card's sustained library rate is 1.72 (it holds the clock to ~1.7 GHz);
// a prompt of 8192 tokens, window 4096, 340 us, 1.21 PFLOP/s: 6.7 items a CTA, whose ends
// cost about four tiles each (the last products, the output's stores: 12 us in all, the
// first softmax) and the masked halves of the tiles at the window's and diagonal's edges.
#include "kv_paged_many.cuh"

namespace kvevict {

cudaError_t launch_attend_many(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                               const AttendIo &io, const AttendWs &ws, cudaStream_t s) {
    return attend_many<kPlain>(C, T, layer, M, ScoreForm{}, io, ws, s);
}

}  // namespace kvevict
