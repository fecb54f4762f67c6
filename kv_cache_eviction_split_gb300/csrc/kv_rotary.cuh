// kv_rotary.cuh -- rotary positions as the kernels see them (not part of the ABI).
#pragma once
#include <type_traits>

#include "kv_paged.cuh"

namespace kvevict {

struct DevRotary {
    int dims, interleaved, backward;
    float factor;
    const float *inv_freq;     // device [dims / 2]
};

// Strides count vectors of 8 elements.
struct RotaryIo {
    const uint4 *x;
    long long x_tok, x_head;
    uint4 *out;                // may be x
    long long out_tok, out_head;
};
struct AppendIo {
    const uint4 *q;            // null: K and V alone
    long long q_stride;
    uint4 *q_out;
    long long q_out_stride;
    const uint4 *k, *v;
    long long k_stride, v_stride;
};

// Blocks that a step's tokens are spread over before a block takes more than one: two an SM.
constexpr long long kRotarySpread = 152 * 2;
constexpr long long kRotaryCtas = 1 << 20;

cudaError_t launch_rotary(const DevRotary &A, long long tokens, int heads, int d, int dtype,
                          const int32_t *positions, const RotaryIo &io, cudaStream_t s);
cudaError_t launch_append_rotary(const DevPaged &C, const DevChunk &T, int layer, const DevRotary &A,
                                 const int32_t *positions, int32_t *row_pos, const AppendIo &io,
                                 cudaStream_t s);

}  // namespace kvevict
