// kv_rotary.cu -- rotary positions: rows turned by the angles of their positions, alone
// (kv_rotary) or on the way into the pages (kv_paged_append_rotary).
//
// Pair i of a row at position p turns by a = p w_i:
//   (x1, x2) -> f (x1 cos a - x2 sin a, x1 sin a + x2 cos a)
// Bound by HBM: every row read once and written once, 32 bytes (eight pairs) a thread and
// step.  The angles belong to a token, not to a head, so a block takes whole tokens and its
// threads compute a token's cosines once, in shared memory, while the rows are on their way.
//
// p w_i in fp32 would be off by 0.06 at a position of a million: the angle is kept in turns,
// as 64 bits after the point.  w_i / 2 pi is taken once a block in fp64 and p times it modulo
// one turn is an integer product, exact but for the 53 bits of the factor (an angle off by at most
// p w_i 2^-52, 2^-21 at the last position); fp64 arithmetic per angle would cost as much as the
// copy does.  Half turns in fp32 (24 bits) then go through sincospif.
#include "kv_paged_attend.cuh"
#include "kv_rotary.cuh"

namespace kvevict {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 8;        // tokens a block takes together
constexpr int kMostPairs = 64;        // d / 2

// Frequencies of the block in turns a position, as 64 bits after the point.
__device__ __forceinline__ void load_turns(const DevRotary &A, unsigned long long *s_turn) {
    const int i = threadIdx.x;
    if (i < A.dims / 2) {
        // what is above the point are whole turns of a whole position
        double t = (double)A.inv_freq[i] * 0.15915494309189535;
        t -= floor(t);
        s_turn[i] = (unsigned long long)(t * 18446744073709551616.0);
    }
}

// Cosine and sine (times the factor) of position p and frequency `turn`.
__device__ __forceinline__ float2 turn_of(const DevRotary &A, unsigned long long turn, int p) {
    const unsigned long long phase = (unsigned long long)(long long)p * turn;
    const float x = (float)(int)(phase >> 32) * 4.656612873077393e-10f;      // half turns
    float2 cs;
    sincospif(x, &cs.y, &cs.x);
    cs.x *= A.factor;
    cs.y *= A.factor;
    return cs;
}

// A row's 16 elements of unit i as two vectors, at a() and b().  Turned units come first: with
// halves paired, elements 8 i and dims / 2 + 8 i; the others are neighbours.
template <bool kInter>
struct Unit {
    int a, b, pair;                   // vectors of the row; the first pair
    bool turned;
    __device__ __forceinline__ Unit(int i, int dims) {
        turned = i * 16 < dims;
        pair = 8 * i;
        const bool apart = !kInter && turned;
        a = apart ? i : 2 * i;
        b = apart ? i + dims / 16 : 2 * i + 1;
    }
};

template <typename E, bool kInter>
__device__ __forceinline__ void turn_unit(uint4 &x, uint4 &y, const float2 *cs) {
    uint32_t *xw = reinterpret_cast<uint32_t *>(&x), *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float2 u = E::unpack(xw[w]), v = E::unpack(yw[w]);
        if (kInter) {
            const float2 c = cs[w], e = cs[w + 4];
            u = make_float2(u.x * c.x - u.y * c.y, u.x * c.y + u.y * c.x);
            v = make_float2(v.x * e.x - v.y * e.y, v.x * e.y + v.y * e.x);
        } else {
            const float2 c = cs[2 * w], e = cs[2 * w + 1];
            const float2 s = u, t = v;
            u = make_float2(s.x * c.x - t.x * c.y, s.y * e.x - t.y * e.y);
            v = make_float2(s.x * c.y + t.x * c.x, s.y * e.y + t.y * e.x);
        }
        xw[w] = E::pack(u.x, u.y);
        yw[w] = E::pack(v.x, v.y);
    }
}

// The block's loop over groups of tokens: `angles` fills the table of a group and `rows` moves its
// units.  Two tables, so that one barrier a group is enough.
template <typename F>
__device__ __forceinline__ void for_groups(const DevRotary &A, long long tokens, int group,
                                           const int32_t *positions, F rows) {
    __shared__ unsigned long long s_turn[kMostPairs];
    __shared__ float2 s_cs[2][kMostTokens][kMostPairs];
    const int half = A.dims / 2;
    load_turns(A, s_turn);
    __syncthreads();
    int which = 0;
    for (long long t0 = (long long)blockIdx.x * group; t0 < tokens;
         t0 += (long long)gridDim.x * group, which ^= 1) {
        const int n = (int)min((long long)group, tokens - t0);
        rows(t0, n, s_cs[which], [&]() {
            for (int i = threadIdx.x; i < n * half; i += kThreads) {
                const int t = i / half, k = i - t * half;
                float2 cs = turn_of(A, s_turn[k], positions[t0 + t]);
                if (A.backward) cs.y = -cs.y;
                s_cs[which][t][k] = cs;
            }
            __syncthreads();
        });
    }
}

constexpr int kUnroll = 3;            // units in flight a thread

template <typename E, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4)
rotary_kernel(const DevRotary A, long long tokens, int heads, int group,
              const int32_t *positions, const uint4 *x, long long x_tok,
              long long x_head, uint4 *out, long long out_tok, long long out_head) {
    constexpr int kU = D / 16;
    pdl_wait();
    pdl_trigger();
    for_groups(A, tokens, group, positions,
               [&](long long t0, int n, const float2 (*cs)[kMostPairs], auto angles) {
                   const int per = heads * kU, all = n * per;
                   bool ready = false;
                   for (int i0 = threadIdx.x; i0 < all || !ready; i0 += kThreads * kUnroll) {
                       uint4 a[kUnroll], b[kUnroll];
                       int tk[kUnroll], hd[kUnroll], un[kUnroll];
#pragma unroll
                       for (int q = 0; q < kUnroll; ++q) {
                           const int i = i0 + q * kThreads;
                           tk[q] = i / per;
                           hd[q] = (i - tk[q] * per) / kU;
                           un[q] = i % kU;
                           if (i >= all) continue;
                           const Unit<kInter> u(un[q], A.dims);
                           const uint4 *src = x + (t0 + tk[q]) * x_tok + hd[q] * x_head;
                           a[q] = src[u.a];
                           b[q] = src[u.b];
                       }
                       if (!ready) angles();
                       ready = true;
#pragma unroll
                       for (int q = 0; q < kUnroll; ++q) {
                           if (i0 + q * kThreads >= all) continue;
                           const Unit<kInter> u(un[q], A.dims);
                           if (u.turned) turn_unit<E, kInter>(a[q], b[q], &cs[tk[q]][u.pair]);
                           uint4 *dst = out + (t0 + tk[q]) * out_tok + hd[q] * out_head;
                           dst[u.a] = a[q];
                           dst[u.b] = b[q];
                       }
                   }
               });
}

// Request of token `tok`, by a warp: 32 offsets at a time.
__device__ __forceinline__ int request_by_warp(const DevChunk &T, int R, long long tok) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int n = __popc(__ballot_sync(0xffffffffu, at < hi && T.off[at] <= tok));
        lo += max(n - 1, 0) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Rows of a token: Hq query heads, then H of K, then H of V.
template <typename E, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4)
append_rotary_kernel(const DevPaged C, const DevChunk T, int layer, const DevRotary A, int group,
                     const int32_t *positions, int32_t *row_pos, const AppendIo io) {
    constexpr int kU = D / 16;
    __shared__ int s_req[kMostTokens];
    pdl_wait();
    pdl_trigger();
    const int Hq = io.q ? C.Hq : 0;
    for_groups(A, T.tokens, group, positions,
               [&](long long t0, int n, const float2 (*cs)[kMostPairs], auto angles) {
                   const int per = (Hq + 2 * C.H) * kU, all = n * per;
                   bool ready = false;
                   for (int i0 = threadIdx.x; i0 < all || !ready; i0 += kThreads * kUnroll) {
                       uint4 a[kUnroll], b[kUnroll];
                       int tk[kUnroll], hd[kUnroll], un[kUnroll];
#pragma unroll
                       for (int q = 0; q < kUnroll; ++q) {
                           const int i = i0 + q * kThreads;
                           tk[q] = i / per;
                           hd[q] = (i - tk[q] * per) / kU;
                           un[q] = i % kU;
                           if (i >= all) continue;
                           const Unit<kInter> u(un[q], A.dims);
                           const long long tok = t0 + tk[q];
                           const int h = hd[q] - Hq;
                           const uint4 *src =
                               h < 0 ? io.q + tok * io.q_stride + hd[q] * (D / 8)
                               : h < C.H ? io.k + tok * io.k_stride + h * (D / 8)
                                         : io.v + tok * io.v_stride + (h - C.H) * (D / 8);
                           a[q] = src[u.a];
                           b[q] = src[u.b];
                       }
                       if (!ready) {
                           const int warp = threadIdx.x >> 5;
                           if (warp < n) {
                               const int r = request_by_warp(T, C.R, t0 + warp);
                               if ((threadIdx.x & 31) == 0) s_req[warp] = r;
                           }
                           angles();
                       }
                       ready = true;
#pragma unroll
                       for (int q = 0; q < kUnroll; ++q) {
                           if (i0 + q * kThreads >= all) continue;
                           const Unit<kInter> u(un[q], A.dims);
                           const long long tok = t0 + tk[q];
                           const int h = hd[q] - Hq;
                           if (u.turned && h < C.H)
                               turn_unit<E, kInter>(a[q], b[q], &cs[tk[q]][u.pair]);
                           uint4 *dst;
                           if (h < 0) {
                               dst = io.q_out + tok * io.q_out_stride + hd[q] * (D / 8);
                           } else {
                               const int r = s_req[tk[q]], head = h < C.H ? h : h - C.H;
                               if (tok >= T.off[C.R]) continue;
                               const long long v = ((long long)r * C.L + layer) * C.H + head;
                               int len;
                               const bool ok = unit_len(C, v, len);
                               const long long j = len - (T.off[r + 1] - tok);
                               if (ok && j < 0) continue;
                               const long long row =
                                   ok ? page_row(C, C.table + v * C.max_pages, (int)j) : -1;
                               if (row < 0) {
                                   post_status(C.status, KV_ERR_INVALID_ARG);
                                   continue;
                               }
                               if (h < C.H && un[q] == 0) {
                                   if (C.mass) C.mass[row] = 0.f;
                                   if (row_pos) row_pos[row] = positions[tok];
                               }
                               dst = static_cast<uint4 *>(h < C.H ? C.k : C.v) + row * (D / 8);
                           }
                           dst[u.a] = a[q];
                           dst[u.b] = b[q];
                       }
                   }
                   // the next group's requests overwrite these
                   __syncthreads();
               });
}

// Tokens a block takes together: enough units for its threads' first step.
int group_of(int rows, int d) {
    const int g = kThreads / (rows * (d / 16));
    return g < 1 ? 1 : g > kMostTokens ? kMostTokens : g;
}
unsigned grid_of(long long tokens, int group) {
    const long long n = (tokens + group - 1) / group;
    return (unsigned)(n < kRotaryCtas ? n : kRotaryCtas);
}

template <typename E, int D, bool kInter>
cudaError_t rotary(const DevRotary &A, long long tokens, int heads, const int32_t *positions,
                   const RotaryIo &io, cudaStream_t s) {
    const int group = group_of(heads, D);
    return launch_dependent(rotary_kernel<E, D, kInter>, dim3(grid_of(tokens, group)), kThreads, 0,
                            s, A, tokens, heads, group, positions, io.x, io.x_tok, io.x_head,
                            io.out, io.out_tok, io.out_head);
}

template <typename E, int D, bool kInter>
cudaError_t append(const DevPaged &C, const DevChunk &T, int layer, const DevRotary &A,
                   const int32_t *positions, int32_t *row_pos, const AppendIo &io, cudaStream_t s) {
    const int group = group_of((io.q ? C.Hq : 0) + 2 * C.H, D);
    return launch_dependent(append_rotary_kernel<E, D, kInter>, dim3(grid_of(T.tokens, group)),
                            kThreads, 0, s, C, T, layer, A, group, positions, row_pos, io);
}

}  // namespace

cudaError_t launch_rotary(const DevRotary &A, long long tokens, int heads, int d, int dtype,
                          const int32_t *positions, const RotaryIo &io, cudaStream_t s) {
    auto go = [&](auto e, auto inter) {
        using E = decltype(e);
        constexpr bool kInter = decltype(inter)::value;
        return d == 64 ? rotary<E, 64, kInter>(A, tokens, heads, positions, io, s)
                       : rotary<E, 128, kInter>(A, tokens, heads, positions, io, s);
    };
    if (dtype == KV_FP16)
        return A.interleaved ? go(Fp16{}, std::true_type{}) : go(Fp16{}, std::false_type{});
    return A.interleaved ? go(Bf16{}, std::true_type{}) : go(Bf16{}, std::false_type{});
}

cudaError_t launch_append_rotary(const DevPaged &C, const DevChunk &T, int layer, const DevRotary &A,
                                 const int32_t *positions, int32_t *row_pos, const AppendIo &io,
                                 cudaStream_t s) {
    auto go = [&](auto e, auto inter) {
        using E = decltype(e);
        constexpr bool kInter = decltype(inter)::value;
        return C.d == 64 ? append<E, 64, kInter>(C, T, layer, A, positions, row_pos, io, s)
                         : append<E, 128, kInter>(C, T, layer, A, positions, row_pos, io, s);
    };
    if (C.dtype == KV_FP16)
        return A.interleaved ? go(Fp16{}, std::true_type{}) : go(Fp16{}, std::false_type{});
    return A.interleaved ? go(Bf16{}, std::true_type{}) : go(Bf16{}, std::false_type{});
}

}  // namespace kvevict
