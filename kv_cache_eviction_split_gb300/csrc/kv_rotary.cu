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
// p w_i 2^-52, 2^-21 at the last position for w_i = 1); fp64 arithmetic per angle would cost as much as
// the copy does.  Half turns in fp32 (24 bits: 2^-23 of an angle) then go through sincospif.
//
// Measured (d = 128, bf16): 8192 tokens of 32 + 8 + 8 heads into the pages 34 us, 5.9 TB/s, 88% of
// what a copy reaches; 2047 tokens of 28 heads (dims 64) 6.5 us, where a launch alone is 2.3; one
// token each of 8 requests 3.5 us.  Three units in flight a thread: two take 35 us, four 34.4 (registers).
#include "kv_paged_attend.cuh"
#include "kv_rotary.cuh"

namespace kvevict {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 8;        // tokens a block takes together
constexpr int kMostPairs = 64;        // d / 2
constexpr int kUnroll = 3;            // units in flight a thread

// x / d for 0 <= x < 2^31 with d's constant from the host.
struct FastDiv {
    unsigned mul, shift, d;
    explicit FastDiv(unsigned n) : d(n) {
        shift = 0;
        while ((1ull << shift) < n) ++shift;
        mul = (unsigned)(((1ull << 32) * ((1ull << shift) - n)) / n + 1);
    }
    __device__ __forceinline__ int operator()(int x) const {
        return (int)((__umulhi((unsigned)x, mul) + (unsigned)x) >> shift);
    }
};

// A row's 16 elements of unit i as two vectors, at a and b.  Turned units come first: with
// halves paired, elements 8 i and dims / 2 + 8 i; the others are neighbours.
template <bool kInter>
struct Unit {
    int a, b;
    bool turned;
    __device__ __forceinline__ Unit(int i, int dims) {
        turned = i * 16 < dims;
        const bool apart = !kInter && turned;
        a = apart ? i : 2 * i;
        b = apart ? i + dims / 16 : 2 * i + 1;
    }
};

// Cosines and sines of a token's pairs.  A unit reads four vectors of two pairs each: word w's pairs,
// which lie a unit apart, so that the threads of a row read side by side.
struct Angles {
    float4 cs[4][kMostPairs / 8];
};

template <typename E, bool kInter>
__device__ __forceinline__ void turn_unit(uint4 &x, uint4 &y, const Angles &A, int unit) {
    uint32_t *xw = reinterpret_cast<uint32_t *>(&x), *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float4 c = A.cs[w][unit];        // two pairs: (cos, sin) twice
        const float2 u = E::unpack(xw[w]), v = E::unpack(yw[w]);
        if (kInter) {
            xw[w] = E::pack(u.x * c.x - u.y * c.y, u.x * c.y + u.y * c.x);
            yw[w] = E::pack(v.x * c.z - v.y * c.w, v.x * c.w + v.y * c.z);
        } else {
            xw[w] = E::pack(u.x * c.x - v.x * c.y, u.y * c.z - v.y * c.w);
            yw[w] = E::pack(u.x * c.y + v.x * c.x, u.y * c.w + v.y * c.z);
        }
    }
}

// The angles of n tokens from t0 on, by all threads.  s_turn: frequencies in turns a position, 64
// bits after the point.
template <bool kInter>
__device__ __forceinline__ void fill_angles(const DevRotary &A, const FastDiv &by_half, int n,
                                            const int32_t *positions,
                                            const unsigned long long *s_turn, Angles *s_cs) {
    const int half = A.dims / 2;
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int t = by_half(i), k = i - t * half;
        const unsigned long long phase = (unsigned long long)(long long)positions[t] * s_turn[k];
        const float x = (float)(int)(phase >> 32) * 4.656612873077393e-10f;      // half turns
        float cos, sin;
        sincospif(x, &sin, &cos);
        if (A.backward) sin = -sin;
        const int j = k & 7, w = kInter ? j & 3 : j >> 1, second = kInter ? j >> 2 : j & 1;
        reinterpret_cast<float2 *>(&s_cs[t].cs[w][k >> 3])[second] =
            make_float2(cos * A.factor, sin * A.factor);
    }
}
__device__ __forceinline__ void load_turns(const DevRotary &A, unsigned long long *s_turn) {
    const int i = threadIdx.x;
    if (i < A.dims / 2) {
        // what is above the point are whole turns of a whole position
        double t = (double)A.inv_freq[i] * 0.15915494309189535;
        t -= floor(t);
        s_turn[i] = (unsigned long long)(t * 18446744073709551616.0);
    }
    __syncthreads();
}

// Rows of a group of tokens, kThreads / (D / 16) at a time: kUnroll of them on their way while the
// group's angles are taken.  place(row) says where a row of the group comes from, once `prepare` has
// run where it goes to (null: nowhere), and whether it is turned.  Two tables of angles, and of
// what `prepare` leaves, so that a barrier a group is enough.
template <typename E, int D, bool kInter, typename S, typename P, typename T>
__device__ __forceinline__ void turn_groups(const DevRotary &A, const FastDiv &by_half,
                                            const FastDiv &by_rows, long long tokens, int group,
                                            const int32_t *positions, S source, P prepare, T target) {
    constexpr int kU = D / 16, kSlots = kThreads / kU;
    __shared__ unsigned long long s_turn[kMostPairs];
    __shared__ Angles s_cs[2][kMostTokens];
    load_turns(A, s_turn);
    const int unit = threadIdx.x % kU, slot = threadIdx.x / kU;
    const Unit<kInter> u(unit, A.dims);
    int which = 0;
    for (long long t0 = (long long)blockIdx.x * group; t0 < tokens;
         t0 += (long long)gridDim.x * group, which ^= 1) {
        const int n = (int)min((long long)group, tokens - t0), all = n * (int)by_rows.d;
        bool ready = false;
        for (int r0 = slot; r0 < all || !ready; r0 += kSlots * kUnroll) {
            uint4 a[kUnroll], b[kUnroll];
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                const int row = r0 + q * kSlots;
                if (row >= all) continue;
                const int t = by_rows(row);
                const uint4 *src = source(t0 + t, row - t * (int)by_rows.d);
                a[q] = src[u.a];
                b[q] = src[u.b];
            }
            if (!ready) {
                prepare(t0, n, which);
                fill_angles<kInter>(A, by_half, n, positions + t0, s_turn, s_cs[which]);
                __syncthreads();
                ready = true;
            }
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                const int row = r0 + q * kSlots;
                if (row >= all) continue;
                const int t = by_rows(row);
                bool turned = u.turned;
                uint4 *dst = target(t0, t, row - t * (int)by_rows.d, unit, which, turned);
                if (turned) turn_unit<E, kInter>(a[q], b[q], s_cs[which][t], unit);
                if (!dst) continue;
                dst[u.a] = a[q];
                dst[u.b] = b[q];
            }
        }
    }
}

template <typename E, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4)
rotary_kernel(const DevRotary A, const FastDiv by_half, const FastDiv by_heads, long long tokens,
              int group, const int32_t *positions, const RotaryIo io) {
    pdl_wait();
    pdl_trigger();
    turn_groups<E, D, kInter>(
        A, by_half, by_heads, tokens, group, positions,
        [&](long long tok, int h) { return io.x + tok * io.x_tok + h * io.x_head; },
        [](long long, int, int) {},
        [&](long long t0, int t, int h, int, int, bool &) {
            return io.out + (t0 + t) * io.out_tok + h * io.out_head;
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

// Rows of a token: Hq query heads (or none), then H of K, then H of V.
constexpr int kMostHeads = 32;        // KV heads of a group's tokens whose places fit shared memory

template <typename E, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4)
append_rotary_kernel(const DevPaged C, const DevChunk T, int layer, const DevRotary A,
                     const FastDiv by_half, const FastDiv by_rows, int group,
                     const int32_t *positions, int32_t *row_pos, const AppendIo io) {
    constexpr int kVecs = D / 8;
    __shared__ int s_req[2][kMostTokens];
    __shared__ int s_row[2][kMostTokens][kMostHeads];        // pool rows; -1: nowhere
    pdl_wait();
    pdl_trigger();
    const int Hq = io.q ? C.Hq : 0;
    const bool none = without_rows(C);
    // Pool row of token tok's new row of head h, -1 if it has none.
    auto place = [&](int r, long long tok, int h) {
        const long long v = ((long long)r * C.L + layer) * C.H + h;
        int len;
        const bool ok = unit_len(C, v, len);
        const long long j = len - (T.off[r + 1] - tok);
        if (tok >= T.off[C.R] || (ok && j < 0) || none) return -1;
        const int row = ok ? (int)page_row(C, C.table + v * C.max_pages, (int)j) : -1;
        if (row < 0) post_status(C.status, KV_ERR_INVALID_ARG);
        return row;
    };
    turn_groups<E, D, kInter>(
        A, by_half, by_rows, T.tokens, group, positions,
        [&](long long tok, int i) {
            const int h = i - Hq;
            return h < 0     ? io.q + tok * io.q_stride + i * kVecs
                   : h < C.H ? io.k + tok * io.k_stride + h * kVecs
                             : io.v + tok * io.v_stride + (h - C.H) * kVecs;
        },
        [&](long long t0, int n, int which) {
            // a warp a token
            const int t = threadIdx.x >> 5, lane = threadIdx.x & 31;
            if (t >= n) return;
            const int r = request_by_warp(T, C.R, t0 + t);
            if (lane == 0) s_req[which][t] = r;
            if (lane < C.H && C.H <= kMostHeads) s_row[which][t][lane] = place(r, t0 + t, lane);
        },
        [&](long long t0, int t, int i, int unit, int which, bool &turned) -> uint4 * {
            const long long tok = t0 + t;
            const int h = i - Hq;
            if (h < 0) return io.q_out + tok * io.q_out_stride + i * kVecs;
            const bool is_k = h < C.H;
            turned = turned && is_k;
            const int head = is_k ? h : h - C.H;
            const int row = C.H <= kMostHeads ? s_row[which][t][head]
                                              : place(s_req[which][t], tok, head);
            if (row < 0) return nullptr;
            if (is_k && unit == 0) {
                if (C.mass) C.mass[row] = 0.f;
                if (row_pos) row_pos[row] = positions[tok];
            }
            return static_cast<uint4 *>(is_k ? C.k : C.v) + (long long)row * kVecs;
        });
}

// Tokens a block takes together: as many as let two blocks an SM take the step at once (a block's
// start, its frequencies and first loads, costs more than another token does: 1000 tokens of 40
// heads 4.7 us so, 6.2 with a block a token), and in longer steps as many as give a block's
// threads two angles each (8192 tokens of 40 heads 27.5 us, 28.0 with 8 a block, 28.3 with an angle each).
int group_of(long long tokens, int dims) {
    const long long g = (tokens + kRotarySpread - 1) / kRotarySpread;
    if (g <= kMostTokens) return (int)g;
    return dims < 64 ? kMostTokens : 2 * kThreads / dims;
}
unsigned grid_of(long long tokens, int group) {
    const long long n = (tokens + group - 1) / group;
    return (unsigned)(n < kRotaryCtas ? n : kRotaryCtas);
}
FastDiv by_half(const DevRotary &A) { return FastDiv(A.dims > 0 ? A.dims / 2 : 1); }

template <typename E, int D, bool kInter>
cudaError_t rotary(const DevRotary &A, long long tokens, int heads, const int32_t *positions,
                   const RotaryIo &io, cudaStream_t s) {
    const int group = group_of(tokens, A.dims);
    return launch_dependent(rotary_kernel<E, D, kInter>, dim3(grid_of(tokens, group)), kThreads, 0, s,
                            A, by_half(A), FastDiv(heads), tokens, group, positions, io);
}

template <typename E, int D, bool kInter>
cudaError_t append(const DevPaged &C, const DevChunk &T, int layer, const DevRotary &A,
                   const int32_t *positions, int32_t *row_pos, const AppendIo &io, cudaStream_t s) {
    const int group = group_of(T.tokens, A.dims);
    return launch_dependent(append_rotary_kernel<E, D, kInter>, dim3(grid_of(T.tokens, group)),
                            kThreads, 0, s, C, T, layer, A, by_half(A),
                            FastDiv((io.q ? C.Hq : 0) + 2 * C.H), group, positions, row_pos, io);
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
