// kv_paged_attend.cuh -- what the attention kernels share: dependent launches, element
// types, the cut of the work into equal runs of key tiles, and the merge's interface.
#pragma once
#include <cuda_fp16.h>

#include "kv_paged.cuh"
#include "kv_sm100.cuh"

namespace kvevict {

// Every kernel of a call is launched as a programmatic dependent of the one before it
// on the stream: its CTAs may be set up early, and wait here, before they touch
// memory, until everything the earlier kernels wrote is visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// cluster > 1: blocks in clusters of that many along x.
template <typename... A, typename... B>
cudaError_t launch_cluster_dependent(void (*kernel)(A...), int cluster, dim3 grid, int threads,
                                     size_t smem, cudaStream_t s, B... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<A>(args)...);
}
template <typename... A, typename... B>
cudaError_t launch_dependent(void (*kernel)(A...), dim3 grid, int threads, size_t smem,
                             cudaStream_t s, B... args) {
    return launch_cluster_dependent(kernel, 1, grid, threads, smem, s, args...);
}

// 16-bit elements: packing of two fp32 values (round to nearest), the first low.
struct Bf16 {
    using T = __nv_bfloat16;
    static constexpr bool kHalf = false;
    static constexpr float kShift = 0.f;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ T one(float x) { return __float2bfloat16_rn(x); }
};
// fp16 has a narrow exponent: weights are taken as 2^(x - m + 7), so that those down to
// 2^-31 of the largest keep a value (a row's maximum is followed to within 2^8: at most
// 2^15).  The factor is common to sums and products and is taken out with the maximum.
struct Fp16 {
    using T = __half;
    static constexpr bool kHalf = true;
    static constexpr float kShift = 7.f;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ T one(float x) { return __float2half_rn(x); }
};

constexpr float kLn2 = 0.6931471805599453f;
// A row's running maximum is raised only when a logit exceeds it by more than this
// (log2 units): sums and weights stay below 2^8 times the count, and the rescaling of
// the accumulators becomes rare.
constexpr float kLazyLog2 = 8.f;

// 2^(a - b) for a running maximum b >= a; 0 when nothing was seen yet.
__device__ __forceinline__ float shrink(float a, float b) {
    return a == -INFINITY ? 0.f : sm100::ex2_approx(a - b);
}

// Requests and rows of unit v = r * H + h of a layer.
struct UnitRows {
    int r, h, n, count;        // rows held, new tokens
    long long tok0;
    bool ok;                   // the length is one a table can hold
    const int32_t *table;
};
__device__ __forceinline__ UnitRows unit_rows(const DevPaged &C, const DevChunk &T, int layer,
                                              int v) {
    UnitRows U;
    U.r = v / C.H;
    U.h = v - U.r * C.H;
    U.tok0 = T.off[U.r];
    U.count = (int)(T.off[U.r + 1] - U.tok0);
    const long long u = ((long long)U.r * C.L + layer) * C.H + U.h;
    U.ok = unit_len(C, u, U.n);
    U.table = C.table + u * C.max_pages;
    return U;
}

// Whether the tensor-memory kernel takes a unit's rows (the few-rows kernels otherwise).
__device__ __forceinline__ bool many_rows(const DevPaged &C, const DevChunk &T,
                                          const UnitRows &U) {
    return (long long)U.count * C.G > T.few_max;
}

// Bits 0 .. n-1 (none for n <= 0).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Query row `row` of unit U in the workspace's packed order: units of a request one after
// another, rows of a unit together.
__device__ __forceinline__ long long packed_row(const DevPaged &C, const UnitRows &U, int row) {
    return U.tok0 * C.Hq + (long long)U.h * U.count * C.G + row;
}

// The run of tiles of one CTA, in the order of all units' parts' tiles.
struct CtaRun {
    int begin, end, per;       // tiles [begin, end) of all; tiles per CTA
    int unit, part;            // the part that holds tile `begin`, and its first tile
    int part_begin;
    int total;
};

// Cuts the tiles of all units of the layer into gridDim.x equal runs.  unit(v) reads what
// is needed of unit v; it consists of parts_of(unit) parts, part i of tiles_of(unit, i)
// tiles.  All kThreads threads call it: a thread sums up its units, or a warp one unit
// where there are few, and a warp finds the run's first part.  s_tiles: kThreads words of
// shared memory (TMA may write there afterwards).
template <int kThreads, typename U, typename P, typename F>
__device__ __forceinline__ CtaRun cut_run(int units, int *s_tiles, U unit, P parts_of,
                                          F tiles_of) {
    constexpr int kWarps = kThreads / 32;
    __shared__ int warp_sums[kWarps];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = (units + kThreads - 1) / kThreads;
    const int v0 = min(units, tid * chunk), v1 = min(units, v0 + chunk);
    auto unit_tiles = [&](int v) {
        int sum = 0;
        const auto u = unit(v);
        const int n = parts_of(u);
        for (int i = 0; i < n; ++i) sum += tiles_of(u, i);
        return sum;
    };
    int mine = 0;
    if (units <= 2 * kWarps) {
        for (int v = warp; v < units; v += kWarps) {
            int sum = 0;
            const auto u = unit(v);
            const int n = parts_of(u);
            for (int i = lane; i < n; i += 32) sum += tiles_of(u, i);
            sum = __reduce_add_sync(0xffffffffu, sum);
            if (lane == 0) s_tiles[v] = sum;
        }
        __syncthreads();
        mine = tid < units ? s_tiles[tid] : 0;
        sm100::fence_proxy_async_smem();
    } else {
        for (int v = v0; v < v1; ++v) mine += unit_tiles(v);
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    CtaRun R;
    R.total = total;
    R.per = max(1, (total + (int)gridDim.x - 1) / (int)gridDim.x);
    R.begin = (int)min((long long)total, (long long)blockIdx.x * R.per);
    R.end = (int)min((long long)total, (long long)R.begin + R.per);
    if (R.begin < R.end && before <= R.begin && R.begin < before + mine) {
        int at = before, v = v0;
        if (chunk > 1)
            for (int t; at + (t = unit_tiles(v)) <= R.begin; ++v) at += t;
        found[0] = v;
        found[2] = at;
    }
    __syncthreads();
    if (R.begin >= R.end) {
        R.unit = units;
        R.part = 0;
        R.part_begin = R.end;
        return R;
    }
    R.unit = found[0];
    if (warp == 0) {
        const auto u = unit(R.unit);
        const int n = parts_of(u);
        int at = found[2];
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int t = i0 + lane < n ? tiles_of(u, i0 + lane) : 0;
            int x = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, at + x > R.begin);
            if (past) {
                if (lane == __ffs(past) - 1) {
                    found[1] = i0 + lane;
                    found[2] = at + x - t;
                }
                break;
            }
            at += __shfl_sync(0xffffffffu, x, 31);
        }
        __syncwarp();
    }
    __syncthreads();
    R.part = found[1];
    R.part_begin = found[2];
    return R;
}

// Cuts the units, in order, into groups of equal rows (rows_of(v) of unit v), at least
// `rows` each and no more groups than `phases`, or than leave each `work` (work_of(v) of
// unit v).  Group g is units [first[g], first[g + 1]) (shared memory, phases + 1 words).
// All kThreads threads call it.
template <int kThreads, typename F, typename W>
__device__ __forceinline__ void cut_units(int units, int phases, long long rows, long long work,
                                          int *first, F rows_of, W work_of) {
    constexpr int kWarps = kThreads / 32;
    __shared__ long long warp_sums[kWarps], warp_work[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid <= phases) first[tid] = tid ? units : 0;
    __syncthreads();
    if (phases == 1) return;
    const int chunk = (units + kThreads - 1) / kThreads;
    const int v0 = min(units, tid * chunk), v1 = min(units, v0 + chunk);
    long long mine = 0, load = 0;
    for (int v = v0; v < v1; ++v) {
        mine += rows_of(v);
        load += work_of(v);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
        load += __shfl_xor_sync(0xffffffffu, load, o);
    }
    if (lane == 31) {
        warp_sums[warp] = incl;
        warp_work[warp] = load;
    }
    __syncthreads();
    long long at = incl - mine, total = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += warp_sums[w];
        total += warp_sums[w];
        all += warp_work[w];
    }
    const long long groups = max(1ll, min((long long)phases, all / work));
    const long long quota = max(rows, (total + groups - 1) / groups);
    for (int v = v0; v < v1; ++v) {
        const long long to = at + rows_of(v);
        for (int g = 1; g < groups; ++g)
            if (at < g * quota && g * quota <= to) first[g] = v + 1;
        at = to;
    }
    __syncthreads();
}

// log2 of a row's softmax sum from its maximum (log2 units) and sum.  A sum is 0 where nothing is seen,
// and NaN, as are then lse and output, where a logit was.
__device__ __forceinline__ float row_lse2(float m, float l) {
    return l == 0.f ? -INFINITY : m + __log2f(l);
}

// Writes a merged row of an item (a warp, D / 32 elements of the sum a lane).
template <typename X, int D>
__device__ __forceinline__ void store_merged(const DevPaged &C, const DevChunk &T, int layer,
                                             const AttendIo &io, float *lse2, const CutItem &it,
                                             int row, float m, float l, const float (&acc)[D / 32]) {
    constexpr int kV = D / 32;
    const int lane = threadIdx.x & 31;
    const UnitRows U = unit_rows(C, T, layer, it.unit);
    const long long tok = U.tok0 + (it.row0 + row) / C.G;
    const int head = U.h * C.G + (it.row0 + row) % C.G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    typename X::T *op = static_cast<typename X::T *>(io.out) + tok * io.out_stride +
                        (long long)head * D + lane * kV;
    static_assert(kV == 2 || kV == 4, "two or four elements a lane");
#pragma unroll
    for (int i = 0; i < kV; i += 2)
        *reinterpret_cast<uint32_t *>(op + i) = X::pack(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0) {
        const float z = row_lse2(m, l);
        if (io.lse) io.lse[tok * C.Hq + head] = z * kLn2;
        if (lse2) lse2[packed_row(C, U, it.row0 + row)] = z;
    }
}

// Merges the many-rows kernel's partials of the items that several CTAs held.
cudaError_t launch_many_merge(const DevPaged &C, const DevChunk &T, int layer, const AttendIo &io,
                              float *lse2, const AttendWs &ws, int phases, cudaStream_t s);
// Requests of at most T.few_max query rows a head: `items` items of at most kFewRows rows
// in all, the largest with max_rows, `blocks` of them at most to a unit, which sees at
// most `seen` rows of it.
cudaError_t launch_attend_few(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                              const AttendIo &io, bool add_mass, long long seen, long long items,
                              int max_rows, int blocks, const AttendWs &ws, cudaStream_t s);
// The others.
cudaError_t launch_attend_many(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                               const AttendIo &io, const AttendWs &ws, cudaStream_t s);
// Their weights, from its packed queries and lse.
cudaError_t launch_many_mass(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                             const AttendWs &ws, cudaStream_t s);

}  // namespace kvevict
