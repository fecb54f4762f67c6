// kv_paged_attention.cu -- attention of new tokens over the pages: which kernel takes a
// request (few or many query rows a head), the merge of items that several CTAs held, and
// the workspace they share.
#include <algorithm>

#include "kv_paged_attend.cuh"

namespace kvevict {
namespace {

// ---------------------------------------------------------------------------
// Merge of cut items.  The CTA that held an item's last tile left its description;
// CTA (b, y) merges rows of the item of slot b.  kSplit: one row a CTA, its warps
// taking every fourth partial (few rows, many partials); else a row per warp.  Partials
// are added in order: the result does not depend on timing.
// ---------------------------------------------------------------------------
template <typename X, int D, int kRowSlots, bool kSplit>
__global__ void __launch_bounds__(128)
merge_kernel(const DevPaged C, const DevChunk T, int layer, const AttendIo io, float *lse2,
             int *status, const int *__restrict__ cta_status, const CutItem *__restrict__ cut,
             const float2 *__restrict__ part_ml, const float *__restrict__ part_o, int ctas,
             bool first) {
    constexpr int kV = D / 32;
    __shared__ float sm_o[4][D], sm_l[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int code = 0;
        for (int i = threadIdx.x; i < ctas; i += 128) code = max(code, cta_status[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) code = max(code, __shfl_xor_sync(0xffffffffu, code, o));
        if (lane == 0) sm_l[warp] = __int_as_float(code);
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 4; ++w) code = max(code, __float_as_int(sm_l[w]));
            if (first || *status == 0) *status = code;
        }
        __syncthreads();
    }
    const CutItem it = cut[blockIdx.x];
    if (it.unit < 0) return;
    const int row = kSplit ? (int)blockIdx.y : (int)blockIdx.y * 4 + warp;
    if (row >= it.rows) return;            // whole CTA where kSplit
    const int parts = (int)blockIdx.x - it.cta0 + 1;
    auto slot_row = [&](int p) {
        return (long long)part_slot(it.cta0 + p, p == 0) * kRowSlots + row;
    };
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, part_ml[slot_row(p)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f, acc[kV] = {};
    constexpr int kStep = kSplit ? 4 : 1;
#pragma unroll 4
    for (int p = kSplit ? warp : 0; p < parts; p += kStep) {
        const long long at = slot_row(p);
        const float2 ml = part_ml[at];
        if (ml.x == -INFINITY) continue;   // nothing seen: its output was not written
        const float w = shrink(ml.x, m);
        l += ml.y * w;
        const float *src = part_o + at * D + lane * kV;
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[i] += src[i] * w;
    }
    if (kSplit) {
#pragma unroll
        for (int i = 0; i < kV; ++i) sm_o[warp][lane * kV + i] = acc[i];
        if (lane == 0) sm_l[warp] = l;
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            l += sm_l[w];
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[i] += sm_o[w][lane * kV + i];
        }
    }
    const UnitRows U = unit_rows(C, T, layer, it.unit);
    const long long tok = U.tok0 + (it.row0 + row) / C.G;
    const int head = U.h * C.G + (it.row0 + row) % C.G;
    const float inv = l > 0.f ? 1.f / l : 0.f;
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

template <typename X, int D>
cudaError_t merge(const DevPaged &C, const DevChunk &T, int layer, const AttendIo &io, float *lse2,
                  const AttendWs &ws, int ctas, int rows, bool first, cudaStream_t s) {
    if (rows == kFewRows)
        return launch_dependent(merge_kernel<X, D, kFewRows, true>,
                                dim3(ctas, std::min<long long>(kFewRows, (long long)T.max_t * C.G)),
                                128, 0, s, C, T, layer, io, lse2, ws.status, ws.cta_status, ws.cut,
                                ws.part_ml, ws.part_o, ctas, first);
    return launch_dependent(merge_kernel<X, D, kManyRows, false>, dim3(ctas, kManyRows / 4), 128, 0,
                            s, C, T, layer, io, lse2, ws.status, ws.cta_status, ws.cut, ws.part_ml,
                            ws.part_o, ctas, first);
}

}  // namespace

cudaError_t launch_attend_merge(const DevPaged &C, const DevChunk &T, int layer,
                                const AttendIo &io, float *lse2, const AttendWs &ws, int ctas,
                                int rows, bool first, cudaStream_t s) {
    if (C.dtype == KV_FP16)
        return C.d == 64 ? merge<Fp16, 64>(C, T, layer, io, lse2, ws, ctas, rows, first, s)
                         : merge<Fp16, 128>(C, T, layer, io, lse2, ws, ctas, rows, first, s);
    return C.d == 64 ? merge<Bf16, 64>(C, T, layer, io, lse2, ws, ctas, rows, first, s)
                     : merge<Bf16, 128>(C, T, layer, io, lse2, ws, ctas, rows, first, s);
}

namespace {
// Requests of the step whose query rows a head fit the few-rows kernel, and the others.
struct Classes {
    int few, few_rows, many;
};
Classes classify(const DevPaged &C, const DevChunk &T) {
    Classes k{0, 0, 0};
    for (int r = 0; r < C.R; ++r) {
        const long long rows = (T.host_off[r + 1] - T.host_off[r]) * C.G;
        if (rows > kFewRows) {
            ++k.many;
        } else if (rows > 0) {
            ++k.few;
            k.few_rows = std::max(k.few_rows, (int)rows);
        }
    }
    return k;
}
}  // namespace

AttendWs attend_ws_layout(const DevPaged &C, const DevChunk &T, bool add_mass, void *base) {
    AttendWs ws{};
    char *b = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = b ? b + off : nullptr;
        off = (off + bytes + 255) / 256 * 256;
        return p;
    };
    const Classes k = classify(C, T);
    // the two kernels run one after the other: they share the partials
    const size_t slots = std::max<size_t>(k.few ? 2 * kFewCtas * (size_t)kFewRows : 0,
                                          k.many ? 2 * kManyCtas * (size_t)kManyRows : 0);
    ws.status = reinterpret_cast<int *>(take(kHeaderBytes));
    ws.cta_status = reinterpret_cast<int *>(take(kFewCtas * sizeof(int)));
    ws.cut = reinterpret_cast<CutItem *>(take(kFewCtas * sizeof(CutItem)));
    ws.part_ml = reinterpret_cast<float2 *>(take(slots * sizeof(float2)));
    ws.part_o = reinterpret_cast<float *>(take(slots * C.d * sizeof(float)));
    if (add_mass) {
        const size_t tiles = (size_t)k.few * C.H * ((C.cap + kFewTile - 1) / kFewTile);
        ws.lse2 = reinterpret_cast<float *>(take((size_t)T.tokens * C.Hq * sizeof(float)));
        ws.q_packed = take(k.many ? (size_t)T.tokens * C.Hq * C.d * 2 : 0);
        ws.tiles = reinterpret_cast<int *>(take(sizeof(int)));
        ws.tile_at = reinterpret_cast<int2 *>(take(tiles * sizeof(int2)));
        ws.logits = reinterpret_cast<float *>(
            take(tiles * kFewRows * kFewTile * sizeof(float)));
    }
    ws.total = off;
    return ws;
}

cudaError_t launch_paged_attention(const DevPaged &C, const DevChunk &T, int layer,
                                   const AttendMask &M, const AttendIo &io, bool add_mass,
                                   const AttendWs &ws, cudaStream_t s) {
    const Classes k = classify(C, T);
    cudaError_t e = cudaSuccess;
    if (k.few) e = launch_attend_few(C, T, layer, M, io, add_mass, k.few_rows, true, ws, s);
    if (e == cudaSuccess && k.many) {
        e = launch_attend_many(C, T, layer, M, io, add_mass, !k.few, ws, s);
        if (e == cudaSuccess && add_mass) e = launch_many_mass(C, T, layer, M, ws, s);
    }
    return e;
}

}  // namespace kvevict
