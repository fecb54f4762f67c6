// kv_paged_copy.cu -- rows into pages: new tokens (append) and packed ragged rows (load).
//
// Bit copies, bound by HBM: every row read once and written once in 16-byte
// vectors.  A row pair (K and V) is 2 d / 8 vectors: one warp's load for d = 128,
// half of one for d = 64, so a warp step moves 512 bytes and addresses are formed
// once per row.  Measured (d = 128, 8 KV heads): load of 256 units of 1638 rows, 430 MB
// moved, 69.6 us (6.2 TB/s; 8 row pairs in flight a lane, 256 rows a CTA); append of 8 tokens
// 2.2 us on the GPU, the launch itself.
#include <algorithm>

#include "kv_compact.cuh"
#include "kv_paged.cuh"

namespace kvevict {
namespace {

constexpr int kWarps = 8;

// Which part of a row pair a lane moves: `sub` of kRows row pairs of the warp step,
// K (which = 0) or V, 16-byte vector `ch` of the row.
template <int D>
struct LanePart {
    static constexpr int kVecs = D / 8;
    static constexpr int kLanes = 2 * kVecs;
    static constexpr int kRows = 32 / kLanes;
    int sub, which, ch;
    __device__ LanePart() {
        const int lane = threadIdx.x & 31;
        sub = lane / kLanes;
        which = (lane % kLanes) / kVecs;
        ch = lane % kVecs;
    }
};

// One row pair per warp part: row i of the call is token i / H, head i % H.
template <int D>
__global__ void __launch_bounds__(kWarps * 32)
append_kernel(const DevPaged C, const DevChunk T, int layer, const uint4 *__restrict__ k_new,
              long long k_stride, const uint4 *__restrict__ v_new, long long v_stride) {
    using Part = LanePart<D>;
    const Part p;
    const long long i = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * Part::kRows + p.sub;
    if (i >= T.tokens * C.H) return;
    const long long tok = i / C.H;
    const int h = (int)(i - tok * C.H);
    const uint4 *src = p.which ? v_new + tok * v_stride : k_new + tok * k_stride;
    const uint4 val = ld_nc(src + h * Part::kVecs + p.ch);
    const bool none = without_rows(C);
    const int r = request_of(T, C.R, tok);
    if (tok >= T.off[C.R] || none) return;
    const long long u = ((long long)r * C.L + layer) * C.H + h;
    int n;
    const bool ok = unit_len(C, u, n);
    const long long j = n - (T.off[r + 1] - tok);
    if (ok && j < 0) return;
    const long long row = ok ? page_row(C, C.table + u * C.max_pages, (int)j) : -1;
    if (row < 0) {
        post_status(C.status, KV_ERR_INVALID_ARG);
        return;
    }
    reinterpret_cast<uint4 *>(p.which ? C.v : C.k)[row * Part::kVecs + p.ch] = val;
    if (C.mass && p.which == 0 && p.ch == 0) C.mass[row] = 0.f;
}

constexpr int kLoadRows = 256;    // packed rows per CTA
constexpr int kLoadUnroll = 8;    // row pairs in flight per lane part

// Rows [r0, r0 + kLoadRows) of the packed arrays; a lane part walks every
// (kWarps * kRows)-th of them and moves on to the next unit as its rows pass one.
template <int D>
__global__ void __launch_bounds__(kWarps * 32)
load_kernel(const DevPaged C, const uint4 *__restrict__ k_rows, const uint4 *__restrict__ v_rows,
            const float *__restrict__ mass_rows, const int64_t *__restrict__ offsets,
            long long total_rows) {
    using Part = LanePart<D>;
    const Part p;
    // whether a unit's rows [a, b) are there and fit its table
    auto fits = [&](long long a, long long b) {
        return a >= 0 && a <= b && b <= total_rows && b - a <= C.cap;
    };
    // lengths: unit u by thread u of the grid
    const long long threads = (long long)gridDim.x * blockDim.x;
    for (long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x; u < C.units; u += threads) {
        const long long a = offsets[u], b = offsets[u + 1];
        C.lens[u] = fits(a, b) ? (int)(b - a) : -1;
    }
    constexpr int kStep = kWarps * Part::kRows;
    const long long r0 = (long long)blockIdx.x * kLoadRows;
    const long long r1 = min(total_rows, r0 + kLoadRows);
    const long long first = r0 + (threadIdx.x >> 5) * Part::kRows + p.sub;
    if (first >= r1) return;
    long long lo = 0, hi = C.units;
    while (hi - lo > 1) {
        const long long mid = (lo + hi) >> 1;
        if (offsets[mid] <= first) lo = mid; else hi = mid;
    }
    long long u = lo, u0 = offsets[u], u1 = offsets[u + 1];
    bool ok = fits(u0, u1), lost = false;
    const uint4 *src = p.which ? v_rows : k_rows;
    uint4 *dst = reinterpret_cast<uint4 *>(p.which ? C.v : C.k);
    for (long long rb = first; rb < r1; rb += kStep * kLoadUnroll) {
        uint4 buf[kLoadUnroll];
        long long to[kLoadUnroll];
#pragma unroll
        for (int i = 0; i < kLoadUnroll; ++i) {
            const long long row = rb + i * kStep;
            if (row < r1) buf[i] = ld_nc(src + row * Part::kVecs + p.ch);
        }
#pragma unroll
        for (int i = 0; i < kLoadUnroll; ++i) {
            const long long row = rb + i * kStep;
            to[i] = -1;
            if (row >= r1) continue;
            while (row >= u1 && u + 1 < C.units) {
                ++u;
                u0 = u1;
                u1 = offsets[u + 1];
                ok = fits(u0, u1);
            }
            if (!ok || row < u0 || row >= u1) continue;
            to[i] = page_row(C, C.table + u * C.max_pages, (int)(row - u0));
            lost |= to[i] < 0;
        }
#pragma unroll
        for (int i = 0; i < kLoadUnroll; ++i) {
            if (to[i] < 0) continue;
            st_cs(dst + to[i] * Part::kVecs + p.ch, buf[i]);
            if (C.mass && p.which == 0 && p.ch == 0)
                C.mass[to[i]] = mass_rows ? mass_rows[rb + i * kStep] : 0.f;
        }
    }
    if (lost && p.which == 0 && p.ch == 0) post_status(C.status, KV_ERR_INVALID_ARG);
}

}  // namespace

cudaError_t launch_paged_append(const DevPaged &C, const DevChunk &T, int layer, const void *k_new,
                                long long k_stride, const void *v_new, long long v_stride,
                                cudaStream_t s) {
    auto k = static_cast<const uint4 *>(k_new);
    auto v = static_cast<const uint4 *>(v_new);
    const long long rows = T.tokens * C.H;
    const int per_cta = C.d == 64 ? kWarps * LanePart<64>::kRows : kWarps * LanePart<128>::kRows;
    const unsigned grid = (unsigned)((rows + per_cta - 1) / per_cta);
    if (C.d == 64)
        append_kernel<64><<<grid, kWarps * 32, 0, s>>>(C, T, layer, k, k_stride / 8, v,
                                                       v_stride / 8);
    else
        append_kernel<128><<<grid, kWarps * 32, 0, s>>>(C, T, layer, k, k_stride / 8, v,
                                                        v_stride / 8);
    return cudaGetLastError();
}

cudaError_t launch_paged_load(const DevPaged &C, const void *k_rows, const void *v_rows,
                              const float *mass_rows, const int64_t *offsets, long long total_rows,
                              cudaStream_t s) {
    auto k = static_cast<const uint4 *>(k_rows);
    auto v = static_cast<const uint4 *>(v_rows);
    const unsigned grid = (unsigned)std::max<long long>(1, (total_rows + kLoadRows - 1) / kLoadRows);
    if (C.d == 64)
        load_kernel<64><<<grid, kWarps * 32, 0, s>>>(C, k, v, mass_rows, offsets, total_rows);
    else
        load_kernel<128><<<grid, kWarps * 32, 0, s>>>(C, k, v, mass_rows, offsets, total_rows);
    return cudaGetLastError();
}

}  // namespace kvevict
