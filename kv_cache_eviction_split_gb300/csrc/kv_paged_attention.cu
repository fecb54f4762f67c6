// kv_paged_attention.cu -- attention of new tokens over the pages, the plain way:
// one CTA per (token, KV head), its warps take every fourth row seen.
#include <cuda_fp16.h>

#include "kv_paged.cuh"

namespace kvevict {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16 *y) { *y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half *y) { *y = __float2half_rn(x); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32)
attend_kernel(const DevPaged C, const DevChunk T, int layer, const AttendMask M, const AttendIo io,
              float *lse2, int *status) {
    constexpr int kE = D / 32;
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tok = blockIdx.x;
    if (tok >= T.off[C.R]) return;
    const int h = blockIdx.y, r = request_of(T, C.R, tok);
    const long long u = ((long long)r * C.L + layer) * C.H + h;
    int n;
    if (!unit_len(C, u, n) && threadIdx.x == 0) post_status(status, KV_ERR_INVALID_ARG);
    const long long t = n - (T.off[r + 1] - tok);
    const int32_t *tab = C.table + u * C.max_pages;
    const int lo = t < 0 ? 0 : window_lo(M, (int)t), sinks = min(M.sinks, lo);
    for (int g = 0; g < C.G; ++g) {
        const int head = h * C.G + g;
        const E *qp = static_cast<const E *>(io.q) + tok * io.q_stride + (long long)head * D;
        float q[kE], o[kE] = {}, m = -INFINITY, l = 0.f;
        for (int e = 0; e < kE; ++e) q[e] = to_f(qp[e * 32 + lane]);
        const int seen = t < 0 ? 0 : sinks + (int)t + 1 - lo;
        for (int x = warp; x < seen; x += kWarps) {
            const int j = x < sinks ? x : lo + x - sinks;
            const long long row = page_row(C, tab, j);
            if (row < 0) {
                if (lane == 0) post_status(status, KV_ERR_INVALID_ARG);
                continue;
            }
            const E *kp = static_cast<const E *>(C.k) + row * D, *vp = static_cast<const E *>(C.v) + row * D;
            float s = 0.f;
            for (int e = 0; e < kE; ++e) s += q[e] * to_f(kp[e * 32 + lane]);
            s = warp_sum(s) * M.scale_log2;
            const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
            l = l * f + p;
            for (int e = 0; e < kE; ++e) o[e] = o[e] * f + p * to_f(vp[e * 32 + lane]);
            m = mn;
        }
        if (lane == 0) {
            sm_m[warp] = m;
            sm_l[warp] = l;
        }
        for (int e = 0; e < kE; ++e) sm_o[warp][e * 32 + lane] = o[e];
        __syncthreads();
        float mm = -INFINITY, ll = 0.f;
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w]);
        for (int w = 0; w < kWarps; ++w) ll += sm_l[w] > 0.f ? sm_l[w] * exp2f(sm_m[w] - mm) : 0.f;
        E *op = static_cast<E *>(io.out) + tok * io.out_stride + (long long)head * D;
        for (int i = threadIdx.x; i < D; i += kWarps * 32) {
            float x = 0.f;
            for (int w = 0; w < kWarps; ++w)
                if (sm_l[w] > 0.f) x += sm_o[w][i] * exp2f(sm_m[w] - mm);
            from_f(ll > 0.f ? x / ll : 0.f, op + i);
        }
        if (threadIdx.x == 0) {
            const float z = ll > 0.f ? mm + log2f(ll) : -INFINITY;
            if (io.lse) io.lse[tok * C.Hq + head] = z * 0.6931471805599453f;
            if (lse2) lse2[tok * C.Hq + head] = z;
        }
        __syncthreads();
    }
}

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32)
mass_kernel(const DevPaged C, const DevChunk T, int layer, const AttendMask M, const AttendIo io,
            const float *lse2, int h) {
    constexpr int kE = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y;
    const long long u = ((long long)r * C.L + layer) * C.H + h;
    const long long t0 = T.off[r];
    const int count = (int)(T.off[r + 1] - t0);
    int n;
    unit_len(C, u, n);
    for (int j = blockIdx.x * kWarps + warp; j < n && count > 0; j += gridDim.x * kWarps) {
        // queries that see row j
        int first = j - (n - count), last = count - 1;
        if (M.window > 0 && j >= M.sinks && j - (n - count) + M.window - 1 < last)
            last = j - (n - count) + M.window - 1;
        if (first < 0) first = 0;
        if (first > last) continue;
        const long long row = page_row(C, C.table + u * C.max_pages, j);
        if (row < 0) continue;
        float k[kE], acc = 0.f;
        for (int e = 0; e < kE; ++e) k[e] = to_f(static_cast<const E *>(C.k)[row * D + e * 32 + lane]);
        for (int i = first; i <= last; ++i)
            for (int g = 0; g < C.G; ++g) {
                const int head = h * C.G + g;
                const E *qp = static_cast<const E *>(io.q) + (t0 + i) * io.q_stride + (long long)head * D;
                float s = 0.f;
                for (int e = 0; e < kE; ++e) s += k[e] * to_f(qp[e * 32 + lane]);
                acc += exp2f(warp_sum(s) * M.scale_log2 - lse2[(t0 + i) * C.Hq + head]);
            }
        if (lane == 0) C.mass[row] += acc;
    }
}

template <typename E, int D>
cudaError_t attend(const DevPaged &C, const DevChunk &T, int layer, const AttendMask &M,
                   const AttendIo &io, bool add_mass, const AttendWs &ws, cudaStream_t s) {
    attend_kernel<E, D><<<dim3((unsigned)T.tokens, C.H), kWarps * 32, 0, s>>>(
        C, T, layer, M, io, add_mass ? ws.lse2 : nullptr, ws.status);
    if (add_mass)
        for (int h = 0; h < C.H; ++h)
            mass_kernel<E, D><<<dim3(1024, C.R), kWarps * 32, 0, s>>>(C, T, layer, M, io, ws.lse2, h);
    return cudaGetLastError();
}

}  // namespace

AttendWs attend_ws_layout(const DevPaged &C, const DevChunk &T, bool add_mass, void *base) {
    AttendWs ws{};
    char *b = static_cast<char *>(base);
    ws.status = reinterpret_cast<int *>(b);
    ws.lse2 = reinterpret_cast<float *>(b + kHeaderBytes);
    ws.total = kHeaderBytes + (add_mass ? (size_t)T.tokens * C.Hq * sizeof(float) : 0);
    return ws;
}

cudaError_t launch_paged_attention(const DevPaged &C, const DevChunk &T, int layer,
                                   const AttendMask &M, const AttendIo &io, bool add_mass,
                                   const AttendWs &ws, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(ws.status, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
    if (C.dtype == KV_FP16)
        return C.d == 64 ? attend<__half, 64>(C, T, layer, M, io, add_mass, ws, s)
                         : attend<__half, 128>(C, T, layer, M, io, add_mass, ws, s);
    return C.d == 64 ? attend<__nv_bfloat16, 64>(C, T, layer, M, io, add_mass, ws, s)
                     : attend<__nv_bfloat16, 128>(C, T, layer, M, io, add_mass, ws, s);
}

}  // namespace kvevict
