// kv_paged_api.cu -- the extern "C" entry points of the paged cache: argument
// checks, workspace carve-up, launches (host code).
#include <algorithm>
#include <cmath>

#include "kv_paged.cuh"
#include "kv_trace.cuh"

using namespace kvevict;

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool bad_ptr(const void *p) { return !p || !aligned16(p); }

kv_status map_cuda(cudaError_t e) { return e == cudaSuccess ? KV_OK : KV_ERR_CUDA; }

// Validates a cache description and fills the device-side copy.
kv_status make_paged(const kv_paged *c, DevPaged *C) {
    if (!c) return KV_ERR_INVALID_ARG;
    if (c->num_requests < 0 || c->num_layers < 1 || c->num_kv_heads < 1 ||
        c->num_q_heads < c->num_kv_heads || c->num_q_heads % c->num_kv_heads != 0 ||
        c->max_pages < 1 || c->num_pages < 1)
        return KV_ERR_INVALID_ARG;
    if (c->dtype != KV_BF16 && c->dtype != KV_FP16) return KV_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return KV_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return KV_ERR_UNSUPPORTED;
    // TMA row coordinates and cache row indices are 32-bit
    const long long kRowLimit = 1LL << 31;
    const long long units = (long long)c->num_requests * c->num_layers * c->num_kv_heads;
    if (c->num_pages >= kRowLimit / c->page_size || c->max_pages >= kRowLimit / c->page_size ||
        (long long)c->num_layers * c->num_kv_heads >= kRowLimit || units >= kRowLimit ||
        (long long)c->num_requests * c->num_kv_heads >= (1 << 20))
        return KV_ERR_UNSUPPORTED;
    C->R = c->num_requests;
    C->L = c->num_layers;
    C->H = c->num_kv_heads;
    C->Hq = c->num_q_heads;
    C->G = c->num_q_heads / c->num_kv_heads;
    C->d = c->head_dim;
    C->ps = c->page_size;
    C->ps_log2 = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
    C->max_pages = c->max_pages;
    C->cap = c->max_pages * c->page_size;
    C->dtype = c->dtype;
    C->num_pages = c->num_pages;
    C->units = units;
    C->table = c->page_table;
    C->lens = c->lens;
    C->k = c->k_pages;
    C->v = c->v_pages;
    C->mass = c->mass;
    C->status = c->status;
    C->wait_ns = kv_get_wait_limit_ns();
    if (units > 0 && (bad_ptr(c->k_pages) || bad_ptr(c->v_pages) || bad_ptr(c->page_table) ||
                      bad_ptr(c->lens) || bad_ptr(c->status) || !aligned16(c->mass)))
        return KV_ERR_INVALID_ARG;
    return KV_OK;
}

kv_status make_chunk(const kv_chunk *t, const DevPaged &C, DevChunk *T) {
    if (!t) return KV_ERR_INVALID_ARG;
    T->off = reinterpret_cast<const long long *>(t->tok_offsets_dev);
    T->host_off = reinterpret_cast<const long long *>(t->tok_offsets_host);
    T->tokens = 0;
    T->max_t = 0;
    if (C.R == 0) return KV_OK;
    if (!t->tok_offsets_host || bad_ptr(t->tok_offsets_dev) || t->tok_offsets_host[0] != 0)
        return KV_ERR_INVALID_ARG;
    long long most = 0;
    for (int r = 0; r < C.R; ++r) {
        const long long n = t->tok_offsets_host[r + 1] - t->tok_offsets_host[r];
        if (n < 0) return KV_ERR_INVALID_ARG;
        most = std::max(most, n);
    }
    T->tokens = t->tok_offsets_host[C.R];
    // query rows (token, head) are counted in 32 bits
    if (T->tokens >= (1LL << 31) / C.Hq) return KV_ERR_UNSUPPORTED;
    T->max_t = (int)most;
    return KV_OK;
}

bool bad_stride(long long stride, long long least) { return stride < least || stride % 8 != 0; }

}  // namespace

extern "C" {

kv_status kv_paged_append(const kv_paged *c, const kv_chunk *t, int32_t layer, const void *k_new,
                          int64_t k_stride, const void *v_new, int64_t v_stride, void *stream) {
    KV_API_RANGE();
    DevPaged C;
    DevChunk T;
    kv_status st = make_paged(c, &C);
    if (st == KV_OK) st = make_chunk(t, C, &T);
    if (st != KV_OK) return st;
    if (layer < 0 || layer >= C.L) return KV_ERR_INVALID_ARG;
    if (T.tokens == 0) return KV_OK;
    const long long row = (long long)C.H * C.d;
    if (bad_ptr(k_new) || bad_ptr(v_new) || bad_stride(k_stride, row) || bad_stride(v_stride, row))
        return KV_ERR_INVALID_ARG;
    return map_cuda(launch_paged_append(C, T, layer, k_new, k_stride, v_new, v_stride,
                                        (cudaStream_t)stream));
}

kv_status kv_paged_load(const kv_paged *c, const void *k_rows, const void *v_rows,
                        const float *mass_rows, const int64_t *offsets_dev, int64_t total_rows,
                        void *stream) {
    KV_API_RANGE();
    DevPaged C;
    kv_status st = make_paged(c, &C);
    if (st != KV_OK || C.units == 0) return st;
    if (total_rows < 0 || total_rows > C.num_pages * C.ps || bad_ptr(offsets_dev))
        return KV_ERR_INVALID_ARG;
    if (total_rows > 0 && (bad_ptr(k_rows) || bad_ptr(v_rows) || !aligned16(mass_rows)))
        return KV_ERR_INVALID_ARG;
    return map_cuda(launch_paged_load(C, k_rows, v_rows, C.mass ? mass_rows : nullptr, offsets_dev,
                                      total_rows, (cudaStream_t)stream));
}

static kv_status check_attention(const kv_paged *c, const kv_chunk *t, int32_t add_mass,
                                 DevPaged *C, DevChunk *T) {
    kv_status st = make_paged(c, C);
    if (st == KV_OK) st = make_chunk(t, *C, T);
    if (st != KV_OK) return st;
    if (add_mass && C->units > 0 && !C->mass) return KV_ERR_INVALID_ARG;
    return KV_OK;
}

kv_status kv_paged_attention_workspace_size(const kv_paged *c, const kv_chunk *t,
                                            int32_t add_mass, size_t *bytes) {
    DevPaged C;
    DevChunk T;
    kv_status st = check_attention(c, t, add_mass, &C, &T);
    if (st != KV_OK) return st;
    if (!bytes) return KV_ERR_INVALID_ARG;
    *bytes = attend_ws_layout(C, T, add_mass != 0, nullptr).total;
    return KV_OK;
}

kv_status kv_paged_attention(const kv_paged *c, const kv_chunk *t, int32_t layer, int32_t window,
                             int32_t num_sinks, float softmax_scale, const void *q,
                             int64_t q_stride, void *out, int64_t out_stride, float *lse,
                             int32_t add_mass, void *workspace, size_t workspace_bytes,
                             void *stream) {
    KV_API_RANGE();
    DevPaged C;
    DevChunk T;
    kv_status st = check_attention(c, t, add_mass, &C, &T);
    if (st != KV_OK) return st;
    if (layer < 0 || layer >= C.L || window < 0 || num_sinks < 0) return KV_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KV_ERR_INVALID_ARG;
    if (T.tokens == 0) return KV_OK;
    const long long row = (long long)C.Hq * C.d;
    if (bad_ptr(q) || bad_ptr(out) || !aligned16(lse) || bad_ptr(workspace) ||
        bad_stride(q_stride, row) || bad_stride(out_stride, row))
        return KV_ERR_INVALID_ARG;
    const AttendWs ws = attend_ws_layout(C, T, add_mass != 0, workspace);
    if (workspace_bytes < ws.total) return KV_ERR_WORKSPACE;
    // a window of the table's length or more hides nothing
    const int w = window >= C.cap ? 0 : window;
    const AttendMask M{w, w > 0 ? num_sinks : 0, softmax_scale * 1.4426950408889634f};
    if (!attend_tiles_fit(C, T, M, add_mass != 0)) return KV_ERR_UNSUPPORTED;
    const AttendIo io{q, out, lse, q_stride, out_stride};
    return map_cuda(launch_paged_attention(C, T, layer, M, io, add_mass != 0, ws,
                                           (cudaStream_t)stream));
}

kv_status kv_paged_evict_workspace_size(const kv_paged *src, size_t *bytes) {
    DevPaged S;
    kv_status st = make_paged(src, &S);
    if (st != KV_OK) return st;
    if (!bytes) return KV_ERR_INVALID_ARG;
    *bytes = kHeaderBytes;
    return KV_OK;
}

kv_status kv_paged_evict(const kv_paged *src, const kv_paged *dst, const int32_t *budgets_dev,
                         int32_t num_sinks, int32_t recent, int32_t *kept, int64_t kept_stride,
                         void *workspace, size_t workspace_bytes, void *stream) {
    KV_API_RANGE();
    DevPaged S, D;
    kv_status st = make_paged(src, &S);
    if (st == KV_OK) st = make_paged(dst, &D);
    if (st != KV_OK) return st;
    if (S.R != D.R || S.L != D.L || S.H != D.H || S.d != D.d || S.dtype != D.dtype || num_sinks < 0 ||
        recent < 0)
        return KV_ERR_INVALID_ARG;
    if (S.units == 0) return KV_OK;
    if (!S.mass || bad_ptr(budgets_dev) || bad_ptr(kept) || bad_ptr(workspace) || kept_stride < 1 ||
        S.lens == D.lens || S.table == D.table)
        return KV_ERR_INVALID_ARG;
    if (workspace_bytes < kHeaderBytes) return KV_ERR_WORKSPACE;
    int *status = static_cast<int *>(workspace);
    if (cudaMemsetAsync(status, 0, sizeof(int), (cudaStream_t)stream) != cudaSuccess)
        return KV_ERR_CUDA;
    return map_cuda(launch_paged_evict(S, D, budgets_dev, num_sinks, recent, kept, kept_stride,
                                       status, (cudaStream_t)stream));
}

}  // extern "C"
