// kv_paged_api.cu -- the extern "C" entry points of the paged cache: argument
// checks, workspace carve-up, launches (host code).
#include <algorithm>
#include <cmath>

#include "kv_paged.cuh"
#include "kv_paged_scores.cuh"
#include "kv_pages.cuh"
#include "kv_rotary.cuh"
#include "kv_trace.cuh"

using namespace kvevict;

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool bad_ptr(const void *p) { return !p || !aligned16(p); }
// whether an entry begins at p (null: none does)
inline bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

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

kv_status make_rotary(const kv_rotation *r, int d, bool backward, DevRotary *A) {
    if (!r || r->dims < 0 || r->dims > d) return KV_ERR_INVALID_ARG;
    if (r->dims % 16 != 0) return KV_ERR_UNSUPPORTED;
    if (!std::isfinite(r->factor) || (r->dims > 0 && !r->inv_freq) ||
        !aligned_to(r->inv_freq, 4))
        return KV_ERR_INVALID_ARG;
    *A = DevRotary{r->dims, r->interleaved != 0, backward, r->factor, r->inv_freq};
    return KV_OK;
}

// The counts of a cache's pages.
bool bad_refs(const DevPaged &C, const int32_t *refs) { return C.units > 0 && bad_ptr(refs); }

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

kv_status kv_paged_attention_scored_workspace_size(const kv_paged *c, const kv_chunk *t,
                                                   int32_t add_mass, size_t *bytes) {
    DevPaged C;
    DevChunk T;
    const kv_status st = check_attention(c, t, add_mass, &C, &T);
    if (st != KV_OK) return st;
    if (!bytes) return KV_ERR_INVALID_ARG;
    if (add_mass && !attend_few_only(C, T)) return KV_ERR_UNSUPPORTED;
    *bytes = attend_ws_layout(C, T, add_mass != 0, nullptr, true).total;
    return KV_OK;
}

kv_status kv_paged_attention_scored(const kv_paged *c, const kv_chunk *t, int32_t layer,
                                    const kv_scoring *f, float softmax_scale, const void *q,
                                    int64_t q_stride, void *out, int64_t out_stride, float *lse,
                                    int32_t add_mass, void *workspace, size_t workspace_bytes,
                                    void *stream) {
    KV_API_RANGE();
    DevPaged C;
    DevChunk T;
    kv_status st = check_attention(c, t, add_mass, &C, &T);
    if (st != KV_OK) return st;
    if (!f || layer < 0 || layer >= C.L || f->window < 0 || f->num_sinks < 0)
        return KV_ERR_INVALID_ARG;
    if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return KV_ERR_INVALID_ARG;
    if (!(f->softcap >= 0.0f) || !std::isfinite(f->softcap)) return KV_ERR_INVALID_ARG;
    if (add_mass && !attend_few_only(C, T)) return KV_ERR_UNSUPPORTED;
    if (T.tokens == 0) return KV_OK;
    const long long row = (long long)C.Hq * C.d;
    if (bad_ptr(q) || bad_ptr(out) || !aligned16(lse) || bad_ptr(workspace) ||
        !aligned16(f->row_pos) || bad_stride(q_stride, row) || bad_stride(out_stride, row) ||
        !aligned_to(f->slopes, 4) || !aligned_to(f->first, 4) || !aligned_to(f->last, 4))
        return KV_ERR_INVALID_ARG;
    // slopes are taken in units of q.k
    if (f->slopes && !std::isfinite(1.0f / softmax_scale)) return KV_ERR_INVALID_ARG;
    const AttendWs ws = attend_ws_layout(C, T, add_mass != 0, workspace, true);
    if (workspace_bytes < ws.total) return KV_ERR_WORKSPACE;
    // a window of the table's length or more hides nothing
    const int w = f->window >= C.cap ? 0 : f->window;
    const AttendMask M{w, w > 0 || f->first ? f->num_sinks : 0, softmax_scale * kLog2e};
    if (!attend_tiles_fit(C, T, M, add_mass != 0)) return KV_ERR_UNSUPPORTED;
    const AttendIo io{q, out, lse, q_stride, out_stride};
    if (!(f->softcap > 0.0f) && !f->slopes && !f->first && !f->last)
        return map_cuda(launch_paged_attention(C, T, layer, M, io, add_mass != 0, ws,
                                               (cudaStream_t)stream));
    ScoreForm form{};
    if (f->softcap > 0.0f) form.set_cap(f->softcap, softmax_scale);
    form.slope_s = 1.0f / softmax_scale;
    form.two_way = f->last != nullptr;
    form.slopes = f->slopes;
    form.pos = f->slopes ? f->row_pos : nullptr;
    return map_cuda(launch_paged_attention_scored(C, T, layer, M, form,
                                                  ScoreBounds{f->row_pos, f->first, f->last}, io,
                                                  add_mass != 0, ws, (cudaStream_t)stream));
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

kv_status kv_rotary_frequencies(int32_t dims, double base, int32_t scaling, double scale,
                                double context, double slow, double fast, float *inv_freq,
                                float *factor) {
    if (dims < 2 || dims % 2 != 0 || !(base > 0) || !std::isfinite(base) || !inv_freq || !factor)
        return KV_ERR_INVALID_ARG;
    if (scaling < KV_ROTARY_NONE || scaling > KV_ROTARY_PARTS) return KV_ERR_INVALID_ARG;
    if (scaling != KV_ROTARY_NONE && (!(scale >= 1) || !std::isfinite(scale)))
        return KV_ERR_INVALID_ARG;
    if (scaling == KV_ROTARY_PARTS && (!(context > 0) || !std::isfinite(context) || !(slow >= 0) ||
                                       !(fast > slow) || !std::isfinite(fast)))
        return KV_ERR_INVALID_ARG;
    if (scaling == KV_ROTARY_BASE && dims > 2) base *= std::pow(scale, dims / (dims - 2.0));
    for (int i = 0; i < dims / 2; ++i) {
        double w = std::pow(base, -2.0 * i / dims);
        if (scaling == KV_ROTARY_LINEAR) {
            w /= scale;
        } else if (scaling == KV_ROTARY_PARTS) {
            const double turns = context * w / 6.283185307179586;
            const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
            w = w * keep + w / scale * (1.0 - keep);
        }
        inv_freq[i] = (float)w;
    }
    *factor = scaling == KV_ROTARY_PARTS ? (float)(0.1 * std::log(scale) + 1.0) : 1.0f;
    return KV_OK;
}

kv_status kv_rotary(const kv_rotation *rot, const int32_t *positions, int64_t tokens, int32_t heads,
                    int32_t head_dim, int32_t dtype, const void *x, int64_t x_stride,
                    int64_t x_head_stride, void *out, int64_t out_stride, int64_t out_head_stride,
                    int32_t backward, void *stream) {
    KV_API_RANGE();
    DevRotary A;
    if (tokens < 0 || heads < 1 || (dtype != KV_BF16 && dtype != KV_FP16)) return KV_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return KV_ERR_UNSUPPORTED;
    const kv_status st = make_rotary(rot, head_dim, backward != 0, &A);
    if (st != KV_OK) return st;
    // a block's rows are counted in 32 bits
    if (heads >= (1 << 24) || tokens >= (1LL << 40)) return KV_ERR_UNSUPPORTED;
    if (tokens == 0) return KV_OK;
    if (!positions || !aligned_to(positions, 4) || bad_ptr(x) || bad_ptr(out))
        return KV_ERR_INVALID_ARG;
    for (long long s : {x_stride, x_head_stride, out_stride, out_head_stride})
        if (s < 0 || s % 8 != 0) return KV_ERR_INVALID_ARG;
    // rows that lie on one another cannot be written: a token's heads together, or a head's tokens
    if ((tokens > 1 && out_stride < head_dim) || (heads > 1 && out_head_stride < head_dim))
        return KV_ERR_INVALID_ARG;
    if (tokens > 1 && heads > 1 && (out_stride - head_dim) / (heads - 1) < out_head_stride &&
        (out_head_stride - head_dim) / (tokens - 1) < out_stride)
        return KV_ERR_INVALID_ARG;
    if (x == out && (x_stride != out_stride || x_head_stride != out_head_stride))
        return KV_ERR_INVALID_ARG;
    const RotaryIo io{static_cast<const uint4 *>(x), x_stride / 8,   x_head_stride / 8,
                      static_cast<uint4 *>(out),     out_stride / 8, out_head_stride / 8};
    return map_cuda(launch_rotary(A, tokens, heads, head_dim, dtype, positions, io,
                                  (cudaStream_t)stream));
}

kv_status kv_paged_append_rotary(const kv_paged *c, const kv_chunk *t, int32_t layer,
                                 const kv_rotation *rot, const int32_t *positions, int32_t *row_pos,
                                 const void *q, int64_t q_stride, void *q_out, int64_t q_out_stride,
                                 const void *k_new, int64_t k_stride, const void *v_new,
                                 int64_t v_stride, void *stream) {
    KV_API_RANGE();
    DevPaged C;
    DevChunk T;
    DevRotary A;
    kv_status st = make_paged(c, &C);
    if (st == KV_OK) st = make_chunk(t, C, &T);
    if (st == KV_OK) st = make_rotary(rot, C.d, false, &A);
    if (st != KV_OK) return st;
    if (layer < 0 || layer >= C.L) return KV_ERR_INVALID_ARG;
    if (C.Hq + 2LL * C.H >= (1 << 24)) return KV_ERR_UNSUPPORTED;
    if (T.tokens == 0) return KV_OK;
    const long long row = (long long)C.H * C.d, q_row = (long long)C.Hq * C.d;
    if (!positions || !aligned_to(positions, 4) || !aligned16(row_pos) || bad_ptr(k_new) ||
        bad_ptr(v_new) || bad_stride(k_stride, row) || bad_stride(v_stride, row))
        return KV_ERR_INVALID_ARG;
    if (q && (bad_ptr(q) || bad_ptr(q_out) || bad_stride(q_stride, q_row) ||
              bad_stride(q_out_stride, q_row) || (q == q_out && q_stride != q_out_stride)))
        return KV_ERR_INVALID_ARG;
    const AppendIo io{static_cast<const uint4 *>(q),     q_stride / 8,
                      static_cast<uint4 *>(q_out),       q_out_stride / 8,
                      static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new),
                      k_stride / 8,                      v_stride / 8};
    return map_cuda(launch_append_rotary(C, T, layer, A, positions, row_pos, io,
                                         (cudaStream_t)stream));
}

kv_status kv_paged_count_refs(const kv_paged *c, int32_t *refs, void *stream) {
    KV_API_RANGE();
    DevPaged C;
    const kv_status st = make_paged(c, &C);
    if (st != KV_OK) return st;
    if (bad_refs(C, refs)) return KV_ERR_INVALID_ARG;
    if (!refs) return KV_OK;
    return map_cuda(launch_count_refs(C, refs, (cudaStream_t)stream));
}

kv_status kv_paged_reserve_workspace_size(const kv_paged *c, size_t *bytes) {
    DevPaged C;
    const kv_status st = make_paged(c, &C);
    if (st != KV_OK) return st;
    if (!bytes) return KV_ERR_INVALID_ARG;
    *bytes = reserve_ws_layout(C, nullptr).total;
    return KV_OK;
}

kv_status kv_paged_reserve(const kv_paged *c, const kv_chunk *t, int32_t *refs, int32_t *row_pos,
                           void *workspace, size_t workspace_bytes, void *stream) {
    KV_API_RANGE();
    DevPaged C;
    DevChunk T;
    kv_status st = make_paged(c, &C);
    if (st == KV_OK) st = make_chunk(t, C, &T);
    if (st != KV_OK) return st;
    if (C.units >= (1 << 28)) return KV_ERR_UNSUPPORTED;
    if (T.tokens == 0) return KV_OK;
    if (bad_refs(C, refs) || !aligned16(row_pos) || bad_ptr(workspace)) return KV_ERR_INVALID_ARG;
    const PagesWs ws = reserve_ws_layout(C, workspace);
    if (workspace_bytes < ws.total) return KV_ERR_WORKSPACE;
    // the pages that the tokens fill in any case
    double least = 0;
    for (int r = 0; r < C.R; ++r)
        least += (double)((T.host_off[r + 1] - T.host_off[r]) / C.ps) * C.L * C.H;
    if (least > (double)C.num_pages) return KV_ERR_BUDGET;
    return map_cuda(launch_reserve(C, T, refs, row_pos, ws, (cudaStream_t)stream));
}

kv_status kv_paged_fork(const kv_paged *c, int32_t *refs, const int32_t *parents, void *stream) {
    KV_API_RANGE();
    DevPaged C;
    const kv_status st = make_paged(c, &C);
    if (st != KV_OK) return st;
    if (C.R > kForkRequests) return KV_ERR_UNSUPPORTED;
    if (C.units == 0) return KV_OK;
    if (bad_refs(C, refs) || !parents || !aligned_to(parents, 4)) return KV_ERR_INVALID_ARG;
    return map_cuda(launch_fork(C, refs, parents, (cudaStream_t)stream));
}

kv_status kv_paged_compact_workspace_size(const kv_paged *c, size_t *bytes) {
    DevPaged C;
    const kv_status st = make_paged(c, &C);
    if (st != KV_OK) return st;
    if (!bytes) return KV_ERR_INVALID_ARG;
    *bytes = compact_ws_layout(C, nullptr).total;
    return KV_OK;
}

kv_status kv_paged_compact(const kv_paged *c, int32_t *refs, int32_t *row_pos, int32_t *live,
                           void *workspace, size_t workspace_bytes, void *stream) {
    KV_API_RANGE();
    DevPaged C;
    const kv_status st = make_paged(c, &C);
    if (st != KV_OK) return st;
    if (!aligned_to(live, 4)) return KV_ERR_INVALID_ARG;
    if (C.units == 0)
        return !live ? KV_OK : map_cuda(cudaMemsetAsync(live, 0, sizeof(int32_t), (cudaStream_t)stream));
    if (bad_refs(C, refs) || !aligned16(row_pos) || bad_ptr(workspace)) return KV_ERR_INVALID_ARG;
    const PagesWs ws = compact_ws_layout(C, workspace);
    if (workspace_bytes < ws.total) return KV_ERR_WORKSPACE;
    return map_cuda(launch_compact_pages(C, refs, row_pos, live, ws, (cudaStream_t)stream));
}

kv_status kv_paged_place_positions(const kv_paged *dst, int32_t *dst_pos, const kv_paged *src,
                                   const int32_t *src_pos, const int32_t *index, int64_t stride,
                                   const int64_t *offsets, void *stream) {
    KV_API_RANGE();
    DevPaged D, S;
    kv_status st = make_paged(dst, &D);
    if (st == KV_OK && src_pos) st = make_paged(src, &S);
    else S = D;
    if (st != KV_OK) return st;
    if (src_pos && (S.R != D.R || S.L != D.L || S.H != D.H || src_pos == dst_pos))
        return KV_ERR_INVALID_ARG;
    if (D.units == 0) return KV_OK;
    if (bad_ptr(dst_pos) || stride < 0 || (src_pos && !index) || (offsets && !index) ||
        !aligned16(src_pos) || !aligned_to(index, 4) || !aligned_to(offsets, 8))
        return KV_ERR_INVALID_ARG;
    return map_cuda(launch_place_positions(D, dst_pos, S, src_pos, index, stride, offsets,
                                           (cudaStream_t)stream));
}

}  // extern "C"
