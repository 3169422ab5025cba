// history_api.hip -- extern "C" entry points of the event-history operators
// (declared in include/dlrm_mi355x.h).  Host code only: argument validation,
// workspace planning and kernel launches on the caller's stream.
#include <stdint.h>

#include "history.h"

#define DLRM_API extern "C" __attribute__((visibility("default")))

using namespace dlrm;

namespace {

constexpr int64_t kIntLimit = (int64_t)1 << 30;
inline dlrm_status_t from_hip(hipError_t e) {
    return e == hipSuccess ? DLRM_OK : (e == kTooLarge ? DLRM_E_UNSUPPORTED : DLRM_E_HIP);
}
inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }

bool known_dtype(int32_t t) { return t == DLRM_DTYPE_F32 || t == DLRM_DTYPE_BF16 || t == DLRM_DTYPE_F16; }
bool known_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }

dlrm_status_t check_attention(const dlrm_attention_t* a) {
    if (!a) return DLRM_E_NULL;
    if (!known_dtype(a->dtype) || a->n_heads < 1 || a->n_kv_heads < 1 || a->n_heads % a->n_kv_heads != 0 ||
        a->head_dim < 1 || a->window < 1 || a->sinks < 0)
        return DLRM_E_SHAPE;
    if (!(a->scale >= -3.0e38f && a->scale <= 3.0e38f)) return DLRM_E_SHAPE;
    if (!known_dim(a->head_dim) || a->n_heads > 4096) return DLRM_E_UNSUPPORTED;
    return DLRM_OK;
}

dlrm_status_t check_cache(const dlrm_history_cache_t* c) {
    if (!c) return DLRM_E_NULL;
    if (c->n_pages < 1 || c->page_events < 1 || c->n_kv_heads < 1 || c->head_dim < 1 || c->n_slots < 1 ||
        c->max_pages < 1)
        return DLRM_E_SHAPE;
    if (!known_dim(c->head_dim) || (c->page_events != 16 && c->page_events != 32 && c->page_events != 64))
        return DLRM_E_UNSUPPORTED;
    if (c->n_kv_heads > 4096 || c->n_pages > kIntLimit || (int64_t)c->max_pages * c->page_events > kIntLimit)
        return DLRM_E_UNSUPPORTED;
    return DLRM_OK;
}
dlrm_status_t check_cache_pointers(const dlrm_history_cache_t* c) {
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->lens || !c->refs || !c->free_pages ||
        !c->counters)
        return DLRM_E_NULL;
    if ((((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->refs) & 15u) != 0) return DLRM_E_SHAPE;
    return DLRM_OK;
}

// Whether the lookup's tiles fit an int and its chunks of query rows a grid.
bool lookup_fits(const dlrm_history_cache_t* c, int64_t batch, int32_t queries, int32_t n_heads) {
    const int64_t rows = (int64_t)queries * (n_heads / c->n_kv_heads);
    const int64_t tiles = ((int64_t)c->max_pages * c->page_events + 63) / 64;
    return (int64_t)queries * batch <= kIntLimit && (rows + 15) / 16 * c->n_kv_heads <= 65535 &&
           batch * tiles <= kIntLimit;
}

// Bytes for the chunk counts and the lists of a compaction.
size_t compact_bytes(const dlrm_history_cache_t* c) {
    return round256(((size_t)3 * c->n_pages + rebuild_chunks(c->n_pages) + 1) * sizeof(int32_t));
}

size_t workspace_bytes(const dlrm_history_cache_t* c, int64_t batch, int32_t queries, int32_t n_heads) {
    size_t n = compact_bytes(c);
    const size_t needs = round256(need_bytes(batch));
    n = needs > n ? needs : n;
    if (queries > 0) {
        const size_t l = round256(lookup_workspace_bytes(*c, batch, queries, n_heads));
        n = l > n ? l : n;
    }
    return n;
}

dlrm_status_t check_workspace(const void* ws, size_t have, size_t need) {
    if (!ws || have < need || ((uintptr_t)ws & 255u) != 0) return DLRM_E_WORKSPACE;
    return DLRM_OK;
}

dlrm_status_t check_ready(const dlrm_history_cache_t* c) {
    const dlrm_status_t st = check_cache(c);
    return st != DLRM_OK ? st : check_cache_pointers(c);
}

}  // namespace

DLRM_API dlrm_status_t dlrm_history_attention(const dlrm_attention_t* a, int64_t batch, int64_t n_events,
                                              const void* offsets, int32_t index_bytes, const void* q, int64_t ld_q,
                                              const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                              const uint8_t* padding, void* out, int64_t ld_out, void* stream) {
    const dlrm_status_t st = check_attention(a);
    if (st != DLRM_OK) return st;
    if (batch < 1 || n_events < 0 || (index_bytes != 4 && index_bytes != 8)) return DLRM_E_SHAPE;
    if (batch > kIntLimit || n_events > kIntLimit) return DLRM_E_UNSUPPORTED;
    if (!offsets) return DLRM_E_NULL;
    if (n_events == 0) return DLRM_OK;
    if (!q || !k || !v || !out) return DLRM_E_NULL;
    const int64_t wq = (int64_t)a->n_heads * a->head_dim, wk = (int64_t)a->n_kv_heads * a->head_dim;
    if (ld_q < wq || ld_k < wk || ld_v < wk || ld_out < wq) return DLRM_E_SHAPE;
    if (ld_k > kIntLimit || ld_v > kIntLimit) return DLRM_E_UNSUPPORTED;
    EncodeArgs e = {};
    e.q = q, e.k = k, e.v = v, e.offsets = offsets, e.padding = padding, e.out = out;
    e.ld_q = ld_q, e.ld_k = ld_k, e.ld_v = ld_v, e.ld_out = ld_out;
    e.n_events = n_events;
    e.window = a->window, e.sinks = a->sinks;
    e.batch = (int)batch, e.n_heads = a->n_heads, e.n_kv = a->n_kv_heads, e.idx32 = index_bytes == 4;
    e.scale = a->scale;
    return from_hip(launch_history_attention(e, a->dtype, a->head_dim, (hipStream_t)stream));
}

DLRM_API size_t dlrm_history_workspace_bytes(const dlrm_history_cache_t* c, int64_t batch, int32_t queries,
                                             int32_t n_heads) {
    if (check_cache(c) != DLRM_OK || batch < 1 || batch > kIntLimit || queries < 0 || n_heads < 0) return 0;
    if (queries > 0 && (n_heads < 1 || n_heads > 4096 || n_heads % c->n_kv_heads != 0)) return 0;
    if (queries > 0 && !lookup_fits(c, batch, queries, n_heads)) return 0;
    return workspace_bytes(c, batch, queries, n_heads);
}

DLRM_API dlrm_status_t dlrm_history_init(const dlrm_history_cache_t* c, void* stream) {
    const dlrm_status_t st = check_ready(c);
    if (st != DLRM_OK) return st;
    return from_hip(launch_history_init(*c, (hipStream_t)stream));
}

DLRM_API dlrm_status_t dlrm_history_append(const dlrm_history_cache_t* c, int64_t batch, const int32_t* slots,
                                           int32_t dtype, int64_t n_events, const void* offsets,
                                           int32_t index_bytes, const void* k, int64_t ld_k, const void* v,
                                           int64_t ld_v, void* workspace, size_t ws_bytes, void* stream) {
    dlrm_status_t st = check_ready(c);
    if (st != DLRM_OK) return st;
    if (batch < 1 || n_events < 0 || !known_dtype(dtype) || (index_bytes != 4 && index_bytes != 8))
        return DLRM_E_SHAPE;
    if (!slots && batch > c->n_slots) return DLRM_E_SHAPE;
    if (batch > kIntLimit / 4 || n_events > kIntLimit) return DLRM_E_UNSUPPORTED;
    if (!offsets || (n_events > 0 && (!k || !v))) return DLRM_E_NULL;
    const int64_t w = (int64_t)c->n_kv_heads * c->head_dim;
    if (ld_k < w || ld_v < w) return DLRM_E_SHAPE;
    st = check_workspace(workspace, ws_bytes, round256(need_bytes(batch)));
    if (st != DLRM_OK) return st;
    AppendArgs a = {};
    a.c = *c;
    a.slots = slots, a.k = k, a.v = v, a.offsets = offsets;
    a.ws.need = (Need*)workspace;
    a.ws.sums = (int2*)(a.ws.need + batch);
    a.ws.n_free = (int*)(a.ws.sums + batch / kNeedBlock + 1);
    a.ld_k = ld_k, a.ld_v = ld_v, a.n_events = n_events;
    a.batch = (int)batch, a.idx32 = index_bytes == 4;
    return from_hip(launch_history_append(a, dtype, (hipStream_t)stream));
}

DLRM_API dlrm_status_t dlrm_history_lookup(const dlrm_history_cache_t* c, const dlrm_attention_t* at, int64_t batch,
                                           const int32_t* slots, int32_t queries, const void* q, int64_t ld_q,
                                           void* out, int64_t ld_out, void* workspace, size_t ws_bytes,
                                           void* stream) {
    dlrm_status_t st = check_ready(c);
    if (st != DLRM_OK) return st;
    st = check_attention(at);
    if (st != DLRM_OK) return st;
    if (!q || !out) return DLRM_E_NULL;
    if (at->n_kv_heads != c->n_kv_heads || at->head_dim != c->head_dim || batch < 1 || queries < 1)
        return DLRM_E_SHAPE;
    if (!slots && batch > c->n_slots) return DLRM_E_SHAPE;
    if (batch > kIntLimit || !lookup_fits(c, batch, queries, at->n_heads)) return DLRM_E_UNSUPPORTED;
    const int64_t w = (int64_t)at->n_heads * at->head_dim;
    if (ld_q < w || ld_out < w) return DLRM_E_SHAPE;
    st = check_workspace(workspace, ws_bytes, round256(lookup_workspace_bytes(*c, batch, queries, at->n_heads)));
    if (st != DLRM_OK) return st;
    LookupArgs a = {};
    a.c = *c;
    a.slots = slots, a.q = q, a.out = out;
    a.partial = (float*)workspace;
    a.ld_q = ld_q, a.ld_out = ld_out;
    a.window = at->window, a.sinks = at->sinks;
    a.batch = (int)batch, a.queries = queries, a.n_heads = at->n_heads;
    const int64_t step = at->dtype == DLRM_DTYPE_F32 ? 4 : 8;
    a.wide = ld_q % step == 0 && ld_out % step == 0 && (((uintptr_t)q | (uintptr_t)out) & 15u) == 0;
    a.scale = at->scale;
    return from_hip(launch_history_lookup(a, at->dtype, (hipStream_t)stream));
}

namespace {

// Checks shared by the calls that release pages.
dlrm_status_t check_release(const dlrm_history_cache_t* c, int64_t n, const int32_t* slots, const void* ws,
                            size_t ws_bytes) {
    const dlrm_status_t st = check_ready(c);
    if (st != DLRM_OK) return st;
    if (n < 1) return DLRM_E_SHAPE;
    if (n > kIntLimit) return DLRM_E_UNSUPPORTED;
    if (!slots) return DLRM_E_NULL;
    return check_workspace(ws, ws_bytes, compact_bytes(c));
}

}  // namespace

DLRM_API dlrm_status_t dlrm_history_fork(const dlrm_history_cache_t* c, int64_t n, const int32_t* src,
                                         const int32_t* dst, void* workspace, size_t ws_bytes, void* stream) {
    const dlrm_status_t st = check_release(c, n, src, workspace, ws_bytes);
    if (st != DLRM_OK) return st;
    if (!dst) return DLRM_E_NULL;
    return from_hip(launch_history_fork(*c, (int)n, src, dst, (int32_t*)workspace, (hipStream_t)stream));
}

DLRM_API dlrm_status_t dlrm_history_truncate(const dlrm_history_cache_t* c, int64_t n, const int32_t* slots,
                                             const int32_t* new_lens, void* workspace, size_t ws_bytes,
                                             void* stream) {
    const dlrm_status_t st = check_release(c, n, slots, workspace, ws_bytes);
    if (st != DLRM_OK) return st;
    return from_hip(launch_history_truncate(*c, (int)n, slots, new_lens, (int32_t*)workspace, (hipStream_t)stream));
}

DLRM_API dlrm_status_t dlrm_history_trim(const dlrm_history_cache_t* c, int64_t n, const int32_t* slots,
                                         int64_t window, int64_t sinks, void* workspace, size_t ws_bytes,
                                         void* stream) {
    const dlrm_status_t st = check_release(c, n, slots, workspace, ws_bytes);
    if (st != DLRM_OK) return st;
    if (window < 1 || sinks < 0) return DLRM_E_SHAPE;
    return from_hip(launch_history_trim(*c, (int)n, slots, window, sinks, (int32_t*)workspace, (hipStream_t)stream));
}

DLRM_API dlrm_status_t dlrm_history_compact(const dlrm_history_cache_t* c, void* workspace, size_t ws_bytes,
                                            void* stream) {
    dlrm_status_t st = check_ready(c);
    if (st != DLRM_OK) return st;
    st = check_workspace(workspace, ws_bytes, compact_bytes(c));
    if (st != DLRM_OK) return st;
    return from_hip(launch_history_compact(*c, (int32_t*)workspace, (hipStream_t)stream));
}
