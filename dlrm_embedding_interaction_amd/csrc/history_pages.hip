// history_pages.hip -- the pages of the 8-bit history cache: appending events
// (reservation, copy of a shared page, quantisation), forking, truncating,
// trimming and compacting.
//
// refs[p] counts the histories that hold page p.  free_pages[0, counters[0])
// lists the pages without a holder in descending order, so that the lowest is
// taken first, from the end.  Every call that releases pages rebuilds the list
// from refs: its order then depends on which pages are free alone, not on the
// order in which the atomics of a call arrived.
#include "history.h"

namespace dlrm {

constexpr int kOneBlockPages = 16384;  // free-list work of one block: 1024 threads x 16 pages

// Exclusive sum of v over the block's threads in order; *total over all.
template <int THREADS>
__device__ __forceinline__ int block_exclusive(int v, int* total) {
    __shared__ int part[THREADS / 64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(inc, d, 64);
        if (lane >= d) inc += o;
    }
    __syncthreads();  // part may still be read from a call before
    if (lane == 63) part[w] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) {
        const int p = part[i];
        before += i < w ? p : 0;
        all += p;
    }
    *total = all;
    return before + inc - v;
}

__global__ __launch_bounds__(256) void history_init_kernel(dlrm_history_cache_t c) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < c.n_pages; i += step) {
        c.refs[i] = 0;
        c.free_pages[i] = c.n_pages - 1 - (int)i;
    }
    for (int64_t i = i0; i < c.n_slots; i += step) c.lens[i] = 0;
    for (int64_t i = i0; i < (int64_t)c.n_slots * c.max_pages; i += step) c.table[i] = -1;
    if (i0 < 4) c.counters[i0] = i0 == 0 ? c.n_pages : 0;
}

// ---- append ------------------------------------------------------------------

// Pages for every history of the call, by one block: a history needs the pages
// its events open, and one more where its last page is part filled and shared.
// Needs are summed in batch order; a history whose sum passes the free count is
// refused whole.  Nothing here changes refs or the table, so that every history
// of the call sees them as they were before it.
__global__ __launch_bounds__(1024) void history_reserve_kernel(AppendArgs a) {
    const dlrm_history_cache_t& c = a.c;
    __shared__ int refused, taken;
    if (threadIdx.x == 0) refused = taken = 0;
    __syncthreads();
    const int n_free = c.counters[0], pe = c.page_events;
    int carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        int need = 0, src = -1, copy = 0, slot = -1;
        int64_t old = 0, count = 0;
        bool ok = false;
        if (b < a.batch) {
            slot = a.slots ? a.slots[b] : b;
            const int64_t begin = history_begin(a.offsets, a.idx32, b, a.n_events);
            count = history_end(a.offsets, a.idx32, b, a.batch, begin, a.n_events) - begin;
            if (slot >= 0 && slot < c.n_slots) {
                old = c.lens[slot];
                ok = old >= 0 && old + count <= (int64_t)c.max_pages * pe;
            }
            if (ok && count > 0) {
                const int part = (int)(old % pe);
                if (part) {
                    src = c.table[(int64_t)slot * c.max_pages + old / pe];
                    ok = src >= 0 && src < c.n_pages;
                    copy = ok && c.refs[src] > 1;
                }
                if (ok) need = (int)((old + count + pe - 1) / pe - (old + pe - 1) / pe) + copy;
            }
        }
        int total;
        const int before = carry + block_exclusive<1024>(need, &total);
        carry += total;
        if (b < a.batch) {
            ok = ok && (need == 0 || before + need <= n_free);
            a.grants[b] = Grant{ok ? (int)old : -1, n_free - 1 - before, src, copy};
            if (ok) {
                c.lens[slot] = (int)(old + count);
                if (need) atomicMax(&taken, before + need);
            } else {
                atomicAdd(&refused, 1);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        c.counters[0] = n_free - taken;
        c.counters[1] += refused;
    }
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, bool wide, float* x) {
    if (wide) {
        if constexpr (sizeof(T) == 2) {
            typedef T v8 __attribute__((ext_vector_type(8)));
            const v8 r = *(const v8*)p;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)r[i];
        } else {
            const floatx4 r0 = *(const floatx4*)p, r1 = *(const floatx4*)(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = r0[i], x[4 + i] = r1[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)p[i];
    }
}

// Four codes of a word times a power of two, rounded to e4m3 again.
__device__ __forceinline__ unsigned rescale4(unsigned w, float f) {
    const float x0 = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * f, x1 = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * f;
    const float x2 = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * f, x3 = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * f;
    return pk_e4m3(x0, x1) | pk_e4m3(x2, x3) << 16;
}

// One block per (page an append touches, kv head, keys or values): the largest
// finite value of the new events sets the block's scale, never below the one it
// has; codes are written from registers, the values' turned through LDS into
// their event-minor order.  Events the page already holds are read only where
// the page is copied or its scale grows.
template <typename T>
__global__ __launch_bounds__(256) void history_append_kernel(AppendArgs a, int wide) {
    const dlrm_history_cache_t& c = a.c;
    __shared__ __attribute__((aligned(16))) uint8_t turned[64 * 128];
    __shared__ float wmax[4];
    const int pe = c.page_events, dim = c.head_dim, hk = blockIdx.y, tid = threadIdx.x;
    const bool minor = blockIdx.z != 0;
    const Unit un = history_of_unit(a.offsets, a.idx32, a.batch, a.n_events, pe, 2, blockIdx.x);
    const int b = un.b;
    const int64_t nth = un.nth, begin = un.begin, count = un.end - un.begin;
    const Grant g = a.grants[b];
    if (g.old_len < 0 || count == 0) return;
    const int slot = a.slots ? a.slots[b] : b;
    const int64_t first = g.old_len / pe, page_no = first + nth, stop = g.old_len + count;
    if (nth < 0 || page_no * pe >= stop) return;
    const int lo = nth == 0 ? g.old_len % pe : 0;                                  // events already in the page
    const int hi = (int)(stop - page_no * pe < pe ? stop - page_no * pe : pe);     // events after the call
    const bool kept = lo > 0 && !g.copy;
    const int opened = (int)nth - (g.src >= 0 && !g.copy ? 1 : 0);                 // of the pages taken from the list
    const int dst = kept ? g.src : c.free_pages[g.pos - opened];
    if (dst < 0 || dst >= c.n_pages) return;
    const int src = lo > 0 ? g.src : dst;

    const int64_t dst_h = (int64_t)dst * c.n_kv_heads + hk, src_h = (int64_t)src * c.n_kv_heads + hk;
    const int64_t page_bytes = (int64_t)pe * dim;
    uint8_t* codes = (minor ? c.v : c.k) + dst_h * page_bytes;
    const uint8_t* held = (minor ? c.v : c.k) + src_h * page_bytes;
    float* scales = minor ? c.v_scale : c.k_scale;
    const int64_t ld = minor ? a.ld_v : a.ld_k;
    // the page's first event stands lo events before the call's first one
    const T* x = (const T*)(minor ? a.v : a.k) + (begin + page_no * pe - g.old_len) * ld + (int64_t)hk * dim;

    const int d8 = dim / 8;               // 8-element pieces of a head: 4, 8 or 16
    const int sh = 31 - __builtin_clz(d8);
    const int lo8 = lo << sh, hi8 = hi << sh;
    float val[4][8];
    float top = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int p = lo8 + tid + r * 256;
        if (p < hi8) {
            load8(x + (int64_t)(p >> sh) * ld + (p & (d8 - 1)) * 8, wide, val[r]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float m = fabsf(val[r][i]);
                top = m < INFINITY ? fmaxf(top, m) : top;
            }
        }
    }
    top = wave_max(top);
    if ((tid & 63) == 0) wmax[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
    const float was = lo > 0 ? scales[src_h] : 0.f;
    float s = page_scale(top);
    s = was > s ? was : s;
    const float inv = 1.f / s;            // a power of two: exact
    const bool rewrite = lo > 0 && (g.copy || s > was);
    const float grown = rewrite ? was * inv : 1.f;

    uint2 code[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int p = lo8 + tid + r * 256;
        if (p < hi8) {
            code[r].x = pk_e4m3(val[r][0] * inv, val[r][1] * inv) | pk_e4m3(val[r][2] * inv, val[r][3] * inv) << 16;
            code[r].y = pk_e4m3(val[r][4] * inv, val[r][5] * inv) | pk_e4m3(val[r][6] * inv, val[r][7] * inv) << 16;
        }
    }
    if (!minor) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int p = lo8 + tid + r * 256;
            if (p < hi8) *(uint2*)(codes + p * 8) = code[r];
        }
        if (rewrite)
            for (int p = tid; p < lo8; p += 256) {
                const uint2 w = *(const uint2*)(held + p * 8);
                *(uint2*)(codes + p * 8) = make_uint2(rescale4(w.x, grown), rescale4(w.y, grown));
            }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int p = lo8 + tid + r * 256;
            if (p < hi8) {
                const int ev = p >> sh, d = (p & (d8 - 1)) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    turned[(d + i) * pe + ev] = (uint8_t)((i < 4 ? code[r].x : code[r].y) >> (8 * (i & 3)));
            }
        }
        __syncthreads();
        const int from = rewrite ? 0 : lo;
        const int pieces = dim * pe / 16;
        for (int p = tid; p < pieces; p += 256) {
            const int e0 = (p * 16) % pe;                    // the piece's first event
            if (e0 >= hi || e0 + 16 <= from) continue;
            uint4 w = *(const uint4*)(turned + p * 16);
            if (rewrite && e0 < lo) {
                const uint4 o = *(const uint4*)(held + p * 16);
                const unsigned old[4] = {rescale4(o.x, grown), rescale4(o.y, grown), rescale4(o.z, grown),
                                         rescale4(o.w, grown)};
                unsigned n[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = lo - (e0 + 4 * i);         // old events of this word
                    const unsigned m = k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
                    n[i] = (old[i] & m) | (n[i] & ~m);
                }
                w = make_uint4(n[0], n[1], n[2], n[3]);
            }
            if (e0 >= from && e0 + 16 <= hi) {
                *(uint4*)(codes + p * 16) = w;
            } else {
                const unsigned n[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (e0 + i >= from && e0 + i < hi) codes[p * 16 + i] = (uint8_t)(n[i / 4] >> (8 * (i & 3)));
            }
        }
    }
    if (tid == 0) {
        if (!kept || s != was) scales[dst_h] = s;
        if (hk == 0 && !minor && !kept) {
            c.table[(int64_t)slot * c.max_pages + page_no] = dst;
            c.refs[dst] = 1;
            if (lo > 0) atomicSub(&c.refs[src], 1);
        }
    }
}

// ---- sharing and releasing -----------------------------------------------------

__device__ __forceinline__ void release_entry(const dlrm_history_cache_t& c, int64_t at) {
    const int p = atomicExch(&c.table[at], -1);
    if (p >= 0 && p < c.n_pages) atomicSub(&c.refs[p], 1);
}

__global__ __launch_bounds__(256) void history_fork_kernel(dlrm_history_cache_t c, const int32_t* src,
                                                           const int32_t* dst) {
    const int from = src[blockIdx.x], to = dst[blockIdx.x];
    if (from < 0 || from >= c.n_slots || to < 0 || to >= c.n_slots) {
        if (threadIdx.x == 0) atomicAdd(&c.counters[1], 1);
        return;
    }
    if (from == to) return;
    const int64_t f = (int64_t)from * c.max_pages, t = (int64_t)to * c.max_pages;
    for (int i = threadIdx.x; i < c.max_pages; i += 256) {
        const int p = c.table[f + i], o = c.table[t + i];
        if (p == o) continue;
        c.table[t + i] = p;
        if (p >= 0 && p < c.n_pages) atomicAdd(&c.refs[p], 1);
        if (o >= 0 && o < c.n_pages) atomicSub(&c.refs[o], 1);
    }
    if (threadIdx.x == 0) c.lens[to] = c.lens[from];
}

__global__ __launch_bounds__(256) void history_truncate_kernel(dlrm_history_cache_t c, const int32_t* slots,
                                                               const int32_t* new_lens) {
    const int slot = slots[blockIdx.x], want = new_lens ? new_lens[blockIdx.x] : 0, pe = c.page_events;
    bool ok = slot >= 0 && slot < c.n_slots && want >= 0;
    if (ok) ok = want <= c.lens[slot] && want <= (int64_t)c.max_pages * pe;
    const int64_t row = (int64_t)slot * c.max_pages;
    // the page that would be filled further may have been trimmed away
    if (ok && want % pe) ok = c.table[row + want / pe] >= 0;
    __syncthreads();  // every thread has read the length
    if (!ok) {
        if (threadIdx.x == 0) atomicAdd(&c.counters[1], 1);
        return;
    }
    for (int64_t i = ((int64_t)want + pe - 1) / pe + threadIdx.x; i < c.max_pages; i += 256) release_entry(c, row + i);
    if (threadIdx.x == 0) c.lens[slot] = want;
}

__global__ __launch_bounds__(256) void history_trim_kernel(dlrm_history_cache_t c, const int32_t* slots,
                                                           int64_t window, int64_t sinks) {
    const int slot = slots[blockIdx.x], pe = c.page_events;
    if (slot < 0 || slot >= c.n_slots) {
        if (threadIdx.x == 0) atomicAdd(&c.counters[1], 1);
        return;
    }
    const int64_t row = (int64_t)slot * c.max_pages;
    // pages whose events all lie behind the sinks and before the window
    const int64_t lo = sinks < (int64_t)c.max_pages * pe ? (sinks + pe - 1) / pe : c.max_pages;
    int64_t hi = c.lens[slot] > window ? (c.lens[slot] - window) / pe : 0;
    hi = hi < c.max_pages ? hi : c.max_pages;
    for (int64_t i = lo + threadIdx.x; i < hi; i += 256) release_entry(c, row + i);
}

// Free pages of each chunk.
__global__ __launch_bounds__(256) void history_count_kernel(dlrm_history_cache_t c, int32_t* counts) {
    const int base = blockIdx.x * kRebuildChunk;
    int n = 0;
    for (int i = threadIdx.x; i < kRebuildChunk; i += 256)
        n += base + i < c.n_pages && c.refs[base + i] == 0 ? 1 : 0;
    int total;
    block_exclusive<256>(n, &total);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// Writes the chunk's free pages: page p goes to the place that counts the free
// pages above it.
template <int THREADS, int PER>
__device__ __forceinline__ void list_free(const dlrm_history_cache_t& c, int base, int above) {
    const int p0 = base + (int)threadIdx.x * PER;
    int n = 0;
    bool free[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        free[i] = p0 + i < c.n_pages && c.refs[p0 + i] == 0;
        n += free[i] ? 1 : 0;
    }
    int total;
    const int before = block_exclusive<THREADS>(n, &total);
    int at = above + total - before - 1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (free[i]) c.free_pages[at--] = p0 + i;
    if (base == 0 && threadIdx.x == 0) c.counters[0] = above + total;
}

__global__ __launch_bounds__(1024) void history_rebuild_one_kernel(dlrm_history_cache_t c) {
    list_free<1024, kOneBlockPages / 1024>(c, 0, 0);
}

__global__ __launch_bounds__(256) void history_rebuild_kernel(dlrm_history_cache_t c, const int32_t* counts) {
    int n = 0;
    for (int i = blockIdx.x + 1 + threadIdx.x; i < (int)gridDim.x; i += 256) n += counts[i];
    int above;
    block_exclusive<256>(n, &above);
    list_free<256, kRebuildChunk / 256>(c, blockIdx.x * kRebuildChunk, above);
}

static hipError_t rebuild(const dlrm_history_cache_t& c, int32_t* counts, hipStream_t s) {
    if (c.n_pages <= kOneBlockPages) {
        hipLaunchKernelGGL(history_rebuild_one_kernel, dim3(1), dim3(1024), 0, s, c);
    } else {
        const int n = rebuild_chunks(c.n_pages);
        hipLaunchKernelGGL(history_count_kernel, dim3(n), dim3(256), 0, s, c, counts);
        hipLaunchKernelGGL(history_rebuild_kernel, dim3(n), dim3(256), 0, s, c, counts);
    }
    return hipGetLastError();
}

// ---- compaction ------------------------------------------------------------------

// With m pages in use, the i-th used page at or above m moves to the i-th free
// page below m.  Workspace: chunk counts, the number of moves, the pages that
// move, the pages they move to, and the new place of each page.
struct MoveWs {
    int32_t *counts, *n, *from, *to, *place;
};
static MoveWs move_ws(const dlrm_history_cache_t& c, int32_t* ws) {
    MoveWs w;
    w.counts = ws;
    w.n = ws + rebuild_chunks(c.n_pages);
    w.from = w.n + 1;
    w.to = w.from + c.n_pages;
    w.place = w.to + c.n_pages;
    return w;
}

__global__ __launch_bounds__(256) void history_plan_kernel(dlrm_history_cache_t c, MoveWs w, int chunks) {
    // free pages in all, before this chunk, and before page m
    int n = 0, nb = 0, total, before;
    for (int i = threadIdx.x; i < chunks; i += 256) {
        const int k = w.counts[i];
        n += k;
        nb += i < (int)blockIdx.x ? k : 0;
    }
    block_exclusive<256>(n, &total);
    block_exclusive<256>(nb, &before);
    const int m = c.n_pages - total, m_chunk = m / kRebuildChunk;
    int nm = 0, holes;
    for (int i = threadIdx.x; i < m_chunk && i < chunks; i += 256) nm += w.counts[i];
    for (int p = m_chunk * kRebuildChunk + threadIdx.x; p < m; p += 256) nm += c.refs[p] == 0 ? 1 : 0;
    block_exclusive<256>(nm, &holes);
    constexpr int PER = kRebuildChunk / 256;
    const int p0 = (int)blockIdx.x * kRebuildChunk + (int)threadIdx.x * PER;
    int k = 0, sum;
    bool free[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        free[i] = p0 + i < c.n_pages && c.refs[p0 + i] == 0;
        k += free[i] ? 1 : 0;
    }
    int fb = before + block_exclusive<256>(k, &sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int p = p0 + i;
        if (p >= c.n_pages) break;
        // used pages before p and at or above m: (p - fb) - (m - holes)
        if (free[i] && p < m) w.to[fb] = p;
        if (!free[i] && p >= m) w.from[p - fb - (m - holes)] = p;
        fb += free[i] ? 1 : 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *w.n = holes;
        c.counters[0] = total;
    }
}

__global__ __launch_bounds__(256) void history_move_kernel(dlrm_history_cache_t c, MoveWs w) {
    const int n = *w.n;
    const int64_t vecs = (int64_t)c.n_kv_heads * c.page_events * c.head_dim / 16;
    for (int r = blockIdx.x; r < n; r += gridDim.x) {
        const int from = w.from[r], to = w.to[r];
        const uint4 *k0 = (const uint4*)c.k + from * vecs, *v0 = (const uint4*)c.v + from * vecs;
        uint4 *k1 = (uint4*)c.k + to * vecs, *v1 = (uint4*)c.v + to * vecs;
        for (int64_t i = threadIdx.x; i < vecs; i += 256) {
            k1[i] = k0[i];
            v1[i] = v0[i];
        }
        for (int h = threadIdx.x; h < c.n_kv_heads; h += 256) {
            c.k_scale[(int64_t)to * c.n_kv_heads + h] = c.k_scale[(int64_t)from * c.n_kv_heads + h];
            c.v_scale[(int64_t)to * c.n_kv_heads + h] = c.v_scale[(int64_t)from * c.n_kv_heads + h];
        }
        if (threadIdx.x == 0) {
            w.place[from] = to;
            c.refs[to] = c.refs[from];
            c.refs[from] = 0;
        }
    }
}

__global__ __launch_bounds__(256) void history_relabel_kernel(dlrm_history_cache_t c, MoveWs w) {
    const int n_free = c.counters[0], m = c.n_pages - n_free;
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < n_free; i += step) c.free_pages[i] = c.n_pages - 1 - (int)i;
    for (int64_t i = i0; i < (int64_t)c.n_slots * c.max_pages; i += step) {
        const int p = c.table[i];
        if (p >= m && p < c.n_pages) c.table[i] = w.place[p];
    }
}

// ---- launches ----------------------------------------------------------------------

static unsigned grid_for(int64_t items, int most) {
    const int64_t g = (items + 255) / 256;
    return (unsigned)(g < 1 ? 1 : (g > most ? most : g));
}

hipError_t launch_history_init(const dlrm_history_cache_t& c, hipStream_t s) {
    hipLaunchKernelGGL(history_init_kernel, dim3(grid_for((int64_t)c.n_slots * c.max_pages + c.n_pages, 2048)),
                       dim3(256), 0, s, c);
    return hipGetLastError();
}

hipError_t launch_history_append(const AppendArgs& a, int dtype, hipStream_t s) {
    hipLaunchKernelGGL(history_reserve_kernel, dim3(1), dim3(1024), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_events == 0) return e;
    const dim3 grid((unsigned)(a.n_events / a.c.page_events + 2 * (int64_t)a.batch), (unsigned)a.c.n_kv_heads, 2);
    const int step = dtype == DLRM_DTYPE_F32 ? 4 : 8;
    const int wide = a.ld_k % step == 0 && a.ld_v % step == 0 && (((uintptr_t)a.k | (uintptr_t)a.v) & 15u) == 0;
    if (dtype == DLRM_DTYPE_F32) hipLaunchKernelGGL(history_append_kernel<float>, grid, dim3(256), 0, s, a, wide);
    else if (dtype == DLRM_DTYPE_BF16) hipLaunchKernelGGL(history_append_kernel<bf16>, grid, dim3(256), 0, s, a, wide);
    else hipLaunchKernelGGL(history_append_kernel<f16>, grid, dim3(256), 0, s, a, wide);
    return hipGetLastError();
}

hipError_t launch_history_fork(const dlrm_history_cache_t& c, int n, const int32_t* src, const int32_t* dst,
                               int32_t* counts, hipStream_t s) {
    hipLaunchKernelGGL(history_fork_kernel, dim3(n), dim3(256), 0, s, c, src, dst);
    hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : rebuild(c, counts, s);
}

hipError_t launch_history_truncate(const dlrm_history_cache_t& c, int n, const int32_t* slots,
                                   const int32_t* new_lens, int32_t* counts, hipStream_t s) {
    hipLaunchKernelGGL(history_truncate_kernel, dim3(n), dim3(256), 0, s, c, slots, new_lens);
    hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : rebuild(c, counts, s);
}

hipError_t launch_history_trim(const dlrm_history_cache_t& c, int n, const int32_t* slots, int64_t window,
                               int64_t sinks, int32_t* counts, hipStream_t s) {
    hipLaunchKernelGGL(history_trim_kernel, dim3(n), dim3(256), 0, s, c, slots, window, sinks);
    hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : rebuild(c, counts, s);
}

hipError_t launch_history_compact(const dlrm_history_cache_t& c, int32_t* ws, hipStream_t s) {
    const MoveWs w = move_ws(c, ws);
    const int chunks = rebuild_chunks(c.n_pages);
    hipLaunchKernelGGL(history_count_kernel, dim3(chunks), dim3(256), 0, s, c, w.counts);
    hipLaunchKernelGGL(history_plan_kernel, dim3(chunks), dim3(256), 0, s, c, w, chunks);
    hipLaunchKernelGGL(history_move_kernel, dim3(c.n_pages < 2048 ? c.n_pages : 2048), dim3(256), 0, s, c, w);
    hipLaunchKernelGGL(history_relabel_kernel,
                       dim3(grid_for((int64_t)c.n_slots * c.max_pages + c.n_pages, 2048)), dim3(256), 0, s, c, w);
    return hipGetLastError();
}

}  // namespace dlrm
