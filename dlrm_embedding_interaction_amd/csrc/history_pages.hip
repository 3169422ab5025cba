// history_pages.hip -- the pages of the 8-bit history cache: appending events
// (reservation, copy of a shared page, quantisation), forking, truncating,
// trimming and compacting.
//
// refs[p] counts the histories that hold page p.  free_pages[0, counters[0])
// lists the pages without a holder in descending order, so that the lowest is
// taken first, from the end.  Every call that releases pages rebuilds the list
// from refs: its order then depends on which pages are free alone, not on the
// order in which the atomics of a call arrived.
//
// Measured on MI355X: appending 128 histories of up to 1000 events, 8 kv heads of
// 128, bf16 (466 MB): 101 us, 4.6 TB/s, against 5.0 for a large copy.  One event for
// each of 512 histories: 8 us, of 1500 with a copied page each 42: there a wave's
// five dependent reads (offsets, need, list, scale, codes) are what it takes.  The
// list of 32000 pages 7 us, of 11000 5.
#include "history.h"

namespace dlrm {

// Pools up to here have their free list written by one block, larger ones in two launches of many.  32768 pages 12 us
// against 9, which a call that is not in a graph loses to the host's time for the launch; 65536 pages 20 against 9.
constexpr int kOneBlockPages = 32768;   // at most 65536, what sixteen waves hold

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

// What each history needs, one thread each: the pages its events open, and one
// more where its last page is part filled and shared.  Nothing here changes refs,
// lengths or the table, so that every history of the call sees them as they were
// before it.  What it takes is the chain slot -> length -> page -> holders of
// dependent reads, spread over as many CUs as there are blocks.
__global__ __launch_bounds__(kNeedBlock) void history_need_kernel(AppendArgs a) {
    const dlrm_history_cache_t& c = a.c;
    const int b = blockIdx.x * kNeedBlock + threadIdx.x, pe = c.page_events;
    const int sh = 31 - __builtin_clz(pe), mask = pe - 1;
    Need d = {-1, -1, 0, 0};
    bool ok = false;
    if (b < a.batch) {
        const int slot = a.slots ? a.slots[b] : b;
        const int64_t begin = history_begin(a.offsets, a.idx32, b, a.n_events);
        const int64_t count = history_end(a.offsets, a.idx32, b, a.batch, begin, a.n_events) - begin;
        if (slot >= 0 && slot < c.n_slots) {
            d.old_len = c.lens[slot];
            ok = d.old_len >= 0 && d.old_len + count <= (int64_t)c.max_pages << sh;
        }
        if (ok && count > 0) {
            if (d.old_len & mask) {
                d.src = c.table[(int64_t)slot * c.max_pages + (d.old_len >> sh)];
                ok = d.src >= 0 && d.src < c.n_pages;
                d.copy = ok && c.refs[d.src] > 1;
            }
            if (ok) d.pages = ((d.old_len + (int)count + mask) >> sh) - ((d.old_len + mask) >> sh) + d.copy;
        }
        if (!ok) d.old_len = -1;
        a.ws.need[b] = d;
    }
    int pages, refused;
    block_exclusive<kNeedBlock>(d.pages, &pages);
    block_exclusive<kNeedBlock>(b < a.batch && !ok ? 1 : 0, &refused);
    if (threadIdx.x == 0) {
        a.ws.sums[blockIdx.x] = make_int2(pages, refused);
        // the list has n_pages places, whatever the counter holds
        if (blockIdx.x == 0) *a.ws.n_free = min(max(c.counters[0], 0), c.n_pages);
    }
}

// Pages of the histories before b, by one wave.
__device__ __forceinline__ int pages_before(const NeedWs& ws, int b) {
    const int lane = threadIdx.x & 63, b0 = b / kNeedBlock * kNeedBlock;
    int n = 0;
    for (int i = lane; i < b / kNeedBlock; i += 64) n += ws.sums[i].x;
#pragma unroll
    for (int i = 0; i < kNeedBlock; i += 64)
        if (b0 + i + lane < b) n += ws.need[b0 + i + lane].pages;
#pragma unroll
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d, 64);
    return n;
}

// Needs are met in batch order; a history whose running sum passes the free
// count is refused whole.
__device__ __forceinline__ bool met(const Need& d, int before, int n_free) {
    return d.old_len >= 0 && (d.pages == 0 || before + d.pages <= n_free);
}

// The free and refused counts after the call, by one block.
__device__ __forceinline__ void settle(const AppendArgs& a) {
    const int tid = threadIdx.x, n_free = *a.ws.n_free;
    int pages = 0, refused = 0, total, no;
    for (int i = tid; i < (a.batch + kNeedBlock - 1) / kNeedBlock; i += 256) {
        const int2 s = a.ws.sums[i];
        pages += s.x;
        refused += s.y;
    }
    block_exclusive<256>(pages, &total);
    block_exclusive<256>(refused, &no);
    int taken = total;
    if (total > n_free) {                   // not everyone is met
        int carry = 0, most = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 256) {
            const int b = b0 + tid;
            const Need d = b < a.batch ? a.ws.need[b] : Need{0, -1, 0, 0};
            int sum, out;
            const int before = carry + block_exclusive<256>(d.pages, &sum);
            carry += sum;
            const bool ok = met(d, before, n_free);
            if (ok && d.pages) most = before + d.pages;
            block_exclusive<256>(d.old_len >= 0 && !ok ? 1 : 0, &out);
            no += out;
        }
        __shared__ int top;
        if (tid == 0) top = 0;
        __syncthreads();
        if (most) atomicMax(&top, most);
        __syncthreads();
        taken = top;
    }
    if (tid == 0) {
        a.c.counters[0] = n_free - taken;
        a.c.counters[1] += no;
    }
}

// Two values over a power-of-two scale as two codes, into the low or high half.
typedef short short2v __attribute__((ext_vector_type(2)));
template <bool HIGH>
__device__ __forceinline__ short2v code2(short2v w, bf16 a, bf16 b, float s) {
    typedef bf16 v __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, v{a, b}, s, HIGH);
}
template <bool HIGH>
__device__ __forceinline__ short2v code2(short2v w, f16 a, f16 b, float s) {
    typedef f16 v __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, v{a, b}, s, HIGH);
}
template <bool HIGH>
__device__ __forceinline__ short2v code2(short2v w, float a, float b, float s) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, s, HIGH);
}
template <typename T>
__device__ __forceinline__ unsigned code4(T a, T b, T c, T d, float s) {
    return __builtin_bit_cast(unsigned, code2<true>(code2<false>(short2v{}, a, b, s), c, d, s));
}

// At the largest scale, 2^120, code 0x78 would stand for 2^128, past every finite
// fp32 and bf16 value: values that would round to it get the code before, 0x77.
constexpr float kLargestScale = 0x1p120f;
__device__ __forceinline__ unsigned keep_finite(unsigned w) {
    const unsigned differ = ((w & 0x7f7f7f7fu) ^ 0x78787878u) + 0x7f7f7f7fu;    // bit 7 of each byte: not 0x78
    return w - (~differ >> 7 & 0x01010101u);
}

// Word k of 16-lane row q goes to word q of row k.
__device__ __forceinline__ void exchange4(unsigned* w) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const auto r = __builtin_amdgcn_permlane32_swap(w[k], w[k + 2], false, false);
        w[k] = r[0];
        w[k + 2] = r[1];
    }
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const auto r = __builtin_amdgcn_permlane16_swap(w[k], w[k + 1], false, false);
        w[k] = r[0];
        w[k + 1] = r[1];
    }
}

// Four codes of a word over a power of two, rounded to e4m3 again.
__device__ __forceinline__ unsigned rescale4(unsigned w, float s) {
    return code4(__builtin_amdgcn_cvt_f32_fp8((int)w, 0), __builtin_amdgcn_cvt_f32_fp8((int)w, 1),
                 __builtin_amdgcn_cvt_f32_fp8((int)w, 2), __builtin_amdgcn_cvt_f32_fp8((int)w, 3), s);
}

// The element with the largest finite magnitude over the wave: bits decide, and
// only where they show an infinity or NaN are the elements looked at one by one.
template <typename T, int N>
__device__ __forceinline__ float wave_magnitude(const Raw<T>* raw, const bool* in) {
    unsigned bits = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (in[i]) top_magnitude(raw[i], bits);
    float top;
    if constexpr (sizeof(T) == 2) {
        const unsigned m = (bits & 0xffffu) > bits >> 16 ? bits & 0xffffu : bits >> 16;
        top = (float)__builtin_bit_cast(T, (unsigned short)m);
    } else {
        top = __uint_as_float(bits);
    }
    if (__any(odd_magnitude<T>(bits))) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (in[i])
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float m = fabsf((float)raw[i].x[x]);
                    top = m < INFINITY ? fmaxf(top, m) : top;
                }
    }
    return wave_max(top);
}

// Bytes of word w of a 16-event group that lie below event `to` of the group.
__device__ __forceinline__ unsigned bytes_below(int to, int w) {
    const int k = to - 4 * w;
    return k >= 4 ? ~0u : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
}

// One wave per (page an append touches, kv head, keys or values).  The largest
// finite value of the new events sets the block's scale, never below the one it has; the events
// stay in registers from the load to the codes.  A lane takes four consecutive
// events of eight elements: the codes of the four events of one element make a
// word of the event-minor value page, and exchanging words between the four
// 16-lane rows makes whole 16-byte pieces of it, without LDS.  Events the page
// already holds are read only where the page is copied, its scale grows, or they
// share a 16-byte piece with new values.  The last block settles the counts.
template <typename T, int D, int PE, bool WIDE>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) void history_append_kernel(AppendArgs a) {
    const dlrm_history_cache_t& c = a.c;
    constexpr int C8 = D / 8;                            // 8-element pieces of a head
    constexpr int EV = 2048 / D;                         // events of one round of the wave
    constexpr int ROUNDS = PE > EV ? PE / EV : 1;
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) settle(a);
        return;
    }
    const int lane = threadIdx.x & 63;
    const int item = __builtin_amdgcn_readfirstlane((int)blockIdx.y * 4 + (int)(threadIdx.x >> 6));
    if (item >= 2 * c.n_kv_heads) return;
    // Units are pages, with room for two more than a history's events fill; or, where that would be more, its
    // events, of which the first in each page does the page's work.
    Unit un = history_of_unit(a.offsets, a.idx32, a.batch, a.n_events, a.per_event ? 1 : PE, a.per_event ? 0 : 2,
                              blockIdx.x);
    const int64_t count = un.end - un.begin;
    const Need g = a.ws.need[un.b];
    const int slot = a.slots ? a.slots[un.b] : un.b;
    if (un.nth < 0 || g.old_len < 0 || count == 0) return;
    if (a.per_event) {
        const int64_t at = g.old_len + un.nth;
        if (un.nth >= count || (un.nth > 0 && at % PE != 0)) return;
        un.nth = at / PE - g.old_len / PE;
    }
    const int64_t page_no = g.old_len / PE + un.nth, stop = g.old_len + count;
    if (page_no * PE >= stop) return;
    const int n_free = *a.ws.n_free, before = pages_before(a.ws, un.b);
    if (!met(g, before, n_free)) return;
    const int lo = un.nth == 0 ? g.old_len % PE : 0;                               // events already in the page
    const int hi = (int)(stop - page_no * PE < PE ? stop - page_no * PE : PE);     // events after the call
    const bool kept = lo > 0 && !g.copy;
    const int opened = (int)un.nth - (g.src >= 0 && !g.copy ? 1 : 0);              // of the pages taken from the list
    const int dst = kept ? g.src : c.free_pages[n_free - 1 - before - opened];
    if (dst < 0 || dst >= c.n_pages) return;
    const int src = lo > 0 ? g.src : dst;
    const int ch = lane % C8, quad = (lane >> 4) + 4 * ((lane & 15) / C8);
    if (item == 0 && lane == 0) {
        if (un.nth == 0) c.lens[slot] = (int)stop;
        if (!kept) {
            c.table[(int64_t)slot * c.max_pages + page_no] = dst;
            c.refs[dst] = 1;
            // the last two holders may both take a copy: the page is then listed as free by the next release
            if (lo > 0) atomicSub(&c.refs[src], 1);
        }
    }
    const int hk = item >> 1;
    const bool minor = item & 1;
    const int64_t ld = minor ? a.ld_v : a.ld_k;
    // the page's first event stands lo events before the call's first one
    const T* x = (const T*)(minor ? a.v : a.k) + (un.begin + page_no * PE - g.old_len) * ld + (int64_t)hk * D;

    // events outside [lo, hi) stand in as the nearest one inside
    Raw<T> raw[ROUNDS][4];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
        if (r * EV < hi && (r + 1) * EV > lo)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int ev = min(max(r * EV + 4 * quad + j, lo), hi - 1);
                raw[r][j] = load_raw<WIDE>(x + (int64_t)ev * ld + ch * 8);
            }
    const int64_t dst_h = (int64_t)dst * c.n_kv_heads + hk, src_h = (int64_t)src * c.n_kv_heads + hk;
    uint8_t* codes = (minor ? c.v : c.k) + dst_h * (PE * D);
    const uint8_t* held = (minor ? c.v : c.k) + src_h * (PE * D);
    float* scales = minor ? c.v_scale : c.k_scale;
    const float was = lo > 0 ? scales[src_h] : 0.f;

    bool in[ROUNDS * 4];
#pragma unroll
    for (int r = 0; r < ROUNDS * 4; ++r) in[r] = r / 4 * EV < hi && (r / 4 + 1) * EV > lo;
    const float top = wave_magnitude<T, ROUNDS * 4>(&raw[0][0], in);
    float s = page_scale(top);
    s = was > s ? was : s;
    const bool rewrite = lo > 0 && (g.copy || s > was);
    // a power of two: exact.  From 2^19 on every code becomes 0, and fp32 does not hold all quotients.
    const float grown = rewrite ? fminf(s / was, 0x1p20f) : 1.f;
    const int from = rewrite ? 0 : lo;
    const bool largest = !__is_same(T, f16) && __builtin_amdgcn_readfirstlane((int)(s == kLargestScale));

#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (r * EV >= hi || (r + 1) * EV <= from) continue;
        if (!minor) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int ev = r * EV + 4 * quad + j;
                if (ev < from || ev >= hi) continue;
                uint2 w;
                if (ev >= lo) {
                    const T* f = raw[r][j].x;
                    w.x = code4(f[0], f[1], f[2], f[3], s);
                    w.y = code4(f[4], f[5], f[6], f[7], s);
                    if (__builtin_expect(largest, 0)) w = make_uint2(keep_finite(w.x), keep_finite(w.y));
                } else {
                    const uint2 o = *(const uint2*)(held + ev * D + ch * 8);
                    w = make_uint2(rescale4(o.x, grown), rescale4(o.y, grown));
                }
                *(uint2*)(codes + ev * D + ch * 8) = w;
            }
        } else {
            unsigned w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = code4(raw[r][0].x[i], raw[r][1].x[i], raw[r][2].x[i], raw[r][3].x[i], s);
            if (__builtin_expect(largest, 0)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = keep_finite(w[i]);
            }
            const int e0 = r * EV + 16 * ((lane & 15) / C8);             // the lane's 16 events after the exchange
            exchange4(w);
            exchange4(w + 4);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (e0 >= hi || e0 + 16 <= from) continue;
                const int at = (ch * 8 + 4 * k + (lane >> 4)) * PE + e0;
                if (lo > e0 || hi < e0 + 16) {
                    const uint4 o = *(const uint4*)(held + at), d = *(const uint4*)(codes + at);
                    const unsigned old[4] = {o.x, o.y, o.z, o.w}, stale[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const unsigned below = bytes_below(lo - e0, y), in = bytes_below(hi - e0, y);
                        w[4 * k + y] = ((rewrite ? rescale4(old[y], grown) : old[y]) & below) | (w[4 * k + y] & in & ~below) |
                                       (stale[y] & ~in);
                    }
                }
                *(uint4*)(codes + at) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
        }
    }
    if (lane == 0 && (!kept || s != was)) scales[dst_h] = s;
}

// ---- sharing and releasing -----------------------------------------------------

__device__ __forceinline__ void drop_page(const dlrm_history_cache_t& c, int p) {
    if (p >= 0 && p < c.n_pages) atomicSub(&c.refs[p], 1);      // its result is not waited for
}

// LANES threads per history.  The list is written by a kernel of its own: a last
// block that wrote it here would need every block to write its caches back first,
// which took 10 to 40 us more than the second launch.  Only where one block can
// do the whole call does it write the list, too.
enum Release { kFork, kTruncate, kTrim };
struct ReleaseArgs {
    dlrm_history_cache_t c;
    const int32_t *slots, *other;       // fork: sources, destinations; truncate: slots, new lengths
    int64_t window, sinks;
    int n;
};

template <Release OP, int LANES>
__device__ __forceinline__ void release_history(const ReleaseArgs& a, int i, int tid) {
    const dlrm_history_cache_t& c = a.c;
    const int sh = 31 - __builtin_clz(c.page_events);
    const int slot = a.slots[i];
    bool ok = slot >= 0 && slot < c.n_slots;
    if constexpr (OP == kFork) {
        const int to = a.other[i];
        ok = ok && to >= 0 && to < c.n_slots;
        if (ok && slot != to) {
            const int64_t f = (int64_t)slot * c.max_pages, t = (int64_t)to * c.max_pages;
            const int len = c.lens[slot];
            for (int x = tid; x < c.max_pages; x += LANES) {
                const int p = c.table[f + x], o = c.table[t + x];
                if (p == o) continue;
                c.table[t + x] = p;
                if (p >= 0 && p < c.n_pages) atomicAdd(&c.refs[p], 1);
                drop_page(c, o);
            }
            if (tid == 0) c.lens[to] = len;
        }
    } else {
        const int len = ok ? c.lens[slot] : 0;
        const int64_t row = (int64_t)slot * c.max_pages;
        int lo, hi = c.max_pages;
        if constexpr (OP == kTruncate) {
            const int want = a.other ? a.other[i] : 0, mask = c.page_events - 1;
            ok = ok && want >= 0 && want <= len && want <= c.max_pages << sh;
            // the page that would be filled further may have been trimmed away
            if (ok && (want & mask)) ok = c.table[row + (want >> sh)] >= 0;
            lo = ok ? (want + mask) >> sh : hi;
            if constexpr (LANES > 64) __syncthreads();      // every thread has read the length
            if (ok && tid == 0) c.lens[slot] = want;
        } else {
            // pages whose events all lie behind the sinks and before the window
            lo = a.sinks < (int64_t)c.max_pages << sh ? (int)((a.sinks + c.page_events - 1) >> sh) : hi;
            const int64_t end = len > a.window ? (len - a.window) >> sh : 0;
            hi = ok && end < hi ? (int)end : (ok ? hi : 0);
        }
        for (int x = lo + tid; x < hi; x += LANES) {
            const int p = c.table[row + x];
            if (p == -1) continue;
            c.table[row + x] = -1;
            drop_page(c, p);
        }
    }
    if (!ok && tid == 0) atomicAdd(&c.counters[1], 1);
}

template <Release OP>
__global__ __launch_bounds__(256) void history_release_kernel(ReleaseArgs a) {
    release_history<OP, 256>(a, blockIdx.x, threadIdx.x);
}

// The free pages of a wave's share of a block, at most 64 words of 64 pages: lane
// k keeps word k, and the free pages of the words above it.
struct FreeWords {
    unsigned long long word;
    int above, n;           // free pages in the words above mine, in all
    int p0, words;          // the share's first page, its words
    __device__ __forceinline__ unsigned long long of(int k) const {
        const unsigned lo = __builtin_amdgcn_readlane((unsigned)word, k);
        const unsigned hi = __builtin_amdgcn_readlane((unsigned)(word >> 32), k);
        return (unsigned long long)hi << 32 | lo;
    }
    __device__ __forceinline__ int above_of(int k) const { return __builtin_amdgcn_readlane(above, k); }
};

__device__ __forceinline__ FreeWords mark_free(const dlrm_history_cache_t& c, int base, int words) {
    constexpr int AT_ONCE = 16;
    FreeWords f;
    const int lane = threadIdx.x & 63;
    f.p0 = base + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) * words * 64;
    f.words = words;
    f.word = 0;
    for (int k0 = 0; k0 < words; k0 += AT_ONCE) {
        int r[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
            r[i] = c.refs[min(f.p0 + (k0 + i) * 64 + lane, c.n_pages - 1)];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            const unsigned long long m =
                __ballot(r[i] == 0 && k0 + i < words && f.p0 + (k0 + i) * 64 + lane < c.n_pages);
            f.word = lane == k0 + i ? m : f.word;
        }
    }
    const int mine = __popcll(f.word);
    int sum = mine;                     // of the words from mine up
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_down(sum, d, 64);
        if (lane + d < 64) sum += o;
    }
    f.above = sum - mine;
    f.n = __builtin_amdgcn_readlane(sum, 0);
    return f;
}

// Sums of one number per wave: over the waves after mine, and over all.
template <int WAVES>
__device__ __forceinline__ int after_mine(int n, int* total) {
    __shared__ int part[WAVES];
    __syncthreads();  // part may still be read from a call before
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = n;
    __syncthreads();
    int after = 0, all = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        after += i > (int)(threadIdx.x >> 6) ? part[i] : 0;
        all += part[i];
    }
    *total = all;
    return after;
}

// Free page p goes to the place that counts the free pages above it.
template <int WAVES>
__device__ __forceinline__ void list_free(const dlrm_history_cache_t& c, int base, int words, int above) {
    const FreeWords f = mark_free(c, base, words);
    int total;
    const int at = above + after_mine<WAVES>(f.n, &total), lane = threadIdx.x & 63;
    for (int k = 0; k < words; ++k) {
        const unsigned long long m = f.of(k);
        if (m >> lane & 1) c.free_pages[at + f.above_of(k) + __popcll(m >> lane >> 1)] = f.p0 + k * 64 + lane;
    }
    if (base == 0 && threadIdx.x == 0) c.counters[0] = above + total;
}

constexpr int kChunkWords = kRebuildChunk / 256;         // of each of four waves
// Words of each of sixteen waves; a pool that one block lists has at most 64.
__device__ __forceinline__ int one_words(int n_pages) { return (n_pages + 1023) / 1024; }

__global__ __launch_bounds__(1024) void history_rebuild_one_kernel(dlrm_history_cache_t c) {
    list_free<16>(c, 0, one_words(c.n_pages), 0);
}

// Free pages of each chunk.
__global__ __launch_bounds__(256) void history_count_kernel(dlrm_history_cache_t c, int32_t* counts) {
    const FreeWords f = mark_free(c, blockIdx.x * kRebuildChunk, kChunkWords);
    int total;
    after_mine<4>(f.n, &total);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

__global__ __launch_bounds__(256) void history_rebuild_kernel(dlrm_history_cache_t c, const int32_t* counts) {
    int n = 0;
    for (int i = blockIdx.x + 1 + threadIdx.x; i < (int)gridDim.x; i += 256) n += counts[i];
    int above;
    block_exclusive<256>(n, &above);
    list_free<4>(c, blockIdx.x * kRebuildChunk, kChunkWords, above);
}

// A wave per history, sixteen at a time, then the list: one launch for a call of a
// few histories of a small pool.  Of 8192 pages, 32 histories: 7.4 us, in launches of
// its own 8.4; 128 histories 9.8 against 7.5.
template <Release OP>
__global__ __launch_bounds__(1024) void history_release_one_kernel(ReleaseArgs a) {
    for (int i = threadIdx.x >> 6; i < a.n; i += 16) release_history<OP, 64>(a, i, threadIdx.x & 63);
    __threadfence_block();      // the holders' counts are changed in the block's own L2 and not cached nearer
    __syncthreads();
    list_free<16>(a.c, 0, one_words(a.c.n_pages), 0);
}

template <Release OP>
static hipError_t release(const ReleaseArgs& a, int32_t* counts, hipStream_t s) {
    if (a.n <= 32 && a.c.max_pages <= 256 && a.c.n_pages <= 8192) {
        hipLaunchKernelGGL(history_release_one_kernel<OP>, dim3(1), dim3(1024), 0, s, a);
        return hipGetLastError();
    }
    if (!grid_fits(a.n, 256)) return kTooLarge;
    hipLaunchKernelGGL(history_release_kernel<OP>, dim3(a.n), dim3(256), 0, s, a);
    if (a.c.n_pages <= kOneBlockPages) {
        hipLaunchKernelGGL(history_rebuild_one_kernel, dim3(1), dim3(1024), 0, s, a.c);
    } else {
        const int n = rebuild_chunks(a.c.n_pages);
        hipLaunchKernelGGL(history_count_kernel, dim3(n), dim3(256), 0, s, a.c, counts);
        hipLaunchKernelGGL(history_rebuild_kernel, dim3(n), dim3(256), 0, s, a.c, counts);
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

// Enters the marked pages into the lists: `before` free pages lie before the
// wave's first one, `holes` below m.
__device__ __forceinline__ void list_moves(const dlrm_history_cache_t& c, const MoveWs& w, const FreeWords& f,
                                           int before, int m, int holes) {
    const int lane = threadIdx.x & 63;
    for (int k = 0; k < f.words; ++k) {
        const unsigned long long b = f.of(k);
        const int p = f.p0 + k * 64 + lane;
        const int fb = before + f.n - f.above_of(k) - __popcll(b >> lane);      // free pages before p
        // used pages before p and at or above m: (p - fb) - (m - holes)
        if (b >> lane & 1) {
            if (p < m) w.to[fb] = p;
        } else if (p >= m && p < c.n_pages) {
            w.from[p - fb - (m - holes)] = p;
        }
    }
}

// The new place and the holders of a page that moves.
__device__ __forceinline__ void pair_move(const dlrm_history_cache_t& c, const MoveWs& w, int i) {
    const int from = w.from[i], to = w.to[i];
    w.place[from] = to;
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
}

__global__ __launch_bounds__(1024) void history_plan_one_kernel(dlrm_history_cache_t c, MoveWs w) {
    const FreeWords f = mark_free(c, 0, one_words(c.n_pages));
    int total, holes;
    const int after = after_mine<16>(f.n, &total);
    const int m = c.n_pages - total;
    const int k = m - (f.p0 + (int)(threadIdx.x & 63) * 64);     // of the lane's word: pages below m
    const int below = __popcll(f.word & (k >= 64 ? ~0ull : (k <= 0 ? 0ull : (1ull << k) - 1)));
    block_exclusive<1024>(below, &holes);
    list_moves(c, w, f, total - after - f.n, m, holes);
    __threadfence_block();      // the lists are read by other threads of the block
    __syncthreads();
    for (int i = threadIdx.x; i < holes; i += 1024) pair_move(c, w, i);
    if (threadIdx.x == 0) {
        *w.n = holes;
        c.counters[0] = total;
    }
}

__global__ __launch_bounds__(256) void history_plan_kernel(dlrm_history_cache_t c, MoveWs w, int chunks) {
    // free pages in all, before this chunk, and below page m
    int n = 0, nb = 0, total, before, sum;
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
    const FreeWords f = mark_free(c, blockIdx.x * kRebuildChunk, kChunkWords);
    const int after = after_mine<4>(f.n, &sum);
    list_moves(c, w, f, before + sum - after - f.n, m, holes);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *w.n = holes;
        c.counters[0] = total;
    }
}

__global__ __launch_bounds__(256) void history_pair_kernel(dlrm_history_cache_t c, MoveWs w) {
    const int n = *w.n;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        pair_move(c, w, (int)i);
}

// Moves the pages and gives them their new numbers in the table and the list.
__global__ __launch_bounds__(256) void history_move_kernel(dlrm_history_cache_t c, MoveWs w) {
    const int n = *w.n;
    const int64_t vecs = (int64_t)c.n_kv_heads * c.page_events * c.head_dim / 16;
    for (int r = blockIdx.x; r < n; r += gridDim.x) {
        const int from = w.from[r], to = w.to[r];
        const uint4 *k0 = (const uint4*)c.k + from * vecs, *v0 = (const uint4*)c.v + from * vecs;
        uint4 *k1 = (uint4*)c.k + to * vecs, *v1 = (uint4*)c.v + to * vecs;
        for (int64_t i = threadIdx.x; i < vecs; i += 256) {
            const uint4 k = k0[i], v = v0[i];
            k1[i] = k;
            v1[i] = v;
        }
        for (int h = threadIdx.x; h < c.n_kv_heads; h += 256) {
            c.k_scale[(int64_t)to * c.n_kv_heads + h] = c.k_scale[(int64_t)from * c.n_kv_heads + h];
            c.v_scale[(int64_t)to * c.n_kv_heads + h] = c.v_scale[(int64_t)from * c.n_kv_heads + h];
        }
    }
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

template <typename T, int D, int PE>
static void launch_append(const AppendArgs& a, bool wide, dim3 grid, hipStream_t s) {
    if (wide) hipLaunchKernelGGL((history_append_kernel<T, D, PE, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((history_append_kernel<T, D, PE, false>), grid, dim3(256), 0, s, a);
}
template <typename T, int D>
static void launch_append(const AppendArgs& a, bool wide, dim3 grid, hipStream_t s) {
    if (a.c.page_events == 16) launch_append<T, D, 16>(a, wide, grid, s);
    else if (a.c.page_events == 32) launch_append<T, D, 32>(a, wide, grid, s);
    else launch_append<T, D, 64>(a, wide, grid, s);
}
template <typename T>
static void launch_append(const AppendArgs& a, dim3 grid, hipStream_t s) {
    const int step = 16 / sizeof(T);
    const bool wide = a.ld_k % step == 0 && a.ld_v % step == 0 && (((uintptr_t)a.k | (uintptr_t)a.v) & 15u) == 0;
    if (a.c.head_dim == 32) launch_append<T, 32>(a, wide, grid, s);
    else if (a.c.head_dim == 64) launch_append<T, 64>(a, wide, grid, s);
    else launch_append<T, 128>(a, wide, grid, s);
}

hipError_t launch_history_append(const AppendArgs& args, int dtype, hipStream_t s) {
    AppendArgs a = args;
    const int64_t by_page = a.n_events / a.c.page_events + 2 * (int64_t)a.batch;
    a.per_event = a.n_events <= by_page;
    const int64_t units = a.per_event ? a.n_events : by_page;
    if (!grid_fits(units + 1, 256)) return kTooLarge;
    hipLaunchKernelGGL(history_need_kernel, dim3((a.batch + kNeedBlock - 1) / kNeedBlock), dim3(kNeedBlock), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(units + 1), (unsigned)((2 * a.c.n_kv_heads + 3) / 4));
    if (dtype == DLRM_DTYPE_F32) launch_append<float>(a, grid, s);
    else if (dtype == DLRM_DTYPE_BF16) launch_append<bf16>(a, grid, s);
    else launch_append<f16>(a, grid, s);
    return hipGetLastError();
}

hipError_t launch_history_fork(const dlrm_history_cache_t& c, int n, const int32_t* src, const int32_t* dst,
                               int32_t* counts, hipStream_t s) {
    return release<kFork>(ReleaseArgs{c, src, dst, 0, 0, n}, counts, s);
}

hipError_t launch_history_truncate(const dlrm_history_cache_t& c, int n, const int32_t* slots,
                                   const int32_t* new_lens, int32_t* counts, hipStream_t s) {
    return release<kTruncate>(ReleaseArgs{c, slots, new_lens, 0, 0, n}, counts, s);
}

hipError_t launch_history_trim(const dlrm_history_cache_t& c, int n, const int32_t* slots, int64_t window,
                               int64_t sinks, int32_t* counts, hipStream_t s) {
    return release<kTrim>(ReleaseArgs{c, slots, nullptr, window, sinks, n}, counts, s);
}

hipError_t launch_history_compact(const dlrm_history_cache_t& c, int32_t* ws, hipStream_t s) {
    const MoveWs w = move_ws(c, ws);
    if (c.n_pages <= kOneBlockPages) {
        hipLaunchKernelGGL(history_plan_one_kernel, dim3(1), dim3(1024), 0, s, c, w);
    } else {
        const int chunks = rebuild_chunks(c.n_pages);
        hipLaunchKernelGGL(history_count_kernel, dim3(chunks), dim3(256), 0, s, c, w.counts);
        hipLaunchKernelGGL(history_plan_kernel, dim3(chunks), dim3(256), 0, s, c, w, chunks);
        hipLaunchKernelGGL(history_pair_kernel, dim3(grid_for(c.n_pages, 1024)), dim3(256), 0, s, c, w);
    }
    const int64_t cells = (int64_t)c.n_slots * c.max_pages + c.n_pages;
    const unsigned movers = (unsigned)(c.n_pages < 2048 ? c.n_pages : 2048), rows = grid_for(cells, 2048);
    hipLaunchKernelGGL(history_move_kernel, dim3(movers > rows ? movers : rows), dim3(256), 0, s, c, w);
    return hipGetLastError();
}

}  // namespace dlrm
