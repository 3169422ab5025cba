// history.h -- launch functions and device helpers of the event-history
// operators: windowed attention over ragged histories, the 8-bit paged cache
// and the management of its pages.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dlrm_mi355x.h"
#include "dlrm_device.h"

namespace dlrm {

constexpr int kScaleFloor = -100;    // smallest exponent of a page's power-of-two scale
constexpr int kRebuildChunk = 4096;  // pages per block of the free-list work on large pools

typedef __bf16 bf16;
typedef _Float16 f16;

// Arguments of the attention over ragged histories.
struct EncodeArgs {
    const void *q, *k, *v, *offsets;
    const uint8_t* padding;
    void* out;
    int64_t ld_q, ld_k, ld_v, ld_out, n_events, window, sinks;
    int batch, n_heads, n_kv, idx32;
    float scale;
};

// Arguments of the attention over the cache.
struct LookupArgs {
    dlrm_history_cache_t c;
    const int32_t* slots;
    const void* q;
    void* out;
    float* partial;
    int64_t ld_q, ld_out, window, sinks;
    int batch, queries, n_heads, wide;      // wide: rows of q and out are 16-byte aligned
    float scale;
};

// What one history of an append needs: its events before (-1: refused), the
// page that holds its last part (-1: none), whether that page is copied because
// other histories hold it too, and how many pages it takes from the list.
struct Need {
    int old_len, src, copy, pages;
};
constexpr int kNeedBlock = 256;      // histories whose needs are summed together

// The needs of all histories, the sums of their pages for each kNeedBlock of them
// and the refusals among them, and the length of the free list before the call.
struct NeedWs {
    Need* need;
    int2* sums;
    int* n_free;
};
inline size_t need_bytes(int64_t batch) {
    return (size_t)batch * sizeof(Need) + ((size_t)batch / kNeedBlock + 1) * sizeof(int2) + 16;
}

struct AppendArgs {
    dlrm_history_cache_t c;
    const int32_t* slots;
    const void *k, *v, *offsets;
    NeedWs ws;
    int64_t ld_k, ld_v, n_events;
    int batch, idx32, per_event;        // per_event: one unit of work per event (see the kernel), not per page
};

// Arguments of the selection of continuations.  ld_allowed 0: one row of bytes for all.
constexpr int kMostBeams = 128, kMostKept = 128, kMostGroup = 128;
constexpr int kItemBits = 25;           // of an item's number among a candidate's bits
constexpr int64_t kMostItems = (int64_t)1 << kItemBits;
struct SelectArgs {
    const void* logits;
    const float* scores;
    const uint8_t *allowed, *ended;
    float* out_scores;
    int32_t *out_parents, *out_items;
    int64_t ld_logits, ld_allowed;
    int batch, beams, items, keep, end_item, segs;
};

// Arguments of the lookup of groups of histories: those of the lookup, and the groups.
struct SharedArgs {
    LookupArgs l;
    const void* groups;                     // offsets, or NULL: batch / n_groups rows each
    int n_groups, idx32;
};

// HIP counts the threads along a dimension of a grid in 32 bits.  Launch functions
// return kTooLarge, having enqueued nothing, where a call would need more.
constexpr hipError_t kTooLarge = hipErrorInvalidConfiguration;
inline bool grid_fits(int64_t blocks, int threads) { return (uint64_t)blocks * threads <= 0xffffffffull; }

hipError_t launch_history_attention(const EncodeArgs& a, int dtype, int dim, hipStream_t s);
hipError_t launch_history_lookup(const LookupArgs& a, int dtype, hipStream_t s);
size_t lookup_workspace_bytes(const dlrm_history_cache_t& c, int64_t batch, int queries, int n_heads);
hipError_t launch_history_lookup_shared(const SharedArgs& a, int dtype, void* workspace, hipStream_t s);
size_t shared_workspace_bytes(const dlrm_history_cache_t& c, int64_t batch, int64_t n_groups, int queries, int n_heads);
hipError_t launch_history_select(const SelectArgs& a, int dtype, void* workspace, hipStream_t s);
size_t select_workspace_bytes(int64_t batch, int beams, int64_t items, int keep);

hipError_t launch_history_init(const dlrm_history_cache_t& c, hipStream_t s);
hipError_t launch_history_append(const AppendArgs& a, int dtype, hipStream_t s);
hipError_t launch_history_fork(const dlrm_history_cache_t& c, int n, const int32_t* src, const int32_t* dst,
                               int32_t* counts, hipStream_t s);
hipError_t launch_history_reorder(const dlrm_history_cache_t& c, int n_groups, int group, const int32_t* slots,
                                  const int32_t* parents, int32_t* counts, hipStream_t s);
hipError_t launch_history_truncate(const dlrm_history_cache_t& c, int n, const int32_t* slots,
                                   const int32_t* new_lens, int32_t* counts, hipStream_t s);
hipError_t launch_history_trim(const dlrm_history_cache_t& c, int n, const int32_t* slots, int64_t window,
                               int64_t sinks, int32_t* counts, hipStream_t s);
hipError_t launch_history_compact(const dlrm_history_cache_t& c, int32_t* ws, hipStream_t s);
inline int rebuild_chunks(int n_pages) { return (n_pages + kRebuildChunk - 1) / kRebuildChunk; }

// Bounds of history b in the packed events, kept inside [0, n] whatever the
// offsets hold.
__device__ __forceinline__ int64_t history_begin(const void* off, int idx32, int64_t b, int64_t n) {
    const int64_t o = ld_index(off, b, idx32);
    return o < 0 ? 0 : (o > n ? n : o);
}
__device__ __forceinline__ int64_t history_end(const void* off, int idx32, int64_t b, int64_t batch, int64_t begin,
                                               int64_t n) {
    const int64_t o = b + 1 < batch ? ld_index(off, b + 1, idx32) : n;
    return o < begin ? begin : (o > n ? n : o);
}

// The history that owns unit u when history b's units begin at
// floor(off[b] / width) + extra * b.  That start grows by at least
// floor(len / width) + extra from one history to the next, so no count of units
// has to be summed over the batch: with extra = 1 there is room for
// ceil(len / width) units, with extra = 2 for the pages an append of len events
// can touch.  Returns the history and u's number within it.
// Called by whole waves: each step reads 64 offsets at once and narrows the
// batch 64-fold, so that 4096 histories take two round trips; the last one
// holds the bounds of the history, too.
struct Unit {
    int b;                  // history
    int64_t nth;            // number of the unit within it; below 0: no one's
    int64_t begin, end;     // the history's rows
};
// A value of one lane, the same for the wave: what follows from it stays in scalar registers.
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
    const unsigned lo = __builtin_amdgcn_readlane((unsigned)v, lane);
    const unsigned hi = __builtin_amdgcn_readlane((unsigned)((uint64_t)v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ Unit history_of_unit(const void* off, int idx32, int batch, int64_t n, int width,
                                                int extra, int64_t u) {
    const int lane = threadIdx.x & 63, sh = 31 - __builtin_clz(width);      // a power of two
    int lo = 0, left = batch;
    Unit r;
    while (true) {
        const int step = (left + 63) / 64, at = lo + lane * step;
        const bool in = lane * step < left;
        const int64_t o = history_begin(off, idx32, in ? at : lo, n);
        const int64_t s = (o >> sh) + (int64_t)extra * at;
        const int k = __popcll(__ballot(in && s <= u));                       // lanes 0 .. k - 1
        const int last = __builtin_amdgcn_readfirstlane(k ? k - 1 : 0);
        lo += last * step;
        if (step == 1) {
            r.b = lo;
            r.nth = u - lane_value(s, last);
            r.begin = lane_value(o, last);
            const int64_t next = lane_value(o, last < 63 ? last + 1 : 63);
            r.end = last < 63 && last + 1 < left ? (next < r.begin ? r.begin : next)
                                                 : lane_value(history_end(off, idx32, lo, batch, r.begin, n), 0);
            return r;
        }
        const int rest = left - last * step;
        left = rest < step ? rest : step;
    }
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
    return v;
}

// c of exp(scale s) = 2^(c s), a negative scale having turned the query's sign.  Never
// 0, which would make NaN of an unseen key's -inf: the smallest fp32 number leaves
// every finite score's weight at 1.  Never infinite, which would make NaN of a 0.
__device__ __forceinline__ float exponent_scale(float scale) {
    return fminf(fmaxf(fabsf(scale) * 1.44269504088896341f, 0x1p-149f), 0x1.fffffep+127f);
}

// Eight consecutive elements of a row, as they are in memory.
template <typename T>
struct Raw {
    T x[8];
};
template <bool WIDE, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
    Raw<T> r;
    if constexpr (WIDE) {
        typedef T v __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
        for (int c = 0; c < (int)sizeof(T) / 2; ++c) {
            const v t = *(const v*)(p + c * (16 / sizeof(T)));
#pragma unroll
            for (int i = 0; i < 16 / (int)sizeof(T); ++i) r.x[c * (16 / sizeof(T)) + i] = t[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.x[i] = p[i];
    }
    return r;
}
// Four consecutive elements, at once where their row is aligned.
template <typename T>
__device__ __forceinline__ void store4(T* p, floatx4 v, int wide) {
    if (wide) {
        typedef T t4 __attribute__((ext_vector_type(4)));
        *(t4*)p = t4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = (T)v[i];
    }
}

// The largest magnitude among elements as bits, without their sign (16-bit
// types: of the even and of the odd elements).  Infinities and NaN come out above
// every finite value.
template <typename T>
__device__ __forceinline__ void top_magnitude(const Raw<T>& r, unsigned& top) {
    if constexpr (sizeof(T) == 2) {
        typedef unsigned short us2 __attribute__((ext_vector_type(2)));
        typedef unsigned u4 __attribute__((ext_vector_type(4)));
        const u4 w = __builtin_bit_cast(u4, r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(us2, top),
                                                                         __builtin_bit_cast(us2, w[i] & 0x7fff7fffu)));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned w = __builtin_bit_cast(unsigned, r.x[i]) & 0x7fffffffu;
            top = top > w ? top : w;
        }
    }
}
template <typename T>
__device__ __forceinline__ bool odd_magnitude(unsigned top) {
    if constexpr (sizeof(T) == 4) return top >= 0x7f800000u;
    const unsigned all = __is_same(T, f16) ? 0x7c00u : 0x7f80u;
    return (top & 0xffffu) >= all || top >> 16 >= all;
}
// The smallest power of two s >= 2^kScaleFloor with amax / s <= 448 (the
// largest e4m3 value, 0.875 x 2^9).  Read off the bits, so exact: amax =
// m 2^x with m in [1, 2) gives 2^(x - 8) for m <= 1.75 and 2^(x - 7) above.
__device__ __forceinline__ float page_scale(float amax) {
    const unsigned bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < kScaleFloor ? kScaleFloor : e;
    return __uint_as_float((unsigned)(e + 127) << 23);
}

}  // namespace dlrm
