// history_tile.h -- one 64-event tile of the 8-bit paged cache in one wave: what
// the lookups share.  The two products, their operands' layout and the parts that
// factors are split into are described in history_lookup.hip.
#pragma once

#include "history.h"

namespace dlrm {

constexpr int kTile = 64;                // events per tile

// The visible tiles of a history: `lead` tiles from its start, then the tiles
// from `first` on, `count` in all.
struct Span {
    int len, low, lead_events, first, lead, count;
};

__device__ __forceinline__ Span span_of(const LookupArgs& a, int b) {
    Span s;
    const int slot = a.slots ? a.slots[b] : b;
    const bool held = slot >= 0 && slot < a.c.n_slots;
    const int most = a.c.max_pages * a.c.page_events;
    int len = held ? a.c.lens[slot] : 0;
    len = len < 0 ? 0 : (len > most ? most : len);
    int low = len > a.window ? len - (int)a.window : 0;
    int lead = (int)(a.sinks < low ? a.sinks : low);
    if (lead == low) low = lead = 0;     // the sinks reach the window: everything is seen
    s.len = len;
    s.low = low;
    s.lead_events = lead;
    s.first = low / kTile;
    s.lead = (lead + kTile - 1) / kTile;
    s.lead = s.lead < s.first ? s.lead : s.first;
    s.count = len ? s.lead + (len + kTile - 1) / kTile - s.first : 0;
    return s;
}

// A history's visible tiles at most, as the host can tell.
inline int64_t most_tiles(const LookupArgs& a) {
    const int64_t span = ((int64_t)a.c.max_pages * a.c.page_events + kTile - 1) / kTile;
    if (a.window >= span * kTile || a.sinks >= span * kTile) return span;
    const int64_t seen = (a.window + kTile - 1) / kTile + 1 + (a.sinks + kTile - 1) / kTile;
    return seen < span ? seen : span;
}

// A slot that is none is counted, by one thread of the history's blocks.
__device__ __forceinline__ void count_refused(const LookupArgs& a, int b) {
    if (a.slots[b] < 0 || a.slots[b] >= a.c.n_slots) atomicAdd(&a.c.counters[1], 1);
}

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// fp32 values as sums of bf16 parts cut off at 8 bits each: the high halves of
// two words, packed.
__device__ __forceinline__ unsigned pack_hi(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

template <int N>
__device__ __forceinline__ void split8(const float* x, bf16x8* part) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_hi(r[2 * i], r[2 * i + 1]);
        part[n] = __builtin_bit_cast(bf16x8, w);
        if (n + 1 < N) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] -= cut(r[i]);
        }
    }
}

// Eight codes times their scale as bf16.
__device__ __forceinline__ bf16x8 decode8(unsigned lo, unsigned hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    const u32x4 w = {__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b),
                     __builtin_bit_cast(unsigned, c), __builtin_bit_cast(unsigned, d)};
    return __builtin_bit_cast(bf16x8, w);
}

template <typename T> struct Parts;
template <> struct Parts<bf16> { static constexpr int q = 1, p = 2; };
template <> struct Parts<f16> { static constexpr int q = 2, p = 2; };
template <> struct Parts<float> { static constexpr int q = 3, p = 3; };

// The codes of one tile as the products take them.
template <int D>
struct Tile {
    static constexpr int KL = D >= 64 ? D / 64 : 1;     // 16-byte loads of a key row per lane (D 32: 8 bytes)
    u32x4 k[4][KL];
    u32x4 v[D / 16];
    float ks, vs;
    bool kin, vin;                                      // the pages are there
};

// The lane's part of a query row, from element 0 of the head: elements l 64 + g 16 +
// 8 u + i (D 32: g 8 + i) for step 2 l + u.  A negative scale turns the query's sign.
template <int D, typename T>
__device__ __forceinline__ void load_query(const T* qp, float scale, int wide, int g,
                                           bf16x8 (&q)[D / 32][Parts<T>::q]) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        const int d0 = D == 32 ? g * 8 : (s >> 1) * 64 + g * 16 + (s & 1) * 8;
        const Raw<T> raw = wide ? load_raw<true>(qp + d0) : load_raw<false>(qp + d0);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = scale < 0.f ? -(float)raw.x[i] : (float)raw.x[i];
        split8<Parts<T>::q>(x, q[s]);
    }
}

// The tile whose first page is p0 of the history with this page list.
template <int D, int PE>
__device__ __forceinline__ void load_tile(const dlrm_history_cache_t& c, const int32_t* table, int p0, int hk, int n,
                                          int g, Tile<D>& t) {
    constexpr int PT = kTile / PE;                      // pages per tile
    int pk, pv;
    if constexpr (PT == 1) {
        pk = pv = table[p0];
    } else {
        const int ik = p0 + (n >> 2) * PT / 4, iv = p0 + g * PT / 4;
        pk = ik < c.max_pages ? table[ik] : -1;
        pv = iv < c.max_pages ? table[iv] : -1;
    }
    t.kin = pk >= 0 && pk < c.n_pages;
    t.vin = pv >= 0 && pv < c.n_pages;
    const int64_t hk_k = (int64_t)(t.kin ? pk : 0) * c.n_kv_heads + hk;
    const int64_t hk_v = (int64_t)(t.vin ? pv : 0) * c.n_kv_heads + hk;
    const uint8_t* kp = c.k + (hk_k * PE + (n >> 2) * 16 % PE + (n & 3)) * D + g * (D == 32 ? 8 : 16);
    const uint8_t* vp = c.v + (hk_v * D + n) * PE + g * 16 % PE;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int x = 0; x < Tile<D>::KL; ++x) {
            if constexpr (D == 32) {
                const u32x2 w = *(const u32x2*)(kp + e * 4 * D);
                t.k[e][x] = u32x4{w[0], w[1], 0u, 0u};
            } else {
                t.k[e][x] = *(const u32x4*)(kp + e * 4 * D + x * 64);
            }
        }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) t.v[j] = *(const u32x4*)(vp + j * 16 * PE);
    t.ks = c.k_scale[hk_k];
    t.vs = c.v_scale[hk_v];
}

// The tile's part of the rows' results: o the weighted sums, m the largest score (before the scale c), l the lane's
// share of the weights' sum.  Events below `len` that are not below `low`, or are below `lead`, are seen; `whole`, the
// same for the wave: all of the tile.  ROWS: low and lead are each row's own, and the
// values of events that some rows do not see are finite.
template <int D, typename T, bool ROWS = false>
__device__ __forceinline__ void use_tile(Tile<D>& t, const bf16x8 (&q)[D / 32][Parts<T>::q], float c, int e0, bool whole,
                                         int low, int lead, int len, int g, floatx4 (&o)[D / 16], float& m, float& l) {
    constexpr int NQ = Parts<T>::q, NP = Parts<T>::p;
    floatx4 s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        s[e] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < Tile<D>::KL; ++x)
#pragma unroll
            for (int u = 0; u < (D == 32 ? 1 : 2); ++u) {
                const bf16x8 kk = decode8(t.k[e][x][2 * u], t.k[e][x][2 * u + 1], t.ks);
#pragma unroll
                for (int y = 0; y < NQ; ++y)
                    s[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[2 * x + u][y], s[e], 0, 0, 0);
            }
    }
    // events of the tile's ends, and of pages that are not there, leave: score -inf, codes 0
    unsigned seen = 0xffffu;                             // of the lane group's 16 events
    if (!whole || __any(!t.vin)) {
        seen = 0;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            const int j = e0 + g * 16 + x;
            seen |= (t.vin && j < len && (j >= low || j < lead)) ? 1u << x : 0u;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x)
            if (!(seen >> x & 1)) s[x >> 2][x & 3] = -INFINITY;
        if constexpr (ROWS) seen = t.vin ? 0xffffu : 0u;
        u32x4 keep;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const unsigned f = seen >> (4 * x) & 15u;
            keep[x] = (f & 1 ? 0xffu : 0u) | (f & 2 ? 0xff00u : 0u) | (f & 4 ? 0xff0000u : 0u) |
                      (f & 8 ? 0xff000000u : 0u);
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) t.v[j] &= keep;
        t.vs = seen ? t.vs : 1.f;
    }
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < 16; ++x) top = fmaxf(top, s[x >> 2][x & 3]);
    top = fmaxf(top, swizzle_xor16(top));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float mx = fmaxf(m, top);
    if (__any(mx > m)) {
        const float alpha = mx == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mx) * c);
        l *= alpha;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[j] *= alpha;
        m = mx;
    }
    const float mc = m == -INFINITY ? 0.f : m * c;
    float p[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
        p[x] = __builtin_amdgcn_exp2f(fmaf(s[x >> 2][x & 3], c, -mc));
        l += p[x];
    }
    bf16x8 pp[2][NP];
    split8<NP>(p, pp[0]);
    split8<NP>(p + 8, pp[1]);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bf16x8 vv = decode8(t.v[j][2 * h], t.v[j][2 * h + 1], t.vs);
#pragma unroll
            for (int y = 0; y < NP; ++y)
                o[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, pp[h][y], o[j], 0, 0, 0);
        }
}

}  // namespace dlrm
