// history_select.hip -- the best continuations of a group of histories: beams x
// items by the sum of a beam's score and an item's log-probability.
//
//   s(w, v) = score_w + x(w, v) - log sum_u exp x(w, u)       over the allowed u
//
// The `keep` largest s of a group, in descending order; equal ones by beam, then
// by logit and item.  Within a beam the order is that of the logits, so that a row's best items
// are found without its sum, in the same pass over it.
//
// What bounds it, and what it reaches: ten fp64 instructions a logit for the sums.  64 groups of 8 beams, 100000 items, bf16,
// 48.5 us: the pass 44 (2.3 TB/s; vector instructions issue in 75% of the cycles), the join 9.  128 rows of 10^6 items, fp32,
// best 100: 122 us, the pass 106 (4.9 TB/s).  16 groups of 64 beams, 20011 items, fp16, best 64: 39 us, 27 and 14.  4 groups of
// 4 beams, 5000 items: 15 us in one launch, a chain of counts and of reads by other waves.
#include "history.h"

namespace dlrm {

typedef unsigned long long u64;

constexpr int kSelectHalf = 512;         // logits of half a tile in the 16-bit types, or of a whole one: eight a lane
constexpr int kSelectRoom = 512;         // candidates a wave has room for
constexpr int kGroups = 16;              // groups of tiles in a wave's part
constexpr int kSelectWaves = 4096;       // waves a launch aims at: sixteen on each CU
constexpr int kBlockWaves = 8;
// Groups of few logits, one part of a row for each wave of a block, and not more groups than CUs, take one launch.  4
// beams of 500 to 5000 items, fp32: 64 groups 12.3 to 16.3 us, in two launches 13.9 to 17.3; 512 groups 22.4 to 32.1
// against 21.2 to 28.9.  Blocks whose waves take several parts lose: 4 groups of 32000 logits 23.3, in two launches 17.5.
constexpr int kOneLogits = 20480, kOneGroups = 256;
constexpr int kMostSegs = 256;           // parts of a row, of all rows of a group
constexpr int kMostLists = 4096;
constexpr int kJoinRoom = 256;           // candidates a wave of the join has room for, and all of them together
constexpr int kPool = 512;

// What one wave leaves of its part of a row: the sum of exponentials against `ref`,
// the largest logit (NaN if one was among them), and how many candidates it lists.
struct __attribute__((aligned(32))) SelectSum {
    double sum;
    float ref, top;
    int n, unused[3];
};

struct SelectWs {
    SelectSum* sums;     // (rows, segs)
    u64* keys;           // (rows, segs, keep)
};

// Bits in the order of the values they stand for; -0 must have become 0.
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned b = __float_as_uint(x);
    return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ u64 ordered(double x) {
    const u64 b = (u64)__double_as_longlong(x);
    return b ^ ((u64)((long long)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered(u64 k) {
    return __longlong_as_double((long long)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// A candidate among all beams: its score, then beam, logit and item, so that equal
// scores have an order, too.
struct Best {
    u64 score, rest;
};
__device__ __forceinline__ bool above(const Best& a, const Best& b) {
    return a.score > b.score || (a.score == b.score && a.rest > b.rest);
}
__device__ __forceinline__ bool reaches(u64 a, u64 b) { return a >= b; }
__device__ __forceinline__ bool reaches(const Best& a, const Best& b) { return !above(b, a); }
__device__ __forceinline__ u64 wave_and(u64 v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v &= (u64)__shfl_xor((long long)v, d, 64);
    return v;
}
__device__ __forceinline__ u64 wave_or(u64 v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v |= (u64)__shfl_xor((long long)v, d, 64);
    return v;
}
__device__ __forceinline__ u64 first_word(u64 k) { return k; }
__device__ __forceinline__ u64 first_word(const Best& k) { return k.score; }

// Keeps the `keep` largest of the n > keep different keys in buf and returns the
// smallest of them.  The bits of the keep-th largest are found from the highest
// in which the keys differ down, until exactly `keep` keys reach what is known of it.
template <int ROOM>
__device__ __forceinline__ u64 kth(const u64 (&e)[ROOM], u64 all, u64 any, int keep) {
    const u64 differ = all ^ any;
    if (!differ) return all;
    u64 bit = 0x8000000000000000ull >> __builtin_clzll(differ);
    u64 t = all & ~(bit | (bit - 1));
    for (; bit; bit >>= 1) {
        int count = 0;
#pragma unroll
        for (int i = 0; i < ROOM; ++i) count += __popcll(__ballot(e[i] >= (t | bit)));
        if (count >= keep) t |= bit;
        if (count == keep) break;
    }
    return t;
}
template <int ROOM>
__device__ __forceinline__ Best kth(const Best (&e)[ROOM], u64 all, u64 any, int keep) {
    // the scores first; where several have the last one, the rest decides
    u64 s[ROOM];
#pragma unroll
    for (int i = 0; i < ROOM; ++i) s[i] = e[i].score;
    Best t = {kth(s, all, any, keep), 0};
    int reach = 0;
#pragma unroll
    for (int i = 0; i < ROOM; ++i) reach += __popcll(__ballot(s[i] >= t.score));
    if (reach == keep) return t;
    for (u64 bit = 0x8000000000000000ull; bit; bit >>= 1) {
        const Best c = {t.score, t.rest | bit};
        int count = 0;
#pragma unroll
        for (int i = 0; i < ROOM; ++i) count += __popcll(__ballot(reaches(e[i], c)));
        if (count >= keep) t = c;
        if (count == keep) break;
    }
    return t;
}
template <int ROOM, typename K>
__device__ __forceinline__ K keep_among(K* buf, int n, int keep) {
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    K e[ROOM / 64];
    u64 all = ~0ull, any = 0;
#pragma unroll
    for (int i = 0; i < ROOM / 64; ++i) {
        const bool in = i * 64 + lane < n;
        e[i] = in ? buf[i * 64 + lane] : K{};
        all &= in ? first_word(e[i]) : ~0ull;
        any |= first_word(e[i]);
    }
    const K t = kth(e, wave_and(all), wave_or(any), keep);
    int at = 0;
#pragma unroll
    for (int i = 0; i < ROOM / 64; ++i) {
        const u64 in = __ballot(i * 64 + lane < n && reaches(e[i], t));
        if (in >> lane & 1) buf[at + __popcll(in & ((1ull << lane) - 1))] = e[i];
        at += __popcll(in);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return t;
}

template <int ROOM, typename K>
__device__ __forceinline__ K keep_largest(K* buf, int n, int keep) {
    return n <= 128 ? keep_among<128>(buf, n, keep) : keep_among<ROOM>(buf, n, keep);
}

// The keep-th largest of two values per lane, 1 <= keep <= 128, or less than that by
// less than 2^-7 of it: the upper half of its bits, two at a time (each step waits some
// 200 cycles for its counts).  ORDERS of them at once, for different `keep`.
template <int ORDERS>
__device__ __forceinline__ void kth_of_lanes(float a, float b, const int (&keep)[ORDERS], float (&r)[ORDERS]) {
    const unsigned x = ordered(a + 0.f), y = ordered(b + 0.f);
    unsigned t[ORDERS] = {};
#pragma unroll
    for (int at = 30; at >= 16; at -= 2)
#pragma unroll
        for (int k = 0; k < ORDERS; ++k) {
            unsigned digit = 0;
#pragma unroll
            for (unsigned d = 1; d < 4; ++d) {
                const unsigned c = t[k] | d << at;
                digit += __popcll(__ballot(x >= c)) + __popcll(__ballot(y >= c)) >= keep[k] ? 1u : 0u;
            }
            t[k] |= digit << at;
        }
#pragma unroll
    for (int k = 0; k < ORDERS; ++k) r[k] = unordered(t[k] > 0x007fffffu ? t[k] : 0x007fffffu);   // below -inf: NaN
}

// Sums of exponentials are held as sum x 2^whole(ref).  ref is a multiple of 512, so
// that it is 0 in ordinary rows and a logit adds the same wherever it stands; logits
// beyond 2^20 (far) are taken less ref before the exponential, and sums stand against
// e^ref.
constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453;
constexpr double kShift = 0x1.8p52;      // adding and taking away: a whole number
__device__ __forceinline__ bool far(float ref) { return !(fabsf(ref) <= 0x1p20f); }
__device__ __forceinline__ double whole(float ref) { return rint((double)ref * kLog2e); }
// The logarithm of what a sum against `ref` is a multiple of, less ref.
__device__ __forceinline__ double beside(float ref) { return far(ref) ? 0. : fma(whole(ref), kLn2, -(double)ref); }

// e^x 2^-w with shift = kShift - w, to 2^-29 of its value, where the result has an
// exponent within double's.  x log2 e is split into a whole number and a rest of at most
// a half; a polynomial of the sixth degree, fitted to the least relative error
// (1.86e-9), gives 2 to the rest.
__device__ __forceinline__ double power(double x, double shift) {
    const double k = fma(x, kLog2e, shift), f = fma(x, kLog2e, shift - k);
    double p = 0x1.41d332c59dceep-13;
    p = fma(p, f, 0x1.5f456a892d64dp-10);
    p = fma(p, f, 0x1.3b2dbbc1f415fp-7);
    p = fma(p, f, 0x1.c6aed4b954ea2p-5);
    p = fma(p, f, 0x1.ebfbdadcaf500p-3);
    p = fma(p, f, 0x1.62e430c7e91f8p-1);
    p = fma(p, f, 0x1.0000000261502p+0);
    return __hiloint2double(__double2hiint(p) + (__double2loint(k) << 20), __double2loint(p));
}
// What a sum against `from` has to be multiplied by to stand against `to`.
__device__ __forceinline__ double moved(float from, float to) {
    if (far(from) || far(to)) return power(fmax((double)from - (double)to + (beside(from) - beside(to)), -690.), kShift);
    const double d = fmax(whole(from) - whole(to), -1000.);
    return __hiloint2double((1023 + (int)d) << 20, 0);
}

// Eight elements of a row at any alignment, and their bytes of a mask.
template <typename T>
struct Eight {
    typedef unsigned words __attribute__((ext_vector_type(sizeof(T) * 2), aligned(sizeof(T))));
    words w;
    uint2 may;
};
template <typename T, bool MASKED>
__device__ __forceinline__ Eight<T> load_eight(const T* x, const uint8_t* may, int at, int items) {
    typedef unsigned two __attribute__((ext_vector_type(2), aligned(1)));
    Eight<T> r;
    if (at + 8 <= items) {
        r.w = *(const typename Eight<T>::words*)(x + at);
        if constexpr (MASKED) {
            const two m = *(const two*)(may + at);
            r.may = make_uint2(m[0], m[1]);
        }
        return r;
    }
    T e[8];
    uint8_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        e[i] = at + i < items ? x[at + i] : (T)-INFINITY;
        m[i] = MASKED && at + i < items ? may[at + i] : 0;
    }
    r.w = __builtin_bit_cast(typename Eight<T>::words, e);
    r.may = __builtin_bit_cast(uint2, m);
    return r;
}
template <typename T, bool MASKED>
__device__ __forceinline__ void values_of(const Eight<T>& r, float* f) {
    struct Elements {
        T x[8];
    };
    const Elements e = __builtin_bit_cast(Elements, r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // bf16 by its bits: a conversion lets the compiler take maxima in bf16, rounding each again
        if constexpr (__is_same(T, bf16)) f[i] = __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
        else f[i] = (float)e.x[i];
        if constexpr (MASKED) f[i] = ((i < 4 ? r.may.x : r.may.y) >> (8 * (i & 3)) & 0xffu) ? f[i] : -INFINITY;
    }
}

// What the waves of a block leave for one another and for themselves.
struct SelectShared {
    u64 room[kBlockWaves][kSelectRoom];
    float tops[kBlockWaves][kGroups][64];  // later the numbers of those that reach the floor
    float found[kBlockWaves];
};

// One wave's part of a row, every wave of the block taking part.
//
// The sum is taken against `ref`, which needs only be near the largest logit: 64 bits
// hold e^300 times too much, so that no tile waits for a maximum over the wave, and
// rows of the same logits in another order have sums that differ by their additions'
// rounding alone (see the join).  Logits more than 690 below ref count as if they were
// 690 below, which is nothing against any sum that counts.
//
// Of the logits themselves the pass over them keeps the largest of each group that a
// lane sees.  Only logits that reach `floor` can be among the best: the keep-th largest
// of 128 of the part's groups, or the least of what the `sharing` waves of the row find
// so for the keep / sharing-th, whichever is larger.  The few groups that reach it are
// then read once more, from a cache.  Collecting candidates on the way took twice as
// long as the sums: nearly every tile has one while the floor still rises.
template <typename T, bool MASKED>
__device__ __forceinline__ void select_part(const SelectArgs& a, const SelectWs& ws, int64_t unit, SelectShared& s) {
    constexpr int HALVES = sizeof(T) == 2 ? 2 : 1, E = 8 * HALVES, TILE = kSelectHalf * HALVES;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t row = unit / a.segs;
    const int seg = (int)(unit - row * a.segs);
    const int sharing = a.segs < kBlockWaves ? a.segs : kBlockWaves, share = (a.keep + sharing - 1) / sharing;
    const bool mine = unit >= 0 && row < (int64_t)a.batch * a.beams;
    const int tiles = (a.items + TILE - 1) / TILE;
    const int t0 = (int)((int64_t)tiles * seg / a.segs);
    int t1 = (int)((int64_t)tiles * (seg + 1) / a.segs);
    const T* x = (const T*)a.logits + row * a.ld_logits;
    const uint8_t* may = MASKED ? a.allowed + row * a.ld_allowed : nullptr;
    Eight<T> next[HALVES];                  // on its way while the row's score is
    if (mine && t0 < t1)
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
            next[h] = load_eight<T, MASKED>(x, may, t0 * TILE + h * kSelectHalf + lane * 8, a.items);
    // of a row without continuations nothing else is read, here or by the join
    const bool live = mine && (!a.scores || fabsf(a.scores[row]) < INFINITY) && !(a.ended && a.ended[row]);
    if (!live) t1 = t0;
    const int group = (t1 - t0 + kGroups - 1) / kGroups;        // tiles

    float ref = -3.4028235e38f, low = -INFINITY, high = -INFINITY, most = -INFINITY;
    double sum[2] = {0., 0.}, least_x = -INFINITY, shift = kShift;
    bool is_far = true;
    int groups = 0, left = group;
    for (int t = t0; t < t1; ++t) {
        const int at = t * TILE + lane * 8;
        float f[E];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            values_of<T, MASKED>(next[h], f + 8 * h);
            if (t + 1 < t1) next[h] = load_eight<T, MASKED>(x, may, at + TILE + h * kSelectHalf, a.items);
        }
        float l = f[0], h = f[E / 2];        // a NaN stays one
#pragma unroll
        for (int i = 1; i < E / 2; ++i) {
            l = __builtin_elementwise_maximum(l, f[i]);
            h = __builtin_elementwise_maximum(h, f[E / 2 + i]);
        }
        low = __builtin_elementwise_maximum(low, l);
        high = __builtin_elementwise_maximum(high, h);
        const float top = __builtin_elementwise_maximum(l, h);
        most = __builtin_elementwise_maximum(most, top);
        if (--left == 0 || t + 1 == t1) {
            s.tops[wave][groups++][lane] = most;
            most = -INFINITY;
            left = group;
        }
        if (__builtin_expect(__any(top > ref + 300.f), 0)) {
            const float to = 512.f * rintf(wave_max(top) / 512.f);
            const double by = moved(ref, to);
            sum[0] *= by;
            sum[1] *= by;
            ref = to;
            is_far = far(ref);
            least_x = (double)ref - 690.;
            shift = kShift - whole(ref);
        }
        if (__builtin_expect(is_far, 0)) {
#pragma unroll
            for (int i = 0; i < E; ++i) sum[0] += power(fmax((double)f[i] - (double)ref, -690.), kShift);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) sum[i & 1] += power(fmax((double)f[i], least_x), shift);
        }
    }
    float kth[2];
    kth_of_lanes(low, high, {a.keep, share}, kth);
    float floor = kth[0];
    if (sharing > 1) {
        if (lane == 0) s.found[wave] = kth[1];
        __syncthreads();
        float every = INFINITY;
        for (int i = 0; i < sharing; ++i) every = fminf(every, s.found[wave / sharing * sharing + i]);
        floor = fmaxf(floor, every);
    }
    if (!live) return;

    // the groups that reach the floor, in order
    unsigned short* which = (unsigned short*)s.tops[wave];
    int reach = 0;
    for (int j = 0; j < groups; ++j) {
        const float top = s.tops[wave][j][lane];
        const bool in = top >= floor && top > -INFINITY;
        const u64 go = __ballot(in);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (in) which[reach + __popcll(go & ((1ull << lane) - 1))] = (unsigned short)(j * 64 + lane);
        reach += __popcll(go);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    u64* buf = s.room[wave];
    int n = 0;
    u64 least = 0;                 // candidates have to be larger
    for (int e = 0; e < reach; e += 64) {
        const int g = e + lane < reach ? (int)which[e + lane] : -1;
        for (int k = 0; k < group; ++k) {
            const int t = t0 + (g >> 6) * group + k;
            const int at = g >= 0 && t < t1 ? t * TILE + (g & 63) * 8 : a.items;
            Eight<T> raw[HALVES];
#pragma unroll
            for (int h = 0; h < HALVES; ++h) raw[h] = load_eight<T, MASKED>(x, may, at + h * kSelectHalf, a.items);
#pragma unroll 1
            for (int h = 0; h < HALVES; ++h) {
                float f[8];
                Eight<T> one = raw[0];
                if (HALVES == 2 && h) {
                    one.w = raw[HALVES - 1].w;
                    one.may = raw[HALVES - 1].may;
                }
                values_of<T, MASKED>(one, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const u64 key = (u64)ordered(f[i] + 0.f) << 32 | (0xffffffffu - (unsigned)(at + h * kSelectHalf + i));
                    const u64 in = __ballot(f[i] >= floor && f[i] > -INFINITY && key > least);
                    if (!in) continue;
                    if (n > kSelectRoom - 64) {
                        least = keep_largest<kSelectRoom>(buf, n, a.keep);
                        n = a.keep;
                    }
                    if (in >> lane & 1) buf[n + __popcll(in & ((1ull << lane) - 1))] = key;
                    n += __popcll(in);
                }
            }
        }
    }
    if (n > a.keep) {
        keep_largest<kSelectRoom>(buf, n, a.keep);
        n = a.keep;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    u64* keys = ws.keys + unit * a.keep;
    for (int i = lane; i < n; i += 64) keys[i] = buf[i];
    most = __builtin_elementwise_maximum(low, high);
    const bool bad = __any(most != most);
    most = wave_max(most);
    double all = sum[0] + sum[1];
#pragma unroll
    for (int d = 32; d; d >>= 1) all += __shfl_xor(all, d, 64);
    if (lane == 0) ws.sums[unit] = SelectSum{all, ref, bad ? NAN : most, n, {}};
}

// The largest fp32 value that is not above x.
__device__ __forceinline__ float round_down(double x) {
    const float f = (float)x;
    if (!((double)f > x)) return f;
    const unsigned k = ordered(f + 0.f) - 1;
    return unordered(k);
}

struct JoinShared {
    double score[kMostBeams], log_sum[kMostBeams];     // log_sum NaN: the beam gives no candidates
    Best room[kBlockWaves][kJoinRoom], pool[kPool];
    double part_sum[kMostLists / 8 + kMostBeams];
    float part_ref[kMostLists / 8 + kMostBeams], part_top[kMostLists / 8 + kMostBeams];
    float best[kMostLists];                 // the best score of a list, rounded down
    unsigned char held[kMostLists];         // its candidates
    unsigned short list[kMostLists];        // the lists that may hold one of the best
    int place[kPool];
    int lists, count[kBlockWaves], joined;  // joined: not one of count, which slower waves may yet read
    float found[kBlockWaves];
};

// Joins the parts of a group's rows, by a block.  No list whose largest logit gives
// less than the keep-th largest of the lists' is read, and no candidate taken further
// that is below what the waves find together.
__device__ __forceinline__ void join_group(const SelectArgs& a, const SelectWs& ws, int group, JoinShared& s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row0 = (int64_t)group * a.beams;
    const int lists = a.beams * a.segs;
    const SelectSum* sums = ws.sums + row0 * a.segs;
    const u64* keys = ws.keys + row0 * a.segs * a.keep;
    auto score_of = [&](int w) { return a.scores ? (double)a.scores[row0 + w] : 0.; };
    auto over = [&](int w) { return a.ended && a.ended[row0 + w]; };
    // a thread for each list: the sums of up to eight neighbours of a row
    const int near = a.segs < 8 ? a.segs : 8, parts = a.segs / near;
    for (int i = tid; i - lane < lists; i += 64 * kBlockWaves) {
        SelectSum p = {0., -3.4028235e38f, -INFINITY, 0, {}};
        if (i < lists) p = sums[i];         // of a row that was not read: anything
        float ref = p.ref, top = p.top;
        for (int d = 1; d < near; d <<= 1) {
            ref = fmaxf(ref, __shfl_xor(ref, d, 64));
            top = __builtin_elementwise_maximum(top, __shfl_xor(top, d, 64));
        }
        double sum = p.sum * moved(p.ref, ref);
        for (int d = 1; d < near; d <<= 1) sum += __shfl_xor(sum, d, 64);
        if (i < lists) {
            s.best[i] = p.top;
            s.held[i] = (unsigned char)p.n;
            if (i % near == 0) {
                s.part_sum[i / near] = sum;
                s.part_ref[i / near] = ref;
                s.part_top[i / near] = top;
            }
        }
    }
    if (tid == 0) s.lists = 0;
    __syncthreads();
    const bool few = lists * a.keep <= 128;      // none is left out before they are ordered
    for (int w = tid; w < a.beams; w += 64 * kBlockWaves) {
        const double score = score_of(w);
        double to = NAN;
        if (fabs(score) < INFINITY && !over(w)) {
            float ref = s.part_ref[w * parts], top = s.part_top[w * parts];
            for (int i = 1; i < parts; ++i) {
                ref = fmaxf(ref, s.part_ref[w * parts + i]);
                top = __builtin_elementwise_maximum(top, s.part_top[w * parts + i]);
            }
            double sum = 0;
            for (int i = 0; i < parts; ++i) sum += s.part_sum[w * parts + i] * moved(s.part_ref[w * parts + i], ref);
            // Rows of the same logits in another order tie, as far as 64 bits tell: their sums are the same but for the
            // additions' rounding and a power of two, which follows from the reference and is taken out first; and the
            // logarithm is rounded to whole multiples of 2^-32, far above its last bits and below the exponentials' 2^-29.
            int up;
            const double part = frexp(sum, &up);
            const double l = far(ref) ? (double)ref + log(sum) : fma(whole(ref) + up, kLn2, log(part));
            if (top < INFINITY) to = rint(l * 0x1p32) * 0x1p-32;
        }
        s.score[w] = score;
        s.log_sum[w] = to;
    }
    __syncthreads();
    for (int i = tid; i < lists; i += 64 * kBlockWaves) {
        const unsigned w = (unsigned)i / (unsigned)a.segs;
        const double l = s.log_sum[w];
        const bool in = l == l && s.best[i] > -INFINITY;
        s.best[i] = in ? round_down(s.score[w] + ((double)s.best[i] - l)) : -INFINITY;
        if (!in) s.held[i] = 0;
    }
    __syncthreads();
    float floor = -INFINITY;
    if (!few && lists >= a.keep) {
        float low = -INFINITY, high = -INFINITY;
        for (int i = lane; i < lists; i += 128) {
            low = fmaxf(low, s.best[i]);
            if (i + 64 < lists) high = fmaxf(high, s.best[i + 64]);
        }
        float kth[1];
        kth_of_lanes(low, high, {a.keep}, kth);
        floor = kth[0];
    }
    for (int i = tid; i < lists; i += 64 * kBlockWaves)
        if (s.held[i] && s.best[i] >= floor) s.list[atomicAdd(&s.lists, 1)] = (unsigned short)i;
    __syncthreads();

    Best* buf = s.room[wave];
    int n = 0;
    Best least{};
    auto enter = [&](bool in, const Best& k) {
        const u64 go = __ballot(in && above(k, least));
        if (!go) return;
        if (n > kJoinRoom - 64) {
            least = keep_largest<kJoinRoom>(buf, n, a.keep);
            n = a.keep;
        }
        if (go >> lane & 1) buf[n + __popcll(go & ((1ull << lane) - 1))] = k;
        n += __popcll(go);
    };
    const int count = s.lists;
    for (int i0 = wave; i0 < count; i0 += 4 * kBlockWaves) {
        int l[4], held[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kBlockWaves;
            l[u] = __builtin_amdgcn_readfirstlane(i < count ? (int)s.list[i] : 0);
            held[u] = __builtin_amdgcn_readfirstlane(i < count ? (int)s.held[l[u]] : 0);
        }
        for (int j0 = 0; j0 < a.keep; j0 += 64) {
            const int j = j0 + lane;
            u64 key[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) key[u] = j < held[u] ? keys[(int64_t)l[u] * a.keep + j] : 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (j0 >= held[u]) continue;
                const int w = l[u] / a.segs;
                const double score = s.score[w] + ((double)unordered((unsigned)(key[u] >> 32)) - s.log_sum[w]) + 0.;
                const unsigned item = 0xffffffffu - (unsigned)key[u];
                enter(key[u] && score >= (double)floor,
                      Best{ordered(score), (u64)(kMostBeams - 1 - w) << 57 | (key[u] >> 32) << kItemBits |
                                               ((1u << kItemBits) - 1 - item)});
            }
        }
    }
    if (a.ended && wave == 0)               // beams that ended carry themselves over
        for (int w0 = 0; w0 < a.beams; w0 += 64) {
            const int w = w0 + lane;
            const bool carry = w < a.beams && over(w);
            const double score = carry ? score_of(w) : 0.;
            enter(carry && fabs(score) < INFINITY, Best{ordered(score + 0.), (u64)(kMostBeams - 1 - w) << 57});
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (!few) {                             // what every wave has keep / kBlockWaves of
        const float x = lane < n ? round_down(unordered(buf[lane].score)) : -INFINITY;
        const float y = lane + 64 < n ? round_down(unordered(buf[lane + 64].score)) : -INFINITY;
        float own[1];
        kth_of_lanes(x, y, {(a.keep + kBlockWaves - 1) / kBlockWaves}, own);
        if (lane == 0) s.found[wave] = own[0];
        __syncthreads();
        floor = s.found[0];
#pragma unroll
        for (int o = 1; o < kBlockWaves; ++o) floor = fminf(floor, s.found[o]);
        int m = 0;                          // that reach it, moved to the front
        for (int i0 = 0; i0 < n; i0 += 64) {
            const Best k = i0 + lane < n ? buf[i0 + lane] : Best{};
            const u64 go = __ballot(i0 + lane < n && unordered(k.score) >= (double)floor);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (go >> lane & 1) buf[m + __popcll(go & ((1ull << lane) - 1))] = k;
            m += __popcll(go);
        }
        n = m;
    }
    if (lane == 0) s.count[wave] = n;
    __syncthreads();
    int first = 0, all = 0;
#pragma unroll
    for (int o = 0; o < kBlockWaves; ++o) {
        first += o < wave ? s.count[o] : 0;
        all += s.count[o];
    }
    if (all <= kPool) {
        for (int i = lane; i < n; i += 64) s.pool[first + i] = buf[i];
    } else if (wave == 0) {                 // many equal ones: the best of two waves at a time
        for (int o = 1; o < kBlockWaves; ++o)
            for (int i0 = 0; i0 < s.count[o]; i0 += 64) {
                const int i = i0 + lane;
                enter(i < s.count[o], i < s.count[o] ? s.room[o][i] : Best{});
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        for (int i = lane; i < n; i += 64) s.pool[i] = buf[i];
        if (lane == 0) s.joined = n;
    }
    for (int i = tid; i < kPool; i += 64 * kBlockWaves) s.place[i] = 0;
    __syncthreads();
    n = all <= kPool ? all : s.joined;
    // each one's place: how many are above it, counted by `split` threads
    const int split = max(64 * kBlockWaves / max(n, 1), 1);
    for (int i = tid; i < n * split; i += 64 * kBlockWaves) {
        const int c = i / split, part = i % split;
        const Best k = s.pool[c];
        int place = 0;
#pragma unroll 4
        for (int j = part; j < n; j += split) place += above(s.pool[j], k) ? 1 : 0;
        atomicAdd(&s.place[c], place);
    }
    __syncthreads();
    const int64_t out = (int64_t)group * a.keep;
    for (int i = tid; i < n; i += 64 * kBlockWaves) {
        const int place = s.place[i];
        if (place >= a.keep) continue;
        const Best k = s.pool[i];
        const int w = kMostBeams - 1 - (int)(k.rest >> 57);
        a.out_scores[out + place] = (float)unordered(k.score);
        a.out_parents[out + place] = w;
        a.out_items[out + place] = over(w) ? a.end_item : (1 << kItemBits) - 1 - (int)(k.rest & ((1u << kItemBits) - 1));
    }
    for (int i = n + tid; i < a.keep; i += 64 * kBlockWaves) {
        a.out_scores[out + i] = -INFINITY;
        a.out_parents[out + i] = a.out_items[out + i] = -1;
    }
}

template <typename T, bool MASKED>
__global__ __launch_bounds__(64 * kBlockWaves, 4) void history_select_kernel(SelectArgs a, SelectWs ws) {
    __shared__ SelectShared s;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    select_part<T, MASKED>(a, ws, (int64_t)blockIdx.x * kBlockWaves + wave, s);
}

__global__ __launch_bounds__(64 * kBlockWaves) void history_select_join_kernel(SelectArgs a, SelectWs ws) {
    __shared__ JoinShared s;
    join_group(a, ws, blockIdx.x, s);
}

// Both steps in one launch, a block per group.
template <typename T, bool MASKED>
__global__ __launch_bounds__(64 * kBlockWaves) void history_select_one_kernel(SelectArgs a, SelectWs ws) {
    __shared__ union Both {
        SelectShared part;
        JoinShared join;
        __device__ Both() {}
    } s;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), units = a.beams * a.segs;
    select_part<T, MASKED>(a, ws, wave < units ? (int64_t)blockIdx.x * units + wave : -1, s.part);
    __threadfence_block();                  // the sums and keys are read by other waves of the block
    __syncthreads();
    join_group(a, ws, blockIdx.x, s.join);
}

// Parts that a row is cut into: enough waves to fill the card, 2048 logits at least for each.  A power of two, or whole
// blocks, so that the waves of a block know each other's rows.
static int segs_of(int64_t batch, int beams, int64_t items) {
    const int64_t rows = batch * beams, least = (items + 2047) / 2048;
    int64_t s = (kSelectWaves + rows - 1) / rows;
    s = s < least ? s : least;
    s = s < kMostSegs ? s : kMostSegs;
    s = s < kMostLists / beams ? s : kMostLists / beams;
    if (s >= kBlockWaves) return (int)(s / kBlockWaves * kBlockWaves);
    return s >= 4 ? 4 : (s >= 2 ? 2 : 1);
}

static size_t sums_bytes(int64_t units) { return ((size_t)units * sizeof(SelectSum) + 255) / 256 * 256; }

size_t select_workspace_bytes(int64_t batch, int beams, int64_t items, int keep) {
    const int64_t units = batch * beams * segs_of(batch, beams, items);
    return sums_bytes(units) + (size_t)units * keep * sizeof(u64);
}

static bool in_one_launch(const SelectArgs& a) {
    return a.beams * a.segs <= kBlockWaves && (int64_t)a.beams * a.items <= kOneLogits && a.batch <= kOneGroups;
}

template <typename T>
static void launch_select(const SelectArgs& a, const SelectWs& ws, int64_t blocks, hipStream_t s) {
    if (in_one_launch(a)) {
        if (a.allowed) hipLaunchKernelGGL((history_select_one_kernel<T, true>), dim3(a.batch), dim3(64 * kBlockWaves), 0, s, a, ws);
        else hipLaunchKernelGGL((history_select_one_kernel<T, false>), dim3(a.batch), dim3(64 * kBlockWaves), 0, s, a, ws);
        return;
    }
    if (a.allowed) hipLaunchKernelGGL((history_select_kernel<T, true>), dim3(blocks), dim3(64 * kBlockWaves), 0, s, a, ws);
    else hipLaunchKernelGGL((history_select_kernel<T, false>), dim3(blocks), dim3(64 * kBlockWaves), 0, s, a, ws);
}

hipError_t launch_history_select(const SelectArgs& args, int dtype, void* workspace, hipStream_t s) {
    SelectArgs a = args;
    a.segs = segs_of(a.batch, a.beams, a.items);
    const int64_t units = (int64_t)a.batch * a.beams * a.segs, blocks = (units + kBlockWaves - 1) / kBlockWaves;
    if (!grid_fits(blocks, 64 * kBlockWaves) || !grid_fits(a.batch, 64 * kBlockWaves)) return kTooLarge;
    SelectWs ws;
    ws.sums = (SelectSum*)workspace;
    ws.keys = (u64*)((char*)workspace + sums_bytes(units));
    if (dtype == DLRM_DTYPE_F32) launch_select<float>(a, ws, blocks, s);
    else if (dtype == DLRM_DTYPE_BF16) launch_select<bf16>(a, ws, blocks, s);
    else launch_select<f16>(a, ws, blocks, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (in_one_launch(a)) return hipSuccess;
    hipLaunchKernelGGL(history_select_join_kernel, dim3(a.batch), dim3(64 * kBlockWaves), 0, s, a, ws);
    return hipGetLastError();
}

}  // namespace dlrm
