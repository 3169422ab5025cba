// history_select.hip -- the best continuations of a group of histories: beams x
// items by the sum of a beam's score and an item's log-probability.
//
//   s(w, v) = score_w + x(w, v) - log sum_u exp x(w, u)       over the allowed u
//
// The `keep` largest s of a group, in descending order; equal ones by beam, then by
// item.  Within a beam the order is that of the logits, so that a row's best items
// are found without its sum, in the same pass over it.
#include "history.h"

namespace dlrm {

typedef unsigned long long u64;

constexpr int kSelectTile = 512;         // logits a wave takes at a time: eight a lane
constexpr int kSelectRoom = 1024;        // candidates a wave has room for
constexpr int kSelectWaves = 4096;       // waves a launch aims at: sixteen on each CU
constexpr int kJoinWaves = 8;
constexpr int kJoinRoom = 512;
constexpr int kMostLists = 4096;         // parts of a group's rows

// What one wave leaves of its part of a row: the sum of exponentials against `ref`,
// the largest logit, and whether a NaN was among them.
struct SelectSum {
    double sum;
    float ref, top;
    int bad;
};

struct SelectWs {
    SelectSum* sums;     // (rows, segs)
    u64* keys;           // (rows, segs, keep): 0 where there is none
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
__device__ __forceinline__ K keep_largest(K* buf, int n, int keep) {
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

// The keep-th largest of two values per lane, 1 <= keep <= 128.
__device__ __forceinline__ float kth_of_lanes(float a, float b, int keep) {
    const unsigned x = ordered(a + 0.f), y = ordered(b + 0.f);
    unsigned t = 0;
    for (unsigned bit = 0x80000000u; bit; bit >>= 1) {
        const int count = __popcll(__ballot(x >= (t | bit))) + __popcll(__ballot(y >= (t | bit)));
        if (count >= keep) t |= bit;
        if (count == keep) break;
    }
    return unordered(t > 0x007fffffu ? t : 0x007fffffu);        // below -inf there are only NaN
}

// e^d for d up to 600, to 2^-34 of its value; below -690 as if it were -690, which is
// nothing against any sum that counts.  d log2 e is split into a whole number and a
// rest of at most a half by adding and taking away 1.5 x 2^52; a polynomial of the
// seventh degree, fitted to the least relative error, gives 2 to the rest.
__device__ __forceinline__ double weight(double d) {
    constexpr double L = 1.4426950408889634, SHIFT = 0x1.8p52;
    d = fmax(d, -690.);
    const double k = fma(d, L, SHIFT), f = fma(d, L, SHIFT - k);
    double p = 0x1.fe17826c2a406p-17;
    p = fma(p, f, 0x1.446a1fd688addp-13);
    p = fma(p, f, 0x1.5d8a708988ddcp-10);
    p = fma(p, f, 0x1.3b29dc40dc8a4p-7);
    p = fma(p, f, 0x1.c6b08aaf2db33p-5);
    p = fma(p, f, 0x1.ebfbe0a4be78ap-3);
    p = fma(p, f, 0x1.62e42ff116296p-1);
    p = fma(p, f, 0x1.ffffffffabbcdp-1);
    return __hiloint2double(__double2hiint(p) + (__double2loint(k) << 20), __double2loint(p));
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
        f[i] = (float)e.x[i];
        if constexpr (MASKED) f[i] = ((i < 4 ? r.may.x : r.may.y) >> (8 * (i & 3)) & 0xffu) ? f[i] : -INFINITY;
    }
}

// One wave's part of a row.  The sum is taken against `ref`, which needs only be near
// the largest logit: 64 bits hold e^300 times too much, so that it moves in no
// ordinary row, and no tile waits for a maximum over the wave.  Only logits that reach
// `floor` can be among the best: the keep-th largest of 128 groups of logits, and of
// the candidates when their room was last full.  Most tiles have none.
template <typename T, bool MASKED>
__device__ __forceinline__ void select_part(const SelectArgs& a, const SelectWs& ws, int64_t unit, u64* buf) {
    const int lane = threadIdx.x & 63;
    const int64_t row = unit / a.segs;
    const int seg = (int)(unit - row * a.segs);
    if (a.scores && !(fabsf(a.scores[row]) < INFINITY)) return;      // nothing of the row is read, here or by the join
    if (a.ended && a.ended[row]) return;
    const int tiles = (a.items + kSelectTile - 1) / kSelectTile;
    const int t0 = (int)((int64_t)tiles * seg / a.segs), t1 = (int)((int64_t)tiles * (seg + 1) / a.segs);
    const T* x = (const T*)a.logits + row * a.ld_logits;
    const uint8_t* may = MASKED ? a.allowed + row * a.ld_allowed : nullptr;

    int n = 0;
    u64 least = 0;                 // candidates have to be larger
    float ref = -3.4028235e38f, floor = -INFINITY, low = -INFINITY, high = -INFINITY;
    double sum = 0;
    bool bad = false;
    Eight<T> next = load_eight<T, MASKED>(x, may, t0 * kSelectTile + lane * 8, a.items);
    for (int t = t0; t < t1; ++t) {
        const int at = t * kSelectTile + lane * 8;
        const Eight<T> raw = next;
        if (t + 1 < t1) next = load_eight<T, MASKED>(x, may, at + kSelectTile, a.items);
        float f[8];
        values_of<T, MASKED>(raw, f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) bad |= __builtin_isunordered(f[i], f[i + 1]);
        const float l = fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), h = fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7]));
        low = fmaxf(low, l);
        high = fmaxf(high, h);
        const float top = fmaxf(l, h);
        if (__builtin_expect(__any(top > ref + 300.f), 0)) {
            const float to = wave_max(top);
            sum *= weight((double)ref - (double)to);
            ref = to;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += weight((double)f[i] - (double)ref);
        const int done = t - t0 + 1;
        if ((done & (done - 1)) == 0) floor = fmaxf(floor, kth_of_lanes(low, high, a.keep));
        if (__any(top >= floor)) {
            if (n > kSelectRoom - kSelectTile) {
                least = keep_largest<kSelectRoom>(buf, n, a.keep);
                floor = fmaxf(floor, unordered((unsigned)(least >> 32)));
                n = a.keep;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u64 key = (u64)ordered(f[i] + 0.f) << 32 | (0xffffffffu - (unsigned)(at + i));
                const u64 in = __ballot(f[i] >= floor && f[i] > -INFINITY && key > least);
                if (in >> lane & 1) buf[n + __popcll(in & ((1ull << lane) - 1))] = key;
                n += __popcll(in);
            }
        }
    }
    if (n > a.keep) {
        keep_largest<kSelectRoom>(buf, n, a.keep);
        n = a.keep;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    u64* keys = ws.keys + unit * a.keep;
    for (int i = lane; i < a.keep; i += 64) keys[i] = i < n ? buf[i] : 0;
    const float most = wave_max(fmaxf(low, high));
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
    const int any = __any(bad);
    if (lane == 0) ws.sums[unit] = SelectSum{sum, ref, most, any};
}

// The largest fp32 value that is not above x.
__device__ __forceinline__ float round_down(double x) {
    const float f = (float)x;
    if (!((double)f > x)) return f;
    const unsigned k = ordered(f + 0.f) - 1;
    return unordered(k);
}

struct JoinShared {
    double base[kMostBeams];                // score - log of the sum; NaN: the beam gives no candidates
    Best room[kJoinWaves][kJoinRoom];
    unsigned short list[kMostLists];        // the lists that may hold one of the best
    int lists, held[kJoinWaves];
};

// Joins the parts of a group's rows, by a block of kJoinWaves waves.  No list whose
// largest logit gives less than the keep-th largest of the lists' is read.
__device__ __forceinline__ void join_group(const SelectArgs& a, const SelectWs& ws, int group, JoinShared& s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row0 = (int64_t)group * a.beams;
    const int lists = a.beams * a.segs;
    const SelectSum* sums = ws.sums + row0 * a.segs;
    const u64* keys = ws.keys + row0 * a.segs * a.keep;
    for (int w = wave; w < a.beams; w += kJoinWaves) {
        const double score = a.scores ? (double)a.scores[row0 + w] : 0.;
        const bool over = a.ended && a.ended[row0 + w];
        double to = NAN;
        if (fabs(score) < INFINITY && !over) {
            const SelectSum* p = sums + w * a.segs;
            float m = -INFINITY;
            bool bad = false;
            for (int i = lane; i < a.segs; i += 64) {
                m = fmaxf(m, p[i].ref);
                bad |= p[i].bad != 0;
            }
            m = wave_max(m);
            double sum = 0;
            for (int i = lane; i < a.segs; i += 64) sum += p[i].sum * weight((double)p[i].ref - (double)m);
#pragma unroll
            for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
            if (!__any(bad) && m < INFINITY) to = score - ((double)m + log(sum));
        }
        if (lane == 0) s.base[w] = to;
    }
    if (tid == 0) s.lists = 0;
    __syncthreads();

    // the best score of list i, rounded down, and whether it has one
    auto best_of = [&](int i, bool* in) {
        const double b = s.base[i / a.segs];
        const float top = b == b ? sums[i].top : -INFINITY;
        *in = top > -INFINITY;
        return *in ? round_down(b + (double)top) : -INFINITY;
    };
    bool in;
    float low = -INFINITY, high = -INFINITY;
    for (int i = lane; i < lists; i += 128) {
        low = fmaxf(low, best_of(i, &in));
        if (i + 64 < lists) high = fmaxf(high, best_of(i + 64, &in));
    }
    const float floor = kth_of_lanes(low, high, a.keep);
    for (int i = tid; i < lists; i += 64 * kJoinWaves) {
        const float b = best_of(i, &in);
        if (in && b >= floor) s.list[atomicAdd(&s.lists, 1)] = (unsigned short)i;
    }
    __syncthreads();

    Best* buf = s.room[wave];
    int n = 0;
    Best least{};
    auto enter = [&](bool in, const Best& k) {
        if (n > kJoinRoom - 64) {
            least = keep_largest<kJoinRoom>(buf, n, a.keep);
            n = a.keep;
        }
        const u64 go = __ballot(in && above(k, least));
        if (go >> lane & 1) buf[n + __popcll(go & ((1ull << lane) - 1))] = k;
        n += __popcll(go);
    };
    auto settle = [&] {
        if (n > a.keep) {
            least = keep_largest<kJoinRoom>(buf, n, a.keep);
            n = a.keep;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    const int count = s.lists;
    for (int i0 = wave; i0 < count; i0 += 2 * kJoinWaves)
        for (int j = lane; j - lane < a.keep; j += 64) {
            u64 key[2];
            int l[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = i0 + u * kJoinWaves;
                l[u] = __builtin_amdgcn_readfirstlane(i < count ? (int)s.list[i] : -1);
                key[u] = l[u] >= 0 && j < a.keep ? keys[(int64_t)l[u] * a.keep + j] : 0;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (l[u] < 0) continue;
                const int w = l[u] / a.segs;
                const double score = s.base[w] + (double)unordered((unsigned)(key[u] >> 32)) + 0.;
                const unsigned item = 0xffffffffu - (unsigned)key[u];
                enter(key[u] && score >= (double)floor,
                      Best{ordered(score), (u64)(kMostBeams - 1 - w) << 57 | (key[u] >> 32) << kItemBits |
                                               ((1u << kItemBits) - 1 - item)});
            }
        }
    if (a.ended && wave == 0)               // beams that ended carry themselves over
        for (int w0 = 0; w0 < a.beams; w0 += 64) {
            const int w = w0 + lane;
            const bool over = w < a.beams && a.ended[row0 + w];
            const double score = over && a.scores ? (double)a.scores[row0 + w] : 0.;
            enter(over && fabs(score) < INFINITY, Best{ordered(score + 0.), (u64)(kMostBeams - 1 - w) << 57});
        }
    settle();
    if (lane == 0) s.held[wave] = n;
    __syncthreads();
    if (wave != 0) return;
    for (int o = 1; o < kJoinWaves; ++o)
        for (int i0 = 0; i0 < s.held[o]; i0 += 64) {
            const int i = i0 + lane;
            enter(i < s.held[o], i < s.held[o] ? s.room[o][i] : Best{});
        }
    settle();
    // each one's place: how many are above it
    const int64_t out = (int64_t)group * a.keep;
    for (int i = lane; i < a.keep; i += 64) {
        if (i >= n) {
            a.out_scores[out + i] = -INFINITY;
            a.out_parents[out + i] = a.out_items[out + i] = -1;
            continue;
        }
        const Best k = buf[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += above(buf[j], k) ? 1 : 0;
        const int w = kMostBeams - 1 - (int)(k.rest >> 57);
        const bool over = a.ended && a.ended[row0 + w];
        a.out_scores[out + place] = (float)unordered(k.score);
        a.out_parents[out + place] = w;
        a.out_items[out + place] = over ? a.end_item : (1 << kItemBits) - 1 - (int)(k.rest & ((1u << kItemBits) - 1));
    }
}

template <typename T, bool MASKED>
__global__ __launch_bounds__(256) void history_select_kernel(SelectArgs a, SelectWs ws) {
    __shared__ u64 room[4][kSelectRoom];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    if (unit < (int64_t)a.batch * a.beams * a.segs) select_part<T, MASKED>(a, ws, unit, room[wave]);
}

__global__ __launch_bounds__(64 * kJoinWaves) void history_select_join_kernel(SelectArgs a, SelectWs ws) {
    __shared__ JoinShared s;
    join_group(a, ws, blockIdx.x, s);
}

// Parts that a row is cut into: enough waves to fill the card, four tiles at least for each, and no more lists and
// candidates than a block can join.
static int segs_of(int64_t batch, int beams, int64_t items, int keep) {
    const int64_t rows = batch * beams, tiles = (items + kSelectTile - 1) / kSelectTile;
    int64_t s = (kSelectWaves + rows - 1) / rows;
    s = s < (tiles + 3) / 4 ? s : (tiles + 3) / 4;
    const int64_t most = kMostLists / beams;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s);
}

static size_t sums_bytes(int64_t units) { return ((size_t)units * sizeof(SelectSum) + 255) / 256 * 256; }

size_t select_workspace_bytes(int64_t batch, int beams, int64_t items, int keep) {
    const int64_t units = batch * beams * segs_of(batch, beams, items, keep);
    return sums_bytes(units) + (size_t)units * keep * sizeof(u64);
}

template <typename T>
static void launch_select(const SelectArgs& a, const SelectWs& ws, int64_t blocks, hipStream_t s) {
    if (a.allowed) hipLaunchKernelGGL((history_select_kernel<T, true>), dim3(blocks), dim3(256), 0, s, a, ws);
    else hipLaunchKernelGGL((history_select_kernel<T, false>), dim3(blocks), dim3(256), 0, s, a, ws);
}

hipError_t launch_history_select(const SelectArgs& args, int dtype, void* workspace, hipStream_t s) {
    SelectArgs a = args;
    a.segs = segs_of(a.batch, a.beams, a.items, a.keep);
    const int64_t units = (int64_t)a.batch * a.beams * a.segs, blocks = (units + 3) / 4;
    if (!grid_fits(blocks, 256) || !grid_fits(a.batch, 64 * kJoinWaves)) return kTooLarge;
    SelectWs ws;
    ws.sums = (SelectSum*)workspace;
    ws.keys = (u64*)((char*)workspace + sums_bytes(units));
    if (dtype == DLRM_DTYPE_F32) launch_select<float>(a, ws, blocks, s);
    else if (dtype == DLRM_DTYPE_BF16) launch_select<bf16>(a, ws, blocks, s);
    else launch_select<f16>(a, ws, blocks, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(history_select_join_kernel, dim3(a.batch), dim3(64 * kJoinWaves), 0, s, a, ws);
    return hipGetLastError();
}

}  // namespace dlrm
