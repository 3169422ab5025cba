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
constexpr int kJoinRoom = 512;

// What one wave leaves of its part of a row: the largest logit, the sum of
// exponentials against it, and whether a NaN was among them.
struct SelectSum {
    double sum;
    float top;
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
__device__ __forceinline__ u64 with_bit(u64 k, int bit) { return k | 1ull << bit; }
__device__ __forceinline__ Best with_bit(Best k, int bit) {
    if (bit >= 64) k.score |= 1ull << (bit - 64);
    else k.rest |= 1ull << bit;
    return k;
}

// Keeps the `keep` largest of the n > keep different keys in buf and returns the
// smallest of them.  The bits of the keep-th largest are found from the highest
// down, until exactly `keep` keys reach what is known of it.
template <int ROOM, int BITS, typename K>
__device__ __forceinline__ K keep_largest(K* buf, int n, int keep) {
    const int lane = threadIdx.x & 63;
    K e[ROOM / 64];
#pragma unroll
    for (int i = 0; i < ROOM / 64; ++i) e[i] = i * 64 + lane < n ? buf[i * 64 + lane] : K{};
    K t{};
    for (int bit = BITS - 1; bit >= 0; --bit) {
        const K c = with_bit(t, bit);
        int count = 0;
#pragma unroll
        for (int i = 0; i < ROOM / 64; ++i) count += __popcll(__ballot(reaches(e[i], c)));
        if (count >= keep) t = c;
        if (count == keep) break;
    }
    int at = 0;
#pragma unroll
    for (int i = 0; i < ROOM / 64; ++i) {
        const u64 in = __ballot(reaches(e[i], t));
        if (in >> lane & 1) buf[at + __popcll(in & ((1ull << lane) - 1))] = e[i];
        at += __popcll(in);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return t;
}

// One wave per (row, part of its items).
template <typename T, bool MASKED>
__global__ __launch_bounds__(256) void history_select_kernel(SelectArgs a, SelectWs ws) {
    __shared__ u64 room[4][kSelectRoom];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
    const int64_t row = unit / a.segs;
    const int seg = (int)(unit % a.segs);
    if (row >= (int64_t)a.batch * a.beams) return;
    const bool live = !a.scores || fabsf(a.scores[row]) < INFINITY;
    if (!live || (a.ended && a.ended[row])) return;          // nothing of the row is read, here or by the join
    u64* buf = room[wave];
    const int tiles = (a.items + kSelectTile - 1) / kSelectTile;
    const int t0 = (int)((int64_t)tiles * seg / a.segs), t1 = (int)((int64_t)tiles * (seg + 1) / a.segs);
    const T* x = (const T*)a.logits + row * a.ld_logits;
    const uint8_t* may = MASKED ? a.allowed + row * a.ld_allowed : nullptr;

    int n = 0;
    u64 least = 0;                 // candidates have to be larger
    float m = -3.4028235e38f, top = -INFINITY;
    double sum = 0;
    bool bad = false;
    for (int t = t0; t < t1; ++t) {
        const int at = t * kSelectTile + lane * 8;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = at + i < a.items && (!MASKED || may[at + i]);
            f[i] = in ? (float)x[at + i] + 0.f : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bad |= f[i] != f[i];
            top = fmaxf(top, f[i]);
        }
        if (top > m) {
            sum *= exp((double)m - (double)top);
            m = top;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += exp((double)f[i] - (double)m);
        if (n > kSelectRoom - kSelectTile) {
            least = keep_largest<kSelectRoom, 64>(buf, n, a.keep);
            n = a.keep;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const u64 key = (u64)ordered(f[i]) << 32 | (0xffffffffu - (unsigned)(at + i));
            const u64 in = __ballot(f[i] > -INFINITY && key > least);
            if (in >> lane & 1) buf[n + __popcll(in & ((1ull << lane) - 1))] = key;
            n += __popcll(in);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (n > a.keep) {
        keep_largest<kSelectRoom, 64>(buf, n, a.keep);
        n = a.keep;
    }
    u64* keys = ws.keys + unit * a.keep;
    for (int i = lane; i < a.keep; i += 64) keys[i] = i < n ? buf[i] : 0;
    const float all = wave_max(top);
    sum = top > -INFINITY ? sum * exp((double)m - (double)all) : 0.;
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
    const int any = __any(bad);
    if (lane == 0) ws.sums[unit] = SelectSum{sum, all, any};
}

// Joins the parts of a group's rows: a block per group.
__global__ __launch_bounds__(256) void history_select_join_kernel(SelectArgs a, SelectWs ws) {
    __shared__ double base[kMostBeams];                     // score - log sum; NaN: the beam gives no candidates
    __shared__ Best room[4][kJoinRoom];
    __shared__ int held[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    for (int w = wave; w < a.beams; w += 4) {
        const double score = a.scores ? (double)a.scores[row0 + w] : 0.;
        const bool over = a.ended && a.ended[row0 + w];
        double to = NAN;
        if (fabs(score) < INFINITY && !over) {
            const SelectSum* s = ws.sums + (row0 + w) * a.segs;
            float m = -INFINITY;
            bool bad = false;
            for (int i = lane; i < a.segs; i += 64) {
                m = fmaxf(m, s[i].top);
                bad |= s[i].bad != 0;
            }
            m = wave_max(m);
            double sum = 0;
            for (int i = lane; i < a.segs; i += 64)
                if (s[i].top > -INFINITY) sum += s[i].sum * exp((double)s[i].top - (double)m);
#pragma unroll
            for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
            if (!__any(bad) && fabsf(m) < INFINITY) to = score - ((double)m + log(sum));
        }
        if (lane == 0) base[w] = to;
    }
    __syncthreads();
    Best* buf = room[wave];
    const int list = a.segs * a.keep, each = a.beams * list;
    int n = 0;
    Best least{};
    auto enter = [&](bool in, const Best& k) {
        if (n > kJoinRoom - 64) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            least = keep_largest<kJoinRoom, 128>(buf, n, a.keep);
            n = a.keep;
        }
        const u64 go = __ballot(in && above(k, least));
        if (go >> lane & 1) buf[n + __popcll(go & ((1ull << lane) - 1))] = k;
        n += __popcll(go);
    };
    auto settle = [&] {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (n > a.keep) {
            least = keep_largest<kJoinRoom, 128>(buf, n, a.keep);
            n = a.keep;
        }
    };
    for (int i0 = wave * 64; i0 < each; i0 += 256) {
        const int i = i0 + lane;
        const int w = i < each ? i / list : 0;
        const double b = base[w];
        const bool in = i < each && b == b;
        const u64 key = in ? ws.keys[row0 * list + i] : 0;
        Best k{};
        if (key) {
            const unsigned item = 0xffffffffu - (unsigned)key;
            k.score = ordered(b + (double)unordered((unsigned)(key >> 32)) + 0.);
            k.rest = (u64)(kMostBeams - 1 - w) << 57 | (key >> 32) << kItemBits | ((1u << kItemBits) - 1 - item);
        }
        enter(key != 0, k);
    }
    if (a.ended && wave == 0)                               // beams that ended carry themselves over
        for (int w0 = 0; w0 < a.beams; w0 += 64) {
            const int w = w0 + lane;
            const bool over = w < a.beams && a.ended[row0 + w];
            const double score = over && a.scores ? (double)a.scores[row0 + w] : 0.;
            enter(over && fabs(score) < INFINITY, Best{ordered(score + 0.), (u64)(kMostBeams - 1 - w) << 57});
        }
    settle();
    if (lane == 0) held[wave] = n;
    __syncthreads();
    if (wave != 0) return;
    for (int o = 1; o < 4; ++o)
        for (int i0 = 0; i0 < held[o]; i0 += 64) {
            const int i = i0 + lane;
            enter(i < held[o], i < held[o] ? room[o][i] : Best{});
        }
    settle();
    // each one's place: how many are above it
    const int64_t out = (int64_t)blockIdx.x * a.keep;
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

// Parts that a row is cut into: enough waves to fill the card, four tiles at least for each, and no more candidates
// than a block can join in a few steps.
static int segs_of(int64_t batch, int beams, int64_t items, int keep) {
    const int64_t rows = batch * beams, tiles = (items + kSelectTile - 1) / kSelectTile;
    int64_t s = (kSelectWaves + rows - 1) / rows;
    s = s < (tiles + 3) / 4 ? s : (tiles + 3) / 4;
    const int64_t most = 16384 / ((int64_t)beams * keep);
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
    if (!grid_fits(blocks, 256) || !grid_fits(a.batch, 256)) return kTooLarge;
    SelectWs ws;
    ws.sums = (SelectSum*)workspace;
    ws.keys = (u64*)((char*)workspace + sums_bytes(units));
    if (dtype == DLRM_DTYPE_F32) launch_select<float>(a, ws, blocks, s);
    else if (dtype == DLRM_DTYPE_BF16) launch_select<bf16>(a, ws, blocks, s);
    else launch_select<f16>(a, ws, blocks, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(history_select_join_kernel, dim3(a.batch), dim3(256), 0, s, a, ws);
    return hipGetLastError();
}

}  // namespace dlrm
