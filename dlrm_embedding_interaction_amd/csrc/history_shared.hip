// history_shared.hip -- the lookup of groups of histories that share what came
// first: beams of one user, sessions opened on one history.
//
// A fork shares pages, so what histories have in common shows in their page lists.
// Per group, a first kernel finds which 64-event tiles lie on the same pages in all of
// its histories.  A second one reads those tiles once for all
// rows of the group (histories x queries x heads per kv head, in chunks of 16, one
// chunk per wave; the waves of a block read the same tiles at the same time).  The
// tiles of all groups make one row, cut into equal runs per block whatever the
// lengths are; every piece of a run that lies in one group leaves its maximum, sum
// and weighted sum in the workspace.  A third kernel, a block for each history, kv
// head and chunk of its rows, reads the tiles that are the history's own and joins
// them with the pieces.
//
// A shared tile is one that every row of the group sees whole.  Where windows or sinks
// of the histories end at different events, the tiles around these ends are each one's
// own: a row that does not see an event must not meet its value, which may be a NaN.
#include "history_tile.h"

namespace dlrm {

constexpr int kTailBlocks = 512;          // rows' blocks of one wave from here on, of four below
constexpr int kSharedWaves = 2048;       // waves the shared tiles' kernel aims at: two on each SIMD

// A group: its rows of the batch, the slot of one of its histories with events, and
// the shared tiles: [0, lead) and [first, common), `count` in all.  All rows see all
// of a shared tile, so that no row's mask is needed there.
struct Group {
    int begin, end, slot, lead, first, common, count;
};
// Where the group stands in the row of all tiles: of its tiles, and of its pieces.
struct Place {
    int64_t tile, piece;
};

struct SharedWs {
    Group* groups;          // (n_groups)
    Place* places;          // (n_groups)
    int* group_of;          // (batch)
    int64_t* per;           // tiles of a run
    int64_t pieces;         // that there is room for: as many as there can be while no two groups overlap
    float* partial;         // (pieces, kv heads, waves of a block, 16 (head_dim + 2))
};

// A block per group: the tiles that lie on the same pages in all of its histories
// and that all of them see whole.  Histories without events see nothing and do not
// count.
constexpr int kGroupThreads = 1024;
__global__ __launch_bounds__(kGroupThreads) void history_group_kernel(SharedArgs a, SharedWs ws) {
    __shared__ int len_min, lead_min, low_max, differs, some;
    __shared__ int slot_of[kGroupThreads];
    const LookupArgs& l = a.l;
    const dlrm_history_cache_t& c = l.c;
    const int g = blockIdx.x, tid = threadIdx.x;
    int begin, end;
    if (a.groups) {
        begin = g == 0 ? 0 : (int)history_begin(a.groups, a.idx32, g, l.batch);
        end = (int)history_end(a.groups, a.idx32, g, a.n_groups, begin, l.batch);
    } else {
        const int each = l.batch / a.n_groups;
        begin = g * each;
        end = begin + each;
    }
    if (tid == 0) {
        len_min = lead_min = differs = 0x7fffffff;
        low_max = 0;
        some = -1;
    }
    __syncthreads();
    for (int b = begin + tid; b < end; b += kGroupThreads) {
        ws.group_of[b] = g;
        const Span s = span_of(l, b);
        if (!s.len) continue;
        atomicMin(&len_min, s.len);
        atomicMin(&lead_min, s.low ? s.lead_events : s.len);
        atomicMax(&low_max, s.low);
        atomicMax(&some, b);
    }
    __syncthreads();
    Group r = {begin, end, 0, 0, 0, 0, 0};
    if (some >= 0) {
        r.slot = l.slots ? l.slots[some] : some;
        const int pt = kTile / c.page_events, tiles = len_min / kTile;
        r.first = min((low_max + kTile - 1) / kTile, tiles);
        r.lead = min(lead_min / kTile, r.first);
        const int lead = r.lead * pt, first = r.first * pt;
        const int n = lead + tiles * pt - first;            // pages [0, lead) and [first, tiles pt)
        const int32_t* one = c.table + (int64_t)r.slot * c.max_pages;
        int least = 0x7fffffff;
        for (int b0 = begin; b0 < end; b0 += kGroupThreads) {
            const int here = min(end - b0, kGroupThreads);
            __syncthreads();
            if (tid < here) {
                const int slot = l.slots ? l.slots[b0 + tid] : b0 + tid;
                slot_of[tid] = slot >= 0 && slot < c.n_slots && c.lens[slot] > 0 ? slot : -1;
            }
            __syncthreads();
            for (int i = tid & 63; i < n; i += 64) {
                const int x = i < lead ? i : first + i - lead, p = one[x];
#pragma unroll 8
                for (int k = tid >> 6; k < here; k += kGroupThreads / 64) {
                    const int slot = slot_of[k];
                    const int q = slot >= 0 ? c.table[(int64_t)slot * c.max_pages + x] : p;
                    least = q != p ? min(least, x) : least;
                }
            }
        }
        if (least < 0x7fffffff) atomicMin(&differs, least);
        __syncthreads();
        r.common = min(differs / pt, tiles);
        r.first = min(r.first, r.common);
        r.lead = min(r.lead, r.common);
        r.count = r.lead + r.common - r.first;
    }
    if (tid == 0) ws.groups[g] = r;
}

// Blocks of `waves` chunks that the group's rows make.
__device__ __forceinline__ int64_t blocks_of(const Group& g, int rows, int waves) {
    return ((int64_t)(g.end - g.begin) * rows + 16 * waves - 1) / (16 * waves);
}

__device__ __forceinline__ int64_t wave_inclusive(int64_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up((long long)v, d, 64);
        if (lane >= d) v += o;
    }
    return v;
}

template <int D, int PE, typename T>
__global__ __launch_bounds__(256, 2) void history_shared_kernel(SharedArgs a, SharedWs ws, int waves) {
    constexpr int NQ = Parts<T>::q, PT = kTile / PE;
    const LookupArgs& l = a.l;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int n = lane & 15, g = lane >> 4, hk = blockIdx.y;
    const int heads = l.n_heads / l.c.n_kv_heads, rows = l.queries * heads;

    // tiles and pieces before each lane's share of the groups
    const int each = (a.n_groups + 63) / 64;
    const int lo = lane * each, hi = lo + each < a.n_groups ? lo + each : a.n_groups;
    int64_t tiles = 0, pieces = 0;
    for (int i = lo; i < hi; ++i) {
        const Group r = ws.groups[i];
        const int64_t blocks = blocks_of(r, rows, waves);
        tiles += blocks * r.count;
        pieces += blocks;
    }
    const int64_t tiles_in = wave_inclusive(tiles), pieces_in = wave_inclusive(pieces);
    const int64_t total = lane_value(tiles_in, 63);
    const int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (blockIdx.x + blockIdx.y + threadIdx.x == 0) *ws.per = per;
    int64_t at = blockIdx.x * per;
    if (at >= total) return;
    const int64_t stop = at + per < total ? at + per : total;
    const int mine = 63 - __builtin_clzll(__ballot(tiles_in - tiles <= at));
    int64_t start = lane_value(tiles_in - tiles, mine), piece = lane_value(pieces_in - pieces, mine);
    int gi = mine * each;

    const float c = exponent_scale(l.scale);
    while (at < stop) {
        const Group r = ws.groups[gi];
        const int64_t blocks = blocks_of(r, rows, waves);
        if (start + blocks * r.count <= at) {
            start += blocks * r.count;
            piece += blocks;
            ++gi;
            continue;
        }
        if (at == start && hk == 0 && threadIdx.x == 0) ws.places[gi] = Place{start, piece};
        const int64_t block = (at - start) / r.count;
        const int i0 = (int)(at - start - block * r.count);
        const int i1 = r.count - i0 < stop - at ? r.count : i0 + (int)(stop - at);
        at += i1 - i0;
        const int64_t chunk = block * waves + wave;
        const int64_t all = (int64_t)(r.end - r.begin) * rows;
        const int64_t place = piece + block + blockIdx.x;
        if (chunk * 16 >= all || place >= ws.pieces) continue;

        // the lane's column: a row of one of the group's histories
        const int64_t row = chunk * 16 + n < all ? chunk * 16 + n : chunk * 16;
        const int b = r.begin + (int)(row / rows), y = (int)(row % rows);
        bf16x8 q[D / 32][NQ];
        load_query<D>((const T*)l.q + ((int64_t)b * l.queries + y / heads) * l.ld_q + (int64_t)(hk * heads + y % heads) * D,
                      l.scale, l.wide, g, q);
        const int32_t* table = l.c.table + (int64_t)r.slot * l.c.max_pages;
        floatx4 o[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[j] = floatx4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, sum = 0.f;
        auto tile_of = [&](int i) { return i < r.lead ? i : r.first + (i - r.lead); };
        auto load = [&](int i, Tile<D>& t) { load_tile<D, PE>(l.c, table, tile_of(i) * PT, hk, n, g, t); };
        auto use = [&](Tile<D>& t) {
            use_tile<D, T>(t, q, c, 0, true, 0, 0, kTile, g, o, m, sum);       // all of it but pages that are not there
        };
        constexpr bool TURNS = D < 128 || NQ == 1;
        Tile<D> cur, nxt;
        load(i0, cur);
        for (int i = i0; i < i1; ++i) {
            if (i + 1 < i1) load(i + 1, nxt);
            use(cur);
            if constexpr (TURNS) {
                if (++i >= i1) break;
                if (i + 1 < i1) load(i + 1, cur);
                use(nxt);
            } else {
                cur = nxt;
            }
        }
        sum += swizzle_xor16(sum);
        sum += __shfl_xor(sum, 32, 64);
        float* part = ws.partial +
                      ((place * gridDim.y + hk) * waves + wave) * (16 * (D + 2));
#pragma unroll
        for (int j = 0; j < D / 16; ++j) *(floatx4*)(part + n * D + 16 * j + 4 * g) = o[j];
        if (g == 0) {
            part[16 * D + n] = m * c;
            part[16 * D + 16 + n] = sum;
        }
    }
}

// A block per (history, kv head, chunk of its rows): the tiles that are its own, and the join.
template <int D, int PE, typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void history_tail_kernel(SharedArgs a, SharedWs ws, int waves) {
    constexpr int NQ = Parts<T>::q, PT = kTile / PE, OP = D + 4;
    __shared__ __attribute__((aligned(16))) float part_o[WAVES > 1 ? WAVES * 16 * OP : 4];
    __shared__ float part_m[16 * WAVES], part_l[16 * WAVES];
    const LookupArgs& l = a.l;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4, b = blockIdx.x;
    const int heads = l.n_heads / l.c.n_kv_heads, rows = l.queries * heads, chunks = (rows + 15) / 16;
    const int hk = blockIdx.y / chunks, r0 = (blockIdx.y % chunks) * 16, y = r0 + n;
    const bool live = y < rows;
    const Span sp = span_of(l, b);
    if (sp.count == 0 && l.slots && blockIdx.y == 0 && tid == 0) count_refused(l, b);

    const int gi = ws.group_of[b];
    Group r = {0, 0, 0, 0, 0, 0, 0};
    if (gi >= 0 && gi < a.n_groups) r = ws.groups[gi];
    if (b < r.begin || b >= r.end || !sp.len) r.lead = r.first = r.common = r.count = 0;
    // the tiles that are the history's own: of its sinks, of its window before the shared ones, and behind them
    const int end = (sp.len + kTile - 1) / kTile;
    const int n0 = max(sp.lead - r.lead, 0), b1 = max(sp.first, r.lead), n1 = max(min(r.first, end) - b1, 0);
    const int b2 = max(sp.first, r.common), n2 = max(end - b2, 0);
    auto tile_of = [&](int i) { return i < n0 ? r.lead + i : (i < n0 + n1 ? b1 + i - n0 : b2 + i - n0 - n1); };
    const int count = n0 + n1 + n2;

    floatx4 o[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[j] = floatx4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, sum = 0.f;
    if (wave < count) {
        bf16x8 q[D / 32][NQ];
        const int yy = live ? y : 0;
        load_query<D>((const T*)l.q + ((int64_t)b * l.queries + yy / heads) * l.ld_q + (int64_t)(hk * heads + yy % heads) * D,
                      l.scale, l.wide, g, q);
        const int slot = l.slots ? l.slots[b] : b;
        const int32_t* table = l.c.table + (int64_t)slot * l.c.max_pages;
        const float c = exponent_scale(l.scale);
        Tile<D> cur, nxt;
        load_tile<D, PE>(l.c, table, tile_of(wave) * PT, hk, n, g, cur);
        for (int i = wave; i < count; i += WAVES) {
            if (i + WAVES < count) load_tile<D, PE>(l.c, table, tile_of(i + WAVES) * PT, hk, n, g, nxt);
            const int e0 = tile_of(i) * kTile;
            const bool whole = (e0 >= sp.low || e0 + kTile <= sp.lead_events) && e0 + kTile <= sp.len;
            use_tile<D, T>(cur, q, c, e0, whole, sp.low, sp.lead_events, sp.len, g, o, m, sum);
            cur = nxt;
        }
        m *= c;                                          // from here on in powers of two
        sum += swizzle_xor16(sum);
        sum += __shfl_xor(sum, 32, 64);
    }
    if (r.count) {
        const Place at = ws.places[gi];
        const int64_t per = *ws.per;
        const int64_t row = (int64_t)(b - r.begin) * rows + (live ? y : 0), chunk = row / 16, block = chunk / waves;
        const int64_t t0 = at.tile + block * r.count, run0 = t0 / per, run1 = (t0 + r.count - 1) / per;
        for (int64_t i = run0 + wave; __any(i <= run1); i += WAVES) {
            const int64_t place = at.piece + block + i;
            if (i > run1 || place < 0 || place >= ws.pieces) continue;
            const float* part = ws.partial + ((place * l.c.n_kv_heads + hk) * waves + chunk % waves) * (16 * (D + 2));
            const int col = (int)(row % 16);
            const float pm = part[16 * D + col], ps = part[16 * D + 16 + col];
            if (pm == -INFINITY) continue;
            const float mx = fmaxf(m, pm), f0 = __builtin_amdgcn_exp2f(m - mx), f1 = __builtin_amdgcn_exp2f(pm - mx);
            m = mx;
            sum = sum * f0 + ps * f1;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[j] = o[j] * f0 + *(const floatx4*)(part + col * D + 16 * j + 4 * g) * f1;
        }
    }
    if constexpr (WAVES == 1) {
        if (live) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            T* op = (T*)l.out + ((int64_t)b * l.queries + y / heads) * l.ld_out + (int64_t)(hk * heads + y % heads) * D;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) store4(op + 16 * j + 4 * g, o[j] * inv, l.wide);
        }
        return;
    }
    if (g == 0) part_m[wave * 16 + n] = m;
    __syncthreads();
    float mx = part_m[n];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) mx = fmaxf(mx, part_m[16 * i + n]);
    const float f = mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mx);
    if (g == 0) part_l[wave * 16 + n] = sum * f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) *(floatx4*)&part_o[(wave * 16 + n) * OP + 16 * j + 4 * g] = o[j] * f;
    __syncthreads();
    for (int x = tid; x < 4 * D; x += 64 * WAVES) {
        const int i = x / (D / 4), d = x % (D / 4) * 4, row = r0 + i;
        if (row >= rows) break;
        float all = part_l[i];
        floatx4 v = *(const floatx4*)&part_o[i * OP + d];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            all += part_l[16 * w + i];
            v += *(const floatx4*)&part_o[(16 * w + i) * OP + d];
        }
        T* op = (T*)l.out + ((int64_t)b * l.queries + row / heads) * l.ld_out + (int64_t)(hk * heads + row % heads) * D + d;
        store4(op, v * (all == 0.f ? 0.f : 1.f / all), l.wide);
    }
}

// Waves of a block, each with a chunk of 16 of its group's rows: as many as a group has chunks on average, up to four.
static int chunk_waves(int64_t batch, int64_t n_groups, int rows) {
    const int64_t chunks = ((batch + n_groups - 1) / n_groups * rows + 15) / 16;
    return chunks > 2 ? 4 : (chunks > 1 ? 2 : 1);
}
static int runs_of(int n_kv_heads, int waves) {
    const int n = kSharedWaves / (n_kv_heads * waves);
    return n < 1 ? 1 : n;
}

static size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Where the parts of the workspace begin.
struct SharedPlan {
    size_t places, group_of, per, partial, end;
    int64_t pieces;
};
static SharedPlan plan_of(const dlrm_history_cache_t& c, int64_t batch, int64_t n_groups, int rows, int waves) {
    SharedPlan p;
    p.places = round256(n_groups * sizeof(Group));
    p.group_of = p.places + round256(n_groups * sizeof(Place));
    p.per = p.group_of + round256(batch * sizeof(int));
    p.partial = p.per + 256;
    p.pieces = runs_of(c.n_kv_heads, waves) + batch * rows / (16 * waves) + n_groups;
    p.end = p.partial + (size_t)p.pieces * c.n_kv_heads * waves * 16 * (c.head_dim + 2) * sizeof(float);
    return p;
}

size_t shared_workspace_bytes(const dlrm_history_cache_t& c, int64_t batch, int64_t n_groups, int queries, int n_heads) {
    const int rows = queries * (n_heads / c.n_kv_heads);
    return plan_of(c, batch, n_groups, rows, chunk_waves(batch, n_groups, rows)).end;
}

template <int D, int PE, typename T>
static hipError_t launch_t(const SharedArgs& a, void* workspace, hipStream_t s) {
    const LookupArgs& l = a.l;
    const int rows = l.queries * (l.n_heads / l.c.n_kv_heads), waves = chunk_waves(l.batch, a.n_groups, rows);
    if (!grid_fits(l.batch, 256) || !grid_fits(a.n_groups, kGroupThreads)) return kTooLarge;
    const SharedPlan p = plan_of(l.c, l.batch, a.n_groups, rows, waves);
    char* const w = (char*)workspace;
    const SharedWs ws = {(Group*)w, (Place*)(w + p.places), (int*)(w + p.group_of), (int64_t*)(w + p.per), p.pieces,
                         (float*)(w + p.partial)};
    hipLaunchKernelGGL(history_group_kernel, dim3(a.n_groups), dim3(kGroupThreads), 0, s, a, ws);
    hipLaunchKernelGGL((history_shared_kernel<D, PE, T>), dim3(runs_of(l.c.n_kv_heads, waves), l.c.n_kv_heads),
                       dim3(64 * waves), 0, s, a, ws, waves);
    const int chunks = (rows + 15) / 16 * l.c.n_kv_heads;
    const dim3 tails(l.batch, chunks);
    if ((int64_t)l.batch * chunks > kTailBlocks)
        hipLaunchKernelGGL((history_tail_kernel<D, PE, T, 1>), tails, dim3(64), 0, s, a, ws, waves);
    else
        hipLaunchKernelGGL((history_tail_kernel<D, PE, T, 4>), tails, dim3(256), 0, s, a, ws, waves);
    return hipGetLastError();
}
template <int D, int PE>
static hipError_t launch_d(const SharedArgs& a, int dtype, void* ws, hipStream_t s) {
    if (dtype == DLRM_DTYPE_F32) return launch_t<D, PE, float>(a, ws, s);
    if (dtype == DLRM_DTYPE_BF16) return launch_t<D, PE, bf16>(a, ws, s);
    return launch_t<D, PE, f16>(a, ws, s);
}
template <int PE>
static hipError_t launch_p(const SharedArgs& a, int dtype, void* ws, hipStream_t s) {
    if (a.l.c.head_dim == 32) return launch_d<32, PE>(a, dtype, ws, s);
    if (a.l.c.head_dim == 64) return launch_d<64, PE>(a, dtype, ws, s);
    return launch_d<128, PE>(a, dtype, ws, s);
}

hipError_t launch_history_lookup_shared(const SharedArgs& a, int dtype, void* ws, hipStream_t s) {
    if (a.l.c.page_events == 16) return launch_p<16>(a, dtype, ws, s);
    if (a.l.c.page_events == 32) return launch_p<32>(a, dtype, ws, s);
    return launch_p<64>(a, dtype, ws, s);
}

}  // namespace dlrm
