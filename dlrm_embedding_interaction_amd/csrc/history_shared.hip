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
// Windows and sinks of a group's histories end at different events, so in the tiles
// around these ends every row has a mask of its own.  The values there are the same for
// all rows, and a row that does not see an event must not meet its value if that is a
// NaN: in such tiles NaN codes are taken out of the product and given to the rows that
// see them by a product of their places.
//
// What bounds it, and what it reaches: 32 users' 16 beams over up to 32000 events, bf16, 32 / 8 heads of 128, 357 us, of
// which the page lists take 6, the shared tiles 299 and the tail 32 (shortest launches; one behind the other the clock falls,
// and they take 9, 422 and 42): 1.35 GB read once (4.5 TB/s), matrix instructions in 46% and vector instructions in 55% of
// the cycles.  64 users' 8 beams over up to 8000 events, 16 / 4 heads of 64, 67 us: 37 and the tail 15.  One row to a history
// and kv head, 1500 sessions: 98 us, where the decoding of tiles is the work (38, and 46 for the sessions' own).
#include "history_tile.h"

namespace dlrm {

// Rows' blocks of the tail have four waves up to here, which share the pieces of long histories, and one beyond, where waves
// of other blocks hide as much.  16 groups of 16, 4 kv heads of 32, fp32 (1024 blocks): four 34 us, one 44; of 64, bf16 49.5
// and 53; 32 groups of 16 (2048 blocks): four 50.7 and 63.2, one 44.3 and 56.4.  Heads of 128, whose waves fill their SIMDs
// sooner: one group of 256, 2 x 4 rows (1024 blocks), four 87 us, one 83; 16 groups of 16, 8 kv heads (2048 blocks), 104 and 97.
constexpr int tail_blocks(int dim) { return dim < 128 ? 1024 : 512; }
constexpr int kSharedWaves = 2048;       // waves of the shared tiles' kernel, where two are resident on each SIMD

// A group: its rows of the batch, the slot of one of its histories with events, and
// the tiles on the same pages in all of them that any of them sees: [0, lead) and
// [first, common), `count` in all.  As written, before the first page on which they
// differ is known: up to the last tile that all have whole.
struct Group {
    int begin, end, slot, lead, first, common, count, unused;
};
constexpr int kParts = 8;                  // blocks that compare the page lists of one group, at most (one of 256: a call of 100 us takes 90)
// Where the group stands in the row of all tiles: of its tiles, and of its pieces.
struct Place {
    int64_t tile, piece;
};

struct SharedWs {
    Group* groups;          // (n_groups)
    int* differs;           // (n_groups, parts): the first tile that a part found to differ
    Place* places;          // (n_groups)
    int* group_of;          // (batch)
    int64_t* per;           // tiles of a run
    int64_t pieces;         // that there is room for: as many as there can be while no two groups overlap
    float* partial;         // (pieces, kv heads, waves of a block, columns (head_dim + 2))
    int waves, cols;        // waves of a block, rows of a wave: 16 or 32
    int parts;
};

__device__ __forceinline__ Group group_at(const SharedWs& ws, int g) {
    Group r = ws.groups[g];
    int differs = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kParts; ++i) differs = min(differs, ws.differs[g * ws.parts + min(i, ws.parts - 1)]);
    r.common = min(r.common, differs);
    r.first = min(r.first, r.common);
    r.lead = min(r.lead, r.common);
    r.count = r.lead + r.common - r.first;
    return r;
}

// Blocks of (group, part of its histories): which tiles lie on the same pages in all of
// them.  Those without events see nothing and do not count.
constexpr int kGroupThreads = 1024;
__global__ __launch_bounds__(kGroupThreads) void history_group_kernel(SharedArgs a, SharedWs ws) {
    __shared__ int len_min, first_min, lead_max, differs, some;
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
        len_min = first_min = differs = 0x7fffffff;
        lead_max = 0;
        some = -1;
    }
    __syncthreads();
    for (int b = begin + tid; b < end; b += kGroupThreads) {
        if (blockIdx.y == 0) ws.group_of[b] = g;
        const Span s = span_of(l, b);
        if (!s.len) continue;
        atomicMin(&len_min, s.len);
        atomicMin(&first_min, s.first);
        atomicMax(&lead_max, s.lead);
        atomicMax(&some, b);
    }
    __syncthreads();
    Group r = {begin, end, 0, 0, 0, 0, 0, 0};
    if (some >= 0) {
        r.slot = l.slots ? l.slots[some] : some;
        const int pt = kTile / c.page_events;
        r.common = len_min / kTile;
        r.first = min(first_min, r.common);
        r.lead = min(lead_max, r.first);
        const int lead = r.lead * pt, first = r.first * pt;
        const int n = lead + r.common * pt - first;         // pages [0, lead) and [first, common pt)
        const int32_t* one = c.table + (int64_t)r.slot * c.max_pages;
        int least = 0x7fffffff;
        for (int b0 = begin + blockIdx.y; b0 < end; b0 += kGroupThreads * ws.parts) {
            const int here = min((end - b0 + ws.parts - 1) / ws.parts, kGroupThreads);
            __syncthreads();
            if (tid < here) {
                const int b = b0 + tid * ws.parts, slot = l.slots ? l.slots[b] : b;
                slot_of[tid] = slot >= 0 && slot < c.n_slots && c.lens[slot] > 0 ? slot : r.slot;
            }
            __syncthreads();
            // a wave for each history and 64 of its pages
            const int chunks = (n + 63) / 64, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll 4
            for (int w = wave; w < here * chunks; w += kGroupThreads / 64) {
                const int i = w / here * 64 + (tid & 63), x = i < lead ? i : first + i - lead;
                const int32_t* row = c.table + (int64_t)slot_of[w % here] * c.max_pages;
                if (i < n) least = row[x] != one[x] ? min(least, x / pt) : least;
            }
        }
        if (least < 0x7fffffff) atomicMin(&differs, least);
        __syncthreads();
    }
    if (tid == 0) {
        ws.differs[g * ws.parts + blockIdx.y] = differs;
        if (blockIdx.y == 0) ws.groups[g] = r;
    }
}

// ---- tiles for 32 rows -----------------------------------------------------------
//
// As in history_tile.h, but with the 32x32x16 instruction, so that codes are decoded
// once for 32 rows:
//   S^T = K Q^T   two products of 32 events each.  Row m of product t is event
//                 32 (m / 4 % 2) + 16 t + 4 (m / 8) + m % 4, so that half h of the wave
//                 ends up with the scores of events 32 h .. 32 h + 31, in order.
//   O^T += V^T P^T  four steps of 16 events, eight of each half.
// K's registers take the next tile as soon as the first product is done, each half of
// V's after its steps, so that one tile's registers are enough.
typedef float floatx16 __attribute__((ext_vector_type(16)));

template <int D>
struct Keys32 {
    u32x4 k[2][D / 32];
    float scale[2];
};
template <int D>
struct Values32 {
    u32x4 v[D / 32][2];
    float scale[2];
    bool in[2];
};

// A value that the whole wave reads, into scalar registers.
template <typename T>
__device__ __forceinline__ T read_scalar(const T* p, int64_t i) {
    return ((const __attribute__((address_space(4))) T*)p)[i];
}

// The pages that a lane reads of a tile, found a tile ahead of the codes, whose
// addresses would otherwise be waited for.  A shared tile lies whole within every
// list; an entry that is no page is only looked at when it is used, so that no load
// under way has to be waited for here.
template <int PE>
struct Pages32 {
    int k[2], v[2];
    __device__ __forceinline__ void find(const int32_t* table, int p0) {
        if constexpr (PE == 64) {
            k[0] = k[1] = v[0] = v[1] = read_scalar(table, p0);
            return;
        }
        const int lane = threadIdx.x & 63;
        asm("" : "+v"(p0));     // a lane's value: one that is the wave's would be waited for, to reach scalar registers
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            k[u] = table[p0 + (32 * (lane >> 2 & 1) + 16 * u) / PE];
            v[u] = table[p0 + (32 * (lane >> 5) + 16 * u) / PE];
        }
    }
};
__device__ __forceinline__ bool is_page(const dlrm_history_cache_t& c, int p) { return p >= 0 && p < c.n_pages; }

template <int D, int PE>
__device__ __forceinline__ void load_keys32(const dlrm_history_cache_t& c, const Pages32<PE>& p, int hk, Keys32<D>& t) {
    const int lane = threadIdx.x & 63, m = lane & 31, h = lane >> 5;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int e = 32 * (m >> 2 & 1) + 16 * u + 4 * (m >> 3) + (m & 3);
        const int64_t at = (int64_t)(is_page(c, p.k[u]) ? p.k[u] : 0) * c.n_kv_heads + hk;
        const uint8_t* k = c.k + (at * PE + e % PE) * D + h * 16;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) t.k[u][x] = *(const u32x4*)(k + 32 * x);
        t.scale[u] = c.k_scale[at];
    }
}
// Half u of them: the events that the second product's steps 2 u and 2 u + 1 take.
template <int D, int PE>
__device__ __forceinline__ void load_values32(const dlrm_history_cache_t& c, const Pages32<PE>& p, int hk, int u,
                                              Values32<D>& t) {
    const int lane = threadIdx.x & 63, m = lane & 31, h = lane >> 5;
    const int e = 32 * h + 16 * u;
    t.in[u] = is_page(c, p.v[u]);
    const int64_t at = (int64_t)(t.in[u] ? p.v[u] : 0) * c.n_kv_heads + hk;
    const uint8_t* v = c.v + (at * D + m) * PE + e % PE;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) t.v[j][u] = *(const u32x4*)(v + j * 32 * PE);
    t.scale[u] = c.v_scale[at];
}

// A tile as the waves of a block share it: every wave reads its part of the codes in
// whole lines and writes it to LDS.  The 16-byte chunks of a row stand in an order that
// follows from the row, so that the sixteen lanes that read at once meet every bank
// once.
template <int D, int PE, int WAVES>
struct Staged {
    static constexpr int CHUNKS = 64 * D / 16 / 64 / WAVES;      // of the keys, and of the values, per lane
    static constexpr int ROW = D / 16;                           // chunks of a key row; a value row has four
    static_assert(CHUNKS >= 1, "a tile has a chunk for every thread of the block");
    u32x4 k[CHUNKS], v[CHUNKS];
    // Place of a chunk within its row.
    __device__ __forceinline__ static int key_place(int row, int chunk) {
        return chunk ^ (ROW == 8 ? (row >> 1 & 3) | (row >> 5 & 1) << 2 : (ROW == 4 ? (row >> 2 & 1) | (row >> 5 & 1) << 1 : row >> 5 & 1));
    }
    __device__ __forceinline__ static int value_place(int d, int chunk) { return chunk ^ (d >> 2 & 3); }

    // A chunk's column of a value row, and so its page, is the same for all chunks of a lane.
    __device__ __forceinline__ static int value_event() { return 16 * value_place(threadIdx.x >> 2, threadIdx.x & 3); }
    // The page of each key chunk and of the value chunks.  A tile on one page: that page, in a scalar register, from
    // which the addresses follow without vector instructions.
    struct Pages {
        int k[PE == 64 ? 1 : CHUNKS], v;
        __device__ __forceinline__ void find(const int32_t* table, int p0) {
            if constexpr (PE == 64) {
                k[0] = v = read_scalar(table, p0);
            } else {
                asm("" : "+v"(p0));     // as in Pages32
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) k[i] = table[p0 + (i * 64 * WAVES + (int)threadIdx.x) / ROW / PE];
                v = table[p0 + value_event() / PE];
            }
        }
    };
    __device__ __forceinline__ void load(const dlrm_history_cache_t& c, const Pages& p, int hk) {
        const int64_t pv = (int64_t)(is_page(c, p.v) ? p.v : 0) * c.n_kv_heads + hk;
        const uint8_t* const vp = c.v + pv * D * PE;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int at = i * 64 * WAVES + threadIdx.x, row = at / ROW, d = at >> 2, pk = p.k[PE == 64 ? 0 : i];
            const uint8_t* const kp = c.k + ((int64_t)(is_page(c, pk) ? pk : 0) * c.n_kv_heads + hk) * D * PE;
            k[i] = *(const u32x4*)(kp + (unsigned)(row % PE * D + 16 * key_place(row, at % ROW)));
            v[i] = *(const u32x4*)(vp + (unsigned)(d * PE + value_event() % PE));
        }
    }
    __device__ __forceinline__ void store(u32x4* lds) const {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int at = i * 64 * WAVES + threadIdx.x;
            lds[at] = k[i];
            lds[4 * D + at] = v[i];
        }
    }
    __device__ __forceinline__ static void keys(const u32x4* lds, Keys32<D>& t) {
        const int lane = threadIdx.x & 63, m = lane & 31, h = lane >> 5;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int e = 32 * (m >> 2 & 1) + 16 * u + 4 * (m >> 3) + (m & 3);
#pragma unroll
            for (int x = 0; x < D / 32; ++x) t.k[u][x] = lds[e * ROW + key_place(e, 2 * x + h)];
        }
    }
    __device__ __forceinline__ static void values(const u32x4* lds, Values32<D>& t) {
        const int lane = threadIdx.x & 63, m = lane & 31, h = lane >> 5;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const int d = 32 * j + m;
                t.v[j][u] = lds[4 * D + 4 * d + value_place(d, 2 * h + u)];
            }
    }
};

// Bytes of a word that are the code of a NaN, as 0xff.
__device__ __forceinline__ unsigned nan_bytes(unsigned w) {
    return (((w & 0x7f7f7f7fu) + 0x01010101u) >> 7 & 0x01010101u) * 0xffu;
}
// Four bytes of 0xff or 0 as four bf16 of 1 or 0, in two words.
__device__ __forceinline__ u32x2 ones_of(unsigned b) {
    return u32x2{(b & 1u) * 0x3f80u | (b >> 8 & 1u) * 0x3f800000u, (b >> 16 & 1u) * 0x3f80u | (b >> 24 & 1u) * 0x3f800000u};
}
// Eight bits as eight bf16 of 1 or 0.
__device__ __forceinline__ bf16x8 ones_of_bits(unsigned b) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (b >> (2 * i) & 1u) * 0x3f80u | (b >> (2 * i + 1) & 1u) * 0x3f800000u;
    return __builtin_bit_cast(bf16x8, w);
}

// ---- the shared tiles --------------------------------------------------------------

// Blocks that the group's rows make, each taking so many of them.
__device__ __forceinline__ int64_t blocks_of(const Group& g, int rows, int taken) {
    return ((int64_t)(g.end - g.begin) * rows + taken - 1) / taken;
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

// What a row sees of the tile at e0.
struct Sight {
    int low, lead;                       // events from low on and those below lead; the lane's row's
    int low_max, lead_min;               // over the rows that read the tiles together
    // Of tiles in rising order, those before number `from` and from number `to` on are seen whole by all rows.
    __device__ __forceinline__ void edges(const Group& r, int* from, int* to) const {
        auto before = [&](int tile) { return tile < r.first ? min(tile, r.lead) : r.lead + tile - r.first; };
        *to = before(low_max / kTile + (low_max % kTile != 0));
        *from = min(before(lead_min / kTile), *to);
    }
    __device__ __forceinline__ void agree() {
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            low_max = max(low_max, __shfl_xor(low_max, d, 64));
            lead_min = min(lead_min, __shfl_xor(lead_min, d, 64));
        }
        low_max = __builtin_amdgcn_readfirstlane(low_max);
        lead_min = __builtin_amdgcn_readfirstlane(lead_min);
    }
    template <int N>
    __device__ __forceinline__ unsigned seen(int e) const {
        unsigned s = 0;
#pragma unroll
        for (int x = 0; x < N; ++x) s |= e + x >= low || e + x < lead ? 1u << x : 0u;
        return s;
    }
};

// Sixteen rows of a group over a run of its tiles.
template <int D, int PE, typename T>
struct Rows16 {
    static constexpr int COLS = 16;
    bf16x8 q[D / 32][Parts<T>::q];
    floatx4 o[D / 16];
    float m = -INFINITY, sum = 0.f;

    __device__ __forceinline__ static int column() { return threadIdx.x & 15; }
    __device__ __forceinline__ void start(const T* qp, float scale, int wide) {
        load_query<D>(qp, scale, wide, (threadIdx.x & 63) >> 4, q);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[j] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    // Some rows do not see some events: masked, NaN values apart.
    __device__ __forceinline__ void use_masked(Tile<D>& t, float c, int e0, const Sight& at) {
        const int g = (threadIdx.x & 63) >> 4;
        unsigned nan = 0;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) nan |= nan_bytes(t.v[j][x]);
        if (__any(t.vin && nan)) {
            const unsigned seen = t.vin ? at.seen<16>(e0 + 16 * g) : 0u;
            const bf16x8 see[2] = {ones_of_bits(seen & 0xffu), ones_of_bits(seen >> 8)};
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                floatx4 n = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const unsigned b0 = nan_bytes(t.v[j][2 * h]), b1 = nan_bytes(t.v[j][2 * h + 1]);
                    const u32x2 w0 = ones_of(b0), w1 = ones_of(b1);
                    const u32x4 w = {w0[0], w0[1], w1[0], w1[1]};
                    n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), see[h], n, 0, 0, 0);
                    t.v[j][2 * h] &= ~b0;
                    t.v[j][2 * h + 1] &= ~b1;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][i] += n[i] > 0.f ? NAN : 0.f;
            }
        }
        use_tile<D, T, true>(t, q, c, e0, false, at.low, at.lead, 0x7fffffff, g, o, m, sum);
    }
    __device__ __forceinline__ void run(const dlrm_history_cache_t& c, const int32_t* table, const Group& r, int hk,
                                        float scale, const Sight& at, int i0, int i1) {
        constexpr bool TURNS = D < 128 || Parts<T>::q == 1;
        const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
        auto tile_of = [&](int i) { return i < r.lead ? i : r.first + (i - r.lead); };
        auto load = [&](int i, Tile<D>& t) { load_tile<D, PE>(c, table, tile_of(i) * (kTile / PE), hk, n, g, t); };
        auto use = [&](Tile<D>& t) { use_tile<D, T>(t, q, scale, 0, true, 0, 0, kTile, g, o, m, sum); };
        int from, to;
        at.edges(r, &from, &to);
        Tile<D> cur, nxt;
        for (int i = max(i0, from); i < min(i1, to); ++i) {
            load(i, cur);
            use_masked(cur, scale, tile_of(i) * kTile, at);
        }
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const int stop = part ? i1 : min(i1, from);
            int i = part ? max(i0, to) : i0;
            if (i < stop) load(i, cur);
            for (; i < stop; ++i) {
                if (i + 1 < stop) load(i + 1, nxt);
                use(cur);
                if constexpr (TURNS) {
                    if (++i >= stop) break;
                    if (i + 1 < stop) load(i + 1, cur);
                    use(nxt);
                } else {
                    cur = nxt;
                }
            }
        }
    }
    // The weighted sums by column, then the maxima in powers of two, then the weights' sums.
    __device__ __forceinline__ void leave(float* part, float c) {
        const int n = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
        sum += swizzle_xor16(sum);
        sum += __shfl_xor(sum, 32, 64);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) *(floatx4*)(part + n * D + 16 * j + 4 * g) = o[j];
        if (g == 0) {
            part[16 * D + n] = m * c;
            part[16 * D + 16 + n] = sum;
        }
    }
};

template <int D, int PE, typename T>
struct Rows32 {
    static constexpr int COLS = 32, NQ = Parts<T>::q, NP = Parts<T>::p;
    bf16x8 q[D / 16][NQ];
    floatx16 o[D / 32];
    float m = -INFINITY, sum = 0.f;

    __device__ __forceinline__ static int column() { return threadIdx.x & 31; }
    __device__ __forceinline__ void start(const T* qp, float scale, int wide) {
        const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            const int d0 = (s >> 1) * 32 + h * 16 + (s & 1) * 8;
            const Raw<T> raw = wide ? load_raw<true>(qp + d0) : load_raw<false>(qp + d0);
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = scale < 0.f ? -(float)raw.x[i] : (float)raw.x[i];
            split8<NQ>(x, q[s]);
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[j][i] = 0.f;
    }
    // Products that follow one another add to different sums: one that adds to the last one's result waits for it.
    __device__ __forceinline__ void scores(const Keys32<D>& k, floatx16 (&s)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int x = 0; x < 16; ++x) s[u][x] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            bf16x8 kk[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) kk[u] = decode8(k.k[u][x / 2][x % 2 * 2], k.k[u][x / 2][x % 2 * 2 + 1], k.scale[u]);
#pragma unroll
            for (int y = 0; y < NQ; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kk[u], q[x][y], s[u], 0, 0, 0);
        }
    }
    // The running maximum, which may lag by 2^kLag, each row's for itself, so that the sums are rescaled in few tiles;
    // what the exponents are taken against.  Weights stay below 1, as against the maximum itself.
    static constexpr float kLag = 8.f;
    __device__ __forceinline__ float raise(const floatx16 (&s)[2], float scale) {
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < 32; ++x) top = fmaxf(top, s[x >> 4][x & 15]);
        const unsigned bits = __float_as_uint(top);
        const auto both = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
        top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1]));
        const bool up = (top - m) * scale > kLag;
        if (__any(up)) {
            const float mx = up ? top : m;
            const float alpha = up ? __builtin_amdgcn_exp2f((m - mx) * scale) : 1.f;
            sum *= alpha;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) o[j] *= alpha;
            m = mx;
        }
        return m == -INFINITY ? 0.f : m * scale + kLag;
    }
    // The second product's steps 2 half and 2 half + 1.
    __device__ __forceinline__ void weigh(const floatx16 (&s)[2], const Values32<D>& v, float scale, float mc, int half) {
#pragma unroll
        for (int u = 2 * half; u < 2 * half + 2; ++u) {
            float p[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                p[x] = __builtin_amdgcn_exp2f(fmaf(s[half][8 * (u & 1) + x], scale, -mc));
                sum += p[x];
            }
            bf16x8 pp[NP];
            split8<NP>(p, pp);
            bf16x8 vv[D / 32];
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                vv[j] = decode8(v.v[j][half][u % 2 * 2], v.v[j][half][u % 2 * 2 + 1], v.scale[half]);
#pragma unroll
            for (int y = 0; y < NP; ++y)
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vv[j], pp[y], o[j], 0, 0, 0);
        }
    }
    __device__ __forceinline__ void run(const dlrm_history_cache_t& c, const int32_t* table, const Group& r, int hk,
                                        float scale, const Sight& at, int i0, int i1) {
        constexpr int PT = kTile / PE;
        auto tile_of = [&](int i) { return i < r.lead ? i : r.first + (i - r.lead); };
        int from, to;
        at.edges(r, &from, &to);
        run_masked(c, table, r, hk, scale, at, max(i0, from), min(i1, to));
        Pages32<PE> page;
        Keys32<D> k;
        Values32<D> v;
        floatx16 s[2];
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const int stop = part ? i1 : min(i1, from);
            int i = part ? max(i0, to) : i0;
            if (i >= stop) continue;
            page.find(table, tile_of(i) * PT);
            load_keys32<D, PE>(c, page, hk, k);
            load_values32<D, PE>(c, page, hk, 0, v);
            load_values32<D, PE>(c, page, hk, 1, v);
            page.find(table, tile_of(min(i + 1, stop - 1)) * PT);
            for (; i < stop; ++i) {
                Pages32<PE> later;
                later.find(table, tile_of(min(i + 2, stop - 1)) * PT);
                scores(k, s);
                load_keys32<D, PE>(c, page, hk, k);
                if (__builtin_expect(__any(!v.in[0] || !v.in[1]), 0)) mask(s, v, ~0u, false);
                const float mc = raise(s, scale);
                weigh(s, v, scale, mc, 0);
                load_values32<D, PE>(c, page, hk, 0, v);
                weigh(s, v, scale, mc, 1);
                load_values32<D, PE>(c, page, hk, 1, v);
                page = later;
            }
        }
    }
    __device__ __forceinline__ void run_masked(const dlrm_history_cache_t& c, const int32_t* table, const Group& r, int hk,
                                               float scale, const Sight& at, int i0, int i1) {
        const int h = (threadIdx.x & 63) >> 5;
        Pages32<PE> page;
        Keys32<D> k;
        Values32<D> v;
        floatx16 s[2];
        for (int i = i0; i < i1; ++i) {
            const int tile = i < r.lead ? i : r.first + (i - r.lead);
            page.find(table, tile * (kTile / PE));
            load_keys32<D, PE>(c, page, hk, k);
            load_values32<D, PE>(c, page, hk, 0, v);
            load_values32<D, PE>(c, page, hk, 1, v);
            scores(k, s);
            mask(s, v, at.seen<32>(tile * kTile + 32 * h), true);
            const float mc = raise(s, scale);
            weigh(s, v, scale, mc, 0);
            weigh(s, v, scale, mc, 1);
        }
    }
    // The scales of the lane's pages, and whether they are there.
    struct Scales {
        float k[2], v[2];
        bool in[2];
        __device__ __forceinline__ void load(const dlrm_history_cache_t& c, const Pages32<PE>& p, int hk) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (PE == 64 && u) {
                    k[u] = k[0], v[u] = v[0], in[u] = in[0];
                    break;
                }
                in[u] = is_page(c, p.v[u]);
                const int64_t ik = (int64_t)(is_page(c, p.k[u]) ? p.k[u] : 0) * c.n_kv_heads + hk;
                const int64_t iv = (int64_t)(in[u] ? p.v[u] : 0) * c.n_kv_heads + hk;
                k[u] = PE == 64 ? read_scalar(c.k_scale, ik) : c.k_scale[ik];
                v[u] = PE == 64 ? read_scalar(c.v_scale, iv) : c.v_scale[iv];
            }
        }
    };
    // All waves of a block over the same tiles, through LDS: while one tile is used the next one is read into
    // registers.  `live`: the wave has rows; `lds`: two tiles.
    template <int WAVES>
    __device__ __forceinline__ void run_staged(const dlrm_history_cache_t& c, const int32_t* table, const Group& r, int hk,
                                               float scale, const Sight& at, int i0, int i1, bool live, u32x4* lds) {
        constexpr int PT = kTile / PE;
        typedef Staged<D, PE, WAVES> S;
        auto tile_of = [&](int i) { return i < r.lead ? i : r.first + (i - r.lead); };
        int from, to;
        at.edges(r, &from, &to);
        if (live) run_masked(c, table, r, hk, scale, at, max(i0, from), min(i1, to));
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const int stop = part ? i1 : min(i1, from);
            int i = part ? max(i0, to) : i0;
            if (i >= stop) continue;
            S staged;
            typename S::Pages page;
            Pages32<PE> mine;
            Scales now, next;
            page.find(table, tile_of(i) * PT);
            mine.find(table, tile_of(i) * PT);
            staged.load(c, page, hk);
            now.load(c, mine, hk);
            page.find(table, tile_of(min(i + 1, stop - 1)) * PT);
            mine.find(table, tile_of(min(i + 1, stop - 1)) * PT);
            __syncthreads();                // the tiles before may still be in use
            staged.store(lds);
            __syncthreads();
            for (int which = 0; i < stop; ++i, which ^= 1) {
                const u32x4* tile = lds + which * (8 * D);
                staged.load(c, page, hk);
                next.load(c, mine, hk);
                page.find(table, tile_of(min(i + 2, stop - 1)) * PT);
                mine.find(table, tile_of(min(i + 2, stop - 1)) * PT);
                if (live) {
                    Keys32<D> k;
                    Values32<D> v;
                    floatx16 s[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) k.scale[u] = now.k[u], v.scale[u] = now.v[u], v.in[u] = now.in[u];
                    S::keys(tile, k);
                    scores(k, s);
                    S::values(tile, v);
                    if (__builtin_expect(__any(!v.in[0] || !v.in[1]), 0)) mask(s, v, ~0u, false);
                    const float mc = raise(s, scale);
                    weigh(s, v, scale, mc, 0);
                    weigh(s, v, scale, mc, 1);
                }
                staged.store(lds + (which ^ 1) * (8 * D));
                now = next;
                __syncthreads();
            }
        }
    }
    // Leaves out the events that a row does not see and those of pages that are not there; `apart`: NaN values leave
    // the product for the rows that see them.
    __device__ __forceinline__ void mask(floatx16 (&s)[2], Values32<D>& v, unsigned seen, bool apart) {
        seen &= (v.in[0] ? 0xffffu : 0u) | (v.in[1] ? 0xffff0000u : 0u);
#pragma unroll
        for (int x = 0; x < 32; ++x)
            if (!(seen >> x & 1)) s[x >> 4][x & 15] = -INFINITY;
        unsigned nan = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            v.scale[u] = v.in[u] ? v.scale[u] : 1.f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    v.v[j][u][x] = v.in[u] ? v.v[j][u][x] : 0u;
                    nan |= nan_bytes(v.v[j][u][x]);
                }
        }
        if (!apart || !__any(nan)) return;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            floatx16 n;
#pragma unroll
            for (int x = 0; x < 16; ++x) n[x] = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const unsigned b0 = nan_bytes(v.v[j][u >> 1][u % 2 * 2]), b1 = nan_bytes(v.v[j][u >> 1][u % 2 * 2 + 1]);
                const u32x2 a0 = ones_of(b0), a1 = ones_of(b1);
                const u32x4 w = {a0[0], a0[1], a1[0], a1[1]};
                n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w),
                                                            ones_of_bits(seen >> (8 * u) & 0xffu), n, 0, 0, 0);
                v.v[j][u >> 1][u % 2 * 2] &= ~b0;
                v.v[j][u >> 1][u % 2 * 2 + 1] &= ~b1;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) o[j][x] += n[x] > 0.f ? NAN : 0.f;
        }
    }
    __device__ __forceinline__ void leave(float* part, float c) {
        const int n = threadIdx.x & 31, h = (threadIdx.x & 63) >> 5;
        sum += __shfl_xor(sum, 32, 64);
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int a = 0; a < 4; ++a)
                *(floatx4*)(part + n * D + 32 * j + 8 * a + 4 * h) =
                    floatx4{o[j][4 * a], o[j][4 * a + 1], o[j][4 * a + 2], o[j][4 * a + 3]};
        if (h == 0) {
            part[32 * D + n] = m * c + kLag;
            part[32 * D + 32 + n] = sum;
        }
    }
};

// Waves on a SIMD.  With 32 rows, heads of 128 pass 256 registers: in fp32, whose scores take three products, and in fp16
// (two) with up to two waves to a block, what is moved to memory costs more than a second wave gives.  Whole calls with two
// waves on a SIMD and with one (and half the runs, see launch_t), 8 kv heads, 3000 events: 32 groups of 16 x 4 rows, fp32 176
// and 125 us, fp16 129 and 95; 16 groups of 64 x 4 rows, whose blocks have four waves, fp32 217 and 190, fp16 148 and 148,
// bf16 122 and 138.  bf16 with fewer waves to a block would gain, too (102 and 86), and is left at two.
template <int D, typename T>
constexpr int resident(int cols, int waves) {
    return D == 128 && cols == 32 && (Parts<T>::q == 3 || (Parts<T>::q == 2 && waves < 4)) ? 1 : 2;
}

// WAVES to a block; where there are more than one they share the tiles.
template <int D, int PE, typename T, template <int, int, typename> class Rows, int WAVES>
__global__ __launch_bounds__(64 * WAVES, (resident<D, T>(Rows<D, PE, T>::COLS, WAVES)))
void history_shared_kernel(SharedArgs a, SharedWs ws) {
    typedef Rows<D, PE, T> R;
    __shared__ u32x4 lds[WAVES > 1 ? 2 * 8 * D : 1];
    const LookupArgs& l = a.l;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), hk = blockIdx.y;
    const int heads = l.n_heads / l.c.n_kv_heads, rows = l.queries * heads, taken = R::COLS * WAVES;

    // tiles and pieces before each lane's share of the groups
    const int each = (a.n_groups + 63) / 64;
    const int lo = lane * each, hi = lo + each < a.n_groups ? lo + each : a.n_groups;
    int64_t tiles = 0, pieces = 0;
    for (int i = lo; i < hi; ++i) {
        const Group r = group_at(ws, i);
        const int64_t blocks = blocks_of(r, rows, taken);
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
        const Group r = group_at(ws, gi);
        const int64_t blocks = blocks_of(r, rows, taken);
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
        const int64_t chunk = block * WAVES + wave, first = chunk * R::COLS;
        const int64_t all = (int64_t)(r.end - r.begin) * rows, place = piece + block + blockIdx.x;
        if (place >= ws.pieces) continue;
        const bool any = first < all;
        if (WAVES == 1 && !any) continue;

        // the lane's column: a row of one of the group's histories
        const int64_t row = any ? (first + R::column() < all ? first + R::column() : first) : 0;
        const int b = r.begin + (int)(row / rows), y = (int)(row % rows);
        const Span sp = span_of(l, b);
        Sight sight;
        sight.low = sp.low;                 // a history without events: as if it saw everything, and not read later
        sight.lead = sp.low ? sp.lead_events : 0x7fffffff;
        sight.low_max = sight.low, sight.lead_min = sight.lead;
        R sums;
        sums.start((const T*)l.q + ((int64_t)b * l.queries + y / heads) * l.ld_q + (int64_t)(hk * heads + y % heads) * D,
                   l.scale, l.wide);
        const int32_t* table = l.c.table + (int64_t)r.slot * l.c.max_pages;
        float* const part = ws.partial + ((place * gridDim.y + hk) * WAVES + wave) * (R::COLS * (D + 2));
        if constexpr (WAVES == 1) {
            sight.agree();
            sums.run(l.c, table, r, hk, c, sight, i0, i1);
        } else {
            __shared__ int low_max, lead_min;   // the same tiles are masked in all waves of the block
            __syncthreads();
            if (threadIdx.x == 0) low_max = 0, lead_min = 0x7fffffff;
            __syncthreads();
            sight.agree();
            if (lane == 0 && any) {
                atomicMax(&low_max, sight.low_max);
                atomicMin(&lead_min, sight.lead_min);
            }
            __syncthreads();
            sight.low_max = __builtin_amdgcn_readfirstlane(low_max);
            sight.lead_min = __builtin_amdgcn_readfirstlane(lead_min);
            sums.template run_staged<WAVES>(l.c, table, r, hk, c, sight, i0, i1, any, lds);
        }
        if (any) sums.leave(part, c);
    }
}

// A block per (history, kv head, chunk of its rows): the tiles that are its own, and the join.
template <int D, int PE, typename T, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void history_tail_kernel(SharedArgs a, SharedWs ws) {
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

    const int gi = a.groups ? ws.group_of[b] : b / (l.batch / a.n_groups);
    Group r = {0, 0, 0, 0, 0, 0, 0, 0};
    Place place_of = {0, 0};
    const int64_t per = *ws.per;
    if (gi >= 0 && gi < a.n_groups) {
        r = group_at(ws, gi);
        place_of = ws.places[gi];           // not written where nothing is shared
    }
    if (b < r.begin || b >= r.end || !sp.len) r.common = r.count = 0;
    // the history's tiles behind the shared ones
    auto tile_of = [&](int i) { return i < sp.lead ? i : sp.first + (i - sp.lead); };
    const int end = (sp.len + kTile - 1) / kTile;
    const int shared = min(sp.lead, r.common) + max(min(end, r.common) - sp.first, 0), own = shared + wave;

    floatx4 o[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[j] = floatx4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, sum = 0.f;
    if (own < sp.count) {
        bf16x8 q[D / 32][NQ];
        const int yy = live ? y : 0;
        load_query<D>((const T*)l.q + ((int64_t)b * l.queries + yy / heads) * l.ld_q + (int64_t)(hk * heads + yy % heads) * D,
                      l.scale, l.wide, g, q);
        const int slot = l.slots ? l.slots[b] : b;
        const int32_t* table = l.c.table + (int64_t)slot * l.c.max_pages;
        const float c = exponent_scale(l.scale);
        // One wave to a block: without a second tile's registers 64 instead of 80 (heads of 64) and eight waves a SIMD, which
        // hide more (1500 sessions' own tiles 53 -> 46 us; with the pieces' reads before the tiles, too, 65).
        Tile<D> cur, nxt;
        if (WAVES > 1) load_tile<D, PE>(l.c, table, tile_of(own) * PT, hk, n, g, cur);
        for (int i = own; i < sp.count; i += WAVES) {
            if (WAVES == 1) load_tile<D, PE>(l.c, table, tile_of(i) * PT, hk, n, g, cur);
            else if (i + WAVES < sp.count) load_tile<D, PE>(l.c, table, tile_of(i + WAVES) * PT, hk, n, g, nxt);
            const int e0 = tile_of(i) * kTile;
            const bool whole = (e0 >= sp.low || e0 + kTile <= sp.lead_events) && e0 + kTile <= sp.len;
            use_tile<D, T>(cur, q, c, e0, whole, sp.low, sp.lead_events, sp.len, g, o, m, sum);
            if (WAVES > 1) cur = nxt;
        }
        m *= c;                                          // from here on in powers of two
        sum += swizzle_xor16(sum);
        sum += __shfl_xor(sum, 32, 64);
    }
    if (r.count) {
        const int64_t row = (int64_t)(b - r.begin) * rows + (live ? y : 0);
        const int64_t chunk = row >> (ws.cols == 32 ? 5 : 4), block = chunk >> (ws.waves >> 1);     // of 16 or 32; 1, 2 or 4
        const int64_t t0 = place_of.tile + block * r.count, run0 = t0 / per, run1 = (t0 + r.count - 1) / per;
        const int col = (int)row & (ws.cols - 1);
        // two pieces at a time, all of their reads on the way together
        for (int64_t i0 = run0 + wave; __any(i0 <= run1); i0 += 2 * WAVES) {
            float pm[2], ps[2];
            bool in[2];
            floatx4 po[2][D / 16];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t place = place_of.piece + block + i0 + u * WAVES;
                in[u] = i0 + u * WAVES <= run1 && place >= 0 && place < ws.pieces;
                const float* part = ws.partial +
                                    (((in[u] ? place : 0) * l.c.n_kv_heads + hk) * ws.waves + (chunk & (ws.waves - 1))) * (ws.cols * (D + 2));
                pm[u] = part[ws.cols * D + col];
                ps[u] = part[ws.cols * D + ws.cols + col];
#pragma unroll
                for (int j = 0; j < D / 16; ++j) po[u][j] = *(const floatx4*)(part + col * D + 16 * j + 4 * g);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (!in[u]) continue;
                // A maximum of -inf is that of a piece without a number among its scores, too: its sums are NaN, and a
                // factor of 0 keeps them so.
                const float mx = fmaxf(m, pm[u]), to = mx == -INFINITY ? 0.f : mx;
                const float f0 = __builtin_amdgcn_exp2f(m - to), f1 = __builtin_amdgcn_exp2f(pm[u] - to);
                m = mx;
                sum = sum * f0 + ps[u] * f1;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) o[j] = o[j] * f0 + po[u][j] * f1;
            }
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

// Rows that a wave takes, and the waves of a block: as many as a group's rows need on average, up to four (heads of 32:
// two, whose tiles have a chunk for each thread of no more).  32 rows where 16 would not hold a group's: 16 groups of 256
// rows, heads of 128, 3000 events, bf16 117 us, in 16 rows 194; 32 groups of 32 rows 63 and 64.  Tiles shared by two waves
// instead of read by each (32 groups of 64 rows, 32000 events, bf16): 430 -> 372 us.
struct Shape {
    int cols, waves;
};
static Shape shape_of(int dim, int64_t batch, int64_t n_groups, int rows) {
    const int64_t mean = (batch + n_groups - 1) / n_groups * rows;
    Shape s;
    s.cols = mean > 16 ? 32 : 16;
    const int64_t chunks = (mean + s.cols - 1) / s.cols;
    s.waves = chunks > 2 && dim > 32 ? 4 : (chunks > 1 ? 2 : 1);
    return s;
}
static int runs_of(int n_kv_heads, int waves) {
    const int n = kSharedWaves / (n_kv_heads * waves);
    return n < 1 ? 1 : n;
}

static size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Where the parts of the workspace begin.
struct SharedPlan {
    size_t differs, places, group_of, per, partial, end;
    int64_t pieces;
};
static SharedPlan plan_of(const dlrm_history_cache_t& c, int64_t batch, int64_t n_groups, int rows, Shape shape) {
    SharedPlan p;
    p.differs = round256(n_groups * sizeof(Group));
    p.places = p.differs + round256(n_groups * kParts * sizeof(int));
    p.group_of = p.places + round256(n_groups * sizeof(Place));
    p.per = p.group_of + round256(batch * sizeof(int));
    p.partial = p.per + 256;
    p.pieces = runs_of(c.n_kv_heads, shape.waves) + batch * rows / (shape.cols * shape.waves) + n_groups;
    p.end = p.partial +
            (size_t)p.pieces * c.n_kv_heads * shape.waves * shape.cols * (c.head_dim + 2) * sizeof(float);
    return p;
}

size_t shared_workspace_bytes(const dlrm_history_cache_t& c, int64_t batch, int64_t n_groups, int queries, int n_heads) {
    const int rows = queries * (n_heads / c.n_kv_heads);
    const size_t shared = plan_of(c, batch, n_groups, rows, shape_of(c.head_dim, batch, n_groups, rows)).end;
    const size_t single = lookup_workspace_bytes(c, batch, queries, n_heads);
    return shared > single ? shared : single;
}

template <int D, int PE, typename T>
static hipError_t launch_t(const SharedArgs& a, void* workspace, hipStream_t s) {
    const LookupArgs& l = a.l;
    const int rows = l.queries * (l.n_heads / l.c.n_kv_heads);
    const Shape shape = shape_of(D, l.batch, a.n_groups, rows);
    const SharedPlan p = plan_of(l.c, l.batch, a.n_groups, rows, shape);
    char* const w = (char*)workspace;
    // enough blocks for every CU
    const int parts = a.n_groups <= 256 / kParts ? kParts : (a.n_groups < 256 ? 256 / a.n_groups : 1);
    const SharedWs ws = {(Group*)w, (int*)(w + p.differs), (Place*)(w + p.places), (int*)(w + p.group_of),
                         (int64_t*)(w + p.per), p.pieces, (float*)(w + p.partial), shape.waves, shape.cols, parts};
    hipLaunchKernelGGL(history_group_kernel, dim3(a.n_groups, parts), dim3(kGroupThreads), 0, s, a, ws);
    // runs that are all resident at once: 32 groups of 8 x 4 rows, fp32 heads of 128, 1024 waves 60 us, 2048 70
    const int all = runs_of(l.c.n_kv_heads, shape.waves), runs = resident<D, T>(shape.cols, shape.waves) == 1 ? (all + 1) / 2 : all;
    const dim3 grid(runs, l.c.n_kv_heads), block(64 * shape.waves);
    if (shape.cols == 16) hipLaunchKernelGGL((history_shared_kernel<D, PE, T, Rows16, 1>), grid, block, 0, s, a, ws);
    else if (shape.waves == 1) hipLaunchKernelGGL((history_shared_kernel<D, PE, T, Rows32, 1>), grid, block, 0, s, a, ws);
    else if (shape.waves == 2) hipLaunchKernelGGL((history_shared_kernel<D, PE, T, Rows32, 2>), grid, block, 0, s, a, ws);
    else if constexpr (D > 32)
        hipLaunchKernelGGL((history_shared_kernel<D, PE, T, Rows32, 4>), grid, block, 0, s, a, ws);
    const int chunks = (rows + 15) / 16 * l.c.n_kv_heads;
    const dim3 tails(l.batch, chunks);
    if ((int64_t)l.batch * chunks > tail_blocks(D))
        hipLaunchKernelGGL((history_tail_kernel<D, PE, T, 1>), tails, dim3(64), 0, s, a, ws);
    else
        hipLaunchKernelGGL((history_tail_kernel<D, PE, T, 4>), tails, dim3(256), 0, s, a, ws);
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

// Whether the groups' histories are looked up one by one: three kernels take 11 to 20 us before they save anything.
// Tiles of all rows' chunks, one by one against shared: 4 kv heads of 32, fp32, 32 groups of 16, 16384 (500 events) 16
// us to 23, 32768 (1000) 29 to 27, 65536 51 to 31; 8 of 128, bf16, 32 groups of 4, 16384 36 to 40, 32768 63 to 44; 4 groups
// of 64, 32768 53 to 53.  Histories of few tiles have most of them to themselves: 32 groups of 64, 8 of 128, up to 204
// events (4 tiles) 83 to 115, up to 504 (8) 154 to 133.
static bool one_by_one(const LookupArgs& l) {
    const int64_t tiles = most_tiles(l), rows = (int64_t)l.queries * (l.n_heads / l.c.n_kv_heads);
    return tiles <= 5 || l.batch * tiles * l.c.n_kv_heads * ((rows + 15) / 16) <= 24576;
}

hipError_t launch_history_lookup_shared(const SharedArgs& a, int dtype, void* ws, hipStream_t s) {
    if (!grid_fits(a.l.batch, 256) || !grid_fits(a.n_groups, kGroupThreads)) return kTooLarge;
    if (one_by_one(a.l)) {
        LookupArgs l = a.l;
        l.partial = (float*)ws;
        return launch_history_lookup(l, dtype, s);
    }
    if (a.l.c.page_events == 16) return launch_p<16>(a, dtype, ws, s);
    if (a.l.c.page_events == 32) return launch_p<32>(a, dtype, ws, s);
    return launch_p<64>(a, dtype, ws, s);
}

}  // namespace dlrm
