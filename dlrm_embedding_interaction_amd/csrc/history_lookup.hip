// history_lookup.hip -- attention of single queries over the 8-bit paged cache.
//
// The queries of history b stand at its last position len - 1 and see event j
// iff j >= len - window or j < sinks.  Keys and values are e4m3 codes times the
// power-of-two scale of their page and head: exact in bf16.
//
// What bounds it is reading the codes, 2 head_dim bytes per visible event and kv
// head, so the work is split over waves that never wait for one another.  The
// visible events of all histories make one row of 64-event tiles, and each wave
// takes an equal, contiguous run of it, whatever the lengths are.  Only the first
// and the last history of a run can be cut; their maximum, sum and weighted sum
// go to the workspace and a second kernel joins them.
//
// One tile in one wave, products on the matrix cores (16x16x32, bf16), with the
// query rows of the kv head (queries x heads per kv head, in chunks of 16) as the
// columns of both products:
//   S^T = K Q^T   four products of 16 events each.  Row m of product t is event
//                 16 (m / 4) + 4 t + m % 4, so that lane group g = lane / 16 ends
//                 up with the scores of events 16 g .. 16 g + 15, in order.
//   O^T += V^T P^T  the sum runs over the events each lane group holds: P^T is the
//                 lane's own scores, V^T sixteen consecutive bytes of the
//                 event-minor value page.
// K, V and P go from memory or registers straight into the products; nothing
// passes through LDS.  Products of the query's 8-bit-mantissa parts (bf16: one
// part, fp16: two, fp32: three, no bit lost) with the codes are exact; the sums
// are fp32.  The weights are kept in two bf16 parts (fp32 queries: three), since
// rounding them to one would add an error as large as the output's own rounding.
//
// Measured on MI355X: 128 histories of up to 32000 events, 8 kv heads of 128, 32
// query heads, bf16: 812 us, 5.8 TB/s of codes, 93% of what a plain read stream
// reaches (6.28 TB/s).  256 histories, window 1024, 4 kv heads of 64: 32 us, 4.0
// TB/s; there the dependent reads length -> page -> codes and the ~300 vector
// instructions a tile (decoding, exponentials, splitting) show.
#include "history_tile.h"

namespace dlrm {

constexpr int kLookupWaves = 2048;       // waves a launch aims at: two on each SIMD
// Histories of at most this many tiles have a block of their own: no second kernel, but the longest history sets the
// time.  The table's room counts, which the host knows, not what is held.  Measured on ragged histories, blocks against
// runs: 96 of up to 24 tiles (4 heads of 64) 16.1 us to 18.8, of up to 32 19.6 to 21.4, of up to 48 26.1 to 25.5; 256 (16
// heads on 4) of up to 24 28.5 to 31.0, of up to 40 42.9 to 43.0, of up to 64 81 to 73.  Where eight waves share a block
// the longest costs less: 64 of up to 40 tiles 15.9 to 20.8, eight of up to 48 12.4 to 13.1, of up to 64 15.2 to 14.3;
// 64 of up to 64 would still be faster in blocks, 21.3 to 24.6, and of up to 96, 28.6 to 31.3.
constexpr int kDirectTiles = 32, kDirectTiles8 = 48;

// Two waves per SIMD: all fits but in the runs of fp32 heads of 128, which keep 12 to 20 bytes a lane in scratch.
// DIRECT waves: one block of so many per (history, chunk of rows), its waves taking
// every DIRECT-th tile and joining their results through LDS.  0: runs of tiles.
template <int D, int PE, typename T, int DIRECT>
__global__ __launch_bounds__(DIRECT ? 64 * DIRECT : 256, 2) void history_lookup_kernel(LookupArgs a, int n_waves, int* __restrict__ meta) {
    constexpr int NQ = Parts<T>::q;
    constexpr int KS = D / 32;                          // 32-element steps of the first product
    constexpr int PT = kTile / PE;                      // pages per tile
    constexpr int OP = D + 4;                           // row stride of the joined results
    __shared__ int before[DIRECT ? 1 : 256];
    __shared__ int wsum[4];
    __shared__ __attribute__((aligned(16))) float part_o[DIRECT > 1 ? DIRECT * 16 * OP : 4];
    __shared__ float part_m[16 * (DIRECT + 1)], part_l[16 * (DIRECT + 1)];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int group = a.n_heads / a.c.n_kv_heads, rows = a.queries * group;
    const int chunks = (rows + 15) / 16;
    const int hk = blockIdx.y / chunks, r = (blockIdx.y % chunks) * 16 + n;
    const int cols = rows < 16 ? rows : 16;             // columns of a partial result

    int w = 0, at = 0, stop = 1, start = 0, b = blockIdx.x, per = 1;
    if constexpr (!DIRECT) {
        // tiles before each thread's share of the histories
        const int each = (a.batch + 255) / 256;
        const int b_lo = tid * each, b_hi = b_lo + each < a.batch ? b_lo + each : a.batch;
        int mine = 0;
        for (int b = b_lo; b < b_hi; ++b) mine += span_of(a, b).count;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(inc, d, 64);
            if (lane >= d) inc += o;
        }
        if (lane == 63) wsum[wave] = inc;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < wave) inc += wsum[i];
            total += wsum[i];
        }
        before[tid] = inc - mine;
        __syncthreads();
        per = total > n_waves ? (total + n_waves - 1) / n_waves : 1;
        w = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + wave);
        if (w == 0 && blockIdx.y == 0 && lane == 0) meta[a.batch] = per;
        int64_t at64 = (int64_t)w * per;
        if (at64 >= total) return;
        at = (int)at64;
        stop = at + per < total ? at + per : total;
        int lo = 0, hi = 255;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        start = __builtin_amdgcn_readfirstlane(before[lo]);       // tiles before history b
        b = __builtin_amdgcn_readfirstlane(lo * each);
    }

    while (at < stop) {
        const Span sp = span_of(a, b);
        if (!DIRECT && start + sp.count <= at) {
            start += sp.count;
            ++b;
            continue;
        }
        // the wave's tiles of the history: a run, or every DIRECT-th
        const int i0 = DIRECT ? wave : at - start;
        const int i1 = DIRECT || sp.count < stop - start ? sp.count : stop - start;
        constexpr int STEP = DIRECT ? DIRECT : 1;
        if (!DIRECT && i0 == 0 && blockIdx.y == 0 && lane == 0) meta[b] = start;
        const int slot = a.slots ? a.slots[b] : b;
        const int32_t* table = a.c.table + (int64_t)slot * a.c.max_pages;

        bf16x8 q[KS][NQ];
        const bool live = r < rows;
        const int64_t qrow = (int64_t)b * a.queries + (live ? r / group : 0);
        const int qhead = hk * group + (live ? r % group : 0);
        load_query<D>((const T*)a.q + qrow * a.ld_q + (int64_t)qhead * D, a.scale, a.wide, g, q);
        floatx4 o[D / 16];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[j] = floatx4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;

        auto tile_of = [&](int i) { return i < sp.lead ? i : sp.first + (i - sp.lead); };
        auto load = [&](int i, Tile<D>& t) { load_tile<D, PE>(a.c, table, tile_of(i) * PT, hk, n, g, t); };
        const float c = exponent_scale(a.scale);
        auto use = [&](int i, Tile<D>& t) {
            const int e0 = tile_of(i) * kTile;
            const bool whole = (e0 >= sp.low || e0 + kTile <= sp.lead_events) && e0 + kTile <= sp.len;
            use_tile<D, T>(t, q, c, e0, whole, sp.low, sp.lead_events, sp.len, g, o, m, l);
        };

        // one tile is on its way while the other is used; where registers allow, the two take turns instead of being
        // moved (windowed batch 33.4 -> 32.3 us)
        constexpr bool TURNS = D < 128 || NQ == 1;
        Tile<D> cur, nxt;
        if (i0 < i1) load(i0, cur);
        for (int i = i0; i < i1; i += STEP) {
            if (i + STEP < i1) load(i + STEP, nxt);
            use(i, cur);
            if constexpr (TURNS) {
                i += STEP;
                if (i >= i1) break;
                if (i + STEP < i1) load(i + STEP, cur);
                use(i, nxt);
            } else {
                cur = nxt;
            }
        }
        m *= c;                                          // from here on in powers of two
        l += swizzle_xor16(l);
        l += __shfl_xor(l, 32, 64);

        if constexpr (DIRECT > 1) {
            if (g == 0) part_m[wave * 16 + n] = m;
            __syncthreads();
            float mx = part_m[n];
#pragma unroll
            for (int i = 1; i < DIRECT; ++i) mx = fmaxf(mx, part_m[16 * i + n]);
            const float f = mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mx);
            if (g == 0) part_l[wave * 16 + n] = l * f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) *(floatx4*)&part_o[(wave * 16 + n) * OP + 16 * j + 4 * g] = o[j] * f;
            __syncthreads();
            for (int x = tid; x < 4 * D; x += 64 * DIRECT) {
                const int y = x / (D / 4), d = x % (D / 4) * 4, row = r - n + y;
                if (row >= rows) break;
                float sum = part_l[y];
                floatx4 v = *(const floatx4*)&part_o[y * OP + d];
#pragma unroll
                for (int i = 1; i < DIRECT; ++i) {
                    sum += part_l[16 * i + y];
                    v += *(const floatx4*)&part_o[(16 * i + y) * OP + d];
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                T* op = (T*)a.out + ((int64_t)b * a.queries + row / group) * a.ld_out +
                        (int64_t)(hk * group + row % group) * D + d;
                store4(op, v * inv, a.wide);
            }
        } else if (DIRECT || (i0 == 0 && i1 == sp.count)) {
            if (live) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                T* op = (T*)a.out + qrow * a.ld_out + (int64_t)qhead * D;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    store4(op + 16 * j + 4 * g, o[j] * inv, a.wide);
            }
        } else if (n < cols) {
            // a run cuts at most the history it begins in and the one it ends in
            float* part = a.partial +
                          (((int64_t)2 * w + (i0 == 0 ? 1 : 0)) * gridDim.y + blockIdx.y) * cols * (D + 2) + n * (D + 2);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[16 * j + 4 * g + i] = o[j][i];
            if (g == 0) {
                part[D] = m;
                part[D + 1] = l;
            }
        }
        if constexpr (DIRECT) {
            if (__builtin_expect(sp.count == 0, 0) && a.slots && blockIdx.y == 0 && tid == 0) count_refused(a, b);
            break;
        }
        at = start + i1;
        start += sp.count;
        ++b;
    }
}

// Joins the runs that share a history: blocks of (history, chunk of rows, every
// gridDim.z-th 64 elements of its result).  The runs' maxima and sums first, then
// each element over four groups of runs, so that the reads of a history cut into
// many runs do not wait for one another.
template <int D, typename T>
__global__ __launch_bounds__(256) void history_join_kernel(LookupArgs a, const int* __restrict__ meta) {
    __shared__ float ms[16][17], ls[16][17], os[4][64];
    const int b = blockIdx.x, tid = threadIdx.x;
    const int group = a.n_heads / a.c.n_kv_heads, rows = a.queries * group;
    const int chunks = (rows + 15) / 16;
    const int hk = blockIdx.y / chunks, r0 = (blockIdx.y % chunks) * 16;
    const int cols = rows < 16 ? rows : 16;
    const int count = span_of(a, b).count;
    const int start = count ? meta[b] : 0, per = meta[a.batch];
    if (a.slots && count == 0 && (int)blockIdx.y + (int)blockIdx.z + tid == 0) count_refused(a, b);
    const int w0 = start / per, w1 = count ? (start + count - 1) / per : 0;
    if (count && w0 == w1) return;                      // one wave had it all
    const int runs = count ? w1 - w0 + 1 : 0;
    // run i of the history: its wave's second place for the first run, which began the history, the first for others
    const int64_t one = (int64_t)cols * (D + 2);
    auto run = [&](int i) {
        return a.partial + ((int64_t)(2 * (w0 + i) + (i == 0 ? 1 : 0)) * gridDim.y + blockIdx.y) * one;
    };
    if (runs <= 8) {                                    // not worth the barriers
        for (int x = blockIdx.z * 256 + tid; x < cols * D; x += gridDim.z * 256) {
            const int n = x / D, d = x % D;
            if (r0 + n >= rows) break;
            float pm[8], pl[8], po[8], m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float* p = run(i < runs ? i : 0) + n * (D + 2);
                pm[i] = runs ? p[D] : -INFINITY, pl[i] = runs ? p[D + 1] : 0.f, po[i] = runs ? p[d] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) m = i < runs ? fmaxf(m, pm[i]) : m;
            const float mf = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = i < runs ? __builtin_amdgcn_exp2f(pm[i] - mf) : 0.f;
                l += i < runs ? pl[i] * f : 0.f;
                o += i < runs ? po[i] * f : 0.f;
            }
            T* out = (T*)a.out + ((int64_t)b * a.queries + (r0 + n) / group) * a.ld_out +
                     (int64_t)(hk * group + (r0 + n) % group) * D;
            out[d] = (T)(l == 0.f ? 0.f : o / l);
        }
        return;
    }
    const int col = tid & 15, sub = tid >> 4;
    float m = -INFINITY, l = 0.f;
    for (int i = sub; i < runs && col < cols; i += 16) m = fmaxf(m, run(i)[col * (D + 2) + D]);
    ms[sub][col] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, ms[i][col]);
    const float mf = m == -INFINITY ? 0.f : m;
    for (int i = sub; i < runs && col < cols; i += 16) {
        const float* p = run(i) + col * (D + 2) + D;
        l += p[1] * __builtin_amdgcn_exp2f(p[0] - mf);
    }
    ls[sub][col] = l;
    __syncthreads();
    if (sub == 0) {
        l = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) l += ls[i][col];
        ls[0][col] = l;
        ms[0][col] = mf;
    }
    __syncthreads();
    const int e = tid & 63, part = tid >> 6;
    for (int x0 = blockIdx.z * 64; x0 < cols * D; x0 += gridDim.z * 64) {
        const int x = x0 + e, n = x / D, d = x % D;
        float o = 0.f;
        if (x < cols * D) {
            const float mn = ms[0][n];
#pragma unroll 8
            for (int i = part; i < runs; i += 4) {
                const float* p = run(i) + n * (D + 2);
                o += p[d] * __builtin_amdgcn_exp2f(p[D] - mn);
            }
        }
        os[part][e] = o;
        __syncthreads();
        if (part == 0 && x < cols * D && r0 + n < rows) {
            o = os[0][e] + os[1][e] + os[2][e] + os[3][e];
            T* out = (T*)a.out + ((int64_t)b * a.queries + (r0 + n) / group) * a.ld_out +
                     (int64_t)(hk * group + (r0 + n) % group) * D;
            const float sum = ls[0][n];
            out[d] = (T)(sum == 0.f ? 0.f : o / sum);
        }
        __syncthreads();
    }
}

// Waves for each chunk of rows of each kv head.
static int waves_of(const dlrm_history_cache_t& c, int64_t batch, int queries, int n_heads) {
    const int64_t rows = (int64_t)queries * (n_heads / c.n_kv_heads);
    const int64_t hc = (rows + 15) / 16 * c.n_kv_heads;
    const int64_t tiles = batch * (((int64_t)c.max_pages * c.page_events + kTile - 1) / kTile);
    int64_t w = (kLookupWaves + hc - 1) / hc;
    w = w < tiles ? w : tiles;
    return (int)((w + 3) / 4 * 4);
}

static size_t meta_bytes(int64_t batch) { return ((size_t)(batch + 1) * sizeof(int) + 255) / 256 * 256; }

size_t lookup_workspace_bytes(const dlrm_history_cache_t& c, int64_t batch, int queries, int n_heads) {
    const int64_t rows = (int64_t)queries * (n_heads / c.n_kv_heads);
    const int64_t hc = (rows + 15) / 16 * c.n_kv_heads, cols = rows < 16 ? rows : 16;
    return meta_bytes(batch) +
           (size_t)2 * waves_of(c, batch, queries, n_heads) * hc * cols * (c.head_dim + 2) * sizeof(float);
}

// Waves of a history's block: as many as let every block be resident at once, with
// `room` waves to a CU.  1024 blocks of up to 18 tiles: 2 waves 33 us, 1 or 4 42;
// 384 blocks of up to 24: 4 waves 18.7 us, 2 or 8 24-25.
static int direct_waves(int64_t blocks, int room) {
    int w = 8;
    while (w > 1 && blocks > 256 * (room / w)) w /= 2;
    return w;
}

template <int D, int PE, typename T>
static hipError_t launch_t(LookupArgs a, hipStream_t s) {
    const int rows = a.queries * (a.n_heads / a.c.n_kv_heads);
    const int hc = (rows + 15) / 16 * a.c.n_kv_heads;
    int* meta = (int*)a.partial;
    a.partial = (float*)((char*)a.partial + meta_bytes(a.batch));
    const int w = direct_waves((int64_t)a.batch * hc, D == 32 || (D == 64 && Parts<T>::q == 1) ? 12 : 8);
    if (most_tiles(a) <= (w == 8 ? kDirectTiles8 : kDirectTiles)) {
        if (!grid_fits(a.batch, 64 * w)) return kTooLarge;
        const dim3 grid(a.batch, hc);
        if (w == 8) hipLaunchKernelGGL((history_lookup_kernel<D, PE, T, 8>), grid, dim3(512), 0, s, a, 0, meta);
        else if (w == 4) hipLaunchKernelGGL((history_lookup_kernel<D, PE, T, 4>), grid, dim3(256), 0, s, a, 0, meta);
        else if (w == 2) hipLaunchKernelGGL((history_lookup_kernel<D, PE, T, 2>), grid, dim3(128), 0, s, a, 0, meta);
        else hipLaunchKernelGGL((history_lookup_kernel<D, PE, T, 1>), grid, dim3(64), 0, s, a, 0, meta);
        return hipGetLastError();
    }
    if (!grid_fits(a.batch, 256)) return kTooLarge;
    const int waves = waves_of(a.c, a.batch, a.queries, a.n_heads);
    hipLaunchKernelGGL((history_lookup_kernel<D, PE, T, 0>), dim3(waves / 4, hc), dim3(256), 0, s, a, waves, meta);
    // A few long histories are cut into many runs each: their elements are then spread over blocks, too.  64 histories
    // of up to 64 tiles, 8 waves each: 27.5 -> 23.0 us; 256, two waves each, would go 50.9 -> 53.3.
    const int cols = rows < 16 ? rows : 16;
    const int z = waves / a.batch >= 8 ? (cols * D + 63) / 64 : 1;
    hipLaunchKernelGGL((history_join_kernel<D, T>), dim3(a.batch, hc, z), dim3(256), 0, s, a, meta);
    return hipGetLastError();
}
template <int D, int PE>
static hipError_t launch_d(const LookupArgs& a, int dtype, hipStream_t s) {
    if (dtype == DLRM_DTYPE_F32) return launch_t<D, PE, float>(a, s);
    if (dtype == DLRM_DTYPE_BF16) return launch_t<D, PE, bf16>(a, s);
    return launch_t<D, PE, f16>(a, s);
}
template <int PE>
static hipError_t launch_p(const LookupArgs& a, int dtype, hipStream_t s) {
    if (a.c.head_dim == 32) return launch_d<32, PE>(a, dtype, s);
    if (a.c.head_dim == 64) return launch_d<64, PE>(a, dtype, s);
    return launch_d<128, PE>(a, dtype, s);
}

hipError_t launch_history_lookup(const LookupArgs& a, int dtype, hipStream_t s) {
    if (a.c.page_events == 16) return launch_p<16>(a, dtype, s);
    if (a.c.page_events == 32) return launch_p<32>(a, dtype, s);
    return launch_p<64>(a, dtype, s);
}

}  // namespace dlrm
