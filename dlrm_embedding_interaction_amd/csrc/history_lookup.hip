// history_lookup.hip -- attention of single queries over the 8-bit paged cache.
//
// The queries of history b stand at its last position len - 1 and see event j
// iff j >= len - window or j < sinks.  Keys and values are e4m3 codes times the
// power-of-two scale of their page and head.
#include "history.h"

namespace dlrm {

template <typename T>
__global__ __launch_bounds__(64) void history_lookup_kernel(LookupArgs a) {
    __shared__ float qs[128];
    __shared__ float ps[64];
    const int lane = threadIdx.x, h = blockIdx.y, hk = h / (a.n_heads / a.c.n_kv_heads);
    const int64_t row = blockIdx.x;
    const int b = (int)(row / a.queries), dim = a.c.head_dim, pe = a.c.page_events;
    const int slot = a.slots ? a.slots[b] : b;
    const bool held = slot >= 0 && slot < a.c.n_slots;
    const int64_t span = (int64_t)a.c.max_pages * pe;
    int64_t len = held ? a.c.lens[slot] : 0;
    len = len < 0 ? 0 : (len > span ? span : len);
    const T* q = (const T*)a.q + row * a.ld_q + (int64_t)h * dim;
    for (int d = lane; d < dim; d += 64) qs[d] = ld_f32(q + d);
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    const int64_t first = len - a.window > 0 ? len - a.window : 0;
    const int64_t lead = a.sinks < first ? a.sinks : first;
    const int64_t lead_tiles = (lead + 63) / 64;
    const int64_t tiles = lead_tiles + (len - first + 63) / 64;
    for (int64_t t = 0; t < tiles; ++t) {
        const int64_t base = t < lead_tiles ? t * 64 : first + (t - lead_tiles) * 64;
        const int64_t stop = t < lead_tiles ? lead : len;
        const int64_t j = base + lane;
        bool seen = j < stop;
        int page = -1;
        if (seen) {
            page = a.c.table[(int64_t)slot * a.c.max_pages + j / pe];
            seen = page >= 0 && page < a.c.n_pages;
        }
        float s = -INFINITY;
        if (seen) {
            const int64_t ph = (int64_t)page * a.c.n_kv_heads + hk;
            const uint8_t* k = a.c.k + (ph * pe + j % pe) * dim;
            float dot = 0.f;
            for (int d = 0; d < dim; ++d) dot = fmaf(qs[d], e4m3_f32(k[d]), dot);
            s = dot * a.c.k_scale[ph] * a.scale;
        }
        const float mt = fmaxf(m, wave_max(s));
        if (mt == -INFINITY) continue;
        const float p = seen ? __expf(s - mt) : 0.f;
        const float alpha = __expf(m - mt);
        l = l * alpha + wave_sum(p);
        m = mt;
        __syncthreads();
        ps[lane] = seen ? p : -1.f;
        __syncthreads();
        for (int c = 0; c < 2; ++c) {
            const int d = lane + c * 64;
            if (d >= dim) continue;
            float o = acc[c] * alpha;
            for (int x = 0; x < 64; ++x)
                if (ps[x] >= 0.f || ps[x] != ps[x]) {
                    const int64_t jj = base + x;
                    const int pg = a.c.table[(int64_t)slot * a.c.max_pages + jj / pe];
                    const int64_t ph = (int64_t)pg * a.c.n_kv_heads + hk;
                    o = fmaf(ps[x], e4m3_f32(a.c.v[(ph * dim + d) * pe + jj % pe]) * a.c.v_scale[ph], o);
                }
            acc[c] = o;
        }
    }
    T* out = (T*)a.out + row * a.ld_out + (int64_t)h * dim;
    for (int c = 0; c < 2; ++c) {
        const int d = lane + c * 64;
        if (d < dim) out[d] = (T)(l == 0.f ? 0.f : acc[c] / l);
    }
}

size_t lookup_workspace_bytes(const dlrm_history_cache_t&, int64_t, int, int) { return 256; }

hipError_t launch_history_lookup(const LookupArgs& a, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)(a.batch * a.queries), (unsigned)a.n_heads);
    if (dtype == DLRM_DTYPE_F32) hipLaunchKernelGGL(history_lookup_kernel<float>, grid, dim3(64), 0, s, a);
    else if (dtype == DLRM_DTYPE_BF16) hipLaunchKernelGGL(history_lookup_kernel<bf16>, grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL(history_lookup_kernel<f16>, grid, dim3(64), 0, s, a);
    return hipGetLastError();
}

}  // namespace dlrm
