// history_attention.hip -- causal attention over ragged event histories with a
// sliding window and first events that stay visible.
//
// Row i of a history sees key j iff j <= i, (i - j < window or j < sinks) and
// event j is not padding:
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale <q_i, k_j> - m_i)
// in one pass over the keys with the running maximum m and sum.  A row that
// sees nothing gives zeros.
#include "history.h"

namespace dlrm {

// One wave per (event, head): lanes over 64 keys for the products, over the
// head's elements for the weighted sum.
template <typename T>
__global__ __launch_bounds__(64) void history_attention_kernel(EncodeArgs a, int dim) {
    __shared__ float qs[128];
    __shared__ float ps[64];
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int h = blockIdx.y, hk = h / (a.n_heads / a.n_kv);
    // the last history that begins at or before the row
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (history_begin(a.offsets, a.idx32, mid, a.n_events) <= row) lo = mid;
        else hi = mid - 1;
    }
    const int64_t begin = history_begin(a.offsets, a.idx32, lo, a.n_events);
    if (begin > row) return;
    const T* q = (const T*)a.q + row * a.ld_q + (int64_t)h * dim;
    for (int d = lane; d < dim; d += 64) qs[d] = ld_f32(q + d);
    __syncthreads();
    const int64_t i = row - begin;
    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    const int64_t first = i - a.window + 1 > 0 ? i - a.window + 1 : 0;
    const int64_t lead = (a.sinks < first ? a.sinks : first + 0);
    const int64_t lead_tiles = (lead + 63) / 64;
    const int64_t tiles = lead_tiles + (i - first) / 64 + 1;
    for (int64_t t = 0; t < tiles; ++t) {
        const int64_t base = t < lead_tiles ? t * 64 : first + (t - lead_tiles) * 64;
        const int64_t stop = t < lead_tiles ? lead : i + 1;
        const int64_t j = base + lane;
        bool seen = j < stop;
        if (seen && a.padding) seen = a.padding[begin + j] == 0;
        float s = -INFINITY;
        if (seen) {
            const T* k = (const T*)a.k + (begin + j) * a.ld_k + (int64_t)hk * dim;
            float dot = 0.f;
            for (int d = 0; d < dim; ++d) dot = fmaf(qs[d], ld_f32(k + d), dot);
            s = dot * a.scale;
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
                if (ps[x] >= 0.f || ps[x] != ps[x])
                    o = fmaf(ps[x], ld_f32((const T*)a.v + (begin + base + x) * a.ld_v + (int64_t)hk * dim + d), o);
            acc[c] = o;
        }
    }
    T* out = (T*)a.out + row * a.ld_out + (int64_t)h * dim;
    for (int c = 0; c < 2; ++c) {
        const int d = lane + c * 64;
        if (d < dim) out[d] = (T)(l == 0.f ? 0.f : acc[c] / l);
    }
}

hipError_t launch_history_attention(const EncodeArgs& a, int dtype, int dim, hipStream_t s) {
    const dim3 grid((unsigned)a.n_events, (unsigned)a.n_heads);
    if (dtype == DLRM_DTYPE_F32) hipLaunchKernelGGL(history_attention_kernel<float>, grid, dim3(64), 0, s, a, dim);
    else if (dtype == DLRM_DTYPE_BF16) hipLaunchKernelGGL(history_attention_kernel<bf16>, grid, dim3(64), 0, s, a, dim);
    else hipLaunchKernelGGL(history_attention_kernel<f16>, grid, dim3(64), 0, s, a, dim);
    return hipGetLastError();
}

}  // namespace dlrm
