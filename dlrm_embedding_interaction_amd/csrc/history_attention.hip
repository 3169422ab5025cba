// history_attention.hip -- causal attention over ragged event histories with a
// sliding window and first events that stay visible.
//
// Row i of a history sees key j iff j <= i, (i - j < window or j < sinks) and
// event j is not padding:
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale <q_i, k_j> - m_i)
// in one pass over the keys with the running maximum m and sum.  A row that
// sees nothing gives zeros.
//
// One block takes 32 W rows of one history and head, one wave 32 of them, and
// walks the tiles of BN keys that any of its rows sees: first those of the
// sinks, then those of the window.  Both products run on the matrix cores
// (32x32x16) with the rows as columns:
//   S^T = K Q^T, O^T += V^T P^T.
// A lane then holds one row's scores of half the tile's keys: the row's maximum
// and sum are the lane's own and its partner's (lane ^ 32), and the scores are
// the second product's operand as they are, in registers.  K and V pass through
// LDS, shared by the block's waves; V is turned by the transposing LDS read.  The
// next tile is on its way from memory while this one is worked on.
//
// fp32 tensors are multiplied as three bf16 parts each (rounded, so that the
// parts hold all 24 bits), in the six products of parts that are not below
// 2^-24 of the whole: 6/16 of the fp32 matrix instructions' time.  16-bit
// tensors round the weights to their own type once: against the 64-bit form
// 0.0020 of the output's size in bf16, where rounding the output alone gives
// 0.0016, 0.00026 against 0.00020 in fp16; maxima, sums and outputs are held in
// fp32.
//
// Measured on MI355X, bf16: 2 histories of up to 12001 events, 8 heads on 2 kv heads
// of 128, window 4096: 279 to 288 us, 810 to 830 TFLOP/s of visible pairs, 67 to 69%
// of a large library product (1204).  Per 32 rows x 32 keys a wave issues 16 products (512 cycles) and
// ~110 vector instructions (~600 cycles with the exponentials); the counters show
// 40% and 40% of the cycles busy with either, the rest waiting for LDS and at
// barriers.  256 histories of up to 512, 4 heads of 64, window 128: 43 us against 29
// for its bytes, the masked edges of the window being most of the work.  Tried and
// not kept: two LDS buffers with one barrier a tile (309 against 293 us), 64 keys at
// a time (304), reads ordered ahead of the products, raised wave priorities.
#include "history.h"

namespace dlrm {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef short shortx8 __attribute__((ext_vector_type(8)));

// How a type is multiplied: as `parts` values of `part` each.
template <typename T> struct Mul;
template <> struct Mul<bf16> { typedef bf16 part; static constexpr int parts = 1; };
template <> struct Mul<f16> { typedef f16 part; static constexpr int parts = 1; };
template <> struct Mul<float> { typedef bf16 part; static constexpr int parts = 3; };

__device__ __forceinline__ floatx16 mfma(shortx8 a, shortx8 b, floatx16 c, bf16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ floatx16 mfma(shortx8 a, shortx8 b, floatx16 c, f16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// Sum of the products of parts: all pairs whose product can matter.
template <typename E, int N>
__device__ __forceinline__ floatx16 mul_parts(const shortx8* a, const shortx8* b, floatx16 c) {
    if constexpr (N == 1) {
        return mfma(a[0], b[0], c, E{});
    } else {
        c = mfma(a[0], b[2], c, E{});
        c = mfma(a[1], b[1], c, E{});
        c = mfma(a[2], b[0], c, E{});
        c = mfma(a[0], b[1], c, E{});
        c = mfma(a[1], b[0], c, E{});
        return mfma(a[0], b[0], c, E{});
    }
}

// The largest fp32 value that rounds to a finite bf16 one.  Finite values beyond it
// would have an infinite first part; cut to it, theirs is the largest bf16 and the
// rest is exact as before.
constexpr float kLargestFirst = 0x1.fefffep+127f;
__device__ __forceinline__ float first_part(float x) { return fminf(fmaxf(x, -kLargestFirst), kLargestFirst); }

// Eight fp32 values as N vectors of parts, the first the rounded values, each
// next one the rounded rest.  LARGE: values beyond kLargestFirst are met.  Returns
// 0, or NaN where a rest is not finite.
template <typename E, int N, bool LARGE = false>
__device__ __forceinline__ float split8(const float* x, shortx8* part) {
    typedef E Ex8 __attribute__((ext_vector_type(8)));
    float r[8], odd = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        Ex8 e;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            e[i] = (E)(LARGE && n == 0 ? first_part(r[i]) : r[i]);
            if (n + 1 < N) r[i] -= (float)e[i];
            if (n + 2 == N) odd = fmaf(r[i], 0.f, odd);
        }
        part[n] = __builtin_bit_cast(shortx8, e);
    }
    return odd;
}

template <bool LARGE = false, typename T>
__device__ __forceinline__ float to_parts(const Raw<T>& r, shortx8* part) {
    if constexpr (Mul<T>::parts == 1) {
        part[0] = __builtin_bit_cast(shortx8, r);
        return 0.f;
    } else {
        return split8<bf16, 3, LARGE>(r.x, part);
    }
}
template <typename T>
__device__ __forceinline__ bool finite_bits(T x) {
    if constexpr (sizeof(T) == 4) return (__builtin_bit_cast(unsigned, x) & 0x7f800000u) != 0x7f800000u;
    const unsigned short all = sizeof(T) == 2 && __is_same(T, f16) ? 0x7c00 : 0x7f80;
    if constexpr (sizeof(T) == 2) return (__builtin_bit_cast(unsigned short, x) & all) != all;
    return true;
}

// Four keys of 16 columns, turned: lane j of a group of 16 points at key
// j / 4, columns 4 (j % 4) .. + 3, and receives column j of the four keys.
__device__ __forceinline__ shortx4 read_turned(const void* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) shortx4*)(__attribute__((address_space(3))) void*)p);
}

// The larger of a value and its partner's in lane ^ 32, and their sum.
__device__ __forceinline__ float halves_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Log2 of what a weight is multiplied by, and with it the row's sum.  Weights taken
// against a maximum that lags by 2^8 then stay below 1: a mean of large values
// passes the type's end on its way only where their sum does.  fp16 values are far
// from the accumulators' end, but its weights would be 0 below 2^-25: they go up to
// 2^15, so that those below 2^-21 are off by 2^-32 at most.
template <typename T> constexpr float kWeightLog2 = __is_same(T, f16) ? 7.f : -8.f;

// Waves per SIMD that the registers are cut to.  All fits but at heads of 128, where 13 of the 99 kernels keep 44 to 140
// bytes a lane in scratch: fp32 in blocks of rows of their own, 16-bit with padding in two waves or with shared keys.
template <typename T, int D> constexpr int kWavesPerSimd = sizeof(T) == 4 || D == 128 ? 2 : (D == 64 ? 3 : 4);

// WIDE: 16-byte loads and stores.  PAD: padding bytes may be given.  KS: waves that
// share the keys of a tile among them for the same rows, and join at the end.
template <typename T, int D, int W, int BN, bool WIDE, bool PAD, int KS>
__global__ __launch_bounds__(64 * W, (kWavesPerSimd<T, D>)) void history_attention_kernel(EncodeArgs a, int heads_log2) {
    typedef typename Mul<T>::part E;
    constexpr int N = Mul<T>::parts;
    constexpr int THREADS = 64 * W;
    constexpr int KP = D + 8;                       // row strides in LDS: 16-byte reads of 8 rows, and the turned
    constexpr int VP = D == 32 ? D : D + 32;        // reads of 4 rows, touch every bank once
    constexpr int VEC = (BN * D / 8 + THREADS - 1) / THREADS;
    static_assert(BN * D / 8 % THREADS == 0, "whole vectors per thread");
    __shared__ __attribute__((aligned(16))) E ks[N][BN][KP];
    __shared__ __attribute__((aligned(16))) E vs[N][BN][VP];
    __shared__ int odd[2];      // even / odd tiles hold an infinity or NaN among their values (fp32: parts of either)

    const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);      // conditions on it are scalar branches
    constexpr int PK = BN / KS;                     // keys of the tile that the wave works on
    const int BM = 32 * (W / KS) >> heads_log2;
    const int ks_at = wave % KS, wr = wave / KS;
    const int head = (blockIdx.y << heads_log2) + (wr & ((1 << heads_log2) - 1)), hk = head / (a.n_heads / a.n_kv);
    // the longest rows first: a history's last tiles see the most keys
    const Unit un = history_of_unit(a.offsets, a.idx32, a.batch, a.n_events, BM, 1,
                                    (int64_t)gridDim.x - 1 - blockIdx.x);
    const int64_t nth = un.nth, begin = un.begin;
    const int len = (int)(un.end - begin);
    if (nth < 0 || nth * BM >= len) return;
    const int q0 = (int)nth * BM, r0 = q0 + (wr >> heads_log2) * 32, row = r0 + n;
    const int last = q0 + BM < len ? q0 + BM - 1 : len - 1;
    const int window = __builtin_amdgcn_readfirstlane((int)a.window);
    const int sinks = __builtin_amdgcn_readfirstlane((int)a.sinks);
    const T* kg = (const T*)a.k + begin * a.ld_k + (int64_t)hk * D;
    const T* vg = (const T*)a.v + begin * a.ld_v + (int64_t)hk * D;
    const uint8_t* pad = PAD && a.padding ? a.padding + begin : nullptr;

    // tiles of keys: `lead` of the sinks, then from `first` on
    int low = q0 >= window ? q0 - window + 1 : 0;
    if (sinks >= low) low = 0;
    const int first = low / BN;
    int lead = low ? (sinks + BN - 1) / BN : 0;
    lead = lead < first ? lead : first;
    const int tiles = lead + last / BN + 1 - first;
    auto key_of = [&](int t) { return (t < lead ? t : first + t - lead) * BN; };

    // the row's elements 16 s + 8 h .. + 7; a negative scale turns their sign, so that scores only grow by it
    shortx8 q[D / 16][N];
    {
        const T* qp = (const T*)a.q + (begin + (row < len ? row : len - 1)) * a.ld_q + (int64_t)head * D;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            Raw<T> r = load_raw<WIDE>(qp + 16 * s + 8 * h);
            to_parts<true>(r, q[s]);
#pragma unroll
            for (int i = 0; i < N; ++i) q[s][i] ^= a.scale < 0.f ? (short)0x8000 : (short)0;
        }
    }
    const float c = exponent_scale(a.scale);

    Raw<T> kr[VEC], vr[VEC];
    uint8_t hide = 0;       // the padding byte of the wave's key `lane`, as loaded: a comparison here would wait for it
    // Rows behind the history's end stand in as its last one: no row sees them.
    auto fetch = [&](int t) {
        const int k0 = key_of(t);
        if (PAD && pad && lane < PK) hide = pad[min(k0 + ks_at * PK + lane, len - 1)];
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
            const int p = tid + x * THREADS, d = p % (D / 8) * 8;
            const int key = min(k0 + p / (D / 8), len - 1);
            kr[x] = load_raw<WIDE>(kg + (int64_t)key * (int)a.ld_k + d);
            vr[x] = load_raw<WIDE>(vg + (int64_t)key * (int)a.ld_v + d);
        }
    };

    floatx16 o[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) o[j] = floatx16{};
    float m = -INFINITY, l = 0.f;

    fetch(0);
    if (tid == 0) odd[0] = 0;
    for (int t = 0; t < tiles; ++t) {
        const int k0 = key_of(t);
        const unsigned long long hidden = PAD ? __ballot(hide != 0) : 0;      // the wave's padding events
        __syncthreads();                            // the tile before has been read
        if (tid == 0) odd[(t + 1) & 1] = 0;
        unsigned big = 0;
        float rest = 0.f;
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
            const int p = tid + x * THREADS, key = p / (D / 8), d = p % (D / 8) * 8;
            shortx8 kp[N], vp[N];
            rest += to_parts(kr[x], kp);
            rest += to_parts(vr[x], vp);
            if constexpr (N == 1) top_magnitude(vr[x], big);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                *(shortx8*)&ks[i][key][d] = kp[i];
                *(shortx8*)&vs[i][key][d] = vp[i];
            }
        }
        if (__builtin_expect(N == 1 ? odd_magnitude<T>(big) : rest != 0.f, 0)) {       // NaN differs from 0
            // infinities and NaN are taken out of the products and added to the rows that see them, fp32 keys' to the
            // scores; finite fp32 keys and values whose first part is not finite are split anew
            odd[t & 1] = 1;
#pragma unroll
            for (int x = 0; x < VEC; ++x) {
                const int p = tid + x * THREADS, key = p / (D / 8), d = p % (D / 8) * 8;
                Raw<T> kf = kr[x], vf = vr[x];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    kf.x[i] = finite_bits(kf.x[i]) ? kf.x[i] : (T)0.f;
                    vf.x[i] = finite_bits(vf.x[i]) ? vf.x[i] : (T)0.f;
                }
                shortx8 kp[N], vp[N];
                to_parts<true>(kf, kp);
                to_parts<true>(vf, vp);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (N > 1) *(shortx8*)&ks[i][key][d] = kp[i];
                    *(shortx8*)&vs[i][key][d] = vp[i];
                }
            }
        }
        __syncthreads();
        if (t + 1 < tiles) fetch(t + 1);
        const bool fix = __builtin_amdgcn_readfirstlane(odd[t & 1]) != 0;
        // 32 keys at a time, those that no row of the wave sees left out
#pragma unroll
        for (int u = 0; u < PK / 32; ++u) {
            const int k1 = k0 + ks_at * PK + 32 * u;
            if (k1 > r0 + 31 || (r0 - (k1 + 31) >= window && k1 >= sinks)) continue;
            floatx16 s = floatx16{};
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                shortx8 kk[N];
#pragma unroll
                for (int i = 0; i < N; ++i) kk[i] = *(const shortx8*)&ks[i][ks_at * PK + u * 32 + n][16 * x + 8 * h];
                s = mul_parts<E, N>(kk, q[x], s);
            }
            if constexpr (N > 1) {
                if (__builtin_expect(fix, 0)) {
                    // infinities and NaN of the keys by the queries' first parts, which have their signs and zeros: with
                    // all parts an infinity would meet the zeros among the others
                    const T* kp = kg + (int64_t)min(k1 + n, len - 1) * a.ld_k + 8 * h;
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        Raw<T> r = load_raw<false>(kp + 16 * x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) r.x[i] = finite_bits(r.x[i]) ? (T)0.f : r.x[i];
                        shortx8 e[N];
                        to_parts(r, e);
                        s = mfma(e[0], q[x][0], s, E{});
                    }
                }
            }
            const unsigned off = PAD ? (unsigned)(hidden >> (32 * u)) : 0;
            if (k1 + 31 > r0 || (r0 + 31 - k1 >= window && k1 + 32 > sinks) || off) {
                // bit y: the row sees key k1 + 4 h + y.  Whatever stands in the other keys leaves here; their values
                // meet weights of 0, and those that are not finite are dealt with apart.
                auto up_to = [](int y) { return y < 0 ? 0u : y > 30 ? ~0u : (2u << y) - 1u; };      // bits 0 .. y
                const int k2 = k1 + 4 * h;
                const unsigned see = up_to(row - k2) & (~up_to(row - window - k2) | up_to(sinks - 1 - k2)) &
                                     ~(off >> (4 * h));
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // the bit spread over a word picks the score's bits or those of -inf, without a condition register
                    const unsigned keep = (unsigned)((int)(see << (31 - (8 * (i >> 2) + (i & 3)))) >> 31);
                    s[i] = __uint_as_float((__float_as_uint(s[i]) & keep) | (0xff800000u & ~keep));
                }
            }
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[i]);
            top = halves_max(top);
            // the maximum a row's weights are taken against may lag the true one by 2^8: weights then stay below
            // that, far from the end of every type, and most tiles leave the sums as they are.  Each row decides for
            // itself, so that its bits do not depend on the rows that share its wave.
            const bool up = (top - m) * c > 8.f;
            if (__any(up)) {
                const float mx = up ? top : m;
                const float alpha = mx == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mx) * c);
                l *= alpha;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) o[j] *= alpha;
                m = mx;
            }
            const float mc = m == -INFINITY ? 0.f : m * c - kWeightLog2<T>;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = __builtin_amdgcn_exp2f(fmaf(s[8 * e + i], c, -mc));
                    l += p[i];
                }
                shortx8 pp[N];
                split8<E, N>(p, pp);
                // keys 16 e + 4 h + {0..3} and + 8 of this half: the lane's own scores
                const int key = ks_at * PK + u * 32 + 16 * e + 4 * h + (n >> 2 & 3), col = 16 * (lane >> 4 & 1) + 4 * (n & 3);
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    shortx8 vv[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const shortx4 v0 = read_turned(&vs[i][key][32 * j + col]);
                        const shortx4 v1 = read_turned(&vs[i][key + 8][32 * j + col]);
                        vv[i] = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                    o[j] = mul_parts<E, N>(vv, pp, o[j]);
                }
            }
        }
        if (__builtin_expect(fix, 0)) {
            for (int key = k0 + ks_at * PK; key < k0 + (ks_at + 1) * PK && key < len; ++key)
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const T v = vg[(int64_t)key * a.ld_v + 32 * j + 8 * (i >> 2) + 4 * h + (i & 3)];
                        const bool sees = key <= row && (row - key < window || key < sinks) && !(pad && pad[key]);
                        if (!finite_bits(v) && sees) o[j][i] += (float)v;
                    }
        }
    }
    l = halves_sum(l);
    if constexpr (KS > 1) {
        // the waves' results against their common maximum: the upper half hands theirs to the lower half, and so on
        // down to the first
        static_assert(sizeof(vs) >= W / 2 * (D / 32) * 4096, "room for the results of half the waves");
        __shared__ float mm[W][32], ll[W][32];
        floatx4* give = (floatx4*)&vs[0][0][0];
        if (h == 0) mm[wave][n] = m;
        __syncthreads();                            // also: the last tile has been read
        const int w0 = wr * KS;
        float mx = mm[w0][n];
#pragma unroll
        for (int i = 1; i < KS; ++i) mx = fmaxf(mx, mm[w0 + i][n]);
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - mx) * c);
        if (h == 0) ll[wave][n] = l * f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) o[j] *= f;
#pragma unroll
        for (int half = KS / 2; half; half /= 2) {
            if (ks_at >= half && ks_at < 2 * half) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        give[((wr * (KS / 2) + ks_at - half) * (D / 32) * 4 + j * 4 + i) * 64 + lane] =
                            floatx4{o[j][4 * i], o[j][4 * i + 1], o[j][4 * i + 2], o[j][4 * i + 3]};
            }
            __syncthreads();
            if (ks_at < half) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const floatx4 v = give[((wr * (KS / 2) + ks_at) * (D / 32) * 4 + j * 4 + i) * 64 + lane];
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[j][4 * i + x] += v[x];
                    }
            }
            __syncthreads();
        }
        if (ks_at != 0) return;
        l = ll[w0][n];
#pragma unroll
        for (int i = 1; i < KS; ++i) l += ll[w0 + i][n];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* op = (T*)a.out + (begin + row) * a.ld_out + (int64_t)head * D;
    if constexpr (WIDE && sizeof(T) == 2) {
        // the two halves of a row hold four elements each of every eight: exchanged, a lane stores eight at once
        typedef unsigned u4 __attribute__((ext_vector_type(4)));
        typedef T t2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                unsigned w[4];          // elements 16 e + 4 h .. + 3, and + 8
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = __builtin_bit_cast(unsigned, t2{(T)(o[j][8 * e + 2 * i] * inv), (T)(o[j][8 * e + 2 * i + 1] * inv)});
                const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                if (row < len) *(u4*)(op + 32 * j + 16 * e + 8 * h) = u4{x[0], y[0], x[1], y[1]};
            }
    } else if (row < len) {
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                T* at = op + 32 * j + 2 * i + 4 * h;
                if constexpr (WIDE) {
                    *(floatx4*)at = floatx4{o[j][i] * inv, o[j][i + 1] * inv, o[j][i + 2] * inv, o[j][i + 3] * inv};
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x) at[x] = (T)(o[j][i + x] * inv);
                }
            }
    }
}

template <typename T, int D, int W, int KS = 1>
static hipError_t launch_w(const EncodeArgs& a, bool wide, int heads_log2, hipStream_t s) {
    constexpr int BN = (sizeof(T) == 4 && D == 128 ? 32 : 64) * KS;
    const int64_t tiles = a.n_events / (32 * (W / KS) >> heads_log2) + a.batch;
    if (!grid_fits(tiles, 64 * W)) return kTooLarge;
    const dim3 grid((unsigned)tiles, (unsigned)(a.n_heads >> heads_log2));
    const dim3 block(64 * W);
    if (!wide) hipLaunchKernelGGL((history_attention_kernel<T, D, W, BN, false, true, KS>), grid, block, 0, s, a, heads_log2);
    else if (a.padding) hipLaunchKernelGGL((history_attention_kernel<T, D, W, BN, true, true, KS>), grid, block, 0, s, a, heads_log2);
    else hipLaunchKernelGGL((history_attention_kernel<T, D, W, BN, true, false, KS>), grid, block, 0, s, a, heads_log2);
    return hipGetLastError();
}
template <typename T, int D>
static hipError_t launch_d(const EncodeArgs& a, bool wide, hipStream_t s) {
    const int64_t mean = a.n_events / a.batch;
    const int group = a.n_heads / a.n_kv;
    // Log2 of the heads that share a block, and its rows in 32s.  Blocks of 32 rows waste fewest on short histories,
    // larger ones share their tiles.  Measured, 32 rows against 64: 1024 histories of 20, 4 heads of 32, fp16 9.2 us to
    // 12.4, of 32 15.9 to 13.2; 2048 of 20, 4 heads of 64, bf16 36 to 31; up to 128 events, 4 heads of 128 on two kv
    // heads, bf16 51 to 52, up to 160 66 to 65; 4 heads of 64 on two, fp32, up to 40 41 to 39.
    const int heads = group % 4 == 0 ? 2 : (group % 2 == 0 ? 1 : 0);
    const bool one = heads ? sizeof(T) == 2 && mean <= 72 : D == 32 && mean <= 24;
    // 64 rows against 128: 2048 of up to 128, 4 heads of 64, bf16 60 us to 64, of up to 192 108 to 111; of 48 37 to 49.
    // Histories that fill their 64 or 96 rows go the other way, and so do small heads: 2048 of 64 65 to 56, of 96 97 to
    // 93; 1024 of 64, 4 heads of 32, fp16 28 to 22, of up to 128 28 to 26; 512 of 64, 2 heads of 64, fp32 39 to 25.  The
    // mean does not tell the two apart.
    const int rows = one ? 1 : (mean <= 96 ? 2 : 4);
    // Blocks of 8 waves read each tile once for twice the rows, blocks of 4 leave two to a CU, one's loads and stores
    // beside the other's products.  Lifelong (66 tiles a block) 8 waves 294 us, 4 waves 312; grouped (10 tiles) 308
    // against 289.
    const int64_t tiles = (a.window < mean ? a.window : mean) / 64;
    // A few long histories do not fill the card, and a block's time is its row of tiles: four waves (two, where three
    // parts of each element fill the LDS) then share each row's keys.  4000 events, 4 heads of 64 (125 blocks)
    // 78 -> 39 us; 8000, one head of 128 (63) 207 -> 112; with 376 blocks it would be 48 -> 77.
    const int rows_log2 = (rows << heads >= 4 ? 7 : (rows << heads == 2 ? 6 : 5)) - heads;      // of a block
    const int64_t blocks = ((a.n_events >> rows_log2) + 1) * (a.n_heads >> heads);
    if (tiles >= 8 && blocks < 256) {
        if constexpr (sizeof(T) == 2 || D == 32) return launch_w<T, D, 8, 4>(a, wide, heads ? 1 : 0, s);
        else return launch_w<T, D, 4, 2>(a, wide, heads ? 1 : 0, s);
    }
    if constexpr (D == 128) {
        if (rows << heads >= 8 && tiles >= 24) return launch_w<T, D, 8>(a, wide, heads, s);
    }
    if (rows << heads >= 4) return launch_w<T, D, 4>(a, wide, heads, s);
    if constexpr (D == 32) {
        if (rows << heads == 1) return launch_w<T, D, 1>(a, wide, heads, s);
    }
    return launch_w<T, D, 2>(a, wide, heads, s);
}
template <typename T>
static hipError_t launch_t(const EncodeArgs& a, int dim, hipStream_t s) {
    const int64_t step = 16 / sizeof(T);
    const bool wide = a.ld_q % step == 0 && a.ld_k % step == 0 && a.ld_v % step == 0 && a.ld_out % step == 0 &&
                      (((uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.out) & 15u) == 0;
    if (dim == 32) return launch_d<T, 32>(a, wide, s);
    if (dim == 64) return launch_d<T, 64>(a, wide, s);
    return launch_d<T, 128>(a, wide, s);
}

hipError_t launch_history_attention(const EncodeArgs& args, int dtype, int dim, hipStream_t s) {
    EncodeArgs a = args;
    const int64_t most = (int64_t)1 << 30;      // no history is longer
    a.window = a.window < most ? a.window : most;
    a.sinks = a.sinks < most ? a.sinks : most;
    if (dtype == DLRM_DTYPE_F32) return launch_t<float>(a, dim, s);
    if (dtype == DLRM_DTYPE_BF16) return launch_t<bf16>(a, dim, s);
    return launch_t<f16>(a, dim, s);
}

}  // namespace dlrm
