// cross_attention_few.cuh - cross attention of few queries: at most 16 rows
// (queries times the query heads that share a key head) per batch row and key
// head, over 16-bit keys or the 8-bit cache: xa_few_kernel.
//
// Every key and value is then used for 16 rows at most, so reading them is the
// bound (84 MB, 13 us, for 2 x 20 heads x 16384 keys x 64 in 8 bits), and a
// 128-row tensor-core tile would be nearly empty and slow to turn round.
// Instead each warp streams key blocks of its own straight from global memory
// into the register fragments of mma.sync (m16n8k16), with no shared memory,
// no barriers and the next block's loads in flight under this one's work:
//
//   S (rows x keys) = Q K^T:  B fragments. The contraction index may be
//     permuted freely, so lane (g, t) = (lane / 4, lane % 4) takes 16
//     contiguous bytes of key g's row, and Q is laid out to match.
//   O^T (d x rows) += V^T P^T: A fragments pair two keys at one d; lane (g, t)
//     takes keys 2t, 2t+1, 2t+8, 2t+9 at contiguous d and interleaves them with
//     byte permutes. P^T's B fragment is S's accumulator as it stands.
//
// 8-bit codes are exact in f16 (one conversion per pair), so that kernel
// multiplies in f16: q is scaled by a power of two per row to be exact there,
// the block's k scale joins the softmax scale and its v scale is applied when a
// step's product is added to O in float32. Powers of two or not, no scale is
// rounded to 16 bits. P is taken at the step's own largest score, and what that
// lies under the row's reference is applied in float32 too: a block's values may
// be as large as its probabilities are small, which f16 P at one reference for
// all keys would lose below 2^-31.
//
// The key range is split over CTAs and over a CTA's four warps; the warps merge
// through shared memory, the CTAs as a cluster through each other's shared
// memory, or, where more than eight of them pay, through a workspace and
// xa_combine_kernel. The softmax reference moves lazily as in npa_fwd_kernel.cuh.
//
// Measured with keys and values in DRAM, then in L2: 22.5 and 19.2 us for the size
// above (17 to 18 us of it this kernel, the rest the merge and the launches), 14.8
// and 12.6 us for 2 x 20 heads x 16 queries x 4111 masked 16-bit keys (42 MB, 6.5
// us; 14.1 and 12.0 without a mask), 3.4 us for one query of 10 heads over 77 keys.
#pragma once

#include <cooperative_groups.h>

#include "cross_attention.cuh"

namespace npa {

// Rows up to which this kernel runs: two 8-row tiles. Against xa_fwd_kernel
// with its cut units (keys in L2): 16 x 4111 keys of 2 x 20 heads at d = 64 12.0
// / 21.6 us, of 24 heads at d = 128 14.5 / 18.5; one query of 10 heads x 77 keys
// 3.3 / 6.7; one query x 16384 cached keys of 2 x 20 heads 19.2 / 66.4.
constexpr int kXaFewRows = 16;
constexpr int kXaFewWarps = 4;
constexpr int kXaFewCluster = 8;  // splits that merge inside a cluster at most (the portable size)
// CTAs that run on a multiprocessor at once, by their registers.
__host__ __device__ constexpr int xa_few_per_sm(int d, int row_tiles) { return d == 64 ? (row_tiles == 1 ? 4 : 3) : 2; }

struct XfParams {
    const void *q, *k, *v;
    void *o;
    long long qsb, qsh, qst, ksb, ksh, kst, vsb, vsh, vst, osb, osh, ost;  // strides in elements
    const int *kv_lens;
    const unsigned char *key_mask;
    const float *k_scale, *v_scale;
    int scale_blocks;
    int B, heads, kv_heads, group, Lq, Lk;
    int n_splits;
    int cluster;  // the splits of a unit are one cluster and merge there
    float scale_log2;
    float *o_part, *ml;  // n_splits > 1 without a cluster, as in XaParams
};

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D: head dimension; NT: 8-row tiles (1 or 2). With an 8-bit cache the
// products run in f16 and q, o are bf16.
template <int D, bool KV8, bool F16, int NT>
struct XfWarp {
    static constexpr bool kF16 = KV8 || F16;                 // type of the products
    static constexpr int kStep = !KV8 && D == 128 ? 16 : 32;  // keys of a step: what the registers hold
    static constexpr int kTiles = kStep / 8, kSubs = kStep / 16;
    static constexpr uint32_t kAll = kStep == 32 ? 0xffffffffu : 0xffffu;  // every key of a step is kept
    static constexpr int kKLoads = KV8 ? D / 64 : D / 32;    // 16-byte pieces of a key row per lane
    static constexpr int kVWords = KV8 ? D / 32 : D / 16;    // 32-bit words of a value row per lane
    static constexpr int kMTiles = D / 16;
    // The reference moves to kBelow under a step's maximum that exceeds it by more
    // than kLead. P of a step reaches 2^15 in f16, 2^7 at its own maximum with an
    // 8-bit cache (where nothing but float32 sums is at the reference, and it
    // stays above the largest score: O overflows only where sum p |v| does).
    static constexpr float kLead = KV8 ? 0.f : kF16 ? 15.f : kRescaleLog2;
    static constexpr float kBelow = KV8 ? -4.f : kF16 ? 7.f : 0.f;
    static constexpr float kTop = 7.f;  // 8-bit: log2 of P at a step's maximum

    uint32_t q[D / 16][NT][2];  // [k step][row tile]: a0, a2 (and a1, a3)
    uint4 kr[kTiles][kKLoads];
    uint32_t vr[kSubs][4][kVWords];
    float ks, vs;               // this step's scales
    unsigned char mask_byte;
    float o[NT][kMTiles][4];
    float R[NT], l[NT], f[NT];  // reference, partial sum, scale of row tile n's row g

    // d of accumulator pair jm, half e, for lane group g
    __device__ static __forceinline__ int d_of(int g, int jm, int e) {
        if (KV8 && D == 128) return 16 * g + 2 * jm + e;
        return (jm >> 2) * 64 + 8 * g + 2 * (jm & 3) + e;
    }

    // row: this lane's bytes of the step's key g (load_k) or 2t (load_v);
    // stride: bytes from key to key; n: keys left from the step's first on.
    template <bool kFull>
    __device__ __forceinline__ void load_k(const char *row, long long stride, int n, int g) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < kKLoads; ++j)
                kr[i][j] = kFull || 8 * i + g < n ? __ldg(reinterpret_cast<const uint4 *>(row + 8 * i * stride + j * 64))
                                                  : make_uint4(0, 0, 0, 0);
    }
    template <bool kFull>
    __device__ __forceinline__ void load_v(const char *row, long long stride, int n, int t) {
#pragma unroll
        for (int s = 0; s < kSubs; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 16 * s + (i & 1) + (i >> 1) * 8;  // past 2t
                const bool in = kFull || key + 2 * t < n;
                if constexpr (KV8 && D == 64) {
                    const uint2 x = in ? __ldg(reinterpret_cast<const uint2 *>(row + key * stride)) : make_uint2(0, 0);
                    vr[s][i][0] = x.x;
                    vr[s][i][1] = x.y;
                } else {
#pragma unroll
                    for (int j = 0; j < kVWords / 4; ++j) {
                        const uint4 x = in ? __ldg(reinterpret_cast<const uint4 *>(row + key * stride + j * 128))
                                           : make_uint4(0, 0, 0, 0);
                        vr[s][i][4 * j] = x.x;
                        vr[s][i][4 * j + 1] = x.y;
                        vr[s][i][4 * j + 2] = x.z;
                        vr[s][i][4 * j + 3] = x.w;
                    }
                }
            }
    }

    // S of the step's keys.
    __device__ __forceinline__ void scores(float (&s)[kTiles][4]) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int j = 0; j < kKLoads; ++j) {
                const uint32_t w[4] = {kr[i][j].x, kr[i][j].y, kr[i][j].z, kr[i][j].w};
                if constexpr (KV8) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int k = j * 4 + u;
                        mma_16816<true>(s[i], q[k][0][0], NT > 1 ? q[k][NT - 1][0] : 0u, q[k][0][1],
                                        NT > 1 ? q[k][NT - 1][1] : 0u, sm100::e4m3x2_to_f16x2(w[u]),
                                        sm100::e4m3x2_to_f16x2(w[u] >> 16));
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int k = j * 2 + u;
                        mma_16816<F16>(s[i], q[k][0][0], NT > 1 ? q[k][NT - 1][0] : 0u, q[k][0][1],
                                       NT > 1 ? q[k][NT - 1][1] : 0u, w[2 * u], w[2 * u + 1]);
                    }
                }
            }
        }
    }

    // O^T += V^T P^T for the step, P as packed pairs [row tile][16 keys][2]; to_R
    // (8-bit): from P's reference to O's, of this lane's two rows of each tile.
    __device__ __forceinline__ void products(const uint32_t (&pb)[NT][kSubs][2], const float (&to_R)[NT][2], uint32_t keep,
                                             int t) {
        // values of keys that are not kept: 0 (P is 0 there, but not 0 * NaN)
        if (keep != kAll) {
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!(keep >> (16 * s + 2 * t + (i & 1) + (i >> 1) * 8) & 1u)) {
#pragma unroll
                        for (int j = 0; j < kVWords; ++j) vr[s][i][j] = 0;
                    }
        }
        if constexpr (KV8) {
#pragma unroll
            for (int jw = 0; jw < kVWords; ++jw) {
                float acc[2][NT][4];  // two 16-row tiles of O^T share a word of codes
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[e][n][0] = acc[e][n][1] = acc[e][n][2] = acc[e][n][3] = 0.f;
#pragma unroll
                for (int s = 0; s < kSubs; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // codes of two keys at one d, next to each other
                        const uint32_t lo = __byte_perm(vr[s][0][jw], vr[s][1][jw], e ? 0x7362 : 0x5140);
                        const uint32_t hi = __byte_perm(vr[s][2][jw], vr[s][3][jw], e ? 0x7362 : 0x5140);
                        const uint32_t a0 = sm100::e4m3x2_to_f16x2(lo), a1 = sm100::e4m3x2_to_f16x2(lo >> 16);
                        const uint32_t a2 = sm100::e4m3x2_to_f16x2(hi), a3 = sm100::e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_16816<true>(acc[e][n], a0, a1, a2, a3, pb[n][s][0], pb[n][s][1]);
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            o[n][2 * jw + e][c] = fmaf(vs, acc[e][n][c] * to_R[n][c & 1], o[n][2 * jw + e][c]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
#pragma unroll
                for (int jw = 0; jw < kVWords; ++jw) {
                    const uint32_t a0 = __byte_perm(vr[s][0][jw], vr[s][1][jw], 0x5410);
                    const uint32_t a1 = __byte_perm(vr[s][0][jw], vr[s][1][jw], 0x7632);
                    const uint32_t a2 = __byte_perm(vr[s][2][jw], vr[s][3][jw], 0x5410);
                    const uint32_t a3 = __byte_perm(vr[s][2][jw], vr[s][3][jw], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_16816<F16>(o[n][jw], a0, a1, a2, a3, pb[n][s][0], pb[n][s][1]);
                }
        }
    }
};

template <int D, bool KV8, bool F16, int NT>
__global__ void __launch_bounds__(32 * kXaFewWarps, xa_few_per_sm(D, NT)) xa_few_kernel(const __grid_constant__ XfParams p) {
    using W = XfWarp<D, KV8, F16, NT>;
    sm100::let_next_kernel_start();
    // [warps][8 NT][D] O, then [warps][8 NT][2] reference and sum, then the block's merged [8 NT][2]
    extern __shared__ float xf_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int unit = blockIdx.x / p.n_splits, split = blockIdx.x - unit * p.n_splits;
    const int b = unit / p.kv_heads, kvh = unit - b * p.kv_heads;
    const int rows = p.group * p.Lq;
    const int len = p.kv_lens ? min(max(__ldg(p.kv_lens + b), 0), p.Lk) : p.Lk;
    const long long steps = ((long long)len + W::kStep - 1) / W::kStep;
    const int j1 = int(steps * (split + 1) / p.n_splits);
    int j = int(steps * split / p.n_splits) + warp;
    // bytes from key to key (a cache's rows are contiguous), and this lane's place in the first
    constexpr int kElem = KV8 ? 1 : 2;
    const long long kst = KV8 ? D : p.kst * 2, vst = KV8 ? D : p.vst * 2;
    const char *kb = static_cast<const char *>(p.k) + (b * p.ksb + kvh * p.ksh) * kElem + g * kst + t * 16;
    const char *vb = static_cast<const char *>(p.v) + (b * p.vsb + kvh * p.vsh) * kElem + 2 * t * vst +
                     g * (KV8 && D == 64 ? 8 : 16);
    const float *ks = p.k_scale + (size_t)unit * p.scale_blocks, *vs = p.v_scale + (size_t)unit * p.scale_blocks;
    const unsigned char *mask = p.key_mask ? p.key_mask + (size_t)b * p.Lk : nullptr;

    W w;
    auto load_keys = [&](int step) {
        const int key0 = bound_coord(step * W::kStep, p.Lk), n = len - key0;
        if (n >= W::kStep)
            w.template load_k<true>(kb + key0 * kst, kst, n, g);
        else
            w.template load_k<false>(kb + key0 * kst, kst, n, g);
        if (KV8) w.ks = __ldg(ks + key0 / kKv8Block);
        if (mask) w.mask_byte = lane < min(n, W::kStep) ? __ldg(mask + key0 + lane) : 0;
    };
    auto load_values = [&](int step) {
        const int key0 = bound_coord(step * W::kStep, p.Lk), n = len - key0;
        if (n >= W::kStep)
            w.template load_v<true>(vb + key0 * vst, vst, n, t);
        else
            w.template load_v<false>(vb + key0 * vst, vst, n, t);
        if (KV8) w.vs = __ldg(vs + key0 / kKv8Block);
    };
    if (j < j1) {
        load_keys(j);
        load_values(j);
    }
    // queries: row r is query r % Lq of head kvh * group + r / Lq
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = n * 8 + g;
        const bool in = r < rows;
        const int hd = in ? r / p.Lq : 0, i = in ? r - hd * p.Lq : 0;
        const uint16_t *src = static_cast<const uint16_t *>(p.q) + b * p.qsb + (kvh * p.group + hd) * p.qsh + i * p.qst;
        w.R[n] = -INFINITY;
        w.l[n] = 0.f;
        w.f[n] = p.scale_log2;
        if constexpr (KV8) {
            // 16 elements per lane and 64 of d, exact in f16 after a power of two
            uint4 x[D / 64][2];
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[c][h] = in ? __ldg(reinterpret_cast<const uint4 *>(src + c * 64 + t * 16 + h * 8)) : make_uint4(0, 0, 0, 0);
                    const uint32_t y[4] = {x[c][h].x, x[c][h].y, x[c][h].z, x[c][h].w};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(y[u] << 16)), fabsf(__uint_as_float(y[u] & 0xffff0000u))));
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // exponent of the row's largest, within what has a normal reciprocal
            const int e = amax > 0.f ? min(max(int(__float_as_uint(amax) >> 23) - 127, -126), 126) : 0;
            const float down = __uint_as_float(uint32_t(127 - e) << 23);
            w.f[n] *= __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t y[4] = {x[c][h].x, x[c][h].y, x[c][h].z, x[c][h].w};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        w.q[c * 4 + h * 2 + (u >> 1)][n][u & 1] = sm100::pack_f16x2(
                            __uint_as_float(y[u] << 16) * down, __uint_as_float(y[u] & 0xffff0000u) * down);
                }
        } else {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint4 x = in ? __ldg(reinterpret_cast<const uint4 *>(src + c * 32 + t * 8)) : make_uint4(0, 0, 0, 0);
                w.q[c * 2][n][0] = x.x;
                w.q[c * 2][n][1] = x.y;
                w.q[c * 2 + 1][n][0] = x.z;
                w.q[c * 2 + 1][n][1] = x.w;
            }
        }
#pragma unroll
        for (int m = 0; m < W::kMTiles; ++m) w.o[n][m][0] = w.o[n][m][1] = w.o[n][m][2] = w.o[n][m][3] = 0.f;
    }

    for (; j < j1; j += kXaFewWarps) {
        const bool more = j + kXaFewWarps < j1;
        float s[W::kTiles][4];
        w.scores(s);
        const int left = len - j * W::kStep;
        const uint32_t keep = mask                 ? __ballot_sync(0xffffffffu, w.mask_byte != 0)
                              : left >= W::kStep ? W::kAll
                                                 : (1u << left) - 1u;
        const float kscale = KV8 ? w.ks : 1.f;
        if (KV8 && keep == 0u) w.vs = 0.f;  // no key of the step: its block's scale may be anything
        if (more) load_keys(j + kXaFewWarps);
        if (keep != W::kAll) {
#pragma unroll
            for (int i = 0; i < W::kTiles; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (!(keep >> (8 * i + 2 * t + (c & 1)) & 1u)) s[i][c] = -INFINITY;
        }
        uint32_t pb[NT][W::kSubs][2];
        bool moved = false;
        float alpha[NT], to_R[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < W::kTiles; ++i) mx = sm100::max3(mx, s[i][2 * n], s[i][2 * n + 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // kept above 0: -inf times it stays -inf
            const float f = KV8 ? fmaxf(w.f[n] * kscale, 1.2e-38f) : w.f[n];
            const float bm = mx * f, before = w.R[n];
            if (bm > w.R[n] + W::kLead) w.R[n] = bm - W::kBelow;
            alpha[n] = w.R[n] == before ? 1.f : sm100::ex2_approx(before - w.R[n]);
            moved = moved || w.R[n] != before;
            const float ref = KV8 ? bm - W::kTop : w.R[n], neg = ref == -INFINITY ? 0.f : -ref;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < W::kTiles; ++i) {
                const float p0 = sm100::ex2_approx(fmaf(s[i][2 * n], f, neg));
                const float p1 = sm100::ex2_approx(fmaf(s[i][2 * n + 1], f, neg));
                sum += p0 + p1;
                pb[n][i >> 1][i & 1] = sm100::pack_16x2<W::kF16>(p0, p1);
            }
            if constexpr (KV8) {
                // 0 where every score is -inf, or NaN, which stays
                const float x = ref == -INFINITY ? 0.f : sm100::ex2_approx(ref - w.R[n]);
                to_R[n][0] = __shfl_sync(0xffffffffu, x, 8 * t);
                to_R[n][1] = __shfl_sync(0xffffffffu, x, 8 * t + 4);
                sum *= x;
            }
            w.l[n] = fmaf(w.l[n], alpha[n], sum);
        }
        if (__any_sync(0xffffffffu, moved)) {
            // accumulator columns are rows 2t and 2t + 1 of a row tile
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float a0 = __shfl_sync(0xffffffffu, alpha[n], 8 * t), a1 = __shfl_sync(0xffffffffu, alpha[n], 8 * t + 4);
#pragma unroll
                for (int m = 0; m < W::kMTiles; ++m) {
                    w.o[n][m][0] *= a0;
                    w.o[n][m][1] *= a1;
                    w.o[n][m][2] *= a0;
                    w.o[n][m][3] *= a1;
                }
            }
        }
        w.products(pb, to_R, keep, t);
        if (more) load_values(j + kXaFewWarps);
    }

    // merge the warps
    constexpr int kRows = 8 * NT;
    float *sm_o = xf_smem + (size_t)warp * kRows * D;
    float2 *sm_ml = reinterpret_cast<float2 *>(xf_smem + kXaFewWarps * kRows * D);
    float2 *merged_ml = sm_ml + kXaFewWarps * kRows;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float l = w.l[n];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) sm_ml[warp * kRows + n * 8 + g] = make_float2(w.R[n], l);
#pragma unroll
        for (int m = 0; m < W::kMTiles; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<float2 *>(sm_o + (n * 8 + 2 * t + c) * D + W::d_of(g, m, 0)) =
                    make_float2(w.o[n][m][c], w.o[n][m][2 + c]);
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < rows * (D / 2); idx += 32 * kXaFewWarps) {
        const int r = idx / (D / 2), d = (idx - r * (D / 2)) * 2;
        float2 ml[kXaFewWarps];
        float m = -INFINITY, L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int i = 0; i < kXaFewWarps; ++i) {
            ml[i] = sm_ml[i * kRows + r];
            m = fmaxf(m, ml[i].x);
        }
#pragma unroll
        for (int i = 0; i < kXaFewWarps; ++i) {
            if (ml[i].x == -INFINITY) {  // no keys: 0; or scores that are all NaN: NaN
                L += ml[i].y;
                continue;
            }
            const float wgt = sm100::ex2_approx(ml[i].x - m);
            const float2 o = *reinterpret_cast<const float2 *>(xf_smem + (i * kRows + r) * D + d);
            L = fmaf(wgt, ml[i].y, L);
            x = fmaf(wgt, o.x, x);
            y = fmaf(wgt, o.y, y);
        }
        const int hd = r / p.Lq, i = r - hd * p.Lq, h = kvh * p.group + hd;
        if (p.cluster) {  // (r, d) of the warps' results is read by this thread alone
            *reinterpret_cast<float2 *>(xf_smem + r * D + d) = make_float2(x, y);
            if (d == 0) merged_ml[r] = make_float2(m, L);
        } else if (p.n_splits > 1) {
            const size_t row = ((size_t)b * p.heads + h) * p.Lq + i;
            const size_t part = (size_t)split * p.B * p.heads * p.Lq + row;
            if (!bound_row(true, part, (size_t)p.n_splits * p.B * p.heads * p.Lq)) continue;
            *reinterpret_cast<float2 *>(p.o_part + part * D + d) = make_float2(x, y);
            if (d == 0) *reinterpret_cast<float2 *>(p.ml + part * 2) = make_float2(m, L);
        } else {
            if (!bound_row(true, ((size_t)b * p.heads + h) * p.Lq + i, (size_t)p.B * p.heads * p.Lq)) continue;
            const float inv = L > 0.f ? 1.f / L : L;
            uint16_t *dst = static_cast<uint16_t *>(p.o) + b * p.osb + h * p.osh + i * p.ost + d;
            *reinterpret_cast<uint32_t *>(dst) = L == 0.f ? 0u : sm100::pack_16x2<F16>(x * inv, y * inv);
        }
    }
    if (!p.cluster) return;
    // the splits are the blocks of a cluster: each merges a share of the row
    // elements from everyone's shared memory
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int idx = split * 32 * kXaFewWarps + threadIdx.x; idx < rows * (D / 2); idx += p.n_splits * 32 * kXaFewWarps) {
        const int r = idx / (D / 2), d = (idx - r * (D / 2)) * 2;
        float2 ml[kXaFewCluster], o[kXaFewCluster];
        float m = -INFINITY, L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int i = 0; i < kXaFewCluster; ++i) {
            const bool in = i < p.n_splits;
            ml[i] = in ? *cluster.map_shared_rank(merged_ml + r, i) : make_float2(-INFINITY, 0.f);
            o[i] = in ? *cluster.map_shared_rank(reinterpret_cast<float2 *>(xf_smem + r * D + d), i) : make_float2(0.f, 0.f);
            m = fmaxf(m, ml[i].x);
        }
#pragma unroll
        for (int i = 0; i < kXaFewCluster; ++i) {
            if (ml[i].x == -INFINITY) {  // no keys: 0; or scores that are all NaN: NaN
                L += ml[i].y;
                continue;
            }
            const float wgt = sm100::ex2_approx(ml[i].x - m);
            L = fmaf(wgt, ml[i].y, L);
            x = fmaf(wgt, o[i].x, x);
            y = fmaf(wgt, o[i].y, y);
        }
        const int hd = r / p.Lq, i = r - hd * p.Lq, h = kvh * p.group + hd;
        if (!bound_row(true, ((size_t)b * p.heads + h) * p.Lq + i, (size_t)p.B * p.heads * p.Lq)) continue;
        const float inv = L > 0.f ? 1.f / L : L;
        uint16_t *dst = static_cast<uint16_t *>(p.o) + b * p.osb + h * p.osh + i * p.ost + d;
        *reinterpret_cast<uint32_t *>(dst) = L == 0.f ? 0u : sm100::pack_16x2<F16>(x * inv, y * inv);
    }
    cluster.sync();  // nobody's shared memory goes while it is read
}

}  // namespace npa
