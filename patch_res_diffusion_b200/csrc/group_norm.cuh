// group_norm.cuh - group norm with an activation, channels last
// (npa_group_norm_act):
//   y[b, n, c] = act((x[b, n, c] - mean[b, g]) * rstd[b, g] * w[c] + bias[c]),  g = c / (C / groups),
// mean and variance over the N tokens and the C / groups channels of a group.
// Bound by memory: x read once and y written once. Two kernels reach that:
//
//  * gn_cluster_kernel: a cluster of up to 8 blocks holds a chunk of whole
//    groups of one batch row in its shared memory, exchanges the groups'
//    statistics through distributed shared memory and normalises from there.
//    One launch, one pass over x. Taken when the chunk fits.
//  * gn_step_kernel: otherwise the work is cut into items (a few batch rows, or
//    a channel chunk of one) small enough to stay in L2 between their two
//    passes. Launch s takes the statistics of item s and normalises item s - 1,
//    so reading new data from memory and writing results overlap; a launch
//    starts under the end of the one before it (programmatic serialisation)
//    and waits for it only between its two halves.
//
// Nothing is accumulated with atomics: results do not depend on the order in
// which blocks run. Statistics are float32 throughout and never a difference
// of large sums: a thread takes the mean and the squared deviations of kBatch
// values of one channel as defined (the values are in registers, so the second
// pass costs no memory), and pairs (n, mean, M2) are merged by
//   mean = sum n_i mean_i / n,   M2 = sum M2_i + sum n_i (mean_i - mean)^2.
//
// A thread owns one 16-byte column of channels (kVec = 8 or 4; 1 where
// alignment or strides forbid it) and walks the tokens of its tile; a block is
// `rows` tokens by `cols` columns, so that neighbouring threads read
// neighbouring channels.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kv8_store.cuh"

namespace npa {

constexpr int kGnThreads = 512;        // threads of a block at most
constexpr int kGnMaxChannels = 4096;   // the block's statistics are kept in shared memory
constexpr int kGnMaxTiles = 320;       // token tiles of an item at most: ten per lane when they are merged
constexpr int kGnMaxCluster = 8;       // the portable cluster size

struct GnParams {
    const void *x;
    void *y;
    const void *w, *bias;  // null: 1 and 0
    int w_f32;             // w, bias are float32 (else of x's type)
    long long xsb, xst, ysb, yst;  // batch and token strides, elements
    int N, G, cpg;         // tokens, groups, channels per group
    int cw;                // channels of a chunk: whole groups
    int cols, rows;        // block shape: columns (of kVec channels) x tokens
    int segs;              // groups that kVec neighbouring channels touch at most
    int tiles, tile_rows;  // token tiles (gn_cluster_kernel: blocks of the cluster) and tokens in each
    float eps;
    int silu;
    // gn_step_kernel: batch rows and first channel of the item whose
    // statistics are taken and of the one that is normalised (rows 0: none)
    int stat_b, stat_nb, stat_c, apply_b, apply_nb, apply_c;
    float2 *part;          // [B][G][tiles] (mean, M2)
};

template <typename T, int kVec>
struct GnVec;
template <>
struct GnVec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void widen(Raw v, float (&f)[8]) { unpack_16x8<false>(v, f); }
    static __device__ __forceinline__ Raw narrow(const float (&f)[8]) {
        return make_uint4(sm100::pack_bf16x2(f[0], f[1]), sm100::pack_bf16x2(f[2], f[3]),
                          sm100::pack_bf16x2(f[4], f[5]), sm100::pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct GnVec<__half, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void widen(Raw v, float (&f)[8]) { unpack_16x8<true>(v, f); }
    static __device__ __forceinline__ Raw narrow(const float (&f)[8]) {
        return make_uint4(sm100::pack_f16x2(f[0], f[1]), sm100::pack_f16x2(f[2], f[3]),
                          sm100::pack_f16x2(f[4], f[5]), sm100::pack_f16x2(f[6], f[7]));
    }
};
template <>
struct GnVec<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ void widen(Raw v, float (&f)[4]) {
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
    static __device__ __forceinline__ Raw narrow(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <typename T>
struct GnVec<T, 1> {
    using Raw = T;
    static __device__ __forceinline__ void widen(Raw v, float (&f)[1]) { f[0] = float(v); }
    static __device__ __forceinline__ Raw narrow(const float (&f)[1]) { return T(f[0]); }
};

// Waits until the kernels before this one on the stream are complete (launched
// with programmatic serialisation, a kernel starts before that).
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Mean and squared deviations of each of a thread's kVec channels, merged over
// the values it has seen.
template <int kVec>
struct GnAcc {
    float mean[kVec], m2[kVec];
    int n = 0;
    __device__ __forceinline__ GnAcc() {
#pragma unroll
        for (int k = 0; k < kVec; ++k) mean[k] = m2[k] = 0.f;
    }
    template <typename V, int kBatch>
    __device__ __forceinline__ void add(const typename V::Raw (&raw)[kBatch], int valid) {
        if (valid >= kBatch) {
            float s[kVec], d2[kVec];
#pragma unroll
            for (int k = 0; k < kVec; ++k) s[k] = d2[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float f[kVec];
                V::widen(raw[i], f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) s[k] += f[k];
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k) s[k] *= 1.f / kBatch;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float f[kVec];
                V::widen(raw[i], f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) d2[k] = fmaf(f[k] - s[k], f[k] - s[k], d2[k]);
            }
            const float share = __fdividef(float(kBatch), float(n + kBatch));
            const float cross = share * float(n);
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const float d = s[k] - mean[k];
                mean[k] = fmaf(d, share, mean[k]);
                m2[k] += fmaf(d * d, cross, d2[k]);
            }
            n += kBatch;
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i >= valid) break;
                float f[kVec];
                V::widen(raw[i], f);
                const float share = __fdividef(1.f, float(n + 1));
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    const float d = f[k] - mean[k];
                    mean[k] = fmaf(d, share, mean[k]);
                    m2[k] = fmaf(d, f[k] - mean[k], m2[k]);
                }
                ++n;
            }
        }
    }
    // One entry (mean, M2) for each group that column `col` touches.
    __device__ __forceinline__ void store(const GnParams &p, int col, float2 *entry) const {
        const int g0 = col * kVec / p.cpg;
        for (int s = 0; s < p.segs; ++s) {
            const int lo = (g0 + s) * p.cpg - col * kVec, hi = lo + p.cpg;  // the group's channels of this column
            float sum = 0.f, cnt = 0.f;
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                if (k >= lo && k < hi) {
                    sum += mean[k];
                    cnt += 1.f;
                }
            const float mu = cnt > 0.f ? __fdividef(sum, cnt) : 0.f;
            float q = 0.f;
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                if (k >= lo && k < hi) q += fmaf(float(n) * (mean[k] - mu), mean[k] - mu, m2[k]);
            entry[s] = make_float2(mu, q);
        }
    }
};

// (mean, M2) of one group over a tile of `tokens` tokens, from the block's
// entries [rows][columns of the chunk][segs]. One warp; every lane gets them.
template <int kVec>
__device__ __forceinline__ float2 gn_group_of_block(const GnParams &p, const float2 *entry, int g, int tokens) {
    const int lane = threadIdx.x & 31;
    const int v0 = g * p.cpg / kVec, v1 = ((g + 1) * p.cpg - 1) / kVec, nv = v1 - v0 + 1;
    const int ncol = p.cw / kVec, entries = p.rows * nv;
    float s = 0.f;
    for (int i = lane; i < entries; i += 32) {
        const int y = i / nv, v = v0 + i - y * nv;
        const int ch = min((v + 1) * kVec, (g + 1) * p.cpg) - max(v * kVec, g * p.cpg);
        const int n = (tokens - y + p.rows - 1) / p.rows;
        s = fmaf(float(n * ch), entry[((size_t)y * ncol + v) * p.segs + g - v * kVec / p.cpg].x, s);
    }
    const float mean = warp_sum(s) / (float(tokens) * float(p.cpg));
    float m2 = 0.f;
    for (int i = lane; i < entries; i += 32) {
        const int y = i / nv, v = v0 + i - y * nv;
        const int ch = min((v + 1) * kVec, (g + 1) * p.cpg) - max(v * kVec, g * p.cpg);
        const int n = (tokens - y + p.rows - 1) / p.rows;
        const float2 e = entry[((size_t)y * ncol + v) * p.segs + g - v * kVec / p.cpg];
        const float d = e.x - mean;
        m2 += fmaf(float(n * ch) * d, d, e.y);
    }
    return make_float2(mean, warp_sum(m2));
}

template <typename T>
__device__ __forceinline__ float gn_weight(const void *w, int f32, int c) {
    return f32 ? __ldg(static_cast<const float *>(w) + c) : float(static_cast<const T *>(w)[c]);
}

__device__ __forceinline__ float silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }

// What a thread needs to normalise its column.
template <typename T, int kVec>
struct GnAffine {
    float mean[kVec], a[kVec], bias[kVec];
    int act;
    __device__ __forceinline__ GnAffine(const GnParams &p, const float *sm_mean, const float *sm_rstd, int col, int c0)
        : act(p.silu) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int g = (col * kVec + k) / p.cpg, c = c0 + col * kVec + k;
            mean[k] = sm_mean[g];
            a[k] = sm_rstd[g] * (p.w ? gn_weight<T>(p.w, p.w_f32, c) : 1.f);
            bias[k] = p.bias ? gn_weight<T>(p.bias, p.w_f32, c) : 0.f;
        }
    }
    __device__ __forceinline__ typename GnVec<T, kVec>::Raw operator()(typename GnVec<T, kVec>::Raw raw) const {
        float f[kVec];
        GnVec<T, kVec>::widen(raw, f);
#pragma unroll
        for (int k = 0; k < kVec; ++k) f[k] = fmaf(f[k] - mean[k], a[k], bias[k]);
        if (act) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) f[k] = silu(f[k]);
        }
        return GnVec<T, kVec>::narrow(f);
    }
};

// ---------------------------------------------------------------------------
// A chunk in a cluster's shared memory
// ---------------------------------------------------------------------------
// Grid (cluster blocks, channel chunks, batch rows). Shared memory: the
// block's tokens, 16 bytes per thread and step (a thread reads back what it
// wrote itself), then the entries, the cluster's pairs [blocks][groups], and
// mean and rstd [groups].
template <typename T, int kVec>
__global__ void __launch_bounds__(kGnThreads) gn_cluster_kernel(const __grid_constant__ GnParams p) {
    using V = GnVec<T, kVec>;
    using Raw = typename V::Raw;
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ uint4 gn_smem16[];
    const int ng = p.cw / p.cpg, threads = p.cols * p.rows;
    const int steps = (p.tile_rows + p.rows - 1) / p.rows;
    Raw *slab = reinterpret_cast<Raw *>(gn_smem16);
    float2 *entry = reinterpret_cast<float2 *>(slab + (size_t)steps * threads);
    float2 *pairs = entry + (size_t)p.rows * (p.cw / kVec) * p.segs;
    float *sm_mean = reinterpret_cast<float *>(pairs + (size_t)p.tiles * ng), *sm_rstd = sm_mean + ng;

    // the other blocks' shared memory is written below: they have to be there
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int rank = blockIdx.x, b = blockIdx.z, c0 = blockIdx.y * p.cw;
    const int tx = threadIdx.x % p.cols, ty = threadIdx.x / p.cols;
    const int r0 = rank * p.tile_rows, tokens = max(0, min(p.tile_rows, p.N - r0));
    constexpr int kBatch = 8;
    const int mine = ty < p.rows ? (tokens - ty + p.rows - 1) / p.rows : 0;  // this thread's tokens
    const long long xstep = (long long)p.rows * p.xst;
    if (ty < p.rows) {
        const T *src = static_cast<const T *>(p.x) + b * p.xsb + c0 + tx * kVec + (long long)(r0 + ty) * p.xst;
        GnAcc<kVec> acc;
        for (int k = 0; k < mine; k += kBatch) {
            Raw raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (k + i < mine) raw[i] = *reinterpret_cast<const Raw *>(src + (k + i) * xstep);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (k + i < mine) slab[(size_t)(k + i) * threads + threadIdx.x] = raw[i];
            acc.template add<V>(raw, mine - k);
        }
        acc.store(p, tx, entry + ((size_t)ty * p.cols + tx) * p.segs);
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int g = threadIdx.x >> 5; g < ng; g += warps) {
        const float2 q = tokens > 0 ? gn_group_of_block<kVec>(p, entry, g, tokens) : make_float2(0.f, 0.f);
        if (lane < p.tiles) cluster.map_shared_rank(pairs, lane)[rank * ng + g] = q;
    }
    cluster.sync();
    for (int g = threadIdx.x; g < ng; g += blockDim.x) {
        const float total = float(p.N);
        float s = 0.f, m2 = 0.f;
        for (int t = 0; t < p.tiles; ++t)
            s = fmaf(float(max(0, min(p.tile_rows, p.N - t * p.tile_rows))), pairs[t * ng + g].x, s);
        const float mean = s / total;
        for (int t = 0; t < p.tiles; ++t) {
            const float2 q = pairs[t * ng + g];
            const float d = q.x - mean;
            m2 += fmaf(float(max(0, min(p.tile_rows, p.N - t * p.tile_rows))) * float(p.cpg) * d, d, q.y);
        }
        sm_mean[g] = mean;
        sm_rstd[g] = rsqrtf(m2 / (total * float(p.cpg)) + p.eps);
    }
    __syncthreads();
    if (ty >= p.rows) return;
    const GnAffine<T, kVec> f(p, sm_mean, sm_rstd, tx, c0);
    T *dst = static_cast<T *>(p.y) + b * p.ysb + c0 + tx * kVec + (long long)(r0 + ty) * p.yst;
#pragma unroll 4
    for (int k = 0; k < mine; ++k)
        *reinterpret_cast<Raw *>(dst + (long long)k * p.rows * p.yst) = f(slab[(size_t)k * threads + threadIdx.x]);
}

// ---------------------------------------------------------------------------
// Items through L2
// ---------------------------------------------------------------------------
template <typename T, int kVec>
__global__ void __launch_bounds__(kGnThreads, 2) gn_step_kernel(const __grid_constant__ GnParams p) {
    using V = GnVec<T, kVec>;
    using Raw = typename V::Raw;
    constexpr int kBatch = 4;  // tokens in flight per thread
    extern __shared__ uint4 gn_smem16[];  // statistics: the entries; normalisation: mean and rstd [groups of the item]
    let_next_kernel_start();
    const int tile = blockIdx.x;
    const int tx = threadIdx.x % p.cols, ty = threadIdx.x / p.cols;
    const int r0 = tile * p.tile_rows, r1 = min(p.N, r0 + p.tile_rows);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, ng = p.cw / p.cpg;
    float2 *entry = reinterpret_cast<float2 *>(gn_smem16);
    const bool stat = blockIdx.y < p.stat_nb;
    if (stat) {
        const T *x = static_cast<const T *>(p.x) + (p.stat_b + blockIdx.y) * p.xsb + p.stat_c;
        for (int col = tx; ty < p.rows && col * kVec < p.cw; col += p.cols) {
            const T *src = x + col * kVec;
            GnAcc<kVec> acc;
            for (int r = r0 + ty; r < r1; r += p.rows * kBatch) {
                Raw raw[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (r + i * p.rows < r1)
                        raw[i] = *reinterpret_cast<const Raw *>(src + (long long)(r + i * p.rows) * p.xst);
                acc.template add<V>(raw, (r1 - r + p.rows - 1) / p.rows);
            }
            acc.store(p, col, entry + ((size_t)ty * (p.cw / kVec) + col) * p.segs);
        }
        __syncthreads();
    }
    // everything launched before is complete: the previous launch's statistics
    // can be read, and a launch that waits for this one waits for those too
    wait_for_previous_kernel();
    if (stat) {
        float2 *out = p.part + ((size_t)(p.stat_b + blockIdx.y) * p.G + p.stat_c / p.cpg) * p.tiles + tile;
        for (int g = threadIdx.x >> 5; g < ng; g += warps) {
            const float2 q = gn_group_of_block<kVec>(p, entry, g, r1 - r0);
            if (lane == 0) out[(size_t)g * p.tiles] = q;
        }
        __syncthreads();
    }
    if (blockIdx.y >= p.apply_nb) return;
    float *sm_mean = reinterpret_cast<float *>(gn_smem16), *sm_rstd = sm_mean + ng;
    const int b = p.apply_b + blockIdx.y;
    for (int g = threadIdx.x >> 5; g < ng; g += warps) {
        const float2 *part = p.part + ((size_t)b * p.G + p.apply_c / p.cpg + g) * p.tiles;
        constexpr int kPer = kGnMaxTiles / 32;
        float2 q[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) q[i] = lane + 32 * i < p.tiles ? part[lane + 32 * i] : make_float2(0.f, 0.f);
        const float total = float(p.N);
        float s = 0.f, m2 = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            s = fmaf(float(max(0, min(p.tile_rows, p.N - (lane + 32 * i) * p.tile_rows))), q[i].x, s);
        const float mean = warp_sum(s) / total;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float d = q[i].x - mean;
            m2 += fmaf(float(max(0, min(p.tile_rows, p.N - (lane + 32 * i) * p.tile_rows))) * float(p.cpg) * d, d, q[i].y);
        }
        m2 = warp_sum(m2);
        if (lane == 0) {
            sm_mean[g] = mean;
            sm_rstd[g] = rsqrtf(m2 / (total * float(p.cpg)) + p.eps);
        }
    }
    __syncthreads();
    if (ty >= p.rows) return;
    for (int col = tx; col * kVec < p.cw; col += p.cols) {
        const GnAffine<T, kVec> f(p, sm_mean, sm_rstd, col, p.apply_c);
        const T *src = static_cast<const T *>(p.x) + b * p.xsb + p.apply_c + col * kVec;
        T *dst = static_cast<T *>(p.y) + b * p.ysb + p.apply_c + col * kVec;
        for (int r = r0 + ty; r < r1; r += p.rows * kBatch) {
            Raw raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (r + i * p.rows < r1)
                    raw[i] = __ldcs(reinterpret_cast<const Raw *>(src + (long long)(r + i * p.rows) * p.xst));
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (r + i * p.rows < r1)
                    __stcs(reinterpret_cast<Raw *>(dst + (long long)(r + i * p.rows) * p.yst), f(raw[i]));
        }
    }
}

}  // namespace npa
