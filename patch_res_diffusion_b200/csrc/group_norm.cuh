// group_norm.cuh - group norm with an activation, channels last
// (npa_group_norm_act):
//   y[b, n, c] = act((x[b, n, c] - mean[b, g]) * rstd[b, g] * w[c] + bias[c]),  g = c / (C / groups),
// mean and variance over the N tokens and the C / groups channels of a group.
// Bound by memory: x read once and y written once at best.
//
//  * gn_cluster_kernel: a cluster of up to 8 blocks holds a chunk of whole
//    groups of one batch row in its shared memory, exchanges the groups'
//    statistics through distributed shared memory and normalises from there.
//    One launch, one pass over x. Taken when the chunk fits.
//  * otherwise gn_stats_kernel (x read, a pair for each token tile and group),
//    gn_merge_kernel (the tiles of a group merged) and gn_apply_kernel (x read
//    again, y written). The last one walks the tokens from the end, so that
//    what the first one read last is still in L2. A launch starts under the end
//    of the one before it (programmatic serialisation) and loads its first
//    tokens before it waits for that one. Cutting x into items that stay in L2
//    between the passes was slower: 258 us instead of 182 for [2, 262144, 320]
//    bf16, whose items of 42 MB leave each launch too little to do.
//    179 us for that size: 64 for the statistics (5.4 TB/s), 110 for the rest
//    (6.1 TB/s), where one pass that cannot be had would take 102.
//    26 us for [2, 16384, 320] in float32 (84 MB, 12.8 us; both passes from L2),
//    36 us for [2, 16384, 321] in bf16, one element to a load (42 MB).
//    The cluster form takes 11 us for [2, 1024, 1280] in float16.
//
// Nothing is accumulated with atomics: results do not depend on the order in
// which blocks run. Statistics are float32 throughout. A thread sums x - K and
// (x - K)^2 of a channel, K the mean of that channel's first kGnBatch values it
// sees, and takes M2 = sum (x - K)^2 - (sum (x - K))^2 / n. The subtraction
// loses at most n (K - mean)^2 2^-24, and since K is the mean of kGnBatch
// members, the group's M2 is at least kGnBatch (K - mean)^2: n is kept to
// kGnRun, so the loss is below 2^-17 of M2 even for the worst data. Pairs
// (n, mean, M2) are then merged by
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
#include <type_traits>

#include "kv8_store.cuh"

namespace npa {

constexpr int kGnThreads = 256;        // threads of a block at most
constexpr int kGnMaxChannels = 4096;   // the block's statistics are kept in shared memory
constexpr int kGnMaxTiles = 512;       // token tiles of a batch row at most
constexpr int kGnMaxCluster = 8;       // the portable cluster size
constexpr int kGnBatch = 4;            // tokens that a thread takes at a time
constexpr int kGnLanes = 8;            // lanes that merge one group's channels
constexpr int kGnRun = 512;            // values that share one shift K at most

// n / d for 0 <= n < 2^16 and 1 <= d < 2^16: with m = floor(2^32 / d) + 1 the
// product's error n (d - 2^32 mod d) / d stays below 2^32 / d.
struct SmallDiv {
    uint32_t m;  // 0: d = 1
    __host__ __device__ SmallDiv() : m(0) {}
    __host__ __device__ explicit SmallDiv(int d) : m(d > 1 ? uint32_t((1ull << 32) / d) + 1 : 0) {}
    __device__ __forceinline__ int operator()(int n) const { return m ? int(__umulhi(uint32_t(n), m)) : n; }
};

struct GnParams {
    const void *x;
    void *y;
    const void *w, *bias;  // null: 1 and 0
    int w_f32;             // w, bias are float32 (else of x's type)
    long long xsb, xst, ysb, yst;  // batch and token strides, elements
    int N, G, cpg;         // tokens, groups, channels per group
    int cw;                // channels of a chunk: whole groups (all but in gn_cluster_kernel)
    int cols, rows;        // block shape: columns (of kVec channels) x tokens
    SmallDiv by_cols, by_cpg;
    int tiles, tile_rows;  // token tiles of the statistics (gn_cluster_kernel: blocks of the cluster), tokens in each
    float eps;
    int silu;
    int apply_tiles, apply_rows;  // token tiles of the normalisation and tokens in each
    float2 *part;          // [B][G][tiles] (mean, M2)
    float2 *mean_rstd;     // [B][G]
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

// Sum over kLanes neighbouring lanes.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of a thread's kVec channels; its entries (mean, M2) in shared memory
// take one run of at most kGnRun values after the other.
template <int kVec>
struct GnAcc {
    float shift[kVec], sum[kVec], square[kVec];  // K, sum (x - K), sum (x - K)^2
    float2 *entry;
    int n = 0, run = 0;  // values in the entries; in the current run
    __device__ __forceinline__ explicit GnAcc(float2 *e) : entry(e) {}
    // kCount more values of each channel.
    template <typename V, int kCount>
    __device__ __forceinline__ void add(const typename V::Raw *raw) {
        if (run == 0) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) shift[k] = sum[k] = square[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kCount; ++i) {
                float f[kVec];
                V::widen(raw[i], f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) shift[k] = fmaf(f[k], 1.f / kCount, shift[k]);
            }
        }
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            float f[kVec];
            V::widen(raw[i], f);
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const float d = f[k] - shift[k];
                sum[k] += d;
                square[k] = fmaf(d, d, square[k]);
            }
        }
        run += kCount;
        if (run >= kGnRun) flush();
    }
    __device__ __forceinline__ void flush() {
        if (run == 0) {  // no values at all: entries of weight 0
            if (n > 0) return;
#pragma unroll
            for (int k = 0; k < kVec; ++k) entry[k] = make_float2(0.f, 0.f);
            return;
        }
        const float inv = __fdividef(1.f, float(run));
        const float share = __fdividef(float(run), float(n + run)), cross = share * float(n);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const float d = sum[k] * inv, mean = d + shift[k], m2 = fmaf(-sum[k], d, square[k]);
            float2 old = make_float2(mean, 0.f);
            if (n) old = entry[k];
            const float e = mean - old.x;
            entry[k] = make_float2(fmaf(e, share, old.x), old.y + fmaf(e * e, cross, m2));
        }
        n += run;
        run = 0;
    }
};

// body(g, lane) for g = 0 .. n - 1, kGnLanes neighbouring threads to a group.
// Every thread of a warp runs the same number of rounds (with the last group
// again where there is none left), so body may exchange values between lanes.
template <typename Body>
__device__ __forceinline__ void for_groups(int n, Body body) {
    const int per_round = blockDim.x / kGnLanes;
    for (int g0 = 0; g0 < n; g0 += per_round)
        body(min(g0 + int(threadIdx.x) / kGnLanes, n - 1), int(threadIdx.x) % kGnLanes);
}

// From a block's entries [rows][cw + 1] (mean, M2) over a tile of `tokens`
// tokens: emit(g, lane, pair) for every group of the chunk, by each of its
// lanes. First the rows of a channel are merged (into its row 0), by one
// thread or, where there are many rows, by kGnLanes, then kGnLanes threads
// merge the channels of a group.
template <int kLanes>
__device__ __forceinline__ void gn_merge_rows(const GnParams &p, float2 *entry, int tokens, int c, int lane) {
    const int base = tokens / p.rows, more = tokens - base * p.rows;  // tokens of row y: base, one more for y < more
    const float n0 = float(base), n1 = float(base + 1);
    float s = 0.f, m2 = 0.f;
#pragma unroll 4
    for (int y = lane; y < p.rows; y += kLanes) s = fmaf(y < more ? n1 : n0, entry[y * (p.cw + 1) + c].x, s);
    const float mean = lanes_sum<kLanes>(s) / float(tokens);
#pragma unroll 4
    for (int y = lane; y < p.rows; y += kLanes) {
        const float2 q = entry[y * (p.cw + 1) + c];
        const float d = q.x - mean;
        m2 += fmaf((y < more ? n1 : n0) * d, d, q.y);
    }
    m2 = lanes_sum<kLanes>(m2);
    if (lane == 0) entry[c] = make_float2(mean, m2);
}

template <typename Emit>
__device__ __forceinline__ void gn_groups_of_block(const GnParams &p, float2 *entry, int tokens, Emit emit) {
    __syncthreads();
    if (p.rows > kGnLanes) {
        const int per_round = blockDim.x / kGnLanes, c = int(threadIdx.x) / kGnLanes, lane = int(threadIdx.x) % kGnLanes;
        // the channels past the last are read and written by nobody, but take part in the exchange
        for (int c0 = 0; c0 < p.cw; c0 += per_round)
            gn_merge_rows<kGnLanes>(p, entry, c0 + c < p.cw ? tokens : 1, min(c0 + c, p.cw), lane);
    } else {
        for (int c = threadIdx.x; c < p.cw; c += blockDim.x) gn_merge_rows<1>(p, entry, tokens, c, 0);
    }
    __syncthreads();
    const float inv_cpg = 1.f / float(p.cpg);
    for_groups(p.by_cpg(p.cw), [&](int g, int lane) {
        const float2 *e = entry + g * p.cpg;
        float s = 0.f, m2 = 0.f;
        for (int c = lane; c < p.cpg; c += kGnLanes) s += e[c].x;
        const float mean = lanes_sum<kGnLanes>(s) * inv_cpg;
        for (int c = lane; c < p.cpg; c += kGnLanes) {
            const float d = e[c].x - mean;
            m2 += fmaf(float(tokens) * d, d, e[c].y);
        }
        emit(g, lane, make_float2(mean, lanes_sum<kGnLanes>(m2)));
    });
}

// (mean, rstd) of a group from its pairs over p.tiles <= kLanes * kPer tiles,
// by kLanes neighbouring lanes. Tiles hold p.tile_rows tokens, the one at
// p.N's end fewer, any after it none.
template <int kLanes, int kPer>
__device__ __forceinline__ float2 gn_merge_tiles(const GnParams &p, const float2 *pair, int pitch, int lane) {
    float2 q[kPer];
    float w[kPer], s = 0.f, m2 = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int t = lane + kLanes * i;
        q[i] = t < p.tiles ? pair[(size_t)t * pitch] : make_float2(0.f, 0.f);
        w[i] = t < p.tiles ? float(min(max(p.N - t * p.tile_rows, 0), p.tile_rows)) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) s = fmaf(w[i], q[i].x, s);
    const float mean = lanes_sum<kLanes>(s) / float(p.N);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float d = q[i].x - mean;
        m2 += w[i] > 0.f ? fmaf(w[i] * float(p.cpg) * d, d, q[i].y) : 0.f;
    }
    return make_float2(mean, rsqrtf(lanes_sum<kLanes>(m2) / (float(p.N) * float(p.cpg)) + p.eps));
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a thread needs to normalise its column: weight and bias are read early,
// the statistics come later.
template <typename T, int kVec>
struct GnAffine {
    float a[kVec], bias[kVec];  // y = x a + bias
    __device__ __forceinline__ void weights(const GnParams &p, int col, int c0) {
        const int c = c0 + col * kVec;
#pragma unroll
        for (int k = 0; k < kVec; ++k) a[k] = 1.f, bias[k] = 0.f;
        if (p.w_f32) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                if (p.w) a[k] = __ldg(static_cast<const float *>(p.w) + c + k);
                if (p.bias) bias[k] = __ldg(static_cast<const float *>(p.bias) + c + k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                if (p.w) a[k] = float(static_cast<const T *>(p.w)[c + k]);
                if (p.bias) bias[k] = float(static_cast<const T *>(p.bias)[c + k]);
            }
        }
    }
    // mean_rstd: of the chunk's groups. x a - mean a costs no more precision
    // than the mean's own rounding.
    __device__ __forceinline__ void statistics(const GnParams &p, const float2 *mean_rstd, int col) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const float2 s = mean_rstd[p.by_cpg(col * kVec + k)];
            a[k] *= s.y;
            bias[k] = fmaf(-s.x, a[k], bias[k]);
        }
    }
    static __device__ __forceinline__ float pair(const float (&u)[kVec], int i) {
        if constexpr (kVec > 1) return u[2 * i] * u[2 * i + 1];
        return u[0];
    }
    template <bool kSilu>
    __device__ __forceinline__ typename GnVec<T, kVec>::Raw apply(typename GnVec<T, kVec>::Raw raw) const {
        float f[kVec];
        GnVec<T, kVec>::widen(raw, f);
#pragma unroll
        for (int k = 0; k < kVec; ++k) f[k] = fmaf(f[k], a[k], bias[k]);
        if constexpr (kSilu) {
            // z / (1 + e^-z), two to a reciprocal: 1 / u = v / (u v). The power
            // is kept below 2^63 so that u v is finite; where that would show,
            // z e^z is the same to 2^-62 (and -0 for the largest -z).
            constexpr int kPairs = (kVec + 1) / 2;
            float u[kVec], uv[kPairs], most = 0.f;
#pragma unroll
            for (int k = 0; k < kVec; ++k) u[k] = 1.f + sm100::ex2_approx(fminf(-1.4426950408889634f * f[k], 63.f));
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                uv[i] = pair(u, i);
                most = fmaxf(most, uv[i]);
            }
            if (most > 0x1p60f) {  // rare
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    if (f[k] < -43.f) {
                        // in two factors: ex2.approx has no results below 2^-126
                        const float h = sm100::ex2_approx(0.5f * 1.4426950408889634f * f[k]);
                        f[k] *= h;
                        f[k] *= h;
                        u[k] = 1.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < kPairs; ++i) uv[i] = pair(u, i);
            }
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const float r = rcp_approx(uv[i]);
                if constexpr (kVec > 1) {
                    f[2 * i] *= r * u[2 * i + 1];
                    f[2 * i + 1] *= r * u[2 * i];
                } else {
                    f[0] *= r;
                }
            }
        }
        return GnVec<T, kVec>::narrow(f);
    }
};

// ---------------------------------------------------------------------------
// Asynchronous copies of 16 bytes into a thread's own shared memory slots
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy16_async(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------------------
// A chunk in a cluster's shared memory
// ---------------------------------------------------------------------------
// Grid (cluster blocks, channel chunks, batch rows). Shared memory: the
// block's tokens, 16 bytes per thread and step, then the entries, the
// cluster's pairs [blocks][groups], and (mean, rstd) [groups].
template <typename T, int kVec>
__global__ void __launch_bounds__(kGnThreads) gn_cluster_kernel(const __grid_constant__ GnParams p) {
    using V = GnVec<T, kVec>;
    using Raw = typename V::Raw;
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ uint4 gn_smem16[];
    const int ng = p.by_cpg(p.cw), threads = p.cols * p.rows;
    const int steps = p.tile_rows / p.rows;
    Raw *slab = reinterpret_cast<Raw *>(gn_smem16);
    float2 *entry = reinterpret_cast<float2 *>(slab + (size_t)steps * threads);
    float2 *pairs = entry + (size_t)p.rows * (p.cw + 1);
    float2 *mean_rstd = pairs + (size_t)p.tiles * ng;

    // the other blocks' shared memory is written below: they have to be there
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int rank = blockIdx.x, b = blockIdx.z, c0 = blockIdx.y * p.cw;
    const int ty = p.by_cols(threadIdx.x), tx = threadIdx.x - ty * p.cols;
    const int r0 = rank * p.tile_rows, tokens = max(0, min(p.tile_rows, p.N - r0));
    const int mine = ty < p.rows ? (tokens - ty + p.rows - 1) / p.rows : 0;  // this thread's tokens
    constexpr int kGroup = 8, kAhead = 4;  // tokens of a copy group, groups in flight
    slab += threadIdx.x;
    GnAffine<T, kVec> f;
    if (ty < p.rows) {
        const long long step = (long long)p.rows * p.xst;
        const T *src = static_cast<const T *>(p.x) + b * p.xsb + c0 + tx * kVec + (long long)(r0 + ty) * p.xst;
        auto fetch = [&](int k) {
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
                if (k + i < mine) copy16_async(slab + (size_t)(k + i) * threads, src + (k + i) * step);
            copy_commit();
        };
#pragma unroll
        for (int a = 0; a < kAhead; ++a) fetch(a * kGroup);
        f.weights(p, tx, c0);
        GnAcc<kVec> acc(entry + (size_t)ty * (p.cw + 1) + tx * kVec);
        for (int k = 0; k < mine; k += kGroup) {
            copy_wait<kAhead - 1>();
            const Raw *at = slab + (size_t)k * threads;
            const int left = min(mine - k, kGroup);
            if (left == kGroup) {
                Raw raw[kGroup];
#pragma unroll
                for (int i = 0; i < kGroup; ++i) raw[i] = at[(size_t)i * threads];
                acc.template add<V, kGroup>(raw);
            } else {
                for (int i = 0; i < left; ++i, at += threads) acc.template add<V, 1>(at);
            }
            fetch(k + kAhead * kGroup);
        }
        acc.flush();
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    // a block without tokens counts with weight 0
    gn_groups_of_block(p, entry, max(tokens, 1), [&](int g, int lane, float2 q) {
        if (lane < p.tiles) cluster.map_shared_rank(pairs, lane)[rank * ng + g] = q;
    });
    cluster.sync();
    for_groups(ng, [&](int g, int lane) {
        const float2 q = gn_merge_tiles<kGnLanes, kGnMaxCluster / kGnLanes>(p, pairs + g, ng, lane);
        if (lane == 0) mean_rstd[g] = q;
    });
    __syncthreads();
    if (ty >= p.rows || !bound_row(true, c0 + tx * kVec + kVec - 1, (size_t)p.G * p.cpg)) return;
    f.statistics(p, mean_rstd, tx);
    T *dst = static_cast<T *>(p.y) + b * p.ysb + c0 + tx * kVec + (long long)(r0 + ty) * p.yst;
    const long long step = (long long)p.rows * p.yst;
    auto write = [&](auto silu) {
#pragma unroll 4
        for (int k = 0; k < mine; ++k, dst += step, slab += threads)
            if (bound_row(true, (size_t)r0 + ty + (size_t)k * p.rows, p.N))
                *reinterpret_cast<Raw *>(dst) = f.template apply<decltype(silu)::value>(*slab);
    };
    if (p.silu)
        write(std::true_type{});
    else
        write(std::false_type{});
}

// ---------------------------------------------------------------------------
// Three launches
// ---------------------------------------------------------------------------
// Grid (token tiles, batch rows). Shared memory: the entries.
template <typename T, int kVec>
__global__ void __launch_bounds__(kGnThreads, 3) gn_stats_kernel(const __grid_constant__ GnParams p) {
    using V = GnVec<T, kVec>;
    using Raw = typename V::Raw;
    extern __shared__ uint4 gn_smem16[];
    float2 *entry = reinterpret_cast<float2 *>(gn_smem16);
    sm100::let_next_kernel_start();
    const int tile = blockIdx.x, b = blockIdx.y;
    const int ty = p.by_cols(threadIdx.x), tx = threadIdx.x - ty * p.cols;
    const int r0 = tile * p.tile_rows, tokens = min(p.N - r0, p.tile_rows);
    const T *src = static_cast<const T *>(p.x) + b * p.xsb + tx * kVec + (long long)(r0 + ty) * p.xst;
    const long long step = (long long)p.rows * p.xst;
    for (int col = tx; ty < p.rows && col * kVec < p.cw; col += p.cols, src += p.cols * kVec) {
        GnAcc<kVec> acc(entry + (size_t)ty * (p.cw + 1) + col * kVec);
        const T *at = src;
        int left = (tokens - ty + p.rows - 1) / p.rows;  // this thread's tokens
        Raw raw[kGnBatch], next[kGnBatch];               // the next batch is on its way while one is summed
        auto fetch = [&](Raw(&to)[kGnBatch]) {
#pragma unroll
            for (int i = 0; i < kGnBatch; ++i, at += step) to[i] = *reinterpret_cast<const Raw *>(at);
        };
        if (left >= kGnBatch) fetch(raw);
        for (; left >= kGnBatch; left -= kGnBatch) {
            if (left >= 2 * kGnBatch) fetch(next);
            acc.template add<V, kGnBatch>(raw);
#pragma unroll
            for (int i = 0; i < kGnBatch; ++i) raw[i] = next[i];
        }
        for (; left > 0; --left, at += step) {
            const Raw one = *reinterpret_cast<const Raw *>(at);
            acc.template add<V, 1>(&one);
        }
        acc.flush();
    }
    float2 *out = p.part + (size_t)b * p.G * p.tiles + tile;
    gn_groups_of_block(p, entry, tokens, [&](int g, int lane, float2 q) {
        if (bound_row(lane == 0, (size_t)g * p.tiles + tile, (size_t)p.G * p.tiles)) out[(size_t)g * p.tiles] = q;
    });
}

// One warp to a (batch row, group).
__global__ void __launch_bounds__(128) gn_merge_kernel(const __grid_constant__ GnParams p, int n) {
    sm100::let_next_kernel_start();
    const int g = blockIdx.x * 4 + (threadIdx.x >> 5);
    sm100::wait_for_previous_kernel();
    if (g >= n) return;
    const float2 q = gn_merge_tiles<32, kGnMaxTiles / 32>(p, p.part + (size_t)g * p.tiles, 1, threadIdx.x & 31);
    if ((threadIdx.x & 31) == 0) p.mean_rstd[g] = q;
}

// Grid (token tiles, batch rows), both from the end.
template <typename T, int kVec>
__global__ void __launch_bounds__(kGnThreads, 3) gn_apply_kernel(const __grid_constant__ GnParams p) {
    using V = GnVec<T, kVec>;
    using Raw = typename V::Raw;
    sm100::let_next_kernel_start();
    const int ty = p.by_cols(threadIdx.x), tx = threadIdx.x - ty * p.cols;
    const int r0 = (gridDim.x - 1 - blockIdx.x) * p.apply_rows, tokens = min(p.N - r0, p.apply_rows);
    const int b = gridDim.y - 1 - blockIdx.y;
    const T *src = static_cast<const T *>(p.x) + b * p.xsb + tx * kVec + (long long)(r0 + ty) * p.xst;
    T *out = static_cast<T *>(p.y) + b * p.ysb + tx * kVec + (long long)(r0 + ty) * p.yst;
    const long long xstep = (long long)p.rows * p.xst, ystep = (long long)p.rows * p.yst;
    const float2 *mean_rstd = p.mean_rstd + (size_t)b * p.G;
    bool waited = false;
    for (int col = tx; ty < p.rows && col * kVec < p.cw; col += p.cols, src += p.cols * kVec, out += p.cols * kVec) {
        const T *at = src;
        T *dst = out;
        int left = (tokens - ty + p.rows - 1) / p.rows;
        // its last token and channel lie in the tensor
        if (!bound_row(left > 0, (size_t)r0 + ty + (size_t)(left - 1) * p.rows, p.N) ||
            !bound_row(true, (size_t)col * kVec + kVec - 1, (size_t)p.G * p.cpg))
            left = 0;
        Raw raw[kGnBatch], next[kGnBatch];  // the next batch is on its way while one is written
        auto fetch = [&](Raw(&to)[kGnBatch]) {
#pragma unroll
            for (int i = 0; i < kGnBatch; ++i, at += xstep) to[i] = __ldcs(reinterpret_cast<const Raw *>(at));
        };
        if (left >= kGnBatch) fetch(raw);
        GnAffine<T, kVec> f;
        f.weights(p, col, 0);
        if (!waited) sm100::wait_for_previous_kernel();
        waited = true;
        f.statistics(p, mean_rstd, col);
        auto write = [&](auto silu) {
            constexpr bool kSilu = decltype(silu)::value;
            for (; left >= kGnBatch; left -= kGnBatch) {
                if (left >= 2 * kGnBatch) fetch(next);
#pragma unroll
                for (int i = 0; i < kGnBatch; ++i, dst += ystep)
                    __stcs(reinterpret_cast<Raw *>(dst), f.template apply<kSilu>(raw[i]));
#pragma unroll
                for (int i = 0; i < kGnBatch; ++i) raw[i] = next[i];
            }
            for (; left > 0; --left, at += xstep, dst += ystep)
                __stcs(reinterpret_cast<Raw *>(dst), f.template apply<kSilu>(__ldcs(reinterpret_cast<const Raw *>(at))));
        };
        if (p.silu)
            write(std::true_type{});
        else
            write(std::false_type{});
    }
}

}  // namespace npa
