// group_norm.cuh - group norm with an activation, channels last
// (npa_group_norm_act):
//   y[b, n, c] = act((x[b, n, c] - mean[b, g]) * rstd[b, g] * w[c] + bias[c]),  g = c / (C / groups),
// mean and variance over the N tokens and the C / groups channels of a group.
// Two kernels: gn_stats_kernel reads x and writes one (mean, M2) pair per
// (batch, group, token tile); gn_apply_kernel merges the tiles' pairs and
// normalises. Nothing is accumulated with atomics, so results do not depend on
// the order in which blocks run.
//
// Statistics are float32 throughout and never a difference of large sums: a
// thread takes the mean and the squared deviations of kBatch values of one
// channel exactly as defined (the values are in registers, so the second pass
// costs no memory), and pairs (n, mean, M2) are merged by
//   mean = sum n_i mean_i / n,   M2 = sum M2_i + sum n_i (mean_i - mean)^2.
//
// A thread owns one 16-byte column of channels (kVec = 8 or 4; 1 where
// alignment or strides forbid it) and walks the tokens of its tile; a block is
// `rows` tokens by `cols` columns, so that neighbouring threads read
// neighbouring channels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kv8_store.cuh"

namespace npa {

struct GnParams {
    const void *x;
    void *y;
    const void *w, *bias;  // null: 1 and 0
    int w_f32;             // w, bias are float32 (else of x's type)
    long long xsb, xst, ysb, yst;  // batch and token strides, elements
    int N, G, cpg;         // tokens, groups, channels per group
    int c0, cw;            // channels of this launch: [c0, c0 + cw), whole groups
    int cols, rows;        // block shape: columns (of kVec channels) x tokens
    int stat_tiles, stat_rows;    // token tiles of the statistics and tokens in each
    int apply_tiles, apply_rows;  // and of the normalisation
    float eps;
    int silu;
    float2 *part;          // [B][G][stat_tiles] (mean, M2)
};

// Threads of a block at most, and values of one channel taken at a time.
constexpr int kGnThreads = 512;
constexpr int kGnMaxChannels = 4096;  // the statistics keep two floats per channel in shared memory
constexpr int kGnBatch = 8;

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

template <typename T, int kVec>
__global__ void __launch_bounds__(kGnThreads) gn_stats_kernel(const __grid_constant__ GnParams p) {
    using V = GnVec<T, kVec>;
    extern __shared__ float gn_smem[];  // [rows][cw] mean, [rows][cw] M2, [rows] count
    float *sm_mean = gn_smem, *sm_m2 = gn_smem + (size_t)p.rows * p.cw, *sm_n = sm_m2 + (size_t)p.rows * p.cw;
    let_next_kernel_start();
    const int tile = blockIdx.x, b = blockIdx.y;
    const int tx = threadIdx.x % p.cols, ty = threadIdx.x / p.cols;
    const int r0 = tile * p.stat_rows, r1 = min(p.N, r0 + p.stat_rows);
    if (ty < p.rows) {
        int n = 0;
        for (int col = tx; col * kVec < p.cw; col += p.cols) {
            const T *src = static_cast<const T *>(p.x) + b * p.xsb + p.c0 + col * kVec;
            float mean[kVec], m2[kVec];
#pragma unroll
            for (int k = 0; k < kVec; ++k) mean[k] = m2[k] = 0.f;
            n = 0;
            for (int r = r0 + ty; r < r1; r += p.rows * kGnBatch) {
                typename V::Raw raw[kGnBatch];
#pragma unroll
                for (int i = 0; i < kGnBatch; ++i)
                    if (r + i * p.rows < r1)
                        raw[i] = *reinterpret_cast<const typename V::Raw *>(src + (long long)(r + i * p.rows) * p.xst);
                if (r + (kGnBatch - 1) * p.rows < r1) {
                    float s[kVec], d2[kVec];
#pragma unroll
                    for (int k = 0; k < kVec; ++k) s[k] = d2[k] = 0.f;
#pragma unroll
                    for (int i = 0; i < kGnBatch; ++i) {
                        float f[kVec];
                        V::widen(raw[i], f);
#pragma unroll
                        for (int k = 0; k < kVec; ++k) s[k] += f[k];
                    }
#pragma unroll
                    for (int k = 0; k < kVec; ++k) s[k] *= 1.f / kGnBatch;
#pragma unroll
                    for (int i = 0; i < kGnBatch; ++i) {
                        float f[kVec];
                        V::widen(raw[i], f);
#pragma unroll
                        for (int k = 0; k < kVec; ++k) d2[k] = fmaf(f[k] - s[k], f[k] - s[k], d2[k]);
                    }
                    const float share = float(kGnBatch) / float(n + kGnBatch);
                    const float cross = share * float(n);
#pragma unroll
                    for (int k = 0; k < kVec; ++k) {
                        const float d = s[k] - mean[k];
                        mean[k] = fmaf(d, share, mean[k]);
                        m2[k] += fmaf(d * d, cross, d2[k]);
                    }
                    n += kGnBatch;
                } else {
#pragma unroll
                    for (int i = 0; i < kGnBatch; ++i) {
                        if (r + i * p.rows >= r1) break;
                        float f[kVec];
                        V::widen(raw[i], f);
                        const float share = 1.f / float(n + 1);
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
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                sm_mean[(size_t)ty * p.cw + col * kVec + k] = mean[k];
                sm_m2[(size_t)ty * p.cw + col * kVec + k] = m2[k];
            }
        }
        if (tx == 0) sm_n[ty] = float(n);
    }
    __syncthreads();
    // the kernels this one may have overtaken are complete before it is, so
    // that a later kernel's wait for this one covers them as well
    wait_for_previous_kernel();
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const float inv_n = 1.f / (float(r1 - r0) * float(p.cpg));
    const int entries = p.rows * p.cpg;
    for (int g = threadIdx.x >> 5; g * p.cpg < p.cw; g += warps) {
        float s = 0.f;
        for (int i = lane; i < entries; i += 32) {
            const int y = i / p.cpg;
            s = fmaf(sm_n[y], sm_mean[(size_t)y * p.cw + g * p.cpg + i - y * p.cpg], s);
        }
        const float mean = warp_sum(s) * inv_n;
        float m2 = 0.f;
        for (int i = lane; i < entries; i += 32) {
            const int y = i / p.cpg;
            const size_t at = (size_t)y * p.cw + g * p.cpg + i - y * p.cpg;
            const float d = sm_mean[at] - mean;
            m2 += sm_n[y] > 0.f ? fmaf(sm_n[y] * d, d, sm_m2[at]) : 0.f;
        }
        m2 = warp_sum(m2);
        if (lane == 0)
            p.part[((size_t)b * p.G + p.c0 / p.cpg + g) * p.stat_tiles + tile] = make_float2(mean, m2);
    }
}

template <typename T>
__device__ __forceinline__ float gn_weight(const void *w, int f32, int c) {
    return f32 ? __ldg(static_cast<const float *>(w) + c) : float(static_cast<const T *>(w)[c]);
}

__device__ __forceinline__ float silu(float y) { return __fdividef(y, 1.f + __expf(-y)); }

template <typename T, int kVec>
__global__ void __launch_bounds__(kGnThreads) gn_apply_kernel(const __grid_constant__ GnParams p) {
    using V = GnVec<T, kVec>;
    extern __shared__ float gn_smem[];  // [groups of this launch] mean, rstd
    const int ng = p.cw / p.cpg;
    float *sm_mean = gn_smem, *sm_rstd = gn_smem + ng;
    let_next_kernel_start();
    const int tile = blockIdx.x, b = blockIdx.y;
    wait_for_previous_kernel();
    // merge the statistics' tiles: one warp per group
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int g = threadIdx.x >> 5; g < ng; g += warps) {
        const float2 *part = p.part + ((size_t)b * p.G + p.c0 / p.cpg + g) * p.stat_tiles;
        const float total = float(p.N);
        float s = 0.f;
        for (int t = lane; t < p.stat_tiles; t += 32)
            s = fmaf(float(min(p.stat_rows, p.N - t * p.stat_rows)), part[t].x, s);
        const float mean = warp_sum(s) / total;
        float m2 = 0.f;
        for (int t = lane; t < p.stat_tiles; t += 32) {
            const float2 q = part[t];
            const float d = q.x - mean;
            m2 += fmaf(float(min(p.stat_rows, p.N - t * p.stat_rows)) * float(p.cpg) * d, d, q.y);
        }
        m2 = warp_sum(m2);
        if (lane == 0) {
            sm_mean[g] = mean;
            sm_rstd[g] = rsqrtf(m2 / (total * float(p.cpg)) + p.eps);
        }
    }
    __syncthreads();
    const int tx = threadIdx.x % p.cols, ty = threadIdx.x / p.cols;
    if (ty >= p.rows) return;
    const int r0 = tile * p.apply_rows, r1 = min(p.N, r0 + p.apply_rows);
    for (int col = tx; col * kVec < p.cw; col += p.cols) {
        const int c = p.c0 + col * kVec;
        float mean[kVec], a[kVec], bias[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int g = (col * kVec + k) / p.cpg;
            mean[k] = sm_mean[g];
            a[k] = sm_rstd[g] * (p.w ? gn_weight<T>(p.w, p.w_f32, c + k) : 1.f);
            bias[k] = p.bias ? gn_weight<T>(p.bias, p.w_f32, c + k) : 0.f;
        }
        const T *src = static_cast<const T *>(p.x) + b * p.xsb + c;
        T *dst = static_cast<T *>(p.y) + b * p.ysb + c;
        constexpr int kB = 4;  // tokens in flight
        for (int r = r0 + ty; r < r1; r += p.rows * kB) {
            typename V::Raw raw[kB];
#pragma unroll
            for (int i = 0; i < kB; ++i)
                if (r + i * p.rows < r1)
                    raw[i] = *reinterpret_cast<const typename V::Raw *>(src + (long long)(r + i * p.rows) * p.xst);
#pragma unroll
            for (int i = 0; i < kB; ++i) {
                if (r + i * p.rows >= r1) break;
                float f[kVec];
                V::widen(raw[i], f);
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    f[k] = fmaf(f[k] - mean[k], a[k], bias[k]);
                    if (p.silu) f[k] = silu(f[k]);
                }
                *reinterpret_cast<typename V::Raw *>(dst + (long long)(r + i * p.rows) * p.yst) = V::narrow(f);
            }
        }
    }
}

}  // namespace npa
