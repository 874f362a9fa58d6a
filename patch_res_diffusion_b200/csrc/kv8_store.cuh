// kv8_store.cuh - writes keys and values into the 8-bit cache
// (npa_kv8_store): e4m3 codes with one scale per 64 tokens and head,
//   s = 2^ceil(log2(amax / 448)),   code = round_to_nearest_even_e4m3(x / s),
// amax the largest finite |x| of the block's written tokens. e4m3 is a
// floating-point format, so a power-of-two scale costs no precision against
// amax / 448 (a block's smallest numbers lie at most one binade lower), x / s
// and code * s are exact in float32. The attention kernels multiply the codes
// in float16, where they are exact, and apply s in float32.
//
// A block that starts inside (the first one, when `start` is not a multiple of
// 64) keeps its earlier tokens: its scale is the larger of the old one and the
// new tokens' (of tokens without a finite number other than 0, the old one), and
// when it grows the earlier codes are rounded again at it.
// Codes past the last written token are left as they were.
//
// One block of 128 threads per (batch, head, 64 tokens, k or v): every element
// is read once, held in registers over the block-wide maximum, and written
// once as 8 codes per store. 26 us for 2 x 10 heads x 16384 tokens x 64 (126 MB,
// 4.8 TB/s, where a copy has 6.6: stores of 8 bytes a thread, issue slots 60%
// busy); one token appended takes 3.5 us, a launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "cross_attention.cuh"

namespace npa {

struct Kv8StoreParams {
    const void *x[2];         // keys, values: 16-bit, strides below
    unsigned char *codes[2];  // [B, heads, capacity, d]
    float *scale[2];          // [B, heads, capacity / 64]
    long long sb[2], sh[2], st[2];
    const int *starts;        // [B] or null: first token of each batch row (else start)
    int start, n, capacity, heads, n_blocks;
    int rows;                 // batch rows times heads
};

// The smallest power of two s (at least 2^-126) with amax / s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ float kv8_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < -126) e = -126;  // subnormal amax included
    return __uint_as_float(uint32_t(e + 127) << 23);
}

// Two floats to two e4m3 codes (nearest even, finite values past 448 and
// infinities to +-448, NaN to the NaN code); `lo` goes to the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint2 kv8_encode(const float (&f)[8], float inv) {
    uint2 c;
    c.x = pack_e4m3x2(f[0] * inv, f[1] * inv) | pack_e4m3x2(f[2] * inv, f[3] * inv) << 16;
    c.y = pack_e4m3x2(f[4] * inv, f[5] * inv) | pack_e4m3x2(f[6] * inv, f[7] * inv) << 16;
    return c;
}

template <bool F16>
__device__ __forceinline__ void unpack_16x8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (F16) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <int D, bool F16>
__global__ void __launch_bounds__(128) kv8_store_kernel(const __grid_constant__ Kv8StoreParams p) {
    constexpr int kPieces = kKv8Block * D / 8 / 128;  // 8-element pieces per thread
    const int t = blockIdx.x & 1;
    const int rest = blockIdx.x >> 1;
    const int bh = rest / p.n_blocks;
    const int b = bh / p.heads, h = bh - b * p.heads;
    const int start = p.starts ? __ldg(p.starts + b) : p.start;
    // tokens [lo, hi) of this row lie inside the cache
    const long long lo = start > 0 ? start : 0;
    const long long end = (long long)start + p.n;
    const long long hi = end < p.capacity ? end : p.capacity;
    const long long blk = lo / kKv8Block + (rest - bh * p.n_blocks);
    const long long t0 = blk * kKv8Block;
    if (t0 >= hi) return;  // uniform over the block
    // (uniform too) the block's tokens and its scale lie in the cache
    if (!bound_row(true, (size_t)bh * p.capacity + t0 + kKv8Block - 1, (size_t)p.rows * p.capacity)) return;
    const uint16_t *x = static_cast<const uint16_t *>(p.x[t]) + b * p.sb[t] + h * p.sh[t];
    unsigned char *codes = p.codes[t] + ((size_t)bh * p.capacity + t0) * D;
    float *scale = p.scale[t] + (size_t)bh * (p.capacity / kKv8Block) + blk;

    uint4 v[kPieces];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int piece = threadIdx.x + 128 * i;
        const long long tok = t0 + piece / (D / 8);
        v[i] = make_uint4(0, 0, 0, 0);
        if (tok >= lo && tok < hi)
            v[i] = __ldg(reinterpret_cast<const uint4 *>(x + (tok - start) * p.st[t] + piece % (D / 8) * 8));
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        float f[8];
        unpack_16x8<F16>(v[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float a = fabsf(f[k]);
            if (a < INFINITY) amax = fmaxf(amax, a);  // false for NaN too
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __shared__ float warp_max[4];
    __shared__ float old_scale;
    const bool inside = t0 < lo;  // earlier tokens of this block stay
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    if (threadIdx.x == 0) old_scale = inside ? *scale : 0.f;
    __syncthreads();
    amax = fmaxf(fmaxf(warp_max[0], warp_max[1]), fmaxf(warp_max[2], warp_max[3]));
    const float old = old_scale;
    float s = amax > 0.f ? kv8_scale(amax) : inside ? old : 1.f;
    // a scale that nobody has set yet may be 0: 1 / s has to be finite
    if (inside) s = fmaxf(fmaxf(s, old), 0x1p-126f);
    const float inv = 1.f / s;
    if (threadIdx.x == 0) *scale = s;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int piece = threadIdx.x + 128 * i;
        const long long tok = t0 + piece / (D / 8);
        uint2 *dst = reinterpret_cast<uint2 *>(codes + piece * 8);
        float f[8];
        if (tok >= lo && tok < hi) {
            unpack_16x8<F16>(v[i], f);
            *dst = kv8_encode(f, inv);
        } else if (inside && tok < lo && s != old) {
            const uint2 c = *dst;
            const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t h2 = sm100::e4m3x2_to_f16x2(w[k]);
                const float2 d2 = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
                f[2 * k] = d2.x * old;
                f[2 * k + 1] = d2.y * old;
            }
            *dst = kv8_encode(f, inv);
        }
    }
}

}  // namespace npa
