// cross_attention_short.cuh - cross attention to at most 128 keys (a text
// encoder's 77 tokens and the like), 16-bit keys: xa_short_kernel.
//
// With so few keys a query row costs more to move than to compute: 4 d bytes
// in and out against 4 d Lk products, so the bound is memory (51 us for 2 x 10
// heads x 65536 queries x 77 keys at d = 64). The kernel is built to keep many
// query tiles moving: keys and values of a (batch, head) are loaded once and
// stay in shared memory while the CTA walks that head's tiles, and NW
// warpgroups work on tiles of their own, each with its own issuing warp, Q
// buffers, tensor memory and barriers. A warpgroup's tile is one pass without a
// running maximum: S = Q K^T, softmax of the whole row, O = P V. A tile's chain
// of waits is long, but NW chains overlap on a multiprocessor.
//
// Warps: 4 * NW compute (NW = 4 at d = 64, 2 at d = 128), NW issuers (one
// thread each: query loads, products, output stores), then one that loads keys
// and values, clears unkept value rows and publishes which keys are kept. An
// issuer starts the next tile's S before it stores this one's output.
// TMEM per warpgroup: S in columns 0..127; P over S's first 64; O in 64..127
// (d = 64, over S: every row of it has been read when P V starts) or 128..255.
// O leaves through the tile's own Q buffer, which the S product has read.
//
// Measured: 87 us for the size above (3.9 TB/s; the general kernel took 155, two
// warpgroups that issue for themselves 107). No unit is busy more than 45% of
// the time: what is left is each tile's chain (load, S, softmax, P V, store),
// of which a multiprocessor has four under way (S of a fifth would fit in the
// tensor memory for 77 keys, its P beside O would not). With 154 keys (two
// blocks) the general kernel runs: 17 us for 2 x 10 heads x 4096 queries, d = 64.
#pragma once

#include "cross_attention.cuh"

namespace npa {

// Keys up to which this kernel runs: one S of the tensor memory's 128 columns.
// Against xa_fwd_kernel: 87 / 155 us for 77 keys (2 x 10 heads x 65536 queries).
constexpr int kXaShortKeys = 128;

template <int D>
struct XsCfg {
    static constexpr int NW = D == 64 ? 4 : 2;
    static constexpr int kChunks = D / 64;
    static constexpr int kChunkBytes = 128 * 128;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    // d = 64: six warpgroups (the issuers and the loader have one each), and
    // the compute ones take the others' registers; d = 128: three.
    static constexpr int kThreads = D == 64 ? 768 : 384;
    static constexpr int kIssueWarp = NW * 4, kLoadWarp = D == 64 ? 20 : 10;
    static constexpr bool kSplitRegs = D == 64;
    static constexpr uint32_t kRegsLaunch = D == 64 ? 80 : 168, kRegsCompute = 104, kRegsOther = 32;
    static_assert(!kSplitRegs || 128 * (4 * kRegsCompute + 2 * kRegsOther) <= kThreads * kRegsLaunch, "register split");
    static constexpr int kTmemCols = 512;
    static constexpr int kColsPerWg = 512 / NW;
    static constexpr int kColO = D == 64 ? 64 : 128;
    // shared memory: Q [NW][2], then the key/value stages (sized by the key count), then this
    static constexpr int kQBytes = NW * 2 * kTileBytes;
    static constexpr int bKVFull = 0;            // [2] copies landed
    static constexpr int bKVReady = 2;           // [2] unkept rows cleared, kept keys published
    static constexpr int bKVEmpty = 4;           // [2] NW arrivals
    static constexpr int bQFull = 6;             // [NW][2]
    static constexpr int bS = bQFull + 2 * NW;   // [NW] S written (MMA commit)
    static constexpr int bP = bS + NW;           // [NW] P written (128 arrivals)
    static constexpr int bO = bP + NW;           // [NW] O written (MMA commit)
    static constexpr int bE = bO + NW;           // [NW] O staged (128 arrivals)
    static constexpr int bSet = bE + NW;         // [NW] the issuer has moved to another key/value set
    static constexpr int bDrain = bSet + NW;     // [NW]
    static constexpr int kNumBars = bDrain + NW;
    static constexpr int kMiscBytes = kNumBars * 8 + 16 + 2 * 32;  // barriers; TMEM base and abort flag; kept keys
    __host__ __device__ static constexpr int kv_stage_bytes(int rows) { return 2 * kChunks * rows * 128; }
    static constexpr int smem_bytes(int rows, int stages) {
        return kQBytes + stages * kv_stage_bytes(rows) + kMiscBytes + 1024;
    }
};

struct XsParams {
    XaParams a;      // tm_q, tm_o: boxes of 128 rows; tm_k, tm_v: boxes of kv_rows rows
    int kv_rows;     // keys rounded up to 16
    int kv_stages;   // 1 or 2
    int n_qtiles;    // ceil(Lq / 128)
    int n_tiles;     // B * heads * n_qtiles
    FastDiv by_qtiles;
};

// The tiles [first, last) of this CTA: contiguous, so that most of them share
// keys and values.
__device__ __forceinline__ void xs_tiles(const XsParams &p, int *first, int *last) {
    const int base = p.n_tiles / gridDim.x, more = p.n_tiles - base * gridDim.x;
    const int c = blockIdx.x;
    *first = c * base + min(c, more);
    *last = *first + base + (c < more);
}

template <int D>
__device__ void xs_loader(const XsParams &p, uint8_t *kv, uint64_t *bars, uint32_t *kept, volatile uint32_t *abort_flag) {
    using C = XsCfg<D>;
    const uint64_t lim = p.a.wait_limit_ns;
    const int lane = threadIdx.x & 31;
    int t0, t1;
    xs_tiles(p, &t0, &t1);
    const int bh0 = p.by_qtiles(t0), n_bh = p.by_qtiles(t1 - 1) - bh0 + 1;
    const int stage_bytes = C::kv_stage_bytes(p.kv_rows), half = stage_bytes / 2, chunk = p.kv_rows * 128;
    int issued = 0;
    bool ok = true;
    auto load = [&](int seq) {  // one lane
        const int s = seq % p.kv_stages;
        const int bh = bh0 + seq, b = p.a.by_heads(bh), h = p.a.by_group(bh - b * p.a.heads);
        const int kb = bound_coord(b, p.a.B), kh = bound_coord(h, p.a.kv_heads);
        uint8_t *dst = kv + s * stage_bytes;
        sm100::mbar_arrive_expect_tx(&bars[C::bKVFull + s], stage_bytes);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
            sm100::tma_load_4d(dst + c * chunk, &p.a.tm_k, &bars[C::bKVFull + s], c * 64, 0, kh * p.a.k_h, kb * p.a.k_b);
            sm100::tma_load_4d(dst + half + c * chunk, &p.a.tm_v, &bars[C::bKVFull + s], c * 64, 0, kh * p.a.v_h,
                               kb * p.a.v_b);
        }
    };
    for (int seq = 0; seq < n_bh; ++seq) {
        // stages are filled ahead as they become free
        while (issued < n_bh && issued < seq + p.kv_stages) {
            const int s = issued % p.kv_stages, use = issued / p.kv_stages;
            ok = use == 0 || sm100::mbar_wait(&bars[C::bKVEmpty + s], (use - 1) & 1, lim);
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            if (!ok) break;
            if (lane == 0) load(issued);
            ++issued;
        }
        if (!ok) break;
        const int s = seq % p.kv_stages;
        ok = __all_sync(0xffffffffu, sm100::mbar_wait(&bars[C::bKVFull + s], (seq / p.kv_stages) & 1, lim));
        if (!ok) break;
        XaUnit u;
        u.b = p.a.by_heads(bh0 + seq);
        u.len = p.a.kv_lens ? min(max(__ldg(p.a.kv_lens + u.b), 0), p.a.Lk) : p.a.Lk;
        uint32_t w[4];
        xa_keep(p.a, u, 0, u.len, w);
        if (lane < 4) kept[s * 8 + lane] = lane == 0 ? w[0] : lane == 1 ? w[1] : lane == 2 ? w[2] : w[3];
        if (lane == 4) kept[s * 8 + 4] = u.len;
        if (p.a.kv_lens || p.a.key_mask) {  // 0 * NaN would reach the sums through the product
            uint8_t *v = kv + s * stage_bytes + half;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int row = 32 * c + lane;
                if (row < p.kv_rows && !(w[c] >> lane & 1)) {
#pragma unroll
                    for (int i = 0; i < 8 * C::kChunks; ++i)
                        *reinterpret_cast<uint4 *>(v + (i >> 3) * chunk + row * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            sm100::fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&bars[C::bKVReady + s]);
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
    // every issued copy must have landed before the CTA may exit
    for (int s = 0; s < p.kv_stages; ++s)
        if (issued > s) sm100::mbar_wait(&bars[C::bKVFull + s], ((issued - 1 - s) / p.kv_stages) & 1, lim);
}

// One thread per warpgroup: query loads, products and output stores of its tiles.
template <int D, bool F16>
__device__ void xs_issue(const XsParams &p, uint8_t *smem, uint8_t *kv, uint64_t *bars, const uint32_t *kept,
                         uint32_t tmem0, volatile uint32_t *abort_flag, int wg) {
    using C = XsCfg<D>;
    const uint64_t lim = p.a.wait_limit_ns;
    const uint32_t tmem = tmem0 + wg * C::kColsPerWg;
    uint8_t *q0 = smem + wg * 2 * C::kTileBytes;
    const int stage_bytes = C::kv_stage_bytes(p.kv_rows), half = stage_bytes / 2, chunk = p.kv_rows * 128;
    const uint64_t q_desc = sm100::sdesc_sw128(sm100::smem_u32(q0), 16, 1024);
    const uint64_t k_desc = sm100::sdesc_sw128(sm100::smem_u32(kv), 16, 1024);
    const uint64_t v_desc = sm100::sdesc_sw128(sm100::smem_u32(kv + half), chunk, 1024);
    int t0, t1;
    xs_tiles(p, &t0, &t1);
    const int bh0 = p.by_qtiles(t0), last_seq = p.by_qtiles(t1 - 1) - bh0;
    auto load_q = [&](int t, int buf) {
        const int bh = p.by_qtiles(t), b = p.a.by_heads(bh);
        const int qb = bound_coord(b, p.a.B), qh = bound_coord(bh - b * p.a.heads, p.a.heads);
        uint64_t *bar = &bars[C::bQFull + 2 * wg + buf];
        sm100::mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
            sm100::tma_load_4d(q0 + buf * C::kTileBytes + c * C::kChunkBytes, &p.a.tm_q, bar, c * 64,
                               bound_coord((t - bh * p.n_qtiles) * 128, p.a.Lq), qh * p.a.q_h, qb * p.a.q_b);
    };
    auto store_o = [&](int t, int buf) {
        const int bh = p.by_qtiles(t), b = p.a.by_heads(bh);
        const int ob = bound_coord(b, p.a.B), oh = bound_coord(bh - b * p.a.heads, p.a.heads);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
            sm100::tma_store_4d(&p.a.tm_o, q0 + buf * C::kTileBytes + c * C::kChunkBytes, c * 64,
                                bound_coord((t - bh * p.n_qtiles) * 128, p.a.Lq), oh, ob);
        sm100::bulk_commit();
    };
    int loaded = 0;  // Q tiles asked for
    for (int t = t0 + wg; t < t1 && loaded < 2; t += C::NW, ++loaded) load_q(t, loaded);
    if (wg == 0) sm100::tma_prefetch_desc(&p.a.tm_o);
    int seq = -1;      // key/value set in use, counted from the CTA's first
    int i = 0, m = 0;  // tiles begun; tiles with keys begun
    bool ok = true;
    // moves on to key/value set `to`, releasing the ones before it
    auto advance = [&](int to) {
        while (ok && seq < to) {
            if (seq >= 0) sm100::mbar_arrive(&bars[C::bKVEmpty + seq % p.kv_stages]);
            ++seq;
            ok = sm100::mbar_wait(&bars[C::bKVReady + seq % p.kv_stages], (seq / p.kv_stages) & 1, lim);
        }
    };
    constexpr uint32_t kIdS0 =
        F16 ? sm100::idesc_f16_f32(128, 0, false, false) : sm100::idesc_bf16_f32(128, 0, false, false);
    constexpr uint32_t kIdO =
        F16 ? sm100::idesc_f16_f32(128, D, false, true) : sm100::idesc_bf16_f32(128, D, false, true);
    for (int t = t0 + wg;; t += C::NW, ++i) {
        const bool more = t < t1;
        const int set = more ? p.by_qtiles(t) - bh0 : seq;
        const uint64_t q = q_desc + uint64_t(((i & 1) * C::kTileBytes) >> 4);
        if (more) ok = ok && sm100::mbar_wait(&bars[C::bQFull + 2 * wg + (i & 1)], (i >> 1) & 1, lim);
        // the previous tile's output is staged: its tensor memory is free
        if (i > 0) ok = ok && sm100::mbar_wait(&bars[C::bE + wg], (i - 1) & 1, lim);
        if (!ok || *abort_flag) {
            ok = false;
            break;
        }
        if (set != seq) {
            advance(set);
            if (!ok) break;
            sm100::mbar_arrive(&bars[C::bSet + wg]);
        }
        const int stage = seq % p.kv_stages;
        const int n = more ? int(kept[stage * 8 + 4]) : 0;
        const uint64_t v = v_desc + uint64_t((stage * stage_bytes) >> 4);
        if (n > 0) {
            const uint32_t id = kIdS0 | (uint32_t((n + 15) >> 4) << 18);
            const uint64_t k = k_desc + uint64_t((stage * stage_bytes) >> 4);
            sm100::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                sm100::mma_ss(tmem, q + uint64_t(((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4),
                              k + uint64_t(((kk >> 2) * chunk + (kk & 3) * 32) >> 4), id, kk > 0 ? 1u : 0u);
            sm100::tc_commit(&bars[C::bS + wg]);
        }
        if (i > 0) {
            store_o(t - C::NW, (i - 1) & 1);
            if (t + C::NW < t1) {  // the tile after next, into the buffer that this store has read
                sm100::bulk_wait_read();
                load_q(t + C::NW, (i - 1) & 1);
                ++loaded;
            }
        }
        if (!more) break;
        if (n > 0) {
            ok = sm100::mbar_wait(&bars[C::bP + wg], m & 1, lim);
            if (!ok) break;
            sm100::tc_fence_after();
            const int steps = (n + 15) >> 4;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                if (kk < steps)
                    sm100::mma_ts(tmem + C::kColO, tmem + kk * 8, v + uint64_t((kk * 2048) >> 4), kIdO, kk > 0 ? 1u : 0u);
            sm100::tc_commit(&bars[C::bO + wg]);
            ++m;
        }
    }
    advance(last_seq);
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
    // products and copies in flight end, stores complete
    sm100::tc_commit(&bars[C::bDrain + wg]);
    sm100::mbar_wait(&bars[C::bDrain + wg], 0, lim);
    for (int k = i; k < loaded; ++k) sm100::mbar_wait(&bars[C::bQFull + 2 * wg + (k & 1)], (k >> 1) & 1, lim);
    sm100::bulk_wait_all();
}

// W scores of a row from TMEM, unkept ones as -inf.
template <int W>
__device__ __forceinline__ void xs_scores(uint32_t t_s, uint32_t keep, float (&s)[W]) {
    uint32_t r[W];
    if constexpr (W == 32)
        sm100::tmem_ld32(t_s, r);
    else
        sm100::tmem_ld16(t_s, r);
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] = __uint_as_float(r[i]);
    if ((keep | (W == 32 ? 0u : 0xffff0000u)) != 0xffffffffu) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (!(keep >> i & 1u)) s[i] = -INFINITY;
    }
}

template <int W>
__device__ __forceinline__ float xs_max(const float (&s)[W]) {
    float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int i = 4; i + 4 < W; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = sm100::max3(m[k], s[i + k], s[i + 4 + k]);
    if (W % 8 == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], s[W - 4 + k]);
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <int D, bool F16>
__device__ void xs_compute(const XsParams &p, uint8_t *smem, uint64_t *bars, const uint32_t *kept, uint32_t tmem0,
                           volatile uint32_t *abort_flag, int wg) {
    using C = XsCfg<D>;
    const uint64_t lim = p.a.wait_limit_ns;
    const int row = threadIdx.x & 127, warp = row >> 5;
    const uint32_t t_row = tmem0 + wg * C::kColsPerWg + (uint32_t(warp) * 32u << 16);
    const float c2 = p.a.scale_log2;
    int t0, t1;
    xs_tiles(p, &t0, &t1);
    const int bh0 = p.by_qtiles(t0);
    int seq = -1, i = 0, m = 0;  // as in xs_issue
    int sets = 0;                // sets used so far
    bool ok = true;
    for (int t = t0 + wg; t < t1; t += C::NW, ++i) {
        const int bh = p.by_qtiles(t);
        const int row0 = (t - bh * p.n_qtiles) * 128;
        if (seq != bh - bh0) {
            // The issuer says when: it walks every set, and it is never more
            // than this tile ahead. The set's own barrier could be a phase or
            // more away from the one wanted, where sets between are skipped.
            // The set is not released before the tile is done.
            seq = bh - bh0;
            ok = warp_wait(&bars[C::bSet + wg], (sets++) & 1, lim);
            if (!ok) break;
        }
        const uint32_t *keep = kept + seq % p.kv_stages * 8;
        const int n = int(keep[4]);
        const bool active = row0 + warp * 32 < p.a.Lq && n > 0;  // some row of this warp is a query with keys
        float l = 0.f;
        if (n > 0) {
            ok = warp_wait(&bars[C::bS + wg], m & 1, lim);
            if (!ok) break;
            sm100::tc_fence_after();
            if (active) {
                // whole 32-key pieces, then the rest as one of 16 or 32
                const int rest = n & 31, pieces = (n >> 5) + (rest > 16);
                const bool half = rest > 0 && rest <= 16;
                float mx = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < pieces; ++c) {
                    float s[32];
                    xs_scores<32>(t_row + 32 * c, keep[c], s);
                    mx = fmaxf(mx, xs_max<32>(s));
                }
                float tail[16];
                if (half) {
                    xs_scores<16>(t_row + 32 * pieces, keep[pieces], tail);
                    mx = fmaxf(mx, xs_max<16>(tail));
                }
                // f16 keeps its probabilities 2^7 higher, as in XaSoftmax
                const float ref = mx * c2 - (F16 ? 7.f : 0.f);
#pragma unroll 1
                for (int c = 0; c < pieces; ++c) {
                    float s[32];
                    xs_scores<32>(t_row + 32 * c, keep[c], s);
                    uint32_t pk[16];
                    l += exp_block<32, F16>(s, c2, ref, pk);
                    sm100::tmem_st16(t_row + 16 * c, pk);
                }
                if (half) {
                    uint32_t pk[8];
                    l += exp_block<16, F16>(tail, c2, ref, pk);
                    sm100::tmem_st8(t_row + 16 * pieces, pk);
                }
            }
            sm100::tc_fence_before();
            sm100::mbar_arrive(&bars[C::bP + wg]);
            ok = warp_wait(&bars[C::bO + wg], m & 1, lim);
            if (!ok) break;
            sm100::tc_fence_after();
            ++m;
        } else {  // the Q tile must have landed before zeros go there
            ok = warp_wait(&bars[C::bQFull + 2 * wg + (i & 1)], (i >> 1) & 1, lim);
            if (!ok) break;
        }
        // O / l into the tile's Q buffer (the S product has read it); without
        // a kept key O is 0, without any key nothing was computed
        uint8_t *dst = smem + (wg * 2 + (i & 1)) * C::kTileBytes + row * 128;
        if (active) {
            const float inv = l > 0.f ? 1.f / l : l;
            const uint64_t inv2 = sm100::pack_f32x2(inv, inv);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                sm100::tmem_ld32(t_row + C::kColO + c * 32, o);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x, y;
                        sm100::unpack_f32x2(sm100::fma_f32x2(sm100::pack_f32x2(__uint_as_float(o[8 * v + 2 * j]),
                                                                               __uint_as_float(o[8 * v + 2 * j + 1])),
                                                             inv2, 0),
                                            x, y);
                        h[j] = sm100::pack_16x2<F16>(x, y);
                    }
                    *reinterpret_cast<uint4 *>(dst + (c >> 1) * C::kChunkBytes + ((((c & 1) * 4 + v) ^ (row & 7)) << 4)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
        } else if (n <= 0) {
#pragma unroll
            for (int v = 0; v < 8 * C::kChunks; ++v)
                *reinterpret_cast<uint4 *>(dst + (v >> 3) * C::kChunkBytes + (v & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        sm100::tc_fence_before();
        sm100::fence_proxy_async();
        sm100::mbar_arrive(&bars[C::bE + wg]);
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
}

template <int D, bool F16>
__global__ void __launch_bounds__(XsCfg<D>::kThreads, 1) xa_short_kernel(const __grid_constant__ XsParams p) {
    using C = XsCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = sm100::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *kv = smem + C::kQBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(kv + p.kv_stages * C::kv_stage_bytes(p.kv_rows));
    uint32_t *misc = reinterpret_cast<uint32_t *>(bars + C::kNumBars);  // [0] TMEM base, [1] abort flag
    uint32_t *kept = misc + 4;                                          // [2][8]: four words of kept keys, key count
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            sm100::mbar_init(&bars[C::bKVFull + s], 1);
            sm100::mbar_init(&bars[C::bKVReady + s], 1);
            sm100::mbar_init(&bars[C::bKVEmpty + s], C::NW);
        }
        for (int w = 0; w < C::NW; ++w) {
            sm100::mbar_init(&bars[C::bQFull + 2 * w], 1);
            sm100::mbar_init(&bars[C::bQFull + 2 * w + 1], 1);
            sm100::mbar_init(&bars[C::bS + w], 1);
            sm100::mbar_init(&bars[C::bP + w], 128);
            sm100::mbar_init(&bars[C::bO + w], 1);
            sm100::mbar_init(&bars[C::bE + w], 128);
            sm100::mbar_init(&bars[C::bSet + w], 1);
            sm100::mbar_init(&bars[C::bDrain + w], 1);
        }
        misc[1] = 0;
        sm100::fence_barrier_init();
    }
    if (warp == C::kLoadWarp) {
        sm100::tmem_alloc(&misc[0], C::kTmemCols);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = misc[0];
    volatile uint32_t *abort_flag = &misc[1];
    if (warp >= C::kIssueWarp) {
        if constexpr (C::kSplitRegs) sm100::setmaxnreg_dec<C::kRegsOther>();
        if (warp == C::kLoadWarp)
            xs_loader<D>(p, kv, bars, kept, abort_flag);
        else if (warp < C::kIssueWarp + C::NW && (threadIdx.x & 31) == 0)
            xs_issue<D, F16>(p, smem, kv, bars, kept, tmem, abort_flag, warp - C::kIssueWarp);
    } else {
        if constexpr (C::kSplitRegs) sm100::setmaxnreg_inc<C::kRegsCompute>();
        xs_compute<D, F16>(p, smem, bars, kept, tmem, abort_flag, warp >> 2);
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    if (warp == C::kLoadWarp) {
        __syncwarp();
        sm100::tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace npa
