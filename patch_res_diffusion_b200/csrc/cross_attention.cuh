// cross_attention.cuh - attention of Lq queries to an encoder's Lk keys and
// values of another length (npa_cross_attention_fwd), and the same over a
// cache held in e4m3 with a scale per 64 tokens and head
// (npa_kv8_cross_attention_fwd).
//
//   o[b, h, i] = sum_j p_ij v[b, h', j],  p_ij = softmax_j(scale q[b, h, i] . k[b, h', j])
//
// over the keys j < kv_lens[b] with key_mask[b, j] != 0; h' = h / (heads /
// kv_heads). A row without keys gives zeros. What it has to read and write is
// q, o, k and v once; the exponentials (one per query and key) bind before the
// products at d = 64, as in the self-attention kernel.
//
// A persistent CTA walks units of 256 query rows (two 128-row tiles, one
// softmax warpgroup each) of one (batch, head), optionally over a part of the
// key range. Warps:
//   0-7    softmax and epilogue, tile 0 and 1 (TMEM lane = query row)
//   8      TMA producer (query tiles; key and value blocks of 128 tokens)
//   9, 10  MMA issuers: d = 64, the S products and the P.V products; d = 128,
//          warp 9 issues both
//   11     16-bit keys: clears the value rows of keys that are not kept
//          (0 * NaN would reach the sums through the product otherwise);
//          8-bit cache: finds how large a block's kept value codes are
//   12-15  8-bit cache: converts code blocks to f16 tiles in shared memory
// TMEM, the aliasing of P at d = 128, the lazily moved softmax reference and
// the turns on the exponential unit are those of npa_fwd_kernel.cuh.
//
// 8-bit cache. e4m3 codes are exact in f16 and one conversion makes two, so
// that kernel multiplies in f16 and leaves every scale to float32: q, scaled by
// a power of two per row, is exact in f16 too (elements 2^-14 under the row's
// largest lose at most 2^-25 of it); the block's k scale joins the softmax
// scale; its v scale shifts the exponent of P (P' = 2^(x + log2 s_v - R)), and
// the row sum divides it out again. (Converting code * scale to bf16 instead
// took 900 instructions of a converting warp per block, and more than twice
// the time of the softmax beside it.)
//   P' is f16: what lies 2^-31 under the reference is lost. So R has to follow
// what blocks contribute, not their scales alone: a block of zeros, one whose
// scale stems from a token that is not kept, or one whose scale has grown may
// have a large scale and small codes. Warp 11 therefore finds, per 64 tokens,
// the power of two by which the largest kept code lies under the format's top
// (where a code of 128 or more is met, as in nearly every block's first rows,
// that is 0 and the search ends); the converter takes it out of the value tile,
// exactly, and the softmax adds it to the scale. Halves without a kept code
// other than 0 count as 2^-80. A key's rounding is then at most 2^-30 of the
// largest p |v| that some 64 tokens' largest p and largest kept |v| make.
//   Scales are taken relative to that of the unit's first 64 tokens with values
// (2^c), so that sums stay within float32 wherever the scales lie; between
// blocks they may differ by 2^100.
//
// What differs from the self-attention kernel: every tensor is a 4D {d, L,
// heads, B} map with the caller's strides (a projection's [B, L, heads * d]
// needs no transposed copy); the last block's products and exponentials stop
// at its last key (rounded up to 16 and 32); the output leaves through shared
// memory as 128-byte rows with TMA stores, whose box the tensor map clips at
// Lq; and Q is double buffered at d = 64, so that a short context (one block
// per unit) streams queries and outputs at memory speed.
//
// Measured, bf16: 24 heads x 4096 x 16384 at d = 128 679 us (1,215 TFLOP/s; 745
// to 754 in a longer run, under the power cap), tensor and exponential units 59%
// busy each; 2 x 10 heads x 4096 x 9216 at d = 64 299 us (646 TFLOP/s),
// exponential unit 66%; over the 8-bit cache 2 x 10 heads x 4096 x 12288 at d =
// 64 464 us (555 TFLOP/s), exponential unit 52%, issue slots 47%, and 24 heads x
// 2048 x 4096 at d = 128 169 us (610 TFLOP/s), no unit above 31%. No unit is
// full: a tile's steps (S, softmax, P V) follow one another, two tiles fill a
// multiprocessor's gaps in part, and half of a cached block's scores are read
// twice.
//
// Tried and slower: dealing a one-tile piece's blocks to both warpgroups in
// turn (77 queries of 24 heads x 4608 cached keys: 36 us instead of 29; the
// code tiles' stages are what such a piece waits for, and the merge doubles).
#pragma once

#include <cuda_fp16.h>

#include "npa_fwd_kernel.cuh"

namespace npa {

constexpr int kKv8Block = 64;  // tokens of one head that share a scale of the 8-bit cache
constexpr int kXaMaxSplits = 64;      // xa_few_kernel's key-range splits at most
constexpr int kXaMaxTailCtas = 160;   // CTAs that cut units are dealt to at most

// n / d for 0 <= n < 2^31, d >= 1: with s = ceil(log2 d) and m = ceil(2^(31 +
// s) / d), the product n m exceeds 2^(31 + s) n / d by less than 2^(31 + s) / d.
struct FastDiv {
    uint32_t m;
    int s;
    FastDiv() = default;
    __host__ explicit FastDiv(int d) : s(0) {
        while ((1ll << s) < d) ++s;
        m = uint32_t(((1ull << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ int operator()(int n) const { return int((uint64_t(uint32_t(n)) * m) >> (31 + s)); }
};

struct XaParams {
    CUtensorMap tm_q;  // 4D {d, Lq, heads, B}, box {64, 128, 1, 1}, 128B swizzle
    CUtensorMap tm_k;  // 4D {d, Lk, kv_heads, B}, box {64, 128, 1, 1}, 128B swizzle; codes: box {d, 128, 1, 1}, none
    CUtensorMap tm_v;
    CUtensorMap tm_o;  // as tm_q
    const int *kv_lens;              // [B] or null: keys of batch row b (clamped to 0 .. Lk)
    const unsigned char *key_mask;   // [B, Lk] or null: 0 = not attended
    const float *k_scale, *v_scale;  // 8-bit cache: [B, kv_heads, scale_blocks]
    int scale_blocks;
    int B, heads, kv_heads, group, Lq, Lk;
    int q_b, q_h, k_b, k_h, v_b, v_h;  // 1, or 0 along an axis that the tensor repeats (stride 0)
    int n_qpairs;                      // ceil(Lq / 256)
    int n_units;                       // 256-row units: B * heads * n_qpairs
    // Every CTA runs `waves` whole units (blockIdx.x, blockIdx.x + gridDim.x,
    // ...). The units after those, fewer than there are CTAs, are cut: their
    // key blocks (n_blk each) go, in order, to the first tail_ctas CTAs (CTA
    // c: tail_start[c] .. tail_start[c + 1]), and the pieces of a unit are
    // merged by xa_tail_kernel. tail_ctas = 0: nothing is cut.
    int waves, tail_ctas, n_blk;
    int tail_start[kXaMaxTailCtas + 1];
    FastDiv by_blk, by_qpairs, by_heads, by_group;
    float scale_log2;
    unsigned long long wait_limit_ns;
    int sort_rows;  // batch rows in the order of their lengths
    int n_splits;   // xa_few_kernel: key-range splits
    // Partial results: unnormalised O [..][d], then reference and row sum
    // [..][2] (cut units over the 8-bit cache: O / l, reference plus log2 l, 1).
    // Cut units: two slots of 256 rows per CTA (its first piece, its last);
    // xa_few_kernel: [n_splits][B * heads * Lq].
    float *o_part, *ml;
};

template <int D, bool KV8>
struct XaCfg {
    static_assert(D == 64 || D == 128, "head dim");
    static constexpr int kChunks = D / 64;
    static constexpr int kChunkBytes = 128 * 128;  // 128 rows x 64 16-bit columns
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kCodeBytes = 128 * D;     // 128 rows of e4m3 codes
    // Shared memory is what sets the depths: 224 KB in every shape.
    static constexpr int kQStages = D == 64 ? 2 : 1;
    static constexpr int kStages = KV8 ? (D == 64 ? 2 : 1) : (D == 64 ? 4 : 2);
    static constexpr int kCodeStages = KV8 ? (D == 64 ? 4 : 2) : 0;
    static constexpr int kThreads = KV8 ? 512 : 384;
    static constexpr int kCtlWarp = 8;
    static constexpr int kConvWarp = 12;
    // Register split, as in KCfg; the 8-bit kernel's four warpgroups start
    // with 128 each, and its converter takes its share from the softmax's.
    static constexpr uint32_t kRegsLaunch = KV8 ? 128 : 168;
    static constexpr uint32_t kRegsSoftmax = KV8 ? 184 : D == 64 ? 216 : 208;
    static constexpr uint32_t kRegsCtl = KV8 ? 64 : D == 64 ? 72 : 88;
    static constexpr uint32_t kRegsConv = 80;
    static_assert(256 * kRegsSoftmax + 128 * kRegsCtl + (KV8 ? 128 * kRegsConv : 0) <= kThreads * kRegsLaunch,
                  "register split");
    static_assert(kThreads * kRegsLaunch <= 65536, "register file");
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kQStages * 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffKC = kOffV + kStages * kTileBytes;
    static constexpr int kOffVC = kOffKC + kCodeStages * kCodeBytes;
    static constexpr int kOffO = kOffVC + kCodeStages * kCodeBytes;  // [2] 128 rows x 64 columns
    static constexpr int kOffBar = kOffO + 2 * kChunkBytes;
    static constexpr int bQFull = 0;                     // [kQStages] both tiles landed
    static constexpr int bQEmpty = bQFull + kQStages;    // [kQStages] S products done (MMA commit)
    static constexpr int bKFull = bQEmpty + kQStages;    // [kStages] key tile there (TMA, or 128 converter arrivals)
    static constexpr int bKEmpty = bKFull + kStages;
    static constexpr int bVFull = bKEmpty + kStages;
    static constexpr int bVEmpty = bVFull + kStages;
    static constexpr int bVReady = bVEmpty + kStages;    // [kStages] rows of unkept keys cleared
    static constexpr int bQReady = bVReady + kStages;    // [kQStages] 8-bit: queries in f16 (128 arrivals)
    static constexpr int bKCFull = bQReady + kQStages;   // [kCodeStages] code blocks landed
    static constexpr int bKCEmpty = bKCFull + kCodeStages;
    static constexpr int bVCFull = bKCEmpty + kCodeStages;
    static constexpr int bVCEmpty = bVCFull + kCodeStages;  // 128 converter arrivals and the look at the values
    static constexpr int bSFull = bVCEmpty + kCodeStages;
    static constexpr int bSFree = bSFull + 2;
    static constexpr int bPFull = bSFree + 2;
    static constexpr int bPFree = bPFull + 2;
    static constexpr int bTurn = bPFree + 2;             // [2][4]
    static constexpr int bEpi = bTurn + 8;               // [2] a softmax warpgroup's own barrier (128 arrivals)
    static constexpr int bDrain = bEpi + 2;              // [2]
    // [4] 8-bit: the row exponents of a unit are written (128 arrivals). Four
    // sets: the converter reaches unit u + 4 only after the S products of unit
    // u + 2, which wait for the softmax of unit u (u + 1 at the latest, where a
    // unit has one tile only).
    static constexpr int kExpSets = 4;
    static constexpr int bExp = bDrain + 2;
    // [kScaleSets] 8-bit: a block's scales (XaBlockScales) are written (one
    // arrival). The converter waits for that before it converts the block's
    // keys, so its scores come later still and the softmax need not wait again.
    // A set is written again when the value codes of block i + kScaleSets are
    // there: behind the value tile of block i + kStages, and so behind the
    // products of block i, for which the softmax has read it.
    static constexpr int kScaleSets = kCodeStages + kStages;
    static constexpr int bScale = bExp + (KV8 ? kExpSets : 0);
    static constexpr int kNumBars = bScale + (KV8 ? kScaleSets : 0);
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kOffExp = kOffMisc + 16;        // [kExpSets][2][128] 8-bit: exponent taken out of a query row
    static constexpr int kOffScale = (kOffExp + (KV8 ? kExpSets * 256 : 0) + 15) & ~15;  // [kScaleSets] XaBlockScales
    static constexpr int kSmemBytes = kOffScale + (KV8 ? kScaleSets * 32 : 0) + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    static constexpr uint32_t kTmemCols = 512;
    static constexpr bool kSeparateP = (D == 64);
    // Turns on the exponential unit: not with the 8-bit cache, where half of a
    // block's scores are read under them (531 us with, 494 without on 2 x 10
    // heads, 4096 queries, 12288 keys).
    static constexpr bool kUseTurn = D == 64 && !KV8;
    __device__ static constexpr uint32_t col_s(int q) { return uint32_t(q * 128); }
    __device__ static constexpr uint32_t col_o(int q) { return uint32_t(256 + q * D); }
    __device__ static constexpr uint32_t col_p(int q) { return kSeparateP ? uint32_t(256 + 2 * D + q * 64) : col_s(q); }
};

// ---------------------------------------------------------------------------
// Units
// ---------------------------------------------------------------------------
struct XaUnit {
    int b, h, kvh;
    int row0;    // first query row
    int nt;      // query tiles (1 or 2)
    int len;     // keys of this batch row
    int jb, je;  // key blocks [jb, je)
    int slot;    // a piece of a unit: where its partial result goes; -1: the whole unit
};

// The batch row with the rank-th fewest keys (the earlier row first where they
// have the same). Units run in this order: a CTA's whole units are then alike,
// and the longest are those that are cut. (Lengths 12288 and 6144 in that order,
// 2 x 10 heads x 4096 queries over the 8-bit cache: 460 us as the rows stand, 358
// so.) For short units the look at the lengths costs more than it gives. As they
// stand / sorted, us, 4096 queries, all and half of the keys kept:
//   blocks                          2          8          12         16         32
//   d = 64, 2 x 10 heads        17 / 19    43 / 44    60 / 54    75 / 66  133 / 111
//   the same over the cache     22 / 24    54 / 56    75 / 68    93 / 84  166 / 142
//   d = 128, 2 x 12 heads       23 / 25    52 / 53    70 / 72    89 / 92  184 / 172
constexpr int kXaMaxSortedRows = 8;
__host__ __device__ constexpr int xa_min_sorted_blocks(int d) { return d == 64 ? 12 : 32; }
__device__ __forceinline__ int xa_row_of_rank(const int *kv_lens, int B, int Lk, int rank) {
    int row = 0;
    for (int b = 0; b < B; ++b) {
        const int len = min(max(__ldg(kv_lens + b), 0), Lk);
        int before = 0;
        for (int c = 0; c < B; ++c) {
            const int other = min(max(__ldg(kv_lens + c), 0), Lk);
            before += other < len || (other == len && c < b);
        }
        if (before == rank) row = b;
    }
    return row;
}

// The units of a CTA, in the order that all of its roles walk them.
struct XaIter {
    const XaParams &p;
    XaUnit u;
    int w = 0, pos = 0, start = 0, end = 0;
    __device__ __forceinline__ explicit XaIter(const XaParams &prm) : p(prm) {
        if (int(blockIdx.x) < p.tail_ctas) {
            pos = start = p.tail_start[blockIdx.x];
            end = p.tail_start[blockIdx.x + 1];
        }
    }
    __device__ __forceinline__ bool next() {
        int unit, jb = 0, je = p.n_blk;
        u.slot = -1;
        if (w < p.waves) {
            unit = blockIdx.x + w * gridDim.x;
            ++w;
            if (unit >= p.n_units) return false;
        } else {
            if (pos >= end) return false;
            const int t = p.by_blk(pos);
            unit = p.waves * gridDim.x + t;
            jb = pos - t * p.n_blk;
            je = min(p.n_blk, jb + end - pos);
            if (je - jb < p.n_blk) u.slot = 2 * blockIdx.x + (pos != start);
            pos += je - jb;
        }
        const int bh = p.by_qpairs(unit);
        u.row0 = (unit - bh * p.n_qpairs) * 256;
        u.b = p.by_heads(bh);
        u.h = bh - u.b * p.heads;
        u.kvh = p.by_group(u.h);
        if (p.sort_rows) u.b = xa_row_of_rank(p.kv_lens, p.B, p.Lk, u.b);
        u.nt = p.Lq - u.row0 > 128 ? 2 : 1;
        u.len = p.kv_lens ? min(max(__ldg(p.kv_lens + u.b), 0), p.Lk) : p.Lk;
        u.je = min(je, (u.len + 127) / 128);
        u.jb = min(jb, u.je);
        return true;
    }
};

__device__ __forceinline__ int xa_block_keys(const XaUnit &u, int j) { return min(128, u.len - j * 128); }

// Which of block j's 128 keys are attended: bit i of w[c] is key 32 c + i.
// Executed by a whole warp; every lane gets all words.
__device__ __forceinline__ void xa_keep(const XaParams &p, const XaUnit &u, int j, int n, uint32_t (&w)[4]) {
    if (p.key_mask) {
        const unsigned char *m = p.key_mask + (size_t)u.b * p.Lk + (size_t)j * 128;
        const int lane = threadIdx.x & 31;
        bool k[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = 32 * c + lane < n && __ldg(m + 32 * c + lane) != 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = __ballot_sync(0xffffffffu, k[c]);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int m = n - 32 * c;
            w[c] = m >= 32 ? 0xffffffffu : m <= 0 ? 0u : (1u << m) - 1u;
        }
    }
}

// ---------------------------------------------------------------------------
// Producer
// ---------------------------------------------------------------------------
template <int D, bool KV8>
__device__ void xa_producer(const XaParams &p, uint8_t *smem, uint64_t *bars, volatile uint32_t *abort_flag) {
    using C = XaCfg<D, KV8>;
    constexpr int kRing = KV8 ? C::kCodeStages : C::kStages;
    constexpr int kBytes = KV8 ? C::kCodeBytes : C::kTileBytes;
    constexpr int kOffKr = KV8 ? C::kOffKC : C::kOffK, kOffVr = KV8 ? C::kOffVC : C::kOffV;
    constexpr int bKF = KV8 ? C::bKCFull : C::bKFull, bKE = KV8 ? C::bKCEmpty : C::bKEmpty;
    constexpr int bVF = KV8 ? C::bVCFull : C::bVFull, bVE = KV8 ? C::bVCEmpty : C::bVEmpty;
    const uint64_t lim = p.wait_limit_ns;
    sm100::tma_prefetch_desc(&p.tm_q);
    sm100::tma_prefetch_desc(&p.tm_k);
    sm100::tma_prefetch_desc(&p.tm_v);
    sm100::tma_prefetch_desc(&p.tm_o);
    int nk = 0, nv = 0, uq = 0;
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        if (u.je <= u.jb) continue;
        const int qs = uq % C::kQStages, quse = uq / C::kQStages;
        if (quse > 0 && !sm100::mbar_wait(&bars[C::bQEmpty + qs], (quse - 1) & 1, lim)) {
            ok = false;
            break;
        }
        sm100::mbar_arrive_expect_tx(&bars[C::bQFull + qs], u.nt * C::kTileBytes);
        for (int t = 0; t < u.nt; ++t) {
            const int r = bound_coord(u.row0 + t * 128, p.Lq);
            uint8_t *dst = smem + C::kOffQ + (qs * 2 + t) * C::kTileBytes;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
                sm100::tma_load_4d(dst + c * C::kChunkBytes, &p.tm_q, &bars[C::bQFull + qs], c * 64, r,
                                   bound_coord(u.h, p.heads) * p.q_h, bound_coord(u.b, p.B) * p.q_b);
        }
        ++uq;
        const int kh = bound_coord(u.kvh, p.kv_heads), kb = bound_coord(u.b, p.B);
        for (int j = u.jb; j < u.je; ++j) {
            if (*abort_flag) {
                ok = false;
                break;
            }
            const int s = nk % kRing, use = nk / kRing;
            const int r = bound_coord(j * 128, p.Lk);
            if (use > 0 && !sm100::mbar_wait(&bars[bKE + s], (use - 1) & 1, lim)) {
                ok = false;
                break;
            }
            sm100::mbar_arrive_expect_tx(&bars[bKF + s], kBytes);
            if (KV8) {
                sm100::tma_load_4d(smem + kOffKr + s * kBytes, &p.tm_k, &bars[bKF + s], 0, r, kh, kb);
            } else {
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c)
                    sm100::tma_load_4d(smem + kOffKr + s * kBytes + c * C::kChunkBytes, &p.tm_k, &bars[bKF + s],
                                       c * 64, r, kh * p.k_h, kb * p.k_b);
            }
            ++nk;
            if (use > 0 && !sm100::mbar_wait(&bars[bVE + s], (use - 1) & 1, lim)) {
                ok = false;
                break;
            }
            sm100::mbar_arrive_expect_tx(&bars[bVF + s], kBytes);
            if (KV8) {
                sm100::tma_load_4d(smem + kOffVr + s * kBytes, &p.tm_v, &bars[bVF + s], 0, r, kh, kb);
            } else {
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c)
                    sm100::tma_load_4d(smem + kOffVr + s * kBytes + c * C::kChunkBytes, &p.tm_v, &bars[bVF + s],
                                       c * 64, r, kh * p.v_h, kb * p.v_b);
            }
            ++nv;
        }
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
    // every issued copy must have landed before the CTA may exit
    for (int s = 0; s < C::kQStages; ++s)
        if (uq > s) sm100::mbar_wait(&bars[C::bQFull + s], ((uq - 1 - s) / C::kQStages) & 1, lim);
    for (int s = 0; s < kRing; ++s) {
        if (nk > s) sm100::mbar_wait(&bars[bKF + s], ((nk - 1 - s) / kRing) & 1, lim);
        if (nv > s) sm100::mbar_wait(&bars[bVF + s], ((nv - 1 - s) / kRing) & 1, lim);
    }
}

// ---------------------------------------------------------------------------
// MMA issuers
// ---------------------------------------------------------------------------
// S_q[:, 0 .. n) = Q K^T for the block's n keys (n rounded up to 16).
template <int D, bool F16>
__device__ __forceinline__ void xa_issue_s(uint32_t d_tmem, uint64_t qdesc, uint64_t kdesc, int n) {
    using C = XaCfg<D, false>;
    constexpr uint32_t kId0 = F16 ? sm100::idesc_f16_f32(128, 0, false, false) : sm100::idesc_bf16_f32(128, 0, false, false);
    const uint32_t id = kId0 | (uint32_t((n + 15) >> 4) << 18);  // N >> 3 at bit 17
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = uint64_t(((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4);
        sm100::mma_ss(d_tmem, qdesc + off, kdesc + off, id, kk > 0 ? 1u : 0u);
    }
}

// O_q (+)= P_q V over the block's n keys (n rounded up to 16; P is 0 and V is
// finite past n).
template <int D, bool F16>
__device__ __forceinline__ void xa_issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint64_t vdesc, int n, bool accumulate) {
    constexpr uint32_t kId = F16 ? sm100::idesc_f16_f32(128, D, false, true) : sm100::idesc_bf16_f32(128, D, false, true);
    const int steps = (n + 15) >> 4;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
        if (kk < steps)
            sm100::mma_ts(o_tmem, p_tmem + kk * 8, vdesc + uint64_t((kk * 2048) >> 4), kId,
                          (accumulate || kk > 0) ? 1u : 0u);
}

template <int D, bool KV8>
struct XaDescs {
    uint64_t q0, k0, v0;
    static constexpr uint64_t tile = uint64_t(XaCfg<D, KV8>::kTileBytes >> 4);
    __device__ explicit XaDescs(uint8_t *smem) {
        using C = XaCfg<D, KV8>;
        q0 = sm100::sdesc_sw128(sm100::smem_u32(smem + C::kOffQ), 16, 1024);
        k0 = sm100::sdesc_sw128(sm100::smem_u32(smem + C::kOffK), 16, 1024);
        v0 = sm100::sdesc_sw128(sm100::smem_u32(smem + C::kOffV), C::kChunkBytes, 1024);
    }
};

// The barrier that says block values are ready for the products: the copy's
// own, or the one of the warp that clears unkept rows.
template <int D, bool KV8>
__device__ __forceinline__ int xa_v_bar(const XaParams &p) {
    using C = XaCfg<D, KV8>;
    return !KV8 && (p.kv_lens || p.key_mask) ? C::bVReady : C::bVFull;
}

// d = 64: the S products.
template <int D, bool KV8, bool F16>
__device__ void xa_mma_s(const XaParams &p, uint8_t *smem, uint64_t *bars, uint32_t tmem,
                         volatile uint32_t *abort_flag) {
    using C = XaCfg<D, KV8>;
    const uint64_t lim = p.wait_limit_ns;
    const XaDescs<D, KV8> dd(smem);
    int kv = 0, uq = 0, g[2] = {0, 0};
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        if (u.je <= u.jb) continue;
        const int qs = uq % C::kQStages;
        ok = sm100::mbar_wait(&bars[(KV8 ? C::bQReady : C::bQFull) + qs], (uq / C::kQStages) & 1, lim);
        ++uq;
        for (int j = u.jb; ok && j < u.je; ++j, ++kv) {
            if (*abort_flag) {
                ok = false;
                break;
            }
            const int s = kv % C::kStages, n = xa_block_keys(u, j);
            ok = sm100::mbar_wait(&bars[C::bKFull + s], (kv / C::kStages) & 1, lim);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (!ok || q >= u.nt) continue;
                if (g[q] > 0) ok = sm100::mbar_wait(&bars[C::bSFree + q], (g[q] - 1) & 1, lim);
                if (!ok) continue;
                sm100::tc_fence_after();
                xa_issue_s<D, KV8 || F16>(tmem + C::col_s(q), dd.q0 + (qs * 2 + q) * dd.tile, dd.k0 + s * dd.tile, n);
                sm100::tc_commit(&bars[C::bSFull + q]);
                ++g[q];
            }
            if (ok) sm100::tc_commit(&bars[C::bKEmpty + s]);
        }
        if (ok) sm100::tc_commit(&bars[C::bQEmpty + qs]);
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
    sm100::tc_commit(&bars[C::bDrain]);
    sm100::mbar_wait(&bars[C::bDrain], 0, lim);
}

// d = 64: the P.V products.
template <int D, bool KV8, bool F16>
__device__ void xa_mma_pv(const XaParams &p, uint8_t *smem, uint64_t *bars, uint32_t tmem,
                          volatile uint32_t *abort_flag) {
    using C = XaCfg<D, KV8>;
    const uint64_t lim = p.wait_limit_ns;
    const XaDescs<D, KV8> dd(smem);
    const int bV = xa_v_bar<D, KV8>(p);
    int kv = 0, g[2] = {0, 0};
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        for (int j = u.jb; ok && j < u.je; ++j, ++kv) {
            if (*abort_flag) {
                ok = false;
                break;
            }
            const int s = kv % C::kStages, n = xa_block_keys(u, j);
            ok = sm100::mbar_wait(&bars[bV + s], (kv / C::kStages) & 1, lim);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (!ok || q >= u.nt) continue;
                ok = sm100::mbar_wait(&bars[C::bPFull + q], g[q] & 1, lim);
                if (!ok) continue;
                sm100::tc_fence_after();
                xa_issue_pv<D, KV8 || F16>(tmem + C::col_o(q), tmem + C::col_p(q), dd.v0 + s * dd.tile, n, j > u.jb);
                sm100::tc_commit(&bars[C::bPFree + q]);
                ++g[q];
            }
            if (ok) sm100::tc_commit(&bars[C::bVEmpty + s]);
        }
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
    sm100::tc_commit(&bars[C::bDrain + 1]);
    sm100::mbar_wait(&bars[C::bDrain + 1], 0, lim);
}

// d = 128 (P aliases S): PV_q(j-1) before S_q(j) from one thread, so that the
// completion of S_q(j) also says that PV_q(j-1) is done.
template <int D, bool KV8, bool F16>
__device__ void xa_mma(const XaParams &p, uint8_t *smem, uint64_t *bars, uint32_t tmem,
                       volatile uint32_t *abort_flag) {
    using C = XaCfg<D, KV8>;
    const uint64_t lim = p.wait_limit_ns;
    const XaDescs<D, KV8> dd(smem);
    const int bV = xa_v_bar<D, KV8>(p);
    int kv0 = 0, uq = 0, g[2] = {0, 0};  // kv0: ring index of the unit's first block; g: P blocks consumed
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        const int n_blk = u.je - u.jb;
        if (n_blk <= 0) continue;
        const int qs = uq % C::kQStages;
        ok = sm100::mbar_wait(&bars[(KV8 ? C::bQReady : C::bQFull) + qs], (uq / C::kQStages) & 1, lim);
        ++uq;
        for (int j = 0; ok && j <= n_blk; ++j) {
            if (*abort_flag) {
                ok = false;
                break;
            }
            const int kv = kv0 + j, s = kv % C::kStages;
            const int sp = (kv + C::kStages - 1) % C::kStages;  // the previous block's stage
            if (j < n_blk) ok = sm100::mbar_wait(&bars[C::bKFull + s], (kv / C::kStages) & 1, lim);
            if (ok && j > 0) ok = sm100::mbar_wait(&bars[bV + sp], ((kv - 1) / C::kStages) & 1, lim);
            if (!ok) break;
            sm100::tc_fence_after();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (!ok || q >= u.nt) continue;
                if (j > 0) {
                    ok = sm100::mbar_wait(&bars[C::bPFull + q], g[q] & 1, lim);
                    if (!ok) continue;
                    sm100::tc_fence_after();
                    xa_issue_pv<D, KV8 || F16>(tmem + C::col_o(q), tmem + C::col_p(q), dd.v0 + sp * dd.tile,
                                        xa_block_keys(u, u.jb + j - 1), j > 1);
                    sm100::tc_commit(&bars[C::bPFree + q]);
                    ++g[q];
                }
                if (j < n_blk) {
                    xa_issue_s<D, KV8 || F16>(tmem + C::col_s(q), dd.q0 + (qs * 2 + q) * dd.tile, dd.k0 + s * dd.tile,
                                       xa_block_keys(u, u.jb + j));
                    sm100::tc_commit(&bars[C::bSFull + q]);
                }
            }
            if (!ok) break;
            if (j < n_blk) sm100::tc_commit(&bars[C::bKEmpty + s]);
            if (j == n_blk - 1) sm100::tc_commit(&bars[C::bQEmpty + qs]);
            if (j > 0) sm100::tc_commit(&bars[C::bVEmpty + sp]);
        }
        kv0 += n_blk;
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
    sm100::tc_commit(&bars[C::bDrain]);
    sm100::mbar_wait(&bars[C::bDrain], 0, lim);
}

// ---------------------------------------------------------------------------
// 16-bit values: rows of unkept keys set to zero (one warp). P is 0 there, but
// a NaN or an infinity in padding would still spread through the product.
// ---------------------------------------------------------------------------
template <int D>
__device__ void xa_clear_unkept(const XaParams &p, uint8_t *smem, uint64_t *bars, volatile uint32_t *abort_flag) {
    using C = XaCfg<D, false>;
    const uint64_t lim = p.wait_limit_ns;
    const int lane = threadIdx.x & 31;
    int kv = 0;
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        for (int j = u.jb; j < u.je; ++j, ++kv) {
            const int s = kv % C::kStages, n = xa_block_keys(u, j);
            uint32_t w[4];
            xa_keep(p, u, j, n, w);
            ok = !*abort_flag && sm100::mbar_wait(&bars[C::bVFull + s], (kv / C::kStages) & 1, lim);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t *tile = smem + C::kOffV + s * C::kTileBytes;
            const int n16 = (n + 15) & ~15;  // rows that the product reads
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int row = 32 * c + lane;
                if (row < n16 && !(w[c] >> lane & 1)) {
#pragma unroll
                    for (int ch = 0; ch < C::kChunks; ++ch)
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *reinterpret_cast<uint4 *>(tile + ch * C::kChunkBytes + row * 128 + v * 16) =
                                make_uint4(0, 0, 0, 0);
                }
            }
            sm100::fence_proxy_async();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&bars[C::bVReady + s]);
        }
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
}

// ---------------------------------------------------------------------------
// 8-bit cache: how large the kept value codes are (one warp)
// ---------------------------------------------------------------------------
constexpr int kXaNoValues = 255;  // no kept code other than 0

// The power of two by which the largest kept code of 64 tokens lies under
// 2^8..2^9, the binade of the format's top: 0 (a code of 128 or more), 2..17 or
// kXaNoValues. Executed by a whole warp.
template <int D>
__device__ __forceinline__ int xa_codes_under_top(const uint8_t *codes, uint32_t w0, uint32_t w1, int lane) {
    if ((w0 | w1) == 0u) return kXaNoValues;
    uint32_t top = 0;  // largest magnitudes, in the upper bytes of two halves
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) {
        const int idx = lane + 32 * i, row = idx / (D / 16);
        uint4 c = *reinterpret_cast<const uint4 *>(codes + idx * 16);
        if (!((row < 32 ? w0 : w1) >> (row & 31) & 1u)) c = make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {c.x, c.y, c.z, c.w};
        uint32_t big = 0;  // codes 0x70 and above, the sign aside: 128 or more
#pragma unroll
        for (int k = 0; k < 4; ++k) big |= x[k] & x[k] << 1 & x[k] << 2 & 0x40404040u;
        if (__any_sync(0xffffffffu, big != 0u)) return 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            top = __vmaxu2(top, x[k] & 0x7f007f00u);
            top = __vmaxu2(top, (x[k] & 0x007f007fu) << 8);
        }
    }
    const int a = int(__reduce_max_sync(0xffffffffu, max(top >> 16, top & 0xffffu)) >> 8);
    if (a == 0) return kXaNoValues;
    return a >= 8 ? 15 - (a >> 3) : 17 - (31 - __clz(a));  // exponent (a >> 3) - 7; subnormals a 2^-9
}

// A block's scales, for each half of its keys: k, the keys'; lv, log2 of what the
// value tile is to be multiplied by, relative to the unit's 2^c; inv_v, 2^-lv.
// (lg2.approx is off by 2^-22, or by 2^-17 at the ends of float32's range: below
// a sixteenth of P's rounding.)
struct alignas(16) XaBlockScales {
    float k[2], lv[2], inv_v[2];
    float c;
    int lift;  // powers of two that the value tile's halves are multiplied by: bits 0-7, 8-15
};
static_assert(sizeof(XaBlockScales) == 32, "two 16-byte loads");
// lv of 64 tokens that contribute nothing: R follows them only where values have
// less than 2^-80 of their probability (a rounding is then 2^-25 2^-87 of the
// unit's first values' scale, below 2^-109 of the largest value), and a row sum
// over them alone stays below 2^(80 + 15) times the number of keys.
constexpr float kXaNoValuesLog2 = -80.f;

template <int D>
__device__ void xa_block_scales(const XaParams &p, uint8_t *smem, uint64_t *bars, volatile uint32_t *abort_flag) {
    using C = XaCfg<D, true>;
    const uint64_t lim = p.wait_limit_ns;
    const int lane = threadIdx.x & 31;
    XaBlockScales *sets = reinterpret_cast<XaBlockScales *>(smem + C::kOffScale);
    int kv = 0;
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        const size_t s0 = ((size_t)u.b * p.kv_heads + u.kvh) * p.scale_blocks;
        float c = -INFINITY;  // log2 of the first values' scale; -inf: none yet
        for (int j = u.jb; j < u.je; ++j, ++kv) {
            const int cs = kv % C::kCodeStages, set = kv % C::kScaleSets;
            const int i0 = 2 * j, i1 = min(i0 + 1, p.scale_blocks - 1);  // past the cache: its keys are not kept
            const float ks[2] = {__ldg(p.k_scale + s0 + i0), __ldg(p.k_scale + s0 + i1)};
            const float vs[2] = {__ldg(p.v_scale + s0 + i0), __ldg(p.v_scale + s0 + i1)};
            ok = !*abort_flag && sm100::mbar_wait_idle(&bars[C::bVCFull + cs], (kv / C::kCodeStages) & 1, lim);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t *codes = smem + C::kOffVC + cs * C::kCodeBytes;
            XaBlockScales out;
            out.lift = 0;
            int tops = 0;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int key = j * 128 + h * 64 + lane;  // this lane's first, the second 32 on
                bool k0 = key < u.len, k1 = key + 32 < u.len;
                if (p.key_mask) {
                    const unsigned char *m = p.key_mask + (size_t)u.b * p.Lk + key;
                    k0 = k0 && __ldg(m) != 0;
                    k1 = k1 && __ldg(m + 32) != 0;
                }
                const uint32_t w0 = __ballot_sync(0xffffffffu, k0), w1 = __ballot_sync(0xffffffffu, k1);
                tops |= xa_codes_under_top<D>(codes + h * 64 * D, w0, w1, lane) << 8 * h;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int top = tops >> 8 * h & 255;
                const bool some = top != kXaNoValues;  // else whatever the scale holds stays out
                const float lv = __log2f(vs[h]) - float(top);
                if (some && c == -INFINITY) c = lv;
                out.k[h] = ks[h];
                out.lv[h] = some ? lv - c : kXaNoValuesLog2;
                out.inv_v[h] = sm100::ex2_approx(-out.lv[h]);
                if (some) out.lift |= top << 8 * h;
            }
            out.c = c;
            __syncwarp();
            if (lane == 0) {
                sets[set] = out;
                sm100::mbar_arrive(&bars[C::bScale + set]);
                sm100::mbar_arrive(&bars[C::bVCEmpty + cs]);
            }
        }
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
}

// ---------------------------------------------------------------------------
// 8-bit cache (one warpgroup): code blocks to f16 tiles, values of unkept keys
// as zeros (a NaN code would reach the sums through the product otherwise), and
// the unit's query rows to f16.
// ---------------------------------------------------------------------------
// The i-th 16-code piece of converting thread tid. Eight lanes take half of an
// even row and the other half of the odd row behind it (d = 128): 128 different
// bytes mod 128 to read, and, as the swizzle puts even rows' pieces in even
// places, eight different places to write.
template <int D>
__device__ __forceinline__ void xa_piece(int i, int tid, int &row, int &piece) {
    const int idx = tid + 128 * i, half = idx >> 2 & 1;
    row = D == 128 ? idx / 16 * 2 + half : idx / (D / 16);
    piece = D == 128 ? (idx & 3) + 4 * (half ^ (idx >> 3 & 1)) : idx % (D / 16);
}

template <int D>
__device__ __forceinline__ void xa_convert_tile(const uint8_t *codes, uint8_t *tile, const uint32_t (&w)[4], int tid) {
    using C = XaCfg<D, true>;
    constexpr int kPerRow = D / 16;  // 16-code pieces of a row
    const bool all = (w[0] & w[1] & w[2] & w[3]) == 0xffffffffu;
    // pieces in flight. d = 64 takes what keeps the code short, which the kernel's
    // roles share a cache for: 463 us with 1, 477 with 2, 487 with 4 (2 x 10 heads x
    // 4096 x 12288); d = 128: 4 against 2, 171 and 173 us (24 heads x 2048 x 4096).
    constexpr int kAhead = D == 128 ? 4 : 1;
#pragma unroll kAhead
    for (int i = 0; i < kPerRow; ++i) {
        int row, piece;
        xa_piece<D>(i, tid, row, piece);
        uint4 c4 = *reinterpret_cast<const uint4 *>(codes + row * D + piece * 16);
        if (!all) {
            const uint32_t word = row < 64 ? (row < 32 ? w[0] : w[1]) : (row < 96 ? w[2] : w[3]);
            if (!(word >> (row & 31) & 1u)) c4 = make_uint4(0, 0, 0, 0);
        }
        uint8_t *dst = tile + (piece >> 2) * C::kChunkBytes + row * 128;
        const int p0 = (piece & 3) * 2;
        *reinterpret_cast<uint4 *>(dst + ((p0 ^ (row & 7)) << 4)) =
            make_uint4(sm100::e4m3x2_to_f16x2(c4.x), sm100::e4m3x2_to_f16x2(c4.x >> 16), sm100::e4m3x2_to_f16x2(c4.y),
                       sm100::e4m3x2_to_f16x2(c4.y >> 16));
        *reinterpret_cast<uint4 *>(dst + (((p0 + 1) ^ (row & 7)) << 4)) =
            make_uint4(sm100::e4m3x2_to_f16x2(c4.z), sm100::e4m3x2_to_f16x2(c4.z >> 16), sm100::e4m3x2_to_f16x2(c4.w),
                       sm100::e4m3x2_to_f16x2(c4.w >> 16));
    }
}

// The values that this thread has converted times 2^lift0 (the first 64 rows) or
// 2^lift1, at most 2^17: exact.
template <int D>
__device__ __forceinline__ void xa_lift_tile(uint8_t *tile, int lift0, int lift1, int tid) {
    using C = XaCfg<D, true>;
#pragma unroll 1
    for (int i = 0; i < D / 2; ++i) {
        int row, piece;
        xa_piece<D>(i >> 3, tid, row, piece);
        const int lift = row < 64 ? lift0 : lift1, p0 = (piece & 3) * 2 + (i >> 2 & 1);
        // in two factors, f16x2: 2^17 is past f16's largest
        const uint32_t f0 = uint32_t(15 + (lift >> 1)) * 0x04000400u, f1 = uint32_t(15 + lift - (lift >> 1)) * 0x04000400u;
        uint8_t *base = tile + (piece >> 2) * C::kChunkBytes + row * 128 + ((p0 ^ (row & 7)) << 4);
        uint32_t *at = reinterpret_cast<uint32_t *>(base) + (i & 3);
        *at = sm100::mul_f16x2(sm100::mul_f16x2(*at, f0), f1);
    }
}

// One query row, bf16 to f16 in place; returns the exponent taken out.
template <int D>
__device__ __forceinline__ int xa_convert_q_row(uint8_t *tile, int row) {
    using C = XaCfg<D, true>;
    uint8_t *base = tile + row * 128;
    auto at = [&](int i) { return reinterpret_cast<uint4 *>(base + (i >> 3) * C::kChunkBytes + (((i & 7) ^ (row & 7)) << 4)); };
    uint32_t top = 0;  // largest magnitude, as bits
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = *at(i);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(x[k] & 0x7fffu, x[k] >> 16 & 0x7fffu));
    }
    const int e = top ? min(max(int(top >> 7) - 127, -126), 126) : 0;
    const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = *at(i);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            h[k] = sm100::pack_f16x2(__uint_as_float(x[k] << 16) * down, __uint_as_float(x[k] & 0xffff0000u) * down);
        *at(i) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    return e;
}

template <int D>
__device__ void xa_convert(const XaParams &p, uint8_t *smem, uint64_t *bars, volatile uint32_t *abort_flag) {
    using C = XaCfg<D, true>;
    const uint64_t lim = p.wait_limit_ns;
    const int tid = threadIdx.x - C::kConvWarp * 32;
    int kv = 0, uq = 0;
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        if (u.je <= u.jb) continue;
        const int qs = uq % C::kQStages;
        ok = warp_wait(&bars[C::bQFull + qs], (uq / C::kQStages) & 1, lim);
        if (!ok) break;
        const int set = uq % C::kExpSets;
        ++uq;
#pragma unroll 1
        for (int t = 0; t < u.nt; ++t)
            reinterpret_cast<int8_t *>(smem + C::kOffExp)[(set * 2 + t) * 128 + tid] =
                int8_t(xa_convert_q_row<D>(smem + C::kOffQ + (qs * 2 + t) * C::kTileBytes, tid));
        sm100::mbar_arrive(&bars[C::bExp + set]);
        sm100::fence_proxy_async();
        sm100::mbar_arrive(&bars[C::bQReady + qs]);
        for (int j = u.jb; ok && j < u.je; ++j, ++kv) {
            uint32_t w[4];
            xa_keep(p, u, j, xa_block_keys(u, j), w);
            const int cs = kv % C::kCodeStages, cpar = (kv / C::kCodeStages) & 1;
            const int s = kv % C::kStages, use = kv / C::kStages;
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {  // keys, values
                // the block's scales come after the copy of its values
                const int set = kv % C::kScaleSets;
                ok = !*abort_flag &&
                     (t || (sm100::mbar_wait(&bars[C::bScale + set], (kv / C::kScaleSets) & 1, lim) &&
                            sm100::mbar_wait(&bars[C::bKCFull + cs], cpar, lim))) &&
                     (use == 0 || sm100::mbar_wait(&bars[(t ? C::bVEmpty : C::bKEmpty) + s], (use - 1) & 1, lim));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t *tile = smem + (t ? C::kOffV : C::kOffK) + s * C::kTileBytes;
                xa_convert_tile<D>(smem + (t ? C::kOffVC : C::kOffKC) + cs * C::kCodeBytes, tile, w, tid);
                if (t) {
                    const int lift = reinterpret_cast<const XaBlockScales *>(smem + C::kOffScale)[set].lift;
                    if (lift) xa_lift_tile<D>(tile, lift & 255, lift >> 8, tid);
                }
                sm100::fence_proxy_async();
                sm100::mbar_arrive(&bars[(t ? C::bVFull : C::bKFull) + s]);
                sm100::mbar_arrive(&bars[(t ? C::bVCEmpty : C::bKCEmpty) + cs]);
            }
        }
    }
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
}

// ---------------------------------------------------------------------------
// Softmax and epilogue
// ---------------------------------------------------------------------------
// 32 * NCH scores of a row, unkept ones as -inf (kMasked: there may be some).
template <int NCH, bool kMasked = true>
__device__ __forceinline__ void xa_load_scores(uint32_t t_s, const uint32_t (&w)[4], float (&s)[32 * NCH]) {
    if constexpr (NCH == 2) {
        uint32_t r[64];
        sm100::tmem_ld64(t_s, r);
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(r[i]);
    } else if constexpr (NCH == 4) {
        uint32_t r[128];
        sm100::tmem_ld128(t_s, r);
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(r[i]);
    } else {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            uint32_t r[32];
            sm100::tmem_ld32(t_s + 32 * c, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[32 * c + i] = __uint_as_float(r[i]);
        }
    }
#pragma unroll
    for (int c = 0; kMasked && c < NCH; ++c) {
        if (w[c] != 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!(w[c] >> i & 1u)) s[32 * c + i] = -INFINITY;
        }
    }
}

template <int NCH>
__device__ __forceinline__ void xa_store_p(uint32_t t_p, const uint32_t (&pk)[16 * NCH]) {
    if constexpr (NCH == 4) {
        sm100::tmem_st64(t_p, pk);
    } else if constexpr (NCH == 2) {
        sm100::tmem_st32(t_p, pk);
    } else {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = pk[16 * c + i];
            sm100::tmem_st16(t_p + 16 * c, r);
        }
    }
}

// The same for one row: f, of the scores to log2 units.
struct XaScales {
    float f[2], lv[2], inv_v[2];
};

template <int D, bool KV8, bool F16>
struct XaSoftmax {
    using C = XaCfg<D, KV8>;
    static constexpr bool kF16 = KV8 || F16;  // type of P
    // A block whose maximum exceeds the reference by more than kLead moves it
    // to kBelow under the maximum: P stays within 2^8 in bf16. In f16 the
    // probabilities are kept 2^7 higher (at most 2^15), so that those 2^-24
    // below the row's largest are still normal numbers.
    static constexpr float kLead = kF16 ? 15.f : kRescaleLog2;
    static constexpr float kBelow = kF16 ? 7.f : 0.f;

    const XaParams &p;
    uint64_t *bars;
    uint64_t lim;
    uint32_t tS, tO, tP;
    int q, warp;  // tile, warp within the warpgroup
    bool lane0;
    int g, tb;    // blocks of this tile so far; blocks of two-tile units so far
    float R, R_prev, l;

    __device__ __forceinline__ bool take_turn() {
        return !C::kUseTurn || (q == 0 && tb == 0) ||
               warp_wait(&bars[C::bTurn + 4 * q + warp], (q == 0 ? tb - 1 : tb) & 1, lim);
    }
    __device__ __forceinline__ void pass_turn() {
        if (C::kUseTurn) {
            __syncwarp();
            if (lane0) sm100::mbar_arrive(&bars[C::bTurn + 4 * (1 - q) + warp]);
        }
    }

    // Maximum of one half's scores in log2 units, value scale included.
    template <int N>
    __device__ __forceinline__ float half_max(const float (&s)[N], const XaScales &sc, int h) {
        float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            m[0] = sm100::max3(m[0], s[i], s[i + 1]);
            m[1] = sm100::max3(m[1], s[i + 2], s[i + 3]);
        }
        return fmaf(fmaxf(m[0], m[1]), sc.f[h], sc.lv[h]);
    }
    // P of one half at reference R; the row sum, without the value scale.
    template <int N>
    __device__ __forceinline__ float half_exp(const float (&s)[N], const XaScales &sc, int h, uint32_t (&pk)[N / 2]) {
        return exp_block<N, true>(s, sc.f[h], R == -INFINITY ? R : R - sc.lv[h], pk) * sc.inv_v[h];
    }

    // The row's scores are in registers: d = 64, the next block's may come.
    __device__ __forceinline__ void release_scores() {
        if (C::kSeparateP) {
            sm100::tc_fence_before();
            sm100::mbar_arrive(&bars[C::bSFree + q]);
        }
    }

    // PV(j-1) is done and O is at the reference R.
    __device__ __forceinline__ bool ready_for_p(bool first, float alpha) {
        if (C::kSeparateP && !first) {
            if (!warp_wait(&bars[C::bPFree + q], (g - 1) & 1, lim)) return false;
            sm100::tc_fence_after();
        }
        if (!first && __any_sync(0xffffffffu, alpha != 1.f)) rescale(alpha);
        return true;
    }

    // A block over the 8-bit cache, half by half (each has its scales): a whole
    // row of scores does not fit in the registers that its 512 threads leave.
    // The second half is read twice; P of the first may overwrite its own
    // scores (d = 128), not the second's.
    template <int NCH, bool kMasked>
    __device__ __forceinline__ bool block8(const uint32_t (&w)[4], const XaScales &sc, bool first, bool turns) {
        constexpr int kA = NCH < 2 ? NCH : 2, kB = NCH - kA;  // 32-key pieces of the halves
        const uint32_t wb[4] = {w[2], w[3], 0, 0};
        float bm = -INFINITY;
        if constexpr (kB > 0) {
            float s[32 * kB];
            xa_load_scores<kB, kMasked>(tS + 64, wb, s);
            bm = half_max(s, sc, 1);
        }
        float s[32 * kA];
        xa_load_scores<kA, kMasked>(tS, w, s);
        if (kB == 0) release_scores();
        bm = fmaxf(bm, half_max(s, sc, 0));
        if (bm > R + kLead) R = bm - kBelow;
        const float alpha = (R == R_prev) ? 1.f : sm100::ex2_approx(R_prev - R);
        if (turns && !take_turn()) return false;
        uint32_t pk[16 * kA];
        l = l * alpha + half_exp(s, sc, 0, pk);
        if (!ready_for_p(first, alpha)) return false;
        xa_store_p<kA>(tP, pk);
        if constexpr (kB > 0) {
            float t[32 * kB];
            xa_load_scores<kB, kMasked>(tS + 64, wb, t);
            release_scores();
            uint32_t pt[16 * kB];
            l += half_exp(t, sc, 1, pt);
            xa_store_p<kB>(tP + 32, pt);
        }
        if (turns) pass_turn();
        sm100::tc_fence_before();
        sm100::mbar_arrive(&bars[C::bPFull + q]);
        R_prev = R;
        return true;
    }

    // One block of at most 32 * NCH keys; false when a wait ran out.
    template <int NCH, bool kMasked = true>
    __device__ __forceinline__ bool block(const uint32_t (&w)[4], const XaScales &sc, bool first, bool turns) {
        if constexpr (KV8) {
            return block8<NCH, kMasked>(w, sc, first, turns);
        } else {
            constexpr int kN = 32 * NCH;
            float s[kN];
            xa_load_scores<NCH, kMasked>(tS, w, s);
            release_scores();
            const float bm = row_max<kN>(s) * p.scale_log2;
            if (bm > R + kLead) R = bm - kBelow;
            if (turns && !take_turn()) return false;
            uint32_t pk[kN / 2];
            const float sum = exp_block<kN, F16>(s, p.scale_log2, R, pk);
            if (turns) pass_turn();
            const float alpha = (R == R_prev) ? 1.f : sm100::ex2_approx(R_prev - R);
            if (!ready_for_p(first, alpha)) return false;
            l = l * alpha + sum;
            xa_store_p<NCH>(tP, pk);
            sm100::tc_fence_before();
            sm100::mbar_arrive(&bars[C::bPFull + q]);
            R_prev = R;
            return true;
        }
    }

    // O *= alpha.
    __device__ __forceinline__ void rescale(float alpha) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            sm100::tmem_ld32(tO + c * 32, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            sm100::tmem_st32(tO + c * 32, o);
        }
    }

    // A warp whose 32 rows lie past the last query keeps the barriers' counts.
    __device__ __forceinline__ bool idle_block(bool first, bool turns) {
        if (C::kSeparateP) sm100::mbar_arrive(&bars[C::bSFree + q]);
        if (turns) {
            if (!take_turn()) return false;
            pass_turn();
        }
        if (C::kSeparateP && !first && !warp_wait(&bars[C::bPFree + q], (g - 1) & 1, lim)) return false;
        sm100::mbar_arrive(&bars[C::bPFull + q]);
        return true;
    }
};

template <int D, bool KV8, bool F16>
__device__ void xa_softmax(const XaParams &p, uint8_t *smem, uint64_t *bars, uint32_t tmem,
                           volatile uint32_t *abort_flag, int q) {
    using C = XaCfg<D, KV8>;
    const uint64_t lim = p.wait_limit_ns;
    const int row = threadIdx.x & 127;
    const int warp = row >> 5;
    const uint32_t lane_off = uint32_t(warp) * 32u << 16;
    XaSoftmax<D, KV8, F16> st{p,    bars, lim,  tmem + lane_off + C::col_s(q), tmem + lane_off + C::col_o(q),
                              tmem + lane_off + C::col_p(q), q, warp, (threadIdx.x & 31) == 0, 0, 0, 0.f, 0.f, 0.f};
    uint8_t *stage = smem + C::kOffO + q * C::kChunkBytes;
    int ep = 0;  // uses of the warpgroup's own barrier
    int uq = -1;  // units with keys so far, the current one included
    int kv = 0;   // 8-bit cache: blocks before the current unit's, of any tile
    auto group_sync = [&]() {
        sm100::mbar_arrive(&bars[C::bEpi + q]);
        return warp_wait(&bars[C::bEpi + q], (ep++) & 1, lim);
    };
    bool ok = true;
    for (XaIter it(p); ok && it.next();) {
        const XaUnit &u = it.u;
        uq += u.je > u.jb;
        const int kv0 = kv - u.jb;
        kv += u.je - u.jb;
        if (q >= u.nt) continue;
        const int grow = u.row0 + q * 128 + row;  // this thread's query
        const bool active = u.row0 + q * 128 + warp * 32 < p.Lq;
        const bool turns = u.nt == 2;
        st.R = st.R_prev = -INFINITY;
        st.l = 0.f;
        XaScales sc;
        float f_row = 0.f, c = -INFINITY;  // 8-bit cache: this row's factor; XaBlockScales::c
        for (int j = u.jb; j < u.je; ++j) {
            const int n = xa_block_keys(u, j);
            uint32_t w[4];
            const bool full = n == 128 && !p.key_mask;
            if (!full) xa_keep(p, u, j, n, w);
            ok = warp_wait(&bars[C::bSFull + q], st.g & 1, lim);
            if (!ok) break;
            if constexpr (KV8) {
                if (j == u.jb) {
                    const int set = uq % C::kExpSets;
                    ok = warp_wait(&bars[C::bExp + set], (uq / C::kExpSets) & 1, lim);
                    if (!ok) break;
                    const int e = reinterpret_cast<const int8_t *>(smem + C::kOffExp)[(set * 2 + q) * 128 + row];
                    f_row = p.scale_log2 * __uint_as_float(uint32_t(127 + e) << 23);
                }
                const float4 *at = reinterpret_cast<const float4 *>(smem + C::kOffScale) + (kv0 + j) % C::kScaleSets * 2;
                const float4 s0 = at[0], s1 = at[1];
                sc.f[0] = fmaxf(f_row * s0.x, 1.2e-38f);  // above 0: -inf times it stays -inf
                sc.f[1] = fmaxf(f_row * s0.y, 1.2e-38f);
                sc.lv[0] = s0.z, sc.lv[1] = s0.w;
                sc.inv_v[0] = s1.x, sc.inv_v[1] = s1.y;
                c = s1.z;
            }
            sm100::tc_fence_after();
            const bool first = j == u.jb;
            if (!active)
                ok = st.idle_block(first, turns);
            else if (full)
                ok = st.template block<4, false>(w, sc, first, turns);
            else if (n > 96)
                ok = st.template block<4>(w, sc, first, turns);
            else if (n > 64)
                ok = st.template block<3>(w, sc, first, turns);
            else if (n > 32)
                ok = st.template block<2>(w, sc, first, turns);
            else
                ok = st.template block<1>(w, sc, first, turns);
            ++st.g;
            st.tb += turns;
            if (!ok) break;
        }
        const bool any = u.je > u.jb;
        // the last P.V product of this tile
        if (ok && any) ok = warp_wait(&bars[C::bPFree + q], (st.g - 1) & 1, lim);
        if (!ok) break;
        sm100::tc_fence_after();
        // 8-bit cache: 2^c in two factors (with 1 / l it may be far from 1)
        const float to_v = KV8 ? (c == -INFINITY ? 0.f : sm100::ex2_approx(0.5f * c)) : 1.f;
        const float inv_l = (st.l > 0.f ? 1.f / st.l : st.l == 0.f ? 0.f : st.l) * to_v;
        if (u.slot >= 0) {
            const size_t prow = (size_t)u.slot * 256 + q * 128 + row;
            const bool valid = bound_row(grow < p.Lq, prow, (size_t)p.tail_ctas * 512);
            // the 8-bit cache's pieces hold O / l, with the sum in the reference:
            // so they lie within float32 wherever the result does
            const bool divided = KV8 && st.l > 0.f;
            const float ref = divided ? st.R_prev + __log2f(st.l) : st.R_prev;
            if (valid) *reinterpret_cast<float2 *>(p.ml + prow * 2) = make_float2(any ? ref : -INFINITY, divided ? 1.f : st.l);
            auto piece = [&](uint32_t x) { return KV8 ? __uint_as_float(x) * to_v * inv_l : __uint_as_float(x); };
            if (any && active) {
                float4 *part = reinterpret_cast<float4 *>(p.o_part + prow * D);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t o[32];
                    sm100::tmem_ld32(st.tO + i * 32, o);
                    if (valid) {
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            part[i * 8 + v] = make_float4(piece(o[4 * v]), piece(o[4 * v + 1]), piece(o[4 * v + 2]),
                                                          piece(o[4 * v + 3]));
                    }
                }
            }
            continue;
        }
        // O / l through shared memory, 64 columns at a time (128-byte rows,
        // the tensor map's swizzle), and out by TMA
        for (int ch = 0; ch < C::kChunks; ++ch) {
            if (row == 0) sm100::bulk_wait_read();  // the previous store has read the stage
            ok = group_sync();
            if (!ok) break;
            if (active) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[32];
                    if (any) {
                        sm100::tmem_ld32(st.tO + ch * 64 + c * 32, o);
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t h[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float a = __uint_as_float(o[8 * v + 2 * i]), b = __uint_as_float(o[8 * v + 2 * i + 1]);
                            if (KV8) a *= to_v, b *= to_v;
                            h[i] = any && st.l != 0.f ? sm100::pack_16x2<F16>(a * inv_l, b * inv_l) : 0u;
                        }
                        *reinterpret_cast<uint4 *>(stage + row * 128 + (((c * 4 + v) ^ (row & 7)) << 4)) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
            }
            sm100::fence_proxy_async();
            ok = group_sync();
            if (!ok) break;
            if (row == 0) {
                sm100::tma_store_4d(&p.tm_o, stage, ch * 64, bound_coord(u.row0 + q * 128, p.Lq),
                                    bound_coord(u.h, p.heads), bound_coord(u.b, p.B));
                sm100::bulk_commit();
            }
        }
    }
    if (row == 0) sm100::bulk_wait_all();
    if (!ok) {
        record_error(kErrDeviceTimeout);
        *abort_flag = 1;
    }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int D, bool KV8, bool F16>
__global__ void __launch_bounds__(XaCfg<D, KV8>::kThreads, 1)
    xa_fwd_kernel(const __grid_constant__ XaParams p) {
    using C = XaCfg<D, KV8>;
    extern __shared__ uint8_t smem_raw[];
    sm100::let_next_kernel_start();
    const uint32_t raw = sm100::smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);  // [0] TMEM base, [1] abort flag
    const int warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kQStages; ++s) {
            sm100::mbar_init(&bars[C::bQFull + s], 1);
            sm100::mbar_init(&bars[C::bQEmpty + s], 1);
            sm100::mbar_init(&bars[C::bQReady + s], 128);
        }
        for (int s = 0; KV8 && s < C::kExpSets; ++s) sm100::mbar_init(&bars[C::bExp + s], 128);
        for (int s = 0; s < C::kStages; ++s) {
            sm100::mbar_init(&bars[C::bKFull + s], KV8 ? 128 : 1);
            sm100::mbar_init(&bars[C::bKEmpty + s], 1);
            sm100::mbar_init(&bars[C::bVFull + s], KV8 ? 128 : 1);
            sm100::mbar_init(&bars[C::bVEmpty + s], 1);
            sm100::mbar_init(&bars[C::bVReady + s], 1);
        }
        for (int s = 0; s < C::kCodeStages; ++s) {
            sm100::mbar_init(&bars[C::bKCFull + s], 1);
            sm100::mbar_init(&bars[C::bKCEmpty + s], 128);
            sm100::mbar_init(&bars[C::bVCFull + s], 1);
            sm100::mbar_init(&bars[C::bVCEmpty + s], 129);
        }
        for (int s = 0; KV8 && s < C::kScaleSets; ++s) sm100::mbar_init(&bars[C::bScale + s], 1);
        for (int q = 0; q < 2; ++q) {
            sm100::mbar_init(&bars[C::bSFull + q], 1);
            sm100::mbar_init(&bars[C::bSFree + q], 128);
            sm100::mbar_init(&bars[C::bPFull + q], 128);
            sm100::mbar_init(&bars[C::bPFree + q], 1);
            for (int k = 0; k < 4; ++k) sm100::mbar_init(&bars[C::bTurn + 4 * q + k], 1);
            sm100::mbar_init(&bars[C::bEpi + q], 128);
            sm100::mbar_init(&bars[C::bDrain + q], 1);
        }
        misc[1] = 0;
        sm100::fence_barrier_init();
    }
    if (warp == C::kCtlWarp) {
        sm100::tmem_alloc(&misc[0], C::kTmemCols);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = misc[0];
    volatile uint32_t *abort_flag = &misc[1];

    if (KV8 && warp >= C::kConvWarp) {
        sm100::setmaxnreg_dec<C::kRegsConv>();
        if constexpr (KV8) xa_convert<D>(p, smem, bars, abort_flag);
    } else if (warp >= C::kCtlWarp) {
        sm100::setmaxnreg_dec<C::kRegsCtl>();
        const int role = warp - C::kCtlWarp;
        if (role == 3) {
            if constexpr (KV8)
                xa_block_scales<D>(p, smem, bars, abort_flag);
            else if (p.kv_lens || p.key_mask)
                xa_clear_unkept<D>(p, smem, bars, abort_flag);
        } else if ((threadIdx.x & 31) == 0) {
            if (role == 0) xa_producer<D, KV8>(p, smem, bars, abort_flag);
            if constexpr (C::kSeparateP) {
                if (role == 1) xa_mma_s<D, KV8, F16>(p, smem, bars, tmem, abort_flag);
                if (role == 2) xa_mma_pv<D, KV8, F16>(p, smem, bars, tmem, abort_flag);
            } else {
                if (role == 1) xa_mma<D, KV8, F16>(p, smem, bars, tmem, abort_flag);
            }
        }
    } else {
        sm100::setmaxnreg_inc<C::kRegsSoftmax>();
        xa_softmax<D, KV8, F16>(p, smem, bars, tmem, abort_flag, warp >> 2);
    }

    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    if (warp == C::kCtlWarp) {
        __syncwarp();
        sm100::tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Merging partial results. With m* the largest reference of a row's pieces,
//   o = sum_s 2^(m_s - m*) O_s / sum_s 2^(m_s - m*) l_s
// (cut units over the 8-bit cache: O_s / l_s, m_s + log2 l_s and 1, `divided`);
// a piece without keys has m_s = -inf and l_s = 0 and wrote no O. One whose
// scores are all NaN has m_s = -inf too (a maximum passes NaN over) and l_s =
// NaN: its sum joins as it stands, so that the row is NaN however it was split.
struct XaCombineParams {
    const float *o_part, *ml;
    void *o;
    long long sb, sh, st;  // strides of o in elements
    int n_splits, rows, heads, Lq;
    // xa_tail_kernel: the first cut unit, and the CTAs that hold a cut unit's
    // first and last block
    int first_unit, n_blk;
    FastDiv by_qpairs, by_heads;
    int n_qpairs;
    const int *kv_lens;  // null: batch rows as they stand
    int B, Lk;
    int divided;         // pieces hold O / l: weights are divided too, so that the sum keeps the result's range
    short first_cta[kXaMaxTailCtas], last_cta[kXaMaxTailCtas];
    int tail_start[kXaMaxTailCtas];
};

// One row by one warp: n <= 32 * kPerLane pieces, row_of(s) the row of piece s
// in o_part and ml. References and sums are read together, O eight pieces at
// a time.
template <int D, bool F16, int kPerLane, typename RowOf>
__device__ __forceinline__ void xa_merge_row(const XaCombineParams &p, int n, RowOf row_of, uint16_t *dst) {
    constexpr int kPer = D / 32;  // elements of O per lane
    constexpr int kAhead = 8;
    const int lane = threadIdx.x & 31;
    float2 ml[kPerLane];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        ml[i] = lane + 32 * i < n ? __ldcg(reinterpret_cast<const float2 *>(p.ml) + row_of(lane + 32 * i))
                                  : make_float2(-INFINITY, 0.f);
        m = fmaxf(m, ml[i].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float w[kPerLane], L = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        w[i] = ml[i].x == -INFINITY ? 0.f : sm100::ex2_approx(ml[i].x - m);
        L = ml[i].x == -INFINITY ? L + ml[i].y : fmaf(w[i], ml[i].y, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = L > 0.f ? 1.f / L : L;
    if (p.divided) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) w[i] *= inv;
    }
    float acc[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    for (int s0 = 0; s0 < n; s0 += kAhead) {
        float o[kAhead][kPer], wgt[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int s = s0 + i;
            float mine = w[0];
#pragma unroll
            for (int k = 1; k < kPerLane; ++k) mine = s >> 5 == k ? w[k] : mine;
            wgt[i] = __shfl_sync(0xffffffffu, mine, s & 31);
            const bool in = s < n && wgt[i] != 0.f;
            const float *src = p.o_part + (in ? (size_t)row_of(s) * D : 0) + lane * kPer;
#pragma unroll
            for (int c = 0; c < kPer; ++c) o[i][c] = in ? __ldcg(src + c) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] = fmaf(wgt[i], o[i][c], acc[c]);
    }
    const float last = p.divided && L > 0.f ? 1.f : inv;
#pragma unroll
    for (int c = 0; c < kPer; c += 2)
        reinterpret_cast<uint32_t *>(dst + lane * kPer)[c / 2] =
            L == 0.f ? 0u : sm100::pack_16x2<F16>(acc[c] * last, acc[c + 1] * last);
}

// xa_few_kernel's key-range splits.
template <int D, bool F16>
__global__ void __launch_bounds__(128) xa_combine_kernel(const __grid_constant__ XaCombineParams p) {
    const int r = blockIdx.x * 4 + (threadIdx.x >> 5);
    sm100::wait_for_previous_kernel();
    if (r >= p.rows) return;
    const int bh = r / p.Lq, i = r - bh * p.Lq, b = bh / p.heads, h = bh - b * p.heads;
    xa_merge_row<D, F16, kXaMaxSplits / 32>(
        p, p.n_splits, [&](int s) { return (size_t)s * p.rows + r; },
        static_cast<uint16_t *>(p.o) + b * p.sb + h * p.sh + i * p.st);
}

// The pieces of cut units: 64 blocks of four rows to a unit.
template <int D, bool F16>
__global__ void __launch_bounds__(128) xa_tail_kernel(const __grid_constant__ XaCombineParams p) {
    const int t = blockIdx.x >> 6, r = (blockIdx.x & 63) * 4 + (threadIdx.x >> 5);
    const int unit = p.first_unit + t, bh = p.by_qpairs(unit), row = (unit - bh * p.n_qpairs) * 256 + r;
    const int c0 = p.first_cta[t], c1 = p.last_cta[t];
    sm100::wait_for_previous_kernel();
    if (row >= p.Lq || c0 == c1) return;  // no row, or the unit was not cut
    const int rank = p.by_heads(bh), h = bh - rank * p.heads;
    const int b = p.kv_lens ? xa_row_of_rank(p.kv_lens, p.B, p.Lk, rank) : rank;
    // a CTA's first piece is in its slot 0: of the unit's CTAs, only the first
    // may have begun with another unit
    const int begun = p.tail_start[c0] < t * p.n_blk;
    xa_merge_row<D, F16, kXaMaxTailCtas / 32>(
        p, c1 - c0 + 1, [&](int s) { return (size_t)(2 * (c0 + s) + (s == 0 ? begun : 0)) * 256 + r; },
        static_cast<uint16_t *>(p.o) + b * p.sb + h * p.sh + row * p.st);
}

}  // namespace npa
