// api.cu - host side of the C ABI declared in include/npa.h: argument
// validation, geometry resolution, TMA tensor-map encoding and the launches of
// the sm_100a kernels. Nothing here computes attention or the combines.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "npa.h"
#include "asg_combine.cuh"
#include "cross_attention.cuh"
#include "cross_attention_few.cuh"
#include "cross_attention_short.cuh"
#include "group_norm.cuh"
#include "kv8_store.cuh"
#include "md_combine.cuh"
#include "npa_fwd_kernel.cuh"

namespace {

using npa::FwdParams;

// The kernel's bounded waits give up after this long (a healthy wait is far
// below a millisecond).
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

#ifdef NPA_DEBUG_BOUNDS
// Bounds-checking build: wait limit (microseconds) of the next attention
// launch whose CTA 0 withholds one arrival; 0 = none pending.
std::atomic<unsigned> g_debug_stall_us{0};
#endif

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_mu;
EncodeTiledFn g_encode = nullptr;
constexpr int kMaxDevices = 64;
struct DeviceState {
    bool checked = false;
    npa_status status = NPA_ERR_UNSUPPORTED;
    int sm_count = 0;
    int l2_bytes = 0;
    bool xa_checked = false;  // the cross-attention kernels (on their first use)
    npa_status xa_status = NPA_ERR_UNSUPPORTED;
    // clusters of xa_few_kernel that run at once: [d = 128][8-bit][two row tiles][size]
    int xf_clusters[2][2][2][npa::kXaFewCluster + 1] = {};
    bool gn_checked = false;  // the group norm's kernels
    npa_status gn_status = NPA_ERR_UNSUPPORTED;
};
DeviceState g_dev[kMaxDevices];

// Sets a kernel's shared-memory limit and checks that it was compiled with the
// register count its warp roles redistribute (0: none): the softmax warpgroups'
// setmaxnreg.inc draws on the registers the block was launched with, and would
// never complete if the launch held fewer. NPA_ERR_UNSUPPORTED is for good;
// NPA_ERR_CUDA, a call that failed, is asked again next time.
npa_status prepare(const void *kernel, int registers, int smem_bytes) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) return NPA_ERR_CUDA;
    if (registers && attr.numRegs != registers) return NPA_ERR_UNSUPPORTED;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) == cudaSuccess
               ? NPA_OK
               : NPA_ERR_CUDA;
}

template <int D, bool GQ, bool MD = false>
npa_status prepare_kernel() {
    using C = npa::KCfg<D, 2, 128>;
    return prepare((const void *)npa::npa_fwd_kernel<D, 2, 128, GQ, MD>, (int)C::kRegsLaunch, C::kSmemBytes);
}

// The first status that is not NPA_OK.
npa_status first_fault(std::initializer_list<npa_status> all) {
    for (const npa_status s : all)
        if (s != NPA_OK) return s;
    return NPA_OK;
}

// Resolves the tensor-map encoder and checks (once per device) that the
// current device is an sm_100 part; sets the kernels' shared-memory limits.
// On success *sm_count holds the device's multiprocessor count.
npa_status ensure_ready(int *sm_count = nullptr, int *l2_bytes = nullptr) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NPA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return NPA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult qres;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &qres) != cudaSuccess ||
            qres != cudaDriverEntryPointSuccess || fn == nullptr)
            return NPA_ERR_CUDA;
        g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    DeviceState &ds = g_dev[dev];
    if (!ds.checked) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return NPA_ERR_CUDA;
        if (cudaDeviceGetAttribute(&ds.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            ds.sm_count < 1 || cudaDeviceGetAttribute(&ds.l2_bytes, cudaDevAttrL2CacheSize, dev) != cudaSuccess)
            return NPA_ERR_CUDA;
        const npa_status st = major != 10 || minor != 0
                                  ? NPA_ERR_UNSUPPORTED
                                  : first_fault({prepare_kernel<64, false>(), prepare_kernel<128, false>(),
                                                 prepare_kernel<64, false, true>(), prepare_kernel<128, false, true>(),
                                                 prepare_kernel<64, true>(), prepare_kernel<128, true>()});
        if (st == NPA_ERR_CUDA) return st;
        ds.status = st;
        ds.checked = true;
    }
    if (sm_count) *sm_count = ds.sm_count;
    if (l2_bytes) *l2_bytes = ds.l2_bytes;
    return ds.status;
}

// The per-CTA unit lists take 0.1-0.5 ms to build on the host, so the last
// few are kept, keyed by everything they depend on.
struct SchedKey {
    int BH, H, W, G, Ph, Pw, mh, mw, kc_log2, kr, n_qblocks, patch_begin, patch_count, grid, head_major;
    bool operator==(const SchedKey &o) const { return std::memcmp(this, &o, sizeof(SchedKey)) == 0; }
};
struct SchedEntry {
    SchedKey key;
    unsigned long long used = 0;  // 0: empty
    int n_sched = 0;
    unsigned short cta_first[npa::kMaxSchedCtas + 1];
    unsigned short sched[npa::kMaxSchedUnits];
};
constexpr int kSchedCacheEntries = 8;
std::mutex g_sched_mu;
SchedEntry g_sched_cache[kSchedCacheEntries];
unsigned long long g_sched_clock = 0;

// Fills prm's per-CTA lists (npa::build_schedule), from the cache when the
// same geometry was scheduled recently.
void schedule_units(FwdParams &prm, int grid, bool head_major) {
    SchedKey key;
    std::memset(&key, 0, sizeof(key));
    key = SchedKey{prm.BH, prm.H,      prm.W,  prm.G,         prm.Ph,          prm.Pw,          prm.mh,          prm.mw,
                   prm.kc_log2, prm.kr, prm.n_qblocks, prm.patch_begin, prm.patch_count, grid, head_major ? 1 : 0};
    std::lock_guard<std::mutex> lock(g_sched_mu);
    SchedEntry *victim = &g_sched_cache[0];
    for (SchedEntry &e : g_sched_cache) {
        if (e.used && e.key == key) {
            e.used = ++g_sched_clock;
            prm.n_sched = e.n_sched;
            std::memcpy(prm.cta_first, e.cta_first, sizeof(e.cta_first));
            std::memcpy(prm.sched, e.sched, sizeof(unsigned short) * (size_t)e.n_sched);
            return;
        }
        if (e.used < victim->used) victim = &e;
    }
    npa::build_schedule(prm, grid, head_major);
    victim->key = key;
    victim->used = ++g_sched_clock;
    victim->n_sched = prm.n_sched;
    std::memcpy(victim->cta_first, prm.cta_first, sizeof(prm.cta_first));
    std::memcpy(victim->sched, prm.sched, sizeof(unsigned short) * (size_t)prm.n_sched);
}

// Rectangle form of both geometries (see npa_geometry.cuh).
struct Geo {
    int H, W, Ph, Pw, mh, mw;
};

// Sum over the patches along one axis of (patch extent) x (window extent).
long long axis_pair_sum(int L, int P, int m) {
    long long s = 0;
    for (int p0 = 0; p0 < L; p0 += P) {
        const int p1 = p0 + P < L ? p0 + P : L;
        const int w0 = p0 - m > 0 ? p0 - m : 0;
        const int w1 = p1 + m < L ? p1 + m : L;
        s += (long long)(p1 - p0) * (w1 - w0);
    }
    return s;
}

// Sum over the patches along one axis of the window extent padded to `tile`.
long long axis_window_sum(int L, int P, int m, int tile, bool padded) {
    long long s = 0;
    for (int p0 = 0; p0 < L; p0 += P) {
        const int p1 = p0 + P < L ? p0 + P : L;
        const int w0 = p0 - m > 0 ? p0 - m : 0;
        const int w1 = p1 + m < L ? p1 + m : L;
        const int e = w1 - w0;
        s += padded ? (long long)((e + tile - 1) / tile) * tile : e;
    }
    return s;
}

// Key block shape for blocks of kb keys: 2^lg columns x kb/2^lg rows, chosen
// to waste the fewest key slots over all windows (ties go to the wider box:
// longer contiguous runs).
int choose_kc_log2(const Geo &g, int kb) {
    const int top = kb == 128 ? 7 : 6;
    int best_lg = top;
    long long best_waste = LLONG_MAX;
    const long long exact = axis_window_sum(g.W, g.Pw, g.mw, 1, false) * axis_window_sum(g.H, g.Ph, g.mh, 1, false);
    for (int lg = top; lg >= top - 3; --lg) {
        const int kc = 1 << lg, kr = kb >> lg;
        const long long padded =
            axis_window_sum(g.W, g.Pw, g.mw, kc, true) * axis_window_sum(g.H, g.Ph, g.mh, kr, true);
        if (padded - exact < best_waste) {
            best_waste = padded - exact;
            best_lg = lg;
        }
    }
    return best_lg;
}

// Query tile shape: qc patch columns x qr patch rows (qc*qr <= 128), chosen to
// need the fewest tiles per patch.
void choose_q_tile(int Ph, int Pw, int *qc_out, int *qr_out) {
    const int cands[6] = {Pw < 128 ? Pw : 128, 128, 64, 32, 16, 8};
    long long best = LLONG_MAX;
    int bc = 128, br = 1;
    for (int i = 0; i < 6; ++i) {
        const int c = cands[i];
        if (c < 1 || c > 128) continue;
        int r = 128 / c;
        if (r > Ph) r = Ph;
        if (r < 1) r = 1;
        const long long tiles = (long long)((Pw + c - 1) / c) * ((Ph + r - 1) / r);
        if (tiles < best) {
            best = tiles;
            bc = c;
            br = r;
        }
    }
    *qc_out = bc;
    *qr_out = br;
}

// Overlapping-window mode: the query tile box (qc columns x qr rows, qc*qr <=
// 128) that needs the fewest tiles over all windows; windows form a grid, so
// the count is (sum over column windows of ceil(width/qc)) x (sum over row
// windows of ceil(height/qr)). tiles_c / tiles_r cover the largest window.
void choose_q_tile_md(const Geo &g, int *qc_out, int *qr_out, int *tiles_c, int *tiles_r) {
    const int nph = (g.H + g.Ph - 1) / g.Ph, npw = (g.W + g.Pw - 1) / g.Pw;
    long long best = LLONG_MAX;
    for (int qc = 128; qc >= 8; qc /= 2) {
        const int qr = 128 / qc;
        long long sc = 0, sr = 0;
        int mc = 0, mr = 0;
        for (int j = 0; j < npw; ++j) {
            const int ww = std::min(g.W, (j + 1) * g.Pw + g.mw) - std::max(0, j * g.Pw - g.mw);
            sc += (ww + qc - 1) / qc;
            mc = std::max(mc, (ww + qc - 1) / qc);
        }
        for (int i = 0; i < nph; ++i) {
            const int wh = std::min(g.H, (i + 1) * g.Ph + g.mh) - std::max(0, i * g.Ph - g.mh);
            sr += (wh + qr - 1) / qr;
            mr = std::max(mr, (wh + qr - 1) / qr);
        }
        if (sc * sr < best) {
            best = sc * sr;
            *qc_out = qc;
            *qr_out = qr;
            *tiles_c = mc;
            *tiles_r = mr;
        }
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

bool encode(CUtensorMap *m, const void *base, cuuint32_t rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

npa_status validate_common(const void *q, const void *k, const void *v, void *o, int B, int heads, int H, int W,
                           int d, const npa_global_kv *gkv, int *G_out) {
    if (!q || !k || !v || !o) return NPA_ERR_INVALID_ARG;
    if (B < 1 || heads < 1 || H < 1 || W < 1 || d < 1) return NPA_ERR_INVALID_ARG;
    int G = 0;
    if (gkv && gkv->n_tokens != 0) {
        if (gkv->n_tokens < 0 || !gkv->k || !gkv->v) return NPA_ERR_INVALID_ARG;
        G = gkv->n_tokens;
    }
    if (d != 64 && d != 128) return NPA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return NPA_ERR_MISALIGNED;
    if (G && (!aligned16(gkv->k) || !aligned16(gkv->v))) return NPA_ERR_MISALIGNED;
    const long long N = (long long)H * W;
    const long long BH = (long long)B * heads;
    // tensor-map limits (strides < 2^40 bytes) and 32-bit unit/coordinate math
    if (N * d * 2 >= (1LL << 40) || BH > INT_MAX / 4 || N > INT_MAX || (long long)G * d * 2 >= (1LL << 40))
        return NPA_ERR_UNSUPPORTED;
    const size_t bytes = (size_t)(BH * N * d * 2);
    const size_t gbytes = (size_t)(BH * G * d * 2);
    if (overlaps(o, bytes, q, bytes) || overlaps(o, bytes, k, bytes) || overlaps(o, bytes, v, bytes))
        return NPA_ERR_INVALID_ARG;
    if (G && (overlaps(o, bytes, gkv->k, gbytes) || overlaps(o, bytes, gkv->v, gbytes))) return NPA_ERR_INVALID_ARG;
    *G_out = G;
    return NPA_OK;
}

// ks / vs (both or neither): previous-step keys/values for the rows of a
// window outside its patch. [patch_begin, patch_begin + patch_count): the
// patches computed, in natural numbering; patch_count < 0 means all.
npa_status launch(const void *q, const void *k, const void *v, const void *ks, const void *vs, void *o, int B,
                  int heads, int d, const Geo &g, int G, const npa_global_kv *gkv, int patch_begin, int patch_count,
                  npa_stream_t stream, float *md_part = nullptr) {
    int sm_count = 0, l2_bytes = 0;
    npa_status st = ensure_ready(&sm_count, &l2_bytes);
    if (st != NPA_OK) return st;
    const int nt = 2;  // query tiles per work unit

    FwdParams prm;
    std::memset(&prm, 0, sizeof(prm));
    prm.o = o;
    prm.H = g.H;
    prm.W = g.W;
    prm.G = G;
    prm.Ph = g.Ph;
    prm.Pw = g.Pw;
    prm.mh = g.mh;
    prm.mw = g.mw;
    prm.nPh = (g.H + g.Ph - 1) / g.Ph;
    prm.nPw = (g.W + g.Pw - 1) / g.Pw;
    if (md_part) {
        if (prm.nPh > npa::kMaxMdAxis || prm.nPw > npa::kMaxMdAxis) return NPA_ERR_UNSUPPORTED;
        choose_q_tile_md(g, &prm.qc, &prm.qr, &prm.tiles_c, &prm.tiles_r);
        prm.md = 1;
        prm.md_part = md_part;
        prm.md_rows = npa::md_axis_offset(g.H, g.Ph, g.mh, prm.nPh);
        prm.md_tw = npa::md_axis_offset(g.W, g.Pw, g.mw, prm.nPw);
    } else {
        choose_q_tile(g.Ph, g.Pw, &prm.qc, &prm.qr);
        prm.tiles_c = (g.Pw + prm.qc - 1) / prm.qc;
        prm.tiles_r = (g.Ph + prm.qr - 1) / prm.qr;
    }
    prm.kb = 128;
    prm.tiles_per_unit = nt;
    prm.kc_log2 = choose_kc_log2(g, prm.kb);
    prm.kr = prm.kb >> prm.kc_log2;
    prm.n_qblocks = (prm.tiles_c * prm.tiles_r + nt - 1) / nt;
    prm.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d));
    prm.wait_limit_ns = kWaitLimitNs;
#ifdef NPA_DEBUG_BOUNDS
    if (const unsigned stall_us = g_debug_stall_us.exchange(0)) {
        prm.debug_stall = 1;
        prm.wait_limit_ns = stall_us * 1000ull;
    }
#endif

    if ((long long)prm.nPh * prm.nPw > INT_MAX / 4) return NPA_ERR_UNSUPPORTED;
    prm.patch_begin = patch_begin;
    prm.patch_count = patch_count < 0 ? prm.nPh * prm.nPw : patch_count;
    prm.two_source = ks != nullptr;
    const long long units = (long long)B * heads * prm.patch_count * prm.n_qblocks;
    if (units > INT_MAX / 2) return NPA_ERR_UNSUPPORTED;

    const int BH = B * heads;
    prm.BH = BH;
    prm.n_units = (int)units;
    npa::order_patches(prm);
    // persistent grid: one CTA per multiprocessor (shared memory and TMEM
    // admit one), each walking its host-built list of units (or every
    // gridDim.x-th unit); when the keys and values of all heads do not fit in
    // L2, the lists run head by head
    const unsigned grid = (unsigned)(units < sm_count ? units : sm_count);
    if (!md_part) {
        const double kv_bytes = 4.0 * BH * (double)g.H * g.W * d + 4.0 * BH * (double)G * d;
        schedule_units(prm, (int)grid, kv_bytes > (double)l2_bytes);
    }
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)g.W, (cuuint64_t)g.H, (cuuint64_t)BH};
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)g.W * d * 2, (cuuint64_t)g.H * g.W * d * 2};
    const cuuint32_t qbox[4] = {64, (cuuint32_t)prm.qc, (cuuint32_t)prm.qr, 1};
    const cuuint32_t kbox[4] = {64, (cuuint32_t)(1 << prm.kc_log2), (cuuint32_t)prm.kr, 1};
    if (!encode(&prm.tm_q, q, 4, dims, strides, qbox) || !encode(&prm.tm_k, k, 4, dims, strides, kbox) ||
        !encode(&prm.tm_v, v, 4, dims, strides, kbox))
        return NPA_ERR_CUDA;
    if (ks && (!encode(&prm.tm_ks, ks, 4, dims, strides, kbox) || !encode(&prm.tm_vs, vs, 4, dims, strides, kbox)))
        return NPA_ERR_CUDA;
    if (G > 0) {
        const cuuint64_t gdims[3] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)BH};
        const cuuint64_t gstrides[2] = {(cuuint64_t)d * 2, (cuuint64_t)G * d * 2};
        const cuuint32_t gbox[3] = {64, (cuuint32_t)prm.kb, 1};
        if (!encode(&prm.tm_gk, gkv->k, 3, gdims, gstrides, gbox) ||
            !encode(&prm.tm_gv, gkv->v, 3, gdims, gstrides, gbox))
            return NPA_ERR_CUDA;
    }

    void *args[1] = {&prm};
    cudaError_t e;
    const void *kernel;
    unsigned threads, smem;
    if (d == 64 && md_part) {
        kernel = (const void *)npa::npa_fwd_kernel<64, 2, 128, false, true>;
        threads = npa::KCfg<64, 2, 128>::kThreads;
        smem = npa::KCfg<64, 2, 128>::kSmemBytes;
    } else if (d == 128 && md_part) {
        kernel = (const void *)npa::npa_fwd_kernel<128, 2, 128, false, true>;
        threads = npa::KCfg<128, 2, 128>::kThreads;
        smem = npa::KCfg<128, 2, 128>::kSmemBytes;
    } else if (d == 64) {
        kernel = (const void *)npa::npa_fwd_kernel<64, 2, 128, false>;
        threads = npa::KCfg<64, 2, 128>::kThreads;
        smem = npa::KCfg<64, 2, 128>::kSmemBytes;
    } else {
        kernel = (const void *)npa::npa_fwd_kernel<128, 2, 128, false>;
        threads = npa::KCfg<128, 2, 128>::kThreads;
        smem = npa::KCfg<128, 2, 128>::kSmemBytes;
    }
    e = cudaLaunchKernel(kernel, dim3(grid), dim3(threads), args, smem, (cudaStream_t)stream);
    if (e != cudaSuccess) return NPA_ERR_CUDA;
    if (md_part) {
        npa::MdCombineParams cp;
        std::memset(&cp, 0, sizeof(cp));
        cp.part = md_part;
        cp.o = static_cast<__nv_bfloat16 *>(o);
        cp.H = g.H;
        cp.W = g.W;
        cp.Ph = g.Ph;
        cp.Pw = g.Pw;
        cp.mh = g.mh;
        cp.mw = g.mw;
        cp.nPh = prm.nPh;
        cp.nPw = prm.nPw;
        cp.BH = BH;
        cp.md_rows = prm.md_rows;
        cp.md_tw = prm.md_tw;
        for (int i = 0; i < prm.nPh; ++i) cp.rh[i] = npa::md_axis_offset(g.H, g.Ph, g.mh, i);
        for (int j = 0; j < prm.nPw; ++j) cp.cw[j] = npa::md_axis_offset(g.W, g.Pw, g.mw, j);
        void *cargs[1] = {&cp};
        const long long tokens = (long long)BH * g.H * g.W;
        const long long per_block = 256 / (d / 4);  // tokens per 256-thread block
        const dim3 cgrid((unsigned)((tokens + per_block - 1) / per_block));
        if (d == 64)
            e = cudaLaunchKernel((const void *)npa::md_combine_kernel<64>, cgrid, dim3(256), cargs, 0,
                                 (cudaStream_t)stream);
        else
            e = cudaLaunchKernel((const void *)npa::md_combine_kernel<128>, cgrid, dim3(256), cargs, 0,
                                 (cudaStream_t)stream);
        if (e != cudaSuccess) return NPA_ERR_CUDA;
    }
    return NPA_OK;
}

// ---------------------------------------------------------------------------
// Global-token queries (text-query half of joint attention)
// ---------------------------------------------------------------------------
struct GqPlan {
    int kc_log2, kr, n_blocks, n_qblocks, base_units, splits;
    size_t split_bytes;  // workspace bytes per key-range split
};

GqPlan plan_gq(int B, int heads, int H, int W, int d, int G, int sm_count) {
    GqPlan pl;
    const Geo g{H, W, H, W, 0, 0};
    pl.kc_log2 = choose_kc_log2(g, 128);
    pl.kr = 128 >> pl.kc_log2;
    pl.n_blocks = ((W + (1 << pl.kc_log2) - 1) >> pl.kc_log2) * ((H + pl.kr - 1) / pl.kr) + (G + 127) / 128;
    const int tiles = (G + 127) / 128;
    pl.n_qblocks = (tiles + 1) / 2;
    pl.base_units = B * heads * pl.n_qblocks;
    // split the key range until the units roughly fill the GPU once
    int s = (sm_count + pl.base_units / 2) / pl.base_units;
    if (s < 1) s = 1;
    if (s > 16) s = 16;
    if (s > pl.n_blocks) s = pl.n_blocks;
    pl.splits = s;
    pl.split_bytes = (size_t)B * heads * G * (d + 2) * sizeof(float);
    return pl;
}

npa_status launch_gq(const void *gq, const void *k, const void *v, const void *gk, const void *gv, void *go, int B,
                     int heads, int H, int W, int d, int G, float *o_part, float *ml, int splits, int sm_count,
                     npa_stream_t stream) {
    const GqPlan pl = plan_gq(B, heads, H, W, d, G, sm_count);
    FwdParams prm;
    std::memset(&prm, 0, sizeof(prm));
    prm.o = go;
    prm.H = H;
    prm.W = W;
    prm.G = G;
    prm.Ph = H;
    prm.Pw = W;
    prm.nPh = prm.nPw = 1;
    prm.kb = 128;
    prm.tiles_per_unit = 2;
    prm.kc_log2 = pl.kc_log2;
    prm.kr = pl.kr;
    prm.n_qblocks = pl.n_qblocks;
    prm.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d));
    prm.wait_limit_ns = kWaitLimitNs;
    prm.BH = B * heads;
    prm.n_splits = splits;
    prm.gq_tiles = (G + 127) / 128;
    prm.o_part = o_part;
    prm.ml = ml;
    const long long units = (long long)prm.BH * pl.n_qblocks * splits;
    if (units > INT_MAX / 2) return NPA_ERR_UNSUPPORTED;
    prm.n_units = (int)units;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)W, (cuuint64_t)H, (cuuint64_t)prm.BH};
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)W * d * 2, (cuuint64_t)H * W * d * 2};
    const cuuint32_t kbox[4] = {64, (cuuint32_t)(1 << pl.kc_log2), (cuuint32_t)pl.kr, 1};
    const cuuint64_t gdims[3] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)prm.BH};
    const cuuint64_t gstrides[2] = {(cuuint64_t)d * 2, (cuuint64_t)G * d * 2};
    const cuuint32_t gbox[3] = {64, 128, 1};
    if (!encode(&prm.tm_k, k, 4, dims, strides, kbox) || !encode(&prm.tm_v, v, 4, dims, strides, kbox) ||
        !encode(&prm.tm_gk, gk, 3, gdims, gstrides, gbox) || !encode(&prm.tm_gv, gv, 3, gdims, gstrides, gbox) ||
        !encode(&prm.tm_gq, gq, 3, gdims, gstrides, gbox))
        return NPA_ERR_CUDA;
    const unsigned grid = (unsigned)(units < sm_count ? units : sm_count);
    void *args[1] = {&prm};
    cudaError_t e;
    if (d == 64) {
        using C = npa::KCfg<64, 2, 128>;
        e = cudaLaunchKernel((const void *)npa::npa_fwd_kernel<64, 2, 128, true>, dim3(grid), dim3(C::kThreads),
                             args, C::kSmemBytes, (cudaStream_t)stream);
    } else {
        using C = npa::KCfg<128, 2, 128>;
        e = cudaLaunchKernel((const void *)npa::npa_fwd_kernel<128, 2, 128, true>, dim3(grid), dim3(C::kThreads),
                             args, C::kSmemBytes, (cudaStream_t)stream);
    }
    if (e != cudaSuccess) return NPA_ERR_CUDA;
    if (splits > 1) {
        const int rows = prm.BH * G;
        const float *op = o_part, *mlp = ml;
        __nv_bfloat16 *gop = static_cast<__nv_bfloat16 *>(go);
        int ns = splits, nr = rows;
        void *cargs[5] = {&op, &mlp, &gop, &ns, &nr};
        const dim3 cgrid((unsigned)((rows + 7) / 8));
        if (d == 64)
            e = cudaLaunchKernel((const void *)npa::gq_combine_kernel<64>, cgrid, dim3(256), cargs, 0,
                                 (cudaStream_t)stream);
        else
            e = cudaLaunchKernel((const void *)npa::gq_combine_kernel<128>, cgrid, dim3(256), cargs, 0,
                                 (cudaStream_t)stream);
        if (e != cudaSuccess) return NPA_ERR_CUDA;
    }
    return NPA_OK;
}

npa_status validate_gq(const void *gq, const void *k, const void *v, const void *gk, const void *gv, void *go,
                       int B, int heads, int H, int W, int d, int G) {
    if (!gq || !k || !v || !gk || !gv || !go) return NPA_ERR_INVALID_ARG;
    if (B < 1 || heads < 1 || H < 1 || W < 1 || G < 1) return NPA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return NPA_ERR_UNSUPPORTED;
    if (!aligned16(gq) || !aligned16(k) || !aligned16(v) || !aligned16(gk) || !aligned16(gv) || !aligned16(go))
        return NPA_ERR_MISALIGNED;
    const long long N = (long long)H * W, BH = (long long)B * heads;
    if (N * d * 2 >= (1LL << 40) || BH > INT_MAX / 64 || N > INT_MAX || (long long)G * d * 2 >= (1LL << 40) ||
        BH * G > INT_MAX / 2)
        return NPA_ERR_UNSUPPORTED;
    const size_t gbytes = (size_t)(BH * G * d * 2), ibytes = (size_t)(BH * N * d * 2);
    if (overlaps(go, gbytes, gq, gbytes) || overlaps(go, gbytes, gk, gbytes) || overlaps(go, gbytes, gv, gbytes) ||
        overlaps(go, gbytes, k, ibytes) || overlaps(go, gbytes, v, ibytes))
        return NPA_ERR_INVALID_ARG;
    return NPA_OK;
}

// ---------------------------------------------------------------------------
// Fixed scratch for npa_global_query_attention_fwd_noalloc: the key-range
// split partials live in this file-scope device array instead of caller
// memory. Every GPU that loads the library holds it until the process exits.
// In host code g_noalloc_scratch only stands for the symbol; its device
// address is fetched once per device with cudaGetSymbolAddress (with that
// device current) and passed to the kernels.
// ---------------------------------------------------------------------------
constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];
void *g_noalloc_addr[kMaxDevices] = {};

int neighbor_rows(int s, double p) {
    if (s < 1 || !(p >= 0.0) || !(p <= 1.0)) return -1;
    int r = (int)std::ceil(p * (double)s - 1e-9);
    if (r < 0) r = 0;
    if (r > s) r = s;
    return r;
}

// Overlapping-window mode: bytes of float32 window partials.
size_t md_workspace_bytes(int B, int heads, int H, int W, int d, int patch, int margin) {
    const long long rows = npa::md_axis_offset(H, patch, margin, (H + patch - 1) / patch);
    const long long cols = npa::md_axis_offset(W, patch, margin, (W + patch - 1) / patch);
    return (size_t)B * heads * rows * cols * d * sizeof(float);
}

double useful_flops(int B, int heads, int d, const Geo &g, int G) {
    const double pairs = (double)axis_pair_sum(g.H, g.Ph, g.mh) * (double)axis_pair_sum(g.W, g.Pw, g.mw) +
                         (double)g.H * g.W * G;
    return 4.0 * d * (double)B * heads * pairs;
}

// ---------------------------------------------------------------------------
// Cross attention, 16-bit keys or the 8-bit cache
// ---------------------------------------------------------------------------
template <int D, bool KV8, bool F16>
npa_status prepare_xa_kernel() {
    using C = npa::XaCfg<D, KV8>;
    return prepare((const void *)npa::xa_fwd_kernel<D, KV8, F16>, (int)C::kRegsLaunch, C::kSmemBytes);
}

constexpr int kMaxSmem = 227 * 1024;

template <int D, bool F16>
npa_status prepare_xs_kernel() {
    using C = npa::XsCfg<D>;
    return prepare((const void *)npa::xa_short_kernel<D, F16>, C::kSplitRegs ? (int)C::kRegsLaunch : 0, kMaxSmem);
}

// xa_few_kernel's dynamic shared memory.
unsigned xf_smem(int d, int tiles) { return 8 * tiles * (npa::kXaFewWarps * (d + 2) + 2) * sizeof(float); }

// How many clusters of each size run at once: out[size], of single blocks out[1].
template <int D, bool KV8, int NT>
npa_status count_xf_clusters(int (&out)[npa::kXaFewCluster + 1]) {
    const void *kernel = (const void *)npa::xa_few_kernel<D, KV8, false, NT>;
    for (int s = 1; s <= npa::kXaFewCluster; ++s) {
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)s;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg;
        std::memset(&cfg, 0, sizeof(cfg));
        cfg.gridDim = dim3((unsigned)s);
        cfg.blockDim = dim3(32 * npa::kXaFewWarps);
        cfg.dynamicSmemBytes = xf_smem(D, NT);
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&out[s], kernel, &cfg) != cudaSuccess) return NPA_ERR_CUDA;
        if (out[s] < 1) return NPA_ERR_UNSUPPORTED;
    }
    return NPA_OK;
}

// ensure_ready plus the cross-attention kernels' limits, once per device.
npa_status ensure_xa_ready(int *sm_count, const DeviceState **state = nullptr) {
    const npa_status st = ensure_ready(sm_count);
    if (st != NPA_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NPA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState &ds = g_dev[dev];
    if (!ds.xa_checked) {
        const npa_status xa = first_fault(
            {prepare_xa_kernel<64, false, false>(), prepare_xa_kernel<64, false, true>(),
             prepare_xa_kernel<128, false, false>(), prepare_xa_kernel<128, false, true>(),
             prepare_xa_kernel<64, true, false>(), prepare_xa_kernel<128, true, false>(), prepare_xs_kernel<64, false>(),
             prepare_xs_kernel<64, true>(), prepare_xs_kernel<128, false>(), prepare_xs_kernel<128, true>(),
             count_xf_clusters<64, false, 1>(ds.xf_clusters[0][0][0]),
             count_xf_clusters<64, false, 2>(ds.xf_clusters[0][0][1]),
             count_xf_clusters<64, true, 1>(ds.xf_clusters[0][1][0]),
             count_xf_clusters<64, true, 2>(ds.xf_clusters[0][1][1]),
             count_xf_clusters<128, false, 1>(ds.xf_clusters[1][0][0]),
             count_xf_clusters<128, false, 2>(ds.xf_clusters[1][0][1]),
             count_xf_clusters<128, true, 1>(ds.xf_clusters[1][1][0]),
             count_xf_clusters<128, true, 2>(ds.xf_clusters[1][1][1])});
        if (xa == NPA_ERR_CUDA) return xa;
        ds.xa_status = xa;
        ds.xa_checked = true;
    }
    if (state) *state = &ds;  // not written again
    return ds.xa_status;
}

// A strided [B, heads, L, d] tensor of 16-bit elements (or 1-byte codes).
struct View {
    const void *ptr;
    long long sb, sh, st;  // strides in elements
    int B, heads, L, d, elem;
    size_t span() const {  // bytes from the first element to the last
        return (size_t)((B - 1) * sb + (heads - 1) * sh + (L - 1) * st + d) * elem;
    }
};

// Strides given by the caller, or those of a contiguous tensor. Axes of one
// entry get a contiguous tensor's stride (theirs is never used).
npa_status make_view(View *v, const void *ptr, const npa_strides *s, int B, int heads, int L, int d, int elem,
                     bool output) {
    *v = View{ptr, (long long)heads * L * d, (long long)L * d, d, B, heads, L, d, elem};
    if (s) {
        if (s->batch < 0 || s->head < 0 || s->token < 0) return NPA_ERR_INVALID_ARG;
        if (B > 1) v->sb = s->batch;
        if (heads > 1) v->sh = s->head;
        if (L > 1) v->st = s->token;
    }
    const int unit = 16 / elem;
    if (v->sb % unit || v->sh % unit || v->st % unit) return NPA_ERR_MISALIGNED;
    if (L > 1 && v->st < d) return NPA_ERR_INVALID_ARG;
    // tensor-map limits (strides < 2^40 bytes), and spans that fit an address
    const long long lim = (1LL << 40) / elem;
    if (v->sb >= lim || v->sh >= lim || v->st >= lim) return NPA_ERR_UNSUPPORTED;
    if ((double)v->sb * B + (double)v->sh * heads + (double)v->st * L >= (double)(1LL << 46)) return NPA_ERR_UNSUPPORTED;
    if (output) {  // no two elements at one place
        long long st[3] = {B > 1 ? v->sb : 0, heads > 1 ? v->sh : 0, L > 1 ? v->st : 0};
        int n[3] = {B, heads, L};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (st[j] < st[i]) std::swap(st[i], st[j]), std::swap(n[i], n[j]);
        long long below = d;  // elements that the faster axes span
        for (int i = 0; i < 3; ++i) {
            if (n[i] == 1) continue;
            if (st[i] < below) return NPA_ERR_INVALID_ARG;
            below += (n[i] - 1) * st[i];
        }
    }
    return NPA_OK;
}

// 4D map {d, L, heads, B}, boxes of `rows` tokens; an axis with stride 0 becomes one entry long (the
// kernel multiplies its coordinate by 0).
bool encode_view(CUtensorMap *m, const View &v, bool f16, int rows = 128) {
    const bool codes = v.elem == 1;
    const cuuint64_t dims[4] = {(cuuint64_t)v.d, (cuuint64_t)v.L, (cuuint64_t)(v.sh ? v.heads : 1),
                                (cuuint64_t)(v.sb ? v.B : 1)};
    const cuuint64_t row = (cuuint64_t)v.d * v.elem;
    const cuuint64_t strides[3] = {(cuuint64_t)v.st * v.elem, v.sh ? (cuuint64_t)v.sh * v.elem : row,
                                   v.sb ? (cuuint64_t)v.sb * v.elem : row};
    const cuuint32_t box[4] = {codes ? (cuuint32_t)v.d : 64u, (cuuint32_t)rows, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return g_encode(m,
                    codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                    : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    4, const_cast<void *>(v.ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    codes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How xa_fwd_kernel's units are shared out: whole units in waves, and whether
// the last wave, which does not fill the GPU, is cut into pieces of the key
// range. In key blocks of one CTA, a unit costs about two beyond its own, a
// piece three, and the merge six. (Uncut / cut: 37 / 44 us for 80 units of 16
// blocks, 866 / 719 us for 384 units of 128.) Cut units are dealt out either
// evenly, where a CTA may hold the end of one unit and the beginning of the
// next, or with the same number of CTAs to every unit, one piece each.
struct XaPlan {
    int grid, waves, tail_ctas, per_unit;  // per_unit: CTAs of a cut unit, 0: dealt evenly
    long long tail_blocks, n_blk;
    int start(int cta) const {  // the first block of a CTA's share of the cut units
        if (per_unit) return (int)(cta / per_unit * n_blk + cta % per_unit * n_blk / per_unit);
        return (int)(tail_blocks * cta / tail_ctas);
    }
};

XaPlan plan_xa(long long units, long long n_blk, int sm_count, bool cut) {
    XaPlan pl;
    std::memset(&pl, 0, sizeof(pl));
    pl.n_blk = n_blk;
    pl.grid = (int)std::min<long long>(units, sm_count);
    pl.waves = (int)((units + sm_count - 1) / sm_count);
    const long long whole = units / sm_count, rest = units % sm_count, blocks = rest * n_blk;
    if (!cut || rest == 0 || blocks > (1 << 30) || sm_count > npa::kXaMaxTailCtas) return pl;
    long long ctas = std::min<long long>(sm_count, (blocks + 1) / 2);  // two blocks each at least
    const long long per_unit = std::min(sm_count / rest, n_blk / 2);
    auto share = [](long long all, long long parts) { return (all + parts - 1) / parts; };
    long long best = n_blk + 2;
    if (ctas > rest && share(blocks, ctas) + 12 < best) {
        best = share(blocks, ctas) + 12;
        pl.tail_ctas = (int)ctas;
    }
    if (per_unit > 1 && share(n_blk, per_unit) + 9 <= best) {
        pl.per_unit = (int)per_unit;
        pl.tail_ctas = (int)(per_unit * rest);
    }
    if (pl.tail_ctas == 0) return pl;
    pl.waves = (int)whole;
    pl.grid = (int)(whole ? sm_count : pl.tail_ctas);
    pl.tail_blocks = blocks;
    return pl;
}

// Key-range splits of xa_few_kernel. In steps of a warp: with the splits as a
// cluster, the longest warp's, times the waves in which the clusters run; with
// as many blocks as run at once and a merge through the workspace, the longest
// warp's and about four more. (Cluster / workspace, us, keys in L2: 12.0 / 14.9
// for 2 x 20 heads, 16 queries, 4111 keys at d = 64, where a warp has 5 or 3 steps;
// 22.5 / 19.2 for one query over 16384 cached keys, 16 or 10 steps. No third size
// was compared.) Without room for the latter in the workspace, the former.
struct XfPlan {
    int splits;
    bool cluster;
};

XfPlan plan_xf(const DeviceState &ds, long long units, int rows, int Lk, int d, bool kv8, size_t held) {
    const int tiles = rows > 8 ? 2 : 1;
    const long long step = !kv8 && d == 128 ? 16 : 32, steps = (Lk + step - 1) / step;
    auto longest = [&](long long splits) { return (steps + splits * npa::kXaFewWarps - 1) / (splits * npa::kXaFewWarps); };
    XfPlan pl{1, false};
    long long best = LLONG_MAX;
    for (int s = 1; s <= npa::kXaFewCluster; ++s) {
        const long long at_once = ds.xf_clusters[d == 128][kv8][tiles - 1][s];
        const long long cost = (units + at_once - 1) / at_once * longest(s);
        if (cost < best) {
            best = cost;
            pl = XfPlan{s, s > 1};
        }
    }
    // a split has two steps or more for every warp
    const long long fit = (long long)npa::xa_few_per_sm(d, tiles) * ds.sm_count / units, most = ((long long)Lk + 255) / 256;
    const long long want = std::min({fit, most, (long long)npa::kXaMaxSplits, (long long)std::min<size_t>(held, npa::kXaMaxSplits)});
    if (want > pl.splits && longest(want) + 4 < best) pl = XfPlan{(int)want, false};
    return pl;
}

bool xa_few_rows(int heads, int kv_heads, int Lq) {
    return (long long)(heads / kv_heads) * Lq <= npa::kXaFewRows;
}

size_t xa_split_bytes(int B, int heads, int Lq, int d) { return (size_t)B * heads * Lq * (d + 2) * sizeof(float); }
size_t xa_tail_bytes(int ctas, int d) { return (size_t)ctas * 512 * (d + 2) * sizeof(float); }

struct XaCall {
    View q, k, v, o;
    const float *k_scale, *v_scale;  // null: 16-bit keys
    int scale_blocks;
    const int *kv_lens;
    const unsigned char *key_mask;
    float scale;
    void *workspace;
    size_t workspace_bytes;
    bool f16;
};

// Sizes, scale and masks (before the views, which need the sizes).
npa_status validate_xa_sizes(int B, int heads, int kv_heads, int Lq, int Lk, int d, float scale,
                             const int32_t *kv_lens) {
    if (B < 1 || heads < 1 || kv_heads < 1 || Lq < 1 || Lk < 1 || d < 1) return NPA_ERR_INVALID_ARG;
    if (heads % kv_heads != 0 || !std::isfinite(scale) || scale < 0.f) return NPA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return NPA_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(kv_lens) & 3u) return NPA_ERR_MISALIGNED;
    const long long units = (long long)B * heads * (((long long)Lq + 255) / 256);
    if ((long long)B * heads > INT_MAX / 64 || units > INT_MAX / 128 || Lq > INT_MAX - 256 || Lk > INT_MAX - 256)
        return NPA_ERR_UNSUPPORTED;
    return NPA_OK;
}

npa_status validate_xa_buffers(const XaCall &c) {
    const int B = c.q.B, Lk = c.k.L;
    if (!aligned16(c.q.ptr) || !aligned16(c.k.ptr) || !aligned16(c.v.ptr) || !aligned16(c.o.ptr) ||
        (c.workspace && !aligned16(c.workspace)))
        return NPA_ERR_MISALIGNED;
    struct { const void *p; size_t n; } in[7] = {
        {c.q.ptr, c.q.span()}, {c.k.ptr, c.k.span()}, {c.v.ptr, c.v.span()},
        {c.kv_lens, (size_t)B * 4}, {c.key_mask, (size_t)B * Lk},
        {c.k_scale, (size_t)B * c.k.heads * c.scale_blocks * 4}, {c.v_scale, (size_t)B * c.k.heads * c.scale_blocks * 4}};
    for (const auto &x : in) {
        if (!x.p) continue;
        if (overlaps(c.o.ptr, c.o.span(), x.p, x.n)) return NPA_ERR_INVALID_ARG;
        if (c.workspace && overlaps(c.workspace, c.workspace_bytes, x.p, x.n)) return NPA_ERR_INVALID_ARG;
    }
    if (c.workspace && overlaps(c.workspace, c.workspace_bytes, c.o.ptr, c.o.span())) return NPA_ERR_INVALID_ARG;
    return NPA_OK;
}

template <int D, bool F16>
npa_status launch_xs_kernel(const XaCall &c, const npa::XaParams &a, int sm_count, npa_stream_t stream) {
    using C = npa::XsCfg<D>;
    npa::XsParams prm;
    std::memset(&prm, 0, sizeof(prm));
    prm.a = a;
    prm.kv_rows = (a.Lk + 15) / 16 * 16;
    prm.kv_stages = C::smem_bytes(prm.kv_rows, 2) <= kMaxSmem ? 2 : 1;
    prm.n_qtiles = (a.Lq + 127) / 128;
    prm.n_tiles = a.B * a.heads * prm.n_qtiles;  // at most twice the units
    prm.by_qtiles = npa::FastDiv(prm.n_qtiles);
    if (!encode_view(&prm.a.tm_k, c.k, F16, prm.kv_rows) || !encode_view(&prm.a.tm_v, c.v, F16, prm.kv_rows))
        return NPA_ERR_CUDA;
    void *args[1] = {&prm};
    const unsigned grid = (unsigned)(prm.n_tiles < sm_count ? prm.n_tiles : sm_count);
    return cudaLaunchKernel((const void *)npa::xa_short_kernel<D, F16>, dim3(grid), dim3(C::kThreads), args,
                            C::smem_bytes(prm.kv_rows, prm.kv_stages), (cudaStream_t)stream) == cudaSuccess
               ? NPA_OK
               : NPA_ERR_CUDA;
}

// The kernel that merges partial results: of cut units (tail_ctas > 0), or of
// xa_few_kernel's splits.
npa_status launch_combine(const XaCall &c, const npa::XaParams &a, npa_stream_t stream) {
    const int d = c.q.d;
    const bool tail = a.tail_ctas > 0;
    npa::XaCombineParams cp;
    std::memset(&cp, 0, sizeof(cp));
    cp.o_part = a.o_part;
    cp.ml = a.ml;
    cp.o = const_cast<void *>(c.o.ptr);
    cp.sb = c.o.sb;
    cp.sh = c.o.sh;
    cp.st = c.o.st;
    cp.n_splits = a.n_splits;
    cp.rows = a.B * a.heads * a.Lq;
    cp.heads = a.heads;
    cp.Lq = a.Lq;
    unsigned grid = (unsigned)((cp.rows + 3) / 4);
    if (tail) {
        const int cut = a.tail_start[a.tail_ctas] / a.n_blk;  // cut units
        cp.first_unit = a.n_units - cut;
        cp.n_blk = a.n_blk;
        cp.by_qpairs = a.by_qpairs;
        cp.by_heads = a.by_heads;
        cp.n_qpairs = a.n_qpairs;
        cp.kv_lens = a.sort_rows ? a.kv_lens : nullptr;
        cp.B = a.B;
        cp.Lk = a.Lk;
        cp.divided = a.k_scale != nullptr;
        std::memcpy(cp.tail_start, a.tail_start, sizeof(cp.tail_start));
        for (int t = 0, cta = 0; t < cut; ++t) {
            while (a.tail_start[cta + 1] <= t * a.n_blk) ++cta;
            cp.first_cta[t] = (short)cta;
            while (a.tail_start[cta + 1] < (t + 1) * a.n_blk) ++cta;
            cp.last_cta[t] = (short)cta;
        }
        grid = 64u * cut;
    }
    void *args[1] = {&cp};
    const void *kernels[2][2][2] = {
        {{(const void *)npa::xa_combine_kernel<64, false>, (const void *)npa::xa_combine_kernel<64, true>},
         {(const void *)npa::xa_combine_kernel<128, false>, (const void *)npa::xa_combine_kernel<128, true>}},
        {{(const void *)npa::xa_tail_kernel<64, false>, (const void *)npa::xa_tail_kernel<64, true>},
         {(const void *)npa::xa_tail_kernel<128, false>, (const void *)npa::xa_tail_kernel<128, true>}}};
    const void *kernel = kernels[tail][d == 128][c.f16];
    // it may start under the attention kernel's end, and waits there
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(128);
    cfg.stream = (cudaStream_t)stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args) == cudaSuccess ? NPA_OK : NPA_ERR_CUDA;
}

template <int D, bool KV8, bool F16>
npa_status launch_xf_kernel(const XaCall &c, const npa::XaParams &a, bool cluster, npa_stream_t stream) {
    npa::XfParams prm;
    std::memset(&prm, 0, sizeof(prm));
    prm.q = c.q.ptr;
    prm.k = c.k.ptr;
    prm.v = c.v.ptr;
    prm.o = const_cast<void *>(c.o.ptr);
    prm.qsb = c.q.sb, prm.qsh = c.q.sh, prm.qst = c.q.st;
    prm.ksb = c.k.sb, prm.ksh = c.k.sh, prm.kst = c.k.st;
    prm.vsb = c.v.sb, prm.vsh = c.v.sh, prm.vst = c.v.st;
    prm.osb = c.o.sb, prm.osh = c.o.sh, prm.ost = c.o.st;
    prm.kv_lens = a.kv_lens;
    prm.key_mask = a.key_mask;
    prm.k_scale = a.k_scale;
    prm.v_scale = a.v_scale;
    prm.scale_blocks = a.scale_blocks;
    prm.B = a.B, prm.heads = a.heads, prm.kv_heads = a.kv_heads, prm.group = a.group, prm.Lq = a.Lq, prm.Lk = a.Lk;
    prm.n_splits = a.n_splits;
    prm.cluster = cluster;
    prm.scale_log2 = a.scale_log2;
    prm.o_part = a.o_part;
    prm.ml = a.ml;
    const int tiles = a.group * a.Lq > 8 ? 2 : 1;
    const void *kernel = tiles == 2 ? (const void *)npa::xa_few_kernel<D, KV8, F16, 2>
                                    : (const void *)npa::xa_few_kernel<D, KV8, F16, 1>;
    void *args[1] = {&prm};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)a.n_splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(a.B * a.kv_heads * a.n_splits));
    cfg.blockDim = dim3(32 * npa::kXaFewWarps);
    cfg.dynamicSmemBytes = xf_smem(D, tiles);
    cfg.stream = (cudaStream_t)stream;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, kernel, args) == cudaSuccess ? NPA_OK : NPA_ERR_CUDA;
}

npa_status launch_xa(const XaCall &c, npa_stream_t stream) {
    int sm_count = 0;
    const DeviceState *ds = nullptr;
    const npa_status st = ensure_xa_ready(&sm_count, &ds);
    if (st != NPA_OK) return st;
    const int B = c.q.B, heads = c.q.heads, Lq = c.q.L, d = c.q.d, Lk = c.k.L;
    npa::XaParams prm;
    std::memset(&prm, 0, sizeof(prm));
    prm.kv_lens = c.kv_lens;
    prm.key_mask = c.key_mask;
    prm.k_scale = c.k_scale;
    prm.v_scale = c.v_scale;
    prm.scale_blocks = c.scale_blocks;
    prm.B = B;
    prm.heads = heads;
    prm.kv_heads = c.k.heads;
    prm.group = heads / c.k.heads;
    prm.Lq = Lq;
    prm.Lk = Lk;
    prm.q_b = c.q.sb != 0;
    prm.q_h = c.q.sh != 0;
    prm.k_b = c.k.sb != 0;
    prm.k_h = c.k.sh != 0;
    prm.v_b = c.v.sb != 0;
    prm.v_h = c.v.sh != 0;
    prm.n_qpairs = (Lq + 255) / 256;
    const double scale = c.scale > 0.f ? (double)c.scale : 1.0 / std::sqrt((double)d);
    // (a scale near float32's largest: finite, so that scores of 0 stay 0)
    prm.scale_log2 = (float)std::min(1.4426950408889634 * scale, (double)FLT_MAX);
    prm.wait_limit_ns = kWaitLimitNs;
    const long long units = (long long)B * heads * prm.n_qpairs;
    prm.n_units = (int)units;
    prm.by_qpairs = npa::FastDiv(prm.n_qpairs);
    prm.by_heads = npa::FastDiv(heads);
    prm.by_group = npa::FastDiv(prm.group);
    prm.o_part = static_cast<float *>(c.workspace);
    const bool kv8 = c.k_scale != nullptr;
    if (xa_few_rows(heads, c.k.heads, Lq)) {
        const size_t held = c.workspace ? c.workspace_bytes / xa_split_bytes(B, heads, Lq, d) : 0;
        const XfPlan pl = plan_xf(*ds, (long long)B * c.k.heads, prm.group * Lq, Lk, d, kv8, held);
        const bool cluster = pl.cluster;
        prm.n_splits = pl.splits;
        prm.ml = pl.splits > 1 && !cluster ? prm.o_part + (size_t)prm.n_splits * B * heads * Lq * d : nullptr;
        npa_status s;
        if (kv8)
            s = d == 64 ? launch_xf_kernel<64, true, false>(c, prm, cluster, stream)
                        : launch_xf_kernel<128, true, false>(c, prm, cluster, stream);
        else if (d == 64)
            s = c.f16 ? launch_xf_kernel<64, false, true>(c, prm, cluster, stream)
                      : launch_xf_kernel<64, false, false>(c, prm, cluster, stream);
        else
            s = c.f16 ? launch_xf_kernel<128, false, true>(c, prm, cluster, stream)
                      : launch_xf_kernel<128, false, false>(c, prm, cluster, stream);
        return s != NPA_OK || !prm.ml ? s : launch_combine(c, prm, stream);
    }
    if (!encode_view(&prm.tm_q, c.q, c.f16) || !encode_view(&prm.tm_o, c.o, c.f16)) return NPA_ERR_CUDA;
    if (!kv8 && Lk <= npa::kXaShortKeys)
        return d == 64 ? (c.f16 ? launch_xs_kernel<64, true>(c, prm, sm_count, stream)
                                : launch_xs_kernel<64, false>(c, prm, sm_count, stream))
                       : (c.f16 ? launch_xs_kernel<128, true>(c, prm, sm_count, stream)
                                : launch_xs_kernel<128, false>(c, prm, sm_count, stream));
    if (!encode_view(&prm.tm_k, c.k, c.f16) || !encode_view(&prm.tm_v, c.v, c.f16)) return NPA_ERR_CUDA;
    prm.n_blk = (Lk + 127) / 128;
    prm.by_blk = npa::FastDiv(prm.n_blk);
    XaPlan pl = plan_xa(units, prm.n_blk, sm_count, true);
    if (pl.tail_ctas && (!c.workspace || c.workspace_bytes < xa_tail_bytes(pl.tail_ctas, d)))
        pl = plan_xa(units, prm.n_blk, sm_count, false);
    prm.sort_rows = prm.kv_lens && B > 1 && B <= npa::kXaMaxSortedRows && units > sm_count &&
                    prm.n_blk >= npa::xa_min_sorted_blocks(d);
    prm.waves = pl.waves;
    prm.tail_ctas = pl.tail_ctas;
    for (int i = 0; i <= pl.tail_ctas && pl.tail_ctas; ++i)
        prm.tail_start[i] = pl.start(i);
    prm.ml = prm.o_part + (size_t)pl.tail_ctas * 512 * d;
    const void *kernel;
    unsigned threads, smem;
    auto pick = [&](const void *k, auto cfg) {
        kernel = k;
        threads = decltype(cfg)::kThreads;
        smem = decltype(cfg)::kSmemBytes;
    };
    if (kv8 && d == 64)
        pick((const void *)npa::xa_fwd_kernel<64, true, false>, npa::XaCfg<64, true>{});
    else if (kv8)
        pick((const void *)npa::xa_fwd_kernel<128, true, false>, npa::XaCfg<128, true>{});
    else if (d == 64)
        pick(c.f16 ? (const void *)npa::xa_fwd_kernel<64, false, true> : (const void *)npa::xa_fwd_kernel<64, false, false>,
             npa::XaCfg<64, false>{});
    else
        pick(c.f16 ? (const void *)npa::xa_fwd_kernel<128, false, true>
                   : (const void *)npa::xa_fwd_kernel<128, false, false>,
             npa::XaCfg<128, false>{});
    void *args[1] = {&prm};
    if (cudaLaunchKernel(kernel, dim3((unsigned)pl.grid), dim3(threads), args, smem, (cudaStream_t)stream) != cudaSuccess)
        return NPA_ERR_CUDA;
    return pl.tail_ctas ? launch_combine(c, prm, stream) : NPA_OK;
}

// A cache's own arguments.
npa_status validate_kv8(const npa_kv8_cache *cache, int B, int kv_heads, int d) {
    if (!cache || !cache->k || !cache->v || !cache->k_scale || !cache->v_scale) return NPA_ERR_INVALID_ARG;
    if (B < 1 || kv_heads < 1 || d < 1 || cache->capacity < npa::kKv8Block || cache->capacity % npa::kKv8Block != 0)
        return NPA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return NPA_ERR_UNSUPPORTED;
    if (!aligned16(cache->k) || !aligned16(cache->v) || !aligned16(cache->k_scale) || !aligned16(cache->v_scale))
        return NPA_ERR_MISALIGNED;
    if ((long long)B * kv_heads > INT_MAX / 64 || (double)B * kv_heads * cache->capacity * d >= (double)(1LL << 46))
        return NPA_ERR_UNSUPPORTED;
    return NPA_OK;
}

// ---------------------------------------------------------------------------
// Group norm
// ---------------------------------------------------------------------------
struct GnPlan {
    int vec, cols, rows, threads;
    int cw;               // channels of a chunk
    int cluster;          // > 0: gn_cluster_kernel with this many blocks (0: three launches)
    int tiles, tile_rows;
    int apply_tiles, apply_rows;
    size_t smem, bytes;   // dynamic shared memory; workspace
};

// Batches of tokens of a normalising thread.
constexpr int kGnApplyBatches = 6;
// Shared memory of a cluster block's share of its chunk at most.
constexpr size_t kGnSlabBytes = 200 * 1024;

void gn_shape(GnPlan *pl) {
    const int ncol = pl->cw / pl->vec;
    pl->cols = ncol < npa::kGnThreads ? ncol : npa::kGnThreads;
    pl->rows = npa::kGnThreads / pl->cols;
    pl->threads = (pl->cols * pl->rows + 31) / 32 * 32;
}

// Tokens cut into `tiles` tiles of whole block rows.
void gn_tiles(GnPlan *pl, int N, long long tiles) {
    long long r = (N + tiles - 1) / tiles;
    if (r < pl->rows) r = pl->rows;
    pl->tile_rows = (int)((r + pl->rows - 1) / pl->rows * pl->rows);
    pl->tiles = (int)(((long long)N + pl->tile_rows - 1) / pl->tile_rows);
}

int lcm(int a, int b) {
    int x = a, y = b;
    while (y) {
        const int t = x % y;
        x = y;
        y = t;
    }
    return a / x * b;
}

GnPlan plan_gn(int B, int N, int C, int groups, int vec, int elem, int sm_count) {
    GnPlan pl;
    std::memset(&pl, 0, sizeof(pl));
    const int cpg = C / groups;
    pl.vec = vec;
    // the narrowest chunk of whole groups and whole 32-byte sectors that
    // divides the channels, widened to 128 bytes where that divides them too
    int chunk = C;
    if (vec > 1) {
        const int unit = lcm(cpg, 32 / elem);
        for (int m = 1; (long long)unit * m <= C; ++m)
            if (C % (unit * m) == 0) {
                chunk = unit * m;
                if (chunk * elem >= 128) break;
            }
    }
    // cluster form: the least number of blocks whose shared memory holds a
    // chunk, or more while the GPU is not full (against the three launches,
    // float16: 10.8 / 14.1 us for [2, 1024, 1280], 17.3 / 19.9 for [2, 4096,
    // 640], 21.3 / 21.5 for [2, 16384, 320], the largest that fits)
    if (vec > 1 && chunk / vec <= npa::kGnThreads && C / chunk <= 65535) {
        pl.cw = chunk;
        gn_shape(&pl);
        for (int s = 1; s <= npa::kGnMaxCluster; s *= 2) {
            gn_tiles(&pl, N, s);
            const size_t ng = chunk / cpg;
            const size_t slab = (size_t)(pl.tile_rows / pl.rows) * pl.cols * pl.rows * 16;
            const size_t smem = slab + (size_t)pl.rows * (chunk + 1) * 8 + (size_t)s * ng * 8 + ng * 8;
            const bool enough = (long long)B * (C / chunk) * s >= sm_count || s == npa::kGnMaxCluster ||
                                N <= 8LL * s * pl.rows;
            if (smem > kGnSlabBytes || !enough) continue;
            pl.cluster = s;
            pl.tiles = s;  // trailing blocks may have no tokens
            pl.smem = smem;
            return pl;
        }
    }
    // three launches. Statistics: about three blocks for every multiprocessor,
    // of a batch of tokens for each thread at least; normalisation: short
    // blocks, many more than fit at once
    pl.cw = C;
    gn_shape(&pl);
    const long long batch = (long long)npa::kGnBatch * pl.rows;
    const long long want = std::min<long long>(npa::kGnMaxTiles, (3LL * sm_count + B - 1) / B);
    gn_tiles(&pl, N, std::max(1LL, std::min(want, (N + batch - 1) / batch)));
    pl.apply_rows = (int)std::min<long long>(kGnApplyBatches * batch, INT_MAX / 2);
    pl.apply_tiles = (int)(((long long)N + pl.apply_rows - 1) / pl.apply_rows);
    pl.smem = (size_t)pl.rows * (C + 1) * 8;
    pl.bytes = (size_t)B * groups * (pl.tiles + 1) * sizeof(float2);
    return pl;
}

int gn_elem(npa_dtype t) { return t == NPA_DTYPE_FP32 ? 4 : 2; }
bool gn_dtype(npa_dtype t) { return t == NPA_DTYPE_BF16 || t == NPA_DTYPE_FP16 || t == NPA_DTYPE_FP32; }

// Tokens of C channels at these strides can be read 16 bytes at a time.
bool gn_vectors(int C, npa_dtype dtype, const void *x, const void *y, const int64_t (&s)[4]) {
    const int unit = 16 / gn_elem(dtype);
    for (const int64_t t : s)
        if (t % unit) return false;
    return C % unit == 0 && aligned16(x) && aligned16(y);
}

template <typename T>
npa_status prepare_gn_kernel() {
    return prepare((const void *)npa::gn_cluster_kernel<T, 16 / sizeof(T)>, 0, (int)kGnSlabBytes);
}

// ensure_ready plus the group norm kernels' shared memory, once per device.
npa_status ensure_gn_ready(int *sm_count) {
    const npa_status st = ensure_ready(sm_count);
    if (st != NPA_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NPA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState &ds = g_dev[dev];
    if (!ds.gn_checked) {
        const npa_status gn =
            first_fault({prepare_gn_kernel<__nv_bfloat16>(), prepare_gn_kernel<__half>(), prepare_gn_kernel<float>()});
        if (gn == NPA_ERR_CUDA) return gn;
        ds.gn_status = gn;
        ds.gn_checked = true;
    }
    return ds.gn_status;
}

template <typename T, int kVec>
npa_status launch_gn(const npa::GnParams &prm, const GnPlan &pl, int B, int C, npa_stream_t stream) {
    npa::GnParams p = prm;
    void *args[1] = {&p};
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.blockDim = dim3(pl.threads);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = (cudaStream_t)stream;
    cfg.attrs = &attr;
    if (pl.cluster) {
        if constexpr (kVec > 1) {
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = pl.cluster;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.numAttrs = 1;
            cfg.gridDim = dim3(pl.cluster, C / pl.cw, B);
            return cudaLaunchKernelExC(&cfg, (const void *)npa::gn_cluster_kernel<T, kVec>, args) == cudaSuccess
                       ? NPA_OK
                       : NPA_ERR_CUDA;
        }
        return NPA_ERR_CUDA;  // not planned
    }
    cfg.gridDim = dim3(pl.tiles, B);
    if (cudaLaunchKernelExC(&cfg, (const void *)npa::gn_stats_kernel<T, kVec>, args) != cudaSuccess) return NPA_ERR_CUDA;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = 0;
    int n = B * p.G;
    void *merge_args[2] = {&p, &n};
    cfg.gridDim = dim3((n + 3) / 4);
    cfg.blockDim = dim3(128);
    if (cudaLaunchKernelExC(&cfg, (const void *)npa::gn_merge_kernel, merge_args) != cudaSuccess) return NPA_ERR_CUDA;
    cfg.gridDim = dim3(pl.apply_tiles, B);
    cfg.blockDim = dim3(pl.threads);
    return cudaLaunchKernelExC(&cfg, (const void *)npa::gn_apply_kernel<T, kVec>, args) == cudaSuccess ? NPA_OK
                                                                                                       : NPA_ERR_CUDA;
}

template <typename T>
npa_status launch_gn_vec(const npa::GnParams &prm, const GnPlan &pl, int B, int C, npa_stream_t stream) {
    return pl.vec == 1 ? launch_gn<T, 1>(prm, pl, B, C, stream) : launch_gn<T, 16 / sizeof(T)>(prm, pl, B, C, stream);
}

}  // namespace

extern "C" {

npa_status npa_attention_fwd(const void *q, const void *k, const void *v, void *o, int B, int heads, int H, int W,
                             int d, int patch, int margin, const npa_global_kv *global_kv, npa_stream_t stream) {
    int G = 0;
    npa_status st = validate_common(q, k, v, o, B, heads, H, W, d, global_kv, &G);
    if (st != NPA_OK) return st;
    if (patch < 1 || margin < 0) return NPA_ERR_INVALID_ARG;
    const Geo g{H, W, patch, patch, margin, margin};
    return launch(q, k, v, nullptr, nullptr, o, B, heads, d, g, G, global_kv, 0, -1, stream);
}

npa_status pcpp_attention_fwd(const void *q, const void *k, const void *v, void *o, int B, int heads, int H, int W,
                              int d, int n_strips, double p, const npa_global_kv *global_kv, npa_stream_t stream) {
    int G = 0;
    npa_status st = validate_common(q, k, v, o, B, heads, H, W, d, global_kv, &G);
    if (st != NPA_OK) return st;
    if (n_strips < 1 || H % n_strips != 0 || !(p >= 0.0) || !(p <= 1.0)) return NPA_ERR_INVALID_ARG;
    const int s = H / n_strips;
    const Geo g{H, W, s, W, neighbor_rows(s, p), 0};
    return launch(q, k, v, nullptr, nullptr, o, B, heads, d, g, G, global_kv, 0, -1, stream);
}

npa_status pcpp_attention_fwd_stale(const void *q, const void *k, const void *v, const void *k_stale,
                                    const void *v_stale, void *o, int B, int heads, int H, int W, int d, int n_strips,
                                    double p, int strip_begin, int strip_count, const npa_global_kv *global_kv,
                                    npa_stream_t stream) {
    int G = 0;
    npa_status st = validate_common(q, k, v, o, B, heads, H, W, d, global_kv, &G);
    if (st != NPA_OK) return st;
    if (!k_stale || !v_stale) return NPA_ERR_INVALID_ARG;
    if (!aligned16(k_stale) || !aligned16(v_stale)) return NPA_ERR_MISALIGNED;
    const size_t bytes = (size_t)B * heads * H * W * d * 2;
    if (overlaps(o, bytes, k_stale, bytes) || overlaps(o, bytes, v_stale, bytes)) return NPA_ERR_INVALID_ARG;
    if (n_strips < 1 || H % n_strips != 0 || !(p >= 0.0) || !(p <= 1.0)) return NPA_ERR_INVALID_ARG;
    if (strip_begin < 0 || strip_count < 1 || strip_begin > n_strips - strip_count) return NPA_ERR_INVALID_ARG;
    const int s = H / n_strips;
    const Geo g{H, W, s, W, neighbor_rows(s, p), 0};
    return launch(q, k, v, k_stale, v_stale, o, B, heads, d, g, G, global_kv, strip_begin, strip_count, stream);
}

size_t npa_global_query_workspace_size(int B, int heads, int H, int W, int d, int G) {
    if (B < 1 || heads < 1 || H < 1 || W < 1 || G < 1 || (d != 64 && d != 128)) return 0;
    int dev = 0, sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    const GqPlan pl = plan_gq(B, heads, H, W, d, G, sm);
    return pl.splits > 1 ? (size_t)pl.splits * pl.split_bytes : 0;
}

npa_status npa_global_query_attention_fwd(const void *gq, const void *k, const void *v, const void *gk,
                                          const void *gv, void *go, int B, int heads, int H, int W, int d, int G,
                                          void *workspace, size_t workspace_bytes, npa_stream_t stream) {
    npa_status st = validate_gq(gq, k, v, gk, gv, go, B, heads, H, W, d, G);
    if (st != NPA_OK) return st;
    if (workspace && !aligned16(workspace)) return NPA_ERR_MISALIGNED;
    int sm_count = 0;
    st = ensure_ready(&sm_count);
    if (st != NPA_OK) return st;
    const GqPlan pl = plan_gq(B, heads, H, W, d, G, sm_count);
    // as many splits as planned and as the workspace holds (one needs none)
    int splits = workspace ? (int)(workspace_bytes / pl.split_bytes) : 1;
    if (splits > pl.splits) splits = pl.splits;
    if (splits < 2) splits = 1;
    float *o_part = static_cast<float *>(workspace);
    float *ml = splits > 1 ? o_part + (size_t)splits * B * heads * G * d : nullptr;
    if (splits > 1) {
        const size_t wsz = (size_t)splits * pl.split_bytes;
        const size_t gbytes = (size_t)B * heads * G * d * 2;
        if (overlaps(workspace, wsz, go, gbytes) || overlaps(workspace, wsz, gq, gbytes)) return NPA_ERR_INVALID_ARG;
    }
    return launch_gq(gq, k, v, gk, gv, go, B, heads, H, W, d, G, o_part, ml, splits, sm_count, stream);
}

npa_status npa_global_query_attention_fwd_noalloc(const void *gq, const void *k, const void *v, const void *gk,
                                                  const void *gv, void *go, int B, int heads, int H, int W, int d,
                                                  int G, npa_stream_t stream) {
    npa_status st = validate_gq(gq, k, v, gk, gv, go, B, heads, H, W, d, G);
    if (st != NPA_OK) return st;
    // the array must hold at least two partial results (the smallest split);
    // the limit does not depend on the device, so it is checked first
    const size_t per_split = (size_t)B * heads * G * (d + 2) * sizeof(float);
    if (2 * per_split > kNoAllocScratchBytes) return NPA_ERR_UNSUPPORTED;
    int sm_count = 0;
    st = ensure_ready(&sm_count);
    if (st != NPA_OK) return st;
    const GqPlan pl = plan_gq(B, heads, H, W, d, G, sm_count);
    int splits = 1;
    if (pl.splits > 1) {
        splits = (int)(kNoAllocScratchBytes / per_split);
        if (splits > pl.splits) splits = pl.splits;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NPA_ERR_CUDA;
    void *base = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        if (!g_noalloc_addr[dev]) {
            void *ptr = nullptr;
            if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || ptr == nullptr) return NPA_ERR_CUDA;
            g_noalloc_addr[dev] = ptr;
        }
        base = g_noalloc_addr[dev];
    }
    float *o_part = splits > 1 ? static_cast<float *>(base) : nullptr;
    float *ml = splits > 1 ? o_part + (size_t)splits * B * heads * G * d : nullptr;
    return launch_gq(gq, k, v, gk, gv, go, B, heads, H, W, d, G, o_part, ml, splits, sm_count, stream);
}

size_t npa_multidiffusion_workspace_size(int B, int heads, int H, int W, int d, int patch, int margin) {
    if (B < 1 || heads < 1 || H < 1 || W < 1 || patch < 1 || margin < 0 || (d != 64 && d != 128)) return 0;
    return md_workspace_bytes(B, heads, H, W, d, patch, margin);
}

npa_status npa_multidiffusion_attention_fwd(const void *q, const void *k, const void *v, void *o, int B, int heads,
                                            int H, int W, int d, int patch, int margin,
                                            const npa_global_kv *global_kv, void *workspace,
                                            size_t workspace_bytes, npa_stream_t stream) {
    int G = 0;
    npa_status st = validate_common(q, k, v, o, B, heads, H, W, d, global_kv, &G);
    if (st != NPA_OK) return st;
    if (patch < 1 || margin < 0 || !workspace) return NPA_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return NPA_ERR_MISALIGNED;
    const long long nph = (H + patch - 1) / patch, npw = (W + patch - 1) / patch;
    if (nph > npa::kMaxMdAxis || npw > npa::kMaxMdAxis) return NPA_ERR_UNSUPPORTED;
    const size_t need = md_workspace_bytes(B, heads, H, W, d, patch, margin);
    if (workspace_bytes < need) return NPA_ERR_INVALID_ARG;
    const size_t bytes = (size_t)B * heads * H * W * d * 2, gbytes = (size_t)B * heads * G * d * 2;
    if (overlaps(workspace, need, q, bytes) || overlaps(workspace, need, k, bytes) ||
        overlaps(workspace, need, v, bytes) || overlaps(workspace, need, o, bytes))
        return NPA_ERR_INVALID_ARG;
    if (G && (overlaps(workspace, need, global_kv->k, gbytes) || overlaps(workspace, need, global_kv->v, gbytes)))
        return NPA_ERR_INVALID_ARG;
    const Geo g{H, W, patch, patch, margin, margin};
    return launch(q, k, v, nullptr, nullptr, o, B, heads, d, g, G, global_kv, 0, -1, stream,
                  static_cast<float *>(workspace));
}

double npa_multidiffusion_useful_flops(int B, int heads, int H, int W, int d, int patch, int margin, int G) {
    if (B < 1 || heads < 1 || H < 1 || W < 1 || d < 1 || patch < 1 || margin < 0 || G < 0) return -1.0;
    double s1r = 0, s2r = 0, s1c = 0, s2c = 0;
    for (int i = 0; i < (H + patch - 1) / patch; ++i) {
        const double w = std::min(H, (i + 1) * patch + margin) - std::max(0, i * patch - margin);
        s1r += w;
        s2r += w * w;
    }
    for (int j = 0; j < (W + patch - 1) / patch; ++j) {
        const double w = std::min(W, (j + 1) * patch + margin) - std::max(0, j * patch - margin);
        s1c += w;
        s2c += w * w;
    }
    return 4.0 * d * (double)B * heads * (s2r * s2c + G * s1r * s1c);
}

npa_status asg_guidance_combine(const void *eps, const void *eps_ref, const void *mask, void *out, int n_patches,
                                int B, int C, int S, float w_t, npa_stream_t stream) {
    if (!eps || !eps_ref || !mask || !out) return NPA_ERR_INVALID_ARG;
    if (n_patches < 1 || B < 1 || C < 1 || S < 1 || !std::isfinite(w_t)) return NPA_ERR_INVALID_ARG;
    if (!aligned16(eps) || !aligned16(eps_ref) || !aligned16(mask) || !aligned16(out)) return NPA_ERR_MISALIGNED;
    const long long nb = (long long)n_patches * B;
    if (nb * C > (1LL << 40) / S || nb > INT_MAX) return NPA_ERR_UNSUPPORTED;
    const size_t e_bytes = (size_t)nb * C * S * 2, r_bytes = (size_t)B * C * S * 2, m_bytes = (size_t)nb * S * 2;
    if (out != eps && overlaps(out, e_bytes, eps, e_bytes)) return NPA_ERR_INVALID_ARG;
    if (overlaps(out, e_bytes, eps_ref, r_bytes) || overlaps(out, e_bytes, mask, m_bytes)) return NPA_ERR_INVALID_ARG;
    int sm_count = 0;
    const npa_status st = ensure_ready(&sm_count);
    if (st != NPA_OK) return st;
    npa::AsgParams prm;
    prm.eps = static_cast<const __nv_bfloat16 *>(eps);
    prm.ref = static_cast<const __nv_bfloat16 *>(eps_ref);
    prm.mask = static_cast<const __nv_bfloat16 *>(mask);
    prm.out = static_cast<__nv_bfloat16 *>(out);
    prm.B = B;
    prm.C = C;
    prm.S = S;
    prm.chunks = (S + 7) / 8;
    prm.n_items = nb * prm.chunks;
    prm.w = w_t;
    prm.vec = S % 8 == 0;
    // enough blocks for every chunk, at most 8 resident 256-thread blocks per
    // multiprocessor (the kernel strides over the rest)
    const long long blocks = (prm.n_items + 255) / 256;
    const unsigned grid = (unsigned)(blocks < 8LL * sm_count ? blocks : 8LL * sm_count);
    void *args[1] = {&prm};
    const cudaError_t e =
        cudaLaunchKernel((const void *)npa::asg_combine_kernel, dim3(grid), dim3(256), args, 0, (cudaStream_t)stream);
    return e == cudaSuccess ? NPA_OK : NPA_ERR_CUDA;
}

npa_status npa_device_ready(void) {
    int sm = 0;
    const npa_status st = ensure_xa_ready(&sm);
    return st != NPA_OK ? st : ensure_gn_ready(&sm);
}

size_t npa_cross_attention_workspace_size(int B, int heads, int kv_heads, int Lq, int Lk, int d) {
    if (validate_xa_sizes(B, heads, kv_heads, Lq, Lk, d, 0.f, nullptr) != NPA_OK) return 0;
    int sm = 0;
    const DeviceState *ds = nullptr;
    if (ensure_xa_ready(&sm, &ds) != NPA_OK) return 0;
    if (xa_few_rows(heads, kv_heads, Lq)) {
        int splits = 0;  // of 16-bit keys or the cache, whichever has more
        for (const bool kv8 : {false, true}) {
            const XfPlan pl = plan_xf(*ds, (long long)B * kv_heads, heads / kv_heads * Lq, Lk, d, kv8, SIZE_MAX);
            if (!pl.cluster && pl.splits > splits) splits = pl.splits;
        }
        return splits > 1 ? (size_t)splits * xa_split_bytes(B, heads, Lq, d) : 0;
    }
    const XaPlan pl = plan_xa((long long)B * heads * ((Lq + 255) / 256), ((long long)Lk + 127) / 128, sm, true);
    return xa_tail_bytes(pl.tail_ctas, d);
}

npa_status npa_cross_attention_fwd(const void *q, const void *k, const void *v, void *o, npa_dtype dtype, int B,
                                   int heads, int kv_heads, int Lq, int Lk, int d, const npa_strides *q_strides,
                                   const npa_strides *k_strides, const npa_strides *v_strides,
                                   const npa_strides *o_strides, const int32_t *kv_lens, const uint8_t *key_mask,
                                   float scale, void *workspace, size_t workspace_bytes, npa_stream_t stream) {
    if (!q || !k || !v || !o) return NPA_ERR_INVALID_ARG;
    npa_status st = validate_xa_sizes(B, heads, kv_heads, Lq, Lk, d, scale, kv_lens);
    if (st != NPA_OK) return st;
    if (dtype != NPA_DTYPE_BF16 && dtype != NPA_DTYPE_FP16) return NPA_ERR_UNSUPPORTED;
    XaCall c;
    std::memset(&c, 0, sizeof(c));
    if ((st = make_view(&c.q, q, q_strides, B, heads, Lq, d, 2, false)) != NPA_OK ||
        (st = make_view(&c.k, k, k_strides, B, kv_heads, Lk, d, 2, false)) != NPA_OK ||
        (st = make_view(&c.v, v, v_strides, B, kv_heads, Lk, d, 2, false)) != NPA_OK ||
        (st = make_view(&c.o, o, o_strides, B, heads, Lq, d, 2, true)) != NPA_OK)
        return st;
    c.kv_lens = kv_lens;
    c.key_mask = key_mask;
    c.scale = scale;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    c.f16 = dtype == NPA_DTYPE_FP16;
    if ((st = validate_xa_buffers(c)) != NPA_OK) return st;
    return launch_xa(c, stream);
}

npa_status npa_kv8_cross_attention_fwd(const void *q, const npa_kv8_cache *cache, void *o, int B, int heads,
                                       int kv_heads, int Lq, int Lk, int d, const npa_strides *q_strides,
                                       const npa_strides *o_strides, const int32_t *kv_lens, const uint8_t *key_mask,
                                       float scale, void *workspace, size_t workspace_bytes, npa_stream_t stream) {
    if (!q || !o) return NPA_ERR_INVALID_ARG;
    npa_status st = validate_xa_sizes(B, heads, kv_heads, Lq, Lk, d, scale, kv_lens);
    if (st != NPA_OK) return st;
    if ((st = validate_kv8(cache, B, kv_heads, d)) != NPA_OK) return st;
    if (Lk > cache->capacity) return NPA_ERR_INVALID_ARG;
    XaCall c;
    std::memset(&c, 0, sizeof(c));
    npa_strides cs;
    cs.token = d;
    cs.head = (int64_t)cache->capacity * d;
    cs.batch = cs.head * kv_heads;
    if ((st = make_view(&c.q, q, q_strides, B, heads, Lq, d, 2, false)) != NPA_OK ||
        (st = make_view(&c.k, cache->k, &cs, B, kv_heads, Lk, d, 1, false)) != NPA_OK ||
        (st = make_view(&c.v, cache->v, &cs, B, kv_heads, Lk, d, 1, false)) != NPA_OK ||
        (st = make_view(&c.o, o, o_strides, B, heads, Lq, d, 2, true)) != NPA_OK)
        return st;
    c.k_scale = cache->k_scale;
    c.v_scale = cache->v_scale;
    c.scale_blocks = cache->capacity / npa::kKv8Block;
    c.kv_lens = kv_lens;
    c.key_mask = key_mask;
    c.scale = scale;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    if ((st = validate_xa_buffers(c)) != NPA_OK) return st;
    return launch_xa(c, stream);
}

npa_status npa_kv8_store(const void *k, const void *v, const npa_kv8_cache *cache, npa_dtype dtype, int B,
                         int kv_heads, int d, int start, const int32_t *starts, int n_tokens,
                         const npa_strides *k_strides, const npa_strides *v_strides, npa_stream_t stream) {
    if (!k || !v) return NPA_ERR_INVALID_ARG;
    npa_status st = validate_kv8(cache, B, kv_heads, d);
    if (st != NPA_OK) return st;
    if (n_tokens < 1 || (!starts && (start < 0 || (long long)start + n_tokens > cache->capacity)))
        return NPA_ERR_INVALID_ARG;
    if (dtype != NPA_DTYPE_BF16 && dtype != NPA_DTYPE_FP16) return NPA_ERR_UNSUPPORTED;
    View kv[2];
    if ((st = make_view(&kv[0], k, k_strides, B, kv_heads, n_tokens, d, 2, false)) != NPA_OK ||
        (st = make_view(&kv[1], v, v_strides, B, kv_heads, n_tokens, d, 2, false)) != NPA_OK)
        return st;
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(starts) & 3u)) return NPA_ERR_MISALIGNED;
    // the four arrays of the cache and the inputs do not share memory
    const size_t codes = (size_t)B * kv_heads * cache->capacity * d;
    const size_t scales = (size_t)B * kv_heads * (cache->capacity / npa::kKv8Block) * 4;
    struct { const void *p; size_t n; } a[7] = {{cache->k, codes}, {cache->v, codes}, {cache->k_scale, scales},
        {cache->v_scale, scales}, {k, kv[0].span()}, {v, kv[1].span()}, {starts, (size_t)B * 4}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 7; ++j)
            if (a[j].p && overlaps(a[i].p, a[i].n, a[j].p, a[j].n)) return NPA_ERR_INVALID_ARG;
    npa::Kv8StoreParams prm;
    std::memset(&prm, 0, sizeof(prm));
    for (int t = 0; t < 2; ++t) {
        prm.x[t] = kv[t].ptr;
        prm.sb[t] = kv[t].sb;
        prm.sh[t] = kv[t].sh;
        prm.st[t] = kv[t].st;
    }
    prm.codes[0] = static_cast<unsigned char *>(cache->k);
    prm.codes[1] = static_cast<unsigned char *>(cache->v);
    prm.scale[0] = cache->k_scale;
    prm.scale[1] = cache->v_scale;
    prm.starts = starts;
    prm.start = start;
    prm.n = n_tokens;
    prm.capacity = cache->capacity;
    prm.heads = kv_heads;
    prm.rows = B * kv_heads;
    // blocks touched: counted from the first one's start, or, with starts on
    // the device, one more than the tokens alone need
    const long long span = starts ? (long long)n_tokens + npa::kKv8Block - 1 : start % npa::kKv8Block + (long long)n_tokens;
    const long long nb = std::min<long long>((span + npa::kKv8Block - 1) / npa::kKv8Block, cache->capacity / npa::kKv8Block);
    prm.n_blocks = (int)nb;
    const long long grid = 2 * nb * B * kv_heads;
    if (grid > INT_MAX) return NPA_ERR_UNSUPPORTED;
    st = ensure_ready();
    if (st != NPA_OK) return st;
    const bool f16 = dtype == NPA_DTYPE_FP16;
    const void *kernel = d == 64 ? (f16 ? (const void *)npa::kv8_store_kernel<64, true>
                                        : (const void *)npa::kv8_store_kernel<64, false>)
                                 : (f16 ? (const void *)npa::kv8_store_kernel<128, true>
                                        : (const void *)npa::kv8_store_kernel<128, false>);
    void *args[1] = {&prm};
    return cudaLaunchKernel(kernel, dim3((unsigned)grid), dim3(128), args, 0, (cudaStream_t)stream) == cudaSuccess
               ? NPA_OK
               : NPA_ERR_CUDA;
}

size_t npa_group_norm_workspace_size(npa_dtype dtype, int B, int N, int C, int groups) {
    if (!gn_dtype(dtype) || B < 1 || N < 1 || C < 1 || groups < 1 || C % groups || C > npa::kGnMaxChannels) return 0;
    int dev = 0, sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    // whichever of the vector and the single-element form needs more
    const int unit = 16 / gn_elem(dtype);
    size_t n = plan_gn(B, N, C, groups, 1, gn_elem(dtype), sm).bytes;
    if (C % unit == 0) n = std::max(n, plan_gn(B, N, C, groups, unit, gn_elem(dtype), sm).bytes);
    return n;
}

npa_status npa_group_norm_act(const void *x, const void *weight, const void *bias, void *y, npa_dtype dtype,
                              npa_dtype weight_dtype, int B, int N, int C, int groups, int64_t x_batch_stride,
                              int64_t x_token_stride, int64_t y_batch_stride, int64_t y_token_stride, float eps,
                              npa_activation act, void *workspace, size_t workspace_bytes, npa_stream_t stream) {
    if (!x || !y) return NPA_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || C < 1 || groups < 1 || C % groups != 0 || !std::isfinite(eps) || eps < 0.f)
        return NPA_ERR_INVALID_ARG;
    if (act != NPA_ACT_NONE && act != NPA_ACT_SILU) return NPA_ERR_INVALID_ARG;
    if (!gn_dtype(dtype) || ((weight || bias) && weight_dtype != dtype && weight_dtype != NPA_DTYPE_FP32))
        return NPA_ERR_UNSUPPORTED;
    if (C > npa::kGnMaxChannels || B > 65535 || N > INT_MAX / 2) return NPA_ERR_UNSUPPORTED;
    int64_t s[4] = {x_batch_stride, x_token_stride, y_batch_stride, y_token_stride};
    for (const int64_t t : s)
        if (t < 0 || t >= (1LL << 40)) return t < 0 ? NPA_ERR_INVALID_ARG : NPA_ERR_UNSUPPORTED;
    // axes of one entry: their stride is never used
    if (N == 1) s[1] = s[3] = C;
    if (B == 1) s[0] = (int64_t)N * s[1], s[2] = (int64_t)N * s[3];
    if (s[1] < C || s[3] < C) return NPA_ERR_INVALID_ARG;
    if (B > 1 && N > 1 && s[2] < (N - 1) * s[3] + C && s[3] < (B - 1) * s[2] + C) return NPA_ERR_INVALID_ARG;
    if (B > 1 && s[2] < C) return NPA_ERR_INVALID_ARG;
    const int elem = gn_elem(dtype), welem = gn_elem(weight_dtype);
    if ((reinterpret_cast<uintptr_t>(x) % elem) || (reinterpret_cast<uintptr_t>(y) % elem) || !aligned16(workspace) ||
        (weight && reinterpret_cast<uintptr_t>(weight) % welem) || (bias && reinterpret_cast<uintptr_t>(bias) % welem))
        return NPA_ERR_MISALIGNED;
    const double ext = (double)B * std::max(s[0], s[2]) + (double)N * std::max(s[1], s[3]);
    if (ext * elem >= (double)(1LL << 46)) return NPA_ERR_UNSUPPORTED;
    const size_t xb = (size_t)((B - 1) * s[0] + (N - 1) * s[1] + C) * elem;
    const size_t yb = (size_t)((B - 1) * s[2] + (N - 1) * s[3] + C) * elem;
    // in place, or apart
    const bool same = x == y && s[0] == s[2] && s[1] == s[3];
    if (!same && overlaps(x, xb, y, yb)) return NPA_ERR_INVALID_ARG;
    const size_t wb = (size_t)C * welem;
    if ((weight && overlaps(y, yb, weight, wb)) || (bias && overlaps(y, yb, bias, wb))) return NPA_ERR_INVALID_ARG;
    int sm_count = 0;
    const npa_status st = ensure_gn_ready(&sm_count);
    if (st != NPA_OK) return st;
    const GnPlan pl = plan_gn(B, N, C, groups, gn_vectors(C, dtype, x, y, s) ? 16 / elem : 1, elem, sm_count);
    if (workspace_bytes < pl.bytes) return NPA_ERR_INVALID_ARG;
    if (pl.bytes && !workspace) return NPA_ERR_INVALID_ARG;
    if (overlaps(workspace, pl.bytes, x, xb) || overlaps(workspace, pl.bytes, y, yb) ||
        (weight && overlaps(workspace, pl.bytes, weight, wb)) || (bias && overlaps(workspace, pl.bytes, bias, wb)))
        return NPA_ERR_INVALID_ARG;
    npa::GnParams prm;
    std::memset(&prm, 0, sizeof(prm));
    prm.x = x;
    prm.y = y;
    prm.w = weight;
    prm.bias = bias;
    prm.w_f32 = weight_dtype == NPA_DTYPE_FP32;
    prm.xsb = s[0];
    prm.xst = s[1];
    prm.ysb = s[2];
    prm.yst = s[3];
    prm.N = N;
    prm.G = groups;
    prm.cpg = C / groups;
    prm.cw = pl.cw;
    prm.cols = pl.cols;
    prm.rows = pl.rows;
    prm.by_cols = npa::SmallDiv(pl.cols);
    prm.by_cpg = npa::SmallDiv(C / groups);
    prm.tiles = pl.tiles;
    prm.tile_rows = pl.tile_rows;
    prm.eps = eps;
    prm.silu = act == NPA_ACT_SILU;
    prm.apply_tiles = pl.apply_tiles;
    prm.apply_rows = pl.apply_rows;
    prm.part = static_cast<float2 *>(workspace);
    prm.mean_rstd = prm.part + (size_t)B * groups * pl.tiles;
    if (dtype == NPA_DTYPE_BF16) return launch_gn_vec<__nv_bfloat16>(prm, pl, B, C, stream);
    if (dtype == NPA_DTYPE_FP16) return launch_gn_vec<__half>(prm, pl, B, C, stream);
    return launch_gn_vec<float>(prm, pl, B, C, stream);
}

int pcpp_neighbor_rows(int strip_rows, double p) { return neighbor_rows(strip_rows, p); }

double npa_useful_flops(int B, int heads, int H, int W, int d, int patch, int margin, int G) {
    if (B < 1 || heads < 1 || H < 1 || W < 1 || d < 1 || patch < 1 || margin < 0 || G < 0) return -1.0;
    return useful_flops(B, heads, d, Geo{H, W, patch, patch, margin, margin}, G);
}

double pcpp_useful_flops(int B, int heads, int H, int W, int d, int n_strips, double p, int G) {
    if (B < 1 || heads < 1 || H < 1 || W < 1 || d < 1 || n_strips < 1 || H % n_strips != 0 || G < 0) return -1.0;
    const int s = H / n_strips;
    const int r = neighbor_rows(s, p);
    if (r < 0) return -1.0;
    return useful_flops(B, heads, d, Geo{H, W, s, W, r, 0}, G);
}

npa_status npa_device_status(npa_stream_t stream) {
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return NPA_ERR_CUDA;
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, npa::g_npa_status, sizeof(v)) != cudaSuccess) return NPA_ERR_CUDA;
    if (v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(npa::g_npa_status, &zero, sizeof(zero)) != cudaSuccess) return NPA_ERR_CUDA;
    }
    return (npa_status)v;
}

npa_status npa_selftest_wait_timeout(uint32_t limit_us, npa_stream_t stream) {
    if (limit_us < 1 || limit_us > 1000000) return NPA_ERR_INVALID_ARG;
    npa_status st = ensure_ready();
    if (st != NPA_OK) return st;
    unsigned long long ns = (unsigned long long)limit_us * 1000ull;
    void *args[1] = {&ns};
    cudaError_t e = cudaLaunchKernel((const void *)npa::npa_wait_selftest_kernel, dim3(1), dim3(32), args, 0,
                                     (cudaStream_t)stream);
    return e == cudaSuccess ? NPA_OK : NPA_ERR_CUDA;
}

#ifdef NPA_DEBUG_BOUNDS
npa_status npa_debug_withhold_arrival_once(uint32_t wait_limit_us) {
    if (wait_limit_us < 1 || wait_limit_us > 1000000) return NPA_ERR_INVALID_ARG;
    g_debug_stall_us.store(wait_limit_us);
    return NPA_OK;
}
#endif

const char *npa_status_string(npa_status status) {
    switch (status) {
        case NPA_OK: return "NPA_OK";
        case NPA_ERR_INVALID_ARG: return "NPA_ERR_INVALID_ARG";
        case NPA_ERR_UNSUPPORTED: return "NPA_ERR_UNSUPPORTED";
        case NPA_ERR_MISALIGNED: return "NPA_ERR_MISALIGNED";
        case NPA_ERR_CUDA: return "NPA_ERR_CUDA";
        case NPA_ERR_DEVICE_TIMEOUT: return "NPA_ERR_DEVICE_TIMEOUT";
        case NPA_ERR_DEVICE_BOUNDS: return "NPA_ERR_DEVICE_BOUNDS";
    }
    return "NPA_ERR_UNKNOWN";
}

}  // extern "C"
