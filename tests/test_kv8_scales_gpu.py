"""Value scales of the 8-bit cache that say little about what their blocks
contribute: blocks of zeros, scales that stem from tokens that are not kept or
that have grown, blocks far apart. The bound knows each row's own probabilities
and kept values, so that what a small block loses cannot hide under a large one."""
import numpy as np
import pytest

from _block import HALF_STEP, HALF_SUB, f64, randn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def npa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from patch_res_diffusion_b200 import build
    build.build()
    import patch_res_diffusion_b200 as m
    assert m.npa_device_status() == m.NPA_OK
    yield m
    assert m.npa_device_status() == m.NPA_OK


def attend_and_check(npa, q, cache, n, keep=None, what="", **kw):
    """Per element: P is f16 (half a step of each p |v|), scores, exponentials
    and sums float32 (2^-12 of sum p |v|), the output bf16. Under f16's normal
    range a key loses at most half of 2^-24 at its block's reference. The
    largest p of some 64 tokens is at least 2^7 there and a block's largest kept
    code 2^7 at least, while a code is 448 at most: 2^-25 2^-7 448 / 2^7 < 2^-30
    of the largest product of a block's largest p and its largest kept |v|."""
    mask = None if keep is None else torch.from_numpy(keep).cuda()
    out = npa.kv8_cross_attention(q, cache, n, key_mask=mask, **kw)
    torch.cuda.synchronize()
    assert npa.npa_device_status() == npa.NPA_OK
    k, v = ((c.cpu().to(torch.float64).numpy() * np.repeat(f64(s), 64, axis=2)[..., None])[:, :, :n]
            for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    got, q = f64(out), f64(q)
    B, heads, Lq, d = q.shape
    per = heads // k.shape[1]
    for b in range(B):
        pick = np.arange(n) if keep is None else np.flatnonzero(keep[b])
        if pick.size == 0:
            assert not got[b].any()
            continue
        starts = np.flatnonzero(np.r_[True, np.diff(pick // 64) > 0])
        for h in range(heads):
            kk, vv = k[b, h // per, pick], v[b, h // per, pick]
            z = q[b, h] @ kk.T / np.sqrt(d)
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            ref, mag = p @ vv, p @ np.abs(vv)
            tops = np.maximum.reduceat(p, starts, axis=1) * np.maximum.reduceat(np.abs(vv).max(1), starts)
            bound = ((HALF_STEP["fp16"] + 2.0 ** -12) * mag + HALF_STEP["bf16"] * np.abs(ref) + HALF_SUB["bf16"] +
                     pick.size * 2.0 ** -30 * tops.max(1, keepdims=True))
            over = np.abs(got[b, h] - ref) / bound
            assert np.isfinite(got[b, h]).all() and over.max() <= 1, (what, b, h, float(over.max()))
    return out


def stored(npa, k, v, capacity=None):
    B, h, n, d = k.shape
    cache = npa.Kv8Cache.empty(B, h, capacity or n, d)
    npa.kv8_store(cache, k, v)
    return cache


def times(x, size):
    return (x.double() * size).bfloat16()


def per_block(*sizes):
    return torch.tensor(sizes, dtype=torch.float64, device="cuda").repeat_interleave(64)[:, None]


# (Lq, n, split): whole units, one and two tiles; cut units with pieces of two blocks
MANY = [(17, 384, False), (150, 384, False), (150, 1536, True), (300, 1500, True)]


def zero_blocks(npa, Lq, n, split, d):
    q, k, v = randn(1, 2, 4, Lq, d), randn(2, 2, 2, n, d), randn(3, 2, 2, n, d)
    nb = -(-n // 64)
    for small in (1e-3, 1e-5, 1e-6, 1e-7, 1e-8, 1e-20, 1e-36):
        for zeros in ((0,), (1, 2), (nb - 1,), tuple(range(0, nb, 2)), tuple(range(1, nb, 2))):
            x = times(v, small)
            for i in zeros:
                x[:, :, 64 * i:64 * i + 64] = 0
            attend_and_check(npa, q, stored(npa, k, x), n, split=split, what=(small, zeros))
    out = attend_and_check(npa, q, stored(npa, k, torch.zeros_like(v)), n, split=split, what="zeros alone")
    assert not out.any()


def unkept_sizes(npa, Lq, n, split, d):
    q, k, v = randn(4, 2, 4, Lq, d), randn(5, 2, 2, n, d), randn(6, 2, 2, n, d)
    keep = np.ones((2, n), dtype=bool)
    for j, size in ((5, 2.0 ** 7), (64 + 63, 2.0 ** 12), (200, 2.0 ** 30), (n - 1, 2.0 ** 100)):
        keep[:, j] = False
        v[:, :, j] = size
    keep[1, 70:130] = False
    # a code's own rounding at such a scale may leave 0: the cache's values are what counts
    attend_and_check(npa, q, stored(npa, k, v), n, keep, split=split)
    attend_and_check(npa, q, stored(npa, k, times(v, 2.0 ** -20)), n, keep, split=split)


def grown_scales(npa, Lq, n, split, d):
    q, k, v = randn(7, 2, 2, Lq, d), randn(8, 2, 2, n, d), times(randn(9, 2, 2, n, d), 2.0 ** -12)
    cache = stored(npa, k, v)
    keep = np.ones((2, n), dtype=bool)
    for j, size in ((40, 1.0), (64 + 50, 2.0 ** 5), (128 + 3, 2.0 ** 9), (n - 2, 2.0 ** 60)):
        npa.kv8_store(cache, k[:, :, j:j + 1], torch.full_like(v[:, :, j:j + 1], size), start=j)
        keep[:, j] = False
    attend_and_check(npa, q, cache, n, keep, split=split)


def far_apart(npa, Lq, n, split, d):
    """A block's values may be as large as its probabilities are small."""
    q, k, v = randn(10, 1, 2, Lq, d), randn(11, 1, 2, n, d), randn(12, 1, 2, n, d)
    nb = -(-n // 64)
    q[..., 0] = 8.0 * d ** 0.5
    for step in (4.0, 24.0, 40.0):
        # the first coordinate lowers block i's scores by i step (base 2); its values rise by as much
        k[..., 0] = -torch.arange(n, device="cuda").div(64, rounding_mode="floor").clamp(max=3) * step / 8.0 * 0.6931
        grow = per_block(*[2.0 ** (step * min(i, 3)) for i in range(nb)])[:n]
        for all_by in (1.0, 2.0 ** -100):
            attend_and_check(npa, q, stored(npa, k, times(v, grow * all_by)), n, split=split, what=(step, all_by))
            fall = times(v, all_by / grow * 2.0 ** 60)
            attend_and_check(npa, q, stored(npa, k, fall), n, split=split, what=(step, all_by, "falling"))


def scales_of_others(npa, Lq, n, split, d):
    """Scales written elsewhere: any positive finite numbers, with any codes."""
    q, k, v = randn(13, 1, 2, Lq, d), randn(14, 1, 2, n, d), randn(15, 1, 2, n, d)
    cache = stored(npa, k, v)
    for s in (2.0 ** -133, 1.3 * 2.0 ** -120, 0.3, 1.9 * 2.0 ** 118):
        scale = torch.full(cache.v_scale.shape, s)
        scale[:, :, ::3] *= 0.77
        cache.v_scale.copy_(scale)
        attend_and_check(npa, q, cache, n, split=split, what=s)
    cache.v_scale.fill_(2.0 ** 127)      # with codes of at most 1/2, and 2^-9 alone in a block
    cache.v.copy_((cache.v.float() / 1024).to(torch.float8_e4m3fn))
    cache.v.view(torch.uint8)[:, :, 64:128] = 1
    attend_and_check(npa, q, cache, n, split=split, what="largest")


def zeros_take_the_weight(npa, Lq, n, split, d):
    """Nearly all of the probability on values of 0; what is left still counts."""
    q, k, v = randn(16, 1, 2, Lq, d), randn(17, 1, 2, n, d), randn(18, 1, 2, n, d)
    q[..., 0] = 8.0 * d ** 0.5
    for zeros in (0, -(-n // 64) - 1):
        x = v.clone()
        x[:, :, 64 * zeros:64 * zeros + 64] = 0
        for gap in (20.0, 50.0, 70.0, 95.0):
            k[..., 0] = 0
            k[:, :, 64 * zeros:64 * zeros + 64, 0] = gap / 8.0 * 0.6931
            attend_and_check(npa, q, stored(npa, k, x), n, split=split, what=(zeros, gap))


CASES = [zero_blocks, unkept_sizes, grown_scales, far_apart, scales_of_others, zeros_take_the_weight]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,n,split", MANY)
@pytest.mark.parametrize("case", CASES)
def test_many_rows(npa, case, Lq, n, split, d):
    case(npa, Lq, n, split, d)


# at most 16 rows: whole, split in a cluster, split through the workspace
FEW = [(1, 384, True), (8, 1536, True), (3, 12000, True), (2, 333, False)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,n,split", FEW)
@pytest.mark.parametrize("case", CASES)
def test_few_rows(npa, case, Lq, n, split, d):
    case(npa, Lq, n, split, d)


def test_checked_build(npa):
    npa.use_bounds_checking(True)
    try:
        for d in (64, 128):
            zero_blocks(npa, 150, 1536, True, d)
            unkept_sizes(npa, 40, 200 + 64, False, d)
    finally:
        npa.use_bounds_checking(False)
