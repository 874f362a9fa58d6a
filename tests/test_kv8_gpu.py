"""The 8-bit key/value cache on the GPU: what npa_kv8_store writes equals the
float64 oracle exactly, and npa_kv8_cross_attention_fwd agrees with the oracle
over the values the cache holds."""
import numpy as np
import pytest

import oracle
from _block import bits, check_attention, f64, randn

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


def codes64(t):
    return t.cpu().to(torch.float64).numpy()


def store_and_check(npa, cache, k, v, start=0, starts=None):
    """Stores, and holds codes and scales of the whole cache to the oracle's."""
    want = [(codes64(c).copy(), f64(s).copy()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    sv = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    npa.kv8_store(cache, k, v, start=start, starts=sv)
    torch.cuda.synchronize()
    for (c, s), x, gc, gs in zip(want, (k, v), (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        x = f64(x)
        for b in range(x.shape[0]):
            oracle.kv8_store(c[b], s[b], x[b], start if starts is None else starts[b])
        np.testing.assert_array_equal(f64(gs), s)
        np.testing.assert_array_equal(codes64(gc), c)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("start,n", [(0, 1), (0, 64), (0, 200), (64, 65), (5, 1), (5, 59), (5, 60), (63, 1), (63, 2),
                                     (100, 156), (255, 1)])
def test_store(npa, dtype, d, start, n):
    cache = npa.Kv8Cache.empty(2, 3, 256, d)
    store_and_check(npa, cache, randn(1, 2, 3, 256, d, dtype=dtype), randn(2, 2, 3, 256, d, dtype=dtype))
    k, v = randn(3, 2, 3, n, d, dtype=dtype, sd=3.0), randn(4, 2, 3, n, d, dtype=dtype, sd=0.1)
    store_and_check(npa, cache, k, v, start)


def test_store_token_by_token(npa):
    """Appending one token at a time with growing magnitudes: every growth of a
    scale rounds the block's earlier codes again."""
    cache = npa.Kv8Cache.empty(1, 2, 128, 64)
    for t in range(100):
        k, v = randn(10 + t, 1, 2, 1, 64, sd=1.04 ** t), randn(300 + t, 1, 2, 1, 64, sd=1.1 ** -t)
        store_and_check(npa, cache, k, v, t)


def test_store_rows_at_their_own_positions(npa):
    cache = npa.Kv8Cache.empty(6, 2, 192, 64)
    store_and_check(npa, cache, randn(20, 6, 2, 192, 64), randn(21, 6, 2, 192, 64))
    for n in (1, 3, 64, 70):
        k, v = randn(22 + n, 6, 2, n, 64, sd=2.0), randn(23 + n, 6, 2, n, 64, sd=2.0)
        store_and_check(npa, cache, k, v, starts=[0, 63, 64, 191, 130, 7])
    # outside the cache: nothing written there
    k, v = randn(50, 6, 2, 10, 64), randn(51, 6, 2, 10, 64)
    store_and_check(npa, cache, k, v, starts=[-20, -3, 192, 100000, 187, -10])


def test_store_values(npa):
    """Zeros, powers of two at the border of a scale, subnormals, the largest
    numbers, infinities and NaN."""
    cache = npa.Kv8Cache.empty(1, 1, 64 * 9, 64)
    x = torch.zeros(1, 1, 64 * 9, 64, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(0)
    r = lambda: torch.randn(64, 64, generator=g)
    x[0, 0, 64:128] = (r().sign() * 448)                          # exactly 448: scale 1
    x[0, 0, 128:192] = (r().sign() * 450)                         # the next bf16 number: scale 2
    x[0, 0, 192:256] = r() * 1e-39                                # bf16 subnormals: the least scale
    x[0, 0, 256:320] = r() * 1e38
    x[0, 0, 320:384] = r()
    x[0, 0, 320, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    x[0, 0, 384:448] = torch.linspace(-1, 1, 64 * 64).reshape(64, 64) ** 9
    x[0, 0, 448, 0] = 2.0 ** -100
    x[0, 0, 512:576] = float("nan")
    store_and_check(npa, cache, x.cuda(), (-x).cuda())
    assert float(cache.k_scale[0, 0, 0]) == 1 and float(cache.k_scale[0, 0, 1]) == 1
    assert float(cache.k_scale[0, 0, 2]) == 2 and float(cache.k_scale[0, 0, 3]) == 2.0 ** -126
    y = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16).cuda()     # a zero token keeps the block's scale
    store_and_check(npa, cache, y, y, 448 + 5)
    assert float(cache.k_scale[0, 0, 7]) == 2.0 ** -108


def test_store_strides_and_neighbours(npa):
    """Projection layouts in; codes outside the written tokens stay bit for bit."""
    B, h, n, d = 2, 3, 90, 64
    kv = randn(30, B, n, 2, h, d)
    k, v = (kv[:, :, i].transpose(1, 2) for i in range(2))
    cache = npa.Kv8Cache.empty(B, h, 256, d)
    cache.k.view(torch.uint8).fill_(0x41)
    cache.v.view(torch.uint8).fill_(0x7F)      # NaN codes
    npa.kv8_store(cache, k, v, start=64)
    torch.cuda.synchronize()
    for t, fill in ((cache.k, 0x41), (cache.v, 0x7F)):
        u = t.view(torch.uint8)
        assert (u[:, :, :64] == fill).all() and (u[:, :, 64 + n:] == fill).all()
    e = npa.Kv8Cache.empty(B, h, 256, d)
    npa.kv8_store(e, k.contiguous(), v.contiguous(), start=64)
    assert torch.equal(e.k.view(torch.uint8)[:, :, 64:64 + n], cache.k.view(torch.uint8)[:, :, 64:64 + n])
    assert torch.equal(e.v.view(torch.uint8)[:, :, 64:64 + n], cache.v.view(torch.uint8)[:, :, 64:64 + n])
    one = randn(31, 1, h, 64, d).expand(B, h, 64, d)
    npa.kv8_store(e, one, one, start=0)
    assert torch.equal(e.k[0].view(torch.uint8)[:, :64], e.k[1].view(torch.uint8)[:, :64])


def filled(npa, seed, B, h, n, d):
    """A cache of n stored tokens with blocks of differing size; past them NaN codes."""
    cache = npa.Kv8Cache.empty(B, h, n + 70, d)
    cache.k.view(torch.uint8).fill_(0x7F)
    cache.v.view(torch.uint8).fill_(0xFF)
    size = torch.from_numpy(np.exp(0.4 * np.random.default_rng(seed).standard_normal((1, 1, n, 1)))).cuda()
    k, v = (randn(seed + i, B, h, n, d).double() * size for i in (1, 2))
    npa.kv8_store(cache, k.bfloat16(), v.bfloat16())
    return cache


def values(codes, scale, n):
    return (codes64(codes) * np.repeat(f64(scale), 64, axis=2)[..., None])[:, :, :n]


def attend_and_check(npa, q, cache, n, kv_lens=None, key_mask=None, scale=None, what="", **kw):
    B = q.shape[0]
    keep = np.ones((B, n), dtype=bool)
    kv = km = None
    if kv_lens is not None:
        keep &= np.arange(n)[None] < np.clip(kv_lens, 0, n)[:, None]
        kv = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    if key_mask is not None:
        keep &= key_mask
        km = torch.from_numpy(key_mask).cuda()
    out = npa.kv8_cross_attention(q, cache, n, kv_lens=kv, key_mask=km, scale=scale, **kw)
    torch.cuda.synchronize()
    assert npa.npa_device_status() == npa.NPA_OK
    v = values(cache.v, cache.v_scale, n)
    ref, mag = oracle.cross_attention(f64(q), values(cache.k, cache.k_scale, n), v, keep=keep, scale=scale)
    check_attention(f64(out), ref, mag, "bf16", n, float(np.nanmax(np.abs(v))), what, kv8=True)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,n", [(1, 1), (1, 77), (16, 64), (128, 65), (129, 128), (257, 129), (300, 500), (40, 192),
                                  (700, 257)])
def test_attention_lengths(npa, d, Lq, n):
    cache = filled(npa, 5 * n, 2, 3, n, d)
    attend_and_check(npa, randn(40, 2, 3, Lq, d), cache, n, what=(Lq, n))


@pytest.mark.parametrize("d", [64, 128])
def test_attention_long(npa, d):
    cache = filled(npa, 60, 1, 2, 4500, d)
    for Lq, split in ((1, True), (1, False), (260, True), (260, False)):
        attend_and_check(npa, randn(61, 1, 2, Lq, d), cache, 4500, split=split, what=(Lq, split))
    cache = filled(npa, 62, 2, 4, 600, d)
    attend_and_check(npa, randn(63, 2, 4, 6000, d), cache, 600)


@pytest.mark.parametrize("d,n,lens", [(64, 2500, None), (128, 1800, [1800, 700])])
def test_attention_more_units_than_multiprocessors(npa, d, n, lens):
    """Whole units in waves, then the rest cut into pieces of the key range."""
    cache = filled(npa, 65, 2, 5, n, d)
    q = randn(66, 2, 5, 4000, d)
    attend_and_check(npa, q, cache, n, kv_lens=lens)
    attend_and_check(npa, q, cache, n, kv_lens=lens, split=False)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_heads_lens_masks(npa, d):
    B, n = 4, 400
    cache = filled(npa, 70, B, 2, n, d)
    rng = np.random.default_rng(5)
    mask = rng.random((B, n)) < 0.5
    mask[1] = False
    lens = [n, 33, 0, 129]
    for Lq in (1, 140):
        q = randn(71, B, 6, Lq, d)
        attend_and_check(npa, q, cache, n)
        out = attend_and_check(npa, q, cache, n, kv_lens=lens)
        assert not out[2].any()
        out = attend_and_check(npa, q, cache, n, key_mask=mask)
        assert not out[1].any()
        attend_and_check(npa, q, cache, n, key_mask=mask, kv_lens=lens, scale=0.3, split=False)


@pytest.mark.parametrize("Lq", [1, 5, 140])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_blocks_without_kept_keys(npa, d, Lq):
    """A block that the mask leaves out altogether was perhaps never stored:
    its scales may hold anything, alone in a 128-key block or with its other half."""
    B, n = 2, 500
    cache = filled(npa, 75, B, 2, n, d)
    mask = np.ones((B, n), dtype=bool)
    nan, inf = float("nan"), float("inf")   # (the bound takes the largest finite value: no inf there)
    for i, bad_k, bad_v in ((0, nan, nan), (3, inf, 0.0), (4, 0.0, nan), (5, -1.0, -1.0)):
        mask[:, 64 * i:64 * i + 64] = False
        cache.k_scale[:, :, i] = bad_k
        cache.v_scale[:, :, i] = bad_v
    mask[0, 64:100] = False
    attend_and_check(npa, randn(76, B, 4, Lq, d), cache, n, key_mask=mask)
    mask[1] = False
    assert not attend_and_check(npa, randn(76, B, 4, Lq, d), cache, n, key_mask=mask)[1].any()


def test_attention_layouts_and_guard(npa):
    B, h, Lq, n, d = 2, 3, 140, 200, 64
    cache = filled(npa, 80, B, h, n, d)
    q = randn(81, B, Lq, h, d).transpose(1, 2)
    buf = torch.full((B, Lq + 2, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
    attend_and_check(npa, q, cache, n, out=buf[:, 1:-1].transpose(1, 2))
    assert (buf[:, 0] == 7.0).all() and (buf[:, -1] == 7.0).all()


@pytest.mark.parametrize("Lq", [3, 50])
def test_other_scales(npa, Lq):
    """Scales that are no powers of two (a cache filled elsewhere) are as exact."""
    B, h, n, d = 1, 2, 300, 64
    cache = filled(npa, 90, B, h, n, d)
    cache.k_scale.mul_(1.2345)
    cache.v_scale.mul_(0.777)
    attend_and_check(npa, randn(91, B, h, Lq, d), cache, n)


@pytest.mark.parametrize("Lq", [2, 150])
def test_sizes_of_values_and_queries(npa, Lq):
    """Blocks whose values differ by 2^60, tiny and huge keys and queries."""
    B, h, n, d = 1, 2, 320, 64
    k, v = randn(95, B, h, n, d), randn(96, B, h, n, d)
    size = torch.tensor([1.0, 2.0 ** -40, 2.0 ** 20, 1.0, 2.0 ** -8], device="cuda").repeat_interleave(64)[:, None]
    for ks, qs in ((1.0, 1.0), (2.0 ** -60, 2.0 ** 60), (2.0 ** 70, 2.0 ** -70)):
        cache = npa.Kv8Cache.empty(B, h, n, d)
        npa.kv8_store(cache, (k.double() * ks).bfloat16(), (v.double() * size).bfloat16())
        attend_and_check(npa, (randn(97, B, h, Lq, d).double() * qs).bfloat16(), cache, n, what=(ks, qs))


def test_a_denoising_loop_in_one_graph(npa):
    """Store and attend captured together, replayed on new states."""
    B, h, n, d = 1, 4, 300, 64
    cache = npa.Kv8Cache.empty(B, h, n, d)
    q, k, v = randn(1, B, h, 200, d), randn(2, B, h, n, d), randn(3, B, h, n, d)
    npa.kv8_store(cache, k, v)
    eager = npa.kv8_cross_attention(q, cache, n)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        npa.kv8_store(cache, k, v)
        npa.kv8_cross_attention(q, cache, n, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(eager))
    k.copy_(randn(4, *k.shape))
    g.replay()
    torch.cuda.synchronize()
    other = npa.Kv8Cache.empty(B, h, n, d)
    npa.kv8_store(other, k, v)
    again = npa.kv8_cross_attention(q, other, n)
    assert torch.equal(bits(out), bits(again)) and not torch.equal(bits(out), bits(eager))


def test_checked_build(npa):
    npa.use_bounds_checking(True)
    try:
        for d in (64, 128):
            for Lq, n in ((1, 1), (130, 515), (2, 3001)):
                cache = filled(npa, Lq, 2, 2, n, d)
                attend_and_check(npa, randn(9, 2, 4, Lq, d), cache, n, kv_lens=[n, n // 2])
    finally:
        npa.use_bounds_checking(False)


@pytest.mark.parametrize("i", range(16))
def test_random_shapes(npa, i):
    rng = np.random.default_rng(900 + i)
    B, kvh, per = int(rng.integers(1, 4)), int(rng.integers(1, 4)), int(rng.choice([1, 1, 2, 3]))
    d = int(rng.choice([64, 128]))
    Lq, n = int(2 ** rng.uniform(0, 9.5)), int(2 ** rng.uniform(0, 11))
    cache = filled(npa, 7 * i, B, kvh, n, d)
    lens = rng.integers(0, n + 1, B) if rng.random() < 0.4 else None
    mask = rng.random((B, n)) < rng.random() if rng.random() < 0.4 else None
    attend_and_check(npa, randn(5, B, kvh * per, Lq, d), cache, n, kv_lens=lens, key_mask=mask,
                     split=bool(rng.random() < 0.7), what=(B, kvh, per, d, Lq, n))
