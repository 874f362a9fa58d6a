"""NaN and infinities in what the attention reads: a NaN in a query row, or in a
key or value that is kept, shows in every output that its formula reaches, in
whichever way a call is split, and in no other."""
import numpy as np
import pytest

import oracle
from _block import attention_bound, f64, randn

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


def check(got, q, k, v, dtype, kv8=False, keep=None, what=""):
    """NaN where the oracle has NaN, the usual bound elsewhere."""
    with np.errstate(invalid="ignore"):
        ref, mag = oracle.cross_attention(q, k, v, keep=keep)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=str(what))
    ok = ~np.isnan(ref)
    vmax = float(np.nanmax(np.abs(v)))
    bound = attention_bound(np.where(ok, ref, 0.0), np.where(ok, mag, 0.0), dtype, k.shape[2], vmax, kv8)
    assert (np.abs(got - ref)[ok] <= bound[ok]).all(), what


# (B, heads, kv_heads, Lq, Lk, split): one way of the kernels each
WAYS = {
    "one step": (2, 2, 2, 1, 20, True),              # a single warp has keys
    "warps": (2, 2, 2, 3, 33, True),                 # ... several do, the last one a single key
    "warps of 300 units": (30, 20, 20, 2, 130, True),
    "cluster": (2, 4, 2, 5, 900, True),
    "cluster, two row tiles": (2, 20, 20, 9, 1500, True),
    "workspace": (1, 2, 1, 8, 6000, True),
    "at most 128 keys": (2, 3, 3, 200, 77, True),    # in the cache: one block
    "whole units": (2, 3, 3, 300, 333, False),
    "cut units": (1, 3, 3, 300, 1500, True),
    "whole and cut units": (1, 5, 5, 4000, 1100, True),
}


def inputs(way, d, dtype, seed=5):
    B, h, hk, Lq, Lk, split = WAYS[way]
    return (randn(seed, B, h, Lq, d, dtype=dtype), randn(seed + 1, B, hk, Lk, d, dtype=dtype),
            randn(seed + 2, B, hk, Lk, d, dtype=dtype), split)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("way", list(WAYS))
def test_nan_query_rows(npa, way, d, dtype):
    q, k, v, split = inputs(way, d, dtype)
    B, h, Lq, _ = q.shape
    q[0, 0, 0, 3] = float("nan")
    q[B - 1, h - 1, Lq - 1] = float("nan")
    out = npa.cross_attention(q, k, v, split=split)
    check(f64(out), f64(q), f64(k), f64(v), dtype, what=way)
    assert torch.isnan(out[0, 0, 0]).all() and torch.isnan(out[B - 1, h - 1, Lq - 1]).all()


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("place", ["first", "last", "all"])
def test_nan_keys(npa, way, d, dtype, place):
    """A kept key that is NaN, alone in the last warp's or piece's share or not:
    every query that reads it is NaN. An unkept one reaches nobody."""
    q, k, v, split = inputs(way, d, dtype, 15)
    Lk = k.shape[2]
    j = {"first": 0, "last": Lk - 1, "all": slice(None)}[place]
    k[0, 0, j, 1] = float("nan")
    out = npa.cross_attention(q, k, v, split=split)
    check(f64(out), f64(q), f64(k), f64(v), dtype, what=(way, place))
    assert torch.isnan(out[0, 0]).all()
    if place == "all":
        return
    mask = torch.ones(q.shape[0], Lk, dtype=torch.bool, device="cuda")
    mask[0, j] = False
    out = npa.cross_attention(q, k, v, key_mask=mask, split=split)
    assert not torch.isnan(out).any()


@pytest.mark.parametrize("way", list(WAYS))
def test_nan_and_infinite_values(npa, way):
    """A kept value's NaN or infinity shows in its column; a kept infinite key
    gives what the formula gives."""
    q, k, v, split = inputs(way, 64, "bf16", 25)
    v[0, 0, 0, 7] = float("nan")
    v[0, 0, -1, 9] = float("inf")
    out = npa.cross_attention(q, k, v, split=split)
    got = f64(out)
    group = q.shape[1] // k.shape[1]
    assert np.isnan(got[0, :group, :, 7]).all() and (got[0, :group, :, 9] == np.inf).all()
    got[0, :group][..., [7, 9]] = 0
    assert np.isfinite(got).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("way", list(WAYS))
def test_cache(npa, way, d):
    """The same over the 8-bit cache: NaN in a query, in a key's codes, in a value's."""
    q, k, v, split = inputs(way, d, "bf16", 35)
    B, h, Lq, _ = q.shape
    Lk = k.shape[2]
    group = h // k.shape[1]

    def run(q, k, v, mask=None):
        cache = npa.Kv8Cache.empty(B, k.shape[1], Lk, d)
        npa.kv8_store(cache, k, v)
        out = npa.kv8_cross_attention(q, cache, Lk, key_mask=mask, split=split)
        kc, vc = ((f64(c.float()) * np.repeat(f64(s), 64, axis=2)[..., None])[:, :, :Lk]
                  for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        check(f64(out), f64(q), kc, vc, "bf16", kv8=True, keep=None if mask is None else mask.cpu().numpy(), what=way)
        return out

    bad = q.clone()
    bad[0, 0, 0, 3] = float("nan")
    bad[B - 1, h - 1, Lq - 1] = float("nan")
    out = run(bad, k, v)
    assert torch.isnan(out[0, 0, 0]).all() and torch.isnan(out[B - 1, h - 1, Lq - 1]).all()
    for j in (0, Lk - 1, slice(None)):
        bad = k.clone()
        bad[0, 0, j, 1] = float("nan")
        assert torch.isnan(run(q, bad, v)[0, :group]).all()
        if j != slice(None):
            mask = torch.ones(B, Lk, dtype=torch.bool, device="cuda")
            mask[0, j] = False
            assert not torch.isnan(run(q, bad, v, mask)).any()
    bad = v.clone()
    bad[0, 0, Lk - 1, 9] = float("nan")
    out = run(q, k, bad)
    assert torch.isnan(out[0, :group, :, 9]).all()


@pytest.mark.parametrize("scale", [3.4e38, 2.4e38, 1e-38, 1e-44])
@pytest.mark.parametrize("way", ["one step", "cluster", "workspace", "at most 128 keys", "whole units", "cut units"])
def test_scales_at_the_ends_of_float32(npa, way, scale):
    """Scores that are all 0, or negligible, give the mean of the kept values."""
    q, k, v, split = inputs(way, 64, "bf16", 45)
    mask = torch.ones(q.shape[0], k.shape[2], dtype=torch.bool, device="cuda")
    mask[:, 1::3] = False
    if scale > 1:
        q.zero_()
    out = f64(npa.cross_attention(q, k, v, key_mask=mask, scale=scale, split=split))
    keep = mask.cpu().numpy()
    ref, mag = oracle.cross_attention(f64(q), f64(k), f64(v), keep=keep, scale=0.0)
    assert (np.abs(out - ref) <= attention_bound(ref, mag, "bf16", k.shape[2], 6.0)).all()
    cache = npa.Kv8Cache.empty(q.shape[0], k.shape[1], k.shape[2], 64)
    npa.kv8_store(cache, k, v)
    out = f64(npa.kv8_cross_attention(q, cache, k.shape[2], key_mask=mask, scale=scale, split=split))
    vc = (f64(cache.v.float()) * np.repeat(f64(cache.v_scale), 64, axis=2)[..., None])[:, :, :k.shape[2]]
    ref, mag = oracle.cross_attention(f64(q), f64(k), vc, keep=keep, scale=0.0)
    assert (np.abs(out - ref) <= attention_bound(ref, mag, "bf16", k.shape[2], 6.0, True)).all()
