"""Group norm with an activation, channels last (npa_group_norm_act) on the
GPU against the float64 oracle."""
import numpy as np
import pytest

import oracle
from _block import HALF_STEP, HALF_SUB, bits, check_attention, f64, randn, torch_dtype

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def npa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from patch_res_diffusion_b200 import build
    build.build()
    import patch_res_diffusion_b200 as m
    yield m
    assert m.npa_device_status() == m.NPA_OK


def bound(y, z, lift, dtype):
    """float32 arithmetic: mean and rstd are within 2^-20 relative of exact
    (pairwise merged sums of at most some thousand terms each), so z is off by
    at most 2^-20 (|z| + lift + |z - b|), where |z - b| <= |z| + |b| is covered
    by taking 2^-19; SiLU's slope is at most 1.1 and its exponential and
    quotient add 2^-20 (1 + |z|) relative; then one rounding."""
    e32 = 2.0 ** -19 * (np.abs(z) + lift + 1.0)
    return 1.1 * e32 + 2.0 ** -20 * (1 + np.abs(z)) * np.abs(y) + HALF_STEP[dtype] * np.abs(y) + HALF_SUB[dtype]


def run_and_check(npa, x, groups, w=None, b=None, eps=1e-5, act=None, dtype="bf16", what="", **kw):
    x64 = f64(x)
    out = npa.group_norm(x, groups, w, b, eps=eps, act=act, **kw)
    torch.cuda.synchronize()
    y, z, lift = oracle.group_norm(x64, groups, None if w is None else f64(w), None if b is None else f64(b), eps, act)
    got = f64(out)
    assert np.isfinite(got).all(), what
    over = np.abs(got - y) / bound(y, z, lift, dtype)
    assert over.max() <= 1, (what, float(over.max()), float(np.abs(got - y).max()))
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("B,N,C,groups", [(1, 1, 8, 1), (2, 1, 64, 32), (2, 64, 320, 32), (1, 1024, 1280, 32),
                                          (3, 257, 640, 32), (2, 31, 96, 8), (1, 5000, 32, 32), (2, 100, 2560, 32),
                                          (1, 333, 4096, 1), (1, 7, 40, 5), (70, 9, 16, 4)])
def test_shapes(npa, dtype, act, B, N, C, groups):
    x = randn(N + C, B, N, C, dtype=dtype) + randn(1, C, dtype=dtype)
    w, b = randn(2, C, dtype=dtype) * 0.2 + 1, randn(3, C, dtype=dtype) * 0.3
    # one element per group: the output is exactly the bias, up to 0 * rstd
    run_and_check(npa, x, groups, w, b, act=act, dtype=dtype, what=(B, N, C, groups))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("C,groups", [(1, 1), (3, 3), (30, 3), (33, 11), (129, 1), (1025, 5), (517, 517)])
def test_odd_channels(npa, dtype, C, groups):
    """Rows that are not made of 16-byte pieces."""
    x = randn(C, 2, 203, C, dtype=dtype)
    run_and_check(npa, x, groups, randn(2, C, dtype=dtype), randn(3, C, dtype=dtype), act="silu", dtype=dtype)
    run_and_check(npa, x, groups, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_float32_weights(npa, dtype):
    x = randn(11, 2, 300, 320, dtype=dtype)
    w, b = randn(12, 320, dtype="fp32"), randn(13, 320, dtype="fp32")
    run_and_check(npa, x, 32, w, b, act="silu", dtype=dtype)
    run_and_check(npa, x, 32, w, None, dtype=dtype)
    run_and_check(npa, x, 32, None, b, dtype=dtype)


@pytest.mark.parametrize("shift,sd", [(1000.0, 1.0), (-3e4, 2.0), (0.0, 1e-6), (5.0, 0.0), (0.0, 1e15)])
def test_means_and_spreads(npa, shift, sd):
    """A mean far from zero, tiny and huge spreads, a constant group."""
    x = (randn(21, 2, 5000, 64, dtype="fp32", sd=1.0) * sd + shift)
    run_and_check(npa, x, 8, dtype="fp32", act="silu" if sd != 1e15 else None)


def test_outliers(npa):
    """One huge element (the first of all among them) does not spoil the variance."""
    for at in (0, 3999):
        x = randn(22, 1, 4000, 32, dtype="fp32")
        x[0, at, 0] = 1e5
        run_and_check(npa, x, 4, dtype="fp32")


def test_extreme_activations(npa):
    x = randn(23, 1, 50, 32, dtype="fp32")
    w = torch.full((32,), 60.0, device="cuda")
    run_and_check(npa, x, 4, w, torch.zeros(32, device="cuda"), act="silu", dtype="fp32")


def test_large(npa):
    """Many tiles, and more rows than one block of each tile takes at a time."""
    x = randn(24, 1, 70000, 320)
    run_and_check(npa, x, 32, randn(25, 320), randn(26, 320), act="silu")


@pytest.mark.parametrize("B,N,C,groups,dtype", [(1, 40000, 128, 32, "bf16"), (3, 20000, 64, 4, "fp16"),
                                                (5, 50000, 128, 32, "bf16"), (2, 300000, 48, 3, "bf16"),
                                                (1, 45000, 320, 32, "fp32"), (2, 4096, 640, 32, "bf16"),
                                                (1, 16384, 320, 32, "bf16"), (9, 1500, 72, 9, "fp32")])
def test_plans(npa, B, N, C, groups, dtype):
    """Sizes on both sides of what a cluster holds: one item, several batch
    rows to an item (a shorter last one), channel chunks, blocks of a cluster
    without tokens."""
    x = randn(70, B, N, C, dtype=dtype) + randn(71, C, dtype=dtype)
    y = x.clone()
    a = run_and_check(npa, x, groups, randn(72, C, dtype=dtype), randn(73, C, dtype=dtype), act="silu", dtype=dtype)
    npa.group_norm(y, groups, randn(72, C, dtype=dtype), randn(73, C, dtype=dtype), act="silu", out=y)
    assert torch.equal(bits(a), bits(y))


def test_workspace(npa):
    """A short workspace is refused; what lies past it stays; none is needed for small tensors."""
    assert npa.npa_group_norm_workspace_size(npa.NPA_DTYPE_BF16, 2, 1024, 1280, 32) > 0   # rows may be misaligned
    x = randn(74, 1, 1024, 1280)
    y, z = torch.empty_like(x), torch.empty_like(x)
    args = (npa.NPA_DTYPE_BF16, npa.NPA_DTYPE_BF16, 1, 1024, 1280, 32, 1024 * 1280, 1280, 1024 * 1280, 1280, 1e-5, 0)
    npa.npa_group_norm_act(x, None, None, y, *args, None, 0)
    x = randn(75, 1, 40000, 320)
    y = torch.empty_like(x)
    args = (npa.NPA_DTYPE_BF16, npa.NPA_DTYPE_BF16, 1, 40000, 320, 32, 40000 * 320, 320, 40000 * 320, 320, 1e-5, 0)
    n = npa.npa_group_norm_workspace_size(npa.NPA_DTYPE_BF16, 1, 40000, 320, 32)
    ws = torch.full((n // 4 + 16,), 7.0, device="cuda")
    with pytest.raises(npa.NpaError):
        npa.npa_group_norm_act(x, None, None, y, *args, ws, n // 2)
    with pytest.raises(npa.NpaError):
        npa.npa_group_norm_act(x, None, None, y, *args, None, 0)
    npa.npa_group_norm_act(x, None, None, y, *args, ws, n)
    torch.cuda.synchronize()
    assert (ws[n // 4:] == 7.0).all()
    assert torch.equal(bits(y), bits(npa.group_norm(x, 32)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_in_place_and_guards(npa, dtype):
    """A slice of a concatenated tensor in, a slice of another out, rest
    untouched; in place; rows that are not 16-byte aligned."""
    B, N, C = 2, 130, 64
    for pad in (64, 3):
        big = randn(31, B, N + 2, C + pad, dtype=dtype)
        x = big[:, 1:-1, pad:]
        out = torch.full((B, N + 3, C + 2 * pad), 7.0, dtype=torch_dtype(dtype), device="cuda")
        view = out[:, 2:-1, pad:pad + C]
        run_and_check(npa, x, 8, randn(32, C, dtype=dtype), None, act="silu", dtype=dtype, out=view)
        view.fill_(7.0)
        assert (out == 7.0).all()
    x = randn(33, B, N, C, dtype=dtype)
    want = npa.group_norm(x, 8, act="silu")
    y = x.clone()
    npa.group_norm(y, 8, act="silu", out=y)
    assert torch.equal(bits(y), bits(want))
    t = randn(34, N, B, C, dtype=dtype).transpose(0, 1)      # tokens outermost
    run_and_check(npa, t, 8, dtype=dtype)


def test_not_finite(npa):
    """A NaN spoils its own group of its own batch row only."""
    x = randn(41, 2, 200, 64)
    clean = npa.group_norm(x, 8)
    x[0, 17, 9] = float("nan")
    y = npa.group_norm(x, 8)
    assert torch.isnan(y[0, :, 8:16]).all()
    y[0, :, 8:16] = clean[0, :, 8:16]
    assert torch.equal(bits(y), bits(clean))


def test_repeatable_streams_and_graph(npa):
    x, w = randn(51, 2, 3000, 320), randn(52, 320)
    a = npa.group_norm(x, 32, w, act="silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [npa.group_norm(x, 32, w, act="silu", stream=s) for _ in range(20)]
    s.synchronize()
    assert all(torch.equal(bits(o), bits(a)) for o in outs)
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        npa.group_norm(x, 32, w, act="silu", out=out)
    for seed in (53, 54):
        x.copy_(randn(seed, *x.shape))
        want = npa.group_norm(x, 32, w, act="silu")
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want))


def test_a_block_of_a_network(npa):
    """Norm, cross attention to a padded prompt, then the result kept in an
    8-bit cache and read by a few latent queries: each step's result against
    the oracle on what the step before returned."""
    B, N, C, h, d = 2, 300, 320, 5, 64
    x = randn(61, B, N, C)
    y = run_and_check(npa, x, 32, randn(62, C), randn(63, C), act="silu")
    q = y.view(B, N, h, d).transpose(1, 2)
    k, v = (randn(64 + i, B, 77, h, d).transpose(1, 2) for i in range(2))
    lens = torch.tensor([77, 20], dtype=torch.int32, device="cuda")
    o = npa.cross_attention(q, k, v, kv_lens=lens)
    keep = np.arange(77)[None] < f64(lens)[:, None]
    check_attention(f64(o), *oracle.cross_attention(f64(q), f64(k), f64(v), keep=keep), "bf16", 77, 6.0)
    cache = npa.Kv8Cache.empty(B, h, N, d)
    npa.kv8_store(cache, o, q)
    z = npa.kv8_cross_attention(randn(66, B, h, 16, d), cache, N)
    val = lambda c, s: (c.cpu().double().numpy() * np.repeat(f64(s), 64, axis=2)[..., None])[:, :, :N]
    vv = val(cache.v, cache.v_scale)
    ref = oracle.cross_attention(f64(randn(66, B, h, 16, d)), val(cache.k, cache.k_scale), vv)
    check_attention(f64(z), *ref, "bf16", N, float(np.abs(vv).max()), kv8=True)
