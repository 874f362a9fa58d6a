"""Cross attention (npa_cross_attention_fwd) on the GPU against the float64
oracle: lengths around the tile and block borders, both dtypes and head
dimensions, shared heads, caller's strides, lengths and masks (rows without
keys, NaN and infinities in what is left out), splits, streams and graphs."""
import numpy as np
import pytest

import oracle
from _block import attention_bound, bits, check_attention, f64, randn, torch_dtype

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


def keep_of(B, Lk, kv_lens=None, key_mask=None):
    keep = np.ones((B, Lk), dtype=bool)
    if kv_lens is not None:
        keep &= np.arange(Lk)[None] < np.clip(np.asarray(kv_lens), 0, Lk)[:, None]
    if key_mask is not None:
        keep &= np.asarray(key_mask, dtype=bool)
    return keep


def run_and_check(npa, q, k, v, dtype, kv_lens=None, key_mask=None, scale=None, what="", **kw):
    B, Lk = q.shape[0], k.shape[2]
    keep = keep_of(B, Lk, kv_lens, key_mask)
    kv = None if kv_lens is None else torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    km = None if key_mask is None else torch.tensor(np.asarray(key_mask, dtype=bool), device="cuda")
    out = npa.cross_attention(q, k, v, kv_lens=kv, key_mask=km, scale=scale, **kw)
    torch.cuda.synchronize()
    assert npa.npa_device_status() == npa.NPA_OK
    v64 = f64(v)
    ref, mag = oracle.cross_attention(f64(q), f64(k), v64, keep=keep, scale=scale)
    vmax = float(np.abs(v64[np.isfinite(v64)]).max())
    check_attention(f64(out), ref, mag, dtype, Lk, vmax, what)
    return out


def qkv(seed, B, heads, kv_heads, Lq, Lk, d, dtype="bf16"):
    return (randn(seed, B, heads, Lq, d, dtype=dtype), randn(seed + 1, B, kv_heads, Lk, d, dtype=dtype),
            randn(seed + 2, B, kv_heads, Lk, d, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (1, 77), (3, 2), (128, 128), (129, 127), (256, 129), (257, 16), (300, 77),
                                   (31, 33), (33, 96), (64, 97), (255, 256), (511, 257), (40, 400)])
def test_lengths(npa, dtype, d, Lq, Lk):
    q, k, v = qkv(100 + Lq + Lk, 2, 3, 3, Lq, Lk, d, dtype)
    run_and_check(npa, q, k, v, dtype, what=(Lq, Lk))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lk", list(range(1, 20)) + [31, 32, 47, 48, 49, 63, 64, 65, 79, 80, 81, 95, 111, 112, 113, 144, 145])
def test_every_tail(npa, d, Lk):
    """The last block's products and exponentials stop at its last key."""
    q, k, v = qkv(Lk, 1, 2, 2, 130, Lk, d)
    run_and_check(npa, q, k, v, "bf16", what=Lk)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16"), (64, "fp16"), (128, "bf16")])
def test_few_rows_split_in_every_way(npa, d, dtype):
    """At most 16 rows: whole, split inside clusters of each size, split through
    the workspace; pieces without keys, rows without keys, more units than run at once."""
    for i, (B, heads, kv_heads, Lq, Lk) in enumerate(((1, 1, 1, 1, 40), (2, 2, 2, 3, 300), (1, 3, 3, 16, 600), (3, 6, 2, 5, 900),
                                                      (4, 20, 20, 1, 1200), (2, 20, 20, 9, 1500), (3, 10, 10, 2, 2100),
                                                      (1, 2, 1, 8, 5000), (30, 20, 20, 1, 260))):
        lens = np.random.default_rng(i).integers(0, Lk + 1, B)
        lens[0] = Lk
        if B > 2:
            lens[1:3] = 0, 1
        mask = np.random.default_rng(i).random((B, Lk)) < 0.3
        q, k, v = qkv(700 + i, B, heads, kv_heads, Lq, Lk, d, dtype)
        for kw in ({}, {"kv_lens": lens.tolist()}, {"key_mask": mask, "split": False}):
            run_and_check(npa, q, k, v, dtype, what=(i, list(kw)), **kw)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
def test_many_rows_of_one_tile(npa, d, dtype):
    """Every tile has keys of its own (at most 128 queries a head), of another
    length than its neighbours': a warpgroup's tiles skip key sets."""
    B, Lk = 1400, 77
    rng = np.random.default_rng(17)
    lens = rng.integers(0, Lk + 1, B)
    lens[rng.random(B) < 0.3] = 0
    mask = rng.random((B, Lk)) < 0.5
    mask[::3] = False
    for heads, kv_heads, Lq, Bi in ((1, 1, 20, B), (2, 1, 17, 700), (3, 3, 128, 300), (1, 1, 130, 700)):
        q, k, v = qkv(800 + Lq, Bi, heads, kv_heads, Lq, Lk, d, dtype)
        run_and_check(npa, q, k, v, dtype, kv_lens=lens[:Bi].tolist(), what=(heads, Lq, "lens"))
        run_and_check(npa, q, k, v, dtype, key_mask=mask[:Bi], what=(heads, Lq, "mask"))
        run_and_check(npa, q, k, v, dtype, what=(heads, Lq))


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
def test_rows_in_the_order_of_their_lengths(npa, d, dtype):
    """More units than multiprocessors: rows run shortest first, whole units and
    cut ones; equal lengths, none at all, and lengths outside the tensor."""
    for B, heads, Lq, Lk in ((2, 5, 4200, 1400), (5, 3, 3000, 700), (8, 4, 1300, 2100), (9, 4, 1300, 600)):
        q, k, v = qkv(900 + B, B, heads, heads, Lq, Lk, d, dtype)
        for lens in ([Lk] + [Lk // 2] * (B - 1), [Lk - 37 * i for i in range(B)], [(91 * i) % 500 for i in range(B)],
                     [0] + [Lk + 5] * (B - 1), [-3] * B):
            run_and_check(npa, q, k, v, dtype, kv_lens=lens, what=(B, lens))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("fp16", 64), ("bf16", 128), ("fp16", 128)])
def test_long_keys(npa, dtype, d):
    """Many blocks: ring wrap-around, rescaling, splits; and many units of
    several blocks without splits."""
    q, k, v = qkv(7, 1, 2, 2, 200, 5000, d, dtype)
    run_and_check(npa, q, k, v, dtype, what="split")
    run_and_check(npa, q, k, v, dtype, split=False, what="unsplit")
    q, k, v = qkv(8, 2, 5, 5, 4000, 640, d, dtype)
    run_and_check(npa, q, k, v, dtype, what="units")


@pytest.mark.parametrize("d,Lk,lens", [(64, 2500, None), (128, 1800, [1800, 700]), (64, 2200, [5, 2200])])
def test_more_units_than_multiprocessors(npa, d, Lk, lens):
    """Whole units in waves, then the rest cut into pieces of the key range;
    batch rows whose keys end inside, before and after a piece."""
    q, k, v = qkv(9, 2, 5, 5, 4000, Lk, d)
    assert npa.npa_cross_attention_workspace_size(2, 5, 5, 4000, Lk, d) > 0
    a = run_and_check(npa, q, k, v, "bf16", kv_lens=lens, what="cut")
    b = npa.cross_attention(q, k, v, kv_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
    assert torch.equal(bits(a), bits(b))
    run_and_check(npa, q, k, v, "bf16", kv_lens=lens, split=False, what="whole")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_scores(npa, d, dtype):
    """Scores that grow along the keys by hundreds: the reference has to move."""
    q, k, v = qkv(21, 1, 2, 2, 257, 900, d, dtype)
    k = (k.float() * torch.linspace(0.1, 12.0, 900, device="cuda")[None, None, :, None]).to(torch_dtype(dtype))
    B = 1
    out = npa.cross_attention(q, k, v)
    torch.cuda.synchronize()
    ref, mag = oracle.cross_attention(f64(q), f64(k), f64(v))
    # scores of size S carry a float32 error of about 2^-22 S (sums of d products, one product with the scale), and
    # a probability that much relative error: S < 2^9 here
    extra = 2.0 ** -12 * mag
    bound = attention_bound(ref, mag, dtype, 900, float(v.abs().max())) + extra
    assert (np.abs(f64(out) - ref) <= bound).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(6, 2), (4, 1)])
def test_shared_heads(npa, d, heads, kv_heads):
    q, k, v = qkv(31, 2, heads, kv_heads, 150, 140, d)
    run_and_check(npa, q, k, v, "bf16")
    q, k, v = qkv(32, 2, heads, kv_heads, 1, 3000, d)
    run_and_check(npa, q, k, v, "bf16")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("split", [True, False])
def test_lengths_per_row(npa, d, split):
    """Rows of every kind of length, none and too large ones among them; what
    lies past a row's length is NaN and infinity."""
    B, Lk = 8, 700
    lens = [700, 0, 1, 128, 129, 5000, -3, 333]
    for Lq in (1, 300):
        q, k, v = qkv(41, B, 2, 2, Lq, Lk, d)
        for b, n in enumerate(np.clip(lens, 0, Lk)):
            k[b, :, n:] = float("nan")
            v[b, :, n:] = float("inf")
            v[b, :, n::2] = float("nan")
        out = run_and_check(npa, q, k, v, "bf16", kv_lens=lens, split=split)
        assert not out[1].any() and not out[6].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lk", [77, 128, 515])
def test_masks(npa, dtype, d, Lk):
    """Scattered masks, an empty row, a row that keeps its last key only, a
    whole block left out; NaN, infinities and the type's lowest value in what
    is left out."""
    B = 5
    rng = np.random.default_rng(Lk + d)
    mask = rng.random((B, Lk)) < 0.5
    mask[1] = False
    mask[2] = False
    mask[2, -1] = True
    if Lk > 300:
        mask[3, 128:256] = False
        mask[4, :256] = False
    q, k, v = qkv(51, B, 2, 2, 140, Lk, d, dtype)
    low = torch.finfo(torch_dtype(dtype)).min
    for b in range(B):
        out_ = torch.from_numpy(np.flatnonzero(~mask[b])).cuda()
        k[b, :, out_] = low
        k[b, :, out_[::3]] = float("nan")
        v[b, :, out_] = low
        v[b, :, out_[::2]] = float("nan")
        v[b, :, out_[1::3]] = float("-inf")
    out = run_and_check(npa, q, k, v, dtype, key_mask=mask)
    assert not out[1].any()
    lens = [Lk, Lk, Lk - 1, Lk // 2, 3]
    out = run_and_check(npa, q, k, v, dtype, key_mask=mask, kv_lens=lens, split=False)
    assert not out[2].any()


def test_mask_as_bytes(npa):
    q, k, v = qkv(55, 2, 2, 2, 33, 90, 64)
    m = torch.from_numpy(np.random.default_rng(3).integers(0, 2, (2, 90)).astype(np.uint8) * 7).cuda()
    a = npa.cross_attention(q, k, v, key_mask=m)
    b = npa.cross_attention(q, k, v, key_mask=m != 0)
    assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("d", [64, 128])
def test_projection_layouts(npa, d):
    """q from [B, L, heads * d], k and v from one [B, L, 2, heads, d] buffer,
    the output into a slice of a larger one whose rest stays as it was."""
    B, h, Lq, Lk = 2, 3, 200, 150
    q = randn(61, B, Lq, h, d).transpose(1, 2)
    kv = randn(62, B, Lk, 2, h, d)
    k, v = (kv[:, :, i].transpose(1, 2) for i in range(2))
    out = run_and_check(npa, q, k, v, "bf16")
    assert out.stride() == q.stride()
    buf = torch.full((B, Lq + 5, h + 1, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    view = buf[:, 2:Lq + 2, :h, :d].transpose(1, 2)
    run_and_check(npa, q, k, v, "bf16", out=view)
    buf[:, 2:Lq + 2, :h, :d] = 7.0
    assert (buf == 7.0).all()
    for Lq_ in (1, 40):     # the merged splits too
        q1 = randn(63, B, h, Lq_, d)
        k1, v1 = randn(64, B, h, 2000, d), randn(65, B, h, 2000, d)
        buf = torch.full((B, Lq_ + 3, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
        run_and_check(npa, q1, k1, v1, "bf16", out=buf[:, 1:Lq_ + 1].transpose(1, 2))
        buf[:, 1:Lq_ + 1] = 7.0
        assert (buf == 7.0).all()


@pytest.mark.parametrize("Lq", [2, 260])
def test_repeated_inputs(npa, Lq):
    """expand()ed states: one prompt for the batch, one head for all."""
    q = randn(71, 3, 4, Lq, 64)
    k, v = randn(72, 1, 4, 300, 64).expand(3, 4, 300, 64), randn(73, 3, 1, 300, 64).expand(3, 4, 300, 64)
    run_and_check(npa, q, k, v, "bf16")


@pytest.mark.parametrize("scale", [0.02, 0.125, 1.5])
def test_scale(npa, scale):
    q, k, v = qkv(81, 1, 2, 2, 100, 200, 64)
    run_and_check(npa, q, k, v, "bf16", scale=scale)


def test_workspace_sizes(npa):
    """No workspace, too small a one and the planned one: the same result up
    to the merge's rounding; what lies past the workspace stays."""
    B, h, Lq, Lk, d = 1, 3, 20, 6000, 64
    q, k, v = qkv(91, B, h, h, Lq, Lk, d)
    ref, mag = oracle.cross_attention(f64(q), f64(k), f64(v))
    full = npa.npa_cross_attention_workspace_size(B, h, h, Lq, Lk, d)
    assert full > 0
    one = B * h * Lq * (d + 2) * 4
    for nbytes in (0, one, 2 * one, 3 * one + 4, full):
        ws = torch.full((full // 4 + 64,), 7.0, device="cuda")
        o = torch.full_like(q, float("nan"))
        npa.npa_cross_attention_fwd(q, k, v, o, npa.NPA_DTYPE_BF16, B, h, h, Lq, Lk, d,
                                    workspace=ws if nbytes else None, workspace_bytes=nbytes)
        torch.cuda.synchronize()
        check_attention(f64(o), ref, mag, "bf16", Lk, 6.0, nbytes)
        assert (ws[nbytes // 4:] == 7.0).all()


def test_repeatable_and_side_stream(npa):
    for shape in ((2, 5, 5, 700, 300, 64), (1, 3, 3, 5, 4000, 128)):
        q, k, v = qkv(95, *shape)
        a = npa.cross_attention(q, k, v)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        outs = [npa.cross_attention(q, k, v, stream=s) for _ in range(3)]
        outs.append(npa.cross_attention(q, k, v, stream=s.cuda_stream))
        s.synchronize()
        for o in outs:
            assert torch.equal(bits(o), bits(a))


def test_two_calls_at_once(npa):
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    qa, ka, va = qkv(96, 1, 4, 4, 3, 9000, 64)
    qb, kb, vb = qkv(97, 1, 4, 4, 3, 9000, 64)
    a, b = npa.cross_attention(qa, ka, va), npa.cross_attention(qb, kb, vb)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = []
    for _ in range(10):
        res.append((npa.cross_attention(qa, ka, va, stream=s), npa.cross_attention(qb, kb, vb, stream=t)))
    torch.cuda.synchronize()
    for x, y in res:
        assert torch.equal(bits(x), bits(a)) and torch.equal(bits(y), bits(b))


@pytest.mark.parametrize("Lq,Lk,masked", [(300, 77, True), (2, 4000, False)])
def test_graph_replay(npa, Lq, Lk, masked):
    q, k, v = qkv(98, 2, 2, 2, Lq, Lk, 64)
    m = torch.ones(2, Lk, dtype=torch.bool, device="cuda") if masked else None
    eager = npa.cross_attention(q, k, v, key_mask=m)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        npa.cross_attention(q, k, v, key_mask=m, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(eager))
    q.copy_(randn(99, *q.shape))
    if masked:
        m[0, Lk // 2:] = False
    again = npa.cross_attention(q, k, v, key_mask=m)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(again)) and not torch.equal(bits(again), bits(eager))


def test_checked_build(npa):
    """The bounds-checking build runs ragged cases without a finding."""
    npa.use_bounds_checking(True)
    try:
        for d in (64, 128):
            for Lq, Lk in ((1, 1), (300, 77), (130, 515), (2, 3001)):
                q, k, v = qkv(Lq, 2, 2, 1, Lq, Lk, d)
                run_and_check(npa, q, k, v, "bf16", kv_lens=[Lk, Lk // 2])
                run_and_check(npa, q, k, v, "bf16")
    finally:
        npa.use_bounds_checking(False)


@pytest.mark.parametrize("i", range(24))
def test_random_shapes(npa, i):
    rng = np.random.default_rng(700 + i)
    B, kvh, per = int(rng.integers(1, 4)), int(rng.integers(1, 4)), int(rng.choice([1, 1, 2, 3]))
    d, dtype = int(rng.choice([64, 128])), str(rng.choice(["bf16", "fp16"]))
    Lq, Lk = int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 11))
    q, k, v = qkv(800 + 3 * i, B, kvh * per, kvh, Lq, Lk, d, dtype)
    lens = rng.integers(0, Lk + 1, B) if rng.random() < 0.4 else None
    mask = rng.random((B, Lk)) < rng.random() if rng.random() < 0.4 else None
    run_and_check(npa, q, k, v, dtype, kv_lens=lens, key_mask=mask, split=bool(rng.random() < 0.7),
                  what=(B, kvh, per, d, dtype, Lq, Lk))
