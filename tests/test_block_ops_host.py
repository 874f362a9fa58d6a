"""Cross attention, the 8-bit cache and group norm on the host: argument
validation before any CUDA call, the helpers' refusals, and the oracle's own
pins. No compute call is made here."""
import ctypes

import numpy as np
import pytest

import oracle
import patch_res_diffusion_b200 as npa

torch = pytest.importorskip("torch")

# fake, never dereferenced addresses
Q, K, V, O, WS, LENS, MASK = (0x10000000 * (i + 1) for i in range(7))
BAD, UNS, MIS = npa.NPA_ERR_INVALID_ARG, npa.NPA_ERR_UNSUPPORTED, npa.NPA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    from patch_res_diffusion_b200 import build
    build.build()
    return npa.lib()


def st(*s):
    return ctypes.byref(npa._Strides(*s))


def cross(L, q=Q, k=K, v=V, o=O, dtype=0, B=2, h=4, kvh=4, Lq=64, Lk=77, d=64, qs=None, ks=None, vs=None, os=None,
          lens=None, mask=None, scale=0.0, ws=None, nb=0):
    return L.npa_cross_attention_fwd(q, k, v, o, dtype, B, h, kvh, Lq, Lk, d, qs, ks, vs, os, lens, mask, scale, ws,
                                     nb, None)


def test_cross_attention_refusals(L):
    for name in "qkvo":
        assert cross(L, **{name: None}) == BAD
    for name in ("B", "h", "kvh", "Lq", "Lk", "d"):
        assert cross(L, **{name: 0}) == BAD
        assert cross(L, **{name: -5}) == BAD
    assert cross(L, h=6, kvh=4) == BAD
    for s in (float("nan"), float("inf"), -0.1):
        assert cross(L, scale=s) == BAD
    for d in (32, 96, 256):
        assert cross(L, d=d) == UNS
    for t in (2, 3, -1):
        assert cross(L, dtype=t) == UNS
    assert cross(L, Lq=2 ** 31 - 1) == UNS and cross(L, Lk=2 ** 31 - 1) == UNS
    assert cross(L, B=1 << 20, h=1 << 10, kvh=1 << 10) == UNS
    for name in "qkvo":
        assert cross(L, **{name: {"q": Q, "k": K, "v": V, "o": O}[name] + 8}) == MIS
    assert cross(L, lens=LENS + 2) == MIS
    assert cross(L, ws=WS + 8, nb=1 << 20) == MIS


def test_cross_attention_strides(L):
    n = 2 * 4 * 64 * 64
    for name in ("qs", "ks", "vs", "os"):
        assert cross(L, **{name: st(-64, 64, 64)}) == BAD
        assert cross(L, **{name: st(16384, 4096, 68)}) == MIS         # rows not 16-byte aligned
        assert cross(L, **{name: st(16384, 4100, 64)}) == MIS
        assert cross(L, **{name: st(16384, 64, 32)}) == BAD           # rows on top of each other
        assert cross(L, **{name: st(1 << 40, 64, 256)}) == UNS
    assert cross(L, os=st(0, 64, 256)) == BAD                          # an output has one place per element
    assert cross(L, os=st(16384, 0, 64)) == BAD
    assert cross(L, os=st(64, 4096, 64)) == BAD
    assert cross(L, os=st(16384, 64, 128)) == BAD                      # heads of one row overlap the next row
    assert n == 32768


def test_cross_attention_overlaps(L):
    nb = 2 * 4 * 64 * 64 * 2
    assert cross(L, o=Q) == BAD and cross(L, o=K + 16) == BAD and cross(L, o=V - nb + 16) == BAD
    assert cross(L, lens=O + 64) == BAD and cross(L, mask=O + 3) == BAD
    assert cross(L, ws=Q, nb=64) == BAD and cross(L, ws=O, nb=64) == BAD and cross(L, ws=K - 64, nb=128) == BAD
    assert cross(L, lens=WS, ws=WS, nb=64) == BAD


def test_workspace_size_of_bad_arguments(L):
    f = L.npa_cross_attention_workspace_size
    assert f(0, 4, 4, 1, 77, 64) == 0 and f(1, 4, 4, 1, 77, 96) == 0 and f(1, 4, 4, -1, 77, 64) == 0
    assert f(1, 4, 3, 1, 77, 64) == 0


def kv8c(k=K, v=V, ks=0xB0000000, vs=0xC0000000, cap=128):
    return ctypes.byref(npa._Kv8Cache(k, v, ks, vs, cap))


def attend8(L, q=Q, c=None, o=O, B=2, h=4, kvh=4, Lq=64, Lk=77, d=64, scale=0.0, lens=None, ws=None, nb=0):
    return L.npa_kv8_cross_attention_fwd(q, c or kv8c(), o, B, h, kvh, Lq, Lk, d, None, None, lens, None, scale, ws,
                                         nb, None)


def store(L, k=Q, v=WS, c=None, dtype=0, B=2, kvh=4, d=64, start=0, starts=None, n=10, ks=None, vs=None):
    return L.npa_kv8_store(k, v, c or kv8c(), dtype, B, kvh, d, start, starts, n, ks, vs, None)


def test_kv8_refusals(L):
    assert L.npa_kv8_cross_attention_fwd(Q, None, O, 2, 4, 4, 64, 77, 64, None, None, None, None, 0.0, None, 0,
                                         None) == BAD
    for bad in (dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(cap=0), dict(cap=100), dict(cap=-64)):
        assert attend8(L, c=kv8c(**bad)) == BAD and store(L, c=kv8c(**bad)) == BAD
    assert attend8(L, c=kv8c(k=K + 8)) == MIS and store(L, c=kv8c(vs=0xC0000004)) == MIS
    assert attend8(L, q=None) == BAD and attend8(L, o=None) == BAD
    assert attend8(L, Lk=129) == BAD and attend8(L, kvh=3) == BAD and attend8(L, d=32) == UNS
    assert attend8(L, o=K) == BAD and attend8(L, o=0xB0000000) == BAD and attend8(L, o=Q + 16) == BAD
    assert attend8(L, ws=V, nb=64) == BAD and attend8(L, ws=0xC0000000, nb=64) == BAD
    assert store(L, k=None) == BAD and store(L, v=None) == BAD and store(L, n=0) == BAD and store(L, start=-1) == BAD
    assert store(L, start=120, n=9) == BAD and store(L, start=2 ** 31 - 1, n=2 ** 31 - 1) == BAD
    assert store(L, dtype=2) == UNS and store(L, d=80) == UNS
    assert store(L, k=Q + 8) == MIS and store(L, starts=LENS + 1) == MIS
    assert store(L, ks=st(1, 64, 64)) == MIS and store(L, ks=st(5120, -64, 64)) == BAD
    assert store(L, k=K) == BAD and store(L, v=0xB0000000) == BAD and store(L, c=kv8c(v=K)) == BAD
    assert store(L, starts=K) == BAD


def norm(L, x=Q, w=V, b=MASK, y=O, dtype=0, wdtype=0, B=2, N=10, C=64, G=8, xs=(640, 64), ys=(640, 64), eps=1e-5,
         act=0, ws=WS, nb=1 << 20):
    return L.npa_group_norm_act(x, w, b, y, dtype, wdtype, B, N, C, G, *xs, *ys, eps, act, ws, nb, None)


def test_group_norm_refusals(L):
    assert norm(L, x=None) == BAD and norm(L, y=None) == BAD
    for name in ("B", "N", "C", "G"):
        assert norm(L, **{name: 0}) == BAD
    assert norm(L, G=7) == BAD and norm(L, eps=-1.0) == BAD and norm(L, eps=float("nan")) == BAD
    assert norm(L, act=2) == BAD and norm(L, act=-1) == BAD
    assert norm(L, dtype=3) == UNS and norm(L, dtype=1, wdtype=0) == UNS and norm(L, wdtype=1) == UNS
    assert norm(L, C=8192, G=8, xs=(81920, 8192), ys=(81920, 8192)) == UNS and norm(L, B=70000) == UNS
    assert norm(L, xs=(640, 32)) == BAD and norm(L, ys=(640, 32)) == BAD and norm(L, ys=(100, 64)) == BAD
    assert norm(L, ys=(0, 64)) == BAD and norm(L, xs=(-1, 64)) == BAD and norm(L, xs=(1 << 41, 64)) == UNS
    assert norm(L, x=Q + 1) == MIS and norm(L, ws=WS + 4) == MIS and norm(L, w=V + 1) == MIS
    assert norm(L, wdtype=2, b=MASK + 2) == MIS
    assert norm(L, y=Q + 128) == BAD and norm(L, y=Q, ys=(1280, 128)) == BAD and norm(L, w=O) == BAD
    assert L.npa_group_norm_workspace_size(0, 2, 10, 64, 7) == 0 and L.npa_group_norm_workspace_size(5, 2, 10, 64, 8) == 0


def test_helpers_refuse(L):
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    q, k = t(2, 4, 8, 64), t(2, 4, 9, 64)
    with pytest.raises(ValueError):      # not on a GPU
        npa.cross_attention(q, k, k)
    with pytest.raises(ValueError):
        npa.cross_attention(q[0], k, k)
    with pytest.raises(ValueError):
        npa.cross_attention(q, t(2, 4, 9, 128), k)
    with pytest.raises(ValueError):
        npa.cross_attention(q, k, t(2, 4, 8, 64))
    with pytest.raises(ValueError):
        npa.cross_attention(q.float(), k, k)
    with pytest.raises(ValueError):
        npa.cross_attention(q.transpose(2, 3), k, k)
    with pytest.raises(ValueError):
        npa.cross_attention(q, k, k, kv_lens=torch.zeros(2))
    with pytest.raises(ValueError):
        npa.cross_attention(q, k, k, kv_lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        npa.cross_attention(q, k, k, key_mask=torch.zeros(2, 8, dtype=torch.bool))
    with pytest.raises(ValueError):
        npa.cross_attention(q, k, k, key_mask=torch.zeros(2, 9))
    with pytest.raises(ValueError):
        npa.Kv8Cache(t(2, 4, 100, 64, dt=torch.uint8), t(2, 4, 100, 64, dt=torch.uint8), torch.ones(2, 4, 2),
                     torch.ones(2, 4, 2))
    with pytest.raises(ValueError):
        npa.Kv8Cache(t(2, 4, 128, 64, dt=torch.uint8), t(2, 4, 128, 64, dt=torch.uint8), torch.ones(2, 4, 1),
                     torch.ones(2, 4, 2))
    with pytest.raises(ValueError):
        npa.group_norm(t(2, 3, 64), 8)
    with pytest.raises(ValueError):
        npa.group_norm(t(2, 3, 64), 8, act="relu")
    with pytest.raises(ValueError):
        npa.group_norm(t(2, 3, 64), 8, weight=torch.zeros(63))
    with pytest.raises(ValueError):
        npa.group_norm(t(2, 3, 64), 8, weight=torch.zeros(64, dtype=torch.float16))


def test_helpers_refuse_numbers_that_the_c_call_would_change():
    """ctypes drops an int's upper bits, and a float32 0 would mean the default scale."""
    assert npa._scale(None) == 0 and npa._scale(0.125) == 0.125
    for bad in (0, -1.0, float("nan"), float("inf"), 1e39, 1e-60):
        with pytest.raises(ValueError):
            npa._scale(bad)
    assert npa._int32("n", 2 ** 31 - 1) == 2 ** 31 - 1
    for bad in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            npa._int32("n", bad)
    shape, strides = (2, 4, 8, 64), (2048, 512, 64, 1)
    for n in (2 ** 32 + 5, 2 ** 32):
        with pytest.raises(ValueError):
            npa._kv8_plan(0, False, shape, strides, (2, 4, 128, 64), n, torch.bfloat16)
        with pytest.raises(ValueError):   # a head axis of stride 0
            npa._kv8_plan(0, False, (2, n, 1, 64), (64, 0, 64, 1), (2, 4, 128, 64), None, torch.bfloat16)
        with pytest.raises(ValueError):
            npa._cross_plan(-1, False, shape, strides, (2, n, 8, 64), (512, 0, 64, 1), (2, n, 8, 64), (512, 0, 64, 1),
                            *[torch.bfloat16] * 3)
        with pytest.raises(ValueError):
            npa._norm_plan(-1, 32 + n, None, (2, 3, 64), (192, 64, 1), torch.bfloat16, *[None] * 6)
    with pytest.raises(TypeError):
        npa._kv8_plan(0, False, shape, strides, (2, 4, 128, 64), 2.5, torch.bfloat16)


def test_helpers_refuse_a_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    class Stream:
        cuda_stream, device_index = 0, 1
    with pytest.raises(ValueError, match="stream of device 1"):
        npa._run_on(0, Stream(), lambda handle: None)


def test_cache_tensors_stay(L):
    """The tensors that were checked are the ones that a call gets."""
    c = object.__new__(npa.Kv8Cache)
    with pytest.raises(AttributeError):
        c.k = torch.zeros(1)
    with pytest.raises(AttributeError):
        c.k_scale = torch.zeros(1)


# ---------------------------------------------------------------------------
# The oracle's pins
# ---------------------------------------------------------------------------

def test_oracle_cross_attention_is_softmax_attention():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((2, 4, 5, 8)), rng.standard_normal((2, 2, 7, 8)), rng.standard_normal((2, 2, 7, 8))
    keep = rng.random((2, 7)) < 0.6
    keep[1] = False
    keep[1, 3] = True
    got, mag = oracle.cross_attention(q, k, v, keep=keep)
    T = torch.from_numpy
    want = torch.nn.functional.scaled_dot_product_attention(
        T(q), T(k).repeat_interleave(2, 1), T(v).repeat_interleave(2, 1), attn_mask=T(keep)[:, None, None, :])
    np.testing.assert_allclose(got, want.numpy(), rtol=0, atol=1e-12)
    np.testing.assert_allclose(got[1], np.repeat(v[1, :, 3], 2, 0)[:, None].repeat(5, 1), rtol=0, atol=1e-15)
    assert (mag >= np.abs(got) - 1e-15).all()
    none, _ = oracle.cross_attention(q, k, v, keep=np.zeros((2, 7), bool))
    assert not none.any()


def test_oracle_e4m3_rounds_like_the_type():
    x = np.concatenate([np.linspace(-460, 460, 20011), np.linspace(-0.05, 0.05, 20011), 2.0 ** np.arange(-14, 9),
                        [0.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(oracle.e4m3_round(x), want)
    assert oracle.e4m3_round(1e9) == 448 and oracle.e4m3_round(-np.inf) == -448 and np.isnan(oracle.e4m3_round(np.nan))


@pytest.mark.parametrize("amax,s", [(0.0, 1.0), (448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (225.0, 1.0),
                                    (2.0 ** -130, 2.0 ** -126), (3e38, 2.0 ** 120)])
def test_oracle_scale(amax, s):
    assert oracle.kv8_scale(amax) == s


def test_oracle_store_by_hand():
    """A block of 4: tokens 3, 1 at scale 1/128 (3 / 448 < 1/128), then 100 appended."""
    c, s = np.zeros((1, 8, 1)), np.ones((1, 2))
    oracle.kv8_store(c, s, np.array([[[3.0], [1.0]]]), 0, block=4)
    assert s[0, 0] == 2.0 ** -7 and c[0, :2, 0].tolist() == [384.0, 128.0]
    oracle.kv8_store(c, s, np.array([[[100.0], [-5.0], [7.0]]]), 2, block=4)
    assert s[0, 0] == 0.25 and c[0, :4, 0].tolist() == [12.0, 4.0, 384.0, -20.0]     # 400 ties to 384
    assert s[0, 1] == 2.0 ** -6 and c[0, 4, 0] == 448.0


def test_oracle_group_norm_matches_torch():
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((2, 9, 12)) + 3, rng.standard_normal(12), rng.standard_normal(12)
    T = torch.from_numpy
    want = torch.nn.functional.group_norm(T(x).transpose(1, 2), 4, T(w), T(b), 1e-5).transpose(1, 2)
    got, _, _ = oracle.group_norm(x, 4, w, b)
    np.testing.assert_allclose(got, want.numpy(), rtol=0, atol=1e-12)
    got, _, _ = oracle.group_norm(x, 4, w, b, act="silu")
    np.testing.assert_allclose(got, torch.nn.functional.silu(want).numpy(), rtol=0, atol=1e-12)
