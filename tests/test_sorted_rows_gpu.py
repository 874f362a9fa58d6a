"""Batch rows of differing lengths beyond the number of blocks from which units
run in the order of the lengths, at both head dimensions and over the cache."""
import numpy as np
import pytest

import oracle
from _block import check_attention, f64, randn

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


@pytest.mark.parametrize("d,heads,Lq,Lk", [(64, 10, 2048, 1600), (128, 10, 1930, 4200)])
@pytest.mark.parametrize("cached", [False, True])
def test_longest_first_row(npa, d, heads, Lq, Lk, cached):
    """Rows given longest first, so that every unit runs at another place than it stands."""
    B = 2
    lens = np.array([Lk, Lk // 3 + 5])
    keep = np.arange(Lk) < lens[:, None]
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = randn(1, B, heads, Lq, d), randn(2, B, heads, Lk, d), randn(3, B, heads, Lk, d)
    if cached:
        cache = npa.Kv8Cache.empty(B, heads, Lk, d)
        npa.kv8_store(cache, k, v)
        out = npa.kv8_cross_attention(q, cache, Lk, kv_lens=kv_lens)
        k, v = ((c.float() * s.repeat_interleave(64, 2)[..., None])[:, :, :Lk]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    else:
        out = npa.cross_attention(q, k, v, kv_lens=kv_lens)
    heads_looked_at = [0, heads - 1]
    ref, mag = oracle.cross_attention(*(f64(x[:, heads_looked_at]) for x in (q, k, v)), keep=keep)
    check_attention(f64(out[:, heads_looked_at]), ref, mag, "bf16", Lk, float(v.abs().max()), kv8=cached)
