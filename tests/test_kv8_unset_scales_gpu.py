"""Tokens appended inside a block whose scale nobody has set (a cache allocated
as zeros), or that is smaller than the store ever writes."""
import numpy as np
import pytest

import oracle
from _block import f64, randn

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


@pytest.mark.parametrize("old", [0.0, 2.0 ** -149, 2.0 ** -130, 2.0 ** -126, 2.0 ** -40])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -133, 2.0 ** -60, 1.0])
@pytest.mark.parametrize("d", [64, 128])
def test_appended_to_an_unset_block(npa, old, size, d):
    B, h, cap, start, n = 2, 2, 192, 37, 40
    codes = torch.zeros(B, h, cap, d, dtype=torch.uint8, device="cuda")
    codes[:, :, ::3] = 0x35
    scales = torch.full((B, h, cap // 64), old)      # on the host, where small numbers stay
    tensors = [codes.view(torch.float8_e4m3fn), codes.clone().view(torch.float8_e4m3fn), scales.cuda(), scales.cuda()]
    cache = npa.Kv8Cache(*tensors)
    k, v = ((randn(i, B, h, n, d, device="cpu").double() * size).bfloat16().cuda() for i in (1, 2))
    want = [(t.cpu().to(torch.float64).numpy().copy(), f64(s).copy())
            for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    npa.kv8_store(cache, k, v, start=start)
    torch.cuda.synchronize()
    for (c, s), x, gc, gs in zip(want, (k, v), (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
        for b in range(B):
            oracle.kv8_store(c[b], s[b], f64(x)[b], start)
        np.testing.assert_array_equal(f64(gs), s)
        np.testing.assert_array_equal(gc.cpu().to(torch.float64).numpy(), c)
        assert (s[:, :, :2] >= 2.0 ** -126).all()
