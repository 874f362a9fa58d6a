"""The helpers' look-up by shape: a number given as a tensor counts by what it
holds at each call."""
import pytest

from _block import bits, randn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def npa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from patch_res_diffusion_b200 import build
    build.build()
    import patch_res_diffusion_b200 as m
    m.npa_device_ready()
    yield m
    assert m.npa_device_status() == m.NPA_OK


@pytest.mark.parametrize("Lq", [1, 40])
def test_token_count_in_a_tensor(npa, Lq):
    cache = npa.Kv8Cache.empty(1, 2, 256, 64)
    npa.kv8_store(cache, randn(1, 1, 2, 256, 64), randn(2, 1, 2, 256, 64))
    q = randn(3, 1, 2, Lq, 64)
    n = torch.tensor(30)
    for tokens in (30, 200, 7):
        n.fill_(tokens)
        assert torch.equal(bits(npa.kv8_cross_attention(q, cache, n)), bits(npa.kv8_cross_attention(q, cache, tokens)))
    with pytest.raises(TypeError):
        npa.kv8_cross_attention(q, cache, 30.0)      # 30 has been looked up before


def test_groups_in_a_tensor(npa):
    x = randn(4, 1, 50, 64)
    g = torch.tensor(8)
    for groups in (8, 16):
        g.fill_(groups)
        assert torch.equal(bits(npa.group_norm(x, g)), bits(npa.group_norm(x, groups)))
    with pytest.raises(TypeError):
        npa.group_norm(x, 8.0)
