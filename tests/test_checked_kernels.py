"""The bounds-checking build checks every kernel that writes an output."""
import glob
import os
import re

import pytest

from _block import bits, randn

torch = pytest.importorskip("torch")
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "patch_res_diffusion_b200", "csrc")

# one row to a thread or warp, compared with the row count in every build
ROW_GUARDED = {"asg_combine.cuh", "md_combine.cuh"}


def test_every_kernel_file_has_checks():
    files = [f for f in glob.glob(os.path.join(CSRC, "*.cuh")) if "__global__" in open(f).read()]
    assert len(files) >= 8
    for f in files:
        if os.path.basename(f) not in ROW_GUARDED:
            assert re.search(r"\bbound_(row|coord)\(", open(f).read()), f


@pytest.fixture(scope="module")
def npa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from patch_res_diffusion_b200 import build
    build.build()
    import patch_res_diffusion_b200 as m
    m.use_bounds_checking(True)
    try:
        yield m
    finally:
        m.use_bounds_checking(False)


def both(npa, run):
    """The checked build's result, found without a failed check, is the normal one's."""
    got = run()
    torch.cuda.synchronize()
    assert npa.npa_device_status() == npa.NPA_OK
    npa.use_bounds_checking(False)
    want = run()
    torch.cuda.synchronize()
    assert npa.npa_device_status() == npa.NPA_OK
    npa.use_bounds_checking(True)
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,N,C,groups", [(2, 100, 320, 32), (1, 3, 24, 3), (1, 40000, 64, 4), (2, 33, 33, 11), (1, 70, 2056, 8)])
def test_group_norm(npa, dtype, B, N, C, groups):
    x = randn(1, B, N, C, dtype=dtype)
    both(npa, lambda: [npa.group_norm(x, groups, act="silu")])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("starts,n", [([0, 0], 192), ([5, 127], 1), ([-20, 150], 60), ([191, 500], 3)])
def test_store(npa, d, starts, n):
    k, v = randn(2, 2, 3, n, d), randn(3, 2, 3, n, d)

    def run():
        cache = npa.Kv8Cache.empty(2, 3, 192, d)
        npa.kv8_store(cache, k, v, starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        return [cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale]
    both(npa, run)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (3, 33), (16, 700), (1, 9000)])
def test_few_rows(npa, d, Lq, Lk):
    q, k, v = randn(4, 2, 4, Lq, d), randn(5, 2, 4, Lk, d), randn(6, 2, 4, Lk, d)
    lens = torch.tensor([Lk, Lk // 2], dtype=torch.int32, device="cuda")
    both(npa, lambda: [npa.cross_attention(q, k, v), npa.cross_attention(q, k, v, kv_lens=lens)])
