"""SiLU behind the group norm over its whole range: with weights of 0 the value
in front of the activation is the bias itself, exactly."""
import numpy as np
import pytest

from _block import HALF_STEP, HALF_SUB, f64, randn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

Z = [-1e30, -3.0, -1e4, 2.0, -43.5, -42.9, 0.0, -87.0, 1e4, -88.5, -0.01, -95.0, -102.0, 50.0, -104.5, -60.0, -1e20, -20.0,
     -43.0, -1.0, -5e3, -149.0, 88.0]


@pytest.fixture(scope="module")
def npa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from patch_res_diffusion_b200 import build
    build.build()
    import patch_res_diffusion_b200 as m
    yield m
    assert m.npa_device_status() == m.NPA_OK


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N,C,groups", [(200, 320, 32), (40000, 64, 4), (200, 33, 11), (3, 8, 1)])
def test_silu_of_the_bias(npa, dtype, N, C, groups):
    """The exponent z log2(e) is off by 1.5 half steps, at most 150 x 1.5 x 2^-24,
    which is below 2^-16 of the result with all the roundings behind it; an
    exponential below 2^-126 is off by half of 2^-149, times z, and is 0 below
    2^-150; then one rounding."""
    z = np.float32([Z[(5 * i + i // len(Z)) % len(Z)] for i in range(C)]).astype(np.float64)
    x = randn(1, 1, N, C, dtype=dtype)
    out = npa.group_norm(x, groups, torch.zeros(C, device="cuda"), torch.from_numpy(z).float().cuda(), act="silu")
    with np.errstate(over="ignore"):
        y = z / (1 + np.exp(-z))
    bound = (2.0 ** -16 + HALF_STEP[dtype]) * np.abs(y) + np.minimum(np.abs(z), 150) * 2.0 ** -149 + HALF_SUB[dtype]
    over = np.abs(f64(out) - y) - bound
    assert (over <= 0).all(), [(z[c], f64(out)[0, n, c], y[c]) for _, n, c in np.argwhere(over > 0)[:5]]


@pytest.mark.parametrize("C", [64, 33])
def test_nan_stays_in_its_channel(npa, C):
    """A NaN bias next to channels far below and above 0."""
    bias = torch.full((C,), -50.0, device="cuda")
    bias[1::3] = float("nan")
    bias[2::3] = 3.0
    out = npa.group_norm(randn(2, 1, 100, C, dtype="fp32"), 1, torch.zeros(C, device="cuda"), bias, act="silu")
    assert torch.equal(torch.isnan(out), torch.isnan(bias).expand(1, 100, C))
