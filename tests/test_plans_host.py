"""What the helpers look up again for a shape: nothing that was found out while
the device could not be asked."""
import pytest

import patch_res_diffusion_b200 as npa

torch = pytest.importorskip("torch")


class Library:
    """Answers as the library does whose device fails once, then is there."""

    def __init__(self, sizes):
        self.sizes, self.ready = list(sizes), [npa.NPA_ERR_CUDA]

    def npa_cross_attention_workspace_size(self, *args):
        return self.sizes.pop(0)

    npa_group_norm_workspace_size = npa_cross_attention_workspace_size

    def npa_device_ready(self):
        return self.ready.pop(0) if self.ready else npa.NPA_OK

    def npa_status_string(self, code):
        return b"error"


def cross(Lk):
    q, k = (2, 4, 8, 64), (2, 4, Lk, 64)
    return npa._cross_plan(0, True, q, (2048, 512, 64, 1), k, (4 * Lk * 64, Lk * 64, 64, 1), k,
                           (4 * Lk * 64, Lk * 64, 64, 1), *[torch.bfloat16] * 3)[3]


def kv8(Lk):
    return npa._kv8_plan(0, True, (2, 4, 8, 64), (2048, 512, 64, 1), (2, 4, 8192, 64), Lk, torch.bfloat16)[3]


def norm(N):
    return npa._norm_plan(0, 8, None, (2, N, 64), (64 * N, 64, 1), torch.bfloat16, *[None] * 6)[3]


@pytest.mark.parametrize("plan", [cross, kv8, norm])
def test_a_size_of_a_device_that_was_not_ready_is_not_kept(monkeypatch, plan):
    fake = Library([0, 4096])
    monkeypatch.setattr(npa, "lib", lambda: fake)
    with pytest.raises(npa.NpaError):
        plan(7001)
    assert plan(7001) == 4096
    assert plan(7001) == 4096 and not fake.sizes      # looked up
    fake.sizes, fake.ready = [0], []
    assert plan(7002) == 0 and plan(7002) == 0        # none needed


def test_device_ready_on_this_machine():
    from patch_res_diffusion_b200 import build
    build.build()
    if not torch.cuda.is_available():
        with pytest.raises(npa.NpaError):
            npa.npa_device_ready()
        with pytest.raises(npa.NpaError):
            npa.npa_device_ready()


def test_groups_are_looked_up_as_a_number(monkeypatch):
    seen = []
    monkeypatch.setattr(npa, "_norm_plan", lambda index, groups, *rest: seen.append(groups) or (None, None, None, 0))
    x = torch.zeros(1, 3, 64)
    for g in (8, torch.tensor(8)):
        with pytest.raises(ValueError):      # not on a GPU
            npa.group_norm(x, g)
    assert [type(g) for g in seen] == [int, int]
    with pytest.raises(TypeError):
        npa.group_norm(x, 8.0)
