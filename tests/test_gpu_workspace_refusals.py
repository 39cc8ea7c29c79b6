"""A workspace that the kernels could not write, or whose bytes are not the ones its size says, is refused
before anything is launched."""
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
BAD = {
    "host": lambda: torch.empty(1 << 22, dtype=torch.uint8),
    "expanded": lambda: torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 22),
    "strided": lambda: torch.empty(1 << 22, 2, dtype=torch.uint8, device="cuda")[:, 0],
}


@pytest.mark.parametrize("kind", BAD)
def test_refused(kind):
    ws = BAD[kind]()
    x, w = torch.zeros(8, 33, dtype=torch.bfloat16, device="cuda"), torch.zeros(16, 33, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(8, 15, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(300, 400, device="cuda")
    calls = (lambda: zc.linear(x, w, workspace=ws), lambda: zc.linear_dgrad(x, w.T.contiguous(), workspace=ws),
             lambda: zc.linear_wgrad(dy, x, torch.zeros(15, 33, device="cuda"), workspace=ws),
             lambda: zc.newton_schulz(g, workspace=ws), lambda: zc.muon_step([g.clone()], [g.clone()], [g], lr=0.1, workspace=ws))
    for call in calls:
        with pytest.raises(ValueError, match="workspace"):
            call()
    assert zc.device_status() == 0


def test_any_type_of_elements():
    x, w = torch.ones(8, 33, dtype=torch.bfloat16, device="cuda"), torch.ones(16, 33, dtype=torch.bfloat16, device="cuda")
    for dtype in (torch.uint8, torch.float32, torch.int64):
        y = zc.linear(x, w, workspace=torch.empty(1 << 12, 2, dtype=dtype, device="cuda"))
        assert bool((y == 33).all())
