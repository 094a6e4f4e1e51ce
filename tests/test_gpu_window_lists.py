"""Offsets that decrease between sequences behind a shared prefix whose own keys are read apart from it."""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# the rows of a sequence in the middle lie among, before and behind those of its group
@pytest.mark.parametrize("at,to", [(11, 9), (11, 0), (11, 50)])
def test_rows_outside_a_group(at, to):
    B, Hq, Hk, D, P = 48, 8, 2, 128, 8000
    cq = list(range(at)) + list(range(to, to + B - at)) + [B]     # one row each, but for the step at `at`
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(128, Hq, D, generator=g, device="cuda").bfloat16()
    k, kp = (torch.randn(n, Hk, D, generator=g, device="cuda").bfloat16() for n in (B, P))
    guard = torch.full((160, Hq, D), 5.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((128, Hq), 5.0, device="cuda")
    status = vit.new_status()
    vit.prefix_attn(q, kp, kp, k, k, ints(cq), ints([0, P // 2, P]), ints(range(B + 1)), ints([0, 5, B]), 1, P, 1,
                    out=guard[16:144], lse=lse, status=status)
    assert vit.read_status(status) in (-10, -11)
    assert (guard == 5).all() and (lse == 5).all()
    status = vit.new_status()
    vit.prefix_attn(q, kp, kp, k, k, ints(range(B + 1)), ints([0, P // 2, P]), ints(range(B + 1)), ints([0, 5, B]), 1, P,
                    1, out=guard[16:144], lse=lse, status=status)
    assert vit.read_status(status) == 0 and (guard[:16] == 5).all() and (guard[16 + B:] == 5).all()
    assert torch.isfinite(guard).all() and (lse[:B] > 5).all()
