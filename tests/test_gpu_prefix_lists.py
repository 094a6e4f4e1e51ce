"""Attention behind shared prefixes where a side of a call holds nothing, or its lists are malformed where no sequence is.
Tolerances are those of test_gpu_window_attn."""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from test_gpu_window_attn import check, make, offsets, reference

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,Hk,m", [(64, 8, 1), (20, 8, 1), (200, 1, 2), (18, 8, 1)])   # 152 pairs of sequence and key head or more; fewer
def test_no_own_keys_behind_a_prefix_read_apart(B, Hk, m):
    """No sequence has a key of its own: the prefixes are all that the queries see."""
    pl = [7000, 2001]
    q, k, v, cq, ck, _ = make([m] * B, [0] * B, 4 * Hk, Hk, 64)
    assert k.shape[0] == 0
    kp, vp = (make(pl, [1], Hk, Hk, 64, seed=s)[0] for s in (1, 2))
    cp, groups = offsets(pl), [B - 5, 5]
    of = [(kp, vp, 0, 7000)] * (B - 5) + [(kp, vp, 7000, 9001)] * 5
    status = vit.new_status()
    out, lse = vit.prefix_attn(q, kp, vp, k, v, cq, cp, ck, offsets(groups), m, 7000, 1, return_lse=True, status=status)
    assert vit.read_status(status) == 0
    check(out, lse, reference(q, k, v, cq, ck, prefix=of))
