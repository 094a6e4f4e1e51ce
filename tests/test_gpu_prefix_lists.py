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


# groups without sequences that are malformed: offsets of prefixes that decrease or leave the tensor, groups that decrease, a
# prefix longer than its bound; few groups and many
EMPTY = [
    ([0, 1, 1, 2], [0, 10, 5, 20], 0, -10),
    ([0, 1, 1, 2], [0, 10, 31, 20], 0, -10),
    ([0, 2, 1, 2], [0, 10, 10, 20], 0, -10),
    ([0, 1, 1, 2], [0, 5, 20, 30], 10, -11),
    ([0, 1, 2, 2], [0, 10, 20, 31], 0, -10),
    ([0, 0, 1, 2], [-4, 0, 10, 20], 0, -10),
    ([0, 1] + [1] * 38 + [2], [0, 10] + [15, 12] * 19 + [20], 0, -10),
    ([0] * 30 + [1] * 10 + [2], [0] * 29 + [10] * 5 + [25] * 7, 10, -11),
]


# few rows; a list of sequences; groups apart from their sequences with many rows and with few
@pytest.mark.parametrize("ql,heads,rows", [([4, 4], 1, 30), ([600, 600], 2, 30), ([40] * 2, 16, 30), ([1, 1], 2, 30000)])
@pytest.mark.parametrize("cg,cp,mp,code", EMPTY)
def test_bad_groups_without_sequences_are_reported(ql, heads, rows, cg, cp, mp, code):
    T = sum(ql)
    q = torch.randn(T, heads, 64, device="cuda").bfloat16()
    k, kp = (torch.randn(n, heads, 64, device="cuda").bfloat16() for n in (T, rows))
    grow = rows // 30                                      # the offsets of thirty rows, in a prefix of `rows`
    guard = torch.full((T + 16, heads, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    status = vit.new_status()
    cp = [x * grow if x >= 0 else x for x in cp]
    call = lambda g, p, m: vit.prefix_attn(q, kp, kp, k, k, offsets(ql), ints(p), offsets(ql), ints(g), max(ql), m * grow,
                                           max(ql), out=guard[8:8 + T], status=status)
    call(cg, cp, mp)
    assert vit.read_status(status) == code
    assert (guard[:8] == 5).all() and (guard[8 + T:] == 5).all()
    status.zero_()
    call([0] * (len(cg) - 2) + [1, 2], [0] * (len(cg) - 2) + [5 * grow, 30 * grow], 0)   # empty groups that are sound
    assert vit.read_status(status) == 0
    check(guard[8:8 + T], None, reference(q, k, k, offsets(ql), offsets(ql),
                                          prefix=[(kp, kp, 0, 5 * grow), (kp, kp, 5 * grow, 30 * grow)]))
