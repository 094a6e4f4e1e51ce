"""Gradient of windowed attention where a query sees one key: its weight is 1 whatever the score, so it gets no dq and gives no
dk. The first token of every text is such a row, and every row of a window of one without first tokens. Exactly 0, where a
difference of two fp32 sums would leave their rounding."""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from test_gpu_window_attn_bwd import check, grads, reference

pytestmark = pytest.mark.gpu


def run(ql, kl, Hq, Hk, D, window, sinks):
    q, k, v, do, cq, ck, mask = grads(ql, kl, Hq, Hk, D, window, sinks)
    out, lse = vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), *mask, return_lse=True)
    got = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), *mask)
    check(got, reference(q, k, v, do, cq, ck, None, window, sinks))
    return got, cq.tolist(), ck.tolist(), do


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3), (1, 1), (2, 0)])
@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 32), (8, 1, 128), (6, 3, 80), (4, 2, 64), (3, 3, 96)])
def test_first_tokens(Hq, Hk, D, window, sinks):
    """Texts of one token, of several and of many; more queries than keys; one key before a long continuation."""
    ql, kl = [1, 40, 1, 300, 7, 1, 130, 5], [1, 40, 0, 300, 3, 1, 130, 900]
    (dq, dk, dv), cq, ck, do = run(ql, kl, Hq, Hk, D, window, sinks)
    for b, (m, n) in enumerate(zip(ql, kl)):
        first = cq[b] + m - n                                 # the row of the sequence's first key, where it is a query
        if cq[b] <= first < cq[b + 1]:
            assert not dq[first].any() and (m < 2 or n < 2 or dq[first + 1].any())
        if n == 1:
            assert not dk[ck[b]].any()
            assert torch.equal(dv[ck[b]], do[first].double().reshape(Hk, Hq // Hk, D).sum(1).bfloat16()) or Hq > Hk


@pytest.mark.parametrize("Hq,Hk,D", [(1, 1, 32), (8, 1, 128), (16, 16, 80), (5, 1, 64)])
def test_a_window_of_one(Hq, Hk, D):
    (dq, dk, dv), _, _, do = run([500, 1, 129], [500, 40, 129], Hq, Hk, D, 1, 0)
    assert not dq.any() and not dk.any() and dv.any()


def test_texts_of_one_token():
    (dq, dk, dv), _, _, do = run([1] * 300, [1] * 300, 4, 2, 64, 0, 0)
    assert not dq.any() and not dk.any()
