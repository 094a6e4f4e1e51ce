"""Integers past 32 bits at the Python binding, on the CPU: a window, a count of first tokens or a bound larger than any
tensor is what it says and not its low 32 bits, and sizes that no call takes stay refused."""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from vision_encoder_varlen_gb300 import _build

MOST = 2 ** 31 - 1
PAST = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 64 + 5, 10 ** 30]


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()


@pytest.mark.parametrize("big", PAST)
def test_windows_and_first_tokens(big):
    assert vit._window(big, 4) == (MOST, 4)
    assert vit._window(5, big) == (5, MOST)
    assert vit._window(None, -big)[1] < 0                      # the library refuses those
    for w in (-big, 0, -1):
        with pytest.raises(ValueError, match="at least 1"):
            vit._window(w, 0)


def test_whole_numbers():
    assert vit._window(7.0, 2) == vit._window(torch.tensor(7), torch.tensor(2)) == (7, 2)
    for w, s in ((2.7, 0), (5, 0.5), (float("nan"), 0)):
        with pytest.raises(ValueError):
            vit._window(w, s)
    with pytest.raises((ValueError, OverflowError)):
        vit._window(float("inf"), 0)


@pytest.mark.parametrize("big", PAST)
def test_sizes(big):
    f, g, h = vit.window_attn_workspace_size, vit.window_attn_bwd_workspace_size, vit.prefix_attn_workspace_size
    for size, Tq, most in ((f, 3, 1), (g, 5000, 5000)):
        of = lambda *a: size(Tq, 40000, 8, 2, 64, 3, *a)
        assert of(most, 40000, big, 4) == of(most, 40000) != of(most, 40000, 5, 4)
        assert of(most, 40000, 30, big) == of(most, 40000, 30, 40000)
        assert of(most, 40000, -big) == 0
        assert of(big, big) == of()
        assert size(50, 400, big, 2, 64, 3) == size(50, 400, 8, 2, 64, big) == 0
    assert h(50, 9000, 400, 8, 2, 64, 30, 1, big, big, big) == h(50, 9000, 400, 8, 2, 64, 30, 1) > 0
    assert h(50, 9000, 400, 8, 2, 64, 30, big) == 0
    assert vit.cross_attn_workspace_size(50, 9000, 8, 2, 64, 3, big, big) == vit.cross_attn_workspace_size(50, 9000, 8, 2, 64, 3)
    assert vit.cross_attn_bwd_workspace_size(50, 9000, 8, 2, 64, 3, big) == vit.cross_attn_bwd_workspace_size(50, 9000, 8, 2, 64, 3)
    assert vit.workspace_size(50, big, 1, 64) == vit.workspace_size(50, 8, big, 64) == 0
    assert vit._max_seqlen(big) == MOST


@pytest.mark.gpu
@pytest.mark.parametrize("big", PAST)
def test_calls(big):
    """The result of a call whose window, first tokens and bounds are larger than anything is that of one without."""
    from test_gpu_window_attn import make
    q, k, v, cq, ck, _ = make([40, 3], [90, 60], 4, 2, 64)
    out, lse = vit.window_attn(q, k, v, cq, ck, return_lse=True)
    for args in ((big, big, big, 0), (None, None, 5, big), (big, big, None, 0)):
        a, b = vit.window_attn(q, k, v, cq, ck, *args, return_lse=True)
        assert args[2] == 5 or (torch.equal(a, out) and torch.equal(b, lse))
        assert torch.allclose(b, lse, atol=1e-4)               # (all keys of the past are first tokens: the same sums)
    do = torch.randn_like(q)
    want = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck)
    got = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, big, big, big, 0)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    want = vit.prefix_attn(q, k, v, k, v, cq, ck[[0, 2]].contiguous(), ck)
    assert torch.equal(want, vit.prefix_attn(q, k, v, k, v, cq, ck[[0, 2]].contiguous(), ck, None, big, big, big))
