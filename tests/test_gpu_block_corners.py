"""Corner calls of the operators around a language model's reading of the encoder's states: no rows, no sequences,
sequences without states beside others, lists that are wrong in one place, infinities.

Expected values are exact (zeros, untouched rows, the same bits as another call) or from the formulas in 64 bits with
the bounds that stand beside them.
"""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit

pytestmark = pytest.mark.gpu

BF16 = dict(dtype=torch.bfloat16, device="cuda")


# ------------------------------------------------------------------ residual step

@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("C", [256, 520, 1280, 6144, 8192])
@pytest.mark.parametrize("post,pre,gate", [(True, False, False), (False, False, True), (True, True, True),
                                           (True, False, True), (False, True, False)])
def test_residual_gradient_of_no_rows(C, post, pre, gate, wide):
    """The sums over no tokens are 0, whichever of the inputs are there."""
    w = torch.ones(C, **BF16)
    dh = torch.empty(0, C, device="cuda", dtype=torch.float32 if wide else torch.bfloat16)
    none = torch.empty(0, C, **BF16)
    dx, dy, dgate, dw_post, dw_pre = vit.norm_residual_bwd(
        none if pre else None, dh, dh if pre else None, none, gate=w if gate else None, w_post=w if post else None,
        w_pre=w if pre else None)
    assert dx.shape == dy.shape == (0, C)
    for asked, s in ((gate, dgate), (post, dw_post), (pre, dw_pre)):
        assert (s is not None) == asked
        if asked:
            assert s.shape == (C,) and not s.any()


# ------------------------------------------------------------------ cross attention

@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("Tq,Tk", [(37, 210), (37, 0), (0, 210)])
def test_gradient_of_no_sequences(Tq, Tk, side):
    """All rows are rows of no sequence: 0 in new tensors, as they were in given ones."""
    q, k = torch.randn(Tq, 4, 64, device="cuda").bfloat16(), torch.randn(Tk, 2, 64, device="cuda").bfloat16()
    lse = torch.zeros(Tq, 4, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for t in [torch.full_like(x, float("nan")) for x in (q, k, k) for _ in range(4)]:
            del t                                             # what the allocator hands out next is not 0
    got = vit.cross_attn_bwd(q, q, k, k, q, lse, cu, cu, stream=stream)
    torch.cuda.synchronize()
    for t, like in zip(got, (q, k, k)):
        assert t.shape == like.shape and not t.any()
    given = [torch.full_like(x, 7) for x in (q, k, k)]
    vit.cross_attn_bwd(q, q, k, k, q, lse, cu, cu, dq=given[0], dk=given[1], dv=given[2], stream=stream)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in given)


def _lists(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device="cuda")


def test_gradients_back_to_back_on_one_workspace():
    """Calls of different lengths that follow one another on one workspace, captured in one graph and replayed
    without a pause, give the bits of separate calls: none reads the lists or statistics of another."""
    g = torch.Generator(device="cuda").manual_seed(5)
    Hq, Hk, D = 8, 2, 64
    calls = []
    for ql, kl in (([300, 1, 77], [900, 40, 333]), ([5, 200], [64, 1500]), ([1] * 40, [1] * 40), ([513], [2049])):
        n = lambda T, H: torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
        q, do, k, v = n(sum(ql), Hq), n(sum(ql), Hq), n(sum(kl), Hk), n(sum(kl), Hk)
        cq, ck = _lists(ql), _lists(kl)
        out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True)
        ref = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl))
        got = [torch.empty_like(t) for t in (q, k, v)]
        calls.append(((do, q, k, v, out, lse, cq, ck, max(ql), max(kl)), ref, got))
    size = max(vit.cross_attn_bwd_workspace_size(a[1].shape[0], a[2].shape[0], Hq, Hk, D, a[6].numel() - 1, a[8], a[9])
               for a, _, _ in calls)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run():
        for a, _, (dq, dk, dv) in calls:
            vit.cross_attn_bwd(*a, dq=dq, dk=dk, dv=dv, workspace=ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(30):
        for _, _, got in calls:
            for t in got:
                t.zero_()
        for _ in range(4):
            graph.replay()
        for _, ref, got in calls:
            for x, y in zip(got, ref):
                assert torch.equal(x, y)
