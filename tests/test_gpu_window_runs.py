"""Gradient of windowed attention over long texts with first tokens: the loops over all queries of the key tiles that
hold first tokens are cut into runs, whose sums are added up. Against the definition in 64 bits, with the tolerances of
test_gpu_window_attn_bwd: the runs' fp32 sums and their sum round by 2^-24 of the partial sums, far below the 2^-8 of
P and dS there."""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from test_gpu_window_attn_bwd import check, grads, reference

pytestmark = pytest.mark.gpu

CASES = [
    ([2500], [2500], 8, 1, 64, 64, 4),
    ([2500, 40], [2600, 40], 4, 4, 128, 100, 150),
    ([1900, 0, 900], [1900, 33, 1000], 6, 2, 80, 1, 1),
    ([2100, 1, 1030], [2100, 700, 1000], 3, 3, 96, 20, 129),
    ([3001], [3007], 16, 1, 32, 7, 16),
    ([2048, 2047, 2049], [2048, 2047, 2049], 5, 1, 128, 64, 1),
]


def joined(call):
    vit.kernel_timing(True)
    r = call()
    torch.cuda.synchronize()
    names = vit.kernel_timing_read()
    vit.kernel_timing(False)
    return r, "window_grad_join" in names


@pytest.mark.parametrize("ql,kl,Hq,Hk,D,window,sinks", CASES)
def test_cut_loops(ql, kl, Hq, Hk, D, window, sinks):
    q, k, v, do, cq, ck, mask = grads(ql, kl, Hq, Hk, D, window, sinks)
    out, lse = vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), *mask, return_lse=True)
    status = vit.new_status()
    got, cut = joined(lambda: vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), *mask, status=status))
    assert cut and vit.read_status(status) == 0
    check(got, reference(q, k, v, do, cq, ck, None, window, sinks))
    for sizes in ((max(ql), max(kl)), (None, None), (2 * max(ql), max(kl) + 5)):   # neither order nor bounds change it
        again = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, *sizes, *mask)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_short_calls_take_no_join():
    for window, sinks in ((0, 0), (64, 0), (256, 4)):
        q, k, v, do, cq, ck, mask = grads([400, 300], [400, 300], 4, 2, 64, window, sinks)
        out, lse = vit.window_attn(q, k, v, cq, ck, 400, 400, *mask, return_lse=True)
        _, cut = joined(lambda: vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, 400, 400, *mask))
        assert not cut


def test_padded_cache_strided_outputs_and_graph():
    """Keys with padding (NaN) behind each sequence, dk and dv inside wider rows, and the call in a graph whose inputs
    change between replays."""
    ql, lens, S, Hq, Hk, D, window, sinks = [1500, 1400], [1520, 1400], 1600, 4, 2, 64, 32, 130
    q, k, v, do, cq, ck, mask = grads(ql, [S, S], Hq, Hk, D, window, sinks)
    k_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        k[b * S + n:(b + 1) * S] = float("nan")
        v[b * S + n:(b + 1) * S] = float("nan")
    wide = [torch.full((2 * S, Hk + 1, D), 7.0, device="cuda").bfloat16() for _ in range(2)]
    dq, dk, dv = torch.empty_like(q), wide[0][:, :Hk], wide[1][:, :Hk]

    def call():
        out, lse = vit.window_attn(q, k, v, cq, ck, max(ql), S, *mask, k_len=k_len, return_lse=True)
        vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), S, *mask, k_len=k_len, dq=dq, dk=dk, dv=dv)

    own = torch.cat([torch.arange(S, device="cuda") < n for n in lens])

    def right(rest):
        for w in wide:
            assert (w[:, Hk] == 7).all() and (w[~own, :Hk] == rest).all()
        ref, tol = reference(q, k, v, do, cq, ck, k_len, window, sinks)
        check((dq, dk[own], dv[own]), ([ref[0], ref[1][own], ref[2][own]], [tol[0], tol[1][own], tol[2][own]]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
        torch.cuda.synchronize()
        right(7)
        with torch.cuda.graph(graph, stream=side):
            call()
    do.mul_(-0.5)
    for w in wide:
        w[:, :Hk] = 3
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    right(3)
