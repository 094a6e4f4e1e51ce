"""Gradient of cross attention against the definition in 64 bits, and against differences.

Tolerances, per element. P and dS are rounded to bf16 (2^-8 of each), o is bf16 (2^-8 of each of its
elements, so delta is off by 2^-8 sum_d |do_d o_d|), scores and dP are fp32 sums of D products
(below D 2^-24 of their magnitudes, relative errors of every p), exp2 is good to 2^-21, results are
rounded once (2^-8). With e = 2 score error + 2^-19:
  |dv err| <= 2^-8 |dv| + (2^-8 + e)(1 + 2^-8) sum p |do|
  |ds err| <= (2^-8 + e)(1 + 2^-8) p (|dP| + |delta| + m) + p 2^-8 sum |do o| =: w,  m = D 2^-24 sum |do v|
  |dq err| <= 2^-8 |dq| + scale sum_j w |k|, likewise dk.
"""
import math

import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from test_gpu_cross_attn import make, many

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def reference(q, k, v, do, cu_q, cu_k, k_len=None, scale=None):
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    G = Hq // Hk
    scale = 1 / math.sqrt(D) if scale is None else scale
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
    g, tol = [z(q), z(k), z(v)], [z(q), z(k), z(v)]
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cq) - 1):
        n = ck[b + 1] - ck[b] if k_len is None else int(k_len[b])
        rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b] + n)
        if n == 0 or cq[b + 1] == cq[b]:
            continue
        Q, DO = (t[rq].double().transpose(0, 1) for t in (q, do))
        K, V = (t[rk].double().transpose(0, 1).repeat_interleave(G, 0) for t in (k, v))
        T = lambda t: t.transpose(1, 2)
        s = Q @ T(K) * scale
        p = torch.softmax(s, -1)
        o = p @ V
        dp = DO @ T(V)
        delta = (DO * o).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        e = 2 * (Q.abs() @ T(K.abs())).amax() * scale * D * 2.0 ** -24 + 2.0 ** -19
        m = D * 2.0 ** -24 * (DO.abs() @ T(V.abs()))
        w = (BF + e) * (1 + BF) * p * (dp.abs() + delta.abs() + m) + p * BF * (DO * o).abs().sum(-1, keepdim=True)
        heads = lambda t: t.reshape(Hk, G, *t.shape[1:]).sum(1).transpose(0, 1)
        g[0][rq] = (scale * ds @ K).transpose(0, 1)
        tol[0][rq] = (scale * w @ K.abs()).transpose(0, 1)
        g[1][rk] = heads(scale * T(ds) @ Q)
        tol[1][rk] = heads(scale * T(w) @ Q.abs())
        g[2][rk] = heads(T(p) @ DO)
        tol[2][rk] = heads((BF + e) * (1 + BF) * T(p) @ DO.abs())
    return g, tol


def check(got, ref, what=""):
    for name, x, y, t in zip(("dq", "dk", "dv"), got, *ref):
        assert torch.isfinite(x).all(), what + name
        err = (x.double() - y).abs() - (BF * y.abs() + t + 2.0 ** -130)
        assert (err <= 0).all(), f"{what}{name}: {float(err.max()):.3e} past its bound"


CASES = [
    ([1], [1], 1, 1, 32),
    ([1, 3], [5, 40], 2, 1, 64),
    ([17], [16], 1, 1, 128),
    ([64, 65, 1, 0, 7], [63, 1, 700, 9, 0], 4, 2, 80),
    ([130, 1, 257, 31], [77, 1111, 0, 128], 8, 1, 128),
    ([300, 200], [113, 513], 6, 2, 96),
    ([1000], [999], 3, 3, 32),
    ([129, 600], [640, 3], 5, 1, 64),
    ([40] * 12, [100] * 12, 8, 2, 64),
    ([513], [2000], 16, 16, 80),
    ([2000, 3], [130, 900], 4, 1, 128),
]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", CASES)
def test_gradient(ql, kl, Hq, Hk, D):
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    g = torch.Generator(device="cuda").manual_seed(9)
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True)
    status = vit.new_status()
    got = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), status=status)
    assert vit.read_status(status) == 0
    check(got, reference(q, k, v, do, cq, ck))
    again = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("D", [64, 80, 128])
def test_padding_strides_and_untouched_rows(D):
    # NaN before, behind and (past k_len) between the sequences; views with their own strides; what belongs to no
    # sequence stays as it was
    ql, S, lens, Hq, Hk, gap = [33, 100, 1], 90, [90, 0, 37], 4, 2, 5
    q, _, _, cq, _ = make(ql, [1] * 3, Hq, Hk, D, gap=gap)
    g = torch.Generator(device="cuda").manual_seed(4)
    kv = torch.randn(3 * S + gap, 2, Hk, D, generator=g, device="cuda").bfloat16()
    for b, n in enumerate(lens):
        kv[b * S + n:(b + 1) * S] = math.nan
    kv[3 * S:] = math.inf
    k, v = kv[:, 0], kv[:, 1]
    ck = torch.arange(4, device="cuda", dtype=torch.int32) * S
    k_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    vit.cross_attn(q, k, v, cq, ck, max(ql), S, 0.2, k_len=k_len, out=out, lse=lse)
    do[:gap] = math.nan
    dq = torch.full_like(q, 7.0)
    dkv = torch.full_like(kv, 7.0)
    vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), S, 0.2, k_len=k_len, dq=dq, dk=dkv[:, 0], dv=dkv[:, 1])
    own_q = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    own_q[gap:gap + sum(ql)] = True
    own_k = torch.zeros(k.shape[0], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        own_k[b * S:b * S + n] = True
    assert (dq[~own_q] == 7).all() and (dkv[~own_k] == 7).all()
    ref, tol = reference(q, k, v, do, cq, ck, lens, 0.2)
    check((dq[own_q], dkv[:, 0][own_k], dkv[:, 1][own_k]),
          ([ref[0][own_q], ref[1][own_k], ref[2][own_k]], [tol[0][own_q], tol[1][own_k], tol[2][own_k]]))
    made = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), S, 0.2, k_len=k_len)
    assert (made[0][~own_q] == 0).all() and (made[1][~own_k] == 0).all() and (made[2][~own_k] == 0).all()
    assert torch.equal(made[0][own_q], dq[own_q])


def test_against_differences():
    ql, kl, Hq, Hk, D = [5, 70], [40, 90], 4, 2, 64
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    g = torch.Generator(device="cuda").manual_seed(11)
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    out, lse = vit.cross_attn(q, k, v, cq, ck, return_lse=True)
    got = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck)
    tol = reference(q, k, v, do, cq, ck)[1]

    def loss(q, k, v):
        total, a, b = 0.0, 0, 0
        for m, n in zip(ql, kl):
            Q, DO = q[a:a + m].transpose(0, 1), do[a:a + m].double().transpose(0, 1)
            K, V = (t[b:b + n].transpose(0, 1).repeat_interleave(Hq // Hk, 0) for t in (k, v))
            total += float((torch.softmax(Q @ K.transpose(1, 2) / math.sqrt(D), -1) @ V * DO).sum())
            a, b = a + m, b + n
        return total

    ins = [t.double() for t in (q, k, v)]
    for i in range(3):
        d = torch.randn(ins[i].shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        slope = (loss(*(t + e * d if j == i else t for j, t in enumerate(ins))) -
                 loss(*(t - e * d if j == i else t for j, t in enumerate(ins)))) / (2 * e)
        bound = float(((BF * got[i].double().abs() + tol[i]) * d.abs()).sum()) + 1e-4
        assert abs(slope - float((got[i].double() * d).sum())) <= bound


def test_one_side_empty():
    z = dict(device="cuda", dtype=torch.bfloat16)
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q, k = torch.randn(70, 4, 64, device="cuda").bfloat16(), torch.randn(150, 2, 64, device="cuda").bfloat16()
    none_q, none_k = torch.empty(0, 4, 64, **z), torch.empty(0, 2, 64, **z)
    out, lse = vit.cross_attn(q, none_k, none_k, cu(0, 70), cu(0, 0), return_lse=True)
    dq, dk, dv = vit.cross_attn_bwd(q, q, none_k, none_k, out, lse, cu(0, 70), cu(0, 0))
    assert (dq == 0).all() and dk.shape == dv.shape == (0, 2, 64)
    buf = torch.full_like(k, 3.0), torch.full_like(k, 3.0)
    vit.cross_attn_bwd(none_q, none_q, k, k, none_q, torch.empty(0, 4, device="cuda"), cu(0, 0), cu(0, 150),
                       dq=torch.empty_like(none_q), dk=buf[0], dv=buf[1])
    assert (buf[0] == 0).all() and (buf[1] == 0).all()


def test_bad_offsets_leave_outputs():
    q, k = torch.randn(8, 4, 64, device="cuda").bfloat16(), torch.randn(30, 4, 64, device="cuda").bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(8, 4, device="cuda")
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for cq, ck in ((t(0, 5, 3), t(0, 10, 20)), (t(0, 4, 8), t(0, 20, 10)), (t(0, 4, 9), t(0, 10, 31))):
        status = vit.new_status()
        outs = [torch.full((24, 4, 64), 5.0, device="cuda", dtype=torch.bfloat16)[8:16]] + [
            torch.full((90, 4, 64), 5.0, device="cuda", dtype=torch.bfloat16)[30:60] for _ in range(2)]
        vit.cross_attn_bwd(q, q, k, k, out, lse, cq, ck, dq=outs[0], dk=outs[1], dv=outs[2], status=status)
        assert vit.read_status(status) == -10
        for o in outs:
            whole = o._base
            assert (whole[:o.storage_offset() // 256] == 5).all()
            assert (whole[o.storage_offset() // 256 + o.shape[0]:] == 5).all()


def test_graph_replays_other_lengths():
    ql, kl, Hq, Hk, D = [150, 150], [400, 400], 4, 2, 80
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    do = torch.randn_like(q)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    g = [torch.empty_like(t) for t in (q, k, v)]
    wf = torch.empty(vit.cross_attn_workspace_size(300, 800, Hq, Hk, D, 2, 150, 400), dtype=torch.uint8, device="cuda")
    wb = torch.empty(vit.cross_attn_bwd_workspace_size(300, 800, Hq, Hk, D, 2, 150, 400), dtype=torch.uint8,
                     device="cuda")

    def step():
        vit.cross_attn(q, k, v, cq, ck, 150, 400, out=out, lse=lse, workspace=wf)
        vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, 150, 400, dq=g[0], dk=g[1], dv=g[2], workspace=wb)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (400, 37, 0):
        ck.copy_(torch.tensor([0, n, n + 400], dtype=torch.int32))
        for t in g:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(g, reference(q, k, v, do, cq, ck), f"{n}: ")


@pytest.mark.parametrize("B,Hq,Hk,D", [(31, 4, 1, 64), (32, 2, 2, 80), (33, 4, 2, 96), (700, 2, 1, 32), (40, 8, 8, 128)])
def test_many_sequences(B, Hq, Hk, D):
    ql, kl = many(B, 0, 60, 0, 150, B)
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    g = torch.Generator(device="cuda").manual_seed(B)
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True)
    status = vit.new_status()
    got = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), status=status)
    assert vit.read_status(status) == 0
    check(got, reference(q, k, v, do, cq, ck))


@pytest.mark.parametrize("D", [32, 64, 80, 96, 128])
def test_every_tail(D):
    """Streamed lengths that end in each 16-row step of a tile, and in each half of the widest."""
    kl = [112 * 2 + n for n in (0, 1, 15, 16, 17, 47, 48, 49, 63, 64, 65, 79, 80, 81, 95, 96, 97, 111)]
    ql = kl[::-1]
    q, k, v, cq, ck = make(ql, kl, 2, 2, D)
    g = torch.Generator(device="cuda").manual_seed(D)
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    out, lse = vit.cross_attn(q, k, v, cq, ck, return_lse=True)
    check(vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck), reference(q, k, v, do, cq, ck))
