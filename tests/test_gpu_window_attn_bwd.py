"""Gradient of causal attention with a sliding window and first tokens kept visible, against the definition in 64 bits
and against differences.

Tolerances, per element, as for cross attention's gradient. P and dS are rounded to bf16 (2^-8 of each), o is bf16
(2^-8 of each of its elements, so delta is off by 2^-8 sum_d |do_d o_d|), scores and dP are fp32 sums of D products
(below D 2^-24 of their magnitudes, relative errors of every p), exp2 is good to 2^-21, results are rounded once (2^-8).
With e = 2 score error + 2^-19:
  |dv err| <= 2^-8 |dv| + (2^-8 + e)(1 + 2^-8) sum p |do|
  |ds err| <= (2^-8 + e)(1 + 2^-8) p (|dP| + |delta| + m) + p 2^-8 sum |do o| =: w,  m = D 2^-24 sum |do v|
  |dq err| <= 2^-8 |dq| + scale sum_j w |k|, likewise dk.
Rows that see 2 to 16 keys have delta from the scores: for them the term with sum |do o| is e p (|dP| + |delta|) instead.
"""
import math
import random

import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from test_gpu_window_attn import make, offsets, visible

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def reference(q, k, v, do, cu_q, cu_k, k_len=None, window=0, sinks=0, scale=None):
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
    g, tol = [z(q), z(k), z(v)], [z(q), z(k), z(v)]
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cq) - 1):
        n = ck[b + 1] - ck[b] if k_len is None else int(k_len[b])
        rq, rk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b] + n)
        if n == 0 or cq[b + 1] == cq[b]:
            continue
        see = visible(cq[b + 1] - cq[b], n, window, sinks)
        few = ((see.sum(1) >= 2) & (see.sum(1) <= 16))[:, None]
        for h in range(Hq):
            Q, DO, K, V = q[rq, h].double(), do[rq, h].double(), k[rk, h * Hk // Hq].double(), v[rk, h * Hk // Hq].double()
            s = (Q @ K.T * scale).masked_fill(~see, -math.inf)
            p = torch.softmax(s, -1).nan_to_num(nan=0.0)
            o, dp = p @ V, DO @ V.T
            delta = (DO * o).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            e = 2 * (Q.abs() @ K.abs().T).masked_fill(~see, 0).amax() * scale * D * 2.0 ** -24 + 2.0 ** -19
            m = D * 2.0 ** -24 * (DO.abs() @ V.abs().T)
            rounded = torch.where(few, e * (dp.abs() + delta.abs()), BF * (DO * o).abs().sum(-1, keepdim=True))
            w = (BF + e) * (1 + BF) * p * (dp.abs() + delta.abs() + m) + p * rounded
            at = h * Hk // Hq
            g[0][rq, h], tol[0][rq, h] = scale * ds @ K, scale * w @ K.abs()
            g[1][rk, at] += scale * ds.T @ Q
            tol[1][rk, at] += scale * w.T @ Q.abs()
            g[2][rk, at] += p.T @ DO
            tol[2][rk, at] += (BF + e) * (1 + BF) * p.T @ DO.abs()
    return g, tol


def check(got, ref, what=""):
    for name, x, y, t in zip(("dq", "dk", "dv"), got, *ref):
        assert torch.isfinite(x).all(), what + name
        err = (x.double() - y).abs() - (BF * y.abs() + t + 2.0 ** -130)
        assert (err <= 0).all(), f"{what}{name}: {float(err.max()):.3e} past its bound"


def grads(ql, kl, Hq, Hk, D, window, sinks, seed=9):
    q, k, v, cq, ck, _ = make(ql, kl, Hq, Hk, D)
    g = torch.Generator(device="cuda").manual_seed(seed)
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    return q, k, v, do, cq, ck, (window or None, sinks)


# packed texts (as many keys as queries), continuations over cached keys, more queries than keys, none of either
CASES = [
    ([1], [1], 1, 1, 32, 0, 0),
    ([1, 3], [1, 40], 2, 1, 64, 5, 1),
    ([17], [16], 1, 1, 128, 0, 0),
    ([64, 65, 1, 0, 7], [64, 1, 700, 9, 0], 4, 2, 80, 20, 3),
    ([130, 1, 257, 31], [130, 1111, 257, 128], 8, 1, 128, 100, 4),
    ([130, 1, 257, 31], [130, 1111, 257, 128], 8, 1, 128, 0, 0),
    ([300, 200], [300, 513], 6, 2, 96, 64, 70),
    ([1000], [999], 3, 3, 32, 7, 0),
    ([1000], [1000], 4, 4, 64, 1, 0),
    ([129, 600], [129, 600], 5, 1, 64, 0, 0),
    ([40] * 12, [40] * 12, 8, 2, 64, 12, 2),
    ([30] * 50, [33] * 50, 4, 4, 96, 16, 0),
    ([513], [2000], 16, 16, 80, 300, 4),
    ([2000, 3], [2000, 900], 4, 1, 128, 256, 4),
    ([1500], [1500], 2, 2, 80, 200, 150),
    ([2100], [2100], 8, 2, 96, 0, 0),
]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D,window,sinks", CASES)
def test_gradient(ql, kl, Hq, Hk, D, window, sinks):
    q, k, v, do, cq, ck, mask = grads(ql, kl, Hq, Hk, D, window, sinks)
    out, lse = vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), *mask, return_lse=True)
    status = vit.new_status()
    got = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), *mask, status=status)
    assert vit.read_status(status) == 0
    check(got, reference(q, k, v, do, cq, ck, None, window, sinks))
    again = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, None, None, *mask)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("D", [64, 80, 128])
def test_padding_strides_and_untouched_rows(D):
    """NaN before, behind and (past k_len) between the sequences; views with their own strides; what belongs to no
    sequence stays as it was. The second sequence has fewer keys than queries, the third keys before its queries."""
    ql, S, lens, Hq, Hk, gap = [33, 100, 1], 190, [190, 60, 137], 4, 2, 5
    q, _, _, cq, _, _ = make(ql, [1] * 3, Hq, Hk, D, gap=gap)
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
    mask = (40, 3)
    vit.window_attn(q, k, v, cq, ck, max(ql), S, *mask, 0.2, k_len=k_len, out=out, lse=lse)
    do[:gap] = math.nan
    dq = torch.full_like(q, 7.0)
    dkv = torch.full_like(kv, 7.0)
    vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), S, *mask, 0.2, k_len=k_len, dq=dq, dk=dkv[:, 0],
                        dv=dkv[:, 1])
    own_q = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    own_q[gap:gap + sum(ql)] = True
    own_k = torch.zeros(k.shape[0], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        own_k[b * S:b * S + n] = True
    assert (dq[~own_q] == 7).all() and (dkv[~own_k] == 7).all()
    ref, tol = reference(q, k, v, do, cq, ck, lens, *mask, 0.2)
    check((dq[own_q], dkv[:, 0][own_k], dkv[:, 1][own_k]),
          ([ref[0][own_q], ref[1][own_k], ref[2][own_k]], [tol[0][own_q], tol[1][own_k], tol[2][own_k]]))
    made = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), S, *mask, 0.2, k_len=k_len)
    assert (made[0][~own_q] == 0).all() and (made[1][~own_k] == 0).all() and (made[2][~own_k] == 0).all()
    assert torch.equal(made[0][own_q], dq[own_q])


def test_values_behind_the_mask_leave_nothing():
    """Scores of masked pairs that are huge (their exp overflows) enter neither side's gradient."""
    n, D, window = 300, 64, 8
    q, k, v, do, cq, ck, mask = grads([n], [n], 2, 2, D, window, 0)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[1::2, :, 0] = 4000.0                             # against keys that most rows of the same tile do not see
    out, lse = vit.window_attn(q, k, v, cq, ck, n, n, *mask, return_lse=True)
    got = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, n, n, *mask)
    check(got, reference(q, k, v, do, cq, ck, None, window, 0))


def test_against_differences():
    ql, kl, Hq, Hk, D, window, sinks = [5, 70], [40, 90], 4, 2, 64, 11, 2
    q, k, v, do, cq, ck, mask = grads(ql, kl, Hq, Hk, D, window, sinks, seed=11)
    out, lse = vit.window_attn(q, k, v, cq, ck, None, None, *mask, return_lse=True)
    got = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, None, None, *mask)
    tol = reference(q, k, v, do, cq, ck, None, window, sinks)[1]

    def loss(q, k, v):
        total, a, b = 0.0, 0, 0
        for m, n in zip(ql, kl):
            hide = ~visible(m, n, window, sinks)
            for h in range(Hq):
                s = (q[a:a + m, h] @ k[b:b + n, h * Hk // Hq].T / math.sqrt(D)).masked_fill(hide, -math.inf)
                total += (torch.softmax(s, -1) @ v[b:b + n, h * Hk // Hq] * do[a:a + m, h].double()).sum()
            a, b = a + m, b + n
        return total

    base = [t.double() for t in (q, k, v)]
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, (x, t) in enumerate(zip(got, tol)):
        for _ in range(8):
            at = tuple(int(torch.randint(0, s, (1,), generator=g, device="cuda")) for s in x.shape)
            moved = [[t.clone() for t in base] for _ in range(2)]
            moved[0][i][at] += 1e-4
            moved[1][i][at] -= 1e-4
            want = float(loss(*moved[0]) - loss(*moved[1])) / 2e-4
            # a central difference of step 1e-4 in 64 bits is good to 1e-6 here
            assert abs(float(x[at]) - want) <= BF * abs(want) + float(t[at]) + 1e-6


def test_random_calls():
    rng = random.Random(12)
    for i in range(40):
        D, Hk = rng.choice([32, 64, 80, 96, 128]), rng.choice([1, 2, 3])
        Hq, B = Hk * rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 5, 40])
        ql = [rng.choice([0, 1, 1, 2, 15, 64, 130]) if B > 5 else rng.choice([1, 3, 33, 128, 400]) for _ in range(B)]
        kl = [max(0, m + rng.choice([0, 0, 0, 1, 100, 700, -2])) for m in ql]
        if not sum(ql) or not sum(kl):
            continue
        window, sinks = rng.choice([0, 1, 2, 9, 64, 200, 2000]), rng.choice([0, 1, 16, 150])
        q, k, v, do, cq, ck, mask = grads(ql, kl, Hq, Hk, D, window, sinks, seed=i)
        out, lse = vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), *mask, return_lse=True)
        got = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), *mask)
        check(got, reference(q, k, v, do, cq, ck, None, window, sinks), f"{i} ")
