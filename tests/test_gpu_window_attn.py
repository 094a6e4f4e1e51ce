"""Causal attention with a sliding window and the first tokens kept visible, and attention behind a shared prefix,
against their definitions in 64 bits.

Tolerances as for cross attention, per element of out = sum_j p_j v_j: P is rounded to bf16 before the product (2^-8 of
each p_j, so 2^-8 sum_j p_j |v_j|), the result once more (2^-8 of it); scores are fp32 sums of products of bf16 values
(D terms: below D 2^-24 of sum |q_d k_d|, a relative error of every p), exp2 is good to 2^-21 of each p. lse moves by
at most the largest score error plus 2^-21.
"""
import math
import random

import pytest
import torch

import vision_encoder_varlen_gb300 as vit

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def offsets(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def make(ql, kl, Hq, Hk, D, seed=0, gap=0, rows=None):
    """Packed inputs; with `gap`, unused rows before the first and behind the last sequence hold NaN, and so do the rows
    of a padded cache (`rows` for each sequence) behind the real ones."""
    g = torch.Generator(device="cuda").manual_seed(seed + sum(ql) + 3 * sum(kl) + D)
    kr = kl if rows is None else [rows] * len(kl)
    n = lambda T, H: torch.randn(T + 2 * gap, H, D, generator=g, device="cuda").bfloat16()
    q, k, v = n(sum(ql), Hq), n(sum(kr), Hk), n(sum(kr), Hk)
    for t in (q, k, v):
        t[:gap] = math.nan
        t[t.shape[0] - gap:] = math.nan
    cu_k = offsets(kr, gap)
    if rows is not None:
        for b, m in enumerate(kl):
            for t in (k, v):
                t[int(cu_k[b]) + m:int(cu_k[b + 1])] = math.nan
    k_len = None if rows is None else torch.tensor(kl, dtype=torch.int32, device="cuda")
    return q, k, v, offsets(ql, gap), cu_k, k_len


def visible(m, n, window, sinks):
    """[m, n]: what each query sees, the queries being the last of the keys."""
    p = torch.arange(n - m, n, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")
    see = j <= p
    return see & ((p - j < window) | (j < sinks)) if window else see


def reference(q, k, v, cu_q, cu_k, k_len=None, window=0, sinks=0, scale=None, prefix=None):
    """out, lse, and the magnitudes sum p|v| and the score error's bound, by sequence in 64 bits. prefix:
    (k_prefix, v_prefix, first row, end row) for each sequence."""
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    serr = torch.zeros_like(lse)
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cq) - 1):
        m, n = cq[b + 1] - cq[b], ck[b + 1] - ck[b] if k_len is None else int(k_len[b])
        if m == 0:
            continue
        see = visible(m, n, window, sinks)
        K, V = k[ck[b]:ck[b] + n].double(), v[ck[b]:ck[b] + n].double()
        if prefix is not None:
            kp, vp, a, z = prefix[b]
            K, V = torch.cat([kp[a:z].double(), K]), torch.cat([vp[a:z].double(), V])
            see = torch.cat([torch.ones(m, z - a, dtype=torch.bool, device="cuda"), see], 1)
        if K.shape[0] == 0:
            continue
        for r0 in range(0, m, 2048):
            r1 = min(m, r0 + 2048)
            Q = q[cq[b] + r0:cq[b] + r1].double().transpose(0, 1)
            at = slice(cq[b] + r0, cq[b] + r1)
            hide = ~see[r0:r1]
            for h in range(Hq):
                Kh, Vh = K[:, h * Hk // Hq], V[:, h * Hk // Hq]
                s = (Q[h] @ Kh.T * scale).masked_fill(hide, -math.inf)
                p = torch.softmax(s, -1).nan_to_num(nan=0.0)
                out[at, h], mag[at, h] = p @ Vh, p @ Vh.abs()
                lse[at, h] = torch.logsumexp(s, -1)
                serr[at, h] = (Q[h].abs() @ Kh.abs().T).masked_fill(hide, 0).amax(-1) * scale * D * 2.0 ** -24
    return out, lse, mag, serr


def check(got, got_lse, ref, rows=slice(None)):
    out, lse, mag, serr = ref
    assert torch.isfinite(got[rows]).all()
    e = 2 * serr[..., None] + 2.0 ** -20
    bound = BF * out.abs() + (BF + e) * (1 + BF) * mag + 2.0 ** -130
    err = ((got.double() - out).abs() - bound)[rows]
    assert (err <= 0).all(), f"out {float(err.max()):.3e} past its bound"
    if got_lse is not None:
        empty = torch.isinf(lse)
        assert torch.equal(torch.isneginf(got_lse)[rows], empty[rows])
        d = (got_lse.double() - lse).abs()[rows]
        tol = (serr + 2.0 ** -19 * (1 + lse.abs()))[rows]
        assert (d <= tol)[~empty[rows]].all()


# query lengths, key lengths, Hq, Hkv, D, window, sinks: single tokens, continuations, prompts; keys equal to, more and
# fewer than queries, and none; windows of one, inside a tile, across tiles and wider than everything; sinks of none, one,
# inside a tile, across tiles, meeting the window
CASES = [
    ([1], [1], 1, 1, 32, 0, 0),
    ([1], [1], 1, 1, 128, 1, 1),
    ([1, 1, 1], [1601, 577, 1], 32, 8, 128, 512, 4),
    ([1] * 9, [0, 63, 64, 65, 127, 128, 129, 5000, 1], 8, 1, 80, 64, 1),
    ([1] * 9, [0, 63, 64, 65, 127, 128, 129, 5000, 1], 8, 2, 80, 100, 70),
    ([1, 0, 1], [700, 300, 0], 4, 4, 96, 1, 0),
    ([2, 5, 1, 0], [33, 1000, 16, 5], 12, 3, 64, 20, 3),
    ([3, 4, 16, 9], [1, 4, 3000, 0], 4, 4, 32, 33, 17),
    ([16, 7], [900, 5000], 2, 1, 128, 0, 0),
    ([13, 31, 7], [900, 15, 2500], 6, 3, 128, 250, 5),
    ([64, 64], [256, 4097], 2, 2, 80, 300, 4),
    ([40, 64], [3, 1700], 2, 2, 32, 0, 0),
    ([65], [65], 1, 1, 64, 7, 2),
    ([9, 70, 1], [100, 1000, 0], 8, 1, 128, 128, 16),
    ([130, 1, 257, 0, 300], [130, 1111, 200, 50, 312], 4, 2, 80, 100, 4),
    ([130, 1, 257, 0, 300], [130, 1111, 257, 50, 300], 4, 4, 80, 0, 0),
    ([513], [6000], 2, 1, 128, 1000, 200),
    ([300, 200], [300, 2000], 6, 2, 96, 96, 96),
    ([1000], [999], 3, 3, 32, 128, 4),
    ([1000], [1000], 8, 1, 128, 1, 0),
    ([129, 2000], [640, 2000], 5, 1, 64, 333, 130),
    ([2000, 1500], [2000, 1500], 16, 16, 64, 256, 4),
    ([200], [20000], 1, 1, 80, 7000, 300),
    ([1537, 300, 77], [1537, 900, 77], 32, 8, 128, 0, 0),
    ([1537, 300, 77], [1537, 900, 77], 32, 8, 128, 400, 4),
]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D,window,sinks", CASES)
def test_forward(ql, kl, Hq, Hk, D, window, sinks):
    q, k, v, cq, ck, _ = make(ql, kl, Hq, Hk, D, gap=3)
    ref = reference(q, k, v, cq, ck, None, window, sinks)
    status = vit.new_status()
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    args = (window or None, sinks)
    vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), *args, out=out, lse=lse, status=status)
    assert vit.read_status(status) == 0
    inside = slice(3, 3 + sum(ql))
    check(out, lse, ref, inside)
    assert (out[:3] == 9).all() and (out[3 + sum(ql):] == 9).all() and (lse[:3] == 9).all()
    # no bounds given, and no lse: still the same rows
    plain = torch.full_like(q, 9.0)
    vit.window_attn(q, k, v, cq, ck, None, None, *args, out=plain)
    check(plain, None, ref, inside)
    again = torch.full_like(q, 9.0)
    vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), *args, out=again)
    assert torch.equal(again, out)                     # the same bits from run to run


@pytest.mark.parametrize("m", [1, 4, 40, 300])
@pytest.mark.parametrize("D", [64, 80])
def test_padded_cache(m, D):
    """A cache of as many rows for every sequence, NaN behind the real ones."""
    ql, kl = [m] * 5, [max(m, n) for n in (m, 77, 400, 511, 512)]
    q, k, v, cq, ck, k_len = make(ql, kl, 8, 2, D, rows=max(512, m))
    ref = reference(q, k, v, cq, ck, k_len, 100, 4)
    out, lse = vit.window_attn(q, k, v, cq, ck, m, max(512, m), 100, 4, k_len=k_len, return_lse=True)
    check(out, lse, ref)


@pytest.mark.parametrize("m", [1, 2, 30, 200])
def test_evicted_rows_are_not_read(m):
    """Rows between the first tokens and the window hold NaN, as in a cache that gave them up."""
    n, window, sinks = 3000, 700, 5
    q, k, v, cq, ck, _ = make([m], [n], 8, 2, 128)
    ref = reference(q, k, v, cq, ck, None, window, sinks)
    for t in (k, v):
        t[sinks:n - m - window + 1] = math.nan
    out, lse = vit.window_attn(q, k, v, cq, ck, m, n, window, sinks, return_lse=True)
    check(out, lse, ref)


@pytest.mark.parametrize("m", [1, 5, 200])
def test_scores_of_minus_infinity_and_huge_scores(m):
    """Keys whose score is -inf have no weight; the running maximum starts from them."""
    n, D = 800, 64
    q, k, v, cq, ck, _ = make([m], [n], 2, 2, D)
    q[..., 0] = 1.0
    k[..., 0] = 0.0
    k[10:700, :, 0] = -math.inf
    k[5:7, :, 0] = 3e4
    see = visible(m, n, 500, 8)
    s = torch.einsum("qhd,khd->hqk", q.double(), k.double()) / math.sqrt(D)
    s.masked_fill_(~see, -math.inf)
    p = torch.softmax(s, -1)
    want = torch.einsum("hqk,khd->qhd", p, v.double())
    out, lse = vit.window_attn(q, k, v, cq, ck, m, n, 500, 8, return_lse=True)
    assert torch.isfinite(out).all()
    mag = torch.einsum("hqk,khd->qhd", p, v.double().abs())
    # two keys with scores of 3750 carry the rows: D terms of fp32 sums are D 2^-24 of that, twice so much moves the
    # weights of one against the other, and what the file's head says of lse holds for it
    serr = D * 2.0 ** -24 * 3750
    assert ((out.double() - want).abs() <= (2 * serr + BF) * (1 + BF) * mag + BF * want.abs()).all()
    lse_want = torch.logsumexp(s, -1)
    assert ((lse.T.double() - lse_want).abs() <= serr + 2.0 ** -19 * (1 + lse_want.abs())).all()


# groups of sequences with query and own key lengths, prefixes: decoding, questions, prompts; no prefix, no own keys,
# neither, fewer keys than queries
PREFIX = [
    ([1, 1, 1], [5, 1, 90], [1601], [3], 32, 8, 128),
    ([1] * 20, [1, 2, 300, 77, 64] * 4, [700, 3000], [15, 5], 8, 2, 64),
    ([1] * 40, [7] * 40, [0, 513, 1, 4000], [3, 20, 0, 17], 8, 1, 80),
    ([3, 1, 8, 0, 5], [3, 0, 2, 0, 100], [129, 0], [3, 2], 4, 4, 96),
    ([20, 131, 7, 64, 33, 90], [20, 131, 7, 64, 33, 90], [777, 2500], [2, 4], 16, 16, 80),
    ([20, 131, 7, 64, 33, 90] * 6, [30, 131, 3, 64, 0, 95] * 6, [777, 0, 2500], [12, 6, 18], 3, 1, 32),
    ([700, 300, 1], [700, 500, 1], [4097], [3], 32, 8, 128),
    ([300, 500], [100, 0], [50, 0], [1, 1], 2, 2, 64),
    ([2000], [2000], [333], [1], 4, 1, 96),
    ([1], [1], [20000], [1], 1, 1, 128),
    ([1] * 200, [3] * 200, [1000], [200], 16, 2, 64),
]


@pytest.mark.parametrize("ql,kl,pl,groups,Hq,Hk,D", PREFIX)
def test_prefix(ql, kl, pl, groups, Hq, Hk, D):
    q, k, v, cq, ck, _ = make(ql, kl, Hq, Hk, D, gap=2)
    kp, vp, _, cp, _, _ = make(pl, [1], Hk, Hk, D, seed=7, gap=2)
    vp = make(pl, [2], Hk, Hk, D, seed=9, gap=2)[0]
    kp = make(pl, [2], Hk, Hk, D, seed=8, gap=2)[0]
    cg, cpl = offsets(groups), cp.tolist()
    of = [(kp, vp, cpl[g], cpl[g + 1]) for g, m in enumerate(groups) for _ in range(m)]
    ref = reference(q, k, v, cq, ck, prefix=of)
    status = vit.new_status()
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    vit.prefix_attn(q, kp, vp, k, v, cq, cp, ck, cg, max(ql), max(pl), max(kl), out=out, lse=lse, status=status)
    assert vit.read_status(status) == 0
    inside = slice(2, 2 + sum(ql))
    check(out, lse, ref, inside)
    assert (out[:2] == 9).all() and (out[2 + sum(ql):] == 9).all() and (lse[:2] == 9).all()
    plain = torch.full_like(q, 9.0)
    vit.prefix_attn(q, kp, vp, k, v, cq, cp, ck, cg if len(pl) > 1 else None, out=plain)
    check(plain, None, ref, inside)
    again = torch.full_like(q, 9.0)
    vit.prefix_attn(q, kp, vp, k, v, cq, cp, ck, cg, max(ql), max(pl), max(kl), out=again)
    assert torch.equal(again, out)


def test_random_calls():
    rng = random.Random(11)
    for i in range(60):
        D, Hk = rng.choice([32, 64, 80, 96, 128]), rng.choice([1, 2, 3])
        Hq, B = Hk * rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 5, 40])
        ql = [rng.choice([0, 1, 1, 2, 15, 64, 130]) if B > 5 else rng.choice([1, 3, 33, 128, 400]) for _ in range(B)]
        kl = [max(0, m + rng.choice([0, 0, 1, 100, 900, -2])) for m in ql]
        window, sinks = rng.choice([0, 1, 9, 64, 200, 3000]), rng.choice([0, 1, 16, 150])
        q, k, v, cq, ck, _ = make(ql, kl, Hq, Hk, D, seed=i, gap=1)
        inside = slice(1, 1 + sum(ql))
        if rng.random() < 0.5:
            ref = reference(q, k, v, cq, ck, None, window, sinks)
            out, lse = vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), window or None, sinks, return_lse=True)
        else:
            G = rng.choice([1, 2])
            cut = rng.randint(0, B)
            pl, groups = [rng.choice([0, 5, 200, 1500]) for _ in range(G)], [cut, B - cut] if G == 2 else [B]
            kp, vp = (make(pl, [1], Hk, Hk, D, seed=s + i, gap=1)[0] for s in (50, 90))
            cp = offsets(pl, 1).tolist()
            of = [(kp, vp, cp[g], cp[g + 1]) for g, m in enumerate(groups) for _ in range(m)]
            ref = reference(q, k, v, cq, ck, prefix=of)
            out, lse = vit.prefix_attn(q, kp, vp, k, v, cq, offsets(pl, 1), ck, offsets(groups), max(ql), max(pl),
                                       max(kl), return_lse=True)
        check(out, lse, ref, inside)
