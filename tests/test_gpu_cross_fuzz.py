"""Seeded random calls of cross attention and its gradient: head groups and sizes, ragged lengths with empty
sequences, padded states, unused rows and loose bounds, against the definition in 64 bits (the tolerances are those
that the tests of the two calls derive), and twice for the same bits."""
import math
import random

import pytest
import torch

import vision_encoder_varlen_gb300 as vit
import test_gpu_cross_attn as forward
import test_gpu_cross_attn_bwd as backward

pytestmark = pytest.mark.gpu


def draw(rng):
    while True:
        Hk = rng.choice([1, 2, 3, 4])
        c = dict(D=rng.choice([32, 64, 80, 96, 128]), Hk=Hk, Hq=Hk * rng.choice([1, 1, 2, 3, 4, 6, 8]),
                 B=rng.choice([1, 2, 3, 5, 9, 20, 33, 40]), gap=rng.choice([0, 0, 3]))
        mq, mk = rng.choice([1, 2, 7, 16, 33, 70, 200, 600]), rng.choice([1, 15, 64, 130, 500, 1500, 4000])
        c["ql"] = [rng.randint(0, mq) for _ in range(c["B"])]
        c["kl"] = [rng.randint(0, mk) for _ in range(c["B"])]
        c["lens"] = [rng.randint(0, n) for n in c["kl"]] if rng.random() < 0.3 else None
        c["mq"], c["mk"] = rng.choice([max(c["ql"]), None, max(c["ql"]) + 5]), rng.choice([max(c["kl"]), None])
        if sum(c["ql"]) and sum(c["kl"]) and c["B"] * mq * mk * c["Hq"] <= 3e8:
            return c


@pytest.mark.parametrize("seed", range(40))
def test_random_call(seed):
    c = draw(random.Random(seed))
    gap, lens, ql, kl = c["gap"], c["lens"], c["ql"], c["kl"]
    q, k, v, cq, ck = forward.make(ql, kl, c["Hq"], c["Hk"], c["D"], seed=seed, gap=gap)
    k_len = None
    if lens is not None:
        k_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):                           # what lies behind the real states enters nothing
            k[int(ck[b]) + n:int(ck[b + 1])] = math.nan
            v[int(ck[b]) + n:int(ck[b + 1])] = math.inf
    status = vit.new_status()
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    call = lambda o, **kw: vit.cross_attn(q, k, v, cq, ck, c["mq"], c["mk"], k_len=k_len, out=o, status=status, **kw)
    call(out, lse=lse)
    inside = slice(gap, gap + sum(ql))
    forward.check(out, lse, forward.reference(q, k, v, cq, ck, lens), inside)
    assert (out[:gap] == 9).all() and (out[inside.stop:] == 9).all()
    assert torch.equal(out, call(torch.full_like(q, 9.0)))
    g = torch.Generator(device="cuda").manual_seed(seed)
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    back = lambda: vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, c["mq"], c["mk"], k_len=k_len, status=status)
    got = back()
    assert vit.read_status(status) == 0
    used_q = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    used_q[inside] = True
    used_k = torch.zeros(k.shape[0], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens or kl):
        used_k[int(ck[b]):int(ck[b]) + n] = True
    used = (used_q, used_k, used_k)
    ref, tol = backward.reference(q, k, v, do, cq, ck, lens)
    pick = lambda ts: [t[u] for t, u in zip(ts, used)]
    backward.check(pick(got), (pick(ref), pick(tol)))
    assert not any(t[~u].any() for t, u in zip(got, used))
    assert all(torch.equal(a, b) for a, b in zip(got, back()))
