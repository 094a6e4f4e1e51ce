"""Model of the work list of a language model's own attention (csrc/window_schedule.cu), CPU only: every query row meets
every key that its mask lets through exactly once, items and partial results stay inside the workspace, and no item is
empty. The model mirrors the plan and the list of the source; that the two agree on the plan is read from the
workspace sizes that the library reports."""
import math
import random

import pytest

import vision_encoder_varlen_gb300 as vit
from vision_encoder_varlen_gb300 import _build

SMS = 152
cdiv = lambda a, b: -(-a // b)
up = lambda x: cdiv(x, 256) * 256


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()


def tile_keys(D):
    return min(128, (512 - 2 * D) // 3 // 16 * 16)


def plan(Tq, B, Hq, Hk, D, max_q, max_k, window, sinks, G, Tp, max_p):
    group = Hq // Hk
    lg = 3 if group % 8 == 0 else 2 if group % 4 == 0 else 1 if group % 2 == 0 else 0
    tok, packs, bn = 128 >> lg, Hq >> lg, tile_keys(D)
    own = min(Tq // tok + B, B * cdiv(max_q, tok))
    grouped = Tq // tok + G
    prefix = G > 0 and Tp > 0
    apart = prefix and own > 2 * grouped
    own_most = cdiv(min(max_k, window + 2 * tok - 1) if window else max_k, bn)
    first_most = cdiv(max_p if prefix else min(sinks, max_k) if window else 0, bn)
    own_few = apart and few(B, Hq, Hk, D, max_q, max_k, 0, 0)
    p = dict(lg=lg, apart=apart, own_few=own_few, units=(G if own_few else G + B if apart else B), run=0, slots=0, tiles=0)
    least = 2 * cdiv(512, 2 * bn)
    if apart:
        own = 0 if own_few else own
        p["run"] = run = max(least, cdiv((own * own_most + grouped * first_most) * packs, 8 * SMS))
        p["items"] = p["slots"] = (grouped * max(1, cdiv(first_most, run)) + own * max(1, cdiv(own_most, run))) * packs
    else:
        tiles, most = own * packs, own_most + first_most
        p["items"] = tiles
        if 0 < 2 * tiles <= SMS:
            run = max(least, cdiv(most, SMS // tiles))
            if cdiv(most, run) > 1:
                p.update(run=run, items=tiles * cdiv(most, run), tiles=tiles, slots=tiles * cdiv(most, run))
    part_s = up(up(up(up(64 + 48 * p["items"]) + 32 * p["tiles"]) + 8 * B) + (16 * p["units"] if apart else 0))
    p["bytes"] = up(up(part_s + p["slots"] * 512) + p["slots"] * 512 * D)
    if own_few:
        p["bytes"] += few_bytes(B, Hq, Hk, D, max_q, max_k)
    return p


def few_bytes(B, Hq, Hk, D, max_q, max_k):
    """Partial results of the kernel for few rows, also where it makes one run."""
    rows, pairs = max_q * (Hq // Hk), B * Hk
    if pairs >= SMS and max_k <= 2048:
        return 4 * pairs * rows * (D + 1)
    fit = SMS * (227 * 1024 // (3 * 256 * D + 2048))   # blocks that run at a time
    n = max(1, min((8 * SMS + pairs // 2) // pairs, cdiv(max_k, max(16 * rows, 128))))
    for _ in range(2):                                 # again with fewer runs where a second round would be a small one
        chunk = max(64, cdiv(cdiv(max_k, n), 64) * 64)
        runs = cdiv(max_k, chunk) if max_k else 1
        if not (pairs <= fit < pairs * runs and 2 * pairs * runs < 3 * fit):
            break
        n = fit // pairs
    return 4 * pairs * runs * rows * (D + 1)


def few(B, Hq, Hk, D, max_q, max_k, window, sinks):
    most = max_k
    if window and window + sinks < max_k:
        most = min(cdiv(sinks, 64) * 64 + window + max_q - 1, max_k + 64)
    rows = max_q * (Hq // Hk)
    return rows <= 16 or (rows <= 32 and B * most * Hk * D * 4 <= 32 << 20)


def span(first, last, window, sinks, prefix):
    """(first tokens read apart, position from which the rest is read, keys read from there) of queries first..last"""
    lo = max(0, first - window + 1) if window and not prefix else 0
    n = sinks if lo > sinks else 0
    lo = lo if lo > sinks else 0
    return n, lo, max(0, last + 1 - lo)


def make_list(p, ql, kl, Hq, D, window, sinks, prefixes=None, groups=None, sms=SMS, longer=0):
    """With a prefix apart the list may take `longer` runs than the plan's. Items as (unit, first query, end, head, tiles, prefix or first keys [a, b), own keys [a, b), slot, two tiles)."""
    bn, lg_tile, packs = tile_keys(D), 7 - p["lg"], Hq >> p["lg"]
    if p["apart"]:
        p = dict(p, run=p["run"] + longer)
    units, at = [], 0
    start = [sum(ql[:i]) for i in range(len(ql))]
    if p["apart"]:                                     # the groups first
        for f, m in zip(prefixes, groups):
            units.append(dict(q=(start[at] if m else 0), n=sum(ql[at:at + m]), f=f, k=0, p0=0))
            at += m
    of = [f for f, m in zip(prefixes or [], groups or []) for _ in range(m)]
    for b, (m, n) in enumerate(zip(ql, kl) if not p["own_few"] else ()):
        f = of[b] if of and not p["apart"] else 0
        none = max(0, m - n) if f == 0 else 0
        units.append(dict(q=start[b] + none, n=m - none, f=f, k=n, p0=n - m + none))

    def tiles_of(u, t, e):
        a, lo, n = (0, 0, 0) if u["k"] == 0 else span(u["p0"] + t, u["p0"] + e - 1, window, sinks, prefixes is not None)
        a = u["f"] if prefixes is not None else a
        return a, lo, n, cdiv(a, bn) + cdiv(n, bn)

    used = [i for i, u in enumerate(units) if u["n"] > 0 and (u["f"] > 0 or u["k"] > 0)]
    longest = {i: tiles_of(units[i], max(0, units[i]["n"] - (1 << lg_tile)), units[i]["n"])[3] for i in used}
    used.sort(key=lambda i: (-longest[i], i))
    full = sum(packs * cdiv(units[i]["n"], 2 << lg_tile) for i in used)
    all_split = p["run"] > 0 or p["apart"] or 2 * full <= sms
    lg = lg_tile if all_split else lg_tile + 1
    listed, slot = [], 0
    for i in used:
        u = units[i]
        nq, runs = cdiv(u["n"], 1 << lg), max(1, cdiv(longest[i], p["run"])) if p["run"] else 1
        for n in range(nq * packs * runs):
            j, run = divmod(n, runs)
            t = (nq - 1 - j // packs) << lg
            e = min(u["n"], t + (1 << lg))
            f, lo, k, tiles = tiles_of(u, t, e)
            use = max(1, cdiv(tiles, p["run"])) if runs > 1 else 1
            assert use <= runs
            if run < use:
                nf, a, b = cdiv(f, bn), tiles * run // use, tiles * (run + 1) // use
                fa, fb = (min(f, min(x, nf) * bn) for x in (a, b))
                ka, kb = (min(k, max(0, x - nf) * bn) for x in (a, b))
                halves = [(t, e)]
                listed.append((i, t, e, j % packs, (fa, fb), (lo + ka, lo + kb),
                               slot + n if runs > 1 or p["apart"] else -1))
        slot += nq * packs * runs
    rest = len(listed) % sms
    cut = rest if not all_split and 2 * rest <= sms else 0
    extra = sum(1 for x in listed[len(listed) - cut:] if x[2] - x[1] > 1 << lg_tile) if cut else 0
    return units, listed, len(listed) + extra, slot


def check(ql, kl, Hq, Hk, D, window=0, sinks=0, prefixes=None, groups=None, loose=False, longer=0):
    Tq, B = sum(ql), len(ql)
    G, Tp = (len(prefixes), sum(prefixes)) if prefixes else (0, 0)
    max_q, max_k = (Tq, sum(kl)) if loose else (max(ql), max(kl))
    max_p = (Tp if loose else max(prefixes)) if prefixes else 0
    window = 0 if window >= max_k else window          # it leaves nothing out
    sinks = sinks if window else 0
    p = plan(Tq, B, Hq, Hk, D, max_q, max_k, window, sinks, G, Tp, max_p)
    rows, keys = max_q * (Hq // Hk), cdiv(max_p, 64) * 64 + max_k
    if prefixes is not None and few(B, Hq, Hk, D, max_q, keys, 0, 0) and B * keys * Hk * D * 4 <= 96 << 20:
        return                                         # each sequence reads its prefix: no list
    if prefixes is not None:
        assert vit.prefix_attn_workspace_size(Tq, Tp, sum(kl), Hq, Hk, D, B, G, max_q, max_p, max_k) == p["bytes"]
    elif not few(B, Hq, Hk, D, max_q, max_k, window, sinks):
        assert vit.window_attn_workspace_size(Tq, sum(kl), Hq, Hk, D, B, max_q, max_k, window, sinks) == p["bytes"]
    units, items, n_items, slots = make_list(p, ql, kl, Hq, D, window, sinks, prefixes if Tp else None, groups, longer=longer)
    assert n_items <= p["items"]
    assert (slots if p["run"] else 0) <= p["slots"]
    seen = {}
    for u, t, e, pack, f, k, slot in items:
        assert f[1] > f[0] or k[1] > k[0]
        assert -1 <= slot < max(p["slots"], 1)
        seen.setdefault((u, t, e, pack), []).append((f, k))
    packs = Hq >> p["lg"]
    for i, u in enumerate(units):
        mine = sorted((t, e) for (x, t, e, pack) in seen if x == i and pack == 0)
        if u["n"] > 0 and (u["f"] > 0 or u["k"] > 0):
            assert mine[0][0] == 0 and mine[-1][1] == u["n"] and all(a[1] == b[0] for a, b in zip(mine, mine[1:]))
        for t, e in mine:
            for pack in range(packs):
                assert sorted(seen[i, t, e, pack]) == sorted(seen[i, t, e, 0])
            parts = seen[i, t, e, 0]
            first = sorted(f for f, _ in parts if f[1] > f[0])
            own = sorted(k for _, k in parts if k[1] > k[0])
            for x in (first, own):                     # pieces that meet
                assert all(a[1] == b[0] for a, b in zip(x, x[1:]))
            lo, hi = (own[0][0], own[-1][1]) if own else (0, 0)
            head = (first[0][0], first[-1][1]) if first else (0, 0)
            if prefixes and Tp:
                assert head == (0, u["f"]) and lo == 0
                head = (0, 0)
            if not u["k"]:
                continue
            for pos in {u["p0"] + t, u["p0"] + (t + e) // 2, u["p0"] + e - 1}:
                for j in {0, 1, sinks - 1, sinks, pos - window, pos - window + 1, pos - 1, pos, lo - 1, lo}:
                    if not 0 <= j < u["k"]:
                        continue
                    visible = j <= pos and (window == 0 or pos - j < window or j < sinks)
                    assert (head[0] <= j < head[1]) + (lo <= j < hi) <= 1
                    if visible:
                        assert head[0] <= j < head[1] or lo <= j < hi


def test_windows():
    rng = random.Random(5)
    for _ in range(400):
        B, Hk, D = rng.choice([1, 2, 3, 9, 40]), rng.choice([1, 2, 3]), rng.choice([32, 64, 80, 96, 128])
        Hq = Hk * rng.choice([1, 2, 3, 4, 8])
        ql = [rng.choice([0, 1, 2, 17, 64, 128, 129, 300, 1000]) for _ in range(B)]
        kl = [max(0, m + rng.choice([0, 0, 5, 1000, 4001, -1, -m])) for m in ql]
        if sum(ql) and sum(kl):
            check(ql, kl, Hq, Hk, D, rng.choice([0, 1, 2, 7, 128, 500, 5000]), rng.choice([0, 1, 4, 113, 600]),
                  loose=rng.random() < 0.3)


def test_prefixes():
    rng = random.Random(6)
    for _ in range(400):
        G, Hk, D = rng.choice([1, 1, 2, 5]), rng.choice([1, 2, 3]), rng.choice([32, 64, 80, 96, 128])
        groups = [rng.choice([0, 1, 2, 12]) for _ in range(G)]
        B = sum(groups)
        most = rng.choice([1, 3, 70, 600])
        ql = [rng.choice([0, 1, 2, most]) for _ in range(B)]
        kl = [max(0, m + rng.choice([0, 0, 3, 900, -1, -m])) for m in ql]
        if B and sum(ql) and sum(kl):
            check(ql, kl, Hk * rng.choice([1, 2, 4, 8]), Hk, D,
                  prefixes=[rng.choice([0, 1, 100, 1601, 9000]) for _ in range(G)], groups=groups,
                  loose=rng.random() < 0.3, longer=rng.choice([0, 1, 5, 40, 127]))
