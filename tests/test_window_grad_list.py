"""Model of the gradient's work lists in a language model's own attention (make_list in csrc/cross_bwd.cu), CPU only, against
the library's own plan: the items of both passes, the key tiles whose loops are cut and their runs stay inside the
workspace, every query tile of a key tile's loop belongs to exactly one run, and no run is empty."""
import os
import random
import re

from vision_encoder_varlen_gb300 import _build
from test_window_plans import plans

cdiv = lambda a, b: -(-a // b)
up = lambda x: cdiv(x, 256) * 256


def streamed(D):
    """Rows of a streamed tile: (dk and dv, dq)."""
    return (112 if D == 32 else 96 if D == 64 else 64 if D == 128 else 80), (112 if D <= 64 else 96 if D == 80 else 80 if D == 96 else 64)


def test_tile_sizes():
    with open(os.path.join(_build.CSRC, "cross_bwd.cu")) as f:
        text = re.sub(r"\s+", " ", f.read())
    assert ("int BN = DKV ? (D == 32 ? 112 : D == 64 ? 96 : D == 128 ? 64 : 80) : (D <= 64 ? 112 : D == 80 ? 96 : D == 96 ? 80 : 64)"
            in text)
    assert "it.tiles = (it.ln + step - 1) / step * (Hq / Hk >> lg_pack);" in text


def key_loops(p, ql, kl, Hq, Hk, D, window, sinks):
    """The loop length in tiles of every key tile, for one key head."""
    tok, packs = streamed(D)[0] >> p["lg_pack"], Hq // Hk >> p["lg_pack"]
    for m, n in zip(ql, kl):
        p0 = n - m
        for a in range(0, n, 128):
            e = min(n, a + 128)
            lo = max(0, a - p0)
            hi = m if window == 0 or a < sinks else e - 1 + window - p0
            yield a, cdiv(max(0, min(m, hi) - lo), tok) * packs


def check(p, ql, kl, Hq, Hk, D, window, sinks):
    lg = p["lg_pack"]
    assert sum(cdiv(m, 128 >> lg) for m in ql) * (Hq >> lg) <= p["max_dq"]
    loops = list(key_loops(p, ql, kl, Hq, Hk, D, window, sinks))
    assert len(loops) * Hk <= p["max_dkv"]
    stats = up(up(256 + 48 * p["max_dq"]) + 48 * (p["max_dkv"] + p["max_slots"]))
    assert p["bytes"] == up(up(stats + 8 * sum(ql) * Hq) + 32 * p["max_cut"]) + 4 * 2 * 128 * D * p["max_slots"]
    if p["cut_over"] == 0:
        assert p["max_cut"] == p["max_slots"] == 0
        return 0
    assert window > 0 and sinks > 0 and 0 < p["run_tiles"] <= p["cut_over"] and p["max_slots"] <= 304
    cut = [t for _, t in loops if t > p["cut_over"]]
    assert all(a < sinks for a, t in loops if t > p["cut_over"])   # only the first tokens' tiles
    runs = [cdiv(t, p["run_tiles"]) for t in cut]
    assert len(cut) * Hk <= p["max_cut"] and sum(runs) * Hk <= p["max_slots"], (p, cut)
    for t, r in zip(cut, runs):
        at = [t * k // r for k in range(r + 1)]
        assert r >= 2 and all(0 < b - a <= p["run_tiles"] for a, b in zip(at, at[1:])) and at[1] == t // r
    return sum(runs) * Hk / p["max_slots"]


def test_lists_stay_inside_the_workspace(plans):
    rng = random.Random(11)
    calls = []
    for i in range(2000):
        D, Hk = rng.choice([32, 64, 80, 96, 128]), rng.choice([1, 1, 2, 3, 8, 16])
        Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8, 16])
        B = rng.choice([1, 1, 2, 3, 9, 40, 300])
        most = rng.choice([40, 700, 5000, 40000, 300000]) // (1 if B < 9 else 10)
        ql = [rng.choice([0, 1, most, rng.randint(1, most), rng.randint(1, most)]) for _ in range(B)]
        kl = [max(0, m + rng.choice([0, 0, 0, 7, most, -1, -m])) for m in ql]
        if sum(ql) and sum(kl):
            calls.append((ql, kl, Hq, Hk, D, rng.choice([0, 1, 16, 64, 128, 500, 5000]),
                          rng.choice([0, 1, 4, 16, 128, 129, 600, 5000, 2 ** 31 - 1]), rng.random() < 0.3))
    lines = []
    for ql, kl, Hq, Hk, D, window, sinks, loose in calls:
        mq, mk = (sum(ql), sum(kl)) if loose else (max(ql), max(kl))
        window = 0 if window >= mk else window                     # as the call does before it makes its plan
        lines.append(("grad", sum(ql), sum(kl), len(ql), Hq, Hk, D, mq, mk, window, sinks if window else 0))
    used = [check(p, *c[:5], x[9], x[10]) for p, c, x in zip(plans(lines), calls, lines)]
    assert sum(u > 0 for u in used) > 50 and max(used) > 0.4      # cut loops are among them
