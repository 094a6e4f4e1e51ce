"""The measured cases of a language model's own attention: a sliding window with the first tokens kept
visible, for prompts, single tokens and training, and attention of a batch that shares a long prefix.

``run`` computes each operator in a plain form (elementary torch operations in 32 bits) or, where
``own`` is true, through the package's entry points.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of three conversations behind a short window: latency
        dict(name="window_step", op="window", batch=3, q_lo=1, q_max=1, k_lo=1, k_max=1601, lens=21, window=512,
             sinks=4, padded=True, empty=False, q_heads=32, k_heads=8, dim=128, lse=False),
        # one decoding step of a full batch; caches padded to a bucket, some shorter than the window
        dict(name="window_step_batch", op="window", batch=48, q_lo=1, q_max=1, k_lo=60, k_max=16383, lens=22,
             window=4096, sinks=4, padded=True, empty=True, q_heads=32, k_heads=8, dim=128, lse=False),
        # continuations of a few tokens each (drafted tokens, tails of prompts) over cached text
        dict(name="window_chunk", op="window", batch=9, q_lo=1, q_max=67, k_lo=100, k_max=6007, lens=23, window=1000,
             sinks=17, padded=True, empty=False, q_heads=16, k_heads=16, dim=80, lse=False),
        # prompts through a windowed layer, part of each cached already, with the log-sum-exp
        dict(name="window_prefill", op="window", batch=3, q_lo=1500, q_max=6007, k_lo=6100, k_max=8191, lens=24,
             window=2048, sinks=4, padded=False, empty=False, q_heads=32, k_heads=8, dim=128, lse=True),
        # prompts through a layer that sees everything before them
        dict(name="causal_prefill", op="window", batch=4, q_lo=700, q_max=4095, k_lo=1, k_max=4095, lens=25, window=0,
             sinks=0, padded=False, empty=False, q_heads=16, k_heads=16, dim=80, lse=False),
        # training, short packed texts
        dict(name="window_train_short", op="window_train", batch=9, q_lo=1, q_max=700, k_lo=1, k_max=1, lens=26,
             window=128, sinks=4, padded=False, empty=False, q_heads=8, k_heads=2, dim=64, lse=True),
        # training, long packed texts through a windowed layer
        dict(name="window_train_long", op="window_train", batch=4, q_lo=2500, q_max=5117, k_lo=1, k_max=1, lens=27,
             window=1024, sinks=4, padded=False, empty=False, q_heads=16, k_heads=16, dim=80, lse=True),
        # training through a layer that sees everything, grouped heads
        dict(name="causal_train", op="window_train", batch=3, q_lo=1500, q_max=2311, k_lo=1, k_max=1, lens=28,
             window=0, sinks=0, padded=False, empty=False, q_heads=32, k_heads=8, dim=128, lse=True),
        # one decoding step of three answers about one image: latency
        dict(name="prefix_step", op="prefix", groups=1, batch=3, q_lo=1, q_max=1, p_lo=1601, p_max=1601, k_lo=1,
             k_max=90, lens=29, padded=True, empty=False, q_heads=32, k_heads=8, dim=128, lse=False),
        # one decoding step of many answers about each of several documents
        dict(name="prefix_step_batch", op="prefix", groups=4, batch=64, q_lo=1, q_max=1, p_lo=3000, p_max=8191, k_lo=5,
             k_max=700, lens=30, padded=True, empty=False, q_heads=32, k_heads=8, dim=128, lse=False),
        # questions about two images, read in one batch, with the log-sum-exp
        dict(name="prefix_questions", op="prefix", groups=2, batch=32, q_lo=8, q_max=131, p_lo=2000, p_max=4097,
             k_lo=1, k_max=131, lens=31, padded=False, empty=False, q_heads=16, k_heads=16, dim=80, lse=True),
        # long prompts behind one shared document
        dict(name="prefix_prompts", op="prefix", groups=1, batch=6, q_lo=300, q_max=2047, p_lo=8191, p_max=8191,
             k_lo=1, k_max=2047, lens=32, padded=False, empty=False, q_heads=32, k_heads=8, dim=128, lse=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _heads(rng):
    k_heads = rng.choice([1, 2, 4, 8, 16])
    q_heads = k_heads * rng.choice([1, 1, 2, 4, 8])
    while q_heads > 32:
        q_heads //= 2
    return max(q_heads, k_heads), k_heads


def draw(rng):
    op = rng.choice(["window", "window", "window_train", "prefix", "prefix"])
    dim = rng.choice([32, 64, 80, 96, 128])
    q_heads, k_heads = _heads(rng)
    batch = _log_int(rng, 1, 64)
    case = dict(op=op, lens=rng.randrange(1 << 30), q_heads=q_heads, k_heads=k_heads, dim=dim,
                lse=op == "window_train" or rng.random() < 0.5)
    if op == "prefix":
        kind = rng.choice(["step", "few", "many"])
        q_max = {"step": 1, "few": _log_int(rng, 2, 100), "many": _log_int(rng, 100, 2047)}[kind]
        p_max, k_max = _log_int(rng, 16, 16000), _log_int(rng, 1, 2047)
        while batch * q_max * (p_max + q_max + k_max) * q_heads > 2e9 or batch * (p_max + k_max) * k_heads > 5e6:
            batch, p_max = max(1, batch // 2), max(1, int(p_max * 0.7))
        groups = min(batch, rng.choice([1, 1, 2, 5]))
        return dict(case, groups=groups, batch=batch, q_lo=max(1, q_max // rng.choice([1, 2, 8])), q_max=q_max,
                    p_lo=max(1, p_max // rng.choice([1, 2, 16])), p_max=p_max, k_lo=max(1, k_max // rng.choice([1, 16])),
                    k_max=k_max, padded=rng.random() < 0.5, empty=rng.random() < 0.2)
    window = 0 if rng.random() < 0.2 else _log_int(rng, 8, 5000)
    sinks = 0 if window == 0 else rng.choice([0, 1, 4, 17, 64, 150])
    if op == "window_train":
        q_max, k_max = _log_int(rng, 1, 5200), 1
        while batch * q_max * q_max * q_heads > 1.6e9:
            batch, q_max = max(1, batch // 2), max(1, int(q_max * 0.8))
        padded, empty = False, False
    else:
        kind = rng.choice(["step", "few", "many"])
        q_max = {"step": 1, "few": _log_int(rng, 2, 100), "many": _log_int(rng, 100, 6000)}[kind]
        k_max = _log_int(rng, 1, 16000)
        while batch * q_max * max(q_max, k_max) * q_heads > 4e9 or batch * max(q_max, k_max) * k_heads > 5e6:
            batch, k_max = max(1, batch // 2), max(1, int(k_max * 0.7))
            q_max = max(1, int(q_max * 0.8))
        padded, empty = rng.random() < 0.5, batch > 1 and rng.random() < 0.3
    return dict(case, batch=batch, q_lo=max(1, q_max // rng.choice([1, 2, 8])), q_max=q_max,
                k_lo=max(1, k_max // rng.choice([1, 2, 16])), k_max=k_max, window=window, sinks=sinks, padded=padded,
                empty=empty)


def _lengths(case):
    """Query and key lengths of a case, the first sequence the longest: keys are the cached ones and the
    queries' own. ``empty``: the last sequence has no keys at all."""
    rng = random.Random(case["lens"])
    n = case["batch"]
    q = [case["q_max"]] + [_log_int(rng, case["q_lo"], case["q_max"]) for _ in range(n - 1)]
    k = [case["k_max"]] + [_log_int(rng, case["k_lo"], case["k_max"]) for _ in range(n - 1)]
    k = [max(a, b) for a, b in zip(q, k)]
    if case["empty"]:
        k[-1] = 0
    return q, k


def _prefixes(case):
    """Lengths of the prefixes, and how many sequences share each."""
    rng = random.Random(case["lens"] + 1)
    p = [case["p_max"]] + [_log_int(rng, case["p_lo"], case["p_max"]) for _ in range(case["groups"] - 1)]
    cuts = sorted(rng.sample(range(1, case["batch"]), case["groups"] - 1))
    return p, [b - a for a, b in zip([0] + cuts, cuts + [case["batch"]])]


# ------------------------------------------------------------------ inputs

def _offsets(lens):
    return torch.tensor([0] + list(lens), device="cuda").cumsum(0).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)

    ql, kl = _lengths(case)
    D, Hq, Hk = case["dim"], case["q_heads"], case["k_heads"]
    s = dict(case=case, q_max=max(ql), k_max=max(kl))
    # a padded cache has as many rows for every sequence, and a list of how many are real
    rows = [max(kl)] * len(kl) if case["padded"] else kl
    s["k_len"] = torch.tensor(kl, device="cuda").int() if case["padded"] else None
    s["q"] = normal(sum(ql), Hq, D)
    s["k"] = normal(max(1, sum(rows)), Hk, D)
    s["v"] = normal(max(1, sum(rows)), Hk, D)
    s["cu_q"], s["cu_k"] = _offsets(ql), _offsets(rows)
    if case["op"] == "window_train":
        s["dout"] = normal(sum(ql), Hq, D, scale=0.1)
    if case["op"] == "prefix":
        pl, members = _prefixes(case)
        s["k_prefix"], s["v_prefix"] = normal(sum(pl), Hk, D), normal(sum(pl), Hk, D)
        s["cu_prefix"], s["cu_group"], s["p_max"] = _offsets(pl), _offsets(members), max(pl)
        cuts = [0]
        for m in members:
            cuts.append(cuts[-1] + m)
        s["group_q_max"] = max(sum(ql[a:b]) for a, b in zip(cuts, cuts[1:]))
    return s


# ------------------------------------------------------------------ the plain forms

def _padded(x, start, n, most):
    """[B, heads, most, dim] in 32 bits, and which places hold a row."""
    at = torch.arange(most, device=x.device)
    held = at < n[:, None]
    rows = x[(start[:, None] + at).clamp(max=x.shape[0] - 1)].float()
    return rows.transpose(1, 2), held


def _packed(x, cu, T):
    """The rows of [B, heads, most, dim], one sequence after the other."""
    t = torch.arange(T, device=x.device)
    i = torch.searchsorted(cu[1:].long(), t, right=True)
    return x.transpose(1, 2)[i, t - cu[i]]


def _grouped(q, Hk):
    """[B, Hq, L, D] with the queries of one key head side by side."""
    B, Hq, L, D = q.shape
    return q.reshape(B, Hk, Hq // Hk * L, D)


def _sums(q, k, v, scale, visible):
    """(scores less their row's maximum, exponentiated, their sums, the maxima)."""
    score = q @ k.transpose(-1, -2)
    score *= scale
    if visible is not None:
        score.masked_fill_(~visible, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = score.sub_(top).exp_()
    return p, p.sum(-1, keepdim=True), top


def _window_mask(n_q, n_k, Lq, Lk, window, sinks):
    """[B, Lq, Lk]: what each query of a sequence sees, its queries being the last of its keys."""
    i = torch.arange(Lq, device=n_q.device)[:, None]
    j = torch.arange(Lk, device=n_q.device)
    p = (n_k - n_q)[:, None, None] + i
    see = (j <= p) & (j < n_k[:, None, None])
    if window > 0:
        see &= (j > p - window) | (j < sinks)
    return see


def _own_keys(s):
    case = s["case"]
    n_q = s["cu_q"].diff().long()
    n_k = (s["k_len"] if s["k_len"] is not None else s["cu_k"].diff()).long()
    q, real = _padded(s["q"], s["cu_q"][:-1].long(), n_q, s["q_max"])
    k, held = _padded(s["k"], s["cu_k"][:-1].long(), n_k, s["k_max"])
    v, _ = _padded(s["v"], s["cu_k"][:-1].long(), n_k, s["k_max"])
    k, v = k * held[:, None, :, None], v * held[:, None, :, None]
    see = _window_mask(n_q, n_k, s["q_max"], s["k_max"], case.get("window", 0), case.get("sinks", 0))
    group = case["q_heads"] // case["k_heads"]
    return _grouped(q, case["k_heads"]), k, v, see.repeat(1, group, 1)[:, None], real, (n_q, n_k)


def _plain_window(s):
    case = s["case"]
    q, k, v, see, real, (n_q, n_k) = _own_keys(s)
    B, Hq, Hk, D, Lq = len(n_q), case["q_heads"], case["k_heads"], case["dim"], s["q_max"]
    scale = 1.0 / math.sqrt(D)
    p, total, top = _sums(q, k, v, scale, see)
    lse = top + total.log()
    p /= torch.where(total > 0, total, 1.0)
    o = p @ v
    T = s["q"].shape[0]
    result = (_packed(o.reshape(B, Hq, Lq, D), s["cu_q"], T).to(BF16),)
    if case["lse"]:
        result += (_packed(lse.reshape(B, Hq, Lq, 1), s["cu_q"], T)[..., 0].contiguous(),)
    if case["op"] == "window":
        return result
    do, _ = _padded(s["dout"], s["cu_q"][:-1].long(), n_q, Lq)
    do = _grouped(do * real[:, None, :, None], Hk)
    dv = p.transpose(-1, -2) @ do
    ds = do @ v.transpose(-1, -2)
    ds -= (do * o).sum(-1, keepdim=True)
    ds *= p
    ds *= scale
    dq = (ds @ k).reshape(B, Hq, Lq, D)
    dk = ds.transpose(-1, -2) @ q
    S = s["k"].shape[0]
    return result + (_packed(dq, s["cu_q"], T).to(BF16), _packed(dk, s["cu_k"], S).to(BF16),
                     _packed(dv, s["cu_k"], S).to(BF16))


def _plain_prefix(s):
    case = s["case"]
    q, k, v, see, _, (n_q, _) = _own_keys(s)
    B, G, Hq, Hk, D, Lq = len(n_q), case["groups"], case["q_heads"], case["k_heads"], case["dim"], s["q_max"]
    scale, T = 1.0 / math.sqrt(D), s["q"].shape[0]
    p, own_total, own_top = _sums(q, k, v, scale, see)
    own_o = p @ v

    def rows(x, cu, L):
        return _packed(x.reshape(-1, Hq, L, x.shape[-1]), cu, T)

    own_o, own_total, own_top = (rows(x, s["cu_q"], Lq) for x in (own_o, own_total, own_top))
    # the prefix of each group, for the queries of all its sequences at once
    cu = s["cu_q"][s["cu_group"].long()]
    L = s["group_q_max"]
    q, _ = _padded(s["q"], cu[:-1].long(), cu.diff().long(), L)
    n_p = s["cu_prefix"].diff().long()
    k, held = _padded(s["k_prefix"], s["cu_prefix"][:-1].long(), n_p, s["p_max"])
    v, _ = _padded(s["v_prefix"], s["cu_prefix"][:-1].long(), n_p, s["p_max"])
    p, total, top = _sums(_grouped(q, Hk), k, v, scale, held[:, None, None])
    o, total, top = (rows(x, cu, L) for x in (p @ v, total, top))
    most = torch.maximum(torch.where(own_total > 0, own_top, -math.inf), torch.where(total > 0, top, -math.inf))
    most = torch.where(torch.isfinite(most), most, 0.0)
    a, b = (own_top - most).exp() * (own_total > 0), (top - most).exp() * (total > 0)
    both = a * own_total + b * total
    out = ((a * own_o + b * o) / torch.where(both > 0, both, 1.0)).to(BF16)
    return (out, (most + both.log())[..., 0].contiguous()) if case["lse"] else (out,)


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import vision_encoder_varlen_gb300 as vit
    case = s["case"]
    if case["op"] == "prefix":
        out = vit.prefix_attn(s["q"], s["k_prefix"], s["v_prefix"], s["k"], s["v"], s["cu_q"], s["cu_prefix"],
                              s["cu_k"], s["cu_group"], s["q_max"], s["p_max"], s["k_max"], k_len=s["k_len"],
                              return_lse=case["lse"])
        return out if case["lse"] else (out,)
    window = case["window"] or None
    out = vit.window_attn(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["q_max"], s["k_max"], window,
                          case["sinks"], k_len=s["k_len"], return_lse=case["lse"])
    if case["op"] == "window":
        return out if case["lse"] else (out,)
    out, lse = out
    return (out, lse) + vit.window_attn_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_q"], s["cu_k"],
                                            s["q_max"], s["k_max"], window, case["sinks"])


def run(state):
    if own:
        return _own(state)
    return _plain_prefix(state) if state["case"]["op"] == "prefix" else _plain_window(state)


# ------------------------------------------------------------------ what a pass cannot do without

def _seen(n_q, n_k, window, sinks):
    """(pairs of query and visible key, keys that some query sees) of one sequence."""
    pairs, first = 0, max(0, n_k - n_q)
    if n_k == 0:
        return 0, 0
    if window == 0:
        return sum(range(first + 1, n_k + 1)), n_k
    for p in range(first, n_k):
        pairs += min(p + 1, window) + min(sinks, max(0, p + 1 - window))
    low = max(0, first - window + 1)
    return pairs, n_k - low + min(sinks, low)


def work(case):
    ql, kl = _lengths(case)
    D, Hq, Hk = case["dim"], case["q_heads"], case["k_heads"]
    seen = [_seen(a, b, case.get("window", 0), case.get("sinks", 0)) for a, b in zip(ql, kl)]
    pairs, keys = sum(x[0] for x in seen), sum(x[1] for x in seen)
    lists = 8 * (case["batch"] + 1) + (4 * case["batch"] if case["padded"] else 0)
    if case["op"] == "prefix":
        pl, members = _prefixes(case)
        at = 0
        for p, m in zip(pl, members):
            pairs += p * sum(ql[at:at + m])
            at += m
        keys += sum(pl)
        lists += 8 * (case["groups"] + 1)
    qn, kn = sum(ql) * Hq * D, keys * Hk * D
    lse = 4 * sum(ql) * Hq if case["lse"] else 0
    if case["op"] == "window_train":
        return {"bytes": 8 * qn + 8 * kn + lse + lists, "flops": 14 * pairs * Hq * D}
    return {"bytes": 4 * qn + 4 * kn + lse + lists, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    """Query block by query block, over the keys that the block can see alone."""
    if work(case)["flops"] > 1.5e12:
        return None
    s = prepare(case, seed)
    ql, kl = _lengths(case)
    D, Hq, Hk = case["dim"], case["q_heads"], case["k_heads"]
    window, sinks, train = case.get("window", 0), case.get("sinks", 0), case["op"] == "window_train"
    out = torch.zeros(*s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(out)
    dk = torch.zeros(*s["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    prefix_of = []
    if case["op"] == "prefix":
        pl, members = _prefixes(case)
        at = 0
        for p, m in zip(pl, members):
            prefix_of += [(at, at + p)] * m
            at += p
    row, key = 0, 0
    for b, (m, n) in enumerate(zip(ql, kl)):
        for i0 in range(0, m, 1024):
            i1 = min(m, i0 + 1024)
            pos = torch.arange(n - m + i0, n - m + i1, device="cuda")
            low = 0 if window == 0 else max(0, n - m + i0 - window + 1)
            j = torch.arange(n, device="cuda")
            j = j[(j >= low) | (j < sinks)]
            behind = pos[:, None] - j[None]
            hidden = behind < 0
            if window > 0:
                hidden |= (behind >= window) & (j >= sinks)
            for h in range(Hq):
                at, of = (slice(row + i0, row + i1), h), (key + j, h // (Hq // Hk))
                q, k, v = s["q"][at].double(), s["k"][of].double(), s["v"][of].double()
                hide = hidden
                if prefix_of:
                    a, z = prefix_of[b]
                    k = torch.cat([s["k_prefix"][a:z, of[1]].double(), k])
                    v = torch.cat([s["v_prefix"][a:z, of[1]].double(), v])
                    hide = torch.cat([hidden.new_zeros(i1 - i0, z - a), hidden], 1)
                if k.shape[0] == 0:
                    continue
                score = (q @ k.T / math.sqrt(D)).masked_fill(hide, -math.inf)
                lse[at] = torch.logsumexp(score, -1)
                p = torch.softmax(score, -1).nan_to_num(nan=0.0)
                out[at] = p @ v
                if train:
                    do = s["dout"][at].double()
                    dv[of] += p.T @ do
                    dp = do @ v.T
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
                    dq[at] = ds @ k
                    dk[of] += ds.T @ q
        row, key = row + m, key + (max(kl) if case["padded"] else n)
    result = (out, lse) if case["lse"] else (out,)
    return result + (dq, dk, dv) if train else result
