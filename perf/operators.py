"""The measured cases of the operators around a language model's reading of the encoder's states:
rotary positions with three axes, cross attention, and the gated residual with its norms.

``run`` computes each operator in a plain form (elementary torch operations in 32 bits) or, where
``own`` is true, through the package's entry points.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of three sequences: latency
        dict(name="mrope_step", op="mrope", tokens=3, q_heads=32, k_heads=8, dim=128, norm=True, cycled=True,
             interleaved=False, far=65536, grid=False),
        # a packed batch of images and short clips, positions made from their grids
        dict(name="mrope_clips", op="mrope", tokens=0, clips=24, side=40, frames=3, q_heads=16, k_heads=16, dim=80,
             norm=True, cycled=False, interleaved=False, far=0, grid=True),
        # the gradient of the same call over long text and video positions
        dict(name="mrope_grad", op="mrope_grad", tokens=40013, q_heads=16, k_heads=4, dim=128, norm=True, cycled=True,
             interleaved=False, far=1 << 20),
        # serving: one new token of each of three sequences reads its image (one has a single state)
        dict(name="cross_step", op="cross", batch=3, q_lo=1, q_max=1, k_lo=1, k_max=1601, lens=11, empty=False,
             q_heads=32, k_heads=8, dim=128, lse=False),
        # serving: a full batch of single tokens over ragged states, one of them without any
        dict(name="cross_step_batch", op="cross", batch=48, q_lo=1, q_max=1, k_lo=60, k_max=8191, lens=12, empty=True,
             q_heads=32, k_heads=8, dim=128, lse=False),
        # a resampler: 64 latent queries read each image
        dict(name="cross_latents", op="cross", batch=16, q_lo=64, q_max=64, k_lo=256, k_max=4097, lens=13, empty=False,
             q_heads=16, k_heads=16, dim=80, lse=False),
        # prefill: prompts over the states of several large images, with the log-sum-exp
        dict(name="cross_prefill", op="cross", batch=4, q_lo=700, q_max=2047, k_lo=6404, k_max=16389, lens=14,
             empty=False, q_heads=32, k_heads=8, dim=128, lse=True),
        # training, short ragged sequences, one without states
        dict(name="cross_train_short", op="cross_train", batch=9, q_lo=1, q_max=131, k_lo=1, k_max=700, lens=15,
             empty=True, q_heads=8, k_heads=2, dim=64, lse=True),
        # training, long sequences
        dict(name="cross_train_long", op="cross_train", batch=4, q_lo=1500, q_max=2311, k_lo=3000, k_max=5117, lens=16,
             empty=False, q_heads=16, k_heads=16, dim=80, lse=True),
        # one decoding step through a gated block: latency
        dict(name="norm_step", op="norm", tokens=4, width=2048, gate="channel", post=True, pre=True, wide=False,
             scale=1.0),
        # the encoder's width over a full packed batch
        dict(name="norm_batch", op="norm", tokens=37007, width=1280, gate="channel", post=True, pre=True, wide=False,
             scale=0.5),
        # the gradient with a 32-bit residual stream and a gate for each token
        dict(name="norm_grad", op="norm_grad", tokens=9001, width=5120, gate="token", post=True, pre=True, wide=True,
             scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["mrope", "mrope_grad", "cross", "cross", "cross_train", "norm", "norm_grad"])
    if op in ("mrope", "mrope_grad"):
        dim = rng.choice([32, 64, 80, 96, 128])
        k_heads = rng.choice([1, 2, 4, 8, 16])
        q_heads = k_heads * rng.choice([1, 1, 2, 4])
        most = min(40000, int(40000 * 20 * 128 / (dim * (q_heads + k_heads))))
        case = dict(op=op, tokens=_log_int(rng, 1, most), q_heads=q_heads, k_heads=k_heads, dim=dim,
                    norm=rng.random() < 0.75, cycled=rng.random() < 0.5, interleaved=rng.random() < 0.3,
                    far=_log_int(rng, 64, 1 << 20))
        return case if op == "mrope_grad" else dict(case, grid=False)
    if op in ("norm", "norm_grad"):
        width = 8 * _log_int(rng, 16, 1024)
        return dict(op=op, tokens=_log_int(rng, 1, min(40000, 45000000 // width)), width=width,
                    gate=rng.choice(["none", "channel", "token"]), post=rng.random() < 0.7, pre=rng.random() < 0.8,
                    wide=rng.random() < 0.4, scale=rng.choice([1.0, 0.5, 0.1]))
    dim = rng.choice([32, 64, 80, 96, 128])
    k_heads = rng.choice([1, 2, 4, 8, 16])
    q_heads = k_heads * rng.choice([1, 1, 2, 4, 8])
    while q_heads > 32:
        q_heads //= 2
    q_heads = max(q_heads, k_heads)
    batch = _log_int(rng, 1, 48)
    kind = rng.choice(["step", "few", "many"]) if op == "cross" else rng.choice(["few", "many"])
    q_max = {"step": 1, "few": _log_int(rng, 2, 100), "many": _log_int(rng, 100, 2300)}[kind]
    k_max = _log_int(rng, 1, 16000)
    # padded scores of the plain form and the products stay within the largest listed cases
    while batch * q_max * k_max * q_heads > 1.2e9 or batch * k_max * k_heads > 3.2e6:
        batch, k_max = max(1, batch // 2), max(1, int(k_max * 0.7))
    return dict(op=op, batch=batch, q_lo=max(1, q_max // rng.choice([1, 2, 8])), q_max=q_max,
                k_lo=max(1, k_max // rng.choice([1, 2, 16])), k_max=k_max, lens=rng.randrange(1 << 30),
                empty=batch > 1 and rng.random() < 0.3, q_heads=q_heads, k_heads=k_heads, dim=dim,
                lse=op == "cross_train" or rng.random() < 0.5)


def _lengths(case):
    """Query and key lengths of a cross-attention case: the first sequence has the longest of each."""
    rng = random.Random(case["lens"])
    q = [case["q_max"]] + [_log_int(rng, case["q_lo"], case["q_max"]) for _ in range(case["batch"] - 1)]
    k = [case["k_max"]] + [_log_int(rng, case["k_lo"], case["k_max"]) for _ in range(case["batch"] - 1)]
    if case["empty"]:
        k[-1] = 0
    return q, k


def _grids(case):
    """(frames, rows, columns) of each clip; a third of them are single images."""
    rng = random.Random(case["clips"] * 1000 + case["side"])
    return [(1 if i % 3 == 0 else case["frames"], rng.randint(case["side"] // 3, case["side"]),
             rng.randint(case["side"] // 3, case["side"])) for i in range(case["clips"])]


def _tokens(case):
    return sum(t * h * w for t, h, w in _grids(case)) if case.get("grid") else case["tokens"]


def _sections(dim, cycled):
    """Pairs turned by time, height and width: about 1/5, 2/5, 2/5 of dim / 2, or nearly equal shares when they cycle."""
    r = dim // 2
    h = 3 * r // 10 if cycled else 2 * r // 5
    return r - 2 * h, h, h


def _axes(sections, cycled):
    """Axis of each pair: the sections one after the other, or t, h, w in turn while height and width last."""
    t, h, w = sections
    if not cycled:
        return [0] * t + [1] * h + [2] * w
    return [1 if m % 3 == 1 and m < 3 * h else 2 if m % 3 == 2 and m < 3 * w else 0 for m in range(t + h + w)]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=BF16, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)

    op = case["op"]
    s = dict(case=case)
    if op in ("mrope", "mrope_grad"):
        T, D = _tokens(case), case["dim"]
        s["q"] = normal(T, case["q_heads"], D, scale=2.0)
        s["k"] = normal(T, case["k_heads"], D, scale=2.0)
        s["norm_w"] = normal(2, D, scale=0.2, shift=1.0) if case["norm"] else None
        s["sections"] = _sections(D, case["cycled"])
        s["axes"] = torch.tensor(_axes(s["sections"], case["cycled"]), device="cuda")
        j = torch.arange(D // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = (THETA ** (-2.0 * j / D)).float()
        if case.get("grid"):
            s["grid"] = torch.tensor(_grids(case), dtype=torch.int32, device="cuda")
        else:
            s["pos"] = torch.randint(0, case["far"], (T, 3), generator=g, device="cuda", dtype=torch.int32)
        if op == "mrope_grad":
            s["dq"] = normal(T, case["q_heads"], D, scale=0.01)
            s["dk"] = normal(T, case["k_heads"], D, scale=0.01)
    elif op in ("cross", "cross_train"):
        ql, kl = _lengths(case)
        D, Hq, Hk = case["dim"], case["q_heads"], case["k_heads"]
        s["q"] = normal(sum(ql), Hq, D)
        s["k"] = normal(max(1, sum(kl)), Hk, D)
        s["v"] = normal(max(1, sum(kl)), Hk, D)
        s["cu_q"] = torch.tensor([0] + ql, device="cuda").cumsum(0).int()
        s["cu_k"] = torch.tensor([0] + kl, device="cuda").cumsum(0).int()
        if op == "cross_train":
            s["dout"] = normal(sum(ql), Hq, D, scale=0.1)
    else:
        T, C = case["tokens"], case["width"]
        res = torch.float32 if case["wide"] else BF16
        s["x"] = normal(T, C, dtype=res, scale=3.0)
        s["y"] = normal(T, C, scale=0.7)
        s["gate"] = None if case["gate"] == "none" else normal(*((C,) if case["gate"] == "channel" else (T, C)),
                                                               scale=0.3, shift=0.5)
        s["w_post"] = normal(C, scale=0.2, shift=1.0) if case["post"] else None
        s["w_pre"] = normal(C, scale=0.2, shift=1.0) if case["pre"] else None
        if op == "norm_grad":
            s["dz"] = normal(T, C, scale=0.01) if case["pre"] else None
            s["dh"] = normal(T, C, dtype=res, scale=0.01)
    return s


# ------------------------------------------------------------------ the plain forms

def _grid_positions(grid, T):
    size = grid.long().prod(1)
    cu = torch.cat([size.new_zeros(1), size.cumsum(0)])
    t = torch.arange(T, device=grid.device)
    i = torch.searchsorted(cu[1:], t, right=True)
    off, h, w = t - cu[i], grid[i, 1].long(), grid[i, 2].long()
    return torch.stack([off // (h * w), off // w % h, off % w], 1).int(), cu.int()


def _cos_sin(s, pos):
    a = pos.double()[:, s["axes"]] * s["inv_freq"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_mrope(s):
    case = s["case"]
    made = ()
    pos = s.get("pos")
    if case.get("grid"):
        pos, cu = _grid_positions(s["grid"], s["q"].shape[0])
        made = (pos, cu)
    cos, sin = _cos_sin(s, pos)

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * _rms(x) * w.float()
        return _turn(x, cos, sin, case["interleaved"]).to(BF16)

    w = s["norm_w"]
    return (one(s["q"], None if w is None else w[0]), one(s["k"], None if w is None else w[1])) + made


def _plain_mrope_grad(s):
    cos, sin = _cos_sin(s, s["pos"])

    def one(dy, x, w):
        dz = _turn(dy.float(), cos, -sin, s["case"]["interleaved"])
        if w is None:
            return dz.to(BF16), None
        x = x.float()
        r = _rms(x)
        xh, dn = x * r, dz * w.float()
        return (r * (dn - xh * (dn * xh).mean(-1, keepdim=True))).to(BF16), (dz * xh).double().sum((0, 1)).float()

    w = s["norm_w"]
    dq, wq = one(s["dq"], s["q"], None if w is None else w[0])
    dk, wk = one(s["dk"], s["k"], None if w is None else w[1])
    return (dq, dk) if w is None else (dq, dk, torch.stack([wq, wk]))


def _padded(x, cu, most):
    """[B, heads, most, dim] in 32 bits, and which places hold a row."""
    start, n = cu[:-1].long(), cu.diff().long()
    at = torch.arange(most, device=x.device)
    held = at < n[:, None]
    rows = x[(start[:, None] + at).clamp(max=x.shape[0] - 1)].float()
    return rows.transpose(1, 2), held


def _packed(x, cu, T):
    """The rows of [B, heads, most, dim], one sequence after the other."""
    t = torch.arange(T, device=x.device)
    i = torch.searchsorted(cu[1:].long(), t, right=True)
    return x.transpose(1, 2)[i, t - cu[i]]


def _plain_cross(s):
    case = s["case"]
    q, _ = _padded(s["q"], s["cu_q"], case["q_max"])
    k, held = _padded(s["k"], s["cu_k"], case["k_max"])
    v, _ = _padded(s["v"], s["cu_k"], case["k_max"])
    B, Hq, Lq, D = q.shape
    Hk = k.shape[1]
    scale = 1.0 / math.sqrt(D)
    # the queries of one key head side by side: [B, Hk, group * Lq, D]
    q = q.reshape(B, Hk, Hq // Hk * Lq, D)
    k, v = k * held[:, None, :, None], v * held[:, None, :, None]
    score = q @ k.transpose(-1, -2)
    score *= scale
    score.masked_fill_(~held[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p /= torch.where(total > 0, total, 1.0)
    o = p @ v
    T = s["q"].shape[0]
    out = _packed(o.reshape(B, Hq, Lq, D), s["cu_q"], T).to(BF16)
    result = (out,)
    if case["lse"]:
        result += (_packed(lse.reshape(B, Hq, Lq, 1), s["cu_q"], T)[..., 0].contiguous(),)
    if case["op"] == "cross":
        return result
    do, real = _padded(s["dout"], s["cu_q"], case["q_max"])
    do = (do * real[:, None, :, None]).reshape(B, Hk, Hq // Hk * Lq, D)
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


def _plain_norm(s):
    u = s["y"].float()
    if s["w_post"] is not None:
        u = u * _rms(u) * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["x"].float() + s["case"]["scale"] * u
    if s["w_pre"] is None:
        return (h.to(s["x"].dtype),)
    return h.to(s["x"].dtype), (h * _rms(h) * s["w_pre"].float()).to(BF16)


def _plain_norm_grad(s):
    case, grads = s["case"], []
    dh = s["dh"].float()
    if s["w_pre"] is not None:
        h, dz = s["x"].float(), s["dz"].float()
        r = _rms(h)
        hh, dn = h * r, dz * s["w_pre"].float()
        dh = dh + r * (dn - hh * (dn * hh).mean(-1, keepdim=True))
        grads.append((dz * hh).double().sum(0).float())
    y = s["y"].float()
    r = _rms(y)
    yh = y * r if s["w_post"] is not None else y
    u = yh * s["w_post"].float() if s["w_post"] is not None else y
    du = case["scale"] * dh
    if s["gate"] is not None:
        dg = du * u
        grads.append(dg.to(BF16) if case["gate"] == "token" else dg.double().sum(0).float())
        du = du * s["gate"].float()
    dy = du
    if s["w_post"] is not None:
        grads.append((du * yh).double().sum(0).float())
        dn = du * s["w_post"].float()
        dy = r * (dn - yh * (dn * yh).mean(-1, keepdim=True))
    return (dh.to(s["x"].dtype), dy.to(BF16), *grads)


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import vision_encoder_varlen_gb300 as vit
    case = s["case"]
    op = case["op"]
    if op == "mrope":
        made, pos = (), s.get("pos")
        if case["grid"]:
            made = vit.grid_positions(s["grid"], s["q"].shape[0])
            pos = made[0]
        return vit.qk_norm_mrope(s["q"], s["k"], pos, s["inv_freq"], s["sections"], s["norm_w"], EPS,
                                 cycled=case["cycled"], interleaved=case["interleaved"]) + tuple(made)
    if op == "mrope_grad":
        dq, dk, dw = vit.qk_norm_mrope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["inv_freq"], s["sections"],
                                           s["norm_w"], EPS, cycled=case["cycled"], interleaved=case["interleaved"])
        return (dq, dk) if dw is None else (dq, dk, dw)
    if op in ("cross", "cross_train"):
        out = vit.cross_attn(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], case["q_max"], case["k_max"],
                             return_lse=case["lse"])
        if op == "cross":
            return out if case["lse"] else (out,)
        out, lse = out
        return (out, lse) + vit.cross_attn_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_q"], s["cu_k"],
                                               case["q_max"], case["k_max"])
    if op == "norm":
        h, z = vit.norm_residual(s["x"], s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"],
                                 scale=case["scale"], eps=EPS)
        return (h,) if z is None else (h, z)
    dx, dy, dgate, dw_post, dw_pre = vit.norm_residual_bwd(s["dz"], s["dh"], s["x"], s["y"], gate=s["gate"],
                                                           w_post=s["w_post"], w_pre=s["w_pre"], scale=case["scale"],
                                                           eps=EPS)
    return (dx, dy) + tuple(t for t in (dw_pre, dgate, dw_post) if t is not None)


def run(state):
    if own:
        return _own(state)
    return {"mrope": _plain_mrope, "mrope_grad": _plain_mrope_grad, "cross": _plain_cross,
            "cross_train": _plain_cross, "norm": _plain_norm, "norm_grad": _plain_norm_grad}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("mrope", "mrope_grad"):
        n = _tokens(case) * (case["q_heads"] + case["k_heads"]) * case["dim"]
        b = 4 * n + 12 * _tokens(case) + 2 * case["dim"] + (4 * case["dim"] if case["norm"] else 0)
        if op == "mrope":
            return {"bytes": b + (24 * case["clips"] if case["grid"] else 0), "flops": (8 if case["norm"] else 3) * n}
        return {"bytes": b + (2 * n + 8 * case["dim"] if case["norm"] else 0), "flops": (16 if case["norm"] else 3) * n}
    if op in ("cross", "cross_train"):
        ql, kl = _lengths(case)
        D, Hq, Hk = case["dim"], case["q_heads"], case["k_heads"]
        qn, kn = sum(ql) * Hq * D, sum(kl) * Hk * D
        products = sum(a * b for a, b in zip(ql, kl)) * Hq * D
        lse = 4 * sum(ql) * Hq if case["lse"] else 0
        cu = 8 * (case["batch"] + 1)
        if op == "cross":
            return {"bytes": 4 * qn + 4 * kn + lse + cu, "flops": 4 * products}
        return {"bytes": 8 * qn + 8 * kn + lse + cu, "flops": 14 * products}
    n, C = case["tokens"] * case["width"], case["width"]
    res = 4 if case["wide"] else 2
    gate = 0 if case["gate"] == "none" else C if case["gate"] == "channel" else n
    if op == "norm":
        return {"bytes": 2 * res * n + 2 * n + (2 * n if case["pre"] else 0) + 2 * gate +
                2 * C * (case["post"] + case["pre"]), "flops": n * (3 + 4 * case["post"] + 4 * case["pre"])}
    b = 2 * res * n + 2 * n + (res * n + 2 * n if case["pre"] else 0) + 2 * gate
    b += 2 * n if case["post"] or gate else 0
    b += 2 * n if case["gate"] == "token" else 4 * gate
    return {"bytes": b + 6 * C * (case["post"] + case["pre"]), "flops": n * (5 + 8 * case["post"] + 9 * case["pre"])}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rotation(case, s):
    """Row t's complex turns exp(i a), one for each pair."""
    if case.get("grid"):
        pos = [(t, h, w) for T, H, W in _grids(case) for t in range(T) for h in range(H) for w in range(W)]
        pos = torch.tensor(pos, device="cuda")
    else:
        pos = s["pos"].long()
    t, h, w = _sections(case["dim"], case["cycled"])
    axis = []
    for m in range(t + h + w):
        if case["cycled"]:
            a = m % 3
            axis.append(a if a and m < 3 * (h if a == 1 else w) else 0)
        else:
            axis.append(0 if m < t else 1 if m < t + h else 2)
    angle = torch.stack([pos[:, a].double() * s["inv_freq"][m].double() for m, a in enumerate(axis)], 1)
    return pos.int(), torch.polar(torch.ones_like(angle), angle)[:, None]


def _exact_mrope(case, s):
    pos, turn = _exact_rotation(case, s)
    R = case["dim"] // 2

    def pairs(x):
        return torch.complex(x[..., 0::2], x[..., 1::2]) if case["interleaved"] else torch.complex(x[..., :R], x[..., R:])

    def flat(z):
        return torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)

    outs, sums = [], []
    for row, name in enumerate("qk"):
        x = s[name].double()
        w = s["norm_w"][row].double() if case["norm"] else torch.ones(case["dim"], dtype=torch.float64, device="cuda")
        r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) if case["norm"] else torch.ones_like(x[..., :1])
        if case["op"] == "mrope":
            outs.append(flat(pairs(x * r * w).mul(turn)))
            continue
        d = flat(pairs(s["d" + name].double()).mul(turn.conj()))
        sums.append((d * x * r).sum((0, 1)))
        if case["norm"]:
            inner = (d * w * x).sum(-1, keepdim=True)
            outs.append(r * d * w - r ** 3 * x * inner / case["dim"])
        else:
            outs.append(d)
    if case["op"] == "mrope":
        if case["grid"]:
            ends = torch.tensor([0] + [t * h * w for t, h, w in _grids(case)]).cumsum(0).int().cuda()
            outs += [pos, ends]
        return tuple(outs)
    return tuple(outs) + ((torch.stack(sums),) if case["norm"] else ())


def _exact_cross(case, s):
    ql, kl = _lengths(case)
    D, Hq, Hk = case["dim"], case["q_heads"], case["k_heads"]
    if sum(a * b for a, b in zip(ql, kl)) * Hq * D * (14 if case["op"] == "cross_train" else 4) > 1.5e12:
        return None
    out = torch.zeros(*s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(out)
    dk = torch.zeros(*s["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    a = b = 0
    for m, n in zip(ql, kl):
        for h in range(Hq if n else 0):
            at = (slice(a, a + m), h)
            of = (slice(b, b + n), h * Hk // Hq)
            q, k, v = s["q"][at].double(), s["k"][of].double(), s["v"][of].double()
            score = q @ k.T / math.sqrt(D)
            lse[at] = torch.logsumexp(score, -1)
            p = torch.softmax(score, -1)
            out[at] = p @ v
            if case["op"] == "cross_train":
                do = s["dout"][at].double()
                dv[of] += p.T @ do
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
                dq[at] = ds @ k
                dk[of] += ds.T @ q
        a, b = a + m, b + n
    result = (out, lse) if case["lse"] else (out,)
    return result if case["op"] == "cross" else result + (dq, dk, dv)


def _exact_norm(case, s):
    one = torch.ones((), dtype=torch.float64, device="cuda")
    x, y = s["x"].double(), s["y"].double()
    gate = one if s["gate"] is None else s["gate"].double()
    post = one if s["w_post"] is None else s["w_post"].double()
    pre = one if s["w_pre"] is None else s["w_pre"].double()
    ry = one if s["w_post"] is None else 1 / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS)
    if case["op"] == "norm":
        h = x + case["scale"] * gate * post * ry * y
        return (h, h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * pre) if case["pre"] else (h,)
    C, dh, more = case["width"], s["dh"].double(), []
    if case["pre"]:
        rx = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        dz = s["dz"].double()
        dh = dh + rx * dz * pre - rx ** 3 * x * (dz * pre * x).sum(-1, keepdim=True) / C
        more.append((dz * x * rx).sum(0))
    back = case["scale"] * dh
    if case["gate"] != "none":
        dg = back * post * ry * y
        more.append(dg if case["gate"] == "token" else dg.sum(0))
    back = back * gate
    if not case["post"]:
        return (dh, back, *more)
    more.append((back * ry * y).sum(0))
    return (dh, ry * back * post - ry ** 3 * y * (back * post * y).sum(-1, keepdim=True) / C, *more)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("mrope", "mrope_grad"):
        return _exact_mrope(case, s)
    return _exact_cross(case, s) if op in ("cross", "cross_train") else _exact_norm(case, s)
