"""The calls around a language model's reading of the encoder's states run together, as a block uses them:
positions of the clips and rotary turns of queries and states, cross attention, the gated residual step; then back
through all of them. Checked end to end against the formulas in 64 bits, and captured in a graph.

Tolerances. Forward: q and k are rounded once (e = 2^-8 of each value), so a score moves by at most
scale 2 e |q| |k| (Cauchy-Schwarz) =: t, plus fp32 sums far below it; p by at most 2.1 t of itself, once more e for
its rounding; out by (2.1 t + e) sum p |v| + e |out|. h and z come from the stored out: h is off by its own rounding,
z = RMSNorm(h) w by r |w| (H + |h| |H|_2 / |h|_2), H the fp32 error of h, and its rounding. Gradient, at the stored q, k, out, h, y: dy is rounded (e |dy|); P and dS are rounded (e of each);
delta is a sum over the stored out, off by e (sum p |v| + |out|). Every bound is carried through the next linear
step by magnitudes, and each stored result adds e of itself. fp32 arithmetic adds less than 2^-15 of the magnitudes.
"""
import math

import pytest
import torch

import vision_encoder_varlen_gb300 as vit

pytestmark = pytest.mark.gpu
E = 2.0 ** -8
F = 2.0 ** -15


def angles(pos, freq, sec):
    D2 = freq.numel()
    axis = torch.zeros(D2, dtype=torch.long, device=pos.device)
    axis[sec[0]:sec[0] + sec[1]] = 1
    axis[sec[0] + sec[1]:] = 2
    return pos.double()[:, axis] * freq.double()             # [T, D/2]


def turned(x, a, sign=1):
    D2 = a.shape[1]
    c, s = a.cos()[:, None], sign * a.sin()[:, None]
    x1, x2 = x[..., :D2], x[..., D2:]
    return torch.cat((x1 * c - x2 * s, x2 * c + x1 * s), -1)


def normed(x, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def norm_back(x, w, g, eps, mag=False):
    """Gradient of normed at x, or a bound of it for |g| <= mag'd g."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    dn = g * (w.abs() if mag else w)
    if mag:
        return r * (dn + xh.abs() * (dn * xh.abs()).mean(-1, keepdim=True))
    return r * (dn - xh * (dn * xh).mean(-1, keepdim=True))


class Block:
    """One reading block's tensors and calls."""

    def __init__(self, grids, q_lens, Hq, Hk, D, wide, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.r = r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        bf = lambda *s: r(*s).bfloat16()
        self.Hq, self.Hk, self.D, self.C, self.eps = Hq, Hk, D, Hq * D, 1e-6
        self.grid = torch.tensor(grids, dtype=torch.int32, device="cuda").reshape(-1, 3)
        self.k_lens = [t * h * w for t, h, w in grids]
        self.q_lens = q_lens
        self.Tq, self.Tk = sum(q_lens), sum(self.k_lens)
        self.cu_q = torch.tensor([0] + list(torch.tensor(q_lens).cumsum(0)), dtype=torch.int32, device="cuda")
        self.q_pos = torch.randint(0, 5000, (self.Tq, 3), generator=g, device="cuda", dtype=torch.int32)
        self.freq = (10000.0 ** (-torch.arange(D // 2, device="cuda").double() / (D // 2))).float()
        self.sec = (D // 2 - 2 * (D // 8), D // 8, D // 8)
        self.q, self.k, self.v = bf(self.Tq, Hq, D), bf(self.Tk, Hk, D), bf(self.Tk, Hk, D)
        self.w = (0.5 + 0.05 * r(2, D)).bfloat16()
        self.x = r(self.Tq, self.C) if wide else bf(self.Tq, self.C)
        self.gate, self.w_post, self.w_pre = bf(self.C), (1 + 0.1 * r(self.C)).bfloat16(), (1 + 0.1 * r(self.C)).bfloat16()
        self.dz, self.dh = bf(self.Tq, self.C), bf(self.Tq, self.C).to(self.x.dtype)
        self.max_q, self.max_k = max(q_lens), max(self.k_lens)

    def forward(self, stream=None):
        n = self
        n.k_pos, n.cu_k = vit.grid_positions(n.grid, n.Tk, stream=stream)
        n.qr, _ = vit.qk_norm_mrope(n.q, None, n.q_pos, n.freq, n.sec, n.w, n.eps, stream=stream)
        _, n.kr = vit.qk_norm_mrope(None, n.k, n.k_pos, n.freq, n.sec, n.w, n.eps, stream=stream)
        n.y, n.lse = vit.cross_attn(n.qr, n.kr, n.v, n.cu_q, n.cu_k, n.max_q, n.max_k, return_lse=True, stream=stream)
        n.h, n.z = vit.norm_residual(n.x, n.y.view(n.Tq, n.C), gate=n.gate, w_post=n.w_post, w_pre=n.w_pre, eps=n.eps,
                                     stream=stream)
        return n.h, n.z

    def backward(self, stream=None):
        n = self
        n.dx, dy, n.dgate, n.dw_post, n.dw_pre = vit.norm_residual_bwd(
            n.dz, n.dh, n.h, n.y.view(n.Tq, n.C), gate=n.gate, w_post=n.w_post, w_pre=n.w_pre, eps=n.eps,
            stream=stream)
        dqr, dkr, n.dv = vit.cross_attn_bwd(dy.view(n.Tq, n.Hq, n.D), n.qr, n.kr, n.v, n.y, n.lse, n.cu_q, n.cu_k,
                                            n.max_q, n.max_k, stream=stream)
        n.dq, _, dw0 = vit.qk_norm_mrope_bwd(dqr, None, n.q, None, n.q_pos, n.freq, n.sec, n.w, n.eps, stream=stream)
        _, n.dk, dw1 = vit.qk_norm_mrope_bwd(None, dkr, None, n.k, n.k_pos, n.freq, n.sec, n.w, n.eps, stream=stream)
        n.dw = torch.stack((dw0[0], dw1[1]))
        return n.dx, n.dgate, n.dw_post, n.dw_pre, n.dq, n.dk, n.dv, n.dw

    def heads(self, k):
        return k.repeat_interleave(self.Hq // self.Hk, 1)

    def pairs(self):
        q0 = k0 = 0
        for a, b in zip(self.q_lens, self.k_lens):
            yield slice(q0, q0 + a), slice(k0, k0 + b)
            q0, k0 = q0 + a, k0 + b


def close(got, want, tol, what):
    bad = (got.double() - want).abs() - tol
    assert not (bad > 0).any() and not torch.isnan(got).any(), (what, bad.max().item())


def check_forward(n):
    D, C = n.D, n.C
    pos = torch.cat([torch.stack(torch.meshgrid(*(torch.arange(s) for s in g), indexing="ij"), -1).reshape(-1, 3)
                     for g in n.grid.tolist()]).to("cuda")
    assert torch.equal(n.k_pos.long(), pos)
    q = turned(normed(n.q.double(), n.w[0].double(), n.eps), angles(n.q_pos, n.freq, n.sec))
    k = turned(normed(n.k.double(), n.w[1].double(), n.eps), angles(pos, n.freq, n.sec))
    v = n.v.double()
    y, Y = torch.zeros_like(q), torch.zeros_like(q)
    scale = 1 / math.sqrt(D)
    for a, b in n.pairs():
        if b.stop == b.start or a.stop == a.start:
            continue
        kk, vv = n.heads(k[b]), n.heads(v[b])
        p = torch.softmax(scale * torch.einsum("qhd,khd->hqk", q[a], kk), -1)
        t = scale * 2 * E * torch.einsum("qh,kh->hqk", q[a].norm(dim=-1), kk.norm(dim=-1)).amax(-1)
        y[a] = torch.einsum("hqk,khd->qhd", p, vv)
        Y[a] = (2.1 * t.T[..., None] + E + F) * torch.einsum("hqk,khd->qhd", p, vv.abs()) + E * y[a].abs()
    close(n.y, y, Y, "y")
    x, w1, w2, g = n.x.double(), n.w_post.double(), n.w_pre.double(), n.gate.double()

    u = g * normed(n.y.double().view(-1, C), w1, n.eps)        # from the stored y
    h = x + u
    close(n.h, h, F * (x.abs() + u.abs()) + (E * h.abs() if n.h.dtype == torch.bfloat16 else 0), "h")
    z = normed(h, w2, n.eps)
    H = F * (x.abs() + u.abs())
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + n.eps)
    moved = r * w2.abs() * (H + h.abs() * H.norm(dim=-1, keepdim=True) / h.norm(dim=-1, keepdim=True))
    close(n.z, z, 1.05 * moved + (E + F) * z.abs(), "z")


def check_backward(n):
    D, C = n.D, n.C
    d = lambda t: t.double()
    q, k, v = d(n.qr), d(n.kr), d(n.v)
    y, h, g, w1, w2 = d(n.y).view(-1, C), d(n.h), d(n.gate), d(n.w_post), d(n.w_pre)
    dH = d(n.dh) + norm_back(h, w2, d(n.dz), n.eps)
    mag = d(n.dh).abs() + norm_back(h, w2, d(n.dz).abs(), n.eps, mag=True)
    close(n.dx, dH, F * mag + (E * dH.abs() if n.dx.dtype == torch.bfloat16 else 0), "dx")
    r1 = torch.rsqrt((y * y).mean(-1, keepdim=True) + n.eps)
    r2 = torch.rsqrt((h * h).mean(-1, keepdim=True) + n.eps)
    close(n.dw_pre, (d(n.dz) * h * r2).sum(0), F * (d(n.dz) * h * r2).abs().sum(0), "dw_pre")
    close(n.dw_post, (dH * g * y * r1).sum(0), F * (mag * (g * y * r1).abs()).sum(0), "dw_post")
    close(n.dgate, (dH * y * r1 * w1).sum(0), F * (mag * (y * r1 * w1).abs()).sum(0), "dgate")
    dy = norm_back(y, w1, dH * g, n.eps).view(-1, n.Hq, D)
    DY = E * dy.abs() + F * norm_back(y, w1, mag * g.abs(), n.eps, mag=True).view(-1, n.Hq, D)
    dq, dk, dv = (torch.zeros_like(t) for t in (q, k, v))
    DQ, DK, DV = (torch.zeros_like(t) for t in (q, k, v))
    scale = 1 / math.sqrt(D)
    grp = lambda t: t.view(t.shape[0], n.Hk, n.Hq // n.Hk, D).sum(2)
    es = lambda p, t: torch.einsum("hqk,qhd->khd", p, t)
    eo = lambda p, t: torch.einsum("hqk,khd->qhd", p, t)
    for a, b in n.pairs():
        if b.stop == b.start or a.stop == a.start:
            continue
        kk, vv, do, DO = n.heads(k[b]), n.heads(v[b]), dy[a], DY[a]
        p = torch.softmax(scale * torch.einsum("qhd,khd->hqk", q[a], kk), -1)
        dp = torch.einsum("qhd,khd->hqk", do, vv)
        o = eo(p, vv)
        delta = (do * o).sum(-1).T[..., None]
        ds = p * (dp - delta)
        O = E * (eo(p, vv.abs()) + o.abs())                   # the stored out
        dp_e = torch.einsum("qhd,khd->hqk", DO + F * do.abs(), vv.abs())
        de_e = (DO * o.abs() + (do.abs() + DO) * O).sum(-1).T[..., None]
        DS = 1.05 * p * (dp_e + de_e) + (E + F) * ds.abs() + F * p * (dp.abs() + delta.abs())
        dv[b] = grp(es(p, do))
        DV[b] = grp(es(p, 1.05 * DO + (E + F) * do.abs())) + E * dv[b].abs()
        dq[a] = scale * eo(ds, kk)
        DQ[a] = scale * eo(DS + F * ds.abs(), kk.abs()) + E * dq[a].abs()
        dk[b] = scale * grp(es(ds, q[a]))
        DK[b] = scale * grp(es(DS + F * ds.abs(), q[a].abs())) + E * dk[b].abs()
    close(n.dv, dv, DV, "dv")
    for name, raw, dr, DR, pos, w, dw in (("dq", n.q, dq, DQ, n.q_pos, n.w[0], n.dw[0]),
                                          ("dk", n.k, dk, DK, n.k_pos, n.w[1], n.dw[1])):
        a, x = angles(pos, n.freq, n.sec), d(raw)
        dz = turned(dr, a, -1)
        half = DR + F * dr.abs()
        DZ = torch.cat((half[..., :D // 2] + half[..., D // 2:],) * 2, -1)     # a turn mixes the two of a pair
        want = norm_back(x, d(w), dz, n.eps)
        tol = norm_back(x, d(w), DZ + F * dz.abs(), n.eps, mag=True)
        close(getattr(n, name), want, tol + E * want.abs(), name)
        xh = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + n.eps)
        close(dw, (dz * xh).sum((0, 1)), ((DZ + F * dz.abs()) * xh.abs()).sum((0, 1)), name + " weight")


SHAPES = {
    "prompts": ([(1, 9, 13), (3, 8, 8), (1, 1, 1)], [70, 33, 5], 8, 2, 64, False),
    "single tokens": ([(1, 16, 16), (4, 10, 11), (1, 20, 21)], [1, 1, 1], 8, 4, 128, False),
    "no states, no queries": ([(1, 6, 7), (0, 4, 4), (2, 5, 5)], [20, 9, 0], 4, 4, 80, True),
    "grouped, wide": ([(2, 12, 12), (1, 30, 30)], [150, 260], 16, 2, 96, True),
    "one small head": ([(1, 3, 3)], [17], 1, 1, 32, False),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_block(name):
    n = Block(*SHAPES[name])
    n.forward()
    n.backward()
    check_forward(n)
    check_backward(n)


def test_block_captured():
    """The whole block, forward and back, in one graph: replayed with other values, the same as the calls made anew."""
    shape = SHAPES["grouped, wide"]
    n = Block(*shape)
    n.forward(), n.backward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n.forward(), n.backward()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = n.forward() + n.backward()
    m = Block(*shape, seed=1)
    # other lengths in the same buffers, within the captured bounds
    m.q_lens, m.cu_q = [155, 255], torch.tensor([0, 155, 410], dtype=torch.int32, device="cuda")
    m.grid, m.k_lens, m.Tk = torch.tensor([[4, 9, 8], [1, 30, 30]], dtype=torch.int32, device="cuda"), [288, 900], 1188
    for t in ("q", "k", "v", "w", "x", "gate", "w_post", "w_pre", "dz", "dh", "q_pos", "grid", "cu_q"):
        getattr(n, t).copy_(getattr(m, t))
    graph.replay()
    torch.cuda.synchronize()
    want = m.forward() + m.backward()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_blocks_on_two_streams():
    """Two blocks at once, each on a stream of its own that it is given, while the current stream reuses memory."""
    blocks = [Block(*SHAPES["prompts"], seed=i) for i in range(2)]
    want = [b.forward() + b.backward() for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(5):
        got = [b.forward(s) for b, s in zip(blocks, streams)]
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        for g, b, s in zip(got, blocks, streams):
            with torch.cuda.stream(s):                         # dw of the block is stacked there
                got[blocks.index(b)] = g + b.backward(s)
        del junk
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """States whose element offsets pass 2^32: a cache of 5 GB each for k and v, read near its end."""
    Hk, D, T = 8, 128, 2 ** 32 // 1024 + 1000
    k = torch.zeros(T, Hk, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = torch.randn(2, 600, Hk, D, generator=g, device="cuda").bfloat16()
    k[-600:], v[-600:] = tail[0], tail[1]
    for Tq in (1, 40):
        q = torch.randn(Tq, 2 * Hk, D, generator=g, device="cuda").bfloat16()
        cu_q = torch.tensor([0, Tq], dtype=torch.int32, device="cuda")
        far = vit.cross_attn(q, k, v, cu_q, torch.tensor([T - 600, T], dtype=torch.int32, device="cuda"), Tq, 600,
                             return_lse=True)
        near = vit.cross_attn(q, tail[0], tail[1], cu_q, torch.tensor([0, 600], dtype=torch.int32, device="cuda"), Tq,
                              600, return_lse=True)
        assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
        do = torch.randn(Tq, 2 * Hk, D, generator=g, device="cuda").bfloat16()
        a = vit.cross_attn_bwd(do, q, tail[0], tail[1], *near, cu_q,
                               torch.tensor([0, 600], dtype=torch.int32, device="cuda"), Tq, 600)
        b = vit.cross_attn_bwd(do, q, k, v, *far, cu_q, torch.tensor([T - 600, T], dtype=torch.int32, device="cuda"),
                               Tq, 600)
        assert torch.equal(a[0], b[0])
        for x, y in zip(a[1:], b[1:]):
            assert torch.equal(x, y[-600:]) and not y[:-600].any()
    x = torch.zeros(T, Hk, D, dtype=torch.bfloat16, device="cuda")
    x[-600:] = tail[0]
    freq = torch.rand(D // 2, generator=g, device="cuda")
    pos = torch.randint(0, 99, (T, 3), generator=g, device="cuda", dtype=torch.int32)
    vit.qk_norm_mrope(None, x, pos, freq, (20, 22, 22), inplace=True)
    _, want = vit.qk_norm_mrope(None, tail[0], pos[-600:].contiguous(), freq, (20, 22, 22))
    assert torch.equal(x[-600:], want) and not x[:-600].any()
    h, _ = vit.norm_residual(k.view(T, -1), x.view(T, -1), scale=2.0)
    # the sum is exact in fp32 (two bf16 values, a power of two) up to its rounding and one more to bf16
    want = (tail[0].double() + 2 * want.double()).view(600, -1)
    close(h[-600:], want, (2.0 ** -8 + 2.0 ** -22) * want.abs() + 1e-30, "h")


@pytest.mark.parametrize("Lq", [1, 33])
def test_most_sequences(Lq):
    """As many sequences as a call takes: 1 or 33 queries each, 0 to 7 states; one more is refused."""
    B, Hq, Hk, D, most = 8192, 2, 1, 64, 7
    g = torch.Generator(device="cuda").manual_seed(5)
    n = torch.randint(0, most + 1, (B,), generator=g, device="cuda")
    cu_k = torch.cat((n.new_zeros(1), n.cumsum(0))).int()
    cu_q = torch.arange(B + 1, device="cuda", dtype=torch.int32) * Lq
    r = lambda T, H: torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    q, k, v, do = r(B * Lq, Hq), r(int(cu_k[-1]), Hk), r(int(cu_k[-1]), Hk), r(B * Lq, Hq)
    status = vit.new_status()
    out, lse = vit.cross_attn(q, k, v, cu_q, cu_k, Lq, most, return_lse=True, status=status)
    dq, dk, dv = vit.cross_attn_bwd(do, q, k, v, out, lse, cu_q, cu_k, Lq, most, status=status)
    assert vit.read_status(status) == 0
    # padded to 7 states in 64 bits
    at = (cu_k[:-1, None] + torch.arange(most, device="cuda")).clamp(max=int(cu_k[-1]) - 1).long()
    there = (torch.arange(most, device="cuda") < n[:, None])[:, None, None]
    K, V = (t[at, 0].double().masked_fill(~there[:, 0, 0, :, None], 0.0) for t in (k, v))
    Q, DO = (t.view(B, Lq, Hq, D).double() for t in (q, do))
    s = (torch.einsum("bqhd,bkd->bqhk", Q, K) / 8).masked_fill(~there, -math.inf)
    p = torch.softmax(s, -1).nan_to_num(0.0)
    o = torch.einsum("bqhk,bkd->bqhd", p, V)
    mag = torch.einsum("bqhk,bkd->bqhd", p, V.abs())
    close(out.view(B, Lq, Hq, D), o, E * o.abs() + 1.01 * E * mag, "out")
    dP = torch.einsum("bqhd,bkd->bqhk", DO, V)
    dl, dm = (DO * o).sum(-1, keepdim=True), (DO.abs() * (o.abs() + mag)).sum(-1, keepdim=True)
    ds = p * (dP - dl)
    DS = 1.01 * (E * ds.abs() + p * E * dm) + F * p * (dP.abs() + dl.abs())
    want = torch.einsum("bqhk,bkd->bqhd", ds, K) / 8
    close(dq.view(B, Lq, Hq, D), want, torch.einsum("bqhk,bkd->bqhd", DS, K.abs()) / 8 + E * want.abs(), "dq")
    rows = there[:, 0, 0]
    want = torch.einsum("bqhk,bqhd->bkd", ds, Q)[rows] / 8
    close(dk[:, 0], want, (torch.einsum("bqhk,bqhd->bkd", DS, Q.abs()) / 8)[rows] + E * want.abs(), "dk")
    want = torch.einsum("bqhk,bqhd->bkd", p, DO)[rows]
    close(dv[:, 0], want, 1.01 * E * torch.einsum("bqhk,bqhd->bkd", p, DO.abs())[rows] + E * want.abs(), "dv")
    with pytest.raises(vit.VitError, match="-7"):
        vit.cross_attn(q, k, v, torch.cat((cu_q, cu_q[-1:])), torch.cat((cu_k, cu_k[-1:])), Lq, most)
