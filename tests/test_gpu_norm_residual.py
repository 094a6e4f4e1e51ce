"""The residual step with the norms on either side, and its gradient, against the formulas in 64 bits.

Tolerances. A bf16 output is rounded once (2^-8 of the value), an fp32 one at 2^-24; before that the
fp32 arithmetic (sums of at most 8192 squares in a tree whose serial part is at most 16 terms per
lane, 5 shuffle steps and 16 warps; rsqrtf to 2 units) is good to 64 * 2^-24 = 2^-18 of the
magnitudes that enter an element. Weight sums over n rows add (n + 64) 2^-24 of the sum of
magnitudes.
"""
import math

import pytest
import torch

import vision_encoder_varlen_gb300 as vit

pytestmark = pytest.mark.gpu
EPS = 1e-6
F32 = 2.0 ** -18


def rms(x, eps=EPS):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def close(got, ref, mag, what):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    assert torch.isfinite(got).all(), what
    err = (got.double() - ref).abs() - (half * ref.abs() + F32 * mag + 2.0 ** -130)
    assert (err <= 0).all(), f"{what}: {float(err.max()):.3e} past its bound"


def make(T, C, gate, post, pre, wide, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T * 7 + C)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = 3 * n(T, C)
    x = x if wide else x.bfloat16()
    y = (0.7 * n(T, C)).bfloat16()
    gt = None if gate is None else (0.5 + 0.3 * n(*((C,) if gate == "channel" else (T, C)))).bfloat16()
    return (x, y, gt, (1 + 0.2 * n(C)).bfloat16() if post else None, (1 + 0.2 * n(C)).bfloat16() if pre else None,
            n(T, C), n(T, C))


CASES = [
    # T, C, gate, post, pre, fp32 residual, scale
    (1, 8, "channel", True, True, False, 1.0),
    (3, 24, None, True, False, True, -0.5),
    (5, 128, "token", False, True, False, 1.0),
    (4, 2048, "channel", True, True, False, 1.0),
    (700, 256, "token", True, True, True, 0.1),
    (333, 520, "channel", False, False, False, 2.0),
    (1000, 1280, "channel", True, True, False, 0.5),
    (65, 1288, None, False, True, True, 1.0),
    (130, 4096, "token", True, True, False, 1.0),
    (77, 4104, "channel", True, True, True, 1.0),
    (400, 5120, "token", True, True, True, 1.0),
    (31, 8192, "channel", True, True, True, 1.0),
    (2, 8192, "token", False, True, False, 1.0),
    (9, 504, None, False, False, False, 1.0),
    # many rows per block (the ring goes round), and widths where the layout changes
    (3001, 5120, "token", True, True, True, 1.0),
    (5003, 640, "channel", True, True, False, 1.0),
    (6001, 512, "token", True, True, True, 1.0),
    (1501, 4096, "channel", True, True, False, 0.5),
    (903, 6144, "channel", True, True, True, 1.0),
    (701, 6152, "token", True, True, True, 1.0),
    (1103, 8192, "token", True, True, True, 1.0),
    (611, 7000, None, False, True, False, 1.0),
    (1200, 2056, "channel", True, False, True, 1.0),
    (1301, 776, "token", False, False, False, 1.0),
]


@pytest.mark.parametrize("T,C,gate,post,pre,wide,scale", CASES)
def test_forward(T, C, gate, post, pre, wide, scale):
    x, y, g, wo, wr, _, _ = make(T, C, gate, post, pre, wide)
    u = y.double()
    if post:
        u = u * rms(u) * wo.double()
    if g is not None:
        u = u * g.double()
    h = x.double() + scale * u
    mag = x.double().abs() + abs(scale) * u.abs()
    got_h, got_z = vit.norm_residual(x, y, gate=g, w_post=wo, w_pre=wr, scale=scale, eps=EPS)
    close(got_h, h, mag, "h")
    assert (got_z is None) == (not pre)
    if pre:
        r = rms(h)
        # an error of 2^-18 mag in h moves z by that times r w, and through r by at most as much in the mean
        close(got_z, h * r * wr.double(), 2 * (mag + h.abs()) * r * wr.double().abs(), "z")
    # in place, z over y, and from rows with a stride of their own: the same bits
    xs = torch.zeros(T, C + 16, device="cuda", dtype=x.dtype)[:, :C]
    xs.copy_(x)
    ys = torch.zeros(T, 2 * C, device="cuda", dtype=y.dtype)[:, C:]
    ys.copy_(y)
    h2, z2 = vit.norm_residual(xs, ys, gate=g, w_post=wo, w_pre=wr, scale=scale, eps=EPS, h_out=xs,
                               z_out=ys if pre else None)
    assert h2 is xs and torch.equal(xs, got_h) and (not pre or torch.equal(ys, got_z))


@pytest.mark.parametrize("T,C,gate,post,pre,wide,scale", CASES)
@pytest.mark.parametrize("stream_grad", [True, False])
def test_gradient(T, C, gate, post, pre, wide, scale, stream_grad):
    if not pre and not stream_grad:
        pytest.skip("no gradient arrives at all")
    h, y, g, wo, wr, dz, dh = make(T, C, gate, post, pre, wide)
    dz = dz.bfloat16() if pre else None
    dh = dh.to(h.dtype) if stream_grad else None
    status = vit.new_status()
    dx, dy, dg, dwo, dwr = vit.norm_residual_bwd(dz, dh, h, y, gate=g, w_post=wo, w_pre=wr, scale=scale, eps=EPS,
                                                 status=status)
    assert vit.read_status(status) == 0
    one = torch.ones(C, device="cuda", dtype=torch.float64)
    H, Y = h.double(), y.double()
    dH = dh.double() if stream_grad else torch.zeros_like(H)
    mH = dH.abs()
    if pre:
        r, w = rms(H), wr.double()
        hh, dn = H * r, dz.double() * w
        dH = dH + r * (dn - hh * (dn * hh).mean(-1, keepdim=True))
        mH = mH + r * (dn.abs() + hh.abs() * (dn * hh).abs().mean(-1, keepdim=True))
        terms = (dz.double() * hh).abs().sum(0)
        assert ((dwr.double() - (dz.double() * hh).sum(0)).abs() <= ((T + 64) * 2.0 ** -24 + F32) * terms).all()
    close(dx, dH, mH, "dx")
    G = one if g is None else g.double()
    W = wo.double() if post else one
    r1 = rms(Y) if post else torch.ones_like(Y[:, :1])
    yh = Y * r1
    du, mu = scale * dH * G, abs(scale) * mH * G.abs()
    if post:
        dn, mn = du * W, mu * W.abs()
        ref = r1 * (dn - yh * (dn * yh).mean(-1, keepdim=True))
        close(dy, ref, r1 * (mn + yh.abs() * (mn * yh.abs()).mean(-1, keepdim=True)), "dy")
        terms = (mu * yh.abs()).sum(0)
        assert ((dwo.double() - (du * yh).sum(0)).abs() <= ((T + 64) * 2.0 ** -24 + 2 * F32) * terms).all()
    else:
        close(dy, du, mu, "dy")
    dgate, mg = scale * dH * yh * W, abs(scale) * mH * (yh * W).abs()
    if gate == "token":
        close(dg, dgate, 2 * mg, "dgate")
    elif gate == "channel":
        assert ((dg.double() - dgate.sum(0)).abs() <= ((T + 64) * 2.0 ** -24 + 2 * F32) * mg.sum(0)).all()
    else:
        assert dg is None
    again = vit.norm_residual_bwd(dz, dh, h, y, gate=g, w_post=wo, w_pre=wr, scale=scale, eps=EPS)
    for a, b in zip((dx, dy, dg, dwo, dwr), again):
        assert (a is None and b is None) or torch.equal(a, b)


def test_gradient_against_differences():
    T, C, scale, e = 6, 640, 0.7, 1e-4
    x, y, g, wo, wr, dz, dh = make(T, C, "channel", True, True, True)
    dz = dz.bfloat16()

    def forward(x, y, g, wo, wr):
        h = x + scale * g * y * rms(y) * wo
        return h, h * rms(h) * wr

    ins = [t.double() for t in (x, y, g, wo, wr)]
    h = forward(*ins)[0].float()
    dx, dy, dg, dwo, dwr = vit.norm_residual_bwd(dz, dh, h, y, gate=g, w_post=wo, w_pre=wr, scale=scale, eps=EPS)
    gen = torch.Generator(device="cuda").manual_seed(8)
    for i, got in enumerate((dx, dy, dg, dwo, dwr)):
        d = torch.randn(ins[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        vals = []
        for s in (1, -1):
            moved = list(ins)
            moved[i] = ins[i] + s * e * d
            hh, zz = forward(*moved)
            vals.append(float((hh * dh.double()).sum() + (zz * dz.double()).sum()))
        slope = (vals[0] - vals[1]) / (2 * e)
        tol = float((got.double().abs() * d.abs()).sum()) * 2.0 ** -7 + 1e-4
        assert abs(slope - float((got.double() * d).sum())) <= tol, i


def test_empty_and_graph():
    x, y, g, wo, wr, dz, dh = make(0, 1280, "channel", True, True, False)
    h, z = vit.norm_residual(x, y, gate=g, w_post=wo, w_pre=wr)
    assert h.shape == z.shape == (0, 1280)
    grads = vit.norm_residual_bwd(dz.bfloat16(), dh.bfloat16(), x, y, gate=g, w_post=wo, w_pre=wr)
    assert all((t == 0).all() for t in grads[2:])
    x, y, g, wo, wr, dz, dh = make(500, 1280, "channel", True, True, False)
    dz, dh = dz.bfloat16(), dh.bfloat16()
    want = vit.norm_residual(x, y, gate=g, w_post=wo, w_pre=wr) + vit.norm_residual_bwd(
        dz, dh, x, y, gate=g, w_post=wo, w_pre=wr)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = vit.norm_residual(x, y, gate=g, w_post=wo, w_pre=wr) + vit.norm_residual_bwd(
            dz, dh, x, y, gate=g, w_post=wo, w_pre=wr)
    for t in got:
        t.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_expanded_gate_is_refused():
    # an expanded row is a gate for all tokens, whose gradient is a [C] sum: it is given as [C]
    x, y, _, wo, wr, dz, dh = make(5, 64, None, True, True, False)
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: vit.norm_residual(x, y, gate=g.expand(5, 64), w_post=wo, w_pre=wr),
                 lambda: vit.norm_residual_bwd(dz.bfloat16(), None, x, y, gate=g.expand(5, 64), w_post=wo, w_pre=wr)):
        with pytest.raises(ValueError, match=r"given as \[C\]"):
            call()


def test_infinity_in_y_without_its_norm():
    # dy is the gradient times the gate where y has no norm: finite whatever y holds
    h, y, g, _, wr, dz, dh = make(300, 1280, "channel", False, True, False)
    y[7, 5], y[200, 1279] = math.inf, math.nan
    dx, dy, *_ = vit.norm_residual_bwd(dz.bfloat16(), dh.bfloat16(), h, y, gate=g, w_pre=wr)
    assert torch.isfinite(dx).all() and torch.isfinite(dy).all()
