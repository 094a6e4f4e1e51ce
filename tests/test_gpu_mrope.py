"""Three-axis rotary positions with the per-head norm, and their gradient, against the formulas in 64 bits.

Tolerances. Outputs are rounded to bf16 once: at most half a step, 2^-8 of the value. Before that:
the angle is exact to 2^-24 of its reduced value (<= pi, so 2^-22), __sincosf adds 2^-21 absolute,
the norm factor and the products a few 2^-23 relative: together below 2^-19 of the magnitudes that
enter an element (the two elements of its pair). Weight sums are fp32 sums of n terms: rounding
errors below (n / parts + 64) 2^-24 of the sum of magnitudes, each term itself good to 2^-18.
"""
import math

import pytest
import torch

import vision_encoder_varlen_gb300 as vit

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8
EPS = 1e-6


def axes(sections, cycled):
    t, h, w = sections
    if not cycled:
        return [0] * t + [1] * h + [2] * w
    return [1 if m % 3 == 1 and m < 3 * h else 2 if m % 3 == 2 and m < 3 * w else 0 for m in range(t + h + w)]


def angles(pos, inv_freq, sections, cycled):
    a = torch.tensor(axes(sections, cycled), device=pos.device)
    return pos.double()[:, a] * inv_freq.double()


def turn(x, a, interleaved):
    c, s = a.cos()[:, None], a.sin()[:, None]
    if interleaved:
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
    u, v = x.chunk(2, -1)
    return torch.cat([u * c - v * s, v * c + u * s], -1)


def partner(x, interleaved):
    if interleaved:
        return torch.stack([x[..., 1::2], x[..., 0::2]], -1).flatten(-2)
    return torch.cat(list(reversed(x.chunk(2, -1))), -1)


def rms(x, eps):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def reference(x, w, a, interleaved, eps=EPS):
    """y, and the magnitude that the tolerance before rounding is relative to."""
    x = x.double()
    if w is not None:
        x = x * rms(x, eps) * w.double()
    return turn(x, a, interleaved), x.abs() + partner(x, interleaved).abs()


def reference_grad(dy, x, w, a, interleaved, eps=EPS):
    dz = turn(dy.double(), -a, interleaved)
    mag = dy.double().abs()
    mag = mag + partner(mag, interleaved)
    if w is None:
        return dz, mag, None, None
    x = x.double()
    r = rms(x, eps)
    xh, dn = x * r, dz * w.double()
    dx = r * (dn - xh * (dn * xh).mean(-1, keepdim=True))
    m = mag * w.double().abs()
    return (dx, r * (m + xh.abs() * (m * xh.abs()).mean(-1, keepdim=True)), (dz * xh).sum((0, 1)),
            (mag * xh.abs()).sum((0, 1)))


def close(got, ref, mag, what):
    err = (got.double() - ref).abs() - (BF * ref.abs() + 2.0 ** -19 * mag + 2.0 ** -130)
    assert torch.isfinite(got).all(), what
    assert (err <= 0).all(), f"{what}: {float(err.max()):.3e} past its bound"


def make(T, Hq, Hk, D, cycled, norm, far, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T + D)
    r = D // 2
    h = 3 * r // 10 if cycled else 2 * r // 5
    sections = (r - 2 * h, h, h)
    q = (2 * torch.randn(T, Hq, D, generator=g, device="cuda")).bfloat16()
    k = (2 * torch.randn(T, Hk, D, generator=g, device="cuda")).bfloat16()
    pos = torch.randint(-far, far, (T, 3), generator=g, device="cuda", dtype=torch.int32)
    inv_freq = (10000.0 ** (-2.0 * torch.arange(r, device="cuda", dtype=torch.float64) / D)).float()
    w = (1 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).bfloat16() if norm else None
    return q, k, pos, inv_freq, sections, w


CASES = [
    # T, Hq, Hk, D, cycled, interleaved, norm, far
    (1, 1, 1, 32, False, False, True, 100),
    (3, 32, 8, 128, True, False, True, 65536),
    (7, 5, 3, 80, False, True, True, 50),
    (130, 16, 16, 80, False, False, True, 4000),
    (33, 12, 1, 96, True, True, False, 1 << 20),
    (257, 9, 2, 64, True, False, False, 1 << 30),
    (2500, 4, 2, 128, False, False, True, 1 << 24),
    (641, 30, 30, 32, False, True, True, 300),
]


@pytest.mark.parametrize("T,Hq,Hk,D,cycled,il,norm,far", CASES)
def test_forward(T, Hq, Hk, D, cycled, il, norm, far):
    q, k, pos, f, sec, w = make(T, Hq, Hk, D, cycled, norm, far)
    a = angles(pos, f, sec, cycled)
    y = vit.qk_norm_mrope(q, k, pos, f, sec, w, EPS, cycled=cycled, interleaved=il)
    for got, x, row in ((y[0], q, 0), (y[1], k, 1)):
        close(got, *reference(x, None if w is None else w[row], a, il), "qk"[row])
    # alone, in place and into views with their own strides: the same bits
    assert torch.equal(vit.qk_norm_mrope(q, None, pos, f, sec, w, EPS, cycled=cycled, interleaved=il)[0], y[0])
    assert torch.equal(vit.qk_norm_mrope(None, k, pos, f, sec, w, EPS, cycled=cycled, interleaved=il)[1], y[1])
    wide = torch.full((T, Hq + 2 * Hk, D), 7.0, device="cuda", dtype=torch.bfloat16)
    wide[:, :Hq], wide[:, Hq:Hq + Hk] = q, k
    qv, kv = wide[:, :Hq], wide[:, Hq:Hq + Hk]
    vit.qk_norm_mrope(qv, kv, pos, f, sec, w, EPS, cycled=cycled, interleaved=il, inplace=True)
    assert torch.equal(qv, y[0]) and torch.equal(kv, y[1]) and (wide[:, Hq + Hk:] == 7).all()


@pytest.mark.parametrize("T,Hq,Hk,D,cycled,il,norm,far", CASES)
def test_gradient(T, Hq, Hk, D, cycled, il, norm, far):
    q, k, pos, f, sec, w = make(T, Hq, Hk, D, cycled, norm, far)
    g = torch.Generator(device="cuda").manual_seed(5)
    dq = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    dk = torch.randn(k.shape, generator=g, device="cuda").bfloat16()
    a = angles(pos, f, sec, cycled)
    gq, gk, dw = vit.qk_norm_mrope_bwd(dq, dk, q, k, pos, f, sec, w, EPS, cycled=cycled, interleaved=il)
    assert (dw is None) == (w is None)
    for row, (got, dy, x) in enumerate(((gq, dq, q), (gk, dk, k))):
        ref, mag, sw, mw = reference_grad(dy, x, None if w is None else w[row], a, il)
        close(got, ref, mag, "qk"[row])
        if w is not None:
            n = T * x.shape[1]
            tol = ((n + 64) * 2.0 ** -24 + 2.0 ** -18) * mw
            assert ((dw[row].double() - sw).abs() <= tol).all()
    again = vit.qk_norm_mrope_bwd(dq, dk, q, k, pos, f, sec, w, EPS, cycled=cycled, interleaved=il)
    assert torch.equal(again[0], gq) and torch.equal(again[1], gk) and (w is None or torch.equal(again[2], dw))
    one = vit.qk_norm_mrope_bwd(dq, None, q, None, pos, f, sec, w, EPS, cycled=cycled, interleaved=il)
    assert torch.equal(one[0], gq) and one[1] is None and (w is None or (one[2][1] == 0).all())
    over = vit.qk_norm_mrope_bwd(dq, dk, q, k, pos, f, sec, w, EPS, cycled=cycled, interleaved=il, inplace=True)
    assert over[0] is dq and torch.equal(dq, gq) and torch.equal(dk, gk)


def test_gradient_against_differences():
    # <dy, y(x + e d) - y(x - e d)> / 2e in 64 bits on the reference that the kernel is held to
    q, k, pos, f, sec, w = make(9, 3, 2, 64, True, True, 1000)
    a = angles(pos, f, sec, True)
    g = torch.Generator(device="cuda").manual_seed(6)
    dy = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    got = vit.qk_norm_mrope_bwd(dy, None, q, None, pos, f, sec, w, EPS, cycled=True)[0]
    for _ in range(4):
        d = torch.randn(q.shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        up, down = (reference(q.double() + s * e * d, w[0], a, False)[0] for s in (1, -1))
        slope = float((dy.double() * (up - down)).sum() / (2 * e))
        ours = float((got.double() * d).sum())
        # every element of the gradient is off by at most 2^-8 of itself plus 2^-19 of its parts
        tol = float((got.double().abs() * d.abs()).sum()) * 2.0 ** -7 + 1e-6
        assert abs(slope - ours) <= tol


def test_zero_rows_and_no_eps():
    # lanes past a token's last head must not leak into the weight sums when eps is 0
    q, k, pos, f, sec, w = make(5, 3, 1, 80, False, True, 10)
    dq, dk = torch.ones_like(q), torch.ones_like(k)
    _, _, dw = vit.qk_norm_mrope_bwd(dq, dk, q, k, pos, f, sec, w, 0.0)
    assert torch.isfinite(dw).all()


def test_empty():
    q, k, pos, f, sec, w = make(0, 4, 2, 64, False, True, 10)
    y = vit.qk_norm_mrope(q, k, pos, f, sec, w)
    assert y[0].shape == (0, 4, 64) and y[1].shape == (0, 2, 64)
    gq, gk, dw = vit.qk_norm_mrope_bwd(q, k, q, k, pos, f, sec, w)
    assert gq.shape == (0, 4, 64) and (dw == 0).all()


def test_captured_graph_and_stream():
    q, k, pos, f, sec, w = make(300, 8, 2, 128, True, True, 1000)
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    want = vit.qk_norm_mrope(q, k, pos, f, sec, w, cycled=True)
    grad = vit.qk_norm_mrope_bwd(dq, dk, q, k, pos, f, sec, w, cycled=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = vit.qk_norm_mrope(q, k, pos, f, sec, w, cycled=True, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = vit.qk_norm_mrope(q, k, pos, f, sec, w, cycled=True)
        d = vit.qk_norm_mrope_bwd(dq, dk, q, k, pos, f, sec, w, cycled=True)
    for t in y + d:
        t.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, z) for x, z in zip(want + grad, y + d))


@pytest.mark.parametrize("grids", [[(1, 1, 1)], [(3, 5, 7), (0, 4, 4), (1, 9, 2), (2, 0, 3), (4, 1, 6)],
                                   [(1, 3, 4)] * 700, []])
def test_grid_positions(grids):
    want = [(t, h, w) for T, H, W in grids for t in range(T) for h in range(H) for w in range(W)]
    grid = torch.tensor(grids, dtype=torch.int32, device="cuda").reshape(-1, 3)
    status = vit.new_status()
    pos, cu = vit.grid_positions(grid, len(want), status=status)
    assert vit.read_status(status) == 0
    assert torch.equal(pos.cpu(), torch.tensor(want, dtype=torch.int32).reshape(-1, 3))
    ends = torch.tensor([0] + [t * h * w for t, h, w in grids]).cumsum(0).int()
    assert torch.equal(cu.cpu(), ends)


@pytest.mark.parametrize("grids,T", [([(1, 2, 3)], 7), ([(1, -2, -3)], 6), ([(2 ** 31 - 1,) * 3], 8), ([], 1),
                                     ([(65536, 65536, 1), (1, 2, 3)], 6)])
def test_grid_mismatch_leaves_outputs(grids, T):
    grid = torch.tensor(grids, dtype=torch.int32, device="cuda").reshape(-1, 3)
    status = vit.new_status()
    vit.grid_positions(grid, T, status=status)
    assert vit.read_status(status) == -12


def test_agrees_with_the_two_axis_call():
    """A still image with no time pairs and both spatial tables side by side turns as vit_qk_norm_rope does."""
    grid = torch.tensor([[5, 6], [4, 4]], dtype=torch.int32, device="cuda")
    T, D = 46, 64
    f, pos, cu = vit.rope_freqs(grid, T, D)
    pos3, cu3 = vit.grid_positions(torch.tensor([[1, 5, 6], [1, 4, 4]], dtype=torch.int32, device="cuda"), T)
    assert torch.equal(pos3[:, 1:], pos) and torch.equal(cu3, cu)
    q = torch.randn(T, 3, D, device="cuda").bfloat16()
    two = vit.qk_norm_rope(q, None, pos, f)[0]
    three = vit.qk_norm_mrope(q, None, pos3, torch.cat([f, f]), (0, D // 4, D // 4))[0]
    # both round once; cos and sin differ by at most 2^-20
    assert ((two.double() - three.double()).abs() <= 2 * BF * two.double().abs() + 2.0 ** -17).all()
    assert math.isclose(float((two == three).double().mean()), 1.0, abs_tol=0.02)


def test_extreme_positions():
    """The largest and smallest positions of an int32, and those around the change to 64-bit angles."""
    D, H = 64, 3
    ends = [2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 2 ** 22 - 1, 2 ** 22, -2 ** 22, -2 ** 22 + 1, 0]
    pos = torch.tensor([[a, b, c] for a in ends for b, c in ((0, 7), (a, -a - 1))], dtype=torch.int32, device="cuda")
    T = pos.shape[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    freq = torch.cat((torch.ones(3), torch.rand(28), torch.tensor([-0.7]))).float().cuda()
    sec = (12, 10, 10)
    y, _ = vit.qk_norm_mrope(x, None, pos, freq, sec)
    close(y, *reference(x, None, angles(pos, freq, sec, False), False), "y")
    dx, _, _ = vit.qk_norm_mrope_bwd(x, None, None, None, pos, freq, sec)
    ref, mag, _, _ = reference_grad(x, None, None, angles(pos, freq, sec, False), False)
    close(dx, ref, mag, "dx")
