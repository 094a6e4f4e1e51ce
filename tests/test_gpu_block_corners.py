"""Corner calls of the operators around a language model's reading of the encoder's states: no rows, no sequences,
sequences without states beside others, lists that are wrong in one place, infinities.

Expected values are exact (zeros, untouched rows, the same bits as another call) or from the formulas in 64 bits with
the bounds that stand beside them.
"""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from test_gpu_cross_attn import check, make, reference

pytestmark = pytest.mark.gpu

BF16 = dict(dtype=torch.bfloat16, device="cuda")


# ------------------------------------------------------------------ residual step

@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("C", [256, 520, 1280, 6144, 8192])
@pytest.mark.parametrize("post,pre,gate", [(True, False, False), (False, False, True), (True, True, True),
                                           (True, False, True), (False, True, False)])
def test_residual_gradient_of_no_rows(C, post, pre, gate, wide):
    """The sums over no tokens are 0, whichever of the inputs are there."""
    w = torch.ones(C, **BF16)
    dh = torch.empty(0, C, device="cuda", dtype=torch.float32 if wide else torch.bfloat16)
    none = torch.empty(0, C, **BF16)
    dx, dy, dgate, dw_post, dw_pre = vit.norm_residual_bwd(
        none if pre else None, dh, dh if pre else None, none, gate=w if gate else None, w_post=w if post else None,
        w_pre=w if pre else None)
    assert dx.shape == dy.shape == (0, C)
    for asked, s in ((gate, dgate), (post, dw_post), (pre, dw_pre)):
        assert (s is not None) == asked
        if asked:
            assert s.shape == (C,) and not s.any()


# ------------------------------------------------------------------ cross attention

@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("Tq,Tk", [(37, 210), (37, 0), (0, 210)])
def test_gradient_of_no_sequences(Tq, Tk, side):
    """All rows are rows of no sequence: 0 in new tensors, as they were in given ones."""
    q, k = torch.randn(Tq, 4, 64, device="cuda").bfloat16(), torch.randn(Tk, 2, 64, device="cuda").bfloat16()
    lse = torch.zeros(Tq, 4, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for t in [torch.full_like(x, float("nan")) for x in (q, k, k) for _ in range(4)]:
            del t                                             # what the allocator hands out next is not 0
    got = vit.cross_attn_bwd(q, q, k, k, q, lse, cu, cu, stream=stream)
    torch.cuda.synchronize()
    for t, like in zip(got, (q, k, k)):
        assert t.shape == like.shape and not t.any()
    given = [torch.full_like(x, 7) for x in (q, k, k)]
    vit.cross_attn_bwd(q, q, k, k, q, lse, cu, cu, dq=given[0], dk=given[1], dv=given[2], stream=stream)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in given)


def _lists(lengths):
    return torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device="cuda")


def test_gradients_back_to_back_on_one_workspace():
    """Calls of different lengths that follow one another on one workspace, captured in one graph and replayed
    without a pause, give the bits of separate calls: none reads the lists or statistics of another."""
    g = torch.Generator(device="cuda").manual_seed(5)
    Hq, Hk, D = 8, 2, 64
    calls = []
    for ql, kl in (([300, 1, 77], [900, 40, 333]), ([5, 200], [64, 1500]), ([1] * 40, [1] * 40), ([513], [2049])):
        n = lambda T, H: torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
        q, do, k, v = n(sum(ql), Hq), n(sum(ql), Hq), n(sum(kl), Hk), n(sum(kl), Hk)
        cq, ck = _lists(ql), _lists(kl)
        out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True)
        ref = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl))
        got = [torch.empty_like(t) for t in (q, k, v)]
        calls.append(((do, q, k, v, out, lse, cq, ck, max(ql), max(kl)), ref, got))
    size = max(vit.cross_attn_bwd_workspace_size(a[1].shape[0], a[2].shape[0], Hq, Hk, D, a[6].numel() - 1, a[8], a[9])
               for a, _, _ in calls)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run():
        for a, _, (dq, dk, dv) in calls:
            vit.cross_attn_bwd(*a, dq=dq, dk=dk, dv=dv, workspace=ws)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(30):
        for _, _, got in calls:
            for t in got:
                t.zero_()
        for _ in range(4):
            graph.replay()
        for _, ref, got in calls:
            for x, y in zip(got, ref):
                assert torch.equal(x, y)


def _cross(ql, kl, Hq, Hk, D, seed=0):
    """q, k, v with rows of no sequence before, behind and around them, and the two lists."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda T, H: torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    return n(sum(ql) + 9, Hq), n(sum(kl) + 5, Hk), n(sum(kl) + 5, Hk), _lists(ql) + 4, _lists(kl) + 2


def _check_rows_without_states(ql, kl, Hq, Hk, D, lse=True):
    """Zeros and -inf for the sequences without states, the bits of the call without them for the others, and the
    rows of no sequence as they were."""
    q, k, v, cq, ck = _cross(ql, kl, Hq, Hk, D)
    out = torch.full_like(q, 3)
    l = torch.full(q.shape[:2], 5.0, device="cuda") if lse else None
    status = vit.new_status()
    vit.cross_attn(q, k, v, cq, ck, max(ql), max(max(kl), 1), out=out, lse=l, status=status)
    assert vit.read_status(status) == 0
    at = [4]
    for n in ql:
        at.append(at[-1] + n)
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    inside[at[0]:at[-1]] = True
    assert (out[~inside] == 3).all() and (not lse or (l[~inside] == 5).all())
    keep = [i for i, n in enumerate(kl) if n]
    for i, n in enumerate(kl):
        if n == 0:
            rows = slice(at[i], at[i + 1])
            assert (out[rows] == 0).all() and (not lse or torch.isneginf(l[rows]).all()), i
    if not keep:
        return
    qs = torch.cat([q[at[i]:at[i + 1]] for i in keep])
    ref, ref_l = vit.cross_attn(qs, k, v, _lists([ql[i] for i in keep]), _lists([kl[i] for i in keep]) + 2,
                                max(ql), max(kl), return_lse=True)
    # The other call may cut the keys differently. Each side then rounds P and its result to bf16 (2^-8 of them), so
    # they are 2 x 2^-8 (max |v| + |out|) apart at most; sums of n <= 2048 exponentials in another order n 2^-24.
    got = torch.cat([out[at[i]:at[i + 1]] for i in keep])
    assert ((got.float() - ref.float()).abs() <= 2.0 ** -7 * (v.float().abs().max() + ref.float().abs())).all()
    if lse:
        got_l = torch.cat([l[at[i]:at[i + 1]] for i in keep])
        assert ((got_l - ref_l).abs() <= 2.0 ** -12 + 2.0 ** -22 * ref_l.abs()).all()


@pytest.mark.parametrize("lse", [True, False])
@pytest.mark.parametrize("ql,kl,Hq,Hk,D", [
    ([300, 257, 64, 500], [700, 0, 1300, 0], 8, 2, 128),          # between and behind others
    ([40, 1, 333], [0, 0, 900], 4, 4, 80),                        # before them
    ([1000], [0], 16, 16, 64),                                    # alone
    ([200, 5, 77], [0, 0, 0], 6, 2, 32),                          # all of them
    ([64] * 18, [500] * 16 + [0, 0], 16, 16, 80),                 # latents
    ([70] * 20 + [3] * 20 + [90] * 60, ([300] * 10 + [0] * 10) * 5, 8, 8, 96),   # more than a warp lists
    ([0, 50, 0, 60], [0, 0, 10, 20], 4, 2, 64),                   # without queries either
])
def test_sequences_without_states(ql, kl, Hq, Hk, D, lse):
    _check_rows_without_states(ql, kl, Hq, Hk, D, lse)


@pytest.mark.parametrize("other", [0, 600])
def test_a_long_sequence_without_states(other):
    """200 000 rows, behind a prompt and alone."""
    _check_rows_without_states([200000, 300], [0, other], 8, 2, 64)


def test_a_text_only_request_costs_no_more_than_its_zeros():
    """A prompt without states beside three others: its rows (17 MB of zeros, some microseconds) are written by all
    SMs beside the others' work, not by one warp at ten times the whole call's time."""
    def time(ql, kl):
        q, k, v, cq, ck = _cross(ql, kl, 32, 8, 128)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        ms = []
        for i in range(8):
            s, e = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            s.record()
            vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), out=out, lse=lse)
            e.record()
            torch.cuda.synchronize()
            ms.append(s.elapsed_time(e))
        return min(ms[2:])

    assert time([2047] * 4, [8000] * 3 + [0]) < 1.5 * time([2047] * 3, [8000] * 3)


def _gradient_into(q, k, v, do, cq, ck, k_len, max_q, max_k, zero_rest, fill=7.0):
    """The C call on buffers full of `fill`: (status code of the device, dq, dk, dv)."""
    (Tq, Hq, D), (Tk, Hk, _) = q.shape, k.shape
    out, lse = vit.cross_attn(q, k, v, cq, ck, max_q, max_k, k_len=k_len, status=vit.new_status(), return_lse=True)
    g = [torch.full_like(t, fill) for t in (q, k, v)]
    status = vit.new_status()
    n = vit.cross_attn_bwd_workspace_size(Tq, Tk, Hq, Hk, D, cq.numel() - 1, max_q, max_k)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()
    code = vit.lib().vit_cross_attn_bwd(
        p(do), p(q), p(k), p(v), p(out), p(lse), Tq, Tk, Hq, Hk, D, *[t.stride(0) for t in (do, q, k, v, out)], p(cq),
        p(ck), p(k_len), cq.numel() - 1, max_q, max_k, 0.0, *[p(t) for t in g], *[t.stride(0) for t in g], zero_rest,
        p(ws), n, p(status), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()
    return vit.read_status(status), *g


@pytest.mark.parametrize("zero_rest", [0, 1])
@pytest.mark.parametrize("bad,code", [(-5, -10), (130, -10), (101, -11)])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_gradient_beside_a_malformed_length(at, bad, code, zero_rest):
    """Real states per sequence: one wrong entry leaves that sequence's rows as they were, whether or not the rest is
    cleared, and nobody else's are touched by it. (101 of 120 rows is sound but above the bound of 100.)"""
    g = torch.Generator(device="cuda").manual_seed(at)
    n = lambda T, H: torch.randn(T, H, 64, generator=g, device="cuda").bfloat16()
    q, do, k, v = n(150, 4), n(150, 4), n(400, 2), n(400, 2)
    cq, ck = _lists([50, 50, 50]), _lists([120, 120, 120]) + 11
    lens = [100, 33, 77]
    fine = torch.tensor(lens, dtype=torch.int32, device="cuda")
    _, *ref = _gradient_into(q, k, v, do, cq, ck, fine, 50, 100, 1, 0.0)
    lens[at] = bad
    status, *got = _gradient_into(q, k, v, do, cq, ck, torch.tensor(lens, dtype=torch.int32, device="cuda"), 50, 100,
                                  zero_rest)
    assert status == code
    rest = 0.0 if zero_rest else 7.0
    for x, y, lo, per in ((got[0], ref[0], 0, 50), (got[1], ref[1], 11, 120), (got[2], ref[2], 11, 120)):
        want = torch.full_like(x, rest)
        for b in range(3):
            rows = slice(lo + b * per, lo + (b + 1) * per)
            if b == at:
                want[rows] = 7.0
            else:
                real = slice(rows.start, rows.start + (per if per == 50 else lens[b]))
                want[real] = y[real]
        # the sound sequences may be left out of such a call; where they are computed they are right
        for b in range(3):
            rows = slice(lo + b * per, lo + (b + 1) * per)
            assert torch.equal(x[rows], want[rows]) or (b != at and (x[rows] == 7.0).all()), (b, per)
        assert (x[:lo] == rest).all() and (x[lo + 3 * per:] == rest).all()


@pytest.mark.parametrize("which", ["q", "k"])
def test_gradient_with_offsets_that_decrease(which):
    """Nothing at all is written, the rest included."""
    q, k = torch.randn(90, 4, 64, device="cuda").bfloat16(), torch.randn(90, 2, 64, device="cuda").bfloat16()
    good = _lists([30, 20, 10]) + 5
    wrong = torch.tensor([5, 35, 25, 65], dtype=torch.int32, device="cuda")
    k_len = torch.tensor([10, 0, 10], dtype=torch.int32, device="cuda")
    status, *got = _gradient_into(q, k, k, q, wrong if which == "q" else good, wrong if which == "k" else good, k_len,
                                  90, 90, 1)
    assert status == -10 and all((t == 7).all() for t in got)


# keys that take no part because their scores are -inf (an infinite component against a positive one of the queries):
# the first ones, up to whole tiles and runs; all but the last; every other group of 16
MINUS = {
    "first_16": lambda n: slice(0, min(16, n - 1)), "first_64": lambda n: slice(0, min(64, n - 1)),
    "first_half": lambda n: slice(0, n // 2), "all_but_the_last": lambda n: slice(0, n - 1),
    "last_half": lambda n: slice((n + 1) // 2, n),
    "every_other_16": lambda n: [i for i in range(n) if (i // 16) % 2 == 0 and i < n - 1],
}
SCORES = [
    # query lengths, key lengths, Hq, Hkv, D
    ([1, 2], [37, 3000], 8, 2, 128),          # few rows, keys split and joined
    ([1], [100000], 2, 1, 64),                # in many runs
    ([1] * 200, [70] * 200, 8, 8, 80),        # in one
    ([64], [6000], 2, 2, 80),                 # one tile, keys cut into runs
    ([300, 130], [900, 113], 4, 2, 96),       # split items
    ([700] * 6, [500] * 6, 16, 4, 128),       # whole items
    ([700] * 6, [300] * 6, 16, 16, 64),
]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", SCORES)
@pytest.mark.parametrize("where", sorted(MINUS))
def test_scores_of_minus_infinity(where, ql, kl, Hq, Hk, D):
    """Such keys have weight 0, wherever they lie: the result is that of the other keys."""
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    q[..., 0] = q[..., 0].abs() + 0.125
    keep = torch.ones(k.shape[0], dtype=torch.bool, device="cuda")
    for b, n in enumerate(kl):
        keep[int(ck[b]):int(ck[b]) + n][MINUS[where](n)] = False
    k[~keep, :, 0] = -float("inf")
    kept = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), keep.long().cumsum(0)])
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True)
    check(out, lse, reference(q, k[keep], v[keep], cq, kept[ck.long()].int()))


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", SCORES)
def test_all_scores_minus_infinity(ql, kl, Hq, Hk, D):
    """0 / 0 and ln 0 by the formulas, in one row; the other rows are as always."""
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    q[..., 0] = 0
    ref = reference(q, k, v, cq, ck)
    t = q.shape[0] // 2
    q[t, 1, 0] = -float("inf")
    k[..., 0] = 1
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True)
    assert torch.isnan(out[t, 1]).all() and torch.isneginf(lse[t, 1])
    rows = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    rows[t, 1] = False
    check(out, lse, ref, rows)


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", SCORES)
def test_a_key_of_nan(ql, kl, Hq, Hk, D):
    """A NaN among the first sequence's keys makes all of its rows NaN, the log-sum-exp too, and no other's."""
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    ref = reference(q, k, v, cq, ck)
    k[int(ck[0]), :, 3] = float("nan")
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True)
    n = ql[0]
    assert torch.isnan(out[:n]).all() and torch.isnan(lse[:n]).all()
    if len(ql) > 1:
        check(out, lse, ref, slice(n, None))


# ------------------------------------------------------------------ as many heads as a call takes

def test_most_heads():
    """65536 heads: the bits of calls on a few of them, first and last."""
    H, D = 65536, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda T: torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    q, do, k, v = n(2), n(2), n(5), n(5)
    pos = torch.tensor([[1, 7, 3], [0, 2, 100000]], dtype=torch.int32, device="cuda")
    freq = torch.logspace(0, -4, D // 2, device="cuda")
    w = torch.ones(2, D, **BF16)
    cq, ck = _lists([2]), _lists([5])
    y, _ = vit.qk_norm_mrope(q, None, pos, freq, (6, 5, 5), w)
    _, yk = vit.qk_norm_mrope(None, q, pos, freq, (6, 5, 5), w)
    back, _, _ = vit.qk_norm_mrope_bwd(do, None, q, None, pos, freq, (6, 5, 5), w)
    out, lse = vit.cross_attn(q, k, v, cq, ck, return_lse=True)
    grad = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck)
    for few in (slice(0, 64), slice(H - 64, H)):
        a, b, c, d = (t[:, few].contiguous() for t in (q, do, k, v))
        assert torch.equal(y[:, few], vit.qk_norm_mrope(a, None, pos, freq, (6, 5, 5), w)[0])
        assert torch.equal(yk[:, few], vit.qk_norm_mrope(None, a, pos, freq, (6, 5, 5), w)[1])
        assert torch.equal(back[:, few], vit.qk_norm_mrope_bwd(b, None, a, None, pos, freq, (6, 5, 5), w)[0])
        o, l = vit.cross_attn(a, c, d, cq, ck, return_lse=True)
        assert torch.equal(out[:, few], o) and torch.equal(lse[:, few], l)
        for x, ref in zip(grad, vit.cross_attn_bwd(b, a, c, d, o, l, cq, ck)):
            assert torch.equal(x[:, few], ref)


# ------------------------------------------------------------------ the residual gradient's other forms

def _norm_bwd(dz, dh, h, y, gate, w_post, w_pre, dx, dy, dgate, dw_post, dw_pre, scale=0.75, eps=1e-6):
    """The C call; strides are the tensors' own."""
    ref = dh if dh is not None else h
    T, C = ref.shape
    p = lambda t: None if t is None else t.data_ptr()
    s = lambda t: 0 if t is None else t.stride(0)
    n = vit.lib().vit_norm_residual_bwd_workspace_size(C)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    status = vit.new_status()
    token = gate is not None and gate.dim() == 2
    code = vit.lib().vit_norm_residual_bwd(
        p(dz), p(dh), p(h), p(y), p(gate), p(w_post), p(w_pre), p(dx), p(dy), p(dgate), p(dw_post), p(dw_pre), T, C,
        vit.RES_FP32 if ref.dtype == torch.float32 else vit.RES_BF16, s(dz), s(dh), s(h), s(y),
        gate.stride(0) if token else 0, s(dx), s(dy), dgate.stride(0) if token and dgate is not None else 0, scale, eps,
        p(ws), n, p(status), torch.cuda.current_stream().cuda_stream)
    assert code == 0 and vit.read_status(status) == 0


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,C", [(1, 8), (37, 256), (333, 512), (700, 520), (3001, 1280), (450, 4096), (333, 6144), (170, 8192)])
def test_residual_gradient_in_place_and_in_part(T, C, wide):
    """dx over dh, dy over y or dz, and any of the sums left out: the bits of the call with tensors of its own."""
    g = torch.Generator(device="cuda").manual_seed(C + T)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")
    res = (lambda t: t) if wide else (lambda t: t.bfloat16())
    rows = lambda t: torch.cat([t, torch.full_like(t[:, :16], 9)], 1)[:, :C]      # a stride above the width
    h, dh, y, dz = rows(res(n(T, C))), rows(res(n(T, C))), rows(n(T, C).bfloat16()), rows(n(T, C).bfloat16())
    w1, w2 = (1 + 0.2 * n(C)).bfloat16(), (1 + 0.2 * n(C)).bfloat16()
    for gate in (None, n(C).bfloat16(), rows(n(T, C).bfloat16())):
        for post, pre, stream in ((w1, w2, True), (w1, None, True), (None, w2, False), (None, None, True), (w1, w2, False)):
            if pre is None and not stream:
                continue
            z, d = dz if pre is not None else None, dh if stream else None
            dx, dy, dgate, dw_post, dw_pre = vit.norm_residual_bwd(z, d, h, y, gate=gate, w_post=post, w_pre=pre, scale=0.75)
            same = lambda t: t if t is None else rows(t.clone())
            # dx over dh; dy over y; the sums one at a time
            for keep in range(4):
                d2, y2, z2 = same(d), same(y), same(z)
                if keep % 2 and z is not None:                # dy over dz
                    over = z2
                else:
                    over = y2
                out = [None if t is None or i != keep else torch.empty_like(t)
                       for i, t in enumerate((dgate, dw_post, dw_pre))]
                x2 = d2 if d2 is not None else torch.empty_like(dx)
                _norm_bwd(z2, d2, h, y2, gate, post, pre, x2, over, *out)
                assert torch.equal(x2, dx) and torch.equal(over, dy), (post is None, pre is None, keep)
                for got, ref in zip(out, (dgate, dw_post, dw_pre)):
                    assert got is None or torch.equal(got, ref)
                for t in (x2, over):                          # what lies between the rows
                    if t.stride(0) > C:
                        assert (t.as_strided((T - 1, 16), (t.stride(0), 1), t.storage_offset() + C) == 9).all()


# ------------------------------------------------------------------ the gradient over few keys

@pytest.mark.parametrize("ql,kl,Hq,Hk,D", [
    ([50, 7, 131, 1], [2, 3, 5, 1], 4, 4, 64),
    ([64] * 6, [1, 2, 4, 8, 15, 16], 8, 1, 128),
    ([33, 200, 3, 90], [13, 16, 17, 900], 6, 2, 80),              # beside longer ones
    ([17, 1, 0, 40], [9, 14, 5, 0], 12, 4, 96),
    ([5] * 100, [1 + i % 16 for i in range(100)], 2, 2, 32),
    ([1000], [3], 16, 4, 64),
])
@pytest.mark.parametrize("padded", [False, True])
def test_gradient_over_few_keys(ql, kl, Hq, Hk, D, padded):
    """Over few keys delta nearly cancels dP, so it is taken from the scores and not from the rounded output: dS is off
    by its own rounding and the fp32 arithmetic alone. With e = 2 (D 2^-24 max sum |q k| scale) + 2^-19 the relative
    error of every p, and 2 m, m = D 2^-24 sum |do v|, that of dP and delta,
      |dS err| <= 2^-8 |dS| + (1 + 2^-8) p (2 m + e (|dP| + sum p |dP|)) =: w
      |dq err| <= 2^-8 |dq| + scale sum_j w |k|, likewise dk."""
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    k_len = None
    if padded:                                                    # twice the rows, the second half not there
        wide = [torch.full((2 * t.shape[0], *t.shape[1:]), float("nan"), **BF16) for t in (k, v)]
        lists = ck.tolist()
        for a, b in zip(lists[:-1], lists[1:]):
            for t, w in zip((k, v), wide):
                w[2 * a:a + b] = t[a:b]
        k, v = wide
        k_len, ck = torch.tensor(kl, dtype=torch.int32, device="cuda"), 2 * ck
    g = torch.Generator(device="cuda").manual_seed(1)
    do = torch.randn(q.shape, generator=g, device="cuda").bfloat16()
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), k_len=k_len, return_lse=True)
    dq, dk, _ = vit.cross_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), k_len=k_len)
    half, G, scale = 2.0 ** -8, Hq // Hk, D ** -0.5
    at, of, T = cq.tolist(), ck.tolist(), lambda t: t.transpose(1, 2)
    for b, n in enumerate(kl):
        if n == 0 or n > 16 or ql[b] == 0:
            continue
        rq, rk = slice(at[b], at[b + 1]), slice(of[b], of[b] + n)
        Q, DO = (t[rq].double().transpose(0, 1) for t in (q, do))
        K, V = (t[rk].double().transpose(0, 1).repeat_interleave(G, 0) for t in (k, v))
        p = torch.softmax(Q @ T(K) * scale, -1)
        dp = DO @ T(V)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        e = 2 * (Q.abs() @ T(K.abs())).amax() * scale * D * 2.0 ** -24 + 2.0 ** -19
        m = D * 2.0 ** -24 * (DO.abs() @ T(V.abs()))
        m = m + (p * m).sum(-1, keepdim=True)
        w = half * ds.abs() + (1 + half) * p * (2 * m + e * (dp.abs() + (p * dp.abs()).sum(-1, keepdim=True)))
        heads = lambda t: t.reshape(Hk, G, *t.shape[1:]).sum(1).transpose(0, 1)
        for name, x, y, t in (("dq", dq[rq], scale * (ds @ K).transpose(0, 1), scale * (w @ K.abs()).transpose(0, 1)),
                              ("dk", dk[rk], heads(scale * T(ds) @ Q), heads(scale * T(w) @ Q.abs()))):
            err = (x.double() - y).abs() - (half * y.abs() + (1 + half) * t + 2.0 ** -130)
            assert (err <= 0).all(), f"{name} over {n} keys: {float(err.max()):.3e} past its bound"
