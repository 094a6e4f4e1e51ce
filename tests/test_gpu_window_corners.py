"""Corners of a language model's own attention: bad lists, graphs, streams, workspaces, many sequences and groups, strides,
long caches, and a run of its calls together as a decoder uses them. Tolerances are those of the two files imported."""
import math

import pytest
import torch

import vision_encoder_varlen_gb300 as vit
import test_gpu_window_attn_bwd as back
from test_gpu_window_attn import BF, check, make, offsets, reference

pytestmark = pytest.mark.gpu


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ lists that are malformed

BAD = [
    # cu_q, cu_k, k_len, max_q, max_k, code
    ([0, 5, 3], [0, 10, 20], None, 0, 0, -10),
    ([0, 5, 9], [0, 10, 20], None, 0, 0, -10),             # past Tq
    ([0, 4, 8], [0, 10, 31], None, 0, 0, -10),             # past Tk
    ([-1, 4, 8], [0, 10, 20], None, 0, 0, -10),
    ([0, 4, 8], [0, 10, 20], [3, 11], 0, 0, -10),
    ([0, 4, 8], [0, 10, 20], [-1, 5], 0, 0, -10),
    ([0, 4, 8], [0, 10, 20], [2 ** 31 - 1, 5], 0, 0, -10),
    ([0, 4, 8], [0, 10, 20], None, 3, 0, -11),
    ([0, 4, 8], [0, 10, 20], None, 0, 9, -11),
]


@pytest.mark.parametrize("cq,ck,kl,mq,mk,code", BAD)
@pytest.mark.parametrize("heads", [1, 32])                 # few rows, many rows
@pytest.mark.parametrize("window,sinks", [(None, 0), (3, 1)])
def test_bad_offsets_are_reported(cq, ck, kl, mq, mk, code, heads, window, sinks):
    q = torch.randn(8, heads, 64, device="cuda").bfloat16()
    k = torch.randn(30, 1, 64, device="cuda").bfloat16()
    guard = torch.full((24, heads, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    grads = [torch.full((24 if i == 0 else 50, heads if i == 0 else 1, 64), 5.0, device="cuda", dtype=torch.bfloat16)
             for i in range(3)]
    lse = torch.zeros(8, heads, device="cuda")
    status = vit.new_status()
    vit.window_attn(q, k, k, ints(cq), ints(ck), mq, mk, window, sinks, k_len=ints(kl), out=guard[8:16], status=status)
    assert vit.read_status(status) == code
    assert (guard[:8] == 5).all() and (guard[16:] == 5).all()
    status = vit.new_status()
    vit.window_attn_bwd(q, q, k, k, q, lse, ints(cq), ints(ck), mq, mk, window, sinks, k_len=ints(kl), dq=grads[0][8:16],
                        dk=grads[1][10:40], dv=grads[2][10:40], status=status)
    assert vit.read_status(status) == code
    for g, n in zip(grads, (8, 30, 30)):
        lo = (g.shape[0] - n) // 2
        assert (g[:lo] == 5).all() and (g[lo + n:] == 5).all()
    status = vit.new_status()
    vit.prefix_attn(q, k, k, k, k, ints(cq), ints([0, 30]), ints(ck), None, mq, 0, mk, k_len=ints(kl), out=guard[8:16],
                    status=status)
    assert vit.read_status(status) == code
    assert (guard[:8] == 5).all() and (guard[16:] == 5).all()
    # a sound call afterwards is not affected
    out = vit.window_attn(q, k, k, ints([0, 4, 8]), ints([0, 10, 20]), None, None, window, sinks)
    check(out, None, reference(q, k, k, ints([0, 4, 8]), ints([0, 10, 20]), None, window or 0, sinks))


BAD_GROUPS = [
    # cu_group, cu_prefix, max_prefix, code
    ([0, 1, 1], [0, 10, 20], 0, -10),                      # ends before the last sequence
    ([1, 1, 2], [0, 10, 20], 0, -10),
    ([0, 3, 2], [0, 10, 20], 0, -10),
    ([0, 1, 3], [0, 10, 20], 0, -10),
    ([0, -1, 2], [0, 10, 20], 0, -10),
    ([0, 1, 2], [0, 20, 10], 0, -10),
    ([0, 1, 2], [0, 10, 31], 0, -10),
    ([0, 1, 2], [-1, 10, 20], 0, -10),
    ([0, 1, 2], [0, 10, 20], 9, -11),
]


# few rows; a list of sequences; groups apart from their sequences with many rows and with few
@pytest.mark.parametrize("ql,heads,rows", [([4, 4], 1, 30), ([600, 600], 2, 30), ([40] * 2, 16, 30), ([1, 1], 2, 30000)])
@pytest.mark.parametrize("cg,cp,mp,code", BAD_GROUPS)
def test_bad_groups_are_reported(ql, heads, rows, cg, cp, mp, code):
    T = sum(ql)
    q = torch.randn(T, heads, 64, device="cuda").bfloat16()
    k, kp = (torch.randn(n, heads, 64, device="cuda").bfloat16() for n in (T, rows))
    grow = rows // 30                                      # the offsets of thirty rows, in a prefix of `rows`
    guard = torch.full((T + 16, heads, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    status = vit.new_status()
    cp = [x * grow if x >= 0 else x for x in cp]
    vit.prefix_attn(q, kp, kp, k, k, offsets(ql), ints(cp), offsets(ql), ints(cg), max(ql), mp * grow, max(ql),
                    out=guard[8:8 + T], status=status)
    assert vit.read_status(status) == code
    assert (guard[:8] == 5).all() and (guard[8 + T:] == 5).all()


# ------------------------------------------------------------------ graphs, streams, workspaces

@pytest.mark.parametrize("Lq", [1, 200])
def test_graph_replays_other_lengths(Lq):
    """Captured once for a bucket, replayed after other lengths were written on the device."""
    q, k, v, cq, ck, _ = make([Lq, Lq], [1200, 1200], 8, 2, 128)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(vit.window_attn_workspace_size(q.shape[0], k.shape[0], 8, 2, 128, 2, Lq, 1200, 300, 4),
                     dtype=torch.uint8, device="cuda")
    run = lambda: vit.window_attn(q, k, v, cq, ck, Lq, 1200, 300, 4, out=out, lse=lse, workspace=ws)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for kl in ([1200, 1200], [37, 900], [0, 1]):
        ck.copy_(torch.tensor([0, kl[0], kl[0] + kl[1]], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, reference(q, k, v, cq, ck, None, 300, 4))


# few rows; a list of sequences; groups apart with few rows and with many
@pytest.mark.parametrize("Lq,Hq,P", [(1, 8, 700), (300, 8, 700), (1, 8, 30000), (20, 2, 3000)])
def test_graph_replays_other_prefixes(Lq, Hq, P):
    q, k, v, cq, ck, _ = make([Lq] * 6, [Lq + 50] * 6, Hq, 2, 128)
    kp, vp = (make([P], [1], 2, 2, 128, seed=s)[0] for s in (1, 2))
    cp, cg = ints([0, P // 2, P]), ints([0, 2, 6])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(vit.prefix_attn_workspace_size(6 * Lq, P, k.shape[0], Hq, 2, 128, 6, 2, Lq, P, Lq + 50),
                     dtype=torch.uint8, device="cuda")
    run = lambda: vit.prefix_attn(q, kp, vp, k, v, cq, cp, ck, cg, Lq, P, Lq + 50, out=out, lse=lse, workspace=ws)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for prefixes, groups in (([0, P // 2, P], [0, 2, 6]), ([5, 5, P - 3], [0, 5, 6]), ([0, P, P], [0, 6, 6]),
                             ([7, 7, 7], [0, 0, 6])):
        cp.copy_(torch.tensor(prefixes, dtype=torch.int32))
        cg.copy_(torch.tensor(groups, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        of = [(kp, vp, prefixes[g], prefixes[g + 1]) for g in range(2) for _ in range(groups[g + 1] - groups[g])]
        check(out, lse, reference(q, k, v, cq, ck, prefix=of))


def test_graphs_on_one_workspace():
    """Graphs of a forward and a backward call that share a workspace, replayed in turn, and calls on two streams with
    workspaces of their own."""
    q, k, v, do, cq, ck, mask = back.grads([300, 77], [300, 77], 4, 2, 80, 50, 3)
    n, size = q.shape[0], vit.window_attn_bwd_workspace_size
    ws = torch.empty(max(size(n, n, 4, 2, 80, 2, 300, 300, *mask), vit.window_attn_workspace_size(n, n, 4, 2, 80, 2, 300, 300,
                                                                                                 *mask)),
                     dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    fwd = lambda: vit.window_attn(q, k, v, cq, ck, 300, 300, *mask, out=out, lse=lse, workspace=ws)
    bwd = lambda: vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, 300, 300, *mask, dq=dq, dk=dk, dv=dv, workspace=ws)
    fwd(), bwd()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, f in zip(graphs, (fwd, bwd)):
        with torch.cuda.graph(g):
            f()
    for seed in (1, 2):
        q.copy_(torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        check(out, lse, reference(q, k, v, cq, ck, None, *mask))
        back.check((dq, dk, dv), back.reference(q, k, v, do, cq, ck, None, *mask))
    want = [t.clone() for t in (out, dq, dk, dv)]
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        for s in side:
            o, l = vit.window_attn(q, k, v, cq, ck, 300, 300, *mask, return_lse=True, stream=s)
            got.append((o,) + vit.window_attn_bwd(do, q, k, v, o, l, cq, ck, 300, 300, *mask, stream=s))
    for s in side:
        s.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))


# ------------------------------------------------------------------ many sequences and groups

# up to 32 sequences by a warp, up to 256 by a thread each, more sorted by the block; lists that end in a small wave;
# cut key ranges with many sequences
MANY = [
    (32, 17, 60, 4, 1, 64, 20, 3),
    (33, 17, 60, 4, 4, 80, 100, 0),
    (256, 0, 40, 2, 1, 32, 7, 2),
    (257, 0, 40, 2, 1, 32, 0, 0),
    (3000, 0, 20, 2, 1, 32, 9, 1),
    (20, 300, 300, 8, 8, 64, 128, 4),
    (5, 1000, 1000, 8, 2, 96, 0, 0),
    (2, 40, 70, 2, 2, 128, 3000, 500),
    (40, 40, 40, 1, 1, 64, 0, 0),
    (40, 40, 40, 1, 1, 64, 1500, 9),
]


@pytest.mark.parametrize("B,lo,hi,Hq,Hk,D,window,sinks", MANY)
def test_many_sequences(B, lo, hi, Hq, Hk, D, window, sinks):
    ql = torch.randint(lo, hi + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    kl = [max(0, m + (7 * i) % 5 - 1) if B > 5 and B != 40 else m + 9000 * (B == 2) + 3000 * (B == 40) for i, m in enumerate(ql)]
    q, k, v, cq, ck, _ = make(ql, kl, Hq, Hk, D)
    ref = reference(q, k, v, cq, ck, None, window, sinks)
    status = vit.new_status()
    out, lse = vit.window_attn(q, k, v, cq, ck, max(ql), max(kl), window or None, sinks, return_lse=True, status=status)
    assert vit.read_status(status) == 0
    check(out, lse, ref)
    do = torch.randn_like(q)
    got = vit.window_attn_bwd(do, q, k, v, out, lse, cq, ck, max(ql), max(kl), window or None, sinks, status=status)
    assert vit.read_status(status) == 0
    back.check(got, back.reference(q, k, v, do, cq, ck, None, window, sinks))


@pytest.mark.parametrize("G,per,m,P", [(31, 3, 1, 200), (32, 3, 1, 200), (40, 2, 20, 90), (1, 700, 1, 3000), (3, 100, 5, 2000),
                                       (2, 300, 20, 500)])
def test_many_groups(G, per, m, P):
    B = G * per
    ql, kl = [m] * B, [m + i % 4 for i in range(B)]
    q, k, v, cq, ck, _ = make(ql, kl, 4, 1, 64)
    pl = [(P * (g + 1)) // G for g in range(G)]
    kp, vp = (make(pl, [1], 1, 1, 64, seed=s)[0] for s in (1, 2))
    cp, cg = offsets(pl), offsets([per] * G)
    at = cp.tolist()
    ref = reference(q, k, v, cq, ck, prefix=[(kp, vp, at[g], at[g + 1]) for g in range(G) for _ in range(per)])
    status = vit.new_status()
    out, lse = vit.prefix_attn(q, kp, vp, k, v, cq, cp, ck, cg, m, max(pl), max(kl), return_lse=True, status=status)
    assert vit.read_status(status) == 0
    check(out, lse, ref)


def test_most_heads():
    q, k, v, cq, ck, _ = make([3, 20], [40, 20], 65536, 8192, 32)
    out, lse = vit.window_attn(q, k, v, cq, ck, 20, 40, 9, 2, return_lse=True)
    for h in (0, 1, 32767, 65535):
        one = reference(q[:, h:h + 1], k[:, h // 8:h // 8 + 1], v[:, h // 8:h // 8 + 1], cq, ck, None, 9, 2)
        check(out[:, h:h + 1], lse[:, h:h + 1].contiguous(), one)


# ------------------------------------------------------------------ layouts and sizes

@pytest.mark.parametrize("m", [1, 150])
def test_views_of_one_projection(m):
    """q, k and v as views of one packed projection, and a cache whose rows hold k and v side by side."""
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(3 * m, 8 + 2 + 2, 64, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    cq = offsets([m] * 3)
    out = torch.full((3 * m, 9, 64), 4.0, device="cuda", dtype=torch.bfloat16)
    vit.window_attn(q, k, v, cq, cq, m, m, 20, 2, out=out[:, 1:])
    check(out[:, 1:], None, reference(q, k, v, cq, cq, None, 20, 2))
    assert (out[:, 0] == 4).all()
    kv = torch.randn(500, 2, 2, 64, generator=g, device="cuda").bfloat16()
    got = vit.prefix_attn(q, kv[:, 0], kv[:, 1], k, v, cq, ints([100, 500]), cq, None, m, 400, m)
    check(got, None, reference(q, k, v, cq, cq, prefix=[(kv[:, 0], kv[:, 1], 100, 500)] * 3))


@pytest.mark.parametrize("m", [1, 60])
def test_nothing_on_a_side(m):
    """No keys anywhere, no prefix anywhere, no queries, no sequences."""
    q = torch.randn(2 * m, 4, 64, device="cuda").bfloat16()
    none, cq, zero = q.new_zeros(0, 2, 64), offsets([m, m]), ints([0, 0, 0])
    k = torch.randn(2 * m, 2, 64, device="cuda").bfloat16()
    out, lse = vit.window_attn(q, none, none, cq, zero, m, 1, 5, 2, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    dq, dk, dv = vit.window_attn_bwd(q, q, none, none, out, lse, cq, zero, m, 1, 5, 2)
    assert not dq.any() and dk.shape == dv.shape == none.shape
    out, lse = vit.prefix_attn(q, none, none, none, none, cq, ints([0, 0]), zero, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    want = vit.window_attn(q, k, k, cq, cq, m, m)
    check(vit.prefix_attn(q, none, none, k, k, cq, ints([0, 0]), cq), None, reference(q, k, k, cq, cq))
    check(want, None, reference(q, k, k, cq, cq))
    out, lse = vit.prefix_attn(q, k, k, none, none, cq, ints([0, 2 * m]), zero, None, m, 2 * m, 1, return_lse=True)
    check(out, lse, reference(q, none, none, cq, zero, prefix=[(k, k, 0, 2 * m)] * 2))
    empty = q[:0]
    assert vit.window_attn(empty, k, k, zero, cq).shape == empty.shape
    dq, dk, dv = vit.window_attn_bwd(empty, empty, k, k, empty, lse[:0], zero, cq, window=3)
    assert not dk.any() and not dv.any()
    one = ints([0])
    dq, dk, dv = vit.window_attn_bwd(q, q, k, k, q, lse, one, one)
    assert not dq.any() and not dk.any() and not dv.any()
    assert vit.prefix_attn(q, k, k, k, k, one, ints([0, 0]), one).shape == q.shape


@pytest.mark.parametrize("m,P,padded", [(1, 900, 64), (1, 30000, 64), (30, 900, 100), (400, 900, 500)])
def test_prefix_before_a_padded_cache(m, P, padded):
    """NaN behind the real rows of each sequence's cache, and around the prefixes."""
    B, Hk = 6, 2
    own = [m + 5 * b for b in range(B - 1)] + [0]
    q, k, v, cq, ck, k_len = make([m] * B, own, 8, Hk, 80, rows=padded)
    kp, vp = (make([P, 33], [1], Hk, Hk, 80, seed=s, gap=4)[0] for s in (1, 2))
    cp, groups = offsets([P, 33], 4), [4, 2]
    of = [(kp, vp, 4, 4 + P)] * 4 + [(kp, vp, 4 + P, 37 + P)] * 2
    out, lse = vit.prefix_attn(q, kp, vp, k, v, cq, cp, ck, offsets(groups), m, P, padded, k_len=k_len, return_lse=True)
    check(out, lse, reference(q, k, v, cq, ck, k_len, prefix=of))


def test_windows_that_leave_nothing_out():
    q, k, v, cq, ck, _ = make([200, 1], [300, 90], 4, 2, 64)
    want = vit.window_attn(q, k, v, cq, ck, 200, 300, return_lse=True)
    for window, sinks in ((300, 0), (301, 7), (2 ** 31 - 1, 2 ** 31 - 1)):
        got = vit.window_attn(q, k, v, cq, ck, 200, 300, window, sinks, return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    # all first tokens stay visible: nothing is left out either, but by the mask
    got = vit.window_attn(q, k, v, cq, ck, 200, 300, 5, 2 ** 31 - 1, return_lse=True)
    check(*got, reference(q, k, v, cq, ck))
    do = torch.randn_like(q)
    a = vit.window_attn_bwd(do, q, k, v, *want, cq, ck, 200, 300)
    b = vit.window_attn_bwd(do, q, k, v, *want, cq, ck, 200, 300, 2 ** 31 - 1, 9)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("m", [1, 40])
def test_offsets_past_32_bits(m):
    """A cache of 2.3 billion elements: sequences at its end, behind a window and without one, and a prefix there."""
    Hk, D, T = 8, 128, 2_300_000
    k = torch.zeros(T, Hk, D, device="cuda", dtype=torch.bfloat16)
    n = [900, 4000]
    g = torch.Generator(device="cuda").manual_seed(8)
    k[T - sum(n):] = torch.randn(sum(n), Hk, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(2 * m, 2 * Hk, D, generator=g, device="cuda").bfloat16()
    cq, ck = offsets([m, m]), offsets(n, T - sum(n))
    tail, ct = k[T - sum(n):], offsets(n)
    for window, sinks in ((0, 0), (500, 4)):
        out, lse = vit.window_attn(q, k, k, cq, ck, m, 4000, window or None, sinks, return_lse=True)
        check(out, lse, reference(q, tail, tail, cq, ct, None, window, sinks))
        if window:
            do = torch.randn_like(q)
            dk, dv = torch.zeros_like(k), torch.zeros_like(k)
            dq = torch.zeros_like(q)
            vit.window_attn_bwd(do, q, k, k, out, lse, cq, ck, m, 4000, window, sinks, dq=dq, dk=dk, dv=dv)
            back.check((dq, dk[T - sum(n):], dv[T - sum(n):]),
                       back.reference(q, tail, tail, do, cq, ct, None, window, sinks))
            assert not dk[:T - sum(n)].any() and not dv[:T - sum(n)].any()
            del dk, dv
    own = torch.randn(2 * m, Hk, D, generator=g, device="cuda").bfloat16()
    out, lse = vit.prefix_attn(q, k, k, own, own, cq, ints([T - 4000, T]), cq, None, m, 4000, m, return_lse=True)
    check(out, lse, reference(q, own, own, cq, cq, prefix=[(tail, tail, 900, 4900)] * 2))


# ------------------------------------------------------------------ a decoder's run of them

def rotated(x, w, pos, freq, sec):
    return vit.qk_norm_mrope(x, None, pos, freq, sec, w)[0]


@pytest.mark.parametrize("captured", [False, True])
def test_a_decoder_layer(captured):
    """Positions and norms of q and k, windowed attention, the residual step, the reading of an encoder's states, and back
    through all of it: each stored result against its definition from the tensors before it."""
    ql, Hq, Hk, D, window, sinks = [150, 37, 1], 8, 2, 64, 40, 4
    T, C = sum(ql), Hq * D
    g = torch.Generator(device="cuda").manual_seed(21)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    qkv, x, dz, dh = bf(T, Hq + 2 * Hk, D), bf(T, C), bf(T, C), bf(T, C)
    w, w_pre = (1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")).bfloat16(), bf(C)
    freq = (1e4 ** (-torch.arange(D // 2, device="cuda").double() / (D // 2))).float()
    pos = torch.cat([torch.arange(m) for m in ql]).int().cuda()[:, None].expand(T, 3).contiguous()
    sec, cu = (D // 2, 0, 0), offsets(ql)
    s = {}

    def run():
        q, k = vit.qk_norm_mrope(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], pos, freq, sec, w)
        v = qkv[:, Hq + Hk:]
        y, lse = vit.window_attn(q, k, v, cu, cu, max(ql), max(ql), window, sinks, return_lse=True)
        h, z = vit.norm_residual(x, y.view(T, C), w_pre=w_pre)
        dx, dy, _, _, dw = vit.norm_residual_bwd(dz, dh, h, y.view(T, C), w_pre=w_pre)
        dq, dk, dv = vit.window_attn_bwd(dy.view(T, Hq, D), q, k, v, y, lse, cu, cu, max(ql), max(ql), window, sinks)
        dq0, dk0, dnorm = vit.qk_norm_mrope_bwd(dq, dk, qkv[:, :Hq], qkv[:, Hq:Hq + Hk], pos, freq, sec, w)
        s.update(q=q, k=k, v=v, y=y, lse=lse, h=h, z=z, dy=dy, dq=dq, dk=dk, dv=dv, dq0=dq0, dk0=dk0, dnorm=dnorm)

    run()
    if captured:
        first = {n: t.clone() for n, t in s.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(first[n], s[n]) for n in s)
    check(s["y"], s["lse"], reference(s["q"], s["k"], s["v"], cu, cu, None, window, sinks))
    back.check((s["dq"], s["dk"], s["dv"]), back.reference(s["q"], s["k"], s["v"], s["dy"].view(T, Hq, D), cu, cu, None,
                                                            window, sinks))
    for n in ("h", "z", "dq0", "dk0", "dnorm"):
        assert torch.isfinite(s[n]).all()


@pytest.mark.parametrize("window,sinks", [(None, 0), (30, 4)])
def test_a_prompt_then_single_tokens(window, sinks):
    """A prompt at once, in pieces over the growing cache, and its last tokens one by one: the same rows."""
    n, Hq, Hk, D = 260, 8, 2, 128
    q, k, v, _, _, _ = make([n], [n], Hq, Hk, D, seed=3)
    ref = reference(q, k, v, offsets([n]), offsets([n]), None, window or 0, sinks)
    check(vit.window_attn(q, k, v, offsets([n]), offsets([n]), n, n, window, sinks), None, ref)
    out, at = torch.empty_like(q), 0
    for m in [100, 1, 7, 33, 64] + [1] * 55:
        done = ints([at + m])
        vit.window_attn(q[at:at + m], k, v, offsets([m]), ints([0, n]), m, n, window, sinks, k_len=done, out=out[at:at + m])
        at += m
    assert at == n
    check(out, None, ref)


@pytest.mark.parametrize("m", [1, 30, 300])
def test_a_shared_prefix_is_the_sequences_with_it(m):
    """prefix_attn against window_attn over caches that hold the prefix in front of every sequence."""
    B, P, Hq, Hk, D = 7, 900, 8, 2, 64
    own = [m + 3 * b for b in range(B)]
    q, k, v, cq, ck, _ = make([m] * B, own, Hq, Hk, D)
    kp, vp = (make([P], [1], Hk, Hk, D, seed=s)[0] for s in (1, 2))
    together = lambda p, x: torch.cat([torch.cat([p, t]) for t in x.split(own)])
    ref = reference(q, k, v, cq, ck, prefix=[(kp, vp, 0, P)] * B)
    a = vit.prefix_attn(q, kp, vp, k, v, cq, ints([0, P]), ck, None, m, P, max(own), return_lse=True)
    b = vit.window_attn(q, together(kp, k), together(vp, v), cq, offsets([P + n for n in own]), m, P + max(own),
                        return_lse=True)
    check(*a, ref)
    check(*b, ref)
