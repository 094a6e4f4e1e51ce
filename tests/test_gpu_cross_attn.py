"""Cross attention between packed sequences of different lengths, against the definition in 64 bits.

Tolerances, per element of out = sum_j p_j v_j: P is rounded to bf16 before the product (2^-8 of each
p_j, so 2^-8 sum_j p_j |v_j|), the result once more (2^-8 of it); scores are fp32 sums of products of
bf16 values (D terms: below D 2^-24 of sum |q_d k_d|, a relative error of every p), exp2 is good to
2^-21 of each p. lse moves by at most the largest score error plus 2^-21.
"""
import math

import pytest
import torch

import vision_encoder_varlen_gb300 as vit

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def make(ql, kl, Hq, Hk, D, seed=0, gap=0):
    """Packed inputs; with `gap`, unused rows before the first and behind the last sequence hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed + sum(ql) + 3 * sum(kl) + D)
    n = lambda T, H: torch.randn(T + 2 * gap, H, D, generator=g, device="cuda").bfloat16()
    q, k, v = n(sum(ql), Hq), n(sum(kl), Hk), n(sum(kl), Hk)
    if gap:
        for t in (q, k, v):
            t[:gap] = math.nan
            t[t.shape[0] - gap:] = math.nan
    cu = lambda x: torch.tensor([gap] + [gap + sum(x[:i + 1]) for i in range(len(x))], dtype=torch.int32, device="cuda")
    return q, k, v, cu(ql), cu(kl)


def reference(q, k, v, cu_q, cu_k, k_len=None, scale=None):
    """out, lse, and the magnitudes sum p|v| and the score error's bound, by sequence and head in 64 bits."""
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    serr = torch.zeros_like(lse)
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cq) - 1):
        n = ck[b + 1] - ck[b] if k_len is None else int(k_len[b])
        if n == 0 or cq[b + 1] == cq[b]:
            continue
        Q = q[cq[b]:cq[b + 1]].double().transpose(0, 1)
        K, V = (t[ck[b]:ck[b] + n].double().transpose(0, 1).repeat_interleave(Hq // Hk, 0) for t in (k, v))
        s = Q @ K.transpose(1, 2) * scale
        p = torch.softmax(s, -1)
        out[cq[b]:cq[b + 1]] = (p @ V).transpose(0, 1)
        mag[cq[b]:cq[b + 1]] = (p @ V.abs()).transpose(0, 1)
        lse[cq[b]:cq[b + 1]] = torch.logsumexp(s, -1).T
        serr[cq[b]:cq[b + 1]] = ((Q.abs() @ K.abs().transpose(1, 2)).amax(-1) * scale * D * 2.0 ** -24).T
    return out, lse, mag, serr


def check(got, got_lse, ref, rows=None):
    out, lse, mag, serr = ref
    rows = slice(None) if rows is None else rows
    assert torch.isfinite(got[rows]).all()
    e = 2 * serr[..., None] + 2.0 ** -20
    bound = BF * out.abs() + (BF + e) * (1 + BF) * mag + 2.0 ** -130
    err = ((got.double() - out).abs() - bound)[rows]
    assert (err <= 0).all(), f"out {float(err.max()):.3e} past its bound"
    if got_lse is not None:
        empty = torch.isinf(lse)
        assert torch.equal(torch.isneginf(got_lse)[rows], empty[rows])
        d = (got_lse.double() - lse).abs()[rows]
        tol = (serr + 2.0 ** -19 * (1 + lse.abs()))[rows]
        assert (d <= tol)[~empty[rows]].all()


# few query rows (split over the keys) and many (tensor-core tiles), lengths of one and none, odd sizes
CASES = [
    # query lengths, key lengths, Hq, Hkv, D
    ([1], [1], 1, 1, 32),
    ([1, 1, 1], [1601, 577, 1], 32, 8, 128),
    ([1] * 9, [0, 63, 64, 65, 127, 128, 129, 5000, 1], 8, 1, 80),
    ([1, 0, 1], [700, 300, 0], 4, 4, 96),
    ([2, 5, 1, 0], [33, 1000, 16, 5], 12, 3, 64),
    ([64, 64], [256, 4097], 2, 2, 80),
    ([13, 31, 7], [900, 15, 2500], 6, 3, 128),
    ([40, 64], [3, 1700], 2, 2, 32),
    ([65], [1], 1, 1, 64),
    ([9, 70, 1], [100, 1000, 0], 8, 1, 128),
    ([130, 1, 257, 0, 300], [77, 1111, 0, 50, 112], 4, 2, 80),
    ([513], [6000], 2, 1, 128),
    ([300, 200], [113, 2000], 6, 2, 96),
    ([1000], [999], 3, 3, 32),
    ([129, 2000], [640, 1], 5, 1, 64),
    ([200], [20000], 1, 1, 80),
]


@pytest.mark.parametrize("ql,kl,Hq,Hk,D", CASES)
def test_forward(ql, kl, Hq, Hk, D):
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D, gap=3)
    ref = reference(q, k, v, cq, ck)
    status = vit.new_status()
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), out=out, lse=lse, status=status)
    assert vit.read_status(status) == 0
    inside = slice(3, 3 + sum(ql))
    check(out, lse, ref, inside)
    assert (out[:3] == 9).all() and (out[3 + sum(ql):] == 9).all() and (lse[:3] == 9).all()
    # no bounds given, and no lse: still the same rows
    plain = torch.full_like(q, 9.0)
    vit.cross_attn(q, k, v, cq, ck, out=plain)
    check(plain, None, ref, inside)
    again = torch.full_like(q, 9.0)
    vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), out=again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("ql", [[1, 1, 1, 1], [9, 1, 33, 100]])
def test_padded_states_and_strides(ql):
    # states padded to a common length: what lies behind k_len (NaN, Inf) enters nothing
    B, S, Hq, Hk, D = 4, 200, 8, 2, 80
    lens = [200, 0, 17, 131]
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.randn(B * S, 2, Hk, D, generator=g, device="cuda").bfloat16()
    for b, n in enumerate(lens):
        kv[b * S + n:(b + 1) * S, 0] = math.nan
        kv[b * S + n:(b + 1) * S, 1] = math.inf
    k, v = kv[:, 0], kv[:, 1]                              # token stride 2 Hk D
    q = torch.randn(sum(ql), 3, Hq, D, generator=g, device="cuda").bfloat16()[:, 1]
    cq = torch.tensor([0] + ql, device="cuda").cumsum(0).int()
    ck = torch.arange(B + 1, device="cuda", dtype=torch.int32) * S
    k_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), S, 0.3, k_len=k_len, return_lse=True)
    check(out, lse, reference(q, k, v, cq, ck, lens, 0.3))


def test_no_states_at_all():
    for n in (1, 300):
        q = torch.randn(n, 4, 64, device="cuda").bfloat16()
        k = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
        cq = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ck = torch.zeros(2, dtype=torch.int32, device="cuda")
        out, lse = vit.cross_attn(q, k, k, cq, ck, return_lse=True)
        assert (out == 0).all() and torch.isneginf(lse).all()
    none = q[:0]
    assert vit.cross_attn(none, k, k, cq * 0, ck).shape == (0, 4, 64)


def test_agrees_with_self_attention_and_large_scores():
    # equal offsets on both sides are self attention; scores of +-60 keep the softmax exact
    ql = [300, 65, 512]
    q, k, v, cq, ck = make(ql, ql, 4, 4, 80)
    q = (8 * q.float()).bfloat16()
    out, lse = vit.cross_attn(q, k, v, cq, ck, 512, 512, return_lse=True)
    check(out, lse, reference(q, k, v, cq, ck))
    mine, l2 = vit.varlen_attn(q, k, v, cq, 512, return_lse=True)
    assert float((out.float() - mine.float()).abs().max()) <= 2 * BF * float(v.float().abs().max())


BAD = [
    # cu_q, cu_k, k_len, max_q, max_k, code
    ([0, 5, 3], [0, 10, 20], None, 0, 0, -10),
    ([0, 5, 9], [0, 10, 20], None, 0, 0, -10),             # past Tq
    ([0, 4, 8], [0, 10, 31], None, 0, 0, -10),             # past Tk
    ([-1, 4, 8], [0, 10, 20], None, 0, 0, -10),
    ([0, 4, 8], [0, 10, 20], [3, 11], 0, 0, -10),
    ([0, 4, 8], [0, 10, 20], [-1, 5], 0, 0, -10),
    ([0, 4, 8], [0, 10, 20], None, 3, 0, -11),
    ([0, 4, 8], [0, 10, 20], None, 0, 9, -11),
]


@pytest.mark.parametrize("cq,ck,kl,mq,mk,code", BAD)
@pytest.mark.parametrize("heads", [1, 32])                 # few rows, many rows
def test_bad_offsets_are_reported(cq, ck, kl, mq, mk, code, heads):
    q = torch.randn(8, heads, 64, device="cuda").bfloat16()
    k = torch.randn(30, 1, 64, device="cuda").bfloat16()
    t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    guard = torch.full((24, heads, 64), 5.0, device="cuda", dtype=torch.bfloat16)
    status = vit.new_status()
    vit.cross_attn(q, k, k, t(cq), t(ck), mq, mk, k_len=t(kl), out=guard[8:16], status=status)
    assert vit.read_status(status) == code
    assert (guard[:8] == 5).all() and (guard[16:] == 5).all()
    # a sound call afterwards is not affected
    out = vit.cross_attn(q, k, k, t([0, 4, 8]), t([0, 10, 20]))
    check(out, None, reference(q, k, k, t([0, 4, 8]), t([0, 10, 20])))


@pytest.mark.parametrize("Lq", [1, 200])
def test_graph_replays_other_lengths(Lq):
    # captured once for a bucket, replayed after other lengths were written on the device
    q, k, v, cq, ck = make([Lq, Lq], [1200, 1200], 8, 2, 128)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(vit.cross_attn_workspace_size(q.shape[0], k.shape[0], 8, 2, 128, 2, Lq, 1200), dtype=torch.uint8,
                     device="cuda")
    vit.cross_attn(q, k, v, cq, ck, Lq, 1200, out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vit.cross_attn(q, k, v, cq, ck, Lq, 1200, out=out, lse=lse, workspace=ws)
    for kl in ([1200, 1200], [37, 900], [0, 1]):
        ck.copy_(torch.tensor([0, kl[0], kl[0] + kl[1]], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, reference(q, k, v, cq, ck))


def test_side_stream():
    q, k, v, cq, ck = make([1] * 5, [900] * 5, 8, 2, 128)
    want = vit.cross_attn(q, k, v, cq, ck, 1, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [vit.cross_attn(q, k, v, cq, ck, 1, 900, stream=side) for _ in range(8)]
    side.synchronize()
    assert all(torch.equal(want, x) for x in got)


def many(B, lo_q, hi_q, lo_k, hi_k, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: torch.randint(lo, hi + 1, (B,), generator=g).tolist()
    return r(lo_q, hi_q), r(lo_k, hi_k)


# up to 32 sequences are ordered by one warp, more by the block; lists that end in a wave for few SMs are cut there
# (20 x 8 heads of 300 rows: 320 items; 5 x 4 x 8 of 1000: 160); chunked keys (few tiles, long keys) with many sequences
MANY = [
    (31, 17, 60, 0, 200, 4, 1, 64),
    (32, 17, 60, 0, 200, 4, 4, 80),
    (33, 17, 60, 0, 200, 4, 1, 64),
    (700, 0, 40, 0, 50, 2, 1, 32),
    (20, 300, 300, 128, 300, 8, 8, 64),
    (5, 1000, 1000, 100, 500, 8, 2, 96),
    (36, 20, 50, 1, 3000, 2, 2, 128),
    (6, 100, 140, 1, 5000, 4, 2, 128),
    (40, 1, 16, 0, 300, 2, 2, 80),
]


@pytest.mark.parametrize("B,lo_q,hi_q,lo_k,hi_k,Hq,Hk,D", MANY)
def test_many_sequences(B, lo_q, hi_q, lo_k, hi_k, Hq, Hk, D):
    ql, kl = many(B, lo_q, hi_q, lo_k, hi_k, B)
    q, k, v, cq, ck = make(ql, kl, Hq, Hk, D)
    status = vit.new_status()
    out, lse = vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl), return_lse=True, status=status)
    assert vit.read_status(status) == 0
    check(out, lse, reference(q, k, v, cq, ck))
    assert torch.equal(out, vit.cross_attn(q, k, v, cq, ck, max(ql), max(kl)))


@pytest.mark.parametrize("B", [20, 50])
def test_one_bad_sequence_among_many(B):
    ql, kl = many(B, 20, 60, 30, 100, 7)
    q, k, v, cq, ck = make(ql, kl, 4, 2, 64)
    ref = reference(q, k, v, cq, ck)
    # a key count past its bound: only that sequence is left alone
    k_len = torch.tensor(kl, dtype=torch.int32, device="cuda")
    k_len[11] += 1
    out, status = torch.full_like(q, 3.0), vit.new_status()
    vit.cross_attn(q, k, v, cq, ck, 60, 200, k_len=k_len, out=out, status=status)
    assert vit.read_status(status) == -10
    a, b = int(cq[11]), int(cq[12])
    assert (out[a:b] == 3).all()
    check(out, None, ref, torch.cat((torch.arange(a), torch.arange(b, q.shape[0]))).cuda())
    # query offsets that decrease: nothing past the tensors, and the error is told
    cq[11] = cq[12] + 1
    status = vit.new_status()
    vit.cross_attn(q, k, v, cq, ck, 200, 200, out=out, status=status)
    assert vit.read_status(status) == -10


@pytest.mark.parametrize("rows", [15, 16, 17, 32, 33])
def test_where_the_kernels_change(rows):
    """Query rows per key head around the sizes at which another kernel takes the call; keys around 32 MiB, and more
    than 16 runs of a sequence."""
    for keys, D in ((400, 64), (65000, 128)):
        q, k, v, cq, ck = make([rows, 1], [keys, 700], 2, 2, D)
        out, lse = vit.cross_attn(q, k, v, cq, ck, rows, max(keys, 700), return_lse=True)
        check(out, lse, reference(q, k, v, cq, ck))
