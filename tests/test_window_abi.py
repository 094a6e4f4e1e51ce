"""Refusals of the calls of a language model's own attention, on the CPU: every bad argument that the host can see is
named by its code and nothing is launched, and the Python binding checks types, shapes and devices before it."""
import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from vision_encoder_varlen_gb300 import _build
from test_block_abi import P, call


@pytest.fixture(scope="module")
def L():
    _build.build()
    return vit.lib()


WINDOW = "q k v Tq Tk Hq Hk D qs ks vs cuq cuk klen B mq mk win sinks scale out os lse ws wsb status stream".split()
GOOD = dict(q=P, k=2 * P, v=3 * P, Tq=100, Tk=200, Hq=8, Hk=2, D=64, qs=512, ks=128, vs=128, cuq=P, cuk=P, klen=None, B=2,
            mq=50, mk=100, win=30, sinks=4, scale=0.0, out=P, os=512, lse=None, ws=P, wsb=1 << 30, status=None, stream=None)
BWD = ("do q k v out lse Tq Tk Hq Hk D dos qs ks vs os cuq cuk klen B mq mk win sinks scale dq dk dv dqs dks dvs zero ws wsb "
       "status stream").split()
GOOD_BWD = dict(GOOD, do=P, lse=P, dos=512, dq=P, dk=P, dv=P, dqs=512, dks=128, dvs=128, zero=1)
PREFIX = ("q kp vp k v Tq Tp Tk Hq Hk D qs kps vps ks vs cuq cug cup cuk klen B G mq mp mk scale out os lse ws wsb status "
          "stream").split()
GOOD_PREFIX = dict(GOOD, kp=4 * P, vp=5 * P, Tp=300, kps=128, vps=128, cug=P, cup=P, G=2, mp=200)


def each(L, **kw):
    """The same code from the three calls, for what they share."""
    codes = [call(f, good, order, **{n: x for n, x in kw.items() if n in order})
             for f, good, order in ((L.vit_window_attn, GOOD, WINDOW), (L.vit_window_attn_bwd, GOOD_BWD, BWD),
                                    (L.vit_prefix_attn, GOOD_PREFIX, PREFIX))]
    assert len(set(codes)) == 1, (kw, codes)
    return codes[0]


def test_what_the_calls_share(L):
    assert each(L, D=72) == -2
    assert each(L, Hq=9) == -3 and each(L, Hk=0) == -3 and each(L, Hq=65537, Hk=65537) == -3
    assert each(L, Tq=-1) == -3 and each(L, Tk=(1 << 31) - (1 << 16) + 1) == -3
    assert each(L, B=-1) == -3 and each(L, B=8193) == -7
    assert each(L, mq=-1) == -14 and each(L, mk=-1) == -14
    assert each(L, scale=float("inf")) == -14 and each(L, scale=float("nan")) == -14
    assert each(L, q=None) == -1 and each(L, v=None) == -1 and each(L, cuk=None) == -1 and each(L, ws=None) == -1
    assert each(L, out=None) == -1
    assert each(L, qs=504) == -4 and each(L, vs=132) == -4 and each(L, os=256) == -4
    assert each(L, k=P + 8) == -5 and each(L, klen=P + 1) == -5 and each(L, ws=P + 4) == -5 and each(L, out=P + 2) == -5
    assert each(L, lse=P + 2) == -5
    assert each(L, wsb=8) == -6
    assert each(L, B=0) == 0


def test_windows(L):
    for f, good, order in ((L.vit_window_attn, GOOD, WINDOW), (L.vit_window_attn_bwd, GOOD_BWD, BWD)):
        assert call(f, good, order, win=-1) == -14 and call(f, good, order, sinks=-1) == -14
        assert call(f, good, order, win=0, sinks=-5) == -14
    assert call(L.vit_window_attn, GOOD, WINDOW, Tq=0) == 0
    g = lambda **kw: call(L.vit_window_attn_bwd, GOOD_BWD, BWD, **kw)
    assert g(do=None) == -1 and g(lse=None) == -1 and g(dv=None) == -1
    assert g(dqs=256) == -4 and g(dks=120) == -4 and g(dk=P + 8) == -5


def test_prefixes(L):
    f = lambda **kw: call(L.vit_prefix_attn, GOOD_PREFIX, PREFIX, **kw)
    assert f(Tp=-1) == -3 and f(Tp=1 << 31) == -3 and f(G=-1) == -3 and f(G=0) == -3 and f(G=8193) == -7
    assert f(mp=-1) == -14
    assert f(cup=None) == -1 and f(cug=None) == -1 and f(kp=None) == -1 and f(vp=None) == -1
    assert f(kps=120) == -4 and f(vps=124) == -4
    assert f(cug=P + 2) == -5 and f(cup=P + 1) == -5 and f(kp=P + 8) == -5
    assert f(B=0, G=0) == 0 and f(Tq=0) == 0
    # no groups but one, or no prefix rows at all: the workspace is the first thing that is missing then
    assert f(cug=None, G=1, wsb=0) == -6 and f(Tp=0, kp=None, vp=None, wsb=0) == -6


def test_workspace_sizes():
    f, g, h = vit.window_attn_workspace_size, vit.window_attn_bwd_workspace_size, vit.prefix_attn_workspace_size
    assert f(100, 200, 8, 3, 64, 2) == 0 and g(100, 200, 8, 3, 64, 2) == 0 and h(100, 50, 200, 8, 3, 64, 2, 1) == 0
    assert f(100, 200, 8, 2, 64, 2, window=-1) == 0 and f(100, 200, 8, 2, 64, 2, window=5, sinks=-1) == 0
    assert h(100, 50, 200, 8, 2, 64, 2, 0) == 0 and h(100, -1, 200, 8, 2, 64, 2, 1) == 0
    # a window that leaves nothing out is none; one of a long cache needs no more than what it lets through
    assert f(4, 40000, 8, 2, 64, 4, 1, 40000, 40000) == f(4, 40000, 8, 2, 64, 4, 1, 40000) > 0
    assert f(4, 40000, 8, 2, 64, 4, 1, 40000, 1000, 4) < f(4, 40000, 8, 2, 64, 4, 1, 40000)
    most = 2 ** 31 - 2 ** 16
    assert f(64, most, 64, 8, 128, 64, 1, most, 5000, 4) > 0 and f(64, most + 1, 64, 8, 128, 64, 1, most, 5000, 4) == 0
    assert f(1, most, 1, 1, 32, 8192, 1, most, most, most) > 0 and g(1, most, 1, 1, 32, 8192, 1, most, 7, 2 ** 31 - 1) > 0
    assert h(64, most, most, 8, 8, 128, 64, 1, 1, most, most) > 0 and h(64, most + 1, 9, 8, 8, 128, 64, 1) == 0


def test_binding_checks():
    bf = dict(dtype=torch.bfloat16)
    q, k = torch.zeros(5, 4, 64, **bf), torch.zeros(9, 2, 64, **bf)
    cu, lse = torch.zeros(2, dtype=torch.int32), torch.zeros(5, 4)
    with pytest.raises(ValueError, match="CUDA"):
        vit.window_attn(q, k, k, cu, cu)
    with pytest.raises(ValueError, match="CUDA"):
        vit.window_attn_bwd(q, q, k, k, q, lse, cu, cu)
    with pytest.raises(ValueError, match="CUDA"):
        vit.prefix_attn(q, k, k, k, k, cu, cu, cu)
    with pytest.raises(ValueError, match="window"):
        vit.window_attn_bwd(q, q, k, k, q, lse, cu, cu, window=0)
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        vit.window_attn(q[0], k, k, cu, cu)
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        vit.prefix_attn(q, k[0], k, k, k, cu, cu, cu)
