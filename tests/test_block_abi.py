"""Refusals of the calls around a language model's reading of the encoder's states, on the CPU: every bad argument
that the host can see is named by its code and nothing is launched, and the Python binding checks types, shapes and
devices before it. The calls' NVTX ranges are closed on every return."""
import ctypes
import json
import os
import shutil
import subprocess
import sys

import pytest
import torch

import vision_encoder_varlen_gb300 as vit
from vision_encoder_varlen_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
SEC = (ctypes.c_int * 3)(8, 16, 16)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return vit.lib()


def call(fn, good, order, **kw):
    a = dict(good, **kw)
    return fn(*(a[n] for n in order))


# addresses that no check dereferences
P = 4096


def test_grid_positions(L):
    f = L.vit_grid_positions
    assert f(P, -1, 4, P, P, None, None) == -3
    assert f(P, 1, -1, P, P, None, None) == -3
    assert f(P, 1, 1 << 31, P, P, None, None) == -3
    assert f(P, 8193, 4, P, P, None, None) == -7
    assert f(None, 1, 4, P, P, None, None) == -1
    assert f(P, 1, 4, P + 2, P, None, None) == -5
    assert f(P, 1, 4, None, None, None, None) == 0


MROPE = ("qi qo ki ko T Hq Hk D qis qos kis kos pos freq sec layout mode w eps stream").split()
GOOD_MROPE = dict(qi=P, qo=2 * P, ki=3 * P, ko=4 * P, T=10, Hq=4, Hk=2, D=80, qis=320, qos=320, kis=160, kos=160,
                  pos=P, freq=P, sec=SEC, layout=0, mode=0, w=None, eps=1e-6, stream=None)


def test_mrope(L):
    f = lambda **kw: call(L.vit_qk_norm_mrope, GOOD_MROPE, MROPE, **kw)
    three = lambda *x: (ctypes.c_int * 3)(*x)
    assert f(D=72) == -2
    assert f(T=-1) == -3 and f(T=1 << 31) == -3 and f(Hq=0) == -3 and f(Hk=70000) == -3
    assert f(eps=-1.0) == -14 and f(eps=float("nan")) == -14
    assert f(mode=2) == -14 and f(layout=2) == -14
    assert f(sec=None) == -1
    assert f(sec=three(8, 16, 15)) == -14 and f(sec=three(-8, 24, 24)) == -14
    assert f(layout=1, sec=three(10, 15, 15)) == -14          # a cycle cannot give 15 of 40 pairs to height
    assert f(pos=None) == -1 and f(freq=None) == -1
    assert f(qo=None) == -1 and f(ki=None) == -1
    assert f(qi=None, qo=None, ki=None, ko=None) == -1
    assert f(qis=312) == -4 and f(kos=162) == -4
    assert f(qo=P, qos=328) == -4                             # in place with another stride
    assert f(qi=P + 8) == -5 and f(w=P + 2) == -5 and f(pos=P + 1) == -5
    assert f(T=0, qi=None, qo=None, ki=None, ko=None) == 0


MROPE_BWD = ("dqo dqi dko dki q k T Hq Hk D dqos dqis dkos dkis qs ks pos freq sec layout mode w eps dw ws wsb "
             "stream").split()
GOOD_MROPE_BWD = dict(dqo=P, dqi=2 * P, dko=3 * P, dki=4 * P, q=5 * P, k=6 * P, T=10, Hq=4, Hk=2, D=80, dqos=320,
                      dqis=320, dkos=160, dkis=160, qs=320, ks=160, pos=P, freq=P, sec=SEC, layout=0, mode=0, w=P,
                      eps=1e-6, dw=P, ws=P, wsb=1 << 30, stream=None)


def test_mrope_gradient(L):
    f = lambda **kw: call(L.vit_qk_norm_mrope_bwd, GOOD_MROPE_BWD, MROPE_BWD, **kw)
    assert f(D=81) == -2 and f(Hq=0) == -3
    assert f(q=None) == -1 and f(dki=None) == -1              # the norm's gradient needs its input
    assert f(qs=8) == -4 and f(dqos=312) == -4
    assert f(k=P + 4) == -5
    assert f(ws=None) == -1 and f(ws=P + 8) == -5 and f(wsb=16) == -6 and f(dw=P + 2) == -5
    assert L.vit_qk_norm_mrope_bwd_workspace_size(80) > 0 and L.vit_qk_norm_mrope_bwd_workspace_size(81) == 0


CROSS = "q k v Tq Tk Hq Hk D qs ks vs cuq cuk klen B mq mk scale out os lse ws wsb status stream".split()
GOOD_CROSS = dict(q=P, k=2 * P, v=3 * P, Tq=100, Tk=200, Hq=8, Hk=2, D=64, qs=512, ks=128, vs=128, cuq=P, cuk=P,
                  klen=None, B=2, mq=50, mk=100, scale=0.0, out=P, os=512, lse=None, ws=P, wsb=1 << 30, status=None,
                  stream=None)
CROSS_BWD = ("do q k v out lse Tq Tk Hq Hk D dos qs ks vs os cuq cuk klen B mq mk scale dq dk dv dqs dks dvs zero ws "
             "wsb status stream").split()
GOOD_CROSS_BWD = dict(GOOD_CROSS, do=P, lse=P, dos=512, dq=P, dk=P, dv=P, dqs=512, dks=128, dvs=128, zero=1)


def both(L, **kw):
    a = call(L.vit_cross_attn, GOOD_CROSS, CROSS, **kw)
    b = call(L.vit_cross_attn_bwd, GOOD_CROSS_BWD, CROSS_BWD, **kw)
    assert a == b, (kw, a, b)
    return a


def test_cross_attention_and_gradient(L):
    assert both(L, D=72) == -2
    assert both(L, Hq=9) == -3 and both(L, Hk=0) == -3 and both(L, Tq=-1) == -3 and both(L, Tk=(1 << 31) - (1 << 16) + 1) == -3
    assert both(L, B=-1) == -3 and both(L, B=8193) == -7
    assert both(L, mq=-1) == -14 and both(L, scale=float("inf")) == -14
    assert both(L, q=None) == -1 and both(L, v=None) == -1 and both(L, cuk=None) == -1 and both(L, ws=None) == -1
    assert both(L, qs=504) == -4 and both(L, vs=132) == -4
    assert both(L, k=P + 8) == -5 and both(L, klen=P + 1) == -5 and both(L, ws=P + 4) == -5
    assert both(L, wsb=8) == -6
    assert both(L, B=0) == 0
    f = lambda **kw: call(L.vit_cross_attn, GOOD_CROSS, CROSS, **kw)
    assert f(out=None) == -1 and f(os=256) == -4 and f(lse=P + 2) == -5
    assert f(Tq=0) == 0
    g = lambda **kw: call(L.vit_cross_attn_bwd, GOOD_CROSS_BWD, CROSS_BWD, **kw)
    assert g(do=None) == -1 and g(lse=None) == -1 and g(dv=None) == -1
    assert g(dqs=256) == -4 and g(dks=120) == -4 and g(dk=P + 8) == -5


def test_cross_workspace_sizes(L):
    f, g = vit.cross_attn_workspace_size, vit.cross_attn_bwd_workspace_size
    assert f(100, 200, 8, 3, 64, 2) == 0 and g(100, 200, 8, 3, 64, 2) == 0       # 8 heads over 3
    assert f(100, 200, 8, 2, 65, 2) == 0 and f(100, 200, 8, 2, 64, 9000) == 0
    # one new token each, long states: a split's partial rows; bounds above the totals are the totals
    assert f(4, 40000, 8, 2, 64, 4, 1, 40000) == f(4, 40000, 8, 2, 64, 4, 1, 1 << 30) > 0
    assert f(5000, 9000, 16, 16, 80, 3) > 0 and g(5000, 9000, 16, 16, 80, 3) >= 5000 * 16 * 8
    # a long cache: element offsets pass 32 bits; rows up to 2^31 - 2^16
    most = 2 ** 31 - 2 ** 16
    assert f(64, most, 64, 8, 128, 64, 1, most) > 0 and f(64, most + 1, 64, 8, 128, 64, 1, most) == 0
    assert f(1, most, 1, 1, 32, 8192, 1, most) > 0 and g(1, most, 1, 1, 32, 8192, 1, most) > 0


NORM = "x y gate wo wr h z T C res xs ys gs hs zs scale eps stream".split()
GOOD_NORM = dict(x=P, y=2 * P, gate=P, wo=P, wr=P, h=3 * P, z=4 * P, T=7, C=1280, res=0, xs=1280, ys=1280, gs=0, hs=1280,
                 zs=1280, scale=1.0, eps=1e-6, stream=None)
NORM_BWD = ("dz dh h y gate wo wr dx dy dg dwo dwr T C res dzs dhs hs ys gs dxs dys dgs scale eps ws wsb status "
            "stream").split()
GOOD_NORM_BWD = dict(dz=P, dh=2 * P, h=3 * P, y=4 * P, gate=P, wo=P, wr=P, dx=5 * P, dy=6 * P, dg=P, dwo=P, dwr=P, T=7,
                     C=1280, res=0, dzs=1280, dhs=1280, hs=1280, ys=1280, gs=0, dxs=1280, dys=1280, dgs=1280,
                     scale=1.0, eps=1e-6, ws=P, wsb=1 << 30, status=None, stream=None)


def test_norm_residual(L):
    f = lambda **kw: call(L.vit_norm_residual, GOOD_NORM, NORM, **kw)
    g = lambda **kw: call(L.vit_norm_residual_bwd, GOOD_NORM_BWD, NORM_BWD, **kw)
    for h in (f, g):
        assert h(C=1284) == -3 and h(C=0) == -3 and h(C=8200) == -3 and h(T=-1) == -3
        assert h(res=2) == -14 and h(scale=float("nan")) == -14 and h(eps=-1e-6) == -14
        assert h(gs=640) == -4 and h(ys=1276) == -4 and h(y=None) == -1 and h(y=P + 2) == -5
    assert f(x=None) == -1 and f(z=None) == -1 and f(wr=None) == -14 and f(h=P, hs=1288) == -4 and f(T=0) == 0
    assert g(dz=None) == -14 and g(wr=None, dwr=None) == -14 and g(h=None) == -1
    assert g(wo=None) == -14 and g(gate=None) == -14          # a gradient of what is not there
    assert g(ws=None) == -1 and g(wsb=64) == -6 and g(dg=P + 4) == -5
    assert g(dx=2 * P, dxs=1288) == -4
    assert g(dz=None, dh=None, wr=None, dwr=None) == -1
    assert L.vit_norm_residual_bwd_workspace_size(1280) > 0 and L.vit_norm_residual_bwd_workspace_size(12) == 0


def test_binding_checks():
    bf = dict(dtype=torch.bfloat16)
    q, k = torch.zeros(5, 4, 64, **bf), torch.zeros(9, 2, 64, **bf)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vit.cross_attn(q, k, k, cu, cu)
    with pytest.raises(ValueError, match="CUDA"):
        vit.norm_residual(q[:, 0], q[:, 1])
    with pytest.raises(ValueError, match="CUDA"):
        vit.qk_norm_mrope(q, None, torch.zeros(5, 3, dtype=torch.int32), torch.zeros(32), (8, 12, 12))
    with pytest.raises(ValueError, match="at least one"):
        vit.qk_norm_mrope(None, None, cu, cu, (1, 1, 1))
    with pytest.raises(ValueError, match=r"\[T, H, D\]"):
        vit.cross_attn(q[0], k, k, cu, cu)
    with pytest.raises(ValueError, match="dz is given exactly"):
        vit.norm_residual_bwd(None, q[:, 0], q[:, 0], q[:, 0], w_pre=torch.zeros(64, **bf))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        vit.norm_residual(torch.zeros(3, 8, dtype=torch.float16), q[:, 0])
    with pytest.raises(ValueError, match="grid_thw"):
        vit.grid_positions(torch.zeros(4, 2, dtype=torch.int32), 0)


_CHILD = r"""
import ctypes, json, sys
L = ctypes.CDLL(sys.argv[1])
rec = ctypes.CDLL(sys.argv[2])
rec.nvtx_recorder_ranges.restype = ctypes.c_char_p
vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
rope = [vp, vp, vp, i32, i32, vp, f32]
T = {
    "vit_grid_positions": [vp, i32, i64, vp, vp, vp, vp],
    "vit_qk_norm_mrope": [vp] * 4 + [i64, i32, i32, i32] + [i64] * 4 + rope + [vp],
    "vit_qk_norm_mrope_bwd": [vp] * 6 + [i64, i32, i32, i32] + [i64] * 6 + rope + [vp, vp, sz, vp],
    "vit_cross_attn": [vp] * 3 + [i64, i64, i32, i32, i32] + [i64] * 3 + [vp] * 3 + [i32, i32, i32, f32, vp, i64, vp,
                                                                                    vp, sz, vp, vp],
    "vit_cross_attn_bwd": [vp] * 6 + [i64, i64, i32, i32, i32] + [i64] * 5 + [vp] * 3 + [i32, i32, i32, f32] + [vp] * 3 +
                          [i64] * 3 + [i32, vp, sz, vp, vp],
    "vit_norm_residual": [vp] * 7 + [i64, i32, i32] + [i64] * 5 + [f32, f32, vp],
    "vit_norm_residual_bwd": [vp] * 12 + [i64, i32, i32] + [i64] * 8 + [f32, f32, vp, sz, vp, vp],
}
codes = {}
for name, types in T.items():
    f = getattr(L, name)
    f.argtypes = types
    codes[name] = f(*(None if t is vp else -1.0 if t is f32 else 0 if t is sz else -1 for t in types))
print(json.dumps({"codes": codes, "ranges": rec.nvtx_recorder_ranges().decode().split(),
                  "pushes": rec.nvtx_recorder_pushes(), "pops": rec.nvtx_recorder_pops()}))
"""


def test_ranges(tmp_path):
    gcc = shutil.which("gcc")
    include = os.path.join(os.path.dirname(os.path.dirname(_build._nvcc())), "include")
    if not gcc or not os.path.exists(os.path.join(include, "nvtx3", "nvToolsExt.h")):
        pytest.skip("gcc or the NVTX 3 headers are missing")
    lib = _build.build()
    rec = str(tmp_path / "librec.so")
    subprocess.run([gcc, "-shared", "-fPIC", "-O2", "-std=c11", "-I", include,
                    os.path.join(HERE, "nvtx_recorder.c"), "-o", rec], check=True, capture_output=True)
    env = dict(os.environ, NVTX_INJECTION64_PATH=rec)
    r = subprocess.run([sys.executable, "-c", _CHILD, lib, rec], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stderr
    got = json.loads(r.stdout.splitlines()[-1])
    assert all(c < 0 for c in got["codes"].values()), got
    assert got["ranges"] == ["vitattn/" + n for n in got["codes"]] and got["pushes"] == got["pops"] == len(got["codes"])
