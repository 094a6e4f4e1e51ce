"""Both sides of the documented limits of the calls around a language model's reading of the encoder's states, on the
CPU: with no rows a call that passes the checks has nothing to do and says so before it looks for a device."""
import ctypes

import pytest

import vision_encoder_varlen_gb300 as vit
from test_block_abi import CROSS, CROSS_BWD, GOOD_CROSS, GOOD_CROSS_BWD, GOOD_MROPE, GOOD_MROPE_BWD, MROPE, MROPE_BWD, L, call

OK, BAD_SHAPE = 0, -3


@pytest.mark.parametrize("heads,code", [(1, OK), (65536, OK), (65537, BAD_SHAPE), (0, BAD_SHAPE)])
def test_heads(L, heads, code):
    for h in ("Hq", "Hk"):
        assert call(L.vit_qk_norm_mrope, GOOD_MROPE, MROPE, T=0, **{h: heads}) == code
        assert call(L.vit_qk_norm_mrope_bwd, GOOD_MROPE_BWD, MROPE_BWD, T=0, dw=None, **{h: heads}) == code
    kw = dict(Hq=heads, Hk=1, Tq=0)
    assert call(L.vit_cross_attn, GOOD_CROSS, CROSS, **kw) == code
    assert call(L.vit_cross_attn_bwd, GOOD_CROSS_BWD, CROSS_BWD, Tk=0, **kw) == code
    assert (vit.cross_attn_workspace_size(5, 7, heads, heads, 64, 1) > 0) == (code == OK)


def test_columns_and_rows(L):
    assert L.vit_norm_residual_bwd_workspace_size(8192) > 0 and L.vit_norm_residual_bwd_workspace_size(8200) == 0
    most = 2 ** 31 - 2 ** 16
    assert vit.cross_attn_workspace_size(most, 7, 1, 1, 32, 1) > 0
    assert vit.cross_attn_workspace_size(most + 1, 7, 1, 1, 32, 1) == 0
    assert vit.cross_attn_workspace_size(5, 7, 1, 1, 32, vit.MAX_SEGMENTS) > 0
    assert vit.cross_attn_workspace_size(5, 7, 1, 1, 32, vit.MAX_SEGMENTS + 1) == 0
