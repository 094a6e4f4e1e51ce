"""Registers of the kernels around a language model's reading of the encoder's states, from the assembler's own report
on the CPU.

The gradient kernel of cross attention splits its launch's registers between its warpgroups with setmaxnreg, which
waits for registers that are not there: every instantiation has to compile to exactly the count that the split was
made for. (The launcher refuses any other count; this finds it when it is built.)
"""
import os

from vision_encoder_varlen_gb300 import _build
from test_ptxas_resources import _constant, kernels

HEAD_DIMS = (32, 64, 80, 96, 128)


def test_every_kernel_is_reported(kernels):
    names = [k["name"] for k in kernels]
    for kern in ("cross_few_kernel", "cross_join_kernel", "cross_tile_join_kernel", "cross_grad_kernel",
                 "cross_grad_prepare_kernel", "mrope_kernel", "mrope_bwd_kernel"):
        for D in HEAD_DIMS:
            assert any(f"{kern}<{D}" in n or f"{kern}<(int){D}" in n for n in names), (kern, D)
    for kern in ("cross_schedule_kernel", "grid_positions_kernel", "norm_residual_kernel", "norm_residual_bwd_kernel",
                 "norm_residual_bwd_ring_kernel", "column_sum_kernel"):
        assert any(kern in n for n in names), kern


def test_gradient_kernel_register_count_matches_its_split(kernels):
    with open(os.path.join(_build.CSRC, "cross_bwd.cu")) as f:
        src = f.read()
    threads, launch = _constant(src, "kThreads"), _constant(src, "kLaunchRegs")
    ctrl, softmax = _constant(src, "kCtrlRegs"), _constant(src, "kSoftmaxRegs")
    # one control warpgroup, two softmax warpgroups
    assert threads == 384 and launch * threads <= 65536 and launch % 8 == ctrl % 8 == softmax % 8 == 0
    assert ctrl * 128 + softmax * 256 <= launch * threads
    grads = [k for k in kernels if "cross_grad_kernel" in k["name"]]
    assert len(grads) == len(HEAD_DIMS)
    assert all(k["regs"] == launch for k in grads), [(k["name"], k["regs"]) for k in grads]


def test_cross_variants_of_the_tcgen05_kernel(kernels):
    """One instantiation of the forward kernel per head size takes the cross-attention list."""
    names = [k["name"].replace("(bool)1", "true").replace("(bool)0", "false").replace("(int)", "") for k in kernels]
    for D in HEAD_DIMS:
        assert any(f"attn_long_kernel<{D}, true, false, true>" in n for n in names), D
