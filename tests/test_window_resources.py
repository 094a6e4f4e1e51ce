"""Registers of the kernels of a language model's own attention, from the assembler's own report on the CPU: those whose
warpgroups share out a launch's registers compile to exactly the count that the split was made for."""
import os

from vision_encoder_varlen_gb300 import _build
from test_ptxas_resources import _constant, kernels

HEAD_DIMS = (32, 64, 80, 96, 128)


def of(kernels, name):
    return [k for k in kernels if name in k["name"]]


def test_every_kernel_is_reported(kernels):
    for name in ("window_long_kernel", "window_grad_kernel", "window_join_kernel"):
        for D in HEAD_DIMS:
            assert any(f"{name}<{D}" in k["name"] or f"{name}<(int){D}" in k["name"] for k in kernels), (name, D)
    assert len(of(kernels, "window_schedule_kernel")) == 6


def test_register_counts_match_their_splits(kernels):
    for name, file in (("window_long_kernel", "attn_long.cu"), ("window_grad_kernel", "cross_bwd.cu")):
        with open(os.path.join(_build.CSRC, file)) as f:
            launch = _constant(f.read(), "kLaunchRegs")
        mine = of(kernels, name)
        assert len(mine) == len(HEAD_DIMS)
        assert all(k["regs"] == launch for k in mine), [(k["name"], k["regs"]) for k in mine]


def test_no_kernel_keeps_arrays_in_local_memory(kernels):
    """A loop that is not unrolled around a row's scores put them there: 3.5 times slower, and no spill told of it."""
    for name in ("window_", "cross_few_kernel", "cross_grad_prepare_kernel"):
        assert of(kernels, name)
        assert all(k["stack"] == 0 for k in of(kernels, name)), [(k["name"], k["stack"]) for k in of(kernels, name)]
