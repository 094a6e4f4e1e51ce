"""The kernel for few query rows in a language model's own attention: how many of its blocks an SM holds, from the
assembler's own report on the CPU, and that the library's plan begins no second round of blocks that would be a small one."""
import math
import os
import random
import subprocess

import pytest

import vision_encoder_varlen_gb300 as vit
from test_ptxas_resources import _ENTRY, _demangle
from test_window_plans import plans
from vision_encoder_varlen_gb300 import _build

SMS, HEAD_DIMS = 152, (32, 64, 80, 96, 128)


def by_smem(D):
    return 227 * 1024 // (3 * 256 * D + 2048)


def by_registers(regs, row_tiles):
    """Warps are dealt to the four quarters of the register file, in units of 8 registers a thread."""
    return 4 * (16384 // (32 * math.ceil(regs / 8) * 8)) // (4 * row_tiles + 1)


def places(D, row_tiles):
    """What the plan counts on."""
    return by_smem(D) if row_tiles == 1 or D < 64 else 2 if D <= 80 else 1


def test_places_that_registers_leave(tmp_path):
    r = subprocess.run([_build._nvcc(), *_build.compile_flags(ptxas_info=True), "-c",
                        os.path.join(_build.CSRC, "cross_few.cu"), "-o", str(tmp_path / "o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    report = _ENTRY.findall(r.stderr)
    found = 0
    for name, (_, _, _, _, regs) in zip(_demangle([x[0] for x in report]), report):
        name = name.replace("(int)", "").replace("(bool)1", "true")
        for D in HEAD_DIMS[1:]:
            for t in (1, 2):
                if f"cross_few_kernel<{D}, {t}, true>" in name:
                    assert min(by_smem(D), by_registers(int(regs), t)) == places(D, t), (name, regs)
                    found += 1
    assert found == 2 * len(HEAD_DIMS[1:])


def test_no_small_second_round(plans):
    rng = random.Random(8)
    lines = []
    for _ in range(4000):
        B, Hk, D = rng.choice([1, 2, 3, 5, 7, 11, 13, 20, 30]), rng.choice([1, 2, 4, 8, 16]), rng.choice(HEAD_DIMS)
        group = rng.choice([1, 2, 4, 8])
        lines.append(("few", B, Hk * group, Hk, D, rng.choice([1, 2, 3, 4, 8, 32]), rng.randint(64, 9000), 0, 0))
    two = 0
    for (_, B, Hq, Hk, D, mq, mk, _, _), p in zip(lines, plans(lines)):
        if not p["takes"]:
            continue
        blocks, fit = B * Hk * p["n_split"], SMS * places(D, p["row_tiles"])
        assert not (fit < blocks < 1.5 * fit and B * Hk <= fit), (B, Hq, Hk, D, mq, mk, p)
        assert p["n_split"] <= p["room"] and p["partial_bytes"] in (0, 4 * B * Hk * p["room"] * p["rows"] * (D + 1))
        assert p["partial_bytes"] > 0 or p["n_split"] == 1
        two += p["row_tiles"] == 2 and D >= 64 and p["n_split"] < p["room"]
    assert two > 5


@pytest.mark.gpu
@pytest.mark.parametrize("B,mk,D,P", [(7, 1100, 128, 0), (13, 1200, 64, 0), (9, 1000, 96, 0), (12, 680, 128, 9000), (20, 800, 64, 9000)])
def test_fewer_runs_than_the_workspace_holds(B, mk, D, P):
    """Two row tiles whose runs are fewer than shared memory alone would allow, alone and beside a prefix read apart."""
    from test_gpu_window_attn import check, make, offsets, reference
    q, k, v, cq, ck, _ = make([8] * B, [mk - b for b in range(B)], 32, 8, D)
    status = vit.new_status()
    if P == 0:
        for window, sinks in ((None, 0), (mk - 70, 9)):
            out, lse = vit.window_attn(q, k, v, cq, ck, 8, mk, window, sinks, return_lse=True, status=status)
            assert vit.read_status(status) == 0
            check(out, lse, reference(q, k, v, cq, ck, None, window or 0, sinks))
    else:
        kp, vp = (make([P], [1], 8, 8, D, seed=s)[0] for s in (1, 2))
        out, lse = vit.prefix_attn(q, kp, vp, k, v, cq, offsets([P]), ck, None, 8, P, mk, return_lse=True, status=status)
        assert vit.read_status(status) == 0
        check(out, lse, reference(q, k, v, cq, ck, prefix=[(kp, vp, 0, P)] * B))
