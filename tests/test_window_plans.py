"""How calls of a language model's own attention are cut, from the library's own plans (functions of the sizes alone), on
the CPU."""
import os
import random
import subprocess

import pytest

from vision_encoder_varlen_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="session")
def plans(tmp_path_factory):
    """A function of lines that name calls: the plan of each, as a dict of whole numbers."""
    _build.build()
    prog = str(tmp_path_factory.mktemp("plans") / "window_plans")
    r = subprocess.run([_build._nvcc(), "-std=c++17", *_build.ARCH, "-I", _build.INCLUDE, "-I", _build.CSRC,
                        os.path.join(HERE, "window_plans.cu"), "-o", prog, "-L", _build.LIBDIR, "-lvitattn",
                        "-Xlinker", "-rpath", "-Xlinker", _build.LIBDIR], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(lines):
        r = subprocess.run([prog], input="\n".join(" ".join(map(str, x)) for x in lines), capture_output=True, text=True)
        out = [dict((n, int(v)) for n, v in (f.split("=") for f in line.split())) for line in r.stdout.splitlines()]
        assert r.returncode == 0 and len(out) == len(lines), r.stderr
        return out

    return ask


def test_runs_have_keys(plans):
    """A run is a whole number of 64-key tiles and at least one, also where no sequence has a key of its own; the runs of
    the longest sequence cover it, and none of them is empty."""
    rng = random.Random(3)
    lines, keys = [], []
    for _ in range(3000):
        B, Hk, D = rng.choice([1, 3, 19, 64, 400]), rng.choice([1, 2, 8, 16]), rng.choice([32, 64, 80, 96, 128])
        Hq, mq = Hk * rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3])
        mk = rng.choice([0, 1, 63, 64, 65, 700, 2048, 2049, 9000])
        G, mp = rng.choice([1, 2]), rng.choice([1, 1601, 9000])
        lines += [("win", B * mq, B, Hq, Hk, D, mq, mk, 0, 0, G, G * mp, mp), ("few", B, Hq, Hk, D, mq, mk, 0, 0),
                  ("prefix_few", B, Hq, Hk, D, mq, mk, mp)]
        keys += [mk, mk, -(-mp // 64) * 64 + mk]
    apart_without_keys = 0
    for line, n, p in zip(lines, keys, plans(lines)):
        if line[0] == "win" and not p["own_few"]:
            continue
        assert p["chunk"] >= 64 and p["chunk"] % 64 == 0, (line, p)
        assert p["n_split"] == max(1, -(-n // p["chunk"])), (line, p)
        apart_without_keys += line[0] == "win" and n == 0 and line[2] * line[4] >= 152
    assert apart_without_keys > 20
