"""The cuts that tests/ffn_cuts.py names are those of the plans (csrc/ffn_plan.cpp, built for the host
with tests/sanitize/ffn_plans.cpp)."""
import os
import shutil
import subprocess

import pytest

from . import ffn_cuts
from .test_sanitizers import CSRC, FLAGS, ROCM_INC, SAN, build

pytestmark = pytest.mark.skipif(not shutil.which("g++") or not os.path.isdir(ROCM_INC),
                                reason="host compiler or HIP headers not found")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plans") / "ffn_plans")
    build(["g++", "-std=c++17", "-I", ROCM_INC, "-I", CSRC, "-D__HIP_PLATFORM_AMD__", *FLAGS,
           os.path.join(CSRC, "ffn_plan.cpp"), os.path.join(SAN, "ffn_plans.cpp"), "-o", exe])

    def ask(kind, sizes):
        lines = "".join("%s %d %d %d\n" % (kind, *s) for s in sizes)
        res = subprocess.run([exe], input=lines, capture_output=True, text=True, timeout=120)
        assert res.returncode == 0, res.stderr[-2000:]
        found = []
        for line in res.stdout.splitlines():
            cuts = {}
            for item in line.split(";")[:-1]:
                name, first, tile, shares = item.split()
                cuts[name] = ("+" if first != "0" else "") + tile + ("s" if shares != "1" else "")
            found.append(cuts)
        return dict(zip(sizes, found, strict=True))

    return ask


def test_named_cuts(plans):
    for kind, table in (("ffn", ffn_cuts.FFN), ("mxffn", ffn_cuts.MX_FFN),
                        ("mxffn", ffn_cuts.MX_VALUES)):
        for sizes, cuts in plans(kind, list(table)).items():
            assert {n: cuts.get(n) for n in table[sizes]} == table[sizes], (kind, sizes, cuts)
    for sizes, cuts in plans("mx", list(ffn_cuts.MX)).items():
        assert cuts["product"] == ffn_cuts.MX[sizes], (sizes, cuts)


def test_every_second_launch_is_there():
    """Each product with a second launch of every tile, in shares and without where plans have them."""
    seen = {(n, c) for cuts in ffn_cuts.FFN.values() for n, c in cuts.items()}
    for name in ("up", "down", "dh", "dx", "dw13", "dw2"):
        assert {c for n, c in seen if n == name} >= {"+0", "+1", "+3"}, name
    for name in ("up", "dh", "dx", "dw13"):
        assert {c for n, c in seen if n == name} >= {"+0s", "+3s"}, name
    whole = {"0", "0s", "1", "2", "3", "3s"}
    assert set(ffn_cuts.MX.values()) >= whole | {"+0", "+3", "+3s"}
    for name in ("up", "down"):
        cuts = {c[name] for c in ffn_cuts.MX_FFN.values() if name in c}
        assert cuts >= whole | {"+0", "+3"}, name
