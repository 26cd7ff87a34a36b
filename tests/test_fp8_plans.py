"""The cuts that tests/fp8_cuts.py names are those of the plan (csrc/fp8_plan.cpp, built for the host with
tests/sanitize/fp8_plans.cpp), and the host code of include/moe_fp8.h and include/moe_balance.h under
AddressSanitizer and UndefinedBehaviorSanitizer, driven by tests/sanitize/fp8_check.cpp."""
import os
import shutil
import subprocess

import pytest

from .fp8_cuts import CUTS
from .test_sanitizers import CSRC, FLAGS, ROCM_INC, ROOT, SAN, build, run

pytestmark = pytest.mark.skipif(not shutil.which("g++") or not os.path.isdir(ROCM_INC),
                                reason="host compiler or HIP headers not found")


def test_named_cuts(tmp_path):
    exe = str(tmp_path / "fp8_plans")
    build(["g++", "-std=c++17", "-I", ROCM_INC, "-I", CSRC, "-D__HIP_PLATFORM_AMD__", *FLAGS,
           os.path.join(CSRC, "fp8_plan.cpp"), os.path.join(SAN, "fp8_plans.cpp"), "-o", exe])
    lines = "".join("%d %d %d %d %d\n" % sizes for sizes in CUTS)
    res = subprocess.run([exe], input=lines, capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr[-2000:]
    found = [("+" if f != "0" else "") + t + ("s" if s != "1" else "")
             for f, t, s in (line.split() for line in res.stdout.splitlines())]
    assert dict(zip(CUTS, found, strict=True)) == CUTS
    for wide in (0, 1):
        for rows in (0, 1):
            cuts = {c for (w, r, *_), c in CUTS.items() if (w, r) == (wide, rows)}
            two = {"+3", "+3s"} if rows and not wide else {"+0", "+0s", "+3", "+3s"}
            assert cuts == {"0", "0s", "1", "3", "3s"} | two | (
                set() if wide else {"2"} if rows else {"2", "+1"})


def test_host_code_under_sanitizers(tmp_path):
    inc = ["-std=c++17", "-I", ROCM_INC, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for src in (os.path.join(CSRC, "fp8_api.cpp"), os.path.join(CSRC, "fp8_plan.cpp"),
                os.path.join(CSRC, "balance_api.cpp"), os.path.join(SAN, "fp8_check.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        build(["g++", *inc, *FLAGS, "-c", src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "fp8_check")
    build(["g++", "-fsanitize=address,undefined", *objs, "-o", exe])
    rc, out = run(exe)
    assert rc == 0, out[-4000:]
    assert "failed: 0" in out and "runtime error" not in out and "Sanitizer" not in out, out[-4000:]
