"""The host code of the feed-forward and MXFP4 entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (host compilers only), driven by tests/sanitize/ffn_check.cpp: argument checks,
workspace layout, launch sequences and the plans of the products, with every launch replaced by a check of
the arrays that it is handed."""
import os
import shutil

import pytest

from .test_sanitizers import CSRC, FLAGS, ROCM_INC, ROOT, SAN, build, run

pytestmark = pytest.mark.skipif(not shutil.which("g++") or not os.path.isdir(ROCM_INC),
                                reason="host compiler or HIP headers not found")


def test_host_code_under_sanitizers(tmp_path):
    inc = ["-std=c++17", "-I", ROCM_INC, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-D__HIP_PLATFORM_AMD__"]
    objs = []
    for src in (os.path.join(CSRC, "ffn_api.cpp"), os.path.join(CSRC, "ffn_plan.cpp"),
                os.path.join(SAN, "ffn_check.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        build(["g++", *inc, *FLAGS, "-c", src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "ffn_check")
    build(["g++", "-fsanitize=address,undefined", *objs, "-o", exe])
    rc, out = run(exe)
    assert rc == 0, out[-4000:]
    assert "failed: 0" in out and "runtime error" not in out and "Sanitizer" not in out, out[-4000:]
