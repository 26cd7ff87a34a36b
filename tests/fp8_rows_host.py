"""The few-row rules of the FP8 products as the library applies them: tests/sanitize/fp8_rows_check.cpp built
with the host code, under AddressSanitizer and UndefinedBehaviorSanitizer."""
import os
import subprocess

from .test_sanitizers import CSRC, ENV, FLAGS, ROCM_INC, ROOT, SAN, build


def build_check(folder):
    """The program; ask(exe, lines) gives its answers, a line each."""
    exe = os.path.join(str(folder), "fp8_rows_check")
    build(["g++", "-std=c++17", "-I", ROCM_INC, "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-D__HIP_PLATFORM_AMD__", *FLAGS, *(os.path.join(CSRC, s) for s in (
               "fp8_api.cpp", "fp8_plan.cpp", "fp8_rows_plan.cpp")),
           os.path.join(SAN, "fp8_rows_check.cpp"), "-o", exe])
    return exe


def ask(exe, lines):
    res = subprocess.run([exe], input="".join(line + "\n" for line in lines), capture_output=True, text=True,
                         timeout=300, env=ENV)
    assert res.returncode == 0, res.stderr[-4000:]
    answers = res.stdout.splitlines()
    assert len(answers) == len(lines)
    return answers
