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


# Experts' calls that take the few-row kernels, and how many slices a work-group has in either product:
# (tokens, hidden, inter, experts, top_k). 8 waves share the stages of 128: more than 3 stages a wave use a place
# of its ring again; 7, 9 and 11 stages leave waves without one or with one more than others.
FEW_EXPERTS = {
    (1, 7168, 2048, 8, 8): "few 1 4", (2, 7168, 1152, 8, 8): "few 1 8", (4, 2048, 1024, 8, 4): "few 2 2",
    (5, 1408, 896, 8, 3): "few 1 1", (4, 4096, 256, 8, 4): "few 1 4", (3, 7168, 128, 8, 5): "few 1 4",
    (2, 1024, 4096, 16, 16): "few 8 2", (16, 2176, 1152, 24, 3): "few 8 4", (8, 2048, 4096, 16, 4): "few 8 4",
    (1, 15104, 128, 1, 1): "few 1 1", (4, 128, 15104, 4, 2): "few 8 1", (4, 1152, 1024, 16, 4): "few 4 2",
    (32, 2048, 512, 64, 4): "few 8 8",
}

# Experts of these many pairs each (in buckets of 256 rows: blocks that are full, of at most 128 and of at most 64
# pairs), 64 blocks, and sizes (hidden, inter) at which the second product takes so many column tiles of
# 256 a work-group in turn: the last tile half or whole, the last group short, stages of 128 odd and even
PAIRS = [1, 64, 65, 128, 129, 256, 257, 300, 0, 40, 90, 200] * 4 + [1, 64, 65, 128, 129, 256, 257, 300, 0, 40, 90]
SPANS = {(1152, 128): 2, (1152, 256): 2, (1408, 384): 2, (2048, 640): 2, (896, 384): 1,
         (3200, 128): 4, (3456, 384): 4, (3712, 256): 4, (3968, 640): 4}
