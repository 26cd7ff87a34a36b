"""The host code of the FP8 products for a few rows, by the library's own rules for sizes (no GPU)."""
import os
import shutil

import pytest

from .fp8_rows_host import FEW_EXPERTS, PAIRS, SPANS, ask, build_check
from .test_sanitizers import ROCM_INC

pytestmark = pytest.mark.skipif(not shutil.which("g++") or not os.path.isdir(ROCM_INC),
                                reason="host compiler or HIP headers not found")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return build_check(tmp_path_factory.mktemp("fp8_rows"))


def longest(exe, source, M):
    """The longest K that the few-row kernels take with M rows of 8 columns."""
    ks = range(16, (1 << 20) + 1, 16)
    fits = ask(exe, [f"f {source} {M} 8 {k}" for k in ks])
    last = max((k for k, f in zip(ks, fits) if f == "1"), default=0)
    assert all((f == "1") == (k <= last) for k, f in zip(ks, fits))
    return last


# 64 KB hold M quantised rows of K rounded up to 256 and 16 bytes more, 4 (M + 2) bytes of scales for each 128
# of K, and 512 M bytes of sums; of codes the scales alone
LONGEST = {(1, 1): 59392, (1, 4): 15104, (0, 1): 699008, (0, 4): 349440, (0, 5): 299520, (0, 16): 116480}


@pytest.mark.parametrize("source,M", list(LONGEST))
def test_longest_rows(exe, source, M):
    assert longest(exe, source, M) == LONGEST[source, M]
    assert longest(exe, source, 17 if source == 0 else 5) == 0


def test_products_on_both_sides_of_the_limits(exe):
    """Arrays and workspaces of every path, at the longest K of each and one step more."""
    lines = [f"m {M} {N} {K} {q} {block} {kind}"
             for M in (1, 2, 4, 5, 16, 17) for N in (8, 264, 4096)
             for top in (*LONGEST.values(), 14000, (1 << 20) - 16) for K in (top, top + 16)
             for q in (0, 1) for block in (1, 128) for kind in (0, 2)]
    answers = dict(zip(lines, ask(exe, lines)))
    for (source, M), K in LONGEST.items():
        if source == 1:  # (codes that long are faster in tiles)
            assert any(answers[f"m {M} {N} {K} 1 128 0"] == "f" for N in (8, 264, 4096)), M
            assert not any(answers[f"m {M} {N} {K + 16} 1 128 {kind}"] == "f" for N in (8, 264, 4096) for kind in (0, 2))
    for line, a in answers.items():
        q, block = line.split()[4:6]
        assert a in (("t", "r") if q == "0" else ("qt", "qr", "f")) and (block == "128" or a in ("t", "qt")), line


def test_a_bf16_operand_and_its_codes_take_the_same_kernel(exe):
    """... few rows or tiles, whose sums differ in their order and, for bf16 results, their accuracy."""
    sizes = [(M, N, K, kind) for M in (1, 2, 3, 4, 5, 8, 16, 17, 64) for kind in (0, 2)
             for N in (8, 256, 1024, 2048, 4096, 7168, 8192, 28672)
             for K in (128, 1024, 2048, 4096, 7168, 8192, 14336, 15104, 15120, 59392)]
    bf16 = ask(exe, [f"m {M} {N} {K} 1 128 {kind}" for M, N, K, kind in sizes])
    codes = ask(exe, [f"m {M} {N} {K} 0 128 {kind}" for M, N, K, kind in sizes])
    differ = [s for s, x, q in zip(sizes, bf16, codes) if q != {"f": "r", "qr": "r", "qt": "t"}[x]]
    assert not differ, (len(differ), len(sizes), differ[:10])
    assert {"f", "qr", "qt"} == set(bf16)


def test_named_experts_take_the_few_row_kernels(exe):
    """... with the slices that they are named for, so that a change of the rules cannot empty the GPU tests."""
    found = ask(exe, ["e %d %d %d %d %d" % size for size in FEW_EXPERTS])
    assert dict(zip(FEW_EXPERTS, found)) == FEW_EXPERTS
    assert {int(s) for a in found for s in a.split()[1:]} == {1, 2, 4, 8}
    # at most two pairs an expert on average, hidden and inter up to 15104
    few = ["e 4 256 128 2 1", "e 12 256 128 48 8", "e 1 15104 128 1 1", "e 1 128 15104 1 1", "e 1 15104 15104 1 1"]
    tiles = ["e 5 256 128 2 1", "e 13 256 128 48 8", "e 1 15232 128 1 1", "e 1 128 15232 1 1"]
    assert all(a.startswith("few") for a in ask(exe, few)) and ask(exe, tiles) == ["tiles"] * len(tiles)


def test_named_sizes_take_their_column_tiles_in_turn(exe):
    blocks = sum(-(-n // 256) for n in PAIRS)
    found = ask(exe, [f"s {blocks} {-(-hidden // 256)}" for hidden, _ in SPANS])
    assert dict(zip(SPANS, map(int, found))) == SPANS
    for hidden, inter in SPANS:  # tiles, not the few-row kernels
        assert ask(exe, [f"e {sum(PAIRS) // 2} {hidden} {inter} {len(PAIRS)} 2"]) == ["tiles"]
    # never a round of work-groups more than 1/32 over one tile each
    sizes = [(tm, tn) for tm in range(1, 200, 3) for tn in range(1, 40)]
    for (tm, tn), a in zip(sizes, ask(exe, [f"s {tm} {tn}" for tm, tn in sizes])):
        rounds = lambda span: -(-tm * -(-tn // span) // 256) * span  # noqa: E731
        best = max(s for s in (1, 2, 4) if rounds(s) * 32 <= rounds(1) * 33)
        assert int(a) == best
