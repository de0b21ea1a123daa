"""Which kernel of the 8-bit product a size selects (csrc/f8_gemm_choice.h, compiled for the host
with g++), and that the GPU tests' sizes reach every kernel, both output types, ragged edges and
every split.  CPU only."""
import os
import shutil
import subprocess

import pytest

from tests import f8_sizes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "flow_matching_mmdit_b200", "csrc")
SMS = 148
FEW, MID64, MID128, PAIR128, PAIR256 = range(5)

PROGRAM = r"""
#include <stdio.h>
#include "f8_gemm_choice.h"
int main() {
  long long m, n, k, sms;
  while (scanf("%lld %lld %lld %lld", &m, &n, &k, &sms) == 4) {
    const lens::F8Choice c = lens::choose_gemm_f8(m, n, k, (int)sms);
    printf("%d %d\n", (int)c.kernel, c.detail);
  }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cc").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "choice.cc"), "-o", str(d / "choice")], check=True)

    def run(sizes, sms=SMS):
        text = "".join(f"{m} {n} {k} {sms}\n" for m, n, k in sizes)
        out = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


def test_each_named_size_reaches_its_kernel(choose):
    names = {"few 8": (FEW, 1), "few 16": (FEW, 2), "few 32": (FEW, 4)}
    got = dict(zip(f8_sizes.KERNELS, choose(f8_sizes.KERNELS.values())))
    for name, choice in names.items():
        assert got.pop(name) == choice, name
    kinds = {"mid 64": MID64, "mid 128": MID128, "pair 128": PAIR128, "pair 256": PAIR256}
    assert {name: kernel for name, (kernel, _) in got.items()} == kinds
    assert got["mid 64"][1] > 0 and got["mid 128"][1] > 0      # with their k blocks split


def test_the_sizes_cover_every_kernel_and_its_edges(choose):
    sizes = f8_sizes.SIZES
    of = dict(zip(sizes, choose(sizes)))
    by = {}
    for size, choice in of.items():
        by.setdefault(choice[0], []).append(size)
    # all rows of the last group of eight, one of them, and several k blocks a warp
    for groups in (1, 2, 4):
        rows = {m for (m, n, k), c in of.items() if c == (FEW, groups) and k > 128}
        assert 8 * groups in rows and any(m < 8 * groups for m in rows), groups
    assert any(m > 24 and m < 32 for m, _, _ in by[FEW]) and any(k > 16 * 128 for _, _, k in by[FEW])
    for kernel in (MID64, MID128):
        assert {0, 1, 2, 3} <= {c[1] for c in of.values() if c[0] == kernel}, kernel
    # the last column block partial: in the first and in the second half of a tile, and not at all there
    assert {n % 256 for _, n, _ in by[PAIR256]} >= {0, 16, 144}
    assert {n % 128 for _, n, _ in by[PAIR128]} >= {0, 16}
    for kernel in (MID64, MID128, PAIR128, PAIR256):
        assert any(k % 128 for _, _, k in by[kernel]) and any(m % 128 for m, _, _ in by[kernel])


def test_choices_are_valid_over_the_whole_range(choose):
    import random
    rng = random.Random(0)
    sizes = [(rng.randint(1, 2 ** rng.randint(1, 22)), 16 * rng.randint(1, 2 ** rng.randint(0, 18)),
              16 * rng.randint(1, 2 ** rng.randint(0, 18))) for _ in range(3000)]
    for sms in (148, 132, 2):
        for (m, n, k), (kernel, detail) in zip(sizes, choose(sizes, sms)):
            if kernel == FEW:
                assert m <= 8 * detail and detail in (1, 2, 4) and n // 16 < 2 ** 31
            elif kernel in (MID64, MID128):
                assert 0 <= detail <= 3 and -(-k // 128) >= 1 << detail       # a k block for every CTA
                assert -(-m // (64 if kernel == MID64 else 128)) <= 65535     # rows of tiles: the grid's y
                assert (kernel == MID64) == (m <= 64)
            else:
                assert detail == 0 and m > 64
