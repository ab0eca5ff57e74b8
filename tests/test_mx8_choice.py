"""Which kernel the 8-bit products run for the cases of their GPU tests: the
library's rule (csrc/mx8_choice.hpp, host code) compiled and asked.  No GPU
needed."""
import os
import shutil
import subprocess

import pytest

from _mx8_cases import CASES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "padding_free_expert_amd", "csrc")
MAIN = r"""
#include <cstdio>
#include "mx8_choice.hpp"
int main() {
    long long rows;
    int E, N, NB;
    while (std::scanf("%lld %d %d %d", &rows, &E, &N, &NB) == 4) {
        const xmoe::Mx8Choice c = xmoe::mx8_choose(rows, E, N, NB);
        std::puts(c.stream == 1 ? "16" : c.stream == 2 ? "32" : c.once ? "tile nt" : "tile");
    }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("choice")
    (at / "main.cpp").write_text(MAIN)
    exe = str(at / "choose")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "main.cpp"), "-o", exe], check=True)

    def ask(calls):
        text = "\n".join(" ".join(map(str, c)) for c in calls)
        return subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
    return ask


def _rows(c):
    return sum(c["counts"]) + c["spare"]


def test_each_case_runs_the_kernel_it_is_for(choose):
    for name, c in CASES.items():
        E = len(c["counts"])
        got = choose([(_rows(c), E, c["h"], 2), (_rows(c), E, c["d"], 1)])
        assert got == [c["up"], c["down"]], name


def test_the_cases_reach_every_kernel_and_form():
    forms = {(which, c[which], c["T"] is not None) for c in CASES.values() for which in ("up", "down")}
    for kernel in ("16", "32", "tile", "tile nt"):
        for gathered in (False, True):
            # the down-projection's rows are never gathered
            assert ("up", kernel, gathered) in forms or kernel in ("16", "32"), (kernel, gathered)
        assert any(w == "up" and k == kernel for w, k, _ in forms) and any(w == "down" and k == kernel for w, k, _ in forms)
    tiles = [c for c in CASES.values() if c["up"].startswith("tile")]
    assert any(c["d"] <= 128 for c in tiles) and any(c["h"] <= 128 for c in tiles)     # one 128-deep step
    assert any(c["d"] % 128 for c in tiles) and any(c["h"] % 128 for c in tiles)       # a last step in part
    assert any(len(c["counts"]) == 1024 for c in tiles) and any(0 in c["counts"] for c in tiles)
    assert any(c["spare"] for c in tiles)
    # rounds of 256 tiles: a last one of at most half the compute units is split
    for width, which, N in ((128, "up", "h"), (256, "down", "d")):
        rest = set()
        for c in CASES.values():
            if c[which].startswith("tile"):
                n = sum(-(-r // 256) for r in c["counts"]) * -(-c[N] // width)
                rest.add((min(n // 256, 2), 2 * (n % 256) <= 256))
        assert {(0, False), (0, True), (1, False), (1, True)} <= rest, (which, rest)
        assert any(r >= 2 for r, _ in rest), which


def test_borders(choose):
    E, N = 64, 1408
    calls = [(0, E, N, 2), (1, E, N, 2), (12 * E, E, N, 2), (12 * E + 1, E, N, 2), (26 * E, E, N, 2), (26 * E + 1, E, N, 2),
             (128 * E, E, N, 2), (128 * E + 1, E, N, 2), (27, 1, N, 2), (2000, 1, N, 2), ((1 << 25) - 1, 1024, 32, 1)]
    assert choose(calls) == ["16", "16", "16", "32", "32", "tile nt", "tile nt", "tile", "32", "tile", "tile"]


def test_the_long_prompt_of_the_serving_block(choose):
    """1500 tokens, top-3 of 8 experts of 224 and one shared of 544, d = 1088."""
    calls = [(4500, 8, 224, 2), (4500, 8, 1088, 1), (1500, 1, 544, 2), (1500, 1, 1088, 1)]
    assert choose(calls) == ["tile"] * 4
