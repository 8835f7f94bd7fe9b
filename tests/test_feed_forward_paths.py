"""The rule that chooses a block-128 product's kernel, as built for the host, for the sizes of tests/feed_forward_paths.py
and, with those of tests/test_gpu_feed_forward.py, for all kernels there are."""

import os
import re
import subprocess

import pytest

import feed_forward_paths as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

SOURCE = r"""
#include "%s"
#include <stdio.h>
using namespace mxg::b128;
int main() {
  char kind;
  long long a, b, c, d;
  int exact;
  while (scanf(" %%c %%lld %%lld %%lld %%lld %%d", &kind, &a, &b, &c, &d, &exact) == 6) {
    const Choice ch = kind == 'l' ? choose(a, b, c, 1, exact) : kind == 'g' ? choose_grouped(a, b, c, d, exact) : choose_deep(a, b, c, d);
    if (ch.rows) printf("rows %%dx%%d\n", kind == 'l' ? a <= 16 ? 16 : 32 : ch.bm, ch.rows);
    else printf("tile %%dx%%d%%s\n", ch.bm, ch.bn, ch.splits > 1 ? " divided" : "");
  }
}
"""


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    """Questions (kind, four sizes, whether C is float32) -> kernels."""
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(SOURCE % os.path.join(ROOT, "block_scaled_precision_e4m3_amd", "csrc", "block128_choose.hpp"))
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__=1", f"-I{ROCM}/include", "-o", str(d / "choice"), str(d / "choice.cpp"),
                    f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib"], check=True, capture_output=True)

    def ask(questions):
        text = "".join(" ".join(map(str, q)) + "\n" for q in questions)
        out = subprocess.run([str(d / "choice")], input=text, check=True, capture_output=True, text=True, timeout=60).stdout.splitlines()
        assert len(out) == len(questions)
        return out
    return ask


def linear(size, exact):
    return ("l", *size, 0, exact)


def grouped(case, exact):
    sizes, n, k, head, tail = case
    return ("g", sum(sizes) + head + tail, len(sizes), n, k, exact)


def deep(case):
    sizes, m, n, head, tail = case
    return ("d", P.blocks(sizes, head, tail), len(sizes), m, n, 1)


def test_sizes_reach_their_kernels(choice):
    for exact in (0, 1):
        for ask, cases in ((linear, P.LINEAR), (grouped, P.GROUPED)):
            assert choice([ask(c[0], exact) for c in cases]) == [c[1 + exact] for c in cases]
    assert choice([deep(c) for c, _ in P.DEEP]) == [to for _, to in P.DEEP]


def parameters(test, which=-1):
    marks = [m for m in test.pytestmark if m.name == "parametrize"]
    return marks[which].args[1]


def test_sizes_of_the_tests_reach_every_kernel(choice):
    import test_gpu_feed_forward as T
    tiles16 = {"tile 64x64", "tile 64x128", "tile 128x128", "tile 128x256", "tile 256x256"}
    rows = {"rows 16x16", "rows 16x32", "rows 32x16", "rows 32x32"}
    tiles32, divided = tiles16 - {"tile 256x256"}, {"tile 64x64 divided", "tile 64x128 divided"}
    for exact, tiles, parts in ((0, tiles16, divided), (1, tiles32, divided | {"tile 128x128 divided"})):
        assert set(choice([linear(s, exact) for s in T.SIZES + [c[0] for c in P.LINEAR]])) == tiles | rows | parts
        assert set(choice([grouped(c, exact) for c in T.GROUPS + [c[0] for c in P.GROUPED]])) == tiles | rows
    cases = [tuple(c) for c in parameters(T.test_weight_gradient_sizes)] + [c for c, _ in P.DEEP]
    assert set(choice([deep(c) for c in cases])) == tiles32 | divided | {"tile 128x128 divided"}


def test_no_other_kernel_is_chosen(choice):
    """Over a wide range of sizes nothing but what the last test names comes up."""
    import random
    rng = random.Random(3)

    def log(a, b):
        return int(a * (b / a) ** rng.random())
    found = set()
    for exact in (0, 1):
        found |= {(k, "l", exact) for k in choice([("l", log(1, 5000), log(1, 9000), 16 * log(1, 500), 0, exact) for _ in range(5000)])}
        found |= {(k, "g", exact) for k in choice([("g", log(1, 20000), log(1, 1024), log(1, 9000), 16 * log(1, 500), exact) for _ in range(5000)])}
    found |= {(k, "d", 1) for k in choice([("d", log(1, 2000), log(1, 1024), log(1, 5000), log(1, 5000), 1) for _ in range(5000)])}
    for kernel, kind, exact in found:
        assert re.fullmatch(r"rows (16|32)x(16|32)|tile (64x64|64x128|128x128|128x256|256x256)( divided)?", kernel)
        assert not (exact and "256x256" in kernel) and not (kind == "g" and "divided" in kernel) and not (kind == "d" and "rows" in kernel)
        if "divided" in kernel:
            assert "x256" not in kernel and (exact or "128x128" not in kernel)
