"""What the entry points take for tensors that lie on each other, against the bytes themselves (host code, built with g++)."""

import itertools
import os
import random
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <stdio.h>
#include "%s"
using namespace mxg::host;
int main() {
  long long at, rows, bytes, step, at2, rows2, bytes2, step2;
  while (scanf("%%lld %%lld %%lld %%lld %%lld %%lld %%lld %%lld", &at, &rows, &bytes, &step, &at2, &rows2, &bytes2, &step2) == 8) {
    const RowsAt a{(const void*)at, rows, bytes, step}, b{(const void*)at2, rows2, bytes2, step2};
    printf("%%d %%d %%d\n", overlap(a, b), overlap(b, a), same(a, b));
  }
}
"""


def touched(at, rows, bytes_, step):
    return {at + i * step + j for i in range(rows) for j in range(bytes_)}


def ask(tmp_path, cases):
    source, program = tmp_path / "ask.cpp", str(tmp_path / "ask")
    source.write_text(SOURCE % os.path.join(ROOT, "block_scaled_precision_e4m3_amd", "csrc", "overlap.hpp"))
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", program, str(source)], check=True)
    text = "".join(" ".join(map(str, a + b)) + "\n" for a, b in cases)
    out = subprocess.run([program], input=text, check=True, capture_output=True, text=True, timeout=60).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_small_tensors(tmp_path):
    rng = random.Random(0)

    def tensor():
        rows, bytes_ = rng.randint(0, 5), rng.randint(0, 6)
        return (1000 + rng.randint(0, 40), rows, bytes_, bytes_ + rng.choice((0, 0, 1, 2, 7)))
    cases = [(tensor(), tensor()) for _ in range(20000)]
    cases += [((1000, r, n, 8), (1000 + d, s, m, 8)) for r, s in itertools.product((1, 2, 3), repeat=2)
              for n, m in ((4, 4), (8, 8), (3, 6)) for d in range(-30, 31)]
    got = ask(tmp_path, cases)
    assert len(got) == len(cases)
    seen = set()
    for (a, b), (ab, ba, same) in zip(cases, got):
        want = bool(touched(*a) & touched(*b))
        assert ab == ba == want, (a, b, want)
        assert same == (a[0] == b[0] and (a[1] <= 1 or a[3] == b[3]))
        seen.add((want, a[3] == b[3]))
    assert len(seen) == 4


def test_large_tensors(tmp_path):
    """Sizes past 32 bits, and the two halves of one matrix's columns over many rows."""
    m, n, base = 1 << 24, 1 << 13, 1 << 40
    halves = ((base, m, n, 2 * n), (base + n, m, n, 2 * n))
    near = ((base, m, n, 2 * n), (base + n - 1, m, n, 2 * n))
    behind = ((base, m, n, n), (base + m * n, m, n, n))
    last = ((base, m, n, n), (base + m * n - 1, 1, n, n))
    # even rows of 8 bytes in 16, and rows of 4 in the gaps of every second one
    gaps = ((base, 1 << 16, 8, 16), (base + 8, 1 << 15, 4, 32))
    meets = ((base, 1 << 16, 8, 16), (base + 8, 1 << 15, 4, 33))
    assert [g[:2] for g in ask(tmp_path, [halves, near, behind, last, gaps, meets])] == [(0, 0), (1, 1), (0, 0), (1, 1), (0, 0), (1, 1)]
